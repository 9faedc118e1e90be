// group_norm.cu -- group norm with an activation, channels last: x [N, S, C], G groups of D = C / G
// channels, statistics over the S positions and D channels of each (sample n, group g).
//
//   xh = (x - mean) rstd,  rstd = 1 / sqrt(var + eps),  z = xh w_c + b_c
//   y  = act(z), or z act(gate) where a gate is given
// and with dz = dy act'(z) (dy act(gate) and dgate = dy z act'(gate) with a gate), dn = dz w_c:
//   dx = rstd (dn - mean(dn) - xh mean(dn xh)),   dw_c = sum dz xh,   db_c = sum dz
//
// Bound by memory: x (and gate, dy) are read and y (dx, dgate) written.  Two forms:
//   rows    S = 1 (every token on its own, the norm of a scan's heads): the D channels of a group lie
//           side by side, a few lanes hold them in registers, one pass over the data.
//   tiles   any S: a first kernel reduces tiles of positions, a second one merges the tiles' results
//           and applies them (its reads of a tensor up to L2's size hit L2).  A thread keeps the same
//           channels (one vector) for all of its positions, so any D works at full vector width.
// Means and variances are merged pairwise from centred sums (count, mean, sum of squares about the
// mean): a mean far above the deviation costs no digits.

#include <algorithm>

#include "api.cuh"
#include "common.cuh"

namespace prism {
namespace {

struct NormArgs {
    int N, S, C, G, act;
    float eps;
    const void *x, *gate, *dy;
    const float *weight, *bias;
    float *mean, *rstd;      // outputs of the forward pass (may be null), inputs of the backward one
    void *y, *dx, *dgate;
    float *stat_parts;       // tiles form: [N][tiles][pieces][2]
    float *chan_parts;       // backward: [parts][2][C] sums of dz and dz xh
    int tiles, parts;
};

// ---- activations -------------------------------------------------------------------------------

__device__ __forceinline__ float act_value(int act, float z) {
    if (act == PRISM_ACT_SILU) return z / (1.f + expf(-z));
    if (act == PRISM_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    return z;
}

// act(z) and act'(z)
__device__ __forceinline__ float act_both(int act, float z, float &slope) {
    if (act == PRISM_ACT_SILU) {
        const float s = 1.f / (1.f + expf(-z));
        slope = s * fmaf(z, 1.f - s, 1.f);
        return z * s;
    }
    if (act == PRISM_ACT_GELU) {
        const float c = 0.5f * (1.f + erff(z * 0.70710678118654752f));
        slope = fmaf(z * 0.39894228040143268f, expf(-0.5f * z * z), c);
        return z * c;
    }
    slope = 1.f;
    return z;
}

// ---- vectors of V consecutive channels -----------------------------------------------------------

template <typename IO, int V>
struct alignas(sizeof(IO) * V) Pack {
    IO v[V];
};

template <typename IO, int V>
__device__ __forceinline__ void load_vec(const void *p, long long at, float (&f)[V]) {
    const Pack<IO, V> r = *reinterpret_cast<const Pack<IO, V> *>((const IO *)p + at);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = ld_io(r.v, i);
}
template <typename IO, int V>
__device__ __forceinline__ void store_vec(void *p, long long at, const float (&f)[V]) {
    Pack<IO, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) st_io(r.v, i, f[i]);
    *reinterpret_cast<Pack<IO, V> *>((IO *)p + at) = r;
}

// dz of one element (before the weight), and its dgate
__device__ __forceinline__ float dz_of(const NormArgs &p, float z, float dy, float gate, float &dgate) {
    float slope;
    if (p.gate) {
        const float a = act_both(p.act, gate, slope);
        dgate = dy * z * slope;
        return dy * a;
    }
    act_both(p.act, z, slope);
    return dy * slope;
}

// ---- rows form -----------------------------------------------------------------------------------

constexpr int kRowThreads = 256;
constexpr int kRowVecs = 4;  // vectors of a lane at most

// Sum over the LG lanes of a group (LG a power of two, groups aligned to it).
__device__ __forceinline__ float lanes_sum(float x, int LG) {
    for (int o = LG >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// LG lanes hold one (row, group) at a time: lane l the vectors l, l + LG, ... of its D / V.  A lane
// group keeps its group g over all of its rows, so the weights are read once.
template <typename IO, int V, int K>
__global__ void __launch_bounds__(kRowThreads) norm_rows_fwd_kernel(NormArgs p, int LG, int row_lanes) {
    const int D = p.C / p.G, nv = D / V;
    const int lane = threadIdx.x & (LG - 1);
    const long long unit = ((long long)blockIdx.x * kRowThreads + threadIdx.x) / LG;
    const int g = (int)(unit % p.G);
    const long long first = unit / p.G;
    float w[K][V], b[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = lane + k * LG, c = g * D + v * V + i;
            w[k][i] = p.weight && v < nv ? p.weight[c] : 1.f;
            b[k][i] = p.bias && v < nv ? p.bias[c] : 0.f;
        }
    const float inv = 1.f / (float)D;
    // the lane groups of one warp take the same number of steps, so that every shuffle has all lanes
    for (long long r0 = 0; r0 < p.N; r0 += row_lanes) {
        const long long row = r0 + first;
        const bool live = first < row_lanes && row < p.N;
        const long long base = row * p.C + (long long)g * D;
        float x[K][V], gt[K][V];
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = lane + k * LG;
            if (live && v < nv) {
                load_vec<IO, V>(p.x, base + v * V, x[k]);
                if (p.gate) load_vec<IO, V>(p.gate, base + v * V, gt[k]);
#pragma unroll
                for (int i = 0; i < V; ++i) s += x[k][i];
            }
        }
        const float mean = lanes_sum(s, LG) * inv;
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (live && lane + k * LG < nv)
#pragma unroll
                for (int i = 0; i < V; ++i) q = fmaf(x[k][i] - mean, x[k][i] - mean, q);
        const float rstd = 1.f / sqrtf(fmaf(lanes_sum(q, LG), inv, p.eps));
        if (!live) continue;
        if (lane == 0) {
            if (p.mean) p.mean[row * p.G + g] = mean;
            if (p.rstd) p.rstd[row * p.G + g] = rstd;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = lane + k * LG;
            if (v >= nv) continue;
            float y[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float z = fmaf((x[k][i] - mean) * rstd, w[k][i], b[k][i]);
                y[i] = p.gate ? z * act_value(p.act, gt[k][i]) : act_value(p.act, z);
            }
            store_vec<IO, V>(p.y, base + v * V, y);
        }
    }
}

// The same lanes for the backward pass; a lane also sums dz and dz xh of its channels over its rows.
template <typename IO, int V, int K>
__global__ void __launch_bounds__(kRowThreads) norm_rows_bwd_kernel(NormArgs p, int LG, int row_lanes) {
    const int D = p.C / p.G, nv = D / V;
    const int lane = threadIdx.x & (LG - 1);
    const long long unit = ((long long)blockIdx.x * kRowThreads + threadIdx.x) / LG;
    const int g = (int)(unit % p.G);
    const long long first = unit / p.G;
    float w[K][V], b[K][V], sz[K][V], szx[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = lane + k * LG, c = g * D + v * V + i;
            w[k][i] = p.weight && v < nv ? p.weight[c] : 1.f;
            b[k][i] = p.bias && v < nv ? p.bias[c] : 0.f;
            sz[k][i] = szx[k][i] = 0.f;
        }
    const float inv = 1.f / (float)D;
    for (long long r0 = 0; r0 < p.N; r0 += row_lanes) {
        const long long row = r0 + first;
        const bool live = first < row_lanes && row < p.N;
        const long long base = row * p.C + (long long)g * D;
        const float mean = live ? p.mean[row * p.G + g] : 0.f, rstd = live ? p.rstd[row * p.G + g] : 0.f;
        float xh[K][V], dn[K][V];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = lane + k * LG;
            if (!live || v >= nv) continue;
            float x[V], dy[V], gt[V] = {}, dg[V];
            load_vec<IO, V>(p.x, base + v * V, x);
            load_vec<IO, V>(p.dy, base + v * V, dy);
            if (p.gate) load_vec<IO, V>(p.gate, base + v * V, gt);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                xh[k][i] = (x[i] - mean) * rstd;
                const float dz = dz_of(p, fmaf(xh[k][i], w[k][i], b[k][i]), dy[i], gt[i], dg[i]);
                sz[k][i] += dz;
                szx[k][i] = fmaf(dz, xh[k][i], szx[k][i]);
                dn[k][i] = dz * w[k][i];
                s1 += dn[k][i];
                s2 = fmaf(dn[k][i], xh[k][i], s2);
            }
            if (p.gate) store_vec<IO, V>(p.dgate, base + v * V, dg);
        }
        s1 = lanes_sum(s1, LG) * inv;
        s2 = lanes_sum(s2, LG) * inv;
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = lane + k * LG;
            if (v >= nv) continue;
            float dx[V];
#pragma unroll
            for (int i = 0; i < V; ++i) dx[i] = rstd * (dn[k][i] - s1 - xh[k][i] * s2);
            store_vec<IO, V>(p.dx, base + v * V, dx);
        }
    }
    if (!p.chan_parts || first >= row_lanes) return;
    float *out = p.chan_parts + first * 2 * p.C + g * D;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = lane + k * LG;
        if (v >= nv) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            out[v * V + i] = sz[k][i];
            out[p.C + v * V + i] = szx[k][i];
        }
    }
}

// dbias, dweight: the parts' sums, a column per thread of x and 8 interleaved ranges of parts.
__global__ void __launch_bounds__(256) norm_channel_sum_kernel(const float *parts, int n, int C, float *dweight, float *dbias) {
    __shared__ float s[8][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;  // col over [dz | dz xh]
    float acc = 0.f;
    if (col < 2 * C)
        for (int i = k; i < n; i += 8) acc += parts[(long long)i * 2 * C + col];
    s[k][threadIdx.x & 31] = acc;
    __syncthreads();
    if (k == 0 && col < 2 * C) {
        for (int i = 1; i < 8; ++i) acc += s[i][threadIdx.x];
        if (col < C) {
            if (dbias) dbias[col] = acc;
        } else if (dweight) {
            dweight[col - C] = acc;
        }
    }
}

// ---- tiles form ----------------------------------------------------------------------------------

constexpr int kTileThreads = 512;
constexpr int kTileCols = 256;  // vector columns of a block

struct Stat {
    float n, mean, m2;
};
__device__ __forceinline__ Stat merge(const Stat &a, const Stat &b) {
    const float n = a.n + b.n;
    if (n == 0.f) return a;
    const float f = b.n / n, d = b.mean - a.mean;
    return Stat{n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * a.n * f};
}
__device__ __forceinline__ Stat shfl(const Stat &a, int o) {
    return Stat{__shfl_xor_sync(0xffffffffu, a.n, o), __shfl_xor_sync(0xffffffffu, a.mean, o), __shfl_xor_sync(0xffffffffu, a.m2, o)};
}

// Geometry of a block: channels [c0, c1) (whole vectors), positions [s0, s1) of sample n; thread
// (col, rl) owns V channels and every RL-th position.
template <int V>
struct Tile {
    int n, tile, cb, c0, c1, cols, RL, col, rl, s0, s1;
    bool live;
    __device__ explicit Tile(const NormArgs &p) {
        n = blockIdx.x / p.tiles;
        tile = blockIdx.x % p.tiles;
        cb = blockIdx.y;
        c0 = cb * kTileCols * V;
        c1 = min(c0 + kTileCols * V, p.C);
        cols = (c1 - c0) / V;
        RL = kTileThreads / cols;
        col = threadIdx.x % cols;
        rl = threadIdx.x / cols;
        live = rl < RL;
        s0 = (int)((long long)p.S * tile / p.tiles);
        s1 = (int)((long long)p.S * (tile + 1) / p.tiles);
    }
    // A group cut by a block's edge leaves one piece in each block: piece g + cb is group g's in block cb.
    __device__ int first_group(int D) const { return c0 / D; }
    __device__ int last_group(int D) const { return (c1 - 1) / D; }
    __device__ long long at(const NormArgs &p, int s) const { return ((long long)n * p.S + s) * p.C + c0 + col * V; }
};

__host__ __device__ inline int norm_pieces(int G, int blocks) { return G + blocks - 1; }

template <typename IO, int V>
__global__ void __launch_bounds__(kTileThreads) norm_tile_stats_kernel(NormArgs p) {
    __shared__ float sh_mean[kTileThreads * V], sh_m2[kTileThreads * V];
    const Tile<V> t(p);
    const int D = p.C / p.G;
    float mean[V] = {}, m2[V] = {};
    float cnt = 0.f;
    if (t.live)
        for (int s = t.s0 + t.rl; s < t.s1; s += t.RL) {
            float x[V];
            load_vec<IO, V>(p.x, t.at(p, s), x);
            cnt += 1.f;
            const float f = 1.f / cnt;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = x[i] - mean[i];
                mean[i] = fmaf(d, f, mean[i]);
                m2[i] = fmaf(d, x[i] - mean[i], m2[i]);
            }
        }
    const int width = t.c1 - t.c0;
    if (t.live)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sh_mean[t.rl * width + t.col * V + i] = mean[i];
            sh_m2[t.rl * width + t.col * V + i] = m2[i];
        }
    __syncthreads();
    // one warp per group piece: the piece's channels times the RL rows of partial results
    const int lane = threadIdx.x & 31;
    for (int g = t.first_group(D) + (threadIdx.x >> 5); g <= t.last_group(D); g += kTileThreads / 32) {
        const int a = max(g * D, t.c0) - t.c0, b = min((g + 1) * D, t.c1) - t.c0;
        Stat st{0.f, 0.f, 0.f};
        for (int e = lane; e < (b - a) * t.RL; e += 32) {
            const int r = e / (b - a), c = a + e % (b - a);
            const int rows = t.s1 - t.s0 - r;  // positions of row lane r: s0 + r, s0 + r + RL, ...
            const float n = rows > 0 ? (float)((rows + t.RL - 1) / t.RL) : 0.f;
            st = merge(st, Stat{n, sh_mean[r * width + c], sh_m2[r * width + c]});
        }
        for (int o = 16; o > 0; o >>= 1) st = merge(st, shfl(st, o));
        if (lane == 0) {
            float *out = p.stat_parts + 2 * (((long long)blockIdx.x) * norm_pieces(p.G, gridDim.y) + g + t.cb);
            out[0] = st.mean;
            out[1] = st.m2;
        }
    }
}

// mean and rstd of group g of sample n from all tiles' pieces, by one warp
template <int V>
__device__ __forceinline__ Stat merge_pieces(const NormArgs &p, int n, int g, int blocks) {
    const int D = p.C / p.G, lane = threadIdx.x & 31;
    const int b0 = g * D / (kTileCols * V), b1 = ((g + 1) * D - 1) / (kTileCols * V), nb = b1 - b0 + 1;
    Stat st{0.f, 0.f, 0.f};
    for (int e = lane; e < p.tiles * nb; e += 32) {
        const int tile = e / nb, cb = b0 + e % nb;
        const int a = max(g * D, cb * kTileCols * V), b = min((g + 1) * D, (cb + 1) * kTileCols * V);
        const int rows = (int)((long long)p.S * (tile + 1) / p.tiles) - (int)((long long)p.S * tile / p.tiles);
        const float *in = p.stat_parts + 2 * (((long long)n * p.tiles + tile) * norm_pieces(p.G, blocks) + g + cb);
        st = merge(st, Stat{(float)(b - a) * (float)rows, in[0], in[1]});
    }
    for (int o = 16; o > 0; o >>= 1) st = merge(st, shfl(st, o));
    return st;
}

template <typename IO, int V>
__global__ void __launch_bounds__(kTileThreads) norm_tile_apply_kernel(NormArgs p) {
    __shared__ float sh_mean[kTileCols * V], sh_rstd[kTileCols * V];
    const Tile<V> t(p);
    const int D = p.C / p.G, g0 = t.first_group(D);
    for (int g = g0 + (threadIdx.x >> 5); g <= t.last_group(D); g += kTileThreads / 32) {
        const Stat st = merge_pieces<V>(p, t.n, g, gridDim.y);
        if ((threadIdx.x & 31) == 0) {
            const float rstd = 1.f / sqrtf(st.m2 / ((float)D * (float)p.S) + p.eps);
            sh_mean[g - g0] = st.mean;
            sh_rstd[g - g0] = rstd;
            if (t.tile == 0 && g * D >= t.c0) {  // the block with the group's first channel
                if (p.mean) p.mean[(long long)t.n * p.G + g] = st.mean;
                if (p.rstd) p.rstd[(long long)t.n * p.G + g] = rstd;
            }
        }
    }
    __syncthreads();
    if (!t.live) return;
    float mean[V], rstd[V], w[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = t.c0 + t.col * V + i, g = c / D - g0;
        mean[i] = sh_mean[g];
        rstd[i] = sh_rstd[g];
        w[i] = p.weight ? p.weight[c] : 1.f;
        b[i] = p.bias ? p.bias[c] : 0.f;
    }
    for (int s = t.s0 + t.rl; s < t.s1; s += t.RL) {
        const long long at = t.at(p, s);
        float x[V], gt[V] = {}, y[V];
        load_vec<IO, V>(p.x, at, x);
        if (p.gate) load_vec<IO, V>(p.gate, at, gt);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float z = fmaf((x[i] - mean[i]) * rstd[i], w[i], b[i]);
            y[i] = p.gate ? z * act_value(p.act, gt[i]) : act_value(p.act, z);
        }
        store_vec<IO, V>(p.y, at, y);
    }
}

// First kernel of the backward pass: per channel sum dz and sum dz xh over the tile, and their sums over
// each group piece with the weights.
template <typename IO, int V>
__global__ void __launch_bounds__(kTileThreads) norm_tile_grad_sums_kernel(NormArgs p) {
    __shared__ float sh1[kTileThreads * V], sh2[kTileThreads * V];
    const Tile<V> t(p);
    const int D = p.C / p.G, width = t.c1 - t.c0;
    if (t.live) {
        float mean[V], rstd[V], w[V], b[V], sz[V] = {}, szx[V] = {};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = t.c0 + t.col * V + i;
            mean[i] = p.mean[(long long)t.n * p.G + c / D];
            rstd[i] = p.rstd[(long long)t.n * p.G + c / D];
            w[i] = p.weight ? p.weight[c] : 1.f;
            b[i] = p.bias ? p.bias[c] : 0.f;
        }
        for (int s = t.s0 + t.rl; s < t.s1; s += t.RL) {
            const long long at = t.at(p, s);
            float x[V], dy[V], gt[V] = {}, dg;
            load_vec<IO, V>(p.x, at, x);
            load_vec<IO, V>(p.dy, at, dy);
            if (p.gate) load_vec<IO, V>(p.gate, at, gt);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float xh = (x[i] - mean[i]) * rstd[i];
                const float dz = dz_of(p, fmaf(xh, w[i], b[i]), dy[i], gt[i], dg);
                sz[i] += dz;
                szx[i] = fmaf(dz, xh, szx[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sh1[t.rl * width + t.col * V + i] = sz[i];
            sh2[t.rl * width + t.col * V + i] = szx[i];
        }
    }
    __syncthreads();
    float *chan = p.chan_parts + (long long)blockIdx.x * 2 * p.C + t.c0;
    for (int c = threadIdx.x; c < width; c += kTileThreads) {
        float a = 0.f, b = 0.f;
        for (int r = 0; r < t.RL; ++r) {
            a += sh1[r * width + c];
            b += sh2[r * width + c];
        }
        chan[c] = a;
        chan[p.C + c] = b;
        const float w = p.weight ? p.weight[t.c0 + c] : 1.f;
        sh1[c] = a * w;  // row lane 0's place, which only this thread reads
        sh2[c] = b * w;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for (int g = t.first_group(D) + (threadIdx.x >> 5); g <= t.last_group(D); g += kTileThreads / 32) {
        const int a = max(g * D, t.c0) - t.c0, b = min((g + 1) * D, t.c1) - t.c0;
        float s1 = 0.f, s2 = 0.f;
        for (int c = a + lane; c < b; c += 32) {
            s1 += sh1[c];
            s2 += sh2[c];
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (lane == 0) {
            float *out = p.stat_parts + 2 * (((long long)blockIdx.x) * norm_pieces(p.G, gridDim.y) + g + t.cb);
            out[0] = s1;
            out[1] = s2;
        }
    }
}

template <typename IO, int V>
__global__ void __launch_bounds__(kTileThreads) norm_tile_grad_apply_kernel(NormArgs p) {
    __shared__ float sh1[kTileCols * V], sh2[kTileCols * V];
    const Tile<V> t(p);
    const int D = p.C / p.G, g0 = t.first_group(D), lane = threadIdx.x & 31;
    const float inv = 1.f / ((float)D * (float)p.S);
    for (int g = g0 + (threadIdx.x >> 5); g <= t.last_group(D); g += kTileThreads / 32) {
        const int b0 = g * D / (kTileCols * V), b1 = ((g + 1) * D - 1) / (kTileCols * V), nb = b1 - b0 + 1;
        float s1 = 0.f, s2 = 0.f;
        for (int e = lane; e < p.tiles * nb; e += 32) {
            const float *in = p.stat_parts + 2 * (((long long)t.n * p.tiles + e / nb) * norm_pieces(p.G, gridDim.y) + g + b0 + e % nb);
            s1 += in[0];
            s2 += in[1];
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (lane == 0) {
            sh1[g - g0] = s1 * inv;
            sh2[g - g0] = s2 * inv;
        }
    }
    __syncthreads();
    if (!t.live) return;
    float mean[V], rstd[V], w[V], b[V], s1[V], s2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = t.c0 + t.col * V + i, g = c / D;
        mean[i] = p.mean[(long long)t.n * p.G + g];
        rstd[i] = p.rstd[(long long)t.n * p.G + g];
        w[i] = p.weight ? p.weight[c] : 1.f;
        b[i] = p.bias ? p.bias[c] : 0.f;
        s1[i] = sh1[g - g0];
        s2[i] = sh2[g - g0];
    }
    for (int s = t.s0 + t.rl; s < t.s1; s += t.RL) {
        const long long at = t.at(p, s);
        float x[V], dy[V], gt[V] = {}, dg[V], dx[V];
        load_vec<IO, V>(p.x, at, x);
        load_vec<IO, V>(p.dy, at, dy);
        if (p.gate) load_vec<IO, V>(p.gate, at, gt);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float xh = (x[i] - mean[i]) * rstd[i];
            const float dz = dz_of(p, fmaf(xh, w[i], b[i]), dy[i], gt[i], dg[i]);
            dx[i] = rstd[i] * (fmaf(dz, w[i], -s1[i]) - xh * s2[i]);
        }
        store_vec<IO, V>(p.dx, at, dx);
        if (p.gate) store_vec<IO, V>(p.dgate, at, dg);
    }
}

// ---- plan and launches -----------------------------------------------------------------------------

struct NormPlan {
    bool rows;
    int V;                   // channels of a vector
    int LG, K;               // rows form: lanes of a group, vectors of a lane at most
    int row_lanes, blocks;   // rows form: rows in work at a time, CTAs
    int tiles, col_blocks;   // tiles form
};

NormPlan plan_of(const prism_norm_shape &s, bool backward) {
    const int D = s.C / s.G, full = s.io == PRISM_F32 ? 4 : 8;
    NormPlan pl{};
    pl.V = D % full == 0 ? full : 1;
    const int nv = D / pl.V;
    pl.rows = s.S == 1 && nv <= 32 * kRowVecs;
    const int sms = sm_count();
    if (pl.rows) {
        pl.LG = 1;
        while (pl.LG < nv && pl.LG < 32) pl.LG *= 2;
        pl.K = nv <= 32 ? 1 : kRowVecs;
        const long long per_block = kRowThreads / pl.LG;
        long long lanes = std::max<long long>(1, (long long)sms * (backward ? 4 : 8) * per_block / s.G);
        lanes = std::min<long long>(lanes, std::max(1, s.N));
        pl.row_lanes = (int)lanes;
        pl.blocks = (int)((lanes * s.G + per_block - 1) / per_block);
        return pl;
    }
    pl.V = s.C % full == 0 ? full : 1;
    pl.col_blocks = (s.C / pl.V + kTileCols - 1) / kTileCols;
    const long long others = std::max(1LL, (long long)s.N * pl.col_blocks);
    pl.tiles = (int)std::max<long long>(1, std::min<long long>((4LL * sms + others - 1) / others, s.S / 16));
    return pl;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t stat_bytes(const prism_norm_shape &s, const NormPlan &pl) {
    return pl.rows ? 0 : align256((size_t)s.N * pl.tiles * norm_pieces(s.G, pl.col_blocks) * 8);
}
int chan_parts(const prism_norm_shape &s, const NormPlan &pl) { return pl.rows ? pl.row_lanes : s.N * pl.tiles; }

prism_status check_shape(const prism_norm_shape *s) {
    if (!s) return PRISM_ERR_INVALID_ARG;
    if (s->N < 0 || s->S < 0 || s->C < 1 || s->G < 1 || s->C % s->G) return PRISM_ERR_INVALID_ARG;
    if (s->io != PRISM_BF16 && s->io != PRISM_F32) return PRISM_ERR_INVALID_ARG;
    if (s->act != PRISM_ACT_NONE && s->act != PRISM_ACT_SILU && s->act != PRISM_ACT_GELU) return PRISM_ERR_INVALID_ARG;
    if (!(s->eps >= 0.f)) return PRISM_ERR_INVALID_ARG;
    if (s->C > (1 << 20) || (long long)s->N * s->G > 0x7fffffffLL || s->N > (1 << 24)) return PRISM_ERR_UNSUPPORTED;
    return PRISM_OK;
}

template <typename IO>
cudaError_t launch_fwd(const NormArgs &a, const NormPlan &pl, cudaStream_t s) {
    constexpr int F = 16 / sizeof(IO);
    launch_probe_mark(s);
    if (pl.rows) {
        auto kern = pl.V == 1 ? (pl.K == 1 ? norm_rows_fwd_kernel<IO, 1, 1> : norm_rows_fwd_kernel<IO, 1, kRowVecs>)
                              : (pl.K == 1 ? norm_rows_fwd_kernel<IO, F, 1> : norm_rows_fwd_kernel<IO, F, kRowVecs>);
        kern<<<pl.blocks, kRowThreads, 0, s>>>(a, pl.LG, pl.row_lanes);
        return cudaGetLastError();
    }
    const dim3 grid(a.N * a.tiles, pl.col_blocks);
    (pl.V == 1 ? norm_tile_stats_kernel<IO, 1> : norm_tile_stats_kernel<IO, F>)<<<grid, kTileThreads, 0, s>>>(a);
    launch_probe_mark(s);
    (pl.V == 1 ? norm_tile_apply_kernel<IO, 1> : norm_tile_apply_kernel<IO, F>)<<<grid, kTileThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t launch_bwd(const NormArgs &a, const NormPlan &pl, float *dweight, float *dbias, cudaStream_t s) {
    constexpr int F = 16 / sizeof(IO);
    launch_probe_mark(s);
    if (pl.rows) {
        auto kern = pl.V == 1 ? (pl.K == 1 ? norm_rows_bwd_kernel<IO, 1, 1> : norm_rows_bwd_kernel<IO, 1, kRowVecs>)
                              : (pl.K == 1 ? norm_rows_bwd_kernel<IO, F, 1> : norm_rows_bwd_kernel<IO, F, kRowVecs>);
        kern<<<pl.blocks, kRowThreads, 0, s>>>(a, pl.LG, pl.row_lanes);
    } else {
        const dim3 grid(a.N * a.tiles, pl.col_blocks);
        (pl.V == 1 ? norm_tile_grad_sums_kernel<IO, 1> : norm_tile_grad_sums_kernel<IO, F>)<<<grid, kTileThreads, 0, s>>>(a);
        launch_probe_mark(s);
        (pl.V == 1 ? norm_tile_grad_apply_kernel<IO, 1> : norm_tile_grad_apply_kernel<IO, F>)<<<grid, kTileThreads, 0, s>>>(a);
    }
    if (dweight || dbias) {
        launch_probe_mark(s);
        norm_channel_sum_kernel<<<(2 * a.C + 31) / 32, 256, 0, s>>>(a.chan_parts, a.parts, a.C, dweight, dbias);
    }
    return cudaGetLastError();
}

NormArgs args_of(const prism_norm_shape &s, const NormPlan &pl, const void *x, const float *weight, const float *bias,
                 const void *gate) {
    NormArgs a{};
    a.N = s.N; a.S = s.S; a.C = s.C; a.G = s.G; a.act = s.act; a.eps = s.eps;
    a.x = x; a.gate = gate; a.weight = weight; a.bias = bias;
    a.tiles = pl.tiles;
    return a;
}

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

}  // namespace
}  // namespace prism

using namespace prism;

extern "C" {

prism_status prism_group_norm_fwd_workspace_size(const prism_norm_shape *shape, size_t *bytes) {
    if (!bytes) return PRISM_ERR_INVALID_ARG;
    const prism_status st = check_shape(shape);
    if (st != PRISM_OK) return st;
    *bytes = std::max<size_t>(256, stat_bytes(*shape, plan_of(*shape, false)));
    return PRISM_OK;
}

prism_status prism_group_norm_fwd(const prism_norm_shape *shape, const void *x, const float *weight, const float *bias,
                                  const void *gate, void *y, float *mean, float *rstd, void *workspace, size_t ws_bytes,
                                  void *stream) {
    const prism_status st = check_shape(shape);
    if (st != PRISM_OK) return st;
    const prism_norm_shape &s = *shape;
    const size_t n = (size_t)s.N * s.S * s.C * (s.io == PRISM_F32 ? 4 : 2), groups = (size_t)s.N * s.G * 4;
    if (n == 0) return PRISM_OK;
    if (!x || !y || !aligned16(x) || !aligned16(y) || !aligned16(gate)) return PRISM_ERR_INVALID_ARG;
    if (!aligned4(weight) || !aligned4(bias) || !aligned4(mean) || !aligned4(rstd)) return PRISM_ERR_INVALID_ARG;
    const NormPlan pl = plan_of(s, false);
    const size_t need = std::max<size_t>(256, stat_bytes(s, pl));
    if (!workspace || ws_bytes < need || ((uintptr_t)workspace & 255u)) return PRISM_ERR_INVALID_ARG;
    const ByteRange outs[] = {{y, n}, {mean, groups}, {rstd, groups}, {workspace, need}};
    const ByteRange ins[] = {{x, n}, {gate, n}, {weight, (size_t)s.C * 4}, {bias, (size_t)s.C * 4}};
    if (outputs_alias(outs, 4, ins, 4)) return PRISM_ERR_INVALID_ARG;
    NormArgs a = args_of(s, pl, x, weight, bias, gate);
    a.y = y; a.mean = mean; a.rstd = rstd; a.stat_parts = (float *)workspace;
    const cudaError_t err = s.io == PRISM_F32 ? launch_fwd<float>(a, pl, (cudaStream_t)stream)
                                              : launch_fwd<__nv_bfloat16>(a, pl, (cudaStream_t)stream);
    probe_finish((cudaStream_t)stream);
    return cuda_status(err);
}

prism_status prism_group_norm_bwd_workspace_size(const prism_norm_shape *shape, size_t *bytes) {
    if (!bytes) return PRISM_ERR_INVALID_ARG;
    const prism_status st = check_shape(shape);
    if (st != PRISM_OK) return st;
    const NormPlan pl = plan_of(*shape, true);
    *bytes = std::max<size_t>(256, stat_bytes(*shape, pl) + (size_t)chan_parts(*shape, pl) * 2 * shape->C * 4);
    return PRISM_OK;
}

prism_status prism_group_norm_bwd(const prism_norm_shape *shape, const void *x, const float *weight, const float *bias,
                                  const void *gate, const float *mean, const float *rstd, const void *dy, void *dx,
                                  void *dgate, float *dweight, float *dbias, void *workspace, size_t ws_bytes, void *stream) {
    const prism_status st = check_shape(shape);
    if (st != PRISM_OK) return st;
    const prism_norm_shape &s = *shape;
    const size_t n = (size_t)s.N * s.S * s.C * (s.io == PRISM_F32 ? 4 : 2), groups = (size_t)s.N * s.G * 4;
    if (!aligned4(weight) || !aligned4(bias) || !aligned4(mean) || !aligned4(rstd) || !aligned4(dweight) || !aligned4(dbias))
        return PRISM_ERR_INVALID_ARG;
    if (n == 0) {  // sums over nothing
        cudaError_t err = cudaSuccess;
        if (dweight) err = cudaMemsetAsync(dweight, 0, (size_t)s.C * 4, (cudaStream_t)stream);
        if (dbias && err == cudaSuccess) err = cudaMemsetAsync(dbias, 0, (size_t)s.C * 4, (cudaStream_t)stream);
        return cuda_status(err);
    }
    if (!x || !dy || !dx || !mean || !rstd || (gate != nullptr) != (dgate != nullptr)) return PRISM_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(dy) || !aligned16(dx) || !aligned16(gate) || !aligned16(dgate)) return PRISM_ERR_INVALID_ARG;
    const NormPlan pl = plan_of(s, true);
    size_t need = 0;
    prism_group_norm_bwd_workspace_size(shape, &need);
    if (!workspace || ws_bytes < need || ((uintptr_t)workspace & 255u)) return PRISM_ERR_INVALID_ARG;
    const size_t chan = (size_t)s.C * 4;
    const ByteRange outs[] = {{dx, n}, {dgate, n}, {dweight, chan}, {dbias, chan}, {workspace, need}};
    const ByteRange ins[] = {{x, n}, {gate, n}, {dy, n}, {mean, groups}, {rstd, groups}, {weight, chan}, {bias, chan}};
    if (outputs_alias(outs, 5, ins, 7)) return PRISM_ERR_INVALID_ARG;
    NormArgs a = args_of(s, pl, x, weight, bias, gate);
    a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
    a.dy = dy; a.dx = dx; a.dgate = dgate;
    a.stat_parts = (float *)workspace;
    a.chan_parts = (float *)((char *)workspace + stat_bytes(s, pl));
    a.parts = chan_parts(s, pl);
    if (pl.rows && !dweight && !dbias) a.chan_parts = nullptr;
    const cudaError_t err = s.io == PRISM_F32 ? launch_bwd<float>(a, pl, dweight, dbias, (cudaStream_t)stream)
                                              : launch_bwd<__nv_bfloat16>(a, pl, dweight, dbias, (cudaStream_t)stream);
    probe_finish((cudaStream_t)stream);
    return cuda_status(err);
}

}  // extern "C"
