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
//           channels (one vector) for all of its positions.  (One kernel whose CTAs keep a sample in the shared
//           memory of a cluster was measured: 53 us against 27 on 8 samples of 4096 x 320, which takes clusters of 16.)
// Vectors are 16 bytes where the channels of a group (rows) or of a position (tiles) divide into them, one
// channel where they do not.
// Every result is (count, mean, sum of squares about the mean), and results are merged by their means' differences
// from the first of them: a mean far above the deviation costs no digits beyond its own rounding.

#include <algorithm>
#include <type_traits>

#include "api.cuh"
#include "common.cuh"
#include "dependent.cuh"
#include "f32x2.cuh"

namespace prism {
namespace {

struct NormArgs {
    int N, S, C, G, act;
    float eps;
    const void *x, *gate, *dy;
    const float *weight, *bias;
    float *mean, *rstd;      // outputs of the forward pass (may be null), inputs of the backward one
    void *y, *dx, *dgate;
    float *stat_parts;       // tiles form: [N][pieces][tiles][2]
    float *chan_parts;       // backward: [parts][2][C] sums of dz and dz xh
    int tiles, parts;
    int tile_len, tile_more;  // tiles form: positions of a tile, and how many first tiles have one more
};

// ---- activations -------------------------------------------------------------------------------

// Kernels for the common vector widths are built for each activation, with and without a gate (a mode);
// kRuntime takes both from the arguments.
constexpr int kRuntime = -1;
template <int MODE>
__device__ __forceinline__ int mode_act(const NormArgs &p) { return MODE == kRuntime ? p.act : MODE >> 1; }
template <int MODE>
__device__ __forceinline__ bool mode_gate(const NormArgs &p) { return MODE == kRuntime ? p.gate != nullptr : MODE & 1; }

// 1 / x to 1 ulp (0 for infinities: what 1 / (1 + exp(-z)) tends to where exp overflows)
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// __expf for bf16 results: its error, about |x| 2^-24, is far below their rounding.
template <typename IO>
__device__ __forceinline__ float exp_io(float x) { return sizeof(IO) == 2 ? __expf(x) : expf(x); }

template <typename IO>
__device__ __forceinline__ float act_value(int act, float z) {
    if (act == PRISM_ACT_SILU) return z * rcp_approx(1.f + exp_io<IO>(-z));
    if (act == PRISM_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    return z;
}

// act(z) and act'(z)
template <typename IO>
__device__ __forceinline__ float act_both(int act, float z, float &slope) {
    if (act == PRISM_ACT_SILU) {
        const float s = rcp_approx(1.f + exp_io<IO>(-z)), a = z * s;
        slope = fmaf(a, 1.f - s, s);
        return a;
    }
    if (act == PRISM_ACT_GELU) {
        const float c = 0.5f * (1.f + erff(z * 0.70710678118654752f));
        slope = fmaf(z * 0.39894228040143268f, exp_io<IO>(-0.5f * z * z), c);
        return z * c;
    }
    slope = 1.f;
    return z;
}

// ---- arithmetic on a vector's elements, two at a time (packed f32x2) where there are two ----------
//
// A unit of one element is a float, of two a 64-bit register pair.

template <int V>
using Unit = std::conditional_t<V == 1, float, F2>;
template <int V>
constexpr int kUnits = V == 1 ? 1 : V / 2;

template <int V>
__device__ __forceinline__ Unit<V> unit_of(const float (&x)[V], int u) {
    if constexpr (V == 1) return x[0];
    else return pack2(x[2 * u], x[2 * u + 1]);
}
template <typename U>
__device__ __forceinline__ U both(float x) {
    if constexpr (sizeof(U) == 4) return x;
    else return pack2(x, x);
}

// ---- vectors of V consecutive channels -----------------------------------------------------------

template <typename IO, int V>
struct alignas(sizeof(IO) * V) Pack {
    IO v[V];
    __device__ __forceinline__ float at(int i) const { return ld_io(v, i); }
    __device__ __forceinline__ Unit<V> unit(int u) const {
        if constexpr (V == 1) return at(0);
        else return pack2(at(2 * u), at(2 * u + 1));
    }
    __device__ __forceinline__ void set(int u, float x) { st_io(v, u, x); }
    __device__ __forceinline__ void set(int u, F2 x) {
        if constexpr (V > 1) {
            if constexpr (sizeof(IO) == 2) {
                reinterpret_cast<__nv_bfloat162 *>(v)[u] = __floats2bfloat162_rn(first(x), second(x));
            } else {
                st_io(v, 2 * u, first(x));
                st_io(v, 2 * u + 1, second(x));
            }
        }
    }
};

template <typename IO, int V>
__device__ __forceinline__ Pack<IO, V> load_pack(const void *p, long long at) {
    return *reinterpret_cast<const Pack<IO, V> *>((const IO *)p + at);
}
template <typename IO, int V>
__device__ __forceinline__ void store_pack(void *p, long long at, const Pack<IO, V> &r) {
    *reinterpret_cast<Pack<IO, V> *>((IO *)p + at) = r;
}
// Unit u of a channel array (parameters), `missing` where there is none.
template <int V>
__device__ __forceinline__ Unit<V> channel_unit(const float *p, int c, float missing) {
    if constexpr (V == 1) return p ? p[c] : missing;
    else return p ? pack2(p[c], p[c + 1]) : pack2(missing, missing);
}

template <typename IO, int MODE>
__device__ __forceinline__ float y_of(const NormArgs &p, float z, float gate) {
    return mode_gate<MODE>(p) ? z * act_value<IO>(mode_act<MODE>(p), gate) : act_value<IO>(mode_act<MODE>(p), z);
}
template <typename IO, int MODE>
__device__ __forceinline__ F2 y_of(const NormArgs &p, F2 z, F2 gate) {
    return pack2(y_of<IO, MODE>(p, first(z), first(gate)), y_of<IO, MODE>(p, second(z), second(gate)));
}

// dz of one element (before the weight), and its dgate
template <typename IO, int MODE>
__device__ __forceinline__ float dz_of(const NormArgs &p, float z, float dy, float gate, float &dgate) {
    float slope;
    if (mode_gate<MODE>(p)) {
        const float a = act_both<IO>(mode_act<MODE>(p), gate, slope);
        dgate = dy * z * slope;
        return dy * a;
    }
    act_both<IO>(mode_act<MODE>(p), z, slope);
    dgate = 0.f;
    return dy * slope;
}
template <typename IO, int MODE>
__device__ __forceinline__ F2 dz_of(const NormArgs &p, F2 z, F2 dy, F2 gate, F2 &dgate) {
    float d0, d1;
    const float a = dz_of<IO, MODE>(p, first(z), first(dy), first(gate), d0);
    const float b = dz_of<IO, MODE>(p, second(z), second(dy), second(gate), d1);
    dgate = pack2(d0, d1);
    return pack2(a, b);
}

// ---- rows form -----------------------------------------------------------------------------------

constexpr int kRowThreads = 256;
constexpr int kRowVecs = 4;  // vectors of a lane at most
constexpr int kRowFwdBlocks = 4, kRowBwdBlocks = 2;  // CTAs of an SM (one vector per lane)

// Sum over the LG lanes of a group (LG a power of two, groups aligned to it).
template <int LG>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int o = LG >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// What a lane of the rows form works on: LG lanes hold one (row, group) at a time, lane l the vectors l,
// l + LG, ... of its D / V.  A lane group keeps its group g over all of its rows, so the weights are read
// once.  Close to both bounds: memory, and the instructions of the activation and of the two
// reductions.  The next row is requested before the current one is reduced, LG is a template
// argument and the arithmetic runs on packed pairs (gated norm of 65536 x 16 heads of 128 at bf16: 365 us
// without the three, 41 instructions an element).
template <int V, int K, int LG>
struct RowLane {
    using U = Unit<V>;
    int D, nv, lane, g, first;  // (row lanes are few: RowLane::first < the number of rows)
    bool mine;
    long long base, step;       // element of this lane's first vector, and to the next row's
    U w[K][kUnits<V>], b[K][kUnits<V>];
    __device__ RowLane(const NormArgs &p, int row_lanes) {
        D = p.C / p.G;
        nv = D / V;
        lane = threadIdx.x & (LG - 1);
        const int unit = (blockIdx.x * kRowThreads + threadIdx.x) / LG;
        g = unit % p.G;
        first = unit / p.G;
        mine = first < row_lanes;
        base = (long long)first * p.C + (long long)g * D + lane * V;
        step = (long long)row_lanes * p.C;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int u = 0; u < kUnits<V>; ++u) {
                const int c = g * D + (lane + k * LG) * V + 2 * u;
                w[k][u] = channel_unit<V>(has(k) ? p.weight : nullptr, c, 1.f);
                b[k][u] = channel_unit<V>(has(k) ? p.bias : nullptr, c, 0.f);
            }
    }
    __device__ __forceinline__ bool has(int k) const { return lane + k * LG < nv; }
};

// A thread's own vectors of the rows to come, NT tensors, kRing - 1 rows ahead: asynchronous copies into
// shared memory (read back by the same thread, so there is nothing to synchronise).  Registers for one row
// ahead kept 32 KB in flight per SM, 4.5 TB/s.
constexpr int kRing = 4;

template <typename IO, int V, int NT>
struct RowRing {
    static_assert(sizeof(Pack<IO, V>) == 16, "16-byte copies");
    Pack<IO, V> (*buf)[NT][kRowThreads];  // [kRing], shared
    __device__ __forceinline__ void copy(int slot, int tensor, const void *p, long long at) const {
        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(&buf[slot][tensor][threadIdx.x]);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"((const IO *)p + at) : "memory");
    }
    __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // every copy but those of the kRing - 1 latest rows has landed
    __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory"); }
    __device__ __forceinline__ Pack<IO, V> get(int slot, int tensor) const { return buf[slot][tensor][threadIdx.x]; }
};

template <typename IO, int V, int K, int LG, int MODE>
__global__ void __launch_bounds__(kRowThreads, K == 1 ? kRowFwdBlocks : 1) norm_rows_fwd_kernel(NormArgs p, int row_lanes) {
    using U = Unit<V>;
    constexpr int NU = kUnits<V>;
    constexpr bool RING = K == 1 && V > 1;
    __shared__ Pack<IO, V> buf[RING ? kRing : 1][2][RING ? kRowThreads : 1];
    const RowLane<V, K, LG> t(p, row_lanes);
    const float inv = 1.f / (float)t.D;
    Pack<IO, V> xr[K], gr[K];
    int slot = 0;
    auto request = [&](int row, long long at, int to) {  // into ring slot `to`, or registers
        if (t.mine && row < p.N)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (t.has(k)) {
                    if constexpr (RING) {
                        const RowRing<IO, V, 2> ring{buf};
                        ring.copy(to, 0, p.x, at);
                        if (mode_gate<MODE>(p)) ring.copy(to, 1, p.gate, at);
                    } else {
                        xr[k] = load_pack<IO, V>(p.x, at + k * LG * V);
                        if (mode_gate<MODE>(p)) gr[k] = load_pack<IO, V>(p.gate, at + k * LG * V);
                    }
                }
        if constexpr (RING) RowRing<IO, V, 2>::commit();
    };
    long long at = t.base;
#pragma unroll
    for (int k = 0; k < (RING ? kRing - 1 : 1); ++k) request(t.first + k * row_lanes, at + k * t.step, k);
    // the lane groups of one warp take the same number of steps, so that every shuffle has all lanes
    for (int r0 = 0; r0 < p.N; r0 += row_lanes, at += t.step) {
        const int row = r0 + t.first;
        const bool live = t.mine && row < p.N;
        U x[K][NU], s = both<U>(0.f);
        Pack<IO, V> gc[K];
        if constexpr (RING) {
            request(row + (kRing - 1) * row_lanes, at + (kRing - 1) * t.step, (slot + kRing - 1) % kRing);
            const RowRing<IO, V, 2> ring{buf};
            ring.wait();
            xr[0] = ring.get(slot, 0);
            if (mode_gate<MODE>(p)) gr[0] = ring.get(slot, 1);
            slot = (slot + 1) % kRing;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            gc[k] = gr[k];
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                x[k][u] = xr[k].unit(u);
                if (t.has(k)) s = add(s, x[k][u]);
            }
        }
        if constexpr (!RING) request(row + row_lanes, at + t.step, 0);
        const float mean = lanes_sum<LG>(total(s)) * inv;
        U q = both<U>(0.f);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                x[k][u] = add(x[k][u], both<U>(-mean));
                if (t.has(k)) q = fma(x[k][u], x[k][u], q);
            }
        const float rstd = rsqrtf(fmaf(lanes_sum<LG>(total(q)), inv, p.eps));
        if (!live) continue;
        if (t.lane == 0) {
            if (p.mean) p.mean[(long long)row * p.G + t.g] = mean;
            if (p.rstd) p.rstd[(long long)row * p.G + t.g] = rstd;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!t.has(k)) continue;
            Pack<IO, V> y;
#pragma unroll
            for (int u = 0; u < NU; ++u)
                y.set(u, y_of<IO, MODE>(p, fma(mul(x[k][u], both<U>(rstd)), t.w[k][u], t.b[k][u]), gc[k].unit(u)));
            store_pack<IO, V>(p.y, at + k * LG * V, y);
        }
    }
}

// The same lanes for the backward pass; a lane also sums dz and dz xh of its channels over its rows.
template <typename IO, int V, int K, int LG, int MODE>
__global__ void __launch_bounds__(kRowThreads, K == 1 ? kRowBwdBlocks : 1) norm_rows_bwd_kernel(NormArgs p, int row_lanes) {
    using U = Unit<V>;
    constexpr int NU = kUnits<V>;
    dependent_wait();
    const RowLane<V, K, LG> t(p, row_lanes);
    const float inv = 1.f / (float)t.D;
    U sz[K][NU], szx[K][NU];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int u = 0; u < NU; ++u) sz[k][u] = szx[k][u] = both<U>(0.f);
    constexpr bool RING = K == 1 && V > 1;
    constexpr int AHEAD = RING ? kRing - 1 : 1;
    __shared__ Pack<IO, V> buf[RING ? kRing : 1][3][RING ? kRowThreads : 1];
    Pack<IO, V> xr[K], dr[K], gr[K];
    float mean_n[AHEAD] = {}, rstd_n[AHEAD] = {};  // of the rows to come, the next one first
    int slot = 0;
    auto request = [&](int row, long long at, int to, float &mean, float &rstd) {
        if (t.mine && row < p.N) {
            mean = p.mean[(long long)row * p.G + t.g];
            rstd = p.rstd[(long long)row * p.G + t.g];
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (t.has(k)) {
                    if constexpr (RING) {
                        const RowRing<IO, V, 3> ring{buf};
                        ring.copy(to, 0, p.x, at);
                        ring.copy(to, 1, p.dy, at);
                        if (mode_gate<MODE>(p)) ring.copy(to, 2, p.gate, at);
                    } else {
                        xr[k] = load_pack<IO, V>(p.x, at + k * LG * V);
                        dr[k] = load_pack<IO, V>(p.dy, at + k * LG * V);
                        if (mode_gate<MODE>(p)) gr[k] = load_pack<IO, V>(p.gate, at + k * LG * V);
                    }
                }
        }
        if constexpr (RING) RowRing<IO, V, 3>::commit();
    };
    long long at = t.base;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) request(t.first + k * row_lanes, at + k * t.step, k, mean_n[k], rstd_n[k]);
    for (int r0 = 0; r0 < p.N; r0 += row_lanes, at += t.step) {
        const int row = r0 + t.first;
        const bool live = t.mine && row < p.N;
        const float mean = mean_n[0], rstd = rstd_n[0];
#pragma unroll
        for (int k = 0; k + 1 < AHEAD; ++k) {
            mean_n[k] = mean_n[k + 1];
            rstd_n[k] = rstd_n[k + 1];
        }
        if constexpr (RING) {
            request(row + AHEAD * row_lanes, at + AHEAD * t.step, (slot + AHEAD) % kRing, mean_n[AHEAD - 1], rstd_n[AHEAD - 1]);
            const RowRing<IO, V, 3> ring{buf};
            ring.wait();
            xr[0] = ring.get(slot, 0);
            dr[0] = ring.get(slot, 1);
            if (mode_gate<MODE>(p)) gr[0] = ring.get(slot, 2);
            slot = (slot + 1) % kRing;
        }
        U xh[K][NU], dn[K][NU], s1 = both<U>(0.f), s2 = both<U>(0.f);
        Pack<IO, V> dg[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!live || !t.has(k)) continue;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                xh[k][u] = mul(add(xr[k].unit(u), both<U>(-mean)), both<U>(rstd));
                U d;
                const U dz = dz_of<IO, MODE>(p, fma(xh[k][u], t.w[k][u], t.b[k][u]), dr[k].unit(u), gr[k].unit(u), d);
                dg[k].set(u, d);
                sz[k][u] = add(sz[k][u], dz);
                szx[k][u] = fma(dz, xh[k][u], szx[k][u]);
                dn[k][u] = mul(dz, t.w[k][u]);
                s1 = add(s1, dn[k][u]);
                s2 = fma(dn[k][u], xh[k][u], s2);
            }
            if (mode_gate<MODE>(p)) store_pack<IO, V>(p.dgate, at + k * LG * V, dg[k]);
        }
        if constexpr (!RING) request(row + row_lanes, at + t.step, 0, mean_n[0], rstd_n[0]);
        const float m1 = lanes_sum<LG>(total(s1)) * inv, m2 = lanes_sum<LG>(total(s2)) * inv;
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!t.has(k)) continue;
            Pack<IO, V> dx;
#pragma unroll
            for (int u = 0; u < NU; ++u)
                dx.set(u, mul(both<U>(rstd), fma(xh[k][u], both<U>(-m2), add(dn[k][u], both<U>(-m1)))));
            store_pack<IO, V>(p.dx, at + k * LG * V, dx);
        }
    }
    if (!p.chan_parts || !t.mine) return;
    float *out = p.chan_parts + (long long)t.first * 2 * p.C + t.g * t.D + t.lane * V;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (!t.has(k)) continue;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            float *o = out + k * LG * V + 2 * u;
            if constexpr (V == 1) {
                o[0] = sz[k][u];
                o[p.C] = szx[k][u];
            } else {
                o[0] = first(sz[k][u]);
                o[1] = second(sz[k][u]);
                o[p.C] = first(szx[k][u]);
                o[p.C + 1] = second(szx[k][u]);
            }
        }
    }
}

// dbias, dweight: the parts' sums, 32 columns of [dz | dz xh] per block and 32 interleaved ranges of parts,
// four loads in flight per thread.
__global__ void __launch_bounds__(1024) norm_channel_sum_kernel(const float *parts, int n, int C, float *dweight, float *dbias) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    dependent_wait();
    float acc[4] = {};
    if (col < 2 * C)
        for (int i = k; i < n; i += 128)
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i + 32 * u < n) acc[u] += parts[(long long)(i + 32 * u) * 2 * C + col];
    s[k][lane] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    __syncthreads();
    const float sum = warp_sum(s[lane][k]);  // warp k: column k of the block
    const int c = blockIdx.x * 32 + k;
    if (lane == 0 && c < 2 * C) {
        if (c < C) {
            if (dbias) dbias[c] = sum;
        } else if (dweight) {
            dweight[c - C] = sum;
        }
    }
}

// ---- tiles form ----------------------------------------------------------------------------------

constexpr int kTileThreads = 256;
constexpr int kTileCols = 256;  // vector columns of a block

// Geometry of a block: channels [c0, c1) (whole vectors), positions [s0, s1) of sample n; thread
// (col, rl) owns V channels and every RL-th position.
template <int V>
struct Tile {
    int n, tile, cb, c0, c1, cols, RL, col, rl, s0, s1;
    bool live;
    __device__ Tile(const NormArgs &p, int unit) {  // unit: n * tiles + tile
        n = unit / p.tiles;
        tile = unit % p.tiles;
        cb = blockIdx.y;
        c0 = cb * kTileCols * V;
        c1 = min(c0 + kTileCols * V, p.C);
        cols = (c1 - c0) / V;
        RL = kTileThreads / cols;
        col = threadIdx.x % cols;
        rl = threadIdx.x / cols;
        live = rl < RL;
        s0 = tile * p.tile_len + min(tile, p.tile_more);
        s1 = s0 + positions(p, tile);
    }
    __device__ __forceinline__ static int positions(const NormArgs &p, int tile) { return p.tile_len + (tile < p.tile_more); }
    // A group cut by a block's edge leaves one piece in each block: piece g + cb is group g's in block cb.
    __device__ int first_group(int D) const { return c0 / D; }
    __device__ int last_group(int D) const { return (c1 - 1) / D; }
    __device__ long long at(const NormArgs &p, int s) const { return ((long long)n * p.S + s) * p.C + c0 + col * V; }
};

// A thread's vectors of the positions s0 + rl, s0 + rl + RL, ... of NT tensors (x, dy, gate; a null one is
// skipped), AHEAD - 1 positions ahead of their use: asynchronous copies into shared memory, read back by the
// same thread.  (Batches of plain loads, each waited for before the next, reached a third of the bandwidth.)
// Vectors of less than 16 bytes are loaded when they are due.
template <typename IO, int V, int NT>
struct PosStream {
    static constexpr bool RING = sizeof(Pack<IO, V>) == 16;
    static constexpr int AHEAD = NT == 3 ? 5 : 8;  // (two blocks of 256 threads fit an SM)
    const void *t[NT];
    Pack<IO, V> *buf;  // shared, [AHEAD][NT][kTileThreads]
    long long at, step;
    int s, end, RL, slot;
    __device__ PosStream(const NormArgs &p, const Tile<V> &tile, Pack<IO, V> *ring) : buf(ring) {
        s = tile.s0 + tile.rl;
        end = tile.live ? tile.s1 : tile.s0;
        RL = tile.RL;
        at = tile.at(p, s);
        step = (long long)RL * p.C;
        slot = 0;
    }
    __device__ __forceinline__ Pack<IO, V> *place(int sl, int k) const { return buf + (sl * NT + k) * kTileThreads + threadIdx.x; }
    __device__ __forceinline__ void request(int ahead, int sl) {
        if constexpr (RING) {
            if (s + ahead * RL < end)
#pragma unroll
                for (int k = 0; k < NT; ++k)
                    if (t[k]) {
                        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(place(sl, k));
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"((const IO *)t[k] + at + ahead * step)
                                     : "memory");
                    }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    __device__ __forceinline__ void start() {
#pragma unroll
        for (int k = 0; k + 1 < AHEAD; ++k) request(k, k);
    }
    __device__ __forceinline__ bool more() const { return s < end; }
    __device__ __forceinline__ int positions() const { return s < end ? (end - s + RL - 1) / RL : 0; }
    // The current position's vectors; requests the one AHEAD - 1 further on.
    __device__ __forceinline__ void get(Pack<IO, V> (&x)[NT]) {
        if constexpr (RING) {
            request(AHEAD - 1, (slot + AHEAD - 1) % AHEAD);
            asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
        }
#pragma unroll
        for (int k = 0; k < NT; ++k)
            if (t[k]) x[k] = RING ? *place(slot, k) : load_pack<IO, V>(t[k], at);
    }
    __device__ __forceinline__ void next() {
        s += RL;
        at += step;
        slot = (slot + 1) % AHEAD;
    }
};
template <typename IO, int V, int NT>
constexpr int kPosBytes = PosStream<IO, V, NT>::RING ? PosStream<IO, V, NT>::AHEAD * NT * kTileThreads * 16 : 0;

__host__ __device__ inline int norm_pieces(int G, int blocks) { return G + blocks - 1; }
// Where the pair of a group's piece in column block cb is, among stat_parts' pairs.
__device__ __forceinline__ long long piece_at(const NormArgs &p, int n, int tile, int g, int cb, int blocks) {
    return ((long long)n * norm_pieces(p.G, blocks) + g + cb) * p.tiles + tile;
}

// The threads of a block over its groups, `lanes` (a power of two up to 32) neighbours for each group, all groups at
// once where they fit.  This code and what uses it run once per block: what they cost are latencies and
// instruction fetches, so all of it is short loops.  (A warp per group, four groups unrolled, and a merge with a
// division for every pair of results: 3 us of each kernel's 13 to 17.)
struct GroupLanes {
    int g0, count, lanes, lane, shift, first, end, step;
    __device__ __forceinline__ GroupLanes(int first_group, int last_group) {
        g0 = first_group;
        count = last_group - first_group + 1;
        shift = 5;
        while (shift > 0 && (count << shift) > kTileThreads) --shift;
        lanes = 1 << shift;
        lane = threadIdx.x & (lanes - 1);
        step = kTileThreads >> shift;
        first = threadIdx.x >> shift;
        end = (count + step - 1) / step * step;  // every thread takes every step: the sums below need all lanes
    }
    __device__ __forceinline__ int group(int k) const { return g0 + min(k, count - 1); }
    __device__ __forceinline__ bool writes(int k) const { return lane == 0 && k < count; }
    __device__ __forceinline__ float total(float x) const {
#pragma unroll 1
        for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    }
};

// f(a float pair, the number of values behind it) for this lane's pieces of group g over all tiles.
template <int V, typename F>
__device__ __forceinline__ void visit_pieces(const NormArgs &p, int n, int g, const GroupLanes &l, int blocks, F f) {
    const int D = p.C / p.G, cb0 = g * D / (kTileCols * V), cb1 = ((g + 1) * D - 1) / (kTileCols * V);
#pragma unroll 1
    for (int cb = cb0; cb <= cb1; ++cb) {
        const float2 *x = reinterpret_cast<const float2 *>(p.stat_parts) + piece_at(p, n, 0, g, cb, blocks);
        const float w = (float)(min((g + 1) * D, (cb + 1) * kTileCols * V) - max(g * D, cb * kTileCols * V));
#pragma unroll 4
        for (int tile = l.lane; tile < p.tiles; tile += l.lanes) f(x[tile], w * (float)Tile<V>::positions(p, tile));
    }
}

// Positions that a thread sums up before it moves its mean.  (A mean moved by d / count at every position stops
// moving once that is below half an ulp of it: 16384 positions of mean 1000 and deviation 0.5 were off by 60
// half-ulps.  A mean in two parts, moved once a block, is off by one.  Blocks of 8: 1 to 2 % slower; of 32: 1 % faster.)
constexpr int kStatBlock = 16;

template <typename IO, int V>
__global__ void __launch_bounds__(kTileThreads, 2) norm_tile_stats_kernel(NormArgs p) {
    __shared__ float sh_mean[kTileThreads * V], sh_m2[kTileThreads * V];
    dependent_wait();
    const Tile<V> t(p, blockIdx.x);
    const int D = p.C / p.G;
    extern __shared__ __align__(16) uint8_t ring[];
    PosStream<IO, V, 1> in(p, t, reinterpret_cast<Pack<IO, V> *>(ring));
    in.t[0] = p.x;
    using U = Unit<V>;
    constexpr int NU = kUnits<V>;
    // The mean so far is lo - neg, m2 the sum of squares about it, both of cnt positions.  A block's sums s of
    // d = x + neg and q of d^2 move the mean by t - lo, t = (cnt lo + s) / (cnt + block), and add
    // q + cnt lo^2 - (cnt + block) t^2 to m2.  It starts with the first position, so d has the size of the deviation.
    U neg[NU], lo[NU], m2[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) neg[u] = lo[u] = m2[u] = both<U>(0.f);
    float cnt = 0.f;
    in.start();
    int left = in.positions();
    if (left > 0) {
        Pack<IO, V> x[1];
        in.get(x);
        in.next();
#pragma unroll
        for (int u = 0; u < NU; ++u) neg[u] = mul(x[0].unit(u), both<U>(-1.f));
        cnt = 1.f;
        --left;
    }
    while (left > 0) {
        // (a first block of 4: about a first value far from the others, sums of 16 would lose five bits to t)
        const int block = min(left, cnt == 1.f ? kStatBlock / 4 : kStatBlock);
        left -= block;
        U s[NU], q[NU];
#pragma unroll
        for (int u = 0; u < NU; ++u) s[u] = q[u] = both<U>(0.f);
#pragma unroll 4
        for (int k = 0; k < block; ++k) {
            Pack<IO, V> x[1];
            in.get(x);
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const U d = add(x[0].unit(u), neg[u]);
                s[u] = add(s[u], d);
                q[u] = fma(d, d, q[u]);
            }
            in.next();
        }
        const U n_old = both<U>(cnt);
        cnt += (float)block;
        const U inv = both<U>(__fdividef(1.f, cnt)), minus = both<U>(-1.f);
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const U w = fma(n_old, lo[u], s[u]), t = mul(w, inv);
            m2[u] = add(m2[u], fma(mul(w, minus), t, fma(mul(n_old, lo[u]), lo[u], q[u])));
            const U at = fma(t, minus, neg[u]);                // minus the new mean, rounded,
            lo[u] = add(t, fma(neg[u], minus, at));            // and what it lacks
            neg[u] = at;
        }
    }
    const int width = t.c1 - t.c0, n = t.s1 - t.s0;
    if (t.live) {
        float *mean_to = sh_mean + t.rl * width + t.col * V, *m2_to = sh_m2 + t.rl * width + t.col * V;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            if constexpr (V == 1) {
                mean_to[0] = -neg[0];
                m2_to[0] = m2[0];
            } else {
                mean_to[2 * u] = -first(neg[u]);
                mean_to[2 * u + 1] = -second(neg[u]);
                m2_to[2 * u] = first(m2[u]);
                m2_to[2 * u + 1] = second(m2[u]);
            }
        }
    }
    __syncthreads();
    // The results of a group piece's channels and row lanes are merged by their mean and the sum of squares about
    // it: two short sums, of differences from the first of them, so that equal values have exactly their mean.
    const GroupLanes l(t.first_group(D), t.last_group(D));
    const int per = n / t.RL, more = n - per * t.RL;  // positions of a row lane, and how many lanes have one more
    for (int k = l.first; k < l.end; k += l.step) {
        const int g = l.group(k);
        const int a = max(g * D, t.c0) - t.c0, w = min((g + 1) * D, t.c1) - t.c0 - a;
        const int r0 = l.lane / w, c0 = l.lane - r0 * w, dr = l.lanes / w, dc = l.lanes - dr * w;
        auto visit = [&](auto f) {
#pragma unroll 2
            for (int r = r0, c = c0; r < t.RL;) {
                f(r * width + a + c, (float)(per + (r < more)));
                r += dr;
                c += dc;
                if (c >= w) {
                    c -= w;
                    ++r;
                }
            }
        };
        const float m0 = sh_mean[a];
        float sum = 0.f, sq = 0.f;
        visit([&](int e, float cnt) { sum = fmaf(cnt, sh_mean[e] - m0, sum); });
        const float mean = m0 + __fdividef(l.total(sum), (float)w * (float)n);
        visit([&](int e, float cnt) {
            const float d = sh_mean[e] - mean;
            sq += fmaf(cnt * d, d, sh_m2[e]);
        });
        sq = l.total(sq);
        if (l.writes(k)) reinterpret_cast<float2 *>(p.stat_parts)[piece_at(p, t.n, t.tile, g, t.cb, gridDim.y)] = make_float2(mean, sq);
    }
}

template <typename IO, int V, int MODE>
__global__ void __launch_bounds__(kTileThreads, 2) norm_tile_apply_kernel(NormArgs p) {
    __shared__ float sh_mean[kTileCols * V], sh_rstd[kTileCols * V];
    const Tile<V> t(p, blockIdx.x);
    const int D = p.C / p.G, g0 = t.first_group(D);
    extern __shared__ __align__(16) uint8_t ring[];
    PosStream<IO, V, 2> in(p, t, reinterpret_cast<Pack<IO, V> *>(ring));
    in.t[0] = p.x;
    in.t[1] = mode_gate<MODE>(p) ? p.gate : nullptr;
    in.start();
    using U = Unit<V>;
    constexpr int NU = kUnits<V>;
    float w[V];
    U scale[NU], shift[NU];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = p.weight && t.live ? p.weight[t.c0 + t.col * V + i] : 1.f;
#pragma unroll
    for (int u = 0; u < NU; ++u) shift[u] = channel_unit<V>(t.live ? p.bias : nullptr, t.c0 + t.col * V + 2 * u, 0.f);
    dependent_wait();
    const GroupLanes l(g0, t.last_group(D));
    const float count = (float)D * (float)p.S;
    for (int k = l.first; k < l.end; k += l.step) {
        const int g = l.group(k);
        const float m0 = p.stat_parts[2 * piece_at(p, t.n, 0, g, g * D / (kTileCols * V), gridDim.y)];
        float sum = 0.f, sq = 0.f;
        visit_pieces<V>(p, t.n, g, l, gridDim.y, [&](const float2 &x, float n) { sum = fmaf(n, x.x - m0, sum); });
        const float mean = m0 + __fdividef(l.total(sum), count);
        visit_pieces<V>(p, t.n, g, l, gridDim.y, [&](const float2 &x, float n) {
            const float d = x.x - mean;
            sq += fmaf(n * d, d, x.y);
        });
        const float rstd = rsqrtf(__fdividef(l.total(sq), count) + p.eps);
        if (l.writes(k)) {
            sh_mean[g - g0] = mean;
            sh_rstd[g - g0] = rstd;
            if (t.tile == 0 && g * D >= t.c0) {  // the block with the group's first channel
                if (p.mean) p.mean[(long long)t.n * p.G + g] = mean;
                if (p.rstd) p.rstd[(long long)t.n * p.G + g] = rstd;
            }
        }
    }
    __syncthreads();
    if (!t.live) return;
    int g = (t.c0 + t.col * V) / D;
    U neg[NU];  // z = (x + neg) scale + shift
    float m[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (t.c0 + t.col * V + i >= (g + 1) * D) ++g;
        m[i] = -sh_mean[g - g0];
        w[i] *= sh_rstd[g - g0];
    }
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        neg[u] = unit_of<V>(m, u);
        scale[u] = unit_of<V>(w, u);
    }
    for (; in.more(); in.next()) {
        Pack<IO, V> x[2], y;
        in.get(x);
#pragma unroll
        for (int u = 0; u < NU; ++u) y.set(u, y_of<IO, MODE>(p, fma(add(x[0].unit(u), neg[u]), scale[u], shift[u]), x[1].unit(u)));
        store_pack<IO, V>(p.y, in.at, y);
    }
}

// What the backward pass needs of a thread's channels, the first of them in group g.
template <int V>
__device__ __forceinline__ void norm_params(const NormArgs &p, const Tile<V> &t, int g, float (&mean)[V], float (&rstd)[V], float (&w)[V],
                                            float (&b)[V]) {
    const int D = p.C / p.G;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = t.c0 + t.col * V + i;
        if (c >= (g + 1) * D) ++g;
        const bool in = t.live;
        mean[i] = in ? p.mean[(long long)t.n * p.G + g] : 0.f;
        rstd[i] = in ? p.rstd[(long long)t.n * p.G + g] : 0.f;
        w[i] = in && p.weight ? p.weight[c] : 1.f;
        b[i] = in && p.bias ? p.bias[c] : 0.f;
    }
}

// First kernel of the backward pass: per channel sum dz and sum dz xh over the tile, and their sums over
// each group piece with the weights.  A block takes every gridDim.x-th tile of all samples and keeps its
// channels' totals, so that the parts of dweight and dbias stay few.
template <typename IO, int V, int MODE>
__global__ void __launch_bounds__(kTileThreads, 2) norm_tile_grad_sums_kernel(NormArgs p) {
    __shared__ float sh1[kTileThreads * V], sh2[kTileThreads * V];
    __shared__ float tot1[kTileCols * V], tot2[kTileCols * V];
    extern __shared__ __align__(16) uint8_t ring[];
    const int D = p.C / p.G;
    dependent_wait();
    for (int i = threadIdx.x; i < kTileCols * V; i += kTileThreads) tot1[i] = tot2[i] = 0.f;
    for (int unit = blockIdx.x; unit < p.N * p.tiles; unit += gridDim.x) {
        const Tile<V> t(p, unit);
        const int width = t.c1 - t.c0;
        PosStream<IO, V, 3> in(p, t, reinterpret_cast<Pack<IO, V> *>(ring));
        in.t[0] = p.x;
        in.t[1] = p.dy;
        in.t[2] = mode_gate<MODE>(p) ? p.gate : nullptr;
        in.start();
        __syncthreads();
        if (t.live) {
            float mean[V], rstd[V], w[V], b[V], sz[V] = {}, szx[V] = {};
            norm_params<V>(p, t, (t.c0 + t.col * V) / D, mean, rstd, w, b);
            for (; in.more(); in.next()) {
                Pack<IO, V> x[3];
                in.get(x);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = (x[0].at(i) - mean[i]) * rstd[i];
                    float dg;
                    const float dz = dz_of<IO, MODE>(p, fmaf(xh, w[i], b[i]), x[1].at(i), x[2].at(i), dg);
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
        for (int c = threadIdx.x; c < width; c += kTileThreads) {
            float a = 0.f, b = 0.f;
            for (int r = 0; r < t.RL; ++r) {
                a += sh1[r * width + c];
                b += sh2[r * width + c];
            }
            tot1[c] += a;
            tot2[c] += b;
            const float w = p.weight ? p.weight[t.c0 + c] : 1.f;
            sh1[c] = a * w;  // row lane 0's place, which only this thread reads
            sh2[c] = b * w;
        }
        __syncthreads();
        const GroupLanes l(t.first_group(D), t.last_group(D));
        for (int k = l.first; k < l.end; k += l.step) {
            const int g = l.group(k);
            const int a = max(g * D, t.c0) - t.c0, b = min((g + 1) * D, t.c1) - t.c0;
            float s1 = 0.f, s2 = 0.f;
#pragma unroll 2
            for (int c = a + l.lane; c < b; c += l.lanes) {
                s1 += sh1[c];
                s2 += sh2[c];
            }
            s1 = l.total(s1);
            s2 = l.total(s2);
            if (l.writes(k)) reinterpret_cast<float2 *>(p.stat_parts)[piece_at(p, t.n, t.tile, g, t.cb, gridDim.y)] = make_float2(s1, s2);
        }
    }
    if (!p.chan_parts) return;
    const int c0 = blockIdx.y * kTileCols * V, width = min(kTileCols * V, p.C - c0);
    float *chan = p.chan_parts + (long long)blockIdx.x * 2 * p.C + c0;
    for (int c = threadIdx.x; c < width; c += kTileThreads) {  // each thread its own totals
        chan[c] = tot1[c];
        chan[p.C + c] = tot2[c];
    }
}

template <typename IO, int V, int MODE>
__global__ void __launch_bounds__(kTileThreads, 2) norm_tile_grad_apply_kernel(NormArgs p) {
    __shared__ float sh1[kTileCols * V], sh2[kTileCols * V];
    const Tile<V> t(p, blockIdx.x);
    const int D = p.C / p.G, g0 = t.first_group(D);
    extern __shared__ __align__(16) uint8_t ring[];
    PosStream<IO, V, 3> in(p, t, reinterpret_cast<Pack<IO, V> *>(ring));
    in.t[0] = p.x;
    in.t[1] = p.dy;
    in.t[2] = mode_gate<MODE>(p) ? p.gate : nullptr;
    in.start();
    const int g_first = (t.c0 + t.col * V) / D;
    float mean[V], rstd[V], w[V], b[V], s1[V], s2[V];
    norm_params<V>(p, t, g_first, mean, rstd, w, b);
    dependent_wait();
    const float inv = 1.f / ((float)D * (float)p.S);
    const GroupLanes l(g0, t.last_group(D));
    for (int k = l.first; k < l.end; k += l.step) {
        const int g = l.group(k);
        float a = 0.f, b = 0.f;
        visit_pieces<V>(p, t.n, g, l, gridDim.y, [&](const float2 &x, float) {
            a += x.x;
            b += x.y;
        });
        a = l.total(a);
        b = l.total(b);
        if (l.writes(k)) {
            sh1[g - g0] = a * inv;
            sh2[g - g0] = b * inv;
        }
    }
    __syncthreads();
    if (!t.live) return;
    int g = g_first;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (t.c0 + t.col * V + i >= (g + 1) * D) ++g;
        s1[i] = sh1[g - g0];
        s2[i] = sh2[g - g0];
    }
    for (; in.more(); in.next()) {
        Pack<IO, V> x[3], dgv, dxv;
        in.get(x);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float xh = (x[0].at(i) - mean[i]) * rstd[i];
            float dg;
            const float dz = dz_of<IO, MODE>(p, fmaf(xh, w[i], b[i]), x[1].at(i), x[2].at(i), dg);
            st_io(dxv.v, i, rstd[i] * (fmaf(dz, w[i], -s1[i]) - xh * s2[i]));
            st_io(dgv.v, i, dg);
        }
        store_pack<IO, V>(p.dx, in.at, dxv);
        if (mode_gate<MODE>(p)) store_pack<IO, V>(p.dgate, in.at, dgv);
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
        pl.LG = 4;
        while (pl.LG < nv && pl.LG < 32) pl.LG *= 2;
        pl.K = nv <= 32 && pl.V > 1 ? 1 : kRowVecs;
        const long long per_block = kRowThreads / pl.LG;
        long long lanes = std::max<long long>(1, (long long)sms * (pl.K > 1 ? 1 : backward ? kRowBwdBlocks : kRowFwdBlocks) * per_block / s.G);
        lanes = std::min<long long>(lanes, std::max(1, s.N));
        pl.row_lanes = (int)lanes;
        pl.blocks = (int)((lanes * s.G + per_block - 1) / per_block);
        return pl;
    }
    pl.V = s.C % full == 0 ? full : 1;
    pl.col_blocks = (s.C / pl.V + kTileCols - 1) / kTileCols;
    const long long others = std::max(1LL, (long long)s.N * pl.col_blocks);
    pl.tiles = (int)std::max<long long>(1, std::min<long long>((2LL * sms + others - 1) / others, s.S / 16));
    return pl;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t stat_bytes(const prism_norm_shape &s, const NormPlan &pl) {
    return pl.rows ? 0 : align256((size_t)s.N * pl.tiles * norm_pieces(s.G, pl.col_blocks) * 8);
}
int chan_parts(const prism_norm_shape &s, const NormPlan &pl) {
    return pl.rows ? pl.row_lanes : (int)std::min<long long>((long long)s.N * pl.tiles, 2LL * sm_count());
}

prism_status check_shape(const prism_norm_shape *s) {
    if (!s) return PRISM_ERR_INVALID_ARG;
    if (s->N < 0 || s->S < 0 || s->C < 1 || s->G < 1 || s->C % s->G) return PRISM_ERR_INVALID_ARG;
    if (s->io != PRISM_BF16 && s->io != PRISM_F32) return PRISM_ERR_INVALID_ARG;
    if (s->act != PRISM_ACT_NONE && s->act != PRISM_ACT_SILU && s->act != PRISM_ACT_GELU) return PRISM_ERR_INVALID_ARG;
    if (!(s->eps >= 0.f)) return PRISM_ERR_INVALID_ARG;
    if (s->C > (1 << 20) || (long long)s->N * s->G > 0x7fffffffLL || s->N > (1 << 24) || s->S > (1 << 30)) return PRISM_ERR_UNSUPPORTED;
    if ((long long)s->N * s->S > (1LL << 40) / s->C) return PRISM_ERR_UNSUPPORTED;  // (sizes in bytes stay far below 2^63)
    return PRISM_OK;
}

// f(mode) with the call's activation and gate as a compile-time mode.
template <typename F>
void with_mode(const NormArgs &a, F f) {
    const bool g = a.gate != nullptr;
    switch (a.act) {
        case PRISM_ACT_SILU: g ? f(std::integral_constant<int, 3>()) : f(std::integral_constant<int, 2>()); break;
        case PRISM_ACT_GELU: g ? f(std::integral_constant<int, 5>()) : f(std::integral_constant<int, 4>()); break;
        default: g ? f(std::integral_constant<int, 1>()) : f(std::integral_constant<int, 0>()); break;
    }
}

// Launch of a tiles kernel with its stream's shared memory.
template <int BYTES, typename K>
cudaError_t launch_tiles(K kern, dim3 grid, const NormArgs &a, cudaStream_t s, bool dependent) {
    if (BYTES > 0) {
        const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
        if (err != cudaSuccess) return err;
    }
    return dependent_launch(kern, grid, kTileThreads, BYTES, s, dependent, a);
}

// f(lanes) with the plan's lanes of a group as a compile-time number.
template <typename F>
void with_lanes(int LG, F f) {
    switch (LG) {
        case 4: f(std::integral_constant<int, 4>()); break;
        case 8: f(std::integral_constant<int, 8>()); break;
        case 16: f(std::integral_constant<int, 16>()); break;
        default: f(std::integral_constant<int, 32>()); break;
    }
}

template <typename IO>
cudaError_t launch_fwd(const NormArgs &a, const NormPlan &pl, cudaStream_t s) {
    constexpr int F = 16 / sizeof(IO);
    if (pl.rows) {
        launch_probe_mark(s);
        with_lanes(pl.LG, [&](auto l) {
            if (pl.V == 1) norm_rows_fwd_kernel<IO, 1, kRowVecs, l.value, kRuntime><<<pl.blocks, kRowThreads, 0, s>>>(a, pl.row_lanes);
            else if (pl.K == 1)
                with_mode(a, [&](auto m) { norm_rows_fwd_kernel<IO, F, 1, l.value, m.value><<<pl.blocks, kRowThreads, 0, s>>>(a, pl.row_lanes); });
            else if constexpr (l.value == 32)  // (several vectors of a lane only where 32 lanes are too few)
                norm_rows_fwd_kernel<IO, F, kRowVecs, 32, kRuntime><<<pl.blocks, kRowThreads, 0, s>>>(a, pl.row_lanes);
        });
        return cudaGetLastError();
    }
    const dim3 grid(a.N * a.tiles, pl.col_blocks);
    cudaError_t err = pl.V == 1 ? launch_tiles<0>(norm_tile_stats_kernel<IO, 1>, grid, a, s, false)
                                : launch_tiles<kPosBytes<IO, F, 1>>(norm_tile_stats_kernel<IO, F>, grid, a, s, false);
    if (err != cudaSuccess) return err;
    if (pl.V == 1) err = launch_tiles<0>(norm_tile_apply_kernel<IO, 1, kRuntime>, grid, a, s, true);
    else with_mode(a, [&](auto m) { err = launch_tiles<kPosBytes<IO, F, 2>>(norm_tile_apply_kernel<IO, F, m.value>, grid, a, s, true); });
    return err;
}

template <typename IO>
cudaError_t launch_bwd(const NormArgs &a, const NormPlan &pl, float *dweight, float *dbias, cudaStream_t s) {
    constexpr int F = 16 / sizeof(IO);
    cudaError_t err = cudaSuccess;
    if (pl.rows) {
        launch_probe_mark(s);
        with_lanes(pl.LG, [&](auto l) {
            if (pl.V == 1) norm_rows_bwd_kernel<IO, 1, kRowVecs, l.value, kRuntime><<<pl.blocks, kRowThreads, 0, s>>>(a, pl.row_lanes);
            else if (pl.K == 1)
                with_mode(a, [&](auto m) { norm_rows_bwd_kernel<IO, F, 1, l.value, m.value><<<pl.blocks, kRowThreads, 0, s>>>(a, pl.row_lanes); });
            else if constexpr (l.value == 32)  // (several vectors of a lane only where 32 lanes are too few)
                norm_rows_bwd_kernel<IO, F, kRowVecs, 32, kRuntime><<<pl.blocks, kRowThreads, 0, s>>>(a, pl.row_lanes);
        });
    } else {
        const dim3 grid(a.N * a.tiles, pl.col_blocks);
        const dim3 some(a.parts, pl.col_blocks);
        if (pl.V == 1) err = launch_tiles<0>(norm_tile_grad_sums_kernel<IO, 1, kRuntime>, some, a, s, false);
        else with_mode(a, [&](auto m) { err = launch_tiles<kPosBytes<IO, F, 3>>(norm_tile_grad_sums_kernel<IO, F, m.value>, some, a, s, false); });
        if (err != cudaSuccess) return err;
        if (pl.V == 1) err = launch_tiles<0>(norm_tile_grad_apply_kernel<IO, 1, kRuntime>, grid, a, s, true);
        else with_mode(a, [&](auto m) { err = launch_tiles<kPosBytes<IO, F, 3>>(norm_tile_grad_apply_kernel<IO, F, m.value>, grid, a, s, true); });
    }
    if (err == cudaSuccess) err = cudaGetLastError();
    if (err == cudaSuccess && (dweight || dbias))
        err = dependent_launch(norm_channel_sum_kernel, dim3((2 * a.C + 31) / 32), 1024, 0, s, true, (const float *)a.chan_parts, a.parts,
                               a.C, dweight, dbias);
    return err;
}

NormArgs args_of(const prism_norm_shape &s, const NormPlan &pl, const void *x, const float *weight, const float *bias,
                 const void *gate) {
    NormArgs a{};
    a.N = s.N; a.S = s.S; a.C = s.C; a.G = s.G; a.act = s.act; a.eps = s.eps;
    a.x = x; a.gate = gate; a.weight = weight; a.bias = bias;
    a.tiles = pl.tiles;
    if (pl.tiles > 0) {
        a.tile_len = s.S / pl.tiles;
        a.tile_more = s.S % pl.tiles;
    }
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
    *bytes = shape->N == 0 || shape->S == 0 ? 0 : stat_bytes(*shape, plan_of(*shape, false));
    return PRISM_OK;
}

prism_status prism_group_norm_fwd(const prism_norm_shape *shape, const void *x, const float *weight, const float *bias,
                                  const void *gate, void *y, float *mean, float *rstd, void *workspace, size_t ws_bytes,
                                  void *stream) {
    const prism_status st = check_shape(shape);
    if (st != PRISM_OK) return st;
    const prism_norm_shape &s = *shape;
    const size_t n = (size_t)s.N * s.S * s.C * (s.io == PRISM_F32 ? 4 : 2), groups = (size_t)s.N * s.G * 4;
    if (!aligned4(weight) || !aligned4(bias) || !aligned4(mean) || !aligned4(rstd)) return PRISM_ERR_INVALID_ARG;
    if (n == 0) {  // statistics over no positions: NaN (every byte 255)
        cudaError_t err = cudaSuccess;
        if (mean && groups > 0) err = cudaMemsetAsync(mean, 255, groups, (cudaStream_t)stream);
        if (rstd && groups > 0 && err == cudaSuccess) err = cudaMemsetAsync(rstd, 255, groups, (cudaStream_t)stream);
        return cuda_status(err);
    }
    if (!x || !y || !aligned16(x) || !aligned16(y) || !aligned16(gate)) return PRISM_ERR_INVALID_ARG;
    const NormPlan pl = plan_of(s, false);
    const size_t need = stat_bytes(s, pl);
    if (need > 0 && (!workspace || ws_bytes < need || ((uintptr_t)workspace & 255u))) return PRISM_ERR_INVALID_ARG;
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
    if (!dweight && !dbias) a.chan_parts = nullptr;
    const cudaError_t err = s.io == PRISM_F32 ? launch_bwd<float>(a, pl, dweight, dbias, (cudaStream_t)stream)
                                              : launch_bwd<__nv_bfloat16>(a, pl, dweight, dbias, (cudaStream_t)stream);
    probe_finish((cudaStream_t)stream);
    return cuda_status(err);
}

}  // extern "C"
