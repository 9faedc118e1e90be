// decay_simt.cu -- the decay scan's kernels on CUDA cores, in fp32 throughout (decay.cuh has the
// formulas): the segment sums and the pass over the tokens for fp32 operands, the carry between
// segments and the sum of shared heads' gradients for both types.

#include "decay.cuh"
#include "f32x2.cuh"

namespace prism {
namespace {

constexpr int CH = kDecayChunkSimt;  // tokens of a chunk
constexpr int NT = 256;              // 16 x 16 threads

// Tile rows [t0, t0 + CH) of one head into shared memory by asynchronous copies, zero beyond `len` tokens and
// beyond the operand's own width d (tiles are D = 64 or 128 columns wide, rows D + 4 floats apart: 16-byte
// aligned, and 16 rows read at one column fall into different banks).
template <int D>
__device__ __forceinline__ void request_tile(float *dst, const DecayTensor &x, int b, int h, int t0, int len, int d) {
    const float *src = (const float *)x.p + b * x.sb + (long long)(h / x.div) * x.sh;
    for (int e = threadIdx.x; e < CH * (D / 4); e += NT) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4;  // (d is a multiple of 32)
        const bool in = t0 + r < len && c < d;
        const float *from = in ? src + (long long)(t0 + r) * x.st + c : src;
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst + r * (D + 4) + c);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
    }
}
__device__ __forceinline__ void request_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // all requests but the N latest have landed (this thread's)
__device__ __forceinline__ void request_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Two rows of four floats as four packed pairs.
__device__ __forceinline__ void lds4(const float *p, F2 (&v)[2]) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(p);
    v[0] = x.x;
    v[1] = x.y;
}

// acc[r][c] += sum_j w_j Y[j][m0 + r] Z[j][n0 + c]: a thread's tile of the state, m along y, n along z
// (4 consecutive columns out of every 64; pairs of columns packed).
template <int D1, int D2>
__device__ __forceinline__ void state_tile(const float *Y, const float *Z, const float *w, F2 (&acc)[D1 / 16][D2 / 32]) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 4
    for (int j = 0; j < CH; ++j) {
        const F2 ww = pack2(w[j], w[j]);
        F2 z[D2 / 64][2];
#pragma unroll
        for (int i = 0; i < D2 / 64; ++i) {
            lds4(Z + j * (D2 + 4) + 64 * i + 4 * tx, z[i]);
            z[i][0] = mul(z[i][0], ww);
            z[i][1] = mul(z[i][1], ww);
        }
#pragma unroll
        for (int i = 0; i < D1 / 64; ++i) {
            const float4 y = *reinterpret_cast<const float4 *>(Y + j * (D1 + 4) + 64 * i + 4 * ty);
            const float yf[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const F2 yy = pack2(yf[r], yf[r]);
#pragma unroll
                for (int c = 0; c < D2 / 32; ++c) acc[4 * i + r][c] = fma(yy, z[c >> 1][c & 1], acc[4 * i + r][c]);
            }
        }
    }
}

// o[r][c] += sum over k in [K0, K1) of A[row r][k] B[k][n0 + c], rows ty + 16 r of A (pitch pa), R0 <= r < R1.
template <int D2, int R0, int R1>
__device__ __forceinline__ void rows_range(const float *A, int pa, const float *B, int K0, int K1, F2 (&o)[4][D2 / 32]) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 4
    for (int k0 = K0; k0 < K1; k0 += 4) {
        float4 a[4];
#pragma unroll
        for (int r = R0; r < R1; ++r) a[r] = *reinterpret_cast<const float4 *>(A + (ty + 16 * r) * pa + k0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            F2 b[D2 / 64][2];
#pragma unroll
            for (int i = 0; i < D2 / 64; ++i) lds4(B + (k0 + k) * (D2 + 4) + 64 * i + 4 * tx, b[i]);
#pragma unroll
            for (int r = R0; r < R1; ++r) {
                const float x = (&a[r].x)[k];
                const F2 xx = pack2(x, x);
#pragma unroll
                for (int c = 0; c < D2 / 32; ++c) o[r][c] = fma(xx, b[c >> 1][c & 1], o[r][c]);
            }
        }
    }
}

// The chunk's own part of a pass: P[i][j] = a^|i-j| x_i . y_j on the causal side, rows i = ty + 16 r, columns
// j = tx + 16 c.  Of the 16 x 16 blocks those on the other side are skipped, here and in P Z: 6 of 16.
// (REV: the causal side is j >= i.)
template <int D1, bool REV>
__device__ __forceinline__ void scores(const float *X, const float *Y, const float *pw, float *P) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    F2 s2[4][4] = {};  // sums over even and odd columns
#pragma unroll 4
    for (int d = 0; d < D1; d += 4) {
        F2 xv[4][2], yv[4][2];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            lds4(X + (ty + 16 * r) * (D1 + 4) + d, xv[r]);
            lds4(Y + (tx + 16 * r) * (D1 + 4) + d, yv[r]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = REV ? r : 0; c < (REV ? 4 : r + 1); ++c) s2[r][c] = fma(xv[r][0], yv[c][0], fma(xv[r][1], yv[c][1], s2[r][c]));
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = REV ? r : 0; c < (REV ? 4 : r + 1); ++c) {
            const int i = ty + 16 * r, j = tx + 16 * c, gap = REV ? j - i : i - j;
            P[i * (CH + 4) + j] = gap >= 0 ? total(s2[r][c]) * pw[gap] : 0.f;
        }
}
template <int D2, bool REV>
__device__ __forceinline__ void causal_rows(const float *P, const float *Z, F2 (&o)[4][D2 / 32]) {
    constexpr int PP = CH + 4;
    if constexpr (REV) {
        rows_range<D2, 0, 1>(P, PP, Z, 0, 16, o);
        rows_range<D2, 0, 2>(P, PP, Z, 16, 32, o);
        rows_range<D2, 0, 3>(P, PP, Z, 32, 48, o);
        rows_range<D2, 0, 4>(P, PP, Z, 48, 64, o);
    } else {
        rows_range<D2, 0, 4>(P, PP, Z, 0, 16, o);
        rows_range<D2, 1, 4>(P, PP, Z, 16, 32, o);
        rows_range<D2, 2, 4>(P, PP, Z, 32, 48, o);
        rows_range<D2, 3, 4>(P, PP, Z, 48, 64, o);
    }
}

// Floats of the chunk buffers (one set of tiles each) and of what follows them.  The next chunk's tiles are
// requested before the current one's products, where two sets fit (all widths but 128 x 128 of the pass).
template <int D1, int D2>
struct SumSizes {
    static constexpr int SET = CH * (D1 + 4) + CH * (D2 + 4), NB = 2;
    static constexpr int TOTAL = NB * SET + (CH + 1) + CH;
};
template <int D1, int D2>
struct PassSizes {
    static constexpr int SET = 2 * CH * (D1 + 4) + CH * (D2 + 4);
    static constexpr int REST = D1 * (D2 + 4) + CH * (CH + 4) + (CH + 1) + CH;
    static constexpr int NB = 4 * (2 * SET + REST) <= 227 * 1024 ? 2 : 1;
    static constexpr int TOTAL = NB * SET + REST;
    static_assert(4 * TOTAL <= 227 * 1024, "shared memory budget");
};

// Column of the register tile's index i along y or z.
__device__ __forceinline__ int tile_col(int i, int t) { return 64 * (i >> 2) + 4 * t + (i & 3); }

// Weight of token j of a chunk with n valid ones in the state that leaves the chunk.
__device__ __forceinline__ int write_exponent(int j, int n, int reverse) { return reverse ? j + 1 : n - 1 - j; }

// F[n][m] of one segment: the state that its tokens alone leave behind.
template <int D1, int D2>
__global__ void __launch_bounds__(NT) decay_sum_simt_kernel(const __grid_constant__ DecayPassSet set) {
    extern __shared__ __align__(16) float sm[];
    using SZ = SumSizes<D1, D2>;
    float *pw = sm + SZ::NB * SZ::SET, *w = pw + CH + 1;
    dependent_wait();
    const DecayPass &p = set.p[blockIdx.x / set.p[0].nseg];
    const int seg = blockIdx.x % p.nseg, h = blockIdx.y, b = blockIdx.z;
    const int len = decay_len(p.lengths, b, p.T);
    const int s0 = seg * p.seg_tokens;
    const int s1 = min(s0 + p.seg_tokens, len);
    const float a = p.decay[h];
    F2 acc[D1 / 16][D2 / 32] = {};
    const int nch = s1 > s0 ? (s1 - s0 + CH - 1) / CH : 0;
    auto token = [&](int cc) { return s0 + (p.reverse ? nch - 1 - cc : cc) * CH; };
    auto request = [&](int cc) {
        float *Y = sm + (cc % SZ::NB) * SZ::SET;
        request_tile<D1>(Y, p.y, b, h, token(cc), len, p.d1);
        request_tile<D2>(Y + CH * (D1 + 4), p.z, b, h, token(cc), len, p.d2);
        request_commit();
    };
    if (nch > 0) request(0);
    for (int i = threadIdx.x; i <= CH; i += NT) pw[i] = decay_pow(a, i);
    for (int cc = 0; cc < nch; ++cc) {
        const int n = min(CH, s1 - token(cc));
        const float *Y = sm + (cc % SZ::NB) * SZ::SET, *Z = Y + CH * (D1 + 4);
        __syncthreads();  // the chunk before is done with
        if (cc + 1 < nch) {
            request(cc + 1);
            request_wait<1>();
        } else {
            request_wait<0>();
        }
        for (int j = threadIdx.x; j < CH; j += NT) w[j] = j < n ? pw[write_exponent(j, n, p.reverse)] : 0.f;
        const F2 an = pack2(pw[n], pw[n]);
#pragma unroll
        for (int r = 0; r < D1 / 16; ++r)
#pragma unroll
            for (int c = 0; c < D2 / 32; ++c) acc[r][c] = mul(acc[r][c], an);
        __syncthreads();
        state_tile<D1, D2>(Y, Z, w, acc);
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float *F = p.F + (((long long)b * p.H + h) * p.nseg + seg) * p.d1 * p.d2;
#pragma unroll
    for (int r = 0; r < D1 / 16; ++r) {
        const int m = tile_col(r, ty);
#pragma unroll
        for (int c = 0; c < D2 / 16; ++c) {
            const int n = tile_col(c, tx);
            if (m < p.d1 && n < p.d2) F[n * p.d1 + m] = c & 1 ? second(acc[r][c >> 1]) : first(acc[r][c >> 1]);
        }
    }
}

// One segment's outputs, chunk by chunk, the state in shared memory (R^T: rows along y, so that the
// entry term X R^T reads like the P Z product).
template <int D1, int D2>
__global__ void __launch_bounds__(NT) decay_pass_simt_kernel(const __grid_constant__ DecayPassSet set) {
    extern __shared__ __align__(16) float sm[];
    using SZ = PassSizes<D1, D2>;
    float *R = sm + SZ::NB * SZ::SET, *P = R + D1 * (D2 + 4), *pw = P + CH * (CH + 4), *w = pw + CH + 1;
    const DecayPass &p = set.p[blockIdx.x / set.p[0].nseg];
    const int seg = blockIdx.x % p.nseg, h = blockIdx.y, b = blockIdx.z;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int len = decay_len(p.lengths, b, p.T);
    const int s0 = seg * p.seg_tokens;
    const int send = min(s0 + p.seg_tokens, p.T), s1 = min(send, len);
    const float a = p.decay[h];
    const int nch = s1 > s0 ? (s1 - s0 + CH - 1) / CH : 0;
    auto token = [&](int cc) { return s0 + (p.reverse ? nch - 1 - cc : cc) * CH; };
    auto request = [&](int cc) {
        float *X = sm + (cc % SZ::NB) * SZ::SET;
        request_tile<D1>(X, p.x, b, h, token(cc), len, p.d1);
        request_tile<D1>(X + CH * (D1 + 4), p.y, b, h, token(cc), len, p.d1);
        request_tile<D2>(X + 2 * CH * (D1 + 4), p.z, b, h, token(cc), len, p.d2);
        request_commit();
    };
    if (SZ::NB == 2 && nch > 0) request(0);
    for (int i = threadIdx.x; i <= CH; i += NT) pw[i] = decay_pow(a, i);
    // (the entry state comes from the call's previous kernel; all that was read so far is older than the call)
    dependent_wait();
    const float *E = p.entry ? p.entry + (((long long)b * p.H + h) * p.nseg + seg) * p.d1 * p.d2 : nullptr;
#pragma unroll 4
    for (int e = threadIdx.x; e < D1 * D2 / 4; e += NT) {  // four values of one row of R at a time
        // rows of E along z (m * d2 + n): n fastest; along y (n * d1 + m): m fastest
        const int m = p.entry_t ? e / (D2 / 4) : e % D1, n = 4 * (p.entry_t ? e % (D2 / 4) : e / D1);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (E && m < p.d1 && n < p.d2) {  // (widths are multiples of 32)
            if (p.entry_t) x = *reinterpret_cast<const float4 *>(E + m * p.d2 + n);
            else x = make_float4(E[n * p.d1 + m], E[(n + 1) * p.d1 + m], E[(n + 2) * p.d1 + m], E[(n + 3) * p.d1 + m]);
        }
        *reinterpret_cast<float4 *>(R + m * (D2 + 4) + n) = x;
    }
    for (int cc = 0; cc < nch; ++cc) {
        const int t0 = token(cc), n = min(CH, s1 - t0);
        const float *X = sm + (cc % SZ::NB) * SZ::SET, *Y = X + CH * (D1 + 4), *Z = Y + CH * (D1 + 4);
        __syncthreads();  // the chunk before is done with
        if (SZ::NB == 1) request(cc);
        if (SZ::NB == 2 && cc + 1 < nch) {
            request(cc + 1);
            request_wait<1>();
        } else {
            request_wait<0>();
        }
        for (int j = threadIdx.x; j < CH; j += NT) w[j] = j < n ? pw[write_exponent(j, n, p.reverse)] : 0.f;
        __syncthreads();
        if (p.reverse) scores<D1, true>(X, Y, pw, P);
        else scores<D1, false>(X, Y, pw, P);
        __syncthreads();
        F2 o[4][D2 / 32] = {};
        // entry term, then scaled by its row's decay, then the chunk's own
        rows_range<D2, 0, 4>(X, D1 + 4, R, 0, D1, o);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = ty + 16 * r;
            const float f = i < n ? pw[p.reverse ? n - 1 - i : i + 1] : 0.f;
#pragma unroll
            for (int c = 0; c < D2 / 32; ++c) o[r][c] = mul(o[r][c], pack2(f, f));
        }
        if (p.reverse) causal_rows<D2, true>(P, Z, o);
        else causal_rows<D2, false>(P, Z, o);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = ty + 16 * r;
            if (i >= n) continue;
#pragma unroll
            for (int c = 0; c < D2 / 64; ++c) {
                const int col = 64 * c + 4 * tx;
                if (col < p.d2)
                    *reinterpret_cast<ulonglong2 *>((float *)p.o + (((long long)b * p.T + t0 + i) * p.H + h) * p.d2 + col) =
                        make_ulonglong2(o[r][2 * c], o[r][2 * c + 1]);
            }
        }
        if (cc + 1 < nch) {
            F2 acc[D1 / 16][D2 / 32] = {};
            state_tile<D1, D2>(Y, Z, w, acc);
            __syncthreads();  // every thread has read R for its outputs
            const F2 an = pack2(pw[n], pw[n]);
#pragma unroll
            for (int r = 0; r < D1 / 16; ++r)
#pragma unroll
                for (int c = 0; c < D2 / 32; ++c) {
                    F2 &x = *reinterpret_cast<F2 *>(R + tile_col(r, ty) * (D2 + 4) + tile_col(2 * c, tx));
                    x = fma(an, x, acc[r][c]);
                }
        }
    }
    // rows behind the sequence's last token
    const int z0 = max(s0, s1);
    for (long long e = threadIdx.x; e < (long long)(send - z0) * p.d2; e += NT) ((float *)p.o)[(((long long)b * p.T + z0 + e / p.d2) * p.H + h) * p.d2 + e % p.d2] = 0.f;
}

template <int D1, int D2>
cudaError_t launch_one(const DecayPassSet &set, bool sum, cudaStream_t s) {
    const DecayPass &p = set.p[0];
    const int bytes = 4 * (sum ? SumSizes<D1, D2>::TOTAL : PassSizes<D1, D2>::TOTAL);
    auto kern = sum ? decay_sum_simt_kernel<D1, D2> : decay_pass_simt_kernel<D1, D2>;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != cudaSuccess) return err;
    return dependent_launch(kern, dim3(set.count * p.nseg, p.H, p.B), NT, bytes, s, set.dependent, set);
}

// Four state elements per thread, walked over the segments in order: entry states replace the sums.  The
// sums do not depend on the walk: kAhead of them are loaded at a time.  The two powers a block needs (of a
// whole segment and of the one that the sequence ends in) are taken once, in 64 bits; taken by every
// thread they were the kernel's time (32 us instead of 6 for 16 heads of 65536 tokens).
constexpr int kAhead = 8;

__global__ void __launch_bounds__(128) decay_carry_kernel(const __grid_constant__ DecayCarry c) {
    dependent_wait();
    const DecayCarryOne &o = c.c[blockIdx.z];
    __shared__ float pw[2];
    const int bh = blockIdx.x, e = 4 * (blockIdx.y * 128 + threadIdx.x);
    const int len = decay_len(c.lengths, bh / c.H, c.T);
    const int last = len / c.seg_tokens, rest = len % c.seg_tokens;  // segment `last` has `rest` tokens
    if (threadIdx.x < 2) pw[threadIdx.x] = decay_pow(c.decay[bh % c.H], threadIdx.x == 0 ? c.seg_tokens : rest);
    __syncthreads();
    if (e >= c.elems) return;
    float4 *F = reinterpret_cast<float4 *>(o.F + (long long)bh * c.nseg * c.elems + e);
    const long long step = c.elems / 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (o.init) s = *reinterpret_cast<const float4 *>(o.init + (long long)bh * c.elems + e);
    for (int i0 = 0; i0 < c.nseg; i0 += kAhead) {
        float4 f[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i0 + k < c.nseg) f[k] = F[(o.reverse ? c.nseg - 1 - i0 - k : i0 + k) * step];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i0 + k >= c.nseg) break;
            const int seg = o.reverse ? c.nseg - 1 - i0 - k : i0 + k;
            F[seg * step] = s;
            if (seg < last || (seg == last && rest > 0)) {
                const float a = pw[seg == last];
                s = make_float4(fmaf(a, s.x, f[k].x), fmaf(a, s.y, f[k].y), fmaf(a, s.z, f[k].z), fmaf(a, s.w, f[k].w));
            }
        }
    }
    if (o.final_state) *reinterpret_cast<float4 *>(o.final_state + (long long)bh * c.elems + e) = s;
}

template <typename IO>
__global__ void decay_group_sum_kernel(const __grid_constant__ DecayGroupSum a) {
    dependent_wait();
    const int which = blockIdx.y, d = a.d[which], div = a.div;
    const float *part = a.part[which];
    IO *out = (IO *)a.out[which];
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;  // over [groups, d / 4]
    if (i >= a.groups * (d / 4)) return;
    const long long g = i / (d / 4);
    const int c = (int)(i % (d / 4)) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < div; ++k) {
        const float4 x = *reinterpret_cast<const float4 *>(part + (g * div + k) * d + c);
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    st_io(out, g * d + c, s.x);
    st_io(out, g * d + c + 1, s.y);
    st_io(out, g * d + c + 2, s.z);
    st_io(out, g * d + c + 3, s.w);
}

}  // namespace

cudaError_t launch_decay_simt(const DecayPassSet &set, bool sum, cudaStream_t s) {
    const int d1 = decay_padded(set.p[0].d1), d2 = decay_padded(set.p[0].d2);
    if (d1 == 64) return d2 == 64 ? launch_one<64, 64>(set, sum, s) : launch_one<64, 128>(set, sum, s);
    return d2 == 64 ? launch_one<128, 64>(set, sum, s) : launch_one<128, 128>(set, sum, s);
}

cudaError_t launch_decay_carry(const DecayCarry &c, cudaStream_t s) {
    return dependent_launch(decay_carry_kernel, dim3(c.BH, (c.elems + 511) / 512, c.count), 128, 0, s, c.dependent, c);
}

cudaError_t launch_decay_group_sum(const DecayGroupSum &g, bool io_f32, cudaStream_t s) {
    const int d = g.d[0] > g.d[1] ? g.d[0] : g.d[1];
    const dim3 grid((unsigned)((g.groups * (d / 4) + 255) / 256), 2);
    return dependent_launch(io_f32 ? decay_group_sum_kernel<float> : decay_group_sum_kernel<__nv_bfloat16>, grid, 256, 0, s, true, g);
}

}  // namespace prism
