// decay_tc.cu -- the decay scan's bf16 kernels on the tensor cores (decay.cuh has the formulas): the
// segment sums and the pass over the tokens, chunks of 128 tokens, one CTA per segment of one (b, h).
//
// Per chunk, with n tokens, weights w_j of the state's write and row factors f_i of its read:
//   P   = X Y^T                 [128 tokens x 128 tokens]   M = 128, N = 128, K = D1
//   O   = f o (X R^T) + P' Z    P' = a^|i-j| P on the causal side, rounded to bf16
//   dR^T = (w o Y)^T Z          [D1 x D2], the write; R^T <- a^n R^T + dR^T in fp32 registers
// Operands that come from registers (P', the weighted Y) go to the tensor core through TMEM, where the
// A operand's row is the lane: no shared memory and no swizzle.  The weighted Y is not rounded to one bf16: a
// state sums thousands of them.  It is split into bf16 terms whose sum has 16 (pass kernel: only outputs
// depend on it) or 24 bits (sum kernel: the fp32 states that the caller gets), each multiplied with the exact Z.
// The state is rounded to bf16 once per chunk as the B operand of X R^T; its fp32 master stays in
// registers, so that no tensor-core accumulation (which truncates) runs longer than one chunk.
//
// Widths of 32 run as 64: the TMA boxes reach past the tensor, where loads give zeros and stores
// write nothing.

#include "decay.cuh"
#include "f32x2.cuh"
#include "tc.cuh"
#include "tensor_map.cuh"

namespace prism {
namespace {

using namespace tc;

constexpr int CT = kDecayChunkTc;

// Polls of a bounded wait (of up to kSuspendNs each), and in the stall test.
constexpr uint32_t kPolls = 1u << 17, kStallPolls = 1u << 6;

// Library status word of these kernels (a bounded wait that gave up), read and cleared by
// prism_query_device_status.
__device__ uint32_t g_decay_status;

struct DecayMaps {
    CUtensorMap x, y, z, o;
};
struct DecayMapSet {
    DecayMaps m[kDecaySet];
};

// Bytes of a tile of 128 tokens, D columns (64-column blocks of 128 rows x 128 bytes).
constexpr uint32_t kBlk = CT * 128;
template <int D>
constexpr uint32_t tile_bytes() { return kBlk * (D / 64); }

// What a CTA works on: segment `seg` of sequence (b, h); chunk i of its walk starts at token t0(i) and
// has n(i) valid tokens.
struct Walk {
    int b, h, seg, len, s0, s1, send, nch, reverse;
    __device__ explicit Walk(const DecayPass &p) {
        seg = blockIdx.x % p.nseg;
        h = blockIdx.y;
        b = blockIdx.z;
        len = decay_len(p.lengths, b, p.T);
        s0 = seg * p.seg_tokens;
        send = min(s0 + p.seg_tokens, p.T);
        s1 = min(send, len);
        nch = s1 > s0 ? (s1 - s0 + CT - 1) / CT : 0;
        reverse = p.reverse;
    }
    __device__ int t0(int i) const { return s0 + (reverse ? nch - 1 - i : i) * CT; }
    __device__ int n(int i) const { return min(CT, s1 - t0(i)); }
};

__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *m, int D, int head, int t, int b, uint64_t *bar) {
    mbar_expect_tx(bar, kBlk * (D / 64));
    for (int c = 0; c < D / 64; ++c) tma_load_4d(dst + c * kBlk, m, 64 * c, head, t, b, bar);
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) { return pack_bf16(a, b); }
__device__ __forceinline__ float lo_f(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float hi_f(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// Powers of a head's decay in shared memory: at(e) = a^e for 0 <= e <= 128 and 0 for -32 < e < 0, and the
// weights of a full chunk's tokens in the state that leaves it, w[j] = a^(127 - j), reversed a^(j + 1).
struct Powers {
    alignas(16) float w[CT];
    alignas(16) float none[32], p[CT + 1];
    __device__ void fill(float a, int reverse, int tid, int nthreads) {
        for (int i = tid; i <= CT; i += nthreads) {
            const float x = decay_pow(a, i);
            p[i] = x;
            if (reverse && i > 0) w[i - 1] = x;
            if (!reverse && i < CT) w[CT - 1 - i] = x;
            if (i < 32) none[i] = 0.f;
        }
    }
    __device__ __forceinline__ float at(int e) const { return p[e]; }
};

// Column m of the Y tile, tokens j0 .. j0 + 15, times their weights w, as TERMS bf16 terms into this
// thread's TMEM lane: term t at column col + 64 t, two tokens per column.  Tokens from n on are zero
// whatever the tile holds there.
constexpr int kWeigh = 16;

template <int TERMS>
__device__ __forceinline__ void weigh(const uint8_t *Y, int m, const float *w, int j0, int n, uint32_t taddr_lane, int col) {
    const uint8_t *base = Y + (m >> 6) * kBlk + ((m & 7) << 1) + j0 * 128;
    const int ch = (m & 63) >> 3;
    float x[kWeigh];
#pragma unroll
    for (int i = 0; i < kWeigh; i += 4) {
        const float4 w4 = *reinterpret_cast<const float4 *>(w + j0 + i);
        const float *wf = &w4.x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = i + e;  // (j0 is a multiple of 8: it does not change the swizzle)
            const uint32_t raw = *reinterpret_cast<const uint16_t *>(base + j * 128 + ((ch ^ (j & 7)) << 4));
            x[j] = __uint_as_float(raw << 16) * wf[e];
        }
    }
    if (j0 + kWeigh > n) {
#pragma unroll
        for (int j = 0; j < kWeigh; ++j) x[j] = j0 + j < n ? x[j] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < TERMS; ++k) {
        uint32_t t[kWeigh / 2];
#pragma unroll
        for (int i = 0; i < kWeigh / 2; ++i) {
            t[i] = bf16_pair(x[2 * i], x[2 * i + 1]);
            x[2 * i] -= lo_f(t[i]);
            x[2 * i + 1] -= hi_f(t[i]);
        }
        tmem_st8(taddr_lane + col + 64 * k + j0 / 2, t);
    }
}

// The same for 64-wide Y (D1 = 64), whose product needs only M = 64 rows: the weighted tile goes to shared
// memory in Y's own layout (an MN-major A operand), TERMS tiles one after the other, 16 bytes at a time by any
// thread.  A TMEM operand's lanes are its rows, so half of the warps had none to write (2400 cycles a chunk).
template <int TERMS>
__device__ __forceinline__ void weigh_tile64(const uint8_t *Y, uint8_t *out, const float *w, int n, int tid, int nthreads) {
    for (int e = tid; e < CT * 8; e += nthreads) {
        const int row = e >> 3;
        const uint4 raw = *reinterpret_cast<const uint4 *>(Y + e * 16);  // (a row's chunks may be read in any order)
        const uint32_t y[4] = {raw.x, raw.y, raw.z, raw.w};
        const F2 ww = pack2(w[row], w[row]);
        F2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = row < n ? mul(pack2(lo_f(y[i]), hi_f(y[i])), ww) : 0ull;
#pragma unroll
        for (int k = 0; k < TERMS; ++k) {
            uint32_t t[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                t[i] = bf16_pair(first(x[i]), second(x[i]));
                if (k + 1 < TERMS) x[i] = add(x[i], pack2(-lo_f(t[i]), -hi_f(t[i])));
            }
            *reinterpret_cast<uint4 *>(out + k * kBlk + e * 16) = make_uint4(t[0], t[1], t[2], t[3]);
        }
    }
}

// Where row m = 16 (lane quarter) + lane of an M = 64 product sits: the first 16 lanes of each quarter.  M = 128:
// row = lane.
template <int D1>
__device__ __forceinline__ int product_row(int q, int lane) { return D1 == 64 ? 16 * q + lane : 32 * q + lane; }
template <int D1>
__device__ __forceinline__ bool product_lane(int lane) { return D1 != 64 || lane < 16; }

// Zero rows n .. 127 of a tile (by `nthreads` threads), so that what lies behind the sequence's end
// reaches no product.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t *tile, int n, int tid, int nthreads) {
    for (int e = tid; e < (CT - n) * (D / 64) * 8; e += nthreads) {
        const int c = e & 7, blk = (e >> 3) % (D / 64), r = n + (e >> 3) / (D / 64);
        *reinterpret_cast<uint4 *>(tile + blk * kBlk + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
}

// ------------------------------------------------------------------------------------------------
// Segment sums.  Per chunk three products of 128 x D2 x 128 against 2 tiles of loads: the loads are
// the bound (at D1 = D2 = 128 about 2700 cycles a chunk at the copy bandwidth, the products 1536).

template <int D1, int D2>
struct SumLayout {
    // Warps that weigh Y, that hold the state.  At 64 x 128 there is one buffer of the weighted Y, and twice the warps
    // do not work ahead of the products.  (16 heads of 65536 tokens, 16 warps against 8: 128 x 128 338 us against 345,
    // 128 x 64 and 64 x 64 the same, 64 x 128 289 against 284; its padded batch of 32 x 4 275 against 272.)
    static constexpr int YW = D1 == 64 && D2 == 128 ? 8 : 16, SW = 8;
    static constexpr int LOADW = YW + SW, MMAW = LOADW + 1;
    // With 16, registers are shared out by role as in the pass (launched with 72), by whole warpgroups: two warps of
    // the last have no role.  With 8 each thread has 96 throughout.
    static constexpr bool SHARED_OUT = YW == 16;
    static constexpr int THREADS = 32 * (SHARED_OUT ? LOADW + 4 : MMAW + 1);
    static constexpr int RS = 112, RY = 56, RM = 40;
    static constexpr int SHARES = SHARED_OUT ? (SW * RS + YW * RY + 4 * RM) * 32 : 0;
    static_assert(!SHARED_OUT || (THREADS == 896 && SHARES <= 72 * THREADS), "register shares");
    // The weighted Y: two buffers of three terms in TMEM, or (D1 = 64) one or two in shared memory.
    static constexpr int NYB = D1 == 64 && D2 == 128 ? 1 : 2;
    static constexpr int NST = 3;
    static constexpr uint32_t STAGE = tile_bytes<D1>() + tile_bytes<D2>();
    static constexpr uint32_t YP = NST * STAGE, YP_BYTES = D1 == 64 ? 3 * kBlk : 0;
    static constexpr uint32_t BYTES = YP + NYB * YP_BYTES + 1024;
    static constexpr uint32_t cY = 0, cD = 384;          // TMEM columns: the weighted Y, the product
    static_assert(BYTES + 2048 <= 227 * 1024, "shared memory budget");
    static_assert(cY + 192 * NYB <= cD && cD + D2 <= 512, "TMEM columns");
};

template <int D1, int D2>
__global__ void __launch_bounds__(SumLayout<D1, D2>::THREADS, 1)
    decay_sum_tc_kernel(const __grid_constant__ DecayPassSet set, const __grid_constant__ DecayMapSet map_set) {
    const DecayPass &p = set.p[blockIdx.x / set.p[0].nseg];
    const DecayMaps &maps = map_set.m[blockIdx.x / set.p[0].nseg];
    using LY = SumLayout<D1, D2>;
    constexpr int NST = LY::NST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[NST], freeb[NST], yp_full[LY::NYB], yp_free[LY::NYB], d_full, d_free, drain;
    __shared__ Powers pw;
    __shared__ __align__(16) float w_last[CT];  // the weights of the walk's last chunk
    __shared__ uint32_t tmem_base_sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    dependent_wait();
    const Walk wk(p);
    uint32_t *status = &g_decay_status;
    const uint32_t lim = p.stall ? kStallPolls : kPolls;
    const float a = p.decay[wk.h];

    auto load = [&](int i) {
        const int st = i % NST;
        uint8_t *s = sm + st * LY::STAGE;
        mbar_expect_tx(&full[st], LY::STAGE);
        for (int c = 0; c < D1 / 64; ++c) tma_load_4d(s + c * kBlk, &maps.y, 64 * c, wk.h / p.y.div, wk.t0(i), wk.b, &full[st]);
        for (int c = 0; c < D2 / 64; ++c)
            tma_load_4d(s + tile_bytes<D1>() + c * kBlk, &maps.z, 64 * c, wk.h / p.z.div, wk.t0(i), wk.b, &full[st]);
    };
    if (warp == LY::MMAW) tmem_alloc(&tmem_base_sh, 512);
    if (warp == LY::LOADW && lane == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&freeb[i], LY::YW + 1);
        }
        for (int i = 0; i < LY::NYB; ++i) {
            mbar_init(&yp_full[i], LY::YW);
            mbar_init(&yp_free[i], 1);
        }
        mbar_init(&d_full, 1);
        mbar_init(&d_free, LY::SW);
        mbar_init(&drain, 1);
        mbar_fence_init();
        // the first loads are on their way while the others set up
        for (int i = 0; i < NST && i < wk.nch && !p.stall; ++i) load(i);
    }
    pw.fill(a, wk.reverse, tid, LY::THREADS);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tb = tmem_base_sh;
    if (wk.nch > 0)
        for (int j = tid; j < CT; j += LY::THREADS)
            w_last[j] = wk.reverse ? pw.w[j] : pw.at(max(wk.n(wk.nch - 1) - 1 - j, 0));
    __syncthreads();

    if constexpr (LY::SHARED_OUT)
        if (warp >= LY::LOADW) setmaxnreg_dec<LY::RM>();
    if (warp == LY::LOADW) {
        if (lane == 0 && !p.stall) {
            int i = min(NST, wk.nch);
            for (; i < wk.nch; ++i) {
                if (!mbar_wait_suspend(&freeb[i % NST], (uint32_t)((i / NST - 1) & 1), status, lim)) break;
                load(i);
            }
            // loads in flight land before the CTA exits
            for (int k = i > NST ? i - NST : 0; k < i; ++k) mbar_wait_suspend(&full[k % NST], (uint32_t)((k / NST) & 1), nullptr, lim);
        }
    } else if (warp == LY::MMAW) {
        {
            const uint32_t id = D1 == 64 ? idesc_bf16(64, D2, 1, 1) : idesc_bf16(128, D2, 0, 1);
            auto oz = [](int ks) { return (uint64_t)koff_mn_sw128(ks); };
            auto oy = [](int ks) { return 8 * ks; };
            for (int i = 0; i < wk.nch; ++i) {
                const int st = i % NST, pb = i % LY::NYB;
                if (!mbar_wait_suspend(&full[st], (uint32_t)((i / NST) & 1), status, lim) ||
                    !mbar_wait_suspend(&yp_full[pb], (uint32_t)((i / LY::NYB) & 1), status, lim) ||
                    (i > 0 && !mbar_wait_suspend(&d_free, (uint32_t)((i - 1) & 1), status, lim)))
                    break;
                fence_after_sync();
                const uint64_t dz = make_desc(smem_u32(sm + st * LY::STAGE + tile_bytes<D1>()), kBlk, 1024, 2);
                // smallest terms first: their sum loses nothing to the large one's magnitude
                if constexpr (D1 == 64) {
                    const uint32_t yp = smem_u32(sm + LY::YP + pb * LY::YP_BYTES);
#pragma unroll
                    for (int k = 2; k >= 0; --k)
                        mma_steps_warp<CT / 16>(tb + LY::cD, id, make_desc(yp + k * kBlk, kBlk, 1024, 2), dz, oz, oz, k < 2);
                } else {
                    const uint32_t ya = tb + LY::cY + pb * 192;
#pragma unroll
                    for (int k = 2; k >= 0; --k)
                        mma_steps_tmem_a_warp<CT / 16>(tb + LY::cD, id, ya + 64 * k, dz, oy, oz, k < 2);
                }
                mma_commit_warp(&d_full);
                mma_commit_warp(&yp_free[pb]);
                mma_commit_warp(&freeb[st]);
            }
            mma_commit_warp(&drain);
            mbar_wait_suspend(&drain, 0, nullptr, lim);
        }
    } else if (warp > LY::MMAW) {
        // (no role)
    } else if (warp < LY::YW) {
        if constexpr (LY::SHARED_OUT) setmaxnreg_dec<LY::RY>();
        const int q = warp & 3, j1 = CT / (LY::YW / 4) * (warp >> 2), m = 32 * q + lane;
        for (int i = 0; i < wk.nch; ++i) {
            const int st = i % NST, pb = i % LY::NYB, n = wk.n(i);
            uint8_t *s = sm + st * LY::STAGE;
            if (!mbar_wait_suspend(&full[st], (uint32_t)((i / NST) & 1), status, lim) ||
                (i >= LY::NYB && !mbar_wait_suspend(&yp_free[pb], (uint32_t)((i / LY::NYB - 1) & 1), status, lim)))
                break;
            fence_after_sync();
            const float *w = i + 1 < wk.nch ? pw.w : w_last;
            if (n < CT) zero_rows<D2>(s + tile_bytes<D1>(), n, tid, 32 * LY::YW);
            if constexpr (D1 == 64) {
                weigh_tile64<3>(s, sm + LY::YP + pb * LY::YP_BYTES, w, n, tid, 32 * LY::YW);
            } else {
#pragma unroll 1
                for (int j0 = j1; j0 < j1 + CT / (LY::YW / 4); j0 += kWeigh)
                    weigh<3>(s, m, w, j0, n, taddr(tb, 32 * q, 0), LY::cY + pb * 192);
                tmem_wait_st();
            }
            if (D1 == 64 || n < CT) fence_async_smem();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&yp_full[pb]);
                mbar_arrive(&freeb[st]);
            }
        }
    } else {
        if constexpr (LY::SHARED_OUT) setmaxnreg_inc<LY::RS>();
        const int sw = warp - LY::YW, q = sw & 3, half = sw >> 2, m = product_row<D1>(q, lane);
        constexpr int NC = D2 / 2;
        float r[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) r[c] = 0.f;
        bool ok = true;
        for (int i = 0; i < wk.nch; ++i) {
            const float an = pw.at(wk.n(i));
            if (!mbar_wait_suspend(&d_full, (uint32_t)(i & 1), status, lim)) { ok = false; break; }
            fence_after_sync();
#pragma unroll
            for (int c = 0; c < NC; c += 32) {
                float d[32];
                tmem_ld32(taddr(tb, 32 * q, LY::cD + half * NC + c), d);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) r[c + k] = fmaf(an, r[c + k], d[k]);
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_free);
        }
        if (ok && product_lane<D1>(lane) && m < p.d1) {
            float *F = p.F + (((long long)wk.b * p.H + wk.h) * p.nseg + wk.seg) * p.d1 * p.d2 + m;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int nn = half * NC + c;
                if (nn < p.d2) F[nn * p.d1] = r[c];
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == LY::MMAW) tmem_dealloc(tb, 512);
}

// ------------------------------------------------------------------------------------------------
// The pass.

template <int D1, int D2>
struct PassLayout {
    static constexpr int PW = 8, OW = 4, SW = 8, YW = 8;  // warps: P', outputs, state, weighted Y
    static constexpr int OW0 = PW, SW0 = OW0 + OW, YW0 = SW0 + SW, LOADW = YW0 + YW, MMAW = LOADW + 1;
    static constexpr int THREADS = 32 * (LOADW + 4);      // whole warpgroups: two warps of the last have no role
    // Registers of a thread by role: the block is launched with 64 each, and what the others give up is what the
    // state warps, which hold D2 / 2 state elements, take on.  A launch is refused where the shares add up to more
    // than the kernel was built with (setmaxnreg would wait for registers that never come).
    static constexpr int RS = 96, RP = 56, RO = 56, RY = 56, RM = 40;
    static constexpr int SHARES = (SW * RS + PW * RP + OW * RO + YW * RY + 4 * RM) * 32;
    static_assert(THREADS == 1024 && SHARES <= 64 * THREADS, "register shares");
    static constexpr int NST = D1 == 64 && D2 == 64 ? 3 : 2;
    static constexpr uint32_t X = 0, Y = tile_bytes<D1>(), Z = 2 * tile_bytes<D1>();
    static constexpr uint32_t STAGE = 2 * tile_bytes<D1>() + tile_bytes<D2>();
    static constexpr uint32_t R = NST * STAGE;            // R^T as bf16: rows along y, columns along z
    static constexpr uint32_t R_BLK = D1 * 128;
    static constexpr uint32_t YP = R + R_BLK * (D2 / 64), YP_BYTES = D1 == 64 ? 2 * kBlk : 0;  // the weighted Y (or in TMEM)
    static constexpr uint32_t BYTES = YP + YP_BYTES + 1024;
    // TMEM columns.  (A second P, for the next chunk's, where there is room for it: no faster at 64 x 64.)
    static constexpr uint32_t cP = 0, cO = 128, cD = cO + D2, cY = cD + D2;
    static_assert(BYTES + 1024 <= 227 * 1024, "shared memory budget");
    static_assert(cY + 128 <= 512, "TMEM columns");
};

template <int D1, int D2>
__global__ void __launch_bounds__(PassLayout<D1, D2>::THREADS, 1)
    decay_pass_tc_kernel(const __grid_constant__ DecayPassSet set, const __grid_constant__ DecayMapSet map_set) {
    const DecayPass &p = set.p[blockIdx.x / set.p[0].nseg];
    const DecayMaps &maps = map_set.m[blockIdx.x / set.p[0].nseg];
    using LY = PassLayout<D1, D2>;
    constexpr int NST = LY::NST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t x_full[NST], y_full[NST], z_full[NST], x_free[NST], y_free[NST], z_free[NST];
    __shared__ uint64_t p_full, p_ready, qs_full, o_scaled, o_full, o_free, s_ready, ds_full, yp_full, yp_free, drain;
    __shared__ Powers pw;
    __shared__ uint32_t tmem_base_sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Walk wk(p);
    uint32_t *status = &g_decay_status;
    const uint32_t lim = p.stall ? kStallPolls : kPolls;
    const float a = p.decay[wk.h];

    auto load_x = [&](int i) { load_tile(sm + i % NST * LY::STAGE + LY::X, &maps.x, D1, wk.h / p.x.div, wk.t0(i), wk.b, &x_full[i % NST]); };
    auto load_y = [&](int i) { load_tile(sm + i % NST * LY::STAGE + LY::Y, &maps.y, D1, wk.h / p.y.div, wk.t0(i), wk.b, &y_full[i % NST]); };
    auto load_z = [&](int i) { load_tile(sm + i % NST * LY::STAGE + LY::Z, &maps.z, D2, wk.h / p.z.div, wk.t0(i), wk.b, &z_full[i % NST]); };
    const int early = p.stall ? 0 : min(NST, wk.nch);
    if (warp == LY::MMAW) tmem_alloc(&tmem_base_sh, 512);
    if (warp == LY::LOADW && lane == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&x_full[i], 1);
            mbar_init(&y_full[i], 1);
            mbar_init(&z_full[i], 1);
            mbar_init(&x_free[i], 1);
            mbar_init(&y_free[i], LY::YW + 1);
            mbar_init(&z_free[i], LY::OW);
        }
        mbar_init(&p_full, 1);
        mbar_init(&p_ready, LY::PW);
        mbar_init(&qs_full, 1);
        mbar_init(&o_scaled, LY::OW);
        mbar_init(&o_full, 1);
        mbar_init(&o_free, LY::OW);
        mbar_init(&s_ready, LY::SW);
        mbar_init(&ds_full, 1);
        mbar_init(&yp_full, LY::YW);
        mbar_init(&yp_free, 1);
        mbar_init(&drain, 1);
        mbar_fence_init();
        // the first loads are on their way while the others set up
        for (int i = 0; i < early; ++i) {
            load_x(i);
            load_y(i);
            load_z(i);
        }
    }
    pw.fill(a, wk.reverse, tid, LY::THREADS);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tb = tmem_base_sh;

    if (warp >= LY::LOADW) setmaxnreg_dec<LY::RM>();
    if (warp == LY::LOADW) {
        if (lane == 0 && !p.stall) {
            int nx = early, ny = early, nz = early;  // tiles requested
            for (int i = early; i < wk.nch; ++i) {
                const int st = i % NST;
                const uint32_t par = (uint32_t)((i / NST - 1) & 1);
                if (!mbar_wait_suspend(&x_free[st], par, status, lim)) break;
                load_x(i);
                ++nx;
                if (!mbar_wait_suspend(&y_free[st], par, status, lim)) break;
                load_y(i);
                ++ny;
                if (!mbar_wait_suspend(&z_free[st], par, status, lim)) break;
                load_z(i);
                ++nz;
            }
            // loads in flight land before the CTA exits
            for (int k = nx > NST ? nx - NST : 0; k < nx; ++k) mbar_wait_suspend(&x_full[k % NST], (uint32_t)((k / NST) & 1), nullptr, lim);
            for (int k = ny > NST ? ny - NST : 0; k < ny; ++k) mbar_wait_suspend(&y_full[k % NST], (uint32_t)((k / NST) & 1), nullptr, lim);
            for (int k = nz > NST ? nz - NST : 0; k < nz; ++k) mbar_wait_suspend(&z_full[k % NST], (uint32_t)((k / NST) & 1), nullptr, lim);
        }
    } else if (warp == LY::MMAW) {
        {
            const uint32_t idP = idesc_bf16(128, 128, 0, 0), idZ = idesc_bf16(128, D2, 0, 1), idY = idesc_bf16(64, D2, 1, 1);
            auto ok_ = [](int ks) { return (uint64_t)koff_k_sw128(ks, kBlk); };
            auto omn = [](int ks) { return (uint64_t)koff_mn_sw128(ks); };
            auto oy = [](int ks) { return 8 * ks; };
            auto op = [](int ks) { return 8 * ks + (ks >= 4 ? 32 : 0); };  // P': 64 tokens in each half of P
            const uint64_t dR = make_desc(smem_u32(sm + LY::R), LY::R_BLK, 1024, 2);
            for (int i = 0; i < wk.nch; ++i) {
                const int st = i % NST;
                const uint32_t par = (uint32_t)((i / NST) & 1), ph = (uint32_t)(i & 1), before = (uint32_t)((i - 1) & 1);
                const uint32_t s = smem_u32(sm + st * LY::STAGE);
                const uint64_t dX = make_desc(s + LY::X, 16, 1024, 2), dY = make_desc(s + LY::Y, 16, 1024, 2),
                               dZ = make_desc(s + LY::Z, kBlk, 1024, 2);
                if (!mbar_wait_suspend(&x_full[st], par, status, lim) || !mbar_wait_suspend(&y_full[st], par, status, lim)) break;
                fence_after_sync();
                // P (its region's last readers were the previous chunk's P' Z products, issued before)
                mma_steps_warp<D1 / 16>(tb + LY::cP, idP, dX, dY, ok_, ok_, false);
                mma_commit_warp(&p_full);
                mma_commit_warp(&y_free[st]);
                // X R^T
                if (!mbar_wait_suspend(&s_ready, ph, status, lim) || (i > 0 && !mbar_wait_suspend(&o_free, before, status, lim))) break;
                fence_after_sync();
                mma_steps_warp<D1 / 16>(tb + LY::cO, idZ, dX, dR, ok_, omn, false);
                mma_commit_warp(&qs_full);
                mma_commit_warp(&x_free[st]);
                // the write (the state warps have read the last one: s_ready)
                if (!mbar_wait_suspend(&yp_full, ph, status, lim) || !mbar_wait_suspend(&z_full[st], par, status, lim)) break;
                fence_after_sync();
                if (i + 1 < wk.nch) {
                    if constexpr (D1 == 64) {
                        const uint32_t yp = smem_u32(sm + LY::YP);
                        mma_steps_warp<CT / 16>(tb + LY::cD, idY, make_desc(yp + kBlk, kBlk, 1024, 2), dZ, omn, omn, false);
                        mma_steps_warp<CT / 16>(tb + LY::cD, idY, make_desc(yp, kBlk, 1024, 2), dZ, omn, omn, true);
                    } else {
                        mma_steps_tmem_a_warp<CT / 16>(tb + LY::cD, idZ, tb + LY::cY + 64, dZ, oy, omn, false);
                        mma_steps_tmem_a_warp<CT / 16>(tb + LY::cD, idZ, tb + LY::cY, dZ, oy, omn, true);
                    }
                    mma_commit_warp(&ds_full);
                    mma_commit_warp(&yp_free);
                }
                // O += P' Z
                if (!mbar_wait_suspend(&p_ready, ph, status, lim) || !mbar_wait_suspend(&o_scaled, ph, status, lim)) break;
                fence_after_sync();
                mma_steps_tmem_a_warp<CT / 16>(tb + LY::cO, idZ, tb + LY::cP, dZ, op, omn, true);
                mma_commit_warp(&o_full);
            }
            mma_commit_warp(&drain);
            mbar_wait_suspend(&drain, 0, nullptr, lim);
        }
    } else if (warp > LY::MMAW) {
        // (no role)
    } else if (warp < LY::OW0) {
        setmaxnreg_dec<LY::RP>();
        // ---------------- P' = a^|i-j| P on the causal side, as bf16 over P ----------------
        // two warps per 32 rows, 64 columns each, whose bf16 values go to the first 32 of the warp's own
        const int q = warp & 3, half = warp >> 2, row = 32 * q + lane;
        for (int i = 0; i < wk.nch; ++i) {
            const int n = wk.n(i);
            const uint32_t tl = taddr(tb, 32 * q, LY::cP);
            if (!mbar_wait_suspend(&p_full, (uint32_t)(i & 1), status, lim)) break;
            fence_after_sync();
            // 16 columns at a time, in a loop: unrolled, the five roles' code of a chunk no longer fits the
            // instruction cache and every role waits for its instructions (P' took 7000 cycles instead of 1400)
#pragma unroll 1
            for (int c0 = 64 * half; c0 < 64 * half + 64; c0 += 16) {
                const int J = c0 >> 5, j0 = c0 & 31;  // 32-column block, and the columns' place in it
                uint32_t out[8];
                if (J == q || (wk.reverse ? J > q : J < q)) {
                    float v[16];
                    tmem_ld16(tl + c0, v);
                    tmem_wait_ld();
                    if (J == q) {
                        // (the powers of the other side of the diagonal are zeros below the table)
                        const float *d = pw.p + (wk.reverse ? j0 - lane : lane - j0);
                        if (wk.reverse) {
#pragma unroll
                            for (int c = 0; c < 16; ++c) v[c] *= d[c];
                        } else {
#pragma unroll
                            for (int c = 0; c < 16; ++c) v[c] *= d[-c];
                        }
                    } else {
                        // a^|row - col| = a^(distance to the block's near column) x a^(near column - col)
                        const float f = pw.at(wk.reverse ? 32 * J - row : row - 32 * J - 31);
                        const float *near = (wk.reverse ? pw.p : pw.w + CT - 32) + j0;  // a^c, a^(31 - c)
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            const float4 u = *reinterpret_cast<const float4 *>(near + c);
                            v[c] *= f * u.x;
                            v[c + 1] *= f * u.y;
                            v[c + 2] *= f * u.z;
                            v[c + 3] *= f * u.w;
                        }
                    }
                    if (c0 + 16 > n) {
#pragma unroll
                        for (int c = 0; c < 16; ++c) v[c] = c0 + c < n ? v[c] : 0.f;
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c) out[c] = bf16_pair(v[2 * c], v[2 * c + 1]);
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c) out[c] = 0u;
                }
                tmem_st8(tl + 64 * half + ((c0 & 63) >> 1), out);  // columns that this lane has read already
            }
            tmem_wait_st();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready);
        }
    } else if (warp < LY::SW0) {
        setmaxnreg_dec<LY::RO>();
        // ---------------- outputs ----------------
        const int q = warp & 3, row = 32 * q + lane;
        const uint32_t tl = taddr(tb, 32 * q, LY::cO);
        for (int i = 0; i < wk.nch; ++i) {
            const int n = wk.n(i), t0 = wk.t0(i), st = i % NST;
            const bool live = row < n;
            const float f = live ? pw.at(wk.reverse ? n - 1 - row : row + 1) : 0.f;
            if (!mbar_wait_suspend(&qs_full, (uint32_t)(i & 1), status, lim)) break;
            fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < D2; c += 32) {
                float v[32];
                tmem_ld32(tl + c, v);
                tmem_wait_ld();
                uint32_t u[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(v[k] * f);
                tmem_st32(tl + c, u);
            }
            tmem_wait_st();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_scaled);
            if (!mbar_wait_suspend(&o_full, (uint32_t)(i & 1), status, lim)) break;
            fence_after_sync();
            // Z has had its last reader: its rows take the output's, as bf16, or (shared heads' gradients) as fp32,
            // 32 columns at a time; rows behind the sequence's end are zeros
            uint8_t *zs = sm + st * LY::STAGE + LY::Z;
            if (p.o_f32) {
                uint8_t *box = zs + q * 4096;
#pragma unroll 1
                for (int c = 0; c < D2 && c < p.d2; c += 32) {
                    if (c > 0) {
                        if (lane == 0) bulk_wait_read();
                        __syncwarp();
                    }
#pragma unroll
                    for (int c16 = 0; c16 < 32; c16 += 16) {
                        float v[16];
                        tmem_ld16(tl + c + c16, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; k += 4)
                            *reinterpret_cast<float4 *>(box + lane * 128 + ((((c16 + k) >> 2) ^ (lane & 7)) << 4)) =
                                live ? make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_4d(&maps.o, box, c, wk.h, t0 + 32 * q, wk.b);
                        bulk_commit();
                    }
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < D2; c += 32) {
                    float v[32];
                    tmem_ld32(tl + c, v);
                    tmem_wait_ld();
                    if (!live)
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = 0.f;
#pragma unroll
                    for (int k = 0; k < 32; k += 8)
                        *reinterpret_cast<uint4 *>(zs + sw128_off(row, c + k, kBlk)) =
                            make_uint4(bf16_pair(v[k], v[k + 1]), bf16_pair(v[k + 2], v[k + 3]),
                                       bf16_pair(v[k + 4], v[k + 5]), bf16_pair(v[k + 6], v[k + 7]));
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
#pragma unroll
                    for (int c = 0; c < D2 / 64; ++c)
                        if (64 * c < p.d2) tma_store_4d(&maps.o, zs + c * kBlk + 32 * q * 128, 64 * c, wk.h, t0 + 32 * q, wk.b);
                    bulk_commit();
                }
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&o_free);
                bulk_wait_read();
                mbar_arrive(&z_free[st]);
            }
        }
        if (lane == 0) bulk_wait_all();
    } else if (warp < LY::YW0) {
        setmaxnreg_inc<LY::RS>();
        // ---------------- the state: row m of R^T, half of the columns ----------------
        const int sw = warp - LY::SW0, q = sw & 3, half = sw >> 2, m = product_row<D1>(q, lane);
        const bool mine = product_lane<D1>(lane);
        constexpr int NC = D2 / 2;
        float r[NC];
        // (the entry state comes from the call's previous kernel; the other roles' inputs are older than the call)
        dependent_wait();
        const float *E = p.entry && mine && m < p.d1
                             ? p.entry + (((long long)wk.b * p.H + wk.h) * p.nseg + wk.seg) * p.d1 * p.d2 : nullptr;
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
            const int nn = half * NC + c;  // (d2 is a multiple of 4)
            if (E && nn < p.d2 && p.entry_t) {
                const float4 e = *reinterpret_cast<const float4 *>(E + m * p.d2 + nn);
                r[c] = e.x;
                r[c + 1] = e.y;
                r[c + 2] = e.z;
                r[c + 3] = e.w;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) r[c + k] = E && nn < p.d2 ? E[(nn + k) * p.d1 + m] : 0.f;
            }
        }
        for (int i = 0; i < wk.nch; ++i) {
            if (i > 0) {
                const float an = pw.at(wk.n(i - 1));
                // the previous chunk's write, and (issued before it) the last read of the bf16 state
                if (!mbar_wait_suspend(&ds_full, (uint32_t)((i - 1) & 1), status, lim)) break;
                fence_after_sync();
#pragma unroll
                for (int c = 0; c < NC; c += 16) {
                    float d[16];
                    tmem_ld16(taddr(tb, 32 * q, LY::cD + half * NC + c), d);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) r[c + k] = fmaf(an, r[c + k], d[k]);
                }
            }
            if (mine) {
#pragma unroll
                for (int c = 0; c < NC; c += 8)
                    *reinterpret_cast<uint4 *>(sm + LY::R + sw128_off(m, half * NC + c, LY::R_BLK)) =
                        make_uint4(bf16_pair(r[c], r[c + 1]), bf16_pair(r[c + 2], r[c + 3]), bf16_pair(r[c + 4], r[c + 5]),
                                   bf16_pair(r[c + 6], r[c + 7]));
            }
            fence_async_smem();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_ready);
        }
    } else {
        setmaxnreg_dec<LY::RY>();
        // ---------------- Y times the write's weights ----------------
        const int yt = tid - 32 * LY::YW0, q = warp & 3, half = (warp - LY::YW0) >> 2, m = 32 * q + lane;
        static_assert(LY::YW0 % 4 == 0, "the warp's TMEM lanes");
        for (int i = 0; i < wk.nch; ++i) {
            const int st = i % NST, n = wk.n(i);
            uint8_t *s = sm + st * LY::STAGE;
            if (!mbar_wait_suspend(&y_full[st], (uint32_t)((i / NST) & 1), status, lim)) break;
            if (n < CT) {
                if (!mbar_wait_suspend(&z_full[st], (uint32_t)((i / NST) & 1), status, lim)) break;
                zero_rows<D2>(s + LY::Z, n, yt, 32 * LY::YW);
                fence_async_smem();
            }
            // (on the last chunk too, where nothing is written: without it a warp could arrive for this chunk
            // before another one has for the last, and complete that phase in its place)
            if (i > 0 && !mbar_wait_suspend(&yp_free, (uint32_t)((i - 1) & 1), status, lim)) break;
            if (i + 1 < wk.nch) {  // (nobody reads the state behind the last chunk)
                fence_after_sync();
                if constexpr (D1 == 64) {
                    weigh_tile64<2>(s + LY::Y, sm + LY::YP, pw.w, n, yt, 32 * LY::YW);
                    fence_async_smem();
                } else {
#pragma unroll 1
                    for (int j0 = 64 * half; j0 < 64 * half + 64; j0 += kWeigh)
                        weigh<2>(s + LY::Y, m, pw.w, j0, n, taddr(tb, 32 * q, 0), LY::cY);
                    tmem_wait_st();
                }
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&yp_full);
                mbar_arrive(&y_free[st]);
            }
        }
    }
    // rows behind the sequence's last token
    const int z0 = max(wk.s0, wk.s1);
    const int row_bytes = p.d2 * (p.o_f32 ? 4 : 2), per_row = row_bytes / 16;
    for (long long e = tid; e < (long long)(wk.send - z0) * per_row; e += LY::THREADS) {
        const long long t = z0 + e / per_row;
        *reinterpret_cast<uint4 *>((uint8_t *)p.o + (((long long)wk.b * p.T + t) * p.H + wk.h) * row_bytes + (e % per_row) * 16) =
            make_uint4(0, 0, 0, 0);
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == LY::MMAW) tmem_dealloc(tb, 512);
}

bool operand_map(CUtensorMap *m, const DecayPass &p, const DecayTensor &t, int d) {
    return rows_map(m, t.p, false, p.B, p.T, p.H / t.div, d, t.sb, t.st, t.sh, CT);
}

template <int D1, int D2>
cudaError_t launch_one(const DecayPassSet &set, bool sum, cudaStream_t s) {
    DecayMapSet maps;
    for (int i = 0; i < set.count; ++i) {
        const DecayPass &p = set.p[i];
        DecayMaps &m = maps.m[i];
        bool ok = operand_map(&m.y, p, p.y, p.d1) && operand_map(&m.z, p, p.z, p.d2);
        if (!sum) {
            ok = ok && operand_map(&m.x, p, p.x, p.d1);
            ok = ok && rows_map(&m.o, p.o, p.o_f32, p.B, p.T, p.H, p.d2, (long long)p.T * p.H * p.d2, (long long)p.H * p.d2, p.d2, 32);
        }
        if (!ok) return cudaErrorInvalidValue;
    }
    const DecayPass &p = set.p[0];
    const int bytes = sum ? (int)SumLayout<D1, D2>::BYTES : (int)PassLayout<D1, D2>::BYTES;
    const int threads = sum ? SumLayout<D1, D2>::THREADS : PassLayout<D1, D2>::THREADS;
    auto kern = sum ? decay_sum_tc_kernel<D1, D2> : decay_pass_tc_kernel<D1, D2>;
    // once per device and kernel: the shared memory limit, and the register count that the shares rely on
    static bool ready[2][64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 64 || !ready[sum][dev]) {
        if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return err;
        cudaFuncAttributes attr;
        if ((err = cudaFuncGetAttributes(&attr, kern)) != cudaSuccess) return err;
        if (attr.numRegs * threads < (sum ? (int)SumLayout<D1, D2>::SHARES : (int)PassLayout<D1, D2>::SHARES)) return cudaErrorInvalidKernelImage;
        if (dev < 64) ready[sum][dev] = true;
    }
    return dependent_launch(kern, dim3(set.count * p.nseg, p.H, p.B), threads, bytes, s, set.dependent, set, maps);
}

}  // namespace

cudaError_t launch_decay_tc(const DecayPassSet &set, bool sum, cudaStream_t s) {
    const int d1 = decay_padded(set.p[0].d1), d2 = decay_padded(set.p[0].d2);
    if (d1 == 64) return d2 == 64 ? launch_one<64, 64>(set, sum, s) : launch_one<64, 128>(set, sum, s);
    return d2 == 64 ? launch_one<128, 64>(set, sum, s) : launch_one<128, 128>(set, sum, s);
}

// Read and clear these kernels' status word (PRISM_OK or PRISM_ERR_TIMEOUT).
cudaError_t decay_status(uint32_t *out) {
    uint32_t word = 0;
    cudaError_t err = cudaMemcpyFromSymbol(&word, g_decay_status, sizeof word);
    if (err != cudaSuccess) return err;
    if (word != 0) {
        const uint32_t zero = 0;
        if ((err = cudaMemcpyToSymbol(g_decay_status, &zero, sizeof zero)) != cudaSuccess) return err;
    }
    *out = word;
    return cudaSuccess;
}

}  // namespace prism
