// decay_step.cu -- one token of the decay scan for every sequence: S <- a S + v k^T in place, o = S q.
//
// Memory-bound: the fp32 state is read once and written once, everything else is a few hundred bytes
// per head.  A row of dk floats is spread over dk / 4 lanes (one 16-byte vector each); a warp takes four vectors
// per lane, 2 KB of state, all of them loaded before any is used.  256 x 32 heads of 128 x 128: 171 us, 6.3 TB/s
// (the copy bandwidth is 6.55).  Measured around it: 8 vectors per lane 192 us, 16 204, 2 198 (at 256 threads
// a block; 4 there: 176), blocks of 512 threads 186.

#include "decay.cuh"

namespace prism {
namespace {

constexpr int NT = 128;

constexpr int kLoads = 4;  // 16-byte vectors of a lane

template <typename IO>
struct StepArgs {
    int B, H, dv;
    DecayTensor q, k, v;
    const float *decay;
    float *S;
    IO *o;
};

template <typename IO, int DK>
__global__ void __launch_bounds__(NT) decay_step_kernel(StepArgs<IO> p) {
    constexpr int LR = DK / 4;        // lanes of a row
    constexpr int PER = 32 / LR;      // rows of one load
    constexpr int NL = kLoads, ROWS = NL * PER;
    const int lane = threadIdx.x & 31;
    const int wph = p.dv / ROWS;      // warps of a head
    const long long warp = (long long)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
    const long long bh = warp / wph;
    if (bh >= (long long)p.B * p.H) return;
    const int b = (int)(bh / p.H), h = (int)(bh % p.H);
    const int r0 = (int)(warp % wph) * ROWS + lane / LR, c0 = (lane % LR) * 4;
    float *S = p.S + (bh * p.dv + r0) * DK + c0;
    float4 s[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) s[i] = __ldcs(reinterpret_cast<const float4 *>(S + (long long)i * PER * DK));
    const IO *q = (const IO *)p.q.p + b * p.q.sb + (long long)(h / p.q.div) * p.q.sh + c0;
    const IO *k = (const IO *)p.k.p + b * p.k.sb + (long long)(h / p.k.div) * p.k.sh + c0;
    const IO *v = (const IO *)p.v.p + b * p.v.sb + (long long)(h / p.v.div) * p.v.sh + r0;
    const float a = p.decay[h];
    float qf[4], kf[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        qf[i] = ld_io(q, i);
        kf[i] = ld_io(k, i);
    }
    float dot[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const float vr = ld_io(v, i * PER);
        s[i].x = fmaf(a, s[i].x, vr * kf[0]);
        s[i].y = fmaf(a, s[i].y, vr * kf[1]);
        s[i].z = fmaf(a, s[i].z, vr * kf[2]);
        s[i].w = fmaf(a, s[i].w, vr * kf[3]);
        __stcs(reinterpret_cast<float4 *>(S + (long long)i * PER * DK), s[i]);
        dot[i] = fmaf(s[i].x, qf[0], fmaf(s[i].y, qf[1], fmaf(s[i].z, qf[2], s[i].w * qf[3])));
    }
#pragma unroll
    for (int o = LR / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < NL; ++i) dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], o);
    if (lane % LR == 0) {
#pragma unroll
        for (int i = 0; i < NL; ++i) st_io(p.o, bh * p.dv + r0 + i * PER, dot[i]);
    }
}

template <typename IO, int DK>
cudaError_t launch_dk(const StepArgs<IO> &a, cudaStream_t s) {
    constexpr int ROWS = kLoads * (128 / DK);  // of a warp: 4, 8 or 16, which divide every dv
    const long long warps = (long long)a.B * a.H * (a.dv / ROWS);
    launch_probe_mark(s);
    decay_step_kernel<IO, DK><<<(unsigned)((warps + NT / 32 - 1) / (NT / 32)), NT, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t launch_io(int B, int H, int dk, int dv, const DecayTensor &q, const DecayTensor &k, const DecayTensor &v,
                      const float *decay, float *S, void *o, cudaStream_t s) {
    const StepArgs<IO> a{B, H, dv, q, k, v, decay, S, (IO *)o};
    switch (dk) {
        case 32: return launch_dk<IO, 32>(a, s);
        case 64: return launch_dk<IO, 64>(a, s);
        default: return launch_dk<IO, 128>(a, s);
    }
}

}  // namespace

cudaError_t launch_decay_step(int B, int H, int dk, int dv, const DecayTensor &q, const DecayTensor &k,
                              const DecayTensor &v, const float *decay, float *S, void *o, bool io_f32,
                              cudaStream_t s) {
    return io_f32 ? launch_io<float>(B, H, dk, dv, q, k, v, decay, S, o, s)
                  : launch_io<__nv_bfloat16>(B, H, dk, dv, q, k, v, decay, S, o, s);
}

}  // namespace prism
