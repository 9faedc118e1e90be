// decay_api.cu -- the C entry points of the decay scan: argument checks, the segment plan, the launches.

#include <algorithm>

#include "api.cuh"
#include "decay.cuh"

namespace prism {
namespace {

// prism_debug_set_flags bit 8: the stall test of the tensor-core kernels.
constexpr int kDebugStallDecay = 256;

size_t io_bytes(prism_dtype io) { return io == PRISM_F32 ? 4 : 2; }

// One operand as the kernels read it, and the bytes from its first to behind its last element.
struct Operand {
    DecayTensor t;
    size_t extent;
};

// Strides of an operand [B, T, heads, d]: all zero stands for the dense layout; along an extent of 0 or 1
// nothing is stepped over and any value goes.  False where a stride does not keep rows 16-byte aligned.
bool make_operand(const prism_decay_shape &s, const void *p, const long long (&st)[3], int heads, int d, Operand *out) {
    const long long dense[3] = {(long long)s.T * heads * d, (long long)heads * d, d};
    const long long n[3] = {s.B, s.T, heads};
    const bool is_dense = st[0] == 0 && st[1] == 0 && st[2] == 0;
    const long long unit = 16 / (long long)io_bytes(s.io);
    long long r[3], last = d;
    for (int i = 0; i < 3; ++i) {
        r[i] = is_dense || n[i] <= 1 ? dense[i] : st[i];
        if (n[i] > 1 && s.T > 0 && (r[i] <= 0 || r[i] % unit || r[i] >= (1LL << 40) / 4)) return false;
        if (n[i] > 1) last += (n[i] - 1) * r[i];
    }
    out->t = DecayTensor{p, r[0], r[1], r[2], heads > 0 ? s.H / heads : 1};
    out->extent = (size_t)last * io_bytes(s.io);
    return true;
}

struct DecayCall {
    Operand q, k, v;
    bool work;  // there is a token to process
};

prism_status check_shape(const prism_decay_shape *s) {
    if (!s) return PRISM_ERR_INVALID_ARG;
    if (s->B < 0 || s->H < 0 || s->Hkv < 0 || s->T < 0 || s->dk < 1 || s->dv < 1) return PRISM_ERR_INVALID_ARG;
    if (s->io != PRISM_BF16 && s->io != PRISM_F32) return PRISM_ERR_INVALID_ARG;
    if (s->H > 0 && (s->Hkv < 1 || s->H % s->Hkv)) return PRISM_ERR_INVALID_ARG;
    if (!width_ok(s->dk) || !width_ok(s->dv)) return PRISM_ERR_UNSUPPORTED;
    if (s->B > 65535 || s->H > 65535 || (long long)s->B * s->H > (1 << 24)) return PRISM_ERR_UNSUPPORTED;
    return PRISM_OK;
}

prism_status check_call(const prism_decay_shape *s, const void *q, const void *k, const void *v, const float *decay,
                        DecayCall *c) {
    prism_status st = check_shape(s);
    if (st != PRISM_OK) return st;
    c->work = (long long)s->B * s->H * s->T > 0;
    if (!make_operand(*s, q, s->q_stride, s->H, s->dk, &c->q) || !make_operand(*s, k, s->k_stride, s->Hkv, s->dk, &c->k) ||
        !make_operand(*s, v, s->v_stride, s->Hkv, s->dv, &c->v))
        return PRISM_ERR_INVALID_ARG;
    if (!c->work) return PRISM_OK;
    if (!q || !k || !v || !decay) return PRISM_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || ((uintptr_t)decay & 3u)) return PRISM_ERR_INVALID_ARG;
    return PRISM_OK;
}

// Segments per sequence.  One CTA per SM walks one segment, chunk after chunk, so a plan's time is about
// (waves of CTAs) x (chunks of a segment + what starting one costs, about kStart chunks).
struct DecayPlan {
    int chunk, nseg, seg_tokens;
};
constexpr int kStart = 2;

DecayPlan plan_of(const prism_decay_shape &s) {
    const int chunk = s.io == PRISM_F32 ? kDecayChunkSimt : kDecayChunkTc;
    const int nch = std::max(1, (s.T + chunk - 1) / chunk);
    const long long bh = std::max(1LL, (long long)s.B * s.H);
    const int sms = sm_count();
    DecayPlan best{chunk, 1, nch * chunk};
    long long least = 0;
    for (int want = 1; want <= std::min(nch, 128); ++want) {
        const int per = (nch + want - 1) / want, nseg = (nch + per - 1) / per;
        const long long cost = (bh * nseg + sms - 1) / sms * (per + kStart);
        if (want == 1 || cost < least) {
            least = cost;
            best = DecayPlan{chunk, nseg, per * chunk};
        }
    }
    return best;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

size_t sums_bytes(const prism_decay_shape &s, const DecayPlan &pl) {
    return align256((size_t)s.B * s.H * pl.nseg * s.dk * s.dv * 4);
}

// fp32 gradients of one operand per query head, where heads share keys and values.
size_t shared_grad_bytes(const prism_decay_shape &s) {
    if (s.H == 0 || s.Hkv == s.H) return 0;
    return align256((size_t)s.B * s.T * s.H * std::max(s.dk, s.dv) * 4);
}

DecayTensor dense(const prism_decay_shape &s, const void *p, int d) {
    return DecayTensor{p, (long long)s.T * s.H * d, (long long)s.H * d, d, 1};
}

struct Runner {
    const prism_decay_shape &s;
    DecayPlan pl;
    const float *decay;
    const int *lengths;
    cudaStream_t stream;
    cudaError_t err = cudaSuccess;

    bool f32() const { return s.io == PRISM_F32; }
    void sum(const DecayTensor &y, const DecayTensor &z, int d1, int d2, bool reverse, float *F) {
        if (err != cudaSuccess) return;
        DecayPass p{};
        p.B = s.B; p.H = s.H; p.T = s.T; p.d1 = d1; p.d2 = d2;
        p.y = y; p.z = z; p.decay = decay; p.lengths = lengths;
        p.F = F; p.reverse = reverse; p.nseg = pl.nseg; p.seg_tokens = pl.seg_tokens;
        p.stall = (debug_flags() & kDebugStallDecay) != 0;
        err = f32() ? launch_decay_sum_simt(p, stream) : launch_decay_sum_tc(p, stream);
    }
    void carry(float *F, const float *init, float *final_state, bool reverse) {
        if (err != cudaSuccess) return;
        DecayCarry c{s.B * s.H, s.H, s.T, s.dk * s.dv, pl.nseg, pl.seg_tokens, reverse ? 1 : 0, decay, lengths, init, F, final_state};
        err = launch_decay_carry(c, stream);
    }
    void pass(const DecayTensor &x, const DecayTensor &y, const DecayTensor &z, int d1, int d2, const float *entry,
              bool entry_t, bool reverse, void *o, bool o_f32) {
        if (err != cudaSuccess) return;
        DecayPass p{};
        p.B = s.B; p.H = s.H; p.T = s.T; p.d1 = d1; p.d2 = d2;
        p.x = x; p.y = y; p.z = z; p.decay = decay; p.lengths = lengths;
        p.entry = entry; p.entry_t = entry_t; p.reverse = reverse; p.o = o; p.o_f32 = o_f32;
        p.nseg = pl.nseg; p.seg_tokens = pl.seg_tokens;
        p.stall = (debug_flags() & kDebugStallDecay) != 0;
        err = f32() ? launch_decay_pass_simt(p, stream) : launch_decay_pass_tc(p, stream);
    }
    // a state without tokens: out = init or zero
    void copy_state(float *out, const float *init) {
        if (err != cudaSuccess || !out || out == init) return;
        const size_t n = (size_t)s.B * s.H * s.dk * s.dv * 4;
        err = init ? cudaMemcpyAsync(out, init, n, cudaMemcpyDeviceToDevice, stream) : cudaMemsetAsync(out, 0, n, stream);
    }
};

}  // namespace
}  // namespace prism

using namespace prism;

extern "C" {

prism_status prism_decay_scan_fwd_workspace_size(const prism_decay_shape *shape, size_t *bytes) {
    if (!bytes) return PRISM_ERR_INVALID_ARG;
    const prism_status st = check_shape(shape);
    if (st != PRISM_OK) return st;
    *bytes = std::max<size_t>(256, sums_bytes(*shape, plan_of(*shape)));
    return PRISM_OK;
}

prism_status prism_decay_scan_fwd(const prism_decay_shape *shape, const void *q, const void *k, const void *v,
                                  const float *decay, const float *S0, const int *lengths, void *o, float *S_final,
                                  void *workspace, size_t ws_bytes, void *stream) {
    DecayCall c;
    prism_status st = check_call(shape, q, k, v, decay, &c);
    if (st != PRISM_OK) return st;
    const prism_decay_shape &s = *shape;
    if ((S0 && !aligned16(S0)) || (S_final && !aligned16(S_final)) || ((uintptr_t)lengths & 3u)) return PRISM_ERR_INVALID_ARG;
    if (c.work && (!o || !aligned16(o))) return PRISM_ERR_INVALID_ARG;
    size_t need = 0;
    prism_decay_scan_fwd_workspace_size(shape, &need);
    if (!workspace || ws_bytes < need || ((uintptr_t)workspace & 255u)) return PRISM_ERR_INVALID_ARG;
    const size_t state = (size_t)s.B * s.H * s.dk * s.dv * 4;
    const ByteRange outs[] = {{o, (size_t)s.B * s.T * s.H * s.dv * io_bytes(s.io)}, {S_final, state}, {workspace, need}};
    const ByteRange ins[] = {{q, c.q.extent}, {k, c.k.extent}, {v, c.v.extent}, {decay, (size_t)s.H * 4},
                         {lengths, (size_t)s.B * 4}, {S_final == S0 ? nullptr : S0, state}};
    if (c.work && outputs_alias(outs, 3, ins, 6)) return PRISM_ERR_INVALID_ARG;
    if (s.B == 0 || s.H == 0) return PRISM_OK;
    Runner r{s, plan_of(s), decay, lengths, (cudaStream_t)stream};
    float *F = (float *)workspace;
    if (s.T == 0) {
        r.copy_state(S_final, S0);
    } else {
        const bool cut = r.pl.nseg > 1;
        if (cut || S_final) r.sum(c.k.t, c.v.t, s.dk, s.dv, false, F);
        if (cut) r.carry(F, S0, S_final, false);
        r.pass(c.q.t, c.k.t, c.v.t, s.dk, s.dv, cut ? F : S0, false, false, o, s.io == PRISM_F32);
        // after the pass, which reads S0: S_final may be S0
        if (!cut && S_final) r.carry(F, S0, S_final, false);
    }
    probe_finish((cudaStream_t)stream);
    return cuda_status(r.err);
}

prism_status prism_decay_scan_bwd_workspace_size(const prism_decay_shape *shape, size_t *bytes) {
    if (!bytes) return PRISM_ERR_INVALID_ARG;
    const prism_status st = check_shape(shape);
    if (st != PRISM_OK) return st;
    *bytes = std::max<size_t>(256, 2 * sums_bytes(*shape, plan_of(*shape)) + shared_grad_bytes(*shape));
    return PRISM_OK;
}

prism_status prism_decay_scan_bwd(const prism_decay_shape *shape, const void *q, const void *k, const void *v,
                                  const float *decay, const float *S0, const int *lengths, const void *dO,
                                  const float *dS_final, void *dq, void *dk, void *dv, float *dS0, void *workspace,
                                  size_t ws_bytes, void *stream) {
    DecayCall c;
    prism_status st = check_call(shape, q, k, v, decay, &c);
    if (st != PRISM_OK) return st;
    const prism_decay_shape &s = *shape;
    if ((S0 && !aligned16(S0)) || (dS_final && !aligned16(dS_final)) || (dS0 && !aligned16(dS0)) || ((uintptr_t)lengths & 3u))
        return PRISM_ERR_INVALID_ARG;
    for (const void *g : {dO, (const void *)dq, (const void *)dk, (const void *)dv})
        if (c.work && (!g || !aligned16(g))) return PRISM_ERR_INVALID_ARG;
    size_t need = 0;
    prism_decay_scan_bwd_workspace_size(shape, &need);
    if (!workspace || ws_bytes < need || ((uintptr_t)workspace & 255u)) return PRISM_ERR_INVALID_ARG;
    const size_t state = (size_t)s.B * s.H * s.dk * s.dv * 4, rows = (size_t)s.B * s.T * io_bytes(s.io);
    const ByteRange outs[] = {{dq, rows * s.H * s.dk}, {dk, rows * s.Hkv * s.dk}, {dv, rows * s.Hkv * s.dv}, {dS0, state},
                          {workspace, need}};
    const ByteRange ins[] = {{q, c.q.extent}, {k, c.k.extent}, {v, c.v.extent}, {decay, (size_t)s.H * 4}, {lengths, (size_t)s.B * 4},
                         {S0, state}, {dO, rows * s.H * s.dv}, {dS_final, state}};
    if (c.work && outputs_alias(outs, 5, ins, 8)) return PRISM_ERR_INVALID_ARG;
    if (s.B == 0 || s.H == 0) return PRISM_OK;
    Runner r{s, plan_of(s), decay, lengths, (cudaStream_t)stream};
    if (s.T == 0) {
        r.copy_state(dS0, dS_final);
    } else {
        const bool cut = r.pl.nseg > 1, f32 = s.io == PRISM_F32, shared = s.Hkv != s.H;
        const size_t sb = sums_bytes(s, r.pl);
        float *FS = (float *)workspace, *FG = (float *)((char *)workspace + sb), *part = (float *)((char *)workspace + 2 * sb);
        const DecayTensor g = dense(s, dO, s.dv);
        const long long tokens = (long long)s.B * s.T;
        if (cut) {
            r.sum(c.k.t, c.v.t, s.dk, s.dv, false, FS);
            r.carry(FS, S0, nullptr, false);
        }
        if (cut || dS0) {
            r.sum(c.q.t, g, s.dk, s.dv, true, FG);
            r.carry(FG, dS_final, dS0, true);
        }
        const float *ES = cut ? FS : S0, *EG = cut ? FG : dS_final;
        r.pass(g, c.v.t, c.k.t, s.dv, s.dk, ES, true, false, dq, f32);
        r.pass(c.v.t, g, c.q.t, s.dv, s.dk, EG, true, true, shared ? part : dk, shared || f32);
        if (shared && r.err == cudaSuccess)
            r.err = launch_decay_group_sum(part, dk, tokens, s.Hkv, s.H / s.Hkv, s.dk, f32, r.stream);
        r.pass(c.k.t, c.q.t, g, s.dk, s.dv, EG, false, true, shared ? part : dv, shared || f32);
        if (shared && r.err == cudaSuccess)
            r.err = launch_decay_group_sum(part, dv, tokens, s.Hkv, s.H / s.Hkv, s.dv, f32, r.stream);
    }
    probe_finish((cudaStream_t)stream);
    return cuda_status(r.err);
}

prism_status prism_decay_step(const prism_decay_shape *shape, const void *q, const void *k, const void *v,
                              const float *decay, float *S, void *o, void *stream) {
    DecayCall c;
    prism_status st = check_call(shape, q, k, v, decay, &c);
    if (st != PRISM_OK) return st;
    const prism_decay_shape &s = *shape;
    if (s.T != 1) return PRISM_ERR_INVALID_ARG;
    if (s.B == 0 || s.H == 0) return PRISM_OK;
    if (!S || !aligned16(S) || !o || !aligned16(o)) return PRISM_ERR_INVALID_ARG;
    const ByteRange outs[] = {{o, (size_t)s.B * s.H * s.dv * io_bytes(s.io)}, {S, (size_t)s.B * s.H * s.dk * s.dv * 4}};
    const ByteRange ins[] = {{q, c.q.extent}, {k, c.k.extent}, {v, c.v.extent}, {decay, (size_t)s.H * 4}};
    if (outputs_alias(outs, 2, ins, 4)) return PRISM_ERR_INVALID_ARG;
    const cudaError_t err = launch_decay_step(s.B, s.H, s.dk, s.dv, c.q.t, c.k.t, c.v.t, decay, S, o, s.io == PRISM_F32,
                                              (cudaStream_t)stream);
    probe_finish((cudaStream_t)stream);
    return cuda_status(err);
}

}  // extern "C"
