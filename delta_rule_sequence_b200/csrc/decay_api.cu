// decay_api.cu -- the C entry points of the decay scan: argument checks, the segment plan, the launches.

#include <algorithm>
#include <initializer_list>

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
    const bool empty = s.B == 0 || s.T == 0 || heads == 0;
    for (int i = 0; i < 3; ++i) {
        r[i] = is_dense || n[i] <= 1 ? dense[i] : st[i];
        if (n[i] > 1 && !empty && (r[i] <= 0 || r[i] % unit || r[i] >= 1LL << 36)) return false;
        if (n[i] > 1) last += (n[i] - 1) * r[i];
    }
    out->t = DecayTensor{p, r[0], r[1], r[2], heads > 0 ? s.H / heads : 1};
    out->extent = empty ? 0 : (size_t)last * io_bytes(s.io);
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
    if (s->B > 65535 || s->H > 65535 || (long long)s->B * s->H > (1 << 24) || s->T > (1 << 26)) return PRISM_ERR_UNSUPPORTED;
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

// Segments per sequence, for a launch of `passes` passes.  One CTA per SM walks one segment, chunk after
// chunk; starting one costs about kStart chunks.  Full sequences: the time is about (waves of CTAs) x (chunks
// of a segment + kStart).  A padded batch, whose lengths only the device knows, is taken to be half full: CTAs
// behind their sequence's end leave at once, so the work spreads evenly and ends with one whole segment more.
// (32 x 4 sequences of up to 8192 tokens, 64 wide, random lengths: one segment each 205 us, eight 174 us.)
struct DecayPlan {
    int chunk, nseg, seg_tokens;
};
constexpr int kStart = 2;

DecayPlan plan_of(const prism_decay_shape &s, int passes, bool padded) {
    const int chunk = s.io == PRISM_F32 ? kDecayChunkSimt : kDecayChunkTc;
    const int nch = std::max(1, (s.T + chunk - 1) / chunk);
    const long long ctas = std::max(1LL, (long long)s.B * s.H * passes);
    const int sms = sm_count();
    DecayPlan best{chunk, 1, nch * chunk};
    long long least = 0;
    for (int want = 1; want <= std::min(nch, 128); ++want) {
        const int per = (nch + want - 1) / want, nseg = (nch + per - 1) / per;
        const long long cost = padded ? ctas * nseg * (per + kStart) / (2 * sms) + per + kStart
                                      : (ctas * nseg + sms - 1) / sms * (per + kStart);
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

// fp32 gradients of k or v (width d) per query head, where heads share keys and values.
size_t shared_grad_bytes(const prism_decay_shape &s, int d) {
    if (s.H == 0 || s.Hkv == s.H) return 0;
    return align256((size_t)s.B * s.T * s.H * d * 4);
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
    bool launched = false;  // a kernel of this call is in the stream

    bool f32() const { return s.io == PRISM_F32; }
    DecayPass common(int d1, int d2, bool reverse) const {
        DecayPass p{};
        p.B = s.B; p.H = s.H; p.T = s.T; p.d1 = d1; p.d2 = d2;
        p.decay = decay; p.lengths = lengths; p.reverse = reverse;
        p.nseg = pl.nseg; p.seg_tokens = pl.seg_tokens;
        p.stall = (debug_flags() & kDebugStallDecay) != 0;
        return p;
    }
    DecayPass sum(const DecayTensor &y, const DecayTensor &z, int d1, int d2, bool reverse, float *F) const {
        DecayPass p = common(d1, d2, reverse);
        p.y = y; p.z = z; p.F = F;
        return p;
    }
    DecayPass pass(const DecayTensor &x, const DecayTensor &y, const DecayTensor &z, int d1, int d2, const float *entry,
                   bool entry_t, bool reverse, void *o, bool o_f32) const {
        DecayPass p = common(d1, d2, reverse);
        p.x = x; p.y = y; p.z = z; p.entry = entry; p.entry_t = entry_t; p.o = o; p.o_f32 = o_f32;
        return p;
    }
    // one launch for neighbours of the same padded widths
    void run(std::initializer_list<DecayPass> list, bool sum) {
        DecayPassSet set{};
        for (const DecayPass *p = list.begin(); p != list.end(); ++p) {
            set.p[set.count++] = *p;
            const bool more = p + 1 != list.end() && decay_padded(p[1].d1) == decay_padded(p->d1) &&
                              decay_padded(p[1].d2) == decay_padded(p->d2);
            if (more && set.count < kDecaySet) continue;
            set.dependent = launched;
            launched = true;
            if (err == cudaSuccess) err = f32() ? launch_decay_simt(set, sum, stream) : launch_decay_tc(set, sum, stream);
            set.count = 0;
        }
    }
    void carry(std::initializer_list<DecayCarryOne> list) {
        DecayCarry c{s.B * s.H, s.H, s.T, s.dk * s.dv, pl.nseg, pl.seg_tokens, decay, lengths, 0, launched, {}};
        launched = true;
        for (const DecayCarryOne &o : list) c.c[c.count++] = o;
        if (err == cudaSuccess) err = launch_decay_carry(c, stream);
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
    *bytes = std::max<size_t>(256, std::max(sums_bytes(*shape, plan_of(*shape, 1, false)), sums_bytes(*shape, plan_of(*shape, 1, true))));
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
    if (outputs_alias(outs, 3, ins, 6)) return PRISM_ERR_INVALID_ARG;
    if (s.B == 0 || s.H == 0) return PRISM_OK;
    Runner r{s, plan_of(s, 1, lengths != nullptr), decay, lengths, (cudaStream_t)stream};
    float *F = (float *)workspace;
    if (s.T == 0) {
        r.copy_state(S_final, S0);
    } else {
        const bool cut = r.pl.nseg > 1;
        if (cut || S_final) r.run({r.sum(c.k.t, c.v.t, s.dk, s.dv, false, F)}, true);
        if (cut) r.carry({{0, S0, F, S_final}});
        r.run({r.pass(c.q.t, c.k.t, c.v.t, s.dk, s.dv, cut ? F : S0, false, false, o, s.io == PRISM_F32)}, false);
        // after the pass, which reads S0: S_final may be S0
        if (!cut && S_final) r.carry({{0, S0, F, S_final}});
    }
    probe_finish((cudaStream_t)stream);
    return cuda_status(r.err);
}

prism_status prism_decay_scan_bwd_workspace_size(const prism_decay_shape *shape, size_t *bytes) {
    if (!bytes) return PRISM_ERR_INVALID_ARG;
    const prism_status st = check_shape(shape);
    if (st != PRISM_OK) return st;
    *bytes = std::max<size_t>(256, 2 * std::max(sums_bytes(*shape, plan_of(*shape, 3, false)), sums_bytes(*shape, plan_of(*shape, 3, true))) +
                                       shared_grad_bytes(*shape, shape->dk) +
                                       shared_grad_bytes(*shape, shape->dv));
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
    if (outputs_alias(outs, 5, ins, 8)) return PRISM_ERR_INVALID_ARG;
    if (s.B == 0 || s.H == 0) return PRISM_OK;
    Runner r{s, plan_of(s, 3, lengths != nullptr), decay, lengths, (cudaStream_t)stream};
    if (s.T == 0) {
        r.copy_state(dS0, dS_final);
    } else {
        const bool cut = r.pl.nseg > 1, f32 = s.io == PRISM_F32, shared = s.Hkv != s.H;
        const size_t sb = sums_bytes(s, r.pl);
        char *ws = (char *)workspace;
        float *FS = (float *)ws, *FG = (float *)(ws + sb), *dk_part = (float *)(ws + 2 * sb),
              *dv_part = (float *)(ws + 2 * sb + shared_grad_bytes(s, s.dk));
        const DecayTensor g = dense(s, dO, s.dv);
        const DecayPass sum_S = r.sum(c.k.t, c.v.t, s.dk, s.dv, false, FS), sum_G = r.sum(c.q.t, g, s.dk, s.dv, true, FG);
        if (cut) {
            r.run({sum_S, sum_G}, true);
            r.carry({{0, S0, FS, nullptr}, {1, dS_final, FG, dS0}});
        } else if (dS0) {
            r.run({sum_G}, true);
            r.carry({{1, dS_final, FG, dS0}});
        }
        const float *ES = cut ? FS : S0, *EG = cut ? FG : dS_final;
        r.run({r.pass(g, c.v.t, c.k.t, s.dv, s.dk, ES, true, false, dq, f32),
               r.pass(c.v.t, g, c.q.t, s.dv, s.dk, EG, true, true, shared ? dk_part : dk, shared || f32),
               r.pass(c.k.t, c.q.t, g, s.dk, s.dv, EG, false, true, shared ? dv_part : dv, shared || f32)},
              false);
        if (shared && r.err == cudaSuccess)
            r.err = launch_decay_group_sum({(long long)s.B * s.T * s.Hkv, s.H / s.Hkv, {dk_part, dv_part}, {dk, dv}, {s.dk, s.dv}},
                                           f32, r.stream);
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
