// decay.cuh -- the decay scan (linear attention with one fixed decay per head): arguments and
// launchers shared by its kernels and its C entry points.
//
//   S_t = a_h S_{t-1} + v_t k_t^T,   o_t = S_t q_t
//
// Every output of the forward and of the backward pass is one "pass" over the tokens with three
// operands x, y [T, d1] and z [T, d2] of a head and a carried state R [d2, d1]:
//   o_i = sum_{j <= i} a^(i-j) (x_i . y_j) z_j + (decayed entry state) x_i
// With n tokens in a chunk, entry state R and the exit state R':
//   forward in time:   o_i = sum_{j<=i} a^(i-j) (x_i.y_j) z_j + a^(i+1) R x_i,
//                      R' = a^n R + sum_j a^(n-1-j) z_j y_j^T
//   backward in time:  o_i = sum_{j>=i} a^(j-i) (x_i.y_j) z_j + a^(n-1-i) R x_i,
//                      R' = a^n R + sum_j a^(j+1) z_j y_j^T
//   o  : (x, y, z) = (q, k, v),  forward,  R = S
//   dq : (dO, v, k),             forward,  R = S^T
//   dk : (v, dO, q),             backward, R = G^T      (G_t = a G_{t+1} + dO_t q_t^T)
//   dv : (k, q, dO),             backward, R = G
// so the backward pass runs on the forward's kernels.
//
// The tokens are cut into segments of whole chunks, so that few sequences still fill the GPU:
//   1. the sum kernel: every segment's contribution F = sum_j a^(...) z_j y_j^T to the state,
//   2. the carry kernel: the segments' entry states from the F (and the exit state),
//   3. the pass kernel: every segment's outputs from its entry state.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "dependent.cuh"

namespace prism {

// One operand [B, T, heads, d] with unit stride along d; head h of the scan reads head h / div.
struct DecayTensor {
    const void *p;
    long long sb, st, sh;  // elements between batches, tokens, heads
    int div;
};

struct DecayPass {
    int B, H, T, d1, d2;
    DecayTensor x, y, z;  // widths d1, d1, d2
    void *o;              // dense [B, T, H, d2]: io type, or fp32 when o_f32
    int o_f32;
    const float *decay;
    const int *lengths;   // or null: every sequence has T tokens
    // entry state of (b, h, segment): null (zero) or fp32 matrices one after the other,
    // R[n][m] at n * d1 + m, or at m * d2 + n when entry_t
    const float *entry;
    int entry_t;
    float *F;             // sum kernel's output, [B, H, nseg] matrices [d2][d1]
    int reverse;
    int nseg, seg_tokens; // segments per sequence, tokens per segment (whole chunks)
    int stall;            // the give-up test: no load is issued, every wait runs out after a short limit
};

// Valid tokens of sequence b.
__device__ __forceinline__ int decay_len(const int *lengths, int b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

// a^n for a whole n >= 0 (0^0 = 1), by squaring in 64 bits: with a near 1 and n in the thousands 32 bits would
// lose the last digits of the power.  (exp2(n log2 a) in 64 bits took 1.5 us of a CTA's start.)
__device__ __forceinline__ float decay_pow(float a, int n) {
    double r = 1.0, s = (double)a;
    for (; n > 0; n >>= 1, s *= s)
        if (n & 1) r *= s;
    return (float)r;
}

// Passes (or segment sums) of one launch, all of the same B, H, T, lengths and segments: the CTAs of one
// after those of the other, grid {count * nseg, H, B}.
constexpr int kDecaySet = 3;
struct DecayPassSet {
    int count;
    bool dependent;  // not the first kernel of its call
    DecayPass p[kDecaySet];
};

// Width that a kernel is built for.
inline int decay_padded(int d) { return d <= 64 ? 64 : 128; }

constexpr int kDecayChunkSimt = 64, kDecayChunkTc = 128;  // tokens of a chunk

// fp32 operands, on CUDA cores; bf16 operands, on the tensor cores.
// Every pass of a set has the same padded widths (decay_padded).
cudaError_t launch_decay_simt(const DecayPassSet &set, bool sum, cudaStream_t s);
cudaError_t launch_decay_tc(const DecayPassSet &set, bool sum, cudaStream_t s);
cudaError_t decay_status(uint32_t *out);  // read and clear the tensor-core kernels' status word

// Entry states of every segment from the segments' sums, in place of them, and the exit state.
struct DecayCarryOne {
    int reverse;
    const float *init;        // [BH][elems] or null (zero)
    float *F;                 // [BH][nseg][elems]: sums in, entry states out
    float *final_state;       // [BH][elems] or null
};
struct DecayCarry {
    int BH, H, T, elems;      // elems = d1 * d2
    int nseg, seg_tokens;
    const float *decay;
    const int *lengths;
    int count;
    bool dependent;
    DecayCarryOne c[2];
};
cudaError_t launch_decay_carry(const DecayCarry &c, cudaStream_t s);

// out[b,t,g,:] = sum over the `div` heads of group g of part[b,t,g*div + i,:] (fp32 -> io), for dk and dv.
struct DecayGroupSum {
    long long groups;         // B * T * Hkv
    int div;
    const float *part[2];
    void *out[2];
    int d[2];
};
cudaError_t launch_decay_group_sum(const DecayGroupSum &g, bool io_f32, cudaStream_t s);

cudaError_t launch_decay_step(int B, int H, int dk, int dv, const DecayTensor &q, const DecayTensor &k,
                              const DecayTensor &v, const float *decay, float *S, void *o, bool io_f32,
                              cudaStream_t s);

}  // namespace prism
