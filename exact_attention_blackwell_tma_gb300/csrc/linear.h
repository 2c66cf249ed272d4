// Linear attention with a decay per head: parameters and launchers of its kernels.
//
// One form serves the forward and the three gradients. Over the positions r =
// 0 .. n - 1 of a sequence (its tokens in order, or backwards),
//   out_i = out_mul (sum_{j <= i} decay^(i-j) <a_i, b_j> c_j + decay^(i+1-e) a_i^T X)
//   X'    = decay^n X + sum_j decay^(n-1-j+e) b_j c_j^T
// with X the state carried in (times init_mul) and X' the one carried out:
//   o   a = q,  b = k,  c = v,  X = S_0,     e = 0               X' = S_n
//   dq  a = dO, b = v,  c = k,  X = S_0^T,   e = 0
//   dk  a = v,  b = dO, c = q,  X = dS_n^T,  e = 1, backwards
//   dv  a = k,  b = q,  c = dO, X = dS_n,    e = 1, backwards    X' = dS_0 / scale
// (dS is the gradient of the state behind a token; that of the state in front of
// it has one more factor of decay, hence e.) Grouped heads: `per` query heads
// share a state. o and dq have an output for each (a differs), dk and dv sum over
// them (b and c differ).
#pragma once

#include "kernels.h"

namespace attn {

constexpr int kLinChunk = 64;   // tokens of a chunk: pairs within it, the state across chunks

struct LinParams {
    const __nv_bfloat16 *a, *b, *c;
    long a_stride, b_stride, c_stride;   // elements between tokens
    __nv_bfloat16* out;                  // tokens of heads x DV, contiguous
    const float* log_decay;              // [Hkv], natural log
    const float* init;                   // [B][Hkv][DK][DV] ([DV][DK] with init_trans), or null
    float* final;                        // [B][Hkv][DK][DV], or null
    float* states;                       // workspace: [segments][Hkv][DK][DV] (segments > 1 for some sequence)
    const int* cu;                       // row offsets, or null (dense)
    int B, rows, total;                  // rows per sequence (dense), rows in all
    int Hkv, per, DK, DV;
    int seg_rows;                        // a segment: what one CTA walks, a multiple of the chunk
    int segments;                        // upper bound of the segments of all sequences
    int init_trans, reverse, e;
    float out_mul, init_mul, final_mul;
    int* status;
};

// Segments. A sequence of n rows has ceil(n / seg_rows), at least one, numbered
// from lin_seg_start on: that leaves gaps but needs no scan over the lengths.
struct LinPlan {
    int seg_rows, segments;
    bool split;   // some sequence may have more than one segment
};
LinPlan lin_plan(int B, int Hkv, int L, bool packed, int d, int dv);

// sum: b and c differ per query head (dk, dv), otherwise a and out do (o, dq)
cudaError_t launch_linear(const LinParams& p, bool split, bool sum, cudaStream_t stream);

struct LinStepParams {
    const __nv_bfloat16 *q, *k, *v;
    long q_stride, k_stride, v_stride;
    const float* log_decay;
    float* state;
    __nv_bfloat16* o;
    int B, Hkv, per, d, dv;
    float scale;
};
cudaError_t launch_linear_step(const LinStepParams& p, cudaStream_t stream);

}  // namespace attn
