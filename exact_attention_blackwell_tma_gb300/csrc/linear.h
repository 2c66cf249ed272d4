// Linear attention with a decay per head: parameters and launchers of its kernels.
//
// One form serves the forward and the three gradients. With the tokens of a sequence
// taken in order (o, dq) or from the last to the first (dk, dv: `back`), token i's
// position r, and D the decay,
//   out_i = out_mul (sum_{j at or before i} D^|r_i - r_j| <a_i, b_j> c_j + D^(r_i + 1 - back) a_i^T X)
//   X'    = D^n X + sum_j D^(n - 1 - r_j + back) b_j c_j^T
// where X is the state carried in (times init_mul) and X' the one carried out:
//   o   a = q,  b = k,  c = v,  X = S_0                    X' = S_n
//   dq  a = dO, b = v,  c = k,  X = S_0^T
//   dk  a = v,  b = dO, c = q,  X = dS_n^T / scale
//   dv  a = k,  b = q,  c = dO, X = dS_n / scale           X' = dS_0 / scale
// (dS is the gradient of the state behind a token; that of the state in front of
// it has one more factor of D, hence `back` in the exponents.) Grouped heads: `per`
// query heads share a state. o and dq have an output for each (a differs), dk and
// dv sum over them (b and c differ): `back` says that, too.
//
// Sequences are cut into segments, numbered and chunked from their first token in
// either direction; three kernels: what each segment adds to the state, the scan that
// turns this into the state each segment starts from, the outputs. A call whose
// sequences have one segment each, and that wants no state back, is the last one alone.
#pragma once

#include "kernels.h"
#include "ptx.cuh"

namespace attn {

struct LinParams {
    __nv_bfloat16* out;                  // tokens of heads x DV, contiguous
    const float* log_decay;              // [Hkv], natural log
    const float* init;                   // [B][Hkv][DK][DV] ([DV][DK] with init_trans), or null
    float* final;                        // [B][Hkv][DK][DV], or null
    float* states;                       // workspace: [segments][Hkv][DK][DV]
    const int* cu;                       // row offsets, or null (dense)
    int B, rows, total;                  // rows per sequence (dense), rows in all
    int Hkv, per, DK, DV;
    int seg_rows;                        // rows of a segment, a multiple of a chunk's
    int segments;                        // upper bound of the segments of all sequences
    int plan_split;                      // some sequence may have more than one
    int init_trans, states_trans;        // (states_trans: [segments][Hkv][DV][DK], the states of the transposed product)
    float out_mul, init_mul, final_mul;
    int* status;
    uint64_t wait_budget_ns;
    // whether the states go through the workspace (with `final`, whose buffer may be init's, they do)
    __host__ __device__ bool split() const { return plan_split || final; }
};

// Segments. A sequence of n rows has ceil(n / seg_rows), at least one, numbered
// from lin_seg_start on: that leaves gaps but needs no scan over the lengths.
struct LinPlan {
    int seg_rows, segments;
    bool split;   // some sequence may have more than one segment
};
LinPlan lin_plan(int B, int Hkv, int L, bool packed, int d, int dv, bool final);   // final: the last states are wanted

// Tensor maps, boxes of 64 channels of a head: a, b and c by 128 tokens, out by 32
struct LinMaps {
    CUtensorMap a, b, c, out;
};

// The states that the segments start from, and the last one (nothing to do without several segments or `final`); the outputs
cudaError_t launch_linear_states(const LinParams& p, const LinMaps& maps, bool back, int num_sms, cudaStream_t stream);
cudaError_t launch_linear_out(const LinParams& p, const LinMaps& maps, bool back, int num_sms, cudaStream_t stream);
// (the first half of the states: what each segment adds)
cudaError_t launch_linear_shares(const LinParams& p, const LinMaps& maps, bool back, int num_sms, cudaStream_t stream);

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

#ifdef __CUDACC__
// A segment of a sequence: rows [r0, r1) of its n, q0 its first row.
struct Segment {
    int b, q0, n, r0, r1;
    bool first, last, live;
};
__device__ __forceinline__ int lin_seg_start(const LinParams& p, int b) {
    return p.cu ? __ldg(p.cu + b) / p.seg_rows + b : b * max(1, (p.rows + p.seg_rows - 1) / p.seg_rows);
}
// Rows [q0, q0 + n) of sequence b. Offsets out of range make an empty sequence (reported).
__device__ __forceinline__ void lin_sequence(const LinParams& p, int b, int* q0, int* n) {
    if (!p.cu) {
        *q0 = b * p.rows;
        *n = p.rows;
        return;
    }
    *q0 = __ldg(p.cu + b);
    *n = __ldg(p.cu + b + 1) - *q0;
    if (*q0 < 0 || *n < 0 || *q0 > p.total - *n) {
        atomicCAS(p.status, kStatusOk, kStatusBadPage);
        *q0 = *n = 0;
    }
}
// (A start that is off for bad offsets only moves segments, which are then not live or read another one's state.)
__device__ __forceinline__ Segment segment_at(const LinParams& p, int s) {
    Segment g;
    if (p.cu) {
        int lo = 0, hi = p.B - 1;   // the last b that starts at s or before
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (lin_seg_start(p, mid) <= s) lo = mid;
            else hi = mid - 1;
        }
        g.b = lo;
    } else {
        g.b = s / max(1, (p.rows + p.seg_rows - 1) / p.seg_rows);
    }
    lin_sequence(p, g.b, &g.q0, &g.n);
    const int i = s - lin_seg_start(p, g.b), count = max(1, (g.n + p.seg_rows - 1) / p.seg_rows);
    g.live = i >= 0 && i < count;
    g.first = i == 0;
    g.last = i == count - 1;
    g.r0 = g.live ? i * p.seg_rows : 0;
    g.r1 = g.live ? min(g.n, g.r0 + p.seg_rows) : 0;
    return g;
}

// The state that segment s (of sequence b) starts from, or null (zeros)
__device__ __forceinline__ const float* lin_state_src(const LinParams& p, int s, int b, int h) {
    const long size = (long)p.DK * p.DV;
    return p.split() ? p.states + ((long)s * p.Hkv + h) * size : p.init ? p.init + ((long)b * p.Hkv + h) * size : nullptr;
}
__device__ __forceinline__ float log2_decay(const LinParams& p, int h) {
    const float l = p.log_decay[h] * kLog2e;
    return l > 0.f ? 0.f : l;   // (a decay above 1 counts as 1; NaN stays)
}
__device__ __forceinline__ float decay_pow(float l2, int n) { return n == 0 ? 1.f : exp2f(l2 * (float)n); }   // (0^0 = 1)
#endif

}  // namespace attn
