// Linear attention with a decay per head: parameters and launchers of its kernels.
//
// One form serves the forward and the three gradients. With the tokens of a sequence
// taken in order (o, dq) or from the last to the first (dk, dv: `back`), token i's
// position r, and D the decay,
//   out_i = scale sum_{j at or before i} D^|r_i - r_j| <a_i, b_j> c_j + x D^(r_i + 1 - back) a_i^T X
//   X'    = D^n X + y sum_j D^(n - 1 - r_j + back) b_j c_j^T
// where X is the state carried in and X' the one carried out, x = scale and y = 1 forwards, x = 1 and y = scale
// backwards (dS arrives at its own size: divided by a small scale it might leave the range):
//   o   a = q,  b = k,  c = v,  X = S_0          X' = S_n
//   dq  a = dO, b = v,  c = k,  X = S_0^T
//   dk  a = v,  b = dO, c = q,  X = dS_n^T
//   dv  a = k,  b = q,  c = dO, X = dS_n         X' = dS_0
// (dS is the gradient of the state behind a token; that of the state in front of
// it has one more factor of D, hence `back` in the exponents.) Grouped heads: `per`
// query heads share a state. o and dq have an output for each (a differs), dk and
// dv sum over them (b and c differ): `back` says that, too.
//
// Segments. A run is a sequence's key/value head; it has a unit for every chunk of kLinChunk tokens, counted from
// the first token in either direction. The runs' units lie in a row, sequence by sequence and head by head, and are cut
// into `ranges` of the same length, so that every CTA has as much to do as the others (the chunks of 32 runs of 8192
// tokens on 152 SMs: 13.5 each; whole segments of one length gave 16 to some). A segment is what a range has of
// a run. Three kernels: what each segment that others follow adds to the state, the scan that turns this into the
// state behind it, the outputs. A call whose runs are not cut (`whole`: range i has runs i, i + ranges, ..) and
// that wants no state back is the last one alone.
#pragma once

#include "kernels.h"
#include "ptx.cuh"

namespace attn {

struct LinParams {
    __nv_bfloat16* out;                  // tokens of heads x DV, contiguous
    const float* log_decay;              // [Hkv], natural log
    const float* init;                   // [B][Hkv][DK][DV] ([DV][DK] with init_trans), or null
    float* final;                        // [B][Hkv][DK][DV], or null
    float* states;                       // workspace: [ranges if cut, and B Hkv with `final`][DK][DV] (see lin_share_slot)
    const int* cu;                       // row offsets, or null (dense)
    int B, rows, total;                  // rows per sequence (dense), rows in all
    int Hkv, per, DK, DV;
    int ranges, whole;
    int init_trans, states_trans;        // (states_trans: [..][DV][DK], the states of the transposed product)
    float scale;
    int* status;
    uint64_t wait_budget_ns;
    // whether there are states to make
    __host__ __device__ bool split() const { return !whole || final; }
    __host__ __device__ int cut_slots() const { return whole ? 0 : ranges; }
};

constexpr int kLinChunk = 128;

struct LinPlan {
    int ranges, whole;
    long slots;   // states of the workspace
};
// final: the last states are wanted; tiles: the most CTAs that a range has in any of the call's products
LinPlan lin_plan(int B, int Hkv, int L, bool packed, int tiles, bool final);
inline int lin_tiles(int DK, int DV) { return DK == 128 && DV == 128 ? 1 : DV / 64; }

// Tensor maps, boxes of 64 channels of a head: a, b and c by 128 tokens, out by 32
struct LinMaps {
    CUtensorMap a, b, c, out;
};

// The states that the segments start from, and the last one (nothing to do without several segments or `final`); the outputs
cudaError_t launch_linear_states(const LinParams& p, const LinMaps& maps, bool back, cudaStream_t stream);
cudaError_t launch_linear_out(const LinParams& p, const LinMaps& maps, bool back, cudaStream_t stream);
// (the first half of the states: what each segment adds)
cudaError_t launch_linear_shares(const LinParams& p, const LinMaps& maps, bool back, cudaStream_t stream);

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
// The kernels of a call start before the one in front of them has ended (its last CTAs, the launch and the first
// instructions of the next overlap: 349 -> 332 us for a training step of ten kernels) and wait for it before they
// touch global memory. A kernel lets the next one start once it has its tensor memory: the next one's CTA, should it find
// room on the same SM, could else take the columns first and hold them while it waits for the CTA that needs them.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <class... P, class... A>
cudaError_t launch_early(void (*kern)(P...), unsigned grid, int threads, int bytes, cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

struct LinSegment {
    int run, h, row0, rows;        // rows row0 .. of the tensors; rows = 0: no more
    int after_start, before_end;   // whether the run has units in front of it, and behind it
};
// Where a segment's share goes, and the state it starts from (-1: the call's initial state). Slot i < cut_slots is range
// i's: what its last segment (backwards: its first), cut off by the range's end, adds, and then, by the scan, the
// state that its neighbour starts from. Slot cut_slots + run: the share of the segment that ends a walk and, by
// the scan, the run's initial state (whose own buffer may be `final`, which is written before the outputs are).
__device__ __forceinline__ int lin_share_slot(const LinParams& p, const LinSegment& g, int range, bool back) {
    return (back ? g.after_start : g.before_end) ? range : p.cut_slots() + g.run;
}
__device__ __forceinline__ int lin_start_slot(const LinParams& p, const LinSegment& g, int range, bool back) {
    // (within the slots whatever the offsets)
    if (back ? g.before_end : g.after_start) return back ? min(range + 1, p.ranges - 1) : max(range - 1, 0);
    return p.final ? p.cut_slots() + g.run : -1;
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
__device__ __forceinline__ int lin_chunks(int n) { return (n + kLinChunk - 1) / kLinChunk; }
// Chunks of the sequences in front of b, and of all (a warp's work; units are Hkv times as many, below 2^30: rows are)
__device__ __forceinline__ void lin_chunks_before(const LinParams& p, int b, int lane, int* before, int* all) {
    if (!p.cu) {
        *before = b * lin_chunks(p.rows);
        *all = p.B * lin_chunks(p.rows);
        return;
    }
    constexpr int kMost = 1 << 25;   // (more than there are for offsets that ascend; the sums stay ints)
    int x = 0, y = 0;
    for (int i = lane; i < p.B; i += 32) {
        int q0, n;
        lin_sequence(p, i, &q0, &n);
        y = min(y + lin_chunks(n), kMost);
        if (i < b) x = min(x + lin_chunks(n), kMost);
    }
    *before = (int)__reduce_add_sync(0xffffffffu, (unsigned)x);
    *all = (int)__reduce_add_sync(0xffffffffu, (unsigned)y);
}
// Units of a range. Bad offsets can overlap, which may make more units than rows: a product that leaves int is capped,
// the units behind it are not worked on.
__device__ __forceinline__ int lin_units(const LinParams& p, int chunks) {
    const long u = (long)chunks * p.Hkv;
    return u < (1L << 30) ? (int)u : 1 << 30;
}
__device__ __forceinline__ int lin_range_units(const LinParams& p, int units) { return max(1, (units + p.ranges - 1) / p.ranges); }

// Yields a range's segments in the order of the units (for one warp, all lanes alike).
struct LinFinder {
    int u, end, b, h, q0, n, c0, step;   // the next unit, that of sequence b and head h at chunk c0
    __device__ __forceinline__ LinFinder(const LinParams& p, int range, int lane) {
        step = p.whole ? p.ranges : 1;
        if (p.whole) {   // u and end count runs
            u = range;
            end = p.B * p.Hkv;
            if (u < end) at_run(p, u);
            return;
        }
        int skip, chunks;
        lin_chunks_before(p, 0, lane, &skip, &chunks);
        const int units = lin_units(p, chunks), each = lin_range_units(p, units);
        u = (int)min((long)range * each, (long)units);
        end = min(units, u + each);
        if (u >= end) return;
        // the sequence that holds unit u, and the units in front of it
        long before = 0;
        if (!p.cu) {
            b = u / p.Hkv / lin_chunks(p.rows);
            before = (long)b * lin_chunks(p.rows) * p.Hkv;
        } else {
            for (int b0 = 0;; b0 += 32) {
                int c = 0;
                if (b0 + lane < p.B) {
                    lin_sequence(p, b0 + lane, &q0, &n);
                    c = lin_chunks(n);
                }
                int sum = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                const unsigned past = __ballot_sync(0xffffffffu, before + (long)sum * p.Hkv > u);
                if (past || b0 + 32 >= p.B) {
                    const int at = past ? __ffs(past) - 1 : 31;
                    before += (long)__shfl_sync(0xffffffffu, sum - c, at) * p.Hkv;
                    b = min(b0 + at, p.B - 1);
                    break;
                }
                before += (long)__shfl_sync(0xffffffffu, sum, 31) * p.Hkv;
            }
        }
        lin_sequence(p, b, &q0, &n);
        const int c = max(1, lin_chunks(n));
        h = min((int)((u - before) / c), p.Hkv - 1);
        c0 = (int)(u - before) - h * c;
    }
    __device__ __forceinline__ void at_run(const LinParams& p, int run) {
        b = run / p.Hkv;
        h = run - b * p.Hkv;
        lin_sequence(p, b, &q0, &n);
        c0 = 0;
    }
    __device__ __forceinline__ LinSegment next(const LinParams& p) {
        while (u < end && b < p.B) {
            const int c = lin_chunks(n), c1 = p.whole ? c : min(c, c0 + end - u);
            const LinSegment g{b * p.Hkv + h, h, q0 + c0 * kLinChunk, min(n, c1 * kLinChunk) - c0 * kLinChunk, c0 > 0, c1 < c};
            if (p.whole) {
                u += step;
                if (u < end) at_run(p, u);
            } else {
                u += c1 - c0;
                c0 = 0;
                if (u < end && ++h == p.Hkv) {
                    h = 0;
                    if (++b < p.B) lin_sequence(p, b, &q0, &n);
                }
            }
            if (g.rows > 0) return g;
        }
        return LinSegment{0, 0, 0, 0, 0, 0};
    }
};

__device__ __forceinline__ float log2_decay(const LinParams& p, int h) {
    const float l = p.log_decay[h] * kLog2e;
    return l > 0.f ? 0.f : l;   // (a decay above 1 counts as 1; NaN stays)
}
__device__ __forceinline__ float decay_pow(float l2, int n) { return n == 0 ? 1.f : exp2f(l2 * (float)n); }   // (0^0 = 1)
#endif

}  // namespace attn
