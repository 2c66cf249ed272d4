// How the kernels that attend over a paged cache share their work: the list of
// (sequence, key/value head, row block, two pages) units, its cut into ranges for
// the CTAs, and the joining of row blocks that several CTAs had a share of. P: the
// kernel's parameters, with the fields s (Kv4Batch), c.Hkv, c.dv, H, group,
// win_left, win_right, sinks, prefix, part_ml, part_o, o, lse, status, and kKeepsNan:
// shares whose weight is nothing in fp32 are multiplied by 0 (NaN stays) instead of left out.
#pragma once

#include "kv4.h"
#include "ptx.cuh"

namespace attn {
namespace {

// A sequence's work: pages 0 .. n_sink - 1, then first .. (the window), `pages` in
// all, in units of two for each of `blocks` row blocks of each key/value head.
struct SeqWork {
    Kv4Seq s;
    int rows, blocks, first, n_sink, pages, units;
};
template <class P>
__device__ __forceinline__ SeqWork seq_work(const P& p, int b, int rows_per_block) {
    SeqWork w;
    w.s = kv4_seq(p.s, b);
    w.rows = w.s.nq * p.group;
    w.blocks = (w.rows + rows_per_block - 1) / rows_per_block;
    const MaskBand m = mask_band(w.s.nq, w.s.lk, p.win_left, p.win_right, p.sinks);
    int hi;
    if (band_key_blocks(m, 0, w.s.nq - 1, kPage, &w.first, &hi)) {
        w.n_sink = band_sink_blocks(m, kPage, w.first);
        w.pages = w.n_sink + hi - w.first;
    } else {
        w.n_sink = w.pages = 0;
    }
    w.units = (w.pages + 1) / 2;
    return w;
}
__device__ __forceinline__ int page_of(const SeqWork& w, int i) { return i < w.n_sink ? i : w.first + i - w.n_sink; }

// How the work list is cut: `per` units per CTA. aligned: every row block's units
// are rounded up to a multiple of `per`, so that no CTA works on two row blocks.
struct Cut {
    int per, aligned;
    __device__ __forceinline__ int span(int units) const { return aligned ? (units + per - 1) / per * per : units; }
};
// With few units per CTA a second row block costs as much as the units do (its
// queries, its first loads, its epilogue), so the aligned cut is taken when it
// needs at most this many units per CTA and fits the grid (16 windows of 4096
// keys at d = 256, 33 units each, in twos: 16.2 us unaligned, 12.3 aligned). Longer ranges balance better uncut.
constexpr int kAlignedMost = 8;
// A unit takes a CTA about 1.5 us and joining a row's shares about 1 us per 8, so
// a row block of U units is not cut into more than U / per with 12 per^2 >= U: the
// sum of the two is least there (4 heads over 16000 keys, d = 64, 125 units each:
// a pass of 23.8 us in ones, 14.6 in fours).
__device__ __forceinline__ int least_per(int units) {
    int per = 1;
    while (12 * per * per < units) ++per;
    return per;
}

// The units of all sequences as a prefix sum in shared memory (every thread of
// the CTA calls); `times` (B more ints) is scratch.
template <int kThreads, class P>
__device__ __forceinline__ Cut build_prefix(const P& p, int* prefix, int* times, int rows_per_block, int ctas) {
    for (int b = threadIdx.x; b < p.s.B; b += kThreads) {
        const SeqWork w = seq_work(p, b, rows_per_block);
        if (w.s.bad && blockIdx.x == 0) atomicCAS(p.status, kStatusOk, kStatusBadPage);
        prefix[b + 1] = w.units;
        times[b] = p.c.Hkv * w.blocks;
    }
    __shared__ Cut s_cut;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        auto total = [&](const Cut& c) {   // units of the list
            long x = 0;
            for (int b = lane; b < p.s.B; b += 32) x += (long)times[b] * c.span(prefix[b + 1]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFullMask, x, o);
            return x;
        };
        const long all = total(Cut{0, 0});
        const bool fits = all <= kKv4MostUnits;
        if (!fits) {   // (see kKv4MostUnits: an empty list, cut into nothing)
            for (int b = lane; b < p.s.B; b += 32) times[b] = 0;
            __syncwarp();
            if (blockIdx.x == 0 && lane == 0) atomicCAS(p.status, kStatusOk, kStatusBadPage);
        }
        int longest = 0;
        for (int b = lane; b < p.s.B; b += 32) longest = max(longest, times[b] > 0 ? prefix[b + 1] : 0);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) longest = max(longest, __shfl_xor_sync(kFullMask, longest, o));
        Cut cut{0, 0};
        cut.per = fits ? max((int)((all + ctas - 1) / ctas), longest > 0 ? least_per(longest) : 0) : 0;
        for (int per = cut.per; per > 0 && per <= kAlignedMost; ++per)
            if (total(Cut{per, 1}) <= (long)per * ctas) {
                cut = Cut{per, 1};
                break;
            }
        int carry = 0;
        for (int b0 = 0; b0 < p.s.B; b0 += 32) {
            const int b = b0 + lane;
            int x = b < p.s.B ? times[b] * cut.span(prefix[b + 1]) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFullMask, x, o);
                if (lane >= o) x += y;
            }
            __syncwarp();
            if (b < p.s.B) prefix[b + 1] = carry + x;
            carry += __shfl_sync(kFullMask, x, 31);
        }
        if (lane == 0) {
            prefix[0] = 0;
            s_cut = cut;
        }
    }
    __syncthreads();
    return s_cut;
}

// Unit u: sequence, head, row block and unit index within the row block.
struct Unit {
    int b, h, rb, i;
};
template <class P>
__device__ __forceinline__ Unit unit_at(const P& p, const int* prefix, const Cut& cut, int u, int rows_per_block,
                                        SeqWork* w) {
    int lo = 0, hi = p.s.B - 1;   // the last b with prefix[b] <= u (and units of its own)
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    *w = seq_work(p, lo, rows_per_block);
    Unit r;
    r.b = lo;
    const int span = cut.span(w->units), rem = u - prefix[lo], per_head = w->blocks * span;
    r.h = rem / per_head;
    const int x = rem - r.h * per_head;
    r.rb = x / span;
    r.i = x - r.rb * span;   // (>= units: the padding behind an aligned row block)
    return r;
}

// Row r of head h of a sequence: which CTAs had a share of its row block.
struct Shares {
    int c0, c1, in_block, rows_per_block;   // c0 == c1: finished by its CTA
    __device__ __forceinline__ long at(int c) const { return (long)(2 * c + (c == c0 ? 1 : 0)) * rows_per_block + in_block; }
};
template <class P>
__device__ __forceinline__ Shares shares_of(const P& p, const SeqWork& w, int b, int h, int r, int rows_per_block) {
    const Cut cut{p.prefix[kKv4MaxBatch + 1], p.prefix[kKv4MaxBatch + 2]};
    const int per = cut.per;
    const int u = p.prefix[b] + (h * w.blocks + r / rows_per_block) * cut.span(w.units);
    return Shares{u / per, (u + w.units - 1) / per, r % rows_per_block, rows_per_block};
}
// (max, sum) of all shares of a row, taken by `lanes` (a power of two) neighbouring
// lanes, of which this is `lane`: every lane of the warp calls and gets its row's.
template <class P>
__device__ __forceinline__ float2 join_ml(const P& p, const Shares& s, int lane, int lanes) {
    float m = -INFINITY, l = 0.f;
    for (int c = s.c0 + lane; c <= s.c1; c += lanes) m = fmaxf(m, p.part_ml[2 * s.at(c)]);
    for (int o = lanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
    for (int c = s.c0 + lane; c <= s.c1; c += lanes) {
        const float2 v = *reinterpret_cast<const float2*>(p.part_ml + 2 * s.at(c));
        l += v.y * (v.x == -INFINITY ? 0.f : ex2_mufu(v.x - m));
    }
    for (int o = lanes / 2; o > 0; o >>= 1) l += __shfl_xor_sync(kFullMask, l, o);
    return make_float2(m, l);
}
template <class P>
__device__ __forceinline__ long lse_at(const P& p, const SeqWork& w, int b, int i, int head) {
    return p.s.cu ? (long)head * p.s.total + w.s.q0 + i : ((long)b * p.H + head) * p.s.rows + i;
}

// One warp joins the partial rows of row `row` (token, head) in CTA order (the same sum on
// every run), if its row block was shared; rows that no key reaches get O = 0, LSE =
// -inf. Waits for the grid before it (every thread: the next kernel counts on it).
template <class P>
__device__ __forceinline__ void finish_row(const P& p, long row, int rows_per_block) {
    const int lane = threadIdx.x & 31;
    const bool live = row < (long)p.s.total * p.H;
    const int tok = live ? (int)(row / p.H) : 0, head = live ? (int)(row % p.H) : 0;
    const int b = live ? kv4_seq_of_row(p.s, tok) : -1;
    const SeqWork w = seq_work(p, b < 0 ? 0 : b, rows_per_block);
    const int i = tok - w.s.q0, dv = p.c.dv;
    __nv_bfloat16* out = p.o + ((long)tok * p.H + head) * dv;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // (see above)
    if (b < 0 || w.s.bad) return;
    float* lse = p.lse + lse_at(p, w, b, i, head);
    if (w.pages == 0) {
        for (int c = lane * 4; c < dv; c += 128) *reinterpret_cast<uint2*>(out + c) = make_uint2(0, 0);
        if (lane == 0) *lse = -INFINITY;
        return;
    }
    if (p.prefix[kKv4MaxBatch + 1] == 0) return;   // (a list that did not fit: nothing to join)
    const Shares s = shares_of(p, w, b, head / p.group, i * p.group + head % p.group, rows_per_block);
    if (s.c0 == s.c1) return;
    const float2 ml = join_ml(p, s, lane, 32);
    float4 o[2] = {};
    for (int c = s.c0; c <= s.c1; c += 4) {   // four shares' loads in flight
        float f[4];
        bool live[4];
        float4 y[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool in = c + k <= s.c1;
            const long at = s.at(in ? c + k : s.c1);
            const float mk = p.part_ml[2 * at];
            live[k] = in && mk != -INFINITY;
            f[k] = live[k] ? ex2_mufu(mk - ml.x) : 0.f;
            if (!P::kKeepsNan) live[k] = f[k] != 0.f;
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (x * 128 + lane * 4 < dv) y[k][x] = *reinterpret_cast<const float4*>(p.part_o + at * dv + x * 128 + lane * 4);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (live[k])
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    o[x].x = fmaf(f[k], y[k][x].x, o[x].x);
                    o[x].y = fmaf(f[k], y[k][x].y, o[x].y);
                    o[x].z = fmaf(f[k], y[k][x].z, o[x].z);
                    o[x].w = fmaf(f[k], y[k][x].w, o[x].w);
                }
    }
    const float inv = ml.y > 0.f ? 1.f / ml.y : (ml.y == 0.f ? 0.f : ml.y);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int col = x * 128 + lane * 4;
        if (col < dv)
            *reinterpret_cast<uint2*>(out + col) =
                make_uint2(pack_bf16x2(o[x].x * inv, o[x].y * inv), pack_bf16x2(o[x].z * inv, o[x].w * inv));
    }
    if (lane == 0) *lse = ml.y == 0.f ? -INFINITY : (ml.x + log2f(ml.y)) * kLn2;
}

}  // namespace
}  // namespace attn
