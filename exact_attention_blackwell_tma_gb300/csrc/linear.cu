// Linear attention with a decay per head: the plan of its segments, the scan over them, and the
// single token by the recurrence. linear.h gives the one form that the forward and the gradients
// share, linear_tc.cu its kernels on the tensor cores.
//
// Mathematics. Within a chunk of 128 tokens the pairs are taken as in attention, P_ij =
// D^|i-j| <a_i, b_j> and out += P c; what lies before the chunk enters through the state
// X, out += D^(..) a X. No factor is larger than 1, so nothing overflows for fast decays.
// Sums, states and decays are fp32. Roundings to bf16, the type of the tensor cores'
// operands: P and X before their products (like P in the exact attention: they reach outputs
// that are bf16 themselves). The weighted b in the state's update is as good as its sum must be:
// two bf16 terms (16 bits) on the way from chunk to chunk, where X is rounded to 8 bits next, and in the shares of a
// call that wants no last state; three (all 24) in the shares that a state which leaves the call is made of.
#include "linear.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kScanThreads = 128;

// Turns the segments' shares into the states that their neighbours start from, in the order of the walk:
// X = init, then X = D^rows X + share; and writes the last one. A thread takes four neighbouring elements.
template <bool kBack>
__global__ void __launch_bounds__(kScanThreads) lin_scan_kernel(const LinParams p) {
    __shared__ int s_before, s_all;
    launch_next();
    wait_for_last();
    const int size = p.DK * p.DV, blocks = size / (4 * kScanThreads);
    const int run = blockIdx.x / blocks, b = run / p.Hkv, h = run - b * p.Hkv;
    const int x = ((blockIdx.x - run * blocks) * kScanThreads + threadIdx.x) * 4;
    float4 X = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.init) {   // (loaded before the offsets are looked at: their latencies overlap)
        const float* src = p.init + (long)run * size;
        if (p.init_trans) {
            const float* t = src + x % p.DV * p.DK + x / p.DV;
            X = make_float4(t[0], t[p.DK], t[2 * p.DK], t[3 * p.DK]);
        } else {
            X = *reinterpret_cast<const float4*>(src + x);
        }
    }
    const float l2 = log2_decay(p, h);
    int q0, n;
    lin_sequence(p, b, &q0, &n);
    // its units: unit0 .. unit0 + chunks - 1, in ranges first .. last
    const int chunks = lin_chunks(n);
    int first = 0, last = 0, each = 1;
    long unit0 = 0;
    if (!p.whole) {
        if (threadIdx.x < 32) {
            int before, all;
            lin_chunks_before(p, b, threadIdx.x, &before, &all);
            if (threadIdx.x == 0) {
                s_before = before;
                s_all = all;
            }
        }
        __syncthreads();
        each = lin_range_units(p, lin_units(p, s_all));
        unit0 = (long)s_before * p.Hkv + (long)h * chunks;
        first = (int)min(unit0 / each, (long)p.ranges - 1);
        last = chunks > 0 ? (int)min((unit0 + chunks - 1) / each, (long)p.ranges - 1) : first;
    }
    const float4 start = X;
    // rows of the run in range i (all of them, if it is not cut)
    auto rows_in = [&](int i) {
        if (first == last) return n;
        const long lo = max(unit0, (long)i * each) - unit0, hi = min(unit0 + chunks, (long)(i + 1) * each) - unit0;
        return (int)(min((long)n, hi * kLinChunk) - lo * kLinChunk);
    };
    float4* slots = reinterpret_cast<float4*>(p.states + x);
    auto move = [&](float f, const float4& y) {
        X = make_float4(fmaf(X.x, f, y.x), fmaf(X.y, f, y.y), fmaf(X.z, f, y.z), fmaf(X.w, f, y.w));
    };
    const int cuts = last - first;
    constexpr int kAhead = 4;
    for (int i = 0; i < cuts; i += kAhead) {   // (step i of the walk)
        float4 y[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k < cuts) y[k] = slots[(long)(kBack ? last - i - k : first + i + k) * (size / 4)];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i + k >= cuts) break;
            const int r = kBack ? last - i - k : first + i + k;
            move(decay_pow(l2, rows_in(r)), y[k]);
            slots[(long)r * (size / 4)] = X;
        }
    }
    if (p.final) {
        float4* at = slots + ((long)p.cut_slots() + run) * (size / 4);
        if (n > 0) move(decay_pow(l2, rows_in(kBack ? first : last)), *at);
        *at = start;
        *reinterpret_cast<float4*>(p.final + (long)run * size + x) = X;
    }
}

// ---------------------------------------------------------------- one token
constexpr int kStepThreads = 256, kStepHeads = 4;   // query heads reduced at once

// S = decay S + k v^T and o = scale q^T S of one sequence and head, 64 columns of S
// per CTA: 16 threads of four columns side by side, 16 rows apart down the state,
// which is read and written once, in registers between.
template <int D>
__global__ void __launch_bounds__(kStepThreads) lin_step_kernel(const LinStepParams p) {
    constexpr int kRows = D / 16;
    __shared__ float kf[D], qf[kStepHeads][D], red[kStepHeads][8][64];
    const int nt = p.dv >> 6, tile = blockIdx.x % nt, bh = blockIdx.x / nt, b = bh / p.Hkv, h = bh % p.Hkv;
    const int c4 = threadIdx.x & 15, rg = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    float* S = p.state + (long)bh * D * p.dv + tile * 64 + c4 * 4;
    float4 x[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) x[i] = __ldcs(reinterpret_cast<const float4*>(S + (long)(rg + 16 * i) * p.dv));
    float l = p.log_decay[h];
    const float decay = l > 0.f ? 1.f : expf(l);
    for (int i = threadIdx.x; i < D; i += kStepThreads) kf[i] = __bfloat162float(p.k[b * p.k_stride + (long)h * D + i]);
    const uint2 vr = *reinterpret_cast<const uint2*>(p.v + b * p.v_stride + (long)h * p.dv + tile * 64 + c4 * 4);
    const float4 v = make_float4(__uint_as_float(vr.x << 16), __uint_as_float(vr.x & 0xffff0000u), __uint_as_float(vr.y << 16),
                                 __uint_as_float(vr.y & 0xffff0000u));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const float k = kf[rg + 16 * i];
        x[i] = make_float4(fmaf(decay, x[i].x, k * v.x), fmaf(decay, x[i].y, k * v.y), fmaf(decay, x[i].z, k * v.z),
                           fmaf(decay, x[i].w, k * v.w));
        __stcs(reinterpret_cast<float4*>(S + (long)(rg + 16 * i) * p.dv), x[i]);
    }
    for (int g0 = 0; g0 < p.per; g0 += kStepHeads) {
        const int heads = min(kStepHeads, p.per - g0);
        __syncthreads();
        for (int i = threadIdx.x; i < heads * D; i += kStepThreads)
            qf[i / D][i % D] = __bfloat162float(p.q[b * p.q_stride + ((long)h * p.per + g0) * D + i]);
        __syncthreads();
        for (int g = 0; g < heads; ++g) {
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const float q = qf[g][rg + 16 * i];
                s.x = fmaf(q, x[i].x, s.x);
                s.y = fmaf(q, x[i].y, s.y);
                s.z = fmaf(q, x[i].z, s.z);
                s.w = fmaf(q, x[i].w, s.w);
            }
            s.x += __shfl_xor_sync(0xffffffffu, s.x, 16);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, 16);
            s.z += __shfl_xor_sync(0xffffffffu, s.z, 16);
            s.w += __shfl_xor_sync(0xffffffffu, s.w, 16);
            if ((threadIdx.x & 16) == 0) *reinterpret_cast<float4*>(&red[g][warp][c4 * 4]) = s;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < heads * 64; i += kStepThreads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) s += red[i >> 6][w][i & 63];
            p.o[((long)b * p.Hkv * p.per + (long)h * p.per + g0 + (i >> 6)) * p.dv + tile * 64 + (i & 63)] = __float2bfloat16_rn(s * p.scale);
        }
    }
}

}  // namespace

LinPlan lin_plan(int B, int Hkv, int L, bool packed, int tiles, bool final) {
    constexpr int kSms = 152;   // CTAs of a wave on a GB300, one per SM
    const long most = kSms / tiles, runs = (long)B * Hkv, longest = ((long)L + kLinChunk - 1) / kLinChunk;
    const long units = (packed ? (long)L / kLinChunk + B : B * longest) * Hkv;   // (packed: at most)
    // Whole runs or ranges of units, whichever takes less time, counted in chunks of the outputs' kernel (3 us): where
    // states are to be made it takes half as long again, and the two launches 18 us (777 tokens, 8 heads, with states:
    // 55 us in whole runs, 33 in ranges).
    const double whole = (double)((runs + most - 1) / most) * longest * (final ? 1.5 : 1.0) + (final ? 6 : 0);
    const double cut = (double)((units + most - 1) / most) * 1.5 + 6;
    LinPlan r;
    r.whole = whole <= cut;
    const long count = r.whole ? runs : units;
    r.ranges = (int)(count < most ? (count < 1 ? 1 : count) : most);
    r.slots = (r.whole ? 0 : r.ranges) + (final ? runs : 0);
    return r;
}

cudaError_t launch_linear_states(const LinParams& p, const LinMaps& maps, bool back, cudaStream_t stream) {
    if (!p.split()) return cudaSuccess;
    if (p.total > 0) {
        const cudaError_t e = launch_linear_shares(p, maps, back, stream);
        if (e != cudaSuccess) return e;
    }
    const unsigned blocks = (unsigned)((long)p.DK * p.DV / (4 * kScanThreads) * p.B * p.Hkv);
    return launch_early(back ? lin_scan_kernel<true> : lin_scan_kernel<false>, blocks, kScanThreads, 0, stream, p);
}

cudaError_t launch_linear_step(const LinStepParams& p, cudaStream_t stream) {
    const unsigned ctas = (unsigned)((long)p.B * p.Hkv * (p.dv / 64));
    if (p.d == 64) lin_step_kernel<64><<<ctas, kStepThreads, 0, stream>>>(p);
    else if (p.d == 128) lin_step_kernel<128><<<ctas, kStepThreads, 0, stream>>>(p);
    else if (p.d == 192) lin_step_kernel<192><<<ctas, kStepThreads, 0, stream>>>(p);
    else if (p.d == 256) lin_step_kernel<256><<<ctas, kStepThreads, 0, stream>>>(p);
    else return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace attn
