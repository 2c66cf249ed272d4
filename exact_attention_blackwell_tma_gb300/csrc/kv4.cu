// The 4-bit key/value cache: append (quantise), read (dequantise) and evict.
// All three are bound by memory: each value is touched once.
#include "kv4.h"
#include "ptx.cuh"

namespace attn {
namespace {

__device__ __forceinline__ void bad_page(int* status) { atomicCAS(status, kStatusOk, kStatusBadPage); }

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// (hi - lo) / 15 rounded once to bf16. The fp32 quotient can only mislead the
// second rounding next to the midpoint of two bf16 values; there the midpoint
// m is compared exactly: 15 m has 13 bits, and hi - lo is carried as d + e
// (Knuth's two-sum), so (d - 15 m) + e has the right sign.
__device__ __forceinline__ float scale_of(float lo, float hi) {
    const float d = hi - lo;
    const float f = __fdiv_rn(d, 15.f);
    const uint32_t u = __float_as_uint(f);
    const int low = (int)(u & 0xffffu) - 0x8000;
    uint32_t up = low > 0 || (low == 0 && (u & 0x10000u)) ? 1u : 0u;
    if (low >= -4 && low <= 4) {
        const float t = d - hi;
        const float e = (hi - (d - t)) - (lo + t);
        const float diff = (d - 15.f * __uint_as_float((u & 0xffff0000u) | 0x8000u)) + e;
        up = diff > 0.f || (diff == 0.f && (u & 0x10000u)) ? 1u : 0u;
    }
    if (!(f <= 3.0e38f)) return f;   // infinity and NaN stay
    return __uint_as_float((u & 0xffff0000u) + (up << 16));
}

// round((x - lo) / s) to 0 .. 15, ties to even, decided exactly: next to a
// border (k + 1/2) s the sign of (x - lo) - (k + 1/2) s is taken as above.
__device__ __forceinline__ uint32_t code_of(float x, float lo, float s, float inv) {
    const float d = x - lo, q = d * inv;
    const float k = floorf(q), frac = q - k;
    float c = rintf(q);
    if (fabsf(frac - 0.5f) < 6.1e-5f) {
        const float t = d - x;
        const float e = (x - (d - t)) - (lo + t);
        const float diff = (d - (k + 0.5f) * s) + e;
        c = diff > 0.f ? k + 1.f : (diff < 0.f ? k : 2.f * rintf(0.5f * (k + 0.5f)));
    }
    return (uint32_t)fminf(fmaxf(c, 0.f), 15.f);   // (NaN gives 0)
}

// Eight lanes quantise one group of 64 channels of one token and head: 16 bytes
// of bf16 in and 4 bytes of codes out per lane, the group's extremes by three
// shuffles.
__global__ void __launch_bounds__(256) kv4_append_kernel(Kv4Cache c, Kv4Batch s, const __nv_bfloat16* k,
                                                         const __nv_bfloat16* v, long k_stride, long v_stride,
                                                         int* status) {
    const int gk = c.d / kKv4Group, gv = c.dv / kKv4Group, per_head = gk + gv;
    const long chunks = (long)s.total * c.Hkv * per_head;
    const long step = (long)gridDim.x * blockDim.x / 8;
    const int l8 = threadIdx.x & 7;
    for (long i0 = ((long)blockIdx.x * blockDim.x + threadIdx.x) / 8; i0 - (threadIdx.x & 31) / 8 < chunks; i0 += step) {
        const bool live = i0 < chunks;   // (the warp's four groups stay together for the shuffles)
        const long i = live ? i0 : 0;
        const int t = (int)(i / (c.Hkv * per_head));
        const int rem = (int)(i - (long)t * c.Hkv * per_head);
        const int h = rem / per_head, gi = rem - h * per_head;
        const bool is_v = gi >= gk;
        const int g = is_v ? gi - gk : gi, groups = is_v ? gv : gk;
        const int width = groups * kKv4Group;
        const __nv_bfloat16* src = (is_v ? v + t * v_stride : k + t * k_stride) + h * width + g * kKv4Group + l8 * 8;
        const uint4 raw = *reinterpret_cast<const uint4*>(src);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
        float lo = x[0], hi = x[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) {
            lo = min_nan(lo, x[j]);
            hi = max_nan(hi, x[j]);
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            lo = min_nan(lo, __shfl_xor_sync(kFullMask, lo, o));
            hi = max_nan(hi, __shfl_xor_sync(kFullMask, hi, o));
        }
        if (!live) continue;
        const float sc = scale_of(lo, hi);
        const float inv = sc > 0.f ? __fdiv_rn(1.f, sc) : 0.f;
        uint32_t codes = 0;
        if (sc > 0.f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) codes |= code_of(x[j], lo, sc, inv) << (4 * j);
        }
        const int b = kv4_seq_of_row(s, t);
        if (b < 0) continue;
        const Kv4Seq q = kv4_seq(s, b);
        const int slot = q.lk - q.nq + t - q.q0;
        int page = -1;
        if (!q.bad && slot >= 0) page = s.table[(long)b * s.width + slot / kPage];
        if (page < 0 || page >= c.n_pages) {
            bad_page(status);
            continue;
        }
        const long row = (((long)page * c.Hkv + h) * groups + g) * kPage + slot % kPage;
        reinterpret_cast<uint32_t*>(is_v ? c.v_codes : c.k_codes)[row * 8 + l8] = codes;
        if (l8 == 0)
            (is_v ? c.v_params : c.k_params)[row] = (__float_as_uint(sc) >> 16) | (__float_as_uint(lo) & 0xffff0000u);
    }
}

// Eight lanes restore one group: 4 bytes of codes in, 16 bytes of bf16 out.
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4Cache c, Kv4Batch s, __nv_bfloat16* k, __nv_bfloat16* v,
                                                       int* status) {
    const int gk = c.d / kKv4Group, gv = c.dv / kKv4Group, per_head = gk + gv;
    const long chunks = (long)s.total * c.Hkv * per_head;
    const long step = (long)gridDim.x * blockDim.x / 8;
    const int l8 = threadIdx.x & 7;
    for (long i = ((long)blockIdx.x * blockDim.x + threadIdx.x) / 8; i < chunks; i += step) {
        const int t = (int)(i / (c.Hkv * per_head));
        const int rem = (int)(i - (long)t * c.Hkv * per_head);
        const int h = rem / per_head, gi = rem - h * per_head;
        const bool is_v = gi >= gk;
        const int g = is_v ? gi - gk : gi, groups = is_v ? gv : gk;
        const int b = kv4_seq_of_row(s, t);
        if (b < 0) continue;
        const Kv4Seq q = kv4_seq(s, b);
        const int slot = q.lk - q.nq + t - q.q0;
        uint4 out = make_uint4(0, 0, 0, 0);
        int page = -1;
        if (!q.bad && slot >= 0) page = s.table[(long)b * s.width + slot / kPage];
        if (page >= 0 && page < c.n_pages) {
            const long row = (((long)page * c.Hkv + h) * groups + g) * kPage + slot % kPage;
            const uint32_t w = reinterpret_cast<const uint32_t*>(is_v ? c.v_codes : c.k_codes)[row * 8 + l8];
            const uint32_t p = (is_v ? c.v_params : c.k_params)[row];
            const float sc = __uint_as_float(p << 16), lo = __uint_as_float(p & 0xffff0000u);
            uint32_t r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r[j] = pack_bf16x2(fmaf((float)((w >> (8 * j)) & 15u), sc, lo),
                                   fmaf((float)((w >> (8 * j + 4)) & 15u), sc, lo));
            out = make_uint4(r[0], r[1], r[2], r[3]);
        } else if (q.bad || slot >= 0) {
            bad_page(status);
        }   // (a row before the cache's first token reads as zero)
        __nv_bfloat16* dst = (is_v ? v : k) + ((long)t * c.Hkv + h) * (groups * kKv4Group) + g * kKv4Group + l8 * 8;
        *reinterpret_cast<uint4*>(dst) = out;
    }
}

// ---------------------------------------------------------------- evict
// The order of weights as unsigned integers: NaN below everything, -0 = +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelThreads = 512;

// One CTA per (sequence, head): the slots it keeps, ascending. The need-th
// largest key of the middle is found by four rounds of 8-bit histograms (radix
// select); then one ordered pass writes the kept slots, equal weights in slot
// order.
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(Kv4EvictParams p) {
    __shared__ int hist[256];
    __shared__ int warp_sum[kSelThreads / 32];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    const int b = blockIdx.x / p.c.Hkv, h = blockIdx.x % p.c.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int n = p.lens[b];
    const long most = (long)p.width * kPage < p.weight_stride ? (long)p.width * kPage : p.weight_stride;
    if (n < 0 || n > most) {
        if (tid == 0) bad_page(p.status);
        n = n < 0 ? 0 : (int)most;
    }
    const int m = n < p.budget ? n : p.budget;
    const float* w = p.weights + ((long)b * p.c.Hkv + h) * p.weight_stride;
    float* nw = p.new_weights + ((long)b * p.c.Hkv + h) * p.new_stride;
    int* kept = p.kept + ((long)b * p.c.Hkv + h) * p.budget;
    if (h == 0 && tid == 0) p.new_lens[b] = m;
    const bool all = n <= p.budget;
    const int lo = all ? n : p.sinks, hi = all ? n : n - p.recent;   // the middle [lo, hi)
    if (tid == 0) {
        s_prefix = 0;
        s_need = all ? 0 : m - p.sinks - p.recent;
    }
    __syncthreads();
    uint32_t prefix = 0;
    int need = s_need;
    // (need == 0: no key of the middle stays)
    for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int j = lo + tid; j < hi; j += kSelThreads) {
            const uint32_t key = weight_key(w[j]);
            if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
        }
        __syncthreads();
        if (warp == 0) {   // from the largest digit down, the one that holds the need-th key
            int cnt[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += cnt[i] = hist[255 - (lane * 8 + i)];
            int before = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(kFullMask, before, o);
                if (lane >= o) before += x;
            }
            before -= sum;
            for (int i = 0; i < 8; ++i) {
                if (before < need && need <= before + cnt[i]) {
                    s_prefix = prefix | (uint32_t)(255 - (lane * 8 + i)) << shift;
                    s_need = need - before;
                }
                before += cnt[i];
            }
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
        __syncthreads();
    }
    // ordered pass: slot j stays if it is outside the middle, above the threshold,
    // or at the threshold among the first `need`
    const bool some = !all && m > p.sinks + p.recent;
    int base = 0, ties = 0;   // kept slots and threshold slots so far
    for (int j0 = 0; j0 < n; j0 += kSelThreads) {
        const int j = j0 + tid;
        const bool in = j < n, mid = in && j >= lo && j < hi;
        const float x = in ? w[j] : 0.f;
        const uint32_t key = mid ? weight_key(x) : 0u;
        const bool tie = mid && some && key == prefix;
        const unsigned tb = __ballot_sync(kFullMask, tie);
        if (lane == 0) warp_sum[warp] = __popc(tb);
        __syncthreads();
        int tie_rank = ties + __popc(tb & ((1u << lane) - 1));
        int tie_total = 0;
#pragma unroll
        for (int i = 0; i < kSelThreads / 32; ++i) {
            if (i < warp) tie_rank += warp_sum[i];
            tie_total += warp_sum[i];
        }
        __syncthreads();
        const bool keep = in && (!mid || (some && (key > prefix || (tie && tie_rank < need))));
        const unsigned kb = __ballot_sync(kFullMask, keep);
        if (lane == 0) warp_sum[warp] = __popc(kb);
        __syncthreads();
        int at = base + __popc(kb & ((1u << lane) - 1)), total = 0;
#pragma unroll
        for (int i = 0; i < kSelThreads / 32; ++i) {
            if (i < warp) at += warp_sum[i];
            total += warp_sum[i];
        }
        if (keep && at < m) {
            kept[at] = j;
            nw[at] = x;
        }
        base += total;
        ties += tie_total;
        __syncthreads();
    }
    for (int i = m + tid; i < p.budget; i += kSelThreads) kept[i] = -1;
    for (long i = m + tid; i < p.new_stride; i += kSelThreads) nw[i] = 0.f;
}

// Two lanes copy one 32-byte row of codes; the first also its parameters.
__global__ void __launch_bounds__(256) kv4_gather_kernel(Kv4EvictParams p) {
    const int gk = p.c.d / kKv4Group, gv = p.c.dv / kKv4Group, per = gk + gv;
    const long rows = (long)p.B * p.c.Hkv * p.budget * per;
    const long step = (long)gridDim.x * blockDim.x / 2;
    const int half = threadIdx.x & 1;
    for (long i = ((long)blockIdx.x * blockDim.x + threadIdx.x) / 2; i < rows; i += step) {
        // consecutive lane pairs: consecutive kept slots of one group
        const long bhg = i / p.budget;
        const int at = (int)(i - bhg * p.budget);
        const int gi = (int)(bhg % per);
        const long bh = bhg / per;
        const int b = (int)(bh / p.c.Hkv), h = (int)(bh % p.c.Hkv);
        const int j = p.kept[bh * p.budget + at];
        if (j < 0) continue;
        const int src = p.table[(long)b * p.width + j / kPage], dst = p.new_table[(long)b * p.new_width + at / kPage];
        if (src < 0 || src >= p.c.n_pages || dst < 0 || dst >= p.c.n_pages) {
            bad_page(p.status);
            continue;
        }
        const bool is_v = gi >= gk;
        const int g = is_v ? gi - gk : gi, groups = is_v ? gv : gk;
        const long from = (((long)src * p.c.Hkv + h) * groups + g) * kPage + j % kPage;
        const long to = (((long)dst * p.c.Hkv + h) * groups + g) * kPage + at % kPage;
        uint4* codes = reinterpret_cast<uint4*>(is_v ? p.c.v_codes : p.c.k_codes);
        codes[to * 2 + half] = codes[from * 2 + half];
        uint32_t* params = is_v ? p.c.v_params : p.c.k_params;
        if (half == 0) params[to] = params[from];
    }
}

int blocks_for(long threads, int block) {
    const long n = (threads + block - 1) / block;
    return (int)(n < 1 ? 1 : (n > 152 * 16 ? 152 * 16 : n));
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Cache& c, const Kv4Batch& s, const __nv_bfloat16* k, const __nv_bfloat16* v,
                              long k_stride, long v_stride, int* status, cudaStream_t stream) {
    const long threads = (long)s.total * c.Hkv * ((c.d + c.dv) / kKv4Group) * 8;
    kv4_append_kernel<<<blocks_for(threads, 256), 256, 0, stream>>>(c, s, k, v, k_stride, v_stride, status);
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4Cache& c, const Kv4Batch& s, __nv_bfloat16* k, __nv_bfloat16* v, int* status,
                            cudaStream_t stream) {
    const long threads = (long)s.total * c.Hkv * ((c.d + c.dv) / kKv4Group) * 8;
    kv4_read_kernel<<<blocks_for(threads, 256), 256, 0, stream>>>(c, s, k, v, status);
    return cudaGetLastError();
}

cudaError_t launch_kv4_evict(const Kv4EvictParams& p, cudaStream_t stream) {
    kv4_select_kernel<<<p.B * p.c.Hkv, kSelThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long threads = (long)p.B * p.c.Hkv * p.budget * ((p.c.d + p.c.dv) / kKv4Group) * 2;
    kv4_gather_kernel<<<blocks_for(threads, 256), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace attn
