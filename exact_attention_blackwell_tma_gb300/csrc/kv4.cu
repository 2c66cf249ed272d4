// The 4-bit key/value cache: append (quantise), read (dequantise) and evict.
// All three are bound by memory: each value is touched once.
#include <type_traits>

#include "kv4.h"
#include "ptx.cuh"

namespace attn {
namespace {

__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {   // of two bf16 each
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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
// border (k + 1/2) s the sign of (x - lo) - (k + 1/2) s is taken as above. It
// divides: the reciprocal of a scale of 2^-128 or less is infinite.
__device__ __forceinline__ uint32_t code_of(float x, float lo, float s) {
    const float d = x - lo, q = __fdiv_rn(d, s);
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

// The codes of eight values, four bits each from the lowest up. The quotient is
// corrected by its own residual (Markstein's division: q + (d - q s) / s, the
// residual exact by the fused multiply-add), so a tie, common between bf16
// values, comes out as exactly k + 1/2 and rounds to even, and other quotients
// stay on their side of the border as long as x - lo has few bits. Values below
// 2^-13 of the spread can make it long: a lane that has one, and a quotient next
// to a border, decides its eight codes by code_of. Rounding by adding 1.5 * 2^23
// and packing by multiply-adds (four codes make an integer below 2^16) keep off
// the conversion unit, which bound the kernel (17000 tokens of 8 heads, d = 128:
// 42 us with floor, rint and integer conversions per value, 34 us this way).
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float lo, float hi, float s) {
    if (!(s > 0.f && s < INFINITY)) return 0;   // (also where s is NaN)
    constexpr float kMagic = 12582912.f;
    float inv;
    asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(s));
    float far = 0.f, tiny = fabsf(lo), half[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float d = x[j] - lo, q0 = d * inv;
        const float q = fmaf(fmaf(-q0, s, d), inv, q0);
        const float k = (q + kMagic) - kMagic;
        far = fmaxf(far, fabsf(q - k));
        tiny = fminf(tiny, fabsf(x[j]));
        half[j >> 2] = fmaf(k, (float)(1 << (4 * (j & 3))), half[j >> 2]);
    }
    const bool sure = far < 0.5f - 6.1e-5f || tiny >= (hi - lo) * 1.2207e-4f;
    if (sure && s >= 1e-30f && s <= 1e30f) return (uint32_t)half[0] | (uint32_t)half[1] << 16;
    uint32_t codes = 0;
#pragma unroll 1
    for (int j = 0; j < 8; ++j) codes |= code_of(x[j], lo, s) << (4 * j);
    return codes;
}

// A warp takes `rows` (1 to 4) consecutive rows, whose places its first lanes
// look up together, and walks their groups of 64 channels four at a time, eight
// lanes per group: 16 bytes of bf16 and 4 bytes of codes per lane, the extremes
// by three shuffles. GK, GV: groups of a head.
template <int GK, int GV>
__global__ void __launch_bounds__(256) kv4_append_kernel(Kv4Cache c, Kv4Batch s, const __nv_bfloat16* k,
                                                         const __nv_bfloat16* v, long k_stride, long v_stride,
                                                         int rows, int* status) {
    const int lane = threadIdx.x & 31, l8 = lane & 7;
    const int t0 = (blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32) * rows;
    RowPlace mine{-2, 0};
    if (lane < rows) {
        mine = place_of(c.n_pages, s, t0 + lane, status);
        if (mine.page == -3) bad_page(status);   // more new rows than the cache holds tokens
    }
    const int chunks = c.Hkv * (GK + GV);
    for (int x = 0; x < rows; ++x) {
        const int page = __shfl_sync(kFullMask, mine.page, x), slot = __shfl_sync(kFullMask, mine.slot, x);
        if (page < 0) continue;
        const long t = t0 + x;
        for (int c0 = 0; c0 < chunks; c0 += 8) {   // two groups per lane octet: their loads go out together
            uint4 raw[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int ch = min(c0 + 4 * y + (lane >> 3), chunks - 1);
                const int h = ch / (GK + GV), gi = ch - h * (GK + GV);
                raw[y] = __ldg(reinterpret_cast<const uint4*>(
                    (gi >= GK ? v + t * v_stride + (h * GV + gi - GK) * kKv4Group : k + t * k_stride + (h * GK + gi) * kKv4Group) +
                    l8 * 8));
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int ch = c0 + 4 * y + (lane >> 3);
                const uint32_t w[4] = {raw[y].x, raw[y].y, raw[y].z, raw[y].w};
                float f[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[2 * j] = __uint_as_float(w[j] << 16);
                    f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                }
                // (min, -max) of the group as one bf16 pair: the shuffles carry both, NaN wins
                uint32_t mn = min2_nan(min2_nan(w[0], w[1]), min2_nan(w[2], w[3]));
                uint32_t mx = min2_nan(min2_nan(w[0] ^ 0x80008000u, w[1] ^ 0x80008000u),
                                       min2_nan(w[2] ^ 0x80008000u, w[3] ^ 0x80008000u));
                uint32_t m = min2_nan(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) m = min2_nan(m, __shfl_xor_sync(kFullMask, m, o));
                const float lo = __uint_as_float(m << 16), hi = -__uint_as_float(m & 0xffff0000u);
                if (ch >= chunks) continue;
                const float sc = scale_of(lo, hi);
                const uint32_t codes = codes_of(f, lo, hi, sc);
                const int h = ch / (GK + GV), gi = ch - h * (GK + GV);
                const bool is_v = gi >= GK;
                const long row = (is_v ? (((long)page * c.Hkv + h) * GV + gi - GK) : (((long)page * c.Hkv + h) * GK + gi)) * kPage + slot;
                reinterpret_cast<uint32_t*>(is_v ? c.v_codes : c.k_codes)[row * 8 + l8] = codes;
                if (l8 == 0)
                    (is_v ? c.v_params : c.k_params)[row] = (__float_as_uint(sc) >> 16) | (__float_as_uint(lo) & 0xffff0000u);
            }
        }
    }
}

// The inverse on the same walk: 4 bytes of codes in, 16 bytes of bf16 out per lane.
template <int GK, int GV>
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4Cache c, Kv4Batch s, __nv_bfloat16* k, __nv_bfloat16* v,
                                                       int rows, int* status) {
    const int lane = threadIdx.x & 31, l8 = lane & 7;
    const int t0 = (blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32) * rows;
    RowPlace mine{-2, 0};
    if (lane < rows) mine = place_of(c.n_pages, s, t0 + lane, status);
    const int chunks = c.Hkv * (GK + GV);
    for (int x = 0; x < rows; ++x) {
        const int page = __shfl_sync(kFullMask, mine.page, x), slot = __shfl_sync(kFullMask, mine.slot, x);
        if (page == -2) continue;
        const long t = t0 + x;
        for (int c0 = 0; c0 < chunks; c0 += 16) {   // four groups per lane octet: their loads go out together
            uint32_t w[4], p[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int ch = c0 + 4 * y + (lane >> 3);
                const int h = ch / (GK + GV), gi = ch - h * (GK + GV);
                const bool is_v = gi >= GK;
                const long row = (is_v ? (((long)page * c.Hkv + h) * GV + gi - GK) : (((long)page * c.Hkv + h) * GK + gi)) * kPage + slot;
                w[y] = p[y] = 0;   // (a row that lies nowhere reads as zero)
                if (page >= 0 && ch < chunks) {
                    w[y] = __ldg(reinterpret_cast<const uint32_t*>(is_v ? c.v_codes : c.k_codes) + row * 8 + l8);
                    p[y] = __ldg((is_v ? c.v_params : c.k_params) + row);
                }
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int ch = c0 + 4 * y + (lane >> 3);
                if (ch >= chunks) continue;
                const int h = ch / (GK + GV), gi = ch - h * (GK + GV);
                const float sc = __uint_as_float(p[y] << 16), lo = __uint_as_float(p[y] & 0xffff0000u);
                uint32_t r[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    r[j] = pack_bf16x2(fmaf((float)((w[y] >> (8 * j)) & 15u), sc, lo),
                                       fmaf((float)((w[y] >> (8 * j + 4)) & 15u), sc, lo));
                __nv_bfloat16* dst = gi >= GK ? v + ((t * c.Hkv + h) * GV + gi - GK) * kKv4Group : k + ((t * c.Hkv + h) * GK + gi) * kKv4Group;
                __stcs(reinterpret_cast<uint4*>(dst + l8 * 8), make_uint4(r[0], r[1], r[2], r[3]));
            }
        }
    }
}

// ---------------------------------------------------------------- evict
// The order of weights as unsigned integers: NaN below everything, -0 = +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelThreads = 1024, kSelBins = 2048;
constexpr int kSelKeys = 49152;   // keys of a row that stay in shared memory; those behind are read again

// One CTA per (sequence, head): the slots it keeps, ascending. The need-th
// largest key of the middle is found digit by digit (11, 11 and 10 bits, a
// histogram each; the first leaves the keys in shared memory for the others);
// then one ordered pass, its weights loaded a step ahead (128 rows of up to
// 32768 weights: 31 -> 28 us), writes the kept slots. Of the keys equal to the threshold the first `need`
// stay, so a slot's place is (slots kept above the threshold before it) +
// min(threshold slots before it, need): one scan of two counts.
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(Kv4EvictParams p, int cap) {
    extern __shared__ uint32_t keys[];   // cap of them
    __shared__ int hist[kSelBins];
    __shared__ int2 warp_sum[kSelThreads / 32];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
    const bool some = !all && m > p.sinks + p.recent;                // some of the middle stay
    uint32_t prefix = 0;
    int need = some ? m - p.sinks - p.recent : 0;
    if (some) {
        auto key_at = [&](int j) { return j < cap ? keys[j] : weight_key(__ldg(w + j)); };
        constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
#pragma unroll
        for (int d = 0; d < 3; ++d) {
            for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            const uint32_t mask = d == 0 ? 0u : 0xffffffffu << kShift[d - 1], digit = (1u << kBits[d]) - 1;
#pragma unroll 8
            for (int j = lo + tid; j < hi; j += kSelThreads) {
                uint32_t key;
                if (d == 0) {
                    key = weight_key(__ldg(w + j));
                    if (j < cap) keys[j] = key;
                } else {
                    key = key_at(j);
                }
                if ((key & mask) == prefix) atomicAdd(&hist[(key >> kShift[d]) & digit], 1);
            }
            __syncthreads();
            // the digit that holds the need-th key, counted from the largest: two bins per thread
            const int bins = 1 << kBits[d], top = bins - 1 - 2 * tid;
            const int c0 = 2 * tid < bins ? hist[top] : 0, c1 = 2 * tid < bins ? hist[top - 1] : 0;
            int before = c0 + c1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(kFullMask, before, o);
                if (lane >= o) before += x;
            }
            if (lane == 31) warp_sum[warp].x = before;
            before -= c0 + c1;
            __syncthreads();
            int sum = warp_sum[lane].x;   // (32 warps) the sums of the warps before this one, by every warp
            const int own = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(kFullMask, sum, o);
                if (lane >= o) sum += x;
            }
            before += __shfl_sync(kFullMask, sum - own, warp);
            if (before < need && need <= before + c0) {
                s_prefix = prefix | (uint32_t)top << kShift[d];
                s_need = need - before;
            } else if (before + c0 < need && need <= before + c0 + c1) {
                s_prefix = prefix | (uint32_t)(top - 1) << kShift[d];
                s_need = need - before - c0;
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;
        }
    }
    int above0 = 0, ties0 = 0;   // slots kept above the threshold, and threshold slots, so far
    float next[4];               // the weights of the next step
    auto fetch = [&](int j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) next[i] = j + i < n ? __ldg(w + j + i) : 0.f;
    };
    fetch(4 * tid);
    for (int j0 = 0; j0 < n; j0 += 4 * kSelThreads) {
        const int j = j0 + 4 * tid;
        const float at_j[4] = {next[0], next[1], next[2], next[3]};
        fetch(j + 4 * kSelThreads);
        uint32_t ab = 0, ti = 0;   // bits: slot j + i stays anyway, is at the threshold
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (j + i >= n) break;
            if (j + i < lo || j + i >= hi) {
                ab |= 1u << i;
            } else if (some) {
                const uint32_t key = weight_key(at_j[i]);
                ab |= (key > prefix ? 1u : 0u) << i;
                ti |= (key == prefix ? 1u : 0u) << i;
            }
        }
        int2 c = make_int2(__popc(ab), __popc(ti));
        const int2 own = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFullMask, c.x, o), y = __shfl_up_sync(kFullMask, c.y, o);
            if (lane >= o) {
                c.x += x;
                c.y += y;
            }
        }
        __syncthreads();   // the sums of the previous step have been read
        if (lane == 31) warp_sum[warp] = c;
        __syncthreads();
        int2 total = warp_sum[lane];   // (32 warps) prefix over the warps by every warp
        const int2 mine = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFullMask, total.x, o), y = __shfl_up_sync(kFullMask, total.y, o);
            if (lane >= o) {
                total.x += x;
                total.y += y;
            }
        }
        int above = above0 + c.x - own.x + __shfl_sync(kFullMask, total.x - mine.x, warp);
        int ties = ties0 + c.y - own.y + __shfl_sync(kFullMask, total.y - mine.y, warp);
        above0 += __shfl_sync(kFullMask, total.x, 31);
        ties0 += __shfl_sync(kFullMask, total.y, 31);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool a = (ab >> i) & 1u, e = (ti >> i) & 1u;
            if (a || (e && ties < need)) {
                const int at = above + min(ties, need);
                if (at < m) {
                    kept[at] = j + i;
                    nw[at] = at_j[i];
                }
            }
            above += a;
            ties += e;
        }
    }
    for (int i = m + tid; i < p.budget; i += kSelThreads) kept[i] = -1;
    for (long i = m + tid; i < p.new_stride; i += kSelThreads) nw[i] = 0.f;
}

// One CTA copies 64 kept tokens of one (sequence, head) to one new page: rows of
// 32 bytes of codes, two lanes each, and their parameters.
template <int GK, int GV>
__global__ void __launch_bounds__(128) kv4_gather_kernel(Kv4EvictParams p, int tiles) {
    __shared__ int src_page[kPage], src_slot[kPage];   // page -1: no such token
    const int bh = blockIdx.x / tiles, tile = blockIdx.x - bh * tiles;
    const int b = bh / p.c.Hkv, h = bh - b * p.c.Hkv, tid = threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int dst = p.new_table[(long)b * p.new_width + tile];
    if (tid < kPage) {
        const int at = tile * kPage + tid;
        const int j = at < p.budget ? p.kept[(long)bh * p.budget + at] : -1;
        int src = -1;
        if (j >= 0) {
            src = p.table[(long)b * p.width + j / kPage];
            if (src < 0 || src >= p.c.n_pages || dst < 0 || dst >= p.c.n_pages) {
                src = -1;
                bad_page(p.status);
            }
        }
        src_page[tid] = src;
        src_slot[tid] = j % kPage;
    }
    __syncthreads();
    constexpr int kGroups = GK + GV;
    // the codes: consecutive lane pairs take consecutive tokens of one group
#pragma unroll
    for (int i = tid; i < kGroups * kPage * 2; i += 128) {
        const int g = i / (2 * kPage), x = (i / 2) % kPage, half = i & 1;
        if (src_page[x] < 0) continue;
        uint4* codes = reinterpret_cast<uint4*>(g >= GK ? p.c.v_codes : p.c.k_codes);
        const int groups = g >= GK ? GV : GK, gi = g >= GK ? g - GK : g;
        const long from = (((long)src_page[x] * p.c.Hkv + h) * groups + gi) * kPage + src_slot[x];
        const long to = (((long)dst * p.c.Hkv + h) * groups + gi) * kPage + x;
        codes[to * 2 + half] = codes[from * 2 + half];
    }
#pragma unroll
    for (int i = tid; i < kGroups * kPage; i += 128) {
        const int g = i / kPage, x = i % kPage;
        if (src_page[x] < 0) continue;
        uint32_t* params = g >= GK ? p.c.v_params : p.c.k_params;
        const int groups = g >= GK ? GV : GK, gi = g >= GK ? g - GK : g;
        params[(((long)dst * p.c.Hkv + h) * groups + gi) * kPage + x] =
            params[(((long)src_page[x] * p.c.Hkv + h) * groups + gi) * kPage + src_slot[x]];
    }
}

// Rows per warp: up to four, which look their places up together, as long as
// that leaves 48 warps per SM (17000 rows of 8 heads, d = 128, append: 34 us with
// four rows per warp, 30 with two).
int rows_per_warp(int total, int num_sms) {
    const int rows = total / (num_sms * 48);
    return rows < 1 ? 1 : (rows > 4 ? 4 : rows);
}

template <int GK, int GV>
cudaError_t append_dims(const Kv4Cache& c, const Kv4Batch& s, const __nv_bfloat16* k, const __nv_bfloat16* v,
                        long k_stride, long v_stride, int* status, int num_sms, cudaStream_t stream) {
    const int rows = rows_per_warp(s.total, num_sms), per_block = 4 * rows;
    kv4_append_kernel<GK, GV><<<(s.total + per_block - 1) / per_block, 128, 0, stream>>>(c, s, k, v, k_stride, v_stride,
                                                                                        rows, status);
    return cudaGetLastError();
}
template <int GK, int GV>
cudaError_t read_dims(const Kv4Cache& c, const Kv4Batch& s, __nv_bfloat16* k, __nv_bfloat16* v, int* status,
                      int num_sms, cudaStream_t stream) {
    const int rows = rows_per_warp(s.total, num_sms), per_block = 4 * rows;
    kv4_read_kernel<GK, GV><<<(s.total + per_block - 1) / per_block, 128, 0, stream>>>(c, s, k, v, rows, status);
    return cudaGetLastError();
}
template <int GK, int GV>
cudaError_t gather_dims(const Kv4EvictParams& p, cudaStream_t stream) {
    const int tiles = (p.budget + kPage - 1) / kPage;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * p.c.Hkv * tiles));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_gather_kernel<GK, GV>, p, tiles);
}

// call(GK, GV) for the head dims of a cache
template <class F>
cudaError_t for_dims(const Kv4Cache& c, F call) {
    if (c.d == 64 && c.dv == 64) return call(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
    if (c.d == 128 && c.dv == 128) return call(std::integral_constant<int, 2>{}, std::integral_constant<int, 2>{});
    if (c.d == 192 && c.dv == 192) return call(std::integral_constant<int, 3>{}, std::integral_constant<int, 3>{});
    if (c.d == 192 && c.dv == 128) return call(std::integral_constant<int, 3>{}, std::integral_constant<int, 2>{});
    if (c.d == 256 && c.dv == 256) return call(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Cache& c, const Kv4Batch& s, const __nv_bfloat16* k, const __nv_bfloat16* v,
                              long k_stride, long v_stride, int* status, int num_sms, cudaStream_t stream) {
    return for_dims(c, [&](auto gk, auto gv) {
        return append_dims<gk.value, gv.value>(c, s, k, v, k_stride, v_stride, status, num_sms, stream);
    });
}

cudaError_t launch_kv4_read(const Kv4Cache& c, const Kv4Batch& s, __nv_bfloat16* k, __nv_bfloat16* v, int* status,
                            int num_sms, cudaStream_t stream) {
    return for_dims(c, [&](auto gk, auto gv) {
        return read_dims<gk.value, gv.value>(c, s, k, v, status, num_sms, stream);
    });
}

cudaError_t launch_kv4_evict(const Kv4EvictParams& p, cudaStream_t stream) {
    const int cap = p.width * kPage < kSelKeys ? p.width * kPage : kSelKeys;
    static std::atomic<unsigned long long> allowed{0};
    cudaError_t e = allow_smem(kv4_select_kernel, kSelKeys * 4, allowed);
    if (e != cudaSuccess) return e;
    kv4_select_kernel<<<p.B * p.c.Hkv, kSelThreads, cap * 4, stream>>>(p, cap);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return for_dims(p.c, [&](auto gk, auto gv) { return gather_dims<gk.value, gv.value>(p, stream); });
}

}  // namespace attn
