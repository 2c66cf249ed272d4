// The paged cache in bf16 or 8 bits: append (quantise) and read. Bound by memory:
// each value is touched once. A warp takes a few consecutive tokens, whose places
// its first lanes look up together, and walks their heads, kAhead of them with
// their loads in flight; a lane holds d / 32 neighbouring channels of a head.
#include <type_traits>

#include <cuda_fp16.h>

#include "paged.h"

namespace attn {
namespace {

constexpr int kPagedThreads = 128, kAhead = 4;

// D / 64 words of two bf16, or as many half words of two codes
template <int W>
struct Words {
    uint32_t x[W];
};
template <int W>
__device__ __forceinline__ Words<W> load_words(const void* p) {
    Words<W> r;
    if constexpr (W == 4) {
        const uint4 v = __ldg(static_cast<const uint4*>(p));
        r.x[0] = v.x, r.x[1] = v.y, r.x[2] = v.z, r.x[3] = v.w;
    } else if constexpr (W == 2) {
        const uint2 v = __ldg(static_cast<const uint2*>(p));
        r.x[0] = v.x, r.x[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) r.x[i] = __ldg(static_cast<const uint32_t*>(p) + i);
    }
    return r;
}
template <int W>
__device__ __forceinline__ void store_words(void* p, const Words<W>& r) {
    if constexpr (W == 4) *static_cast<uint4*>(p) = make_uint4(r.x[0], r.x[1], r.x[2], r.x[3]);
    else if constexpr (W == 2) *static_cast<uint2*>(p) = make_uint2(r.x[0], r.x[1]);
    else {
#pragma unroll
        for (int i = 0; i < W; ++i) static_cast<uint32_t*>(p)[i] = r.x[i];
    }
}
// W pairs of codes, 2 W bytes
template <int W>
__device__ __forceinline__ void load_codes(const unsigned char* p, uint16_t (&c)[W]) {
    if constexpr (W == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        c[0] = v.x & 0xffff, c[1] = v.x >> 16, c[2] = v.y & 0xffff, c[3] = v.y >> 16;
    } else if constexpr (W == 2) {
        const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(p));
        c[0] = v & 0xffff, c[1] = v >> 16;
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) c[i] = __ldg(reinterpret_cast<const uint16_t*>(p) + i);
    }
}
template <int W>
__device__ __forceinline__ void store_codes(unsigned char* p, const uint16_t (&c)[W]) {
    if constexpr (W == 4)
        *reinterpret_cast<uint2*>(p) = make_uint2(c[0] | (uint32_t)c[1] << 16, c[2] | (uint32_t)c[3] << 16);
    else if constexpr (W == 2) *reinterpret_cast<uint32_t*>(p) = c[0] | (uint32_t)c[1] << 16;
    else {
#pragma unroll
        for (int i = 0; i < W; ++i) reinterpret_cast<uint16_t*>(p)[i] = c[i];
    }
}
__device__ __forceinline__ uint16_t e4m3_pair(float lo, float hi) {   // round to nearest even, |x| <= 448
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 e4m3_values(uint16_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Quantise one head's row, 2 W channels per lane. With |x| at most m = 1.f 2^(E - 127)
// the scale's exponent is the least e with m <= 448 2^e = 1.75 2^(8 + e): E - 8 as a
// biased byte, one more where f > 1.75; from 1 (2^-126) up. x 2^-e is exact in fp32.
template <int W>
__device__ __forceinline__ void quantise(const Words<W>& r, unsigned char* codes, unsigned char* scale) {
    uint32_t m = 0;   // the largest magnitude of both halves, as bf16 bits
#pragma unroll
    for (int i = 0; i < W; ++i) m = __vmaxu2(m, r.x[i] & 0x7fff7fffu);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = max(m & 0xffffu, m >> 16);
    const bool finite = m < 0x7f80u;
    const int e = finite ? max(1, (int)(m >> 7) - 8 + ((m & 0x7fu) > 0x60u ? 1 : 0)) : 255;
    const float inv = finite ? __uint_as_float((uint32_t)(254 - e) << 23) : 0.f;
    uint16_t c[W];
#pragma unroll
    for (int i = 0; i < W; ++i)
        c[i] = finite ? e4m3_pair(__uint_as_float(r.x[i] << 16) * inv, __uint_as_float(r.x[i] & 0xffff0000u) * inv) : (uint16_t)0;
    store_codes<W>(codes, c);
    if ((threadIdx.x & 31) == 0) *scale = (unsigned char)e;
}

// Heads of one token's K or V: D channels each
template <bool kCodes, int D>
__device__ __forceinline__ void append_row(const __nv_bfloat16* src, unsigned char* rows, unsigned char* scales, int Hkv,
                                           long page, int slot, int lane) {
    constexpr int W = D / 64;
    for (int h0 = 0; h0 < Hkv; h0 += kAhead) {
        Words<W> r[kAhead];
#pragma unroll
        for (int y = 0; y < kAhead; ++y) r[y] = load_words<W>(src + (long)min(h0 + y, Hkv - 1) * D + lane * 2 * W);
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            if (h0 + y >= Hkv) break;
            const long at = (page * Hkv + h0 + y) * kPage + slot;
            if constexpr (kCodes) quantise<W>(r[y], rows + at * D + lane * 2 * W, scales + at);
            else store_words<W>(rows + (at * D + lane * 2 * W) * 2, r[y]);
        }
    }
}
template <bool kCodes, int D>
__device__ __forceinline__ void read_row(__nv_bfloat16* dst, const unsigned char* rows, const unsigned char* scales, int Hkv,
                                         long page, int slot, int lane) {
    constexpr int W = D / 64;
    for (int h0 = 0; h0 < Hkv; h0 += kAhead) {
        Words<W> r[kAhead];
        uint16_t c[kAhead][W];
        uint32_t e[kAhead];
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            const long at = (max(page, 0l) * Hkv + min(h0 + y, Hkv - 1)) * kPage + slot;
            if constexpr (kCodes) {
                load_codes<W>(rows + at * D + lane * 2 * W, c[y]);
                e[y] = __ldg(scales + at);
            } else {
                r[y] = load_words<W>(rows + (at * D + lane * 2 * W) * 2);
            }
        }
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            if (h0 + y >= Hkv) break;
            if constexpr (kCodes) {
                const float f = __uint_as_float(e[y] << 23);   // (255: infinity, times codes of 0: NaN)
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const float2 x = e4m3_values(c[y][i]);
                    r[y].x[i] = pack_bf16x2(x.x * f, x.y * f);
                }
            }
            if (page < 0) {   // (a row that lies nowhere reads as zero)
#pragma unroll
                for (int i = 0; i < W; ++i) r[y].x[i] = 0u;
            }
            store_words<W>(dst + (long)(h0 + y) * D + lane * 2 * W, r[y]);
        }
    }
}

template <bool kCodes, int D, int DV>
__global__ void __launch_bounds__(kPagedThreads) paged_append_kernel(PagedCache c, Kv4Batch s, const __nv_bfloat16* k,
                                                                     const __nv_bfloat16* v, long k_stride, long v_stride,
                                                                     int rows, int* status) {
    const int lane = threadIdx.x & 31;
    const int t0 = (blockIdx.x * (kPagedThreads / 32) + threadIdx.x / 32) * rows;
    RowPlace mine{-2, 0};
    if (lane < rows) {
        mine = place_of(c.n_pages, s, t0 + lane, status);
        if (mine.page == -3) bad_page(status);   // more new rows than the cache holds tokens
    }
    for (int x = 0; x < rows; ++x) {
        const int page = __shfl_sync(0xffffffffu, mine.page, x), slot = __shfl_sync(0xffffffffu, mine.slot, x);
        if (page < 0) continue;
        append_row<kCodes, D>(k + (t0 + x) * k_stride, c.k, c.k_scales, c.Hkv, page, slot, lane);
        append_row<kCodes, DV>(v + (t0 + x) * v_stride, c.v, c.v_scales, c.Hkv, page, slot, lane);
    }
}

template <bool kCodes, int D, int DV>
__global__ void __launch_bounds__(kPagedThreads) paged_read_kernel(PagedCache c, Kv4Batch s, __nv_bfloat16* k,
                                                                   __nv_bfloat16* v, int rows, int* status) {
    const int lane = threadIdx.x & 31;
    const int t0 = (blockIdx.x * (kPagedThreads / 32) + threadIdx.x / 32) * rows;
    RowPlace mine{-2, 0};
    if (lane < rows) mine = place_of(c.n_pages, s, t0 + lane, status);
    for (int x = 0; x < rows; ++x) {
        const int page = __shfl_sync(0xffffffffu, mine.page, x), slot = __shfl_sync(0xffffffffu, mine.slot, x);
        if (page == -2) continue;
        read_row<kCodes, D>(k + (long)(t0 + x) * c.Hkv * D, c.k, c.k_scales, c.Hkv, page, slot, lane);
        read_row<kCodes, DV>(v + (long)(t0 + x) * c.Hkv * DV, c.v, c.v_scales, c.Hkv, page, slot, lane);
    }
}

// Tokens per warp: up to four, as long as that leaves 48 warps per SM
int tokens_per_warp(int total, int num_sms) {
    const int rows = total / (num_sms * 48);
    return rows < 1 ? 1 : (rows > 4 ? 4 : rows);
}

// call(D, DV) for the head dims of a cache
template <class F>
cudaError_t for_dims(const PagedCache& c, F call) {
    if (c.d == 64 && c.dv == 64) return call(std::integral_constant<int, 64>{}, std::integral_constant<int, 64>{});
    if (c.d == 128 && c.dv == 128) return call(std::integral_constant<int, 128>{}, std::integral_constant<int, 128>{});
    if (c.d == 192 && c.dv == 192) return call(std::integral_constant<int, 192>{}, std::integral_constant<int, 192>{});
    if (c.d == 192 && c.dv == 128) return call(std::integral_constant<int, 192>{}, std::integral_constant<int, 128>{});
    if (c.d == 256 && c.dv == 256) return call(std::integral_constant<int, 256>{}, std::integral_constant<int, 256>{});
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_append(const PagedCache& c, bool codes, const Kv4Batch& s, const __nv_bfloat16* k,
                                const __nv_bfloat16* v, long k_stride, long v_stride, int* status, int num_sms,
                                cudaStream_t stream) {
    const int rows = tokens_per_warp(s.total, num_sms), per_block = kPagedThreads / 32 * rows;
    const int grid = (s.total + per_block - 1) / per_block;
    return for_dims(c, [&](auto d, auto dv) {
        auto kern = codes ? paged_append_kernel<true, d.value, dv.value> : paged_append_kernel<false, d.value, dv.value>;
        kern<<<grid, kPagedThreads, 0, stream>>>(c, s, k, v, k_stride, v_stride, rows, status);
        return cudaGetLastError();
    });
}

cudaError_t launch_paged_read(const PagedCache& c, bool codes, const Kv4Batch& s, __nv_bfloat16* k, __nv_bfloat16* v,
                              int* status, int num_sms, cudaStream_t stream) {
    const int rows = tokens_per_warp(s.total, num_sms), per_block = kPagedThreads / 32 * rows;
    const int grid = (s.total + per_block - 1) / per_block;
    return for_dims(c, [&](auto d, auto dv) {
        auto kern = codes ? paged_read_kernel<true, d.value, dv.value> : paged_read_kernel<false, d.value, dv.value>;
        kern<<<grid, kPagedThreads, 0, stream>>>(c, s, k, v, rows, status);
        return cudaGetLastError();
    });
}

}  // namespace attn
