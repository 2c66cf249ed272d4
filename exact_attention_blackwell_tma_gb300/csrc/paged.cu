// The paged cache in bf16 or 8 bits: append (quantise) and read. Bound by memory:
// each value is touched once. A warp takes a few consecutive tokens, whose places
// its first lanes look up together. An append walks their heads, kAhead of them with
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
// One token's K and V rows, all heads, in pieces of eight channels (16 bytes of output): a lane's pieces
// lie 32 apart, kPieces of them with their loads in flight (two: 112 us; four 119, eight 135, see tokens_per_warp).
template <bool kCodes, int D, int DV>
__device__ __forceinline__ void read_token(__nv_bfloat16* k, __nv_bfloat16* v, const PagedCache& c, long page, int slot, int lane) {
    constexpr int PK = D / 8, PV = DV / 8, kPieces = 2;
    const int of_k = c.Hkv * PK, all = of_k + c.Hkv * PV;
    for (int p0 = lane; p0 < all; p0 += 32 * kPieces) {
        uint4 x[kPieces];
        uint32_t e[kPieces];
#pragma unroll
        for (int y = 0; y < kPieces; ++y) {
            const int p = min(p0 + 32 * y, all - 1), q = p < of_k ? p : p - of_k, h = p < of_k ? q / PK : q / PV;
            const long row = (max(page, 0l) * c.Hkv + h) * kPage + slot;
            const long at = p < of_k ? row * D + (q - h * PK) * 8 : row * DV + (q - h * PV) * 8;   // channels
            const unsigned char* src = p < of_k ? c.k : c.v;
            if constexpr (kCodes) {
                const uint2 w = __ldg(reinterpret_cast<const uint2*>(src + at));
                x[y].x = w.x, x[y].y = w.y;
                e[y] = __ldg((p < of_k ? c.k_scales : c.v_scales) + row);
            } else {
                x[y] = __ldg(reinterpret_cast<const uint4*>(src + 2 * at));
            }
        }
#pragma unroll
        for (int y = 0; y < kPieces; ++y) {
            const int p = p0 + 32 * y;
            if (p >= all) break;
            if constexpr (kCodes) {
                const float f = paged_scale(e[y]);
                const uint32_t w[2] = {x[y].x, x[y].y};
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 z = e4m3_values((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
                    o[i] = pack_bf16x2(z.x * f, z.y * f);
                }
                x[y] = make_uint4(o[0], o[1], o[2], o[3]);
            }
            if (page < 0) x[y] = make_uint4(0, 0, 0, 0);   // (a row that lies nowhere reads as zero)
            *reinterpret_cast<uint4*>(p < of_k ? k + p * 8 : v + (p - of_k) * 8) = x[y];
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
        read_token<kCodes, D, DV>(k + (long)(t0 + x) * c.Hkv * D, v + (long)(t0 + x) * c.Hkv * DV, c, page, slot, lane);
    }
}

// Tokens per warp: two where that leaves 48 warps per SM (a chunked prefill of 12000 tokens and the 70000 of its prefix
// read back, 8 heads, 8 bits: 112 us; 119 with four, 153 with all in one wave: neighbouring tokens of a page should be
// read together)
int tokens_per_warp(int total, int num_sms) {
    const int rows = total / (num_sms * 48);
    return rows < 1 ? 1 : (rows > 2 ? 2 : rows);
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
