// Linear attention with a decay per head on tcgen05: head dims 128, 128 tokens a chunk.
// linear.h gives the form (a, b, c, the state X) that the forward and the gradients share,
// linear.cu the scan between the two kernels and the roundings.
//
// What bounds it: each chunk of a head brings 96 KB (32 KB each of a, b and c) and takes 32 KB
// of output; at HBM speed an SM gets that in about 5600 cycles, of which the four products of
// 128 x 128 x 128 take 2100 on the tensor cores (mma.sync, at a quarter of the rate and with its
// operands through registers, set the time). So one CTA per SM walks segments, with the
// next chunk's tiles in flight, and the roles
//   warps 0-3  P: scores from tensor memory, times the decays, back as bf16 (the next
//              product's A operand, over the scores' columns); b times the state's weights, in
//              place in shared memory, once the scores have been taken from it
//   warps 4-7  the state: X = D^n X + (the chunk's share), in registers in fp32, written to shared
//              memory in bf16 for the next chunk; and the outputs, P c + D^(..) a X
//   warp 8     tile loads (TMA), two stages
//   warp 9     the products:  P = a b^T;  O2 = a X;  O1 = P c;  KV = (w b)^T c
// Tensor memory: P (128 columns), O1, O2, KV: all 512. The tensor pipe executes in issue order,
// so the next chunk's scores may be issued behind the product that reads P. Every wait is bounded.
#include <atomic>

#include "kv4.h"
#include "linear.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kCh = 128;                 // tokens of a chunk
constexpr int kBox = 16384;              // 128 rows x 64 columns
constexpr int kTile = 2 * kBox;          // 128 x 128
constexpr uint32_t kTmemCols = 512, kTmP = 0, kTmO1 = 128, kTmO2 = 256, kTmKV = 384;

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ float lo16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi16(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// 16 bytes of a tile: row, piece of eight columns (128-byte swizzle, boxes of 64 columns)
__device__ __forceinline__ uint4* piece_at(uint8_t* tile, int row, int piece) {
    return reinterpret_cast<uint4*>(tile + (piece >> 3) * kBox + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}

// The walk over the CTA's (segment, head) pairs, the same for every warp.
struct Walk {
    int s, h, chunks, items, per;
    Segment g;
};
template <bool kBack>
__device__ __forceinline__ bool next_pair(const LinParams& p, int& k, Walk& w, bool all) {
    for (; k < p.segments * p.Hkv; k += gridDim.x) {
        w.s = k / p.Hkv;
        w.h = k - w.s * p.Hkv;
        w.g = segment_at(p, w.s);
        if (!w.g.live || w.g.r0 == w.g.r1) continue;
        if (!all && (kBack ? w.g.first : w.g.last)) continue;
        w.chunks = (w.g.r1 - w.g.r0 + kCh - 1) / kCh;
        k += gridDim.x;
        return true;
    }
    return false;
}
template <bool kBack>
__device__ __forceinline__ int chunk_row(const Walk& w, int chunk) {   // of the sequence
    return w.g.r0 + (kBack ? w.chunks - 1 - chunk : chunk) * kCh;
}

// ---------------------------------------------------------------- outputs
struct OutLay {
    static constexpr int kStage = 3 * kTile, kXOff = 2 * kStage, kBarOff = kXOff + kTile;
    static constexpr int kFull = 0, kEmpty = 2, kPFull = 4, kPReady = 5, kOFull = 6, kOFree = 7, kXReady = 8, kDrain = 9, kNumBars = 10;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8, kPowOff = kMiscOff + 16;   // D^0 .. D^31, per warp
    static constexpr int kBytes = kPowOff + 4 * 32 * 4 + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory budget");
};
constexpr int kOutThreads = 320;

template <bool kBack>
__global__ void __launch_bounds__(kOutThreads, 1)
lin_out_tc_kernel(const __grid_constant__ LinMaps maps, const LinParams p) {
    using Lay = OutLay;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) -> uint32_t { return base + Lay::kBarOff + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::kMiscOff + 4);
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(Lay::kFull + s), 1);
            mbar_init(bar(Lay::kEmpty + s), 1);
        }
        mbar_init(bar(Lay::kPFull), 1);
        mbar_init(bar(Lay::kPReady), 128);
        mbar_init(bar(Lay::kOFull), 1);
        mbar_init(bar(Lay::kOFree), 128);
        mbar_init(bar(Lay::kXReady), 128);
        mbar_init(bar(Lay::kDrain), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&maps.a);
        tma_prefetch_desc(&maps.b);
        tma_prefetch_desc(&maps.c);
    }
    if (warp == 9) {
        tmem_alloc(smem_addr(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx w{abort_flag, p.status, p.wait_budget_ns};
    const int per = p.per;
    Walk at;
    int k = blockIdx.x;

    if (warp == 8) {
        // ------------------------------------------------------------ loads
        uint32_t it = 0;
        bool ok = true;
        while (ok && next_pair<kBack>(p, k, at, true)) {
            for (int i = 0; i < at.chunks * per && ok; ++i, ++it) {
                const int chunk = i / per, x = i - chunk * per, row = at.g.q0 + chunk_row<kBack>(at, chunk);
                const int ha = kBack ? at.h : at.h * per + x, hb = kBack ? at.h * per + x : at.h;
                const uint32_t st = it & 1u;
                ok = warp_wait(bar(Lay::kEmpty + st), ((it >> 1) & 1u) ^ 1u, w, lane);
                if (ok && lane == 0) {
                    const uint32_t to = base + st * Lay::kStage, full = bar(Lay::kFull + st);
                    mbar_expect_tx(full, 3 * kTile);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        tma_load_3d(to + y * kBox, &maps.a, full, y * 64, ha, row);
                        tma_load_3d(to + kTile + y * kBox, &maps.b, full, y * 64, hb, row);
                        tma_load_3d(to + 2 * kTile + y * kBox, &maps.c, full, y * 64, hb, row);
                    }
                }
                __syncwarp();
            }
        }
        if (lane == 0)   // (a pending load must land before the CTA gives up its memory)
            for (uint32_t i = 0; i < 2 && i < it; ++i) {
                const uint32_t n = it - 1 - i;
                if (ok || i > 0) drain_wait(bar(Lay::kFull + (n & 1u)), (n >> 1) & 1u, p.wait_budget_ns);
            }
        __syncwarp();
    } else if (warp == 9) {
        // ------------------------------------------------------------ products
        constexpr uint32_t kIdP = idesc_bf16_f32(128, 128, false, false);    // a, b: rows of channels
        constexpr uint32_t kIdN = idesc_bf16_f32(128, 128, false, true);     // B (X, c): rows along the sum
        constexpr uint32_t kIdKV = idesc_bf16_f32(128, 128, true, true);     // (w b)^T, c: rows of tokens
        const SmemDesc a_km = sdesc_sw128_split(base, 16, 1024), b_km = sdesc_sw128_split(base + kTile, 16, 1024);
        const SmemDesc b_mn = sdesc_sw128_split(base + kTile, kBox, 1024), c_mn = sdesc_sw128_split(base + 2 * kTile, kBox, 1024);
        const SmemDesc x_mn = sdesc_sw128_split(base + Lay::kXOff, kBox, 1024);
        uint32_t it = 0, outs = 0, xs = 0;   // items, rounds of the outputs' columns, states
        bool ok = true;
        while (ok && next_pair<kBack>(p, k, at, true)) {
            for (int i = 0; i < at.chunks * per; ++i, ++it) {
                const int x = i % per;
                const uint32_t st = it & 1u, off = desc_step(st * Lay::kStage);
                const bool head = !kBack || x == 0, tail = !kBack || x == per - 1;   // of a round of the outputs
                const bool shares = kBack || x == per - 1;                          // this item adds to the state
                if (!(ok = warp_wait(bar(Lay::kFull + st), (it >> 1) & 1u, w, lane))) break;
                tc_fence_after_sync();
                if (lane == 0) {
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const uint32_t step = desc_step((y >> 2) * kBox + (y & 3) * 32);
                        mma_ss(tmem + kTmP, a_km, off + step, b_km, off + step, kIdP, y > 0);
                    }
                    tc_commit(bar(Lay::kPFull));
                }
                __syncwarp();
                if (head) {
                    if (x == 0) {
                        if (!(ok = warp_wait(bar(Lay::kXReady), xs & 1u, w, lane))) break;
                        ++xs;
                    }
                    if (!(ok = warp_wait(bar(Lay::kOFree), (outs & 1u) ^ 1u, w, lane))) break;
                    tc_fence_after_sync();
                    if (lane == 0)
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            mma_ss(tmem + kTmO2, a_km, off + desc_step((y >> 2) * kBox + (y & 3) * 32), x_mn, desc_step(y * 2048),
                                   kIdN, y > 0);
                    __syncwarp();
                }
                if (!(ok = warp_wait(bar(Lay::kPReady), it & 1u, w, lane))) break;
                tc_fence_after_sync();
                if (lane == 0) {
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        mma_ts(tmem + kTmO1, tmem + kTmP + y * 8, c_mn, off + desc_step(y * 2048), kIdN, !head || y > 0);
                    if (shares)
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            mma_ss(tmem + kTmKV, b_mn, off + desc_step(y * 2048), c_mn, off + desc_step(y * 2048), kIdKV,
                                   (kBack && x > 0) || y > 0);
                    tc_commit(bar(Lay::kEmpty + st));
                    if (tail) tc_commit(bar(Lay::kOFull));
                }
                __syncwarp();
                if (tail) ++outs;
            }
        }
        if (lane == 0) {
            tc_commit(bar(Lay::kDrain));
            drain_wait(bar(Lay::kDrain), 0, p.wait_budget_ns);
        }
        __syncwarp();
    } else if (warp < 4) {
        // ------------------------------------------------------------ P, and the weights on b
        const uint32_t t_p = tmem + ((uint32_t)(warp * 32) << 16) + kTmP;
        float* pow = reinterpret_cast<float*>(smem + Lay::kPowOff) + warp * 32;
        uint32_t it = 0;
        bool ok = true;
        float l2 = 0.f;
        int head_of = -1;
        while (ok && next_pair<kBack>(p, k, at, true)) {
            if (at.h != head_of) {
                l2 = log2_decay(p, at.h);
                head_of = at.h;
                __syncwarp();
                pow[lane] = decay_pow(l2, lane);
                __syncwarp();
            }
            const int row = warp * 32 + lane;
            // to columns of a block of 32 on the near side: the distance to the block's nearer end, then pow[]
            float far[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int d = kBack ? 32 * b - row : row - 32 * b - 31;
                far[b] = d >= 0 ? decay_pow(l2, d) : 0.f;
            }
            for (int i = 0; i < at.chunks * per; ++i, ++it) {
                const int chunk = i / per, x = i - chunk * per;
                const int n = min(kCh, at.g.r1 - chunk_row<kBack>(at, chunk));
                const bool shares = kBack || x == per - 1;
                const float weight = row < n ? decay_pow(l2, kBack ? row + 1 : n - 1 - row) : 0.f;
                uint8_t* tiles = smem + (it & 1u) * Lay::kStage;
                if (!(ok = warp_wait(bar(Lay::kPFull), it & 1u, w, lane))) break;
                tc_fence_after_sync();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t out[32];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int b = 2 * half + y;   // columns 32 b .. + 31
                        const bool near = kBack ? b > warp : b < warp;
                        if (near || b == warp) {
                            uint32_t r[32];
                            tmem_ld32(t_p + 32 * b, r);
                            if (near) {
                                const float f = far[b];
                                const int end = n - 32 * b;   // (backwards: the columns that exist)
#pragma unroll
                                for (int c = 0; c < 32; c += 4) {
                                    const float4 t = *reinterpret_cast<const float4*>(pow + (kBack ? c : 28 - c));
                                    const float q[4] = {kBack ? t.x : t.w, kBack ? t.y : t.z, kBack ? t.z : t.y, kBack ? t.w : t.x};
                                    float v[4];
#pragma unroll
                                    for (int z = 0; z < 4; ++z)
                                        v[z] = kBack && c + z >= end ? 0.f : __uint_as_float(r[c + z]) * (f * q[z]);
                                    out[16 * y + c / 2] = pack_bf16x2(v[0], v[1]);
                                    out[16 * y + c / 2 + 1] = pack_bf16x2(v[2], v[3]);
                                }
                            } else {
#pragma unroll
                                for (int c = 0; c < 32; c += 2) {
                                    const int d0 = kBack ? c - lane : lane - c, d1 = kBack ? d0 + 1 : d0 - 1;
                                    const float v0 = d0 >= 0 && (!kBack || 32 * b + c < n) ? __uint_as_float(r[c]) * pow[d0] : 0.f;
                                    const float v1 = d1 >= 0 && (!kBack || 32 * b + c + 1 < n) ? __uint_as_float(r[c + 1]) * pow[d1] : 0.f;
                                    out[16 * y + c / 2] = pack_bf16x2(v0, v1);
                                }
                            }
                        } else {
#pragma unroll
                            for (int c = 0; c < 16; ++c) out[16 * y + c] = 0u;
                        }
                    }
                    tmem_st32(t_p + 32 * half, out);
                }
                if (n < kCh && row >= n) {   // c's rows past the sequence's end, whatever they hold
#pragma unroll
                    for (int c = 0; c < 16; ++c) *piece_at(tiles + 2 * kTile, row, c) = make_uint4(0, 0, 0, 0);
                }
                if (shares) {   // (the scores have been taken: b may change)
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        uint4* at16 = piece_at(tiles + kTile, row, c);
                        const uint4 v = *at16;
                        auto scaled = [&](uint32_t u) { return pack_bf16x2(lo16(u) * weight, hi16(u) * weight); };
                        *at16 = row < n ? make_uint4(scaled(v.x), scaled(v.y), scaled(v.z), scaled(v.w)) : make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tmem_st_wait();
                tc_fence_before_sync();
                mbar_arrive(bar(Lay::kPReady));
            }
        }
    } else {
        // ------------------------------------------------------------ the state and the outputs
        const int row = (warp & 3) * 32 + lane;   // of X (a channel) and of the outputs (a token)
        const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        uint8_t* xs = smem + Lay::kXOff;
        uint32_t outs = 0;
        bool ok = true;
        float X[128];
        auto store_x = [&] {
#pragma unroll
            for (int c = 0; c < 16; ++c)
                *piece_at(xs, row, c) = make_uint4(pack_bf16x2(X[8 * c], X[8 * c + 1]), pack_bf16x2(X[8 * c + 2], X[8 * c + 3]),
                                                   pack_bf16x2(X[8 * c + 4], X[8 * c + 5]), pack_bf16x2(X[8 * c + 6], X[8 * c + 7]));
            fence_proxy_async_smem();
            mbar_arrive(bar(Lay::kXReady));
        };
        while (ok && next_pair<kBack>(p, k, at, true)) {
            const float l2 = log2_decay(p, at.h);
            const float* src = lin_state_src(p, at.s, at.g.b, at.h);
            const float mul = p.split() ? 1.f : p.init_mul;
            if (!src) {
#pragma unroll
                for (int c = 0; c < 128; ++c) X[c] = 0.f;
            } else if (p.split() ? p.states_trans : p.init_trans) {
#pragma unroll
                for (int c = 0; c < 128; ++c) X[c] = mul * src[c * 128 + row];
            } else {
#pragma unroll
                for (int c = 0; c < 128; c += 4) {
                    const float4 y = *reinterpret_cast<const float4*>(src + row * 128 + c);
                    X[c] = mul * y.x, X[c + 1] = mul * y.y, X[c + 2] = mul * y.z, X[c + 3] = mul * y.w;
                }
            }
            store_x();   // (the products that read the last pair's are done: its last round of outputs was waited for)
            for (int chunk = 0; chunk < at.chunks && ok; ++chunk) {
                const int r0 = chunk_row<kBack>(at, chunk), n = min(kCh, at.g.r1 - r0);
                const float into = row < n ? decay_pow(l2, kBack ? n - 1 - row : row + 1) : 0.f;
                for (int x = 0; x < (kBack ? 1 : per); ++x, ++outs) {
                    if (!(ok = warp_wait(bar(Lay::kOFull), outs & 1u, w, lane))) break;
                    tc_fence_after_sync();
                    if ((kBack || x == per - 1) && chunk + 1 < at.chunks) {
                        const float over = decay_pow(l2, n);
#pragma unroll
                        for (int c = 0; c < 128; c += 16) {
                            uint32_t r[16];
                            tmem_ld16(t_row + kTmKV + c, r);
#pragma unroll
                            for (int z = 0; z < 16; ++z) X[c + z] = fmaf(X[c + z], over, __uint_as_float(r[z]));
                        }
                        store_x();
                    }
                    __nv_bfloat16* out = p.out + ((long)(at.g.q0 + r0 + row) * (kBack ? p.Hkv : p.Hkv * per) + (kBack ? at.h : at.h * per + x)) * 128;
#pragma unroll
                    for (int c = 0; c < 128; c += 16) {
                        uint32_t o1[16], o2[16], o[8];
                        tmem_ld16(t_row + kTmO1 + c, o1);
                        tmem_ld16(t_row + kTmO2 + c, o2);
#pragma unroll
                        for (int z = 0; z < 8; ++z)
                            o[z] = pack_bf16x2(p.out_mul * fmaf(into, __uint_as_float(o2[2 * z]), __uint_as_float(o1[2 * z])),
                                               p.out_mul * fmaf(into, __uint_as_float(o2[2 * z + 1]), __uint_as_float(o1[2 * z + 1])));
                        if (row < n) {
                            *reinterpret_cast<uint4*>(out + c) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4*>(out + c + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                    }
                    tc_fence_before_sync();
                    mbar_arrive(bar(Lay::kOFree));
                }
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- segments' shares
// X' of a segment for X = 0: one sum over its tokens in tensor memory, each weighted by the
// decay up to the segment's end (backwards: its start), b times that weight in three bf16 terms
// (all of its 24 bits): the first in place, the others in buffers of 64 tokens, two of each.
struct StateLay {
    static constexpr int kStage = 2 * kTile, kTermOff = 2 * kStage, kTerm = kTile / 2;   // [buffer][term] of 64 x 128
    static constexpr int kBarOff = kTermOff + 4 * kTerm;
    static constexpr int kFull = 0, kEmpty = 2, kWReady = 4, kWFree = 6, kSFull = 8, kSFree = 10, kDrain = 12, kNumBars = 13;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8, kBytes = kMiscOff + 16 + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory budget");
};
constexpr int kStateThreads = 448;   // warps 0-7: weights, 8-11: results, 12: loads, 13: products

template <bool kBack>
__global__ void __launch_bounds__(kStateThreads, 1)
lin_state_tc_kernel(const __grid_constant__ LinMaps maps, const LinParams p) {
    using Lay = StateLay;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) -> uint32_t { return base + Lay::kBarOff + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::kMiscOff + 4);
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(Lay::kFull + s), 1);
            mbar_init(bar(Lay::kEmpty + s), 1);
            mbar_init(bar(Lay::kWReady + s), 256);
            mbar_init(bar(Lay::kWFree + s), 1);
            mbar_init(bar(Lay::kSFull + s), 1);
            mbar_init(bar(Lay::kSFree + s), 128);
        }
        mbar_init(bar(Lay::kDrain), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 12 && lane == 0) {
        tma_prefetch_desc(&maps.b);
        tma_prefetch_desc(&maps.c);
    }
    if (warp == 13) {
        tmem_alloc(smem_addr(tmem_slot), 256);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx w{abort_flag, p.status, p.wait_budget_ns};
    const int per = kBack ? p.per : 1;
    const bool all = p.final != nullptr;
    Walk at;
    int k = blockIdx.x;

    if (warp == 12) {
        // ------------------------------------------------------------ loads
        uint32_t it = 0;
        bool ok = true;
        while (ok && next_pair<kBack>(p, k, at, all)) {
            for (int i = 0; i < at.chunks * per && ok; ++i, ++it) {
                const int chunk = i / per, x = i - chunk * per, row = at.g.q0 + chunk_row<kBack>(at, chunk);
                const int hb = at.h * per + x;
                const uint32_t st = it & 1u;
                ok = warp_wait(bar(Lay::kEmpty + st), ((it >> 1) & 1u) ^ 1u, w, lane);
                if (ok && lane == 0) {
                    const uint32_t to = base + st * Lay::kStage, full = bar(Lay::kFull + st);
                    mbar_expect_tx(full, 2 * kTile);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        tma_load_3d(to + y * kBox, &maps.b, full, y * 64, hb, row);
                        tma_load_3d(to + kTile + y * kBox, &maps.c, full, y * 64, hb, row);
                    }
                }
                __syncwarp();
            }
        }
        if (lane == 0)
            for (uint32_t i = 0; i < 2 && i < it; ++i) {
                const uint32_t n = it - 1 - i;
                if (ok || i > 0) drain_wait(bar(Lay::kFull + (n & 1u)), (n >> 1) & 1u, p.wait_budget_ns);
            }
        __syncwarp();
    } else if (warp == 13) {
        // ------------------------------------------------------------ products
        constexpr uint32_t kIdKV = idesc_bf16_f32(128, 128, true, true);
        const SmemDesc b_mn = sdesc_sw128_split(base, kBox, 1024), c_mn = sdesc_sw128_split(base + kTile, kBox, 1024);
        const SmemDesc t_mn = sdesc_sw128_split(base + Lay::kTermOff, Lay::kTerm / 2, 1024);   // (boxes of 64 rows)
        uint32_t it = 0, pairs = 0;
        bool ok = true;
        while (ok && next_pair<kBack>(p, k, at, all)) {
            const uint32_t acc = tmem + (pairs & 1u) * 128;
            if (!(ok = warp_wait(bar(Lay::kSFree + (pairs & 1u)), ((pairs >> 1) & 1u) ^ 1u, w, lane))) break;
            for (int i = 0; i < at.chunks * per && ok; ++i, ++it) {
                const uint32_t st = it & 1u, off = desc_step(st * Lay::kStage);
                for (int half = 0; half < 2; ++half) {
                    if (!(ok = warp_wait(bar(Lay::kWReady + half), it & 1u, w, lane))) break;
                    tc_fence_after_sync();
                    if (lane == 0) {
                        const uint32_t c0 = off + desc_step(half * 8192);
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            mma_ss(acc, b_mn, c0 + desc_step(y * 2048), c_mn, c0 + desc_step(y * 2048), kIdKV, i > 0 || half > 0 || y > 0);
#pragma unroll
                        for (int term = 0; term < 2; ++term)
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                mma_ss(acc, t_mn, desc_step((2 * half + term) * Lay::kTerm + y * 2048), c_mn, c0 + desc_step(y * 2048), kIdKV, 1);
                        tc_commit(bar(Lay::kWFree + half));
                        if (half == 1) tc_commit(bar(Lay::kEmpty + st));
                        if (half == 1 && i + 1 == at.chunks * per) tc_commit(bar(Lay::kSFull + (pairs & 1u)));
                    }
                    __syncwarp();
                }
            }
            ++pairs;
        }
        if (lane == 0) {
            tc_commit(bar(Lay::kDrain));
            drain_wait(bar(Lay::kDrain), 0, p.wait_budget_ns);
        }
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------------------ weights
        // a thread takes pieces x, x + 4, .. of a row, so that eight neighbouring rows lie in eight banks
        const int r64 = tid & 63, p0 = tid >> 6;
        uint32_t it = 0;
        bool ok = true;
        while (ok && next_pair<kBack>(p, k, at, all)) {
            const float l2 = log2_decay(p, at.h);
            for (int i = 0; i < at.chunks * per && ok; ++i, ++it) {
                const int r0 = chunk_row<kBack>(at, i / per);
                const uint32_t st = it & 1u;
                uint8_t* tiles = smem + st * Lay::kStage;
                if (!(ok = warp_wait(bar(Lay::kFull + st), (it >> 1) & 1u, w, lane))) break;
                for (int half = 0; half < 2; ++half) {
                    const int row = half * 64 + r64, r = r0 + row;
                    const bool in = r < at.g.r1;
                    const float weight = in ? decay_pow(l2, kBack ? r - at.g.r0 + 1 : at.g.r1 - 1 - r) : 0.f;
                    uint8_t* terms = smem + Lay::kTermOff + 2 * half * Lay::kTerm;
                    if (!(ok = warp_wait(bar(Lay::kWFree + half), (it & 1u) ^ 1u, w, lane))) break;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int c = p0 + 4 * y;
                        uint4* at16 = piece_at(tiles, row, c);
                        const uint4 v = *at16;
                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                        uint32_t o[3][4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            float f0 = lo16(u[z]) * weight, f1 = hi16(u[z]) * weight;
#pragma unroll
                            for (int term = 0; term < 3; ++term) {
                                o[term][z] = in ? pack_bf16x2(f0, f1) : 0u;
                                f0 -= lo16(o[term][z]);
                                f1 -= hi16(o[term][z]);
                            }
                        }
                        *at16 = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
#pragma unroll
                        for (int term = 1; term < 3; ++term)
                            *reinterpret_cast<uint4*>(terms + (term - 1) * Lay::kTerm + (c >> 3) * (Lay::kTerm / 2) + r64 * 128 +
                                                      (((c & 7) ^ (r64 & 7)) << 4)) =
                                make_uint4(o[term][0], o[term][1], o[term][2], o[term][3]);
                        if (!in) *piece_at(tiles + kTile, row, c) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(bar(Lay::kWReady + half));
                }
            }
        }
    } else {
        // ------------------------------------------------------------ results
        const int row = (warp & 3) * 32 + lane;
        uint32_t pairs = 0;
        bool ok = true;
        while (ok && next_pair<kBack>(p, k, at, all)) {
            if (!(ok = warp_wait(bar(Lay::kSFull + (pairs & 1u)), (pairs >> 1) & 1u, w, lane))) break;
            tc_fence_after_sync();
            float* dst = p.states + (((long)at.s * p.Hkv + at.h) * 128 + row) * 128;
            const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (pairs & 1u) * 128;
#pragma unroll
            for (int c = 0; c < 128; c += 16) {
                uint32_t r[16];
                tmem_ld16(t_row + c, r);
#pragma unroll
                for (int z = 0; z < 16; z += 4) *reinterpret_cast<uint4*>(dst + c + z) = make_uint4(r[z], r[z + 1], r[z + 2], r[z + 3]);
            }
            tc_fence_before_sync();
            mbar_arrive(bar(Lay::kSFree + (pairs & 1u)));
            ++pairs;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 256);
    }
}

template <class Kernel>
cudaError_t launch_tc(Kernel kern, int threads, int bytes, std::atomic<unsigned long long>& allowed, const LinParams& p,
                      const LinMaps& maps, int num_sms, cudaStream_t stream) {
    cudaError_t e = allow_smem(kern, bytes, allowed);
    if (e != cudaSuccess) return e;
    const long pairs = (long)p.segments * p.Hkv;
    kern<<<(unsigned)(pairs < num_sms ? pairs : num_sms), threads, bytes, stream>>>(maps, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_state_tc(const LinParams& p, const LinMaps& maps, bool back, int num_sms, cudaStream_t stream) {
    static std::atomic<unsigned long long> allowed[2];
    return launch_tc(back ? lin_state_tc_kernel<true> : lin_state_tc_kernel<false>, kStateThreads, StateLay::kBytes, allowed[back],
                     p, maps, num_sms, stream);
}
cudaError_t launch_linear_out_tc(const LinParams& p, const LinMaps& maps, bool back, int num_sms, cudaStream_t stream) {
    static std::atomic<unsigned long long> allowed[2];
    return launch_tc(back ? lin_out_tc_kernel<true> : lin_out_tc_kernel<false>, kOutThreads, OutLay::kBytes, allowed[back], p, maps,
                     num_sms, stream);
}

}  // namespace attn
