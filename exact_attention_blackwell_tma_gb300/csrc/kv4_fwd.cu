// Attention of a few new tokens per sequence over the 4-bit key/value cache.
//
// Mathematics. A code c of key j, channel group g stands for a_jg c + b_jg, so
//   s_ij = scale * sum_g ( a_jg <q_ig, c_jg> + b_jg sum(q_ig) )
//   O_i  = sum_j p_ij v_j,   v_j = a'_jg c'_jg + b'_jg:
// the products run on the 4-bit codes themselves and the parameters enter as one
// factor per (key, group) in fp32 (scores) or fold into P (values); nothing is
// dequantised element by element.
//
// What bounds it: the cache is read once (4.5 bits per element) by 152 SMs at
// HBM speed, about 45 bytes per ns and SM, i.e. 80 codes per ns to turn into
// MMA operands. So the layout of the products is chosen for cheap operands and
// small row counts: keys (channels for PV) take the M side and the query rows
// the N side of mma.sync m16n8k16,
//   S^T[key, row] = codes[key, ch] q^T[ch, row],
//   O^T[ch, row] += codes^T[ch, key] P^T[key, row],
// which pads rows to 8 instead of 16 (64 or 128 for a tcgen05 tile, whose
// operands would also have to pass through shared memory again as 16-bit
// values: more shared-memory traffic than the cache itself). A code becomes an
// fp16 operand by one AND: the bits 0-3 (4-7) of a half are the subnormal
// c 2^-24 (c 2^-20), which the tensor cores take exactly; the powers of two go
// into q and the epilogue. Two codes per AND, one shift per eight.
//
// P^T: the accumulator tile of S^T (row = key) is transposed in registers by
// movmatrix; before that p is multiplied by a'_jg. That product is rounded to
// fp16 (11 bits), scaled by a power of two per group that follows the largest
// a' seen, so that p a' keeps full precision 2^-19 below it. Scores, statistics
// and accumulators are fp32; q is rounded to fp16 after scaling its row to
// 2^14 .. 2^15, which keeps all 8 bits of every bf16 element down to 2^-28 of
// the row's largest.
//
// Work: a unit is two pages of one (sequence, key/value head, row block); all
// units form one list, cut into equal ranges for the CTAs (long and short
// caches balance, one long cache uses every SM). A row block that lies in one
// CTA's range is finished there; others leave (max, sum, O) in the workspace
// for the finishing kernel. Within a CTA each of four warps takes 32 of a unit's
// 128 tokens, with softmax statistics and a ring of asynchronous copies of its
// own, so that nothing synchronises the warps until they add their rows up at the
// end of a row block.
#include <type_traits>

#include <cuda_fp16.h>

#include "kv4.h"
#include "paged_work.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kKv4Threads = 32 * kWarps;
constexpr float kKv4Tau = 8.f;                   // a row's max moves when it grows by more (log2 units)
constexpr int kWTargetLog = 5;                   // the largest a' of a group is scaled to [16, 32) = [2^4, 2^5)
constexpr float kWMost = 128.f;                  // ... and rescaled past this: p a' <= 2^8 * 2^7 in fp16

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the first step of a sum: no accumulator to clear
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ void lds64(uint32_t a, uint32_t& x, uint32_t& y) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(x), "=r"(y) : "r"(a));
}
// 16 bytes per lane from global to shared memory, past L1. (Bulk copies want
// their operands in uniform registers: eight of them per half page, with sources
// of their own, cost a loop of about 100 instructions.)
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ float lo_bf16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// 2^e for an unbiased exponent in the normal range
__device__ __forceinline__ float pow2(int e) {
    return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23);
}

template <int D, int DV, int NR>
struct Kv4Layout {
    static constexpr int kRows = 8 * NR, GK = D / kKv4Group, GV = DV / kKv4Group;
    // a slot: 32 tokens of a page and head, group by group: K codes, V codes, K and V parameters
    static constexpr int kCodes = 32 * 32, kParams = 32 * 4;   // of one group
    static constexpr int kVOff = GK * kCodes, kKpOff = kVOff + GV * kCodes, kVpOff = kKpOff + GK * kParams,
                         kSlot = kVpOff + GV * kParams;
    static constexpr int kSlots = D + DV <= 128 ? 4 : (D + DV <= 256 ? 3 : 2);   // per warp
    static constexpr int kQOff = kWarps * kSlots * kSlot;         // q fragments [NR][GK][2][32 lanes] x 16 bytes
    static constexpr int kQSumOff = kQOff + NR * GK * 1024;       // q's (sum, largest |q|) per row and group
    static constexpr int kKeysOff = kQSumOff + kRows * GK * 8;    // the keys [lo, hi) of each row's window
    static constexpr int kMlOff = kKeysOff + kRows * 8;           // (max, sum) per warp and row
    static constexpr int kPrefixOff = (kMlOff + kWarps * kRows * 8 + 15) / 16 * 16;
    // at the end of a row block each warp's O rows go where its slots were
    static_assert(kRows * DV * 4 <= kSlots * kSlot, "O rows of a warp");
    static constexpr int smem(int B) { return kPrefixOff + (2 * B + 1) * 4; }   // the work prefix, row blocks per sequence
    // accumulators take NR * DV / 4 registers of a thread
    static constexpr int kRegCtas = NR * DV <= 64 ? 4 : (NR * DV <= 256 && DV < 256 ? 3 : 2);
    static constexpr int kSmemCtas = 227 * 1024 / (smem(64) + 1024);   // (with up to 64 sequences)
    static constexpr int kCtas = kRegCtas < kSmemCtas ? kRegCtas : kSmemCtas;
    static_assert(kCtas >= 1 && smem(kKv4MaxBatch) <= 227 * 1024, "shared memory budget");
};

// kScores: key weights are wanted, the scores go to the workspace.
template <int D, int DV, int NR, bool kScores>
__global__ void __launch_bounds__(kKv4Threads, Kv4Layout<D, DV, NR>::kCtas) kv4_fwd_kernel(const Kv4FwdParams p) {
    using Lay = Kv4Layout<D, DV, NR>;
    constexpr int GK = Lay::GK, GV = Lay::GV, S = Lay::kSlots, kRows = Lay::kRows;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int* prefix = reinterpret_cast<int*>(smem + Lay::kPrefixOff);
    const uint32_t ring = base + warp * S * Lay::kSlot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (the finishing kernel waits for this grid's end)
    const Cut cut = build_prefix<kKv4Threads>(p, prefix, prefix + p.s.B + 1, kRows, gridDim.x);   // (ends with __syncthreads)
    const int per = cut.per;
    const int total = prefix[p.s.B];
    if (blockIdx.x == 0) {   // for the kernel that follows
        for (int i = tid; i <= p.s.B; i += kKv4Threads) p.prefix[i] = prefix[i];
        if (tid == 0) {
            p.prefix[kKv4MaxBatch + 1] = per;
            p.prefix[kKv4MaxBatch + 2] = cut.aligned;
        }
    }
    const int u0 = min(total, (int)blockIdx.x * per), u1 = min(total, u0 + per);

    const int g8 = lane >> 2, t4 = lane & 3;
    // This warp's 32 tokens of a unit (half warp % 2 of page warp / 2), in two chunks of 16. S^T
    // row r of a chunk is token t + 4 e + 8 h (r = 2 t + e + 8 h): then the V words of a lane (rows
    // 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of P^T) lie 4 tokens apart and a warp's 32-bit loads hit 32 banks.
    const int half = warp & 1, tok0 = (g8 >> 1) + 4 * (g8 & 1);   // keys tok0, + 8 (chunk 0), + 16, + 24
    float acc[GV * 4][NR][4];
    float qsum[NR][2][GK], qscale[NR][2], m_run[NR][2], mu[NR][2], l_run[NR][2], zb[NR][2][GV], wsc[GV];
    int2* row_keys = reinterpret_cast<int2*>(smem + Lay::kKeysOff);
    float2* qstat = reinterpret_cast<float2*>(smem + Lay::kQSumOff);
    float2* ml = reinterpret_cast<float2*>(smem + Lay::kMlOff);
    const long row_len = (long)p.s.width * kPage;
    for (int u = u0; u < u1;) {
        // ------------------------------------------------ a row block (this CTA's share of it): units i0 .. i1 - 1
        SeqWork w;
        const Unit t = unit_at(p, prefix, cut, u, kRows, &w);
        const int i0 = t.i, i1 = min(w.units, i0 + u1 - u);
        u += min(cut.span(w.units) - i0, u1 - u);   // (with its padding)
        // this warp's pages: index 2 i + warp / 2; lane l holds the id of the unit l % 16 of the current
        // sixteen, and of the next sixteen
        const int* table = p.s.table + (long)t.b * p.s.width;
        auto page_id = [&](int i) {
            const int x = 2 * i + (warp >> 1);
            if (i >= i1 || x >= w.pages) return -2;   // no such page
            const int id = table[page_of(w, x)];
            if (id >= 0 && id < p.c.n_pages) return id;
            atomicCAS(p.status, kStatusOk, kStatusBadPage);
            return -1;
        };
        int ids = 0, ids_next = page_id(i0 + (lane & 15));
        uint32_t live = 0;   // bit (i - i0) % 32: unit i's page is in range
        // A lane's 16-byte pieces of a slot: piece `lane` and `lane` + 32 of every group's codes, and
        // of the 8 (GK + GV) pieces of parameters number `lane`.
        constexpr uint32_t kGroupCodes = kPage * 32, kGroupParams = kPage * 4;   // of a page
        const uint32_t kc_page = (uint32_t)p.c.Hkv * GK * kGroupCodes, vc_page = (uint32_t)p.c.Hkv * GV * kGroupCodes;
        const uint8_t* kc = p.c.k_codes + (size_t)t.h * GK * kGroupCodes + half * Lay::kCodes + lane * 16;
        const uint8_t* vc = p.c.v_codes + (size_t)t.h * GV * kGroupCodes + half * Lay::kCodes + lane * 16;
        const bool par = lane < 8 * (GK + GV), par_v = lane >= 8 * GK;
        const int par_g = lane / 8 - (par_v ? GK : 0);
        const uint32_t par_page = (uint32_t)p.c.Hkv * (par_v ? GV : GK) * kGroupParams;
        const uint8_t* par_src = reinterpret_cast<const uint8_t*>(par_v ? p.c.v_params : p.c.k_params) +
                                 (size_t)(t.h * (par_v ? GV : GK) + par_g) * kGroupParams + half * Lay::kParams + (lane & 7) * 16;
        const uint32_t code_dst = ring + lane * 16, par_dst = ring + Lay::kKpOff + lane * 16;   // (V's parameters follow K's)
        uint32_t slot_in = 0, slot_out = 0;   // slots written to and read from next, as byte offsets
        auto issue = [&](int i) {   // the loads of unit i into the next slot (i - i0 = 0, 1, 2, ...), one group of copies
            const int n = i - i0;
            if (i < i1) {
                if ((n & 15) == 0) {
                    ids = ids_next;
                    ids_next = page_id(i + 16 + (lane & 15));
                    const uint32_t in = __ballot_sync(kFullMask, ids >= 0) & 0xffffu;
                    live = (live & (0xffff0000u >> (n & 16))) | in << (n & 16);
                }
                const int id = __shfl_sync(kFullMask, ids, n & 15);
                if (id >= 0) {
                    const uint8_t *k = kc + (size_t)id * kc_page, *v = vc + (size_t)id * vc_page;
#pragma unroll
                    for (int x = 0; x < 2 * GK; ++x)
                        copy16(code_dst + slot_in + x * 512, k + (x >> 1) * kGroupCodes + (x & 1) * 512);
#pragma unroll
                    for (int x = 0; x < 2 * GV; ++x)
                        copy16(code_dst + slot_in + Lay::kVOff + x * 512, v + (x >> 1) * kGroupCodes + (x & 1) * 512);
                    if (par) copy16(par_dst + slot_in, par_src + (size_t)id * par_page);
                    if constexpr (GK + GV > 4) {   // the parameters past the first 32 pieces
                        constexpr int kRest = 8 * (GK + GV) - 32;   // all of V's last groups
                        if (lane < kRest) {
                            const int g = GV - kRest / 8 + lane / 8;
                            copy16(par_dst + slot_in + 512, reinterpret_cast<const uint8_t*>(p.c.v_params) +
                                                                ((size_t)id * p.c.Hkv + t.h) * GV * kGroupParams + g * kGroupParams +
                                                                half * Lay::kParams + (lane & 7) * 16);
                        }
                    }
                }
                slot_in = slot_in == (S - 1) * Lay::kSlot ? 0 : slot_in + Lay::kSlot;
            }
            copy_commit();
        };
#pragma unroll
        for (int x = 0; x < S - 1; ++x) issue(i0 + x);
        // ------------------------------------------------ its queries
        const MaskBand mb = mask_band(w.s.nq, w.s.lk, p.win_left, p.win_right, p.sinks);
        if (tid < kRows) {
            const int row = t.rb * kRows + tid, i = row / p.group;
            row_keys[tid] = row < w.rows ? make_int2(band_key_lo(mb, i), band_key_hi(mb, i)) : make_int2(0, 0);
        }
        {
            // (n, g) = 8 rows x 64 channels each, dealt to the warps; a lane takes row g8's channels 16 t4 ..
            constexpr int kTasks = (NR * GK + kWarps - 1) / kWarps;
            uint4 raw[kTasks][2];
#pragma unroll
            for (int y = 0; y < kTasks; ++y) {
                const int task = y * kWarps + warp, n = task / GK, g = task % GK;
                const int r = t.rb * kRows + n * 8 + g8;
                raw[y][0] = raw[y][1] = make_uint4(0, 0, 0, 0);
                if (task < NR * GK && r < w.rows) {
                    const uint4* src = reinterpret_cast<const uint4*>(p.q + (long)(w.s.q0 + r / p.group) * p.q_stride +
                                                                      (long)(t.h * p.group + r % p.group) * D + g * kKv4Group + 16 * t4);
                    raw[y][0] = src[0];
                    raw[y][1] = src[1];
                }
            }
#pragma unroll
            for (int y = 0; y < kTasks; ++y) {
                const int task = y * kWarps + warp, n = task / GK, g = task % GK;
                const uint32_t ws[8] = {raw[y][0].x, raw[y][0].y, raw[y][0].z, raw[y][0].w,
                                        raw[y][1].x, raw[y][1].y, raw[y][1].z, raw[y][1].w};
                float part = 0.f, top = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float a = lo_bf16(ws[i]), b = hi_bf16(ws[i]);
                    top = fmaxf(top, fmaxf(fabsf(a), fabsf(b)));
                    part += a;
                    part += b;
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    part += __shfl_xor_sync(kFullMask, part, o);
                    top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
                }
                if (t4 == 0 && task < NR * GK) qstat[(n * 8 + g8) * GK + g] = make_float2(part, top);
            }
            __syncthreads();
            // row r times 2^e has its largest element in [2^14, 2^15) (both powers stay in the float range;
            // a row of its own exponent, so that whatever an unused row of a padded batch holds stays there)
            auto row_exponent = [&](int r) {
                float top = 0.f;
#pragma unroll
                for (int g = 0; g < GK; ++g) top = fmaxf(top, qstat[r * GK + g].y);
                return top > 0.f && top < INFINITY ? min(max(14 - ((int)(__float_as_uint(top) >> 23) - 127), -100), 126) : 0;
            };
#pragma unroll
            for (int y = 0; y < kTasks; ++y) {
                const int task = y * kWarps + warp;
                if (task >= NR * GK) break;
                const float f = pow2(row_exponent(task / GK * 8 + g8)), f16 = f * 0.0625f;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    // word x holds channels 8 x .. 8 x + 7; step 2 x takes (0, 4) and (1, 5), step 2 x + 1 (2, 6) and (3, 7);
                    // odd nibbles read 16 times too large
                    const uint4 v = raw[y][x];
                    *reinterpret_cast<uint4*>(smem + Lay::kQOff + ((task * 2 + x) * 32 + lane) * 16) =
                        make_uint4(pack_f16x2(lo_bf16(v.x) * f, lo_bf16(v.z) * f), pack_f16x2(hi_bf16(v.x) * f16, hi_bf16(v.z) * f16),
                                   pack_f16x2(lo_bf16(v.y) * f, lo_bf16(v.w) * f), pack_f16x2(hi_bf16(v.y) * f16, hi_bf16(v.w) * f16));
                }
            }
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int g = 0; g < GK; ++g) qsum[n][c][g] = p.scale_log2 * qstat[(n * 8 + 2 * t4 + c) * GK + g].x;
                    qscale[n][c] = p.scale_log2 * pow2(24 - row_exponent(n * 8 + 2 * t4 + c));
                    m_run[n][c] = -INFINITY;
                    mu[n][c] = l_run[n][c] = 0.f;
#pragma unroll
                    for (int g = 0; g < GV; ++g) zb[n][c][g] = 0.f;
                }
        }
        // keys that the block's first and last rows (hence all) see
        const int full_lo = band_key_lo(mb, (min(w.rows, t.rb * kRows + kRows) - 1) / p.group);
        const int full_hi = band_key_hi(mb, t.rb * kRows / p.group);
        float* score_at = nullptr;   // the scores of row 2 t4, token tok0 of a half page
        uint32_t rows_in = 0;        // bit 2 n + c: row 8 n + 2 t4 + c exists
        if constexpr (kScores) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
                for (int c = 0; c < 2; ++c) rows_in |= (t.rb * kRows + n * 8 + 2 * t4 + c < w.rows ? 1u : 0u) << (2 * n + c);
            score_at = p.scores + ((long)t.h * p.s.total * p.group + (long)w.s.q0 * p.group + t.rb * kRows + 2 * t4) * row_len + tok0;
        }
#pragma unroll
        for (int g = 0; g < GV; ++g) wsc[g] = INFINITY;
#pragma unroll
        for (int j = 0; j < GV * 4; ++j)
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) acc[j][n][x] = 0.f;
        __syncthreads();   // the q fragments are in place
        const uint32_t qfrag = base + Lay::kQOff + lane * 16;

        // One half page of 32 keys from slot `st`, its first key key0. kWhole: every row sees all of
        // them (the common case, kept free of masks and branches).
        bool force = true;   // some row has yet to see its first key
        auto half_page = [&](auto whole_tag, const uint32_t st, const int key0) {
            constexpr bool kWhole = decltype(whole_tag)::value;
            float sc[2][NR][4];   // s - mu: per chunk [key g8, g8 + 8][row 2 t4, 2 t4 + 1] at 2 * key + row
#pragma unroll
            for (int g = 0; g < GK; ++g) {
                uint4 qf[NR][2];
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) qf[n][x] = lds128(qfrag + ((n * GK + g) * 2 + x) * 512);
#pragma unroll
                for (int ck = 0; ck < 2; ++ck) {
                    const uint32_t row = st + g * Lay::kCodes + (tok0 + 16 * ck) * 32 + 8 * t4;
                    uint32_t wa[2], wb[2];
                    lds64(row, wa[0], wa[1]);
                    lds64(row + 8 * 32, wb[0], wb[1]);
                    const uint32_t par = st + Lay::kKpOff + g * Lay::kParams + (tok0 + 16 * ck) * 4;
                    const uint32_t pa = lds32(par), pb = lds32(par + 32);
                    float d[NR][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t xa = (k & 1) ? wa[k >> 1] >> 8 : wa[k >> 1], xb = (k & 1) ? wb[k >> 1] >> 8 : wb[k >> 1];
                        const uint32_t a0 = xa & 0x000f000fu, a1 = xb & 0x000f000fu, a2 = xa & 0x00f000f0u, a3 = xb & 0x00f000f0u;
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
                            const uint4 q4 = qf[n][k >> 1];
                            if (k == 0) mma_f16_first(d[n], a0, a1, a2, a3, q4.x, q4.y);
                            else mma_f16(d[n], a0, a1, a2, a3, (k & 1) ? q4.z : q4.x, (k & 1) ? q4.w : q4.y);
                        }
                    }
                    const float aa = lo_bf16(pa), ba = hi_bf16(pa), ab = lo_bf16(pb), bb = hi_bf16(pb);
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            sc[ck][n][c] = fmaf(d[n][c] * qscale[n][c], aa, fmaf(qsum[n][c][g], ba, g ? sc[ck][n][c] : -mu[n][c]));
                            sc[ck][n][2 + c] = fmaf(d[n][2 + c] * qscale[n][c], ab, fmaf(qsum[n][c][g], bb, g ? sc[ck][n][2 + c] : -mu[n][c]));
                        }
                }
            }
            if constexpr (!kWhole) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int2 k = row_keys[n * 8 + 2 * t4 + c];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int j = key0 + tok0 + 8 * x;
                            if (!(j < k.y && (j >= k.x || j < p.sinks))) sc[x >> 1][n][2 * (x & 1) + c] = -INFINITY;
                        }
                    }
            }
            if constexpr (kScores) {
                float* dst = score_at + key0;
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if ((rows_in >> (2 * n + c)) & 1u) {
#pragma unroll
                            for (int ck = 0; ck < 2; ++ck) {
                                dst[16 * ck] = sc[ck][n][c] + mu[n][c];
                                dst[16 * ck + 8] = sc[ck][n][2 + c] + mu[n][c];
                            }
                        }
                        dst += c ? 7 * row_len : row_len;
                    }
            }
            // ---------------------------------------- V's parameters; does a maximum or a scale have to move?
            uint32_t vp[2][GV][2];
            bool move = force;
#pragma unroll
            for (int g = 0; g < GV; ++g) {
#pragma unroll
                for (int ck = 0; ck < 2; ++ck)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        vp[ck][g][x] = lds32(st + Lay::kVpOff + g * Lay::kParams + (tok0 + 16 * ck + 8 * x) * 4);
                        if constexpr (!kWhole) {   // a key that none of this lane's rows sees: its parameters may hold anything
                            bool seen = false;
#pragma unroll
                            for (int n = 0; n < NR; ++n) seen |= sc[ck][n][2 * x] != -INFINITY || sc[ck][n][2 * x + 1] != -INFINITY;
                            if (!seen) vp[ck][g][x] = 0u;
                        }
                    }
                const float top = max3(fmaxf(fabsf(lo_bf16(vp[0][g][0])), fabsf(lo_bf16(vp[0][g][1]))),
                                       fabsf(lo_bf16(vp[1][g][0])), fabsf(lo_bf16(vp[1][g][1])));
                move |= !(top * wsc[g] <= kWMost);
            }
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    move |= max3(fmaxf(sc[0][n][c], sc[0][n][2 + c]), sc[1][n][c], sc[1][n][2 + c]) > kKv4Tau;
                }
            if (__any_sync(kFullMask, move)) {
                bool unset = false;
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    float al[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = fmaxf(fmaxf(sc[0][n][c], sc[0][n][2 + c]), fmaxf(sc[1][n][c], sc[1][n][2 + c]));
                        mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 16));
                        const float m_new = fmaxf(m_run[n][c], mx + mu[n][c]);
                        al[c] = m_new == -INFINITY ? 1.f : ex2_mufu(m_run[n][c] - m_new);
                        const float mu_new = m_new == -INFINITY ? 0.f : m_new;
#pragma unroll
                        for (int ck = 0; ck < 2; ++ck) {
                            sc[ck][n][c] += mu[n][c] - mu_new;
                            sc[ck][n][2 + c] += mu[n][c] - mu_new;
                        }
                        unset |= m_new == -INFINITY && row_keys[n * 8 + 2 * t4 + c].y > 0;
                        m_run[n][c] = m_new;
                        mu[n][c] = mu_new;
                        l_run[n][c] *= al[c];
#pragma unroll
                        for (int g = 0; g < GV; ++g) zb[n][c][g] *= al[c];
                    }
#pragma unroll
                    for (int j = 0; j < GV * 4; ++j)
#pragma unroll
                        for (int x = 0; x < 4; ++x) acc[j][n][x] *= al[x & 1];
                }
                force = __any_sync(kFullMask, unset);
#pragma unroll
                for (int g = 0; g < GV; ++g) {
                    // a new power of two for the group's a'; infinities and NaN do not set it
                    float top = 0.f;
#pragma unroll
                    for (int ck = 0; ck < 2; ++ck)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float v = fabsf(lo_bf16(vp[ck][g][x]));
                            top = fmaxf(top, v < INFINITY ? v : 0.f);
                        }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
                    if (!(top * wsc[g] <= kWMost) && top > 0.f) {
                        // (at most 2^127, as infinity means none yet: of scales below 2^-123 p a' is then off by up
                        // to 2^-152, an eighth of the smallest fp32)
                        const float now = pow2(kWTargetLog + 126 - (int)(__float_as_uint(top) >> 23));
                        const float r = wsc[g] == INFINITY ? 1.f : now / wsc[g];
                        wsc[g] = now;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int n = 0; n < NR; ++n)
#pragma unroll
                                for (int x = 0; x < 4; ++x) acc[4 * g + j][n][x] *= r;
                    }
                }
            }
#pragma unroll
            for (int ck = 0; ck < 2; ++ck)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        sc[ck][n][x] = ex2_mufu(sc[ck][n][x]);
                        l_run[n][x & 1] += sc[ck][n][x];
                    }
            // ---------------------------------------- values
#pragma unroll
            for (int g = 0; g < GV; ++g) {
                const float ws = wsc[g] == INFINITY ? 1.f : wsc[g];
#pragma unroll
                for (int ck = 0; ck < 2; ++ck) {
                    const float fa = lo_bf16(vp[ck][g][0]) * ws, fb = lo_bf16(vp[ck][g][1]) * ws;
                    const float ba = hi_bf16(vp[ck][g][0]), bb = hi_bf16(vp[ck][g][1]);
                    uint32_t b0[NR], b1[NR];
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        const float* s4 = sc[ck][n];
                        float x[4] = {s4[0] * fa, s4[1] * fa, s4[2] * fb, s4[3] * fb};
                        if constexpr (kWhole) {
                            zb[n][0][g] = fmaf(s4[0], ba, fmaf(s4[2], bb, zb[n][0][g]));
                            zb[n][1][g] = fmaf(s4[1], ba, fmaf(s4[3], bb, zb[n][1][g]));
                        } else {   // p = 0 times an infinity or a NaN of a masked key stays 0
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const bool zero = s4[y] == 0.f;
                                x[y] = zero ? 0.f : x[y];
                                zb[n][y & 1][g] += zero ? 0.f : s4[y] * (y < 2 ? ba : bb);
                            }
                        }
                        b0[n] = transpose8x8(pack_f16x2(x[0], x[1]));
                        b1[n] = transpose8x8(pack_f16x2(x[2], x[3]));
                    }
                    const uint32_t row = st + Lay::kVOff + g * Lay::kCodes + (16 * ck + t4) * 32 + 4 * g8;
                    const uint32_t w0 = lds32(row), w1 = lds32(row + 4 * 32), w2 = lds32(row + 8 * 32), w3 = lds32(row + 12 * 32);
                    // channels 8 g8 + 2 j (accumulator rows g8) and + 1 (rows g8 + 8, 16 times too large) of the group
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t sel = j < 2 ? 0x5410u : 0x7632u;
                        uint32_t xa = __byte_perm(w0, w1, sel), xb = __byte_perm(w2, w3, sel);
                        if (j & 1) {
                            xa >>= 8;
                            xb >>= 8;
                        }
                        const uint32_t a0 = xa & 0x000f000fu, a1 = xa & 0x00f000f0u, a2 = xb & 0x000f000fu, a3 = xb & 0x00f000f0u;
#pragma unroll
                        for (int n = 0; n < NR; ++n) mma_f16(acc[4 * g + j][n], a0, a1, a2, a3, b0[n], b1[n]);
                    }
                }
            }
        };

        for (int i = i0; i < i1; ++i) {
            // -------------------------------------------- this warp's half page of unit i
            copy_wait<S - 2>();
            __syncwarp();   // the slot is full, and every lane has read the one before
            issue(i + S - 1);
            const bool valid = (live >> ((i - i0) & 31)) & 1u;
            const uint32_t st = ring + slot_out;
            slot_out = slot_out == (S - 1) * Lay::kSlot ? 0 : slot_out + Lay::kSlot;
            const int key0 = page_of(w, 2 * i + (warp >> 1)) * kPage + 32 * half;
            if (valid) {
                if (key0 >= full_lo && key0 + 32 <= full_hi) half_page(std::true_type{}, st, key0);
                else half_page(std::false_type{}, st, key0);
            } else if (kScores && 2 * i + (warp >> 1) < w.pages) {   // no key of a page that is out of range counts
                float* dst = score_at + key0;
                for (int n = 0; n < 2 * NR; ++n) {
                    if ((rows_in >> n) & 1u)
                        for (int x = 0; x < 4; ++x) dst[8 * x] = -INFINITY;
                    dst += n & 1 ? 7 * row_len : row_len;
                }
            }
        }
        // ------------------------------------------------ the four warps' rows become one
        // (every copy into the slots has landed and been read: each warp's O rows go there)
        const bool ends = i1 == w.units, starts = i0 == 0;
        __syncwarp();
        float* mine = reinterpret_cast<float*>(smem + warp * S * Lay::kSlot);
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = l_run[n][c];
                l += __shfl_xor_sync(kFullMask, l, 4);
                l += __shfl_xor_sync(kFullMask, l, 8);
                l += __shfl_xor_sync(kFullMask, l, 16);
                const int row = n * 8 + 2 * t4 + c;
                if (g8 == 0) ml[warp * kRows + row] = make_float2(m_run[n][c], l);
#pragma unroll
                for (int g = 0; g < GV; ++g) {
                    float z = zb[n][c][g];
                    z += __shfl_xor_sync(kFullMask, z, 4);
                    z += __shfl_xor_sync(kFullMask, z, 8);
                    z += __shfl_xor_sync(kFullMask, z, 16);
                    const float inv = wsc[g] == INFINITY ? 1.f : 1.f / wsc[g];   // (a power of two)
                    float4* at = reinterpret_cast<float4*>(mine + row * DV + g * kKv4Group + 8 * g8);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        at[j] = make_float4(fmaf(acc[4 * g + 2 * j][n][c] * 16777216.f, inv, z),   // (inv may be up to 2^123)
                                            fmaf(acc[4 * g + 2 * j][n][2 + c] * 1048576.f, inv, z),
                                            fmaf(acc[4 * g + 2 * j + 1][n][c] * 16777216.f, inv, z),
                                            fmaf(acc[4 * g + 2 * j + 1][n][2 + c] * 1048576.f, inv, z));
                }
            }
        __syncthreads();
        const int part = 2 * blockIdx.x + (starts ? 1 : 0);
        const int n_rows = min(kRows, w.rows - t.rb * kRows);
        for (int x = tid; x < n_rows * (DV / 4); x += kKv4Threads) {
            const int row = x / (DV / 4), c4 = x % (DV / 4);
            float2 v[kWarps];
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int y = 0; y < kWarps; ++y) {
                v[y] = ml[y * kRows + row];
                m = fmaxf(m, v[y].x);
            }
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int y = 0; y < kWarps; ++y) {   // in warp order: the same sum on every run
                const float f = v[y].x == -INFINITY ? 0.f : ex2_mufu(v[y].x - m);
                l += v[y].y * f;
                if (f != 0.f) {
                    const float4 z = *reinterpret_cast<const float4*>(smem + y * S * Lay::kSlot + (row * DV + 4 * c4) * 4);
                    o.x = fmaf(f, z.x, o.x);
                    o.y = fmaf(f, z.y, o.y);
                    o.z = fmaf(f, z.z, o.z);
                    o.w = fmaf(f, z.w, o.w);
                }
            }
            if (starts && ends) {
                const int r = t.rb * kRows + row, i = r / p.group, head = t.h * p.group + r % p.group;
                const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // (NaN stays)
                const long tok = w.s.q0 + i;
                *reinterpret_cast<uint2*>(p.o + (tok * p.H + head) * DV + 4 * c4) =
                    make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
                if (c4 == 0) {
                    float* dst = p.s.cu ? p.lse + (long)head * p.s.total + tok : p.lse + ((long)t.b * p.H + head) * p.s.rows + i;
                    *dst = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                }
            } else {
                *reinterpret_cast<float4*>(p.part_o + ((long)part * kRows + row) * DV + 4 * c4) = o;
                if (c4 == 0) *reinterpret_cast<float2*>(p.part_ml + ((long)part * kRows + row) * 2) = make_float2(m, l);
            }
        }
        __syncthreads();   // the next row block's copies come after these reads
    }
}

// ---------------------------------------------------------------- finish
constexpr int kFinishThreads = 128;
constexpr int kFinishKeys = 4 * kFinishThreads;   // keys of a tile
constexpr int kFinishRows = 64;                   // rows whose LSE it holds at a time

// Blocks [0, row_blocks): one warp per (token, head) whose row block several CTAs
// shared joins their partial rows in CTA order (the same sum on every run); rows
// that no key reaches get O = 0, LSE = -inf. The other blocks update key weights:
//   key_weights[b][h][j] = decay * key_weights + sum over rows of exp(s - LSE),
// four keys per thread and tile, rows in order: four tiles of one row at a time, or,
// when that makes too few blocks for the SMs, one tile of four rows; a block's rows
// get their LSE all at once, several lanes each (4 caches of up to 2253 keys, 8 heads
// of 88 rows, d = 128, the wait for the attention kernel's 25 us included: 38 us, 95
// with four tiles and a warp per row). Scores of pages that no row block visited
// were not written and count as nothing. Launched while the attention kernel
// runs (programmatic dependent launch); what it left is read after the wait.
template <int kTiles>
__global__ void __launch_bounds__(kFinishThreads, 7) kv4_finish_kernel(const Kv4FwdParams p, int rows_per_block,
                                                                    int row_blocks, int key_blocks) {
    __shared__ float lse2[kFinishRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if ((int)blockIdx.x < row_blocks) {
        finish_row(p, (long)blockIdx.x * (kFinishThreads / 32) + warp, rows_per_block);
        return;
    }
    const int id = blockIdx.x - row_blocks;
    const int bh = id / key_blocks, b = bh / p.c.Hkv, h = bh % p.c.Hkv;
    const SeqWork w = seq_work(p, b, rows_per_block);
    const int j0 = (id % key_blocks) * kTiles * kFinishKeys + 4 * threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (j0 == 0 && w.s.lk > p.weight_stride) atomicCAS(p.status, kStatusOk, kStatusBadPage);
    const int keys = (int)min((long)w.s.lk, p.weight_stride);
    if (w.s.bad || (id % key_blocks) * kTiles * kFinishKeys >= keys) return;
    if (w.units > 0 && w.rows > 0 && p.prefix[kKv4MaxBatch + 1] == 0) return;   // (a list that did not fit)
    bool seen[kTiles];
    float sum[kTiles][4] = {};
#pragma unroll
    for (int x = 0; x < kTiles; ++x) {
        const int j = j0 + x * kFinishKeys, page = j / kPage;
        seen[x] = j < keys && (page < w.n_sink || (page >= w.first && page < w.first + w.pages - w.n_sink));
    }
    const long row_len = (long)p.s.width * kPage;
    const float* src = p.scores + ((long)h * p.s.total * p.group + (long)w.s.q0 * p.group) * row_len + j0;
    for (int r0 = 0; r0 < w.rows && w.pages > 0; r0 += kFinishRows) {
        const int nr = min(kFinishRows, w.rows - r0);
        int lanes = 32;   // of a row
        while (lanes > 1 && kFinishThreads / lanes < nr) lanes >>= 1;
        __syncthreads();
        {
            const int r = min((int)threadIdx.x / lanes, nr - 1);   // (at most 64 rows: two lanes or more)
            const Shares s = shares_of(p, w, b, h, r0 + r, rows_per_block);
            const float2 ml = join_ml(p, Shares{s.c0, s.c0 == s.c1 ? s.c0 - 1 : s.c1, s.in_block, s.rows_per_block},
                                      lane & (lanes - 1), lanes);
            const float v = s.c0 == s.c1 ? p.lse[lse_at(p, w, b, (r0 + r) / p.group, h * p.group + (r0 + r) % p.group)] * kLog2e
                                         : (ml.y == 0.f ? -INFINITY : ml.x + log2f(ml.y));
            if ((lane & (lanes - 1)) == 0) lse2[r] = v;
        }
        __syncthreads();
        constexpr int kAhead = 4 / kTiles;
        for (int r = 0; r < nr; r += kAhead) {
            float4 s[kAhead][kTiles];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
#pragma unroll
                for (int x = 0; x < kTiles; ++x)
                    if (seen[x] && (kAhead == 1 || r + k < nr))
                        s[k][x] = __ldcs(reinterpret_cast<const float4*>(src + (r0 + r + k) * row_len + x * kFinishKeys));
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (kAhead > 1 && r + k >= nr) break;
                const float e = lse2[r + k];
#pragma unroll
                for (int x = 0; x < kTiles; ++x) {
                    if (!seen[x]) continue;
                    const float4 y = s[k][x];
                    sum[x][0] += y.x == -INFINITY ? 0.f : ex2_mufu(y.x - e);
                    sum[x][1] += y.y == -INFINITY ? 0.f : ex2_mufu(y.y - e);
                    sum[x][2] += y.z == -INFINITY ? 0.f : ex2_mufu(y.z - e);
                    sum[x][3] += y.w == -INFINITY ? 0.f : ex2_mufu(y.w - e);
                }
            }
        }
    }
    float* dst = p.key_weights + ((long)b * p.c.Hkv + h) * p.weight_stride + j0;
#pragma unroll
    for (int x = 0; x < kTiles; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int k = x * kFinishKeys + y;
            if (j0 + k < keys) dst[k] = p.weight_decay == 0.f ? sum[x][y] : fmaf(p.weight_decay, dst[k], sum[x][y]);
        }
}

template <int D, int DV, int NR>
cudaError_t launch_one(const Kv4FwdParams& p, int num_sms, cudaStream_t stream) {
    using Lay = Kv4Layout<D, DV, NR>;
    static std::atomic<unsigned long long> allowed[2];
    const bool scores = p.key_weights != nullptr;
    auto kern = scores ? kv4_fwd_kernel<D, DV, NR, true> : kv4_fwd_kernel<D, DV, NR, false>;
    const int smem = Lay::smem(p.s.B);
    cudaError_t e = allow_smem(kern, Lay::smem(kKv4MaxBatch), allowed[scores]);
    if (e != cudaSuccess) return e;
    int grid = num_sms * Lay::kCtas;
    if (grid > kKv4MaxCtas) grid = kKv4MaxCtas;
    kern<<<grid, kKv4Threads, smem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int row_blocks = (int)(((long)p.s.total * p.H + kFinishThreads / 32 - 1) / (kFinishThreads / 32));
    const long key_tiles = p.key_weights ? ((long)p.s.width * kPage + kFinishKeys - 1) / kFinishKeys : 0;
    const int tiles = (key_tiles + 3) / 4 * p.c.Hkv * p.s.B >= 7 * num_sms ? 4 : 1;
    const int key_blocks = (int)((key_tiles + tiles - 1) / tiles);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(row_blocks + (long)key_blocks * p.c.Hkv * p.s.B));
    cfg.blockDim = dim3(kFinishThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tiles == 4 ? kv4_finish_kernel<4> : kv4_finish_kernel<1>, p, Lay::kRows, row_blocks, key_blocks);
}

template <int D, int DV>
cudaError_t launch_dims(const Kv4FwdParams& p, int num_sms, cudaStream_t stream) {
    return kv4_row_tiles(p.group, p.s.B, p.s.total) == 1 ? launch_one<D, DV, 1>(p, num_sms, stream)
                                                         : launch_one<D, DV, 2>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_kv4_fwd(const Kv4FwdParams& p, int num_sms, cudaStream_t stream) {
    const int d = p.c.d, dv = p.c.dv;
    if (d == 64 && dv == 64) return launch_dims<64, 64>(p, num_sms, stream);
    if (d == 128 && dv == 128) return launch_dims<128, 128>(p, num_sms, stream);
    if (d == 192 && dv == 192) return launch_dims<192, 192>(p, num_sms, stream);
    if (d == 192 && dv == 128) return launch_dims<192, 128>(p, num_sms, stream);
    if (d == 256 && dv == 256) return launch_dims<256, 256>(p, num_sms, stream);
    return cudaErrorInvalidValue;
}

}  // namespace attn
