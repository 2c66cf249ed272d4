// Attention of a few new tokens per sequence over the paged cache in bf16 or 8 bits.
//
// Mathematics. s_ij = scale <q_i, k_j>, O_i = sum_j p_ij v_j with p = exp(s - LSE), in one
// pass over the keys: a running maximum (moved when a row's grows by more than
// 2^kPagedTau) and sum per row, in fp32, as are all accumulators. With 8 bits k_j = 2^e c_j
// with codes c_j: the power enters the score in fp32, and that of v_j the bf16 operands of the
// product, v up to 2^7 and p beyond it, whose rounding it does not change. (All of it in p, whose
// weights are 2^-16 and less, would take scales below 2^-102 out of bf16's normal numbers.)
//
// What bounds it: the cache is read once. As in the 4-bit kernel, keys (channels for PV)
// take the M side of mma.sync m16n8k16 and the query rows the N side,
//   S^T[key, row] = K[key, ch] q^T[ch, row],   O^T[ch, row] += V^T[ch, key] P^T[key, row],
// which pads a handful of rows to 8 (a tcgen05 tile: to 64 or 128 on its M side, and on
// its N side it would write S to tensor memory and read it back for every 128 keys).
// bf16 operands come by ldmatrix. K's codes are converted to f16, two at a time and exactly, NaN
// included, and q too, by a power of two of each row's own: 8 bits keep all of themselves
// down to 2^-31 of the row's largest, and what is lost below is under 2^-39 of it.
// V's go to bf16, as p needs its exponents: a byte seeeemmm in the upper half of a 16-bit
// lane, its exponent and mantissa moved down by four, is the bf16 c 2^-120, subnormal codes
// included (the bf16 is subnormal too): a shift and two logic operations per pair, then
// one multiplication by the tokens' scales times 2^120. The codes 7f and ff, which
// are NaN and would count as 480 so, are looked for in every word of V, two operations for four
// codes; a step that has some makes the channels they stand in NaN for the rows that see
// their keys. (64 caches of 4096 to 16384, H32/8, d = 128: K by shifts as well and nothing
// looked for 222 us, with both looked for 251, as it is 218.)
//
// Work: paged_work.cuh. Each of four warps loads 32 of a unit's 128 tokens in steps of
// kTok, through a ring of asynchronous copies of its own. A block of up to 8 NR rows is every warp's,
// for its own tokens, with statistics of its own; in a larger one (16 to 32 rows) the two warps of a page
// take half of the rows each, for the tokens of both, so that the cache is read once for twice the rows.
#include <type_traits>

#include "paged.h"
#include "paged_work.cuh"

namespace attn {
namespace {

constexpr int kWarps = 4, kPagedThreads = 32 * kWarps;
constexpr float kPagedTau = 8.f;   // a row's max moves when it grows by more (log2 units)
// p is held 2^16 times smaller than exp(s - max), so that sums of p v stay finite for any N
// keys with N max|v| below 2^136; at the other end a sum holds its fp32's 2^-149, which is 2^-133 of O.
constexpr float kPagedShift = 16.f;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint16_t r;
    asm volatile("ld.shared.u8 %0, [%1];" : "=h"(r) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ uint4 ldsm4(uint32_t a) {
    uint4 r;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ uint4 ldsm4t(uint32_t a) {
    uint4 r;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
    return r;
}
// 16 bytes to shared memory past L1, the first `bytes` of them from memory, zeros behind
__device__ __forceinline__ void copy16n(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23); }
// codes in the upper bytes of both halves: the bf16 pair c 2^-120 (NaN: 480 2^-120)
__device__ __forceinline__ uint32_t codes_bf16(uint32_t x) { return (x & 0x80008000u) | ((x >> 4) & 0x07f007f0u); }
// Bits 80808080 of the words' `or` tell whether a code is NaN: adding one to a byte changes its eighth bit if the seven below
// are set. (Only whether there are any: the carry out of an ff reaches the bytes above it.)
__device__ __forceinline__ uint32_t changed(uint32_t codes) { return codes ^ (codes + 0x01010101u); }
// Exactly: 80 in each byte whose code is NaN, 0 in the others
__device__ __forceinline__ uint32_t nan_codes(uint32_t codes) { return ((codes & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t codes_f16(uint16_t x) {   // two codes, exactly; NaN stays
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t y) {   // bf16 pairs
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
// V's scale is split: 2^(min(e, kInV) - 127) goes to v, the rest to p, which is 1 for rows of values below 448 2^7
constexpr uint32_t kInV = 134;
__device__ __forceinline__ float scale_of_p(uint32_t e) { return e == 255 ? NAN : fmaxf(__uint_as_float(e << 23) * 0x1p-7f, 1.f); }
// Byte t of a and of b, in the halves of a word; such a pair's scales of v times 2^120, in bf16; bits 01000100: past kInV
__device__ __forceinline__ uint32_t byte_pair(uint32_t a, uint32_t b, int t) { return __byte_perm(a, b, (4 + t) << 8 | t) & 0x00ff00ffu; }
__device__ __forceinline__ uint32_t scales_of_v(uint32_t e) { return __vminu2(e, kInV * 0x10001u) * 128u + 120u * 128u * 0x10001u; }
__device__ __forceinline__ uint32_t past_v(uint32_t e) { return e + (255u - kInV) * 0x10001u; }

// Rows of `bytes` in shared memory, kTok tokens: panels of 128 bytes a row (and one of 64
// behind them where they do not divide), their 16-byte pieces permuted by the token so
// that neither eight tokens of one piece (ldmatrix) nor a warp's reads of codes (tokens t and
// t + 4 together in QK; tokens t, two pieces each, in PV) meet in a bank.
template <int kBytes, int kTok>
__device__ __forceinline__ uint32_t row_piece(uint32_t base, int tok, int piece) {
    constexpr int kFull = kBytes / 128;
    if (kBytes % 128 == 0 || piece < 8 * kFull) {
        const int sw = ((tok & 3) << 1) ^ ((tok & 4) ? 5 : 0);
        return base + (piece >> 3) * (kTok * 128) + tok * 128 + (((piece & 7) ^ sw) << 4);
    }
    const int slot = ((tok >> 2) & 1) * 4 + (piece & 3), line = (tok & 3) + 4 * (tok >> 3);
    return base + kFull * (kTok * 128) + line * 128 + ((slot ^ ((tok & 3) << 1)) << 4);
}

template <bool kCodes, int D, int DV, int NR>
struct PagedLayout {
    static constexpr int kGroups = NR == 1 ? 1 : 2, kWarpRows = 8 * NR, kRows = kWarpRows * kGroups, kElt = kCodes ? 1 : 2;
    static constexpr int kKRow = D * kElt, kVRow = DV * kElt;
    // a slot: kTok tokens, about 8 KB, so that a warp's copies in flight cover the latency
    static constexpr int kTok = 32 * (kKRow + kVRow) <= 8192 ? 32 : 16, kSteps = 32 / kTok;   // steps per unit
    static constexpr int kVOff = kTok * kKRow, kKsOff = kVOff + kTok * kVRow, kVsOff = kKsOff + kTok;
    static constexpr int kSlot = kVOff + kTok * kVRow + (kCodes ? 128 : 0);   // (scales padded to a line)
    static constexpr int kSlots = 3;
    static constexpr int kQOff = kWarps * kSlots * kSlot;          // q fragments [kGroups NR][D / 32][32 lanes] x 16 bytes
    static constexpr int kQExpOff = kQOff + kGroups * NR * (D / 32) * 512;   // row exponents of q
    static constexpr int kKeysOff = kQExpOff + kRows * 4;
    static constexpr int kMlOff = kKeysOff + kRows * 8;
    static constexpr int kPrefixOff = (kMlOff + kWarps * kWarpRows * 8 + 15) / 16 * 16;
    static_assert(kWarpRows * DV * 4 <= kSlots * kSlot, "O rows of a warp");
    static constexpr int smem(int B) { return kPrefixOff + (2 * B + 1) * 4; }
    static constexpr int kRegCtas = NR * DV <= 128 ? 4 : (NR * DV <= 256 ? 3 : 2);
    static constexpr int kSmemCtas = 227 * 1024 / (smem(64) + 1024);
    static constexpr int kCtas = kRegCtas < kSmemCtas ? kRegCtas : kSmemCtas;
    static_assert(kCtas >= 1 && smem(kKv4MaxBatch) <= 227 * 1024, "shared memory budget");
};

template <bool kCodes, int D, int DV, int NR>
__global__ void __launch_bounds__(kPagedThreads, PagedLayout<kCodes, D, DV, NR>::kCtas) paged_fwd_kernel(const PagedFwdParams p) {
    using Lay = PagedLayout<kCodes, D, DV, NR>;
    constexpr int S = Lay::kSlots, kRows = Lay::kRows, kWarpRows = Lay::kWarpRows, kTok = Lay::kTok, CK = kTok / 16, kSteps = Lay::kSteps;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int* prefix = reinterpret_cast<int*>(smem + Lay::kPrefixOff);
    const uint32_t ring = base + warp * S * Lay::kSlot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (the finishing kernel waits for this grid's end)
    const Cut cut = build_prefix<kPagedThreads>(p, prefix, prefix + p.s.B + 1, kRows, gridDim.x);   // (ends with __syncthreads)
    const int per = cut.per;
    const int total = prefix[p.s.B];
    if (blockIdx.x == 0) {   // for the kernel that follows
        for (int i = tid; i <= p.s.B; i += kPagedThreads) p.prefix[i] = prefix[i];
        if (tid == 0) {
            p.prefix[kKv4MaxBatch + 1] = per;
            p.prefix[kKv4MaxBatch + 2] = cut.aligned;
        }
    }
    const int u0 = min(total, (int)blockIdx.x * per), u1 = min(total, u0 + per);
    const int g8 = lane >> 2, t4 = lane & 3, half = warp & 1;
    // the tokens of S^T's rows g8 and g8 + 8 of a chunk: with codes, row 2 t + e + 8 h is token t + 4 e + 8 h
    const int tok0 = kCodes ? (g8 >> 1) + 4 * (g8 & 1) : g8;
    float acc[DV / 16][NR][4];
    float qscale[NR][2], m_run[NR][2], mu[NR][2], l_run[NR][2];   // m_run: the max plus the shift; mu: it, or 0
    int2* row_keys = reinterpret_cast<int2*>(smem + Lay::kKeysOff);
    int* q_exp = reinterpret_cast<int*>(smem + Lay::kQExpOff);
    float2* ml = reinterpret_cast<float2*>(smem + Lay::kMlOff);
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
        uint32_t slot_in = 0, slot_out = 0;
        auto issue = [&](int n) {   // the copies of step n (0, 1, 2, ...) of this share into the next slot
            const int x = n / kSteps, i = i0 + x, part = n % kSteps;
            if (i < i1) {
                if (part == 0 && (x & 15) == 0) {
                    ids = ids_next;
                    ids_next = page_id(i + 16 + (lane & 15));
                    const uint32_t in = __ballot_sync(kFullMask, ids >= 0) & 0xffffu;
                    live = (live & (0xffff0000u >> (x & 16))) | in << (x & 16);
                }
                const int id = __shfl_sync(kFullMask, ids, x & 15);
                if (id >= 0) {
                    const int tok = 32 * half + part * kTok;   // of the page
                    const int left = w.s.lk - page_of(w, 2 * i + (warp >> 1)) * kPage - tok;   // tokens that exist: what
                    const long row0 = ((long)id * p.c.Hkv + t.h) * kPage + tok;                // lies behind may be anything
                    const unsigned char *k = p.c.k + row0 * Lay::kKRow, *v = p.c.v + row0 * Lay::kVRow;
                    const uint32_t st = ring + slot_in;
                    constexpr int kKP = Lay::kKRow / 16, kVP = Lay::kVRow / 16;   // pieces of a row
#pragma unroll
                    for (int y = 0; y < kTok * kKP / 32; ++y) {
                        const int z = y * 32 + lane, r = z / kKP, c = z % kKP;
                        copy16n(row_piece<Lay::kKRow, kTok>(st, r, c), k + z * 16, r < left ? 16 : 0);
                    }
#pragma unroll
                    for (int y = 0; y < kTok * kVP / 32; ++y) {
                        const int z = y * 32 + lane, r = z / kVP, c = z % kVP;
                        copy16n(row_piece<Lay::kVRow, kTok>(st + Lay::kVOff, r, c), v + z * 16, r < left ? 16 : 0);
                    }
                    if (kCodes && lane < 2 * CK) {
                        const int c = lane % CK;
                        copy16n(st + (lane < CK ? Lay::kKsOff : Lay::kVsOff) + c * 16,
                                (lane < CK ? p.c.k_scales : p.c.v_scales) + row0 + c * 16, min(max(left - c * 16, 0), 16));
                    }
                }
                slot_in = slot_in == (S - 1) * Lay::kSlot ? 0 : slot_in + Lay::kSlot;
            }
            copy_commit();
        };
#pragma unroll
        for (int x = 0; x < S - 1; ++x) issue(x);
        // ------------------------------------------------ its queries
        const int n_rows = min(kRows, w.rows - t.rb * kRows);
        const bool pairs = Lay::kGroups > 1 && n_rows > kWarpRows;   // rows by the warps of a page
        const int row0 = pairs ? (warp & 1) * kWarpRows : 0;         // this warp's first row of the block
        const int row_end = min(n_rows, row0 + kWarpRows);
        auto sync_page = [&] {   // the warps that read each other's slots
            if (pairs) asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory");
            else __syncwarp();
        };
        const MaskBand mb = mask_band(w.s.nq, w.s.lk, p.win_left, p.win_right, p.sinks);
        if (tid < kRows) {
            const int row = t.rb * kRows + tid, i = row / p.group;
            row_keys[tid] = row < w.rows ? make_int2(band_key_lo(mb, i), band_key_hi(mb, i)) : make_int2(0, 0);
        }
        auto q_row = [&](int r) {   // row r of the block, or null
            r += t.rb * kRows;
            return r < w.rows ? p.q + (long)(w.s.q0 + r / p.group) * p.q_stride + (long)(t.h * p.group + r % p.group) * D : nullptr;
        };
        if constexpr (kCodes) {   // row r times 2^e has its largest element in [2^14, 2^15) (its own exponent per row)
            for (int r = warp; r < kRows; r += kWarps) {
                const __nv_bfloat16* src = q_row(r);
                uint32_t m = 0;
                if (src) {
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) m = __vmaxu2(m, reinterpret_cast<const uint32_t*>(src)[x * 32 + lane] & 0x7fff7fffu);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(kFullMask, m, o));
                const int top = (int)(max(m & 0xffffu, m >> 16) >> 7);   // (biased; 255, an infinity or a NaN: as the largest number's)
                if (lane == 0) q_exp[r] = min(max(14 - (top - 127), -113), 126);
            }
            __syncthreads();
        }
        for (int task = warp; task < (pairs ? Lay::kGroups : 1) * NR * (D / 32); task += kWarps) {   // 8 rows x 32 channels
            const int n = task / (D / 32), kk = task % (D / 32), r = n * 8 + g8;
            const __nv_bfloat16* src = q_row(r);
            uint32_t f[4] = {0u, 0u, 0u, 0u};
            if (src) {
                if constexpr (kCodes) {
                    // channels 64 G + 16 t4 + 8 (kk % 2) .. + 7; word i of a code row's piece serves k step i:
                    // its bytes (0, 1) and (2, 3) are the two pairs of a step
                    const uint4 v = *reinterpret_cast<const uint4*>(src + (kk >> 1) * 64 + 16 * t4 + 8 * (kk & 1));
                    const float e = pow2(q_exp[r]);
                    auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
                    auto hi = [](uint32_t x) { return __uint_as_float(x & 0xffff0000u); };
                    f[0] = pack_f16x2(lo(v.x) * e, hi(v.x) * e);
                    f[1] = pack_f16x2(lo(v.y) * e, hi(v.y) * e);
                    f[2] = pack_f16x2(lo(v.z) * e, hi(v.z) * e);
                    f[3] = pack_f16x2(lo(v.w) * e, hi(v.w) * e);
                } else {
                    const uint32_t* x = reinterpret_cast<const uint32_t*>(src + kk * 32) + t4;
                    f[0] = x[0], f[1] = x[4], f[2] = x[8], f[3] = x[12];
                }
            }
            *reinterpret_cast<uint4*>(smem + Lay::kQOff + (task * 32 + lane) * 16) = make_uint4(f[0], f[1], f[2], f[3]);
        }
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                qscale[n][c] = kCodes ? p.scale_log2 * pow2(-q_exp[row0 + n * 8 + 2 * t4 + c]) : p.scale_log2;
                m_run[n][c] = -INFINITY;
                mu[n][c] = l_run[n][c] = 0.f;
            }
        // keys that this warp's first and last rows (hence all) see
        const int q_first = (t.rb * kRows + row0) / p.group, q_last = (t.rb * kRows + row_end - 1) / p.group;
        const int full_lo = band_key_lo(mb, q_last), full_hi = band_key_hi(mb, q_first);
        // ... and that some row sees, sinks aside
        const int some_lo = band_key_lo(mb, q_first), some_hi = band_key_hi(mb, q_last);
#pragma unroll
        for (int j = 0; j < DV / 16; ++j)
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) acc[j][n][x] = 0.f;
        __syncthreads();   // the q fragments are in place
        const uint32_t qfrag = base + Lay::kQOff + row0 / 8 * (D / 32) * 512 + lane * 16;

        // kTok keys from slot `st`, the first key0. kWhole: every row sees all of them.
        bool force = true;   // some row has yet to see its first key
        auto step = [&](auto whole_tag, const uint32_t st, const int key0) {
            constexpr bool kWhole = decltype(whole_tag)::value;
            float sc[CK][NR][4];   // s - mu: per chunk [key tok0, tok0 + 8][row 2 t4, 2 t4 + 1] at 2 * key + row
#pragma unroll
            for (int ck = 0; ck < CK; ++ck)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) sc[ck][n][x] = 0.f;
            if constexpr (kCodes) {
#pragma unroll
                for (int G = 0; G < D / 64; ++G) {
                    uint4 q0[NR], q1[NR];
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        q0[n] = lds128(qfrag + (n * (D / 32) + 2 * G) * 512);
                        q1[n] = lds128(qfrag + (n * (D / 32) + 2 * G + 1) * 512);
                    }
#pragma unroll
                    for (int ck = 0; ck < CK; ++ck) {
                        const uint4 a = lds128(row_piece<Lay::kKRow, kTok>(st, tok0 + 16 * ck, 4 * G + t4));
                        const uint4 b = lds128(row_piece<Lay::kKRow, kTok>(st, tok0 + 16 * ck + 8, 4 * G + t4));
                        const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a0 = codes_f16((uint16_t)wa[i]), a1 = codes_f16((uint16_t)wb[i]),
                                           a2 = codes_f16((uint16_t)(wa[i] >> 16)), a3 = codes_f16((uint16_t)(wb[i] >> 16));
#pragma unroll
                            for (int n = 0; n < NR; ++n) {
                                const uint4 q = i < 2 ? q0[n] : q1[n];
                                mma_f16(sc[ck][n], a0, a1, a2, a3, (i & 1) ? q.z : q.x, (i & 1) ? q.w : q.y);
                            }
                        }
                    }
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk) {
                    uint4 q[NR];
#pragma unroll
                    for (int n = 0; n < NR; ++n) q[n] = lds128(qfrag + (n * (D / 32) + kk) * 512);
#pragma unroll
                    for (int ck = 0; ck < CK; ++ck)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint4 a = ldsm4(row_piece<Lay::kKRow, kTok>(st, ck * 16 + (lane & 15), kk * 4 + y * 2 + (lane >> 4)));
#pragma unroll
                            for (int n = 0; n < NR; ++n) mma_bf16(sc[ck][n], a.x, a.y, a.z, a.w, y ? q[n].z : q[n].x, y ? q[n].w : q[n].y);
                        }
                }
            }
            uint32_t v_scales[CK][2], past = 0;   // of tokens t4 and t4 + 4, t4 + 8 and t4 + 12
#pragma unroll
            for (int ck = 0; ck < CK; ++ck) {
                if constexpr (kCodes) {
                    const uint4 e = lds128(st + Lay::kVsOff + ck * 16);
                    const uint32_t e0 = byte_pair(e.x, e.y, t4), e1 = byte_pair(e.z, e.w, t4);
                    v_scales[ck][0] = scales_of_v(e0), v_scales[ck][1] = scales_of_v(e1);
                    past |= past_v(e0) | past_v(e1);
                }
                float ks[2] = {1.f, 1.f};
                if constexpr (kCodes) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) ks[x] = paged_scale(lds8(st + Lay::kKsOff + ck * 16 + tok0 + 8 * x));
                }
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float s = sc[ck][n][x] * qscale[n][x & 1];
                        sc[ck][n][x] = kCodes ? fmaf(s, ks[x >> 1], -mu[n][x & 1]) : s - mu[n][x & 1];
                    }
            }
            if constexpr (!kWhole) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int2 k = row_keys[row0 + n * 8 + 2 * t4 + c];
#pragma unroll
                        for (int x = 0; x < 2 * CK; ++x) {
                            const int j = key0 + tok0 + 8 * x;
                            if (!(j < k.y && (j >= k.x || j < p.sinks))) sc[x >> 1][n][2 * (x & 1) + c] = -INFINITY;
                        }
                    }
            }
            const bool some_past = kCodes && (past & 0x01000100u) != 0;
            bool move = force || some_past, scale_p = false;
#pragma unroll
            for (int ck = 0; ck < CK; ++ck)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) move |= sc[ck][n][x] > kPagedTau - kPagedShift;
            if (__any_sync(kFullMask, move)) {
                bool unset = false;
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    float al[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int ck = 0; ck < CK; ++ck) mx = fmaxf(mx, fmaxf(sc[ck][n][c], sc[ck][n][2 + c]));
                        mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 16));
                        // (a row whose own maximum has not moved stays as it is, whatever its neighbours do)
                        const bool moves = mx > kPagedTau - kPagedShift || m_run[n][c] == -INFINITY;
                        const float m_new = moves ? fmaxf(m_run[n][c], mx + mu[n][c] + kPagedShift) : m_run[n][c];
                        al[c] = m_new == -INFINITY ? 1.f : ex2_mufu(m_run[n][c] - m_new);
                        const float mu_new = m_new == -INFINITY ? 0.f : m_new;
#pragma unroll
                        for (int ck = 0; ck < CK; ++ck) {
                            sc[ck][n][c] += mu[n][c] - mu_new;
                            sc[ck][n][2 + c] += mu[n][c] - mu_new;
                        }
                        unset |= m_new == -INFINITY && row_keys[row0 + n * 8 + 2 * t4 + c].y > 0;
                        m_run[n][c] = m_new;
                        mu[n][c] = mu_new;
                        l_run[n][c] *= al[c];
                    }
#pragma unroll
                    for (int j = 0; j < DV / 16; ++j)
#pragma unroll
                        for (int x = 0; x < 4; ++x) acc[j][n][x] *= al[x & 1];
                }
                force = __any_sync(kFullMask, unset);
                scale_p = kCodes && __any_sync(kFullMask, some_past);   // (rows whose maximum stays have changed nothing)
            }
            uint32_t b0[CK][NR], b1[CK][NR];
            auto weights = [&](auto scaled_tag) {
#pragma unroll
                for (int ck = 0; ck < CK; ++ck)
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        float x[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float e = ex2_mufu(sc[ck][n][y]);
                            l_run[n][y & 1] += e;
                            x[y] = e;
                            if constexpr (decltype(scaled_tag)::value) {   // (0 for a masked key, whose scale may be NaN)
                                const float f = scale_of_p(lds8(st + Lay::kVsOff + ck * 16 + tok0 + 8 * (y >> 1)));
                                if (kWhole || sc[ck][n][y] != -INFINITY) x[y] = e * f;
                            }
                        }
                        b0[ck][n] = transpose8x8(pack_bf16x2(x[0], x[1]));
                        b1[ck][n] = transpose8x8(pack_bf16x2(x[2], x[3]));
                    }
            };
            if (scale_p) {
                if constexpr (kCodes) weights(std::true_type{});
            } else {
                weights(std::false_type{});
            }
            // ---------------------------------------- values
            const uint32_t sv = st + Lay::kVOff;
            uint32_t nans = 0;
#pragma unroll
            for (int ck = 0; ck < CK; ++ck) {
                if constexpr (kCodes) {
#pragma unroll
                    for (int x = 0; x < DV / 32; ++x) {   // channels 32 x + 4 g8 .. + 3
                        const int piece = 2 * x + (g8 >> 2), at = (g8 & 3) * 4;
                        uint32_t wv[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) wv[y] = lds32(row_piece<Lay::kVRow, kTok>(sv, ck * 16 + t4 + 4 * y, piece) + at);
#pragma unroll
                        for (int y = 0; y < 4; ++y) nans |= changed(wv[y]);
                        uint32_t f[4][2];   // channel c: tokens (t, t + 4), (t + 8, t + 12)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int y = 0; y < 2; ++y)
                                f[c][y] = times(codes_bf16(__byte_perm(wv[2 * y], wv[2 * y + 1], (4 + c) << 12 | c << 4)), v_scales[ck][y]);
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
                            mma_bf16(acc[2 * x][n], f[0][0], f[1][0], f[0][1], f[1][1], b0[ck][n], b1[ck][n]);
                            mma_bf16(acc[2 * x + 1][n], f[2][0], f[3][0], f[2][1], f[3][1], b0[ck][n], b1[ck][n]);
                        }
                    }
                } else {
                    uint32_t in[2] = {~0u, ~0u};   // values that no row sees may hold anything: they read as zero
                    if constexpr (!kWhole) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int j = key0 + ck * 16 + 8 * (y >> 1) + 2 * t4 + (y & 1);
                            if (!(j < some_hi && (j >= some_lo || j < p.sinks))) in[y >> 1] &= (y & 1) ? 0x0000ffffu : 0xffff0000u;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < DV / 16; ++j) {
                        uint4 a = ldsm4t(row_piece<Lay::kVRow, kTok>(sv, ck * 16 + (lane & 7) + ((lane >> 4) << 3),
                                                                           2 * j + ((lane >> 3) & 1)));
                        if constexpr (!kWhole) a = make_uint4(a.x & in[0], a.y & in[0], a.z & in[1], a.w & in[1]);
#pragma unroll
                        for (int n = 0; n < NR; ++n) mma_bf16(acc[j][n], a.x, a.y, a.z, a.w, b0[ck][n], b1[ck][n]);
                    }
                }
            }
            if constexpr (kCodes) {
                if (__any_sync(kFullMask, (nans & 0x80808080u) != 0)) {
                    // the same products, of 1 for a NaN code with 1 for a row that sees the key (with p the rows that do not
                    // would get 0 times NaN)
#pragma unroll 1
                    for (int ck = 0; ck < CK; ++ck) {
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
                            uint32_t x[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const int2 k = row_keys[row0 + n * 8 + 2 * t4 + (y & 1)];
                                const int j = key0 + ck * 16 + tok0 + 8 * (y >> 1);
                                x[y] = kWhole || (j < k.y && (j >= k.x || j < p.sinks)) ? 0x3f80u : 0u;
                            }
                            b0[0][n] = transpose8x8(x[0] | x[1] << 16);
                            b1[0][n] = transpose8x8(x[2] | x[3] << 16);
                        }
#pragma unroll
                        for (int x = 0; x < DV / 32; ++x) {
                            const int piece = 2 * x + (g8 >> 2), at = (g8 & 3) * 4;
                            uint32_t wv[4], f[4][2];
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                wv[y] = nan_codes(lds32(row_piece<Lay::kVRow, kTok>(sv, ck * 16 + t4 + 4 * y, piece) + at));
#pragma unroll
                            for (int c = 0; c < 4; ++c)
#pragma unroll
                                for (int y = 0; y < 2; ++y)   // (1 in bf16 for a NaN code)
                                    f[c][y] = (__byte_perm(wv[2 * y], wv[2 * y + 1], (4 + c) << 12 | c << 4) >> 15 & 0x00010001u) * 0x3f80u;
#pragma unroll
                            for (int n = 0; n < NR; ++n)
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    float hits[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma_bf16(hits, f[2 * y][0], f[2 * y + 1][0], f[2 * y][1], f[2 * y + 1][1], b0[0][n], b1[0][n]);
#pragma unroll
                                    for (int z = 0; z < 4; ++z)
                                        if (hits[z] > 0.f) acc[2 * x + y][n][z] = __uint_as_float(0x7fc00000u);
                                }
                        }
                    }
                }
            }
        };

        const int steps = (i1 - i0) * kSteps;
        for (int n = 0; n < steps; ++n) {
            copy_wait<S - 2>();
            sync_page();   // the slot is full, and whoever reads it has read the one before
            issue(n + S - 1);
            const int x = n / kSteps, i = i0 + x;
            const bool valid = (live >> (x & 31)) & 1u;
            const uint32_t slot = slot_out;
            slot_out = slot_out == (S - 1) * Lay::kSlot ? 0 : slot_out + Lay::kSlot;
            const int page0 = page_of(w, 2 * i + (warp >> 1)) * kPage + n % kSteps * kTok;
#pragma unroll 1
            for (int x0 = pairs ? 0 : half, x1 = pairs ? 2 : half + 1; x0 < x1; ++x0) {   // (half a page each)
                const uint32_t st = base + ((warp & 2) + x0) * S * Lay::kSlot + slot;
                const int key0 = page0 + 32 * x0;
                if (valid && key0 < w.s.lk) {
                    if (key0 >= full_lo && key0 + kTok <= full_hi) step(std::true_type{}, st, key0);
                    else step(std::false_type{}, st, key0);
                }
            }
        }
        // ------------------------------------------------ the four warps' rows become one
        // (every copy into the slots has landed and been read: each warp's O rows go there)
        const bool ends = i1 == w.units, starts = i0 == 0;
        copy_wait<0>();
        sync_page();
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
                if (g8 == 0) ml[warp * kWarpRows + row] = make_float2(m_run[n][c], l);
                if constexpr (kCodes) {
#pragma unroll
                    for (int x = 0; x < DV / 32; ++x)
                        *reinterpret_cast<float4*>(mine + row * DV + 32 * x + 4 * g8) =
                            make_float4(acc[2 * x][n][c], acc[2 * x][n][2 + c], acc[2 * x + 1][n][c], acc[2 * x + 1][n][2 + c]);
                } else {
#pragma unroll
                    for (int j = 0; j < DV / 16; ++j) {
                        mine[row * DV + j * 16 + g8] = acc[j][n][c];
                        mine[row * DV + j * 16 + g8 + 8] = acc[j][n][2 + c];
                    }
                }
            }
        __syncthreads();
        const int part = 2 * blockIdx.x + (starts ? 1 : 0);
        for (int x = tid; x < n_rows * (DV / 4); x += kPagedThreads) {
            const int row = x / (DV / 4), c4 = x % (DV / 4), at = pairs ? row % kWarpRows : row;
            float2 v[kWarps];
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int y = 0; y < kWarps; ++y) {   // (a warp without this row has no share)
                v[y] = pairs && (y & 1) != row / kWarpRows ? make_float2(-INFINITY, 0.f) : ml[y * kWarpRows + at];
                m = fmaxf(m, v[y].x);
            }
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int y = 0; y < kWarps; ++y) {   // in warp order: the same sum on every run
                const float f = v[y].x == -INFINITY ? 0.f : ex2_mufu(v[y].x - m);
                l += v[y].y * f;
                if (v[y].x != -INFINITY) {   // (a factor of 0 leaves a NaN)
                    const float4 z = *reinterpret_cast<const float4*>(smem + y * S * Lay::kSlot + (at * DV + 4 * c4) * 4);
                    o.x = fmaf(f, z.x, o.x);
                    o.y = fmaf(f, z.y, o.y);
                    o.z = fmaf(f, z.z, o.z);
                    o.w = fmaf(f, z.w, o.w);
                }
            }
            if (starts && ends) {
                const int r = t.rb * kRows + row, i = r / p.group, head = t.h * p.group + r % p.group;
                const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // (NaN stays)
                *reinterpret_cast<uint2*>(p.o + ((long)(w.s.q0 + i) * p.H + head) * DV + 4 * c4) =
                    make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
                if (c4 == 0) p.lse[lse_at(p, w, t.b, i, head)] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            } else {
                *reinterpret_cast<float4*>(p.part_o + ((long)part * kRows + row) * DV + 4 * c4) = o;
                if (c4 == 0) *reinterpret_cast<float2*>(p.part_ml + ((long)part * kRows + row) * 2) = make_float2(m, l);
            }
        }
        __syncthreads();   // the next row block's copies come after these reads
    }
}

constexpr int kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads) paged_finish_kernel(const PagedFwdParams p, int rows_per_block) {
    finish_row(p, (long)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5), rows_per_block);
}

template <bool kCodes, int D, int DV, int NR>
cudaError_t launch_one(const PagedFwdParams& p, int num_sms, cudaStream_t stream) {
    using Lay = PagedLayout<kCodes, D, DV, NR>;
    static std::atomic<unsigned long long> allowed;
    auto kern = paged_fwd_kernel<kCodes, D, DV, NR>;
    cudaError_t e = allow_smem(kern, Lay::smem(kKv4MaxBatch), allowed);
    if (e != cudaSuccess) return e;
    int grid = num_sms * Lay::kCtas;
    if (grid > kKv4MaxCtas) grid = kKv4MaxCtas;
    kern<<<grid, kPagedThreads, Lay::smem(p.s.B), stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long)p.s.total * p.H + kJoinThreads / 32 - 1) / (kJoinThreads / 32)));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_finish_kernel, p, Lay::kRows);
}

template <bool kCodes, int D, int DV>
cudaError_t launch_dims(const PagedFwdParams& p, int num_sms, cudaStream_t stream) {
    return paged_row_tiles(p.group, p.s.B, p.s.total) == 1 ? launch_one<kCodes, D, DV, 1>(p, num_sms, stream)
                                                           : launch_one<kCodes, D, DV, 2>(p, num_sms, stream);
}
template <bool kCodes>
cudaError_t launch_form(const PagedFwdParams& p, int num_sms, cudaStream_t stream) {
    const int d = p.c.d, dv = p.c.dv;
    if (d == 64 && dv == 64) return launch_dims<kCodes, 64, 64>(p, num_sms, stream);
    if (d == 128 && dv == 128) return launch_dims<kCodes, 128, 128>(p, num_sms, stream);
    if (d == 192 && dv == 192) return launch_dims<kCodes, 192, 192>(p, num_sms, stream);
    if (d == 192 && dv == 128) return launch_dims<kCodes, 192, 128>(p, num_sms, stream);
    if (d == 256 && dv == 256) return launch_dims<kCodes, 256, 256>(p, num_sms, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_fwd(const PagedFwdParams& p, bool codes, int num_sms, cudaStream_t stream) {
    return codes ? launch_form<true>(p, num_sms, stream) : launch_form<false>(p, num_sms, stream);
}

}  // namespace attn
