// Linear attention with a decay per head on tcgen05, 128 tokens a chunk. linear.h gives the form
// (a, b, c, the state X) that the forward and the gradients share, linear.cu the scan between
// the two kernels and the roundings.
//
// What bounds it: for head dims of 128 a chunk of a head brings 96 KB (32 KB each of a, b and c)
// and takes 32 KB of output, which is 5600 cycles of an SM's share of HBM's rate; its products take 2600
// on the tensor cores (mma.sync, at a quarter of the rate and with its operands through
// registers, set the time there). What costs is the chain through the chunks: scores, decays, product,
// state, and the next chunk's product with it. So one CTA per SM walks segments with the
// next tiles in flight, in roles that each take less than the loads do:
//   warps 0-7    the outputs, P c + D^(..) a X, and the state, X = D^n X + (the chunk's share), in registers in
//                fp32, written to shared memory in bf16 for the next chunk
//   warps 8-15   P: scores from tensor memory, times the decays, back as bf16 over their columns (the
//                next product's A operand); then b times the state's weights, in two bf16 terms,
//                the first in place once the scores are taken
//   warp 16      tile loads (TMA), a ring for each of a, b and c
//   warp 17      the products, each issued by an elected lane of the converged warp:
//                P = a b^T;  O2 = a X;  O1 = P c;  KV = (w b)^T c
//   warp 18      which segments come next
// The tensor pipe executes in issue order, so the next scores may be issued behind the product
// that reads P. Every wait is bounded.
//
// DT of the output's columns per CTA: all 128 of them for head dims of 128, else 64, which is what
// tensor memory (P 128 columns, O1, O2 and KV's two tiles of 128 channels) and shared memory hold at
// 192 and 256; a and b are then read again, from L2, for the next columns.
#include <atomic>

#include "kv4.h"
#include "linear.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kCh = kLinChunk;           // tokens of a chunk (the tiles below are for 128)
static_assert(kCh == 128, "tiles of 128 tokens");
constexpr int kBox = 16384;              // 128 rows x 64 columns
constexpr int kHalf = kBox / 2;          // 64 rows

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// Two loads of 16 columns and one wait
__device__ __forceinline__ void tmem_ld16x2(uint32_t t0, uint32_t t1, uint32_t (&r)[16], uint32_t (&s)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(s[0]), "=r"(s[1]),
          "=r"(s[2]), "=r"(s[3]), "=r"(s[4]), "=r"(s[5]), "=r"(s[6]), "=r"(s[7]), "=r"(s[8]), "=r"(s[9]), "=r"(s[10]),
          "=r"(s[11]), "=r"(s[12]), "=r"(s[13]), "=r"(s[14]), "=r"(s[15])
        : "r"(t0), "r"(t1)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 32 bytes to memory, a whole sector per lane (the segments' shares: a row of a state per lane)
__device__ __forceinline__ void store32(void* dst, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// 32 bytes from memory. A row per lane by 16 bytes fetched each sector twice (shared memory leaves L1 little room), which
// held up the SM's other loads and barriers for 15 000 cycles wherever a segment began.
__device__ __forceinline__ void load32(const float* src, float* v) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(src)
                 : "memory");
}
// A box of shared memory to the tensor of the map, tracked by this thread's bulk groups
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
// tc_commit by the lane that the mma_.._w calls elect
__device__ __forceinline__ void commit_w(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}
// A value that all lanes have, from an instruction whose result the compiler knows to be one for the warp: what
// follows from it (loops, stages, descriptors) then stays in uniform registers, which the products take their operands from.
__device__ __forceinline__ int uniform(int x) { return (int)__reduce_or_sync(kFullMask, (unsigned)x); }
// A bounded wait of the whole warp. All lanes poll (one access for the warp, no branch around it), and the clock is
// read only after some polls: reading it first delays the warp's resumption.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, const WaitCtx& w) {
    uint64_t deadline = 0;
    bool ok = true;
    for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
        if ((it & 63u) == 0) {
            const uint64_t now = global_timer_ns();
            if (deadline == 0) {
                deadline = now + w.budget_ns;
            } else if (*w.abort_flag || now > deadline) {
                *w.abort_flag = 1;
                atomicCAS(w.status, kStatusOk, kStatusWaitTimeout);
                ok = false;
                break;
            }
        }
    }
    return __all_sync(kFullMask, ok);
}
// Whether the phase has completed, without waiting. (Tests of several barriers ahead of their waits overlap: under
// the other warps' shared-memory traffic each takes some 250 cycles.)
__device__ __forceinline__ bool test_phase(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_unless(bool done, uint32_t bar, uint32_t parity, const WaitCtx& w) {
    return __all_sync(kFullMask, done) || wait_all(bar, parity, w);
}
__device__ __forceinline__ float lo16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi16(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// 16 bytes of a tile of boxes of `rows` rows x 64 columns (128-byte swizzle): row, piece of eight columns
template <int kBoxBytes = kBox>
__device__ __forceinline__ uint4* piece_at(uint8_t* tile, int row, int piece) {
    return reinterpret_cast<uint4*>(tile + (piece >> 3) * kBoxBytes + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}

// The CTA's segments. One warp finds them (LinFinder searches the offsets) and hands them to the others through a
// ring in shared memory: the search in each role's loop made the code several times as long, and warps that resume from
// a wait missed the instruction cache.
constexpr int kSegments = 4;   // entries of the ring
struct SegmentRing {
    LinSegment at[kSegments];
};
template <bool kBack>
__device__ __forceinline__ void find_segments(const LinParams& p, int range, SegmentRing* ring, uint32_t full, uint32_t empty,
                                              const WaitCtx& w, int lane, bool shares) {
    LinFinder finder(p, range, lane);
    LinSegment g;
    for (uint32_t i = 0;; ++i) {
        // (only those whose share somebody wants: the next segment, or who wants the last state)
        do g = finder.next(p);
        while (shares && g.rows > 0 && !(kBack ? g.after_start : g.before_end) && !p.final);
        if (!wait_all(empty + 8 * (i % kSegments), ((i / kSegments) & 1u) ^ 1u, w)) return;
        if (lane == 0) {
            ring->at[i % kSegments] = g;
            mbar_arrive(full + 8 * (i % kSegments));
        }
        __syncwarp();
        if (g.rows == 0) return;
    }
}
// A role's place in the walk. An item is a chunk (the outputs forwards, shares backwards: of one query head, x).
struct Walk {
    LinSegment t;
    int chunks, chunk, x, per;
    uint32_t taken;
    bool live;
};
__device__ __forceinline__ bool next_segment(Walk& i, const SegmentRing* ring, uint32_t full, uint32_t empty, const WaitCtx& w,
                                             int lane) {
    const uint32_t slot = i.taken % kSegments;
    if (!wait_all(full + 8 * slot, (i.taken / kSegments) & 1u, w)) return false;
    const LinSegment& t = ring->at[slot];
    i.t = LinSegment{uniform(t.run), uniform(t.h), uniform(t.row0), uniform(t.rows), uniform(t.after_start), uniform(t.before_end)};
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + 8 * slot);
    ++i.taken;
    i.chunks = (i.t.rows + kCh - 1) / kCh;
    i.chunk = i.x = 0;
    i.live = i.t.rows > 0;
    return true;
}
template <bool kBack>
__device__ __forceinline__ int chunk_row(const Walk& i) {   // of the segment
    return (kBack ? i.chunks - 1 - i.chunk : i.chunk) * kCh;
}

// Rows of (w b)^T c, the state's channels, come in tiles of 128. At 192 the second tile starts 64 early (its first
// 64 rows are the first tile's), at 64 the tile's other rows are of whatever lies behind b (kTailPad: within the
// buffers); neither are looked at.
template <int DK>
__host__ __device__ constexpr int tile_channel(int mt) { return DK > 128 && 128 * mt + 128 > DK ? DK - 128 : 128 * mt; }
template <int DK>
__device__ __forceinline__ bool tile_row(int mt, int row) { return tile_channel<DK>(mt) + row >= 128 * mt && tile_channel<DK>(mt) + row < DK; }
template <int DK>
__device__ __forceinline__ SmemDesc weighted_desc(uint32_t base, int mt, int box_bytes) {
    return sdesc_sw128_split(base + tile_channel<DK>(mt) / 64 * box_bytes, box_bytes, 1024);
}
template <int DK>
constexpr int kTailPad = DK == 64 ? kHalf : 0;

// ---------------------------------------------------------------- outputs
template <int DK, int DT>
struct OutLay {
    static constexpr int MT = (DK + 127) / 128, kB = DK / 64 * kBox, kC = DT / 64 * kBox, kX = DT / 64 * DK * 128;
    // Stages of a, b and c: two where the 227 KB allow it (a load takes 2000 to 3500 cycles under load). The second
    // term has buffers of 64 tokens or, where all of a, b and c have two stages of 32 KB (kShareA), goes where a
    // was once a X is done.
    static constexpr bool kShareA = DK == 128 && DT == 128;
    static constexpr int kRingA = DK <= 128 ? 2 : 1, kRingB = DK <= 192 ? 2 : 1, kRingC = 2;
    static constexpr int kTerm = DK / 64 * kHalf, kTerms = DK <= 128 ? 2 : 1;
    static constexpr int kAOff = kRingB * kB, kCOff = kAOff + kRingA * kB, kXOff = kCOff + kRingC * kC, kTermOff = kXOff + kX;
    // a chunk's outputs pass through X's place on their way to memory, which no product needs then (at 64 it is too small)
    static constexpr int kOutOff = DK == 64 ? kTermOff + kTerms * kTerm + kTailPad<DK> : kXOff, kOutBox = DK == 64 ? kBox : DK * 128;
    static constexpr int kBarOff = DK == 64 ? kOutOff + kBox : kTermOff + (kShareA ? 0 : kTerms * kTerm);
    // warps 0-3 and 4-7 share the columns, or the tiles of X's channels, or have work for the first four alone
    static constexpr int kWarpsX = DT == 128 || MT == 2 ? 8 : 4, kWarpsO = DT == 128 ? 8 : 4;
    static constexpr int kAFull = 0, kAFree = 2, kBFull = 4, kBFree = 6, kCFull = 8, kCFree = 10, kPFull = 12, kPReady = 13,
                         kWReady = 14, kTFree = 16, kOFull = 18, kOFree = 19, kXReady = 20, kKVFull = 21, kDrain = 22,
                         kRFull = 23,
                         kREmpty = kRFull + kSegments, kNumBars = kREmpty + kSegments;
    static constexpr int kMiscOff = kBarOff + (kNumBars + 1) / 2 * 16, kRingOff = kMiscOff + 16;
    static constexpr int kPowOff = kRingOff + (int)sizeof(SegmentRing), kBytes = kPowOff + 8 * 64 * 4;   // 64 floats for each of warps 8-15
    static_assert(kBytes <= 227 * 1024, "shared memory budget");
    static_assert(kXOff % 1024 == 0 && kTermOff % 1024 == 0 && kBarOff % 16 == 0 && kPowOff % 16 == 0, "alignment of tiles and tables");
    static constexpr uint32_t kTmP = 0, kTmO1 = 128, kTmO2 = 128 + DT, kTmKV = 128 + 2 * DT;
    static_assert(kTmKV + MT * DT <= 512, "tensor memory budget");
};
constexpr int kOutThreads = 640;
// registers per thread: at launch, and as the roles share them (their sum over the five warpgroups is the launch's)
constexpr int kOutRegs = 96, kOutRegsX = 120, kOutRegsP = 88, kOutRegsRest = 64;
static_assert(2 * kOutRegsX + 2 * kOutRegsP + kOutRegsRest <= 5 * kOutRegs, "registers of the launch");

template <int DK, int DT, bool kBack>
__global__ void __launch_bounds__(kOutThreads, 1)
lin_out_tc_kernel(const __grid_constant__ LinMaps maps, const LinParams p) {
    using Lay = OutLay<DK, DT>;
    constexpr int MT = Lay::MT;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_addr(smem);
    if (base & 1023u) {
        if (threadIdx.x == 0) atomicCAS(p.status, kStatusOk, kStatusMisaligned);
        return;
    }
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    auto bar = [&](int i) -> uint32_t { return base + Lay::kBarOff + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::kMiscOff + 4);
    SegmentRing* ring = reinterpret_cast<SegmentRing*>(smem + Lay::kRingOff);
    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < Lay::kNumBars; ++i) {
            const bool by_p = i == Lay::kPReady || i == Lay::kWReady || i == Lay::kWReady + 1;
            mbar_init(bar(i), by_p ? 256 : i == Lay::kOFree ? 32 * Lay::kWarpsO : i == Lay::kXReady ? 32 * Lay::kWarpsX
                              : i >= Lay::kREmpty ? 10 + Lay::kWarpsX : 1);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 16 && lane == 0) {
        tma_prefetch_desc(&maps.out);
        tma_prefetch_desc(&maps.a);
        tma_prefetch_desc(&maps.b);
        tma_prefetch_desc(&maps.c);
    }
    if (warp == 17) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    launch_next();   // (see launch_early)
    wait_for_last();
    const WaitCtx w{abort_flag, p.status, p.wait_budget_ns};
    const int per = p.per;
    const int nt = p.DV / DT, range = blockIdx.x / nt, tile = blockIdx.x - range * nt;
    Walk at;
    at.per = per;
    at.taken = 0;
    bool ok = true;
    auto take = [&] { return next_segment(at, ring, bar(Lay::kRFull), bar(Lay::kREmpty), w, lane); };
    auto advance = [&] {   // to the next item; true where a new segment is due
        if (++at.x < at.per) return false;
        at.x = 0;
        return ++at.chunk == at.chunks;
    };
    constexpr uint32_t RB = Lay::kRingB, RC = Lay::kRingC;
    // where the second term goes: backwards with several query heads a is read for each of them, so that it keeps to
    // the first stage and the term to the second; else the term follows a X in its stage
    const bool follows = Lay::kShareA && !(kBack && per > 1);
    const uint32_t RA = Lay::kShareA && !follows ? 1 : Lay::kRingA;

    if (warp >= 16) {
        setmaxnreg_dec<kOutRegsRest>();
        if (warp == 18) {
            find_segments<kBack>(p, range, ring, bar(Lay::kRFull), bar(Lay::kREmpty), w, lane, false);
        } else if (warp == 16) {
            // ------------------------------------------------------------ loads
            uint32_t na = 0, nb = 0, sent_b = 0;   // tiles of a, of b and c
            for (bool fresh = true;; fresh = advance()) {
                if (fresh && !(ok = take())) break;
                if (!at.live) break;
                const int row = at.t.row0 + chunk_row<kBack>(at);
                const int ha = kBack ? at.t.h : at.t.h * per + at.x, hb = kBack ? at.t.h * per + at.x : at.t.h;
                const bool new_a = !kBack || at.x == 0, new_b = kBack || at.x == 0;
                if (new_b) {
                    const uint32_t st = nb % RB, full = bar(Lay::kBFull + st), to = base + st * Lay::kB;
                    if (!(ok = wait_all(bar(Lay::kBFree + st), ((nb / RB) & 1u) ^ 1u, w))) break;
                    if (lane == 0) {
                        mbar_expect_tx(full, Lay::kB);
#pragma unroll
                        for (int y = 0; y < DK / 64; ++y) tma_load_3d(to + y * kBox, &maps.b, full, y * 64, hb, row);
                        ++sent_b;
                    }
                    __syncwarp();
                }
                if (new_a) {
                    const uint32_t st = na % RA, full = bar(Lay::kAFull + st), to = base + Lay::kAOff + st * Lay::kB;
                    if (!(ok = wait_all(bar(Lay::kAFree + st), ((na / RA) & 1u) ^ 1u, w))) break;
                    if (lane == 0) {
                        mbar_expect_tx(full, Lay::kB);
#pragma unroll
                        for (int y = 0; y < DK / 64; ++y) tma_load_3d(to + y * kBox, &maps.a, full, y * 64, ha, row);
                    }
                    __syncwarp();
                    ++na;
                }
                if (new_b) {
                    const uint32_t st = nb % RC, full = bar(Lay::kCFull + st), to = base + Lay::kCOff + st * Lay::kC;
                    if (!(ok = wait_all(bar(Lay::kCFree + st), ((nb / RC) & 1u) ^ 1u, w))) break;
                    if (lane == 0) {
                        mbar_expect_tx(full, Lay::kC);
#pragma unroll
                        for (int y = 0; y < DT / 64; ++y)
                            tma_load_3d(to + y * kBox, &maps.c, full, tile * DT + y * 64, hb, row);
                    }
                    __syncwarp();
                    ++nb;
                }
            }
            if (lane == 0) {   // (a pending load must land before the CTA gives up its memory)
                for (uint32_t i = na > RA ? na - RA : 0; i < na; ++i) drain_wait(bar(Lay::kAFull + i % RA), (i / RA) & 1u, p.wait_budget_ns);
                for (uint32_t i = sent_b > RB ? sent_b - RB : 0; i < sent_b; ++i)
                    drain_wait(bar(Lay::kBFull + i % RB), (i / RB) & 1u, p.wait_budget_ns);
                for (uint32_t i = nb > RC ? nb - RC : 0; i < nb; ++i) drain_wait(bar(Lay::kCFull + i % RC), (i / RC) & 1u, p.wait_budget_ns);
            }
            __syncwarp();
        } else if (warp == 17) {
            // ------------------------------------------------------------ products
            constexpr uint32_t kIdP = idesc_bf16_f32(128, 128, false, false);    // a, b: rows of channels
            constexpr uint32_t kIdN = idesc_bf16_f32(128, DT, false, true);      // B (X, c): rows along the sum
            constexpr uint32_t kIdKV = idesc_bf16_f32(128, DT, true, true);      // (w b)^T, c: rows of tokens
            const SmemDesc a_km = sdesc_sw128_split(base + Lay::kAOff, 16, 1024), b_km = sdesc_sw128_split(base, 16, 1024);
            const SmemDesc c_mn = sdesc_sw128_split(base + Lay::kCOff, kBox, 1024);
            const SmemDesc x_mn = sdesc_sw128_split(base + Lay::kXOff, DK * 128, 1024);
            uint32_t na = 0, nb = 0, nc = 0, it = 0, outs = 0, xs = 0, shared = 0;   // tiles taken, items, rounds of O, states, shares
            // `at` is an item ahead: what is finished here is the one before, if any, with its tiles in a_st and b_st
            bool some = false, shares = false, last_x = false;
            int x = 0;
            uint32_t a_st = 0, b_st = 0;
            for (bool fresh = true;; fresh = advance()) {
                const uint32_t a_off = desc_step(a_st * Lay::kB), c_st = (nc - 1 + (kBack || x == 0)) % RC,
                               c_off = desc_step(c_st * Lay::kC);
                const bool head = !kBack || x == 0, tail = !kBack || last_x;   // of a round of the outputs
                if (some) {
                    const bool new_c = kBack || x == 0;
                    const uint32_t c_full = bar(Lay::kCFull + nc % RC), c_parity = (nc / RC) & 1u;
                    const bool x_done = test_phase(bar(Lay::kXReady), xs & 1u), o_done = test_phase(bar(Lay::kOFree), (outs & 1u) ^ 1u),
                               c_done = test_phase(c_full, c_parity), p_done = test_phase(bar(Lay::kPReady), it & 1u);
                    if (head) {
                        if (!(ok = wait_unless(x_done, bar(Lay::kXReady), xs & 1u, w))) break;
                        ++xs;
                        if (!(ok = wait_unless(o_done, bar(Lay::kOFree), (outs & 1u) ^ 1u, w))) break;
                        tc_fence_after_sync();
#pragma unroll
                        for (int y = 0; y < DK / 16; ++y)
                            mma_ss_w(tmem + Lay::kTmO2, a_km, a_off + desc_step((y >> 2) * kBox + (y & 3) * 32), x_mn,
                                     desc_step(y * 2048), kIdN, y > 0);
                        if (follows && shares) commit_w(bar(Lay::kTFree + 1));
                        else if (!kBack || per == 1) commit_w(bar(Lay::kAFree + a_st));
                    }
                    if (new_c) {
                        if (!(ok = wait_unless(c_done, c_full, c_parity, w))) break;
                        ++nc;
                    }
                    if (!(ok = wait_unless(p_done, bar(Lay::kPReady), it & 1u, w))) break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        mma_ts_w(tmem + Lay::kTmO1, tmem + Lay::kTmP + (y >> 1) * 32 + (y & 1) * 8, c_mn, c_off + desc_step(y * 2048),
                                 kIdN, !head || y > 0);
                    ++it;
                    if (tail) {
                        commit_w(bar(Lay::kOFull));
                        ++outs;
                    }
                }
                if (fresh && !(ok = take())) break;
                const bool new_a = !kBack || at.x == 0, new_b = kBack || at.x == 0;
                const uint32_t a_full = bar(Lay::kAFull + na % RA), a_parity = (na / RA) & 1u;
                const uint32_t b_full = bar(Lay::kBFull + nb % RB), b_parity = (nb / RB) & 1u;
                const uint32_t a_was = a_st, b_was = b_st, rows0 = desc_step(b_st * Lay::kB);
                // the next scores come now if their tiles have come: they have the longer way to go
                const bool a_done = test_phase(a_full, a_parity), b_done = test_phase(b_full, b_parity),
                           w_done = test_phase(bar(Lay::kWReady), shared & 1u);
                const bool early = __all_sync(kFullMask, some && at.live && (!new_a || a_done) && (!new_b || b_done));
#pragma unroll 1
                for (int turn = 0; turn < 2 && ok; ++turn) {
                    if ((turn == 0) == early) {
                        if (!at.live) continue;
                        if (new_a && !(ok = wait_unless(early, a_full, a_parity, w))) break;
                        if (new_b && !(ok = wait_unless(early, b_full, b_parity, w))) break;
                        na += new_a;
                        nb += new_b;
                        a_st = (na - 1) % RA;
                        b_st = (nb - 1) % RB;
                        tc_fence_after_sync();
                        const uint32_t next_a = desc_step(a_st * Lay::kB), next_b = desc_step(b_st * Lay::kB);
#pragma unroll
                        for (int y = 0; y < DK / 16; ++y) {
                            const uint32_t step = desc_step((y >> 2) * kBox + (y & 3) * 32);
                            mma_ss_w(tmem + Lay::kTmP, a_km, next_a + step, b_km, next_b + step, kIdP, y > 0);
                        }
                        commit_w(bar(Lay::kPFull));
                        if (kBack && per > 1 && at.x == per - 1) commit_w(bar(Lay::kAFree + a_st));   // (a X came with x = 0)
                    } else if (some) {
                        if (shares) {
#pragma unroll 1
                            for (int half = 0; half < 2; ++half) {
                                if (half < 3 - Lay::kTerms) {   // (one pass over all rows, or two over 64)
                                    if (!(ok = wait_unless(half == 0 && w_done, bar(Lay::kWReady + half), shared & 1u, w))) break;
                                    tc_fence_after_sync();
                                }
                                const uint32_t rows = desc_step(half * kHalf), buf = Lay::kTerms == 2 ? half : 0;
                                const uint32_t more = (kBack && x > 0) || half > 0;
#pragma unroll 1
                                for (int mt = 0; mt < MT; ++mt) {
                                    const SmemDesc b_mn = weighted_desc<DK>(base, mt, kBox);
                                    const uint32_t t_at = Lay::kShareA ? base + Lay::kAOff + (follows ? a_was : 1) * Lay::kB + half * kHalf
                                                                       : base + Lay::kTermOff + buf * Lay::kTerm;
                                    const SmemDesc t_mn = weighted_desc<DK>(t_at, mt, Lay::kShareA ? kBox : kHalf);
                                    const uint32_t kv = tmem + Lay::kTmKV + mt * DT;
#pragma unroll
                                    for (int y = 0; y < 4; ++y)
                                        mma_ss_w(kv, b_mn, rows0 + rows + desc_step(y * 2048), c_mn, c_off + rows + desc_step(y * 2048),
                                                 kIdKV, y > 0 ? 1u : more);
#pragma unroll
                                    for (int y = 0; y < 4; ++y)
                                        mma_ss_w(kv, t_mn, desc_step(y * 2048), c_mn, c_off + rows + desc_step(y * 2048), kIdKV, 1);
                                }
                                if (!follows && half >= Lay::kTerms - 1) commit_w(bar(Lay::kTFree + Lay::kTerms - 1));
                            }
                            if (follows) commit_w(bar(Lay::kAFree + a_was));
                            if (!ok) break;
                            ++shared;
                            if (tail) commit_w(bar(Lay::kKVFull));
                        }
                        if (kBack || last_x) {
                            commit_w(bar(Lay::kBFree + b_was));
                            commit_w(bar(Lay::kCFree + c_st));
                        }
                    }
                }
                if (!ok || !at.live) break;
                some = true;
                x = at.x;
                last_x = x == per - 1;
                shares = (kBack || last_x) && at.chunk + 1 < at.chunks;   // the item adds to the state
            }
            commit_w(bar(Lay::kDrain));
            if (lane == 0) drain_wait(bar(Lay::kDrain), 0, p.wait_budget_ns);
            __syncwarp();
        }
    } else if (warp >= 8) {
        // ------------------------------------------------------------ P, and the weights on b
        setmaxnreg_dec<kOutRegsP>();
        const int q4 = warp & 3, hf = (warp - 8) >> 2, t = tid - 256, row = q4 * 32 + lane;
        const uint32_t t_p = tmem + ((uint32_t)(q4 * 32) << 16) + Lay::kTmP;
        // Decays of at least 2^-4 keep the factor 2^(31 * 4) that a row's own block needs in range; the others look each power up
        constexpr float kSlowest = -4.f;
        // pw[c]: forwards D^(31 - c), zeros from 32 on; backwards D^(c - 32), zeros up to there
        float* pw = reinterpret_cast<float*>(smem + Lay::kPowOff) + (warp - 8) * 64;
        const float* near_pw = pw + (kBack ? 32 : 0);
        const float* own_pw = pw + (kBack ? 32 - lane : 31 - lane);
        uint32_t it = 0, na = 0, nb = 0, shared = 0;
        float l2 = 0.f, far0 = 0.f, far1 = 0.f, diag = 0.f;
        for (bool fresh = true;; fresh = advance(), ++it) {
            if (fresh) {
                if (!(ok = take()) || !at.live) break;
                l2 = log2_decay(p, at.t.h);
                __syncwarp();
                pw[lane] = kBack ? 0.f : decay_pow(l2, 31 - lane);
                pw[32 + lane] = kBack ? decay_pow(l2, lane) : 0.f;
                __syncwarp();
                // to a block of 32 columns on the near side: the distance to its nearer end, then near_pw
                const int d0 = kBack ? 32 * hf - row : row - 32 * hf - 31, d1 = kBack ? d0 + 64 : d0 - 64;
                far0 = d0 >= 0 ? decay_pow(l2, d0) : 0.f;
                far1 = d1 >= 0 ? decay_pow(l2, d1) : 0.f;
                diag = exp2f(l2 * (kBack ? -lane : lane - 31));   // (the same, to the block that holds the row: not below 1)
            }
            const int n = min(kCh, at.t.rows - chunk_row<kBack>(at));
            const bool shares = (kBack || at.x == per - 1) && at.chunk + 1 < at.chunks;
            if (kBack || at.x == 0) ++nb;
            if (!kBack || at.x == 0) ++na;
            uint8_t* b_tile = smem + (nb - 1) % RB * Lay::kB;
            if (!(ok = wait_all(bar(Lay::kPFull), it & 1u, w))) break;
            tc_fence_after_sync();
#pragma unroll 1
            for (int b = hf; b < 4; b += 2) {   // columns 32 b .. + 31; P goes to the first 16 of them
                uint32_t out[16];
                if (b == q4 || (kBack ? b > q4 : b < q4)) {
                    uint32_t r[32];
                    tmem_ld32(t_p + 32 * b, r);
                    if (kBack && n < 32 * b + 32) {   // columns past the sequence's end, whatever they hold
                        const int end = n - 32 * b;
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (c >= end) r[c] = 0u;
                    }
                    if (b != q4 || l2 >= kSlowest) {
                        const float far = b == q4 ? diag : b == hf ? far0 : far1;
                        const uint64_t f = f32x2(far, far);
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const ulonglong2 g = *reinterpret_cast<const ulonglong2*>(near_pw + c);
                            float v[4];
                            f32x2_split(fmul2(f32x2(u2f(r[c]), u2f(r[c + 1])), fmul2(f, g.x)), v[0], v[1]);
                            f32x2_split(fmul2(f32x2(u2f(r[c + 2]), u2f(r[c + 3])), fmul2(f, g.y)), v[2], v[3]);
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                if (b == q4 && (kBack ? c + z < lane : c + z > lane)) v[z] = 0.f;
                            out[c / 2] = pack_bf16x2(v[0], v[1]);
                            out[c / 2 + 1] = pack_bf16x2(v[2], v[3]);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            const float v0 = (kBack ? c >= lane : c <= lane) ? u2f(r[c]) * own_pw[c] : 0.f;
                            const float v1 = (kBack ? c + 1 >= lane : c + 1 <= lane) ? u2f(r[c + 1]) * own_pw[c + 1] : 0.f;
                            out[c / 2] = pack_bf16x2(v0, v1);
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c) out[c] = 0u;
                }
                tmem_st16(t_p + 32 * b, out);
            }
            if (n < kCh && (kBack || at.x == 0)) {   // c's rows past the sequence's end, whatever they hold
                const int r = t & 127;
                if (!(ok = wait_all(bar(Lay::kCFull + (nb - 1) % RC), ((nb - 1) / RC) & 1u, w))) break;
                if (r >= n)
                    for (int c = t >> 7; c < DT / 8; c += 2)
                        *piece_at(smem + Lay::kCOff + (nb - 1) % RC * Lay::kC, r, c) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            tmem_st_wait();
            tc_fence_before_sync();
            mbar_arrive(bar(Lay::kPReady));
            if (!shares) continue;
            // as many rows at a time as there are buffers for; a thread takes every kLanes-th piece of its row, so that
            // eight neighbouring rows lie in eight banks
            constexpr int kRows = 64 * Lay::kTerms, kLanes = 256 / kRows, kPieces = DK / 8 / kLanes, kAtOnce = kPieces % 3 == 0 ? 3 : 4;
#pragma unroll 1
            for (int r0 = 0; r0 < kCh; r0 += kRows) {
                const int r = r0 + (t & (kRows - 1)), p0 = t / kRows;
                const uint32_t use = r0 == 0 ? 0 : 1, round = Lay::kTerms == 2 ? shared : 2 * shared + use;
                const float weight = r < n ? decay_pow(l2, kBack ? r + 1 : n - 1 - r) : 0.f;
                uint4 lo[kPieces];
#pragma unroll
                for (int y0 = 0; y0 < kPieces; y0 += kAtOnce) {
                    uint4 v[kAtOnce];
#pragma unroll
                    for (int y = 0; y < kAtOnce; ++y) v[y] = *piece_at(b_tile, r, p0 + kLanes * (y0 + y));
#pragma unroll
                    for (int y = 0; y < kAtOnce; ++y) {
                        const uint32_t u[4] = {v[y].x, v[y].y, v[y].z, v[y].w};
                        uint32_t h[4], l[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const float f0 = lo16(u[z]) * weight, f1 = hi16(u[z]) * weight;
                            h[z] = pack_bf16x2(f0, f1);
                            l[z] = pack_bf16x2(f0 - lo16(h[z]), f1 - hi16(h[z]));
                        }
                        if (kBack && r >= n) h[0] = h[1] = h[2] = h[3] = l[0] = l[1] = l[2] = l[3] = 0u;
                        *piece_at(b_tile, r, p0 + kLanes * (y0 + y)) = make_uint4(h[0], h[1], h[2], h[3]);
                        lo[y0 + y] = make_uint4(l[0], l[1], l[2], l[3]);
                    }
                }
                // the second term, once its place is free
                if (!(ok = wait_all(bar(Lay::kTFree + Lay::kTerms - 1), (round & 1u) ^ (follows ? 0u : 1u), w))) break;
                uint8_t* second = Lay::kShareA ? smem + Lay::kAOff + (follows ? (na - 1) % RA : 1) * Lay::kB
                                               : smem + Lay::kTermOff + (Lay::kTerms == 2 ? (r >> 6) * Lay::kTerm : 0);
#pragma unroll
                for (int y = 0; y < kPieces; ++y) {
                    const int c = p0 + kLanes * y;
                    *(Lay::kShareA ? piece_at(second, r, c) : piece_at<kHalf>(second, r & 63, c)) = lo[y];
                }
                fence_proxy_async_smem();
                mbar_arrive(bar(Lay::kWReady + use));
            }
            if (!ok) break;
            ++shared;
        }
    } else {
        // ------------------------------------------------------------ the outputs and the state
        setmaxnreg_inc<kOutRegsX>();
        const int q4 = warp & 3, group = warp >> 2, row = q4 * 32 + lane;   // of X (a tile's) and of the outputs
        const int col0 = DT == 128 ? 64 * group : 0, mt = DT == 128 ? 0 : group;
        const bool has_x = tile_row<DK>(mt, row);
        const int channel = tile_channel<DK>(mt) + row;
        const uint32_t t_row = tmem + ((uint32_t)(q4 * 32) << 16) + col0;
        // (32 rows of 128 bytes that are this warp's alone, as X's rows and then as those of the outputs)
        uint8_t* staged = smem + Lay::kOutOff + (col0 >> 6) * Lay::kOutBox + q4 * 4096;
        at.per = kBack ? 1 : per;   // (backwards one round of outputs for all query heads)
        uint32_t outs = 0, moved = 0;
        float X[64];
        float l2 = 0.f, into = 0.f, over = 0.f;
        // `at` is an item ahead: the outputs are those of the one before, if any; `last`: of a segment
        int n = 0, token0 = 0, head = 0, column = 0;   // its tokens, where the outputs go
        bool some = false, moves = false, last = true;
        for (bool fresh = true; warp < Lay::kWarpsX; fresh = advance()) {
            if (fresh && !(ok = take())) break;
            if (last && at.live) {   // (X is in shared memory: the registers take the next segment's)
                l2 = log2_decay(p, at.t.h);
                // forwards it starts behind the range before's last segment, backwards in front of the one after's first
                const int slot = lin_start_slot(p, at.t, range, kBack);
                const bool trans = slot >= 0 ? p.states_trans : p.init_trans;
                const long size = (long)DK * p.DV;
                const float* src = slot >= 0 ? p.states + slot * size : p.init ? p.init + at.t.run * size : nullptr;
                const int c0 = tile * DT + col0;
                if (!src || !has_x) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) X[c] = 0.f;
                } else if (trans) {
                    const float* from = src + (long)c0 * DK + channel;
#pragma unroll
                    for (int c = 0; c < 64; ++c) X[c] = from[c * DK];
                } else {
                    const float* from = src + (long)channel * p.DV + c0;
                    if ((reinterpret_cast<uintptr_t>(src) & 31u) == 0) {
#pragma unroll
                        for (int c = 0; c < 64; c += 8) load32(from + c, X + c);
                    } else {
#pragma unroll
                        for (int c = 0; c < 64; c += 4) {
                            const float4 y = *reinterpret_cast<const float4*>(from + c);
                            X[c] = y.x, X[c + 1] = y.y, X[c + 2] = y.z, X[c + 3] = y.w;
                        }
                    }
                }
            }
            if (some) {
                if (!(ok = wait_all(bar(Lay::kOFull), outs & 1u, w))) break;
                tc_fence_after_sync();
                if (warp < Lay::kWarpsO) {
                    // all 32 rows by one copy from shared memory (row by row from registers the stores alone took a third
                    // of the shared memory's time); at a sequence's end those that exist, one by one
                    const bool whole = q4 * 32 + 32 <= n;
                    uint8_t* direct = reinterpret_cast<uint8_t*>(
                        p.out + ((long)(token0 + row) * (kBack ? p.Hkv : p.Hkv * per) + head) * p.DV + column);
#pragma unroll 1
                    for (int c = 0; c < 64; c += 16) {
                        uint32_t o1[16], o2[16], o[8];
                        tmem_ld16x2(t_row + Lay::kTmO1 + c, t_row + Lay::kTmO2 + c, o1, o2);
#pragma unroll
                        for (int z = 0; z < 8; ++z)
                            o[z] = pack_bf16x2(fmaf(into, u2f(o2[2 * z]), p.scale * u2f(o1[2 * z])),
                                               fmaf(into, u2f(o2[2 * z + 1]), p.scale * u2f(o1[2 * z + 1])));
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            uint8_t* to = whole ? staged + lane * 128 + ((((c >> 3) + z) ^ (lane & 7)) << 4) : direct + 2 * c + 16 * z;
                            if (row < n) *reinterpret_cast<uint4*>(to) = make_uint4(o[4 * z], o[4 * z + 1], o[4 * z + 2], o[4 * z + 3]);
                        }
                    }
                    tc_fence_before_sync();
                    mbar_arrive(bar(Lay::kOFree));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (whole && lane == 0) {
                        tma_store_3d(&maps.out, smem_addr(staged), column, head, token0 + q4 * 32);
                        bulk_commit_group();
                    }
                }
                ++outs;
                if (moves && !last) {
                    if (!(ok = wait_all(bar(Lay::kKVFull), moved & 1u, w))) break;
                    ++moved;
                    tc_fence_after_sync();
#pragma unroll
                    for (int c = 0; c < 64; c += 32) {
                        uint32_t r[32];
                        tmem_ld32(t_row + Lay::kTmKV + mt * DT + c, r);
#pragma unroll
                        for (int z = 0; z < 32; ++z) X[c + z] = fmaf(X[c + z], over, kBack ? p.scale * u2f(r[z]) : u2f(r[z]));
                    }
                    tc_fence_before_sync();
                }
                if (lane == 0) bulk_wait_group_read0();
                __syncwarp();
            }
            // (the products with the last X are done: the outputs that use it have been here)
            if (!last || at.live) {
                if (has_x) {
#pragma unroll
                    for (int c = 0; c < 64; c += 8)
                        *piece_at<DK * 128>(smem + Lay::kXOff, channel, (col0 + c) >> 3) =
                            make_uint4(pack_bf16x2(X[c], X[c + 1]), pack_bf16x2(X[c + 2], X[c + 3]), pack_bf16x2(X[c + 4], X[c + 5]),
                                       pack_bf16x2(X[c + 6], X[c + 7]));
                }
                fence_proxy_async_smem();
                mbar_arrive(bar(Lay::kXReady));
            }
            if (!at.live) break;
            some = true;
            const int r0 = chunk_row<kBack>(at);
            n = min(kCh, at.t.rows - r0);
            moves = at.x == at.per - 1;
            last = moves && at.chunk + 1 == at.chunks;
            into = (kBack ? 1.f : p.scale) * (row < n ? decay_pow(l2, kBack ? n - 1 - row : row + 1) : 0.f);
            over = decay_pow(l2, n);
            token0 = at.t.row0 + r0;
            head = kBack ? at.t.h : at.t.h * per + at.x;
            column = tile * DT + col0;
        }
        if (lane == 0) bulk_wait_group0();
        __syncwarp();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- segments' shares
// X' of a segment for X = 0. An item's sum is made in tensor memory, its tokens weighted by the decay up to the
// chunk's end (backwards: its start), and added to the segment's in registers: the tensor cores' sums are cut off rather
// than rounded, which over 5000 tokens of four query heads in one sum made 4e-6 of a state. b times the weight is in
// bf16 terms: the first in place, the others in buffers of 64 tokens. Three terms (all 24 bits) where a state leaves the call, else two
// (the states are rounded to 8 bits by the products that use them).
template <int DK, int DT>
struct StateLay {
    static constexpr int MT = (DK + 127) / 128, kB = DK / 64 * kBox, kC = DT / 64 * kBox, kStage = kB + kC;
    static constexpr int kTerm = DK / 64 * kHalf, kSets = DK <= 192 ? 2 : 1;   // sets of buffers
    static constexpr int kTermOff = 2 * kStage, kBarOff = kTermOff + kSets * 2 * kTerm + kTailPad<DK>;
    static constexpr int kFull = 0, kEmpty = 2, kWReady = 4, kWFree = 6, kSFull = 8, kSFree = 10, kDrain = 12, kRFull = 13,
                         kREmpty = kRFull + kSegments, kNumBars = kREmpty + kSegments;
    static constexpr int kMiscOff = kBarOff + (kNumBars + 1) / 2 * 16, kRingOff = kMiscOff + 16;
    static constexpr int kBytes = kRingOff + (int)sizeof(SegmentRing);
    static_assert(kBytes <= 227 * 1024, "shared memory budget");
    static_assert(kTermOff % 1024 == 0 && kBarOff % 16 == 0 && kRingOff % 8 == 0, "alignment of tiles and tables");
    static constexpr int kWarpsR = DT == 128 || MT == 2 ? 8 : 4;   // as in OutLay
    static constexpr uint32_t kAcc = MT * DT, kCols = 2 * kAcc <= 128 ? 128 : 256;
    static_assert(2 * kAcc <= kCols, "tensor memory budget");
};
constexpr int kStateThreads = 608;   // warps 0-7: weights, 8-15: the segment's sum, 16: loads, 17: products, 18: segments

template <int DK, int DT, bool kBack>
__global__ void __launch_bounds__(kStateThreads, 1)
lin_state_tc_kernel(const __grid_constant__ LinMaps maps, const LinParams p) {
    using Lay = StateLay<DK, DT>;
    constexpr int MT = Lay::MT;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_addr(smem);
    if (base & 1023u) {
        if (threadIdx.x == 0) atomicCAS(p.status, kStatusOk, kStatusMisaligned);
        return;
    }
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    auto bar = [&](int i) -> uint32_t { return base + Lay::kBarOff + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::kMiscOff + 4);
    SegmentRing* ring = reinterpret_cast<SegmentRing*>(smem + Lay::kRingOff);
    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < Lay::kNumBars; ++i) {
            const bool by_w = i == Lay::kWReady || i == Lay::kWReady + 1, by_r = i == Lay::kSFree || i == Lay::kSFree + 1;
            mbar_init(bar(i), by_w ? 256 : by_r ? 32 * Lay::kWarpsR : i >= Lay::kREmpty ? 10 + Lay::kWarpsR : 1);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 16 && lane == 0) {
        tma_prefetch_desc(&maps.b);
        tma_prefetch_desc(&maps.c);
    }
    if (warp == 17) {
        tmem_alloc(smem_addr(tmem_slot), Lay::kCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    launch_next();
    wait_for_last();
    const WaitCtx w{abort_flag, p.status, p.wait_budget_ns};
    const int nt = p.DV / DT, range = blockIdx.x / nt, tile = blockIdx.x - range * nt;
    Walk at;
    at.per = kBack ? p.per : 1;
    at.taken = 0;
    bool ok = true;
    auto take = [&] { return next_segment(at, ring, bar(Lay::kRFull), bar(Lay::kREmpty), w, lane); };
    auto advance = [&] {   // to the next item; true where a new segment is due
        if (++at.x < at.per) return false;
        at.x = 0;
        return ++at.chunk == at.chunks;
    };
    const int terms = p.final ? 3 : 2;   // of the weighted b
    uint32_t it = 0;

    if (warp == 18) {
        find_segments<kBack>(p, range, ring, bar(Lay::kRFull), bar(Lay::kREmpty), w, lane, true);
    } else if (warp == 16) {
        // ------------------------------------------------------------ loads
        for (bool fresh = true;; fresh = advance(), ++it) {
            if (fresh && !(ok = take())) break;
            if (!at.live) break;
            const int row = at.t.row0 + chunk_row<kBack>(at), hb = at.t.h * at.per + at.x;
            const uint32_t st = it & 1u;
            if (!(ok = wait_all(bar(Lay::kEmpty + st), ((it >> 1) & 1u) ^ 1u, w))) break;
            if (lane == 0) {
                const uint32_t to = base + st * Lay::kStage, full = bar(Lay::kFull + st);
                mbar_expect_tx(full, Lay::kStage);
#pragma unroll
                for (int y = 0; y < DK / 64; ++y) tma_load_3d(to + y * kBox, &maps.b, full, y * 64, hb, row);
#pragma unroll
                for (int y = 0; y < DT / 64; ++y)
                    tma_load_3d(to + Lay::kB + y * kBox, &maps.c, full, tile * DT + y * 64, hb, row);
            }
            __syncwarp();
        }
        if (lane == 0)
            for (uint32_t i = it > 2 ? it - 2 : 0; i < it; ++i)
                drain_wait(bar(Lay::kFull + (i & 1u)), (i >> 1) & 1u, p.wait_budget_ns);
        __syncwarp();
    } else if (warp == 17) {
        // ------------------------------------------------------------ products
        constexpr uint32_t kIdKV = idesc_bf16_f32(128, DT, true, true);
        const SmemDesc c_mn = sdesc_sw128_split(base + Lay::kB, kBox, 1024);
        for (bool fresh = true;; fresh = advance(), ++it) {
            if (fresh && !(ok = take())) break;
            if (!at.live) break;
            const uint32_t st = it & 1u, acc = tmem + st * Lay::kAcc, off = desc_step(st * Lay::kStage);
            if (!(ok = wait_all(bar(Lay::kSFree + st), ((it >> 1) & 1u) ^ 1u, w))) break;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                if (!(ok = wait_all(bar(Lay::kWReady + half), it & 1u, w))) break;
                tc_fence_after_sync();
                const uint32_t c0 = off + desc_step(half * kHalf), set = Lay::kSets == 2 ? half : 0, more = half > 0;
#pragma unroll 1
                for (int mt = 0; mt < MT; ++mt) {
                    const SmemDesc b_mn = weighted_desc<DK>(base, mt, kBox);
                    const SmemDesc t_mn = weighted_desc<DK>(base + Lay::kTermOff + 2 * set * Lay::kTerm, mt, kHalf);
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        mma_ss_w(acc + mt * DT, b_mn, c0 + desc_step(y * 2048), c_mn, c0 + desc_step(y * 2048), kIdKV, y > 0 ? 1u : more);
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        if (y < 4 * (terms - 1))
                            mma_ss_w(acc + mt * DT, t_mn, desc_step((y >> 2) * Lay::kTerm + (y & 3) * 2048), c_mn,
                                 c0 + desc_step((y & 3) * 2048), kIdKV, 1);
                }
                commit_w(bar(Lay::kWFree + set));
            }
            if (!ok) break;
            commit_w(bar(Lay::kEmpty + st));
            commit_w(bar(Lay::kSFull + st));
        }
        commit_w(bar(Lay::kDrain));
        if (lane == 0) drain_wait(bar(Lay::kDrain), 0, p.wait_budget_ns);
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------------------ weights
        // a thread takes pieces x, x + 4, .. of a row, so that eight neighbouring rows lie in eight banks
        const int r64 = tid & 63, p0 = tid >> 6;
        float l2 = 0.f;
        for (bool fresh = true;; fresh = advance(), ++it) {
            if (fresh) {
                if (!(ok = take()) || !at.live) break;
                l2 = log2_decay(p, at.t.h);
            }
            const int n = min(kCh, at.t.rows - chunk_row<kBack>(at));
            const uint32_t st = it & 1u;
            uint8_t* tiles = smem + st * Lay::kStage;
            if (!(ok = wait_all(bar(Lay::kFull + st), (it >> 1) & 1u, w))) break;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                const int row = half * 64 + r64;
                const uint32_t use = 2 * it + half, set = use % Lay::kSets;
                const bool in = row < n;
                const float weight = in ? decay_pow(l2, kBack ? row + 1 : n - 1 - row) : 0.f;
                uint8_t* buf = smem + Lay::kTermOff + 2 * set * Lay::kTerm;
                if (!(ok = wait_all(bar(Lay::kWFree + set), ((use / Lay::kSets) & 1u) ^ 1u, w))) break;
                constexpr int kPieces = DK / 32, kAtOnce = kPieces % 3 == 0 ? 3 : 2;
#pragma unroll 1
                for (int y0 = 0; y0 < kPieces; y0 += kAtOnce) {
                    uint4 v[kAtOnce];
#pragma unroll
                    for (int y = 0; y < kAtOnce; ++y) v[y] = *piece_at(tiles, row, p0 + 4 * (y0 + y));
#pragma unroll
                    for (int y = 0; y < kAtOnce; ++y) {
                        const uint32_t u[4] = {v[y].x, v[y].y, v[y].z, v[y].w};
                        const int c = p0 + 4 * (y0 + y);
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
                        *piece_at(tiles, row, c) = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
#pragma unroll
                        for (int term = 1; term < 3; ++term)
                            if (term < terms) *piece_at<kHalf>(buf + (term - 1) * Lay::kTerm, r64, c) =
                                make_uint4(o[term][0], o[term][1], o[term][2], o[term][3]);
                    }
                }
                if (!in)
                    for (int c = p0; c < DT / 8; c += 4) *piece_at(tiles + Lay::kB, row, c) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                mbar_arrive(bar(Lay::kWReady + half));
            }
            if (!ok) break;
        }
    } else {
        // ------------------------------------------------------------ the segment's sum
        const int q4 = warp & 3, group = (warp - 8) >> 2, row = q4 * 32 + lane;
        const int col0 = DT == 128 ? 64 * group : 0, mt = DT == 128 ? 0 : group;
        const uint32_t t_row = tmem + ((uint32_t)(q4 * 32) << 16) + mt * DT + col0;
        float X[64];
        float l2 = 0.f;
        for (bool fresh = true; warp < 8 + Lay::kWarpsR; ++it) {
            if (fresh) {
                if (!(ok = take()) || !at.live) break;
                l2 = log2_decay(p, at.t.h);
#pragma unroll
                for (int c = 0; c < 64; ++c) X[c] = 0.f;
            }
            const float over = at.x == 0 ? decay_pow(l2, min(kCh, at.t.rows - chunk_row<kBack>(at))) : 1.f;
            const uint32_t st = it & 1u;
            if (!(ok = wait_all(bar(Lay::kSFull + st), (it >> 1) & 1u, w))) break;
            tc_fence_after_sync();
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
                uint32_t r[16];
                tmem_ld16(t_row + st * Lay::kAcc + c, r);
#pragma unroll
                for (int z = 0; z < 16; ++z) X[c + z] = fmaf(X[c + z], over, u2f(r[z]));
            }
            tc_fence_before_sync();
            mbar_arrive(bar(Lay::kSFree + st));
            const int slot = lin_share_slot(p, at.t, range, kBack);
            if (!(fresh = advance()) || !tile_row<DK>(mt, row)) continue;
            if (kBack) {
#pragma unroll
                for (int c = 0; c < 64; ++c) X[c] *= p.scale;
            }
            float* dst = p.states + ((long)slot * DK + tile_channel<DK>(mt) + row) * p.DV + tile * DT + col0;
#pragma unroll
            for (int c = 0; c < 64; c += 8)   // (the workspace is 256-byte aligned)
                store32(dst + c, {f2u(X[c]), f2u(X[c + 1]), f2u(X[c + 2]), f2u(X[c + 3]), f2u(X[c + 4]), f2u(X[c + 5]), f2u(X[c + 6]),
                                  f2u(X[c + 7])});
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, Lay::kCols);
    }
}

template <class Kernel>
cudaError_t launch_tc(Kernel kern, int threads, int bytes, int tiles, std::atomic<unsigned long long>& allowed,
                      const LinParams& p, const LinMaps& maps, cudaStream_t stream) {
    cudaError_t e = allow_smem(kern, bytes, allowed);
    if (e != cudaSuccess) return e;
    return launch_early(kern, (unsigned)(p.ranges * tiles), threads, bytes, stream, maps, p);
}
// The registers that the roles share out must be those of the launch (asked once per kernel and device set)
template <class Kernel>
cudaError_t check_regs(Kernel kern, std::atomic<int>& done) {
    if (done.load(std::memory_order_relaxed)) return cudaSuccess;
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < kOutRegs) return cudaErrorInvalidConfiguration;
    done.store(1, std::memory_order_relaxed);
    return cudaSuccess;
}

template <int DK, int DT, bool kBack>
cudaError_t launch_one(bool outputs, const LinParams& p, const LinMaps& maps, cudaStream_t stream) {
    static std::atomic<unsigned long long> allowed[2];
    static std::atomic<int> regs;
    const int tiles = p.DV / DT;
    if (!outputs)
        return launch_tc(lin_state_tc_kernel<DK, DT, kBack>, kStateThreads, StateLay<DK, DT>::kBytes, tiles, allowed[0], p, maps, stream);
    const cudaError_t e = check_regs(lin_out_tc_kernel<DK, DT, kBack>, regs);
    if (e != cudaSuccess) return e;
    return launch_tc(lin_out_tc_kernel<DK, DT, kBack>, kOutThreads, OutLay<DK, DT>::kBytes, tiles, allowed[1], p, maps, stream);
}
template <bool kBack>
cudaError_t launch_dims(bool outputs, const LinParams& p, const LinMaps& maps, cudaStream_t stream) {
    if (p.DK == 64) return launch_one<64, 64, kBack>(outputs, p, maps, stream);
    if (p.DK == 128 && p.DV == 128) return launch_one<128, 128, kBack>(outputs, p, maps, stream);
    if (p.DK == 128) return launch_one<128, 64, kBack>(outputs, p, maps, stream);
    if (p.DK == 192) return launch_one<192, 64, kBack>(outputs, p, maps, stream);
    if (p.DK == 256) return launch_one<256, 64, kBack>(outputs, p, maps, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_linear_shares(const LinParams& p, const LinMaps& maps, bool back, cudaStream_t stream) {
    return back ? launch_dims<true>(false, p, maps, stream) : launch_dims<false>(false, p, maps, stream);
}
cudaError_t launch_linear_out(const LinParams& p, const LinMaps& maps, bool back, cudaStream_t stream) {
    if (p.total == 0) return cudaSuccess;
    return back ? launch_dims<true>(true, p, maps, stream) : launch_dims<false>(true, p, maps, stream);
}

}  // namespace attn
