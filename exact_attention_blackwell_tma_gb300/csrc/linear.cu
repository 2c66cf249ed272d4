// Linear attention with a decay per head: the plan of its segments, the scan over them, the
// kernels on mma.sync for the head dims that linear_tc.cu does not take, and the single
// token by the recurrence. linear.h gives the one form that the forward and the gradients share.
//
// Mathematics. Within a chunk of 64 tokens the pairs are taken as in attention, P_ij =
// D^|i-j| <a_i, b_j> and out += P c; what lies before the chunk enters through the state
// X, out += D^(..) a X. No factor is larger than 1, so nothing overflows for fast decays.
// Sums, states and decays are fp32. Roundings to bf16, the type of the tensor cores'
// operands: P, X before its product with a, and the weighted b in the state's update within
// a segment (like P in the exact attention: they reach outputs that are bf16 themselves).
// The segments' shares, which the states that leave a call are made of, take the weighted b
// as three bf16 terms, all 24 bits of it.
#include <atomic>

#include "kv4.h"
#include "linear.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kLinThreads = 256, kC = 64;
constexpr int kPanel = kC * 128;   // bytes of 64 rows x 64 columns

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes to shared memory, zeros where !in
__device__ __forceinline__ void copy16z(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait0() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Tiles in shared memory: panels of 64 columns, rows of 128 bytes whose 16-byte
// pieces are permuted by the row, so that eight rows of one piece (an ldmatrix
// phase) lie in different banks. Column `col` is a multiple of 8.
__device__ __forceinline__ uint32_t tile_at(uint32_t base, int row, int col, int rows = kC) {
    return base + (col >> 6) * (rows * 128) + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4);
}

// 64 tokens from row r0 of a sequence on (zeros past its end), `width` columns
__device__ __forceinline__ void load_tile(uint32_t dst, const __nv_bfloat16* src, long stride, int width, const Segment& g,
                                          int r0) {
    const int pieces = width >> 3, shift = 31 - __clz(pieces);
    for (int x = threadIdx.x; x < kC * pieces; x += kLinThreads) {
        const int row = (pieces & (pieces - 1)) == 0 ? x >> shift : x / pieces, col = (x - row * pieces) * 8, r = r0 + row;
        const bool in = r < g.n;
        copy16z(tile_at(dst, row, col), in ? src + (long)(g.q0 + r) * stride + col : src, in);
    }
}

// X = decay X + (weights b)^T c over a chunk. Warp w owns rows 16 MT (w % 4) .. of
// X and columns 32 (w / 4) ..; w_tab[j] is token j's weight.
// kTerms bf16 terms of the weighted b.
template <int MT, int kTerms>
__device__ __forceinline__ void update_state(float (&X)[MT][4][4], uint32_t b_tile, uint32_t c_tile, const float* w_tab,
                                             float decay) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t4 = lane & 3;
    const int m0 = (warp & 3) * 16 * MT, n0 = (warp >> 2) * 32;
    uint32_t cf[4][2][4];   // [16 tokens][16 columns]
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int x = 0; x < 2; ++x) ldsm4t(tile_at(c_tile, ks * 16 + (lane & 15), n0 + x * 16 + (lane >> 4) * 8), cf[ks][x]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float acc[4][4] = {};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t raw[4];
            float f[4][2];
            ldsm4t(tile_at(b_tile, ks * 16 + (lane & 7) + ((lane >> 4) << 3), m0 + mt * 16 + ((lane >> 3) & 1) * 8), raw);
#pragma unroll
            for (int x = 0; x < 4; ++x) {   // raw[x]: tokens 16 ks + 2 t4 + 8 (x / 2), + 1
                const int j = ks * 16 + 2 * t4 + 8 * (x >> 1);
                f[x][0] = __uint_as_float(raw[x] << 16) * w_tab[j];
                f[x][1] = __uint_as_float(raw[x] & 0xffff0000u) * w_tab[j + 1];
            }
#pragma unroll
            for (int term = 0; term < kTerms; ++term) {
                uint32_t w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    w[x] = pack_bf16x2(f[x][0], f[x][1]);
                    if (term + 1 < kTerms) {
                        f[x][0] -= __uint_as_float(w[x] << 16);
                        f[x][1] -= __uint_as_float(w[x] & 0xffff0000u);
                    }
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) mma_bf16(acc[n], w, cf[ks][n >> 1][(n & 1) * 2], cf[ks][n >> 1][(n & 1) * 2 + 1]);
            }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) X[mt][n][x] = fmaf(X[mt][n][x], decay, acc[n][x]);
    }
}

// Visits a thread's elements of X as f(row, column, x0, x1) of two neighbouring columns.
template <int MT, class F>
__device__ __forceinline__ void each_pair(float (&X)[MT][4][4], F f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int m0 = (warp & 3) * 16 * MT + (lane >> 2), n0 = (warp >> 2) * 32 + 2 * (lane & 3);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) f(m0 + mt * 16 + 8 * x, n0 + n * 8, X[mt][n][2 * x], X[mt][n][2 * x + 1]);
}

// Powers of the decay for a chunk whose tokens i < n (all 64, but for a sequence's last)
// exist. Token i's weight in the state: in order D^(n - 1 - i), backwards D^(i + 1).
struct Tables {
    float w[2 * kC];       // in order: D^(63 - x), zero from x = 64 on (read from x = 64 - n); backwards: D^(x + 1)
    float pow[kC + 1];     // D^x
};
template <bool kBack>
__device__ __forceinline__ void fill_tables(Tables* t, float l2) {
    for (int x = threadIdx.x; x < 2 * kC; x += kLinThreads) {
        t->w[x] = x < kC ? decay_pow(l2, kBack ? x + 1 : kC - 1 - x) : 0.f;
        if (x <= kC) t->pow[x] = decay_pow(l2, x);
    }
}
template <bool kBack>
__device__ __forceinline__ const float* weights(const Tables* t, int n) { return kBack ? t->w : t->w + kC - n; }

template <int DK>
struct StateSmem {
    static constexpr int kB = kC * DK * 2, kStage = kB + kPanel, kTables = 2 * kStage, kBytes = kTables + (int)sizeof(Tables);
};

// What each segment adds to the state (carried in: nothing); without a final state to
// return, the segment that a walk visits last is not needed.
template <int DK, bool kBack>
__global__ void __launch_bounds__(kLinThreads, DK <= 128 ? 2 : 1) lin_state_kernel(const LinParams p) {
    using Lay = StateSmem<DK>;
    constexpr int MT = DK / 64;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t base = smem_addr(smem);
    Tables* tab = reinterpret_cast<Tables*>(smem + Lay::kTables);
    const int nt = p.DV >> 6, tile = blockIdx.x % nt, h = blockIdx.x / nt % p.Hkv, s = blockIdx.x / nt / p.Hkv;
    const Segment g = segment_at(p, s);
    if (!g.live || (!p.final && (kBack ? g.first : g.last))) return;
    const float l2 = log2_decay(p, h);
    fill_tables<kBack>(tab, l2);
    const int per = kBack ? p.per : 1, chunks = (g.r1 - g.r0 + kC - 1) / kC, items = chunks * per;
    auto row_of = [&](int it) { return g.r0 + (kBack ? chunks - 1 - it / per : it / per) * kC; };
    auto issue = [&](int it) {
        if (it < items) {
            const int r = row_of(it), head = h * per + it % per;
            const uint32_t at = base + (it & 1) * Lay::kStage;
            load_tile(at, p.b + (long)head * DK, p.b_stride, DK, g, r);
            load_tile(at + Lay::kB, p.c + (long)head * p.DV + tile * 64, p.c_stride, 64, g, r);
        }
        copy_commit();
    };
    float X[MT][4][4] = {};
    issue(0);
    for (int it = 0; it < items; ++it) {
        copy_wait0();
        __syncthreads();
        issue(it + 1);
        const uint32_t at = base + (it & 1) * Lay::kStage;
        const int n = min(kC, g.r1 - row_of(it));
        update_state<MT, 3>(X, at, at + Lay::kB, weights<kBack>(tab, n), it % per == 0 ? tab->pow[n] : 1.f);
    }
    copy_wait0();
    float* dst = p.states + ((long)s * p.Hkv + h) * DK * p.DV + tile * 64;
    each_pair<MT>(X, [&](int row, int col, float x0, float x1) {
        *reinterpret_cast<float2*>(dst + (long)row * p.DV + col) = make_float2(x0, x1);
    });
}

// Turns the segments' shares into the state that each of them starts from, in the
// order of the walk: X = init, then X = D^rows X + share; and writes the last one. A
// thread takes one element.
template <bool kBack>
__global__ void __launch_bounds__(kLinThreads) lin_scan_kernel(const LinParams p) {
    const int size = p.DK * p.DV, blocks = size / kLinThreads;
    const int bh = blockIdx.x / blocks, b = bh / p.Hkv, h = bh % p.Hkv, x = blockIdx.x % blocks * kLinThreads + threadIdx.x;
    const int s0 = lin_seg_start(p, b);
    if (s0 < 0 || s0 >= p.segments) return;
    const Segment g = segment_at(p, s0);
    if (g.b != b) return;   // (offsets that do not ascend)
    const int count = min(max(1, (g.n + p.seg_rows - 1) / p.seg_rows), p.segments - s0);
    float X = 0.f;
    if (p.init) X = p.init_mul * p.init[(long)bh * size + (p.init_trans ? x % p.DV * p.DK + x / p.DV : x)];
    const float l2 = log2_decay(p, h), whole = decay_pow(l2, p.seg_rows);
    const int rest = g.n - (count - 1) * p.seg_rows;   // rows of the segment that ends the sequence
    const float part = decay_pow(l2, rest);
    float* at = p.states + ((long)s0 * p.Hkv + h) * size + x;
    const long step = (long)p.Hkv * size;
    constexpr int kAhead = 8;
    for (int i = 0; i < count; i += kAhead) {   // (step i of the walk)
        float y[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int s = kBack ? count - 1 - i - k : i + k;
            const bool in = i + k < count && (p.final || i + k < count - 1) && g.n > 0;
            y[k] = in ? at[s * step] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i + k >= count) break;
            const int s = kBack ? count - 1 - i - k : i + k;
            at[s * step] = X;
            X = fmaf(X, s == count - 1 ? part : whole, y[k]);
        }
    }
    if (p.final) p.final[(long)bh * size + x] = X * p.final_mul;
}

template <int DK>
struct OutSmem {
    static constexpr int kA = kC * DK * 2, kBC = kA + kPanel;
    static constexpr int kBCOff = 2 * kA, kX = kBCOff + 2 * kBC, kP = kX + DK * 128, kTables = kP + kPanel,
                         kBytes = kTables + (int)sizeof(Tables);
};

// The outputs of a segment: 64 tokens at a time, 64 of the DV columns per CTA.
// kBack: one a and out for the group, b and c per query head; else the reverse.
// Warps: P and out in tiles of 16 rows (warp % 4) x 32 columns (warp / 4), the
// state as in update_state.
template <int DK, bool kBack>
__global__ void __launch_bounds__(kLinThreads, DK <= 128 ? 2 : 1) lin_out_kernel(const LinParams p) {
    using Lay = OutSmem<DK>;
    constexpr int MT = DK / 64;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t base = smem_addr(smem);
    Tables* tab = reinterpret_cast<Tables*>(smem + Lay::kTables);
    const int nt = p.DV >> 6, tile = blockIdx.x % nt, h = blockIdx.x / nt % p.Hkv, s = blockIdx.x / nt / p.Hkv;
    const Segment g = segment_at(p, s);
    if (!g.live || g.r0 == g.r1) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, t4 = lane & 3;
    const int per = p.per, chunks = (g.r1 - g.r0 + kC - 1) / kC, items = chunks * per;
    const int i0 = (warp & 3) * 16, j0 = (warp >> 2) * 32;   // this warp's rows and columns
    auto row_of = [&](int chunk) { return g.r0 + (kBack ? chunks - 1 - chunk : chunk) * kC; };
    auto issue = [&](int it) {
        if (it < items) {
            const int chunk = it / per, x = it - chunk * per, r = row_of(chunk), head = h * per + x;
            const uint32_t a_at = base + ((kBack ? chunk : it) & 1) * Lay::kA;
            const uint32_t b_at = base + Lay::kBCOff + ((kBack ? it : chunk) & 1) * Lay::kBC;
            if (!kBack || x == 0) load_tile(a_at, p.a + (long)(kBack ? h : head) * DK, p.a_stride, DK, g, r);
            if (kBack || x == 0) {
                const long hb = kBack ? head : h;
                load_tile(b_at, p.b + hb * DK, p.b_stride, DK, g, r);
                load_tile(b_at + Lay::kA, p.c + hb * p.DV + tile * 64, p.c_stride, 64, g, r);
            }
        }
        copy_commit();
    };
    issue(0);
    fill_tables<kBack>(tab, log2_decay(p, h));
    float X[MT][4][4];
    {
        const float* src = lin_state_src(p, s, g.b, h);
        const bool trans = p.split() ? p.states_trans : p.init_trans;
        const float mul = p.split() ? 1.f : p.init_mul;
        each_pair<MT>(X, [&](int row, int col, float& x0, float& x1) {
            col += tile * 64;
            if (!src) {
                x0 = x1 = 0.f;
            } else if (trans) {
                x0 = mul * src[(long)col * DK + row];
                x1 = mul * src[(long)(col + 1) * DK + row];
            } else {
                const float2 y = *reinterpret_cast<const float2*>(src + (long)row * p.DV + col);
                x0 = mul * y.x;
                x1 = mul * y.y;
            }
        });
    }
    float acc[4][4];
    for (int it = 0; it < items; ++it) {
        const int chunk = it / per, x = it - chunk * per, r0 = row_of(chunk), n = min(kC, g.r1 - r0);
        const uint32_t a_at = base + ((kBack ? chunk : it) & 1) * Lay::kA;
        const uint32_t b_at = base + Lay::kBCOff + ((kBack ? it : chunk) & 1) * Lay::kBC, c_at = b_at + Lay::kA;
        const uint32_t x_at = base + Lay::kX, p_at = base + Lay::kP;
        copy_wait0();
        __syncthreads();   // this item's tiles are there; everyone is done with the one before
        issue(it + 1);
        if (x == 0)
            each_pair<MT>(X, [&](int row, int col, float x0, float x1) {
                *reinterpret_cast<uint32_t*>(smem + Lay::kX + row * 128 + (((col >> 3) ^ (row & 7)) << 4) + (col & 7) * 2) =
                    pack_bf16x2(x0, x1);
            });
        {   // P: rows i0 .. + 15, columns j0 .. + 31 (nothing on the far side of the diagonal)
            float P[4][4] = {};
            if (kBack ? j0 + 31 >= i0 : j0 <= i0 + 15) {
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks) {
                    uint32_t af[4];
                    ldsm4(tile_at(a_at, i0 + (lane & 15), ks * 16 + (lane >> 4) * 8), af);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        uint32_t bf[4];
                        ldsm4(tile_at(b_at, j0 + y * 16 + (lane & 7) + ((lane >> 4) << 3), ks * 16 + ((lane >> 3) & 1) * 8), bf);
                        mma_bf16(P[2 * y], af, bf[0], bf[1]);
                        mma_bf16(P[2 * y + 1], af, bf[2], bf[3]);
                    }
                }
            }
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int i = i0 + g8 + 8 * z, j = j0 + y * 8 + 2 * t4;
                    const int gap = kBack ? j - i : i - j, next = kBack ? gap + 1 : gap - 1;   // of columns j and j + 1
                    const float p0 = gap >= 0 ? P[y][2 * z] * tab->pow[gap] : 0.f;
                    const float p1 = next >= 0 ? P[y][2 * z + 1] * tab->pow[next] : 0.f;
                    *reinterpret_cast<uint32_t*>(smem + Lay::kP + i * 128 + (((j >> 3) ^ (i & 7)) << 4) + (j & 7) * 2) =
                        pack_bf16x2(p0, p1);
                }
        }
        __syncthreads();
        if (!kBack || x == 0) {   // what the state gives: a X
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int z = 0; z < 4; ++z) acc[y][z] = 0.f;
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks) {
                uint32_t af[4];
                ldsm4(tile_at(a_at, i0 + (lane & 15), ks * 16 + (lane >> 4) * 8), af);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t bf[4];
                    ldsm4t(tile_at(x_at, ks * 16 + (lane & 15), j0 + y * 16 + (lane >> 4) * 8), bf);
                    mma_bf16(acc[2 * y], af, bf[0], bf[1]);
                    mma_bf16(acc[2 * y + 1], af, bf[2], bf[3]);
                }
            }
            const int i = i0 + g8;
            const float f0 = tab->pow[kBack ? max(n - 1 - i, 0) : i + 1], f1 = tab->pow[kBack ? max(n - 9 - i, 0) : i + 9];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                acc[y][0] *= f0;
                acc[y][1] *= f0;
                acc[y][2] *= f1;
                acc[y][3] *= f1;
            }
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {   // P c, tokens up to (backwards: from) the rows' own
            if (kBack ? ks * 16 + 15 < i0 : ks * 16 > i0) continue;
            uint32_t af[4];
            ldsm4(tile_at(p_at, i0 + (lane & 15), ks * 16 + (lane >> 4) * 8), af);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t bf[4];
                ldsm4t(tile_at(c_at, ks * 16 + (lane & 15), j0 + y * 16 + (lane >> 4) * 8), bf);
                mma_bf16(acc[2 * y], af, bf[0], bf[1]);
                mma_bf16(acc[2 * y + 1], af, bf[2], bf[3]);
            }
        }
        if (!kBack || x == per - 1) {
            const long heads = kBack ? p.Hkv : (long)p.Hkv * per;
            __nv_bfloat16* out = p.out + (kBack ? h : (long)h * per + x) * p.DV + tile * 64 + j0 + 2 * t4;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int i = i0 + g8 + 8 * z;
                if (i >= n) continue;
                const long t = g.q0 + r0 + i;
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    *reinterpret_cast<uint32_t*>(out + t * heads * p.DV + y * 8) =
                        pack_bf16x2(acc[y][2 * z] * p.out_mul, acc[y][2 * z + 1] * p.out_mul);
            }
        }
        if (chunk < chunks - 1 && (kBack || x == per - 1))
            update_state<MT, 1>(X, b_at, c_at, weights<kBack>(tab, n), kBack && x > 0 ? 1.f : tab->pow[n]);
    }
    copy_wait0();
}

template <int DK, bool kBack>
cudaError_t launch_dk(const LinParams& p, bool state, cudaStream_t stream) {
    static std::atomic<unsigned long long> allowed[2];
    const unsigned ctas = (unsigned)((long)p.segments * p.Hkv * (p.DV / 64));
    cudaError_t e;
    if (state) {
        if ((e = allow_smem(lin_state_kernel<DK, kBack>, StateSmem<DK>::kBytes, allowed[0])) != cudaSuccess) return e;
        lin_state_kernel<DK, kBack><<<ctas, kLinThreads, StateSmem<DK>::kBytes, stream>>>(p);
    } else {
        if ((e = allow_smem(lin_out_kernel<DK, kBack>, OutSmem<DK>::kBytes, allowed[1])) != cudaSuccess) return e;
        lin_out_kernel<DK, kBack><<<ctas, kLinThreads, OutSmem<DK>::kBytes, stream>>>(p);
    }
    return cudaGetLastError();
}
template <bool kBack>
cudaError_t launch_sync(const LinParams& p, bool state, cudaStream_t stream) {
    if (p.DK == 64) return launch_dk<64, kBack>(p, state, stream);
    if (p.DK == 128) return launch_dk<128, kBack>(p, state, stream);
    if (p.DK == 192) return launch_dk<192, kBack>(p, state, stream);
    if (p.DK == 256) return launch_dk<256, kBack>(p, state, stream);
    return cudaErrorInvalidValue;
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

LinPlan lin_plan(int B, int Hkv, int L, bool packed, int d, int dv) {
    constexpr int kUnit = 128;   // a chunk of the tcgen05 kernels, two of the others
    const long units = packed ? (long)L / kUnit + 1 : (long)B * ((L + kUnit - 1) / kUnit);
    const long tiles = (long)Hkv * ((d < dv ? d : dv) / 64);
    const long longest = (L + kUnit - 1) / kUnit;   // units that a sequence can have
    long seg = (units * tiles + 1215) / 1216;
    if (seg < 2) seg = 2;
    if (!packed && (long)B * tiles >= 304) seg = longest;
    if (seg > longest) seg = longest;
    if (seg < 1) seg = 1;
    LinPlan r;
    r.split = seg < longest;
    r.seg_rows = (int)(seg * kUnit);
    r.segments = packed ? L / r.seg_rows + B : B * (int)(L > 0 ? ((long)L + r.seg_rows - 1) / r.seg_rows : 1);
    return r;
}

cudaError_t launch_linear_states(const LinParams& p, const LinMaps& maps, bool back, int num_sms, cudaStream_t stream) {
    if (!p.split()) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    if (p.total > 0)
        e = lin_on_tc(p.DK, p.DV) ? launch_linear_state_tc(p, maps, back, num_sms, stream)
                                  : back ? launch_sync<true>(p, true, stream) : launch_sync<false>(p, true, stream);
    if (e != cudaSuccess) return e;
    const unsigned blocks = (unsigned)((long)p.DK * p.DV / kLinThreads * p.B * p.Hkv);
    if (back) lin_scan_kernel<true><<<blocks, kLinThreads, 0, stream>>>(p);
    else lin_scan_kernel<false><<<blocks, kLinThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_linear_out(const LinParams& p, const LinMaps& maps, bool back, int num_sms, cudaStream_t stream) {
    if (p.total == 0) return cudaSuccess;
    return lin_on_tc(p.DK, p.DV) ? launch_linear_out_tc(p, maps, back, num_sms, stream)
                                 : back ? launch_sync<true>(p, false, stream) : launch_sync<false>(p, false, stream);
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
