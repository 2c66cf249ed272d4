// The 4-bit key/value cache: its layout and the launchers of its kernels.
//
// Pages of 64 tokens. Of one page and key/value head, the channels (d of K, dv
// of V) split into groups of 64; a group holds 32 bytes of codes per token
// (channel 2 i in the low half of byte i) and one (scale, minimum) pair of bf16
// per token: a code c stands for scale * c + minimum. Group-major, so that one
// page of one head is one contiguous block per tensor (one bulk copy) and a
// warp's fragment loads from shared memory touch consecutive 32-byte rows:
//   codes  [pages][Hkv][groups][64][32] bytes
//   params [pages][Hkv][groups][64][2]  bf16
#pragma once

#include <atomic>

#include "kernels.h"
#include "mask.cuh"
#include "ptx.cuh"

namespace attn {

constexpr int kPage = 64;            // tokens of a page
constexpr int kKv4Group = 64;        // channels that share a (scale, minimum) pair
constexpr int kKv4MaxBatch = 1024;   // sequences per call (the work prefix lives in shared memory)

struct Kv4Cache {
    unsigned char* k_codes;
    unsigned int* k_params;    // scale in the low half, minimum in the high half
    unsigned char* v_codes;
    unsigned int* v_params;
    int n_pages, Hkv, d, dv;
};

// Which rows belong to which sequence and where its keys are: packed (cu, B + 1
// offsets) or dense (cu null, `rows` rows per sequence). Sequence b's rows are
// the last ones of its lens[b] cached tokens.
struct Kv4Batch {
    const int* table;   // [B][width] page ids
    const int* lens;    // [B] tokens in the cache, the new ones included
    const int* cu;      // row offsets, or null
    int B, width, rows, total;   // total: packed rows (B * rows when dense)
};

struct Kv4FwdParams {
    static constexpr bool kKeepsNan = false;   // paged_work.cuh
    Kv4Cache c;
    Kv4Batch s;
    const __nv_bfloat16* q;
    long q_stride;             // elements between tokens of q
    __nv_bfloat16* o;
    float* lse;
    float* key_weights;        // [B][Hkv][weight_stride], or null
    long weight_stride;
    float weight_decay;
    int H, group;
    int win_left, win_right, sinks;
    float scale_log2;
    int* prefix;               // workspace: B + 1 work offsets, then the units per CTA
    float* part_ml;            // workspace: (max, sum) of partial rows
    float* part_o;             // workspace: partial rows
    float* scores;             // workspace: [total * H][width * 64] log2-unit scores (key weights only)
    int* status;
};

// Row blocks: a CTA holds 8 * kv4_row_tiles(...) (query, head-of-the-group) rows
// of one key/value head at once. Blocks of 16 rows when an average sequence has
// more than 8 (32 sequences, group 4, 1 to 16 tokens each, d = 128: 111 us, 123 with
// 8 rows at once); blocks of 32 took so many registers from the number of warps
// that they lost more than they saved by reading the codes less often.
inline int kv4_row_tiles(int group, int B, int total) {
    const long rows = B > 0 ? (long)group * ((total + B - 1) / B) : group;
    return rows <= 8 ? 1 : 2;
}
constexpr int kKv4MaxCtas = 640;
// The work list counts (row block, two pages) units in an int. A batch of rows
// that follow one another stays below this (checked on the host); offsets that
// run backwards can make sequences share rows and pass it: such a call does no work.
constexpr long kKv4MostUnits = 2000000000;
// Workspace parts in bytes.
inline size_t kv4_prefix_bytes() { return (kKv4MaxBatch + 8) * sizeof(int); }
inline size_t kv4_ml_bytes(int nr) { return (size_t)kKv4MaxCtas * 2 * nr * 8 * 2 * sizeof(float); }
inline size_t kv4_part_bytes(int nr, int dv) { return (size_t)kKv4MaxCtas * 2 * nr * 8 * dv * sizeof(float); }

cudaError_t launch_kv4_fwd(const Kv4FwdParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_kv4_append(const Kv4Cache& c, const Kv4Batch& s, const __nv_bfloat16* k, const __nv_bfloat16* v,
                              long k_stride, long v_stride, int* status, int num_sms, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4Cache& c, const Kv4Batch& s, __nv_bfloat16* k, __nv_bfloat16* v, int* status,
                            int num_sms, cudaStream_t stream);
struct Kv4EvictParams {
    Kv4Cache c;
    const int* table;
    const int* lens;
    const float* weights;      // [B][Hkv][weight_stride]
    const int* new_table;
    int* new_lens;
    int* kept;                 // [B][Hkv][budget]
    float* new_weights;        // [B][Hkv][new_stride]
    long weight_stride, new_stride;
    int B, width, new_width, budget, sinks, recent;
    int* status;
};
cudaError_t launch_kv4_evict(const Kv4EvictParams& p, cudaStream_t stream);

// Allow a kernel `bytes` of dynamic shared memory, asked for once per device
// (the attribute stays with the kernel; setting it on every call costs a
// small call's launch a microsecond).
template <class... Args>
cudaError_t allow_smem(void (*kernel)(Args...), int bytes, std::atomic<unsigned long long>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
    if (bit & done.load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

#ifdef __CUDACC__
// A sequence of a batch: rows [q0, q0 + nq) and lk cached tokens. Lengths out
// of range are clamped (and reported by the caller through the status word).
struct Kv4Seq {
    int q0, nq, lk;
    bool bad;
};
__device__ __forceinline__ Kv4Seq kv4_seq(const Kv4Batch& s, int b) {
    Kv4Seq r;
    r.q0 = s.cu ? s.cu[b] : b * s.rows;
    r.nq = s.cu ? s.cu[b + 1] - r.q0 : s.rows;
    r.lk = s.lens[b];
    r.bad = false;
    if (r.q0 < 0 || r.nq < 0 || r.q0 > s.total - r.nq) {
        r.bad = true;
        r.q0 = r.nq = 0;
    }
    if (r.lk < 0 || r.lk > s.width * kPage) {
        r.bad = true;
        r.lk = r.lk < 0 ? 0 : s.width * kPage;
    }
    return r;
}
// Sequence of packed row t (the last b with start(b) <= t), or -1 for a row past the last sequence.
__device__ __forceinline__ int kv4_seq_of_row(const Kv4Batch& s, int t) {
    if (!s.cu) return t / s.rows;
    if (t >= s.cu[s.B] || t < s.cu[0]) return -1;
    int lo = 0, hi = s.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return t < s.cu[lo + 1] ? lo : -1;   // (offsets that do not ascend: no sequence)
}
__device__ __forceinline__ void bad_page(int* status) { atomicCAS(status, kStatusOk, kStatusBadPage); }

// Where a packed row lives: its page and slot, or page -1: nowhere (out of
// range, reported), -2: no such row (past the last sequence), -3: before the
// sequence's first token (a padded dense batch).
struct RowPlace {
    int page, slot;
};
__device__ __forceinline__ RowPlace place_of(int n_pages, const Kv4Batch& s, int t, int* status) {
    RowPlace r{-2, 0};
    if (t >= s.total) return r;
    const int b = kv4_seq_of_row(s, t);
    if (b < 0) return r;
    const Kv4Seq q = kv4_seq(s, b);
    const int slot = q.lk - q.nq + t - q.q0;
    r.page = -1;
    if (!q.bad && slot < 0) r.page = -3;
    if (!q.bad && slot >= 0) {
        r.slot = slot % kPage;
        r.page = s.table[(long)b * s.width + slot / kPage];
        if (r.page < 0 || r.page >= n_pages) r.page = -1;
    }
    if (r.page == -1) bad_page(status);
    return r;
}
#endif

}  // namespace attn
