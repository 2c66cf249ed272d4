// The paged key/value cache in bf16 or 8 bits: its layout and the launchers of its kernels.
//
// Pages of 64 tokens, [pages][Hkv][64][channels] for K (d) and V (dv), in bf16 or in
// e4m3. With e4m3, bytes e [pages][Hkv][64] give each token and head a scale of
// 2^(e - 127) for its codes, e from 1 up (255: the row held an infinity or a NaN and is
// NaN throughout, whatever its codes are; an append makes them 0). A power of two costs a code that has an exponent of its own
// nothing, and makes quantising exact up to the one rounding of the code.
// Batches (tables, lengths, rows) are those of the 4-bit cache.
#pragma once

#include "kv4.h"

namespace attn {

struct PagedCache {
    unsigned char* k;          // bf16 or e4m3 rows, by `bits`
    unsigned char* v;
    unsigned char* k_scales;   // (8 bits)
    unsigned char* v_scales;
    int n_pages, Hkv, d, dv;
};

struct PagedFwdParams {
    static constexpr bool kKeepsNan = true;   // paged_work.cuh
    PagedCache c;
    Kv4Batch s;
    const __nv_bfloat16* q;
    long q_stride;             // elements between tokens of q
    __nv_bfloat16* o;
    float* lse;
    int H, group;
    int win_left, win_right, sinks;
    float scale_log2;
    int* prefix;               // workspace: as in Kv4FwdParams
    float* part_ml;
    float* part_o;
    int* status;
};

// Tiles of 8 (query, head-of-the-group) rows that a CTA holds at once: four when an average sequence has more than 8 rows
// (32 sequences, group 4, 1 to 16 tokens, bf16, d = 128: 188 us in blocks of two tiles, 143 of four).
inline int paged_row_tiles(int group, int B, int total) { return kv4_row_tiles(group, B, total) == 1 ? 1 : 4; }

#ifdef __CUDACC__
__device__ __forceinline__ float paged_scale(uint32_t e) { return __uint_as_float(e == 255 ? 0x7fc00000u : e << 23); }
#endif

cudaError_t launch_paged_append(const PagedCache& c, bool codes, const Kv4Batch& s, const __nv_bfloat16* k,
                                const __nv_bfloat16* v, long k_stride, long v_stride, int* status, int num_sms,
                                cudaStream_t stream);
cudaError_t launch_paged_read(const PagedCache& c, bool codes, const Kv4Batch& s, __nv_bfloat16* k, __nv_bfloat16* v,
                              int* status, int num_sms, cudaStream_t stream);
cudaError_t launch_paged_fwd(const PagedFwdParams& p, bool codes, int num_sms, cudaStream_t stream);

}  // namespace attn
