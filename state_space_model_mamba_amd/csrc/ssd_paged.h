// Internal launchers of the paged-cache entry points and of the norm and rotation of
// queries and keys (not part of the C ABI; see include/ssd.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

// Pages [num_pages, Hkv, page rows, D] of keys and values in the input type, or in 4
// bits ([.., D / 2] bytes with scales [.., D / 64] of a step and a least value in half
// precision, one dword each); row r of sequence b is line r % (1 << shift) of page
// table[b * max_pages + (r >> shift)].
struct PagedCache {
    void *k, *v;
    uint32_t *ks, *vs;        // NULL: the input type
    const int32_t *table;
    int64_t num_pages, max_pages;
    int shift;
};

// Norm and rotation of queries and keys (any of it may be absent).
struct QkTurn {
    const float *inv_freq, *q_weight, *k_weight;   // NULL: not rotated / not normed
    const int32_t *positions;                      // one per token; NULL: its row in the cache
    int rot;                                       // rotated values of a head
    int next;                                      // pairs (2 i, 2 i + 1) instead of (i, i + rot / 2)
    float eps;
};

// Rows of q (q_heads), k and v (kv_heads) to q_out, k_out (either may be NULL) and, with
// a cache, the keys and values to rows lengths[b] + j of it.  cu: host offsets of the
// sequences' tokens, NULL for one token each.
struct TurnRows {
    const void *q, *k, *v;
    void *q_out, *k_out;
    int64_t q_stride, k_stride, v_stride, qo_stride, ko_stride;
    int64_t rows, Hq, Hkv, D;
};
hipError_t launch_qk_turn(int bf16, const TurnRows &r, const QkTurn &turn, hipStream_t s);
hipError_t launch_paged_append(int bf16, int64_t batch, const int64_t *cu, const TurnRows &r,
                               const QkTurn &turn, const PagedCache &cache, const int32_t *lengths,
                               hipStream_t s);

// Rows starts[b] .. (0 ..; NULL) of the sequences' keys and values to packed rows cu[b] ..
// cu[b + 1] - 1 of k and v [*, Hkv, D].  starts and cu are host arrays.
hipError_t launch_paged_gather(int bf16, int64_t batch, const int64_t *cu, const int64_t *starts,
                               int64_t Hkv, int64_t D, const PagedCache &cache, void *k, void *v,
                               hipStream_t s);

// One query token per sequence over rows 0 .. lengths[b] of the cache.
size_t paged_decode_workspace(int bf16, int q4, int64_t B, int64_t Hq, int64_t Hkv, int64_t D);
hipError_t launch_paged_decode(int bf16, int64_t B, int64_t Hq, int64_t Hkv, int64_t D,
                               int64_t q_stride, float scale, const void *q, const PagedCache &cache,
                               const int32_t *lengths, void *o, void *ws, hipStream_t s);

}  // namespace ssd
