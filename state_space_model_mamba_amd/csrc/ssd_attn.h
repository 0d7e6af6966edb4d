// Internal launchers of the linear-attention and softmax-attention entry
// points (not part of the C ABI; see include/ssd.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace ssd {

// Lets `kernel` be launched with `bytes` of dynamic LDS, once per device (`done`:
// a bit per device, one word for each kernel).
inline hipError_t allow_lds(const void *kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
    if ((done.load(std::memory_order_acquire) & bit) != 0)
        return hipSuccess;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess)
        done.fetch_or(bit, std::memory_order_release);
    return e;
}

// One packed sequence of an attention launch.
struct AttnSeq {
    int64_t q0, k0;   // first query / key row
    int32_t lq, lk;   // rows
};

// Causal attention of packed prompts: q, o [*, Hq, D], k, v [*, Hkv, D], rows
// `*_stride` elements apart (o contiguous).  seqs is a host array.
hipError_t launch_attn_prefill(int bf16, int64_t nseq, const AttnSeq *seqs, int64_t Hq, int64_t Hkv,
                               int64_t D, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                               float scale, const void *q, const void *k, const void *v, void *o,
                               hipStream_t s);

// One decode token per sequence over a padded cache [B, M, Hkv, D].
int64_t attn_decode_splits(int64_t B, int64_t M, int64_t Hq, int64_t Hkv);
size_t attn_decode_workspace(int64_t B, int64_t M, int64_t Hq, int64_t Hkv, int64_t D);
hipError_t launch_attn_decode(int bf16, int64_t B, int64_t M, int64_t Hq, int64_t Hkv, int64_t D,
                              int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                              const void *q, const void *k, const void *v, void *k_cache,
                              void *v_cache, const int32_t *lengths, void *o, void *ws,
                              hipStream_t s);

// Linear attention with one decay per head over packed sequences; sequence i is
// rows tok[i] .. tok[i] + len[i] - 1 of q, k [*, Hk, dk] and v, o [*, Hv, dv].
struct LinSeq {
    int64_t tok;
    int64_t len;
};
struct LinPlan {
    int64_t seg_tokens;   // tokens per segment (a multiple of the tile), same for all sequences
    int64_t nslot;        // segments whose end state is kept, over all sequences
    int cols;             // value columns per work-group
    size_t ws_bytes;
};
LinPlan plan_linattn(int bf16, int64_t nseq, const LinSeq *seqs, int64_t Hk, int64_t Hv, int64_t dk,
                     int64_t dv);
hipError_t launch_linattn_scan(int bf16, const LinPlan &plan, int64_t nseq, const LinSeq *seqs,
                               int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t q_stride,
                               int64_t k_stride, int64_t v_stride, float scale, const void *q,
                               const void *k, const void *v, const float *log_decay,
                               const float *init, void *o, float *fin, void *ws, hipStream_t s);
hipError_t launch_linattn_decode(int bf16, int64_t B, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv,
                                 int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                                 const void *q, const void *k, const void *v,
                                 const float *log_decay, float *state, void *o, hipStream_t s);

}  // namespace ssd
