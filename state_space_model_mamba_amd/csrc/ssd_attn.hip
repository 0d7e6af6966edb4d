// Causal softmax attention on gfx950: packed prompts (prefill) and one decode
// token per sequence over a padded key/value cache.
//
// For query token t of a sequence with lq queries and lk keys, query head h and
// key head h / (Hq / Hkv), keys s <= t + lk - lq being visible:
//     a_s = scale q_t . k_s,   o_t = sum_s exp(a_s - m) v_s / sum_s exp(a_s - m)
// for any m; a row that sees no key is 0.  One pass over the keys carries
// (m, l = sum exp(a_s - m), acc = sum exp(a_s - m) v_s) per row in fp32: when m
// grows by more than kSlack (log2 units) l and acc are rescaled, otherwise the
// old m is kept -- the result does not depend on m, and exp(a - m) <= 2^kSlack
// stays far from overflow -- so that the rescaling pass over acc is rare.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ssd_attn.h"
#include "ssd_mma.h"

namespace ssd {
namespace {

using namespace mx;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;
constexpr float kNoMax = -3e38f;   // m before the first visible key (finite: m - m is 0)
// |scale| log2 e.  A scale of 0 weights all visible keys alike; it is kept off 0 so
// that a masked score (-inf) times it stays -inf, and finite so that a score of 0 times
// it stays 0.
float score_factor(float scale)
{
    return std::clamp(std::abs(scale) * kLog2e, 1.17549435e-38f, 3.40282347e38f);
}

// s c - m, the product rounded before the difference as it is in m: for the largest
// score of a row exactly 0 however large it is.  (Fused, the rounding of m remains;
// the row's weights have it in common, but past 2^30 it overflows the exponential.)
__device__ __forceinline__ float below_max(float s, float c, float m)
{
#pragma clang fp contract(off)
    return s * c - m;
}

// A 32-key tile in a wave's own LDS, for 32 rows (score columns): updates (m, l,
// acc).  Keys from `see` (per lane) on are masked if `masked` (wave-uniform).  The
// probabilities, unnormalised, are the second product's operand as kTerms numbers of
// its type: in bf16 one is off by up to 2^-8, as the output's own rounding, two by up
// to 2^-17.  (The sum l takes them unrounded.)
template <typename T, int D, int kTerms>
__device__ __forceinline__ void tile32(const unsigned char *Kt, const unsigned char *Vt,
                                       const typename Piece<T>::V (&qf)[Tile<T, D>::kPieces], bool masked,
                                       int see, float c,
                                       int lane, float &m, float &l, f32x16 (&acc)[D / 32])
{
    typedef Tile<T, D> TL;
    constexpr int DB = D / 32, PC = 16 / Piece<T>::E;
    const int cl = lane & 31, hh = lane >> 5;
    f32x16 s = {};
#pragma unroll
    for (int p = 0; p < TL::kPieces; ++p)
        s = mma(TL::row_nat(Kt, cl, p, hh), qf[p], s);
    if (masked) {
        const int lim = see - 4 * hh;
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (8 * (r >> 2) + (r & 3) >= lim)
                s[r] = -__builtin_inff();
    }
    float t = s[0];
#pragma unroll
    for (int r = 1; r < 16; ++r)
        t = fmaxf(t, s[r]);
    t = half_max(t) * c;
    if (__any(t > m + kSlack)) {
        const float mn = fmaxf(m, t), al = exp2_fast(m - mn);
        m = mn;
        l *= al;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[d][r] *= al;
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        s[r] = exp2_fast(below_max(s[r], c, m));
        l += s[r];
    }
#pragma unroll
    for (int p = 0; p < PC; ++p) {
        typename Piece<T>::V pf[kTerms];
#pragma unroll
        for (int i = 0; i < kTerms; ++i) {
            pf[i] = acc_piece(s, p, (const T *)nullptr);
            if (i + 1 < kTerms)
#pragma unroll
                for (int e = 0; e < Piece<T>::E; ++e)
                    s[Piece<T>::E * p + e] -= (float)pf[i][e];
        }
#pragma unroll
        for (int d = 0; d < DB; ++d) {
            const typename Piece<T>::V v = TL::col_acc(Vt, p, 32 * d, lane);
#pragma unroll
            for (int i = 0; i < kTerms; ++i)
                acc[d] = mma(v, pf[i], acc[d]);
        }
    }
}

// The LDS of kernels whose waves work on tiles of their own: two slots of a K and a
// V tile per wave, as many waves as fit.
template <typename T, int D> struct WaveTiles {
    static constexpr int kPitch = Tile<T, D>::kPitch;
    static constexpr int kWaves = kPitch <= 256 ? 4 : kPitch == 512 ? 2 : 1;
    static constexpr int kTileBytes = 32 * kPitch;
    static constexpr unsigned kWaveSmem = 4u * kTileBytes;
    static constexpr unsigned kSmem = kWaves * kWaveSmem;
};

// Joins the waves' results for the same 32 rows: each scales its sums to the common
// m and leaves them in its part of the LDS as [row][D]; then out(i, v, m, l) is
// called with four consecutive sums of the work-group for each i = row D + d.
template <typename T, int D, typename Out>
__device__ __forceinline__ void join_waves(unsigned char *smem, float (&sm)[WaveTiles<T, D>::kWaves][32],
                                           float (&sl)[WaveTiles<T, D>::kWaves][32], int w, int lane, int rows,
                                           float m, float l, const f32x16 (&acc)[D / 32], Out out)
{
    typedef WaveTiles<T, D> GM;
    constexpr int NW = GM::kWaves, DB = D / 32;
    const int cl = lane & 31, hh = lane >> 5;
    l = half_sum(l);
    if (hh == 0) {
        sm[w][cl] = m;
        sl[w][cl] = l;
    }
    __syncthreads();
    float mt = sm[0][cl];
#pragma unroll
    for (int i = 1; i < NW; ++i)
        mt = fmaxf(mt, sm[i][cl]);
    const float f = exp2_fast(m - mt);
    float *wp = reinterpret_cast<float *>(smem + w * GM::kWaveSmem);
    if (cl < rows)
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<f32x4 *>(wp + cl * D + 32 * d + 8 * g + 4 * hh) =
                    f32x4{acc[d][4 * g] * f, acc[d][4 * g + 1] * f, acc[d][4 * g + 2] * f,
                          acc[d][4 * g + 3] * f};
    __syncthreads();
    for (int i = 4 * (64 * w + lane); i < rows * D; i += 4 * 64 * NW) {
        const int row = i / D;
        f32x4 v = *reinterpret_cast<const f32x4 *>(smem + i * 4);
#pragma unroll
        for (int j = 1; j < NW; ++j)
            v += *reinterpret_cast<const f32x4 *>(smem + j * GM::kWaveSmem + i * 4);
        float mr = sm[0][row];
#pragma unroll
        for (int j = 1; j < NW; ++j)
            mr = fmaxf(mr, sm[j][row]);
        float lr = 0.f;
#pragma unroll
        for (int j = 0; j < NW; ++j)
            lr += sl[j][row] * exp2_fast(sm[j][row] - mr);
        out(i, v, mr, lr);
    }
}

// ---------------------------------------------------------------------------
// Prefill
// ---------------------------------------------------------------------------
// Rows of a sequence are its (token, head of the group) pairs, token-major, so
// that all query heads of a key head share its K and V tiles and short prompts
// still fill the 32-row blocks.  A work-group takes kRows consecutive rows, 32 per
// wave; the scores are formed transposed (keys x rows): a lane then holds one row,
// its statistics are per-lane scalars, and the probabilities are the second
// product's operand as they stand.  K and V tiles go from memory straight into two
// LDS slots, a tile ahead.
//
// Bound by the matrix and vector units: one prompt of 8192 tokens, 32 heads over 8
// of 128 in bf16, takes 500 - 540 us, 1.02 - 1.10 PFLOP/s; a large library product
// (8192 x 8192 x 8192) reaches 1.20 on the same card.  The matrix units are busy 48%
// of the time and the vector units 44%.  Tried and no faster: the eight waves'
// pairs staggered by half a tile (554 us), 64 rows per wave with the two blocks'
// steps interleaved in one stream (729 us: registers spill), raised priority
// around the products (545), the K operands of a tile read together (510).
struct SeqTab {
    static constexpr int kMax = 120;          // sequences per launch (kernel arguments: 4 KB)
    AttnSeq seq[kMax];
    int32_t pre[128];                         // first work item of each sequence; then INT32_MAX
};

struct PrefillArgs {
    SeqTab tab;
    const void *q, *k, *v;
    void *o;
    int64_t q_stride, k_stride, v_stride;     // elements between rows
    int Hq, Hkv, grp;
    float c;                                  // |scale| log2 e
    int neg;                                  // scale < 0: the queries' signs are flipped
};

typedef const __attribute__((address_space(4))) PrefillArgs *PrefillArgsPtr;

template <typename T> __device__ __forceinline__ typename Piece<T>::V flip(typename Piece<T>::V v);
template <> __device__ __forceinline__ bf16x8 flip<__bf16>(bf16x8 v)
{
    u32x4 u = __builtin_bit_cast(u32x4, v);
    return __builtin_bit_cast(bf16x8, u ^ 0x80008000u);
}
template <> __device__ __forceinline__ f32x4 flip<float>(f32x4 v)
{
    return -v;
}

template <typename T, int D, int NW>
__global__ __launch_bounds__(64 * NW, D <= 128 ? 2 : 1) void attn_prefill_kernel(
    PrefillArgs args_in_kernarg)
{
    constexpr int KT = sizeof(T) == 2 ? 64 : 32;          // keys per tile
    constexpr int KB = KT / 32, DB = D / 32;
    constexpr int E = Piece<T>::E, PC = 16 / E;           // pieces per 32-key block of P
    constexpr int kRows = 32 * NW;
    typedef Tile<T, D> TL;
    typedef typename Piece<T>::V V;
    constexpr int kTileBytes = KT * TL::kPitch;
    extern __shared__ __align__(1024) unsigned char smem[];   // [2][K tile, V tile]

    const PrefillArgsPtr a = (PrefillArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    const int tid = threadIdx.x, lane = tid & 63, w = uniform_int(tid >> 6);
    const int cl = lane & 31, hh = lane >> 5;

    // heads of one row block next to each other: with 8 key heads each XCD
    // keeps one head's K and V in its L2
    const int Hkv = a->Hkv, grp = a->grp;
    const int item = (int)(blockIdx.x / (unsigned)Hkv), hk = (int)(blockIdx.x % (unsigned)Hkv);
    const int below = __popcll(__ballot(a->tab.pre[lane] <= item)) +
                      __popcll(__ballot(a->tab.pre[64 + lane] <= item));
    const int si = uniform_int(below - 1);
    const int lq = a->tab.seq[si].lq, lk = a->tab.seq[si].lk;
    const int64_t nrow = (int64_t)lq * grp;
    const int nblk = (int)((nrow + kRows - 1) / kRows);
    // the last rows see the most keys: they start first
    const int blk = nblk - 1 - (item - a->tab.pre[si]);
    const int64_t row0 = (int64_t)blk * kRows;
    const T *kp = (const T *)a->k + a->tab.seq[si].k0 * a->k_stride + (int64_t)hk * D;
    const T *vp = (const T *)a->v + a->tab.seq[si].k0 * a->v_stride + (int64_t)hk * D;

    const int64_t row = row0 + w * 32 + cl;
    const bool valid = row < nrow;
    const unsigned rr = (unsigned)(valid ? row : nrow - 1);
    const unsigned tok = rr / (unsigned)grp, head = hk * grp + rr % (unsigned)grp;
    const int64_t qt = a->tab.seq[si].q0 + tok;
    const int lim = valid ? std::max(0, lk - lq + (int)tok + 1) : 0;   // keys the lane's row sees
    V qf[TL::kPieces];
    const T *qp = (const T *)a->q + qt * a->q_stride + (int64_t)head * D;
#pragma unroll
    for (int p = 0; p < TL::kPieces; ++p) {
        qf[p] = *reinterpret_cast<const V *>(qp + (2 * p + hh) * E);
        if (a->neg)
            qf[p] = flip<T>(qf[p]);
    }
    // keys that any / every row of the wave sees, and any row of the work-group
    const int64_t wfirst = row0 + (int64_t)w * 32, wlast = std::min<int64_t>(nrow, wfirst + 32) - 1;
    const int wmax = wfirst >= nrow ? 0 : std::max(0, lk - lq + (int)((unsigned)wlast / (unsigned)grp) + 1);
    const int wmin = std::max(0, lk - lq + (int)((unsigned)wfirst / (unsigned)grp) + 1);
    const int64_t glast = std::min<int64_t>(nrow, row0 + kRows) - 1;
    const int gmax = std::max(0, lk - lq + (int)((unsigned)glast / (unsigned)grp) + 1);
    const int ntile = uniform_int((gmax + KT - 1) / KT);
    const float c = a->c;

    f32x16 acc[DB] = {};
    float m = kNoMax, l = 0.f;
    const unsigned lds0 = lds_addr(smem);
    auto issue = [&](int n) {
        const unsigned dst = lds0 + (n & 1) * 2 * kTileBytes;
        TileLoad<T, D, KT, NW>::issue(dst, kp, a->k_stride, (int64_t)n * KT, lk, w, lane);
        TileLoad<T, D, KT, NW>::issue(dst + kTileBytes, vp, a->v_stride, (int64_t)n * KT, lk, w, lane);
    };
    if (ntile > 0)
        issue(0);

    for (int n = 0; n < ntile; ++n) {
        wait_vmcnt<0>();      // this wave's share of tile n has landed
        lds_barrier();        // everyone's has, and tile n - 1 has been read
        if (n + 1 < ntile)
            issue(n + 1);
        if (n * KT >= wmax)
            continue;
        const unsigned char *Kt = smem + (n & 1) * 2 * kTileBytes, *Vt = Kt + kTileBytes;

        f32x16 s[KB] = {};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int p = 0; p < TL::kPieces; ++p)
                s[kb] = mma(TL::row_nat(Kt, kb * 32 + cl, p, hh), qf[p], s[kb]);
        if ((n + 1) * KT > wmin) {
            const int see = lim - n * KT - 4 * hh;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (32 * kb + 8 * (r >> 2) + (r & 3) >= see)
                        s[kb][r] = -__builtin_inff();
        }
        float t = s[0][0];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                t = fmaxf(t, s[kb][r]);
        t = half_max(t) * c;
        if (__any(t > m + kSlack)) {
            const float mn = fmaxf(m, t), al = exp2_fast(m - mn);
            m = mn;
            l *= al;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[d][r] *= al;
        }
        // the exponents as one fused operation each (3% of the kernel's time), but for
        // huge scores
        float ec = c, em = m;
        if (__any(fabsf(m) > 16777216.f && m != kNoMax)) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    s[kb][r] = below_max(s[kb][r], c, m);
            ec = 1.f;
            em = 0.f;
        }
        V pf[KB * PC];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float e = exp2_fast(__builtin_fmaf(s[kb][r], ec, -em));
                l += e;
                s[kb][r] = e;
            }
            // (one operand each, as in tile32: two would be half as many matrix
            // instructions again in a kernel that they bound)
#pragma unroll
            for (int p = 0; p < PC; ++p)
                pf[kb * PC + p] = acc_piece(s[kb], p, (const T *)nullptr);
        }
#pragma unroll
        for (int p = 0; p < KB * PC; ++p)
#pragma unroll
            for (int d = 0; d < DB; ++d)
                acc[d] = mma(TL::col_acc(Vt, p, 32 * d, lane), pf[p], acc[d]);
    }

    const float tot = half_sum(l);
    const float inv = tot > 0.f ? 1.f / tot : 0.f;
    T *op = (T *)a->o + (qt * a->Hq + head) * D;
#pragma unroll
    for (int d = 0; d < DB; ++d) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
            acc[d][r] *= inv;
        store_row(op, 32 * d, hh, valid, acc[d]);
    }
}

// Few rows (short prompts, or few heads): 32 rows per work-group, the waves taking
// every kWaves-th 32-key tile of them, each with its own running (m, l, acc), joined
// at the end.  Four to eight times as many work-groups then share the chip, and each
// walks its keys in a kWaves-th of the tiles (four waves; two for rows of 512 bytes
// and one for rows of 1 KB, whose tiles fill the LDS).  Bound by each work-group's
// chain of steps: 1.3 us each at 128 in bf16, 5 at 128 in fp32, 13 at 256 in fp32 (64
// queries on 4000 keys: 40, 320 and 1670 us; figures at the rule that chooses it).
// The keys are not split over work-groups: the time grows with the prefix whatever
// the chip has free.
template <typename T, int D>
__global__ __launch_bounds__((64 * WaveTiles<T, D>::kWaves), 1) void attn_prefill_few_kernel(
    PrefillArgs args_in_kernarg)
{
    typedef WaveTiles<T, D> GM;
    typedef Tile<T, D> TL;
    typedef typename Piece<T>::V V;
    constexpr int E = Piece<T>::E, NW = GM::kWaves, DB = D / 32;
    constexpr int kLoads = 2 * TileLoad<T, D, 32, 1>::kPer;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ float sm[NW][32], sl[NW][32];
    __shared__ int64_t srow[32];

    const PrefillArgsPtr a = (PrefillArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    const int tid = threadIdx.x, lane = tid & 63, w = uniform_int(tid >> 6);
    const int cl = lane & 31, hh = lane >> 5;
    const int Hkv = a->Hkv, grp = a->grp;
    const int item = (int)(blockIdx.x / (unsigned)Hkv), hk = (int)(blockIdx.x % (unsigned)Hkv);
    const int below = __popcll(__ballot(a->tab.pre[lane] <= item)) +
                      __popcll(__ballot(a->tab.pre[64 + lane] <= item));
    const int si = uniform_int(below - 1);
    const int lq = a->tab.seq[si].lq, lk = a->tab.seq[si].lk;
    const int64_t nrow = (int64_t)lq * grp;
    const int blk = (int)((nrow + 31) / 32) - 1 - (item - a->tab.pre[si]);
    const int64_t row0 = (int64_t)blk * 32;
    const int rows = (int)std::min<int64_t>(32, nrow - row0);
    const T *kp = (const T *)a->k + a->tab.seq[si].k0 * a->k_stride + (int64_t)hk * D;
    const T *vp = (const T *)a->v + a->tab.seq[si].k0 * a->v_stride + (int64_t)hk * D;

    const unsigned rr = (unsigned)(row0 + std::min(cl, rows - 1));
    const unsigned tok = rr / (unsigned)grp, head = hk * grp + rr % (unsigned)grp;
    const int64_t qt = a->tab.seq[si].q0 + tok;
    if (w == 0 && hh == 0)
        srow[cl] = (qt * a->Hq + head) * D;
    const int lim = std::max(0, lk - lq + (int)tok + 1);
    V qf[TL::kPieces];
    const T *qp = (const T *)a->q + qt * a->q_stride + (int64_t)head * D;
#pragma unroll
    for (int p = 0; p < TL::kPieces; ++p) {
        qf[p] = *reinterpret_cast<const V *>(qp + (2 * p + hh) * E);
        if (a->neg)
            qf[p] = flip<T>(qf[p]);
    }
    const int kend = uniform_int(std::max(0, lk - lq + (int)((unsigned)(row0 + rows - 1) / (unsigned)grp) + 1));
    const int kall = uniform_int(std::max(0, lk - lq + (int)((unsigned)row0 / (unsigned)grp) + 1));

    unsigned char *mine = smem + w * GM::kWaveSmem;
    const unsigned lds0 = lds_addr(mine);
    auto issue = [&](int t0, int slot) {
        const unsigned dst = lds0 + slot * 2 * GM::kTileBytes;
        TileLoad<T, D, 32, 1>::issue(dst, kp, a->k_stride, t0, lk, 0, lane);
        TileLoad<T, D, 32, 1>::issue(dst + GM::kTileBytes, vp, a->v_stride, t0, lk, 0, lane);
    };
    f32x16 acc[DB] = {};
    float m = kNoMax, l = 0.f;
    int t0 = 32 * w;
    if (t0 < kend)
        issue(t0, 0);
    for (int n = 0; t0 < kend; ++n, t0 += 32 * NW) {
        const int tn = t0 + 32 * NW;
        // the slot issued next was read by this wave before: its reads are done
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (tn < kend) {
            issue(tn, (n + 1) & 1);
            wait_vmcnt<(kLoads < 63 ? kLoads : 63)>();
        } else {
            wait_vmcnt<0>();
        }
        const unsigned char *Kt = mine + (n & 1) * 2 * GM::kTileBytes, *Vt = Kt + GM::kTileBytes;
        tile32<T, D, 1>(Kt, Vt, qf, t0 + 32 > kall, lim - t0, a->c, lane, m, l, acc);
    }
    T *o = (T *)a->o;
    join_waves<T, D>(smem, sm, sl, w, lane, rows, m, l, acc, [&](int i, f32x4 v, float, float lr) {
        const float inv = lr > 0.f ? 1.f / lr : 0.f;
        T *op = o + srow[i / D] + i % D;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            op[e] = (T)(v[e] * inv);
    });
}

// Launches `kernel` with work-groups of `rows` rows.
hipError_t prefill_launch(void (*kernel)(PrefillArgs), int64_t rows, int threads, unsigned smem,
                          std::atomic<uint64_t> &allowed, PrefillArgs &args, int64_t nseq, const AttnSeq *seqs,
                          hipStream_t s)
{
    hipError_t e = allow_lds(reinterpret_cast<const void *>(kernel), (int)smem, allowed);
    if (e != hipSuccess)
        return e;
    // launches of at most SeqTab::kMax sequences and 2^32 - 1 threads, the sequences
    // with the most work per row block first
    for (int64_t at = 0; at < nseq;) {
        int n = 0;
        int64_t items = 0;
        const int64_t most = (int64_t)UINT32_MAX / threads / args.Hkv;
        while (at < nseq && n < SeqTab::kMax) {
            const int64_t blocks = (seqs[at].lq * (int64_t)args.grp + rows - 1) / rows;
            if (blocks > most - items)
                break;
            args.tab.seq[n++] = seqs[at++];
            items += blocks;
        }
        if (n == 0)
            return hipErrorInvalidValue;                  // one sequence alone is too much
        std::stable_sort(args.tab.seq, args.tab.seq + n,
                         [](const AttnSeq &x, const AttnSeq &y) { return x.lk > y.lk; });
        items = 0;
        for (int i = 0; i < n; ++i) {
            args.tab.pre[i] = (int32_t)items;
            items += (args.tab.seq[i].lq * (int64_t)args.grp + rows - 1) / rows;
        }
        for (int i = n; i < 128; ++i)
            args.tab.pre[i] = INT32_MAX;
        kernel<<<dim3((unsigned)(items * args.Hkv)), dim3(threads), smem, s>>>(args);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
    }
    return hipSuccess;
}

template <typename T, int D, int NW>
hipError_t prefill(PrefillArgs &args, int64_t nseq, const AttnSeq *seqs, hipStream_t s)
{
    static std::atomic<uint64_t> allowed{0}, allowed_few{0};
    constexpr int64_t kRows = 32 * NW;
    // Few rows go to the kernel of 32-row work-groups.  Measured (us, few against
    // many, 32 heads over 8) at n work-groups of 32 rows, a prompt alone (n tokens) and
    // n queries after 4000 cached keys:
    //            n     256              512              768              1024
    //   bf16  64  11/11, 33/80     11/14, 46/85     17/18, 72/90     21/23, 88/94
    //        128  11/12, 47/109    19/19, 89/116    31/25, 130/123   43/32, 172/130
    //        256  17/20, 120/213   33/33, 232/227   59/45, 355/242   88/58, 483/259
    //   fp32  64  12/24, 116/323   25/43, 222/342   47/63, 331/364   72/82, 453/385
    //        128  28/52, 343/761   58/97, 675/804   122/143, 1053/850  192/188, 1433/896
    //        256  115/152, 1762/2590  242/321, 3547/2736  555/485, 5415/2886  905/639, 7430/3037
    // 8 heads over 8 (longer sequences at the same n) cross at the same n or up to half
    // as much again later.  Prompts alone cross later than queries after cached keys
    // (their row blocks differ in length and even out): the limits lie between.
    constexpr int64_t kFew = sizeof(T) == 2 ? 512 : D == 64 ? 1024 : D == 128 ? 768 : 512;
    int64_t blocks = 0;
    for (int64_t i = 0; i < nseq && blocks < (int64_t(1) << 32); ++i)
        blocks += (seqs[i].lq * (int64_t)args.grp + 31) / 32;
    if (blocks * args.Hkv <= kFew)
        return prefill_launch(&attn_prefill_few_kernel<T, D>, 32, 64 * WaveTiles<T, D>::kWaves,
                              WaveTiles<T, D>::kSmem, allowed_few, args, nseq, seqs, s);
    constexpr unsigned kSmem = 4u * (sizeof(T) == 2 ? 64 : 32) * D * sizeof(T);
    return prefill_launch(&attn_prefill_kernel<T, D, NW>, kRows, 64 * NW, kSmem, allowed, args, nseq, seqs, s);
}

// ---------------------------------------------------------------------------
// One decode token per sequence
// ---------------------------------------------------------------------------
// The new token's k and v go to row `at` = lengths[b] of the cache and rows
// 0 .. at are attended.  The rows are cut into chunks of a fixed size (so that
// every work-group does about the same work whatever the lengths are, which
// the host does not know); a work-group takes one chunk of one key head, its
// waves every kWaves-th 32-key tile of it, each with its own running (m, l,
// acc), double-buffered in a part of the LDS that only it touches.  The query
// heads of the group are the columns of the score block.  Chunks are joined by
// a second small kernel.
struct DecodeArgs {
    const void *q, *k, *v;
    void *kc, *vc;
    const int32_t *lengths;
    void *o;
    float *part;                              // [item][split][rows][D] accumulators
    float2 *ml;                               // [item][split][rows] (m, l)
    int64_t q_stride, k_stride, v_stride;
    int64_t M;
    int Hq, Hkv, grp, rtiles;                 // rtiles: 32-row tiles of a group
    int chunk, nsplit;
    float c;
    int neg;
};

// Rows first .. 31 of a wave's K (or V) tile become the new token's.
template <typename T, int D>
__device__ __forceinline__ void put_rows(unsigned char *tile, const T *src, int first, int lane)
{
    typedef Tile<T, D> TL;
    for (int i = lane; i < (32 - first) * TL::kChunks; i += 64) {
        const int row = first + i / TL::kChunks, ch = i % TL::kChunks;
        *reinterpret_cast<uint4 *>(tile + TL::off(row, ch)) =
            *reinterpret_cast<const uint4 *>(src + ch * (16 / (int)sizeof(T)));
    }
}

template <typename T, int D>
__global__ __launch_bounds__((64 * WaveTiles<T, D>::kWaves), 1) void attn_decode_kernel(DecodeArgs a)
{
    typedef WaveTiles<T, D> GM;
    typedef Tile<T, D> TL;
    typedef typename Piece<T>::V V;
    constexpr int E = Piece<T>::E, NW = GM::kWaves, DB = D / 32;
    constexpr int kLoads = 2 * TileLoad<T, D, 32, 1>::kPer;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ float sm[NW][32], sl[NW][32];

    const int tid = threadIdx.x, lane = tid & 63, w = uniform_int(tid >> 6);
    const int cl = lane & 31, hh = lane >> 5;
    // (sequence, key head, row tile) fastest: the chunks of long sequences, which
    // are few in a mixed batch, spread over the launch
    const int items = gridDim.x / a.nsplit;
    const int item = blockIdx.x % items, split = blockIdx.x / items;
    const int rt = item % a.rtiles, hk = (item / a.rtiles) % a.Hkv;
    const int64_t b = item / (a.rtiles * a.Hkv);
    const int at = uniform_int(a.lengths[b]);
    const int rows = std::min(32, a.grp - 32 * rt);       // query heads of this tile
    const int64_t h0 = (int64_t)hk * a.grp + 32 * rt;
    T *op = (T *)a.o + (b * a.Hq + h0) * D;

    if (at < 0 || at >= a.M) {                            // inactive slot
        if (a.nsplit == 1)
            for (int i = tid; i < rows * D; i += 64 * NW)
                op[i] = (T)0.f;
        return;
    }
    const int64_t kbeg = (int64_t)split * a.chunk;
    if (kbeg > at)
        return;
    const int kend = (int)std::min<int64_t>(kbeg + a.chunk, (int64_t)at + 1);   // keys [kbeg, kend)

    V qf[TL::kPieces];
    const T *qp = (const T *)a.q + b * a.q_stride + (h0 + std::min(cl, rows - 1)) * D;
#pragma unroll
    for (int p = 0; p < TL::kPieces; ++p) {
        qf[p] = *reinterpret_cast<const V *>(qp + (2 * p + hh) * E);
        if (a.neg)
            qf[p] = flip<T>(qf[p]);
    }
    const T *kn = (const T *)a.k + b * a.k_stride + (int64_t)hk * D;
    const T *vn = (const T *)a.v + b * a.v_stride + (int64_t)hk * D;
    const int64_t cstride = (int64_t)a.Hkv * D;
    T *kc = (T *)a.kc + b * a.M * cstride + (int64_t)hk * D;
    T *vc = (T *)a.vc + b * a.M * cstride + (int64_t)hk * D;
    if (kend == at + 1 && rt == 0) {                      // the chunk that holds the new row stores it
        for (int i = tid; i < TL::kChunks; i += 64 * NW) {
            *reinterpret_cast<uint4 *>((unsigned char *)(kc + at * cstride) + 16 * i) =
                *reinterpret_cast<const uint4 *>((const unsigned char *)kn + 16 * i);
            *reinterpret_cast<uint4 *>((unsigned char *)(vc + at * cstride) + 16 * i) =
                *reinterpret_cast<const uint4 *>((const unsigned char *)vn + 16 * i);
        }
    }

    unsigned char *mine = smem + w * GM::kWaveSmem;
    const unsigned lds0 = lds_addr(mine);
    // rows of the tile at key t0 that are in the cache already: those before `at`
    auto issue = [&](int t0, int slot) {
        if (t0 >= at)
            return;
        const unsigned dst = lds0 + slot * 2 * GM::kTileBytes;
        TileLoad<T, D, 32, 1>::issue(dst, kc, cstride, t0, at, 0, lane);
        TileLoad<T, D, 32, 1>::issue(dst + GM::kTileBytes, vc, cstride, t0, at, 0, lane);
    };

    f32x16 acc[DB] = {};
    float m = kNoMax, l = 0.f;
    int t0 = (int)kbeg + 32 * w;
    if (t0 < kend)
        issue(t0, 0);
    for (int n = 0; t0 < kend; ++n, t0 += 32 * NW) {
        const int tn = t0 + 32 * NW;
        // the slot issued next was read by this wave before: its reads are done
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (tn < kend && tn < at) {
            issue(tn, (n + 1) & 1);
            wait_vmcnt<(kLoads < 63 ? kLoads : 63)>();
        } else {
            wait_vmcnt<0>();
        }
        unsigned char *Kt = mine + (n & 1) * 2 * GM::kTileBytes, *Vt = Kt + GM::kTileBytes;
        if (t0 + 32 > at) {
            // the new token, and after it (masked rows) its copies
            put_rows<T, D>(Kt, kn, at - t0, lane);
            put_rows<T, D>(Vt, vn, at - t0, lane);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        // (two terms: the matrix units are idle most of the time here)
        tile32<T, D, sizeof(T) == 2 ? 2 : 1>(Kt, Vt, qf, t0 + 32 > kend, kend - t0, a.c, lane, m, l, acc);
    }
    const int64_t slot = ((int64_t)item * a.nsplit + split) * 32;
    join_waves<T, D>(smem, sm, sl, w, lane, rows, m, l, acc, [&](int i, f32x4 v, float mr, float lr) {
        if (a.nsplit == 1) {
            const float inv = lr > 0.f ? 1.f / lr : 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                op[i + e] = (T)(v[e] * inv);
        } else {
            *reinterpret_cast<f32x4 *>(a.part + slot * D + i) = v;
            if (i % D == 0)
                a.ml[slot + i / D] = make_float2(mr, lr);
        }
    });
}

// Joins the chunks of one query head: o = sum_i 2^(m_i - m) acc_i / sum_i 2^(m_i - m) l_i.
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(DecodeArgs a)
{
    constexpr int LPR = D / 4, G = 256 / LPR;             // lanes per row, chunk groups
    __shared__ float4 sacc[G][LPR];
    __shared__ float sl[G], smax[4];
    const int tid = threadIdx.x, g = tid / LPR, d4 = tid % LPR;
    const int64_t b = blockIdx.x / a.Hq;
    const int h = blockIdx.x % a.Hq;
    const int at = a.lengths[b];
    const int ns = at < 0 || at >= a.M ? 0 : at / a.chunk + 1;
    const int hk = h / a.grp, rt = (h % a.grp) / 32, row = h % a.grp % 32;
    const int64_t slot = (((b * a.Hkv + hk) * a.rtiles + rt) * a.nsplit) * 32 + row;
    float mx = kNoMax;
    for (int i = tid; i < ns; i += 256)
        mx = fmaxf(mx, a.ml[slot + (int64_t)i * 32].x);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        mx = fmaxf(mx, __shfl_xor(mx, off, 64));
    if ((tid & 63) == 0)
        smax[tid >> 6] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(smax[0], smax[1]), fmaxf(smax[2], smax[3]));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    // eight chunks in flight per lane (their loads are independent, and few
    // work-groups run)
    constexpr int U = 8;
    for (int i0 = g; i0 < ns; i0 += G * U) {
        float2 ml[U];
        float4 p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = std::min(i0 + u * G, ns - 1);
            ml[u] = a.ml[slot + (int64_t)i * 32];
            p[u] = *reinterpret_cast<const float4 *>(a.part + (slot + (int64_t)i * 32) * D + 4 * d4);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float f = i0 + u * G < ns ? exp2_fast(ml[u].x - mx) : 0.f;
            v.x += f * p[u].x; v.y += f * p[u].y; v.z += f * p[u].z; v.w += f * p[u].w;
            l += f * ml[u].y;
        }
    }
    sacc[g][d4] = v;
    if (d4 == 0)
        sl[g] = l;
    __syncthreads();
    if (tid < LPR) {
        for (int i = 1; i < G; ++i) {
            const float4 p = sacc[i][d4];
            v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
            l += sl[i];
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        T *op = (T *)a.o + (b * a.Hq + h) * D + 4 * d4;
        op[0] = (T)(v.x * inv);
        op[1] = (T)(v.y * inv);
        op[2] = (T)(v.z * inv);
        op[3] = (T)(v.w * inv);
    }
}

// Keys per work-group: about 2048 work-groups when the cache is full (eight
// rounds of the chip, so that unequal lengths even out), 128 keys at least.
int64_t decode_chunk(int64_t B, int64_t M, int64_t Hkv, int64_t rtiles)
{
    const int64_t want = (M * B * Hkv * rtiles + 2047) / 2048;
    return std::max<int64_t>(128, (want + 127) / 128 * 128);
}

template <typename T, int D> hipError_t decode(const DecodeArgs &a, int64_t B, hipStream_t s)
{
    typedef WaveTiles<T, D> GM;
    static std::atomic<uint64_t> allowed{0};
    hipError_t e = allow_lds(reinterpret_cast<const void *>(&attn_decode_kernel<T, D>), (int)GM::kSmem, allowed);
    if (e != hipSuccess)
        return e;
    const unsigned grid = (unsigned)(B * a.Hkv * a.rtiles * a.nsplit);
    attn_decode_kernel<T, D><<<dim3(grid), dim3(64 * GM::kWaves), GM::kSmem, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess || a.nsplit == 1)
        return e;
    attn_join_kernel<T, D><<<dim3((unsigned)(B * a.Hq)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_prefill(int bf16, int64_t nseq, const AttnSeq *seqs, int64_t Hq, int64_t Hkv,
                               int64_t D, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                               float scale, const void *q, const void *k, const void *v, void *o,
                               hipStream_t s)
{
    PrefillArgs args = {};
    args.q = q;
    args.k = k;
    args.v = v;
    args.o = o;
    args.q_stride = q_stride;
    args.k_stride = k_stride;
    args.v_stride = v_stride;
    args.Hq = (int)Hq;
    args.Hkv = (int)Hkv;
    args.grp = (int)(Hq / Hkv);
    args.c = score_factor(scale);
    args.neg = scale < 0.f;
    if (bf16) {
        switch (D) {
        case 64: return prefill<__bf16, 64, 8>(args, nseq, seqs, s);
        case 128: return prefill<__bf16, 128, 8>(args, nseq, seqs, s);
        case 256: return prefill<__bf16, 256, 4>(args, nseq, seqs, s);
        }
    } else {
        switch (D) {
        case 64: return prefill<float, 64, 4>(args, nseq, seqs, s);
        case 128: return prefill<float, 128, 4>(args, nseq, seqs, s);
        case 256: return prefill<float, 256, 4>(args, nseq, seqs, s);
        }
    }
    return hipErrorInvalidValue;
}


int64_t attn_decode_splits(int64_t B, int64_t M, int64_t Hq, int64_t Hkv)
{
    const int64_t rtiles = (Hq / Hkv + 31) / 32;
    const int64_t chunk = decode_chunk(B, M, Hkv, rtiles);
    return std::max<int64_t>(1, (M + chunk - 1) / chunk);
}

size_t attn_decode_workspace(int64_t B, int64_t M, int64_t Hq, int64_t Hkv, int64_t D)
{
    if (B == 0 || M == 0)
        return 0;
    const int64_t ns = attn_decode_splits(B, M, Hq, Hkv);
    if (ns <= 1)
        return 0;
    const int64_t slots = B * Hkv * ((Hq / Hkv + 31) / 32) * ns * 32;
    return (size_t)(slots * (D * 4 + 8));
}

hipError_t launch_attn_decode(int bf16, int64_t B, int64_t M, int64_t Hq, int64_t Hkv, int64_t D,
                              int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                              const void *q, const void *k, const void *v, void *k_cache,
                              void *v_cache, const int32_t *lengths, void *o, void *ws,
                              hipStream_t s)
{
    DecodeArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.kc = k_cache;
    a.vc = v_cache;
    a.lengths = lengths;
    a.o = o;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.M = M;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.grp = (int)(Hq / Hkv);
    a.rtiles = (a.grp + 31) / 32;
    a.chunk = (int)decode_chunk(B, M, Hkv, a.rtiles);
    a.nsplit = (int)attn_decode_splits(B, M, Hq, Hkv);
    a.c = score_factor(scale);
    a.neg = scale < 0.f;
    a.part = static_cast<float *>(ws);
    a.ml = reinterpret_cast<float2 *>(a.part + B * Hkv * a.rtiles * (int64_t)a.nsplit * 32 * D);
    if (bf16) {
        switch (D) {
        case 64: return decode<__bf16, 64>(a, B, s);
        case 128: return decode<__bf16, 128>(a, B, s);
        case 256: return decode<__bf16, 256>(a, B, s);
        }
    } else {
        switch (D) {
        case 64: return decode<float, 64>(a, B, s);
        case 128: return decode<float, 128>(a, B, s);
        case 256: return decode<float, 256>(a, B, s);
        }
    }
    return hipErrorInvalidValue;
}

}  // namespace ssd
