// Linear attention with one decay per head on gfx950: the chunked form over
// prompts (batched or packed) and the recurrent step for single tokens.
//
// Per value head j with query/key head i = j / (Hv / Hk) and lambda = e^g_j:
//     S_t = lambda S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t       (S: dk x dv, fp32)
// Over a tile of n tokens entered with state S (t, s = 0 .. n - 1):
//     o_t = scale (lambda^(t+1) S^T q_t + sum_{s<=t} lambda^(t-s) (q_t . k_s) v_s)
//     S  <- lambda^n S + sum_s lambda^(n-1-s) k_s v_s^T
// The decay is the same for every token, so the scan keeps the state as R with
// S = lambda^(e-N) R, e the tokens since the last rescale and N those of an epoch: a
// tile then adds lambda^(N-e-s-1) k_s v_s^T to R without touching the rest of it,
// with weights from a table, and R is multiplied by lambda^N once per epoch: every
// kEpochTiles tiles, or sooner, before the weights would fall below 2^-kEpoch.  A head
// that forgets more than that within a tile is scaled every tile instead.  No weight
// passes 1, so R overflows only where S does; below, terms of S (three bf16 numbers)
// keep their 24 bits down to 2^(kEpoch-110) and those of q . S down to 2^(kEpoch-102).
// Powers of lambda are formed from the exponent in fp64 (in fp32 they would be off by
// up to kEpoch 2^-24 relative).
//
// Rounding (bf16): q, k, v are exact operands.  The state and the masked scores
// are each rounded once to bf16 on their way into the products that form o
// (each about as large as the rounding of o itself); the state update takes
// lambda^.. v as the sum of three bf16 numbers, which hold an fp32 product
// whole, so that the end state keeps fp32 accuracy, or of two (off by up to 2^-17)
// where the end state has forgotten the tokens below 2^-kForget, or none is wanted:
// no token's rounding is larger than 2^-24 of its product, whatever follows it.  (Three
// throughout: 273 against 255 us for the scan below.)
//
// q, k, v and o move once in the scan; a sequence cut into segments, to fill the chip,
// has all but its last segment's k and v read a second time by the state kernel.  4 x
// 8192 tokens of 32 heads of 128 x 128 over 16 (bf16, 4 segments): 250 - 256 us in all,
// the scan 134 - 180 us of it for 850 MB counted (bound by memory: a copy moves 4.8
// TB/s on the same card, 180 us; part of k and v is still in the memory-side cache),
// the state kernel 87 - 102 us for 223 MB (bound by its chain of up to 64 tiles, about
// 1.4 us each; heads that forget fast stop early).  What the scan needed for that: two
// work-groups per CU (32-token tiles; 64-token ones left room for one, 450 us in all),
// every wave forming a share of the next tile's scores (338 us before), no register
// spilled inside the loop (a spill's reload waits for the tiles on their way: 2 to 3
// times slower), few vector instructions beside the products (one base register per LDS
// operand, weights from a table).  With 256 keys the registers do not suffice: bf16
// reloads 20 from scratch in each tile and moves 520 to or from the accumulators (6 us
// a tile), fp32 reloads up to 9, and 3 with 128 keys by 64 columns.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>
#include <utility>
#include <vector>

#include "ssd_attn.h"
#include "ssd_mma.h"

namespace ssd {
namespace {

using namespace mx;

constexpr double kLog2e = 1.4426950408889634;
// Powers of two that an epoch's weights span.  Larger spans lose small terms, smaller
// ones rescale more heads in every tile: 8 x 2048 tokens of 24 heads (log decays -0.8
// to -1/256) 67.0 us with 40, 69.4 with 24.
constexpr float kEpoch = 40.f;
constexpr int kEpochTiles = 8;
// Chained states times keys from which lin_chain_kernel runs (us without and with
// it): bf16, one sequence, 4 heads of 256 x 64, 6 segments 514 and 496, 16 segments
// 295 and 207, 64 segments 493 and 83; 32 heads of 128 x 128, 6 segments 394 and 399,
// 12 segments (2048 tokens) 52 and 45; fp32, 8 heads of 64 x 64, 11 segments 29 and 32.
constexpr int64_t kChain = 1024;
constexpr float kForget = 7.f;                // two terms leave 2^-17 of a product: 2^-24 by then

struct LinTab {
    static constexpr int kMax = 96;           // sequences per launch (kernel arguments: 4 KB)
    int64_t tok[kMax];
    int32_t len[kMax];
    int32_t slot[kMax];                       // first state slot of the sequence
    int32_t pre[128];                         // first work item of each sequence; then INT32_MAX
    int32_t id[kMax];                         // the sequence's index among all (states)
};

struct LinArgs {
    LinTab tab;
    const void *q, *k, *v;
    const float *g;
    const float *init;
    void *o;
    float *fin;
    float *ws;                                // [slot][Hv][column tile][dk x columns], fragment order
    int64_t q_stride, k_stride, v_stride;
    int32_t seg_tokens, Hk, Hv, dv;
    float scale;
    int copy_init;                            // fin is init: segment 0 starts from its slot's copy
    int chained;                              // slots hold entering states (lin_chain_kernel)
};

typedef const __attribute__((address_space(4))) LinArgs *LinArgsPtr;

// lambda^n for an exponent of any size, g2 = log2 lambda.
__device__ __forceinline__ float pow_of(double g2, double n)
{
    double x = g2 * n;
    x = x < -2000.0 ? -2000.0 : x > 2000.0 ? 2000.0 : x;
    const double r = __builtin_rint(x);
    return __builtin_ldexpf(exp2_fast((float)(x - r)), (int)r);
}

template <typename T, int DK, int NW> struct LinSmem {
    static constexpr int C = 32, CT = 32 * NW;   // tokens per tile, value columns
    static constexpr int kK = C * DK * (int)sizeof(T), kV = C * CT * (int)sizeof(T);
    static constexpr int kP = C * C * (int)sizeof(T);
    static constexpr int kScanSlot = 2 * kK + kV, kStateSlot = kK + kV;
    // tiles in LDS: in use, landed, on its way.  Work-groups of two waves do without
    // the one between, so that three instead of two share a CU (8 x 2048 tokens of 24
    // heads of 128 x 64 in bf16: 75 us against 94), as does whatever has no room for it.
    static constexpr int kRing = 3 * (kScanSlot + kP) <= 158 * 1024 && NW == 4 ? 3 : 2;
    static constexpr int kScan = kRing * (kScanSlot + kP);
    static constexpr int kStateRing = 3 * kStateSlot <= 159 * 1024 ? 3 : 2, kState = kStateRing * kStateSlot;
    static constexpr int kTables = ((kEpochTiles + 1) * C + kEpochTiles + 1) * 4;
    static constexpr int kScanBytes = kScan + kTables;
};

// The state row (of a 32-row block) that register r of lane half hh holds.
template <typename T> __device__ __forceinline__ int state_row(int r, int hh)
{
    if constexpr (sizeof(T) == 2)
        return 16 * (r >> 3) + 8 * hh + (r & 7);
    else
        return 8 * (r >> 2) + 4 * hh + (r & 3);
}

// v * u as the sum of kTerms bf16 numbers (three hold an fp32 product whole).
template <int kTerms>
__device__ __forceinline__ void weigh(bf16x8 v, const f32x4 &u0, const f32x4 &u1, bf16x8 (&x)[kTerms])
{
    const u32x4 vb = __builtin_bit_cast(u32x4, v);
    u32x4 xb[kTerms];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float p = __builtin_bit_cast(float, vb[j] << 16) * (j < 2 ? u0[2 * j] : u1[2 * j - 4]);
        float q = __builtin_bit_cast(float, vb[j] & 0xffff0000u) * (j < 2 ? u0[2 * j + 1] : u1[2 * j - 3]);
#pragma unroll
        for (int i = 0; i < kTerms; ++i) {
            xb[i][j] = pack_bf16(p, q);
            if (i + 1 == kTerms)
                break;
            p -= __builtin_bit_cast(float, xb[i][j] << 16);
            q -= __builtin_bit_cast(float, xb[i][j] & 0xffff0000u);
        }
    }
#pragma unroll
    for (int i = 0; i < kTerms; ++i)
        x[i] = __builtin_bit_cast(bf16x8, xb[i]);
}

// What a work-group of either kernel works on.
struct Work {
    int si, seg, head, ct, hk;                // sequence, segment, value head, column tile, query/key head
    int len, nseg, beg, end;                  // the sequence's tokens and segments, the segment's tokens
};
template <int CT> __device__ __forceinline__ Work work_of(LinArgsPtr a, int lane)
{
    // value heads of a query/key head, and their column tiles, next to each other
    // on one XCD: they read the same q and k
    const unsigned nb = gridDim.x, per = nb / 8;
    const unsigned bid = blockIdx.x < per * 8 ? (blockIdx.x % 8) * per + blockIdx.x / 8 : blockIdx.x;
    const int Hv = a->Hv, nct = a->dv / CT, hc = Hv * nct;
    const int item = (int)(bid / (unsigned)hc), hx = (int)(bid % (unsigned)hc);
    const int below = __popcll(__ballot(a->tab.pre[lane] <= item)) +
                      __popcll(__ballot(a->tab.pre[64 + lane] <= item));
    Work k;
    k.si = uniform_int(below - 1);
    k.seg = item - a->tab.pre[k.si];
    k.head = hx / nct;
    k.ct = hx % nct;
    k.hk = k.head / (Hv / a->Hk);
    k.len = a->tab.len[k.si];
    k.nseg = std::max(1, (k.len + a->seg_tokens - 1) / a->seg_tokens);
    k.beg = k.seg * a->seg_tokens;
    k.end = std::min(k.len, k.beg + a->seg_tokens);
    return k;
}

// A wave's 32 columns of a state: element (row, column) of the [dk][dv] matrix of
// init and fin, and its slot in the workspace (fragment order: coalesced).
template <typename T, int DK>
__device__ __forceinline__ void load_state(f32x16 (&R)[DK / 32], const float *p, int dv, int hh)
{
#pragma unroll
    for (int d = 0; d < DK / 32; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            R[d][r] = p[(int64_t)(32 * d + state_row<T>(r, hh)) * dv];
}
template <int DK> __device__ __forceinline__ void store_slot(float *p, const f32x16 (&R)[DK / 32])
{
#pragma unroll
    for (int d = 0; d < DK / 32; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *reinterpret_cast<f32x4 *>(p + (d * 4 + g) * 256) =
                f32x4{R[d][4 * g], R[d][4 * g + 1], R[d][4 * g + 2], R[d][4 * g + 3]};
}
template <int DK> __device__ __forceinline__ void add_slot(f32x16 (&R)[DK / 32], const float *p, float f)
{
#pragma unroll
    for (int d = 0; d < DK / 32; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x4 z = *reinterpret_cast<const f32x4 *>(p + (d * 4 + g) * 256);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                R[d][4 * g + e] = __builtin_fmaf(z[e], f, R[d][4 * g + e]);
        }
}

// A tile's update of the wave's state columns, from its K tile in LDS (lane offset
// `bk` included) and its V operands: R += sum_s u_s k_s v_s^T, u being the lane's
// weights of the tokens (u4(i, j): four of piece i).
template <typename T, int DK, int kTerms, typename U>
__device__ __forceinline__ void update(f32x16 (&R)[DK / 32], unsigned bk,
                                       const typename Piece<T>::V (&vf)[16 / Piece<T>::E],
                                       typename Piece<T>::V (&kf)[DK / 32], U u4)
{
    typedef LaneBase<T, DK> BK;
    constexpr int DB = DK / 32, PT = 16 / Piece<T>::E;
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        if constexpr (sizeof(T) == 2) {
            bf16x8 x[kTerms];
            weigh(vf[i], u4(i, 0), u4(i, 1), x);
#pragma unroll
            for (int j = 0; j < kTerms; ++j)
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    R[d] = mma(kf[d], x[j], R[d]);
        } else {
            const f32x4 x = vf[i] * u4(i, 0);
#pragma unroll
            for (int d = 0; d < DB; ++d)
                R[d] = mma(kf[d], x, R[d]);
        }
        if (i + 1 < PT)
#pragma unroll
            for (int d = 0; d < DB; ++d)
                kf[d] = BK::col_piece(0, bk, i + 1, d);
    }
}

// The end state of a segment (every segment but its sequence's last, so a whole
// number of tiles) into its slot: sum_t lambda^(T-1-t) k_t v_t^T, with the first
// segment's initial state.  The tiles are walked from the end: the weights then
// only shrink, R needs no rescaling, the walk ends where lambda^(T-1-t) is 0 in
// fp32, and the tokens read last are those the scan reads first.
template <typename T, int DK, int NW>
__global__ __launch_bounds__(64 * NW, DK == 256 || sizeof(T) == 4 ? 1 : 2) void lin_state_kernel(
    LinArgs args_in_kernarg)
{
    typedef LinSmem<T, DK, NW> SM;
    constexpr int C = SM::C, CT = SM::CT, DB = DK / 32, PT = 16 / Piece<T>::E, E = Piece<T>::E;
    typedef typename Piece<T>::V V;
    typedef LaneBase<T, DK> BK;
    typedef LaneBase<T, CT> BV;
    typedef TileLoad<T, DK, C, NW> LK;
    typedef TileLoad<T, CT, C, NW> LV;
    constexpr int kLoads = LK::kPer + LV::kPer, kSlot = SM::kStateSlot, kRing = SM::kStateRing;
    extern __shared__ __align__(1024) unsigned char smem[];   // the ring, then lambda^(C-1-s)
    float *su = reinterpret_cast<float *>(smem + SM::kState);

    const LinArgsPtr a = (LinArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    const int tid = threadIdx.x, lane = tid & 63, w = uniform_int(tid >> 6), hh = lane >> 5;
    const Work k = work_of<CT>(a, lane);
    const int dv = a->dv, Hv = a->Hv, ntile = (k.end - k.beg) / C;
    const double g2 = std::max(a->g[k.head] * kLog2e, -1e5);
    const float g2f = (float)g2;
    const T *kp = (const T *)a->k + a->tab.tok[k.si] * a->k_stride + (int64_t)k.hk * DK;
    const T *vp = (const T *)a->v + a->tab.tok[k.si] * a->v_stride + (int64_t)k.head * dv + k.ct * CT;
    float *slot0 = a->ws + (((int64_t)a->tab.slot[k.si] * Hv + k.head) * (dv / CT) + k.ct) * ((int64_t)DK * CT) +
                   w * (DK * 32) + lane * 4;
    const int64_t wslot = (int64_t)Hv * DK * dv;          // floats between slots

    if (tid < C)
        su[tid] = pow_of(g2, C - 1 - tid);
    // tiles that count: lambda^(n C) >= 2^-150
    const int cnt = g2f * (float)C * (float)ntile < -150.f
                        ? std::max(1, std::min(ntile, (int)std::min(1e6f, -150.f / (g2f * (float)C)) + 1))
                        : ntile;
    f32x16 R[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            R[d][r] = 0.f;
    if (k.seg == 0 && a->init) {
        load_state<T, DK>(R, a->init + (a->tab.id[k.si] * (int64_t)Hv + k.head) * DK * dv + k.ct * CT + 32 * w +
                                 (lane & 31), dv, hh);
        if (a->copy_init)
            store_slot<DK>(slot0 + (k.nseg - 1) * wslot, R);
        const float f = pow_of(g2, k.end - k.beg);
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                R[d][r] *= f;
    }

    const unsigned lds0 = lds_addr(smem);
    auto issue = [&](int n) {                             // the n-th tile from the end
        const unsigned dst = lds0 + (n % kRing) * kSlot;
        const int t0 = k.end - (n + 1) * C;
        LK::issue(dst, kp, a->k_stride, t0, k.end, w, lane);
        LV::issue(dst + SM::kK, vp, a->v_stride, t0, k.end, w, lane);
    };
    const unsigned bk = lds0 + BK::template col<true>(lane);
    const unsigned bv = lds0 + (BV::template col<false>(lane) ^ (sizeof(T) == 2 ? (unsigned)w << 6 : (unsigned)w << 7));
    auto tile = [&](int n, auto terms) {
        // this wave's share of the tile has landed (the next one's loads are on their
        // way), then everyone's has, and the tile before has been read
        if (kRing == 3 && n + 1 < cnt)
            wait_vmcnt<kRing == 3 ? kLoads : 0>();
        else
            wait_vmcnt<0>();
        lds_barrier();
        if (n + kRing - 1 < cnt)
            issue(n + kRing - 1);
        const unsigned ring = (unsigned)(n % kRing) * kSlot, b = opaque(bk) + ring, c = opaque(bv) + ring;
        V vf[PT], kf[DB];
#pragma unroll
        for (int i = 0; i < PT; ++i)
            vf[i] = BV::col_piece(SM::kK, c, i, 0);
#pragma unroll
        for (int d = 0; d < DB; ++d)
            kf[d] = BK::col_piece(0, b, 0, d);
        const float f = pow_of(g2, (double)n * C);
        update<T, DK, decltype(terms)::value>(R, b, vf, kf, [&](int i, int j) {
            return f * *reinterpret_cast<const f32x4 *>(su + 2 * E * i + E * hh + 4 * j);
        });
    };
    if (cnt > 0)
        issue(0);
    if (kRing == 3 && cnt > 1)
        issue(1);
    // tokens that the segment's end has forgotten below 2^-kForget take two terms
    const int keep = sizeof(T) == 2 && g2f <= 0.f
                         ? std::min(cnt, (int)std::min(1e6f, kForget / (1e-9f - g2f * (float)C)) + 1)
                         : cnt;
    int n = 0;
    for (; n < keep; ++n)
        tile(n, std::integral_constant<int, 3>());
    for (; n < cnt; ++n)
        tile(n, std::integral_constant<int, 2>());
    store_slot<DK>(slot0 + k.seg * wslot, R);
}

// The slots of long chains made running states in place: slot j becomes the state
// after segment j, slot j-1 lambda^T0 + slot j (the factor to more than fp32, as its
// rounding would be repeated).  Every segment of the scan then reads one slot instead
// of all before its own.  One thread takes four elements of all segments, eight
// segments' loads in flight.
template <int DK> __global__ __launch_bounds__(256) void lin_chain_kernel(LinArgs args_in_kernarg)
{
    const LinArgsPtr a = (LinArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    const int per = a->Hv * a->dv * (DK / 64) / 16;       // work-groups of a sequence: 1024 elements each
    const int si = blockIdx.x / (unsigned)per, at = (blockIdx.x % (unsigned)per) * 1024;
    const int last = (a->tab.len[si] + a->seg_tokens - 1) / a->seg_tokens - 1;   // slots 0 .. last - 1
    if (last < 2)
        return;
    const double g2 = std::max(a->g[at / (DK * a->dv)] * kLog2e, -1e5);
    const double fd = exp2(g2 * (double)a->seg_tokens);
    const float fhi = (float)fd, flo = fhi < 3e38f ? (float)(fd - (double)fhi) : 0.f;
    const int64_t wslot = (int64_t)a->Hv * DK * a->dv;
    float *p = a->ws + (int64_t)a->tab.slot[si] * wslot + at + 4 * threadIdx.x;
    constexpr int U = 8;
    f32x4 acc = *reinterpret_cast<const f32x4 *>(p);
    for (int j0 = 1; j0 < last; j0 += U) {
        f32x4 z[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            z[u] = *reinterpret_cast<const f32x4 *>(p + std::min(j0 + u, last - 1) * wslot);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j0 + u >= last)
                break;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[e] = __builtin_fmaf(acc[e], fhi, __builtin_fmaf(acc[e], flo, z[u][e]));
            *reinterpret_cast<f32x4 *>(p + (j0 + u) * wslot) = acc;
        }
    }
}

// o over one segment of one (sequence, value head, column tile), and the end state
// for a sequence's last segment.
//
// A wave owns 32 value columns: its dk x 32 slice of R stays in the result
// registers and is the operand of the state product as it stands (contraction
// over its rows), and the scores of a tile, the same for all columns, are shared
// through LDS.  Outputs are formed transposed (columns x tokens): a lane holds
// one token, so its power of lambda is one per-lane factor.
template <typename T, int DK, int NW>
__global__ __launch_bounds__(64 * NW, DK == 256 || sizeof(T) == 4 ? 1 : 2) void lin_scan_kernel(LinArgs args_in_kernarg)
{
    typedef LinSmem<T, DK, NW> SM;
    constexpr int C = SM::C, CT = SM::CT, DB = DK / 32;
    static_assert(C == 32, "a tile is one 32-token block");
    constexpr int E = Piece<T>::E, PB = 16 / E;           // pieces per 32-row block
    constexpr int PT = C / (2 * E);                       // pieces over a tile's tokens
    typedef Tile<T, DK> TK;
    typedef Tile<T, C> TP;
    typedef LaneBase<T, DK> BK;
    typedef LaneBase<T, CT> BV;
    typedef LaneBase<T, C> BP;
    typedef typename Piece<T>::V V;
    constexpr int kStores = sizeof(T) == 2 ? 2 : 4;       // per wave and tile
    extern __shared__ __align__(1024) unsigned char smem[];
    // after the ring: update weights of an epoch's tokens, lambda^(N-1-(i C+s))
    // (direct: those of a tile, lambda^(C-1-s); the last C: a ragged tile's), and
    // lambda^(i C-N).  (All of it dynamic, so that the ring starts at LDS address 0 and
    // its offsets are immediates.)
    float *su = reinterpret_cast<float *>(smem + SM::kScan);
    float *spow = su + (kEpochTiles + 1) * C;

    const LinArgsPtr a = (LinArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    const int tid = threadIdx.x, lane = tid & 63, w = uniform_int(tid >> 6);
    const int cl = lane & 31, hh = lane >> 5;
    const Work k = work_of<CT>(a, lane);
    const int seg = k.seg, nseg = k.nseg, beg = k.beg, end = k.end, head = k.head, T0 = a->seg_tokens;
    const int Hv = a->Hv, dv = a->dv;
    const double g2 = std::max(a->g[head] * kLog2e, -1e5);
    const float g2f = (float)g2;
    const int col0 = k.ct * CT + 32 * w;                  // the wave's first column of dv

    const int64_t tok0 = a->tab.tok[k.si];
    const T *qp = (const T *)a->q + tok0 * a->q_stride + (int64_t)k.hk * DK;
    const T *kp = (const T *)a->k + tok0 * a->k_stride + (int64_t)k.hk * DK;
    const T *vp = (const T *)a->v + tok0 * a->v_stride + (int64_t)head * dv + k.ct * CT;
    const int64_t sbase = (a->tab.id[k.si] * (int64_t)Hv + head) * DK * dv + col0 + cl;   // of init and fin
    const float *slot0 = a->ws + (((int64_t)a->tab.slot[k.si] * Hv + head) * (dv / CT) + k.ct) * ((int64_t)DK * CT) +
                         w * (DK * 32) + lane * 4;
    const int64_t wslot = (int64_t)Hv * DK * dv;          // floats between slots

    // ---- the state entering the segment ----
    f32x16 R[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            R[d][r] = 0.f;
    if (seg == 0) {
        if (a->copy_init && nseg > 1)
            add_slot<DK>(R, slot0 + (nseg - 1) * wslot, 1.f);
        else if (a->init)
            load_state<T, DK>(R, a->init + sbase, dv, hh);
    } else {
        // slot 0 holds the state after segment 0 (the initial one included), slot
        // j segment j's from zero; those forgotten below 2^-150 are left out
        int j = a->chained ? seg - 1 : 0;
        while (j < seg - 1 && g2f * (float)T0 * (float)(seg - 1 - j) < -150.f)
            ++j;
        for (; j < seg; ++j)
            add_slot<DK>(R, slot0 + j * wslot, pow_of(g2, (double)T0 * (seg - 1 - j)));
    }

    const unsigned lds0 = lds_addr(smem);
    constexpr int kSlot = SM::kScanSlot, kRing = SM::kRing;
    constexpr bool kAhead = kRing == 3;                   // scores are formed a tile ahead
    auto issue = [&](int t0, int slot) {
        const unsigned dst = lds0 + slot * kSlot;
        TileLoad<T, DK, C, NW>::issue(dst, kp, a->k_stride, t0, end, w, lane);
        TileLoad<T, CT, C, NW>::issue(dst + SM::kK, vp, a->v_stride, t0, end, w, lane);
        TileLoad<T, DK, C, NW>::issue(dst + SM::kK + SM::kV, qp, a->q_stride, t0, end, w, lane);
    };

    const bool direct = -g2f * (float)C > kEpoch || g2f > 0.f;   // scaled every tile
    const int epoch =
        direct ? 0 : std::max(1, (int)std::min((float)kEpochTiles, kEpoch / (1e-9f - g2f * (float)C)));
    const int N = C * epoch;
    // what R is multiplied by when it is rescaled, to more than fp32
    float fhi = pow_of(g2, direct ? C : N), flo = 0.f;
    if (epoch == kEpochTiles) {
        const double fd = exp2(g2 * (double)N);
        fhi = (float)fd;
        flo = (float)(fd - (double)fhi);
    }
    const float scale = a->scale;
    for (int i = tid; i < kEpochTiles * C; i += 64 * NW)
        su[i] = pow_of(g2, (direct ? C : N) - 1 - i);
    if (tid <= kEpochTiles)
        spow[tid] = direct ? 1.f : pow_of(g2, tid * C - N);
    const float ft = scale * pow_of(g2, cl + 1);          // scale lambda^(t+1), the lane's token t
    const bool wide = fabsf(scale) > 0x1p80f;             // times lambda^-N may pass fp32
    // the wave's 16 x 16 blocks of a tile's masked scores (transposed: s x t): factors
    // scale lambda^(t-s), and the scores of the tile in `slot` into its P buffer
    constexpr int kBlk = 4 / NW;
    const int c16 = lane & 15, g16 = lane >> 4;
    float fp[kBlk][4];
#pragma unroll
    for (int j = 0; j < kBlk; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tb = (w * kBlk + j) >> 1, sb = (w * kBlk + j) & 1;
            const int d = 16 * (tb - sb) + c16 - 4 * g16 - i;       // t - s
            fp[j][i] = d < 0 ? 0.f : scale * exp2_fast(g2f * (float)d);
        }
    constexpr int kSp = TK::kChunks / 4;                  // pieces of a 16-row operand
    const unsigned bsk = BK::row16(c16, g16);             // the lane's offsets of each operand
    const unsigned bq = BK::row32(cl, hh), bk = BK::template col<true>(lane);
    const unsigned bv = BV::template col<false>(lane) ^ (sizeof(T) == 2 ? (unsigned)w << 6 : (unsigned)w << 7);
    const unsigned bp = BP::row32(cl, hh);
    struct ScoreIn {
        V k[kSp], q[kSp];
    };
    const int tb = (w * kBlk) >> 1;                       // the blocks' tokens t
    auto score_load_k = [&](int slot, int j, ScoreIn &in) {
        const unsigned b =
            opaque(bsk) + (unsigned)(slot * kSlot) + (((unsigned)(w * kBlk + j) & 1) * 16u) * TK::kPitch;
#pragma unroll
        for (int i = 0; i < kSp; ++i)
            in.k[i] = BK::piece16(0, b, i);
    };
    auto score_load = [&](int slot, ScoreIn &in) {
        const unsigned b = opaque(bsk) + (unsigned)(slot * kSlot) + (unsigned)tb * 16u * TK::kPitch;
#pragma unroll
        for (int i = 0; i < kSp; ++i)
            in.q[i] = BK::piece16(SM::kK + SM::kV, b, i);
        score_load_k(slot, 0, in);
    };
    auto score_store = [&](int slot, ScoreIn &in) {
        unsigned char *Pt = smem + kRing * kSlot + slot * SM::kP;
#pragma unroll
        for (int j = 0; j < kBlk; ++j) {
            const int sb = (w * kBlk + j) & 1;
            f32x4 p = {};
#pragma unroll
            for (int i = 0; i < kSp; ++i)
                p = mma16(in.k[i], in.q[i], p);
            if (j + 1 < kBlk)
                score_load_k(slot, j + 1, in);
#pragma unroll
            for (int i = 0; i < 4; ++i)                   // (a masked score may be infinite: no 0 times it)
                p[i] = fp[j][i] == 0.f ? 0.f : p[i] * fp[j][i];
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<uint2 *>(Pt + TP::off(16 * tb + c16, 2 * sb + (g16 >> 1)) + 8 * (g16 & 1)) =
                    make_uint2(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]));
            else
                *reinterpret_cast<f32x4 *>(Pt + TP::off(16 * tb + c16, 4 * sb + g16)) = p;
        }
    };

    if (beg < end) {
        issue(beg, 0);
        if (kAhead && beg + C < end)
            issue(beg + C, 1);
        wait_vmcnt<0>();
        if constexpr (kAhead) {
            lds_barrier();                                // (the tables are written, too)
            ScoreIn in;
            score_load(0, in);
            score_store(0, in);
        }
    }
    T *const out = (T *)a->o;
    // tiles done; S = lambda^(e-N) R, ep = e / C (entered with R = S: rescaled at once)
    int n = 0, ep = epoch, e = N;
    int64_t orow = ((tok0 + beg) * Hv + head) * (int64_t)dv + col0;
    const unsigned ostride = (unsigned)(Hv * dv * (int)sizeof(T));
    const unsigned olane = (unsigned)cl * ostride + 16u * (unsigned)hh;

    // one tile; mode 0: the head is scaled every tile, else the bf16 terms of the
    // update's weighted values
    int slot = 0;
    auto tile = [&](auto mode) {
        constexpr int kMode = decltype(mode)::value;
        constexpr bool kDirect = kMode == 0;
        constexpr int kTerms = kDirect ? 3 : kMode;
        const int next = slot == kRing - 1 ? 0 : slot + 1, last = slot == 0 ? kRing - 1 : slot - 1;
        const int t0 = beg + n * C, rows = std::min(C, end - t0);
        // the next tile's loads of this wave have landed (this tile's were waited for
        // before; the last tile's stores, issued after them, may still be on their
        // way), then everyone's have, the last tile has been read and this one's
        // scores are there
        if (n > 0)
            wait_vmcnt<kStores>();
        lds_barrier();
        if (t0 + (kRing - 1) * C < end)
            issue(t0 + (kRing - 1) * C, last);
        const unsigned ring = (unsigned)(slot * kSlot), pring = (unsigned)(slot * SM::kP);
        if (!kDirect && ep == epoch) {
            if (epoch == kEpochTiles) {
                // a slowly forgetting head: the factor to more than fp32, since its
                // rounding would be repeated over many epochs
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        R[d][r] = __builtin_fmaf(R[d][r], fhi, R[d][r] * flo);
            } else {
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        R[d][r] *= fhi;
            }
            ep = 0;
            e = 0;
        }
        int ub = ep * C;
        if (rows < C) {   // the tokens past the end weigh 0 (every wave writes the same)
            ub = kEpochTiles * C;
            if (lane < C)
                su[ub + lane] = lane < rows ? su[ep * C + lane + (kDirect ? C - rows : 0)] : 0.f;
            lds_barrier();
        }

        // The LDS reads of a step are issued together ahead of the products (one at a
        // time before its product, as the compiler would have them, each costs its
        // latency); for fp32 and 256 keys there are not the registers for it.
        constexpr bool kBatch = sizeof(T) == 2 && DK <= 128 && NW == 4;
        auto step = [] {
            if constexpr (kBatch)
                __builtin_amdgcn_sched_barrier(0);
        };
        V vf[PT], kf[DB];
        f32x4 uw[E / 4];
        V pf[PT];
        f32x16 y = {};
        const unsigned bvo = opaque(bv) + ring;
#pragma unroll
        for (int i = 0; i < PT; ++i)
            vf[i] = BV::col_piece(SM::kK, bvo, i, 0);
        const unsigned bko = opaque(bk) + ring;
        auto weight4 = [&](int i, int j) {
            return *reinterpret_cast<const f32x4 *>(su + ub + 2 * E * i + E * hh + 4 * j);
        };
        // the (next) tile's scores (past the last tile: of whatever is there, not
        // used) and the state's part
        ScoreIn in;
        score_load(kAhead ? next : slot, in);
        constexpr bool kHold = DK <= 128 && NW == 4;
        V qf[kHold ? TK::kPieces : 1];
        const unsigned bqo = opaque(bq) + ring;
        if constexpr (kHold)
#pragma unroll
            for (int i = 0; i < TK::kPieces; ++i)
                qf[i] = BK::piece32(SM::kK + SM::kV, bqo, i);
        float f = ft * spow[ep];
        step();
        score_store(kAhead ? next : slot, in);
#pragma unroll
        for (int j = 0; j < E / 4; ++j)
            uw[j] = weight4(0, j);
#pragma unroll
        for (int d = 0; d < DB; ++d)
            kf[d] = BK::col_piece(0, bko, 0, d);
        if constexpr (!kAhead)
            lds_barrier();
#pragma unroll
        for (int i = 0; i < PT; ++i)
            pf[i] = BP::piece32(kRing * kSlot, opaque(bp) + pring, i);
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < PB; ++i)
                y = mma(acc_piece(R[d], i, (const T *)nullptr),
                        kHold ? qf[kHold ? d * PB + i : 0] : BK::piece32(SM::kK + SM::kV, bqo, d * PB + i), y);
        step();

        // the state update (issued ahead of the other wave of the SIMD)
        __builtin_amdgcn_s_setprio(1);
        if constexpr (kDirect) {
            const float fd = rows < C ? su[C - 1 - rows] : fhi;   // lambda^rows
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    R[d][r] *= fd;
        }
        update<T, DK, kTerms>(R, bko, vf, kf, [&](int i, int j) { return i == 0 ? uw[j] : weight4(i, j); });

        if (wide) {
#pragma unroll
            for (int r = 0; r < 16; ++r)
                y[r] *= spow[ep];
            f = ft;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r)
            y[r] *= f;
#pragma unroll
        for (int i = 0; i < PT; ++i)
            y = mma(vf[i], pf[i], y);
        // stores through a descriptor that ends at the segment's last row: always the
        // same number of store instructions (see the wait above); a row past the last
        // lies past the descriptor's end whatever the column
        const __amdgpu_buffer_rsrc_t orr = __builtin_amdgcn_make_buffer_rsrc(
            out + orow, (short)0, (int)((unsigned)(rows - 1) * ostride + 32 * (unsigned)sizeof(T)), 0x00020000);
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                unsigned o4[4];
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {
                    const auto sw = __builtin_amdgcn_permlane32_swap(
                        pack_bf16(y[4 * g + 2 * h2], y[4 * g + 2 * h2 + 1]),
                        pack_bf16(y[4 * g + 4 + 2 * h2], y[4 * g + 5 + 2 * h2]), false, false);
                    o4[h2] = sw[0];
                    o4[2 + h2] = sw[1];
                }
                __builtin_amdgcn_raw_buffer_store_b128(u32x4{o4[0], o4[1], o4[2], o4[3]}, orr,
                                                       olane + 16u * (unsigned)g, 0, 0);
            }
        } else {
#pragma unroll
            for (int g = 0; g < 4; ++g)
                __builtin_amdgcn_raw_buffer_store_b128(
                    __builtin_bit_cast(u32x4, f32x4{y[4 * g], y[4 * g + 1], y[4 * g + 2], y[4 * g + 3]}), orr,
                    olane + 32u * (unsigned)g, 0, 0);
        }
        orow += (int64_t)C * Hv * dv;
        __builtin_amdgcn_s_setprio(0);
        if constexpr (!kDirect) {
            ++ep;
            e += rows;
        }
        slot = next;
        ++n;
    };
    const int ntile = (end - beg + C - 1) / C;
    auto tiles = [&](auto mode, int upto) {
        while (n < upto)
            tile(mode);
    };
    if (direct) {
        tiles(std::integral_constant<int, 0>(), ntile);
    } else {
        // tokens that the end of the segment's state has forgotten below 2^-kForget
        // take two terms
        const int keep = seg < nseg - 1 ? 0 : (int)std::min(1e6f, kForget / (1e-9f - g2f * (float)C)) + 1;
        if constexpr (sizeof(T) == 2)
            tiles(std::integral_constant<int, 2>(), ntile - keep);
        tiles(std::integral_constant<int, 3>(), ntile);
    }
    if (seg == nseg - 1) {
        const float fe = pow_of(g2, e - N);
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                a->fin[sbase + (int64_t)(32 * d + state_row<T>(r, hh)) * dv] = R[d][r] * fe;
    }
}

hipError_t launch_part(void (*kernel)(LinArgs), int threads, int smem, std::atomic<uint64_t> &allowed,
                       const LinArgs &args, int64_t groups, hipStream_t s)
{
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(kernel), smem, allowed);
    if (e != hipSuccess)
        return e;
    kernel<<<dim3((unsigned)groups), dim3(threads), smem, s>>>(args);
    return hipGetLastError();
}

// LDS bytes of a scan work-group, for the planner.
template <typename T> int scan_lds_of(int64_t dk, int cols)
{
    if (cols == 128)
        return dk == 64 ? LinSmem<T, 64, 4>::kScanBytes : LinSmem<T, 128, 4>::kScanBytes;
    return dk == 64 ? LinSmem<T, 64, 2>::kScanBytes
                    : dk == 128 ? LinSmem<T, 128, 2>::kScanBytes : LinSmem<T, 256, 2>::kScanBytes;
}
int scan_lds(int bf16, int64_t dk, int cols)
{
    return bf16 ? scan_lds_of<__bf16>(dk, cols) : scan_lds_of<float>(dk, cols);
}

template <typename T, int DK, int NW>
hipError_t scan(LinArgs &args, int64_t nseq, const LinSeq *seqs, hipStream_t s)
{
    typedef LinSmem<T, DK, NW> SM;
    static_assert(SM::kScanBytes <= 160 * 1024, "LDS of a CU");
    static std::atomic<uint64_t> allow_state{0}, allow_scan{0};
    const int64_t T0 = args.seg_tokens, groups = (int64_t)args.Hv * (args.dv / (32 * NW));
    const int64_t most = (int64_t)UINT32_MAX / (64 * NW) / groups;   // a launch holds fewer than 2^32 threads
    int64_t slot = 0;
    for (int64_t at = 0; at < nseq;) {
        int n = 0;
        int64_t items = 0, states = 0, longest = 0;
        int32_t segs[LinTab::kMax];
        while (at < nseq && n < LinTab::kMax) {
            const int64_t ns = std::max<int64_t>(1, (seqs[at].len + T0 - 1) / T0);
            if (items + ns > most)
                break;
            args.tab.tok[n] = seqs[at].tok;
            args.tab.len[n] = (int32_t)seqs[at].len;
            args.tab.id[n] = (int32_t)at;
            args.tab.slot[n] = (int32_t)slot;
            segs[n] = (int32_t)ns;
            slot += ns > 1 ? ns : 0;
            items += ns;
            states += ns - 1;
            longest = std::max(longest, ns);
            ++n;
            ++at;
        }
        if (n == 0)
            return hipErrorInvalidValue;
        hipError_t e;
        args.chained = (longest - 1) * DK >= kChain;
        for (int pass = states > 0 ? 0 : 1; pass < 2; ++pass) {
            int32_t sum = 0;
            for (int i = 0; i < 128; ++i) {
                args.tab.pre[i] = i < n ? sum : INT32_MAX;
                if (i < n)
                    sum += pass == 0 ? segs[i] - 1 : segs[i];
            }
            e = pass == 0 ? launch_part(&lin_state_kernel<T, DK, NW>, 64 * NW, SM::kState + SM::C * 4, allow_state,
                                        args, states * groups, s)
                          : launch_part(&lin_scan_kernel<T, DK, NW>, 64 * NW, SM::kScanBytes, allow_scan,
                                        args, items * groups, s);
            if (e != hipSuccess)
                return e;
            if (pass == 0 && args.chained) {
                lin_chain_kernel<DK><<<dim3((unsigned)(n * (args.Hv * args.dv * (DK / 64) / 16))), dim3(256), 0, s>>>(args);
                if ((e = hipGetLastError()) != hipSuccess)
                    return e;
            }
        }
    }
    return hipSuccess;
}

template <typename T, int DK>
hipError_t scan_cols(int cols, LinArgs &args, int64_t nseq, const LinSeq *seqs, hipStream_t s)
{
    if constexpr (DK <= 128)   // (256 keys by 128 columns do not fit the LDS)
        if (cols == 128)
            return scan<T, DK, 4>(args, nseq, seqs, s);
    return scan<T, DK, 2>(args, nseq, seqs, s);
}

// ---------------------------------------------------------------------------
// One token per sequence
// ---------------------------------------------------------------------------
// A work-group takes CT columns of one value head's state: each lane four
// consecutive columns of DK / (4 RPI) rows.  The state is read once and written
// once; every element is updated, stored, and added to its column's output sum
// from the same register.  Bound by memory: 256 sequences of 32 heads of 128 x 128
// (1.08 GB) in 184 us, 5.9 TB/s.
constexpr int kStepThreads = 256;
// State above the 256 MB memory-side cache streams through HBM on every step:
// its accesses carry non-temporal hints; a smaller one stays cache-resident.
constexpr int64_t kStepNTBytes = 256ll << 20;

template <bool kNT> __device__ __forceinline__ f32x4 step_ld(const float *p)
{
    if constexpr (kNT)
        return __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p));
    return *reinterpret_cast<const f32x4 *>(p);
}
template <bool kNT> __device__ __forceinline__ void step_st(float *p, f32x4 v)
{
    if constexpr (kNT)
        __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(p));
    else
        *reinterpret_cast<f32x4 *>(p) = v;
}

template <typename T, int DK, int CT, bool kNT>
__global__ __launch_bounds__(kStepThreads) void lin_step_kernel(
    int Hk, int Hv, int dv, int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
    const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
    const float *__restrict__ g, float *__restrict__ state, T *__restrict__ o)
{
    constexpr int LPR = CT / 4, RPI = 64 / LPR, ROWS = DK / (4 * RPI);
    static_assert(ROWS * 4 * RPI == DK, "rows split over 4 waves x RPI");
    __shared__ f32x4 part[4][LPR];
    const int tiles = dv / CT;
    const int64_t bj = blockIdx.x / (unsigned)tiles;
    const int tile = blockIdx.x % (unsigned)tiles;
    const int64_t b = bj / Hv;
    const int j = (int)(bj - b * Hv), i = j / (Hv / Hk);
    const int tid = threadIdx.x, w = uniform_int(tid >> 6), lane = tid & 63;
    const int lg = lane / LPR, lc = lane % LPR;
    const int c0 = tile * CT + 4 * lc, r0 = (w * RPI + lg) * ROWS;

    float *S = state + (bj * DK + r0) * dv + c0;
    f32x4 s[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
        s[r] = step_ld<kNT>(S + (int64_t)r * dv);
    const T *qi = q + b * q_stride + (int64_t)i * DK + r0, *ki = k + b * k_stride + (int64_t)i * DK + r0;
    const T *vj = v + b * v_stride + (int64_t)j * dv + c0;
    f32x4 vv;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        vv[e] = (float)vj[e];
    const float lam = pow_of(std::max(g[j] * kLog2e, -1e5), 1.0);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const float kr = (float)ki[r], qr = (float)qi[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[r][e] = __builtin_fmaf(lam, s[r][e], kr * vv[e]);
            acc[e] = __builtin_fmaf(qr, s[r][e], acc[e]);
        }
        step_st<kNT>(S + (int64_t)r * dv, s[r]);
    }
    // sum over the wave's row groups, then over the waves
#pragma unroll
    for (int off = 32; off >= LPR; off >>= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[e] += __shfl_xor(acc[e], off, 64);
    if (lg == 0)
        part[w][lc] = acc;
    __syncthreads();
    if (tid < LPR) {
        const f32x4 t = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
        T *oj = o + bj * dv + tile * CT + 4 * tid;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            oj[e] = (T)(t[e] * scale);
    }
}

template <typename T, int DK>
hipError_t step(int64_t B, int64_t Hk, int64_t Hv, int64_t dv, int64_t qs, int64_t ks, int64_t vs,
                float scale, const void *q, const void *k, const void *v, const float *g, float *state,
                void *o, hipStream_t s)
{
    // few heads: narrow column tiles, so that more work-groups share the state (32
    // heads of 128 x 128: 3.4 us)
    const bool nt = B * Hv * DK * dv * 4 > kStepNTBytes;
    const int ct = B * Hv * (dv / 64) >= 1024 ? 64 : 32;
    const dim3 grid((unsigned)(B * Hv * (dv / ct)));
#define SSD_LIN_STEP(CT, NT)                                                                       \
    lin_step_kernel<T, DK, CT, NT><<<grid, dim3(kStepThreads), 0, s>>>(                            \
        (int)Hk, (int)Hv, (int)dv, qs, ks, vs, scale, (const T *)q, (const T *)k, (const T *)v, g, \
        state, (T *)o)
    if (ct == 64) {
        if (nt)
            SSD_LIN_STEP(64, true);
        else
            SSD_LIN_STEP(64, false);
    } else {
        if (nt)
            SSD_LIN_STEP(32, true);
        else
            SSD_LIN_STEP(32, false);
    }
#undef SSD_LIN_STEP
    return hipGetLastError();
}

}  // namespace

// Segment length and column tile by a model of the two launches.  A work-group's
// 32-token tile takes at least `chain` us (its own dependent steps), and with the
// chip's slots full at least slots x `rate` us (memory: the bytes of a tile at
// 4.8 TB/s, q and k once per head group; or the matrix and vector work).  A launch
// runs in rounds of `slots` work-groups; a chained state costs its reader 1, 2.5 or 6
// us at 64, 128 and 256 keys, unless lin_chain_kernel has joined them, which moves
// every slot three times over (with the state kernel's writes).  Measured at 4 x 8192
// tokens (32 heads of 128 x 128, bf16, 512 slots): 259 us with 4 segments per sequence
// (one round of the scan) against 285 with 8 and 304 with 2; at 8 x 2048 (24 heads of
// 128 x 64, 768 slots): 73 us with 4 against 103 with 2 and 88 with 8; one sequence of
// 13384 (4 heads of 256 x 64): 79 us with 84 or more, 207 with 16.
LinPlan plan_linattn(int bf16, int64_t nseq, const LinSeq *seqs, int64_t Hk, int64_t Hv, int64_t dk,
                     int64_t dv)
{
    // the lengths, runs of equal ones taken together: the host's time grows with their
    // number
    std::vector<std::pair<uint32_t, int64_t>> lens;
    int64_t longest = 0;
    for (int64_t i = 0; i < nseq; ++i) {
        longest = std::max(longest, seqs[i].len);
        if (lens.empty() || lens.back().first != (uint32_t)seqs[i].len)
            lens.emplace_back((uint32_t)seqs[i].len, 0);
        ++lens.back().second;
    }
    LinPlan best = {};
    double best_us = 1e300;
    const int64_t esz = bf16 ? 2 : 4;
    const int64_t trials = std::clamp<int64_t>(4096 / std::max<int64_t>(1, (int64_t)lens.size()), 16, 128);
    const int64_t kmax = std::max<int64_t>(1, std::min<int64_t>(trials, (longest + 31) / 32));
    for (int cols = dv % 128 == 0 && dk <= 128 ? 128 : 64; cols >= 64; cols /= 2) {
        const int64_t heads = Hv * (dv / cols);
        // work-groups of a CU: by LDS, and by registers (8 waves; 4 of the large heads
        // and of fp32)
        const int64_t nw = cols / 32;
        const int64_t per_cu = std::max<int64_t>(
            1, std::min<int64_t>((bf16 && dk <= 128 ? 8 : 4) / nw, 160 * 1024 / scan_lds(bf16, dk, cols)));
        const double slots = 256.0 * per_cu, w = dk / 128.0, waves = (double)nw;
        const double chain = !bf16 ? 1.8 + 4.6 * w : dk <= 128 ? 0.6 + 0.9 * w : 5.8;
        const double chain_state = !bf16 ? 0.7 + 2.4 * w : dk <= 128 ? 0.4 + 0.6 * w : 3.5;
        const double chain_slot = dk == 64 ? 1.0 : dk == 128 ? 2.5 : 6.0;
        const double shared = (double)dk * Hk / Hv;       // q (or k) columns a work-group pays for
        const double us_byte = 1.0 / 4.8e6;
        const double rate = std::max(32 * esz * (2 * shared + 2 * cols) * us_byte,
                                     (bf16 ? 0.9e-3 : 4e-3) * waves * w);
        const double rate_state = std::max(32 * esz * (shared + cols) * us_byte,
                                           (bf16 ? 0.7e-3 : 2e-3) * waves * w);
        for (int64_t k = 1; k <= kmax; ++k) {
            const int64_t T0 = std::max<int64_t>(32, ((longest + k - 1) / k + 31) / 32 * 32);
            int64_t segs = 0, slot = 0;
            for (const auto &[len, count] : lens) {
                const int64_t ns = std::max<int64_t>(1, (len + (uint32_t)T0 - 1) / (uint32_t)T0);
                segs += count * ns;
                slot += ns > 1 ? count * ns : 0;
            }
            // rounds of a launch of n work-groups of at most T0 tokens (a partly filled
            // one gains about half of what it leaves free)
            auto launch = [&](double n, double ch, double rt) {
                const double tiles = T0 / 32.0, full = (double)(int64_t)(n / slots);
                const double rest = n - full * slots;
                return tiles * (full * std::max(ch, slots * rt) +
                                (rest > 0 ? std::max(ch, 0.5 * (slots + rest) * rt) : 0.0));
            };
            double us = launch((double)(segs * heads), chain, rate);
            if (segs > nseq) {
                const int64_t prior = (longest + T0 - 1) / T0 - 1;
                us += 4.0 + launch((double)((segs - nseq) * heads), chain_state, rate_state);
                if (prior * dk >= kChain)
                    us += 9.0 + 0.3 * (double)prior + 3.0 * (double)(slot * Hv * dk * dv * 4) * us_byte;
                else
                    us += chain_slot * (double)prior;
            }
            if (us < best_us) {
                best_us = us;
                best.seg_tokens = T0;
                best.nslot = slot;
                best.cols = cols;
            }
        }
    }
    best.ws_bytes = (size_t)(best.nslot * Hv * dk * dv * 4);
    return best;
}

hipError_t launch_linattn_scan(int bf16, const LinPlan &plan, int64_t nseq, const LinSeq *seqs,
                               int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t q_stride,
                               int64_t k_stride, int64_t v_stride, float scale, const void *q,
                               const void *k, const void *v, const float *log_decay,
                               const float *init, void *o, float *fin, void *ws, hipStream_t s)
{
    LinArgs args = {};
    args.q = q;
    args.k = k;
    args.v = v;
    args.g = log_decay;
    args.init = init;
    args.o = o;
    args.fin = fin;
    args.ws = static_cast<float *>(ws);
    args.q_stride = q_stride;
    args.k_stride = k_stride;
    args.v_stride = v_stride;
    args.seg_tokens = (int32_t)plan.seg_tokens;
    args.Hk = (int32_t)Hk;
    args.Hv = (int32_t)Hv;
    args.dv = (int32_t)dv;
    args.scale = scale;
    args.copy_init = init != nullptr && init == fin;
    if (bf16) {
        switch (dk) {
        case 64: return scan_cols<__bf16, 64>(plan.cols, args, nseq, seqs, s);
        case 128: return scan_cols<__bf16, 128>(plan.cols, args, nseq, seqs, s);
        case 256: return scan_cols<__bf16, 256>(plan.cols, args, nseq, seqs, s);
        }
    } else {
        switch (dk) {
        case 64: return scan_cols<float, 64>(plan.cols, args, nseq, seqs, s);
        case 128: return scan_cols<float, 128>(plan.cols, args, nseq, seqs, s);
        case 256: return scan_cols<float, 256>(plan.cols, args, nseq, seqs, s);
        }
    }
    return hipErrorInvalidValue;
}

hipError_t launch_linattn_decode(int bf16, int64_t B, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv,
                                 int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                                 const void *q, const void *k, const void *v,
                                 const float *log_decay, float *state, void *o, hipStream_t s)
{
    if (bf16) {
        switch (dk) {
        case 64: return step<__bf16, 64>(B, Hk, Hv, dv, q_stride, k_stride, v_stride, scale, q, k, v, log_decay, state, o, s);
        case 128: return step<__bf16, 128>(B, Hk, Hv, dv, q_stride, k_stride, v_stride, scale, q, k, v, log_decay, state, o, s);
        case 256: return step<__bf16, 256>(B, Hk, Hv, dv, q_stride, k_stride, v_stride, scale, q, k, v, log_decay, state, o, s);
        }
    } else {
        switch (dk) {
        case 64: return step<float, 64>(B, Hk, Hv, dv, q_stride, k_stride, v_stride, scale, q, k, v, log_decay, state, o, s);
        case 128: return step<float, 128>(B, Hk, Hv, dv, q_stride, k_stride, v_stride, scale, q, k, v, log_decay, state, o, s);
        case 256: return step<float, 256>(B, Hk, Hv, dv, q_stride, k_stride, v_stride, scale, q, k, v, log_decay, state, o, s);
        }
    }
    return hipErrorInvalidValue;
}

}  // namespace ssd
