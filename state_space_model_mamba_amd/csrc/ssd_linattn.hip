// Linear attention with one decay per head on gfx950: the chunked form over
// prompts (batched or packed) and the recurrent step for single tokens.
//
// Per value head j with query/key head i = j / (Hv / Hk) and lambda = e^g_j:
//     S_t = lambda S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t       (S: dk x dv, fp32)
// Over a tile of n tokens entered with state S (t, s = 0 .. n - 1):
//     o_t = scale (lambda^(t+1) S^T q_t + sum_{s<=t} lambda^(t-s) (q_t . k_s) v_s)
//     S  <- lambda^n S + sum_s lambda^(n-1-s) k_s v_s^T
// The decay is the same for every token, so the state is kept as R with
// S = lambda^e R, e the tokens since the last rescale: a tile then adds
// lambda^-(e+s+1) k_s v_s^T to R without touching the rest of it, and R is
// multiplied by lambda^e only when that falls below 2^-kEpoch (kEpoch = 24: the
// weights stay within 2^24, and rescales, whose rounding would add up over the
// tiles of a slowly forgetting head, are a memory length apart).  A head that
// forgets faster than 2^-kEpoch within a tile is scaled every tile instead.
// Powers of lambda are formed from the exponent in fp64 (fp32 would be off by
// up to kEpoch 2^-24 relative).
//
// Rounding (bf16): q, k, v are exact operands.  The state and the masked scores
// are each rounded once to bf16 on their way into the products that form o
// (each about as large as the rounding of o itself); the state update takes
// lambda^.. v as the sum of three bf16 numbers, which hold an fp32 product
// whole: the fp32 state keeps fp32 accuracy (two left it 2.5e-6 off, relative).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ssd_attn.h"
#include "ssd_mma.h"

namespace ssd {
namespace {

using namespace mx;

constexpr double kLog2e = 1.4426950408889634;
constexpr float kEpoch = 24.f;

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

template <typename T> struct LinGeom {
    static constexpr int C = sizeof(T) == 2 ? 64 : 32;    // tokens per tile
};

template <typename T, int DK, int NW> struct LinSmem {
    static constexpr int C = LinGeom<T>::C, CT = 32 * NW;
    static constexpr int kK = C * DK * (int)sizeof(T), kV = C * CT * (int)sizeof(T);
    static constexpr int kP = C * C * (int)sizeof(T);
    static constexpr int kScanSlot = 2 * kK + kV, kStateSlot = kK + kV;
    static constexpr int kScan = 2 * kScanSlot + kP, kState = 2 * kStateSlot;
};

// v * u, rounded to fp32, as the sum of three bf16 numbers.
__device__ __forceinline__ void weigh(bf16x8 v, const f32x4 &u0, const f32x4 &u1, bf16x8 (&x)[3])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float p = (float)v[e] * (e < 4 ? u0[e & 3] : u1[e & 3]);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            x[i][e] = (__bf16)p;
            p -= (float)x[i][e];
        }
    }
}

// The work of one segment of one (sequence, value head, column tile): with
// kScan, o over the segment (and the end state for a sequence's last segment);
// without, its end state into the workspace.
//
// A wave owns 32 value columns: its dk x 32 slice of R stays in the result
// registers and is the operand of the state product as it stands (contraction
// over its rows), and the scores of a tile, the same for all columns, are shared
// through LDS.  Outputs are formed transposed (columns x tokens): a lane holds
// one token, so its power of lambda is one per-lane factor.
template <typename T, int DK, int NW, bool kScan>
__global__ __launch_bounds__(64 * NW) void lin_scan_kernel(LinArgs args_in_kernarg)
{
    typedef LinSmem<T, DK, NW> SM;
    constexpr int C = SM::C, TB = C / 32, CT = SM::CT, DB = DK / 32;
    constexpr int E = Piece<T>::E, PB = 16 / E;           // pieces per 32-row block
    constexpr int PT = C / (2 * E);                       // pieces over a tile's tokens
    typedef Tile<T, DK> TK;
    typedef Tile<T, CT> TV;
    typedef Tile<T, C> TP;
    typedef typename Piece<T>::V V;
    constexpr int kStores = kScan ? TB * (sizeof(T) == 2 ? 2 : 4) : 0;   // per wave and tile
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(16) float su[NW][C];             // the tokens' update weights

    const LinArgsPtr a = (LinArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    const int tid = threadIdx.x, lane = tid & 63, w = uniform_int(tid >> 6);
    const int cl = lane & 31, hh = lane >> 5;

    // value heads of a query/key head, and their column tiles, next to each other
    // on one XCD: they read the same q and k
    const unsigned nb = gridDim.x, per = nb / 8;
    const unsigned bid = blockIdx.x < per * 8 ? (blockIdx.x % 8) * per + blockIdx.x / 8 : blockIdx.x;
    const int Hv = a->Hv, nct = a->dv / CT, hc = Hv * nct;
    const int item = (int)(bid / (unsigned)hc), hx = (int)(bid % (unsigned)hc);
    const int head = hx / nct, ct = hx % nct, hk = head / (Hv / a->Hk);
    const int below = __popcll(__ballot(a->tab.pre[lane] <= item)) +
                      __popcll(__ballot(a->tab.pre[64 + lane] <= item));
    const int si = uniform_int(below - 1);
    const int seg = item - a->tab.pre[si];
    const int len = a->tab.len[si], T0 = a->seg_tokens;
    const int nseg = std::max(1, (len + T0 - 1) / T0);
    const int beg = seg * T0, end = std::min(len, beg + T0);
    const int64_t sid = a->tab.id[si];
    const double g2 = std::max(a->g[head] * kLog2e, -1e5);
    const float g2f = (float)g2;
    const int col0 = ct * CT + 32 * w;                    // the wave's first column of dv
    const int dv = a->dv;

    const T *qp = (const T *)a->q + a->tab.tok[si] * a->q_stride + (int64_t)hk * DK;
    const T *kp = (const T *)a->k + a->tab.tok[si] * a->k_stride + (int64_t)hk * DK;
    const T *vp = (const T *)a->v + a->tab.tok[si] * a->v_stride + (int64_t)head * dv + ct * CT;
    const int64_t sbase = (sid * Hv + head) * (int64_t)DK * dv + col0 + cl;   // of init and fin
    const int64_t frag = (int64_t)DK * CT;                // floats of a slot's (head, column tile)
    float *wsp = a->ws + (((int64_t)a->tab.slot[si] * Hv + head) * nct + ct) * frag +
                 w * (DK * 32) + lane * 4;
    const int64_t wslot = (int64_t)Hv * nct * frag;

    f32x16 R[DB];
    // ---- the state entering the segment ----
    const bool use_init = a->init != nullptr;
    auto from_ws = [&](int j, float f) {                  // R = f R + slot j
        const float *p = wsp + j * wslot;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 z = *reinterpret_cast<const f32x4 *>(p + (d * 4 + g) * 256);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    R[d][4 * g + e] = __builtin_fmaf(R[d][4 * g + e], f, z[e]);
            }
    };
    auto to_ws = [&](int j, float f) {
        float *p = wsp + j * wslot;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<f32x4 *>(p + (d * 4 + g) * 256) =
                    f32x4{R[d][4 * g] * f, R[d][4 * g + 1] * f, R[d][4 * g + 2] * f, R[d][4 * g + 3] * f};
    };
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            R[d][r] = 0.f;
    if (seg == 0) {
        if (kScan && a->copy_init && nseg > 1) {
            from_ws(nseg - 1, 0.f);
        } else if (use_init) {
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    R[d][r] = a->init[sbase + (int64_t)(32 * d + 8 * (r >> 2) + 4 * hh + (r & 3)) * dv];
        }
        if (!kScan && a->copy_init)
            to_ws(nseg - 1, 1.f);
    } else if (kScan) {
        // slot 0 holds the state after segment 0 (the initial one included), slot
        // j segment j's from zero; those forgotten below 2^-150 are left out
        const float fT = pow_of(g2, T0);
        int j = 0;
        while (j < seg - 1 && g2f * (float)T0 * (float)(seg - 1 - j) < -150.f)
            ++j;
        for (; j < seg; ++j)
            from_ws(j, fT);
    }

    const unsigned lds0 = lds_addr(smem);
    constexpr int kSlot = kScan ? SM::kScanSlot : SM::kStateSlot;
    auto issue = [&](int t0, int slot) {
        unsigned dst = lds0 + slot * kSlot;
        TileLoad<T, DK, C, NW>::issue(dst, kp, a->k_stride, t0, end, w, lane);
        TileLoad<T, CT, C, NW>::issue(dst + SM::kK, vp, a->v_stride, t0, end, w, lane);
        if constexpr (kScan)
            TileLoad<T, DK, C, NW>::issue(dst + SM::kK + SM::kV, qp, a->q_stride, t0, end, w, lane);
    };

    const bool direct = -g2f * (float)C > kEpoch || g2f > 0.f;   // scaled every tile
    const float scale = a->scale;
    int e = 0;                                            // S = lambda^e R
    if (beg < end)
        issue(beg, 0);
    bool first = true;
    for (int t0 = beg, n = 0; t0 < end; t0 += C, ++n) {
        const int rows = std::min(C, end - t0);
        // this wave's share of the tile has landed (the last tile's stores, issued
        // after its loads, may still be on their way), then everyone's has
        if (first)
            wait_vmcnt<0>();
        else
            wait_vmcnt<kStores>();
        first = false;
        lds_barrier();
        if (t0 + C < end)
            issue(t0 + C, (n + 1) & 1);
        const unsigned char *Kt = smem + (n & 1) * kSlot, *Vt = Kt + SM::kK, *Qt = Vt + SM::kV;
        unsigned char *Pt = smem + 2 * SM::kScanSlot;

        if (!direct && e > 0 && -g2f * (float)(e + C) > kEpoch) {
            const float f = pow_of(g2, e);
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    R[d][r] *= f;
            e = 0;
        }
        // update weights of the tile's tokens (lane = token), 0 past the end
        if (lane < C)
            su[w][lane] = lane < rows ? (direct ? pow_of(g2, rows - 1 - lane) : pow_of(g2, -(e + lane + 1)))
                                      : 0.f;

        V vf[PT];
        if constexpr (kScan) {
            // masked scores (transposed: s x t): one 32 x 32 block per wave
            constexpr int kBlocks = TB * (TB + 1) / 2;
            for (int blk = w; blk < kBlocks; blk += NW) {
                const int tb = blk == 0 ? 0 : 1, sb = blk == 2 ? 1 : 0;
                f32x16 p = {};
#pragma unroll
                for (int i = 0; i < TK::kPieces; ++i)
                    p = mma(TK::row_nat(Kt, 32 * sb + cl, i, hh), TK::row_nat(Qt, 32 * tb + cl, i, hh), p);
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int d = 32 * (tb - sb) + cl - (8 * (r >> 2) + 4 * hh + (r & 3));   // t - s
                    p[r] = d < 0 ? 0.f : p[r] * (scale * exp2_fast(g2f * (float)d));
                }
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    unsigned char *dst = Pt + TP::off(32 * tb + cl, (32 * sb + 8 * g) * (int)sizeof(T) / 16);
                    if constexpr (sizeof(T) == 2)
                        *reinterpret_cast<uint2 *>(dst + 8 * hh) =
                            make_uint2(pack_bf16(p[4 * g], p[4 * g + 1]), pack_bf16(p[4 * g + 2], p[4 * g + 3]));
                    else
                        *reinterpret_cast<f32x4 *>(
                            Pt + TP::off(32 * tb + cl, (32 * sb + 8 * g + 4 * hh) / 4)) =
                            f32x4{p[4 * g], p[4 * g + 1], p[4 * g + 2], p[4 * g + 3]};
                }
            }
            // the state's part
            f32x16 y[TB] = {};
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int i = 0; i < PB; ++i) {
                    const V rf = acc_piece(R[d], i, (const T *)nullptr);
#pragma unroll
                    for (int tb = 0; tb < TB; ++tb)
                        y[tb] = mma(rf, TK::row_acc(Qt, 32 * tb + cl, d * PB + i, hh), y[tb]);
                }
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
                const float f = scale * pow_of(g2, (direct ? 0 : e) + 32 * tb + cl + 1);
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    y[tb][r] *= f;
            }
#pragma unroll
            for (int i = 0; i < PT; ++i)
                vf[i] = TV::col_acc(Vt, i, 32 * w, lane);
            lds_barrier();                                // the scores are there
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int i = 0; i < (tb + 1) * PB; ++i)
                    y[tb] = mma(vf[i], TP::row_acc(Pt, 32 * tb + cl, i, hh), y[tb]);
            // stores through a descriptor that ends at the segment's last row: always the
            // same number of store instructions (see the wait above)
            T *ob = (T *)a->o + ((a->tab.tok[si] + t0) * Hv + head) * (int64_t)dv + col0;
            const unsigned ostride = (unsigned)(Hv * dv * (int)sizeof(T));
            const __amdgpu_buffer_rsrc_t orr = __builtin_amdgcn_make_buffer_rsrc(
                ob, (short)0, (int)((unsigned)(rows - 1) * ostride + 32 * (unsigned)sizeof(T)), 0x00020000);
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
                // a row past the last lies past the descriptor's end whatever the column
                const unsigned ro = (unsigned)(32 * tb + cl) * ostride;
                if constexpr (sizeof(T) == 2) {
#pragma unroll
                    for (int g = 0; g < 4; g += 2) {
                        unsigned out[4];
#pragma unroll
                        for (int h2 = 0; h2 < 2; ++h2) {
                            const auto sw = __builtin_amdgcn_permlane32_swap(
                                pack_bf16(y[tb][4 * g + 2 * h2], y[tb][4 * g + 2 * h2 + 1]),
                                pack_bf16(y[tb][4 * g + 4 + 2 * h2], y[tb][4 * g + 5 + 2 * h2]), false, false);
                            out[h2] = sw[0];
                            out[2 + h2] = sw[1];
                        }
                        __builtin_amdgcn_raw_buffer_store_b128(u32x4{out[0], out[1], out[2], out[3]}, orr,
                                                               ro + (unsigned)(8 * g + 8 * hh) * 2u, 0, 0);
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        __builtin_amdgcn_raw_buffer_store_b128(
                            __builtin_bit_cast(u32x4, f32x4{y[tb][4 * g], y[tb][4 * g + 1], y[tb][4 * g + 2],
                                                            y[tb][4 * g + 3]}),
                            orr, ro + (unsigned)(8 * g + 4 * hh) * 4u, 0, 0);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < PT; ++i)
                vf[i] = TV::col_acc(Vt, i, 32 * w, lane);
        }

        // the state update
        if (direct) {
            const float f = pow_of(g2, rows);
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    R[d][r] *= f;
        } else {
            e += rows;
        }
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            if constexpr (sizeof(T) == 2) {
                const f32x4 u0 = *reinterpret_cast<const f32x4 *>(&su[w][16 * i + 4 * hh]);
                const f32x4 u1 = *reinterpret_cast<const f32x4 *>(&su[w][16 * i + 8 + 4 * hh]);
                V x[3];
                weigh(vf[i], u0, u1, x);
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    const V kf = TK::col_acc(Kt, i, 32 * d, lane);
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        R[d] = mma(kf, x[j], R[d]);
                }
            } else {
                const f32x4 u = *reinterpret_cast<const f32x4 *>(&su[w][8 * i + 4 * hh]);
                const V x = vf[i] * u;
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    R[d] = mma(TK::col_acc(Kt, i, 32 * d, lane), x, R[d]);
            }
        }
    }

    if constexpr (kScan) {
        if (seg == nseg - 1) {
            const float f = pow_of(g2, e);
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    a->fin[sbase + (int64_t)(32 * d + 8 * (r >> 2) + 4 * hh + (r & 3)) * dv] = R[d][r] * f;
        }
    } else {
        to_ws(seg, pow_of(g2, e));
    }
}

template <typename T, int DK, int NW, bool kScan>
hipError_t launch_part(const LinArgs &args, int64_t items, hipStream_t s)
{
    typedef LinSmem<T, DK, NW> SM;
    constexpr int kSmem = kScan ? SM::kScan : SM::kState;
    static_assert(kSmem + NW * SM::C * 4 <= 160 * 1024, "LDS of a CU");
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void *>(&lin_scan_kernel<T, DK, NW, kScan>),
        hipFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != hipSuccess)
        return e;
    const int64_t grid = items * args.Hv * (args.dv / (32 * NW));
    lin_scan_kernel<T, DK, NW, kScan><<<dim3((unsigned)grid), dim3(64 * NW), kSmem, s>>>(args);
    return hipGetLastError();
}

template <typename T, int DK, int NW>
hipError_t scan(LinArgs &args, int64_t nseq, const LinSeq *seqs, hipStream_t s)
{
    const int64_t T0 = args.seg_tokens;
    const int64_t most = INT32_MAX / ((int64_t)args.Hv * (args.dv / (32 * NW)));
    int64_t slot = 0;
    for (int64_t at = 0; at < nseq;) {
        int n = 0;
        int64_t items = 0, states = 0;
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
            ++n;
            ++at;
        }
        if (n == 0)
            return hipErrorInvalidValue;
        hipError_t e;
        for (int pass = states > 0 ? 0 : 1; pass < 2; ++pass) {
            int32_t sum = 0;
            for (int i = 0; i < 128; ++i) {
                args.tab.pre[i] = i < n ? sum : INT32_MAX;
                if (i < n)
                    sum += pass == 0 ? segs[i] - 1 : segs[i];
            }
            e = pass == 0 ? launch_part<T, DK, NW, false>(args, states, s)
                          : launch_part<T, DK, NW, true>(args, items, s);
            if (e != hipSuccess)
                return e;
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
// from the same register.
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
    // few heads: narrow column tiles, so that more work-groups share the state
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

LinPlan plan_linattn(int bf16, int64_t nseq, const LinSeq *seqs, int64_t Hk, int64_t Hv, int64_t dk,
                     int64_t dv)
{
    LinPlan p = {};
    p.cols = dv % 128 == 0 && dk <= 128 ? 128 : 64;
    const int64_t heads = Hv * (dv / p.cols);
    int64_t total = 0, longest = 0;
    for (int64_t i = 0; i < nseq; ++i) {
        total += seqs[i].len;
        longest = std::max(longest, seqs[i].len);
    }
    const int64_t tile = bf16 ? 64 : 32;
    // work-groups wanted: one per CU
    int64_t T0 = total * heads / 256;
    T0 = std::max<int64_t>(4 * tile, (T0 + tile - 1) / tile * tile);
    T0 = std::min(T0, (std::max<int64_t>(longest, 1) + tile - 1) / tile * tile);
    p.seg_tokens = T0;
    for (int64_t i = 0; i < nseq; ++i) {
        const int64_t ns = (seqs[i].len + T0 - 1) / T0;
        p.nslot += ns > 1 ? ns : 0;
    }
    p.ws_bytes = (size_t)(p.nslot * Hv * dk * dv * 4);
    return p;
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
