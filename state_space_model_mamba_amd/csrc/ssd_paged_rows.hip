// Rows of queries, keys and values on their way into a softmax layer and into its paged
// cache, and back (gfx950).
//
// Norm and rotation.  For a head x of D values of a token at position t, with weights w:
//     n = x w / sqrt(mean(x^2) + eps)
//     (n_a, n_b) <- (n_a cos f_i t - n_b sin f_i t, n_b cos f_i t + n_a sin f_i t)
// for the pairs (a, b) = (i, i + R / 2) or (2 i, 2 i + 1), i < R / 2.  Everything is
// fp32 but the angle: f_i t is formed in fp64 in turns and reduced to half a turn there
// (in fp32 it would be off by 2^-24 of itself, a hundredth of a radian at t = 131072).
// Results are rounded once, to the output type.
//
// 4-bit rows.  Every 64 values of a row have a least value m = f16(min) and a step
// s = f16((max - min) / 15), the fifteenth as a product with 1/15 in fp32 (as torch divides by
// a number); code = round((x - m) / s) in 0 .. 15, value = code s + m.
// Half precision holds the pair in a dword and is an operand of the mixed-precision
// multiply-add as it stands; its 11 bits keep the codes' range within 1% of a step.  A NaN
// among the values makes both NaN, infinities of one sign alone the step (inf - inf): the
// group comes back as NaN, as it would by the formula.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ssd_mma.h"
#include "ssd_paged.h"

namespace ssd {
namespace {

using namespace mx;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kHalfMax = 65504.f;
constexpr int kGroup = 64;                    // 4-bit values that share a step and a least value

// The sequences of a launch (kernel arguments: 4 KB).
struct RowTab {
    static constexpr int kMax = 120;
    int64_t tok[kMax];                        // first packed token
    int32_t row[kMax], n[kMax];               // first row in the cache (gather), tokens
    int32_t pre[128];                         // first unit of each sequence; then INT32_MAX
};

// The sequence of unit `u`.
template <typename Tab> __device__ __forceinline__ int seq_of(const Tab &tab, int u, int lane)
{
    return uniform_int(__popcll(__ballot(tab.pre[lane] <= u)) +
                       __popcll(__ballot(tab.pre[64 + lane] <= u)) - 1);
}

// Page of a row, or -1 where the table has none.
__device__ __forceinline__ int page_of(const PagedCache &c, int64_t b, int64_t row)
{
    if (row < 0 || (row >> c.shift) >= c.max_pages)
        return -1;
    const int page = c.table[b * c.max_pages + (row >> c.shift)];
    return page >= 0 && page < c.num_pages ? page : -1;
}

template <int kCtrl> __device__ __forceinline__ float dpp(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl,
                                                                 0xf, 0xf, true));
}
// Reduces over kLanes (8, 16 or 32) neighbouring lanes; all of them get the result.
template <int kLanes, typename Op> __device__ __forceinline__ float across(float v, Op op)
{
    v = op(v, dpp<0xb1>(v));                  // lane ^ 1
    v = op(v, dpp<0x4e>(v));                  // lane ^ 2
    v = op(v, dpp<0x141>(v));                 // 7 - lane of 8: the other four
    if constexpr (kLanes > 8)
        v = op(v, dpp<0x140>(v));             // 15 - lane of 16: the other eight
    if constexpr (kLanes > 16)                // lane ^ 16
        v = op(v, __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v), 0x401f)));
    return v;
}

// The lesser and the greater of two numbers, NaN if either is.
__device__ __forceinline__ float least_of(float p, float q)
{
    return __builtin_elementwise_minimum(p, q);
}
__device__ __forceinline__ float most_of(float p, float q)
{
    return __builtin_elementwise_maximum(p, q);
}

// The sum of four squares, each rounded.  A head's fours are then added in pairs, of neighbours
// but where half pairs turn a part of the head: a turned lane's two, R / 2 apart there, come
// first.  With neighbours that is the order of torch's mean for D = 128.  4-bit codes depend on
// the last bits where a value lies between two: with sums in another order, the hardware's
// reciprocal root and sincospif 17 - 28 of 21.7 million (heads turned whole) differed from those
// of the formula written in torch, now none to two (for 3 us in 138).
__device__ __forceinline__ float four_squares(const float *x)
{
#pragma clang fp contract(off)
    return x[0] * x[0] + x[1] * x[1] + x[2] * x[2] + x[3] * x[3];
}

// 1 / sqrt(z), the hardware's estimate and a Newton step whose residual 1 - z y^2 is exact to
// second order.  (0 and infinity: as the estimate; its residual would be NaN.)
__device__ __forceinline__ float rsqrt_near(float z)
{
    const float y = rsqrtf(z), t = z * y;
    const float e = __builtin_fmaf(-__builtin_fmaf(z, y, -t), y, __builtin_fmaf(-t, y, 1.f));
    return fabsf(e) < 1.f ? __builtin_fmaf(0.5f * y, e, y) : y;
}

// Sine and cosine of x turns, |x| <= 1/2: the Taylor series about the nearest quarter turn, with
// the leading terms as sums of two fp32 numbers, so that only their last addition rounds.  (All
// in fp64 the constants' registers make the appends spill: 117 us instead of 106 for 21150 tokens.)
__device__ __forceinline__ void sincos_turns(double x, float &sine, float &cosine)
{
    const double q = __builtin_rint(4.0 * x), ud = 6.283185307179586 * __builtin_fma(-0.25, q, x);
    const float u = (float)ud, ul = (float)(ud - (double)u);
    const float v = u * u, vl = __builtin_fmaf(2.f * u, ul, __builtin_fmaf(u, u, -v));
    float s = __builtin_fmaf(v, -1.f / 39916800, 1.f / 362880);
    s = __builtin_fmaf(v, s, -1.f / 5040);
    s = __builtin_fmaf(v, s, 1.f / 120);
    s = __builtin_fmaf(v, s, -1.f / 6);
    s = u + __builtin_fmaf(u * v, s, ul);
    float c = __builtin_fmaf(v, -1.f / 3628800, 1.f / 40320);
    c = __builtin_fmaf(v, c, -1.f / 720);
    c = __builtin_fmaf(v, c, 1.f / 24);
    const float h = __builtin_fmaf(-0.5f, v, 1.f), hl = __builtin_fmaf(-0.5f, v, 1.f - h);
    c = h + __builtin_fmaf(v * v, c, __builtin_fmaf(-0.5f, vl, hl));
    const int k = (int)q;
    const float a = k & 1 ? c : s, b = k & 1 ? s : c;
    sine = k & 2 ? -a : a;
    cosine = (k + 1) & 2 ? -b : b;
}

// Four values of T.
template <typename T> struct Four;
template <> struct Four<__bf16> {
    typedef uint2 V;
    static __device__ __forceinline__ void open(V u, float *x)
    {
        x[0] = __uint_as_float(u.x << 16);
        x[1] = __uint_as_float(u.x & 0xffff0000u);
        x[2] = __uint_as_float(u.y << 16);
        x[3] = __uint_as_float(u.y & 0xffff0000u);
    }
    static __device__ __forceinline__ V close(const float *x)
    {
        return make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    }
};
template <> struct Four<float> {
    typedef float4 V;
    static __device__ __forceinline__ void open(V u, float *x)
    {
        x[0] = u.x;
        x[1] = u.y;
        x[2] = u.z;
        x[3] = u.w;
    }
    static __device__ __forceinline__ V close(const float *x)
    {
        return make_float4(x[0], x[1], x[2], x[3]);
    }
};

// ---------------------------------------------------------------------------
// Norm, rotation, append
// ---------------------------------------------------------------------------
struct TurnArgs {
    RowTab tab;                               // tok[0]: the launch's first token; row, n: not used
    TurnRows r;
    QkTurn turn;
    PagedCache c;
    const int32_t *lengths;
    int64_t ntok, seq0;                       // tokens and first sequence of the launch
    int one;                                  // one token per sequence: no table
    int chunks, per;                          // work items per token, head groups of each
};
typedef const __attribute__((address_space(4))) TurnArgs *TurnArgsPtr;

enum { kNoPages, kPages, kPages4 };

// A wave takes one token's heads (or a part of them, where there are few tokens), D / 8
// lanes to a head, 8 values to a lane: for halves paired over R / 2 the four at 4 j and
// the four at R / 2 + 4 j, so that a lane has both of a pair and nothing moves between
// lanes but the sum of squares; otherwise 8 j .. 8 j + 7.  The angles' sines and cosines
// are formed once per token and wave, one or two angles to a lane (each lane its own four
// took 8 us more in 138).
//
// Bound by memory: 32768 tokens of 32 + 8 heads of 128 in bf16 take 130 us, 5.2 TB/s (a large
// copy 5.08); with the append of 21150 tokens 107 us, 4.8 TB/s.  Into 4 bits 114 us for 12%
// fewer bytes, the vector units 68% busy and rows of 64 bytes written one by one.  Five waves
// per SIMD in bf16, 96 registers each: with four (102, the compiler's own choice for the 4-bit
// append) it and the reading back took 142 us, with five 138 (now 139, and one register of it
// spills), with six, which spill more, 154.
// One token takes 4.6 us, most of it the look-ups, one after the other.
template <typename T, int D, int kKind>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 5 : 1) void turn_kernel(TurnArgs args_in_kernarg)
{
    constexpr int LPH = D / 8, HW = 64 / LPH; // lanes of a head, heads at once
    constexpr int U = 4;                      // head groups of a round; the next round's loads are in flight
    constexpr int NA = D > 128 ? D / 128 : 1; // angles a lane forms
    typedef Four<T> F;
    __shared__ float ex[kKind == kPages4 ? 4 : 1][kKind == kPages4 ? 512 : 1];

    const TurnArgsPtr a = (TurnArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    const int lane = threadIdx.x & 63, w = uniform_int((int)threadIdx.x >> 6);
    const int j = lane % LPH, hl = lane / LPH;
    const int Hq = (int)a->r.Hq, Hkv = (int)a->r.Hkv;
    const int NH = Hq + (kKind == kNoPages ? Hkv : 2 * Hkv);
    const int rot = a->turn.rot;
    const bool next = a->turn.next != 0, turned = j < rot / 8;
    const bool apart = !next && rot == D;     // a lane's fours lie half a head apart: no neighbours
    const int oa = !next && turned ? 4 * j : 8 * j, ob = !next && turned ? rot / 2 + 4 * j : 8 * j + 4;

    const float *qw = a->turn.q_weight, *kw = a->turn.k_weight;
    float wq[8], wk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int d = (e < 4 ? oa : ob - 4) + e;
        wq[e] = qw ? qw[d] : 1.f;
        wk[e] = kw ? kw[d] : 1.f;
    }
    // angles i = lane + 64 n, each formed by one lane
    double freq[NA];
#pragma unroll
    for (int n = 0; n < NA; ++n)
        freq[n] = lane + 64 * n < rot / 2 ? (double)a->turn.inv_freq[lane + 64 * n] * 0.15915494309189535 : 0.0;
    const float eps = a->turn.eps;

    const int64_t nunit = a->ntok * a->chunks;
    for (int64_t unit = (int64_t)blockIdx.x * 4 + w; unit < nunit; unit += (int64_t)gridDim.x * 4) {
        const int64_t rel = unit / a->chunks;
        const int h0 = (int)(unit % a->chunks) * a->per * HW;
        const int h1 = std::min(NH, h0 + a->per * HW);
        const int64_t t = a->tab.tok[0] + rel;
        const T *qp = (const T *)a->r.q + t * a->r.q_stride, *kp = (const T *)a->r.k + t * a->r.k_stride;
        const T *vp = (const T *)a->r.v + t * a->r.v_stride;
        typename F::V raw[U][2];
        const auto fetch = [&](int hb) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = hb + u * HW + hl;
                if (h < h1) {
                    const T *src = h < Hq ? qp + (int64_t)h * D
                                 : h < Hq + Hkv ? kp + (int64_t)(h - Hq) * D : vp + (int64_t)(h - Hq - Hkv) * D;
                    const bool isv = h >= Hq + Hkv;
                    raw[u][0] = *reinterpret_cast<const typename F::V *>(src + (isv ? 8 * j : oa));
                    raw[u][1] = *reinterpret_cast<const typename F::V *>(src + (isv ? 8 * j + 4 : ob));
                }
            }
        };
        fetch(h0);                            // (ahead of the look-ups, which wait for one another)
        __builtin_amdgcn_sched_barrier(0);
        // where the token goes
        int64_t pos = 0, line = 0;
        bool stored = false;
        if constexpr (kKind != kNoPages) {
            const int si = a->one ? 0 : seq_of(a->tab, (int)rel, lane);
            const int64_t b = a->one ? a->seq0 + rel : a->seq0 + si;
            const int length = a->lengths[b];
            const int64_t row = (int64_t)length + (a->one ? 0 : rel - a->tab.pre[si]);
            const int page = length < 0 ? -1 : page_of(*(const PagedCache *)&a->c, b, row);
            stored = page >= 0;
            line = ((int64_t)std::max(page, 0) * Hkv << a->c.shift) + (row & ((1 << a->c.shift) - 1));
            pos = row;
        }
        if (a->turn.positions)
            pos = a->turn.positions[t];
        float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {};
        if (rot > 0) {
            float c1[NA], s1[NA];
#pragma unroll
            for (int n = 0; n < NA; ++n) {
                const double turns = (double)pos * freq[n];
                sincos_turns(turns - __builtin_rint(turns), s1[n], c1[n]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int from = (4 * j + e) & 63;
                cs[e] = __shfl(c1[0], from, 64);
                sn[e] = __shfl(s1[0], from, 64);
                if constexpr (NA == 2) {
                    const float c2 = __shfl(c1[1], from, 64), s2 = __shfl(s1[1], from, 64);
                    cs[e] = j < 16 ? cs[e] : c2;
                    sn[e] = j < 16 ? sn[e] : s2;
                }
            }
        }

        for (int hb = h0; hb < h1; hb += U * HW) {
            typename F::V now[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                now[u][0] = raw[u][0];
                now[u][1] = raw[u][1];
            }
            if (hb + U * HW < h1)
                fetch(hb + U * HW);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (hb + u * HW >= h1)
                    continue;
                const int h = hb + u * HW + hl;
                const bool live = h < h1, isq = h < Hq, isv = h >= Hq + Hkv;
                float x[8];
                F::open(now[u][0], x);
                F::open(now[u][1], x + 4);
                if (live ? (isq ? qw : isv ? nullptr : kw) != nullptr : false) {
                    const auto add = [](float p, float q) { return p + q; };
                    float ss = four_squares(x);
                    const float s4 = four_squares(x + 4);
                    ss = apart ? across<LPH>(ss, add) + across<LPH>(s4, add) : across<LPH>(ss + s4, add);
                    const float rs = rsqrt_near(ss * (1.f / D) + eps);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = x[e] * rs * (isq ? wq[e] : wk[e]);
                }
                if (turned && !isv) {
#pragma clang fp contract(off)                // (each product rounded: both of a pair alike)
                    if (next) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float p = x[2 * e], q = x[2 * e + 1];
                            x[2 * e] = p * cs[e] - q * sn[e];
                            x[2 * e + 1] = q * cs[e] + p * sn[e];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float p = x[e], q = x[4 + e];
                            x[e] = p * cs[e] - q * sn[e];
                            x[4 + e] = q * cs[e] + p * sn[e];
                        }
                    }
                }
                const int da = isv ? 8 * j : oa, db = isv ? 8 * j + 4 : ob;
                if (live && !isv) {           // packed rows
                    T *dst = isq ? (T *)a->r.q_out + t * a->r.qo_stride + (int64_t)h * D
                                 : (T *)a->r.k_out + t * a->r.ko_stride + (int64_t)(h - Hq) * D;
                    if (isq || a->r.k_out) {
                        *reinterpret_cast<typename F::V *>(dst + da) = F::close(x);
                        *reinterpret_cast<typename F::V *>(dst + db) = F::close(x + 4);
                    }
                }
                if (kKind == kPages && live && !isq && stored) {
                    const int64_t at = line + ((int64_t)(isv ? h - Hq - Hkv : h - Hq) << a->c.shift);
                    T *dst = (T *)(isv ? a->c.v : a->c.k) + at * D;
                    *reinterpret_cast<typename F::V *>(dst + da) = isv ? now[u][0] : F::close(x);
                    *reinterpret_cast<typename F::V *>(dst + db) = isv ? now[u][1] : F::close(x + 4);
                }
                if constexpr (kKind == kPages4) {
                    if (!stored || hb + (u + 1) * HW <= Hq)
                        continue;             // (the whole wave: no keys or values among its heads)
                    // to consecutive values 8 j .. through the wave's own LDS
                    float *m = ex[w] + hl * D;
                    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                    *reinterpret_cast<float4 *>(m + da) = make_float4(x[0], x[1], x[2], x[3]);
                    *reinterpret_cast<float4 *>(m + db) = make_float4(x[4], x[5], x[6], x[7]);
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = m[8 * j + e];
                    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
                    float lo = y[0], hi = y[0];
#pragma unroll
                    for (int e = 1; e < 8; ++e) {
                        lo = least_of(lo, y[e]);
                        hi = most_of(hi, y[e]);
                    }
                    lo = across<8>(lo, least_of);
                    hi = across<8>(hi, most_of);
                    const _Float16 least = (_Float16)least_of(most_of(lo, -kHalfMax), kHalfMax);
                    const _Float16 step = (_Float16)least_of((hi - lo) * (1.f / 15), kHalfMax);
                    const float fl = (float)least, fs = (float)step;
                    // The quotients, rounded as a division rounds them (Markstein's correction: the
                    // residual n - q s, exact, times the refined reciprocal, which is one for all)
                    // and to whole numbers by adding 3 2^22, whose low bits they become: its own
                    // bits, eight times shifted, add up to 0x3f400000.  (A step of 0 or NaN: all
                    // codes 0.)
                    const float est = __builtin_amdgcn_rcpf(fs), top = 15.f * fs;
                    const float inv = __builtin_fmaf(__builtin_fmaf(-fs, est, 1.f), est, est);
                    unsigned codes = 0u - 0x3f400000u;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float n = __builtin_amdgcn_fmed3f(y[e] - fl, 0.f, top), q = n * inv;
                        const float r = __builtin_fmaf(__builtin_fmaf(-q, fs, n), inv, q) + 12582912.f;
                        codes += __float_as_uint(r) << (4 * e);
                    }
                    codes = fs > 0.f ? codes : 0u;
                    if (live && !isq) {
                        const int64_t at = line + ((int64_t)(isv ? h - Hq - Hkv : h - Hq) << a->c.shift);
                        reinterpret_cast<uint32_t *>(isv ? a->c.v : a->c.k)[at * (D / 8) + j] = codes;
                        if (j % 8 == 0)
                            (isv ? a->c.vs : a->c.ks)[at * (D / kGroup) + j / 8] =
                                __builtin_bit_cast(unsigned, f16x2{step, least});
                    }
                }
            }
        }
    }
}

// About 8192 waves when there are few tokens (32 to a CU), whole tokens otherwise.
template <typename T, int D, int kKind> hipError_t turn_launch(TurnArgs &args, hipStream_t s)
{
    constexpr int64_t HW = 512 / D;
    const int64_t heads = args.r.Hq + (kKind == kNoPages ? 1 : 2) * args.r.Hkv;
    const int64_t groups = (heads + HW - 1) / HW;
    const int64_t per = std::clamp<int64_t>(args.ntok * groups / 8192, 1, groups);
    args.per = (int)per;
    args.chunks = (int)((groups + per - 1) / per);
    const int64_t blocks = std::min<int64_t>((args.ntok * args.chunks + 3) / 4, 1 << 20);
    turn_kernel<T, D, kKind><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(args);
    return hipGetLastError();
}

template <int kKind> hipError_t turn_any(int bf16, TurnArgs &args, hipStream_t s)
{
    switch (args.r.D) {
    case 64: return bf16 ? turn_launch<__bf16, 64, kKind>(args, s) : turn_launch<float, 64, kKind>(args, s);
    case 128: return bf16 ? turn_launch<__bf16, 128, kKind>(args, s) : turn_launch<float, 128, kKind>(args, s);
    case 256: return bf16 ? turn_launch<__bf16, 256, kKind>(args, s) : turn_launch<float, 256, kKind>(args, s);
    }
    return hipErrorInvalidValue;
}

// ---------------------------------------------------------------------------
// Rows back from pages
// ---------------------------------------------------------------------------
struct GatherArgs {
    RowTab tab;                               // pre: in blocks of 16 rows
    PagedCache c;
    void *k, *v;
    int64_t seq0, nblk;
    int Hkv;
};
typedef const __attribute__((address_space(4))) GatherArgs *GatherArgsPtr;

// A wave takes 16 consecutive lines of a page (lines 16 n .., of one head) of k or of v:
// contiguous there, one segment per line in the output.  26300 rows of 8 heads of 128 from
// 4 bits to bf16: 26 us, 5.2 TB/s.
template <typename T, int D, bool kQ4>
__global__ __launch_bounds__(256) void gather_kernel(GatherArgs args_in_kernarg)
{
    constexpr int E = kQ4 ? 8 : 16 / (int)sizeof(T);          // values of a lane
    constexpr int LPR = D / E, RW = 64 / LPR, N = 16 / RW;    // lanes of a row, rows at once, steps
    const GatherArgsPtr a = (GatherArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    const int lane = threadIdx.x & 63, w = uniform_int((int)threadIdx.x >> 6);
    const int Hkv = a->Hkv, j = lane % LPR;
    const int64_t nunit = a->nblk * 2 * Hkv;
    for (int64_t unit = (int64_t)blockIdx.x * 4 + w; unit < nunit; unit += (int64_t)gridDim.x * 4) {
        const int hk = (int)(unit % Hkv);
        const int64_t blk = unit / Hkv >> 1;
        const bool isv = (unit / Hkv & 1) != 0;
        const int si = seq_of(a->tab, (int)blk, lane);
        const int first = a->tab.row[si];
        const int64_t r0 = ((int64_t)(first >> 4) + (blk - a->tab.pre[si])) << 4;
        const int page = page_of(*(const PagedCache *)&a->c, a->seq0 + si, r0);
        const int64_t line = ((((int64_t)std::max(page, 0) * Hkv + hk) << a->c.shift)) +
                             (r0 & ((1 << a->c.shift) - 1));
        const int64_t out0 = a->tab.tok[si] + (r0 - first);
        T *op = (T *)(isv ? a->v : a->k);
        const int lo = (int)std::max<int64_t>(0, first - r0),
                  hi = (int)std::min<int64_t>(16, (int64_t)first + a->tab.n[si] - r0);
        uint4 out[N];
        if constexpr (kQ4) {
            uint32_t codes[N], sc[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int64_t at = line + n * RW + lane / LPR;
                codes[n] = page < 0 ? 0u : reinterpret_cast<const uint32_t *>(isv ? a->c.v : a->c.k)[at * (D / 8) + j];
                sc[n] = page < 0 ? 0u : (isv ? a->c.vs : a->c.ks)[at * (D / kGroup) + j / 8];
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const f16x2 s = __builtin_bit_cast(f16x2, sc[n]);
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = __builtin_fmaf((float)(codes[n] >> (4 * e) & 15u), (float)s[0], (float)s[1]);
                const int r = n * RW + lane / LPR;
                if (r < lo || r >= hi)
                    continue;
                T *dst = op + ((out0 + r) * Hkv + hk) * D + 8 * j;
                *reinterpret_cast<typename Four<T>::V *>(dst) = Four<T>::close(x);
                *reinterpret_cast<typename Four<T>::V *>(dst + 4) = Four<T>::close(x + 4);
            }
        } else {
            const uint4 *src = reinterpret_cast<const uint4 *>((const T *)(isv ? a->c.v : a->c.k) + line * D) + lane;
#pragma unroll
            for (int n = 0; n < N; ++n)
                out[n] = page < 0 ? make_uint4(0, 0, 0, 0) : src[n * 64];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int r = n * RW + lane / LPR;
                if (r >= lo && r < hi)
                    *reinterpret_cast<uint4 *>(op + ((out0 + r) * Hkv + hk) * D + E * j) = out[n];
            }
        }
    }
}

template <typename T, int D> hipError_t gather_launch(const GatherArgs &args, hipStream_t s)
{
    const int64_t blocks = std::min<int64_t>((args.nblk * 2 * args.Hkv + 3) / 4, 1 << 20);
    if (args.c.ks)
        gather_kernel<T, D, true><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(args);
    else
        gather_kernel<T, D, false><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(args);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_turn(int bf16, const TurnRows &r, const QkTurn &turn, hipStream_t s)
{
    TurnArgs args = {};
    args.r = r;
    args.turn = turn;
    args.ntok = r.rows;
    return turn_any<kNoPages>(bf16, args, s);
}

hipError_t launch_paged_append(int bf16, int64_t batch, const int64_t *cu, const TurnRows &r,
                               const QkTurn &turn, const PagedCache &cache, const int32_t *lengths,
                               hipStream_t s)
{
    TurnArgs args = {};
    args.r = r;
    args.turn = turn;
    args.c = cache;
    args.lengths = lengths;
    args.one = cu == nullptr;
    for (int64_t at = 0; at < batch;) {
        int64_t n = args.one ? batch : std::min<int64_t>(batch - at, RowTab::kMax);
        args.seq0 = at;
        args.tab.tok[0] = cu ? cu[at] : 0;
        args.ntok = cu ? cu[at + n] - cu[at] : batch;
        if (cu) {
            for (int i = 0; i < 128; ++i)
                args.tab.pre[i] = i < n ? (int32_t)(cu[at + i] - cu[at]) : INT32_MAX;
        }
        at += n;
        if (args.ntok == 0)
            continue;
        const hipError_t e = cache.ks ? turn_any<kPages4>(bf16, args, s) : turn_any<kPages>(bf16, args, s);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_paged_gather(int bf16, int64_t batch, const int64_t *cu, const int64_t *starts,
                               int64_t Hkv, int64_t D, const PagedCache &cache, void *k, void *v,
                               hipStream_t s)
{
    GatherArgs args = {};
    args.c = cache;
    args.k = k;
    args.v = v;
    args.Hkv = (int)Hkv;
    for (int64_t at = 0; at < batch;) {
        const int64_t n = std::min<int64_t>(batch - at, RowTab::kMax);
        args.seq0 = at;
        args.nblk = 0;
        for (int64_t i = 0; i < n; ++i) {
            const int64_t first = starts ? starts[at + i] : 0, rows = cu[at + i + 1] - cu[at + i];
            args.tab.tok[i] = cu[at + i];
            args.tab.row[i] = (int32_t)first;
            args.tab.n[i] = (int32_t)rows;
            args.tab.pre[i] = (int32_t)args.nblk;
            args.nblk += rows > 0 ? ((first + rows + 15) >> 4) - (first >> 4) : 0;
        }
        for (int64_t i = n; i < 128; ++i)
            args.tab.pre[i] = INT32_MAX;
        at += n;
        if (args.nblk == 0)
            continue;
        hipError_t e = hipErrorInvalidValue;
        switch (D) {
        case 64: e = bf16 ? gather_launch<__bf16, 64>(args, s) : gather_launch<float, 64>(args, s); break;
        case 128: e = bf16 ? gather_launch<__bf16, 128>(args, s) : gather_launch<float, 128>(args, s); break;
        case 256: e = bf16 ? gather_launch<__bf16, 256>(args, s) : gather_launch<float, 256>(args, s); break;
        }
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace ssd
