// Softmax attention of one query token per sequence over a paged key/value cache
// (gfx950), the pages holding the input type or 4-bit codes.
//
// For query head h, key head h / (Hq / Hkv) and the rows s = 0 .. lengths[b]:
//     a_s = scale q . k_s,   o = sum_s exp(a_s - m) v_s / sum_s exp(a_s - m)
// in one pass with a running maximum, as in the kernels over padded caches.
//
// Work.  The host knows neither the lengths nor, therefore, the work: the launch has a
// fixed number of work-groups W, and each takes an equal share of the units of all
// (sequence, key head, 16 or 32 query heads) items laid end to end, a unit being kNW
// tiles of kKT keys or the start of an item.  A share may end inside an item; what a
// work-group has of an item that others continue goes to the workspace, and a second small
// kernel joins those.  So tables much wider than the sequences are long cost nothing, and sequences of any
// mix of lengths spread evenly.
//
// Scores are formed transposed (keys x query heads, 16 x 16 blocks): lane c + 16 g holds
// the scores of query head c for keys 16 kb + 4 g + i, its maximum and sums are per-lane
// scalars, and the probabilities are the second product's operand as they stand.  Tiles
// go from memory straight into LDS, two deep per wave, in parts of 16 rows: a part never
// crosses a page, so pages of 16 rows and more need no care.
//
// Bound by memory over pages of the input type: one sequence of 131000 rows, 32 heads over
// 8 of 128 in bf16, 98 us and the join's 5 (537 MB at 5.5 TB/s; a large copy reaches 5.08
// on the same card); 64 of 100 - 8190 rows 193 - 211 with the append in front, by the lengths.
// Over 4-bit pages a tile's instructions and waits take longer than its bytes: vector units 47%
// busy, matrix units 16%, 38 us for the long sequence's 151 MB (4.0 TB/s) and 5 for the join,
// 74 and 5 for the 64.  Small calls take 6 - 12 us: the look-ups in front of the first tile, a
// tile, and the join's launch.  Tried and no better: twice and four times as many work-groups
// (8 and 25 us more: each starts with look-ups and an empty pipeline), a second round of small
// work-groups for the end (4 - 8 us more for even batches).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ssd_attn.h"
#include "ssd_mma.h"
#include "ssd_paged.h"
#include "ssd_softmax.h"

namespace ssd {
namespace {

using namespace mx;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v2i lds_v2i;

struct PagedArgs {
    PagedCache c;
    const void *q;
    const int32_t *lengths;
    void *o;
    float *part;                              // [2 W][rows][D] sums of the items' pieces
    float2 *ml;                               // [2 W][rows] (m, l)
    int4 *rec;                                // (sequence or -1, item of it, first and last work-group) of what is
                                              // to be joined: [B HR] by item where that is no more than W
    int by_item;                              // .. else [W] by the work-group that began it
    int spare;                                // bytes of a wave's sums beside its tiles, 0: in their place
    int64_t q_stride;
    int64_t B, cap;                           // sequences; rows that a table has pages for
    int Hq, Hkv, grp, rtiles, logw;
    float scale;                              // |scale| log2 e
    int neg;                                  // scale < 0
};

// Maximum / sum over the four lanes c, c + 16, c + 32, c + 48.  (The swaps' second
// results go through an empty asm statement, as in half_max.)
__device__ __forceinline__ float quad_sum(float v)
{
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    unsigned b = s[1];
    asm volatile("" : "+v"(b));
    return half_sum(__builtin_bit_cast(float, (unsigned)s[0]) + __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float quad_max(float v)
{
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    unsigned b = s[1];
    asm volatile("" : "+v"(b));
    return half_max(fmaxf(__builtin_bit_cast(float, (unsigned)s[0]), __builtin_bit_cast(float, b)));
}

// Where the 16-row parts of a tile come from: the line of the first row among all pages'
// (of all heads), how many of the part's rows exist (1 .. 16), and whether its table entry
// was no page.  A part past the end stands for the tile's first.
template <int kParts> struct Parts {
    int64_t line[kParts];
    int rows[kParts];
    unsigned bad;
};

typedef const __attribute__((address_space(4))) int32_t *ConstInts;

__device__ __forceinline__ int64_t first_line(const PagedArgs &a, int page, int hk, int row)
{
    return (int64_t)(((uint64_t)(unsigned)page * (unsigned)a.Hkv + (unsigned)hk) << a.c.shift) +
           (row & ((1 << a.c.shift) - 1));
}

// The parts of the tile of keys t0 .. (scalar loads: vector ones would wait for the tiles
// in flight).  0 <= t0 < len <= cap.  A tile that lies in one page needs one entry.
template <int kParts>
__device__ __forceinline__ Parts<kParts> parts_of(const PagedArgs &a, int64_t b, int hk, int t0, int len)
{
    Parts<kParts> p;
    p.bad = 0;
    const ConstInts tab = (ConstInts)(uintptr_t)(a.c.table + b * a.c.max_pages);
    const unsigned npages = (unsigned)a.c.num_pages;
    if ((16 * kParts) >> a.c.shift <= 1) {
        int page = tab[uniform_int(t0) >> a.c.shift];
        if ((unsigned)page >= npages) {
            page = 0;
            p.bad = (1u << kParts) - 1;
        }
        const int64_t line = first_line(a, page, hk, t0);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const bool there = t0 + 16 * i < len;
            p.line[i] = there ? line + 16 * i : line;
            p.rows[i] = std::min(16, len - (there ? t0 + 16 * i : t0));
        }
        return p;
    }
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const int r0 = uniform_int(t0 + 16 * i < len ? t0 + 16 * i : t0);
        int page = tab[r0 >> a.c.shift];
        if ((unsigned)page >= npages) {
            page = 0;
            p.bad |= 1u << i;
        }
        p.rows[i] = std::min(16, len - r0);
        p.line[i] = first_line(a, page, hk, r0);
    }
    return p;
}

// What a lane carries of its query heads (CB columns of a block each).
template <int D, int CB> struct Sums {
    f32x4 acc[CB][D / 16];                    // acc[.][d][i]: value 16 d + 4 g + i
    float m[CB], l[CB];
};

// Raises the running maxima if a score of the tile passes one by kSlack, and turns the
// scores into unnormalised probabilities.  more(cb, f): sums to be rescaled by f.
template <int D, int CB, int KB, typename More>
__device__ __forceinline__ void soften(f32x4 (&s)[CB][KB], float c, Sums<D, CB> &st, More more)
{
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        float t = s[cb][0][0];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                t = fmaxf(t, s[cb][kb][i]);
        t *= c;
        if (__any(t > st.m[cb] + kSlack)) {
            const float mn = fmaxf(st.m[cb], quad_max(t)), al = exp2_fast(st.m[cb] - mn);
            st.m[cb] = mn;
            st.l[cb] *= al;
            more(cb, al);
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    st.acc[cb][d][i] *= al;
        }
        // the exponents as one fused operation each, but for huge scores
        float ec = c, em = st.m[cb];
        if (__builtin_expect(__any(fabsf(em) > 16777216.f && em != kNoMax), 0)) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[cb][kb][i] = below_max(s[cb][kb][i], c, st.m[cb]);
            ec = 1.f;
            em = 0.f;
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = exp2_fast(__builtin_fmaf(s[cb][kb][i], ec, -em));
                st.l[cb] += e;
                s[cb][kb][i] = e;
            }
    }
}

// Scores of keys from `see` on and of parts in `bad` become -infinity.
template <int CB, int KB>
__device__ __forceinline__ void hide(f32x4 (&s)[CB][KB], int see, unsigned bad, int g)
{
    asm volatile("" : "+v"(g));               // (nothing of this ahead of the branch that leads here)
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        const int lim = bad >> kb & 1u ? -64 : see - 16 * kb - 4 * g;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i >= lim)
#pragma unroll
                for (int cb = 0; cb < CB; ++cb)
                    s[cb][kb][i] = -__builtin_inff();
    }
}

// x as kTerms bf16 numbers, the first its rounding and the others that of what is left: x - t,
// exact, as a dot product with (-1, 0) or (0, -1), one instruction where taking the half out and
// subtracting would be two.  (The pairs are kept in registers: the compiler would write (-1, 0)
// as the inline constant -1.0, whose -1 the hardware has in the upper half.)
template <int kTerms> __device__ __forceinline__ void terms_of(const float (&x)[8], bf16x8 (&t)[kTerms])
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    unsigned lo = 0x0000bf80u, hi = 0xbf800000u;
    asm("" : "+s"(lo), "+s"(hi));
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        r[e] = x[e];
#pragma unroll
    for (int n = 0; n < kTerms; ++n) {
        u32x4 u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            u[e] = opaque(pack_bf16(r[2 * e], r[2 * e + 1]));
            if (n + 1 < kTerms) {
                const bf16x2 two = __builtin_bit_cast(bf16x2, (unsigned)u[e]);
                r[2 * e] = __builtin_amdgcn_fdot2_f32_bf16(two, __builtin_bit_cast(bf16x2, lo), r[2 * e], false);
                r[2 * e + 1] = __builtin_amdgcn_fdot2_f32_bf16(two, __builtin_bit_cast(bf16x2, hi), r[2 * e + 1], false);
            }
        }
        t[n] = __builtin_bit_cast(bf16x8, u);
    }
}

// ---------------------------------------------------------------------------
// Pages of the input type
// ---------------------------------------------------------------------------
// bf16: tiles of 32 keys, probabilities as three bf16 numbers, which hold an fp32 number (two
// leave 2^-17 of it: 0.2 - 0.3% of the outputs then differ from the rounded formula instead of
// 0.01 - 0.04%, in the same time).  fp32: tiles of 16, fp32 products.
template <typename T_, int D, int CB> struct WideTile {
    typedef T_ T;
    typedef Tile<T, D> TL;
    typedef typename Piece<T>::V V;
    static constexpr bool kHalf = sizeof(T) == 2;
    static constexpr int kKT = kHalf ? 32 : 16, kParts = kKT / 16, NP = TL::kPitch / 64;
    static constexpr int kTileBytes = kKT * TL::kPitch, kBuf = 2 * kTileBytes;
    static constexpr int kNW = 2 * kBuf * 4 <= 128 * 1024 ? 4 : 2;
    static constexpr int kMost = 4;
    static constexpr bool kTurns = false;
    static constexpr int kLoads = 2 * kParts * TileLoad<T, D, 16, 1>::kPer;

    V qf[CB][NP];

    // The queries, out of the LDS tiles at `at`.
    __device__ __forceinline__ void begin(const PagedArgs &a, unsigned at, int lane)
    {
        typedef LaneBase<T, D> LB;
        const unsigned qr = LB::row16(lane & 15, lane >> 4);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                qf[cb][p] = LB::piece16(at + 16 * cb * TL::kPitch, qr, p);
                if (a.neg)
                    qf[cb][p] = flip<T>(qf[cb][p]);
            }
    }

    static constexpr int kWhole = kLoads;
    static __device__ __forceinline__ bool whole(const PagedArgs &, int, int)
    {
        return false;
    }

    static __device__ __forceinline__ void issue(const PagedArgs &a, unsigned dst, const Parts<kParts> &p, bool,
                                                 int lane)
    {
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const unsigned at = dst + (unsigned)(16 * i * TL::kPitch);
            TileLoad<T, D, 16, 1>::issue(at, (const T *)a.c.k + p.line[i] * D, D, 0, p.rows[i], 0, lane);
            TileLoad<T, D, 16, 1>::issue(at + kTileBytes, (const T *)a.c.v + p.line[i] * D, D, 0, p.rows[i], 0, lane);
        }
    }

    // Values of parts that are no page: 0 (their scores are hidden, and 0 times them must be 0).
    static __device__ __forceinline__ void clear(unsigned char *buf, unsigned bad, int lane)
    {
        for (int i = 0; i < kParts; ++i)
            if (bad >> i & 1u)
                for (int x = 16 * lane; x < 16 * TL::kPitch; x += 1024)
                    *reinterpret_cast<uint4 *>(buf + kTileBytes + 16 * i * TL::kPitch + x) = make_uint4(0, 0, 0, 0);
    }

    __device__ __forceinline__ void tile(unsigned buf, bool masked, int see, unsigned bad, float c, int lane,
                                         Sums<D, CB> &st)
    {
        typedef LaneBase<T, D> LB;
        const int cl = lane & 15, g = lane >> 4;
        f32x4 s[CB][kParts] = {};
        const unsigned kr = opaque(LB::row16(cl, g));
#pragma unroll
        for (int kb = 0; kb < kParts; ++kb)
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const V k = LB::piece16(buf + 16 * kb * TL::kPitch, kr, p);
#pragma unroll
                for (int cb = 0; cb < CB; ++cb)
                    s[cb][kb] = mma16(k, qf[cb][p], s[cb][kb]);
            }
        if (masked)
            hide(s, see, bad, g);
        soften<D, CB, kParts>(s, c, st, [](int, float) {});
        const unsigned vt = buf + kTileBytes;
        if constexpr (kHalf) {
            bf16x8 pt[CB][3];
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = s[cb][e >> 2][e & 3];
                terms_of<3>(x, pt[cb]);
            }
            const int r = 4 * g + ((lane >> 2) & 3), q = lane & 3;
            const unsigned vr = opaque((unsigned)TL::off(r, q >> 1) + (q & 1) * 8);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                const unsigned at = vt + (vr ^ ((unsigned)d << 5));
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)at);
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s16x4 *)(uintptr_t)(at + 16 * TL::kPitch));
                const bf16x8 v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                    for (int n = 0; n < 3; ++n)
                        st.acc[cb][d] = mma16(v, pt[cb][n], st.acc[cb][d]);
            }
        } else {
            // row 4 g + i, column 16 d + c
            const unsigned vr = opaque((unsigned)(4 * g * TL::kPitch + (((cl >> 2) ^ g) << 4) + (cl & 3) * 4));
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                f32x4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = *(const __attribute__((address_space(3))) float *)(uintptr_t)(
                        vt + i * TL::kPitch + (vr ^ (unsigned)((d ^ i) << 6)));
#pragma unroll
                for (int cb = 0; cb < CB; ++cb)
                    st.acc[cb][d] = mma16(v, s[cb][0], st.acc[cb][d]);
            }
        }
    }

    __device__ __forceinline__ void finish(Sums<D, CB> &) {}
};

// ---------------------------------------------------------------------------
// Pages of 4-bit codes
// ---------------------------------------------------------------------------
// A value costs one instruction to unpack where a bf16 page costs none, so the work around it
// is kept off the vector units.  A byte n < 16 taken as an fp8 number (e4m3) is n 2^-9, so a
// dword's codes, four to a masked dword, become bf16 numbers n by conversions from fp8 with a
// scale of 2^9, two each, and those are the products' operand: with step s and least value m of
// the 64 values of group G,
//     q . k_G = s (sum q n) + m sum q
//     sum_t p_t v_t = sum_t (p_t s_t) n_t + sum_t p_t m_t
// so that scales cost one multiply-add per score or probability and group instead of one
// per value.  The second line's two sums grow with the number of keys where their sum need not
// (values about 0), and their roundings with them.  So two of every four keys count from the top,
//     p v = -(p s) (15 - n) + p (m + 15 s),
// whose sums run the other way; the complement is part of the mask.  p s enters as three bf16
// numbers, which hold all of an fp32 number.  (With codes as 16 + n, all keys alike and two
// terms, 0.4 - 1.6% of the outputs differed from the rounded formula, now 0.01 - 0.07% as of
// fp32 products; 78 -> 82 us for 64 sequences of 100 - 8190 rows.)  Where queries are fp32 both
// enter as three terms, and codes as (n - 8) / 16 with m + 8 s for m: 2.5 instructions a value.
// Keys are read as stored; values through the 4-bit transpose read, 16 keys of one column at a
// time.
//
// Tiles of 64 keys, or 32 where one is 5 KB and more (shorter chains in front of a wave's
// first result and fewer registers; 131000 keys of 128: 46 -> 42 us): [keys][D / 2] bytes
// of keys, the same of values, then the scales [part][group][16 keys] of both.  Rows are not
// padded; their 16-byte chunks are permuted by an XOR with swz(row), so that reads of 16
// rows cover the banks evenly.
template <typename T_, int D, int CB> struct CodeTile {
    typedef T_ T;
    static constexpr bool kShort = D > 64 && CB == 1;
    static constexpr int kKT = kShort ? 32 : 64, kParts = kKT / 16, G = D / 64;
    static constexpr int kRow = D / 2, kPart = 16 * kRow, kSide = kParts * kPart, kScales = kKT * 4 * G;
    static constexpr int kBuf = 2 * kSide + 2 * kScales;
    static constexpr int kNW = 4;
    // Work-groups of a CU: two at 256 registers a wave, or one at 512 where two blocks of columns
    // of wide heads, or fp32 queries of 256, take more (with bf16 queries 292 at 128, 476 at 256).
    // 16 sequences of 8000 rows in fp32: 16 heads over 4 of 256 77 us, with two 90; 32 heads over
    // one of 128 27, with two 47.  In bf16 64 of 100 - 8190 rows, 32 heads over one of 128, 36 and
    // 38, but 32 of 8000, 60 heads over 3, 66 and 62.  Registers that spill all the same: six of
    // fp32 queries of 64 and 127 of those of 256, both with two blocks of columns.
    static constexpr int kMost = (CB == 2 && D > 64) || (D == 256 && sizeof(T) == 4) ? 1 : 2;
    // Work-groups of a CU raise their priority in every other tile, in turn: the older one would
    // otherwise finish first and leave the other alone (2 - 5% of the time; with two blocks of
    // columns no difference).
    static constexpr bool kTurns = CB == 1;
    static constexpr int kPer = kPart > 1024 ? kPart / 1024 : 1;          // loads of a part's codes
    static constexpr int kLoads = kParts * (2 * kPer + 2);
    static constexpr int kQ = sizeof(T) == 2 ? 1 : 3, kP = 3;
    static constexpr bool kCentred = sizeof(T) == 4;

    // (constants kept in registers: as literals they would be part of every instruction)
    unsigned low, top;                        // codes of a dword in its bytes; which of them count from the top
    float zero;
    bf16x8 qf[CB][D / 32][kQ];                // queries, in the order of opened()
    float qs[CB][G];                          // their sums over a group
    float rest[CB][G];                        // sum of p m or p (m + 15 s) (centred: p (m + 8 s))

    static __device__ __forceinline__ int swz(int row)
    {
        return D == 64 ? 0 : D == 128 ? (row >> 2) & 3 : (row >> 1) & 7;
    }

    // The code that element e of opened() is.
    static __host__ __device__ constexpr int code_of(int e)
    {
        return kCentred ? (e >> 1) + 4 * (e & 1) : e < 4 ? 2 * e : 2 * e - 7;
    }
    // Whether a value's code counts from the top there.
    static __host__ __device__ constexpr bool from_top(int code)
    {
        return !kCentred && ((code & 3) == 1 || (code & 3) == 2);
    }

    // Codes 0 .. 7 of a dword, keys' as they are and some of the values' from the top; centred:
    // (code - 8) / 16.
    template <bool kKey> __device__ __forceinline__ bf16x8 opened(unsigned w) const
    {
        u32x4 v;
        if constexpr (kCentred) {
            w ^= 0x88888888u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = pack_bf16(__builtin_amdgcn_cvt_off_f32_i4((int)(w >> (4 * i))),
                                 __builtin_amdgcn_cvt_off_f32_i4((int)(w >> (4 * i + 16))));
            return __builtin_bit_cast(bf16x8, v);
        }
        const unsigned even = (kKey ? w : w ^ top) & low, odd = (kKey ? w >> 4 : (w >> 4) ^ ~top) & low;
        v[0] = pair<false>(even);
        v[1] = pair<true>(even);
        v[2] = pair<false>(odd);
        v[3] = pair<true>(odd);
        return __builtin_bit_cast(bf16x8, v);
    }

    // Two bytes below 16 of a dword's lower or upper half as bf16 numbers.
    template <bool kUpper> static __device__ __forceinline__ unsigned pair(unsigned bytes)
    {
        return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, 512.f, kUpper));
    }

    __device__ __forceinline__ void begin(const PagedArgs &a, unsigned at, int lane)
    {
        typedef Tile<T, D> TL;
        constexpr int kRaw = sizeof(T) == 2 ? 1 : 2;             // 16-byte pieces of eight queries
        const int c = lane & 15, g = lane >> 4;
        low = 0x0f0f0f0fu;
        top = 0xff00ff00u;                    // codes 2 and 6 of the even ones, and the others of the odd ones: 1 and 5
        zero = 0.f;
        asm volatile("" : "+s"(low), "+s"(top), "+v"(zero));
        const unsigned sign = a.neg ? 0x80000000u : 0u;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int s = 0; s < G; ++s) {
                float sum = 0.f;
#pragma unroll
                for (int p = 2 * s; p < 2 * s + 2; ++p) {
                    float x[8], y[8];
                    u32x4 raw[kRaw];
#pragma unroll
                    for (int n = 0; n < kRaw; ++n)
                        raw[n] = *(const __attribute__((address_space(3))) u32x4 *)(uintptr_t)(
                            at + 16 * cb * TL::kPitch + TL::off(c, ((p / 2 * 8 + 2 * g + p % 2) * kRaw) + n));
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const unsigned u = sizeof(T) == 4 ? raw[e / 4 % kRaw][e % 4]
                                           : e & 1 ? raw[0][e / 2] & 0xffff0000u : raw[0][e / 2] << 16;
                        x[e] = __uint_as_float(u ^ sign);
                        sum += x[e];
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = x[code_of(e)];
                    terms_of<kQ>(y, qf[cb][p]);
                }
                qs[cb][s] = quad_sum(sum);
                rest[cb][s] = 0.f;
            }
    }

    // 16 or 4 bytes per lane of the first kLanes lanes from base + voff into LDS (assembly for
    // the reasons given at lds_load16).
    template <int kLanes> static __device__ __forceinline__ void load16(unsigned dst, const unsigned char *base, unsigned voff, int lane)
    {
        if (kLanes >= 64 || lane < kLanes)
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
                         :: "s"(uniform_int((int)dst)), "v"(voff), "s"(base) : "memory", "m0");
    }
    template <int kLanes> static __device__ __forceinline__ void load4(unsigned dst, const unsigned char *base, unsigned voff, int lane)
    {
        if (kLanes >= 64 || lane < kLanes)
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, %2"
                         :: "s"(uniform_int((int)dst)), "v"(voff), "s"(base) : "memory", "m0");
    }

    // A tile's loads: kWhole where its 64 rows exist and lie in one page, else part by part.
    static constexpr int kWhole = 2 * (kSide / 1024) + 2 * (kScales / 256);
    static __device__ __forceinline__ bool whole(const PagedArgs &a, int t0, int len)
    {
        return kKT >> a.c.shift <= 1 && t0 + kKT <= len;
    }

    static __device__ __forceinline__ void issue(const PagedArgs &a, unsigned dst, const Parts<kParts> &p, bool all,
                                                 int lane)
    {
        constexpr int CPR = kRow / 16;                       // chunks of a row
        // (kRow is 32 G and a row's scales take 4 G bytes)
        if (all) {
            const unsigned char *kp = (const unsigned char *)a.c.k + p.line[0] * kRow;
            const unsigned char *vp = (const unsigned char *)a.c.v + p.line[0] * kRow;
            const unsigned char *ks = (const unsigned char *)a.c.ks + p.line[0] * (4 * G);
            const unsigned char *vs = (const unsigned char *)a.c.vs + p.line[0] * (4 * G);
#pragma unroll
            for (int n = 0; n < kSide / 1024; ++n) {
                const int x = n * 64 + lane, row = x / CPR;
                const unsigned off = (unsigned)(row * kRow + (((x % CPR) ^ swz(row)) << 4));
                load16<64>(dst + n * 1024, kp, off, lane);
                load16<64>(dst + kSide + n * 1024, vp, off, lane);
            }
#pragma unroll
            for (int n = 0; n < kScales / 256; ++n) {
                // dword [part][group][key] <- [key][group]
                const int x = n * 64 + lane, key = 16 * (x / (16 * G)) + x % 16, grp = x % (16 * G) / 16;
                const unsigned off = (unsigned)(key * G + grp) * 4u;
                load4<64>(dst + 2 * kSide + n * 256, ks, off, lane);
                load4<64>(dst + 2 * kSide + kScales + n * 256, vs, off, lane);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int last = p.rows[i] - 1;
            const unsigned char *kp = (const unsigned char *)a.c.k + p.line[i] * kRow;
            const unsigned char *vp = (const unsigned char *)a.c.v + p.line[i] * kRow;
#pragma unroll
            for (int n = 0; n < kPer; ++n) {
                const int x = n * 64 + lane, row = x / CPR;
                const unsigned off = (unsigned)(std::min(row, last) * kRow + (((x % CPR) ^ swz(row)) << 4));
                load16<kPart / 16>(dst + i * kPart + n * 1024, kp, off, lane);
                load16<kPart / 16>(dst + kSide + i * kPart + n * 1024, vp, off, lane);
            }
            const unsigned off = (unsigned)(std::min(lane & 15, last) * G + (lane >> 4)) * 4u;
            const unsigned at = dst + 2 * kSide + i * 64 * G;
            load4<16 * G>(at, (const unsigned char *)a.c.ks + p.line[i] * (4 * G), off, lane);
            load4<16 * G>(at + kScales, (const unsigned char *)a.c.vs + p.line[i] * (4 * G), off, lane);
        }
    }

    // Scales of values of parts that are no page: 0.
    static __device__ __forceinline__ void clear(unsigned char *buf, unsigned bad, int lane)
    {
        for (int i = 0; i < kParts; ++i)
            if ((bad >> i & 1u) && lane < 16 * G)
                *reinterpret_cast<unsigned *>(buf + 2 * kSide + kScales + i * 64 * G + 4 * lane) = 0u;
    }

    static __device__ __forceinline__ u32x4 scales(unsigned at)
    {
        return *(const __attribute__((address_space(3))) u32x4 *)(uintptr_t)at;
    }

    __device__ __forceinline__ void tile(unsigned buf, bool masked, int see, unsigned bad, float c, int lane,
                                         Sums<D, CB> &st)
    {
        const int cl = lane & 15, g = lane >> 4;
        f32x4 sc[CB][kParts];
        const unsigned kr = opaque((unsigned)(cl * kRow + ((((g >> 1)) ^ swz(cl)) << 4) + (g & 1) * 8));
#pragma unroll
        for (int kb = 0; kb < kParts; ++kb)
#pragma unroll
            for (int s = 0; s < G; ++s) {
                const u32x2 w = *(const __attribute__((address_space(3))) u32x2 *)(uintptr_t)(
                    buf + kb * kPart + (kr ^ (unsigned)(s << 5)));
                const bf16x8 k0 = opened<true>(w[0]), k1 = opened<true>(w[1]);
                const u32x4 ws = scales(buf + 2 * kSide + (unsigned)(kb * 64 * G + s * 64 + 16 * g));
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) {
                    f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int n = 0; n < kQ; ++n) {
                        d = mma16(k0, qf[cb][2 * s][n], d);
                        d = mma16(k1, qf[cb][2 * s + 1][n], d);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f16x2 h = __builtin_bit_cast(f16x2, (unsigned)ws[i]);
                        const float step = kCentred ? 16.f * (float)h[0] : (float)h[0];
                        const float least = kCentred ? __builtin_fmaf(8.f, (float)h[0], (float)h[1]) : (float)h[1];
                        const float r = __builtin_fmaf(least, qs[cb][s], s == 0 ? zero : sc[cb][kb][i]);
                        sc[cb][kb][i] = __builtin_fmaf(step, d[i], r);
                    }
                }
            }
        if (masked)
            hide(sc, see, bad, g);
        soften<D, CB, kParts>(sc, c, st, [&](int cb, float al) {
#pragma unroll
            for (int s = 0; s < G; ++s)
                rest[cb][s] *= al;
        });
        // within 16 lanes, lane r addresses the row of key 16 (r / 4) + 4 g + r % 4 (of tiles of 32
        // keys: r % 8, and the upper eight lanes the next 16 columns)
        constexpr bool kTall = kKT == 64;
        const int r = 16 * (kTall ? cl >> 2 : cl >> 2 & 1) + 4 * g + (cl & 3);
        const unsigned vr = opaque((unsigned)(r * kRow + (swz(r) << 4) + (kTall ? 0 : (cl >> 3) * 8)));
#pragma unroll
        for (int s = 0; s < G; ++s) {
            bf16x8 pt[CB][kParts / 2][kP];
#pragma unroll
            for (int kb = 0; kb < kParts; kb += 2) {
                const u32x4 w0 = scales(buf + 2 * kSide + kScales + (unsigned)(kb * 64 * G + s * 64 + 16 * g));
                const u32x4 w1 = scales(buf + 2 * kSide + kScales + (unsigned)((kb + 1) * 64 * G + s * 64 + 16 * g));
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int code = code_of(e);             // (of eight keys: four of block kb, four of the next)
                        const f16x2 h = __builtin_bit_cast(f16x2, (unsigned)(code >> 2 ? w1 : w0)[code & 3]);
                        const float p = sc[cb][kb + (code >> 2)][code & 3];
                        const float base = kCentred ? __builtin_fmaf(8.f, (float)h[0], (float)h[1])
                                         : from_top(code) ? __builtin_fmaf(15.f, (float)h[0], (float)h[1]) : (float)h[1];
                        rest[cb][s] = __builtin_fmaf(p, base, rest[cb][s]);
                        x[e] = kCentred ? p * (16.f * (float)h[0])
                                        : __builtin_fmaf(from_top(code) ? -p : p, (float)h[0], zero);
                    }
                    terms_of<kP>(x, pt[cb][kb / 2]);
                }
            }
#pragma unroll
            for (int d = 4 * s; d < 4 * s + 4; d += kTall ? 1 : 2) {
                const v2i w = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                    (lds_v2i *)(uintptr_t)(buf + kSide + (vr ^ (unsigned)((d >> 1) << 4)) + (d & 1) * 8));
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const bf16x8 v = opened<false>((unsigned)w[x]);
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                        for (int n = 0; n < kP; ++n) {
                            f32x4 &acc = st.acc[cb][kTall ? d : d + x];
                            acc = mma16(v, pt[cb][kTall ? x : 0][n], acc);
                        }
                }
            }
        }
    }

    __device__ __forceinline__ void finish(Sums<D, CB> &st)
    {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int s = 0; s < G; ++s) {
                const float r = quad_sum(rest[cb][s]);
#pragma unroll
                for (int d = 4 * s; d < 4 * s + 4; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        st.acc[cb][d][i] += r;
            }
    }
};

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
// Tokens of sequence b, 0 for an unused slot.
__device__ __forceinline__ int filled(const PagedArgs &a, int64_t b)
{
    const int at = a.lengths[b];
    return at < 0 || at >= a.cap ? 0 : at + 1;
}

template <typename Eng, int D, int CB, int kOcc>
__global__ __launch_bounds__((64 * Eng::kNW), (kOcc * Eng::kNW / 4 > 0 ? kOcc * Eng::kNW / 4 : 1))
void paged_decode_kernel(PagedArgs a)
{
    typedef typename Eng::T T;
    constexpr int NW = Eng::kNW, NT = 64 * NW, KT = Eng::kKT, STEP = KT * NW;
    constexpr unsigned kWave = 2u * Eng::kBuf;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ float sm[NW][16 * CB], sl[NW][16 * CB];
    __shared__ int64_t wsum[NW];
    __shared__ int where[2];

    const int tid = threadIdx.x, lane = tid & 63, w = uniform_int(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int W = 1 << a.logw, HR = a.Hkv * a.rtiles;

    // This work-group's units [u0, u1) of all, and the sequence b that u0 lies in with the
    // units before it.  Beginning an item takes about as long as a unit (`extra`, its first unit
    // then: without it work-groups with many short sequences end last, 94 us instead of 82 for 64
    // sequences of 100 - 8190 rows in 4 bits).  Up to 64 sequences of the same number of units do
    // without: their items divide evenly more often (16 of 8000 rows, 32 heads over one of 256: 36
    // us, 43 with).  Where there are no more units than work-groups each gets one, so that every
    // work-group of an item has a piece of it.  Up to 64 sequences: every wave finds its share from
    // its own lanes.
    int before = 0, found, mylen = 0, extra;
    int64_t all, u0, u1;
    const auto share = [&](int total, int count, bool alike) {
        const bool few = (int64_t)total * HR <= W;
        extra = few || alike ? 0 : 1;
        all = (int64_t)(total + extra * count) * HR;
        u0 = few ? std::min<int64_t>(all, blockIdx.x) : (all * blockIdx.x) >> a.logw;
        u1 = few ? std::min<int64_t>(all, blockIdx.x + 1) : (all * (blockIdx.x + 1)) >> a.logw;
    };
    if (a.B <= 64) {
        mylen = lane < a.B ? filled(a, lane) : 0;
        const int mine = (mylen + STEP - 1) / STEP;
        int incl = mine;
        incl += __builtin_amdgcn_update_dpp(0, incl, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8
        incl += __builtin_amdgcn_update_dpp(0, incl, 0x112, 0xf, 0xf, false);
        incl += __builtin_amdgcn_update_dpp(0, incl, 0x114, 0xf, 0xf, false);
        incl += __builtin_amdgcn_update_dpp(0, incl, 0x118, 0xf, 0xf, false);
        incl += __builtin_amdgcn_update_dpp(0, incl, 0x142, 0xa, 0xf, false);   // row_bcast 15, 31
        incl += __builtin_amdgcn_update_dpp(0, incl, 0x143, 0xc, 0xf, false);
        const uint64_t some = __ballot(mylen > 0);
        const int one = __builtin_amdgcn_readlane(mine, some ? __builtin_ctzll(some) : 0);
        share(__builtin_amdgcn_readlane(incl, 63), __popcll(some), __all(mine == 0 || mine == one));
        incl += extra * __popcll(some & (~uint64_t(0) >> (63 - lane)));
        const uint64_t past = __ballot((int64_t)incl * HR > u0);
        found = past ? __builtin_ctzll(past) : -1;
        before = __builtin_amdgcn_readlane(incl - mine - (mylen > 0 ? extra : 0), past ? found : 0);
    } else {
        // (units below 2^32, and sequences above)
        const int per = (int)((a.B + NT - 1) / NT), b0 = tid * per, b1 = std::min((int)a.B, b0 + per);
        const auto units_of = [&](int b) {
            const int n = (filled(a, b) + STEP - 1) / STEP;
            return n > 0 ? (int64_t(1) << 32) + n : 0;
        };
        int64_t mine = 0;
        for (int b = b0; b < b1; ++b)
            mine += units_of(b);
        int64_t incl = mine;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int64_t up = __shfl_up(incl, off, 64);
            if (lane >= off)
                incl += up;
        }
        if (lane == 63)
            wsum[w] = incl;
        if (tid == 0)
            where[0] = -1;
        __syncthreads();
        int64_t excl = incl - mine, total = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            if (i < w)
                excl += wsum[i];
            total += wsum[i];
        }
        share(uniform_int((int)total), uniform_int((int)(total >> 32)), false);
        const auto weight = [&](int64_t x) { return (int64_t)((int)x + extra * (int)(x >> 32)) * HR; };
        if (u0 >= weight(excl) && u0 < weight(excl + mine)) {
            int b = b0;
            for (; b + 1 < b1; ++b) {
                const int64_t n = units_of(b);
                if (u0 < weight(excl + n))
                    break;
                excl += n;
            }
            where[0] = b;
            where[1] = (int)excl + extra * (int)(excl >> 32);
        }
        __syncthreads();
        found = uniform_int(where[0]);
        before = uniform_int(where[1]);
    }
    if (!a.by_item && tid == 0)
        a.rec[blockIdx.x] = make_int4(-1, 0, 0, 0);

    unsigned char *own = smem + w * kWave;
    const unsigned lds0 = lds_addr(own);
    // (lengths that change under the kernel end it early)
    int64_t b = found;
    int64_t first = (int64_t)before * HR;                     // first unit of the sequence
    const auto len_of = [&](int64_t i) {
        return a.B <= 64 ? __builtin_amdgcn_readlane(mylen, (int)i) : uniform_int(filled(a, i));
    };
    int len = u0 < u1 && found >= 0 ? len_of(b) : 0;
    int units = (len + STEP - 1) / STEP;
    int item = 0, from = 0;                                   // from: among units + extra
    if (units > 0) {
        const unsigned at = (unsigned)(u0 - first);           // (below 2^31: checked on the host)
        item = (int)(at / (unsigned)(units + extra));
        from = (int)(at % (unsigned)(units + extra));
        if (item >= HR)
            units = 0;
    }

    // The queries go through LDS as the tiles do (loads into registers would wait for the tiles
    // in flight): they land in the second slot while the first tile is on its way, and the
    // second tile follows them.  Where the LDS has room for the waves' sums beside their tiles
    // (a.spare), both are sent for ahead of the end of the item before.
    constexpr bool kBeside = 16 * CB * D * (int)sizeof(T) <= Eng::kBuf;
    const bool ahead = kBeside && a.spare > 0;
    Parts<Eng::kParts> nxt = {};
    bool sent = false;
    const auto send = [&](int64_t b_, int item_, int t_, int kend_, int len_) {
        const int rt_ = item_ % a.rtiles, hk_ = item_ / a.rtiles, rows_ = std::min(16 * CB, a.grp - 16 * CB * rt_);
        const T *qp = (const T *)a.q + b_ * a.q_stride + ((int64_t)hk_ * a.grp + 16 * CB * rt_) * D;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
            TileLoad<T, D, 16, 1>::issue(lds0 + (kBeside ? Eng::kBuf : 0) + 16 * cb * D * (int)sizeof(T), qp, D,
                                         std::min(16 * cb, rows_ - 1), rows_, 0, lane);
        if (t_ < kend_) {
            nxt = parts_of<Eng::kParts>(a, b_, hk_, t_, len_);
            if (kBeside)
                Eng::issue(a, lds0, nxt, Eng::whole(a, t_, len_), lane);
        }
    };

    for (int64_t u = u0; u < u1 && units > 0;) {
        const int end = (int)std::min<int64_t>(units + extra, from + (u1 - u));
        const int begin = std::max(0, from - extra), to = end - extra;    // units of keys
        if (begin >= to)
            break;
        const int rt = item % a.rtiles, hk = item / a.rtiles;
        const int rows = std::min(16 * CB, a.grp - 16 * CB * rt);
        const int64_t h0 = (int64_t)hk * a.grp + 16 * CB * rt;
        const int kend = (int)std::min<int64_t>((int64_t)to * STEP, len);

        Eng eng;
        int t0 = begin * STEP + KT * w;
        if (!sent) {
            wait_vmcnt<0>();                                  // (stores of the item before)
            send(b, item, t0, kend, len);
        }
        Parts<Eng::kParts> second = {};
        if (t0 + STEP < kend)
            second = parts_of<Eng::kParts>(a, b, hk, t0 + STEP, len);
        unsigned bad = t0 < kend ? nxt.bad : 0u, bad_next = second.bad;
        if (!kBeside || sent || t0 >= kend)
            wait_vmcnt<0>();
        else if (Eng::whole(a, t0, len))
            wait_vmcnt<Eng::kWhole>();
        else
            wait_vmcnt<Eng::kLoads>();
        eng.begin(a, lds0 + (kBeside ? Eng::kBuf : 0), lane);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (!kBeside && t0 < kend)
            Eng::issue(a, lds0, nxt, Eng::whole(a, t0, len), lane);
        if (t0 + STEP < kend)
            Eng::issue(a, lds0 + Eng::kBuf, second, Eng::whole(a, t0 + STEP, len), lane);
        if (t0 + 2 * STEP < kend)
            nxt = parts_of<Eng::kParts>(a, b, hk, t0 + 2 * STEP, len);
        Sums<D, CB> st;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
            st.m[cb] = kNoMax;
            st.l[cb] = 0.f;
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
                st.acc[cb][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        for (int n = 0; t0 < kend; ++n, t0 += STEP) {
            const unsigned slot = (unsigned)(n & 1) * Eng::kBuf;
            // this tile has landed (the next may be in flight)
            if (t0 + STEP >= kend)
                wait_vmcnt<0>();
            else if (Eng::whole(a, t0 + STEP, len))
                wait_vmcnt<Eng::kWhole>();
            else
                wait_vmcnt<Eng::kLoads>();
            if (bad) {
                Eng::clear(own + slot, bad, lane);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            }
            if constexpr (Eng::kTurns)                        // (two work-groups to a CU: W / 2 apart)
                if (((unsigned)n + (blockIdx.x >> (a.logw - 1))) & 1u)
                    __builtin_amdgcn_s_setprio(1);
                else
                    __builtin_amdgcn_s_setprio(0);
            eng.tile(lds0 + slot, t0 + KT > len || bad != 0, len - t0, bad, a.scale, lane, st);
            bad = bad_next;
            if (t0 + 2 * STEP < kend) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");    // the slot's reads are done
                Eng::issue(a, lds0 + slot, nxt, Eng::whole(a, t0 + 2 * STEP, len), lane);
                bad_next = nxt.bad;
                if (t0 + 3 * STEP < kend)
                    nxt = parts_of<Eng::kParts>(a, b, hk, t0 + 3 * STEP, len);
            }
        }
        eng.finish(st);

        // what comes next: the next item, of the next sequence that has tokens if need be
        const bool began = begin == 0, complete = began && to == units;
        const int64_t ob = b, last = first + (int64_t)(item + 1) * (units + extra) - 1;
        const int oitem = item;
        u += end - from;
        from = 0;
        if (u < u1 && ++item == HR) {
            item = 0;
            first += (int64_t)HR * (units + extra);
            for (b += 1; b < a.B; b += 64) {
                const uint64_t some = a.B <= 64 ? __ballot(mylen > 0) >> b
                                                : __ballot(b + lane < a.B && filled(a, std::min(a.B - 1, b + lane)) > 0);
                if (some) {
                    b += __builtin_ctzll(some);
                    break;
                }
            }
            len = b < a.B ? len_of(b) : 0;
            units = (len + STEP - 1) / STEP;
        }
        sent = ahead && u1 - u > extra && units > 0;
        if (sent) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");        // the slots' reads are done
            send(b, item, KT * w, (int)std::min<int64_t>(std::min<int64_t>(units, u1 - u - extra) * STEP, len), len);
        }

        // the waves' sums to a common maximum
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
            const float l = quad_sum(st.l[cb]);
            if (g == 0) {
                sm[w][16 * cb + c] = st.m[cb];
                sl[w][16 * cb + c] = l;
            }
        }
        __syncthreads();
        unsigned char *sums = ahead ? smem + NW * kWave : smem;
        const unsigned pitch = ahead ? (unsigned)a.spare : kWave;     // between the waves' sums
        float *wp = reinterpret_cast<float *>(sums + w * pitch);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
            float mt = sm[0][16 * cb + c];
#pragma unroll
            for (int i = 1; i < NW; ++i)
                mt = fmaxf(mt, sm[i][16 * cb + c]);
            const float f = exp2_fast(st.m[cb] - mt);
            if (16 * cb + c < rows)
#pragma unroll
                for (int d = 0; d < D / 16; ++d)
                    *reinterpret_cast<f32x4 *>(wp + (16 * cb + c) * D + 16 * d + 4 * g) =
                        f32x4{st.acc[cb][d][0] * f, st.acc[cb][d][1] * f, st.acc[cb][d][2] * f, st.acc[cb][d][3] * f};
        }
        __syncthreads();
        const int64_t slot = (2 * (int64_t)blockIdx.x + (began ? 1 : 0)) * 16 * CB;
        T *op = (T *)a.o + (ob * a.Hq + h0) * D;
        for (int i = 4 * tid; i < rows * D; i += 4 * NT) {
            const int row = i / D;
            f32x4 v = *reinterpret_cast<const f32x4 *>(sums + i * 4);
#pragma unroll
            for (int k = 1; k < NW; ++k)
                v += *reinterpret_cast<const f32x4 *>(sums + k * pitch + i * 4);
            float mr = sm[0][row], lr = 0.f;
#pragma unroll
            for (int k = 1; k < NW; ++k)
                mr = fmaxf(mr, sm[k][row]);
#pragma unroll
            for (int k = 0; k < NW; ++k)
                lr += sl[k][row] * exp2_fast(sm[k][row] - mr);
            if (complete) {
                const float inv = lr > 0.f ? 1.f / lr : 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    op[i + e] = (T)(v[e] * inv);
            } else {
                *reinterpret_cast<f32x4 *>(a.part + slot * D + i) = v;
                if (i % D == 0)
                    a.ml[slot + row] = make_float2(mr, lr);
            }
        }
        if (began && tid == 0 && (!complete || a.by_item)) {
            // the work-group of the item's last unit
            const int64_t wl = all <= W ? last : (((last + 1) << a.logw) - 1) / all;
            a.rec[a.by_item ? ob * HR + oitem : blockIdx.x] =
                make_int4(complete ? -1 : (int)ob, oitem, (int)blockIdx.x, (int)wl);
        }
        __syncthreads();                                      // (the LDS is written again)
    }

    // unused slots
    for (int64_t i = blockIdx.x; i < a.B; i += W)
        if (filled(a, i) == 0) {
            for (int64_t j = tid; j < (int64_t)a.Hq * D; j += NT)
                ((T *)a.o)[i * a.Hq * D + j] = (T)0.f;
            if (a.by_item && tid < HR)
                for (int j = tid; j < HR; j += NT)
                    a.rec[i * HR + j] = make_int4(-1, 0, 0, 0);
        }
}

// Joins the pieces of an item that several work-groups have: one row per work-group, the
// loads of up to 16 kT / D pieces in flight together.
template <typename T, int D, int CB, int kT> __global__ __launch_bounds__(kT) void paged_join_kernel(PagedArgs a)
{
    constexpr int LPR = D / 4, G = kT / LPR;
    __shared__ float4 sacc[G][LPR];
    __shared__ float sl[G];
    const int4 rec = a.rec[blockIdx.x];
    if (rec.x < 0 || rec.x >= a.B || rec.z < 0 || rec.w >= 1 << a.logw)   // (lengths that changed under the kernel)
        return;
    const int tid = threadIdx.x, gr = tid / LPR, d4 = tid % LPR;
    const int w0 = rec.z, n = rec.w - w0 + 1;
    const int rt = rec.y % a.rtiles, hk = rec.y / a.rtiles, row = blockIdx.y;
    if (row >= std::min(16 * CB, a.grp - 16 * CB * rt))
        return;
    const int64_t h = (int64_t)hk * a.grp + 16 * CB * rt + row;
    // piece 0: the second slot of w0; piece i: the first of w0 + i
    auto at = [&](int i) { return (2 * (int64_t)(w0 + i) + (i == 0 ? 1 : 0)) * 16 * CB + row; };
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f, m = kNoMax;
    constexpr int U = 4;
    for (int i0 = gr; i0 < n; i0 += G * U) {
        float2 ml[U];
        float4 p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t s = at(std::min(i0 + u * G, n - 1));
            ml[u] = a.ml[s];
            p[u] = *reinterpret_cast<const float4 *>(a.part + s * D + 4 * d4);
        }
        float mn = m;
#pragma unroll
        for (int u = 0; u < U; ++u)
            mn = fmaxf(mn, ml[u].x);
        const float old = exp2_fast(m - mn);
        v.x *= old; v.y *= old; v.z *= old; v.w *= old;
        l *= old;
        m = mn;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float f = i0 + u * G < n ? exp2_fast(ml[u].x - m) : 0.f;
            v.x += f * p[u].x; v.y += f * p[u].y; v.z += f * p[u].z; v.w += f * p[u].w;
            l += f * ml[u].y;
        }
    }
    // to a common maximum over the groups that had pieces
    __shared__ float smax[G];
    if (d4 == 0)
        smax[gr] = m;
    __syncthreads();
    float mx = kNoMax;
    for (int i = 0; i < G; ++i)
        mx = fmaxf(mx, smax[i]);
    const float f = exp2_fast(m - mx);
    sacc[gr][d4] = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
    if (d4 == 0)
        sl[gr] = l * f;
    __syncthreads();
    if (tid < LPR) {
        v = sacc[0][d4];
        l = sl[0];
        for (int i = 1; i < G; ++i) {
            const float4 p = sacc[i][d4];
            v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
            l += sl[i];
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        T *op = (T *)a.o + ((int64_t)rec.x * a.Hq + h) * D + 4 * d4;
        op[0] = (T)(v.x * inv);
        op[1] = (T)(v.y * inv);
        op[2] = (T)(v.z * inv);
        op[3] = (T)(v.w * inv);
    }
}

// Work-groups of a CU: as many as fit by their LDS and registers; and 256 CUs of them.
template <typename Eng> constexpr int occupancy()
{
    const int n = std::min(Eng::kMost, 160 * 1024 / (Eng::kNW * 2 * Eng::kBuf + 2048));
    return n >= 4 ? 4 : n >= 2 ? 2 : 1;
}
template <typename Eng> constexpr int log_groups()
{
    return occupancy<Eng>() == 4 ? 10 : occupancy<Eng>() == 2 ? 9 : 8;
}

// Calls f(engine, D, CB) for the call's types and sizes.
template <typename F> auto with_engine(int bf16, int q4, int64_t D, bool two, F f)
{
#define SSD_PAGED(T, D_)                                                                                 \
    (q4 ? (two ? f((CodeTile<T, D_, 2> *)nullptr, std::integral_constant<int, D_>(), std::integral_constant<int, 2>()) \
               : f((CodeTile<T, D_, 1> *)nullptr, std::integral_constant<int, D_>(), std::integral_constant<int, 1>())) \
        : (two ? f((WideTile<T, D_, 2> *)nullptr, std::integral_constant<int, D_>(), std::integral_constant<int, 2>()) \
               : f((WideTile<T, D_, 1> *)nullptr, std::integral_constant<int, D_>(), std::integral_constant<int, 1>())))
    if (bf16)
        return D == 64 ? SSD_PAGED(__bf16, 64) : D == 128 ? SSD_PAGED(__bf16, 128) : SSD_PAGED(__bf16, 256);
    return D == 64 ? SSD_PAGED(float, 64) : D == 128 ? SSD_PAGED(float, 128) : SSD_PAGED(float, 256);
#undef SSD_PAGED
}

}  // namespace

// (Up to 16 query heads of a key head are one block of columns, more are items of 32.)
size_t paged_decode_workspace(int bf16, int q4, int64_t B, int64_t Hq, int64_t Hkv, int64_t D)
{
    if (B == 0)
        return 0;
    return with_engine(bf16, q4, D, Hq / Hkv > 16, [D](auto *e, auto, auto cb) {
        const size_t W = size_t(1) << log_groups<std::remove_pointer_t<decltype(e)>>();
        return W * (2 * 16 * decltype(cb)::value * (size_t)(D * 4 + 8) + 16);
    });
}

hipError_t launch_paged_decode(int bf16, int64_t B, int64_t Hq, int64_t Hkv, int64_t D,
                               int64_t q_stride, float scale, const void *q, const PagedCache &cache,
                               const int32_t *lengths, void *o, void *ws, hipStream_t s)
{
    PagedArgs a = {};
    a.c = cache;
    a.q = q;
    a.lengths = lengths;
    a.o = o;
    a.q_stride = q_stride;
    a.B = B;
    a.cap = cache.max_pages << cache.shift;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.grp = (int)(Hq / Hkv);
    a.scale = score_factor(scale);
    a.neg = scale < 0.f;
    return with_engine(bf16, cache.ks != nullptr, D, a.grp > 16, [&](auto *e, auto dim, auto cols) {
        typedef std::remove_pointer_t<decltype(e)> Eng;
        constexpr int kD = decltype(dim)::value, CB = decltype(cols)::value, kOcc = occupancy<Eng>();
        constexpr unsigned kTiles = Eng::kNW * 2u * Eng::kBuf, kMost = 157u * 1024u / occupancy<Eng>();
        const unsigned sums = (unsigned)std::min(a.grp, 16 * CB) * kD * 4u;
        a.spare = kTiles + Eng::kNW * sums <= kMost ? (int)sums : 0;
        const unsigned smem = kTiles + Eng::kNW * (unsigned)a.spare;
        static_assert(16 * CB * kD * 4 <= 2 * Eng::kBuf, "a wave's sums, and its queries, fit its tiles");
        a.rtiles = (a.grp + 16 * CB - 1) / (16 * CB);
        a.logw = log_groups<Eng>();
        const unsigned W = 1u << a.logw;
        a.part = static_cast<float *>(ws);
        a.ml = reinterpret_cast<float2 *>(a.part + (size_t)2 * W * 16 * CB * kD);
        a.rec = reinterpret_cast<int4 *>(a.ml + (size_t)2 * W * 16 * CB);
        const int64_t items = B * Hkv * a.rtiles;
        a.by_item = items <= W;
        static std::atomic<uint64_t> allowed{0};
        const auto kernel = &paged_decode_kernel<Eng, kD, CB, kOcc>;
        hipError_t err = allow_lds(reinterpret_cast<const void *>(kernel), (int)kMost, allowed);
        if (err != hipSuccess)
            return err;
        kernel<<<dim3(W), dim3(64 * Eng::kNW), smem, s>>>(a);
        if ((err = hipGetLastError()) != hipSuccess || a.cap <= Eng::kNW * Eng::kKT)
            return err;                       // (items of one unit are never cut)
        // (few items have many pieces each; starting many large work-groups takes longer than
        // they save: 6 us for 512 items of 4 heads)
        const int64_t heads = std::min(a.grp, 16 * CB), groups = (a.by_item ? items : W) * heads;
        const dim3 grid((unsigned)(a.by_item ? items : W), (unsigned)heads);
        if (groups <= 256)
            paged_join_kernel<typename Eng::T, kD, CB, 1024><<<grid, dim3(1024), 0, s>>>(a);
        else
            paged_join_kernel<typename Eng::T, kD, CB, 256><<<grid, dim3(256), 0, s>>>(a);
        return hipGetLastError();
    });
}

}  // namespace ssd
