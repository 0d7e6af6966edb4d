// Device helpers shared by the linear-attention and softmax-attention kernels:
// 32 x 32 matrix-instruction operands for bf16 and fp32, the LDS tiles they
// are read from, and loads from memory straight into those tiles.
//
// Operand conventions (wave64).  A product D += A B of 32 x 32 blocks takes
// from lane l = c + 32 hh row c of A (column c of B) at E values of the
// contraction index and leaves D[8 (r / 4) + 4 hh + r % 4][c] in the lane's
// register r of 16.  One "piece" is 16 bytes per lane: E = 8 bf16 values (one
// v_mfma_f32_32x32x16_bf16) or E = 4 fp32 values (four v_mfma_f32_32x32x2_f32),
// i.e. 2 E values of the contraction index over the two lane halves.  The
// index may be dealt to the slots in any order as long as A and B agree; two
// orders are used, e being the slot:
//   natural      piece p, half hh, slot e  <->  2 E p + E hh + e
//   accumulator  the rows a result register holds: for bf16
//                16 p + 8 (e / 4) + 4 hh + e % 4, for fp32 the natural order
// so that a result, converted to the operand type, is an operand of the next
// product without moving between lanes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {
namespace mx {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((__vector_size__(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

template <typename T> struct Piece;
template <> struct Piece<__bf16> {
    typedef bf16x8 V;
    static constexpr int E = 8;
};
template <> struct Piece<float> {
    typedef f32x4 V;
    static constexpr int E = 4;
};

__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(f32x4 a, f32x4 b, f32x16 c)
{
#pragma unroll
    for (int e = 0; e < 4; ++e)
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

// 16 x 16 blocks: lane l = c + 16 g holds row c of A (column c of B), natural
// order over the four lane groups, and D[4 g + i][c] in register i.
__device__ __forceinline__ f32x4 mma16(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma16(f32x4 a, f32x4 b, f32x4 c)
{
#pragma unroll
    for (int e = 0; e < 4; ++e)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

// Piece p of a 32-row result block as an operand (accumulator order), rounded
// once to the operand type.
__device__ __forceinline__ bf16x8 acc_piece(const f32x16 &d, int p, const __bf16 *)
{
    bf16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = (__bf16)d[8 * p + e];
    return v;
}
__device__ __forceinline__ f32x4 acc_piece(const f32x16 &d, int p, const float *)
{
    return f32x4{d[4 * p], d[4 * p + 1], d[4 * p + 2], d[4 * p + 3]};
}

// A [rows][D] tile of T in LDS.  Rows are not padded (a row is what a direct
// load writes); instead the 16-byte chunks of a row are permuted by an XOR
// with swz(row), chosen so that 16 consecutive rows' reads of one chunk, and
// the transpose reads of four rows by four chunks, each cover all 64 banks.
template <typename T, int D> struct Tile {
    static constexpr int kPitch = D * (int)sizeof(T);
    static constexpr int kChunks = kPitch / 16;
    static constexpr int kPieces = kPitch / 32;      // pieces of a row as an operand
    static_assert(kChunks >= 4, "a row is a quarter of the banks or more");

    static __device__ __forceinline__ int swz(int row)
    {
        if constexpr (kChunks >= 16)
            return ((row & 3) << 2) | ((row >> 2) & 3);
        else if constexpr (kChunks == 8)   // two rows per 256 bytes: row bit 0 is the upper half already
            return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
        else
            return (row >> 2) & 3;
    }
    static __device__ __forceinline__ int off(int row, int chunk)
    {
        return row * kPitch + ((chunk ^ swz(row)) << 4);
    }
    // operand over the columns, natural order: row `row` (lane % 32 of a block)
    static __device__ __forceinline__ typename Piece<T>::V row_nat(const unsigned char *t, int row,
                                                                   int p, int hh)
    {
        return *reinterpret_cast<const typename Piece<T>::V *>(t + off(row, 2 * p + hh));
    }
    // operand over the rows (transposed), accumulator order: column col0 + lane % 32.
    // bf16 through the transpose read: within 16 lanes, lane i gets element i % 4
    // of the 8 bytes that lanes i / 4, i / 4 + 4, .. + 12 address (one per row), so
    // a read turns 4 rows x 16 columns.
    static __device__ __forceinline__ typename Piece<T>::V col_acc(const unsigned char *t, int p,
                                                                   int col0, int lane)
    {
        if constexpr (sizeof(T) == 4) {
            const int col = col0 + (lane & 31), r0 = 8 * p + 4 * (lane >> 5);
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = *reinterpret_cast<const float *>(t + off(r0 + e, col >> 2) + (col & 3) * 4);
            return v;
        } else {
            const int row = 16 * p + 4 * (lane >> 5) + ((lane >> 2) & 3);
            const int col = col0 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
            const unsigned char *a = t + off(row, col >> 3) + (col & 7) * 2;
            const unsigned char *b = t + off(row + 8, col >> 3) + (col & 7) * 2;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)a);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)b);
            return __builtin_bit_cast(
                bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

// A lane's byte offset into a tile, from which an operand's pieces follow by an
// XOR with a constant (the chunk permutation is an XOR itself) and a constant
// row offset: one register per operand instead of one per read.  opaque() keeps
// the XORs where they are used.
__device__ __forceinline__ unsigned opaque(unsigned v)
{
    asm volatile("" : "+v"(v));
    return v;
}
template <typename T, int D> struct LaneBase {
    typedef Tile<T, D> TL;
    typedef typename Piece<T>::V V;
    // (t: the tile's LDS address, a constant, which ends up in the instruction)
    static __device__ __forceinline__ V at(unsigned t, unsigned off)
    {
        return *(const __attribute__((address_space(3))) V *)(uintptr_t)(t + off);
    }
    // 32-row operand over the columns, natural order: piece p of row `row`
    static __device__ __forceinline__ unsigned row32(int row, int hh)
    {
        return (unsigned)TL::off(row, hh);
    }
    static __device__ __forceinline__ V piece32(unsigned t, unsigned base, int p)
    {
        return at(t, base ^ ((unsigned)p << 5));
    }
    // 16-row operand
    static __device__ __forceinline__ unsigned row16(int row, int g)
    {
        return (unsigned)TL::off(row, g);
    }
    static __device__ __forceinline__ V piece16(unsigned t, unsigned base, int p)
    {
        return at(t, base ^ ((unsigned)p << 6));
    }
    // transposed operand, natural order (bf16): rows 16 p + 8 hh + e of column
    // 32 d + lane % 32, or with kPerm of the column that makes a result's register
    // 8 j + i of lane half hh stand for column 16 j + 8 hh + i (so that the result, as
    // an operand, meets a natural-order operand: in each 16 columns the middle two
    // groups of four trade places).  fp32: the accumulator order is the natural one,
    // and register r stands for column 8 (r / 4) + 4 hh + r % 4.
    template <bool kPerm> static __device__ __forceinline__ unsigned col(int lane)
    {
        if constexpr (sizeof(T) == 4) {
            const int c = lane & 31;
            return (unsigned)(TL::off(4 * (lane >> 5), c >> 2) + (c & 3) * 4);
        } else {
            const int q = lane & 3, g4 = kPerm ? ((q & 1) << 1) | (q >> 1) : q;
            const int c = 16 * ((lane >> 4) & 1) + 4 * g4;
            return (unsigned)(TL::off(8 * (lane >> 5) + ((lane >> 2) & 3), c >> 3) + (c & 7) * 2);
        }
    }
    static __device__ __forceinline__ V col_piece(unsigned t, unsigned base, int p, int d)
    {
        if constexpr (sizeof(T) == 4) {
            // rows 8 p + 4 hh + e: e changes the permutation's upper two bits, 8 p its lower
            V v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 8 * p + e;
                v[e] = *(const __attribute__((address_space(3))) float *)(uintptr_t)(
                    (base ^ (unsigned)((d << 7) ^ (TL::swz(r) << 4))) + (t + (unsigned)(r * TL::kPitch)));
            }
            return v;
        } else {
            const unsigned a = base ^ ((unsigned)d << 6);
            const unsigned x = a + (t + 16u * p * TL::kPitch), y = (a ^ 16u) + (t + (16u * p + 4) * TL::kPitch);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)x);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)y);
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

__device__ __forceinline__ float exp2_fast(float v)
{
    return __builtin_amdgcn_exp2f(v);
}

__device__ __forceinline__ int uniform_int(int v)
{
    return __builtin_amdgcn_readfirstlane(v);
}
// Maximum / sum of a value and the one the lane 32 away holds, kept by both.
// (The second result of the swap goes through an empty asm statement: read by
// one instruction directly, the two have been taken for the same register.)
__device__ __forceinline__ float half_max(float v)
{
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    unsigned b = s[1];
    asm volatile("" : "+v"(b));
    return fmaxf(__builtin_bit_cast(float, (unsigned)s[0]), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float half_sum(float v)
{
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    unsigned b = s[1];
    asm volatile("" : "+v"(b));
    return __builtin_bit_cast(float, (unsigned)s[0]) + __builtin_bit_cast(float, b);
}

__device__ __forceinline__ unsigned pack_bf16(float a, float b)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(unsigned, bf16x2{(__bf16)a, (__bf16)b});
}

// Writes columns col0 .. col0 + 31 of the lane's row from a transposed result
// block (rows = columns of the output): `row` points at the row's column 0.
// fp32 registers 4 g .. 4 g + 3 are four consecutive columns; for bf16 the two
// lane halves trade pairs of them so that each lane writes 16 bytes.
__device__ __forceinline__ void store_row(float *row, int col0, int hh, bool valid, const f32x16 &d)
{
    if (!valid)
        return;
#pragma unroll
    for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4 *>(row + col0 + 8 * g + 4 * hh) =
            f32x4{d[4 * g], d[4 * g + 1], d[4 * g + 2], d[4 * g + 3]};
}
__device__ __forceinline__ void store_row(__bf16 *row, int col0, int hh, bool valid, const f32x16 &d)
{
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
        unsigned out[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const auto s = __builtin_amdgcn_permlane32_swap(
                pack_bf16(d[4 * g + 2 * e], d[4 * g + 2 * e + 1]),
                pack_bf16(d[4 * g + 4 + 2 * e], d[4 * g + 4 + 2 * e + 1]), false, false);
            out[e] = s[0];
            out[2 + e] = s[1];
        }
        if (valid)
            *reinterpret_cast<u32x4 *>(row + col0 + 8 * g + 8 * hh) =
                u32x4{out[0], out[1], out[2], out[3]};
    }
}

// Raw buffer descriptor over `bytes` bytes from `base` (both wave-uniform).
__device__ __forceinline__ u32x4 buffer_words(const void *base, unsigned bytes)
{
    const uint64_t a = (uint64_t)(uintptr_t)base;
    u32x4 w;
    w[0] = (unsigned)uniform_int((int)(unsigned)a);
    w[1] = (unsigned)uniform_int((int)(unsigned)(a >> 32)) & 0xffffu;
    w[2] = (unsigned)uniform_int((int)bytes);
    w[3] = 0x00020000u;
    return w;
}

// 16 bytes per lane from the buffer into LDS at dst + 16 lane.  Written as
// assembly because the compiler waits for every such load before any LDS read;
// the reader waits with wait_vmcnt and a barrier instead.  (One wait state
// between writing m0 and the load that reads it.)
__device__ __forceinline__ void lds_load16(unsigned dst, u32x4 rsrc, unsigned voff, unsigned soff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(uniform_int((int)dst)), "v"(voff), "s"(rsrc), "s"(uniform_int((int)soff)) : "memory", "m0");
}

template <int n> __device__ __forceinline__ void wait_vmcnt()
{
    static_assert(n >= 0 && n < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" :: "n"(n) : "memory");
}

// Barrier for LDS hand-offs only: this wave's LDS accesses are done; global
// loads and stores stay in flight.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ unsigned lds_addr(const void *p)
{
    return (unsigned)uniform_int(
        (int)(unsigned)(uintptr_t)(const __attribute__((address_space(3))) void *)p);
}

// A wave's share of loading a [kRows][D] tile: the 1 KB blocks from w kPer on, lane l
// writing bytes 16 l .. 16 l + 15 of each, so the chunk permutation is
// applied to the source.  Rows past the last valid one repeat it: what is
// masked afterwards is then finite whenever the sequence's own values are, and
// nothing outside the sequence is read.
template <typename T, int D, int kRows, int kWaves> struct TileLoad {
    typedef Tile<T, D> TL;
    static constexpr int kBlocks = kRows * TL::kPitch / 1024;
    static_assert(kBlocks % kWaves == 0, "whole blocks per wave");
    static constexpr int kPer = kBlocks / kWaves;    // load instructions per wave

    static __device__ __forceinline__ void issue(unsigned dst, const T *base, int64_t stride,
                                                 int64_t row0, int64_t nrows, int w, int lane)
    {
        const int rows = uniform_int((int)(nrows - row0 < kRows ? nrows - row0 : kRows));   // >= 1
        const unsigned sb = (unsigned)uniform_int((int)((unsigned)stride * (unsigned)sizeof(T)));
        const u32x4 rs = buffer_words(base + row0 * stride, (unsigned)(rows - 1) * sb + TL::kPitch);
        constexpr int kBlkRows = TL::kPitch >= 1024 ? 1 : 1024 / TL::kPitch;   // rows of a 1 KB block
        if (TL::kPitch <= 1024 && rows == kRows) {
            // whole: block b's rows are kBlkRows b further on, a scalar offset, and only
            // the chunk permutation differs
            const int row = 16 * lane / TL::kPitch, chunk = 16 * lane % TL::kPitch / 16;
            const unsigned lo = (unsigned)row * sb;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int b = w * kPer + i;
                lds_load16(dst + 1024u * (unsigned)b, rs,
                           lo + (unsigned)((chunk ^ TL::swz(row + b * kBlkRows)) << 4),
                           (unsigned)(b * kBlkRows) * sb);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = w * kPer + i;
            const int row = (b * 1024 + 16 * lane) / TL::kPitch;
            const int chunk = ((b * 1024 + 16 * lane) % TL::kPitch) / 16;
            const int src = row < rows ? row : rows - 1;
            lds_load16(dst + 1024u * (unsigned)b, rs,
                       (unsigned)src * sb + (unsigned)((chunk ^ TL::swz(row)) << 4), 0);
        }
    }
};

}  // namespace mx
}  // namespace ssd
