// Device helpers of the scalar-gated delta rule's kernels: two-part bf16
// operands, staged tiles and MFMA fragments. Not part of the ABI.
//
// Precision. Every product of the rule runs on bf16 MFMA with float32
// accumulation, and a float32 operand is taken as two bf16 parts, x = h + l
// with h = bf16(x), l = bf16(x - h): 16 significant bits, 2^-18 relative.
// Products of two such operands drop l l (2^-18 of the product). bf16 inputs
// are one part, fp16 inputs are exactly two. The state, the chunk's WY
// solution and all sums are float32.
//
// Fragments (lane = 16 q4 + l16). A 16x16 accumulator tile holds rows
// 4 q4 + e (e = 0..3) of column l16. As the right operand of the next product
// (32 contracted rows = two stacked tiles) the lane's eight values are rows
// 4 q4 + e of the first and of the second tile: the contraction runs in that
// order on both sides, so an accumulator becomes an operand without leaving
// its lane. The left operand then reads two runs of four columns,
// 4 q4 .. and 16 + 4 q4 .. of the 32.
#pragma once

#include "gdn2_delta.h"
#include "gdn2_device.h"

namespace gdn2 {
namespace dev {

constexpr float LOG2E = 1.44269504088896340736f;
constexpr int PSTR = 144;  // LDS row stride of a 64-column bf16 plane (bytes): 16 rows apart in banks by 16 bytes

// x = h + l
__device__ __forceinline__ void split4(f32x4 x, bf16x4 &h, bf16x4 &l)
{
    h = f32x4_to_bf16(x);
    l = f32x4_to_bf16(x - __builtin_convertvector(h, f32x4));
}
__device__ __forceinline__ void split8(f32x8 x, bf16x8 &h, bf16x8 &l)
{
    h = f32x8_to_bf16(x);
    l = f32x8_to_bf16(x - __builtin_convertvector(h, f32x8));
}

template <int IO>
__device__ __forceinline__ float io_f32(uint16_t b)
{
    if constexpr (IO == IO_F16) return (float)__builtin_bit_cast(_Float16, b);
    else return __uint_as_float((uint32_t)b << 16);
}
template <int IO>
__device__ __forceinline__ uint16_t f32_io(float x)  // rounded to nearest even
{
    if constexpr (IO == IO_F16) return __builtin_bit_cast(uint16_t, (_Float16)x);
    else return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// The left operand of one 32-wide step from a row-major tile in LDS: row
// `row`, columns c0 + 4 q4 .. + 3 and c0 + 16 + 4 q4 .. + 3.
__device__ __forceinline__ bf16x8 ld_row(const char *base, int stride, int row, int c0, int q4)
{
    const char *a = base + row * stride + 2 * (c0 + 4 * q4);
    return cat4(*reinterpret_cast<const bf16x4 *>(a), *reinterpret_cast<const bf16x4 *>(a + 32));
}
// The same operand of the transposed tile: element (m, k) is tile[k][m],
// rows k = k0 + 4 q4 .. and k0 + 16 + 4 q4 .., columns m = c0 + l16.
__device__ __forceinline__ bf16x8 ld_col(const char *base, int stride, int k0, int c0, int q4, int l16)
{
    const int a = (k0 + 4 * q4 + (l16 >> 2)) * stride + 2 * (c0 + 4 * (l16 & 3));
    return cat4(lds_tr(base, a), lds_tr(base, a + 16 * stride));
}
// As ld_row and ld_col with the contraction in plain order (8 q4 .. 8 q4 + 7).
__device__ __forceinline__ bf16x8 ld_row_plain(const char *base, int stride, int row, int c0, int q4)
{
    return *reinterpret_cast<const bf16x8 *>(base + row * stride + 2 * (c0 + 8 * q4));
}
__device__ __forceinline__ bf16x8 ld_col_plain(const char *base, int stride, int k0, int c0, int q4, int l16)
{
    const int a = (k0 + 8 * q4 + (l16 >> 2)) * stride + 2 * (c0 + 4 * (l16 & 3));
    return cat4(lds_tr(base, a), lds_tr(base, a + 4 * stride));
}

// acc + (ah [+ al]) (bh + bl), without al bl
template <bool TWO>
__device__ __forceinline__ f32x4 mfma_split(bf16x8 ah, bf16x8 al, bf16x8 bh, bf16x8 bl, f32x4 acc)
{
    acc = mfma_bf16(ah, bh, acc);
    acc = mfma_bf16(ah, bl, acc);
    if constexpr (TWO) acc = mfma_bf16(al, bh, acc);
    return acc;
}

// 16 bytes of io values as one bf16 plane (bf16) or two (fp16: exact).
template <int NP>
__device__ __forceinline__ void st_parts(char *base, int plane_bytes, int off, i32x4 raw)
{
    if constexpr (NP == 1) {
        *reinterpret_cast<i32x4 *>(base + off) = raw;
    } else {
        bf16x8 h, l;
        split8(__builtin_convertvector(__builtin_bit_cast(f16x8, raw), f32x8), h, l);
        *reinterpret_cast<bf16x8 *>(base + off) = h;
        *reinterpret_cast<bf16x8 *>(base + plane_bytes + off) = l;
    }
}

// Row and 16-byte column of chunk ci (0 .. 383) of a record's plane.
__device__ __forceinline__ void plane_pos(int ci, int &row, int &col)
{
    if (ci < 128) {
        row = ci >> 2;
        col = ci & 3;
    } else {
        row = 32 + ((ci - 128) >> 3);
        col = (ci - 128) & 7;
    }
}

__device__ __forceinline__ int64_t delta_item(const DeltaParams &p, int64_t slot, int hv) { return slot * p.HV + hv; }

// Sum over the 16 lanes of a row (lanes with equal q4); every lane gets it.
__device__ __forceinline__ float sum16(float x)
{
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x128, 0xf, 0xf, true));  // row_ror:8
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x124, 0xf, 0xf, true));  // row_ror:4
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x122, 0xf, 0xf, true));  // row_ror:2
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x121, 0xf, 0xf, true));  // row_ror:1
    return x;
}

}  // namespace dev
}  // namespace gdn2
