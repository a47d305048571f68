// Device helpers of the recurrence's and the convolution's kernels: elements
// of any type one or two at a time. Not part of the ABI.
//
// Lanes own channels: a wave reads 64 (or 128, two per lane) neighbouring
// channels of a token at once and walks along the tokens, so that a channel's
// whole arithmetic stays in one lane. With an odd number of channels the last
// pair begins at the last but one, which two lanes then have: both compute and
// store the same values. (Rows of 2047 channels one per lane: convolution of
// 37,000 tokens 123 us, gradients 209; in pairs 76 and 133.)
#pragma once

#include <stdint.h>

#include <type_traits>

#include <hip/hip_runtime.h>

#include "gdn2_device.h"
#include "gdn2_mixer.h"
#include "gdn2_packed.h"

namespace gdn2 {
namespace dev {

// VEC elements of type E as they lie in memory.
template <int E, int VEC>
using Raw = std::conditional_t<E == E_F32, std::conditional_t<VEC == 2, f32x2, float>,
                               std::conditional_t<VEC == 2, uint32_t, uint16_t>>;
template <int E>
using Elem = std::conditional_t<E == E_F32, float, uint16_t>;

template <int E>
__device__ __forceinline__ float el_f32(uint16_t b)
{
    if constexpr (E == E_F16) return (float)__builtin_bit_cast(_Float16, b);
    else return __uint_as_float((uint32_t)b << 16);
}
template <int E>
__device__ __forceinline__ uint16_t f32_el(float x)  // rounded to nearest even
{
    if constexpr (E == E_F16) return __builtin_bit_cast(uint16_t, (_Float16)x);
    else return __builtin_bit_cast(uint16_t, (__bf16)x);
}
template <int E, int VEC>
__device__ __forceinline__ Raw<E, VEC> ld_raw(const void *p, int64_t row, uint32_t col)
{
    Raw<E, VEC> r;  // (at any element's address)
    __builtin_memcpy(&r, static_cast<const Elem<E> *>(p) + row + col, sizeof r);
    return r;
}
// R rows from t0 on (those from hi on read row hi - 1).
template <int E, int VEC, int R>
__device__ __forceinline__ void ld_rows(const void *p, int64_t stride, int t0, int hi, uint32_t col, Raw<E, VEC> (&r)[R])
{
    if (t0 + R <= hi) {
        int64_t row = t0 * stride;
#pragma unroll
        for (int i = 0; i < R; ++i, row += stride) r[i] = ld_raw<E, VEC>(p, row, col);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) r[i] = ld_raw<E, VEC>(p, (int64_t)(t0 + i < hi ? t0 + i : hi - 1) * stride, col);
    }
}
template <int E, int VEC>
__device__ __forceinline__ void widen(Raw<E, VEC> r, float (&o)[VEC])
{
    if constexpr (E == E_F32) {
        if constexpr (VEC == 2) {
            o[0] = r[0];
            o[1] = r[1];
        } else {
            o[0] = r;
        }
    } else if constexpr (VEC == 2) {
        o[0] = el_f32<E>((uint16_t)r);
        o[1] = el_f32<E>((uint16_t)(r >> 16));
    } else {
        o[0] = el_f32<E>(r);
    }
}
template <int E, int VEC>
__device__ __forceinline__ void st_el(void *p, int64_t row, uint32_t col, const float (&x)[VEC])
{
    Raw<E, VEC> r;
    if constexpr (E == E_F32) {
        if constexpr (VEC == 2) r = f32x2{x[0], x[1]};
        else r = x[0];
    } else if constexpr (VEC == 2) {
        r = (uint32_t)f32_el<E>(x[0]) | (uint32_t)f32_el<E>(x[1]) << 16;
    } else {
        r = f32_el<E>(x[0]);
    }
    __builtin_memcpy(static_cast<Elem<E> *>(p) + row + col, &r, sizeof r);
}
template <int E, int VEC>
__device__ __forceinline__ void ld_el(const void *p, int64_t row, uint32_t col, float (&x)[VEC])
{
    widen<E, VEC>(ld_raw<E, VEC>(p, row, col), x);
}
// An element of one of two types (float32 or E).
template <int E>
__device__ __forceinline__ float ld_either(const void *p, bool f32, int64_t i)
{
    if constexpr (E == E_F32) return static_cast<const float *>(p)[i];
    else return f32 ? static_cast<const float *>(p)[i] : el_f32<E>(static_cast<const uint16_t *>(p)[i]);
}
template <int E>
__device__ __forceinline__ void st_either(void *p, bool f32, int64_t i, float x)
{
    if constexpr (E == E_F32) static_cast<float *>(p)[i] = x;
    else if (f32) static_cast<float *>(p)[i] = x;
    else static_cast<uint16_t *>(p)[i] = f32_el<E>(x);
}

// Workgroups are dealt to the eight XCDs in turn; this hands each XCD a run
// of consecutive work items, so that neighbours in memory share an L2 (rows
// that are not multiples of a cache line have lines in two workgroups).
__device__ __forceinline__ uint32_t xcd_run(uint32_t id, uint32_t count)
{
    const uint32_t q = count / 8, r = count % 8, x = id % 8;
    return x * q + (x < r ? x : r) + id / 8;
}

// Calls f(n) for every empty sequence among a workgroup's share of all
// sequences (share `part` of `parts`), each by one wave, with n wave-uniform.
template <class F>
__device__ __forceinline__ void for_empty(const Packed &b, uint32_t part, uint32_t parts, F f)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    if (!b.cu) {
        if (b.T == 0 && part == 0 && wave == 0) f(0);
        return;
    }
    const int n0 = (int)((int64_t)b.N * part / parts), n1 = (int)((int64_t)b.N * (part + 1) / parts);
    for (int n = n0 + 64 * wave; n < n1; n += 64 * waves) {
        uint64_t m = __ballot(n + lane < n1 && b.entry(n + lane) >= b.entry(n + lane + 1));
        while (m) {
            f(n + __builtin_ctzll(m));
            m &= m - 1;
        }
    }
}

}  // namespace dev
}  // namespace gdn2
