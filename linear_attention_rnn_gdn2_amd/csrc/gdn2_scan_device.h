// The gated linear recurrence per channel (CDNA4, gfx950):
//
//     h_t = a_t h_{t-1} + u_t,   a = e^g,   u = m w x,
//     m = 1, 1 - a or sqrt(1 - a^2);   out_t = h_t
//
// and its gradients, with c_t what reaches h_{t-1} from behind:
//
//     dh_t = dout_t + c_{t+1},   c_t = a_t dh_t,
//     dx = m w dh,   dw = m x dh,   dg = dh (a h_{t-1} + m' w x),
//     m' = 0, -a or -a^2 / m (0 where m is 0)
//
// Tokens depend on each other through pairs (A, H) alone, the product of the
// decays and the end state from zero: (A2, H2) after (A1, H1) is (A1 A2, A2 H1
// + H2); a sequence's start cuts the product off. The gradients' pairs are
// (A, C), joined from the other end. A wave holds 8 tokens of 64
// (or 128) channels in registers, makes its pair, the workgroup's waves
// exchange pairs through LDS, and each walks its tokens a second time from its
// true entering state.
//
// Slow decays: a near 1 is rounded to 2^-25, which moves the rate of a decay
// of 2^-10 by 3e-5, all steps alike where g stays the same. A decay is
// therefore held in two parts, a = hi + lo, and a product of decays as the sum
// of its g.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

#include "../../include/gdn2.h"
#include "gdn2_internal.h"
#include "gdn2_mixer_device.h"

namespace gdn2 {
namespace scan {

using namespace dev;

constexpr int R = 8;  // tokens per wave and tile

// e^g in two parts. For |g| < 1/4 the second is what the first leaves of 1 +
// (e^g - 1), the bracket g times a polynomial fitted to (e^g - 1) / g on [-1/4,
// 0] (at most 4.7e-9 off there, relative; 1e-7 as float32 evaluates it); a
// faster decay forgets a state within four steps, and the first part's 2^-24
// is enough.
struct Decay {
    float hi, lo;
};
__device__ __forceinline__ Decay decay(float g)
{
    float e = fmaf(g, 0.007513605989515781f, 0.04149065539240837f);
    e = fmaf(g, e, 0.16665108501911163f);
    e = fmaf(g, e, 0.4999995231628418f);
    e = fmaf(g, e, 1.0f);
    Decay a;
    a.hi = ex2(g * 1.44269504088896340736f);
    a.lo = fabsf(g) < 0.25f ? fmaf(g, e, 1.0f - a.hi) : 0.0f;
    return a;
}
__device__ __forceinline__ float advance(Decay a, float h, float u) { return fmaf(a.hi, h, fmaf(a.lo, h, u)); }  // a h + u
__device__ __forceinline__ float times(Decay a, float x) { return fmaf(a.hi, x, a.lo * x); }
template <int KIND>
__device__ __forceinline__ float factor(Decay a)
{
    if constexpr (KIND == GDN2_SCAN_INPUT_NONE) return 1.0f;
    const float rest = (1.0f - a.hi) - a.lo;  // 1 - a
    if constexpr (KIND == GDN2_SCAN_INPUT_CONVEX) return rest;
    return __builtin_amdgcn_sqrtf(rest * (1.0f + a.hi));
}
// The derivative of the factor m by g.
template <int KIND>
__device__ __forceinline__ float factor_slope(Decay a, float m)
{
    if constexpr (KIND == GDN2_SCAN_INPUT_NONE) return 0.0f;
    if constexpr (KIND == GDN2_SCAN_INPUT_CONVEX) return -a.hi;
    return m > 0.0f ? -a.hi * a.hi * __builtin_amdgcn_rcpf(m) : 0.0f;
}

// A state's VEC values: float32 or bf16 at element `at`; zero without a state.
template <int VEC>
__device__ __forceinline__ void state_in(const ScanParams &p, int n, uint32_t col, float (&h)[VEC])
{
#pragma unroll
    for (int v = 0; v < VEC; ++v)
        h[v] = p.h0 ? state_ld(static_cast<const float *>(p.h0), p.h0_bf16, (int64_t)n * p.D + col + v) : 0.0f;
}
template <int VEC>
__device__ __forceinline__ void state_out(const ScanParams &p, int n, uint32_t col, const float (&h)[VEC])
{
#pragma unroll
    for (int v = 0; v < VEC; ++v) state_st(static_cast<float *>(p.ht), p.ht_bf16, (int64_t)n * p.D + col + v, h[v]);
}

// The inputs of a wave's R tokens as loaded (rows past `hi` read row hi - 1).
template <int E, int G, int VEC>
struct Rows {
    Raw<E, VEC> x[R], w[R];
    Raw<G, VEC> g[R];

    __device__ __forceinline__ void load(const ScanParams &p, int t0, int hi, uint32_t col)
    {
        ld_rows<E, VEC, R>(p.x, p.sx, t0, hi, col, x);
        ld_rows<G, VEC, R>(p.g, p.sg, t0, hi, col, g);
        if (p.w) ld_rows<E, VEC, R>(p.w, p.sw, t0, hi, col, w);
    }
    __device__ __forceinline__ void wide(const ScanParams &p, int i, float (&gf)[VEC], float (&wf)[VEC], float (&xf)[VEC]) const
    {
        widen<E, VEC>(x[i], xf);
        widen<G, VEC>(g[i], gf);
        if (p.w) {
            widen<E, VEC>(w[i], wf);
        } else {
#pragma unroll
            for (int v = 0; v < VEC; ++v) wf[v] = 1.0f;
        }
    }
    // The tokens' decays and gated inputs u, and the sum of g over the first cnt.
    template <int KIND>
    __device__ __forceinline__ void inputs(const ScanParams &p, int cnt, Decay (&a)[R][VEC], float (&u)[R][VEC], float (&sum)[VEC]) const
    {
#pragma unroll
        for (int v = 0; v < VEC; ++v) sum[v] = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float gf[VEC], wf[VEC], xf[VEC];
            wide(p, i, gf, wf, xf);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                a[i][v] = decay(gf[v]);
                u[i][v] = factor<KIND>(a[i][v]) * (wf[v] * xf[v]);
                sum[v] += i < cnt ? gf[v] : 0.0f;
            }
        }
    }
};

// Where a workgroup works: channels of a lane, and its range of tokens.
template <int VEC>
struct Place {
    uint32_t parts, range, col;
    bool on;
    int lane, wave;
    __device__ __forceinline__ explicit Place(const ScanParams &p, bool groups = false)
    {
        const uint32_t cols = (p.D + 64 * VEC - 1) / (64 * VEC);
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        parts = gridDim.x / cols;
        uint32_t cb;
        if (groups) {
            // groups of sequences by length: the columns of a group one after the other
            const uint32_t id = snake(blockIdx.x, gridDim.x);
            range = id / cols;
            cb = id % cols;
        } else {
            const uint32_t id = xcd_run(blockIdx.x, gridDim.x);
            range = id / cols;
            cb = id % cols;
        }
        const uint32_t c0 = (cb * 64 + lane) * VEC, last = p.D - VEC;
        on = c0 < (uint32_t)p.D;
        col = c0 < last ? c0 : last;  // lanes past the last channel read it and store nothing
    }
    // Workgroups that share a compute unit are 256 apart: every other 256 in reverse.
    __device__ static __forceinline__ uint32_t snake(uint32_t id, uint32_t count)
    {
        const uint32_t row = id / 256, left = count - row * 256, n = left < 256 ? left : 256;
        return row & 1 ? row * 256 + n - 1 - id % 256 : id;
    }
};

__device__ __forceinline__ Packed packed(const ScanParams &p) { return Packed{p.cu, p.cu64, p.N, p.T}; }

// A sum of g that stands for: a sequence begins among these tokens.
constexpr float CUT = INFINITY;

// The state (or gradient) behind some tokens, from h before them.
__device__ __forceinline__ float join(const float *s, float h)  // s: hi (CUT: a start), lo, end state
{
    const float e = advance(Decay{s[0], s[1]}, h, s[2]);
    return s[0] == CUT ? s[2] : e;
}

// R tokens from an entering state to the one behind them: f(i, h) sees the
// state behind token i. PLAIN: the tokens all exist and none begins a sequence.
template <int VEC, bool PLAIN, class F>
__device__ __forceinline__ void walk(const ScanParams &p, const Slice<R> &s, uint32_t col, const Decay (&a)[R][VEC],
                                     const float (&u)[R][VEC], float (&h)[VEC], F f)
{
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (!PLAIN && i >= s.cnt) break;
        if (!PLAIN && s.starts >> i & 1) state_in<VEC>(p, s.seq(i), col, h);
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = advance(a[i][v], h[v], u[i][v]);
        f(i, h);
    }
}

// f<E, G, VEC, KIND>() for the call's types and options.
template <class F>
hipError_t for_types(const ScanParams &p, bool pairs, F f)
{
    auto kind = [&](auto e, auto g, auto vec) {
        if (p.scale == GDN2_SCAN_INPUT_NONE) f(e, g, vec, std::integral_constant<int, GDN2_SCAN_INPUT_NONE>{});
        else if (p.scale == GDN2_SCAN_INPUT_CONVEX) f(e, g, vec, std::integral_constant<int, GDN2_SCAN_INPUT_CONVEX>{});
        else f(e, g, vec, std::integral_constant<int, GDN2_SCAN_INPUT_UNIT>{});
    };
    auto vec = [&](auto e, auto g) {
        if (pairs) kind(e, g, std::integral_constant<int, 2>{});
        else kind(e, g, std::integral_constant<int, 1>{});
    };
    constexpr std::integral_constant<int, E_F32> f32{};
    constexpr std::integral_constant<int, E_F16> f16{};
    constexpr std::integral_constant<int, E_BF16> bf16{};
    if (p.io == E_F32) vec(f32, f32);
    else if (p.io == E_F16 && p.g_f32) vec(f16, f32);
    else if (p.io == E_F16) vec(f16, f16);
    else if (p.g_f32) vec(bf16, f32);
    else vec(bf16, bf16);
    return hipGetLastError();
}
inline int64_t column_blocks(const ScanParams &p, int per) { return ((int64_t)p.D + per - 1) / per; }

}  // namespace scan
}  // namespace gdn2
