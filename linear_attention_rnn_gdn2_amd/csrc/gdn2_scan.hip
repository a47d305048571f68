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
// of 2^-10 by 3e-5, all steps alike where g stays the same. For -ln 2 < g <= 0
// the step is therefore h + (e h + u) with e = e^g - 1 (a polynomial, relative
// error 1e-7), and a product of decays is held as the sum of its g.
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "../../include/gdn2.h"
#include "gdn2_internal.h"
#include "gdn2_mixer_device.h"

namespace gdn2 {
namespace {

using namespace dev;

constexpr int R = 8;  // tokens per wave and tile

// A token's decay in one register: e^g - 1 with the sign bit set where -ln 2
// < g <= 0, else e^g.
__device__ __forceinline__ float decay(float g)
{
    float e = fmaf(g, 0.0010361977620050311f, 0.008072594180703163f);
    e = fmaf(g, e, 0.04157528653740883f);
    e = fmaf(g, e, 0.16665200889110565f);
    e = fmaf(g, e, 0.49999913573265076f);
    e = fmaf(g, e, 1.0f) * g;
    const float a = ex2(g * 1.44269504088896340736f);
    return g > -0.69314718f && g <= 0.0f ? __uint_as_float(__float_as_uint(e) | 0x80000000u) : a;
}
__device__ __forceinline__ bool slow(float c) { return (int)__float_as_uint(c) < 0; }
__device__ __forceinline__ float advance(float c, float h, float u)  // a h + u
{
    return fmaf(c, h, u) + (slow(c) ? h : 0.0f);
}
__device__ __forceinline__ float times_a(float c, float x) { return fmaf(c, x, slow(c) ? x : 0.0f); }
__device__ __forceinline__ float rate(float c) { return slow(c) ? 1.0f + c : c; }
__device__ __forceinline__ float factor(int kind, float c)
{
    if (kind == GDN2_SCAN_INPUT_NONE) return 1.0f;
    if (kind == GDN2_SCAN_INPUT_CONVEX) return slow(c) ? -c : 1.0f - c;
    return __builtin_amdgcn_sqrtf(slow(c) ? -c * (2.0f + c) : (1.0f - c) * (1.0f + c));
}
__device__ __forceinline__ float factor_slope(int kind, float c, float m)
{
    if (kind == GDN2_SCAN_INPUT_NONE) return 0.0f;
    const float a = rate(c);
    if (kind == GDN2_SCAN_INPUT_CONVEX) return -a;
    return m > 0.0f ? -a * a * __builtin_amdgcn_rcpf(m) : 0.0f;
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
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t t = t0 + i < hi ? t0 + i : hi - 1;
            x[i] = ld_raw<E, VEC>(p.x, t * p.sx, col);
            g[i] = ld_raw<G, VEC>(p.g, t * p.sg, col);
        }
        if (p.w) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int64_t t = t0 + i < hi ? t0 + i : hi - 1;
                w[i] = ld_raw<E, VEC>(p.w, t * p.sw, col);
            }
        }
    }
    // Token i's g, decay, w and x.
    __device__ __forceinline__ void at(const ScanParams &p, int i, float (&gf)[VEC], float (&c)[VEC], float (&wf)[VEC],
                                       float (&xf)[VEC]) const
    {
        widen<E, VEC>(x[i], xf);
        widen<G, VEC>(g[i], gf);
        if (p.w) {
            widen<E, VEC>(w[i], wf);
        } else {
#pragma unroll
            for (int v = 0; v < VEC; ++v) wf[v] = 1.0f;
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) c[v] = decay(gf[v]);
    }
};

// Where a workgroup works: channels of a lane, and its range of tokens.
template <int VEC>
struct Place {
    uint32_t id, parts, range, c0, col;
    bool on;
    int lane, wave;
    __device__ __forceinline__ explicit Place(const ScanParams &p)
    {
        const uint32_t cols = (p.D + 64 * VEC - 1) / (64 * VEC);
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        parts = gridDim.x / cols;
        id = xcd_run(blockIdx.x, gridDim.x);
        range = id / cols;
        c0 = (id % cols * 64 + lane) * VEC;
        on = c0 < (uint32_t)p.D;
        col = on ? c0 : p.D - VEC;  // lanes past the last channel read it and store nothing
    }
};

__device__ __forceinline__ Packed packed(const ScanParams &p) { return Packed{p.cu, p.cu64, p.N, p.T}; }

// The mark of a pair whose tokens begin a sequence: in the place of a decay
// (which is above -0.5), and in the place of a sum of g.
constexpr float CUT = -1.0f, CUT_SUM = INFINITY;

// Joins the waves' pairs (decay, end state) in order: the state that enters
// wave `wave` and the one behind the last wave, from h.
template <int NW, int VEC>
__device__ __forceinline__ void join_waves(const float (*pair)[64 * VEC * 2], int wave, int lane, float (&enter)[VEC], float (&h)[VEC])
{
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const float *s = &pair[w][lane * VEC * 2];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            if (w == wave) enter[v] = h[v];
            const float c = s[2 * v], H = s[2 * v + 1];
            h[v] = c == CUT ? H : advance(c, h[v], H);
        }
    }
}

// The forward over a range of tokens: a group of whole sequences, or a tile
// whose entering state is known.
template <int E, int G, int VEC, int NW>
__global__ __launch_bounds__(NW * 64) void scan_fwd_kernel(ScanParams p)
{
    __shared__ float pair[2][NW][64 * VEC * 2];
    const Place<VEC> at(p);
    const Packed b = packed(p);
    const int tokens = b.tokens(), lane = at.lane, wave = at.wave;
    if (p.ht)
        for_empty(b, at.range, at.parts, [&](int n) {
            float h[VEC];
            state_in<VEC>(p, n, at.col, h);
            if (at.on) state_out<VEC>(p, n, at.c0, h);
        });
    int lo, hi;
    float h[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = 0.0f;
    if (p.groups) {
        lo = b.start_from((int)((int64_t)p.T * at.range / p.groups));
        hi = (int)at.range + 1 < p.groups ? b.start_from((int)((int64_t)p.T * (at.range + 1) / p.groups)) : tokens;
    } else {
        lo = at.range * SCAN_TILE;
        hi = lo + SCAN_TILE < tokens ? lo + SCAN_TILE : tokens;
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = p.end[(int64_t)at.range * p.D + at.col + v];
    }
    if (lo >= hi) return;
    Cursor cur(b);
    Slice<R> s, next;
    Rows<E, G, VEC> rows;
    next.set(cur, lo + wave * R, hi, tokens);
    rows.load(p, lo + wave * R, hi, at.col);
    int buf = 0;
    for (int t = lo; t < hi; t += NW * R, buf ^= 1) {
        s = next;
        float c[R][VEC], u[R][VEC], sum[VEC], H[VEC], enter[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) sum[v] = H[v] = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float g[VEC], w[VEC], x[VEC];
            rows.at(p, i, g, c[i], w, x);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                u[i][v] = factor(p.scale, c[i][v]) * (w[v] * x[v]);
                if (i < s.cnt) sum[v] += g[v];
            }
        }
        const int tn = t + NW * R;
        if (tn < hi) {
            rows.load(p, tn + wave * R, hi, at.col);
            next.set(cur, tn + wave * R, hi, tokens);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (i >= s.cnt) break;
            if (s.starts >> i & 1) state_in<VEC>(p, s.seq(i), at.col, H);
#pragma unroll
            for (int v = 0; v < VEC; ++v) H[v] = advance(c[i][v], H[v], u[i][v]);
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            pair[buf][wave][(lane * VEC + v) * 2] = s.starts ? CUT : decay(sum[v]);
            pair[buf][wave][(lane * VEC + v) * 2 + 1] = H[v];
        }
        __syncthreads();
        join_waves<NW, VEC>(pair[buf], wave, lane, enter, h);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (i >= s.cnt) break;
            if (s.starts >> i & 1) state_in<VEC>(p, s.seq(i), at.col, enter);
#pragma unroll
            for (int v = 0; v < VEC; ++v) enter[v] = advance(c[i][v], enter[v], u[i][v]);
            if (at.on) st_el<E, VEC>(p.out, (int64_t)(s.t0 + i) * p.so, at.c0, enter);
            if (s.lasts >> i & 1 && p.ht && at.on) state_out<VEC>(p, s.seq(i), at.c0, enter);
        }
    }
}

// What the gradient needs of dout: the loaded rows, and dout plus, on a
// sequence's last token, the final state's gradient.
template <int E, int VEC>
struct OutRows {
    Raw<E, VEC> d[R];
    __device__ __forceinline__ void load(const ScanParams &p, int t0, int hi, uint32_t col)
    {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t t = t0 + i < hi ? t0 + i : hi - 1;
            d[i] = ld_raw<E, VEC>(p.dout, t * p.sdo, col);
        }
    }
    __device__ __forceinline__ void at(const ScanParams &p, int i, const Slice<R> &s, uint32_t col, float (&o)[VEC]) const
    {
        widen<E, VEC>(d[i], o);
        if (s.lasts >> i & 1 && p.dht) {
            const float *q = p.dht + (int64_t)s.seq(i) * p.D + col;
#pragma unroll
            for (int v = 0; v < VEC; ++v) o[v] += q[v];
        }
    }
};

// What R tokens are to the others: the end state from zero, and (BWD) the
// gradient that leaves the first of them backwards, nothing reaching the last.
template <int VEC, bool BWD>
__device__ __forceinline__ void summarise(const ScanParams &p, const Slice<R> &s, uint32_t col, const float (&c)[R][VEC],
                                          const float (&u)[R][VEC], const float (&d)[R][VEC], float (&H)[VEC], float (&C)[VEC])
{
#pragma unroll
    for (int v = 0; v < VEC; ++v) H[v] = C[v] = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (i >= s.cnt) break;
        if (s.starts >> i & 1) state_in<VEC>(p, s.seq(i), col, H);
#pragma unroll
        for (int v = 0; v < VEC; ++v) H[v] = advance(c[i][v], H[v], u[i][v]);
    }
    if constexpr (BWD) {
#pragma unroll
        for (int i = R - 1; i >= 0; --i) {
            if (i >= s.cnt) continue;
            // a sequence's first token hands nothing to the token before it
            const bool cut = s.starts >> i & 1;
#pragma unroll
            for (int v = 0; v < VEC; ++v) C[v] = cut ? 0.0f : times_a(c[i][v], d[i][v] + C[v]);
        }
    }
}

// The tiles' sums of g and end states (and, for the gradients, what leaves
// each backwards).
template <int E, int G, int VEC, bool BWD>
__global__ __launch_bounds__(512) void scan_tiles_kernel(ScanParams p)
{
    constexpr int NW = SCAN_TILE / R, F = BWD ? 3 : 2;
    __shared__ float tri[NW][F][64 * VEC];
    const Place<VEC> at(p);
    const Packed b = packed(p);
    const int tokens = b.tokens(), lane = at.lane, wave = at.wave;
    const int lo = at.range * SCAN_TILE, hi = lo + SCAN_TILE < tokens ? lo + SCAN_TILE : tokens;
    float sum[VEC] = {}, H[VEC] = {}, C[VEC] = {};
    if (lo < hi) {
        Rows<E, G, VEC> rows;
        OutRows<E, VEC> outs;
        rows.load(p, lo + wave * R, hi, at.col);
        if constexpr (BWD) outs.load(p, lo + wave * R, hi, at.col);
        Cursor cur(b);
        Slice<R> s;
        s.set(cur, lo + wave * R, hi, tokens);
        float c[R][VEC], u[R][VEC], d[R][VEC];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float g[VEC], w[VEC], x[VEC];
            rows.at(p, i, g, c[i], w, x);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                u[i][v] = factor(p.scale, c[i][v]) * (w[v] * x[v]);
                if (i < s.cnt) sum[v] += g[v];
            }
            if constexpr (BWD) outs.at(p, i, s, at.col, d[i]);
        }
        summarise<VEC, BWD>(p, s, at.col, c, u, d, H, C);
        if (s.starts) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) sum[v] = CUT_SUM;
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        tri[wave][0][lane * VEC + v] = sum[v];
        tri[wave][1][lane * VEC + v] = H[v];
        if constexpr (BWD) tri[wave][2][lane * VEC + v] = C[v];
    }
    __syncthreads();
    if (wave != 0 || !at.on) return;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        float g = 0.0f, h = 0.0f, c = 0.0f, cw[NW];
        bool cut = false;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float gw = tri[w][0][lane * VEC + v], hw = tri[w][1][lane * VEC + v];
            const bool start = gw == CUT_SUM;
            cw[w] = start ? CUT : decay(gw);
            h = start ? hw : advance(cw[w], h, hw);
            g += gw;
            cut |= start;
        }
        if constexpr (BWD) {
#pragma unroll
            for (int w = NW - 1; w >= 0; --w) {
                const float e = tri[w][2][lane * VEC + v];
                c = cw[w] == CUT ? e : advance(cw[w], c, e);
            }
        }
        const int64_t o = (int64_t)at.range * p.D + at.c0 + v;
        p.sums[o] = cut ? CUT_SUM : g;
        p.end[o] = h;
        if constexpr (BWD) p.back[o] = c;
    }
}

// Joins the tiles of 64 channels: the state that enters each (in p.end), or,
// for blockIdx.y = 1 and from the last tile on, the gradient that reaches its
// last token from behind (in p.back). 16 waves, each a run of tiles.
__global__ __launch_bounds__(1024) void scan_join_kernel(ScanParams p)
{
    __shared__ float pair[16][64][2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t c0 = (int64_t)blockIdx.x * 64 + lane, col = c0 < p.D ? c0 : p.D - 1;
    const bool rev = blockIdx.y;
    float *val = rev ? p.back : p.end;
    const int k0 = (int)((int64_t)p.tiles * wave / 16), k1 = (int)((int64_t)p.tiles * (wave + 1) / 16);
    auto index = [&](int k) { return (int64_t)(rev ? p.tiles - 1 - k : k) * p.D + col; };
    constexpr int U = 8;
    float G = 0.0f, H = 0.0f;
    bool cut = false;
    for (int k = k0; k < k1; k += U) {
        float a[U], h[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t o = index(k + i < k1 ? k + i : k1 - 1);
            a[i] = p.sums[o];
            h[i] = val[o];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (k + i >= k1) break;
            const bool r = a[i] == CUT_SUM;
            cut |= r;
            H = r ? h[i] : advance(decay(a[i]), H, h[i]);
            G += a[i];
        }
    }
    pair[wave][lane][0] = cut ? CUT : decay(G);
    pair[wave][lane][1] = H;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < wave; ++w) {
        const float a = pair[w][lane][0], h = pair[w][lane][1];
        s = a == CUT ? h : advance(a, s, h);
    }
    for (int k = k0; k < k1; k += U) {
        float a[U], h[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t o = index(k + i < k1 ? k + i : k1 - 1);
            a[i] = p.sums[o];
            h[i] = val[o];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (k + i >= k1) break;
            if (c0 < p.D) val[index(k + i)] = s;
            s = a[i] == CUT_SUM ? h[i] : advance(decay(a[i]), s, h[i]);
        }
    }
}

// The gradients of a tile, from the state that enters it and the gradient
// that reaches it from behind.
template <int E, int G, int VEC>
__global__ __launch_bounds__(512) void scan_bwd_kernel(ScanParams p)
{
    constexpr int NW = SCAN_TILE / R;
    __shared__ float tri[NW][3][64 * VEC];
    const Place<VEC> at(p);
    const Packed b = packed(p);
    const int tokens = b.tokens(), lane = at.lane, wave = at.wave;
    if (p.dh0)
        for_empty(b, at.range, at.parts, [&](int n) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const int64_t o = (int64_t)n * p.D + at.c0 + v;
                if (at.on) p.dh0[o] = p.dht ? p.dht[o] : 0.0f;
            }
        });
    const int lo = at.range * SCAN_TILE, hi = lo + SCAN_TILE < tokens ? lo + SCAN_TILE : tokens;
    if (lo >= hi) return;
    Rows<E, G, VEC> rows;
    OutRows<E, VEC> outs;
    rows.load(p, lo + wave * R, hi, at.col);
    outs.load(p, lo + wave * R, hi, at.col);
    float h[VEC], after[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        h[v] = p.tiles > 1 ? p.end[(int64_t)at.range * p.D + at.col + v] : 0.0f;
        after[v] = p.tiles > 1 ? p.back[(int64_t)at.range * p.D + at.col + v] : 0.0f;
    }
    Cursor cur(b);
    Slice<R> s;
    s.set(cur, lo + wave * R, hi, tokens);
    float c[R][VEC], w[R][VEC], x[R][VEC], u[R][VEC], d[R][VEC], before[R][VEC], sum[VEC] = {}, H[VEC], C[VEC];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float g[VEC];
        rows.at(p, i, g, c[i], w[i], x[i]);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            u[i][v] = factor(p.scale, c[i][v]) * (w[i][v] * x[i][v]);
            if (i < s.cnt) sum[v] += g[v];
        }
        outs.at(p, i, s, at.col, d[i]);
    }
    summarise<VEC, true>(p, s, at.col, c, u, d, H, C);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        tri[wave][0][lane * VEC + v] = s.starts ? CUT : decay(sum[v]);
        tri[wave][1][lane * VEC + v] = H[v];
        tri[wave][2][lane * VEC + v] = C[v];
    }
    __syncthreads();
    // the waves before this one, then those behind it from the last on
#pragma unroll
    for (int k = 0; k < NW; ++k) {
        if (k >= wave) break;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float a = tri[k][0][lane * VEC + v], e = tri[k][1][lane * VEC + v];
            h[v] = a == CUT ? e : advance(a, h[v], e);
        }
    }
#pragma unroll
    for (int k = NW - 1; k >= 0; --k) {
        if (k <= wave) break;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float a = tri[k][0][lane * VEC + v], e = tri[k][2][lane * VEC + v];
            after[v] = a == CUT ? e : advance(a, after[v], e);
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (i >= s.cnt) continue;
        if (s.starts >> i & 1) state_in<VEC>(p, s.seq(i), at.col, h);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            before[i][v] = h[v];
            h[v] = advance(c[i][v], h[v], u[i][v]);
        }
    }
#pragma unroll
    for (int i = R - 1; i >= 0; --i) {
        if (i >= s.cnt) continue;
        // nothing reaches a sequence's last token from behind
        const bool last = s.lasts >> i & 1;
        float dx[VEC], dw[VEC], dg[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float dh = last ? d[i][v] : d[i][v] + after[v], m = factor(p.scale, c[i][v]);
            after[v] = times_a(c[i][v], dh);
            dx[v] = m * w[i][v] * dh;
            dw[v] = m * x[i][v] * dh;
            dg[v] = dh * fmaf(factor_slope(p.scale, c[i][v], m), w[i][v] * x[i][v], rate(c[i][v]) * before[i][v]);
        }
        const int64_t t = s.t0 + i;
        if (at.on) {
            st_el<E, VEC>(p.dx, t * p.sdx, at.c0, dx);
            if (p.dw) st_el<E, VEC>(p.dw, t * p.sdw, at.c0, dw);
            st_el<G, VEC>(p.dg, t * p.sdg, at.c0, dg);
            if (s.starts >> i & 1 && p.dh0) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) p.dh0[(int64_t)s.seq(i) * p.D + at.c0 + v] = after[v];
            }
        }
    }
}

// Token by token: a thread owns VEC channels of one sequence and reads their
// state before it writes it (so that it may be updated in place).
template <int E, int G, int VEC>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanParams p)
{
    const uint32_t cols = (p.D + 256 * VEC - 1) / (256 * VEC);
    const int n = blockIdx.x / cols;
    const uint32_t col = (blockIdx.x % cols * 256 + threadIdx.x) * VEC;
    if (col >= (uint32_t)p.D) return;
    const SeqRange r = seq_range(p.cu, p.cu64, p.T, n);
    float h[VEC];
    state_in<VEC>(p, n, col, h);
    for (int64_t t = r.b; t < r.e; ++t) {
        float g[VEC], x[VEC], w[VEC];
        ld_el<E, VEC>(p.x, t * p.sx, col, x);
        ld_el<G, VEC>(p.g, t * p.sg, col, g);
        if (p.w) ld_el<E, VEC>(p.w, t * p.sw, col, w);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float c = decay(g[v]);
            h[v] = advance(c, h[v], factor(p.scale, c) * (p.w ? w[v] * x[v] : x[v]));
        }
        st_el<E, VEC>(p.out, t * p.so, col, h);
    }
    if (p.ht) state_out<VEC>(p, n, col, h);
}

// f<E, G, VEC>() for the call's types.
template <class F>
hipError_t for_types(const ScanParams &p, F f)
{
    auto vec = [&](auto e, auto g) {
        if (p.vec2) f(e, g, std::integral_constant<int, 2>{});
        else f(e, g, std::integral_constant<int, 1>{});
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
int64_t column_blocks(const ScanParams &p, int per) { return (p.D + (int64_t)per * (p.vec2 ? 2 : 1) - 1) / (per * (p.vec2 ? 2 : 1)); }

hipError_t launch_tiles(const ScanParams &p, bool bwd, hipStream_t stream)
{
    const dim3 grid((unsigned)(column_blocks(p, 64) * p.tiles));
    hipError_t e = for_types(p, [&](auto io, auto g, auto vec) {
        if (bwd) hipLaunchKernelGGL((scan_tiles_kernel<io(), g(), vec(), true>), grid, dim3(512), 0, stream, p);
        else hipLaunchKernelGGL((scan_tiles_kernel<io(), g(), vec(), false>), grid, dim3(512), 0, stream, p);
    });
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(scan_join_kernel, dim3((unsigned)((p.D + 63) / 64), bwd ? 2 : 1), dim3(1024), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

int32_t scan_groups(int64_t T, int64_t N, int64_t D)
{
    const int64_t cols = (D + 63) / 64;
    if (T <= 512) return 1;
    if (N * cols >= 256) {
        const int64_t s = (2048 + cols - 1) / cols;
        return (int32_t)(s < N ? s : N);
    }
    return 0;
}

hipError_t launch_scan_fwd(const ScanParams &p, hipStream_t stream)
{
    if (!p.groups) {
        if (hipError_t e = launch_tiles(p, false, stream); e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)(column_blocks(p, 64) * (p.groups ? p.groups : p.tiles)));
    return for_types(p, [&](auto io, auto g, auto vec) {
        hipLaunchKernelGGL((scan_fwd_kernel<io(), g(), vec(), SCAN_TILE / R>), grid, dim3(SCAN_TILE / R * 64), 0, stream, p);
    });
}

hipError_t launch_scan_step(const ScanParams &p, hipStream_t stream)
{
    const dim3 grid((unsigned)(column_blocks(p, 256) * p.N));
    return for_types(p, [&](auto io, auto g, auto vec) {
        hipLaunchKernelGGL((scan_step_kernel<io(), g(), vec()>), grid, dim3(256), 0, stream, p);
    });
}

hipError_t launch_scan_bwd(const ScanParams &p, hipStream_t stream)
{
    if (p.tiles > 1) {
        if (hipError_t e = launch_tiles(p, true, stream); e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)(column_blocks(p, 64) * (p.tiles ? p.tiles : 1)));
    return for_types(p, [&](auto io, auto g, auto vec) {
        hipLaunchKernelGGL((scan_bwd_kernel<io(), g(), vec()>), grid, dim3(512), 0, stream, p);
    });
}

}  // namespace gdn2
