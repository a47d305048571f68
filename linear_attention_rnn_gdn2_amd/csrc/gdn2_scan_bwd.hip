// The gated linear recurrence's gradients, and the join of tiles that both
// directions use (see gdn2_scan_device.h).
#include "gdn2_scan_device.h"

namespace gdn2 {
namespace {

using namespace scan;

// What the gradient needs of dout: the loaded rows, and dout plus, on a
// sequence's last token, the final state's gradient.
template <int E, int VEC>
struct OutRows {
    Raw<E, VEC> d[R];
    __device__ __forceinline__ void load(const ScanParams &p, int t0, int hi, uint32_t col)
    {
        ld_rows<E, VEC, R>(p.dout, p.sdo, t0, hi, col, d);
    }
    // Token i's (widened where it is used: registers decide the workgroups per compute unit).
    template <bool PLAIN>
    __device__ __forceinline__ void wide(const ScanParams &p, const Slice<R> &s, uint32_t col, int i, float (&o)[VEC]) const
    {
        widen<E, VEC>(d[i], o);
        if (!PLAIN && p.dht && s.lasts >> i & 1) {
            const float *q = p.dht + (int64_t)s.seq(i) * p.D + col;
#pragma unroll
            for (int v = 0; v < VEC; ++v) o[v] += q[v];
        }
    }
};

// The gradient through R tokens backwards: `after` is what reaches the last
// of them from behind, and becomes what leaves the first; f(i, dh) sees the
// state's gradient at token i, g(i, c) what leaves a sequence's first token
// (for its initial state). PLAIN: the tokens all exist, and no sequence
// begins or ends among them.
template <int E, int VEC, bool PLAIN, class F, class G>
__device__ __forceinline__ void walk_back(const ScanParams &p, const Slice<R> &s, uint32_t col, const Decay (&a)[R][VEC],
                                          const OutRows<E, VEC> &outs, float (&after)[VEC], F f, G g)
{
#pragma unroll
    for (int i = R - 1; i >= 0; --i) {
        if (!PLAIN && i >= s.cnt) continue;
        float d[VEC], dh[VEC];
        outs.template wide<PLAIN>(p, s, col, i, d);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            dh[v] = !PLAIN && s.lasts >> i & 1 ? d[v] : d[v] + after[v];
            after[v] = times(a[i][v], dh[v]);
        }
        f(i, dh);
        if (!PLAIN && s.starts >> i & 1) {
            g(i, after);
#pragma unroll
            for (int v = 0; v < VEC; ++v) after[v] = 0.0f;  // nothing reaches the sequence before
        }
    }
}

// The gradients' tiles: sums of g, end states, and what leaves each backwards.
template <int E, int G, int VEC, int KIND>
__global__ __launch_bounds__(512) void scan_tiles_kernel(ScanParams p)
{
    constexpr int NW = SCAN_TILE / R;
    __shared__ float trio[NW][3][64 * VEC];
    const Place<VEC> at(p);
    const Packed b = packed(p);
    const int tokens = b.tokens(), lane = at.lane, wave = at.wave;
    const int lo = at.range * SCAN_TILE, hi = lo + SCAN_TILE < tokens ? lo + SCAN_TILE : tokens;
    float sum[VEC] = {}, H[VEC] = {}, C[VEC] = {};
    if (lo < hi) {
        Rows<E, G, VEC> rows;
        OutRows<E, VEC> outs;
        rows.load(p, lo + wave * R, hi, at.col);
        outs.load(p, lo + wave * R, hi, at.col);
        Cursor cur(b);
        Slice<R> s;
        s.set(cur, lo + wave * R, hi, tokens);
        Decay a[R][VEC];
        float u[R][VEC];
        rows.template inputs<KIND>(p, s.cnt, a, u, sum);
        auto none = [](int, float (&)[VEC]) {};
        if (s.cnt == R && !s.starts) walk<VEC, true>(p, s, at.col, a, u, H, none);
        else walk<VEC, false>(p, s, at.col, a, u, H, none);
        if (s.cnt == R && !s.starts && !s.lasts) walk_back<E, VEC, true>(p, s, at.col, a, outs, C, none, none);
        else walk_back<E, VEC, false>(p, s, at.col, a, outs, C, none, none);
        if (s.starts) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) sum[v] = CUT;
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        trio[wave][0][lane * VEC + v] = sum[v];
        trio[wave][1][lane * VEC + v] = H[v];
        trio[wave][2][lane * VEC + v] = C[v];
    }
    __syncthreads();
    if (wave != 0 || !at.on) return;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        float g = 0.0f, h = 0.0f, c = 0.0f;
        Decay a[NW];
        bool cut = false;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float gw = trio[w][0][lane * VEC + v], hw = trio[w][1][lane * VEC + v];
            a[w] = decay(gw);
            h = gw == CUT ? hw : advance(a[w], h, hw);
            cut |= gw == CUT;
            a[w].hi = gw == CUT ? CUT : a[w].hi;
            g += gw;
        }
#pragma unroll
        for (int w = NW - 1; w >= 0; --w) {
            const float e[3] = {a[w].hi, a[w].lo, trio[w][2][lane * VEC + v]};
            c = join(e, c);
        }
        const int64_t o = (int64_t)at.range * p.D + at.col + v;
        p.sums[o] = cut ? CUT : g;
        p.end[o] = h;
        p.back[o] = c;
    }
}

// Joins the tiles of COLS channels: the state that enters each (in p.end),
// or, for blockIdx.y = 1 and from the last tile on, the gradient that reaches
// its last token from behind (in p.back). 1024 / COLS runs of tiles side by
// side: what costs is the loads' latency, and with many channels their lines
// (1024 tiles of 1024 channels 12 us in 16 channels a workgroup, 23 in 64;
// 578 tiles of 4096, both directions, 30 in 16, 15 in 32, 19 in 64).
template <int COLS>
__global__ __launch_bounds__(1024) void scan_join_kernel(ScanParams p)
{
    constexpr int RUNS = 1024 / COLS;
    __shared__ float trio[RUNS][3][COLS];
    const int c = threadIdx.x % COLS, run = threadIdx.x / COLS;
    const int64_t c0 = (int64_t)blockIdx.x * COLS + c, col = c0 < p.D ? c0 : p.D - 1;
    const bool rev = blockIdx.y;
    float *val = rev ? p.back : p.end;
    const int k0 = (int)((int64_t)p.tiles * run / RUNS), k1 = (int)((int64_t)p.tiles * (run + 1) / RUNS);
    constexpr int U = 8;
    auto tiles = [&](float s, auto f) {  // f(place, sum of g, state that enters) for this run's tiles, from state s
        for (int k = k0; k < k1; k += U) {
            float g[U], h[U];
            int64_t o[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int q = k + i < k1 ? k + i : k1 - 1;
                o[i] = (int64_t)(rev ? p.tiles - 1 - q : q) * p.D + col;
                g[i] = p.sums[o[i]];
                h[i] = val[o[i]];
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (k + i >= k1) break;
                f(o[i], g[i], s);
                s = g[i] == CUT ? h[i] : advance(decay(g[i]), s, h[i]);
            }
        }
        return s;
    };
    float sum = 0.0f;
    bool cut = false;
    trio[run][2][c] = tiles(0.0f, [&](int64_t, float g, float) {
        sum += g;
        cut |= g == CUT;
    });
    const Decay d = decay(sum);
    trio[run][0][c] = cut ? CUT : d.hi;
    trio[run][1][c] = d.lo;
    __syncthreads();
    if (k0 == k1) return;
    float s = 0.0f;
    for (int w = 0; w < run; ++w) {
        const float e[3] = {trio[w][0][c], trio[w][1][c], trio[w][2][c]};
        s = join(e, s);
    }
    tiles(s, [&](int64_t o, float, float h) {
        if (c0 < p.D) val[o] = h;
    });
}

// The gradients of a tile, from the state that enters it and the gradient
// that reaches it from behind.
// Registers decide: m, x, w and dout are made again from what was loaded where
// they are needed (16-bit types: 108 to 110 registers, two workgroups per
// compute unit: 36,962 tokens of 4096 channels 514 us, 5.3 TB/s; held from the
// first walk on 162 registers, 640 us). float32 takes 130 and one workgroup
// (all three kernels of that batch 1,274 us, 1.43 times what their bytes take).
template <int E, int G, int VEC, int KIND>
__global__ __launch_bounds__(512) void scan_bwd_kernel(ScanParams p)
{
    constexpr int NW = SCAN_TILE / R;
    __shared__ float quad[NW][4][64 * VEC];  // as join() takes them, with the state's and the gradient's
    const Place<VEC> at(p);
    const Packed b = packed(p);
    const int tokens = b.tokens(), lane = at.lane, wave = at.wave;
    if (p.dh0)
        for_empty(b, at.range, at.parts, [&](int n) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const int64_t o = (int64_t)n * p.D + at.col + v;
                if (at.on) p.dh0[o] = p.dht ? p.dht[o] : 0.0f;
            }
        });
    const uint32_t tile = at.parts - 1 - at.range;  // (the last tiles' inputs were read last)
    const int lo = tile * SCAN_TILE, hi = lo + SCAN_TILE < tokens ? lo + SCAN_TILE : tokens;
    if (lo >= hi) return;
    Rows<E, G, VEC> rows;
    OutRows<E, VEC> outs;
    rows.load(p, lo + wave * R, hi, at.col);
    outs.load(p, lo + wave * R, hi, at.col);
    float h[VEC], after[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        h[v] = p.tiles > 1 ? p.end[(int64_t)tile * p.D + at.col + v] : 0.0f;
        after[v] = p.tiles > 1 ? p.back[(int64_t)tile * p.D + at.col + v] : 0.0f;
    }
    Cursor cur(b);
    Slice<R> s;
    s.set(cur, lo + wave * R, hi, tokens);
    Decay a[R][VEC];
    float u[R][VEC], before[R][VEC], sum[VEC], H[VEC] = {}, C[VEC] = {};
    rows.template inputs<KIND>(p, s.cnt, a, u, sum);
    const bool plain = s.cnt == R && !s.starts && !s.lasts;
    auto none = [](int, float (&)[VEC]) {};
    if (plain) {
        walk<VEC, true>(p, s, at.col, a, u, H, none);
        walk_back<E, VEC, true>(p, s, at.col, a, outs, C, none, none);
    } else {
        walk<VEC, false>(p, s, at.col, a, u, H, none);
        walk_back<E, VEC, false>(p, s, at.col, a, outs, C, none, none);
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        const Decay w = decay(sum[v]);
        quad[wave][0][lane * VEC + v] = s.starts ? CUT : w.hi;
        quad[wave][1][lane * VEC + v] = w.lo;
        quad[wave][2][lane * VEC + v] = H[v];
        quad[wave][3][lane * VEC + v] = C[v];
    }
    __syncthreads();
    if constexpr (sizeof(rows.x[0]) >= 4) {
        // (x and w widened again where the gradients need them)
#pragma unroll
        for (int i = 0; i < R; ++i) {
            asm("" : "+v"(rows.x[i]));
            asm("" : "+v"(rows.w[i]));
        }
    }
    // the waves before this one, then those behind it from the last on
    auto from = [&](int k, int which, float (&x)[VEC]) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const int c = lane * VEC + v;
            const float e[3] = {quad[k][0][c], quad[k][1][c], quad[k][which][c]};
            x[v] = join(e, x[v]);
        }
    };
    for (int k = 0; k < wave; ++k) from(k, 2, h);
    for (int k = NW - 1; k > wave; --k) from(k, 3, after);
    auto gradients = [&](int i, float (&dh)[VEC]) {
        float gf[VEC], w[VEC], x[VEC], dx[VEC], dw[VEC], dg[VEC];
        rows.wide(p, i, gf, w, x);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            Decay ai = a[i][v];
            asm("" : "+v"(ai.hi));  // (keeps m from being held since u was made)
            const float m = factor<KIND>(ai), mdh = m * dh[v];
            dx[v] = w[v] * mdh;
            dw[v] = x[v] * mdh;
            dg[v] = dh[v] * fmaf(factor_slope<KIND>(ai, m), w[v] * x[v], ai.hi * before[i][v]);
        }
        if (!at.on) return;
        const int64_t t = s.t0 + i;
        st_el<E, VEC>(p.dx, t * p.sdx, at.col, dx);
        if (p.dw) st_el<E, VEC>(p.dw, t * p.sdw, at.col, dw);
        st_el<G, VEC>(p.dg, t * p.sdg, at.col, dg);
    };
    auto first = [&](int i, float (&c)[VEC]) {
        if (!p.dh0 || !at.on) return;
#pragma unroll
        for (int v = 0; v < VEC; ++v) p.dh0[(int64_t)s.seq(i) * p.D + at.col + v] = c[v];
    };
    // the states before the tokens, then the gradients from the last token on
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (!plain && s.starts >> i & 1) state_in<VEC>(p, s.seq(i), at.col, h);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            before[i][v] = h[v];
            h[v] = advance(a[i][v], h[v], u[i][v]);
        }
    }
    if (plain) walk_back<E, VEC, true>(p, s, at.col, a, outs, after, gradients, first);
    else walk_back<E, VEC, false>(p, s, at.col, a, outs, after, gradients, first);
}

}  // namespace

hipError_t launch_scan_join(const ScanParams &p, bool bwd, hipStream_t stream)
{
    auto go = [&](auto cols) {
        const dim3 grid((unsigned)column_blocks(p, cols()), bwd ? 2 : 1);
        hipLaunchKernelGGL((scan_join_kernel<cols()>), grid, dim3(1024), 0, stream, p);
    };
    if (p.D <= 2048) go(std::integral_constant<int, 16>{});
    else go(std::integral_constant<int, 32>{});
    return hipGetLastError();
}

hipError_t launch_scan_bwd(const ScanParams &p, hipStream_t stream)
{
    const dim3 grid((unsigned)(column_blocks(p, p.vec2 ? 128 : 64) * (p.tiles ? p.tiles : 1)));
    if (p.tiles > 1) {
        hipError_t e = for_types(p, p.vec2, [&](auto io, auto g, auto vec, auto kind) {
            hipLaunchKernelGGL((scan_tiles_kernel<io(), g(), vec(), kind()>), grid, dim3(512), 0, stream, p);
        });
        if (e == hipSuccess) e = launch_scan_join(p, true, stream);
        if (e != hipSuccess) return e;
    }
    return for_types(p, p.vec2, [&](auto io, auto g, auto vec, auto kind) {
        hipLaunchKernelGGL((scan_bwd_kernel<io(), g(), vec(), kind()>), grid, dim3(512), 0, stream, p);
    });
}

}  // namespace gdn2
