// The gated linear recurrence forward: groups of whole sequences, two passes
// over few long ones, and token by token (see gdn2_scan_device.h).
#include "gdn2_scan_device.h"

namespace gdn2 {
namespace {

using namespace scan;

// The forward over a group of whole sequences: the waves take 8 tokens each in
// turn, loading the next 8 while they join these.
template <int E, int G, int KIND>
__global__ __launch_bounds__(512) void scan_groups_kernel(ScanParams p)
{
    constexpr int NW = 8, VEC = 1;
    __shared__ float trio[2][NW][3][64 * VEC];
    const Place<VEC> at(p, true);
    const Packed b = packed(p);
    const int tokens = b.tokens(), lane = at.lane, wave = at.wave;
    if (p.ht)
        for_empty(b, at.range, at.parts, [&](int n) {
            float h[VEC];
            state_in<VEC>(p, n, at.col, h);
            if (at.on) state_out<VEC>(p, n, at.col, h);
        });
    int lo, hi;
    float h[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = 0.0f;
    if (p.groups > 1 && p.groups == p.N && p.N <= 64) {
        b.by_length(at.range, lo, hi);
    } else {
        lo = b.start_from((int)((int64_t)p.T * at.range / p.groups));
        hi = (int)at.range + 1 < p.groups ? b.start_from((int)((int64_t)p.T * (at.range + 1) / p.groups)) : tokens;
    }
    if (lo >= hi) return;
    Cursor cur(b);
    Slice<R> s, next;
    Rows<E, G, VEC> rows;
    rows.load(p, lo + wave * R, hi, at.col);
    next.set(cur, lo + wave * R, hi, tokens);
    int buf = 0;
    for (int t = lo; t < hi; t += NW * R, buf ^= 1) {
        s = next;
        Decay a[R][VEC];
        float u[R][VEC], sum[VEC], H[VEC] = {}, enter[VEC];
        rows.template inputs<KIND>(p, s.cnt, a, u, sum);
        const int tn = t + NW * R;
        if (tn < hi) {
            rows.load(p, tn + wave * R, hi, at.col);
            next.set(cur, tn + wave * R, hi, tokens);
        }
        const bool plain = s.cnt == R && !s.starts;
        auto none = [](int, float (&)[VEC]) {};
        if (plain) walk<VEC, true>(p, s, at.col, a, u, H, none);
        else walk<VEC, false>(p, s, at.col, a, u, H, none);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const Decay d = decay(sum[v]);
            trio[buf][wave][0][lane * VEC + v] = s.starts ? CUT : d.hi;
            trio[buf][wave][1][lane * VEC + v] = d.lo;
            trio[buf][wave][2][lane * VEC + v] = H[v];
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float e[3] = {trio[buf][w][0][lane * VEC + v], trio[buf][w][1][lane * VEC + v], trio[buf][w][2][lane * VEC + v]};
                if (w == wave) enter[v] = h[v];
                h[v] = join(e, h[v]);
            }
        auto store = [&](int i, float (&o)[VEC]) {
            if (at.on) st_el<E, VEC>(p.out, (int64_t)(s.t0 + i) * p.so, at.col, o);
        };
        if (plain) {
            walk<VEC, true>(p, s, at.col, a, u, enter, store);
            if (s.lasts >> (R - 1) && p.ht && at.on) state_out<VEC>(p, s.seq(R - 1), at.col, enter);
        } else {
            walk<VEC, false>(p, s, at.col, a, u, enter, [&](int i, float (&o)[VEC]) {
                store(i, o);
                if (s.lasts >> i & 1 && p.ht && at.on) state_out<VEC>(p, s.seq(i), at.col, o);
            });
        }
    }
}

// The forward over few long sequences, in two passes. A wave takes p.chunk
// consecutive tokens, a workgroup eight such chunks (a range). The first pass
// leaves the sum of g and the end state from zero of every chunk and every
// range, the second walks each chunk from its entering state. f(s, a, u) sees
// 8 tokens. With 16-bit x and g two workgroups share a compute unit (124 and
// 112 registers); 65,536 tokens of 1024 channels: the first pass 81 us, 3.3 TB/s
// of reads beside 25 vector instructions per element that hold the vector units
// for 54 % of that time, the second 77 us, 5.3 TB/s. float32 takes 151 and 134
// to 136 registers and one workgroup (303 us in all for 170 of bytes).
template <int E, int G, int VEC, int KIND, class F>
__device__ __forceinline__ void walk_chunk(const ScanParams &p, const Packed &b, int lo, int hi, int tokens, uint32_t col, F f)
{
    if (lo >= hi) return;
    Cursor cur(b);
    Slice<R> s, next;
    Rows<E, G, VEC> rows;
    rows.load(p, lo, hi, col);
    next.set(cur, lo, hi, tokens);
    for (int t = lo; t < hi; t += R) {
        s = next;
        Decay a[R][VEC];
        float u[R][VEC], sum[VEC];
        rows.template inputs<KIND>(p, s.cnt, a, u, sum);
        if (t + R < hi) {
            rows.load(p, t + R, hi, col);
            next.set(cur, t + R, hi, tokens);
        }
        f(s, a, u, sum);
    }
}

template <int E, int G, int VEC, int KIND>
__global__ __launch_bounds__(512) void scan_sums_kernel(ScanParams p)
{
    __shared__ float duo[8][2][64 * VEC];
    const Place<VEC> at(p);
    const Packed b = packed(p);
    const int tokens = b.tokens(), lane = at.lane, wave = at.wave;
    const int64_t chunk = (int64_t)at.range * 8 + wave, lo64 = chunk * p.chunk;
    const int lo = lo64 < tokens ? (int)lo64 : tokens, hi = lo64 + p.chunk < tokens ? lo + p.chunk : tokens;
    float sum[VEC] = {}, H[VEC] = {};
    bool cut = false;
    walk_chunk<E, G, VEC, KIND>(p, b, lo, hi, tokens, at.col,
                                [&](const Slice<R> &s, const Decay(&a)[R][VEC], const float(&u)[R][VEC], const float(&g)[VEC]) {
                                    auto none = [](int, float(&)[VEC]) {};
                                    if (s.cnt == R && !s.starts) walk<VEC, true>(p, s, at.col, a, u, H, none);
                                    else walk<VEC, false>(p, s, at.col, a, u, H, none);
                                    cut |= s.starts != 0;
#pragma unroll
                                    for (int v = 0; v < VEC; ++v) sum[v] += g[v];
                                });
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        const float g = cut ? CUT : sum[v];
        duo[wave][0][lane * VEC + v] = g;
        duo[wave][1][lane * VEC + v] = H[v];
        if (at.on) {
            p.chunk_sums[chunk * p.D + at.col + v] = g;
            p.chunk_end[chunk * p.D + at.col + v] = H[v];
        }
    }
    __syncthreads();
    if (wave != 0 || !at.on) return;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        float g = 0.0f, h = 0.0f;
        bool any = false;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const float gw = duo[w][0][lane * VEC + v], hw = duo[w][1][lane * VEC + v];
            h = gw == CUT ? hw : advance(decay(gw), h, hw);
            any |= gw == CUT;
            g += gw;
        }
        const int64_t o = (int64_t)at.range * p.D + at.col + v;
        p.sums[o] = any ? CUT : g;
        p.end[o] = h;
    }
}

template <int E, int G, int VEC, int KIND>
__global__ __launch_bounds__(512) void scan_chunks_kernel(ScanParams p)
{
    const Place<VEC> at(p);
    const Packed b = packed(p);
    const int tokens = b.tokens(), wave = at.wave;
    if (p.ht)
        for_empty(b, at.range, at.parts, [&](int n) {
            float h[VEC];
            state_in<VEC>(p, n, at.col, h);
            if (at.on) state_out<VEC>(p, n, at.col, h);
        });
    const uint32_t range = at.parts - 1 - at.range;  // (from the end: the first pass read that last)
    const int64_t first = (int64_t)range * 8, lo64 = (first + wave) * p.chunk;
    if (lo64 >= tokens) return;
    const int lo = (int)lo64, hi = lo64 + p.chunk < tokens ? lo + p.chunk : tokens;
    float h[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        const int64_t c = at.col + v;
        h[v] = p.end[range * (int64_t)p.D + c];
        float g[7], e[7];
#pragma unroll
        for (int w = 0; w < 7; ++w) {  // the range's chunks before this one (the others' own again, unused)
            const int64_t o = (first + (w < wave ? w : wave)) * p.D + c;
            g[w] = p.chunk_sums[o];
            e[w] = p.chunk_end[o];
        }
#pragma unroll
        for (int w = 0; w < 7; ++w) {
            const float x = g[w] == CUT ? e[w] : advance(decay(g[w]), h[v], e[w]);
            h[v] = w < wave ? x : h[v];
        }
    }
    walk_chunk<E, G, VEC, KIND>(p, b, lo, hi, tokens, at.col,
                                [&](const Slice<R> &s, const Decay(&a)[R][VEC], const float(&u)[R][VEC], const float(&)[VEC]) {
                                    auto store = [&](int i, float(&o)[VEC]) {
                                        if (at.on) st_el<E, VEC>(p.out, (int64_t)(s.t0 + i) * p.so, at.col, o);
                                    };
                                    if (s.cnt == R && !s.starts) {
                                        walk<VEC, true>(p, s, at.col, a, u, h, store);
                                        if (s.lasts >> (R - 1) && p.ht && at.on) state_out<VEC>(p, s.seq(R - 1), at.col, h);
                                    } else {
                                        walk<VEC, false>(p, s, at.col, a, u, h, [&](int i, float(&o)[VEC]) {
                                            store(i, o);
                                            if (s.lasts >> i & 1 && p.ht && at.on) state_out<VEC>(p, s.seq(i), at.col, o);
                                        });
                                    }
                                });
}

// Token by token: a thread owns VEC channels of one sequence and reads their
// state before it writes it (so that it may be updated in place).
template <int E, int G, int VEC, int KIND>
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
            const Decay a = decay(g[v]);
            h[v] = advance(a, h[v], factor<KIND>(a) * (p.w ? w[v] * x[v] : x[v]));
        }
        st_el<E, VEC>(p.out, t * p.so, col, h);
    }
    if (p.ht) state_out<VEC>(p, n, col, h);
}

}  // namespace

// Tokens per wave: about 8192 waves of 64 channels (65,536 tokens of 1024
// channels in 128: 163 us, in 64 164, in 32 174; 8192 tokens 43, 53, 53).
int32_t scan_chunk(int64_t T, int64_t D)
{
    const int64_t c = T * ((D + 63) / 64) / 8192 / R * R;
    return (int32_t)(c < R ? R : c > 256 ? 256 : c);
}

// Whole sequences take 2.2 us per 64 tokens of the longest, all side by side,
// or the time of their bytes; two passes read x, w and g twice and take a
// launch or two more. Measured, two passes / whole in us: one sequence of 8192
// tokens, 4096 channels 124 / 284, two 240 / 287, three 372 / 292, four 484 /
// 297; 8 and 12 of 1024 channels 270 / 290 and 387 / 294; one of 256 and of
// 1024 tokens 22 / 14 and 22 / 39; five of 700, 2048 channels 53 / 32; 300 of
// 20 to 200 310 / 178. The lengths are not known here, and taken as equal: one
// sequence of 30,000 tokens among seven of 500 takes 1023, in two passes 607.
// Groups: each sequence its own where there are few, the longest first; else
// as many as make 1024 workgroups, four for each of 256 compute units, of 64
// tokens and more (1000 sequences of 20 tokens, 1024 channels: 32 groups 65,
// 128 83).
int32_t scan_groups(int64_t T, int64_t N, int64_t D)
{
    const double bytes = (double)T * (double)D, walk = 0.035 * (double)T / (double)N, move = bytes * 10 / 4.6e6;
    if (8 + (walk > move ? walk : move) > 18 + bytes * 18 / 4.9e6) return 0;
    if (N <= 64 && T / N >= 64) return (int32_t)N;
    const int64_t cols = (D + 63) / 64, fill = (1024 + cols - 1) / cols, most = T / 64 < N ? T / 64 : N;
    const int64_t s = fill < most ? fill : most;
    return (int32_t)(s < 1 ? 1 : s);
}

hipError_t launch_scan_fwd(const ScanParams &p, hipStream_t stream)
{
    if (p.groups) {
        const dim3 grid((unsigned)(column_blocks(p, 64) * p.groups));
        return for_types(p, false, [&](auto io, auto g, auto vec, auto kind) {
            if constexpr (vec() == 1) hipLaunchKernelGGL((scan_groups_kernel<io(), g(), kind()>), grid, dim3(512), 0, stream, p);
        });
    }
    const dim3 grid((unsigned)(column_blocks(p, p.vec2 ? 128 : 64) * p.tiles));
    hipError_t e = for_types(p, p.vec2, [&](auto io, auto g, auto vec, auto kind) {
        hipLaunchKernelGGL((scan_sums_kernel<io(), g(), vec(), kind()>), grid, dim3(512), 0, stream, p);
    });
    if (e == hipSuccess) e = launch_scan_join(p, false, stream);
    if (e != hipSuccess) return e;
    return for_types(p, p.vec2, [&](auto io, auto g, auto vec, auto kind) {
        hipLaunchKernelGGL((scan_chunks_kernel<io(), g(), vec(), kind()>), grid, dim3(512), 0, stream, p);
    });
}

hipError_t launch_scan_step(const ScanParams &p, hipStream_t stream)
{
    const dim3 grid((unsigned)(column_blocks(p, p.vec2 ? 512 : 256) * p.N));
    return for_types(p, p.vec2, [&](auto io, auto g, auto vec, auto kind) {
        hipLaunchKernelGGL((scan_step_kernel<io(), g(), vec(), kind()>), grid, dim3(256), 0, stream, p);
    });
}

}  // namespace gdn2
