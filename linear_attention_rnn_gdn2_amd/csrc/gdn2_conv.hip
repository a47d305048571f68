// The short causal convolution per channel (CDNA4, gfx950), K = 2, 3 or 4 taps:
//
//     p_t = b + sum_j W_j x_{t-(K-1)+j},   y = p or p sigmoid(p)
//
// where a sequence's first tokens see the rows of its initial state, the K - 1
// inputs before them. The final state is the last K - 1 inputs. Gradients:
//
//     dp = dy y'(p),   dx_s = sum_i W_{K-1-i} dp_{s+i} (inside the sequence),
//     dW_j = sum_t dp_t x_{t-(K-1)+j},   db = sum_t dp_t,
//
// dx of the last K - 1 rows takes the final state's gradient, and the initial
// state's rows are rows before the first: the same sum.
//
// Bound by HBM: every row is read once and written once, but for the K - 1 rows
// that a wave reads of its neighbour. A wave holds 64 (or 128) channels and
// walks along the tokens with the last K - 1 rows in registers.
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "../../include/gdn2.h"
#include "gdn2_mixer_device.h"

namespace gdn2 {
namespace {

using namespace dev;

constexpr int R = 8;  // tokens loaded at once, while the 8 before are worked on

__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + ex2(x * -1.44269504088896340736f)); }

__device__ __forceinline__ Packed packed(const ConvParams &p) { return Packed{p.cu, p.cu64, p.N, p.T}; }

// The first token of sequence n, which holds token t.
__device__ __forceinline__ int start_of(const Packed &b, int n, int t)
{
    const int s = b.cu ? b.entry(n) : 0;
    return s < t ? s : t;
}

// A lane's taps and bias.
template <int E, int K, int VEC>
struct Taps {
    float w[K][VEC], b[VEC];
    __device__ __forceinline__ Taps(const ConvParams &p, uint32_t col)
    {
        // the taps of neighbouring channels lie one after the other
        auto get = [&](auto *raw, auto wide) {
            __builtin_memcpy(raw, static_cast<decltype(raw)>(const_cast<void *>(p.weight)) + (int64_t)col * K, VEC * K * sizeof *raw);
#pragma unroll
            for (int v = 0; v < VEC; ++v)
#pragma unroll
                for (int j = 0; j < K; ++j) w[j][v] = wide(raw[v * K + j]);
        };
        if (E == E_F32 || p.w_f32) {
            float raw[VEC * K];
            get(raw, [](float x) { return x; });
        } else if constexpr (E != E_F32) {
            uint16_t raw[VEC * K];
            get(raw, [](uint16_t x) { return el_f32<E>(x); });
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) b[v] = p.bias ? ld_either<E>(p.bias, p.w_f32, col + v) : 0.0f;
    }
};

// The K - 1 inputs before a token, the oldest first, of a lane's channels.
template <int E, int K, int VEC>
struct Window {
    float x[K - 1][VEC];

    // As they are before the first token of sequence n.
    __device__ __forceinline__ void begin(const ConvParams &p, int n, uint32_t col)
    {
#pragma unroll
        for (int r = 0; r < K - 1; ++r) {
            if (p.s0) {
                ld_el<E, VEC>(p.s0, ((int64_t)n * (K - 1) + r) * p.D, col, x[r]);
            } else {
#pragma unroll
                for (int v = 0; v < VEC; ++v) x[r][v] = 0.0f;
            }
        }
    }
    // As they are before token t of sequence n, which begins at token b <= t.
    __device__ __forceinline__ void at(const ConvParams &p, int n, int b, int t, uint32_t col)
    {
#pragma unroll
        for (int r = 0; r < K - 1; ++r) {
            const int s = t - (K - 1) + r, q = s - b + K - 1;  // the token, or the row of the state where it lies before b
            if (s >= b) {
                ld_el<E, VEC>(p.x, (int64_t)s * p.sx, col, x[r]);
            } else if (p.s0) {
                ld_el<E, VEC>(p.s0, ((int64_t)n * (K - 1) + q) * p.D, col, x[r]);
            } else {
#pragma unroll
                for (int v = 0; v < VEC; ++v) x[r][v] = 0.0f;
            }
        }
    }
    __device__ __forceinline__ void push(const float (&xt)[VEC])
    {
#pragma unroll
        for (int r = 0; r < K - 1; ++r)
#pragma unroll
            for (int v = 0; v < VEC; ++v) x[r][v] = r + 1 < K - 1 ? x[r + 1][v] : xt[v];
    }
    __device__ __forceinline__ void product(const Taps<E, K, VEC> &w, const float (&xt)[VEC], float (&o)[VEC]) const
    {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float s = w.b[v];
#pragma unroll
            for (int j = 0; j < K - 1; ++j) s = fmaf(w.w[j][v], x[j][v], s);
            o[v] = fmaf(w.w[K - 1][v], xt[v], s);
        }
    }
    // Stored as sequence n's final state.
    __device__ __forceinline__ void end(const ConvParams &p, int n, uint32_t col) const
    {
#pragma unroll
        for (int r = 0; r < K - 1; ++r) st_el<E, VEC>(p.st, ((int64_t)n * (K - 1) + r) * p.D, col, x[r]);
    }
};

template <int VEC>
__device__ __forceinline__ void activate(const ConvParams &p, float (&y)[VEC])
{
    if (p.silu) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[v] *= sigmoid(y[v]);
    }
}

// Channels of a lane and the part along the tokens of a workgroup.
__device__ __forceinline__ uint32_t work_id() { return xcd_run(blockIdx.x, gridDim.x); }
template <int VEC>
struct Place : Channels<VEC> {
    uint32_t parts, part;
    int wave;
    __device__ __forceinline__ explicit Place(const ConvParams &p) : Place(p, (p.D + 64 * VEC - 1) / (64 * VEC)) {}

private:
    __device__ __forceinline__ Place(const ConvParams &p, uint32_t cols)
        : Channels<VEC>(work_id() % cols, threadIdx.x & 63, p.D), parts(gridDim.x / cols), part(work_id() / cols),
          wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6))
    {
    }
};

template <int E, int K, int VEC>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvParams p)
{
    const Place<VEC> at(p);
    const Packed b = packed(p);
    const int tokens = b.tokens();
    Window<E, K, VEC> win;
    if (p.st)
        for_empty(b, at.part, at.parts, [&](int n) {
            win.begin(p, n, at.col);
            if (at.on) win.end(p, n, at.col);
        });
    const int64_t lo64 = ((int64_t)at.part * 4 + at.wave) * p.slice_tokens;
    if (lo64 >= tokens) return;
    const int lo = (int)lo64, hi = lo64 + p.slice_tokens < tokens ? lo + p.slice_tokens : tokens;
    const Taps<E, K, VEC> taps(p, at.col);
    Cursor cur(b);
    const int n0 = cur.at(lo);
    win.at(p, n0, start_of(b, n0, lo), lo, at.col);
    Raw<E, VEC> raw[R];
    Slice<R> s;
    ld_rows<E, VEC, R>(p.x, p.sx, lo, hi, at.col, raw);
    s.set(cur, lo, hi, tokens);
    for (int t = lo; t < hi; t += R) {
        float x[R][VEC];
#pragma unroll
        for (int i = 0; i < R; ++i) widen<E, VEC>(raw[i], x[i]);
        const Slice<R> now = s;
        if (t + R < hi) {
            ld_rows<E, VEC, R>(p.x, p.sx, t + R, hi, at.col, raw);
            s.set(cur, t + R, hi, tokens);
        }
        auto token = [&](int i) {
            float y[VEC];
            win.product(taps, x[i], y);
            win.push(x[i]);
            activate<VEC>(p, y);
            if (at.on) st_el<E, VEC>(p.out, (int64_t)(t + i) * p.so, at.col, y);
        };
        if (now.cnt == R && !now.starts) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                token(i);
                if (now.lasts >> i & 1 && p.st && at.on) win.end(p, now.seq(i), at.col);
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (i >= now.cnt) break;
                if (now.starts >> i & 1) win.begin(p, now.seq(i), at.col);
                token(i);
                if (now.lasts >> i & 1 && p.st && at.on) win.end(p, now.seq(i), at.col);
            }
        }
    }
}

// Token by token: a thread owns VEC channels of one sequence and reads their
// state before it writes it (so that it may be updated in place).
template <int E, int K, int VEC>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvParams p)
{
    const uint32_t cols = (p.D + 256 * VEC - 1) / (256 * VEC);
    const int n = blockIdx.x / cols;
    const uint32_t col = (blockIdx.x % cols * 256 + threadIdx.x) * VEC;
    if (col >= (uint32_t)p.D) return;
    const SeqRange r = seq_range(p.cu, p.cu64, p.T, n);
    const Taps<E, K, VEC> taps(p, col);
    Window<E, K, VEC> win;
    win.begin(p, n, col);
    for (int64_t t = r.b; t < r.e; ++t) {
        float x[VEC], y[VEC];
        ld_el<E, VEC>(p.x, t * p.sx, col, x);
        win.product(taps, x, y);
        win.push(x);
        activate<VEC>(p, y);
        st_el<E, VEC>(p.out, t * p.so, col, y);
    }
    if (p.st) win.end(p, n, col);
}

// The gradients: a wave walks along its tokens and K - 1 more (whose dp its
// own last rows need). A row's dx is complete once the K - 1 tokens after it
// are through; until then its sum is one of the K - 1 in `sum`, the oldest
// row's first.
template <int E, int K, int VEC>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvParams p)
{
    __shared__ float red[4][K + 1][64 * VEC];
    const Place<VEC> at(p);
    const Packed b = packed(p);
    const int tokens = b.tokens();
    if (p.ds0)
        for_empty(b, at.part, at.parts, [&](int n) {
#pragma unroll
            for (int r = 0; r < K - 1; ++r) {
                float x[VEC] = {};
                const int64_t row = ((int64_t)n * (K - 1) + r) * p.D;
                if (p.dst) ld_el<E, VEC>(p.dst, row, at.col, x);
                if (at.on) st_el<E, VEC>(p.ds0, row, at.col, x);
            }
        });
    float dw[K + 1][VEC] = {};
    const int64_t lo64 = ((int64_t)at.part * 4 + at.wave) * p.slice_tokens;
    const int lo = lo64 < tokens ? (int)lo64 : tokens;
    const int hi = lo64 + p.slice_tokens < tokens ? lo + p.slice_tokens : tokens;
    if (lo < hi) {
        const Taps<E, K, VEC> taps(p, at.col);
        Cursor cur(b);
        int n = cur.at(lo), begin = start_of(b, n, lo);
        Window<E, K, VEC> win;
        win.at(p, n, begin, lo, at.col);
        float sum[K - 1][VEC] = {};
        // Row t - (K - 1) + r, with its sum: stored where this wave owns it.
        auto emit = [&](int row, const float (&x)[VEC]) {
            if (row >= begin) {
                if (row >= lo && row < hi && at.on) st_el<E, VEC>(p.dx, (int64_t)row * p.sdx, at.col, x);
            } else if (begin >= lo && begin < hi && p.ds0 && at.on) {
                st_el<E, VEC>(p.ds0, ((int64_t)n * (K - 1) + row - begin + K - 1) * p.D, at.col, x);
            }
        };
        const int stop = hi + K - 1 < tokens ? hi + K - 1 : tokens;
        Raw<E, VEC> rx[R], rd[R];
        Slice<R> s;
        ld_rows<E, VEC, R>(p.x, p.sx, lo, stop, at.col, rx);
        ld_rows<E, VEC, R>(p.dout, p.sdo, lo, stop, at.col, rd);
        s.set(cur, lo, stop, tokens);
        bool done = false;
        for (int t = lo; t < stop && !done; t += R) {
            float x[R][VEC], dp[R][VEC];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                widen<E, VEC>(rx[i], x[i]);
                widen<E, VEC>(rd[i], dp[i]);
            }
            const Slice<R> now = s;
            if (t + R < stop) {
                ld_rows<E, VEC, R>(p.x, p.sx, t + R, stop, at.col, rx);
                ld_rows<E, VEC, R>(p.dout, p.sdo, t + R, stop, at.col, rd);
                s.set(cur, t + R, stop, tokens);
            }
            // Token i: dp, its share of the weights' sums, and the row that is complete with it.
            auto token = [&](int i, bool own, float(&row)[VEC]) {
                if (p.silu) {
                    float y[VEC];
                    win.product(taps, x[i], y);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        const float sg = sigmoid(y[v]);
                        dp[i][v] *= sg * fmaf(y[v], 1.0f - sg, 1.0f);
                    }
                }
                if (own) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
#pragma unroll
                        for (int j = 0; j < K - 1; ++j) dw[j][v] = fmaf(dp[i][v], win.x[j][v], dw[j][v]);
                        dw[K - 1][v] = fmaf(dp[i][v], x[i][v], dw[K - 1][v]);
                        dw[K][v] += dp[i][v];
                    }
                }
                win.push(x[i]);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    row[v] = fmaf(taps.w[0][v], dp[i][v], sum[0][v]);
#pragma unroll
                    for (int r = 0; r < K - 1; ++r)
                        sum[r][v] = fmaf(taps.w[r + 1][v], dp[i][v], r + 1 < K - 1 ? sum[r + 1][v] : 0.0f);
                }
            };
            const int before = t - (K - 1);  // the first row that these tokens complete
            if (now.cnt == R && !now.starts && !now.lasts && before >= lo && before >= begin && t + R <= hi) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    float row[VEC];
                    token(i, true, row);
                    if (at.on) st_el<E, VEC>(p.dx, (int64_t)(before + i) * p.sdx, at.col, row);
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (i >= now.cnt) break;
                if (now.starts >> i & 1) {
                    if (t + i >= hi) {  // the rows behind belong to others
                        done = true;
                        break;
                    }
                    n = now.seq(i);
                    begin = t + i;
                    win.begin(p, n, at.col);
#pragma unroll
                    for (int r = 0; r < K - 1; ++r)
#pragma unroll
                        for (int v = 0; v < VEC; ++v) sum[r][v] = 0.0f;
                }
                float row[VEC];
                token(i, t + i < hi, row);
                emit(before + i, row);
                if (now.lasts >> i & 1) {
                    // the sequence's last K - 1 rows, with the final state's gradient
#pragma unroll
                    for (int r = 0; r < K - 1; ++r) {
                        float f[VEC] = {};
                        if (p.dst) ld_el<E, VEC>(p.dst, ((int64_t)n * (K - 1) + r) * p.D, at.col, f);
#pragma unroll
                        for (int v = 0; v < VEC; ++v) f[v] += sum[r][v];
                        emit(t + i - (K - 2) + r, f);
                    }
                }
            }
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        const int c = at.place(v);
#pragma unroll
        for (int j = 0; j <= K; ++j)
            if (c >= 0) red[at.wave][j][c] = dw[j][v];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (K + 1) * 64 * VEC; i += 256) {
        const int j = i / (64 * VEC), c = i % (64 * VEC);
        const uint32_t col = at.base + c;
        if (col < (uint32_t)p.D)
            p.part[((int64_t)at.part * (K + 1) + j) * p.D + col] = red[0][j][c] + red[1][j][c] + (red[2][j][c] + red[3][j][c]);
    }
}

// The workgroups' partial sums joined in a fixed order: 64 channels of one
// tap (or the bias) per workgroup, 16 waves.
template <int E>
__global__ __launch_bounds__(1024) void conv_dw_kernel(ConvParams p)
{
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, K = p.taps, j = blockIdx.y;
    const int64_t c0 = (int64_t)blockIdx.x * 64 + lane, col = c0 < p.D ? c0 : p.D - 1;
    float s = 0.0f;
    for (int g0 = wave; g0 < p.slices; g0 += 128) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int g = g0 + 16 * i;
            x[i] = g < p.slices ? p.part[((int64_t)g * (K + 1) + j) * p.D + col] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[i];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c0 >= p.D) return;
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x += red[i][lane];
    if (j < K) {
        if (p.dweight) st_either<E>(p.dweight, p.w_f32, c0 * K + j, x);
    } else if (p.dbias) {
        st_either<E>(p.dbias, p.w_f32, c0, x);
    }
}

// f<E, K, VEC>() for the call's types and taps.
template <class F>
hipError_t for_types(const ConvParams &p, F f)
{
    auto vec = [&](auto e, auto k) {
        if (p.vec2) f(e, k, std::integral_constant<int, 2>{});
        else f(e, k, std::integral_constant<int, 1>{});
    };
    auto taps = [&](auto e) {
        if (p.taps == 2) vec(e, std::integral_constant<int, 2>{});
        else if (p.taps == 3) vec(e, std::integral_constant<int, 3>{});
        else vec(e, std::integral_constant<int, 4>{});
    };
    if (p.io == E_F32) taps(std::integral_constant<int, E_F32>{});
    else if (p.io == E_F16) taps(std::integral_constant<int, E_F16>{});
    else taps(std::integral_constant<int, E_BF16>{});
    return hipGetLastError();
}
int64_t column_blocks(const ConvParams &p, int per) { return (p.D + (int64_t)per * (p.vec2 ? 2 : 1) - 1) / (per * (p.vec2 ? 2 : 1)); }

}  // namespace

// (Long slices read few rows twice, short ones fill the GPU with little work:
// forward 36,962 tokens of 8192 channels in slices of 32 269 us, of 64 252, of
// 128 261.)
int32_t conv_slice_tokens(int64_t T, int64_t D, bool bwd)
{
    int32_t l = bwd ? 256 : 64;
    while (l > (bwd ? 16 : 8) && T * ((D + 63) / 64) < (int64_t)l * 4096) l /= 2;
    return l;
}

int32_t conv_slices(int64_t T, int64_t D, bool bwd)
{
    const int64_t l = 4 * (int64_t)conv_slice_tokens(T, D, bwd);
    return (int32_t)((T + l - 1) / l);
}

hipError_t launch_conv_fwd(const ConvParams &p, hipStream_t stream)
{
    const dim3 grid((unsigned)(column_blocks(p, 64) * (p.slices ? p.slices : 1)));
    return for_types(p, [&](auto e, auto k, auto vec) {
        hipLaunchKernelGGL((conv_fwd_kernel<e(), k(), vec()>), grid, dim3(256), 0, stream, p);
    });
}

hipError_t launch_conv_step(const ConvParams &p, hipStream_t stream)
{
    const dim3 grid((unsigned)(column_blocks(p, 256) * p.N));
    return for_types(p, [&](auto e, auto k, auto vec) {
        hipLaunchKernelGGL((conv_step_kernel<e(), k(), vec()>), grid, dim3(256), 0, stream, p);
    });
}

hipError_t launch_conv_bwd(const ConvParams &p, hipStream_t stream)
{
    const dim3 grid((unsigned)(column_blocks(p, 64) * (p.slices ? p.slices : 1)));
    hipError_t e = for_types(p, [&](auto e, auto k, auto vec) {
        hipLaunchKernelGGL((conv_bwd_kernel<e(), k(), vec()>), grid, dim3(256), 0, stream, p);
    });
    if (e != hipSuccess || !(p.dweight || p.dbias)) return e;
    const dim3 dw((unsigned)((p.D + 63) / 64), p.taps + 1);
    if (p.io == E_F32) hipLaunchKernelGGL((conv_dw_kernel<E_F32>), dw, dim3(1024), 0, stream, p);
    else if (p.io == E_F16) hipLaunchKernelGGL((conv_dw_kernel<E_F16>), dw, dim3(1024), 0, stream, p);
    else hipLaunchKernelGGL((conv_dw_kernel<E_BF16>), dw, dim3(1024), 0, stream, p);
    return hipGetLastError();
}

}  // namespace gdn2
