// Per-head norms of q and k with the position rotation in the same pass, and
// their gradients (CDNA4, gfx950). Per row x of K elements:
//
//     z = x r w;   y = z, its first `rot` elements turned in pairs (a, b) by
//     the position's angle: (a c - b s, a s + b c)
//
// with r = 1 / max(|x|, eps), 1 / sqrt(mean x^2 + eps) or 1. The gradients,
// with dz = dy turned back, m = w dz:
//
//     dx = r m - x r^3 <x, m> / n   (n = 1, or K for the mean; no second term
//     where eps holds the norm),    dw = sum over all rows of dz x r
//
// Bound by HBM: every row is read once and written once. A row is K / 8 lanes
// of 8 elements (16 bytes per lane), so that a wave covers 64 * 8 / K rows and
// its loads are contiguous over heads; sums are float32 lane exchanges. Pairs
// (i, i + rot / 2) lie in two lanes rot / 16 apart and are exchanged through
// the lanes, pairs (2 i, 2 i + 1) in one.
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "gdn2_delta_device.h"

namespace gdn2 {
namespace {

using namespace dev;

template <int IO>
__device__ __forceinline__ f32x8 ldx8(const uint16_t *p)
{
    if constexpr (IO == IO_F16) return __builtin_convertvector(*reinterpret_cast<const f16x8 *>(p), f32x8);
    else return __builtin_convertvector(*reinterpret_cast<const bf16x8 *>(p), f32x8);
}
template <int IO>
__device__ __forceinline__ void stx8(uint16_t *p, f32x8 x)
{
    if constexpr (IO == IO_F16) *reinterpret_cast<f16x8 *>(p) = __builtin_convertvector(x, f16x8);
    else *reinterpret_cast<bf16x8 *>(p) = f32x8_to_bf16(x);
}

template <int LANES>
__device__ __forceinline__ float row_sum(float x)  // over LANES neighbouring lanes
{
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) x += __shfl_xor(x, d);
    return x;
}

template <int IO>
__device__ __forceinline__ f32x8 weight8(const QkParams &p, int which, int c0)
{
    f32x8 w;
    if (!p.w[which]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    } else if (p.w_f32[which]) {
        const f32x4 *a = reinterpret_cast<const f32x4 *>(static_cast<const float *>(p.w[which]) + c0);
        w = __builtin_shufflevector(a[0], a[1], 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        w = ldx8<IO>(static_cast<const uint16_t *>(p.w[which]) + c0);
    }
    return w;
}

// The table row of token t: positions outside the table read its first or last row.
__device__ __forceinline__ const float *rope_row(const QkParams &p, int64_t t)
{
    int64_t pos = p.pos64 ? static_cast<const int64_t *>(p.pos)[t] : (int64_t) static_cast<const int32_t *>(p.pos)[t];
    pos = pos < 0 ? 0 : pos >= p.P ? p.P - 1 : pos;
    return p.rope + pos * p.rot;
}

// z (8 elements from column c0 of a row) turned by the row's angles; back: by the negative angles.
__device__ __forceinline__ f32x8 turn(const QkParams &p, const float *row, f32x8 z, int c0, bool back)
{
    const int half = p.rot / 2;
    if (p.interleaved) {
        if (c0 < p.rot) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (c0 + 2 * i < p.rot) {
                    const float c = row[c0 / 2 + i], s0 = row[half + c0 / 2 + i], s = back ? -s0 : s0;
                    const float a = z[2 * i], b = z[2 * i + 1];
                    z[2 * i] = a * c - b * s;
                    z[2 * i + 1] = a * s + b * c;
                }
            }
        }
        return z;
    }
    // element i < half pairs with i + half: half is a multiple of 8, so that pairs are whole lanes apart
    const int d = half / 8, l = c0 / 8;
    const int lane = threadIdx.x & 63;
    const int partner = l < d ? lane + d : l < 2 * d ? lane - d : lane;
    f32x8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __shfl(z[i], partner);
    if (c0 < p.rot) {
        const int f = c0 < half ? c0 : c0 - half;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = row[f + i], s0 = row[half + f + i], s = (c0 < half) == back ? s0 : -s0;
            z[i] = z[i] * c + o[i] * s;
        }
    }
    return z;
}

template <int K>
__device__ __forceinline__ float norm_rate(const QkParams &p, f32x8 x, bool &held)
{
    held = false;
    if (p.norm == 0) return 1.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
    s = row_sum<K / 8>(s);
    if (p.norm == 2) return 1.0f / sqrtf(s * (1.0f / K) + p.eps);
    const float nrm = sqrtf(s);
    held = !(nrm > p.eps);
    return 1.0f / (held ? p.eps : nrm);
}

// Row `id` of the call: token-major over the heads of q, then of k.
__device__ __forceinline__ void row_of(const QkParams &p, int64_t id, int &which, int64_t &tok, int &head)
{
    const int both = p.heads[0] + p.heads[1];
    tok = id / both;
    head = (int)(id - tok * both);
    which = head >= p.heads[0];
    if (which) head -= p.heads[0];
}

template <int K, int IO>
__global__ __launch_bounds__(256) void qk_fwd_kernel(QkParams p)
{
    constexpr int LPR = K / 8, RPB = 256 / LPR;
    const int64_t rows = p.T * (p.heads[0] + p.heads[1]);
    const int c0 = (threadIdx.x % LPR) * 8;
    for (int64_t id0 = (int64_t)blockIdx.x * RPB; id0 < rows; id0 += (int64_t)gridDim.x * RPB) {
        int64_t id = id0 + threadIdx.x / LPR;
        const bool on = id < rows;
        if (!on) id = rows - 1;
        int which, head;
        int64_t tok;
        row_of(p, id, which, tok, head);
        const f32x8 x = ldx8<IO>(p.x[which] + tok * p.sx[which] + head * p.hsx[which] + c0);
        bool held;
        const float r = norm_rate<K>(p, x, held);
        f32x8 z = x * r * weight8<IO>(p, which, c0);
        if (p.rope) z = turn(p, rope_row(p, tok), z, c0, false);
        if (on) stx8<IO>(p.y[which] + tok * p.sy[which] + head * p.hsy[which] + c0, z);
    }
}

template <int K, int IO, bool DW>
__global__ __launch_bounds__(256) void qk_bwd_kernel(QkParams p)
{
    constexpr int LPR = K / 8, RPB = 256 / LPR;
    const int64_t rows = p.T * (p.heads[0] + p.heads[1]);
    const int c0 = (threadIdx.x % LPR) * 8;
    f32x8 dw[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.0f;
    for (int64_t id0 = (int64_t)blockIdx.x * RPB; id0 < rows; id0 += (int64_t)gridDim.x * RPB) {
        int64_t id = id0 + threadIdx.x / LPR;
        const bool on = id < rows;
        if (!on) id = rows - 1;
        int which, head;
        int64_t tok;
        row_of(p, id, which, tok, head);
        const f32x8 x = ldx8<IO>(p.x[which] + tok * p.sx[which] + head * p.hsx[which] + c0);
        f32x8 dz = ldx8<IO>(p.dy[which] + tok * p.sdy[which] + head * p.hsdy[which] + c0);
        bool held;
        const float r = norm_rate<K>(p, x, held);
        if (p.rope) dz = turn(p, rope_row(p, tok), dz, c0, true);
        if constexpr (DW) {
            if (on) dw[which] += dz * x * r;
        }
        const f32x8 m = dz * weight8<IO>(p, which, c0);
        f32x8 dx = m * r;
        if (p.norm != 0) {
            float d = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) d = fmaf(x[i], m[i], d);
            d = row_sum<LPR>(d) * (p.norm == 2 ? 1.0f / K : 1.0f);
            if (!held) dx -= x * (r * (r * (r * d)));
        }
        if (on) stx8<IO>(p.y[which] + tok * p.sy[which] + head * p.hsy[which] + c0, dx);
    }
    if constexpr (DW) {
        // the block's rows joined in a fixed order: part[block][which][K]
        __shared__ float red[RPB][K];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) red[threadIdx.x / LPR][c0 + i] = dw[w][i];
            __syncthreads();
            if (threadIdx.x < K) {
                float s = 0.0f;
                for (int i = 0; i < RPB; ++i) s += red[i][threadIdx.x];
                p.part[((int64_t)blockIdx.x * 2 + w) * K + threadIdx.x] = s;
            }
        }
    }
}

// The blocks' partial weight gradients joined, in a fixed order: one
// workgroup per 16 columns, 16 threads per column.
template <int IO>
__global__ __launch_bounds__(256) void qk_dw_kernel(QkParams p)
{
    __shared__ float red[16][17];
    const int c = threadIdx.x & 15, part = threadIdx.x >> 4;
    const int id = blockIdx.x * 16 + c, which = id / p.K, col = id % p.K;
    float s = 0.0f;
    for (int g = part; g < p.groups; g += 16) s += p.part[((int64_t)g * 2 + which) * p.K + col];
    red[part][c] = s;
    __syncthreads();
    if (part == 0 && p.dw[which]) {
        float x = 0.0f;
        for (int i = 0; i < 16; ++i) x += red[i][c];
        if (p.w_f32[which]) static_cast<float *>(p.dw[which])[col] = x;
        else static_cast<uint16_t *>(p.dw[which])[col] = f32_io<IO>(x);
    }
}

int64_t qk_blocks(int64_t T, int32_t hq, int32_t hk, int32_t K)
{
    const int64_t rpb = 256 / (K / 8);
    return (T * ((int64_t)hq + hk) + rpb - 1) / rpb;
}

}  // namespace

int qk_bwd_groups(int64_t T, int32_t heads_q, int32_t heads_k, int32_t K)
{
    const int64_t b = qk_blocks(T, heads_q, heads_k, K);
    return (int)(b < 2048 ? b : 2048);
}

hipError_t launch_qk_fwd(const QkParams &p, hipStream_t stream)
{
    const int64_t b = qk_blocks(p.T, p.heads[0], p.heads[1], p.K);
    if (b == 0) return hipSuccess;
    const dim3 grid((unsigned)(b < 16384 ? b : 16384));
    if (p.K == 128) {
        if (p.io == IO_F16) hipLaunchKernelGGL((qk_fwd_kernel<128, IO_F16>), grid, dim3(256), 0, stream, p);
        else hipLaunchKernelGGL((qk_fwd_kernel<128, IO_BF16>), grid, dim3(256), 0, stream, p);
    } else {
        if (p.io == IO_F16) hipLaunchKernelGGL((qk_fwd_kernel<64, IO_F16>), grid, dim3(256), 0, stream, p);
        else hipLaunchKernelGGL((qk_fwd_kernel<64, IO_BF16>), grid, dim3(256), 0, stream, p);
    }
    return hipGetLastError();
}

template <int K, int IO>
static void launch_qk_bwd_dw(const QkParams &p, dim3 grid, hipStream_t stream)
{
    if (p.dw[0] || p.dw[1]) hipLaunchKernelGGL((qk_bwd_kernel<K, IO, true>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((qk_bwd_kernel<K, IO, false>), grid, dim3(256), 0, stream, p);
}

hipError_t launch_qk_bwd(const QkParams &p, hipStream_t stream)
{
    if (p.groups > 0) {
        const dim3 grid((unsigned)p.groups);
        if (p.K == 128) {
            if (p.io == IO_F16) launch_qk_bwd_dw<128, IO_F16>(p, grid, stream);
            else launch_qk_bwd_dw<128, IO_BF16>(p, grid, stream);
        } else {
            if (p.io == IO_F16) launch_qk_bwd_dw<64, IO_F16>(p, grid, stream);
            else launch_qk_bwd_dw<64, IO_BF16>(p, grid, stream);
        }
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (!p.dw[0] && !p.dw[1]) return hipSuccess;
    const dim3 grid((unsigned)(2 * p.K / 16));
    if (p.io == IO_F16) hipLaunchKernelGGL((qk_dw_kernel<IO_F16>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((qk_dw_kernel<IO_BF16>), grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace gdn2
