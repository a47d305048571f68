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
// of 8 elements (16 bytes per lane), a wave takes one token and 512 / K of its
// rows (heads of q, then of k) at a time, four such loads in flight, and holds
// what the token's rows share: its angles and the weights. Few tokens are
// split over several waves. Sums are lane exchanges in float32. Pairs (i, i +
// rot / 2) lie in two lanes rot / 16 apart and are exchanged through the
// lanes, pairs (2 i, 2 i + 1) in one. 37,517 tokens of 32 + 32 heads of 128 take
// 225 us (5.5 TB/s; with two rows in flight a tenth longer), their gradients for
// 16,384 tokens of 32 + 8 heads 107 us and 7 for the weights' (4.8 TB/s).
#include <stdint.h>

#include <type_traits>

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
__device__ __forceinline__ float row_sum(float x)  // over the LANES (8 or 16) lanes of a row
{
    auto dpp = [&](auto ctrl) {
        x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    dpp(std::integral_constant<int, 0xB1>{});   // lane ^ 1
    dpp(std::integral_constant<int, 0x4E>{});   // lane ^ 2
    dpp(std::integral_constant<int, 0x141>{});  // mirrored in 8
    if constexpr (LANES == 16) dpp(std::integral_constant<int, 0x140>{});  // mirrored in 16
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

// What a token's rows share in one lane: the angles of its 8 columns (a
// column that is not turned has cosine 1 and sine 0), with the sine's sign.
struct Turn {
    f32x8 c, s;
    int partner;  // lane that holds the pairs' other elements (halves)
    int n;        // columns of the lane that are turned (the others are left as they are, infinities too)

    // Token t's; back: by the negative angles. Positions outside the table
    // read its first or last row.
    template <bool INTER>
    __device__ __forceinline__ void set(const QkParams &p, int64_t t, int c0, bool back)
    {
        int64_t pos = p.pos64 ? static_cast<const int64_t *>(p.pos)[t] : (int64_t) static_cast<const int32_t *>(p.pos)[t];
        pos = pos < 0 ? 0 : pos >= p.P ? p.P - 1 : pos;
        const float *row = p.rope + pos * p.rot;
        const int half = p.rot / 2, lane = threadIdx.x & 63;
        partner = lane;
        n = p.rot - c0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = 1.0f;
            s[i] = 0.0f;
        }
        if (c0 >= p.rot) return;
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c0 + 2 * i < p.rot) {
                    const float x = row[half + c0 / 2 + i];
                    c[2 * i] = c[2 * i + 1] = row[c0 / 2 + i];
                    s[2 * i] = back ? x : -x;
                    s[2 * i + 1] = back ? -x : x;
                }
        } else {
            // element i < half pairs with i + half: half is a multiple of 8, so that pairs are whole lanes apart
            const bool first = c0 < half;
            const int f = first ? c0 : c0 - half;
            partner = first ? lane + half / 8 : lane - half / 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = row[half + f + i];
                c[i] = row[f + i];
                s[i] = first == back ? x : -x;
            }
        }
    }
    template <bool INTER>
    __device__ __forceinline__ f32x8 apply(f32x8 z) const
    {
        f32x8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = INTER ? z[i ^ 1] : __shfl(z[i], partner);
            o[i] = i < n ? x : 0.0f;
        }
        return z * c + o * s;
    }
};

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

constexpr int UNR = 4;  // rows per lane in flight

// Rows of one token that a wave's lanes take: row r of q's heads, then of k's
// (past the last: the last again, not stored).
template <int K>
struct Rows {
    static constexpr int LPR = K / 8, RPW = 64 / LPR;
    const QkParams &p;
    int64_t tok;
    int c0, sub, both;

    __device__ __forceinline__ Rows(const QkParams &q, int64_t t, int lane)
        : p(q), tok(t), c0(lane % LPR * 8), sub(lane / LPR), both(q.heads[0] + q.heads[1])
    {
    }
    struct At {
        bool on, second;
        int head;
    };
    __device__ __forceinline__ At at(int r0) const
    {
        const int r = r0 + sub, c = r < both ? r : both - 1;
        return At{r < both, c >= p.heads[0], c >= p.heads[0] ? c - p.heads[0] : c};
    }
    template <class P>
    __device__ __forceinline__ P *ptr(P *const (&base)[2], const int64_t (&st)[2], const int64_t (&hs)[2], At a) const
    {
        return (a.second ? base[1] + tok * st[1] + a.head * hs[1] : base[0] + tok * st[0] + a.head * hs[0]) + c0;
    }
};

template <int K, int IO, bool ROPE, bool INTER>
__global__ __launch_bounds__(256) void qk_fwd_kernel(QkParams p)
{
    using R = Rows<K>;
    const int lane = threadIdx.x & 63, c0 = lane % R::LPR * 8;
    const f32x8 w0 = weight8<IO>(p, 0, c0), w1 = weight8<IO>(p, 1, c0);
    const int step = R::RPW << p.split;
    const int64_t units = p.T << p.split;
    for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < units; u += (int64_t)gridDim.x * 4) {
        const int64_t tok = u >> p.split;
        const int part = (int)(u & ((1 << p.split) - 1));
        const R rows(p, tok, lane);
        Turn turn;
        if constexpr (ROPE) turn.set<INTER>(p, tok, c0, false);
        for (int r0 = part * R::RPW; r0 < rows.both; r0 += UNR * step) {
            typename R::At a[UNR];
            f32x8 x[UNR];
#pragma unroll
            for (int i = 0; i < UNR; ++i) {
                a[i] = rows.at(r0 + i * step);
                x[i] = ldx8<IO>(rows.ptr(p.x, p.sx, p.hsx, a[i]));
            }
#pragma unroll
            for (int i = 0; i < UNR; ++i) {
                bool held;
                const float r = norm_rate<K>(p, x[i], held);
                f32x8 z = x[i] * r * (a[i].second ? w1 : w0);
                if constexpr (ROPE) z = turn.apply<INTER>(z);
                if (a[i].on) stx8<IO>(rows.ptr(p.y, p.sy, p.hsy, a[i]), z);
            }
        }
    }
}

template <int K, int IO, bool ROPE, bool INTER, bool DW>
__global__ __launch_bounds__(256) void qk_bwd_kernel(QkParams p)
{
    using R = Rows<K>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    f32x8 dw0, dw1;
#pragma unroll
    for (int i = 0; i < 8; ++i) dw0[i] = dw1[i] = 0.0f;
    const int c0 = lane % R::LPR * 8;
    const f32x8 w0 = weight8<IO>(p, 0, c0), w1 = weight8<IO>(p, 1, c0);
    const int64_t units = p.T << p.split;
    for (int64_t u = (int64_t)blockIdx.x * 4 + wave; u < units; u += (int64_t)gridDim.x * 4) {
        const int64_t tok = u >> p.split;
        const int part = (int)(u & ((1 << p.split) - 1));
        const R rows(p, tok, lane);
        Turn turn;
        if constexpr (ROPE) turn.set<INTER>(p, tok, c0, true);
        const int step = R::RPW << p.split;
        for (int r0 = part * R::RPW; r0 < rows.both; r0 += 2 * step) {
            typename R::At a[2];
            f32x8 x[2], dz[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[i] = rows.at(r0 + i * step);
                x[i] = ldx8<IO>(rows.ptr(p.x, p.sx, p.hsx, a[i]));
                dz[i] = ldx8<IO>(rows.ptr(p.dy, p.sdy, p.hsdy, a[i]));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                bool held;
                const float r = norm_rate<K>(p, x[i], held);
                if constexpr (ROPE) dz[i] = turn.apply<INTER>(dz[i]);
                if constexpr (DW) {
                    const f32x8 d = dz[i] * x[i] * (a[i].on ? r : 0.0f);
                    if (a[i].on) {  // (a row past the last could hold infinities)
                        if (a[i].second) dw1 += d;
                        else dw0 += d;
                    }
                }
                const f32x8 m = dz[i] * (a[i].second ? w1 : w0);
                f32x8 dx = m * r;
                if (p.norm != 0) {
                    float d = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) d = fmaf(x[i][j], m[j], d);
                    d = row_sum<R::LPR>(d) * (p.norm == 2 ? 1.0f / K : 1.0f);
                    if (!held) dx -= x[i] * (r * (r * (r * d)));
                }
                if (a[i].on) stx8<IO>(rows.ptr(p.y, p.sy, p.hsy, a[i]), dx);
            }
        }
    }
    if constexpr (DW) {
        // the block's rows joined in a fixed order: part[block][which][K]
        constexpr int RPB = 4 * R::RPW;
        __shared__ float red[RPB][K];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) red[threadIdx.x / R::LPR][c0 + i] = w ? dw1[i] : dw0[i];
            __syncthreads();
            if (threadIdx.x < K) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < RPB; ++i) s += red[i][threadIdx.x];
                p.part[((int64_t)blockIdx.x * 2 + w) * K + threadIdx.x] = s;
            }
        }
    }
}

// The blocks' partial weight gradients joined, in a fixed order: one
// workgroup per 16 columns, 64 threads per column, eight loads in flight.
template <int IO>
__global__ __launch_bounds__(1024) void qk_dw_kernel(QkParams p)
{
    __shared__ float red[64][17];
    const int c = threadIdx.x & 15, part = threadIdx.x >> 4;
    const int id = blockIdx.x * 16 + c, which = id / p.K, col = id % p.K;
    float s = 0.0f;
    for (int g0 = part; g0 < p.groups; g0 += 512) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int g = g0 + 64 * i;
            x[i] = g < p.groups ? p.part[((int64_t)g * 2 + which) * p.K + col] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[i];
    }
    red[part][c] = s;
    __syncthreads();
    if (part == 0 && p.dw[which]) {
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < 64; ++i) x += red[i][c];
        if (p.w_f32[which]) static_cast<float *>(p.dw[which])[col] = x;
        else static_cast<uint16_t *>(p.dw[which])[col] = f32_io<IO>(x);
    }
}

constexpr int64_t FWD_GROUPS = 1 << 20, BWD_GROUPS = 2048;

// Waves per token, as a power of two: enough for 4096 waves, at most one per
// 512 / K rows.
int qk_split(int64_t T, int32_t heads, int32_t K)
{
    int s = 0;
    while ((T << s) < 4096 && (512 / K << s) < heads) ++s;
    return s;
}

template <int K, int IO>
void launch_fwd(const QkParams &p, dim3 grid, hipStream_t stream)
{
    if (!p.rope) hipLaunchKernelGGL((qk_fwd_kernel<K, IO, false, false>), grid, dim3(256), 0, stream, p);
    else if (p.interleaved) hipLaunchKernelGGL((qk_fwd_kernel<K, IO, true, true>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((qk_fwd_kernel<K, IO, true, false>), grid, dim3(256), 0, stream, p);
}
template <int K, int IO, bool DW>
void launch_bwd(const QkParams &p, dim3 grid, hipStream_t stream)
{
    if (!p.rope) hipLaunchKernelGGL((qk_bwd_kernel<K, IO, false, false, DW>), grid, dim3(256), 0, stream, p);
    else if (p.interleaved) hipLaunchKernelGGL((qk_bwd_kernel<K, IO, true, true, DW>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((qk_bwd_kernel<K, IO, true, false, DW>), grid, dim3(256), 0, stream, p);
}
template <int K, int IO>
void launch_bwd_dw(const QkParams &p, dim3 grid, hipStream_t stream)
{
    if (p.dw[0] || p.dw[1]) launch_bwd<K, IO, true>(p, grid, stream);
    else launch_bwd<K, IO, false>(p, grid, stream);
}

}  // namespace

int qk_bwd_groups(int64_t T, int32_t heads_q, int32_t heads_k, int32_t K)
{
    const int64_t b = ((T << qk_split(T, heads_q + heads_k, K)) + 3) / 4;
    return (int)(b < BWD_GROUPS ? b : BWD_GROUPS);
}

hipError_t launch_qk_fwd(const QkParams &p0, hipStream_t stream)
{
    QkParams p = p0;
    if (p.T == 0) return hipSuccess;
    p.split = qk_split(p.T, p.heads[0] + p.heads[1], p.K);
    const int64_t b = ((p.T << p.split) + 3) / 4;
    const dim3 grid((unsigned)(b < FWD_GROUPS ? b : FWD_GROUPS));
    if (p.K == 128) {
        if (p.io == IO_F16) launch_fwd<128, IO_F16>(p, grid, stream);
        else launch_fwd<128, IO_BF16>(p, grid, stream);
    } else {
        if (p.io == IO_F16) launch_fwd<64, IO_F16>(p, grid, stream);
        else launch_fwd<64, IO_BF16>(p, grid, stream);
    }
    return hipGetLastError();
}

hipError_t launch_qk_bwd(const QkParams &p0, hipStream_t stream)
{
    QkParams p = p0;
    if (p.groups > 0) {
        p.split = qk_split(p.T, p.heads[0] + p.heads[1], p.K);
        const dim3 grid((unsigned)p.groups);
        if (p.K == 128) {
            if (p.io == IO_F16) launch_bwd_dw<128, IO_F16>(p, grid, stream);
            else launch_bwd_dw<128, IO_BF16>(p, grid, stream);
        } else {
            if (p.io == IO_F16) launch_bwd_dw<64, IO_F16>(p, grid, stream);
            else launch_bwd_dw<64, IO_BF16>(p, grid, stream);
        }
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (!p.dw[0] && !p.dw[1]) return hipSuccess;
    const dim3 grid((unsigned)(2 * p.K / 16));
    if (p.io == IO_F16) hipLaunchKernelGGL((qk_dw_kernel<IO_F16>), grid, dim3(1024), 0, stream, p);
    else hipLaunchKernelGGL((qk_dw_kernel<IO_BF16>), grid, dim3(1024), 0, stream, p);
    return hipGetLastError();
}

}  // namespace gdn2
