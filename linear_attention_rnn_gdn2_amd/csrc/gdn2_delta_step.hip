// Scalar-gated delta rule token by token (CDNA4, gfx950), for decode and
// short spans:
//
//     S <- e^g S;  u = beta (v - S^T k);  S <- S + k u^T;  o = scale S^T q
//
// in float32 throughout. Every value column of S evolves on its own: a wave
// takes 32 columns of one (sequence, value head) and keeps that K x 32 block
// in registers for the whole span, so that the state is read once and written
// once. Lane 8 i + j owns rows i K / 8 .. of columns 4 j .. 4 j + 3; the two
// column sums per token join the 8 row groups by three lane exchanges, and no
// wave waits for another. Bound by HBM, the states' bytes: 128 sequences of 32
// heads (K = V = 128, 541 MB) take 100 us, 5.4 TB/s; spans of 1 to 8 tokens of
// 48 sequences 29 us, 3.6 TB/s (a token's loads in flight over the token
// before it measured slower, 31 us: the waves beside a waiting one cover it,
// and it costs registers); one sequence of 32 heads 6.0 us, all of it latency.
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "gdn2_delta_device.h"

namespace gdn2 {
namespace {

using namespace dev;

constexpr int SW_COLS = 32;  // value columns per wave

template <int IO>
__device__ __forceinline__ f32x8 ld8(const uint16_t *p)
{
    if constexpr (IO == IO_F16) return __builtin_convertvector(*reinterpret_cast<const f16x8 *>(p), f32x8);
    else return __builtin_convertvector(*reinterpret_cast<const bf16x8 *>(p), f32x8);
}

// x summed over the 8 row groups (lanes with equal lane % 8); every lane gets it.
__device__ __forceinline__ float group_sum(float x)
{
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x128, 0xf, 0xf, true));  // row_ror:8
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Four state values from element offset e (float32 or bf16).
__device__ __forceinline__ f32x4 state_ld4(const float *s, bool b16, int64_t e)
{
    if (b16) return __builtin_convertvector(*reinterpret_cast<const bf16x4 *>(reinterpret_cast<const uint16_t *>(s) + e), f32x4);
    return *reinterpret_cast<const f32x4 *>(s + e);
}
__device__ __forceinline__ void state_st4(float *s, bool b16, int64_t e, f32x4 x)
{
    if (b16) *reinterpret_cast<bf16x4 *>(reinterpret_cast<uint16_t *>(s) + e) = f32x4_to_bf16(x);
    else *reinterpret_cast<f32x4 *>(s + e) = x;
}

template <int K, int IO, bool VK, bool L2N>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaParams p, int64_t waves)
{
    constexpr int RPG = K / 8;  // rows per lane
    int64_t item = (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
    if (item >= waves) return;
    const int nvb = p.V / SW_COLS;
    const int vb = (int)(item % nvb);
    item /= nvb;
    const int hv = (int)(item % p.HV), n = (int)(item / p.HV);
    const int hk = hv / (p.HV / p.H);
    const SeqRange rng = seq_of(p, n);
    const int lane = threadIdx.x & 63, rg = lane >> 3, cg = lane & 7;
    const int r0 = rg * RPG, col = vb * SW_COLS + 4 * cg;
    const int64_t shead = ((int64_t)n * p.HV + hv) * K * p.V;

    f32x4 S[RPG];  // row r0 + i, columns col ..
    if (!p.h0) {
#pragma unroll
        for (int i = 0; i < RPG; ++i) S[i] = f32x4{0, 0, 0, 0};
    } else if constexpr (VK) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < RPG / 4; ++i) {
                const f32x4 x = state_ld4(p.h0, p.h0_bf16, shead + (int64_t)(col + j) * K + r0 + 4 * i);
#pragma unroll
                for (int e = 0; e < 4; ++e) S[4 * i + e][j] = x[e];
            }
    } else {
#pragma unroll
        for (int i = 0; i < RPG; ++i) S[i] = state_ld4(p.h0, p.h0_bf16, shead + (int64_t)(r0 + i) * p.V + col);
    }

    for (int64_t tok = rng.b; tok < rng.e; ++tok) {
        f32x8 k[RPG / 8], q[RPG / 8];
#pragma unroll
        for (int i = 0; i < RPG / 8; ++i) {
            k[i] = ld8<IO>(p.k + tok * p.sk + hk * p.hsk + r0 + 8 * i);
            q[i] = ld8<IO>(p.q + tok * p.sq + hk * p.hsq + r0 + 8 * i);
        }
        const uint16_t *vp = p.v + tok * p.sv + hv * p.hsv + col;
        f32x4 v;
        if constexpr (IO == IO_F16) v = __builtin_convertvector(*reinterpret_cast<const f16x4 *>(vp), f32x4);
        else v = __builtin_convertvector(*reinterpret_cast<const bf16x4 *>(vp), f32x4);
        float g = 0.0f;
        if (p.g) {
            const int64_t o = tok * p.sg + hv * p.hsg;
            if (p.gtype == G_F32) g = static_cast<const float *>(p.g)[o];
            else if (p.gtype == G_F16) g = io_f32<IO_F16>(static_cast<const uint16_t *>(p.g)[o]);
            else g = io_f32<IO_BF16>(static_cast<const uint16_t *>(p.g)[o]);
        }
        float bt = p.beta ? io_f32<IO>(p.beta[tok * p.sb + hv * p.hsb]) : 1.0f;
        const float decay = expf(g);
        f32x4 e = {0, 0, 0, 0};
        float nk = 0.0f, nq = 0.0f;
#pragma unroll
        for (int i = 0; i < RPG; ++i) {
            const float ki = k[i / 8][i % 8];
            S[i] *= decay;
            e += S[i] * ki;
            if constexpr (L2N) {
                nk = fmaf(ki, ki, nk);
                nq = fmaf(q[i / 8][i % 8], q[i / 8][i % 8], nq);
            }
        }
        float rk = 1.0f, rq = p.scale;
        if constexpr (L2N) {
            rk = 1.0f / fmaxf(sqrtf(group_sum(nk)), 1e-12f);
            rq = p.scale / fmaxf(sqrtf(group_sum(nq)), 1e-12f);
        }
        f32x4 u, o = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = bt * (v[j] - rk * group_sum(e[j])) * rk;  // k u^T of the unit row: k (rk u)
#pragma unroll
        for (int i = 0; i < RPG; ++i) {
            S[i] += u * k[i / 8][i % 8];
            o += S[i] * q[i / 8][i % 8];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = group_sum(o[j]) * rq;
        if (rg == 0) {
            uint16_t *op = p.out + tok * p.so + hv * p.hso + col;
            if constexpr (IO == IO_F16) *reinterpret_cast<f16x4 *>(op) = __builtin_convertvector(o, f16x4);
            else *reinterpret_cast<bf16x4 *>(op) = f32x4_to_bf16(o);
        }
    }
    if (!p.ht) return;
    if constexpr (VK) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < RPG / 4; ++i)
                state_st4(p.ht, p.ht_bf16, shead + (int64_t)(col + j) * K + r0 + 4 * i,
                          f32x4{S[4 * i][j], S[4 * i + 1][j], S[4 * i + 2][j], S[4 * i + 3][j]});
    } else {
#pragma unroll
        for (int i = 0; i < RPG; ++i) state_st4(p.ht, p.ht_bf16, shead + (int64_t)(r0 + i) * p.V + col, S[i]);
    }
}

template <int K, int IO>
void launch_step(const DeltaParams &p, dim3 grid, dim3 block, int64_t waves, hipStream_t stream)
{
    if (p.state_vmajor) {
        if (p.qk_l2norm) hipLaunchKernelGGL((delta_step_kernel<K, IO, true, true>), grid, block, 0, stream, p, waves);
        else hipLaunchKernelGGL((delta_step_kernel<K, IO, true, false>), grid, block, 0, stream, p, waves);
    } else {
        if (p.qk_l2norm) hipLaunchKernelGGL((delta_step_kernel<K, IO, false, true>), grid, block, 0, stream, p, waves);
        else hipLaunchKernelGGL((delta_step_kernel<K, IO, false, false>), grid, block, 0, stream, p, waves);
    }
}

}  // namespace

hipError_t launch_delta_step(const DeltaParams &p, hipStream_t stream)
{
    const int64_t waves = (int64_t)p.N * p.HV * (p.V / SW_COLS);
    constexpr int wpg = 4;  // waves per workgroup (they share nothing)
    const dim3 grid((unsigned)((waves + wpg - 1) / wpg)), block(64 * wpg);
    if (p.K == 128) {
        if (p.io == IO_F16) launch_step<128, IO_F16>(p, grid, block, waves, stream);
        else launch_step<128, IO_BF16>(p, grid, block, waves, stream);
    } else {
        if (p.io == IO_F16) launch_step<64, IO_F16>(p, grid, block, waves, stream);
        else launch_step<64, IO_BF16>(p, grid, block, waves, stream);
    }
    return hipGetLastError();
}

}  // namespace gdn2
