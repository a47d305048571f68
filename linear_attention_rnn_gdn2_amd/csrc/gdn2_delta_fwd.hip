// Scalar-gated delta rule, chunked (CDNA4, gfx950): the chunk-parallel
// preparation and the sequential pass over the chunks.
//
// Per sequence and value head, with a K x V float32 state S and scalars
// g <= 0 and beta per token (the channel-wise rule of this library with one
// gate for all channels, and the write gate equal to beta):
//
//     S' = e^g S;  u = beta (v - S'^T k);  S = S' + k u^T;  o = scale S^T q
//
// A chunk of 64 tokens with G the running sum of g and D_rs = e^(G_r - G_s):
//
//     A_rs = beta_r D_rs (k_r . k_s), s < r;      T = (I + A)^-1
//     P_rs = scale D_rs (q_r . k_s), s <= r
//     R = beta (V - e^G (K S));   U = T R;   O = scale e^G (Q S) + P U
//     S <- e^(G_C) S + K^T (e^(G_C - G) U)
//
// T and P depend on q, k and the gates alone, so a first kernel computes them
// for all chunks at once (delta_wy_kernel, one record per chunk and value
// head), and the sequential kernel (delta_state_kernel) is left with products
// of small operands in which every 16 value columns are independent: a wave
// keeps its K x 16 columns of S in registers for the whole sequence and needs
// nothing from other waves but the staged tiles of K, Q, T and P.
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "gdn2_delta_device.h"

namespace gdn2 {
namespace {

using namespace dev;

// ------------------------------------------------------------ preparation --
// One workgroup (4 waves) per (chunk, value head). Wave w owns block row w
// (16 tokens) of the two score products, inverts the diagonal block w by
// forward substitution, and then carries block column w of the inverse:
//     T_ij = -T_ii (sum_{j <= m < i} A_im T_mj)
// in float32 MFMA (16x16x4), whose accumulators are its next right operands.
template <int K>
struct WyLds {
    static constexpr int RS = 2 * K + 16;  // row stride of a staged tile (bytes): rows 16 bytes apart in banks
    static constexpr int TILE = 64 * RS;
    static constexpr int K0 = 0, Q0 = TILE;
    static constexpr int PL = 0;           // output planes, over the tiles once both products are done
    static constexpr int PLANE = 64 * PSTR;
    static constexpr int AS = 68;          // floats per row of A
    static constexpr int A0 = 2 * TILE > 4 * PLANE ? 2 * TILE : 4 * PLANE;
    static constexpr int TS = 20;          // floats per row of an inverted diagonal block
    static constexpr int T0 = A0 + 64 * AS * 4;
    static constexpr int V0 = T0 + 4 * 16 * TS * 4;
    static constexpr int SIZE = V0 + 6 * 256;
};

template <int K, int IO, bool L2N>
__global__ __launch_bounds__(256) void delta_wy_kernel(DeltaParams p)
{
    using L = WyLds<K>;
    __shared__ __attribute__((aligned(16))) char sm[L::SIZE];
    const int hv = (int)(blockIdx.x % (unsigned)p.HV);
    const int64_t slot = blockIdx.x / (unsigned)p.HV;
    int n;
    int64_t c;
    if (!slot_owner(p.cu, p.cu64, p.T, p.N, slot, &n, &c)) return;
    const SeqRange rng = seq_of(p, n);
    const int64_t t0 = rng.b + c * CHUNK;
    const int len = (int)(rng.e - t0 < CHUNK ? rng.e - t0 : CHUNK);
    const int hk = hv / (p.HV / p.H);
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63, q4 = lane >> 4, l16 = lane & 15;

    // the tiles (rows past the chunk's end are zeros by the buffers' range)
    {
        const __amdgpu_buffer_rsrc_t rk = buf_rsrc(p.k + t0 * p.sk + hk * p.hsk, (int)(((len - 1) * p.sk + K) * 2));
        const __amdgpu_buffer_rsrc_t rq = buf_rsrc(p.q + t0 * p.sq + hk * p.hsq, (int)(((len - 1) * p.sq + K) * 2));
        constexpr int CPT = 64 * K / 8 / 256;
        i32x4 a[CPT], b[CPT];
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int ci = t + 256 * i, row = ci / (K / 8), col = ci % (K / 8);
            a[i] = buf_ld16<i32x4>(rk, (uint32_t)(row * (int)p.sk + col * 8) * 2);
            b[i] = buf_ld16<i32x4>(rq, (uint32_t)(row * (int)p.sq + col * 8) * 2);
        }
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int ci = t + 256 * i, row = ci / (K / 8), col = ci % (K / 8);
            lds_st(sm, L::K0 + row * L::RS + col * 16, a[i]);
            lds_st(sm, L::Q0 + row * L::RS + col * 16, b[i]);
        }
    }
    float *vec = reinterpret_cast<float *>(sm + L::V0);  // G hi, G lo, beta, e^G (unscaled), rk, rq
    char *rec = p.rec + delta_item(p, slot, hv) * (int64_t)DeltaRecord::BYTES;
    float *rvec = reinterpret_cast<float *>(rec + DeltaRecord::VEC);
    double G = 0.0, GC = 0.0;
    float bt = 0.0f;
    if (wave == 0) {
        // running sum of g in 64 bits: its differences are exponents, and a
        // strongly decayed chunk's sum is far larger than they are
        float g = 0.0f;
        if (lane < len) {
            const int64_t tok = t0 + lane;
            if (p.g) {
                const int64_t o = tok * p.sg + hv * p.hsg;
                if (p.gtype == G_F32) g = static_cast<const float *>(p.g)[o];
                else if (p.gtype == G_F16) g = io_f32<IO_F16>(static_cast<const uint16_t *>(p.g)[o]);
                else g = io_f32<IO_BF16>(static_cast<const uint16_t *>(p.g)[o]);
            }
            bt = p.beta ? io_f32<IO>(p.beta[tok * p.sb + hv * p.hsb]) : 1.0f;
        }
        G = (double)g * 1.4426950408889634074;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double x = __shfl_up(G, d);
            if (lane >= d) G += x;
        }
        GC = __shfl(G, 63);
        const float gh = (float)G;
        vec[lane] = gh;
        vec[64 + lane] = (float)(G - (double)gh);
        vec[128 + lane] = bt;
    }
    __syncthreads();
    float rkv = 1.0f, rqv = 1.0f;
    if constexpr (L2N) {
        // reciprocal norms of the rows of q and k: four threads per row
        const int row = t >> 2, part = t & 3;
        float sk = 0.0f, sq = 0.0f;
#pragma unroll
        for (int i = 0; i < K / 32; ++i) {
            const uint16_t *a = reinterpret_cast<const uint16_t *>(sm + L::K0 + row * L::RS) + part * (K / 4) + 8 * i;
            const uint16_t *b = reinterpret_cast<const uint16_t *>(sm + L::Q0 + row * L::RS) + part * (K / 4) + 8 * i;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = io_f32<IO>(a[j]), y = io_f32<IO>(b[j]);
                sk = fmaf(x, x, sk);
                sq = fmaf(y, y, sq);
            }
        }
        sk += __shfl_xor(sk, 1);
        sq += __shfl_xor(sq, 1);
        sk += __shfl_xor(sk, 2);
        sq += __shfl_xor(sq, 2);
        if (part == 0) {
            vec[256 + row] = 1.0f / fmaxf(sqrtf(sk), 1e-12f);
            vec[320 + row] = 1.0f / fmaxf(sqrtf(sq), 1e-12f);
        }
        __syncthreads();
    }
    if (wave == 0) {
        if constexpr (L2N) {
            rkv = vec[256 + lane];
            rqv = vec[320 + lane];
        }
        const float eg = ex2((float)G);
        rvec[DeltaRecord::EG * 64 + lane] = eg * rkv;
        rvec[DeltaRecord::EQ * 64 + lane] = eg * rqv * p.scale;
        rvec[DeltaRecord::ED * 64 + lane] = ex2((float)(GC - G)) * rkv;
        rvec[DeltaRecord::BT * 64 + lane] = bt;
        rvec[DeltaRecord::GH * 64 + lane] = (float)G;
        rvec[DeltaRecord::GL * 64 + lane] = (float)(G - (double)(float)G);
        if (lane == 0) *reinterpret_cast<float *>(rec + DeltaRecord::GAMMA) = ex2((float)GC);
    }

    // block row `wave` of K K^T and Q K^T, decayed and masked
    float *A = reinterpret_cast<float *>(sm + L::A0);
    f32x4 P[4];
    {
        auto mm = [](i32x4 a, i32x4 b, f32x4 acc) {
            if constexpr (IO == IO_F16)
                return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), acc, 0, 0, 0);
            else return mfma_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc);
        };
        i32x4 ka[K / 32], qa[K / 32];
#pragma unroll
        for (int j = 0; j < K / 32; ++j) {
            ka[j] = lds_ld<i32x4>(sm, L::K0 + (16 * wave + l16) * L::RS + 64 * j + 16 * q4);
            qa[j] = lds_ld<i32x4>(sm, L::Q0 + (16 * wave + l16) * L::RS + 64 * j + 16 * q4);
        }
        const f32x4 gh = lds_ld<f32x4>(sm, L::V0 + (16 * wave + 4 * q4) * 4);
        const f32x4 gl = lds_ld<f32x4>(sm, L::V0 + 256 + (16 * wave + 4 * q4) * 4);
        const f32x4 b4 = lds_ld<f32x4>(sm, L::V0 + 512 + (16 * wave + 4 * q4) * 4);
        f32x4 rk4 = {1, 1, 1, 1}, rq4 = {1, 1, 1, 1};
        if constexpr (L2N) {
            rk4 = lds_ld<f32x4>(sm, L::V0 + 1024 + (16 * wave + 4 * q4) * 4);
            rq4 = lds_ld<f32x4>(sm, L::V0 + 1280 + (16 * wave + 4 * q4) * 4);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            P[s] = f32x4{0, 0, 0, 0};
            if (s > wave) continue;
            f32x4 kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < K / 32; ++j) {
                const i32x4 b = lds_ld<i32x4>(sm, L::K0 + (16 * s + l16) * L::RS + 64 * j + 16 * q4);
                kk = mm(ka[j], b, kk);
                qk = mm(qa[j], b, qk);
            }
            const int col = 16 * s + l16;
            const float gsh = vec[col], gsl = vec[64 + col];
            float rks = 1.0f;
            if constexpr (L2N) rks = vec[256 + col];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 16 * wave + 4 * q4 + e;
                // the exponent is not positive for s <= r; above the diagonal the product is not used
                const float d = ex2(fminf((gh[e] - gsh) + (gl[e] - gsl), 0.0f)) * rks;
                A[row * L::AS + col] = col < row ? b4[e] * d * rk4[e] * kk[e] : 0.0f;
                P[s][e] = col <= row ? p.scale * d * rq4[e] * qk[e] : 0.0f;
            }
        }
    }
    __syncthreads();  // A is complete; the tiles are done with

    // P and the zero blocks above the diagonal
    auto st_plane = [&](int plane, int brow, int bcol, f32x4 x) {
        bf16x4 h, l;
        split4(x, h, l);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int o = L::PL + plane * L::PLANE + (16 * brow + 4 * q4 + e) * PSTR + 2 * (16 * bcol + l16);
            lds_st(sm, o, h[e]);
            lds_st(sm, o + L::PLANE, l[e]);
        }
    };
#pragma unroll
    for (int s = 0; s < 4; ++s)
        if (s <= wave) st_plane(2, wave, s, P[s]);
    if (!(wave & 1)) {
        st_plane(2, wave, wave + 1, f32x4{0, 0, 0, 0});
        st_plane(0, wave, wave + 1, f32x4{0, 0, 0, 0});
    }

    // diagonal block `wave` of T: column l16 by forward substitution
    float *TD = reinterpret_cast<float *>(sm + L::T0);
    {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == l16 ? 1.0f : 0.0f;
        const float *Ad = A + 16 * wave * L::AS + 16 * wave;
#pragma unroll
        for (int i = 1; i < 16; ++i) {
            float s = x[i];
#pragma unroll
            for (int m4 = 0; m4 < (i + 3) / 4; ++m4) {
                const f32x4 a = *reinterpret_cast<const f32x4 *>(Ad + i * L::AS + 4 * m4);
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    if (4 * m4 + m < i) s = fmaf(-a[m], x[4 * m4 + m], s);
            }
            x[i] = s;
        }
        if (q4 == 0)
#pragma unroll
            for (int i = 0; i < 16; ++i) TD[(16 * wave + i) * L::TS + l16] = x[i];
    }
    __syncthreads();
    // block column `wave`
    {
        f32x4 Tc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < wave) continue;
            if (i == wave) {
#pragma unroll
                for (int e = 0; e < 4; ++e) Tc[i][e] = TD[(16 * i + 4 * q4 + e) * L::TS + l16];
            } else {
                f32x4 acc = {0, 0, 0, 0}, res = {0, 0, 0, 0};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    if (m < wave || m >= i) continue;
                    const f32x4 a = *reinterpret_cast<const f32x4 *>(A + (16 * i + l16) * L::AS + 16 * m + 4 * q4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], Tc[m][e], acc, 0, 0, 0);
                }
                const f32x4 td = *reinterpret_cast<const f32x4 *>(TD + (16 * i + l16) * L::TS + 4 * q4);
#pragma unroll
                for (int e = 0; e < 4; ++e) res = __builtin_amdgcn_mfma_f32_16x16x4f32(td[e], acc[e], res, 0, 0, 0);
                Tc[i] = -res;
            }
            st_plane(0, i, wave, Tc[i]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 6; ++i) {
        const int id = t + 256 * i, plane = id / 384, ci = id % 384;
        int row, col;
        plane_pos(ci, row, col);
        *reinterpret_cast<i32x4 *>(rec + plane * DeltaRecord::PLANE + 16 * ci) =
            lds_ld<i32x4>(sm, L::PL + plane * L::PLANE + row * PSTR + 16 * col);
    }
}

// -------------------------------------------------------- sequential pass --
// One workgroup per (sequence, value head, 16 NW value columns); wave w owns
// 16 columns. The next chunk's tiles are loaded into registers while the
// current one is computed from LDS.
template <int K, int NP, int NW, bool CKPT>
struct StateLds {
    static constexpr int RS = 2 * K + 16;
    static constexpr int TILE = 64 * RS;
    static constexpr int K0 = 0;
    static constexpr int Q0 = NP * TILE;
    static constexpr int PLANE = 64 * PSTR;
    static constexpr int NPL = CKPT ? 2 : 4;  // T only, or T and P
    static constexpr int P0 = (CKPT ? 1 : 2) * NP * TILE;
    static constexpr int V0 = P0 + NPL * PLANE;
    static constexpr int VB = DeltaRecord::NVEC * 256 + 16;  // vectors and gamma
    static constexpr int SIZE = V0 + VB;
};

template <int K, int IO, int NW, bool CKPT>
__global__ __launch_bounds__(64 * NW) void delta_state_kernel(DeltaParams p)
{
    constexpr int NP = IO == IO_F16 ? 2 : 1;
    using L = StateLds<K, NP, NW, CKPT>;
    constexpr int NT = 64 * NW;
    constexpr int KT = K / 16, KS = K / 32;
    __shared__ __attribute__((aligned(16))) char sm[L::SIZE];
    const int nvb = p.V / (16 * NW);
    int item = blockIdx.x;
    const int vb = item % nvb;
    item /= nvb;
    const int hv = item % p.HV, n = item / p.HV;
    const int hk = hv / (p.HV / p.H);
    const SeqRange rng = seq_of(p, n);
    const int64_t nch = chunks_of(rng);
    const int64_t slot0 = chunk_slot(rng.b, n, 0);
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63, q4 = lane >> 4, l16 = lane & 15;
    const int col = (vb * NW + wave) * 16 + l16;
    const int64_t shead = ((int64_t)n * p.HV + hv) * K * p.V;
    const int64_t sr = p.state_vmajor ? 1 : p.V, sc = p.state_vmajor ? K : 1;

    f32x4 S[KT];
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            S[i][e] = p.h0 ? state_ld(p.h0, p.h0_bf16, shead + (16 * i + 4 * q4 + e) * sr + col * sc) : 0.0f;

    constexpr int CPT = 64 * K / 8 / NT;                    // 16-byte chunks of a tile per thread
    constexpr int RCH = L::NPL * 384;
    constexpr int RPT = (RCH + NT - 1) / NT;                // ... of the record's planes
    constexpr int VCH = DeltaRecord::NVEC * 16 + 1;         // ... of its vectors
    static_assert(NT >= VCH, "one vector chunk per thread");
    i32x4 fk[CPT], fq[CKPT ? 1 : CPT], fr[RPT], fv;
    uint16_t vv[16];

    auto fetch = [&](int64_t c) {
        const int64_t t0 = rng.b + c * CHUNK;
        const int len = (int)(rng.e - t0 < CHUNK ? rng.e - t0 : CHUNK);
        const __amdgpu_buffer_rsrc_t rk = buf_rsrc(p.k + t0 * p.sk + hk * p.hsk, (int)(((len - 1) * p.sk + K) * 2));
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int ci = t + NT * i, row = ci / (K / 8), cc = ci % (K / 8);
            fk[i] = buf_ld16<i32x4>(rk, (uint32_t)(row * (int)p.sk + cc * 8) * 2);
        }
        if constexpr (!CKPT) {
            const __amdgpu_buffer_rsrc_t rq = buf_rsrc(p.q + t0 * p.sq + hk * p.hsq, (int)(((len - 1) * p.sq + K) * 2));
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                const int ci = t + NT * i, row = ci / (K / 8), cc = ci % (K / 8);
                fq[i] = buf_ld16<i32x4>(rq, (uint32_t)(row * (int)p.sq + cc * 8) * 2);
            }
        }
        const char *rec = p.rec + delta_item(p, slot0 + c, hv) * (int64_t)DeltaRecord::BYTES;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int id = t + NT * i;
            if (RCH % NT == 0 || id < RCH) fr[i] = *reinterpret_cast<const i32x4 *>(rec + 16 * id);
        }
        if (t < VCH) fv = *reinterpret_cast<const i32x4 *>(rec + DeltaRecord::VEC + 16 * t);
        const __amdgpu_buffer_rsrc_t rv = buf_rsrc(p.v + t0 * p.sv + hv * p.hsv, (int)(((len - 1) * p.sv + p.V) * 2));
#pragma unroll
        for (int i = 0; i < 16; ++i)
            vv[i] = __builtin_amdgcn_raw_buffer_load_b16(rv, (uint32_t)((16 * (i >> 2) + 4 * q4 + (i & 3)) * (int)p.sv + col) * 2, 0, 0);
    };
    auto stage = [&]() {
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int ci = t + NT * i, row = ci / (K / 8), cc = ci % (K / 8);
            st_parts<NP>(sm + L::K0, L::TILE, row * L::RS + cc * 16, fk[i]);
            if constexpr (!CKPT) st_parts<NP>(sm + L::Q0, L::TILE, row * L::RS + cc * 16, fq[i]);
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int id = t + NT * i;
            if (RCH % NT == 0 || id < RCH) {
                const int plane = id / 384;
                int row, cc;
                plane_pos(id % 384, row, cc);
                lds_st(sm, L::P0 + plane * L::PLANE + row * PSTR + 16 * cc, fr[i]);
            }
        }
        if (t < VCH) lds_st(sm, L::V0 + 16 * t, fv);
    };

    if (nch > 0) fetch(0);
    for (int64_t c = 0; c < nch; ++c) {
        const int64_t t0 = rng.b + c * CHUNK;
        const int len = (int)(rng.e - t0 < CHUNK ? rng.e - t0 : CHUNK);
        float v32[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v32[i] = io_f32<IO>(vv[i]);
        stage();
        __syncthreads();
        if (c + 1 < nch) fetch(c + 1);

        const int64_t frag = delta_item(p, slot0 + c, hv) * (p.V / 16) + (vb * NW + wave);
        auto vec4 = [&](int which, int mt) { return lds_ld<f32x4>(sm, L::V0 + which * 256 + (16 * mt + 4 * q4) * 4); };
        const float gamma = lds_ld<float>(sm, L::V0 + DeltaRecord::NVEC * 256);

        bf16x8 Sh[KS], Sl[KS];
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            bf16x4 h0, l0, h1, l1;
            split4(S[2 * j], h0, l0);
            split4(S[2 * j + 1], h1, l1);
            Sh[j] = cat4(h0, h1);
            Sl[j] = cat4(l0, l1);
        }
        if constexpr (CKPT) {
            f32x4 *dst = reinterpret_cast<f32x4 *>(p.s_ck) + frag * (KT * 64) + lane;
#pragma unroll
            for (int i = 0; i < KT; ++i) dst[64 * i] = S[i];
        }
        // [tile] S for the K (and Q) tile at LDS offset `base`: rows 16 mt ..
        auto times_state = [&](int base, int mt) {
            f32x4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                const bf16x8 a = ld_row(sm + base, L::RS, 16 * mt + l16, 32 * j, q4);
                bf16x8 al = a;
                if constexpr (NP == 2) al = ld_row(sm + base + L::TILE, L::RS, 16 * mt + l16, 32 * j, q4);
                acc = mfma_split<NP == 2>(a, al, Sh[j], Sl[j], acc);
            }
            return acc;
        };
        // R = beta (V - e^G K S) as a right operand
        bf16x8 Rh[2], Rl[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            bf16x4 h[2], l[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int mt = 2 * j + i;
                const f32x4 x = times_state(L::K0, mt), eg = vec4(DeltaRecord::EG, mt), bt = vec4(DeltaRecord::BT, mt);
                f32x4 r;
#pragma unroll
                for (int e = 0; e < 4; ++e) r[e] = bt[e] * (v32[4 * mt + e] - eg[e] * x[e]);
                split4(r, h[i], l[i]);
            }
            Rh[j] = cat4(h[0], h[1]);
            Rl[j] = cat4(l[0], l[1]);
        }
        // U = T R, and e^(G_C - G) U
        bf16x8 Uh[2], Ul[2], Wh[2], Wl[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            bf16x4 h[2], l[2], wh[2], wl[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int mt = 2 * j + i;
                f32x4 u = {0, 0, 0, 0};
#pragma unroll
                for (int jj = 0; jj <= j; ++jj)
                    u = mfma_split<true>(ld_row(sm + L::P0, PSTR, 16 * mt + l16, 32 * jj, q4),
                                         ld_row(sm + L::P0 + L::PLANE, PSTR, 16 * mt + l16, 32 * jj, q4), Rh[jj], Rl[jj], u);
                if constexpr (CKPT) reinterpret_cast<f32x4 *>(p.u_ck)[frag * 256 + 64 * mt + lane] = u;
                const f32x4 ed = vec4(DeltaRecord::ED, mt);
                split4(u, h[i], l[i]);
                split4(u * ed, wh[i], wl[i]);
            }
            Uh[j] = cat4(h[0], h[1]);
            Ul[j] = cat4(l[0], l[1]);
            Wh[j] = cat4(wh[0], wh[1]);
            Wl[j] = cat4(wl[0], wl[1]);
        }
        if constexpr (!CKPT) {
            const __amdgpu_buffer_rsrc_t ro = buf_rsrc(p.out + t0 * p.so + hv * p.hso, (int)(((len - 1) * p.so + p.V) * 2));
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                f32x4 o = times_state(L::Q0, mt) * vec4(DeltaRecord::EQ, mt);
#pragma unroll
                for (int jj = 0; jj <= mt / 2; ++jj)
                    o = mfma_split<true>(ld_row(sm + L::P0 + 2 * L::PLANE, PSTR, 16 * mt + l16, 32 * jj, q4),
                                         ld_row(sm + L::P0 + 3 * L::PLANE, PSTR, 16 * mt + l16, 32 * jj, q4), Uh[jj], Ul[jj], o);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // a row past the chunk's end lies past the buffer's range and is dropped
                    __builtin_amdgcn_raw_buffer_store_b16(f32_io<IO>(o[e]), ro, (uint32_t)((16 * mt + 4 * q4 + e) * (int)p.so + col) * 2, 0, 0);
                }
            }
        }
        // S <- e^(G_C) S + K^T (e^(G_C - G) U)
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            f32x4 s = S[i] * gamma;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bf16x8 a = ld_col(sm + L::K0, L::RS, 32 * j, 16 * i, q4, l16);
                bf16x8 al = a;
                if constexpr (NP == 2) al = ld_col(sm + L::K0 + L::TILE, L::RS, 32 * j, 16 * i, q4, l16);
                s = mfma_split<NP == 2>(a, al, Wh[j], Wl[j], s);
            }
            S[i] = s;
        }
        __syncthreads();  // everybody is done with this chunk's tiles
    }
    if (p.ht)
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                state_st(p.ht, p.ht_bf16, shead + (16 * i + 4 * q4 + e) * sr + col * sc, S[i][e]);
}

template <int K, int IO>
void launch_wy_l2(const DeltaParams &p, dim3 grid, hipStream_t stream)
{
    if (p.qk_l2norm) hipLaunchKernelGGL((delta_wy_kernel<K, IO, true>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((delta_wy_kernel<K, IO, false>), grid, dim3(256), 0, stream, p);
}

template <int K, int IO, int NW>
void launch_state_ck(const DeltaParams &p, bool ckpt, hipStream_t stream)
{
    const dim3 grid((unsigned)((int64_t)p.N * p.HV * (p.V / (16 * NW))));
    if (ckpt) hipLaunchKernelGGL((delta_state_kernel<K, IO, NW, true>), grid, dim3(64 * NW), 0, stream, p);
    else hipLaunchKernelGGL((delta_state_kernel<K, IO, NW, false>), grid, dim3(64 * NW), 0, stream, p);
}

}  // namespace

hipError_t launch_delta_wy(const DeltaParams &p, hipStream_t stream)
{
    if (p.T == 0) return hipSuccess;
    const dim3 grid((unsigned)((int64_t)p.nslots * p.HV));
    if (p.K == 128) {
        if (p.io == IO_F16) launch_wy_l2<128, IO_F16>(p, grid, stream);
        else launch_wy_l2<128, IO_BF16>(p, grid, stream);
    } else {
        if (p.io == IO_F16) launch_wy_l2<64, IO_F16>(p, grid, stream);
        else launch_wy_l2<64, IO_BF16>(p, grid, stream);
    }
    return hipGetLastError();
}

hipError_t launch_delta_state(const DeltaParams &p, bool ckpt, int ncu, hipStream_t stream)
{
    (void)ncu;
    if (p.K == 128) {
        if (p.io == IO_F16) launch_state_ck<128, IO_F16, 4>(p, ckpt, stream);
        else launch_state_ck<128, IO_BF16, 4>(p, ckpt, stream);
    } else {
        if (p.io == IO_F16) launch_state_ck<64, IO_F16, 4>(p, ckpt, stream);
        else launch_state_ck<64, IO_BF16, 4>(p, ckpt, stream);
    }
    return hipGetLastError();
}

}  // namespace gdn2
