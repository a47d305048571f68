// Scalar-gated delta rule, gradients (CDNA4, gfx950). After the preparation
// (T, P) and the sequential pass with checkpoints (the state S entering each
// chunk, and U), with dS the gradient of the state that leaves a chunk:
//
//     dU = P^T dO + e^(G_C - G) (K dS);   dY = T^T dU;   dV = beta dY
//     dS <- e^(G_C) dS + Q^T (scale e^G dO) - K^T (e^G dV)
//
// runs over the chunks in reverse (delta_bwd_state_kernel: like the forward
// pass, every 16 value columns are independent), and then, for every chunk at
// once (delta_bwd_grad_kernel), with dP_rs = scale D_rs (dO_r . u_s), s <= r,
// and dA_rs = -beta_r D_rs (dY_r . u_s), s < r, the gradients of the scores:
//
//     dQ = scale e^G (dO S^T) + dP K
//     dK = dP^T Q + (dA + dA^T) K + e^(G_C - G) (U dS^T) - e^G beta (dY S^T)
//     dbeta_r = dY_r . v_r - e^G_r k_r . (S dY_r) - sum_{s<r} D_rs (k_r . k_s) (dY_r . u_s)
//     dg_t = sum_{r >= t > s} E_rs + sum_{r >= t} I_r + sum_{s < t} X_s + e^(G_C) <S, dS>
//
// where E = dP (q k) + dA (k k) below the diagonal, I_r is what enters row r
// from the state and X_s what row s leaves in it: dg_t sums every product
// of decays that spans token t, so that no two sums are subtracted.
#include <stdint.h>

#include <type_traits>

#include <hip/hip_runtime.h>

#include "gdn2_delta_device.h"

namespace gdn2 {
namespace {

using namespace dev;

// ----------------------------------------------------- reverse sequential --
// As the forward's sequential pass: NC computing waves of 16 value columns
// each, 4 staging waves. T and P are used transposed, through transpose reads
// of their planes, which are staged row-major for that (PlaneTile).
constexpr int LW = 4;  // staging waves

// A record's plane, row-major: columns 0 .. 31 of all rows, then columns
// 32 .. 63 of rows 32 .. 63 (the others are above the diagonal), in rows of 64
// bytes whose 16-byte pieces are permuted so that a transpose read touches
// every bank once.
struct PlaneTile {
    static constexpr int BYTES = 6144;
    __device__ static __forceinline__ int swz(int r) { return (r >> 2 & 1) << 1 | (r >> 3 & 1); }
    // byte offset of the four columns 4 c .. of row r
    __device__ static __forceinline__ int quad(int r, int c)
    {
        return c / 8 * 2048 + r * 64 + (((c % 8 >> 1) ^ swz(r)) << 4) + 8 * (c & 1);
    }
    // transposed: element (m, k) = plane[k][m], rows k = 32 j + 4 q4 .. and 32 j + 16 + 4 q4 .., columns m = 16 i + l16, i <= 2 j + 1
    __device__ static __forceinline__ bf16x8 col(const char *plane, int i, int j, int q4, int l16)
    {
        const int a = quad(4 * q4 + (l16 >> 2), 4 * (i & 1) + (l16 & 3)) + i / 2 * 2048 + 32 * 64 * j;
        return cat4(lds_tr(plane, a), lds_tr(plane, a + 16 * 64));
    }
};

template <int K, int COLS>
struct BwdStateLds {
    static constexpr int TILE = Tile<K>::BYTES;
    static constexpr int OS = 2 * COLS + 16;  // row stride of the dO tile (later the chunk's dV)
    static constexpr int K0 = 0, Q0 = TILE;
    static constexpr int O0 = 2 * TILE;
    static constexpr int R0 = O0 + 64 * OS;   // planes of T and P
    static constexpr int G0 = R0 + 4 * PlaneTile::BYTES;
    static constexpr int VCH = (DeltaRecord::GAMMA + 16 - DeltaRecord::VEC) / 16;
    static constexpr int HALF = (G0 + 16 * VCH + 511) / 512 * 512;
    static constexpr int SIZE = 2 * HALF;
};

template <int K, int IO, int NC>
__global__ __launch_bounds__(64 * (NC + LW)) void delta_bwd_state_kernel(DeltaParams p)
{
    constexpr int COLS = 16 * NC;
    using L = BwdStateLds<K, COLS>;
    using TL = Tile<K>;
    constexpr int KT = K / 16, KS = K / 32;
    __shared__ __attribute__((aligned(16))) char sm[L::SIZE];
    const int nvb = p.V / COLS;
    int item = blockIdx.x;
    const int vb = item % nvb;
    item /= nvb;
    const int hv = item % p.HV, n = item / p.HV;
    const int hk = hv / (p.HV / p.H);
    const SeqRange rng = seq_of(p, n);
    const int64_t nch = chunks_of(rng);
    const int64_t slot0 = chunk_slot(rng.b, n, 0);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;

    if (wave >= NC) {
        const int t = threadIdx.x - 64 * NC;
        constexpr int TH = 64 * LW;
        constexpr int CPT = 64 * K / 8 / TH;
        constexpr int OCH = 64 * COLS / 8, OPT = (OCH + TH - 1) / TH;
        constexpr int RPT = 4 * DeltaRecord::PLANE / 16 / TH;  // 6
        static_assert(L::VCH <= TH && 4 * DeltaRecord::PLANE == 16 * RPT * TH, "pieces per thread");
        i32x4 fk[CPT], fq[CPT], fo[OPT], fr[RPT], fv;
        auto fetch = [&](int64_t c) {
            const int64_t t0 = rng.b + c * CHUNK;
            const int len = (int)(rng.e - t0 < CHUNK ? rng.e - t0 : CHUNK);
            const __amdgpu_buffer_rsrc_t rk = buf_rsrc(p.k + t0 * p.sk + hk * p.hsk, (int)(((len - 1) * p.sk + K) * 2));
            const __amdgpu_buffer_rsrc_t rq = buf_rsrc(p.q + t0 * p.sq + hk * p.hsq, (int)(((len - 1) * p.sq + K) * 2));
            const __amdgpu_buffer_rsrc_t ro = buf_rsrc(p.dout + t0 * p.sv + hv * p.hsv, (int)(((len - 1) * p.sv + p.V) * 2));
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                const int ci = t + TH * i, row = ci / (K / 8), cc = ci % (K / 8);
                fk[i] = buf_ld16<i32x4>(rk, (uint32_t)(row * (int)p.sk + cc * 8) * 2);
                fq[i] = buf_ld16<i32x4>(rq, (uint32_t)(row * (int)p.sq + cc * 8) * 2);
            }
#pragma unroll
            for (int i = 0; i < OPT; ++i) {
                const int ci = t + TH * i, row = ci / (COLS / 8), cc = ci % (COLS / 8);
                if (OCH % TH == 0 || ci < OCH)
                    fo[i] = buf_ld16<i32x4>(ro, (uint32_t)(row * (int)p.sv + vb * COLS + cc * 8) * 2);
            }
            const char *rec = p.rec + delta_item(p, slot0 + c, hv) * (int64_t)DeltaRecord::BYTES;
#pragma unroll
            for (int i = 0; i < RPT; ++i) fr[i] = *reinterpret_cast<const i32x4 *>(rec + 16 * (t + TH * i));
            if (t < L::VCH) fv = *reinterpret_cast<const i32x4 *>(rec + DeltaRecord::VEC + 16 * t);
        };
        auto stage = [&](char *half) {
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                const int ci = t + TH * i, row = ci / (K / 8), cc = ci % (K / 8);
                lds_st(half, L::K0 + TL::piece(row, cc), fk[i]);
                lds_st(half, L::Q0 + TL::piece(row, cc), fq[i]);
            }
#pragma unroll
            for (int i = 0; i < OPT; ++i) {
                const int ci = t + TH * i, row = ci / (COLS / 8), cc = ci % (COLS / 8);
                if (OCH % TH == 0 || ci < OCH) lds_st(half, L::O0 + row * L::OS + cc * 16, fo[i]);
            }
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                // 16 bytes of a fragment: two runs of four columns of one row
                const int id = t + TH * i, plane = id / 384, f = id % 384 >> 6, ln = id & 63;
                const int mt = f < 2 ? f : (f + 2) / 2, j = f < 2 ? 0 : f & 1, r = 16 * mt + (ln & 15), c4 = 8 * j + (ln >> 4);
                char *dst = half + L::R0 + plane * PlaneTile::BYTES;
                const bf16x8 x = __builtin_bit_cast(bf16x8, fr[i]);
                lds_st(dst, PlaneTile::quad(r, c4), __builtin_shufflevector(x, x, 0, 1, 2, 3));
                lds_st(dst, PlaneTile::quad(r, c4 + 4), __builtin_shufflevector(x, x, 4, 5, 6, 7));
            }
            if (t < L::VCH) lds_st(half, L::G0 + 16 * t, fv);
        };
        // dV of chunk c, left where its dO tile was (read and later overwritten by the same thread)
        auto flush = [&](int64_t c) {
            const char *half = sm + (c & 1) * L::HALF;
            const int64_t t0 = rng.b + c * CHUNK;
            const int len = (int)(rng.e - t0 < CHUNK ? rng.e - t0 : CHUNK);
#pragma unroll
            for (int i = 0; i < OPT; ++i) {
                const int ci = t + TH * i, row = ci / (COLS / 8), cc = ci % (COLS / 8);
                if (ci < OCH && row < len)
                    *reinterpret_cast<i32x4 *>(p.dv + (t0 + row) * p.sv + hv * p.hsv + vb * COLS + cc * 8) =
                        lds_ld<i32x4>(half, L::O0 + row * L::OS + cc * 16);
            }
        };
        if (nch > 0) {
            fetch(nch - 1);
            stage(sm + ((nch - 1) & 1) * L::HALF);
            if (nch > 1) fetch(nch - 2);
        }
        __syncthreads();
        for (int64_t c = nch - 1; c >= 0; --c) {
            if (c + 1 < nch) flush(c + 1);
            if (c > 0) stage(sm + ((c - 1) & 1) * L::HALF);
            if (c > 1) fetch(c - 2);
            __syncthreads();
        }
        if (nch > 0) flush(0);
        return;
    }

    const int q4 = lane >> 4, l16 = lane & 15;
    const int col = (vb * NC + wave) * 16 + l16;
    const int64_t shead = ((int64_t)n * p.HV + hv) * K * p.V;
    f32x4 dS[KT];
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) dS[i][e] = p.dht ? p.dht[shead + (int64_t)(state_row(i, q4) + e) * p.V + col] : 0.0f;
    RightOp<IO, KS> So;
    So.set(dS);
    __syncthreads();
    for (int64_t c = nch - 1; c >= 0; --c) {
        char *half = sm + (c & 1) * L::HALF;
        const char *KL = half + L::K0, *QL = half + L::Q0;
        const char *TH = half + L::R0, *PH = TH + 2 * PlaneTile::BYTES;
        const int64_t frag = delta_item(p, slot0 + c, hv) * (p.V / 16) + (vb * NC + wave);
        auto vec = [&](int which, f32x4 (&x)[4]) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) x[mt] = lds_ld<f32x4>(half, L::G0 + which * 256 + (16 * mt + 4 * q4) * 4);
        };
        const float gamma = lds_ld<float>(half, L::G0 + DeltaRecord::NVEC * 256);
        {
            f32x4 *dst = reinterpret_cast<f32x4 *>(p.ds_ck) + frag * (KT * 64) + lane;
#pragma unroll
            for (int i = 0; i < KT; ++i) dst[64 * i] = dS[i];
        }
        constexpr f32x4 zero = {0, 0, 0, 0};
        // dU = e^(G_C - G) (K dS) + P^T dO
        f32x4 U[4] = {zero, zero, zero, zero}, x4[4];
        bf16x8 a[4], b[4], Uh[2], Ul[2];
#pragma unroll
        for (int j = 0; j < KS; ++j) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) a[mt] = TL::row(KL, mt, j, q4, l16);
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) U[mt] = So.mul1(a[mt], j, part, U[mt]);
        }
        vec(DeltaRecord::ED, x4);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) U[mt] = So.scaled(U[mt]) * x4[mt];
        bf16x4 raw[4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
            raw[mt] = lds_tr(half, L::O0 + (16 * mt + 4 * q4 + (l16 >> 2)) * L::OS + 2 * (16 * wave + 4 * (l16 & 3)));
        f32x4 dO[4];
        bf16x8 Oh[2], Ol[2];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) dO[mt] = io4_f32<IO>(raw[mt]);
        if constexpr (IO == IO_F16) {
            split_rows(dO, Oh, Ol);
        } else {
            Oh[0] = cat4(raw[0], raw[1]);
            Oh[1] = cat4(raw[2], raw[3]);
        }
        // y += (plane pair)^T (h + l); two: l is there
        auto upper = [&](const char *plane, const bf16x8 (&h)[2], const bf16x8 (&l)[2], auto two, f32x4 (&y)[4]) {
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const int top = jj ? 4 : 2;
#pragma unroll
                for (int mt = 0; mt < top; ++mt) {
                    a[mt] = PlaneTile::col(plane, mt, jj, q4, l16);
                    b[mt] = PlaneTile::col(plane + PlaneTile::BYTES, mt, jj, q4, l16);
                }
#pragma unroll
                for (int mt = 0; mt < top; ++mt) y[mt] = mfma_bf16(a[mt], h[jj], y[mt]);
#pragma unroll
                for (int mt = 0; mt < top; ++mt) y[mt] = mfma_bf16(b[mt], h[jj], y[mt]);
                if constexpr (decltype(two)::value)
#pragma unroll
                    for (int mt = 0; mt < top; ++mt) y[mt] = mfma_bf16(a[mt], l[jj], y[mt]);
            }
        };
        upper(PH, Oh, Ol, std::integral_constant<bool, IO == IO_F16>{}, U);
        split_rows(U, Uh, Ul);
        // dY = T^T dU
        f32x4 Y[4] = {zero, zero, zero, zero};
        upper(TH, Uh, Ul, std::true_type{}, Y);
        // dV = beta dY; the right operands e^G dV (negated) and scale e^G dO
        RightOp<IO, 2> E, F;
        {
            f32x4 dv[4];
            vec(DeltaRecord::BT, x4);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                reinterpret_cast<f32x4 *>(p.y_ck)[frag * 256 + 64 * mt + lane] = Y[mt];
                dv[mt] = Y[mt] * x4[mt];
                st_rows16<IO>(half + L::O0 + (16 * mt + 4 * q4) * L::OS + 32 * wave, L::OS, dv[mt], l16);
            }
            vec(DeltaRecord::EG, x4);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) dv[mt] *= -x4[mt];
            E.set(dv);
            vec(DeltaRecord::EQ, x4);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) dO[mt] *= x4[mt];
            F.set(dO);
        }
#pragma unroll
        for (int i0 = 0; i0 < KT; i0 += 4) {
            f32x4 s[4], w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i] = IO == IO_F16 ? zero : dS[i0 + i] * gamma;
                w[i] = zero;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = TL::col(KL, i0 + i, j, q4, l16);
                    b[i] = TL::col(QL, i0 + i, j, q4, l16);
                }
#pragma unroll
                for (int part = 0; part < 2; ++part) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i] = E.mul1(a[i], j, part, s[i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (IO == IO_F16) w[i] = F.mul1(b[i], j, part, w[i]);
                        else s[i] = F.mul1(b[i], j, part, s[i]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dS[i0 + i] = IO == IO_F16 ? dS[i0 + i] * gamma + s[i] * E.inv + w[i] * F.inv : s[i];
        }
        So.set(dS);
        __syncthreads();
    }
    if (p.dh0)
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) p.dh0[shead + (int64_t)(state_row(i, q4) + e) * p.V + col] = dS[i][e];
}

// --------------------------------------------------------- all gradients --
// One workgroup of D / 16 waves per (chunk, value head) (K = V = D). The
// products that contract the value dimension run over 32 columns at a time,
// staged value-major ([v][k] and [v][token], as the checkpoints' fragments
// hold them); wave w owns key columns 16 w .. 16 w + 15 of dQ and dK and
// every (D / 16)-th 16x16 tile of the two score gradients.
template <int D, int NP>
struct GradLds {
    static constexpr int RS = 2 * D + 16;
    static constexpr int TILE = 64 * RS;
    static constexpr int K0 = 0, Q0 = NP * TILE;
    static constexpr int W0 = 2 * NP * TILE;  // the block of 32 value columns
    static constexpr int OS = 80;             // row stride of the dO block (bytes)
    static constexpr int OT = 64 * OS;
    static constexpr int O0 = W0, VT0 = O0 + NP * OT;  // dO and V: [token][32]
    static constexpr int VP = 32 * PSTR;      // a plane of U or dY: [v][64 tokens]
    static constexpr int U0 = VT0 + NP * OT, Y0 = U0 + 2 * VP;
    static constexpr int SP = 32 * RS;        // a plane of S or dS: [v][D]
    static constexpr int S0 = Y0 + 2 * VP, DS0 = S0 + 2 * SP;
    static constexpr int WEND = DS0 + 2 * SP;
    // over it, once all value columns are done: E, and the score gradients' planes
    static constexpr int ES = 65;             // floats per row of E
    static constexpr int E0 = W0;
    static constexpr int PLANE = 64 * PSTR;
    static constexpr int DP0 = (E0 + 64 * ES * 4 + 15) / 16 * 16, DA0 = DP0 + 2 * PLANE;
    static constexpr int XEND = DA0 + 2 * PLANE;
    static constexpr int R0 = WEND > XEND ? WEND : XEND;  // vectors, and sums to join over waves and tiles
    static constexpr int NWV = D / 16;
    static constexpr int VEC = R0;
    static constexpr int RED = VEC + DeltaRecord::NVEC * 256 + 16;  // [wave][3][64]
    static constexpr int ROW = RED + NWV * 3 * 256;                 // [4][64]
    static constexpr int YV = ROW + 4 * 256;                        // [64]
    static constexpr int DOT = YV + 256;                            // [wave]
    static constexpr int SIZE = DOT + 16 * NWV;
};

template <int D, int IO>
__global__ __launch_bounds__(4 * D) void delta_bwd_grad_kernel(DeltaParams p)
{
    constexpr int NP = IO == IO_F16 ? 2 : 1;
    using L = GradLds<D, NP>;
    constexpr int NW = D / 16, NT = 64 * NW;
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
    const int64_t item = delta_item(p, slot, hv);
    const char *rec = p.rec + item * (int64_t)DeltaRecord::BYTES;

    constexpr int CPT = 64 * D / 8 / NT;  // 2
    {
        const __amdgpu_buffer_rsrc_t rk = buf_rsrc(p.k + t0 * p.sk + hk * p.hsk, (int)(((len - 1) * p.sk + D) * 2));
        const __amdgpu_buffer_rsrc_t rq = buf_rsrc(p.q + t0 * p.sq + hk * p.hsq, (int)(((len - 1) * p.sq + D) * 2));
        i32x4 a[CPT], b[CPT];
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int ci = t + NT * i, row = ci / (D / 8), cc = ci % (D / 8);
            a[i] = buf_ld16<i32x4>(rk, (uint32_t)(row * (int)p.sk + cc * 8) * 2);
            b[i] = buf_ld16<i32x4>(rq, (uint32_t)(row * (int)p.sq + cc * 8) * 2);
        }
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int ci = t + NT * i, row = ci / (D / 8), cc = ci % (D / 8);
            st_parts<NP>(sm + L::K0, L::TILE, row * L::RS + cc * 16, a[i]);
            st_parts<NP>(sm + L::Q0, L::TILE, row * L::RS + cc * 16, b[i]);
        }
    }
    constexpr int VCH = DeltaRecord::NVEC * 16 + 1;
    if (t < VCH) lds_st(sm, L::VEC + 16 * t, *reinterpret_cast<const i32x4 *>(rec + DeltaRecord::VEC + 16 * t));

    const __amdgpu_buffer_rsrc_t ro = buf_rsrc(p.dout + t0 * p.sv + hv * p.hsv, (int)(((len - 1) * p.sv + D) * 2));
    const __amdgpu_buffer_rsrc_t rv = buf_rsrc(p.v + t0 * p.sv + hv * p.hsv, (int)(((len - 1) * p.sv + D) * 2));
    const f32x4 *s_ck = reinterpret_cast<const f32x4 *>(p.s_ck) + item * (D / 16) * (D / 16 * 64);
    const f32x4 *ds_ck = reinterpret_cast<const f32x4 *>(p.ds_ck) + item * (D / 16) * (D / 16 * 64);
    const f32x4 *u_ck = reinterpret_cast<const f32x4 *>(p.u_ck) + item * (D / 16) * 256;
    const f32x4 *y_ck = reinterpret_cast<const f32x4 *>(p.y_ck) + item * (D / 16) * 256;

    // fragments of a block of 32 value columns: 2 (D / 16) 64 of S and dS, 512 of U and dY
    constexpr int SPT = 2 * (D / 16) * 64 / NT;  // 2
    constexpr int UPT = 512 / NT;                // 1 (D = 128), 2 (D = 64)
    f32x4 fs[SPT], fd[SPT], fu[UPT], fy[UPT];
    i32x4 fo, fv;
    auto fetch = [&](int vb) {
#pragma unroll
        for (int i = 0; i < SPT; ++i) {
            fs[i] = s_ck[vb * 2 * (D / 16) * 64 + t + NT * i];
            fd[i] = ds_ck[vb * 2 * (D / 16) * 64 + t + NT * i];
        }
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            fu[i] = u_ck[vb * 512 + t + NT * i];
            fy[i] = y_ck[vb * 512 + t + NT * i];
        }
        if (t < 256) {
            const uint32_t off = (uint32_t)((t >> 2) * (int)p.sv + vb * 32 + (t & 3) * 8) * 2;
            fo = buf_ld16<i32x4>(ro, off);
            fv = buf_ld16<i32x4>(rv, off);
        }
    };
    auto st_frag = [&](int base, int plane, int stride, f32x4 x, int id, int tiles, bool state) {
        // fragment id -> (16 columns, tile, lane): 4 consecutive rows of one value column
        const int ln = id & 63, tile = (id >> 6) % tiles, v = (id >> 6) / tiles * 16 + (ln & 15);
        const int r = state ? state_row(tile, ln >> 4) : 16 * tile + 4 * (ln >> 4);
        bf16x4 h, l;
        split4(x, h, l);
        lds_st(sm, base + v * stride + 2 * r, h);
        lds_st(sm, base + plane + v * stride + 2 * r, l);
    };

    f32x4 aq[4], ay[4], au[4];  // dO S^T, dY S^T, U dS^T: rows 16 mt .., key columns 16 wave ..
    constexpr int TPW = (10 + NW - 1) / NW;
    f32x4 ou[TPW], yu[TPW];     // dO U^T, dY U^T
#pragma unroll
    for (int i = 0; i < 4; ++i) aq[i] = ay[i] = au[i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < TPW; ++i) ou[i] = yu[i] = f32x4{0, 0, 0, 0};
    // tile id of the lower triangle -> block row and column
    auto tri = [](int id, int &br, int &bc) {
        br = id < 1 ? 0 : id < 3 ? 1 : id < 6 ? 2 : 3;
        bc = id - br * (br + 1) / 2;
    };
    f32x4 yv = {0, 0, 0, 0};
    float dot = 0.0f;  // <S, dS>
    fetch(0);
    for (int vb = 0; vb < D / 32; ++vb) {
#pragma unroll
        for (int i = 0; i < SPT; ++i) {
            st_frag(L::S0, L::SP, L::RS, fs[i], t + NT * i, D / 16, true);
            st_frag(L::DS0, L::SP, L::RS, fd[i], t + NT * i, D / 16, true);
#pragma unroll
            for (int e = 0; e < 4; ++e) dot = fmaf(fs[i][e], fd[i][e], dot);
        }
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            st_frag(L::U0, L::VP, PSTR, fu[i], t + NT * i, 4, false);
            st_frag(L::Y0, L::VP, PSTR, fy[i], t + NT * i, 4, false);
        }
        if (t < 256) {
            st_parts<NP>(sm + L::O0, L::OT, (t >> 2) * L::OS + (t & 3) * 16, fo);
            st_parts<NP>(sm + L::VT0, L::OT, (t >> 2) * L::OS + (t & 3) * 16, fv);
        }
        __syncthreads();
        if (vb + 1 < D / 32) fetch(vb + 1);
        const bf16x8 sh = ld_col_plain(sm + L::S0, L::RS, 0, 16 * wave, q4, l16);
        const bf16x8 sl = ld_col_plain(sm + L::S0 + L::SP, L::RS, 0, 16 * wave, q4, l16);
        const bf16x8 dh = ld_col_plain(sm + L::DS0, L::RS, 0, 16 * wave, q4, l16);
        const bf16x8 dl = ld_col_plain(sm + L::DS0 + L::SP, L::RS, 0, 16 * wave, q4, l16);
        auto o_row = [&](int part, int mt) { return ld_row_plain(sm + L::O0 + part * L::OT, L::OS, 16 * mt + l16, 0, q4); };
        auto v_col = [&](int base, int part, int mt) { return ld_col_plain(sm + base + part * L::VP, PSTR, 0, 16 * mt, q4, l16); };
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const bf16x8 o = o_row(0, mt);
            bf16x8 o2 = o;
            if constexpr (NP == 2) o2 = o_row(1, mt);
            aq[mt] = mfma_split<NP == 2>(o, o2, sh, sl, aq[mt]);
            ay[mt] = mfma_split<true>(v_col(L::Y0, 0, mt), v_col(L::Y0, 1, mt), sh, sl, ay[mt]);
            au[mt] = mfma_split<true>(v_col(L::U0, 0, mt), v_col(L::U0, 1, mt), dh, dl, au[mt]);
        }
#pragma unroll
        for (int i = 0; i < TPW; ++i) {
            const int id = wave + NW * i;
            if (id < 10) {
                int br, bc;
                tri(id, br, bc);
                const bf16x8 uh = v_col(L::U0, 0, bc), ul = v_col(L::U0, 1, bc), o = o_row(0, br);
                bf16x8 o2 = o;
                if constexpr (NP == 2) o2 = o_row(1, br);
                ou[i] = mfma_split<NP == 2>(o, o2, uh, ul, ou[i]);
                yu[i] = mfma_split<true>(v_col(L::Y0, 0, br), v_col(L::Y0, 1, br), uh, ul, yu[i]);
            }
        }
        if (wave < 4) {  // the diagonal of dY V^T, block `wave`
            const bf16x8 vh = ld_row_plain(sm + L::VT0, L::OS, 16 * wave + l16, 0, q4);
            const bf16x8 yh = v_col(L::Y0, 0, wave), yl = v_col(L::Y0, 1, wave);
            yv = mfma_bf16(yh, vh, yv);
            yv = mfma_bf16(yl, vh, yv);
            if constexpr (NP == 2) yv = mfma_bf16(yh, ld_row_plain(sm + L::VT0 + L::OT, L::OS, 16 * wave + l16, 0, q4), yv);
        }
        __syncthreads();
    }
    if (wave < 4 && l16 >> 2 == q4)  // row 4 q4 + e = column l16
        *reinterpret_cast<float *>(sm + L::YV + 4 * (16 * wave + l16)) = l16 & 2 ? (l16 & 1 ? yv[3] : yv[2]) : (l16 & 1 ? yv[1] : yv[0]);

    // score gradients: the same tiles of Q K^T and K K^T, decayed
    const float *vec = reinterpret_cast<const float *>(sm + L::VEC);
    float *E = reinterpret_cast<float *>(sm + L::E0);
    float *rowsum = reinterpret_cast<float *>(sm + L::ROW);
    auto st_plane = [&](int base, int row, int col, float x) {
        const __bf16 h = (__bf16)x, l = (__bf16)(x - (float)h);
        lds_st(sm, base + row * PSTR + 2 * col, h);
        lds_st(sm, base + L::PLANE + row * PSTR + 2 * col, l);
    };
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
        const int id = wave + NW * i;
        if (id < 10) {
            int br, bc;
            tri(id, br, bc);
            f32x4 kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const bf16x8 b = ld_row_plain(sm + L::K0, L::RS, 16 * bc + l16, 32 * j, q4);
                const bf16x8 ka = ld_row_plain(sm + L::K0, L::RS, 16 * br + l16, 32 * j, q4);
                const bf16x8 qa = ld_row_plain(sm + L::Q0, L::RS, 16 * br + l16, 32 * j, q4);
                kk = mfma_bf16(ka, b, kk);
                qk = mfma_bf16(qa, b, qk);
                if constexpr (NP == 2) {
                    const bf16x8 b2 = ld_row_plain(sm + L::K0 + L::TILE, L::RS, 16 * bc + l16, 32 * j, q4);
                    kk = mfma_bf16(ka, b2, kk);
                    qk = mfma_bf16(qa, b2, qk);
                    kk = mfma_bf16(ld_row_plain(sm + L::K0 + L::TILE, L::RS, 16 * br + l16, 32 * j, q4), b, kk);
                    qk = mfma_bf16(ld_row_plain(sm + L::Q0 + L::TILE, L::RS, 16 * br + l16, 32 * j, q4), b, qk);
                }
            }
            const int s = 16 * bc + l16;
            const float gsh = vec[DeltaRecord::GH * 64 + s], gsl = vec[DeltaRecord::GL * 64 + s];
            f32x4 rs;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 16 * br + 4 * q4 + e;
                const float d = ex2(fminf((vec[DeltaRecord::GH * 64 + r] - gsh) + (vec[DeltaRecord::GL * 64 + r] - gsl), 0.0f));
                const float dp = s <= r ? p.scale * d * ou[i][e] : 0.0f;
                const float yd = s < r ? d * yu[i][e] : 0.0f;
                const float da = -vec[DeltaRecord::BT * 64 + r] * yd;
                rs[e] = sum16(yd * kk[e]);
                E[r * L::ES + s] = s < r ? dp * qk[e] + da * kk[e] : 0.0f;
                st_plane(L::DP0, r, s, dp);
                if (s <= r) st_plane(L::DA0, r, s, da);  // zero on the diagonal
                if (s < r) st_plane(L::DA0, s, r, da);
            }
            if (l16 == 0) *reinterpret_cast<f32x4 *>(rowsum + bc * 64 + 16 * br + 4 * q4) = rs;
            if (br == bc && !(br & 1)) {  // the zero block right of it
#pragma unroll
                for (int e = 0; e < 4; ++e) st_plane(L::DP0, 16 * br + 4 * q4 + e, 16 * (br + 1) + l16, 0.0f);
            }
        }
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
    if (lane == 0) *reinterpret_cast<float *>(sm + L::DOT + 4 * wave) = dot;
    __syncthreads();

    // dQ and dK of this wave's key columns, and their rows' products with q and k
    const int kc = 16 * wave + l16;
    const int64_t w0 = (t0 * p.HV + hv) * D + kc;                     // per value head (float32)
    const int64_t o0 = (t0 * p.H + hk) * D + kc;
    const bool grouped = p.H != p.HV;
    float *red = reinterpret_cast<float *>(sm + L::RED) + wave * 192;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
        auto vec4 = [&](int which) { return lds_ld<f32x4>(sm, L::VEC + which * 256 + (16 * mt + 4 * q4) * 4); };
        const f32x4 eg = vec4(DeltaRecord::EG), bt = vec4(DeltaRecord::BT);
        f32x4 dq = aq[mt] * vec4(DeltaRecord::EQ), y = ay[mt] * eg, x = au[mt] * vec4(DeltaRecord::ED);
        f32x4 si, sy, sx;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 16 * mt + 4 * q4 + e;
            const int o = r * L::RS + 2 * kc;
            float qv = bf16_bits_to_f32(lds_ld<uint16_t>(sm, L::Q0 + o)), kv = bf16_bits_to_f32(lds_ld<uint16_t>(sm, L::K0 + o));
            if constexpr (NP == 2) {
                qv += bf16_bits_to_f32(lds_ld<uint16_t>(sm, L::Q0 + L::TILE + o));
                kv += bf16_bits_to_f32(lds_ld<uint16_t>(sm, L::K0 + L::TILE + o));
            }
            si[e] = sum16(qv * dq[e]);
            sy[e] = sum16(kv * y[e]);
            sx[e] = sum16(kv * x[e]);
        }
        if (l16 == 0) {
            *reinterpret_cast<f32x4 *>(red + 16 * mt + 4 * q4) = si;
            *reinterpret_cast<f32x4 *>(red + 64 + 16 * mt + 4 * q4) = sy;
            *reinterpret_cast<f32x4 *>(red + 128 + 16 * mt + 4 * q4) = sx;
        }
        f32x4 dk = x - bt * y;
        auto part2 = [&](int base, int j, int which) {  // right operand: rows 32 j .. of K or Q, the wave's columns
            return ld_col(sm + base + which * L::TILE, L::RS, 32 * j, 16 * wave, q4, l16);
        };
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const bf16x8 k0 = part2(L::K0, j, 0), q0 = part2(L::Q0, j, 0);
            bf16x8 k1 = k0, q1 = q0;
            if constexpr (NP == 2) {
                k1 = part2(L::K0, j, 1);
                q1 = part2(L::Q0, j, 1);
            }
            auto add = [&](bf16x8 ah, bf16x8 al, bf16x8 bh, bf16x8 bl, f32x4 acc) {
                acc = mfma_bf16(ah, bh, acc);
                acc = mfma_bf16(al, bh, acc);
                if constexpr (NP == 2) acc = mfma_bf16(ah, bl, acc);
                return acc;
            };
            if (j <= mt / 2)
                dq = add(ld_row(sm + L::DP0, PSTR, 16 * mt + l16, 32 * j, q4),
                         ld_row(sm + L::DP0 + L::PLANE, PSTR, 16 * mt + l16, 32 * j, q4), k0, k1, dq);
            if (j >= mt / 2)
                dk = add(ld_col(sm + L::DP0, PSTR, 32 * j, 16 * mt, q4, l16),
                         ld_col(sm + L::DP0 + L::PLANE, PSTR, 32 * j, 16 * mt, q4, l16), q0, q1, dk);
            dk = add(ld_row(sm + L::DA0, PSTR, 16 * mt + l16, 32 * j, q4),
                     ld_row(sm + L::DA0 + L::PLANE, PSTR, 16 * mt + l16, 32 * j, q4), k0, k1, dk);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 16 * mt + 4 * q4 + e;
            if (r < len) {
                if (grouped) {
                    p.dq_ws[w0 + (int64_t)r * p.HV * D] = dq[e];
                    p.dk_ws[w0 + (int64_t)r * p.HV * D] = dk[e];
                } else {
                    p.dq[o0 + (int64_t)r * p.H * D] = f32_io<IO>(dq[e]);
                    p.dk[o0 + (int64_t)r * p.H * D] = f32_io<IO>(dk[e]);
                }
            }
        }
    }
    __syncthreads();
    if (wave != 0) return;

    // the scalars: lane = token
    float I = 0.0f, Y = 0.0f, X = 0.0f, sd = 0.0f, rs = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const float *r = reinterpret_cast<const float *>(sm + L::RED) + w * 192;
        I += r[lane];
        Y += r[64 + lane];
        X += r[128 + lane];
        sd += lds_ld<float>(sm, L::DOT + 4 * w);
    }
    for (int b = 0; b <= lane >> 4; ++b) rs += rowsum[b * 64 + lane];
    const float bt = vec[DeltaRecord::BT * 64 + lane];
    const float dbeta = lds_ld<float>(sm, L::YV + 4 * lane) - Y - rs;
    I -= bt * Y;
    // row `lane` of E to sums over the columns before each
    float run = 0.0f;
    for (int s = 0; s <= lane; ++s) {
        const float x = E[lane * L::ES + s];
        E[lane * L::ES + s] = run;
        run += x;
    }
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    float pairs = 0.0f;
    for (int r = 0; r < 64; ++r)
        if (r >= lane) pairs += E[r * L::ES + lane];
    float Isum = I, Xsum = X;  // suffix sum of I, inclusive prefix of X
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const float a = __shfl_down(Isum, d), b = __shfl_up(Xsum, d);
        if (lane + d < 64) Isum += a;
        if (lane >= d) Xsum += b;
    }
    const float xb = __shfl_up(Xsum, 1);
    const float dg = pairs + Isum + (lane > 0 ? xb : 0.0f) + vec[DeltaRecord::NVEC * 64] * sd;
    if (lane < len) {
        const int64_t o = (t0 + lane) * p.HV + hv;
        p.dbeta[o] = f32_io<IO>(dbeta);
        if (p.gtype == G_F32) static_cast<float *>(p.dg)[o] = dg;
        else static_cast<uint16_t *>(p.dg)[o] = p.gtype == G_F16 ? f32_io<IO_F16>(dg) : f32_io<IO_BF16>(dg);
    }
}

}  // namespace

template <int K, int IO>
static void launch_bwd_state_cols(const DeltaParams &p, int cols, hipStream_t stream)
{
    const dim3 grid((unsigned)((int64_t)p.N * p.HV * (p.V / cols)));
    if (cols == 128) {
        // (K = V: 128 columns only with 128 key rows)
        if constexpr (K == 128) hipLaunchKernelGGL((delta_bwd_state_kernel<K, IO, 8>), grid, dim3(64 * (8 + LW)), 0, stream, p);
    } else if (cols == 64) {
        hipLaunchKernelGGL((delta_bwd_state_kernel<K, IO, 4>), grid, dim3(64 * (4 + LW)), 0, stream, p);
    } else {
        hipLaunchKernelGGL((delta_bwd_state_kernel<K, IO, 2>), grid, dim3(64 * (2 + LW)), 0, stream, p);
    }
}

hipError_t launch_delta_bwd_state(const DeltaParams &p, int ncu, hipStream_t stream)
{
    const int cols = delta_columns(p, ncu);
    if (p.K == 128) {
        if (p.io == IO_F16) launch_bwd_state_cols<128, IO_F16>(p, cols, stream);
        else launch_bwd_state_cols<128, IO_BF16>(p, cols, stream);
    } else {
        if (p.io == IO_F16) launch_bwd_state_cols<64, IO_F16>(p, cols, stream);
        else launch_bwd_state_cols<64, IO_BF16>(p, cols, stream);
    }
    return hipGetLastError();
}

hipError_t launch_delta_bwd_grad(const DeltaParams &p, hipStream_t stream)
{
    if (p.T == 0) return hipSuccess;
    const dim3 grid((unsigned)((int64_t)p.nslots * p.HV));
    if (p.K == 128) {
        if (p.io == IO_F16) hipLaunchKernelGGL((delta_bwd_grad_kernel<128, IO_F16>), grid, dim3(512), 0, stream, p);
        else hipLaunchKernelGGL((delta_bwd_grad_kernel<128, IO_BF16>), grid, dim3(512), 0, stream, p);
    } else {
        if (p.io == IO_F16) hipLaunchKernelGGL((delta_bwd_grad_kernel<64, IO_F16>), grid, dim3(256), 0, stream, p);
        else hipLaunchKernelGGL((delta_bwd_grad_kernel<64, IO_BF16>), grid, dim3(256), 0, stream, p);
    }
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (p.H == p.HV) return hipSuccess;
    BwdParams r{};
    r.T = p.T;
    r.H = p.H;
    r.HV = p.HV;
    r.K = p.K;
    r.io = p.io;
    r.dq_ws = p.dq_ws;
    r.dk_ws = p.dk_ws;
    r.dq = p.dq;
    r.dk = p.dk;
    return launch_bwd_reduce(r, stream);
}

}  // namespace gdn2
