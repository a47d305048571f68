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

#include <hip/hip_runtime.h>

#include "gdn2_delta_device.h"

namespace gdn2 {
namespace {

using namespace dev;

// ----------------------------------------------------- reverse sequential --
template <int K, int NP, int NW>
struct BwdStateLds {
    static constexpr int RS = 2 * K + 16;
    static constexpr int TILE = 64 * RS;
    static constexpr int K0 = 0, Q0 = NP * TILE;
    static constexpr int PLANE = DeltaRecord::PLANE;
    static constexpr int P0 = 2 * NP * TILE;
    static constexpr int V0 = P0 + 4 * PLANE;
    static constexpr int SIZE = V0 + DeltaRecord::NVEC * 256 + 16;
};

template <int K, int IO, int NW>
__global__ __launch_bounds__(64 * NW) void delta_bwd_state_kernel(DeltaParams p)
{
    constexpr int NP = IO == IO_F16 ? 2 : 1;
    using L = BwdStateLds<K, NP, NW>;
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

    f32x4 dS[KT];
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) dS[i][e] = p.dht ? p.dht[shead + (int64_t)(16 * i + 4 * q4 + e) * p.V + col] : 0.0f;

    constexpr int CPT = 64 * K / 8 / NT;
    constexpr int RCH = 4 * DeltaRecord::PLANE / 16, RPT = (RCH + NT - 1) / NT;
    constexpr int VCH = DeltaRecord::NVEC * 16 + 1;
    static_assert(NT >= VCH, "one vector chunk per thread");
    i32x4 fk[CPT], fq[CPT], fr[RPT], fv;
    uint16_t vv[16], oo[16];

    auto fetch = [&](int64_t c) {
        const int64_t t0 = rng.b + c * CHUNK;
        const int len = (int)(rng.e - t0 < CHUNK ? rng.e - t0 : CHUNK);
        const __amdgpu_buffer_rsrc_t rk = buf_rsrc(p.k + t0 * p.sk + hk * p.hsk, (int)(((len - 1) * p.sk + K) * 2));
        const __amdgpu_buffer_rsrc_t rq = buf_rsrc(p.q + t0 * p.sq + hk * p.hsq, (int)(((len - 1) * p.sq + K) * 2));
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int ci = t + NT * i, row = ci / (K / 8), cc = ci % (K / 8);
            fk[i] = buf_ld16<i32x4>(rk, (uint32_t)(row * (int)p.sk + cc * 8) * 2);
            fq[i] = buf_ld16<i32x4>(rq, (uint32_t)(row * (int)p.sq + cc * 8) * 2);
        }
        const char *rec = p.rec + delta_item(p, slot0 + c, hv) * (int64_t)DeltaRecord::BYTES;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int id = t + NT * i;
            if (RCH % NT == 0 || id < RCH) fr[i] = *reinterpret_cast<const i32x4 *>(rec + 16 * id);
        }
        if (t < VCH) fv = *reinterpret_cast<const i32x4 *>(rec + DeltaRecord::VEC + 16 * t);
        const int bytes = (int)(((len - 1) * p.sv + p.V) * 2);
        const __amdgpu_buffer_rsrc_t rv = buf_rsrc(p.v + t0 * p.sv + hv * p.hsv, bytes);
        const __amdgpu_buffer_rsrc_t ro = buf_rsrc(p.dout + t0 * p.sv + hv * p.hsv, bytes);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t off = (uint32_t)((16 * (i >> 2) + 4 * q4 + (i & 3)) * (int)p.sv + col) * 2;
            vv[i] = __builtin_amdgcn_raw_buffer_load_b16(rv, off, 0, 0);
            oo[i] = __builtin_amdgcn_raw_buffer_load_b16(ro, off, 0, 0);
        }
    };
    auto stage = [&]() {
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int ci = t + NT * i, row = ci / (K / 8), cc = ci % (K / 8);
            st_parts<NP>(sm + L::K0, L::TILE, row * L::RS + cc * 16, fk[i]);
            st_parts<NP>(sm + L::Q0, L::TILE, row * L::RS + cc * 16, fq[i]);
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int id = t + NT * i;
            if (RCH % NT == 0 || id < RCH) {
                lds_st(sm, L::P0 + 16 * id, fr[i]);
            }
        }
        if (t < VCH) lds_st(sm, L::V0 + 16 * t, fv);
    };

    if (nch > 0) fetch(nch - 1);
    for (int64_t c = nch - 1; c >= 0; --c) {
        const int64_t t0 = rng.b + c * CHUNK;
        const int len = (int)(rng.e - t0 < CHUNK ? rng.e - t0 : CHUNK);
        float v32[16];
        f32x4 dO[4];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            v32[i] = io_f32<IO>(vv[i]);
            dO[i >> 2][i & 3] = io_f32<IO>(oo[i]);
        }
        stage();
        __syncthreads();
        if (c > 0) fetch(c - 1);

        const int64_t frag = delta_item(p, slot0 + c, hv) * (p.V / 16) + (vb * NW + wave);
        auto vec4 = [&](int which, int mt) { return lds_ld<f32x4>(sm, L::V0 + which * 256 + (16 * mt + 4 * q4) * 4); };
        const float gamma = lds_ld<float>(sm, L::V0 + DeltaRecord::NVEC * 256);
        {
            f32x4 *dst = reinterpret_cast<f32x4 *>(p.ds_ck) + frag * (KT * 64) + lane;
#pragma unroll
            for (int i = 0; i < KT; ++i) dst[64 * i] = dS[i];
        }
        bf16x8 Sh[KS], Sl[KS];
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            bf16x4 h0, l0, h1, l1;
            split4(dS[2 * j], h0, l0);
            split4(dS[2 * j + 1], h1, l1);
            Sh[j] = cat4(h0, h1);
            Sl[j] = cat4(l0, l1);
        }
        bf16x8 Oh[2], Ol[2];  // dO as a right operand (one part when it is bf16)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            bf16x4 h0, l0, h1, l1;
            split4(dO[2 * j], h0, l0);
            split4(dO[2 * j + 1], h1, l1);
            Oh[j] = cat4(h0, h1);
            Ol[j] = cat4(l0, l1);
        }
        // dU = P^T dO + e^(G_C - G) (K dS)
        bf16x8 Uh[2], Ul[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            bf16x4 h[2], l[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int mt = 2 * j + i;
                f32x4 u = {0, 0, 0, 0};
#pragma unroll
                for (int jj = 0; jj < KS; ++jj) {
                    const bf16x8 a = ld_row(sm + L::K0, L::RS, 16 * mt + l16, 32 * jj, q4);
                    bf16x8 al = a;
                    if constexpr (NP == 2) al = ld_row(sm + L::K0 + L::TILE, L::RS, 16 * mt + l16, 32 * jj, q4);
                    u = mfma_split<NP == 2>(a, al, Sh[jj], Sl[jj], u);
                }
                u *= vec4(DeltaRecord::ED, mt);
#pragma unroll
                for (int jj = j; jj < 2; ++jj) {
                    const bf16x8 ph = ld_frag_t(sm + L::P0 + 2 * L::PLANE, mt, jj, q4, l16);
                    const bf16x8 pl = ld_frag_t(sm + L::P0 + 3 * L::PLANE, mt, jj, q4, l16);
                    u = mfma_bf16(ph, Oh[jj], u);
                    if constexpr (NP == 2) u = mfma_bf16(ph, Ol[jj], u);
                    u = mfma_bf16(pl, Oh[jj], u);
                }
                split4(u, h[i], l[i]);
            }
            Uh[j] = cat4(h[0], h[1]);
            Ul[j] = cat4(l[0], l[1]);
        }
        // dY = T^T dU, dV = beta dY; the right operands e^G dV (negated) and scale e^G dO
        bf16x8 Eh[2], El[2], Fh[2], Fl[2];
        const __amdgpu_buffer_rsrc_t rdv = buf_rsrc(p.dv + t0 * p.sv + hv * p.hsv, (int)(((len - 1) * p.sv + p.V) * 2));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            bf16x4 h[2], l[2], fh[2], fl[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int mt = 2 * j + i;
                f32x4 y = {0, 0, 0, 0};
#pragma unroll
                for (int jj = j; jj < 2; ++jj)
                    y = mfma_split<true>(ld_frag_t(sm + L::P0, mt, jj, q4, l16),
                                         ld_frag_t(sm + L::P0 + L::PLANE, mt, jj, q4, l16), Uh[jj], Ul[jj], y);
                reinterpret_cast<f32x4 *>(p.y_ck)[frag * 256 + 64 * mt + lane] = y;
                const f32x4 dv = y * vec4(DeltaRecord::BT, mt), eg = vec4(DeltaRecord::EG, mt), eq = vec4(DeltaRecord::EQ, mt);
                f32x4 yv;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    __builtin_amdgcn_raw_buffer_store_b16(f32_io<IO>(dv[e]), rdv, (uint32_t)((16 * mt + 4 * q4 + e) * (int)p.sv + col) * 2, 0, 0);
                    yv[e] = sum16(y[e] * v32[4 * mt + e]);
                }
                if (l16 == 0) *reinterpret_cast<f32x4 *>(p.yv + frag * 64 + 16 * mt + 4 * q4) = yv;
                split4(-(eg * dv), h[i], l[i]);
                split4(eq * dO[mt], fh[i], fl[i]);
            }
            Eh[j] = cat4(h[0], h[1]);
            El[j] = cat4(l[0], l[1]);
            Fh[j] = cat4(fh[0], fh[1]);
            Fl[j] = cat4(fl[0], fl[1]);
        }
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            f32x4 s = dS[i] * gamma;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bf16x8 a = ld_col(sm + L::K0, L::RS, 32 * j, 16 * i, q4, l16);
                const bf16x8 b = ld_col(sm + L::Q0, L::RS, 32 * j, 16 * i, q4, l16);
                bf16x8 al = a, bl = b;
                if constexpr (NP == 2) {
                    al = ld_col(sm + L::K0 + L::TILE, L::RS, 32 * j, 16 * i, q4, l16);
                    bl = ld_col(sm + L::Q0 + L::TILE, L::RS, 32 * j, 16 * i, q4, l16);
                }
                s = mfma_split<NP == 2>(a, al, Eh[j], El[j], s);
                s = mfma_split<NP == 2>(b, bl, Fh[j], Fl[j], s);
            }
            dS[i] = s;
        }
        __syncthreads();
    }
    if (p.dh0)
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) p.dh0[shead + (int64_t)(16 * i + 4 * q4 + e) * p.V + col] = dS[i][e];
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
    static constexpr int O0 = W0;
    static constexpr int VP = 32 * PSTR;      // a plane of U or dY: [v][64 tokens]
    static constexpr int U0 = O0 + NP * OT, Y0 = U0 + 2 * VP;
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
    static constexpr int DOT = ROW + 4 * 256;                       // [wave]
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
    const f32x4 *s_ck = reinterpret_cast<const f32x4 *>(p.s_ck) + item * (D / 16) * (D / 16 * 64);
    const f32x4 *ds_ck = reinterpret_cast<const f32x4 *>(p.ds_ck) + item * (D / 16) * (D / 16 * 64);
    const f32x4 *u_ck = reinterpret_cast<const f32x4 *>(p.u_ck) + item * (D / 16) * 256;
    const f32x4 *y_ck = reinterpret_cast<const f32x4 *>(p.y_ck) + item * (D / 16) * 256;

    // fragments of a block of 32 value columns: 2 (D / 16) 64 of S and dS, 512 of U and dY
    constexpr int SPT = 2 * (D / 16) * 64 / NT;  // 2
    constexpr int UPT = 512 / NT;                // 1 (D = 128), 2 (D = 64)
    f32x4 fs[SPT], fd[SPT], fu[UPT], fy[UPT];
    i32x4 fo;
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
        if (t < 256) fo = buf_ld16<i32x4>(ro, (uint32_t)((t >> 2) * (int)p.sv + vb * 32 + (t & 3) * 8) * 2);
    };
    auto st_frag = [&](int base, int plane, int stride, f32x4 x, int id, int tiles) {
        // fragment id -> (16 columns, tile, lane): 4 consecutive rows of one value column
        const int ln = id & 63, tile = (id >> 6) % tiles, v = (id >> 6) / tiles * 16 + (ln & 15), r = 16 * tile + 4 * (ln >> 4);
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
    float dot = 0.0f;  // <S, dS>
    fetch(0);
    for (int vb = 0; vb < D / 32; ++vb) {
#pragma unroll
        for (int i = 0; i < SPT; ++i) {
            st_frag(L::S0, L::SP, L::RS, fs[i], t + NT * i, D / 16);
            st_frag(L::DS0, L::SP, L::RS, fd[i], t + NT * i, D / 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) dot = fmaf(fs[i][e], fd[i][e], dot);
        }
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            st_frag(L::U0, L::VP, PSTR, fu[i], t + NT * i, 4);
            st_frag(L::Y0, L::VP, PSTR, fy[i], t + NT * i, 4);
        }
        if (t < 256) st_parts<NP>(sm + L::O0, L::OT, (t >> 2) * L::OS + (t & 3) * 16, fo);
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
        __syncthreads();
    }

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
    float I = 0.0f, Y = 0.0f, X = 0.0f, sd = 0.0f, yv = 0.0f, rs = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const float *r = reinterpret_cast<const float *>(sm + L::RED) + w * 192;
        I += r[lane];
        Y += r[64 + lane];
        X += r[128 + lane];
        sd += lds_ld<float>(sm, L::DOT + 4 * w);
        yv += p.yv[(item * NW + w) * 64 + lane];
    }
    for (int b = 0; b <= lane >> 4; ++b) rs += rowsum[b * 64 + lane];
    const float bt = vec[DeltaRecord::BT * 64 + lane];
    const float dbeta = yv - Y - rs;
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

hipError_t launch_delta_bwd_state(const DeltaParams &p, int ncu, hipStream_t stream)
{
    (void)ncu;
    const dim3 grid((unsigned)((int64_t)p.N * p.HV * (p.V / 64)));
    if (p.K == 128) {
        if (p.io == IO_F16) hipLaunchKernelGGL((delta_bwd_state_kernel<128, IO_F16, 4>), grid, dim3(256), 0, stream, p);
        else hipLaunchKernelGGL((delta_bwd_state_kernel<128, IO_BF16, 4>), grid, dim3(256), 0, stream, p);
    } else {
        if (p.io == IO_F16) hipLaunchKernelGGL((delta_bwd_state_kernel<64, IO_F16, 4>), grid, dim3(256), 0, stream, p);
        else hipLaunchKernelGGL((delta_bwd_state_kernel<64, IO_BF16, 4>), grid, dim3(256), 0, stream, p);
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
