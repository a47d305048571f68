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
// Bound by HBM with many chains: 190 KiB per item, of which dS and dY, 96 KiB,
// are left for the gradients (8 sequences, 36,962 tokens, 32 heads: 775 us,
// 4.6 TB/s; the checkpoints of the forward's pass, 140 KiB per item, 535 us).
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
    __device__ static __forceinline__ i32x4 col(const char *plane, int i, int j, int q4, int l16)
    {
        const int a = quad(4 * q4 + (l16 >> 2), 4 * (i & 1) + (l16 & 3)) + i / 2 * 2048 + 32 * 64 * j;
        return __builtin_bit_cast(i32x4, cat4(lds_tr(plane, a), lds_tr(plane, a + 16 * 64)));
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
    static constexpr int VCH = (DeltaRecord::SCAL + 16 - DeltaRecord::VEC) / 16;
    static constexpr int HALF = (G0 + 16 * VCH + 511) / 512 * 512;
    static constexpr int SIZE = 2 * HALF;
};

// A split run's segments are entered from their ends: SEG walks those but the
// first, the last from the given gradient and the others from zero, and
// leaves what comes out of each (rseg); the transition of the gradient over a
// segment is the state's transposed.
template <int K, int IO, int NC, int MODE>
__global__ __launch_bounds__(64 * (NC + LW)) void delta_bwd_state_kernel(DeltaParams p)
{
    constexpr int COLS = 16 * NC;
    using L = BwdStateLds<K, COLS>;
    using TL = Tile<K>;
    constexpr int KT = K / 16, KS = K / 32;
    __shared__ __attribute__((aligned(16))) char sm[L::SIZE];
    const int nvb = p.V / COLS;
    const int nseg = MODE == SEG ? p.nseg - 1 : MODE == JOIN ? p.nseg : 1;
    const Chain chain = chain_of(p, nvb * nseg);
    const int vb = chain.part % nvb, hv = chain.hv, n = chain.n;
    const int seg = chain.part / nvb + (MODE == SEG ? 1 : 0);
    const bool last = MODE == OUT || seg == p.nseg - 1;
    const int hk = hv / (p.HV / p.H);
    SeqRange rng = chain.rng;
    int64_t nch = chunks_of(rng);
    int64_t slot0 = chunk_slot(rng.b, n, 0);
    if constexpr (MODE != OUT) segment_of(p.nseg, seg, rng, nch, slot0);
    // where a split run keeps what enters segment s - 1 from its end: at s - 1
    float *rseg = MODE == OUT ? nullptr : p.rseg + ((int64_t)n * p.HV + hv) * (p.nseg - 1) * K * p.V;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;

    if (wave >= NC) {
        const int t = threadIdx.x - 64 * NC;
        constexpr int TH = 64 * LW;
        constexpr int CPT = 64 * K / 8 / TH;
        constexpr int OCH = 64 * COLS / 8, OPT = (OCH + TH - 1) / TH;
        constexpr int RPT = 4 * DeltaRecord::PLANE / 16 / TH;  // 6
        static_assert(L::VCH <= TH && 4 * DeltaRecord::PLANE == 16 * RPT * TH, "pieces per thread");
        i32x4 fk[CPT], fq[CPT], fo[OPT], fr[RPT], fv;
        float ck[CPT], cq[CPT];  // the rows' powers of two
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
            if constexpr (IO == IO_BF16) {
                const float *v2 = reinterpret_cast<const float *>(rec + DeltaRecord::VEC2);
#pragma unroll
                for (int i = 0; i < CPT; ++i) {
                    ck[i] = v2[DeltaRecord::CK * 64 + (t + TH * i) / (K / 8)];
                    cq[i] = v2[DeltaRecord::CQ * 64 + (t + TH * i) / (K / 8)];
                }
            }
#pragma unroll
            for (int i = 0; i < RPT; ++i) fr[i] = *reinterpret_cast<const i32x4 *>(rec + 16 * (t + TH * i));
            if (t < L::VCH) fv = *reinterpret_cast<const i32x4 *>(rec + DeltaRecord::VEC + 16 * t);
        };
        auto stage = [&](char *half) {
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                const int ci = t + TH * i, row = ci / (K / 8), cc = ci % (K / 8);
                lds_st(half, L::K0 + TL::piece(row, cc), row_f16<IO>(fk[i], ck[i]));
                lds_st(half, L::Q0 + TL::piece(row, cc), row_f16<IO>(fq[i], cq[i]));
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
            if constexpr (MODE != SEG)
                if (c + 1 < nch) flush(c + 1);
            if (c > 0) stage(sm + ((c - 1) & 1) * L::HALF);
            if (c > 1) fetch(c - 2);
            __syncthreads();
        }
        if constexpr (MODE != SEG)
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
        for (int e = 0; e < 4; ++e) {
            const int64_t o = (int64_t)(state_row(i, q4) + e) * p.V + col;
            dS[i][e] = !last ? (MODE == JOIN ? rseg[(int64_t)seg * K * p.V + o] : 0.0f) : p.dht ? p.dht[shead + o] : 0.0f;
        }
    RightOp<KS> So;
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
        const f32x4 scal = lds_ld<f32x4>(half, L::G0 + DeltaRecord::SCAL - DeltaRecord::VEC);  // e^(G_C), 1 / scales of T and P
        const float gamma = scal[0];
        if constexpr (MODE != SEG) {
            f32x4 *dst = reinterpret_cast<f32x4 *>(p.ds_ck) + frag * (KT * 64) + lane;
#pragma unroll
            for (int i = 0; i < KT; ++i) dst[64 * i] = dS[i];
        }
        const float smax = So.mx;
        constexpr f32x4 zero = {0, 0, 0, 0};
        // dU = e^(G_C - G) (K dS) + P^T dO
        f32x4 U[4] = {zero, zero, zero, zero}, Y[4] = {zero, zero, zero, zero}, x4[4], dO[4];
        i32x4 a[4], b[4];
#pragma unroll
        for (int j = 0; j < KS; ++j) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) a[mt] = TL::row(KL, mt, j, q4, l16);
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) U[mt] = So.mul1(a[mt], j, part, U[mt]);
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
            dO[mt] = io4_f32<IO>(lds_tr(half, L::O0 + (16 * mt + 4 * q4 + (l16 >> 2)) * L::OS + 2 * (16 * wave + 4 * (l16 & 3))));
        RightOp<2, 1> Oo;  // (16-bit values: one part is all of them)
        Oo.set(dO);
        // y += (plane pair)^T op
        auto upper = [&](const char *plane, const auto &op, int parts, f32x4 (&y)[4]) {
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const int top = jj ? 4 : 2;
#pragma unroll
                for (int mt = 0; mt < top; ++mt) {
                    a[mt] = PlaneTile::col(plane, mt, jj, q4, l16);
                    b[mt] = PlaneTile::col(plane + PlaneTile::BYTES, mt, jj, q4, l16);
                }
#pragma unroll
                for (int mt = 0; mt < top; ++mt) y[mt] = op.mul1(a[mt], jj, 0, y[mt]);
#pragma unroll
                for (int mt = 0; mt < top; ++mt) y[mt] = op.mul1(b[mt], jj, 0, y[mt]);
                if (parts == 2)
#pragma unroll
                    for (int mt = 0; mt < top; ++mt) y[mt] = op.mul1(a[mt], jj, 1, y[mt]);
            }
        };
        upper(PH, Oo, 1, Y);
        vec(DeltaRecord::ED, x4);
        const float pinv = Oo.inv * scal[2];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            U[mt] = U[mt] * (x4[mt] * So.inv) + Y[mt] * pinv;
            Y[mt] = zero;
        }
        // dY = T^T dU
        {
            RightOp<2> Uo;
            Uo.set(U);
            upper(TH, Uo, 2, Y);
            const float tinv = Uo.inv * scal[1];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) Y[mt] *= tinv;
        }
        if constexpr (MODE != SEG) {
            const f32x4 m = {max16(smax), max16(col_max(Y)), max16(Oo.mx), 0.0f};
            if (lane == 0) *reinterpret_cast<f32x4 *>(p.mx + frag * 8 + 4) = m;
        }
        // dS <- e^(G_C) dS + tile^T x
        auto add_outer = [&](const char *tile, const f32x4 (&x)[4], float g) {
            RightOp<2> op;
            op.set(x);
#pragma unroll
            for (int i0 = 0; i0 < KT; i0 += 4) {
                f32x4 s[4] = {zero, zero, zero, zero};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = TL::col(tile, i0 + i, j, q4, l16);
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[i] = op.mul1(a[i], j, part, s[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) dS[i0 + i] = dS[i0 + i] * g + s[i] * op.inv;
            }
        };
        vec(DeltaRecord::EQ, x4);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) dO[mt] *= x4[mt];
        add_outer(QL, dO, gamma);  // scale e^G dO
        // dV = beta dY, left where this wave's columns of dO were, and -e^G dV
        vec(DeltaRecord::BT, x4);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            if constexpr (MODE != SEG) reinterpret_cast<f32x4 *>(p.y_ck)[frag * 256 + 64 * mt + lane] = Y[mt];
            Y[mt] *= x4[mt];
            if constexpr (MODE != SEG) st_rows16<IO>(half + L::O0 + (16 * mt + 4 * q4) * L::OS + 32 * wave, L::OS, Y[mt], l16);
        }
        vec(DeltaRecord::EG, x4);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) Y[mt] *= -x4[mt];
        add_outer(KL, Y, 1.0f);
        So.set(dS);
        __syncthreads();
    }
    float *dst = MODE == SEG ? rseg + (int64_t)(seg - 1) * K * p.V : p.dh0 && seg == 0 ? p.dh0 + shead : nullptr;
    if (dst)
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[(int64_t)(state_row(i, q4) + e) * p.V + col] = dS[i][e];
}

// --------------------------------------------------------- all gradients --
// One workgroup of D / 16 waves per (chunk, value head) (K = V = D). The
// products that contract the value dimension run over 32 columns at a time,
// staged value-major ([v][k] and [v][token], as the checkpoints' fragments
// hold them); wave w owns key columns 16 w .. 16 w + 15 of dQ and dK and
// every (D / 16)-th 16x16 tile of the two score gradients, computed
// transposed: a lane then holds four columns of one row r. All operands are
// fp16 parts under one power of two per operand and chunk (the sequential
// passes leave the largest magnitudes). Two workgroups share a compute unit
// and hide each other's loads; one with the next block's loads in registers
// took three tenths longer. Bound by HBM, 310 KiB per item at 4.2 TB/s (8
// sequences, 36,962 tokens, 32 heads: 1.40 ms), and by the loads' latency in
// what is left of the copy rate.

// 32 rows (v) of C 16-bit values, written 8 bytes at a time down 16 rows and
// read transposed from 4 rows and the 4 rows 8 further on: pieces of 16 bytes
// permuted by the row, their halves by the piece, both without conflicts.
template <int C>
struct ValueTile {
    static constexpr int BYTES = 64 * C;
    __device__ static __forceinline__ int swz(int r)
    {
        return C == 128 ? (r >> 3 & 1) << 3 | (r & 3) << 1 | (r >> 2 & 1) : (r >> 1 & 1) << 2 | (r >> 3 & 1) << 1 | (r >> 2 & 1);
    }
    // byte offset of the four columns 4 c .. of row r
    __device__ static __forceinline__ int quad(int r, int c)
    {
        return r * 2 * C + (((c >> 1) ^ swz(r)) << 4) + 8 * ((c ^ c >> 1) & 1);
    }
    // transposed: element (m, k) = tile[k][m], rows k = 8 q4 .., columns m = 16 w + l16
    __device__ static __forceinline__ i32x4 col(const char *tile, int w, int q4, int l16)
    {
        const int r = 8 * q4 + (l16 >> 2), c = 4 * w + (l16 & 3);
        return __builtin_bit_cast(i32x4, cat4(lds_tr(tile, quad(r, c)), lds_tr(tile, quad(r + 4, c))));
    }
};
// 64 rows (tokens) of 32 16-bit values: 16-byte piece c of row r.
__device__ __forceinline__ int token_piece(int r, int c) { return r * 64 + ((c ^ (r >> 2 & 3)) << 4); }

template <int D>
struct GradLds {
    // the block of 32 value columns
    static constexpr int OT = 64 * 64;        // dO or V
    static constexpr int O0 = 0, VT0 = OT;
    static constexpr int VP = ValueTile<64>::BYTES;
    static constexpr int U0 = 2 * OT, Y0 = U0 + 2 * VP;
    static constexpr int SP = ValueTile<D>::BYTES;
    static constexpr int S0 = Y0 + 2 * VP, DS0 = S0 + 2 * SP;
    static constexpr int WEND = DS0 + 2 * SP;
    // over it, once all value columns are done: K, Q, and the score gradients' planes
    static constexpr int TILE = Tile<D>::BYTES;
    static constexpr int K0 = 0, Q0 = TILE;
    static constexpr int DP0 = 2 * TILE, DA0 = DP0 + 2 * PlaneTile::BYTES;
    static constexpr int XEND = DA0 + 2 * PlaneTile::BYTES;
    // vectors, and sums to join over waves and tiles
    static constexpr int NWV = D / 16;
    static constexpr int VEC = WEND > XEND ? WEND : XEND;
    static constexpr int RED = VEC + DeltaRecord::BYTES - DeltaRecord::VEC;  // [wave][3][64]
    static constexpr int ES = 20;                                   // floats per row of a diagonal block of E
    static constexpr int ED = RED + NWV * 3 * 256;                  // the four diagonal blocks: [64][ES]
    static constexpr int ROW = ED + 64 * ES * 4;                    // row sums of the tiles of E, by block column: [3][64]
    static constexpr int COL = ROW + 3 * 256;                       // column sums, by block row - 1: [3][64]
    static constexpr int KKR = COL + 3 * 256;                       // row sums of D kk (dY U^T): [4][64]
    static constexpr int YV = KKR + 4 * 256;                        // [64]
    static constexpr int DOT = YV + 256;                            // [wave]
    static constexpr int PMX = DOT + 32;                            // largest of dP, dA: [2][wave]
    static constexpr int SIZE = PMX + 64;
};

// Sum over the four lanes of a column (equal l16); every lane gets it.
__device__ __forceinline__ float sum_q4(float x)
{
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

template <int D, int IO>
__global__ __launch_bounds__(4 * D, D == 64 ? 2 : 4) void delta_bwd_grad_kernel(DeltaParams p)
{
    using L = GradLds<D>;
    using TL = Tile<D>;
    constexpr int NW = D / 16, NT = 64 * NW;
    __shared__ __attribute__((aligned(16))) char sm[L::SIZE];
    const int hv = (int)(blockIdx.x % (unsigned)p.HV);
    const int64_t slot = blockIdx.x / (unsigned)p.HV;
    SeqRange rng;
    int64_t c;
    if (!chunk_of(p, slot, &rng, &c)) return;
    const int64_t t0 = rng.b + c * CHUNK;
    const int len = (int)(rng.e - t0 < CHUNK ? rng.e - t0 : CHUNK);
    const int hk = hv / (p.HV / p.H);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int t = threadIdx.x, lane = t & 63, q4 = lane >> 4, l16 = lane & 15;
    auto again = [&]() {
        lane = fresh(threadIdx.x & 63);
        t = 64 * wave + lane;
        q4 = lane >> 4;
        l16 = lane & 15;
    };
    const int64_t item = delta_item(p, slot, hv);
    const char *rec = p.rec + item * (int64_t)DeltaRecord::BYTES;

    constexpr int VCH = (DeltaRecord::BYTES - DeltaRecord::VEC) / 16;
    static_assert(VCH <= NT, "one piece per thread");
    if (t < VCH) lds_st(sm, L::VEC + 16 * t, *reinterpret_cast<const i32x4 *>(rec + DeltaRecord::VEC + 16 * t));

    const int vbytes = (int)(((len - 1) * p.sv + D) * 2);
    const __amdgpu_buffer_rsrc_t ro = buf_rsrc(p.dout + t0 * p.sv + hv * p.hsv, vbytes);
    const __amdgpu_buffer_rsrc_t rv = buf_rsrc(p.v + t0 * p.sv + hv * p.hsv, vbytes);
    // (buffers: one offset register per access, where a flat address takes two)
    const __amdgpu_buffer_rsrc_t s_ck = buf_rsrc(p.s_ck + item * D * D, 4 * D * D), ds_ck = buf_rsrc(p.ds_ck + item * D * D, 4 * D * D);
    const __amdgpu_buffer_rsrc_t u_ck = buf_rsrc(p.u_ck + item * 64 * D, 256 * D), y_ck = buf_rsrc(p.y_ck + item * 64 * D, 256 * D);

    // the operands' powers of two and what undoes them, from the sequential passes' maxima
    enum { MS = 0, MU = 1, MV = 2, MD = 4, MY = 5, MO = 6 };
    float m8 = lane < D / 2 ? p.mx[item * (D / 2) + lane] : 0.0f;  // [D / 16][8]
    m8 = fmaxf(m8, __shfl_xor(m8, 8));
    m8 = fmaxf(m8, __shfl_xor(m8, 16));
    m8 = fmaxf(m8, __shfl_xor(m8, 32));
    const int ex8 = IO == IO_F16 && ((lane & 7) == MV || (lane & 7) == MO) ? 0 : scale_exp(m8);
    auto exp_of = [&](int which) { return __builtin_amdgcn_readlane(ex8, which); };
    const int eS = exp_of(MS), eU = exp_of(MU), eV = exp_of(MV), eD = exp_of(MD), eY = exp_of(MY), eO = exp_of(MO);
    // (by its bits: a uniform value that takes no vector register; -114 <= e <= 120)
    auto two = [](int e) { return __uint_as_float((uint32_t)(127 + e) << 23); };

    // fragment id -> (16 columns, tile, lane): 4 consecutive rows of one value column
    auto st_frag = [&](int base, int plane, auto tile_of, f32x4 x, float sc, int id, int tiles, bool state) {
        using VT = decltype(tile_of);
        const int ln = id & 63, tile = (id >> 6) % tiles, v = (id >> 6) / tiles * 16 + (ln & 15);
        const int r = state ? state_row(tile, ln >> 4) : 16 * tile + 4 * (ln >> 4);
        uint32_t h0, l0, h1, l1;
        split2_f16(x[0] * sc, x[1] * sc, h0, l0);
        split2_f16(x[2] * sc, x[3] * sc, h1, l1);
        lds_st(sm, base + VT::quad(v, r >> 2), u32x2{h0, h1});
        lds_st(sm, base + plane + VT::quad(v, r >> 2), u32x2{l0, l1});
    };

    f32x4 aq[4], ay[4], au[4];  // dO S^T, dY S^T, U dS^T: rows 16 mt .., key columns 16 wave ..
    constexpr int TPW = (10 + NW - 1) / NW;
    f32x4 ou[TPW], yu[TPW];     // (dO U^T)^T, (dY U^T)^T
    f32x4 yv = {0, 0, 0, 0};
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
    for (int vb = 0; vb < D / 32; ++vb) {
        again();
        // fragments of 32 value columns: 2 (D / 16) 64 of S and dS, 512 of U and dY
        constexpr int SPT = 2 * (D / 16) * 64 / NT;  // 2
        constexpr int UPT = 512 / NT;                // 1 (D = 128), 2 (D = 64)
        // (dY and V follow once S has left its registers: all at once is no faster, after the stores 5% slower)
        {
            f32x4 fs[SPT], fd[SPT], fu[UPT], fy[UPT];
            i32x4 fo = {}, fv = {};
#pragma unroll
            for (int i = 0; i < SPT; ++i) fs[i] = buf_ld16<f32x4>(s_ck, 16 * (uint32_t)(vb * 2 * (D / 16) * 64 + t + NT * i));
#pragma unroll
            for (int i = 0; i < SPT; ++i) fd[i] = buf_ld16<f32x4>(ds_ck, 16 * (uint32_t)(vb * 2 * (D / 16) * 64 + t + NT * i));
#pragma unroll
            for (int i = 0; i < UPT; ++i) fu[i] = buf_ld16<f32x4>(u_ck, 16 * (uint32_t)(vb * 512 + t + NT * i));
            const uint32_t off = (uint32_t)((t >> 2) * (int)p.sv + vb * 32 + (t & 3) * 8) * 2;
            if (t < 256) fo = buf_ld16<i32x4>(ro, off);
            if (vb > 0) __syncthreads();  // the block before is done with
#pragma unroll
            for (int i = 0; i < SPT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) dot = fmaf(fs[i][e], fd[i][e], dot);
#pragma unroll
            for (int i = 0; i < SPT; ++i) st_frag(L::S0, L::SP, ValueTile<D>{}, fs[i], two(eS), t + NT * i, D / 16, true);
            region();
#pragma unroll
            for (int i = 0; i < UPT; ++i) fy[i] = buf_ld16<f32x4>(y_ck, 16 * (uint32_t)(vb * 512 + t + NT * i));
            if (t < 256) fv = buf_ld16<i32x4>(rv, off);
#pragma unroll
            for (int i = 0; i < SPT; ++i) st_frag(L::DS0, L::SP, ValueTile<D>{}, fd[i], two(eD), t + NT * i, D / 16, true);
#pragma unroll
            for (int i = 0; i < UPT; ++i) st_frag(L::U0, L::VP, ValueTile<64>{}, fu[i], two(eU), t + NT * i, 4, false);
            if (t < 256) lds_st(sm, L::O0 + token_piece(t >> 2, t & 3), row_f16<IO>(fo, two(eO)));
#pragma unroll
            for (int i = 0; i < UPT; ++i) st_frag(L::Y0, L::VP, ValueTile<64>{}, fy[i], two(eY), t + NT * i, 4, false);
            if (t < 256) lds_st(sm, L::VT0 + token_piece(t >> 2, t & 3), row_f16<IO>(fv, two(eV)));
        }
        __syncthreads();
        again();
        const i32x4 sh = ValueTile<D>::col(sm + L::S0, wave, q4, l16), sl = ValueTile<D>::col(sm + L::S0 + L::SP, wave, q4, l16);
        const i32x4 dh = ValueTile<D>::col(sm + L::DS0, wave, q4, l16), dl = ValueTile<D>::col(sm + L::DS0 + L::SP, wave, q4, l16);
        auto o_row = [&](int base, int mt) { return lds_ld<i32x4>(sm, base + token_piece(16 * mt + l16, q4)); };
        auto v_col = [&](int base, int part, int mt) { return ValueTile<64>::col(sm + base + part * L::VP, mt, q4, l16); };
        // acc + (ah + al) (bh + bl), without al bl
        auto split = [](i32x4 ah, i32x4 al, i32x4 bh, i32x4 bl, f32x4 acc) {
            return mfma_f16(al, bh, mfma_f16(ah, bl, mfma_f16(ah, bh, acc)));
        };
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const i32x4 o = o_row(L::O0, mt);
            aq[mt] = mfma_f16(o, sl, mfma_f16(o, sh, aq[mt]));
            ay[mt] = split(v_col(L::Y0, 0, mt), v_col(L::Y0, 1, mt), sh, sl, ay[mt]);
            au[mt] = split(v_col(L::U0, 0, mt), v_col(L::U0, 1, mt), dh, dl, au[mt]);
            if (mt & 1) region();
        }
#pragma unroll
        for (int i = 0; i < TPW; ++i) {
            const int id = wave + NW * i;
            if (id < 10) {
                int br, bc;
                tri(id, br, bc);
                const i32x4 uh = v_col(L::U0, 0, bc), ul = v_col(L::U0, 1, bc), o = o_row(L::O0, br);
                ou[i] = mfma_f16(ul, o, mfma_f16(uh, o, ou[i]));
                yu[i] = split(uh, ul, v_col(L::Y0, 0, br), v_col(L::Y0, 1, br), yu[i]);
            }
            region();
        }
        if (wave < 4) {  // the diagonal of dY V^T, block `wave`
            const i32x4 vh = o_row(L::VT0, wave);
            yv = mfma_f16(v_col(L::Y0, 1, wave), vh, mfma_f16(v_col(L::Y0, 0, wave), vh, yv));
        }
    }
    again();
    if (wave < 4 && l16 >> 2 == q4)  // row 4 q4 + e = column l16
        *reinterpret_cast<float *>(sm + L::YV + 4 * (16 * wave + l16)) =
            (l16 & 2 ? (l16 & 1 ? yv[3] : yv[2]) : (l16 & 1 ? yv[1] : yv[0])) * two(-eY) * two(-eV);
    const float *vec = reinterpret_cast<const float *>(sm + L::VEC), *vec2 = vec + (DeltaRecord::VEC2 - DeltaRecord::VEC) / 4;
    // one power of two for all rows of K, and one for Q's: the smallest of the rows'
    float uk = 1.0f, uq = 1.0f;
    if constexpr (IO == IO_BF16) {
        uk = vec2[DeltaRecord::CK * 64 + lane];
        uq = vec2[DeltaRecord::CQ * 64 + lane];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            uk = fminf(uk, __shfl_xor(uk, d));
            uq = fminf(uq, __shfl_xor(uq, d));
        }
        uk = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(uk)));
        uq = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(uq)));
    }
    // (powers of two: the reciprocal has the exponent's complement)
    const float ik = __uint_as_float((254u << 23) - __float_as_uint(uk)), iq = __uint_as_float((254u << 23) - __float_as_uint(uq));
    {
        constexpr int CPT = 64 * D / 8 / NT;  // 2
        const __amdgpu_buffer_rsrc_t rk = buf_rsrc(p.k + t0 * p.sk + hk * p.hsk, (int)(((len - 1) * p.sk + D) * 2));
        const __amdgpu_buffer_rsrc_t rq = buf_rsrc(p.q + t0 * p.sq + hk * p.hsq, (int)(((len - 1) * p.sq + D) * 2));
        i32x4 a[CPT], b[CPT];
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int ci = t + NT * i, row = ci / (D / 8), cc = ci % (D / 8);
            a[i] = buf_ld16<i32x4>(rk, (uint32_t)(row * (int)p.sk + cc * 8) * 2);
            b[i] = buf_ld16<i32x4>(rq, (uint32_t)(row * (int)p.sq + cc * 8) * 2);
        }
        __syncthreads();  // the last block is done with
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int ci = t + NT * i, row = ci / (D / 8), cc = ci % (D / 8);
            lds_st(sm, L::K0 + TL::piece(row, cc), row_f16<IO>(a[i], uk));
            lds_st(sm, L::Q0 + TL::piece(row, cc), row_f16<IO>(b[i], uq));
        }
    }
    __syncthreads();

    again();
    // score gradients, rows r = 16 br + l16, columns s = 16 bc + 4 q4 + e: the same tiles of Q K^T and K K^T, decayed
    float pm = 0.0f, am = 0.0f;
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
        const int id = wave + NW * i;
        if (id < 10) {
            int br, bc;
            tri(id, br, bc);
            f32x4 kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const i32x4 a = TL::row(sm + L::K0, bc, j, q4, l16);
                kk = mfma_f16(a, TL::row(sm + L::K0, br, j, q4, l16), kk);
                qk = mfma_f16(a, TL::row(sm + L::Q0, br, j, q4, l16), qk);
                if (j & 1) region();
            }
            kk = kk * ik * ik;
            qk = qk * ik * iq;
            const int r = 16 * br + l16, s0 = 16 * bc + 4 * q4;
            const float gh = vec2[DeltaRecord::GH * 64 + r], gl = vec2[DeltaRecord::GL * 64 + r], bt = vec[DeltaRecord::BT * 64 + r];
            const f32x4 sh = *reinterpret_cast<const f32x4 *>(vec2 + DeltaRecord::GH * 64 + s0), sl = *reinterpret_cast<const f32x4 *>(vec2 + DeltaRecord::GL * 64 + s0);
            ou[i] = ou[i] * two(-eO) * two(-eU) * p.scale;
            yu[i] = yu[i] * two(-eY) * two(-eU);
            f32x4 dp, da, E;
            float kkr = 0.0f, er = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float d = ex2(fminf((gh - sh[e]) + (gl - sl[e]), 0.0f));
                const bool below = s0 + e < r;
                const float yd = below ? d * yu[i][e] : 0.0f;
                dp[e] = s0 + e <= r ? d * ou[i][e] : 0.0f;
                da[e] = -bt * yd;
                E[e] = below ? dp[e] * qk[e] + da[e] * kk[e] : 0.0f;
                kkr = fmaf(yd, kk[e], kkr);
                er += E[e];
                pm = fmaxf(pm, fabsf(dp[e]));
                am = fmaxf(am, fabsf(da[e]));
            }
            kkr = sum_q4(kkr);
            if (q4 == 0) *reinterpret_cast<float *>(sm + L::KKR + 256 * bc + 4 * r) = kkr;
            if (br == bc) {
                lds_st(sm, L::ED + (r * L::ES + 4 * q4) * 4, E);
            } else {
                er = sum_q4(er);
                if (q4 == 0) *reinterpret_cast<float *>(sm + L::ROW + 256 * bc + 4 * r) = er;
                f32x4 ec;
#pragma unroll
                for (int e = 0; e < 4; ++e) ec[e] = sum16(E[e]);
                if (l16 == 0) lds_st(sm, L::COL + 256 * (br - 1) + 4 * s0, ec);
            }
            ou[i] = dp;
            yu[i] = da;
        }
        region();
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        pm = fmaxf(pm, __shfl_xor(pm, d));
        am = fmaxf(am, __shfl_xor(am, d));
    }
    if (lane == 0) {
        *reinterpret_cast<float *>(sm + L::PMX + 4 * wave) = pm;
        *reinterpret_cast<float *>(sm + L::PMX + 32 + 4 * wave) = am;
    }
    __syncthreads();
    pm = am = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        pm = fmaxf(pm, lds_ld<float>(sm, L::PMX + 4 * w));
        am = fmaxf(am, lds_ld<float>(sm, L::PMX + 32 + 4 * w));
    }
    const int eP = __builtin_amdgcn_readfirstlane(scale_exp(pm)), eA = __builtin_amdgcn_readfirstlane(scale_exp(am));
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
        const int id = wave + NW * i;
        if (id < 10) {
            int br, bc;
            tri(id, br, bc);
            const int r = 16 * br + l16, c4 = 4 * bc + q4;
            auto st_plane = [&](int base, int col4, f32x4 x, float sc) {
                uint32_t h0, l0, h1, l1;
                split2_f16(x[0] * sc, x[1] * sc, h0, l0);
                split2_f16(x[2] * sc, x[3] * sc, h1, l1);
                lds_st(sm, base + PlaneTile::quad(r, col4), u32x2{h0, h1});
                lds_st(sm, base + PlaneTile::BYTES + PlaneTile::quad(r, col4), u32x2{l0, l1});
            };
            st_plane(L::DP0, c4, ou[i], two(eP));
            st_plane(L::DA0, c4, yu[i], two(eA));
            if (br == bc && !(br & 1)) {  // the zero block right of it
                st_plane(L::DP0, c4 + 4, f32x4{0, 0, 0, 0}, 1.0f);
                st_plane(L::DA0, c4 + 4, f32x4{0, 0, 0, 0}, 1.0f);
            }
        }
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
    if (lane == 0) *reinterpret_cast<float *>(sm + L::DOT + 4 * wave) = dot;
    __syncthreads();

    again();
    // dQ and dK of this wave's key columns, and their rows' products with q and k
    const bool grouped = p.H != p.HV;
    __amdgpu_buffer_rsrc_t rdq, rdk;  // per value head in float32, or the gradients themselves
    if (grouped) {
        const int64_t o = (t0 * p.HV + hv) * D;
        const int bytes = (int)(uint32_t)(((int64_t)(len - 1) * p.HV * D + D) * 4);
        rdq = buf_rsrc(p.dq_ws + o, bytes);
        rdk = buf_rsrc(p.dk_ws + o, bytes);
    } else {
        const int64_t o = (t0 * p.H + hk) * D;
        const int bytes = ((len - 1) * p.H * D + D) * 2;
        rdq = buf_rsrc(p.dq + o, bytes);
        rdk = buf_rsrc(p.dk + o, bytes);
    }
    float *red = reinterpret_cast<float *>(sm + L::RED) + wave * 192;
    // right operands: rows 32 j .. of K and Q, the wave's columns
    bf16x4 kc[4], qc[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
        kc[mt] = TL::quad(sm + L::K0, mt, wave, q4, l16);
        qc[mt] = TL::quad(sm + L::Q0, mt, wave, q4, l16);
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
        auto vec4 = [&](int which) { return lds_ld<f32x4>(sm, L::VEC + which * 256 + (16 * mt + 4 * q4) * 4); };
        auto pow2 = [&](int which) { return *reinterpret_cast<const f32x4 *>(vec2 + which * 64 + 16 * mt + 4 * q4); };
        // (the vectors without the rows' powers of two)
        const f32x4 ck = pow2(DeltaRecord::CK);
        f32x4 dq = aq[mt] * two(-eO) * two(-eS) * (vec4(DeltaRecord::EQ) * pow2(DeltaRecord::CQ));
        f32x4 y = ay[mt] * two(-eY) * two(-eS) * (vec4(DeltaRecord::EG) * ck), x = au[mt] * two(-eU) * two(-eD) * (vec4(DeltaRecord::ED) * ck);
        f32x4 si, sy, sx, dk = x - vec4(DeltaRecord::BT) * y;
        // q and k of rows 16 mt + 4 q4 .., column 16 wave + l16
        const f32x4 qv = __builtin_convertvector(__builtin_bit_cast(f16x4, qc[mt]), f32x4) * iq;
        const f32x4 kv = __builtin_convertvector(__builtin_bit_cast(f16x4, kc[mt]), f32x4) * ik;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            si[e] = sum16(qv[e] * dq[e]);
            sy[e] = sum16(kv[e] * y[e]);
            sx[e] = sum16(kv[e] * x[e]);
        }
        if (l16 == 0) {
            *reinterpret_cast<f32x4 *>(red + 16 * mt + 4 * q4) = si;
            *reinterpret_cast<f32x4 *>(red + 64 + 16 * mt + 4 * q4) = sy;
            *reinterpret_cast<f32x4 *>(red + 128 + 16 * mt + 4 * q4) = sx;
        }
        auto prow = [&](int base, int j) {
            const int a = base + 64 * 16 * mt + 2048 * j;
            return __builtin_bit_cast(i32x4, cat4(lds_ld<bf16x4>(sm, a + PlaneTile::quad(l16, q4)), lds_ld<bf16x4>(sm, a + PlaneTile::quad(l16, 4 + q4))));
        };
        auto pcol = [&](int base, int j) { return PlaneTile::col(sm + base, mt, j, q4, l16); };
        constexpr int PB = PlaneTile::BYTES;
        f32x4 pk = {0, 0, 0, 0}, pq = {0, 0, 0, 0}, ak = {0, 0, 0, 0};  // dP K, dP^T Q, (dA + dA^T) K
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const i32x4 k8 = __builtin_bit_cast(i32x4, cat4(kc[2 * j], kc[2 * j + 1])), q8 = __builtin_bit_cast(i32x4, cat4(qc[2 * j], qc[2 * j + 1]));
            if (j <= mt / 2) {
                pk = mfma_f16(prow(L::DP0, j), k8, pk);
                pk = mfma_f16(prow(L::DP0 + PB, j), k8, pk);
                ak = mfma_f16(prow(L::DA0, j), k8, ak);
                ak = mfma_f16(prow(L::DA0 + PB, j), k8, ak);
            }
            if (j >= mt / 2) {
                pq = mfma_f16(pcol(L::DP0, j), q8, pq);
                pq = mfma_f16(pcol(L::DP0 + PB, j), q8, pq);
                ak = mfma_f16(pcol(L::DA0, j), k8, ak);
                ak = mfma_f16(pcol(L::DA0 + PB, j), k8, ak);
            }
        }
        dq += pk * two(-eP) * ik;
        dk += pq * two(-eP) * iq + ak * two(-eA) * ik;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // (rows past the chunk's end lie past the buffers' range)
            const uint32_t r = 16 * mt + 4 * q4 + e;
            if (grouped) {
                const uint32_t o = 4 * (r * (uint32_t)(p.HV * D) + 16 * wave + l16);
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(dq[e]), rdq, o, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(dk[e]), rdk, o, 0, 0);
            } else {
                const uint32_t o = 2 * (r * (uint32_t)(p.H * D) + 16 * wave + l16);
                __builtin_amdgcn_raw_buffer_store_b16(f32_io<IO>(dq[e]), rdq, o, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b16(f32_io<IO>(dk[e]), rdk, o, 0, 0);
            }
        }
        region();
    }
    __syncthreads();
    if (wave != 0) return;

    // the scalars: lane = token
    float I = 0.0f, Y = 0.0f, X = 0.0f, sd = 0.0f, kkr = 0.0f;
    auto f32_at = [&](int base, int i) { return lds_ld<float>(sm, base + 4 * i); };
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        I += f32_at(L::RED + w * 768, lane);
        Y += f32_at(L::RED + w * 768 + 256, lane);
        X += f32_at(L::RED + w * 768 + 512, lane);
        sd += f32_at(L::DOT, w);
    }
#pragma unroll
    for (int b = 0; b < 4; ++b)
        if (b <= q4) kkr += f32_at(L::KKR + 256 * b, lane);
    const float bt = vec[DeltaRecord::BT * 64 + lane];
    const float dbeta = f32_at(L::YV, lane) - Y - kkr;
    I -= bt * Y;
    // sum of E over r >= t > s, t = lane = 16 q4 + l16: whole tiles left of
    // and below t's block, the rows from t on of the tiles left of the
    // diagonal, the columns before t of the tiles under it, and the diagonal
    float rows_left = 0.0f, cols_under = 0.0f, tiles = 0.0f;
#pragma unroll
    for (int b = 0; b < 3; ++b) {
        if (b < q4) rows_left += f32_at(L::ROW + 256 * b, lane);
        if (b >= q4) cols_under += f32_at(L::COL + 256 * b, lane);
    }
    // (row sums of the blocks further down, columns left of t's block)
    float below[3];
#pragma unroll
    for (int br = 1; br < 4; ++br) {
        float s = 0.0f;
#pragma unroll
        for (int b = 0; b < 3; ++b)
            if (b < br && b < q4 && br > q4) s += f32_at(L::ROW + 256 * b, 16 * br + l16);
        below[br - 1] = sum16(s);
    }
    tiles = below[0] + below[1] + below[2];
    // suffix sum of rows_left and exclusive prefix of cols_under within the 16 lanes of the block
    float suf = rows_left, pre = cols_under;
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) {
        const float a = __shfl_down(suf, d, 16), b = __shfl_up(pre, d, 16);
        if (l16 + d < 16) suf += a;
        if (l16 >= d) pre += b;
    }
    pre -= cols_under;
    // the diagonal block: this lane's row summed up to each column, then down the columns
    f32x4 row[4];
    float run = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) row[i] = lds_ld<f32x4>(sm, L::ED + (lane * L::ES + 4 * i) * 4);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float x = row[i / 4][i % 4];
        row[i / 4][i % 4] = run;
        run += x;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) lds_st(sm, L::ED + (lane * L::ES + 4 * i) * 4, row[i]);
    float pairs = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const float x = f32_at(L::ED, (16 * q4 + r) * L::ES + l16);
        if (r >= l16) pairs += x;
    }
    float Isum = I, Xsum = X;  // suffix sum of I, inclusive prefix of X
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const float a = __shfl_down(Isum, d), b = __shfl_up(Xsum, d);
        if (lane + d < 64) Isum += a;
        if (lane >= d) Xsum += b;
    }
    const float xb = __shfl_up(Xsum, 1);
    const float dg = pairs + suf + pre + tiles + Isum + (lane > 0 ? xb : 0.0f) + vec[(DeltaRecord::SCAL - DeltaRecord::VEC) / 4] * sd;
    if (lane < len) {
        const int64_t o = (t0 + lane) * p.HV + hv;
        p.dbeta[o] = f32_io<IO>(dbeta);
        if (p.gtype == G_F32) static_cast<float *>(p.dg)[o] = dg;
        else static_cast<uint16_t *>(p.dg)[o] = p.gtype == G_F16 ? f32_io<IO_F16>(dg) : f32_io<IO_BF16>(dg);
    }
}

// dq, dk of a q/k head with several value heads: the sums over them, in their
// order, of the sequences' tokens (what lies behind the last one is left as
// it is). Eight columns per thread.
template <int IO>
__global__ __launch_bounds__(256) void delta_bwd_reduce_kernel(DeltaParams p)
{
    const int m = p.HV / p.H, pieces = p.K / 8;
    const int64_t b = seq_of(p, 0).b, e = seq_of(p, p.N - 1).e, total = (e - b) * p.H * pieces;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / pieces + b * p.H;  // (token, q/k head): its value heads' rows follow each other
        const int c = (int)(i % pieces) * 8;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const float *src = (w ? p.dk_ws : p.dq_ws) + row * m * p.K + c;
            f32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
            for (int j = 0; j < m; ++j) {
                lo += *reinterpret_cast<const f32x4 *>(src + (int64_t)j * p.K);
                hi += *reinterpret_cast<const f32x4 *>(src + (int64_t)j * p.K + 4);
            }
            uint16_t *dst = (w ? p.dk : p.dq) + row * p.K + c;
            u32x2 a, d;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                a[x] = (uint32_t)f32_io<IO>(lo[2 * x]) | (uint32_t)f32_io<IO>(lo[2 * x + 1]) << 16;
                d[x] = (uint32_t)f32_io<IO>(hi[2 * x]) | (uint32_t)f32_io<IO>(hi[2 * x + 1]) << 16;
            }
            *reinterpret_cast<i32x4 *>(dst) = i32x4{(int)a[0], (int)a[1], (int)d[0], (int)d[1]};
        }
    }
}

}  // namespace

template <int K, int IO, int NC>
static hipError_t launch_bwd_state_nc(const DeltaParams &p, hipStream_t stream)
{
    const int64_t chains = (int64_t)p.N * p.HV;
    const dim3 grid((unsigned)(chains * (p.V / (16 * NC)) * p.nseg)), block(64 * (NC + LW));
    if constexpr (NC < 8) {
        if (p.nseg > 1) {
            const dim3 grid1((unsigned)(chains * (p.V / 64) * (p.nseg - 1)));
            hipLaunchKernelGGL((delta_bwd_state_kernel<K, IO, 4, SEG>), grid1, dim3(64 * (4 + LW)), 0, stream, p);
            if (hipError_t e = launch_delta_join_bwd(p, stream); e != hipSuccess) return e;
            hipLaunchKernelGGL((delta_bwd_state_kernel<K, IO, NC, JOIN>), grid, block, 0, stream, p);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((delta_bwd_state_kernel<K, IO, NC, OUT>), grid, block, 0, stream, p);
    return hipGetLastError();
}

template <int K, int IO>
static hipError_t launch_bwd_state_cols(const DeltaParams &p, int cols, hipStream_t stream)
{
    // (K = V: 128 columns only with 128 key rows)
    if constexpr (K == 128)
        if (cols == 128) return launch_bwd_state_nc<K, IO, 8>(p, stream);
    return cols == 64 ? launch_bwd_state_nc<K, IO, 4>(p, stream) : launch_bwd_state_nc<K, IO, 2>(p, stream);
}

hipError_t launch_delta_bwd_state(const DeltaParams &p, int ncu, hipStream_t stream)
{
    const int cols = delta_columns(p, ncu);
    if (p.K == 128) return p.io == IO_F16 ? launch_bwd_state_cols<128, IO_F16>(p, cols, stream) : launch_bwd_state_cols<128, IO_BF16>(p, cols, stream);
    return p.io == IO_F16 ? launch_bwd_state_cols<64, IO_F16>(p, cols, stream) : launch_bwd_state_cols<64, IO_BF16>(p, cols, stream);
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
    const int64_t blocks = (p.T * p.H * p.K / 8 + 255) / 256;
    const dim3 rgrid((unsigned)(blocks < 65536 ? blocks : 65536));
    if (p.io == IO_F16) hipLaunchKernelGGL((delta_bwd_reduce_kernel<IO_F16>), rgrid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((delta_bwd_reduce_kernel<IO_BF16>), rgrid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace gdn2
