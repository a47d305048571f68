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
// One workgroup (4 waves) per (chunk, value head). Wave w owns the rows
// r = 16 w .. of both score products, computed transposed (the left operand
// is the earlier token's key), so that a lane holds four consecutive columns
// of one row: that is its share of the record's fragments, stored from
// registers. T follows by blocks of 16, also transposed: the diagonal blocks
// by forward substitution, one per wave, and then for wave i, column by
// column towards the left,
//     T_ij^T = -T_jj^T (sum_{j < m <= i} A_mj^T T_im^T)
// on float32 MFMA (16x16x4), whose accumulators are its next right operands.
// Bound by HBM (57 KiB read and written per item): 18,700 items of 8 packed
// sequences (36,962 tokens, 32 heads) take 210 us, 5.2 TB/s; with three waves
// per SIMD instead of four, whose registers spill nothing either, a seventh
// longer.
template <int K>
struct WyLds {
    static constexpr int RS = 2 * K + 16;  // row stride of a staged tile (bytes): rows 16 bytes apart in banks
    static constexpr int TILE = 64 * RS;
    static constexpr int K0 = 0, Q0 = TILE;
    // over the tiles, once both products are done
    static constexpr int AS = 68;          // floats per row of A^T
    static constexpr int A0 = 0;
    static constexpr int TS = 20;          // floats per row of a transposed diagonal block of T
    static constexpr int T0 = A0 + 64 * AS * 4;
    static constexpr int TEND = T0 + 64 * TS * 4;
    static constexpr int V0 = 2 * TILE > TEND ? 2 * TILE : TEND;
    static constexpr int SIZE = V0 + 8 * 256;  // G in two parts, beta, rk, rq, ck, cq; the waves' maxima
};

template <int K, int IO, bool L2N>
__global__ __launch_bounds__(256, 4) void delta_wy_kernel(DeltaParams p)
{
    using L = WyLds<K>;
    __shared__ __attribute__((aligned(16))) char sm[L::SIZE];
    const int hv = (int)(blockIdx.x % (unsigned)p.HV);
    const int64_t slot = blockIdx.x / (unsigned)p.HV;
    SeqRange rng;
    int64_t c;
    if (!chunk_of(p, slot, &rng, &c)) return;
    const int64_t t0 = rng.b + c * CHUNK;
    const int len = (int)(rng.e - t0 < CHUNK ? rng.e - t0 : CHUNK);
    const int hk = hv / (p.HV / p.H);
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63, q4 = lane >> 4, l16 = lane & 15;

    // the gates first (their wait is then the tiles')
    float g = 0.0f, bt = 0.0f;
    if (wave == 0 && lane < len) {
        const int64_t tok = t0 + lane;
        if (p.g) {
            const int64_t o = tok * p.sg + hv * p.hsg;
            if (p.gtype == G_F32) g = static_cast<const float *>(p.g)[o];
            else if (p.gtype == G_F16) g = io_f32<IO_F16>(static_cast<const uint16_t *>(p.g)[o]);
            else g = io_f32<IO_BF16>(static_cast<const uint16_t *>(p.g)[o]);
        }
        bt = p.beta ? io_f32<IO>(p.beta[tok * p.sb + hv * p.hsb]) : 1.0f;
    }
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
            if constexpr (IO == IO_BF16) {
                // the powers of two for the sequential passes' fp16 rows, from the largest magnitude
                // (as integers: bf16 magnitudes order like their bits)
                auto row_max = [](i32x4 x) {
                    uint32_t m = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t lo = (uint32_t)x[e] & 0x7fffu, hi = (uint32_t)x[e] >> 16 & 0x7fffu;
                        m = max(m, max(lo, hi));
                    }
                    // over the K / 8 lanes of the row
                    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, true));   // lane ^ 1
                    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, true));   // lane ^ 2
                    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xf, 0xf, true));  // mirrored in 8
                    if (K == 128) m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xf, 0xf, true));  // in 16
                    return ldexpf(1.0f, scale_exp(__uint_as_float(m << 16)));
                };
                const float ck = row_max(a[i]), cq = row_max(b[i]);
                if (col == 0) {
                    lds_st(sm, L::V0 + 5 * 256 + 4 * row, ck);
                    lds_st(sm, L::V0 + 6 * 256 + 4 * row, cq);
                }
            }
        }
    }
    float *vec = reinterpret_cast<float *>(sm + L::V0);
    char *rec = p.rec + delta_item(p, slot, hv) * (int64_t)DeltaRecord::BYTES;
    float *rvec = reinterpret_cast<float *>(rec + DeltaRecord::VEC);
    double G = 0.0, GC = 0.0;
    if (wave == 0) {
        // running sum of g in 64 bits: its differences are exponents, and a
        // strongly decayed chunk's sum is far larger than they are. Every g is
        // bounded from below first: e^-200 is 0 in float32 as all beneath it
        // are, and the other tokens' decays are not lost next to a state reset
        // written as the type's lowest value (NaN stays).
        g = g < -200.0f ? -200.0f : g;
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
            // (a row of zeros stays one: its factor must not set the scale of an fp16 operand)
            vec[192 + row] = sk == 0.0f ? 0.0f : 1.0f / fmaxf(sqrtf(sk), 1e-12f);
            vec[256 + row] = 1.0f / fmaxf(sqrtf(sq), 1e-12f);
        }
        __syncthreads();
    }
    if (wave == 0) {
        const float ck = IO == IO_BF16 ? vec[320 + lane] : 1.0f, cq = IO == IO_BF16 ? vec[384 + lane] : 1.0f;
        const float rk = (L2N ? vec[192 + lane] : 1.0f) / ck, rq = (L2N ? vec[256 + lane] : 1.0f) / cq;  // (exact)
        const float eg = ex2((float)G), gh = (float)G;
        rvec[DeltaRecord::EG * 64 + lane] = eg * rk;
        rvec[DeltaRecord::EQ * 64 + lane] = eg * rq * p.scale;
        rvec[DeltaRecord::ED * 64 + lane] = ex2((float)(GC - G)) * rk;
        rvec[DeltaRecord::BT * 64 + lane] = bt;
        float *rvec2 = reinterpret_cast<float *>(rec + DeltaRecord::VEC2);
        rvec2[DeltaRecord::GH * 64 + lane] = gh;
        rvec2[DeltaRecord::GL * 64 + lane] = (float)(G - (double)gh);
        rvec2[DeltaRecord::CK * 64 + lane] = ck;
        rvec2[DeltaRecord::CQ * 64 + lane] = cq;
        if (lane == 0) *reinterpret_cast<float *>(rec + DeltaRecord::SCAL) = ex2((float)GC);
    }

    // rows r = 16 wave + l16 of A and P, columns 16 s + 4 q4 + e
    auto mm = [](i32x4 a, i32x4 b, f32x4 acc) {
        if constexpr (IO == IO_F16)
            return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), acc, 0, 0, 0);
        else return mfma_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc);
    };
    const int r = 16 * wave + l16;
    f32x4 At[4], Pt[4];
    {
        i32x4 kb[K / 32], qb[K / 32];
#pragma unroll
        for (int j = 0; j < K / 32; ++j) {
            kb[j] = lds_ld<i32x4>(sm, L::K0 + r * L::RS + 64 * j + 16 * q4);
            qb[j] = lds_ld<i32x4>(sm, L::Q0 + r * L::RS + 64 * j + 16 * q4);
        }
        const float gh = vec[r], gl = vec[64 + r], br = vec[128 + r] * (L2N ? vec[192 + r] : 1.0f);
        const float sr = p.scale * (L2N ? vec[256 + r] : 1.0f);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            At[s] = Pt[s] = f32x4{0, 0, 0, 0};
            if (s > wave) continue;
            f32x4 kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < K / 32; ++j) {
                const i32x4 a = lds_ld<i32x4>(sm, L::K0 + (16 * s + l16) * L::RS + 64 * j + 16 * q4);
                kk = mm(a, kb[j], kk);
                qk = mm(a, qb[j], qk);
            }
            const f32x4 gsh = lds_ld<f32x4>(sm, L::V0 + (16 * s + 4 * q4) * 4);
            const f32x4 gsl = lds_ld<f32x4>(sm, L::V0 + 256 + (16 * s + 4 * q4) * 4);
            f32x4 rks = {1, 1, 1, 1};
            if constexpr (L2N) rks = lds_ld<f32x4>(sm, L::V0 + 768 + (16 * s + 4 * q4) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = 16 * s + 4 * q4 + e;
                // the exponent is not positive for col <= r; above the diagonal the product is not used
                const float d = ex2(fminf((gh - gsh[e]) + (gl - gsl[e]), 0.0f)) * rks[e];
                At[s][e] = col < r ? br * d * kk[e] : 0.0f;
                Pt[s][e] = col <= r ? sr * d * qk[e] : 0.0f;
            }
        }
    }
    // blocks 2 j and 2 j + 1 of block row `wave`, times sc, to the record's planes
    auto st_pair = [&](int plane, int j, f32x4 x0, f32x4 x1, float sc, bool low) {
        i32x4 h, l;
        split8_f16(x0, x1, sc, h, l);
        char *dst = rec + plane + DeltaRecord::frag(wave, j) + 16 * lane;
        *reinterpret_cast<i32x4 *>(dst) = h;
        if (low) *reinterpret_cast<i32x4 *>(dst + DeltaRecord::PLANE) = l;
    };
    // the waves' largest magnitudes, at vec[448 + 4 which + wave]
    auto put_max = [&](int which, const f32x4 (&x)[4]) {
        const float m = max16(col_max(x));
        if (lane == 0) vec[448 + 4 * which + wave] = m;
    };
    auto chunk_exp = [&](int which) {
        const f32x4 m = lds_ld<f32x4>(sm, L::V0 + (448 + 4 * which) * 4);
        return scale_exp(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
    };
    put_max(0, Pt);
    __syncthreads();  // the tiles are done with
    {
        const int ex = chunk_exp(0);
        const float sc = ldexpf(1.0f, ex);
        st_pair(DeltaRecord::PH, 0, Pt[0], Pt[1], sc, p.low_p);
        if (wave >= 2) st_pair(DeltaRecord::PH, 1, Pt[2], Pt[3], sc, p.low_p);
        if (t == 0) *reinterpret_cast<float *>(rec + DeltaRecord::SCAL + 8) = ldexpf(1.0f, -ex);
    }

    float *A = reinterpret_cast<float *>(sm + L::A0), *TD = reinterpret_cast<float *>(sm + L::T0);
#pragma unroll
    for (int s = 0; s < 4; ++s)
        if (s <= wave)
#pragma unroll
            for (int e = 0; e < 4; ++e) A[(16 * s + 4 * q4 + e) * L::AS + r] = At[s][e];
    __syncthreads();
    // diagonal block `wave` of T: column l16 by forward substitution
    {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == l16 ? 1.0f : 0.0f;
        const float *Ad = A + 16 * wave * L::AS + 16 * wave;
#pragma unroll
        for (int m = 0; m < 15; ++m)
#pragma unroll
            for (int i4 = (m + 1) / 4; i4 < 4; ++i4) {
                const f32x4 a = *reinterpret_cast<const f32x4 *>(Ad + m * L::AS + 4 * i4);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * i4 + e > m) x[4 * i4 + e] = fmaf(-a[e], x[m], x[4 * i4 + e]);
            }
        if (q4 == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f32x4 *>(TD + (16 * wave + l16) * L::TS + 4 * i) = f32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    }
    __syncthreads();
    // block row `wave`, from the diagonal to the left
    f32x4 Tt[4];
#pragma unroll
    for (int s = 3; s >= 0; --s) {
        Tt[s] = f32x4{0, 0, 0, 0};
        if (s > wave) continue;
        if (s == wave) {
#pragma unroll
            for (int e = 0; e < 4; ++e) Tt[s][e] = TD[(16 * s + 4 * q4 + e) * L::TS + l16];
        } else {
            f32x4 acc = {0, 0, 0, 0}, res = {0, 0, 0, 0};
#pragma unroll
            for (int m = 3; m > s; --m) {
                if (m > wave) continue;
                const f32x4 a = *reinterpret_cast<const f32x4 *>(A + (16 * s + l16) * L::AS + 16 * m + 4 * q4);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], Tt[m][e], acc, 0, 0, 0);
            }
            const f32x4 td = *reinterpret_cast<const f32x4 *>(TD + (16 * s + l16) * L::TS + 4 * q4);
#pragma unroll
            for (int e = 0; e < 4; ++e) res = __builtin_amdgcn_mfma_f32_16x16x4f32(td[e], acc[e], res, 0, 0, 0);
            Tt[s] = -res;
        }
    }
    put_max(1, Tt);
    __syncthreads();
    const int ex = chunk_exp(1);
    const float sc = ldexpf(1.0f, ex);
    st_pair(DeltaRecord::TH, 0, Tt[0], Tt[1], sc, true);
    if (wave >= 2) st_pair(DeltaRecord::TH, 1, Tt[2], Tt[3], sc, true);
    if (t == 0) *reinterpret_cast<float *>(rec + DeltaRecord::SCAL + 4) = ldexpf(1.0f, -ex);
}

// -------------------------------------------------------- sequential pass --
// One workgroup per (sequence, value head, 16 NC value columns): NC
// computing waves, each with 16 columns of S in registers, and 4
// waves that stage the chunks two ahead of them (loads a chunk ahead in
// registers, tiles a chunk ahead in the other half of LDS) and store the
// outputs of the chunk before. One barrier per chunk; the computing waves
// touch no global memory but for the states.
//
// Bound, with many chains, by HBM: a chunk's tiles, record and outputs are 85
// KiB per item (the packed batch above: 480 us, of which its longest chain of
// 128 chunks sets 270; equal lengths in 128 columns 390 us, 4.1 TB/s). With few
// chains by a chunk's chain of products, 2.1 us at 32 columns: see the split run
// (delta_join_kernel).
constexpr int LW = 4;  // staging waves

// For a bf16 output, which is rounded by up to 2^-8 of itself, the high parts of
// S, P and U do: to nearest, they are off by up to 2^-11, as likely up as down
// (outputs are off by 1.68e-3 in the 2-norm, 1.66e-3 of it their own rounding;
// with the low parts a call takes 3 to 9% longer, in 128 columns 20%). Next to
// fp16 rounding they do not.
template <int K, int IO, int COLS, bool CKPT>
struct StateLds {
    static constexpr int TILE = Tile<K>::BYTES;
    static constexpr int VS = 2 * COLS + 16;  // row stride of the V tile (later the chunk's outputs)
    static constexpr int K0 = 0;
    static constexpr int Q0 = TILE;           // (outputs only)
    static constexpr int V0 = CKPT ? TILE : 2 * TILE;
    static constexpr int R0 = V0 + 64 * VS;   // the record: planes of T (and P), vectors
    static constexpr int RP = CKPT ? DeltaRecord::PH : IO == IO_BF16 ? DeltaRecord::PL : DeltaRecord::VEC;  // bytes of planes
    static constexpr int RCH = (RP + DeltaRecord::SCAL + 16 - DeltaRecord::VEC) / 16;
    static constexpr int G0 = R0 + RP;        // its vectors
    static constexpr int HALF = (R0 + 16 * RCH + 511) / 512 * 512;
    static constexpr int SIZE = 2 * HALF;
};

// (SEG: end states and transitions, the K columns of the transition after the
// V of the state)
template <int K, int IO, int NC, int MODE>
__global__ __launch_bounds__(64 * (NC + LW)) void delta_state_kernel(DeltaParams p)
{
    constexpr int COLS = 16 * NC;
    constexpr bool SPLIT = MODE == SEG || MODE == JOIN || MODE == JOIN_CKPTS;
    constexpr bool STORE = MODE == CKPTS || MODE == JOIN_CKPTS, CKPT = STORE || MODE == SEG;  // (CKPT: no outputs)
    using L = StateLds<K, IO, COLS, CKPT>;
    using TL = Tile<K>;
    constexpr int KT = K / 16, KS = K / 32;
    constexpr bool AHEAD = NC < 8;
    __shared__ __attribute__((aligned(16))) char sm[L::SIZE];
    const int nvb = p.V / COLS;
    const int blocks = MODE == SEG ? nvb + K / COLS : nvb;
    const int nseg = !SPLIT ? 1 : MODE == SEG ? p.nseg - 1 : p.nseg;
    const Chain chain = chain_of(p, blocks * nseg);
    const int hv = chain.hv, n = chain.n, seg = chain.part / blocks, vb = chain.part % blocks;
    const bool transition = MODE == SEG && vb >= nvb;
    if (transition && seg == 0) return;  // (entered with the known initial state)
    const int hk = hv / (p.HV / p.H);
    SeqRange rng = chain.rng;
    int64_t nch = chunks_of(rng);
    int64_t slot0 = chunk_slot(rng.b, n, 0);
    if constexpr (SPLIT) segment_of(p.nseg, seg, rng, nch, slot0);
    // where a split run keeps segment s of this chain
    const int64_t seg_size = (int64_t)K * p.V + K * K;
    float *segs = SPLIT ? p.seg + ((int64_t)n * p.HV + hv) * (p.nseg - 1) * seg_size : nullptr;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;

    if (wave >= NC) {
        const int t = threadIdx.x - 64 * NC;
        constexpr int TH = 64 * LW;
        constexpr int CPT = 64 * K / 8 / TH;             // 16-byte pieces of a K or Q tile per thread
        constexpr int VCH = 64 * COLS / 8;               // pieces of the V tile
        constexpr int VPT = (VCH + TH - 1) / TH;
        constexpr int RPT = (L::RCH + TH - 1) / TH;
        i32x4 fk[CPT], fq[CPT], fv[VPT], fr[RPT];
        float ck[CPT], cq[CPT];  // the rows' powers of two
        auto fetch = [&](int64_t c) {
            const int64_t t0 = rng.b + c * CHUNK;
            const int len = (int)(rng.e - t0 < CHUNK ? rng.e - t0 : CHUNK);
            const __amdgpu_buffer_rsrc_t rk = buf_rsrc(p.k + t0 * p.sk + hk * p.hsk, (int)(((len - 1) * p.sk + K) * 2));
            const __amdgpu_buffer_rsrc_t rq = buf_rsrc(p.q + t0 * p.sq + hk * p.hsq, (int)(((len - 1) * p.sq + K) * 2));
            const __amdgpu_buffer_rsrc_t rv = buf_rsrc(p.v + t0 * p.sv + hv * p.hsv, transition ? 0 : (int)(((len - 1) * p.sv + p.V) * 2));
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                const int ci = t + TH * i, row = ci / (K / 8), cc = ci % (K / 8);
                fk[i] = buf_ld16<i32x4>(rk, (uint32_t)(row * (int)p.sk + cc * 8) * 2);
                if constexpr (!CKPT) fq[i] = buf_ld16<i32x4>(rq, (uint32_t)(row * (int)p.sq + cc * 8) * 2);
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int ci = t + TH * i, row = ci / (COLS / 8), cc = ci % (COLS / 8);
                if (VCH % TH == 0 || ci < VCH)
                    fv[i] = buf_ld16<i32x4>(rv, (uint32_t)(row * (int)p.sv + vb * COLS + cc * 8) * 2);
            }
            const char *rec = p.rec + delta_item(p, slot0 + c, hv) * (int64_t)DeltaRecord::BYTES;
            if constexpr (IO == IO_BF16) {
                const float *v2 = reinterpret_cast<const float *>(rec + DeltaRecord::VEC2);
#pragma unroll
                for (int i = 0; i < CPT; ++i) {
                    const int row = (t + TH * i) / (K / 8);
                    ck[i] = v2[DeltaRecord::CK * 64 + row];
                    if constexpr (!CKPT) cq[i] = v2[DeltaRecord::CQ * 64 + row];
                }
            }
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int id = t + TH * i;  // the planes that are used, then the vectors
                if (id < L::RCH)
                    fr[i] = *reinterpret_cast<const i32x4 *>(rec + 16 * id + (16 * id >= L::RP ? DeltaRecord::VEC - L::RP : 0));
            }
        };
        auto stage = [&](char *half) {
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                const int ci = t + TH * i, row = ci / (K / 8), cc = ci % (K / 8);
                lds_st(half, L::K0 + TL::piece(row, cc), row_f16<IO>(fk[i], ck[i]));
                if constexpr (!CKPT) lds_st(half, L::Q0 + TL::piece(row, cc), row_f16<IO>(fq[i], cq[i]));
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int ci = t + TH * i, row = ci / (COLS / 8), cc = ci % (COLS / 8);
                if (VCH % TH == 0 || ci < VCH) lds_st(half, L::V0 + row * L::VS + cc * 16, fv[i]);
            }
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int id = t + TH * i;
                if (id < L::RCH) lds_st(half, L::R0 + 16 * id, fr[i]);
            }
        };
        // the outputs of chunk c, left where its V tile was (read and later overwritten by the same thread)
        auto flush = [&](int64_t c) {
            const char *half = sm + (c & 1) * L::HALF;
            const int64_t t0 = rng.b + c * CHUNK;
            const int len = (int)(rng.e - t0 < CHUNK ? rng.e - t0 : CHUNK);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int ci = t + TH * i, row = ci / (COLS / 8), cc = ci % (COLS / 8);
                if (ci < VCH && row < len)
                    *reinterpret_cast<i32x4 *>(p.out + (t0 + row) * p.so + hv * p.hso + vb * COLS + cc * 8) =
                        lds_ld<i32x4>(half, L::V0 + row * L::VS + cc * 16);
            }
        };
        if (nch > 0) {
            fetch(0);
            stage(sm);
            if (nch > 1) fetch(1);
        }
        __syncthreads();
        for (int64_t c = 0; c < nch; ++c) {
            if constexpr (!CKPT)
                if (c > 0) flush(c - 1);
            if (c + 1 < nch) stage(sm + ((c + 1) & 1) * L::HALF);
            if (c + 2 < nch) fetch(c + 2);
            __syncthreads();
        }
        if constexpr (!CKPT)
            if (nch > 0) flush(nch - 1);
        return;
    }

    const int q4 = lane >> 4, l16 = lane & 15;
    const int col = (vb * NC + wave) * 16 + l16;
    const int64_t shead = ((int64_t)n * p.HV + hv) * K * p.V;
    const int64_t sr = p.state_vmajor ? 1 : p.V, sc = p.state_vmajor ? K : 1;
    f32x4 S[KT];
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            S[i][e] = transition ? (state_row(i, q4) + e == col - p.V ? 1.0f : 0.0f)
                      : seg > 0  ? (MODE != SEG ? segs[(seg - 1) * seg_size + (state_row(i, q4) + e) * (int64_t)p.V + col] : 0.0f)
                      : p.h0     ? state_ld(p.h0, p.h0_bf16, shead + (state_row(i, q4) + e) * sr + col * sc) : 0.0f;
    constexpr int OP = IO == IO_BF16 ? 1 : 2;  // parts of what only the outputs need
    RightOp<KS> So;
    So.set(S);
    __syncthreads();
    for (int64_t c = 0; c < nch; ++c) {
        char *half = sm + (c & 1) * L::HALF;
        const char *KL = half + L::K0, *QL = half + L::Q0;
        const char *TH = half + L::R0, *PH = TH + 2 * DeltaRecord::PLANE;
        const int64_t frag = delta_item(p, slot0 + c, hv) * (p.V / 16) + (vb * NC + wave);
        auto vec = [&](int which, f32x4 (&x)[4]) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) x[mt] = lds_ld<f32x4>(half, L::G0 + which * 256 + (16 * mt + 4 * q4) * 4);
        };
        // the left operands of four independent products, and the products
        auto rows = [&](const char *tile, int j, i32x4 (&a)[4]) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) a[mt] = TL::row(tile, mt, j, q4, l16);
        };
        auto cols = [&](int i0, int j, i32x4 (&a)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = TL::col(KL, i0 + i, j, q4, l16);
        };
        auto times = [&](const auto &op, int parts, const i32x4 (&a)[4], int j, f32x4 (&y)[4]) {
#pragma unroll
            for (int part = 0; part < parts; ++part)
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = op.mul1(a[i], j, part, y[i]);
        };
        auto frags = [&](const char *plane, int j, i32x4 (&a)[4]) {
#pragma unroll
            for (int mt = 2 * j; mt < 4; ++mt) a[mt] = ld_frag(plane, mt, j, lane);
        };
        // (parts of the plane and of the operand: 2, or 1 of each)
        auto lower = [&](const i32x4 (&ah)[4], const i32x4 (&al)[4], const auto &op, int parts, int j, f32x4 (&y)[4]) {
#pragma unroll
            for (int mt = 2 * j; mt < 4; ++mt) y[mt] = op.mul1(ah[mt], j, 0, y[mt]);
            if (parts == 2) {
#pragma unroll
                for (int mt = 2 * j; mt < 4; ++mt) y[mt] = op.mul1(ah[mt], j, 1, y[mt]);
#pragma unroll
                for (int mt = 2 * j; mt < 4; ++mt) y[mt] = op.mul1(al[mt], j, 0, y[mt]);
            }
        };
        constexpr f32x4 zero = {0, 0, 0, 0};
        f32x4 R[4] = {zero, zero, zero, zero}, o[4] = {zero, zero, zero, zero}, U[4] = {zero, zero, zero, zero};
        f32x4 v[4], bt[4], eg[4], ed[4], eq[4];
        i32x4 a0[4], a1[4], b0[4], b1[4];
        // Every block of loads stands where the products two regions before
        // its use begin (AHEAD), or at its use: two computing waves per SIMD
        // hide each other's waits, and have a third fewer registers.
        auto early = [&](auto load) {
            if constexpr (AHEAD) load();
        };
        auto late = [&](auto load) {
            if constexpr (!AHEAD) load();
        };
        auto fence = [&]() {
            if constexpr (AHEAD) region();
        };
        auto rv = [&]() {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
                v[mt] = io4_f32<IO>(lds_tr(half, L::V0 + (16 * mt + 4 * q4 + (l16 >> 2)) * L::VS + 2 * (16 * wave + 4 * (l16 & 3))));
            vec(DeltaRecord::EG, eg);
            vec(DeltaRecord::BT, bt);
        };
        auto planes = [&](const char *plane, int parts, int j, i32x4 (&a)[4], i32x4 (&b)[4]) {
            frags(plane, j, a);
            if (parts == 2) frags(plane + DeltaRecord::PLANE, j, b);
        };
        const f32x4 scal = lds_ld<f32x4>(half, L::G0 + DeltaRecord::SCAL - DeltaRecord::VEC);  // e^(G_C), 1 / scales of T and P
        const float gamma = scal[0];

        // K S
        early([&] { rows(KL, 0, a0), rows(KL, 1, a1); });
        if constexpr (STORE) {
            f32x4 *dst = reinterpret_cast<f32x4 *>(p.s_ck) + frag * (KT * 64) + lane;
#pragma unroll
            for (int i = 0; i < KT; ++i) dst[64 * i] = S[i];
        }
        const float smax = So.mx;
        fence();
#pragma unroll
        for (int j = 0; j < KS; j += 2) {
            late([&] { rows(KL, j, a0); });
            times(So, 2, a0, j, R);
            early([&] {
                if (j + 2 < KS) rows(KL, j + 2, a0);
                else if (!CKPT) rows(QL, 0, a0);
            });
            fence();
            late([&] { rows(KL, j + 1, a1); });
            times(So, 2, a1, j + 1, R);
            early([&] {
                if (j + 2 < KS) rows(KL, j + 3, a1);
                else rv();
                if (j + 2 >= KS && !CKPT) rows(QL, 1, a1);
            });
            fence();
        }
        // R = beta (V - e^G K S) as a right operand, beside half of Q S
        late(rv);
        early([&] { planes(TH, 2, 0, b0, b1); });
        if constexpr (!CKPT && AHEAD) {
            times(So, OP, a0, 0, o);
            if (KS > 2) rows(QL, 2, a0);
            times(So, OP, a1, 1, o);
            if (KS > 2) rows(QL, 3, a1);
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) R[mt] = bt[mt] * (v[mt] - eg[mt] * So.inv * R[mt]);
        RightOp<2> Ro;
        Ro.set(R);
        fence();
        // U = T R, and e^(G_C - G) U, beside the other half
        late([&] { planes(TH, 2, 0, b0, b1); });
        lower(b0, b1, Ro, 2, 0, U);
        early([&] { planes(TH, 2, 1, b0, b1), vec(DeltaRecord::ED, ed); });
        fence();
        late([&] { planes(TH, 2, 1, b0, b1); });
        lower(b0, b1, Ro, 2, 1, U);
        early([&] { cols(0, 0, b0), cols(0, 1, b1); });
        fence();
        if constexpr (!CKPT && KS > 2 && AHEAD) {
            times(So, OP, a0, 2, o);
            times(So, OP, a1, 3, o);
        }
        const float tinv = Ro.inv * scal[1];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) U[mt] *= tinv;
        // O = scale e^G Q S + P U, left where this wave's columns of V were
        RightOp<2, OP> Uo;
        auto outputs = [&](int j) {
            if (j == 0) {
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) o[mt] = o[mt] * (eq[mt] * So.inv);
            }
            f32x4 y[4] = {zero, zero, zero, zero};
            lower(j ? a0 : b0, j ? a1 : b1, Uo, OP, j, y);
            const float s = Uo.inv * scal[2];
#pragma unroll
            for (int mt = 2 * j; mt < 4; ++mt) o[mt] += y[mt] * s;
        };
        auto store_out = [&]() {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) st_rows16<IO>(half + L::V0 + (16 * mt + 4 * q4) * L::VS + 32 * wave, L::VS, o[mt], l16);
        };
        if constexpr (!CKPT && !AHEAD) {
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                rows(QL, j, a0);
                times(So, OP, a0, j, o);
            }
            vec(DeltaRecord::EQ, eq);
            Uo.set(U);
            planes(PH, OP, 0, b0, b1);
            outputs(0);
            planes(PH, OP, 1, a0, a1);
            outputs(1);
            store_out();
        }
        late([&] { vec(DeltaRecord::ED, ed); });
        RightOp<2> Wo;
        {
            f32x4 W[4];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                if constexpr (STORE) reinterpret_cast<f32x4 *>(p.u_ck)[frag * 256 + 64 * mt + lane] = U[mt];
                W[mt] = U[mt] * ed[mt];
            }
            Wo.set(W);
            if constexpr (STORE) {
                const f32x4 m = {max16(smax), max16(col_max(U)), max16(col_max(v)), 0.0f};
                if (lane == 0) *reinterpret_cast<f32x4 *>(p.mx + frag * 8) = m;
            }
        }
        fence();
        // S <- e^(G_C) S + K^T (e^(G_C - G) U)
#pragma unroll
        for (int i0 = 0; i0 < KT; i0 += 4) {
            f32x4 s[4] = {zero, zero, zero, zero};
            late([&] { cols(i0, 0, b0); });
            times(Wo, 2, b0, 0, s);
            early([&] {
                if (i0 + 4 < KT) cols(i0 + 4, 0, b0);
                else if (!CKPT) planes(PH, OP, 0, b0, a0);
            });
            fence();
            late([&] { cols(i0, 1, b1); });
            times(Wo, 2, b1, 1, s);
            early([&] {
                if (i0 + 4 < KT) cols(i0 + 4, 1, b1);
                else if (!CKPT) vec(DeltaRecord::EQ, eq);
            });
            if (!CKPT && AHEAD && i0 == 0) Uo.set(U);
            fence();
#pragma unroll
            for (int i = 0; i < 4; ++i) S[i0 + i] = S[i0 + i] * gamma + s[i] * Wo.inv;
        }
        if constexpr (!CKPT && AHEAD) {
            // beside the next chunk's operand of S
            if constexpr (OP == 2) {
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) b1[mt] = a0[mt];
            }
            planes(PH, OP, 1, a0, a1);
            outputs(0);
            So.set(S);
            outputs(1);
            store_out();
        } else {
            So.set(S);
        }
        __syncthreads();
    }
    if constexpr (MODE == SEG) {
        float *dst = segs + seg * seg_size + (transition ? (int64_t)K * p.V + col - p.V : col);
        const int64_t row = transition ? K : p.V;
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[(state_row(i, q4) + e) * row] = S[i][e];
    } else if (p.ht && seg == nseg - 1)
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) state_st(p.ht, p.ht_bf16, shead + (state_row(i, q4) + e) * sr + col * sc, S[i][e]);
}

// A split run's segments joined, one after the other, in float32 (16x16x4
// MFMA): end state s <- end state s + transition s times end state s - 1, or,
// of the gradients (BACK), what enters segment s from its end <- that + the
// transposed transition times what enters segment s + 1 (rseg[s - 1] is
// segment s's). Columns are independent: a workgroup takes 16 of a chain's, a
// wave 16 of the rows; the state passes between the waves through LDS,
// transposed, so that four rows of a column are one read. A step's wait is
// the transition (64 KiB a chain), which is loaded a step ahead.
template <int K, bool BACK>
__global__ __launch_bounds__(4 * K) void delta_join_kernel(DeltaParams p)
{
    constexpr int KT = K / 16, RS = K + 4;
    __shared__ __attribute__((aligned(16))) float sm[2][16 * RS];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, q4 = lane >> 4, l16 = lane & 15;
    const int col = (int)(blockIdx.x % (unsigned)(p.V / 16)) * 16 + l16, row = 16 * wave + 4 * q4;
    const int64_t size = (int64_t)K * p.V + K * K, chain = blockIdx.x / (unsigned)(p.V / 16);
    const int steps = p.nseg - 2;
    const float *tr = p.seg + chain * (p.nseg - 1) * size + (int64_t)K * p.V;  // transitions, `size` apart
    // the states that are joined, in order: end states, or rseg from its last on
    float *at = BACK ? p.rseg + (chain * (p.nseg - 1) + steps) * K * p.V : p.seg + chain * (p.nseg - 1) * size;
    const int64_t next = BACK ? -(int64_t)K * p.V : size;
    auto load = [&](int s) {
        f32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = at[s * next + (row + e) * (int64_t)p.V + col];
        return x;
    };
    auto fetch = [&](int s, f32x4 (&m)[KT]) {  // rows 16 wave + l16 of step s's matrix
        const float *t = tr + (BACK ? p.nseg - 1 - s : s) * size;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            if constexpr (BACK) {
#pragma unroll
                for (int e = 0; e < 4; ++e) m[i][e] = t[(16 * i + 4 * q4 + e) * K + 16 * wave + l16];
            } else {
                m[i] = *reinterpret_cast<const f32x4 *>(t + (16 * wave + l16) * K + 16 * i + 4 * q4);
            }
        }
    };
    f32x4 m[KT], x = load(0), y = load(1);
    fetch(1, m);
    *reinterpret_cast<f32x4 *>(&sm[0][l16 * RS + row]) = x;
    for (int s = 1; s <= steps; ++s) {
        f32x4 ahead[KT];
        const int s1 = s < steps ? s + 1 : s;
        x = y;
        y = load(s1);
        fetch(s1, ahead);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const f32x4 b = *reinterpret_cast<const f32x4 *>(&sm[(s - 1) & 1][l16 * RS + 16 * i + 4 * q4]);
#pragma unroll
            for (int e = 0; e < 4; ++e) x = __builtin_amdgcn_mfma_f32_16x16x4f32(m[i][e], b[e], x, 0, 0, 0);
        }
        *reinterpret_cast<f32x4 *>(&sm[s & 1][l16 * RS + row]) = x;
#pragma unroll
        for (int e = 0; e < 4; ++e) at[s * next + (row + e) * (int64_t)p.V + col] = x[e];
#pragma unroll
        for (int i = 0; i < KT; ++i) m[i] = ahead[i];
    }
}

template <int K, int IO>
void launch_wy_l2(const DeltaParams &p, dim3 grid, hipStream_t stream)
{
    if (p.qk_l2norm) hipLaunchKernelGGL((delta_wy_kernel<K, IO, true>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((delta_wy_kernel<K, IO, false>), grid, dim3(256), 0, stream, p);
}

template <int K, int IO, int NC>
void launch_state_ck(const DeltaParams &p, bool ckpt, hipStream_t stream)
{
    const int64_t chains = (int64_t)p.N * p.HV;
    const dim3 grid((unsigned)(chains * (p.V / (16 * NC)))), block(64 * (NC + LW));
    if constexpr (NC < 8) {
        if (p.nseg > 1) {
            const dim3 grid1((unsigned)(chains * ((p.V + p.K) / 64) * (p.nseg - 1)));
            hipLaunchKernelGGL((delta_state_kernel<K, IO, 4, SEG>), grid1, dim3(64 * (4 + LW)), 0, stream, p);
            hipLaunchKernelGGL((delta_join_kernel<K, false>), dim3((unsigned)(chains * (p.V / 16))), dim3(4 * K), 0, stream, p);
            const dim3 grid2(grid.x * p.nseg);
            if (ckpt) hipLaunchKernelGGL((delta_state_kernel<K, IO, NC, JOIN_CKPTS>), grid2, block, 0, stream, p);
            else hipLaunchKernelGGL((delta_state_kernel<K, IO, NC, JOIN>), grid2, block, 0, stream, p);
            return;
        }
    }
    if constexpr (16 * NC <= K)  // (gradients: K = V)
        if (ckpt) {
            hipLaunchKernelGGL((delta_state_kernel<K, IO, NC, CKPTS>), grid, block, 0, stream, p);
            return;
        }
    hipLaunchKernelGGL((delta_state_kernel<K, IO, NC, OUT>), grid, block, 0, stream, p);
}

template <int K, int IO>
void launch_state_cols(const DeltaParams &p, bool ckpt, int cols, hipStream_t stream)
{
    if (cols == 128) launch_state_ck<K, IO, 8>(p, ckpt, stream);
    else if (cols == 64) launch_state_ck<K, IO, 4>(p, ckpt, stream);
    else launch_state_ck<K, IO, 2>(p, ckpt, stream);
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

hipError_t launch_delta_join_bwd(const DeltaParams &p, hipStream_t stream)
{
    const dim3 grid((unsigned)((int64_t)p.N * p.HV * (p.V / 16))), block(4 * p.K);
    if (p.K == 128) hipLaunchKernelGGL((delta_join_kernel<128, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((delta_join_kernel<64, true>), grid, block, 0, stream, p);
    return hipGetLastError();
}

int delta_columns(const DeltaParams &p, int ncu)
{
    const int64_t chains = (int64_t)p.N * p.HV * p.nseg;
    if (p.nseg > 1) return chains * (p.V / 32) <= ncu ? 32 : 64;
    for (int cols = 32; cols < p.V; cols *= 2)
        if (chains * (p.V / cols) <= (cols == 64 ? 2 : 1) * (int64_t)ncu) return cols;
    return p.V;
}

int delta_segments(int64_t T, int64_t N, int64_t HV, int64_t K, int64_t V)
{
    if (T <= 0 || N <= 0 || HV <= 0) return 1;
    const int64_t chunks = T / CHUNK / N;  // of a sequence of mean length
    int64_t s = 1 + 256 / (N * HV * ((V + K) / 64));
    if (s == 3 && chunks < 32) return 1;
    if (s > 32) s = 32;
    if (s > chunks / 8) s = chunks / 8;
    return s < 3 ? 1 : (int)s;
}

hipError_t launch_delta_state(const DeltaParams &p, bool ckpt, int ncu, hipStream_t stream)
{
    const int cols = delta_columns(p, ncu);
    if (p.K == 128) {
        if (p.io == IO_F16) launch_state_cols<128, IO_F16>(p, ckpt, cols, stream);
        else launch_state_cols<128, IO_BF16>(p, ckpt, cols, stream);
    } else {
        if (p.io == IO_F16) launch_state_cols<64, IO_F16>(p, ckpt, cols, stream);
        else launch_state_cols<64, IO_BF16>(p, ckpt, cols, stream);
    }
    return hipGetLastError();
}

}  // namespace gdn2
