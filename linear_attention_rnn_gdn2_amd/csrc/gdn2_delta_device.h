// Device helpers of the scalar-gated delta rule's kernels: two-part fp16
// operands, staged tiles and MFMA fragments. Not part of the ABI.
//
// Precision. The sequential passes run on fp16 MFMA with float32 accumulation
// and take a float32 operand as two fp16 parts, x = h + l, each rounded to
// nearest, after a power of two has brought the largest value of its column (or
// chunk) near 2^14: 22 significant bits next to that value, 2^-38 of it at the
// bottom. Products of two such operands drop l l. Rows of q and k that are fp16
// values are used as they are; bf16 rows are brought into fp16's range by a
// power of two (exactly, but for values under 2^-30 of the row's largest, which
// lose bits under fp16's smallest step, 2^-38 of it). The state, the chunk's WY
// solution and all sums are float32.
//
// Fragments (lane = 16 q4 + l16). A 16x16 accumulator tile holds rows
// 4 q4 + e (e = 0..3) of column l16. As the right operand of the next product
// (32 contracted rows = two stacked tiles) the lane's eight values are rows
// 4 q4 + e of the first and of the second tile: the contraction runs in that
// order on both sides, so an accumulator becomes an operand without leaving
// its lane. The left operand then reads two runs of four columns,
// 4 q4 .. and 16 + 4 q4 .. of the 32.
#pragma once

#include "gdn2_delta.h"
#include "gdn2_device.h"

namespace gdn2 {
namespace dev {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int IO>
__device__ __forceinline__ float io_f32(uint16_t b)
{
    if constexpr (IO == IO_F16) return (float)__builtin_bit_cast(_Float16, b);
    else return __uint_as_float((uint32_t)b << 16);
}
template <int IO>
__device__ __forceinline__ uint16_t f32_io(float x)  // rounded to nearest even
{
    if constexpr (IO == IO_F16) return __builtin_bit_cast(uint16_t, (_Float16)x);
    else return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// The state's rows in accumulator tiles: rows 4 q4 .. of tile i are key rows
// state_row(i, q4) .. + 3, so that two tiles (2 j, 2 j + 1) as a right operand
// hold eight consecutive key rows per lane, and the left operand beside them
// is one 16-byte read of a row of K or Q.
__device__ __forceinline__ int state_row(int i, int q4) { return 32 * (i >> 1) + 8 * q4 + 4 * (i & 1); }

// A staged tile of 64 rows of K 16-bit values, read in two ways: 16 rows at 8
// columns (left operands of K S), and transposed, 8 rows at 4 runs of 4
// columns (of K^T U). The 16-byte pieces of a row are permuted by the row's
// bits (swz): the first read then touches every bank once, the second twice
// at most (its runs all lie in one half of their pieces).
template <int K>
struct Tile {
    static constexpr int RS = 2 * K;
    static constexpr int BYTES = 64 * RS;
    __device__ static __forceinline__ int swz(int r)
    {
        return K == 128 ? (r >> 1 & 3) << 2 | (r & 1) << 1 | (r >> 3 & 1) : (r >> 1 & 1) << 2 | (r >> 2 & 3);
    }
    // byte offset of 16-byte piece c of row r
    __device__ static __forceinline__ int piece(int r, int c) { return r * RS + ((c ^ swz(r)) << 4); }
    // rows 16 mt + l16, columns 32 j + 8 q4 ..
    __device__ static __forceinline__ i32x4 row(const char *tile, int mt, int j, int q4, int l16)
    {
        return lds_ld<i32x4>(tile, l16 * RS + (((4 * j + q4) ^ swz(l16)) << 4) + 16 * RS * mt);
    }
    // 4 rows 16 mt + 4 q4 .. of column 16 w + l16
    __device__ static __forceinline__ bf16x4 quad(const char *tile, int mt, int w, int q4, int l16)
    {
        const int r = 4 * q4 + (l16 >> 2);
        return lds_tr(tile, r * RS + (((2 * w + (l16 >> 1 & 1)) ^ swz(r)) << 4) + 8 * (l16 & 1) + 16 * RS * mt);
    }
    // transposed: element (m, k) = tile[k][m], rows k = 32 j + 4 q4 .. and 32 j + 16 + 4 q4 .., columns those of state tile i
    __device__ static __forceinline__ i32x4 col(const char *tile, int i, int j, int q4, int l16)
    {
        const int r = 4 * q4 + (l16 >> 2);
        const int a = r * RS + (((4 * (i >> 1) + (l16 & 3)) ^ swz(r)) << 4) + 8 * (i & 1) + 32 * RS * j;
        return __builtin_bit_cast(i32x4, cat4(lds_tr(tile, a), lds_tr(tile, a + 16 * RS)));
    }
};

// A record's fragment as a left operand.
__device__ __forceinline__ i32x4 ld_frag(const char *plane, int mt, int j, int lane)
{
    return *reinterpret_cast<const i32x4 *>(plane + DeltaRecord::frag(mt, j) + 16 * lane);
}

__device__ __forceinline__ int64_t delta_item(const DeltaParams &p, int64_t slot, int hv) { return slot * p.HV + hv; }

__device__ __forceinline__ f32x4 mfma_f16(i32x4 a, i32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// The exponent of the power of two that brings m near 2^14 (2^13 <= m 2^e <
// 2^14; zero, infinity and NaN count as values near 1).
__device__ __forceinline__ int scale_exp(float m)
{
    const int e = 14 - __builtin_amdgcn_frexp_expf(m);
    return e > 120 ? 120 : e;
}

// y0, y1 in fp16, packed, and what is left of them. (To nearest, which
// gfx950 does for the pair in one instruction: the bf16 outputs use high parts
// without their low ones, and cut off they were 3.5e-4 too small, all alike.)
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_f16(float y0, float y1)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{y0, y1}), f16x2));
}
__device__ __forceinline__ void split2_f16(float y0, float y1, uint32_t &h, uint32_t &l)
{
    h = pack_f16(y0, y1);
    const f16x2 f = __builtin_bit_cast(f16x2, h);
    l = pack_f16(fmaf((float)f[0], -1.0f, y0), fmaf((float)f[1], -1.0f, y1));
}
// Two tiles of a column as an operand: parts of x0 and x1 times sc.
__device__ __forceinline__ void split8_f16(f32x4 x0, f32x4 x1, float sc, i32x4 &h, i32x4 &l)
{
    uint32_t a[4], b[4];
    x0 *= sc;
    x1 *= sc;
    split2_f16(x0[0], x0[1], a[0], b[0]);
    split2_f16(x0[2], x0[3], a[1], b[1]);
    split2_f16(x1[0], x1[1], a[2], b[2]);
    split2_f16(x1[2], x1[3], a[3], b[3]);
    h = i32x4{(int)a[0], (int)a[1], (int)a[2], (int)a[3]};
    l = i32x4{(int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// The largest magnitude of 4 M values per lane over the lane's column (the
// four lanes of equal l16).
template <int M>
__device__ __forceinline__ float col_max(const f32x4 (&x)[M])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
        for (int e = 0; e < 4; e += 2) m = fmaxf(m, fmaxf(fabsf(x[i][e]), fabsf(x[i][e + 1])));
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    m = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// The largest of the 16 lanes of a row; every lane gets it.
__device__ __forceinline__ float max16(float x)
{
    x = fmaxf(x, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x128, 0xf, 0xf, true)));  // row_ror:8
    x = fmaxf(x, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x124, 0xf, 0xf, true)));  // row_ror:4
    x = fmaxf(x, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x122, 0xf, 0xf, true)));  // row_ror:2
    return fmaxf(x, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x121, 0xf, 0xf, true)));  // row_ror:1
}

// A float32 right operand of N 32-row steps (step j: tiles 2 j and 2 j + 1) in
// PARTS fp16 parts, scaled per column.
template <int N, int PARTS = 2>
struct RightOp {
    i32x4 h[N], l[PARTS == 2 ? N : 1];
    float inv;  // what a product is multiplied by
    float mx;   // the column's largest magnitude

    __device__ __forceinline__ void set(const f32x4 (&x)[2 * N])
    {
        mx = col_max(x);
        const int ex = scale_exp(mx);
        const float sc = ldexpf(1.0f, ex);
        inv = ldexpf(1.0f, -ex);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if constexpr (PARTS == 2) {
                split8_f16(x[2 * j], x[2 * j + 1], sc, h[j], l[j]);
            } else {
                const f32x4 y0 = x[2 * j] * sc, y1 = x[2 * j + 1] * sc;
                const f16x4 a = __builtin_convertvector(y0, f16x4), b = __builtin_convertvector(y1, f16x4);  // to nearest
                h[j] = __builtin_bit_cast(i32x4, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
            }
        }
    }
    // acc + a times the high (part 0) or low part of step j
    __device__ __forceinline__ f32x4 mul1(i32x4 a, int j, int part, f32x4 acc) const
    {
        return mfma_f16(a, PARTS == 2 && part ? l[j] : h[j], acc);
    }
};

// 16 bytes of a row of q or k as fp16: as they are, or bf16 times the row's power of two.
template <int IO>
__device__ __forceinline__ i32x4 row_f16(i32x4 raw, float c)
{
    if constexpr (IO == IO_F16) return raw;
    i32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = (int)pack_f16(__uint_as_float((uint32_t)raw[i] << 16) * c, __uint_as_float((uint32_t)raw[i] & 0xffff0000u) * c);
    return y;
}

// Four 16-bit io values as float32.
template <int IO>
__device__ __forceinline__ f32x4 io4_f32(bf16x4 x)
{
    if constexpr (IO == IO_F16) return __builtin_convertvector(__builtin_bit_cast(f16x4, x), f32x4);
    else return __builtin_convertvector(x, f32x4);
}

// Four rows (4 q4 ..) of a wave's 16 columns, rounded to the io type, into a
// row-major tile of 16-bit values at `at` (the byte of row 4 q4's column 0).
// Neighbouring lanes trade halves of their rows, so that every store is a
// whole dword (16-bit stores cost bank conflicts: measured 2200 cycles per
// chunk with eight waves).
template <int IO>
__device__ __forceinline__ void st_rows16(char *at, int stride, f32x4 x, int l16)
{
    const uint32_t p0 = (uint32_t)f32_io<IO>(x[0]) | (uint32_t)f32_io<IO>(x[1]) << 16;
    const uint32_t p1 = (uint32_t)f32_io<IO>(x[2]) | (uint32_t)f32_io<IO>(x[3]) << 16;
    const bool odd = l16 & 1;
    const uint32_t keep = odd ? p1 : p0;
    const uint32_t got = __builtin_amdgcn_update_dpp(0, odd ? p0 : p1, 0xB1, 0xf, 0xf, true);  // lane ^ 1
    const uint32_t first = odd ? got : keep, second = odd ? keep : got;                        // columns l16 & ~1, | 1
    char *a = at + (odd ? 2 * stride : 0) + 2 * (l16 & ~1);
    *reinterpret_cast<uint32_t *>(a) = __builtin_amdgcn_perm(second, first, 0x05040100u);
    *reinterpret_cast<uint32_t *>(a + stride) = __builtin_amdgcn_perm(second, first, 0x07060302u);
}

// The value again, as one the compiler knows nothing of: what is computed
// from it stays where it is used (the lanes' LDS addresses, held over the
// whole kernel, would take a quarter more registers than there are).
__device__ __forceinline__ int fresh(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// Nothing moves across: the sequential passes are latency-bound, and a
// region's loads are those of the products two regions on.
__device__ __forceinline__ void region() { __builtin_amdgcn_sched_barrier(0); }

// Sum over the 16 lanes of a row (lanes with equal q4); every lane gets it.
__device__ __forceinline__ float sum16(float x)
{
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x128, 0xf, 0xf, true));  // row_ror:8
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x124, 0xf, 0xf, true));  // row_ror:4
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x122, 0xf, 0xf, true));  // row_ror:2
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x121, 0xf, 0xf, true));  // row_ror:1
    return x;
}

// What a sequential pass is for: its results (OUT); the forward's walk for
// the gradients' checkpoints (CKPTS); a split run's segments from zero (SEG)
// and its results, each segment entered with the joined state (JOIN, and
// JOIN_CKPTS for checkpoints).
enum { OUT, CKPTS, SEG, JOIN, JOIN_CKPTS };

// The chain (sequence, value head) of a workgroup of the sequential passes
// and which of the chain's `per` workgroups it is. The workgroups that read
// the same tiles of k and q run on one XCD, whose L2 they share (consecutive
// workgroups go to the 8 XCDs in turn), where that leaves every XCD the same
// number of them; up to 64 sequences start longest first, so that with more
// workgroups than compute units the short ones fill the end.
struct Chain {
    int part, hv, n;
    SeqRange rng;
};
// The range that lane i holds (T fits 32 bits).
__device__ __forceinline__ SeqRange range_of(SeqRange r, int i)
{
    return SeqRange{__builtin_amdgcn_readlane((int)r.b, i), __builtin_amdgcn_readlane((int)r.e, i)};
}
__device__ __forceinline__ Chain chain_of(const DeltaParams &p, int per)
{
    const unsigned b = blockIdx.x;
    const int rep = p.HV / p.H, same = per * rep, pairs = p.N * p.H;
    int u, pair;
    if (pairs % 8 == 0) {
        u = (int)(b / 8 % (unsigned)same);
        pair = (int)(b / 8 / (unsigned)same * 8 + b % 8);
    } else {
        u = (int)(b % (unsigned)same);
        pair = (int)(b / (unsigned)same);
    }
    int n = pair / p.H;
    SeqRange rng;
    if (p.N > 1 && p.N <= 64) {
        const int lane = threadIdx.x & 63;
        int len = -1, rank = 0;
        const SeqRange r = seq_of(p, lane < p.N ? lane : 0);
        if (lane < p.N) len = (int)chunks_of(r);
        for (int j = 0; j < p.N; ++j) {
            const int x = __builtin_amdgcn_readlane(len, j);
            rank += x > len || (x == len && j < lane);
        }
        n = __builtin_ctzll(__ballot(lane < p.N && rank == n));
        rng = range_of(r, n);
    } else {
        rng = seq_of(p, n);
    }
    return Chain{u % per, pair % p.H * rep + u / per, n, rng};
}

// Of a chain's chunks, those of segment seg of a split run.
__device__ __forceinline__ void segment_of(int nseg, int seg, SeqRange &rng, int64_t &nch, int64_t &slot0)
{
    const int64_t per = (nch + nseg - 1) / nseg, c0 = seg * per < nch ? seg * per : nch;
    nch = nch - c0 < per ? nch - c0 : per;
    slot0 += c0;
    rng.b += c0 * CHUNK;
    if (rng.e > rng.b + nch * CHUNK) rng.e = rng.b + nch * CHUNK;
}

// The chunk of a checkpoint slot: false where the slot holds none. 64
// sequences at a time are looked at, so that up to 64 cost one load's wait.
__device__ __forceinline__ bool chunk_of(const DeltaParams &p, int64_t slot, SeqRange *rng, int64_t *c)
{
    const int lane = threadIdx.x & 63;
    int n = 0, count = p.N, step;
    do {
        step = (count + 63) / 64;
        const int i = lane * step;
        const SeqRange r = seq_of(p, n + (i < count ? i : 0));
        const uint64_t m = __ballot(i < count && chunk_slot(r.b, n + i, 0) <= slot);
        const int k = m ? 63 - __builtin_clzll(m) : 0;
        *rng = range_of(r, k);
        n += k * step;
        count = count - k * step < step ? count - k * step : step;
    } while (step > 1);
    *c = slot - chunk_slot(rng->b, n, 0);
    return *c >= 0 && *c < chunks_of(*rng);
}

}  // namespace dev
}  // namespace gdn2
