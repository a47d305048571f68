// Layer and RMS norm of rows with weight, bias and a SiLU gate, and their
// gradients (CDNA4, gfx950). Per row x of D elements:
//
//     n = (x - mean) r, r = 1 / sqrt(var + eps)   or   n = x r, r = 1 / sqrt(mean x^2 + eps)
//     q = n w + b,   y = q   or   q z sigmoid(z)
//
// and with s = z sigmoid(z), dq = dy s, m = dq w:
//
//     dz = dy q s'(z),   dw = sum over rows of dq n,   db = sum of dq,
//     dx = r (m - mean m - n mean(m n))   or   r (m - n mean(m n))
//
// Bound by HBM: a row stays in the registers of the lanes that share it (8 to
// 64 lanes, or a whole workgroup), is read once and written once; the
// backward makes the row's statistics again from x, which it needs anyway.
// A lane takes 16 bytes of each of its pieces. The variance is that of the
// differences from the mean: waves that share a row exchange their own means
// and squares about them (and, backward, sums of m and of m times the same
// differences), which are joined without subtracting large sums.
#include <stdint.h>

#include <type_traits>

#include <hip/hip_runtime.h>

#include "../../include/gdn2.h"
#include "gdn2_mixer_device.h"

namespace gdn2 {
namespace {

using namespace dev;

__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + ex2(x * -1.44269504088896340736f)); }

// a b, rounded (not fused with what it is added to).
__device__ __forceinline__ float product(float a, float b)
{
#pragma clang fp contract(off)
    return a * b;
}

template <int LANES>
__device__ __forceinline__ float lane_sum(float x)  // over aligned groups of LANES lanes
{
    auto dpp = [&](auto ctrl) {
        x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    if constexpr (LANES >= 2) dpp(std::integral_constant<int, 0xB1>{});   // lane ^ 1
    if constexpr (LANES >= 4) dpp(std::integral_constant<int, 0x4E>{});   // lane ^ 2
    if constexpr (LANES >= 8) dpp(std::integral_constant<int, 0x141>{});  // mirrored in 8
    if constexpr (LANES >= 16) dpp(std::integral_constant<int, 0x140>{}); // mirrored in 16
    if constexpr (LANES >= 32) x += __shfl_xor(x, 16);
    if constexpr (LANES >= 64) x += __shfl_xor(x, 32);
    return x;
}

// A lane's piece of a row: P elements, 16 bytes, at any element's address (the
// hardware takes 16-byte accesses off their lines; rows of 2047 elements in
// pieces on the lines, with single elements at both ends, take twice as long).
template <int E>
constexpr int PIECE = E == E_F32 ? 4 : 8;

template <int E>
struct Bits {
    typedef uint16_t type __attribute__((ext_vector_type(8)));
};
template <>
struct Bits<E_F32> {
    typedef float type __attribute__((ext_vector_type(4)));
};

// The first `count` of the elements at p exist (P, but in rows narrower than P).
template <int E>
__device__ __forceinline__ typename Bits<E>::type ld_piece(const void *base, int64_t at, int count)
{
    const Elem<E> *p = static_cast<const Elem<E> *>(base) + at;
    typename Bits<E>::type r = {};
    if (count >= PIECE<E>) {
        __builtin_memcpy(&r, p, 16);
    } else {
#pragma unroll
        for (int i = 0; i < PIECE<E> - 1; ++i)
            if (i < count) r[i] = p[i];
    }
    return r;
}
template <int E>
__device__ __forceinline__ void st_piece(void *base, int64_t at, int count, const float (&x)[PIECE<E>])
{
    constexpr int P = PIECE<E>;
    Elem<E> *p = static_cast<Elem<E> *>(base) + at;
    typename Bits<E>::type r;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if constexpr (E == E_F32) r[i] = x[i];
        else r[i] = f32_el<E>(x[i]);
    }
    if (count >= P) {
        __builtin_memcpy(p, &r, 16);
    } else {
#pragma unroll
        for (int i = 0; i < P - 1; ++i)
            if (i < count) p[i] = r[i];
    }
}
template <int E>
__device__ __forceinline__ void widen_piece(typename Bits<E>::type r, float (&x)[PIECE<E>])
{
#pragma unroll
    for (int i = 0; i < PIECE<E>; ++i) {
        if constexpr (E == E_F32) x[i] = r[i];
        else x[i] = el_f32<E>(r[i]);
    }
}

// Rows as lanes see them: LPR lanes share a row, each with NV pieces LPR apart.
// The row's last piece ends with the row: where the width is no multiple of P
// it begins inside the piece before it, whose elements it has again (and does
// not count again; both lanes store the same values). FULL: it is a multiple.
template <int E, int LPR, int NV, bool FULL>
struct Lanes {
    static constexpr int P = PIECE<E>;
    int sub, D;
    __device__ __forceinline__ explicit Lanes(const NormParams &p) : sub(threadIdx.x % LPR), D(p.D) {}
    __device__ __forceinline__ int begin(int k) const { return (k * LPR + sub) * P; }
    __device__ __forceinline__ bool on(int k) const { return begin(k) < D; }
    __device__ __forceinline__ int first(int k) const { return FULL || begin(k) + P <= D || D < P ? begin(k) : D - P; }
    // whether element i of piece k is one of the row's, and the piece's own
    __device__ __forceinline__ bool in(int k, int i) const
    {
        return on(k) && (FULL || (first(k) + i >= begin(k) && first(k) + i < D));
    }
    __device__ __forceinline__ int own(int k) const { return !on(k) ? 0 : !FULL && D - begin(k) < P ? D - begin(k) : P; }
    __device__ __forceinline__ void load(const void *base, int64_t at, typename Bits<E>::type (&r)[NV]) const
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            r[k] = typename Bits<E>::type{};
            if (on(k)) r[k] = ld_piece<E>(base, at + first(k), FULL ? P : D);
        }
    }
};

template <int E, class L, int NV>
__device__ __forceinline__ void ld_vector(const L &l, const void *v, bool f32, float absent, float (&o)[NV][PIECE<E>])
{
    constexpr int P = PIECE<E>;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < P; ++i) o[k][i] = absent;
        if (!v || !l.on(k)) continue;
        if (E == E_F32 || f32) {
#pragma unroll
            for (int h = 0; h < P; h += 4) {
                const f32x4 x = ld_piece<E_F32>(v, l.first(k) + h, l.D - h);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[k][h + i] = x[i];
            }
        } else {
            widen_piece<E>(ld_piece<E>(v, l.first(k), l.D), o[k]);
        }
    }
}

__device__ __forceinline__ int64_t row_at(const NormParams &p, int which, int64_t row)
{
    if (p.H == 1) return row * p.st[which];
    const uint32_t r = (uint32_t)row, t = r / (uint32_t)p.H;
    return (int64_t)t * p.st[which] + (int64_t)(r - t * (uint32_t)p.H) * p.sh[which];
}

template <int LPR>
constexpr int WAVES = LPR <= 64 ? 1 : LPR / 64;
template <int LPR>
constexpr int WLANES = LPR < 64 ? LPR : 64;

// Count, mean and squares about the mean over the lanes of a wave that share a
// row; a row's waves exchange them through LDS.
template <int E, int LPR, class L, int NV>
__device__ __forceinline__ void own_stats(const NormParams &p, const L &l, const float (&x)[NV][PIECE<E>], float &count, float &mean,
                                          float &sq)
{
    float s = 0.0f, n = 0.0f;
    mean = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) n += (float)l.own(k);
    if (LPR <= 64) count = (float)p.D;
    else count = lane_sum<WLANES<LPR>>(n);
    if (!p.rms) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < PIECE<E>; ++i) s += l.in(k, i) ? x[k][i] : 0.0f;
        s = lane_sum<WLANES<LPR>>(s);
        mean = count > 0.0f ? s / count : 0.0f;
    }
    sq = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < PIECE<E>; ++i) {
            const float d = l.in(k, i) ? x[k][i] - mean : 0.0f;
            sq = fmaf(d, d, sq);
        }
    sq = lane_sum<WLANES<LPR>>(sq);
}

template <int E, int LPR, int NV, int THREADS, bool GATE, bool FULL>
__global__ __launch_bounds__(THREADS) void norm_fwd_kernel(NormParams p)
{
    constexpr int P = PIECE<E>, RPB = THREADS / LPR, W = WAVES<LPR>;
    __shared__ float part[2][THREADS / 64][4];
    const Lanes<E, LPR, NV, FULL> l(p);
    float w[NV][P], b[NV][P];
    typename Bits<E>::type rx[NV], rz[NV];
    // (rows past the last: the last again, not stored)
    auto load = [&](int64_t row) {
        const int64_t r = row < p.rows ? row : p.rows - 1;
        l.load(p.x, row_at(p, NORM_X, r), rx);
        if constexpr (GATE) l.load(p.z, row_at(p, NORM_Z, r), rz);
    };
    const int64_t mine = threadIdx.x / LPR, step = (int64_t)gridDim.x * RPB;
    load((int64_t)blockIdx.x * RPB + mine);
    ld_vector<E>(l, p.w, p.w_f32, 1.0f, w);
    ld_vector<E>(l, p.b, p.b_f32, 0.0f, b);
    const int wave = threadIdx.x >> 6;
    int buf = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < p.rows; r0 += step, buf ^= 1) {
        const int64_t row = r0 + mine;
        const bool on = row < p.rows;
        const int64_t ya = row_at(p, NORM_Y, on ? row : p.rows - 1);
        float x[NV][P], z[NV][P];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            widen_piece<E>(rx[k], x[k]);
            if constexpr (GATE) widen_piece<E>(rz[k], z[k]);
        }
        if (r0 + step < p.rows) load(row + step);
        float count, mean, sq;
        own_stats<E, LPR>(p, l, x, count, mean, sq);
        if constexpr (W > 1) {
            if ((threadIdx.x & 63) == 0) {
                part[buf][wave][0] = count;
                part[buf][wave][1] = mean;
                part[buf][wave][2] = sq;
            }
            __syncthreads();
            const int w0 = wave / W * W;
            float total = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) total = fmaf(part[buf][w0 + i][0], part[buf][w0 + i][1], total);
            mean = total / (float)p.D;
            sq = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float d = part[buf][w0 + i][1] - mean;
                sq += fmaf(part[buf][w0 + i][0] * d, d, part[buf][w0 + i][2]);
            }
        }
        const float rate = 1.0f / sqrtf(sq / (float)p.D + p.eps);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float y[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                y[i] = fmaf((x[k][i] - mean) * rate, w[k][i], b[k][i]);
                if constexpr (GATE) y[i] *= z[k][i] * sigmoid(z[k][i]);
            }
            if (on && l.on(k)) st_piece<E>(p.y, ya + l.first(k), FULL ? P : l.D, y);
        }
    }
}

template <int E, int LPR, int NV, int THREADS, bool GATE, bool FULL>
__global__ __launch_bounds__(THREADS) void norm_bwd_kernel(NormParams p)
{
    constexpr int P = PIECE<E>, RPB = THREADS / LPR, W = WAVES<LPR>;
    __shared__ float part[2][THREADS / 64][6];
    const Lanes<E, LPR, NV, FULL> l(p);
    constexpr bool HOLD = THREADS <= 512 || NV * P <= 8;  // the weights stay in registers (else they are read again for every row)
    float w[NV][P], b[NV][P], dw[NV][P] = {}, db[NV][P] = {};
    typename Bits<E>::type rx[NV], rd[NV], rz[NV];
    auto vectors = [&]() {
        ld_vector<E>(l, p.w, p.w_f32, 1.0f, w);
        if constexpr (GATE) ld_vector<E>(l, p.b, p.b_f32, 0.0f, b);
    };
    if constexpr (HOLD) vectors();
    const int wave = threadIdx.x >> 6;
    const float over = 1.0f / (float)p.D;
    int buf = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < p.rows; r0 += (int64_t)gridDim.x * RPB, buf ^= 1) {
        const int64_t row = r0 + threadIdx.x / LPR;
        const bool on = row < p.rows;
        const int64_t rr = on ? row : p.rows - 1;  // (rows past the last: the last again, not stored)
        float x[NV][P], dy[NV][P];
        l.load(p.x, row_at(p, NORM_X, rr), rx);
        l.load(p.dy, row_at(p, NORM_DY, rr), rd);
        if constexpr (GATE) l.load(p.z, row_at(p, NORM_Z, rr), rz);
        if constexpr (!HOLD) vectors();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            widen_piece<E>(rx[k], x[k]);
            widen_piece<E>(rd[k], dy[k]);
        }
        float count, mean, sq;
        own_stats<E, LPR>(p, l, x, count, mean, sq);
        // sums of m and of m (x - mean), about this wave's mean
        float sm = 0.0f, sx = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float z[P];
            if constexpr (GATE) widen_piece<E>(rz[k], z);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float m = dy[k][i];
                if constexpr (GATE) m *= z[i] * sigmoid(z[i]);
                m = l.in(k, i) ? product(m, w[k][i]) : 0.0f;
                sm += m;
                sx = fmaf(m, l.in(k, i) ? x[k][i] - mean : 0.0f, sx);
            }
        }
        sm = lane_sum<WLANES<LPR>>(sm);
        sx = lane_sum<WLANES<LPR>>(sx);
        if constexpr (W > 1) {
            if ((threadIdx.x & 63) == 0) {
                part[buf][wave][0] = count;
                part[buf][wave][1] = mean;
                part[buf][wave][2] = sq;
                part[buf][wave][3] = sm;
                part[buf][wave][4] = sx;
            }
            __syncthreads();
            const int w0 = wave / W * W;
            float total = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) total = fmaf(part[buf][w0 + i][0], part[buf][w0 + i][1], total);
            mean = total / (float)p.D;
            sq = sm = sx = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float d = part[buf][w0 + i][1] - mean;
                sq += fmaf(part[buf][w0 + i][0] * d, d, part[buf][w0 + i][2]);
                sm += part[buf][w0 + i][3];
                sx += fmaf(d, part[buf][w0 + i][3], part[buf][w0 + i][4]);
            }
        }
        const float rate = 1.0f / sqrtf(sq * over + p.eps);
        const float m0 = p.rms ? 0.0f : sm * over, m1 = sx * rate * over;  // the means of m and of m n
        const int64_t oa = row_at(p, NORM_Y, rr), ga = GATE ? row_at(p, NORM_DZ, rr) : 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float z[P], dx[P], dz[P];
            if constexpr (GATE) widen_piece<E>(rz[k], z);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float n = (x[k][i] - mean) * rate;
                float dq = dy[k][i];
                if constexpr (GATE) {
                    const float sg = sigmoid(z[i]);
                    dz[i] = dq * fmaf(n, w[k][i], b[k][i]) * (sg * fmaf(z[i], 1.0f - sg, 1.0f));
                    dq *= z[i] * sg;
                }
                // (m rounded as it was summed: in a row of one element m - mean m is 0)
                const float m = product(dq, w[k][i]);
                dx[i] = rate * ((m - m0) - n * m1);
                if (on) {  // (the last row again in lanes past it)
                    dw[k][i] = fmaf(dq, n, dw[k][i]);
                    db[k][i] += dq;
                }
            }
            if (on && l.on(k)) {
                st_piece<E>(p.y, oa + l.first(k), FULL ? P : l.D, dx);
                if constexpr (GATE) st_piece<E>(p.dz, ga + l.first(k), FULL ? P : l.D, dz);
            }
        }
    }
    if (!p.part) return;
    // the rows that the workgroup held side by side, joined in a fixed order
    float *out = p.part + (int64_t)blockIdx.x * 2 * p.D;
    if constexpr (RPB == 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (l.in(k, i)) {
                    out[l.first(k) + i] = dw[k][i];
                    out[p.D + l.first(k) + i] = db[k][i];
                }
    } else {
        constexpr int C = LPR * P;  // columns of one piece of all lanes
        __shared__ float red[RPB][C + 4];
        const int sub = threadIdx.x / LPR;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < P; ++i)
                    if (l.in(k, i)) red[sub][l.first(k) + i - k * C] = which ? db[k][i] : dw[k][i];
                __syncthreads();
                for (int c = threadIdx.x; c < C && k * C + c < p.D; c += THREADS) {
                    float s = 0.0f;
#pragma unroll 8
                    for (int r = 0; r < RPB; ++r) s += red[r][c];
                    out[(int64_t)which * p.D + k * C + c] = s;
                }
            }
    }
}

// The workgroups' partial sums joined in a fixed order: COLS columns of dw or
// db per workgroup, 1024 / COLS threads per column, eight loads in flight. Few
// columns need many threads each (1024 rows of partial sums of 128 columns: 64
// columns per workgroup 7.4 us, 16 5.4), many read whole lines.
template <int E, int COLS>
__global__ __launch_bounds__(1024) void norm_dw_kernel(NormParams p)
{
    constexpr int RUNS = 1024 / COLS;
    __shared__ float red[RUNS][COLS + 1];
    const int c = threadIdx.x % COLS, run = threadIdx.x / COLS, which = blockIdx.y;
    const int c0 = blockIdx.x * COLS + c, col = c0 < p.D ? c0 : p.D - 1;
    float s = 0.0f;
    for (int g0 = run; g0 < p.groups; g0 += 8 * RUNS) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int g = g0 + RUNS * i;
            x[i] = g < p.groups ? p.part[((int64_t)g * 2 + which) * p.D + col] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[i];
    }
    red[run][c] = s;
    __syncthreads();
    if (run != 0 || c0 >= p.D) return;
    float x = 0.0f;
#pragma unroll 16
    for (int i = 0; i < RUNS; ++i) x += red[i][c];
    void *out = which ? p.db : p.dw;
    if (out) st_either<E>(out, which ? p.b_f32 : p.w_f32, c0, x);
}

// f<E, LPR, NV, THREADS>() for the call's type, `pieces` of a row and direction.
// (Backward a lane holds the weights and six values per element: one piece
// per lane where 512 lanes reach, so that two and more workgroups share a
// compute unit. 8192 rows of 4096 in 32 bits with a gate: 512 lanes of two
// pieces 146 us, 1024 of one 198; 16,384 of 4096 in 16 bits: 512 of one 108,
// 256 of two 112. Forward a half-idle workgroup costs most: 16,384 rows of
// 2047 elements in 256 lanes of two pieces 55 us, in 128 of two 27.)
template <int E, bool BWD, class F>
void for_width(int pieces, F f)
{
    const int want = pieces;
    bool done = false;
    // the first of the sizes, smallest first, that holds the row
    auto go = [&](auto lpr, auto nv, auto threads) {
        if (done || want > lpr() * nv()) return;
        done = true;
        f(std::integral_constant<int, E>{}, lpr, nv, threads);
    };
    auto in_wave = [&](auto lpr, auto nv) { go(lpr, nv, std::integral_constant<int, 256>{}); };
    auto whole = [&](auto lpr, auto nv) { go(lpr, nv, lpr); };
    constexpr std::integral_constant<int, 1> one{};
    constexpr std::integral_constant<int, 2> two{};
    in_wave(std::integral_constant<int, 8>{}, one);
    in_wave(std::integral_constant<int, 16>{}, one);
    in_wave(std::integral_constant<int, 32>{}, one);
    in_wave(std::integral_constant<int, 64>{}, one);
    if constexpr (BWD) {
        in_wave(std::integral_constant<int, 128>{}, one);
        whole(std::integral_constant<int, 192>{}, one);
        whole(std::integral_constant<int, 256>{}, one);
        whole(std::integral_constant<int, 384>{}, one);
        whole(std::integral_constant<int, 512>{}, one);
        whole(std::integral_constant<int, 384>{}, two);
        whole(std::integral_constant<int, 512>{}, two);
    } else {
        in_wave(std::integral_constant<int, 64>{}, two);
        in_wave(std::integral_constant<int, 128>{}, two);
        whole(std::integral_constant<int, 192>{}, two);
        whole(std::integral_constant<int, 256>{}, two);
        whole(std::integral_constant<int, 384>{}, two);
        whole(std::integral_constant<int, 512>{}, two);
        whole(std::integral_constant<int, 768>{}, two);
    }
    whole(std::integral_constant<int, 1024>{}, two);
    if constexpr (E == E_F32) whole(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
}
template <bool BWD, class F>
hipError_t for_types(const NormParams &p, F f)
{
    const int pieces = norm_pieces(p.D, p.io);
    if (p.io == E_F32) for_width<E_F32, BWD>(pieces, f);
    else if (p.io == E_F16) for_width<E_F16, BWD>(pieces, f);
    else for_width<E_BF16, BWD>(pieces, f);
    return hipGetLastError();
}
// f(a, b) with both known when compiled.
template <class F>
void by_flags(bool a, bool b, F f)
{
    if (a && b) f(std::true_type{}, std::true_type{});
    else if (a) f(std::true_type{}, std::false_type{});
    else if (b) f(std::false_type{}, std::true_type{});
    else f(std::false_type{}, std::false_type{});
}
// Workgroups: at most what stays resident (each backward one leaves a row of
// partial sums).
template <bool BWD>
int64_t row_groups(int64_t rows, int pieces, int io)
{
    int64_t side = 1, wide = 256;
    auto f = [&](auto, auto lpr, auto, auto threads) {
        side = threads() / lpr();
        wide = threads();
    };
    if (io == E_F32) for_width<E_F32, BWD>(pieces, f);
    else for_width<E_BF16, BWD>(pieces, f);
    const int64_t most = BWD ? (wide <= 256 ? 1024 : wide <= 512 ? 512 : 256) : wide <= 512 ? 2048 : 1024;
    const int64_t all = (rows + side - 1) / side;
    return all < most ? all : most;
}

}  // namespace

int32_t norm_bwd_groups(int64_t rows, int32_t D, int32_t io)
{
    return (int32_t)row_groups<true>(rows, norm_pieces(D, io), io);
}

hipError_t launch_norm_fwd(const NormParams &p, hipStream_t stream)
{
    if (p.rows == 0) return hipSuccess;
    const int pieces = norm_pieces(p.D, p.io);
    const dim3 grid((unsigned)row_groups<false>(p.rows, pieces, p.io));
    return for_types<false>(p, [&](auto e, auto lpr, auto nv, auto threads) {
        auto go = [&](auto gate, auto full) {
            hipLaunchKernelGGL((norm_fwd_kernel<e(), lpr(), nv(), threads(), gate(), full()>), grid, dim3(threads()), 0, stream, p);
        };
        by_flags(p.z != nullptr, p.D % PIECE<e()> == 0, go);
    });
}

hipError_t launch_norm_bwd(const NormParams &p, hipStream_t stream)
{
    if (p.rows > 0) {
        const dim3 grid((unsigned)p.groups);
        hipError_t e = for_types<true>(p, [&](auto e, auto lpr, auto nv, auto threads) {
            auto go = [&](auto gate, auto full) {
                hipLaunchKernelGGL((norm_bwd_kernel<e(), lpr(), nv(), threads(), gate(), full()>), grid, dim3(threads()), 0, stream, p);
            };
            by_flags(p.z != nullptr, p.D % PIECE<e()> == 0, go);
        });
        if (e != hipSuccess) return e;
    }
    if (!p.dw && !p.db) return hipSuccess;
    auto sums = [&](auto e) {
        const dim3 few((unsigned)((p.D + 15) / 16), 2), many((unsigned)((p.D + 63) / 64), 2);
        if (p.D <= 1024) hipLaunchKernelGGL((norm_dw_kernel<e(), 16>), few, dim3(1024), 0, stream, p);
        else hipLaunchKernelGGL((norm_dw_kernel<e(), 64>), many, dim3(1024), 0, stream, p);
    };
    if (p.io == E_F32) sums(std::integral_constant<int, E_F32>{});
    else if (p.io == E_F16) sums(std::integral_constant<int, E_F16>{});
    else sums(std::integral_constant<int, E_BF16>{});
    return hipGetLastError();
}

}  // namespace gdn2
