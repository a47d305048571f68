// Internal interface between the C-ABI layer (gdn2_delta_api.cpp) and the
// gfx950 kernels of the scalar-gated delta rule and of the q/k preparation.
// Not installed, not part of the ABI.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

#include "gdn2_internal.h"

namespace gdn2 {

// Validated arguments of one call of the scalar-gated delta rule. Pointers
// are device pointers; optional ones are nullptr when omitted.
struct DeltaParams {
    const uint16_t *q, *k;  // [T, H, K] io
    const uint16_t *v;      // [T, HV, V] io
    const void *g;          // [T, HV] g type, or nullptr (= 0)
    const uint16_t *beta;   // [T, HV] io, or nullptr (= 1)
    const float *h0;        // [N, HV, K, V] (or [N, HV, V, K]) float32 or bf16, or nullptr (= 0)
    const void *cu;         // [N + 1] int32 or int64, or nullptr (one sequence of T tokens)
    uint16_t *out;          // [T, HV, V] io
    float *ht;              // as h0, or nullptr (not written)
    int64_t T;
    int32_t N, H, HV, K, V;
    float scale;            // resolved (never 0)
    int32_t io, gtype;      // IO_*, G_*
    int32_t cu64;
    int32_t h0_bf16, ht_bf16;
    // element strides of the token and head dimensions
    int64_t sq, sk, sv, so, sg, sb;
    int64_t hsq, hsk, hsv, hso, hsg, hsb;
    int32_t state_vmajor;
    int32_t qk_l2norm;
    int32_t nslots;         // slot_count(T, N)
    // workspace (chunked calls): every chunk's record, DeltaRecord::BYTES per (slot, value head)
    char *rec;
    int32_t low_p;          // the record's low plane of P is used
    // a run split along the sequences: segments of every sequence (1: whole sequences), and per (sequence, value
    // head, segment but the last) its end state from zero [K, V] and its transition [K, K], float32; backward: per
    // segment but the first the gradient that leaves it towards the one before [K, V]
    int32_t nseg;
    float *seg, *rseg;
    // backward only. The checkpoints are in accumulator order: per (slot,
    // value head, 16 value columns) the float32 fragments f32x4[tile][lane]
    // of a wave: lane 16 q4 + l16 holds four rows of column l16, key rows
    // state_row(tile, q4) .. or tokens 16 tile + 4 q4 ..
    const uint16_t *dout;   // [T, HV, V] io
    const float *dht;       // [N, HV, K, V] or nullptr (zero)
    float *dh0;             // [N, HV, K, V] or nullptr (not written)
    uint16_t *dq, *dk;      // [T, H, K] io
    uint16_t *dv;           // [T, HV, V] io
    void *dg;               // [T, HV] gtype
    uint16_t *dbeta;        // [T, HV] io
    float *s_ck, *ds_ck;    // state entering / gradient of the state leaving each chunk: K x V per item
    float *u_ck, *y_ck;     // U and dY of each chunk: 64 x V per item
    float *mx;              // [item][V / 16][8]: largest magnitudes of S, U, v, (0), dS, dY, dO, (0) in 16 columns of a chunk
    float *dq_ws, *dk_ws;   // [T, HV, K] per value head (grouped heads only)
};

// One chunk's record, K-independent: the lower triangles of T and P as fp16
// planes (high and low part: 22 significant bits next to the largest value,
// scaled for that by a power of two of the chunk's own), then float32 vectors
// over the chunk's 64 tokens. A plane is a sequence of left-operand fragments
// of 1 KiB, one per 16 rows and 32 columns on or below the diagonal (the
// upper block of a pair on the diagonal is zero): lane 16 q4 + l16 holds row
// l16, columns 4 q4 .. + 3 and 16 + 4 q4 .. + 3 in 16 bytes.
struct DeltaRecord {
    // fragment of rows 16 mt .., columns 32 j .. (j <= mt / 2)
    __host__ __device__ static constexpr int frag(int mt, int j) { return (mt < 2 ? mt : 2 * mt - 2 + j) * 1024; }
    static constexpr int PLANE = 6 * 1024;  // bytes
    static constexpr int TH = 0, TL = PLANE, PH = 2 * PLANE, PL = 3 * PLANE;
    static constexpr int VEC = 4 * PLANE;
    // vectors: e^G rk / ck, scale e^G rq / cq, e^(G_C - G) rk / ck, beta (rk,
    // rq: the reciprocal norms with in-kernel normalisation, else 1; ck, cq:
    // the powers of two that bring a bf16 row of k or q into fp16's range)
    enum { EG = 0, EQ = 1, ED = 2, BT = 3 };
    static constexpr int SCAL = VEC + 4 * 256;  // e^(G_C), and what T and P are multiplied by to undo their scales
    static constexpr int VEC2 = SCAL + 256;
    enum { GH = 0, GL = 1, CK = 2, CQ = 3 };    // G log2(e) in two parts, ck, cq
    static constexpr int BYTES = VEC2 + 4 * 256;
};

// Arguments of the q/k preparation (forward and backward).
struct QkParams {
    const uint16_t *x[2];        // q, k: [T, H or HK, K] io
    uint16_t *y[2];              // outputs (forward: rows; backward: dq, dk)
    const uint16_t *dy[2];       // backward: gradients of the outputs
    const void *w[2];            // weights [K] float32 or io, or nullptr
    void *dw[2];                 // gradients of the weights, the weights' type, or nullptr
    int32_t w_f32[2];
    const float *rope;           // [P, rot]: cos then sin, or nullptr
    const void *pos;             // [T] int32 or int64
    int32_t pos64;
    int64_t P;                   // rows of the table
    int64_t T;
    int32_t heads[2];
    int32_t K, rot;
    int32_t norm, interleaved, io;
    float eps;
    int64_t sx[2], hsx[2], sy[2], hsy[2], sdy[2], hsdy[2];
    float *part;                 // backward with weights: [groups][2][K] partial sums
    int32_t groups;
    int32_t split;               // log2 of the waves per token
};

// Value columns per workgroup of the sequential passes (they hold most of a
// compute unit's LDS each): 32 where every workgroup is resident at once, 64
// where two rounds of them run, else 128. Few chains spread over the device,
// many do not load a chunk's tiles more often than they must, and between
// the two, chains of unlike lengths share the compute units better in halves
// (K = V = 128, bf16, forward and gradients: 256 chains of 20 to 128 chunks in
// 64 columns 681 and 2952 us, in 128 733 and 3216; all of 73 chunks 670 and
// 2939, 609 and 2905; 1024 chains of 16 chunks 630 and 2629, 561 and 2576; 64
// chains of 64 chunks in 32 columns 195 and 762, in 64 215 and 820. The fp16
// forward in 128 columns holds the low parts of its outputs' operands beside
// them and spills: 1024 chains of 16 chunks 657 in 64 columns, 683 in 128; of 64
// chunks 1236, 1290; 19,200 of one chunk 1431, 1202).
int delta_columns(const DeltaParams &p, int ncu);
// Segments of each sequence of a chunked call (1: not split), and the bytes
// of DeltaParams::seg. A split costs a second walk over every chunk and pays
// where the compute units would be idle: as many segments as keep the first
// walk's workgroups (64 columns of the state or of the transition) resident
// at once, of at least 8 chunks; where no more than three are, the sequences
// need 32 chunks. Measured split / whole in us: 16 heads of 4096 tokens 98 /
// 158, 4 of 32768 215 / 1106, 32 of 8192 255 / 325, 16 of 2304 75 / 93;
// gradients 299 / 425, 662 / 2736, 918 / 1028 and 209 / 259. The shortest that
// are split, 1536 tokens: 8 heads of 64 46 / 52 and 112 / 120, of 128 63 / 65
// and 156 / 167. 32 heads of 128, of which three segments are resident: 1536
// tokens 73 / 71 and 217 / 207, 1792 82 / 81 and 253 / 244, 2048 87 / 91 and
// 275 / 271, 2304 95 / 102 and 319 / 316.
int delta_segments(int64_t T, int64_t N, int64_t HV, int64_t K, int64_t V);
inline int64_t delta_segment_bytes(int64_t N, int64_t HV, int64_t K, int64_t V, int nseg)
{
    return N * HV * (nseg - 1) * (K * V + K * K) * 4;
}
hipError_t launch_delta_wy(const DeltaParams &p, hipStream_t stream);
hipError_t launch_delta_state(const DeltaParams &p, bool ckpt, int ncu, hipStream_t stream);
hipError_t launch_delta_bwd_state(const DeltaParams &p, int ncu, hipStream_t stream);
hipError_t launch_delta_join_bwd(const DeltaParams &p, hipStream_t stream);
hipError_t launch_delta_bwd_grad(const DeltaParams &p, hipStream_t stream);
hipError_t launch_delta_step(const DeltaParams &p, hipStream_t stream);
hipError_t launch_qk_fwd(const QkParams &p, hipStream_t stream);
hipError_t launch_qk_bwd(const QkParams &p, hipStream_t stream);
// Workgroups of the q/k backward (each leaves one row of partial weight gradients).
int qk_bwd_groups(int64_t T, int32_t heads_q, int32_t heads_k, int32_t K);

__host__ __device__ inline SeqRange seq_of(const DeltaParams &p, int64_t n) { return seq_range(p.cu, p.cu64, p.T, n); }

}  // namespace gdn2
