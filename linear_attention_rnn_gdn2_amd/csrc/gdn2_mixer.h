// Internal interface between the C-ABI layer (gdn2_mixer_api.cpp) and the
// gfx950 kernels of what stands around a token mixer's rule: the gated linear
// recurrence, the short causal convolution and the layer norm. Not installed,
// not part of the ABI.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace gdn2 {

enum { E_BF16 = 0, E_F16 = 1, E_F32 = 2 };  // element types of these operators

// Tokens of a tile of the recurrence's gradients: what one workgroup joins (8
// waves of 8 tokens).
constexpr int SCAN_TILE = 64;

struct ScanParams {
    const void *x, *w;      // [T, D] io; w nullptr: 1
    const void *g;          // [T, D] float32 or io
    const void *h0;         // [N, D] float32 or bf16, or nullptr (zero)
    const void *cu;         // [N + 1] int32 or int64, or nullptr (one sequence of T tokens)
    void *out;              // [T, D] io
    void *ht;               // [N, D] float32 or bf16, or nullptr
    int64_t sx, sw, sg, so; // token strides in elements
    int32_t T, N, D;
    int32_t io, g_f32, cu64, h0_bf16, ht_bf16;
    int32_t scale;          // GDN2_SCAN_INPUT_*
    int32_t vec2;           // two channels per lane (token by token, where states may be updated in place: no channel twice)
    int32_t groups;         // whole-sequence groups (0: two passes)
    // workspace: per tile (a range of 8 chunks forward, SCAN_TILE tokens
    // backward) and channel the sum of its g (infinity: a sequence begins in
    // it), its end state from zero, and (backward) the gradient that leaves it
    // towards the token before it; the join replaces the last two by the state
    // that enters the tile and the gradient that reaches it from behind.
    // Forward: the same of every chunk too, as the first pass leaves it.
    float *sums, *end, *back, *chunk_sums, *chunk_end;
    int32_t tiles, chunk;
    // backward
    const void *dout;       // [T, D] io
    const float *dht;       // [N, D] or nullptr
    void *dx, *dw, *dg;     // [T, D]; dw nullptr with w
    float *dh0;             // [N, D] or nullptr
    int64_t sdo, sdx, sdw, sdg;
};

// How a forward call runs: the number of whole-sequence groups (0: in two
// passes over chunks of scan_chunk() tokens, eight of them to a range).
int32_t scan_groups(int64_t T, int64_t N, int64_t D);
int32_t scan_chunk(int64_t T, int64_t D);
inline int64_t scan_ranges(int64_t T, int64_t D)
{
    const int64_t r = 8 * scan_chunk(T, D);
    return (T + r - 1) / r;
}
inline int64_t scan_tiles(int64_t T) { return (T + SCAN_TILE - 1) / SCAN_TILE; }
hipError_t launch_scan_fwd(const ScanParams &p, hipStream_t stream);
hipError_t launch_scan_step(const ScanParams &p, hipStream_t stream);
hipError_t launch_scan_bwd(const ScanParams &p, hipStream_t stream);
hipError_t launch_scan_join(const ScanParams &p, bool bwd, hipStream_t stream);

struct ConvParams {
    const void *x;          // [T, D] io
    const void *weight;     // [D, taps] float32 or io
    const void *bias;       // [D], the weight's type, or nullptr
    const void *s0;         // [N, taps - 1, D] io, or nullptr (zero)
    const void *cu;
    void *out;              // [T, D] io
    void *st;               // [N, taps - 1, D] io, or nullptr
    int64_t sx, so;
    int32_t T, N, D, taps;
    int32_t io, w_f32, cu64, silu, vec2;
    // backward
    const void *dout, *dst; // [T, D], [N, taps - 1, D] io (dst nullptr: zero)
    void *dx, *ds0;         // ds0 nullptr: not written
    void *dweight, *dbias;  // the weight's type, or nullptr
    int64_t sdo, sdx;
    float *part;            // [slices][taps + 1][D]
    int32_t slices, slice_tokens;  // both directions
};

// Tokens that one wave of the convolution (or of its gradients) walks over,
// and the workgroups of four along the tokens (backward each leaves one row of
// partial sums).
int32_t conv_slice_tokens(int64_t T, int64_t D, bool bwd);
int32_t conv_slices(int64_t T, int64_t D, bool bwd);
hipError_t launch_conv_fwd(const ConvParams &p, hipStream_t stream);
hipError_t launch_conv_step(const ConvParams &p, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvParams &p, hipStream_t stream);

struct NormParams {
    const void *x, *z;      // [T, H, D] io; z nullptr: no gate
    const void *w, *b;      // [D] float32 or io, or nullptr
    void *y;                // forward: the output; backward: dx
    const void *dy;         // backward
    void *dz;               // backward with z
    void *dw, *db;          // [D], the types of w and b, or nullptr
    int64_t st[5], sh[5];   // token and head strides of x, z, y, dy, dz
    int64_t rows;
    int32_t H, D;
    int32_t io, w_f32, b_f32, rms;
    float eps;
    float *part;            // backward: [groups][2][D]
    int32_t groups;
};
enum { NORM_X = 0, NORM_Z = 1, NORM_Y = 2, NORM_DY = 3, NORM_DZ = 4 };
constexpr int NORM_MAX_D = 16384;

// 16-byte pieces of a row of D elements.
inline int32_t norm_pieces(int32_t D, int32_t io) { return io == E_F32 ? (D + 3) / 4 : (D + 7) / 8; }
// Workgroups of the norm's backward (each leaves one row of partial sums).
int32_t norm_bwd_groups(int64_t rows, int32_t D, int32_t io);
hipError_t launch_norm_fwd(const NormParams &p, hipStream_t stream);
hipError_t launch_norm_bwd(const NormParams &p, hipStream_t stream);

}  // namespace gdn2
