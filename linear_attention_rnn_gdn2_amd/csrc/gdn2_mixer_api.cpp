// C-ABI entry points of the gated linear recurrence, the short causal
// convolution and the layer norm: argument validation and kernel dispatch.
// Every check runs on the host before anything is enqueued. These entries
// allocate nothing: workspaces are the caller's.
#include <math.h>

#include "../../include/gdn2.h"
#include "gdn2_check.h"
#include "gdn2_mixer.h"

namespace {

using namespace gdn2::api;
using gdn2::ConvParams;
using gdn2::NormParams;
using gdn2::ScanParams;

constexpr int64_t kMaxTokens = INT32_MAX - 65536;  // (the kernels' token indices run past the last one by less)
constexpr int64_t kMaxD = 1 << 24;

int32_t elem(int32_t dtype)
{
    return dtype == GDN2_DTYPE_F32 ? gdn2::E_F32 : dtype == GDN2_DTYPE_F16 ? gdn2::E_F16 : gdn2::E_BF16;
}
int64_t up256(int64_t x) { return (x + 255) & ~(int64_t)255; }

// Whether one launch holds `parts` workgroups of `threads` threads per `per` channels.
bool fits_launch(int64_t parts, int64_t D, int64_t per, int64_t threads)
{
    const int64_t cols = (D + per - 1) / per;
    return parts <= (int64_t)UINT32_MAX / threads && parts * cols <= (int64_t)UINT32_MAX / threads;
}
bool fits_sizes(int64_t T, int64_t N, int64_t D) { return T >= 0 && T <= kMaxTokens && N >= 1 && N <= kMaxTokens && D >= 1 && D <= kMaxD; }
bool fits_scan(int64_t T, int64_t N, int64_t D)
{
    if (!fits_sizes(T, N, D)) return false;
    const int64_t tiles = gdn2::scan_tiles(T), groups = gdn2::scan_groups(T, N, D);
    return fits_launch(tiles > groups ? tiles : groups, D, 64, 512);
}
bool fits_conv(int64_t T, int64_t N, int64_t D) { return fits_sizes(T, N, D) && fits_launch(T / 32 + 1, D, 64, 256); }
bool fits_step(int64_t T, int64_t N, int64_t D) { return fits_sizes(T, N, D) && fits_launch(N, D, 256, 256); }

// An io tensor: its type from bf16, float16, float32 (io 0) or the given one.
int check_io(const gdn2_tensor *t, const char *name, int32_t io, int ndim, const int64_t *want, bool output)
{
    if (!t) return fail(GDN2_ERR_NULL_ARG, "%s is NULL", name);
    if (io == 0 && t->dtype != GDN2_DTYPE_BF16 && t->dtype != GDN2_DTYPE_F16 && t->dtype != GDN2_DTYPE_F32)
        return fail(GDN2_ERR_DTYPE, "%s: expected bf16, float16 or float32, got %s", name, dtype_name(t->dtype));
    if (int rc = check_tensor(t, name, io ? io : t->dtype, -1, ndim, want, VECTORS)) return rc;
    if (!output || numel(t) == 0) return GDN2_OK;
    const bool apart = ndim == 3 ? rows_disjoint(t) : t->shape[0] <= 1 || t->stride[0] >= t->shape[1];
    return apart ? GDN2_OK : fail(GDN2_ERR_LAYOUT, "%s: rows overlap each other", name);
}

int64_t row_stride(const gdn2_tensor *t) { return t->shape[0] > 1 ? t->stride[0] : t->shape[t->ndim - 1]; }

// The number of sequences, after x's own check.
int check_packed(const gdn2_tensor *x, const gdn2_tensor *cu, int64_t *N_out)
{
    int64_t N = 1;
    if (cu) {
        if (int rc = check_tensor(cu, "cu_seqlens", GDN2_DTYPE_I32, GDN2_DTYPE_I64, 1, nullptr)) return rc;
        N = cu->shape[0] - 1;
        if (N < 1) return fail(GDN2_ERR_SHAPE, "cu_seqlens needs at least 2 entries (N >= 1)");
    }
    if (!fits_sizes(x->shape[0], N, x->shape[1]))
        return fail(GDN2_ERR_SHAPE, "T = %lld, N = %lld, D = %lld: T and N may reach %lld, D 1 to %lld", (long long)x->shape[0],
                    (long long)N, (long long)x->shape[1], (long long)kMaxTokens, (long long)kMaxD);
    *N_out = N;
    return GDN2_OK;
}

int too_large(const gdn2_tensor *x, int64_t N)
{
    return fail(GDN2_ERR_SHAPE, "T = %lld, N = %lld, D = %lld exceed the threads of one launch", (long long)x->shape[0], (long long)N,
                (long long)x->shape[1]);
}

// Outputs ts[first ..] against every other tensor; `inplace`: the pair that may be one buffer.
int check_overlaps(const gdn2_tensor *const *ts, const char *const *names, int count, int first, const gdn2_tensor *in = nullptr,
                   const gdn2_tensor *out = nullptr)
{
    for (int o = first; o < count; ++o)
        for (int i = 0; i < count; ++i) {
            if (i == o || (i >= first && i < o)) continue;
            if (in && ts[o] == out && ts[i] == in) continue;
            if (overlaps(ts[o], ts[i])) return fail(GDN2_ERR_ALIAS, "%s overlaps %s", names[o], names[i]);
        }
    return GDN2_OK;
}

int launched(hipError_t e)
{
    return e == hipSuccess ? GDN2_OK : fail(GDN2_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
}

const void *data_of(const gdn2_tensor *t) { return t ? t->data : nullptr; }
void *out_of(const gdn2_tensor *t) { return t ? t->data : nullptr; }

// ------------------------------------------------------------ recurrence --

struct Scan {
    const gdn2_tensor *x, *g, *w, *h0, *cu, *out, *ht;  // (backward: out is d_out, ht d_final_state)
    const gdn2_tensor *dx, *dg, *dw, *dh0;
    const gdn2_scan_options *opts;
};
enum Form { SCAN, STEP, BACK };

// Byte offsets of the recurrence's workspace.
struct ScanSpace {
    int64_t sums, end, back, chunk_sums, chunk_end, total = 0;
    ScanSpace(int64_t T, int64_t D, bool bwd)
    {
        const int64_t tile = up256((bwd ? gdn2::scan_tiles(T) : gdn2::scan_ranges(T, D)) * D * 4);
        const int64_t chunk = bwd ? 0 : up256(8 * gdn2::scan_ranges(T, D) * D * 4);
        auto take = [&](int64_t bytes) {
            const int64_t o = total;
            total += bytes;
            return o;
        };
        sums = take(tile);
        end = take(tile);
        back = take(bwd ? tile : 0);
        chunk_sums = take(chunk);
        chunk_end = take(chunk);
    }
};

int validate(const Scan &a, Form form, void *ws, int64_t ws_bytes, ScanParams *p)
{
    clear_error();
    int32_t scale = GDN2_SCAN_INPUT_NONE;
    if (a.opts) {
        if (a.opts->struct_size < (int32_t)sizeof(gdn2_scan_options))
            return fail(GDN2_ERR_SHAPE, "options: struct_size %d is smaller than %d", a.opts->struct_size, (int)sizeof(gdn2_scan_options));
        scale = a.opts->input_scale;
        if (scale < GDN2_SCAN_INPUT_NONE || scale > GDN2_SCAN_INPUT_UNIT)
            return fail(GDN2_ERR_SHAPE, "options: input_scale must be 0, 1 or 2 (got %d)", scale);
    }
    const bool back = form == BACK;
    int rc;
    if ((rc = check_io(a.x, "x", 0, 2, nullptr, false))) return rc;
    const int32_t io = a.x->dtype;
    const int64_t T = a.x->shape[0], D = a.x->shape[1], rows[2] = {T, D};
    if (!a.g) return fail(GDN2_ERR_NULL_ARG, "g is NULL");
    if ((rc = check_tensor(a.g, "g", GDN2_DTYPE_F32, io, 2, rows, VECTORS))) return rc;
    if (a.w && (rc = check_io(a.w, "w", io, 2, rows, false))) return rc;
    int64_t N;
    if ((rc = check_packed(a.x, a.cu, &N))) return rc;
    if (form == STEP ? !fits_step(T, N, D) : !fits_scan(T, N, D)) return too_large(a.x, N);
    const int64_t states[2] = {N, D};
    if ((rc = check_io(a.out, back ? "d_out" : "out", io, 2, rows, !back))) return rc;
    if (a.h0 && (rc = check_tensor(a.h0, "initial_state", GDN2_DTYPE_F32, GDN2_DTYPE_BF16, 2, states))) return rc;
    if (a.ht && (rc = check_tensor(a.ht, back ? "d_final_state" : "final_state", GDN2_DTYPE_F32, back ? -1 : GDN2_DTYPE_BF16, 2, states)))
        return rc;
    if (back) {
        if ((rc = check_io(a.dx, "dx", io, 2, rows, true))) return rc;
        if ((rc = check_io(a.dg, "dg", a.g->dtype, 2, rows, true))) return rc;
        if (a.dw && !a.w) return fail(GDN2_ERR_NULL_ARG, "dw without w");
        if (a.dw && (rc = check_io(a.dw, "dw", io, 2, rows, true))) return rc;
        if (a.dh0 && (rc = check_tensor(a.dh0, "d_initial_state", GDN2_DTYPE_F32, -1, 2, states))) return rc;
    }
    const gdn2_tensor *fwd[] = {a.x, a.g, a.w, a.h0, a.cu, a.out, a.ht};
    const char *fwd_names[] = {"x", "g", "w", "initial_state", "cu_seqlens", "out", "final_state"};
    const gdn2_tensor *bwd[] = {a.x, a.g, a.w, a.h0, a.cu, a.out, a.ht, a.dx, a.dg, a.dw, a.dh0};
    const char *bwd_names[] = {"x", "g", "w", "initial_state", "cu_seqlens", "d_out", "d_final_state",
                               "dx", "dg", "dw", "d_initial_state"};
    // in place only where a thread holds the state that it writes (token by token)
    const bool inplace = form == STEP && a.h0 && a.ht && a.h0->data == a.ht->data && a.h0->dtype == a.ht->dtype;
    rc = back ? check_overlaps(bwd, bwd_names, 11, 7)
              : check_overlaps(fwd, fwd_names, 7, 5, inplace ? a.h0 : nullptr, inplace ? a.ht : nullptr);
    if (rc || !p) return rc;
    int64_t need = 0;
    if (form == SCAN) need = gdn2_linear_scan_fwd_workspace(T, (int32_t)N, (int32_t)D);
    if (back) need = gdn2_linear_scan_bwd_workspace(T, (int32_t)N, (int32_t)D);
    if ((rc = check_workspace(ws, ws_bytes, need, back ? bwd : fwd, back ? bwd_names : fwd_names, back ? 11 : 7))) return rc;

    *p = ScanParams{};
    p->x = a.x->data;
    p->g = a.g->data;
    p->w = data_of(a.w);
    p->h0 = data_of(a.h0);
    p->cu = data_of(a.cu);
    p->sx = row_stride(a.x);
    p->sg = row_stride(a.g);
    p->sw = a.w ? row_stride(a.w) : 0;
    p->T = (int32_t)T;
    p->N = (int32_t)N;
    p->D = (int32_t)D;
    p->io = elem(io);
    p->g_f32 = a.g->dtype == GDN2_DTYPE_F32;
    p->cu64 = a.cu && a.cu->dtype == GDN2_DTYPE_I64;
    p->h0_bf16 = a.h0 && a.h0->dtype == GDN2_DTYPE_BF16;
    p->scale = scale;
    p->vec2 = form == STEP ? D % 2 == 0 : D >= 2;
    p->chunk = gdn2::scan_chunk(T, D);
    p->tiles = (int32_t)(back ? gdn2::scan_tiles(T) : gdn2::scan_ranges(T, D));
    const ScanSpace space(T, D, back);
    char *b = static_cast<char *>(ws);
    p->sums = reinterpret_cast<float *>(b + space.sums);
    p->end = reinterpret_cast<float *>(b + space.end);
    p->chunk_sums = reinterpret_cast<float *>(b + space.chunk_sums);
    p->chunk_end = reinterpret_cast<float *>(b + space.chunk_end);
    if (back) {
        p->back = reinterpret_cast<float *>(b + space.back);
        p->dout = a.out->data;
        p->sdo = row_stride(a.out);
        p->dht = static_cast<const float *>(data_of(a.ht));
        p->dx = a.dx->data;
        p->dg = a.dg->data;
        p->dw = out_of(a.dw);
        p->dh0 = static_cast<float *>(out_of(a.dh0));
        p->sdx = row_stride(a.dx);
        p->sdg = row_stride(a.dg);
        p->sdw = a.dw ? row_stride(a.dw) : 0;
    } else {
        p->out = a.out->data;
        p->so = row_stride(a.out);
        p->ht = out_of(a.ht);
        p->ht_bf16 = a.ht && a.ht->dtype == GDN2_DTYPE_BF16;
        p->groups = form == SCAN ? gdn2::scan_groups(T, N, D) : 0;
    }
    return GDN2_OK;
}

// ----------------------------------------------------------- convolution --

struct Conv {
    const gdn2_tensor *x, *weight, *bias, *s0, *cu, *out, *st;  // (backward: out is d_out, st d_final_state)
    const gdn2_tensor *dx, *dweight, *dbias, *ds0;
    const gdn2_conv_options *opts;
};

int validate(const Conv &a, Form form, void *ws, int64_t ws_bytes, ConvParams *p)
{
    clear_error();
    int32_t act = GDN2_CONV_SILU;
    if (a.opts) {
        if (a.opts->struct_size < (int32_t)sizeof(gdn2_conv_options))
            return fail(GDN2_ERR_SHAPE, "options: struct_size %d is smaller than %d", a.opts->struct_size, (int)sizeof(gdn2_conv_options));
        act = a.opts->activation;
        if (act != GDN2_CONV_NONE && act != GDN2_CONV_SILU)
            return fail(GDN2_ERR_SHAPE, "options: activation must be 0 or 1 (got %d)", act);
    }
    const bool back = form == BACK;
    int rc;
    if ((rc = check_io(a.x, "x", 0, 2, nullptr, false))) return rc;
    const int32_t io = a.x->dtype;
    const int64_t T = a.x->shape[0], D = a.x->shape[1], rows[2] = {T, D}, wants[2] = {D, -1};
    if (!a.weight) return fail(GDN2_ERR_NULL_ARG, "weight is NULL");
    if ((rc = check_tensor(a.weight, "weight", GDN2_DTYPE_F32, io, 2, wants))) return rc;
    const int64_t K = a.weight->shape[1];
    if (K < 2 || K > 4) return fail(GDN2_ERR_UNSUPPORTED, "weight: %lld taps; 2, 3 and 4 are supported", (long long)K);
    const int32_t wt = a.weight->dtype;
    if (a.bias && (rc = check_tensor(a.bias, "bias", wt, -1, 1, &D))) return rc;
    int64_t N;
    if ((rc = check_packed(a.x, a.cu, &N))) return rc;
    if (form == STEP ? !fits_step(T, N, D) : !fits_conv(T, N, D)) return too_large(a.x, N);
    const int64_t states[3] = {N, K - 1, D};
    if ((rc = check_io(a.out, back ? "d_out" : "out", io, 2, rows, !back))) return rc;
    if (a.s0 && (rc = check_tensor(a.s0, "initial_state", io, -1, 3, states))) return rc;
    if (a.st && (rc = check_tensor(a.st, back ? "d_final_state" : "final_state", io, -1, 3, states))) return rc;
    if (back) {
        if ((rc = check_io(a.dx, "dx", io, 2, rows, true))) return rc;
        if (a.dweight && (rc = check_tensor(a.dweight, "dweight", wt, -1, 2, a.weight->shape))) return rc;
        if (a.dbias && !a.bias) return fail(GDN2_ERR_NULL_ARG, "dbias without bias");
        if (a.dbias && (rc = check_tensor(a.dbias, "dbias", wt, -1, 1, &D))) return rc;
        if (a.ds0 && (rc = check_tensor(a.ds0, "d_initial_state", io, -1, 3, states))) return rc;
    }
    const gdn2_tensor *fwd[] = {a.x, a.weight, a.bias, a.s0, a.cu, a.out, a.st};
    const char *fwd_names[] = {"x", "weight", "bias", "initial_state", "cu_seqlens", "out", "final_state"};
    const gdn2_tensor *bwd[] = {a.x, a.weight, a.bias, a.s0, a.cu, a.out, a.st, a.dx, a.dweight, a.dbias, a.ds0};
    const char *bwd_names[] = {"x", "weight", "bias", "initial_state", "cu_seqlens", "d_out", "d_final_state",
                               "dx", "dweight", "dbias", "d_initial_state"};
    const bool inplace = form == STEP && a.s0 && a.st && a.s0->data == a.st->data;
    rc = back ? check_overlaps(bwd, bwd_names, 11, 7)
              : check_overlaps(fwd, fwd_names, 7, 5, inplace ? a.s0 : nullptr, inplace ? a.st : nullptr);
    if (rc || !p) return rc;
    const bool sums = back && (a.dweight || a.dbias);
    if (sums && (rc = check_workspace(ws, ws_bytes, gdn2_short_conv_bwd_workspace(T, (int32_t)D, (int32_t)K), bwd, bwd_names, 11)))
        return rc;

    *p = ConvParams{};
    p->x = a.x->data;
    p->weight = a.weight->data;
    p->bias = data_of(a.bias);
    p->s0 = data_of(a.s0);
    p->cu = data_of(a.cu);
    p->sx = row_stride(a.x);
    p->T = (int32_t)T;
    p->N = (int32_t)N;
    p->D = (int32_t)D;
    p->taps = (int32_t)K;
    p->io = elem(io);
    p->w_f32 = wt == GDN2_DTYPE_F32;
    p->cu64 = a.cu && a.cu->dtype == GDN2_DTYPE_I64;
    p->silu = act == GDN2_CONV_SILU;
    p->slice_tokens = gdn2::conv_slice_tokens(T, D, back);
    p->slices = gdn2::conv_slices(T, D, back);
    p->vec2 = form == STEP ? D % 2 == 0 : D >= 2;
    if (back) {
        p->dout = a.out->data;
        p->sdo = row_stride(a.out);
        p->dst = data_of(a.st);
        p->dx = a.dx->data;
        p->sdx = row_stride(a.dx);
        p->ds0 = out_of(a.ds0);
        p->dweight = out_of(a.dweight);
        p->dbias = out_of(a.dbias);
        p->part = sums && T > 0 ? static_cast<float *>(ws) : nullptr;  // (without tokens there is nothing to sum, and no room is asked for)
    } else {
        p->out = a.out->data;
        p->so = row_stride(a.out);
        p->st = out_of(a.st);
    }
    return GDN2_OK;
}

// ------------------------------------------------------------------ norm --

struct Norm {
    const gdn2_tensor *x, *z, *w, *b, *dy, *y, *dz, *dw, *db;  // y: out or dx
    const gdn2_norm_options *opts;
};

bool fits_norm(int64_t T, int64_t H, int64_t D)
{
    return T >= 0 && H >= 1 && D >= 1 && D <= gdn2::NORM_MAX_D && H <= INT32_MAX && T <= INT32_MAX && T * H <= INT32_MAX;
}

int validate(const Norm &a, bool back, void *ws, int64_t ws_bytes, NormParams *p)
{
    clear_error();
    int32_t norm = GDN2_NORM_LAYER;
    float eps = 0.0f;
    if (a.opts) {
        if (a.opts->struct_size < (int32_t)sizeof(gdn2_norm_options))
            return fail(GDN2_ERR_SHAPE, "options: struct_size %d is smaller than %d", a.opts->struct_size, (int)sizeof(gdn2_norm_options));
        norm = a.opts->norm;
        eps = a.opts->eps;
    }
    if (norm != GDN2_NORM_LAYER && norm != GDN2_NORM_RMS) return fail(GDN2_ERR_SHAPE, "options: norm must be 0 or 1 (got %d)", norm);
    if (!(eps >= 0.0f) || isinf(eps)) return fail(GDN2_ERR_SHAPE, "options: eps must be finite and not negative");
    if (eps == 0.0f) eps = norm == GDN2_NORM_RMS ? 1e-6f : 1e-5f;
    int rc;
    if ((rc = check_io(a.x, "x", 0, 3, nullptr, false))) return rc;
    const int32_t io = a.x->dtype;
    const int64_t T = a.x->shape[0], H = a.x->shape[1], D = a.x->shape[2];
    if (D < 1 || D > gdn2::NORM_MAX_D)
        return fail(GDN2_ERR_UNSUPPORTED, "D = %lld not supported; rows of 1 to %d elements are", (long long)D, gdn2::NORM_MAX_D);
    if (!fits_norm(T, H, D)) return fail(GDN2_ERR_SHAPE, "T * H = %lld * %lld rows: 2^31 - 1 at most, of at least one head", (long long)T, (long long)H);
    if (a.z && (rc = check_io(a.z, "gate", io, 3, a.x->shape, false))) return rc;
    if (a.w && (rc = check_tensor(a.w, "weight", GDN2_DTYPE_F32, io, 1, &D))) return rc;
    if (a.b && (rc = check_tensor(a.b, "bias", GDN2_DTYPE_F32, io, 1, &D))) return rc;
    if (back && (rc = check_io(a.dy, "d_out", io, 3, a.x->shape, false))) return rc;
    if ((rc = check_io(a.y, back ? "dx" : "out", io, 3, a.x->shape, true))) return rc;
    if (back) {
        if (a.z && (rc = check_io(a.dz, "dgate", io, 3, a.x->shape, true))) return rc;
        if (!a.z && a.dz) return fail(GDN2_ERR_NULL_ARG, "dgate without gate");
        if (a.dw && !a.w) return fail(GDN2_ERR_NULL_ARG, "dweight without weight");
        if (a.db && !a.b) return fail(GDN2_ERR_NULL_ARG, "dbias without bias");
        if (a.dw && (rc = check_tensor(a.dw, "dweight", a.w->dtype, -1, 1, &D))) return rc;
        if (a.db && (rc = check_tensor(a.db, "dbias", a.b->dtype, -1, 1, &D))) return rc;
    }
    const gdn2_tensor *ts[] = {a.x, a.z, a.w, a.b, a.dy, a.y, a.dz, a.dw, a.db};
    const char *names[] = {"x", "gate", "weight", "bias", "d_out", back ? "dx" : "out", "dgate", "dweight", "dbias"};
    if ((rc = check_overlaps(ts, names, 9, 5)) || !p) return rc;
    const bool sums = a.dw || a.db;
    if (sums && (rc = check_workspace(ws, ws_bytes, gdn2_layer_norm_bwd_workspace(T, (int32_t)H, (int32_t)D), ts, names, 9))) return rc;

    *p = NormParams{};
    const gdn2_tensor *io_ts[5] = {a.x, a.z, a.y, a.dy, a.dz};
    bool flat = true;  // every tensor's rows one stride apart
    for (int i = 0; i < 5; ++i) {
        if (!io_ts[i]) continue;
        p->st[i] = T > 1 ? io_ts[i]->stride[0] : 0;
        p->sh[i] = H > 1 ? io_ts[i]->stride[1] : 0;
        flat = flat && (H == 1 || T == 1 || p->st[i] == H * p->sh[i]);
    }
    if (flat && H > 1)
        for (int i = 0; i < 5; ++i) p->st[i] = p->sh[i];
    p->x = a.x->data;
    p->z = data_of(a.z);
    p->w = data_of(a.w);
    p->b = data_of(a.b);
    p->y = a.y->data;
    p->dy = data_of(a.dy);
    p->dz = out_of(a.dz);
    p->dw = out_of(a.dw);
    p->db = out_of(a.db);
    p->rows = T * H;
    p->H = flat ? 1 : (int32_t)H;
    p->D = (int32_t)D;
    p->io = elem(io);
    p->w_f32 = a.w && a.w->dtype == GDN2_DTYPE_F32;
    p->b_f32 = a.b && a.b->dtype == GDN2_DTYPE_F32;
    p->rms = norm == GDN2_NORM_RMS;
    p->eps = eps;
    p->groups = back ? gdn2::norm_bwd_groups(p->rows, p->D, p->io) : 0;
    p->part = sums ? static_cast<float *>(ws) : nullptr;
    return GDN2_OK;
}

}  // namespace

extern "C" {

int64_t gdn2_linear_scan_fwd_workspace(int64_t T, int32_t N, int32_t D)
{
    if (T <= 0 || !fits_scan(T, N, D) || gdn2::scan_groups(T, N, D) != 0) return 0;
    return ScanSpace(T, D, false).total;
}

int64_t gdn2_linear_scan_bwd_workspace(int64_t T, int32_t N, int32_t D)
{
    if (T <= 0 || !fits_scan(T, N, D) || gdn2::scan_tiles(T) <= 1) return 0;
    return ScanSpace(T, D, true).total;
}

int gdn2_linear_scan_fwd(const gdn2_tensor *x, const gdn2_tensor *g, const gdn2_tensor *w, const gdn2_tensor *initial_state,
                         const gdn2_tensor *cu_seqlens, const gdn2_tensor *out, const gdn2_tensor *final_state,
                         const gdn2_scan_options *opts, void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    ScanParams p;
    if (int rc = validate(Scan{x, g, w, initial_state, cu_seqlens, out, final_state, nullptr, nullptr, nullptr, nullptr, opts}, SCAN,
                          workspace, workspace_bytes, &p))
        return rc;
    return launched(gdn2::launch_scan_fwd(p, stream));
}

int gdn2_linear_scan_fwd_check(const gdn2_tensor *x, const gdn2_tensor *g, const gdn2_tensor *w, const gdn2_tensor *initial_state,
                               const gdn2_tensor *cu_seqlens, const gdn2_tensor *out, const gdn2_tensor *final_state,
                               const gdn2_scan_options *opts)
{
    return validate(Scan{x, g, w, initial_state, cu_seqlens, out, final_state, nullptr, nullptr, nullptr, nullptr, opts}, SCAN, nullptr,
                    0, nullptr);
}

int gdn2_linear_scan_recurrent_fwd(const gdn2_tensor *x, const gdn2_tensor *g, const gdn2_tensor *w,
                                   const gdn2_tensor *initial_state, const gdn2_tensor *cu_seqlens, const gdn2_tensor *out,
                                   const gdn2_tensor *final_state, const gdn2_scan_options *opts, hipStream_t stream)
{
    ScanParams p;
    if (int rc = validate(Scan{x, g, w, initial_state, cu_seqlens, out, final_state, nullptr, nullptr, nullptr, nullptr, opts}, STEP,
                          nullptr, 0, &p))
        return rc;
    return launched(gdn2::launch_scan_step(p, stream));
}

int gdn2_linear_scan_recurrent_fwd_check(const gdn2_tensor *x, const gdn2_tensor *g, const gdn2_tensor *w,
                                         const gdn2_tensor *initial_state, const gdn2_tensor *cu_seqlens, const gdn2_tensor *out,
                                         const gdn2_tensor *final_state, const gdn2_scan_options *opts)
{
    return validate(Scan{x, g, w, initial_state, cu_seqlens, out, final_state, nullptr, nullptr, nullptr, nullptr, opts}, STEP, nullptr,
                    0, nullptr);
}

int gdn2_linear_scan_bwd(const gdn2_tensor *x, const gdn2_tensor *g, const gdn2_tensor *w, const gdn2_tensor *initial_state,
                         const gdn2_tensor *cu_seqlens, const gdn2_tensor *d_out, const gdn2_tensor *d_final_state,
                         const gdn2_tensor *dx, const gdn2_tensor *dg, const gdn2_tensor *dw, const gdn2_tensor *d_initial_state,
                         const gdn2_scan_options *opts, void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    ScanParams p;
    if (int rc = validate(Scan{x, g, w, initial_state, cu_seqlens, d_out, d_final_state, dx, dg, dw, d_initial_state, opts}, BACK,
                          workspace, workspace_bytes, &p))
        return rc;
    return launched(gdn2::launch_scan_bwd(p, stream));
}

int gdn2_linear_scan_bwd_check(const gdn2_tensor *x, const gdn2_tensor *g, const gdn2_tensor *w, const gdn2_tensor *initial_state,
                               const gdn2_tensor *cu_seqlens, const gdn2_tensor *d_out, const gdn2_tensor *d_final_state,
                               const gdn2_tensor *dx, const gdn2_tensor *dg, const gdn2_tensor *dw,
                               const gdn2_tensor *d_initial_state, const gdn2_scan_options *opts)
{
    return validate(Scan{x, g, w, initial_state, cu_seqlens, d_out, d_final_state, dx, dg, dw, d_initial_state, opts}, BACK, nullptr, 0,
                    nullptr);
}

int gdn2_short_conv_fwd(const gdn2_tensor *x, const gdn2_tensor *weight, const gdn2_tensor *bias, const gdn2_tensor *initial_state,
                        const gdn2_tensor *cu_seqlens, const gdn2_tensor *out, const gdn2_tensor *final_state,
                        const gdn2_conv_options *opts, hipStream_t stream)
{
    ConvParams p;
    if (int rc = validate(Conv{x, weight, bias, initial_state, cu_seqlens, out, final_state, nullptr, nullptr, nullptr, nullptr, opts},
                          SCAN, nullptr, 0, &p))
        return rc;
    return launched(gdn2::launch_conv_fwd(p, stream));
}

int gdn2_short_conv_fwd_check(const gdn2_tensor *x, const gdn2_tensor *weight, const gdn2_tensor *bias,
                              const gdn2_tensor *initial_state, const gdn2_tensor *cu_seqlens, const gdn2_tensor *out,
                              const gdn2_tensor *final_state, const gdn2_conv_options *opts)
{
    return validate(Conv{x, weight, bias, initial_state, cu_seqlens, out, final_state, nullptr, nullptr, nullptr, nullptr, opts}, SCAN,
                    nullptr, 0, nullptr);
}

int gdn2_short_conv_recurrent_fwd(const gdn2_tensor *x, const gdn2_tensor *weight, const gdn2_tensor *bias,
                                  const gdn2_tensor *initial_state, const gdn2_tensor *cu_seqlens, const gdn2_tensor *out,
                                  const gdn2_tensor *final_state, const gdn2_conv_options *opts, hipStream_t stream)
{
    ConvParams p;
    if (int rc = validate(Conv{x, weight, bias, initial_state, cu_seqlens, out, final_state, nullptr, nullptr, nullptr, nullptr, opts},
                          STEP, nullptr, 0, &p))
        return rc;
    return launched(gdn2::launch_conv_step(p, stream));
}

int gdn2_short_conv_recurrent_fwd_check(const gdn2_tensor *x, const gdn2_tensor *weight, const gdn2_tensor *bias,
                                        const gdn2_tensor *initial_state, const gdn2_tensor *cu_seqlens, const gdn2_tensor *out,
                                        const gdn2_tensor *final_state, const gdn2_conv_options *opts)
{
    return validate(Conv{x, weight, bias, initial_state, cu_seqlens, out, final_state, nullptr, nullptr, nullptr, nullptr, opts}, STEP,
                    nullptr, 0, nullptr);
}

int64_t gdn2_short_conv_bwd_workspace(int64_t T, int32_t D, int32_t K)
{
    if (T <= 0 || K < 2 || K > 4 || !fits_conv(T, 1, D)) return 0;
    return up256(gdn2::conv_slices(T, D, true) * (int64_t)(K + 1) * D * 4);
}

int gdn2_short_conv_bwd(const gdn2_tensor *x, const gdn2_tensor *weight, const gdn2_tensor *bias, const gdn2_tensor *initial_state,
                        const gdn2_tensor *cu_seqlens, const gdn2_tensor *d_out, const gdn2_tensor *d_final_state,
                        const gdn2_tensor *dx, const gdn2_tensor *dweight, const gdn2_tensor *dbias,
                        const gdn2_tensor *d_initial_state, const gdn2_conv_options *opts, void *workspace, int64_t workspace_bytes,
                        hipStream_t stream)
{
    ConvParams p;
    if (int rc = validate(Conv{x, weight, bias, initial_state, cu_seqlens, d_out, d_final_state, dx, dweight, dbias, d_initial_state, opts},
                          BACK, workspace, workspace_bytes, &p))
        return rc;
    return launched(gdn2::launch_conv_bwd(p, stream));
}

int gdn2_short_conv_bwd_check(const gdn2_tensor *x, const gdn2_tensor *weight, const gdn2_tensor *bias,
                              const gdn2_tensor *initial_state, const gdn2_tensor *cu_seqlens, const gdn2_tensor *d_out,
                              const gdn2_tensor *d_final_state, const gdn2_tensor *dx, const gdn2_tensor *dweight,
                              const gdn2_tensor *dbias, const gdn2_tensor *d_initial_state, const gdn2_conv_options *opts)
{
    return validate(Conv{x, weight, bias, initial_state, cu_seqlens, d_out, d_final_state, dx, dweight, dbias, d_initial_state, opts},
                    BACK, nullptr, 0, nullptr);
}

int gdn2_layer_norm_fwd(const gdn2_tensor *x, const gdn2_tensor *gate, const gdn2_tensor *weight, const gdn2_tensor *bias,
                        const gdn2_tensor *out, const gdn2_norm_options *opts, hipStream_t stream)
{
    NormParams p;
    if (int rc = validate(Norm{x, gate, weight, bias, nullptr, out, nullptr, nullptr, nullptr, opts}, false, nullptr, 0, &p)) return rc;
    return launched(gdn2::launch_norm_fwd(p, stream));
}

int gdn2_layer_norm_fwd_check(const gdn2_tensor *x, const gdn2_tensor *gate, const gdn2_tensor *weight, const gdn2_tensor *bias,
                              const gdn2_tensor *out, const gdn2_norm_options *opts)
{
    return validate(Norm{x, gate, weight, bias, nullptr, out, nullptr, nullptr, nullptr, opts}, false, nullptr, 0, nullptr);
}

int64_t gdn2_layer_norm_bwd_workspace(int64_t T, int32_t H, int32_t D)
{
    if (T <= 0 || !fits_norm(T, H, D)) return 0;
    const int64_t a = gdn2::norm_bwd_groups(T * H, D, gdn2::E_BF16), b = gdn2::norm_bwd_groups(T * H, D, gdn2::E_F32);
    const int64_t most = a > b ? a : b;  // the more that either width of an element takes
    return up256(most * 2 * D * 4);
}

int gdn2_layer_norm_bwd(const gdn2_tensor *x, const gdn2_tensor *gate, const gdn2_tensor *weight, const gdn2_tensor *bias,
                        const gdn2_tensor *d_out, const gdn2_tensor *dx, const gdn2_tensor *dgate, const gdn2_tensor *dweight,
                        const gdn2_tensor *dbias, const gdn2_norm_options *opts, void *workspace, int64_t workspace_bytes,
                        hipStream_t stream)
{
    NormParams p;
    if (int rc = validate(Norm{x, gate, weight, bias, d_out, dx, dgate, dweight, dbias, opts}, true, workspace, workspace_bytes, &p))
        return rc;
    return launched(gdn2::launch_norm_bwd(p, stream));
}

int gdn2_layer_norm_bwd_check(const gdn2_tensor *x, const gdn2_tensor *gate, const gdn2_tensor *weight, const gdn2_tensor *bias,
                              const gdn2_tensor *d_out, const gdn2_tensor *dx, const gdn2_tensor *dgate,
                              const gdn2_tensor *dweight, const gdn2_tensor *dbias, const gdn2_norm_options *opts)
{
    return validate(Norm{x, gate, weight, bias, d_out, dx, dgate, dweight, dbias, opts}, true, nullptr, 0, nullptr);
}

}  // extern "C"
