// C-ABI entry points of the scalar-gated delta rule and of the q/k
// preparation: argument validation and kernel dispatch. As for the
// channel-wise rule, every check runs on the host before anything is
// enqueued. These entries allocate nothing: workspaces are the caller's.
#include <math.h>
#include <stddef.h>

#include "../../include/gdn2.h"
#include "gdn2_check.h"
#include "gdn2_delta.h"

namespace {

using namespace gdn2::api;
using gdn2::DeltaParams;
using gdn2::DeltaRecord;
using gdn2::QkParams;

// One kernel launch holds up to 2^32 - 1 threads: 512 per (chunk, value head)
// and 768 per (sequence, value head).
constexpr int64_t kMaxItems = UINT32_MAX / 768;

int check_io(const gdn2_tensor *t, const char *name, int32_t io, const int64_t *want, Layout layout)
{
    return check_tensor(t, name, io, -1, 3, want, layout);
}

int check_g(const gdn2_tensor *g, const char *name, const int64_t *want, Layout layout)
{
    if (g->dtype != GDN2_DTYPE_F32 && g->dtype != GDN2_DTYPE_BF16 && g->dtype != GDN2_DTYPE_F16)
        return fail(GDN2_ERR_DTYPE, "%s: expected float32, bf16 or float16, got %s", name, dtype_name(g->dtype));
    return check_tensor(g, name, g->dtype, -1, 2, want, layout);
}

int32_t g_type(const gdn2_tensor *g)
{
    if (!g || g->dtype == GDN2_DTYPE_F32) return gdn2::G_F32;
    return g->dtype == GDN2_DTYPE_BF16 ? gdn2::G_BF16 : gdn2::G_F16;
}

// Whether one launch holds a call's chains and chunks (T within int32, N, HV > 0).
bool fits_grid(int64_t T, int64_t N, int64_t HV)
{
    return N <= kMaxItems && HV <= kMaxItems && N * HV <= kMaxItems && gdn2::slot_count(T, N) * HV <= kMaxItems;
}

// (64 rows of the value heads are addressed with 32-bit byte offsets in the backward)
bool fits_rows(int64_t HV, int64_t V) { return HV * V * 128 <= INT32_MAX; }

// Sizes shared by the rule's entries, after q's, k's and v's own checks.
int check_sizes(const gdn2_tensor *q, const gdn2_tensor *v, const gdn2_tensor *cu, int64_t *N_out)
{
    const int64_t T = q->shape[0], H = q->shape[1], K = q->shape[2], HV = v->shape[1], V = v->shape[2];
    if (H < 1 || HV < H || HV % H != 0)
        return fail(GDN2_ERR_HEADS, "value heads (%lld) must be a positive multiple of q/k heads (%lld)", (long long)HV,
                    (long long)H);
    if ((K != 64 && K != 128) || (V != 64 && V != 128))
        return fail(GDN2_ERR_UNSUPPORTED, "(K, V) = (%lld, %lld) not supported; K and V must each be 64 or 128", (long long)K,
                    (long long)V);
    if (T > INT32_MAX) return fail(GDN2_ERR_SHAPE, "T = %lld exceeds the int32 range of cu_seqlens", (long long)T);
    int64_t N = 1;
    if (cu) {
        if (int rc = check_tensor(cu, "cu_seqlens", GDN2_DTYPE_I32, GDN2_DTYPE_I64, 1, nullptr)) return rc;
        N = cu->shape[0] - 1;
        if (N < 1) return fail(GDN2_ERR_SHAPE, "cu_seqlens needs at least 2 entries (N >= 1)");
        if (!cu->data) return fail(GDN2_ERR_NULL_ARG, "cu_seqlens: data is NULL");
    }
    if (!fits_grid(T, N, HV))
        return fail(GDN2_ERR_SHAPE, "N * HV or the chunk count times HV exceeds the grid limit (%lld)", (long long)kMaxItems);
    *N_out = N;
    return GDN2_OK;
}

int64_t tok_stride(const gdn2_tensor *t) { return t->shape[0] > 1 ? t->stride[0] : t->ndim == 3 ? t->shape[2] : 0; }
int64_t head_stride(const gdn2_tensor *t) { return t->shape[1] > 1 ? t->stride[1] : 0; }

int64_t up256(int64_t x) { return (x + 255) & ~(int64_t)255; }

// The forward's workspace: the records, then a split run's segments (the
// most that any K and V of this T, N and HV take).
int64_t fwd_records(int64_t T, int64_t N, int64_t HV) { return gdn2::slot_count(T, N) * HV * DeltaRecord::BYTES; }
int64_t fwd_segments(int64_t T, int64_t N, int64_t HV)
{
    int64_t most = 0;
    for (int64_t K = 64; K <= 128; K += 64)
        for (int64_t V = 64; V <= 128; V += 64) {
            const int64_t b = gdn2::delta_segment_bytes(N, HV, K, V, gdn2::delta_segments(T, N, HV, K, V));
            if (b > most) most = b;
        }
    return most;
}

struct DeltaFwd {
    const gdn2_tensor *q, *k, *v, *g, *beta;
    float scale;
    const gdn2_tensor *h0, *cu, *out, *ht;
    const gdn2_fwd_options *opts;
};

int validate(const DeltaFwd &a, bool chunked, void *ws, int64_t ws_bytes, DeltaParams *p)
{
    clear_error();
    Options o;
    int rc;
    if ((rc = read_options(a.opts, &o))) return rc;
    if (chunked && o.split > 0)
        return fail(GDN2_ERR_UNSUPPORTED, "seq_split_chunks %d: the scalar-gated rule takes 0 (automatic) or -1 (whole sequences)", o.split);
    if (!a.q) return fail(GDN2_ERR_NULL_ARG, "q is NULL");
    if (!a.k) return fail(GDN2_ERR_NULL_ARG, "k is NULL");
    if (!a.v) return fail(GDN2_ERR_NULL_ARG, "v is NULL");
    if (!a.out) return fail(GDN2_ERR_NULL_ARG, "out is NULL");
    if ((rc = check_tensor(a.q, "q", GDN2_DTYPE_BF16, GDN2_DTYPE_F16, 3, nullptr, ROWS))) return rc;
    const int32_t io = a.q->dtype;
    const int64_t T = a.q->shape[0], H = a.q->shape[1], K = a.q->shape[2];
    const int64_t qs[3] = {T, H, K}, v_any[3] = {T, -1, -1};
    if ((rc = check_io(a.k, "k", io, qs, ROWS))) return rc;
    if ((rc = check_io(a.v, "v", io, v_any, ROWS))) return rc;
    int64_t N;
    if ((rc = check_sizes(a.q, a.v, a.cu, &N))) return rc;
    const int64_t HV = a.v->shape[1], V = a.v->shape[2];
    const int64_t gs[2] = {T, HV}, vs[3] = {T, HV, V}, ss[4] = {N, HV, o.vmajor ? V : K, o.vmajor ? K : V};
    if (a.g && (rc = check_g(a.g, "g", gs, GATES))) return rc;
    if (a.beta && (rc = check_tensor(a.beta, "beta", io, -1, 2, gs, GATES))) return rc;
    if ((rc = check_io(a.out, "out", io, vs, ROWS))) return rc;
    if (!rows_disjoint(a.out)) return fail(GDN2_ERR_LAYOUT, "out: rows overlap each other");
    if (a.h0 && (rc = check_tensor(a.h0, "initial_state", GDN2_DTYPE_F32, GDN2_DTYPE_BF16, 4, ss))) return rc;
    if (a.ht && (rc = check_tensor(a.ht, "final_state", GDN2_DTYPE_F32, GDN2_DTYPE_BF16, 4, ss))) return rc;

    const gdn2_tensor *ts[] = {a.q, a.k, a.v, a.g, a.beta, a.h0, a.cu, a.out, a.ht};
    const char *names[] = {"q", "k", "v", "g", "beta", "initial_state", "cu_seqlens", "out", "final_state"};
    // in place only where a wave holds every element it writes before it writes (token by token)
    const bool inplace = !chunked && a.h0 && a.ht && a.h0->data == a.ht->data && a.h0->dtype == a.ht->dtype;
    for (int i = 0; i < 7; ++i) {
        if (overlaps(a.out, ts[i])) return fail(GDN2_ERR_ALIAS, "out overlaps %s", names[i]);
        if (overlaps(a.ht, ts[i]) && !(inplace && ts[i] == a.h0)) return fail(GDN2_ERR_ALIAS, "final_state overlaps %s", names[i]);
    }
    if (overlaps(a.out, a.ht)) return fail(GDN2_ERR_ALIAS, "out overlaps final_state");
    if (!p) return GDN2_OK;
    if (chunked && (rc = check_workspace(ws, ws_bytes, gdn2_delta_chunk_fwd_workspace(T, (int32_t)N, (int32_t)HV), ts, names, 9)))
        return rc;

    *p = DeltaParams{};
    p->q = static_cast<const uint16_t *>(a.q->data);
    p->k = static_cast<const uint16_t *>(a.k->data);
    p->v = static_cast<const uint16_t *>(a.v->data);
    p->g = a.g ? a.g->data : nullptr;
    p->beta = a.beta ? static_cast<const uint16_t *>(a.beta->data) : nullptr;
    p->h0 = a.h0 ? static_cast<const float *>(a.h0->data) : nullptr;
    p->cu = a.cu ? a.cu->data : nullptr;
    p->out = static_cast<uint16_t *>(a.out->data);
    p->ht = a.ht ? static_cast<float *>(a.ht->data) : nullptr;
    p->T = T;
    p->N = (int32_t)N;
    p->H = (int32_t)H;
    p->HV = (int32_t)HV;
    p->K = (int32_t)K;
    p->V = (int32_t)V;
    p->scale = a.scale == 0.0f ? (float)(1.0 / sqrt((double)K)) : a.scale;
    p->io = io == GDN2_DTYPE_F16 ? gdn2::IO_F16 : gdn2::IO_BF16;
    p->gtype = g_type(a.g);
    p->cu64 = a.cu && a.cu->dtype == GDN2_DTYPE_I64;
    p->h0_bf16 = a.h0 && a.h0->dtype == GDN2_DTYPE_BF16;
    p->ht_bf16 = a.ht && a.ht->dtype == GDN2_DTYPE_BF16;
    p->sq = tok_stride(a.q);
    p->sk = tok_stride(a.k);
    p->sv = tok_stride(a.v);
    p->so = tok_stride(a.out);
    p->sg = a.g ? tok_stride(a.g) : 0;
    p->sb = a.beta ? tok_stride(a.beta) : 0;
    p->hsq = head_stride(a.q);
    p->hsk = head_stride(a.k);
    p->hsv = head_stride(a.v);
    p->hso = head_stride(a.out);
    p->hsg = a.g ? head_stride(a.g) : 0;
    p->hsb = a.beta ? head_stride(a.beta) : 0;
    p->state_vmajor = o.vmajor;
    p->qk_l2norm = o.l2norm;
    p->nslots = (int32_t)gdn2::slot_count(T, N);
    p->rec = static_cast<char *>(ws);
    p->low_p = p->io == gdn2::IO_F16;
    p->nseg = chunked && o.split == 0 && T > 0 ? gdn2::delta_segments(T, N, HV, K, V) : 1;
    p->seg = p->nseg > 1 ? reinterpret_cast<float *>(p->rec + fwd_records(T, N, HV)) : nullptr;
    return GDN2_OK;
}

struct DeltaBwd {
    const gdn2_tensor *q, *k, *v, *g, *beta;
    float scale;
    const gdn2_tensor *h0, *cu, *dout, *dht, *dq, *dk, *dv, *dg, *dbeta, *dh0;
};

// Byte offsets of the backward's workspace.
struct BwdSpace {
    int64_t rec, s, ds, u, y, mx, dq, dk, seg, rseg, total;
    int nseg;
    BwdSpace(int64_t T, int64_t N, int64_t H, int64_t HV, int64_t K, int64_t V)
    {
        const int64_t items = gdn2::slot_count(T, N) * HV;
        int64_t at = 0;
        auto take = [&](int64_t bytes) {
            const int64_t o = at;
            at += up256(bytes);
            return o;
        };
        rec = take(T > 0 ? items * DeltaRecord::BYTES : 0);
        s = take(T > 0 ? items * K * V * 4 : 0);
        ds = take(T > 0 ? items * K * V * 4 : 0);
        u = take(T > 0 ? items * 64 * V * 4 : 0);
        y = take(T > 0 ? items * 64 * V * 4 : 0);
        mx = take(T > 0 ? items * (V / 16) * 32 : 0);
        dq = take(H != HV ? T * HV * K * 4 : 0);
        dk = take(H != HV ? T * HV * K * 4 : 0);
        nseg = gdn2::delta_segments(T, N, HV, K, V);
        seg = take(gdn2::delta_segment_bytes(N, HV, K, V, nseg));
        rseg = take(N * HV * (nseg - 1) * K * V * 4);
        total = at;
    }
};

int validate(const DeltaBwd &a, void *ws, int64_t ws_bytes, DeltaParams *p)
{
    clear_error();
    const gdn2_tensor *req[] = {a.q, a.k, a.v, a.g, a.beta, a.dout, a.dq, a.dk, a.dv, a.dg, a.dbeta};
    const char *req_names[] = {"q", "k", "v", "g", "beta", "d_out", "dq", "dk", "dv", "dg", "dbeta"};
    for (int i = 0; i < 11; ++i)
        if (!req[i]) return fail(GDN2_ERR_NULL_ARG, "%s is NULL (required by the backward)", req_names[i]);
    int rc;
    if ((rc = check_tensor(a.q, "q", GDN2_DTYPE_BF16, GDN2_DTYPE_F16, 3, nullptr))) return rc;
    const int32_t io = a.q->dtype;
    const int64_t T = a.q->shape[0], H = a.q->shape[1], K = a.q->shape[2];
    const int64_t qs[3] = {T, H, K}, v_any[3] = {T, -1, -1};
    if ((rc = check_io(a.k, "k", io, qs, DENSE))) return rc;
    if ((rc = check_io(a.v, "v", io, v_any, DENSE))) return rc;
    int64_t N;
    if ((rc = check_sizes(a.q, a.v, a.cu, &N))) return rc;
    const int64_t HV = a.v->shape[1], V = a.v->shape[2];
    if (K != V)
        return fail(GDN2_ERR_UNSUPPORTED, "(K, V) = (%lld, %lld) not supported by the backward; it takes (64, 64) or (128, 128)",
                    (long long)K, (long long)V);
    if (!fits_rows(HV, V)) return fail(GDN2_ERR_SHAPE, "HV = %lld: 64 rows of the value heads must span under 2 GiB", (long long)HV);
    const int64_t gs[2] = {T, HV}, vs[3] = {T, HV, V}, ss[4] = {N, HV, K, V};
    if ((rc = check_g(a.g, "g", gs, DENSE))) return rc;
    if ((rc = check_tensor(a.beta, "beta", io, -1, 2, gs))) return rc;
    if ((rc = check_io(a.dout, "d_out", io, vs, DENSE))) return rc;
    if ((rc = check_io(a.dq, "dq", io, qs, DENSE))) return rc;
    if ((rc = check_io(a.dk, "dk", io, qs, DENSE))) return rc;
    if ((rc = check_io(a.dv, "dv", io, vs, DENSE))) return rc;
    if ((rc = check_tensor(a.dg, "dg", a.g->dtype, -1, 2, gs))) return rc;
    if ((rc = check_tensor(a.dbeta, "dbeta", io, -1, 2, gs))) return rc;
    if (a.h0 && (rc = check_tensor(a.h0, "initial_state", GDN2_DTYPE_F32, -1, 4, ss))) return rc;
    if (a.dht && (rc = check_tensor(a.dht, "d_final_state", GDN2_DTYPE_F32, -1, 4, ss))) return rc;
    if (a.dh0 && (rc = check_tensor(a.dh0, "d_initial_state", GDN2_DTYPE_F32, -1, 4, ss))) return rc;

    const gdn2_tensor *ts[] = {a.q, a.k, a.v, a.g, a.beta, a.h0, a.cu, a.dout, a.dht, a.dq, a.dk, a.dv, a.dg, a.dbeta, a.dh0};
    const char *names[] = {"q", "k", "v", "g", "beta", "initial_state", "cu_seqlens", "d_out", "d_final_state",
                           "dq", "dk", "dv", "dg", "dbeta", "d_initial_state"};
    for (int o = 9; o < 15; ++o)
        for (int i = 0; i < 15; ++i)
            if (i != o && (i < 9 || i > o) && overlaps(ts[o], ts[i]))
                return fail(GDN2_ERR_ALIAS, "%s overlaps %s", names[o], names[i]);
    if (!p) return GDN2_OK;
    const BwdSpace w(T, N, H, HV, K, V);
    if ((rc = check_workspace(ws, ws_bytes, w.total, ts, names, 15))) return rc;

    *p = DeltaParams{};
    p->q = static_cast<const uint16_t *>(a.q->data);
    p->k = static_cast<const uint16_t *>(a.k->data);
    p->v = static_cast<const uint16_t *>(a.v->data);
    p->g = a.g->data;
    p->beta = static_cast<const uint16_t *>(a.beta->data);
    p->h0 = a.h0 ? static_cast<const float *>(a.h0->data) : nullptr;
    p->cu = a.cu ? a.cu->data : nullptr;
    p->cu64 = a.cu && a.cu->dtype == GDN2_DTYPE_I64;
    p->T = T;
    p->N = (int32_t)N;
    p->H = (int32_t)H;
    p->HV = (int32_t)HV;
    p->K = (int32_t)K;
    p->V = (int32_t)V;
    p->scale = a.scale == 0.0f ? (float)(1.0 / sqrt((double)K)) : a.scale;
    p->io = io == GDN2_DTYPE_F16 ? gdn2::IO_F16 : gdn2::IO_BF16;
    p->gtype = g_type(a.g);
    p->sq = p->sk = H * K;
    p->hsq = p->hsk = K;
    p->sv = p->so = HV * V;
    p->hsv = p->hso = V;
    p->sg = p->sb = HV;
    p->hsg = p->hsb = 1;
    p->nslots = (int32_t)gdn2::slot_count(T, N);
    p->dout = static_cast<const uint16_t *>(a.dout->data);
    p->dht = a.dht ? static_cast<const float *>(a.dht->data) : nullptr;
    p->dh0 = a.dh0 ? static_cast<float *>(a.dh0->data) : nullptr;
    p->dq = static_cast<uint16_t *>(a.dq->data);
    p->dk = static_cast<uint16_t *>(a.dk->data);
    p->dv = static_cast<uint16_t *>(a.dv->data);
    p->dg = a.dg->data;
    p->dbeta = static_cast<uint16_t *>(a.dbeta->data);
    char *b = static_cast<char *>(ws);
    p->rec = b + w.rec;
    p->low_p = 1;
    p->nseg = w.nseg;
    p->seg = reinterpret_cast<float *>(b + w.seg);
    p->rseg = reinterpret_cast<float *>(b + w.rseg);
    p->s_ck = reinterpret_cast<float *>(b + w.s);
    p->ds_ck = reinterpret_cast<float *>(b + w.ds);
    p->u_ck = reinterpret_cast<float *>(b + w.u);
    p->y_ck = reinterpret_cast<float *>(b + w.y);
    p->mx = reinterpret_cast<float *>(b + w.mx);
    p->dq_ws = reinterpret_cast<float *>(b + w.dq);
    p->dk_ws = reinterpret_cast<float *>(b + w.dk);
    return GDN2_OK;
}

struct Qk {
    const gdn2_tensor *x[2], *dy[2], *w[2], *rope, *pos, *y[2], *dw[2];
    const gdn2_qk_options *opts;
};

const char *kQkIn[2] = {"q", "k"};
const char *kQkDy[2] = {"dq_out", "dk_out"};
const char *kQkW[2] = {"q_weight", "k_weight"};
const char *kQkDw[2] = {"dq_weight", "dk_weight"};

// Heads of q and k together.
bool fits_heads(int64_t heads) { return heads <= INT32_MAX / 2; }

// (backward: a.dy and a.dw are used, and y are the gradients dq, dk)
int validate(const Qk &a, bool backward, void *ws, int64_t ws_bytes, QkParams *p)
{
    clear_error();
    const char *y_names[2] = {backward ? "dq" : "q_out", backward ? "dk" : "k_out"};
    int32_t norm = GDN2_QK_NORM_L2, inter = 0;
    float eps = 0.0f;
    if (a.opts) {
        if (a.opts->struct_size < (int32_t)sizeof(gdn2_qk_options))
            return fail(GDN2_ERR_SHAPE, "options: struct_size %d is smaller than %d", a.opts->struct_size, (int)sizeof(gdn2_qk_options));
        norm = a.opts->norm;
        inter = a.opts->interleaved;
        eps = a.opts->eps;
    }
    if (norm != GDN2_QK_NORM_NONE && norm != GDN2_QK_NORM_L2 && norm != GDN2_QK_NORM_RMS)
        return fail(GDN2_ERR_SHAPE, "options: norm must be 0, 1 or 2 (got %d)", norm);
    if (inter != 0 && inter != 1) return fail(GDN2_ERR_SHAPE, "options: interleaved must be 0 or 1 (got %d)", inter);
    if (!(eps >= 0.0f) || isinf(eps)) return fail(GDN2_ERR_SHAPE, "options: eps must be finite and not negative");
    if (eps == 0.0f) eps = norm == GDN2_QK_NORM_RMS ? 1e-6f : 1e-12f;
    for (int i = 0; i < 2; ++i) {
        if (!a.x[i]) return fail(GDN2_ERR_NULL_ARG, "%s is NULL", kQkIn[i]);
        if (!a.y[i]) return fail(GDN2_ERR_NULL_ARG, "%s is NULL", y_names[i]);
        if (backward && !a.dy[i]) return fail(GDN2_ERR_NULL_ARG, "%s is NULL", kQkDy[i]);
    }
    int rc;
    if ((rc = check_tensor(a.x[0], "q", GDN2_DTYPE_BF16, GDN2_DTYPE_F16, 3, nullptr, ROWS))) return rc;
    const int32_t io = a.x[0]->dtype;
    const int64_t T = a.x[0]->shape[0], K = a.x[0]->shape[2];
    const int64_t k_any[3] = {T, -1, K};
    if ((rc = check_io(a.x[1], "k", io, k_any, ROWS))) return rc;
    if (K != 64 && K != 128) return fail(GDN2_ERR_UNSUPPORTED, "K = %lld not supported; K must be 64 or 128", (long long)K);
    if (a.x[0]->shape[1] < 1 || a.x[1]->shape[1] < 1) return fail(GDN2_ERR_HEADS, "q and k need at least one head each");
    const int64_t heads = a.x[0]->shape[1] + a.x[1]->shape[1];
    if (T > INT32_MAX || !fits_heads(heads)) return fail(GDN2_ERR_SHAPE, "T or the head count exceeds the int32 range");
    for (int i = 0; i < 2; ++i) {
        const int64_t want[3] = {T, a.x[i]->shape[1], K};
        if ((rc = check_io(a.y[i], y_names[i], io, want, ROWS))) return rc;
        if (!rows_disjoint(a.y[i])) return fail(GDN2_ERR_LAYOUT, "%s: rows overlap each other", y_names[i]);
        if (backward && (rc = check_io(a.dy[i], kQkDy[i], io, want, ROWS))) return rc;
        if (a.w[i] && (rc = check_tensor(a.w[i], kQkW[i], GDN2_DTYPE_F32, io, 1, &K))) return rc;
        if (backward && a.dw[i]) {
            if (!a.w[i]) return fail(GDN2_ERR_NULL_ARG, "%s without %s", kQkDw[i], kQkW[i]);
            if ((rc = check_tensor(a.dw[i], kQkDw[i], a.w[i]->dtype, -1, 1, &K))) return rc;
        }
    }
    int64_t P = 0, rot = 0;
    if (a.rope) {
        if ((rc = check_tensor(a.rope, "rope", GDN2_DTYPE_F32, -1, 2, nullptr))) return rc;
        P = a.rope->shape[0];
        rot = a.rope->shape[1];
        if (rot < 2 || rot > K || rot % (inter ? 2 : 16) != 0)
            return fail(GDN2_ERR_UNSUPPORTED, "rope: %lld rotated elements; a positive multiple of %d up to K = %lld is supported",
                        (long long)rot, inter ? 2 : 16, (long long)K);
        if (P < 1) return fail(GDN2_ERR_SHAPE, "rope: the table has no rows");
        if (!a.pos) return fail(GDN2_ERR_NULL_ARG, "positions is NULL, rope is given");
        if ((rc = check_tensor(a.pos, "positions", GDN2_DTYPE_I32, GDN2_DTYPE_I64, 1, &T))) return rc;
    } else if (a.pos) {
        return fail(GDN2_ERR_NULL_ARG, "rope is NULL, positions are given");
    }
    const gdn2_tensor *ts[] = {a.x[0], a.x[1], a.w[0], a.w[1], a.rope, a.pos, backward ? a.dy[0] : nullptr,
                               backward ? a.dy[1] : nullptr, a.y[0], a.y[1], backward ? a.dw[0] : nullptr, backward ? a.dw[1] : nullptr};
    const char *names[] = {"q", "k", "q_weight", "k_weight", "rope", "positions", "dq_out", "dk_out",
                           y_names[0], y_names[1], "dq_weight", "dk_weight"};
    for (int o = 8; o < 12; ++o)
        for (int i = 0; i < 12; ++i)
            if (i != o && (i < 8 || i > o) && overlaps(ts[o], ts[i]))
                return fail(GDN2_ERR_ALIAS, "%s overlaps %s", names[o], names[i]);
    if (!p) return GDN2_OK;
    const bool dw = backward && (a.dw[0] || a.dw[1]);
    if (dw && (rc = check_workspace(ws, ws_bytes,
                                    gdn2_qk_norm_rope_bwd_workspace(T, (int32_t)a.x[0]->shape[1], (int32_t)a.x[1]->shape[1], (int32_t)K),
                                    ts, names, 12)))
        return rc;

    *p = QkParams{};
    for (int i = 0; i < 2; ++i) {
        p->x[i] = static_cast<const uint16_t *>(a.x[i]->data);
        p->y[i] = static_cast<uint16_t *>(a.y[i]->data);
        p->sx[i] = tok_stride(a.x[i]);
        p->hsx[i] = head_stride(a.x[i]);
        p->sy[i] = tok_stride(a.y[i]);
        p->hsy[i] = head_stride(a.y[i]);
        p->heads[i] = (int32_t)a.x[i]->shape[1];
        p->w[i] = a.w[i] ? a.w[i]->data : nullptr;
        p->w_f32[i] = a.w[i] && a.w[i]->dtype == GDN2_DTYPE_F32;
        if (backward) {
            p->dy[i] = static_cast<const uint16_t *>(a.dy[i]->data);
            p->sdy[i] = tok_stride(a.dy[i]);
            p->hsdy[i] = head_stride(a.dy[i]);
            p->dw[i] = a.dw[i] ? a.dw[i]->data : nullptr;
        }
    }
    p->rope = a.rope ? static_cast<const float *>(a.rope->data) : nullptr;
    p->pos = a.pos ? a.pos->data : nullptr;
    p->pos64 = a.pos && a.pos->dtype == GDN2_DTYPE_I64;
    p->P = P;
    p->rot = (int32_t)rot;
    p->T = T;
    p->K = (int32_t)K;
    p->norm = norm;
    p->interleaved = inter;
    p->io = io == GDN2_DTYPE_F16 ? gdn2::IO_F16 : gdn2::IO_BF16;
    p->eps = eps;
    p->part = static_cast<float *>(ws);
    p->groups = backward ? gdn2::qk_bwd_groups(T, p->heads[0], p->heads[1], p->K) : 0;
    return GDN2_OK;
}

int launched(hipError_t e)
{
    return e == hipSuccess ? GDN2_OK : fail(GDN2_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
}

int current_cus()
{
    int dev = 0;
    return hipGetDevice(&dev) == hipSuccess ? cu_count(dev) : 0;
}

}  // namespace

extern "C" {

int64_t gdn2_delta_chunk_fwd_workspace(int64_t T, int32_t N, int32_t HV)
{
    if (T <= 0 || T > INT32_MAX || N <= 0 || HV <= 0 || !fits_grid(T, N, HV)) return 0;
    return fwd_records(T, N, HV) + fwd_segments(T, N, HV);
}

int64_t gdn2_delta_chunk_bwd_workspace(int64_t T, int32_t N, int32_t H, int32_t HV, int32_t K, int32_t V)
{
    if (T <= 0 || T > INT32_MAX || N <= 0 || H <= 0 || HV <= 0 || HV % H != 0 || (K != 64 && K != 128) || V != K) return 0;
    if (!fits_grid(T, N, HV) || !fits_rows(HV, V)) return 0;
    return BwdSpace(T, N, H, HV, K, V).total;
}

int gdn2_delta_chunk_fwd(const gdn2_tensor *q, const gdn2_tensor *k, const gdn2_tensor *v, const gdn2_tensor *g,
                         const gdn2_tensor *beta, float scale, const gdn2_tensor *initial_state,
                         const gdn2_tensor *cu_seqlens, const gdn2_tensor *out, const gdn2_tensor *final_state,
                         const gdn2_fwd_options *opts, void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    DeltaParams p;
    if (int rc = validate(DeltaFwd{q, k, v, g, beta, scale, initial_state, cu_seqlens, out, final_state, opts}, true, workspace,
                          workspace_bytes, &p))
        return rc;
    const int ncu = current_cus();
    hipError_t e = gdn2::launch_delta_wy(p, stream);
    if (e == hipSuccess) e = gdn2::launch_delta_state(p, false, ncu, stream);
    return launched(e);
}

int gdn2_delta_chunk_fwd_check(const gdn2_tensor *q, const gdn2_tensor *k, const gdn2_tensor *v, const gdn2_tensor *g,
                               const gdn2_tensor *beta, float scale, const gdn2_tensor *initial_state,
                               const gdn2_tensor *cu_seqlens, const gdn2_tensor *out, const gdn2_tensor *final_state,
                               const gdn2_fwd_options *opts)
{
    return validate(DeltaFwd{q, k, v, g, beta, scale, initial_state, cu_seqlens, out, final_state, opts}, true, nullptr, 0, nullptr);
}

int gdn2_delta_recurrent_fwd(const gdn2_tensor *q, const gdn2_tensor *k, const gdn2_tensor *v, const gdn2_tensor *g,
                             const gdn2_tensor *beta, float scale, const gdn2_tensor *initial_state,
                             const gdn2_tensor *cu_seqlens, const gdn2_tensor *out, const gdn2_tensor *final_state,
                             const gdn2_fwd_options *opts, hipStream_t stream)
{
    DeltaParams p;
    if (int rc = validate(DeltaFwd{q, k, v, g, beta, scale, initial_state, cu_seqlens, out, final_state, opts}, false, nullptr, 0, &p))
        return rc;
    return launched(gdn2::launch_delta_step(p, stream));
}

int gdn2_delta_recurrent_fwd_check(const gdn2_tensor *q, const gdn2_tensor *k, const gdn2_tensor *v, const gdn2_tensor *g,
                                   const gdn2_tensor *beta, float scale, const gdn2_tensor *initial_state,
                                   const gdn2_tensor *cu_seqlens, const gdn2_tensor *out, const gdn2_tensor *final_state,
                                   const gdn2_fwd_options *opts)
{
    return validate(DeltaFwd{q, k, v, g, beta, scale, initial_state, cu_seqlens, out, final_state, opts}, false, nullptr, 0, nullptr);
}

int gdn2_delta_chunk_bwd(const gdn2_tensor *q, const gdn2_tensor *k, const gdn2_tensor *v, const gdn2_tensor *g,
                         const gdn2_tensor *beta, float scale, const gdn2_tensor *initial_state,
                         const gdn2_tensor *cu_seqlens, const gdn2_tensor *d_out, const gdn2_tensor *d_final_state,
                         const gdn2_tensor *dq, const gdn2_tensor *dk, const gdn2_tensor *dv, const gdn2_tensor *dg,
                         const gdn2_tensor *dbeta, const gdn2_tensor *d_initial_state, void *workspace,
                         int64_t workspace_bytes, hipStream_t stream)
{
    DeltaParams p;
    if (int rc = validate(DeltaBwd{q, k, v, g, beta, scale, initial_state, cu_seqlens, d_out, d_final_state, dq, dk, dv, dg, dbeta,
                                   d_initial_state},
                          workspace, workspace_bytes, &p))
        return rc;
    const int ncu = current_cus();
    hipError_t e = gdn2::launch_delta_wy(p, stream);
    if (e == hipSuccess && p.T > 0) e = gdn2::launch_delta_state(p, true, ncu, stream);
    if (e == hipSuccess) e = gdn2::launch_delta_bwd_state(p, ncu, stream);
    if (e == hipSuccess) e = gdn2::launch_delta_bwd_grad(p, stream);
    return launched(e);
}

int gdn2_delta_chunk_bwd_check(const gdn2_tensor *q, const gdn2_tensor *k, const gdn2_tensor *v, const gdn2_tensor *g,
                               const gdn2_tensor *beta, float scale, const gdn2_tensor *initial_state,
                               const gdn2_tensor *cu_seqlens, const gdn2_tensor *d_out, const gdn2_tensor *d_final_state,
                               const gdn2_tensor *dq, const gdn2_tensor *dk, const gdn2_tensor *dv, const gdn2_tensor *dg,
                               const gdn2_tensor *dbeta, const gdn2_tensor *d_initial_state)
{
    return validate(DeltaBwd{q, k, v, g, beta, scale, initial_state, cu_seqlens, d_out, d_final_state, dq, dk, dv, dg, dbeta,
                             d_initial_state},
                    nullptr, 0, nullptr);
}

int gdn2_qk_norm_rope_fwd(const gdn2_tensor *q, const gdn2_tensor *k, const gdn2_tensor *q_weight, const gdn2_tensor *k_weight,
                          const gdn2_tensor *rope, const gdn2_tensor *positions, const gdn2_tensor *q_out,
                          const gdn2_tensor *k_out, const gdn2_qk_options *opts, hipStream_t stream)
{
    QkParams p;
    if (int rc = validate(Qk{{q, k}, {}, {q_weight, k_weight}, rope, positions, {q_out, k_out}, {}, opts}, false, nullptr, 0, &p))
        return rc;
    return launched(gdn2::launch_qk_fwd(p, stream));
}

int gdn2_qk_norm_rope_fwd_check(const gdn2_tensor *q, const gdn2_tensor *k, const gdn2_tensor *q_weight,
                                const gdn2_tensor *k_weight, const gdn2_tensor *rope, const gdn2_tensor *positions,
                                const gdn2_tensor *q_out, const gdn2_tensor *k_out, const gdn2_qk_options *opts)
{
    return validate(Qk{{q, k}, {}, {q_weight, k_weight}, rope, positions, {q_out, k_out}, {}, opts}, false, nullptr, 0, nullptr);
}

int64_t gdn2_qk_norm_rope_bwd_workspace(int64_t T, int32_t H, int32_t HK, int32_t K)
{
    if (T <= 0 || T > INT32_MAX || H <= 0 || HK <= 0 || !fits_heads((int64_t)H + HK) || (K != 64 && K != 128)) return 0;
    return up256((int64_t)gdn2::qk_bwd_groups(T, H, HK, K) * 2 * K * 4);
}

int gdn2_qk_norm_rope_bwd(const gdn2_tensor *q, const gdn2_tensor *k, const gdn2_tensor *dq_out, const gdn2_tensor *dk_out,
                          const gdn2_tensor *q_weight, const gdn2_tensor *k_weight, const gdn2_tensor *rope,
                          const gdn2_tensor *positions, const gdn2_tensor *dq, const gdn2_tensor *dk,
                          const gdn2_tensor *dq_weight, const gdn2_tensor *dk_weight, const gdn2_qk_options *opts,
                          void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    QkParams p;
    if (int rc = validate(Qk{{q, k}, {dq_out, dk_out}, {q_weight, k_weight}, rope, positions, {dq, dk}, {dq_weight, dk_weight}, opts},
                          true, workspace, workspace_bytes, &p))
        return rc;
    return launched(gdn2::launch_qk_bwd(p, stream));
}

int gdn2_qk_norm_rope_bwd_check(const gdn2_tensor *q, const gdn2_tensor *k, const gdn2_tensor *dq_out, const gdn2_tensor *dk_out,
                                const gdn2_tensor *q_weight, const gdn2_tensor *k_weight, const gdn2_tensor *rope,
                                const gdn2_tensor *positions, const gdn2_tensor *dq, const gdn2_tensor *dk,
                                const gdn2_tensor *dq_weight, const gdn2_tensor *dk_weight, const gdn2_qk_options *opts)
{
    return validate(Qk{{q, k}, {dq_out, dk_out}, {q_weight, k_weight}, rope, positions, {dq, dk}, {dq_weight, dk_weight}, opts}, true,
                    nullptr, 0, nullptr);
}

}  // extern "C"
