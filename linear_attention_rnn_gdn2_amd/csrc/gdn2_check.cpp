// Argument checks shared by the C-ABI entry points (see gdn2_check.h).
#include "gdn2_check.h"

#include <stdarg.h>
#include <stddef.h>
#include <stdio.h>

#include <atomic>
#include <string>
#include <utility>

#include <hip/hip_runtime.h>

namespace gdn2 {
namespace api {

static thread_local std::string g_last_error;

void clear_error() { g_last_error.clear(); }
const char *last_error() { return g_last_error.c_str(); }

int fail(int code, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return code;
}

const char *dtype_name(int32_t d)
{
    switch (d) {
    case GDN2_DTYPE_BF16: return "bf16";
    case GDN2_DTYPE_F32: return "float32";
    case GDN2_DTYPE_I32: return "int32";
    case GDN2_DTYPE_F16: return "float16";
    case GDN2_DTYPE_I64: return "int64";
    default: return "unknown";
    }
}

int64_t elem_size(int32_t d)
{
    switch (d) {
    case GDN2_DTYPE_BF16:
    case GDN2_DTYPE_F16: return 2;
    case GDN2_DTYPE_I64: return 8;
    default: return 4;
    }
}

int64_t numel(const gdn2_tensor *t)
{
    int64_t n = 1;
    for (int d = 0; d < t->ndim; ++d) n *= t->shape[d];
    return n;
}

// Rank, dtype (one of two accepted: dtype2 < 0 for one), extents (-1 = any),
// non-negative extents, layout, non-NULL data when non-empty, 16-byte
// alignment.
int check_tensor(const gdn2_tensor *t, const char *name, int32_t dtype, int32_t dtype2, int ndim,
                 const int64_t *want, Layout layout)
{
    if (t->ndim != ndim)
        return fail(GDN2_ERR_SHAPE, "%s: expected %d dimensions, got %d", name, ndim, t->ndim);
    if (t->dtype != dtype && t->dtype != dtype2) {
        if (dtype2 >= 0)
            return fail(GDN2_ERR_DTYPE, "%s: expected %s or %s, got %s", name, dtype_name(dtype), dtype_name(dtype2),
                        dtype_name(t->dtype));
        return fail(GDN2_ERR_DTYPE, "%s: expected %s, got %s", name, dtype_name(dtype), dtype_name(t->dtype));
    }
    for (int d = 0; d < ndim; ++d) {
        if (t->shape[d] < 0)
            return fail(GDN2_ERR_SHAPE, "%s: negative extent in dimension %d", name, d);
        if (want && want[d] >= 0 && t->shape[d] != want[d])
            return fail(GDN2_ERR_SHAPE, "%s: dimension %d is %lld, expected %lld", name, d,
                        (long long)t->shape[d], (long long)want[d]);
    }
    const int64_t es = elem_size(t->dtype);
    if (layout == ROWS) {
        const int64_t D = t->shape[2];
        if (D > 1 && t->stride[2] != 1)
            return fail(GDN2_ERR_LAYOUT, "%s: the last dimension must be contiguous (stride %lld)", name,
                        (long long)t->stride[2]);
        for (int d = 0; d < 2; ++d) {
            if (t->shape[d] <= 1) continue;
            if (t->stride[d] < 0 || (t->stride[d] * es) % 16 != 0)
                return fail(GDN2_ERR_LAYOUT, "%s: dimension %d stride %lld must be non-negative and a multiple of 16 bytes",
                            name, d, (long long)t->stride[d]);
        }
        if (t->shape[0] > 1) {
            if (t->stride[0] < D)
                return fail(GDN2_ERR_LAYOUT, "%s: token stride %lld is shorter than a row (%lld elements)", name,
                            (long long)t->stride[0], (long long)D);
            if (t->stride[0] * es * 64 > INT32_MAX)
                return fail(GDN2_ERR_LAYOUT, "%s: token stride %lld is too large (64 rows must span under 2 GiB)",
                            name, (long long)t->stride[0]);
        }
    } else if (layout == GATES || layout == VECTORS) {
        if (layout == VECTORS && t->shape[ndim - 1] > 1 && t->stride[ndim - 1] != 1)
            return fail(GDN2_ERR_LAYOUT, "%s: the last dimension must be contiguous (stride %lld)", name,
                        (long long)t->stride[ndim - 1]);
        for (int d = 0; d < ndim; ++d)
            if (t->shape[d] > 1 && t->stride[d] < 0)
                return fail(GDN2_ERR_LAYOUT, "%s: dimension %d stride %lld must be non-negative", name, d,
                            (long long)t->stride[d]);
    } else {
        int64_t expect = 1;
        for (int d = ndim - 1; d >= 0; --d) {
            if (t->shape[d] > 1 && t->stride[d] != expect)
                return fail(GDN2_ERR_LAYOUT, "%s: not row-major contiguous (dimension %d stride %lld, expected %lld)",
                            name, d, (long long)t->stride[d], (long long)expect);
            expect *= t->shape[d];
        }
    }
    if (numel(t) > 0) {
        if (!t->data)
            return fail(GDN2_ERR_NULL_ARG, "%s: data is NULL but the tensor has elements", name);
        const int64_t align = layout == GATES || layout == VECTORS ? es : 16;
        if (reinterpret_cast<uintptr_t>(t->data) % align != 0)
            return fail(GDN2_ERR_LAYOUT, "%s: data pointer is not %lld-byte aligned", name, (long long)align);
    }
    return GDN2_OK;
}

// Whether the [tokens, heads, D] rows of a ROWS tensor are pairwise disjoint:
// with the token and head dimensions taken in order of increasing stride,
// each stride must reach past everything the smaller ones span.
bool rows_disjoint(const gdn2_tensor *t)
{
    int64_t st[2] = {t->stride[0], t->stride[1]}, ex[2] = {t->shape[0], t->shape[1]};
    if (st[0] > st[1]) {
        std::swap(st[0], st[1]);
        std::swap(ex[0], ex[1]);
    }
    int64_t span = t->shape[2];  // elements one row covers
    for (int d = 0; d < 2; ++d) {
        if (ex[d] <= 1) continue;
        if (st[d] < span) return false;
        span += (ex[d] - 1) * st[d];
    }
    return true;
}

// Bytes from the first to one past the last element (strided tensors: the
// whole span, which is conservative for interleaved views).
int64_t span_bytes(const gdn2_tensor *t)
{
    if (numel(t) == 0) return 0;
    int64_t last = 0;
    for (int d = 0; d < t->ndim; ++d) last += (t->shape[d] - 1) * t->stride[d];
    return (last + 1) * elem_size(t->dtype);
}

bool overlaps(const gdn2_tensor *a, const gdn2_tensor *b)
{
    if (!a || !b || !a->data || !b->data) return false;
    const int64_t na = span_bytes(a), nb = span_bytes(b);
    if (na == 0 || nb == 0) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a->data), pb = reinterpret_cast<uintptr_t>(b->data);
    return pa < pb + (uintptr_t)nb && pb < pa + (uintptr_t)na;
}

// A byte range as a tensor, for the overlap checks.
static gdn2_tensor bytes_of(void *data, int64_t bytes)
{
    gdn2_tensor t = {};
    t.data = data;
    t.dtype = GDN2_DTYPE_F16;  // two bytes
    t.ndim = 1;
    t.shape[0] = bytes / 2;
    t.stride[0] = 1;
    return t;
}

int check_workspace(void *ws, int64_t have, int64_t need, const gdn2_tensor *const *ts, const char *const *names, int count)
{
    if (need == 0) return GDN2_OK;
    if (!ws) return fail(GDN2_ERR_WORKSPACE, "workspace is NULL, %lld bytes are needed", (long long)need);
    if (have < need)
        return fail(GDN2_ERR_WORKSPACE, "workspace of %lld bytes is too small, %lld are needed", (long long)have, (long long)need);
    if (reinterpret_cast<uintptr_t>(ws) % 256 != 0) return fail(GDN2_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    const gdn2_tensor w = bytes_of(ws, need);
    for (int i = 0; i < count; ++i)
        if (overlaps(&w, ts[i])) return fail(GDN2_ERR_ALIAS, "workspace overlaps %s", names[i]);
    return GDN2_OK;
}

int read_options(const gdn2_fwd_options *opts, Options *o)
{
    *o = Options{};
    if (!opts) return GDN2_OK;
    const int32_t sz = opts->struct_size;
    if (sz < (int32_t)(2 * sizeof(int32_t)))
        return fail(GDN2_ERR_SHAPE, "options: struct_size %d is smaller than %d", sz, (int)(2 * sizeof(int32_t)));
    if (opts->seq_split_chunks < -1)
        return fail(GDN2_ERR_SHAPE, "options: seq_split_chunks must be -1, 0 or positive (got %d)",
                    opts->seq_split_chunks);
    o->split = opts->seq_split_chunks;
    if (sz >= (int32_t)(offsetof(gdn2_fwd_options, state_layout) + sizeof(int32_t))) {
        if (opts->state_layout != GDN2_STATE_KV && opts->state_layout != GDN2_STATE_VK)
            return fail(GDN2_ERR_SHAPE, "options: state_layout must be GDN2_STATE_KV or GDN2_STATE_VK (got %d)",
                        opts->state_layout);
        o->vmajor = opts->state_layout == GDN2_STATE_VK;
    }
    if (sz >= (int32_t)(offsetof(gdn2_fwd_options, qk_l2norm) + sizeof(int32_t))) {
        if (opts->qk_l2norm != 0 && opts->qk_l2norm != 1)
            return fail(GDN2_ERR_SHAPE, "options: qk_l2norm must be 0 or 1 (got %d)", opts->qk_l2norm);
        o->l2norm = opts->qk_l2norm;
    }
    return GDN2_OK;
}

// Compute-unit count per device, looked up once.
int cu_count(int dev)
{
    static std::atomic<int> cache[64];
    if (dev < 0 || dev >= 64) return 0;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace api
}  // namespace gdn2
