// Argument checks shared by the C-ABI entry points: the calling thread's
// error message, tensor descriptors, options. Host only, not part of the ABI.
#pragma once

#include <stdint.h>

#include "../../include/gdn2.h"

namespace gdn2 {
namespace api {

// Set the thread's error message and return `code`.
int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
void clear_error();
const char *last_error();

const char *dtype_name(int32_t d);
int64_t elem_size(int32_t d);
int64_t numel(const gdn2_tensor *t);

// How a tensor may be laid out in memory.
enum Layout {
    DENSE,  // row-major contiguous
    ROWS,   // [tokens, heads, D]: the D elements of a row contiguous, token
            // and head strides free (non-negative, multiples of 16 bytes,
            // the token stride at least one row), rows 16-byte aligned
    GATES   // [tokens, heads], read an element at a time: any non-negative
            // strides, aligned to the element
};

// Rank, dtype (one of two accepted: dtype2 < 0 for one), extents (-1 = any),
// non-negative extents, layout, non-NULL data when non-empty, 16-byte
// alignment (GATES: the element's).
int check_tensor(const gdn2_tensor *t, const char *name, int32_t dtype, int32_t dtype2, int ndim,
                 const int64_t *want, Layout layout = DENSE);
// Whether the [tokens, heads, D] rows of a ROWS tensor are pairwise disjoint.
bool rows_disjoint(const gdn2_tensor *t);
bool overlaps(const gdn2_tensor *a, const gdn2_tensor *b);

// Options: fields past struct_size keep their defaults, so that callers
// built against an older, shorter struct keep working.
struct Options {
    int32_t split = 0, vmajor = 0, l2norm = 0;
};

int read_options(const gdn2_fwd_options *opts, Options *o);

// Compute-unit count of a device, looked up once (0: unknown).
int cu_count(int dev);

}  // namespace api
}  // namespace gdn2
