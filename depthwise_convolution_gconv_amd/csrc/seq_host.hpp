// seq_host.hpp -- what the C entry points of the sequence operators share: errors, strides,
// ranges of memory, workspaces.  Host code only.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "gconv.h"
#include "seq.hpp"

namespace gconv {
namespace host {

inline gconv_status_t fail(gconv_status_t s, const char *fmt, ...)
{
    char text[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
    gconv::set_last_error(text);
    return s;
}

inline gconv_status_t done(hipError_t err, const char *kname)
{
    if (err != hipSuccess) return fail(GCONV_ERR_LAUNCH, "kernel launch failed: HIP error %d", (int)err);
    gconv::set_last_kernel(kname);
    return GCONV_OK;
}

inline bool bad_dtype(gconv_dtype_t d) { return d != GCONV_F32 && d != GCONV_F16 && d != GCONV_BF16; }
inline size_t elem(gconv_dtype_t d) { return d == GCONV_F32 ? 4 : 2; }

// Memory a call reads or writes.
struct Range {
    const char *name;
    const void *p;
    size_t bytes;
    bool out;
};

inline gconv_status_t check_ranges(const Range *r, int n)
{
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            if (i == j || !r[i].out || !r[i].p || !r[j].p || !r[i].bytes || !r[j].bytes) continue;
            const uintptr_t a = (uintptr_t)r[i].p, b = (uintptr_t)r[j].p;
            if (a < b + r[j].bytes && b < a + r[i].bytes)
                return fail(GCONV_ERR_INVALID_ARG, "%s overlaps %s", r[i].name, r[j].name);
        }
    return GCONV_OK;
}

// Bytes from the first to past the last element of a strided [n0][n1][n2][len] view.
inline size_t extent(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t len, size_t es)
{
    if (n0 == 0 || n1 == 0 || n2 == 0 || len == 0) return 0;
    return es * (size_t)((n0 - 1) * s0 + (n1 - 1) * s1 + (n2 - 1) * s2 + len);
}

constexpr int64_t kMax = (int64_t(1) << 31) - 1;
constexpr double kCells = 4.0e18;   // element offsets stay in int64

inline gconv_status_t check_strides(const int64_t *strides, int n)
{
    if (!strides) return fail(GCONV_ERR_INVALID_ARG, "NULL strides");
    for (int i = 0; i < n; ++i)
        if (strides[i] < 0) return fail(GCONV_ERR_INVALID_ARG, "stride %d is negative", i);
    return GCONV_OK;
}

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

inline gconv_status_t check_workspace(const void *ws, size_t have, size_t need)
{
    if (need > 0 && !ws) return fail(GCONV_ERR_INVALID_ARG, "NULL workspace");
    if (((uintptr_t)ws & 15) != 0) return fail(GCONV_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    if (have < need) return fail(GCONV_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", have, need);
    return GCONV_OK;
}

}  // namespace host
}  // namespace gconv
