// Argument checks that the C ABI layers of the operators share.
#pragma once
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/gdn.h"

namespace gdn {
void set_last_error(const char* msg);
}

namespace {

gdn_status fail(gdn_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    gdn::set_last_error(buf);
    return st;
}
// No C++ exception crosses the C ABI: the launches' tables of kernel attributes allocate.
[[maybe_unused]] gdn_status no_host_memory() { return fail(GDN_ERR_CUDA, "out of host memory"); }
gdn_status done(cudaError_t e) {
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "CUDA error: %s", cudaGetErrorString(e));
    gdn::set_last_error("");
    return GDN_OK;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t elem(int dt) { return dt == GDN_FP32 ? 4 : dt == GDN_BF16 ? 2 : 1; }

// A required (or, with optional set, possibly NULL) pointer of the given alignment.
gdn_status check_ptr(const char* name, const void* p, size_t align, bool optional = false) {
    if (!p) return optional ? GDN_OK : fail(GDN_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, align)) return fail(GDN_ERR_INVALID_ARG, "%s must be %zu-byte aligned", name, align);
    return GDN_OK;
}
// A row stride: 0 stands for `dense`; never below it, and a multiple of `unit` elements.
gdn_status check_stride(const char* name, int64_t& stride, int64_t dense, int64_t unit) {
    if (stride == 0) stride = dense;
    if (stride < dense) return fail(GDN_ERR_INVALID_ARG, "%s (%lld) is below the row's %lld values", name, (long long)stride, (long long)dense);
    if (stride % unit) return fail(GDN_ERR_INVALID_ARG, "%s (%lld) must be a multiple of %lld elements (16 bytes)", name, (long long)stride, (long long)unit);
    return GDN_OK;
}
gdn_status check_scale(float scale) {
    if (!isfinite(scale) || !(scale > 0.f)) return fail(GDN_ERR_INVALID_ARG, "scale must be finite and > 0 (got %g)", double(scale));
    return GDN_OK;
}

#define TRY(x)                            \
    do {                                  \
        const gdn_status try_st = (x);    \
        if (try_st != GDN_OK) return try_st; \
    } while (0)

}  // namespace
