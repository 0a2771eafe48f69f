// Host helpers of the language-model operators' entry points: errors, sizes and
// alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/muon.h"
#include "internal.hpp"

namespace muon {

namespace {

int refuse(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int refuse(int status, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return fail_status(status, buf);
}
int done() { return fail_status(MUON_OK, ""); }
int launched(hipError_t e, const char* what) {
    return e == hipSuccess ? MUON_OK : refuse(MUON_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

constexpr int64_t kMaxSeq = int64_t{1} << 29;
constexpr int64_t kMaxRowStride = int64_t{1} << 24;
constexpr int64_t kMaxBlocks = (int64_t{1} << 31) - 1;

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int64_t div_up(int64_t x, int64_t y) { return (x + y - 1) / y; }
// x * y, or -1 where it passes 2^62 (both >= 0)
int64_t times(int64_t x, int64_t y) {
    int64_t r;
    return x < 0 || y < 0 || __builtin_mul_overflow(x, y, &r) || r > (int64_t{1} << 62) ? -1 : r;
}
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_workspace(const void* ws, size_t have, size_t need) {
    if (!ws || have < need)
        return refuse(MUON_ERR_WORKSPACE, "workspace of %zu bytes is needed (got %zu)", need, ws ? have : 0);
    if (!aligned(ws, 256)) return refuse(MUON_ERR_WORKSPACE, "the workspace is not aligned to 256 bytes");
    return MUON_OK;
}

}  // namespace

}  // namespace muon
