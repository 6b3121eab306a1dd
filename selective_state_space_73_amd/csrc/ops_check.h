// What the C ABI files of the operators share: error texts, rounding of sizes, overlaps, workspaces.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstddef>
#include <cstdint>
#include <cstdio>

#include "selscan_internal.h"

namespace {

[[maybe_unused]] ss_status fail(ss_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return selscan::set_error(s, buf);
}

[[maybe_unused]] size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
[[maybe_unused]] size_t io_size(int dt) { return dt == SS_BF16 ? 2 : 4; }
[[maybe_unused]] int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Range { const void* p; size_t bytes; const char* name; };
[[maybe_unused]] bool overlap(const Range& a, const Range& b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Every output apart from every input, from every other output and from the workspace.
[[maybe_unused]] ss_status check_overlaps(const Range* outs, int n_out, const Range* ins, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlap(outs[i], ins[j])) return fail(SS_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, ins[j].name);
        for (int j = i + 1; j < n_out; ++j)
            if (overlap(outs[i], outs[j])) return fail(SS_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
    }
    return SS_OK;
}

[[maybe_unused]] ss_status check_workspace(const void* workspace, size_t given, size_t need) {
    if (need > 0 && (!workspace || given < need))
        return fail(SS_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", given, need);
    if (need > 0 && ((uintptr_t)workspace & 255u)) return fail(SS_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    return SS_OK;
}

[[maybe_unused]] ss_status launched(hipError_t e) {
    return e == hipSuccess ? SS_OK : fail(SS_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
}

}  // namespace
