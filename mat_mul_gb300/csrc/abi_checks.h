// abi_checks.h -- what the C entry points outside qmm_abi.cu share: refusals
// and the checks of types and pointers.
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "f8_internal.h"
#include "qmm_internal.h"

namespace {

int refuse(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int refuse(int code, const char *fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return qk::record_error(code, msg);
}
int cuda_error(cudaError_t e, const char *what) { return refuse(QMM_ECUDA, "%s: %s", what, cudaGetErrorString(e)); }

using ll = long long;
[[maybe_unused]] constexpr int64_t I31 = int64_t(1) << 31;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_ftype(int t, const char *what) {
    if (t != QMM_F32 && t != QMM_F16 && t != QMM_BF16) return refuse(QMM_EINVAL_TYPE, "%s: unknown value type %d", what, t);
    return QMM_OK;
}
int check_words(const void *p, const char *what) {
    if (!p) return refuse(QMM_EINVAL_PTR, "%s is null", what);
    if (!aligned(p, 4)) return refuse(QMM_EINVAL_PTR, "%s must be 4-byte aligned", what);
    return QMM_OK;
}

}  // namespace
