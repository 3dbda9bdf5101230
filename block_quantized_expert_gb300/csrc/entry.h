// entry.h -- what the C entries of calls without a layer share: the thread's error
// message and the status of a launch.
#pragma once

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "layer.h"

namespace moe {

inline moe_status refuse(moe_status st, const char* fmt, ...) {
    char buf[200];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    set_thread_error(buf);
    return st;
}

inline moe_status status_of(cudaError_t e, const char* what) {
    return e == cudaSuccess ? MOE_OK : refuse(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Whether these pointers to 4-byte elements are all aligned to them (NULL is).
template <typename... P>
bool aligned4(const P*... p) {
    return ((reinterpret_cast<uintptr_t>(p) | ... | uintptr_t(0)) & 3) == 0;
}

constexpr long long kMostStride = 1LL << 40;

}  // namespace moe
