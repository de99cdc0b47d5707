// What the entry points' argument checks share.
#pragma once
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "internal.h"

namespace sdv2 {

__attribute__((format(printf, 2, 3))) inline sdv2_status refuse(sdv2_status s, const char* fmt, ...)
{
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return s;
}

inline sdv2_status launched(cudaError_t e, const char* what)
{
    if (e != cudaSuccess) return refuse(SDV2_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    set_last_error("");
    return SDV2_OK;
}

inline bool on_16_bytes(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool given(const void* p) { return p && on_16_bytes(p); }

}  // namespace sdv2
