// vpa_host.h -- host-side helpers shared by the sources that implement the C
// ABI (api.hip, head_api.hip): error reporting and the argument checks both
// need.  Defined in api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "vpa.h"

namespace vpa {

// Sets the calling thread's vpa_last_error() message and returns `st`.
vpa_status fail(vpa_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
vpa_status hip_fail(hipError_t e, const char* what);

inline vpa_status ok() {
    return VPA_OK;
}

// The dtype argument's integer value.  A C caller may pass any int as a
// vpa_dtype, but in C++ loading an enum outside the range of its
// enumerators is undefined (even to pass it on), so every entry point reads
// its dtype argument's bytes as an int first and works with that int.
int dtype_value(const vpa_dtype* dt);

inline int esize_of(int dt) {
    return dt == VPA_BF16 ? 2 : (dt == VPA_F32 ? 4 : 0);
}

inline bool aligned(const void* p, size_t a) {
    return ((uintptr_t)p % a) == 0;
}

vpa_status check_vocab(const vpa_vocab& v);
vpa_status check_dtype(int dt);
vpa_status check_dispatch(int64_t threads, const char* what);

}  // namespace vpa
