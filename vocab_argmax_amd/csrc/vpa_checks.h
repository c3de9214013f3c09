// vpa_checks.h -- argument checks shared by the sources that implement the C
// ABI of the head's and the draft head's operators (head_api.hip,
// draft_api.hip).
#pragma once

#include "vpa_head.h"
#include "vpa_host.h"

namespace vpa {

constexpr int64_t kMaxSize = INT32_MAX;

inline size_t round256(size_t n) {
    return (n + 255) / 256 * 256;
}

// A matrix argument: a pointer aligned to its element, rows that do not
// overlap.
inline vpa_status check_matrix(const char* name, const void* p, int esize, int64_t ld, int64_t cols) {
    if (!p)
        return fail(VPA_ERR_INVALID, "%s is NULL", name);
    if (!aligned(p, (size_t)esize))
        return fail(VPA_ERR_INVALID, "%s not aligned to its element size", name);
    if (ld < cols || ld > ((int64_t)1 << 40))
        return fail(VPA_ERR_INVALID, "%s: row stride %lld outside [%lld, 2^40]", name,
                    (long long)ld, (long long)cols);
    return ok();
}

inline vpa_status check_vector(const char* name, const void* p, int esize) {
    if (!p)
        return fail(VPA_ERR_INVALID, "%s is NULL", name);
    if (!aligned(p, (size_t)esize))
        return fail(VPA_ERR_INVALID, "%s not aligned to its element size", name);
    return ok();
}

inline vpa_status check_workspace(const char* call, const void* ws, size_t have, size_t need) {
    if (need == 0)
        return ok();
    if (have < need)
        return fail(VPA_ERR_INVALID, "%s: workspace of %zu bytes, needs %zu", call, have, need);
    if (!ws || !aligned(ws, 16))
        return fail(VPA_ERR_INVALID, "%s: workspace is NULL or not 16-byte aligned", call);
    return ok();
}

inline vpa_status check_rows(const char* call, int64_t rows) {
    if (rows < 0 || rows > kMaxSize)
        return fail(VPA_ERR_INVALID, "%s: %lld rows outside [0, 2^31)", call, (long long)rows);
    return ok();
}

inline vpa_status check_sizes(const char* call, int64_t rows, int64_t outer, int64_t inner) {
    vpa_status st = check_rows(call, rows);
    if (st != VPA_OK)
        return st;
    if (outer < 1 || outer > kMaxSize || inner < 1 || inner > kMaxSize)
        return fail(VPA_ERR_INVALID, "%s: outer %lld or inner %lld outside [1, 2^31)", call,
                    (long long)outer, (long long)inner);
    return ok();
}

inline vpa_status check_act(int32_t act) {
    if (act < VPA_ACT_NONE || act > VPA_ACT_SILU)
        return fail(VPA_ERR_UNSUPPORTED, "activation %d is unknown", (int)act);
    return ok();
}

}  // namespace vpa
