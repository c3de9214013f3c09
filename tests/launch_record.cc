// launch_record.cc -- a preloaded library that stands in front of the HIP
// runtime's kernel launch on a host without a GPU: launches of the head's
// operators are written down, with the memory their arguments say they use,
// and report success.  Built and read by test_launches_cpu.py.
#include <dlfcn.h>
#include <stdint.h>
#include <string.h>

#include <map>
#include <string>
#include <vector>

#include "vpa_head_internal.h"

namespace {

// One launch.  `part` .. `part + part_bytes` is what it writes or reads of the
// call's workspace for partial results (0 bytes: none).
struct Launch {
    char name[192];
    uint32_t grid[3], block[3];
    int64_t m, n, k, slices;
    uint64_t part;
    int64_t part_bytes;
    int64_t chunks;             // of a segment of a row of log probabilities
};

std::map<const void*, std::string>& names() {
    static std::map<const void*, std::string> m;
    return m;
}
std::vector<Launch>& launches() {
    static std::vector<Launch> v;
    return v;
}

template <typename T>
const T& arg(void** args, int i) {
    return *(const T*)args[i];
}

void gemm(Launch& l, const vpa::GemmTask& t, int64_t slices, const void* part) {
    l.m = t.m;
    l.n = t.n;
    l.k = t.k;
    l.slices = slices;
    l.part = (uint64_t)part;
    l.part_bytes = part ? slices * t.m * t.n * 4 : 0;
}

}  // namespace

extern "C" {

int launches_count() {
    return (int)launches().size();
}
const Launch* launches_get(int i) {
    return &launches()[(size_t)i];
}
void launches_clear() {
    launches().clear();
}

void __hipRegisterFunction(void** modules, const void* host, char* device, const char* name,
                           unsigned limit, void* tid, void* bid, void* bdim, void* gdim,
                           int* wsize) {
    names()[host] = name;
    static const auto real = (decltype(&__hipRegisterFunction))dlsym(RTLD_NEXT,
                                                                    "__hipRegisterFunction");
    if (real)
        real(modules, host, device, name, limit, tid, bid, bdim, gdim, wsize);
}

hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t,
                           hipStream_t) {
    Launch l{};
    const std::string& name = names()[f];
    strncpy(l.name, name.c_str(), sizeof(l.name) - 1);
    const uint32_t g[3] = {grid.x, grid.y, grid.z}, b[3] = {block.x, block.y, block.z};
    memcpy(l.grid, g, sizeof(g));
    memcpy(l.block, b, sizeof(b));
    const auto is = [&](const char* s) { return name.find(s) != std::string::npos; };
    if (is("gemm_tile_kernel"))
        gemm(l, arg<vpa::GemmTask>(args, 0),
             grid.x / (arg<uint32_t>(args, 1) * arg<uint32_t>(args, 2)), arg<float*>(args, 4));
    else if (is("gemm_few_rows_kernel"))
        gemm(l, arg<vpa::GemmTask>(args, 0), grid.y, arg<float*>(args, 2));
    else if (is("gemm_join_kernel"))
        gemm(l, arg<vpa::GemmTask>(args, 0), arg<int32_t>(args, 1),
             arg<vpa::GemmTask>(args, 0).ws);
    else if (is("linear_rows_kernel"))
        gemm(l, arg<vpa::GemmTask>(args, 0), 1, nullptr);
    else if (is("logprob_part_kernel")) {
        const auto& cut = arg<vpa::LogprobCut>(args, 1);
        l.slices = cut.segments;
        l.chunks = cut.chunks_per_segment;
        l.k = cut.vecs;
    }
    launches().push_back(l);
    return hipSuccess;
}

}  // extern "C"
