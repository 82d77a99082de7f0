// allow_smem: cudaFuncSetAttribute costs about a microsecond, as much as a small operator runs.
#include "launch.h"

#include <mutex>

namespace redmoe {
namespace {

struct Allowed {
    const void* kern;
    int dev, bytes;
};
constexpr int MAX_ALLOWED = 512;  // kernels times devices; beyond that every call asks the runtime
std::mutex allowed_mutex;
Allowed allowed[MAX_ALLOWED];
int n_allowed = 0;

}  // namespace

bool allow_smem(const void* kern, int bytes) {
    if (bytes <= 40 * 1024) return true;  // within what a launch gets without asking, static part included
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> lock(allowed_mutex);
    Allowed* at = nullptr;
    for (int i = 0; i < n_allowed && !at; ++i)
        if (allowed[i].kern == kern && allowed[i].dev == dev) at = &allowed[i];
    if (at && at->bytes >= bytes) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (at) at->bytes = bytes;
    else if (n_allowed < MAX_ALLOWED) allowed[n_allowed++] = {kern, dev, bytes};
    return true;
}

}  // namespace redmoe
