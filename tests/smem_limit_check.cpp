// A kernel's shared-memory limit belongs to the device's context: it is asked
// for at every launch, so a context made anew (cudaDeviceReset) has it too.
// The runtime's calls are stand-ins here.
#include <cstdio>
#include <map>
#include <set>

#include "fp8q_internal.h"

static int device = 0, calls = 0;
static std::map<int, std::set<const void*>> allowed;       // by device: kernels that have the limit
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int bytes) {
    ++calls;
    if (a != cudaFuncAttributeMaxDynamicSharedMemorySize || bytes > 232448) return cudaErrorInvalidValue;
    allowed[device].insert(f);
    return cudaSuccess;
}

static void kernel() {}

int main() {
    bool ok = true;
    for (device = 0; device < 2; ++device)
        for (int call = 0; call < 3; ++call) {
            ok = ok && fp8q::allow_smem(kernel, 1024) == cudaSuccess;
            ok = ok && allowed[device].count(reinterpret_cast<const void*>(kernel));
            allowed[device].clear();                       // the device is reset
        }
    device = 0;
    ok = ok && fp8q::allow_smem(kernel, 1 << 20) != cudaSuccess;      // refused: handed on
    std::printf("%s: %d calls\n", ok ? "ok" : "a launch without its limit", calls);
    return !ok;
}
