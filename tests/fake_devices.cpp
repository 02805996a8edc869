// A stand-in for the runtime calls that the library's launches make: two devices that run nothing,
// keep attributes of kernels per device as real ones do, and list what was launched.  The
// library's objects are linked with it (ld --wrap), so their host code runs as it is.
#include <cuda_runtime.h>

#include <cstring>
#include <map>
#include <mutex>
#include <vector>

namespace {

struct Launch {
    int device;
    unsigned grid[3], block;
    unsigned long long smem;
};
constexpr int kSms[2] = {152, 80};
std::mutex lock;
int device = 0, fail_attributes = 0, fail_launches = 0;
cudaError_t last = cudaSuccess;
std::map<const void*, int> allowed[2];   // dynamic shared memory of a kernel, where set
std::vector<Launch> launches;
thread_local struct {
    dim3 grid, block;
    size_t smem;
    cudaStream_t stream;
} config;

cudaError_t launch(const void* kernel, dim3 grid, dim3 block, size_t smem) {
    std::lock_guard<std::mutex> hold(lock);
    if (fail_launches > 0) {
        --fail_launches;
        return last = cudaErrorInvalidValue;
    }
    const auto it = allowed[device].find(kernel);
    const size_t most = it == allowed[device].end() ? 48 * 1024 : it->second;
    if (smem > most || !grid.x || !grid.y || !grid.z || grid.x > 0x7fffffffu || grid.y > 65535)
        return last = cudaErrorInvalidValue;
    launches.push_back({device, {grid.x, grid.y, grid.z}, block.x, smem});
    return cudaSuccess;
}

}  // namespace

extern "C" {

// ---- for the test ----
void fake_reset() {
    std::lock_guard<std::mutex> hold(lock);
    launches.clear();
    last = cudaSuccess;
    fail_attributes = fail_launches = 0;
}
void fake_use(int d) { device = d; }
void fake_fail_attributes(int n) { fail_attributes = n; }
void fake_fail_launches(int n) { fail_launches = n; }
int fake_sms(int d) { return kSms[d]; }
int fake_launches(Launch* out, int most) {
    const int n = (int)launches.size();
    for (int i = 0; i < n && i < most; ++i) out[i] = launches[i];
    return n;
}

// ---- for the library ----
cudaError_t __wrap_cudaGetDevice(int* d) {
    *d = device;
    return cudaSuccess;
}
cudaError_t __wrap_cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int d) {
    *v = a == cudaDevAttrMultiProcessorCount ? kSms[d] : 0;
    return cudaSuccess;
}
cudaError_t __wrap_cudaGetLastError() {
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
cudaError_t __wrap_cudaFuncSetAttribute(const void* kernel, cudaFuncAttribute a, int v) {
    std::lock_guard<std::mutex> hold(lock);
    if (fail_attributes > 0) {
        --fail_attributes;
        return last = cudaErrorInvalidValue;
    }
    if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) allowed[device][kernel] = v;
    return cudaSuccess;
}
cudaError_t __wrap_cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t,
                                                                         unsigned) {
    *n = 2;
    return cudaSuccess;
}
cudaError_t __wrap_cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* cfg) {
    *n = kSms[device] / (int)cfg->attrs[0].val.clusterDim.x;
    return cudaSuccess;
}
unsigned __wrap___cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, cudaStream_t stream) {
    config = {grid, block, smem, stream};
    return 0;
}
cudaError_t __wrap___cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* smem, void* stream) {
    *grid = config.grid;
    *block = config.block;
    *smem = config.smem;
    std::memcpy(stream, &config.stream, sizeof(cudaStream_t));
    return cudaSuccess;
}
cudaError_t __wrap___cudaGetKernel(cudaKernel_t* handle, const void* kernel) {
    *handle = reinterpret_cast<cudaKernel_t>(const_cast<void*>(kernel));
    return cudaSuccess;
}
cudaError_t __wrap___cudaLaunchKernel(cudaKernel_t kernel, dim3 grid, dim3 block, void**, size_t smem,
                                      cudaStream_t) {
    return launch(kernel, grid, block, smem);
}
cudaError_t __wrap_cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void* kernel, void**) {
    return launch(kernel, cfg->gridDim, cfg->blockDim, cfg->dynamicSmemBytes);
}

}  // extern "C"
