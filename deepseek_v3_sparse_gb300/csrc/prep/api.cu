// api.cu -- the status word and the device queries of libdsix_prep (the library
// is linked by itself, so it keeps its own).
#include <atomic>

#include "prep.cuh"

namespace {
__device__ int g_status = 0;

constexpr int kMaxDevices = 64;

int current_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
    return dev;
}
}  // namespace

namespace dsix {

int* status_ptr() {
    static std::atomic<int*> cache[kMaxDevices];
    const int dev = current_device();
    if (dev < 0) return nullptr;
    int* p = cache[dev].load(std::memory_order_relaxed);
    if (!p) {
        void* q = nullptr;
        if (cudaGetSymbolAddress(&q, g_status) != cudaSuccess) return nullptr;
        p = static_cast<int*>(q);
        cache[dev].store(p, std::memory_order_relaxed);
    }
    return p;
}

int num_sms() {
    static std::atomic<int> cache[kMaxDevices];
    const int dev = current_device();
    if (dev < 0) return -1;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n <= 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return -1;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

int launch_status() { return cudaGetLastError() == cudaSuccess ? IX_OK : IX_ERR_CUDA; }

}  // namespace dsix

extern "C" int ix_prep_device_status(int* status_out) {
    int v = 0;
    if (cudaDeviceSynchronize() != cudaSuccess) return IX_ERR_CUDA;
    if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return IX_ERR_CUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_status, &zero, sizeof(int)) != cudaSuccess) return IX_ERR_CUDA;
    if (status_out) *status_out = v;
    return v ? IX_ERR_DEVICE_CHECK : IX_OK;
}
