// The status word of the int8 product's and the attention's kernels: bit 0 (kStatusTimeout) after a
// wait that ran out.  In a file of its own: its address is asked for without
// loading kernels, the product's or the fused step's (14 ms).
#include <cuda_runtime.h>

#include <atomic>

#include "token_ops.h"

namespace trfn {
namespace {

__device__ unsigned int g_product_status;

std::atomic<unsigned*> g_word[kMaxDevices];   // null: no product has been launched on the device

}  // namespace

int product_status_word(int dev, unsigned** word) {
    unsigned* p = g_word[dev].load(std::memory_order_relaxed);
    if (p == nullptr) {
        void* at = nullptr;
        const cudaError_t e = cudaGetSymbolAddress(&at, g_product_status);
        if (e != cudaSuccess) return cuda_failed("cudaGetSymbolAddress(int8 product)", (int)e);
        p = static_cast<unsigned*>(at);
        g_word[dev].store(p, std::memory_order_relaxed);
    }
    *word = p;
    return TR_OK;
}

int read_product_status(int* flags, bool clear) {
    *flags = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev >= kMaxDevices) return TR_OK;   // no product runs there
    unsigned* const p = e == cudaSuccess ? g_word[dev].load(std::memory_order_relaxed) : nullptr;
    unsigned v = 0;
    if (p != nullptr) e = cudaMemcpy(&v, p, sizeof v, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && clear && v != 0) e = cudaMemset(p, 0, sizeof v);
    if (e != cudaSuccess) return cuda_failed("tr_device_status (int8 product)", (int)e);
    *flags = (int)v;
    return TR_OK;
}

}  // namespace trfn
