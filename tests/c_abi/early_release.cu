// A kernel that lets the next one in the stream start at once, works for `ns`
// nanoseconds more (at most about four times that), and writes its output, n
// bytes of known values, at the end.
#include <cuda_runtime.h>

#include <cstdint>

namespace {

__global__ void work(int8_t* out, long long n, unsigned long long ns) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (unsigned long long i = 0; i < ns / 500; ++i) {
        __nanosleep(1000);
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t - t0 >= ns) break;
    }
    for (long long i = threadIdx.x; i < n; i += blockDim.x) out[i] = (int8_t)(i * 7 % 251 - 125);
}

}  // namespace

extern "C" int early_release(void* out, long long n, unsigned long long ns, void* stream) {
    work<<<1, 256, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<int8_t*>(out), n, ns);
    return (int)cudaGetLastError();
}
