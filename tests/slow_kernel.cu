// A kernel for tests: lets its dependents start at once (programmatic dependent
// launch), runs for `ns` nanoseconds, and copies n bytes at its end.  It holds one
// warp of one SM and always ends (the sleeps are counted).
#include <cuda_runtime.h>
#include <stdint.h>

__global__ void slow_copy_kernel(const uint8_t *src, uint8_t *dst, long long n, long long ns) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (int i = 0; i < 1000000; i++) {
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if ((long long)(t - t0) >= ns) break;
        __nanosleep(1000);
    }
    for (long long i = threadIdx.x; i < n; i += 32) dst[i] = src[i];
}

extern "C" int slow_copy(const void *src, void *dst, long long n, long long ns, void *stream) {
    slow_copy_kernel<<<1, 32, 0, (cudaStream_t)stream>>>((const uint8_t *)src, (uint8_t *)dst, n, ns);
    return (int)cudaGetLastError();
}
