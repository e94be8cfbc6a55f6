/* A CUDA runtime of several devices for host tests: a kernel may be launched with more than 48 KB of dynamic shared memory only on a
   device on which its limit was raised before.  Preloaded over libcudart; nothing runs. */
#include <cuda_runtime_api.h>
#include <stddef.h>

static int current;
static struct { const void* func; int device, bytes; } raised[256];
static int count;
static cudaError_t last;

void fake_set_device(int d) { current = d; }
int fake_raised(void) { return count; }

cudaError_t CUDARTAPI cudaGetDevice(int* d) {
    *d = current;
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaFuncSetAttribute(const void* func, enum cudaFuncAttribute attr, int value) {
    if (attr != cudaFuncAttributeMaxDynamicSharedMemorySize || count == 256) return cudaErrorInvalidValue;
    raised[count].func = func;
    raised[count].device = current;
    raised[count++].bytes = value;
    return cudaSuccess;
}
static cudaError_t launch(const void* func, size_t bytes) {
    int limit = 48 * 1024;
    for (int i = 0; i < count; ++i)
        if (raised[i].func == func && raised[i].device == current) limit = raised[i].bytes;
    return last = bytes <= (size_t)limit ? cudaSuccess : cudaErrorInvalidValue;
}
cudaError_t CUDARTAPI cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* func, void** args) {
    (void)args;
    return launch(func, c->dynamicSmemBytes);
}
/* what a <<< >>> launch calls */
cudaError_t CUDARTAPI __cudaGetKernel(cudaKernel_t* kernel, const void* func) {
    *kernel = (cudaKernel_t)func;
    return cudaSuccess;
}
cudaError_t CUDARTAPI __cudaLaunchKernel(cudaKernel_t kernel, dim3 grid, dim3 block, void** args, size_t bytes, cudaStream_t s) {
    (void)grid, (void)block, (void)args, (void)s;
    return launch((const void*)kernel, bytes);
}
cudaError_t CUDARTAPI cudaGetLastError(void) {
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}

static int encode(void) { return 0; }                    /* a tensor map: any arguments, success */
cudaError_t CUDARTAPI cudaGetDriverEntryPointByVersion(const char* name, void** fn, unsigned version, unsigned long long flags,
                                                       enum cudaDriverEntryPointQueryResult* status) {
    (void)name, (void)version, (void)flags;
    *fn = (void*)encode;
    *status = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
