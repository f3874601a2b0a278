// The runtime calls that cluster_grid makes, for cluster_grid.cu: what fits is told by the
// kernel's address and the device.
#include <cuda_runtime_api.h>

void wide(int) {}
void narrow(int) {}
void never(int) {}

int device = 0, asked = 0;

extern "C" cudaError_t cudaGetDevice(int* d)
{
    *d = device;
    return cudaSuccess;
}

extern "C" cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int)
{
    *v = 152;
    return cudaSuccess;
}

extern "C" cudaError_t cudaGetLastError() { return cudaSuccess; }

extern "C" cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t*)
{
    ++asked;
    *n = f == (const void*)wide ? 76 - device : f == (const void*)narrow ? 40 : 0;
    return cudaSuccess;
}
