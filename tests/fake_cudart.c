/*
 * The part of the CUDA runtime that libfp8q.so's host code calls, without a GPU:
 * two devices of compute capability 10.0, and launches that are checked instead of
 * run. Function attributes belong to the device that is current when they are set,
 * as the runtime has it, and a launch that needs one its device has not been given
 * answers cudaErrorInvalidValue. Linked with the library's objects (built without a
 * runtime of their own) by test_devices_host.py.
 */
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <string.h>

#define DEVICES 2
#define FUNCTIONS 256

static int current;
static struct {
    const void *fn;
    int smem[DEVICES], wide[DEVICES];
} table[FUNCTIONS];
static int launches[DEVICES], refused;

static int find(const void *fn) {
    int i = 0;
    while (i < FUNCTIONS - 1 && table[i].fn && table[i].fn != fn) ++i;
    table[i].fn = fn;
    return i;
}

/* For the test. */
void fake_set_device(int d) { current = d; }
int fake_launches(int d) { return launches[d]; }
int fake_refused(void) { return refused; }

static CUresult encode(CUtensorMap *map, CUtensorMapDataType type, cuuint32_t rank, void *base, const cuuint64_t *dims,
                       const cuuint64_t *strides, const cuuint32_t *box, const cuuint32_t *estr, CUtensorMapInterleave il,
                       CUtensorMapSwizzle sw, CUtensorMapL2promotion l2, CUtensorMapFloatOOBfill fill) {
    cuuint32_t i;
    (void)type, (void)estr, (void)il, (void)sw, (void)l2, (void)fill;
    memset(map, 0, sizeof *map);
    if ((size_t)base % 16) return CUDA_ERROR_INVALID_VALUE;
    for (i = 0; i < rank; ++i)
        if (!dims[i] || dims[i] > 1ull << 32 || !box[i] || box[i] > 256) return CUDA_ERROR_INVALID_VALUE;
    for (i = 0; i + 1 < rank; ++i)
        if (strides[i] % 16 || strides[i] >= 1ull << 40) return CUDA_ERROR_INVALID_VALUE;
    return CUDA_SUCCESS;
}

cudaError_t CUDARTAPI cudaGetDevice(int *d) {
    *d = current;
    return cudaSuccess;
}

cudaError_t CUDARTAPI cudaDeviceGetAttribute(int *v, enum cudaDeviceAttr a, int d) {
    if (d < 0 || d >= DEVICES) return cudaErrorInvalidDevice;
    switch (a) {
    case cudaDevAttrComputeCapabilityMajor: *v = 10; return cudaSuccess;
    case cudaDevAttrComputeCapabilityMinor: *v = 0; return cudaSuccess;
    case cudaDevAttrMultiProcessorCount: *v = 148; return cudaSuccess;
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t CUDARTAPI cudaFuncSetAttribute(const void *fn, enum cudaFuncAttribute a, int v) {
    const int i = find(fn);
    if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) {
        if (v > 227 * 1024) return cudaErrorInvalidValue;
        table[i].smem[current] = v;
    } else if (a == cudaFuncAttributeNonPortableClusterSizeAllowed) {
        table[i].wide[current] = v;
    }
    return cudaSuccess;
}

cudaError_t CUDARTAPI cudaFuncGetAttributes(struct cudaFuncAttributes *a, const void *fn) {
    (void)fn;
    memset(a, 0, sizeof *a);
    a->numRegs = 168;
    return cudaSuccess;
}

static cudaError_t launch(const void *fn, dim3 grid, dim3 block, size_t smem, unsigned cluster) {
    const int i = find(fn);
    if (!grid.x || grid.x > 0x7FFFFFFFu || grid.y != 1 || grid.z != 1 || !block.x || block.x > 1024 || grid.x % cluster ||
        (smem > 48 * 1024 && smem > (size_t)table[i].smem[current]) || cluster > 16 || (cluster > 8 && !table[i].wide[current])) {
        ++refused;
        return cudaErrorInvalidValue;
    }
    ++launches[current];
    return cudaSuccess;
}

cudaError_t CUDARTAPI cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *fn, void **args) {
    unsigned i, cluster = 1;
    (void)args;
    for (i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[i].val.clusterDim.x;
    return launch(fn, c->gridDim, c->blockDim, c->dynamicSmemBytes, cluster ? cluster : 1);
}

static struct {
    dim3 grid, block;
    size_t smem;
    void *stream;
} pushed;

unsigned CUDARTAPI __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, void *stream) {
    pushed.grid = grid, pushed.block = block, pushed.smem = smem, pushed.stream = stream;
    return 0;
}

cudaError_t CUDARTAPI __cudaPopCallConfiguration(dim3 *grid, dim3 *block, size_t *smem, void *stream) {
    *grid = pushed.grid, *block = pushed.block, *smem = pushed.smem, *(void **)stream = pushed.stream;
    return cudaSuccess;
}

cudaError_t CUDARTAPI cudaLaunchKernel(const void *fn, dim3 grid, dim3 block, void **args, size_t smem, cudaStream_t s) {
    (void)args, (void)s;
    return launch(fn, grid, block, smem, 1);
}

cudaError_t CUDARTAPI cudaGetDriverEntryPoint(const char *name, void **fn, unsigned long long flags, enum cudaDriverEntryPointQueryResult *q) {
    (void)flags;
    *fn = strcmp(name, "cuTensorMapEncodeTiled") ? 0 : (void *)encode;
    *q = *fn ? cudaDriverEntryPointSuccess : cudaDriverEntryPointSymbolNotFound;
    return cudaSuccess;
}

cudaError_t CUDARTAPI cudaGetLastError(void) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaGetSymbolAddress(void **p, const void *symbol) {
    *p = (void *)symbol;
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaMemcpyFromSymbol(void *to, const void *symbol, size_t n, size_t at, enum cudaMemcpyKind kind) {
    (void)symbol, (void)at, (void)kind;
    memset(to, 0, n);
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaMemcpyToSymbol(const void *symbol, const void *from, size_t n, size_t at, enum cudaMemcpyKind kind) {
    (void)symbol, (void)from, (void)n, (void)at, (void)kind;
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaMemsetAsync(void *p, int v, size_t n, cudaStream_t s) {
    (void)p, (void)v, (void)n, (void)s;
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaStreamSynchronize(cudaStream_t s) {
    (void)s;
    return cudaSuccess;
}

static void *handle;
void **CUDARTAPI __cudaRegisterFatBinary(void *bin) {
    (void)bin;
    return &handle;
}
void CUDARTAPI __cudaRegisterFatBinaryEnd(void **h) { (void)h; }
void CUDARTAPI __cudaUnregisterFatBinary(void **h) { (void)h; }
void CUDARTAPI __cudaRegisterFunction(void **h, const char *host, char *dev, const char *name, int limit, uint3 *tid, uint3 *bid,
                                      dim3 *bdim, dim3 *gdim, int *wsize) {
    (void)h, (void)host, (void)dev, (void)name, (void)limit, (void)tid, (void)bid, (void)bdim, (void)gdim, (void)wsize;
}
void CUDARTAPI __cudaRegisterVar(void **h, char *host, char *dev, const char *name, int ext, size_t size, int constant, int global) {
    (void)h, (void)host, (void)dev, (void)name, (void)ext, (void)size, (void)constant, (void)global;
}
