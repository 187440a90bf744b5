/* A CUDA runtime for host code without a GPU: memory of the host, one device of
 * compute capability 10.3 with 152 SMs, launches that only leave a line in a log.
 * Copies and fills reach their destination when the stream that they are queued
 * on (the legacy one) is synchronised, which is the least that CUDA promises of
 * a copy from pageable memory and of a fill. */
#include <cuda_runtime_api.h>
#include <stdarg.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

static char log_text[1 << 20];
static size_t log_at;
static void note(const char *f, ...) {
    va_list v;
    va_start(v, f);
    const int n = vsnprintf(log_text + log_at, sizeof(log_text) - log_at, f, v);
    va_end(v);
    if (n > 0 && log_at + n < sizeof(log_text)) log_at += n;
}
const char *fake_log(void) { return log_text; }
void fake_clear(void) { log_text[log_at = 0] = 0; }

static struct Queued { void *dst, *src; int value; size_t bytes; } queued[64];
static int waiting;
int fake_queued(void) { return waiting; }
static cudaError_t later(void *dst, const void *src, int value, size_t bytes) {
    if (waiting == 64) return cudaErrorMemoryAllocation;
    struct Queued q = {dst, 0, value, bytes};
    if (src) memcpy(q.src = malloc(bytes), src, bytes);
    queued[waiting++] = q;
    return cudaSuccess;
}
static void finish(void) {
    for (int i = 0; i < waiting; ++i) {
        if (queued[i].src) memcpy(queued[i].dst, queued[i].src, queued[i].bytes);
        else memset(queued[i].dst, queued[i].value, queued[i].bytes);
        free(queued[i].src);
    }
    waiting = 0;
}

static int *word; /* the last allocation of four bytes */
void fake_set_word(int v) { finish(); *word = v; }

cudaError_t cudaMalloc(void **p, size_t bytes) {
    *p = aligned_alloc(256, (bytes + 255) / 256 * 256);
    if (*p) memset(*p, 0xcd, bytes);
    if (bytes == 4) word = *p;
    return *p ? cudaSuccess : cudaErrorMemoryAllocation;
}
cudaError_t cudaFree(void *p) { finish(); free(p); return cudaSuccess; }
cudaError_t cudaMemcpy(void *dst, const void *src, size_t bytes, enum cudaMemcpyKind kind) {
    if (kind == cudaMemcpyHostToDevice) return later(dst, src, 0, bytes);
    finish();
    memcpy(dst, src, bytes);
    return cudaSuccess;
}
cudaError_t cudaMemset(void *p, int value, size_t bytes) { return later(p, 0, value, bytes); }
cudaError_t cudaMemsetAsync(void *p, int value, size_t bytes, cudaStream_t st) {
    note("memset %zu\n", bytes);
    memset(p, value, bytes);
    return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t st) {
    if (st == 0 || st == cudaStreamLegacy) finish();
    return cudaSuccess;
}
cudaError_t cudaDeviceSynchronize(void) { finish(); return cudaSuccess; }
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, enum cudaDeviceAttr a, int device) {
    switch (a) {
    case cudaDevAttrComputeCapabilityMajor: *v = 10; return cudaSuccess;
    case cudaDevAttrComputeCapabilityMinor: *v = 3; return cudaSuccess;
    case cudaDevAttrMultiProcessorCount: *v = 152; return cudaSuccess;
    case cudaDevAttrMaxSharedMemoryPerBlockOptin: *v = 227 * 1024; return cudaSuccess;
    case cudaDevAttrMaxSharedMemoryPerMultiprocessor: *v = 228 * 1024; return cudaSuccess;
    default: return cudaErrorInvalidValue;
    }
}
cudaError_t cudaGetDeviceProperties(struct cudaDeviceProp *p, int device) {
    memset(p, 0, sizeof(*p));
    p->major = 10;
    p->minor = 3;
    p->multiProcessorCount = 152;
    p->sharedMemPerBlockOptin = 227 * 1024;
    return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(struct cudaFuncAttributes *a, const void *f) {
    memset(a, 0, sizeof(*a));
    a->numRegs = 128;
    a->maxThreadsPerBlock = 512;
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void *f, enum cudaFuncAttribute a, int v) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *f, const cudaLaunchConfig_t *c) {
    *n = 1;
    return cudaSuccess;
}
static int encode(void) { return 0; } /* (a tensor map of nothing) */
cudaError_t cudaGetDriverEntryPointByVersion(const char *name, void **f, unsigned version, unsigned long long flags,
                                             enum cudaDriverEntryPointQueryResult *found) {
    *f = (void *)encode;
    *found = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void **p, const void *symbol) { return cudaErrorNotSupported; }

static struct { const void *host; char name[256]; } kernels[2048];
static int known;
const char *fake_kernel(int i) { return i < known ? kernels[i].name : 0; }
static const char *name_of(const void *f) {
    for (int i = 0; i < known; ++i)
        if (kernels[i].host == f) return kernels[i].name;
    return "?";
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **args) {
    unsigned cluster = 1;
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[i].val.clusterDim.x;
    note("%s %u,%u,%u %u %zu %u\n", name_of(f), c->gridDim.x, c->gridDim.y, c->gridDim.z, c->blockDim.x, c->dynamicSmemBytes, cluster);
    return cudaSuccess;
}
cudaError_t cudaLaunchKernel(const void *f, dim3 grid, dim3 block, void **args, size_t smem, cudaStream_t st) {
    note("%s %u,%u,%u %u %zu 1\n", name_of(f), grid.x, grid.y, grid.z, block.x, smem);
    return cudaSuccess;
}

/* What nvcc's host code registers itself with. */
void **__cudaRegisterFatBinary(void *p) { static void *handle; return &handle; }
void __cudaRegisterFatBinaryEnd(void **h) {}
void __cudaUnregisterFatBinary(void **h) {}
void __cudaRegisterVar(void **h, char *v, char *a, const char *n, int e, size_t s, int c, int g) {}
void __cudaRegisterFunction(void **h, const char *host, char *dev, const char *name, int limit, void *t, void *b, void *bd, void *gd, int *w) {
    if (known == 2048) return;
    kernels[known].host = host;
    strncpy(kernels[known++].name, name, sizeof(kernels[0].name) - 1);
}
cudaError_t __cudaGetKernel(cudaKernel_t *k, const void *f) { *k = (cudaKernel_t)f; return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 grid, dim3 block, void **args, size_t smem, cudaStream_t st) {
    return cudaLaunchKernel((const void *)k, grid, block, args, smem, st);
}
unsigned __cudaPopCallConfiguration(dim3 *g, dim3 *b, size_t *s, void *st) { return 0; }
unsigned __cudaPushCallConfiguration(dim3 g, dim3 b, size_t s, void *st) { return 0; }
