// The runtime calls of the library's host code, on a machine without a GPU: questions get a
// GB300's answers or fail, and a launch is noted instead of made.  Linked in place of the CUDA
// runtime with objects of the library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <cstring>
#include <map>
#include <string>

namespace fake {

int device = 0;
bool no_clusters = false;     // the occupancy calculator fails
bool no_registers = false;    // the attribute query fails
int refuse = 0;               // launches that fail before one is made
cudaError_t pending = cudaSuccess;

struct Launch {
    std::string kernel;
    unsigned grid, block, cluster;
    size_t smem;
    char args[256];           // of the kernel's first parameter
};
Launch last;
int launches = 0;
std::map<const void*, std::string> names;

inline cudaError_t fail(cudaError_t e) {
    pending = e;
    return e;
}

// Clusters of n CTAs resident at once, as a GB300 of 152 SMs answered.
inline int clusters(const std::string& kernel, int n) {
    static const int tensor[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
    static const int any[9] = {0, 456, 228, 148, 110, 87, 74, 59, 51};
    return (kernel.find("matmul_any_kernel") != std::string::npos ? any : tensor)[n];
}

}  // namespace fake

extern "C" {
void** __cudaRegisterFatBinary(void*) {
    static void* handle;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* fn, char*, const char* name, int, void*, void*, void*, void*, int*) {
    fake::names[fn] = name;
}
cudaError_t cudaGetDevice(int* d) {
    *d = fake::device;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
    *v = a == cudaDevAttrMultiProcessorCount ? 152 : 0;
    return cudaSuccess;
}
cudaError_t cudaGetLastError() {
    const cudaError_t e = fake::pending;
    fake::pending = cudaSuccess;
    return e;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* f, const void*) {
    if (fake::no_registers) return fake::fail(cudaErrorUnknown);
    f->numRegs = 80;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* fn, const cudaLaunchConfig_t* cfg) {
    if (fake::no_clusters) return fake::fail(cudaErrorUnknown);
    *n = fake::clusters(fake::names[fn], (int)cfg->attrs[0].val.clusterDim.x);
    return cudaSuccess;
}
static CUresult fake_encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return CUDA_SUCCESS;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
    *f = (void*)fake_encode;
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void* fn, void** args) {
    if (fake::refuse > 0) {
        --fake::refuse;
        return fake::fail(cudaErrorLaunchOutOfResources);
    }
    fake::Launch l = {fake::names[fn], cfg->gridDim.x, cfg->blockDim.x * cfg->blockDim.y, 1, cfg->dynamicSmemBytes, {}};
    for (unsigned i = 0; i < cfg->numAttrs; ++i) {
        if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension) l.cluster = cfg->attrs[i].val.clusterDim.x;
    }
    std::memcpy(l.args, args[0], 88);
    fake::last = l;
    ++fake::launches;
    return cudaSuccess;
}
}
