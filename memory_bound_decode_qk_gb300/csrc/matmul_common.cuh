// matmul_common.cuh -- what the kernels of the 8-bit product share: its parameters,
// the scales' epilogue, warp-level products and clusters.
#pragma once

#include "edge_common.cuh"
#include "launch.h"

namespace edge {

struct MatmulP {
    const char* a;         // [tokens, k]
    const char* w;         // [n, k]
    const float* sa;
    const float* sw;
    const char* bias;      // nullable
    char* out;
    int tokens, n, k;
    int out_dt;
};

__device__ __forceinline__ float load_out(const char* p, int64_t i, int dt) {
    if (dt == kF32) return reinterpret_cast<const float*>(p)[i];
    if (dt == kF16) return to_f(reinterpret_cast<const __half*>(p)[i]);
    return to_f(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_out(char* p, int64_t i, float v, int dt) {
    if (dt == kF32) {
        reinterpret_cast<float*>(p)[i] = v;
    } else if (dt == kF16) {
        reinterpret_cast<__half*>(p)[i] = from_f<__half>(v);
    } else {
        reinterpret_cast<__nv_bfloat16*>(p)[i] = from_f<__nv_bfloat16>(v);
    }
}
// The sum (fp32, or int32 rounded to it) times both scales, plus the bias.
__device__ __forceinline__ float scaled(float sum, float sa, float sw, float bias) {
    return __fadd_rn(__fmul_rn(__fmul_rn(sum, sa), sw), bias);
}

// Four int8 to four fp16 numbers: a byte with its sign bit turned, in the low bits of
// an fp16 number of exponent 2^10, is 1024 + 128 + the value.
__device__ __forceinline__ void widen4(uint32_t v, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = v ^ 0x80808080u;
    const __half2 bias = __floats2half2_rn(-1152.0f, -1152.0f);
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hadd2(*reinterpret_cast<const __half2*>(&a), bias);
    const __half2 y = __hadd2(*reinterpret_cast<const __half2*>(&b), bias);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

// d += A B of one warp, 16 rows, 8 columns and 16 terms.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// All threads of the cluster.  The barrier takes whole warps, whose lanes may come here one
// by one from the stores of a ragged tile.
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// This CTA's shared-memory address as CTA `rank` of the cluster has it.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, int rank) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    return at;
}
__device__ __forceinline__ uint32_t peer_word(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint4 peer_vector(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// A few tokens (matmul_q8_few.cu).
bool matmul_few_suits(const MatmulP& m);
cudaError_t launch_matmul_few(const MatmulP& m, int q_dt, cudaLaunchConfig_t cfg);

// On the tensor memory (matmul_q8_tc.cu).  cfg has room for one more attribute.
bool matmul_tc_suits(const MatmulP& m);
cudaError_t launch_matmul_tc(const MatmulP& m, int q_dt, cudaLaunchConfig_t cfg);

}  // namespace edge
