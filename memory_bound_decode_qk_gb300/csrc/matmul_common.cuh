// matmul_common.cuh -- what the kernels of the 8-bit product share: its parameters
// and the scales' epilogue.
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

// On the tensor memory (matmul_q8_tc.cu).  cfg has room for one more attribute.
bool matmul_tc_suits(const MatmulP& m);
cudaError_t launch_matmul_tc(const MatmulP& m, int q_dt, cudaLaunchConfig_t cfg);

}  // namespace edge
