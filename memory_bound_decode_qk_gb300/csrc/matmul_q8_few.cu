// matmul_q8_few.cu -- the 8-bit product of a few tokens (sm_103a): a stream of weights.
//
// With up to 8 tokens a weight byte takes part in 16 operations at most, so the call is
// bound by reading the weights once, and a small one by the round trip to memory.  They
// go from global memory straight into the registers of the warp-level matrix
// instructions: the order of the summed dimension is free as long as both operands
// share it, so a lane's 16 bytes of a row are the operand registers of two (E4M3,
// m16n8k32) or four (int8, widened to fp16, m16n8k16) instructions, and no shared
// memory is passed.  The weights are the operand with 16 rows: a CTA owns 16 channels
// and all of the summed dimension, cut over its warps, and each lane has 8 loads of 16
// bytes in flight.  The warps' sums are added in a fixed order.  Measured on GB300, one
// token, 6144 channels, 2560 terms (15.8 MB): E4M3 5.8 us (2.7 TB/s; 80 registers put two
// CTAs of 10 warps on an SM, 304 of the 384), int8 6.4 (8 warps, all 384 at once); 2560 x
// 2560: 3.1 and 5.3.
//
// int8 goes through fp16 as in matmul_q8_tc.cu: sums of at most 1024 terms are exact
// in fp32 and then join an int32.
#include "matmul_common.cuh"

namespace edge {
namespace {

constexpr int kStepBytes = 64;  // of a row, for the four lanes that share it

__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 load_stream(const char* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }

// Warps of a CTA, each with at least 4 steps.  Measured on GB300, one token: E4M3 with 8
// warps 3.9 us (2560 x 2560), with 12 2.9; int8, whose widening needs more registers, with
// 8 warps 7.0 us (6144 x 2560), with 12 9.5.
template <bool INT8> constexpr int kWarps = INT8 ? 8 : 12;

template <bool INT8>
__global__ void __launch_bounds__(32 * kWarps<INT8>, 768 / (32 * kWarps<INT8>)) matmul_few_kernel(MatmulP p) {
    constexpr int U = 4, PART = 16 * 8;
    __shared__ uint32_t parts[kWarps<INT8> * PART];  // [warps][tokens][channels]
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int n0 = blockIdx.x * 16;
    if (threadIdx.x == 0) {
        // this CTA's weights into L2 while the preceding grid drains
        prefetch_l2(p.w, (int64_t)n0 * p.k, (int64_t)min(n0 + 16, p.n) * p.k);
    }
    pdl_wait();
    pdl_launch_dependents();

    const int steps = (p.k + kStepBytes - 1) / kStepBytes;
    const int s0 = steps * wid / warps, s1 = steps * (wid + 1) / warps;
    const char* wrow = p.w + (int64_t)(n0 + g) * p.k;
    const char* arow = p.a + (int64_t)g * p.k;
    const bool row0 = n0 + g < p.n, row1 = n0 + g + 8 < p.n;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int whole[4] = {0, 0, 0, 0};
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    int terms = 0;
    for (int s = s0; s < s1; s += U) {
        uint4 w[U][2], a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s + u) * kStepBytes + c * 16;
            const bool ok = s + u < s1 && k < p.k;
            w[u][0] = ok && row0 ? load_stream(wrow + k) : zero;
            w[u][1] = ok && row1 ? load_stream(wrow + (int64_t)8 * p.k + k) : zero;
            a[u] = ok && g < p.tokens ? __ldg(reinterpret_cast<const uint4*>(arow + k)) : zero;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&w[u][0]);
            const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&w[u][1]);
            const uint32_t* b = reinterpret_cast<const uint32_t*>(&a[u]);
            if constexpr (INT8) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t x[4], lo, hi;
                    widen4(w0[q], x[0], x[2]);
                    widen4(w1[q], x[1], x[3]);
                    widen4(b[q], lo, hi);
                    mma_f16(acc, x, lo, hi);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    const uint32_t x[4] = {w0[q], w1[q], w0[q + 1], w1[q + 1]};
                    mma_e4m3(acc, x, b[q], b[q + 1]);
                }
            }
        }
        if constexpr (INT8) {
            terms += U * kStepBytes;
            if (terms + U * kStepBytes > 1024) {
                terms = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    whole[i] += __float2int_rn(acc[i]);
                    acc[i] = 0.0f;
                }
            }
        }
    }
    // parts in shared memory: the channel runs fastest, as in the output
    uint32_t* mine = parts + wid * PART;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int ch = g + 8 * (e >> 1), t = 2 * c + (e & 1);
        mine[t * 16 + ch] = INT8 ? (uint32_t)(whole[e] + __float2int_rn(acc[e])) : __float_as_uint(acc[e]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < PART; i += blockDim.x) {
        const int t = i / 16, n = n0 + i % 16;
        if (t >= p.tokens || n >= p.n) continue;
        float sum = 0.0f;
        int exact = 0;
        for (int k = 0; k < warps; ++k) {
            const uint32_t v = parts[k * PART + i];
            if constexpr (INT8) {
                exact += (int)v;
            } else {
                sum = __fadd_rn(sum, __uint_as_float(v));
            }
        }
        if constexpr (INT8) sum = __int2float_rn(exact);
        const float bias = p.bias != nullptr ? load_out(p.bias, n, p.out_dt) : 0.0f;
        store_out(p.out, (int64_t)t * p.n + n, scaled(sum, __ldg(p.sa + t), __ldg(p.sw + n), bias), p.out_dt);
    }
}

template <bool INT8>
cudaError_t launch_kind(const MatmulP& p, cudaLaunchConfig_t cfg) {
    const int steps = (p.k + kStepBytes - 1) / kStepBytes, warps = (steps + 3) / 4;
    cfg.gridDim = dim3((unsigned)((p.n + 15) / 16));
    cfg.blockDim = dim3(32 * (warps < kWarps<INT8> ? warps : kWarps<INT8>));
    return cudaLaunchKernelEx(&cfg, matmul_few_kernel<INT8>, p);
}

}  // namespace

// At most 8 tokens and 16 MB of weights, rows and addresses on 16 bytes.  Measured on
// GB300 against the kernel on tensor memory, us, E4M3 with one and eight tokens and int8 (the
// same with one and eight):
//                      E4M3 1       E4M3 8       int8
//      512 x 2560    2.2   4.7    2.4   4.7    3.9   6.5
//     2560 x 2560    3.1   5.3    3.3   5.3    5.3   7.1
//     2560 x 4096    4.7   5.6    5.0   5.7    5.9   8.1
//     6144 x 2560    5.8   6.1    6.2   6.1    6.4   8.6 to 8.9
//   16,384 x 1024    5.0   5.1    5.2   4.9    7.2   6.4
//     1600 x 9728    6.2   7.2    6.4   7.2   12.2   9.5
//     2560 x 9728    8.5   8.7    8.8   8.7   13.1  10.8    (above 16 MB)
//   19,456 x 2560   12.8  10.6   13.2  10.6   18.4  12.0    (above 16 MB)
// Where the rule loses: few channels with a long sum, which the other kernel cuts over a
// cluster and this one only over a CTA's warps (512 x 9728 5.7 and 5.4, int8 11.6 and 7.8;
// 256 x 16,384 8.2 and 6.1, int8 18.5 and 9.3).
bool matmul_few_suits(const MatmulP& m) {
    return m.tokens <= 8 && (int64_t)m.n * m.k <= (16 << 20) && m.k % 16 == 0 &&
           reinterpret_cast<uintptr_t>(m.a) % 16 == 0 && reinterpret_cast<uintptr_t>(m.w) % 16 == 0;
}

cudaError_t launch_matmul_few(const MatmulP& m, int q_dt, cudaLaunchConfig_t cfg) {
    return q_dt == kInt8 ? launch_kind<true>(m, cfg) : launch_kind<false>(m, cfg);
}

}  // namespace edge
