// glu.cu -- SiLU / tanh-GELU gated activations of a merged gate+up row (sm_103a).
//
// What it computes ("thox-edge-ops v2", section 5.1; FlashRT
// gate_geglu_merged_fp8): out[t, i] = act(g) * u with g = gate_up[t, i],
// u = gate_up[t, d + i].  The gate is the first half of each row.
// The two activations and their two precisions are in glu_math.cuh.
//
// GB300 design.  It is a pure stream: it reads 2 elements and writes 1 per
// output.  The rows are flattened into one index space of 16-byte vectors.
// Each thread issues its U gate and U up loads before any arithmetic.  A
// multiply-high divide turns a flat index into (row, column).  Stores are
// 16 bytes, or 8 bytes of E4M3 codes: four codes per 32-bit word.
#include "edge_common.cuh"
#include "fastdiv.h"
#include "glu_math.cuh"
#include "launch.h"

namespace edge {
namespace {

struct GluP {
    const char* gu;
    char* out;
    uint32_t total;   // rows * dvec (vector path) or rows * d (generic, 64-bit below)
    FastDiv dv;       // 16-byte vectors per half row
    int64_t rows;
    int64_t d;
    float inv;
};

template <typename T, bool FP8, int ACT, int U>
__global__ void __launch_bounds__(256) glu_vec_kernel(GluP p) {
    constexpr int N = vec_elems<T>();
    const uint32_t dv = p.dv.d;
    const uint4* gu = reinterpret_cast<const uint4*>(p.gu);
    const uint32_t stride = gridDim.x * blockDim.x * U;

    if (threadIdx.x == 0) {
        // this CTA's first vectors into L2 while the preceding grid drains:
        // flat vectors [i0, i1) lie in rows r0..r1, gate then up in each row
        const uint32_t i0 = blockIdx.x * blockDim.x * U;
        const uint32_t i1 = i0 + blockDim.x * U < p.total ? i0 + blockDim.x * U : p.total;
        if (i0 < i1) {
            const int64_t r0 = fast_div(i0, p.dv), r1 = fast_div(i1 - 1, p.dv);
            const int64_t row = 32 * (int64_t)dv;  // bytes of one [g | u] row
            if (r1 > r0 + 1) {
                prefetch_l2(p.gu, r0 * row, (r1 + 1) * row);
            } else {
                for (int64_t r = r0; r <= r1; ++r) {
                    const int64_t c0 = (int64_t)i0 > r * dv ? (int64_t)i0 - r * dv : 0;
                    const int64_t c1 = (int64_t)i1 < (r + 1) * dv ? (int64_t)i1 - r * dv : dv;
                    prefetch_l2(p.gu, r * row + 16 * c0, r * row + 16 * c1);
                    prefetch_l2(p.gu, r * row + 16 * (dv + c0), r * row + 16 * (dv + c1));
                }
            }
        }
    }
    pdl_wait();
    pdl_launch_dependents();

    for (uint32_t b0 = blockIdx.x * blockDim.x * U + threadIdx.x; b0 < p.total; b0 += stride) {
        uint4 gv[U], uv[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const uint32_t i = b0 + k * blockDim.x;
            if (i < p.total) {
                const uint32_t row = fast_div(i, p.dv);
                const uint32_t col = i - row * dv;
                const uint4* g = gu + (size_t)row * 2 * dv + col;
                gv[k] = __ldcs(g);
                uv[k] = __ldcs(g + dv);
            } else {
                gv[k] = make_uint4(0u, 0u, 0u, 0u);
                uv[k] = gv[k];
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const uint32_t i = b0 + k * blockDim.x;
            if (i >= p.total) continue;
            if constexpr (std::is_same<T, float>::value && !FP8) {
                float g[N], u[N], y[N];
                unpack_vec<T, N>(gv[k], g);
                unpack_vec<T, N>(uv[k], u);
#pragma unroll
                for (int e = 0; e < N; ++e) y[e] = gate_accurate<ACT>(g[e], u[e]);
                reinterpret_cast<uint4*>(p.out)[i] = pack_vec<T, N>(y);
            } else {
                // the fast form on element pairs
                float2 g[N / 2], u[N / 2], y[N / 2];
                unpack_pairs<T, N>(gv[k], g);
                unpack_pairs<T, N>(uv[k], u);
#pragma unroll
                for (int j = 0; j < N / 2; ++j) y[j] = gate_fast2<ACT>(g[j], u[j]);
                if constexpr (FP8) {
                    auto q8 = quantize_pairs<N>(y, p.inv);
                    reinterpret_cast<decltype(q8)*>(p.out)[i] = q8;
                } else {
                    reinterpret_cast<uint4*>(p.out)[i] = pack_pairs<T, N>(y);
                }
            }
        }
    }
}

template <typename T, bool FP8, int ACT>
__global__ void __launch_bounds__(256) glu_generic_kernel(GluP p) {
    const T* gu = reinterpret_cast<const T*>(p.gu);
    const int64_t total = p.rows * p.d;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;

    pdl_wait();
    pdl_launch_dependents();

    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
        const int64_t row = i / p.d;
        const int64_t col = i - row * p.d;
        const float g = to_f(gu[row * 2 * p.d + col]);
        const float u = to_f(gu[row * 2 * p.d + p.d + col]);
        const float y = gate<T, FP8, ACT>(g, u);
        if constexpr (FP8) {
            reinterpret_cast<uint8_t*>(p.out)[i] = quantize1(y, p.inv);
        } else {
            reinterpret_cast<T*>(p.out)[i] = from_f<T>(y);
        }
    }
}

template <typename T, bool FP8, int ACT>
cudaError_t launch_typed(const GluArgs& a, GluP& p, cudaStream_t s) {
    constexpr int N = vec_elems<T>();
    auto aligned = [](const void* ptr, uintptr_t n) {
        return (reinterpret_cast<uintptr_t>(ptr) % n) == 0;
    };
    const int sms = sm_count();
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;

    const int64_t dvec = a.d / N;
    const bool vec = (a.d * (int64_t)sizeof(T)) % 16 == 0 && aligned(a.gate_up, 16) &&
                     aligned(a.out, FP8 ? N : 16) && a.rows * dvec <= kMaxUnits;
    if (vec) {
        p.dv = make_fastdiv((uint32_t)dvec);
        p.total = (uint32_t)(a.rows * dvec);
        const int threads = 256;
        // one vector per thread and a one-shot grid (measured on GB300: 2 or 4
        // vectors per thread were slower at every size timed on its own,
        // 1.1x to 1.2x for the tanh-GELU gate with FP8 output)
        int64_t blocks = ((int64_t)p.total + threads - 1) / threads;
        const int64_t cap = (int64_t)sms * (2048 / threads) * 64;
        if (blocks > cap) blocks = cap;
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(threads);
        return cudaLaunchKernelEx(&cfg, glu_vec_kernel<T, FP8, ACT, 1>, p);
    }
    const int64_t total = a.rows * a.d;
    int64_t blocks = (total + 255) / 256;
    const int64_t cap = (int64_t)sms * 64;
    if (blocks > cap) blocks = cap;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&cfg, glu_generic_kernel<T, FP8, ACT>, p);
}

template <typename T>
cudaError_t launch_dt(const GluArgs& a, GluP& p, cudaStream_t s) {
    const bool fp8 = a.out_dt == kFP8;
    if (a.act == kSilu) {
        return fp8 ? launch_typed<T, true, kSilu>(a, p, s) : launch_typed<T, false, kSilu>(a, p, s);
    }
    return fp8 ? launch_typed<T, true, kGelu>(a, p, s) : launch_typed<T, false, kGelu>(a, p, s);
}

}  // namespace

cudaError_t launch_glu(const GluArgs& a, cudaStream_t s) {
    GluP p;
    p.gu = static_cast<const char*>(a.gate_up);
    p.out = static_cast<char*>(a.out);
    p.total = 0;
    p.dv = make_fastdiv(1);
    p.rows = a.rows;
    p.d = a.d;
    p.inv = a.inv_scale;
    switch (a.dt) {
        case kF32: return launch_dt<float>(a, p, s);
        case kF16: return launch_dt<__half>(a, p, s);
        default: return launch_dt<__nv_bfloat16>(a, p, s);
    }
}

}  // namespace edge
