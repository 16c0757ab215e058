// matmul_q8.cu -- product of 8-bit operands with a scale for each token and output
// channel (sm_103a): the choice of a kernel, and the kernel for any size.
//
//   out[t, j] = round((sum_i a[t, i] w[j, i]) sa[t] sw[j] + bias[j])
//
// Rows and addresses on 16 bytes take the stream of weights (matmul_q8_few.cu: up to 8
// tokens and 16 MB of weights) or the tensor memory (matmul_q8_tc.cu); the rest the
// kernel here.
#include "matmul_common.cuh"

namespace edge {
namespace {

// d += A B of one warp, A 16 x 32 and B 32 x 8 bytes.
template <bool INT8>
__device__ __forceinline__ void mma_16x8x32(uint32_t (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    if constexpr (INT8) {
        asm volatile(
            "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
    } else {
        float* f = reinterpret_cast<float*>(d);
        asm volatile(
            "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(f[0]), "+f"(f[1]), "+f"(f[2]), "+f"(f[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
    }
}

template <bool INT8>
__device__ __forceinline__ float sum_of(uint32_t v) {
    return INT8 ? __int2float_rn((int)v) : __uint_as_float(v);
}

// ---------------------------------------------------------------- any size

// Tiles of 64 tokens x 64 channels, 64 bytes of the summed dimension at a time, on
// the warp-level matrix instructions: 2 x 2 warps of 32 x 32 each.  The next bytes
// are fetched into registers while the tile in shared memory is multiplied.  VW:
// bytes of one load, 4 where they divide the row length and both addresses, else 1.
constexpr int kTileAny = 64;
constexpr int kRowAny = 80;  // bytes of a row in shared memory: fragments without bank conflicts

template <bool INT8, int VW>
__global__ void __launch_bounds__(128) matmul_any_kernel(MatmulP p) {
    __shared__ __align__(16) uint8_t as[2][kTileAny * kRowAny], ws[2][kTileAny * kRowAny];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int tiles_n = (p.n + kTileAny - 1) / kTileAny;
    const int t0 = (int)(blockIdx.x / tiles_n) * kTileAny, n0 = (int)(blockIdx.x % tiles_n) * kTileAny;
    const int row = tid >> 1, half = (tid & 1) * 32;  // this thread's 32 bytes of each tile
    pdl_wait();
    pdl_launch_dependents();

    auto fetch = [&](const char* base, int r, int rows, int k0, uint32_t (&v)[8]) {
        const char* src = base + (int64_t)r * p.k;
        const bool ok = r < rows;
        if constexpr (VW == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = k0 + half + 4 * i;
                v[i] = ok && k < p.k ? __ldg(reinterpret_cast<const uint32_t*>(src + k)) : 0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = k0 + half + 4 * i + j;
                    if (ok && k < p.k) v[i] |= (uint32_t)__ldg(reinterpret_cast<const uint8_t*>(src + k)) << (8 * j);
                }
            }
        }
    };
    auto put = [&](uint8_t* tile, const uint32_t (&v)[8]) {
        uint4* dst = reinterpret_cast<uint4*>(tile + row * kRowAny + half);
        dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
        dst[1] = make_uint4(v[4], v[5], v[6], v[7]);
    };

    uint32_t acc[2][4][4];
#pragma unroll
    for (int i = 0; i < 32; ++i) (&acc[0][0][0])[i] = 0u;
    uint32_t av[8], wv[8];
    fetch(p.a, t0 + row, p.tokens, 0, av);
    fetch(p.w, n0 + row, p.n, 0, wv);
    const int steps = (p.k + 63) / 64;
    const int tw = (wid >> 1) * 32, nw = (wid & 1) * 32, g = lane >> 2, c = (lane & 3) * 4;
    for (int s = 0; s < steps; ++s) {
        uint8_t *at = as[s & 1], *wt = ws[s & 1];
        put(at, av);
        put(wt, wv);
        __syncthreads();  // (the buffer written next was last read before this barrier)
        if (s + 1 < steps) {
            fetch(p.a, t0 + row, p.tokens, (s + 1) * 64, av);
            fetch(p.w, n0 + row, p.n, (s + 1) * 64, wv);
        }
#pragma unroll
        for (int k = 0; k < 64; k += 32) {
            uint32_t a[2][4], b[4][2];
            auto word = [&](const uint8_t* tile, int r, int at_k) {
                return *reinterpret_cast<const uint32_t*>(tile + r * kRowAny + at_k + c);
            };
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[i][0] = word(at, tw + 16 * i + g, k);
                a[i][1] = word(at, tw + 16 * i + g + 8, k);
                a[i][2] = word(at, tw + 16 * i + g, k + 16);
                a[i][3] = word(at, tw + 16 * i + g + 8, k + 16);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                b[j][0] = word(wt, nw + 8 * j + g, k);
                b[j][1] = word(wt, nw + 8 * j + g, k + 16);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_16x8x32<INT8>(acc[i][j], a[i], b[j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = t0 + tw + 16 * i + g + 8 * e;
            if (t >= p.tokens) continue;
            const float sa = p.sa[t];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const int n = n0 + nw + 8 * j + (lane & 3) * 2 + o;
                    if (n >= p.n) continue;
                    const float bias = p.bias != nullptr ? load_out(p.bias, n, p.out_dt) : 0.0f;
                    store_out(p.out, (int64_t)t * p.n + n, scaled(sum_of<INT8>(acc[i][j][2 * e + o]), sa, p.sw[n], bias), p.out_dt);
                }
            }
        }
    }
}

template <bool INT8>
cudaError_t launch_any(const MatmulP& p, cudaLaunchConfig_t cfg) {
    auto fits = [&](int n) {
        return p.k % n == 0 && reinterpret_cast<uintptr_t>(p.a) % n == 0 && reinterpret_cast<uintptr_t>(p.w) % n == 0;
    };
    const int64_t tiles = ((int64_t)(p.tokens + kTileAny - 1) / kTileAny) * ((p.n + kTileAny - 1) / kTileAny);
    if (tiles > INT32_MAX) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3((unsigned)tiles);
    cfg.blockDim = dim3(128);
    if (fits(4)) return cudaLaunchKernelEx(&cfg, matmul_any_kernel<INT8, 4>, p);
    return cudaLaunchKernelEx(&cfg, matmul_any_kernel<INT8, 1>, p);
}

}  // namespace

cudaError_t launch_matmul_q8(const MatmulQ8Args& a, cudaStream_t s) {
    MatmulP p;
    p.a = static_cast<const char*>(a.a);
    p.w = static_cast<const char*>(a.w);
    p.sa = a.a_scales;
    p.sw = a.w_scales;
    p.bias = static_cast<const char*>(a.bias);
    p.out = static_cast<char*>(a.out);
    p.tokens = (int)a.tokens;
    p.n = (int)a.n;
    p.k = (int)a.k;
    p.out_dt = a.out_dt;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    if (matmul_few_suits(p)) return launch_matmul_few(p, a.q_dt, cfg);
    if (matmul_tc_suits(p)) return launch_matmul_tc(p, a.q_dt, cfg);
    return a.q_dt == kInt8 ? launch_any<true>(p, cfg) : launch_any<false>(p, cfg);
}

}  // namespace edge
