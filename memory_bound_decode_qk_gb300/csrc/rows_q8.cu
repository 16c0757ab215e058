// rows_q8.cu -- rows in 8 bits with a scale for each row: RMSNorm with or without
// the residual's addition, gated activation, and quantization alone (sm_103a).
//
// What they compute.  Every row has products p_i:
//   norm       p_i = s_i (w_i + delta), s = x or round_dt(x + residual)
//   gate       p_i = act(g_i) u_i
//   quantize   p_i = x_i
// and from m = max |p_i|, with Q = 127 (int8) or 448 (E4M3),
//   code_i = rne(fl(p_i * inv)),  inv = min(Q / m, 2^126),
//   scale  = step (gate, quantize) or r * step (norm),  step = max(m / Q, 2^-126),
// with fl the rounding to fp32 and inv in fp32 for E4M3, in twice fp32's precision for int8
// so that code_i * scale stands for the row's value.  The norm's factor
// r = 1 / sqrt(mean(s^2) + eps) is common to a row: it leaves the codes as they are
// and enters the scale alone.  So one reduction (the sum of squares and the
// maximum together) is enough where norm-then-quantize would take two, and the
// codes do not depend on the order of any sum.  The bound on the step keeps inv
// finite: rows whose largest product is below Q 2^-126 (an empty row among them)
// lose relative precision instead of dividing by zero.
//
// NaN and infinities.  The maximum is taken so that NaN stays NaN, so the scale of
// a row that holds one is NaN or infinite and the row, multiplied back, is NaN
// wherever its codes are zero.  The codes of such a row mean nothing.
//
// GB300 design.  2 (bf16, fp16) to 4 bytes read per element and input, one
// written: the kernels are bound by HBM, and at few rows by one memory round trip.
// As in rows.cu a row stays in registers from its load to its store: a CTA is
// (32 W) x R threads, W warps share a row and every load of a thread is issued
// before any arithmetic.  The products are held in fp32 from the maximum to the
// codes.  Measured with E4M3 and int8 codes: norm of 4096 x 4096 bf16 10.3 and 10.5 us (4.9
// TB/s, 0.72 of a copy's rate: a CTA that reduces has no next row in flight), with the residual
// 19.1 and 19.2 (6.1), tanh-GELU gate of 4001 x 10,240 35.8 and 36.8 (5.7), quantized 4096 x
// 4096 bf16 9.0 and 9.2 (5.6), 2500 x 4096 fp32 8.1 and 8.2 (6.3).  Rows longer than a CTA
// holds, or of a length or alignment that 16-byte vectors do not suit, take a kernel of one
// CTA per row.
#include "edge_common.cuh"
#include "glu_math.cuh"
#include "launch.h"

namespace edge {
namespace {

enum RowKind { kQuant = 0, kNorm = 1, kAddNorm = 2, kGateSilu = 3, kGateGelu = 4 };

template <int KIND> constexpr bool kIsNorm = KIND == kNorm || KIND == kAddNorm;
template <int KIND> constexpr bool kIsGate = KIND == kGateSilu || KIND == kGateGelu;

struct RowsQ8P {
    const char* x;      // the gate: rows of [gate | up]
    char* res;
    const char* w;      // nullable
    char* out;
    float* scales;
    int64_t rows;
    int n;              // codes per row
    int nvec;           // 16-byte vectors of them
    int fp8;
    float eps, delta, inv_n;
};

// ---------------------------------------------------------------- maximum and codes

// max(a, |b|, |c|) in which NaN stays NaN.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float y;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float max_abs(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(fabsf(b)));
    return y;
}
// The maximum of a warp's values, none negative (NaN above all): their bits are
// ordered as they are.
__device__ __forceinline__ float warp_max(float v) {
    uint32_t y;
    asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(y) : "r"(__float_as_uint(v)));
    return __uint_as_float(y);
}

constexpr float kStepFloor = 1.1754943508222875e-38f;  // 2^-126
constexpr float kInvCeiling = 8.507059173023462e37f;   // 2^126

// The inverse of a row's step: a number for E4M3, for int8 one and what it leaves over.
struct Inverse {
    float inv, rest;
};
// E4M3 takes an IEEE division (and so does the step): a plain evaluation of the formulas
// gives the same codes.  For int8 an approximate quotient h and the residual 127 - h m,
// which a fused operation rounds only once, give 127 / m = h + (127 - h m) h / 127 to 2^-44
// of itself (to 2^-29 for m above 2^113, where the rest is subnormal: still less than the
// rounding of a product).  m is scaled so that its reciprocal is normal wherever the
// quotient is not above the ceiling; a maximum that is infinite has inv = 0, NaN the
// ceiling.
__device__ __forceinline__ Inverse inverse_of(float most, int fp8) {
    if (fp8) return {fminf(__fdiv_rn(448.0f, most), kInvCeiling), 0.0f};
    float h;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(__fmul_rn(most, 1.0f / 64.0f)));
    h = __fmul_rn(h, 127.0f / 64.0f);
    const float left = __fmaf_rn(-h, fminf(most, 3.4028234663852886e38f), 127.0f);
    const Inverse q = {h, __fmul_rn(__fmul_rn(left, h), 1.0f / 127.0f)};
    return most >= 127.0f * kStepFloor ? q : Inverse{kInvCeiling, 0.0f};
}
__device__ __forceinline__ float step_of(float most, int fp8) {
    const float step = __fdiv_rn(most, fp8 ? 448.0f : 127.0f);
    return step < kStepFloor ? kStepFloor : step;  // (NaN stays)
}

// int8 codes of y * (inv + rest), at most 127 in size: the products rounded to fp32, then
// 1.5 * 2^23 added, which rounds them to the nearest even integer and leaves it in the
// low bits.  A value halfway between two codes (half of the row's maximum is 63.5 steps) is
// common where inputs have few bits, and with the rest its product is that half exactly.
// With 127 / m in fp32 alone the rounding of the quotient chose the code: of all bf16 and
// fp16 numbers that m can be, the half went to the odd code for 52 and 48% when p * inv was
// not rounded, and for 11 and 15% when it was.
constexpr float kMagic = 12582912.0f;
__device__ __forceinline__ uint32_t int8x4(float2 a, float2 b, Inverse q) {
    const float2 inv = splat2(q.inv), rest = splat2(q.rest), magic = splat2(kMagic);
    a = __fadd2_rn(__ffma2_rn(a, inv, __fmul2_rn(a, rest)), magic);
    b = __fadd2_rn(__ffma2_rn(b, inv, __fmul2_rn(b, rest)), magic);
    const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}
__device__ __forceinline__ uint8_t int8x1(float y, Inverse q) {
    return (uint8_t)__float_as_uint(__fadd_rn(__fmaf_rn(y, q.inv, __fmul_rn(y, q.rest)), kMagic));
}

template <int N>
__device__ __forceinline__ typename Fp8Pack<N>::type codes_of(const float2 (&y)[N / 2], Inverse q, int fp8) {
    if (fp8) return quantize_pairs<N>(y, q.inv);
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        w[i] = int8x4(y[2 * i], y[2 * i + 1], q);
    }
    if constexpr (N == 4) {
        return w[0];
    } else {
        return make_uint2(w[0], w[1]);
    }
}
__device__ __forceinline__ uint8_t code_of(float y, Inverse q, int fp8) {
    return fp8 ? quantize1(y, q.inv) : int8x1(y, q);
}

// ---------------------------------------------------------------- rows in registers

template <typename T, int KIND, int V>
__global__ void __launch_bounds__(512) rows_q8_kernel(RowsQ8P p) {
    constexpr int N = vec_elems<T>();
    constexpr int P = N / 2;
    constexpr bool NORM = kIsNorm<KIND>, ADD = KIND == kAddNorm, GATE = kIsGate<KIND>;
    __shared__ float2 red[16];
    const int tid = threadIdx.x, tpr = blockDim.x;
    const int64_t row0 = (int64_t)blockIdx.x * blockDim.y;
    const int64_t row = row0 + threadIdx.y;
    const bool active = row < p.rows;
    const int64_t in_row = (int64_t)p.nvec * (GATE ? 32 : 16);

    if (tid == 0 && threadIdx.y == 0) {
        // this CTA's rows into L2 while the preceding grid drains
        const int64_t r1 = row0 + blockDim.y < p.rows ? row0 + blockDim.y : p.rows;
        prefetch_l2(p.x, row0 * in_row, r1 * in_row);
        if (ADD) prefetch_l2(p.res, row0 * in_row, r1 * in_row);
    }
    pdl_wait();
    pdl_launch_dependents();

    const int64_t rsafe = active ? row : row0;
    const uint4* xr = reinterpret_cast<const uint4*>(p.x + rsafe * in_row);
    uint4* rr = ADD ? reinterpret_cast<uint4*>(p.res + rsafe * in_row) : nullptr;
    const uint4* wv = NORM ? reinterpret_cast<const uint4*>(p.w) : nullptr;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    // xv: the row, or its gate half; yv: the residual, the weight's place is wr, or
    // the up half
    uint4 xv[V], yv[ADD || GATE ? V : 1], wr[NORM ? V : 1];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int idx = tid + i * tpr;
        const bool ok = active && idx < p.nvec;
        xv[i] = ok ? __ldcs(xr + idx) : zero;
        if constexpr (ADD) yv[i] = ok ? __ldcs(rr + idx) : zero;
        if constexpr (GATE) yv[i] = ok ? __ldcs(xr + p.nvec + idx) : zero;
        if constexpr (NORM) wr[i] = ok && wv != nullptr ? __ldg(wv + idx) : zero;
    }

    // the products are held from here to the codes.  The sum of squares runs in the two
    // lanes of a pair, and beyond 32 terms per thread in two pairs alternating by vector
    constexpr bool kSplit = V * N > 32;
    const float2 delta = splat2(p.delta);
    float2 y[V][P];
    float2 ss[2] = {splat2(0.0f), splat2(0.0f)};
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        unpack_pairs<T, N>(xv[i], y[i]);
        if constexpr (ADD) {
            // eager semantics: widen, add in fp32, round once to the dtype
            float2 b[P];
            unpack_pairs<T, N>(yv[i], b);
#pragma unroll
            for (int j = 0; j < P; ++j) y[i][j] = __fadd2_rn(y[i][j], b[j]);
            const uint4 sum = pack_pairs<T, N>(y[i]);
            const int idx = tid + i * tpr;
            if (active && idx < p.nvec) rr[idx] = sum;
            unpack_pairs<T, N>(sum, y[i]);
        }
        if constexpr (NORM) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                ss[kSplit ? (i & 1) : 0] = __ffma2_rn(y[i][j], y[i][j], ss[kSplit ? (i & 1) : 0]);
            }
            if (wv != nullptr) {
                float2 w[P];
                unpack_pairs<T, N>(wr[i], w);
#pragma unroll
                for (int j = 0; j < P; ++j) y[i][j] = __fmul2_rn(y[i][j], __fadd2_rn(w[j], delta));
            }
        }
        if constexpr (GATE) {
            float2 u[P];
            unpack_pairs<T, N>(yv[i], u);
#pragma unroll
            for (int j = 0; j < P; ++j) y[i][j] = gate_fast2<KIND == kGateSilu ? kSilu : kGelu>(y[i][j], u[j]);
        }
#pragma unroll
        for (int j = 0; j < P; ++j) most = max_abs(most, y[i][j].x, y[i][j].y);
    }
    // over the warps that share the row: sum and maximum with one barrier
    float sum = 0.0f;
    if constexpr (NORM) {
        const float2 s2 = kSplit ? __fadd2_rn(ss[0], ss[1]) : ss[0];
        sum = group_sum<32>(__fadd_rn(s2.x, s2.y));
    }
    float top = warp_max(most);
    const int W = tpr >> 5;
    if ((tid & 31) == 0) red[(threadIdx.y * tpr + tid) >> 5] = make_float2(sum, top);
    __syncthreads();
    sum = top = 0.0f;
    for (int k = 0; k < W; ++k) {
        const float2 v = red[threadIdx.y * W + k];
        if constexpr (NORM) sum = __fadd_rn(sum, v.x);
        top = max_abs(top, v.y);
    }
    if (tid == 0 && active) {
        const float step = step_of(top, p.fp8);
        p.scales[row] = NORM ? __fmul_rn(inv_rms(sum, p.inv_n, p.eps), step) : step;
    }
    const Inverse inv = inverse_of(top, p.fp8);
    char* orow = p.out + rsafe * p.n;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int idx = tid + i * tpr;
        if (!(active && idx < p.nvec)) continue;
        auto c = codes_of<N>(y[i], inv, p.fp8);
        reinterpret_cast<decltype(c)*>(orow)[idx] = c;
    }
}

// ---------------------------------------------------------------- any row

// Any length and alignment: one CTA per row, an element per load.  A thread issues the
// loads of 8 elements before it uses one and holds the products of its first 16; a
// longer row's are loaded and computed again for the codes.  8 squares are summed in fp32
// and those sums in fp64 (a thread has up to 32,768 terms, and this GPU is slow in fp64:
// with every square added there, 4096 rows of 4095 bf16 took 93 us, now 41).  Measured too:
// tanh-GELU gate of 4001 rows of 10,239 84 us, 2500 rows of 4095 fp32 quantized 13.5.  An
// element per load is the bound: 2 or 4 bytes where the aligned kernel has 16.
template <typename T, int KIND>
__global__ void __launch_bounds__(512, 2) rows_q8_any_kernel(RowsQ8P p) {
    constexpr bool NORM = kIsNorm<KIND>, ADD = KIND == kAddNorm, GATE = kIsGate<KIND>;
    constexpr int U = 8, HELD = 2;
    __shared__ double red[16];
    __shared__ float red_top[16];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int stride = U * blockDim.x;

    pdl_wait();
    pdl_launch_dependents();

    const T* w = reinterpret_cast<const T*>(p.w);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* x = reinterpret_cast<const T*>(p.x) + row * p.n * (GATE ? 2 : 1);
        T* res = ADD ? reinterpret_cast<T*>(p.res) + row * p.n : nullptr;
        uint8_t* out = reinterpret_cast<uint8_t*>(p.out) + row * p.n;
        double ss = 0.0;
        float top = 0.0f;
        // the products of 8 elements from i0 on, zeros behind the row; `again`: of a row whose
        // sum and maximum are known (and stored)
        auto products = [&](int i0, bool again, float (&y)[U]) {
            T a[U], b[U], c[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * blockDim.x + threadIdx.x;
                const bool ok = i < p.n;
                if (!ADD || !again) a[u] = ok ? __ldg(x + i) : from_f<T>(0.0f);
                if constexpr (ADD) b[u] = ok ? res[i] : from_f<T>(0.0f);
                if constexpr (GATE) b[u] = ok ? __ldg(x + (int64_t)p.n + i) : from_f<T>(0.0f);
                if constexpr (NORM) c[u] = ok && w != nullptr ? __ldg(w + i) : from_f<T>(0.0f);
            }
            float part = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * blockDim.x + threadIdx.x;
                if constexpr (ADD) {
                    if (again) {
                        y[u] = to_f(b[u]);
                    } else {
                        const T sum = from_f<T>(__fadd_rn(to_f(a[u]), to_f(b[u])));
                        if (i < p.n) res[i] = sum;
                        y[u] = to_f(sum);
                    }
                } else {
                    y[u] = to_f(a[u]);
                }
                if constexpr (NORM) {
                    part = __fmaf_rn(y[u], y[u], part);
                    if (w != nullptr) y[u] = __fmul_rn(y[u], __fadd_rn(to_f(c[u]), p.delta));
                }
                if constexpr (GATE) {
                    if (u % 2 == 1) {
                        const float2 v = gate_fast2<KIND == kGateSilu ? kSilu : kGelu>(
                            make_float2(y[u - 1], y[u]), make_float2(to_f(b[u - 1]), to_f(b[u])));
                        y[u - 1] = v.x;
                        y[u] = v.y;
                        if (!again) top = max_abs(top, v.x, v.y);
                    }
                    continue;
                }
                if (i >= p.n) y[u] = 0.0f;
                if (!again) top = max_abs(top, y[u]);
            }
            if (NORM && !again) ss = __dadd_rn(ss, (double)part);
        };
        float held[HELD][U];
#pragma unroll
        for (int h = 0; h < HELD; ++h) {
            if (h * stride < p.n) products(h * stride, false, held[h]);
        }
        for (int i0 = HELD * stride; i0 < p.n; i0 += stride) {
            float y[U];
            products(i0, false, y);
        }
        if constexpr (NORM) ss = group_sum<32>(ss);
        top = warp_max(top);
        if (lane == 0) {
            red[wid] = ss;
            red_top[wid] = top;
        }
        __syncthreads();
        ss = 0.0;
        top = 0.0f;
        for (int k = 0; k < nw; ++k) {
            if constexpr (NORM) ss = __dadd_rn(ss, red[k]);
            top = max_abs(top, red_top[k]);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            const float step = step_of(top, p.fp8);
            p.scales[row] = NORM ? __fmul_rn(inv_rms((float)ss, p.inv_n, p.eps), step) : step;
        }
        const Inverse inv = inverse_of(top, p.fp8);
        auto codes = [&](int i0, const float (&y)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * blockDim.x + threadIdx.x;
                if (i < p.n) out[i] = code_of(y[u], inv, p.fp8);
            }
        };
#pragma unroll
        for (int h = 0; h < HELD; ++h) {
            if (h * stride < p.n) codes(h * stride, held[h]);
        }
        for (int i0 = HELD * stride; i0 < p.n; i0 += stride) {
            float y[U];
            products(i0, true, y);
            codes(i0, y);
        }
    }
}

// ---------------------------------------------------------------- launch

template <typename T, int KIND>
cudaError_t launch_kind(const RowsQ8Args& a, RowsQ8P& p, cudaStream_t s) {
    constexpr int N = vec_elems<T>();
    const int sms = sm_count();
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;

    auto aligned = [](const void* ptr, uintptr_t n) { return (reinterpret_cast<uintptr_t>(ptr) % n) == 0; };
    const int64_t nvec = a.n / N;
    const bool vec = a.n % N == 0 && aligned(a.x, 16) && aligned(a.residual, 16) && aligned(a.w, 16) &&
                     aligned(a.out, N) && nvec <= 16 * 32 * 8;
    if (vec) {
        // Vectors per thread.  With few rows, or few vectors in all, as many warps to a row
        // as it fills (one vector each); else the number with the least cost for a vector: a
        // warp's reduction and divisions count for 0.88 of the work on one vector, spread
        // over V, and lanes behind the row's end are lost.  8 is for rows that 16 warps do not
        // hold with 4: the products of 16-bit types take 81 to 124 registers a thread, so an
        // SM has one such CTA (fp32 quantized 51, two), and the other choice is to read the
        // row again, below.  Measured on GB300 (E4M3): 64 rows of 32,768 bf16 quantized 2.7 us
        // against 12.2, normed 3.7 and 15.3; 1024 of 20,480 normed 23 and 52, SiLU gate 36 and
        // 42.  Between 1 and 4: the norm of 4096 rows of 4096 bf16 takes 11.0 us with V = 4, 12.9 with 2 and 17.0 with 1, of
        // 1024 rows of 2560 (320 vectors, a sixth of the lanes lost with 3 or 4) 2.9 with 2 and
        // 3.4 with 4; the gate of 512 rows of 2048 2.4 with 1 and 3.0 with 4, of 4096 rows of
        // 9728 34.7 with 4, 39.9 with 3 and 47.4 with rows of 16 warps.
        int V = 8, W = 16;
        double least = 1e30;
        const bool few = a.rows < 2 * (int64_t)sms || a.rows * nvec < 1024 * (int64_t)sms;
        for (int v = 1; v <= 4; ++v) {
            const int w = (int)((nvec + 32 * v - 1) / (32 * v));
            if (w > 16) continue;
            const double cost = few ? v : (1.0 + 0.88 / v) * w * v;
            if (cost < least) {
                least = cost;
                V = v;
                W = w;
            }
        }
        const int R = 128 / (32 * W) > 1 ? 128 / (32 * W) : 1;
        const int64_t blocks = (a.rows + R - 1) / R;
        if (blocks <= (int64_t)INT32_MAX) {
            p.nvec = (int)nvec;
            cfg.gridDim = dim3((unsigned)blocks);
            cfg.blockDim = dim3(32 * W, R);
            switch (V) {
                case 1: return cudaLaunchKernelEx(&cfg, rows_q8_kernel<T, KIND, 1>, p);
                case 2: return cudaLaunchKernelEx(&cfg, rows_q8_kernel<T, KIND, 2>, p);
                case 3: return cudaLaunchKernelEx(&cfg, rows_q8_kernel<T, KIND, 3>, p);
                case 4: return cudaLaunchKernelEx(&cfg, rows_q8_kernel<T, KIND, 4>, p);
                default: return cudaLaunchKernelEx(&cfg, rows_q8_kernel<T, KIND, 8>, p);
            }
        }
    }
    // 16 elements per thread, in 2 to 16 warps
    int64_t warps = (a.n + 32 * 16 - 1) / (32 * 16);
    warps = warps < 2 ? 2 : warps > 16 ? 16 : warps;
    const int64_t cap = (int64_t)sms * 32;
    cfg.gridDim = dim3((unsigned)(a.rows < cap ? a.rows : cap));
    cfg.blockDim = dim3((unsigned)(32 * warps));
    return cudaLaunchKernelEx(&cfg, rows_q8_any_kernel<T, KIND>, p);
}

template <typename T>
cudaError_t launch_dt(const RowsQ8Args& a, RowsQ8P& p, cudaStream_t s) {
    if (a.act == kSilu) return launch_kind<T, kGateSilu>(a, p, s);
    if (a.act == kGelu) return launch_kind<T, kGateGelu>(a, p, s);
    if (a.residual != nullptr) return launch_kind<T, kAddNorm>(a, p, s);
    return a.norm ? launch_kind<T, kNorm>(a, p, s) : launch_kind<T, kQuant>(a, p, s);
}

}  // namespace

cudaError_t launch_rows_q8(const RowsQ8Args& a, cudaStream_t s) {
    RowsQ8P p;
    p.x = static_cast<const char*>(a.x);
    p.res = static_cast<char*>(a.residual);
    p.w = static_cast<const char*>(a.w);
    p.out = static_cast<char*>(a.out);
    p.scales = a.scales;
    p.rows = a.rows;
    p.n = (int)a.n;
    p.nvec = 0;
    p.fp8 = a.out_dt == kFP8;
    p.eps = a.eps;
    p.delta = (float)a.weight_offset;
    p.inv_n = 1.0f / (float)a.n;
    switch (a.dt) {
        case kF32: return launch_dt<float>(a, p, s);
        case kF16: return launch_dt<__half>(a, p, s);
        default: return launch_dt<__nv_bfloat16>(a, p, s);
    }
}

}  // namespace edge
