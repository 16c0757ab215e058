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

// ---------------------------------------------------------------- any size

// Rows and addresses of any alignment, which no tensor map takes.  A tile is 64 tokens
// by 64 channels, 64 terms at a time.  The bytes come as aligned vectors, are shifted
// into place with the neighbouring lane's, turned to fp16 once (exact for both types)
// and laid into shared memory, from where eight warps of 32 x 16 outputs multiply them.
// Few tiles are cut along the sum over the CTAs of a cluster.  int8 sums join an int32
// every 1024 terms, as in matmul_q8_tc.cu.
//
// The shifting and laying out bounds it, several times the products' instructions.
// Measured on GB300 (E4M3, int8): one token, 2560 channels, 9725 terms 22 and 25 us, 64
// tokens 32 and 36, 512 tokens 171 and 196 (149 and 130 TFLOP/s).  Byte loads and an uncut
// sum took 463 and 671 for the first two, and 366 for 1201 x 5120 x 2045 (now 161 and 186).
constexpr int kTile = 64;       // tokens and channels of a CTA
constexpr int kStepAny = 64;    // terms of the sum in one step
constexpr int kRowAny = 144;    // bytes of a row in shared memory, of fp16: no bank conflicts
constexpr int kThreadsAny = 256;

// Four codes to fp16, in which both types' values are exact.
template <bool INT8>
__device__ __forceinline__ void to_half4(uint32_t v, uint32_t& lo, uint32_t& hi) {
    if constexpr (INT8) {
        widen4(v, lo, hi);
    } else {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)v));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(v >> 16)));
    }
}
template <bool INT8>
__device__ __forceinline__ void put_half16(uint4 v, uint8_t* dst) {
    uint32_t h[8];
    to_half4<INT8>(v.x, h[0], h[1]);
    to_half4<INT8>(v.y, h[2], h[3]);
    to_half4<INT8>(v.z, h[4], h[5]);
    to_half4<INT8>(v.w, h[6], h[7]);
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(h[0], h[1], h[2], h[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(h[4], h[5], h[6], h[7]);
}
// Four 8 x 8 matrices of fp16: fragments of 16 rows and terms (the tokens), or of 16
// channels in two operands of 8.
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], const uint8_t* p) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(p);
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

__device__ __forceinline__ const char* round_up(const char* p) { return p + (-reinterpret_cast<uintptr_t>(p) & 15); }
__device__ __forceinline__ const char* round_down(const char* p) { return p - (reinterpret_cast<uintptr_t>(p) & 15); }

// 16 of every 64 bytes of a row that starts at any address, loaded as the aligned
// vectors in which they begin.  Four neighbouring lanes have a row.
struct RowBytes {
    const char* at;      // this lane's first vector
    int off;             // bytes of it before the lane's own
    int lo;              // first step whose vector is inside the operand
    unsigned n;          // steps from there on whose vector is needed and inside
    bool edge;           // the operand begins or ends inside vectors of this row

    // Row r of the operand from base to end, for steps up to s1.
    __device__ RowBytes(const char* base, const char* end, int64_t r, int64_t rows, int k, int s1, int lane) {
        const char* src = base + (r < rows ? r : 0) * k;
        const int col = 16 * (lane & 3);
        off = (int)(reinterpret_cast<uintptr_t>(src) & 15);
        at = src - off + col;
        lo = at < base ? 1 : 0;
        // vectors that begin in the row, of step s1 the first alone
        int64_t hi = (k - col + off + kStepAny - 1) / kStepAny;
        hi = min(hi, (int64_t)(col == 0 ? s1 + 1 : s1));
        const int64_t room = end - at - 16;
        hi = min(hi, room < 0 ? 0 : room / kStepAny + 1);
        n = r < rows && hi > lo ? (unsigned)(hi - lo) : 0u;
        edge = r < rows && (src < round_up(base) || src + k > round_down(end));
    }
    __device__ __forceinline__ uint4 load(int s) const {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if ((unsigned)(s - lo) < n) v = __ldg(reinterpret_cast<const uint4*>(at + s * kStepAny));
        return v;
    }
    // The lane's 16 bytes of a step from its vector and the next one: the next lane's, or of
    // the row's last lane the first lane's of the step after.
    __device__ __forceinline__ uint4 bytes(uint4 now, uint4 then, int lane) const {
        const bool head = (lane & 3) == 0;
        const int from = (lane & 28) | ((lane + 1) & 3);
        uint32_t w[8] = {now.x, now.y, now.z, now.w};
        w[4] = __shfl_sync(0xffffffffu, head ? then.x : now.x, from);
        w[5] = __shfl_sync(0xffffffffu, head ? then.y : now.y, from);
        w[6] = __shfl_sync(0xffffffffu, head ? then.z : now.z, from);
        w[7] = __shfl_sync(0xffffffffu, head ? then.w : now.w, from);
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (off & 3));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // Of those bytes (k0.. of the row) the ones in vectors that the operand begins or ends inside.
    template <bool INT8>
    __device__ __forceinline__ void patch(int k0, int k, const char* base, const char* end, uint8_t* dst, int s) const {
        const char* p = at + off + s * kStepAny;
        const int count = min(16, k - k0);
        if (p >= round_up(base) && p + count <= round_down(end)) return;
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
            if (p + i >= round_up(base) && p + i < round_down(end)) continue;
            uint32_t lo4, hi4;
            to_half4<INT8>(__ldg(reinterpret_cast<const uint8_t*>(p + i)), lo4, hi4);
            reinterpret_cast<uint16_t*>(dst)[i] = (uint16_t)lo4;
        }
    }
};
// The first `left` of 16 bytes, zeros for the others.
__device__ __forceinline__ uint4 first_bytes(uint4 v, int left) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = left - 4 * i;
        w[i] = n >= 4 ? w[i] : n <= 0 ? 0u : w[i] & ((1u << (8 * n)) - 1u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool INT8>
__global__ void __launch_bounds__(kThreadsAny, 3) matmul_any_kernel(MatmulP p, int split) {
    // two steps of both operands, then the sums [token][channel] of a part
    __shared__ __align__(16) uint8_t room[4 * kTile * kRowAny];
    static_assert(sizeof(room) >= kTile * kTile * 4, "a part of a cut tile does not fit");
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int tiles_n = (p.n + kTile - 1) / kTile, tile = (int)blockIdx.x / split, rank = (int)blockIdx.x % split;
    const int t0 = tile / tiles_n * kTile, n0 = tile % tiles_n * kTile;
    const int steps = (p.k + kStepAny - 1) / kStepAny, s0 = steps * rank / split, s1 = steps * (rank + 1) / split;
    const char *a_end = p.a + (int64_t)p.tokens * p.k, *w_end = p.w + (int64_t)p.n * p.k;
    const int row = tid >> 2;  // of both operands
    const RowBytes ar(p.a, a_end, t0 + row, p.tokens, p.k, s1, lane), wr(p.w, w_end, n0 + row, p.n, p.k, s1, lane);
    const bool a_warp = t0 + wid * 8 < p.tokens;  // of this warp's eight rows of tokens there is one
    if (tid < kTile && n0 + tid < p.n) {
        // this CTA's weights into L2 while the preceding grid drains
        const int64_t at = (int64_t)(n0 + tid) * p.k;
        prefetch_l2(p.w, at + s0 * kStepAny, at + min(s1 * kStepAny, p.k));
    }
    pdl_wait();
    pdl_launch_dependents();

    float acc[2][2][4];
    int whole[2][2][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        (&acc[0][0][0])[i] = 0.0f;
        (&whole[0][0][0])[i] = 0;
    }
    const int tw = (wid >> 2) * 32, nw = (wid & 3) * 16, g = lane >> 2;
    const int most = p.tokens - t0 - tw;  // tokens of this warp
    const int a_at = (tw + (lane & 15)) * kRowAny + (lane >> 4) * 16;
    const int w_at = (kTile + nw + (lane & 7) + (lane >> 4) * 8) * kRowAny + ((lane >> 3) & 1) * 16;
    constexpr int DEPTH = 2;  // steps in registers (with 4 the E4M3 kernel took 8 to 15% longer)
    uint4 va[DEPTH], vw[DEPTH];
    auto step = [&](int s, uint4& a, uint4& w, const uint4& a_then, const uint4& w_then) {
        uint8_t* at = room + (s & 1) * 2 * kTile * kRowAny;
        uint8_t* wt = at + kTile * kRowAny;
        const int to = row * kRowAny + 32 * (lane & 3), k0 = s * kStepAny + 16 * (lane & 3);
        const bool last = (s + 1) * kStepAny > p.k;
        if (a_warp) {
            uint4 x = ar.bytes(a, a_then, lane);
            if (last) x = first_bytes(x, p.k - k0);
            put_half16<INT8>(x, at + to);
            if (ar.edge) ar.patch<INT8>(k0, p.k, p.a, a_end, at + to, s);
        }
        uint4 x = wr.bytes(w, w_then, lane);
        if (last) x = first_bytes(x, p.k - k0);
        put_half16<INT8>(x, wt + to);
        if (wr.edge) wr.patch<INT8>(k0, p.k, p.w, w_end, wt + to, s);
        __syncthreads();  // (the buffer written next was last read before this barrier)
        a = ar.load(s + DEPTH);
        w = wr.load(s + DEPTH);
#pragma unroll
        for (int k = 0; k < kStepAny; k += 16) {
            if (most <= 0) break;
            uint32_t b[4];
            load_matrices(b, at + w_at + 2 * k);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (16 * i >= most) break;
                uint32_t x[4];
                load_matrices(x, at + a_at + i * 16 * kRowAny + 2 * k);
                mma_f16(acc[i][0], x, b[0], b[1]);
                mma_f16(acc[i][1], x, b[2], b[3]);
            }
        }
        if (INT8 && (s - s0) % (1024 / kStepAny) == 1024 / kStepAny - 1) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                (&whole[0][0][0])[i] += __float2int_rn((&acc[0][0][0])[i]);
                (&acc[0][0][0])[i] = 0.0f;
            }
        }
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
        va[i] = ar.load(s0 + i);
        vw[i] = wr.load(s0 + i);
    }
    for (int s = s0; s < s1; s += DEPTH) {
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            if (s + i < s1) step(s + i, va[i], vw[i], va[(i + 1) % DEPTH], vw[(i + 1) % DEPTH]);
        }
    }
    auto sum = [&](int i, int j, int e) {
        return INT8 ? (uint32_t)(whole[i][j][e] + __float2int_rn(acc[i][j][e])) : __float_as_uint(acc[i][j][e]);
    };
    auto store = [&](int t, int n, uint32_t x) {
        const float y = INT8 ? __int2float_rn((int)x) : __uint_as_float(x);
        const float bias = p.bias != nullptr ? load_out(p.bias, n, p.out_dt) : 0.0f;
        store_out(p.out, (int64_t)t * p.n + n, scaled(y, __ldg(p.sa + t), __ldg(p.sw + n), bias), p.out_dt);
    };
    uint32_t* part = reinterpret_cast<uint32_t*>(room);
    if (split > 1) __syncthreads();  // every warp has read the last step
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = tw + 16 * i + g + 8 * (e >> 1), n = nw + 8 * j + (lane & 3) * 2 + (e & 1);
                if (split > 1) {
                    part[t * kTile + n] = sum(i, j, e);
                } else if (t0 + t < p.tokens && n0 + n < p.n) {
                    store(t0 + t, n0 + n, sum(i, j, e));
                }
            }
        }
    }
    if (split > 1) {
        cluster_sync();
        // this CTA's share of the outputs, the parts added in rank order
        const int outs = min(kTile, p.tokens - t0) * kTile;
        for (int i = rank * kThreadsAny + tid; i < outs; i += split * kThreadsAny) {
            const uint32_t at = (uint32_t)__cvta_generic_to_shared(part + i);
            uint32_t x[8], total = 0u;
#pragma unroll
            for (int r = 0; r < 8; ++r) x[r] = r < split ? peer_word(peer_addr(at, r)) : 0u;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                if (r >= split) break;
                total = INT8 ? total + x[r] : __float_as_uint(__fadd_rn(__uint_as_float(total), __uint_as_float(x[r])));
            }
            if (n0 + i % kTile < p.n) store(t0 + i / kTile, n0 + i % kTile, total);
        }
        cluster_sync();  // peers read this CTA's shared memory until here
    }
}

template <bool INT8>
cudaError_t launch_any(const MatmulP& p, cudaLaunchConfig_t cfg) {
    const int64_t tiles = (int64_t)((p.tokens + kTile - 1) / kTile) * ((p.n + kTile - 1) / kTile);
    if (tiles > INT32_MAX / 8) return cudaErrorInvalidConfiguration;
    const void* fn = reinterpret_cast<const void*>(matmul_any_kernel<INT8>);
    cfg.blockDim = dim3(kThreadsAny);
    // The cut with the least time in units of a step: the rounds of CTAs times the steps of a
    // part, 4 for its beginning and end, and 3 for the join.
    const int steps = (p.k + kStepAny - 1) / kStepAny;
    int split = 1;
    int64_t best = INT64_MAX;
    for (int s = 1; s <= 8 && (s == 1 || s * 4 <= steps); ++s) {
        const int64_t slots = resident_clusters(fn, cfg, s);
        if (s > 1 && slots < 1) continue;
        const int64_t rounds = slots < 1 ? 1 : (tiles + slots - 1) / slots;
        const int64_t cost = rounds * ((steps + s - 1) / s + 4 + (s > 1 ? 3 : 0));
        if (cost < best) {
            best = cost;
            split = s;
        }
    }
    cfg.gridDim = dim3((unsigned)(tiles * split));
    if (split > 1) {
        cfg.attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        cfg.attrs[cfg.numAttrs].val.clusterDim.x = (unsigned)split;
        cfg.attrs[cfg.numAttrs].val.clusterDim.y = 1;
        cfg.attrs[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, matmul_any_kernel<INT8>, p, split);
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
