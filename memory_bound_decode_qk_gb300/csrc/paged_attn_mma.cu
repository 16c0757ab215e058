// paged_attn_mma.cu -- paged attention of 16-bit heads with few query rows per
// key head (sm_103a).
//
// A decode step reads every key and value once and does 4 G flops for each of
// their elements (G query heads per key head), so it is bound by HBM.  The
// matrix products run on the warp-level tensor instructions (m16n8k16): 16 rows
// are the smallest tile they have, and a decode step seldom fills even those,
// so the wide tcgen05 tiles would have nothing to gain here.
//
// attn_few_kernel (16 rows): a worker is one warp, with a piece of the line and a
// ring of cp.async stages of its own, so no warp ever waits for another.  The
// loads run ahead over the ends of units: the walk of the loads is a copy of
// the walk of the products.  (Four warps that split each tile of one piece and
// joined at the ends of units reached 2.7 TB/s on a ragged batch; this form
// has no such joins.)
// Measured on GB300: 64 sequences of 64 to 8192 keys, 32/8 heads of 128, 558 MB
// in 98 us (5.7 TB/s, 84% of the copy bandwidth); three sequences of 30 to 131
// thousand keys, 24/4 heads of 256, 967 MB in 164 us (5.9 TB/s); blocks of 16
// tokens, 32/32 heads of 128, 248 MB in 55 us (4.5 TB/s).  Up to 8 rows the
// weights keep two 16-bit parts, the second in the rows that are free: 0.5% and
// 1 to 2% of the time of the first two, and their error against 64 bits falls
// from 1.35 times that of the output's rounding alone to 1.0.  16 keys a stage
// and three stages hold 96 KB of copies in flight per CTA of 128-channel heads,
// two CTAs to an SM.
// attn_more_kernel (64 rows): a warp has 16 rows each and the CTA shares the
// tiles, so that a key is read once for 64 rows.  For chunks over pages that TMA
// boxes do not tile; the products run at about 160 TFLOP/s, which bounds it (two
// chunks of 1024 tokens over 16,384 keys in pages of 13 tokens, 32/8 heads of 128:
// 3.05 ms, where pages of 16 take 0.41 with tcgen05).
//
// Both keep the running maximum lazily: the accumulators are rescaled only when
// a row's maximum grew by more than 2^8, which leaves the weights at most 256
// and the result unchanged (numerator and sum carry the same factor).
#include "paged_common.cuh"

namespace edge {
namespace {

// ---------------------------------------------------------------- instructions

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

// 16 bytes from global to shared memory, asynchronously; zeros if !ok.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (std::is_same<T, __half>::value) {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    } else {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    }
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (std::is_same<T, __half>::value) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    } else {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
    }
}
// What rounding a and b to the pair `w` left over, rounded in turn.  (A weight
// that is NaN has NaN here as well.)
template <typename T>
__device__ __forceinline__ uint32_t remainder2(float a, float b, uint32_t w) {
    const float2 r = unpack2<T>(w);
    return pack2<T>(a - r.x, b - r.y);
}

// Whether one of the two values in a word is infinite or NaN.
template <typename T>
__device__ __forceinline__ bool unbounded(uint32_t w) {
    constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7C007C00u : 0x7F807F80u;
    return __vcmpeq2(w & e, e) != 0;
}

// Byte offset of 16-byte chunk c of row r in a tile of DP-element rows; the
// chunk index is xored with the row, so the 8 rows of an ldmatrix lie in
// different banks.
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return (uint32_t)(r * (DP / 8) + (c ^ (r & 7))) * 16u;
}

// ---------------------------------------------------------------- softmax state of two rows

// A thread of a 16-row tile holds columns of rows lane / 4 and lane / 4 + 8.
struct RowState {
    float ref[2], sum[2];  // the reference maximum (base 2) and the sum of this thread's columns
};

constexpr float kLazy = 8.0f;

// Scores s (scaled, base 2, masked to -inf) of NT column tiles -> weights, in
// place; o is rescaled where a row's reference moves.
template <int NT, int NO>
__device__ __forceinline__ void soft_tile(float (&s)[NT][4], float (&o)[NO][4], RowState& st) {
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        top[0] = fmaxf(top[0], fmaxf(s[n][0], s[n][1]));
        top[1] = fmaxf(top[1], fmaxf(s[n][2], s[n][3]));
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
    }
    const bool grow = top[0] > st.ref[0] + kLazy || top[1] > st.ref[1] + kLazy;
    if (__any_sync(0xffffffffu, grow)) {
        float keep[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float next = fmaxf(st.ref[r], top[r]);
            keep[r] = next == -INFINITY ? 1.0f : ex2(st.ref[r] - next);
            st.ref[r] = next;
            st.sum[r] *= keep[r];
        }
#pragma unroll
        for (int n = 0; n < NO; ++n) {
            o[n][0] *= keep[0];
            o[n][1] *= keep[0];
            o[n][2] *= keep[1];
            o[n][3] *= keep[1];
        }
    }
    const float r0 = st.ref[0] == -INFINITY ? 0.0f : st.ref[0];
    const float r1 = st.ref[1] == -INFINITY ? 0.0f : st.ref[1];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        s[n][0] = ex2(s[n][0] - r0);
        s[n][1] = ex2(s[n][1] - r0);
        s[n][2] = ex2(s[n][2] - r1);
        s[n][3] = ex2(s[n][3] - r1);
        st.sum[0] += s[n][0] + s[n][1];
        st.sum[1] += s[n][2] + s[n][3];
    }
}

// Weights times values for a tile that holds infinities or NaN where some rows
// are masked: one key at a time, skipping those that a row does not see (their
// weights are set to -1), so a masked value leaves no trace, and one whose weight
// underflowed to zero leaves 0 times it.  ps: this warp's [16][KN] floats.
template <typename T, int DP, int KN, int NT, int NO>
__device__ void careful_values(const float (&s)[NT][4], float (&o)[NO][4], const char* vt, float* ps,
                               int lane) {
    const int g = lane >> 2, q = (lane & 3) * 2;
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        ps[g * KN + n * 8 + q] = s[n][0];
        ps[g * KN + n * 8 + q + 1] = s[n][1];
        ps[(g + 8) * KN + n * 8 + q] = s[n][2];
        ps[(g + 8) * KN + n * 8 + q + 1] = s[n][3];
    }
    __syncwarp();
    for (int j = 0; j < KN; ++j) {
        const float w0 = ps[g * KN + j], w1 = ps[(g + 8) * KN + j];
#pragma unroll
        for (int n = 0; n < NO; ++n) {
            const T* v = reinterpret_cast<const T*>(vt + chunk_at<DP>(j, n)) + q;
            const float a = to_f(v[0]), b = to_f(v[1]);
            if (!(w0 < 0.0f)) {
                o[n][0] = fmaf(w0, a, o[n][0]);
                o[n][1] = fmaf(w0, b, o[n][1]);
            }
            if (!(w1 < 0.0f)) {
                o[n][2] = fmaf(w1, a, o[n][2]);
                o[n][3] = fmaf(w1, b, o[n][3]);
            }
        }
    }
    __syncwarp();
}

// Two neighbouring outputs of a row.
template <typename T>
__device__ __forceinline__ void store_two(const AttnP& p, int64_t e, float a, float b) {
    if (p.out_fp8) {
        store_one<T>(p, e, a);
        store_one<T>(p, e + 1, b);
    } else {
        reinterpret_cast<T*>(p.out)[e] = from_f<T>(a);
        reinterpret_cast<T*>(p.out)[e + 1] = from_f<T>(b);
    }
}

// Writes a 16-row tile (unnormalized o, reference, full row sums) as partials or
// outputs.  row0: the tile's first row in the unit, nrows: rows of the unit.
template <typename T, int M, int NO>
__device__ __forceinline__ void write_tile(const AttnP& p, const Walk& w, const float (&o)[NO][4],
                                           const float (&ref)[2], const float (&sum)[2], int row0,
                                           int nrows, int lane) {
    const int slot = walk_slot(w);
    float* part = slot < 0 ? nullptr : part_of<M>(p, w.piece, slot);
    const int q = (lane & 3) * 2;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = row0 + (lane >> 2) + 8 * r;
        if (row >= nrows) continue;
        if (part != nullptr) {
#pragma unroll
            for (int n = 0; n < NO; ++n) {
                if (n * 8 < p.D) {
                    *reinterpret_cast<float2*>(part + (int64_t)row * p.D + n * 8 + q) =
                        make_float2(o[n][2 * r], o[n][2 * r + 1]);
                }
            }
            if (q == 0) {
                part[(int64_t)M * p.D + row] = ref[r];
                part[(int64_t)M * p.D + M + row] = sum[r];
            }
        } else {
            const int64_t orow = out_row(p, w.s, w.h, w.rt * M + row);
            const float inv = sum[r] == 0.0f ? 0.0f : 1.0f / sum[r];
#pragma unroll
            for (int n = 0; n < NO; ++n) {
                if (n * 8 < p.D) {
                    store_two<T>(p, orow * p.D + n * 8 + q, o[n][2 * r] * inv, o[n][2 * r + 1] * inv);
                }
            }
            if (q == 0 && p.lse != nullptr) p.lse[orow] = row_lse(ref[r], sum[r]);
        }
    }
}

// ---------------------------------------------------------------- few rows

constexpr int kFewWarps = 4;
constexpr int kFewKeys = 16;  // keys of a warp's stage
constexpr int kFewStages = 3;
constexpr int kFewUC = 2;

// Wide heads keep the queries in shared memory: beside 16 rows of output
// accumulators the registers do not hold them.
template <int DP>
constexpr size_t few_smem() {
    return (size_t)kFewWarps * (kFewStages * 2 * kFewKeys * DP * 2 + (DP > 128 ? 16 * DP * 2 : 0));
}

template <typename T, int DP>
__global__ void __launch_bounds__(kFewWarps * 32, DP <= 128 ? 2 : 1) attn_few_kernel(AttnP p) {
    constexpr int M = 16, KT = kFewKeys, ST = kFewStages, UC = kFewUC;
    constexpr int KS = DP / 16, NO = DP / 8, NT = KT / 8;
    constexpr bool kQS = DP > 128;
    constexpr int kTile = KT * DP * 2;  // bytes of a K (or V) stage
    extern __shared__ __align__(128) char smem[];
    __shared__ WalkSmem<kFewWarps> wsm;
    __shared__ uint32_t dead_of[kFewWarps][ST];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    char* ring = smem + wid * ST * 2 * kTile;
    char* qt = smem + kFewWarps * ST * 2 * kTile + wid * 16 * DP * 2;

    pdl_wait();
    pdl_launch_dependents();
    if (lane == 0) clear_desc(p, blockIdx.x + gridDim.x * wid);

    Walk w;
    if (!walk_begin<M, KT, UC, kFewWarps>(p, w, wsm, kFewWarps * 32, wid)) return;

    // the loads' own walk: `off` is the element offset of this lane's key in
    // the next stage to load (-1: a key no row sees), looked up one stage ahead
    Walk lw = w;
    int lt = 0;
    bool live = true;
    int64_t off = -1;
    auto look = [&] {
        const int j = (lw.k0 + lw.off + lt) * KT + lane;
        off = -1;
        if (lane < KT && j >= lw.keys.lo && j < lw.keys.hi) {
            const int64_t slot = key_slot(p, lw.b, j);
            if (slot >= 0) off = (slot * p.hk + lw.h) * p.D;
        }
    };
    look();
    auto issue = [&](int st) {
        if (live) {
            const uint32_t dead = __ballot_sync(0xffffffffu, off < 0);
            if (lane == 0) dead_of[wid][st] = dead;
            const uint32_t kb = smem_addr(ring + st * 2 * kTile), vb = kb + kTile;
#pragma unroll
            for (int i = 0; i < KT * (DP / 8) / 32; ++i) {
                const int e = lane + 32 * i;
                const int r = e / (DP / 8), c = e % (DP / 8);
                const int64_t o = __shfl_sync(0xffffffffu, off, r);
                const bool ok = o >= 0 && c * 8 < p.D;
                const int64_t at = ok ? (o + c * 8) * 2 : 0;
                const uint32_t to = chunk_at<DP>(r, c);
                cp_async16(kb + to, p.k + at, ok);
                cp_async16(vb + to, p.v + at, ok);
            }
            if (++lt == lw.cnt) {
                lt = 0;
                live = walk_next<M, KT, UC>(p, lw);
                if (live) {
                    // the next unit's queries into L1, a line per lane
                    const int rows = min(lw.s.n * p.G - lw.rt * M, M);
                    const int lines = (p.D * 2 + 127) / 128;
                    for (int i = lane; i < rows * lines; i += 32) {
                        const int r = i / lines;
                        prefetch_l1_line(p.q + out_row(p, lw.s, lw.h, lw.rt * M + r) * p.D * 2 + (i - r * lines) * 128);
                    }
                }
            }
            if (live) look();
        }
        cp_async_commit();
    };
    // wide heads: a unit's queries into shared memory
    auto queries = [&] {
        const int rows = w.s.n * p.G - w.rt * M;
#pragma unroll 4
        for (int i = lane; i < 16 * (DP / 8); i += 32) {
            const int r = i / (DP / 8), c = i % (DP / 8);
            const bool ok = r < rows && c * 8 < p.D;
            const int64_t e = ok ? out_row(p, w.s, w.h, w.rt * M + r) * p.D + c * 8 : 0;
            cp_async16(smem_addr(qt) + chunk_at<DP>(r, c), p.q + e * 2, ok);
        }
        cp_async_commit();
    };
    if constexpr (kQS) queries();
    for (int i = 0; i < ST - 1; ++i) issue(i);

    int stage = 0;
    bool again = false;
    do {
        const int rows = w.s.n * p.G - w.rt * M;  // rows of the unit (may exceed 16)
        uint32_t qf[kQS ? 1 : KS][4];
        if constexpr (kQS) {
            if (again) {
                // behind the stages of this unit that are on their way
                __syncwarp();
                queries();
                cp_async_wait<0>();
                __syncwarp();
            }
            again = true;
        } else {
            // queries straight into the fragments of the first product
            const int g = lane >> 2, q = (lane & 3) * 2;
            const T* qp[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = g + 8 * r;
                qp[r] = row < rows ? reinterpret_cast<const T*>(p.q) + out_row(p, w.s, w.h, w.rt * M + row) * p.D
                                   : nullptr;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = k * 16 + (i >> 1) * 8 + q;
                    const T* x = qp[i & 1];
                    qf[k][i] = x != nullptr && d < p.D ? __ldg(reinterpret_cast<const uint32_t*>(x + d)) : 0u;
                }
            }
        }
        // with up to 8 rows, rows 8 to 15 of the products are free
        const bool half = rows <= 8;
        float o[NO][4];
        RowState st;
#pragma unroll
        for (int n = 0; n < NO; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;
        }
        int at[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            st.ref[r] = -INFINITY;
            st.sum[r] = 0.0f;
            at[r] = w.s.L - w.s.n + (int)fast_div((uint32_t)(w.rt * M + (lane >> 2) + 8 * r), p.gdiv);
        }
        for (int t = 0; t < w.cnt; ++t) {
            cp_async_wait<ST - 2>();
            __syncwarp();
            issue(stage == 0 ? ST - 1 : stage - 1);
            char* kt = ring + stage * 2 * kTile;
            const char* vt = kt + kTile;
            const uint32_t ka = smem_addr(kt), va = smem_addr(vt), qa = smem_addr(qt);
            const uint32_t dead = dead_of[wid][stage] & ((1u << KT) - 1u);
            const int j0 = (w.k0 + w.off + t) * KT;
            stage = stage + 1 == ST ? 0 : stage + 1;

            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][i] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t a[4];
                if constexpr (kQS) {
                    ldsm4(qa + chunk_at<DP>(lane & 15, 2 * k + (lane >> 4)), a);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = qf[k][i];
                }
                // keys 0-7 and 8-15 by channel halves of the step
                uint32_t b[4];
                const int r = (lane & 7) + ((lane >> 4) << 3);
                ldsm4(ka + chunk_at<DP>(r, 2 * k + ((lane >> 3) & 1)), b);
                mma16816<T>(s[0], a, b[0], b[1]);
                mma16816<T>(s[1], a, b[2], b[3]);
            }
            const bool part = j0 < w.keys.flo || j0 + KT > w.keys.fhi;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[n][i] *= p.scale_log2;
                    if (part || dead) {
                        const int c = n * 8 + (lane & 3) * 2 + (i & 1);
                        if (((dead >> c) & 1u) || !sees(p, at[i >> 1], j0 + c)) s[n][i] = -INFINITY;
                    }
                }
            }
            if (half) {
                // row r + 8 is row r again, for the remainders of its weights
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    s[n][2] = s[n][0];
                    s[n][3] = s[n][1];
                }
            }
            soft_tile<NT, NO>(s, o, st);
            // several tokens: values that only some rows see
            bool odd = false;
            if (part && w.s.n > 1) {
                for (int i = lane; i < kTile / 16; i += 32) {
                    const uint4 x = reinterpret_cast<const uint4*>(vt)[i];
                    odd |= unbounded<T>(x.x) || unbounded<T>(x.y) || unbounded<T>(x.z) || unbounded<T>(x.w);
                }
                odd = __any_sync(0xffffffffu, odd);
            }
            if (odd) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = n * 8 + (lane & 3) * 2 + (i & 1);
                        if ((half && i > 1) || ((dead >> c) & 1u) || !sees(p, at[i >> 1], j0 + c)) s[n][i] = -1.0f;
                    }
                }
                careful_values<T, DP, KT, NT, NO>(s, o, vt, reinterpret_cast<float*>(kt), lane);  // the keys are done with
                continue;
            }
            uint32_t a[4] = {pack2<T>(s[0][0], s[0][1]), pack2<T>(s[0][2], s[0][3]),
                             pack2<T>(s[1][0], s[1][1]), pack2<T>(s[1][2], s[1][3])};
            if (half) {
                // what the rounding of the weights left over, in the free rows: it
                // does not show in the output then (relative 2^-16 with bf16, 2^-22
                // with fp16).  With more rows it would take products of its own
                // (14% of the time of long sequences of 256 channels) and outputs
                // of its own: in common ones an infinite value would meet
                // remainders of either sign.
                a[1] = remainder2<T>(s[0][2], s[0][3], a[1]);
                a[3] = remainder2<T>(s[1][2], s[1][3], a[3]);
            }
#pragma unroll
            for (int n = 0; n < NO; n += 2) {
                uint32_t b[4];
                ldsm4t(va + chunk_at<DP>(lane & 15, n + (lane >> 4)), b);
                mma16816<T>(o[n], a, b[0], b[1]);
                mma16816<T>(o[n + 1], a, b[2], b[3]);
            }
        }
        if (half) {
            // an infinity is one in the first part; the second has either sign of
            // it, or NaN
#pragma unroll
            for (int n = 0; n < NO; ++n) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (fabsf(o[n][i]) < INFINITY) o[n][i] += o[n][i + 2];
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            st.sum[r] += __shfl_xor_sync(0xffffffffu, st.sum[r], 1);
            st.sum[r] += __shfl_xor_sync(0xffffffffu, st.sum[r], 2);
        }
        write_tile<T, M, NO>(p, w, o, st.ref, st.sum, 0, rows < M ? rows : M, lane);
        if (lane == 0 && walk_slot(w) == 1) write_desc(p, w);
    } while (walk_next<M, KT, UC>(p, w));
    cp_async_wait<0>();
}

// ---------------------------------------------------------------- more rows

constexpr int kMoreKeys = 64;

constexpr int kMoreStages = 2;
constexpr int kMoreUC = 1;

template <int DP>
constexpr size_t more_smem() {
    return (size_t)64 * DP * 2 + (size_t)kMoreStages * 2 * kMoreKeys * DP * 2;
}

template <typename T, int DP>
__global__ void __launch_bounds__(128, DP <= 128 ? 2 : 1) attn_more_kernel(AttnP p) {
    constexpr int M = 64, KT = kMoreKeys, ST = kMoreStages;
    constexpr int KS = DP / 16, NO = DP / 8, NT = KT / 8;
    constexpr int kTile = KT * DP * 2;
    extern __shared__ __align__(128) char smem[];
    __shared__ WalkSmem<1> wsm;
    __shared__ uint32_t dead_of[ST][KT / 32];
    __shared__ int64_t off_of[KT];
    __shared__ float ps[4][16 * 16];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    char* qt = smem;
    char* ring = smem + M * DP * 2;

    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) clear_desc(p, blockIdx.x);

    Walk w;
    if (!walk_begin<M, KT, kMoreUC, 1>(p, w, wsm, 128, 0)) return;
    do {
        const int rows = w.s.n * p.G - w.rt * M;
        __syncthreads();  // the unit before is done with the queries and the ring
        for (int i = tid; i < M * (DP / 8); i += 128) {
            const int r = i / (DP / 8), c = i % (DP / 8);
            const bool ok = r < rows && c * 8 < p.D;
            const int64_t e = ok ? out_row(p, w.s, w.h, w.rt * M + r) * p.D + c * 8 : 0;
            cp_async16(smem_addr(qt) + chunk_at<DP>(r, c), p.q + e * 2, ok);
        }
        const int t0 = w.k0 + w.off;
        auto issue = [&](int t, int st) {  // every thread of the block
            if (t < w.cnt) {
                if (tid < KT) {
                    const int j = (t0 + t) * KT + tid;
                    int64_t off = -1;
                    if (j >= w.keys.lo && j < w.keys.hi) {
                        const int64_t slot = key_slot(p, w.b, j);
                        if (slot >= 0) off = (slot * p.hk + w.h) * p.D;
                    }
                    off_of[tid] = off;
                    const uint32_t dead = __ballot_sync(0xffffffffu, off < 0);
                    if (lane == 0) dead_of[st][wid] = dead;
                }
                __syncthreads();
                const uint32_t kb = smem_addr(ring + st * 2 * kTile), vb = kb + kTile;
#pragma unroll 4
                for (int i = 0; i < KT * (DP / 8) / 128; ++i) {
                    const int e = tid + 128 * i;
                    const int r = e / (DP / 8), c = e % (DP / 8);
                    const int64_t o = off_of[r];
                    const bool ok = o >= 0 && c * 8 < p.D;
                    const int64_t src = ok ? (o + c * 8) * 2 : 0;
                    const uint32_t to = chunk_at<DP>(r, c);
                    cp_async16(kb + to, p.k + src, ok);
                    cp_async16(vb + to, p.v + src, ok);
                }
            }
            cp_async_commit();
        };
        issue(0, 0);

        float o[NO][4];
        RowState st;
#pragma unroll
        for (int n = 0; n < NO; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;
        }
        int at[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            st.ref[r] = -INFINITY;
            st.sum[r] = 0.0f;
            at[r] = w.s.L - w.s.n +
                    (int)fast_div((uint32_t)(w.rt * M + wid * 16 + (lane >> 2) + 8 * r), p.gdiv);
        }
        for (int t = 0; t < w.cnt; ++t) {
            const int stage = t % ST;
            __syncthreads();  // the other stage is consumed
            issue(t + 1, (t + 1) % ST);
            cp_async_wait<1>();
            __syncthreads();  // this stage is complete for every thread
            const char* kt = ring + stage * 2 * kTile;
            const char* vt = kt + kTile;
            const uint32_t ka = smem_addr(kt), va = smem_addr(vt), qa = smem_addr(qt);
            const uint64_t dead = dead_of[stage][0] | ((uint64_t)dead_of[stage][1] << 32);
            const int j0 = (t0 + t) * KT;

            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][i] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t a[4];
                ldsm4(qa + chunk_at<DP>(wid * 16 + (lane & 15), 2 * k + (lane >> 4)), a);
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t b[4];
                    const int r = n * 8 + (lane & 7) + ((lane >> 4) << 3);
                    ldsm4(ka + chunk_at<DP>(r, 2 * k + ((lane >> 3) & 1)), b);
                    mma16816<T>(s[n], a, b[0], b[1]);
                    mma16816<T>(s[n + 1], a, b[2], b[3]);
                }
            }
            const bool part = j0 < w.keys.flo || j0 + KT > w.keys.fhi;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[n][i] *= p.scale_log2;
                    if (part || dead) {
                        const int c = n * 8 + (lane & 3) * 2 + (i & 1);
                        if (((dead >> c) & 1u) || !sees(p, at[i >> 1], j0 + c)) s[n][i] = -INFINITY;
                    }
                }
            }
            soft_tile<NT, NO>(s, o, st);
            bool odd = false;
            if (part) {
                for (int i = lane; i < kTile / 16; i += 32) {
                    const uint4 x = reinterpret_cast<const uint4*>(vt)[i];
                    odd |= unbounded<T>(x.x) || unbounded<T>(x.y) || unbounded<T>(x.z) || unbounded<T>(x.w);
                }
                odd = __any_sync(0xffffffffu, odd);
            }
#pragma unroll
            for (int k = 0; k < KT / 16; ++k) {
                if (odd) {
                    float two[2][4];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int c = (2 * k + n) * 8 + (lane & 3) * 2 + (i & 1);
                            const bool gone = ((dead >> c) & 1u) || !sees(p, at[i >> 1], j0 + c);
                            two[n][i] = gone ? -1.0f : s[2 * k + n][i];
                        }
                    }
                    careful_values<T, DP, 16, 2, NO>(two, o, vt + k * 16 * DP * 2, ps[wid], lane);
                    continue;
                }
                const uint32_t a[4] = {pack2<T>(s[2 * k][0], s[2 * k][1]), pack2<T>(s[2 * k][2], s[2 * k][3]),
                                       pack2<T>(s[2 * k + 1][0], s[2 * k + 1][1]),
                                       pack2<T>(s[2 * k + 1][2], s[2 * k + 1][3])};
#pragma unroll
                for (int n = 0; n < NO; n += 2) {
                    uint32_t b[4];
                    ldsm4t(va + chunk_at<DP>(k * 16 + (lane & 15), n + (lane >> 4)), b);
                    mma16816<T>(o[n], a, b[0], b[1]);
                    mma16816<T>(o[n + 1], a, b[2], b[3]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            st.sum[r] += __shfl_xor_sync(0xffffffffu, st.sum[r], 1);
            st.sum[r] += __shfl_xor_sync(0xffffffffu, st.sum[r], 2);
        }
        write_tile<T, M, NO>(p, w, o, st.ref, st.sum, wid * 16, rows < M ? rows : M, lane);
        if (tid == 0 && walk_slot(w) == 1) write_desc(p, w);
    } while (walk_next<M, KT, kMoreUC>(p, w));
    cp_async_wait<0>();
}

// ---------------------------------------------------------------- launch

int padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : D <= 192 ? 192 : 256; }

template <typename T>
cudaError_t launch_typed(const AttnP& p, const AttnShape& sh, cudaLaunchConfig_t cfg) {
    void (*fn)(AttnP) = nullptr;
    size_t smem = 0;
    const bool few = sh.path == kPathFew;
    switch (padded(p.D)) {
        case 64: fn = few ? attn_few_kernel<T, 64> : attn_more_kernel<T, 64>; smem = few ? few_smem<64>() : more_smem<64>(); break;
        case 128: fn = few ? attn_few_kernel<T, 128> : attn_more_kernel<T, 128>; smem = few ? few_smem<128>() : more_smem<128>(); break;
        case 192: fn = few ? attn_few_kernel<T, 192> : attn_more_kernel<T, 192>; smem = few ? few_smem<192>() : more_smem<192>(); break;
        default: fn = few ? attn_few_kernel<T, 256> : attn_more_kernel<T, 256>; smem = few ? few_smem<256>() : more_smem<256>(); break;
    }
    const cudaError_t e = allow_smem((const void*)fn, (int)smem);
    if (e != cudaSuccess) return e;
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = smem;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace

AttnShape mma_shape(AttnPath path, int dt, int head_dim) {
    (void)dt;
    const int per_sm = padded(head_dim) <= 128 ? 2 : 1;
    const bool few = path == kPathFew;
    return AttnShape{path, few ? 16 : 64, few ? kFewKeys : kMoreKeys, few ? kFewUC : kMoreUC, per_sm * sm_count(),
                     few ? kFewWarps : 1};
}

cudaError_t launch_attn_mma(const AttnP& p, const AttnShape& sh, int dt, cudaLaunchConfig_t cfg) {
    return dt == kF16 ? launch_typed<__half>(p, sh, cfg) : launch_typed<__nv_bfloat16>(p, sh, cfg);
}

}  // namespace edge
