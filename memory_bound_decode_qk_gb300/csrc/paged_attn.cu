// paged_attn.cu -- attention of a chunk of new tokens over a paged KV cache
// (sm_103a): dispatch, the kernel for any type and head size, and the join of
// split units.
//
// What it computes.  Sequence b has L_b keys in the cache and n_b new queries,
// the last n_b of its positions: query i sits at L_b - n_b + i.  Key j lies in
// slot table[b][j / page] * page + j % page of k_cache and v_cache.  For query
// head h with key head h / G:
//   s_j = scale q . k_j over the keys the query sees (j < L_b, a page inside
//         the pool, and when causal j <= position and, with a window, fewer
//         than `window` positions back)
//   out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),   lse = m + ln sum
// One pass over the keys with the running maximum m and sum (online softmax,
// Milakov and Gimelshein 2018), both in fp32 and in base 2.  A query that
// sees no key gives 0 and lse -inf.
#include "paged_common.cuh"

namespace edge {
namespace {

constexpr int kAnyM = 16;       // query rows of a unit
constexpr int kAnyKT = 32;      // keys of a tile: one per lane
constexpr int kAnyThreads = 256;
constexpr int kAnyRows = 2;     // rows of a warp
constexpr int kAnyUC = 1;

// floats per staged row: a multiple of 4 whose quarter is odd, so that 8
// lanes reading 16 bytes of 8 rows touch all banks once
__host__ __device__ constexpr int any_stride(int D) {
    return (((D + 3) / 4) | 1) * 4;
}

// fp32 rows of whole 16-byte vectors are copied asynchronously into two stages.
template <typename T, bool VEC>
constexpr __host__ __device__ int any_stages() {
    return std::is_same<T, float>::value && VEC ? 2 : 1;
}
__host__ __device__ constexpr int any_smem_floats(int D, int stages) {
    return (kAnyM + 2 * stages * kAnyKT) * any_stride(D) + kAnyM * kAnyKT;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
}

// Any type, head size up to 128 NC and alignment.  Eight warps of two rows each;
// a tile's keys and values are staged as fp32 in shared memory.  Scores: lane =
// key, so a key's 16 bytes serve two rows.  Values: four channels per lane, two
// rows per load.  A key that a row does not see (its weight is noted as -1) is
// skipped, so what the cache holds there does not matter.  Bound by the latency
// of a tile's steps at small sizes and by shared-memory reads at large ones (per
// key and channel quarter of two rows: one 16-byte read for 8 products).
// Measured on GB300: five fp32 chunks of 1 to 37 tokens over up to 999 keys, 8/2
// heads of 128, 24 us (36 us with four warps of four rows and one stage).
template <typename T, int NC, bool VEC>
__global__ void __launch_bounds__(kAnyThreads) attn_any_kernel(AttnP p) {
    constexpr int M = kAnyM, KT = kAnyKT, R = kAnyRows, ST = any_stages<T, VEC>();
    extern __shared__ __align__(16) float smem[];
    __shared__ WalkSmem<1> wsm;
    // of three tiles: one is written while the slowest warp is a tile behind
    __shared__ int64_t slot_of[3][KT];
    const int D = p.D, ds = any_stride(D);
    float* qs = smem;
    float* ring = qs + M * ds;  // stages of [keys | values]
    float* ps = ring + 2 * ST * KT * ds;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;

    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) clear_desc(p, blockIdx.x);
    // the padding channels stay zero
    for (int i = tid; i < (M + 2 * ST * KT) * ds; i += kAnyThreads) smem[i] = 0.0f;

    Walk w;
    if (!walk_begin<M, KT, kAnyUC, 1>(p, w, wsm, kAnyThreads, 0)) return;
    do {
        const int rows = w.s.n * p.G;
        const int r0 = w.rt * M;
        const int t0 = w.k0 + w.off;
        __syncthreads();
        // slots of tile t's keys, by the first warp
        auto look = [&](int t) {
            if (tid < KT) {
                const int j = (t0 + t) * KT + tid;
                slot_of[t % 3][tid] = j < w.s.L ? key_slot(p, w.b, j) : -1;
            }
        };
        // tile t into its stage (asynchronously with two stages)
        auto load = [&](int t) {
            float* ks = ring + (ST == 2 ? (t & 1) * 2 * KT * ds : 0);
            float* vs = ks + KT * ds;
            const int64_t* slots = slot_of[t % 3];
            if constexpr (VEC) {
                constexpr int N = vec_elems<T>();
                const int nv = D / N;
                for (int i = tid; i < KT * nv; i += kAnyThreads) {
                    const int j = i / nv, c = i - j * nv;
                    const int64_t slot = slots[j];
                    const int64_t e = slot >= 0 ? (slot * p.hk + w.h) * nv + c : 0;
                    if constexpr (ST == 2) {
                        cp_async16(ks + j * ds + c * N, reinterpret_cast<const uint4*>(p.k) + e, slot >= 0);
                        cp_async16(vs + j * ds + c * N, reinterpret_cast<const uint4*>(p.v) + e, slot >= 0);
                    } else {
                        uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
                        if (slot >= 0) {
                            x = __ldg(reinterpret_cast<const uint4*>(p.k) + e);
                            y = __ldg(reinterpret_cast<const uint4*>(p.v) + e);
                        }
                        float f[N], g[N];
                        unpack_vec<T, N>(x, f);
                        unpack_vec<T, N>(y, g);
#pragma unroll
                        for (int z = 0; z < N; ++z) {
                            ks[j * ds + c * N + z] = f[z];
                            vs[j * ds + c * N + z] = g[z];
                        }
                    }
                }
            } else {
                for (int i = tid; i < KT * D; i += kAnyThreads) {
                    const int j = i / D, d = i - j * D;
                    const int64_t slot = slots[j];
                    float a = 0.0f, b = 0.0f;
                    if (slot >= 0) {
                        const int64_t e = (slot * p.hk + w.h) * D + d;
                        a = to_f(reinterpret_cast<const T*>(p.k)[e]);
                        b = to_f(reinterpret_cast<const T*>(p.v)[e]);
                    }
                    ks[j * ds + d] = a;
                    vs[j * ds + d] = b;
                }
            }
            if constexpr (ST == 2) asm volatile("cp.async.commit_group;" ::: "memory");
        };
        look(0);
        for (int i = tid; i < M * D; i += kAnyThreads) {
            const int r = i / D, d = i - r * D;
            float x = 0.0f;
            if (r0 + r < rows) {
                x = to_f(reinterpret_cast<const T*>(p.q)[out_row(p, w.s, w.h, r0 + r) * D + d]);
            }
            qs[r * ds + d] = x;
        }
        float4 acc[R][NC];
        float m[R], l[R];
        int at[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.0f;
            at[r] = w.s.L - w.s.n + (int)fast_div((uint32_t)(r0 + wid * R + r), p.gdiv);
#pragma unroll
            for (int i = 0; i < NC; ++i) acc[r][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        __syncthreads();
        if constexpr (ST == 2) load(0);
        for (int t = 0; t < w.cnt; ++t) {
            const int j0 = (t0 + t) * KT;
            if constexpr (ST == 2) {
                if (t + 1 < w.cnt) look(t + 1);
                __syncthreads();  // the slots of t + 1; the tile before is consumed
                if (t + 1 < w.cnt) {
                    load(t + 1);
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                } else {
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                }
            } else {
                if (t > 0) {
                    __syncthreads();  // the tile before is consumed
                    look(t);
                    __syncthreads();
                }
                load(t);
            }
            __syncthreads();
            const float* ks = ring + (ST == 2 ? (t & 1) * 2 * KT * ds : 0);
            const float* vs = ks + KT * ds;
            const bool in = slot_of[t % 3][lane] >= 0;
            // two sums per row, of even and odd quarters
            float s[R][2] = {};
            const float4* kr = reinterpret_cast<const float4*>(ks + lane * ds);
            const int nq = (D + 3) / 4;
#pragma unroll 4
            for (int c = 0; c < nq; ++c) {
                const float4 kk = kr[c];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float4 qq = reinterpret_cast<const float4*>(qs + (wid * R + r) * ds)[c];
                    float& x = s[r][c & 1];
                    x = fmaf(qq.x, kk.x, x);
                    x = fmaf(qq.y, kk.y, x);
                    x = fmaf(qq.z, kk.z, x);
                    x = fmaf(qq.w, kk.w, x);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool seen = in && sees(p, at[r], j0 + lane);
                const float x = seen ? (s[r][0] + s[r][1]) * p.scale_log2 : -INFINITY;
                const float top = fmaxf(m[r], group_max<32>(x));
                const float ref = top == -INFINITY ? 0.0f : top;
                const float keep = ex2(m[r] - ref);
                const float e = ex2(x - ref);
                m[r] = top;
                l[r] = l[r] * keep + group_sum<32>(e);
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    acc[r][i].x *= keep;
                    acc[r][i].y *= keep;
                    acc[r][i].z *= keep;
                    acc[r][i].w *= keep;
                }
                ps[(wid * R + r) * KT + lane] = seen ? e : -1.0f;
            }
            __syncwarp();
#pragma unroll 2
            for (int j = 0; j < KT; j += 4) {
                float4 e[R];
#pragma unroll
                for (int r = 0; r < R; ++r) e[r] = *reinterpret_cast<const float4*>(ps + (wid * R + r) * KT + j);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    float4 vv[NC];
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        const int d = 4 * lane + 128 * i;
                        vv[i] = d < D ? *reinterpret_cast<const float4*>(vs + (j + z) * ds + d) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float x = z == 0 ? e[r].x : z == 1 ? e[r].y : z == 2 ? e[r].z : e[r].w;
                        if (!(x < 0.0f)) {
#pragma unroll
                            for (int i = 0; i < NC; ++i) {
                                acc[r][i].x = fmaf(x, vv[i].x, acc[r][i].x);
                                acc[r][i].y = fmaf(x, vv[i].y, acc[r][i].y);
                                acc[r][i].z = fmaf(x, vv[i].z, acc[r][i].z);
                                acc[r][i].w = fmaf(x, vv[i].w, acc[r][i].w);
                            }
                        }
                    }
                }
            }
        }
        const int slot = walk_slot(w);
        float* part = slot < 0 ? nullptr : part_of<M>(p, w.piece, slot);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = wid * R + r;
            if (r0 + row >= rows) continue;
            const int64_t orow = out_row(p, w.s, w.h, r0 + row);
            const float inv = part != nullptr ? 1.0f : l[r] == 0.0f ? 0.0f : 1.0f / l[r];
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const float y[4] = {acc[r][i].x, acc[r][i].y, acc[r][i].z, acc[r][i].w};
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int d = 4 * lane + 128 * i + z;
                    if (d >= D) continue;
                    if (part != nullptr) {
                        part[row * D + d] = y[z];
                    } else {
                        store_one<T>(p, orow * D + d, y[z] * inv);
                    }
                }
            }
            if (lane == 0) {
                if (part != nullptr) {
                    part[M * D + row] = m[r];
                    part[M * D + M + row] = l[r];
                } else if (p.lse != nullptr) {
                    p.lse[orow] = row_lse(m[r], l[r]);
                }
            }
        }
        if (slot == 1 && tid == 0) write_desc(p, w);
    } while (walk_next<M, KT, kAnyUC>(p, w));
}

// Joins the parts of the unit that started in piece blockIdx.x without ending
// there: with M = max m_i, out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.  Eight
// warps; W of them share a row's parts (a lane has every 32nd channel, the
// warps' sums are added in their order), so a CTA does 8 / W rows at a time.
constexpr int kJoinWarps = 8;
template <typename T, int M, int W>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(AttnP p) {
    constexpr int R = kJoinWarps / W;
    __shared__ float acc_of[W > 1 ? kJoinWarps : 1][256];
    __shared__ float top_of[kJoinWarps], sum_of[kJoinWarps];
    pdl_wait();
    pdl_launch_dependents();
    const int c0 = blockIdx.x, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int sub = wid % W, set = wid / W * W;
    const int4 u = p.desc[2 * c0], v = p.desc[2 * c0 + 1];
    if (u.x < 0) return;
    const Seq s{v.x, v.y, 0};
    const int rows = min(M, s.n * p.G - u.z * M);
    const int64_t rec = M * (int64_t)p.D + 2 * M;
    // parts: slot 1 of c0, then slot 0 of c0 + 1 .. u.x
    const float* base = p.part + ((int64_t)c0 * 2 + 1) * rec;
    const int n = u.x - c0 + 1;
    // whether warp i's parts saw anything (as for a part)
    auto counts = [&](int i) { return top_of[i] != -INFINITY || sum_of[i] != 0.0f; };
    for (int r0 = blockIdx.y * R; r0 < rows; r0 += gridDim.y * R) {
        const int r = min(r0 + wid / W, rows - 1);  // warps past the last row repeat it
        // one pass over this warp's parts with their running maximum
        float top = -INFINITY, l = 0.0f, acc[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
#pragma unroll 2
        for (int i = sub; i < n; i += W) {
            const float* pc = base + (i == 0 ? 0 : (2 * i - 1) * rec);
            const float m = pc[M * p.D + r], li = pc[M * p.D + M + r];
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int d = lane + 32 * k;
                x[k] = d < p.D ? pc[(int64_t)r * p.D + d] : 0.0f;
            }
            // a part that saw nothing has m = -inf and a sum of zero; one whose
            // scores are all NaN has m = -inf (maxima pass NaN over) and the NaN in
            // its sum, which the row takes on
            if (m == -INFINITY && li == 0.0f) continue;
            const float next = fmaxf(top, m);
            const float keep = ex2(top - next), f = ex2(m - next);
            top = next;
            l = fmaf(l, keep, f * li);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = fmaf(acc[k], keep, f * x[k]);
        }
        if constexpr (W > 1) {
            if (lane == 0) {
                top_of[wid] = top;
                sum_of[wid] = l;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) acc_of[wid][lane + 32 * k] = acc[k];
            __syncthreads();
            float all = -INFINITY;
            for (int i = 0; i < W; ++i) all = fmaxf(all, top_of[set + i]);
            top = all;
            l = 0.0f;
            for (int i = 0; i < W; ++i) {
                if (counts(set + i)) l = fmaf(ex2(top_of[set + i] - top), sum_of[set + i], l);
            }
        }
        const int64_t orow = out_row(p, s, u.y, u.z * M + r);
        const bool mine = r0 + wid / W < rows;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        if constexpr (W > 1) {
            for (int d = sub * 32 + lane; mine && d < p.D; d += 32 * W) {
                float y = 0.0f;
                for (int i = 0; i < W; ++i) {
                    if (counts(set + i)) y = fmaf(ex2(top_of[set + i] - top), acc_of[set + i][d], y);
                }
                store_one<T>(p, orow * p.D + d, y * inv);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int d = lane + 32 * k;
                if (mine && d < p.D) store_one<T>(p, orow * p.D + d, acc[k] * inv);
            }
        }
        if (mine && sub == 0 && lane == 0 && p.lse != nullptr) p.lse[orow] = row_lse(top, l);
        if constexpr (W > 1) __syncthreads();  // the shared sums are read before the next rows'
    }
}

template <typename T>
cudaError_t launch_any(const AttnP& p, bool vec, cudaLaunchConfig_t cfg) {
    cfg.blockDim = dim3(kAnyThreads);
    cfg.dynamicSmemBytes = (size_t)any_smem_floats(p.D, vec ? any_stages<T, true>() : 1) * 4;
    void (*fn)(AttnP);
    if (p.D <= 128) fn = vec ? attn_any_kernel<T, 1, true> : attn_any_kernel<T, 1, false>;
    else fn = vec ? attn_any_kernel<T, 2, true> : attn_any_kernel<T, 2, false>;
    const cudaError_t e = allow_smem((const void*)fn, (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

template <typename T, int W>
cudaError_t launch_join_of(const AttnP& p, int M, cudaLaunchConfig_t cfg) {
    switch (M) {
        case 16: return cudaLaunchKernelEx(&cfg, attn_join_kernel<T, 16, W>, p);
        case 64: return cudaLaunchKernelEx(&cfg, attn_join_kernel<T, 64, W>, p);
        case 128: return cudaLaunchKernelEx(&cfg, attn_join_kernel<T, 128, W>, p);
        default: return cudaLaunchKernelEx(&cfg, attn_join_kernel<T, 256, W>, p);
    }
}

template <typename T>
cudaError_t launch_join(const AttnP& p, const AttnShape& sh, cudaLaunchConfig_t cfg) {
    const int64_t all = p.tokens * (int64_t)p.G;
    const int rows = sh.M < all ? sh.M : (int)all;
    const int pieces = sh.ctas * sh.per_cta;
    // a unit spans few pieces when there are about as many units: a warp per
    // row then (one CTA per unit), else the eight warps of a CTA share a row
    const bool few = pieces <= 8 * (int64_t)p.num_seqs * p.hk;
    const int r = few ? kJoinWarps : 1;
    const int y = (rows + r - 1) / r;
    cfg.gridDim = dim3((unsigned)pieces, y < 16 ? y : 16);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.dynamicSmemBytes = 0;
    return few ? launch_join_of<T, 1>(p, sh.M, cfg) : launch_join_of<T, kJoinWarps>(p, sh.M, cfg);
}

// Two CTAs per SM fit up to 128 channels (at most 78 KB each; 152 KB at 256).
AttnShape any_shape() { return AttnShape{kPathAny, kAnyM, kAnyKT, kAnyUC, 2 * sm_count(), 1}; }

int64_t shape_bytes(const AttnShape& sh, int head_dim) {
    return (int64_t)sh.ctas * sh.per_cta * (32 + 2 * 4 * ((int64_t)sh.M * head_dim + 2 * sh.M));
}

}  // namespace

int64_t attn_workspace(int dt, int q_heads, int kv_heads, int head_dim) {
    (void)q_heads;
    (void)kv_heads;
    int64_t n = shape_bytes(any_shape(), head_dim);
    if (dt != kF32 && head_dim % 8 == 0) {
        for (AttnPath path : {kPathFew, kPathMore}) {
            const int64_t b = shape_bytes(mma_shape(path, dt, head_dim), head_dim);
            if (b > n) n = b;
        }
        const int64_t b = shape_bytes(tc_shape(head_dim), head_dim);
        if (b > n) n = b;
    }
    return n;
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s) {
    AttnP p;
    p.q = static_cast<const char*>(a.q);
    p.k = static_cast<const char*>(a.k_cache);
    p.v = static_cast<const char*>(a.v_cache);
    p.out = static_cast<char*>(a.out);
    p.lse = a.lse;
    p.table = a.table;
    p.lens = a.lens;
    p.starts = a.starts;
    p.num_seqs = a.num_seqs;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.page_size = a.page_size;
    p.tokens = (int)a.tokens;
    p.hq = a.q_heads;
    p.hk = a.kv_heads;
    p.G = a.q_heads / a.kv_heads;
    p.D = a.head_dim;
    p.gdiv = make_fastdiv((uint32_t)p.G);
    p.pdiv = make_fastdiv((uint32_t)a.page_size);
    p.causal = a.causal;
    // positions and keys are below 2^30, so a wider window is none, and the
    // kernels' differences stay inside 32 bits
    p.window = a.causal ? (a.window < (1 << 30) ? a.window : 1 << 30) : 0;
    p.out_fp8 = a.out_dt == kFP8;
    p.max_len = a.max_pages * a.page_size;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.inv = a.inv_scale;
    const int es = a.dt == kF32 ? 4 : 2;
    auto aligned = [](const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) % 16) == 0; };
    const bool vec = (a.head_dim * es) % 16 == 0 && aligned(a.k_cache) && aligned(a.v_cache);
    AttnShape sh = any_shape();
    if (a.dt != kF32 && vec && aligned(a.q)) {
        // Packed (token, head of the group) rows of the average sequence: the
        // lengths are on the device.  Measured on GB300 with every path for the
        // same batches (21 each: 1 to 256 sequences of 64 to 16,000 keys, three
        // head shapes), the geometric mean of the times over that of the
        // tcgen05 kernel: 16-row kernel 0.99 at 16 rows (0.27 to 1.84: many short
        // sequences want it, few long ones do not), 1.20 at 24, 1.42 at 48 and
        // 1.59 at 64; 64-row kernel 1.41, 1.43, 1.45 and 1.50.  Of these two,
        // for what tcgen05 does not serve, the first takes 0.70, 0.84, 0.97 and
        // 1.06 times the second's time.  A batch of sequences of very different
        // numbers of new tokens still goes one way: 63 decode tokens with a
        // chunk of 150 are one for the 16-row kernel.
        const int64_t rows = a.tokens * p.G / a.num_seqs;
        if (rows > 16 && aligned(a.out) && tc_suits(p)) sh = tc_shape(a.head_dim);
        else sh = mma_shape(rows <= 48 ? kPathFew : kPathMore, a.dt, a.head_dim);
    }
    p.min_per = sh.path == kPathFew ? 2 : 1;
    // no more CTAs than there can be pieces: the table's width bounds the tiles
    // of a unit, the tokens the units
    {
        const int64_t units = a.num_seqs + a.tokens * p.G / sh.M;
        const int64_t tiles = p.max_len / sh.KT + 2 + sh.UC;
        const int64_t most = (units * a.kv_heads * tiles + p.min_per - 1) / p.min_per;
        const int64_t ctas = (most + sh.per_cta - 1) / sh.per_cta;
        if (ctas < sh.ctas) sh.ctas = ctas > 1 ? (int)ctas : 1;
    }
    p.desc = static_cast<int4*>(a.workspace);
    p.part = reinterpret_cast<float*>(p.desc + 2 * (int64_t)sh.ctas * sh.per_cta);

    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    cfg.gridDim = dim3((unsigned)sh.ctas);
    cudaError_t e;
    if (sh.path == kPathMany) e = launch_attn_tc(p, a.dt, cfg);
    else if (sh.path != kPathAny) e = launch_attn_mma(p, sh, a.dt, cfg);
    else if (a.dt == kF32) e = launch_any<float>(p, vec, cfg);
    else if (a.dt == kF16) e = launch_any<__half>(p, vec, cfg);
    else e = launch_any<__nv_bfloat16>(p, vec, cfg);
    if (e != cudaSuccess) return e;
    if (a.dt == kF32) return launch_join<float>(p, sh, cfg);
    if (a.dt == kF16) return launch_join<__half>(p, sh, cfg);
    return launch_join<__nv_bfloat16>(p, sh, cfg);
}

}  // namespace edge
