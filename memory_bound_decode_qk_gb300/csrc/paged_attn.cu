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
constexpr int kAnyThreads = 128;
constexpr int kAnyUC = 1;

// floats per staged row: a multiple of 4 whose quarter is odd, so that 8
// lanes reading 16 bytes of 8 rows touch all banks once
__host__ __device__ constexpr int any_stride(int D) {
    return (((D + 3) / 4) | 1) * 4;
}

__host__ __device__ constexpr int any_smem_floats(int D) {
    return (kAnyM + 2 * kAnyKT) * any_stride(D) + kAnyM * kAnyKT;
}

// Any type, head size up to 32 NV and alignment.  Four warps; a tile's keys
// and values are staged as fp32 in shared memory.  Scores: lane = key, a warp
// does its four rows, so a key's 16 bytes serve four rows.  Values: lane =
// channel, four rows per load.  A key of weight zero (masked, or underflowed)
// is skipped, so what the cache holds there does not matter.
template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(kAnyThreads) attn_any_kernel(AttnP p) {
    constexpr int M = kAnyM, KT = kAnyKT;
    extern __shared__ __align__(16) float smem[];
    __shared__ WalkSmem<1> wsm;
    __shared__ int64_t slot_of[KT];
    const int D = p.D, ds = any_stride(D);
    float* qs = smem;
    float* ks = qs + M * ds;
    float* vs = ks + KT * ds;
    float* ps = vs + KT * ds;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;

    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) clear_desc(p, blockIdx.x);
    // the padding channels stay zero
    for (int i = tid; i < (M + 2 * KT) * ds; i += kAnyThreads) smem[i] = 0.0f;

    Walk w;
    if (!walk_begin<M, KT, kAnyUC, 1>(p, w, wsm, kAnyThreads, 0)) return;
    do {
        const int rows = w.s.n * p.G;
        const int r0 = w.rt * M;
        __syncthreads();
        for (int i = tid; i < M * D; i += kAnyThreads) {
            const int r = i / D, d = i - r * D;
            float x = 0.0f;
            if (r0 + r < rows) {
                x = to_f(reinterpret_cast<const T*>(p.q)[out_row(p, w.s, w.h, r0 + r) * D + d]);
            }
            qs[r * ds + d] = x;
        }
        float acc[4][NV], m[4], l[4];
        int at[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.0f;
            at[r] = w.s.L - w.s.n + (int)fast_div((uint32_t)(r0 + wid * 4 + r), p.gdiv);
#pragma unroll
            for (int i = 0; i < NV; ++i) acc[r][i] = 0.0f;
        }
        for (int kt = w.k0 + w.off; kt < w.k0 + w.off + w.cnt; ++kt) {
            const int j0 = kt * KT;
            __syncthreads();  // the tile before is consumed
            if (tid < KT) slot_of[tid] = j0 + tid < w.s.L ? key_slot(p, w.b, j0 + tid) : -1;
            __syncthreads();
            if constexpr (VEC) {
                constexpr int N = vec_elems<T>();
                const int nv = D / N;
                for (int i = tid; i < 2 * KT * nv; i += kAnyThreads) {
                    const bool isv = i >= KT * nv;
                    const int e = isv ? i - KT * nv : i;
                    const int j = e / nv, c = e - j * nv;
                    const int64_t slot = slot_of[j];
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (slot >= 0) {
                        x = __ldg(reinterpret_cast<const uint4*>(isv ? p.v : p.k) +
                                  (slot * p.hk + w.h) * nv + c);
                    }
                    float f[N];
                    unpack_vec<T, N>(x, f);
                    float* dst = (isv ? vs : ks) + j * ds + c * N;
#pragma unroll
                    for (int t = 0; t < N; ++t) dst[t] = f[t];
                }
            } else {
                for (int i = tid; i < KT * D; i += kAnyThreads) {
                    const int j = i / D, d = i - j * D;
                    const int64_t slot = slot_of[j];
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
            __syncthreads();
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            const float4* kr = reinterpret_cast<const float4*>(ks + lane * ds);
            for (int c = 0; c < (D + 3) / 4; ++c) {
                const float4 kk = kr[c];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 qq = reinterpret_cast<const float4*>(qs + (wid * 4 + r) * ds)[c];
                    s[r] = fmaf(qq.x, kk.x, s[r]);
                    s[r] = fmaf(qq.y, kk.y, s[r]);
                    s[r] = fmaf(qq.z, kk.z, s[r]);
                    s[r] = fmaf(qq.w, kk.w, s[r]);
                }
            }
            const bool in = slot_of[lane] >= 0;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float x = in && sees(p, at[r], j0 + lane) ? s[r] * p.scale_log2 : -INFINITY;
                const float top = fmaxf(m[r], group_max<32>(x));
                const float ref = top == -INFINITY ? 0.0f : top;
                const float keep = ex2(m[r] - ref);
                const float e = ex2(x - ref);
                m[r] = top;
                l[r] = l[r] * keep + group_sum<32>(e);
#pragma unroll
                for (int i = 0; i < NV; ++i) acc[r][i] *= keep;
                ps[(wid * 4 + r) * KT + lane] = e;
            }
            __syncwarp();
            for (int j = 0; j < KT; ++j) {
                float vv[NV];
#pragma unroll
                for (int i = 0; i < NV; ++i) vv[i] = lane + 32 * i < D ? vs[j * ds + lane + 32 * i] : 0.0f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = ps[(wid * 4 + r) * KT + j];
                    if (e != 0.0f) {
#pragma unroll
                        for (int i = 0; i < NV; ++i) acc[r][i] = fmaf(e, vv[i], acc[r][i]);
                    }
                }
            }
        }
        const int slot = walk_slot(w);
        float* part = slot < 0 ? nullptr : part_of<M>(p, w.piece, slot);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = wid * 4 + r;
            if (r0 + row >= rows) continue;
            if (part != nullptr) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (lane + 32 * i < D) part[row * D + lane + 32 * i] = acc[r][i];
                }
                if (lane == 0) {
                    part[M * D + row] = m[r];
                    part[M * D + M + row] = l[r];
                }
            } else {
                const int64_t orow = out_row(p, w.s, w.h, r0 + row);
                const float inv = l[r] == 0.0f ? 0.0f : 1.0f / l[r];
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (lane + 32 * i < D) store_one<T>(p, orow * D + lane + 32 * i, acc[r][i] * inv);
                }
                if (lane == 0 && p.lse != nullptr) p.lse[orow] = row_lse(m[r], l[r]);
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
            // (a part that saw nothing has m = -inf and wrote no outputs)
            if (m == -INFINITY) continue;
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
                if (top_of[set + i] != -INFINITY) l = fmaf(ex2(top_of[set + i] - top), sum_of[set + i], l);
            }
        }
        const int64_t orow = out_row(p, s, u.y, u.z * M + r);
        const bool mine = r0 + wid / W < rows;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        if constexpr (W > 1) {
            for (int d = sub * 32 + lane; mine && d < p.D; d += 32 * W) {
                float y = 0.0f;
                for (int i = 0; i < W; ++i) {
                    if (top_of[set + i] != -INFINITY) y = fmaf(ex2(top_of[set + i] - top), acc_of[set + i][d], y);
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
    cfg.dynamicSmemBytes = (size_t)any_smem_floats(p.D) * 4;
    void (*fn)(AttnP);
    if (p.D <= 64) fn = vec ? attn_any_kernel<T, 2, true> : attn_any_kernel<T, 2, false>;
    else if (p.D <= 128) fn = vec ? attn_any_kernel<T, 4, true> : attn_any_kernel<T, 4, false>;
    else fn = vec ? attn_any_kernel<T, 8, true> : attn_any_kernel<T, 8, false>;
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

// Two CTAs per SM fit at every head size (at most 88 KB each).
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
    p.window = a.causal ? a.window : 0;
    p.out_fp8 = a.out_dt == kFP8;
    p.max_len = a.max_pages * a.page_size;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.inv = a.inv_scale;
    const int es = a.dt == kF32 ? 4 : 2;
    auto aligned = [](const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) % 16) == 0; };
    const bool vec = (a.head_dim * es) % 16 == 0 && aligned(a.k_cache) && aligned(a.v_cache);
    AttnShape sh = any_shape();
    if (a.dt != kF32 && vec && aligned(a.q)) {
        // rows of a unit: packed (token, head of the group) rows of the
        // average sequence
        const int64_t rows = a.tokens * p.G / a.num_seqs;
        if (rows > 64 && tc_suits(p)) sh = tc_shape(a.head_dim);
        else sh = mma_shape(rows <= 16 ? kPathFew : kPathMore, a.dt, a.head_dim);
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
