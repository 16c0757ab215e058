// pages.cu -- copying, forking, freeing and compacting pages of a KV cache (sm_103a).
//
// A pool of pages is common to any number of caches (the key and value caches
// of every layer): page p of a cache is its bytes [p B, (p + 1) B).  Sequences
// hold pages through a block table; refs[p] counts the entries that name page
// p, and a page with no reference is free.  All of that lives on the device,
// so a step that forks or frees sequences needs no host synchronization and can
// be captured into a graph.
//
// GB300 design.  The data moves are HBM-bound: a page is read once and written
// once.  Work items are 16 KB of one page of one cache; a resident grid strides
// over them, every thread with four 16-byte loads in flight before its first
// store.  All caches of a move are served by one launch (their addresses are
// kernel parameters), so a small move costs one launch, not one per layer.
// Measured on GB300: 1000 pages of 32 KB in 16 caches (1.05 GB read and written)
// 174 us, 6.0 TB/s, 89% of the copy bandwidth; compaction of a pool of 4096 such
// pages (0.77 GB moved) 130 us, 5.9 TB/s.
// A caller's list of pairs is checked where it is carried out, each pair against
// all others for every 16 KB that a CTA takes.  That hides up to about a thousand
// pairs and is the bound beyond: pages of 2 KB in 4 caches, 1000 pairs 10 us,
// 10,000 293 us, 65,536 11.9 ms.
// The bookkeeping is integer work on a few KB: one CTA decides it (so that
// results do not depend on any order of atomics), and the copies follow as a
// dependent launch that reads the pairs it wrote.
#include "edge_common.cuh"
#include "fastdiv.h"
#include "launch.h"

namespace edge {
namespace {

constexpr int kMaxCaches = 64;      // of one launch
constexpr int kMoveThreads = 256;
constexpr int kMoveVecs = 4;
constexpr int kPlanThreads = 1024;

struct MoveP {
    char* cache[kMaxCaches];
    const int32_t* src;    // page of pair k at src[k stride], dst[k stride]
    const int32_t* dst;
    const int32_t* count;  // pairs, on the device; nullptr: n
    int stride, n;
    int num_pages;
    int64_t page_bytes;
    uint32_t units;        // 16-byte vectors, or bytes, of a page
    FastDiv pieces, caches;
};

// One pair's fate when the caller wrote the list: of pairs with one destination
// the last is carried out, and a pair whose source is the destination of
// another is not.  Pairs that name a page outside the pool, or one page twice,
// do not count.  Every thread of the block calls it.
__device__ bool pair_stands(const MoveP& p, int k) {
    auto in = [&](int x) { return x >= 0 && x < p.num_pages; };
    const int s = __ldg(p.src + (int64_t)k * p.stride), d = __ldg(p.dst + (int64_t)k * p.stride);
    bool bad = !in(s) || !in(d) || s == d;
    for (int j = threadIdx.x; j < p.n; j += blockDim.x) {
        const int t = __ldg(p.dst + (int64_t)j * p.stride);
        if (j == k || (t != d && t != s)) continue;
        const int f = __ldg(p.src + (int64_t)j * p.stride);
        if (!in(f) || f == t) continue;
        bad = bad || t == s || j > k;
    }
    return !__syncthreads_or(bad);
}

// CHECK: the pairs are the caller's (pair_stands); else they are this file's
// own, disjoint, with -1 where nothing is to be copied.  V: 16-byte vectors.
template <bool CHECK, bool V>
__global__ void __launch_bounds__(kMoveThreads) pages_move_kernel(const __grid_constant__ MoveP p) {
    pdl_wait();
    pdl_launch_dependents();
    const int n = p.count != nullptr ? __ldg(p.count) : p.n;
    const uint32_t items = (uint32_t)n * p.caches.d * p.pieces.d;
    int last = -1;
    bool stands = false;
    for (uint32_t it = blockIdx.x; it < items; it += gridDim.x) {
        const uint32_t t = fast_div(it, p.pieces);
        const uint32_t piece = it - t * p.pieces.d;
        const int k = (int)fast_div(t, p.caches);
        const uint32_t c = t - k * p.caches.d;
        if constexpr (CHECK) {
            if (k != last) {
                stands = pair_stands(p, k);
                last = k;
            }
            if (!stands) continue;
        }
        const int s = __ldg(p.src + (int64_t)k * p.stride), d = __ldg(p.dst + (int64_t)k * p.stride);
        if (!CHECK && (s < 0 || d < 0)) continue;
        const char* from = p.cache[c] + s * p.page_bytes;
        char* to = p.cache[c] + d * p.page_bytes;
        const uint32_t base = piece * (kMoveThreads * kMoveVecs) + threadIdx.x;
        if constexpr (V) {
            uint4 v[kMoveVecs];
#pragma unroll
            for (int i = 0; i < kMoveVecs; ++i) {
                const uint32_t e = base + i * kMoveThreads;
                if (e < p.units) v[i] = __ldcs(reinterpret_cast<const uint4*>(from) + e);
            }
#pragma unroll
            for (int i = 0; i < kMoveVecs; ++i) {
                const uint32_t e = base + i * kMoveThreads;
                if (e < p.units) reinterpret_cast<uint4*>(to)[e] = v[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < kMoveVecs; ++i) {
                const uint32_t e = base + i * kMoveThreads;
                if (e < p.units) to[e] = from[e];
            }
        }
    }
}

// Inclusive sum over the block's threads, in thread order; `total` is the sum.
__device__ __forceinline__ int block_scan(int v, int* warp, int& total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += up;
    }
    __syncthreads();  // the readers of the scan before
    if (lane == 31) warp[wid] = v;
    __syncthreads();
    total = 0;
    int before = 0;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) {
        if (i < wid) before += warp[i];
        total += warp[i];
    }
    return v + before;
}

// ---------------------------------------------------------------- free

struct RowsP {
    int32_t* table;
    int32_t* lens;
    int32_t* refs;
    const int32_t* rows;
    int num_rows, max_pages, num_pages;
};

// A CTA per listed row.  An entry is taken by exchange, so a row that is listed
// twice gives its pages back once.
__global__ void __launch_bounds__(128) pages_free_kernel(RowsP p) {
    pdl_wait();
    pdl_launch_dependents();
    const int row = __ldg(p.rows + blockIdx.x);
    if (row < 0 || row >= p.num_rows) return;
    int32_t* t = p.table + (int64_t)row * p.max_pages;
    for (int i = threadIdx.x; i < p.max_pages; i += blockDim.x) {
        const int page = atomicExch(t + i, -1);
        if (page >= 0 && page < p.num_pages) atomicSub(p.refs + page, 1);
    }
    if (threadIdx.x == 0) p.lens[row] = 0;
}

// ---------------------------------------------------------------- fork

constexpr int kMaxForks = (int)kMaxPageForks;

struct ForkP {
    int32_t* table;
    int32_t* lens;
    int32_t* refs;
    const int32_t* parents;
    const int32_t* children;
    int32_t* status;
    int32_t* pairs;
    int num_rows, max_pages, num_pages, page_size, n;
};

enum { kForked = 0, kNoPage = 1, kRefused = 2 };

__global__ void __launch_bounds__(kPlanThreads) pages_fork_kernel(ForkP p) {
    __shared__ int fresh[kMaxForks];  // the free pages taken, lowest first
    __shared__ int warp[32];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, nw = kPlanThreads / 32;
    const int64_t max_len = (int64_t)p.max_pages * p.page_size;
    auto in_pool = [&](int x) { return x >= 0 && x < p.num_pages; };

    // which forks stand, and which of them copy a partly filled page; a warp each
    for (int i = wid; i < p.n; i += nw) {
        const int par = p.parents[i], chi = p.children[i];
        bool bad = par < 0 || par >= p.num_rows || chi < 0 || chi >= p.num_rows;
        for (int j = lane; j < p.n; j += 32) {
            bad = bad || p.parents[j] == chi || (j < i && p.children[j] == chi);
        }
        bad = __any_sync(0xffffffffu, bad);
        if (!bad) {
            bad = p.lens[chi] != 0;
            for (int e = lane; e < p.max_pages; e += 32) {
                bad = bad || in_pool(p.table[(int64_t)chi * p.max_pages + e]);
            }
            bad = __any_sync(0xffffffffu, bad);
        }
        if (lane == 0) {
            int last = -1;
            if (!bad) {
                const int len = (int)min((int64_t)max(p.lens[par], 0), max_len);
                if (len % p.page_size != 0) last = p.table[(int64_t)par * p.max_pages + len / p.page_size];
            }
            const bool copies = in_pool(last);
            p.status[i] = bad ? kRefused : copies ? kNoPage : kForked;
            p.pairs[2 * i] = copies ? last : -1;
            p.pairs[2 * i + 1] = -1;
        }
    }
    __syncthreads();
    // the order in which the copying forks take pages
    int want = 0;
    for (int b = 0; b < p.n; b += kPlanThreads) {
        const int i = b + tid;
        const int copies = i < p.n && p.status[i] == kNoPage;
        int total;
        const int rank = want + block_scan(copies, warp, total) - 1;
        if (copies) p.pairs[2 * i + 1] = rank;
        want += total;
    }
    // the lowest free pages
    int found = 0;
    for (int b = 0; b < p.num_pages && found < want; b += 4 * kPlanThreads) {
        int free[4], mine = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int page = b + 4 * tid + k;
            free[k] = page < p.num_pages && p.refs[page] <= 0;
            mine += free[k];
        }
        int total;
        int rank = found + block_scan(mine, warp, total) - mine;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (free[k]) {
                if (rank < want) fresh[rank] = b + 4 * tid + k;
                ++rank;
            }
        }
        found += total;
    }
    __syncthreads();
    // the rows; no child is a parent, so what is read here is not written
    for (int i = wid; i < p.n; i += nw) {
        const int st = p.status[i], rank = p.pairs[2 * i + 1];
        __syncwarp();
        if (st == kRefused) continue;
        if (st == kNoPage && rank >= found) {
            if (lane == 0) {
                p.pairs[2 * i] = -1;
                p.pairs[2 * i + 1] = -1;
            }
            continue;
        }
        const int par = p.parents[i], chi = p.children[i];
        const int page = st == kNoPage ? fresh[rank] : -1;
        const int len = (int)min((int64_t)max(p.lens[par], 0), max_len);
        const int full = len / p.page_size;
        for (int e = lane; e < p.max_pages; e += 32) {
            int x = -1;
            if (e < full) {
                x = p.table[(int64_t)par * p.max_pages + e];
                if (in_pool(x)) atomicAdd(p.refs + x, 1);
            } else if (e == full) {
                x = page;
            }
            p.table[(int64_t)chi * p.max_pages + e] = x;
        }
        if (lane == 0) {
            p.lens[chi] = len;
            if (page >= 0) p.refs[page] = 1;
            p.pairs[2 * i + 1] = page;
            p.status[i] = kForked;
        }
    }
}

// ---------------------------------------------------------------- compact

struct CompactP {
    const int32_t* refs;
    int32_t* refs_out;
    int32_t* map;    // [num_pages]: new number of each page, -1 if free
    int32_t* pairs;  // [2 k], [2 k + 1]: source and destination of move k
    int32_t* count;
    int num_pages;
};

// L pages in use: the k-th page in use from L on moves to the k-th free page
// below L.  One CTA, two passes over refs: a few microseconds for the pools of
// thousands of pages that models serve from, beside moves of 100 and more.
__global__ void __launch_bounds__(kPlanThreads) pages_compact_kernel(CompactP p) {
    __shared__ int warp[32];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    int used = 0, total;
    for (int i = tid; i < p.num_pages; i += kPlanThreads) used += p.refs[i] > 0;
    block_scan(used, warp, total);
    const int L = total;
    int holes = 0, strays = 0;
    for (int b = 0; b < p.num_pages; b += 4 * kPlanThreads) {
        bool hole[4], stray[4];
        int nh = 0, ns = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int page = b + 4 * tid + k;
            const bool live = page < p.num_pages && p.refs[page] > 0;
            hole[k] = page < L && !live;
            stray[k] = live && page >= L;
            nh += hole[k];
            ns += stray[k];
            if (page < p.num_pages) p.map[page] = live ? page : -1;
        }
        int rh = holes + block_scan(nh, warp, total) - nh;
        holes += total;
        int rs = strays + block_scan(ns, warp, total) - ns;
        strays += total;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int page = b + 4 * tid + k;
            if (hole[k]) p.pairs[2 * rh++ + 1] = page;
            if (stray[k]) p.pairs[2 * rs++] = page;
        }
    }
    // holes == strays: both are L less the pages in use below L
    __syncthreads();
    for (int k = tid; k < strays; k += kPlanThreads) {
        const int s = p.pairs[2 * k], d = p.pairs[2 * k + 1];
        p.map[s] = d;
        p.refs_out[d] = p.refs[s];
    }
    __syncthreads();
    for (int i = tid; i < p.num_pages; i += kPlanThreads) {
        if (i >= L) {
            p.refs_out[i] = 0;
        } else if (p.refs_out != p.refs && p.map[i] == i) {
            p.refs_out[i] = p.refs[i];
        }
    }
    if (tid == 0) *p.count = strays;
}

__global__ void __launch_bounds__(256) pages_renumber_kernel(int32_t* out, const int32_t* table, const int32_t* map,
                                                             int64_t entries, int num_pages) {
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < entries; i += (int64_t)gridDim.x * blockDim.x) {
        const int x = table[i];
        out[i] = x >= 0 && x < num_pages ? __ldg(map + x) : x;
    }
}

// ---------------------------------------------------------------- launch

void dependent(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, cudaStream_t s) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
}

// Copies n pairs (or *count of them, at most n) in every cache.
cudaError_t launch_move(const PagePool& pool, const int32_t* src, const int32_t* dst, int stride, int n,
                        const int32_t* count, bool check, cudaStream_t s) {
    if (n == 0) return cudaSuccess;
    bool vec = pool.page_bytes % 16 == 0;
    for (int i = 0; i < pool.num_caches; ++i) vec = vec && (reinterpret_cast<uintptr_t>(pool.caches[i]) % 16) == 0;
    MoveP p;
    p.src = src;
    p.dst = dst;
    p.count = count;
    p.stride = stride;
    p.n = n;
    p.num_pages = pool.num_pages;
    p.page_bytes = pool.page_bytes;
    p.units = (uint32_t)(vec ? pool.page_bytes / 16 : pool.page_bytes);
    const uint32_t per = kMoveThreads * kMoveVecs;
    const uint32_t pieces = (p.units + per - 1) / per;
    p.pieces = make_fastdiv(pieces);
    // items are counted in 32 bits
    int64_t most = ((int64_t(1) << 31) - 1) / ((int64_t)n * pieces);
    if (most > kMaxCaches) most = kMaxCaches;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    dependent(cfg, attr, s);
    cfg.blockDim = dim3(kMoveThreads);
    for (int c0 = 0; c0 < pool.num_caches; c0 += (int)most) {
        const int nc = pool.num_caches - c0 < most ? pool.num_caches - c0 : (int)most;
        for (int i = 0; i < nc; ++i) p.cache[i] = static_cast<char*>(pool.caches[c0 + i]);
        p.caches = make_fastdiv((uint32_t)nc);
        int64_t blocks = (int64_t)n * nc * pieces;
        const int64_t cap = (int64_t)sm_count() * 8;
        if (blocks > cap) blocks = cap;
        cfg.gridDim = dim3((unsigned)blocks);
        cudaError_t e;
        if (check) e = vec ? cudaLaunchKernelEx(&cfg, pages_move_kernel<true, true>, p) : cudaLaunchKernelEx(&cfg, pages_move_kernel<true, false>, p);
        else e = vec ? cudaLaunchKernelEx(&cfg, pages_move_kernel<false, true>, p) : cudaLaunchKernelEx(&cfg, pages_move_kernel<false, false>, p);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

bool pages_fit(int64_t page_bytes, int64_t pairs) {
    // items of one cache, counted in vectors or (unaligned caches) in bytes
    const int64_t pieces = page_bytes / (kMoveThreads * kMoveVecs) + 1;
    return page_bytes < (int64_t(1) << 31) && pairs <= ((int64_t(1) << 31) - 1) / pieces;
}

cudaError_t launch_pages_copy(const PagePool& pool, const int32_t* src, const int32_t* dst, int n, cudaStream_t s) {
    return launch_move(pool, src, dst, 1, n, nullptr, true, s);
}

cudaError_t launch_pages_free(const PageRows& r, int32_t* refs, int num_pages, const int32_t* seqs, int n, cudaStream_t s) {
    RowsP p{r.table, r.lens, refs, seqs, r.num_seqs, r.max_pages, num_pages};
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    dependent(cfg, attr, s);
    cfg.gridDim = dim3((unsigned)n);
    cfg.blockDim = dim3(128);
    return cudaLaunchKernelEx(&cfg, pages_free_kernel, p);
}

cudaError_t launch_pages_fork(const PagePool& pool, const PageRows& r, int page_size, int32_t* refs, const int32_t* parents,
                              const int32_t* children, int n, int32_t* status, int32_t* pairs, cudaStream_t s) {
    ForkP p{r.table, r.lens, refs, parents, children, status, pairs, r.num_seqs, r.max_pages, pool.num_pages, page_size, n};
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    dependent(cfg, attr, s);
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cudaError_t e = cudaLaunchKernelEx(&cfg, pages_fork_kernel, p);
    if (e != cudaSuccess) return e;
    return launch_move(pool, pairs, pairs + 1, 2, n, nullptr, false, s);
}

// The workspace: map [num_pages], count (16 bytes), pairs [2 (num_pages / 2)].
int64_t pages_compact_workspace(int num_pages) { return ((int64_t)num_pages * 4 + 15) / 16 * 16 + 16 + (int64_t)num_pages * 4; }

cudaError_t launch_pages_compact(const PagePool& pool, int32_t* table_out, const PageRows& r, int32_t* refs_out,
                                 const int32_t* refs, void* workspace, cudaStream_t s) {
    CompactP p;
    p.refs = refs;
    p.refs_out = refs_out;
    p.map = static_cast<int32_t*>(workspace);
    p.count = p.map + ((int64_t)pool.num_pages + 3) / 4 * 4;
    p.pairs = p.count + 4;
    p.num_pages = pool.num_pages;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    dependent(cfg, attr, s);
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cudaError_t e = cudaLaunchKernelEx(&cfg, pages_compact_kernel, p);
    if (e != cudaSuccess) return e;
    const int64_t entries = (int64_t)r.num_seqs * r.max_pages;
    if (entries > 0) {
        int64_t blocks = (entries + 255) / 256;
        const int64_t cap = (int64_t)sm_count() * 8;
        cfg.gridDim = dim3((unsigned)(blocks < cap ? blocks : cap));
        cfg.blockDim = dim3(256);
        e = cudaLaunchKernelEx(&cfg, pages_renumber_kernel, table_out, (const int32_t*)r.table, (const int32_t*)p.map, entries,
                               pool.num_pages);
        if (e != cudaSuccess) return e;
    }
    return launch_move(pool, p.pairs, p.pairs + 1, 2, pool.num_pages / 2, p.count, false, s);
}

}  // namespace edge
