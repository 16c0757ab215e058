// paged_common.cuh -- what the paged-attention kernels share: parameters, key
// visibility, the work schedule and the partial results.
//
// Schedule.  A unit is M packed query rows of one sequence and one key head
// (rows are (token, query head of the group), token-major), and its work is a
// run of key tiles of KT keys.  The tiles of all units form one line, and every
// CTA takes an equal piece of it, wherever that starts and ends, so a batch of
// ragged lengths or one long sequence fills the GPU alike.  The lengths live on
// the device, so each CTA finds its piece itself: a block-wide sum of the
// sequences' tiles and a scan up to its own start.  A unit that lies in one
// CTA is written directly.  The pieces of a unit that spans several CTAs go to
// the workspace as (row maximum, row sum, unnormalized output) and a second
// kernel joins them.  At most one unit starts in a CTA without ending there
// (partial slot 1), and at most one ends there that started earlier (slot 0).
#pragma once

#include "edge_common.cuh"
#include "fastdiv.h"
#include "launch.h"

namespace edge {

// Kernel parameters (validated by the C ABI layer).
struct AttnP {
    const char* q;
    const char* k;
    const char* v;
    char* out;
    float* lse;         // nullable
    const int32_t* table;
    const int32_t* lens;
    const int32_t* starts;  // nullable: one token per sequence
    float* part;        // [ctas][2][M * D + 2 M] fp32
    int4* desc;         // [ctas]: unit of slot 1 (b, h, rt) and its last CTA, or w < 0
    int num_seqs, max_pages, num_pages, page_size;
    int tokens, hq, hk, G, D;
    FastDiv gdiv, pdiv;  // by G and by page_size
    int causal, window, out_fp8;
    int max_len;        // max_pages * page_size
    int min_per;        // fewest key tiles a CTA takes
    float scale_log2;   // scale * log2(e): scores are kept in base 2
    float inv;
};

struct Seq {
    int q0, n, L;  // first query row, new tokens, keys
};

// Every value read from the device is clamped, so a wrong one gives wrong
// rows and no access out of range.
__device__ __forceinline__ Seq load_seq(const AttnP& p, int b) {
    Seq s;
    if (p.starts == nullptr) {
        s.q0 = b;
        s.n = 1;
    } else {
        const int a = min(max(__ldg(p.starts + b), 0), p.tokens);
        const int e = min(max(__ldg(p.starts + b + 1), a), p.tokens);
        s.q0 = a;
        s.n = e - a;
    }
    s.L = min(max(__ldg(p.lens + b), 0), p.max_len);
    return s;
}

// Cache slot of key j of sequence b, or -1 if its page is not in the pool.
__device__ __forceinline__ int64_t key_slot(const AttnP& p, int b, int j) {
    const int pi = (int)fast_div((uint32_t)j, p.pdiv);
    const int page = __ldg(p.table + (int64_t)b * p.max_pages + pi);
    if (page < 0 || page >= p.num_pages) return -1;
    return (int64_t)page * p.page_size + (j - pi * p.page_size);
}

// Whether the query at position `at` sees key j < L.
__device__ __forceinline__ bool sees(const AttnP& p, int at, int j) {
    return !p.causal || (j <= at && (p.window <= 0 || at - j < p.window));
}

// Keys of row tile rt: [lo, hi) are seen by at least one of its rows (pages
// outside the pool apart), [flo, fhi) by all of them.
struct Keys {
    int lo, hi, flo, fhi;
};

template <int M>
__device__ __forceinline__ Keys tile_keys(const AttnP& p, const Seq& s, int rt) {
    Keys k{0, s.L, 0, s.L};
    if (p.causal) {
        const int r0 = rt * M;
        const int r1 = min(r0 + M, s.n * p.G);
        const int base = s.L - s.n;
        const int t0 = (int)fast_div((uint32_t)r0, p.gdiv);
        const int t1 = (int)fast_div((uint32_t)(r1 - 1), p.gdiv);
        k.hi = max(base + t1 + 1, 0);
        k.fhi = max(base + t0 + 1, 0);
        if (p.window > 0) {
            k.lo = max(base + t0 - p.window + 1, 0);
            k.flo = max(base + t1 - p.window + 1, 0);
        }
    }
    return k;
}

// Key tiles [k0, k1) of row tile rt; at least one, so that rows that see
// nothing are still written.
template <int M, int KT>
__device__ __forceinline__ Keys tile_range(const AttnP& p, const Seq& s, int rt, int& k0, int& k1) {
    const Keys k = tile_keys<M>(p, s, rt);
    k0 = k.lo / KT;
    k1 = max((k.hi + KT - 1) / KT, k0 + 1);
    return k;
}

template <int M, int KT>
__device__ __forceinline__ int64_t seq_tiles(const AttnP& p, const Seq& s) {
    int64_t c = 0;
    const int nrt = (s.n * p.G + M - 1) / M;
    for (int rt = 0; rt < nrt; ++rt) {
        int k0, k1;
        tile_range<M, KT>(p, s, rt, k0, k1);
        c += k1 - k0;
    }
    return c;
}

// This CTA's walk over its piece of the line.  Every thread holds the same
// copy.
struct Walk {
    int64_t left;  // tiles of the piece still to do, this unit's included
    int64_t after; // line position at which this unit ends
    int64_t per;   // tiles per CTA
    int b, h, rt;
    Seq s;
    int k0, k1;    // the unit's key tiles
    int off, cnt;  // the part of them done here: [k0 + off, k0 + off + cnt)
    Keys keys;
};

template <int M, int KT>
__device__ __forceinline__ void walk_enter(const AttnP& p, Walk& w, int64_t pos) {
    const int len = w.k1 - w.k0;
    w.cnt = (int)(w.left < (int64_t)(len - w.off) ? w.left : (int64_t)(len - w.off));
    w.after = pos + (len - w.off);
}

struct WalkSmem {
    int64_t warp[32];
    int64_t rel;
    int b;
};

// Finds this CTA's piece.  Every thread of the block calls it; false if the
// piece is empty.  `threads` is the block size, a multiple of 32.
template <int M, int KT>
__device__ bool walk_begin(const AttnP& p, Walk& w, WalkSmem& sm, int threads) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, nw = threads >> 5;
    int64_t first = 0, mine = 0;
    for (int b = tid; b < p.num_seqs; b += threads) {
        const int64_t c = seq_tiles<M, KT>(p, load_seq(p, b));
        if (b == tid) first = c;
        mine += c;
    }
    int64_t tot = group_sum<32>(mine);
    if (lane == 0) sm.warp[wid] = tot;
    __syncthreads();
    tot = 0;
    for (int i = 0; i < nw; ++i) tot += sm.warp[i];
    const int64_t total = tot * p.hk;
    int64_t per = (total + gridDim.x - 1) / gridDim.x;
    if (per < p.min_per) per = p.min_per;
    const int64_t start = per * blockIdx.x;
    if (start >= total) return false;
    w.per = per;
    w.left = total - start < per ? total - start : per;
    int64_t base = 0;
    for (int b0 = 0; b0 < p.num_seqs; b0 += threads) {
        const int b = b0 + tid;
        int64_t c = 0;
        if (b0 == 0) {
            c = first;
        } else if (b < p.num_seqs) {
            c = seq_tiles<M, KT>(p, load_seq(p, b));
        }
        int64_t inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        __syncthreads();  // sm.warp's readers of the round before are done
        if (lane == 31) sm.warp[wid] = inc;
        if (tid == 0) sm.b = -1;
        __syncthreads();
        int64_t before = base, all = 0;
        for (int i = 0; i < nw; ++i) {
            if (i < wid) before += sm.warp[i];
            all += sm.warp[i];
        }
        const int64_t hi = (before + inc) * p.hk, lo = (before + inc - c) * p.hk;
        if (lo <= start && start < hi) {
            sm.b = b;
            sm.rel = start - lo;
        }
        __syncthreads();
        if (sm.b >= 0) break;
        base += all;
    }
    w.b = sm.b;
    int64_t rel = sm.rel;
    w.s = load_seq(p, w.b);
    const int64_t per_head = seq_tiles<M, KT>(p, w.s);
    w.h = (int)(rel / per_head);
    rel -= w.h * per_head;
    w.rt = 0;
    for (;;) {
        w.keys = tile_range<M, KT>(p, w.s, w.rt, w.k0, w.k1);
        if (rel < w.k1 - w.k0) break;
        rel -= w.k1 - w.k0;
        ++w.rt;
    }
    w.off = (int)rel;
    walk_enter<M, KT>(p, w, start);
    return true;
}

// The next unit; false at the end of the piece.
template <int M, int KT>
__device__ bool walk_next(const AttnP& p, Walk& w) {
    w.left -= w.cnt;
    if (w.left <= 0) return false;
    if ((++w.rt) * M >= w.s.n * p.G) {
        w.rt = 0;
        if (++w.h == p.hk) {
            w.h = 0;
            do {
                w.s = load_seq(p, ++w.b);
            } while (w.s.n == 0);
        }
    }
    w.keys = tile_range<M, KT>(p, w.s, w.rt, w.k0, w.k1);
    w.off = 0;
    walk_enter<M, KT>(p, w, w.after);
    return true;
}

// Where this CTA's part of the unit goes: -1 the output itself, else the
// partial slot.
__device__ __forceinline__ int walk_slot(const Walk& w) {
    if (w.cnt == w.k1 - w.k0) return -1;
    return w.off == 0 ? 1 : 0;
}

// The partial record of (cta, slot): M * D outputs, M maxima, M sums.
template <int M>
__device__ __forceinline__ float* part_of(const AttnP& p, int cta, int slot) {
    return p.part + ((int64_t)cta * 2 + slot) * (M * (int64_t)p.D + 2 * M);
}

// Names the unit of slot 1 and the last CTA that holds a piece of it (called
// by one thread).
__device__ __forceinline__ void write_desc(const AttnP& p, const Walk& w) {
    p.desc[blockIdx.x] = make_int4(w.b, w.h, w.rt, (int)((w.after - 1) / w.per));
}

// Row r (of the sequence's packed rows) -> element offset of its output row.
__device__ __forceinline__ int64_t out_row(const AttnP& p, const Seq& s, int h, int r) {
    const int tok = (int)fast_div((uint32_t)r, p.gdiv);
    return ((int64_t)(s.q0 + tok) * p.hq + h * p.G + (r - tok * p.G));
}

__device__ __forceinline__ float ex2(float x) { return exp2f(x); }

template <int N>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

constexpr float kLn2 = 0.6931471805599453f;

// Natural log of the row's sum of exponentials from its base-2 maximum and sum.
__device__ __forceinline__ float row_lse(float m, float l) {
    return l > 0.0f ? (m + log2f(l)) * kLn2 : (l == 0.0f ? -INFINITY : l);
}

template <typename T>
__device__ __forceinline__ void store_one(const AttnP& p, int64_t e, float y) {
    if (p.out_fp8) {
        reinterpret_cast<uint8_t*>(p.out)[e] = quantize1(y, p.inv);
    } else {
        reinterpret_cast<T*>(p.out)[e] = from_f<T>(y);
    }
}

// A path of the operator: its rows per unit and its grid (CTAs that are resident
// together, so that no piece waits for another's end).
enum AttnPath { kPathAny = 0, kPathFew = 1, kPathMore = 2 };
struct AttnShape {
    AttnPath path;
    int M;
    int ctas;
};

// The 16-bit tile kernels (paged_attn_mma.cu): head sizes that are a multiple of
// 8, 16-byte aligned tensors.
AttnShape mma_shape(AttnPath path, int dt, int head_dim);
cudaError_t launch_attn_mma(const AttnP& p, const AttnShape& sh, int dt, cudaLaunchConfig_t cfg);

}  // namespace edge
