// paged_common.cuh -- what the paged-attention kernels share: parameters, key
// visibility, the work schedule and the partial results.
//
// Schedule.  A unit is M packed query rows of one sequence and one key head
// (rows are (token, query head of the group), token-major), and its work is a
// run of key tiles of KT keys.  The units stand in one line, each as long as
// its tiles and a constant for its start and end (UC tiles' worth, measured),
// and every worker (a CTA, or a warp) takes an equal piece of it, wherever that
// starts and ends, so a batch of ragged lengths or one long sequence fills the
// GPU alike.  The lengths live on the device, so each CTA finds its pieces
// itself: a block-wide sum over the sequences and a scan up to its own starts.
// A unit that lies in one piece is written directly.  The parts of a unit that
// spans several pieces go to the workspace as (row maximum, row sum,
// unnormalized output) and a second kernel joins them.  At most one unit starts
// in a piece without ending there (partial slot 1), and at most one ends there
// that started earlier (slot 0).
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
    float* part;        // [pieces][2][M * D + 2 M] fp32
    int4* desc;         // [pieces][2]: unit of slot 1: (last piece or < 0, key head, row
                        // tile, -) and (first query row, tokens, -, -) of its sequence
    int num_seqs, max_pages, num_pages, page_size;
    int tokens, hq, hk, G, D;
    FastDiv gdiv, pdiv;  // by G and by page_size
    int causal, window, out_fp8;
    int max_len;        // max_pages * page_size
    int min_per;        // shortest piece, in tiles
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

// a / b of non-negative values, which seldom need 64 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if ((((uint64_t)a | (uint64_t)b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// Length of sequence b's units of one key head in the line.
template <int M, int KT, int UC>
__device__ __forceinline__ int64_t seq_length(const AttnP& p, const Seq& s) {
    int64_t c = 0;
    const int nrt = (s.n * p.G + M - 1) / M;
    for (int rt = 0; rt < nrt; ++rt) {
        int k0, k1;
        tile_range<M, KT>(p, s, rt, k0, k1);
        c += UC + k1 - k0;
    }
    return c;
}

// A worker's walk over its piece of the line.  Every thread of the worker holds
// the same copy.
struct Walk {
    int64_t left;  // length of the piece behind this unit
    int64_t after; // line position at which this unit ends
    int64_t per;   // length of a piece
    int piece;
    int b, h, rt;
    Seq s;
    int k0, k1;    // the unit's key tiles
    int off, cnt;  // the part of them done here: [k0 + off, k0 + off + cnt)
    Keys keys;
};

// Takes the unit (b, h, rt), of which the line position `at` lies `rel` behind
// the start, as far as the piece reaches.  False if that is no tile of it.
template <int M, int KT, int UC>
__device__ __forceinline__ bool walk_enter(const AttnP& p, Walk& w, int64_t at, int64_t rel) {
    w.keys = tile_range<M, KT>(p, w.s, w.rt, w.k0, w.k1);
    const int64_t len = UC + w.k1 - w.k0;
    const int64_t share = w.left < len - rel ? w.left : len - rel;
    w.off = (int)(rel > UC ? rel - UC : 0);
    const int64_t end = rel + share - UC;
    w.cnt = end > w.off ? (int)(end - w.off) : 0;
    w.left -= share;
    w.after = at + len - rel;
    return w.cnt > 0;
}

template <int PP>
struct WalkSmem {
    int64_t warp[32];
    int64_t rel[PP];
    int b[PP];
};

// The unit and tile at `rel` behind the start of sequence w.b's part of the line,
// of which one key head takes per_head.
template <int M, int KT, int UC>
__device__ __forceinline__ bool walk_settle(const AttnP& p, Walk& w, int64_t total, int64_t per, int piece,
                                            int64_t rel, int64_t per_head) {
    const int64_t start = per * piece;
    w.piece = piece;
    w.per = per;
    w.left = total - start < per ? total - start : per;
    w.h = (int)quotient(rel, per_head);
    rel -= w.h * per_head;
    w.rt = 0;
    for (;;) {
        int k0, k1;
        tile_range<M, KT>(p, w.s, w.rt, k0, k1);
        const int len = UC + k1 - k0;
        if (rel < len) break;
        rel -= len;
        ++w.rt;
    }
    return walk_enter<M, KT, UC>(p, w, start, rel);
}

// The line's pieces: equal lengths, at least min_per.
__device__ __forceinline__ int64_t piece_length(const AttnP& p, int64_t total, int pieces) {
    const int64_t per = quotient(total + pieces - 1, pieces);
    return per > p.min_per ? per : p.min_per;
}

// Finds the pieces blockIdx.x + gridDim.x i, i < PP, of this CTA; the calling
// thread's worker takes the one of i = `mine`.  Every thread of the block calls
// it; false if the worker's piece is empty.  `threads` is the block size, a
// multiple of 32.
template <int M, int KT, int UC, int PP>
__device__ bool walk_begin(const AttnP& p, Walk& w, WalkSmem<PP>& sm, int threads, int mine) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, nw = threads >> 5;
    const int pieces = gridDim.x * PP;
    const int piece = blockIdx.x + gridDim.x * mine;
    if (p.num_seqs <= 32) {
        // a lane per sequence: no shared memory, no barrier
        Seq s{0, 0, 0};
        int64_t c = 0;
        if (lane < p.num_seqs) {
            s = load_seq(p, lane);
            c = seq_length<M, KT, UC>(p, s);
        }
        int64_t inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        const int64_t total = __shfl_sync(0xffffffffu, inc, 31) * p.hk;
        const int64_t per = piece_length(p, total, pieces);
        const int64_t start = per * piece;
        if (start >= total) return false;
        const int64_t lo = (inc - c) * p.hk;
        const int from = __ffs(__ballot_sync(0xffffffffu, lo <= start && start < inc * p.hk)) - 1;
        w.b = from;
        w.s.q0 = __shfl_sync(0xffffffffu, s.q0, from);
        w.s.n = __shfl_sync(0xffffffffu, s.n, from);
        w.s.L = __shfl_sync(0xffffffffu, s.L, from);
        const int64_t rel = start - __shfl_sync(0xffffffffu, lo, from);
        return walk_settle<M, KT, UC>(p, w, total, per, piece, rel, __shfl_sync(0xffffffffu, c, from));
    }
    int64_t first = 0, own = 0;
    for (int b = tid; b < p.num_seqs; b += threads) {
        const int64_t c = seq_length<M, KT, UC>(p, load_seq(p, b));
        if (b == tid) first = c;
        own += c;
    }
    int64_t tot = group_sum<32>(own);
    if (lane == 0) sm.warp[wid] = tot;
    if (tid < PP) sm.b[tid] = -1;
    __syncthreads();
    tot = 0;
    for (int i = 0; i < nw; ++i) tot += sm.warp[i];
    const int64_t total = tot * p.hk;
    const int64_t per = piece_length(p, total, pieces);
    const int64_t low = per * blockIdx.x;  // the first of the CTA's pieces
    if (low >= total) return false;
    const int64_t high = per * ((int64_t)blockIdx.x + (int64_t)gridDim.x * (PP - 1));
    int64_t base = 0;
    for (int b0 = 0; b0 < p.num_seqs; b0 += threads) {
        const int b = b0 + tid;
        int64_t c = 0;
        if (b0 == 0) {
            c = first;
        } else if (b < p.num_seqs) {
            c = seq_length<M, KT, UC>(p, load_seq(p, b));
        }
        int64_t inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        __syncthreads();  // the readers of sm.warp before are done
        if (lane == 31) sm.warp[wid] = inc;
        __syncthreads();
        int64_t before = base, all = 0;
        for (int i = 0; i < nw; ++i) {
            if (i < wid) before += sm.warp[i];
            all += sm.warp[i];
        }
        const int64_t hi = (before + inc) * p.hk, lo = (before + inc - c) * p.hk;
#pragma unroll
        for (int i = 0; i < PP; ++i) {
            const int64_t start = low + per * gridDim.x * i;
            if (lo <= start && start < hi) {
                sm.b[i] = b;
                sm.rel[i] = start - lo;
            }
        }
        base += all;
        if (base * p.hk > high) break;
    }
    __syncthreads();
    w.b = sm.b[mine];
    if (w.b < 0) return false;
    w.s = load_seq(p, w.b);
    return walk_settle<M, KT, UC>(p, w, total, per, piece, sm.rel[mine], seq_length<M, KT, UC>(p, w.s));
}

// The next unit; false at the end of the piece.
template <int M, int KT, int UC>
__device__ bool walk_next(const AttnP& p, Walk& w) {
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
    return walk_enter<M, KT, UC>(p, w, w.after, 0);
}

// Where the worker's part of the unit goes: -1 the output itself, else the
// partial slot.
__device__ __forceinline__ int walk_slot(const Walk& w) {
    if (w.cnt == w.k1 - w.k0) return -1;
    return w.off == 0 ? 1 : 0;
}

// The partial record of (piece, slot): M * D outputs, M maxima, M sums.
template <int M>
__device__ __forceinline__ float* part_of(const AttnP& p, int piece, int slot) {
    return p.part + ((int64_t)piece * 2 + slot) * (M * (int64_t)p.D + 2 * M);
}

// Names the unit of slot 1 and the last piece that holds a part of it (called
// by one thread).
__device__ __forceinline__ void write_desc(const AttnP& p, const Walk& w) {
    p.desc[2 * w.piece] = make_int4((int)quotient(w.after - 1, w.per), w.h, w.rt, 0);
    p.desc[2 * w.piece + 1] = make_int4(w.s.q0, w.s.n, 0, 0);
}
__device__ __forceinline__ void clear_desc(const AttnP& p, int piece) {
    p.desc[2 * piece] = make_int4(-1, 0, 0, 0);
}

// Row r (of the sequence's packed rows) -> element offset of its output row.
__device__ __forceinline__ int64_t out_row(const AttnP& p, const Seq& s, int h, int r) {
    const int tok = (int)fast_div((uint32_t)r, p.gdiv);
    return ((int64_t)(s.q0 + tok) * p.hq + h * p.G + (r - tok * p.G));
}

// 2^x by the hardware's approximation (relative error about 2^-22, results
// below the normal range flushed to zero).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

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

// A path of the operator: rows of a unit, keys of a tile, a unit's constant in the
// line, its grid (CTAs that are resident together) and the pieces each takes.
enum AttnPath { kPathAny = 0, kPathFew = 1, kPathMore = 2, kPathMany = 3 };
struct AttnShape {
    AttnPath path;
    int M, KT, UC;
    int ctas;
    int per_cta;
};

// The 16-bit tile kernels (paged_attn_mma.cu): head sizes that are a multiple of
// 8, 16-byte aligned tensors.
AttnShape mma_shape(AttnPath path, int dt, int head_dim);
cudaError_t launch_attn_mma(const AttnP& p, const AttnShape& sh, int dt, cudaLaunchConfig_t cfg);

// The tcgen05 kernel (paged_attn_tc.cu), where tc_suits says that it serves the
// head and page size.
AttnShape tc_shape(int head_dim);
bool tc_suits(const AttnP& p);
cudaError_t launch_attn_tc(const AttnP& p, int dt, cudaLaunchConfig_t cfg);

}  // namespace edge
