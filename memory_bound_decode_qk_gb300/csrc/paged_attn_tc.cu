// paged_attn_tc.cu -- paged attention of 16-bit chunks with many query rows per
// key head, on the 5th-generation tensor cores (sm_103a).
//
// Work per key tile (128 keys) and query tile (128 packed rows of one key head):
// S = Q K^T and O += P V, 4 * 128 * 128 * D flops, against 128 * 128
// exponentials, so the kernel is bound by the matrix pipe if the softmax of one
// tile runs under the products of another.  Two forms, by what TMEM's 512
// columns hold:
//   heads to 128 channels: a unit is two query tiles, S0 | S1 | O0 | O1.  A key
//     tile is fetched once for 256 rows, and the products alternate,
//     PV0 S0' PV1 S1': while a tile's softmax runs the pipe works for the other.
//   heads to 256 channels: a unit is one query tile, S | S' | O (256 columns).
//     The scores of the next key tile are computed ahead, S' PV S'' PV', so the
//     softmax of one key tile runs under the products of its neighbours.
// Roles of the warps:
//   warp 0        copies keys and values by TMA into a ring in shared memory
//   warp 1        issues tcgen05.mma (one thread)
//   warps 2, 3    values at the edges of what the rows see (below)
//   warps 4-7     softmax, a thread per row;  warps 8-11: of the second tile
// P goes back to TMEM over S as 16-bit values and is the A operand of the
// second product.
//
// Measured on GB300: two chunks of 1024 tokens over 16384 keys, 32/8 heads of 128,
// 533 GFLOP: 334 us as one launch (1595 TFLOP/s, matrix pipe busy 75%), 436 us back
// to back (1220 TFLOP/s; the power limit lowers the clock, 1.77 GHz in the middle
// of four seconds of it against 2.07).  Four prompts of 1201 to 5003 tokens with a
// window of 1024, 16/8 heads of 256, 213 GFLOP seen: 362 us (588 TFLOP/s at 2.07
// GHz), bound by the fetches of key tiles for 128 rows only and by shared-memory
// operands.
//
// Pages.  The cache is a 3-d tensor (channel, head, slot) to TMA; a page (or 128
// rows of it) is one box per 64 channels, stored with the 128-byte swizzle.  A
// page outside the pool or outside the keys that the unit sees is copied from
// behind the tensor's end, which fills zeros.  A page that is seen in part
// brings rows that no query may touch, and rows that only some see: warps 2
// and 3 zero the first before the tile is used, and in the second every infinity
// and NaN, since 0 * NaN is NaN in a matrix product.  If they found any, the
// rows that see such a key add its infinities and NaN at the unit's end (its
// weight is positive, so they reach the sum as they are).  Only the keys that
// some rows of the unit see and others do not are searched for that, at most two
// for each of its tokens, so the time it takes does not depend on how long the
// context is.
//
// Every wait has a limit of two seconds.  A wait that runs out (which correct
// operation never does) ends all later waits of the CTA at once and makes its
// rows NaN.
#include "paged_common.cuh"
#include "tc_common.cuh"

namespace edge {
namespace {

constexpr int kTile = 128;  // query rows of a tile, and keys of a tile

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar,
                                         uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(lead)
        : "memory");
}

// 16 bytes from global to shared memory, asynchronously; zeros if !ok.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ---------------------------------------------------------------- tcgen05

// d[128, N] (+)= A B, both operands in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
        : "memory");
}
// The same with A in TMEM.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
        : "memory");
}

// Instruction descriptor: fp32 accumulator, A and B of type T, M = 128, N = n;
// bmn: B runs along n.
template <typename T>
constexpr __host__ __device__ uint32_t instr_desc(int n, int bmn) {
    const uint32_t f = std::is_same<T, __half>::value ? 0u : 1u;
    return (1u << 4) | (f << 7) | (f << 10) | ((uint32_t)bmn << 16) | ((uint32_t)(n / 8) << 17) | ((uint32_t)(kTile / 16) << 24);
}

// Byte offset of channel chunk c (16 bytes) of row r in a tile of R rows, stored
// as panels of 64 channels with the 128-byte swizzle.
template <int R>
__device__ __forceinline__ uint32_t panel_at(int r, int c) {
    return (uint32_t)((c >> 3) * (R * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
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

// Bits 15 and 31 are set where the exponent of the pair's value is all ones (an
// infinity or NaN): the exponent field plus one at its lowest bit carries there.
template <typename T>
__device__ __forceinline__ uint32_t exponent_bits(uint32_t w) {
    return std::is_same<T, __half>::value ? (w & 0x7C007C00u) + 0x04000400u : (w & 0x7F807F80u) + 0x00800080u;
}

// A pair with its infinities and NaN replaced by zero.
template <typename T>
__device__ __forceinline__ uint32_t bounded(uint32_t w) {
    return w & ~(((exponent_bits<T>(w) >> 15) & 0x00010001u) * 0xFFFFu);
}

// The lowest n bits (n clamped to 0 .. 32).
__device__ __forceinline__ uint32_t bits_below(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// ---------------------------------------------------------------- the kernel

template <int DP>
struct Tc {
    static constexpr int kNQ = DP <= 128 ? 2 : 1;       // query tiles of a unit
    static constexpr int kM = kNQ * kTile;
    // A unit's start and end, in key tiles.  Measured on GB300 over 20 batches for
    // each form (1 to 16 prompts or chunks of 200 to 16,000 keys, with and without
    // windows, five head shapes): with 2, 3, 4, 5, 6 and 8 the geometric mean of
    // the times is 1.08, 1.05, 1.03, 1.03, 1.016 and 1.034 of each batch's best
    // (one query tile), and 1.09, 1.06, 1.03, 1.03, 1.016 and 1.020 (two).  A
    // single batch moves by up to 20% with where the cuts happen to fall.
    static constexpr int kUC = 6;
    // a ring entry: 128 keys and CW channels of them.  Wide heads are cut by
    // channels, not by keys: 64-key operands made the pipe read Q twice as often
    // from shared memory, whose bandwidth then bound it (3100 cycles a tile).
    static constexpr int kCW = DP == 192 ? 64 : DP <= 128 ? DP : 128;
    static constexpr int kParts = DP / kCW;             // entries of a key tile
    static constexpr int kStages = DP == 64 ? 8 : DP == 192 ? 10 : 5;
    static constexpr int kPanels = kCW / 64;            // of an entry
    static constexpr int kQPanels = DP / 64;
    static constexpr int kQ = kTile * DP * 2;           // bytes of a query tile
    static constexpr int kBytes = kTile * kCW * 2;      // bytes of an entry
    static constexpr int kSmem = kNQ * kQ + kStages * kBytes + 1024;
    static constexpr int kThreads = 128 + 128 * kNQ;
};

struct TcSmem {
    uint64_t full[10], empty[10], edge[10];
    uint64_t q_full[2], s_full[2], p_half[2], p_full[2], o_full[2];
    uint32_t tmem;
    uint32_t failed;
    // the last unit, counted from 1, with infinities or NaN taken out of its values
    uint32_t taken;
};

// The tiles [a, b) of the unit's part (relative to its first tile) of which query
// tile i sees anything.
template <int NQ>
__device__ __forceinline__ void tile_span(const AttnP& p, const Walk& w, int i, int& a, int& b) {
    const int t0 = w.k0 + w.off;
    const Keys k = tile_keys<kTile>(p, w.s, w.rt * NQ + i);
    a = max(k.lo / kTile - t0, 0);
    b = min((k.hi + kTile - 1) / kTile - t0, w.cnt);
    if ((w.rt * NQ + i) * kTile >= w.s.n * p.G || b < a) b = a;
}

// Whether the n keys from j on hold some that not every row of the unit sees.
__device__ __forceinline__ bool is_edge(const Walk& w, int j, int n) {
    return j < w.keys.flo || j + n > w.keys.fhi;
}

// The ring positions (in key tiles, from the unit's first) of the keys and the
// values of tile t of cnt: the order in which the products take them, K0 V0 K1
// V1 .. with two query tiles, K0 K1 V0 K2 V1 .. with one.
template <int NQ>
__device__ __forceinline__ uint32_t value_place(int t, int cnt) {
    return NQ == 2 || t + 1 == cnt ? 2 * t + 1 : 2 * t + 2;
}

// Adds the infinities and NaN of the values of keys [first, behind) that the
// thread's row sees, [from, upto), to its outputs o of channels ch .. ch + 31.  All
// lanes of the warp call it with the same first, behind and ch: a lane looks at
// every 32nd key, and all take what a lane has found.
template <typename T>
__device__ __forceinline__ void add_unbounded(const AttnP& p, const Walk& w, int first, int behind, int from, int upto,
                                              int ch, uint32_t (&o)[32]) {
    const int lane = threadIdx.x & 31;
    for (int j0 = first; j0 < behind; j0 += 32) {
        const int64_t slot = j0 + lane < behind ? key_slot(p, w.b, j0 + lane) : -1;
        uint32_t odd = 0;
        if (slot >= 0) {
            const char* v = p.v + ((slot * p.hk + w.h) * p.D + ch) * 2;
            for (int k = 0; k < 32 && ch + k < p.D; k += 8) {
                const uint4 y = __ldg(reinterpret_cast<const uint4*>(v + 2 * k));
                odd |= exponent_bits<T>(y.x) | exponent_bits<T>(y.y) | exponent_bits<T>(y.z) | exponent_bits<T>(y.w);
            }
        }
        uint32_t keys = __ballot_sync(0xffffffffu, (odd & 0x80008000u) != 0);
        for (; keys != 0; keys &= keys - 1) {
            const int src = __ffs(keys) - 1;
            const int64_t at = __shfl_sync(0xffffffffu, slot, src);
            const bool see = j0 + src >= from && j0 + src < upto;
            const T* v = reinterpret_cast<const T*>(p.v) + (at * p.hk + w.h) * p.D + ch;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                const float y = ch + k < p.D ? to_f(v[k]) : 0.0f;
                if (see && !(fabsf(y) < INFINITY)) o[k] = __float_as_uint(__uint_as_float(o[k]) + y);
            }
        }
    }
}

template <typename T, int DP>
__global__ void __launch_bounds__(Tc<DP>::kThreads, 1)
attn_tc_kernel(AttnP p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
               const __grid_constant__ CUtensorMap qmap, int q_boxes) {
    using C = Tc<DP>;
    constexpr int NQ = C::kNQ, M = C::kM, KT = kTile, CW = C::kCW, ST = C::kStages;
    extern __shared__ char raw[];
    __shared__ WalkSmem<1> wsm;
    __shared__ TcSmem sh;
    const int tid = threadIdx.x, lane = tid & 31, wid = uniform(tid >> 5);
    // the swizzle works on address bits: tiles start on 1024 bytes
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    char* tiles = raw + (base - smem_addr(raw));
    const uint32_t ring = base + NQ * C::kQ;

    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) clear_desc(p, blockIdx.x);
    Walk w;
    if (!walk_begin<M, KT, C::kUC, 1>(p, w, wsm, C::kThreads, 0)) return;

    if (wid == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            bar_init(smem_addr(&sh.full[i]), 1);
            bar_init(smem_addr(&sh.empty[i]), 1);
            bar_init(smem_addr(&sh.edge[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_addr(&sh.q_full[i]), q_boxes ? 1 : kTile);
            bar_init(smem_addr(&sh.s_full[i]), 1);
            bar_init(smem_addr(&sh.p_half[i]), kTile);
            bar_init(smem_addr(&sh.p_full[i]), kTile);
            bar_init(smem_addr(&sh.o_full[i]), 1);
        }
        sh.failed = 0;
        sh.taken = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = (uint32_t)uniform((int)sh.tmem);
    volatile uint32_t* failed = &sh.failed;
    // registers with two softmax groups: 128 threads at 88 and 256 at 208 are
    // the launch's 384 at 168
    if (wid < 4) {
        if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (wid == 0) {
            // ---- copies
            const int rows = p.page_size < KT ? p.page_size : KT;  // rows of a box
            const int np = KT / rows;                              // boxes per panel
            const int oob = p.num_pages * p.page_size;             // a slot behind the tensor
            const uint32_t lead = elect_lane();
            uint32_t e = 0;
            int head = 0;
            // the slot of this lane's page of tile t (lane l < np: page l), looked
            // up a tile ahead of its copies
            auto look = [&](int t) {
                const int j = (w.k0 + w.off + t) * KT + lane * rows;
                if (lane < np && j + rows > w.keys.lo && j < w.keys.hi) {
                    const int64_t x = key_slot(p, w.b, j);
                    if (x >= 0) return (int)x;
                }
                return oob;
            };
            auto copy = [&](int t, bool isv, int slot) {
                const bool at_edge = isv && uniform(is_edge(w, (w.k0 + w.off + t) * KT, KT));
#pragma unroll
                for (int h = 0; h < C::kParts; ++h, ++e) {
                    const uint32_t st = e % ST;
                    const uint32_t dst = ring + st * C::kBytes;
                    bar_wait(smem_addr(&sh.empty[st]), ((e / ST) & 1) ^ 1, failed);
                    const uint32_t bar = smem_addr(at_edge ? &sh.edge[st] : &sh.full[st]);
                    bar_expect(bar, C::kBytes, lead);
                    for (int page = 0; page < np; ++page) {
                        const int z = __shfl_sync(0xffffffffu, slot, page);
#pragma unroll
                        for (int panel = 0; panel < C::kPanels; ++panel) {
                            tma_load(dst + panel * (KT * 128) + page * rows * 128, isv ? &vmap : &kmap, h * CW + panel * 64, head,
                                     z, bar, lead);
                        }
                    }
                }
            };
            bool go = true;
            do {
                head = uniform(w.h);
                const int cnt = uniform(w.cnt);
                int now = look(0);
                if constexpr (NQ == 1) copy(0, false, now);
                for (int t = 0; t < cnt; ++t) {
                    const bool more = t + 1 < cnt;
                    int next = now;
                    if (more) next = look(t + 1);
                    if constexpr (NQ == 2) {
                        copy(t, false, now);
                    } else if (more) {
                        copy(t + 1, false, next);
                    }
                    copy(t, true, now);
                    now = next;
                }
                go = uniform(walk_next<M, KT, C::kUC>(p, w));
            } while (go);
        } else if (wid == 1) {
            // ---- products
            {
                const uint32_t lead = elect_lane();
                constexpr uint32_t is = instr_desc<T>(KT, 0), io = instr_desc<T>(CW, 1);
                // descriptors of the first query tile and the first ring entry, as keys
                // and as values; an offset in the tile is added in 16-byte units
                const uint64_t dq = smem_desc(base, 16), dk = smem_desc(ring, 16), dv = smem_desc(ring, KT * 128);
                auto entry = [&](uint32_t e) { return (uint64_t)((e % ST) * (uint32_t)(C::kBytes >> 4)); };
                // S (at column ts of TMEM) of query tile i and the keys of entries e ..
                auto scores = [&](uint32_t ts, int i, uint32_t e) {
#pragma unroll
                    for (int h = 0; h < C::kParts; ++h) {
                        const uint64_t b = dk + entry(e + h);
#pragma unroll 1
                        for (int panel = 0; panel < C::kPanels; ++panel) {
                            const uint32_t qo = (uint32_t)(i * C::kQ + (h * C::kPanels + panel) * (kTile * 128)) >> 4;
                            const uint32_t ko = (uint32_t)(panel * (KT * 128)) >> 4;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                mma_ss(tmem + ts, dq + (qo + k * 2), b + (ko + k * 2), is, h > 0 || k > 0 ? 1u : (uint32_t)(panel > 0), lead);
                            }
                        }
                    }
                };
                // O (at column to) += P (over S) times the values of entries e ..,
                // half of the keys
                auto values = [&](uint32_t to, uint32_t ts, uint32_t e, int half, bool add) {
#pragma unroll
                    for (int h = 0; h < C::kParts; ++h) {
                        const uint64_t b = dv + entry(e + h) + (uint32_t)(half * ((64 * 128) >> 4));
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            mma_ts(tmem + to + h * CW, tmem + ts + half * 32 + k * 8, b + (uint32_t)((k * 16 * 128) >> 4), io,
                                   k > 0 ? 1u : (uint32_t)(add || half > 0), lead);
                        }
                    }
                };
                auto wait_full = [&](uint32_t e) {
#pragma unroll
                    for (int h = 0; h < C::kParts; ++h) bar_wait(smem_addr(&sh.full[(e + h) % ST]), ((e + h) / ST) & 1, failed);
                };
                auto give_back = [&](uint32_t e) {
#pragma unroll
                    for (int h = 0; h < C::kParts; ++h) tc_commit(smem_addr(&sh.empty[(e + h) % ST]), lead);
                };
                uint32_t e = 0, unit[2] = {0, 0}, step[2] = {0, 0};
                bool go = true;
                do {
                    int a[NQ], b[NQ];
#pragma unroll
                    for (int i = 0; i < NQ; ++i) {
                        tile_span<NQ>(p, w, i, a[i], b[i]);
                        a[i] = uniform(a[i]);
                        b[i] = uniform(b[i]);
                    }
                    const int cnt = uniform(w.cnt);
                    for (int t = -1; t < cnt; ++t) {
                        const bool next = t + 1 < cnt;
                        const uint32_t ek = e + C::kParts * (NQ == 2 || t < 0 ? 2 * (t + 1) : 2 * t + 1);
                        const uint32_t ev = e + C::kParts * value_place<NQ>(t, cnt);
                        if constexpr (NQ == 2) {
                            if (t >= 0) wait_full(ev);
                            if (next) wait_full(ek);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                if (t >= a[i] && t < b[i]) {
#pragma unroll 1
                                    for (int half = 0; half < 2; ++half) {
                                        bar_wait(smem_addr(half == 0 ? &sh.p_half[i] : &sh.p_full[i]), step[i] & 1, failed);
                                        tc_after();
                                        values(256 + i * 128, i * 128, ev, half, t > a[i]);
                                    }
                                    ++step[i];
                                    if (t == b[i] - 1) tc_commit(smem_addr(&sh.o_full[i]), lead);
                                }
                                if (t + 1 >= a[i] && t + 1 < b[i]) {
                                    if (t + 1 == a[i]) {
                                        bar_wait(smem_addr(&sh.q_full[i]), unit[i] & 1, failed);
                                        ++unit[i];
                                        tc_after();
                                    }
                                    scores(i * 128, i, ek);
                                    tc_commit(smem_addr(&sh.s_full[i]), lead);
                                }
                            }
                            if (t >= 0) give_back(ev);
                            if (next) give_back(ek);
                        } else {
                            // unit[1] counts the score tiles, step[0] the value tiles
                            if (next) {
                                wait_full(ek);
                                if (t + 1 < b[0]) {
                                    if (t < 0) {
                                        bar_wait(smem_addr(&sh.q_full[0]), unit[0] & 1, failed);
                                        ++unit[0];
                                        tc_after();
                                    }
                                    scores((unit[1] & 1) * 128, 0, ek);
                                    tc_commit(smem_addr(&sh.s_full[unit[1] & 1]), lead);
                                    ++unit[1];
                                }
                                give_back(ek);
                            }
                            if (t >= 0) {
                                wait_full(ev);
                                if (t < b[0]) {
                                    const uint32_t u = step[0]++;
#pragma unroll 1
                                    for (int half = 0; half < 2; ++half) {
                                        bar_wait(smem_addr(&sh.p_full[0]), half, failed);
                                        tc_after();
                                        values(256, (u & 1) * 128, ev, half, t > 0);
                                        tc_commit(smem_addr(&sh.o_full[0]), lead);
                                    }
                                }
                                give_back(ev);
                            }
                        }
                    }
                    e += 2 * C::kParts * cnt;
                    go = uniform(walk_next<M, KT, C::kUC>(p, w));
                } while (go);
            }
        } else {
            // ---- values at an edge (warps 2 and 3, half of the rows each): rows
            // that no query sees become zero, and so do infinities and NaN in rows
            // that some see; the unit's number is noted for those
            uint32_t e = 0, phase = 0, unit = 0;
            do {
                for (int t = 0; t < w.cnt; ++t) {
                    const int j0 = (w.k0 + w.off + t) * KT;
                    if (!is_edge(w, j0, KT)) continue;
                    // rows [0, a) and [d, KT) are nobody's, [a, b) and [c, d) some rows'
                    const int a = min(max(w.keys.lo - j0, 0), KT), d = min(max(w.keys.hi - j0, a), KT);
                    const int b = min(max(w.keys.flo - j0, a), d), c = min(max(w.keys.fhi - j0, b), d);
#pragma unroll 1
                    for (int h = 0; h < C::kParts; ++h) {
                        const uint32_t st = (e + C::kParts * value_place<NQ>(t, w.cnt) + h) % ST;
                        bar_wait(smem_addr(&sh.edge[st]), (phase >> st) & 1, failed);
                        phase ^= 1u << st;
                        char* v = tiles + NQ * C::kQ + st * C::kBytes;
                        constexpr int kRow = CW / 8;  // chunks of a row
                        const int me = tid - 64;
                        uint32_t odd = 0;
                        auto wipe = [&](int from, int to) {
                            for (int i = from * kRow + me; i < to * kRow; i += 64) {
                                *reinterpret_cast<uint4*>(v + panel_at<KT>(i / kRow, i % kRow)) = make_uint4(0u, 0u, 0u, 0u);
                            }
                        };
                        auto scan = [&](int from, int to) {
#pragma unroll 8
                            for (int i = from * kRow + me; i < to * kRow; i += 64) {
                                const uint4 y = *reinterpret_cast<const uint4*>(v + panel_at<KT>(i / kRow, i % kRow));
                                odd |= exponent_bits<T>(y.x) | exponent_bits<T>(y.y) | exponent_bits<T>(y.z) | exponent_bits<T>(y.w);
                            }
                        };
                        auto clean = [&](int from, int to) {
                            for (int i = from * kRow + me; i < to * kRow; i += 64) {
                                uint4* y = reinterpret_cast<uint4*>(v + panel_at<KT>(i / kRow, i % kRow));
                                *y = make_uint4(bounded<T>(y->x), bounded<T>(y->y), bounded<T>(y->z), bounded<T>(y->w));
                            }
                        };
                        wipe(0, a);
                        wipe(d, KT);
                        scan(a, b);
                        scan(c, d);
                        if ((odd & 0x80008000u) != 0) {
                            clean(a, b);
                            clean(c, d);
                        }
                        if (__any_sync(0xffffffffu, (odd & 0x80008000u) != 0) && lane == 0) atomicMax(&sh.taken, unit + 1);
                        fence_async_smem();
                        asm volatile("bar.sync 2, 64;" ::: "memory");
                        if (me == 0) bar_arrive(smem_addr(&sh.full[st]));
                    }
                }
                e += 2 * C::kParts * w.cnt;
                ++unit;
            } while (walk_next<M, KT, C::kUC>(p, w));
        }
    } else {
        if constexpr (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---- softmax of query tile i, a thread per row
        const int i = (wid - 4) >> 2;
        const int row = tid & 127;
        const uint32_t lanes = (uint32_t)(wid & 3) << 21;  // 32 lanes of TMEM per warp
        const uint32_t to = tmem + 256 + i * 128 + lanes;
        char* qt = tiles + i * C::kQ;
        // products given (tiles, or half tiles with one query tile), tiles, units
        uint32_t step = 0, tiles_done = 0, done = 0, unit = 0;
        // this group's queries of a unit into shared memory: one box per 64
        // channels where the heads of the group divide a tile, else row by row
        auto fetch = [&](const Walk& u) {
            const int r0 = u.rt * M + i * kTile;
            if (q_boxes) {
                if (row == 0) {
                    const uint32_t bar = smem_addr(&sh.q_full[i]);
                    const int tok = u.s.q0 + (int)fast_div((uint32_t)r0, p.gdiv);
                    bar_expect(bar, C::kQ, 1);
#pragma unroll
                    for (int panel = 0; panel < C::kQPanels; ++panel) {
                        tma_load(smem_addr(qt) + panel * (kTile * 128), &qmap, panel * 64, u.h * p.G, tok, bar, 1);
                    }
                }
                return;
            }
            const int rows = u.s.n * p.G - r0;
#pragma unroll 4
            for (int x = row; x < kTile * (DP / 8); x += kTile) {
                const int r = x / (DP / 8), c = x % (DP / 8);
                const bool ok = r < rows && c * 8 < p.D;
                const int64_t e = ok ? out_row(p, u.s, u.h, r0 + r) * p.D + c * 8 : 0;
                cp_async16(smem_addr(qt) + panel_at<kTile>(r, c), p.q + e * 2, ok);
            }
        };
        // queries that came row by row are in place
        auto give_queries = [&] {
            if (q_boxes) return;
            cp_async_wait_all();
            fence_async_smem();
            bar_arrive(smem_addr(&sh.q_full[i]));
        };
        int a, b;
        tile_span<NQ>(p, w, i, a, b);
        if (a < b) {
            fetch(w);
            give_queries();
        }
        for (bool go = true; go;) {
            Walk nw = w;
            go = walk_next<M, KT, C::kUC>(p, nw);
            int na = 0, nb = 0;
            if (go) tile_span<NQ>(p, nw, i, na, nb);
            const int r0 = w.rt * M + i * kTile;
            const int rows = min(w.s.n * p.G - r0, kTile);  // may be <= 0
            float ref = -INFINITY, sum = 0.0f;
            const int at = w.s.L - w.s.n + (int)fast_div((uint32_t)(r0 + row), p.gdiv);
            // keys [from, upto) are this row's
            const int upto = p.causal ? min(at + 1, w.s.L) : w.s.L;
            const int from = p.causal && p.window > 0 ? at - p.window + 1 : 0;
            const Keys keys = tile_keys<kTile>(p, w.s, w.rt * NQ + i);
            const int box = p.page_size < kTile ? p.page_size : kTile;
            const int box_shift = 31 - __clz(box);
            // whether this lane's page of tile t is outside the pool, looked up a
            // tile ahead
            auto missing = [&](int t) {
                const int j = (w.k0 + w.off + t) * KT + lane * box;
                return t < b && lane * box < kTile && j < w.s.L && key_slot(p, w.b, j) < 0;
            };
            bool gone = missing(a);
            const uint32_t first_step = step;
            for (int t = a; t < b; ++t) {
                const int j0 = (w.k0 + w.off + t) * KT;
                const uint32_t lost = __ballot_sync(0xffffffffu, gone);
                gone = missing(t + 1);
                // two query tiles: each its own S; one: the two S in turn
                const uint32_t buf = NQ == 2 ? i : tiles_done & 1;
                const uint32_t ts = tmem + buf * 128 + lanes;
                bar_wait(smem_addr(&sh.s_full[buf]), (NQ == 2 ? tiles_done : tiles_done >> 1) & 1, failed);
                tc_after();
                // the last scores of the unit are computed: its queries are done with
                if (t == b - 1 && na < nb) fetch(nw);
                const bool masked = lost || j0 < keys.flo || j0 + KT > keys.fhi;
                // the columns first .. first + 31 that this row sees
                auto seen_of = [&](int first) {
                    uint32_t seen = bits_below(upto - j0 - first) & ~bits_below(from - j0 - first);
                    if (lost) {
                        for (int k = 0; k < 32; k += 8) {  // a page is 8 keys at least
                            if ((lost >> ((first + k) >> box_shift)) & 1u) seen &= ~(0xffu << k);
                        }
                    }
                    return seen;
                };
                if constexpr (NQ == 2) {
                    float s[KT];
#pragma unroll
                    for (int c = 0; c < KT / 32; ++c) tc_ld32(ts + c * 32, reinterpret_cast<uint32_t*>(s) + c * 32);
                    tc_wait_ld();
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < KT / 32; ++c) {
                            const uint32_t seen = seen_of(c * 32);
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                if (!((seen >> k) & 1u)) s[c * 32 + k] = -INFINITY;
                            }
                        }
                    }
                    float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int c = 4; c < KT; c += 4) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) top[k] = fmaxf(top[k], s[c + k]);
                    }
                    const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2;
                    if (t == a) {
                        ref = high;
                    } else if (__any_sync(0xffffffffu, high > ref + 8.0f)) {
                        // lazily: the reference moves only when the weights would
                        // pass 2^8.  The products into O before must be complete:
                        // with two query tiles the commit of S is behind them
                        const float next = fmaxf(ref, high);
                        const float keep = next == -INFINITY ? 1.0f : ex2(ref - next);
                        ref = next;
                        sum *= keep;
#pragma unroll 1
                        for (int c = 0; c < DP / 16; ++c) {
                            uint32_t o[16];
                            tc_ld16(to + c * 16, o);
                            tc_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
                            tc_st16(to + c * 16, o);
                        }
                        tc_wait_st();
                    }
                    const float sub = ref == -INFINITY ? 0.0f : -ref;
                    const float2 f2 = splat2(p.scale_log2), r2 = splat2(sub);
                    float2 acc[2] = {splat2(0.0f), splat2(0.0f)};
#pragma unroll
                    for (int c = 0; c < KT / 32; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float2 x = __ffma2_rn(make_float2(s[c * 32 + 2 * k], s[c * 32 + 2 * k + 1]), f2, r2);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            acc[k & 1] = __fadd2_rn(acc[k & 1], x);
                            pk[k] = pack2<T>(x.x, x.y);
                        }
                        tc_st16(ts + c * 16, pk);
                        if (c & 1) {
                            // half of the weights: their product runs under the
                            // other half's exponentials.  A barrier for each
                            // half, since one warp may be a half ahead
                            tc_wait_st();
                            tc_before();
                            bar_arrive(smem_addr(c == 1 ? &sh.p_half[i] : &sh.p_full[i]));
                        }
                    }
                    sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                    ++step;
                } else {
                    // Half of the tile at a time, so that the product with the first
                    // 64 values runs under the second half's exponentials.  One pass
                    // with the reference as it is; only where a row's maximum passes
                    // it by more than 2^8 (or it is the unit's first half) is the
                    // reference moved, O rescaled and the half done again: the result
                    // carries the same factor in numerator and sum.  The code is kept
                    // short: a form unrolled over all 128 columns outgrew the
                    // instruction cache beside the other roles, and the same
                    // arithmetic took two to three times as long.
#pragma unroll 1
                    for (int half = 0; half < 2; ++half, ++step) {
                        uint32_t x[64], pk[32];
                        tc_ld32(ts + half * 64, x);
                        tc_ld32(ts + half * 64 + 32, x + 32);
                        tc_wait_ld();
                        if (masked) {
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const uint32_t seen = seen_of(half * 64 + c * 32);
#pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    if (!((seen >> k) & 1u)) x[c * 32 + k] = __float_as_uint(-INFINITY);
                                }
                            }
                        }
                        float2 acc[2];
                        bool early = step != first_step;
                        for (;;) {
                            const float2 f2 = splat2(p.scale_log2), r2 = splat2(ref == -INFINITY ? 0.0f : -ref);
                            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                            acc[0] = splat2(0.0f);
                            acc[1] = splat2(0.0f);
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                const float2 s2 = make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
                                top[k & 3] = fmaxf(top[k & 3], fmaxf(s2.x, s2.y));
                                float2 y = __ffma2_rn(s2, f2, r2);
                                y.x = ex2(y.x);
                                y.y = ex2(y.y);
                                acc[k & 1] = __fadd2_rn(acc[k & 1], y);
                                pk[k] = pack2<T>(y.x, y.y);
                            }
                            if (early) {
                                // the product before is complete (every phase of the
                                // barrier is waited for, so a parity names one phase)
                                bar_wait(smem_addr(&sh.o_full[i]), (step - 1) & 1, failed);
                                tc_after();
                                early = false;
                            }
                            const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2;
                            if (!__any_sync(0xffffffffu, high > ref + 8.0f)) break;
                            const float next = fmaxf(ref, high);
                            const float keep = next == -INFINITY ? 1.0f : ex2(ref - next);
                            ref = next;
                            sum *= keep;
                            if (step != first_step) {
#pragma unroll 1
                                for (int c = 0; c < DP / 16; ++c) {
                                    uint32_t o[16];
                                    tc_ld16(to + c * 16, o);
                                    tc_wait_ld();
#pragma unroll
                                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
                                    tc_st16(to + c * 16, o);
                                }
                            }
                        }
                        sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                        // over scores that are read: the halves' weights lie in the
                        // first half's columns
                        tc_st32(ts + half * 32, pk);
                        tc_wait_st();
                        tc_before();
                        bar_arrive(smem_addr(&sh.p_full[i]));
                    }
                }
                ++tiles_done;
            }
            // ---- the unit's end
            if (a < b) {
                bar_wait(smem_addr(&sh.o_full[i]), (NQ == 2 ? done++ : step - 1) & 1, failed);
                tc_after();
            } else if (na < nb) {
                fetch(nw);
            }
            // the next unit's scores may start (they overwrite weights that are used
            // up); its values wait for its weights, which come after this unit's end
            if (na < nb) give_queries();
            if (rows > 0) {
                const bool mine = row < rows;
                // `taken` only grows, and is set before a tile that it speaks of is
                // given to the products: it has reached this unit's number if
                // anything was taken out of its tiles.  These warps may be units
                // ahead or behind the edge warps; if it has passed the number for
                // the sake of a later unit, the search finds nothing to add
                const bool again = a < b && *(volatile uint32_t*)&sh.taken > unit;
                const int slot = walk_slot(w);
                const float nan = *failed ? NAN : 0.0f;
                float* part = slot < 0 ? nullptr : part_of<M>(p, w.piece, slot);
                const int64_t orow = mine ? out_row(p, w.s, w.h, r0 + row) : 0;
                const float scale = (part != nullptr ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum) + nan;
#pragma unroll 1
                for (int c = 0; c < DP / 32; ++c) {
                    uint32_t o[32];
                    if (a < b) {
                        tc_ld32(to + c * 32, o);
                        tc_wait_ld();
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = 0u;
                    }
                    if (again) {
                        // the keys that some rows see: before flo, and from fhi on
                        const int t0 = (w.k0 + w.off + a) * KT, t1 = (w.k0 + w.off + b) * KT;
                        const int end = mine ? upto : 0;
                        add_unbounded<T>(p, w, max(w.keys.lo, t0), min(w.keys.flo, t1), from, end, c * 32, o);
                        add_unbounded<T>(p, w, max(max(w.keys.flo, w.keys.fhi), t0), min(w.keys.hi, t1), from, end, c * 32, o);
                    }
                    if (mine) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8) {
                            const int d = c * 32 + k;
                            if (d >= p.D) continue;
                            float y[8];
#pragma unroll
                            for (int z = 0; z < 8; ++z) y[z] = __uint_as_float(o[k + z]) * scale;
                            if (part != nullptr) {
                                float4* dst = reinterpret_cast<float4*>(part + (int64_t)(i * kTile + row) * p.D + d);
                                dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                                dst[1] = make_float4(y[4], y[5], y[6], y[7]);
                            } else if (p.out_fp8) {
                                *reinterpret_cast<uint2*>(p.out + orow * p.D + d) = quantize_vec<8>(y, p.inv);
                            } else {
                                *reinterpret_cast<uint4*>(p.out + (orow * p.D + d) * 2) = pack_vec<T, 8>(y);
                            }
                        }
                    }
                }
                if (mine && part != nullptr) {
                    part[(int64_t)M * p.D + (i * kTile + row)] = ref;
                    part[(int64_t)M * p.D + M + (i * kTile + row)] = sum + nan;
                } else if (mine && p.lse != nullptr) {
                    p.lse[orow] = row_lse(ref, sum) + nan;
                }
                if (slot == 1 && row == 0 && i == 0) write_desc(p, w);
                tc_before();
            }
            ++unit;
            w = nw;
            a = na;
            b = nb;
        }
    }
    tc_before();
    __syncthreads();
    if (*failed) {
        // copies that nobody waited for end before the shared memory is given up
        for (const uint64_t t0 = now_ns(); now_ns() - t0 < 1000000ull;) {
        }
        __syncthreads();
    }
    if (wid == 1) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ---------------------------------------------------------------- launch

bool query_map(CUtensorMap* map, const AttnP& p, int dt) {
    const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.hq, (cuuint64_t)p.tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)p.D * 2, (cuuint64_t)p.hq * p.D * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(kTile / p.G)};
    const cuuint32_t ones[3] = {1, 1, 1};
    return encoder()(map, dt == kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                     const_cast<char*>(p.q), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool cache_map(CUtensorMap* map, const AttnP& p, const char* base, int dt) {
    const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.hk, (cuuint64_t)p.num_pages * p.page_size};
    const cuuint64_t strides[2] = {(cuuint64_t)p.D * 2, (cuuint64_t)p.hk * p.D * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)(p.page_size < kTile ? p.page_size : kTile)};
    const cuuint32_t ones[3] = {1, 1, 1};
    return encoder()(map, dt == kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                     const_cast<char*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DP>
cudaError_t launch_typed(const AttnP& p, const CUtensorMap (&m)[3], int q_boxes, cudaLaunchConfig_t cfg) {
    const cudaError_t e = allow_smem((const void*)attn_tc_kernel<T, DP>, Tc<DP>::kSmem);
    if (e != cudaSuccess) return e;
    cfg.blockDim = dim3(Tc<DP>::kThreads);
    cfg.dynamicSmemBytes = Tc<DP>::kSmem;
    return cudaLaunchKernelEx(&cfg, attn_tc_kernel<T, DP>, p, m[0], m[1], m[2], q_boxes);
}

}  // namespace

AttnShape tc_shape(int head_dim) {
    const bool wide = head_dim > 128;
    return AttnShape{kPathMany, wide ? Tc<256>::kM : Tc<128>::kM, kTile, wide ? Tc<256>::kUC : Tc<128>::kUC, sm_count(), 1};
}

// 16-byte aligned 16-bit tensors of heads of at least 64 channels (a multiple of
// 8); pages of 8, 16, 32, 64 or a multiple of 128 tokens, so that a ring entry
// is made of whole boxes of at least one swizzle atom; at most 4 million sequences,
// since a walk over empty ones (100 cycles each at most, while other warps of the
// CTA wait for this one) has to end well within the waits' limit.
constexpr int kMaxSeqs = 1 << 22;
bool tc_suits(const AttnP& p) {
    const bool page = p.page_size % kTile == 0 || (p.page_size >= 8 && p.page_size < kTile && kTile % p.page_size == 0);
    return page && p.D >= 64 && p.num_pages > 0 && p.num_seqs <= kMaxSeqs &&
           (int64_t)p.num_pages * p.page_size <= (int64_t)INT32_MAX - kTile && encoder() != nullptr;
}

template <typename T>
cudaError_t launch_by_size(const AttnP& p, const CUtensorMap (&m)[3], int q_boxes, cudaLaunchConfig_t cfg) {
    if (p.D <= 64) return launch_typed<T, 64>(p, m, q_boxes, cfg);
    if (p.D <= 128) return launch_typed<T, 128>(p, m, q_boxes, cfg);
    if (p.D <= 192) return launch_typed<T, 192>(p, m, q_boxes, cfg);
    return launch_typed<T, 256>(p, m, q_boxes, cfg);
}

cudaError_t launch_attn_tc(const AttnP& p, int dt, cudaLaunchConfig_t cfg) {
    CUtensorMap m[3];
    const int q_boxes = kTile % p.G == 0;
    if (!cache_map(&m[0], p, p.k, dt) || !cache_map(&m[1], p, p.v, dt)) return cudaErrorInvalidValue;
    m[2] = m[0];
    if (q_boxes && !query_map(&m[2], p, dt)) return cudaErrorInvalidValue;
    return dt == kF16 ? launch_by_size<__half>(p, m, q_boxes, cfg) : launch_by_size<__nv_bfloat16>(p, m, q_boxes, cfg);
}

}  // namespace edge
