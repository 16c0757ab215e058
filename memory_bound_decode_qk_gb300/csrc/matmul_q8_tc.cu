// matmul_q8_tc.cu -- the 8-bit product on the 5th-generation tensor cores (sm_103a).
//
// A tile is 128 output channels (the rows of the accumulator, so that a thread's
// channel scale is one register) by nt tokens (its columns).  Two forms:
//   one CTA     nt of 16, 32 or 64, for few tokens: E4M3 keeps two CTAs on an SM.  Few
//               tiles are cut along the sum over the CTAs of a cluster, which add
//               their parts through distributed shared memory in a fixed order.
//   a pair      256 channels by up to 256 tokens (int8: 192), each CTA of the pair with
//               128 of the channels and half of the tokens (tcgen05 .cta_group::2):
//               a byte of either operand is fetched for twice as many products.
// Roles of the warps:
//   warp 0      copies both operands by TMA into a ring in shared memory
//   warp 1      issues tcgen05.mma (one thread; of a pair, the first CTA's)
//   warps 4..   scale and store, a thread per channel and all or half of the tokens
//   the last    int8 only: widen the ring's bytes to fp16
// The accumulator is held twice, so the tile that is stored does not stop the next
// one's products.  CTAs are persistent over the tiles.
//
// E4M3 products are the matrix unit's own (kind::f8f6f4).  It has no int8 form on
// this GPU, and the warp-level int8 instruction runs at the rate of the scalar dot
// product (148 TOPS measured).  But every int8 is an fp16 number, a product of two is
// at most 2^14 in size, and fp32 sums of whole numbers are exact up to 2^24: so int8
// operands go through kind::f16 exactly, 1024 terms at a time.  Every 1024 terms the
// accumulator is emptied into int32 registers.  The widened weights go to TMEM, where
// the unit reads them without taking bandwidth from shared memory (which a product of
// few tokens needs whole: 128 rows of 32 bytes took 64 cycles whatever nt was), the
// tokens back to shared memory.
//
// Measured on GB300, back to back: 4096 tokens, 19,456 channels, 2560 terms in E4M3 111 to
// 115 us (3550 to 3670 TFLOP/s), in int8 246 (1657), bound by the matrix pipe and for int8
// the widening beside it; 64 tokens, 2560 channels, 9728 terms 11.0 and 13.3 us (2.3 and 1.9
// TB/s), bound by the launch's beginning, the join and the bytes a CTA has in flight.
//
// Every wait has a limit of two seconds.  A wait that runs out (which correct
// operation never does) ends all later waits of the CTA, and of a pair's other CTA, at
// once and makes their outputs NaN; a cluster that shares a tile reads every flag.
#include <cmath>

#include "matmul_common.cuh"
#include "tc_common.cuh"

namespace edge {
namespace {

constexpr int kRows = 128;  // channels of a CTA's tile
constexpr int kStep = 128;  // terms of a ring entry, the bytes of a swizzled row

// NT: tokens of a tile, for a pair the most.
template <bool INT8, int NT, bool PAIR>
struct Mm {
    static constexpr int kCtas = PAIR || INT8 ? 1 : 2;            // on an SM
    static constexpr int kRoom = (kCtas == 2 ? 110 : PAIR ? 205 : 222) * 1024 - 1024;
    static constexpr int kTokens = PAIR ? NT / 2 : NT;            // of this CTA's part of the operand
    static constexpr int kRaw = (kRows + kTokens) * kStep;        // bytes of a ring entry
    // int8: half an entry (64 terms) widened, the weights in TMEM, the tokens here
    static constexpr int kWides = !INT8 ? 0 : PAIR ? 4 : 8;
    static constexpr int kWide = kTokens * 128;
    static constexpr int kFit = (kRoom - kWides * kWide) / kRaw;
    static constexpr int kStages = kFit < 10 ? kFit : 10;
    static constexpr int kSmem = kStages * kRaw + kWides * kWide + 1024;
    static constexpr int kUnit = INT8 ? 1024 / kStep : 1 << 30;   // entries until a sum is emptied
    // columns of TMEM: two sums, and the widened weights (32 for 64 terms)
    static constexpr int kNeed = 2 * NT + 32 * kWides;
    static constexpr int kColumns = kNeed <= 32 ? 32 : kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
    // warps: 4 for copies and products, those of the sums, groups of 4 that widen
    static constexpr int kSumWarps = PAIR ? 8 : 4;
    static constexpr int kGroups = !INT8 ? 0 : PAIR ? 3 : 4;
    static constexpr int kThreads = 128 + 32 * kSumWarps + 128 * kGroups;
    // int8: registers of the three kinds of warps; together at most the launch's, 768
    // threads at 80
    enum : int { kRegsFew = 40, kRegsSums = PAIR ? 144 : 120, kRegsWide = PAIR ? 48 : 80 };
    static_assert(kStages >= 3 && kStages <= 10 && kNeed <= 512, "the ring or the accumulators do not fit");
    static_assert(PAIR || NT * kRows * 4 <= kSmem - 1024, "a part of a cut tile does not fit");
};

struct MmSmem {
    uint64_t full[10], empty[10];      // the ring
    uint64_t wide[8], narrow[8];       // widened halves of entries: full, empty
    uint64_t sum[2], taken[2];         // accumulators: full, empty
    uint32_t tmem, failed;
};

struct TcP {
    MatmulP m;
    int nt;          // tokens of a tile
    int tiles_n, tiles_t;
    int split;       // one CTA: CTAs of a cluster that share a tile
    int pairs;       // 16-bit outputs whose channel pairs start on 4 bytes
    int whole;       // and fours of channels on 8
};

// Tiles in groups of 16 token tiles, the token tile running fastest: a wave's
// operands stay in L2.
__device__ __forceinline__ void tile_at(const TcP& p, int i, int& tn, int& tt) {
    const int per = 16 * p.tiles_n, group = i / per, first = group * 16;
    const int wide = min(16, p.tiles_t - first), at = i - group * per;
    tn = at / wide;
    tt = first + at - tn * wide;
}

// ---------------------------------------------------------------- instructions

// d (+)= A B: E4M3 with A in shared memory, fp16 with A in TMEM.
template <bool INT8, bool PAIR>
__device__ __forceinline__ void mma_8bit(uint32_t d, uint64_t a, uint32_t ta, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
    if constexpr (INT8 && PAIR) {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(ta), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
            : "memory");
    } else if constexpr (INT8) {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(ta), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
            : "memory");
    } else if constexpr (PAIR) {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
            : "memory");
    }
}
// Arrives, once every product issued before is complete, on the barrier: of a pair, on
// that of both CTAs.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t lead) {
    if constexpr (PAIR) {
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}" ::"r"(bar),
            "r"(lead), "h"((uint16_t)3)
            : "memory");
    } else {
        tc_commit(bar, lead);
    }
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar), "r"(lead)
        : "memory");
}
// The same to this CTA's shared memory, with the barrier of either CTA of the pair.
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

// Arrives on a barrier of any CTA of the cluster.  The default scope, the CTA, is enough
// because no thread of the other CTA reads memory of this one on the strength of it: what it
// announces stays in the SM that made it.  The widened halves lie in this CTA's own shared
// and tensor memory, where the pair's products read them, complete (tcgen05.wait::st, the
// proxy fence) before the arrival is issued; an emptied sum is in registers (wait::ld).  A
// failure is fenced by itself (fail_pair).  Measured with release at the cluster's scope: about
// 2000 cycles for each arrival.
__device__ __forceinline__ void cluster_bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

__device__ __forceinline__ uint4 lds_vector(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts_vector(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// ---------------------------------------------------------------- the kernel

template <bool INT8, int NT, bool PAIR>
__global__ void __launch_bounds__(Mm<INT8, NT, PAIR>::kThreads, Mm<INT8, NT, PAIR>::kCtas)
matmul_tc_kernel(TcP p, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap) {
    using C = Mm<INT8, NT, PAIR>;
    constexpr int ST = C::kStages, WD = C::kWides > 0 ? C::kWides : 1, SW = C::kSumWarps;
    constexpr int TILE = PAIR ? 2 * kRows : kRows;
    extern __shared__ char raw[];
    __shared__ MmSmem sh;
    __shared__ __align__(16) float scales[SW][NT / (SW / 4)];  // of a warp's tokens
    // outputs on their way: by half of the tokens, twice, 8 pairs of tokens x 128 channels
    __shared__ __align__(16) uint32_t staged[PAIR ? 2 : 1][2][PAIR ? 8 : 1][PAIR ? kRows : 1];
    const int tid = threadIdx.x, lane = tid & 31, wid = uniform(tid >> 5);
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;  // the swizzle works on address bits
    const uint32_t wides = base, ring = base + C::kWides * C::kWide;
    const int nt = PAIR ? p.nt : NT, part = PAIR ? nt / 2 : NT;  // tokens of the tile, and this CTA's
    const int split = PAIR ? 1 : p.split, cluster = PAIR ? 2 : split;
    const int rank = cluster > 1 ? (int)(blockIdx.x % cluster) : 0;
    const int tiles = p.tiles_n * p.tiles_t;
    const int first = blockIdx.x / cluster, step = gridDim.x / cluster;
    const int entries = (p.m.k + kStep - 1) / kStep;
    const int e0 = PAIR ? 0 : (int)((int64_t)entries * rank / split);
    const int e1 = PAIR ? entries : (int)((int64_t)entries * (rank + 1) / split);
    const int mine_n = PAIR ? rank * kRows : 0;  // this CTA's channels in the tile

    if (wid == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)), "n"(C::kColumns) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)), "n"(C::kColumns) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            bar_init(smem_addr(&sh.full[i]), 1);
            bar_init(smem_addr(&sh.empty[i]), INT8 ? 8 : 1);
        }
        for (int i = 0; i < WD; ++i) {
            bar_init(smem_addr(&sh.wide[i]), PAIR ? 8 : 4);
            bar_init(smem_addr(&sh.narrow[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_addr(&sh.sum[i]), 1);
            bar_init(smem_addr(&sh.taken[i]), PAIR ? 2 * SW : SW);
        }
        sh.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        // the first weights into L2 while the preceding grid drains
        int tn, tt;
        tile_at(p, first, tn, tt);
        for (int e = e0; e < e1 && e < e0 + ST; ++e) tma_prefetch_2d(&wmap, e * kStep, tn * TILE + mine_n);
    }
    tc_before();
    if constexpr (PAIR) {
        cluster_sync();  // both CTAs' barriers are there
    } else {
        __syncthreads();
    }
    tc_after();
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t tmem = (uint32_t)uniform((int)sh.tmem);
    const uint32_t tmem_w = tmem + 2 * NT;  // widened weights
    volatile uint32_t* failed = &sh.failed;

    if (wid < 4) {
        if constexpr (INT8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"((int)C::kRegsFew));
        if (wid == 0) {
            // ---- copies
            const uint32_t lead = elect_lane();
            const uint32_t bytes = (uint32_t)(kRows + part) * kStep;
            uint32_t st = 0, phase = 1;
            for (int i = first; i < tiles; i += step) {
                int tn, tt;
                tile_at(p, i, tn, tt);
                const int y = tn * TILE + mine_n, t = tt * nt + (PAIR ? rank * part : 0);
                for (int e = e0; e < e1; ++e) {
                    const uint32_t dst = ring + st * C::kRaw, bar = smem_addr(&sh.full[st]);
                    bar_wait<PAIR>(smem_addr(&sh.empty[st]), phase, failed);
                    if constexpr (PAIR && !INT8) {
                        // the products wait for both CTAs' operands on the first one's barrier
                        if (rank == 0) bar_expect(bar, 2 * bytes, lead);
                        const uint32_t at = peer_addr(bar, 0);
                        tma_2d_pair(dst, &wmap, e * kStep, y, at, lead);
                        tma_2d_pair(dst + kRows * kStep, &amap, e * kStep, t, at, lead);
                    } else {
                        bar_expect(bar, bytes, lead);
                        tma_2d(dst, &wmap, e * kStep, y, bar, lead);
                        tma_2d(dst + kRows * kStep, &amap, e * kStep, t, bar, lead);
                    }
                    if (++st == ST) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            if constexpr (PAIR && !INT8) {
                // the other CTA's last arrivals on this one's barriers
                for (int i = 0; i < ST; ++i) {
                    bar_wait<PAIR>(smem_addr(&sh.empty[st]), phase, failed);
                    if (++st == ST) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
        } else if (wid == 1 && (!PAIR || rank == 0)) {
            // ---- products
            const uint32_t lead = elect_lane();
            const uint32_t idesc = (1u << 4) | ((uint32_t)(nt / 8) << 17) | ((uint32_t)(TILE / 16) << 24);
            constexpr int DEPTH = INT8 ? WD : ST, HALVES = INT8 ? 2 : 1;
            const uint64_t dw = smem_desc(ring, 16), dt = smem_desc(INT8 ? wides : ring + kRows * kStep, 16);
            constexpr uint32_t BYTES = INT8 ? C::kWide : C::kRaw;
            uint32_t st = 0, phase = 0, unit = 0;
            for (int i = first; i < tiles; i += step) {
                for (int e = e0; e < e1; ++unit) {
                    const uint32_t buf = unit & 1, d = tmem + buf * NT;
                    bar_wait<PAIR>(smem_addr(&sh.taken[buf]), ((unit >> 1) & 1) ^ 1, failed);
                    tc_after();
                    const int end = min(e1, e + C::kUnit);
                    uint32_t more = 0;
                    for (int count = (end - e) * HALVES; count > 0; --count) {
                        bar_wait<PAIR>(smem_addr(INT8 ? &sh.wide[st] : &sh.full[st]), phase, failed);
                        tc_after();
                        const uint64_t at = st * (uint64_t)(BYTES >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            mma_8bit<INT8, PAIR>(d, dw + (at + k * 2), tmem_w + st * 32 + k * 8, dt + (at + k * 2), idesc, k > 0 ? 1u : more, lead);
                        }
                        more = 1;
                        mma_commit<PAIR>(smem_addr(INT8 ? &sh.narrow[st] : &sh.empty[st]), lead);
                        if (++st == DEPTH) {
                            st = 0;
                            phase ^= 1;
                        }
                    }
                    e = end;
                    mma_commit<PAIR>(smem_addr(&sh.sum[buf]), lead);
                }
            }
        }
    } else if (wid < 4 + SW) {
        if constexpr (INT8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"((int)C::kRegsSums));
        // ---- sums: this thread's channel, and all or half of the tokens
        constexpr int H = NT / (SW / 4), CH = 16;
        const int h = nt / (SW / 4);
        const int quad = wid & 3, half = (wid - 4) >> 2;
        const int row = quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + half * h;
        auto release = [&](uint32_t buf) {
            tc_before();
            __syncwarp();
            if (lane != 0) return;
            if constexpr (PAIR) {
                cluster_bar_arrive(peer_addr(smem_addr(&sh.taken[buf]), 0));
            } else {
                bar_arrive(smem_addr(&sh.taken[buf]));
            }
        };
        uint32_t unit = 0, gives = 0;
        for (int i = first; i < tiles; i += step) {
            int tn, tt;
            tile_at(p, i, tn, tt);
            const int ch = tn * TILE + mine_n + row, t0 = tt * nt + half * h;
            const bool mine = ch < p.m.n;
            const float sw = mine ? __ldg(p.m.sw + ch) : 0.0f;
            const float bias = mine && p.m.bias != nullptr ? load_out(p.m.bias, ch, p.m.out_dt) : 0.0f;
            __syncwarp();  // every lane has read the last tile's scales
            for (int c = lane; c < h; c += 32) scales[wid - 4][c] = t0 + c < p.m.tokens ? __ldg(p.m.sa + t0 + c) : 0.0f;
            __syncwarp();
            // the sums of tokens t0 + c ..: to the output, or to this CTA's part of the tile
            auto give = [&](int c, const uint32_t (&v)[CH]) {
                if (split > 1) {
#pragma unroll
                    for (int j = 0; j < CH; ++j) {
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + (uint32_t)(((half * h + c + j) * kRows + row) * 4)), "r"(v[j]) : "memory");
                    }
                    return;
                }
                const float nsw = *failed ? NAN : sw;
                char* dst = p.m.out + ((int64_t)(t0 + c) * p.m.n + ch) * (p.m.out_dt == kF32 ? 4 : 2);
                const int64_t next = (int64_t)p.m.n * (p.m.out_dt == kF32 ? 4 : 2);
                const int count = min(CH, p.m.tokens - t0 - c);
                float sa[CH];
#pragma unroll
                for (int j = 0; j < CH; j += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(&scales[wid - 4][c + j]);
                    sa[j] = x.x;
                    sa[j + 1] = x.y;
                    sa[j + 2] = x.z;
                    sa[j + 3] = x.w;
                }
                auto value = [&](int j) {
                    return scaled(INT8 ? __int2float_rn((int)v[j]) : __uint_as_float(v[j]), sa[j], nsw, bias);
                };
                if (PAIR && p.whole) {
                    // pairs of tokens of a channel to shared memory; from there a warp has
                    // the 128 channels of two tokens, whole lines of the output
                    uint32_t (&at)[PAIR ? 8 : 1][PAIR ? kRows : 1] = staged[half][gives & 1];
                    ++gives;
#pragma unroll
                    for (int j = 0; j < CH; j += 2) {
                        const float x = value(j), y = value(j + 1);
                        at[PAIR ? j / 2 : 0][PAIR ? row : 0] = p.m.out_dt == kF16 ? pack16<__half>(x, y) : pack16<__nv_bfloat16>(x, y);
                    }
                    asm volatile("bar.sync %0, 128;" ::"r"(half + 1) : "memory");
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int pair = quad * 2 + i, t = t0 + c + 2 * pair, first_ch = ch - row + lane * 4;
                        const uint4 x = *reinterpret_cast<const uint4*>(&at[PAIR ? pair : 0][PAIR ? lane * 4 : 0]);
                        char* to = p.m.out + ((int64_t)t * p.m.n + first_ch) * 2;
                        if (first_ch < p.m.n && t < p.m.tokens) {
                            *reinterpret_cast<uint2*>(to) = make_uint2(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.z, x.w, 0x5410));
                        }
                        if (first_ch < p.m.n && t + 1 < p.m.tokens) {
                            *reinterpret_cast<uint2*>(to + next) = make_uint2(__byte_perm(x.x, x.y, 0x7632), __byte_perm(x.z, x.w, 0x7632));
                        }
                    }
                    return;
                }
                if (!PAIR && p.pairs) {
                    // even lanes store token j of their and their neighbour's channel, odd
                    // lanes token j + 1: 4 bytes (16-bit outputs) of two rows at a time
                    dst += (lane & 1) ? next - 2 : 0;
#pragma unroll
                    for (int j = 0; j < CH; j += 2) {
                        const float x = value(j), y = value(j + 1);
                        const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? x : y, 1);
                        const float lo = (lane & 1) ? other : x, hi = (lane & 1) ? y : other;
                        if (mine && j + (lane & 1) < count) {
                            if (p.m.out_dt == kF16) {
                                *reinterpret_cast<__half2*>(dst) = __floats2half2_rn(lo, hi);
                            } else {
                                *reinterpret_cast<__nv_bfloat162*>(dst) = __floats2bfloat162_rn(lo, hi);
                            }
                        }
                        dst += 2 * next;
                    }
                    return;
                }
#pragma unroll
                for (int j = 0; j < CH; ++j) {
                    const float y = value(j);
                    if (mine && j < count) store_out(dst, 0, y, p.m.out_dt);
                    dst += next;
                }
            };
            if constexpr (INT8) {
                uint32_t acc[H];
#pragma unroll
                for (int c = 0; c < H; ++c) acc[c] = 0u;
                for (int e = e0; e < e1; e += C::kUnit, ++unit) {
                    const uint32_t buf = unit & 1;
                    bar_wait<PAIR>(smem_addr(&sh.sum[buf]), (unit >> 1) & 1, failed);
                    tc_after();
                    if constexpr (H >= 32) {
                        // (h is a multiple of 16: the last columns may be those of nobody)
#pragma unroll
                        for (int c = 0; c < H; c += 32) {
                            if (c >= h) continue;
                            uint32_t v[32];
                            tc_ld32(lanes + buf * NT + c, v);
                            tc_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) acc[c + j] += (uint32_t)__float2int_rn(__uint_as_float(v[j]));
                        }
                    } else {
                        uint32_t v[CH];
                        tc_ld16(lanes + buf * NT, v);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < CH; ++j) acc[j] += (uint32_t)__float2int_rn(__uint_as_float(v[j]));
                    }
                    release(buf);
                }
#pragma unroll
                for (int c = 0; c < H; c += CH) {
                    if (c >= h) continue;
                    uint32_t v[CH];
#pragma unroll
                    for (int j = 0; j < CH; ++j) v[j] = acc[c + j];
                    give(c, v);
                }
            } else {
                const uint32_t buf = unit & 1;
                bar_wait<PAIR>(smem_addr(&sh.sum[buf]), (unit >> 1) & 1, failed);
                tc_after();
#pragma unroll 1
                for (int c = 0; c < h; c += CH) {
                    uint32_t v[CH];
                    tc_ld16(lanes + buf * NT + c, v);
                    tc_wait_ld();
                    give(c, v);
                }
                release(buf);
                ++unit;
            }
        }
    } else if constexpr (INT8) {
        if constexpr (C::kRegsWide < 80) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"((int)C::kRegsWide));
        // ---- widening.  Groups of four warps take the halves of the entries in turn.
        // Weights: a thread's row to its lane of TMEM, two numbers to a column.  Tokens: a
        // 16-byte piece of half a row to two of fp16, both with the 128-byte swizzle; eight
        // threads take four pieces of rows r and r + 4, and those of r + 4 store their
        // second piece first, so that loads and stores are free of bank conflicts.
        const int group = (wid - 4 - SW) >> 2, quad = wid & 3, mine = tid & 127;
        const uint32_t wrow = ring + mine * 128, wx = (uint32_t)(mine & 7);
        const uint32_t wlane = tmem_w + ((uint32_t)(quad * 32) << 16);
        const int odd = (mine >> 2) & 1, r = odd * 4 + ((mine >> 3) & 3) + (mine >> 5) * 8, c = mine & 3;
        const uint32_t from = ring + kRows * kStep + r * 128 + ((c ^ (r & 7)) << 4);
        const uint32_t to = wides + r * 128 + (((c * 2 + odd) ^ (r & 7)) << 4);
        const int pieces = part * 4;
        const uint32_t mine_of = first < tiles ? (uint32_t)((tiles - 1 - first) / step + 1) : 0u;  // tiles
        const uint32_t halves = mine_of * 2u * (uint32_t)(e1 - e0);
        uint32_t n = group;
        for (; n < halves; n += C::kGroups) {
            const uint32_t st = (n >> 1) % ST, wd = n % WD;
            bar_wait<PAIR>(smem_addr(&sh.full[st]), ((n >> 1) / ST) & 1, failed);
            bar_wait<PAIR>(smem_addr(&sh.narrow[wd]), ((n / WD) & 1) ^ 1, failed);
            tc_after();
            const uint32_t entry = st * C::kRaw, half = n & 1;
            const uint32_t src = (from + entry) ^ (half << 6), dst = to + wd * C::kWide;
            // every load before the first number is turned
            constexpr int EACH = C::kTokens * 4 / 128 > 0 ? C::kTokens * 4 / 128 : 1;
            uint4 x[4], v[EACH];
#pragma unroll
            for (int b = 0; b < 4; ++b) x[b] = lds_vector(wrow + entry + (((half * 4 + b) ^ wx) << 4));
#pragma unroll
            for (int u = 0; u < EACH; ++u) {
                if (mine + 128 * u < pieces) v[u] = lds_vector(src + u * 4096);
            }
#pragma unroll
            for (int b = 0; b < 4; b += 2) {
                uint32_t o[16];
                widen4(x[b].x, o[0], o[1]);
                widen4(x[b].y, o[2], o[3]);
                widen4(x[b].z, o[4], o[5]);
                widen4(x[b].w, o[6], o[7]);
                widen4(x[b + 1].x, o[8], o[9]);
                widen4(x[b + 1].y, o[10], o[11]);
                widen4(x[b + 1].z, o[12], o[13]);
                widen4(x[b + 1].w, o[14], o[15]);
                tc_st16(wlane + wd * 32 + b * 8, o);
            }
#pragma unroll
            for (int u = 0; u < EACH; ++u) {
                if (mine + 128 * u < pieces) {
                    uint4 lo, hi;
                    widen4(odd ? v[u].z : v[u].x, lo.x, lo.y);
                    widen4(odd ? v[u].w : v[u].y, lo.z, lo.w);
                    widen4(odd ? v[u].x : v[u].z, hi.x, hi.y);
                    widen4(odd ? v[u].y : v[u].w, hi.z, hi.w);
                    sts_vector(dst + u * 4096, lo);
                    sts_vector((dst + u * 4096) ^ 16, hi);
                }
            }
            tc_wait_st();
            tc_before();
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) {
                    cluster_bar_arrive(peer_addr(smem_addr(&sh.wide[wd]), 0));
                } else {
                    bar_arrive(smem_addr(&sh.wide[wd]));
                }
                bar_arrive(smem_addr(&sh.empty[st]));
            }
        }
        if constexpr (PAIR) {
            // the other CTA's last arrivals on this one's barriers
            n = halves;
            for (int i = 0; i < WD; ++i, ++n) bar_wait<PAIR>(smem_addr(&sh.narrow[n % WD]), ((n / WD) & 1) ^ 1, failed);
        }
    }
    tc_before();
    // (one answer for the CTA: the other one of a pair can set the flag at any time)
    if (__syncthreads_or((int)*failed)) {
        // copies that nobody waited for end before the shared memory is given up
        for (const uint64_t t0 = now_ns(); now_ns() - t0 < 1000000ull;) {
        }
        __syncthreads();
    }
    if constexpr (PAIR) cluster_sync();  // products read both CTAs' memory until here
    if (wid == 1) {
        tc_after();
        if constexpr (PAIR) {
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kColumns) : "memory");
        } else {
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kColumns) : "memory");
        }
    }
    if (!PAIR && split > 1) {
        // the parts lie where the ring was, [token][channel]; every product is done
        cluster_sync();
        constexpr int FROM = INT8 ? 4 : 0;  // the warps that have the launch's registers
        if (wid >= FROM) {
            // this CTA's share of the tile's tokens, the parts added in rank order; a lane has
            // four channels of a token, a warp all
            int tn, tt;
            tile_at(p, first, tn, tt);
            const int c0 = NT * rank / split, c1 = min(NT * (rank + 1) / split, p.m.tokens - tt * NT);
            const int ch = tn * kRows + lane * 4;
            float nan = 0.0f;
            for (int r = 0; r < split; ++r) nan = peer_word(peer_addr(smem_addr(&sh.failed), r)) ? NAN : nan;
            for (int c = c0 + (wid - FROM); c < c1; c += C::kThreads / 32 - FROM) {
                uint4 v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    v[r] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < split) v[r] = peer_vector(peer_addr(base + (uint32_t)((c * kRows + lane * 4) * 4), r));
                }
                const float sa = __ldg(p.m.sa + tt * NT + c);
                char* dst = p.m.out + ((int64_t)(tt * NT + c) * p.m.n + ch) * (p.m.out_dt == kF32 ? 4 : 2);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t sum = 0u;
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const uint32_t x = reinterpret_cast<const uint32_t*>(&v[r])[j];
                        sum = INT8 ? sum + x : __float_as_uint(__fadd_rn(__uint_as_float(sum), __uint_as_float(x)));
                    }
                    if (ch + j >= p.m.n) continue;
                    const float y = INT8 ? __int2float_rn((int)sum) : __uint_as_float(sum);
                    const float bias = p.m.bias != nullptr ? load_out(p.m.bias, ch + j, p.m.out_dt) : 0.0f;
                    store_out(dst, j, scaled(y + nan, sa, __ldg(p.m.sw + ch + j), bias), p.m.out_dt);
                }
            }
        }
        cluster_sync();  // peers read this CTA's shared memory until here
    }
}

// ---------------------------------------------------------------- launch

bool operand_map(CUtensorMap* map, const char* base, int rows, int k, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)k};
    const cuuint32_t box[2] = {kStep, (cuuint32_t)box_rows};
    const cuuint32_t ones[2] = {1, 1};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<char*>(base), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a call is cut: tiles of nt tokens by one CTA (split over a cluster) or a pair.
struct Cut {
    bool pair;
    int nt, split;
};

template <bool INT8, int NT, bool PAIR>
cudaError_t launch_tile(const MatmulP& m, const Cut& cut, cudaLaunchConfig_t cfg) {
    using C = Mm<INT8, NT, PAIR>;
    const void* fn = (const void*)matmul_tc_kernel<INT8, NT, PAIR>;
    constexpr int TILE = PAIR ? 2 * kRows : kRows;
    const int nt = cut.nt;
    TcP p;
    p.m = m;
    p.nt = nt;
    p.tiles_n = (m.n + TILE - 1) / TILE;
    p.tiles_t = (m.tokens + nt - 1) / nt;
    p.pairs = m.out_dt != kF32 && m.n % 2 == 0 && reinterpret_cast<uintptr_t>(m.out) % 4 == 0;
    p.whole = m.out_dt != kF32 && m.n % 4 == 0 && reinterpret_cast<uintptr_t>(m.out) % 8 == 0;
    CUtensorMap wmap, amap;
    if (!operand_map(&wmap, m.w, m.n, m.k, kRows) || !operand_map(&amap, m.a, m.tokens, m.k, PAIR ? nt / 2 : nt)) {
        return cudaErrorInvalidValue;
    }
    cudaError_t e = allow_smem(fn, C::kSmem);
    if (e != cudaSuccess) return e;
    if constexpr (INT8) {
        // the registers that the warps ask for have to be there, or they would wait for ever
        constexpr int need = 4 * C::kRegsFew + C::kSumWarps * C::kRegsSums + 4 * C::kGroups * C::kRegsWide;
        int registers = 0;
        e = kernel_registers(fn, &registers);
        if (e != cudaSuccess) return e;
        if (registers * (C::kThreads / 32) < need) return cudaErrorLaunchOutOfResources;
    }
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    const int64_t tiles = (int64_t)p.tiles_n * p.tiles_t;
    int cluster = 2;
    int64_t slots = (int64_t)sm_count() * C::kCtas;
    if constexpr (PAIR) {
        slots = resident_clusters(fn, cfg, 2);
        if (slots < 1) return cudaErrorLaunchOutOfResources;
    } else {
        cluster = cut.split;
        while (cluster > 1 && tiles > resident_clusters(fn, cfg, cluster)) --cluster;
    }
    p.split = PAIR ? 1 : cluster;
    cfg.gridDim = dim3((unsigned)(cluster * (p.split > 1 || tiles < slots ? tiles : slots)));
    if (cluster > 1) {
        cfg.attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        cfg.attrs[cfg.numAttrs].val.clusterDim.x = (unsigned)cluster;
        cfg.attrs[cfg.numAttrs].val.clusterDim.y = 1;
        cfg.attrs[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, matmul_tc_kernel<INT8, NT, PAIR>, p, wmap, amap);
}

// The quickest cut by a model of the times in us, whose numbers are fits to
// measurements on GB300 (back-to-back launches, weights from memory; 1 to 4096 tokens,
// 1024 to 19,456 channels, sums of 1024 to 9728 terms):
//   a ring entry (128 terms)
//     E4M3: the bytes that an SM takes in, 110 to 120 GB/s; a pair's products need 1.13 ns
//     a token
//     int8: widening, 0.35 us (one CTA, 64 tokens 0.44) and 0.47 to 0.55 us (pair)
//   a launch with its first fetch and last store: 2.4 to 5 us and some ns a token
//   the sum over a cluster: 2 us and 30 ns a token
//   a tile among others: no less than its store, 0.4 us and 9 ns a token (one CTA), 1.3 us
//   and 6 ns (pair)
// The time that memory takes for the weights (5.5 TB/s) runs beside the entries, the
// longer of the two and a quarter of the other count.  Over 22 drawn calls of each type its
// choices took 1.02 (E4M3) and 0.99 (int8) times the best of a sweep of up to 20 cuts in
// the geometric mean, at worst 1.16.  Measured around them: 2560 x 9728 in E4M3, 64
// tokens, 11.1 us split over six CTAs against 21.4 unsplit and 17.5 by pairs of 96 tokens;
// 1024 tokens, 20.7 us with pairs of 160 tokens (70 tiles on 76 pairs) against 27.4 with
// 256 (40 tiles) and 29.4 with 128 (80).
template <bool INT8>
Cut choose(const MatmulP& m, bool pairs) {
    const double sms = sm_count();
    const int entries = (m.k + kStep - 1) / kStep;
    const double memory = ((double)m.n * m.k + (double)m.tokens * m.k) / 5.5e6;
    Cut best = {false, 16, 1};
    double least = 1e30;
    auto consider = [&](const Cut& c) {
        const double tile = c.pair ? 2 * kRows : kRows;
        const double tiles = std::ceil(m.n / tile) * std::ceil((double)m.tokens / c.nt);
        const double rounds = std::ceil(tiles * (c.pair ? 2 : c.split) / sms);
        double entry, ends;
        if (INT8) {
            entry = c.pair ? 0.45 + 0.0005 * c.nt : c.nt <= 32 ? 0.35 : 0.44;
            ends = c.pair ? 5.0 + 0.01 * c.nt : 3.6 + 0.02 * c.nt;
        } else {
            entry = c.pair ? std::fmax((kRows + c.nt / 2) * 0.00105, c.nt * 0.00113) : (kRows + c.nt) * 0.00117;
            ends = c.pair ? 3.0 + 0.008 * c.nt : 2.4 + 0.01 * c.nt;
        }
        if (c.split > 1) ends += 2.0 + 0.03 * c.nt;
        double tile_time = std::ceil((double)entries / c.split) * entry;
        if (rounds > 1) tile_time = std::fmax(tile_time, c.pair ? 1.3 + 0.006 * c.nt : 0.4 + 0.009 * c.nt);
        const double work = rounds * tile_time;
        const double t = ends + std::fmax(work, memory) + 0.25 * std::fmin(work, memory);
        if (t < least) {
            least = t;
            best = c;
        }
    };
    for (int nt = 16; nt <= 64; nt *= 2) {
        if (nt > 16 && m.tokens <= nt / 2) break;
        const int64_t tiles = (int64_t)((m.n + kRows - 1) / kRows) * ((m.tokens + nt - 1) / nt);
        for (int split = 1; split <= 8; ++split) {
            // at least 4 entries for each CTA, and all CTAs at once
            if (split > 1 && (split * 4 > entries || tiles * split > (int64_t)sms)) break;
            consider(Cut{false, nt, split});
        }
    }
    for (int nt = 32; pairs && nt <= (INT8 ? 192 : 256); nt += 32) {
        if (m.tokens <= 32 || (nt > 32 && m.tokens <= nt - 32)) break;
        consider(Cut{true, nt, 1});
    }
    return best;
}

template <bool INT8>
cudaError_t launch_kind(const MatmulP& m, cudaLaunchConfig_t cfg) {
    Cut cut = choose<INT8>(m, true);
    if (cut.pair) {
        const cudaError_t e = launch_tile<INT8, INT8 ? 192 : 256, true>(m, cut, cfg);
        // no room for pairs (or none that the runtime knows of just now): single CTAs serve
        // every call
        if (e != cudaErrorLaunchOutOfResources) return e;
        (void)cudaGetLastError();
        cut = choose<INT8>(m, false);
    }
    if (cut.nt == 16) return launch_tile<INT8, 16, false>(m, cut, cfg);
    if (cut.nt == 32) return launch_tile<INT8, 32, false>(m, cut, cfg);
    return launch_tile<INT8, 64, false>(m, cut, cfg);
}

}  // namespace

// Rows and addresses on 16 bytes, which TMA wants; sizes whose tiles a 32-bit number
// counts.
bool matmul_tc_suits(const MatmulP& m) {
    return m.k % 16 == 0 && reinterpret_cast<uintptr_t>(m.a) % 16 == 0 && reinterpret_cast<uintptr_t>(m.w) % 16 == 0 &&
           ((int64_t)m.n + kRows) / kRows * (((int64_t)m.tokens + 31) / 32) < (int64_t(1) << 27) && encoder() != nullptr;
}

cudaError_t launch_matmul_tc(const MatmulP& m, int q_dt, cudaLaunchConfig_t cfg) {
    return q_dt == kInt8 ? launch_kind<true>(m, cfg) : launch_kind<false>(m, cfg);
}

}  // namespace edge
