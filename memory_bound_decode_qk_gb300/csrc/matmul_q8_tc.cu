// matmul_q8_tc.cu -- the 8-bit product on the 5th-generation tensor cores (sm_103a).
//
// A tile is 128 output channels (the rows of the accumulator, so that a thread's
// channel scale is one register) by NT tokens (its columns).  Roles of the warps:
//   warp 0        copies both operands by TMA into a ring in shared memory
//   warp 1        issues tcgen05.mma (one thread)
//   warps 4-11    scales and stores, a thread per channel and half of the tokens
//   warps 12-19   int8 only: widen the ring's bytes to fp16
// The accumulator is held twice, so the tile that is stored does not stop the next
// one's products.  CTAs are persistent over the tiles.
//
// E4M3 products are the matrix unit's own (kind::f8f6f4).  It has no int8 form on
// this GPU, and the warp-level int8 instruction runs at the rate of the scalar dot
// product (148 TOPS measured).  But every int8 is an fp16 number, a product of two is
// at most 2^14 in size, and fp32 sums of whole numbers are exact up to 2^24: so int8
// operands go through kind::f16 exactly, 1024 terms at a time.  Every 1024 terms the
// accumulator is emptied into int32 registers.
//
// Few tiles are cut along the summed dimension over the CTAs of a cluster (SPLIT),
// which then add their parts through distributed shared memory in a fixed order.
//
// Every wait has a limit of two seconds.  A wait that runs out (which correct
// operation never does) ends all later waits of the CTA at once and makes its
// outputs NaN.
#include "matmul_common.cuh"
#include "tc_common.cuh"

namespace edge {
namespace {

constexpr int kRows = 128;  // channels of a tile

template <bool INT8, int NT>
struct Mm {
    static constexpr int kStep = INT8 ? 64 : 128;                 // terms of a ring entry
    static constexpr int kRaw = (kRows + NT) * kStep;             // bytes that TMA writes
    static constexpr int kWide = (kRows + NT) * 128;              // fp16 bytes of an int8 entry
    static constexpr int kWides = INT8 ? (NT >= 128 ? 3 : 4) : 0;
    static constexpr int kLeft = 220 * 1024 - kWides * kWide;
    static constexpr int kStages = kLeft / kRaw < 10 ? kLeft / kRaw : 10;
    static constexpr int kSmem = kStages * kRaw + kWides * kWide + 1024;
    static constexpr int kThreads = INT8 ? 640 : 384;
    static constexpr int kColumns = 2 * NT;                       // of TMEM
    static constexpr int kUnit = INT8 ? 1024 / kStep : 1 << 30;   // entries until the sum is emptied
    static_assert(kStages >= 3 && kSmem <= 227 * 1024, "the ring does not fit");
    static_assert(NT * kRows * 4 <= kSmem - 1024, "a part of a cut tile does not fit");
};

struct MmSmem {
    uint64_t full[10], empty[10];      // the ring
    uint64_t wide[4], narrow[4];       // widened entries: full, empty
    uint64_t sum[2], taken[2];         // accumulators: full, empty
    uint32_t tmem, failed;
};

struct TcP {
    MatmulP m;
    int tiles_n, tiles_t;
    int split;       // CTAs of a cluster that share a tile
};

// Tiles in groups of 16 token tiles, the token tile running fastest: a wave's
// operands stay in L2.
__device__ __forceinline__ void tile_at(const TcP& p, int i, int& tn, int& tt) {
    const int per = 16 * p.tiles_n, group = i / per, first = group * 16;
    const int wide = min(16, p.tiles_t - first), at = i - group * per;
    tn = at / wide;
    tt = first + at - tn * wide;
}

template <bool INT8>
__device__ __forceinline__ void mma_8bit(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
    if constexpr (INT8) {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
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

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A 32-bit word of shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_word(uint32_t addr, int rank) {
    uint32_t at, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// Four int8 to four fp16 numbers: a byte with its sign bit turned, in the low bits of
// an fp16 number of exponent 2^10, is 1024 + 128 + the value.
__device__ __forceinline__ void widen4(uint32_t v, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = v ^ 0x80808080u;
    const __half2 bias = __floats2half2_rn(-1152.0f, -1152.0f);
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hadd2(*reinterpret_cast<const __half2*>(&a), bias);
    const __half2 y = __hadd2(*reinterpret_cast<const __half2*>(&b), bias);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

template <bool INT8, int NT>
__global__ void __launch_bounds__(Mm<INT8, NT>::kThreads, 1)
matmul_tc_kernel(TcP p, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap) {
    using C = Mm<INT8, NT>;
    constexpr int ST = C::kStages, WD = C::kWides > 0 ? C::kWides : 1;
    extern __shared__ char raw[];
    __shared__ MmSmem sh;
    const int tid = threadIdx.x, lane = tid & 31, wid = uniform(tid >> 5);
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;  // the swizzle works on address bits
    const uint32_t wides = base, ring = base + C::kWides * C::kWide;
    const int split = p.split, rank = split > 1 ? (int)(blockIdx.x % split) : 0;
    const int tiles = p.tiles_n * p.tiles_t;
    const int first = blockIdx.x / split, step = gridDim.x / split;
    const int entries = (p.m.k + C::kStep - 1) / C::kStep;
    const int e0 = (int)((int64_t)entries * rank / split), e1 = (int)((int64_t)entries * (rank + 1) / split);

    if (wid == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)), "n"(C::kColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            bar_init(smem_addr(&sh.full[i]), 1);
            bar_init(smem_addr(&sh.empty[i]), INT8 ? 8 : 1);
        }
        for (int i = 0; i < WD; ++i) {
            bar_init(smem_addr(&sh.wide[i]), 8);
            bar_init(smem_addr(&sh.narrow[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_addr(&sh.sum[i]), 1);
            bar_init(smem_addr(&sh.taken[i]), 8);
        }
        sh.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        // the first weights into L2 while the preceding grid drains
        int tn, tt;
        tile_at(p, first, tn, tt);
        for (int e = e0; e < e1 && e < e0 + ST; ++e) tma_prefetch_2d(&wmap, e * C::kStep, tn * kRows);
    }
    tc_before();
    __syncthreads();
    tc_after();
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t tmem = (uint32_t)uniform((int)sh.tmem);
    volatile uint32_t* failed = &sh.failed;

    if (wid < 4) {
        if constexpr (INT8) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (wid == 0) {
            // ---- copies
            const uint32_t lead = elect_lane();
            uint32_t n = 0;
            for (int i = first; i < tiles; i += step) {
                int tn, tt;
                tile_at(p, i, tn, tt);
                for (int e = e0; e < e1; ++e, ++n) {
                    const uint32_t st = n % ST, dst = ring + st * C::kRaw, bar = smem_addr(&sh.full[st]);
                    bar_wait(smem_addr(&sh.empty[st]), ((n / ST) & 1) ^ 1, failed);
                    bar_expect(bar, C::kRaw, lead);
                    tma_2d(dst, &wmap, e * C::kStep, tn * kRows, bar, lead);
                    tma_2d(dst + kRows * C::kStep, &amap, e * C::kStep, tt * NT, bar, lead);
                }
            }
        } else if (wid == 1) {
            // ---- products
            const uint32_t lead = elect_lane();
            constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(NT / 8) << 17) | ((uint32_t)(kRows / 16) << 24);
            constexpr int DEPTH = INT8 ? WD : ST;
            constexpr int BYTES = INT8 ? C::kWide : C::kRaw;
            const uint64_t dw = smem_desc(INT8 ? wides : ring, 16);
            const uint64_t da = dw + ((kRows * 128) >> 4);
            uint32_t n = 0, unit = 0;
            for (int i = first; i < tiles; i += step) {
                for (int e = e0; e < e1; ++unit) {
                    const uint32_t buf = unit & 1, d = tmem + buf * NT;
                    bar_wait(smem_addr(&sh.taken[buf]), ((unit >> 1) & 1) ^ 1, failed);
                    tc_after();
                    const int end = min(e1, e + C::kUnit), begin = e;
                    for (; e < end; ++e, ++n) {
                        const uint32_t st = n % DEPTH;
                        bar_wait(smem_addr(INT8 ? &sh.wide[st] : &sh.full[st]), (n / DEPTH) & 1, failed);
                        tc_after();
                        const uint64_t at = st * (uint32_t)(BYTES >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            mma_8bit<INT8>(d, dw + (at + k * 2), da + (at + k * 2), idesc, k > 0 ? 1u : (uint32_t)(e > begin), lead);
                        }
                        tc_commit(smem_addr(INT8 ? &sh.narrow[st] : &sh.empty[st]), lead);
                    }
                    tc_commit(smem_addr(&sh.sum[buf]), lead);
                }
            }
        }
    } else if (wid < 12) {
        if constexpr (INT8) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        // ---- sums: this thread's channel, and half of the tokens
        constexpr int H = NT / 2, CH = H < 32 ? H : 32;
        const int quad = wid & 3, half = (wid - 4) >> 2;
        const int row = quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + half * H;
        auto load = [&](uint32_t at, uint32_t (&v)[CH]) {
            if constexpr (CH == 32) {
                tc_ld32(at, v);
            } else {
                tc_ld16(at, v);
            }
            tc_wait_ld();
        };
        uint32_t unit = 0;
        for (int i = first; i < tiles; i += step) {
            int tn, tt;
            tile_at(p, i, tn, tt);
            const int ch = tn * kRows + row, t0 = tt * NT + half * H;
            const bool mine = ch < p.m.n;
            const float sw = mine ? __ldg(p.m.sw + ch) : 0.0f;
            const float bias = mine && p.m.bias != nullptr ? load_out(p.m.bias, ch, p.m.out_dt) : 0.0f;
            // CH sums of tokens t0 + c ..: to the output, or to this CTA's part of the tile
            auto give = [&](int c, const uint32_t (&v)[CH]) {
                if (split > 1) {
#pragma unroll
                    for (int j = 0; j < CH; ++j) {
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + (uint32_t)(((half * H + c + j) * kRows + row) * 4)), "r"(v[j]) : "memory");
                    }
                    return;
                }
                if (!mine) return;
                const float nan = *failed ? NAN : 0.0f;
#pragma unroll
                for (int j = 0; j < CH; ++j) {
                    const int t = t0 + c + j;
                    if (t >= p.m.tokens) break;
                    const float sum = (INT8 ? __int2float_rn((int)v[j]) : __uint_as_float(v[j])) + nan;
                    store_out(p.m.out, (int64_t)t * p.m.n + ch, scaled(sum, __ldg(p.m.sa + t), sw, bias), p.m.out_dt);
                }
            };
            if constexpr (INT8) {
                uint32_t acc[H];
#pragma unroll
                for (int c = 0; c < H; ++c) acc[c] = 0u;
                for (int e = e0; e < e1; e += C::kUnit, ++unit) {
                    const uint32_t buf = unit & 1;
                    bar_wait(smem_addr(&sh.sum[buf]), (unit >> 1) & 1, failed);
                    tc_after();
#pragma unroll
                    for (int c = 0; c < H; c += CH) {
                        uint32_t v[CH];
                        load(lanes + buf * NT + c, v);
#pragma unroll
                        for (int j = 0; j < CH; ++j) acc[c + j] += (uint32_t)__float2int_rn(__uint_as_float(v[j]));
                    }
                    tc_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(smem_addr(&sh.taken[buf]));
                }
#pragma unroll
                for (int c = 0; c < H; c += CH) {
                    uint32_t v[CH];
#pragma unroll
                    for (int j = 0; j < CH; ++j) v[j] = acc[c + j];
                    give(c, v);
                }
            } else {
                const uint32_t buf = unit & 1;
                bar_wait(smem_addr(&sh.sum[buf]), (unit >> 1) & 1, failed);
                tc_after();
#pragma unroll 1
                for (int c = 0; c < H; c += CH) {
                    uint32_t v[CH];
                    load(lanes + buf * NT + c, v);
                    give(c, v);
                }
                tc_before();
                __syncwarp();
                if (lane == 0) bar_arrive(smem_addr(&sh.taken[buf]));
                ++unit;
            }
        }
    } else if constexpr (INT8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        // ---- widening: a 16-byte piece of a row to two of fp16, stored with the 128-byte
        // swizzle that the products read
        const int mine = tid - 384;
        uint32_t n = 0;
        for (int i = first; i < tiles; i += step) {
            for (int e = e0; e < e1; ++e, ++n) {
                const uint32_t st = n % ST, wd = n % WD;
                bar_wait(smem_addr(&sh.full[st]), (n / ST) & 1, failed);
                bar_wait(smem_addr(&sh.narrow[wd]), ((n / WD) & 1) ^ 1, failed);
                const uint32_t src = ring + st * C::kRaw, dst = wides + wd * C::kWide;
#pragma unroll 2
                for (int q = mine; q < (kRows + NT) * 4; q += 256) {
                    uint4 v;
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src + q * 16) : "memory");
                    const int r = q >> 2, c = (q & 3) * 2;
                    uint32_t o[8];
                    widen4(v.x, o[0], o[1]);
                    widen4(v.y, o[2], o[3]);
                    widen4(v.z, o[4], o[5]);
                    widen4(v.w, o[6], o[7]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t at = dst + r * 128 + (((c + h) ^ (r & 7)) << 4);
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(o[4 * h]), "r"(o[4 * h + 1]), "r"(o[4 * h + 2]), "r"(o[4 * h + 3]) : "memory");
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(smem_addr(&sh.empty[st]));
                    bar_arrive(smem_addr(&sh.wide[wd]));
                }
            }
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
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kColumns) : "memory");
    }
    if (split > 1) {
        cluster_sync();
        if (wid >= 4 && wid < 12) {
            // this CTA's share of the tile's tokens, summed over the parts in rank order
            // (on the warps that have the registers)
            int tn, tt;
            tile_at(p, first, tn, tt);
            const int row = tid & 127, ch = tn * kRows + row;
            const int c0 = NT * rank / split, c1 = NT * (rank + 1) / split;
            float nan = 0.0f;
            for (int r = 0; r < split; ++r) nan = peer_word(smem_addr(&sh.failed), r) ? NAN : nan;
            const bool mine = ch < p.m.n;
            const float sw = mine ? __ldg(p.m.sw + ch) : 0.0f;
            const float bias = mine && p.m.bias != nullptr ? load_out(p.m.bias, ch, p.m.out_dt) : 0.0f;
            for (int c = c0 + ((wid - 4) >> 2); c < c1; c += 2) {
                const int t = tt * NT + c;
                if (!mine || t >= p.m.tokens) break;
                float sum = 0.0f;
                int whole = 0;
                for (int r = 0; r < split; ++r) {
                    const uint32_t v = peer_word(base + (uint32_t)((c * kRows + row) * 4), r);
                    if constexpr (INT8) {
                        whole += (int)v;
                    } else {
                        sum = __fadd_rn(sum, __uint_as_float(v));
                    }
                }
                if constexpr (INT8) sum = __int2float_rn(whole);
                store_out(p.m.out, (int64_t)t * p.m.n + ch, scaled(sum + nan, __ldg(p.m.sa + t), sw, bias), p.m.out_dt);
            }
        }
        cluster_sync();  // peers read this CTA's shared memory until here
    }
}

// ---------------------------------------------------------------- launch

bool operand_map(CUtensorMap* map, const char* base, int rows, int k, int box_rows, int box_k, bool swizzle) {
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)k};
    const cuuint32_t box[2] = {(cuuint32_t)box_k, (cuuint32_t)box_rows};
    const cuuint32_t ones[2] = {1, 1};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<char*>(base), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool INT8, int NT>
cudaError_t launch_tile(const MatmulP& m, int split, cudaLaunchConfig_t cfg) {
    using C = Mm<INT8, NT>;
    TcP p;
    p.m = m;
    p.tiles_n = (m.n + kRows - 1) / kRows;
    p.tiles_t = (m.tokens + NT - 1) / NT;
    p.split = split;
    CUtensorMap wmap, amap;
    if (!operand_map(&wmap, m.w, m.n, m.k, kRows, C::kStep, !INT8) ||
        !operand_map(&amap, m.a, m.tokens, m.k, NT, C::kStep, !INT8)) {
        return cudaErrorInvalidValue;
    }
    const cudaError_t e = allow_smem((const void*)matmul_tc_kernel<INT8, NT>, C::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)p.tiles_n * p.tiles_t;
    const int sms = sm_count();
    cfg.gridDim = dim3((unsigned)(split > 1 ? tiles * split : tiles < sms ? tiles : sms));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    if (split > 1) {
        cfg.attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        cfg.attrs[cfg.numAttrs].val.clusterDim.x = (unsigned)split;
        cfg.attrs[cfg.numAttrs].val.clusterDim.y = 1;
        cfg.attrs[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, matmul_tc_kernel<INT8, NT>, p, wmap, amap);
}

template <bool INT8>
cudaError_t launch_kind(const MatmulP& m, cudaLaunchConfig_t cfg) {
    const int sms = sm_count();
    const int nt = m.tokens <= 32 ? 32 : m.tokens <= 64 ? 64 : m.tokens <= 128 ? 128 : 256;
    const int64_t tiles = (int64_t)((m.n + kRows - 1) / kRows) * ((m.tokens + nt - 1) / nt);
    const int entries = (m.k + (INT8 ? 63 : 127)) / (INT8 ? 64 : 128);
    int split = 1;
    while (split < 8 && tiles * (split + 1) <= sms && (split + 1) * 4 <= entries) ++split;
    if (split == 7 || split == 5) --split;
    if (nt == 32) return launch_tile<INT8, 32>(m, split, cfg);
    if (nt == 64) return launch_tile<INT8, 64>(m, split, cfg);
    if (nt == 128) return launch_tile<INT8, 128>(m, split, cfg);
    return launch_tile<INT8, 256>(m, split, cfg);
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
