// edge_ops.cu -- the C ABI of libedge_ops.so: validation, then dispatch.
//
// Every entry point validates its arguments completely before any pointer
// arithmetic or launch ("thox-edge-ops v2", section 5.5): dtypes, NULL
// pointers, sizes, scalars, alignment, and overlap between written and read
// buffers.  An invalid call launches nothing and returns an edge_status.  The
// launchers in qk_norm_rope.cu, rows.cu and glu.cu then choose the kernel and
// launch shape.  Nothing here allocates, synchronizes or copies.
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <atomic>
#include <mutex>

#include "../../include/edge_ops.h"
#include "answers.h"
#include "launch.h"

namespace edge {

int sm_count() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    if (dev >= 0 && dev < 64) {
        int v = cache[dev].load(std::memory_order_relaxed);
        if (v > 0) return v;
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
        (void)cudaGetLastError();
        n = 148;
    }
    if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

int resident_ctas(const void* fn, int threads) {
    struct Entry {
        const void* fn;
        int threads, dev, n;
    };
    static std::mutex mu;
    static Entry table[128];
    static int used = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i) {
        if (table[i].fn == fn && table[i].threads == threads && table[i].dev == dev) {
            return table[i].n;
        }
    }
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, 0) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
    }
    if (n < 1) n = 1;
    if (used < 128) table[used++] = Entry{fn, threads, dev, n};
    return n;
}

int resident_clusters(const void* fn, const cudaLaunchConfig_t& cfg, int n) {
    static Answers<256> answers;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    const int clusters = answers.get(fn, n, dev, [&] {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)n;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t one = {};
        one.gridDim = dim3((unsigned)n);
        one.blockDim = cfg.blockDim;
        one.dynamicSmemBytes = cfg.dynamicSmemBytes;
        one.attrs = attr;
        one.numAttrs = 1;
        int found = 0;
        if (cudaOccupancyMaxActiveClusters(&found, fn, &one) == cudaSuccess) return found;
        (void)cudaGetLastError();
        return -1;
    });
    return clusters > 0 ? clusters : 0;
}

cudaError_t kernel_registers(const void* fn, int* registers) {
    static Answers<128> answers;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    *registers = answers.get(fn, 0, dev, [&] {
        cudaFuncAttributes f;
        e = cudaFuncGetAttributes(&f, fn);
        return e == cudaSuccess ? f.numRegs : -1;
    });
    return e;
}

cudaError_t allow_smem(const void* fn, int bytes) {
    if (bytes <= 40 * 1024) return cudaSuccess;  // 48 KB with the static part need no leave
    struct Entry {
        const void* fn;
        int dev, bytes;
    };
    static std::mutex mu;
    static Entry table[128];
    static int used = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    int at = used;
    for (int i = 0; i < used; ++i) {
        if (table[i].fn == fn && table[i].dev == dev) {
            if (table[i].bytes >= bytes) return cudaSuccess;
            at = i;
            break;
        }
    }
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && at < 128) {
        table[at] = Entry{fn, dev, bytes};
        if (at == used) ++used;
    }
    return e;
}

bool pdl_enabled() {
    static const bool on = [] {
        const char* v = std::getenv("EDGE_OPS_PDL");
        return !(v != nullptr && v[0] == '0');
    }();
    return on;
}

}  // namespace edge

namespace {

thread_local int g_last_cuda_error = 0;

bool act_dtype(edge_dtype dt) { return dt == EDGE_F32 || dt == EDGE_F16 || dt == EDGE_BF16; }

bool q8_dtype(edge_dtype dt) { return dt == EDGE_INT8 || dt == EDGE_FP8_E4M3; }

int64_t esize(edge_dtype dt) { return dt == EDGE_F32 ? 4 : (q8_dtype(dt) ? 1 : 2); }

bool aligned(const void* p, int64_t n) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % (uintptr_t)n) == 0;
}

// Byte range [p, p + n) of a buffer; empty ranges never overlap.
struct Span {
    uintptr_t lo, hi;
};

Span span(const void* p, int64_t bytes) {
    uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Span{lo, p == nullptr ? lo : lo + (uintptr_t)bytes};
}

bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

// A written buffer may coincide with one input exactly (in place), else must not overlap it.
bool bad_alias(Span out, Span in, bool exact_ok) {
    if (!overlap(out, in)) return false;
    return !(exact_ok && out.lo == in.lo && out.hi == in.hi);
}

bool finite_nonneg(float v) { return std::isfinite(v) && v >= 0.0f; }

// rows * cols * bytes without overflow; false if it would exceed int64.
bool checked_bytes(int64_t rows, int64_t cols, int64_t bytes, int64_t* out) {
    if (rows < 0 || cols < 0) return false;
    if (cols != 0 && rows > INT64_MAX / cols) return false;
    const int64_t n = rows * cols;
    if (bytes != 0 && n > INT64_MAX / bytes) return false;
    *out = n * bytes;
    return true;
}

edge_status finish(cudaError_t e) {
    // (taken from the runtime in either case: the next call is not to find it there)
    const cudaError_t last = cudaGetLastError();
    if (e == cudaSuccess) e = last;
    if (e != cudaSuccess) {
        g_last_cuda_error = (int)e;
        return EDGE_ERR_CUDA;
    }
    return EDGE_OK;
}

edge_status check_out_dt(edge_dtype out_dt, edge_dtype dt) {
    if (!act_dtype(dt)) return EDGE_ERR_DTYPE;
    if (out_dt != dt && out_dt != EDGE_FP8_E4M3) return EDGE_ERR_DTYPE;
    return EDGE_OK;
}

edge_status check_scale(edge_dtype out_dt, float inv_scale) {
    if (out_dt == EDGE_FP8_E4M3 && !(std::isfinite(inv_scale) && inv_scale > 0.0f)) {
        return EDGE_ERR_VALUE;
    }
    return EDGE_OK;
}

edge_status rows_entry(void* out, edge_dtype out_dt, const void* x, void* residual, bool fused,
                       const void* w, edge_dtype dt, int64_t rows, int64_t hidden, float eps,
                       int weight_offset, float inv_scale, void* stream) {
    edge_status st = check_out_dt(out_dt, dt);
    if (st != EDGE_OK) return st;
    if (x == nullptr || out == nullptr || (fused && residual == nullptr)) return EDGE_ERR_NULL;
    if (rows < 0 || hidden <= 0) return EDGE_ERR_SHAPE;
    if (!finite_nonneg(eps) || (weight_offset != 0 && weight_offset != 1)) return EDGE_ERR_VALUE;
    if ((st = check_scale(out_dt, inv_scale)) != EDGE_OK) return st;
    int64_t in_bytes = 0, out_bytes = 0;
    if (!checked_bytes(rows, hidden, esize(dt), &in_bytes) ||
        !checked_bytes(rows, hidden, esize(out_dt), &out_bytes)) {
        return EDGE_ERR_SHAPE;
    }
    if (hidden > edge::kMaxHidden) return EDGE_ERR_UNSUPPORTED;
    const int64_t es = esize(dt);
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(w, es) || !aligned(out, esize(out_dt))) {
        return EDGE_ERR_ALIGN;
    }
    const Span so = span(out, out_bytes), sx = span(x, in_bytes), sw = span(w, hidden * es);
    const Span sr = span(fused ? residual : nullptr, in_bytes);
    const bool same_dt = out_dt == dt;
    if (bad_alias(so, sx, same_dt) || overlap(so, sw) || overlap(so, sr)) return EDGE_ERR_ALIAS;
    if (fused && (overlap(sr, sx) || overlap(sr, sw))) return EDGE_ERR_ALIAS;
    if (rows == 0) return EDGE_OK;

    edge::RowsArgs a;
    a.x = x;
    a.residual = fused ? residual : nullptr;
    a.w = w;
    a.beta = nullptr;
    a.layernorm = 0;
    a.out = out;
    a.rows = rows;
    a.hidden = hidden;
    a.dt = (int)dt;
    a.out_dt = (int)out_dt;
    a.eps = eps;
    a.inv_scale = inv_scale;
    a.weight_offset = weight_offset;
    return finish(edge::launch_rows(a, static_cast<cudaStream_t>(stream)));
}

// Rows in 8 bits with a scale each.  act: -1 without a gate.
edge_status rows_q8_entry(void* out, edge_dtype q_dt, float* scales, const void* x, void* residual,
                          bool fused, const void* w, bool norm, edge_dtype dt, int64_t rows,
                          int64_t n, float eps, int weight_offset, int act, void* stream) {
    if (!act_dtype(dt) || !q8_dtype(q_dt)) return EDGE_ERR_DTYPE;
    if (x == nullptr || out == nullptr || scales == nullptr || (fused && residual == nullptr)) {
        return EDGE_ERR_NULL;
    }
    if (rows < 0 || n <= 0) return EDGE_ERR_SHAPE;
    if (!finite_nonneg(eps) || (weight_offset != 0 && weight_offset != 1)) return EDGE_ERR_VALUE;
    const int64_t es = esize(dt);
    int64_t in_bytes = 0, out_bytes = 0, scale_bytes = 0;
    if (!checked_bytes(rows, n, es * (act >= 0 ? 2 : 1), &in_bytes) ||
        !checked_bytes(rows, n, 1, &out_bytes) || !checked_bytes(rows, 1, 4, &scale_bytes)) {
        return EDGE_ERR_SHAPE;
    }
    if (n > edge::kMaxHidden) return EDGE_ERR_UNSUPPORTED;
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(w, es) || !aligned(scales, 4)) {
        return EDGE_ERR_ALIGN;
    }
    const Span so = span(out, out_bytes), ss = span(scales, scale_bytes), sx = span(x, in_bytes);
    const Span sw = span(w, n * es), sr = span(fused ? residual : nullptr, in_bytes);
    if (overlap(so, ss)) return EDGE_ERR_ALIAS;
    for (const Span& written : {so, ss}) {
        if (overlap(written, sx) || overlap(written, sw) || overlap(written, sr)) return EDGE_ERR_ALIAS;
    }
    if (fused && (overlap(sr, sx) || overlap(sr, sw))) return EDGE_ERR_ALIAS;
    if (rows == 0) return EDGE_OK;

    edge::RowsQ8Args a;
    a.x = x;
    a.residual = fused ? residual : nullptr;
    a.w = w;
    a.out = out;
    a.scales = scales;
    a.rows = rows;
    a.n = n;
    a.dt = (int)dt;
    a.out_dt = (int)q_dt;
    a.norm = norm ? 1 : 0;
    a.act = act;
    a.eps = eps;
    a.weight_offset = weight_offset;
    return finish(edge::launch_rows_q8(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

namespace {

const edge::Axes kOneAxis = {0, 0, {0, 0, 0, 0}};

// The sections of a rotary embedding with several axes.
edge_status read_axes(int32_t axes, const int32_t* sections, edge_axis_order order,
                      int32_t rotary_dim, edge::Axes* out) {
    if (sections == nullptr) return EDGE_ERR_NULL;
    if (axes < 1 || axes > 4) return EDGE_ERR_SHAPE;
    if (order != EDGE_AXES_BLOCKS && order != EDGE_AXES_CYCLED) return EDGE_ERR_VALUE;
    *out = edge::Axes{axes, order == EDGE_AXES_CYCLED, {0, 0, 0, 0}};
    const int64_t half = rotary_dim / 2;
    int64_t sum = 0;
    for (int a = 0; a < axes; ++a) {
        if (sections[a] < 0) return EDGE_ERR_SHAPE;
        // dealt in turn, the last pair of every axis but the first is named
        if (out->cycled && a > 0 && sections[a] > 0 &&
            ((int64_t)sections[a] - 1) * axes + a >= half) {
            return EDGE_ERR_SHAPE;
        }
        out->count[a] = sections[a];
        sum += sections[a];
    }
    return sum == half ? EDGE_OK : EDGE_ERR_SHAPE;
}

static edge_status qk_entry(void* q_out, void* k_out, edge_dtype out_dt, const void* q,
                            const void* k, const void* wq, const void* wk, edge_dtype dt,
                            int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                            int32_t rotary_dim, edge_rope_layout layout, const int64_t* positions,
                            const float* cos, const float* sin, int64_t cache_len, float eps,
                            int weight_offset, float inv_scale, int mode, const edge::Axes& axes,
                            void* stream) {
    edge_status st = check_out_dt(out_dt, dt);
    if (st != EDGE_OK) return st;
    if (q == nullptr || q_out == nullptr) return EDGE_ERR_NULL;
    if (k_heads > 0 && (k == nullptr || k_out == nullptr)) return EDGE_ERR_NULL;
    if (tokens < 0 || q_heads < 1 || k_heads < 0 || head_dim < 1 || cache_len < 0) {
        return EDGE_ERR_SHAPE;
    }
    if (rotary_dim < 0 || rotary_dim > head_dim || (rotary_dim & 1)) return EDGE_ERR_SHAPE;
    if (layout != EDGE_ROPE_ROTATE_HALF && layout != EDGE_ROPE_INTERLEAVED) return EDGE_ERR_VALUE;
    if (!finite_nonneg(eps) || (weight_offset != 0 && weight_offset != 1)) return EDGE_ERR_VALUE;
    if ((st = check_scale(out_dt, inv_scale)) != EDGE_OK) return st;
    const bool may_rotate = rotary_dim > 0 && cache_len > 0;
    const int64_t per_token = axes.n > 0 ? axes.n : 1;
    if (may_rotate && (positions == nullptr || cos == nullptr || sin == nullptr)) {
        return EDGE_ERR_NULL;
    }
    const int64_t es = esize(dt), eo = esize(out_dt);
    int64_t qb = 0, kb = 0, qob = 0, kob = 0, cb = 0;
    if (!checked_bytes(tokens, (int64_t)q_heads * head_dim, es, &qb) ||
        !checked_bytes(tokens, (int64_t)k_heads * head_dim, es, &kb) ||
        !checked_bytes(tokens, (int64_t)q_heads * head_dim, eo, &qob) ||
        !checked_bytes(tokens, (int64_t)k_heads * head_dim, eo, &kob) ||
        !checked_bytes(cache_len, rotary_dim / 2, 4, &cb)) {
        return EDGE_ERR_SHAPE;
    }
    if (head_dim > edge::kMaxQKHeadDim) return EDGE_ERR_UNSUPPORTED;
    if (tokens > edge::kMaxUnits / ((int64_t)q_heads + k_heads)) return EDGE_ERR_UNSUPPORTED;
    if (!aligned(q, es) || !aligned(k, es) || !aligned(wq, es) || !aligned(wk, es) ||
        !aligned(q_out, eo) || !aligned(k_out, eo) || !aligned(positions, 8) || !aligned(cos, 4) ||
        !aligned(sin, 4)) {
        return EDGE_ERR_ALIGN;
    }
    const bool same_dt = out_dt == dt;
    const Span sq = span(q, qb), sk = span(k_heads ? k : nullptr, kb);
    const Span sqo = span(q_out, qob), sko = span(k_heads ? k_out : nullptr, kob);
    const Span ro[] = {span(wq, head_dim * es), span(wk, head_dim * es),
                       span(may_rotate ? positions : nullptr, per_token * tokens * 8),
                       span(may_rotate ? cos : nullptr, cb), span(may_rotate ? sin : nullptr, cb)};
    if (bad_alias(sqo, sq, same_dt) || bad_alias(sko, sk, same_dt) || overlap(sqo, sk) ||
        overlap(sko, sq) || overlap(sqo, sko)) {
        return EDGE_ERR_ALIAS;
    }
    for (const Span& r : ro) {
        if (overlap(sqo, r) || overlap(sko, r)) return EDGE_ERR_ALIAS;
    }
    if (tokens == 0) return EDGE_OK;

    edge::QKArgs a;
    a.q = q;
    a.k = k_heads ? k : nullptr;
    a.q_out = q_out;
    a.k_out = k_heads ? k_out : nullptr;
    a.wq = wq;
    a.wk = wk;
    a.pos = may_rotate ? positions : nullptr;
    a.cos = may_rotate ? cos : nullptr;
    a.sin = may_rotate ? sin : nullptr;
    a.tokens = tokens;
    a.cache_len = cache_len;
    a.q_heads = q_heads;
    a.k_heads = k_heads;
    a.head_dim = head_dim;
    a.rotary_dim = rotary_dim;
    a.layout = (int)layout;
    a.dt = (int)dt;
    a.out_dt = (int)out_dt;
    a.eps = eps;
    a.inv_scale = inv_scale;
    a.weight_offset = weight_offset;
    a.mode = mode;
    a.axes = axes;
    return finish(edge::launch_qk(a, static_cast<cudaStream_t>(stream)));
}

static edge_status qkv_entry(void* q_out, void* k_cache, void* v_cache, const void* qkv,
                             const void* wq, const void* wk, edge_dtype dt, int64_t tokens,
                             int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                             int32_t rotary_dim, edge_rope_layout layout,
                             const int64_t* positions, const float* cos, const float* sin,
                             int64_t cache_len, const int64_t* slots, int64_t num_slots,
                             float eps, int weight_offset, int normalize, const edge::Axes& axes,
                             void* stream) {
    if (!act_dtype(dt)) return EDGE_ERR_DTYPE;
    if (qkv == nullptr || q_out == nullptr) return EDGE_ERR_NULL;
    const bool writes_cache = kv_heads > 0 && num_slots > 0;
    if (writes_cache && (k_cache == nullptr || v_cache == nullptr || slots == nullptr)) {
        return EDGE_ERR_NULL;
    }
    if (tokens < 0 || q_heads < 1 || kv_heads < 0 || head_dim < 1 || cache_len < 0 ||
        num_slots < 0) {
        return EDGE_ERR_SHAPE;
    }
    if (rotary_dim < 0 || rotary_dim > head_dim || (rotary_dim & 1)) return EDGE_ERR_SHAPE;
    if (layout != EDGE_ROPE_ROTATE_HALF && layout != EDGE_ROPE_INTERLEAVED) return EDGE_ERR_VALUE;
    if (!finite_nonneg(eps) || (weight_offset != 0 && weight_offset != 1) ||
        (normalize != 0 && normalize != 1)) {
        return EDGE_ERR_VALUE;
    }
    const bool may_rotate = rotary_dim > 0 && cache_len > 0;
    if (may_rotate && (positions == nullptr || cos == nullptr || sin == nullptr)) {
        return EDGE_ERR_NULL;
    }
    const int64_t per_token = axes.n > 0 ? axes.n : 1;
    const int64_t es = esize(dt);
    const int64_t heads_row = (int64_t)q_heads + 2 * (int64_t)kv_heads;
    int64_t in_b = 0, q_b = 0, c_b = 0, cs_b = 0;
    if (!checked_bytes(tokens, heads_row * head_dim, es, &in_b) ||
        !checked_bytes(tokens, (int64_t)q_heads * head_dim, es, &q_b) ||
        !checked_bytes(num_slots, (int64_t)kv_heads * head_dim, es, &c_b) ||
        !checked_bytes(cache_len, rotary_dim / 2, 4, &cs_b)) {
        return EDGE_ERR_SHAPE;
    }
    if (head_dim > edge::kMaxQKHeadDim) return EDGE_ERR_UNSUPPORTED;
    if (tokens > edge::kMaxUnits / heads_row) return EDGE_ERR_UNSUPPORTED;
    if (!aligned(qkv, es) || !aligned(q_out, es) || !aligned(k_cache, es) ||
        !aligned(v_cache, es) || !aligned(wq, es) || !aligned(wk, es) || !aligned(positions, 8) ||
        !aligned(slots, 8) || !aligned(cos, 4) || !aligned(sin, 4)) {
        return EDGE_ERR_ALIGN;
    }
    const Span sq = span(q_out, q_b);
    const Span sk = span(writes_cache ? k_cache : nullptr, c_b);
    const Span sv = span(writes_cache ? v_cache : nullptr, c_b);
    const Span ro[] = {span(qkv, in_b), span(wq, head_dim * es), span(wk, head_dim * es),
                       span(may_rotate ? positions : nullptr, per_token * tokens * 8),
                       span(may_rotate ? cos : nullptr, cs_b), span(may_rotate ? sin : nullptr, cs_b),
                       span(writes_cache ? slots : nullptr, tokens * 8)};
    if (overlap(sq, sk) || overlap(sq, sv) || overlap(sk, sv)) return EDGE_ERR_ALIAS;
    for (const Span& r : ro) {
        if (overlap(sq, r) || overlap(sk, r) || overlap(sv, r)) return EDGE_ERR_ALIAS;
    }
    if (tokens == 0) return EDGE_OK;
    edge::QKVArgs a;
    a.qkv = qkv;
    a.q_out = q_out;
    a.k_cache = writes_cache ? k_cache : nullptr;
    a.v_cache = writes_cache ? v_cache : nullptr;
    a.wq = wq;
    a.wk = wk;
    a.pos = may_rotate ? positions : nullptr;
    a.cos = may_rotate ? cos : nullptr;
    a.sin = may_rotate ? sin : nullptr;
    a.slots = writes_cache ? slots : nullptr;
    a.tokens = tokens;
    a.cache_len = cache_len;
    a.num_slots = writes_cache ? num_slots : 0;
    a.q_heads = q_heads;
    a.kv_heads = kv_heads;
    a.head_dim = head_dim;
    a.rotary_dim = rotary_dim;
    a.layout = (int)layout;
    a.dt = (int)dt;
    a.normalize = normalize;
    a.weight_offset = weight_offset;
    a.eps = eps;
    a.axes = axes;
    bool handled = false;
    cudaError_t e = edge::launch_qkv_cache(a, static_cast<cudaStream_t>(stream), &handled);
    if (e == cudaSuccess && !handled) return EDGE_ERR_UNSUPPORTED;
    return finish(e);
}

// The caches of a page pool: none overlaps another, or one of `other`.
edge_status check_pool(void* const* caches, int32_t num_caches, int64_t page_bytes,
                       int32_t num_pages, int64_t pairs, const Span* other, int others) {
    if (num_caches < 0 || page_bytes < 1 || num_pages < 0) return EDGE_ERR_SHAPE;
    if (num_caches > 0 && caches == nullptr) return EDGE_ERR_NULL;
    int64_t bytes = 0;
    if (!checked_bytes(num_pages, page_bytes, 1, &bytes)) return EDGE_ERR_SHAPE;
    if (!edge::pages_fit(page_bytes, pairs)) return EDGE_ERR_UNSUPPORTED;
    for (int i = 0; i < num_caches; ++i) {
        if (caches[i] == nullptr) return EDGE_ERR_NULL;
    }
    for (int i = 0; i < num_caches; ++i) {
        const Span c = span(caches[i], bytes);
        for (int j = 0; j < i; ++j) {
            if (overlap(c, span(caches[j], bytes))) return EDGE_ERR_ALIAS;
        }
        for (int j = 0; j < others; ++j) {
            if (overlap(c, other[j])) return EDGE_ERR_ALIAS;
        }
    }
    return EDGE_OK;
}

// Whether two of the spans overlap.
bool any_overlap(const Span* s, int n) {
    for (int i = 0; i < n; ++i) {
        for (int j = 0; j < i; ++j) {
            if (overlap(s[i], s[j])) return true;
        }
    }
    return false;
}

}  // namespace

extern "C" {

edge_status edge_rmsnorm(void* out, edge_dtype out_dt, const void* x, const void* w, edge_dtype dt,
                         int64_t rows, int64_t hidden, float eps, int weight_offset,
                         float inv_scale, void* stream) {
    return rows_entry(out, out_dt, x, nullptr, false, w, dt, rows, hidden, eps, weight_offset,
                      inv_scale, stream);
}

edge_status edge_add_rmsnorm(void* out, edge_dtype out_dt, const void* x, void* residual,
                             const void* w, edge_dtype dt, int64_t rows, int64_t hidden, float eps,
                             int weight_offset, float inv_scale, void* stream) {
    return rows_entry(out, out_dt, x, residual, true, w, dt, rows, hidden, eps, weight_offset,
                      inv_scale, stream);
}

edge_status edge_qkv_rope_cache(void* q_out, void* k_cache, void* v_cache, const void* qkv,
                                const void* wq, const void* wk, edge_dtype dt, int64_t tokens,
                                int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                int32_t rotary_dim, edge_rope_layout layout,
                                const int64_t* positions, const float* cos, const float* sin,
                                int64_t cache_len, const int64_t* slots, int64_t num_slots,
                                float eps, int weight_offset, int normalize, void* stream) {
    return qkv_entry(q_out, k_cache, v_cache, qkv, wq, wk, dt, tokens, q_heads, kv_heads, head_dim,
                     rotary_dim, layout, positions, cos, sin, cache_len, slots, num_slots, eps,
                     weight_offset, normalize, kOneAxis, stream);
}

edge_status edge_qkv_rope_cache_axes(void* q_out, void* k_cache, void* v_cache, const void* qkv,
                                     const void* wq, const void* wk, edge_dtype dt, int64_t tokens,
                                     int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                     int32_t rotary_dim, edge_rope_layout layout,
                                     const int64_t* positions, int32_t axes,
                                     const int32_t* sections, edge_axis_order order,
                                     const float* cos, const float* sin, int64_t cache_len,
                                     const int64_t* slots, int64_t num_slots, float eps,
                                     int weight_offset, int normalize, void* stream) {
    edge::Axes ax;
    const edge_status st = read_axes(axes, sections, order, rotary_dim, &ax);
    if (st != EDGE_OK) return st;
    return qkv_entry(q_out, k_cache, v_cache, qkv, wq, wk, dt, tokens, q_heads, kv_heads, head_dim,
                     rotary_dim, layout, positions, cos, sin, cache_len, slots, num_slots, eps,
                     weight_offset, normalize, ax, stream);
}

edge_status edge_layernorm(void* out, edge_dtype out_dt, const void* x, const void* gamma,
                           const void* beta, edge_dtype dt, int64_t rows, int64_t hidden,
                           float eps, float inv_scale, void* stream) {
    edge_status st = check_out_dt(out_dt, dt);
    if (st != EDGE_OK) return st;
    if (x == nullptr || out == nullptr) return EDGE_ERR_NULL;
    if (rows < 0 || hidden <= 0) return EDGE_ERR_SHAPE;
    if (!finite_nonneg(eps)) return EDGE_ERR_VALUE;
    if ((st = check_scale(out_dt, inv_scale)) != EDGE_OK) return st;
    int64_t in_bytes = 0, out_bytes = 0;
    if (!checked_bytes(rows, hidden, esize(dt), &in_bytes) ||
        !checked_bytes(rows, hidden, esize(out_dt), &out_bytes)) {
        return EDGE_ERR_SHAPE;
    }
    if (hidden > edge::kMaxHidden) return EDGE_ERR_UNSUPPORTED;
    const int64_t es = esize(dt);
    if (!aligned(x, es) || !aligned(gamma, es) || !aligned(beta, es) ||
        !aligned(out, esize(out_dt))) {
        return EDGE_ERR_ALIGN;
    }
    const Span so = span(out, out_bytes);
    if (bad_alias(so, span(x, in_bytes), out_dt == dt) || overlap(so, span(gamma, hidden * es)) ||
        overlap(so, span(beta, hidden * es))) {
        return EDGE_ERR_ALIAS;
    }
    if (rows == 0) return EDGE_OK;
    edge::RowsArgs a;
    a.x = x;
    a.residual = nullptr;
    a.w = gamma;
    a.beta = beta;
    a.layernorm = 1;
    a.out = out;
    a.rows = rows;
    a.hidden = hidden;
    a.dt = (int)dt;
    a.out_dt = (int)out_dt;
    a.eps = eps;
    a.inv_scale = inv_scale;
    a.weight_offset = 0;
    return finish(edge::launch_rows(a, static_cast<cudaStream_t>(stream)));
}

edge_status edge_quantize_fp8(void* out, const void* x, edge_dtype dt, int64_t n, float inv_scale,
                              void* stream) {
    if (!act_dtype(dt)) return EDGE_ERR_DTYPE;
    if (out == nullptr || x == nullptr) return EDGE_ERR_NULL;
    if (n < 0) return EDGE_ERR_SHAPE;
    if (!(std::isfinite(inv_scale) && inv_scale > 0.0f)) return EDGE_ERR_VALUE;
    int64_t in_bytes = 0;
    if (!checked_bytes(n, 1, esize(dt), &in_bytes)) return EDGE_ERR_SHAPE;
    if (n > edge::kMaxUnits * 8) return EDGE_ERR_UNSUPPORTED;
    if (!aligned(x, esize(dt))) return EDGE_ERR_ALIGN;
    if (overlap(span(out, n), span(x, in_bytes))) return EDGE_ERR_ALIAS;
    if (n == 0) return EDGE_OK;
    edge::QuantArgs a;
    a.x = x;
    a.out = out;
    a.n = n;
    a.dt = (int)dt;
    a.inv_scale = inv_scale;
    return finish(edge::launch_quant(a, static_cast<cudaStream_t>(stream)));
}

edge_status edge_glu_act(void* out, edge_dtype out_dt, const void* gate_up, edge_dtype dt,
                         int64_t rows, int64_t d, edge_act act, float inv_scale, void* stream) {
    edge_status st = check_out_dt(out_dt, dt);
    if (st != EDGE_OK) return st;
    if (out == nullptr || gate_up == nullptr) return EDGE_ERR_NULL;
    if (rows < 0 || d <= 0) return EDGE_ERR_SHAPE;
    if (act != EDGE_ACT_SILU && act != EDGE_ACT_GELU_TANH) return EDGE_ERR_VALUE;
    if ((st = check_scale(out_dt, inv_scale)) != EDGE_OK) return st;
    int64_t in_bytes = 0, out_bytes = 0;
    if (d > INT64_MAX / 2 || !checked_bytes(rows, 2 * d, esize(dt), &in_bytes) ||
        !checked_bytes(rows, d, esize(out_dt), &out_bytes)) {
        return EDGE_ERR_SHAPE;
    }
    if (!aligned(gate_up, esize(dt)) || !aligned(out, esize(out_dt))) return EDGE_ERR_ALIGN;
    if (overlap(span(out, out_bytes), span(gate_up, in_bytes))) return EDGE_ERR_ALIAS;
    if (rows == 0) return EDGE_OK;

    edge::GluArgs a;
    a.gate_up = gate_up;
    a.out = out;
    a.rows = rows;
    a.d = d;
    a.dt = (int)dt;
    a.out_dt = (int)out_dt;
    a.act = (int)act;
    a.inv_scale = inv_scale;
    return finish(edge::launch_glu(a, static_cast<cudaStream_t>(stream)));
}

edge_status edge_qk_norm_rope(void* q_out, void* k_out, edge_dtype out_dt, const void* q,
                              const void* k, const void* wq, const void* wk, edge_dtype dt,
                              int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                              int32_t rotary_dim, edge_rope_layout layout,
                              const int64_t* positions, const float* cos, const float* sin,
                              int64_t cache_len, float eps, int weight_offset, float inv_scale,
                              void* stream) {
    return qk_entry(q_out, k_out, out_dt, q, k, wq, wk, dt, tokens, q_heads, k_heads, head_dim,
                    rotary_dim, layout, positions, cos, sin, cache_len, eps, weight_offset,
                    inv_scale, 1 /* normalize */, kOneAxis, stream);
}

edge_status edge_qk_norm_rope_ex(void* q_out, void* k_out, edge_dtype out_dt, const void* q,
                                 const void* k, const void* wq, const void* wk, edge_dtype dt,
                                 int64_t tokens, int32_t q_heads, int32_t k_heads,
                                 int32_t head_dim, int32_t rotary_dim, edge_rope_layout layout,
                                 const int64_t* positions, const float* cos, const float* sin,
                                 int64_t cache_len, float eps, int weight_offset, float inv_scale,
                                 uint32_t flags, void* stream) {
    if ((flags & ~(uint32_t)EDGE_QK_ROTATE_UNROUNDED) != 0) return EDGE_ERR_VALUE;
    const int mode = 1 | ((flags & EDGE_QK_ROTATE_UNROUNDED) ? 2 : 0);
    return qk_entry(q_out, k_out, out_dt, q, k, wq, wk, dt, tokens, q_heads, k_heads, head_dim,
                    rotary_dim, layout, positions, cos, sin, cache_len, eps, weight_offset,
                    inv_scale, mode, kOneAxis, stream);
}

edge_status edge_qk_norm_rope_axes(void* q_out, void* k_out, edge_dtype out_dt, const void* q,
                                   const void* k, const void* wq, const void* wk, edge_dtype dt,
                                   int64_t tokens, int32_t q_heads, int32_t k_heads,
                                   int32_t head_dim, int32_t rotary_dim, edge_rope_layout layout,
                                   const int64_t* positions, int32_t axes, const int32_t* sections,
                                   edge_axis_order order, const float* cos, const float* sin,
                                   int64_t cache_len, float eps, int weight_offset,
                                   float inv_scale, uint32_t flags, void* stream) {
    if ((flags & ~(uint32_t)EDGE_QK_ROTATE_UNROUNDED) != 0) return EDGE_ERR_VALUE;
    edge::Axes ax;
    const edge_status st = read_axes(axes, sections, order, rotary_dim, &ax);
    if (st != EDGE_OK) return st;
    const int mode = 1 | ((flags & EDGE_QK_ROTATE_UNROUNDED) ? 2 : 0);
    return qk_entry(q_out, k_out, out_dt, q, k, wq, wk, dt, tokens, q_heads, k_heads, head_dim,
                    rotary_dim, layout, positions, cos, sin, cache_len, eps, weight_offset,
                    inv_scale, mode, ax, stream);
}

edge_status edge_rope_axes(void* q_out, void* k_out, edge_dtype out_dt, const void* q,
                           const void* k, edge_dtype dt, int64_t tokens, int32_t q_heads,
                           int32_t k_heads, int32_t head_dim, int32_t rotary_dim,
                           edge_rope_layout layout, const int64_t* positions, int32_t axes,
                           const int32_t* sections, edge_axis_order order, const float* cos,
                           const float* sin, int64_t cache_len, float inv_scale, void* stream) {
    edge::Axes ax;
    const edge_status st = read_axes(axes, sections, order, rotary_dim, &ax);
    if (st != EDGE_OK) return st;
    return qk_entry(q_out, k_out, out_dt, q, k, nullptr, nullptr, dt, tokens, q_heads, k_heads,
                    head_dim, rotary_dim, layout, positions, cos, sin, cache_len, 0.0f, 0,
                    inv_scale, 0 /* rotate only */, ax, stream);
}

edge_status edge_rope(void* q_out, void* k_out, edge_dtype out_dt, const void* q, const void* k,
                      edge_dtype dt, int64_t tokens, int32_t q_heads, int32_t k_heads,
                      int32_t head_dim, int32_t rotary_dim, edge_rope_layout layout,
                      const int64_t* positions, const float* cos, const float* sin,
                      int64_t cache_len, float inv_scale, void* stream) {
    return qk_entry(q_out, k_out, out_dt, q, k, nullptr, nullptr, dt, tokens, q_heads, k_heads,
                    head_dim, rotary_dim, layout, positions, cos, sin, cache_len, 0.0f, 0,
                    inv_scale, 0 /* rotate only */, kOneAxis, stream);
}

int64_t edge_paged_attention_workspace(edge_dtype dt, int32_t q_heads, int32_t kv_heads,
                                       int32_t head_dim) {
    if (!act_dtype(dt) || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || head_dim < 1 ||
        head_dim > edge::kMaxAttnHeadDim) {
        return -1;
    }
    return edge::attn_workspace((int)dt, q_heads, kv_heads, head_dim);
}

edge_status edge_paged_attention(void* out, edge_dtype out_dt, float* lse, const void* q,
                                 const void* k_cache, const void* v_cache, edge_dtype dt,
                                 int64_t tokens, int32_t q_heads, int32_t kv_heads,
                                 int32_t head_dim, int64_t num_slots, int32_t page_size,
                                 const int32_t* block_table, int32_t num_seqs, int32_t max_pages,
                                 const int32_t* lens, const int32_t* q_starts, float scale,
                                 int causal, int32_t window, float inv_scale, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
    edge_status st = check_out_dt(out_dt, dt);
    if (st != EDGE_OK) return st;
    if (q == nullptr || out == nullptr) return EDGE_ERR_NULL;
    if (tokens < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || head_dim < 1 ||
        num_slots < 0 || page_size < 1 || num_seqs < 0 || max_pages < 0) {
        return EDGE_ERR_SHAPE;
    }
    if (num_seqs > 0 && lens == nullptr) return EDGE_ERR_NULL;
    if (num_slots > 0 && (k_cache == nullptr || v_cache == nullptr)) return EDGE_ERR_NULL;
    if (num_seqs > 0 && max_pages > 0 && block_table == nullptr) return EDGE_ERR_NULL;
    if (q_starts == nullptr && tokens != num_seqs) return EDGE_ERR_SHAPE;
    if (!(std::isfinite(scale) && scale > 0.0f) || (causal != 0 && causal != 1) || window < 0 ||
        (window > 0 && causal == 0)) {
        return EDGE_ERR_VALUE;
    }
    if ((st = check_scale(out_dt, inv_scale)) != EDGE_OK) return st;
    const int64_t es = esize(dt);
    int64_t q_b = 0, o_b = 0, c_b = 0, t_b = 0;
    if (!checked_bytes(tokens, (int64_t)q_heads * head_dim, es, &q_b) ||
        !checked_bytes(tokens, (int64_t)q_heads * head_dim, esize(out_dt), &o_b) ||
        !checked_bytes(num_slots, (int64_t)kv_heads * head_dim, es, &c_b) ||
        !checked_bytes(num_seqs, max_pages, 4, &t_b)) {
        return EDGE_ERR_SHAPE;
    }
    if (head_dim > edge::kMaxAttnHeadDim || tokens > edge::kMaxAttnRows / q_heads ||
        (int64_t)max_pages * page_size > edge::kMaxAttnRows ||
        num_slots / page_size > edge::kMaxUnits) {
        return EDGE_ERR_UNSUPPORTED;
    }
    if (!aligned(q, es) || !aligned(k_cache, es) || !aligned(v_cache, es) ||
        !aligned(out, esize(out_dt)) || !aligned(lse, 4) || !aligned(block_table, 4) ||
        !aligned(lens, 4) || !aligned(q_starts, 4) || !aligned(workspace, 16)) {
        return EDGE_ERR_ALIGN;
    }
    const Span so = span(out, o_b), sl = span(lse, tokens * q_heads * 4);
    const Span sw = span(workspace, workspace_bytes < 0 ? 0 : workspace_bytes);
    const Span ro[] = {span(q, q_b), span(num_slots ? k_cache : nullptr, c_b),
                       span(num_slots ? v_cache : nullptr, c_b), span(block_table, t_b),
                       span(lens, (int64_t)num_seqs * 4),
                       span(q_starts, ((int64_t)num_seqs + 1) * 4)};
    if (overlap(so, sl) || overlap(so, sw) || overlap(sl, sw)) return EDGE_ERR_ALIAS;
    for (const Span& r : ro) {
        if (overlap(so, r) || overlap(sl, r) || overlap(sw, r)) return EDGE_ERR_ALIAS;
    }
    if (tokens == 0 || num_seqs == 0) return EDGE_OK;
    if (workspace == nullptr) return EDGE_ERR_NULL;
    if (workspace_bytes < edge::attn_workspace((int)dt, q_heads, kv_heads, head_dim)) {
        return EDGE_ERR_SHAPE;
    }
    edge::AttnArgs a;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.out = out;
    a.lse = lse;
    a.table = block_table;
    a.lens = lens;
    a.starts = q_starts;
    a.workspace = workspace;
    a.tokens = tokens;
    a.q_heads = q_heads;
    a.kv_heads = kv_heads;
    a.head_dim = head_dim;
    a.num_seqs = num_seqs;
    a.max_pages = max_pages;
    a.num_pages = (int)(num_slots / page_size);
    a.page_size = page_size;
    a.dt = (int)dt;
    a.out_dt = (int)out_dt;
    a.causal = causal;
    a.window = window;
    a.scale = scale;
    a.inv_scale = inv_scale;
    return finish(edge::launch_attn(a, static_cast<cudaStream_t>(stream)));
}

edge_status edge_pages_copy(void* const* caches, int32_t num_caches, int64_t page_bytes,
                            int32_t num_pages, const int32_t* src, const int32_t* dst, int32_t n,
                            void* stream) {
    if (n < 0) return EDGE_ERR_SHAPE;
    if (n > 0 && (src == nullptr || dst == nullptr)) return EDGE_ERR_NULL;
    if (n > edge::kMaxPagePairs) return EDGE_ERR_UNSUPPORTED;
    if (!aligned(src, 4) || !aligned(dst, 4)) return EDGE_ERR_ALIGN;
    const Span lists[] = {span(src, (int64_t)n * 4), span(dst, (int64_t)n * 4)};
    const edge_status st = check_pool(caches, num_caches, page_bytes, num_pages, n, lists, 2);
    if (st != EDGE_OK) return st;
    if (n == 0 || num_caches == 0 || num_pages == 0) return EDGE_OK;
    const edge::PagePool pool{caches, num_caches, num_pages, page_bytes};
    return finish(edge::launch_pages_copy(pool, src, dst, n, static_cast<cudaStream_t>(stream)));
}

edge_status edge_pages_free(int32_t* block_table, int32_t num_seqs, int32_t max_pages,
                            int32_t* lens, int32_t* refs, int32_t num_pages, const int32_t* seqs,
                            int32_t n, void* stream) {
    if (num_seqs < 0 || max_pages < 0 || num_pages < 0 || n < 0) return EDGE_ERR_SHAPE;
    if (n > 0 && (seqs == nullptr || (num_seqs > 0 && lens == nullptr) ||
                  (num_pages > 0 && refs == nullptr) ||
                  (num_seqs > 0 && max_pages > 0 && block_table == nullptr))) {
        return EDGE_ERR_NULL;
    }
    int64_t t_b = 0;
    if (!checked_bytes(num_seqs, max_pages, 4, &t_b)) return EDGE_ERR_SHAPE;
    if (!aligned(block_table, 4) || !aligned(lens, 4) || !aligned(refs, 4) || !aligned(seqs, 4)) {
        return EDGE_ERR_ALIGN;
    }
    const Span s[] = {span(block_table, t_b), span(lens, (int64_t)num_seqs * 4),
                      span(refs, (int64_t)num_pages * 4), span(seqs, (int64_t)n * 4)};
    if (any_overlap(s, 4)) return EDGE_ERR_ALIAS;
    if (n == 0 || num_seqs == 0) return EDGE_OK;
    const edge::PageRows rows{block_table, lens, num_seqs, max_pages};
    return finish(edge::launch_pages_free(rows, refs, num_pages, seqs, n,
                                          static_cast<cudaStream_t>(stream)));
}

edge_status edge_pages_fork(void* const* caches, int32_t num_caches, int64_t page_bytes,
                            int32_t num_pages, int32_t page_size, int32_t* block_table,
                            int32_t num_seqs, int32_t max_pages, int32_t* lens, int32_t* refs,
                            const int32_t* parents, const int32_t* children, int32_t n,
                            int32_t* status, int32_t* pairs, void* stream) {
    if (num_seqs < 0 || max_pages < 0 || n < 0 || page_size < 1 || num_pages < 0) {
        return EDGE_ERR_SHAPE;
    }
    if (n > 0 && (parents == nullptr || children == nullptr || status == nullptr ||
                  pairs == nullptr || (num_seqs > 0 && lens == nullptr) ||
                  (num_pages > 0 && refs == nullptr) ||
                  (num_seqs > 0 && max_pages > 0 && block_table == nullptr))) {
        return EDGE_ERR_NULL;
    }
    int64_t t_b = 0;
    if (!checked_bytes(num_seqs, max_pages, 4, &t_b)) return EDGE_ERR_SHAPE;
    if (n > edge::kMaxPageForks || (int64_t)max_pages * page_size > edge::kMaxAttnRows) {
        return EDGE_ERR_UNSUPPORTED;
    }
    if (!aligned(block_table, 4) || !aligned(lens, 4) || !aligned(refs, 4) ||
        !aligned(parents, 4) || !aligned(children, 4) || !aligned(status, 4) || !aligned(pairs, 4)) {
        return EDGE_ERR_ALIGN;
    }
    const int64_t n_b = (int64_t)n * 4;
    const Span s[] = {span(block_table, t_b), span(lens, (int64_t)num_seqs * 4),
                      span(refs, (int64_t)num_pages * 4), span(status, n_b), span(pairs, 2 * n_b),
                      span(parents, n_b), span(children, n_b)};
    // the two lists may be one
    if (any_overlap(s, 6)) return EDGE_ERR_ALIAS;
    for (int i = 0; i < 5; ++i) {
        if (overlap(s[i], s[6])) return EDGE_ERR_ALIAS;
    }
    const edge_status st = check_pool(caches, num_caches, page_bytes, num_pages, n, s, 7);
    if (st != EDGE_OK) return st;
    if (n == 0) return EDGE_OK;
    const edge::PagePool pool{caches, num_caches, num_pages, page_bytes};
    const edge::PageRows rows{block_table, lens, num_seqs, max_pages};
    return finish(edge::launch_pages_fork(pool, rows, page_size, refs, parents, children, n, status,
                                          pairs, static_cast<cudaStream_t>(stream)));
}

int64_t edge_pages_compact_workspace(int32_t num_pages) {
    return num_pages < 0 ? -1 : edge::pages_compact_workspace(num_pages);
}

edge_status edge_pages_compact(void* const* caches, int32_t num_caches, int64_t page_bytes,
                               int32_t num_pages, int32_t* block_table_out,
                               const int32_t* block_table, int32_t num_seqs, int32_t max_pages,
                               int32_t* refs_out, const int32_t* refs, void* workspace,
                               int64_t workspace_bytes, void* stream) {
    if (num_seqs < 0 || max_pages < 0 || num_pages < 0) return EDGE_ERR_SHAPE;
    if (num_pages > 0 && (refs == nullptr || refs_out == nullptr || workspace == nullptr)) {
        return EDGE_ERR_NULL;
    }
    if (num_seqs > 0 && max_pages > 0 && (block_table == nullptr || block_table_out == nullptr)) {
        return EDGE_ERR_NULL;
    }
    int64_t t_b = 0;
    if (!checked_bytes(num_seqs, max_pages, 4, &t_b)) return EDGE_ERR_SHAPE;
    if (num_pages > 0 && workspace_bytes < edge::pages_compact_workspace(num_pages)) {
        return EDGE_ERR_SHAPE;
    }
    if (!aligned(block_table, 4) || !aligned(block_table_out, 4) || !aligned(refs, 4) ||
        !aligned(refs_out, 4) || !aligned(workspace, 16)) {
        return EDGE_ERR_ALIGN;
    }
    const int64_t r_b = (int64_t)num_pages * 4;
    const Span to = span(block_table_out, t_b), ti = span(block_table, t_b);
    const Span ro = span(refs_out, r_b), ri = span(refs, r_b);
    const Span ws = span(workspace, workspace_bytes < 0 ? 0 : workspace_bytes);
    if (bad_alias(to, ti, true) || bad_alias(ro, ri, true) || overlap(to, ro) || overlap(to, ri) ||
        overlap(ti, ro) || overlap(ws, to) || overlap(ws, ti) || overlap(ws, ro) ||
        overlap(ws, ri)) {
        return EDGE_ERR_ALIAS;
    }
    const Span s[] = {to, ti, ro, ri, ws};
    const edge_status st =
        check_pool(caches, num_caches, page_bytes, num_pages, num_pages / 2, s, 5);
    if (st != EDGE_OK) return st;
    if (num_pages == 0) return EDGE_OK;
    const edge::PagePool pool{caches, num_caches, num_pages, page_bytes};
    const edge::PageRows rows{const_cast<int32_t*>(block_table), nullptr, num_seqs, max_pages};
    return finish(edge::launch_pages_compact(pool, block_table_out, rows, refs_out, refs, workspace,
                                             static_cast<cudaStream_t>(stream)));
}

edge_status edge_rmsnorm_q8(void* out, edge_dtype q_dt, float* scales, const void* x,
                            const void* w, edge_dtype dt, int64_t rows, int64_t n, float eps,
                            int weight_offset, void* stream) {
    return rows_q8_entry(out, q_dt, scales, x, nullptr, false, w, true, dt, rows, n, eps,
                         weight_offset, -1, stream);
}

edge_status edge_add_rmsnorm_q8(void* out, edge_dtype q_dt, float* scales, const void* x,
                                void* residual, const void* w, edge_dtype dt, int64_t rows,
                                int64_t n, float eps, int weight_offset, void* stream) {
    return rows_q8_entry(out, q_dt, scales, x, residual, true, w, true, dt, rows, n, eps,
                         weight_offset, -1, stream);
}

edge_status edge_glu_act_q8(void* out, edge_dtype q_dt, float* scales, const void* gate_up,
                            edge_dtype dt, int64_t rows, int64_t n, edge_act act, void* stream) {
    if (act != EDGE_ACT_SILU && act != EDGE_ACT_GELU_TANH) return EDGE_ERR_VALUE;
    return rows_q8_entry(out, q_dt, scales, gate_up, nullptr, false, nullptr, false, dt, rows, n,
                         0.0f, 0, (int)act, stream);
}

edge_status edge_quantize_q8(void* out, edge_dtype q_dt, float* scales, const void* x,
                             edge_dtype dt, int64_t rows, int64_t n, void* stream) {
    return rows_q8_entry(out, q_dt, scales, x, nullptr, false, nullptr, false, dt, rows, n, 0.0f,
                         0, -1, stream);
}

edge_status edge_matmul_q8(void* out, edge_dtype out_dt, const void* a, const void* w,
                           edge_dtype q_dt, const float* a_scales, const float* w_scales,
                           const void* bias, int64_t tokens, int64_t n, int64_t k, void* stream) {
    if (!act_dtype(out_dt) || !q8_dtype(q_dt)) return EDGE_ERR_DTYPE;
    if (out == nullptr || a == nullptr || w == nullptr || a_scales == nullptr ||
        w_scales == nullptr) {
        return EDGE_ERR_NULL;
    }
    if (tokens < 0 || n < 1 || k < 1) return EDGE_ERR_SHAPE;
    if (k > edge::kMaxMatmulK || tokens > edge::kMaxMatmulRows || n > edge::kMaxMatmulRows) {
        return EDGE_ERR_UNSUPPORTED;
    }
    const int64_t es = esize(out_dt);
    if (!aligned(out, es) || !aligned(bias, es) || !aligned(a_scales, 4) || !aligned(w_scales, 4)) {
        return EDGE_ERR_ALIGN;
    }
    // (at most 2^24 rows of 2^24 elements of 4 bytes: no overflow)
    const Span so = span(out, tokens * n * es);
    if (overlap(so, span(a, tokens * k)) || overlap(so, span(w, n * k)) ||
        overlap(so, span(a_scales, 4 * tokens)) || overlap(so, span(w_scales, 4 * n)) ||
        overlap(so, span(bias, n * es))) {
        return EDGE_ERR_ALIAS;
    }
    if (tokens == 0) return EDGE_OK;

    edge::MatmulQ8Args m;
    m.a = a;
    m.w = w;
    m.a_scales = a_scales;
    m.w_scales = w_scales;
    m.bias = bias;
    m.out = out;
    m.tokens = tokens;
    m.n = n;
    m.k = k;
    m.q_dt = (int)q_dt;
    m.out_dt = (int)out_dt;
    return finish(edge::launch_matmul_q8(m, static_cast<cudaStream_t>(stream)));
}

edge_status edge_copy(void* dst, const void* src, int64_t bytes, void* stream) {
    if (dst == nullptr || src == nullptr) return EDGE_ERR_NULL;
    if (bytes < 0) return EDGE_ERR_SHAPE;
    if (overlap(span(dst, bytes), span(src, bytes))) return EDGE_ERR_ALIAS;
    if (bytes == 0) return EDGE_OK;
    return finish(edge::launch_copy(dst, src, bytes, static_cast<cudaStream_t>(stream)));
}

const char* edge_status_str(edge_status status) {
    switch (status) {
        case EDGE_OK: return "ok";
        case EDGE_ERR_NULL: return "a required pointer is NULL";
        case EDGE_ERR_DTYPE: return "unsupported dtype combination";
        case EDGE_ERR_SHAPE: return "invalid or inconsistent sizes";
        case EDGE_ERR_ALIGN: return "pointer not aligned to its element size";
        case EDGE_ERR_ALIAS: return "a written buffer overlaps another buffer";
        case EDGE_ERR_UNSUPPORTED: return "valid call beyond this build's limits";
        case EDGE_ERR_CUDA: return "CUDA launch failed";
        case EDGE_ERR_VALUE: return "invalid scalar argument";
        default: return "unknown status";
    }
}

int edge_last_cuda_error(void) { return g_last_cuda_error; }

int edge_version(void) { return 100; }

}  // extern "C"
