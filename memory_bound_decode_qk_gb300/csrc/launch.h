// launch.h -- internal interface between the C ABI layer and the kernels.
// Arguments arrive here validated; each launcher picks a kernel and launch
// shape for its op and enqueues it on the caller's stream.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace edge {

enum Dt { kF32 = 0, kF16 = 1, kBF16 = 2, kFP8 = 3, kInt8 = 4 };

// Rotary positions with several axes: pair j of the rotary channels turns by
// the position of its axis.  n = 0: one position per token.
struct Axes {
    int n;          // axes, 0 or 1 .. 4
    int cycled;     // pairs dealt in turn instead of in blocks
    int count[4];   // pairs of each axis
};

struct QKArgs {
    const void* q;
    const void* k;
    void* q_out;
    void* k_out;
    const void* wq;          // nullable
    const void* wk;          // nullable
    const int64_t* pos;      // nullable when no rotation can happen
    const float* cos;
    const float* sin;
    int64_t tokens;
    int64_t cache_len;
    int q_heads, k_heads, head_dim, rotary_dim, layout;
    int dt, out_dt;
    float eps, inv_scale;
    int weight_offset;
    int mode;                // kModeNorm (1) | kModeUnrounded (2), qk_common.cuh
    Axes axes;
};

struct RowsArgs {
    const void* x;
    void* residual;          // nullptr: plain RMSNorm
    const void* w;           // nullable (LayerNorm: gamma)
    const void* beta;        // LayerNorm only, nullable
    int layernorm;           // 1: LayerNorm (no residual)
    void* out;
    int64_t rows;
    int64_t hidden;
    int dt, out_dt;
    float eps, inv_scale;
    int weight_offset;
};

struct GluArgs {
    const void* gate_up;
    void* out;
    int64_t rows;
    int64_t d;
    int dt, out_dt, act;
    float inv_scale;
};

// Launch-shape limits of the paths, checked by the ABI layer.
constexpr int64_t kMaxQKHeadDim = 2048;       // generic prologue path (smem per warp)
constexpr int64_t kMaxHidden = int64_t(1) << 24;  // row length, exact as fp32
constexpr int64_t kMaxUnits = (int64_t(1) << 31) - 1;

cudaError_t launch_qk(const QKArgs& a, cudaStream_t s);
cudaError_t launch_rows(const RowsArgs& a, cudaStream_t s);
cudaError_t launch_glu(const GluArgs& a, cudaStream_t s);

struct QKVArgs {
    const void* qkv;
    void* q_out;
    void* k_cache;
    void* v_cache;
    const void* wq;          // nullable
    const void* wk;          // nullable
    const int64_t* pos;
    const float* cos;
    const float* sin;
    const int64_t* slots;
    int64_t tokens, cache_len, num_slots;
    int q_heads, kv_heads, head_dim, rotary_dim, layout, dt;
    int normalize, weight_offset;
    float eps;
    Axes axes;
};
// *handled is false when the geometry or alignment has no vector path.
cudaError_t launch_qkv_cache(const QKVArgs& a, cudaStream_t s, bool* handled);

struct QuantArgs {
    const void* x;
    void* out;
    int64_t n;
    int dt;
    float inv_scale;
};
cudaError_t launch_quant(const QuantArgs& a, cudaStream_t s);

// Rows in 8 bits with a scale each (rows_q8.cu).
struct RowsQ8Args {
    const void* x;           // the gate: [rows, 2 n]
    void* residual;          // nullptr: no residual
    const void* w;           // norms, nullable
    void* out;
    float* scales;
    int64_t rows, n;
    int dt, out_dt;
    int norm;                // 1: RMSNorm
    int act;                 // -1: no gate
    float eps;
    int weight_offset;
};
cudaError_t launch_rows_q8(const RowsQ8Args& a, cudaStream_t s);

// Product of 8-bit operands with scales (matmul_q8.cu).
struct MatmulQ8Args {
    const void* a;
    const void* w;
    const float* a_scales;
    const float* w_scales;
    const void* bias;        // nullable
    void* out;
    int64_t tokens, n, k;
    int q_dt, out_dt;
};
constexpr int64_t kMaxMatmulK = 131071;   // int8 sums stay below 2^31
constexpr int64_t kMaxMatmulRows = int64_t(1) << 24;  // tokens, n
cudaError_t launch_matmul_q8(const MatmulQ8Args& a, cudaStream_t s);

// Attention over a paged KV cache (paged_attn.cu).
struct AttnArgs {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    void* out;
    float* lse;              // nullable
    const int32_t* table;
    const int32_t* lens;
    const int32_t* starts;   // nullable: one token per sequence
    void* workspace;
    int64_t tokens;
    int q_heads, kv_heads, head_dim;
    int num_seqs, max_pages, num_pages, page_size;
    int dt, out_dt, causal, window;
    float scale, inv_scale;
};
constexpr int64_t kMaxAttnHeadDim = 256;
constexpr int64_t kMaxAttnRows = int64_t(1) << 30;  // tokens * q_heads, max_pages * page_size
int64_t attn_workspace(int dt, int q_heads, int kv_heads, int head_dim);
cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s);

// Pages of a KV cache (pages.cu).
struct PagePool {
    void* const* caches;     // host array of device pointers
    int num_caches, num_pages;
    int64_t page_bytes;
};
struct PageRows {
    int32_t* table;          // [num_seqs, max_pages]
    int32_t* lens;           // [num_seqs]
    int num_seqs, max_pages;
};
constexpr int64_t kMaxPageForks = 8192;   // of one call
constexpr int64_t kMaxPagePairs = 65536;  // each pair is held against all of a call
bool pages_fit(int64_t page_bytes, int64_t pairs);
int64_t pages_compact_workspace(int num_pages);
cudaError_t launch_pages_copy(const PagePool& pool, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t s);
cudaError_t launch_pages_free(const PageRows& r, int32_t* refs, int num_pages,
                              const int32_t* seqs, int n, cudaStream_t s);
cudaError_t launch_pages_fork(const PagePool& pool, const PageRows& r, int page_size,
                              int32_t* refs, const int32_t* parents, const int32_t* children,
                              int n, int32_t* status, int32_t* pairs, cudaStream_t s);
cudaError_t launch_pages_compact(const PagePool& pool, int32_t* table_out, const PageRows& r,
                                 int32_t* refs_out, const int32_t* refs, void* workspace,
                                 cudaStream_t s);

// The yardstick copy (copy.cu): bytes from src to dst, validated.
cudaError_t launch_copy(void* dst, const void* src, int64_t bytes, cudaStream_t s);

// Streaming multiprocessors of the current device (cached per device).
int sm_count();

// CTAs of kernel `fn` resident per SM at `threads` threads and no dynamic
// shared memory (the occupancy calculator, cached per kernel and device).
int resident_ctas(const void* fn, int threads);

// Clusters of `n` CTAs of kernel `fn` resident at the same time, launched as `cfg`
// says (the occupancy calculator, cached per kernel, size and device); 0 if it cannot be
// asked just now.
int resident_clusters(const void* fn, const cudaLaunchConfig_t& cfg, int n);

// Registers of a thread of kernel `fn` (cached per kernel and device).  An error if the
// runtime does not say just now.
cudaError_t kernel_registers(const void* fn, int* registers);

// Lets kernel `fn` use `bytes` of dynamic shared memory (asked of the runtime
// once per kernel and device).
cudaError_t allow_smem(const void* fn, int bytes);

// Programmatic dependent launch for all ops (on unless EDGE_OPS_PDL=0 in the
// environment, read once per process).  Every kernel executes
// griddepcontrol.wait before its first global load whose value it uses, so
// it is always safe as a dependent; it triggers its own dependents at its
// start.
bool pdl_enabled();

}  // namespace edge
