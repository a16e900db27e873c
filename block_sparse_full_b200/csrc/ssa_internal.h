// Internal declarations shared by the host-side translation units of libssa.
// Kernels live in their own .cu files; each exposes one host launcher here.
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

#include "ssa.h"

namespace ssa {

// Records a detail message for ssa_last_error() and returns `status`.
int fail(int status, const char* fmt, ...);

// Turns a pending launch/runtime error into SSA_ERR_CUDA (with detail).
int check_launch(const char* what);

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Shared memory a CTA may hold on sm_100 (227 KB).
constexpr size_t kMaxSmemPerCta = 232448;

// Lets kernel K take dynamic shared memory up to the per-CTA maximum less its
// static shared memory (once per process and device; launches above the default
// 48 KB of dynamic plus static shared memory fail without it).  Call it before
// any stream capture.  Returns an SSA status; *dyn_limit receives the limit.
template <auto K>
int opt_in_max_smem(const char* what, size_t* dyn_limit = nullptr) {
    constexpr int kDevices = 64;
    struct State {
        std::once_flag once;
        cudaError_t err = cudaSuccess;
        size_t limit = 0;
    };
    static State states[kDevices];
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail(SSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    if (dev >= kDevices) return fail(SSA_ERR_UNSUPPORTED, "%s: device %d of more than %d", what, dev, kDevices);
    State& s = states[dev];
    std::call_once(s.once, [&s] {
        cudaFuncAttributes fa;
        s.err = cudaFuncGetAttributes(&fa, K);
        if (s.err == cudaSuccess) {
            s.limit = kMaxSmemPerCta - fa.sharedSizeBytes;
            s.err = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s.limit);
        }
    });
    if (dyn_limit) *dyn_limit = s.limit;
    if (s.err != cudaSuccess)
        return fail(SSA_ERR_CUDA, "%s: shared memory attribute: %s", what, cudaGetErrorString(s.err));
    return SSA_OK;
}

// Launch that may begin while the kernel before it in the stream still runs; the
// kernel itself waits (griddepcontrol.wait) before it touches that one's results.
// cluster: CTAs of a cluster, along x.
template <typename... Params, typename... Args>
int launch_beside_clusters(const char* what, void (*kernel)(Params...), dim3 grid, unsigned cluster, unsigned threads,
                           size_t smem, cudaStream_t s, const Args&... args) {
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&c, kernel, args...);
    if (e != cudaSuccess) return fail(SSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return check_launch(what);
}
template <typename... Params, typename... Args>
int launch_beside(const char* what, void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s,
                  const Args&... args) {
    return launch_beside_clusters(what, kernel, grid, 1u, threads, smem, s, args...);
}

// Wall-clock limit of the kernels' bounded waits (default 2 s; tests shorten it).
unsigned long long wait_limit_ns();
// Under this limit the window and prefix kernels on the tensor cores set up the
// barrier of the scores with one arrival more than it gets, so that the waits for
// them do run out (ssa_debug_set_wait_limit_ns).
constexpr unsigned long long kLostScoresNs = 1;

// Byte budget of the tensor-core backward's dS workspace (default 4 GiB;
// tests shrink it so that small problems run in several head groups).
unsigned long long ds_budget_bytes();

// Measurement hook (ssa_debug_set_kernel_events): records caller event i on
// stream s when the hook is enabled, else does nothing.
constexpr int kKernelEvents = 4;
void mark_kernel_event(int i, cudaStream_t s);

inline size_t num_rows(const ssa_params_t& p) {
    return (size_t)p.B * p.H * p.T;
}
inline size_t num_elems(const ssa_params_t& p) { return num_rows(p) * p.D; }
inline int num_blocks(const ssa_params_t& p) { return p.T / p.block; }
inline int mask_words(const ssa_params_t& p) { return (num_blocks(p) + 31) / 32; }

// ---- selection (select.cu)
size_t select_workspace(const ssa_params_t& p);
int launch_select(const ssa_params_t& p, const void* q, const void* k, int32_t* idx,
                  int32_t* cnt, uint32_t* mask, void* ws, cudaStream_t s);

// ---- forward, CUDA-core path (fwd_simt.cu)
int launch_fwd_simt(const ssa_params_t& p, const void* q, const void* k, const void* v,
                    const uint32_t* mask, void* h_full, void* h_sparse, float* delta,
                    float* lse_full, float* lse_sparse, float* sqdiff, cudaStream_t s);

// ---- forward, tcgen05 path (fwd_tc.cu)
bool fwd_tc_supported(const ssa_params_t& p);
size_t fwd_tc_workspace(const ssa_params_t& p);
int launch_fwd_tc(const ssa_params_t& p, const void* q, const void* k, const void* v,
                  const uint32_t* mask, void* h_full, void* h_sparse, float* delta,
                  float* lse_full, float* lse_sparse, float* sqdiff, float* sink, void* ws,
                  cudaStream_t s);  // sink: optional block-0 mass per row
int fwd_tc_take_status(cudaStream_t s);  // SSA_ERR_TIMEOUT if a wait expired
// the sparse stream alone (inference): h_sparse and lse_sparse only
int launch_fwd_sparse_tc(const ssa_params_t& p, const void* q, const void* k, const void* v,
                         const uint32_t* mask, void* h_sparse, float* lse_sparse, cudaStream_t s);

// ---- decode over a key/value cache (decode.cu)
size_t decode_workspace(const ssa_params_t& p);
int launch_decode_pool(const ssa_params_t& p, int j0, int j1, const void* k, double* kbar,
                       cudaStream_t s);
int launch_decode_step(const ssa_params_t& p, int t, const void* q, const void* k, const void* v,
                       const double* kbar, void* h, float* lse, int32_t* idx, void* ws,
                       cudaStream_t s);

// ---- attention diagnostics (diag.cu)
int launch_diagnostics(const ssa_params_t& p, const void* q, const void* k, const float* lse_full,
                       const float* delta, float* sink, float* stats, cudaStream_t s);
// per-head means of delta and of the sink mass from the row vectors (fixed-order float64)
int launch_diag_heads(const ssa_params_t& p, const float* delta, const float* sink, float* stats,
                      cudaStream_t s);

// ---- alignment loss (loss.cu)
size_t loss_workspace(const ssa_params_t& p);
int launch_loss(const ssa_params_t& p, const float* sqdiff, float w_s, float w_c,
                float* loss_out, void* ws, cudaStream_t s);

// ---- backward, CUDA-core path (bwd_simt.cu)
size_t bwd_simt_workspace(const ssa_params_t& p);
int launch_bwd_simt(const ssa_params_t& p, const void* q, const void* k, const void* v,
                    const uint32_t* mask, const void* h_full, const void* h_sparse,
                    const float* lse_full, const float* lse_sparse, const void* dh_full,
                    const void* dh_sparse, float w_s, float w_c, void* dq, void* dk,
                    void* dv, void* ws, cudaStream_t s);

// ---- backward, tcgen05 path (bwd_tc.cu)
bool bwd_tc_supported(const ssa_params_t& p);
size_t bwd_tc_workspace(const ssa_params_t& p);
int launch_bwd_tc(const ssa_params_t& p, const void* q, const void* k, const void* v,
                  const uint32_t* mask, const void* h_full, const void* h_sparse,
                  const float* lse_full, const float* lse_sparse, const void* dh_full,
                  const void* dh_sparse, float w_s, float w_c, void* dq, void* dk, void* dv,
                  void* ws, cudaStream_t s);
int bwd_tc_take_status(cudaStream_t s);  // SSA_ERR_TIMEOUT if a wait expired
int bwd_tc_heads_per_group(const ssa_params_t& p);  // heads sharing the dS workspace

// ---- paged cache and window attention
// A checked ssa_view_t (data NULL: an optional tensor that is absent).
struct View {
    void* data;
    long long sb, sh, st;  // strides in elements: batch, head, token
};

// appending to a paged cache (cache_append.cu)
int launch_cache_append(const ssa_cache_params_t& p, int n, const View& k, const View& v, const View& q,
                        void* k_pages, void* v_pages, const int32_t* table, const int32_t* lens,
                        int32_t* new_lens, const int32_t* q_start, const double* inv_freq, int rot,
                        int interleaved, int pos_offset, const View& q_out, const View& k_out,
                        cudaStream_t s);
int append_take_status();  // SSA_ERR_INVALID_ARG if a length, slot or page was out of range

// single tokens over a paged cache, with or without a shared prefix (paged_decode.cu)
size_t paged_decode_workspace(const ssa_cache_params_t& p, int prefix_len);
int launch_paged_decode(const ssa_cache_params_t& p, const View& q, const void* k_pages, const void* v_pages,
                        const int32_t* prefix_pages, int prefix_len, const int32_t* table,
                        const int32_t* lens, const View& h, float* lse, void* ws, cudaStream_t s);
int paged_take_status();  // SSA_ERR_INVALID_ARG if a length or page was out of range

// sliding-window attention over sequences, CUDA-core path (window_simt.cu)
int launch_window_fwd_simt(const ssa_window_params_t& p, const View& q, const View& k, const View& v,
                           const int32_t* lens, const View& h, float* lse, cudaStream_t s);
size_t window_bwd_simt_workspace(const ssa_window_params_t& p);
int launch_window_bwd_simt(const ssa_window_params_t& p, const View& q, const View& k, const View& v,
                           const int32_t* lens, const View& h, const float* lse, const View& dh,
                           const View& dq, const View& dk, const View& dv, void* ws, cudaStream_t s);
// the same on the tensor cores (window_fwd_tc.cu)
bool window_tc_supported(const ssa_window_params_t& p);
int launch_window_fwd_tc(const ssa_window_params_t& p, const View& q, const View& k, const View& v,
                         const int32_t* lens, const View& h, float* lse, cudaStream_t s);
bool window_bwd_tc_supported(const ssa_window_params_t& p);  // (window_bwd_tc.cu)
size_t window_bwd_tc_workspace(const ssa_window_params_t& p);
int launch_window_bwd_tc(const ssa_window_params_t& p, const View& q, const View& k, const View& v,
                         const int32_t* lens, const View& h, const float* lse, const View& dh, const View& dq,
                         const View& dk, const View& dv, void* ws, cudaStream_t s);
int window_bwd_take_status();  // SSA_ERR_TIMEOUT, or SSA_ERR_INVALID_ARG as below
// the pass of a batch over its shared prefix on the tensor cores (window_fwd_tc.cu):
// `splits` partials for each of Hkv x ntq row tiles of nb batch entries, 128 rows of D
// outputs, then 128 (maximum, sum) pairs, float32
struct PrefixPlan {
    int splits, ntq, nb;
    size_t bytes;
};
bool prefix_tc_supported(const ssa_cache_params_t& p);
PrefixPlan prefix_tc_plan(const ssa_cache_params_t& p, int prefix_len);
int launch_prefix_tc(const ssa_cache_params_t& p, const View& q, const void* k_pages, const void* v_pages,
                     const int32_t* prefix_pages, int prefix_len, void* ws, cudaStream_t s);
int attn_tc_take_status();  // SSA_ERR_TIMEOUT, or SSA_ERR_INVALID_ARG as below
int window_take_status();  // SSA_ERR_INVALID_ARG if a length was out of range

// ---- self-tests (selftest.cu)
int select_take_status();  // SSA_ERR_TIMEOUT if a pooling wait expired
int decode_take_status();  // SSA_ERR_TIMEOUT if a decode-step wait expired
int selftest_take_status();  // SSA_ERR_TIMEOUT if the self-test wait expired

}  // namespace ssa
