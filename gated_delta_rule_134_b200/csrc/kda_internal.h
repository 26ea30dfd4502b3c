// Internal launch interface between the C-ABI layer and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include <atomic>

#include "kda.h"

namespace kda {

// Raises a kernel's limit of dynamic shared memory once a device (a bit each in
// `raised`, a static of the caller for this kernel; devices past 63 every time).
template <typename Kernel>
inline cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<unsigned long long>& raised) {
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err != cudaSuccess) return err;
    const unsigned long long bit = device < 64 ? 1ull << device : 0;
    if (raised.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess) raised.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

struct ChunkArgs {
    const void *q, *k, *v, *log_alpha, *beta;
    const float* S0;
    void* o;
    float* ST;
    int B, T, H, dk, dv, chunk;
    int bf16;
    int erase;  // 1: delta-rule family (I - beta k k^T), 0: additive write beta k v^T
    int gate;   // 0: log_alpha per key channel [.., dk]; 1: one per token and head [B, T, H]; 2: none
    // Packed variable-length sequences (NULL: dense [B, T, H, .] batch). When
    // set, B is the number of sequences, T the packed token count, and
    // sequence b owns tokens [cu_seqlens[b], cu_seqlens[b+1]) of the [1, T, H, .]
    // tensors; kernels clamp the offsets into [0, T].
    const int* cu_seqlens;
    void* workspace;
    size_t workspace_bytes;
    // Fault injection for the timeout test (tensor-core prefill only): withhold
    // the first k/q load of every CTA and bound each wait by this many SM
    // cycles, so the first wait expires. Zero in every other call.
    int test_withhold_first_load = 0;
    long long test_wait_budget = 0;
};

// Synchronous argument validation shared by every prefill entry point
// (sizes, dtype, head and chunk sizes, variant switches, required pointers
// and their 16-byte alignment). Launches nothing.
kda_status_t check_chunk_args(const ChunkArgs& a, kda_dtype_t dtype);

cudaError_t launch_decode(const void* q, const void* k, const void* v, const void* la, const void* beta,
                          const float* S_in, float* S_out, void* o, int N, int H, int dk, int dv, int bf16,
                          int erase, int gate, cudaStream_t stream);

cudaError_t launch_chunk_simt(const ChunkArgs& a, cudaStream_t stream);

// Fused tensor-core prefill (bf16, dk = dv = 128, chunk = 64).
bool chunk_tc_supported(const ChunkArgs& a);
// scan_mode: 0 one pass per sequence; 1 the chunk-parallel segment scan where
// it pays (dense batch, few heads, long T); 2 the scan whenever T has 3 chunks.
size_t chunk_tc_workspace_bytes(const ChunkArgs& a, int scan_mode);
cudaError_t launch_chunk_tc(const ChunkArgs& a, int scan_mode, cudaStream_t stream);

// Backward of the chunkwise prefill (SIMT fp32, any variant, dk = dv = d in {64, 128}).
struct BwdArgs {
    const void *q, *k, *v, *log_alpha, *beta, *dO;
    const float *S0, *dST;
    void *g_q, *g_k, *g_v, *g_log_alpha, *g_beta;  // gradients (input dtype)
    float* g_S0;
    int B, T, H, d, bf16, erase, gate;
    int mode;  // 0: keep every chunk's state while that fits 16 GB; 1: always; 2: one per 64 tokens
    void* workspace;
    size_t workspace_bytes;
};
size_t chunk_bwd_workspace_bytes(int B, int T, int H, int d, int mode);
cudaError_t launch_chunk_bwd(const BwdArgs& a, cudaStream_t stream);

// Gated linear recurrence h_t = exp(log_alpha_t) h_{t-1} + x_t. Dense [N, T, D],
// or packed [T, D] with cu_seqlens [N + 1].
struct RecurrenceArgs {
    const void *log_alpha, *x;  // backward: x is the gradient of h
    const void* h_fwd;          // backward: the forward pass's h
    const float *state0;        // forward: h0; backward: d_h_T (the state the reverse recurrence starts from)
    const float* h0;            // backward: h0, the h_{t-1} of a first token
    void *out, *out_la;         // forward: h; backward: d_x, d_log_alpha
    float* state_end;           // forward: h_T; backward: d_h0
    const int* cu_seqlens;
    int N, T, D, bf16;
    long long wait_cycles = 1ll << 31;  // SM cycles that a wait within a cluster lasts at most: about a second
    int test_withhold = 0;              // fault injection: the first CTA of a cluster sends nothing
};
// Tokens of a sequence, of a packed batch on average (T and N reach 2^31 and 2^26: their sum leaves int).
inline long long tokens_of(const RecurrenceArgs& a) { return a.cu_seqlens ? ((long long)a.T + a.N - 1) / a.N : a.T; }
// Whether a wait gave up on the current device since the last call; clears it.
cudaError_t recurrence_late(unsigned* flag);
cudaError_t launch_recurrence_fwd(const RecurrenceArgs& a, cudaStream_t stream);
cudaError_t launch_recurrence_bwd(const RecurrenceArgs& a, cudaStream_t stream);
cudaError_t launch_recurrence_step(const void* la, const void* x, const float* h_in, float* h_out, void* y,
                                   long long cells, int bf16, cudaStream_t stream);

// Per-head norm of queries and keys with the position rotation.
struct QkArgs {
    const void *q, *k, *q_weight, *k_weight;
    const float *cos, *sin;
    const void* positions;  // NULL: no rotation
    int pos_bytes;
    const void *d_q_out, *d_k_out;  // backward only
    void *q_out, *k_out;            // backward: d_q, d_k
    float *d_q_weight, *d_k_weight;
    int n, Hq, Hk, d, rot, max_pos;
    long long q_stride_t, q_stride_h, k_stride_t, k_stride_h;
    int norm;
    float eps, q_scale;
    int interleaved, bf16;
    void* workspace;
};
size_t qk_norm_rope_bwd_workspace_bytes(int n, int Hq, int Hk, int d);
cudaError_t launch_qk_norm_rope(const QkArgs& a, cudaStream_t stream);
cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, cudaStream_t stream);

// One new token's attention over a paged key-value cache.
struct AttnDecodeArgs {
    const void *q, *k_new, *v_new;
    void *k_cache, *v_cache;
    const int *page_table, *seq_lens;
    void* o;
    float* lse;
    int N, Hq, Hk, d, n_pages, page_size, max_pages, window;
    float scale;
    int bf16;
    void* workspace;
};
size_t attn_decode_workspace_bytes(int N, int Hq, int Hk, int d);
cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t stream);

}  // namespace kda
