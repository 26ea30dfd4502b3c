// C-ABI layer of libkda.so: argument validation, workspace sizing and
// dispatch to the kernels. Declarations and contracts are in include/kda.h.
#include <stdint.h>

#include "kda.h"
#include "kda_internal.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool head_dims_ok(int dk, int dv) { return dk == dv && (dk == 64 || dk == 128); }

// 0: one pass per sequence; 1: the segment scan where it pays; 2: the scan forced.
int scan_mode_of(kda_algo_t algo) { return algo == KDA_ALGO_TC_SCAN ? 2 : (algo == KDA_ALGO_AUTO ? 1 : 0); }

kda_status_t run_chunk(const kda::ChunkArgs& a, kda_dtype_t dtype, kda_algo_t algo, void* stream);

}  // namespace

kda_status_t kda::check_chunk_args(const kda::ChunkArgs& a, kda_dtype_t dtype) {
    if (a.B < 0 || a.T < 0 || a.H < 0) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (!head_dims_ok(a.dk, a.dv)) return KDA_ERR_UNSUPPORTED;
    if (a.chunk != 16 && a.chunk != 32 && a.chunk != 64) return KDA_ERR_UNSUPPORTED;
    if ((long long)a.B * a.H > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
    if (a.erase != 0 && a.erase != 1) return KDA_ERR_INVALID_ARG;
    if (a.gate < KDA_GATE_CHANNEL || a.gate > KDA_GATE_NONE) return KDA_ERR_INVALID_ARG;
    const bool has_tokens = (long long)a.B * a.T * a.H > 0;
    if (has_tokens) {
        const void* req[] = {a.q, a.k, a.v, a.beta, a.o};
        for (const void* p : req)
            if (p == nullptr || !aligned16(p)) return KDA_ERR_INVALID_ARG;
        if (a.gate != KDA_GATE_NONE && (a.log_alpha == nullptr || !aligned16(a.log_alpha)))
            return KDA_ERR_INVALID_ARG;
    }
    if (a.S0 && !aligned16(a.S0)) return KDA_ERR_INVALID_ARG;
    if (a.ST && !aligned16(a.ST)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

extern "C" {

const char* kda_status_string(kda_status_t s) {
    switch (s) {
        case KDA_OK: return "KDA_OK";
        case KDA_ERR_INVALID_ARG: return "KDA_ERR_INVALID_ARG: null/misaligned pointer, bad size or workspace too small";
        case KDA_ERR_UNSUPPORTED: return "KDA_ERR_UNSUPPORTED: head size, chunk size or algorithm not implemented";
        case KDA_ERR_CUDA: return "KDA_ERR_CUDA: CUDA launch or query failed";
        case KDA_ERR_TIMEOUT: return "KDA_ERR_TIMEOUT: a bounded device-side wait expired";
    }
    return "KDA: unknown status";
}

size_t kda_chunk_fwd_workspace_size(int B, int T, int H, int dk, int dv, int chunk, kda_dtype_t dtype,
                                    kda_algo_t algo) {
    kda::ChunkArgs a{};
    a.B = B; a.T = T; a.H = H; a.dk = dk; a.dv = dv; a.chunk = chunk; a.bf16 = dtype == KDA_BF16;
    a.erase = 1; a.gate = KDA_GATE_CHANNEL; a.cu_seqlens = nullptr;
    if (B < 0 || T < 0 || H < 0 || !head_dims_ok(dk, dv)) return 0;
    const bool tc = (algo == KDA_ALGO_TC) || (algo == KDA_ALGO_TC_SCAN) ||
                    (algo == KDA_ALGO_AUTO && kda::chunk_tc_supported(a));
    return tc ? kda::chunk_tc_workspace_bytes(a, scan_mode_of(algo)) : 0;
}

kda_status_t kda_chunk_fwd_v(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                             const float* S0, void* o, float* S_T, int B, int T, int H, int dk, int dv, int chunk,
                             kda_dtype_t dtype, int erase, kda_gate_t gate, void* workspace, size_t workspace_bytes,
                             kda_algo_t algo, void* stream) {
    kda::ChunkArgs a;
    a.q = q; a.k = k; a.v = v; a.log_alpha = log_alpha; a.beta = beta; a.S0 = S0; a.o = o; a.ST = S_T;
    a.B = B; a.T = T; a.H = H; a.dk = dk; a.dv = dv; a.chunk = chunk; a.bf16 = dtype == KDA_BF16;
    a.erase = erase; a.gate = (int)gate;
    a.cu_seqlens = nullptr;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes;
    return run_chunk(a, dtype, algo, stream);
}

kda_status_t kda_chunk_fwd_varlen(const void* q, const void* k, const void* v, const void* log_alpha,
                                  const void* beta, const float* S0, void* o, float* S_T, const int* cu_seqlens,
                                  int N, int total_T, int H, int dk, int dv, int chunk, kda_dtype_t dtype, int erase,
                                  kda_gate_t gate, void* workspace, size_t workspace_bytes, kda_algo_t algo,
                                  void* stream) {
    if (N < 0 || total_T < 0) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (cu_seqlens == nullptr || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0))
        return KDA_ERR_INVALID_ARG;
    kda::ChunkArgs a;
    a.q = q; a.k = k; a.v = v; a.log_alpha = log_alpha; a.beta = beta; a.S0 = S0; a.o = o; a.ST = S_T;
    a.B = N; a.T = total_T; a.H = H; a.dk = dk; a.dv = dv; a.chunk = chunk; a.bf16 = dtype == KDA_BF16;
    a.erase = erase; a.gate = (int)gate;
    a.cu_seqlens = cu_seqlens;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes;
    return run_chunk(a, dtype, algo, stream);
}

}  // extern "C"

namespace {

kda_status_t run_chunk(const kda::ChunkArgs& a, kda_dtype_t dtype, kda_algo_t algo, void* stream) {
    const int B = a.B, T = a.T, H = a.H, dk = a.dk, dv = a.dv;
    void* workspace = a.workspace;
    const size_t workspace_bytes = a.workspace_bytes;
    kda_status_t st = kda::check_chunk_args(a, dtype);
    if (st != KDA_OK) return st;
    if (algo != KDA_ALGO_AUTO && algo != KDA_ALGO_SIMT && algo != KDA_ALGO_TC && algo != KDA_ALGO_TC_SCAN)
        return KDA_ERR_INVALID_ARG;
    const bool tc = (algo == KDA_ALGO_TC) || (algo == KDA_ALGO_TC_SCAN) ||
                    (algo == KDA_ALGO_AUTO && kda::chunk_tc_supported(a));
    if (tc && !kda::chunk_tc_supported(a)) return KDA_ERR_UNSUPPORTED;
    if (algo == KDA_ALGO_TC_SCAN && a.cu_seqlens) return KDA_ERR_UNSUPPORTED;
    if (tc) {
        const size_t need = kda::chunk_tc_workspace_bytes(a, scan_mode_of(algo));
        if (need > 0 && (workspace == nullptr || workspace_bytes < need ||
                         (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
            return KDA_ERR_INVALID_ARG;
    }
    if ((long long)B * H == 0) return KDA_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t err = tc ? kda::launch_chunk_tc(a, scan_mode_of(algo), s) : kda::launch_chunk_simt(a, s);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

extern "C" {

kda_status_t kda_chunk_fwd_ex(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                              const float* S0, void* o, float* S_T, int B, int T, int H, int dk, int dv, int chunk,
                              kda_dtype_t dtype, void* workspace, size_t workspace_bytes, kda_algo_t algo,
                              void* stream) {
    return kda_chunk_fwd_v(q, k, v, log_alpha, beta, S0, o, S_T, B, T, H, dk, dv, chunk, dtype, 1, KDA_GATE_CHANNEL,
                           workspace, workspace_bytes, algo, stream);
}

kda_status_t kda_chunk_fwd(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                           const float* S0, void* o, float* S_T, int B, int T, int H, int dk, int dv, int chunk,
                           kda_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
    return kda_chunk_fwd_ex(q, k, v, log_alpha, beta, S0, o, S_T, B, T, H, dk, dv, chunk, dtype, workspace,
                            workspace_bytes, KDA_ALGO_AUTO, stream);
}

kda_status_t kda_chunk_fwd_timeout_test(const void* q, const void* k, const void* v, const void* log_alpha,
                                       const void* beta, const float* S0, void* o, float* S_T, int B, int T, int H,
                                       int dk, int dv, int chunk, kda_dtype_t dtype, void* workspace,
                                       size_t workspace_bytes, long long wait_budget_cycles, void* stream) {
    if (wait_budget_cycles <= 0 || wait_budget_cycles > (1ll << 31)) return KDA_ERR_INVALID_ARG;
    kda::ChunkArgs a;
    a.q = q; a.k = k; a.v = v; a.log_alpha = log_alpha; a.beta = beta; a.S0 = S0; a.o = o; a.ST = S_T;
    a.B = B; a.T = T; a.H = H; a.dk = dk; a.dv = dv; a.chunk = chunk; a.bf16 = dtype == KDA_BF16;
    a.erase = 1;
    a.gate = KDA_GATE_CHANNEL;
    a.cu_seqlens = nullptr;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes;
    a.test_withhold_first_load = 1;
    a.test_wait_budget = wait_budget_cycles;
    // Only the single-pass tensor-core kernel has the waits this exercises.
    if (T == 0) return KDA_ERR_INVALID_ARG;
    return run_chunk(a, dtype, KDA_ALGO_TC, stream);
}

kda_status_t kda_workspace_status(const void* workspace, size_t workspace_bytes, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return KDA_ERR_CUDA;
    if (workspace == nullptr || workspace_bytes < sizeof(unsigned)) return KDA_OK;
    unsigned flag = 0;
    if (cudaMemcpy(&flag, workspace, sizeof(flag), cudaMemcpyDeviceToHost) != cudaSuccess) return KDA_ERR_CUDA;
    return flag ? KDA_ERR_TIMEOUT : KDA_OK;
}

kda_status_t kda_decode_step_v(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                               const float* S_in, float* S_out, void* o, int N, int H, int dk, int dv,
                               kda_dtype_t dtype, int erase, kda_gate_t gate, void* stream) {
    if (N < 0 || H < 0) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (erase != 0 && erase != 1) return KDA_ERR_INVALID_ARG;
    if (gate < KDA_GATE_CHANNEL || gate > KDA_GATE_NONE) return KDA_ERR_INVALID_ARG;
    if (!head_dims_ok(dk, dv)) return KDA_ERR_UNSUPPORTED;
    if ((long long)N * H * (dv / 32) > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
    if ((long long)N * H == 0) return KDA_OK;
    const void* req[] = {q, k, v, beta, S_in, S_out, o};
    for (const void* p : req)
        if (p == nullptr || !aligned16(p)) return KDA_ERR_INVALID_ARG;
    if (gate != KDA_GATE_NONE && (log_alpha == nullptr || !aligned16(log_alpha))) return KDA_ERR_INVALID_ARG;
    const cudaError_t err = kda::launch_decode(q, k, v, log_alpha, beta, S_in, S_out, o, N, H, dk, dv,
                                               dtype == KDA_BF16, erase, (int)gate, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_decode_step(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                             const float* S_in, float* S_out, void* o, int N, int H, int dk, int dv,
                             kda_dtype_t dtype, void* stream) {
    return kda_decode_step_v(q, k, v, log_alpha, beta, S_in, S_out, o, N, H, dk, dv, dtype, 1, KDA_GATE_CHANNEL,
                             stream);
}

size_t kda_chunk_bwd_workspace_size_ex(int B, int T, int H, int dk, int dv, kda_bwd_mode_t mode) {
    if (B < 0 || T < 0 || H < 0 || !head_dims_ok(dk, dv)) return 0;
    if (mode < KDA_BWD_AUTO || mode > KDA_BWD_LOW_MEMORY) return 0;
    return kda::chunk_bwd_workspace_bytes(B, T, H, dk, (int)mode);
}

size_t kda_chunk_bwd_workspace_size(int B, int T, int H, int dk, int dv) {
    return kda_chunk_bwd_workspace_size_ex(B, T, H, dk, dv, KDA_BWD_AUTO);
}

kda_status_t kda_chunk_bwd(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                           const float* S0, const void* dO, const float* dS_T, void* d_q, void* d_k, void* d_v,
                           void* d_log_alpha, void* d_beta, float* d_S0, int B, int T, int H, int dk, int dv,
                           kda_dtype_t dtype, int erase, kda_gate_t gate, void* workspace, size_t workspace_bytes,
                           void* stream) {
    return kda_chunk_bwd_ex(q, k, v, log_alpha, beta, S0, dO, dS_T, d_q, d_k, d_v, d_log_alpha, d_beta, d_S0, B, T,
                            H, dk, dv, dtype, erase, gate, KDA_BWD_AUTO, workspace, workspace_bytes, stream);
}

kda_status_t kda_chunk_bwd_ex(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                              const float* S0, const void* dO, const float* dS_T, void* d_q, void* d_k, void* d_v,
                              void* d_log_alpha, void* d_beta, float* d_S0, int B, int T, int H, int dk, int dv,
                              kda_dtype_t dtype, int erase, kda_gate_t gate, kda_bwd_mode_t mode, void* workspace,
                              size_t workspace_bytes, void* stream) {
    if (B < 0 || T < 0 || H < 0) return KDA_ERR_INVALID_ARG;
    if (mode < KDA_BWD_AUTO || mode > KDA_BWD_LOW_MEMORY) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (!head_dims_ok(dk, dv)) return KDA_ERR_UNSUPPORTED;
    if ((long long)B * H > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
    if (erase != 0 && erase != 1) return KDA_ERR_INVALID_ARG;
    if (gate < KDA_GATE_CHANNEL || gate > KDA_GATE_NONE) return KDA_ERR_INVALID_ARG;
    if ((long long)B * T * H > 0) {
        const void* req[] = {q, k, v, beta, dO, d_q, d_k, d_v, d_beta};
        for (const void* p : req)
            if (p == nullptr || !aligned16(p)) return KDA_ERR_INVALID_ARG;
        if (gate != KDA_GATE_NONE &&
            (log_alpha == nullptr || !aligned16(log_alpha) || d_log_alpha == nullptr || !aligned16(d_log_alpha)))
            return KDA_ERR_INVALID_ARG;
    }
    const float* opt[] = {S0, dS_T, d_S0};
    for (const float* p : opt)
        if (p && !aligned16(p)) return KDA_ERR_INVALID_ARG;
    const size_t need = kda::chunk_bwd_workspace_bytes(B, T, H, dk, (int)mode);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)))
        return KDA_ERR_INVALID_ARG;
    if ((long long)B * H == 0) return KDA_OK;
    kda::BwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.log_alpha = log_alpha; a.beta = beta; a.dO = dO; a.S0 = S0; a.dST = dS_T;
    a.g_q = d_q; a.g_k = d_k; a.g_v = d_v; a.g_log_alpha = d_log_alpha; a.g_beta = d_beta; a.g_S0 = d_S0;
    a.B = B; a.T = T; a.H = H; a.d = dk; a.bf16 = dtype == KDA_BF16; a.erase = erase; a.gate = (int)gate;
    a.mode = (int)mode;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes;
    const cudaError_t err = kda::launch_chunk_bwd(a, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// ---------------------------------------------------------------- gated linear recurrence

static bool dtype_ok(kda_dtype_t dtype) { return dtype == KDA_F32 || dtype == KDA_BF16; }
static bool good(const void* p) { return p != nullptr && aligned16(p); }

static kda_status_t check_recurrence(const kda::RecurrenceArgs& a, kda_dtype_t dtype, bool bwd) {
    if (a.N < 0 || a.T < 0 || a.D < 1 || a.D > 1 << 30) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return KDA_ERR_INVALID_ARG;
    if ((long long)a.N * ((a.D + 31) / 32) > 0x3ffffffLL) return KDA_ERR_INVALID_ARG;  // grid limit, clusters included
    if (a.cu_seqlens && (reinterpret_cast<uintptr_t>(a.cu_seqlens) & 3u) != 0) return KDA_ERR_INVALID_ARG;
    if ((long long)a.N * a.T > 0) {
        if (!good(a.log_alpha) || !good(a.x) || !good(a.out)) return KDA_ERR_INVALID_ARG;
        if (bwd && (!good(a.h_fwd) || !good(a.out_la))) return KDA_ERR_INVALID_ARG;
    }
    const float* opt[] = {a.state0, a.h0, a.state_end};
    for (const float* p : opt)
        if (p && !aligned16(p)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

kda_status_t kda_recurrence_fwd(const void* log_alpha, const void* x, const float* h0, void* h, float* h_T,
                                const int* cu_seqlens, int N, int T, int D, kda_dtype_t dtype, void* stream) {
    kda::RecurrenceArgs a{};
    a.log_alpha = log_alpha; a.x = x; a.state0 = h0; a.out = h; a.state_end = h_T; a.cu_seqlens = cu_seqlens;
    a.N = N; a.T = T; a.D = D; a.bf16 = dtype == KDA_BF16;
    const kda_status_t st = check_recurrence(a, dtype, false);
    if (st != KDA_OK) return st;
    if (N == 0) return KDA_OK;
    return kda::launch_recurrence_fwd(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_recurrence_timeout_test(const void* log_alpha, const void* x, void* h, int N, int T, int D,
                                         kda_dtype_t dtype, long long wait_budget_cycles, void* stream) {
    if (wait_budget_cycles <= 0 || wait_budget_cycles > (1ll << 31)) return KDA_ERR_INVALID_ARG;
    kda::RecurrenceArgs a{};
    a.log_alpha = log_alpha; a.x = x; a.out = h;
    a.N = N; a.T = T; a.D = D; a.bf16 = dtype == KDA_BF16;
    a.wait_cycles = wait_budget_cycles;
    a.test_withhold = 1;
    const kda_status_t st = check_recurrence(a, dtype, false);
    if (st != KDA_OK) return st;
    // Only a cluster waits: a few rows of at least 512 tokens.
    if (N < 1 || T < 512 || (long long)N * ((D + 31) / 32) >= 75) return KDA_ERR_INVALID_ARG;
    return kda::launch_recurrence_fwd(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_recurrence_status(void* stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return KDA_ERR_CUDA;
    unsigned flag = 0;
    if (kda::recurrence_late(&flag) != cudaSuccess) return KDA_ERR_CUDA;
    return flag ? KDA_ERR_TIMEOUT : KDA_OK;
}

kda_status_t kda_recurrence_bwd(const void* log_alpha, const void* h, const float* h0, const void* d_h,
                                const float* d_h_T, void* d_x, void* d_log_alpha, float* d_h0,
                                const int* cu_seqlens, int N, int T, int D, kda_dtype_t dtype, void* stream) {
    kda::RecurrenceArgs a{};
    a.log_alpha = log_alpha; a.x = d_h; a.h_fwd = h; a.h0 = h0; a.state0 = d_h_T; a.out = d_x;
    a.out_la = d_log_alpha; a.state_end = d_h0; a.cu_seqlens = cu_seqlens;
    a.N = N; a.T = T; a.D = D; a.bf16 = dtype == KDA_BF16;
    const kda_status_t st = check_recurrence(a, dtype, true);
    if (st != KDA_OK) return st;
    if (N == 0) return KDA_OK;
    return kda::launch_recurrence_bwd(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_recurrence_step(const void* log_alpha, const void* x, const float* h_in, float* h_out, void* y,
                                 int N, int D, kda_dtype_t dtype, void* stream) {
    if (N < 0 || D < 1 || !dtype_ok(dtype)) return KDA_ERR_INVALID_ARG;
    if (N == 0) return KDA_OK;
    const void* req[] = {log_alpha, x, h_in, h_out, y};
    for (const void* p : req)
        if (!good(p)) return KDA_ERR_INVALID_ARG;
    const cudaError_t err = kda::launch_recurrence_step(log_alpha, x, h_in, h_out, y, (long long)N * D,
                                                        dtype == KDA_BF16, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// ---------------------------------------------------------------- query/key norm and rotation

static kda_status_t check_qk(const kda::QkArgs& a, kda_dtype_t dtype, kda_norm_t norm, bool bwd) {
    if (a.n < 0 || a.Hq < 0 || a.Hk < 0 || !dtype_ok(dtype)) return KDA_ERR_INVALID_ARG;
    if (a.Hq > 65535 || a.Hk > 65535) return KDA_ERR_INVALID_ARG;
    if (norm != KDA_NORM_L2 && norm != KDA_NORM_RMS) return KDA_ERR_INVALID_ARG;
    if (a.interleaved != 0 && a.interleaved != 1) return KDA_ERR_INVALID_ARG;
    if (!(a.eps > 0.f) || a.eps > 3.0e38f) return KDA_ERR_INVALID_ARG;
    if (a.d < 8 || a.d > 256 || a.d % 8 != 0) return KDA_ERR_UNSUPPORTED;
    if (a.positions) {
        if (a.pos_bytes != 4 && a.pos_bytes != 8) return KDA_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(a.positions) & (uintptr_t)(a.pos_bytes - 1)) != 0) return KDA_ERR_INVALID_ARG;
        if (a.rot < 16 || a.rot > a.d || a.rot % 16 != 0) return KDA_ERR_UNSUPPORTED;
        if (a.max_pos < 1 || !good(a.cos) || !good(a.sin)) return KDA_ERR_INVALID_ARG;
    }
    if (a.n == 0) return KDA_OK;
    const long long unit = dtype == KDA_BF16 ? 8 : 4;  // elements of 16 bytes
    if (a.Hq > 0) {
        if (!good(a.q) || !good(a.q_out) || (bwd && !good(a.d_q_out))) return KDA_ERR_INVALID_ARG;
        if (a.q_stride_t % unit != 0 || a.q_stride_h % unit != 0) return KDA_ERR_INVALID_ARG;
    }
    if (a.Hk > 0) {
        if (!good(a.k) || !good(a.k_out) || (bwd && !good(a.d_k_out))) return KDA_ERR_INVALID_ARG;
        if (a.k_stride_t % unit != 0 || a.k_stride_h % unit != 0) return KDA_ERR_INVALID_ARG;
    }
    const void* opt[] = {a.q_weight, a.k_weight, a.d_q_weight, a.d_k_weight};
    for (const void* p : opt)
        if (p && !aligned16(p)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

kda_status_t kda_qk_norm_rope(const void* q, const void* k, const void* q_weight, const void* k_weight,
                              const float* cos, const float* sin, const void* positions, int pos_bytes, void* q_out,
                              void* k_out, int n, int Hq, int Hk, int d, int rot, int max_pos, long long q_stride_t,
                              long long q_stride_h, long long k_stride_t, long long k_stride_h, kda_norm_t norm,
                              float eps, float q_scale, int interleaved, kda_dtype_t dtype, void* stream) {
    kda::QkArgs a{};
    a.q = q; a.k = k; a.q_weight = q_weight; a.k_weight = k_weight; a.cos = cos; a.sin = sin;
    a.positions = positions; a.pos_bytes = pos_bytes; a.q_out = q_out; a.k_out = k_out;
    a.n = n; a.Hq = Hq; a.Hk = Hk; a.d = d; a.rot = positions ? rot : 0; a.max_pos = max_pos;
    a.q_stride_t = q_stride_t; a.q_stride_h = q_stride_h; a.k_stride_t = k_stride_t; a.k_stride_h = k_stride_h;
    a.norm = (int)norm; a.eps = eps; a.q_scale = q_scale; a.interleaved = interleaved; a.bf16 = dtype == KDA_BF16;
    const kda_status_t st = check_qk(a, dtype, norm, false);
    if (st != KDA_OK) return st;
    if (n == 0 || Hq + Hk == 0) return KDA_OK;
    return kda::launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_qk_norm_rope_bwd_workspace_size(int n, int Hq, int Hk, int d) {
    if (n < 0 || Hq < 0 || Hk < 0 || d < 8 || d > 256 || d % 8 != 0) return 0;
    return kda::qk_norm_rope_bwd_workspace_bytes(n, Hq, Hk, d);
}

kda_status_t kda_qk_norm_rope_bwd(const void* d_q_out, const void* d_k_out, const void* q, const void* k,
                                  const void* q_weight, const void* k_weight, const float* cos, const float* sin,
                                  const void* positions, int pos_bytes, void* d_q, void* d_k, float* d_q_weight,
                                  float* d_k_weight, int n, int Hq, int Hk, int d, int rot, int max_pos,
                                  long long q_stride_t, long long q_stride_h, long long k_stride_t,
                                  long long k_stride_h, kda_norm_t norm, float eps, float q_scale, int interleaved,
                                  kda_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
    kda::QkArgs a{};
    a.q = q; a.k = k; a.q_weight = q_weight; a.k_weight = k_weight; a.cos = cos; a.sin = sin;
    a.positions = positions; a.pos_bytes = pos_bytes; a.d_q_out = d_q_out; a.d_k_out = d_k_out;
    a.q_out = d_q; a.k_out = d_k; a.d_q_weight = d_q_weight; a.d_k_weight = d_k_weight;
    a.n = n; a.Hq = Hq; a.Hk = Hk; a.d = d; a.rot = positions ? rot : 0; a.max_pos = max_pos;
    a.q_stride_t = q_stride_t; a.q_stride_h = q_stride_h; a.k_stride_t = k_stride_t; a.k_stride_h = k_stride_h;
    a.norm = (int)norm; a.eps = eps; a.q_scale = q_scale; a.interleaved = interleaved; a.bf16 = dtype == KDA_BF16;
    a.workspace = workspace;
    const kda_status_t st = check_qk(a, dtype, norm, true);
    if (st != KDA_OK) return st;
    if (d_q_weight || d_k_weight) {
        const size_t need = kda::qk_norm_rope_bwd_workspace_bytes(n, Hq, Hk, d);
        if (need > 0 && (!good(workspace) || workspace_bytes < need)) return KDA_ERR_INVALID_ARG;
    }
    return kda::launch_qk_norm_rope_bwd(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// ---------------------------------------------------------------- paged decode attention

static bool attn_heads_ok(int Hq, int Hk) { return Hk > 0 && Hq > 0 && Hq % Hk == 0; }

size_t kda_attn_decode_workspace_size(int N, int Hq, int Hk, int d) {
    if (N <= 0 || !attn_heads_ok(Hq, Hk) || (d != 64 && d != 128)) return 0;
    return kda::attn_decode_workspace_bytes(N, Hq, Hk, d);
}

kda_status_t kda_attn_decode(const void* q, const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                             const int* page_table, const int* seq_lens, void* o, float* lse, int N, int Hq, int Hk,
                             int d, int n_pages, int page_size, int max_pages, int window, float scale,
                             kda_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (N < 0 || !attn_heads_ok(Hq, Hk) || n_pages < 0 || page_size < 1 || max_pages < 0 || window < 0)
        return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || !(scale == scale)) return KDA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return KDA_ERR_UNSUPPORTED;
    // positions, and the work items of all rows, are counted in int32
    if ((long long)max_pages * page_size > 0x3fffffffLL || (long long)N * Hq > 0xffffffLL) return KDA_ERR_INVALID_ARG;
    // so are the rows of a cache (one of more would not fit the device)
    if ((long long)n_pages * page_size > 0x7fffffffLL || (long long)n_pages * page_size * Hk > 0x7fffffffLL)
        return KDA_ERR_INVALID_ARG;
    // a worker's share of the work (one of 592 at least) is counted in int32: reached only by capacities that no run ends
    const long long tiles = (long long)max_pages * page_size / 16 + 4, pairs = (long long)N * Hk * ((Hq / Hk + 15) / 16);
    if (pairs > 0 && tiles > 0x7fffffffLL * 512 / pairs) return KDA_ERR_INVALID_ARG;
    if (N == 0) return KDA_OK;
    if (!good(q) || !good(o)) return KDA_ERR_INVALID_ARG;
    if ((k_new == nullptr) != (v_new == nullptr)) return KDA_ERR_INVALID_ARG;
    if (k_new && (!aligned16(k_new) || !aligned16(v_new))) return KDA_ERR_INVALID_ARG;
    if (n_pages > 0 && (!good(k_cache) || !good(v_cache))) return KDA_ERR_INVALID_ARG;
    if (seq_lens == nullptr || (reinterpret_cast<uintptr_t>(seq_lens) & 3u) != 0) return KDA_ERR_INVALID_ARG;
    if (max_pages > 0 && (page_table == nullptr || (reinterpret_cast<uintptr_t>(page_table) & 3u) != 0))
        return KDA_ERR_INVALID_ARG;
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return KDA_ERR_INVALID_ARG;
    const size_t need = kda::attn_decode_workspace_bytes(N, Hq, Hk, d);
    if (need > 0 && (!good(workspace) || workspace_bytes < need)) return KDA_ERR_INVALID_ARG;
    kda::AttnDecodeArgs a{};
    a.q = q; a.k_new = k_new; a.v_new = v_new; a.k_cache = k_cache; a.v_cache = v_cache;
    a.page_table = page_table; a.seq_lens = seq_lens; a.o = o; a.lse = lse;
    a.N = N; a.Hq = Hq; a.Hk = Hk; a.d = d; a.n_pages = n_pages; a.page_size = page_size; a.max_pages = max_pages;
    a.window = window; a.scale = scale; a.bf16 = dtype == KDA_BF16; a.workspace = workspace;
    return kda::launch_attn_decode(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
