// kda_abi.cu -- the extern "C" entry points of libkda: argument checks,
// path selection and launches.  Every check here runs on the host before
// anything is enqueued; the kernels themselves live in the other files.
#include <limits.h>

#include <initializer_list>

#include "kda_internal.cuh"
#include "kda_linear.cuh"
#include "kda_testing.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool supported_d(int32_t d) { return d == 16 || d == 64 || d == 128; }
bool supported_chunk(int32_t L) { return L == 16 || L == 32 || L == 64; }
bool valid_dtype(kda_dtype dt) { return dt == KDA_F32 || dt == KDA_BF16; }

kda::Path prefill_path(int32_t d, kda_dtype dt, int32_t L) {
    return (dt == KDA_BF16 && d == 128 && L == 64) ? kda::PATH_TC : kda::PATH_SIMT;
}

kda_status shape_check(int32_t total_tokens, int32_t num_seqs, int32_t H, int32_t d_k, int32_t d_v,
                       kda_dtype dt, int32_t chunk) {
    if (total_tokens < 0 || num_seqs < 0 || H <= 0 || H > 65535) return KDA_ERR_INVALID_ARG;
    if (!valid_dtype(dt)) return KDA_ERR_INVALID_ARG;
    if (d_k != d_v || !supported_d(d_k) || !supported_chunk(chunk)) return KDA_ERR_UNSUPPORTED;
    // every row index (token * H + head) * d must fit the kernels' 32-bit token arithmetic
    if ((int64_t)total_tokens * H > INT_MAX || (int64_t)num_seqs * H * 8 > INT_MAX) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// The fused prologue / epilogue options, checked (pointers only when the call has rows to process).
kda_status fusion_from(const kda_fusion_opts *opts, bool any_rows, const void *o, kda::Fusion *fu) {
    *fu = kda::Fusion{};
    if (!opts) return KDA_OK;
    if (opts->qk_l2norm) {
        if (!(opts->qk_eps >= 0.f)) return KDA_ERR_INVALID_ARG;
        fu->qk_norm = 1;
        fu->qk_eps = opts->qk_eps;
    }
    if (opts->out_gate) {
        if (!(opts->out_eps > 0.f)) return KDA_ERR_INVALID_ARG;
        if (any_rows && (!aligned16(opts->out_gate) || opts->out_gate == o)) return KDA_ERR_INVALID_ARG;
        if (!aligned16(opts->out_weight)) return KDA_ERR_INVALID_ARG;  // (null passes)
        fu->gate = opts->out_gate;
        fu->weight = opts->out_weight;
        fu->out_eps = opts->out_eps;
    }
    return KDA_OK;
}

}  // namespace

extern "C" {

const char *kda_status_string(kda_status status) {
    switch (status) {
        case KDA_OK: return "KDA_OK";
        case KDA_ERR_INVALID_ARG: return "KDA_ERR_INVALID_ARG";
        case KDA_ERR_UNSUPPORTED: return "KDA_ERR_UNSUPPORTED";
        case KDA_ERR_CUDA: return "KDA_ERR_CUDA";
        case KDA_ERR_TIMEOUT: return "KDA_ERR_TIMEOUT";
        case KDA_ERR_BOUNDS: return "KDA_ERR_BOUNDS";
        default: return "KDA_ERR_UNKNOWN";
    }
}

size_t kda_prefill_workspace_size(int32_t total_tokens, int32_t num_seqs, int32_t H, int32_t d_k, int32_t d_v,
                                  kda_dtype in_dtype, int32_t chunk_size) {
    const int32_t L = chunk_size == 0 ? 64 : chunk_size;
    if (shape_check(total_tokens, num_seqs, H, d_k, d_v, in_dtype, L) != KDA_OK) return 0;
    return kda::ws_layout(total_tokens, num_seqs, H, d_k, d_v, L, prefill_path(d_k, in_dtype, L)).total;
}

}  // extern "C"

namespace {

kda_status prefill_impl(const void *q, const void *k, const void *v, const float *g, const float *beta,
                        const int32_t *cu_seqlens, int32_t num_seqs, int32_t total_tokens, int32_t H, int32_t d_k,
                        int32_t d_v, kda_dtype in_dtype, int32_t chunk_size, const float *S0, void *o,
                        float *S_final, void *workspace, size_t workspace_bytes, void *stream, kda::Marks &marks,
                        const kda_fusion_opts *opts = nullptr) {
    const int32_t L = chunk_size == 0 ? 64 : chunk_size;
    kda_status st = shape_check(total_tokens, num_seqs, H, d_k, d_v, in_dtype, L);
    if (st != KDA_OK) return st;
    kda::Fusion fu;
    if ((st = fusion_from(opts, total_tokens > 0, o, &fu)) != KDA_OK) return st;
    if (!cu_seqlens || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0) {
        if (!q || !k || !v || !g || !beta || !o) return KDA_ERR_INVALID_ARG;
        if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(o)) return KDA_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(beta) & 3u) return KDA_ERR_INVALID_ARG;
        if (o == q || o == k || o == v || o == (const void *)g) return KDA_ERR_INVALID_ARG;
    }
    if (!aligned16(S0) || !aligned16(S_final)) return KDA_ERR_INVALID_ARG;
    const kda::Path path = prefill_path(d_k, in_dtype, L);
    const kda::WsLayout lay = kda::ws_layout(total_tokens, num_seqs, H, d_k, d_v, L, path);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < lay.total)
        return KDA_ERR_INVALID_ARG;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const kda::TcPlan plan =
        path == kda::PATH_TC ? kda::tc_plan(num_seqs, H, total_tokens) : kda::TC_THREE;
    const bool flags = plan != kda::TC_THREE;
    cudaError_t e = cudaSuccess;
    if (!(path == kda::PATH_TC && kda::pipe_self_indexed(plan, num_seqs)))
        e = kda::launch_chunk_index(cu_seqlens, num_seqs, total_tokens, L, workspace,
                                    flags ? static_cast<char *>(workspace) + lay.flags_off : nullptr,
                                    flags ? lay.flags_bytes : 0, s, marks);
    if (e != cudaSuccess) return KDA_ERR_CUDA;
    if (path == kda::PATH_TC)
        e = kda::launch_prefill_tc(q, k, v, g, beta, cu_seqlens, num_seqs, total_tokens, H, S0, o, S_final, workspace,
                                   plan, fu, s, marks);
    else
        e = kda::launch_prefill_simt(q, k, v, g, beta, cu_seqlens, num_seqs, total_tokens, H, d_k, in_dtype, L, S0,
                                     o, S_final, workspace, fu, s, marks);
    marks.end(s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

extern "C" {

kda_status kda_prefill_chunked(const void *q, const void *k, const void *v, const float *g, const float *beta,
                               const int32_t *cu_seqlens, int32_t num_seqs, int32_t total_tokens, int32_t H,
                               int32_t d_k, int32_t d_v, kda_dtype in_dtype, int32_t chunk_size, const float *S0,
                               void *o, float *S_final, void *workspace, size_t workspace_bytes, void *stream) {
    kda::Marks marks;
    return prefill_impl(q, k, v, g, beta, cu_seqlens, num_seqs, total_tokens, H, d_k, d_v, in_dtype, chunk_size, S0,
                        o, S_final, workspace, workspace_bytes, stream, marks);
}

kda_status kda_prefill_chunked_ex(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                  const int32_t *cu_seqlens, int32_t num_seqs, int32_t total_tokens, int32_t H,
                                  int32_t d_k, int32_t d_v, kda_dtype in_dtype, int32_t chunk_size, const float *S0,
                                  void *o, float *S_final, void *workspace, size_t workspace_bytes, void *stream,
                                  const kda_fusion_opts *opts) {
    kda::Marks marks;
    return prefill_impl(q, k, v, g, beta, cu_seqlens, num_seqs, total_tokens, H, d_k, d_v, in_dtype, chunk_size, S0,
                        o, S_final, workspace, workspace_bytes, stream, marks, opts);
}

kda_status kda_prefill_chunked_profiled(const void *q, const void *k, const void *v, const float *g,
                                        const float *beta, const int32_t *cu_seqlens, int32_t num_seqs,
                                        int32_t total_tokens, int32_t H, int32_t d_k, int32_t d_v,
                                        kda_dtype in_dtype, int32_t chunk_size, const float *S0, void *o,
                                        float *S_final, void *workspace, size_t workspace_bytes, void *stream,
                                        void *const *events, int32_t *num_kernels, const char **kernel_names) {
    kda::Marks marks;
    marks.ev = events;
    marks.names = kernel_names;
    const kda_status st = prefill_impl(q, k, v, g, beta, cu_seqlens, num_seqs, total_tokens, H, d_k, d_v, in_dtype,
                                       chunk_size, S0, o, S_final, workspace, workspace_bytes, stream, marks);
    if (num_kernels) *num_kernels = marks.n;
    return st;
}

kda_status kda_prefill_check(const void *workspace, void *stream) {
    if (!workspace) return KDA_ERR_INVALID_ARG;
    int32_t flag = -1;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(&flag, workspace, sizeof(flag), cudaMemcpyDeviceToHost, s) != cudaSuccess) return KDA_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return KDA_ERR_CUDA;
    return kda::status_from_word(flag);
}

kda_status kda_testing_set_plan(int32_t plan) {
    if (plan != -1 && plan != KDA_TESTING_PLAN_THREE && plan != KDA_TESTING_PLAN_CHAIN && plan != KDA_TESTING_PLAN_PIPE)
        return KDA_ERR_INVALID_ARG;
    kda::testing_set_plan(plan == KDA_TESTING_PLAN_THREE   ? kda::TC_THREE
                          : plan == KDA_TESTING_PLAN_CHAIN ? kda::TC_CHAIN
                          : plan == KDA_TESTING_PLAN_PIPE  ? kda::TC_PIPE
                                                           : -1);
    return KDA_OK;
}

kda_status kda_testing_set_fault(int32_t fault, int64_t wait_limit_ns) {
    if ((fault != KDA_TESTING_FAULT_NONE && fault != KDA_TESTING_FAULT_NO_PUBLISH &&
         fault != KDA_TESTING_FAULT_CHUNK_TABLE) ||
        wait_limit_ns < 0)
        return KDA_ERR_INVALID_ARG;
    kda::testing_set_fault(fault, (long long)wait_limit_ns);
    return KDA_OK;
}

kda_status kda_decode_step(const void *q, const void *k, const void *v, const float *g, const float *beta,
                           int32_t num_seqs, int32_t H, int32_t d_k, int32_t d_v, kda_dtype in_dtype,
                           float *S_inout, void *o, void *stream) {
    return kda_decode_step_ex(q, k, v, g, beta, num_seqs, H, d_k, d_v, in_dtype, S_inout, o, stream, nullptr);
}

kda_status kda_decode_step_ex(const void *q, const void *k, const void *v, const float *g, const float *beta,
                              int32_t num_seqs, int32_t H, int32_t d_k, int32_t d_v, kda_dtype in_dtype,
                              float *S_inout, void *o, void *stream, const kda_fusion_opts *opts) {
    if (num_seqs < 0 || H <= 0 || !valid_dtype(in_dtype)) return KDA_ERR_INVALID_ARG;
    kda::Fusion fu;
    if (kda_status st = fusion_from(opts, num_seqs > 0, o, &fu)) return st;
    if (d_k != d_v || !supported_d(d_k)) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)num_seqs * H > INT_MAX) return KDA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return KDA_OK;
    if (!q || !k || !v || !g || !beta || !S_inout || !o) return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(S_inout) || !aligned16(o))
        return KDA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(beta) & 3u) return KDA_ERR_INVALID_ARG;
    if (o == q || o == k || o == v || o == (const void *)S_inout) return KDA_ERR_INVALID_ARG;
    cudaError_t e = kda::launch_decode(q, k, v, g, beta, num_seqs, H, d_k, in_dtype, S_inout, o, nullptr, num_seqs,
                                       nullptr, fu, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_decode_step_indexed(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                   const int32_t *seq_idx, int32_t num_active, int32_t num_slots, int32_t H,
                                   int32_t d_k, int32_t d_v, kda_dtype in_dtype, float *S_pool, void *o,
                                   int32_t *status, void *stream) {
    if (num_active < 0 || num_slots < 0 || H <= 0 || !valid_dtype(in_dtype)) return KDA_ERR_INVALID_ARG;
    if (d_k != d_v || !supported_d(d_k)) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)num_active * H > INT_MAX || (int64_t)num_slots * H > INT_MAX) return KDA_ERR_UNSUPPORTED;
    if (num_active == 0) return KDA_OK;
    if (!q || !k || !v || !g || !beta || !seq_idx || !S_pool || !o) return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(S_pool) || !aligned16(o))
        return KDA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(beta) & 3u) || (reinterpret_cast<uintptr_t>(seq_idx) & 3u) ||
        (reinterpret_cast<uintptr_t>(status) & 3u))
        return KDA_ERR_INVALID_ARG;
    if (o == q || o == k || o == v || o == (const void *)S_pool) return KDA_ERR_INVALID_ARG;
    cudaError_t e = kda::launch_decode(q, k, v, g, beta, num_active, H, d_k, in_dtype, S_pool, o, seq_idx, num_slots,
                                       status, kda::Fusion{}, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

static kda_status state_copy(const float *src, float *dst, const int32_t *seq_idx, int32_t n, int32_t num_slots,
                             int32_t H, int32_t d_k, int32_t d_v, bool scatter, int32_t *status, void *stream) {
    if (n < 0 || num_slots < 0 || H <= 0) return KDA_ERR_INVALID_ARG;
    if (d_k != d_v || !supported_d(d_k)) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)H * d_k * d_v > INT_MAX || (int64_t)n * H > INT_MAX) return KDA_ERR_UNSUPPORTED;
    if (n == 0) return KDA_OK;
    if (!src || !dst || !seq_idx || !aligned16(src) || !aligned16(dst) || (reinterpret_cast<uintptr_t>(seq_idx) & 3u) ||
        (reinterpret_cast<uintptr_t>(status) & 3u) || src == dst)
        return KDA_ERR_INVALID_ARG;
    cudaError_t e = kda::launch_state_copy(src, dst, seq_idx, n, num_slots, H, d_k, scatter, status,
                                           static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_short_conv_prefill(const void *x, const float *w, const int32_t *cu_seqlens, int32_t num_seqs,
                                  int32_t total_tokens, int32_t C, int32_t W, kda_dtype in_dtype,
                                  const float *conv_state, void *y, float *conv_state_out, void *stream) {
    if (total_tokens < 0 || num_seqs < 0 || C <= 0 || !valid_dtype(in_dtype)) return KDA_ERR_INVALID_ARG;
    if (W < 1 || W > KDA_SHORT_CONV_MAX_W) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)total_tokens * C > INT_MAX || (int64_t)num_seqs * W * C > INT_MAX) return KDA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return total_tokens == 0 ? KDA_OK : KDA_ERR_INVALID_ARG;
    const uintptr_t el = in_dtype == KDA_BF16 ? 1u : 3u;
    if (!cu_seqlens || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!x || !w || !y || (reinterpret_cast<uintptr_t>(x) & el) ||
                             (reinterpret_cast<uintptr_t>(y) & el) || x == y))
        return KDA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(w) & 3u) || (reinterpret_cast<uintptr_t>(conv_state) & 3u) ||
        (reinterpret_cast<uintptr_t>(conv_state_out) & 3u))
        return KDA_ERR_INVALID_ARG;
    if (W > 1 && conv_state && conv_state == conv_state_out) return KDA_ERR_INVALID_ARG;
    cudaError_t e = kda::launch_conv_prefill(x, w, cu_seqlens, num_seqs, total_tokens, C, W, in_dtype,
                                             W > 1 ? conv_state : nullptr, y, W > 1 ? conv_state_out : nullptr,
                                             static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_short_conv_decode(const void *x, const float *w, int32_t N, int32_t C, int32_t W, kda_dtype in_dtype,
                                 float *conv_state, void *y, void *stream) {
    if (N < 0 || C <= 0 || !valid_dtype(in_dtype)) return KDA_ERR_INVALID_ARG;
    if (W < 1 || W > KDA_SHORT_CONV_MAX_W) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)N * W * C > INT_MAX) return KDA_ERR_UNSUPPORTED;
    if (N == 0) return KDA_OK;
    const uintptr_t el = in_dtype == KDA_BF16 ? 1u : 3u;
    if (!x || !w || !y || (W > 1 && !conv_state) || (reinterpret_cast<uintptr_t>(x) & el) ||
        (reinterpret_cast<uintptr_t>(y) & el) || (reinterpret_cast<uintptr_t>(w) & 3u) ||
        (reinterpret_cast<uintptr_t>(conv_state) & 3u) || x == y)
        return KDA_ERR_INVALID_ARG;
    cudaError_t e = kda::launch_conv_decode(x, w, N, C, W, in_dtype, conv_state, y, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_state_snapshot(const float *S_pool, const int32_t *seq_idx, int32_t n, int32_t num_slots, int32_t H,
                              int32_t d_k, int32_t d_v, float *S_saved, int32_t *status, void *stream) {
    return state_copy(S_pool, S_saved, seq_idx, n, num_slots, H, d_k, d_v, false, status, stream);
}

kda_status kda_state_restore(const float *S_saved, const int32_t *seq_idx, int32_t n, int32_t num_slots, int32_t H,
                             int32_t d_k, int32_t d_v, float *S_pool, int32_t *status, void *stream) {
    return state_copy(S_saved, S_pool, seq_idx, n, num_slots, H, d_k, d_v, true, status, stream);
}

// What the tree entry points share: sizes, then the packed layout's pointers (only when there are requests).
static kda_status tree_check(int32_t num_seqs, int32_t total_nodes, int32_t bound, int32_t num_slots,
                             kda_dtype in_dtype) {
    if (num_seqs < 0 || total_nodes < 0 || num_slots < 0 || !valid_dtype(in_dtype)) return KDA_ERR_INVALID_ARG;
    if (bound < 1) return KDA_ERR_INVALID_ARG;
    return bound > KDA_TREE_MAX_NODES ? KDA_ERR_UNSUPPORTED : KDA_OK;
}
static bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
static bool given4(const void *p) { return p && aligned4(p); }
static bool given16(const void *p) { return p && aligned16(p); }

kda_status kda_tree_step(const void *q, const void *k, const void *v, const float *g, const float *beta,
                         const int32_t *parent, const int32_t *cu_nodes, const int32_t *seq_idx, int32_t num_seqs,
                         int32_t total_nodes, int32_t max_nodes, int32_t num_slots, int32_t H, int32_t d_k,
                         int32_t d_v, kda_dtype in_dtype, const float *S_pool, void *o, float *u, int32_t *status,
                         void *stream, const kda_fusion_opts *opts) {
    if (kda_status st = tree_check(num_seqs, total_nodes, max_nodes, num_slots, in_dtype)) return st;
    if (H <= 0) return KDA_ERR_INVALID_ARG;
    kda::Fusion fu;
    if (kda_status st = fusion_from(opts, total_nodes > 0, o, &fu)) return st;
    if (d_k != d_v || !supported_d(d_k)) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)total_nodes * H > INT_MAX || (int64_t)num_seqs * H > INT_MAX || (int64_t)num_slots * H > INT_MAX)
        return KDA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_nodes == 0) return KDA_OK;
    if (!given16(q) || !given16(k) || !given16(v) || !given16(g) || !given4(beta) || !given4(parent) ||
        !given4(cu_nodes) || !aligned4(seq_idx) || !given16(S_pool) || !given16(o) || !aligned16(u) ||
        !aligned4(status))
        return KDA_ERR_INVALID_ARG;
    for (const void *out : {(const void *)o, (const void *)u})
        if (out && (out == q || out == k || out == v || out == (const void *)g || out == (const void *)S_pool ||
                    out == (const void *)beta || out == fu.gate))
            return KDA_ERR_INVALID_ARG;
    if (o == (const void *)u) return KDA_ERR_INVALID_ARG;
    const kda::TreeStepArgs a{q, k, v, g, beta, parent, cu_nodes, seq_idx, num_seqs, total_nodes, max_nodes,
                              num_slots, H, d_k, S_pool, o, u, status, fu};
    return kda::launch_tree_step(a, in_dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK
                                                                                                : KDA_ERR_CUDA;
}

kda_status kda_tree_commit(const void *k, const float *g, const float *u, const int32_t *cu_nodes,
                           const int32_t *path, const int32_t *path_len, const int32_t *seq_idx, int32_t num_seqs,
                           int32_t total_nodes, int32_t path_stride, int32_t num_slots, int32_t H, int32_t d_k,
                           int32_t d_v, kda_dtype in_dtype, float *S_pool, int32_t *status, void *stream,
                           const kda_fusion_opts *opts) {
    if (kda_status st = tree_check(num_seqs, total_nodes, path_stride, num_slots, in_dtype)) return st;
    if (H <= 0) return KDA_ERR_INVALID_ARG;
    const bool qk_norm = opts && opts->qk_l2norm;
    if (qk_norm && !(opts->qk_eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (d_k != d_v || !supported_d(d_k)) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)total_nodes * H > INT_MAX || (int64_t)num_seqs * H > INT_MAX || (int64_t)num_slots * H > INT_MAX)
        return KDA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_nodes == 0) return KDA_OK;
    if (!given16(k) || !given16(g) || !given16(u) || !given4(cu_nodes) || !given4(path) || !given4(path_len) ||
        !aligned4(seq_idx) || !given16(S_pool) || !aligned4(status))
        return KDA_ERR_INVALID_ARG;
    const void *out = S_pool;
    if (out == k || out == (const void *)g || out == (const void *)u) return KDA_ERR_INVALID_ARG;
    const kda::TreeCommitArgs a{k, g, u, cu_nodes, path, path_len, seq_idx, num_seqs, total_nodes, path_stride,
                                num_slots, H, d_k, S_pool, status, qk_norm ? 1 : 0, qk_norm ? opts->qk_eps : 0.f};
    return kda::launch_tree_commit(a, in_dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK
                                                                                                  : KDA_ERR_CUDA;
}

static kda_status tree_conv_check(int32_t num_seqs, int32_t total_nodes, int32_t num_slots, int32_t C, int32_t W) {
    if (C <= 0) return KDA_ERR_INVALID_ARG;
    if (W < 1 || W > KDA_SHORT_CONV_MAX_W) return KDA_ERR_UNSUPPORTED;
    // the grid's second dimension is the request; the last block's channel numbers, past C by less than a block's 512,
    // have to fit an int
    if (num_seqs > 65535 || (int64_t)C * W > INT_MAX || C > INT_MAX - 512) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status kda_tree_conv(const void *x, const float *w, const int32_t *parent, const int32_t *cu_nodes,
                         const int32_t *seq_idx, int32_t num_seqs, int32_t total_nodes, int32_t max_nodes,
                         int32_t num_slots, int32_t C, int32_t W, kda_dtype in_dtype, const float *conv_pool, void *y,
                         int32_t *status, void *stream) {
    if (kda_status st = tree_check(num_seqs, total_nodes, max_nodes, num_slots, in_dtype)) return st;
    if (kda_status st = tree_conv_check(num_seqs, total_nodes, num_slots, C, W)) return st;
    if (num_seqs == 0 || total_nodes == 0) return KDA_OK;
    const uintptr_t el = in_dtype == KDA_BF16 ? 1u : 3u;
    if (!x || !y || x == y || (reinterpret_cast<uintptr_t>(x) & el) || (reinterpret_cast<uintptr_t>(y) & el) ||
        !given4(w) || !given4(parent) || !given4(cu_nodes) || !aligned4(seq_idx) || !aligned4(conv_pool) ||
        (W > 1 && !conv_pool) || y == (const void *)conv_pool || y == (const void *)w || !aligned4(status))
        return KDA_ERR_INVALID_ARG;
    const kda::TreeConvArgs a{x, w, parent, cu_nodes, seq_idx, num_seqs, total_nodes, max_nodes, num_slots, C, W,
                              conv_pool, y, status};
    return kda::launch_tree_conv(a, in_dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK
                                                                                                : KDA_ERR_CUDA;
}

kda_status kda_tree_conv_commit(const void *x, const int32_t *cu_nodes, const int32_t *path, const int32_t *path_len,
                                const int32_t *seq_idx, int32_t num_seqs, int32_t total_nodes, int32_t path_stride,
                                int32_t num_slots, int32_t C, int32_t W, kda_dtype in_dtype, float *conv_pool,
                                int32_t *status, void *stream) {
    if (kda_status st = tree_check(num_seqs, total_nodes, path_stride, num_slots, in_dtype)) return st;
    if (kda_status st = tree_conv_check(num_seqs, total_nodes, num_slots, C, W)) return st;
    if (num_seqs == 0 || total_nodes == 0 || W == 1) return KDA_OK;  // a width of one carries nothing
    const uintptr_t el = in_dtype == KDA_BF16 ? 1u : 3u;
    if (!x || (reinterpret_cast<uintptr_t>(x) & el) || !given4(cu_nodes) || !given4(path) || !given4(path_len) ||
        !aligned4(seq_idx) || !given4(conv_pool) || x == (const void *)conv_pool || !aligned4(status))
        return KDA_ERR_INVALID_ARG;
    const kda::TreeConvCommitArgs a{x, cu_nodes, path, path_len, seq_idx, num_seqs, total_nodes, path_stride,
                                    num_slots, C, W, conv_pool, status};
    return kda::launch_tree_conv_commit(a, in_dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

kda_status kda_draft_verify(const void *logits, const float *draft_probs, const int32_t *tokens, const int32_t *parent,
                            const int32_t *cu_nodes, const float *temperature, const float *u_accept,
                            const float *u_next, int32_t num_seqs, int32_t total_nodes, int32_t V, kda_dtype in_dtype,
                            int32_t path_stride, int32_t *path, int32_t *path_len, int32_t *next_token,
                            int32_t *status, void *stream) {
    if (kda_status st = tree_check(num_seqs, total_nodes, path_stride, 0, in_dtype)) return st;
    if (V <= 0) return KDA_ERR_INVALID_ARG;
    if (V > KDA_VERIFY_MAX_VOCAB || num_seqs > INT_MAX / 8) return KDA_ERR_UNSUPPORTED;  // up to 8 CTAs a request
    if (num_seqs == 0) return KDA_OK;
    const uintptr_t el = in_dtype == KDA_BF16 ? 1u : 3u;
    if (total_nodes > 0 && (!logits || (reinterpret_cast<uintptr_t>(logits) & el) || !aligned4(draft_probs) ||
                            !given4(tokens) || !given4(parent) || !aligned4(temperature) || !given4(u_accept) ||
                            !given4(u_next)))
        return KDA_ERR_INVALID_ARG;
    if (!given4(cu_nodes) || !given4(path) || !given4(path_len) || !given4(next_token) || !aligned4(status))
        return KDA_ERR_INVALID_ARG;
    const kda::DraftVerifyArgs a{logits, draft_probs, tokens, parent, cu_nodes, temperature, u_accept, u_next,
                                 num_seqs, total_nodes, V, path_stride, path, path_len, next_token, status};
    return kda::launch_draft_verify(a, in_dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK
                                                                                                   : KDA_ERR_CUDA;
}

// Sizes that the linear-attention entry points share.
static kda_status linear_check(int32_t rows, int32_t H, int32_t H_qk, int32_t d_k, int32_t d_v, kda_dtype in_dtype) {
    if (rows < 0 || H <= 0 || H > 65535 || H_qk <= 0 || H % H_qk || !valid_dtype(in_dtype)) return KDA_ERR_INVALID_ARG;
    if (d_k != d_v || !supported_d(d_k)) return KDA_ERR_UNSUPPORTED;
    return (int64_t)rows * H > INT_MAX ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

// Segments of a prefill call and where its workspace holds them.
static bool linear_on_tensor_cores(int32_t d, kda_dtype dt) { return dt == KDA_BF16 && d == 128; }
static kda_status linear_plan(int32_t total_tokens, int32_t num_seqs, int32_t H, int32_t d, kda_dtype dt, int32_t *seg,
                              int32_t *slots, kda::linear::Layout *lay) {
    if (num_seqs < 0) return KDA_ERR_INVALID_ARG;
    *seg = kda::linear::plan_segment(total_tokens, num_seqs, H, d, linear_on_tensor_cores(d, dt));
    if ((int64_t)total_tokens + *seg > INT_MAX) return KDA_ERR_UNSUPPORTED;  // kernels round token counts up to segments
    const int64_t n = total_tokens / *seg + (int64_t)num_seqs;
    if (n * H > INT_MAX - 4096) return KDA_ERR_UNSUPPORTED;  // units are counted past their end by a grid or two
    *slots = (int32_t)n;
    *lay = kda::linear::layout(n, H, d, total_tokens > *seg);
    return KDA_OK;
}

size_t kda_linear_workspace_size(int32_t total_tokens, int32_t num_seqs, int32_t H, int32_t d_k, int32_t d_v, kda_dtype in_dtype) {
    int32_t seg, slots;
    kda::linear::Layout lay;
    if (linear_check(total_tokens, H, H, d_k, d_v, in_dtype) || linear_plan(total_tokens, num_seqs, H, d_k, in_dtype, &seg, &slots, &lay)) return 0;
    return lay.total;
}

kda_status kda_linear_prefill(const void *q, const void *k, const void *v, const float *g, int32_t g_per_token,
                              const int32_t *cu_seqlens, int32_t num_seqs, int32_t total_tokens, int32_t H, int32_t H_qk,
                              int32_t d_k, int32_t d_v, kda_dtype in_dtype, const float *S0, void *o, float *S_final,
                              void *workspace, size_t workspace_bytes, void *stream, const kda_fusion_opts *opts) {
    if (kda_status st = linear_check(total_tokens, H, H_qk, d_k, d_v, in_dtype)) return st;
    int32_t seg, slots;
    kda::linear::Layout lay;
    if (kda_status st = linear_plan(total_tokens, num_seqs, H, d_k, in_dtype, &seg, &slots, &lay)) return st;
    kda::Fusion fu;
    if (kda_status st = fusion_from(opts, total_tokens > 0, o, &fu)) return st;
    if (num_seqs == 0) return total_tokens == 0 ? KDA_OK : KDA_ERR_INVALID_ARG;
    if (!given4(cu_seqlens)) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0) {
        if (!given16(q) || !given16(k) || !given16(v) || !given4(g) || !given16(o)) return KDA_ERR_INVALID_ARG;
        if (o == q || o == k || o == v || o == (const void *)g || o == (const void *)S0) return KDA_ERR_INVALID_ARG;
    }
    if (!aligned16(S0) || !aligned16(S_final)) return KDA_ERR_INVALID_ARG;
    const void *end = S_final;
    if (end && (end == q || end == k || end == v || end == o || end == (const void *)g || end == fu.gate)) return KDA_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < lay.total) return KDA_ERR_INVALID_ARG;
    char *ws = static_cast<char *>(workspace);
    kda::linear::Args a{};
    a.q = q, a.k = k, a.v = v, a.g = g, a.per_token = g_per_token != 0, a.cu = cu_seqlens;
    a.num_seqs = num_seqs, a.total = total_tokens, a.H = H, a.Hqk = H_qk, a.seg = seg, a.slots = slots;
    a.S0 = S0, a.o = o, a.S_final = S_final, a.aliased = S0 && S0 == S_final;
    a.seg_decay = reinterpret_cast<float *>(ws + lay.decay_off);
    a.seg_state = reinterpret_cast<float *>(ws + lay.state_off);
    a.status = reinterpret_cast<int32_t *>(ws), a.ticket = a.status + kda::linear::kTicketWord, a.fu = fu;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = linear_on_tensor_cores(d_k, in_dtype) ? kda::launch_linear_tc(a, s) : kda::launch_linear_simt(a, d_k, in_dtype, s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_linear_decode_step(const void *q, const void *k, const void *v, const float *g, int32_t g_per_token,
                                  const int32_t *seq_idx, int32_t num_active, int32_t num_slots, int32_t H, int32_t H_qk,
                                  int32_t d_k, int32_t d_v, kda_dtype in_dtype, float *S_pool, void *o, int32_t *status,
                                  void *stream, const kda_fusion_opts *opts) {
    if (kda_status st = linear_check(num_active, H, H_qk, d_k, d_v, in_dtype)) return st;
    if (num_slots < 0) return KDA_ERR_INVALID_ARG;
    if ((int64_t)num_slots * H > INT_MAX) return KDA_ERR_UNSUPPORTED;
    kda::Fusion fu;
    if (kda_status st = fusion_from(opts, num_active > 0, o, &fu)) return st;
    if (num_active == 0) return KDA_OK;
    if (!given16(q) || !given16(k) || !given16(v) || !given4(g) || !aligned4(seq_idx) || !given16(S_pool) || !given16(o) || !aligned4(status))
        return KDA_ERR_INVALID_ARG;
    if (o == q || o == k || o == v || o == (const void *)g || o == (const void *)S_pool) return KDA_ERR_INVALID_ARG;
    const void *pool = S_pool;
    if (pool == q || pool == k || pool == v || pool == (const void *)g || pool == fu.gate) return KDA_ERR_INVALID_ARG;
    const kda::LinearDecodeArgs a{q, k, v, g, g_per_token != 0, seq_idx, num_active, num_slots, H, H_qk, d_k, S_pool, o, status, fu};
    return kda::launch_linear_decode(a, in_dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_rope(const void *q, const void *k, const int32_t *positions, const uint64_t *steps, int32_t total_tokens,
                    int32_t H_q, int32_t H_k, int32_t d, int32_t rot, int32_t interleaved, float scale, kda_dtype in_dtype,
                    void *q_out, void *k_out, void *stream) {
    if (total_tokens < 0 || H_q < 0 || H_k < 0 || H_q > 65535 || H_k > 65535 || H_q + H_k == 0 || d <= 0 || rot < 2 || rot > d || rot % 2 ||
        !valid_dtype(in_dtype))
        return KDA_ERR_INVALID_ARG;
    if ((int64_t)total_tokens * (H_q + H_k) > INT_MAX || d > KDA_ROPE_MAX_D) return KDA_ERR_UNSUPPORTED;
    if (total_tokens == 0) return KDA_OK;
    const uintptr_t el = in_dtype == KDA_BF16 ? 1u : 3u;
    const auto given = [el](const void *p, int32_t heads) { return heads == 0 || (p && (reinterpret_cast<uintptr_t>(p) & el) == 0); };
    if (!given4(positions) || !steps || (reinterpret_cast<uintptr_t>(steps) & 7u) || !given(q, H_q) || !given(q_out, H_q) ||
        !given(k, H_k) || !given(k_out, H_k))
        return KDA_ERR_INVALID_ARG;
    // in place or apart, but not one in the other's place
    if (H_q && H_k && (q == k || q_out == k_out || q_out == k || k_out == q)) return KDA_ERR_INVALID_ARG;
    const kda::RopeArgs a{q, k, positions, reinterpret_cast<const unsigned long long *>(steps), total_tokens, H_q, H_k, d, rot,
                          interleaved != 0, scale, q_out, k_out};
    return kda::launch_rope(a, in_dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
