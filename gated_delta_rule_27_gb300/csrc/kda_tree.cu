// kda_tree.cu -- KDA attention for a tree of drafted tokens over the state pool, and the pool's move along
// the accepted path.
//
// Speculative serving (Lecture 11, section 2, "Serving state" row: rollback must reconcile the KDA state)
// runs the target model once over every drafted token and keeps one path.  A copy of the d_k x d_v state per
// node would cost 64 KB each way per (node, head); but every node's state is the pool's state, decayed, plus
// one rank-one term per node of its path.  With b_i the log-decay summed along the path to node i and S the
// pool's state, which is read once and left alone:
//
//     u_i = beta_i (v_i - (k_i e^{b_i})^T S - sum_{a above i} (k_i . k_a e^{b_i - b_a}) u_a)
//     o_i = (q_i e^{b_i})^T S + sum_{a above i, and i} (q_i . k_a e^{b_i - b_a}) u_a
//
// and the state after the path that ends in node l is  e^{b_l} S + sum_a (k_a e^{b_l - b_a}) u_a^T, so the
// commit needs the stored u and no second recurrence: it is one pass over the state.
#include "kda_tree.cuh"

namespace kda {
namespace {

// ---------------------------------------------------------------------------
// Step, fp32 on the CUDA cores: any supported d and type
// ---------------------------------------------------------------------------
// One CTA per (request, head), one thread per state column.  Nodes go in blocks of kNB: a block's products
// with the state are accumulated in registers over one sweep of the state's rows, then its u follow by
// forward substitution in node order (a node's ancestors all have lower indices).
constexpr int kNB = 8;

template <typename Tin, int D>
__global__ void __launch_bounds__(D < 32 ? 32 : D)
tree_step_kernel(const Tin *__restrict__ q, const Tin *__restrict__ k, const Tin *__restrict__ v,
                 const float *__restrict__ g, const float *__restrict__ beta, const int32_t *__restrict__ parent,
                 const int32_t *__restrict__ cu, const int32_t *__restrict__ seq_idx, int H, int total_nodes,
                 int max_nodes, int num_slots, const float *__restrict__ S_pool, Tin *__restrict__ o,
                 float *__restrict__ u, int32_t *__restrict__ status, int qk_norm, float qk_eps,
                 const Tin *__restrict__ gate, const float *__restrict__ weight, float out_eps) {
    constexpr int NT = D < 32 ? 32 : D;
    extern __shared__ float sm[];
    __shared__ TreeShared ts;
    const int n = blockIdx.x / H, h = blockIdx.x % H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Tree t = read_tree(ts, parent, cu, n, total_nodes, max_nodes, true);
    const int slot = slot_of(seq_idx, n, num_slots);
    if (t.nodes < 0 || slot < 0) {
        if (tid == 0) report_invalid(status);
        return;
    }
    const int M = t.nodes;
    float *s_k = sm, *s_q = s_k + max_nodes * D, *s_b = s_q + max_nodes * D, *s_u = s_b + max_nodes * D;
    float *s_A = s_u + max_nodes * D, *s_P = s_A + max_nodes * max_nodes, *s_beta = s_P + max_nodes * max_nodes;
    const size_t row_stride = (size_t)H * D;
    const size_t base = ((size_t)t.row0 * H + h) * D;

    for (int i = tid; i < M; i += NT) s_beta[i] = beta[(size_t)(t.row0 + i) * H + h];
    for (int i = tid; i < M * D; i += NT) {
        const size_t at = base + (size_t)(i / D) * row_stride + i % D;
        s_k[i] = to_f32(k[at]);
        s_q[i] = to_f32(q[at]);
    }
    __syncthreads();
    if (qk_norm) {  // q, k L2-normalised in fp32: a warp per row
        for (int r = warp; r < 2 * M; r += NT / 32) {
            float *x = r < M ? s_k + r * D : s_q + (r - M) * D;
            float ss = 0.f;
            for (int c = lane; c < D; c += 32) ss = fmaf(x[c], x[c], ss);
#pragma unroll
            for (int off = 16; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float inv = rsqrtf(ss + qk_eps);
            for (int c = lane; c < D; c += 32) x[c] *= inv;
        }
    }
    // log-decay along the paths: each channel by its own thread, parents before children
    for (int c = tid; c < D; c += NT)
        for (int i = 0; i < M; ++i)
            s_b[i * D + c] = log_decay(g[base + (size_t)i * row_stride + c]) + (i ? s_b[ts.parent[i] * D + c] : 0.f);
    __syncthreads();
    // A and P: a warp per (node, ancestor); the exponent b_i - b_a is one of the path's own decays, so no
    // reference point is needed and no factor leaves the range of the decays themselves
    for (int p = warp; p < M * M; p += NT / 32) {
        const int i = p / M, a = p % M;
        if (!((ts.anc[i] >> a) & 1)) continue;
        float sa = 0.f, sp = 0.f;
        for (int c = lane; c < D; c += 32) {
            const float kd = s_k[a * D + c] * expf(s_b[i * D + c] - s_b[a * D + c]);
            sa = fmaf(s_k[i * D + c], kd, sa);
            sp = fmaf(s_q[i * D + c], kd, sp);
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) {
            sa += __shfl_xor_sync(0xffffffffu, sa, off);
            sp += __shfl_xor_sync(0xffffffffu, sp, off);
        }
        if (lane == 0) {
            s_A[i * M + a] = s_beta[i] * sa;
            s_P[i * M + a] = sp;
        }
    }
    __syncthreads();
    for (int i = tid; i < M * D; i += NT) {
        const float e = expf(s_b[i]);
        s_k[i] *= e;
        s_q[i] *= e;
    }
    __syncthreads();

    const float *S = S_pool + ((size_t)slot * H + h) * D * D;
    const int col = tid;
    for (int i0 = 0; i0 < M; i0 += kNB) {
        float x[kNB], y[kNB];
#pragma unroll
        for (int r = 0; r < kNB; ++r) x[r] = y[r] = 0.f;
        if (col < D) {
#pragma unroll 4
            for (int c = 0; c < D; ++c) {
                const float s = S[(size_t)c * D + col];
#pragma unroll
                for (int r = 0; r < kNB; ++r) {
                    if (i0 + r < M) {
                        x[r] = fmaf(s_k[(i0 + r) * D + c], s, x[r]);
                        y[r] = fmaf(s_q[(i0 + r) * D + c], s, y[r]);
                    }
                }
            }
        }
        __syncthreads();  // the block's rows of s_q are read: they take its outputs below
        if (col < D) {
#pragma unroll
            for (int r = 0; r < kNB; ++r) {
                const int i = i0 + r;
                if (i < M) {
                    const size_t at = base + (size_t)i * row_stride + col;
                    const unsigned long long anc = ts.anc[i];
                    float w = s_beta[i] * (to_f32(v[at]) - x[r]), out = y[r];
                    for (int a = 0; a < i; ++a) {
                        if ((anc >> a) & 1) {
                            w = fmaf(-s_A[i * M + a], s_u[a * D + col], w);
                            out = fmaf(s_P[i * M + a], s_u[a * D + col], out);
                        }
                    }
                    s_u[i * D + col] = w;
                    out = fmaf(s_P[i * M + i], w, out);
                    if (u) u[at] = w;
                    if (gate) s_q[i * D + col] = out;
                    else o[at] = from_f32<Tin>(out);
                }
            }
        }
    }
    if (gate) {  // gated output normalisation: a warp per row
        __syncthreads();
        for (int i = warp; i < M; i += NT / 32) {
            const float *x = s_q + i * D;
            float ss = 0.f;
            for (int c = lane; c < D; c += 32) ss = fmaf(x[c], x[c], ss);
#pragma unroll
            for (int off = 16; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float inv = rsqrtf(ss / (float)D + out_eps);
            for (int c = lane; c < D; c += 32) {
                const size_t at = base + (size_t)i * row_stride + c;
                o[at] = from_f32<Tin>(x[c] * inv * (weight ? weight[c] : 1.f) * sigmoidf(to_f32(gate[at])));
            }
        }
    }
}

template <typename Tin, int D>
cudaError_t launch_step_d(const TreeStepArgs &a, cudaStream_t st) {
    const size_t smem = ((size_t)4 * a.max_nodes * D + 2 * (size_t)a.max_nodes * a.max_nodes + a.max_nodes) * 4;
    auto *kernel = tree_step_kernel<Tin, D>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<a.num_seqs * a.H, D < 32 ? 32 : D, smem, st>>>(
        (const Tin *)a.q, (const Tin *)a.k, (const Tin *)a.v, a.g, a.beta, a.parent, a.cu, a.seq_idx, a.H,
        a.total_nodes, a.max_nodes, a.num_slots, a.S_pool, (Tin *)a.o, a.u, a.status, a.fu.qk_norm, a.fu.qk_eps,
        (const Tin *)a.fu.gate, a.fu.weight, a.fu.out_eps);
    return cudaGetLastError();
}

template <typename Tin>
cudaError_t launch_step_t(const TreeStepArgs &a, cudaStream_t st) {
    switch (a.d) {
        case 16: return launch_step_d<Tin, 16>(a, st);
        case 64: return launch_step_d<Tin, 64>(a, st);
        case 128: return launch_step_d<Tin, 128>(a, st);
        default: return cudaErrorInvalidValue;
    }
}

// ---------------------------------------------------------------------------
// Commit
// ---------------------------------------------------------------------------
// One CTA per (request, head), laid out like the decode step: each thread holds 16 rows by four columns of the
// state in registers, loaded before anything else.  The path is taken kChunk nodes at a time: with the decay
// to the chunk's end folded into its keys, a chunk is  S <- e^{b} S + sum_a (k_a e^{b - b_a}) u_a^T.
constexpr int kRows = 16, kChunk = 8;

template <typename Tin, int D>
__global__ void __launch_bounds__((D / 4) * (D / kRows))
tree_commit_kernel(const Tin *__restrict__ k, const float *__restrict__ g, const float *__restrict__ u,
                   const int32_t *__restrict__ cu, const int32_t *__restrict__ path,
                   const int32_t *__restrict__ path_len, const int32_t *__restrict__ seq_idx, int H, int total_nodes,
                   int path_stride, int num_slots, float *__restrict__ S_pool, int32_t *__restrict__ status,
                   int qk_norm, float qk_eps) {
    constexpr int CG = D / 4, NT = CG * (D / kRows);
    __shared__ float s_k[kChunk][D], s_dec[D];
    __shared__ __align__(16) float s_u[kChunk][D];
    __shared__ float s_scale[kChunk];
    __shared__ int s_row[kChunk];
    const int n = blockIdx.x / H, h = blockIdx.x % H, tid = threadIdx.x;
    const int len = path_len[n];
    if (len == 0) return;
    const Tree t = tree_rows(cu, n, total_nodes, kMaxNodes);
    const int slot = slot_of(seq_idx, n, num_slots);
    int bad = t.nodes < 0 || slot < 0 || len < 0 || len > path_stride || len > t.nodes;
    for (int i = tid; i < len && !bad; i += NT) {
        const int node = path[(size_t)n * path_stride + i];
        bad = node < 0 || node >= t.nodes;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) report_invalid(status);
        return;
    }
    const int cg = tid % CG, rg = tid / CG;
    float4 *Sv = reinterpret_cast<float4 *>(S_pool + ((size_t)slot * H + h) * D * D);
    float4 s[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) s[j] = __ldcs(&Sv[(size_t)(rg * kRows + j) * CG + cg]);

    for (int l0 = 0; l0 < len; l0 += kChunk) {
        const int L = min(kChunk, len - l0);
        __syncthreads();
        for (int i = tid; i < L; i += NT)  // (d = 16 runs four threads, fewer than a chunk has nodes)
            s_row[i] = t.row0 + path[(size_t)n * path_stride + l0 + i];
        __syncthreads();
        for (int i = tid; i < L * D; i += NT) {
            const size_t at = ((size_t)s_row[i / D] * H + h) * D + i % D;
            s_k[i / D][i % D] = to_f32(k[at]);
            s_u[i / D][i % D] = u[at];
        }
        __syncthreads();
        if (qk_norm) {  // a group of min(NT, 32) threads per row
            constexpr int G = NT < 32 ? NT : 32;
            const int lane = tid % G;
            for (int r = tid / G; r < kChunk; r += NT / G) {
                float ss = 0.f;
                if (r < L)
                    for (int c = lane; c < D; c += G) ss = fmaf(s_k[r][c], s_k[r][c], ss);
#pragma unroll
                for (int off = G / 2; off; off >>= 1)
                    ss += __shfl_xor_sync(G == 32 ? 0xffffffffu : (1u << G) - 1u, ss, off);
                if (lane == 0) s_scale[r] = rsqrtf(ss + qk_eps);
            }
            __syncthreads();
        }
        for (int c = tid; c < D; c += NT) {  // decays to the chunk's end, per channel
            float b = 0.f;
            for (int r = L - 1; r >= 0; --r) {
                s_k[r][c] *= expf(b) * (qk_norm ? s_scale[r] : 1.f);
                b += log_decay(g[((size_t)s_row[r] * H + h) * D + c]);
            }
            s_dec[c] = expf(b);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const float d = s_dec[rg * kRows + j];
            s[j].x *= d; s[j].y *= d; s[j].z *= d; s[j].w *= d;
        }
        for (int r = 0; r < L; ++r) {
            const float4 w = *reinterpret_cast<const float4 *>(&s_u[r][cg * 4]);
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                const float kr = s_k[r][rg * kRows + j];
                s[j].x = fmaf(kr, w.x, s[j].x); s[j].y = fmaf(kr, w.y, s[j].y);
                s[j].z = fmaf(kr, w.z, s[j].z); s[j].w = fmaf(kr, w.w, s[j].w);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) __stcs(&Sv[(size_t)(rg * kRows + j) * CG + cg], s[j]);
}

template <typename Tin, int D>
cudaError_t launch_commit_d(const TreeCommitArgs &a, cudaStream_t st) {
    tree_commit_kernel<Tin, D><<<a.num_seqs * a.H, (D / 4) * (D / kRows), 0, st>>>(
        (const Tin *)a.k, a.g, a.u, a.cu, a.path, a.path_len, a.seq_idx, a.H, a.total_nodes, a.path_stride,
        a.num_slots, a.S_pool, a.status, a.qk_norm, a.qk_eps);
    return cudaGetLastError();
}

template <typename Tin>
cudaError_t launch_commit_t(const TreeCommitArgs &a, cudaStream_t st) {
    switch (a.d) {
        case 16: return launch_commit_d<Tin, 16>(a, st);
        case 64: return launch_commit_d<Tin, 64>(a, st);
        case 128: return launch_commit_d<Tin, 128>(a, st);
        default: return cudaErrorInvalidValue;
    }
}

// ---------------------------------------------------------------------------
// Short convolution along the paths
// ---------------------------------------------------------------------------
// y_i[c] = sum_j w[c, j] x_{j-th ancestor of i}[c]; past the root the request's carried inputs follow, newest
// first.  One CTA per (request, 128 channels).
constexpr int kConvThreads = 128;

template <typename Tin, int W>
__global__ void __launch_bounds__(kConvThreads)
tree_conv_kernel(const Tin *__restrict__ x, const float *__restrict__ w, const int32_t *__restrict__ parent,
                 const int32_t *__restrict__ cu, const int32_t *__restrict__ seq_idx, int total_nodes, int max_nodes,
                 int num_slots, int C, const float *__restrict__ pool, Tin *__restrict__ y,
                 int32_t *__restrict__ status) {
    __shared__ TreeShared ts;
    const int n = blockIdx.y, c = blockIdx.x * kConvThreads + threadIdx.x;
    const Tree t = read_tree(ts, parent, cu, n, total_nodes, max_nodes, false);
    const int slot = slot_of(seq_idx, n, num_slots);
    if (t.nodes < 0 || slot < 0) {
        if (threadIdx.x == 0) report_invalid(status);
        return;
    }
    if (c >= C) return;
    float wt[W], past[W];  // past[j]: the j-th input before the root
#pragma unroll
    for (int j = 0; j < W; ++j) {
        wt[j] = w[(size_t)c * W + j];
        past[j] = j < W - 1 ? pool[((size_t)slot * (W - 1) + (W - 2 - j)) * C + c] : 0.f;
    }
    for (int i = 0; i < t.nodes; ++i) {
        float acc = 0.f;
        int at = i, carried = 0;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float xv = 0.f;
            if (at >= 0) {
                xv = to_f32(x[(size_t)(t.row0 + at) * C + c]);
                at = ts.parent[at];
            } else {
#pragma unroll
                for (int m = 0; m < W; ++m) xv = m == carried ? past[m] : xv;
                ++carried;
            }
            acc = fmaf(wt[j], xv, acc);
        }
        y[(size_t)(t.row0 + i) * C + c] = from_f32<Tin>(acc);
    }
}

// The carried inputs after a path: the last W - 1 of [carried inputs, the path's inputs].
template <typename Tin>
__global__ void __launch_bounds__(kConvThreads)
tree_conv_commit_kernel(const Tin *__restrict__ x, const int32_t *__restrict__ cu, const int32_t *__restrict__ path,
                        const int32_t *__restrict__ path_len, const int32_t *__restrict__ seq_idx, int total_nodes,
                        int path_stride, int num_slots, int C, int W, float *__restrict__ pool,
                        int32_t *__restrict__ status) {
    const int n = blockIdx.y, c = blockIdx.x * kConvThreads + threadIdx.x;
    const int len = path_len[n];
    if (len == 0) return;
    const Tree t = tree_rows(cu, n, total_nodes, kMaxNodes);
    const int slot = slot_of(seq_idx, n, num_slots);
    bool bad = t.nodes < 0 || slot < 0 || len < 0 || len > path_stride || len > t.nodes;
    int node[KDA_SHORT_CONV_MAX_W - 1];  // node of the new carried input j, or -1 for an old one
    for (int j = 0; j < W - 1 && !bad; ++j) {
        const int l = len - (W - 1) + j;
        node[j] = -1;
        if (l >= 0) {
            node[j] = path[(size_t)n * path_stride + l];
            bad = node[j] < 0 || node[j] >= t.nodes;
        }
    }
    if (bad) {
        if (threadIdx.x == 0) report_invalid(status);
        return;
    }
    if (c >= C) return;
    float next[KDA_SHORT_CONV_MAX_W - 1];
    for (int j = 0; j < W - 1; ++j)
        next[j] = node[j] >= 0 ? to_f32(x[(size_t)(t.row0 + node[j]) * C + c])
                               : pool[((size_t)slot * (W - 1) + j + len) * C + c];
    for (int j = 0; j < W - 1; ++j) pool[((size_t)slot * (W - 1) + j) * C + c] = next[j];
}

template <typename Tin>
cudaError_t launch_conv_t(const TreeConvArgs &a, cudaStream_t st) {
    const dim3 grid((a.C + kConvThreads - 1) / kConvThreads, a.num_seqs);
#define KDA_TREE_CONV(WW)                                                                                          \
    case WW:                                                                                                       \
        tree_conv_kernel<Tin, WW><<<grid, kConvThreads, 0, st>>>((const Tin *)a.x, a.w, a.parent, a.cu, a.seq_idx, \
                                                                 a.total_nodes, a.max_nodes, a.num_slots, a.C,     \
                                                                 a.pool, (Tin *)a.y, a.status);                    \
        break;
    switch (a.W) {
        KDA_TREE_CONV(1) KDA_TREE_CONV(2) KDA_TREE_CONV(3) KDA_TREE_CONV(4)
        KDA_TREE_CONV(5) KDA_TREE_CONV(6) KDA_TREE_CONV(7) KDA_TREE_CONV(8)
        default: return cudaErrorInvalidValue;
    }
#undef KDA_TREE_CONV
    return cudaGetLastError();
}

template <typename Tin>
cudaError_t launch_conv_commit_t(const TreeConvCommitArgs &a, cudaStream_t st) {
    const dim3 grid((a.C + kConvThreads - 1) / kConvThreads, a.num_seqs);
    tree_conv_commit_kernel<Tin><<<grid, kConvThreads, 0, st>>>((const Tin *)a.x, a.cu, a.path, a.path_len, a.seq_idx,
                                                                a.total_nodes, a.path_stride, a.num_slots, a.C, a.W,
                                                                a.pool, a.status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_step(const TreeStepArgs &a, kda_dtype dt, cudaStream_t st) {
    if (dt == KDA_BF16 && a.d == 128) return launch_tree_step_tc(a, st);
    return dt == KDA_BF16 ? launch_step_t<__nv_bfloat16>(a, st) : launch_step_t<float>(a, st);
}
cudaError_t launch_tree_commit(const TreeCommitArgs &a, kda_dtype dt, cudaStream_t st) {
    return dt == KDA_BF16 ? launch_commit_t<__nv_bfloat16>(a, st) : launch_commit_t<float>(a, st);
}
cudaError_t launch_tree_conv(const TreeConvArgs &a, kda_dtype dt, cudaStream_t st) {
    return dt == KDA_BF16 ? launch_conv_t<__nv_bfloat16>(a, st) : launch_conv_t<float>(a, st);
}
cudaError_t launch_tree_conv_commit(const TreeConvCommitArgs &a, kda_dtype dt, cudaStream_t st) {
    return dt == KDA_BF16 ? launch_conv_commit_t<__nv_bfloat16>(a, st) : launch_conv_commit_t<float>(a, st);
}

}  // namespace kda
