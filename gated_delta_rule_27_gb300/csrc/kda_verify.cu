// kda_verify.cu -- verification of drafted tokens against the target's probabilities, from given random numbers.
//
// Rejection sampling over a draft tree keeps the target's distribution.  At a node with target weights
// w_t = 2^{(l_t - max l) log2(e) / T} and the draft distribution q its children were drawn from, the children
// are tried in order; with r = w, s = sum w, C = 0 at first:
//     accept child c if u_c q_c s < r_c;  else  C += s,  r_t = max(w_t - C q_t, 0),  s = sum r.
// (After a rejection the target is the normalised excess max(p - q, 0) of p = r / s; in units of w that excess
// is max(w - C q, 0) with C the sum of all s before it, so one scalar carries any number of rejections.)
// Without q the drafts were chosen, not drawn: q is one at the child, and a rejection removes its token from r.
// At the node that accepts no child the next token is drawn from r by inversion of its cumulative sum.
//
// Sums over the vocabulary are exact: every term is cut to a multiple of 2^-40 and added as an integer, so
// neither the split of the row nor the order of the additions can change a decision.
#include "kda_tree.cuh"

namespace kda {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kVec = 4;
constexpr float kFixed = 1099511627776.f;  // 2^40

__device__ __forceinline__ unsigned long long fixed40(float x) { return __float2ull_rz(x * kFixed); }

// What a row's weights are computed from.
struct RowStats {
    float top, scale;
    int best;   // the lowest index of the largest logit; -1: no logit above -inf
    int onehot; // all the weight at `best` (temperature 0)
};
// w_t.  NaN logits weigh nothing; logits of +inf share the weight.
__device__ __forceinline__ float weight_of(const RowStats &r, float l, int t) {
    if (r.onehot) return t == r.best ? 1.f : 0.f;
    if (l == r.top) return 1.f;  // also where both are +inf
    return fmaxf(exp2f(__fmul_rn(__fsub_rn(l, r.top), r.scale)), 0.f);
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long x) {
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

struct Shared {
    TreeShared tree;
    unsigned long long sum[kWarps];
    float top[kWarps];
    int best[kWarps];
    int removed[kMaxNodes];
    int found;
};

__device__ __forceinline__ unsigned long long block_sum(Shared &sh, unsigned long long x) {
    x = warp_sum(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.sum[threadIdx.x >> 5] = x;
    __syncthreads();
    unsigned long long total = 0;
    for (int w = 0; w < kWarps; ++w) total += sh.sum[w];
    return total;
}

// r_t of the row after its rejections
template <typename Tin>
__device__ __forceinline__ float rest_of(const Shared &sh, const RowStats &st, const Tin *row, const float *q, float C,
                                         int removed, int t) {
    const float w = weight_of(st, to_f32(row[t]), t);
    if (q) return C > 0.f ? fmaxf(__fsub_rn(w, __fmul_rn(C, q[t])), 0.f) : w;
    for (int i = 0; i < removed; ++i)
        if (sh.removed[i] == t) return 0.f;
    return w;
}

template <typename Tin>
__global__ void __launch_bounds__(kThreads)
draft_verify_kernel(const Tin *__restrict__ logits, const float *__restrict__ probs, const int32_t *__restrict__ tokens,
                    const int32_t *__restrict__ parent, const int32_t *__restrict__ cu,
                    const float *__restrict__ temperature, const float *__restrict__ u,
                    const float *__restrict__ u_next, int total_nodes, int V, int path_stride,
                    int32_t *__restrict__ path, int32_t *__restrict__ path_len, int32_t *__restrict__ next_token,
                    int32_t *__restrict__ status) {
    __shared__ Shared sh;
    const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Tree t = read_tree(sh.tree, parent, cu, n, total_nodes, min(path_stride, kMaxNodes), false);
    if (t.nodes < 0 && tid == 0) report_invalid(status);
    int len = 0, next = -1;
    if (t.nodes > 0) {
        const float temp = temperature ? temperature[n] : 1.f;
        int node = 0;
        for (;;) {
            if (tid == 0) path[(size_t)n * path_stride + len] = node;
            ++len;
            const Tin *row = logits + (size_t)(t.row0 + node) * V;
            const float *q = probs ? probs + (size_t)(t.row0 + node) * V : nullptr;
            // the largest logit and its lowest index
            RowStats st;
            st.top = -INFINITY;
            st.best = -1;
            for (int i = tid; i < V; i += kThreads) {
                const float l = to_f32(row[i]);
                if (l > st.top) { st.top = l; st.best = i; }
            }
#pragma unroll
            for (int off = 16; off; off >>= 1) {
                const float l = __shfl_xor_sync(0xffffffffu, st.top, off);
                const int b = __shfl_xor_sync(0xffffffffu, st.best, off);
                if (l > st.top || (l == st.top && b < st.best)) { st.top = l; st.best = b; }
            }
            __syncthreads();
            if (lane == 0) { sh.top[warp] = st.top; sh.best[warp] = st.best; }
            __syncthreads();
            st.top = -INFINITY;
            st.best = -1;
            for (int w = 0; w < kWarps; ++w)
                if (sh.top[w] > st.top || (sh.top[w] == st.top && sh.best[w] < st.best)) {
                    st.top = sh.top[w];
                    st.best = sh.best[w];
                }
            st.onehot = !(temp > 0.f);
            st.scale = st.onehot ? 0.f : 1.4426950408889634f / temp;
            if (st.best < 0) break;  // no weight anywhere
            unsigned long long part = 0;
            for (int i = tid; i < V; i += kThreads) part += fixed40(weight_of(st, to_f32(row[i]), i));
            const unsigned long long Z = block_sum(sh, part);
            unsigned long long s = Z;
            float C = 0.f;
            int removed = 0, accepted = -1;
            for (int j = node + 1; j < t.nodes && accepted < 0; ++j) {
                if (sh.tree.parent[j] != node) continue;
                const int token = tokens[t.row0 + j];
                if (token < 0 || token >= V) {
                    if (tid == 0) report_invalid(status);
                    continue;
                }
                const float r = rest_of(sh, st, row, q, C, removed, token);
                const float sf = __ull2float_rn(s) * (1.f / kFixed), qc = q ? q[token] : 1.f;
                if (__fmul_rn(__fmul_rn(u[t.row0 + j], qc), sf) < r) {
                    accepted = j;
                } else if (q) {
                    C = __fadd_rn(C, sf);
                    part = 0;
                    for (int i = tid; i < V; i += kThreads) part += fixed40(rest_of(sh, st, row, q, C, 0, i));
                    s = block_sum(sh, part);
                } else {
                    s -= fixed40(r);
                    __syncthreads();
                    if (tid == 0) sh.removed[removed] = token;
                    ++removed;
                    __syncthreads();
                }
            }
            if (accepted >= 0) {
                node = accepted;
                continue;
            }
            if (s == 0) {  // nothing is left of the target: its own distribution
                s = Z;
                C = 0.f;
                removed = 0;
                q = nullptr;
            }
            // the next token: the first one whose cumulative sum is above u s
            const double un = (double)u_next[n];
            unsigned long long at = un > 0.0 ? (unsigned long long)(un * (double)s) : 0ull;
            if (at >= s) at = s - 1;
            unsigned long long before = 0;
            for (int i0 = 0; i0 < V && next < 0; i0 += kThreads * kVec) {
                unsigned long long f[kVec], mine = 0;
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const int i = i0 + tid * kVec + e;
                    f[e] = i < V ? fixed40(rest_of(sh, st, row, q, C, removed, i)) : 0ull;
                    mine += f[e];
                }
                unsigned long long upto = mine;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const unsigned long long x = __shfl_up_sync(0xffffffffu, upto, off);
                    if (lane >= off) upto += x;
                }
                __syncthreads();
                if (lane == 31) sh.sum[warp] = upto;
                if (tid == 0) sh.found = -1;
                __syncthreads();
                unsigned long long base = before + upto - mine;
                for (int w = 0; w < kWarps; ++w) {
                    if (w < warp) base += sh.sum[w];
                    before += sh.sum[w];
                }
                if (base <= at && at < base + mine) {
                    int e = 0;
                    while (base + f[e] <= at) base += f[e++];
                    sh.found = i0 + tid * kVec + e;
                }
                __syncthreads();
                next = sh.found;
            }
            break;
        }
    }
    for (int i = len + tid; i < path_stride; i += kThreads) path[(size_t)n * path_stride + i] = -1;
    if (tid == 0) {
        path_len[n] = len;
        next_token[n] = next;
    }
}

}  // namespace

cudaError_t launch_draft_verify(const DraftVerifyArgs &a, kda_dtype dt, cudaStream_t st) {
    if (dt == KDA_BF16)
        draft_verify_kernel<__nv_bfloat16><<<a.num_seqs, kThreads, 0, st>>>(
            (const __nv_bfloat16 *)a.logits, a.probs, a.tokens, a.parent, a.cu, a.temperature, a.u, a.u_next,
            a.total_nodes, a.V, a.path_stride, a.path, a.path_len, a.next_token, a.status);
    else
        draft_verify_kernel<float><<<a.num_seqs, kThreads, 0, st>>>(
            (const float *)a.logits, a.probs, a.tokens, a.parent, a.cu, a.temperature, a.u, a.u_next, a.total_nodes,
            a.V, a.path_stride, a.path, a.path_len, a.next_token, a.status);
    return cudaGetLastError();
}

}  // namespace kda
