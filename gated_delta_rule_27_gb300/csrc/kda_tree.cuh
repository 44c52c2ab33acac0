// kda_tree.cuh -- packed draft trees, as the tree kernels read them.
//
// Request n owns rows [cu[n], cu[n + 1]) of every packed tensor; its first row is the tree's root and
// parent[row] is a local index below the row's own (-1: the root).  A tree is used only after
// read_tree() has found it inside these rules, so no index taken from it can leave its tensors.
#pragma once

#include "kda_internal.cuh"

namespace kda {

constexpr int kMaxNodes = KDA_TREE_MAX_NODES;

struct TreeShared {
    unsigned long long anc[kMaxNodes];  // bit a of anc[i]: node a lies on the path from the root to node i (i included)
    int parent[kMaxNodes];
    int bad;
};

struct Tree {
    int row0, nodes;
};

// Rows of request n, or nodes = -1 where cu breaks the rules (any thread; the same answer in all of them).
__device__ __forceinline__ Tree tree_rows(const int32_t *__restrict__ cu, int n, int total_nodes, int max_nodes) {
    const int lo = cu[n], hi = cu[n + 1];
    if (lo < 0 || hi < lo || hi > total_nodes || hi - lo > max_nodes) return Tree{0, -1};
    return Tree{lo, hi - lo};
}

// The parents of the nodes that a lane of warp `reader` checks (i = lane, lane + 32), asked for as early as the rows are
// known: read_tree() would wait for them alone.
struct Links {
    int p[2];
};
__device__ __forceinline__ Links load_links(const int32_t *__restrict__ parent, const Tree &t, int reader = 0) {
    const int lane = (int)threadIdx.x - 32 * reader;
    Links l{{-1, -1}};
#pragma unroll
    for (int r = 0; r < 2; ++r)
        if (lane >= 0 && lane < 32 && lane + 32 * r < t.nodes) l.p[r] = parent[t.row0 + lane + 32 * r];
    return l;
}

// Warp `reader` checks request n's tree, the block waits for it (one block barrier).  Returns false where it breaks
// the rules.  The paths (where they are wanted) come from pointer doubling: after r rounds a node's mask covers its 2^r
// nearest ancestors.  Trees of up to 16 nodes have mask and link in one word, so that a round is one exchange.
__device__ __forceinline__ bool read_tree(TreeShared &ts, const Tree &t, const Links &links, bool want_paths, int reader = 0) {
    const int lane = (int)threadIdx.x - 32 * reader;
    if (lane >= 0 && lane < 32) {
        bool bad = t.nodes < 0;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = lane + 32 * r, p = links.p[r];
            if (i < t.nodes) {
                bad |= i == 0 ? p != -1 : (p < 0 || p >= i);
                ts.parent[i] = p;
            }
        }
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) ts.bad = bad;
        if (want_paths && !bad) {
            if (t.nodes <= 16) {
                uint32_t w = lane < t.nodes ? 1u << lane | (uint32_t)(links.p[0] + 1) << 16 : 0u;
                for (int span = 1; span < t.nodes; span <<= 1) {
                    const uint32_t up = __shfl_sync(0xffffffffu, w, (int)(w >> 16) - 1);
                    if (w >> 16) w = ((w | up) & 0xffffu) | (up & 0xffff0000u);
                }
                if (lane < t.nodes) ts.anc[lane] = w & 0xffffu;
            } else {
                unsigned long long m[2] = {1ull << lane, 1ull << (lane + 32)};
                int jump[2] = {links.p[0], links.p[1]};
                for (int span = 1; span < t.nodes; span <<= 1) {
                    unsigned long long up[2];
                    int next[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int j = jump[r] < 0 ? 0 : jump[r];
                        const unsigned long long lo = __shfl_sync(0xffffffffu, m[0], j & 31);
                        const unsigned long long hi = __shfl_sync(0xffffffffu, m[1], j & 31);
                        const int nlo = __shfl_sync(0xffffffffu, jump[0], j & 31);
                        const int nhi = __shfl_sync(0xffffffffu, jump[1], j & 31);
                        up[r] = j < 32 ? lo : hi;
                        next[r] = j < 32 ? nlo : nhi;
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        if (jump[r] >= 0) {
                            m[r] |= up[r];
                            jump[r] = next[r];
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    if (lane + 32 * r < t.nodes) ts.anc[lane + 32 * r] = m[r];
            }
        }
    }
    __syncthreads();
    return !ts.bad;
}

// A log-decay, cut where its exponential is zero in fp32, so that sums along a path stay finite for a decay of -inf.
__device__ __forceinline__ float log_decay(float g) { return g < -110.f ? -110.f : g; }

// Row i of A (without beta) and of P by one warp, from the exponents of the path itself: going up from node i the decays
// between the two nodes are summed anew, so that the sum is no larger than what it says, however much the path as a whole
// decays (differences of sums from the root are off by 2^-24 of those sums: 1.4e-4 in o below 32 tokens of -200).  Some
// ancestors at a time, whose rows come with one wait and whose sums over the lanes share their exchanges (nine for four).
//   rows(a, k, g)  the lane's channels of a node's key (before its norm) and log-decay
//   factor(b)      the exponential of a log-decay
//   put(a, x, is_p)  takes the entry of ancestor a (node i itself among them), called by one lane for each
template <int Some, int C, typename Rows, typename Factor, typename Put>
__device__ __forceinline__ void pairs_of_node(const TreeShared &ts, int i, const float (&ki)[C], const float (&qi)[C], Rows rows,
                                              Factor factor, Put put) {
    static_assert(Some == 2 || Some == 4, "one of these many ancestors at a time");
    const int lane = threadIdx.x & 31;
    float b[C];
#pragma unroll
    for (int x = 0; x < C; ++x) b[x] = 0.f;
    for (int top = i; top >= 0;) {
        int at[Some];
        float k[Some][C], g[Some][C], v[2 * Some];
#pragma unroll
        for (int j = 0; j < Some; ++j) {
            at[j] = top;
#pragma unroll
            for (int x = 0; x < C; ++x) k[j][x] = g[j][x] = 0.f;
            if (top >= 0) {
                rows(top, k[j], g[j]);
                top = ts.parent[top];
            }
        }
#pragma unroll
        for (int j = 0; j < Some; ++j) {
            v[j] = v[Some + j] = 0.f;
#pragma unroll
            for (int x = 0; x < C; ++x) {
                const float e = k[j][x] * factor(b[x]);
                v[j] = fmaf(ki[x], e, v[j]);
                v[Some + j] = fmaf(qi[x], e, v[Some + j]);
                b[x] += g[j][x];
            }
        }
        // each exchange halves what a lane still sums: of 2 Some groups of lanes, group j ends up with v[j]
        constexpr int kLanes = 32 / (2 * Some);
#pragma unroll
        for (int half = Some; half; half >>= 1) {
            const bool upper = lane & (half * kLanes);
#pragma unroll
            for (int j = 0; j < half; ++j) {
                const float mine = upper ? v[j + half] : v[j], other = upper ? v[j] : v[j + half];
                v[j] = mine + __shfl_xor_sync(0xffffffffu, other, half * kLanes);
            }
        }
#pragma unroll
        for (int off = kLanes / 2; off; off >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
        const int j = lane / kLanes & (Some - 1);
        int a = j & 1 ? at[1] : at[0];
        if constexpr (Some == 4) a = j & 2 ? (j & 1 ? at[3] : at[2]) : a;
        if (lane % kLanes == 0 && a >= 0) put(a, v[0], lane >= 16);
    }
}

__device__ __forceinline__ void report_invalid(int32_t *status) {
    if (status) atomicCAS(status, 0, (int32_t)KDA_ERR_INVALID_ARG);
}

// The pool slot of request n, or -1 for one outside the pool.
__device__ __forceinline__ int slot_of(const int32_t *__restrict__ seq_idx, int n, int num_slots) {
    const int slot = seq_idx ? seq_idx[n] : n;
    return slot < 0 || slot >= num_slots ? -1 : slot;
}

}  // namespace kda
