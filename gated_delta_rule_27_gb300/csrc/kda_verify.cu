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
//
// Only the rows that the walk visits are read.  One cluster of CTAs serves a request; each CTA keeps its part of
// the visited row in shared memory, so that the maximum, the sum, the excess after a rejection and the search
// for the next token all work on one read of the row.
//
// What bounds it is the walk's length: visited nodes, one after the other, each with an exchange between the
// cluster's CTAs.  So a node's first trial is decided from an fp32 sum that comes with the maximum in one exchange,
// wherever that decides it; the exact sums are formed only where a trial is closer than that, or lost.  (kMargin covers
// the sum's error: of a row of 2^22 logits, the longest, a thread adds 1024 values to each of two sums, 6e-5 of them at
// worst, and the cuts to 2^-40 take 4e-6; at 131072 logits it is below 5e-6 in all.)  Meanwhile the first child's row is
// on its way to L2.
// Measured: one request, a chain of 5 drafted from given distributions, 32768 fp32 logits a row: 9 to 15 us with the walk's length; 64 requests with
// trees of 9 to 16 nodes over 131072 bf16 logits 45 to 55 us; 256 chains of 4 to 8 without distributions over 100003 56 to 60 us.
// The others wait for the longest walk of the batch, several rejections among its trials at about 5 us each: DRAM is
// 17% busy.
#include <cooperative_groups.h>

#include "kda_tc.cuh"
#include "kda_tree.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kMaxCluster = 8;
constexpr uint32_t kMaxPart = 65536;  // bytes of a row that a CTA keeps; a longer part is read again by every pass
constexpr int kRuns = kMaxPart / 16 / 32;  // a run: the 32 vectors of 16 bytes that a warp takes at once
constexpr float kFixed = 1099511627776.f;  // 2^40
constexpr float kMargin = 1e-4f;
constexpr uint64_t kWaitNs = 1000000000ull;  // for an exchange

__device__ __forceinline__ unsigned long long fixed40(float x) { return __float2ull_rz(x * kFixed); }

// A sum of at most 8 values in [0, 1] cut to multiples of 2^-40, without 64-bit conversions: adding 1 with rounding
// towards zero leaves the first 23 bits of the value in the sum's mantissa, adding 2^-17 to the rest the next 17;
// the bit patterns add up as integers, and so do 32 lanes' (8 x 32 x 2^23 fits 32 bits).
struct FixedSum {
    uint32_t hi = 0, lo = 0;
    __device__ __forceinline__ void add2(float2 x) {
        const float2 a = tc::add_rz2(x, make_float2(1.f, 1.f));
        const float2 b = tc::add_rz2(tc::sub2(x, tc::sub2(a, make_float2(1.f, 1.f))), make_float2(0x1p-17f, 0x1p-17f));
        hi += __float_as_uint(a.x) + __float_as_uint(a.y) - 2 * 0x3f800000u;
        lo += __float_as_uint(b.x) + __float_as_uint(b.y) - 2 * 0x37000000u;
    }
    __device__ __forceinline__ unsigned long long mine() const { return ((unsigned long long)hi << 17) + lo; }
    __device__ __forceinline__ unsigned long long of_warp() const {
        return ((unsigned long long)__reduce_add_sync(0xffffffffu, hi) << 17) + __reduce_add_sync(0xffffffffu, lo);
    }
};

// What a row's weights are computed from.
struct Row {
    float top, scale;
    int best;    // the lowest index of the largest logit; -1: no logit above -inf
    bool onehot; // all the weight at `best` (temperature 0)
    bool flat;   // top is +inf: the weight is one at +inf and zero elsewhere
};
// 2^x; below 2^-126, far below the sums' resolution, it is zero
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// w_t of a row with a spread-out weight; a NaN logit weighs nothing
__device__ __forceinline__ float weight_of(const Row &r, float l) {
    if (r.flat) return l == r.top ? 1.f : 0.f;
    return fmaxf(exp2_of(__fmul_rn(__fsub_rn(l, r.top), r.scale)), 0.f);
}
__device__ __forceinline__ float excess_of(float w, float C, float q) { return fmaxf(__fsub_rn(w, __fmul_rn(C, q)), 0.f); }
// Pairs of the same.  `plain`: the row has neither a NaN nor a +inf logit.
__device__ __forceinline__ float2 weights_of(const Row &r, bool plain, float2 l) {
    if (!plain) return make_float2(weight_of(r, l.x), weight_of(r, l.y));
    const float2 x = tc::mul2(tc::sub2(l, make_float2(r.top, r.top)), make_float2(r.scale, r.scale));
    return make_float2(exp2_of(x.x), exp2_of(x.y));
}
__device__ __forceinline__ float2 excesses_of(float2 w, float C, float2 q) {
    const float2 x = tc::sub2(w, tc::mul2(make_float2(C, C), q));
    return make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f));
}

struct __align__(16) Found {  // a maximum, its lowest index, and (to fp32) the sum of the weights relative to it
    float top;
    int best;
    float sum;
    float unused;
};
// The largest of the warp's values, and the lowest index that goes with it.
__device__ __forceinline__ Found best_of_warp(float top, int best) {
    const uint32_t bits = __float_as_uint(top + 0.f);  // (-0 becomes 0)
    const uint32_t key = bits & 0x80000000u ? ~bits : bits | 0x80000000u;  // ordered as the values are
    const uint32_t most = __reduce_max_sync(0xffffffffu, key);
    Found f;
    f.top = __uint_as_float(most & 0x80000000u ? most & 0x7fffffffu : ~most);
    f.best = (int)__reduce_min_sync(0xffffffffu, key == most ? (uint32_t)best : 0xffffffffu);
    f.sum = f.unused = 0.f;
    return f;
}
// The same over the entries that the lanes hold, lane l the entry l mod n (n a power of two), with the sums, which
// become NaN where a logit is NaN or +inf.
__device__ __forceinline__ Found merged(Found f, int n, float scale) {
    Found a = best_of_warp(f.top, f.best);
    a.sum = f.top > -INFINITY ? f.sum * exp2_of((f.top - a.top) * scale) : f.sum;  // (there: zero or NaN)
    for (int off = n >> 1; off; off >>= 1) a.sum += __shfl_xor_sync(0xffffffffu, a.sum, off);
    return a;
}

struct Shared {
    TreeShared tree;
    unsigned long long child[kMaxNodes];            // children of each node
    int token[kMaxNodes];                           // each node's token, or -1 for one outside the vocabulary
    float u[kMaxNodes], logit[kMaxNodes], q[kMaxNodes];  // its number, and its parent's logit and q for its token
    int path[kMaxNodes];                            // the nodes visited
    int removed[kMaxNodes];                         // tokens rejected at the visited node, when there is no q
    unsigned long long removed_w[kMaxNodes];
    unsigned long long part[kRuns];                 // the exact sums of the CTA's runs (of a part that is kept)
    unsigned long long warp_sum[kWarps];
    Found warp_max[kWarps];
    Found cta_max[2][kMaxCluster];                  // exchanged: two places, taken in turn, each with its barrier
    unsigned long long cta_sum[2][kMaxCluster];
    uint64_t bar[2];
    unsigned long long sum_w[kMaxCluster], sum_r[kMaxCluster];
};

// An exchange between the cluster's CTAs: each sends its value to every other's place for it, and goes on once its
// own places are filled.  Two sets of places are enough: a CTA sends for exchange e + 2 only with all values of
// e + 1 in hand, whose senders had read theirs of e.
struct Exchange {
    int count = 0, size = 1, rank = 0;
    bool ok = true;  // every wait so far was met (the same in all threads of the CTA)
    __device__ __forceinline__ int turn() const { return count & 1; }
    __device__ __forceinline__ void expect(Shared &sh, uint32_t bytes) const {
        if (threadIdx.x == 0) tc::mbar_arrive_expect_tx(&sh.bar[turn()], bytes * size);
    }
    __device__ __forceinline__ void wait(Shared &sh, uint64_t wait_ns) {
        ok = __syncthreads_and(ok && tc::mbar_wait(&sh.bar[turn()], (count >> 1) & 1, wait_ns));
        ++count;
    }
};

// Every thread gets the CTAs' sums in sums[] (shared memory) and their total; x is the warp's sum (in lane 0).
__device__ __forceinline__ unsigned long long cluster_sum(Shared &sh, Exchange &ex, uint64_t wait_ns, unsigned long long x,
                                                          unsigned long long *sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, turn = ex.turn();
    if (lane == 0) sh.warp_sum[warp] = x;
    ex.expect(sh, 8);
    __syncthreads();
    if (threadIdx.x < ex.size) {
        unsigned long long total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) total += sh.warp_sum[w];
        tc::st_async_b64(tc::map_to_cta(&sh.cta_sum[turn][ex.rank], threadIdx.x), total,
                         tc::map_to_cta(&sh.bar[turn], threadIdx.x));
    }
    ex.wait(sh, wait_ns);
    unsigned long long total = 0;
    for (int r = 0; r < ex.size; ++r) total += sh.cta_sum[turn][r];
    if (threadIdx.x < ex.size) sums[threadIdx.x] = sh.cta_sum[turn][threadIdx.x];
    return total;
}

// f.top and f.best are the thread's, f.sum the thread's relative to its warp's maximum (which f.top has become).
__device__ __forceinline__ Found cluster_max(Shared &sh, Exchange &ex, uint64_t wait_ns, float scale, Found f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, turn = ex.turn();
    float sum = f.sum;
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    f = best_of_warp(f.top, f.best);
    f.sum = sum;
    if (lane == 0) sh.warp_max[warp] = f;
    ex.expect(sh, 16);
    __syncthreads();
    if (warp == 0) {
        const Found a = merged(sh.warp_max[lane % kWarps], kWarps, scale);
        if (lane < ex.size)
            tc::st_async_b32x4(tc::map_to_cta(&sh.cta_max[turn][ex.rank], lane), __float_as_uint(a.top), (uint32_t)a.best,
                               __float_as_uint(a.sum), 0u, tc::map_to_cta(&sh.bar[turn], lane));
    }
    ex.wait(sh, wait_ns);
    return merged(sh.cta_max[turn][lane & (ex.size - 1)], ex.size, scale);
}

// A CTA's part of one row.  The row is cut at 16-byte boundaries of memory into vectors of `kVec` logits, of which
// the first and last may be partial; `lead` is the number of places before the row's first logit in vector 0.
template <typename Tin>
struct Part {
    static constexpr int kVec = 16 / sizeof(Tin);
    const Tin *row;
    uint4 *kept;  // the part in shared memory, or null
    int lead, V, v0, v1;

    __device__ __forceinline__ uint4 load(int v) const {
        const int i0 = v * kVec - lead;
        if (i0 >= 0 && i0 + kVec <= V) return __ldg(reinterpret_cast<const uint4 *>(row + i0));
        union {
            uint4 vec;
            Tin x[kVec];
        } out;
#pragma unroll
        for (int e = 0; e < kVec; ++e) out.x[e] = i0 + e >= 0 && i0 + e < V ? row[i0 + e] : from_f32<Tin>(-INFINITY);
        return out.vec;
    }
    // Starts the copy of the part to shared memory (complete after cp_async_wait_all and a block barrier).
    __device__ __forceinline__ void fetch() const {
        if (!kept) return;
        for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
            const int i0 = v * kVec - lead;
            if (i0 >= 0 && i0 + kVec <= V) tc::cp_async16(kept + (v - v0), row + i0);
            else kept[v - v0] = load(v);
        }
    }
    // Asks L2 for the part of another row (its 128-byte lines).
    __device__ __forceinline__ void ask(const Tin *other) const {
        const char *first = reinterpret_cast<const char *>(other) + (size_t)max(0, v0 * kVec - lead) * sizeof(Tin);
        const char *end = reinterpret_cast<const char *>(other) + (size_t)min(V, v1 * kVec - lead) * sizeof(Tin);
        for (const char *at = first + threadIdx.x * 128; at < end; at += kThreads * 128) tc::prefetch_l2(at);
    }
    __device__ __forceinline__ void ask_q(const float *q) const {
        for (int i = max(0, v0 * kVec - lead) + threadIdx.x * 32; i < min(V, v1 * kVec - lead); i += kThreads * 32)
            tc::prefetch_l2(q + i);
    }
    __device__ __forceinline__ void get(int v, float (&l)[kVec]) const {
        const uint4 x = kept ? kept[v - v0] : load(v);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (sizeof(Tin) == 4) {
                l[e] = __uint_as_float(w[e]);
            } else {
                l[2 * e] = __uint_as_float(w[e] << 16);
                l[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
            }
        }
    }
    // The largest of a vector's logits (of NaN and a number, the number).
    __device__ __forceinline__ float top(int v) const {
        const uint4 x = kept ? kept[v - v0] : load(v);
        if constexpr (sizeof(Tin) == 4) {
            return fmaxf(fmaxf(__uint_as_float(x.x), __uint_as_float(x.y)), fmaxf(__uint_as_float(x.z), __uint_as_float(x.w)));
        } else {
            const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&x);
            const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
            return fmaxf(__bfloat162float(m.x), __bfloat162float(m.y));
        }
    }
    __device__ __forceinline__ void get_q(const float *q, int v, float (&x)[kVec]) const {
        const int i0 = v * kVec - lead;
        const float *at = q + i0;
        if (i0 >= 0 && i0 + kVec <= V && (reinterpret_cast<uintptr_t>(at) & 15u) == 0) {
#pragma unroll
            for (int e = 0; e < kVec / 4; ++e) {
                const float4 y = __ldg(reinterpret_cast<const float4 *>(at) + e);
                x[4 * e] = y.x; x[4 * e + 1] = y.y; x[4 * e + 2] = y.z; x[4 * e + 3] = y.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[e] = i0 + e >= 0 && i0 + e < V ? __ldg(at + e) : 0.f;
        }
    }
};

// The sum of the lanes up to this one.
__device__ __forceinline__ unsigned long long scan(unsigned long long x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    return x;
}

struct Args {
    const void *logits;
    const float *probs;
    const int32_t *tokens, *parent, *cu;
    const float *temperature, *u, *u_next;
    int total_nodes, V, path_stride;
    uint32_t part_bytes;  // of dynamic shared memory: 0 where a part would not fit
    uint64_t wait_ns;     // how long an exchange is waited for
    bool silent;          // tests of the failure path: each request's last CTA leaves its exchanges unsent
    int32_t *path, *path_len, *next_token, *status;
};

template <typename Tin>
__global__ void __launch_bounds__(kThreads, 4) draft_verify_kernel(const Args p) {
    using P = Part<Tin>;
    constexpr int kBatch = 16 / P::kVec;
    extern __shared__ uint4 kept[];
    __shared__ Shared sh;
    tc::grid_dep_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const int size = cluster.num_blocks(), rank = cluster.block_rank();
    const int n = blockIdx.x / size, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool writer = rank == 0 && tid == 0;
    Row r{};
    P part{};
    part.V = p.V;
    part.kept = p.part_bytes ? kept : nullptr;
    int each = 0;
    auto place = [&](int row) {  // this CTA's part of a row
        part.row = reinterpret_cast<const Tin *>(p.logits) + (size_t)row * p.V;
        part.lead = (int)((reinterpret_cast<uintptr_t>(part.row) & 15u) / sizeof(Tin));
        const int vectors = (part.lead + p.V + P::kVec - 1) / P::kVec;
        each = (vectors + size - 1) / size;
        part.v0 = min(vectors, rank * each);
        part.v1 = min(vectors, part.v0 + each);
    };
    const Tree root = tree_rows(p.cu, n, p.total_nodes, min(p.path_stride, kMaxNodes));
    if (root.nodes > 0) {  // its row is on its way before the tree has been read
        place(root.row0);
        part.fetch();
    }
    if (tid == 0) {
        tc::mbar_init(&sh.bar[0], 1);
        tc::mbar_init(&sh.bar[1], 1);
        tc::fence_mbar_init();
    }
    cluster.barrier_arrive();  // (awaited before the first write to another CTA)
    // the nodes' tokens and numbers, a thread each
    const int mine = tid - (kThreads - kMaxNodes);
    int token = -1;
    float number = 0.f;
    if (mine > 0 && mine < root.nodes) {
        token = p.tokens[root.row0 + mine];
        number = p.u[root.row0 + mine];
    }
    const Links links = load_links(p.parent, root);
    const Tree t = read_tree(sh.tree, root, links, false) ? root : Tree{0, -1};
    if (t.nodes < 0 && writer) report_invalid(p.status);
    if (tid < t.nodes) {
        unsigned long long mask = 0;
        for (int j = tid + 1; j < t.nodes; ++j) mask |= (unsigned long long)(sh.tree.parent[j] == tid) << j;
        sh.child[tid] = mask;
    }
    float logit = 0.f, qt = 1.f;
    if (mine > 0 && mine < t.nodes) {
        if (token < 0 || token >= p.V) token = -1;
        if (token >= 0) {
            const size_t from = (size_t)(t.row0 + sh.tree.parent[mine]) * p.V + token;
            logit = to_f32(reinterpret_cast<const Tin *>(p.logits)[from]);
            if (p.probs) qt = p.probs[from];
        }
    }
    cluster.barrier_wait();
    int len = 0, next = -1;
    Exchange ex;
    ex.size = size;
    ex.rank = rank;
    int owner = -1;  // the CTA that finds the next token in its part of the row; none: `next` is it
    const float *q = nullptr;
    float C = 0.f;
    int removed = 0;
    unsigned long long at = 0;
    bool plain = false;       // the row has neither NaN nor +inf
    bool runs_known = false;  // sh.part holds the sums of the runs of r
    if (t.nodes > 0) {
        const float temp = p.temperature ? p.temperature[n] : 1.f;
        r.onehot = !(temp > 0.f);
        r.scale = r.onehot ? 0.f : 1.4426950408889634f / fmaxf(temp, 1e-30f);
        int node = 0;
        for (;;) {
            if (p.silent && rank == size - 1) {
                ex.ok = false;
                break;
            }
            if (tid == 0) sh.path[len] = node;  // (written out at the end: an exchange would wait for the store)
            ++len;
            if (node > 0) {
                place(t.row0 + node);
                part.fetch();
            }
            q = p.probs ? p.probs + (size_t)(t.row0 + node) * p.V : nullptr;
            C = 0.f;
            removed = 0;
            tc::cp_async_wait_all();
            if (len == 1 && mine > 0 && mine < t.nodes) {  // the gathered values have come with the first row
                sh.token[mine] = token;
                sh.u[mine] = number;
                sh.logit[mine] = logit;
                sh.q[mine] = qt;
            }
            __syncthreads();
            const unsigned long long children = sh.child[node];
            const int trials = __popcll(children), first = __ffsll((long long)children) - 1;
            if (trials) part.ask(part.row + (ptrdiff_t)(first - node) * p.V);
            Found f{-INFINITY, -1, 0.f, 0.f};
            for (int v = part.v0 + tid; v < part.v1; v += kThreads) {
                if (r.onehot) {
                    float l[P::kVec];
                    part.get(v, l);
#pragma unroll
                    for (int e = 0; e < P::kVec; ++e)
                        if (l[e] > f.top) f = Found{l[e], v * P::kVec - part.lead + e, 0.f, 0.f};
                } else {
                    f.top = fmaxf(f.top, part.top(v));
                }
            }
            if (!r.onehot) {
                if (f.top > -INFINITY) f.best = 0;  // only `onehot` uses the place
                f.top = best_of_warp(f.top, 0).top;
                if (trials && f.top == -INFINITY) {
                    // nothing to add up, but a NaN among these logits has to show in the row's sum
                    for (int v = part.v0 + tid; v < part.v1; v += kThreads) {
                        float l[P::kVec];
                        part.get(v, l);
#pragma unroll
                        for (int e = 0; e < P::kVec; ++e)
                            if (l[e] != l[e]) f.sum = l[e];
                    }
                } else if (trials) {
                    float2 sum = make_float2(0.f, 0.f);
                    const Row warps{f.top, r.scale, 0, false, false};
#pragma unroll 2
                    for (int v = part.v0 + tid; v < part.v1; v += kThreads) {
                        float l[P::kVec];
                        part.get(v, l);
#pragma unroll
                        for (int e = 0; e < P::kVec; e += 2)
                            sum = tc::add2(sum, weights_of(warps, true, make_float2(l[e], l[e + 1])));
                    }
                    f.sum = sum.x + sum.y;
                }
            }
            f = cluster_max(sh, ex, p.wait_ns, r.scale, f);
            r.top = f.top;
            r.best = f.best;
            r.flat = f.top == INFINITY;
            plain = trials && f.sum < INFINITY;
            if (r.best < 0 || !ex.ok) break;  // no weight anywhere
            if (trials && !r.onehot && sh.token[first] >= 0) {
                const float w = exp2f(__fmul_rn(__fsub_rn(sh.logit[first], r.top), r.scale));
                if (sh.u[first] * sh.q[first] * f.sum < w * (1.f - kMargin)) {  // never where the sum is NaN
                    node = first;
                    __syncthreads();  // the row's part is free
                    continue;
                }
            }
            // The exact sum of r over the CTA's part, its runs' sums kept in sh.part; batches of kBatch vectors, so
            // that as many reads of q are under way at once.
            auto exact = [&](bool with_q) {
                unsigned long long sum = 0;
                for (int v = part.v0 + warp * 32; v < part.v1; v += kBatch * kThreads) {
                    float x[kBatch][P::kVec];
                    if (with_q) {
#pragma unroll
                        for (int i = 0; i < kBatch; ++i)
                            if (v + i * kThreads + lane < part.v1) part.get_q(q, v + i * kThreads + lane, x[i]);
                    }
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int at = v + i * kThreads;
                        FixedSum f;
                        if (at + lane < part.v1) {
                            float l[P::kVec];
                            part.get(at + lane, l);
#pragma unroll
                            for (int e = 0; e < P::kVec; e += 2) {
                                float2 w = weights_of(r, plain, make_float2(l[e], l[e + 1]));
                                if (with_q) w = excesses_of(w, C, make_float2(x[i][e], x[i][e + 1]));
                                f.add2(w);
                            }
                        }
                        if (at < part.v1) {
                            const unsigned long long run = f.of_warp();
                            sum += run;
                            if (lane == 0 && part.kept) sh.part[(at - part.v0) >> 5] = run;
                        }
                    }
                }
                return sum;
            };
            unsigned long long Z = 1ull << 40;
            if (!r.onehot) {
                if (q && trials) part.ask_q(q);
                Z = cluster_sum(sh, ex, p.wait_ns, exact(false), sh.sum_w);
            }
            if (!ex.ok) break;
            unsigned long long s = Z, *sums = sh.sum_w;
            runs_known = part.kept != nullptr;
            int accepted = -1;
            unsigned long long untried = children;
            while (untried && accepted < 0) {
                const int c = __ffsll((long long)untried) - 1;
                untried &= untried - 1;
                const int token = sh.token[c];
                if (token < 0) {
                    if (writer) report_invalid(p.status);
                    continue;
                }
                const float w = r.onehot ? (token == r.best ? 1.f : 0.f)
                                : r.flat ? weight_of(r, sh.logit[c])
                                         : fmaxf(exp2f(__fmul_rn(__fsub_rn(sh.logit[c], r.top), r.scale)), 0.f);
                const float sf = __ull2float_rn(s) * (1.f / kFixed), qc = sh.q[c];
                float rest = w;
                if (q && C > 0.f) rest = excess_of(w, C, qc);
                for (int i = 0; i < removed; ++i) rest = sh.removed[i] == token ? 0.f : rest;
                if (__fmul_rn(__fmul_rn(sh.u[c], qc), sf) < rest) {
                    accepted = c;
                } else if (!q) {
                    const unsigned long long cut = fixed40(rest);
                    s -= cut;
                    __syncthreads();
                    if (tid == 0) {
                        sh.removed[removed] = token;
                        sh.removed_w[removed] = cut;
                    }
                    ++removed;
                    __syncthreads();
                } else {
                    C = __fadd_rn(C, sf);
                    if (r.onehot) {
                        s = fixed40(excess_of(1.f, C, q[r.best]));
                    } else {
                        s = cluster_sum(sh, ex, p.wait_ns, exact(true), sh.sum_r);
                        sums = sh.sum_r;
                        if (!ex.ok) break;
                    }
                }
            }
            if (!ex.ok) break;
            if (accepted >= 0) {
                node = accepted;
                __syncthreads();  // the row's part is free
                continue;
            }
            if (s == 0) {  // nothing is left of the target: its own distribution
                s = Z;
                C = 0.f;
                removed = 0;
                runs_known &= sums == sh.sum_w;
                sums = sh.sum_w;
            }
            if (r.onehot) {  // all that is left is at one place, unless that was removed
                next = r.best;
                break;
            }
            // the next token: the first one whose cumulative sum is above u s
            const double un = (double)p.u_next[n];
            at = un > 0.0 ? (unsigned long long)(un * (double)s) : 0ull;
            if (at >= s) at = s - 1;
            __syncthreads();  // sums[] is written
            for (owner = 0; owner < size - 1; ++owner) {
                unsigned long long here = sums[owner];
                const int first = owner * each * P::kVec - part.lead, end = first + each * P::kVec;
                for (int i = 0; i < removed; ++i)
                    if (sh.removed[i] >= first && sh.removed[i] < end) here -= sh.removed_w[i];
                if (at < here) break;
                at -= here;
            }
            break;
        }
    }
    if (owner == rank) {
        auto rest = [&](int v, float (&x)[P::kVec]) {
            float l[P::kVec];
            part.get(v, l);
            if (q && C > 0.f) {
                float y[P::kVec];
                part.get_q(q, v, y);
#pragma unroll
                for (int e = 0; e < P::kVec; ++e) x[e] = excess_of(weight_of(r, l[e]), C, y[e]);
            } else {
#pragma unroll
                for (int e = 0; e < P::kVec; ++e) {
                    x[e] = weight_of(r, l[e]);
                    for (int i = 0; i < removed; ++i)
                        if (sh.removed[i] == v * P::kVec - part.lead + e) x[e] = 0.f;
                }
            }
        };
        // The run, the vector and the logit that pass `at`.  A part that is not kept is searched kRuns runs at a time.
        for (int v0 = part.v0; v0 < part.v1; v0 += kRuns * 32) {
            if (!runs_known) {
                __syncthreads();
                for (int run = warp; run < kRuns; run += kWarps) {
                    const int v = v0 + run * 32 + lane;
                    FixedSum sum;
                    if (v < part.v1) {
                        float x[P::kVec];
                        rest(v, x);
#pragma unroll
                        for (int e = 0; e < P::kVec; e += 2) sum.add2(make_float2(x[e], x[e + 1]));
                    }
                    const unsigned long long total = sum.of_warp();
                    if (lane == 0) sh.part[run] = total;
                }
                __syncthreads();
            } else if (removed) {
                if (tid == 0)
                    for (int i = 0; i < removed; ++i) {
                        const int v = (sh.removed[i] + part.lead) / P::kVec;
                        if (v >= part.v0 && v < part.v1) sh.part[(v - part.v0) >> 5] -= sh.removed_w[i];
                    }
                __syncthreads();
            }
            // every warp finds the run (kRuns / 32 entries a lane), the first goes on to the logit
            constexpr int kEach = kRuns / 32;
            unsigned long long own[kEach], sum = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int run = lane * kEach + i;
                own[i] = v0 + run * 32 < part.v1 ? sh.part[run] : 0ull;
                sum += own[i];
            }
            unsigned long long upto = scan(sum);
            const uint32_t here = __ballot_sync(0xffffffffu, at < upto);
            if (!here) {
                at -= __shfl_sync(0xffffffffu, upto, 31);
                continue;
            }
            const int who = __ffs((int)here) - 1;
            int run = lane * kEach;
            unsigned long long left = at - (upto - sum);
#pragma unroll
            for (int i = 0; i < kEach - 1; ++i)
                if (run == lane * kEach + i && left >= own[i]) {
                    left -= own[i];
                    ++run;
                }
            run = __shfl_sync(0xffffffffu, run, who);
            left = __shfl_sync(0xffffffffu, left, who);
            if (warp == 0) {
                const int v = v0 + run * 32 + lane;
                float x[P::kVec];
                FixedSum f;
                if (v < part.v1) {
                    rest(v, x);
#pragma unroll
                    for (int e = 0; e < P::kVec; e += 2) f.add2(make_float2(x[e], x[e + 1]));
                }
                upto = scan(f.mine());
                if (left < upto && left >= upto - f.mine()) {
                    left -= upto - f.mine();
                    int found = 0;
                    bool passed = false;
#pragma unroll
                    for (int e = 0; e < P::kVec; ++e) {
                        const unsigned long long w = fixed40(x[e]);
                        if (!passed && left < w) {
                            passed = true;
                            found = e;
                        }
                        left -= passed ? 0ull : w;
                    }
                    p.next_token[n] = v * P::kVec - part.lead + found;
                }
            }
            break;
        }
    } else if (writer && owner < 0) {
        p.next_token[n] = next;
    }
    // (Let in at the start, the next kernel's clusters would take the places of the first walks to end and lie uneven
    // over the SMs: 64 requests over 131072 tokens 48.4, 56.5 and 45.5 us on three draws, here 48.0, 52.7 and 44.8.)
    tc::grid_dep_launch();
    if (!ex.ok) {  // an exchange that never came: an empty path
        len = 0;
        if (tid == 0 && p.status) atomicCAS(p.status, 0, (int32_t)KDA_ERR_TIMEOUT);
    }
    tc::cp_async_wait_all();  // (a root's row that was fetched for a tree that is not one)
    __syncthreads();
    if (!ex.ok) {
        // A CTA that was only late may still send to this one, whose shared memory has to be there: it stays until the
        // others have left or come here too.  (Each of their waits has its limit.)
        cluster.barrier_arrive();
        cluster.barrier_wait();
    }
    for (int i = tid; i < p.path_stride && rank == 0; i += kThreads)
        p.path[(size_t)n * p.path_stride + i] = i < len ? sh.path[i] : -1;
    if (writer) p.path_len[n] = len;
    // (else every CTA has all values of the last exchange: none writes to another's shared memory any more)
}

template <typename Tin>
cudaError_t launch_t(Args p, int num_seqs, cudaStream_t st) {
    constexpr int kVec = 16 / sizeof(Tin);
    // CTAs per request: a row is split as long as a part has two vectors per thread (64 requests over 131072 tokens:
    // 189, 109, 48 and 59 us with 2, 4, 8 and 16); half as many once each SM has a request, where they would only
    // queue (256 requests over 100003 tokens: 127, 61, 69 and 115 us), if a part can then still be kept.
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    int size = 1;
    while (size < kMaxCluster && p.V >= 2 * size * kThreads * kVec) size *= 2;
    const int vectors = (p.V + 2 * (kVec - 1)) / kVec;
    if (size == kMaxCluster && num_seqs >= sms && (uint32_t)(vectors + size / 2 - 1) / (size / 2) * 16 <= kMaxPart) size /= 2;
    const int each = (vectors + size - 1) / size;
    p.part_bytes = (uint32_t)each * 16 <= kMaxPart ? (uint32_t)each * 16 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)num_seqs * size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = p.part_bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    e = allow_smem<draft_verify_kernel<Tin>>(kMaxPart);
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, draft_verify_kernel<Tin>, (const Args)p);
}

}  // namespace

cudaError_t launch_draft_verify(const DraftVerifyArgs &a, kda_dtype dt, cudaStream_t st) {
    const long long wait_ns = testing_wait_ns();
    const Args p{a.logits, a.probs, a.tokens, a.parent, a.cu, a.temperature, a.u, a.u_next, a.total_nodes, a.V,
                 a.path_stride, 0, wait_ns > 0 ? (uint64_t)wait_ns : kWaitNs, testing_fault() == kFaultNoPublish, a.path,
                 a.path_len, a.next_token, a.status};
    return dt == KDA_BF16 ? launch_t<__nv_bfloat16>(p, a.num_seqs, st) : launch_t<float>(p, a.num_seqs, st);
}

}  // namespace kda
