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
#include <type_traits>

#include "kda_tc.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace {

// ---------------------------------------------------------------------------
// Step, fp32 on the CUDA cores: any supported d and type
// ---------------------------------------------------------------------------
// One CTA of NT threads per (request, head).  With K~ = k e^b, Q~ = q e^b, K^ = k e^{-b} in shared memory, A and P
// are one dot product per (node, ancestor) and thread; the products with the state go in register tiles of TN nodes
// by four columns, which read a vector of shared memory for every eight multiply-adds or more; the substitution has
// a thread per column, eight nodes at a time.  Where the decays along a path sum to more than kMaxRange, so that
// e^{-b} would overflow, A and P take the path's own exponents instead.
// Bound by the multiply-adds with the state, 4 d^2 for each node, and their operands' way from shared memory; with few
// requests by the latency of its dependent steps (17 requests of up to 13 nodes, 5 heads of d = 64, fp32: 6.8 us, of
// which the states' way from HBM is 0.2).
constexpr float kMaxRange = 80.f;

template <int D>
struct StepLayout {  // offsets in floats; R: rows, max_nodes rounded up to eight
    static constexpr int kPitch = D + 4;  // rows of K~, Q~, K^ start on distinct banks
    int R, ap_stride, ke, qe, ki, gb, A, P, beta, scale, S, total;
    __host__ __device__ explicit StepLayout(int max_nodes) {
        R = (max_nodes + 7) & ~7;
        ap_stride = R + 4;
        ke = 0;
        qe = ke + R * kPitch;
        ki = qe + R * kPitch;   // K^, then r [R][D]
        gb = ki + R * kPitch;   // g, then b, then y [R][D]
        A = gb + R * D;
        P = A + R * ap_stride;
        beta = P + R * ap_stride;
        scale = beta + R;
        S = scale + 2 * R;
        total = S + D * D;
    }
    // the state is read through L1 where it would not fit beside the rest
    __host__ __device__ bool keeps_state() const { return total * 4 <= 225 * 1024; }
    __host__ __device__ int bytes() const { return (keeps_state() ? total : S) * 4; }
};

// N neighbouring values of a row, read and written at once.
template <typename T, int N>
struct __align__(N * sizeof(T)) Some {
    T v[N];
};
template <int N, typename T>
__device__ __forceinline__ Some<T, N> load_some(const T *p, bool in) {
    Some<T, N> x;
    if (in) {
        x = *reinterpret_cast<const Some<T, N> *>(p);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) x.v[e] = from_f32<T>(0.f);
    }
    return x;
}

template <int N, typename T>
__device__ __forceinline__ void load_floats(const T *p, bool in, float (&f)[N]) {
    const Some<T, N> x = load_some<N>(p, in);
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = to_f32(x.v[e]);
}

// Adds up[r] * M[row + r][a] * u[a][c] over a < end (a multiple of four) for ROWS rows; M's rows and u lie in shared
// memory.  Masked: entries off the path are skipped instead of multiplied by zero, which a non-finite u of another
// branch would turn into NaN.
template <int D, int ROWS, bool Masked>
__device__ __forceinline__ void add_rows(float (&acc)[ROWS], float sign, const float *M, int stride, const float *u, int end,
                                         const unsigned long long *anc, int row, int nodes) {
    for (int a = 0; a < end; a += 4) {
        float ua[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) ua[e] = sign * u[(a + e) * D];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const float4 m = *reinterpret_cast<const float4 *>(&M[(row + r) * stride + a]);
            const float mv[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!Masked || (row + r < nodes && ((anc[row + r] >> (a + e)) & 1))) acc[r] = fmaf(mv[e], ua[e], acc[r]);
        }
    }
}

// u and o from r and y (all threads).  Forward substitution over blocks of eight nodes: the products with the u of
// earlier blocks are shared out, D threads by NT / D groups of rows, then a thread per column solves the block's own
// triangle.  o follows from all of u at once.  Returns false if a u is not finite (to every thread).
template <int D, int NT, bool Masked>
__device__ __forceinline__ bool substitute(float *sm, const StepLayout<D> &L, const TreeShared &ts, int M) {
    constexpr int RG = NT / D, ROWS = 8 / RG;
    const float *sA = sm + L.A, *sP = sm + L.P;
    const int c = threadIdx.x % D, first = threadIdx.x / D * ROWS;
    const float *s_r = sm + L.ki + c, *s_y = sm + L.gb + c;
    float *s_u = sm + L.ke + c, *s_o = sm + L.qe + c;
    bool finite = true;
    for (int i0 = 0; i0 < M; i0 += 8) {
        float w[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int i = i0 + first + r;
            w[r] = i < M ? s_r[i * D] : 0.f;
        }
        add_rows<D, ROWS, Masked>(w, -1.f, sA, L.ap_stride, s_u, i0, ts.anc, i0 + first, M);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) s_u[(i0 + first + r) * D] = w[r];
        if (RG > 1) __syncthreads();
        if (first == 0) {
            float t[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                t[r] = s_u[(i0 + r) * D];
#pragma unroll
                for (int a = 0; a < r; ++a)
                    if (!Masked || (i0 + r < M && ((ts.anc[i0 + r] >> (i0 + a)) & 1)))
                        t[r] = fmaf(-sA[(i0 + r) * L.ap_stride + i0 + a], t[a], t[r]);
                finite &= i0 + r >= M || fabsf(t[r]) < INFINITY;
                s_u[(i0 + r) * D] = t[r];
            }
        }
        if (RG > 1) __syncthreads();
    }
    for (int i0 = 0; i0 < M; i0 += 8) {
        float out[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) out[r] = i0 + first + r < M ? s_y[(i0 + first + r) * D] : 0.f;
        add_rows<D, ROWS, Masked>(out, 1.f, sP, L.ap_stride, s_u, i0 + 8, ts.anc, i0 + first, M);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) s_o[(i0 + first + r) * D] = out[r];
    }
    return __syncthreads_and(finite);
}

template <typename Tin, int D, int NT>
__global__ void __launch_bounds__(NT)
tree_step_kernel(const Tin *__restrict__ q, const Tin *__restrict__ k, const Tin *__restrict__ v,
                 const float *__restrict__ g, const float *__restrict__ beta, const int32_t *__restrict__ parent,
                 const int32_t *__restrict__ cu, const int32_t *__restrict__ seq_idx, int H, int total_nodes,
                 int max_nodes, int num_slots, const float *__restrict__ S_pool, Tin *__restrict__ o,
                 float *__restrict__ u, int32_t *__restrict__ status, int qk_norm, float qk_eps,
                 const Tin *__restrict__ gate, const float *__restrict__ weight, float out_eps) {
    constexpr int kWarps = NT / 32, CG = D / 4, NG = NT / CG, kTile = D == 128 ? 4 : 2;  // products: column groups, node groups
    constexpr int CPL = D < 32 ? 1 : D / 32, LANES = D / CPL;                 // rows: channels per lane
    constexpr int kPitch = StepLayout<D>::kPitch;
    extern __shared__ __align__(16) float sm[];
    __shared__ TreeShared ts;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const StepLayout<D> L(max_nodes);
    const int n = blockIdx.x / H, h = blockIdx.x % H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Tree t = tree_rows(cu, n, total_nodes, max_nodes);
    const int slot = slot_of(seq_idx, n, num_slots);
    if (t.nodes < 0 || slot < 0) {
        if (tid == 0) report_invalid(status);
        return;
    }
    if (t.nodes == 0) return;
    const Links links = load_links(parent, t);
    const int M = t.nodes;
    const size_t row_stride = (size_t)H * D, base = ((size_t)t.row0 * H + h) * D;
    const float *S = S_pool + ((size_t)slot * H + h) * D * D;
    for (int i = tid; i < M * CG; i += NT)
        tc::cp_async16(sm + L.gb + i * 4, g + base + (size_t)(i / CG) * row_stride + i % CG * 4);
    tc::cp_async_commit();
    if (L.keeps_state()) {
        for (int i = tid; i < D * CG; i += NT) tc::cp_async16(sm + L.S + i * 4, S + i * 4);
        S = sm + L.S;
    }
    tc::cp_async_commit();
    // a thread's rows of k and q for the first 16 nodes
    constexpr int kPer = 16 / kWarps;
    const int c0 = lane * CPL;
    Some<Tin, CPL> kr[kPer], qr[kPer];
    auto fetch = [&](int first) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = first + warp + e * kWarps;
            const size_t at = base + (size_t)i * row_stride + c0;
            kr[e] = load_some<CPL>(k + at, i < M && lane < LANES);
            qr[e] = load_some<CPL>(q + at, i < M && lane < LANES);
        }
    };
    fetch(0);
    for (int i = tid; i < M; i += NT) sm[L.beta + i] = beta[(size_t)(t.row0 + i) * H + h];
    tc::cp_async_wait<1>();
    if (!read_tree(ts, t, links, true)) {  // a block barrier
        tc::cp_async_wait_all();
        if (tid == 0) report_invalid(status);
        return;
    }

    // K~, Q~, K^, a warp per node.  b sums g over the path, 16 nodes at a time, from the b of the nearest ancestor
    // in an earlier group.
    float range = 0.f;
    for (int first = 0; first < M; first += 16) {
        float b[kPer][CPL];
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = first + warp + e * kWarps;
#pragma unroll
            for (int x = 0; x < CPL; ++x) b[e][x] = 0.f;
            if (i < M && lane < LANES) {
                const unsigned long long anc = ts.anc[i], before = anc & ((1ull << first) - 1);
                uint32_t here = (uint32_t)(anc >> first) & 0xffffu;
                if (before) {
                    const float *from = sm + L.gb + (63 - __clzll((long long)before)) * D + c0;
#pragma unroll
                    for (int x = 0; x < CPL; ++x) b[e][x] = from[x];
                }
                while (here) {
                    const float *from = sm + L.gb + (first + __ffs((int)here) - 1) * D + c0;
                    here &= here - 1;
#pragma unroll
                    for (int x = 0; x < CPL; ++x) b[e][x] += log_decay(from[x]);
                }
            }
        }
        __syncthreads();  // every sum of this group is formed
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = first + warp + e * kWarps;
            if (i >= M) break;
            float kf[CPL], qf[CPL];
#pragma unroll
            for (int x = 0; x < CPL; ++x) {
                kf[x] = to_f32(kr[e].v[x]);
                qf[x] = to_f32(qr[e].v[x]);
            }
            float sk = 1.f, sq = 1.f;
            if (qk_norm) {
                sk = sq = 0.f;
#pragma unroll
                for (int x = 0; x < CPL; ++x) {
                    sk = fmaf(kf[x], kf[x], sk);
                    sq = fmaf(qf[x], qf[x], sq);
                }
#pragma unroll
                for (int off = 16; off; off >>= 1) {
                    sk += __shfl_xor_sync(0xffffffffu, sk, off);
                    sq += __shfl_xor_sync(0xffffffffu, sq, off);
                }
                sk = rsqrtf(sk + qk_eps);
                sq = rsqrtf(sq + qk_eps);
                if (lane == 0) {
                    sm[L.scale + i] = sk;
                    sm[L.scale + L.R + i] = sq;
                }
            }
            if (lane < LANES) {
#pragma unroll
                for (int x = 0; x < CPL; ++x) {
                    const float up = expf(b[e][x]), key = kf[x] * sk;
                    range = fmaxf(range, fabsf(b[e][x]));
                    sm[L.gb + i * D + c0 + x] = b[e][x];
                    sm[L.ke + i * kPitch + c0 + x] = key * up;
                    sm[L.qe + i * kPitch + c0 + x] = qf[x] * sq * up;
                    sm[L.ki + i * kPitch + c0 + x] = key * expf(-b[e][x]);
                }
            }
        }
        if (first + 16 < M) {
            fetch(first + 16);
            __syncthreads();
        }
    }
    tc::cp_async_wait_all();
    const bool pairwise = __syncthreads_or(!(range <= kMaxRange));

    // A and P: a thread per (node, ancestor), with zeros up to a multiple of eight
    const int M8 = (M + 7) & ~7;
    for (int p = tid; p < M8 * M8; p += NT) {
        const int i = p / M8, a = p % M8;
        float sa = 0.f, sp = 0.f;
        if (!pairwise && i < M && ((ts.anc[i] >> a) & 1)) {
            const float *x = sm + L.ke + i * kPitch, *y = sm + L.qe + i * kPitch, *z = sm + L.ki + a * kPitch;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                const float4 x4 = *reinterpret_cast<const float4 *>(x + c), y4 = *reinterpret_cast<const float4 *>(y + c),
                             z4 = *reinterpret_cast<const float4 *>(z + c);
                sa = fmaf(x4.x, z4.x, sa); sa = fmaf(x4.y, z4.y, sa); sa = fmaf(x4.z, z4.z, sa); sa = fmaf(x4.w, z4.w, sa);
                sp = fmaf(y4.x, z4.x, sp); sp = fmaf(y4.y, z4.y, sp); sp = fmaf(y4.z, z4.z, sp); sp = fmaf(y4.w, z4.w, sp);
            }
            sa = a == i ? 0.f : sa * sm[L.beta + i];
        }
        sm[L.A + i * L.ap_stride + a] = sa;
        sm[L.P + i * L.ap_stride + a] = sp;
    }
    if (pairwise) {  // a warp per node
        __syncthreads();  // the zeros lie
        for (int i = warp; i < M; i += kWarps) {
            const size_t own = base + (size_t)i * row_stride + c0;
            float ki[CPL], qi[CPL];
            load_floats(k + own, lane < LANES, ki);
            load_floats(q + own, lane < LANES, qi);
            pairs_of_node<4>(ts, i, ki, qi,
                             [&](int a, float (&ka)[CPL], float (&ga)[CPL]) {
                                 const size_t at = base + (size_t)a * row_stride + c0;
                                 load_floats(k + at, lane < LANES, ka);
                                 load_floats(g + at, lane < LANES, ga);
   #pragma unroll
                                 for (int e = 0; e < CPL; ++e) ga[e] = log_decay(ga[e]);
                             },
                             [](float x) { return expf(x); },
                             [&](int a, float x, bool is_p) {
                                 if (qk_norm) x *= sm[L.scale + (is_p ? L.R : 0) + i] * sm[L.scale + a];
                                 if (!is_p) x = a == i ? 0.f : x * sm[L.beta + i];
                                 sm[(is_p ? L.P : L.A) + i * L.ap_stride + a] = x;
                             });
        }
    }
    __syncthreads();  // K^ and b are no longer needed

    // r and y, TN nodes by four columns a thread; v is asked for before the sums
    const int cg = tid % CG, ng = tid / CG;
    auto products = [&](auto tile) {
        constexpr int TN = decltype(tile)::value;
        for (int i0 = ng * TN; i0 < M; i0 += NG * TN) {
            Some<Tin, 4> vr[TN];
#pragma unroll
            for (int r = 0; r < TN; ++r) vr[r] = load_some<4>(v + base + (size_t)(i0 + r) * row_stride + cg * 4, i0 + r < M);
            float x[TN][4], y[TN][4];
#pragma unroll
            for (int r = 0; r < TN; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[r][e] = y[r][e] = 0.f;
            const float *ke[TN], *qe[TN];
#pragma unroll
            for (int r = 0; r < TN; ++r) {
                ke[r] = sm + L.ke + min(i0 + r, M - 1) * kPitch;
                qe[r] = sm + L.qe + min(i0 + r, M - 1) * kPitch;
            }
#pragma unroll 2
            for (int c = 0; c < D; c += 4) {
                float4 s[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] = *reinterpret_cast<const float4 *>(S + (size_t)(c + j) * D + cg * 4);
#pragma unroll
                for (int r = 0; r < TN; ++r) {
                    const float4 kk = *reinterpret_cast<const float4 *>(ke[r] + c), qq = *reinterpret_cast<const float4 *>(qe[r] + c);
                    const float kv[4] = {kk.x, kk.y, kk.z, kk.w}, qv[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[r][0] = fmaf(kv[j], s[j].x, x[r][0]); x[r][1] = fmaf(kv[j], s[j].y, x[r][1]);
                        x[r][2] = fmaf(kv[j], s[j].z, x[r][2]); x[r][3] = fmaf(kv[j], s[j].w, x[r][3]);
                        y[r][0] = fmaf(qv[j], s[j].x, y[r][0]); y[r][1] = fmaf(qv[j], s[j].y, y[r][1]);
                        y[r][2] = fmaf(qv[j], s[j].z, y[r][2]); y[r][3] = fmaf(qv[j], s[j].w, y[r][3]);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < TN; ++r) {
                if (i0 + r < M) {
                    const float w = sm[L.beta + i0 + r];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[r][e] = w * (to_f32(vr[r].v[e]) - x[r][e]);
                    *reinterpret_cast<float4 *>(sm + L.ki + (i0 + r) * D + cg * 4) = make_float4(x[r][0], x[r][1], x[r][2], x[r][3]);
                    *reinterpret_cast<float4 *>(sm + L.gb + (i0 + r) * D + cg * 4) = make_float4(y[r][0], y[r][1], y[r][2], y[r][3]);
                }
            }
        }
    };
    // few nodes: every thread group gets some (256 requests x 32 heads of d = 128, fp32, 3-6 nodes: 284 us for 328)
    if (M <= NG * kTile / 2) products(std::integral_constant<int, kTile / 2>{});
    else products(std::integral_constant<int, kTile>{});
    // the gate's rows for the first 16 nodes and its weight, asked for ahead
    Some<Tin, CPL> zr[kPer];
    float wt[CPL];
    auto fetch_gate = [&](int first) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = first + warp + e * kWarps;
            zr[e] = load_some<CPL>(gate + base + (size_t)i * row_stride + c0, gate && i < M && lane < LANES);
        }
    };
    fetch_gate(0);
#pragma unroll
    for (int a = 0; a < CPL; ++a) wt[a] = gate && weight && lane < LANES ? weight[c0 + a] : 1.f;
    __syncthreads();  // K~ and Q~ are no longer needed: u and o take their place
    if (!substitute<D, NT, false>(sm, L, ts, M)) substitute<D, NT, true>(sm, L, ts, M);
    for (int first = 0; first < M; first += 16) {  // a warp per row
        float x[kPer][CPL], inv[kPer];
        if (first > 0) fetch_gate(first);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = first + warp + e * kWarps;
            inv[e] = 0.f;
#pragma unroll
            for (int a = 0; a < CPL; ++a) {
                x[e][a] = i < M && lane < LANES ? sm[L.qe + i * D + c0 + a] : 0.f;
                inv[e] = fmaf(x[e][a], x[e][a], inv[e]);
            }
        }
        if (gate) {
#pragma unroll
            for (int off = 16; off; off >>= 1)
#pragma unroll
                for (int e = 0; e < kPer; ++e) inv[e] += __shfl_xor_sync(0xffffffffu, inv[e], off);
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = first + warp + e * kWarps;
            if (i >= M || lane >= LANES) continue;
            const size_t at = base + (size_t)i * row_stride + c0;
            const float scale = rsqrtf(inv[e] / (float)D + out_eps);
            Some<Tin, CPL> out;
            Some<float, CPL> ui;
#pragma unroll
            for (int a = 0; a < CPL; ++a) {
                out.v[a] = from_f32<Tin>(gate ? x[e][a] * scale * wt[a] * sigmoidf(to_f32(zr[e].v[a])) : x[e][a]);
                ui.v[a] = sm[L.ke + i * D + c0 + a];
            }
            *reinterpret_cast<Some<Tin, CPL> *>(o + at) = out;
            if (u) *reinterpret_cast<Some<float, CPL> *>(u + at) = ui;
        }
    }
}

template <typename Tin, int D, int NT>
cudaError_t launch_step_n(const TreeStepArgs &a, cudaStream_t st) {
    const int smem = StepLayout<D>(a.max_nodes).bytes();
    const cudaError_t e = allow_smem<tree_step_kernel<Tin, D, NT>>(smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(tree_step_kernel<Tin, D, NT>, a.num_seqs * a.H, NT, smem, st, (const Tin *)a.q,
                            (const Tin *)a.k, (const Tin *)a.v, a.g, a.beta, a.parent, a.cu, a.seq_idx, a.H,
                            a.total_nodes, a.max_nodes, a.num_slots, a.S_pool, (Tin *)a.o, a.u, a.status, a.fu.qk_norm,
                            a.fu.qk_eps, (const Tin *)a.fu.gate, a.fu.weight, a.fu.out_eps);
}

// 256 threads where shared memory leaves room for few CTAs on an SM (d = 128: 137 us with 128 and 123 with 256, 64
// requests x 9-16 nodes x 32 heads, fp32; d = 64, bf16: 124 and 91, 16 requests x 33-64 nodes), or where there are few
// CTAs (8, of 8 nodes: 6.5 and 5.6); else 128, whose barriers stop fewer warps (256 requests x 9-16 nodes, d = 64: 150 and
// 169).
template <typename Tin, int D>
cudaError_t launch_step_d(const TreeStepArgs &a, cudaStream_t st) {
    if constexpr (D == 128) {
        return launch_step_n<Tin, D, 256>(a, st);
    } else if constexpr (D == 64) {
        int sms = 0;
        const cudaError_t e = sm_count(&sms);
        if (e != cudaSuccess) return e;
        return a.max_nodes > 16 || a.num_seqs * a.H <= 2 * sms ? launch_step_n<Tin, D, 256>(a, st)
                                                               : launch_step_n<Tin, D, 128>(a, st);
    } else {
        return launch_step_n<Tin, D, 128>(a, st);
    }
}

template <typename Tin>
cudaError_t launch_step_t(const TreeStepArgs &a, cudaStream_t st) {
    switch (a.d) {
        case 16: return launch_step_d<Tin, 16>(a, st);
        case 64: return launch_step_d<Tin, 64>(a, st);
        case 128:
            if constexpr (sizeof(Tin) == 4) return launch_step_d<Tin, 128>(a, st);
            // (256 requests x 32 heads: 3-6 nodes 99 us with the state in registers, 241 with tcgen05; 9-16 nodes 163
            // and 273; with a variant of the former for 32 nodes, 64 requests of 20-32 took 138 and 98)
            else return a.max_nodes <= 16 ? launch_tree_step_mma(a, st) : launch_tree_step_tc(a, st);
        default: return cudaErrorInvalidValue;
    }
}

// ---------------------------------------------------------------------------
// Commit
// ---------------------------------------------------------------------------
// One CTA per (request, head), laid out like the decode step: each thread holds 16 rows by four columns of the
// state in registers.  The state's loads are issued before anything else that takes time, and the path's rows of
// k, g and u follow as asynchronous copies, so one wait covers both.  The path is taken CHUNK nodes at a time (8, or 16
// where paths may be longer than 8, which would otherwise wait for their rows twice):
// with the decay to the chunk's end folded into its keys, a chunk is  S <- e^{b} S + sum_a (k_a e^{b - b_a}) u_a^T.
// Bound by HBM: the state once each way.  Measured, 256 requests x 32 heads of d = 128, bf16, paths of 0 to 6 nodes:
// 148 us, DRAM busy 78% of the time; 24 warps an SM wait for loads in flight most of theirs.
constexpr int kRows = 16;

template <typename Tin, int D, int CHUNK>
__global__ void __launch_bounds__((D / 4) * (D / kRows), D == 128 ? 3 : 1)
tree_commit_kernel(const Tin *__restrict__ k, const float *__restrict__ g, const float *__restrict__ u,
                   const int32_t *__restrict__ cu, const int32_t *__restrict__ path,
                   const int32_t *__restrict__ path_len, const int32_t *__restrict__ seq_idx, int H, int total_nodes,
                   int path_stride, int num_slots, float *__restrict__ S_pool, int32_t *__restrict__ status,
                   int qk_norm, float qk_eps) {
    constexpr int CG = D / 4, NT = CG * (D / kRows);
    constexpr int KV = D * (int)sizeof(Tin) / 16, FV = D / 4;  // 16-byte vectors of a row of k; of g or u
    __shared__ __align__(16) float s_k[CHUNK][D], s_u[CHUNK][D], s_g[CHUNK][D];
    __shared__ __align__(16) float s_dec[D];
    __shared__ __align__(16) Tin s_raw[CHUNK][D];
    __shared__ float s_scale[CHUNK];
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int n = blockIdx.x / H, h = blockIdx.x % H, tid = threadIdx.x;
    const int len = path_len[n], slot = slot_of(seq_idx, n, num_slots);
    const Tree t = tree_rows(cu, n, total_nodes, kMaxNodes);
    if (len == 0) return;
    if (t.nodes < 0 || slot < 0 || len < 0 || len > path_stride || len > t.nodes) {
        if (tid == 0) report_invalid(status);
        return;
    }
    const int cg = tid % CG, rg = tid / CG;
    float4 *Sv = reinterpret_cast<float4 *>(S_pool + ((size_t)slot * H + h) * D * D);
    float4 s[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) s[j] = __ldcs(&Sv[(size_t)(rg * kRows + j) * CG + cg]);

    const int32_t *nodes = path + (size_t)n * path_stride;
    for (int l0 = 0; l0 < len; l0 += CHUNK) {
        const int L = min(CHUNK, len - l0);
        int bad = 0;
        for (int i = tid; i < L * (KV + 2 * FV); i += NT) {
            const int r = i / (KV + 2 * FV), e = i % (KV + 2 * FV);
            const int node = nodes[l0 + r];
            if (node < 0 || node >= t.nodes) {
                bad = 1;
                continue;
            }
            const size_t at = ((size_t)(t.row0 + node) * H + h) * D;
            if (e < KV) tc::cp_async16(reinterpret_cast<char *>(s_raw[r]) + e * 16, reinterpret_cast<const char *>(k + at) + e * 16);
            else if (e < KV + FV) tc::cp_async16(&s_g[r][(e - KV) * 4], g + at + (e - KV) * 4);
            else tc::cp_async16(&s_u[r][(e - KV - FV) * 4], u + at + (e - KV - FV) * 4);
        }
        if (l0 == 0)  // the whole path is checked before anything is written
            for (int i = CHUNK + tid; i < len; i += NT) bad |= nodes[i] < 0 || nodes[i] >= t.nodes;
        tc::cp_async_wait_all();
        if (__syncthreads_or(bad)) {
            if (tid == 0) report_invalid(status);
            return;
        }
        if (qk_norm) {  // a group of min(NT, 32) threads per row
            constexpr int G = NT < 32 ? NT : 32;
            const int lane = tid % G;
            for (int r = tid / G; r < CHUNK; r += NT / G) {
                float ss = 0.f;
                if (r < L)
                    for (int c = lane; c < D; c += G) ss = fmaf(to_f32(s_raw[r][c]), to_f32(s_raw[r][c]), ss);
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
                s_k[r][c] = to_f32(s_raw[r][c]) * (expf(b) * (qk_norm ? s_scale[r] : 1.f));
                b += log_decay(s_g[r][c]);
            }
            s_dec[c] = expf(b);
        }
        __syncthreads();
#pragma unroll
        for (int j0 = 0; j0 < kRows; j0 += 4) {
            const float4 d4 = *reinterpret_cast<const float4 *>(&s_dec[rg * kRows + j0]);
            const float d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[j0 + e].x *= d[e]; s[j0 + e].y *= d[e]; s[j0 + e].z *= d[e]; s[j0 + e].w *= d[e];
            }
        }
        for (int r = 0; r < L; ++r) {
            const float4 w = *reinterpret_cast<const float4 *>(&s_u[r][cg * 4]);
#pragma unroll
            for (int j0 = 0; j0 < kRows; j0 += 4) {
                const float4 k4 = *reinterpret_cast<const float4 *>(&s_k[r][rg * kRows + j0]);
                const float kr[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float4 &x = s[j0 + e];
                    x.x = fmaf(kr[e], w.x, x.x); x.y = fmaf(kr[e], w.y, x.y);
                    x.z = fmaf(kr[e], w.z, x.z); x.w = fmaf(kr[e], w.w, x.w);
                }
            }
        }
        if (l0 + CHUNK < len) __syncthreads();  // the chunk's rows are free
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) __stcs(&Sv[(size_t)(rg * kRows + j) * CG + cg], s[j]);
}

template <typename Tin, int D, int CHUNK>
cudaError_t launch_commit_c(const TreeCommitArgs &a, cudaStream_t st) {
    return launch_dependent(tree_commit_kernel<Tin, D, CHUNK>, a.num_seqs * a.H, (D / 4) * (D / kRows), 0, st,
                            (const Tin *)a.k, a.g, a.u, a.cu, a.path, a.path_len, a.seq_idx, a.H, a.total_nodes,
                            a.path_stride, a.num_slots, a.S_pool, a.status, a.qk_norm, a.qk_eps);
}
template <typename Tin, int D>
cudaError_t launch_commit_d(const TreeCommitArgs &a, cudaStream_t st) {
    return a.path_stride > 8 ? launch_commit_c<Tin, D, 16>(a, st) : launch_commit_c<Tin, D, 8>(a, st);
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
// first.  One CTA per (request, channel block); a thread owns VEC neighbouring channels, whose rows it reads as
// 16 bytes (VEC = 8 of bf16, 4 of fp32; VEC = 1 where C or an address does not allow that).  All of the block's
// rows are on their way to shared memory at once, each read once; a thread copies what it will use itself.
// Bound by latency: one CTA's loads, then its sums, with 9 CTAs an SM.  Measured, 256 requests x 9 to 16 nodes x 4096
// channels, bf16: 21 us, for 53 MB of x and y and 12.6 MB of carried inputs.
constexpr int kConvThreads = 64;

template <typename Tin, int VEC>
__device__ __forceinline__ void load_row(const Tin *p, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] = to_f32(*p);
    } else {
        union {
            uint4 v;
            Tin x[VEC];
        } r;
        r.v = *reinterpret_cast<const uint4 *>(p);
        if constexpr (sizeof(Tin) == 2) {
            const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[2 * e] = __uint_as_float(w[e] << 16);
                f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = to_f32(r.x[e]);
        }
    }
}
template <typename Tin, int VEC>
__device__ __forceinline__ void store_row(Tin *p, const float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        *p = from_f32<Tin>(f[0]);
    } else {
        union {
            uint4 v;
            Tin x[VEC];
        } r;
#pragma unroll
        for (int e = 0; e < VEC; ++e) r.x[e] = from_f32<Tin>(f[e]);
        *reinterpret_cast<uint4 *>(p) = r.v;
    }
}
template <int VEC>
__device__ __forceinline__ void load_f32(const float *p, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] = *p;
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + e);
            f[e] = v.x; f[e + 1] = v.y; f[e + 2] = v.z; f[e + 3] = v.w;
        }
    }
}
template <int VEC>
__device__ __forceinline__ void store_f32(float *p, const float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        *p = f[0];
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 4)
            *reinterpret_cast<float4 *>(p + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    }
}

// One CTA's rows in shared memory: max_nodes of x, then the W - 1 carried ones (fp32).
template <typename Tin, int VEC>
constexpr size_t conv_row_bytes() { return (size_t)kConvThreads * VEC * sizeof(Tin); }

template <typename Tin, int VEC>
__device__ __forceinline__ void fetch_row(Tin *to, const Tin *from) {
    if constexpr (VEC == 1) *to = *from;
    else
#pragma unroll
        for (int e = 0; e < VEC * (int)sizeof(Tin); e += 16)
            tc::cp_async16(reinterpret_cast<char *>(to) + e, reinterpret_cast<const char *>(from) + e);
}

template <typename Tin, int W, int VEC>
__global__ void __launch_bounds__(kConvThreads)
tree_conv_kernel(const Tin *__restrict__ x, const float *__restrict__ w, const int32_t *__restrict__ parent,
                 const int32_t *__restrict__ cu, const int32_t *__restrict__ seq_idx, int total_nodes, int max_nodes,
                 int num_slots, int C, const float *__restrict__ pool, Tin *__restrict__ y,
                 int32_t *__restrict__ status) {
    __shared__ TreeShared ts;
    // where the j-th input before node i lies: its row's offset in bytes, or -1 - the offset of a carried row
    __shared__ __align__(16) int s_tap[kMaxNodes][W];
    extern __shared__ uint4 rows[];
    Tin *s_x = reinterpret_cast<Tin *>(rows) + threadIdx.x * VEC;
    float *s_past = reinterpret_cast<float *>(reinterpret_cast<char *>(rows) + max_nodes * conv_row_bytes<Tin, VEC>()) + threadIdx.x * VEC;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    constexpr int kStride = kConvThreads * VEC;
    const int n = blockIdx.y, tid = threadIdx.x, c = (blockIdx.x * kConvThreads + tid) * VEC;
    const int slot = slot_of(seq_idx, n, num_slots);
    const Tree t = tree_rows(cu, n, total_nodes, max_nodes);
    const Links links = load_links(parent, t);
    float wt[W][VEC];
    if (c < C && t.nodes > 0 && slot >= 0) {
        for (int i = 0; i < t.nodes; ++i)
            fetch_row<Tin, VEC>(s_x + i * kStride, x + (size_t)(t.row0 + i) * C + c);
        for (int m = 0; m < W - 1; ++m)  // the newest first
            fetch_row<float, VEC>(s_past + m * kStride, pool + ((size_t)slot * (W - 1) + (W - 2 - m)) * C + c);
        float all[W * VEC];
        if constexpr (VEC == 1) {
#pragma unroll
            for (int j = 0; j < W; ++j) all[j] = w[(size_t)c * W + j];
        } else {
            load_f32<W * VEC>(w + (size_t)c * W, all);
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) wt[j][e] = all[e * W + j];
    }
    if (!read_tree(ts, t, links, false) || slot < 0) {
        if (tid == 0) report_invalid(status);
        tc::cp_async_wait_all();
        return;
    }
    for (int i = tid; i < t.nodes; i += kConvThreads) {
        int at = i, m = 0;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            s_tap[i][j] = at >= 0 ? at * (int)conv_row_bytes<Tin, VEC>() : -1 - m++ * (int)conv_row_bytes<float, VEC>();
            at = at >= 0 ? ts.parent[at] : -1;
        }
    }
    tc::cp_async_wait_all();
    __syncthreads();
    if (c >= C) return;
    Tin *out = y + (size_t)t.row0 * C + c;
    const char *xs = reinterpret_cast<const char *>(s_x), *ps = reinterpret_cast<const char *>(s_past);
#pragma unroll 2
    for (int i = 0; i < t.nodes; ++i, out += C) {
        int tap[W];
        if constexpr (W % 4 == 0) {
#pragma unroll
            for (int j = 0; j < W; j += 4) *reinterpret_cast<int4 *>(&tap[j]) = *reinterpret_cast<const int4 *>(&s_tap[i][j]);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) tap[j] = s_tap[i][j];
        }
        float acc[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float v[VEC];
            if (tap[j] >= 0) load_row<Tin, VEC>(reinterpret_cast<const Tin *>(xs + tap[j]), v);
            else load_f32<VEC>(reinterpret_cast<const float *>(ps + (-1 - tap[j])), v);
            if constexpr (VEC == 1) {
                acc[0] = fmaf(wt[j][0], v[0], acc[0]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; e += 2) {  // two multiply-adds an instruction
                    const float2 r = tc::fma2(make_float2(wt[j][e], wt[j][e + 1]), make_float2(v[e], v[e + 1]),
                                              make_float2(acc[e], acc[e + 1]));
                    acc[e] = r.x;
                    acc[e + 1] = r.y;
                }
            }
        }
        store_row<Tin, VEC>(out, acc);
    }
}

// The carried inputs after a path: the last W - 1 of [carried inputs, the path's inputs].
template <typename Tin, int VEC>
__global__ void __launch_bounds__(kConvThreads)
tree_conv_commit_kernel(const Tin *__restrict__ x, const int32_t *__restrict__ cu, const int32_t *__restrict__ path,
                        const int32_t *__restrict__ path_len, const int32_t *__restrict__ seq_idx, int total_nodes,
                        int path_stride, int num_slots, int C, int W, float *__restrict__ pool,
                        int32_t *__restrict__ status) {
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int n = blockIdx.y, c = (blockIdx.x * kConvThreads + threadIdx.x) * VEC;
    const int len = path_len[n], slot = slot_of(seq_idx, n, num_slots);
    const Tree t = tree_rows(cu, n, total_nodes, kMaxNodes);
    if (len == 0) return;
    bool bad = t.nodes < 0 || slot < 0 || len < 0 || len > path_stride || len > t.nodes;
    int node[KDA_SHORT_CONV_MAX_W - 1];  // node of the new carried input j, or -1 for an old one
#pragma unroll
    for (int j = 0; j < KDA_SHORT_CONV_MAX_W - 1; ++j) {
        const int l = len - (W - 1) + j;
        node[j] = -1;
        if (j < W - 1 && l >= 0 && !bad) {
            node[j] = path[(size_t)n * path_stride + l];
            bad = node[j] < 0 || node[j] >= t.nodes;
        }
    }
    // the nodes before those count too: a path is refused here where the state's commit refuses it
    static_assert(kConvThreads >= kMaxNodes, "a thread per node of the path");
    if (!bad && (int)threadIdx.x < len) {
        const int at = path[(size_t)n * path_stride + threadIdx.x];
        bad = at < 0 || at >= t.nodes;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) report_invalid(status);
        return;
    }
    if (c >= C) return;
    float next[KDA_SHORT_CONV_MAX_W - 1][VEC];
    float *mine = pool + (size_t)slot * (W - 1) * C + c;
#pragma unroll
    for (int j = 0; j < KDA_SHORT_CONV_MAX_W - 1; ++j) {
        if (j < W - 1) {
            if (node[j] >= 0) load_row<Tin, VEC>(x + (size_t)(t.row0 + node[j]) * C + c, next[j]);
            else load_f32<VEC>(mine + (size_t)(j + len) * C, next[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < KDA_SHORT_CONV_MAX_W - 1; ++j)
        if (j < W - 1) store_f32<VEC>(mine + (size_t)j * C, next[j]);
}

// Whether rows of C elements and their fp32 counterparts can be taken 16 bytes at a time.
template <typename Tin>
bool rows_of_vectors(int C, const void *a, const void *b, const void *c, const void *d) {
    const uintptr_t any = (uintptr_t)a | (uintptr_t)b | (uintptr_t)c | (uintptr_t)d;
    return C % (16 / (int)sizeof(Tin)) == 0 && (any & 15u) == 0;
}

template <typename Tin, int VEC>
cudaError_t launch_conv_v(const TreeConvArgs &a, cudaStream_t st) {
    const dim3 grid((a.C + kConvThreads * VEC - 1) / (kConvThreads * VEC), a.num_seqs);
    const size_t smem = a.max_nodes * conv_row_bytes<Tin, VEC>() + (size_t)(a.W - 1) * conv_row_bytes<float, VEC>();
    cudaError_t e = cudaSuccess;
#define KDA_TREE_CONV(WW)                                                                                          \
    case WW:                                                                                                       \
        e = allow_smem<tree_conv_kernel<Tin, WW, VEC>>((int)smem);                                                 \
        if (e != cudaSuccess) return e;                                                                            \
        return launch_dependent(tree_conv_kernel<Tin, WW, VEC>, grid, kConvThreads, smem, st, (const Tin *)a.x,    \
                                a.w, a.parent, a.cu, a.seq_idx, a.total_nodes, a.max_nodes, a.num_slots, a.C,      \
                                a.pool, (Tin *)a.y, a.status);
    switch (a.W) {
        KDA_TREE_CONV(1) KDA_TREE_CONV(2) KDA_TREE_CONV(3) KDA_TREE_CONV(4)
        KDA_TREE_CONV(5) KDA_TREE_CONV(6) KDA_TREE_CONV(7) KDA_TREE_CONV(8)
        default: return cudaErrorInvalidValue;
    }
#undef KDA_TREE_CONV
}

template <typename Tin, int VEC>
cudaError_t launch_conv_commit_v(const TreeConvCommitArgs &a, cudaStream_t st) {
    const dim3 grid((a.C + kConvThreads * VEC - 1) / (kConvThreads * VEC), a.num_seqs);
    return launch_dependent(tree_conv_commit_kernel<Tin, VEC>, grid, kConvThreads, 0, st, (const Tin *)a.x, a.cu,
                            a.path, a.path_len, a.seq_idx, a.total_nodes, a.path_stride, a.num_slots, a.C, a.W, a.pool,
                            a.status);
}

template <typename Tin>
cudaError_t launch_conv_t(const TreeConvArgs &a, cudaStream_t st) {
    constexpr int VEC = 16 / (int)sizeof(Tin);
    return rows_of_vectors<Tin>(a.C, a.x, a.y, a.pool, a.w) ? launch_conv_v<Tin, VEC>(a, st) : launch_conv_v<Tin, 1>(a, st);
}
template <typename Tin>
cudaError_t launch_conv_commit_t(const TreeConvCommitArgs &a, cudaStream_t st) {
    constexpr int VEC = 16 / (int)sizeof(Tin);
    return rows_of_vectors<Tin>(a.C, a.x, a.pool, nullptr, nullptr) ? launch_conv_commit_v<Tin, VEC>(a, st)
                                                                    : launch_conv_commit_v<Tin, 1>(a, st);
}

}  // namespace

cudaError_t launch_tree_step(const TreeStepArgs &a, kda_dtype dt, cudaStream_t st) {
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
