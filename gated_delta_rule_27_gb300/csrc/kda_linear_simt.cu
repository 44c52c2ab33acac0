// kda_linear_simt.cu -- chunked linear attention on the CUDA cores: fp32 inputs, and d = 16 or 64; and the chaining of
// the segments' states, which the tensor-core path shares.
//
// The recurrence itself, token by token, with the state in registers: a thread owns a tile of the state, so
// S_t = a S + k v needs the token's k and v of that tile and no other thread.  o = S^T q is added up among the threads of a
// column (lanes of one warp), two tokens at a time: each exchange leaves a lane half of the sums.  q, k and v of 16 or 32
// tokens are staged in shared memory as fp32 while those before them are worked on.
//
// Arithmetic bounds it at its best, 2 d^2 multiply-adds a token and head in fp32; what it takes in fact is the registers'
// share of shared memory, 128 bytes a clock whoever else wants the same: with one column a thread (64 bytes of k and q for
// 8 elements) a token took 300 clocks of an SM at d = 64, with tiles of 8 x 4 it takes a quarter of that.  1501 tokens x 5 heads,
// fp32, d = 64: 27 us for the three launches, where HBM would need 0.8: 235 CTAs of four warps, each of which goes through its 32
// tokens one after the other.
#include <type_traits>

#include "kda_linear.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

using linear::Args;
using linear::Segment;

constexpr float kGentle = 24.f;  // largest range of the decays' sums (log2) over the staged tokens that the state's units may follow

// A thread's tile: kRows x kCols of the state; the D / kRows threads of a column are neighbours in a warp, and hold a sum for
// each of two tokens' kCols columns in the end.
template <int D>
struct Tile {
    static constexpr int kRows = D == 16 ? 4 : 8, kCols = D == 16 ? 2 : D == 64 ? 4 : 8;
    static constexpr int kLanes = D / kRows, kThreads = kLanes * (D / kCols);
    static constexpr int kTok = D == 128 ? 16 : 32;              // tokens staged at once
    static constexpr int kVecs = kTok * D / 4 / kThreads;        // vectors of four elements of a staged tensor a thread loads
    static_assert(kLanes == 2 * kCols && kLanes <= 32);
};

template <typename Tin>
struct alignas(4 * sizeof(Tin)) Four {
    Tin x[4];
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// OUT: the outputs and final states; else what each segment but a document's last adds to the state.  (Three blocks an SM have to
// be asked for where the compiler aims at four, with 128 registers and some spilled: 1501 tokens x 5 heads 27.4 us, else 29.8.)
template <typename Tin, int D, bool OUT>
__global__ void __launch_bounds__(Tile<D>::kThreads, D == 64 && !OUT ? 3 : 0)
linear_simt_kernel(const Args a) {
    using T = Tile<D>;
    constexpr int NT = T::kThreads, R = T::kRows, C = T::kCols, kTok = T::kTok, kWarps = NT / 32;
    __shared__ __align__(16) float s_q[kTok][D], s_k[kTok][D], s_v[kTok][D], s_o[OUT ? kTok : 1][D];
    __shared__ float s_a[kTok], s_in[kTok], s_out[kTok], s_first, s_last;
    __shared__ bool s_gentle;
    __shared__ linear::Repeated s_repeated;  // of one decay for a head: a stage's
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int part = tid % T::kLanes, row0 = part * R, col0 = tid / T::kLanes * C;
    // (behind the segments' kernels, which have waited for everything before them, only the states have to be waited for)
    if (a.first) tc::grid_dep_wait();
    tc::grid_dep_launch();
    const bool valid = linear::valid_table(a.cu, a.num_seqs, a.total);
    if (a.first && blockIdx.x == 0 && tid == 0) *a.status = valid ? (int32_t)KDA_OK : (int32_t)KDA_ERR_INVALID_ARG;
    const int slot = blockIdx.x / a.H, h = blockIdx.x - slot * a.H, hq = h / (a.H / a.Hqk);
    Segment sg;
    if (!valid || !linear::find_segment(a.cu, a.num_seqs, a.seg, slot, &sg) || (!OUT && sg.last)) {
        if (!a.first) tc::grid_dep_wait();  // so that this kernel's end means the end of the ones before it
        return;
    }
    const Tin *q = static_cast<const Tin *>(a.q), *k = static_cast<const Tin *>(a.k), *v = static_cast<const Tin *>(a.v);
    const size_t doc_state = ((size_t)sg.doc * a.H + h) * D * D, seg_state = ((size_t)slot * a.H + h) * D * D;
    const float *init = OUT ? linear::segment_start(a, sg, slot, h, (size_t)D * D) : nullptr;
    double total = 0.0;  // log2 of the segment's decay

    Four<Tin> nq[T::kVecs], nk[T::kVecs], nv[T::kVecs];
    float ng = 0.f;
    auto fetch = [&](int c0) {
#pragma unroll
        for (int e = 0; e < T::kVecs; ++e) {
            const int i = (e * NT + tid) * 4, t = c0 + i / D, c = i % D;
            if (t < sg.len) {
                const size_t at = ((size_t)(sg.t0 + t) * a.Hqk + hq) * D + c;
                if (OUT) nq[e] = *reinterpret_cast<const Four<Tin> *>(q + at);
                nk[e] = *reinterpret_cast<const Four<Tin> *>(k + at);
                nv[e] = *reinterpret_cast<const Four<Tin> *>(v + ((size_t)(sg.t0 + t) * a.H + h) * D + c);
            }
        }
        if (tid < kTok && c0 + tid < sg.len) ng = linear::log2_decay(a.per_token ? a.g[(size_t)(sg.t0 + c0 + tid) * a.H + h] : a.g[h]);
    };
    // (rows behind the segment are staged as zeros, which add nothing to the state)
    const auto stage = [](float *to, const Four<Tin> &x, bool there) {
        *reinterpret_cast<float4 *>(to) = there ? make_float4(to_f32(x.x[0]), to_f32(x.x[1]), to_f32(x.x[2]), to_f32(x.x[3])) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    fetch(0);
    if (!a.first) tc::grid_dep_wait();
    float2 S[R / 2][C];  // pairs of rows
#pragma unroll
    for (int r = 0; r < R / 2; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const size_t at = (size_t)(row0 + 2 * r) * D + col0 + c;
            S[r][c] = init ? make_float2(init[at], init[at + D]) : make_float2(0.f, 0.f);
        }
    float unit = 1.f;  // of the state in S
    const bool repeats = !a.per_token && sg.len >= 2 * kTok;
    for (int c0 = 0; c0 < sg.len; c0 += kTok) {
        const int n = min(kTok, sg.len - c0);
#pragma unroll
        for (int e = 0; e < T::kVecs; ++e) {
            const int i = (e * NT + tid) * 4, t = i / D, c = i % D;
            if (OUT) stage(&s_q[t][c], nq[e], t < n);
            stage(&s_k[t][c], nk[e], t < n);
            stage(&s_v[t][c], nv[e], t < n);
        }
        if (tid < 32) {  // the decays' sums from the first staged token on
            float b = tid < n ? ng : 0.f;
#pragma unroll
            for (int off = 1; off < kTok; off <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, b, off);
                if (tid >= off) b += up;
            }
            const float end = __shfl_sync(0xffffffffu, b, kTok - 1);
            total += (double)end;
            // the least and the most of 0 and the sums (as integers: bits of floats of one sign are in their absolute values' order)
            const float mine = tid < kTok ? b : 0.f;
            const float least = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fminf(mine, 0.f))));
            const float most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(mine, 0.f))));
            const bool gentle = !__any_sync(0xffffffffu, b != b) && most - least < kGentle;
            if (tid < kTok) {
                s_a[tid] = tid < n ? exp2f(ng) : 1.f;
                s_in[tid] = exp2f(b - least);
                s_out[tid] = exp2f(least - b);
            }
            if (tid == 0) {
                s_gentle = gentle;
                s_first = exp2f(least);
                s_last = exp2f(end - least);
                if (repeats) {  // (the end is the least of the sums, or the start is)
                    if (c0 == 0) s_repeated = linear::Repeated::of((double)ng * kTok);
                    if (n == kTok) (ng < 0.f ? s_first : s_last) = s_repeated.next();
                }
            }
        }
        __syncthreads();
        if (c0 + kTok < sg.len) fetch(c0 + kTok);
        if (a.fu.qk_norm) {
            for (int r = warp; r < (OUT ? 2 : 1) * n; r += kWarps) {
                float *row = r < n ? s_k[r] : s_q[r - n];
                float ss = 0.f;
                for (int c = lane; c < D; c += 32) ss = fmaf(row[c], row[c], ss);
                const float scale = rsqrtf(warp_sum(ss) + a.fu.qk_eps);
                for (int c = lane; c < D; c += 32) row[c] *= scale;
            }
            __syncthreads();
        }
        // The state is kept in units of the decay since the first of these tokens, where that is not too strong: it saves the
        // product with each token's decay, and the rounding of that decay, which a slow one would pile up token after token.
        // The unit is the smallest of those decays (the last one's, unless something grows), so that nothing is above what the
        // recurrence itself holds; what falls below fp32's numbers by it is 2^-125 at most.
        const bool gentle = s_gentle;
        const float change = gentle ? unit * s_first : unit;
#pragma unroll
        for (int r = 0; r < R / 2; ++r)
#pragma unroll
            for (int c = 0; c < C; ++c) S[r][c] = tc::mul2(S[r][c], make_float2(change, change));
        unit = gentle ? s_last : 1.f;
        // (A loop for each kind, and two pairs of tokens unrolled: 33000 tokens x 32 heads, d = 64, bf16 1190 us, with the choice
        // inside 1250; 1501 x 16 40 us, without unrolling 50, with four pairs 44.)
        const auto tokens = [&](auto kind) {
            constexpr bool gentle = decltype(kind)::value;
#pragma unroll(D == 128 ? 1 : 2)
            for (int t0 = 0; t0 < n; t0 += 2) {
                float x[2 * C];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = t0 + u;
                    float vv[C];
#pragma unroll
                    for (int c = 0; c < C; c += 2) *reinterpret_cast<float2 *>(vv + c) = *reinterpret_cast<const float2 *>(&s_v[t][col0 + c]);
                    if (gentle) {
                        const float w = s_out[t];
#pragma unroll
                        for (int c = 0; c < C; ++c) vv[c] *= w;
                    } else {
                        const float2 av = make_float2(s_a[t], s_a[t]);
#pragma unroll
                        for (int r = 0; r < R / 2; ++r)
#pragma unroll
                            for (int c = 0; c < C; ++c) S[r][c] = tc::mul2(av, S[r][c]);
                    }
                    float2 acc[C];
#pragma unroll
                    for (int c = 0; c < C; ++c) acc[c] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int r = 0; r < R / 2; r += 2) {
                        const float4 kk = *reinterpret_cast<const float4 *>(&s_k[t][row0 + 2 * r]);
                        const float4 qq = OUT ? *reinterpret_cast<const float4 *>(&s_q[t][row0 + 2 * r]) : kk;
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            const float2 vc = make_float2(vv[c], vv[c]);
                            S[r][c] = tc::fma2(make_float2(kk.x, kk.y), vc, S[r][c]);
                            S[r + 1][c] = tc::fma2(make_float2(kk.z, kk.w), vc, S[r + 1][c]);
                            if (OUT) {
                                acc[c] = tc::fma2(make_float2(qq.x, qq.y), S[r][c], acc[c]);
                                acc[c] = tc::fma2(make_float2(qq.z, qq.w), S[r + 1][c], acc[c]);
                            }
                        }
                    }
#pragma unroll
                    for (int c = 0; c < C; ++c) x[u * C + c] = acc[c].x + acc[c].y;
                }
                if (OUT) {
#pragma unroll
                    for (int half = C; half; half >>= 1) {
                        const bool up = part & half;
#pragma unroll
                        for (int i = 0; i < half; ++i) {
                            const float give = up ? x[i] : x[i + half], keep = up ? x[i + half] : x[i];
                            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, half);
                        }
                    }
                    const int t = t0 + part / C;  // the lane's sum is token part / C's of column part % C
                    s_o[t][col0 + part % C] = gentle ? x[0] * s_in[t] : x[0];
                }
            }
        };
        if (gentle) tokens(std::true_type());
        else tokens(std::false_type());
        __syncthreads();
        if (OUT) {
            Tin *o = static_cast<Tin *>(a.o);
            const Tin *z = static_cast<const Tin *>(a.fu.gate);
            for (int t = warp; t < n; t += kWarps) {
                const size_t at = ((size_t)(sg.t0 + c0 + t) * a.H + h) * D;
                float scale = 1.f;
                if (z) {
                    float ss = 0.f;
                    for (int c = lane; c < D; c += 32) ss = fmaf(s_o[t][c], s_o[t][c], ss);
                    scale = rsqrtf(warp_sum(ss) * (1.f / D) + a.fu.out_eps);
                }
                for (int c = lane; c < D; c += 32) {
                    float x = s_o[t][c];
                    if (z) x = x * scale * (a.fu.weight ? a.fu.weight[c] : 1.f) * sigmoidf(to_f32(z[at + c]));
                    o[at + c] = from_f32<Tin>(x);
                }
            }
            __syncthreads();
        }
    }
    float *to = OUT ? (sg.last && a.S_final ? a.S_final + doc_state : nullptr) : a.seg_state + seg_state;
    if (to) {
#pragma unroll
        for (int r = 0; r < R / 2; ++r)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const size_t at = (size_t)(row0 + 2 * r) * D + col0 + c;
                to[at] = S[r][c].x * unit;
                to[at + D] = S[r][c].y * unit;
            }
    }
    // (one decay for a head: a factor that the chain of segments repeats)
    if (!OUT && tid == 0)
        a.seg_decay[(size_t)slot * a.H + h] =
            a.per_token ? exp2f((float)total) : linear::Repeated::of((double)linear::log2_decay(a.g[h]) * sg.len).at(sg.index);
}

// The state behind each segment but a document's last, in place of what the segment adds: S <- decay S + added, from
// the document's incoming state on.  Block x looks after document x, or where documents outnumber segments after the one
// that holds the first token of the x-th stretch of `seg` tokens, if that is the first such token in it: every document of
// more than one segment holds one.
constexpr int kChainThreads = 256, kLinks = 8;
__global__ void __launch_bounds__(kChainThreads) linear_chain_kernel(const Args a, int vecs, int by_document) {
    tc::grid_dep_launch();  // (the kernel before this one has waited for all that the next one reads, but the states)
    const int h = blockIdx.y, token = blockIdx.x * a.seg;
    int doc = blockIdx.x;
    if (!by_document) {
        int hi = a.num_seqs;  // cu[doc] <= token < cu[hi]
        doc = 0;
        while (hi - doc > 1) {
            const int mid = (doc + hi) >> 1;
            if (a.cu[mid] <= token) doc = mid;
            else hi = mid;
        }
    }
    const int begin = a.cu[doc], len = a.cu[doc + 1] - begin;
    const bool mine = len > a.seg && (by_document || (token >= begin && token - begin < a.seg));
    if (!mine || !linear::valid_table(a.cu, a.num_seqs, a.total)) {
        tc::grid_dep_wait();  // (so that this kernel's end means the end of the one before it)
        return;
    }
    const int links = (len + a.seg - 1) / a.seg - 1, slot = begin / a.seg + doc;
    const int e = blockIdx.z * kChainThreads + threadIdx.x;
    tc::grid_dep_wait();
    if (e >= vecs) return;
    float4 s = a.S0 ? reinterpret_cast<const float4 *>(a.S0)[((size_t)doc * a.H + h) * vecs + e] : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 *p = reinterpret_cast<float4 *>(a.seg_state) + ((size_t)slot * a.H + h) * vecs + e;
    const float *decay = a.seg_decay + (size_t)slot * a.H + h;
    const size_t step = (size_t)a.H * vecs;
    if (a.aliased) p[links * step] = s;
    // eight links' loads at a time: one after another, each would wait for memory
    for (int i = 0; i < links; i += kLinks) {
        float4 add[kLinks];
        float d[kLinks];
#pragma unroll
        for (int l = 0; l < kLinks; ++l)
            if (i + l < links) {
                add[l] = __ldcg(p + l * step);
                d[l] = __ldcg(decay + l * a.H);
            }
#pragma unroll
        for (int l = 0; l < kLinks; ++l)
            if (i + l < links) {
                s.x = fmaf(d[l], s.x, add[l].x);
                s.y = fmaf(d[l], s.y, add[l].y);
                s.z = fmaf(d[l], s.z, add[l].z);
                s.w = fmaf(d[l], s.w, add[l].w);
                p[l * step] = s;
            }
        p += kLinks * step;
        decay += kLinks * a.H;
    }
}

template <typename Tin, int D>
cudaError_t launch_d(const Args &args, cudaStream_t st) {
    Args a = args;
    a.first = 1;
    const dim3 grid((unsigned)(a.slots * a.H));
    if (a.total > a.seg) {
        cudaError_t e = launch_dependent(linear_simt_kernel<Tin, D, false>, grid, dim3(Tile<D>::kThreads), 0, st, a);
        if (e == cudaSuccess) e = launch_linear_chain(a, D, st);
        if (e != cudaSuccess) return e;
        a.first = 0;
    }
    return launch_dependent(linear_simt_kernel<Tin, D, true>, grid, dim3(Tile<D>::kThreads), 0, st, a);
}

template <typename Tin>
cudaError_t launch_t(const Args &a, int d, cudaStream_t st) {
    switch (d) {
        case 16: return launch_d<Tin, 16>(a, st);
        case 64: return launch_d<Tin, 64>(a, st);
        case 128: return launch_d<Tin, 128>(a, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_linear_simt(const linear::Args &a, int d, kda_dtype dt, cudaStream_t st) {
    return dt == KDA_BF16 ? launch_t<__nv_bfloat16>(a, d, st) : launch_t<float>(a, d, st);
}

cudaError_t launch_linear_chain(const linear::Args &a, int d, cudaStream_t st) {
    const int vecs = d * d / 4, stretches = (a.total + a.seg - 1) / a.seg;
    const bool by_document = a.num_seqs <= stretches;
    const dim3 grid((unsigned)(by_document ? a.num_seqs : stretches), (unsigned)a.H, (unsigned)((vecs + kChainThreads - 1) / kChainThreads));
    return launch_dependent(linear_chain_kernel, grid, dim3(kChainThreads), 0, st, a, vecs, by_document ? 1 : 0);
}

}  // namespace kda
