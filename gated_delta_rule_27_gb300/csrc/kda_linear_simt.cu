// kda_linear_simt.cu -- chunked linear attention on the CUDA cores: fp32 inputs, and d = 16 or 64; and the chaining of
// the segments' states, which the tensor-core path shares.
//
// The recurrence itself, token by token, with the state in registers: a thread owns D / 4 of one column's rows (column
// = value dimension), so S_t = a S + k v needs the token's k rows, one v and no other thread, and o = S^T q is finished
// among the column's four threads by two exchanges.  q, k and v of 16 or 32 tokens are staged in shared memory as
// fp32 while those before them are worked on.  Arithmetic bounds it: 3 d^2 operations a token and head, all in fp32.
#include "kda_linear.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

using linear::Args;
using linear::Segment;

constexpr int kSplit = 4;   // threads of a column
constexpr float kGentle = 24.f;  // largest log2 of a decay over the staged tokens that the state's units may follow

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// OUT: the outputs and final states; else what each segment but a document's last adds to the state.
template <typename Tin, int D, bool OUT>
__global__ void __launch_bounds__(D * kSplit)
linear_simt_kernel(const Args a) {
    constexpr int NT = D * kSplit, R = D / kSplit, kWarps = NT / 32;
    constexpr int kTok = D == 128 ? 16 : 32;  // tokens staged at once
    constexpr int kLoads = kTok * D / NT;  // elements of a staged tensor a thread loads
    __shared__ __align__(16) float s_q[kTok][D], s_k[kTok][D], s_v[kTok][D], s_o[OUT ? kTok : 1][D];
    __shared__ float s_a[kTok], s_in[kTok], s_out[kTok];
    __shared__ bool s_gentle;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col = tid / kSplit, part = tid % kSplit;  // rows 4 (i kSplit + part) .. + 3 for i < R / 4
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const bool valid = linear::valid_table(a.cu, a.num_seqs, a.total);
    if (a.first && blockIdx.x == 0 && tid == 0) *a.status = valid ? (int32_t)KDA_OK : (int32_t)KDA_ERR_INVALID_ARG;
    if (!valid) return;
    const int slot = blockIdx.x / a.H, h = blockIdx.x - slot * a.H, hq = h / (a.H / a.Hqk);
    Segment sg;
    if (!linear::find_segment(a.cu, a.num_seqs, a.seg, slot, &sg) || (!OUT && sg.last)) return;
    const Tin *q = static_cast<const Tin *>(a.q), *k = static_cast<const Tin *>(a.k), *v = static_cast<const Tin *>(a.v);
    const size_t doc_state = ((size_t)sg.doc * a.H + h) * D * D, seg_state = ((size_t)slot * a.H + h) * D * D;
    const float *init = OUT ? linear::segment_start(a, sg, slot, h, (size_t)D * D) : nullptr;

    float2 S[R / 2];
#pragma unroll
    for (int i = 0; i < R / 4; ++i) {
        const size_t r = (size_t)4 * (i * kSplit + part) * D + col;
        S[2 * i] = init ? make_float2(init[r], init[r + D]) : make_float2(0.f, 0.f);
        S[2 * i + 1] = init ? make_float2(init[r + 2 * D], init[r + 3 * D]) : make_float2(0.f, 0.f);
    }
    double total = 0.0;  // log2 of the segment's decay

    Tin nq[kLoads], nk[kLoads], nv[kLoads];
    float ng = 0.f;
    auto fetch = [&](int c0) {
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
            const int i = e * NT + tid, t = c0 + i / D, c = i % D;
            if (t < sg.len) {
                const size_t at = ((size_t)(sg.t0 + t) * a.Hqk + hq) * D + c;
                if (OUT) nq[e] = q[at];
                nk[e] = k[at];
                nv[e] = v[((size_t)(sg.t0 + t) * a.H + h) * D + c];
            }
        }
        if (tid < kTok && c0 + tid < sg.len) ng = linear::log2_decay(a.per_token ? a.g[(size_t)(sg.t0 + c0 + tid) * a.H + h] : a.g[h]);
    };
    fetch(0);
    for (int c0 = 0; c0 < sg.len; c0 += kTok) {
        const int n = min(kTok, sg.len - c0);
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
            const int i = e * NT + tid;
            if (OUT) s_q[i / D][i % D] = to_f32(nq[e]);
            s_k[i / D][i % D] = to_f32(nk[e]);
            s_v[i / D][i % D] = to_f32(nv[e]);
        }
        if (tid < 32) {  // the decays' sums from the first staged token on
            float b = tid < n ? ng : 0.f;
#pragma unroll
            for (int off = 1; off < kTok; off <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, b, off);
                if (tid >= off) b += up;
            }
            const float all = __shfl_sync(0xffffffffu, b, kTok - 1);
            total += (double)all;
            float most = fabsf(b);  // (growth and decay may cancel in the whole)
#pragma unroll
            for (int off = 16; off; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
            const bool nan = __any_sync(0xffffffffu, b != b);
            if (tid < kTok) {
                s_a[tid] = exp2f(ng);
                s_in[tid] = exp2f(b);
                s_out[tid] = exp2f(-b);
            }
            if (tid == 0) s_gentle = !nan && most < kGentle;
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
        // The state is kept in units of the decay since the first of these tokens, where that is not so strong that the
        // units overflow: it saves the product with each token's decay, and the rounding of that decay, which a slow one
        // would pile up token after token.
        if (s_gentle) {
#pragma unroll 4
            for (int t = 0; t < n; ++t) {
                const float vo = s_v[t][col] * s_out[t];
                const float2 vv = make_float2(vo, vo);
                float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < R / 4; ++i) {
                    const float4 kk = *reinterpret_cast<const float4 *>(&s_k[t][4 * (i * kSplit + part)]);
                    S[2 * i] = tc::fma2(make_float2(kk.x, kk.y), vv, S[2 * i]);
                    S[2 * i + 1] = tc::fma2(make_float2(kk.z, kk.w), vv, S[2 * i + 1]);
                    if (OUT) {
                        const float4 qq = *reinterpret_cast<const float4 *>(&s_q[t][4 * (i * kSplit + part)]);
                        acc = tc::fma2(make_float2(qq.x, qq.y), S[2 * i], acc);
                        acc = tc::fma2(make_float2(qq.z, qq.w), S[2 * i + 1], acc);
                    }
                }
                if (OUT) {
                    float x = acc.x + acc.y;
                    x += __shfl_xor_sync(0xffffffffu, x, 1);
                    x += __shfl_xor_sync(0xffffffffu, x, 2);
                    if (part == 0) s_o[t][col] = x * s_in[t];
                }
            }
            const float2 end = make_float2(s_in[n - 1], s_in[n - 1]);
#pragma unroll
            for (int i = 0; i < R / 2; ++i) S[i] = tc::mul2(S[i], end);
        } else {
            for (int t = 0; t < n; ++t) {
                const float2 av = make_float2(s_a[t], s_a[t]), vv = make_float2(s_v[t][col], s_v[t][col]);
                float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < R / 4; ++i) {
                    const float4 kk = *reinterpret_cast<const float4 *>(&s_k[t][4 * (i * kSplit + part)]);
                    S[2 * i] = tc::fma2(make_float2(kk.x, kk.y), vv, tc::mul2(av, S[2 * i]));
                    S[2 * i + 1] = tc::fma2(make_float2(kk.z, kk.w), vv, tc::mul2(av, S[2 * i + 1]));
                    if (OUT) {
                        const float4 qq = *reinterpret_cast<const float4 *>(&s_q[t][4 * (i * kSplit + part)]);
                        acc = tc::fma2(make_float2(qq.x, qq.y), S[2 * i], acc);
                        acc = tc::fma2(make_float2(qq.z, qq.w), S[2 * i + 1], acc);
                    }
                }
                if (OUT) {
                    float x = acc.x + acc.y;
                    x += __shfl_xor_sync(0xffffffffu, x, 1);
                    x += __shfl_xor_sync(0xffffffffu, x, 2);
                    if (part == 0) s_o[t][col] = x;
                }
            }
        }
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
        for (int i = 0; i < R / 4; ++i) {
            const size_t r = (size_t)4 * (i * kSplit + part) * D + col;
            to[r] = S[2 * i].x;
            to[r + D] = S[2 * i].y;
            to[r + 2 * D] = S[2 * i + 1].x;
            to[r + 3 * D] = S[2 * i + 1].y;
        }
    }
    if (!OUT && tid == 0) a.seg_decay[(size_t)slot * a.H + h] = exp2f((float)total);
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
        cudaError_t e = launch_dependent(linear_simt_kernel<Tin, D, false>, grid, dim3(D * kSplit), 0, st, a);
        if (e == cudaSuccess) e = launch_linear_chain(a, D, st);
        if (e != cudaSuccess) return e;
        a.first = 0;
    }
    return launch_dependent(linear_simt_kernel<Tin, D, true>, grid, dim3(D * kSplit), 0, st, a);
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
