// kda_rope.cu -- rotary positions of q and k: pair i of a head turned by position x frequency_i.
//
// A frequency is held as the part of a turn that one position adds, in steps of 2^-64 turn.  Position times step in
// 64-bit integers, whole turns falling off the top, is the angle to within position x 2^-65 turn: no far position
// loses anything, and no 64-bit floating point is needed.  The upper 32 bits, as a signed part of half a turn, go to
// sincospi in fp32.
//
// Bound by HBM: q and k are read and written once.  A block works out the sines and cosines of a few tokens once, in
// shared memory, and turns those tokens' heads, 16 bytes a load: of two vectors half the rotated part apart, or of one that
// holds whole pairs.  (One thread for each pair with its own sine and cosine took 53 us for 4096 tokens of 32 heads, two
// thirds of it in the functions.)  65536 tokens x 32 heads of 128, bf16: 164 us in halves, 180 interleaved (158 at a plain copy's
// rate); 4096 tokens 15.6 and 17.2 for 9.9, caches cold (14.8 in halves among other calls on other inputs).  (A thread that
// keeps its place in the head and goes through the heads issues fewer instructions and took longer: 178 us for 169 at the time, 222
// for 199.)
#include "kda_linear.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;       // (256 at up to 64 registers: 16.1 and 17.7 us for the 15.6 and 17.2 of 4096 tokens, 169 and 186
                                    // for the 164 and 179 of 65536; without the bound on registers 21 and 200 interleaved)
constexpr int kMaxTokens = 4;       // tokens of a block
constexpr int kTable = 4096;        // sines and cosines that a block may hold

template <typename Tin, int N>
struct alignas(N * sizeof(Tin)) Vec {
    Tin x[N];
};
// N elements; one by one where they may start anywhere.
template <bool ANYWHERE, typename Tin, int N>
__device__ __forceinline__ void copy(Tin *to, const Tin *from) {
    if constexpr (ANYWHERE) {
#pragma unroll
        for (int i = 0; i < N; ++i) to[i] = from[i];
    } else if constexpr (N * sizeof(Tin) == 16) {
        *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from);
    } else if constexpr (N * sizeof(Tin) == 8) {
        *reinterpret_cast<uint2 *>(to) = *reinterpret_cast<const uint2 *>(from);
    } else {
        static_assert(N * sizeof(Tin) == 4);
        *reinterpret_cast<uint32_t *>(to) = *reinterpret_cast<const uint32_t *>(from);
    }
}
template <typename Tin, int N, bool ANYWHERE>
__device__ __forceinline__ Vec<Tin, N> load(const Tin *p) {
    Vec<Tin, N> v;
    copy<ANYWHERE, Tin, N>(v.x, p);
    return v;
}
template <bool ANYWHERE, typename Tin, int N>
__device__ __forceinline__ void store(Tin *p, const Vec<Tin, N> &v) {
    copy<ANYWHERE, Tin, N>(p, v.x);
}

// Block (x, y): tokens x `tokens` on, heads y `heads` on (q's first, then k's).  A head is `turned` items that turn VEC
// pairs (VEC / 2 if INTERLEAVED) and `copied` items of VEC elements behind them.
template <typename Tin, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 8) rope_kernel(const RopeArgs a, int tokens, int heads, int turned, int copied) {
    constexpr int W = INTERLEAVED && VEC == 1 ? 2 : VEC, kBatch = INTERLEAVED ? 4 : 2;  // elements of a load; items at once
    extern __shared__ float2 s_turn[];  // [tokens, pairs]: cosine, sine
    tc::grid_dep_launch();
    tc::grid_dep_wait();
    const int pairs = a.rot / 2, t0 = blockIdx.x * tokens, h0 = blockIdx.y * heads;
    const int nt = min(tokens, a.total - t0), nh = min(heads, a.Hq + a.Hk - h0);
    for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
        const int t = i / pairs, p = i - t * pairs;
        const unsigned long long turn = (unsigned long long)(long long)a.positions[t0 + t] * a.steps[p];
        float sn, cs;
        sincospif((float)(int)(turn >> 32) * 0x1p-31f, &sn, &cs);
        s_turn[i] = make_float2(cs * a.scale, sn * a.scale);
    }
    __syncthreads();
    // Each thread has kBatch loads under way before it turns the first (outputs may be in place, so the compiler cannot tell
    // that they could be): one at a time left the copy at 63% of HBM's rate.
    const int items = turned + copied, all = nt * nh * items;
    const int item_step = kThreads % items, head_step = kThreads / items;
    int item = threadIdx.x % items, h = threadIdx.x / items, t = h / nh;
    h -= t * nh;
    for (int i = threadIdx.x; i < all; i += kBatch * kThreads) {
        Tin *to[kBatch];
        const float2 *turn[kBatch];  // null: a copy
        Vec<Tin, W> lo[kBatch], hi[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (i + b * kThreads < all) {
                const bool is_q = h0 + h < a.Hq, turns = item < turned;
                const size_t at = ((size_t)(t0 + t) * (is_q ? a.Hq : a.Hk) + (is_q ? h0 + h : h0 + h - a.Hq)) * a.d +
                                  (turns ? item * (INTERLEAVED ? W : VEC) : a.rot + (item - turned) * VEC);
                const Tin *x = static_cast<const Tin *>(is_q ? a.q : a.k) + at;
                to[b] = static_cast<Tin *>(is_q ? a.q_out : a.k_out) + at;
                turn[b] = turns ? s_turn + t * pairs + item * (INTERLEAVED ? W / 2 : VEC) : nullptr;
                if (turns || W == VEC) lo[b] = load<Tin, W, VEC == 1>(x);
                else lo[b].x[0] = x[0];
                if (!INTERLEAVED && turns) hi[b] = load<Tin, W, VEC == 1>(x + pairs);
            }
            item += item_step;
            h += head_step;
            if (item >= items) {
                item -= items;
                ++h;
            }
            while (h >= nh) {
                h -= nh;
                ++t;
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (i + b * kThreads >= all) break;
            if (!turn[b]) {
                if (W == VEC) store<VEC == 1>(to[b], lo[b]);
                else to[b][0] = lo[b].x[0];
                continue;
            }
            if constexpr (INTERLEAVED) {
#pragma unroll
                for (int e = 0; e < W; e += 2) {
                    const float u = to_f32(lo[b].x[e]), w = to_f32(lo[b].x[e + 1]);
                    const float2 f = turn[b][e / 2];
                    lo[b].x[e] = from_f32<Tin>(u * f.x - w * f.y);
                    lo[b].x[e + 1] = from_f32<Tin>(w * f.x + u * f.y);
                }
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    const float u = to_f32(lo[b].x[e]), w = to_f32(hi[b].x[e]);
                    const float2 f = turn[b][e];
                    lo[b].x[e] = from_f32<Tin>(u * f.x - w * f.y);
                    hi[b].x[e] = from_f32<Tin>(w * f.x + u * f.y);
                }
                store<VEC == 1>(to[b] + pairs, hi[b]);
            }
            store<VEC == 1>(to[b], lo[b]);
        }
    }
}

template <typename Tin, int VEC, bool INTERLEAVED>
cudaError_t launch_v(const RopeArgs &a, cudaStream_t st) {
    const int pairs = a.rot / 2, all = a.Hq + a.Hk;
    // Few tokens: a block for each and for part of its heads, so that every SM has eight (512 tokens x 32 heads 3.1 us; four
    // 4.0, sixteen 3.9); else up to four tokens, which share
    // what a block costs (65536 tokens x 32 heads, blocks of 256 threads: 344 us one by one, 205 four, 192 eight; of 128: 164 four, 165 eight).
    int tokens = a.total / 1024;
    tokens = tokens < 1 ? 1 : tokens > kMaxTokens ? kMaxTokens : tokens;
    while (tokens > 1 && tokens * pairs > kTable) --tokens;
    const int blocks = (a.total - 1) / tokens + 1;
    int parts = 152 * 8 / blocks;
    parts = parts < 1 ? 1 : parts > all ? all : parts;
    const int heads = (all + parts - 1) / parts;
    const bool in_place = (a.Hq == 0 || a.q == a.q_out) && (a.Hk == 0 || a.k == a.k_out);
    const int turned = INTERLEAVED ? (VEC == 1 ? pairs : a.rot / VEC) : pairs / VEC, copied = in_place ? 0 : (a.d - a.rot) / VEC;
    const dim3 grid((unsigned)blocks, (unsigned)((all + heads - 1) / heads));
    return launch_dependent(rope_kernel<Tin, VEC, INTERLEAVED>, grid, dim3(kThreads), (size_t)tokens * pairs * sizeof(float2), st, a, tokens, heads,
                            turned, copied);
}

// The widest vectors, 16 bytes at most, of which every one of a head starts on its own size and turns as a whole (20 of 80
// elements turned, halves: fp32, 1001 tokens x 12 heads 6.5 us element by element, 4.7 by two; bf16, 4096 x 32 heads 48 and 30).
template <typename Tin, int VEC, bool INTERLEAVED>
cudaError_t launch_t(const RopeArgs &a, cudaStream_t st) {
    if constexpr (VEC > 1) {
        const auto aligned = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % (VEC * sizeof(Tin)) == 0; };
        if (a.d % VEC || (INTERLEAVED ? a.rot : a.rot / 2) % VEC || !aligned(a.q) || !aligned(a.k) || !aligned(a.q_out) || !aligned(a.k_out))
            return launch_t<Tin, VEC / 2, INTERLEAVED>(a, st);
    }
    return launch_v<Tin, VEC, INTERLEAVED>(a, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, kda_dtype dt, cudaStream_t st) {
    if (dt == KDA_BF16) return a.interleaved ? launch_t<__nv_bfloat16, 8, true>(a, st) : launch_t<__nv_bfloat16, 8, false>(a, st);
    return a.interleaved ? launch_t<float, 4, true>(a, st) : launch_t<float, 4, false>(a, st);
}

}  // namespace kda
