// kda_rope.cu -- rotary positions of q and k: pair i of a head turned by position x frequency_i.
//
// A frequency is held as the part of a turn that one position adds, in steps of 2^-64 turn.  Position times step in
// 64-bit integers, whole turns falling off the top, is the angle to within position x 2^-65 turn: no far position
// loses anything, and no 64-bit floating point is needed.  The upper 32 bits, as a signed part of half a turn, go to
// sincospi in fp32.
//
// Bound by HBM: q and k are read and written once.  A thread works out the angles of V pairs of one token once and
// turns those pairs in all of the token's heads that fall to it.
#include "kda_linear.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// Pairs: (2i, 2i + 1) interleaved, else (i, i + rot / 2).
template <typename Tin>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
    tc::grid_dep_launch();
    tc::grid_dep_wait();
    const int pairs = a.rot / 2, heads = a.Hq + a.Hk;
    const int64_t all = (int64_t)a.total * heads * pairs;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kThreads) {
        const int p = (int)(i % pairs);
        const int64_t row = i / pairs;
        const int h = (int)(row % heads);
        const int64_t t = row / heads;
        const unsigned long long turn = (unsigned long long)(long long)a.positions[t] * a.steps[p];
        float sn, cs;
        sincospif((float)(int)(turn >> 32) * 0x1p-31f, &sn, &cs);
        sn *= a.scale;
        cs *= a.scale;
        const bool is_q = h < a.Hq;
        const size_t at = is_q ? ((size_t)t * a.Hq + h) * a.d : ((size_t)t * a.Hk + (h - a.Hq)) * a.d;
        const Tin *x = static_cast<const Tin *>(is_q ? a.q : a.k) + at;
        Tin *y = static_cast<Tin *>(is_q ? a.q_out : a.k_out) + at;
        const int lo = a.interleaved ? 2 * p : p, hi = a.interleaved ? 2 * p + 1 : p + pairs;
        const float u = to_f32(x[lo]), w = to_f32(x[hi]);
        y[lo] = from_f32<Tin>(u * cs - w * sn);
        y[hi] = from_f32<Tin>(w * cs + u * sn);
        if (x != y)
            for (int c = a.rot + p; c < a.d; c += pairs) y[c] = x[c];
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, kda_dtype dt, cudaStream_t st) {
    const int64_t all = (int64_t)a.total * (a.Hq + a.Hk) * (a.rot / 2);
    const int64_t blocks = (all + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20));
    return dt == KDA_BF16 ? launch_dependent(rope_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, a)
                          : launch_dependent(rope_kernel<float>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace kda
