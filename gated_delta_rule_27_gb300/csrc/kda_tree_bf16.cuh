// kda_tree_bf16.cuh -- what the bf16 tree-step kernels share: bf16 parts of fp32 values, arithmetic on eights, the
// decays in base 2, the inverse of I + A.
#pragma once

#include "kda_tc.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace tree16 {

// Largest |b| (powers of two) for which A and P are formed from the factors e^b and e^{-b}.  The second bf16 part of q e^b
// ends 17 bits below the value and bf16 at 2^-133, so a query keeps all its bits down to 2^-20 at the range's end (with
// 2^-115 one of 1e-5 kept four: o off by 8%).
constexpr float kMaxRange = 96.f;

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void unpack8(const uint4 &x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
// Eight values as bf16 parts: hi the nearest bf16, lo the nearest to what is left.
__device__ __forceinline__ void split8(const float (&f)[8], uint4 &hi, uint4 &lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = pack2(f[2 * i], f[2 * i + 1]);
        const float2 rest = tc::sub2(make_float2(f[2 * i], f[2 * i + 1]),
                                     make_float2(__uint_as_float(h[i] << 16), __uint_as_float(h[i] & 0xffff0000u)));
        l[i] = pack2(rest.x, rest.y);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}
// Eight values as four pairs.
template <typename Op>
__device__ __forceinline__ void pairs8(float (&f)[8], const float (&a)[8], const float (&b)[8], Op op) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const float2 r = op(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
        f[e] = r.x;
        f[e + 1] = r.y;
    }
}
__device__ __forceinline__ void add8(float (&f)[8], const float (&a)[8], const float (&b)[8]) {
    pairs8(f, a, b, [](float2 x, float2 y) { return tc::add2(x, y); });
}
__device__ __forceinline__ void mul8(float (&f)[8], const float (&a)[8], const float (&b)[8]) {
    pairs8(f, a, b, [](float2 x, float2 y) { return tc::mul2(x, y); });
}
__device__ __forceinline__ void scale8(float (&f)[8], const float (&a)[8], float b) {
    pairs8(f, a, a, [b](float2 x, float2) { return tc::mul2(x, make_float2(b, b)); });
}
__device__ __forceinline__ float sum_squares8(const float (&f)[8]) {
    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 8; e += 2) ss = tc::fma2(make_float2(f[e], f[e + 1]), make_float2(f[e], f[e + 1]), ss);
    return ss.x + ss.y;
}
__device__ __forceinline__ void read8(const float *p, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// The decays' exponents are kept in base 2, the hardware's exponential.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float4 log2_decay4(const float4 &g) {
    return make_float4(log_decay(g.x) * kLog2e, log_decay(g.y) * kLog2e, log_decay(g.z) * kLog2e,
                       log_decay(g.w) * kLog2e);
}
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The logistic function to about 2^-21, for a bf16 result.
__device__ __forceinline__ float gate_of(float z) { return __fdividef(1.f, 1.f + exp2_of(-kLog2e * z)); }

// A launch of a bf16 tree step.
struct Args {
    const __nv_bfloat16 *q, *k, *v;
    const float *g, *beta;
    const int32_t *parent, *cu, *seq_idx;
    int H, total_nodes, max_nodes, num_slots, ahead;
    const float *S_pool;
    __nv_bfloat16 *o;
    float *u;
    int32_t *status;
    int qk_norm;
    float qk_eps;
    const __nv_bfloat16 *gate;
    const float *weight;
    float out_eps;
};

// sum_{a < n} x_a t_a, x a 16-byte aligned row in shared memory whose entries at and behind n are zero (up to the
// next multiple of four)
template <int n>
__device__ __forceinline__ float row_dot(const float *x, const float *t) {
    float2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
    for (int a = 0; a < n; a += 4) {
        const float4 y = *reinterpret_cast<const float4 *>(x + a);
        acc[0] = tc::fma2(make_float2(y.x, y.y), make_float2(t[a], t[a + 1]), acc[0]);
        if (a + 2 < n) acc[1] = tc::fma2(make_float2(y.z, y.w), make_float2(t[a + 2], t[a + 3]), acc[1]);
    }
    return (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
}

// T = (I + A)^{-1} of an NB x NB diagonal block of A (zero on and above its diagonal), one column per lane:
// T_ij = [i = j] - sum_{a < i} A_ia T_aj.
template <int NB, int I = 0>
__device__ __forceinline__ void invert_block(const float *A, int stride, int lane, float (&t)[NB]) {
    if constexpr (I == 0) {
#pragma unroll
        for (int i = 0; i < NB; ++i) t[i] = 0.f;  // what a row's last vector reaches past its entries
    }
    if constexpr (I < NB) {
        t[I] = (I == lane ? 1.f : 0.f) - row_dot<I>(A + I * stride, t);
        invert_block<NB, I + 1>(A, stride, lane, t);
    }
}
}  // namespace tree16
}  // namespace kda
