// kda_tree_tc.cu -- the draft-tree step on the Blackwell tensor cores (tcgen05): bf16 inputs, d = 128.
//
// With b_i the log-decay along the path to node i, K~ = k e^b, Q~ = q e^b and K^ = k e^{-b} (kda_tree.cu has the
// recurrence), one CTA per (request, head) forms
//     [A | P]^T-rows:  D1 = [K~ ; Q~] K^T        (nodes x nodes, masked to the paths; A scaled by beta)
//     state products:  D2 = S^T [K~ ; Q~]^T      (128 state columns x 2 M)
//     u_i = beta_i v_i - beta_i x_i - sum_a A_ia u_a,   o_i = y_i + sum_a P_ia u_a
// so the pool's state is read once, whatever the tree's size.  The floor is that read, 64 KB per (request, head).
//
// u moves the fp32 state, so it is formed to fp32 accuracy: every operand is split into two bf16 parts, hi + lo,
// and each product takes hi hi + hi lo + lo hi with fp32 accumulators (2^-17 relative to a term; one part alone
// would leave 2^-9).  The substitution runs in fp32 on the CUDA cores: D2's lanes are state columns, so a thread owns a column and needs
// no other thread's results.  A factor e^{-b} would overflow where the decays along a path sum to more than
// kMaxRange; such a request takes its A and P pairwise from the path's own exponents instead.
#include "kda_tc.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace {

constexpr int kD = 128, kThreads = 256;
constexpr float kMaxRange = 80.f;

// Shared memory for trees of at most MP nodes, in bytes.  Operand images are K-major with the 128-byte swizzle in
// two panels of 64 channels, but the state's, which is read as the MN-major A operand (two groups of 64 state
// columns by 128 rows).  MMAs with fewer than 128 valid A rows read past their image, never past the allocation;
// what they read there only reaches accumulator rows that nobody looks at.
template <int MP>
struct Layout {
    static constexpr uint32_t kq_panel = 4 * MP * 128;   // rows: K~ hi, Q~ hi, K~ lo, Q~ lo
    static constexpr uint32_t ki_panel = 2 * MP * 128;   // rows: K^ hi, K^ lo
    static constexpr int ap_stride = MP + 4;             // floats; 16-byte rows on distinct banks
    static constexpr uint32_t ap_bytes = 2 * MP * ap_stride * 4;
    static constexpr uint32_t kq = 0;
    static constexpr uint32_t s_hi = kq + 2 * kq_panel;
    static constexpr uint32_t s_lo = s_hi + 32768;
    static constexpr uint32_t ki = s_lo + 32768;
    static constexpr uint32_t ki_bytes = 2 * ki_panel > ap_bytes ? 2 * ki_panel : (ap_bytes + 1023) / 1024 * 1024;
    static constexpr uint32_t b = ki + ki_bytes;         // fp32 [MP][128]
    static constexpr uint32_t v = b + MP * 512;          // bf16 [MP][128]
    static constexpr uint32_t total = v + MP * 256;
    static constexpr uint32_t ap = ki;                   // fp32 A [MP][ap_stride], then P: once D1 has been formed
    static constexpr uint32_t u = s_hi;                  // fp32 [MP][128], once D2 has been formed
    static constexpr uint32_t o = s_lo;                  // fp32 [MP][128]
    static constexpr uint32_t d2_cols = 4 * MP;
    static constexpr uint32_t tmem_cols = MP == 8 ? 64 : MP == 16 ? 128 : MP == 32 ? 256 : 512;
};

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
        l[i] = pack2(f[2 * i] - __uint_as_float(h[i] << 16), f[2 * i + 1] - __uint_as_float(h[i] & 0xffff0000u));
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}
__device__ __forceinline__ void ldg8(const float *p, float (&f)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                 : "l"(p));
}

struct Args {
    const __nv_bfloat16 *q, *k, *v;
    const float *g, *beta;
    const int32_t *parent, *cu, *seq_idx;
    int H, total_nodes, max_nodes, num_slots;
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

// Forward substitution of one state column (thread) over all nodes, eight at a time: the products with the u of
// earlier blocks, then the block's own triangle.  Masked: entries off the path are skipped instead of
// multiplied by zero, which a non-finite u of another branch would turn into NaN.  Returns false if a u is not
// finite (never in the masked form).
template <int MP, bool Masked>
__device__ __forceinline__ bool substitute(uint8_t *sm, const TreeShared &ts, const float *s_beta, uint32_t d2, int M,
                                           int c) {
    using L = Layout<MP>;
    const float *sA = reinterpret_cast<const float *>(sm + L::ap), *sP = sA + MP * L::ap_stride;
    float *s_u = reinterpret_cast<float *>(sm + L::u), *s_o = reinterpret_cast<float *>(sm + L::o);
    const __nv_bfloat16 *s_v = reinterpret_cast<const __nv_bfloat16 *>(sm + L::v);
    bool finite = true;
    for (int i0 = 0; i0 < M; i0 += 8) {
        float t[4][8], w[8], out[8];
        tc::tmem_ld8x4(d2 + i0, MP, t);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            w[r] = s_beta[i0 + r] * (__bfloat162float(s_v[(i0 + r) * kD + c]) - (t[0][r] + t[2][r]));
            out[r] = t[1][r] + t[3][r];
        }
        for (int a = 0; a < i0; a += 4) {
            float ua[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) ua[e] = s_u[(a + e) * kD + c];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float4 A = *reinterpret_cast<const float4 *>(&sA[(i0 + r) * L::ap_stride + a]);
                const float4 P = *reinterpret_cast<const float4 *>(&sP[(i0 + r) * L::ap_stride + a]);
                const float Av[4] = {A.x, A.y, A.z, A.w}, Pv[4] = {P.x, P.y, P.z, P.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (!Masked || (i0 + r < M && ((ts.anc[i0 + r] >> (a + e)) & 1))) {
                        w[r] = fmaf(-Av[e], ua[e], w[r]);
                        out[r] = fmaf(Pv[e], ua[e], out[r]);
                    }
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            float Av[8], Pv[8];
#pragma unroll
            for (int h = 0; h <= r / 4; ++h) {
                const float4 A = *reinterpret_cast<const float4 *>(&sA[(i0 + r) * L::ap_stride + i0 + 4 * h]);
                const float4 P = *reinterpret_cast<const float4 *>(&sP[(i0 + r) * L::ap_stride + i0 + 4 * h]);
                Av[4 * h] = A.x; Av[4 * h + 1] = A.y; Av[4 * h + 2] = A.z; Av[4 * h + 3] = A.w;
                Pv[4 * h] = P.x; Pv[4 * h + 1] = P.y; Pv[4 * h + 2] = P.z; Pv[4 * h + 3] = P.w;
            }
#pragma unroll
            for (int a = 0; a < r; ++a) {
                if (!Masked || (i0 + r < M && ((ts.anc[i0 + r] >> (i0 + a)) & 1))) {
                    w[r] = fmaf(-Av[a], w[a], w[r]);
                    out[r] = fmaf(Pv[a], w[a], out[r]);
                }
            }
            out[r] = fmaf(Pv[r], w[r], out[r]);
            finite &= i0 + r >= M || fabsf(w[r]) < INFINITY;
            s_u[(i0 + r) * kD + c] = w[r];
            s_o[(i0 + r) * kD + c] = out[r];
        }
    }
    return Masked || finite;
}

template <int MP>
__global__ void __launch_bounds__(kThreads, MP == 64 ? 1 : 2) tree_step_tc_kernel(const Args p) {
    using L = Layout<MP>;
    extern __shared__ uint8_t raw[];
    __shared__ TreeShared ts;
    __shared__ float s_beta[MP], s_scale[2 * MP];
    __shared__ uint64_t bars[2];
    __shared__ uint32_t s_tmem;
    const int n = blockIdx.x / p.H, h = blockIdx.x % p.H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Tree t = tree_rows(p.cu, n, p.total_nodes, p.max_nodes);
    const int slot = slot_of(p.seq_idx, n, p.num_slots);
    if (t.nodes < 0 || slot < 0) {
        if (tid == 0) report_invalid(p.status);
        return;
    }
    if (t.nodes == 0) return;
    const int M = t.nodes;
    uint8_t *sm = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
    const size_t base = ((size_t)t.row0 * p.H + h) * kD, row_stride = (size_t)p.H * kD;

    // All of the CTA's reads, issued at once: g and v on their way to shared memory, k, q and the state in registers.
    for (int i = tid; i < M * 32; i += kThreads)
        tc::cp_async16(sm + L::b + i * 16, p.g + base + (size_t)(i >> 5) * row_stride + (i & 31) * 4);
    for (int i = tid; i < M * 16; i += kThreads)
        tc::cp_async16(sm + L::v + i * 16, p.v + base + (size_t)(i >> 4) * row_stride + (i & 15) * 8);
    constexpr int kUnits = MP * 16 > kThreads ? MP * 16 / kThreads : 1;  // (node, 8 channels) per thread
    uint4 kr[kUnits], qr[kUnits];
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
        const int i = (tid + e * kThreads) >> 4, ch = tid & 15;
        kr[e] = qr[e] = make_uint4(0, 0, 0, 0);
        if (i < M) {
            kr[e] = __ldg(reinterpret_cast<const uint4 *>(p.k + base + (size_t)i * row_stride) + ch);
            qr[e] = __ldg(reinterpret_cast<const uint4 *>(p.q + base + (size_t)i * row_stride) + ch);
        }
    }
    if (tid < MP) s_beta[tid] = tid < M ? p.beta[(size_t)(t.row0 + tid) * p.H + h] : 0.f;
    const float *S = p.S_pool + ((size_t)slot * p.H + h) * kD * kD;
    float s[8][8];  // row (tid / 16) + 16 j, columns 8 (tid % 16) on
#pragma unroll
    for (int j = 0; j < 8; ++j) ldg8(S + (size_t)((tid >> 4) + 16 * j) * kD + (tid & 15) * 8, s[j]);

    if (warp == 0) {
        tc::tmem_alloc(&s_tmem, L::tmem_cols);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        tc::mbar_init(&bars[0], 1);
        tc::mbar_init(&bars[1], 1);
        tc::fence_mbar_init();
    }
    tc::cp_async_wait_all();
    tc::tc_fence_before();
    const bool good = read_tree(ts, p.parent, p.cu, n, p.total_nodes, p.max_nodes, true).nodes > 0;  // a block barrier
    tc::tc_fence_after();
    const uint32_t tmem = s_tmem, d2 = tmem, d1 = tmem + L::d2_cols;
    if (!good) {
        if (tid == 0) report_invalid(p.status);
        if (warp == 0) tc::tmem_dealloc(tmem, L::tmem_cols);
        return;
    }

    // log-decays along the paths, each channel by its own thread, parents before children
    float *s_b = reinterpret_cast<float *>(sm + L::b);
    float range = 0.f;
    if (tid < kD) {
        float b = 0.f;
        for (int i = 0; i < M; ++i) {
            const int par = ts.parent[i];
            b = s_b[i * kD + tid] + (par < 0 ? 0.f : par == i - 1 ? b : s_b[par * kD + tid]);
            s_b[i * kD + tid] = b;
            range = fmaxf(range, fabsf(b));
        }
    }
    const bool pairwise = __syncthreads_or(!(range <= kMaxRange));

    // operand images of K~, Q~ and K^
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
        const int i = (tid + e * kThreads) >> 4, ch = tid & 15;
        if (MP * 16 < kThreads && i >= MP) break;  // warp-uniform
        float kf[8], qf[8], ki[8], b[8];
        unpack8(kr[e], kf);
        unpack8(qr[e], qf);
        if (p.qk_norm) {  // 16 threads hold a row
            float sk = 0.f, sq = 0.f;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                sk = fmaf(kf[x], kf[x], sk);
                sq = fmaf(qf[x], qf[x], sq);
            }
#pragma unroll
            for (int off = 8; off; off >>= 1) {
                sk += __shfl_xor_sync(0xffffffffu, sk, off);
                sq += __shfl_xor_sync(0xffffffffu, sq, off);
            }
            sk = rsqrtf(sk + p.qk_eps);
            sq = rsqrtf(sq + p.qk_eps);
            if (ch == 0) {
                s_scale[i] = sk;
                s_scale[MP + i] = sq;
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                kf[x] *= sk;
                qf[x] *= sq;
            }
        }
        if (i < M) {
            const float4 b0 = *reinterpret_cast<const float4 *>(&s_b[i * kD + ch * 8]);
            const float4 b1 = *reinterpret_cast<const float4 *>(&s_b[i * kD + ch * 8 + 4]);
            b[0] = b0.x; b[1] = b0.y; b[2] = b0.z; b[3] = b0.w;
            b[4] = b1.x; b[5] = b1.y; b[6] = b1.z; b[7] = b1.w;
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            ki[x] = 0.f;
            if (i < M) {
                const float up = expf(b[x]);
                ki[x] = kf[x] * expf(-b[x]);
                kf[x] *= up;
                qf[x] *= up;
            }
        }
        uint4 hi, lo;
        uint8_t *kq = sm + L::kq + (ch >> 3) * L::kq_panel, *kin = sm + L::ki + (ch >> 3) * L::ki_panel;
        const uint32_t at = tc::sw128_offset(i, (ch & 7) * 8);  // the row groups below are multiples of eight rows
        split8(kf, hi, lo);
        *reinterpret_cast<uint4 *>(kq + at) = hi;
        *reinterpret_cast<uint4 *>(kq + 2 * MP * 128 + at) = lo;
        split8(qf, hi, lo);
        *reinterpret_cast<uint4 *>(kq + MP * 128 + at) = hi;
        *reinterpret_cast<uint4 *>(kq + 3 * MP * 128 + at) = lo;
        split8(ki, hi, lo);
        *reinterpret_cast<uint4 *>(kin + at) = hi;
        *reinterpret_cast<uint4 *>(kin + MP * 128 + at) = lo;
    }
    tc::fence_async_smem();
    __syncthreads();
    constexpr uint64_t kKmaj = tc::smem_desc_base(16, 1024, tc::SW_128B);
    constexpr uint64_t kSmn = tc::smem_desc_base(16384, 1024, tc::SW_128B);
    if (tid == 0 && !pairwise) {  // D1: hi x [hi | lo], then lo x [hi | lo]
        constexpr uint32_t id = tc::idesc_bf16_f32(128, 2 * MP, false, false);
        for (int part = 0; part < 2; ++part)
            for (int c = 0; c < 8; ++c) {
                const uint32_t a = tc::smem_u32(sm) + L::kq + (c >> 2) * L::kq_panel + part * 2 * MP * 128 + (c & 3) * 32;
                const uint32_t b = tc::smem_u32(sm) + L::ki + (c >> 2) * L::ki_panel + (c & 3) * 32;
                tc::mma_bf16(d1, tc::smem_desc(kKmaj, a), tc::smem_desc(kKmaj, b), id, part + c > 0);
            }
        tc::mma_commit(&bars[0]);
    }
    // the state's images
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int row = (tid >> 4) + 16 * j, col = (tid & 15) * 8;
        uint4 hi, lo;
        split8(s[j], hi, lo);
        const uint32_t at = (col >> 6) * 16384 + tc::sw128_offset(row, col & 63);
        *reinterpret_cast<uint4 *>(sm + L::s_hi + at) = hi;
        *reinterpret_cast<uint4 *>(sm + L::s_lo + at) = lo;
    }
    tc::fence_async_smem();
    __syncthreads();
    if (tid == 0) {  // D2: S hi x [hi | lo], then S lo x hi
        constexpr uint32_t id4 = tc::idesc_bf16_f32(128, 4 * MP, true, false);
        constexpr uint32_t id2 = tc::idesc_bf16_f32(128, 2 * MP, true, false);
        for (int part = 0; part < 2; ++part)
            for (int c = 0; c < 8; ++c) {
                const uint32_t a = tc::smem_u32(sm) + (part ? L::s_lo : L::s_hi) + c * 2048;
                const uint32_t b = tc::smem_u32(sm) + L::kq + (c >> 2) * L::kq_panel + (c & 3) * 32;
                tc::mma_bf16(d2, tc::smem_desc(kSmn, a), tc::smem_desc(kKmaj, b), part ? id2 : id4, part + c > 0);
            }
        tc::mma_commit(&bars[1]);
    }
    __syncwarp();

    float *sA = reinterpret_cast<float *>(sm + L::ap), *sP = sA + MP * L::ap_stride;
    bool ok = true;
    if (!pairwise) {
        if (warp * 32 < 2 * MP && warp < 4) {  // lanes are the rows of [K~ ; Q~]
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars[0], 0));
            tc::tc_fence_after();
            const int r = warp * 32 + lane, i = r % MP;
            const unsigned long long anc = i < M ? ts.anc[i] : 0ull;
            const bool is_a = r < MP;
            const float scale = is_a ? s_beta[i] : 1.f;
            for (int a0 = 0; a0 < MP; a0 += 8) {
                float x[4][8];  // columns a0 on of the hi part, then of the lo part; the other two runs are not used
                if (ok) tc::tmem_ld8x4(d1 + ((uint32_t)(warp * 32) << 16) + a0, MP == 8 ? 8 : MP, x);
                float val[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int a = a0 + e;
                    val[e] = ((anc >> a) & 1) && !(is_a && a == i) ? scale * (x[0][e] + x[1][e]) : 0.f;
                }
                if (r < 2 * MP) {
                    float4 *dst = reinterpret_cast<float4 *>((is_a ? sA : sP) + i * L::ap_stride + a0);
                    dst[0] = make_float4(val[0], val[1], val[2], val[3]);
                    dst[1] = make_float4(val[4], val[5], val[6], val[7]);
                }
            }
        }
    } else {
        // a warp per (node, ancestor), four channels a lane; K^ is not used, so A and P go over it
        for (int x = warp; x < M * M; x += kThreads / 32) {
            const int i = x / M, a = x % M;
            float sa = 0.f, sp = 0.f;
            if ((ts.anc[i] >> a) & 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = lane + 32 * e;
                    const float ka = __bfloat162float(p.k[base + (size_t)a * row_stride + c]) *
                                     expf(s_b[i * kD + c] - s_b[a * kD + c]);
                    sa = fmaf(__bfloat162float(p.k[base + (size_t)i * row_stride + c]), ka, sa);
                    sp = fmaf(__bfloat162float(p.q[base + (size_t)i * row_stride + c]), ka, sp);
                }
#pragma unroll
                for (int off = 16; off; off >>= 1) {
                    sa += __shfl_xor_sync(0xffffffffu, sa, off);
                    sp += __shfl_xor_sync(0xffffffffu, sp, off);
                }
                if (p.qk_norm) {
                    sa *= s_scale[i] * s_scale[a];
                    sp *= s_scale[MP + i] * s_scale[a];
                }
            }
            if (lane == 0) {
                sA[i * L::ap_stride + a] = a == i ? 0.f : s_beta[i] * sa;
                sP[i * L::ap_stride + a] = sp;
            }
        }
    }
    ok &= __all_sync(0xffffffffu, tc::mbar_wait(&bars[1], 0));
    tc::tc_fence_after();
    ok = __syncthreads_and(ok);  // every wait was met, A and P are complete, and the state's images are free
    if (ok && warp < 4) {
        const uint32_t lanes = d2 + ((uint32_t)(warp * 32) << 16);
        if (!__all_sync(0xffffffffu, substitute<MP, false>(sm, ts, s_beta, lanes, M, tid)))
            substitute<MP, true>(sm, ts, s_beta, lanes, M, tid);
        tc::tc_fence_before();
    }
    __syncthreads();
    if (warp == 0) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, L::tmem_cols);
    }
    if (!ok) {
        if (tid == 0 && p.status) atomicCAS(p.status, 0, (int32_t)KDA_ERR_TIMEOUT);
        return;
    }
    for (int i = warp; i < M; i += kThreads / 32) {
        const size_t at = base + (size_t)i * row_stride + lane * 4;
        if (p.u)
            *reinterpret_cast<float4 *>(p.u + at) = *reinterpret_cast<const float4 *>(sm + L::u + i * 512 + lane * 16);
        float4 x = *reinterpret_cast<const float4 *>(sm + L::o + i * 512 + lane * 16);
        if (p.gate) {
            const uint2 z = __ldg(reinterpret_cast<const uint2 *>(p.gate + at));
            float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
            if (p.weight) w = __ldg(reinterpret_cast<const float4 *>(p.weight) + lane);
            float ss = fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, x.w * x.w)));
#pragma unroll
            for (int off = 16; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float inv = rsqrtf(ss / (float)kD + p.out_eps);
            x.x *= inv * w.x * sigmoidf(__uint_as_float(z.x << 16));
            x.y *= inv * w.y * sigmoidf(__uint_as_float(z.x & 0xffff0000u));
            x.z *= inv * w.z * sigmoidf(__uint_as_float(z.y << 16));
            x.w *= inv * w.w * sigmoidf(__uint_as_float(z.y & 0xffff0000u));
        }
        *reinterpret_cast<uint2 *>(p.o + at) = make_uint2(pack2(x.x, x.y), pack2(x.z, x.w));
    }
}

template <int MP>
cudaError_t launch_mp(const Args &p, int ctas, cudaStream_t st) {
    constexpr int smem = Layout<MP>::total + 1024;
    cudaError_t e =
        cudaFuncSetAttribute(tree_step_tc_kernel<MP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    tree_step_tc_kernel<MP><<<ctas, kThreads, smem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_step_tc(const TreeStepArgs &a, cudaStream_t st) {
    const Args p{(const __nv_bfloat16 *)a.q, (const __nv_bfloat16 *)a.k, (const __nv_bfloat16 *)a.v, a.g, a.beta,
                 a.parent, a.cu, a.seq_idx, a.H, a.total_nodes, a.max_nodes, a.num_slots, a.S_pool,
                 (__nv_bfloat16 *)a.o, a.u, a.status, a.fu.qk_norm, a.fu.qk_eps, (const __nv_bfloat16 *)a.fu.gate,
                 a.fu.weight, a.fu.out_eps};
    const int ctas = a.num_seqs * a.H;
    if (a.max_nodes <= 8) return launch_mp<8>(p, ctas, st);
    if (a.max_nodes <= 16) return launch_mp<16>(p, ctas, st);
    if (a.max_nodes <= 32) return launch_mp<32>(p, ctas, st);
    return launch_mp<64>(p, ctas, st);
}

}  // namespace kda
