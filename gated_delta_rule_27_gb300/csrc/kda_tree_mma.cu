// kda_tree_mma.cu -- the draft-tree step with the state in registers: bf16 inputs, d = 128, trees of up to 16 nodes.
//
// The mathematics is that of kda_tree_tc.cu: with K~ = k e^b, Q~ = q e^b, K^ = k e^{-b},
//     A, P = [K~ ; Q~] K^^T (masked to the paths),   X^T, Y^T = S^T [K~ ; Q~]^T,
//     R = beta (V - X),   U^T = R^T + R^T (T - I)^T with T = (I + A)^{-1},   O^T = Y^T + U^T P^T.
// Small trees leave each state element a few multiply-adds; what bounds the step is the state's way to the tensor
// core.  Here a warp owns 32 state columns and loads them as the MMA's A fragments: a lane's float4 of four
// neighbouring columns is four rows of two 16-column tiles, and state rows 2t, 2t + 1 pair up as bf16.  X and Y come out as
// fragments that are R's and U's A operands as they are,
// and from the state's load to the stores of u and o a warp waits for no other but for T and the norm of o.
// (The legacy MMA is the right one here: 16 nodes take 1728 clocks of it per head, below the 4000 in which the
// SM's share of HBM delivers the head's state; through tcgen05 the operand's conversion and staging took longer
// than the products.)  Each warp's rows come through a ring of its own in shared memory: loaded straight to
// registers, the lanes of a fragment read four rows that lie on the same banks of L1, 16 data cycles a load for 4,
// and the L1 data pipe was what bounded the step.
//
// Every operand is taken in two bf16 parts as there, hi hi + hi lo + lo hi with fp32 sums: u is off by 3e-7 of its size
// where fp32 products leave 0.5e-7 (2-norm; states of 0.1.  States of 1 and a twentieth of the decay: 3e-6 and 1.6e-7).
//
// Measured (32 heads, 9 to 16 nodes): 64 requests 46 us, 256 requests 162 us where the bytes' way takes 114.  Issue slots
// are 48% busy, the tensor pipe 33%, DRAM 59%: with four CTAs an SM the phases that load (the state) and those that only
// compute (the decays, A, P, T, the stores) overlap in part.
#include "kda_tree_bf16.cuh"

namespace kda {
namespace {
using namespace tree16;

constexpr int kD = 128, kThreads = 128, kWarps = 4;

// Shared memory for trees of at most MP nodes, in bytes.  A fragment tile holds eight nodes (rows of K~, then Q~,
// then K^) by 16 channels: for lane l the bf16 pairs of node l / 4, channels 2 (l % 4) on and 8 further, hi parts
// then lo parts.  It is a B operand, and two of them, for 16 nodes, an A operand.
template <int MP>
struct Layout {
    static constexpr int tiles = MP / 8;
    static constexpr uint32_t frag_bytes = 528;          // 32 lanes x 16 bytes, and 16 against bank conflicts
    static constexpr int ap_stride = MP + 4;
    static constexpr uint32_t ap_bytes = 2 * MP * ap_stride * 4;
    static constexpr uint32_t frag = 0;
    static constexpr uint32_t inv = frag + 2 * tiles * 8 * frag_bytes;  // K^'s tiles
    static constexpr uint32_t b = inv + tiles * 8 * frag_bytes;         // fp32 [MP][128]: g
    static constexpr uint32_t b_bytes = MP * 512;
    static_assert(ap_bytes <= b_bytes, "A and P take the place of g");
    static constexpr int stages = MP == 8 ? 3 : 2;       // (six CTAs fit an SM; MP = 16: four)
    static constexpr uint32_t ring = b + b_bytes;        // per warp `stages` x 16 rows of its 32 columns
    static constexpr uint32_t total = ring + kWarps * stages * 2048;
    // later uses of the same bytes
    static constexpr uint32_t ap = b;                    // fp32 A [MP][ap_stride], then P (once the tiles are built)
    static constexpr uint32_t t = inv;                   // fp32 T - I [MP][ap_stride] (once A and P are formed)
    static constexpr uint32_t x = frag;                  // the masked solve's r, then y: fp32 [MP][128] each
};

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c += hi hi + lo hi + hi lo; b: {hi, hi, lo, lo}
__device__ __forceinline__ void mma_split(float (&c)[4], const uint32_t (&hi)[4], const uint32_t (&lo)[4], const uint4 &b) {
    mma(c, hi, b.x, b.y);
    mma(c, lo, b.x, b.y);
    mma(c, hi, b.z, b.w);
}
// A pair of values as bf16 pairs, hi and lo.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack2(x, y);
    const float2 rest = tc::sub2(make_float2(x, y), make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)));
    lo = pack2(rest.x, rest.y);
}
__device__ __forceinline__ float4 four(uint2 x) {  // of bf16
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                       __uint_as_float(x.y & 0xffff0000u));
}

// Place of the 16-byte vector u of a row of g or b: a thread's two vectors (eight channels) lie half a row apart, so
// that 16 threads read a row without bank conflicts.
__device__ __forceinline__ int spread(int u) { return (u & 1) * 16 + (u >> 1); }
__device__ __forceinline__ void read_row8(const float *row, int ch, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(row)[ch], b = reinterpret_cast<const float4 *>(row)[16 + ch];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Writes eight channels (chunk ch of 16) of node i to its fragment tile.
template <int MP>
__device__ __forceinline__ void store_frag(uint8_t *tiles, int i, int ch, const float (&f)[8]) {
    uint8_t *at = tiles + ((i >> 3) * 8 + (ch >> 1)) * Layout<MP>::frag_bytes + (i & 7) * 64 + (ch & 1) * 4;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        uint32_t hi, lo;
        split2(f[2 * t], f[2 * t + 1], hi, lo);
        *reinterpret_cast<uint32_t *>(at + t * 16) = hi;
        *reinterpret_cast<uint32_t *>(at + t * 16 + 8) = lo;
    }
}
template <int MP>
__device__ __forceinline__ uint4 load_frag(const uint8_t *tiles, int tile, int step) {
    return *reinterpret_cast<const uint4 *>(tiles + (tile * 8 + step) * Layout<MP>::frag_bytes + (threadIdx.x & 31) * 16);
}

// The fragments c of a product over nodes, as the A operand of the next: node tiles 2 s and 2 s + 1.
template <int NT>
__device__ __forceinline__ void as_operand(const float (&c)[NT][4], int s, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split2(c[2 * s][0], c[2 * s][1], hi[0], lo[0]);
    split2(c[2 * s][2], c[2 * s][3], hi[1], lo[1]);
    if (2 * s + 1 < NT) {
        split2(c[(2 * s + 1) % NT][0], c[(2 * s + 1) % NT][1], hi[2], lo[2]);
        split2(c[(2 * s + 1) % NT][2], c[(2 * s + 1) % NT][3], hi[3], lo[3]);
    } else {
        hi[2] = hi[3] = lo[2] = lo[3] = 0u;
    }
}
// c[m][n] += A[m] M^T over the nodes, M a lower triangular fp32 matrix in shared memory.
template <int NT>
__device__ __forceinline__ void times_transposed(float (&c)[2][NT][4], const float (&a)[2][NT][4], const float *M, int stride) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
    for (int s = 0; s < (NT + 1) / 2; ++s) {
        uint32_t hi[2][4], lo[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) as_operand<NT>(a[m], s, hi[m], lo[m]);
#pragma unroll
        for (int n = 2 * s; n < NT; ++n) {
            const float *at = M + (n * 8 + g) * stride + 16 * s + 2 * t;
            const float2 x = *reinterpret_cast<const float2 *>(at);
            uint4 b;
            split2(x.x, x.y, b.x, b.z);
            b.y = b.w = 0u;
            if (2 * s + 1 < NT) {
                const float2 y = *reinterpret_cast<const float2 *>(at + 8);
                split2(y.x, y.y, b.y, b.w);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) mma_split(c[m][n], hi[m], lo[m], b);
        }
    }
}

// u and o of one state column by forward substitution over the paths' entries only (r and y in shared memory; u
// goes back to r's place, o to y's).
template <int MP>
__device__ void solve_masked(uint8_t *sm, const TreeShared &ts, int M, int c) {
    using L = Layout<MP>;
    const float *sA = reinterpret_cast<const float *>(sm + L::ap), *sP = sA + MP * L::ap_stride;
    float *r = reinterpret_cast<float *>(sm + L::x), *y = r + MP * kD;
    for (int i = 0; i < M; ++i) {
        float w = r[i * kD + c], out = y[i * kD + c];
        for (int a = 0; a < i; ++a) {
            if ((ts.anc[i] >> a) & 1) {
                w = fmaf(-sA[i * L::ap_stride + a], r[a * kD + c], w);
                out = fmaf(sP[i * L::ap_stride + a], r[a * kD + c], out);
            }
        }
        r[i * kD + c] = w;
        y[i * kD + c] = fmaf(sP[i * L::ap_stride + i], w, out);
    }
}

template <int MP>
__global__ void __launch_bounds__(kThreads, MP == 8 ? 6 : 4) tree_step_mma_kernel(const Args p) {
    using L = Layout<MP>;
    constexpr int NT = MP / 8, kStages = L::stages;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ TreeShared ts;
    __shared__ __align__(16) float s_beta[MP];
    __shared__ float s_scale[2 * MP], s_square[kWarps][MP];
    __shared__ int s_wild;  // A, P or T holds something that is not finite
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int n = blockIdx.x / p.H, h = blockIdx.x % p.H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    const Tree t = tree_rows(p.cu, n, p.total_nodes, p.max_nodes);
    const int slot = slot_of(p.seq_idx, n, p.num_slots);
    if (t.nodes < 0 || slot < 0) {
        if (tid == 0) report_invalid(p.status);
        return;
    }
    if (t.nodes == 0) return;
    const Links links = load_links(p.parent, t);
    const int M = t.nodes;
    const size_t base = ((size_t)t.row0 * p.H + h) * kD, row_stride = (size_t)p.H * kD;

    // The CTA's first reads, issued at once: g on its way to shared memory, k and q to registers, the first rows of
    // the warp's state columns to its ring.
    constexpr int kUnits = MP / 8;  // (node, 8 channels) per thread: node (tid / 16) + 8 e, channels 8 (tid % 16) on
    uint4 kr[kUnits], qr[kUnits];
    for (int i = tid; i < M * 32; i += kThreads)
        tc::cp_async16(sm + L::b + ((i & ~31) + spread(i & 31)) * 16, p.g + base + (size_t)(i >> 5) * row_stride + (i & 31) * 4);
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
        const int i = (tid >> 4) + 8 * e;
        kr[e] = qr[e] = make_uint4(0, 0, 0, 0);
        if (i < M) {
            kr[e] = __ldg(reinterpret_cast<const uint4 *>(p.k + base + (size_t)i * row_stride) + (tid & 15));
            qr[e] = __ldg(reinterpret_cast<const uint4 *>(p.q + base + (size_t)i * row_stride) + (tid & 15));
        }
    }
    tc::cp_async_commit();
    // Step ks of 16 state rows: eight lanes copy a row's 128 bytes (16-byte vectors XORed with the row's number), four
    // rows at once.
    const float *S = p.S_pool + ((size_t)slot * p.H + h) * kD * kD + (size_t)(lane >> 3) * kD + warp * 32 + (lane & 7) * 4;
    uint8_t *ring = sm + L::ring + warp * kStages * 2048;
    auto load_state = [&](int ks) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 4 * j + (lane >> 3);
            tc::cp_async16(ring + (ks % kStages) * 2048 + row * 128 + (((lane & 7) ^ row) & 7) * 16, S + (size_t)(16 * ks + 4 * j) * kD);
        }
        tc::cp_async_commit();
    };
#pragma unroll
    for (int ks = 0; ks < kStages; ++ks) load_state(ks);
    if (warp == 2) {
        for (int i = lane; i < MP; i += 32) s_beta[i] = i < M ? p.beta[(size_t)(t.row0 + i) * p.H + h] : 0.f;
        if (lane == 0) s_wild = 0;
    }
    tc::cp_async_wait<kStages>();
    for (int i = tid; i < M * 32; i += kThreads) {  // the vectors that this thread copied
        float4 *x = reinterpret_cast<float4 *>(sm + L::b + ((i & ~31) + spread(i & 31)) * 16);
        *x = log2_decay4(*x);
    }
    if (!read_tree(ts, t, links, true)) {  // a block barrier
        tc::cp_async_wait_all();
        if (tid == 0) report_invalid(p.status);
        return;
    }

    // Fragment tiles of K~, Q~ and K^; b sums g over the path.
    float *s_b = reinterpret_cast<float *>(sm + L::b);
    float range = 0.f;
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
        const int i = (tid >> 4) + 8 * e, ch = tid & 15;
        if ((warp << 1) + 8 * e >= M) break;  // (of the warp's two nodes; what the tiles hold past the tree is not looked at)
        float b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (uint32_t here = i < M ? (uint32_t)ts.anc[i] : 0u; here; here &= here - 1) {
            float x[8];
            read_row8(s_b + (__ffs((int)here) - 1) * kD, ch, x);
            add8(b, b, x);
        }
        float kf[8], qf[8], ki[8], up[8], down[8];
        unpack8(kr[e], kf);
        unpack8(qr[e], qf);
        float sk = 1.f, sq = 1.f;
        if (p.qk_norm) {  // 16 threads hold a row
            sk = sum_squares8(kf);
            sq = sum_squares8(qf);
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
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            up[x] = exp2_of(b[x]);
            down[x] = exp2_of(-b[x]);  // used while b is within +-kMaxRange
            range = fmaxf(range, fabsf(b[x]));
        }
        scale8(kf, kf, sk);
        scale8(qf, qf, sq);
        mul8(ki, kf, down);
        mul8(kf, kf, up);
        mul8(qf, qf, up);
        store_frag<MP>(sm + L::frag, i, ch, kf);
        store_frag<MP>(sm + L::frag + NT * 8 * L::frag_bytes, i, ch, qf);
        store_frag<MP>(sm + L::inv, i, ch, ki);
    }
    const bool pairwise = __syncthreads_or(!(range <= kMaxRange));

    float *sA = reinterpret_cast<float *>(sm + L::ap), *sP = sA + MP * L::ap_stride;
    if (pairwise) {
        // A warp per node, four neighbouring channels a lane.  The results' own place holds g, so they pass through the
        // place of K^, which is not used.
        float *xA = reinterpret_cast<float *>(sm + L::inv);
        static_assert(2 * MP * MP * 4 <= NT * 8 * L::frag_bytes, "A and P pass through the place of K^");
        for (int x = tid; x < 2 * MP * MP; x += kThreads) xA[x] = 0.f;
        __syncthreads();
        for (int i = warp; i < M; i += kWarps) {
            auto row4 = [&](const __nv_bfloat16 *x, int a, float (&f)[4]) {
                const float4 y = four(__ldg(reinterpret_cast<const uint2 *>(x + base + (size_t)a * row_stride) + lane));
                f[0] = y.x; f[1] = y.y; f[2] = y.z; f[3] = y.w;
            };
            float ki[4], qi[4];
            row4(p.k, i, ki);
            row4(p.q, i, qi);
            pairs_of_node<4>(ts, i, ki, qi,
                             [&](int a, float (&ka)[4], float (&ga)[4]) {
                                 row4(p.k, a, ka);
                                 const float4 y = reinterpret_cast<const float4 *>(s_b + a * kD)[spread(lane)];
                                 ga[0] = y.x; ga[1] = y.y; ga[2] = y.z; ga[3] = y.w;
                             },
                             [](float x) { return exp2_of(x); },
                             [&](int a, float x, bool is_p) {
                                 if (p.qk_norm) x *= s_scale[is_p ? MP + i : i] * s_scale[a];
                                 if (!is_p) x = a == i ? 0.f : s_beta[i] * x;
                                 xA[(is_p ? MP * MP : 0) + i * MP + a] = x;
                                 if (x * 0.f != 0.f) s_wild = 1;
                             });
        }
        __syncthreads();
        for (int x = tid; x < 2 * MP * MP; x += kThreads) sA[x / MP * L::ap_stride + x % MP] = xA[x];
    } else {
        // 16 rows of [K~ ; Q~] by eight nodes a warp and turn (MP = 8: the rows of K~ and Q~ in one)
        constexpr int kRowTiles = MP == 8 ? 1 : 2 * NT / 2;
        float zero = 0.f;
        for (int task = warp; task < kRowTiles * NT; task += kWarps) {
            const int m = task / NT, nt = task % NT;  // rows 16 m on of [K~ ; Q~], ancestors 8 nt on
            float c[3][4] = {};
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint4 lo_rows = load_frag<MP>(sm + L::frag, 2 * m, ks), hi_rows = load_frag<MP>(sm + L::frag, 2 * m + 1, ks);
                const uint4 b = load_frag<MP>(sm + L::inv, nt, ks);
                const uint32_t hi[4] = {lo_rows.x, hi_rows.x, lo_rows.y, hi_rows.y}, lo[4] = {lo_rows.z, hi_rows.z, lo_rows.w, hi_rows.w};
                mma(c[0], hi, b.x, b.y);
                mma(c[1], lo, b.x, b.y);
                mma(c[2], hi, b.z, b.w);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 16 * m + g + 8 * e, i = row % MP, a = 8 * nt + 2 * t4;
                const bool is_a = row < MP;
                const unsigned long long anc = i < M ? ts.anc[i] : 0ull;
                const float scale = is_a ? s_beta[i] : 1.f;
                float2 val;
                val.x = (anc >> a) & 1 && !(is_a && a == i) ? scale * (c[0][2 * e] + c[1][2 * e] + c[2][2 * e]) : 0.f;
                val.y = (anc >> (a + 1)) & 1 && !(is_a && a + 1 == i) ? scale * (c[0][2 * e + 1] + c[1][2 * e + 1] + c[2][2 * e + 1]) : 0.f;
                zero = fmaf(val.x, 0.f, fmaf(val.y, 0.f, zero));
                *reinterpret_cast<float2 *>((is_a ? sA : sP) + i * L::ap_stride + a) = val;
            }
        }
        if (zero != 0.f) s_wild = 1;
    }
    __syncthreads();  // A and P are complete, and K^ is no longer needed
    if (warp == 0) {  // T - I
        // the blocks of eight on the diagonal, a column a lane, then (MP = 16) the one below it, T21 = -T22 (A21 T11)
        constexpr int kS = L::ap_stride;
        float *sT = reinterpret_cast<float *>(sm + L::t);
        const int block = MP == 8 ? 0 : lane & 8, c = lane & 7;
        float t[8], zero = 0.f;
        invert_block<8>(sA + block * (kS + 1), kS, c, t);
        if (lane < MP) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                zero = fmaf(t[i], 0.f, zero);
                sT[(block + i) * kS + block + c] = MP == 8 && i == c ? 0.f : t[i];
            }
        } else if (MP == 16 && block == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sT[i * kS + 8 + c] = 0.f;
        }
        if constexpr (MP == 16) {
            const int r = 8 + g, j = 2 * t4;  // two entries of T21 a lane
            float2 *w = reinterpret_cast<float2 *>(sT + r * kS + j);
            auto row_times = [&](const float *left, const float *right) {
                float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                for (int a = 0; a < 8; ++a)
                    acc = tc::fma2(make_float2(left[a], left[a]), *reinterpret_cast<const float2 *>(right + a * kS), acc);
                return acc;
            };
            __syncwarp();
            const float2 x = row_times(sA + r * kS, sT + j);
            *w = x;
            __syncwarp();
            const float2 y = row_times(sT + r * kS + 8, sT + 8 * kS + j);
            __syncwarp();
            *w = make_float2(-y.x, -y.y);
            if (lane < MP) sT[lane * (kS + 1)] = 0.f;
            zero = fmaf(y.x, 0.f, fmaf(y.y, 0.f, zero));
        }
        if (zero != 0.f) s_wild = 1;
    }

    // X^T and Y^T of the warp's 32 columns, 16 state rows at a time.  Of node tile j a lane holds nodes
    // 8 j + 2 t4 + {0, 1}, four neighbouring columns of each; their v and gate are asked for now
    // (at their use they cost 12% of the step).
    const int col = warp * 32 + g * 4;
    uint2 vr[NT][2], zr[NT][2];
    float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
    if (p.gate && p.weight) w = __ldg(reinterpret_cast<const float4 *>(p.weight + col));
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 8 * j + 2 * t4 + e;
            vr[j][e] = zr[j][e] = make_uint2(0u, 0u);
            if (i < M) {
                vr[j][e] = __ldg(reinterpret_cast<const uint2 *>(p.v + base + (size_t)i * row_stride + col));
                if (p.gate) zr[j][e] = __ldg(reinterpret_cast<const uint2 *>(p.gate + base + (size_t)i * row_stride + col));
            }
        }
    float x[2][NT][4], y[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[m][j][e] = y[m][j][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        // tile m holds the lane's columns 2 m (rows g of the tile) and 2 m + 1 (rows g + 8)
        uint32_t hi[2][4], lo[2][4];
        // the lane's rows 2 t, 2 t + 1 and 8 further, columns 4 g on of the warp's 32
        if (ks + kStages <= 8) tc::cp_async_wait<kStages - 1>();
        else if (ks == 8 - kStages + 1) tc::cp_async_wait_all();
        __syncwarp();
        float4 r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 2 * t4 + (j & 1) + 8 * (j >> 1);
            r[j] = *reinterpret_cast<const float4 *>(ring + (ks % kStages) * 2048 + row * 128 + ((g ^ row) & 7) * 16);
        }
        __syncwarp();
        if (ks + kStages < 8) load_state(ks + kStages);
#pragma unroll
        for (int k8 = 0; k8 < 2; ++k8) {
            split2(r[2 * k8].x, r[2 * k8 + 1].x, hi[0][2 * k8], lo[0][2 * k8]);
            split2(r[2 * k8].y, r[2 * k8 + 1].y, hi[0][2 * k8 + 1], lo[0][2 * k8 + 1]);
            split2(r[2 * k8].z, r[2 * k8 + 1].z, hi[1][2 * k8], lo[1][2 * k8]);
            split2(r[2 * k8].w, r[2 * k8 + 1].w, hi[1][2 * k8 + 1], lo[1][2 * k8 + 1]);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (MP > 8 && 8 * j >= M) break;
            const uint4 bk = load_frag<MP>(sm + L::frag, j, ks), bq = load_frag<MP>(sm + L::frag, NT + j, ks);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                mma_split(x[m][j], hi[m], lo[m], bk);
                mma_split(y[m][j], hi[m], lo[m], bq);
            }
        }
    }
    // R
    float zero = 0.f;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 8 * j + 2 * t4 + e;
            const float4 v = four(vr[j][e]);
            const float beta = s_beta[i];
            const bool in = i < M;
            x[0][j][e] = in ? beta * (v.x - x[0][j][e]) : 0.f;
            x[0][j][2 + e] = in ? beta * (v.y - x[0][j][2 + e]) : 0.f;
            x[1][j][e] = in ? beta * (v.z - x[1][j][e]) : 0.f;
            x[1][j][2 + e] = in ? beta * (v.w - x[1][j][2 + e]) : 0.f;
            zero = fmaf(x[0][j][e], 0.f, fmaf(x[0][j][2 + e], 0.f, zero));
            zero = fmaf(x[1][j][e], 0.f, fmaf(x[1][j][2 + e], 0.f, zero));
        }
    if (zero != 0.f) s_wild = 1;
    __syncthreads();  // T is complete
    if (!s_wild) {
        float u[2][NT][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) u[m][j][e] = x[m][j][e];
        times_transposed<NT>(u, x, reinterpret_cast<const float *>(sm + L::t), L::ap_stride);
        if (p.u) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 8 * j + 2 * t4 + e;
                    if (i < M)
                        *reinterpret_cast<float4 *>(p.u + base + (size_t)i * row_stride + col) =
                            make_float4(u[0][j][e], u[0][j][2 + e], u[1][j][e], u[1][j][2 + e]);
                }
        }
        times_transposed<NT>(y, u, sP, L::ap_stride);
    } else {
        float *sr = reinterpret_cast<float *>(sm + L::x), *sy = sr + MP * kD;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 8 * j + 2 * t4 + e;
                *reinterpret_cast<float4 *>(sr + i * kD + col) = make_float4(x[0][j][e], x[0][j][2 + e], x[1][j][e], x[1][j][2 + e]);
                *reinterpret_cast<float4 *>(sy + i * kD + col) = make_float4(y[0][j][e], y[0][j][2 + e], y[1][j][e], y[1][j][2 + e]);
            }
        __syncthreads();
        solve_masked<MP>(sm, ts, M, tid);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 8 * j + 2 * t4 + e;
                const float4 o = *reinterpret_cast<const float4 *>(sy + i * kD + col);
                y[0][j][e] = o.x; y[0][j][2 + e] = o.y; y[1][j][e] = o.z; y[1][j][2 + e] = o.w;
                if (p.u && i < M)
                    *reinterpret_cast<float4 *>(p.u + base + (size_t)i * row_stride + col) = *reinterpret_cast<const float4 *>(sr + i * kD + col);
            }
    }
    if (p.gate) {  // the rows' squares: this lane's columns, the warp's, all
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float ss = fmaf(y[0][j][e], y[0][j][e], fmaf(y[0][j][2 + e], y[0][j][2 + e],
                                                             fmaf(y[1][j][e], y[1][j][e], y[1][j][2 + e] * y[1][j][2 + e])));
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                if (g == 0) s_square[warp][8 * j + 2 * t4 + e] = ss;
            }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 8 * j + 2 * t4 + e;
            if (i >= M) continue;
            float4 o = make_float4(y[0][j][e], y[0][j][2 + e], y[1][j][e], y[1][j][2 + e]);
            if (p.gate) {
                const float4 z = four(zr[j][e]);
                const float ss = (s_square[0][i] + s_square[1][i]) + (s_square[2][i] + s_square[3][i]);
                const float inv = rsqrtf(ss * (1.f / kD) + p.out_eps);
                o.x *= inv * w.x * gate_of(z.x);
                o.y *= inv * w.y * gate_of(z.y);
                o.z *= inv * w.z * gate_of(z.z);
                o.w *= inv * w.w * gate_of(z.w);
            }
            *reinterpret_cast<uint2 *>(p.o + base + (size_t)i * row_stride + col) = make_uint2(pack2(o.x, o.y), pack2(o.z, o.w));
        }
}

template <int MP>
cudaError_t launch_mp(const Args &p, int ctas, cudaStream_t st) {
    constexpr int smem = Layout<MP>::total;
    const cudaError_t e = allow_smem<tree_step_mma_kernel<MP>>(smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(tree_step_mma_kernel<MP>, ctas, kThreads, smem, st, p);
}

}  // namespace

cudaError_t launch_tree_step_mma(const TreeStepArgs &a, cudaStream_t st) {
    const Args p{(const __nv_bfloat16 *)a.q, (const __nv_bfloat16 *)a.k, (const __nv_bfloat16 *)a.v, a.g, a.beta,
                 a.parent, a.cu, a.seq_idx, a.H, a.total_nodes, a.max_nodes, a.num_slots, 0, a.S_pool,
                 (__nv_bfloat16 *)a.o, a.u, a.status, a.fu.qk_norm, a.fu.qk_eps, (const __nv_bfloat16 *)a.fu.gate,
                 a.fu.weight, a.fu.out_eps};
    const int ctas = a.num_seqs * a.H;
    return a.max_nodes <= 8 ? launch_mp<8>(p, ctas, st) : launch_mp<16>(p, ctas, st);
}

}  // namespace kda
