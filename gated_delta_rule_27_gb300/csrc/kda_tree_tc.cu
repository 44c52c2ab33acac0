// kda_tree_tc.cu -- the draft-tree step on the Blackwell tensor cores (tcgen05): bf16 inputs, d = 128, trees of 17 to
// 64 nodes.
//
// With b_i the log-decay along the path to node i, K~ = k e^b, Q~ = q e^b and K^ = k e^{-b} (kda_tree.cu has the
// recurrence), one CTA per (request, head) forms, for a tree of at most MP nodes,
//     D1 = [K~ ; Q~] K^^T      A and P: masked to the paths, A scaled by beta
//     D2 = S^T [K~ ; Q~]^T     x and y: the pool's state, 128 columns, times every node's decayed key and query
//     r  = beta (v - x),  T = (I + A)^{-1}
//     D3 = r^T [T - I ; P T]^T   u = r + D3,  o = y + D3     (MP = 64: u first, then o = y + u^T P^T as D4)
// so the state is read once, whatever the tree's size.  The floor is that read, 64 KB per (request, head).
//
// u moves the fp32 state, so one bf16 part (2^-9 of a term) is not enough for it: every operand is split into two, hi +
// lo, 16 bits of the 24, and each product takes hi hi + hi lo + lo hi with fp32 accumulators.  That leaves 3 x 2^-18 of a
// term at most; u is off by 2.4e-7 of its size where fp32 products leave 0.6e-7 (2-norm; states of 0.1.  States of 1 and a
// twentieth of the decay: 3e-6 and 1.5e-7).  A third part
// would close that gap, but its images (32 to 48 KB at MP = 64) do not fit a CTA's shared memory, nor two such CTAs at
// MP = 32.  T comes from fp32 substitutions in blocks of 16 nodes and products of the blocks in the same
// two parts.  A, P and T are done while the state arrives.  Where the decays along a path sum to more than kMaxRange, the
// factors e^b and e^{-b} would leave their range; such a request takes its A and P node by node from the path's own
// exponents instead (16 requests of 33 to 64 nodes: 124 us for 61).
//
// D3 and D4 multiply entries off the paths by zero.  Where an operand is not finite that would carry a NaN from
// one branch into another, so such a request or column takes a substitution that skips them (solve_masked).
//
// What bounds it is the length of one CTA's dependent steps, so CTAs of up to 32 nodes are kept small enough for two to
// share an SM (the state passes through shared memory in two halves of 64 rows, half 1 loading while half 0 is
// multiplied), and a CTA pulls the inputs of the one that will take its place into L2 (without that 233 us for 207 when
// a variant for 16 nodes took 256 requests of 9 to 16, 32 heads).  Above 32 nodes the operands' two bf16 parts take a whole SM's shared memory.
//
// Measured (32 heads): 64 requests of 20 to 32 nodes 88 us, 16 requests of 33 to 64 nodes 62 us, four turns of one CTA
// an SM.  A CTA's time goes in about equal parts to its first reads and the images of K~, Q~ and K^, to the state's
// images with A, P and T (all eight warps; four of them form r meanwhile), and to u, o and their stores.
#include "kda_tree_bf16.cuh"

namespace kda {
namespace {
using namespace tree16;

// Eight worker warps; warp 8 reads the tree and asks for a later CTA's inputs; warp 9 issues the MMAs.
constexpr int kD = 128, kWorkers = 256, kThreads = 320;

// Shared memory for trees of at most MP nodes, in bytes.  Operand images are K-major with the 128-byte swizzle, 64
// elements to a row (keys and queries: two panels of 64 channels), but the state's, which is read as the MN-major
// A operand (two groups of 64 state columns by 64 rows, a half of the state).  MMAs with fewer than 128 valid A rows
// read past their image, never past the allocation; what they read there only reaches accumulator rows that nobody looks at.
template <int MP>
struct Layout {
    static constexpr uint32_t kq_panel = 4 * MP * 128;   // rows: K~ hi, Q~ hi, K~ lo, Q~ lo
    static constexpr uint32_t ki_panel = 2 * MP * 128;   // rows: K^ hi, K^ lo
    static constexpr int ap_stride = MP + 4;             // floats; 16-byte rows on distinct banks
    static constexpr uint32_t ap_bytes = 2 * MP * ap_stride * 4;
    static constexpr uint32_t kq = 0;
    static constexpr uint32_t s_hi = kq + 2 * kq_panel;
    static constexpr uint32_t s_lo = s_hi + 16384;
    static constexpr uint32_t ki = s_lo + 16384;
    static constexpr uint32_t b = ki + 2 * ki_panel;     // fp32 [MP][128]: g, then the paths' sums b
    static constexpr uint32_t ap_tg = MP == 64 ? ap_bytes : 2 * ap_bytes;
    static constexpr uint32_t b_bytes = MP * 512 > ap_tg ? MP * 512 : (ap_tg + 1023) / 1024 * 1024;
    static constexpr uint32_t v = b + b_bytes;           // bf16 [MP][128]
    static constexpr uint32_t w = v + MP * 256;          // fp32 [128]: the output weight
    static constexpr uint32_t tb = w + 512;              // MP = 64: T and the place of a product, below
    static constexpr uint32_t total = MP == 64 ? tb + (64 * ap_stride + 32 * 36) * 4 : tb;
    // later uses of the same bytes
    static constexpr uint32_t t_img = ki;                // rows T - I hi, P T hi, T - I lo, P T lo (MP = 64: T - I hi, lo)
    static constexpr uint32_t p_img = ki + MP * 256;     // MP = 64: P hi, lo   (both once D1 is done)
    static constexpr uint32_t ap = b;                    // fp32 A [MP][ap_stride], then P (once the images are built)
    static constexpr uint32_t tg = MP < 64 ? ap + ap_bytes : tb;  // fp32 T [MP][ap_stride], then P T (MP = 64: a product)
    static constexpr uint32_t r_img = s_hi;              // r: 128 rows hi, 128 rows lo (once D2 is done)
    static constexpr uint32_t u_img = s_hi;              // MP = 64: u, the same way (once D3 is done)
    static constexpr uint32_t z = kq;                    // bf16 [MP][128]: the gate (once D2 is done)
    static constexpr uint32_t o = kq + MP * 256;         // fp32 [MP][128] (once D2 is done)
    // accumulator columns: D2 at 0; D1 and, once it has been read, D3 (then D4) behind it
    static constexpr uint32_t d1 = 4 * MP, d3 = 4 * MP, d4 = 6 * MP;
    static constexpr uint32_t tmem_cols = 8 * MP;
};

// Writes eight consecutive values of an image row, hi at `img` and lo `lo_rows` rows further.
__device__ __forceinline__ void store_split8(uint8_t *img, int row, int col, int lo_rows, const float (&f)[8]) {
    uint4 hi, lo;
    split8(f, hi, lo);
    const uint32_t at = tc::sw128_offset(row, col);
    *reinterpret_cast<uint4 *>(img + at) = hi;
    *reinterpret_cast<uint4 *>(img + lo_rows * 128 + at) = lo;
}
// Eight floats of the state: one 32-byte load where the pool is aligned to that, else two of 16 bytes (all that a pool's
// address promises; 61.1 and 63.9 us for 16 requests of 33 to 64 nodes, 88.7 and 99.0 for 64 of 20 to 32).
__device__ __forceinline__ void ldg8(const float *p, bool aligned32, float (&f)[8]) {
    if (aligned32) {
        asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                     : "l"(p));
    } else {
        asm volatile("ld.global.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%8];\n"
                     "ld.global.L1::no_allocate.v4.f32 {%4,%5,%6,%7}, [%8 + 16];"
                     : "=&f"(f[0]), "=&f"(f[1]), "=&f"(f[2]), "=&f"(f[3]), "=&f"(f[4]), "=&f"(f[5]), "=&f"(f[6]), "=&f"(f[7])
                     : "l"(p));
    }
}
// r of eight nodes for the thread's state column, from the accumulator's hi and lo columns
template <int MP>
__device__ __forceinline__ void residual8(const uint8_t *sm, const float *s_beta, const float (&x_hi)[8],
                                          const float (&x_lo)[8], int i0, int c, float (&r)[8]) {
    const __nv_bfloat16 *s_v = reinterpret_cast<const __nv_bfloat16 *>(sm + Layout<MP>::v);
    float x[8], v[8], beta[8];
    add8(x, x_hi, x_lo);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __bfloat162float(s_v[(i0 + e) * kD + c]);
    read8(s_beta + i0, beta);
    pairs8(r, v, x, [](float2 a, float2 b) { return tc::sub2(a, b); });
    mul8(r, r, beta);
}

// u and o of the thread's state column by forward substitution over the paths' entries only.  u is kept in the
// thread's own two rows of the image of r (or u), whose products are then not used.
template <int MP>
__device__ void solve_masked(uint8_t *sm, const TreeShared &ts, const float *s_beta, uint32_t tmem, int M, int c,
                             float *u_out, size_t row_stride) {
    using L = Layout<MP>;
    const float *sA = reinterpret_cast<const float *>(sm + L::ap), *sP = sA + MP * L::ap_stride;
    auto mine = [&](int a) {
        return reinterpret_cast<float *>(sm + L::r_img + (a >> 5) * 16384 + c * 128 + (a & 31) * 4);
    };
    float *s_o = reinterpret_cast<float *>(sm + L::o);
    for (int i0 = 0; i0 < M; i0 += 8) {
        float t[4][8], r[8];
        tc::tmem_ld8x4(tmem + i0, MP, t);
        residual8<MP>(sm, s_beta, t[0], t[2], i0, c, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = i0 + e;
            if (i < M) {
                float w = r[e], out = t[1][e] + t[3][e];
                for (int a = 0; a < i; ++a) {
                    if ((ts.anc[i] >> a) & 1) {
                        w = fmaf(-sA[i * L::ap_stride + a], *mine(a), w);
                        out = fmaf(sP[i * L::ap_stride + a], *mine(a), out);
                    }
                }
                *mine(i) = w;
                s_o[i * kD + c] = fmaf(sP[i * L::ap_stride + i], w, out);
                if (u_out) u_out[(size_t)i * row_stride] = w;
            }
        }
    }
}

__device__ __forceinline__ void warp_mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack2(x, y);
    lo = pack2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}
// The 16 x 8 tile  sum_{a < K} left[.][a] right[a][.]  of two fp32 matrices in shared memory, in two bf16 parts, as
// T's image will hold it (on the CUDA cores in fp32 the joins took 3 of 65 us, 16 requests of 33 to 64 nodes).
template <int K>
__device__ __forceinline__ void tile_product(const float *left, int ls, const float *right, int rs, float (&c)[4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = (lane & 3) * 2;
    float d[3][4] = {};
#pragma unroll
    for (int k = 0; k < K; k += 16) {
        uint32_t ahi[4], alo[4], bhi[2], blo[2];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float2 x = *reinterpret_cast<const float2 *>(left + (g + 8 * (r & 1)) * ls + k + t + 8 * (r >> 1));
            split2(x.x, x.y, ahi[r], alo[r]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float *y = right + (k + t + 8 * r) * rs + g;
            split2(y[0], y[rs], bhi[r], blo[r]);
        }
        warp_mma(d[0], ahi, bhi);
        warp_mma(d[1], alo, bhi);
        warp_mma(d[2], ahi, blo);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = d[0][e] + d[1][e] + d[2][e];
}
// The blocks below the diagonal of T = (I + A)^{-1}, from those on it:  T21 = -T22 (A21 T11), for each pair of NB x NB
// blocks, a 16 x 8 tile a warp; `tmp` holds the product in brackets, [32][36].
template <int MP, int NB>
__device__ __forceinline__ void join_blocks(const float *A, float *T, float *tmp, int tid) {
    constexpr int kStride = Layout<MP>::ap_stride, kTiles = NB * NB / 128;
    const int warp = tid >> 5, pair = warp / kTiles, i = warp % kTiles / (NB / 8) * 16, j = warp % (NB / 8) * 8;
    const int r = i + ((tid & 31) >> 2), cc = j + (tid & 3) * 2;
    const bool in = pair < MP / (2 * NB);
    const int at = (2 * pair * NB) * (kStride + 1);  // of the pair's first block
    float x[4];
    if (in) {
        tile_product<NB>(A + at + (NB + i) * kStride, kStride, T + at + j, kStride, x);
        float *w = tmp + (pair * NB + r) * 36 + cc;
        w[0] = x[0]; w[1] = x[1]; w[8 * 36] = x[2]; w[8 * 36 + 1] = x[3];
    }
    tc::named_barrier(1, kWorkers);
    if (in) {
        tile_product<NB>(T + at + (NB + i) * kStride + NB, kStride, tmp + pair * NB * 36 + j, 36, x);
        float *w = T + at + (NB + r) * kStride + cc;
        w[0] = -x[0]; w[1] = -x[1]; w[8 * kStride] = -x[2]; w[8 * kStride + 1] = -x[3];
    }
    tc::named_barrier(1, kWorkers);
}

// The MMAs of D = A_hi B^T + A_lo B'^T over MP / 16 slices of 16 elements; B' is the first part of B's rows.
template <int MP, uint32_t IdHi, uint32_t IdLo>
__device__ __forceinline__ void mma_split(uint32_t d, uint32_t a_hi, uint32_t a_lo, uint32_t b, bool elected) {
    constexpr uint64_t kKmaj = tc::smem_desc_base(16, 1024, tc::SW_128B);
#pragma unroll
    for (int c = 0; c < MP / 16; ++c)
        tc::mma_bf16_warp(d, tc::smem_desc(kKmaj, a_hi + c * 32), tc::smem_desc(kKmaj, b + c * 32), IdHi, c > 0, elected);
#pragma unroll
    for (int c = 0; c < MP / 16; ++c)
        tc::mma_bf16_warp(d, tc::smem_desc(kKmaj, a_lo + c * 32), tc::smem_desc(kKmaj, b + c * 32), IdLo, true, elected);
}

// Reads one half of the columns of the rows of D1 that belong to this warp's lanes (row r of [K~ ; Q~]), masks and
// scales them into A and P.
template <int MP>
__device__ __forceinline__ void read_paths(uint8_t *sm, const TreeShared &ts, const float *s_beta, uint32_t tmem, int M,
                                           int row, int half, bool pairwise, int *s_wild) {
    using L = Layout<MP>;
    const bool is_a = row < MP;
    const int i = is_a ? row : row - MP;
    const unsigned long long anc = i < M ? ts.anc[i] : 0ull;
    const float scale = is_a ? s_beta[i] : 1.f;
    float *dst = reinterpret_cast<float *>(sm + L::ap) + ((is_a ? 0 : MP) + i) * L::ap_stride;
    float zero = 0.f;  // NaN once it has met something that is not finite
#pragma unroll 2
    for (int a0 = half * (MP / 2); a0 < (half + 1) * (MP / 2); a0 += 8) {
        float val[8];
        if (!pairwise) {
            float x[2][8];
            tc::tmem_ld8x2(tmem + L::d1 + ((uint32_t)(row & ~31) << 16) + a0, MP, x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                val[e] = ((anc >> (a0 + e)) & 1) && !(is_a && a0 + e == i) ? scale * (x[0][e] + x[1][e]) : 0.f;
            reinterpret_cast<float4 *>(dst + a0)[0] = make_float4(val[0], val[1], val[2], val[3]);
            reinterpret_cast<float4 *>(dst + a0)[1] = make_float4(val[4], val[5], val[6], val[7]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) val[e] = dst[a0 + e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) zero = fmaf(val[e], 0.f, zero);
        if (MP == 64 && !is_a) store_split8(sm + L::p_img, i, a0, MP, val);
    }
    if (zero != 0.f) *s_wild = 1;
}

template <int MP>
__global__ void __launch_bounds__(kThreads, MP == 64 ? 1 : 2) tree_step_tc_kernel(const Args p) {
    using L = Layout<MP>;
    extern __shared__ uint8_t raw[];
    __shared__ TreeShared ts;
    __shared__ __align__(16) float s_beta[MP];
    __shared__ float s_scale[2 * MP];
    __shared__ uint64_t bar_d1, bar_d3, bar_d4, bar_half[2], bar_rows;
    __shared__ uint32_t s_tmem;
    __shared__ int s_wild;    // A, P, T or P T holds something that is not finite
    __shared__ int s_bad[4];  // r does, in the columns of one quarter of the lanes
    tc::grid_dep_wait();
    const int n = blockIdx.x / p.H, h = blockIdx.x % p.H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Tree t = tree_rows(p.cu, n, p.total_nodes, p.max_nodes);
    const int slot = slot_of(p.seq_idx, n, p.num_slots);
    if (t.nodes < 0 || slot < 0) {
        if (tid == 0) report_invalid(p.status);
        return;
    }
    if (t.nodes == 0) return;
    const Links links = load_links(p.parent, t, 8);
    const int M = t.nodes;
    uint8_t *sm = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t sa = tc::smem_u32(sm);
    const size_t base = ((size_t)t.row0 * p.H + h) * kD, row_stride = (size_t)p.H * kD;

    // The CTA's reads, issued at once: g, v, the gate and its weight on their way to shared memory, k, q and half of
    // the state in registers.
    constexpr int kUnits = MP / 16;  // (node, 8 channels) per worker: node (tid / 16) + 16 e, channels 8 (tid % 16) on
    uint4 kr[kUnits], qr[kUnits];
    float s[4][8];                   // state row (tid / 16) + 16 j of the half, columns 8 (tid % 16) on
    const float *S = p.S_pool + ((size_t)slot * p.H + h) * kD * kD + (size_t)(tid >> 4) * kD + (tid & 15) * 8;
    const bool aligned32 = (reinterpret_cast<uintptr_t>(p.S_pool) & 31u) == 0;
    if (warp < 8) {
        for (int i = tid; i < M * 32; i += kWorkers)
            tc::cp_async16(sm + L::b + i * 16, p.g + base + (size_t)(i >> 5) * row_stride + (i & 31) * 4);
#pragma unroll
        for (int e = 0; e < kUnits; ++e) {
            const int i = (tid >> 4) + 16 * e, ch = tid & 15;
            kr[e] = qr[e] = make_uint4(0, 0, 0, 0);
            if (i < M) {
                kr[e] = __ldg(reinterpret_cast<const uint4 *>(p.k + base + (size_t)i * row_stride) + ch);
                qr[e] = __ldg(reinterpret_cast<const uint4 *>(p.q + base + (size_t)i * row_stride) + ch);
            }
        }
        for (int i = tid; i < M * 16; i += kWorkers)
            tc::cp_async16(sm + L::v + i * 16, p.v + base + (size_t)(i >> 4) * row_stride + (i & 15) * 8);
#pragma unroll
        for (int j = 0; j < 4; ++j) ldg8(S + (size_t)(16 * j) * kD, aligned32, s[j]);
        if (p.gate && warp == 0) {
            if (p.weight) tc::cp_async16(sm + L::w + lane * 16, p.weight + lane * 4);
            else *reinterpret_cast<float4 *>(sm + L::w + lane * 16) = make_float4(1.f, 1.f, 1.f, 1.f);
        }
        tc::cp_async_wait_all();
        for (int i = tid; i < M * 32; i += kWorkers) {  // the vectors that this thread copied
            float4 *x = reinterpret_cast<float4 *>(sm + L::b + i * 16);
            *x = log2_decay4(*x);
        }
    } else if (warp == 9) {
        if (lane == 0) tc::bulk_prefetch_l2(p.S_pool + (((size_t)slot * p.H + h) * kD + 64) * kD, 32768);
        tc::tmem_alloc(&s_tmem, L::tmem_cols);
        tc::tmem_relinquish();
        if (lane == 0) {
            tc::mbar_init(&bar_d1, 1);
            tc::mbar_init(&bar_d3, 1);
            tc::mbar_init(&bar_d4, 1);
            tc::mbar_init(&bar_half[0], 1);
            tc::mbar_init(&bar_half[1], 1);
            tc::mbar_init(&bar_rows, 8);
            tc::fence_mbar_init();
            s_wild = 0;
            for (int i = 0; i < 4; ++i) s_bad[i] = 0;
        }
        for (int i = lane; i < MP; i += 32) s_beta[i] = i < M ? p.beta[(size_t)(t.row0 + i) * p.H + h] : 0.f;
        tc::tc_fence_before();
    }
    // Warp 8 looks up the CTA that starts about when this one ends, and asks for its inputs once they will not be in
    // the way of this one's.
    const int later = blockIdx.x + p.ahead;
    Tree lt{0, 0};
    int lslot = -1;
    if (warp == 8 && later < gridDim.x) {
        lt = tree_rows(p.cu, later / p.H, p.total_nodes, p.max_nodes);
        lslot = slot_of(p.seq_idx, later / p.H, p.num_slots);
    }
    const bool good = read_tree(ts, t, links, true, 8);  // a block barrier
    tc::tc_fence_after();
    tc::grid_dep_launch();  // not before this CTA has its tensor memory
    const uint32_t tmem = s_tmem;
    if (!good) {
        if (tid == 0) report_invalid(p.status);
        if (warp == 9) tc::tmem_dealloc(tmem, L::tmem_cols);
        return;
    }
    // Operand images of K~, Q~ and K^.  b sums g over the path, 16 nodes at a time, from the b of the nearest ancestor
    // in an earlier group.
    float *s_b = reinterpret_cast<float *>(sm + L::b);
    float range = 0.f;
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
        const int i = (tid >> 4) + 16 * e, ch = tid & 15;
        float b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (warp < 8 && i < M) {
            const unsigned long long anc = ts.anc[i];
            uint32_t here = (uint32_t)(anc >> (16 * e)) & 0xffffu;
            const unsigned long long before = anc & ((1ull << (16 * e)) - 1);
            if (e > 0 && before) {
                read8(s_b + (63 - __clzll((long long)before)) * kD + ch * 8, b);
            }
            while (here) {
                const int a = 16 * e + __ffs((int)here) - 1;
                here &= here - 1;
                float g[8];
                read8(s_b + a * kD + ch * 8, g);
                add8(b, b, g);
            }
        }
        __syncthreads();  // every sum of this group is formed
        if (warp < 8 && i < M) {
            float4 *x = reinterpret_cast<float4 *>(s_b + i * kD + ch * 8);
            x[0] = make_float4(b[0], b[1], b[2], b[3]);
            x[1] = make_float4(b[4], b[5], b[6], b[7]);
        }
        __syncthreads();
        if (warp < 8 && (warp << 1) + 16 * e < M) {  // what the images hold past the tree is never looked at
            float kf[8], qf[8], ki[8];
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
            float up[8], down[8];
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
            uint8_t *kq = sm + L::kq + (ch >> 3) * L::kq_panel;
            store_split8(kq, i, (ch & 7) * 8, 2 * MP, kf);
            store_split8(kq, MP + i, (ch & 7) * 8, 2 * MP, qf);
            store_split8(sm + L::ki + (ch >> 3) * L::ki_panel, i, (ch & 7) * 8, MP, ki);
        }
    }
    // The state's images, half by half; half 1 is asked for once half 0 is out of the registers (and behind the fence,
    // which waits for the loads before it).
    auto state_images = [&] {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = (tid >> 4) + 16 * j, col = (tid & 15) * 8;
            uint4 hi, lo;
            split8(s[j], hi, lo);
            const uint32_t at = (col >> 6) * 8192 + tc::sw128_offset(row, col & 63);
            *reinterpret_cast<uint4 *>(sm + L::s_hi + at) = hi;
            *reinterpret_cast<uint4 *>(sm + L::s_lo + at) = lo;
        }
        tc::fence_async_smem();
    };
    if (warp < 8) {
        state_images();
#pragma unroll
        for (int j = 0; j < 4; ++j) ldg8(S + (size_t)(64 + 16 * j) * kD, aligned32, s[j]);
    }
    const bool pairwise = __syncthreads_or(!(range <= kMaxRange));
    float *sA = reinterpret_cast<float *>(sm + L::ap), *sP = sA + MP * L::ap_stride;
    if (pairwise) {
        // A warp per node, four neighbouring channels a lane; the results take b's place.  (MP = 32: four ancestors at a
        // time would spill registers of the ordinary case: 92.9 us for 89.4 where 64 requests have 20 to 32 nodes.)
        if (warp < 8) {
            for (int x = tid; x < 2 * MP * L::ap_stride; x += kWorkers) sA[x] = 0.f;
            tc::named_barrier(1, kWorkers);
            for (int i = warp; i < M; i += 8) {
                auto row4 = [&](const __nv_bfloat16 *x, int a, float (&f)[4]) {
                    const uint2 y = __ldg(reinterpret_cast<const uint2 *>(x + base + (size_t)a * row_stride) + lane);
                    f[0] = __uint_as_float(y.x << 16); f[1] = __uint_as_float(y.x & 0xffff0000u);
                    f[2] = __uint_as_float(y.y << 16); f[3] = __uint_as_float(y.y & 0xffff0000u);
                };
                float ki[4], qi[4];
                row4(p.k, i, ki);
                row4(p.q, i, qi);
                pairs_of_node<MP == 64 ? 4 : 2>(ts, i, ki, qi,
                                                [&](int a, float (&ka)[4], float (&ga)[4]) {
                                                    row4(p.k, a, ka);
                                                    const float4 y = log2_decay4(__ldg(reinterpret_cast<const float4 *>(p.g + base + (size_t)a * row_stride) + lane));
                                                    ga[0] = y.x; ga[1] = y.y; ga[2] = y.z; ga[3] = y.w;
                                                },
                                                [](float x) { return exp2_of(x); },
                                                [&](int a, float x, bool is_p) {
                                                    if (p.qk_norm) x *= s_scale[is_p ? MP + i : i] * s_scale[a];
                                                    if (!is_p) x = a == i ? 0.f : s_beta[i] * x;
                                                    (is_p ? sP : sA)[i * L::ap_stride + a] = x;
                                                });
            }
        }
        __syncthreads();
    }

    if (warp == 8 && lslot >= 0 && lt.nodes > 0) {
        const int lh = later % p.H;
        if (lane < 2)
            tc::bulk_prefetch_l2(p.S_pool + (((size_t)lslot * p.H + lh) * kD + 64 * lane) * kD, 32768);
        // the nodes' rows by 128-byte lines: four of g, two each of k, q, v and the gate (one bulk request per row
        // held the warp for 60 clocks each)
        for (int i = lane; i < lt.nodes * 4; i += 32) {
            const size_t at = ((size_t)(lt.row0 + (i >> 2)) * p.H + lh) * kD;
            tc::prefetch_l2(p.g + at + (i & 3) * 32);
            const __nv_bfloat16 *x = i & 2 ? p.k : p.q, *y = i & 2 ? p.v : p.gate;
            tc::prefetch_l2(x + at + (i & 1) * 64);
            if (y) tc::prefetch_l2(y + at + (i & 1) * 64);
        }
    }

    bool ok = true;
    if (warp == 9) {
        constexpr uint64_t kKmaj = tc::smem_desc_base(16, 1024, tc::SW_128B);
        constexpr uint64_t kSmn = tc::smem_desc_base(8192, 1024, tc::SW_128B);
        constexpr uint32_t id1 = tc::idesc_bf16_f32(128, 2 * MP, false, false);
        constexpr uint32_t id4 = tc::idesc_bf16_f32(128, 4 * MP, true, false);
        constexpr uint32_t id2 = tc::idesc_bf16_f32(128, 2 * MP, true, false);
        const bool elected = tc::elect_one();
        if (!pairwise) {  // D1: hi x [hi | lo], then lo x [hi | lo]
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const uint32_t a = sa + L::kq + (c >> 3) * 2 * MP * 128 + ((c >> 2) & 1) * L::kq_panel + (c & 3) * 32;
                const uint32_t b = sa + L::ki + ((c >> 2) & 1) * L::ki_panel + (c & 3) * 32;
                tc::mma_bf16_warp(tmem + L::d1, tc::smem_desc(kKmaj, a), tc::smem_desc(kKmaj, b), id1, c > 0, elected);
            }
            if (elected) tc::mma_commit(&bar_d1);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // D2, half by half, 16 state rows at a time: S hi x [hi | lo] + S lo x hi
            if (c == 4) {
                ok &= __all_sync(0xffffffffu, tc::mbar_wait(&bar_rows, 0));
                tc::tc_fence_after();
            }
            const uint32_t a = (c & 3) * 2048, b = sa + L::kq + (c >> 2) * L::kq_panel + (c & 3) * 32;
            tc::mma_bf16_warp(tmem, tc::smem_desc(kSmn, sa + L::s_hi + a), tc::smem_desc(kKmaj, b), id4, c > 0, elected);
            tc::mma_bf16_warp(tmem, tc::smem_desc(kSmn, sa + L::s_lo + a), tc::smem_desc(kKmaj, b), id2, true, elected);
            if ((c & 3) == 3 && elected) tc::mma_commit(&bar_half[c >> 2]);
        }
        __syncwarp();
    } else if (warp < 8) {
        ok &= __all_sync(0xffffffffu, tc::mbar_wait(&bar_half[0], 0));  // the images' place is free
        state_images();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar_rows);
    }
    float *sT = reinterpret_cast<float *>(sm + L::tg), *tmp = sT + MP * L::ap_stride;
    if (warp < 8) {  // A and P
        if (!pairwise) ok &= __all_sync(0xffffffffu, tc::mbar_wait(&bar_d1, 0));
        tc::tc_fence_after();
        if ((warp & 3) * 32 < 2 * MP) read_paths<MP>(sm, ts, s_beta, tmem, M, (warp & 3) * 32 + lane, warp >> 2, pairwise, &s_wild);
        tc::named_barrier(1, kWorkers);
    }
    if (warp >= 4 && warp < 8) {
        // T's blocks of 16 on the diagonal, one a warp, while the other warps form r
        const int b0 = (warp - 4) * 16;
        if (b0 < MP) {
            float t[16];
            invert_block<16>(sA + b0 * (L::ap_stride + 1), L::ap_stride, lane, t);
            if (lane < 16 || (b0 & 16) == 0) {  // (the zeros beside an upper block are read with it)
#pragma unroll
                for (int i = 0; i < 16; ++i) sT[(b0 + i) * L::ap_stride + b0 + lane] = t[i];
            }
        }
        if (p.gate) {  // the gate, into the place of D2's operands
            ok &= __all_sync(0xffffffffu, tc::mbar_wait(&bar_half[1], 0));
            for (int i = tid - 128; i < M * 16; i += 128)
                tc::cp_async16(sm + L::z + i * 16, p.gate + base + (size_t)(i >> 4) * row_stride + (i & 15) * 8);
        }
    }
    // A thread is a state column from here on.  Four warps form r; for u and o two warps share a quarter of TMEM's
    // lanes and take half of the nodes each.
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int col = tid & (kD - 1), side = warp >> 2;
    constexpr int kHalf = MP / 2;
    if (warp < 4) {  // r, for D3
        ok &= __all_sync(0xffffffffu, tc::mbar_wait(&bar_half[1], 0));
        tc::tc_fence_after();
        float zero = 0.f;
        for (int i0 = 0; i0 < MP; i0 += 8) {
            float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (i0 < M) {
                float x[2][8];
                tc::tmem_ld8x2(lanes + i0, 2 * MP, x);
                residual8<MP>(sm, s_beta, x[0], x[1], i0, col, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    r[e] = i0 + e < M ? r[e] : 0.f;
                    zero = fmaf(r[e], 0.f, zero);
                }
            }
            store_split8(sm + L::r_img, col, i0, 128, r);
        }
        if (zero != 0.f) s_bad[warp & 3] = 1;
    }
    if (warp < 8) {  // the rest of T, and the images that u and o are formed with
        tc::named_barrier(1, kWorkers);
        join_blocks<MP, 16>(sA, sT, tmp, tid);
        if constexpr (MP == 64) {
            join_blocks<MP, 32>(sA, sT, tmp, tid);
        } else {  // P T
            float x[4];
            const int i = (warp >> 2) * 16, j = (warp & 3) * 8;
            tile_product<32>(sP + i * L::ap_stride, L::ap_stride, sT + j, L::ap_stride, x);
            float *to = tmp + (i + (lane >> 2)) * L::ap_stride + j + (lane & 3) * 2;
            to[0] = x[0]; to[1] = x[1]; to[8 * L::ap_stride] = x[2]; to[8 * L::ap_stride + 1] = x[3];
            tc::named_barrier(1, kWorkers);
        }
        float zero = 0.f;
        constexpr int kRows = MP == 64 ? MP : 2 * MP;  // T - I (and P T behind it)
#pragma unroll
        for (int x = tid; x < kRows * (MP / 8); x += kWorkers) {
            const int row = x / (MP / 8), c0 = x % (MP / 8) * 8;
            float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (row >= MP || c0 <= row) read8(sT + row * L::ap_stride + c0, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (c0 + e == row) f[e] = 0.f;
                zero = fmaf(f[e], 0.f, zero);
            }
            store_split8(sm + L::t_img, row, c0, kRows, f);
        }
        if (zero != 0.f) s_wild = 1;
        tc::fence_async_smem();
        tc::tc_fence_before();
    }
    ok = __syncthreads_and(ok);  // every wait so far was met; r, T, P T and P are complete
    constexpr uint32_t id_2mp = tc::idesc_bf16_f32(128, 2 * MP, false, false);
    if (ok && warp == 9) {
        tc::tc_fence_after();
        // MP = 64: columns u hi, u lo; else u hi, o hi, u lo, o lo
        constexpr uint32_t id_hi = MP == 64 ? id_2mp : tc::idesc_bf16_f32(128, 4 * MP, false, false);
        const bool elected = tc::elect_one();
        mma_split<MP, id_hi, id_2mp>(tmem + L::d3, sa + L::r_img, sa + L::r_img + 16384, sa + L::t_img, elected);
        if (elected) tc::mma_commit(&bar_d3);
        __syncwarp();
    }
    const bool masked = s_wild || s_bad[warp & 3];
    float *u_out = p.u ? p.u + base + col : nullptr;
    float *s_o = reinterpret_cast<float *>(sm + L::o);
    if (ok && warp < 8) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&bar_d3, 0));
        tc::tc_fence_after();
        if (masked) {
            if (side == 0) solve_masked<MP>(sm, ts, s_beta, lanes, M, col, u_out, row_stride);
        } else {
            for (int i0 = side * kHalf; i0 < (side + 1) * kHalf; i0 += 8) {
                float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (i0 < M) {
                    if constexpr (MP == 64) {
                        float x[2][8], d[2][8];
                        tc::tmem_ld8x2(lanes + i0, 2 * MP, x);
                        tc::tmem_ld8x2(lanes + L::d3 + i0, MP, d);
                        residual8<MP>(sm, s_beta, x[0], x[1], i0, col, u);
#pragma unroll
                        for (int e = 0; e < 8; ++e) u[e] = i0 + e < M ? u[e] + (d[0][e] + d[1][e]) : 0.f;
                    } else {
                        float x[4][8], d[4][8];
                        tc::tmem_ld8x4(lanes + i0, MP, x);
                        tc::tmem_ld8x4(lanes + L::d3 + i0, MP, d);
                        residual8<MP>(sm, s_beta, x[0], x[2], i0, col, u);
                        float y[8], out[8];
                        add8(out, d[0], d[2]);
                        add8(u, u, out);
                        add8(y, x[1], x[3]);
                        add8(out, d[1], d[3]);
                        add8(out, out, y);
#pragma unroll
                        for (int e = 0; e < 8; ++e) s_o[(i0 + e) * kD + col] = out[e];
                    }
                    if (u_out) {
                        float *out = u_out + (size_t)i0 * row_stride;
#pragma unroll
                        for (int e = 0; e < 8; ++e, out += row_stride)
                            if (i0 + e < M) *out = u[e];
                    }
                }
                if (MP == 64) store_split8(sm + L::u_img, col, i0, 128, u);
            }
        }
        if (MP == 64) tc::fence_async_smem();
        tc::tc_fence_before();
    }
    if (MP == 64) {
        ok = __syncthreads_and(ok);
        if (ok && warp == 9) {
            tc::tc_fence_after();
            const bool elected = tc::elect_one();
            mma_split<MP, id_2mp, id_2mp>(tmem + L::d4, sa + L::u_img, sa + L::u_img + 16384, sa + L::p_img, elected);
            if (elected) tc::mma_commit(&bar_d4);
            __syncwarp();
        }
        if (ok && warp < 8) {
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&bar_d4, 0));
            tc::tc_fence_after();
            for (int i0 = side * kHalf; i0 < min(M, (side + 1) * kHalf) && !masked; i0 += 8) {
                float y[2][8], d[2][8];
                tc::tmem_ld8x2(lanes + MP + i0, 2 * MP, y);
                tc::tmem_ld8x2(lanes + L::d4 + i0, MP, d);
#pragma unroll
                for (int e = 0; e < 8; ++e) s_o[(i0 + e) * kD + col] = (y[0][e] + y[1][e]) + (d[0][e] + d[1][e]);
            }
            tc::tc_fence_before();
        }
    }
    tc::cp_async_wait_all();
    ok = __syncthreads_and(ok);
    if (warp == 9) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, L::tmem_cols);
    }
    if (!ok) {
        if (tid == 0 && p.status) atomicCAS(p.status, 0, (int32_t)KDA_ERR_TIMEOUT);
        return;
    }
    if (warp < 8) {
        const float4 w = *reinterpret_cast<const float4 *>(sm + L::w + lane * 16);
        __nv_bfloat16 *out = p.o + base + (size_t)warp * row_stride + lane * 4;
#pragma unroll 2
        for (int i = warp; i < M; i += 8, out += 8 * row_stride) {
            float4 x = *reinterpret_cast<const float4 *>(sm + L::o + i * 512 + lane * 16);
            if (p.gate) {
                const uint2 z = *reinterpret_cast<const uint2 *>(sm + L::z + i * 256 + lane * 8);
                float ss = fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, x.w * x.w)));
#pragma unroll
                for (int off = 16; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                const float inv = rsqrtf(ss * (1.f / kD) + p.out_eps);
                x.x *= inv * w.x * gate_of(__uint_as_float(z.x << 16));
                x.y *= inv * w.y * gate_of(__uint_as_float(z.x & 0xffff0000u));
                x.z *= inv * w.z * gate_of(__uint_as_float(z.y << 16));
                x.w *= inv * w.w * gate_of(__uint_as_float(z.y & 0xffff0000u));
            }
            *reinterpret_cast<uint2 *>(out) = make_uint2(pack2(x.x, x.y), pack2(x.z, x.w));
        }
    }
}

template <int MP>
cudaError_t launch_mp(Args p, int ctas, cudaStream_t st) {
    constexpr int smem = Layout<MP>::total + 1024;
    int sms = 0;
    cudaError_t e = allow_smem<tree_step_tc_kernel<MP>>(smem);
    if (e == cudaSuccess) e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    p.ahead = sms * (MP == 64 ? 1 : 2);  // the CTAs that run at once
    return launch_dependent(tree_step_tc_kernel<MP>, ctas, kThreads, smem, st, p);
}

}  // namespace

cudaError_t launch_tree_step_tc(const TreeStepArgs &a, cudaStream_t st) {
    const Args p{(const __nv_bfloat16 *)a.q, (const __nv_bfloat16 *)a.k, (const __nv_bfloat16 *)a.v, a.g, a.beta,
                 a.parent, a.cu, a.seq_idx, a.H, a.total_nodes, a.max_nodes, a.num_slots, 0, a.S_pool,
                 (__nv_bfloat16 *)a.o, a.u, a.status, a.fu.qk_norm, a.fu.qk_eps, (const __nv_bfloat16 *)a.fu.gate,
                 a.fu.weight, a.fu.out_eps};
    const int ctas = a.num_seqs * a.H;
    return a.max_nodes <= 32 ? launch_mp<32>(p, ctas, st) : launch_mp<64>(p, ctas, st);
}

}  // namespace kda
