// kda_linear_tc.cu -- chunked linear attention on the tensor cores: bf16, d = 128.
//
// A document is walked in chunks of 64 tokens.  With S the state before a chunk and b, w the chunk's decays,
//     P_ij = 2^(b_i - b_j) (q_i . k_j)        (j <= i, else 0)
//     O^T  = 2^(b_i) S^T Q^T + V^T P^T
//     S^T <- 2^(b_64) S^T + V'^T K,           V'_j = 2^(b_64 - b_j) v_j
// so each product has 128 rows (the value dimension) or the chunk's 64 tokens.  S^T stays in the registers of one warpgroup
// for a whole segment: the tensor core cuts its sums off instead of rounding them, which a sum over thousands of tokens
// would show (8e-6 of S after 4096 tokens), so it forms each chunk's V'^T K by itself and the sum over chunks is rounded.
// q, k, v are read once, o is written once: 1 KB a token and head against 98 kFLOP, so HBM is the bound to reach, 1.45 us a
// chunk for a CTA with its SM's share.  The output kernel takes 1.77 (65536 tokens x 16 heads: 203 us, 5.3 TB/s; 2.6 with both
// fused normalisations): its warps issue in half of all clocks, some 1600 instructions a chunk and SM sub-partition, and the
// longest of the roles (V', 2400 clocks, and 200 for each of its waits) paces the others.  What a CTA does is spread over
// warps that each do one thing, chunk after chunk, across segments:
//     warps 0-1    P: Q K^T from tensor memory, times the decays, to shared memory in bf16
//     warp 2       copies of q, k, v (and of the output gate) by TMA, three chunks ahead, and the decays' sums
//     warp 3       issues the MMAs of the state (V'^T K, S^T Q^T)
//     warps 4-7    the norms of q and k (fused normalisation only); V': v times its decay, in three bf16 parts (the A operand
//                  of the state's product)
//     warps 8-11   S: the state, decayed and added to, and its bf16 copy (the A operand of S^T Q^T)
//     warps 12-15  O: the two parts of o added, to shared memory and out by TMA
//     warps 16-19  one warp that issues the outputs' MMAs (Q K^T, V^T P^T): a warp that issues all of them waits for so many
//                  things in turn that the tensor core stands still (204 us against 200); with the gated normalisation,
//                  which takes twice as long, O of every other chunk instead, and warp 3 issues all MMAs
//
// Measured and not kept: the outputs' MMAs issued by a P warp (230 us); V' by eight warps, one of which issues the state's
// MMAs (225); more registers for V' and O (201).
//
// Roundings to bf16: P and the copy of S, which only reach o, itself rounded to bf16 (each adds an error of the size
// of that rounding in its part of o).  V' reaches the state, which is fp32: it is taken in three parts, all its 24 bits.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "kda_linear.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

using linear::Args;
using linear::Segment;

constexpr int kC = 64;    // tokens of a chunk
constexpr int kDim = 128;
constexpr int kTile = kC * kDim * 2;
constexpr int kRing = 4;  // chunks whose decays are kept
constexpr int kUnits = 4;  // units known ahead

// A whole warp's wait.  One that runs out, after about a second (each try is suspended for 4 us), ends the warp's work, and
// so the waits of the others, one second on: until all have left their work, warps meet at such waits only, or as at MEET below.
// (The outputs' kernel waits for the segments' within that second: their launch takes 25 ms for as many tokens as memory
// holds.)  The loop is small on purpose, see tile_lane.
constexpr int kTries = 1 << 18;
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, tc::mbar_wait_suspended(bar, parity, kTries));
}
#define WAIT(bar, n_uses) \
    if (!wait_warp(&(bar), (uint32_t)(n_uses) & 1u)) goto LEAVE
#define LEAVE died

// One arrival for the warp, once all its lanes are here.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What the other warps need of a chunk's decays (in base 2) and norms.
struct __align__(16) Gates {
    float b[kC];               // sums of log-decays from the chunk's start
    float in[kC];              // 2^b: decay of the incoming state
    float out[kC];             // 2^(b_64 - b): decay to the chunk's end; 1 behind the segment
    float rq[kC], rk[kC];      // 1 / norm of q and k, 0 behind the segment (fused normalisation only)
    float all, pad[3];         // 2^b_64
};

// What a CTA works on: a segment of a head.
struct Unit {
    Segment sg;
    int slot, h;  // slot -1: no more
};

struct OutShared {
    Gates gates[kRing];
    float red[2][4][kC], rms[2][kC];  // of the two groups of O
    uint64_t full[3], empty[3];           // q, k, v of a chunk
    uint64_t gfull[kRing], gempty[kRing];
    uint64_t fixed[2];                    // rows behind a segment cleared (turn by turn: V' can be a chunk ahead)
    uint64_t pfull[2], pready[2], ofull[2], ofree[2];
    uint64_t vready[2], kv[2], sready, dfree, qs, pused;
    uint64_t zfull[3], zfree[3];          // output tiles (and the gate's values before them)
    uint64_t ufull[kUnits], uempty[kUnits];
    uint64_t drain;
    Unit unit[kUnits];
    uint32_t tmem;
    volatile int dead, left[2];  // whether a wait has run out: any warp's, one's of a group of O
};
constexpr int kStage = 3 * kTile;
constexpr int kOutP = 3 * kStage, kOutO = kOutP + 8192, kOutV3 = kOutO + 3 * kTile, kOutShared = kOutV3 + kTile;
constexpr int kOutSmem = kOutShared + (int)sizeof(OutShared) + 1024;
static_assert(kOutSmem <= 232448, "shared memory of a CTA");
constexpr int kOutThreads = 640;
// Registers a thread of each warpgroup, see more_registers.
constexpr int kOutOthers = 72, kOutS = 184, kOutRegs = 128 * (4 * kOutOthers + kOutS);
// The warp that issues the outputs' MMAs.
template <bool GATE>
constexpr int kOutSecond = GATE ? 3 : 16;

// Tensor memory: V'^T K, S^T in bf16, V'^T's first two parts, two buffers each of P (then V^T P^T) and S^T Q^T.
enum : uint32_t { kTmD = 0, kTmSb = 128, kTmVhi = 192, kTmVlo = 224, kTmP = 256, kTmO = 384 };

constexpr uint64_t kKmajor = tc::smem_desc_base(16, 1024, tc::SW_128B);
constexpr uint64_t kMNmajor = tc::smem_desc_base(8192, 1024, tc::SW_128B);
constexpr uint32_t kId64 = tc::idesc_bf16_f32(128, 64, false, false);

__device__ __forceinline__ uint32_t lane_base(int warp) { return (uint32_t)((warp & 3) * 32) << 16; }

// Sums of log2-decays of a chunk's tokens, in steps of 2^-44: lane l holds tokens 2l and 2l + 1.  Whole numbers, so that
// behind a token that forgets everything differences of small decays survive (fp64 would do, at ten times the latency).
constexpr float kFixed = 17592186044416.f;
struct Sums {
    long long b0, b1, all;
    bool nan0, nan1, nan;  // whether one of the tokens up to here is NaN, or any
};
__device__ __forceinline__ float from_fixed(long long x) { return __ll2float_rn(x) * (1.f / kFixed); }
__device__ __forceinline__ Sums chunk_sums(float x0, float x1) {
    const int lane = threadIdx.x & 31;
    const unsigned n0 = __ballot_sync(0xffffffffu, x0 != x0), n1 = __ballot_sync(0xffffffffu, x1 != x1);
    const long long f0 = __float2ll_rn(x0 * kFixed), f1 = __float2ll_rn(x1 * kFixed);
    long long s = f0 + f1;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += up;
    }
    Sums r;
    r.b0 = s - f1;
    r.b1 = s;
    r.all = __shfl_sync(0xffffffffu, s, 31);
    const unsigned upto = 0xffffffffu >> (31 - lane);
    r.nan0 = (n0 & upto) | (n1 & (upto >> 1));
    r.nan1 = (n0 | n1) & upto;
    r.nan = n0 | n1;
    return r;
}

// 1 / sqrt(sum of squares + eps) of 16 of the tile's rows, half a row a lane; 0 from row n on, whose tokens are not the
// segment's (of a cleared row without eps it would be infinite, and the product with its zeros NaN).
__device__ __forceinline__ void row_norms(const uint8_t *tile, int first, int n, float eps, float *out) {
    const int lane = threadIdx.x & 31, r = first + (lane & 15);
    const uint8_t *row = tile + (lane >> 4) * 8192 + r * 128;
    float2 ss = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int c = 0; c < 8; ++c) {
        const uint4 x = *reinterpret_cast<const uint4 *>(row + ((c ^ (r & 7)) << 4));
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 y = make_float2(bf16_lo(u[i]), bf16_hi(u[i]));
            ss = tc::fma2(y, y, ss);
        }
    }
    float all = ss.x + ss.y;
    all += __shfl_xor_sync(0xffffffffu, all, 16);
    out[r] = r < n ? rsqrtf(all + eps) : 0.f;
}

// Clears rows n..63 of a q, k or v tile (tokens of another document, or none): they would meet zeros in the products,
// but infinities and NaN among them would not vanish.
__device__ __forceinline__ void clear_rows(uint8_t *tile, int n, int thread, int threads) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int i = n * 8 + thread; i < kC * 8; i += threads) {
        *reinterpret_cast<uint4 *>(tile + i * 16) = zero;
        *reinterpret_cast<uint4 *>(tile + 8192 + i * 16) = zero;
    }
}

// (The code of this file is kept short on purpose, loops not unrolled unless registers ask for it.  A warp of each kind
// shares an SM sub-partition and its instruction cache: an instruction takes 1.5 clocks of a warp from code of 8 KB, 4
// from 24 KB and 5 to 7 from 48 KB on, and the first version, 120 KB unrolled, took 4 times as long for want of them.)

// What a lane addresses when its warp moves four 8 x 8 tiles between registers and a chunk's tile of `dim` 16 on: tokens
// 0 to 15, in the order (first 8 dims, first 8 tokens), (next 8 dims, first 8 tokens), then the next 8 tokens.  Tokens 16 t
// on are 2048 t bytes further.
__device__ __forceinline__ uint32_t tile_lane(int dim) {
    const int lane = threadIdx.x & 31, token = (lane & 7) + (lane >> 4) * 8, chunk = ((dim & 63) >> 3) + ((lane >> 3) & 1);
    return (uint32_t)((dim >> 6) * 8192 + token * 128 + ((chunk ^ (token & 7)) << 4));
}

// 32 lanes of V'^T (value dimensions 32 (warp % 4) on) for the chunk's tokens, in three bf16 parts: v's tile is read
// transposed, so that a register holds two tokens of a value dimension, as the MMA wants A.  The third part goes back to
// shared memory, a tile like v's: tensor memory has no room for it beside the outputs.  The first 32 tokens are `ready`
// before the others: their MMAs run meanwhile; and each half waits for the MMAs of the `uses`-th one in its place to be `done`.
// False if a wait ran out.  (Two parts would do with 8 MMAs instead of 12 and take 5 to 12% less time of long prompts, but
// their 16 bits put S off by 2.2e-6 of its size; all 24 by 4e-7, like fp32 sums.)
template <bool NORM>
__device__ __forceinline__ bool decayed_values(const uint8_t *v, uint8_t *third, const Gates &g, int warp, uint32_t hi_col, uint32_t lo_col,
                                               uint64_t *ready, uint64_t *done, int uses) {
    const int c2 = (threadIdx.x & 3) * 2, dim = (warp & 3) * 32;
    uint32_t from0 = tc::smem_u32(v) + tile_lane(dim), from1 = tc::smem_u32(v) + tile_lane(dim + 16);
    const uint32_t to_third = tc::smem_u32(third) - tc::smem_u32(v);
    hi_col += lane_base(warp);
    lo_col += lane_base(warp);
#pragma unroll 1
    for (int j = c2; j < kC; j += 16, from0 += 2048, from1 += 2048, hi_col += 8, lo_col += 8) {
        if (!(j & 16) && uses > 0) {
            if (!wait_warp(done + (j >> 5), (uint32_t)(uses - 1) & 1u)) return false;
            tc::tc_fence_after();
        }
        uint32_t x[2][4];
        tc::ldmatrix_t4(from0, x[0]);
        tc::ldmatrix_t4(from1, x[1]);
        float2 w[2] = {*reinterpret_cast<const float2 *>(&g.out[j]), *reinterpret_cast<const float2 *>(&g.out[j + 8])};
        if (NORM) {
            w[0] = tc::mul2(w[0], *reinterpret_cast<const float2 *>(&g.rk[j]));
            w[1] = tc::mul2(w[1], *reinterpret_cast<const float2 *>(&g.rk[j + 8]));
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t hi[4], mid[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 y = tc::mul2(make_float2(bf16_lo(x[half][e]), bf16_hi(x[half][e])), w[e >> 1]);
                hi[e] = pack_bf16(y.x, y.y);
                const float2 r = tc::sub2(y, make_float2(bf16_lo(hi[e]), bf16_hi(hi[e])));
                mid[e] = pack_bf16(r.x, r.y);
                const float2 rr = tc::sub2(r, make_float2(bf16_lo(mid[e]), bf16_hi(mid[e])));
                lo[e] = pack_bf16(rr.x, rr.y);
            }
            tc::tmem_st_16x8(hi_col + (half << 20), hi);
            tc::tmem_st_16x8(lo_col + (half << 20), mid);
            tc::stmatrix_t4((half ? from1 : from0) + to_third, lo);
        }
        if (j & 16) {
            tc::fence_async_smem();
            tc::tmem_wait_st();
            tc::tc_fence_before();
            warp_arrive(ready + (j >> 5));
        }
    }
    return true;
}

// A value that all lanes of the warp have, in a register of the whole warp: what an MMA takes has to be in those, and from
// values that the compiler cannot tell to be the same in all lanes it moves every operand of every MMA there (24
// instructions an MMA, of which the issuing warp did not get enough: 100 to 140 clocks for one that runs for 32 to 64).
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(0xffffffffu, x); }

// The lower half of a shared-memory descriptor; the upper one is the layout's alone.
__device__ __forceinline__ uint32_t desc_lo(uint64_t base, uint32_t smem_addr) { return (uint32_t)base | ((smem_addr & 0x3FFFF) >> 4); }
__device__ __forceinline__ uint64_t desc(uint64_t base, uint32_t lo) { return (base & 0xffffffff00000000ull) | lo; }

// MMAs over consecutive slices of 16 of K: A in tensor memory (8 columns a slice) or in shared memory, B in shared memory,
// slices `a_step` and `b_step` (in 16 bytes) apart.
template <int STEPS>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_base, uint32_t b, uint32_t b_step, uint32_t id, bool accumulate, bool one) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) tc::mma_bf16_ts_warp(d, a + 8 * i, desc(b_base, b + b_step * i), id, accumulate || i > 0, one);
}
template <int STEPS>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a_base, uint32_t a, uint32_t a_step, uint64_t b_base, uint32_t b, uint32_t b_step,
                                       uint32_t id, bool accumulate, bool one) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) tc::mma_bf16_warp(d, desc(a_base, a + a_step * i), desc(b_base, b + b_step * i), id, accumulate || i > 0, one);
}

// V'^T K over the first or last 32 of the chunk's tokens, all parts of V'.
__device__ __forceinline__ void mma_state(int half, uint32_t d_col, uint32_t hi_col, uint32_t lo_col, uint32_t third, uint32_t k, bool one) {
    constexpr uint32_t id = tc::idesc_bf16_f32(128, 128, false, true);
    const uint32_t kd = desc_lo(kMNmajor, k + half * 4096);
    mma_ts<2>(d_col, hi_col + half * 16, kMNmajor, kd, 128, id, half > 0, one);
    mma_ts<2>(d_col, lo_col + half * 16, kMNmajor, kd, 128, id, true, one);
    mma_ss<2>(d_col, kMNmajor, desc_lo(kMNmajor, third + half * 4096), 128, kMNmajor, kd, 128, tc::idesc_bf16_f32(128, 128, true, true), true, one);
}

// The registers of a warpgroup's threads, changed by all its warps.  What the groups have afterwards must not be more than
// the block was launched with, or the group that asks for more waits for ever: the host compares the sums below with the
// built kernel's registers before it launches it.
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// This thread's column of a state in memory (rows of kDim), as pairs of rows.
__device__ __forceinline__ void load_column(float2 (&S)[kDim / 2], const float *p) {
#pragma unroll
    for (int k = 0; k < kDim / 2; ++k) S[k] = p ? make_float2(p[(size_t)2 * k * kDim], p[(size_t)(2 * k + 1) * kDim]) : make_float2(0.f, 0.f);
}
__device__ __forceinline__ void store_column(const float2 (&S)[kDim / 2], float *p) {
#pragma unroll
    for (int k = 0; k < kDim / 2; ++k) {
        p[(size_t)2 * k * kDim] = S[k].x;
        p[(size_t)(2 * k + 1) * kDim] = S[k].y;
    }
}

// S <- all S + V'^T K of this thread's lane.
__device__ __forceinline__ void add_products(float2 (&S)[kDim / 2], float2 all, uint32_t col) {
#pragma unroll
    for (int k = 0; k < kDim; k += 32) {
        float x[32];
        tc::tmem_ld32(col + k, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) S[k / 2 + e] = tc::fma2(S[k / 2 + e], all, make_float2(x[2 * e], x[2 * e + 1]));
    }
    tc::tc_fence_before();
}

// The unit behind `u` for a warp's CTA.
__device__ __forceinline__ int next_unit(const Args &a, int u) {
    if (!a.ticket) return u + (int)gridDim.x;
    int t = 0;
    if ((threadIdx.x & 31) == 0) {
        tc::grid_dep_wait();  // the kernel that sets the ticket to 0
        t = atomicAdd(a.ticket, 1);
    }
    return (int)gridDim.x + __shfl_sync(0xffffffffu, t, 0);
}

template <bool NORM, bool GATE>
__global__ void __launch_bounds__(kOutThreads, 1)
linear_out_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
              const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ CUtensorMap tm_z, const Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    OutShared &sh = *reinterpret_cast<OutShared *>(sm + kOutShared);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) {
            tc::mbar_init(&sh.full[i], 1);
            tc::mbar_init(&sh.empty[i], GATE ? 1 : 2);
            tc::mbar_init(&sh.zfull[i], 1);
            tc::mbar_init(&sh.zfree[i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(&sh.gfull[i], NORM ? 5 : 1);
            tc::mbar_init(&sh.gempty[i], 14);  // V', S and O warps, the two of P
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.fixed[i], 4);
            tc::mbar_init(&sh.pfull[i], 1);
            tc::mbar_init(&sh.pready[i], 2);
            tc::mbar_init(&sh.ofull[i], GATE ? 1 : 2);
            tc::mbar_init(&sh.ofree[i], 4);
            sh.left[i] = 0;
        }
        for (int i = 0; i < kUnits; ++i) {
            tc::mbar_init(&sh.ufull[i], 1);
            tc::mbar_init(&sh.uempty[i], GATE ? 19 : 16);  // all warps at work but the copies'
        }
        tc::mbar_init(&sh.vready[0], 4);
        tc::mbar_init(&sh.vready[1], 4);
        tc::mbar_init(&sh.sready, 4);
        tc::mbar_init(&sh.dfree, 4);
        tc::mbar_init(&sh.kv[0], 1);
        tc::mbar_init(&sh.kv[1], 1);
        tc::mbar_init(&sh.qs, 1);
        tc::mbar_init(&sh.pused, 1);
        tc::mbar_init(&sh.drain, GATE ? 1 : 2);
        sh.dead = 0;
        tc::fence_mbar_init();
    }
    if (warp == 3) {
        tc::tmem_alloc(&sh.tmem, 512);
        tc::tmem_relinquish();
    }
    // Behind the segments' kernels, which have waited for everything before them, only the states have to be waited for: the
    // S warps do.  (All of them, whatever they read: this kernel's end then means the end of the ones before it.)
    if (a.first) tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (threadIdx.x == 0 && a.total > 0) {
        tc::prefetch_map(&tm_q);
        tc::prefetch_map(&tm_k);
        tc::prefetch_map(&tm_v);
        tc::prefetch_map(&tm_o);
        if (GATE) tc::prefetch_map(&tm_z);
    }
    tc::tc_fence_before();
    const bool valid = linear::valid_table(a.cu, a.num_seqs, a.total);  // also the barrier behind the set-up
    tc::tc_fence_after();
    if (a.first && blockIdx.x == 0 && threadIdx.x == 0) *a.status = valid ? (int32_t)KDA_OK : (int32_t)KDA_ERR_INVALID_ARG;
    const uint32_t tm = sh.tmem;
    const int units = valid ? a.slots * a.H : 0;
    const int share = a.H / a.Hqk;

// The units of a CTA, as the copies' warp hands them out, and their chunks.
#define NEXT_UNIT                                                    \
    WAIT(sh.ufull[turn % kUnits], turn / kUnits);                    \
    const Segment sg = sh.unit[turn % kUnits].sg;                    \
    [[maybe_unused]] const int slot = sh.unit[turn % kUnits].slot, h = sh.unit[turn % kUnits].h; \
    warp_arrive(&sh.uempty[turn % kUnits]);                          \
    ++turn;
#define CHUNKS                                                       \
    for (int c0 = 0; c0 < sg.len; c0 += kC, ++n) {                   \
        [[maybe_unused]] const int t0 = sg.t0 + c0, rows = min(kC, sg.len - c0), st = n % 3;
#define FOR_SEGMENTS                                                 \
    for (;;) {                                                       \
        NEXT_UNIT                                                    \
        if (slot < 0) break;                                         \
        CHUNKS
#define END_SEGMENTS \
    }                \
    }

    int turn = 0;  // units so far
    int n = 0;  // chunks so far: each barrier's phase follows from it
    if (warp < 8 || warp >= 12) fewer_registers<kOutOthers>();
    if (warp == 2) {
        // ---- units, copies and decays; a chunk's decays are read while the one before it is worked on.  Documents are of
        // any length, so behind its first unit a CTA takes the next that nobody has: dealt out in turn, the CTA with the
        // most chunks had half as many again as the mean (8 documents, 33000 tokens x 32 heads).
        float g0 = 0.f, g1 = 0.f;
        linear::Repeated all{};  // 2^b_64 where it is the same for chunk after chunk
        for (int u = blockIdx.x;; ++turn) {
            Segment sg;
            while (u < units && !linear::find_segment(a.cu, a.num_seqs, a.seg, u / a.H, &sg)) u = next_unit(a, u);
            const int slot = u / a.H, h = u - slot * a.H;
            if (turn >= kUnits) WAIT(sh.uempty[turn % kUnits], turn / kUnits - 1);
            if (lane == 0) {
                sh.unit[turn % kUnits] = Unit{sg, u < units ? slot : -1, h};
                tc::mbar_arrive(&sh.ufull[turn % kUnits]);
            }
            if (u >= units) break;
            CHUNKS
            const bool last_chunk = c0 + kC >= sg.len;
        if (n >= 3) WAIT(sh.empty[st], n / 3 - 1);
        if (lane == 0) {
            uint8_t *to = sm + st * kStage;
            tc::mbar_arrive_expect_tx(&sh.full[st], kStage);
            for (int p = 0; p < 2; ++p) {
                tc::tma_load_3d(to + p * 8192, &tm_q, p * 64, h / share, t0, &sh.full[st]);
                tc::tma_load_3d(to + kTile + p * 8192, &tm_k, p * 64, h / share, t0, &sh.full[st]);
                tc::tma_load_3d(to + 2 * kTile + p * 8192, &tm_v, p * 64, h, t0, &sh.full[st]);
            }
        }
        const auto fetch = [&](int t, int count) {
            const float *p = a.per_token ? a.g + (size_t)(t + 2 * lane) * a.H + h : a.g + h;
            g0 = 2 * lane < count ? *p : 0.f;
            g1 = 2 * lane + 1 < count ? p[a.per_token ? a.H : 0] : 0.f;
        };
        if (c0 == 0) fetch(t0, rows);
        Gates &g = sh.gates[n % kRing];
        const float x0 = linear::log2_decay(g0), x1 = linear::log2_decay(g1);
        if (!last_chunk) fetch(t0 + kC, min(kC, sg.len - c0 - kC));
        const Sums s = chunk_sums(x0, x1);
        if (n >= kRing) WAIT(sh.gempty[n % kRing], n / kRing - 1);
        {
            const float nan = __int_as_float(0x7fffffff);
            const float2 b = make_float2(s.nan0 ? nan : from_fixed(s.b0), s.nan1 ? nan : from_fixed(s.b1));
            reinterpret_cast<float2 *>(g.b)[lane] = b;
            reinterpret_cast<float2 *>(g.in)[lane] = make_float2(ex2(b.x), ex2(b.y));
            reinterpret_cast<float2 *>(g.out)[lane] = make_float2(ex2(from_fixed(s.all - s.b0)), ex2(from_fixed(s.all - s.b1)));
            const bool repeats = !a.per_token && sg.len >= 2 * kC;
            if (repeats && c0 == 0) all = linear::Repeated::of((double)s.all * (1. / kFixed));
            const float x = repeats && rows == kC ? all.next() : exp2f(from_fixed(s.all));
            if (lane == 0) g.all = s.nan ? nan : x;
        }
        if (!a.withheld) warp_arrive(&sh.gfull[n % kRing]);
        if (GATE) {
            if (n >= 3) WAIT(sh.zfree[st], n / 3 - 1);
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&sh.zfull[st], kTile);
                for (int p = 0; p < 2; ++p) tc::tma_load_3d(sm + kOutO + st * kTile + p * 8192, &tm_z, p * 64, h, t0, &sh.zfull[st]);
            }
        }
            }
            u = next_unit(a, u);
        }
    } else if (warp == 3 || warp == kOutSecond<GATE>) {
        // ---- MMAs, in the order in which they can start: V'^T K and S^T Q^T of a chunk, Q K^T of the next, whose scores are
        // worked out meanwhile, V^T P^T of the first
        const bool one = tc::elect_one(), state = warp == 3, out = GATE || !state;
        const uint32_t base = uniform(tc::smem_u32(sm)), tu = uniform(tm);
        int fixes = 0, left = 0;  // tokens of the segment that are left
        for (bool more = true; more; ++n) {
            while (more && left <= 0) {
                NEXT_UNIT
                more = slot >= 0;
                left = more ? sg.len : 0;
            }
            const uint32_t un = uniform(n), um = un - 1, s = um % 3, b = um & 1, before = base + s * kStage;
            if (state && n > 0) {  // of the chunk before
                WAIT(sh.dfree, um);
#pragma unroll 1
                for (uint32_t half = 0; half < 2; ++half) {
                    WAIT(sh.vready[half], um);
                    tc::tc_fence_after();
                    mma_state(half, tu + kTmD, tu + kTmVhi, tu + kTmVlo, base + kOutV3, before + kTile, one);
                    if (one) tc::mma_commit(&sh.kv[half]);
                    __syncwarp();
                }
                if (!GATE && n >= 3) WAIT(sh.ofree[b], um / 2 - 1);
                WAIT(sh.sready, um);
                tc::tc_fence_after();
                const uint32_t qd = desc_lo(kKmajor, before);
#pragma unroll(GATE ? 1 : 2)
                for (uint32_t p = 0; p < 2; ++p) mma_ts<4>(tu + kTmO + b * 64, tu + kTmSb + p * 32, kKmajor, qd + p * 512, 2, kId64, p, one);
                if (one) {
                    tc::mma_commit(&sh.qs);
                    if (!GATE) {
                        tc::mma_commit(&sh.ofull[b]);
                        tc::mma_commit(&sh.empty[s]);
                    }
                }
                __syncwarp();
            }
            if (!out) {
                left -= kC;
                continue;
            }
            // the next Q K^T waits for the output that was in its place: a quick one is gone before P is there, while
            // a gated one takes longer than P
            const int second = GATE && n >= 2;
#pragma unroll 1
            for (int go = 0; go < 2; ++go) {
                if (go == second && more) {
                    const uint32_t st = un % 3;
                    WAIT(sh.full[st], un / 3);
                    if (left < kC) {
                        WAIT(sh.fixed[fixes & 1], fixes >> 1);
                        ++fixes;
                    }
                    left -= kC;
                    if (n >= 2) WAIT(sh.ofree[un & 1], un / 2 - 1);
                    tc::tc_fence_after();
                    // (rows 64 to 127 of the result come of what follows the tile's half, and nobody reads them)
                    const uint32_t qd = desc_lo(kKmajor, base + st * kStage), kd = desc_lo(kKmajor, base + st * kStage + kTile), d = tu + kTmP + (un & 1) * 64;
#pragma unroll(GATE ? 1 : 2)
                    for (uint32_t p = 0; p < 2; ++p) mma_ss<4>(d, kKmajor, qd + p * 512, 2, kKmajor, kd + p * 512, 2, kId64, p, one);
                    if (one) tc::mma_commit(&sh.pfull[un & 1]);
                    __syncwarp();
                }
                if (go != second && n > 0) {
                    WAIT(sh.pready[b], um >> 1);
                    tc::tc_fence_after();
                    mma_ss<4>(tu + kTmP + b * 64, kMNmajor, desc_lo(kMNmajor, before + 2 * kTile), 128, kKmajor, desc_lo(kKmajor, base + kOutP), 2,
                            tc::idesc_bf16_f32(128, 64, true, false), false, one);
                    if (one) {
                        tc::mma_commit(&sh.ofull[b]);
                        tc::mma_commit(&sh.pused);
                        tc::mma_commit(&sh.empty[s]);
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp < 2) {
        // ---- P
        const int i = warp * 32 + lane;
        FOR_SEGMENTS
        WAIT(sh.gfull[n % kRing], n / kRing);
        WAIT(sh.pfull[n & 1], n / 2);
        if (n >= 1) WAIT(sh.pused, n - 1);
        tc::tc_fence_after();
        {
            const Gates &g = sh.gates[n % kRing];
            // (the sums' rounding, 2^-24 of up to 64 x 160, costs a score at most a part in 2^11: less than its bf16)
            const float bi = g.b[i];
            const uint32_t from = tm + kTmP + (n & 1) * 64 + lane_base(warp);
            uint8_t *row = sm + kOutP + i * 128;
            const int end = min(i + 1, rows);
#pragma unroll 1
            for (int j = 0; j < kC; j += 8) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (j < 32 * (warp + 1)) {  // (warp 0 holds the first 32 rows, which end at column 32)
                    float x[8], b[8];
                    tc::tmem_ld8(from + j, x);
                    *reinterpret_cast<float4 *>(b) = *reinterpret_cast<const float4 *>(&g.b[j]);
                    *reinterpret_cast<float4 *>(b + 4) = *reinterpret_cast<const float4 *>(&g.b[j + 4]);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float2 d = tc::sub2(make_float2(bi, bi), make_float2(b[e], b[e + 1]));
                        float2 y = tc::mul2(make_float2(x[e], x[e + 1]), make_float2(ex2(d.x), ex2(d.y)));
                        if (NORM) y = tc::mul2(y, *reinterpret_cast<const float2 *>(&g.rk[j + e]));
                        x[e] = y.x;
                        x[e + 1] = y.y;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (j + e >= end) x[e] = 0.f;
                    u = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
                }
                *reinterpret_cast<uint4 *>(row + (((j >> 3) ^ (i & 7)) << 4)) = u;
            }
        }
        tc::fence_async_smem();
        tc::tc_fence_before();
        warp_arrive(&sh.pready[n & 1]);
        if (lane == 0) tc::mbar_arrive(&sh.gempty[n % kRing]);
        END_SEGMENTS
    } else if (warp < 8) {
        // ---- V'
        int fixes = 0;
        FOR_SEGMENTS
        WAIT(sh.full[st], n / 3);
        if (rows < kC) {
            clear_rows(sm + st * kStage + kTile, rows, threadIdx.x - 128, 128);
            clear_rows(sm + st * kStage + 2 * kTile, rows, threadIdx.x - 128, 128);
            tc::fence_async_smem();
            warp_arrive(&sh.fixed[fixes & 1]);
            WAIT(sh.fixed[fixes & 1], fixes >> 1);
            ++fixes;
        }
        if (NORM) {
            if (n >= kRing) WAIT(sh.gempty[n % kRing], n / kRing - 1);
#pragma unroll 1
            for (int k = 0; k < 2; ++k)
                row_norms(sm + st * kStage + k * kTile, (warp & 3) * 16, rows, a.fu.qk_eps, k ? sh.gates[n % kRing].rk : sh.gates[n % kRing].rq);
            warp_arrive(&sh.gfull[n % kRing]);
        }
        WAIT(sh.gfull[n % kRing], n / kRing);
        if (!decayed_values<NORM>(sm + st * kStage + 2 * kTile, sm + kOutV3, sh.gates[n % kRing], warp, tm + kTmVhi, tm + kTmVlo, sh.vready, sh.kv, n))
            goto died;
        if (lane == 0) tc::mbar_arrive(&sh.gempty[n % kRing]);
        END_SEGMENTS
    } else if (warp < 12) {
        // ---- S
        more_registers<kOutS>();
        tc::grid_dep_wait();
        const int dv = (warp & 3) * 32 + lane;
        const uint32_t d_col = tm + kTmD + lane_base(warp), sb_col = tm + kTmSb + lane_base(warp);
        for (;;) {
            NEXT_UNIT
            if (slot < 0) break;
            const float *init = linear::segment_start(a, sg, slot, h, (size_t)kDim * kDim);
            float2 S[kDim / 2], all = make_float2(1.f, 1.f);
            load_column(S, init ? init + dv : nullptr);
            for (int c0 = 0; c0 < sg.len; c0 += kC, ++n) {
                if (c0 > 0) {
                    WAIT(sh.kv[1], n - 1);
                    tc::tc_fence_after();
                    add_products(S, all, d_col);
                }
                warp_arrive(&sh.dfree);
                if (n > 0) WAIT(sh.qs, n - 1);
                tc::tc_fence_after();
#pragma unroll
                for (int k = 0; k < kDim; k += 16) {
                    uint32_t p[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[e] = pack_bf16(S[k / 2 + e].x, S[k / 2 + e].y);
                    tc::tmem_st8(sb_col + k / 2, p);
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                warp_arrive(&sh.sready);
                WAIT(sh.gfull[n % kRing], n / kRing);
                const float x = sh.gates[n % kRing].all;
                all = make_float2(x, x);
                warp_arrive(&sh.gempty[n % kRing]);
            }
            if (sg.len > 0) {
                WAIT(sh.kv[1], n - 1);
                tc::tc_fence_after();
                add_products(S, all, d_col);
            }
            if (sg.last && a.S_final) store_column(S, a.S_final + ((size_t)sg.doc * a.H + h) * kDim * kDim + dv);
        }
    } else if (GATE || warp < 16) {
        // ---- O; with the gated normalisation two groups of four warps, every other chunk each
        const int group = GATE ? (warp >> 2) - 3 : 0, first = 384 + group * 128, tid = (int)threadIdx.x - first;
        const int dim = (warp & 3) * 32, c2 = (lane & 3) * 2;
        float (&red)[4][kC] = sh.red[group], (&rms)[kC] = sh.rms[group];
        int going = -1;  // the tile whose copy out is not known to have read it
// All four warps of the group here, with what they have written for each other.  The barrier has no limit of its own: a warp
// whose wait has run out says so and arrives once more, so that the others, each of which gets here or gives up in the end, are
// all let go, see it, and follow it.  That is looked at where a chunk's waits lie before the barrier; none lies between its others.
#define MEET tc::named_barrier(2 + group, 128)
#define MEET_BEHIND_WAITS \
    MEET;                 \
    if (sh.left[group]) goto LEAVE
#undef LEAVE
#define LEAVE left_behind
        float2 weight[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)};  // of dimensions dim + 16 h + lane / 4 and 8 on
        if (GATE && a.fu.weight)
            for (int h = 0; h < 2; ++h)
                weight[h] = make_float2(a.fu.weight[dim + 16 * h + (lane >> 2)], a.fu.weight[dim + 16 * h + 8 + (lane >> 2)]);
        FOR_SEGMENTS
        if (GATE && (n & 1) != group) continue;
        uint8_t *tile = sm + kOutO + st * kTile;
        WAIT(sh.gfull[n % kRing], n / kRing);
        if (GATE) {
            WAIT(sh.zfull[st], n / 3);
        } else {
            if (n >= 3) WAIT(sh.zfree[st], n / 3 - 1);
        }
        WAIT(sh.ofull[n & 1], n / 2);
        tc::tc_fence_after();
        {
            const Gates &g = sh.gates[n % kRing];
            const uint32_t t1 = tm + kTmO + (n & 1) * 64 + lane_base(warp), t2 = tm + kTmP + (n & 1) * 64 + lane_base(warp);
            uint32_t to[2] = {tc::smem_u32(tile) + tile_lane(dim), tc::smem_u32(tile) + tile_lane(dim + 16)};
            // o of 16 tokens and 32 value dimensions from its two parts, two fragments of 16 x 8 for each 16 dimensions
            const auto part = [&](int i, float2 (&z)[2][4]) {
                float x[2][8], y[2][8];
                tc::tmem_ld_16x16x4(t1 + i, t2 + i, x, y);
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const float2 in = *reinterpret_cast<const float2 *>(&g.in[i + 8 * f + c2]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int h = e >> 1, at = 4 * f + 2 * (e & 1);
                        z[h][2 * f + (e & 1)] = tc::fma2(in, make_float2(x[h][at], x[h][at + 1]), make_float2(y[h][at], y[h][at + 1]));
                    }
                    if (NORM) {
                        const float2 rq = *reinterpret_cast<const float2 *>(&g.rq[i + 8 * f + c2]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) z[e >> 1][2 * f + (e & 1)] = tc::mul2(z[e >> 1][2 * f + (e & 1)], rq);
                    }
                }
            };
            const auto put = [&](const float2 (&z)[2][4]) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t u[4] = {pack_bf16(z[h][0].x, z[h][0].y), pack_bf16(z[h][1].x, z[h][1].y), pack_bf16(z[h][2].x, z[h][2].y),
                                           pack_bf16(z[h][3].x, z[h][3].y)};
                    tc::stmatrix_t4(to[h], u);
                    to[h] += 2048;
                }
            };
            if (GATE) {
                // sums of squares over the value dimension: over a thread's four, its warp's 32 (each exchange leaves a lane
                // half of the tokens), and the four warps'
                const bool up1 = lane & 4, up2 = lane & 8;
#pragma unroll 1
                for (int i = 0; i < kC; i += 16) {
                    float2 z[2][4], sq[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    part(i, z);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sq[(e & 3) >> 1] = tc::fma2(z[e >> 2][e & 3], z[e >> 2][e & 3], sq[(e & 3) >> 1]);
                    float2 x = up1 ? sq[1] : sq[0];
                    const float2 give = up1 ? sq[0] : sq[1];
                    x.x += __shfl_xor_sync(0xffffffffu, give.x, 4);
                    x.y += __shfl_xor_sync(0xffffffffu, give.y, 4);
                    float y = up2 ? x.y : x.x;
                    y += __shfl_xor_sync(0xffffffffu, up2 ? x.x : x.y, 8);
                    y += __shfl_xor_sync(0xffffffffu, y, 16);
                    if (lane < 16) red[warp & 3][i + (up1 ? 8 : 0) + c2 + (up2 ? 1 : 0)] = y;
                }
                MEET_BEHIND_WAITS;
                if (tid < kC) {
                    const int i = tid;
                    rms[i] = rsqrtf(((red[0][i] + red[1][i]) + (red[2][i] + red[3][i])) * (1.f / kDim) + a.fu.out_eps);
                }
                MEET;
            }
#pragma unroll 1
            for (int i = 0; i < kC; i += 16) {
                float2 z[2][4];
                part(i, z);
                if (GATE) {
                    const float2 r[2] = {*reinterpret_cast<const float2 *>(&rms[i + c2]), *reinterpret_cast<const float2 *>(&rms[i + 8 + c2])};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t gate[4];
                        tc::ldmatrix_t4(to[h], gate);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 x = tc::mul2(make_float2(bf16_lo(gate[e]), bf16_hi(gate[e])), make_float2(-linear::kLog2e, -linear::kLog2e));
                            const float2 y = tc::add2(make_float2(ex2(x.x), ex2(x.y)), make_float2(1.f, 1.f));
                            const float w = e & 1 ? weight[h].y : weight[h].x;
                            z[h][e] = tc::mul2(tc::mul2(z[h][e], make_float2(rcp(y.x), rcp(y.y))), tc::mul2(r[e >> 1], make_float2(w, w)));
                        }
                    }
                }
                put(z);
            }
            tc::tc_fence_before();
            warp_arrive(&sh.ofree[n & 1]);
        }
        if (lane == 0) tc::mbar_arrive(&sh.gempty[n % kRing]);
        tc::fence_async_smem();
        if (GATE) {
            MEET;
        } else {
            MEET_BEHIND_WAITS;
        }
        // a tile is free again once its copy out has read it: seen to when the next one is on its way
        if (rows == kC) {
            if (tid == 0) {
                tc::tma_store_3d(&tm_o, 0, h, t0, tile);
                tc::tma_store_3d(&tm_o, 64, h, t0, tile + 8192);
                tc::bulk_commit();
                if (GATE) {  // the gate's values of three chunks on wait for the tile
                    tc::bulk_wait_read();
                    tc::mbar_arrive(&sh.zfree[st]);
                } else {
                    if (going >= 0) {
                        tc::bulk_wait_read_all_but_one();
                        tc::mbar_arrive(&sh.zfree[going]);
                    }
                    going = st;
                }
            }
        } else {
#pragma unroll 1
            for (int i = tid; i < rows * 16; i += 128) {
                const int t = i >> 4, c = i & 15;
                reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + ((size_t)(t0 + t) * a.H + h) * kDim)[c] =
                    *reinterpret_cast<const uint4 *>(tile + (c >> 3) * 8192 + t * 128 + (((c & 7) ^ (t & 7)) << 4));
            }
            tc::fence_async_smem();
            MEET;
            if (tid == 0) {
                if (going >= 0) {
                    tc::bulk_wait_read();
                    tc::mbar_arrive(&sh.zfree[going]);
                    going = -1;
                }
                tc::mbar_arrive(&sh.zfree[st]);
            }
        }
        __syncwarp();
        END_SEGMENTS
        goto done;
    left_behind:
        sh.left[group] = 1;
        __threadfence_block();
        __syncwarp();
        tc::named_barrier_arrive(2 + group, 128);
        goto died;
#undef LEAVE
#define LEAVE died
    }
    goto done;
died:
    sh.dead = 1;
done:
    __syncwarp();
    if (warp == 3 || warp == kOutSecond<GATE>) {  // every MMA done before the tensor memory goes
        if (tc::elect_one()) tc::mma_commit(&sh.drain);
        __syncwarp();
        tc::mbar_wait(&sh.drain, 0);
    }
    if (warp >= 12 && threadIdx.x % 128 == 0) tc::bulk_wait_read();
    tc::tc_fence_before();
    __syncthreads();
    if (sh.dead && warp == 2) {  // copies in flight: each stage's last one, which ends a phase of either parity
        for (int i = 0; i < 3; ++i)
            for (int p = 0; p < 2; ++p) {
                tc::mbar_wait(&sh.full[i], p, 1000000);
                tc::mbar_wait(&sh.zfull[i], p, 1000000);
            }
    }
    __syncthreads();
    if (warp == 3) tc::tmem_dealloc(tm, 512);
    if (sh.dead && threadIdx.x == 0) atomicExch(a.status, (int32_t)KDA_ERR_TIMEOUT);
}

// ---------------------------------------------------------------------------
// What each segment but a document's last adds to the state by its end, S^T = sum_j 2^(b_end - b_j) v_j k_j^T.  The
// chunks are taken from the last to the first, so that every weight is known when its chunk is reached and the sum is
// never rescaled; it also leaves the segment's first rows in L2 for the pass that forms the outputs.
// Only k and v are read: 512 bytes a token and head; and only as far back as weights are above 2^-126, below which they are
// zero here (exp2 flushes what fp32 holds no normal number for).
//     warp 0  copies   warp 2  decays   warps 1, 3  MMAs, and warps 4-7, 8-11  V' (and norms of k), of every other chunk
//     warps 12-15  the sums over the chunks, in registers
// 65536 tokens x 16 heads, none forgotten: 103 us, 1.0 a chunk against the 0.7 of an SM's share of HBM (one warp for all MMAs:
// 106 us); V' is the longest role here too.
// ---------------------------------------------------------------------------
constexpr int kSegStages = 5, kTold = 8;
struct SegShared {
    Gates gates[kRing];
    uint64_t full[kSegStages], empty[kSegStages];
    uint64_t gfull[kRing], gempty[kRing];
    uint64_t vready[2][2], vfree[2][2], dfull[2], dfree[2], drain;
    uint64_t told[kTold];  // whether a chunk is its segment's last one that counts
    int stop[kTold];
    uint32_t tmem;
    volatile int dead;
};
constexpr int kSegStage = 2 * kTile;
constexpr int kSegV3 = kSegStages * kSegStage, kSegShared = kSegV3 + 2 * kTile;
constexpr int kSegSmem = kSegShared + (int)sizeof(SegShared) + 1024;
static_assert(kSegSmem <= 232448, "shared memory of a CTA");
constexpr int kSegThreads = 16 * 32;
constexpr int kSegOthers = 104, kSegSums = 184, kSegRegs = 128 * (3 * kSegOthers + kSegSums);

constexpr long long kGone = -(127ll << 44);  // in the sums' fixed point

template <bool NORM>
__global__ void __launch_bounds__(kSegThreads, 1)
linear_segment_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    SegShared &sh = *reinterpret_cast<SegShared *>(sm + kSegShared);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSegStages; ++i) {
            tc::mbar_init(&sh.full[i], 1);
            tc::mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kTold; ++i) tc::mbar_init(&sh.told[i], 1);
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(&sh.gfull[i], NORM ? 5 : 1);
            tc::mbar_init(&sh.gempty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.vready[i][0], 4);
            tc::mbar_init(&sh.vready[i][1], 4);
            tc::mbar_init(&sh.vfree[i][0], 1);
            tc::mbar_init(&sh.vfree[i][1], 1);
            tc::mbar_init(&sh.dfull[i], 1);
            tc::mbar_init(&sh.dfree[i], 4);
        }
        tc::mbar_init(&sh.drain, 2);
        sh.dead = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(&sh.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::grid_dep_wait();
    tc::grid_dep_launch();  // (not before the wait: the kernels behind this one read q, k, v and g without one)
    tc::tc_fence_before();
    const bool valid = linear::valid_table(a.cu, a.num_seqs, a.total);  // also the barrier behind the set-up
    tc::tc_fence_after();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *a.status = valid ? (int32_t)KDA_OK : (int32_t)KDA_ERR_INVALID_ARG;
        *a.ticket = 0;
    }
    const uint32_t tm = sh.tmem, tm_vhi = tm + 256, tm_vlo = tm + 288;  // V'^T K at 0 and 128, V' at 256 and 320
    const int units = valid ? a.slots * a.H : 0;
    const int share = a.H / a.Hqk;

// a segment that is not its document's last has a.seg tokens, a whole number of chunks
#define FOR_FULL_SEGMENTS                                                                                      \
    for (int u = blockIdx.x; u < units; u += gridDim.x) {                                                      \
        Segment sg;                                                                                            \
        const int slot = u / a.H, h = u - slot * a.H;                                                          \
        if (!linear::find_segment(a.cu, a.num_seqs, a.seg, slot, &sg) || sg.last) continue;
#define FOR_CHUNKS                                                                                             \
        for (int c0 = sg.len - kC; c0 >= 0; c0 -= kC, ++n) {                                                   \
            [[maybe_unused]] const int t0 = sg.t0 + c0, st = n % kSegStages, b = n & 1;

    if (warp < 12) fewer_registers<kSegOthers>();
    int n = 0;  // chunks so far
    if (warp == 0) {
        FOR_FULL_SEGMENTS
        FOR_CHUNKS
        if (c0 + kC < sg.len) {
            // (the decays are at most four chunks ahead of what has been copied: `told` goes round in eight)
            WAIT(sh.told[(n - 1) % kTold], (n - 1) / kTold);
            if (sh.stop[(n - 1) % kTold]) break;
        }
        if (n >= kSegStages) WAIT(sh.empty[st], n / kSegStages - 1);
        if (lane == 0) {
            uint8_t *to = sm + st * kSegStage;
            tc::mbar_arrive_expect_tx(&sh.full[st], kSegStage);
            for (int p = 0; p < 2; ++p) {
                tc::tma_load_3d(to + p * 8192, &tm_k, p * 64, h / share, t0, &sh.full[st]);
                tc::tma_load_3d(to + kTile + p * 8192, &tm_v, p * 64, h, t0, &sh.full[st]);
            }
        }
        END_SEGMENTS
    } else if (warp == 1 || warp == 3) {
        const bool one = tc::elect_one();
        const uint32_t base = uniform(tc::smem_u32(sm)), tu = uniform(tm);
        FOR_FULL_SEGMENTS
        FOR_CHUNKS
        if (b != warp >> 1) {
            WAIT(sh.told[n % kTold], n / kTold);
            if (sh.stop[n % kTold]) c0 = 0;
            continue;
        }
        WAIT(sh.full[st], n / kSegStages);
        if (n >= 2) WAIT(sh.dfree[b], n / 2 - 1);
        const uint32_t un = uniform(n), ub = un & 1, v = tu + 256 + ub * 64;
#pragma unroll 1
        for (uint32_t half = 0; half < 2; ++half) {
            WAIT(sh.vready[b][half], n / 2);
            tc::tc_fence_after();
            mma_state(half, tu + ub * 128, v, v + 32, base + kSegV3 + ub * kTile, base + un % kSegStages * kSegStage, one);
            if (one) tc::mma_commit(&sh.vfree[b][half]);
            __syncwarp();
        }
        if (one) {
            tc::mma_commit(&sh.empty[st]);
            tc::mma_commit(&sh.dfull[b]);
        }
        __syncwarp();
        if (sh.stop[n % kTold]) c0 = 0;
        END_SEGMENTS
    } else if (warp == 2) {
        // decays; a chunk's are read while the one before it is worked on
        float g0 = 0.f, g1 = 0.f;
        FOR_FULL_SEGMENTS
        long long later = 0;  // the log-decays of the chunks behind this one, held short of overflow
        bool nan = false;
        FOR_CHUNKS
        const auto fetch = [&](int t) {
            const float *p = a.per_token ? a.g + (size_t)(t + 2 * lane) * a.H + h : a.g + h;
            g0 = *p;
            g1 = p[a.per_token ? a.H : 0];
        };
        if (c0 == sg.len - kC) fetch(t0);
        Gates &g = sh.gates[n % kRing];
        const float x0 = linear::log2_decay(g0), x1 = linear::log2_decay(g1);
        if (c0 > 0) fetch(t0 - kC);
        const Sums s = chunk_sums(x0, x1);
        if (n >= kRing) WAIT(sh.gempty[n % kRing], n / kRing - 1);
        reinterpret_cast<float2 *>(g.out)[lane] =
            nan ? make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff))
                : make_float2(ex2(from_fixed(later + (s.all - s.b0))), ex2(from_fixed(later + (s.all - s.b1))));
        later = min(max(later + s.all, -(1ll << 60)), 1ll << 60);
        nan = nan || s.nan;
        const bool stop = c0 == 0 || (!nan && later < kGone);
        if (lane == 0) sh.stop[n % kTold] = stop;
        if (!a.withheld) warp_arrive(&sh.gfull[n % kRing]);
        if (lane == 0) tc::mbar_arrive(&sh.told[n % kTold]);
        if (stop) c0 = 0;
        }
        if (lane == 0) {
            // (one decay for a head: a factor that the chain of segments repeats)
            const float x = a.per_token ? exp2f(from_fixed(later)) : linear::Repeated::of((double)later * (1. / kFixed)).at(sg.index);
            a.seg_decay[(size_t)slot * a.H + h] = nan ? __int_as_float(0x7fffffff) : x;
        }
        }
    } else if (warp < 12) {
        const int group = (warp >> 2) - 1;
        FOR_FULL_SEGMENTS
        FOR_CHUNKS
        if (b != group) {
            WAIT(sh.told[n % kTold], n / kTold);
            if (sh.stop[n % kTold]) c0 = 0;
            continue;
        }
        WAIT(sh.full[st], n / kSegStages);
        if (NORM) {
            if (n >= kRing) WAIT(sh.gempty[n % kRing], n / kRing - 1);
            row_norms(sm + st * kSegStage, (warp & 3) * 16, kC, a.fu.qk_eps, sh.gates[n % kRing].rk);
            warp_arrive(&sh.gfull[n % kRing]);
        }
        WAIT(sh.gfull[n % kRing], n / kRing);
        if (!decayed_values<NORM>(sm + st * kSegStage + kTile, sm + kSegV3 + b * kTile, sh.gates[n % kRing], warp, tm_vhi + b * 64, tm_vlo + b * 64, sh.vready[b],
                                  sh.vfree[b], n / 2))
            goto died;
        const bool stop = sh.stop[n % kTold];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.gempty[n % kRing]);
        if (stop) c0 = 0;
        END_SEGMENTS
    } else if (warp < 16) {
        more_registers<kSegSums>();
        FOR_FULL_SEGMENTS
        float2 S[kDim / 2];
#pragma unroll
        for (int k = 0; k < kDim / 2; ++k) S[k] = make_float2(0.f, 0.f);
        FOR_CHUNKS
        WAIT(sh.dfull[b], n / 2);
        tc::tc_fence_after();
        add_products(S, make_float2(1.f, 1.f), tm + b * 128 + lane_base(warp));
        const bool stop = sh.stop[n % kTold];
        warp_arrive(&sh.dfree[b]);
        if (stop) c0 = 0;
        }
        store_column(S, a.seg_state + ((size_t)slot * a.H + h) * kDim * kDim + (warp & 3) * 32 + lane);
        }
    }
    goto done;
died:
    sh.dead = 1;
done:
    __syncwarp();
    if (warp == 1 || warp == 3) {
        if (tc::elect_one()) tc::mma_commit(&sh.drain);
        __syncwarp();
        tc::mbar_wait(&sh.drain, 0);
    }
    tc::tc_fence_before();
    __syncthreads();
    if (sh.dead && warp == 0) {
        for (int i = 0; i < kSegStages; ++i)
            for (int p = 0; p < 2; ++p) tc::mbar_wait(&sh.full[i], p, 1000000);
    }
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tm, 512);
    if (sh.dead && threadIdx.x == 0) atomicExch(a.status, (int32_t)KDA_ERR_TIMEOUT);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// [total, heads, 128] bf16 tensor in boxes of 64 channels of one head of a chunk's tokens, 128-byte swizzle.
bool make_map(CUtensorMap *map, const void *base, int total, int heads) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)kDim, (cuuint64_t)heads, (cuuint64_t)total};
    cuuint64_t strides[2] = {(cuuint64_t)kDim * 2, (cuuint64_t)heads * kDim * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)kC};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether a kernel was built with the registers that its warpgroups share out.
template <auto Kernel>
cudaError_t enough_registers(int threads, int wanted) {
    static const int regs = [] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, Kernel) == cudaSuccess ? (at.numRegs + 7) / 8 * 8 : 0;
    }();
    return regs * threads >= wanted ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <bool NORM, bool GATE>
cudaError_t launch_out(const CUtensorMap *m, const Args &a, int grid, cudaStream_t st) {
    cudaError_t e = enough_registers<linear_out_tc<NORM, GATE>>(kOutThreads, kOutRegs);
    if (e == cudaSuccess) e = allow_smem<linear_out_tc<NORM, GATE>>(kOutSmem);
    return e != cudaSuccess ? e : launch_dependent(linear_out_tc<NORM, GATE>, dim3(grid), dim3(kOutThreads), kOutSmem, st, m[0], m[1], m[2], m[3], m[4], a);
}
template <bool NORM>
cudaError_t launch_segment(const CUtensorMap *m, const Args &a, int grid, cudaStream_t st) {
    cudaError_t e = enough_registers<linear_segment_tc<NORM>>(kSegThreads, kSegRegs);
    if (e == cudaSuccess) e = allow_smem<linear_segment_tc<NORM>>(kSegSmem);
    return e != cudaSuccess ? e : launch_dependent(linear_segment_tc<NORM>, dim3(grid), dim3(kSegThreads), kSegSmem, st, m[1], m[2], a);
}

}  // namespace

cudaError_t launch_linear_tc(const linear::Args &args, cudaStream_t st) {
    Args a = args;
    CUtensorMap m[5] = {};
    // (a map of an empty tensor cannot be made; with no tokens nothing is copied and any map will do)
    if (a.total > 0 && (!make_map(&m[0], a.q, a.total, a.Hqk) || !make_map(&m[1], a.k, a.total, a.Hqk) || !make_map(&m[2], a.v, a.total, a.H) ||
                        !make_map(&m[3], a.o, a.total, a.H) || !make_map(&m[4], a.fu.gate ? a.fu.gate : a.o, a.total, a.H)))
        return cudaErrorInvalidValue;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.slots * a.H;
    const int grid = (int)(units < sms ? units : sms);
    a.first = 1;
    a.withheld = testing_fault() == kFaultNoPublish;
    if (a.total > a.seg) {  // some document may have more than one segment
        e = a.fu.qk_norm ? launch_segment<true>(m, a, grid, st) : launch_segment<false>(m, a, grid, st);
        if (e == cudaSuccess) e = launch_linear_chain(a, kDim, st);
        if (e != cudaSuccess) return e;
        a.first = 0;
    } else {
        a.ticket = nullptr;
    }
    if (a.fu.qk_norm) return a.fu.gate ? launch_out<true, true>(m, a, grid, st) : launch_out<true, false>(m, a, grid, st);
    return a.fu.gate ? launch_out<false, true>(m, a, grid, st) : launch_out<false, false>(m, a, grid, st);
}

}  // namespace kda
