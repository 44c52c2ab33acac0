// kda_linear_tc.cu -- chunked linear attention on the tensor cores: bf16, d = 128.
//
// A document is walked in chunks of 64 tokens.  With S the state before a chunk and b, w the chunk's decays,
//     P_ij = 2^(b_i - b_j) (q_i . k_j)        (j <= i, else 0)
//     O^T  = 2^(b_i) S^T Q^T + V^T P^T
//     S^T <- 2^(b_64) S^T + V'^T K,           V'_j = 2^(b_64 - b_j) v_j
// so each product has 128 rows (the value dimension) or the chunk's 64 tokens, and S^T stays in tensor memory for a
// whole segment.  q, k, v are read once, o is written once: 1 KB a token and head against 98 kFLOP, so HBM bounds
// it and the work per chunk only has to hide behind the copies (a CTA with its SM's share of HBM takes 1.45 us a
// chunk).  What a CTA does is spread over warps that each do one thing, chunk after chunk, across segments:
//     warps 0-1    P: Q K^T from tensor memory, times the decays, to shared memory in bf16
//     warp 2       copies of q, k, v (and of the output gate) by TMA, three chunks ahead
//     warp 3       issues all MMAs
//     warps 4-7    V': v times its decay, in two bf16 parts, to tensor memory (the A operand of the state's product)
//     warps 8-11   S: the state's decay in place, and its bf16 copy (the A operand of S^T Q^T)
//     warps 12-15  O: the two parts of o added, normalised, to shared memory and out by TMA
//     warp 16      the decays' sums; warps 17-18 the norms of q and k (fused normalisation only)
//
// Roundings to bf16: P and the copy of S, which only reach o, itself rounded to bf16 (each adds an error of the size
// of that rounding in its part of o).  V' reaches the state, which is fp32: it is taken in two parts (16 bits of 24).
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
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kRing = 4;  // chunks whose decays are kept

// A wait that ran out ends the whole CTA: everyone polls `dead`.
__device__ __forceinline__ bool wait_or_dead(uint64_t *bar, uint32_t parity, volatile int *dead) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = tc::globaltimer_ns();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (tc::mbar_try_wait(bar, parity)) return true;
        if (*dead) return false;
        if (tc::globaltimer_ns() - t0 > kWaitNs) {
            *dead = 1;
            return false;
        }
    }
}
#define WAIT(bar, n_uses) \
    if (!__all_sync(0xffffffffu, wait_or_dead(&(bar), (uint32_t)(n_uses) & 1u, &sh.dead))) goto done

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

// What the other warps need of a chunk's decays (in base 2) and norms.
struct __align__(16) Gates {
    float b_hi[kC], b_lo[kC];  // sums of log-decays from the chunk's start, in two parts
    float in[kC];              // 2^b: decay of the incoming state
    float out[kC];             // 2^(b_64 - b): decay to the chunk's end; 0 behind the segment
    float rq[kC], rk[kC];      // 1 / norm of q and k (fused normalisation only)
    float all, pad[3];         // 2^b_64
};

struct OutShared {
    Gates gates[kRing];
    float red[4][kC];
    float rms[kC];
    uint64_t full[3], empty[3];           // q, k, v of a chunk
    uint64_t gfull[kRing], gempty[kRing];
    uint64_t fixed;                       // rows behind a segment cleared
    uint64_t pfull[2], pready[2], ofull[2], ofree[2];
    uint64_t vready, sready, kv;
    uint64_t zfull[3], zfree[3];          // output tiles (and the gate's values before them)
    uint64_t drain;
    uint32_t tmem;
    volatile int dead;
};
constexpr int kStage = 3 * kTile;
constexpr int kOutP = 3 * kStage, kOutO = kOutP + 2 * 8192, kOutShared = kOutO + 3 * kTile;
constexpr int kOutSmem = kOutShared + (int)sizeof(OutShared) + 1024;
static_assert(kOutSmem <= 232448, "shared memory of a CTA");
constexpr int kOutThreads = 19 * 32;

// Tensor memory: S^T in fp32 and bf16, V'^T in two parts, two buffers each of P (then V^T P^T) and S^T Q^T.
enum : uint32_t { kTmS = 0, kTmSb = 128, kTmVhi = 192, kTmVlo = 224, kTmP = 256, kTmO = 384 };

constexpr uint64_t kKmajor = tc::smem_desc_base(16, 1024, tc::SW_128B);
constexpr uint64_t kMNmajor = tc::smem_desc_base(8192, 1024, tc::SW_128B);
constexpr uint32_t kId64 = tc::idesc_bf16_f32(128, 64, false, false);

__device__ __forceinline__ uint32_t lane_base(int warp) { return (uint32_t)((warp & 3) * 32) << 16; }

// Sums of log2-decays of a chunk's `n` tokens: lane l holds tokens 2l and 2l + 1 (x0, x1; 0 behind the segment).
// Sums in 64 bits: behind a token that forgets everything, differences of small decays have to survive.
struct Sums {
    double b0, b1, all;
};
__device__ __forceinline__ Sums chunk_sums(float x0, float x1) {
    const int lane = threadIdx.x & 31;
    double s = (double)x0 + (double)x1;
    const double own = s;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += up;
    }
    Sums r;
    r.b0 = s - own + (double)x0;
    r.b1 = s;
    r.all = __shfl_sync(0xffffffffu, s, 31);
    return r;
}

// 1 / sqrt(sum of squares + eps) of the tile's 64 rows, two rows a lane.
__device__ __forceinline__ void row_norms(const uint8_t *tile, float eps, float *out) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int r = lane; r < kC; r += 32) {
        float ss = 0.f;
#pragma unroll 4
        for (int c = 0; c < 16; ++c) {
            const uint4 x = *reinterpret_cast<const uint4 *>(tile + (c >> 3) * 8192 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ss = fmaf(bf16_lo(u[i]), bf16_lo(u[i]), ss);
                ss = fmaf(bf16_hi(u[i]), bf16_hi(u[i]), ss);
            }
        }
        out[r] = rsqrtf(ss + eps);
    }
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

// This thread's lane of V'^T (value dimension 32 (warp % 4) + lane) for the chunk's tokens, in two bf16 parts.
template <bool NORM>
__device__ __forceinline__ void decayed_values(const uint8_t *v, const Gates &g, int n, int warp, uint32_t hi_col, uint32_t lo_col) {
    const int dv = (warp & 3) * 32 + (threadIdx.x & 31);
    const uint8_t *col = v + (dv >> 6) * 8192;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int j = half * 32 + 2 * i;
            float w0 = g.out[j], w1 = g.out[j + 1];
            if (NORM) {
                w0 *= g.rk[j];
                w1 *= g.rk[j + 1];
            }
            const float v0 = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(col + tc::sw128_offset(j, dv & 63)));
            const float v1 = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(col + tc::sw128_offset(j + 1, dv & 63)));
            const float x0 = j < n ? w0 * v0 : 0.f, x1 = j + 1 < n ? w1 * v1 : 0.f;
            hi[i] = pack_bf16(x0, x1);
            lo[i] = pack_bf16(x0 - bf16_lo(hi[i]), x1 - bf16_hi(hi[i]));
        }
        tc::tmem_st16(hi_col + lane_base(warp) + half * 16, hi);
        tc::tmem_st16(lo_col + lane_base(warp) + half * 16, lo);
    }
    tc::tmem_wait_st();
    tc::tc_fence_before();
}

// S^T += V'^T K over the chunk's tokens, both parts of V'.
__device__ __forceinline__ void mma_state(uint32_t s_col, uint32_t hi_col, uint32_t lo_col, const uint8_t *k, bool accumulate, bool elected) {
    constexpr uint32_t id = tc::idesc_bf16_f32(128, 128, false, true);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const uint64_t kd = tc::smem_desc(kMNmajor, tc::smem_u32(k + s * 2048));
        tc::mma_bf16_ts_warp(s_col, hi_col + s * 8, kd, id, accumulate || s > 0, elected);
        tc::mma_bf16_ts_warp(s_col, lo_col + s * 8, kd, id, true, elected);
    }
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
            tc::mbar_init(&sh.empty[i], 1);
            tc::mbar_init(&sh.zfull[i], 1);
            tc::mbar_init(&sh.zfree[i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(&sh.gfull[i], NORM ? 3 : 1);
            tc::mbar_init(&sh.gempty[i], 14);  // V', S and O warps, the two of P
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.pfull[i], 1);
            tc::mbar_init(&sh.pready[i], 2);
            tc::mbar_init(&sh.ofull[i], 1);
            tc::mbar_init(&sh.ofree[i], 4);
        }
        tc::mbar_init(&sh.fixed, 4);
        tc::mbar_init(&sh.vready, 4);
        tc::mbar_init(&sh.sready, 4);
        tc::mbar_init(&sh.kv, 1);
        tc::mbar_init(&sh.drain, 1);
        sh.dead = 0;
        tc::fence_mbar_init();
    }
    if (warp == 3) {
        tc::tmem_alloc(&sh.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::grid_dep_launch();
    tc::grid_dep_wait();
    tc::tc_fence_before();
    const bool valid = linear::valid_table(a.cu, a.num_seqs, a.total);  // also the barrier behind the set-up
    tc::tc_fence_after();
    if (a.first && blockIdx.x == 0 && threadIdx.x == 0) *a.status = valid ? (int32_t)KDA_OK : (int32_t)KDA_ERR_INVALID_ARG;
    const uint32_t tm = sh.tmem;
    const int units = valid ? a.slots * a.H : 0;
    const int share = a.H / a.Hqk;

#define FOR_SEGMENTS                                                                               \
    for (int u = blockIdx.x; u < units; u += gridDim.x) {                                          \
        Segment sg;                                                                                \
        const int slot = u / a.H, h = u - slot * a.H;                                              \
        if (!linear::find_segment(a.cu, a.num_seqs, a.seg, slot, &sg)) continue;                   \
        for (int c0 = 0; c0 < sg.len; c0 += kC, ++n) {                                             \
            [[maybe_unused]] const int t0 = sg.t0 + c0, rows = min(kC, sg.len - c0), st = n % 3;   \
            [[maybe_unused]] const bool last_chunk = c0 + kC >= sg.len;
#define END_SEGMENTS \
    }                \
    }

    int n = 0;  // chunks so far: each barrier's phase follows from it
    if (warp == 2) {
        // ---- copies
        FOR_SEGMENTS
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
        if (GATE) {
            if (n >= 3) WAIT(sh.zfree[st], n / 3 - 1);
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&sh.zfull[st], kTile);
                tc::tma_load_3d(sm + kOutO + st * kTile, &tm_z, 0, h, t0, &sh.zfull[st]);
            }
        }
        END_SEGMENTS
    } else if (warp == 3) {
        // ---- MMAs.  A chunk's Q K^T goes out before the products of the chunk before it, which wait for more.
        const bool one = tc::elect_one();
        int fixes = 0, prev = -1;
        auto rest = [&](int m) -> bool {  // the products of chunk m after its Q K^T
            const int s = m % 3, b = m & 1;
            const uint8_t *at = sm + s * kStage;
            if (!__all_sync(0xffffffffu, wait_or_dead(&sh.vready, m & 1, &sh.dead))) return false;
            if (!__all_sync(0xffffffffu, wait_or_dead(&sh.sready, m & 1, &sh.dead))) return false;
            tc::tc_fence_after();
            mma_state(tm + kTmS, tm + kTmVhi, tm + kTmVlo, at + kTile, true, one);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                tc::mma_bf16_ts_warp(tm + kTmO + b * 64, tm + kTmSb + i * 8,
                                     tc::smem_desc(kKmajor, tc::smem_u32(at + (i >> 2) * 8192 + (i & 3) * 32)), kId64, i > 0, one);
            if (one) tc::mma_commit(&sh.kv);
            if (!__all_sync(0xffffffffu, wait_or_dead(&sh.pready[b], (m >> 1) & 1, &sh.dead))) return false;
            tc::tc_fence_after();
            constexpr uint32_t id = tc::idesc_bf16_f32(128, 64, true, false);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                tc::mma_bf16_warp(tm + kTmP + b * 64, tc::smem_desc(kMNmajor, tc::smem_u32(at + 2 * kTile + i * 2048)),
                                  tc::smem_desc(kKmajor, tc::smem_u32(sm + kOutP + b * 8192 + i * 32)), id, i > 0, one);
            if (one) {
                tc::mma_commit(&sh.ofull[b]);
                tc::mma_commit(&sh.empty[s]);
            }
            __syncwarp();
            return true;
        };
        FOR_SEGMENTS
        WAIT(sh.full[st], n / 3);
        if (rows < kC) {
            WAIT(sh.fixed, fixes);
            ++fixes;
        }
        if (n >= 2) WAIT(sh.ofree[n & 1], n / 2 - 1);
        tc::tc_fence_after();
        {
            const uint8_t *at = sm + st * kStage;
            // (rows 64 to 127 of the result come of what follows the tile's half, and nobody reads them)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t off = (i >> 2) * 8192 + (i & 3) * 32;
                tc::mma_bf16_warp(tm + kTmP + (n & 1) * 64, tc::smem_desc(kKmajor, tc::smem_u32(at + off)),
                                  tc::smem_desc(kKmajor, tc::smem_u32(at + kTile + off)), kId64, i > 0, one);
            }
            if (one) tc::mma_commit(&sh.pfull[n & 1]);
            __syncwarp();
        }
        if (prev >= 0 && !rest(prev)) goto done;
        prev = n;
        END_SEGMENTS
        if (prev >= 0 && !rest(prev)) goto done;
    } else if (warp < 2) {
        // ---- P
        const int i = warp * 32 + lane;
        FOR_SEGMENTS
        WAIT(sh.gfull[n % kRing], n / kRing);
        WAIT(sh.pfull[n & 1], n / 2);
        tc::tc_fence_after();
        {
            const Gates &g = sh.gates[n % kRing];
            const float bh = g.b_hi[i], bl = g.b_lo[i];
            uint8_t *row = sm + kOutP + (n & 1) * 8192 + i * 128;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                float x[32];
                if (part <= warp) tc::tmem_ld32(tm + kTmP + (n & 1) * 64 + lane_base(warp) + part * 32, x);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t u[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float y[2];
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const int at = c * 8 + e * 2 + f, j = part * 32 + at;
                            float z = x[at] * ex2((bh - g.b_hi[j]) + (bl - g.b_lo[j]));
                            if (NORM) z *= g.rk[j];
                            y[f] = part <= warp && j <= i && j < rows ? z : 0.f;
                        }
                        u[e] = pack_bf16(y[0], y[1]);
                    }
                    *reinterpret_cast<uint4 *>(row + (((part * 4 + c) ^ (i & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
                }
            }
        }
        tc::fence_async_smem();
        tc::tc_fence_before();
        warp_arrive(&sh.pready[n & 1]);
        if (lane == 0) tc::mbar_arrive(&sh.gempty[n % kRing]);
        END_SEGMENTS
    } else if (warp < 8) {
        // ---- V'
        FOR_SEGMENTS
        WAIT(sh.full[st], n / 3);
        if (rows < kC) {
            clear_rows(sm + st * kStage + kTile, rows, threadIdx.x - 128, 128);
            clear_rows(sm + st * kStage + 2 * kTile, rows, threadIdx.x - 128, 128);
            tc::fence_async_smem();
            tc::named_barrier(1, 128);
            if (lane == 0) tc::mbar_arrive(&sh.fixed);
        }
        WAIT(sh.gfull[n % kRing], n / kRing);
        if (n >= 1) WAIT(sh.kv, n - 1);
        tc::tc_fence_after();
        decayed_values<NORM>(sm + st * kStage + 2 * kTile, sh.gates[n % kRing], rows, warp, tm + kTmVhi, tm + kTmVlo);
        warp_arrive(&sh.vready);
        if (lane == 0) tc::mbar_arrive(&sh.gempty[n % kRing]);
        END_SEGMENTS
    } else if (warp < 12) {
        // ---- S
        const int dv = (warp & 3) * 32 + lane;
        for (int u = blockIdx.x; u < units; u += gridDim.x) {
            Segment sg;
            const int slot = u / a.H, h = u - slot * a.H;
            if (!linear::find_segment(a.cu, a.num_seqs, a.seg, slot, &sg)) continue;
            const size_t doc_state = ((size_t)sg.doc * a.H + h) * kDim * kDim + dv;
            const float *init = linear::segment_start(a, sg, slot, h, (size_t)kDim * kDim);
            if (init) init += dv;
            if (sg.len == 0) {
                if (a.S_final)
                    for (int k = 0; k < kDim; ++k) a.S_final[doc_state + (size_t)k * kDim] = init ? init[(size_t)k * kDim] : 0.f;
                continue;
            }
            for (int c0 = 0; c0 < sg.len; c0 += kC, ++n) {
                WAIT(sh.gfull[n % kRing], n / kRing);
                const float all = sh.gates[n % kRing].all;
                if (c0 > 0) {
                    WAIT(sh.kv, n - 1);
                    tc::tc_fence_after();
                }
#pragma unroll 1
                for (int part = 0; part < 4; ++part) {
                    float x[32];
                    if (c0 == 0) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) x[k] = init ? init[(size_t)(part * 32 + k) * kDim] : 0.f;
                    } else {
                        tc::tmem_ld32(tm + kTmS + lane_base(warp) + part * 32, x);
                    }
                    uint32_t p[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        p[k] = pack_bf16(x[2 * k], x[2 * k + 1]);
                        x[2 * k] *= all;
                        x[2 * k + 1] *= all;
                    }
                    tc::tmem_st16(tm + kTmSb + lane_base(warp) + part * 16, p);
                    tc::tmem_st32(tm + kTmS + lane_base(warp) + part * 32, x);
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                warp_arrive(&sh.sready);
                if (lane == 0) tc::mbar_arrive(&sh.gempty[n % kRing]);
            }
            WAIT(sh.kv, n - 1);
            if (sg.last && a.S_final) {
                tc::tc_fence_after();
#pragma unroll 1
                for (int part = 0; part < 4; ++part) {
                    float x[32];
                    tc::tmem_ld32(tm + kTmS + lane_base(warp) + part * 32, x);
#pragma unroll
                    for (int k = 0; k < 32; ++k) a.S_final[doc_state + (size_t)(part * 32 + k) * kDim] = x[k];
                }
                tc::tc_fence_before();
            }
        }
    } else if (warp < 16) {
        // ---- O
        const int dv = (warp & 3) * 32 + lane;
        const float weight = GATE && a.fu.weight ? a.fu.weight[dv] : 1.f;
        FOR_SEGMENTS
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
            __nv_bfloat16 *col = reinterpret_cast<__nv_bfloat16 *>(tile) + dv;
            if constexpr (!GATE) {
#pragma unroll
                for (int part = 0; part < 4; ++part) {
                    float x[16], y[16];
                    tc::tmem_ld16x2(t1 + part * 16, t2 + part * 16, x, y);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const int i = part * 16 + k;
                        float z = fmaf(g.in[i], x[k], y[k]);
                        if (NORM) z *= g.rq[i];
                        col[i * kDim] = __float2bfloat16_rn(z);
                    }
                }
                tc::tc_fence_before();
                warp_arrive(&sh.ofree[n & 1]);
            } else {
                float z[kC], sq[kC];
#pragma unroll
                for (int part = 0; part < 4; ++part) {
                    float x[16], y[16];
                    tc::tmem_ld16x2(t1 + part * 16, t2 + part * 16, x, y);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const int i = part * 16 + k;
                        z[i] = fmaf(g.in[i], x[k], y[k]);
                        if (NORM) z[i] *= g.rq[i];
                        sq[i] = z[i] * z[i];
                    }
                }
                tc::tc_fence_before();
                warp_arrive(&sh.ofree[n & 1]);
                // sums over the warp's 32 value dimensions: each exchange halves the tokens that a lane holds
#pragma unroll
                for (int half = 32; half >= 2; half >>= 1) {
                    const bool up = lane & (half >> 1);
#pragma unroll
                    for (int i = 0; i < half; ++i) {
                        const float give = up ? sq[i] : sq[i + half], keep = up ? sq[i + half] : sq[i];
                        sq[i] = keep + __shfl_xor_sync(0xffffffffu, give, half >> 1);
                    }
                }
                // lane's bits 4..0 chose halves of 64, 32, 16, 8, 4 tokens: it holds tokens 2 lane and 2 lane + 1
                sh.red[warp & 3][2 * lane] = sq[0];
                sh.red[warp & 3][2 * lane + 1] = sq[1];
                tc::named_barrier(2, 128);
                if (threadIdx.x - 384 < kC) {
                    const int i = threadIdx.x - 384;
                    sh.rms[i] = rsqrtf(((sh.red[0][i] + sh.red[1][i]) + (sh.red[2][i] + sh.red[3][i])) * (1.f / kDim) + a.fu.out_eps);
                }
                tc::named_barrier(2, 128);
#pragma unroll
                for (int i = 0; i < kC; ++i)
                    col[i * kDim] = __float2bfloat16_rn(z[i] * sh.rms[i] * weight * sigmoidf(__bfloat162float(col[i * kDim])));
            }
        }
        if (lane == 0) tc::mbar_arrive(&sh.gempty[n % kRing]);
        tc::fence_async_smem();
        tc::named_barrier(2, 128);
        if (rows == kC) {
            if (threadIdx.x == 384) {
                tc::tma_store_3d(&tm_o, 0, h, t0, tile);
                tc::bulk_commit();
                tc::bulk_wait_read();
                tc::mbar_arrive(&sh.zfree[st]);
            }
        } else {
            for (int i = threadIdx.x - 384; i < rows * 16; i += 128)
                reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + ((size_t)(t0 + (i >> 4)) * a.H + h) * kDim)[i & 15] =
                    reinterpret_cast<const uint4 *>(tile)[i];
            tc::fence_async_smem();
            tc::named_barrier(2, 128);
            if (threadIdx.x == 384) tc::mbar_arrive(&sh.zfree[st]);
        }
        __syncwarp();
        END_SEGMENTS
    } else if (warp == 16) {
        // ---- decays
        FOR_SEGMENTS
        Gates &g = sh.gates[n % kRing];
        const int j = 2 * lane;
        float x0 = 0.f, x1 = 0.f;
        if (a.per_token) {
            if (j < rows) x0 = linear::log2_decay(a.g[(size_t)(t0 + j) * a.H + h]);
            if (j + 1 < rows) x1 = linear::log2_decay(a.g[(size_t)(t0 + j + 1) * a.H + h]);
        } else {
            const float x = linear::log2_decay(a.g[h]);
            if (j < rows) x0 = x;
            if (j + 1 < rows) x1 = x;
        }
        const Sums s = chunk_sums(x0, x1);
        if (n >= kRing) WAIT(sh.gempty[n % kRing], n / kRing - 1);
        {
            const float2 hi = make_float2((float)s.b0, (float)s.b1);
            reinterpret_cast<float2 *>(g.b_hi)[lane] = hi;
            reinterpret_cast<float2 *>(g.b_lo)[lane] = make_float2((float)(s.b0 - (double)hi.x), (float)(s.b1 - (double)hi.y));
            reinterpret_cast<float2 *>(g.in)[lane] = make_float2(exp2f(hi.x), exp2f(hi.y));
            reinterpret_cast<float2 *>(g.out)[lane] = make_float2(exp2f((float)(s.all - s.b0)), exp2f((float)(s.all - s.b1)));
            if (lane == 0) g.all = exp2f((float)s.all);
        }
        warp_arrive(&sh.gfull[n % kRing]);
        END_SEGMENTS
    } else if (NORM) {
        // ---- norms of q (warp 17) and k (warp 18)
        FOR_SEGMENTS
        WAIT(sh.full[st], n / 3);
        if (n >= kRing) WAIT(sh.gempty[n % kRing], n / kRing - 1);
        Gates &g = sh.gates[n % kRing];
        row_norms(sm + st * kStage + (warp - 17) * kTile, a.fu.qk_eps, warp == 17 ? g.rq : g.rk);
        warp_arrive(&sh.gfull[n % kRing]);
        END_SEGMENTS
    }
done:
    __syncwarp();
    if (warp == 3) {  // every MMA done before the tensor memory goes
        if (tc::elect_one()) tc::mma_commit(&sh.drain);
        __syncwarp();
        tc::mbar_wait(&sh.drain, 0);
    }
    if (threadIdx.x == 384) tc::bulk_wait_all();
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
// chunks are taken from the last to the first, so that every weight is known when its chunk is reached and the sum in
// tensor memory is never rescaled; it also leaves the segment's first rows in L2 for the pass that forms the outputs.
// Only k and v are read: 512 bytes a token and head.
//     warp 0  copies   warp 1  MMAs   warp 2  decays   warp 3  norms of k   warps 4-7, 8-11  V' of every other chunk
//     warps 12-15  the finished sums to memory
// ---------------------------------------------------------------------------
constexpr int kSegStages = 6;
struct SegShared {
    Gates gates[kRing];
    uint64_t full[kSegStages], empty[kSegStages];
    uint64_t gfull[kRing], gempty[kRing];
    uint64_t vready[2], vfree[2], sfull[2], sfree[2], drain;
    uint32_t tmem;
    volatile int dead;
};
constexpr int kSegStage = 2 * kTile;
constexpr int kSegShared = kSegStages * kSegStage;
constexpr int kSegSmem = kSegShared + (int)sizeof(SegShared) + 1024;
static_assert(kSegSmem <= 232448, "shared memory of a CTA");
constexpr int kSegThreads = 16 * 32;

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
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(&sh.gfull[i], NORM ? 2 : 1);
            tc::mbar_init(&sh.gempty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.vready[i], 4);
            tc::mbar_init(&sh.vfree[i], 1);
            tc::mbar_init(&sh.sfull[i], 1);
            tc::mbar_init(&sh.sfree[i], 4);
        }
        tc::mbar_init(&sh.drain, 1);
        sh.dead = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(&sh.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::grid_dep_launch();
    tc::grid_dep_wait();
    tc::tc_fence_before();
    const bool valid = linear::valid_table(a.cu, a.num_seqs, a.total);  // also the barrier behind the set-up
    tc::tc_fence_after();
    if (a.first && blockIdx.x == 0 && threadIdx.x == 0) *a.status = valid ? (int32_t)KDA_OK : (int32_t)KDA_ERR_INVALID_ARG;
    const uint32_t tm = sh.tmem, tm_vhi = tm + 256, tm_vlo = tm + 288;  // sums at 0 and 128, V' at 256 and 320
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

    int n = 0, m = 0;  // chunks and segments so far
    if (warp == 0) {
        FOR_FULL_SEGMENTS
        FOR_CHUNKS
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
    } else if (warp == 1) {
        const bool one = tc::elect_one();
        FOR_FULL_SEGMENTS
        if (m >= 2) WAIT(sh.sfree[m & 1], m / 2 - 1);
        FOR_CHUNKS
        WAIT(sh.full[st], n / kSegStages);
        WAIT(sh.vready[b], n / 2);
        tc::tc_fence_after();
        mma_state(tm + (m & 1) * 128, tm_vhi + b * 64, tm_vlo + b * 64, sm + st * kSegStage, c0 + kC < sg.len, one);
        if (one) {
            tc::mma_commit(&sh.empty[st]);
            tc::mma_commit(&sh.vfree[b]);
            if (c0 == 0) tc::mma_commit(&sh.sfull[m & 1]);
        }
        __syncwarp();
        }
        ++m;
        }
    } else if (warp == 2) {
        FOR_FULL_SEGMENTS
        double later = 0.0;  // the log-decays of the chunks behind this one
        FOR_CHUNKS
        Gates &g = sh.gates[n % kRing];
        float x0, x1;
        if (a.per_token) {
            x0 = linear::log2_decay(a.g[(size_t)(t0 + 2 * lane) * a.H + h]);
            x1 = linear::log2_decay(a.g[(size_t)(t0 + 2 * lane + 1) * a.H + h]);
        } else {
            x0 = x1 = linear::log2_decay(a.g[h]);
        }
        const Sums s = chunk_sums(x0, x1);
        if (n >= kRing) WAIT(sh.gempty[n % kRing], n / kRing - 1);
        reinterpret_cast<float2 *>(g.out)[lane] = make_float2(exp2f((float)(later + (s.all - s.b0))), exp2f((float)(later + (s.all - s.b1))));
        later += s.all;
        warp_arrive(&sh.gfull[n % kRing]);
        }
        if (lane == 0) a.seg_decay[(size_t)slot * a.H + h] = exp2f((float)later);
        }
    } else if (warp == 3) {
        if (NORM) {
            FOR_FULL_SEGMENTS
            FOR_CHUNKS
            WAIT(sh.full[st], n / kSegStages);
            if (n >= kRing) WAIT(sh.gempty[n % kRing], n / kRing - 1);
            row_norms(sm + st * kSegStage, a.fu.qk_eps, sh.gates[n % kRing].rk);
            warp_arrive(&sh.gfull[n % kRing]);
            END_SEGMENTS
        }
    } else if (warp < 12) {
        const int group = (warp >> 2) - 1;
        FOR_FULL_SEGMENTS
        FOR_CHUNKS
        if (b != group) continue;
        WAIT(sh.full[st], n / kSegStages);
        WAIT(sh.gfull[n % kRing], n / kRing);
        if (n >= 2) WAIT(sh.vfree[b], n / 2 - 1);
        tc::tc_fence_after();
        decayed_values<NORM>(sm + st * kSegStage + kTile, sh.gates[n % kRing], kC, warp, tm_vhi + b * 64, tm_vlo + b * 64);
        warp_arrive(&sh.vready[b]);
        if (lane == 0) tc::mbar_arrive(&sh.gempty[n % kRing]);
        END_SEGMENTS
    } else {
        FOR_FULL_SEGMENTS
        WAIT(sh.sfull[m & 1], m / 2);
        tc::tc_fence_after();
        float *to = a.seg_state + ((size_t)slot * a.H + h) * kDim * kDim + (warp & 3) * 32 + lane;
#pragma unroll 1
        for (int part = 0; part < 4; ++part) {
            float x[32];
            tc::tmem_ld32(tm + (m & 1) * 128 + lane_base(warp) + part * 32, x);
#pragma unroll
            for (int k = 0; k < 32; ++k) to[(size_t)(part * 32 + k) * kDim] = x[k];
        }
        tc::tc_fence_before();
        warp_arrive(&sh.sfree[m & 1]);
        ++m;
        }
    }
done:
    __syncwarp();
    if (warp == 1) {
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

// [total, heads, 128] bf16 tensor in boxes of a chunk's tokens of one head: halves of 64 channels with the 128-byte
// swizzle (operands of MMAs), or whole rows as they are (the output, and the gate).
bool make_map(CUtensorMap *map, const void *base, int total, int heads, bool operand) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)kDim, (cuuint64_t)heads, (cuuint64_t)total};
    cuuint64_t strides[2] = {(cuuint64_t)kDim * 2, (cuuint64_t)heads * kDim * 2};
    cuuint32_t box[3] = {operand ? 64u : (cuuint32_t)kDim, 1, (cuuint32_t)kC};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, operand ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool NORM, bool GATE>
cudaError_t launch_out(const CUtensorMap *m, const Args &a, int grid, cudaStream_t st) {
    const cudaError_t e = allow_smem<linear_out_tc<NORM, GATE>>(kOutSmem);
    return e != cudaSuccess ? e : launch_dependent(linear_out_tc<NORM, GATE>, dim3(grid), dim3(kOutThreads), kOutSmem, st, m[0], m[1], m[2], m[3], m[4], a);
}
template <bool NORM>
cudaError_t launch_segment(const CUtensorMap *m, const Args &a, int grid, cudaStream_t st) {
    const cudaError_t e = allow_smem<linear_segment_tc<NORM>>(kSegSmem);
    return e != cudaSuccess ? e : launch_dependent(linear_segment_tc<NORM>, dim3(grid), dim3(kSegThreads), kSegSmem, st, m[1], m[2], a);
}

}  // namespace

cudaError_t launch_linear_tc(const linear::Args &args, cudaStream_t st) {
    Args a = args;
    CUtensorMap m[5];
    // (a map of an empty tensor cannot be made; with no tokens nothing is copied and any map will do)
    const int rows = a.total > 0 ? a.total : 1;
    if (a.total > 0) {
        if (!make_map(&m[0], a.q, rows, a.Hqk, true) || !make_map(&m[1], a.k, rows, a.Hqk, true) || !make_map(&m[2], a.v, rows, a.H, true) ||
            !make_map(&m[3], a.o, rows, a.H, false) || !make_map(&m[4], a.fu.gate ? a.fu.gate : a.o, rows, a.H, false))
            return cudaErrorInvalidValue;
    }
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.slots * a.H;
    const int grid = (int)(units < sms ? units : sms);
    a.first = 1;
    if (a.total > a.seg) {  // some document may have more than one segment
        e = a.fu.qk_norm ? launch_segment<true>(m, a, grid, st) : launch_segment<false>(m, a, grid, st);
        if (e == cudaSuccess) e = launch_linear_chain(a, kDim, st);
        if (e != cudaSuccess) return e;
        a.first = 0;
    }
    if (a.fu.qk_norm) return a.fu.gate ? launch_out<true, true>(m, a, grid, st) : launch_out<true, false>(m, a, grid, st);
    return a.fu.gate ? launch_out<false, true>(m, a, grid, st) : launch_out<false, false>(m, a, grid, st);
}

}  // namespace kda
