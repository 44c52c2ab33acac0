// kda_linear.cuh -- linear attention with one decay per head: what its kernels share.
//
// Per (document, head), with g one log-decay of a token (or of the head):
//     S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t.
// A run of tokens 1..n behind a state S is, with b_i = g_1 + ... + g_i,
//     o_i = exp(b_i) S^T q_i + sum_{j <= i} exp(b_i - b_j) (q_i . k_j) v_j,
//     S_n = exp(b_n) S + sum_j exp(b_n - b_j) k_j v_j^T,
// all exponents at most 0 where no log-decay is positive, so nothing overflows on the way.
//
// A document of more than `seg` tokens is split into segments that run side by side: a first kernel forms what each
// adds to the state by its end, a second chains those into the state before each segment, and the last forms the
// outputs.  Segments are numbered without a table: document n owns slots cu[n] / seg + n and on, one for each of its
// segments (an empty document one): cu[n + 1] / seg + n + 1 is never below the end of that run, and the last slot is
// below total / seg + num_seqs.  The document of a slot is the last one whose first slot is not above it.
#pragma once

#include "kda_internal.cuh"

namespace kda {
namespace linear {

constexpr float kLog2e = 1.4426950408889634f;
// Log2-decays are taken as at least this: 2^-160 is 0 in fp32 (down to its smallest subnormal), as a decay of minus
// infinity is, and differences of their sums stay numbers.  (At most its opposite, which is infinite in fp32.)
constexpr float kMinLog2 = -160.f;

// A token's log-decay in base 2 (NaN stays NaN).
__device__ __forceinline__ float log2_decay(float g) {
    const float x = g * kLog2e;
    return x < kMinLog2 ? kMinLog2 : x > -kMinLog2 ? -kMinLog2 : x;
}

// A factor 2^log2 that is multiplied in again and again (one decay for a head: each chunk's, stage's or segment's).  Rounded once
// and for all, its error adds up: S of 65536 tokens off by up to 3e-5 of its size, after 1024 factors.  So it is one of the two
// floats beside the true value each time, the upper one as often as that is near it: every product of them is right to one step.
struct Repeated {
    float down, up;
    uint32_t part, sum;  // how far up the true value is, in steps of 2^-32, and the parts so far
    static __device__ Repeated of(double log2) {
        const double x = exp2(log2);
        Repeated r;
        r.down = r.up = (float)x;
        r.part = r.sum = 0;
        if (x < 1e38) {
            r.down = __double2float_rd(x);
            r.up = __uint_as_float(__float_as_uint(r.down) + 1);
            r.part = __double2uint_rd((x - r.down) / ((double)r.up - r.down) * 4294967296.0);
        }
        return r;
    }
    __device__ float next() {
        sum += part;
        return sum < part ? up : down;
    }
    // The factor of the use behind `before` others.
    __device__ float at(uint32_t before) const { return before * part + part < part ? up : down; }
};

// Whether cu_seqlens describes num_seqs documents of total tokens in all; every thread of the block calls it and gets
// the answer.
__device__ __forceinline__ bool valid_table(const int32_t *__restrict__ cu, int num_seqs, int total) {
    bool ok = true;
    for (int n = threadIdx.x; n <= num_seqs; n += blockDim.x) {
        const int here = cu[n];
        ok = ok && here >= 0 && here <= total;
        if (n == 0) ok = ok && here == 0;
        ok = ok && (n == num_seqs ? here == total : here <= cu[n + 1]);
    }
    return __syncthreads_and(ok);
}

struct Segment {
    int doc, t0, len;   // document, first token, tokens (0 for an empty document)
    int index, count;   // which of its document's segments it is, and of how many
    bool first, last;   // of them
};

// The segment of a slot; false if the slot has none.  Called by a whole warp: 32 documents are looked at at once.
__device__ __forceinline__ bool find_segment(const int32_t *__restrict__ cu, int num_seqs, int seg, int slot, Segment *s) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = num_seqs;  // the document is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const bool below = lane * step < n && cu[at] / seg + at <= slot;
        const int hit = __popc(__ballot_sync(0xffffffffu, below)) - 1;  // the first is always below
        lo += hit * step;
        n = min(step, n - hit * step);
    }
    const int begin = cu[lo], len = cu[lo + 1] - begin, i = slot - (begin / seg + lo), count = len > seg ? (len + seg - 1) / seg : 1;
    if (i >= count) return false;
    s->doc = lo;
    s->t0 = begin + i * seg;
    s->len = min(seg, len - i * seg);
    s->index = i;
    s->count = count;
    s->first = i == 0;
    s->last = i == count - 1;
    return true;
}

// Where a segment's state begins: its document's incoming state (null: zeros), or what the chain left in the slot
// before it.  With S_final in S0's place the last segment's end could overtake the first one's start, so the chain
// leaves a copy of S0 in the document's last slot, which has no other use.
struct Args;
__device__ __forceinline__ const float *segment_start(const Args &a, const Segment &s, int slot, int h, size_t state);

// Tokens of a segment, which are chosen without the documents' lengths.  Tensor cores: one document is cut into as many
// segments of all heads as there are SMs, or a small multiple of that where they do not fit the SMs well, of 256 tokens at
// least.  Several make segments of their own by ending: the batch is cut into as many as leave an SM four in all, so that
// the longest document leaves no SM alone for long, of 512 tokens at least (8 documents at random places, 33000 tokens x 32 heads: 278 us
// in pieces of 3008 tokens, 315 of 8256, 313 of 1216).  From 608 / H documents on that splits none, which suits equal ones (18 x 1833
// tokens x 32 heads: 207 us, in pieces of 1216 310) and not a long one among short (16 x 1000 and 17000: 540 us and 276).
//
// CUDA cores, which take a token some ten times as long: four segments an SM, of 64 tokens at least at d = 128.  Below that a
// state is a quarter or less, and segments are short where there are few tokens (32 at least: d = 64, fp32, 5 heads, 400 tokens
// 13.9 us for 19.7; 1501 tokens 27.4 for 26.5, at d = 128 80.6 for 53.6), and eight an SM where those still have 64 tokens and the four
// have 128 (33000 tokens x 32 heads, d = 64, bf16, 1200 us for 1450; 4096 x 16, d = 128, fp32, 351 for 293).
inline int plan_segment(int64_t total, int64_t num_seqs, int64_t H, int d, bool tensor_cores) {
    constexpr int64_t kSms = 152;
    const auto cut = [&](int64_t parts, int64_t unit, int64_t least) {
        const int64_t seg = parts < 1 ? total : ((total + parts - 1) / parts);
        return seg < least ? least : (seg + unit - 1) / unit * unit;
    };
    int64_t seg;
    if (tensor_cores && num_seqs > 1) {
        seg = cut(4 * kSms / H - num_seqs, 64, 512);
    } else if (tensor_cores) {
        int64_t parts = 0;
        for (int64_t r = 1; r <= 3; ++r) {
            parts = r * kSms / H;
            if (10 * parts * H >= 9 * r * kSms) break;
        }
        seg = cut(parts, 64, 256);
    } else if (d == 128) {
        seg = cut(4 * kSms / H, 64, 64);
    } else {
        seg = cut(4 * kSms / H, 32, 32);
        if (seg >= 128) seg = cut(8 * kSms / H, 32, 64);
    }
    return (int)(seg < 0x7fffffc0 ? seg : 0x7fffffc0);
}

struct Args {
    const void *q, *k, *v;
    const float *g;       // [total, H], or [H] where !per_token
    int per_token;
    const int32_t *cu;
    int num_seqs, total, H, Hqk;  // head h of v reads head h / (H / Hqk) of q and k
    int seg, slots;       // tokens of a segment (a multiple of 64, or 32 on the CUDA cores), slots of segments
    const float *S0;      // [num_seqs, H, d, d] or null
    void *o;
    float *S_final;       // or null
    float *seg_state;     // [slots, H, d, d]: first what a segment adds, then the state behind it
    float *seg_decay;     // [slots, H]: the product of its decays
    int32_t *status;
    int32_t *ticket;      // the output kernel's next unit (null: units are dealt out in turn)
    int aliased;          // S_final is S0: a document of several segments starts from a copy of it
    int first;            // whether the kernel is its call's first, which sets the status word
    int withheld;         // in tests of waits that run out only (tensor cores): no chunk's decays are published
    Fusion fu;
};

__device__ __forceinline__ const float *segment_start(const Args &a, const Segment &s, int slot, int h, size_t state) {
    if (s.first && !(a.aliased && s.count > 1)) return a.S0 ? a.S0 + ((size_t)s.doc * a.H + h) * state : nullptr;
    return a.seg_state + ((size_t)(s.first ? slot + s.count - 1 : slot - 1) * a.H + h) * state;
}

// Workspace: the status word and the ticket (256 bytes), then the segments' decays and states.
constexpr int kTicketWord = 32;
struct Layout {
    size_t decay_off, state_off, total;
};
inline Layout layout(int64_t slots, int64_t H, int d, bool split) {
    Layout l;
    l.decay_off = 256;
    l.state_off = l.decay_off + (split ? align256((size_t)slots * H * 4) : 0);
    l.total = l.state_off + (split ? (size_t)slots * H * d * d * 4 : 0);
    return l;
}

}  // namespace linear

// Chunked linear attention (kda_linear_tc.cu: bf16, d = 128; kda_linear_simt.cu: the rest), and the chaining of the
// segments' states between its two passes.
cudaError_t launch_linear_tc(const linear::Args &a, cudaStream_t st);
cudaError_t launch_linear_simt(const linear::Args &a, int d, kda_dtype dt, cudaStream_t st);
cudaError_t launch_linear_chain(const linear::Args &a, int d, cudaStream_t st);
// One token of each listed slot of a pool (kda_linear_decode.cu).
struct LinearDecodeArgs {
    const void *q, *k, *v;
    const float *g;
    int per_token;
    const int32_t *idx;  // or null: sequence i is slot i
    int num_active, num_slots, H, Hqk, d;
    float *S;
    void *o;
    int32_t *status;
    Fusion fu;
};
cudaError_t launch_linear_decode(const LinearDecodeArgs &a, kda_dtype dt, cudaStream_t st);
// Rotary positions (kda_rope.cu).
struct RopeArgs {
    const void *q, *k;
    const int32_t *positions;
    const unsigned long long *steps;
    int total, Hq, Hk, d, rot, interleaved;
    float scale;
    void *q_out, *k_out;
};
cudaError_t launch_rope(const RopeArgs &a, kda_dtype dt, cudaStream_t st);

}  // namespace kda
