// kda_linattn.h -- shared parts of the chunked linear-attention kernels.
#pragma once

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

struct ChunkParams {
    const void *q, *k, *v;
    const float *g;
    const void *s_in;
    void *s_out, *o;
    const int32_t *cu, *slots;
    int64_t total, qs, ks, vs, gs;  // strides in elements; gs 0: one decay per head
    int N, H, rep, num_slots, dv, tiles, units;
    int state_bf16;
    float scale;
    // segments: tokens in each (0: whole sequences), their number, the states they
    // start from in accumulator order and their decay products, both [segment][head]
    int seg, segs;
    int joined;  // a scan joins them; else every segment sums the ones before it
    float *ws, *wdec;
};

inline ChunkParams chunk_params(const kda_linattn_prefill_args *a) {
    ChunkParams p = {};
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->log_decay;
    p.s_in = a->state_in; p.s_out = a->state_out; p.o = a->o; p.cu = a->cu_seqlens;
    p.slots = a->state_slots; p.num_slots = a->num_slots;
    p.total = a->total_tokens; p.N = a->num_seqs; p.H = a->num_heads; p.rep = a->num_heads / a->num_k_heads;
    p.qs = a->q_stride; p.ks = a->k_stride; p.vs = a->v_stride;
    p.gs = (a->flags & KDA_F_DECAY_PER_HEAD) ? 0 : a->num_heads;
    p.dv = a->head_dim_v; p.state_bf16 = (a->flags & KDA_F_STATE_BF16) != 0; p.scale = a->scale;
    return p;
}

// The workspace of a plan: (segments + 1) x H states, then the decay products.
inline void use_segments(ChunkParams &p, const kda_linattn_prefill_args *a, const LinattnPlan &plan) {
    p.seg = plan.tokens;
    p.segs = (int)plan.segments;
    p.joined = plan.longest > kJoinSegments;
    p.ws = static_cast<float *>(a->workspace);
    p.wdec = p.ws + (size_t)(plan.segments + 1) * p.H * a->head_dim_k * p.dv;
}
// Joins the segments' states along every sequence (`elems` floats each).
hipError_t launch_segment_scan(const ChunkParams &p, int elems, hipStream_t s);

// Workgroup barrier behind this wave's own LDS accesses.  (A fence would also
// wait for stores and LDS DMA.)
__device__ __forceinline__ void bar() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// First token of sequence n (n = N: the end of the last one).
__device__ __forceinline__ int64_t seq_start(const ChunkParams &p, int n) {
    return p.cu ? min((int64_t)max(p.cu[n], 0), p.total) : p.total / p.N * n;
}

// Segments are numbered with room for one partial one per sequence: sequence n's
// begin at seq_start / seg + n, and numbers past its last are unused.
__device__ __forceinline__ int seg_base(const ChunkParams &p, int n) { return (int)(seq_start(p, n) / p.seg) + n; }

// The sequence that segment number s belongs to: sixty-four probes at a time.
__device__ __forceinline__ int seg_seq(const ChunkParams &p, int s, int lane) {
    int lo = 0, cnt = p.N;
    while (cnt > 1) {
        const int step = (cnt + 63) / 64, i = lo + lane * step;
        const bool below = i < lo + cnt && seg_base(p, i) <= s;
        const int m = __popcll(__ballot(below));
        lo += m > 1 ? (m - 1) * step : 0;
        cnt = min(step, p.N - lo);
    }
    return lo;
}

// What a workgroup works on, from its block index: segment s (a whole sequence
// without segments), number j of its sequence's `nseg`.  The rep * tiles workgroups
// that read the same keys are `units` neighbours on one XCD (blocks go round the
// eight XCDs), where they share its L2.
struct Work {
    int n, h, tile, s, j, nseg;
    int64_t t0;
    int len;
};
__device__ __forceinline__ bool locate(const ChunkParams &p, Work &w, int lane) {
    const int U = p.rep * p.tiles, xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
    const int unit = (idx / U) * 8 + xcd, member = idx % U;
    if (unit >= p.units) return false;
    const int Hk = p.H / p.rep;
    w.s = unit / Hk;
    w.h = (unit - w.s * Hk) * p.rep + member / p.tiles;
    w.tile = member % p.tiles;
    w.n = p.seg ? __builtin_amdgcn_readfirstlane(seg_seq(p, w.s, lane)) : w.s;
    w.t0 = seq_start(p, w.n);
    w.len = (int)max(seq_start(p, w.n + 1) - w.t0, (int64_t)0);
    w.j = 0;
    w.nseg = 1;
    if (p.seg) {
        w.j = w.s - seg_base(p, w.n);
        w.nseg = max((w.len + p.seg - 1) / p.seg, 1);
        if (w.j < 0 || w.j >= w.nseg) return false;
        w.t0 += (int64_t)w.j * p.seg;
        w.len = min(w.len - w.j * p.seg, p.seg);
    }
    return true;
}

constexpr int kFactorTokens = 64;  // most tokens of a chunk

// Factors of one chunk: bh + bl (the decay sums, base 2), eb = 2^b, w = 2^(b_n - b), 2^(b_n)
// last; w and the last also over `after`, the sum of the chunks behind it.  Rows past the
// sequence repeat its last token, whose w is 1, or hold zeros: their w of 2^-60 adds 2^-54 of
// that token's product at most, which fp32 does not see, where a zero would make NaN of an
// infinity in it.
struct Factors {
    float bh[kFactorTokens], bl[kFactorTokens], eb[kFactorTokens], w[kFactorTokens], total, pad[3];
};

// DPP move of a double, zero where a lane has no source or its row is masked off.
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_f64(double x) {
    typedef __attribute__((ext_vector_type(2))) int i32x2;
    const i32x2 v = __builtin_bit_cast(i32x2, x);
    i32x2 r;
    r.x = __builtin_amdgcn_update_dpp(0, v.x, CTRL, ROWS, 0xf, false);
    r.y = __builtin_amdgcn_update_dpp(0, v.y, CTRL, ROWS, 0xf, false);
    return __builtin_bit_cast(double, r);
}
__device__ __forceinline__ double lane63_f64(double x) {
    typedef __attribute__((ext_vector_type(2))) int i32x2;
    i32x2 v = __builtin_bit_cast(i32x2, x);
    v.x = __builtin_amdgcn_readlane(v.x, 63);
    v.y = __builtin_amdgcn_readlane(v.y, 63);
    return __builtin_bit_cast(double, v);
}

// x: the log-decay of token `lane` of the chunk (ignored past its n tokens).  Returns
// the chunk's sum.
__device__ __forceinline__ double chunk_factors(float x, Factors *f, int n, int lane, double after = 0.0) {
    x = x > 0.f ? 0.f : x;                   // NaN stays
    x = x < -1e6f ? -1e6f : x;               // 2^(-1e6) is 0 as well; sums stay finite
    double b = lane < n ? (double)x * 1.4426950408889634 : 0.0;
    b += dpp_f64<0x111, 0xf>(b);  // row_shr 1, 2, 4, 8: sums inside 16 lanes
    b += dpp_f64<0x112, 0xf>(b);
    b += dpp_f64<0x114, 0xf>(b);
    b += dpp_f64<0x118, 0xf>(b);
    b += dpp_f64<0x142, 0xa>(b);  // lane 15 and 47 into the next 16
    b += dpp_f64<0x143, 0xc>(b);  // lane 31 into the upper half
    const double e = lane63_f64(b);
    const float hi = (float)b;
    f->bh[lane] = hi;
    f->bl[lane] = (float)(b - (double)hi);
    f->eb[lane] = exp2_fast(hi);
    f->w[lane] = lane < n ? exp2_fast((float)(e - b + after)) : 0x1p-60f;
    if (lane == 0) f->total = exp2_fast((float)(e + after));
    return e;
}

}  // namespace kda
