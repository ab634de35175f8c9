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

// Workgroup barrier behind this wave's own LDS accesses.  (A fence would also
// wait for stores and LDS DMA.)
__device__ __forceinline__ void bar() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// First token of sequence n (n = N: the end of the last one).
__device__ __forceinline__ int64_t seq_start(const ChunkParams &p, int n) {
    return p.cu ? min((int64_t)max(p.cu[n], 0), p.total) : p.total / p.N * n;
}

constexpr int kFactorTokens = 64;  // most tokens of a chunk

// Factors of one chunk: bh + bl (the decay sums, base 2), eb = 2^b, w = 2^(b_n - b)
// (0 past the sequence), 2^(b_n) last.
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

// x: the log-decay of token `lane` of the chunk (ignored past its n tokens).
__device__ __forceinline__ void chunk_factors(float x, Factors *f, int n, int lane) {
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
    f->w[lane] = lane < n ? exp2_fast((float)(e - b)) : 0.f;
    if (lane == 0) f->total = exp2_fast((float)e);
}

}  // namespace kda
