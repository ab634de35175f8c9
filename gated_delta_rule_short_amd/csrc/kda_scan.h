// kda_scan.h -- what the gated scan's kernels share: decays and input factors, the cut
// of the packed tokens into tiles, and the chain of states from tile to tile.
#pragma once

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

constexpr int kWaves = 8;    // waves of a workgroup, one behind the other along the tokens
constexpr int kRows = 16;    // tokens of a wave
constexpr uint32_t kEmpty = 0xffffffffu, kState = 0xbf800000u;  // see chain_carry

struct ScanParams {
    const void *x, *g, *d;
    void *o, *dx, *dg;
    int64_t xs, gs, ds, os, dxs, dgs;  // elements per token
    const void *state_in;
    void *state_out;
    const float *dstate_out;
    float *dstate_in;
    const int32_t *cu, *slots;
    int64_t T, tiles;
    uint32_t *ticket;
    uint64_t *words;
    int N, C, groups, num_slots, state_bf16, polls;
};

constexpr float kLog2e = 1.4426950408889634f;

// log2(1 + e), 0 <= e <= 1, to 2e-7 of itself: a polynomial times e (least maximal
// relative error, by reweighted least squares).  The logarithm of a rounded 1 + e would
// lose e's low bits, and with them the memory of a gate near 1.
__device__ __forceinline__ float log2_1p(float e) {
    float q = 0.007549080532044172f;
    q = fmaf(q, e, -0.042566657066345215f);
    q = fmaf(q, e, 0.11285553127527237f);
    q = fmaf(q, e, -0.19711840152740479f);
    q = fmaf(q, e, 0.27564114332199097f);
    q = fmaf(q, e, -0.3584083914756775f);
    q = fmaf(q, e, 0.48069295287132263f);
    q = fmaf(q, e, -0.7213401794433594f);
    return e * fmaf(q, e, 1.4426950216293335f);
}

// 1 - exp(g) for g <= 0: the Taylor series near 0 (to 4e-8 of itself), where the
// difference from a rounded exponential would lose it.
__device__ __forceinline__ float one_minus_exp(float g) {
    float q = fmaf(g, 1.f / 720.f, 1.f / 120.f);
    q = fmaf(q, g, 1.f / 24.f);
    q = fmaf(q, g, 1.f / 6.f);
    q = fmaf(q, g, 0.5f);
    q = fmaf(q, g, 1.f);
    return g > -0.125f ? -g * q : 1.f - exp2_fast(g * kLog2e);
}

// Of one gate value: l = log2 a, c = 1 - a (only where it is used), and what follows.
template <int GATE, int INPUT> struct Factors {
    float l, c, b;
    bool clamped;
    __device__ __forceinline__ explicit Factors(float z) {
        if (GATE == KDA_GATE_LOG) {
            clamped = z > 0.f;
            const float g = clamped ? 0.f : z;  // NaN stays
            l = g * kLog2e;
            c = one_minus_exp(g);
        } else {
            clamped = false;
            const float y = z * kLog2e, s = log2_1p(exp2_fast(-fabsf(y)));
            l = fminf(y, 0.f) - s;                // log2 of 1 / (1 + e^-z)
            c = exp2_fast(-fmaxf(y, 0.f) - s);    // 1 / (1 + e^z)
        }
        b = INPUT == KDA_INPUT_PLAIN ? 1.f : INPUT == KDA_INPUT_COMPLEMENT ? c : __builtin_amdgcn_sqrtf(c * (2.f - c));
    }
    __device__ __forceinline__ float input(float x) const { return INPUT == KDA_INPUT_PLAIN ? x : b * x; }
    // dx = b dh;  dgate = dh a' (before - x q) with a' = da/dgate and q = -db/da
    __device__ __forceinline__ void gradient(float a, float dh, float before, float x, float &dx, float &dg) const {
        dx = INPUT == KDA_INPUT_PLAIN ? dh : b * dh;
        if (INPUT == KDA_INPUT_COMPLEMENT) before -= x;
        if (INPUT == KDA_INPUT_NORM) before -= b > 0.f ? x * (a * __builtin_amdgcn_rcpf(b)) : 0.f;
        dg = dh * (GATE == KDA_GATE_LOG ? a : a * c) * before;
        if (clamped) dg = 0.f;
    }
};

__device__ __forceinline__ float2 load_state(const void *p, size_t at, int bf16) {
    float2 h;
    if (bf16) Pair<__bf16>::load(static_cast<const __bf16 *>(p) + at, h.x, h.y);
    else Pair<float>::load(static_cast<const float *>(p) + at, h.x, h.y);
    return h;
}
__device__ __forceinline__ void store_state(void *p, size_t at, int bf16, float2 h) {
    if (bf16) Pair<__bf16>::store(static_cast<__bf16 *>(p) + at, h.x, h.y);
    else Pair<float>::store(static_cast<float *>(p) + at, h.x, h.y);
}

// A run's step (sum: log2 of its decay, add) continued by the step s of the run behind it.
__device__ __forceinline__ void append(float4 s, float2 &sum, float2 &add) {
    sum.x += s.x;
    sum.y += s.y;
    add.x = fmaf(exp2_fast(s.x), add.x, s.z);
    add.y = fmaf(exp2_fast(s.y), add.y, s.w);
}

struct TileId {
    int64_t start, len;     // the sequence's tokens
    int64_t m;              // number of the tile
    int n, group, index;    // sequence (-1: nothing to do), channel group, tile in the sequence
};

// Tokens of sequence n, kept inside the call's whatever cu_seqlens holds.
__device__ __forceinline__ void sequence(const ScanParams &p, int n, TileId &id) {
    seq_bounds(p.cu, p.T, p.N, n, id.start, id.len);
    id.start = min(max(id.start, (int64_t)0), p.T);
    id.len = min(max(id.len, (int64_t)0), p.T - id.start);
}

__device__ __forceinline__ TileId whole_sequence(const ScanParams &p) {
    TileId id = {};
    id.n = blockIdx.x / p.groups;
    id.group = blockIdx.x - id.n * p.groups;
    sequence(p, id.n, id);
    return id;
}

// First tile number of sequence n.  Tiles T / TILE + N suffice: a sequence of L tokens
// from s has (s + L) / TILE - s / TILE + 1 of them, at least ceil(L / TILE) and one.
template <int TILE> __device__ __forceinline__ int64_t first_tile(const ScanParams &p, int n) {
    return (p.cu ? min(max((int64_t)p.cu[n], (int64_t)0), p.T) : p.T / p.N * n) / TILE + n;
}

__device__ __forceinline__ int64_t uniform64(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// The tile that this workgroup takes: tickets count (tile, channel group), a tile behind
// the one that its state comes from, so that whatever a workgroup waits for belongs to a
// smaller ticket, held by a workgroup that runs or has run.  The smallest unfinished
// ticket never waits, hence every wait ends.
template <int TILE>
__device__ __forceinline__ TileId chained_tile(const ScanParams &p, int wave, int lane, TileId *shared, bool backward) {
    if (wave == 0) {
        TileId id = {};
        unsigned ticket = 0;
        if (lane == 0) ticket = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        ticket = __builtin_amdgcn_readfirstlane(ticket);
        const int64_t k = ticket / (unsigned)p.groups;
        id.group = ticket - (unsigned)k * p.groups;
        id.m = backward ? p.tiles - 1 - k : k;
        int lo = 0, hi = p.N;  // the last sequence whose first tile is at or before m
        while (hi - lo > 1) {
            const int step = (hi - lo + 63) / 64, at = lo + lane * step;
            const bool before = at < hi && (lane == 0 || first_tile<TILE>(p, at) <= id.m);
            lo += (__popcll(__ballot(before)) - 1) * step;
            hi = min(lo + step, hi);
        }
        const int64_t i = id.m - first_tile<TILE>(p, lo);
        id.n = lo;
        sequence(p, lo, id);
        id.index = (int)i;
        if (i < 0 || (i > 0 && i * TILE >= id.len)) id.n = -1;
        if (lane == 0) *shared = id;
    }
    __syncthreads();
    TileId id = *shared;
    id.start = uniform64(id.start);
    id.len = uniform64(id.len);
    id.m = uniform64(id.m);
    id.n = __builtin_amdgcn_readfirstlane(id.n);
    id.group = __builtin_amdgcn_readfirstlane(id.group);
    id.index = __builtin_amdgcn_readfirstlane(id.index);
    return id;
}

// The state before a tile (wave 0, two channels a lane).  `edge` is the tile index at
// which the chain begins, there with the state `h`; from it the chain runs towards the
// other end of the sequence.
//
// A tile first publishes its own step (P, H) and, once it knows the state before it, the
// state behind it.  Both are one 64-bit word for each channel, value and kind together,
// so relaxed atomics suffice and no cache is flushed: {P, H} with P >= 0 (a NaN has the
// usual bits), {kState, h}, or kEmpty from the clearing launch.  A tile reads its
// kLook predecessors at once; from the nearest that shows a state it goes forward with
// h -> P h + H, which is what those tiles compute themselves: the result does not depend
// on how far the others have come.
constexpr int kLook = 8;
__device__ __forceinline__ uint64_t word(uint32_t kind, float v) {
    return (uint64_t)__builtin_bit_cast(uint32_t, v) << 32 | kind;
}
__device__ __forceinline__ float word_value(uint64_t w) { return __builtin_bit_cast(float, (uint32_t)(w >> 32)); }
__device__ __forceinline__ uint32_t decay_bits(float p) {
    return p == p ? __builtin_bit_cast(uint32_t, p) : 0x7fc00000u;
}
__device__ __forceinline__ void publish(uint64_t *at, uint64_t a, uint64_t b) {
    __hip_atomic_store(at, a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(at + 1, b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int WAVES>
__device__ __forceinline__ float2 chain_carry(const ScanParams &p, const TileId &id, int lane, int edge, int tiles,
                                              const float4 (*steps)[64], float2 h) {
    float2 sum = {0.f, 0.f}, add = {0.f, 0.f};
#pragma unroll
    for (int q = 0; q < WAVES; ++q) append(steps[q][lane], sum, add);
    const float2 dec = {exp2_fast(sum.x), exp2_fast(sum.y)};
    const int64_t row = (int64_t)p.groups * 128;
    uint64_t *mine = p.words + id.m * row + id.group * 128 + 2 * lane;
    const int done = abs(id.index - edge), back = edge == 0 ? -1 : 1;  // tiles before this one; where they are
    const bool last = done == tiles - 1;
    if (done > 0) {
        if (!last) publish(mine, word(decay_bits(dec.x), add.x), word(decay_bits(dec.y), add.y));
        const int look = min(done, kLook);
        for (int polls = 0;; ++polls) {
            uint64_t wx[kLook], wy[kLook];
#pragma unroll
            for (int k = 0; k < kLook; ++k) {
                const uint64_t *at = mine + back * (int64_t)min(k + 1, look) * row;
                wx[k] = __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                wy[k] = __hip_atomic_load(at + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
            int found = -1;
            bool open = true;
#pragma unroll
            for (int k = 0; k < kLook; ++k)
                if (open && found < 0 && k < look) {
                    const uint32_t a = (uint32_t)wx[k], b = (uint32_t)wy[k];
                    if (__all(a == kState && b == kState)) found = k;
                    else if (!__all(a != kEmpty && b != kEmpty)) open = false;
                }
            if (found >= 0) {
#pragma unroll
                for (int k = kLook - 1; k >= 0; --k)
                    if (k <= found) {
                        const uint32_t a = (uint32_t)wx[k], b = (uint32_t)wy[k];
                        h.x = a == kState ? word_value(wx[k]) : fmaf(__builtin_bit_cast(float, a), h.x, word_value(wx[k]));
                        h.y = b == kState ? word_value(wy[k]) : fmaf(__builtin_bit_cast(float, b), h.y, word_value(wy[k]));
                    }
                break;
            }
            if (polls >= p.polls) {  // never reached by a correct chain; a wait that gives up says so
                h = make_float2(__builtin_nanf(""), __builtin_nanf(""));
                break;
            }
            __builtin_amdgcn_s_sleep(2);
        }
    }
    if (!last) publish(mine, word(kState, fmaf(dec.x, h.x, add.x)), word(kState, fmaf(dec.y, h.y, add.y)));
    return h;
}

}  // namespace kda
