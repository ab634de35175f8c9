// kda_scan.h -- what the gated scan's kernels share: decays and input factors, the cut
// of the packed tokens into tiles, and the chain of states from tile to tile.
#pragma once

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

// A workgroup: waves with rows of a tile, one behind the other along the tokens, and
// one that holds none and finds the tiles and their states.  Waves with rows: 15 where a
// sequence's tiles are chained (7: 1 x 65,536 tokens x 4096 354 us instead of 337, 1 x 32,768
// x 512 69 instead of 45: longer tiles make shorter chains), 7 in one pass (15: 40 sequences
// of 0 to 90 tokens 26 us instead of 13.6), and 3 there where the sequences have no more
// tokens on average than they hold (7: 256 of 1 to 60 tokens x 4096 channels 73 us instead
// of 47).
constexpr int kWavesChained = 15, kWavesOnePass = 7, kWavesShort = 3;

// A wave goes over its rows twice.  Either it keeps two registers for every element from
// one pass to the other, or it forms the factors again from the rows as they were read:
// where they are cheap, so that 64 registers do and two workgroups of 16 waves fit a
// compute unit (16 ragged sequences x 4096, log-decays 343 us, kept 372; pre-activations
// with complement kept 337, formed again in 64 registers 977, most of it spills).  The
// gradients of fp32, half as many rows to a wave, fit either way (8192 x 4096 160, kept 171).
constexpr bool scan_cheap(int gate, int input) { return gate == KDA_GATE_LOG && input == KDA_INPUT_PLAIN; }
constexpr bool scan_again(size_t elem, bool backward, bool cheap) { return cheap || (backward && elem == 4); }
// Waves on a SIMD that the registers are cut for.
constexpr int scan_occupancy(size_t elem, bool backward, bool cheap) { return elem == 4 || cheap ? 8 : 4; }
// Tokens of a wave: about what the registers hold (32,768 x 4096 bf16, pre-activations with
// norm: 16 rows 227 us, 14 194; their gradients 10 rows 441, 8 345; gradients of log-decays
// with complement 8 rows 328, 12 312, of pre-activations alone 8 289, 10 277, 12 298; 8192 x
// 4096 fp32 with norm 8 rows 92.6, 6 88.9).  Not to the last register: bf16 log-decays with
// complement or norm take all 128 at 16 rows, and the forms of 7 and 3 waves keep 12 bytes a
// lane in scratch (14 rows would take 121 and none); of the fp32 gradients log-decays with norm
// at 7 and 3 waves and pre-activations alone at 15 keep 36.  Log-decays alone would hold more
// than 16: 20 rows, 60 registers, are the same for wide prompts (1 x 4096 x 8192 51.4 us
// either way, 16 ragged sequences x 4096 342 and 343) and better for long narrow ones (1 x
// 32,768 x 512 40.4 instead of 44.7); their gradients are the same with 8 or 10.  In one pass
// more rows leave waves without any (40 sequences of 40 tokens x 2048, gradients of log-decays
// with complement 8 rows 12.3, 12 14.4).
constexpr int scan_rows(size_t elem, bool backward, bool chained, int gate, int input) {
    const bool log = gate == KDA_GATE_LOG, plain = input == KDA_INPUT_PLAIN;
    if (backward) return elem == 4 ? 4 : chained && log != plain ? (log ? 12 : 10) : 8;
    return elem == 2 ? (!log && input == KDA_INPUT_NORM ? 14 : 16) : scan_cheap(gate, input) ? 8 : 6;
}
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
    int64_t T;
    uint32_t *ticket, *flags;
    uint64_t *words;
    int N, C, groups, num_slots, state_bf16, polls, tiles;
};

constexpr float kLog2e = 1.4426950408889634f;

// log2(1 + e), 0 <= e <= 1, to 2.1e-7 of itself as evaluated here in fp32: a polynomial times
// e (least maximal relative error, by reweighted least squares).  The logarithm of a rounded
// 1 + e would lose e's low bits.
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

// Of one gate value: a, c = 1 - a and the input factor b; l = log2 a for KDA_GATE_LOG.
template <int GATE, int INPUT> struct Factors {
    float a, c, b, l;
    bool clamped;
    __device__ __forceinline__ Factors() {}
    __device__ __forceinline__ explicit Factors(float z) {
        if (GATE == KDA_GATE_LOG) {
            clamped = z > 0.f;
            const float g = clamped ? 0.f : z;  // NaN stays
            l = g * kLog2e;
            a = exp2_fast(l);
            c = g > -0.125f ? near_zero(g) : 1.f - a;
        } else {
            clamped = false;
            const float e = exp2_fast(-fabsf(z) * kLog2e), r = __builtin_amdgcn_rcpf(1.f + e), er = e * r;
            // 1 / (1 + e^-z) and 1 / (1 + e^z), both to (6 + 1.3 |z|) 2^-24 of themselves: the argument
            // of the exponential is rounded, which costs more the farther out z lies
            a = z > 0.f ? r : er;
            c = z > 0.f ? er : r;
        }
        b = INPUT == KDA_INPUT_PLAIN ? 1.f : INPUT == KDA_INPUT_COMPLEMENT ? c : __builtin_amdgcn_sqrtf(c * (1.f + a));
    }
    __device__ __forceinline__ float input(float x) const { return INPUT == KDA_INPUT_PLAIN ? x : b * x; }
    // dx = b dh;  dgate = dh a' (before - x q) with a' = da/dgate and q = -db/da
    __device__ __forceinline__ void gradient(float dh, float before, float x, float &dx, float &dg) const {
        dx = INPUT == KDA_INPUT_PLAIN ? dh : b * dh;
        if (INPUT == KDA_INPUT_COMPLEMENT) before -= x;
        if (INPUT == KDA_INPUT_NORM) before -= b > 0.f ? x * (a * __builtin_amdgcn_rcpf(b)) : 0.f;
        dg = dh * (GATE == KDA_GATE_LOG ? a : a * c) * before;
        if (clamped) dg = 0.f;
    }
    // 1 - e^g near 0, to 9e-8 of itself as evaluated here (the last product's rounding alone is
    // 6e-8): the difference from a rounded exponential would lose its low bits
    static __device__ __forceinline__ float near_zero(float g) {
        float q = fmaf(g, 1.f / 720.f, 1.f / 120.f);
        q = fmaf(q, g, 1.f / 24.f);
        q = fmaf(q, g, 1.f / 6.f);
        q = fmaf(q, g, 0.5f);
        q = fmaf(q, g, 1.f);
        return -g * q;
    }
};

// The gate value whose step leaves the state alone (a = 1, 1 - a = 0).
template <int GATE> __device__ __forceinline__ float open_gate() { return GATE == KDA_GATE_LOG ? 0.f : __builtin_inff(); }

// The step of a run of tokens, grown at one end.  The running product weighs the inputs;
// what is handed on is its logarithm, which must not gather the rounding of every a = 1 -
// small: a sum of the log-decays, or for pre-activations the product's own complement
// 1 - prod a = sum c prod a, exact where it is small, and one logarithm of it at the end.
template <int GATE> struct Run {
    float prod = 1.f, add = 0.f, acc = 0.f;
    template <typename F> __device__ __forceinline__ void decay(const F &f) {
        acc = GATE == KDA_GATE_LOG ? acc + f.l : fmaf(f.c, prod, acc);
        prod *= f.a;
    }
    // a token before the run (the state passes it first)
    template <typename F> __device__ __forceinline__ void before(const F &f, float u) {
        add = fmaf(u, prod, add);
        decay(f);
    }
    // in the gradients' direction: a token after it, whose value passes its own decay too
    template <typename F> __device__ __forceinline__ void behind(const F &f, float d) {
        decay(f);
        add = fmaf(d, prod, add);
    }
    __device__ __forceinline__ float log2_decay() const {
        if (GATE == KDA_GATE_LOG) return acc;
        return prod > 0.5f ? -log2_1p(acc * __builtin_amdgcn_rcpf(prod)) : __builtin_amdgcn_logf(prod);
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

// A tile of a sequence: tokens index * TILE and on of its `len`, which begin at `start` of
// the call's; 128 channels.
struct alignas(16) Tile {
    int n, group, start, len, index, slot;  // n: sequence, -1: no tile
    int m;                                  // number of the tile in the call (chained)
    int count;                              // tiles of the sequence
};

// The sequences' bounds and slots, as one wave reads them: of up to 63 sequences from a
// register of each lane, filled once; of more from memory.
struct Sequences {
    const ScanParams &p;
    int lane, bound, slot;
    __device__ __forceinline__ Sequences(const ScanParams &p, int lane) : p(p), lane(lane) {
        bound = lane <= p.N ? cu(lane) : 0;
        slot = lane < p.N ? pool_slot(p.slots, p.num_slots, lane) : -1;
    }
    // kept inside the call's tokens whatever cu_seqlens holds
    __device__ __forceinline__ int cu(int n) const {
        return p.cu ? (int)min(max((int64_t)p.cu[n], (int64_t)0), p.T) : (int)(p.T / p.N * n);
    }
    __device__ __forceinline__ bool held() const { return p.N < 64; }
    template <int TILE> __device__ __forceinline__ void fill(int n, Tile &t) const {
        t.n = n;
        t.start = held() ? __builtin_amdgcn_readlane(bound, n) : cu(n);
        t.len = max((held() ? __builtin_amdgcn_readlane(bound, n + 1) : cu(n + 1)) - t.start, 0);
        t.count = (t.len + TILE - 1) / TILE;
        t.slot = held() ? __builtin_amdgcn_readlane(slot, n) : pool_slot(p.slots, p.num_slots, n);
    }
    // First tile number of sequence n.  Tiles T / TILE + N suffice: a sequence of L tokens
    // from s has (s + L) / TILE - s / TILE + 1 of them, at least ceil(L / TILE) and one.
    template <int TILE> static __device__ __forceinline__ int first_tile(int start, int n) { return start / TILE + n; }
    // The tile of number m (n: -1 where no tile has that number).
    template <int TILE> __device__ __forceinline__ void find(int m, Tile &t) const {
        int lo = 0, hi = p.N;  // the last sequence whose first tile is at or before m
        if (held()) {
            lo = max(__popcll(__ballot(lane < p.N && (lane == 0 || first_tile<TILE>(bound, lane) <= m))) - 1, 0);
        } else {
            while (hi - lo > 1) {
                const int step = (hi - lo + 63) / 64, at = lo + lane * step;
                const bool before = at < hi && (lane == 0 || first_tile<TILE>(cu(at), at) <= m);
                lo += (__popcll(__ballot(before)) - 1) * step;
                hi = min(lo + step, hi);
            }
        }
        lo = __builtin_amdgcn_readfirstlane(lo);
        fill<TILE>(lo, t);
        t.m = m;
        t.index = m - first_tile<TILE>(t.start, lo);
        if (t.index < 0 || t.index >= max(t.count, 1)) t.n = -1;
    }
};

// Takes a ticket (lane 0's result).  Tickets count (tile, channel group), a tile behind the
// one that its state comes from, so that whatever a workgroup waits for belongs to a
// smaller ticket, held by a workgroup that runs or has run.  The smallest unfinished
// ticket never waits, hence every wait ends, however few workgroups run at a time.
__device__ __forceinline__ uint32_t take_ticket(const ScanParams &p, int lane) {
    uint32_t ticket = 0;
    if (lane == 0) ticket = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return ticket;
}
// Its tile (n: -1 for a number that no tile has).
template <int TILE, bool BACKWARD>
__device__ __forceinline__ Tile ticket_tile(const ScanParams &p, const Sequences &seq, uint32_t taken) {
    Tile t = {};
    const uint32_t ticket = __builtin_amdgcn_readfirstlane(taken), k = ticket / (uint32_t)p.groups;
    t.group = ticket - k * p.groups;
    seq.find<TILE>(BACKWARD ? p.tiles - 1 - (int)k : (int)k, t);
    return t;
}

__device__ __forceinline__ Tile uniform(const Tile &t) {
    Tile u;
    u.n = __builtin_amdgcn_readfirstlane(t.n);
    u.group = __builtin_amdgcn_readfirstlane(t.group);
    u.start = __builtin_amdgcn_readfirstlane(t.start);
    u.len = __builtin_amdgcn_readfirstlane(t.len);
    u.index = __builtin_amdgcn_readfirstlane(t.index);
    u.slot = __builtin_amdgcn_readfirstlane(t.slot);
    u.m = __builtin_amdgcn_readfirstlane(t.m);
    u.count = __builtin_amdgcn_readfirstlane(t.count);
    return u;
}

// Two neighbouring elements as they were read.  (bf16: one register and no vector of two
// halves, which the compiler would take apart where control flow joins.)
template <typename T> struct Two;
template <> struct Two<__bf16> {
    typedef uint32_t bits;
    static __device__ __forceinline__ float get(bits x, int v) {
        return __builtin_bit_cast(float, v ? x & 0xffff0000u : x << 16);
    }
    static __device__ __forceinline__ bits both(float x) {
        const uint32_t b = __builtin_bit_cast(uint32_t, x) >> 16;  // (of values that bf16 holds)
        return b << 16 | b;
    }
    static __device__ __forceinline__ void hold(bits &x) { asm volatile("" : "+v"(x)); }
};
template <> struct Two<float> {
    struct bits { float x, y; };
    static __device__ __forceinline__ float get(bits x, int v) { return v ? x.y : x.x; }
    static __device__ __forceinline__ bits both(float x) { return bits{x, x}; }
    static __device__ __forceinline__ void hold(bits &x) { asm volatile("" : "+v"(x.x), "+v"(x.y)); }
};

// A wave's rows of one tensor as a bounded buffer: rows past the last one are read as it
// and written nowhere, whatever lies behind it.  (The hardware compares a lane's offset
// with the bytes left behind the row's, so a row's offset stays inside.)
template <typename T> struct RowBuffer {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    static constexpr uint32_t kNowhere = 0x7ffffff0u;  // past every buffer: 2^31 bytes at most
    __amdgpu_buffer_rsrc_t rsrc;
    int stride, last;
    __device__ __forceinline__ RowBuffer(const void *p, int64_t token, int64_t elems, int C, int rows)
        : stride((int)elems * (int)sizeof(T)), last(__builtin_amdgcn_readfirstlane(max(rows, 1) - 1)) {
        const uint64_t base = reinterpret_cast<uint64_t>(p) + token * elems * (int64_t)sizeof(T);
        const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)base), hi = __builtin_amdgcn_readfirstlane((uint32_t)(base >> 32));
        const int bytes = __builtin_amdgcn_readfirstlane(rows > 0 ? last * stride + C * (int)sizeof(T) : 0);
        rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>((uint64_t)hi << 32 | lo), 0, bytes, 0x00020000);
    }
    __device__ __forceinline__ typename Two<T>::bits load(uint32_t off, int row) const {
        const int at = __builtin_amdgcn_readfirstlane(min(max(row, 0), last) * stride);
        if constexpr (sizeof(T) == 2) return __builtin_amdgcn_raw_buffer_load_b32(rsrc, off, at, 0);
        else return __builtin_bit_cast(typename Two<T>::bits, __builtin_amdgcn_raw_buffer_load_b64(rsrc, off, at, 0));
    }
    __device__ __forceinline__ void store(uint32_t off, int row, float a, float b) const {
        const uint32_t o = row <= last ? off : kNowhere;
        const int at = __builtin_amdgcn_readfirstlane(min(row, last) * stride);
        typename Pair<T>::vec v;
        v.x = from_f32<T>(a);
        v.y = from_f32<T>(b);
        if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), rsrc, o, at, 0);
        else __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, v), rsrc, o, at, 0);
    }
};

// The state before a tile whose step is (dec, add), two channels a lane.  `h` is the state
// before the sequence where the chain begins with this tile (`done` = 0 tiles before it);
// the `done` tiles before it have the numbers m + way, m + 2 way, ..
//
// A tile first publishes its own step (P, H) and, once it knows the state before it, the
// state behind it.  Both are one 64-bit word for each channel, value and kind together,
// so relaxed atomics suffice and no cache is flushed: {P, H} with P >= 0 (a NaN has the
// usual bits), {kState, h}, or kEmpty from the clearing launch.  A flag for the tile says
// which to expect; neighbours' flags lie side by side, so that a waiting tile polls 256
// bytes for the 64 before it (the words of eight of them, 8 KB, took a third of the
// memory's time from those that work).  From the nearest tile that shows a state it goes
// forward with h -> P h + H, which is what those tiles compute themselves: the result does
// not depend on how far the others have come.
constexpr int kLook = 8;  // rows of words read at once
__device__ __forceinline__ uint64_t word(uint32_t kind, float v) {
    return (uint64_t)__builtin_bit_cast(uint32_t, v) << 32 | kind;
}
__device__ __forceinline__ float word_value(uint64_t w) { return __builtin_bit_cast(float, (uint32_t)(w >> 32)); }
__device__ __forceinline__ uint32_t decay_bits(float p) {
    return p == p ? __builtin_bit_cast(uint32_t, p) : 0x7fc00000u;
}
__device__ __forceinline__ void publish(uint64_t *at, uint64_t a, uint64_t b, uint32_t *flag, uint32_t kind, int lane) {
    __hip_atomic_store(at, a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(at + 1, b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (lane == 0) __hip_atomic_store(flag, kind, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ float2 chain_carry(const ScanParams &p, const Tile &t, int lane, int done, int way,
                                              float2 dec, float2 add, float2 h) {
    const int64_t row = (int64_t)p.groups * 128 * way;  // words from a tile's to those of the one before
    uint64_t *mine = p.words + ((int64_t)t.m * p.groups + t.group) * 128 + 2 * lane;
    uint32_t *flag = p.flags + (int64_t)t.group * p.tiles + t.m;
    const bool last = done == t.count - 1;
    if (done > 0) {
        if (!last) publish(mine, word(decay_bits(dec.x), add.x), word(decay_bits(dec.y), add.y), flag, 1, lane);
        for (int polls = 0;; ++polls) {
            uint32_t f = 0;
            if (lane < done) f = __hip_atomic_load(flag + way * (lane + 1), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const uint64_t states = __ballot(f == 2), steps = __ballot(f != 0);
            const int from = states ? __builtin_ctzll(states) : 64;
            bool good = from < 64 && (~steps & ((1ull << from) - 1)) == 0;
            float2 s = h;
            for (int k0 = from; k0 >= 0 && good; k0 -= kLook) {
                uint64_t wx[kLook], wy[kLook];
#pragma unroll
                for (int i = 0; i < kLook; ++i) {
                    const uint64_t *at = mine + row * (max(k0 - i, 0) + 1);
                    wx[i] = __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    wy[i] = __hip_atomic_load(at + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    if (k0 - i <= 0) break;
                }
#pragma unroll
                for (int i = 0; i < kLook; ++i) {
                    const uint32_t a = (uint32_t)wx[i], b = (uint32_t)wy[i];
                    // a flag may be seen before its words
                    if (!__all(k0 - i == from ? a == kState && b == kState : a != kEmpty && b != kEmpty)) good = false;
                    s.x = a == kState ? word_value(wx[i]) : fmaf(__builtin_bit_cast(float, a), s.x, word_value(wx[i]));
                    s.y = b == kState ? word_value(wy[i]) : fmaf(__builtin_bit_cast(float, b), s.y, word_value(wy[i]));
                    if (k0 - i <= 0) break;
                }
            }
            if (good) {
                h = s;
                break;
            }
            if (polls >= p.polls) {  // never reached by a correct chain; a wait that gives up says so
                h = make_float2(__builtin_nanf(""), __builtin_nanf(""));
                break;
            }
            __builtin_amdgcn_s_sleep(1);
        }
    }
    if (!last) publish(mine, word(kState, fmaf(dec.x, h.x, add.x)), word(kState, fmaf(dec.y, h.y, add.y)), flag, 2, lane);
    return h;
}

}  // namespace kda
