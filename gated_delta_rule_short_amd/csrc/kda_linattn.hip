// kda_linattn.hip -- chunked linear attention with one decay per head, bf16 tokens.
//
// With b_r the sum of a chunk's log-decays up to token r (64 tokens a chunk):
//     o_r = scale (e^{b_r} S^T q_r + sum_{s <= r} e^{b_r - b_s} (q_r . k_s) v_s)
//     S   <- e^{b_64} S + sum_s k_s (e^{b_64 - b_s} v_s)^T
// so a chunk is five small matrix products: K Q^T, S^T Q^T, V^T P^T (the outputs,
// transposed) and K^T V' (the state).
//
// A workgroup owns DVT columns of one (sequence, head) state and carries it over
// the chunks in registers.  A wave holds 16 columns of a 1/DKS part of the rows,
// laid out so that its accumulators, rounded to bf16, are the operand of S^T Q^T
// as they stand: the state never passes through LDS.  P = K Q^T is formed once
// and reaches the waves through LDS in operand order.  Four more waves serve the
// others: two stream q, k, v and g from memory into a ring of LDS stages (LDS DMA,
// NS - 1 chunks ahead; one wave alone would stall at 63 loads in flight and hold the
// others at their next barrier), two form P and turn the decays of the next chunk
// into the factors above.
//
// With few (sequence, head) pairs the sequences are cut into segments, and three
// launches spread them over the GPU: every segment's state from nothing (the same
// kernel without q, P and outputs), a scan of those states along each sequence, and
// the outputs with every segment starting from its scanned state.  The keys and
// values are read twice for it, first from the last chunk to the first: what the
// outputs begin with was read last and is still cached (1 x 65,536 tokens x 8 heads
// 202 -> 197 us, 1 x 4096 x 64 92.6 -> 92.2; and the state needs no decay on the way).
// Where sequences have few segments, the third launch joins them itself.
//
// Rounding: P and the state under q are rounded to bf16 once as operands (the
// outputs are bf16 themselves).  The decayed values of the state's own product
// are split into three bf16 parts, which hold an fp32 value exactly, because the
// state is returned in fp32 and one rounded part would leave it with 2^-9.  The
// decay sums run in 64 bits and are kept as two floats: b_r - b_s stays exact
// behind a token that clears the state (a large |g|).
//
// What bounds it: 16 sequences of 4096 tokens x 64 heads x 128 x 128 (4.3 GB) take 0.98
// to 1.27 ms, 3.4 to 4.4 TB/s against 5.2 of a large copy, at 1.2 to 1.6 GHz: the power
// that the state's products draw (0.91 ms at 2.3 GHz without them).  A lone sequence is
// bound by the chain of its chunks, 1.4 us each; cut into many segments, by the scan that
// joins them, whose steps of eight segments follow one another at 1.25 us (1 x 16,384
// tokens x 1 head: 256 segments, 53 us).
//
// A future token has a zero in P, but zero times a non-finite value is not
// zero: products never run over whole 16-token blocks of the future, and a NaN or
// infinity among a chunk's values is left out of them and added on its own to the
// rows that see it.  In the state's product an infinity must not meet a zero that the
// recurrence does not have: neither the parts of a value (split3) nor the weights of the
// rows past the sequence are zeros.  (Those parts cost the large calls up to 1 % and 40
// short sequences 0.6 of 13.3 us.)
#include <type_traits>

#include "kda_linattn.h"

namespace kda {

namespace {

constexpr int C = kFactorTokens;  // tokens per chunk

typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

// Piece c (16 bytes) of row r lies at piece c ^ swz(r) of its row of CPR pieces, with
// the bits of r permuted so that no two lanes served in one cycle meet in a bank:
// for q and k a 16-byte read of rows l % 16 at one piece (cycles take l % 16 of
// 0..3 and 12..15 with the next sixteen lanes' 4..11) and a transposed read of four
// rows by four pieces' halves, for v the transposed read of two whole pieces.
template <int CPR> __device__ __forceinline__ int swz(int r) {
    const int lo = CPR == 16 ? (r & 1) | (r >> 1 & 1) << 3 : r >> 1 & 1;
    return lo | (r >> 3 & 1) << 1 | (r >> 2 & 1) << 2;
}
template <int CPR> __device__ __forceinline__ int swz_v(int r) {
    return CPR == 16 ? (r & 7) << 1 | (r >> 3 & 1) : CPR == 8 ? (r & 6) | (r >> 3 & 1) : (r >> 2 & 1) << 1;
}

// Transposed read: lane l gets rows 4 (l / 16) + 0..3 of column l % 16, from four
// neighbouring elements at p in row 4 (l / 16) + l % 16 / 4 each.
__device__ __forceinline__ bf16x4 read_tr(const unsigned char *p) {
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)p));
}

// 16 bytes of each lane's address to 16 * lane behind dst (the same for every lane).
__device__ __forceinline__ void dma16(unsigned char *dst, const unsigned char *src) {
    __builtin_amdgcn_global_load_lds(src, (lds_void *)dst, 16, 0, 0);
}

// DMA of the chunk's first n rows of CPR pieces at `src` (rows `stride` bytes apart)
// into LDS; rows past them repeat the last one, which a weight of next to nothing or a row
// that is not stored makes harmless.
template <int CPR, bool V, int I0 = 0, int I1 = CPR>  // instructions I0 .. I1 - 1 of CPR
__device__ __forceinline__ void dma_rows(unsigned char *dst, const unsigned char *src, int64_t stride, int n,
                                         int lane) {
    constexpr int RPI = 64 / CPR;  // rows per instruction
    const int lr = lane / CPR, pc = lane % CPR;
    if (n == C) {
        const unsigned char *row = src + (I0 * RPI + lr) * stride;
#pragma unroll
        for (int i = I0; i < I1; ++i) {
            dma16(dst + i * 1024, row + (pc ^ (V ? swz_v<CPR>(i * RPI + lr) : swz<CPR>(i * RPI + lr))) * 16);
            row += RPI * stride;
        }
    } else {
#pragma unroll 1
        for (int i = I0; i < I1; ++i) {
            const int row = i * RPI + lr;
            dma16(dst + i * 1024, src + (int64_t)min(row, n - 1) * stride + (pc ^ (V ? swz_v<CPR>(row) : swz<CPR>(row))) * 16);
        }
    }
}

// LDS of a workgroup.  OUT false: the state alone, without q and P.
template <int DK, int DVT, int DKS, int NS, bool OUT> struct Lay {
    static constexpr int NCT = DVT / 16, NW = NCT * DKS;  // column tiles, compute waves
    static constexpr int STAGES = NS, UD = DK / 32 / DKS; // 32-row groups of the state per wave
    static constexpr bool Q = OUT;
    static constexpr int QB = C * DK * 2, VB = C * DVT * 2;
    static constexpr int K = OUT ? QB : 0, V = K + QB, STAGE = V + VB;  // q, k, v in a stage
    static constexpr int CPR = DK / 8, CPV = DVT / 8;     // 16-byte pieces of a row
    static constexpr int G = NS * STAGE, NG = NS < 2 ? 2 : NS;  // ring of raw decays
    static constexpr int P = G + NG * 256;                // P of two chunks, six operand pairs of 1 KiB each
    static constexpr int B = P + (OUT ? 2 * 6144 : 0);    // decay factors of three chunks
    static constexpr int X = B + 3 * 1040;                // partial outputs of two chunks when DKS > 1
    static constexpr int XB = OUT && DKS > 1 ? NCT * 4 * DKS * 1024 : 0;
    static constexpr int TOTAL = X + 2 * XB;
    static constexpr int SERVE = OUT ? 2 : 1;             // waves that form factors and P
    static constexpr int THREADS = (NW + SERVE + 2) * 64;
    static constexpr int DMAS = OUT ? CPR + CPV / 2 : (CPR + CPV) / 2;  // loads per chunk and streaming wave
    static_assert(UD >= 1 && TOTAL <= 160 * 1024, "LDS");
};

// A streaming wave's view of its sequence and head (strides in bytes, g's in
// elements): the first takes q, g and the upper half of v, the second k and the rest;
// without q they share k like v.
struct Stream {
    const unsigned char *x, *v;
    const float *g;
    int64_t xs, vs, gs;
    int len, nc;
};
// (One past the last chunk is fetched too, from tokens that are there, so that every
// chunk comes with the same number of loads.)  Without q the chunks come last to first
// and are whole ones.
template <typename L> __device__ __forceinline__ void fetch_g(const Stream &m, unsigned char *lds, int c, int lane) {
    if (c > m.nc) return;
    const int t = L::Q ? min(c * C + lane, m.len - 1) : max(m.nc - 1 - c, 0) * C + lane;
    __builtin_amdgcn_global_load_lds(m.g + (int64_t)t * m.gs, (lds_void *)(lds + L::G + (c % L::NG) * 256), 4, 0, 0);
}
template <typename L, int SW>
__device__ __forceinline__ void fetch(const Stream &m, unsigned char *lds, int c, int lane) {
    if (c >= m.nc) return;
    unsigned char *st = lds + (c % L::STAGES) * L::STAGE;
    const int n = L::Q ? min(m.len - c * C, C) : C;
    const int64_t t = (int64_t)(L::Q ? c : m.nc - 1 - c) * C;
    if constexpr (L::Q) dma_rows<L::CPR, false>(st + SW * L::K, m.x + t * m.xs, m.xs, n, lane);
    else dma_rows<L::CPR, false, SW * L::CPR / 2, (SW + 1) * L::CPR / 2>(st, m.x + t * m.xs, m.xs, n, lane);
    dma_rows<L::CPV, true, SW * L::CPV / 2, (SW + 1) * L::CPV / 2>(st + L::V, m.v + t * m.vs, m.vs, n, lane);
}
template <typename L, int SW>
__device__ __forceinline__ void stream(const Stream &m, unsigned char *lds, int lane) {
    constexpr int NS = L::STAGES, EACH = L::DMAS + (SW == 0);
    // issued in order g0, then (g of chunk c + 1, chunk c): when chunk c has
    // landed, so has the next chunk's g
    if (SW == 0) fetch_g<L>(m, lds, 0, lane);
    auto next = [&](int c) __attribute__((always_inline)) {
        if (SW == 0) fetch_g<L>(m, lds, c + 1, lane);
        fetch<L, SW>(m, lds, c, lane);
    };
    // chunk c has landed when only the chunks behind it are outstanding
    auto landed = [&](int c, auto behind) __attribute__((always_inline)) {
        constexpr int N = decltype(behind)::value * EACH;
        static_assert(N + EACH < 64, "loads in flight");
        if (c + decltype(behind)::value < m.nc) wait_vmcnt<N>();
        else wait_vmcnt<0>();
    };
    next(0);
    if (SW == 0) wait_vmcnt<EACH>();
    bar();  // g0 is there
    for (int c = 1; c < NS - 1; ++c) next(c);
    landed(0, std::integral_constant<int, (NS > 2 ? NS - 2 : 0)>{});
    bar();
    if (NS > 1) next(NS - 1);
    for (int c = 0; c < m.nc; ++c) {
        if constexpr (NS == 1) {
            bar();  // c: the slot is free
            if (c + 1 == m.nc) break;
            next(c + 1);
            landed(c + 1, std::integral_constant<int, 0>{});
            bar();
        } else {
            landed(c + 1, std::integral_constant<int, NS - 2>{});
            bar();  // c: the slot of chunk c is free, chunk c + 1 is there
            next(c + NS);
        }
    }
}

// v w, never -0.  (Not fused: a product that underflows would keep its sign.)
__device__ __forceinline__ float weighted(float v, float w) {
#pragma clang fp contract(off)
    const float x = v * w;
    return x + 0.f;
}
// x = a + b + c exactly, each the upper half of its word a bf16 (8 bits of x's 24).  a and
// b are cut from the value one step nearer to zero, so that no part of a number is zero and
// none has another sign: an infinite key times the parts, and a key times the parts of an
// infinity (twice the largest finite value, and itself), sum to what x itself gives and
// not to NaN.  x must not be -0; y is exact and never is.
__device__ __forceinline__ void split3(float x, uint32_t &a, uint32_t &b, uint32_t &c) {
    a = __builtin_elementwise_sub_sat(__builtin_bit_cast(uint32_t, x), 1u);
    const float y = x - __builtin_bit_cast(float, a & 0xffff0000u);
    b = __builtin_elementwise_sub_sat(__builtin_bit_cast(uint32_t, y), 1u);
    c = __builtin_bit_cast(uint32_t, y - __builtin_bit_cast(float, b & 0xffff0000u));
}
__device__ __forceinline__ bf16x8 upper_halves(const uint32_t *x) {
    typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x07060302u);
    return __builtin_bit_cast(bf16x8, r);
}

// Whether any of four tokens' values is not finite.
__device__ __forceinline__ bool has_non_finite(const bf16x4 (&v)[4]) {
    typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
    typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
    u16x2 most = {0, 0};  // of the moduli, two at a time
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, __builtin_bit_cast(u32x2, v[t])[i] & 0x7fff7fffu));
    return max(most.x, most.y) >= 0x7f80;
}

// Five of the ten 16 x 16 blocks of P at or below the diagonal: row blocks 0..2 against
// key blocks 0 and 1, or (2, 2) and the last row block.  Lane: token 16 rt + l % 16,
// keys 16 st + 4 (l / 16) + 0..3, the operand order of V^T P^T.
template <int DK, int HALF>
__device__ __forceinline__ void scores(const unsigned char *lq, const unsigned char *lk, const Factors *f,
                                       unsigned char *pl, int lane) {
    constexpr int RT[2][5] = {{0, 1, 1, 2, 2}, {2, 3, 3, 3, 3}}, ST[2][5] = {{0, 0, 1, 0, 1}, {2, 0, 1, 2, 3}};
    const int r16 = lane & 15, g4 = lane >> 4, frow = swz<DK / 8>(r16);
    f32x4 d[5];
#pragma unroll
    for (int b = 0; b < 5; ++b) d[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < DK / 32; ++u) {
        const int off = r16 * (DK * 2) + ((4 * u + g4) ^ frow) * 16;
        bf16x8 q[4], k[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (HALF ? t >= 2 : t < 3) q[t] = *reinterpret_cast<const bf16x8 *>(lq + 16 * t * (DK * 2) + off);
            if (HALF || t < 2) k[t] = *reinterpret_cast<const bf16x8 *>(lk + 16 * t * (DK * 2) + off);
        }
#pragma unroll
        for (int b = 0; b < 5; ++b) d[b] = mma_k32(k[ST[HALF][b]], q[RT[HALF][b]], d[b]);
    }
#pragma unroll
    for (int b = 0; b < 5; ++b) {
        const int rt = RT[HALF][b], st = ST[HALF][b], s = 16 * st + 4 * g4;
        const float rh = f->bh[16 * rt + r16], rl = f->bl[16 * rt + r16];
        const f32x4 sh = *reinterpret_cast<const f32x4 *>(f->bh + s), sl = *reinterpret_cast<const f32x4 *>(f->bl + s);
        f32x4 x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = d[b][i] * exp2_fast((rh - sh[i]) + (rl - sl[i]));
            if (rt == st) x[i] = r16 >= 4 * g4 + i ? x[i] : 0.f;
        }
        const int pair = (rt < 2 ? rt : 2 * rt - 2) + (st >> 1);
        *reinterpret_cast<bf16x4 *>(pl + pair * 1024 + lane * 16 + (st & 1) * 8) = pack4(x);
    }
}

// The finite values of x, or (BAD) the others; zeros in the place of the rest.
template <bool BAD> __device__ __forceinline__ bf16x4 part_of(bf16x4 x) {
    const i16x4 b = __builtin_bit_cast(i16x4, x);
    i16x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = ((b[i] & 0x7f80) == 0x7f80) == BAD ? b[i] : (short)0;
    return __builtin_bit_cast(bf16x4, r);
}

// What the chunk's non-finite values add to V^T P^T of row block rt: earlier blocks
// whole, the diagonal block token by token, to the rows that see it.
__device__ __forceinline__ f32x4 add_bad(f32x4 acc, const bf16x4 *vt, const unsigned char *pl, int rt, int lane) {
    const int r16 = lane & 15, g4 = lane >> 4;
    const bf16x4 z = {};
    for (int st = 0; st <= rt; ++st) {
        const bf16x4 pp = *reinterpret_cast<const bf16x4 *>(pl + (st >> 1) * 1024 + lane * 16 + (st & 1) * 8);
        bf16x4 vv = vt[0];
        vv = part_of<true>(st == 1 ? vt[1] : st == 2 ? vt[2] : st == 3 ? vt[3] : vv);
        if (st < rt) {
            acc = acc + mma_k16w(vv, pp, f32x4{0.f, 0.f, 0.f, 0.f});
            continue;
        }
        for (int s = 0; s < 16; ++s) {
            bf16x4 one = z;
#pragma unroll
            for (int i = 0; i < 4; ++i) one[i] = (g4 == s >> 2 && i == (s & 3)) ? vv[i] : one[i];
            const f32x4 d = mma_k16w(one, pp, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] += r16 >= s ? d[i] : 0.f;
        }
    }
    return acc;
}

template <int DK, int DVT, int DKS, int NS, bool OUT>
__global__ void __launch_bounds__((Lay<DK, DVT, DKS, NS, OUT>::THREADS), (NS == 1 ? 4 : 1)) chunk_kernel(ChunkParams p) {
    typedef Lay<DK, DVT, DKS, NS, OUT> L;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[L::TOTAL];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Work wk;
    if (!locate(p, wk, lane)) return;
    if (!OUT && wk.j + 1 >= wk.nseg) return;  // nothing starts from the last segment
    const int slot = pool_slot(p.slots, p.num_slots, wk.n);
    if (slot < 0) return;
    const int nc = (wk.len + C - 1) / C;

    // Barriers: one when g of chunk 0 has landed, one when chunk 0 has and its factors
    // are formed, then one at the end of every interval c, in which chunk c is worked on
    // (and with one stage another when chunk c + 1 has landed in it).
    if (wave >= L::NW && nc == 0) return;
    if (wave >= L::NW + L::SERVE) {  // the streaming waves: they read no LDS
        const int hk = wk.h / p.rep, sw = wave - L::NW - L::SERVE;
        const bool keys = sw || !OUT;
        Stream m;
        m.xs = (keys ? p.ks : p.qs) * 2; m.vs = p.vs * 2; m.gs = p.gs;
        m.x = static_cast<const unsigned char *>(keys ? p.k : p.q) + wk.t0 * m.xs + (int64_t)hk * DK * 2;
        m.v = static_cast<const unsigned char *>(p.v) + wk.t0 * m.vs + ((int64_t)wk.h * p.dv + wk.tile * DVT) * 2;
        m.g = p.g + wk.t0 * p.gs + wk.h;
        m.len = wk.len; m.nc = nc;
        if (sw == 0) stream<L, 0>(m, lds, lane);
        else stream<L, 1>(m, lds, lane);
        return;
    }
    Factors *fac = reinterpret_cast<Factors *>(lds + L::B);
    if (wave >= L::NW) {  // the score waves; the first also forms the factors of chunk c + 1
        double after = 0.0;  // the decays of the chunks behind (already worked on without q)
        auto form = [&](int c) __attribute__((always_inline)) {
            if (c >= nc) return;
            const float x = reinterpret_cast<const float *>(lds + L::G + (c % L::NG) * 256)[lane];
            const double e = chunk_factors(x, fac + c % 3, OUT ? min(wk.len - c * C, C) : C, lane, after);
            if (!OUT) after += e;
        };
        bar();
        if (wave == L::NW) form(0);
        bar();
        for (int c = 0; c < nc; ++c) {
            const unsigned char *lq = lds + (c % NS) * L::STAGE;
            unsigned char *pl = lds + L::P + (c & 1) * 6144;
            if (wave == L::NW) {
                if constexpr (OUT) scores<DK, 0>(lq, lq + L::K, fac + c % 3, pl, lane);
                form(c + 1);
            } else if constexpr (OUT) {
                scores<DK, 1>(lq, lq + L::K, fac + c % 3, pl, lane);
            }
            bar();
            if (NS == 1 && c + 1 < nc) bar();
        }
        return;
    }

    const int r16 = lane & 15, g4 = lane >> 4;
    const int ct = wave % L::NCT, hh = wave / L::NCT;
    const int col = wk.tile * DVT + 16 * ct;
    // Without q, S begins at zero and the start is added behind the last chunk.
    // S[u][e][i]: row 32 (hh UD + u) + 8 g4 + 4 (e ^ g4 % 2) + i, column col + r16 (the
    // exchanged halves keep the transposed reads of k off each other's banks)
    f32x4 S[L::UD][2];
    const size_t sbase = ((size_t)slot * p.H + wk.h) * DK * p.dv + (size_t)(32 * hh * L::UD + 8 * g4) * p.dv + col + r16;
    // a segment's starting state: the user's for a sequence in one piece; else the
    // first segment keeps a copy for the outputs, which may replace the user's
    const size_t wbase = ((size_t)wk.s * p.H + wk.h) * DK * p.dv + ((size_t)wk.tile * L::NW + wave) * L::UD * 512 + lane * 4;
    const size_t wnext = (size_t)p.H * DK * p.dv;
    if (OUT && wk.nseg > 1) {
        // (without a scan, the segments before this one are joined here)
        const int first = p.joined || wk.j < 2 ? 0 : wk.j - 1;  // segments back to where the sum begins
#pragma unroll
        for (int u = 0; u < L::UD; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                S[u][e] = *reinterpret_cast<const f32x4 *>(p.ws + wbase - first * wnext + (2 * u + e) * 256);
#pragma unroll 2
        for (int b = first - 1; b >= 0; --b) {
            const float d = p.wdec[(size_t)(wk.s - b - 1) * p.H + wk.h];
#pragma unroll
            for (int u = 0; u < L::UD; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    S[u][e] = S[u][e] * d + *reinterpret_cast<const f32x4 *>(p.ws + wbase - b * wnext + (2 * u + e) * 256);
        }
    } else {
        auto read = [&](auto *x) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < L::UD; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        S[u][e][i] = to_f32(x[sbase + (size_t)(32 * u + 4 * (e ^ (g4 & 1)) + i) * p.dv]);
        };
        if (!p.s_in || wk.j > 0) {
#pragma unroll
            for (int u = 0; u < L::UD; ++u) S[u][0] = S[u][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        } else if (p.state_bf16) {
            read(static_cast<const __bf16 *>(p.s_in));
        } else {
            read(static_cast<const float *>(p.s_in));
        }
        if (!OUT && wk.j == 0) {
#pragma unroll
            for (int u = 0; u < L::UD; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) *reinterpret_cast<f32x4 *>(p.ws + wbase + (2 * u + e) * 256) = S[u][e];
        }
    }

    __bf16 *o = static_cast<__bf16 *>(p.o) + ((size_t)wk.t0 * p.H + wk.h) * p.dv + col + 4 * g4;
    const size_t orow = (size_t)p.H * p.dv;
    const int frow = swz<L::CPR>(r16), trow = 4 * g4 + (r16 >> 2), ftr = swz<L::CPR>(trow);
    const int voff = trow * (DVT * 2) + ((2 * ct + (r16 >> 1 & 1)) ^ swz_v<L::CPV>(trow)) * 16 + (r16 & 1) * 8;

    bf16x4 vt[4];     // the chunk's values: column r16, tokens 16 t + 4 g4 + i
    f32x4 acc[4];     // S^T q of row block t, decayed (DKS 1)
    bool odd = false; // a value is not finite

    // Interval c: everything of chunk c that needs no other wave.
    auto own_part = [&](int c) __attribute__((always_inline)) {
        const unsigned char *lq = lds + (c % NS) * L::STAGE, *lk = lq + L::K, *lv = lq + L::V;
        const Factors *f = fac + c % 3;
#pragma unroll
        for (int t = 0; t < 4; ++t) vt[t] = read_tr(lv + 16 * t * (DVT * 2) + voff);
        if constexpr (OUT) {
        // S^T q over this wave's rows, four row blocks side by side
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < L::UD; ++u) {
            const bf16x4 s0 = pack4(S[u][0]), s1 = pack4(S[u][1]);
            const bf16x8 sb = (g4 & 1) ? join8(s1, s0) : join8(s0, s1);
            const unsigned char *qr = lq + r16 * (DK * 2) + ((4 * (hh * L::UD + u) + g4) ^ frow) * 16;
#pragma unroll
            for (int t = 0; t < 4; ++t)
                acc[t] = mma_k32(sb, *reinterpret_cast<const bf16x8 *>(qr + 16 * t * (DK * 2)), acc[t]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t] = acc[t] * f->eb[16 * t + r16];
        if constexpr (DKS > 1) {
            f32x4 *xs = reinterpret_cast<f32x4 *>(lds + L::X + (c & 1) * L::XB) + (size_t)ct * 4 * DKS * 64;
#pragma unroll
            for (int t = 0; t < 4; ++t) xs[(t * DKS + hh) * 64 + lane] = acc[t];
        }
        odd = __any(has_non_finite(vt));
        }
        // the state over the chunk: K^T V' with V' in three exact parts
        if constexpr (OUT) {
            const float tot = f->total;
#pragma unroll
            for (int u = 0; u < L::UD; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) S[u][e] = S[u][e] * tot;
        }
#pragma unroll
        for (int kp = 0; kp < 2; ++kp) {
            bf16x8 v3[3];
            {
                uint32_t x[8], y[8], z[8];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const f32x4 w = *reinterpret_cast<const f32x4 *>(f->w + 32 * kp + 16 * t + 4 * g4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) split3(weighted((float)vt[2 * kp + t][i], w[i]), x[4 * t + i], y[4 * t + i], z[4 * t + i]);
                }
                v3[0] = upper_halves(x);
                v3[1] = upper_halves(y);
                v3[2] = upper_halves(z);
            }
#pragma unroll
            for (int u0 = 0; u0 < L::UD; u0 += 2) {
                constexpr int W = L::UD < 2 ? 1 : 2;
                bf16x8 kt[W][2];
#pragma unroll
                for (int u = 0; u < W; ++u)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const unsigned char *kr = lk + (32 * kp + trow) * (DK * 2) +
                                                  ((4 * (hh * L::UD + u0 + u) + (r16 & 3)) ^ ftr) * 16 + 8 * (e ^ (r16 & 1));
                        kt[u][e] = join8(read_tr(kr), read_tr(kr + 16 * DK * 2));
                    }
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int u = 0; u < W; ++u)
#pragma unroll
                        for (int e = 0; e < 2; ++e) S[u0 + u][e] = mma_k32(kt[u][e], v3[i], S[u0 + u][e]);
            }
        }
    };
    // Behind barrier c: P's part of a row block, and its store (only the last chunk can
    // end early).
    auto finish = [&](int c, int rt, f32x4 d, auto guarded, auto last) __attribute__((always_inline)) {
        const unsigned char *pr = lds + L::P + (c & 1) * 6144 + (rt < 2 ? rt : 2 * rt - 2) * 1024;
        constexpr bool G = decltype(guarded)::value;  // values that are not finite come apart
        bf16x4 vv[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) vv[t] = G ? part_of<false>(vt[t]) : vt[t];
        // a half pair past the diagonal drops out on both sides
        const bf16x4 z = {};
        const bf16x8 p0 = *reinterpret_cast<const bf16x8 *>(pr + lane * 16);
        const bf16x4 a0 = {p0[0], p0[1], p0[2], p0[3]}, a1 = {p0[4], p0[5], p0[6], p0[7]};
        d = mma_k32(join8(vv[0], rt >= 1 ? vv[1] : z), join8(a0, rt >= 1 ? a1 : z), d);
        if (rt >= 2) {
            const bf16x8 p1 = *reinterpret_cast<const bf16x8 *>(pr + 1024 + lane * 16);
            const bf16x4 b0 = {p1[0], p1[1], p1[2], p1[3]}, b1 = {p1[4], p1[5], p1[6], p1[7]};
            d = mma_k32(join8(vv[2], rt >= 3 ? vv[3] : z), join8(b0, rt >= 3 ? b1 : z), d);
        }
        if (G) d = add_bad(d, vt, pr, rt, lane);
        const int t = c * C + 16 * rt + r16;
        if (!decltype(last)::value || t < wk.len)
            *reinterpret_cast<bf16x4 *>(o + (size_t)t * orow) = pack4(d * p.scale);
    };
    auto outputs = [&](int c, auto guarded, auto last) __attribute__((always_inline)) {
        if constexpr (DKS == 1) {
            if constexpr (decltype(guarded)::value) {
#pragma unroll 1
                for (int rt = 0; rt < 4; ++rt)
                    finish(c, rt, rt == 0 ? acc[0] : rt == 1 ? acc[1] : rt == 2 ? acc[2] : acc[3], guarded, last);
            } else {
#pragma unroll
                for (int rt = 0; rt < 4; ++rt) finish(c, rt, acc[rt], guarded, last);
            }
        } else {
            // row block rt of column tile ct is finished by one of its DKS waves, from
            // the partial sums of all of them in order
            const f32x4 *xs = reinterpret_cast<const f32x4 *>(lds + L::X + (c & 1) * L::XB) + (size_t)ct * 4 * DKS * 64;
#pragma unroll
            for (int j = 0; j < 4 / DKS; ++j) {
                const int rt = DKS == 4 ? hh : (j == 0 ? hh : 3 - hh);
                f32x4 d = xs[rt * DKS * 64 + lane];
#pragma unroll
                for (int i = 1; i < DKS; ++i) d = d + xs[(rt * DKS + i) * 64 + lane];
                finish(c, rt, d, guarded, last);
            }
        }
    };
    f32x4 start[L::UD][2];
    if constexpr (!OUT) {
#pragma unroll
        for (int u = 0; u < L::UD; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                start[u][e] = S[u][e];
                S[u][e] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
    }
    if (nc > 0) {
        bar();
        bar();
        // the first chunk apart where sequences are short (40 of them 14.4 -> 13.9 us); in the
        // loop else (16 ragged sequences 1515 -> 1472 us)
        if constexpr (NS == 1) {
            own_part(0);
            bar();
        }
#pragma unroll 1
        for (int c = NS == 1; c < nc; ++c) {
            if (c > 0) {
                if constexpr (OUT) {
                    if (odd) outputs(c - 1, std::true_type{}, std::false_type{});
                    else outputs(c - 1, std::false_type{}, std::false_type{});
                }
                if (NS == 1) bar();
            }
            own_part(c);
            bar();
        }
        if constexpr (OUT) {
            if (odd) outputs(nc - 1, std::true_type{}, std::true_type{});
            else outputs(nc - 1, std::false_type{}, std::true_type{});
        }
    }
    if constexpr (!OUT) {
        const float kept = fac[(nc - 1) % 3].total;  // the decays of all chunks
#pragma unroll
        for (int u = 0; u < L::UD; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<f32x4 *>(p.ws + wnext + wbase + (2 * u + e) * 256) = S[u][e] + start[u][e] * kept;
        if (threadIdx.x == 0 && wk.tile == 0) p.wdec[(size_t)wk.s * p.H + wk.h] = kept;
        return;
    }
    if (wk.j + 1 < wk.nseg) return;
    if (!p.s_out) return;
    auto write = [&](auto *x) __attribute__((always_inline)) {
        typedef typename std::remove_pointer<decltype(x)>::type E;
#pragma unroll
        for (int u = 0; u < L::UD; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[sbase + (size_t)(32 * u + 4 * (e ^ (g4 & 1)) + i) * p.dv] = from_f32<E>(S[u][e][i]);
    };
    if (p.state_bf16) write(static_cast<__bf16 *>(p.s_out));
    else write(static_cast<float *>(p.s_out));
}

template <int DK, int DVT, int DKS, int NS, bool OUT> hipError_t launch(ChunkParams p, hipStream_t s) {
    typedef Lay<DK, DVT, DKS, NS, OUT> L;
    p.tiles = p.dv / DVT;
    p.units = (p.seg ? p.segs : p.N) * (p.H / p.rep);
    const unsigned blocks = (unsigned)((p.units + 7) / 8) * 8 * p.rep * p.tiles;
    hipLaunchKernelGGL((chunk_kernel<DK, DVT, DKS, NS, OUT>), dim3(blocks), dim3(L::THREADS), 0, s, p);
    trace("chunk_kernel<%d, %d, %d, %d, %d> grid=(%u) block=%d lds=%d", DK, DVT, DKS, NS, (int)OUT, blocks, L::THREADS,
          L::TOTAL);
    return hipGetLastError();
}

// Whole states per workgroup.  (A 128 x 64 tile is split over twice the waves.)
hipError_t launch_wide(const ChunkParams &p, int dk, hipStream_t s) {
    if (dk == 64) return p.dv == 128 ? launch<64, 128, 1, 3, true>(p, s) : launch<64, 64, 1, 3, true>(p, s);
    return p.dv == 128 ? launch<128, 128, 1, 3, true>(p, s) : launch<128, 64, 2, 2, true>(p, s);
}

// Whole states over segments; of 64 columns two workgroups to a compute unit, with fewer
// stages of loads in each (8 sequences of 36,559 tokens in all, 5 heads, dk 128 79 -> 73 us).
template <bool OUT> hipError_t launch_segments(const ChunkParams &p, int dk, hipStream_t s) {
    constexpr int NS = OUT ? 3 : 4, NS64 = OUT ? 1 : 2;
    if (dk == 64) return p.dv == 128 ? launch<64, 128, 1, NS, OUT>(p, s) : launch<64, 64, 1, NS64, OUT>(p, s);
    return p.dv == 128 ? launch<128, 128, 1, NS, OUT>(p, s) : launch<128, 64, 1, NS64, OUT>(p, s);
}

}  // namespace

namespace {

// Along each sequence: the state that segment j + 1 starts from is its own from
// nothing (there already) plus segment j's start decayed over segment j, j >= 1.  One
// element a thread, eight segments in flight: 32 segments x 8 heads (17 MB read and
// written): 10 us.
__global__ void __launch_bounds__(256) segment_scan_kernel(ChunkParams p, int elems) {
    const int per = elems / 256, part = blockIdx.x % per, pair = blockIdx.x / per;
    const int n = pair / p.H, h = pair - n * p.H;
    const int64_t len = seq_start(p, n + 1) - seq_start(p, n);
    const int s0 = seg_base(p, n);
    const int nseg = (int)min((len + p.seg - 1) / p.seg, (int64_t)(p.segs - s0));
    if (nseg < 3 || pool_slot(p.slots, p.num_slots, n) < 0) return;
    const size_t step = (size_t)p.H * elems;
    float *w = p.ws + ((size_t)s0 * p.H + h) * elems + part * 256 + threadIdx.x;
    const float *dec = p.wdec + (size_t)s0 * p.H + h;
    float run = w[step];
    for (int j = 2; j < nseg; j += 8) {
        float x[8], d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // clamped, so that no branch stands between the loads
            const int at = min(j + i, nseg - 1);
            x[i] = w[(size_t)at * step];
            d[i] = dec[(size_t)(at - 1) * p.H];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            run = fmaf(run, d[i], x[i]);
            if (j + i < nseg) w[(size_t)(j + i) * step] = run;
        }
    }
}

}  // namespace

hipError_t launch_segment_scan(const ChunkParams &p, int elems, hipStream_t s) {
    const unsigned blocks = (unsigned)(p.N * p.H * (elems / 256));
    hipLaunchKernelGGL(segment_scan_kernel, dim3(blocks), dim3(256), 0, s, p, elems);
    trace("segment_scan_kernel grid=(%u) block=256", blocks);
    return hipGetLastError();
}

hipError_t launch_linattn_chunks(const kda_linattn_prefill_args *a, const LinattnPlan &plan, hipStream_t s) {
    ChunkParams p = chunk_params(a);
    if (plan.tokens) {
        use_segments(p, a, plan);
        hipError_t e = launch_segments<false>(p, a->head_dim_k, s);
        if (e != hipSuccess) return e;
        e = p.joined ? launch_segment_scan(p, a->head_dim_k * p.dv, s) : hipSuccess;
        if (e != hipSuccess) return e;
        return launch_segments<true>(p, a->head_dim_k, s);
    }
    const int64_t pairs = (int64_t)a->num_seqs * a->num_heads;
    // Many short sequences: one stage and 64 columns, so that a compute unit holds two
    // workgroups and one's loads run under the other's work.  640 workgroups (40
    // sequences x 16 heads, dv 64, with states) of 64 and 128 tokens each, nothing cached: dk
    // 128 26.7 -> 23.8 and 32.9 -> 33.7 us, dk 64 20.5 -> 15.3 and 25.6 -> 24.9; no gain with
    // 128 columns.
    if (pairs >= 256 && p.dv == 64 && p.total <= 128 * (int64_t)p.N)
        return a->head_dim_k == 64 ? launch<64, 64, 1, 1, true>(p, s) : launch<128, 64, 1, 1, true>(p, s);
    if (pairs * (p.dv / 64) >= 256) return launch_wide(p, a->head_dim_k, s);
    return a->head_dim_k == 64 ? launch<64, 32, 2, 3, true>(p, s) : launch<128, 32, 2, 3, true>(p, s);
}

}  // namespace kda
