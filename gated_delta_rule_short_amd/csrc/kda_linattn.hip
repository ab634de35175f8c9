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
// as they stand: the state never passes through LDS.  P = K Q^T is formed once,
// its 16 x 16 blocks shared out over the waves, and reaches them through LDS in
// operand order.  Two more waves serve the others: one streams q, k, v and g from
// memory into a ring of LDS stages (LDS DMA, NS - 1 chunks ahead), one turns the
// decays of the next chunk into the factors above.
//
// Rounding: P and the state under q are rounded to bf16 once as operands (the
// outputs are bf16 themselves).  The decayed values of the state's own product
// are split into three bf16 parts, which hold an fp32 value exactly, because the
// state is returned in fp32 and one rounded part would leave it with 2^-9.  The
// decay sums run in 64 bits and are kept as two floats: b_r - b_s stays exact
// behind a token that clears the state (a large |g|).
//
// A future token has a zero in P, but zero times a non-finite value is not
// zero: products never run over whole 16-token blocks of the future, and a chunk
// whose values hold a NaN or infinity takes its diagonal blocks token by token.
#include <type_traits>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int C = 64;  // tokens per chunk

typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
typedef __attribute__((ext_vector_type(8))) unsigned short u16x8;

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
};

// Workgroup barrier behind this wave's own LDS accesses.  (A fence would also
// wait for stores and LDS DMA.)
__device__ __forceinline__ void bar() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Position of 16-byte piece c of row r in a row of CPR pieces: the sixteen rows a
// wave reads at one piece, and the four rows by four pieces of a transposed read,
// fall on different banks.
template <int CPR> __device__ __forceinline__ int swz(int r) {
    return CPR == 16 ? ((r & 3) << 2 | (r >> 2 & 3)) : CPR == 8 ? ((r >> 1 & 1) << 2 | (r >> 2 & 3)) : 0;
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
// into LDS; rows past them repeat the last one, which a zero weight or a row that
// is not stored makes harmless.
template <int CPR>
__device__ __forceinline__ void dma_rows(unsigned char *dst, const unsigned char *src, int64_t stride, int n,
                                         int lane) {
    constexpr int RPI = 64 / CPR;  // rows per instruction
    const int lr = lane / CPR, pc = lane % CPR;
    if (n == C) {
        const unsigned char *row = src + lr * stride;
#pragma unroll
        for (int i = 0; i < CPR; ++i) {
            dma16(dst + i * 1024, row + (pc ^ swz<CPR>(i * RPI + lr)) * 16);
            row += RPI * stride;
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < CPR; ++i) {
            const int row = i * RPI + lr;
            dma16(dst + i * 1024, src + (int64_t)min(row, n - 1) * stride + (pc ^ swz<CPR>(row)) * 16);
        }
    }
}

// What a workgroup works on, from its block index.  The rep * tiles workgroups
// that read the same keys are `units` neighbours on one XCD (blocks go round the
// eight XCDs), where they share its L2.
struct Work {
    int n, h, tile;
    int64_t t0;
    int len;
};
__device__ __forceinline__ bool locate(const ChunkParams &p, Work &w) {
    const int U = p.rep * p.tiles, xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
    const int unit = (idx / U) * 8 + xcd, member = idx % U;
    if (unit >= p.units) return false;
    const int Hk = p.H / p.rep;
    w.n = unit / Hk;
    w.h = (unit - w.n * Hk) * p.rep + member / p.tiles;
    w.tile = member % p.tiles;
    if (p.cu) {
        w.t0 = min((int64_t)max(p.cu[w.n], 0), p.total);
        w.len = (int)max(min((int64_t)max(p.cu[w.n + 1], 0), p.total) - w.t0, (int64_t)0);
    } else {
        w.len = (int)(p.total / p.N);
        w.t0 = (int64_t)w.len * w.n;
    }
    return true;
}

template <int DK, int DVT, int DKS, int NS> struct Lay {
    static constexpr int NCT = DVT / 16, NW = NCT * DKS;  // column tiles, compute waves
    static constexpr int STAGES = NS;
    static constexpr int UD = DK / 32 / DKS;              // 32-row groups of the state per wave
    static constexpr int QB = C * DK * 2, VB = C * DVT * 2, STAGE = 2 * QB + VB;
    static constexpr int CPR = DK / 8, CPV = DVT / 8;     // 16-byte pieces of a row
    static constexpr int G = NS * STAGE;                  // ring of raw decays
    static constexpr int P = G + NS * 256;                // P, six operand pairs of 1 KiB
    static constexpr int B = P + 6144;                    // decay factors, two chunks
    static constexpr int X = B + 2 * 1040;                // partial outputs when DKS > 1
    static constexpr int TOTAL = X + (DKS > 1 ? NCT * 4 * DKS * 1024 : 0);
    static constexpr int THREADS = (NW + 2) * 64;
    static constexpr int DMAS = STAGE / 1024 + 1;         // DMA instructions per chunk
    static_assert(UD >= 1 && TOTAL <= 160 * 1024, "LDS");
};

// The streaming wave's view of its sequence and head (strides in bytes, g's in
// elements).
struct Stream {
    const unsigned char *q, *k, *v;
    const float *g;
    int64_t qs, ks, vs, gs;
    int len, nc;
};
template <typename L> __device__ __forceinline__ void fetch_g(const Stream &m, unsigned char *lds, int c, int lane) {
    if (c < m.nc)
        __builtin_amdgcn_global_load_lds(m.g + (int64_t)min(c * C + lane, m.len - 1) * m.gs,
                                         (lds_void *)(lds + L::G + (c % L::STAGES) * 256), 4, 0, 0);
}
template <typename L> __device__ __forceinline__ void fetch(const Stream &m, unsigned char *lds, int c, int lane) {
    if (c >= m.nc) return;
    unsigned char *st = lds + (c % L::STAGES) * L::STAGE;
    const int n = min(m.len - c * C, C);
    const int64_t t = (int64_t)c * C;
    dma_rows<L::CPR>(st, m.q + t * m.qs, m.qs, n, lane);
    dma_rows<L::CPR>(st + L::QB, m.k + t * m.ks, m.ks, n, lane);
    dma_rows<L::CPV>(st + 2 * L::QB, m.v + t * m.vs, m.vs, n, lane);
}

// Factors of one chunk: bh + bl (the decay sums, base 2), eb = 2^b, w = 2^(b_n - b)
// (0 past the sequence), 2^(b_n) last.
struct Factors {
    float bh[C], bl[C], eb[C], w[C], total, pad[3];
};

__device__ __forceinline__ void chunk_factors(const float *g, Factors *f, int n, int lane) {
    float x = g[lane];
    x = x > 0.f ? 0.f : x;                   // NaN stays
    x = x < -1e6f ? -1e6f : x;               // 2^(-1e6) is 0 as well; sums stay finite
    double b = lane < n ? (double)x * 1.4426950408889634 : 0.0;
#pragma unroll
    for (int d = 1; d < C; d *= 2) {
        const double y = __shfl_up(b, d);
        if (lane >= d) b += y;
    }
    const double e = __shfl(b, C - 1);
    const float hi = (float)b;
    f->bh[lane] = hi;
    f->bl[lane] = (float)(b - (double)hi);
    f->eb[lane] = exp2_fast(hi);
    f->w[lane] = lane < n ? exp2_fast((float)(e - b)) : 0.f;
    if (lane == 0) f->total = exp2_fast((float)e);
}

__device__ __forceinline__ bool has_non_finite(bf16x8 a, bf16x8 b) {
    const u16x8 m = {0x7fff, 0x7fff, 0x7fff, 0x7fff, 0x7fff, 0x7fff, 0x7fff, 0x7fff};
    const u16x8 x = __builtin_elementwise_max(__builtin_bit_cast(u16x8, a) & m, __builtin_bit_cast(u16x8, b) & m);
    unsigned r = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) r = max(r, (unsigned)x[i]);
    return r >= 0x7f80;
}

// acc += V^T P^T of row block rt when the values hold a non-finite one: earlier
// blocks whole, the diagonal block token by token, added to the rows that see it.
__device__ __forceinline__ f32x4 guarded_pv(f32x4 acc, const bf16x4 *vt, const unsigned char *pl, int rt, int lane) {
    const int r16 = lane & 15, g4 = lane >> 4;
    const bf16x4 z = {};
    for (int st = 0; st <= rt; ++st) {
        const bf16x4 pp = *reinterpret_cast<const bf16x4 *>(pl + (st >> 1) * 1024 + lane * 16 + (st & 1) * 8);
        bf16x4 vv = vt[0];
        vv = st == 1 ? vt[1] : st == 2 ? vt[2] : st == 3 ? vt[3] : vv;
        if (st < rt) {
            acc = mma_k16w(vv, pp, acc);
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

template <int DK, int DVT, int DKS, int NS>
__global__ void __launch_bounds__((Lay<DK, DVT, DKS, NS>::THREADS)) chunk_kernel(ChunkParams p) {
    typedef Lay<DK, DVT, DKS, NS> L;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[L::TOTAL];
    Work wk;
    if (!locate(p, wk)) return;
    const int slot = pool_slot(p.slots, p.num_slots, wk.n);
    if (slot < 0) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nc = (wk.len + C - 1) / C;

    if (wave == L::NW) {  // the streaming wave: it reads no LDS
        const int hk = wk.h / p.rep;
        Stream sm;
        sm.q = static_cast<const unsigned char *>(p.q) + ((int64_t)wk.t0 * p.qs + hk * DK) * 2;
        sm.k = static_cast<const unsigned char *>(p.k) + ((int64_t)wk.t0 * p.ks + hk * DK) * 2;
        sm.v = static_cast<const unsigned char *>(p.v) +
               ((int64_t)wk.t0 * p.vs + (int64_t)wk.h * p.dv + wk.tile * DVT) * 2;
        sm.g = p.g + wk.t0 * p.gs + wk.h;
        sm.qs = p.qs * 2; sm.ks = p.ks * 2; sm.vs = p.vs * 2; sm.gs = p.gs;
        sm.len = wk.len; sm.nc = nc;
        // issued in order g0, then (g of chunk c + 1, chunk c): when chunk c has
        // landed, so has the next chunk's g
        fetch_g<L>(sm, lds, 0, lane);
        for (int c = 0; c < NS - 1; ++c) {
            fetch_g<L>(sm, lds, c + 1, lane);
            fetch<L>(sm, lds, c, lane);
        }
        for (int c = 0; c < nc; ++c) {
            // chunk c has landed when only the NS - 2 chunks behind it are outstanding
            constexpr int AHEAD = (NS - 2) * L::DMAS;
            if (c + NS - 1 < nc) wait_vmcnt<(AHEAD < 63 ? AHEAD : 63)>();
            else wait_vmcnt<0>();
            if (c == 0) bar();  // g0 is there: its factors are formed now
            bar();  // A
            fetch_g<L>(sm, lds, c + NS, lane);
            fetch<L>(sm, lds, c + NS - 1, lane);
            bar();  // B
            if (DKS > 1) bar();  // C
        }
        return;
    }
    Factors *fac = reinterpret_cast<Factors *>(lds + L::B);
    if (wave == L::NW + 1) {  // the decay wave
        for (int c = 0; c < nc; ++c) {
            if (c == 0) {
                bar();
                chunk_factors(reinterpret_cast<const float *>(lds + L::G), fac, min(wk.len, C), lane);
            }
            bar();  // A
            if (c + 1 < nc)
                chunk_factors(reinterpret_cast<const float *>(lds + L::G + ((c + 1) % NS) * 256), fac + ((c + 1) & 1),
                              min(wk.len - (c + 1) * C, C), lane);
            bar();  // B
            if (DKS > 1) bar();  // C
        }
        return;
    }

    const int r16 = lane & 15, g4 = lane >> 4;
    const int ct = wave % L::NCT, hh = wave / L::NCT;
    const int col = wk.tile * DVT + 16 * ct;
    // S[u][e][i]: row 32 (hh UD + u) + 8 g4 + 4 e + i, column col + r16
    f32x4 S[L::UD][2];
    const size_t sbase = ((size_t)slot * p.H + wk.h) * DK * p.dv + (size_t)(32 * hh * L::UD + 8 * g4) * p.dv + col + r16;
#pragma unroll
    for (int u = 0; u < L::UD; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const size_t at = sbase + (size_t)(32 * u + 4 * e + i) * p.dv;
                S[u][e][i] = !p.s_in ? 0.f
                             : p.state_bf16 ? (float)static_cast<const __bf16 *>(p.s_in)[at]
                                            : static_cast<const float *>(p.s_in)[at];
            }

    __bf16 *o = static_cast<__bf16 *>(p.o) + ((size_t)wk.t0 * p.H + wk.h) * p.dv + col + 4 * g4;
    const size_t orow = (size_t)p.H * p.dv;
    unsigned char *pl = lds + L::P;
    const int frow = swz<L::CPR>(r16);
    for (int c = 0; c < nc; ++c) {
        const unsigned char *lq = lds + (c % NS) * L::STAGE, *lk = lq + L::QB, *lv = lk + L::QB;
        const Factors *f = fac + (c & 1);
        const int n = min(wk.len - c * C, C);
        if (c == 0) bar();
        bar();  // A: chunk c and its factors are in LDS
        for (int b = wave; b < 10; b += L::NW) {
            const int rt = b >= 6 ? 3 : b >= 3 ? 2 : b >= 1 ? 1 : 0, st = b - rt * (rt + 1) / 2;
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < DK / 32; ++u) {
                const int off = ((4 * u + g4) ^ frow) * 16;
                acc = mma_k32(*reinterpret_cast<const bf16x8 *>(lk + (16 * st + r16) * (DK * 2) + off),
                              *reinterpret_cast<const bf16x8 *>(lq + (16 * rt + r16) * (DK * 2) + off), acc);
            }
            // lane: token r = 16 rt + r16, keys s = 16 st + 4 g4 + i
            const int r = 16 * rt + r16, s = 16 * st + 4 * g4;
            const float rh = f->bh[r], rl = f->bl[r];
            const f32x4 sh = *reinterpret_cast<const f32x4 *>(f->bh + s), sl = *reinterpret_cast<const f32x4 *>(f->bl + s);
            f32x4 pv;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = acc[i] * exp2_fast((rh - sh[i]) + (rl - sl[i]));
                pv[i] = r >= s + i ? x : 0.f;
            }
            const int pair = (rt < 2 ? rt : 2 * rt - 2) + (st >> 1);
            *reinterpret_cast<bf16x4 *>(pl + pair * 1024 + lane * 16 + (st & 1) * 8) = pack4(pv);
        }
        bar();  // B: P is in LDS
        bf16x4 vt[4];
        {
            const int row = 4 * g4 + (r16 >> 2);
            const int off = ((2 * ct + (r16 >> 1 & 1)) ^ swz<L::CPV>(row)) * 16 + (r16 & 1) * 8;
#pragma unroll
            for (int t = 0; t < 4; ++t) vt[t] = read_tr(lv + (16 * t + row) * (DVT * 2) + off);
        }
        const bool odd = __any(has_non_finite(join8(vt[0], vt[1]), join8(vt[2], vt[3])));
        bf16x8 sb[L::UD];
#pragma unroll
        for (int u = 0; u < L::UD; ++u) sb[u] = join8(pack4(S[u][0]), pack4(S[u][1]));
        const float tot = f->total;

        // partial S^T q of the row block (this wave's part of the state rows)
        auto inter = [&](int rt) {
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < L::UD; ++u)
                acc = mma_k32(sb[u], *reinterpret_cast<const bf16x8 *>(
                                         lq + (16 * rt + r16) * (DK * 2) + ((4 * (hh * L::UD + u) + g4) ^ frow) * 16), acc);
            return acc;
        };
        // the decayed partial sum, P's part, the store
        auto finish = [&](int rt, f32x4 acc, auto guarded) {
            const int r = 16 * rt + r16;
            acc = acc * f->eb[r];
            const unsigned char *pr = pl + (rt < 2 ? rt : 2 * rt - 2) * 1024;
            if constexpr (decltype(guarded)::value) {
                acc = guarded_pv(acc, vt, pr, rt, lane);
            } else {
                const bf16x8 p0 = *reinterpret_cast<const bf16x8 *>(pr + lane * 16);
                const bf16x4 p0l = {p0[0], p0[1], p0[2], p0[3]};
                if (rt == 0) {
                    acc = mma_k16w(vt[0], p0l, acc);
                } else {
                    acc = mma_k32(join8(vt[0], vt[1]), p0, acc);
                    if (rt >= 2) {
                        const bf16x8 p1 = *reinterpret_cast<const bf16x8 *>(pr + 1024 + lane * 16);
                        const bf16x4 p1l = {p1[0], p1[1], p1[2], p1[3]};
                        acc = rt == 2 ? mma_k16w(vt[2], p1l, acc) : mma_k32(join8(vt[2], vt[3]), p1, acc);
                    }
                }
            }
            if (r < n) *reinterpret_cast<bf16x4 *>(o + (size_t)(c * C + r) * orow) = pack4(acc * p.scale);
        };
        auto update = [&]() {
#pragma unroll
            for (int u = 0; u < L::UD; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) S[u][e] = S[u][e] * tot;
#pragma unroll
            for (int kp = 0; kp < 2; ++kp) {
                bf16x8 v3[3];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const f32x4 w = *reinterpret_cast<const f32x4 *>(f->w + 32 * kp + 16 * t + 4 * g4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = (float)vt[2 * kp + t][i] * w[i];
                        const __bf16 a = (__bf16)x;
                        const float y = x - (float)a;
                        const __bf16 b = (__bf16)y;
                        v3[0][4 * t + i] = a;
                        v3[1][4 * t + i] = b;
                        v3[2][4 * t + i] = (__bf16)(y - (float)b);
                    }
                }
                const int row = 4 * g4 + (r16 >> 2), sw = swz<L::CPR>(row);
#pragma unroll
                for (int u = 0; u < L::UD; ++u)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const unsigned char *kr = lk + (32 * kp + row) * (DK * 2) +
                                                  ((4 * (hh * L::UD + u) + (r16 & 3)) ^ sw) * 16 + 8 * e;
                        const bf16x8 kt = join8(read_tr(kr), read_tr(kr + 16 * DK * 2));
#pragma unroll
                        for (int i = 0; i < 3; ++i) S[u][e] = mma_k32(kt, v3[i], S[u][e]);
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if constexpr (DKS == 1) {
            if (odd) {
#pragma unroll 1
                for (int rt = 0; rt < 4; ++rt) finish(rt, inter(rt), std::true_type{});
            } else {
#pragma unroll
                for (int rt = 0; rt < 4; ++rt) {
                    finish(rt, inter(rt), std::false_type{});
                    __builtin_amdgcn_sched_barrier(0);  // operands of one row block at a time
                }
            }
            update();
        } else {
            // row block rt of column tile ct is finished by one of its DKS waves, from
            // the partial sums of all of them in order
            f32x4 *xs = reinterpret_cast<f32x4 *>(lds + L::X) + (size_t)ct * 4 * DKS * 64;
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) xs[(rt * DKS + hh) * 64 + lane] = inter(rt);
            update();
            bar();  // C: the partial sums are in LDS
#pragma unroll 1
            for (int j = 0; j < 4 / DKS; ++j) {
                const int rt = DKS == 4 ? hh : (j == 0 ? hh : 3 - hh);
                f32x4 acc = xs[rt * DKS * 64 + lane];
#pragma unroll
                for (int d = 1; d < DKS; ++d) acc = acc + xs[(rt * DKS + d) * 64 + lane];
                if (odd) finish(rt, acc, std::true_type{});
                else finish(rt, acc, std::false_type{});
            }
        }
    }
    if (!p.s_out) return;
#pragma unroll
    for (int u = 0; u < L::UD; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const size_t at = sbase + (size_t)(32 * u + 4 * e + i) * p.dv;
                if (p.state_bf16) static_cast<__bf16 *>(p.s_out)[at] = (__bf16)S[u][e][i];
                else static_cast<float *>(p.s_out)[at] = S[u][e][i];
            }
}

template <int DK, int DVT, int DKS, int NS> hipError_t launch(ChunkParams p, hipStream_t s) {
    typedef Lay<DK, DVT, DKS, NS> L;
    p.tiles = p.dv / DVT;
    p.units = p.N * (p.H / p.rep);
    const unsigned blocks = (unsigned)((p.units + 7) / 8) * 8 * p.rep * p.tiles;
    hipLaunchKernelGGL((chunk_kernel<DK, DVT, DKS, NS>), dim3(blocks), dim3(L::THREADS), 0, s, p);
    trace("chunk_kernel<%d, %d, %d, %d> grid=(%u) block=%d lds=%d", DK, DVT, DKS, NS, blocks, L::THREADS, L::TOTAL);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linattn_chunks(const kda_linattn_prefill_args *a, hipStream_t s) {
    ChunkParams p = {};
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->log_decay;
    p.s_in = a->state_in; p.s_out = a->state_out; p.o = a->o; p.cu = a->cu_seqlens;
    p.slots = a->state_slots; p.num_slots = a->num_slots;
    p.total = a->total_tokens; p.N = a->num_seqs; p.H = a->num_heads; p.rep = a->num_heads / a->num_k_heads;
    p.qs = a->q_stride; p.ks = a->k_stride; p.vs = a->v_stride;
    p.gs = (a->flags & KDA_F_DECAY_PER_HEAD) ? 0 : a->num_heads;
    p.dv = a->head_dim_v; p.state_bf16 = (a->flags & KDA_F_STATE_BF16) != 0; p.scale = a->scale;
    const int64_t pairs = (int64_t)a->num_seqs * a->num_heads;
    if (a->head_dim_k == 64) {
        if (pairs * (p.dv / 64) >= 256) return p.dv == 128 ? launch<64, 128, 1, 3>(p, s) : launch<64, 64, 1, 3>(p, s);
        return launch<64, 32, 2, 3>(p, s);
    }
    if (pairs * (p.dv / 64) >= 256) return p.dv == 128 ? launch<128, 128, 1, 3>(p, s) : launch<128, 64, 2, 2>(p, s);
    return launch<128, 32, 2, 3>(p, s);
}

}  // namespace kda
