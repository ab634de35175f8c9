// kda_linattn_f32.hip -- chunked linear attention with one decay per head for fp32
// tokens.
//
// The sums are those of kda_linattn.hip over chunks of 32 tokens, on the fp32 matrix
// instructions (no operand is rounded; at 157 TFLOP/s the chip's fp32 rate is a
// sixteenth of its bf16 rate, so a shorter chunk with fewer products inside it pays).
// Those instructions are the bound of large calls: 16 sequences of 4096 tokens x 64 heads
// x 128 x 128, 354 GFLOP with P formed for each half of the columns, take 3.4 to 3.5 ms, 104
// to 101 TFLOP/s of the 143 that a large fp32 product reaches; with few heads the bound is a
// chunk's chain of three barriers, 3.2 us, which segments shorten.
// A workgroup carries 32 or 64 columns of a (sequence, head) state, two waves to a tile
// of 16: each makes the outputs of one block of 16 tokens, and holds the state rows of
// every second 16-row tile.  The state reaches the other waves, and P the outputs,
// through LDS in operand order; q, k, v and g of the next chunk are loaded into
// registers while the current one is worked on.
#include <type_traits>

#include "kda_linattn.h"

namespace kda {

namespace {

constexpr int C = 32;

__device__ __forceinline__ bool finite4(f32x4 x) {
    const f32x4 z = x * 0.f;  // NaN where x is not finite
    return (z.x + z.y) + (z.z + z.w) == 0.f;
}

// x if it is finite, or (BAD) if it is not; else zero.
template <bool BAD> __device__ __forceinline__ float part_of(float x) {
    return (x * 0.f == 0.f) != BAD ? x : 0.f;
}

// OUT false: a segment's state alone, without q, P and outputs.
template <int DK, int DVT, bool OUT>
__global__ void __launch_bounds__(8 * DVT) chunk_f32_kernel(ChunkParams p) {
    constexpr int NCT = DVT / 16, NW = 2 * NCT;  // column tiles, waves
    constexpr int VP = DVT + 4;
    constexpr int QP = DK + 4;          // row pitch: rows 4 apart fall on different banks
    constexpr int QN = DK / DVT;        // 16-byte pieces of a 32 x DK tensor per thread
    constexpr int NT = DK / 16, NH = NT / 2;  // 16-row tiles of the state, and per wave
    __shared__ __attribute__((aligned(16))) float lq[C * QP], lk[C * QP], lv[C * VP];
    __shared__ f32x4 lp[3][64];         // P blocks (0,0), (1,0), (1,1)
    __shared__ f32x4 ls[NCT][NT][64];     // the state, operand order
    __shared__ Factors fac;
    __shared__ int bad[NW];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g4 = lane >> 4, rt = wave / NCT, ct = wave % NCT;
    Work wk;
    if (!locate(p, wk, lane)) return;
    if (!OUT && wk.j + 1 >= wk.nseg) return;  // nothing starts from the last segment
    const int slot = pool_slot(p.slots, p.num_slots, wk.n);
    if (slot < 0) return;
    const int h = wk.h, tile = wk.tile, len = wk.len, nc = (len + C - 1) / C;
    const int64_t t0 = wk.t0;
    const float *q = static_cast<const float *>(p.q) + t0 * p.qs + (int64_t)(h / p.rep) * DK;
    const float *k = static_cast<const float *>(p.k) + t0 * p.ks + (int64_t)(h / p.rep) * DK;
    const float *v = static_cast<const float *>(p.v) + t0 * p.vs + (int64_t)h * p.dv + tile * DVT;
    const float *g = p.g + t0 * p.gs + h;
    float *o = static_cast<float *>(p.o) + ((size_t)t0 * p.H + h) * p.dv + tile * DVT + 16 * ct + 4 * g4;

    // state rows 16 (rt + 2 j) + 4 g4 + i, column r16 of tile ct
    f32x4 S[NH];
    const size_t sbase = (((size_t)slot * p.H + h) * DK + 16 * rt + 4 * g4) * p.dv + tile * DVT + 16 * ct + r16;
    auto read = [&](auto *x) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NH; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[j][i] = to_f32(x[sbase + (size_t)(32 * j + i) * p.dv]);
    };
    // where a segment starts from: see the workspace of kda_linattn.hip
    float *ws = p.ws + ((size_t)wk.s * p.H + h) * DK * p.dv + (size_t)(tile * NW + wave) * NH * 256 + lane * 4;
    const size_t next = (size_t)p.H * DK * p.dv;
    if (OUT && wk.nseg > 1) {
        const int first = p.joined || wk.j < 2 ? 0 : wk.j - 1;
#pragma unroll
        for (int j = 0; j < NH; ++j) S[j] = *reinterpret_cast<const f32x4 *>(ws - first * next + j * 256);
#pragma unroll 2
        for (int b = first - 1; b >= 0; --b) {
            const float x = p.wdec[(size_t)(wk.s - b - 1) * p.H + h];
#pragma unroll
            for (int j = 0; j < NH; ++j) S[j] = S[j] * x + *reinterpret_cast<const f32x4 *>(ws - b * next + j * 256);
        }
    } else if (!p.s_in || wk.j > 0) {
#pragma unroll
        for (int j = 0; j < NH; ++j) S[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    } else if (p.state_bf16) {
        read(static_cast<const __bf16 *>(p.s_in));
    } else {
        read(static_cast<const float *>(p.s_in));
    }
    if (!OUT && wk.j == 0) {
#pragma unroll
        for (int j = 0; j < NH; ++j) *reinterpret_cast<f32x4 *>(ws + j * 256) = S[j];
    }
    if (OUT) {
#pragma unroll
        for (int j = 0; j < NH; ++j) ls[ct][rt + 2 * j][lane] = S[j];
    }

    // this thread's pieces of the next chunk (zeros past the sequence)
    f32x4 nq[QN], nk[QN], nv;
    float ng = 0.f;
    const int vr = tid / (DVT / 4), vc = 4 * (tid % (DVT / 4));
    auto load = [&](int c) __attribute__((always_inline)) {
        const f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < QN; ++i) {
            const int e = tid + 64 * NW * i, r = c * C + e / (DK / 4), d = 4 * (e % (DK / 4));
            if (OUT) nq[i] = r < len ? *reinterpret_cast<const f32x4 *>(q + r * p.qs + d) : z;
            nk[i] = r < len ? *reinterpret_cast<const f32x4 *>(k + r * p.ks + d) : z;
        }
        nv = c * C + vr < len ? *reinterpret_cast<const f32x4 *>(v + (c * C + vr) * p.vs + vc) : z;
        if (wave == 3) ng = lane < C && c * C + lane < len ? g[(c * C + lane) * p.gs] : 0.f;
    };
    float kept = 1.f;  // the decays of all chunks
    if (nc > 0) load(0);
    for (int c = 0; c < nc; ++c) {
        const int m = min(len - c * C, C);
#pragma unroll
        for (int i = 0; i < QN; ++i) {
            const int e = tid + 64 * NW * i, at = e / (DK / 4) * QP + 4 * (e % (DK / 4));
            if (OUT) *reinterpret_cast<f32x4 *>(lq + at) = nq[i];
            *reinterpret_cast<f32x4 *>(lk + at) = nk[i];
        }
        *reinterpret_cast<f32x4 *>(lv + vr * VP + vc) = nv;
        const bool some = __any(!finite4(nv));
        if (lane == 0) bad[wave] = some;
        const float gc = ng;
        bar();
        if (c + 1 < nc) load(c + 1);

        // values of column r16, tokens 16 st + 4 g4 + i
        f32x4 vt[2];
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int i = 0; i < 4; ++i) vt[st][i] = lv[(16 * st + 4 * g4 + i) * VP + 16 * ct + r16];
        // P block of waves 0..2: row block pr, key block ps; wave 3 forms the factors
        const int pr = wave > 0, ps = wave > 1;
        f32x4 d = {0.f, 0.f, 0.f, 0.f}, acc = d;
        if (wave == 3) {
            chunk_factors(gc, &fac, m, lane);
        } else if (OUT && wave < 3) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const f32x4 a = *reinterpret_cast<const f32x4 *>(lk + (16 * ps + r16) * QP + 16 * t + 4 * g4);
                const f32x4 b = *reinterpret_cast<const f32x4 *>(lq + (16 * pr + r16) * QP + 16 * t + 4 * g4);
#pragma unroll
                for (int i = 0; i < 4; ++i) d = mma_f32(a[i], b[i], d);
            }
        }
        if (OUT) {
            // S^T q of this wave's token block and column tile
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const f32x4 a = ls[ct][t][lane];
                const f32x4 b = *reinterpret_cast<const f32x4 *>(lq + (16 * rt + r16) * QP + 16 * t + 4 * g4);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc = mma_f32(a[i], b[i], acc);
            }
        }
        bar();
        if constexpr (OUT) {
        acc = acc * fac.eb[16 * rt + r16];
        if (wave < 3) {
            const int r = 16 * pr + r16, s = 16 * ps + 4 * g4;
            const float rh = fac.bh[r], rl = fac.bl[r];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = d[i] * exp2_fast((rh - fac.bh[s + i]) + (rl - fac.bl[s + i]));
                d[i] = r >= s + i ? x : 0.f;
            }
            lp[wave][lane] = d;
        }
        bar();
        const f32x4 p1 = lp[rt][lane], p2 = lp[2][lane];  // (rt, 0), (1, 1)
        // a value that is not finite is left out of the products, where zeros of the
        // future would not stay zeros, and added to the rows that see it
        bool odd = false;
#pragma unroll
        for (int i = 0; i < NW; ++i) odd |= bad[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = mma_f32(odd ? part_of<false>(vt[0][i]) : vt[0][i], p1[i], acc);
        if (rt == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = mma_f32(odd ? part_of<false>(vt[1][i]) : vt[1][i], p2[i], acc);
        }
        if (odd) {
            for (int st = 0; st <= rt; ++st) {
                const f32x4 pp = st ? p2 : p1, vv = st ? vt[1] : vt[0];
                for (int s = 0; s < 16; ++s) {
                    // the key slot of this token alone: lanes of group s / 4, element s % 4
                    const int i0 = s & 3;
                    const float x = part_of<true>(i0 == 0 ? vv[0] : i0 == 1 ? vv[1] : i0 == 2 ? vv[2] : vv[3]);
                    const float y = i0 == 0 ? pp[0] : i0 == 1 ? pp[1] : i0 == 2 ? pp[2] : pp[3];
                    const f32x4 e = mma_f32(g4 == s >> 2 ? x : 0.f, g4 == s >> 2 ? y : 0.f, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] += (st < rt || r16 >= s) ? e[i] : 0.f;
                }
            }
        }
        const int t = c * C + 16 * rt + r16;
        if (t < len) *reinterpret_cast<f32x4 *>(o + (size_t)t * p.H * p.dv) = acc * p.scale;

        }
        // the state over the chunk
        f32x4 w0 = *reinterpret_cast<const f32x4 *>(fac.w + 4 * g4) * vt[0];
        f32x4 w1 = *reinterpret_cast<const f32x4 *>(fac.w + 16 + 4 * g4) * vt[1];
        const float tot = fac.total;
#pragma unroll
        for (int j = 0; j < NH; ++j) {
            const float *kr = lk + 4 * g4 * QP + 16 * (rt + 2 * j) + r16;
            S[j] = S[j] * tot;
#pragma unroll
            for (int i = 0; i < 4; ++i) S[j] = mma_f32(kr[i * QP], w0[i], S[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) S[j] = mma_f32(kr[(16 + i) * QP], w1[i], S[j]);
            if (OUT) ls[ct][rt + 2 * j][lane] = S[j];
        }
        if (!OUT) kept *= tot;
        bar();
    }
    if constexpr (!OUT) {
        ws += next;  // what the next segment starts from
#pragma unroll
        for (int j = 0; j < NH; ++j) *reinterpret_cast<f32x4 *>(ws + j * 256) = S[j];
        if (tid == 0 && tile == 0) p.wdec[(size_t)wk.s * p.H + h] = kept;
        return;
    }
    if (wk.j + 1 < wk.nseg) return;
    if (!p.s_out) return;
    auto write = [&](auto *x) __attribute__((always_inline)) {
        typedef typename std::remove_pointer<decltype(x)>::type E;
#pragma unroll
        for (int j = 0; j < NH; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[sbase + (size_t)(32 * j + i) * p.dv] = from_f32<E>(S[j][i]);
    };
    if (p.state_bf16) write(static_cast<__bf16 *>(p.s_out));
    else write(static_cast<float *>(p.s_out));
}

template <int DVT, bool OUT> hipError_t launch(ChunkParams p, int dk, hipStream_t s) {
    p.tiles = p.dv / DVT;
    const unsigned blocks = (unsigned)((p.units + 7) / 8) * 8 * p.rep * p.tiles;
    if (dk == 64) hipLaunchKernelGGL((chunk_f32_kernel<64, DVT, OUT>), dim3(blocks), dim3(8 * DVT), 0, s, p);
    else hipLaunchKernelGGL((chunk_f32_kernel<128, DVT, OUT>), dim3(blocks), dim3(8 * DVT), 0, s, p);
    trace("chunk_f32_kernel<%d, %d, %d> grid=(%u) block=%d", dk, DVT, (int)OUT, blocks, 8 * DVT);
    return hipGetLastError();
}
template <int DVT> hipError_t launch(ChunkParams &p, const kda_linattn_prefill_args *a, const LinattnPlan &plan,
                                     hipStream_t s) {
    if (plan.tokens) {
        use_segments(p, a, plan);
        hipError_t e = launch<DVT, false>(p, a->head_dim_k, s);
        if (e != hipSuccess) return e;
        e = p.joined ? launch_segment_scan(p, a->head_dim_k * p.dv, s) : hipSuccess;
        if (e != hipSuccess) return e;
    }
    return launch<DVT, true>(p, a->head_dim_k, s);
}

}  // namespace

hipError_t launch_linattn_f32(const kda_linattn_prefill_args *a, const LinattnPlan &plan, hipStream_t s) {
    ChunkParams p = chunk_params(a);
    p.units = (plan.tokens ? (int)plan.segments : p.N) * a->num_k_heads;
    // 32 columns while a compute unit has one workgroup at most; beyond it 64, which form
    // P half as often.  dk = dv = 128, one pass, us (32/64 columns): 16 heads of 2048
    // tokens 211/257, 128 heads of 256 tokens 47/41, 1024 heads of 4096 4638/3505.  The
    // segment numbers that several sequences leave unused crowd the others on fewer units:
    // two passes, 4096 tokens x 8 heads, 256 workgroups of 64 columns: one sequence 66/61,
    // four 66/88; dk 64 45/44 and 50/58.
    const int64_t states = (plan.tokens ? p.total / plan.tokens : p.N) * (int64_t)p.H;
    const int64_t narrow = plan.tokens && p.N > 1 ? 256 : 128;
    return states * (p.dv / 64) > narrow ? launch<64>(p, a, plan, s) : launch<32>(p, a, plan, s);
}

}  // namespace kda
