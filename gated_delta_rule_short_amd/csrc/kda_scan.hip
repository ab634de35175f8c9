// kda_scan.hip -- the gated scan over packed prompts and its gradients, a channel's
// state a single number: h_t = a_t h_{t-1} + b_t x_t.
//
// The recurrence is linear in the state, so a run of tokens acts on the state before it
// as one step (P, H): h -> P h + H, and runs are joined by (P2 P1, P2 H1 + H2).  A tile
// is kRows tokens x kWaves waves of 128 channels: a lane owns two neighbouring channels
// and a wave kRows tokens of them.  In a tile
//   1. each wave forms its rows' step from its last row to its first,
//      H = sum_t exp2(l_{t+1} + .. + l_last) u_t,  log2 P = sum l_t, with l = log2 a and
//      u = b x, all rows independent but for a running sum of l;
//   2. the waves' steps are joined through LDS with the state before the tile;
//   3. each wave runs the recurrence over its rows from its own first state.
// Decays are summed as logarithms over a tile, so a decay near 1 loses nothing to the
// rounding of a = 1 - small: that error would grow with the length of the memory.
//
// One pass: a workgroup walks the tiles of one (sequence, 128 channels).  Chained: a
// workgroup takes one tile and waits for the state before it (see chain_carry).  Either
// way every element is read once and written once: the bound is HBM.
#include <algorithm>

#include "kda_scan.h"

namespace kda {

namespace {

// From the state `h` before the tile: the state before chain position `pos`, and in h the
// one behind the tile (the whole tile's decay rounded once, as chain_carry does).
template <int WAVES>
__device__ __forceinline__ void join(const float4 (*steps)[64], int lane, int pos, float2 &h, float2 &mine) {
    float2 sum = {0.f, 0.f}, add = {0.f, 0.f};
#pragma unroll
    for (int q = 0; q < WAVES; ++q) {
        if (q == pos) mine = make_float2(fmaf(exp2_fast(sum.x), h.x, add.x), fmaf(exp2_fast(sum.y), h.y, add.y));
        append(steps[q][lane], sum, add);
    }
    h = make_float2(fmaf(exp2_fast(sum.x), h.x, add.x), fmaf(exp2_fast(sum.y), h.y, add.y));
}

template <typename T, int GATE, int INPUT, bool CHAINED>
__global__ void __launch_bounds__(64 * kWaves, sizeof(T) == 2 ? 4 : 2) scan_kernel(ScanParams p) {
    typedef typename Pair<T>::vec vec;
    constexpr int S = kRows, TILE = S * kWaves;
    __shared__ float4 steps[2][kWaves][64];
    __shared__ float2 carry[64];
    __shared__ TileId shared_id;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const TileId id = CHAINED ? chained_tile<TILE>(p, wave, lane, &shared_id, false) : whole_sequence(p);
    if (id.n < 0) return;
    const int slot = pool_slot(p.slots, p.num_slots, id.n);
    if (slot < 0) return;
    const int c = id.group * 128 + 2 * lane;
    const bool on = c < p.C;
    const int cl = on ? c : p.C - 2;
    const size_t srow = (size_t)slot * p.C + cl;
    const int tiles = (int)((id.len + TILE - 1) / TILE);

    vec rx[S], rg[S];
    auto load = [&](int i) __attribute__((always_inline)) {
        const int64_t t0 = (int64_t)i * TILE + wave * S;
#pragma unroll
        for (int j = 0; j < S; ++j) {
            const int64_t t = id.start + min(t0 + j, id.len - 1);
            rx[j] = *reinterpret_cast<const vec *>(static_cast<const T *>(p.x) + t * p.xs + cl);
            rg[j] = *reinterpret_cast<const vec *>(static_cast<const T *>(p.g) + t * p.gs + cl);
        }
    };
    float2 h = {0.f, 0.f};
    const int first = CHAINED ? id.index : 0, end = CHAINED ? min(id.index + 1, tiles) : tiles;
    if (first < end) load(first);
    if (p.state_in && first == 0) h = load_state(p.state_in, srow, p.state_bf16);
    for (int i = first; i < end; ++i) {
        const int64_t t0 = (int64_t)i * TILE + wave * S;
        float l[S][2], u[S][2];
#pragma unroll
        for (int j = 0; j < S; ++j) {
            const bool in = t0 + j < id.len;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const Factors<GATE, INPUT> f(to_f32(rg[j][v]));
                l[j][v] = in ? f.l : 0.f;
                u[j][v] = in ? f.input(to_f32(rx[j][v])) : 0.f;
            }
        }
        if (!CHAINED && i + 1 < end) load(i + 1);
        float sum[2] = {0.f, 0.f}, add[2] = {u[S - 1][0], u[S - 1][1]};
#pragma unroll
        for (int j = S - 1; j >= 0; --j)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if (j < S - 1) add[v] = fmaf(u[j][v], exp2_fast(sum[v]), add[v]);
                sum[v] += l[j][v];
            }
        float4(*st)[64] = steps[CHAINED ? 0 : i & 1];
        st[wave][lane] = make_float4(sum[0], sum[1], add[0], add[1]);
        __syncthreads();
        float2 mine = {0.f, 0.f};
        if (CHAINED) {
            if (wave == 0) {
                const float2 before = chain_carry<kWaves>(p, id, lane, 0, tiles, st, h);
                carry[lane] = before;
                float2 after = before;
                if (i == tiles - 1 && p.state_out) {
                    join<kWaves>(st, lane, 0, after, mine);
                    if (on) store_state(p.state_out, srow, p.state_bf16, after);
                }
            }
            __syncthreads();
            h = carry[lane];
        }
        join<kWaves>(st, lane, wave, h, mine);
        T *o = static_cast<T *>(p.o) + (id.start + t0) * p.os + cl;
#pragma unroll
        for (int j = 0; j < S; ++j) {
            mine.x = fmaf(exp2_fast(l[j][0]), mine.x, u[j][0]);
            mine.y = fmaf(exp2_fast(l[j][1]), mine.y, u[j][1]);
            if (t0 + j < id.len && on) Pair<T>::store(o + j * p.os, mine.x, mine.y);
        }
    }
    // (a chained tile's state went out with its carry; a sequence without tokens passes its own on)
    if (p.state_out && on && wave == 0 && (!CHAINED || tiles == 0)) store_state(p.state_out, srow, p.state_bf16, h);
}

// The gradients: r_t, what the tokens behind t leave for h_t, runs the other way,
//     dh_t = do_t + r_t,  r_{t-1} = a_t dh_t,
// as steps (P, H) of r -> P r + H with H = sum_t do_t exp2(l_first + .. + l_t).  The chain
// position of a wave counts from the tile's end, that of a tile from the sequence's end.
template <typename T, int GATE, int INPUT, bool CHAINED>
__global__ void __launch_bounds__(64 * kWaves, sizeof(T) == 2 ? 4 : 2) scan_backward_kernel(ScanParams p) {
    typedef typename Pair<T>::vec vec;
    constexpr int S = sizeof(T) == 2 ? kRows : kRows / 2, TILE = S * kWaves;
    constexpr bool X = INPUT != KDA_INPUT_PLAIN;
    __shared__ float4 steps[2][kWaves][64];
    __shared__ float2 carry[64];
    __shared__ TileId shared_id;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const TileId id = CHAINED ? chained_tile<TILE>(p, wave, lane, &shared_id, true) : whole_sequence(p);
    if (id.n < 0) return;
    const int c = id.group * 128 + 2 * lane;
    const bool on = c < p.C;
    const int cl = on ? c : p.C - 2;
    const size_t srow = (size_t)id.n * p.C + cl;
    const int tiles = (int)((id.len + TILE - 1) / TILE);

    vec rd[S], rg[S], rh[S], rx[X ? S : 1];
    auto load = [&](int i) __attribute__((always_inline)) {
        const int64_t t0 = (int64_t)i * TILE + wave * S;
#pragma unroll
        for (int j = 0; j < S; ++j) {
            const int64_t t = id.start + min(t0 + j, id.len - 1);
            rd[j] = *reinterpret_cast<const vec *>(static_cast<const T *>(p.d) + t * p.ds + cl);
            rg[j] = *reinterpret_cast<const vec *>(static_cast<const T *>(p.g) + t * p.gs + cl);
            rh[j] = *reinterpret_cast<const vec *>(static_cast<const T *>(p.o) + max(t - 1, id.start) * p.os + cl);
            if (X) rx[j] = *reinterpret_cast<const vec *>(static_cast<const T *>(p.x) + t * p.xs + cl);
        }
    };
    float2 r = {0.f, 0.f}, h0 = {0.f, 0.f};
    const int last = CHAINED ? min(id.index, tiles - 1) : tiles - 1, end = CHAINED ? id.index : 0;
    if (last >= end) load(last);
    if (p.dstate_out && last == tiles - 1) r = *reinterpret_cast<const float2 *>(p.dstate_out + srow);
    if (p.state_in && end == 0) h0 = load_state(p.state_in, srow, p.state_bf16);
    for (int i = last; i >= end; --i) {
        const int64_t t0 = (int64_t)i * TILE + wave * S;
        float sum[2] = {0.f, 0.f}, add[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < S; ++j)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const bool in = t0 + j < id.len;
                const Factors<GATE, INPUT> f(to_f32(rg[j][v]));
                sum[v] += in ? f.l : 0.f;
                add[v] = fmaf(in ? to_f32(rd[j][v]) : 0.f, exp2_fast(sum[v]), add[v]);
            }
        const int pos = kWaves - 1 - wave;
        float4(*st)[64] = steps[CHAINED ? 0 : i & 1];
        st[pos][lane] = make_float4(sum[0], sum[1], add[0], add[1]);
        __syncthreads();
        float2 mine = {0.f, 0.f};
        if (CHAINED) {
            if (wave == 0) {
                const float2 before = chain_carry<kWaves>(p, id, lane, tiles - 1, tiles, st, r);
                carry[lane] = before;
                float2 after = before;
                if (i == 0 && p.dstate_in) {
                    join<kWaves>(st, lane, 0, after, mine);
                    if (on) *reinterpret_cast<float2 *>(p.dstate_in + srow) = after;
                }
            }
            __syncthreads();
            r = carry[lane];
        }
        join<kWaves>(st, lane, pos, r, mine);
        T *dx = static_cast<T *>(p.dx) + (id.start + t0) * p.dxs + cl;
        T *dg = static_cast<T *>(p.dg) + (id.start + t0) * p.dgs + cl;
#pragma unroll
        for (int j = S - 1; j >= 0; --j) {
            const bool in = t0 + j < id.len;
            float m[2] = {mine.x, mine.y}, ox[2], og[2];
            const float hs[2] = {h0.x, h0.y};
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const Factors<GATE, INPUT> f(to_f32(rg[j][v]));
                const float dh = to_f32(rd[j][v]) + m[v], a = exp2_fast(f.l);
                const float before = t0 + j == 0 ? hs[v] : to_f32(rh[j][v]);
                f.gradient(a, dh, before, X ? to_f32(rx[X ? j : 0][v]) : 0.f, ox[v], og[v]);
                if (in) m[v] = a * dh;
            }
            mine = make_float2(m[0], m[1]);
            if (in && on) {
                Pair<T>::store(dx + j * p.dxs, ox[0], ox[1]);
                Pair<T>::store(dg + j * p.dgs, og[0], og[1]);
            }
        }
        if (!CHAINED && i > end) load(i - 1);
    }
    if (p.dstate_in && on && wave == 0 && (!CHAINED || tiles == 0))
        *reinterpret_cast<float2 *>(p.dstate_in + srow) = r;
}

// Marks every word of the workspace as not yet written and sets the ticket to 0.
__global__ void __launch_bounds__(256) scan_clear_kernel(uint4 *words, int64_t count, uint32_t *ticket) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256)
        words[i] = make_uint4(kEmpty, kEmpty, kEmpty, kEmpty);
    if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
}

template <typename T, int GATE, int INPUT> void launch(const ScanParams &p, bool chained, bool backward, unsigned blocks, hipStream_t s) {
    const dim3 grid(blocks), block(64 * kWaves);
    if (backward) {
        if (chained) hipLaunchKernelGGL((scan_backward_kernel<T, GATE, INPUT, true>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((scan_backward_kernel<T, GATE, INPUT, false>), grid, block, 0, s, p);
    } else {
        if (chained) hipLaunchKernelGGL((scan_kernel<T, GATE, INPUT, true>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((scan_kernel<T, GATE, INPUT, false>), grid, block, 0, s, p);
    }
}
template <typename T, int GATE> void launch(const ScanParams &p, int input, bool chained, bool backward, unsigned blocks, hipStream_t s) {
    if (input == KDA_INPUT_PLAIN) launch<T, GATE, KDA_INPUT_PLAIN>(p, chained, backward, blocks, s);
    else if (input == KDA_INPUT_COMPLEMENT) launch<T, GATE, KDA_INPUT_COMPLEMENT>(p, chained, backward, blocks, s);
    else launch<T, GATE, KDA_INPUT_NORM>(p, chained, backward, blocks, s);
}

hipError_t launch_any(ScanParams p, const ScanPlan &plan, kda_dtype dt, int gate, int input, bool backward, hipStream_t s) {
    unsigned blocks = (unsigned)((int64_t)p.N * p.groups);
    if (plan.chained) {
        p.tiles = plan.tiles;
        p.ticket = static_cast<uint32_t *>(plan.workspace);
        p.words = reinterpret_cast<uint64_t *>(static_cast<char *>(plan.workspace) + 256);
        p.polls = spin_limit();
        blocks = (unsigned)(plan.tiles * p.groups);
        const int64_t count = plan.tiles * p.groups * 64;
        const unsigned cb = (unsigned)std::min<int64_t>((count + 255) / 256, 4096);
        hipLaunchKernelGGL(scan_clear_kernel, dim3(cb), dim3(256), 0, s, reinterpret_cast<uint4 *>(p.words), count, p.ticket);
        trace("scan_clear_kernel grid=(%u) block=256", cb);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (dt == KDA_BF16) gate == KDA_GATE_LOG ? launch<__bf16, KDA_GATE_LOG>(p, input, plan.chained, backward, blocks, s)
                                             : launch<__bf16, KDA_GATE_SIGMOID>(p, input, plan.chained, backward, blocks, s);
    else gate == KDA_GATE_LOG ? launch<float, KDA_GATE_LOG>(p, input, plan.chained, backward, blocks, s)
                              : launch<float, KDA_GATE_SIGMOID>(p, input, plan.chained, backward, blocks, s);
    trace("scan%s_kernel<%s> grid=(%u) block=%d", backward ? "_backward" : "", plan.chained ? "chained" : "one pass", blocks, 64 * kWaves);
    return hipGetLastError();
}

}  // namespace

int scan_tile(kda_dtype dt, bool backward) { return kWaves * (backward && dt == KDA_F32 ? kRows / 2 : kRows); }

hipError_t launch_gated_scan(const kda_gated_scan_args *a, const ScanPlan &plan, hipStream_t s) {
    ScanParams p = {};
    p.x = a->x; p.g = a->gate; p.o = a->o;
    p.xs = a->x_stride; p.gs = a->gate_stride; p.os = a->o_stride;
    p.state_in = a->state_in; p.state_out = a->state_out; p.state_bf16 = (a->flags & KDA_F_STATE_BF16) != 0;
    p.slots = a->state_slots; p.num_slots = a->num_slots;
    p.cu = a->cu_seqlens; p.T = a->total_tokens; p.N = a->num_seqs; p.C = a->channels;
    p.groups = (a->channels + 127) / 128;
    return launch_any(p, plan, a->dtype, a->gate_kind, a->input_kind, false, s);
}

hipError_t launch_gated_scan_backward(const kda_gated_scan_backward_args *a, const ScanPlan &plan, hipStream_t s) {
    ScanParams p = {};
    p.d = a->d_o; p.x = a->x; p.g = a->gate; p.o = const_cast<void *>(a->o); p.dx = a->dx; p.dg = a->dgate;
    p.ds = a->d_o_stride; p.xs = a->x_stride; p.gs = a->gate_stride; p.os = a->o_stride;
    p.dxs = a->dx_stride; p.dgs = a->dgate_stride;
    p.state_in = a->state_in; p.state_bf16 = (a->flags & KDA_F_STATE_BF16) != 0;
    p.dstate_out = a->dstate_out; p.dstate_in = a->dstate_in;
    p.cu = a->cu_seqlens; p.T = a->total_tokens; p.N = a->num_seqs; p.C = a->channels;
    p.groups = (a->channels + 127) / 128;
    return launch_any(p, plan, a->dtype, a->gate_kind, a->input_kind, true, s);
}

}  // namespace kda
