// kda_scan.hip -- the gated scan over packed prompts and its gradients, a channel's
// state a single number: h_t = a_t h_{t-1} + b_t x_t.
//
// The recurrence is linear in the state, so a run of tokens acts on the state before it
// as one step (P, H): h -> P h + H, and runs are joined by (P2 P1, P2 H1 + H2).  A tile
// is S tokens x 3, 7 or 15 waves of 128 channels: a lane owns two neighbouring channels and a
// wave S tokens of them.  For each tile
//   1. every wave forms its rows' step and leaves it in LDS;
//   2. the manager, a wave of its own without rows, joins the steps, finds the state
//      before the tile and leaves each wave the state that it begins from;
//   3. every wave runs the recurrence over its rows and writes them.
// Between waves and tiles decays are handed on as logarithms, and only a whole tile's is
// rounded as a decay: the rounding of every a = 1 - small, the same for every token of a
// steady gate, would grow with the length of the memory.
//
// One pass: a workgroup walks the tiles of one (sequence, 128 channels), the manager keeps
// the state.  Chained: a workgroup takes one tile by ticket, and the state comes from the
// workgroup before it through the workspace (chain_carry).  Either way every element is
// read once and written once: the bound is HBM (figures at the kernels).  Workgroups that
// stay and take tile after tile were slower, also with the next rows on their way (16 ragged
// sequences of 75,926 tokens in all x 4096 channels 430 to 499 us, one tile each 391): a
// ticket taken early waits for a tile that has not begun.
#include <algorithm>

#include "kda_scan.h"

namespace kda {

namespace {

template <int WAVES> struct Shared {
    Tile tile[2];             // of iterations i (i & 1)
    float4 steps[WAVES][64];  // from the waves: log2 P and H; to them: P and H of the rows before theirs
    float2 carry[64];         // the state before the tile
};

// The manager's part.  `edge` is where a sequence's chain begins: its first tile, or for
// the gradients its last.  `first` and `final` are the states there and at the other end.
template <int TILE, bool BACKWARD, bool CHAINED, int WAVES, typename First, typename Final>
__device__ __forceinline__ void manage(const ScanParams &p, Shared<WAVES> &sh, int lane, First first, Final final) {
    const uint32_t taken = CHAINED ? take_ticket(p, lane) : 0;
    const Sequences seq(p, lane);
    float2 running = {0.f, 0.f};
    auto next = [&](const Tile &before) __attribute__((always_inline)) {
        Tile t = before;
        if (before.n >= 0) {  // one pass: the sequence goes on, or ends
            t.index += BACKWARD ? -1 : 1;
            if (CHAINED || t.index < 0 || t.index >= t.count) t.n = -1;
            return t;
        }
        if (CHAINED) {
            t = ticket_tile<TILE, BACKWARD>(p, seq, taken);
        } else {
            t.m = blockIdx.x / p.groups;
            t.group = blockIdx.x - t.m * p.groups;
            seq.fill<TILE>(t.m, t);
            t.index = BACKWARD ? t.count - 1 : 0;
        }
        if (t.slot < 0) t.n = -1;
        if (t.n >= 0 && t.count == 0) {  // no tokens: the state is passed on
            final(t, first(t));
            t.n = -1;
        }
        return t;
    };
    Tile cur = {};
    cur.n = -1;
    cur = next(cur);
    if (lane == 0) sh.tile[0] = cur;
    barrier_lds();
    for (int i = 1; cur.n >= 0; ++i) {
        const int edge = BACKWARD ? cur.count - 1 : 0, done = BACKWARD ? edge - cur.index : cur.index;
        float2 h = done == 0 ? first(cur) : running;
        const Tile after = next(cur);
        if (lane == 0) sh.tile[i & 1] = after;
        barrier_lds();
        float2 sum = {0.f, 0.f}, add = {0.f, 0.f};
#pragma unroll
        for (int q = 0; q < WAVES; ++q) {
            const float4 s = sh.steps[q][lane];
            sh.steps[q][lane] = make_float4(exp2_fast(sum.x), exp2_fast(sum.y), add.x, add.y);
            sum.x += s.x;
            sum.y += s.y;
            add.x = fmaf(exp2_fast(s.x), add.x, s.z);
            add.y = fmaf(exp2_fast(s.y), add.y, s.w);
        }
        const float2 dec = {exp2_fast(sum.x), exp2_fast(sum.y)};
        if (CHAINED) h = chain_carry(p, cur, lane, done, BACKWARD ? 1 : -1, dec, add, h);
        sh.carry[lane] = h;
        barrier_lds();
        running = make_float2(fmaf(dec.x, h.x, add.x), fmaf(dec.y, h.y, add.y));
        if (done == cur.count - 1) final(cur, running);
        cur = after;
    }
}

// The state that the rows at chain position `pos` begin from.
template <int WAVES> __device__ __forceinline__ float2 begin_state(const Shared<WAVES> &sh, int lane, int pos) {
    const float4 s = sh.steps[pos][lane];
    const float2 c = sh.carry[lane];
    return make_float2(fmaf(s.x, c.x, s.z), fmaf(s.y, c.y, s.w));
}

// Byte offset of a lane's channels in a row; past every buffer where there are none.
template <typename T> __device__ __forceinline__ uint32_t lane_offset(const ScanParams &p, const Tile &t, int lane) {
    const int c = t.group * 128 + 2 * lane;
    return c < p.C ? (uint32_t)c * sizeof(T) : RowBuffer<T>::kNowhere;
}

// bf16, inputs not cached, bytes past L2: 1 x 4096 tokens x 8192 channels, log-decays, 208 MB
// (1.03 of the least) in 51 us, 4.1 TB/s (1152 workgroups, 512 at a time: the ramps count);
// 16 sequences of 75,926 tokens x 4096 343 us, 5.45 TB/s.  1 x 65,536 x 4096, pre-activations
// with complement, 1.66 GB in 337 to 357 us, 4.7 to 4.9 TB/s: 126 registers leave a compute
// unit one workgroup, and nothing is on its way while that one computes (VALU slots half
// taken).  Half the rows in 64 registers, two workgroups: 354, and 179 instead of 184 for
// 1 x 32,768 x 4096 log-decays with complement, 223 instead of 194 for pre-activations with norm.
template <typename T, int GATE, int INPUT, int WAVES>
__global__ void __launch_bounds__(64 * (WAVES + 1), scan_occupancy(sizeof(T), false, scan_cheap(GATE, INPUT))) scan_kernel(ScanParams p) {
    typedef Two<T> two;
    constexpr bool CHEAP = scan_cheap(GATE, INPUT), AGAIN = scan_again(sizeof(T), false, CHEAP);
    constexpr bool CHAINED = WAVES == kWavesChained;
    constexpr int S = scan_rows(sizeof(T), false, CHAINED, GATE, INPUT), TILE = S * WAVES;
    __shared__ Shared<WAVES> sh;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    if (wave == WAVES) {
        auto at = [&](const Tile &t) { return (size_t)t.slot * p.C + t.group * 128 + 2 * lane; };
        auto on = [&](const Tile &t) { return t.group * 128 + 2 * lane < p.C; };
        manage<TILE, false, CHAINED, WAVES>(
            p, sh, lane,
            [&](const Tile &t) { return p.state_in && on(t) ? load_state(p.state_in, at(t), p.state_bf16) : float2{0.f, 0.f}; },
            [&](const Tile &t, float2 h) { if (p.state_out && on(t)) store_state(p.state_out, at(t), p.state_bf16, h); });
        return;
    }
    barrier_lds();
    Tile cur = uniform(sh.tile[0]);
    for (int i = 1; cur.n >= 0; ++i) {
        const int rows = min(max(cur.len - cur.index * TILE - wave * S, 0), S);  // of this wave
        const uint32_t off = lane_offset<T>(p, cur, lane);
        const int64_t token = (int64_t)cur.start + cur.index * TILE + wave * S;
        typename two::bits rx[S], rg[S];
        {
            const RowBuffer<T> x(p.x, token, p.xs, p.C, rows), g(p.g, token, p.gs, p.C, rows);
#pragma unroll
            for (int j = S - 1; j >= 0; --j) {
                rg[j] = g.load(off, j);
                rx[j] = x.load(off, j);
            }
        }
        if (rows < S) {
#pragma unroll
            for (int j = 0; j < S; ++j)
                if (j >= rows) {
                    rx[j] = two::both(0.f);
                    rg[j] = two::both(open_gate<GATE>());
                }
        }
        float a[S][2], u[S][2];
        Run<GATE> run[2];
        auto factors = [&](int j, int v) __attribute__((always_inline)) {
            const Factors<GATE, INPUT> f(two::get(rg[j], v));
            a[j][v] = f.a;
            u[j][v] = f.input(two::get(rx[j], v));
            return f;
        };
#pragma unroll
        for (int j = S - 1; j >= 0; --j) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const Factors<GATE, INPUT> f = factors(j, v);
                run[v].before(f, u[j][v]);
            }
        }
        sh.steps[wave][lane] = make_float4(run[0].log2_decay(), run[1].log2_decay(), run[0].add, run[1].add);
        barrier_lds();
        const Tile after = uniform(sh.tile[i & 1]);
        barrier_lds();
        if (AGAIN) {
#pragma unroll
            for (int j = 0; j < S; ++j) {
                two::hold(rg[j]);
                two::hold(rx[j]);
            }
        }
        float2 h = begin_state(sh, lane, wave);
        const RowBuffer<T> o(p.o, token, p.os, p.C, rows);
#pragma unroll
        for (int j = 0; j < S; ++j) {
            if (AGAIN) {
                factors(j, 0);
                factors(j, 1);
            }
            h.x = fmaf(a[j][0], h.x, u[j][0]);
            h.y = fmaf(a[j][1], h.y, u[j][1]);
            o.store(off, j, h.x, h.y);
        }
        cur = after;
    }
}

// The gradients: r_t, what the tokens behind t leave for h_t, runs the other way,
//     dh_t = do_t + r_t,  r_{t-1} = a_t dh_t,
// as steps (P, H) of r -> P r + H with H = sum_t do_t a_first .. a_t.  The chain position
// of a wave counts from the tile's end, that of a tile from the sequence's end.
// bf16: 1 x 4096 x 8192, log-decays, 349 MB in 76 us, 4.6 TB/s; 16 sequences of 92,117 tokens
// x 4096, pre-activations with complement, 4.67 GB (1.03 of the least) in 884 us, 5.3 TB/s.
template <typename T, int GATE, int INPUT, int WAVES>
__global__ void __launch_bounds__(64 * (WAVES + 1), scan_occupancy(sizeof(T), true, scan_cheap(GATE, INPUT))) scan_backward_kernel(ScanParams p) {
    typedef Two<T> two;
    constexpr bool CHEAP = scan_cheap(GATE, INPUT), AGAIN = scan_again(sizeof(T), true, CHEAP);
    constexpr bool CHAINED = WAVES == kWavesChained;
    constexpr int S = scan_rows(sizeof(T), true, CHAINED, GATE, INPUT), TILE = S * WAVES;
    constexpr bool X = INPUT != KDA_INPUT_PLAIN;
    __shared__ Shared<WAVES> sh;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    auto at = [&](const Tile &t) { return (size_t)t.n * p.C + t.group * 128 + 2 * lane; };
    auto on = [&](const Tile &t) { return t.group * 128 + 2 * lane < p.C; };
    if (wave == WAVES) {
        manage<TILE, true, CHAINED, WAVES>(
            p, sh, lane,
            [&](const Tile &t) { return p.dstate_out && on(t) ? *reinterpret_cast<const float2 *>(p.dstate_out + at(t)) : float2{0.f, 0.f}; },
            [&](const Tile &t, float2 r) { if (p.dstate_in && on(t)) *reinterpret_cast<float2 *>(p.dstate_in + at(t)) = r; });
        return;
    }
    const int pos = WAVES - 1 - wave;
    barrier_lds();
    Tile cur = uniform(sh.tile[0]);
    for (int i = 1; cur.n >= 0; ++i) {
        const int t0 = cur.index * TILE + wave * S, rows = min(max(cur.len - t0, 0), S);  // of this wave
        const int first = t0 == 0;
        const uint32_t off = lane_offset<T>(p, cur, lane);
        const int64_t token = (int64_t)cur.start + t0;
        typename two::bits rd[S], rg[S], rh[S], rx[X ? S : 1];
        {
            const RowBuffer<T> d(p.d, token, p.ds, p.C, rows), g(p.g, token, p.gs, p.C, rows);
#pragma unroll
            for (int j = 0; j < S; ++j) {
                rg[j] = g.load(off, j);
                rd[j] = d.load(off, j);
            }
            const RowBuffer<T> h(p.o, token - 1 + first, p.os, p.C, rows);  // the tokens before
            const RowBuffer<T> x(p.x, token, p.xs, p.C, X ? rows : 0);
#pragma unroll
            for (int j = 0; j < S; ++j) {
                rh[j] = h.load(off, j - first);
                if (X) rx[X ? j : 0] = x.load(off, j);
            }
        }
        const float2 h0 = first && p.state_in && on(cur) ? load_state(p.state_in, at(cur), p.state_bf16) : float2{0.f, 0.f};
        if (rows < S) {
#pragma unroll
            for (int j = 0; j < S; ++j)
                if (j >= rows) {
                    rd[j] = two::both(0.f);
                    rg[j] = two::both(open_gate<GATE>());
                }
        }
        Factors<GATE, INPUT> f[S][2];
        Run<GATE> run[2];
#pragma unroll
        for (int j = 0; j < S; ++j) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                f[j][v] = Factors<GATE, INPUT>(two::get(rg[j], v));
                run[v].behind(f[j][v], two::get(rd[j], v));
            }
        }
        sh.steps[pos][lane] = make_float4(run[0].log2_decay(), run[1].log2_decay(), run[0].add, run[1].add);
        barrier_lds();
        const Tile after = uniform(sh.tile[i & 1]);
        barrier_lds();
#pragma unroll
        for (int j = 0; j < S; ++j) {
            two::hold(rd[j]);
            two::hold(rh[j]);
            if (X) two::hold(rx[X ? j : 0]);
            if (AGAIN) two::hold(rg[j]);
        }
        float2 r = begin_state(sh, lane, pos);
        const RowBuffer<T> dx(p.dx, token, p.dxs, p.C, rows), dg(p.dg, token, p.dgs, p.C, rows);
#pragma unroll
        for (int j = S - 1; j >= 0; --j) {
            float m[2] = {r.x, r.y}, ox[2], og[2];
            const float hs[2] = {h0.x, h0.y};
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if (AGAIN) f[j][v] = Factors<GATE, INPUT>(two::get(rg[j], v));
                const float dh = two::get(rd[j], v) + m[v];
                const float before = j == 0 && first ? hs[v] : two::get(rh[j], v);
                f[j][v].gradient(dh, before, X ? two::get(rx[X ? j : 0], v) : 0.f, ox[v], og[v]);
                m[v] = f[j][v].a * dh;  // (a row that only pads has an open gate and no gradient of its own)
            }
            r = make_float2(m[0], m[1]);
            dx.store(off, j, ox[0], ox[1]);
            dg.store(off, j, og[0], og[1]);
        }
        cur = after;
    }
}

// Workspace of the chained schedule: the ticket, the flags [groups][tiles] and the words
// [tiles][groups][128].
struct ChainLayout {
    int64_t flags, words, bytes;  // byte offsets, all of 256
    ChainLayout(int64_t tiles, int64_t groups) {
        flags = 256;
        words = flags + (groups * tiles * 4 + 255) / 256 * 256;
        bytes = words + tiles * groups * 128 * 8;
    }
};

// Marks every word as not yet written, and sets flags and ticket to 0: 5 to 7 us, most of
// them the launch (26 MB for 1 x 65,536 x 4096).  A kernel and no fill of the runtime's,
// which a captured graph does not replay reliably.
__global__ void __launch_bounds__(256) scan_clear_kernel(uint4 *ws, int64_t words, int64_t end) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < end; i += (int64_t)gridDim.x * 256) {
        const uint32_t v = i < words ? 0u : kEmpty;
        ws[i] = make_uint4(v, v, v, v);
    }
}

template <typename T, int GATE, int INPUT, int WAVES> void launch(const ScanParams &p, bool backward, unsigned blocks, hipStream_t s) {
    const dim3 grid(blocks), block(64 * (WAVES + 1));
    if (backward) hipLaunchKernelGGL((scan_backward_kernel<T, GATE, INPUT, WAVES>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((scan_kernel<T, GATE, INPUT, WAVES>), grid, block, 0, s, p);
}
template <typename T, int GATE, int INPUT> void launch(const ScanParams &p, int waves, bool backward, unsigned blocks, hipStream_t s) {
    if (waves == kWavesChained) launch<T, GATE, INPUT, kWavesChained>(p, backward, blocks, s);
    else if (waves == kWavesOnePass) launch<T, GATE, INPUT, kWavesOnePass>(p, backward, blocks, s);
    else launch<T, GATE, INPUT, kWavesShort>(p, backward, blocks, s);
}
template <typename T, int GATE> void launch(const ScanParams &p, int input, int waves, bool backward, unsigned blocks, hipStream_t s) {
    if (input == KDA_INPUT_PLAIN) launch<T, GATE, KDA_INPUT_PLAIN>(p, waves, backward, blocks, s);
    else if (input == KDA_INPUT_COMPLEMENT) launch<T, GATE, KDA_INPUT_COMPLEMENT>(p, waves, backward, blocks, s);
    else launch<T, GATE, KDA_INPUT_NORM>(p, waves, backward, blocks, s);
}

hipError_t launch_any(ScanParams p, const ScanPlan &plan, kda_dtype dt, int gate, int input, bool backward, hipStream_t s) {
    unsigned blocks = (unsigned)((int64_t)p.N * p.groups);
    const int rows = scan_rows(dt == KDA_BF16 ? 2 : 4, backward, plan.chained, gate, input);
    const int waves = plan.chained ? kWavesChained : p.T <= (int64_t)p.N * kWavesShort * rows ? kWavesShort : kWavesOnePass;
    if (plan.chained) {
        p.tiles = (int)plan.tiles;
        char *ws = static_cast<char *>(plan.workspace);
        const ChainLayout at(plan.tiles, p.groups);
        p.ticket = reinterpret_cast<uint32_t *>(ws);
        p.flags = reinterpret_cast<uint32_t *>(ws + at.flags);
        p.words = reinterpret_cast<uint64_t *>(ws + at.words);
        p.polls = spin_limit();
        blocks = (unsigned)(plan.tiles * p.groups);
        const unsigned cb = (unsigned)std::min<int64_t>((at.bytes / 16 + 255) / 256, 2048);
        hipLaunchKernelGGL(scan_clear_kernel, dim3(cb), dim3(256), 0, s, reinterpret_cast<uint4 *>(ws), at.words / 16, at.bytes / 16);
        trace("scan_clear_kernel grid=(%u) block=256", cb);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (dt == KDA_BF16) gate == KDA_GATE_LOG ? launch<__bf16, KDA_GATE_LOG>(p, input, waves, backward, blocks, s)
                                             : launch<__bf16, KDA_GATE_SIGMOID>(p, input, waves, backward, blocks, s);
    else gate == KDA_GATE_LOG ? launch<float, KDA_GATE_LOG>(p, input, waves, backward, blocks, s)
                              : launch<float, KDA_GATE_SIGMOID>(p, input, waves, backward, blocks, s);
    trace("scan%s_kernel<%s> grid=(%u) block=%d", backward ? "_backward" : "", plan.chained ? "chained" : "one pass", blocks, 64 * (waves + 1));
    return hipGetLastError();
}

}  // namespace

int scan_tile(kda_dtype dt, int gate, int input, bool backward) {
    return kWavesChained * scan_rows(dt == KDA_BF16 ? 2 : 4, backward, true, gate, input);
}

size_t scan_chain_bytes(int64_t tiles, int C) { return (size_t)ChainLayout(tiles, ((int64_t)C + 127) / 128).bytes; }

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
