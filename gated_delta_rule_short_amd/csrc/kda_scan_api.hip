// kda_scan_api.hip -- the extern "C" entry points of the gated scan and of the norm with
// the residual's addition (declared in kda.h).
//
// Every argument is checked on the host before anything is enqueued, as in
// kda_api.hip; the library allocates nothing and never synchronises the stream.
#include <algorithm>
#include <cmath>

#include "kda.h"
#include "kda_checks.h"
#include "kda_internal.h"

namespace {

using namespace kda::checks;

// A launch holds fewer than 2^32 threads, up to 1024 of them in a workgroup.
constexpr int64_t kMaxGroups = (int64_t)1 << 22;
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - 512;

int64_t channel_groups(int32_t C) { return ((int64_t)C + 127) / 128; }

kda_status check_scan(int32_t N, int32_t C, kda_dtype dt, int gate, int input, uint32_t flags) {
    if (N < 1) return fail(KDA_ERR_INVALID_ARG, "num_seqs = %d, must be >= 1", N);
    if (C < 1 || C % 8) return fail(KDA_ERR_INVALID_ARG, "channels = %d, must be a positive multiple of 8", C);
    if (dt != KDA_F32 && dt != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    if (gate != KDA_GATE_LOG && gate != KDA_GATE_SIGMOID)
        return fail(KDA_ERR_INVALID_ARG, "gate_kind %d: use a KDA_GATE_* value", gate);
    if (input != KDA_INPUT_PLAIN && input != KDA_INPUT_COMPLEMENT && input != KDA_INPUT_NORM)
        return fail(KDA_ERR_INVALID_ARG, "input_kind %d: use a KDA_INPUT_* value", input);
    if (flags & ~(uint32_t)KDA_F_STATE_BF16) return fail(KDA_ERR_UNSUPPORTED, "unsupported flags 0x%x", flags);
    if (N * channel_groups(C) >= kMaxGroups) return fail(KDA_ERR_INVALID_ARG, "num_seqs * channels too large");
    return KDA_OK;
}

// Tokens a wave's buffer spans at once, times this many elements, stay below 2^31 bytes.
constexpr int64_t kMaxStride = (int64_t)1 << 22;
kda_status check_strides(const Rows *r, int n) {
    for (int i = 0; i < n; ++i)
        if (r[i].stride > kMaxStride)
            return fail(KDA_ERR_UNSUPPORTED, "%s_stride = %lld, at most %lld", r[i].name, (long long)r[i].stride, (long long)kMaxStride);
    return KDA_OK;
}

// Checks of the packed tokens, shared by the prompts and their gradients.
template <typename A> kda_status check_tokens(const A &a) {
    const int64_t T = a.total_tokens;
    if (T < 0) return fail(KDA_ERR_INVALID_ARG, "total_tokens < 0");
    // token positions inside a sequence are 32-bit in the kernels, up to a tile past its end
    if (T > kMaxTokens) return fail(KDA_ERR_INVALID_ARG, "total_tokens too large");
    if (a.cu_seqlens_host && !a.cu_seqlens) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens_host needs cu_seqlens");
    if (!a.cu_seqlens && T % a.num_seqs)
        return fail(KDA_ERR_INVALID_ARG, "cu_seqlens NULL needs total_tokens %% num_seqs == 0");
    if (a.schedule != KDA_SCHEDULE_AUTO && a.schedule != KDA_SCHEDULE_ONE_PASS && a.schedule != KDA_SCHEDULE_CHAINED)
        return fail(KDA_ERR_UNSUPPORTED, "schedule %d: automatic, one pass or chained", a.schedule);
    return check_cu_host(a.cu_seqlens_host, a.num_seqs, T);
}

// Tokens of the longest sequence as far as the host knows it.
template <typename A> int64_t longest_sequence(const A &a) {
    if (!a.cu_seqlens) return a.total_tokens / a.num_seqs;
    if (!a.cu_seqlens_host) return a.total_tokens;
    int64_t longest = 0;
    for (int64_t n = 0; n < a.num_seqs; ++n)
        longest = std::max<int64_t>(longest, (int64_t)a.cu_seqlens_host[n + 1] - a.cu_seqlens_host[n]);
    return longest;
}

// Tokens that the tiles of a chained call hold, the half-empty last ones among them.
template <typename A> double padded_tokens(const A &a, int tile) {
    const int64_t T = a.total_tokens, N = a.num_seqs;
    if (a.cu_seqlens && !a.cu_seqlens_host) return (double)T + 0.5 * tile * (double)N;
    int64_t tiles = 0;
    for (int64_t n = 0; n < N; ++n) {
        const int64_t len = a.cu_seqlens ? (int64_t)a.cu_seqlens_host[n + 1] - a.cu_seqlens_host[n] : T / N;
        tiles += (len + tile - 1) / tile;
    }
    return (double)tiles * tile;
}

// The automatic choice compares a cost of both sides (us).  One pass takes the longer of
// its longest sequence, token behind token, and of the memory's time for everything, at
// 4.8 TB/s.  Chained takes 8 for its second launch and its workspace, and the memory's
// time at 4.7 to 5.2 TB/s, of which a row that only pads a last tile costs half.  Measured,
// one pass / chained, 4096 channels of bf16: 1 sequence of 224 tokens 10.5/14.0, 448
// 16.6/14.5, 4096 137/35; 8 of 1000 47/52; 64 of 1000, log-decays 326/309, pre-activations
// with complement 320/375; backward, 8 of 2000 142/137.  Called one after another neither
// side takes less than its fixed part, about 10 and 14, so the choice is early for one
// sequence of a few hundred tokens: fp32, 224 x 512, takes chained, 14.4, and one pass would
// take 10.7.  Lengths that only the device knows count as one sequence: chained loses up to
// a third on many short ones, one pass any factor on a long one among them.
template <typename A> bool prefer_chained(const A &a, bool backward, int tile) {
    const bool half = a.dtype == KDA_BF16, cheap = a.gate_kind == KDA_GATE_LOG && a.input_kind == KDA_INPUT_PLAIN;
    const double row = (double)a.channels * (half ? 2 : 4) * (!backward ? 3 : a.input_kind == KDA_INPUT_PLAIN ? 5 : 6);
    const double token = backward ? (half ? 0.051 : 0.072) : (half ? 0.031 : 0.042);
    const double rate = backward ? 5.0e6 : cheap ? 5.2e6 : 4.7e6;
    const double T = (double)a.total_tokens;
    const double one = std::max((double)longest_sequence(a) * token, T * row / 4.8e6);
    return 8.0 + 0.5 * (T + padded_tokens(a, tile)) * row / rate < one;
}

// The schedule of a call that has a workspace.
template <typename A> kda::ScanPlan scan_plan(const A &a, bool backward) {
    const kda::ScanPlan one{false, 0, nullptr};
    if (a.schedule == KDA_SCHEDULE_ONE_PASS || a.total_tokens < 1) return one;
    const int tile = kda::scan_tile(a.dtype, a.gate_kind, a.input_kind, backward);
    const kda::ScanPlan chained{true, a.total_tokens / tile + a.num_seqs, a.workspace};
    if (chained.tiles * channel_groups(a.channels) >= kMaxGroups) return one;
    return a.schedule == KDA_SCHEDULE_CHAINED || prefer_chained(a, backward, tile) ? chained : one;
}

size_t plan_bytes(const kda::ScanPlan &plan, int32_t C) {
    return plan.chained ? kda::scan_chain_bytes(plan.tiles, C) : 0;
}

template <typename A> size_t scan_workspace(const A *a, bool backward) {
    if (!a || a->num_seqs < 1 || a->channels < 1 || a->total_tokens < 0 || a->total_tokens > kMaxTokens) return 0;
    return plan_bytes(scan_plan(*a, backward), a->channels);
}

// The schedule of this call and the checks of its workspace.
template <typename A> kda_status resolve_plan(const A &a, bool backward, kda::ScanPlan &plan, size_t &bytes) {
    plan = kda::ScanPlan{false, 0, nullptr};
    bytes = 0;
    if (a.schedule == KDA_SCHEDULE_CHAINED && a.total_tokens > 0) {
        if (!a.workspace)
            return fail(KDA_ERR_INVALID_ARG, "the chained schedule needs a workspace (kda_gated_scan%s_workspace_size)",
                        backward ? "_backward" : "");
        if (!scan_plan(a, backward).chained) return fail(KDA_ERR_INVALID_ARG, "too many tiles for the chained schedule");
    }
    if (!a.workspace) return KDA_OK;
    plan = scan_plan(a, backward);
    bytes = plan_bytes(plan, a.channels);
    if (a.workspace_bytes < bytes)
        return fail(KDA_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", a.workspace_bytes, bytes);
    if (plan.chained && (uintptr_t)a.workspace % 16)
        return fail(KDA_ERR_INVALID_ARG, "the workspace must be 16-byte aligned");
    return KDA_OK;
}

// Written tensors (the first n_written) against each other and every other, and all of
// them against the plain buffers, of which the first b_written are written.
kda_status check_disjoint(const Rows *r, int n, int n_written, const int *same, const Buf *b, int nb, int b_written) {
    kda_status st = check_rows_written(r, n, n_written, same);
    if (st != KDA_OK) return st;
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < nb; ++j)
            if ((i < n_written || j < b_written) && overlap(r[i].p, rows_bytes(r[i]), b[j].p, b[j].bytes))
                return fail(KDA_ERR_INVALID_ARG, "%s overlaps %s", r[i].name, b[j].name);
    return check_written(b, nb, b_written);
}

kda_status scan_prefill_impl(kda_gated_scan_args a, hipStream_t stream) {
    kda_status st = check_scan(a.num_seqs, a.channels, a.dtype, a.gate_kind, a.input_kind, a.flags);
    if (st != KDA_OK) return st;
    st = check_tokens(a);
    if (st != KDA_OK) return st;
    const int64_t T = a.total_tokens, C = a.channels, N = a.num_seqs;
    if (T > 0 && (!a.x || !a.gate || !a.o)) return fail(KDA_ERR_INVALID_ARG, "x, gate and o must be non-NULL");
    size_t rows = 0;
    st = pool_rows(a.state_slots, a.num_slots, a.num_seqs, rows);
    if (st != KDA_OK) return st;
    const size_t sb = rows * C * state_esize(a.flags), es = esize(a.dtype);
    Rows r[3] = {{a.o, T, a.o_stride, C, es, "o"}, {a.x, T, a.x_stride, C, es, "x"}, {a.gate, T, a.gate_stride, C, es, "gate"}};
    for (Rows &x : r) {
        st = check_rows(x);
        if (st != KDA_OK) return st;
    }
    st = check_strides(r, 3);
    if (st != KDA_OK) return st;
    a.o_stride = r[0].stride; a.x_stride = r[1].stride; a.gate_stride = r[2].stride;
    if ((uintptr_t)a.state_in % 16 || (uintptr_t)a.state_out % 16)
        return fail(KDA_ERR_INVALID_ARG, "the states must be 16-byte aligned");
    const bool in_place = a.state_out && (const void *)a.state_out == a.state_in;
    kda::ScanPlan plan;
    size_t wb;
    st = resolve_plan(a, false, plan, wb);
    if (st != KDA_OK) return st;
    const Buf bufs[] = {{a.state_out, sb, "state_out"}, {a.workspace, wb, "workspace"},
                        {a.state_in, in_place ? 0 : sb, "state_in"},
                        {a.cu_seqlens, a.cu_seqlens ? (size_t)(N + 1) * 4 : 0, "cu_seqlens"},
                        {a.state_slots, a.state_slots ? (size_t)N * 4 : 0, "state_slots"}};
    const int same[1] = {-1};
    st = check_disjoint(r, 3, 1, same, bufs, 5, 2);
    if (st != KDA_OK) return st;
    if (T == 0 && !a.state_out) return KDA_OK;
    const hipError_t e = kda::launch_gated_scan(&a, plan, stream);
    if (e != hipSuccess) return hip_fail(e, "gated_scan_prefill launch");
    return KDA_OK;
}

kda_status scan_decode_impl(kda_gated_scan_decode_args a, hipStream_t stream) {
    kda_status st = check_scan(a.num_seqs, a.channels, a.dtype, a.gate_kind, a.input_kind, a.flags);
    if (st != KDA_OK) return st;
    if (!a.x || !a.gate || !a.state || !a.o) return fail(KDA_ERR_INVALID_ARG, "x, gate, state and o must be non-NULL");
    const int64_t C = a.channels, N = a.num_seqs;
    size_t rows = 0;
    st = pool_rows(a.state_slots, a.num_slots, a.num_seqs, rows);
    if (st != KDA_OK) return st;
    const size_t es = esize(a.dtype);
    Rows r[3] = {{a.o, N, a.o_stride, C, es, "o"}, {a.x, N, a.x_stride, C, es, "x"}, {a.gate, N, a.gate_stride, C, es, "gate"}};
    for (Rows &x : r) {
        st = check_rows(x);
        if (st != KDA_OK) return st;
    }
    a.o_stride = r[0].stride; a.x_stride = r[1].stride; a.gate_stride = r[2].stride;
    if ((uintptr_t)a.state % 16) return fail(KDA_ERR_INVALID_ARG, "the states must be 16-byte aligned");
    const Buf bufs[] = {{a.state, rows * C * state_esize(a.flags), "state"},
                        {a.state_slots, a.state_slots ? (size_t)N * 4 : 0, "state_slots"}};
    const int same[1] = {-1};
    st = check_disjoint(r, 3, 1, same, bufs, 2, 1);
    if (st != KDA_OK) return st;
    const hipError_t e = kda::launch_gated_scan_decode(&a, stream);
    if (e != hipSuccess) return hip_fail(e, "gated_scan_decode launch");
    return KDA_OK;
}

kda_status scan_backward_impl(kda_gated_scan_backward_args a, hipStream_t stream) {
    kda_status st = check_scan(a.num_seqs, a.channels, a.dtype, a.gate_kind, a.input_kind, a.flags);
    if (st != KDA_OK) return st;
    st = check_tokens(a);
    if (st != KDA_OK) return st;
    const int64_t T = a.total_tokens, C = a.channels, N = a.num_seqs;
    if (a.input_kind == KDA_INPUT_PLAIN && a.x) return fail(KDA_ERR_INVALID_ARG, "KDA_INPUT_PLAIN takes no x");
    if (T > 0 && (!a.d_o || !a.gate || !a.o || !a.dx || !a.dgate || (a.input_kind != KDA_INPUT_PLAIN && !a.x)))
        return fail(KDA_ERR_INVALID_ARG, "d_o, gate, o, x, dx and dgate must be non-NULL");
    const size_t es = esize(a.dtype), sb = (size_t)N * C * state_esize(a.flags), gb = (size_t)N * C * 4;
    Rows r[6] = {{a.dx, T, a.dx_stride, C, es, "dx"}, {a.dgate, T, a.dgate_stride, C, es, "dgate"},
                 {a.d_o, T, a.d_o_stride, C, es, "d_o"}, {a.gate, T, a.gate_stride, C, es, "gate"},
                 {a.o, T, a.o_stride, C, es, "o"}, {a.x, T, a.x ? a.x_stride : 0, C, es, "x"}};
    for (Rows &x : r) {
        st = check_rows(x);
        if (st != KDA_OK) return st;
    }
    st = check_strides(r, 6);
    if (st != KDA_OK) return st;
    a.dx_stride = r[0].stride; a.dgate_stride = r[1].stride; a.d_o_stride = r[2].stride;
    a.gate_stride = r[3].stride; a.o_stride = r[4].stride; a.x_stride = r[5].stride;
    if ((uintptr_t)a.state_in % 16 || (uintptr_t)a.dstate_out % 16 || (uintptr_t)a.dstate_in % 16)
        return fail(KDA_ERR_INVALID_ARG, "the states must be 16-byte aligned");
    kda::ScanPlan plan;
    size_t wb;
    st = resolve_plan(a, true, plan, wb);
    if (st != KDA_OK) return st;
    const Buf bufs[] = {{a.dstate_in, gb, "dstate_in"}, {a.workspace, wb, "workspace"}, {a.state_in, sb, "state_in"},
                        {a.dstate_out, a.dstate_out == a.dstate_in ? 0 : gb, "dstate_out"},
                        {a.cu_seqlens, a.cu_seqlens ? (size_t)(N + 1) * 4 : 0, "cu_seqlens"}};
    const int same[2] = {-1, -1};
    st = check_disjoint(r, 6, 2, same, bufs, 5, 2);
    if (st != KDA_OK) return st;
    if (T == 0 && !a.dstate_in) return KDA_OK;
    const hipError_t e = kda::launch_gated_scan_backward(&a, plan, stream);
    if (e != hipSuccess) return hip_fail(e, "gated_scan_backward launch");
    return KDA_OK;
}

kda_status check_rms(int64_t T, int32_t C, kda_dtype dt, float eps) {
    if (T < 0) return fail(KDA_ERR_INVALID_ARG, "total_tokens < 0");
    if (T > ((int64_t)1 << 31) - 64) return fail(KDA_ERR_INVALID_ARG, "total_tokens too large");
    if (C < 1 || C % 8 || C > KDA_ADD_NORM_MAX_CHANNELS)
        return fail(KDA_ERR_UNSUPPORTED, "channels = %d: a multiple of 8 up to %d", C, KDA_ADD_NORM_MAX_CHANNELS);
    if (dt != KDA_F32 && dt != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    if (!std::isfinite(eps) || !(eps > 0.f)) return fail(KDA_ERR_INVALID_ARG, "eps must be finite and > 0");
    return KDA_OK;
}

kda_status add_norm_impl(kda_add_norm_args a, hipStream_t stream) {
    kda_status st = check_rms(a.total_tokens, a.channels, a.dtype, a.eps);
    if (st != KDA_OK) return st;
    const int64_t T = a.total_tokens, C = a.channels;
    if (a.quant != KDA_QUANT_NONE && a.quant != KDA_QUANT_TOKEN && a.quant != KDA_QUANT_GROUP)
        return fail(KDA_ERR_INVALID_ARG, "quant %d: use a KDA_QUANT_* value", (int)a.quant);
    if (a.quant == KDA_QUANT_GROUP && C % 128)
        return fail(KDA_ERR_UNSUPPORTED, "KDA_QUANT_GROUP needs channels in multiples of 128, got %d", a.channels);
    if (T == 0) return KDA_OK;  // empty tensors may be NULL
    if (!a.x || !a.y) return fail(KDA_ERR_INVALID_ARG, "x and y must be non-NULL");
    if ((a.quant == KDA_QUANT_NONE) != !a.scale)
        return fail(KDA_ERR_INVALID_ARG, "scale goes with an 8-bit y, and only with it");
    const size_t es = esize(a.dtype), ys = a.quant == KDA_QUANT_NONE ? es : 1;
    Rows r[4] = {{a.residual_out, T, a.residual_out ? a.residual_out_stride : 0, C, es, "residual_out"},
                 {a.y, T, a.y_stride, C, ys, "y"}, {a.x, T, a.x_stride, C, es, "x"},
                 {a.residual, T, a.residual ? a.residual_stride : 0, C, es, "residual"}};
    for (Rows &x : r) {
        st = check_rows(x, &x == r + 1 && ys == 1 ? 8 : 16);
        if (st != KDA_OK) return st;
    }
    a.residual_out_stride = r[0].stride; a.y_stride = r[1].stride; a.x_stride = r[2].stride; a.residual_stride = r[3].stride;
    if ((uintptr_t)a.weight % 16) return fail(KDA_ERR_INVALID_ARG, "the weight must be 16-byte aligned");
    if ((uintptr_t)a.scale % 4) return fail(KDA_ERR_INVALID_ARG, "the scales must be 4-byte aligned");
    const Buf bufs[] = {{a.scale, a.quant == KDA_QUANT_TOKEN ? (size_t)T * 4 : (size_t)T * (C / 128) * 4, "scale"},
                        {a.weight, (size_t)C * 4, "weight"}};
    // residual_out may be x or residual: take the one that it is out of the comparison
    Rows q[4] = {r[0], r[1], r[2], r[3]};
    int n = 2;
    for (int i = 2; i < 4; ++i)
        if (r[i].p && !(r[i].p == r[0].p && r[i].stride == r[0].stride)) q[n++] = r[i];
    const int same[2] = {-1, -1};
    st = check_disjoint(q, n, 2, same, bufs, 2, 1);
    if (st != KDA_OK) return st;
    const hipError_t e = kda::launch_add_norm(&a, stream);
    if (e != hipSuccess) return hip_fail(e, "add_norm launch");
    return KDA_OK;
}

kda_status add_norm_backward_impl(kda_add_norm_backward_args a, hipStream_t stream) {
    kda_status st = check_rms(a.total_tokens, a.channels, a.dtype, a.eps);
    if (st != KDA_OK) return st;
    const int64_t T = a.total_tokens, C = a.channels;
    if (T == 0 && !a.dweight) return KDA_OK;  // empty tensors may be NULL
    if (T > 0 && (!a.dy || !a.s || !a.dx)) return fail(KDA_ERR_INVALID_ARG, "dy, s and dx must be non-NULL");
    const size_t es = esize(a.dtype);
    Rows r[4] = {{a.dx, T, a.dx_stride, C, es, "dx"}, {a.dy, T, a.dy_stride, C, es, "dy"}, {a.s, T, a.s_stride, C, es, "s"},
                 {a.dresidual, T, a.dresidual ? a.dresidual_stride : 0, C, es, "dresidual"}};
    for (Rows &x : r) {
        st = check_rows(x);
        if (st != KDA_OK) return st;
    }
    a.dx_stride = r[0].stride; a.dy_stride = r[1].stride; a.s_stride = r[2].stride; a.dresidual_stride = r[3].stride;
    if ((uintptr_t)a.weight % 16 || (uintptr_t)a.dweight % 16)
        return fail(KDA_ERR_INVALID_ARG, "weight and dweight must be 16-byte aligned");
    const size_t wb = a.dweight ? kda::add_norm_backward_workspace_bytes(T, a.channels) : 0;
    if (wb && (!a.workspace || a.workspace_bytes < wb))
        return fail(KDA_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", a.workspace ? a.workspace_bytes : 0, wb);
    if (wb && (uintptr_t)a.workspace % 16) return fail(KDA_ERR_INVALID_ARG, "the workspace must be 16-byte aligned");
    const Buf bufs[] = {{a.dweight, (size_t)C * 4, "dweight"}, {a.workspace, wb, "workspace"}, {a.weight, (size_t)C * 4, "weight"}};
    Rows q[4] = {r[0]};
    int n = 1;
    for (int i = 1; i < 4; ++i)
        if (r[i].p && !(r[i].p == r[0].p && r[i].stride == r[0].stride)) q[n++] = r[i];
    const int same[1] = {-1};
    st = check_disjoint(q, n, 1, same, bufs, 3, 2);
    if (st != KDA_OK) return st;
    const hipError_t e = kda::launch_add_norm_backward(&a, stream);
    if (e != hipSuccess) return hip_fail(e, "add_norm_backward launch");
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_gated_scan_prefill(const kda_gated_scan_args *a, hipStream_t stream) {
    clear_error();
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    return scan_prefill_impl(*a, stream);
}

size_t kda_gated_scan_workspace_size(const kda_gated_scan_args *a) { return scan_workspace(a, false); }

kda_status kda_gated_scan_decode(const kda_gated_scan_decode_args *a, hipStream_t stream) {
    clear_error();
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    return scan_decode_impl(*a, stream);
}

kda_status kda_gated_scan_backward(const kda_gated_scan_backward_args *a, hipStream_t stream) {
    clear_error();
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    return scan_backward_impl(*a, stream);
}

size_t kda_gated_scan_backward_workspace_size(const kda_gated_scan_backward_args *a) { return scan_workspace(a, true); }

kda_status kda_add_norm(const kda_add_norm_args *a, hipStream_t stream) {
    clear_error();
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    return add_norm_impl(*a, stream);
}

kda_status kda_add_norm_backward(const kda_add_norm_backward_args *a, hipStream_t stream) {
    clear_error();
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    return add_norm_backward_impl(*a, stream);
}

size_t kda_add_norm_backward_workspace_size(const kda_add_norm_backward_args *a) {
    if (!a || !a->dweight || a->total_tokens < 1 || a->total_tokens > ((int64_t)1 << 31) - 64 || a->channels < 1 ||
        a->channels > KDA_ADD_NORM_MAX_CHANNELS)
        return 0;
    return kda::add_norm_backward_workspace_bytes(a->total_tokens, a->channels);
}

}  // extern "C"
