// kda_linattn_api.hip -- the extern "C" entry points of the linear attention and
// the per-head norms (declared in kda.h).
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

// (Sequence, head) pairs of a grid, which holds a multiple of eight key heads.
int64_t grid_pairs(int64_t N, int32_t H, int32_t Hk) { return (N * Hk + 7) / 8 * 8 * (H / Hk); }

// Pairs of the two-pass schedule: its scan takes 16,384 threads for each, and a launch
// holds fewer than 2^32.
constexpr int64_t kMaxSegmentPairs = (int64_t)1 << 18;

kda_status check_linattn(int32_t N, int32_t H, int32_t Hk, int32_t dk, int32_t dv, kda_dtype dt, uint32_t flags,
                         float scale) {
    if (N < 1) return fail(KDA_ERR_INVALID_ARG, "num_seqs = %d, must be >= 1", N);
    if (H < 1) return fail(KDA_ERR_INVALID_ARG, "num_heads = %d, must be >= 1", H);
    if (Hk < 1 || H % Hk)
        return fail(KDA_ERR_INVALID_ARG, "num_k_heads = %d, must divide num_heads = %d", Hk, H);
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128))
        return fail(KDA_ERR_UNSUPPORTED, "head dims %d x %d: 64 and 128 are supported", dk, dv);
    if (dt != KDA_F32 && dt != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    if (flags & ~(uint32_t)(KDA_F_STATE_BF16 | KDA_F_DECAY_PER_HEAD))
        return fail(KDA_ERR_UNSUPPORTED, "unsupported flags 0x%x", flags);
    if (!std::isfinite(scale) || scale < 0.f)
        return fail(KDA_ERR_INVALID_ARG, "scale must be finite and >= 0 (0 = default)");
    // a launch holds fewer than 2^32 threads, up to 1024 of them for each pair
    if (grid_pairs(N, H, Hk) >= (int64_t)1 << 22)
        return fail(KDA_ERR_INVALID_ARG, "num_seqs * num_heads too large");
    return KDA_OK;
}

// Tokens of the longest sequence; `unknown` when the lengths are only on the device.
int64_t longest_sequence(const kda_linattn_prefill_args &a, int64_t unknown) {
    if (!a.cu_seqlens) return a.total_tokens / a.num_seqs;
    if (!a.cu_seqlens_host) return unknown;
    int64_t longest = 0;
    for (int64_t n = 0; n < a.num_seqs; ++n)
        longest = std::max<int64_t>(longest, (int64_t)a.cu_seqlens_host[n + 1] - a.cu_seqlens_host[n]);
    return longest;
}

// Segments of the two-pass schedule: whole chunks of 64 tokens, one workgroup for each
// of the 256 compute units (bf16: whole states; fp32: 64 columns).  Two fit one unit,
// except of 128-column states in bf16, and are taken where a segment keeps 256 tokens
// (fp32, 1 sequence of 8192 tokens x 16 heads 220 -> 195 us, bf16 x 64 columns, 2
// sequences of 13,438 tokens x 15 heads 80 -> 76; shorter ones cost more than they fill:
// fp32 1 x 32,768 x 1 77 -> 86, bf16 36 of 31,407 x 2 38 -> 44).
kda::LinattnPlan segment_plan(const kda_linattn_prefill_args &a) {
    const int64_t T = a.total_tokens, N = a.num_seqs, H = a.num_heads;
    const int64_t work = (T + 63) / 64 * H;  // chunks of all heads
    int64_t groups = a.dtype == KDA_F32 && a.head_dim_v > 64 ? 256 : 512;
    if ((a.dtype == KDA_BF16 && a.head_dim_v > 64) || work < 4 * groups) groups /= 2;
    kda::LinattnPlan plan;
    const int64_t chunks = (work + groups - 1) / groups;  // in each
    plan.tokens = (int)std::min<int64_t>(std::max<int64_t>(chunks, 1), (int64_t)1 << 24) * 64;
    plan.segments = T / plan.tokens + N;
    plan.bytes = ((size_t)(plan.segments + 1) * a.head_dim_k * a.head_dim_v + (size_t)plan.segments) * H * 4;
    plan.longest = (longest_sequence(a, T) + plan.tokens - 1) / plan.tokens;
    return plan;
}

// The automatic choice compares a cost of both sides (us; dk = dv = 128; L tokens and
// `pairs` segments x heads in two passes).  In one pass the longest sequence's chunks
// follow one another; segments run side by side but read the keys and values twice, in
// two more launches:
//   bf16  one pass  5 + 1.33 longest / 64 (32-column tiles; 2.4 for whole states)
//         two       10.5 + 0.045 pairs + 3.9 L / 64, and 3.5 for a launch that joins
//   fp32  one pass  4 + 6.2 longest / 64 (8.1 with 64 columns)
//         two        7 + 12 L / 64 (20 with two workgroups to a compute unit)
// The constants were fitted to calls on cached inputs.  Both sides on distinct tensors
// that are not cached, 1 sequence of 1024, 2048, 4096 and 32,768 tokens, bf16: 8 heads
// 28/22, 51/33, 99/40, 750/112; 64 heads 33/39, 59/58, 120/105, 939/632; fp32, 8 heads
// 105/26, 209/40, 412/66, 3311/371.  There, over 1, 4 and 16 sequences x 1, 8, 16, 64 and 128
// heads x 512 to 32,768 tokens, the choice is within 10 % of the better side but for bf16
// 1 x 2048 x 128 (one pass 97, two 88), 16 x 1024 x 1 (28, 40), and 16 sequences x 8 heads from
// 4096 tokens on (191, 244; of 16,384 705, 916), where it takes the other one.
bool prefer_segments(const kda_linattn_prefill_args &a, const kda::LinattnPlan &plan) {
    if (plan.bytes > KDA_PREFILL_WORKSPACE_CAP) return false;
    const int64_t T = a.total_tokens, N = a.num_seqs, H = a.num_heads, L = plan.tokens;
    const int64_t longest = longest_sequence(a, (T + N - 1) / N);  // the average where lengths are not known
    const int64_t halves = N * H * (a.head_dim_v / 64);
    if (a.dtype == KDA_F32)
        return (halves > 128 ? 81 : 62) * longest > (L < 256 || T / L * H * (a.head_dim_v / 64) <= 256 ? 120 : 200) * L + 2000;
    const bool wide = halves >= 256;
    return (wide ? 240 : 133) * longest > 390 * L + 290 * (T / L * H) + (plan.longest > kda::kJoinSegments ? 57600 : 35200);
}

// Whether a call with a workspace runs two passes, and how (tokens 0: one pass).
kda::LinattnPlan linattn_plan(const kda_linattn_prefill_args &a) {
    const kda::LinattnPlan none{0, 0, 0, 0};
    if (a.schedule == KDA_SCHEDULE_ONE_PASS || a.total_tokens < 1) return none;
    if ((int64_t)a.num_seqs * a.num_heads >= kMaxSegmentPairs) return none;
    const kda::LinattnPlan plan = segment_plan(a);
    return a.schedule == KDA_SCHEDULE_TWO_PASS || prefer_segments(a, plan) ? plan : none;
}

kda_status linattn_prefill_impl(kda_linattn_prefill_args a, hipStream_t stream) {
    kda_status st = check_linattn(a.num_seqs, a.num_heads, a.num_k_heads, a.head_dim_k, a.head_dim_v, a.dtype,
                                  a.flags, a.scale);
    if (st != KDA_OK) return st;
    const int64_t T = a.total_tokens, H = a.num_heads, N = a.num_seqs;
    if (T < 0) return fail(KDA_ERR_INVALID_ARG, "total_tokens < 0");
    // token positions inside a sequence are 32-bit in the kernels (cu_seqlens is int32)
    if (T > ((int64_t)1 << 31) - 64) return fail(KDA_ERR_INVALID_ARG, "total_tokens too large");
    if (T > 0 && (!a.q || !a.k || !a.v || !a.o))
        return fail(KDA_ERR_INVALID_ARG, "q, k, v and o must be non-NULL");
    if (T > 0 && !a.log_decay) return fail(KDA_ERR_INVALID_ARG, "log_decay is NULL");
    if (a.cu_seqlens_host && !a.cu_seqlens)
        return fail(KDA_ERR_INVALID_ARG, "cu_seqlens_host needs cu_seqlens");
    if (!a.cu_seqlens && T % N)
        return fail(KDA_ERR_INVALID_ARG, "cu_seqlens NULL needs total_tokens %% num_seqs == 0");
    st = check_cu_host(a.cu_seqlens_host, a.num_seqs, T);
    if (st != KDA_OK) return st;
    const size_t es = esize(a.dtype);
    size_t rows = 0;
    st = pool_rows(a.state_slots, a.num_slots, a.num_seqs, rows);
    if (st != KDA_OK) return st;
    const size_t sb = rows * H * a.head_dim_k * a.head_dim_v * state_esize(a.flags);
    const int64_t wk = (int64_t)a.num_k_heads * a.head_dim_k, wv = H * a.head_dim_v;
    Rows r[4] = {{a.o, T, wv, wv, es, "o"}, {a.q, T, a.q_stride, wk, es, "q"}, {a.k, T, a.k_stride, wk, es, "k"},
                 {a.v, T, a.v_stride, wv, es, "v"}};
    for (Rows &x : r) {
        st = check_rows(x);
        if (st != KDA_OK) return st;
    }
    a.q_stride = r[1].stride; a.k_stride = r[2].stride; a.v_stride = r[3].stride;
    if ((uintptr_t)a.state_in % 16 || (uintptr_t)a.state_out % 16)
        return fail(KDA_ERR_INVALID_ARG, "the states must be 16-byte aligned");
    const bool in_place = a.state_out && (const void *)a.state_out == a.state_in;
    if (a.state_out && !in_place && overlap(a.state_out, sb, a.state_in, sb))
        return fail(KDA_ERR_INVALID_ARG, "state_out partially overlaps state_in");
    const size_t gb = (size_t)H * ((a.flags & KDA_F_DECAY_PER_HEAD) ? 1 : T) * 4;
    if (a.schedule != KDA_SCHEDULE_AUTO && a.schedule != KDA_SCHEDULE_ONE_PASS && a.schedule != KDA_SCHEDULE_TWO_PASS)
        return fail(KDA_ERR_UNSUPPORTED, "schedule %d: automatic, one pass or two passes", a.schedule);
    if (a.schedule == KDA_SCHEDULE_TWO_PASS && T > 0) {  // (no tokens, no passes)
        if (!a.workspace)
            return fail(KDA_ERR_INVALID_ARG, "the two-pass schedule needs a workspace (kda_linattn_workspace_size)");
        if (N * H >= kMaxSegmentPairs) return fail(KDA_ERR_INVALID_ARG, "too many pairs for the two-pass schedule");
    }
    const kda::LinattnPlan plan = a.workspace ? linattn_plan(a) : kda::LinattnPlan{0, 0, 0, 0};
    if (a.workspace && a.workspace_bytes < plan.bytes)
        return fail(KDA_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", a.workspace_bytes, plan.bytes);
    if (plan.tokens && (uintptr_t)a.workspace % 16)
        return fail(KDA_ERR_INVALID_ARG, "the workspace must be 16-byte aligned");
    const Buf bufs[] = {{a.o, rows_bytes(r[0]), "o"}, {a.state_out, sb, "state_out"},
                        {a.workspace, plan.bytes, "workspace"},
                        {a.q, rows_bytes(r[1]), "q"}, {a.k, rows_bytes(r[2]), "k"}, {a.v, rows_bytes(r[3]), "v"},
                        {a.log_decay, gb, "log_decay"}, {a.state_in, in_place ? 0 : sb, "state_in"},
                        {a.cu_seqlens, a.cu_seqlens ? (size_t)(N + 1) * 4 : 0, "cu_seqlens"},
                        {a.state_slots, a.state_slots ? (size_t)N * 4 : 0, "state_slots"}};
    st = check_written(bufs, 10, 3);
    if (st != KDA_OK) return st;
    if (T == 0 && !a.state_out) return KDA_OK;
    if (a.scale == 0.f) a.scale = 1.0f / std::sqrt((float)a.head_dim_k);
    hipError_t e = a.dtype == KDA_BF16 ? kda::launch_linattn_chunks(&a, plan, stream) : kda::launch_linattn_f32(&a, plan, stream);
    if (e != hipSuccess) return hip_fail(e, "linattn_prefill launch");
    return KDA_OK;
}

kda_status linattn_decode_impl(kda_linattn_decode_args a, hipStream_t stream) {
    kda_status st = check_linattn(a.num_seqs, a.num_heads, a.num_k_heads, a.head_dim_k, a.head_dim_v, a.dtype,
                                  a.flags, a.scale);
    if (st != KDA_OK) return st;
    if (!a.q || !a.k || !a.v || !a.log_decay || !a.state || !a.o)
        return fail(KDA_ERR_INVALID_ARG, "q, k, v, log_decay, state and o must be non-NULL");
    const size_t es = esize(a.dtype);
    const int64_t N = a.num_seqs, H = a.num_heads;
    size_t rows = 0;
    st = pool_rows(a.state_slots, a.num_slots, a.num_seqs, rows);
    if (st != KDA_OK) return st;
    const size_t sb = rows * H * a.head_dim_k * a.head_dim_v * state_esize(a.flags);
    const int64_t wk = (int64_t)a.num_k_heads * a.head_dim_k, wv = H * a.head_dim_v;
    Rows r[4] = {{a.o, N, wv, wv, es, "o"}, {a.q, N, a.q_stride, wk, es, "q"}, {a.k, N, a.k_stride, wk, es, "k"},
                 {a.v, N, a.v_stride, wv, es, "v"}};
    for (Rows &x : r) {
        st = check_rows(x);
        if (st != KDA_OK) return st;
    }
    a.q_stride = r[1].stride; a.k_stride = r[2].stride; a.v_stride = r[3].stride;
    if ((uintptr_t)a.state % 16) return fail(KDA_ERR_INVALID_ARG, "the states must be 16-byte aligned");
    const Buf bufs[] = {{a.o, rows_bytes(r[0]), "o"}, {a.state, sb, "state"},
                        {a.q, rows_bytes(r[1]), "q"}, {a.k, rows_bytes(r[2]), "k"}, {a.v, rows_bytes(r[3]), "v"},
                        {a.log_decay, (size_t)H * ((a.flags & KDA_F_DECAY_PER_HEAD) ? 1 : N) * 4, "log_decay"},
                        {a.state_slots, a.state_slots ? (size_t)N * 4 : 0, "state_slots"}};
    st = check_written(bufs, 7, 2);
    if (st != KDA_OK) return st;
    if (a.scale == 0.f) a.scale = 1.0f / std::sqrt((float)a.head_dim_k);
    hipError_t e = kda::launch_linattn_decode(&a, stream);
    if (e != hipSuccess) return hip_fail(e, "linattn_decode launch");
    return KDA_OK;
}

// Checks shared by the two norms.
kda_status check_norm(int64_t T, int32_t D, kda_dtype dt, float eps) {
    if (T < 0) return fail(KDA_ERR_INVALID_ARG, "total_tokens < 0");
    if (T > ((int64_t)1 << 31) - 64) return fail(KDA_ERR_INVALID_ARG, "total_tokens too large");
    if (D != 64 && D != 128) return fail(KDA_ERR_UNSUPPORTED, "head_dim %d: 64 and 128 are supported", D);
    if (dt != KDA_F32 && dt != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    if (!std::isfinite(eps) || !(eps > 0.f)) return fail(KDA_ERR_INVALID_ARG, "eps must be finite and > 0");
    return KDA_OK;
}

kda_status qk_norm_rope_impl(kda_qk_norm_rope_args a, hipStream_t stream) {
    kda_status st = check_norm(a.total_tokens, a.head_dim, a.dtype, a.eps);
    if (st != KDA_OK) return st;
    const int64_t T = a.total_tokens;
    const int32_t D = a.head_dim, R = a.rotary_dim;
    if (a.num_q_heads < 1 || a.num_q_heads > 1 << 16)
        return fail(KDA_ERR_INVALID_ARG, "num_q_heads = %d, must be in 1..65536", a.num_q_heads);
    if (a.num_k_heads < 0 || a.num_k_heads > 1 << 16)
        return fail(KDA_ERR_INVALID_ARG, "num_k_heads = %d, must be in 0..65536", a.num_k_heads);
    if (a.norm != KDA_NORM_NONE && a.norm != KDA_NORM_RMS && a.norm != KDA_NORM_L2)
        return fail(KDA_ERR_INVALID_ARG, "norm %d: use a KDA_NORM_* value", (int)a.norm);
    if (a.flags & ~(uint32_t)KDA_F_ROPE_INTERLEAVED)
        return fail(KDA_ERR_UNSUPPORTED, "unsupported flags 0x%x", a.flags);
    if (R < 0 || R > D || R % 16)
        return fail(KDA_ERR_UNSUPPORTED, "rotary_dim %d: a multiple of 16 up to head_dim = %d", R, D);
    if (a.norm != KDA_NORM_RMS && (a.q_weight || a.k_weight))
        return fail(KDA_ERR_INVALID_ARG, "weights need KDA_NORM_RMS");
    if (T == 0) return KDA_OK;  // empty tensors may be NULL
    if ((R == 0) != !a.positions || (R == 0) != !a.inv_freq)
        return fail(KDA_ERR_INVALID_ARG, "positions and inv_freq go with rotary_dim > 0, and only with it");
    if (a.num_k_heads == 0 && (a.k || a.k_out || a.k_weight))
        return fail(KDA_ERR_INVALID_ARG, "num_k_heads = 0 takes no k, k_out or k_weight");
    if (!a.q || !a.q_out || (a.num_k_heads > 0 && (!a.k || !a.k_out)))
        return fail(KDA_ERR_INVALID_ARG, "q, q_out, k and k_out must be non-NULL");
    const size_t es = esize(a.dtype);
    const int64_t wq = (int64_t)a.num_q_heads * D, wk = (int64_t)a.num_k_heads * D;
    Rows r[4] = {{a.q_out, T, a.q_out_stride, wq, es, "q_out"}, {a.k_out, T, a.k_out_stride, wk, es, "k_out"},
                 {a.q, T, a.q_stride, wq, es, "q"}, {a.k, T, a.k_stride, wk, es, "k"}};
    for (Rows &x : r) {
        st = check_rows(x);
        if (st != KDA_OK) return st;
    }
    a.q_out_stride = r[0].stride; a.k_out_stride = r[1].stride;
    a.q_stride = r[2].stride; a.k_stride = r[3].stride;
    const int same[2] = {2, 3};
    st = check_rows_written(r, 4, 2, same);
    if (st != KDA_OK) return st;
    if ((uintptr_t)a.q_weight % 16 || (uintptr_t)a.k_weight % 16)
        return fail(KDA_ERR_INVALID_ARG, "the weights must be 16-byte aligned");
    const Buf aux[] = {{a.q_out, rows_bytes(r[0]), "q_out"}, {a.k_out, rows_bytes(r[1]), "k_out"},
                       {a.q_weight, a.q_weight ? (size_t)D * 4 : 0, "q_weight"},
                       {a.k_weight, a.k_weight ? (size_t)D * 4 : 0, "k_weight"},
                       {a.positions, a.positions ? (size_t)T * 4 : 0, "positions"},
                       {a.inv_freq, (size_t)R * 2, "inv_freq"}};
    for (int i = 0; i < 2; ++i)
        for (int j = 2; j < 6; ++j)
            if (overlap(aux[i].p, aux[i].bytes, aux[j].p, aux[j].bytes))
                return fail(KDA_ERR_INVALID_ARG, "%s overlaps %s", aux[i].name, aux[j].name);
    hipError_t e = kda::launch_qk_norm_rope(&a, stream);
    if (e != hipSuccess) return hip_fail(e, "qk_norm_rope launch");
    return KDA_OK;
}

kda_status gated_norm_impl(kda_gated_norm_args a, hipStream_t stream) {
    kda_status st = check_norm(a.total_tokens, a.head_dim, a.dtype, a.eps);
    if (st != KDA_OK) return st;
    const int64_t T = a.total_tokens;
    if (a.num_heads < 1 || a.num_heads > 1 << 16)
        return fail(KDA_ERR_INVALID_ARG, "num_heads = %d, must be in 1..65536", a.num_heads);
    if (a.flags & ~(uint32_t)(KDA_F_SILU | KDA_F_WEIGHT_PER_HEAD))
        return fail(KDA_ERR_UNSUPPORTED, "unsupported flags 0x%x", a.flags);
    if (T == 0) return KDA_OK;  // empty tensors may be NULL
    if ((a.flags & KDA_F_WEIGHT_PER_HEAD) && !a.weight)
        return fail(KDA_ERR_INVALID_ARG, "KDA_F_WEIGHT_PER_HEAD needs a weight");
    if ((a.flags & KDA_F_SILU) && !a.z) return fail(KDA_ERR_INVALID_ARG, "KDA_F_SILU needs z");
    if (!a.x || !a.y) return fail(KDA_ERR_INVALID_ARG, "x and y must be non-NULL");
    const size_t es = esize(a.dtype);
    const int64_t w = (int64_t)a.num_heads * a.head_dim;
    Rows r[3] = {{a.y, T, a.y_stride, w, es, "y"}, {a.x, T, a.x_stride, w, es, "x"},
                 {a.z, T, a.z ? a.z_stride : 0, w, es, "z"}};
    for (Rows &x : r) {
        st = check_rows(x);
        if (st != KDA_OK) return st;
    }
    a.y_stride = r[0].stride; a.x_stride = r[1].stride; a.z_stride = r[2].stride;
    for (int j = 1; j < 3; ++j) {  // y may be x or z, element for element
        if (r[0].p == r[j].p && r[0].stride == r[j].stride) continue;
        if (rows_overlap(r[0], r[j])) return fail(KDA_ERR_INVALID_ARG, "y overlaps %s", r[j].name);
    }
    if ((uintptr_t)a.weight % 16) return fail(KDA_ERR_INVALID_ARG, "the weight must be 16-byte aligned");
    const size_t wb = !a.weight ? 0 : (size_t)a.head_dim * ((a.flags & KDA_F_WEIGHT_PER_HEAD) ? a.num_heads : 1) * 4;
    if (overlap(a.y, rows_bytes(r[0]), a.weight, wb)) return fail(KDA_ERR_INVALID_ARG, "y overlaps weight");
    hipError_t e = kda::launch_gated_norm(&a, stream);
    if (e != hipSuccess) return hip_fail(e, "gated_norm launch");
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_linattn_prefill(const kda_linattn_prefill_args *a, hipStream_t stream) {
    clear_error();
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    return linattn_prefill_impl(*a, stream);
}

size_t kda_linattn_workspace_size(const kda_linattn_prefill_args *a) {
    if (!a || a->num_seqs < 1 || a->num_heads < 1 || a->total_tokens < 0 || a->total_tokens > ((int64_t)1 << 31) - 64 ||
        a->head_dim_k < 1 || a->head_dim_v < 1 || a->head_dim_k > 128 || a->head_dim_v > 128)
        return 0;
    return linattn_plan(*a).bytes;
}

kda_status kda_linattn_decode(const kda_linattn_decode_args *a, hipStream_t stream) {
    clear_error();
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    return linattn_decode_impl(*a, stream);
}

kda_status kda_qk_norm_rope(const kda_qk_norm_rope_args *a, hipStream_t stream) {
    clear_error();
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    return qk_norm_rope_impl(*a, stream);
}

kda_status kda_gated_norm(const kda_gated_norm_args *a, hipStream_t stream) {
    clear_error();
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    return gated_norm_impl(*a, stream);
}

}  // extern "C"
