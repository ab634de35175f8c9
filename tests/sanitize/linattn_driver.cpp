// Host-only sanitizer run of the linear-attention and per-head norm entry points:
// kda_linattn_api.hip's host code against stub launchers that record the call.
// Good arguments must reach their launcher with strides and scale resolved; bad
// ones must fail before it.
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "kda.h"
#include "kda_checks.h"
#include "kda_internal.h"

static int g_launch = 0;
static kda_linattn_prefill_args g_prefill;
static kda::LinattnPlan g_plan;
static kda_linattn_decode_args g_decode;
static kda_qk_norm_rope_args g_qk;
static kda_gated_norm_args g_gated;
static char g_msg[512];

namespace kda {
hipError_t launch_linattn_chunks(const kda_linattn_prefill_args *a, const LinattnPlan &p, hipStream_t) {
    ++g_launch; g_prefill = *a; g_plan = p; return hipSuccess;
}
hipError_t launch_linattn_f32(const kda_linattn_prefill_args *a, const LinattnPlan &p, hipStream_t) {
    ++g_launch; g_prefill = *a; g_plan = p; return hipSuccess;
}
hipError_t launch_linattn_decode(const kda_linattn_decode_args *a, hipStream_t) { ++g_launch; g_decode = *a; return hipSuccess; }
hipError_t launch_qk_norm_rope(const kda_qk_norm_rope_args *a, hipStream_t) { ++g_launch; g_qk = *a; return hipSuccess; }
hipError_t launch_gated_norm(const kda_gated_norm_args *a, hipStream_t) { ++g_launch; g_gated = *a; return hipSuccess; }
namespace checks {
kda_status fail(kda_status st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
    va_end(ap);
    return st;
}
void clear_error() { g_msg[0] = 0; }
}  // namespace checks
}  // namespace kda

static int failures = 0;
#define CHECK(cond) do { if (!(cond)) { ++failures; std::fprintf(stderr, "FAIL line %d: %s (%s)\n", __LINE__, #cond, g_msg); } } while (0)

// fake device addresses, far apart: never dereferenced by the host code
static void *addr(int i) { return reinterpret_cast<void *>((uintptr_t)(i + 1) << 40); }

int main() {
    kda_linattn_prefill_args p;
    std::memset(&p, 0, sizeof(p));
    p.num_seqs = 2; p.num_heads = 6; p.num_k_heads = 3; p.head_dim_k = 64; p.head_dim_v = 128; p.dtype = KDA_BF16;
    p.total_tokens = 100; p.q = addr(0); p.k = addr(1); p.v = addr(2); p.log_decay = (const float *)addr(3);
    p.state_in = addr(4); p.state_out = addr(4); p.o = addr(5); p.cu_seqlens = (const int32_t *)addr(6);
    const int32_t cu[3] = {0, 0, 100};
    p.cu_seqlens_host = cu;
    CHECK(kda_linattn_prefill(&p, nullptr) == KDA_OK && g_launch == 1);
    CHECK(g_prefill.q_stride == 192 && g_prefill.v_stride == 768 && g_prefill.scale == 0.125f);
    p.total_tokens = (int64_t)1 << 31;
    CHECK(kda_linattn_prefill(&p, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 1);
    p.total_tokens = 100;
    p.q_stride = (int64_t)1 << 62;  // products of sizes stay in range
    CHECK(kda_linattn_prefill(&p, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 1);
    // q, k and v as views of one packed projection
    p.q_stride = p.k_stride = p.v_stride = 1152;
    p.k = (const char *)addr(0) + 192 * 2; p.v = (const char *)addr(0) + 384 * 2; p.scale = 2.f;
    CHECK(kda_linattn_prefill(&p, nullptr) == KDA_OK && g_launch == 2 && g_prefill.scale == 2.f);
    p.num_seqs = 1; p.cu_seqlens = p.cu_seqlens_host = nullptr; p.total_tokens = 0;
    CHECK(kda_linattn_prefill(&p, nullptr) == KDA_OK && g_launch == 3);  // passes the state through
    p.state_out = nullptr;
    CHECK(kda_linattn_prefill(&p, nullptr) == KDA_OK && g_launch == 3);

    // segments: chosen for one long sequence of few heads, never without a workspace
    p.total_tokens = 65536; p.num_heads = p.num_k_heads = 8; p.head_dim_k = p.head_dim_v = 128;
    p.k = addr(1); p.v = addr(2); p.q_stride = p.k_stride = p.v_stride = 0;
    const size_t need = kda_linattn_workspace_size(&p);
    CHECK(need > (size_t)8 * 128 * 128 * 4 * 32);
    CHECK(kda_linattn_prefill(&p, nullptr) == KDA_OK && g_launch == 4 && g_plan.tokens == 0);
    p.workspace = addr(7); p.workspace_bytes = need - 1;
    CHECK(kda_linattn_prefill(&p, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 4);
    p.workspace_bytes = need;
    CHECK(kda_linattn_prefill(&p, nullptr) == KDA_OK && g_launch == 5 && g_plan.tokens == 2048 && g_plan.segments == 33);
    p.schedule = KDA_SCHEDULE_ONE_PASS;
    CHECK(kda_linattn_workspace_size(&p) == 0);
    CHECK(kda_linattn_prefill(&p, nullptr) == KDA_OK && g_launch == 6 && g_plan.tokens == 0);
    p.schedule = KDA_SCHEDULE_TWO_PASS; p.total_tokens = 100; p.workspace = nullptr;
    CHECK(kda_linattn_prefill(&p, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 6);
    p.workspace = addr(2);
    CHECK(kda_linattn_prefill(&p, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 6);  // overlaps v
    p.schedule = KDA_SCHEDULE_FUSED;
    CHECK(kda_linattn_prefill(&p, nullptr) == KDA_ERR_UNSUPPORTED && g_launch == 6);

    kda_linattn_decode_args d;
    std::memset(&d, 0, sizeof(d));
    d.num_seqs = 5; d.num_heads = 2; d.num_k_heads = 1; d.head_dim_k = 128; d.head_dim_v = 64; d.dtype = KDA_F32;
    d.flags = KDA_F_DECAY_PER_HEAD | KDA_F_STATE_BF16;
    d.q = addr(0); d.k = addr(1); d.v = addr(2); d.log_decay = (const float *)addr(3); d.state = addr(4); d.o = addr(5);
    CHECK(kda_linattn_decode(&d, nullptr) == KDA_OK && g_launch == 7 && g_decode.k_stride == 128);
    d.state_slots = (const int32_t *)addr(6); d.num_slots = 2147483647;
    CHECK(kda_linattn_decode(&d, nullptr) == KDA_ERR_INVALID_ARG);  // a pool that size covers the other tensors
    d.num_slots = 1000;
    CHECK(kda_linattn_decode(&d, nullptr) == KDA_OK && g_launch == 8);

    kda_qk_norm_rope_args k;
    std::memset(&k, 0, sizeof(k));
    k.total_tokens = 7; k.num_q_heads = 4; k.num_k_heads = 2; k.head_dim = 64; k.rotary_dim = 32; k.dtype = KDA_BF16;
    k.norm = KDA_NORM_L2; k.eps = 1e-6f; k.positions = (const int32_t *)addr(8); k.inv_freq = (const float *)addr(9);
    // in place, inside one packed projection of 512 elements a token
    k.q = k.q_out = addr(0); k.k = k.k_out = (char *)addr(0) + 256 * 2;
    k.q_stride = k.k_stride = k.q_out_stride = k.k_out_stride = 512;
    CHECK(kda_qk_norm_rope(&k, nullptr) == KDA_OK && g_launch == 9);
    k.k = k.k_out = (char *)addr(0) + 248 * 2;  // shares eight elements with q
    CHECK(kda_qk_norm_rope(&k, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 9);
    k.k = k.k_out = (char *)addr(0) + 392 * 2;  // runs into the next token's q
    CHECK(kda_qk_norm_rope(&k, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 9);
    k.k = k.k_out = (char *)addr(0) + (384 + 512 * 3) * 2;  // rows three tokens on, beside every q
    CHECK(kda_qk_norm_rope(&k, nullptr) == KDA_OK && g_launch == 10);
    k.k = k.k_out = nullptr; k.num_k_heads = 0; k.k_stride = k.k_out_stride = 0;
    CHECK(kda_qk_norm_rope(&k, nullptr) == KDA_OK && g_launch == 11);

    kda_gated_norm_args g;
    std::memset(&g, 0, sizeof(g));
    g.total_tokens = 7; g.num_heads = 3; g.head_dim = 128; g.dtype = KDA_F32; g.eps = 1e-6f;
    g.x = g.y = addr(0);
    CHECK(kda_gated_norm(&g, nullptr) == KDA_OK && g_launch == 12 && g_gated.y_stride == 384);
    g.z = (char *)addr(0) + 16;
    CHECK(kda_gated_norm(&g, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 12);
    g.total_tokens = 0;
    CHECK(kda_gated_norm(&g, nullptr) == KDA_OK && g_launch == 12);

    if (failures) return 1;
    std::printf("linattn sanitizer run ok\n");
    return 0;
}
