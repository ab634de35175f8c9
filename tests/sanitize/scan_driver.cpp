// Host-only sanitizer run of the gated-scan and residual-norm entry points:
// kda_scan_api.hip's host code against stub launchers that record the call.  Good
// arguments must reach their launcher with strides and schedule resolved; bad ones must
// fail before it.
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "kda.h"
#include "kda_checks.h"
#include "kda_internal.h"

static int g_launch = 0;
static kda_gated_scan_args g_scan;
static kda_gated_scan_backward_args g_grad;
static kda_gated_scan_decode_args g_step;
static kda_add_norm_args g_norm;
static kda_add_norm_backward_args g_norm_grad;
static kda::ScanPlan g_plan;
static char g_msg[512];

namespace kda {
int scan_tile(kda_dtype dt, int, int, bool backward) { return 30 * (dt == KDA_F32 ? 1 : 2) * (backward ? 2 : 4); }
size_t scan_chain_bytes(int64_t tiles, int C) { return 256 + (size_t)((C + 127) / 128) * tiles * 1024; }
hipError_t launch_gated_scan(const kda_gated_scan_args *a, const ScanPlan &p, hipStream_t) {
    ++g_launch; g_scan = *a; g_plan = p; return hipSuccess;
}
hipError_t launch_gated_scan_backward(const kda_gated_scan_backward_args *a, const ScanPlan &p, hipStream_t) {
    ++g_launch; g_grad = *a; g_plan = p; return hipSuccess;
}
hipError_t launch_gated_scan_decode(const kda_gated_scan_decode_args *a, hipStream_t) { ++g_launch; g_step = *a; return hipSuccess; }
size_t add_norm_backward_workspace_bytes(int64_t T, int C) { return (size_t)(T < 512 ? T : 512) * C * 4; }
hipError_t launch_add_norm(const kda_add_norm_args *a, hipStream_t) { ++g_launch; g_norm = *a; return hipSuccess; }
hipError_t launch_add_norm_backward(const kda_add_norm_backward_args *a, hipStream_t) { ++g_launch; g_norm_grad = *a; return hipSuccess; }
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
static const int32_t *iaddr(int i) { return static_cast<const int32_t *>(addr(i)); }

int main() {
    const int32_t cu[3] = {0, 0, 1000};
    kda_gated_scan_args s;
    std::memset(&s, 0, sizeof(s));
    s.num_seqs = 2; s.channels = 200; s.total_tokens = 1000; s.dtype = KDA_BF16;
    s.x = addr(0); s.gate = static_cast<char *>(addr(0)) + 400; s.x_stride = s.gate_stride = 408;
    s.state_in = s.state_out = addr(2); s.o = addr(3); s.cu_seqlens = iaddr(4); s.cu_seqlens_host = cu;
    CHECK(kda_gated_scan_prefill(&s, nullptr) == KDA_OK && g_launch == 1 && !g_plan.chained);
    CHECK(g_scan.x_stride == 408 && g_scan.o_stride == 200);
    const size_t need = kda_gated_scan_workspace_size(&s);
    CHECK(need == 256 + 2 * (size_t)(1000 / 240 + 2) * 1024);
    s.workspace = addr(5); s.workspace_bytes = need;
    CHECK(kda_gated_scan_prefill(&s, nullptr) == KDA_OK && g_plan.chained && g_plan.tiles == 6 && g_plan.workspace == addr(5));
    s.workspace_bytes = need - 1;
    CHECK(kda_gated_scan_prefill(&s, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 2);
    s.schedule = KDA_SCHEDULE_ONE_PASS;
    CHECK(kda_gated_scan_prefill(&s, nullptr) == KDA_OK && !g_plan.chained);
    s.o = const_cast<void *>(s.gate);
    CHECK(kda_gated_scan_prefill(&s, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 3);
    CHECK(kda_gated_scan_prefill(nullptr, nullptr) == KDA_ERR_INVALID_ARG);

    kda_gated_scan_decode_args d;
    std::memset(&d, 0, sizeof(d));
    d.num_seqs = 5; d.channels = 64; d.dtype = KDA_F32; d.x = addr(0); d.gate = addr(1); d.state = addr(2); d.o = addr(3);
    CHECK(kda_gated_scan_decode(&d, nullptr) == KDA_OK && g_step.x_stride == 64 && g_launch == 4);
    d.state = addr(3);
    CHECK(kda_gated_scan_decode(&d, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 4);

    kda_gated_scan_backward_args b;
    std::memset(&b, 0, sizeof(b));
    b.num_seqs = 2; b.channels = 128; b.total_tokens = 1000; b.dtype = KDA_F32; b.input_kind = KDA_INPUT_NORM;
    b.d_o = addr(0); b.gate = addr(1); b.o = addr(2); b.x = addr(3); b.dx = addr(4); b.dgate = addr(5);
    b.dstate_out = static_cast<const float *>(addr(6)); b.dstate_in = static_cast<float *>(addr(6));
    b.cu_seqlens = iaddr(7); b.workspace = addr(8);
    b.workspace_bytes = kda_gated_scan_backward_workspace_size(&b);
    CHECK(b.workspace_bytes == 256 + (size_t)(1000 / 60 + 2) * 1024);
    CHECK(kda_gated_scan_backward(&b, nullptr) == KDA_OK && g_plan.chained && g_grad.dgate_stride == 128 && g_launch == 5);
    b.x = nullptr;
    CHECK(kda_gated_scan_backward(&b, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 5);

    kda_add_norm_args n;
    std::memset(&n, 0, sizeof(n));
    n.total_tokens = 9; n.channels = 72; n.dtype = KDA_BF16; n.quant = KDA_QUANT_TOKEN; n.eps = 1e-6f;
    n.x = addr(0); n.residual = addr(1); n.residual_out = addr(1); n.y = static_cast<char *>(addr(2)) + 8;
    n.scale = static_cast<float *>(addr(3));
    CHECK(kda_add_norm(&n, nullptr) == KDA_OK && g_norm.y_stride == 72 && g_launch == 6);
    n.residual_out = addr(2);
    CHECK(kda_add_norm(&n, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 6);

    kda_add_norm_backward_args g;
    std::memset(&g, 0, sizeof(g));
    g.total_tokens = 9; g.channels = 72; g.dtype = KDA_BF16; g.eps = 1e-6f; g.dy = addr(0); g.s = addr(1); g.dx = addr(0);
    g.dweight = static_cast<float *>(addr(3)); g.workspace = addr(4);
    g.workspace_bytes = kda_add_norm_backward_workspace_size(&g);
    CHECK(kda_add_norm_backward(&g, nullptr) == KDA_OK && g_norm_grad.s_stride == 72 && g_launch == 7);
    g.workspace_bytes -= 1;
    CHECK(kda_add_norm_backward(&g, nullptr) == KDA_ERR_INVALID_ARG && g_launch == 7);
    g.dweight = nullptr;
    CHECK(kda_add_norm_backward(&g, nullptr) == KDA_OK && g_launch == 8);
    if (failures) return 1;
    std::printf("scan sanitizer run ok\n");
    return 0;
}
