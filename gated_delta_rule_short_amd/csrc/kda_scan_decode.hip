// kda_scan_decode.hip -- one token of the gated scan for each of N sequences:
// h <- a h + b x, o = h, the states updated in place.
//
// A lane owns four neighbouring channels of one sequence.  The bound is HBM (every state
// is read once and written once) or, long before it, latency: 1 x 8192 channels 3.0 us, 256 x
// 8192 with slots 7.1 us for 29 MB, 4.1 TB/s, in fp32 8.4 us for 42 MB, 5.0 TB/s.  2048
// workgroups are one round of them, and with slots each makes two trips to memory, one behind
// the other: the slot, which decides whether the sequence is there at all, then x, gate and
// state.  A channel that remembers long is stepped as h - (1 - a) h: over thousands of calls
// the rounding of a itself, the same at every step of a steady gate, would change its memory's
// length.
#include "kda_scan.h"

namespace kda {

namespace {

struct StepParams {
    const void *x, *g;
    void *state, *o;
    const int32_t *slots;
    int64_t xs, gs, os;
    unsigned items;  // sequences x C / 4: fewer than 2^27, since sequences x groups of 128 are fewer than 2^22
    int C, num_slots;
};

template <typename T> struct Four { typedef f32x4 vec; };
template <> struct Four<__bf16> { typedef bf16x4 vec; };
template <typename T> __device__ __forceinline__ f32x4 load4(const T *p) {
    const typename Four<T>::vec v = *reinterpret_cast<const typename Four<T>::vec *>(p);
    return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}
__device__ __forceinline__ void store4(__bf16 *p, f32x4 v) { *reinterpret_cast<bf16x4 *>(p) = pack4(v); }
__device__ __forceinline__ void store4(float *p, f32x4 v) { *reinterpret_cast<f32x4 *>(p) = v; }

template <typename T, typename S, int GATE, int INPUT>
__global__ void __launch_bounds__(256) scan_step_kernel(StepParams p) {
    const unsigned item = blockIdx.x * 256 + threadIdx.x, runs = p.C / 4;
    if (item >= p.items) return;
    const int n = (int)(item / runs), c = 4 * (int)(item - n * runs);
    const int slot = pool_slot(p.slots, p.num_slots, n);
    if (slot < 0) return;
    S *state = static_cast<S *>(p.state) + (size_t)slot * p.C + c;
    const f32x4 x = load4(static_cast<const T *>(p.x) + n * p.xs + c), z = load4(static_cast<const T *>(p.g) + n * p.gs + c);
    f32x4 h = load4(state);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Factors<GATE, INPUT> f(z[i]);
        const float u = f.input(x[i]), limited = __builtin_amdgcn_fmed3f(h[i], -3.4028234663852886e38f, 3.4028234663852886e38f);
        // (an infinite state stays one: infinity minus a part of itself would not)
        h[i] = f.c < 0.5f ? h[i] + fmaf(-f.c, limited, u) : fmaf(f.a, h[i], u);
    }
    store4(state, h);
    store4(static_cast<T *>(p.o) + n * p.os + c, h);
}

template <typename T, typename S, int GATE> void launch(const StepParams &p, int input, unsigned blocks, hipStream_t s) {
    if (input == KDA_INPUT_PLAIN) hipLaunchKernelGGL((scan_step_kernel<T, S, GATE, KDA_INPUT_PLAIN>), dim3(blocks), dim3(256), 0, s, p);
    else if (input == KDA_INPUT_COMPLEMENT) hipLaunchKernelGGL((scan_step_kernel<T, S, GATE, KDA_INPUT_COMPLEMENT>), dim3(blocks), dim3(256), 0, s, p);
    else hipLaunchKernelGGL((scan_step_kernel<T, S, GATE, KDA_INPUT_NORM>), dim3(blocks), dim3(256), 0, s, p);
}
template <typename T, typename S> void launch(const StepParams &p, int gate, int input, unsigned blocks, hipStream_t s) {
    gate == KDA_GATE_LOG ? launch<T, S, KDA_GATE_LOG>(p, input, blocks, s) : launch<T, S, KDA_GATE_SIGMOID>(p, input, blocks, s);
}

}  // namespace

hipError_t launch_gated_scan_decode(const kda_gated_scan_decode_args *a, hipStream_t s) {
    StepParams p = {};
    p.x = a->x; p.g = a->gate; p.state = a->state; p.o = a->o;
    p.xs = a->x_stride; p.gs = a->gate_stride; p.os = a->o_stride;
    p.slots = a->state_slots; p.num_slots = a->num_slots; p.C = a->channels;
    p.items = (unsigned)a->num_seqs * (unsigned)(a->channels / 4);
    const unsigned blocks = (p.items + 255) / 256;
    const bool half = (a->flags & KDA_F_STATE_BF16) != 0;
    if (a->dtype == KDA_BF16) half ? launch<__bf16, __bf16>(p, a->gate_kind, a->input_kind, blocks, s) : launch<__bf16, float>(p, a->gate_kind, a->input_kind, blocks, s);
    else half ? launch<float, __bf16>(p, a->gate_kind, a->input_kind, blocks, s) : launch<float, float>(p, a->gate_kind, a->input_kind, blocks, s);
    trace("scan_step_kernel grid=(%u) block=256", blocks);
    return hipGetLastError();
}

}  // namespace kda
