// kda_add_norm.hip -- residual addition, RMS norm of whole rows and 8-bit output with
// scales, and the gradients of the norm.
//
// A row of C channels lies in the registers of WPR waves, one or two runs of eight channels
// a lane, from its read to its last write: every element is read once and written once and
// the bound is HBM.
#include <algorithm>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

namespace {

template <typename T> __device__ __forceinline__ void load8(const T *p, float (&x)[8]);
template <> __device__ __forceinline__ void load8<__bf16>(const __bf16 *p, float (&x)[8]) {
    const bf16x8 v = *reinterpret_cast<const bf16x8 *>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
}
template <> __device__ __forceinline__ void load8<float>(const float *p, float (&x)[8]) {
    const f32x4 a = reinterpret_cast<const f32x4 *>(p)[0], b = reinterpret_cast<const f32x4 *>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[i] = a[i]; x[4 + i] = b[i]; }
}
// Eight elements as they were read.
template <typename T> struct Eight;
template <> struct Eight<__bf16> {
    bf16x8 v;
    __device__ __forceinline__ void load(const __bf16 *p) { v = *reinterpret_cast<const bf16x8 *>(p); }
    __device__ __forceinline__ float get(int i) const { return (float)v[i]; }
};
template <> struct Eight<float> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const f32x4 *>(p)[0];
        b = reinterpret_cast<const f32x4 *>(p)[1];
    }
    __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i] : b[i - 4]; }
};
__device__ __forceinline__ void store8(__bf16 *p, const float (&x)[8]) {
    *reinterpret_cast<bf16x8 *>(p) = pack8(f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]});
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    reinterpret_cast<f32x4 *>(p)[0] = f32x4{x[0], x[1], x[2], x[3]};
    reinterpret_cast<f32x4 *>(p)[1] = f32x4{x[4], x[5], x[6], x[7]};
}

// Largest over the 16 lanes of a DPP row, in each of them; then over the wave.
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
    x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xb1, 0xf, 0xf, true));   // quad_perm [1,0,3,2]
    x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4e, 0xf, 0xf, true));   // quad_perm [2,3,0,1]
    x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141, 0xf, 0xf, true));  // row_half_mirror
    x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x140, 0xf, 0xf, true));  // row_mirror
    return x;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = row_max(x);
    return max(max((uint32_t)__builtin_amdgcn_readlane((int)x, 0), (uint32_t)__builtin_amdgcn_readlane((int)x, 16)),
               max((uint32_t)__builtin_amdgcn_readlane((int)x, 32), (uint32_t)__builtin_amdgcn_readlane((int)x, 48)));
}

// The scale of values whose largest modulus has the bits `top` (NaN bits are above all
// others), and the factor that takes them to +-448.  A value at the border leaves 448 by
// its rounding only, and e4m3 rounds up to 464 down to 448.
__device__ __forceinline__ float quant_scale(uint32_t top, float &inverse) {
    const float m = __builtin_bit_cast(float, top);
    const float scale = top == 0 ? 1.f : top >= 0x7f800000u ? __builtin_nanf("") : fmaxf(m * (1.f / 448.f), 0x1p-126f);
    inverse = 1.f / scale;
    return scale;
}
__device__ __forceinline__ uint2 pack_e4m3(const float (&y)[8], float k) {
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * k, y[1] * k, 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * k, y[3] * k, lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4] * k, y[5] * k, 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6] * k, y[7] * k, hi, true);
    return make_uint2((unsigned)lo, (unsigned)hi);
}

struct NormParams {
    const void *x, *r;
    const float *w;
    void *s, *y;
    float *scale;
    int64_t T, xs, rs, ss, ys;
    int C;
    float eps;
};

// A workgroup takes one row (waves_of has the choice measured), eight or more stand on a
// compute unit at a time and cover each other's sums.  The largest magnitude of a scale is
// the largest of the bits, so that a NaN is above all others.  16,384 x 4096 bf16, 8-bit
// groups: 472 MB in 84 to 87 us, 5.5 TB/s; one row of 4096 2.8 us.  A grid of workgroups that
// stay was slower.
template <typename T, int QUANT, int WPR, int NC>
__global__ void __launch_bounds__(64 * WPR) add_norm_kernel(NormParams p) {
    __shared__ float part[2][WPR];
    __shared__ uint32_t tops[2][WPR];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    int buf = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, buf ^= 1) {
        const T *x = static_cast<const T *>(p.x) + t * p.xs, *r = static_cast<const T *>(p.r) + t * p.rs;
        float v[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = 8 * (lane + 64 * (wave + WPR * i));
            if (c < p.C) {
                load8<T>(x + c, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
            }
        }
        if (p.r) {
            float o[NC][8];
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = 8 * (lane + 64 * (wave + WPR * i));
                if (c < p.C) load8<T>(r + c, o[i]);
            }
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (8 * (lane + 64 * (wave + WPR * i)) < p.C) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] += o[i][j];
                }
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
        ss = wave_sum(ss);
        if (WPR > 1) {
            if (lane == 0) part[buf][wave] = ss;
            barrier_lds();
            ss = 0.f;
#pragma unroll
            for (int q = 0; q < WPR; ++q) ss += part[buf][q];
        }
        const float rs = rsqrtf(ss / (float)p.C + p.eps);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = 8 * (lane + 64 * (wave + WPR * i));
            if (c >= p.C) continue;
            if (p.s) store8(static_cast<T *>(p.s) + t * p.ss + c, v[i]);
            float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
            if (p.w) load8<float>(p.w + c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= rs * w[j];
            if (QUANT == KDA_QUANT_NONE) {
                store8(static_cast<T *>(p.y) + t * p.ys + c, v[i]);
            } else {
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = max(m, __builtin_bit_cast(uint32_t, v[i][j]) & 0x7fffffffu);
                if (QUANT == KDA_QUANT_TOKEN) {
                    top = max(top, m);
                } else {  // 16 lanes hold the 128 channels of a scale, all of them or none inside C
                    float k;
                    const float scale = quant_scale(row_max(m), k);
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.y) + t * p.ys + c) = pack_e4m3(v[i], k);
                    if (lane % 16 == 0) p.scale[t * (p.C / 128) + c / 128] = scale;
                }
            }
        }
        if (QUANT == KDA_QUANT_TOKEN) {
            top = wave_max(top);
            if (WPR > 1) {
                if (lane == 0) tops[buf][wave] = top;
                barrier_lds();
#pragma unroll
                for (int q = 0; q < WPR; ++q) top = max(top, tops[buf][q]);
            }
            float k;
            const float scale = quant_scale(top, k);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = 8 * (lane + 64 * (wave + WPR * i));
                if (c < p.C) *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.y) + t * p.ys + c) = pack_e4m3(v[i], k);
            }
            if (threadIdx.x == 0) p.scale[t] = scale;
        }
    }
}

struct GradParams {
    const void *dy, *s, *dr;
    const float *w;
    void *dx;
    float *part;  // [blocks][C], or NULL
    int64_t T, dys, ss, drs, dxs;
    int C;
    float eps;
};

__device__ __forceinline__ void weights(const float *p, int at, float (&w)[8]) {
    if (p) {
        load8<float>(p + at, w);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 1.f;
    }
}

// A workgroup of ROWS x WPR waves takes rows blockIdx x ROWS and on, a grid's rows apart,
// with the next ones on their way while it works on these, and keeps the sums of dy n of
// its channels in registers; its waves' sums meet in LDS at the end, one after another.
// 16,384 x 4096 bf16: 541 MB in 94 us, 5.75 TB/s, and 5 for weight_grad_kernel; without the
// next rows on their way 116 in all instead of 96.
template <typename T, int WPR, int NC, int ROWS>
__global__ void __launch_bounds__(64 * WPR * ROWS) add_norm_backward_kernel(GradParams p) {
    __shared__ float2 part[2][ROWS][WPR];
    __shared__ float meet[ROWS > 1 ? ROWS - 1 : 1][ROWS > 1 ? 512 * WPR * NC : 1];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64 % WPR, sub = threadIdx.x / (64 * WPR);
    const int64_t step = (int64_t)gridDim.x * ROWS;
    // (sixteen waves leave a lane 128 registers: there the weights are read again, the
    // residual's gradient when it is needed, and in fp32 no row ahead)
    constexpr bool KEEP = WPR < 16, AHEAD = KEEP || sizeof(T) == 2;
    float dw[NC][8] = {}, w[KEEP ? NC : 1][8];
    Eight<T> ns[NC], ng[NC], nr[NC];
    bool on[NC];
    int at[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = 8 * (lane + 64 * (wave + WPR * i));
        on[i] = c < p.C;
        at[i] = on[i] ? c : 0;
        if (KEEP) weights(p.w, at[i], w[KEEP ? i : 0]);
    }
    auto load = [&](int64_t t) __attribute__((always_inline)) {
        t = min(t, p.T - 1);  // (rows past the last one read it again and leave nothing)
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            ns[i].load(static_cast<const T *>(p.s) + t * p.ss + at[i]);
            ng[i].load(static_cast<const T *>(p.dy) + t * p.dys + at[i]);
            if (KEEP && p.dr) nr[i].load(static_cast<const T *>(p.dr) + t * p.drs + at[i]);
        }
    };
    int64_t t = (int64_t)blockIdx.x * ROWS + sub;
    if (AHEAD) load(t);
    // every wave of a workgroup makes the same turns: barriers stand inside
    int buf = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * ROWS; t0 < p.T; t0 += step, t += step, buf ^= 1) {
        if (!AHEAD) load(t);
        Eight<T> s[NC], g[NC], r[NC];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            s[i] = ns[i];
            g[i] = ng[i];
            if (KEEP) r[i] = nr[i];
            float a = 0.f, b = 0.f;
            if (!KEEP) weights(p.w, at[i], w[0]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = s[i].get(j);
                a = fmaf(x, x, a);
                b = fmaf(x, g[i].get(j) * w[KEEP ? i : 0][j], b);
            }
            ss += on[i] ? a : 0.f;
            dot += on[i] ? b : 0.f;
        }
        if (AHEAD) load(t + step);
        ss = wave_sum(ss);
        dot = wave_sum(dot);
        if (WPR > 1) {
            if (lane == 0) part[buf][sub][wave] = make_float2(ss, dot);
            barrier_lds();
            ss = dot = 0.f;
#pragma unroll
            for (int q = 0; q < WPR; ++q) { ss += part[buf][sub][q].x; dot += part[buf][sub][q].y; }
        }
        const float rs = rsqrtf(ss / (float)p.C + p.eps), k = dot / (float)p.C * rs * rs;
        if (t < p.T) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float d[8];
                if (!KEEP) {
                    weights(p.w, at[i], w[0]);
                    if (p.dr) r[i].load(static_cast<const T *>(p.dr) + t * p.drs + at[i]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float x = s[i].get(j), y = g[i].get(j);
                    dw[i][j] = fmaf(y, x * rs, dw[i][j]);
                    d[j] = rs * (y * w[KEEP ? i : 0][j] - k * x);
                    if (p.dr) d[j] += r[i].get(j);
                }
                if (on[i]) store8(static_cast<T *>(p.dx) + t * p.dxs + at[i], d);
            }
        }
    }
    if (p.part) {
        if (ROWS > 1 && sub > 0) {
#pragma unroll
            for (int i = 0; i < NC; ++i) store8(&meet[sub - 1][8 * (lane + 64 * (wave + WPR * i))], dw[i]);
        }
        if (ROWS > 1) __syncthreads();
        if (sub == 0) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                for (int q = 0; q < ROWS - 1; ++q) {
                    float o[8];
                    load8<float>(&meet[q][8 * (lane + 64 * (wave + WPR * i))], o);
#pragma unroll
                    for (int j = 0; j < 8; ++j) dw[i][j] += o[j];
                }
                if (on[i]) store8(p.part + (size_t)blockIdx.x * p.C + at[i], dw[i]);
            }
        }
    }
}

// dweight: 32 channels a workgroup, 8 lanes of four, 128 slices of the partial rows joined
// through LDS in order (4.8 us for 256 rows of 4096: the launch and one trip to memory).
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float *part, int rows, int C, float *dw) {
    __shared__ f32x4 sums[128][8];
    const int lane = threadIdx.x % 8, slice = threadIdx.x / 8, c = blockIdx.x * 32 + 4 * lane;
    f32x4 a = {0.f, 0.f, 0.f, 0.f};
    if (c < C)
        for (int r = slice; r < rows; r += 128) a = a + *reinterpret_cast<const f32x4 *>(part + (size_t)r * C + c);
    sums[slice][lane] = a;
    __syncthreads();
#pragma unroll
    for (int half = 64; half > 0; half /= 2) {
        if (slice < half) sums[slice][lane] = sums[slice][lane] + sums[slice + half][lane];
        __syncthreads();
    }
    if (slice == 0 && c < C) *reinterpret_cast<f32x4 *>(dw + c) = sums[0][lane];
}

// Waves a row takes: so many that a lane holds one run of eight channels, up to eight
// waves, two above.  16,384 rows of 4096 in bf16 with 8-bit groups: 84 us with eight waves
// of one run, 87 with four of two, 142 with one of eight; the gradients, which hold three
// tensors and the next row's, 96, 105 and 158; 8192 rows of 8192, gradients, 103 with eight
// waves of two runs, 107 with sixteen of one.
int waves_of(int C) { return C <= 512 ? 1 : C <= 1024 ? 2 : C <= 2048 ? 4 : C <= 8192 ? 8 : 16; }
// Of waves_of(C) waves, a lane holds one run (else two): only eight waves have both.
template <int WPR> constexpr bool one_run(int C) { return WPR < 8 || (WPR == 8 && C <= 4096); }
constexpr unsigned kMaxBlocks = 1u << 20;

template <typename T, int QUANT, int WPR> void launch_norm(const NormParams &p, hipStream_t s) {
    const unsigned blocks = (unsigned)std::min<int64_t>(p.T, kMaxBlocks);
    const dim3 grid(blocks), block(64 * WPR);
    if (one_run<WPR>(p.C)) hipLaunchKernelGGL((add_norm_kernel<T, QUANT, WPR, one_run<WPR>(1) ? 1 : 2>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((add_norm_kernel<T, QUANT, WPR, one_run<WPR>(1 << 30) ? 1 : 2>), grid, block, 0, s, p);
    trace("add_norm_kernel<waves=%d> grid=(%u) block=%d", WPR, blocks, 64 * WPR);
}
template <typename T, int QUANT> void launch_norm(const NormParams &p, hipStream_t s) {
    switch (waves_of(p.C)) {
    case 1: return launch_norm<T, QUANT, 1>(p, s);
    case 2: return launch_norm<T, QUANT, 2>(p, s);
    case 4: return launch_norm<T, QUANT, 4>(p, s);
    case 8: return launch_norm<T, QUANT, 8>(p, s);
    default: return launch_norm<T, QUANT, 16>(p, s);
    }
}
template <typename T> void launch_norm(const NormParams &p, int quant, hipStream_t s) {
    if (quant == KDA_QUANT_NONE) launch_norm<T, KDA_QUANT_NONE>(p, s);
    else if (quant == KDA_QUANT_TOKEN) launch_norm<T, KDA_QUANT_TOKEN>(p, s);
    else launch_norm<T, KDA_QUANT_GROUP>(p, s);
}

// Rows side by side in a workgroup of the gradients (four waves at least), and workgroups:
// twelve waves or one workgroup for each of the 256 compute units (more of them add to the
// partial sums of dweight: sixteen waves 104 us instead of 96).
int grad_rows(int C) { return std::max(4 / waves_of(C), 1); }
unsigned grad_blocks(int64_t T, int C) {
    const int rows = grad_rows(C), waves = rows * waves_of(C);
    return (unsigned)std::min<int64_t>((T + rows - 1) / rows, 256 * std::max(12 / waves, 1));
}

template <typename T, int WPR, int ROWS> void launch_grad(const GradParams &p, unsigned blocks, hipStream_t s) {
    const dim3 grid(blocks), block(64 * WPR * ROWS);
    if (one_run<WPR>(p.C)) hipLaunchKernelGGL((add_norm_backward_kernel<T, WPR, one_run<WPR>(1) ? 1 : 2, ROWS>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((add_norm_backward_kernel<T, WPR, one_run<WPR>(1 << 30) ? 1 : 2, ROWS>), grid, block, 0, s, p);
    trace("add_norm_backward_kernel<waves=%d, rows=%d> grid=(%u) block=%d", WPR, ROWS, blocks, 64 * WPR * ROWS);
}
template <typename T> void launch_grad(const GradParams &p, unsigned blocks, hipStream_t s) {
    switch (waves_of(p.C)) {
    case 1: return launch_grad<T, 1, 4>(p, blocks, s);
    case 2: return launch_grad<T, 2, 2>(p, blocks, s);
    case 4: return launch_grad<T, 4, 1>(p, blocks, s);
    case 8: return launch_grad<T, 8, 1>(p, blocks, s);
    default: return launch_grad<T, 16, 1>(p, blocks, s);
    }
}

}  // namespace

size_t add_norm_backward_workspace_bytes(int64_t T, int C) { return T > 0 ? (size_t)grad_blocks(T, C) * C * 4 : 0; }

hipError_t launch_add_norm(const kda_add_norm_args *a, hipStream_t s) {
    NormParams p = {};
    p.x = a->x; p.r = a->residual; p.w = a->weight; p.s = a->residual_out; p.y = a->y; p.scale = a->scale;
    p.T = a->total_tokens; p.C = a->channels; p.eps = a->eps;
    p.xs = a->x_stride; p.rs = a->residual_stride; p.ss = a->residual_out_stride; p.ys = a->y_stride;
    a->dtype == KDA_BF16 ? launch_norm<__bf16>(p, a->quant, s) : launch_norm<float>(p, a->quant, s);
    return hipGetLastError();
}

hipError_t launch_add_norm_backward(const kda_add_norm_backward_args *a, hipStream_t s) {
    GradParams p = {};
    p.dy = a->dy; p.s = a->s; p.dr = a->dresidual; p.w = a->weight; p.dx = a->dx;
    p.T = a->total_tokens; p.C = a->channels; p.eps = a->eps;
    p.dys = a->dy_stride; p.ss = a->s_stride; p.drs = a->dresidual_stride; p.dxs = a->dx_stride;
    p.part = a->dweight ? static_cast<float *>(a->workspace) : nullptr;
    const unsigned blocks = grad_blocks(p.T, p.C);
    if (p.T > 0) {
        a->dtype == KDA_BF16 ? launch_grad<__bf16>(p, blocks, s) : launch_grad<float>(p, blocks, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a->dweight) {
        hipLaunchKernelGGL(weight_grad_kernel, dim3((p.C + 31) / 32), dim3(1024), 0, s, p.part, (int)blocks, p.C, a->dweight);
        trace("weight_grad_kernel grid=(%d) block=1024", (p.C + 31) / 32);
    }
    return hipGetLastError();
}

}  // namespace kda
