// kda_add_norm.hip -- residual addition, RMS norm of whole rows and 8-bit output with
// scales, and the gradients of the norm.
//
// A row of C channels lies in the registers of WPR waves, NC runs of eight channels a
// lane, from its read to its last write: every element is read once and written once and
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
            __syncthreads();
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
                __syncthreads();
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

// A workgroup takes rows blockIdx, blockIdx + gridDim, .. and keeps the sums of dy n of its
// own channels in registers.
template <typename T, int WPR, int NC>
__global__ void __launch_bounds__(64 * WPR) add_norm_backward_kernel(GradParams p) {
    __shared__ float2 part[2][WPR];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    float dw[NC][8] = {};
    int buf = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, buf ^= 1) {
        float s[NC][8], g[NC][8];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = 8 * (lane + 64 * (wave + WPR * i));
            if (c < p.C) {
                load8<T>(static_cast<const T *>(p.s) + t * p.ss + c, s[i]);
                load8<T>(static_cast<const T *>(p.dy) + t * p.dys + c, g[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) s[i][j] = g[i][j] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = 8 * (lane + 64 * (wave + WPR * i));
            float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
            if (p.w && c < p.C) load8<float>(p.w + c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss = fmaf(s[i][j], s[i][j], ss);
                dot = fmaf(s[i][j], g[i][j] * w[j], dot);
            }
        }
        ss = wave_sum(ss);
        dot = wave_sum(dot);
        if (WPR > 1) {
            if (lane == 0) part[buf][wave] = make_float2(ss, dot);
            __syncthreads();
            ss = dot = 0.f;
#pragma unroll
            for (int q = 0; q < WPR; ++q) { ss += part[buf][q].x; dot += part[buf][q].y; }
        }
        const float rs = rsqrtf(ss / (float)p.C + p.eps), k = dot / (float)p.C * rs * rs;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = 8 * (lane + 64 * (wave + WPR * i));
            if (c >= p.C) continue;
            float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, d[8];
            if (p.w) load8<float>(p.w + c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[i][j] = fmaf(g[i][j], s[i][j] * rs, dw[i][j]);
                d[j] = rs * (g[i][j] * w[j] - k * s[i][j]);
            }
            if (p.dr) {
                float r[8];
                load8<T>(static_cast<const T *>(p.dr) + t * p.drs + c, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] += r[j];
            }
            store8(static_cast<T *>(p.dx) + t * p.dxs + c, d);
        }
    }
    if (p.part) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = 8 * (lane + 64 * (wave + WPR * i));
            if (c < p.C) store8(p.part + (size_t)blockIdx.x * p.C + c, dw[i]);
        }
    }
}

// dweight: 32 channels a workgroup, 8 lanes of four, 32 slices of the partial rows joined
// through LDS in order.
__global__ void __launch_bounds__(256) weight_grad_kernel(const float *part, int rows, int C, float *dw) {
    __shared__ f32x4 sums[32][8];
    const int lane = threadIdx.x % 8, slice = threadIdx.x / 8, c = blockIdx.x * 32 + 4 * lane;
    f32x4 a = {0.f, 0.f, 0.f, 0.f};
    if (c < C) {
        const int per = (rows + 31) / 32, end = min(rows, (slice + 1) * per);
        for (int r = slice * per; r < end; ++r) a = a + *reinterpret_cast<const f32x4 *>(part + (size_t)r * C + c);
    }
    sums[slice][lane] = a;
    __syncthreads();
    if (slice == 0 && c < C) {
        for (int q = 1; q < 32; ++q) a = a + sums[q][lane];
        *reinterpret_cast<f32x4 *>(dw + c) = a;
    }
}

// Waves a row takes: one where its channels fit one wave's registers (eight runs of 512)
// and there are rows enough to fill the GPU with such waves, else four.
constexpr int64_t kManyRows = 2048;
constexpr unsigned kMaxBlocks = 1u << 20;

template <typename T, int QUANT, int WPR> void launch_norm(const NormParams &p, hipStream_t s) {
    const unsigned blocks = (unsigned)std::min<int64_t>(p.T, kMaxBlocks);
    const int runs = (p.C + 512 * WPR - 1) / (512 * WPR);
    const dim3 grid(blocks), block(64 * WPR);
    if (runs <= 1) hipLaunchKernelGGL((add_norm_kernel<T, QUANT, WPR, 1>), grid, block, 0, s, p);
    else if (runs <= 2) hipLaunchKernelGGL((add_norm_kernel<T, QUANT, WPR, 2>), grid, block, 0, s, p);
    else if (runs <= 4) hipLaunchKernelGGL((add_norm_kernel<T, QUANT, WPR, 4>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((add_norm_kernel<T, QUANT, WPR, 8>), grid, block, 0, s, p);
    trace("add_norm_kernel<waves=%d, runs=%d> grid=(%u) block=%d", WPR, runs, blocks, 64 * WPR);
}
template <typename T, int QUANT> void launch_norm(const NormParams &p, hipStream_t s) {
    p.C <= 4096 && p.T >= kManyRows ? launch_norm<T, QUANT, 1>(p, s) : launch_norm<T, QUANT, 4>(p, s);
}
template <typename T> void launch_norm(const NormParams &p, int quant, hipStream_t s) {
    if (quant == KDA_QUANT_NONE) launch_norm<T, KDA_QUANT_NONE>(p, s);
    else if (quant == KDA_QUANT_TOKEN) launch_norm<T, KDA_QUANT_TOKEN>(p, s);
    else launch_norm<T, KDA_QUANT_GROUP>(p, s);
}

template <typename T> void launch_grad(const GradParams &p, unsigned blocks, hipStream_t s) {
    const int runs = (p.C + 2047) / 2048;
    const dim3 grid(blocks), block(256);
    if (runs <= 1) hipLaunchKernelGGL((add_norm_backward_kernel<T, 4, 1>), grid, block, 0, s, p);
    else if (runs <= 2) hipLaunchKernelGGL((add_norm_backward_kernel<T, 4, 2>), grid, block, 0, s, p);
    else if (runs <= 4) hipLaunchKernelGGL((add_norm_backward_kernel<T, 4, 4>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((add_norm_backward_kernel<T, 4, 8>), grid, block, 0, s, p);
}

unsigned grad_blocks(int64_t T) { return (unsigned)std::min<int64_t>(T, 512); }

}  // namespace

size_t add_norm_backward_workspace_bytes(int64_t T, int C) { return (size_t)grad_blocks(T) * C * 4; }

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
    const unsigned blocks = grad_blocks(p.T);
    if (p.T > 0) {
        a->dtype == KDA_BF16 ? launch_grad<__bf16>(p, blocks, s) : launch_grad<float>(p, blocks, s);
        trace("add_norm_backward_kernel grid=(%u) block=256", blocks);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a->dweight) {
        hipLaunchKernelGGL(weight_grad_kernel, dim3((p.C + 31) / 32), dim3(256), 0, s, p.part, (int)blocks, p.C, a->dweight);
        trace("weight_grad_kernel grid=(%d) block=256", (p.C + 31) / 32);
    }
    return hipGetLastError();
}

}  // namespace kda
