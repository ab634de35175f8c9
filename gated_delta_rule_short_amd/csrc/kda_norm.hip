// kda_norm.hip -- per-head norms around the mixers: queries and keys with their
// position rotation, and the gated norm of the mixer's output.
//
// A head row of D elements belongs to D / 8 neighbouring lanes, eight elements
// each, so a wave of 64 holds 512 / D rows and a row's sum of squares stays inside
// a 16-lane DPP row.  Both kernels stream: every element is read once and
// written once and the bound is HBM.
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

// Sum of squares over the D / 8 lanes of a row, in every lane of it.
template <int D> __device__ __forceinline__ float row_sumsq(const float (&x)[8]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
    s += KDA_DPP(s, 0xb1);   // quad_perm [1,0,3,2]
    s += KDA_DPP(s, 0x4e);   // quad_perm [2,3,0,1]
    s += KDA_DPP(s, 0x141);  // row_half_mirror
    if (D == 128) s += KDA_DPP(s, 0x140);  // row_mirror
    return s;
}

struct QkParams {
    const void *q, *k;
    void *qo, *ko;
    const float *wq, *wk, *inv_freq;
    const int32_t *pos;
    int64_t T, qs, ks, qos, kos;
    int Hq, Hk, groups, per_group;  // a token's rows in `groups` runs of `per_group`
    int R, norm, interleaved;
    float eps;
};

// One wave per (token, run of heads).  Lane i < R / 2 forms the angle of pair i:
// the turns pos * inv_freq / 2 pi are reduced in 64 bits, so the 32-bit sine and
// cosine see an argument below one half.  The pairs reach the lanes that need
// them through the wave's own LDS.
template <typename T, int D>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(QkParams p) {
    constexpr int LPR = D / 8, RPW = 64 / LPR;
    __shared__ float2 cs[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t first = (int64_t)blockIdx.x * 4; first < p.T * p.groups; first += (int64_t)gridDim.x * 4) {
    const int64_t item = first + wave;
    const int64_t t = item / p.groups;
    const bool live = t < p.T;
    const int g = (int)(item - t * p.groups);
    __syncthreads();
    if (p.R && live && lane < p.R / 2) {
        const double turns = (double)p.pos[t] * (double)p.inv_freq[lane] * 0.15915494309189535;
        const float fr = (float)(turns - rint(turns));
        float s, c;
        sincospif(2.f * fr, &s, &c);
        cs[wave][lane] = make_float2(c, s);
    }
    __syncthreads();
    if (!live) continue;
    const int e = lane % LPR, c0 = 8 * e, sub = lane / LPR;
    // this lane's eight elements: pair index of each, and its partner's lane
    const int half = p.R / 2;
    const bool rot = c0 < p.R;
    float co[8], si[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int j = p.interleaved ? (c0 + i) >> 1 : (c0 < half ? c0 + i : c0 + i - half);
        const float2 v = rot ? cs[wave][j] : make_float2(1.f, 0.f);
        co[i] = v.x;
        // the first of a pair takes -sin times its partner, the second +sin
        si[i] = (p.interleaved ? (i & 1) == 0 : c0 < half) ? -v.y : v.y;
    }
    const int partner = p.interleaved || !rot ? lane : (c0 < half ? lane + half / 8 : lane - half / 8);
    float w[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[0][i] = p.wq ? p.wq[c0 + i] : 1.f;
        w[1][i] = p.wk ? p.wk[c0 + i] : 1.f;
    }
    const int r1 = min((g + 1) * p.per_group, p.Hq + p.Hk);
    for (int r0 = g * p.per_group; r0 < r1; r0 += RPW) {
        const int r = r0 + sub;
        const bool on = r < r1, isk = r >= p.Hq;
        const int hh = isk ? r - p.Hq : r;
        float x[8] = {};
        if (on)
            load8<T>((isk ? static_cast<const T *>(p.k) + t * p.ks : static_cast<const T *>(p.q) + t * p.qs) +
                         (size_t)hh * D + c0, x);
        if (p.norm != KDA_NORM_NONE) {
            const float ss = row_sumsq<D>(x);
            const float rs = p.norm == KDA_NORM_RMS ? rsqrtf(ss * (1.f / D) + p.eps) : rsqrtf(ss + p.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= rs * (isk ? w[1][i] : w[0][i]);
        }
        if (p.R) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = p.interleaved ? x[i ^ 1] : __shfl(x[i], partner);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = rot ? fmaf(x[i], co[i], y[i] * si[i]) : x[i];
        }
        if (on)
            store8((isk ? static_cast<T *>(p.ko) + t * p.kos : static_cast<T *>(p.qo) + t * p.qos) +
                       (size_t)hh * D + c0, x);
    }
    }
}

struct GatedParams {
    const void *x, *z;
    void *y;
    const float *w;
    int64_t rows, xs, zs, ys;  // rows = T * H
    int H, w_head, silu;
    float eps;
};

template <typename T, int D>
__device__ __forceinline__ void gated_row(const GatedParams &p, int64_t r, int c0) {
    const int64_t t = r / p.H;
    const int h = (int)(r - t * p.H);
    const size_t at = (size_t)h * D + c0;
    float x[8];
    load8<T>(static_cast<const T *>(p.x) + t * p.xs + at, x);
    const float rs = rsqrtf(row_sumsq<D>(x) * (1.f / D) + p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= rs;
    if (p.w) {
        float w[8];
        load8<float>(p.w + (p.w_head ? at : (size_t)c0), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= w[i];
    }
    if (p.z) {
        float z[8];
        load8<T>(static_cast<const T *>(p.z) + t * p.zs + at, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= p.silu ? z[i] * sigmoidf_dev(z[i]) : sigmoidf_dev(z[i]);
    }
    store8(static_cast<T *>(p.y) + t * p.ys + at, x);
}

template <typename T, int D>
__global__ void __launch_bounds__(256) gated_norm_kernel(GatedParams p) {
    constexpr int LPR = D / 8, RPB = 256 / LPR;
    const int64_t step = (int64_t)gridDim.x * RPB;
    for (int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR; r < p.rows; r += step)
        gated_row<T, D>(p, r, 8 * (threadIdx.x % LPR));
}

// A launch holds fewer than 2^32 threads; items past that many workgroups are
// taken by the same ones in turn.
constexpr int64_t kMaxBlocks = 1 << 22;

}  // namespace

hipError_t launch_qk_norm_rope(const kda_qk_norm_rope_args *a, hipStream_t s) {
    QkParams p = {};
    p.q = a->q; p.k = a->k; p.qo = a->q_out; p.ko = a->k_out;
    p.wq = a->q_weight; p.wk = a->k_weight; p.inv_freq = a->inv_freq; p.pos = a->positions;
    p.T = a->total_tokens;
    p.qs = a->q_stride; p.ks = a->k_stride; p.qos = a->q_out_stride; p.kos = a->k_out_stride;
    p.Hq = a->num_q_heads; p.Hk = a->num_k_heads;
    p.R = a->rotary_dim; p.norm = a->norm; p.interleaved = (a->flags & KDA_F_ROPE_INTERLEAVED) != 0;
    p.eps = a->eps;
    const int rows = p.Hq + p.Hk;
    p.per_group = 16;
    p.groups = (rows + p.per_group - 1) / p.per_group;
    const int64_t items = p.T * p.groups;
    const unsigned blocks = (unsigned)std::min<int64_t>((items + 3) / 4, kMaxBlocks);
    if (a->dtype == KDA_BF16) {
        if (a->head_dim == 64) hipLaunchKernelGGL((qk_norm_rope_kernel<__bf16, 64>), dim3(blocks), dim3(256), 0, s, p);
        else hipLaunchKernelGGL((qk_norm_rope_kernel<__bf16, 128>), dim3(blocks), dim3(256), 0, s, p);
    } else {
        if (a->head_dim == 64) hipLaunchKernelGGL((qk_norm_rope_kernel<float, 64>), dim3(blocks), dim3(256), 0, s, p);
        else hipLaunchKernelGGL((qk_norm_rope_kernel<float, 128>), dim3(blocks), dim3(256), 0, s, p);
    }
    trace("qk_norm_rope_kernel<D=%d> grid=(%u) block=256", a->head_dim, blocks);
    return hipGetLastError();
}

hipError_t launch_gated_norm(const kda_gated_norm_args *a, hipStream_t s) {
    GatedParams p = {};
    p.x = a->x; p.z = a->z; p.y = a->y; p.w = a->weight;
    p.rows = a->total_tokens * a->num_heads;
    p.xs = a->x_stride; p.zs = a->z_stride; p.ys = a->y_stride;
    p.H = a->num_heads; p.w_head = (a->flags & KDA_F_WEIGHT_PER_HEAD) != 0; p.silu = (a->flags & KDA_F_SILU) != 0;
    p.eps = a->eps;
    const int rpb = 2048 / a->head_dim;
    const unsigned blocks = (unsigned)std::min<int64_t>((p.rows + rpb - 1) / rpb, kMaxBlocks);
    if (a->dtype == KDA_BF16) {
        if (a->head_dim == 64) hipLaunchKernelGGL((gated_norm_kernel<__bf16, 64>), dim3(blocks), dim3(256), 0, s, p);
        else hipLaunchKernelGGL((gated_norm_kernel<__bf16, 128>), dim3(blocks), dim3(256), 0, s, p);
    } else {
        if (a->head_dim == 64) hipLaunchKernelGGL((gated_norm_kernel<float, 64>), dim3(blocks), dim3(256), 0, s, p);
        else hipLaunchKernelGGL((gated_norm_kernel<float, 128>), dim3(blocks), dim3(256), 0, s, p);
    }
    trace("gated_norm_kernel<D=%d> grid=(%u) block=256", a->head_dim, blocks);
    return hipGetLastError();
}

}  // namespace kda
