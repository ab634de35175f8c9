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

// Sum over the D / 8 lanes of a row, in every lane of it.
template <int D> __device__ __forceinline__ float row_total(float s) {
    s += KDA_DPP(s, 0xb1);   // quad_perm [1,0,3,2]
    s += KDA_DPP(s, 0x4e);   // quad_perm [2,3,0,1]
    s += KDA_DPP(s, 0x141);  // row_half_mirror
    if (D == 128) s += KDA_DPP(s, 0x140);  // row_mirror
    return s;
}
template <int D> __device__ __forceinline__ float row_sumsq(const float (&x)[8]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
    return row_total<D>(s);
}

template <typename T> struct Quad;  // four neighbouring elements
template <> struct Quad<__bf16> { typedef bf16x4 vec; };
template <> struct Quad<float> { typedef f32x4 vec; };
template <typename T> __device__ __forceinline__ f32x4 wide(typename Quad<T>::vec x) {
    return f32x4{(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
}
__device__ __forceinline__ void store4(__bf16 *p, f32x4 x) { *reinterpret_cast<bf16x4 *>(p) = pack4(x); }
__device__ __forceinline__ void store4(float *p, f32x4 x) { *reinterpret_cast<f32x4 *>(p) = x; }

struct QkParams {
    const void *x[2];        // q, k
    void *y[2];
    const float *w[2], *inv_freq;
    const int32_t *pos;
    int64_t T, xs[2], ys[2];
    int H[2], qgroups;       // heads; runs of kRun heads that q takes
    int R, norm;
    float eps;
};
constexpr int kRun = 32;     // heads of one wave

// One wave per (token, run of heads of q or of k).  A row's D / 8 lanes hold two quads
// of elements each: lane e of a rotated part the quads of pairs 4 e .. 4 e + 3 (both
// halves of the pair, whichever way they are paired), the others neighbouring quads of
// the unrotated rest, so no element crosses lanes.  Lane i < R / 2 forms the angle of
// pair i once for the whole run: the turns pos * inv_freq / 2 pi are reduced in 64
// bits, so the 32-bit sine and cosine see an argument of at most one half; the pairs
// reach the lanes that rotate by them through LDS.  4096 tokens x (64 + 64) heads x 128
// (268 MB moved): 53 us, 5.0 TB/s, the rate of a large copy; 88 us with one quad of rows
// in flight, pairs exchanged between lanes and cosines held for eight elements.
template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(64) qk_norm_rope_kernel(QkParams p) {
    typedef typename Quad<T>::vec vec;
    constexpr int LPR = D / 8, RPW = 64 / LPR, ITER = kRun / RPW, BATCH = ITER < 4 ? ITER : 4;
    __shared__ float2 cs[64];
    const int lane = threadIdx.x, e = lane % LPR, sub = lane / LPR;
    const int half = p.R / 2;
    const bool rot = 8 * e < p.R;
    const int at0 = rot && !INTERLEAVED ? 4 * e : 8 * e, at1 = rot && !INTERLEAVED ? half + 4 * e : 8 * e + 4;
    const int isk = (int)blockIdx.y >= p.qgroups, h0 = (blockIdx.y - (isk ? p.qgroups : 0)) * kRun;
    const int heads = min(p.H[isk] - h0, kRun);
    f32x4 w0 = {1.f, 1.f, 1.f, 1.f}, w1 = w0;
    if (p.w[isk]) {
        w0 = *reinterpret_cast<const f32x4 *>(p.w[isk] + at0);
        w1 = *reinterpret_cast<const f32x4 *>(p.w[isk] + at1);
    }
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const T *x = static_cast<const T *>(p.x[isk]) + t * p.xs[isk] + (int64_t)(h0 + sub) * D;
        T *y = static_cast<T *>(p.y[isk]) + t * p.ys[isk] + (int64_t)(h0 + sub) * D;
        f32x4 co = {1.f, 1.f, 1.f, 1.f}, si = {0.f, 0.f, 0.f, 0.f};
        vec v0[BATCH], v1[BATCH];
        auto load = [&](int b) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if ((b + i) * RPW + sub < heads) {
                    v0[i] = *reinterpret_cast<const vec *>(x + (b + i) * RPW * D + at0);
                    v1[i] = *reinterpret_cast<const vec *>(x + (b + i) * RPW * D + at1);
                }
        };
        load(0);  // under the angles
        if (p.R) {
            __syncthreads();
            if (lane < half) {
                const double turns = (double)p.pos[t] * (double)p.inv_freq[lane] * 0.15915494309189535;
                float s, c;
                sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
                cs[lane] = make_float2(c, s);
            }
            __syncthreads();
            if (rot) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    co[i] = cs[4 * e + i].x;
                    si[i] = cs[4 * e + i].y;
                }
            }
        }
#pragma unroll
        for (int b = 0; b < ITER; b += BATCH) {
            if (b > 0) {
                if (b * RPW >= heads) break;
                load(b);
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if ((b + i) * RPW >= heads) break;  // (30,000 tokens x 4 + 2 heads of 64: 32 -> 20 us)
                const bool on = (b + i) * RPW + sub < heads;
                f32x4 a = on ? wide<T>(v0[i]) : f32x4{}, c = on ? wide<T>(v1[i]) : f32x4{};
                if (p.norm != KDA_NORM_NONE) {
                    float ss = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) ss = fmaf(a[j], a[j], fmaf(c[j], c[j], ss));
                    ss = row_total<D>(ss);
                    const float rs = rsqrtf((p.norm == KDA_NORM_RMS ? ss * (1.f / D) : ss) + p.eps);
                    a = a * (w0 * rs);
                    c = c * (w1 * rs);
                }
                if (rot) {  // (never of an infinity by a zero sine in the unrotated rest)
                    const f32x4 u = a, z = c;
                    if (INTERLEAVED) {
                        a = f32x4{u[0] * co[0] - u[1] * si[0], u[1] * co[0] + u[0] * si[0],
                                  u[2] * co[1] - u[3] * si[1], u[3] * co[1] + u[2] * si[1]};
                        c = f32x4{z[0] * co[2] - z[1] * si[2], z[1] * co[2] + z[0] * si[2],
                                  z[2] * co[3] - z[3] * si[3], z[3] * co[3] + z[2] * si[3]};
                    } else {
                        a = u * co - z * si;
                        c = z * co + u * si;
                    }
                }
                if (on) {
                    store4(y + (b + i) * RPW * D + at0, a);
                    store4(y + (b + i) * RPW * D + at1, c);
                }
            }
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

// One row of one head.  16,384 tokens x 64 heads x 128 in bf16 with the gate (805 MB
// moved): 142 us, 5.65 TB/s, above the 5.2 of a large copy, which writes half of what it
// moves where this writes a third.
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

template <typename T, bool INTERLEAVED> void launch_qk(const QkParams &p, int D, dim3 grid, hipStream_t s) {
    if (D == 64) hipLaunchKernelGGL((qk_norm_rope_kernel<T, 64, INTERLEAVED>), grid, dim3(64), 0, s, p);
    else hipLaunchKernelGGL((qk_norm_rope_kernel<T, 128, INTERLEAVED>), grid, dim3(64), 0, s, p);
}

}  // namespace

hipError_t launch_qk_norm_rope(const kda_qk_norm_rope_args *a, hipStream_t s) {
    QkParams p = {};
    p.x[0] = a->q; p.x[1] = a->k; p.y[0] = a->q_out; p.y[1] = a->k_out;
    p.w[0] = a->q_weight; p.w[1] = a->k_weight; p.inv_freq = a->inv_freq; p.pos = a->positions;
    p.T = a->total_tokens;
    p.xs[0] = a->q_stride; p.xs[1] = a->k_stride; p.ys[0] = a->q_out_stride; p.ys[1] = a->k_out_stride;
    p.H[0] = a->num_q_heads; p.H[1] = a->num_k_heads;
    p.qgroups = (p.H[0] + kRun - 1) / kRun;
    p.R = a->rotary_dim; p.norm = a->norm; p.eps = a->eps;
    const bool pairs = (a->flags & KDA_F_ROPE_INTERLEAVED) != 0;
    const dim3 grid((unsigned)std::min<int64_t>(p.T, kMaxBlocks), p.qgroups + (p.H[1] + kRun - 1) / kRun);
    if (a->dtype == KDA_BF16) pairs ? launch_qk<__bf16, true>(p, a->head_dim, grid, s) : launch_qk<__bf16, false>(p, a->head_dim, grid, s);
    else pairs ? launch_qk<float, true>(p, a->head_dim, grid, s) : launch_qk<float, false>(p, a->head_dim, grid, s);
    trace("qk_norm_rope_kernel<D=%d> grid=(%u, %u) block=64", a->head_dim, grid.x, grid.y);
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
