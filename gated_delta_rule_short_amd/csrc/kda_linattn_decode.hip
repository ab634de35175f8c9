// kda_linattn_decode.hip -- recurrent form of the linear attention with one decay
// per head: S <- exp(g) S + k v^T, o = scale S^T q, token by token.
//
// A workgroup owns DVT columns of one (sequence, head) state: the columns of a
// state never mix, so any split over them is exact.  The state stays in
// registers from its read to its write; thread t owns VEC neighbouring columns
// (16 bytes of storage) of rows t / LPR + RG m.  Per element and token: the decay,
// the write k v and the read q are one multiply and two FMAs, and the column
// sums cross the lanes of a wave, then the waves through LDS.  The bound is HBM:
// every state is read once and written once.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

namespace {

struct RecurParams {
    const void *q, *k, *v;
    const float *g;
    const void *s_in;
    void *s_out, *o;
    const int32_t *cu, *slots;
    int64_t total, qs, ks, vs, gs;  // gs: elements of g per token (0: one decay per head)
    int N, H, rep, num_slots, dv, tiles;
    float scale;
};

template <typename S> struct StateVec;
template <> struct StateVec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float *p, float (&f)[4]) {
        const f32x4 v = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = v[i];
    }
    static __device__ __forceinline__ void store(float *p, const float (&f)[4]) {
        *reinterpret_cast<f32x4 *>(p) = f32x4{f[0], f[1], f[2], f[3]};
    }
};
template <> struct StateVec<__bf16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const __bf16 *p, float (&f)[8]) {
        const bf16x8 v = *reinterpret_cast<const bf16x8 *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)v[i];
    }
    static __device__ __forceinline__ void store(__bf16 *p, const float (&f)[8]) {
        *reinterpret_cast<bf16x8 *>(p) = pack8(f32x4{f[0], f[1], f[2], f[3]}, f32x4{f[4], f[5], f[6], f[7]});
    }
};

// exp(min(g, 0)); a NaN stays one.
__device__ __forceinline__ float decay_of(float g) {
    g = g > 0.f ? 0.f : g;
    return exp2_fast(g * 1.4426950408889634f);
}

template <typename T, typename S, int DK, int DVT, int NT>
__global__ void __launch_bounds__(NT) recurrent_kernel(RecurParams p) {
    constexpr int VEC = StateVec<S>::N;
    constexpr int LPR = DVT / VEC;     // lanes of a state row
    constexpr int RG = NT / LPR;       // rows held side by side
    constexpr int M = DK / RG;         // rows per thread
    constexpr int NW = NT / 64;
    static_assert(M * RG == DK && LPR <= 64 && DK <= NT && DVT <= NT, "thread layout");
    __shared__ float sq[2][DK], sk[2][DK], part[NW][DVT];
    const int tid = threadIdx.x, tile = blockIdx.x % p.tiles;
    const int pair = blockIdx.x / p.tiles, n = pair / p.H, h = pair - n * p.H;
    const int slot = pool_slot(p.slots, p.num_slots, n);
    if (slot < 0) return;
    int64_t t0, len;
    if (p.cu) {
        t0 = min((int64_t)max(p.cu[n], 0), p.total);
        len = min((int64_t)max(p.cu[n + 1], 0), p.total) - t0;
    } else {
        len = p.total / p.N;
        t0 = len * n;
    }
    const int cl = tid % LPR, rg = tid / LPR, col = tile * DVT + cl * VEC;
    const size_t base = (((size_t)slot * p.H + h) * DK + rg) * p.dv + col;
    float f[M][VEC];
    const S *si = static_cast<const S *>(p.s_in);
    if (si) {
#pragma unroll
        for (int m = 0; m < M; ++m) StateVec<S>::load(si + base + (size_t)m * RG * p.dv, f[m]);
    } else {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[m][i] = 0.f;
    }
    const int hk = h / p.rep;
    const T *q = static_cast<const T *>(p.q) + (size_t)hk * DK, *k = static_cast<const T *>(p.k) + (size_t)hk * DK;
    const T *v = static_cast<const T *>(p.v) + (size_t)h * p.dv + col;
    T *o = static_cast<T *>(p.o);
    for (int64_t t = t0; t < t0 + len; ++t) {
        const int b = (int)(t - t0) & 1;
        if (tid < DK) {
            sq[b][tid] = to_f32(q[t * p.qs + tid]) * p.scale;
            sk[b][tid] = to_f32(k[t * p.ks + tid]);
        }
        const float a = decay_of(p.g[t * p.gs + h]);
        float vv[VEC], acc[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            vv[i] = to_f32(v[t * p.vs + i]);
            acc[i] = 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const float kr = sk[b][rg + RG * m], qr = sq[b][rg + RG * m];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                f[m][i] = fmaf(kr, vv[i], a * f[m][i]);
                acc[i] = fmaf(qr, f[m][i], acc[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i)
#pragma unroll
            for (int d = LPR; d < 64; d *= 2) acc[i] += __shfl_xor(acc[i], d);
        if (tid % 64 < LPR) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) part[tid / 64][cl * VEC + i] = acc[i];
        }
        __syncthreads();
        if (tid < DVT) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) s += part[w][tid];
            o[((size_t)t * p.H + h) * p.dv + tile * DVT + tid] = from_f32<T>(s);
        }
    }
    S *so = static_cast<S *>(p.s_out);
    if (so) {
#pragma unroll
        for (int m = 0; m < M; ++m) StateVec<S>::store(so + base + (size_t)m * RG * p.dv, f[m]);
    }
}

template <typename T, typename S, int DK>
hipError_t launch(RecurParams p, hipStream_t s) {
    // 64-column tiles: two workgroups per 128-wide state
    p.tiles = p.dv / 64;
    const unsigned blocks = (unsigned)p.N * p.H * p.tiles;
    hipLaunchKernelGGL((recurrent_kernel<T, S, DK, 64, 256>), dim3(blocks), dim3(256), 0, s, p);
    trace("recurrent_kernel<dk=%d> grid=(%u) block=256", DK, blocks);
    return hipGetLastError();
}

hipError_t dispatch(const RecurParams &p, kda_dtype dt, uint32_t flags, int dk, hipStream_t s) {
    const bool sb = flags & KDA_F_STATE_BF16;
    if (dt == KDA_BF16) {
        if (dk == 64) return sb ? launch<__bf16, __bf16, 64>(p, s) : launch<__bf16, float, 64>(p, s);
        return sb ? launch<__bf16, __bf16, 128>(p, s) : launch<__bf16, float, 128>(p, s);
    }
    if (dk == 64) return sb ? launch<float, __bf16, 64>(p, s) : launch<float, float, 64>(p, s);
    return sb ? launch<float, __bf16, 128>(p, s) : launch<float, float, 128>(p, s);
}

}  // namespace

hipError_t launch_linattn_decode(const kda_linattn_decode_args *a, hipStream_t s) {
    RecurParams p = {};
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->log_decay;
    p.s_in = a->state; p.s_out = a->state; p.o = a->o;
    p.slots = a->state_slots; p.num_slots = a->num_slots;
    p.total = a->num_seqs; p.N = a->num_seqs; p.H = a->num_heads; p.rep = a->num_heads / a->num_k_heads;
    p.qs = a->q_stride; p.ks = a->k_stride; p.vs = a->v_stride;
    p.gs = (a->flags & KDA_F_DECAY_PER_HEAD) ? 0 : a->num_heads;
    p.dv = a->head_dim_v; p.scale = a->scale;
    return dispatch(p, a->dtype, a->flags, a->head_dim_k, s);
}

}  // namespace kda
