// kda_linattn_decode.hip -- one token of the linear attention with one decay per
// head: S <- exp(min(g, 0)) S + k v^T, o = scale S^T q.
//
// A workgroup of four threads to a column owns 64 or 128 columns of one (sequence, head)
// state: the columns of a state never mix, so any split over them is exact.  The state
// stays in registers from its read to its write; thread t owns 16 bytes of neighbouring
// columns in rows t / LPR + RG m.  Per element: one multiply and two FMAs (the decay,
// the write k v, the read q); the column sums cross the lanes of a wave, then the
// waves through LDS.
//
// The bound is HBM: every state is read once and written once, with non-temporal
// accesses (a step's states are not read again before every other layer's).  256
// sequences x 64 heads of fp32 states (2.16 GB): 366 to 373 us, 5.9 TB/s, the rate of a bare
// read-and-write-back of such states; 409 us without the hint.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

namespace {

struct DecodeParams {
    const void *q, *k, *v;
    const float *g;
    void *state, *o;
    const int32_t *slots;
    int64_t qs, ks, vs, gs;  // elements per sequence (gs 0: one decay per head)
    int H, rep, num_slots, dv, tiles;
    float scale;
};

// Sixteen bytes of a stored state.
template <typename S> struct StateVec;
template <> struct StateVec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float *p, float (&f)[4]) {
        const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p));
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = v[i];
    }
    static __device__ __forceinline__ void store(float *p, const float (&f)[4]) {
        __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4 *>(p));
    }
};
template <> struct StateVec<__bf16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const __bf16 *p, float (&f)[8]) {
        const bf16x8 v = __builtin_nontemporal_load(reinterpret_cast<const bf16x8 *>(p));
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)v[i];
    }
    static __device__ __forceinline__ void store(__bf16 *p, const float (&f)[8]) {
        __builtin_nontemporal_store(pack8(f32x4{f[0], f[1], f[2], f[3]}, f32x4{f[4], f[5], f[6], f[7]}),
                                    reinterpret_cast<bf16x8 *>(p));
    }
};

template <typename T, typename S, int DK, int DVT>
__global__ void __launch_bounds__(4 * DVT) decode_kernel(DecodeParams p) {
    constexpr int VEC = StateVec<S>::N, WAVES = DVT / 16;
    constexpr int LPR = DVT / VEC;     // lanes of a state row
    constexpr int RG = 4 * DVT / LPR;     // rows held side by side
    constexpr int M = DK / RG;         // rows per thread
    static_assert(M * RG == DK, "thread layout");
    __shared__ float sq[DK], sk[DK], part[WAVES][DVT];
    const int tid = threadIdx.x, tile = blockIdx.x % p.tiles;
    const int pair = blockIdx.x / p.tiles, n = pair / p.H, h = pair - n * p.H;
    const int slot = pool_slot(p.slots, p.num_slots, n);
    if (slot < 0) return;
    const int cl = tid % LPR, rg = tid / LPR, col = tile * DVT + cl * VEC;
    S *s = static_cast<S *>(p.state) + (((size_t)slot * p.H + h) * DK + rg) * p.dv + col;
    float f[M][VEC];
#pragma unroll
    for (int m = 0; m < M; ++m) StateVec<S>::load(s + (size_t)m * RG * p.dv, f[m]);
    if (tid < DK) {
        const int64_t hk = (int64_t)(h / p.rep) * DK + tid;
        sq[tid] = to_f32(static_cast<const T *>(p.q)[n * p.qs + hk]) * p.scale;
        sk[tid] = to_f32(static_cast<const T *>(p.k)[n * p.ks + hk]);
    }
    const T *v = static_cast<const T *>(p.v) + n * p.vs + (int64_t)h * p.dv + col;
    float g = p.g[n * p.gs + h], vv[VEC], acc[VEC];
    g = g > 0.f ? 0.f : g;  // NaN stays
    const float a = exp2_fast(g * 1.4426950408889634f);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        vv[i] = to_f32(v[i]);
        acc[i] = 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const float kr = sk[rg + RG * m], qr = sq[rg + RG * m];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            f[m][i] = fmaf(kr, vv[i], a * f[m][i]);
            acc[i] = fmaf(qr, f[m][i], acc[i]);
        }
    }
#pragma unroll
    for (int m = 0; m < M; ++m) StateVec<S>::store(s + (size_t)m * RG * p.dv, f[m]);
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
        float o = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
        if constexpr (WAVES == 8) o += (part[4][tid] + part[5][tid]) + (part[6][tid] + part[7][tid]);
        static_cast<T *>(p.o)[((size_t)n * p.H + h) * p.dv + tile * DVT + tid] = from_f32<T>(o);
    }
}

template <typename T, typename S, int DK, int DVT> hipError_t launch(DecodeParams p, int N, hipStream_t s) {
    p.tiles = p.dv / DVT;
    const unsigned blocks = (unsigned)N * p.H * p.tiles;
    hipLaunchKernelGGL((decode_kernel<T, S, DK, DVT>), dim3(blocks), dim3(4 * DVT), 0, s, p);
    trace("decode_kernel<dk=%d, %d columns> grid=(%u) block=%d", DK, DVT, blocks, 4 * DVT);
    return hipGetLastError();
}
// 128 columns where there are states enough, us (64/128 columns, 512 threads; states not
// cached): 64 heads, 1 sequence 4.3/5.0, 4 7.4/7.8, 8 13.5/13.2, 256 381/373, with bf16
// states 195/182.
template <typename T, typename S, int DK> hipError_t launch(const DecodeParams &p, int N, hipStream_t s) {
    return p.dv == 128 && (int64_t)N * p.H >= 512 ? launch<T, S, DK, 128>(p, N, s) : launch<T, S, DK, 64>(p, N, s);
}
template <typename T> hipError_t launch(const DecodeParams &p, const kda_linattn_decode_args *a, hipStream_t s) {
    const int N = a->num_seqs;
    if (a->flags & KDA_F_STATE_BF16)
        return a->head_dim_k == 64 ? launch<T, __bf16, 64>(p, N, s) : launch<T, __bf16, 128>(p, N, s);
    return a->head_dim_k == 64 ? launch<T, float, 64>(p, N, s) : launch<T, float, 128>(p, N, s);
}

}  // namespace

hipError_t launch_linattn_decode(const kda_linattn_decode_args *a, hipStream_t s) {
    DecodeParams p = {};
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->log_decay;
    p.state = a->state; p.o = a->o;
    p.slots = a->state_slots; p.num_slots = a->num_slots;
    p.H = a->num_heads; p.rep = a->num_heads / a->num_k_heads;
    p.qs = a->q_stride; p.ks = a->k_stride; p.vs = a->v_stride;
    p.gs = (a->flags & KDA_F_DECAY_PER_HEAD) ? 0 : a->num_heads;
    p.dv = a->head_dim_v; p.scale = a->scale;
    return a->dtype == KDA_BF16 ? launch<__bf16>(p, a, s) : launch<float>(p, a, s);
}

}  // namespace kda
