// ssm_token.cuh -- selective state space scan: arguments shared by its kernels,
// and the kernel of single tokens,
//   d = softplus(dt + bias_h)   (or dt + bias_h),   a = e^{d A_h}
//   S <- a S + d k v^T ,   o = S^T q + D_h v
//
// Bound by the state's traffic (read and written once in fp32: 268 MB for 128
// sequences of 32 heads of 128 x 64 take 43 us, 6.2 TB/s; with an L2 full of
// other data 47, and 55 with 256 threads a block).  A CTA holds CW of the d_v columns of one (b, h) state in registers:
// thread (row group rg, column group cg) has rows rg, rg + RG, ... of four
// consecutive columns, so that state loads and stores are 16 bytes a thread
// and whole rows a warp, all of them in flight before the first is used.  The
// readout is a sum over the row groups: shuffles inside a warp, then one row of
// partials per warp in shared memory.
#pragma once

#include "common.cuh"

namespace gdn {
namespace ssm {

struct Args {
    const void *q, *k, *v, *dt;
    size_t q_bs, q_ts, k_bs, k_ts, v_bs, v_ts, dt_bs, dt_ts;   // elements
    const float *A, *D, *dt_bias;      // [H]; D and dt_bias may be NULL
    const float *state_in;             // [B, H, dk, dv] or NULL
    float *state_out;                  // or NULL; may be state_in
    void *o;                           // [B, T, H, dv]
    const int *lengths;                // [B] or NULL
    int B, T, H, G, softplus;
};

__device__ __forceinline__ int live_tokens(const Args &a, int b) {
    return a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
}

// Step size of a token: softplus(x) = max(x, 0) + log(1 + e^-|x|).
__device__ __forceinline__ float step_size(float x, int softplus) {
    return softplus ? fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))) : x;
}

// Log decay of a token.  A token without a step (and a place behind the
// sequence's end) forgets nothing, whatever A is: -inf times 0 would be NaN.
__device__ __forceinline__ float log_decay(float d, float A) { return d == 0.f ? 0.f : d * A; }
// A token's decay, to the nearest: near one expf is off by a quarter of a step in
// the mean, to one side, and a state that forgets slowly adds that up.
__device__ __forceinline__ float decay(float d, float A) {
    const float x = log_decay(d, A);
    return x > -0.5f ? 1.f + expm1f(x) : expf(x);
}
// A decay as a + e, a the fp32 below it: S <- a S + (e S + d k v^T).  Near one even the
// nearest fp32 is off by up to 2^-25, as much as a slow head forgets: 2e-5 of the
// state's norm behind 3,000 tokens, 6e-5 with expf, 1.4e-6 in this form.  It costs a
// multiply-add for each element of the state, which is free where the state comes
// from memory for every token.  e stays above zero: zero times an infinite element
// would be NaN.
struct Decay {
    float a, e;
};
constexpr float kTiny = 1e-30f;
// From the decay less one, in [-1/2, 0].
__device__ __forceinline__ Decay decay_near_one(float m) {
    float a = 1.f + m, e = (1.f - a) + m;
    if (e < 0.f) {
        a -= 0x1p-24f;
        e += 0x1p-24f;
    }
    return {a, fmaxf(e, kTiny)};
}
__device__ __forceinline__ Decay split_decay(float d, float A) {
    const float x = log_decay(d, A);
    return x > -0.6931471805599453f ? decay_near_one(expm1f(x)) : Decay{expf(x), kTiny};
}

constexpr int kTokThreads = 128;

// grid (DV / CW, B * H)
template <int DK, int DV, int CW, typename T, typename Td>
__global__ void __launch_bounds__(kTokThreads)
token_kernel(const Args a)
{
    constexpr int NC = CW / 4;                    // column groups
    constexpr int RG = kTokThreads / NC;          // row groups
    constexpr int RPT = DK / RG;                  // rows per thread
    constexpr int NW = kTokThreads / 32;
    static_assert(RPT >= 1 && NC <= 32, "layout");
    __shared__ __align__(16) float ks[DK], qs[DK], vs[CW], part[NW][CW];

    const int tid = threadIdx.x, cg = tid % NC, rg = tid / NC, warp = tid >> 5;
    const int b = blockIdx.y / a.H, h = blockIdx.y % a.H, g = h / (a.H / a.G);
    const int c0 = blockIdx.x * CW;
    const int n = live_tokens(a, b);              // 0 or 1
    const size_t sbase = ((size_t)blockIdx.y * DK) * DV + c0 + cg * 4;
    float4 S[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m)
        S[m] = a.state_in ? *reinterpret_cast<const float4 *>(a.state_in + sbase + (size_t)(rg + RG * m) * DV)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    if (n > 0) {
        const T *q = static_cast<const T *>(a.q) + b * a.q_bs + (size_t)g * DK;
        const T *k = static_cast<const T *>(a.k) + b * a.k_bs + (size_t)g * DK;
        const T *v = static_cast<const T *>(a.v) + b * a.v_bs + (size_t)h * DV + c0;
        for (int i = tid; i < DK; i += kTokThreads) {
            ks[i] = to_f32(k[i]);
            qs[i] = to_f32(q[i]);
        }
        for (int i = tid; i < CW; i += kTokThreads) vs[i] = to_f32(v[i]);
        const float bias = a.dt_bias ? a.dt_bias[h] : 0.f;
        const float d = step_size(to_f32(static_cast<const Td *>(a.dt)[b * a.dt_bs + h]) + bias, a.softplus);
        const Decay al = split_decay(d, a.A[h]);
        __syncthreads();
        const float4 vv = *reinterpret_cast<const float4 *>(&vs[cg * 4]);
        const float4 u = make_float4(d * vv.x, d * vv.y, d * vv.z, d * vv.w);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int m = 0; m < RPT; ++m) {
            const float kr = ks[rg + RG * m], qr = qs[rg + RG * m];
            S[m].x = fmaf(al.a, S[m].x, fmaf(al.e, S[m].x, kr * u.x));
            S[m].y = fmaf(al.a, S[m].y, fmaf(al.e, S[m].y, kr * u.y));
            S[m].z = fmaf(al.a, S[m].z, fmaf(al.e, S[m].z, kr * u.z));
            S[m].w = fmaf(al.a, S[m].w, fmaf(al.e, S[m].w, kr * u.w));
            y.x = fmaf(qr, S[m].x, y.x);
            y.y = fmaf(qr, S[m].y, y.y);
            y.z = fmaf(qr, S[m].z, y.z);
            y.w = fmaf(qr, S[m].w, y.w);
        }
#pragma unroll
        for (int s = NC; s < 32; s <<= 1) {
            y.x += __shfl_xor_sync(0xffffffffu, y.x, s);
            y.y += __shfl_xor_sync(0xffffffffu, y.y, s);
            y.z += __shfl_xor_sync(0xffffffffu, y.z, s);
            y.w += __shfl_xor_sync(0xffffffffu, y.w, s);
        }
        if ((tid & 31) < NC) *reinterpret_cast<float4 *>(&part[warp][cg * 4]) = y;
        __syncthreads();
        if (tid < CW) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) s += part[w][tid];
            const float D = a.D ? a.D[h] : 0.f;
            static_cast<T *>(a.o)[((size_t)b * a.H + h) * DV + c0 + tid] = from_f32<T>(fmaf(D, vs[tid], s));
        }
    }
    if (a.state_out)
#pragma unroll
        for (int m = 0; m < RPT; ++m)
            *reinterpret_cast<float4 *>(a.state_out + sbase + (size_t)(rg + RG * m) * DV) = S[m];
}

}  // namespace ssm
}  // namespace gdn
