// ssm_token.cuh -- selective state space scan, token by token on the CUDA
// cores (any length; the single-token and fp32 path):
//   d_t = softplus(dt_t + bias_h)   (or dt_t + bias_h),   a_t = e^{d_t A_h}
//   S_t = a_t S_{t-1} + d_t k_t v_t^T ,   o_t = S_t^T q_t + D_h v_t
//
// A single token is bound by the state's traffic (read and written once in
// fp32), a long call by the three multiply-adds per state element and token.
// A CTA holds CW of the d_v columns of one (b, h) state in registers: thread
// (row group rg, column group cg) has rows rg, rg + RG, ... of four
// consecutive columns, so that state loads and stores are 16 bytes a thread
// and whole rows a warp.  Tokens are staged kStage at a time in shared
// memory; a token's readout is a sum over the row groups (shuffles inside a
// warp, one double-buffered row of partials per warp).
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

constexpr int kTokThreads = 256;
constexpr int kStage = 16;

template <int DK, int DV, int CW, typename T, typename Td>
__global__ void __launch_bounds__(kTokThreads)
token_kernel(const Args a)
{
    constexpr int NC = CW / 4;                    // column groups
    constexpr int RG = kTokThreads / NC;          // row groups
    constexpr int RPT = DK / RG;                  // rows per thread
    constexpr int LPW = 32 / NC;                  // row groups per warp
    constexpr int NW = kTokThreads / 32;
    static_assert(RPT >= 1 && LPW >= 1, "layout");
    __shared__ __align__(16) float ks[kStage][DK], qs[kStage][DK], vs[kStage][CW];
    __shared__ __align__(16) float part[2][NW][CW];
    __shared__ float as[kStage], ds[kStage];

    const int tid = threadIdx.x, cg = tid % NC, rg = tid / NC, warp = tid >> 5;
    const int b = blockIdx.y / a.H, h = blockIdx.y % a.H, g = h / (a.H / a.G);
    const int c0 = blockIdx.x * CW;
    const int n = live_tokens(a, b);
    const size_t sbase = ((size_t)blockIdx.y * DK) * DV + c0 + cg * 4;
    float4 S[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m)
        S[m] = a.state_in ? *reinterpret_cast<const float4 *>(a.state_in + sbase + (size_t)(rg + RG * m) * DV)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    const T *q = static_cast<const T *>(a.q) + b * a.q_bs + (size_t)g * DK;
    const T *k = static_cast<const T *>(a.k) + b * a.k_bs + (size_t)g * DK;
    const T *v = static_cast<const T *>(a.v) + b * a.v_bs + (size_t)h * DV + c0;
    const Td *dt = static_cast<const Td *>(a.dt) + b * a.dt_bs + h;
    T *o = static_cast<T *>(a.o) + ((size_t)b * a.T * a.H + h) * DV + c0;
    const float A = a.A[h], D = a.D ? a.D[h] : 0.f, bias = a.dt_bias ? a.dt_bias[h] : 0.f;

    for (int t0 = 0; t0 < n; t0 += kStage) {
        const int nt = min(kStage, n - t0);
        for (int e = tid; e < nt * DK; e += kTokThreads) {
            const int t = e / DK, i = e % DK;
            ks[t][i] = to_f32(k[(size_t)(t0 + t) * a.k_ts + i]);
            qs[t][i] = to_f32(q[(size_t)(t0 + t) * a.q_ts + i]);
        }
        for (int e = tid; e < nt * CW; e += kTokThreads) {
            const int t = e / CW, i = e % CW;
            vs[t][i] = to_f32(v[(size_t)(t0 + t) * a.v_ts + i]);
        }
        if (tid < nt) {
            const float d = step_size(to_f32(dt[(size_t)(t0 + tid) * a.dt_ts]) + bias, a.softplus);
            ds[tid] = d;
            as[tid] = expf(d * A);
        }
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            const float al = as[t], d = ds[t];
            const float4 vv = *reinterpret_cast<const float4 *>(&vs[t][cg * 4]);
            const float4 u = make_float4(d * vv.x, d * vv.y, d * vv.z, d * vv.w);
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int m = 0; m < RPT; ++m) {
                const float kr = ks[t][rg + RG * m], qr = qs[t][rg + RG * m];
                S[m].x = fmaf(al, S[m].x, kr * u.x);
                S[m].y = fmaf(al, S[m].y, kr * u.y);
                S[m].z = fmaf(al, S[m].z, kr * u.z);
                S[m].w = fmaf(al, S[m].w, kr * u.w);
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
            float (*pb)[CW] = part[t & 1];
            if ((tid & 31) < NC) *reinterpret_cast<float4 *>(&pb[warp][cg * 4]) = y;
            __syncthreads();
            if (tid < CW) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) s += pb[w][tid];
                o[(size_t)(t0 + t) * a.H * DV + tid] = from_f32<T>(fmaf(D, vs[t][tid], s));
            }
        }
        __syncthreads();   // the staged tokens and partials are free again
    }
    if (a.state_out)
#pragma unroll
        for (int m = 0; m < RPT; ++m)
            *reinterpret_cast<float4 *>(a.state_out + sbase + (size_t)(rg + RG * m) * DV) = S[m];
}

}  // namespace ssm
}  // namespace gdn
