// ssm_cols.cuh -- selective state space scan, token by token with the state in
// registers: calls of a few tokens and fp32 inputs of any length.
//
// The columns of the state are independent, so a warp keeps 8 of them to
// itself: lane (cg, rg) holds four columns and the rows of every 16th group of
// four (group 16 m + rg), two rows to a register pair, and a token is
//   S <- a S + k (d v) ,  y += q S
// three packed operations for two rows and a column.  q and k come from shared
// memory, 16 bytes for four rows of four columns (with one column a lane the
// same reads, four times as many, were the bound: 256 shared-memory cycles a
// token), staged kStages x kTok tokens ahead by bulk copies of whole rows in
// the inputs' own type.  The readout of four tokens and four columns is summed
// over the row groups at once: 15 shuffles leave each lane with one sum.
//
// Bound by the latency of a warp's own chain while each has a scheduler to itself
// (0.21 us a token at d_k = 128: 512 tokens of 16 heads of 128 x 128 114 us), then
// by issue, about 24 + 0.4 d_k instructions a token and warp.  fp32 throughout,
// sums of d_k / 16 terms per lane; decays are the nearest fp32 (with what they leave,
// as for single tokens, each state element costs an operation more: 202 -> 229 us
// for 128 sequences of 24 tokens, 32 heads of 128 x 64).
#pragma once

#include "packed.cuh"
#include "sm100.cuh"
#include "ssm_token.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace ssm {
namespace cols {

using namespace gdn::sm100;

constexpr int kTok = 16;       // tokens of a stage
constexpr int kStages = 4;
constexpr int kMaxWarps = 8;
constexpr unsigned long long kWaitNs = 1000000000ull;   // a wait gives up after 1 s

// Stage: rows of k and q (a token's two behind one another), rows of v, then
// {decay, step size} of the tokens.
template <int DK, typename T>
__host__ __device__ constexpr int stage_bytes(int warps) {
    return kTok * (2 * DK + 8 * warps) * (int)sizeof(T) + kTok * 8;
}
template <int DK, typename T>
constexpr int smem_bytes(int warps) { return kStages * stage_bytes<DK, T>(warps) + 64; }

// Four consecutive elements from shared memory.
__device__ __forceinline__ void load4(const float *p, float2 &a, float2 &b) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    a = make_float2(v.x, v.y);
    b = make_float2(v.z, v.w);
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float2 &a, float2 &b) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    a = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
    b = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}

// grid (DV / (8 warps), B * H), block 32 * warps.
template <int DK, int DV, typename T, typename Td>
__global__ void __launch_bounds__(kMaxWarps * 32)
cols_kernel(const Args a, unsigned int *err)
{
    constexpr int NM = DK / 64;                   // groups of four rows a lane
    extern __shared__ __align__(128) unsigned char smem[];
    const int warps = blockDim.x >> 5, cw = 8 * warps;
    const int tid = threadIdx.x, lane = tid & 31, rg = lane & 15, col = (tid >> 5) * 8 + (lane >> 4) * 4;
    const int b = blockIdx.y / a.H, h = blockIdx.y % a.H, g = h / (a.H / a.G);
    const int c0 = blockIdx.x * cw;
    const int n = live_tokens(a, b);
    const T *q = static_cast<const T *>(a.q) + b * a.q_bs + (size_t)g * DK;
    const T *k = static_cast<const T *>(a.k) + b * a.k_bs + (size_t)g * DK;
    const T *v = static_cast<const T *>(a.v) + b * a.v_bs + (size_t)h * DV + c0;
    const Td *dt = static_cast<const Td *>(a.dt) + b * a.dt_bs + h;
    T *o = static_cast<T *>(a.o) + ((size_t)b * a.T * a.H + h) * DV + c0 + col + (rg & 3);
    const float A = a.A[h], D = a.D ? a.D[h] : 0.f, bias = a.dt_bias ? a.dt_bias[h] : 0.f;
    const size_t sbase = (size_t)blockIdx.y * DK * DV + c0 + col;
    const int sb = stage_bytes<DK, T>(warps), row = 2 * DK;
    const int v_off = kTok * row * (int)sizeof(T), g_off = v_off + kTok * cw * (int)sizeof(T);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * sb);
    if (tid == 0) {
#pragma unroll
        for (int s = 0; s < kStages; ++s) mbar_init(full + s, 1);
        fence_mbar_init();
    }
    __syncthreads();

    // Stage s, by the first warp: one row copy a lane for k and q, one for v.
    // Tokens behind the end become ones that change nothing (decay 1, step 0,
    // zero rows), so that the walk takes whole groups of tokens.
    auto load_dt = [&](int s) {                   // a stage ahead of its use: a long wait for its warp otherwise
        const int t = s * kTok + (lane & (kTok - 1));
        return t < n ? to_f32(dt[(size_t)t * a.dt_ts]) : 0.f;
    };
    float raw = 0.f;
    auto fetch = [&](int s) {
        const int t0 = s * kTok, nt = min(kTok, n - t0);
        if (nt <= 0) return;
        const float x = raw + bias;
        raw = load_dt(s + 1);
        unsigned char *st = smem + (s % kStages) * sb;
        const int t = lane & (kTok - 1), half = lane / kTok;
        T *rowp = reinterpret_cast<T *>(st) + t * row + half * DK;
        T *vp = reinterpret_cast<T *>(st + v_off) + t * cw;
        const uint32_t kb = DK * sizeof(T), vb = cw * sizeof(T);
        if (lane == 0) mbar_arrive_expect_tx(full + s % kStages, nt * (2 * kb + vb));
        __syncwarp();
        if (t < nt) {
            gdn::tc2::bulk_load(rowp, half ? q + (size_t)(t0 + t) * a.q_ts : k + (size_t)(t0 + t) * a.k_ts, kb,
                                full + s % kStages);
            if (half == 0) gdn::tc2::bulk_load(vp, v + (size_t)(t0 + t) * a.v_ts, vb, full + s % kStages);
        } else {
            for (int i = 0; i < DK; ++i) rowp[i] = from_f32<T>(0.f);
            if (half == 0)
                for (int i = 0; i < cw; ++i) vp[i] = from_f32<T>(0.f);
        }
        if (half == 0) {
            const float d = t < nt ? step_size(x, a.softplus) : 0.f;
            reinterpret_cast<float2 *>(st + g_off)[t] = make_float2(decay(d, A), d);
        }
    };
    const int ns = (n + kTok - 1) / kTok;
    if (tid < 32) {
        raw = load_dt(0);
        for (int s = 0; s < kStages - 1; ++s) fetch(s);
    }

    float2 S[NM][2][4];                           // [group][row pair][column]
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const size_t r = sbase + (size_t)(64 * m + 4 * rg + 2 * i) * DV;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (a.state_in) {
                x = *reinterpret_cast<const float4 *>(a.state_in + r);
                y = *reinterpret_cast<const float4 *>(a.state_in + r + DV);
            }
            S[m][i][0] = make_float2(x.x, y.x);
            S[m][i][1] = make_float2(x.y, y.y);
            S[m][i][2] = make_float2(x.z, y.z);
            S[m][i][3] = make_float2(x.w, y.w);
        }

    bool gave_up = false;                         // the same in every thread
    int s = 0;
    for (; s < ns; ++s) {
        const bool there = mbar_wait_ns(full + s % kStages, (s / kStages) & 1, kWaitNs);
        gave_up = __syncthreads_or(!there);       // stage s and its gates are there, stage s - 1 is read
        if (gave_up) break;
        if (tid < 32) fetch(s + kStages - 1);
        const unsigned char *st = smem + (s % kStages) * sb;
        const T *kq = reinterpret_cast<const T *>(st) + 4 * rg;
        const T *vs = reinterpret_cast<const T *>(st + v_off) + col;
        const float2 *gt = reinterpret_cast<const float2 *>(st + g_off);
        const int t0 = s * kTok, nt = min(kTok, n - t0);
#pragma unroll 1
        for (int t = 0; t < nt; t += 4) {
            float y[16];                          // [token][column]
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const T *kt = kq + (t + j) * row, *qt = kt + DK;
                const float2 ad = gt[t + j], al2 = make_float2(ad.x, ad.x);
                float2 v0, v1, u2[4], yy[4];
                load4(vs + (t + j) * cw, v0, v1);
                const float u[4] = {ad.y * v0.x, ad.y * v0.y, ad.y * v1.x, ad.y * v1.y};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    u2[c] = make_float2(u[c], u[c]);
                    yy[c] = make_float2(0.f, 0.f);
                }
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    float2 k0, k1, q0, q1;
                    load4(kt + 64 * m, k0, k1);
                    load4(qt + 64 * m, q0, q1);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        S[m][0][c] = fma2(al2, S[m][0][c], mul2(k0, u2[c]));
                        S[m][1][c] = fma2(al2, S[m][1][c], mul2(k1, u2[c]));
                        yy[c] = fma2(q0, S[m][0][c], yy[c]);
                        yy[c] = fma2(q1, S[m][1][c], yy[c]);
                    }
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) y[4 * j + c] = yy[c].x + yy[c].y;
            }
            // sums over the row groups: lane rg ends with (token t + rg / 4, column rg % 4)
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) {
                const bool up = rg & d;
#pragma unroll
                for (int i = 0; i < d; ++i) {
                    const float got = __shfl_xor_sync(0xffffffffu, up ? y[i] : y[i + d], d);
                    y[i] = (up ? y[i + d] : y[i]) + got;
                }
            }
            const int tt = t + (rg >> 2);
            if (tt < nt)
                o[(size_t)(t0 + tt) * a.H * DV] = from_f32<T>(fmaf(D, to_f32(vs[tt * cw + (rg & 3)]), y[0]));
        }
    }
    if (gave_up) {
        if (tid == 0) atomicAdd(err, 1u);
        // the copies in flight land before shared memory goes
        const int issued = min(ns, s + kStages - 1);
        for (int i = 0; i < kStages; ++i) mbar_drain(full + i, (issued + kStages - 1 - i) / kStages);
        return;
    }
    if (a.state_out)
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const size_t r = sbase + (size_t)(64 * m + 4 * rg + 2 * i) * DV;
                *reinterpret_cast<float4 *>(a.state_out + r) =
                    make_float4(S[m][i][0].x, S[m][i][1].x, S[m][i][2].x, S[m][i][3].x);
                *reinterpret_cast<float4 *>(a.state_out + r + DV) =
                    make_float4(S[m][i][0].y, S[m][i][1].y, S[m][i][2].y, S[m][i][3].y);
            }
}

}  // namespace cols
}  // namespace ssm
}  // namespace gdn
