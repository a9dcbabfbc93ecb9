// ssm_chunk.cuh -- selective state space scan of fp32 inputs in chunks of 64
// tokens on the CUDA cores, three launches:
//   state   dS_c = sum_j w_j k_j v_j^T  of every chunk at once,
//           w_j = d_j a_{j+1} ... a_end
//   carry   S_{c+1} = a_c S_c + dS_c over the chunks, one thread for four state
//           elements; each dS_c is replaced by the state S_c the chunk starts from
//   out     o_i = P(i, start) q_i S_c + sum_{j<=i} P(i, j) d_j (q_i . k_j) v_j + D v_i
// so that all but the carry is parallel over the chunks and made of products
// with a register tile a thread (two columns to a packed multiply-add).
//
// fp32 throughout.  Decays P(i, j) inside a chunk are 2^(c_i - c_j) with the
// prefix sums c in 64 bits: in 32 the difference of two sums near 64 would be
// off by 4e-6.  Weights to the end and from the start are sums of their own.
//
// A chunk costs 64 (64 d_k + 64 d_v + 2 d_k d_v) multiply-adds.  Bound by the
// shared-memory reads that feed them (a 16-byte read of a warp takes four cycles
// even where all its lanes want the same) and, with few chunks, by the chain of
// loads and barriers of one block: 5 sequences of up to 777 tokens, 6 heads of
// 64 x 64, 28 us; 2,048 tokens of 24 heads of 128 x 64 110 us.
#pragma once

#include "packed.cuh"
#include "ssm_token.cuh"

namespace gdn {
namespace ssm {
namespace chunk {

constexpr int kTok = 64;
constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinLog = -1024.f;      // a token's log2 decay: far below what fp32 holds

// Rows t0 .. t0 + 63 of a [T, ts] matrix, D columns, into rows of LD floats;
// rows from n on are zero.
template <int D, int LD>
__device__ __forceinline__ void load_rows(float *dst, const float *src, size_t ts, int t0, int n) {
    for (int i = threadIdx.x; i < kTok * (D / 4); i += kThreads) {
        const int t = i / (D / 4), c = (i % (D / 4)) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t0 + t < n) x = *reinterpret_cast<const float4 *>(src + (size_t)(t0 + t) * ts + c);
        *reinterpret_cast<float4 *>(dst + t * LD + c) = x;
    }
}

// Step size and log2 decay of the chunk's token `lane + 32 half` (warps 0, 1).
__device__ __forceinline__ void gate(const Args &a, int b, int h, int t, int n, float &d, float &la) {
    d = 0.f;
    la = 0.f;
    if (t < n) {
        const float bias = a.dt_bias ? a.dt_bias[h] : 0.f;
        d = step_size(static_cast<const float *>(a.dt)[b * a.dt_bs + (size_t)t * a.dt_ts + h] + bias, a.softplus);
        la = fmaxf(log_decay(d, a.A[h]) * kLog2e, kMinLog);
    }
}

template <int DK, int DV>
struct StateSmem {
    static constexpr int kK = 0, kV = kK + kTok * DK, kW = kV + kTok * DV, kFloats = kW + kTok + 4;
};

// grid (chunks, B * H)
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads)
state_kernel(const Args a, float *__restrict__ ds, float *__restrict__ decs, int nc)
{
    using SM = StateSmem<DK, DV>;
    constexpr int TN = DV == 128 ? 8 : 4, TM = DK * DV / kThreads / TN;     // thread tile
    extern __shared__ __align__(16) float sm[];
    const int c = blockIdx.x, b = blockIdx.y / a.H, h = blockIdx.y % a.H, g = h / (a.H / a.G);
    const int n = live_tokens(a, b), t0 = c * kTok, tid = threadIdx.x, lane = tid & 31;
    if (t0 >= n) return;
    float *ks = sm + SM::kK, *vs = sm + SM::kV, *ws = sm + SM::kW;
    if (tid < 64) {
        float d, la;
        gate(a, b, h, t0 + tid, n, d, la);
        float suf = __shfl_down_sync(0xffffffffu, la, 1);
        if (lane == 31) suf = 0.f;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const float x = __shfl_down_sync(0xffffffffu, suf, s);
            if (lane + s < 32) suf += x;
        }
        if (lane == 0) ws[kTok + (tid >> 5)] = suf + la;      // the half's sum
        asm volatile("bar.sync 1, 64;" ::: "memory");
        if (tid < 32) suf += ws[kTok + 1];
        ws[tid] = d * exp2f(suf);
        if (tid == 0) decs[(size_t)blockIdx.y * nc + c] = suf + la;
    }
    load_rows<DK, DK>(ks, static_cast<const float *>(a.k) + b * a.k_bs + (size_t)g * DK, a.k_ts, t0, n);
    __syncthreads();
    // weighted values
    const float *v = static_cast<const float *>(a.v) + b * a.v_bs + (size_t)h * DV;
    for (int i = tid; i < kTok * (DV / 4); i += kThreads) {
        const int t = i / (DV / 4), col = (i % (DV / 4)) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t0 + t < n) x = *reinterpret_cast<const float4 *>(v + (size_t)(t0 + t) * a.v_ts + col);
        const float w = ws[t];
        *reinterpret_cast<float4 *>(vs + t * DV + col) = make_float4(w * x.x, w * x.y, w * x.z, w * x.w);
    }
    __syncthreads();
    const int tx = tid % (DV / TN), ty = tid / (DV / TN);
    float2 acc[TM][TN / 2];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) acc[i][j] = make_float2(0.f, 0.f);
    const float *kp = ks + ty * TM, *vp = vs + tx * 4;
    const int nt = min(kTok, n - t0);
#pragma unroll 4
    for (int t = 0; t < nt; ++t) {
        float kr[TM];
        float2 vr[TN / 2];
#pragma unroll
        for (int i = 0; i < TM; i += 4) *reinterpret_cast<float4 *>(kr + i) = *reinterpret_cast<const float4 *>(kp + t * DK + i);
#pragma unroll
        for (int j = 0; j < TN; j += 4) {          // columns tx 4 .. and (TN = 8) 64 further on
            const float4 x = *reinterpret_cast<const float4 *>(vp + t * DV + j * (DV / TN));
            vr[j / 2] = make_float2(x.x, x.y);
            vr[j / 2 + 1] = make_float2(x.z, x.w);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN / 2; ++j) acc[i][j] = fma2(kr[i], vr[j], acc[i][j]);
    }
    float *dst = ds + ((size_t)blockIdx.y * nc + c) * DK * DV + tx * 4;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; j += 4)
            *reinterpret_cast<float4 *>(dst + (ty * TM + i) * DV + j * (DV / TN)) =
                make_float4(acc[i][j / 2].x, acc[i][j / 2].y, acc[i][j / 2 + 1].x, acc[i][j / 2 + 1].y);
}

// grid (DK * DV / 4 / kThreads, B * H): the chunks' start states, over their dS.
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads)
carry_kernel(const Args a, float *__restrict__ ds, const float *__restrict__ decs, int nc)
{
    const int b = blockIdx.y / a.H, n = live_tokens(a, b), m = (n + kTok - 1) / kTok;
    const int e = blockIdx.x * kThreads + threadIdx.x;
    const size_t sidx = (size_t)blockIdx.y * (DK * DV / 4) + e;
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.state_in) S = reinterpret_cast<const float4 *>(a.state_in)[sidx];
    float4 *p = reinterpret_cast<float4 *>(ds) + (size_t)blockIdx.y * nc * (DK * DV / 4) + e;
    const float *dec = decs + (size_t)blockIdx.y * nc;
    constexpr int kAhead = 8;
    for (int c = 0; c < m; c += kAhead) {
        float4 x[kAhead];
        float f[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (c + i < m) {
                x[i] = p[(size_t)(c + i) * (DK * DV / 4)];
                f[i] = exp2f(dec[c + i]);
            }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (c + i < m) {
                p[(size_t)(c + i) * (DK * DV / 4)] = S;
                S = make_float4(fmaf(f[i], S.x, x[i].x), fmaf(f[i], S.y, x[i].y), fmaf(f[i], S.z, x[i].z),
                                fmaf(f[i], S.w, x[i].w));
            }
    }
    if (a.state_out) reinterpret_cast<float4 *>(a.state_out)[sidx] = S;
}

template <int DK, int DV>
struct OutSmem {
    static constexpr int LQ = DK + 4, LM = kTok + 4;      // padded rows: 16-byte reads of 8 rows spread over the banks
    static constexpr int kQ = 0, kK = kQ + kTok * LQ;
    static constexpr int kKS = kTok * (LQ > DV ? LQ : DV);     // k, then the state 64 rows at a time, then v:
    static constexpr int kM = kK + kKS, kC = kM + kTok * LM;   // one buffer, so that two blocks fit an SM
    static constexpr int kFloats = kC + 2 * kTok + 2 * kTok + 4;              // c (64 bits), d, P(i, start)
};

// grid (chunks, B * H)
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads)
out_kernel(const Args a, const float *__restrict__ starts, int nc)
{
    using SM = OutSmem<DK, DV>;
    constexpr int TN = DV == 128 ? 8 : 4, TM = kTok * DV / kThreads / TN;     // thread tile of the output: 4 rows
    static_assert(TM == 4, "tile");
    extern __shared__ __align__(16) float sm[];
    const int c = blockIdx.x, b = blockIdx.y / a.H, h = blockIdx.y % a.H, g = h / (a.H / a.G);
    const int n = live_tokens(a, b), t0 = c * kTok, tid = threadIdx.x, lane = tid & 31;
    if (t0 >= n) return;
    float *qs = sm + SM::kQ, *ks = sm + SM::kK, *vs = ks, *ms = sm + SM::kM;
    double *cs = reinterpret_cast<double *>(sm + SM::kC);
    float *dsz = sm + SM::kC + 2 * kTok, *es = dsz + kTok, *half = es + kTok;
    if (tid < 64) {
        float d, la;
        gate(a, b, h, t0 + tid, n, d, la);
        double s = la;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, s, k);
            if (lane >= k) s += x;
        }
        if (tid == 31) *reinterpret_cast<double *>(half) = s;
        asm volatile("bar.sync 1, 64;" ::: "memory");
        if (tid >= 32) s += *reinterpret_cast<const double *>(half);
        cs[tid] = s;
        dsz[tid] = d;
        es[tid] = exp2f((float)s);
    }
    load_rows<DK, SM::LQ>(qs, static_cast<const float *>(a.q) + b * a.q_bs + (size_t)g * DK, a.q_ts, t0, n);
    load_rows<DK, SM::LQ>(ks, static_cast<const float *>(a.k) + b * a.k_bs + (size_t)g * DK, a.k_ts, t0, n);
    __syncthreads();
    // ---- M = (Q K^T) * decay * d, rows gy + 16 i, columns gx + 16 j
    {
        const int gx = tid % 16, gy = tid / 16;
        float2 acc[4][4];                          // two partial sums over d_k
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int d = 0; d < DK; d += 4) {
            float4 x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(qs + (gy + 16 * i) * SM::LQ + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(ks + (gx + 16 * j) * SM::LQ + d);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j].x = fmaf(x[i].x, y[j].x, fmaf(x[i].z, y[j].z, acc[i][j].x));
                    acc[i][j].y = fmaf(x[i].y, y[j].y, fmaf(x[i].w, y[j].w, acc[i][j].y));
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = gy + 16 * i, t = gx + 16 * j;
                float m = 0.f;
                if (t <= r) m = (acc[i][j].x + acc[i][j].y) * dsz[t] * exp2f((float)(cs[r] - cs[t]));
                ms[r * SM::LM + t] = m;
            }
    }
    __syncthreads();
    // ---- the output's tile: rows ty 4 .., columns tx 4 .. (and 64 further on)
    const int tx = tid % (DV / TN), ty = tid / (DV / TN), r0 = ty * TM;
    float2 acc[TM][TN / 2];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) acc[i][j] = make_float2(0.f, 0.f);
    auto add = [&](const float *x, int ldx, const float *y, int m) {    // acc += X[rows][m] Y[m][columns]
#pragma unroll 2
        for (int t = 0; t < m; t += 4) {
            float4 xr[TM];
#pragma unroll
            for (int i = 0; i < TM; ++i) xr[i] = *reinterpret_cast<const float4 *>(x + (r0 + i) * ldx + t);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float2 yr[TN / 2];
#pragma unroll
                for (int j = 0; j < TN; j += 4) {
                    const float4 z = *reinterpret_cast<const float4 *>(y + (t + u) * DV + tx * 4 + j * (DV / TN));
                    yr[j / 2] = make_float2(z.x, z.y);
                    yr[j / 2 + 1] = make_float2(z.z, z.w);
                }
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const float s = u == 0 ? xr[i].x : u == 1 ? xr[i].y : u == 2 ? xr[i].z : xr[i].w;
#pragma unroll
                    for (int j = 0; j < TN / 2; ++j) acc[i][j] = fma2(s, yr[j], acc[i][j]);
                }
            }
        }
    };
    // Q S, the state 64 rows at a time over k's place
    const float *S = starts + ((size_t)blockIdx.y * nc + c) * DK * DV;
#pragma unroll 1
    for (int k0 = 0; k0 < DK; k0 += kTok) {
        if (k0) __syncthreads();
        for (int i = tid; i < kTok * DV / 4; i += kThreads)
            reinterpret_cast<float4 *>(ks)[i] = reinterpret_cast<const float4 *>(S + (size_t)k0 * DV)[i];
        __syncthreads();
        add(qs + k0, SM::LQ, ks, kTok);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const float e = es[r0 + i];
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) acc[i][j] = make_float2(e * acc[i][j].x, e * acc[i][j].y);
    }
    __syncthreads();
    load_rows<DV, DV>(vs, static_cast<const float *>(a.v) + b * a.v_bs + (size_t)h * DV, a.v_ts, t0, n);
    __syncthreads();
    add(ms, SM::LM, vs, r0 + TM);                  // (rows up to the tile's last: the rest of M is zero)
    const float D = a.D ? a.D[h] : 0.f;
    float *o = static_cast<float *>(a.o) + (((size_t)b * a.T + t0) * a.H + h) * DV + tx * 4;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        if (t0 + r0 + i >= n) break;
#pragma unroll
        for (int j = 0; j < TN; j += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(vs + (r0 + i) * DV + tx * 4 + j * (DV / TN));
            *reinterpret_cast<float4 *>(o + (size_t)(r0 + i) * a.H * DV + j * (DV / TN)) =
                make_float4(fmaf(D, x.x, acc[i][j / 2].x), fmaf(D, x.y, acc[i][j / 2].y),
                            fmaf(D, x.z, acc[i][j / 2 + 1].x), fmaf(D, x.w, acc[i][j / 2 + 1].y));
        }
    }
}

}  // namespace chunk
}  // namespace ssm
}  // namespace gdn
