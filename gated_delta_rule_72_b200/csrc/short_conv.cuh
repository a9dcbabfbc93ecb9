// short_conv.cuh -- short causal convolution over time, one filter per
// channel (depthwise), the inputs' last K-1 rows carried as a state:
//   y[b,t,c] = act(bias[c] + sum_{j<K} w[c,j] x[b, t-(K-1)+j, c])
// with x before token 0 read from the state (zero without one) and act the
// identity or silu(y) = y / (1 + e^-y).
//
// HBM-bound: every x is read once and every y written once; K multiply-adds
// and one silu per element stay below that (two special-function operations
// an element, 16 per SM and cycle, are 0.7 of the time of the bytes at bf16).
// A thread owns V consecutive channels (16 bytes) for a tile of tokens: the
// filter and the K-1 inputs before stay in registers, a row is loaded kBatch
// rows before it is used, so that a thread has kBatch independent 16-byte loads
// in flight all the time, and two channels share a multiply-add.  A tile
// re-reads the K-1 rows before it.  Rows or bases that are not 16-byte aligned,
// and channel counts that are no multiple of V, take the V = 1 form.
// 32,760 x 4,608 bf16, K = 4 with silu: 118 us, 5.1 TB/s (a copy of the same
// bytes takes 98); in the V = 1 form, rows off 16 bytes, 140 us, fp32 214 (195).  Three blocks an SM; with four the filter spills (155 us).  Batches
// of 4 and 6 rows take 125 and 127 us.  The rows of all but the last two batches
// of a tile go without bounds checks (127 us with them).
//
// The state out is written by the threads of the first tile, which are also
// the only readers of the state in: each thread has read its channels' state
// before it writes them, so the state may be updated in place.
#pragma once

#include "packed.cuh"
#include "vecio.cuh"

namespace gdn {
namespace conv {

constexpr int kThreads = 128;
template <int V> constexpr int kBlocks = V == 1 ? 10 : 3;     // per SM
constexpr int kBatch = 8;      // rows loaded ahead

struct Args {
    const void *x;
    size_t x_bs, x_ts;         // strides of the batch and of the tokens, elements
    const float *w, *bias;     // [C, K]; [C] or NULL
    const void *state_in;      // [B, K-1, C] or NULL
    void *state_out;           // [B, K-1, C] or NULL
    void *y;                   // [B, T, C]
    const int *lengths;        // [B] or NULL
    int B, T, C, tile, ntile;  // tile: tokens per thread, a multiple of kBatch
};

// y / (1 + e^-y), the exponential and the reciprocal in their forms without
// denormals (those with them are several instructions each; below y = -87 the
// result is -0 instead of -1e-36 and less).
__device__ __forceinline__ float silu(float y) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return y * r;
}

template <typename T, int K, int V, bool kSilu>
__global__ void __launch_bounds__(kThreads, kBlocks<V>)
conv_kernel(const Args a)
{
    using P = Pack<T, V>;
    using Row = typename P::Raw;
    // thread -> (sequence, tile, channels), channels fastest
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int groups = (a.C + V - 1) / V;
    const long long bt = id / groups;
    const int b = (int)(bt / a.ntile);
    if (b >= a.B) return;
    const int c = (int)(id - bt * groups) * V;
    int n = a.T;
    if (a.lengths) n = min(max(a.lengths[b], 0), a.T);
    const int t0 = (int)(bt - (long long)b * a.ntile) * a.tile;
    if (t0 >= n && t0 > 0) return;
    const T *x = static_cast<const T *>(a.x) + (size_t)b * a.x_bs + c;
    T *y = static_cast<T *>(a.y) + (size_t)b * a.T * a.C + c;

    float w[K][V], bias[V];
    if (V % 4 == 0) {
        // V filters of K taps: V K consecutive floats
        float f[V * K];
        const float4 *wp = reinterpret_cast<const float4 *>(a.w + (size_t)c * K);
#pragma unroll
        for (int i = 0; i < V * K / 4; ++i) *reinterpret_cast<float4 *>(f + 4 * i) = wp[i];
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < K; ++j) w[j][i] = f[i * K + j];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < K; ++j) w[j][i] = a.w[(size_t)(c + i) * K + j];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = a.bias ? a.bias[c + i] : 0.f;
    const int t1 = min(n, t0 + a.tile);
    Row r[kBatch];
#pragma unroll
    for (int m = 0; m < kBatch; ++m)
        if (t0 + m < t1) r[m] = *reinterpret_cast<const Row *>(x + (size_t)(t0 + m) * a.x_ts);
    // the K-1 rows before the tile, oldest first
    float h[K - 1][V];
    if (t0 == 0) {
        Row s[K - 1];
        const T *si = static_cast<const T *>(a.state_in);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            s[j] = P::zero();
            if (si) s[j] = *reinterpret_cast<const Row *>(si + ((size_t)b * (K - 1) + j) * a.C + c);
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) P::unpack(s[j], h[j]);
        if (a.state_out) {
            T *so = static_cast<T *>(a.state_out);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                // position n - (K-1) + j; negative ones are in the state in
                const int p = n - (K - 1) + j;
                Row r;
                if (p >= 0) {
                    r = *reinterpret_cast<const Row *>(x + (size_t)p * a.x_ts);
                } else {
#pragma unroll
                    for (int m = 0; m < K - 1; ++m)
                        if (m == p + K - 1) r = s[m];
                }
                *reinterpret_cast<Row *>(so + ((size_t)b * (K - 1) + j) * a.C + c) = r;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int p = t0 - (K - 1) + j;   // tiles are longer than K-1 rows
            P::unpack(*reinterpret_cast<const Row *>(x + (size_t)p * a.x_ts), h[j]);
        }
    }

    // one row: the sums of the row's inputs and the K-1 before, the activation
    auto row = [&](const Row &in, T *dst) {
        float xi[V], out[V];
        P::unpack(in, xi);
        // two channels an instruction
        if (V % 2 == 0) {
#pragma unroll
            for (int i = 0; i + 1 < V; i += 2) {
                float2 acc = make_float2(bias[i], bias[i + 1]);
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
                    acc = fma2(make_float2(w[j][i], w[j][i + 1]), make_float2(h[j][i], h[j][i + 1]), acc);
                acc = fma2(make_float2(w[K - 1][i], w[K - 1][i + 1]), make_float2(xi[i], xi[i + 1]), acc);
                out[i] = acc.x;
                out[i + 1] = acc.y;
            }
        } else {
            float acc = bias[0];
#pragma unroll
            for (int j = 0; j < K - 1; ++j) acc = fmaf(w[j][0], h[j][0], acc);
            out[0] = fmaf(w[K - 1][0], xi[0], acc);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j + 1 < K - 1; ++j) h[j][i] = h[j + 1][i];
            h[K - 2][i] = xi[i];
            if (kSilu) out[i] = silu(out[i]);
        }
        *reinterpret_cast<Row *>(dst) = P::pack(out);
    };
    int t = t0;
    const T *xp = x + (size_t)(t0 + kBatch) * a.x_ts;      // (only read where the row exists)
    T *yp = y + (size_t)t0 * a.C;
    for (; t + 2 * kBatch <= t1; t += kBatch) {            // batches with a whole batch behind them
#pragma unroll
        for (int m = 0; m < kBatch; ++m) {
            const Row cur = r[m];
            r[m] = *reinterpret_cast<const Row *>(xp);
            xp += a.x_ts;
            row(cur, yp);
            yp += a.C;
        }
    }
#pragma unroll 1
    for (; t < t1; t += kBatch) {
#pragma unroll
        for (int m = 0; m < kBatch; ++m) {
            if (t + m >= t1) break;
            const Row cur = r[m];
            if (t + m + kBatch < t1) r[m] = *reinterpret_cast<const Row *>(xp);
            xp += a.x_ts;
            row(cur, yp);
            yp += a.C;
        }
    }
}

}  // namespace conv
}  // namespace gdn
