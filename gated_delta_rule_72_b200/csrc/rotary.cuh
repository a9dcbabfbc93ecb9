// rotary.cuh -- rotary positions: pair j of a head is turned by the angle
// pos * theta_j,
//   (x0, x1) -> scale * (x0 cos - x1 sin, x0 sin + x1 cos),
// pairs (2j, 2j+1) (interleaved) or (j, j + rot/2) (halves) of the first rot
// channels; the channels behind them pass through.
//
// The angle is kept in turns as a 64-bit fixed-point fraction: the table
// holds round(theta_j / 2 pi * 2^64) and the product with the integer
// position wraps modulo one turn exactly, so a position of a million or a
// billion costs no accuracy (fp32 angles are off by 0.06 rad at a million).
// The top 32 bits, as a signed fraction of a turn, give cos and sin.
//
// HBM-bound: q and k are read once and written once.  A block takes `tok`
// tokens: it makes the tokens' cos and sin once in shared memory (they serve
// every head of q and k), then its threads stride over (token, head, vector)
// with 16-byte accesses.  Rows that are not 16-byte aligned, and sizes that
// are no multiple of the vector, take the element-wise form.
#pragma once

#include "common.cuh"

namespace gdn {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxTok = 8;        // tokens per block
constexpr int kMaxRot = 256;      // rotated channels of a head

struct Part {
    const void *in;
    void *out;
    size_t in_bs, in_ts, in_hs, out_bs, out_ts, out_hs;   // elements
    int heads;
};
struct Args {
    Part q, k;
    const void *pos;               // [B, T, axes] int32 or int64
    const long long *freqs;        // [2, rot/2]: phase per position, axis
    float scale;
    long long rows;                // B * T
    int T, d, rot, axes, tok;
    bool pos64, copy;              // copy: the channels behind rot are written too
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec { T e[V]; };

// V elements from p: one vector access, or element by element (kElem).
template <typename T, int V, bool kElem>
__device__ __forceinline__ void load(const T *p, float (&x)[V]) {
    if (kElem) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = to_f32(p[i]);
    } else {
        const Vec<T, V> v = *reinterpret_cast<const Vec<T, V> *>(p);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = to_f32(v.e[i]);
    }
}
template <typename T, int V, bool kElem>
__device__ __forceinline__ void store(T *p, const float (&x)[V]) {
    Vec<T, V> v;
#pragma unroll
    for (int i = 0; i < V; ++i) v.e[i] = from_f32<T>(x[i]);
    if (kElem) {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = v.e[i];
    } else {
        *reinterpret_cast<Vec<T, V> *>(p) = v;
    }
}

template <typename T, int V, bool kInter, bool kElem>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(const Args a)
{
    __shared__ float2 cs[kMaxTok * kMaxRot / 2];
    const int pairs = a.rot / 2;
    const long long row0 = (long long)blockIdx.x * a.tok;
    const int nt = (int)min((long long)a.tok, a.rows - row0);
    for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
        const int t = i / pairs, j = i - t * pairs;
        long long ax = a.freqs[pairs + j];
        ax = ax < 0 ? 0 : (ax >= a.axes ? a.axes - 1 : ax);
        const size_t pi = (size_t)(row0 + t) * a.axes + (size_t)ax;
        const long long p = a.pos64 ? static_cast<const long long *>(a.pos)[pi]
                                    : (long long)static_cast<const int *>(a.pos)[pi];
        const unsigned long long ph = (unsigned long long)p * (unsigned long long)a.freqs[j];
        // the nearest signed 32-bit fraction of a turn
        const int turn = (int)((ph + 0x80000000ull) >> 32);
        float s, c;
        sincospif((float)turn * 0x1p-31f, &s, &c);
        cs[i] = make_float2(c * a.scale, s * a.scale);
    }
    __syncthreads();

    // groups of a head: rotated ones (halves: V channels and their partners),
    // then the channels behind rot
    const int ng = kInter ? a.rot / V : pairs / V;
    const int nv = ng + (a.copy ? (a.d - a.rot + V - 1) / V : 0);
    const int heads = a.q.heads + a.k.heads;
    const int items = nt * heads * nv;
    for (int it = threadIdx.x; it < items; it += kThreads) {
        const int th = it / nv, g = it - th * nv;
        const int t = th / heads;
        int h = th - t * heads;
        const bool isq = h < a.q.heads;
        if (!isq) h -= a.q.heads;
        const Part &P = isq ? a.q : a.k;
        const long long row = row0 + t;
        const long long b = row / a.T, tt = row - b * a.T;
        const T *in = static_cast<const T *>(P.in) + b * P.in_bs + tt * P.in_ts + h * P.in_hs;
        T *out = static_cast<T *>(P.out) + b * P.out_bs + tt * P.out_ts + h * P.out_hs;
        if (g >= ng) {
            const int e = a.rot + (g - ng) * V;
            if (kElem) {
                for (int i = e; i < min(e + V, a.d); ++i) out[i] = in[i];
            } else {
                float x[V];
                load<T, V, kElem>(in + e, x);
                store<T, V, kElem>(out + e, x);
            }
        } else if (kInter) {
            float x[V];
            load<T, V, kElem>(in + g * V, x);
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const float2 z = cs[t * pairs + (g * V + i) / 2];
                const float x0 = x[i], x1 = x[i + 1];
                x[i] = fmaf(x0, z.x, -x1 * z.y);
                x[i + 1] = fmaf(x0, z.y, x1 * z.x);
            }
            store<T, V, kElem>(out + g * V, x);
        } else {
            float x0[V], x1[V];
            load<T, V, kElem>(in + g * V, x0);
            load<T, V, kElem>(in + pairs + g * V, x1);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float2 z = cs[t * pairs + g * V + i];
                const float u = x0[i], w = x1[i];
                x0[i] = fmaf(u, z.x, -w * z.y);
                x1[i] = fmaf(u, z.y, w * z.x);
            }
            store<T, V, kElem>(out + g * V, x0);
            store<T, V, kElem>(out + pairs + g * V, x1);
        }
    }
}

}  // namespace rope
}  // namespace gdn
