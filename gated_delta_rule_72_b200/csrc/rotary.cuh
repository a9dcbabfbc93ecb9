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

#include "vecio.cuh"

namespace gdn {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxTok = 8;        // tokens per block
constexpr int kUnroll = 4;        // heads in flight a thread
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

// V elements: one 16-byte access, or element by element (V = 1 or 2).
template <typename T, int V>
struct Io {
    using Raw = typename Pack<T, V>::Raw;
    static __device__ __forceinline__ Raw load(const T *p) { return *reinterpret_cast<const Raw *>(p); }
    static __device__ __forceinline__ void store(T *p, const Raw &r) { *reinterpret_cast<Raw *>(p) = r; }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[V]) { Pack<T, V>::unpack(r, x); }
    static __device__ __forceinline__ Raw pack(const float (&x)[V]) { return Pack<T, V>::pack(x); }
};
template <typename T>
struct Io<T, 2> {
    struct Raw { T a, b; };
    static __device__ __forceinline__ Raw load(const T *p) { return {p[0], p[1]}; }
    static __device__ __forceinline__ void store(T *p, const Raw &r) { p[0] = r.a; p[1] = r.b; }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[2]) { x[0] = to_f32(r.a); x[1] = to_f32(r.b); }
    static __device__ __forceinline__ Raw pack(const float (&x)[2]) { return {from_f32<T>(x[0]), from_f32<T>(x[1])}; }
};
// N (cos, sin) pairs from shared memory.
template <int N>
__device__ __forceinline__ void load_cs(const float2 *z, float2 (&c)[N]) {
    if (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i + 1 < N; i += 2) {
            const float4 f = *reinterpret_cast<const float4 *>(z + i);
            c[i] = make_float2(f.x, f.y);
            c[i + 1] = make_float2(f.z, f.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = z[i];
    }
}

template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreads, 3)
rotary_kernel(const Args a)
{
    using IO = Io<T, V>;
    using Raw = typename IO::Raw;
    constexpr bool kElem = V <= 2;
    __shared__ __align__(16) float2 cs[kMaxTok * kMaxRot / 2];
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
    // then the channels behind rot.  A thread keeps its group and strides over
    // the (token, head) pairs, kUnroll of them in flight.
    const int ng = kInter ? a.rot / V : pairs / V;
    const int nv = ng + (a.copy ? (a.d - a.rot + V - 1) / V : 0);
    const int heads = a.q.heads + a.k.heads;
    const int slots = nv < kThreads ? kThreads / nv : 1;
    const int slot = threadIdx.x / nv;
    if (slot >= slots) return;
    for (int g = threadIdx.x - slot * nv; g < nv; g += kThreads) {       // (one, unless nv > kThreads)
        const int total = nt * heads;
        int t = slot / heads, h = slot - t * heads;
        for (int it = slot; it < total; it += slots * kUnroll) {
            const T *in[kUnroll];
            T *out[kUnroll];
            int tk[kUnroll];
            Raw x0[kUnroll], x1[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                in[u] = nullptr;
                if (it + u * slots < total) {
                    const bool isq = h < a.q.heads;
                    const Part &P = isq ? a.q : a.k;
                    const int hh = isq ? h : h - a.q.heads;
                    const long long row = row0 + t;
                    const long long b = a.rows == a.T ? 0 : row / a.T, tt = row - b * a.T;
                    in[u] = static_cast<const T *>(P.in) + b * P.in_bs + tt * P.in_ts + hh * P.in_hs;
                    out[u] = static_cast<T *>(P.out) + b * P.out_bs + tt * P.out_ts + hh * P.out_hs;
                    tk[u] = t;
                }
                h += slots;
                while (h >= heads) {
                    h -= heads;
                    ++t;
                }
            }
            if (g >= ng) {
                const int e = a.rot + (g - ng) * V;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    if (!in[u]) continue;
                    if (kElem) {
                        for (int i = e; i < min(e + V, a.d); ++i) out[u][i] = in[u][i];
                    } else {
                        x0[u] = IO::load(in[u] + e);
                    }
                }
                if (!kElem)
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u)
                        if (in[u]) IO::store(out[u] + e, x0[u]);
                continue;
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (in[u]) {
                    x0[u] = IO::load(in[u] + g * V);
                    if (!kInter) x1[u] = IO::load(in[u] + pairs + g * V);
                }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (!in[u]) continue;
                if (kInter) {
                    float2 c[(V + 1) / 2];
                    float y[V];
                    load_cs(cs + tk[u] * pairs + g * V / 2, c);
                    IO::unpack(x0[u], y);
#pragma unroll
                    for (int i = 0; i + 1 < V; i += 2) {
                        const float y0 = y[i], y1 = y[i + 1];
                        y[i] = fmaf(y0, c[i / 2].x, -y1 * c[i / 2].y);
                        y[i + 1] = fmaf(y0, c[i / 2].y, y1 * c[i / 2].x);
                    }
                    x0[u] = IO::pack(y);
                } else {
                    float2 c[V];
                    float y[V], z[V];
                    load_cs(cs + tk[u] * pairs + g * V, c);
                    IO::unpack(x0[u], y);
                    IO::unpack(x1[u], z);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float y0 = y[i], y1 = z[i];
                        y[i] = fmaf(y0, c[i].x, -y1 * c[i].y);
                        z[i] = fmaf(y0, c[i].y, y1 * c[i].x);
                    }
                    x0[u] = IO::pack(y);
                    IO::store(out[u] + pairs + g * V, IO::pack(z));
                }
                IO::store(out[u] + g * V, x0[u]);
            }
        }
    }
}

}  // namespace rope
}  // namespace gdn
