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
// HBM-bound: q and k are read once and written once.  A thread keeps one group
// of channels of one token: it makes the group's cos and sin once, in
// registers, and turns that group of every head of q and k (few tokens: of
// every hsplit-th head), kUnroll 16-byte loads in flight and no barrier (with the
// cosines of a block's tokens in shared memory: 96 us for what takes 68).  Rows
// that are not 16-byte aligned, and sizes that are no multiple of the vector,
// take the element-wise form.  32,760 tokens, 12 + 12 heads of 128, bf16: 68 us,
// 6.0 TB/s (off 16 bytes 99 us, fp32 131, 6.1 TB/s); 2 x 4,099 tokens, 24 + 4 heads of 128 with 64 turned, fp32: 45 us, 5.3 TB/s.
#pragma once

#include "vecio.cuh"

namespace gdn {
namespace rope {

constexpr int kThreads = 256;
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
    int T, d, rot, axes, hsplit;
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
// Every hsplit-th head of one tensor (q or k) from h0 on: in, out at this
// thread's token and channels, cs the group's (cos, sin).  Halves: the second
// V channels stand `off` behind the first (two: they exist).  A group behind
// rot is copied by the same accesses, so that a warp of both kinds does not
// take two paths.
template <typename T, int V, bool kInter, int N>
__device__ __forceinline__ void turn_heads(const T *in, T *out, size_t in_hs, size_t out_hs, int h0, int hsplit,
                                           int heads, int off, bool two, bool behind, const float2 (&cs)[N])
{
    using IO = Io<T, V>;
    using Raw = typename IO::Raw;
    in += h0 * in_hs;
    out += h0 * out_hs;
    in_hs *= hsplit;
    out_hs *= hsplit;
    for (int h = h0; h < heads; h += hsplit * kUnroll) {
        Raw x0[kUnroll], x1[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (h + u * hsplit < heads) {
                x0[u] = IO::load(in + u * in_hs);
                if (!kInter && two) x1[u] = IO::load(in + u * in_hs + off);
            }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (h + u * hsplit >= heads) break;
            if (!behind) {
                float y[V], w[V];
                IO::unpack(x0[u], y);
                if (kInter) {
#pragma unroll
                    for (int i = 0; i + 1 < V; i += 2) {
                        const float y0 = y[i], y1 = y[i + 1];
                        y[i] = fmaf(y0, cs[i / 2].x, -y1 * cs[i / 2].y);
                        y[i + 1] = fmaf(y0, cs[i / 2].y, y1 * cs[i / 2].x);
                    }
                } else {
                    IO::unpack(x1[u], w);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float y0 = y[i], y1 = w[i];
                        y[i] = fmaf(y0, cs[i].x, -y1 * cs[i].y);
                        w[i] = fmaf(y0, cs[i].y, y1 * cs[i].x);
                    }
                    x1[u] = IO::pack(w);
                }
                x0[u] = IO::pack(y);
            }
            IO::store(out + u * out_hs, x0[u]);
            if (!kInter && two) IO::store(out + u * out_hs + off, x1[u]);
        }
        in += kUnroll * in_hs;
        out += kUnroll * out_hs;
    }
}

// Groups of V channels (halves: twice V) of a head of d channels.
__host__ __device__ __forceinline__ int rotated_groups(int rot, int V, bool inter) {
    return inter ? rot / V : rot / 2 / V;
}
__host__ __device__ __forceinline__ int copied_groups(int rest, int V, bool inter) {
    const int w = inter ? V : 2 * V;
    return (rest + w - 1) / w;
}

// Threads: groups of channels fastest, then head splits, then tokens.
template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(const Args a)
{
    constexpr int N = kInter ? (V + 1) / 2 : V;       // pairs of a group
    const int pairs = a.rot / 2;
    const int ng = rotated_groups(a.rot, V, kInter);
    const int nc = a.copy ? copied_groups(a.d - a.rot, V, kInter) : 0, nv = ng + nc;
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int per = nv * a.hsplit;
    const long long row = id / per;
    if (row >= a.rows) return;
    const int rest = (int)(id - row * per), h0 = rest / nv, g = rest - h0 * nv;
    const long long b = row / a.T, t = row - b * a.T;
    const bool behind = g >= ng;
    const int e = behind ? a.rot + (g - ng) * V : g * V;
    const T *qi = static_cast<const T *>(a.q.in) + b * a.q.in_bs + t * a.q.in_ts + e;
    T *qo = static_cast<T *>(a.q.out) + b * a.q.out_bs + t * a.q.out_ts + e;
    const T *ki = static_cast<const T *>(a.k.in) + b * a.k.in_bs + t * a.k.in_ts + e;
    T *ko = static_cast<T *>(a.k.out) + b * a.k.out_bs + t * a.k.out_ts + e;
    // the second half of a group (halves); V = 1, 2 groups may end inside d
    const int off = behind ? nc * V : pairs;
    const bool two = !kInter && e + off < a.d;
    if (kInter && V == 2 && behind && e + 1 >= a.d) {      // the last channel of an odd rest
        for (int h = h0; h < a.q.heads; h += a.hsplit) qo[h * a.q.out_hs] = qi[h * a.q.in_hs];
        for (int h = h0; h < a.k.heads; h += a.hsplit) ko[h * a.k.out_hs] = ki[h * a.k.in_hs];
        return;
    }
    float2 cs[N];
    const int j0 = kInter ? e / 2 : e;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (behind) break;
        const int j = j0 + i;
        long long ax = 0;
        if (a.axes > 1) {
            ax = a.freqs[pairs + j];
            ax = ax < 0 ? 0 : (ax >= a.axes ? a.axes - 1 : ax);
        }
        const size_t pi = (size_t)row * a.axes + (size_t)ax;
        const long long p = a.pos64 ? static_cast<const long long *>(a.pos)[pi]
                                    : (long long)static_cast<const int *>(a.pos)[pi];
        const unsigned long long ph = (unsigned long long)p * (unsigned long long)a.freqs[j];
        // the nearest signed 32-bit fraction of a turn
        const int turn = (int)((ph + 0x80000000ull) >> 32);
        float s, c;
        sincospif((float)turn * 0x1p-31f, &s, &c);
        cs[i] = make_float2(c * a.scale, s * a.scale);
    }
    turn_heads<T, V, kInter>(qi, qo, a.q.in_hs, a.q.out_hs, h0, a.hsplit, a.q.heads, off, two, behind, cs);
    if (a.k.heads) turn_heads<T, V, kInter>(ki, ko, a.k.in_hs, a.k.out_hs, h0, a.hsplit, a.k.heads, off, two, behind, cs);
}

}  // namespace rope
}  // namespace gdn
