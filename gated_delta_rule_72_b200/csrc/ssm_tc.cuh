// ssm_tc.cuh -- selective state space scan of bf16 inputs on the tensor cores,
// in chunks of 128 tokens.
//
// With a_t = e^{d_t A} and, inside a chunk, P(i, j) = a_{j+1} ... a_i:
//   o_i   = P(i, start) q_i S_in + sum_{j<=i} P(i, j) d_j (q_i . k_j) v_j
//   S_out = P(end, start) S_in  + sum_j P(end, j) d_j k_j v_j^T
// One CTA walks the chunks of a head block: W = 128 value columns (one head of
// d_v = 128 or two heads of 64 that share q and k; W = 64 when no such pair
// exists).  Per chunk, all tcgen05 with fp32 accumulators in TMEM:
//   G  = Q K^T                            [128 x 128], shared by the heads
//   M  = G * decay * d, lower triangle, bf16, written over G in TMEM
//   R  = Q S                              [128 x W],   S a bf16 copy of the state
//   Y  = M V                              [128 x W],   A operand from TMEM
//   dS = (w V)^T K                        [W x d_k],   w V as three bf16 terms
//   o  = P(i, start) R + Y + D v ,   S <- P(end, start) S + dS  (fp32 registers)
//
// Precision.  q, k, v are exact bf16 operands, so G is exact to fp32; M and the
// operand copy of S are rounded once to bf16 (o itself is bf16: the roundings of
// the terms stay at the size of the output's own).  The state is fp32: its
// update takes the weighted values as three bf16 terms (24 significant bits).  Decays
// are products of factors in (0, 1] only: a row factor (from the start of the
// row's 32-token block) times a column factor (to that start), each a sum of
// log-decays that is summed directly, so nothing over- or underflows that the
// product does not; inside a 32 x 32 diagonal block 2^(c_i - c_j).
//
// Bound by shared-memory bandwidth (operand reads and writes), then HBM: a
// chunk of 128 columns moves 64 KB of v and o through HBM (1,490 cycles of an
// SM's share at 1.9 GHz) and about 580 KB through shared memory (4,500 cycles
// at 128 B).  128-token chunks of 128 columns are the largest whose G/M, R, Y
// and dS fit TMEM's 512 columns; sharing G between two heads of 64 halves its
// cost and the q, k traffic.
//
// Long walks are cut into segments that run in parallel: tail_kernel makes
// each segment's own contribution to its final state, walking back from its
// end until the decay has gone to zero, and the walk of segment g starts from
// the decayed sum of the contributions before it.
//
// Warps: 0 loads and stores (TMA), 1 issues every MMA, 2 makes the decay
// tables, 3-10 make M and the output, 11-18 the weighted values and the state.
#pragma once

#include "sm100.cuh"
#include "ssm_token.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace ssmtc {

using namespace gdn::sm100;
using gdn::tc2::pack_bf16;
using gdn::tc2::sdesc_sw128_mn;
using gdn::tc2::swz128;
using gdn::tc2::unpack_bf16;

constexpr int kTok = 128;                  // tokens per chunk
constexpr int kThreads = 608;              // 19 warps: up to 104 registers a thread
constexpr int kTailThreads = 256;
constexpr unsigned long long kWaitNs = 1000000000ull;   // a wait gives up after 1 s
constexpr float kLog2e = 1.4426950408889634f;
// Decays below 2^-256 are zero in fp32 many times over: per-token log-decays
// are clamped there, which keeps the block sums exact to 2^-10.
constexpr float kMinLog = -256.f;
// Contributions decayed below this are dropped at a segment's start.
constexpr float kForgetLog = -100.f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, r;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 r, a, b;\n\t"
        "mov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
// One lane of a converged warp, in the form that lets the compiler keep MMA
// operands in uniform registers: behind a plain `lane == 0` each MMA cost
// 150-180 cycles to issue, 62 (its execution time at N = 128) behind this.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
// The slow part of a wait: until the phase completes, for at most kWaitNs (the
// clock and the abort flag are read once in 64 polls).  Out of line: the roles
// of a CTA run different code, and what is inlined at every wait pushes the
// others out of the instruction cache.
static __device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort_s,
                                              unsigned int *err) {
    const unsigned long long t0 = global_ns();
    for (;;) {
        if (mbar_wait(bar, parity, 64)) return true;
        if (*abort_s) return false;
        if (global_ns() - t0 >= kWaitNs) {
            *abort_s = 1;
            atomicAdd(err, 1u);
            return false;
        }
    }
}
// Bounded wait; false when it, or another role's, gave up.
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t ph, volatile int *abort_s, unsigned int *err) {
    return mbar_try_wait(bar, ph & 1u) || wait_slow(bar, ph & 1u, abort_s, err);
}
// D[tmem] (+)= A[tmem] * B[smem]: A is M x 16 bf16, two K elements a column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, r;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "sub.rn.f32x2 r, a, b;\n\t"
        "mov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
// x = hi + mid + lo, three bf16 terms for 24 significant bits: hi and mid are
// cut off (their rest is exact), lo is rounded.
__device__ __forceinline__ void split3(float2 x, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    auto top = [](float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); };
    auto pack = [](float2 v) { return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632); };
    hi = pack(x);
    x = sub2(x, make_float2(top(x.x), top(x.y)));
    mid = pack(x);
    x = sub2(x, make_float2(top(x.x), top(x.y)));
    lo = pack_bf16(x.x, x.y);
}
// Eight bf16 values times w as three terms of 16 bytes.
__device__ __forceinline__ void weigh8(const uint4 &v, float w, uint4 &hi, uint4 &mid, uint4 &lo) {
    const uint32_t *x = reinterpret_cast<const uint32_t *>(&v);
    uint32_t *h = reinterpret_cast<uint32_t *>(&hi), *m = reinterpret_cast<uint32_t *>(&mid),
             *l = reinterpret_cast<uint32_t *>(&lo);
#pragma unroll
    for (int i = 0; i < 4; ++i) split3(mul2(unpack_bf16(x[i]), make_float2(w, w)), h[i], m[i], l[i]);
}

// S += f x, x a column of stride `ld`, eight loads in flight.
template <int N>
__device__ __forceinline__ void add_scaled(float (&S)[N], float f, const float *x, int ld) {
#pragma unroll
    for (int k = 0; k < N; k += 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) S[k + i] = fmaf(f, x[(size_t)(k + i) * ld], S[k + i]);
        asm volatile("" ::: "memory");   // keeps later loads from being hoisted into more registers
    }
}

// Decay tables of one chunk and head.  Blocks of 32 tokens; c: log2 decay from
// the block's start to the token (included).
struct Table {
    float cf[192];      // d_j times the decay from token j to the start of block b > 0, at cf_off(b) + j
    float e[kTok];      // c_j - log2 d_j
    float c[kTok];
    float w[kTok];      // d_j P(end, j)
    float pre[4];       // log2 decay from the chunk's start to the block's
    float dec, pad[3];  // P(end, start)
};
__device__ __forceinline__ int cf_off(int b) { return 16 * b * (b - 1); }   // 0, 32, 96

template <int DK, int W>
struct Smem {
    static constexpr int kXSlot = (W / 64) * 16384;
    static constexpr int kX = 0;                              // 2 slots: v, then the output tile
    static constexpr int kK = kX + 2 * kXSlot;
    static constexpr int kQ = kK + (DK / 64) * 16384;
    static constexpr int kWX = kQ + (DK / 64) * 16384;        // 2 x 3 terms of 32 tokens x 128 columns (8 KB)
    static constexpr int kWXBuf = 3 * 8192;
    static constexpr int kS = kWX + 2 * kWXBuf;               // [W][DK] bf16, blocks of 64 d_k
    static constexpr int kTab = kS + (DK / 64) * W * 128;     // [2][2] tables
    static constexpr int kBar = kTab + 4 * (int)sizeof(Table);
    static constexpr int kCtl = kBar + 256;
    static constexpr int kBytes = kCtl + 32;
    static_assert(kBytes <= 232448, "shared memory budget");
    static_assert(kS % 1024 == 0 && kWX % 1024 == 0 && kTab % 16 == 0, "alignment");
};

struct Params {
    gdn::ssm::Args a;
    int dt_f32;
    int nhb;              // head blocks per sequence
    int nseg, L;          // segments of L chunks
    const float *tails;   // [B * H][nseg - 1] [DK][DV] contributions, or NULL
    const float *decs;    // [B * H][nseg - 1] log2 decay of a segment
    const float *init;    // initial state (a copy when the state is updated in place)
    unsigned int *err;
};

__device__ __forceinline__ float load_dt(const Params &p, int b, int t, int h) {
    const size_t i = (size_t)b * p.a.dt_bs + (size_t)t * p.a.dt_ts + h;
    return p.dt_f32 ? static_cast<const float *>(p.a.dt)[i] : to_f32(static_cast<const __nv_bfloat16 *>(p.a.dt)[i]);
}

// Step size and log2 decay of a token (zero behind the sequence's end).
__device__ __forceinline__ void gate(const Params &p, float x, bool live, float A2, float &d, float &la) {
    d = live ? gdn::ssm::step_size(x, p.a.softplus) : 0.f;
    la = fmaxf(d * A2, kMinLog);
}

// ---------------------------------------------------------------------------
// The walk
// ---------------------------------------------------------------------------
template <int DK, int DV, int HB>
__global__ void __launch_bounds__(kThreads, 1)
walk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const Params p)
{
    constexpr int W = DV * HB;
    using SM = Smem<DK, W>;
    constexpr uint32_t cG = 0, cR = 128, cY = 256, cS = 384;     // TMEM columns
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_u32(smem);
    if (sbase & 1023u) {
        if (threadIdx.x == 0) atomicAdd(p.err, 1u);
        return;
    }
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SM::kBar);
    uint64_t *x_full = bars, *kq_full = bars + 2, *kq_free = bars + 3, *fixed = bars + 4, *g_full = bars + 5,
             *m_ready = bars + 6, *y_full = bars + 7, *y_free = bars + 8, *y_staged = bars + 9, *r_done = bars + 10,
             *s_ready = bars + 11, *wx_ready = bars + 12, *wx_free = bars + 14, *ds_full = bars + 16,
             *ds_free = bars + 17, *tab_full = bars + 18, *tab_free = bars + 20;
    uint32_t *tmem_s = reinterpret_cast<uint32_t *>(smem + SM::kCtl);
    volatile int *abort_s = reinterpret_cast<volatile int *>(smem + SM::kCtl + 4);
    Table *tabs = reinterpret_cast<Table *>(smem + SM::kTab);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp & 3;
    const int b = blockIdx.y / p.nhb, hb = blockIdx.y % p.nhb, h0 = hb * HB;
    const int grp = h0 / (p.a.H / p.a.G);
    const int n = gdn::ssm::live_tokens(p.a, b);
    const int nC = (n + kTok - 1) / kTok;
    const int seg = blockIdx.x, c0 = seg * p.L, c1 = min(nC, c0 + p.L);
    const int nch = c1 - c0;
    // the segment that holds the last token (segment 0 of an empty sequence) writes the final state
    const bool last = nC == 0 ? seg == 0 : (c0 < nC && c1 == nC);
    if (nch <= 0 && !last) return;

    if (tid == 0) {
        mbar_init(&x_full[0], 1);
        mbar_init(&x_full[1], 1);
        mbar_init(kq_full, 1);
        mbar_init(kq_free, 1);
        mbar_init(fixed, 8);
        mbar_init(g_full, 1);
        mbar_init(m_ready, 8);
        mbar_init(y_full, 1);
        mbar_init(y_free, 8);
        mbar_init(y_staged, 8);
        mbar_init(r_done, 1);
        mbar_init(s_ready, 8);
        mbar_init(&wx_ready[0], 4);
        mbar_init(&wx_ready[1], 4);
        mbar_init(&wx_free[0], 1);
        mbar_init(&wx_free[1], 1);
        mbar_init(ds_full, 1);
        mbar_init(ds_free, 8);
        mbar_init(&tab_full[0], 1);
        mbar_init(&tab_full[1], 1);
        mbar_init(&tab_free[0], 16);
        mbar_init(&tab_free[1], 16);
        fence_mbar_init();
        *abort_s = 0;
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_o);
    }
    if (warp == 0) {
        tmem_alloc(tmem_s, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;

    auto wait = [&](uint64_t *bar, uint32_t ph) { return wait_phase(bar, ph, abort_s, p.err); };
    auto partial = [&](int c) { return (c0 + c + 1) * kTok > n; };          // chunk with tokens behind the end
    // its rows behind the end are other sequences' memory only when n < T
    auto own_rows = [&](int c) { return partial(c) && n < p.a.T; };

    if (warp == 0) {
        // ============================ loads and stores ==============================
        if (lane == 0) {
            auto load_x = [&](int c) {
                uint64_t *bar = &x_full[c & 1];
                mbar_arrive_expect_tx(bar, SM::kXSlot);
#pragma unroll
                for (int x = 0; x < W / 64; ++x)
                    tma_load_4d(smem + SM::kX + (c & 1) * SM::kXSlot + x * 16384, &tm_v, bar, h0 * DV + 64 * x,
                                (c0 + c) * kTok, b, 0);
            };
            auto load_kq = [&](int c) {
                mbar_arrive_expect_tx(kq_full, 2 * (DK / 64) * 16384);
#pragma unroll
                for (int x = 0; x < DK / 64; ++x) {
                    tma_load_4d(smem + SM::kK + x * 16384, &tm_k, kq_full, grp * DK + 64 * x, (c0 + c) * kTok, b, 0);
                    tma_load_4d(smem + SM::kQ + x * 16384, &tm_q, kq_full, grp * DK + 64 * x, (c0 + c) * kTok, b, 0);
                }
            };
            if (nch > 0) { load_kq(0); load_x(0); }
            if (nch > 1) load_x(1);
            for (int c = 0; c < nch; ++c) {
                if (c + 1 < nch) {
                    if (!wait(kq_free, c)) break;
                    load_kq(c + 1);
                }
                if (!wait(y_staged, c)) break;
                if (!own_rows(c)) {
#pragma unroll
                    for (int x = 0; x < W / 64; ++x)
                        tma_store_4d(&tm_o, smem + SM::kX + (c & 1) * SM::kXSlot + x * 16384, h0 * DV + 64 * x,
                                     (c0 + c) * kTok, b, 0);
                    bulk_commit_group();
                }
                if (c + 2 < nch) {
                    bulk_wait_read_all();
                    load_x(c + 2);
                }
            }
            bulk_wait_all();
        }
        __syncwarp();
    } else if (warp == 1) {
        // ============================ MMA issue =====================================
        if (elect_one()) {
            constexpr uint32_t idG = idesc(128, 128, 1, 0, 0);
            constexpr uint32_t idR = idesc(128, W, 1, 0, 0);
            constexpr uint32_t idS = idesc(128, DK, 1, 1, 1);
            constexpr uint32_t idY = idesc(128, DV, 1, 0, 1);
            const uint64_t dQ = sdesc_sw128(sbase + SM::kQ), dK = sdesc_sw128(sbase + SM::kK);
            const uint64_t dS = sdesc_sw128(sbase + SM::kS), dKm = sdesc_sw128_mn(sbase + SM::kK, 16384);
            const uint64_t dX = sdesc_sw128_mn(sbase + SM::kX, 16384), dWX = sdesc_sw128_mn(sbase + SM::kWX, 4096);
            auto adv = [](uint64_t d, uint32_t bytes) { return d + (uint64_t)(bytes >> 4); };
            uint32_t wph = 0;      // quarters issued
            for (int c = 0; c < nch; ++c) {
                if (!wait(kq_full, c)) break;
                if (partial(c) && !wait(fixed, 0)) break;
                if (c > 0 && !wait(y_full, c - 1)) break;                     // M (over G) has been read
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) {
                    const uint32_t o = (k >> 2) * 16384 + (k & 3) * 32;
                    mma_bf16(tmem + cG, adv(dQ, o), adv(dK, o), idG, k > 0);
                }
                mma_commit(g_full);
                // R = Q S
                if (!wait(s_ready, c)) break;
                if (c > 0 && !wait(y_free, c - 1)) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)
                    mma_bf16(tmem + cR, adv(dQ, (k >> 2) * 16384 + (k & 3) * 32),
                             adv(dS, (k >> 2) * (W * 128) + (k & 3) * 32), idR, k > 0);
                mma_commit(r_done);
                // dS, 32 tokens at a time
                if (c > 0 && !wait(ds_free, c - 1)) break;
                bool ok = true;
#pragma unroll 1
                for (int q = 0; q < 4; ++q, ++wph) {
                    if (!(ok = wait(&wx_ready[q & 1], wph >> 1))) break;
                    tc_fence_after();
                    const uint64_t wx = adv(dWX, (q & 1) * SM::kWXBuf);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint64_t bk = adv(dKm, (2 * q + s) * 2048);
                        mma_bf16(tmem + cS, adv(wx, s * 2048), bk, idS, q + s > 0);
                        mma_bf16(tmem + cS, adv(wx, 8192 + s * 2048), bk, idS, 1);
                        mma_bf16(tmem + cS, adv(wx, 16384 + s * 2048), bk, idS, 1);
                    }
                    mma_commit(&wx_free[q & 1]);
                }
                if (!ok) break;
                mma_commit(ds_full);
                mma_commit(kq_free);
                // Y = M V
                if (!wait(m_ready, c)) break;
                tc_fence_after();
                const uint64_t dV = adv(dX, (c & 1) * SM::kXSlot);
#pragma unroll
                for (int h = 0; h < HB; ++h)
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_bf16_ta(tmem + cY + h * DV, tmem + cG + 32 * (s >> 1) + 16 * h + 8 * (s & 1),
                                    adv(dV, h * 16384 + s * 2048), idY, s > 0);
                mma_commit(y_full);
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // ============================ decay tables ==================================
        float A2[HB], bias[HB], raw[HB][4];
#pragma unroll
        for (int h = 0; h < HB; ++h) {
            A2[h] = p.a.A[h0 + h] * kLog2e;
            bias[h] = p.a.dt_bias ? p.a.dt_bias[h0 + h] : 0.f;
        }
        auto fetch = [&](int c) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int t = (c0 + c) * kTok + q * 32 + lane;
#pragma unroll
                for (int h = 0; h < HB; ++h) raw[h][q] = t < n ? load_dt(p, b, t, h0 + h) : 0.f;
            }
        };
        if (nch > 0) fetch(0);
        for (int c = 0; c < nch; ++c) {
            float d[HB][4], la[HB][4];
#pragma unroll
            for (int h = 0; h < HB; ++h)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    gate(p, raw[h][q] + bias[h], (c0 + c) * kTok + q * 32 + lane < n, A2[h], d[h][q], la[h][q]);
            if (c + 1 < nch) fetch(c + 1);
            if (c >= 2 && !wait(&tab_free[c & 1], (c >> 1) - 1)) break;
#pragma unroll
            for (int h = 0; h < HB; ++h) {
                float suf[4], cc[4], sum[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    cc[q] = la[h][q];
                    suf[q] = __shfl_down_sync(0xffffffffu, la[h][q], 1);
                    if (lane == 31) suf[q] = 0.f;
                }
#pragma unroll
                for (int s = 1; s < 32; s <<= 1)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float u = __shfl_up_sync(0xffffffffu, cc[q], s);
                        const float v = __shfl_down_sync(0xffffffffu, suf[q], s);
                        if (lane >= s) cc[q] += u;
                        if (lane + s < 32) suf[q] += v;
                    }
#pragma unroll
                for (int q = 0; q < 4; ++q) sum[q] = __shfl_sync(0xffffffffu, cc[q], 31);
                Table &tb = tabs[(c & 1) * 2 + h];
                float post = 0.f;
#pragma unroll
                for (int q = 3; q >= 0; --q) {
                    tb.w[q * 32 + lane] = d[h][q] * ex2(suf[q] + post);
                    tb.c[q * 32 + lane] = cc[q];
                    tb.e[q * 32 + lane] = cc[q] - __log2f(d[h][q]);
                    float gap = 0.f;
#pragma unroll
                    for (int r = q + 1; r < 4; ++r) {
                        tb.cf[cf_off(r) + q * 32 + lane] = d[h][q] * ex2(suf[q] + gap);
                        gap += sum[r];
                    }
                    post += sum[q];
                }
                if (lane == 0) {
                    tb.pre[0] = 0.f;
                    tb.pre[1] = sum[0];
                    tb.pre[2] = sum[0] + sum[1];
                    tb.pre[3] = sum[0] + sum[1] + sum[2];
                    tb.dec = ex2(post);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&tab_full[c & 1]);
        }
    } else if (warp < 11) {
        // ============================ M and the output ==============================
        const int u = (warp - 3) >> 2;               // pieces u, u + 2; columns u W/2 ..
        const int row = quarter * 32 + lane;
        constexpr int NCOL = W / 2;
        const int hcol = (u * NCOL) / DV;            // this warp group's head (of HB) in the output
        const float D = p.a.D ? p.a.D[h0 + hcol] : 0.f;
        for (int c = 0; c < nch; ++c) {
            const Table *tb = tabs + (c & 1) * 2;
            if (!wait(&tab_full[c & 1], c >> 1)) break;
            float ci[HB], rf[HB];
#pragma unroll
            for (int h = 0; h < HB; ++h) {
                ci[h] = tb[h].c[row];
                rf[h] = ex2(ci[h]);
            }
            if (!wait(g_full, c)) break;
            tc_fence_after();
#pragma unroll 1
            for (int pp = 0; pp < 2; ++pp) {
                const int pc = u + 2 * pp;           // 32 tokens j of this piece
                const uint32_t col = tmem + lane_base + cG + pc * 32;
                float g[32];
                if (pc <= quarter) {
                    tmem_ld16(col, g);
                    tmem_ld16(col + 16, g + 16);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int h = 0; h < HB; ++h) {
                    float m[16];                     // packed pairs
                    if (pc < quarter) {
                        const float4 *cf = reinterpret_cast<const float4 *>(tb[h].cf + cf_off(quarter) + pc * 32);
                        const float2 r2 = make_float2(rf[h], rf[h]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 f = cf[j];
                            const float2 x = mul2(make_float2(g[4 * j], g[4 * j + 1]), mul2(make_float2(f.x, f.y), r2));
                            const float2 y =
                                mul2(make_float2(g[4 * j + 2], g[4 * j + 3]), mul2(make_float2(f.z, f.w), r2));
                            m[2 * j] = __uint_as_float(pack_bf16(x.x, x.y));
                            m[2 * j + 1] = __uint_as_float(pack_bf16(y.x, y.y));
                        }
                    } else if (pc == quarter) {
                        const float4 *ej = reinterpret_cast<const float4 *>(tb[h].e + pc * 32);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 e = ej[j];
                            const float x0 = 4 * j <= lane ? g[4 * j] * ex2(ci[h] - e.x) : 0.f;
                            const float x1 = 4 * j + 1 <= lane ? g[4 * j + 1] * ex2(ci[h] - e.y) : 0.f;
                            const float x2 = 4 * j + 2 <= lane ? g[4 * j + 2] * ex2(ci[h] - e.z) : 0.f;
                            const float x3 = 4 * j + 3 <= lane ? g[4 * j + 3] * ex2(ci[h] - e.w) : 0.f;
                            m[2 * j] = __uint_as_float(pack_bf16(x0, x1));
                            m[2 * j + 1] = __uint_as_float(pack_bf16(x2, x3));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) m[j] = 0.f;
                    }
                    tmem_st16(col + 16 * h, m);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(m_ready);
            const float rs = ex2(tb[hcol].pre[quarter] + tb[hcol].c[row]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&tab_free[c & 1]);
            // ---- o = P(i, start) R + Y + D v, over v in its slot
            if (!wait(y_full, c)) break;
            tc_fence_after();
            const bool direct = own_rows(c);
            const int t = (c0 + c) * kTok + row;
            __nv_bfloat16 *orow = static_cast<__nv_bfloat16 *>(p.a.o) +
                                  (((size_t)b * p.a.T + t) * p.a.H + h0) * DV + u * NCOL;
#pragma unroll 1
            for (int k = 0; k < NCOL; k += 16) {
                const int col = u * NCOL + k;
                float r[16], y[16];
                tmem_ld16(tmem + lane_base + cR + col, r);
                tmem_ld16(tmem + lane_base + cY + col, y);
                unsigned char *xs = smem + SM::kX + (c & 1) * SM::kXSlot + (col >> 6) * 16384;
                const uint32_t o0 = swz128(row * 128 + (col & 63) * 2);
                uint4 *slot[2] = {reinterpret_cast<uint4 *>(xs + o0), reinterpret_cast<uint4 *>(xs + (o0 ^ 16))};
                const uint4 v[2] = {*slot[0], *slot[1]};
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t vv[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = unpack_bf16(vv[i]);
                        const int j = 8 * e + 2 * i;
                        w[i] = pack_bf16(fmaf(D, x.x, fmaf(rs, r[j], y[j])), fmaf(D, x.y, fmaf(rs, r[j + 1], y[j + 1])));
                    }
                    const uint4 out = make_uint4(w[0], w[1], w[2], w[3]);
                    if (!direct) *slot[e] = out;
                    else if (t < n) *reinterpret_cast<uint4 *>(orow + k + 8 * e) = out;
                }
            }
            tc_fence_before();
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(y_free);                 // R and Y are read out
                mbar_arrive(y_staged);
            }
        }
    } else {
        // ================= weighted values and the state ============================
        const int u = (warp - 11) >> 2;              // d_k half of the state
        constexpr int NK = DK / 2;
        const int v = quarter * 32 + lane;           // value column of the state (TMEM lane)
        const bool live = v < W;
        const int hv = v / DV < HB ? v / DV : 0, vcol = v % DV;
        const size_t sidx = ((size_t)(b * p.a.H + h0 + hv) * DK + u * NK) * DV + vcol;
        float S[NK];
#pragma unroll
        for (int k = 0; k < NK; ++k) S[k] = 0.f;
        if (live) {
            float f = 1.f;
            int g = seg - 1;
            for (float lg = 0.f; g >= 0; --g) {       // contributions of the segments before, latest first
                const size_t ti = (size_t)(b * p.a.H + h0 + hv) * (p.nseg - 1) + g;
                const float *src = p.tails + (ti * DK + u * NK) * DV + vcol;
                add_scaled<NK>(S, f, src, DV);
                lg += p.decs[ti];
                f = ex2(lg);
                if (lg < kForgetLog) break;
            }
            if (seg == 0 && p.init)                  // (segment 0's contribution holds it for the others)
                add_scaled<NK>(S, f, p.init + sidx, DV);
        }
        auto stage_state = [&]() {
            if (live)
#pragma unroll
                for (int k = 0; k < NK; k += 8) {
                    const int kk = u * NK + k;
                    const uint4 x = make_uint4(pack_bf16(S[k], S[k + 1]), pack_bf16(S[k + 2], S[k + 3]),
                                               pack_bf16(S[k + 4], S[k + 5]), pack_bf16(S[k + 6], S[k + 7]));
                    *reinterpret_cast<uint4 *>(smem + SM::kS + (kk >> 6) * (W * 128) +
                                               swz128(v * 128 + (kk & 63) * 2)) = x;
                }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_ready);
        };
        stage_state();
        const int xcol = quarter * 32;               // this warp's 32 value columns; quarters u and u + 2 of the tokens
        unsigned char *wx = smem + SM::kWX + u * SM::kWXBuf + (xcol >> 6) * 4096;
        uint32_t wph = 0;
        bool ok = true;
        for (int c = 0; c < nch && ok; ++c) {
            unsigned char *xs = smem + SM::kX + (c & 1) * SM::kXSlot;
            const Table *tb = tabs + (c & 1) * 2;
            if (!wait(&tab_full[c & 1], c >> 1) || !wait(&x_full[c & 1], c >> 1)) break;
            if (partial(c)) {
                // rows behind the end: zero, so that nothing there (NaN too) enters a product
                if (!wait(kq_full, c)) break;
                const int first = n - (c0 + c) * kTok;
                for (int i = (warp - 11) * 32 + lane; i < kTok * 8; i += 256) {
                    const int r = i >> 3, ch = (i & 7) * 16;
                    if (r < first) continue;
#pragma unroll
                    for (int x = 0; x < W / 64; ++x)
                        *reinterpret_cast<uint4 *>(xs + x * 16384 + r * 128 + ch) = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int x = 0; x < DK / 64; ++x)
                        *reinterpret_cast<uint4 *>(smem + SM::kK + x * 16384 + r * 128 + ch) = make_uint4(0, 0, 0, 0);
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(fixed);
                if (!wait(fixed, 0)) break;          // every row is zero before any is read
            }
#pragma unroll 1
            for (int q = u; q < 4; q += 2, ++wph) {
                if (wph >= 1 && !(ok = wait(&wx_free[u], wph - 1))) break;
                const int r = q * 32 + lane;
                if (xcol < W) {
                    const float w = tb[xcol / DV].w[r];
#pragma unroll 1
                    for (int e = 0; e < 4; e += 2) {
                        const uint32_t o0 = swz128(lane * 128 + ((xcol & 63) + 8 * e) * 2), o1 = o0 ^ 16;
                        const unsigned char *src = xs + (xcol >> 6) * 16384 + q * 4096;
                        const uint4 x0 = *reinterpret_cast<const uint4 *>(src + o0);
                        const uint4 x1 = *reinterpret_cast<const uint4 *>(src + o1);
                        uint4 t[3];
                        weigh8(x0, w, t[0], t[1], t[2]);
#pragma unroll
                        for (int i = 0; i < 3; ++i) *reinterpret_cast<uint4 *>(wx + o0 + i * 8192) = t[i];
                        weigh8(x1, w, t[0], t[1], t[2]);
#pragma unroll
                        for (int i = 0; i < 3; ++i) *reinterpret_cast<uint4 *>(wx + o1 + i * 8192) = t[i];
                    }
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&wx_ready[u]);
            }
            if (!ok) break;
            const float dec = tb[hv].dec;
            __syncwarp();
            if (lane == 0) mbar_arrive(&tab_free[c & 1]);
            // ---- S <- P(end, start) S + dS
            if (!wait(ds_full, c)) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < NK; k += 16) {
                float x[16];
                tmem_ld16(tmem + lane_base + cS + u * NK + k, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) S[k + i] = fmaf(dec, S[k + i], x[i]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ds_free);
            if (c + 1 < nch) {
                if (!wait(r_done, c)) break;         // Q S has read the copy before
                stage_state();
            }
        }
        if (last && live && p.a.state_out && *abort_s == 0) {
#pragma unroll
            for (int k = 0; k < NK; ++k) p.a.state_out[sidx + (size_t)k * DV] = S[k];
        }
    }

    __syncthreads();
    if (*abort_s && tid == 0) {
        // a wait gave up: let copies and MMAs in flight land before shared memory and TMEM go
        uint64_t *in_flight[] = {&x_full[0], &x_full[1], kq_full, g_full, r_done, ds_full, y_full, kq_free};
        for (uint64_t *bar : in_flight) mbar_wait(bar, 0, 64);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Contributions of the segments to the states after them
// ---------------------------------------------------------------------------
template <int DK, int W>
struct TailSmem {
    static constexpr int kX = 0;                              // v: W/64 blocks
    static constexpr int kK = kX + (W / 64) * 16384;
    static constexpr int kWX = kK + (DK / 64) * 16384;        // 3 terms of 128 tokens x 128 columns each
    static constexpr int kW = kWX + 3 * 32768;                // weights [2][128]
    static constexpr int kRed = kW + 2 * kTok * 4;            // log-decay sums [2 heads][8 warps]
    static constexpr int kBar = kRed + 64;
    static constexpr int kCtl = kBar + 16;
    static constexpr int kBytes = kCtl + 16;
};

// grid (nseg - 1, B * nhb): segment g of a head block: tails[g] = the state
// after it when it starts from zero (segment 0: from the initial state),
// decs[g] = its log2 decay.  Segments without a successor do nothing.
template <int DK, int DV, int HB>
__global__ void __launch_bounds__(kTailThreads, 1)
tail_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Params p,
            float *__restrict__ tails, float *__restrict__ decs, float *__restrict__ init_copy)
{
    constexpr int W = DV * HB;
    using SM = TailSmem<DK, W>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_u32(smem);
    if (sbase & 1023u) {
        if (threadIdx.x == 0) atomicAdd(p.err, 1u);
        return;
    }
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + SM::kBar), *done = full + 1;
    uint32_t *tmem_s = reinterpret_cast<uint32_t *>(smem + SM::kCtl);
    volatile int *abort_s = reinterpret_cast<volatile int *>(smem + SM::kCtl + 4);
    float *ws = reinterpret_cast<float *>(smem + SM::kW);
    float *red = reinterpret_cast<float *>(smem + SM::kRed);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp & 3;
    const int b = blockIdx.y / p.nhb, hb = blockIdx.y % p.nhb, h0 = hb * HB, seg = blockIdx.x;
    const int grp = h0 / (p.a.H / p.a.G);
    const int n = gdn::ssm::live_tokens(p.a, b);
    const int nC = (n + kTok - 1) / kTok;
    const int c0 = seg * p.L, c1 = c0 + p.L;
    if (seg == 0 && init_copy) {
        // the walk's start state, kept from its in-place update
        const size_t base = (size_t)(b * p.a.H + h0) * DK * DV;
        for (int i = tid; i < HB * DK * DV / 4; i += kTailThreads)
            reinterpret_cast<float4 *>(init_copy + base)[i] = reinterpret_cast<const float4 *>(p.a.state_in + base)[i];
    }
    if (c1 >= nC) return;      // the last segment of its sequence, or behind it: whole chunks only from here

    if (tid == 0) {
        mbar_init(full, 1);
        mbar_init(done, 1);
        fence_mbar_init();
        *abort_s = 0;
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    if (warp == 0) {
        tmem_alloc(tmem_s, 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    auto wait = [&](uint64_t *bar, uint32_t ph) { return wait_phase(bar, ph, abort_s, p.err); };
    constexpr uint32_t idS = idesc(128, DK, 1, 1, 1);
    // this thread's token of a chunk, and its head (threads 0-127: the first, 128-255: the second)
    const int hh = tid >> 7, j = tid & 127;
    const bool has = hh < HB;
    const float A2 = has ? p.a.A[h0 + hh] * kLog2e : 0.f;
    const float bias = has && p.a.dt_bias ? p.a.dt_bias[h0 + hh] : 0.f;
    float after[HB];           // log2 decay from the end of the chunk to the end of the segment
#pragma unroll
    for (int h = 0; h < HB; ++h) after[h] = 0.f;
    int steps = 0;
    bool forgot = false;
    for (int c = c1 - 1; c >= c0; --c) {
        float d = 0.f, la = 0.f;
        if (has) gate(p, load_dt(p, b, c * kTok + j, h0 + hh) + bias, true, A2, d, la);   // whole chunks only
        // once everything is forgotten only the segment's decay is of interest: it is zero as well
        if (!forgot) {
            if (tid == 0) {
                mbar_arrive_expect_tx(full, (W / 64 + DK / 64) * 16384);
#pragma unroll
                for (int x = 0; x < W / 64; ++x)
                    tma_load_4d(smem + SM::kX + x * 16384, &tm_v, full, h0 * DV + 64 * x, c * kTok, b, 0);
#pragma unroll
                for (int x = 0; x < DK / 64; ++x)
                    tma_load_4d(smem + SM::kK + x * 16384, &tm_k, full, grp * DK + 64 * x, c * kTok, b, 0);
            }
        }
        // suffix sums of the chunk's log-decays
        float suf = __shfl_down_sync(0xffffffffu, la, 1);
        if (lane == 31) suf = 0.f;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const float x = __shfl_down_sync(0xffffffffu, suf, s);
            if (lane + s < 32) suf += x;
        }
        if (lane == 0) red[warp] = suf + la;
        __syncthreads();
        float post = hh == 0 ? after[0] : after[HB - 1];
        for (int q = quarter + 1; q < 4; ++q) post += red[(warp & 4) + q];
        if (has) ws[tid] = d * ex2(suf + post);
        forgot = true;
#pragma unroll
        for (int h = 0; h < HB; ++h) {
            after[h] += red[4 * h] + red[4 * h + 1] + red[4 * h + 2] + red[4 * h + 3];
            forgot = forgot && after[h] < kForgetLog;
        }
        __syncthreads();
        wait(full, steps);
        // weighted values, hi and lo
        for (int i = tid; i < kTok * (W / 8); i += kTailThreads) {
            const int r = i & 127, cb = i >> 7;          // token, 8-column chunk
            const int col = cb * 8;
            const uint32_t off = (col >> 6) * 16384 + swz128(r * 128 + (col & 63) * 2);
            const uint4 x = *reinterpret_cast<const uint4 *>(smem + SM::kX + off);
            const float w = ws[(col / DV) * 128 + r];
            uint4 t[3];
            weigh8(x, w, t[0], t[1], t[2]);
#pragma unroll
            for (int e = 0; e < 3; ++e) *reinterpret_cast<uint4 *>(smem + SM::kWX + e * 32768 + off) = t[e];
        }
        fence_async_shared();
        __syncthreads();
        if (*abort_s) break;
        if (warp == 0 && elect_one()) {
            tc_fence_after();
            const uint64_t dK = sdesc_sw128_mn(sbase + SM::kK, 16384), dW = sdesc_sw128_mn(sbase + SM::kWX, 16384);
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                mma_bf16(tmem, dW + s * 128, dK + s * 128, idS, steps + s > 0);
                mma_bf16(tmem, dW + 2048 + s * 128, dK + s * 128, idS, 1);
                mma_bf16(tmem, dW + 4096 + s * 128, dK + s * 128, idS, 1);
            }
            mma_commit(done);
        }
        wait(done, steps);
        ++steps;
        __syncthreads();
        if (*abort_s) break;
        if (forgot) {
            // the chunks before it only add to a decay that is zero already
            break;
        }
    }
    if (!*abort_s) {
        tc_fence_after();
        constexpr int NK = DK / 2;
        const int u = warp >> 2, v = quarter * 32 + lane;
        const int hv = v / DV < HB ? v / DV : 0, vcol = v % DV;
        const size_t bh = (size_t)(b * p.a.H + h0 + hv);
        const float f = HB == 2 && hv == 1 ? ex2(after[HB - 1]) : ex2(after[0]);
        const bool add = seg == 0 && p.a.state_in && v < W;
        float *dst = tails + ((bh * (p.nseg - 1) + seg) * DK + u * NK) * DV + vcol;
        const float *src = p.a.state_in ? p.a.state_in + (bh * DK + u * NK) * DV + vcol : nullptr;
#pragma unroll 1
        for (int k = 0; k < NK; k += 16) {
            float x[16];
            tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + u * NK + k, x);
            tmem_wait_ld();
            if (v < W)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    dst[(size_t)(k + i) * DV] = add ? fmaf(f, src[(size_t)(k + i) * DV], x[i]) : x[i];
        }
        if (tid < HB) decs[(size_t)(b * p.a.H + h0 + tid) * (p.nseg - 1) + seg] = tid == 0 ? after[0] : after[HB - 1];
    } else if (tid == 0) {
        mbar_wait(full, 0, 64);
        mbar_wait(done, 0, 64);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 128);
}

}  // namespace ssmtc
}  // namespace gdn
