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
//   dS = (w V)^T K                        [W x d_k],   w V as three bf16 terms in TMEM
//   o  = P(i, start) R + Y + D v ,   S <- P(end, start) S + dS
// R is scaled where it lies and Y accumulates onto it; S stays in the registers of
// four warps in fp32, a value column a thread, and takes in each chunk's dS there.
//
// Precision.  q, k, v are exact bf16 operands, so G is exact to fp32; M and the
// operand copy of S are rounded once to bf16 (o itself is bf16: the roundings of
// the terms stay at the size of the output's own; o ends 1.2 times as far from
// its exact value as the rounding of o alone puts it).  The state is fp32: its
// update takes the weighted values as three bf16 terms, 24 significant bits, and
// sums 24 products from zero in TMEM, whose accumulators cut off what does not fit
// 24 bits, small terms first, before the registers' addition rounds to nearest: 5e-7 of
// its norm off at most, however long the walk (accumulated in TMEM from chunk to chunk
// every product's cut was one of the whole state: 2e-5 behind 22 chunks of a head
// that never forgets, and growing with their number).  Decays are products
// of factors in (0, 1] only: a row factor (from the start of the row's 32-token
// block) times a column factor (to that start), each a sum of log-decays that
// is summed directly, so nothing over- or underflows that the product does
// not; inside a 32 x 32 diagonal block 2^(c_i - c_j).
//
// What bounds it.  A chunk of 128 columns moves 64 KB of v and o through HBM
// (1,490 cycles of an SM's share at 1.9 GHz), keeps the tensor cores busy for
// about 3,100 cycles (dS, three terms, half of it) and takes 5,600 to 6,600: the products, the
// warps between them and the tiles' latency wait for one another in turn.
// 4 x 16,384 tokens of 32 heads of 128 x 128 take 437 us at 1,965 MHz, 3.1 TB/s, and
// 511 us call upon call, where the power limit (1,000 W) holds the clock at 1,620.
// Left out in turn, with the state still in TMEM (438 us): the products 350, the
// warps' arithmetic 336, both 275; v loaded a chunk earlier, into a slot still in use, 426.
// 128-token chunks of 128 columns are the largest whose G/M, R/Y, dS and
// weighted values fit TMEM's 512 columns; sharing G between two heads of 64
// halves its cost and the q, k traffic.
//
// Long walks are cut into segments that run in parallel: tail_kernel makes
// each segment's own contribution to its final state, walking back from its
// end until the decay has gone to zero, and the walk of segment g starts from
// the decayed sum of the contributions before it.
//
// Warps: 0-3 keep the state, 4 loads and stores (TMA), 5 issues every MMA, 6 and 7
// make the decay tables, 8-11 the weighted values, 12-19 M and the output.
// The state's warps come first because the next chunk waits for them, and release
// what they have read of dS before they write the state's copy (together 515
// us for what took 502).
#pragma once

#include "packed.cuh"
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
// Warps of the walk: 4 for the state, loads and stores, MMA issue, two for decay
// tables (a head each), kCW for the weighted values, kMW for M and the output.
constexpr int kCW = 4, kMW = 8;
constexpr int kThreads = 32 * (8 + kCW + kMW);
constexpr uint32_t kWaitNs = 1000000000u;   // a wait gives up after 1 s
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Decays below 2^-256 are zero in fp32 many times over: per-token log-decays
// are clamped there, which keeps the block sums exact to 2^-10.
constexpr float kMinLog = -256.f;
// Contributions decayed below 2^-100 are dropped at a segment's start.
constexpr float kForgetLog = -100.f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^x - 1 for x in [-1, 0], to fp32: the exponential's series, x ln2 / 1! + ... (the
// twelfth term is 1e-9 of the value; a call of expm1f costs the walk's tables registers).
__device__ __forceinline__ float ex2m1(float x) {
    x *= kLn2;
    float y = 1.f;
#pragma unroll
    for (int i = 11; i > 1; --i) y = fmaf(x * (1.f / i), y, 1.f);
    return x * y;
}
// One lane of a converged warp, in the form that lets the compiler keep MMA
// operands in uniform registers: behind a plain `lane == 0` each MMA cost
// 150-180 cycles to issue, 62 (its execution time at N = 128) behind this.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ uint32_t global_ns_lo() {
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}
// Wait for a phase, for at most kWaitNs; false when it, or another role's, gave up
// (counted once, at the kernel's end).  Short, for it is inlined at every wait: the
// roles of a CTA run different code that shares the instruction cache.
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t ph, volatile int *abort_s) {
    if (mbar_try_wait(bar, ph & 1u)) return true;
    const uint32_t t0 = global_ns_lo();
    while (!mbar_try_wait(bar, ph & 1u))
        if (*abort_s || global_ns_lo() - t0 >= kWaitNs) {
            *abort_s = 1;
            return false;
        }
    return true;
}
// A wait gave up: the products issued by this thread end before shared memory and TMEM go.
__device__ __forceinline__ void drain_products(uint64_t *bar) {
    mma_commit(bar);
    mbar_drain(bar, 1);
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
// Four 8 x 8 blocks of 16-bit values, transposed: lane l gives the address of
// row l % 8 of block l / 8 and gets column l / 4, rows 2 (l % 4) and one more.
__device__ __forceinline__ void ldmatrix_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16 lanes x 16 columns: r[2 i + j] of lane l goes to TMEM lane 8 j + l / 4, column 4 i + l % 4.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// One warp's 32 tokens x 32 value columns of v times the tokens' weights, as
// three terms of 16 TMEM columns (two tokens a column): src is this lane's row
// (token) of the 128B-swizzled tile at the columns' start, w the weights of
// tokens 2 (lane % 4), + 1 of each block of 8.
__device__ __forceinline__ void weigh_block(uint32_t src, uint32_t dst, const float2 (&w)[4]) {
#pragma unroll 1
    for (int l = 0; l < 2; ++l) {    // 16 columns = lanes
        uint32_t x[2][4], t[3][8];
#pragma unroll
        for (int i = 0; i < 2; ++i) ldmatrix_t(src ^ (32 * l + 16 * i), x[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                split3(mul2(unpack_bf16(x[i][k]), w[k]), t[0][2 * k + i], t[1][2 * k + i], t[2][2 * k + i]);
#pragma unroll
        for (int i = 0; i < 3; ++i) tmem_st_16x128b_x4(dst + ((uint32_t)(16 * l) << 16) + 16 * i, t[i]);
    }
    tmem_wait_st();
}

// Decay tables of one chunk and head.  Blocks of 32 tokens; c: log2 decay from
// the block's start to the token (included).
struct Table {
    float cf[192];      // d_j times the decay from token j to the start of block b > 0, at cf_off(b) + j
    float e[kTok];      // c_j - log2 d_j
    float c[kTok];
    float w[kTok];      // d_j P(end, j)
    float pre[4];       // log2 decay from the chunk's start to the block's
    gdn::ssm::Decay dec;   // P(end, start)
    float pad[2];
};
__device__ __forceinline__ int cf_off(int b) { return 16 * b * (b - 1); }   // 0, 32, 96

// Registers a thread of the walk's warp groups, out of the launch's: the state's
// warps hold 128 values of it.
constexpr int kRegsLaunch = 96;
constexpr int kRegsState = 176, kRegsSupport = 56, kRegsWeights = 72, kRegsOutput = 88;
static_assert(kRegsState + kRegsSupport + (kCW / 4) * kRegsWeights + (kMW / 4) * kRegsOutput <=
                  kRegsLaunch * (kThreads / 128), "register shares");
template <int N, bool kInc>
__device__ __forceinline__ void set_registers() {
    if (kInc) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Wait for tmem_ld16; x is not read before it.
__device__ __forceinline__ void tmem_wait_ld16(float (&x)[16]) {
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+f"(x[i]));
}

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
    la = fmaxf(gdn::ssm::log_decay(d, A2), kMinLog);
}

// ---------------------------------------------------------------------------
// The walk
// ---------------------------------------------------------------------------
template <int DK, int W>
struct Smem {
    static constexpr int kXSlot = (W / 64) * 16384;
    static constexpr int kKSlot = (DK / 64) * 16384;
    static constexpr int kX = 0;                              // 2 slots: v, then the output tile
    static constexpr int kK = kX + 2 * kXSlot;                // 2 slots
    static constexpr int kQ = kK + 2 * kKSlot;
    static constexpr int kS = kQ + kKSlot;                    // [W][DK] bf16, blocks of 64 d_k
    static constexpr int kTab = kS + (DK / 64) * W * 128;     // [2][2] tables
    static constexpr int kBar = kTab + 4 * (int)sizeof(Table);
    static constexpr int kCtl = kBar + 256;
    static constexpr int kBytes = kCtl + 32;
    static_assert(kBytes <= 232448, "shared memory budget");
    static_assert(kS % 1024 == 0 && kTab % 16 == 0, "alignment");
};

template <int DK, int DV, int HB>
__global__ void __launch_bounds__(kThreads, 1)
walk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const Params p)
{
    constexpr int W = DV * HB;
    using SM = Smem<DK, W>;
    // TMEM columns: G / M, R / Y, dS (the start state at first), two buffers of three 16-column terms of weighted values
    constexpr uint32_t cG = 0, cY = 128, cS = 256, cW = 384;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_u32(smem);
    if (sbase & 1023u) {
        if (threadIdx.x == 0) atomicAdd(p.err, 1u);
        return;
    }
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SM::kBar);
    uint64_t *x_full = bars;           // [2] v loaded
    uint64_t *k_full = bars + 2;       // [2] k loaded
    uint64_t *k_free = bars + 4;       // [2] dS done with k
    uint64_t *q_full = bars + 6;       // q loaded
    uint64_t *r_done = bars + 7;       // R complete: q and the state's copy are read
    uint64_t *fixed = bars + 8;        // rows behind the end are zero (last chunk)
    uint64_t *g_full = bars + 9;       // G complete
    uint64_t *m_ready = bars + 10;     // M written, R scaled
    uint64_t *y_full = bars + 11;      // Y complete
    uint64_t *y_free = bars + 12;      // Y read out
    uint64_t *y_staged = bars + 13;    // [2] output tile written (a barrier a slot: chunk c + 1 may be done before
                                       // the storing warp looks at chunk c's, chunk c + 2 not)
    uint64_t *s_ready = bars + 15;     // the state's copy written
    uint64_t *wx_ready = bars + 16;    // [2] weighted values written
    uint64_t *wx_free = bars + 18;     // [2] ... and read
    uint64_t *s_full = bars + 20;      // what a chunk adds to the state complete
    uint64_t *tab_full = bars + 21;    // [2] decay tables written
    uint64_t *tab_free = bars + 23;    // [2] ... and read
    uint64_t *drained = bars + 25;     // products complete, when a wait gave up
    uint64_t *ds_free = bars + 26;     // what a chunk adds to the state has been read
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

    auto load_x = [&](int c) {
        uint64_t *bar = &x_full[c & 1];
        mbar_arrive_expect_tx(bar, SM::kXSlot);
#pragma unroll
        for (int x = 0; x < W / 64; ++x)
            tma_load_4d(smem + SM::kX + (c & 1) * SM::kXSlot + x * 16384, &tm_v, bar, h0 * DV + 64 * x,
                        (c0 + c) * kTok, b, 0);
    };
    auto load_k = [&](int c) {
        uint64_t *bar = &k_full[c & 1];
        mbar_arrive_expect_tx(bar, SM::kKSlot);
#pragma unroll
        for (int x = 0; x < DK / 64; ++x)
            tma_load_4d(smem + SM::kK + (c & 1) * SM::kKSlot + x * 16384, &tm_k, bar, grp * DK + 64 * x,
                        (c0 + c) * kTok, b, 0);
    };
    auto load_q = [&](int c) {
        mbar_arrive_expect_tx(q_full, SM::kKSlot);
#pragma unroll
        for (int x = 0; x < DK / 64; ++x)
            tma_load_4d(smem + SM::kQ + x * 16384, &tm_q, q_full, grp * DK + 64 * x, (c0 + c) * kTok, b, 0);
    };
    if (tid == 0) {
        const uint8_t counts[27] = {1, 1, 1, 1, 1, 1, 1, 1, kCW, 1, kMW, 1, kMW, kMW, kMW, 4, 4, 4, 1, 1, 1, HB, HB,
                                    4 + kCW + kMW, 4 + kCW + kMW, 1, 4};
#pragma unroll
        for (int i = 0; i < 27; ++i) mbar_init(bars + i, counts[i]);
        fence_mbar_init();
        *abort_s = 0;
        // the first chunks' tiles, while the start state is gathered
        if (nch > 0) { load_k(0); load_q(0); load_x(0); }
        if (nch > 1) { load_k(1); load_x(1); }
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

    // with segments this grid starts beside the contributions' last blocks: what they wrote is read from here on
    if (p.nseg > 1) asm volatile("griddepcontrol.wait;" ::: "memory");
    // The walk's start state, warps 0-15: 32 TMEM lanes (value columns) x DK/4
    // rows each, every load of a segment's contribution in flight at once.
    if (warp < 16) {
        constexpr int NR = DK / 4;
        const int v = quarter * 32 + lane, r0 = (warp >> 2) * NR;
        const int hv = v / DV < HB ? v / DV : 0, vcol = v % DV;
        const size_t bh = (size_t)(b * p.a.H + h0 + hv);
        float x[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) x[i] = 0.f;
        // contributions of the segments before, latest first, down to the one
        // behind which all has decayed; behind the first, the initial state
        float carry = 0.f;
        for (int g1 = seg; g1 > 0 && carry >= kForgetLog; g1 -= 32) {
            const int g = g1 - 1 - lane;
            const float own = g >= 0 ? p.decs[bh * (p.nseg - 1) + g] : 0.f;
            // decay behind this segment, summed without its own: taking that off again would
            // leave nothing of small decays behind one that forgets all
            float lg = __shfl_up_sync(0xffffffffu, own, 1);
            if (lane == 0) lg = 0.f;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const float y = __shfl_up_sync(0xffffffffu, lg, s);
                if (lane >= s) lg += y;
            }
            const float before = carry + lg;
            const int cnt = __popc(__ballot_sync(0xffffffffu, g >= 0 && before >= kForgetLog));
            for (int k = 0; k < cnt; ++k) {
                const float f = ex2(__shfl_sync(0xffffffffu, before, k));
                const float *src = p.tails + ((bh * (p.nseg - 1) + g1 - 1 - k) * DK + r0) * DV + vcol;
                if (v < W)
#pragma unroll
                    for (int i = 0; i < NR; ++i) x[i] = fmaf(f, src[(size_t)i * DV], x[i]);
            }
            carry = __shfl_sync(0xffffffffu, before + own, 31);
        }
        if (p.init && carry >= kForgetLog && v < W) {
            const float f = ex2(carry), *src = p.init + (bh * DK + r0) * DV + vcol;
#pragma unroll
            for (int i = 0; i < NR; ++i) x[i] = fmaf(f, src[(size_t)i * DV], x[i]);
        }
        if (nch > 0) {
#pragma unroll
            for (int i = 0; i < NR; i += 16) tmem_st16(tmem + lane_base + cS + r0 + i, x + i);
            tmem_wait_st();
        } else if (p.a.state_out && v < W) {          // no tokens: the state passes through
#pragma unroll
            for (int i = 0; i < NR; ++i) p.a.state_out[(bh * DK + r0 + i) * DV + vcol] = x[i];
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    auto wait = [&](uint64_t *bar, uint32_t ph) { return wait_phase(bar, ph, abort_s); };
    auto partial = [&](int c) { return (c0 + c + 1) * kTok > n; };          // chunk with tokens behind the end
    // its rows behind the end are other sequences' memory only when n < T
    auto own_rows = [&](int c) { return partial(c) && n < p.a.T; };

    if (warp >= 4 && warp < 8) {
        set_registers<kRegsSupport, false>();
    }
    if (warp == 4) {
        // ============================ loads and stores ==============================
        if (lane == 0) {
            int nq = min(nch, 1), nk = min(nch, 2), nx = nk;         // loads issued
            for (int c = 0; c < nch; ++c) {
                if (c + 1 < nch) {
                    if (!wait(r_done, c)) break;
                    load_q(c + 1);
                    ++nq;
                }
                if (c + 2 < nch) {
                    if (!wait(&k_free[c & 1], c >> 1)) break;
                    load_k(c + 2);
                    ++nk;
                }
                if (!wait(&y_staged[c & 1], c >> 1)) break;
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
                    ++nx;
                }
            }
            bulk_wait_all();
            if (*abort_s) {        // a wait gave up: the loads land before shared memory goes
                mbar_drain(q_full, nq);
                for (int s = 0; s < 2; ++s) {
                    mbar_drain(&k_full[s], (nk + 1 - s) >> 1);
                    mbar_drain(&x_full[s], (nx + 1 - s) >> 1);
                }
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        // ============================ MMA issue =====================================
        if (elect_one()) {
            constexpr uint32_t idG = idesc(128, 128, 1, 0, 0);
            constexpr uint32_t idR = idesc(128, W, 1, 0, 0);
            constexpr uint32_t idS = idesc(128, DK, 1, 0, 1);
            constexpr uint32_t idY = idesc(128, DV, 1, 0, 1);
            const uint64_t dQ = sdesc_sw128(sbase + SM::kQ), dK = sdesc_sw128(sbase + SM::kK);
            const uint64_t dS = sdesc_sw128(sbase + SM::kS), dKm = sdesc_sw128_mn(sbase + SM::kK, 16384);
            const uint64_t dX = sdesc_sw128_mn(sbase + SM::kX, 16384);
            auto adv = [](uint64_t d, uint32_t bytes) { return d + (uint64_t)(bytes >> 4); };
            uint32_t wph = 0;      // quarters issued
            for (int c = 0; c < nch; ++c) {
                const uint32_t ks = (c & 1) * SM::kKSlot;
                if (!wait(q_full, c) || !wait(&k_full[c & 1], c >> 1)) break;
                if (partial(c) && !wait(fixed, 0)) break;
                if (c > 0 && !wait(y_full, c - 1)) break;                     // M (over G) has been read
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) {
                    const uint32_t o = (k >> 2) * 16384 + (k & 3) * 32;
                    mma_bf16(tmem + cG, adv(dQ, o), adv(dK, ks + o), idG, k > 0);
                }
                mma_commit(g_full);
                if (!wait(ds_free, c)) break;
                // dS, 32 tokens at a time
                bool ok = true;
#pragma unroll 1
                for (int q = 0; q < 4; ++q, ++wph) {
                    // R = Q S, over the output before, once the first product of dS keeps
                    // the tensor cores busy (before it: 453 us on 4 x 16,384 x 32 x 128, so 440)
                    if (q == 1) {
                        if (c > 0 && !(ok = wait(y_free, c - 1))) break;
                        if (!(ok = wait(s_ready, c))) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < DK / 16; ++k)
                            mma_bf16(tmem + cY, adv(dQ, (k >> 2) * 16384 + (k & 3) * 32),
                                     adv(dS, (k >> 2) * (W * 128) + (k & 3) * 32), idR, k > 0);
                        mma_commit(r_done);
                    }
                    if (!(ok = wait(&wx_ready[q & 1], wph >> 1))) break;
                    tc_fence_after();
                    const uint32_t wx = tmem + cW + (q & 1) * 48;
#pragma unroll
                    for (int t = 2; t >= 0; --t)      // the small terms first
#pragma unroll
                        for (int s = 0; s < 2; ++s)
                            mma_bf16_ta(tmem + cS, wx + 16 * t + 8 * s, adv(dKm, ks + (2 * q + s) * 2048), idS,
                                        q + s + (2 - t) > 0);
                    mma_commit(&wx_free[q & 1]);
                }
                if (!ok) break;
                mma_commit(s_full);
                mma_commit(&k_free[c & 1]);
                // Y = scaled R + M V
                if (!wait(m_ready, c)) break;
                tc_fence_after();
                const uint64_t dV = adv(dX, (c & 1) * SM::kXSlot);
#pragma unroll
                for (int h = 0; h < HB; ++h)
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_bf16_ta(tmem + cY + h * DV, tmem + cG + 32 * (s >> 1) + 16 * h + 8 * (s & 1),
                                    adv(dV, h * 16384 + s * 2048), idY, 1);
                mma_commit(y_full);
            }
            if (*abort_s) drain_products(drained);
        }
        __syncwarp();
    } else if (warp == 6 || (HB == 2 && warp == 7)) {
        // ============================ decay tables ==================================
        // A warp for each head (one for both: 157 us, so 140, on 32,760 tokens of
        // 24 heads of 128 x 64).
        const int h = warp - 6;
        const float A2 = p.a.A[h0 + h] * kLog2e;
        const float bias = p.a.dt_bias ? p.a.dt_bias[h0 + h] : 0.f;
        float raw[4];
        auto fetch = [&](int c) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int t = (c0 + c) * kTok + q * 32 + lane;
                raw[q] = t < n ? load_dt(p, b, t, h0 + h) : 0.f;
            }
        };
        if (nch > 0) fetch(0);
        for (int c = 0; c < nch; ++c) {
            float d[4], la[4], suf[4], cc[4], sum[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                gate(p, raw[q] + bias, (c0 + c) * kTok + q * 32 + lane < n, A2, d[q], la[q]);
            if (c + 1 < nch) fetch(c + 1);
            if (c >= 2 && !wait(&tab_free[c & 1], (c >> 1) - 1)) break;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                cc[q] = la[q];
                suf[q] = __shfl_down_sync(0xffffffffu, la[q], 1);
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
                tb.w[q * 32 + lane] = d[q] * ex2(suf[q] + post);
                tb.c[q * 32 + lane] = cc[q];
                tb.e[q * 32 + lane] = cc[q] - __log2f(d[q]);
                float gap = 0.f;
#pragma unroll
                for (int r = q + 1; r < 4; ++r) {
                    tb.cf[cf_off(r) + q * 32 + lane] = d[q] * ex2(suf[q] + gap);
                    gap += sum[r];
                }
                post += sum[q];
            }
            if (lane == 0) {
                tb.pre[0] = 0.f;
                tb.pre[1] = sum[0];
                tb.pre[2] = sum[0] + sum[1];
                tb.pre[3] = sum[0] + sum[1] + sum[2];
                tb.dec = post > -1.f ? gdn::ssm::decay_near_one(ex2m1(post))
                                     : gdn::ssm::Decay{ex2(post), gdn::ssm::kTiny};
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&tab_full[c & 1]);
        }
    } else if (warp >= 8 + kCW) {
        // ============================ M and the output ==============================
        set_registers<kRegsOutput, false>();
        constexpr int NG = kMW / 4;                  // warp groups
        const int u = (warp - 8 - kCW) >> 2;         // tokens 32 u .. of M (and every NG-th block), columns u NCOL ..
        const int row = quarter * 32 + lane;
        constexpr int NCOL = W / NG;
        const int hcol = (u * NCOL) / DV;            // this warp group's head (of HB) in the output
        const float D = p.a.D ? p.a.D[h0 + hcol] : 0.f;
        const uint32_t ycol = tmem + lane_base + cY + u * NCOL;
        const uint32_t o0 = ((u * NCOL) >> 6) * 16384 + swz128(row * 128 + ((u * NCOL) & 63) * 2);
        for (int c = 0; c < nch; ++c) {
            const Table *tb = tabs + (c & 1) * 2;
            if (!wait(&tab_full[c & 1], c >> 1)) break;
            const float rs = ex2(tb[hcol].pre[quarter] + tb[hcol].c[row]);
            if (!wait(g_full, c)) break;
            tc_fence_after();
#pragma unroll 1
            for (int pc = u; pc < 4; pc += NG) {
                const uint32_t gcol = tmem + lane_base + cG + pc * 32;
                float g[32];
                if (pc <= quarter) {
                    tmem_ld16(gcol, g);
                    tmem_ld16(gcol + 16, g + 16);
                    tmem_wait_ld();
                }
#pragma unroll 1
                for (int h = 0; h < HB; ++h) {
                    const float ci = tb[h].c[row];
                    float m[16];                         // packed pairs
                    if (pc < quarter) {
                        const float4 *cf = reinterpret_cast<const float4 *>(tb[h].cf + cf_off(quarter) + pc * 32);
                        const float rf = ex2(ci);
                        const float2 r2 = make_float2(rf, rf);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 f = cf[j];
                            const float2 x = mul2(make_float2(g[4 * j], g[4 * j + 1]), mul2(make_float2(f.x, f.y), r2));
                            const float2 y = mul2(make_float2(g[4 * j + 2], g[4 * j + 3]), mul2(make_float2(f.z, f.w), r2));
                            m[2 * j] = __uint_as_float(pack_bf16(x.x, x.y));
                            m[2 * j + 1] = __uint_as_float(pack_bf16(y.x, y.y));
                        }
                    } else if (pc == quarter) {
                        const float4 *ej = reinterpret_cast<const float4 *>(tb[h].e + pc * 32);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 e = ej[j];
                            const float x0 = 4 * j <= lane ? g[4 * j] * ex2(ci - e.x) : 0.f;
                            const float x1 = 4 * j + 1 <= lane ? g[4 * j + 1] * ex2(ci - e.y) : 0.f;
                            const float x2 = 4 * j + 2 <= lane ? g[4 * j + 2] * ex2(ci - e.z) : 0.f;
                            const float x3 = 4 * j + 3 <= lane ? g[4 * j + 3] * ex2(ci - e.w) : 0.f;
                            m[2 * j] = __uint_as_float(pack_bf16(x0, x1));
                            m[2 * j + 1] = __uint_as_float(pack_bf16(x2, x3));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) m[j] = 0.f;
                    }
                    tmem_st16(gcol + 16 * h, m);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&tab_free[c & 1]);
            // ---- R <- P(i, start) R
            if (!wait(r_done, c)) break;
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < NCOL; k += 16) {
                float r[16];
                tmem_ld16(ycol + k, r);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 x = mul2(make_float2(r[i], r[i + 1]), make_float2(rs, rs));
                    r[i] = x.x;
                    r[i + 1] = x.y;
                }
                tmem_st16(ycol + k, r);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(m_ready);
            // ---- o = Y + D v, over v in its slot
            if (!wait(y_full, c)) break;
            tc_fence_after();
            const bool direct = own_rows(c);
            unsigned char *xs = smem + SM::kX + (c & 1) * SM::kXSlot;
#pragma unroll 1
            for (int k = 0; k < NCOL; k += 16) {
                float y[16];
                tmem_ld16(ycol + k, y);
                uint4 *slot[2] = {reinterpret_cast<uint4 *>(xs + (o0 ^ (2 * k))),
                                  reinterpret_cast<uint4 *>(xs + (o0 ^ (2 * k) ^ 16))};
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
                        w[i] = pack_bf16(fmaf(D, x.x, y[j]), fmaf(D, x.y, y[j + 1]));
                    }
                    const uint4 out = make_uint4(w[0], w[1], w[2], w[3]);
                    if (!direct) {
                        *slot[e] = out;
                    } else {
                        const int t = (c0 + c) * kTok + row;
                        if (t < n)
                            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.a.o) +
                                                       (((size_t)b * p.a.T + t) * p.a.H + h0) * DV + u * NCOL + k +
                                                       8 * e) = out;
                    }
                }
            }
            fence_async_shared();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(y_free);
                mbar_arrive(&y_staged[c & 1]);
            }
        }
    } else if (warp >= 8) {
        // ============================ weighted values ===============================
        // This warp's 32 value columns are its 32 TMEM lanes: the values come out
        // of shared memory transposed (8 x 8 blocks), and the blocks of 8 tokens
        // are 16x128b pieces of the operand.
        set_registers<kRegsWeights, false>();
        constexpr int NG = kCW / 4;
        const int u = (warp - 8) >> 2;               // blocks of 32 tokens u, u + NG, ..
        const int xcol = quarter * 32;
        bool ok = true;
        for (int c = 0; c < nch && ok; ++c) {
            unsigned char *xs = smem + SM::kX + (c & 1) * SM::kXSlot;
            const Table *tb = tabs + (c & 1) * 2;
            if (!wait(&tab_full[c & 1], c >> 1) || !wait(&x_full[c & 1], c >> 1)) break;
            if (partial(c)) {
                // rows behind the end: zero, so that nothing there (NaN too) enters a product
                if (!wait(&k_full[c & 1], c >> 1)) break;
                const int first = n - (c0 + c) * kTok;
                for (int i = (warp - 8) * 32 + lane; i < kTok * 8; i += 32 * kCW) {
                    const int r = i >> 3, ch = (i & 7) * 16;
                    if (r < first) continue;
#pragma unroll
                    for (int x = 0; x < W / 64; ++x)
                        *reinterpret_cast<uint4 *>(xs + x * 16384 + r * 128 + ch) = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int x = 0; x < DK / 64; ++x)
                        *reinterpret_cast<uint4 *>(smem + SM::kK + (c & 1) * SM::kKSlot + x * 16384 + r * 128 + ch) =
                            make_uint4(0, 0, 0, 0);
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(fixed);
                if (!wait(fixed, 0)) break;          // every row is zero before any is read
            }
#pragma unroll 1
            for (int q = u; q < 4; q += NG) {
                const uint32_t use = 2 * c + (q >> 1);   // of buffer q & 1
                const uint32_t dst = tmem + lane_base + cW + (q & 1) * 48;
                if (use >= 1 && !(ok = wait(&wx_free[q & 1], use - 1))) break;
                tc_fence_after();
                if (xcol < W) {
                    const float2 *wt = reinterpret_cast<const float2 *>(tb[xcol / DV].w + q * 32) + (lane & 3);
                    const float2 w[4] = {wt[0], wt[4], wt[8], wt[12]};
                    const uint32_t src =
                        smem_u32(xs) + (xcol >> 6) * 16384 + swz128((q * 32 + lane) * 128 + (xcol & 63) * 2);
                    weigh_block(src, dst, w);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&wx_ready[q & 1]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&tab_free[c & 1]);
        }
    } else if (warp < 4) {
        // ============================ the state =====================================
        // A thread's column of the state stays in its registers; TMEM holds what the
        // chunk before adds to it (at first the start state).
        set_registers<kRegsState, true>();
        const int v = quarter * 32 + lane;           // value column (TMEM lane)
        const bool live = v < W;
        const int hv = v / DV < HB ? v / DV : 0, vcol = v % DV;
        const size_t bh = (size_t)(b * p.a.H + h0 + hv);
        const uint32_t scol = tmem + lane_base + cS;
        const uint32_t sdst = SM::kS;
        float2 S[DK / 2];
        gdn::ssm::Decay dec{0.f, 0.f};               // of the chunk before
#pragma unroll
        for (int i = 0; i < DK / 2; ++i) S[i] = make_float2(0.f, 0.f);
        // S <- P S + dS, 16 rows
        auto add = [&](int k, const float *x) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                S[k / 2 + i] = fma2(dec.a, S[k / 2 + i],
                                    fma2(dec.e, S[k / 2 + i], make_float2(x[2 * i], x[2 * i + 1])));
        };
        for (int c = 0; c < nch; ++c) {
            // ---- the state after chunk c - 1
            if (c > 0 && !wait(s_full, c - 1)) break;
            tc_fence_after();
            float x[2][16];
            tmem_ld16(scol, x[0]);
            tmem_wait_ld16(x[0]);
#pragma unroll
            for (int k = 0; k < DK; k += 16) {
                if (k + 16 < DK) tmem_ld16(scol + k + 16, x[((k >> 4) + 1) & 1]);
                add(k, x[(k >> 4) & 1]);
                if (k + 16 < DK) tmem_wait_ld16(x[((k >> 4) + 1) & 1]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ds_free);
            // ---- its bf16 copy for R
            if (c > 0 && !wait(r_done, c - 1)) break;
            if (live)
#pragma unroll
                for (int k = 0; k < DK; k += 8) {
                    const float2 *y = S + k / 2;
                    *reinterpret_cast<uint4 *>(smem + sdst + (k >> 6) * (W * 128) + swz128(v * 128 + (k & 63) * 2)) =
                        make_uint4(pack_bf16(y[0].x, y[0].y), pack_bf16(y[1].x, y[1].y), pack_bf16(y[2].x, y[2].y),
                                   pack_bf16(y[3].x, y[3].y));
                }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_ready);
            if (!wait(&tab_full[c & 1], c >> 1)) break;
            dec = tabs[(c & 1) * 2 + hv].dec;
            __syncwarp();
            if (lane == 0) mbar_arrive(&tab_free[c & 1]);
        }
        if (last && p.a.state_out && nch > 0 && wait(s_full, nch - 1)) {
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < DK; k += 16) {
                float x[16];
                tmem_ld16(scol + k, x);
                tmem_wait_ld16(x);
                add(k, x);
                if (live)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        p.a.state_out[(bh * DK + k + 2 * i) * DV + vcol] = S[k / 2 + i].x;
                        p.a.state_out[(bh * DK + k + 2 * i + 1) * DV + vcol] = S[k / 2 + i].y;
                    }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_s && tid == 0) atomicAdd(p.err, 1u);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Contributions of the segments to the states after them
// ---------------------------------------------------------------------------
constexpr int kTailStages = 3;
constexpr int kTailBars = 17;              // barriers
constexpr int kTailThreads = 32 * 22;      // 16 warps of weighted values, loads, MMA issue, 4 of weights
constexpr int kMaxSegChunks = 256;         // longest segment (its blocks' decays are kept in shared memory)

template <int DK, int W>
struct TailSmem {
    static constexpr int kStage = (W / 64 + DK / 64) * 16384;   // v, then k
    static constexpr int kW = kTailStages * kStage;              // weights [2][2][128]
    static constexpr int kSum = kW + 4 * kTok * 4;               // log2 decay of each 32-token block [2][4 kMaxSegChunks]
    static constexpr int kBar = kSum + 8 * kMaxSegChunks * 4;
    static constexpr int kCtl = kBar + 8 * kTailBars;
    static constexpr int kBytes = kCtl + 32;
    static_assert(kBytes <= 232448, "shared memory budget");
};

// grid (nseg - 1, B * nhb): segment g of a head block: tails[g] = the state
// after it when it starts from zero, decs[g] = its log2 decay.  Segments without a successor do nothing.  The
// chunks are taken from the last one back, until what is before has decayed
// below kForgetLog; each is summed from zero in TMEM and added in registers (as the
// walk does, and for the same reason), behind the next one's weighted values, so
// that these are made while a chunk is multiplied (between their halves: 152 us for
// what takes 146 of 32,760 tokens of 24 heads of 128 x 64; all chunks in one
// accumulator, with its cuts: 142).  A chunk costs about 1.9 us (three products over k,
// 1,500 cycles of them); 256 chunks of 12 head blocks in 11 segments take 47 us, 49
// where no head forgets.
template <int DK, int DV, int HB>
__global__ void __launch_bounds__(kTailThreads, 1)
tail_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Params p,
            float *__restrict__ tails, float *__restrict__ decs, float *__restrict__ init_copy)
{
    constexpr int W = DV * HB;
    using SM = TailSmem<DK, W>;
    constexpr uint32_t cS = 0, cW = 128;       // TMEM columns: state, two buffers of 4 x 3 x 16
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_u32(smem);
    if (sbase & 1023u) {
        if (threadIdx.x == 0) atomicAdd(p.err, 1u);
        return;
    }
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SM::kBar);
    uint64_t *full = bars;             // [3] v and k loaded
    uint64_t *freed = bars + 3;        // [3] ... and read
    uint64_t *w_full = bars + 6;       // [2] weights written
    uint64_t *w_free = bars + 8;       // [2] ... and read
    uint64_t *wx_ready = bars + 10;    // [2] weighted values written
    uint64_t *wx_free = bars + 12;     // [2] ... and read
    uint64_t *s_full = bars + 14;      // a chunk's sum complete
    uint64_t *s_free = bars + 15;      // ... and read
    uint64_t *drained = bars + 16;     // products complete, when a wait gave up
    uint32_t *tmem_s = reinterpret_cast<uint32_t *>(smem + SM::kCtl);
    volatile int *abort_s = reinterpret_cast<volatile int *>(smem + SM::kCtl + 4);
    float *after_s = reinterpret_cast<float *>(smem + SM::kCtl + 8);     // [2]
    int *steps_s = reinterpret_cast<int *>(smem + SM::kCtl + 16);         // [2]
    float *ws = reinterpret_cast<float *>(smem + SM::kW);
    float *sums = reinterpret_cast<float *>(smem + SM::kSum);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp & 3;
    const int b = blockIdx.y / p.nhb, hb = blockIdx.y % p.nhb, h0 = hb * HB, seg = blockIdx.x;
    const int grp = h0 / (p.a.H / p.a.G);
    const int n = gdn::ssm::live_tokens(p.a, b);
    const int nC = (n + kTok - 1) / kTok;
    const int c0 = seg * p.L, c1 = c0 + p.L;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the walk's blocks may start on free SMs
    if (seg == 0 && init_copy) {
        // the walk's start state, kept from its in-place update
        const size_t base = (size_t)(b * p.a.H + h0) * DK * DV;
        for (int i = tid; i < HB * DK * DV / 4; i += kTailThreads)
            reinterpret_cast<float4 *>(init_copy + base)[i] = reinterpret_cast<const float4 *>(p.a.state_in + base)[i];
    }
    if (c1 >= nC) return;      // the last segment of its sequence, or behind it: whole chunks only from here

    auto load = [&](int i) {   // chunk i from the end
        const int st = i % kTailStages, t0 = (c1 - 1 - i) * kTok;
        unsigned char *dst = smem + st * SM::kStage;
        mbar_arrive_expect_tx(&full[st], SM::kStage);
#pragma unroll
        for (int x = 0; x < W / 64; ++x) tma_load_4d(dst + x * 16384, &tm_v, &full[st], h0 * DV + 64 * x, t0, b, 0);
#pragma unroll
        for (int x = 0; x < DK / 64; ++x)
            tma_load_4d(dst + (W / 64 + x) * 16384, &tm_k, &full[st], grp * DK + 64 * x, t0, b, 0);
    };
    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < kTailBars; ++i)
            mbar_init(bars + i, (i >= 8 && i < 12) || i == 15 ? 16 : (i == 6 || i == 7 ? 4 : 1));
        fence_mbar_init();
        *abort_s = 0;
        load(0);               // the last chunk counts whatever the decays are
    }
    if (warp == 0) {
        tmem_alloc(tmem_s, 512);
        tmem_relinquish();
    }
    // every 32-token block's log2 decay
    float A2[HB], bias[HB];
#pragma unroll
    for (int h = 0; h < HB; ++h) {
        A2[h] = p.a.A[h0 + h] * kLog2e;
        bias[h] = p.a.dt_bias ? p.a.dt_bias[h0 + h] : 0.f;
    }
    const int nb = 4 * p.L;
    constexpr int kNW = kTailThreads / 32, kAhead = 4;        // blocks a warp loads at once
    for (int i0 = warp; i0 < nb; i0 += kNW * kAhead) {
        float x[kAhead][HB];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int h = 0; h < HB; ++h)
                x[k][h] = i0 + k * kNW < nb ? load_dt(p, b, c0 * kTok + (i0 + k * kNW) * 32 + lane, h0 + h) : 0.f;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int h = 0; h < HB; ++h) {
                float d, s;
                gate(p, x[k][h] + bias[h], true, A2[h], d, s);
#pragma unroll
                for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                if (lane == 0 && i0 + k * kNW < nb) sums[h * 4 * kMaxSegChunks + i0 + k * kNW] = s;
            }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    // from the last block back: the decay behind each (in place of its own),
    // and the chunks that are not forgotten at the segment's end
    if (warp < HB) {
        float *sum = sums + warp * 4 * kMaxSegChunks, carry = 0.f;
        int need = 0;
        for (int i = 0; i < nb; i += 32) {
            const int blk = nb - 1 - i - lane;
            const float own = blk >= 0 ? sum[blk] : 0.f;
            float inc = own;
#pragma unroll
            for (int k = 1; k < 32; k <<= 1) {
                const float y = __shfl_up_sync(0xffffffffu, inc, k);
                if (lane >= k) inc += y;
            }
            float ex = __shfl_up_sync(0xffffffffu, inc, 1);
            if (lane == 0) ex = 0.f;
            if (blk >= 0) sum[blk] = carry + ex;
            // a chunk counts while what is behind it has not decayed
            need += __popc(__ballot_sync(0xffffffffu, blk >= 0 && (blk & 3) == 3 && carry + ex >= kForgetLog));
            carry += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) {
            after_s[warp] = carry;
            steps_s[warp] = need;
        }
    }
    __syncthreads();
    const int steps = max(1, max(steps_s[0], steps_s[HB - 1]));   // (the first tile is on its way)
    auto wait = [&](uint64_t *bar, uint32_t ph) { return wait_phase(bar, ph, abort_s); };
    int issued = 1;                                               // loads (known to lane 0 of warp 16)

    if (warp == 16) {
        if (lane == 0) {
            for (int i = 1; i < steps; ++i) {
                if (i >= kTailStages && !wait(&freed[i % kTailStages], i / kTailStages - 1)) break;
                load(i);
                ++issued;
            }
        }
        __syncwarp();
    } else if (warp == 17) {
        if (elect_one()) {
            constexpr uint32_t idS = idesc(128, DK, 1, 0, 1);
            for (int i = 0; i < steps; ++i) {
                const int st = i % kTailStages;
                if (!wait(&full[st], i / kTailStages) || !wait(&wx_ready[i & 1], i >> 1)) break;
                if (i > 0 && !wait(s_free, i - 1)) break;
                tc_fence_after();
                const uint64_t dK = sdesc_sw128_mn(sbase + st * SM::kStage + (W / 64) * 16384, 16384);
                const uint32_t wx = tmem + cW + (i & 1) * 192;
#pragma unroll
                for (int t = 2; t >= 0; --t)      // the small terms first
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_bf16_ta(tmem + cS, wx + (s >> 1) * 48 + t * 16 + (s & 1) * 8, dK + s * 128, idS,
                                    s + (2 - t) > 0);
                mma_commit(&freed[st]);
                mma_commit(&wx_free[i & 1]);
                mma_commit(s_full);
            }
            if (*abort_s) drain_products(drained);
        }
        __syncwarp();
    } else if (warp >= 18) {
        // weights of token block q: d_j times the decay from token j to the segment's end
        const int q = warp - 18;
        float raw[HB];
        auto fetch = [&](int i) {
#pragma unroll
            for (int h = 0; h < HB; ++h) raw[h] = load_dt(p, b, (c1 - 1 - i) * kTok + q * 32 + lane, h0 + h);
        };
        if (steps > 0) fetch(0);
        for (int i = 0; i < steps; ++i) {
            float d[HB], suf[HB];
#pragma unroll
            for (int h = 0; h < HB; ++h) {
                float la;
                gate(p, raw[h] + bias[h], true, A2[h], d[h], la);
                suf[h] = __shfl_down_sync(0xffffffffu, la, 1);
                if (lane == 31) suf[h] = 0.f;
            }
            if (i + 1 < steps) fetch(i + 1);
#pragma unroll
            for (int s = 1; s < 32; s <<= 1)
#pragma unroll
                for (int h = 0; h < HB; ++h) {
                    const float x = __shfl_down_sync(0xffffffffu, suf[h], s);
                    if (lane + s < 32) suf[h] += x;
                }
            if (i >= 2 && !wait(&w_free[i & 1], (i >> 1) - 1)) break;
#pragma unroll
            for (int h = 0; h < HB; ++h)
                ws[((i & 1) * 2 + h) * kTok + q * 32 + lane] =
                    d[h] * ex2(suf[h] + sums[h * 4 * kMaxSegChunks + (p.L - 1 - i) * 4 + q]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&w_full[i & 1]);
        }
    } else {
        // weighted values: token block warp / 4, value columns 32 quarter ..; behind
        // them the sum of the chunk before, a quarter of d_k, onto the registers'
        constexpr int NK = DK / 4;
        const int q = warp >> 2, xcol = quarter * 32;
        float2 acc[NK / 2];
#pragma unroll
        for (int k = 0; k < NK / 2; ++k) acc[k] = make_float2(0.f, 0.f);
        bool ok = true;
        for (int i = 0; i <= steps; ++i) {
            if (i < steps) {
                const int st = i % kTailStages;
                if (!(ok = wait(&w_full[i & 1], i >> 1) && wait(&full[st], i / kTailStages))) break;
                float2 w[4] = {};
                if (xcol < W) {
                    const float2 *wt =
                        reinterpret_cast<const float2 *>(ws + ((i & 1) * 2 + xcol / DV) * kTok + q * 32) + (lane & 3);
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = wt[4 * k];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&w_free[i & 1]);
                if (i >= 2 && !(ok = wait(&wx_free[i & 1], (i >> 1) - 1))) break;
                tc_fence_after();
                if (xcol < W)
                    weigh_block(sbase + st * SM::kStage + (xcol >> 6) * 16384 +
                                    swz128((q * 32 + lane) * 128 + (xcol & 63) * 2),
                                tmem + ((uint32_t)(quarter * 32) << 16) + cW + (i & 1) * 192 + q * 48, w);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&wx_ready[i & 1]);
            }
            if (i > 0) {
                if (!(ok = wait(s_full, i - 1))) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < NK; k += 16) {
                    float x[16];
                    tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + cS + q * NK + k, x);
                    tmem_wait_ld16(x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        acc[k / 2 + j].x += x[2 * j];
                        acc[k / 2 + j].y += x[2 * j + 1];
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free);
            }
        }
        // ---- out
        const int v = quarter * 32 + lane;
        if (ok && v < W) {
            const int hv = v / DV < HB ? v / DV : 0, vcol = v % DV;
            const size_t bh = (size_t)(b * p.a.H + h0 + hv);
            float *dst = tails + ((bh * (p.nseg - 1) + seg) * DK + q * NK) * DV + vcol;
#pragma unroll
            for (int k = 0; k < NK / 2; ++k) {
                dst[(size_t)(2 * k) * DV] = acc[k].x;
                dst[(size_t)(2 * k + 1) * DV] = acc[k].y;
            }
        }
        if (tid < HB) decs[(size_t)(b * p.a.H + h0 + tid) * (p.nseg - 1) + seg] = after_s[tid];
    }
    __syncthreads();
    if (*abort_s && warp == 16 && lane == 0) {
        // a wait gave up: the copies land before shared memory goes
        for (int s = 0; s < kTailStages; ++s) mbar_drain(&full[s], (issued + kTailStages - 1 - s) / kTailStages);
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_s && tid == 0) atomicAdd(p.err, 1u);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace ssmtc
}  // namespace gdn
