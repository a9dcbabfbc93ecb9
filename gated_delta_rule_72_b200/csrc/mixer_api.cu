// mixer_api.cu -- C-ABI entry points of the operators around the gated scan:
// the short causal convolution, rotary positions and the selective state
// space scan (argument checks and kernel dispatch).  See include/gdn.h.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/gdn.h"
#include "common.cuh"
#include "host.cuh"
#include "launch_stats.cuh"
#include "rotary.cuh"
#include "short_conv.cuh"
#include "ssm_chunk.cuh"
#include "ssm_cols.cuh"
#include "ssm_tc.cuh"
#include "ssm_token.cuh"

namespace {

using bf16 = __nv_bfloat16;

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool known(gdn_dtype d) { return d == GDN_F32 || d == GDN_BF16; }
size_t esize(gdn_dtype d) { return d == GDN_F32 ? 4 : 2; }

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const char *p = static_cast<const char *>(a), *q = static_cast<const char *>(b);
    return p && q && na && nb && p < q + nb && q < p + na;
}
// Bytes from the first to behind the last element of a [B, T, H, d] view.
size_t span(int B, size_t bs, int T, size_t ts, int H, size_t hs, size_t d, size_t es) {
    return ((size_t)(B - 1) * bs + (size_t)(T - 1) * ts + (size_t)(H - 1) * hs + d) * es;
}

// A dimension of one entry has no stride of its own: whatever the caller gives
// for it is replaced by the row's width.
void settle(int n, size_t &stride, size_t width) {
    if (n <= 1) stride = width;
}

// A [B, T, H, d] view, strides in elements.
struct View {
    const void *p;
    int B;
    size_t bs;
    int T;
    size_t ts;
    int H;
    size_t hs;
    int d;
    size_t row() const { return (size_t)(H - 1) * hs + d; }
    size_t batch() const { return (size_t)(T - 1) * ts + row(); }
    size_t all() const { return (size_t)(B - 1) * bs + batch(); }
};

// No two elements of a view share memory.
bool distinct(const View &v) {
    size_t n[3] = {(size_t)v.B, (size_t)v.T, (size_t)v.H};
    const size_t st[3] = {v.bs, v.ts, v.hs};
    size_t extent = v.d;
    for (int pass = 0; pass < 3; ++pass) {
        int m = -1;   // the smallest stride left
        for (int i = 0; i < 3; ++i)
            if (n[i] > 1 && (m < 0 || st[i] < st[m])) m = i;
        if (m < 0) break;
        if (st[m] < extent) return false;
        extent += (n[m] - 1) * st[m];
        n[m] = 1;
    }
    return true;
}

// A dimension in which two views step alike, and what the smaller ones span in each.
struct Step {
    long long nx, ny, stride, ext_x, ext_y;
};
// Blocks of two views, `off` elements apart, share an element: for each
// difference of the two indices in the largest dimension at which what lies below may
// meet, look there.
bool blocks_meet(const Step *st, int n, long long off, long long ext_x, long long ext_y) {
    if (off >= ext_x || off + ext_y <= 0) return false;
    if (n == 0) return true;
    const long long p = st->stride;
    long long lo = (-off - st->ext_y) / p - 1, hi = (st->ext_x - off) / p + 1;    // (one more on either side)
    if (lo < -(st->nx - 1)) lo = -(st->nx - 1);
    if (hi > st->ny - 1) hi = st->ny - 1;
    if (hi - lo > 8) return true;                 // views that overlap themselves: not told apart
    for (long long m = lo; m <= hi; ++m)
        if (blocks_meet(st + 1, n - 1, off + m * p, st->ext_x, st->ext_y)) return true;
    return false;
}

// Two views may share memory.  Exact where their strides are the same (one
// tensor's heads, columns or rows, in any order of the dimensions); a dimension in
// which the strides differ counts as one solid block.
bool clash(const View &x, const View &y, size_t es) {
    if (!overlap(x.p, x.all() * es, y.p, y.all() * es)) return false;
    const long long bytes = static_cast<const char *>(y.p) - static_cast<const char *>(x.p);
    if (bytes % (long long)es) return true;
    const int nx[3] = {x.B, x.T, x.H}, ny[3] = {y.B, y.T, y.H};
    const size_t sx[3] = {x.bs, x.ts, x.hs}, sy[3] = {y.bs, y.ts, y.hs};
    Step st[3];
    int n = 0;
    long long ext_x = x.d, ext_y = y.d;
    for (int i = 0; i < 3; ++i) {
        const long long s = (long long)(nx[i] > 1 ? sx[i] : sy[i]);
        if (s == 0 || (nx[i] == 1 && ny[i] == 1)) continue;
        if (nx[i] > 1 && ny[i] > 1 && sx[i] != sy[i]) {
            ext_x += (nx[i] - 1) * (long long)sx[i];
            ext_y += (ny[i] - 1) * (long long)sy[i];
            continue;
        }
        int at = n++;
        for (; at > 0 && st[at - 1].stride < s; --at) st[at] = st[at - 1];
        st[at] = {nx[i], ny[i], s, 0, 0};
    }
    for (int i = n - 1; i >= 0; --i) {
        st[i].ext_x = ext_x;
        st[i].ext_y = ext_y;
        ext_x += (st[i].nx - 1) * st[i].stride;
        ext_y += (st[i].ny - 1) * st[i].stride;
    }
    return blocks_meet(st, n, bytes / (long long)es, ext_x, ext_y);
}

gdn_status launch_status() { return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

constexpr int kMaxTokens = 1 << 30;

// Allow `kern` the dynamic shared memory it needs, once per device.
template <typename K>
bool allow_smem(K *kern, int bytes, std::atomic<unsigned long long> &done) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// A kernel that shares its registers out anew was launched with what the shares
// need: with fewer, the warps that ask for more would wait for good.
template <typename K>
bool has_registers(K *kern, int need, std::atomic<int> &known) {
    int n = known.load(std::memory_order_relaxed);
    if (n == 0) {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, kern) != cudaSuccess) return false;
        known.store(n = at.numRegs, std::memory_order_relaxed);
    }
    return n >= need;
}

// ---------------------------------------------------------------------------
// Short convolution
// ---------------------------------------------------------------------------
template <typename T, int K, int V, bool kSilu>
gdn_status launch_conv(gdn::conv::Args a, int B, cudaStream_t s) {
    using namespace gdn::conv;
    // One wave of threads (kBlocks blocks an SM), each with one tile of tokens:
    // the longest tiles that fill the GPU re-read the fewest rows.
    const long long groups = ((long long)a.C + V - 1) / V * B;
    const long long threads = (long long)gdn::device_sm_count() * kBlocks<V> * kThreads;
    long long tile = (groups * a.T + threads - 1) / threads;
    tile = (tile + kBatch - 1) / kBatch * kBatch;
    if (tile < kBatch) tile = kBatch;
    a.tile = (int)tile;
    a.ntile = a.T > 0 ? (int)((a.T + tile - 1) / tile) : 1;
    const long long blocks = (groups * a.ntile + kThreads - 1) / kThreads;
    gdn::LaunchScope ls("short_conv", s);
    conv_kernel<T, K, V, kSilu><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return launch_status();
}

template <typename T, int K, int V>
gdn_status conv_act(const gdn::conv::Args &a, int B, int silu, cudaStream_t s) {
    return silu ? launch_conv<T, K, V, true>(a, B, s) : launch_conv<T, K, V, false>(a, B, s);
}

template <typename T, int K>
gdn_status conv_vec(const gdn::conv::Args &a, int B, int silu, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = a.C % V == 0 && aligned(a.w, 16) && (a.T == 0 || (aligned(a.x, 16) && a.x_ts % V == 0 && a.x_bs % V == 0));
    return vec ? conv_act<T, K, V>(a, B, silu, s) : conv_act<T, K, 1>(a, B, silu, s);
}

template <typename T>
gdn_status conv_width(const gdn::conv::Args &a, int B, int K, int silu, cudaStream_t s) {
    if (K == 2) return conv_vec<T, 2>(a, B, silu, s);
    if (K == 3) return conv_vec<T, 3>(a, B, silu, s);
    return conv_vec<T, 4>(a, B, silu, s);
}

// ---------------------------------------------------------------------------
// Rotary positions
// ---------------------------------------------------------------------------
template <typename T, int V, bool kInter>
gdn_status launch_rotary(gdn::rope::Args a, cudaStream_t s) {
    using namespace gdn::rope;
    const int nv = rotated_groups(a.rot, V, kInter) + (a.copy ? copied_groups(a.d - a.rot, V, kInter) : 0);
    // split the heads of a token over as many threads as leave four blocks an SM
    const int heads = a.q.heads > a.k.heads ? a.q.heads : a.k.heads;
    const long long want = 4ll * gdn::device_sm_count() * kThreads;
    long long split = want / (a.rows * nv);
    a.hsplit = (int)(split < 1 ? 1 : (split > heads ? heads : split));
    const long long blocks = (a.rows * nv * a.hsplit + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffll) return GDN_ERR_SHAPE;
    gdn::LaunchScope ls("rotary", s);
    rotary_kernel<T, V, kInter><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return launch_status();
}

template <typename T>
gdn_status rotary_type(const gdn::rope::Args &a, int inter, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    bool vec = a.rot % V == 0 && (inter || (a.rot / 2) % V == 0) && (!a.copy || (a.d - a.rot) % (inter ? V : 2 * V) == 0);
    const gdn::rope::Part *ps[2] = {&a.q, &a.k};
    for (const gdn::rope::Part *p : ps)
        if (p->heads) {
            vec = vec && aligned(p->in, 16) && aligned(p->out, 16);
            const size_t st[6] = {p->in_bs, p->in_ts, p->in_hs, p->out_bs, p->out_ts, p->out_hs};
            for (size_t x : st) vec = vec && x % V == 0;
        }
    if (inter) return vec ? launch_rotary<T, V, true>(a, s) : launch_rotary<T, 2, true>(a, s);
    return vec ? launch_rotary<T, V, false>(a, s) : launch_rotary<T, 1, false>(a, s);
}

// ---------------------------------------------------------------------------
// Selective state space scan
// ---------------------------------------------------------------------------
struct Scan {
    gdn::ssm::Args a;
    int dk, dv;
    gdn_dtype t, dt_t;
    cudaStream_t stream;
};

template <int DK, int DV, int CW, typename T, typename Td>
gdn_status launch_token(const Scan &c) {
    gdn::LaunchScope ls("ssm_token", c.stream);
    gdn::ssm::token_kernel<DK, DV, CW, T, Td>
        <<<dim3(DV / CW, c.a.B * c.a.H), gdn::ssm::kTokThreads, 0, c.stream>>>(c.a);
    return launch_status();
}

template <int DK, int DV, typename T, typename Td>
gdn_status token_cols(const Scan &c) {
    // slices of 64 columns when they fill the GPU twice, else of 32
    if ((long long)c.a.B * c.a.H * (DV / 64) >= 2ll * gdn::device_sm_count()) return launch_token<DK, DV, 64, T, Td>(c);
    return launch_token<DK, DV, 32, T, Td>(c);
}

// Several tokens: a warp for every 8 columns, in blocks as large as leave one
// for every SM (the warps of a block share the staged q and k).
template <int DK, int DV, typename T, typename Td>
gdn_status launch_cols(const Scan &c) {
    using namespace gdn::ssm::cols;
    const long long all = (long long)c.a.B * c.a.H * (DV / 8);
    int warps = kMaxWarps;
    while (warps > 1 && all / warps < gdn::device_sm_count()) warps /= 2;
    const int smem = smem_bytes<DK, T>(warps);
    unsigned int *err = gdn::wait_timeout_counter();
    if (!err) return GDN_ERR_CUDA;
    auto kern = cols_kernel<DK, DV, T, Td>;
    static std::atomic<unsigned long long> done;
    if (!allow_smem(kern, smem_bytes<DK, T>(kMaxWarps), done)) return GDN_ERR_CUDA;
    gdn::LaunchScope ls("ssm_cols", c.stream);
    kern<<<dim3(DV / (8 * warps), c.a.B * c.a.H), 32 * warps, smem, c.stream>>>(c.a, err);
    return launch_status();
}

template <int DK, int DV, typename T, typename Td>
gdn_status token_path(const Scan &c) {
    return c.a.T == 1 ? token_cols<DK, DV, T, Td>(c) : launch_cols<DK, DV, T, Td>(c);
}

template <typename T, typename Td>
gdn_status token_dims(const Scan &c) {
    if (c.dk == 128) return c.dv == 128 ? token_path<128, 128, T, Td>(c) : token_path<128, 64, T, Td>(c);
    return c.dv == 128 ? token_path<64, 128, T, Td>(c) : token_path<64, 64, T, Td>(c);
}

// ---------------------------------------------------------------------------
// Tensor-core path of the scan (bf16)
// ---------------------------------------------------------------------------
// Calls of at most this many tokens run token by token.
constexpr int kTokenCall = 32;
// Fewest chunks of a walk that is cut, down to segments of one chunk: with them
// the contributions' launch takes about 5 us and a chunk of the walk 3.0 (16 heads of
// 128 x 128: 3 chunks 16.9 us whole, 20.2 cut; 4 chunks 18.8 and 18.1, where a
// state is updated in place 19.8 and 20.8; 6 chunks 24.7 and 20.0, in place 25.8
// and 22.2; 13 chunks 30.0 in segments of 3, 26.9 of 2).
constexpr int kMinSegmented = 4;
// A segment starts from the sum of the contributions before it (0.6 us each
// where nothing has been forgotten), so more segments shorten the walk up to about
// sqrt(12 chunks) of them: 18,944 tokens of one head that never forgets 49 us in
// 37 segments of 4 chunks, 92 in 148 of one.
constexpr int kSegSquare = 12;

bool use_tc(int T, gdn_dtype t) { return t == GDN_BF16 && T > kTokenCall; }

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// ---------------------------------------------------------------------------
// Chunked path of the scan on the CUDA cores (fp32)
// ---------------------------------------------------------------------------
// In chunks, or token by token with a warp for 8 columns?  From B200 timings:
// the walk takes 0.21 us a token at d_k = 128 (0.18 at 64) while every warp has
// a scheduler of its own (4 an SM), and 0.23 of that more for each further warp
// there; the chunks take 30 us (three launches) and 0.16 us for every block of 64
// tokens x 128 x 64, 0.19 at d_k = 64 (2,048 tokens: 24 heads of 128 x 64 110 us
// against 436; 384 heads of 64 x 64 1,130 us against 717).
bool use_chunks(int B, int T, int H, int dk, int dv, gdn_dtype t) {
    if (t != GDN_F32 || T <= kTokenCall) return false;
    const double warps = (double)B * H * dv / 8, per = warps / (4.0 * gdn::device_sm_count());
    const double walk = T * (dk == 128 ? 0.21 : 0.18) * (per > 1 ? 0.77 + 0.23 * per : 1.0);
    const double blocks = (double)B * H * ((T + 63) / 64) * dk * dv / (128 * 64);
    return 30.0 + (dk == 128 ? 0.16 : 0.19) * blocks < walk;
}

struct ChunkPlan {
    int nc;
    size_t decs, bytes;
};
ChunkPlan plan_chunks(int B, int T, int H, int dk, int dv) {
    ChunkPlan p{};
    p.nc = (T + gdn::ssm::chunk::kTok - 1) / gdn::ssm::chunk::kTok;
    const size_t n = (size_t)B * H * p.nc;
    p.decs = round_up(n * dk * dv * 4, 256);
    p.bytes = p.decs + round_up(n * 4, 256);
    return p;
}

template <int DK, int DV>
gdn_status launch_chunks(const Scan &c, const ChunkPlan &pl, void *ws) {
    using namespace gdn::ssm::chunk;
    float *ds = static_cast<float *>(ws);
    float *decs = reinterpret_cast<float *>(static_cast<char *>(ws) + pl.decs);
    const dim3 grid(pl.nc, c.a.B * c.a.H);
    constexpr int s1 = StateSmem<DK, DV>::kFloats * 4, s3 = OutSmem<DK, DV>::kFloats * 4;
    static_assert(s1 <= 232448 && s3 <= 232448, "shared memory budget");
    static std::atomic<unsigned long long> done1, done3;
    if (!allow_smem(state_kernel<DK, DV>, s1, done1) || !allow_smem(out_kernel<DK, DV>, s3, done3)) return GDN_ERR_CUDA;
    {
        gdn::LaunchScope ls("ssm_chunk_state", c.stream);
        state_kernel<DK, DV><<<grid, kThreads, s1, c.stream>>>(c.a, ds, decs, pl.nc);
    }
    if (launch_status() != GDN_OK) return GDN_ERR_CUDA;
    {
        gdn::LaunchScope ls("ssm_chunk_carry", c.stream);
        carry_kernel<DK, DV><<<dim3(DK * DV / 4 / kThreads, c.a.B * c.a.H), kThreads, 0, c.stream>>>(c.a, ds, decs,
                                                                                                     pl.nc);
    }
    if (launch_status() != GDN_OK) return GDN_ERR_CUDA;
    gdn::LaunchScope ls("ssm_chunk_out", c.stream);
    out_kernel<DK, DV><<<grid, kThreads, s3, c.stream>>>(c.a, ds, pl.nc);
    return launch_status();
}

gdn_status chunk_dims(const Scan &c, const ChunkPlan &pl, void *ws) {
    if (c.dk == 128) return c.dv == 128 ? launch_chunks<128, 128>(c, pl, ws) : launch_chunks<128, 64>(c, pl, ws);
    return c.dv == 128 ? launch_chunks<64, 128>(c, pl, ws) : launch_chunks<64, 64>(c, pl, ws);
}

// Head blocks (128 value columns: two heads of 64 that share a group, else one
// head) and the segments of their walks, the same number for each: as many as
// leave one wave of CTAs where there are fewer head blocks than SMs, else one.  So
// SMs stand idle where the SMs are no multiple of the head blocks: 16,384 tokens of
// heads of 128 x 128, 0.19 ns a token and head of 148 or 296 heads, 0.21 of 128,
// 0.33 of 76 (one walk a head on half of the GPU) and 0.35 of 149 (a second wave
// of one).
struct TcPlan {
    int hb, nhb, nC, nseg, L;
    size_t tails, decs, init, bytes;   // workspace offsets and size
};
TcPlan plan_tc(int B, int T, int H, int G, int dk, int dv) {
    TcPlan p{};
    p.hb = dv == 64 && (H / G) % 2 == 0 ? 2 : 1;
    p.nhb = H / p.hb;
    p.nC = (T + gdn::ssmtc::kTok - 1) / gdn::ssmtc::kTok;
    int g = gdn::device_sm_count() / (B * p.nhb);
    if (g > p.nC) g = p.nC;
    while (g > 1 && g * g > kSegSquare * p.nC) --g;
    if (g < 1 || p.nC < kMinSegmented) g = 1;
    const int least = (p.nC + gdn::ssmtc::kMaxSegChunks - 1) / gdn::ssmtc::kMaxSegChunks;
    if (g < least) g = least;
    p.L = (p.nC + g - 1) / g;
    p.nseg = (p.nC + p.L - 1) / p.L;
    if (p.nseg > 1) {
        const size_t bh = (size_t)B * H, st = (size_t)dk * dv * 4;
        p.decs = round_up(bh * (p.nseg - 1) * st, 256);
        p.init = p.decs + round_up(bh * (p.nseg - 1) * 4, 256);
        p.bytes = p.init + round_up(bh * st, 256);
    }
    return p;
}

// [B, T, D] view as tiles of 64 columns x 128 tokens, 128B swizzle.
bool encode_rows(CUtensorMap *m, const void *base, int B, size_t bs, int T, size_t ts, int D) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = gdn::driver_tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t sb = B > 1 ? bs * 2 : ts * 2;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)T, (cuuint64_t)B, 1};
    const cuuint64_t strides[3] = {ts * 2, sb, sb};
    const cuuint32_t box[4] = {64, gdn::ssmtc::kTok, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, int HB>
gdn_status launch_tc(const Scan &c, const TcPlan &pl, void *ws) {
    using namespace gdn::ssmtc;
    const gdn::ssm::Args &a = c.a;
    CUtensorMap mq, mk, mv, mo;
    const int D = a.H * DV;
    if (!encode_rows(&mq, a.q, a.B, a.q_bs, a.T, a.q_ts, a.G * DK) ||
        !encode_rows(&mk, a.k, a.B, a.k_bs, a.T, a.k_ts, a.G * DK) ||
        !encode_rows(&mv, a.v, a.B, a.v_bs, a.T, a.v_ts, D) ||
        !encode_rows(&mo, a.o, a.B, (size_t)a.T * D, a.T, D, D))
        return GDN_ERR_CUDA;
    Params p{};
    p.a = a;
    p.dt_f32 = c.dt_t == GDN_F32;
    p.nhb = pl.nhb;
    p.nseg = pl.nseg;
    p.L = pl.L;
    p.init = a.state_in;
    p.err = gdn::wait_timeout_counter();
    if (!p.err) return GDN_ERR_CUDA;
    if (pl.nseg > 1) {
        char *base = static_cast<char *>(ws);
        float *tails = reinterpret_cast<float *>(base + pl.tails);
        float *decs = reinterpret_cast<float *>(base + pl.decs);
        float *copy = a.state_in && a.state_in == a.state_out ? reinterpret_cast<float *>(base + pl.init) : nullptr;
        auto kern = tail_kernel<DK, DV, HB>;
        constexpr int smem = TailSmem<DK, DV * HB>::kBytes;
        static std::atomic<unsigned long long> done;
        if (!allow_smem(kern, smem, done)) return GDN_ERR_CUDA;
        gdn::LaunchScope ls("ssm_tail", c.stream);
        kern<<<dim3(pl.nseg - 1, a.B * pl.nhb), kTailThreads, smem, c.stream>>>(mk, mv, p, tails, decs, copy);
        if (launch_status() != GDN_OK) return GDN_ERR_CUDA;
        p.tails = tails;
        p.decs = decs;
        if (copy) p.init = copy;
    }
    auto kern = walk_kernel<DK, DV, HB>;
    constexpr int smem = Smem<DK, DV * HB>::kBytes;
    static std::atomic<unsigned long long> done;
    static std::atomic<int> regs;
    if (!allow_smem(kern, smem, done) || !has_registers(kern, kRegsLaunch, regs)) return GDN_ERR_CUDA;
    gdn::LaunchScope ls("ssm_walk", c.stream);
    // behind the contributions' launch the walk may start before they have all
    // finished (it waits for them before it reads anything of theirs)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pl.nseg, a.B * pl.nhb);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pl.nseg > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, mo, p) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <int DK>
gdn_status tc_dims(const Scan &c, const TcPlan &pl, void *ws) {
    if (c.dv == 128) return launch_tc<DK, 128, 1>(c, pl, ws);
    return pl.hb == 2 ? launch_tc<DK, 64, 2>(c, pl, ws) : launch_tc<DK, 64, 1>(c, pl, ws);
}

gdn_status check_ws(const void *ws, size_t have, size_t need) {
    if (need == 0) return GDN_OK;
    if (!ws) return GDN_ERR_NULL;
    if (!aligned(ws, 256)) return GDN_ERR_ALIGN;
    return have < need ? GDN_ERR_WORKSPACE : GDN_OK;
}

gdn_status run_scan(const Scan &c, void *ws, size_t ws_bytes) {
    if (use_tc(c.a.T, c.t)) {
        const TcPlan pl = plan_tc(c.a.B, c.a.T, c.a.H, c.a.G, c.dk, c.dv);
        const gdn_status s = check_ws(ws, ws_bytes, pl.bytes);
        if (s != GDN_OK) return s;
        return c.dk == 128 ? tc_dims<128>(c, pl, ws) : tc_dims<64>(c, pl, ws);
    }
    if (use_chunks(c.a.B, c.a.T, c.a.H, c.dk, c.dv, c.t)) {
        const ChunkPlan pl = plan_chunks(c.a.B, c.a.T, c.a.H, c.dk, c.dv);
        const gdn_status s = check_ws(ws, ws_bytes, pl.bytes);
        return s != GDN_OK ? s : chunk_dims(c, pl, ws);
    }
    if (c.t == GDN_F32) return token_dims<float, float>(c);
    return c.dt_t == GDN_F32 ? token_dims<bf16, float>(c) : token_dims<bf16, bf16>(c);
}

bool scan_sizes(int B, int T, int H, int G) {
    return B >= 1 && H >= 1 && G >= 1 && T >= 0 && T <= kMaxTokens && H % G == 0 && (long long)B * H <= 65535;
}

}  // namespace

extern "C" {

gdn_status gdn_short_conv(const void *x, size_t x_batch_stride, size_t x_token_stride, const float *w,
                          const float *bias, const void *state_in, void *state_out, void *y, const int *lengths,
                          int B, int T, int C, int K, int silu, gdn_dtype dt, void *stream) {
    if (!known(dt)) return GDN_ERR_DTYPE;
    if (B < 1 || B > 65535 || T < 0 || T > kMaxTokens || C < 1 || C > kMaxTokens) return GDN_ERR_SHAPE;
    if (K < 2 || K > 4) return GDN_ERR_UNSUPPORTED;
    if (T == 0 && !state_out) return GDN_OK;
    if (!w || (T > 0 && (!x || !y))) return GDN_ERR_NULL;
    const size_t es = esize(dt);
    if (!aligned(w, 4) || !aligned(bias, 4) || !aligned(lengths, 4) || !aligned(x, es)) return GDN_ERR_ALIGN;
    if (!aligned(y, 16) || !aligned(state_in, 16) || !aligned(state_out, 16)) return GDN_ERR_ALIGN;
    settle(T, x_token_stride, C);
    settle(B, x_batch_stride, C);
    if (T > 0 && ((T > 1 && x_token_stride < (size_t)C) || (B > 1 && x_batch_stride < (size_t)C)))
        return GDN_ERR_SHAPE;
    const size_t nx = T > 0 ? span(B, x_batch_stride, T, x_token_stride, 1, 0, C, es) : 0;
    const size_t ny = (size_t)B * T * C * es, ns = (size_t)B * (K - 1) * C * es;
    if (overlap(y, ny, x, nx) || overlap(y, ny, state_in, ns) || overlap(y, ny, state_out, ns) ||
        overlap(state_out, ns, x, nx) || (overlap(state_out, ns, state_in, ns) && state_out != state_in))
        return GDN_ERR_SHAPE;
    const gdn::conv::Args a{x, x_batch_stride, x_token_stride, w, bias, state_in, state_out, y, lengths, B, T, C, 0, 0};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dt == GDN_F32 ? conv_width<float>(a, B, K, silu, s) : conv_width<bf16>(a, B, K, silu, s);
}

gdn_status gdn_rotary(const void *q, size_t q_batch_stride, size_t q_token_stride, size_t q_head_stride, void *q_out,
                      size_t q_out_batch_stride, size_t q_out_token_stride, size_t q_out_head_stride, int Hq,
                      const void *k, size_t k_batch_stride, size_t k_token_stride, size_t k_head_stride, void *k_out,
                      size_t k_out_batch_stride, size_t k_out_token_stride, size_t k_out_head_stride, int Hk,
                      const void *pos, int pos_bits, int axes, const void *freqs, float scale, int B, int T, int d,
                      int rot, int interleaved, gdn_dtype dt, void *stream) {
    if (!known(dt)) return GDN_ERR_DTYPE;
    if (pos_bits != 32 && pos_bits != 64) return GDN_ERR_DTYPE;
    if (B < 1 || T < 0 || T > kMaxTokens || Hq < 1 || Hk < 0 || Hq > 65535 || Hk > 65535 || d < 2 || axes < 1 ||
        axes > 8 || (long long)B * T > (1ll << 31))
        return GDN_ERR_SHAPE;
    if (rot < 2 || rot % 2 || rot > d || rot > gdn::rope::kMaxRot || d > 1024) return GDN_ERR_UNSUPPORTED;
    if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f) return GDN_ERR_SHAPE;
    if (T == 0) return GDN_OK;
    if (!q || !q_out || !pos || !freqs || (Hk > 0 && (!k || !k_out))) return GDN_ERR_NULL;
    const size_t es = esize(dt);
    size_t *bst[4] = {&q_batch_stride, &q_out_batch_stride, &k_batch_stride, &k_out_batch_stride};
    size_t *tst[4] = {&q_token_stride, &q_out_token_stride, &k_token_stride, &k_out_token_stride};
    size_t *hst[4] = {&q_head_stride, &q_out_head_stride, &k_head_stride, &k_out_head_stride};
    for (int i = 0; i < 4; ++i) {
        settle(B, *bst[i], d);
        settle(T, *tst[i], d);
        settle(i < 2 ? Hq : Hk, *hst[i], d);
    }
    const void *ps[4] = {q, q_out, Hk ? k : q, Hk ? k_out : q};
    for (const void *p : ps)
        if (!aligned(p, es)) return GDN_ERR_ALIGN;
    if (!aligned(pos, pos_bits / 8) || !aligned(freqs, 8)) return GDN_ERR_ALIGN;
    gdn::rope::Args a{};
    a.q = {q, q_out, q_batch_stride, q_token_stride, q_head_stride, q_out_batch_stride, q_out_token_stride,
           q_out_head_stride, Hq};
    a.k = {k, k_out, k_batch_stride, k_token_stride, k_head_stride, k_out_batch_stride, k_out_token_stride,
           k_out_head_stride, Hk};
    // an output is its own input exactly (in place), or overlaps neither
    // input; the two outputs do not overlap
    const View in[2] = {{q, B, q_batch_stride, T, q_token_stride, Hq, q_head_stride, d},
                        {k, B, k_batch_stride, T, k_token_stride, Hk, k_head_stride, d}};
    const View out[2] = {{q_out, B, q_out_batch_stride, T, q_out_token_stride, Hq, q_out_head_stride, d},
                         {k_out, B, k_out_batch_stride, T, k_out_token_stride, Hk, k_out_head_stride, d}};
    const int np = Hk ? 2 : 1;
    bool copy = false;
    for (int i = 0; i < np; ++i) {
        if (!distinct(out[i])) return GDN_ERR_SHAPE;
        const bool inplace = out[i].p == in[i].p && out[i].bs == in[i].bs && out[i].ts == in[i].ts &&
                             out[i].hs == in[i].hs;
        copy = copy || (!inplace && rot < d);
        for (int j = 0; j < np; ++j)
            if (!(i == j && inplace) && clash(out[i], in[j], es)) return GDN_ERR_SHAPE;
    }
    if (np == 2 && clash(out[0], out[1], es)) return GDN_ERR_SHAPE;
    a.pos = pos;
    a.freqs = static_cast<const long long *>(freqs);
    a.scale = scale;
    a.T = T;
    a.d = d;
    a.rot = rot;
    a.axes = axes;
    a.pos64 = pos_bits == 64;
    a.copy = copy;
    a.rows = (long long)B * T;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dt == GDN_F32 ? rotary_type<float>(a, interleaved, s) : rotary_type<bf16>(a, interleaved, s);
}

gdn_status gdn_ssm_scan(const void *q, size_t q_batch_stride, size_t q_token_stride, const void *k,
                        size_t k_batch_stride, size_t k_token_stride, const void *v, size_t v_batch_stride,
                        size_t v_token_stride, const void *dt, size_t dt_batch_stride, size_t dt_token_stride,
                        const float *A, const float *D, const float *dt_bias, const float *state_in,
                        float *state_out, void *o, const int *lengths, int B, int T, int H, int G, int dk, int dv,
                        int softplus, gdn_dtype t, gdn_dtype dt_t, void *workspace, size_t ws_bytes, void *stream) {
    if (!known(t) || !known(dt_t) || (t == GDN_F32 && dt_t != GDN_F32)) return GDN_ERR_DTYPE;
    if (!scan_sizes(B, T, H, G)) return GDN_ERR_SHAPE;
    if (!((dk == 64 || dk == 128) && (dv == 64 || dv == 128))) return GDN_ERR_UNSUPPORTED;
    if (T == 0 && !state_out) return GDN_OK;
    const size_t es = esize(t), de = esize(dt_t);
    if (!aligned(state_in, 16) || !aligned(state_out, 16)) return GDN_ERR_ALIGN;
    const size_t ns = (size_t)B * H * dk * dv * 4;
    if (overlap(state_in, ns, state_out, ns) && state_in != state_out) return GDN_ERR_SHAPE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (state_out == state_in) return GDN_OK;
        const cudaError_t e = state_in ? cudaMemcpyAsync(state_out, state_in, ns, cudaMemcpyDeviceToDevice, s)
                                       : cudaMemsetAsync(state_out, 0, ns, s);
        return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    if (!q || !k || !v || !dt || !A || !o) return GDN_ERR_NULL;
    const void *ps[4] = {q, k, v, o};
    for (const void *p : ps)
        if (!aligned(p, 16)) return GDN_ERR_ALIGN;
    size_t *bst[4] = {&q_batch_stride, &k_batch_stride, &v_batch_stride, &dt_batch_stride};
    size_t *tst[4] = {&q_token_stride, &k_token_stride, &v_token_stride, &dt_token_stride};
    const size_t width[4] = {(size_t)G * dk, (size_t)G * dk, (size_t)H * dv, (size_t)H};
    for (int i = 0; i < 4; ++i) {
        settle(B, *bst[i], width[i]);
        settle(T, *tst[i], width[i]);
    }
    // whole 16-byte rows: tile copies need them
    const size_t st[6] = {q_batch_stride, q_token_stride, k_batch_stride, k_token_stride, v_batch_stride,
                          v_token_stride};
    for (size_t x : st)
        if (x * es % 16) return GDN_ERR_ALIGN;
    if (!aligned(dt, de) || !aligned(A, 4) || !aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(lengths, 4))
        return GDN_ERR_ALIGN;
    const size_t row[3] = {(size_t)G * dk, (size_t)G * dk, (size_t)H * dv};
    for (int i = 0; i < 3; ++i)
        if ((B > 1 && st[2 * i] < row[i]) || (T > 1 && st[2 * i + 1] < row[i])) return GDN_ERR_SHAPE;
    if ((B > 1 && dt_batch_stride < (size_t)H) || (T > 1 && dt_token_stride < (size_t)H)) return GDN_ERR_SHAPE;
    const size_t no = (size_t)B * T * H * dv * es;
    const void *in[3] = {q, k, v};
    for (int i = 0; i < 3; ++i) {
        const size_t n = span(B, st[2 * i], T, st[2 * i + 1], 1, 0, row[i], es);
        if (overlap(o, no, in[i], n) || overlap(state_out, ns, in[i], n)) return GDN_ERR_SHAPE;
    }
    const size_t nd = span(B, dt_batch_stride, T, dt_token_stride, 1, 0, H, de);
    if (overlap(o, no, dt, nd) || overlap(state_out, ns, dt, nd) || overlap(o, no, state_in, ns) ||
        overlap(o, no, state_out, ns))
        return GDN_ERR_SHAPE;
    Scan c{{q, k, v, dt, q_batch_stride, q_token_stride, k_batch_stride, k_token_stride, v_batch_stride,
            v_token_stride, dt_batch_stride, dt_token_stride, A, D, dt_bias, state_in, state_out, o, lengths, B, T, H,
            G, softplus},
           dk, dv, t, dt_t, s};
    return run_scan(c, workspace, ws_bytes);
}

size_t gdn_ssm_workspace_size(int B, int T, int H, int G, int dk, int dv, gdn_dtype t) {
    if (!known(t) || !scan_sizes(B, T, H, G) || !((dk == 64 || dk == 128) && (dv == 64 || dv == 128))) return 0;
    if (use_tc(T, t)) return plan_tc(B, T, H, G, dk, dv).bytes;
    return use_chunks(B, T, H, dk, dv, t) ? plan_chunks(B, T, H, dk, dv).bytes : 0;
}

}  // extern "C"
