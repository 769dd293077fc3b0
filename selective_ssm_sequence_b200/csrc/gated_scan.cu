// gated_scan.cu -- the channel-wise gated recurrence: forward, backward, one
// token (hm_gated_scan_fwd, _bwd, _step).
//
//   z = dt + bias, Delta = softplus(z), a = exp(-Delta exp(A_log))
//   h_t = a_t h_{t-1} + beta_t x_t
//
// A run of tokens acts on the state as h -> A h + B with A the product of its
// decays, and runs compose: (A2, B2) o (A1, B1) = (A2 A1, A2 B1 + B2).  A warp
// takes 64 channels (two per lane) and a run of consecutive tokens, whose
// decays and inputs stay in registers; the block's warps stand one behind the
// other in time, the blocks of a cluster likewise, and the cluster walks the
// sequence a window at a time.  In a window each warp forms its run's (A, B),
// the block composes them through shared memory and hands its own to every
// block of the cluster (st.async into their shared memory, counted by an
// mbarrier there), and each warp, now knowing its entering state, runs its
// tokens once more out of registers.  So each input is read once from HBM in
// one launch without scratch (but for the backward of long sequences of few
// channels), and every sum has a fixed order.
#include <mutex>
#include <type_traits>

#include "cluster_fit.h"
#include "packed.cuh"
#include "tc_common.cuh"

namespace hm {

namespace {

constexpr int kChunk = 64;   // tokens between two stored states
constexpr int kCols = 64;    // channels of a warp
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int64_t clamped_len(const int32_t *lengths, int64_t b, int64_t L) {
    if (!lengths) return L;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n > L ? L : n;
}


// ------------------------------------------------------------------ gates

__device__ __forceinline__ F2 ex2(F2 a) {
    const float2 u = un(a);
    return pk(tc::ex2_approx(u.x), tc::ex2_approx(u.y));
}
__device__ __forceinline__ float sqrt_approx(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Latency bounds this pass at the 16 warps that an SM holds of it (half of the
// issue slots and a third of the special-function unit are used), so fewer
// instructions are less time: the gates are formed in the log2 domain with two
// special-function instructions per element (three with HM_INPUT_UNIT) and
// packed fp32 arithmetic:
//   e = 2^-|z'|, z' = z / ln 2;   softplus(z) / ln 2 = max(z', 0) + log2(1 + e)
// with log2(1 + e) = e P(e) a polynomial on the whole [0, 1], which keeps its
// relative precision where e (and the decay's distance from one) is tiny.  No
// input overflows: an infinite z gives e = 0, and a NaN goes through e.
struct ChanParams {
    F2 bias, nrate;                   // bias / ln 2; -exp(A_log)
};
struct Gate2 {
    F2 z, e, step, la, a;             // z, step and la divided by ln 2
};

__device__ __forceinline__ ChanParams params_of(float A0, float A1, float bias0, float bias1) {
    ChanParams p;
    float r0 = expf(A0), r1 = expf(A1);
    if (r0 > 3e38f) r0 = 3e38f;       // finite, so that a step of zero decays nothing
    if (r1 > 3e38f) r1 = 3e38f;
    p.nrate = pk(-r0, -r1);
    // below infinity: tokens behind a sequence's end enter as dt = -inf, and must come out as z = -inf
    bias0 *= kLog2e, bias1 *= kLog2e;
    p.bias = pk(bias0 > 3e38f ? 3e38f : bias0, bias1 > 3e38f ? 3e38f : bias1);
    return p;
}
__device__ __forceinline__ ChanParams chan_params(const float *A_log, const float *dt_bias, int64_t c, int64_t c1,
                                                  int64_t D) {
    if (c >= D) return params_of(0.f, 0.f, 0.f, 0.f);
    if (c1 >= D) c1 = c;
    return params_of(A_log[c], A_log[c1], dt_bias ? dt_bias[c] : 0.f, dt_bias ? dt_bias[c1] : 0.f);
}

// log2(1 + e) / e for 0 <= e <= 1: the degree-7 polynomial of least maximal
// relative error (2e-7; fitted to log1p(e) / (e ln 2)).
__device__ __forceinline__ F2 log2_1p_over(F2 e) {
    F2 p = fma(splat(-0.012319470755755901f), e, splat(0.06360787898302078f));
    p = fma(p, e, splat(-0.15535186231136322f));
    p = fma(p, e, splat(0.25600969791412354f));
    p = fma(p, e, splat(-0.35339483618736267f));
    p = fma(p, e, splat(0.48006370663642883f));
    p = fma(p, e, splat(-0.7213100790977478f));
    return fma(p, e, splat(1.4426947832107544f));
}

__device__ __forceinline__ Gate2 gates2(F2 dt, const ChanParams &p) {
    Gate2 g;
    g.z = fma(dt, splat(kLog2e), p.bias);
    const float2 z = un(g.z);
    g.e = pk(tc::ex2_approx(-fabsf(z.x)), tc::ex2_approx(-fabsf(z.y)));
    g.step = fma(log2_1p_over(g.e), g.e, pk(fmaxf(z.x, 0.f), fmaxf(z.y, 0.f)));
    g.la = g.step * p.nrate;
    g.a = ex2(g.la);
    return g;
}

// beta^2 = 1 - a^2 = 1 - 2^w, w = 2 la.  Above -1/2 it is -w times a degree-4
// polynomial fitted to (2^w - 1) / w (relative error 3.2e-8), since the
// difference would lose the bits of a step that hardly decays.
__device__ __forceinline__ F2 unit_sq(const Gate2 &g) {
    const F2 w = g.la + g.la;
    F2 p = fma(splat(-0.0011544522130861878f), w, splat(-0.009541281498968601f));
    p = fma(p, w, splat(-0.0554904080927372f));
    p = fma(p, w, splat(-0.2402256429195404f));
    p = fma(p, w, splat(-0.6931471824645996f));
    const float2 s = un(p * w), u = un(w), a = un(g.a);
    return pk(u.x > -0.5f ? s.x : fmaf(-a.x, a.x, 1.f), u.y > -0.5f ? s.y : fmaf(-a.y, a.y, 1.f));
}

// beta x
template <int SCALE>
__device__ __forceinline__ F2 input2(const Gate2 &g, F2 x) {
    if (SCALE == HM_INPUT_PLAIN) return x;
    if (SCALE == HM_INPUT_STEP) return x * (g.step * splat(kLn2));
    const float2 q = un(unit_sq(g));
    return x * pk(sqrt_approx(q.x), sqrt_approx(q.y));
}

// two channels of a row as loaded: one word of bf16, two of fp32
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    uint32_t w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = *reinterpret_cast<const uint32_t *>(p); }
    __device__ __forceinline__ void set(float x, float y) { w = tc::pack_bf16x2(x, y); }
    __device__ __forceinline__ F2 pair() const { return pk(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
};
template <>
struct Raw<float> {
    float2 w;
    __device__ __forceinline__ void load(const float *p) { w = *reinterpret_cast<const float2 *>(p); }
    __device__ __forceinline__ void set(float x, float y) { w = make_float2(x, y); }
    __device__ __forceinline__ F2 pair() const { return pk(w.x, w.y); }
};
__device__ __forceinline__ void st_pair(__nv_bfloat16 *p, F2 v) {
    const float2 u = un(v);
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(u.x, u.y);
}
__device__ __forceinline__ void st_pair(float *p, F2 v) { *reinterpret_cast<float2 *>(p) = un(v); }

// How a block's tiles come and go.  kTma: boxes by TMA, where rows start on
// 16-byte boundaries.  kAsync: each thread's own elements by cp.async, ahead
// by the same number of windows: fp32 rows at any offset, bf16 rows on 4-byte
// boundaries.  kOdd (bf16 rows at odd offsets): the aligned words that hold a
// warp's 64 elements of a row, 32 or 33 of them, by cp.async from its lanes
// together; an aligned word with an element of the row in it is always readable.
enum Mode { kOdd = 0, kAsync = 1, kTma = 2 };

// A lane's two channels: neighbours where they move as one word or box; else
// 32 apart, so that a warp's single elements are neighbours in memory.
template <typename T, int MODE>
struct Lanes {
    static constexpr bool kSplit = MODE == kOdd || (MODE == kAsync && sizeof(T) == 4);
    static constexpr int kPitch = MODE == kOdd ? kCols + 2 : kCols;              // of a tile's rows
    static constexpr int kFirst = kSplit ? 1 : 2, kSecond = kSplit ? 32 : 1;     // 1st: lane * kFirst; 2nd: that + kSecond
    static __device__ __forceinline__ Raw<T> load(const T *p) {
        Raw<T> r;
        if constexpr (kSplit) r.set(hm_ld(p, 0), hm_ld(p, 32));
        else r.load(p);
        return r;
    }
};

__device__ __forceinline__ void cp_async4(void *dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// a thread's two elements of one row; in0: the first is there, in1: the second too
template <typename T, int MODE>
__device__ __forceinline__ void own_pair(T *dst, const T *src, bool in1) {
    if constexpr (Lanes<T, MODE>::kSplit) {
        cp_async4(dst, src, 4);
        if (in1) cp_async4(dst + 32, src + 32, 4);
    } else {
        cp_async4(dst, src, in1 ? 4 : 2);
    }
}

// whether a bf16 row starts in the upper half of a word
__device__ __forceinline__ int odd_half(const void *p) { return (int)((uintptr_t)p >> 1) & 1; }
// kOdd: the words of a row's elements [0, min(left, 64)) from `src` on
template <typename T>
__device__ __forceinline__ void own_words(T *dst, const T *src, int lane, int64_t left) {
    const int off = odd_half(src);
    src -= off;
    if (2 * lane - off < left) cp_async4(dst + 2 * lane, src + 2 * lane, 4);
    if (lane == 0 && off && left >= kCols) cp_async4(dst + kCols, src + kCols, 4);
}

// ------------------------------------------------------------------ exchange

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a run's (A, B), 16 bytes per lane
struct __align__(16) Map2 {
    F2 A, B;
};
__device__ __forceinline__ F2 apply(const Map2 &m, F2 h) { return fma(m.A, h, m.B); }
// m, then n
__device__ __forceinline__ Map2 then(const Map2 &m, const Map2 &n) { return {m.A * n.A, fma(n.A, m.B, n.B)}; }

// 16 bytes into block `rank`'s shared memory (at this block's address `dst`),
// counted by that block's mbarrier `bar`
__device__ __forceinline__ void st_async16(uint32_t dst, uint32_t bar, uint32_t rank, const Map2 &m) {
    asm volatile(
        "{\n\t.reg .b32 d, b;\n\t"
        "mapa.shared::cluster.u32 d, %0, %2;\n\t"
        "mapa.shared::cluster.u32 b, %1, %2;\n\t"
        "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [d], {%3, %4}, [b];\n\t}" ::"r"(dst),
        "r"(bar), "r"(rank), "l"(m.A.v), "l"(m.B.v)
        : "memory");
}

// ------------------------------------------------------------------ time split

// A sequence is walked in windows of `cluster` x W runs, W the warps of a
// block; block `rank` of the cluster takes its W runs of each.  What a block
// needs of a window are the maps of the blocks in front of it, and of the
// window before those of all others, so two mbarriers count the arrivals: `low`
// from the blocks in front (waited for in the same window), `high` from this
// block and those behind (waited for one window later, when they have long
// arrived).  No block waits for one behind it in the same window, so a
// block's latency to the others is hidden as long as they lag less than a
// window.
//
// Two slots per sender are enough: a block passes on its map of window i + 2
// only after it has seen all maps of window i + 1, and each block hands its own
// on only after all its warps have read everything of window i.
struct Exchange {
    Map2 *agg;                // [2][W][32] by parity of the window: the block's warps
    Map2 *ctas;               // [2][cluster][32]: the cluster's blocks
    uint64_t *low, *high;     // [2] each
    int rank, cluster;
    volatile int *abort_flag;
    DevErr err;
};

constexpr int kR = 16;        // tokens of a warp's run
constexpr int kStages = 2;

// One poll for a phase that other blocks of the cluster complete: their maps come
// by st.async, whose complete_tx releases at cluster scope, so the wait acquires
// at that scope (the plain form acquires within the block only, which is enough
// for the block's own TMA loads).
__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 P, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, P;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// what a barrier counts: this block's TMA loads, or maps of the cluster's blocks
enum Source { kOwnLoads, kClusterMaps };
template <Source S>
__device__ __forceinline__ bool try_wait(uint64_t *bar, uint32_t parity) {
    return S == kClusterMaps ? try_wait_cluster(bar, parity) : tc::mbar_try_wait(bar, parity);
}

// Bounded wait of every thread of the block.  After a timeout the kernel keeps
// its control flow (its loops are bounded and every block of a cluster must
// reach the barriers), with short waits that let its own copies land.
template <Source S>
__device__ __noinline__ void wait_bar_slow(uint64_t *bar, uint32_t parity, volatile int *abort_flag, DevErr err,
                                           unsigned site) {
    const uint32_t polls = *abort_flag ? 1u << 10 : tc::kWaitPolls;
    for (uint32_t i = 0; i < polls; ++i)
        if (try_wait<S>(bar, parity)) return;
    *abort_flag = 1;
    report_error(err, HM_ERR_TIMEOUT, KID_GATED_SCAN, site);
}
template <Source S>
__device__ __forceinline__ void wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort_flag, DevErr err,
                                         unsigned site) {
    if (!try_wait<S>(bar, parity)) wait_bar_slow<S>(bar, parity, abort_flag, err, site);
}

// State at the start of window `it` from that at this block's runs of the
// window before (`hb`); it > 0, cluster > 1.
__device__ __forceinline__ F2 finish_window(const Exchange &x, int it, F2 hb) {
    const int i = it - 1;
    wait_bar<kClusterMaps>(&x.high[i & 1], (i >> 1) & 1, x.abort_flag, x.err, 1);
    const Map2 *m = x.ctas + ((i & 1) * x.cluster + x.rank) * 32 + (threadIdx.x & 31);
#pragma unroll 2
    for (int r = x.rank; r < x.cluster; ++r, m += 32) hb = apply(*m, hb);
    return hb;
}

// After the block barrier of window `it` (all warps' maps in agg): the state
// entering this warp's run, from `h`, the state at the start of the window.
// h becomes the state at the block's runs (cluster > 1) or behind the window.
// Only the last warp composes all the block's maps and hands them on.
template <int W>
__device__ __forceinline__ F2 enter_run(const Exchange &x, int it, int warp, F2 &h) {
    const int lane = threadIdx.x & 31;
    const Map2 *agg = x.agg + (it & 1) * W * 32 + lane;
    if (x.cluster == 1) {
        F2 hin = h;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == warp) hin = h;
            h = apply(agg[w * 32], h);
        }
        return hin;
    }
    Map2 before = {splat(1.f), splat(0.f)};
    if (warp > 0) {
        before = agg[0];
#pragma unroll 1
        for (int w = 1; w < warp; ++w) before = then(before, agg[w * 32]);
    }
    if (warp == W - 1) {
        const Map2 q = then(before, agg[(W - 1) * 32]);
        const uint32_t slot = tc::smem_u32(x.ctas + ((it & 1) * x.cluster + x.rank) * 32 + lane);
        const uint32_t lo = tc::smem_u32(&x.low[it & 1]), hi = tc::smem_u32(&x.high[it & 1]);
        if (lane == 0) {
            tc::mbar_arrive_expect_tx(&x.high[it & 1], (uint32_t)(x.cluster - x.rank) * 512u);
            if (x.rank) tc::mbar_arrive_expect_tx(&x.low[it & 1], (uint32_t)x.rank * 512u);
        }
#pragma unroll 1
        for (int r = 0; r < x.cluster; ++r) st_async16(slot, x.rank < r ? lo : hi, (uint32_t)r, q);
    }
    if (x.rank) {
        wait_bar<kClusterMaps>(&x.low[it & 1], (it >> 1) & 1, x.abort_flag, x.err, 2);
        const Map2 *m = x.ctas + (it & 1) * x.cluster * 32 + lane;
#pragma unroll 2
        for (int r = 0; r < x.rank; ++r, m += 32) h = apply(*m, h);
    }
    return warp ? apply(before, h) : h;
}

// ------------------------------------------------------------------ forward

struct FwdArgs {
    hm_gated_scan_args p;
    int64_t groups;           // column groups of a sequence
    int64_t nchunk;
};

// blockIdx.x = (sequence, column group, rank in cluster).  With kTma and kAsync
// the window after the next is on its way while one is computed (two stages);
// with kTma each warp sends its run's results from a staging tile of its own,
// except the run in which a sequence ends; else element stores.
//
// The run's composed maps live in registers (64 of them): 16 warps on an SM.
template <typename T, int SCALE, int MODE, int W>
__global__ void __launch_bounds__(W * 32, 16 / W)
gated_fwd_kernel(const __grid_constant__ CUtensorMap map_dt, const __grid_constant__ CUtensorMap map_x,
                 const __grid_constant__ CUtensorMap map_y, FwdArgs f, int cluster, DevErr err) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kStages], low[2], high[2];
    __shared__ int abort_flag;
    constexpr bool WIDE = MODE == kTma;
    constexpr int kFirst = Lanes<T, MODE>::kFirst, kSecond = Lanes<T, MODE>::kSecond;
    constexpr int kPitch = Lanes<T, MODE>::kPitch;
    constexpr int kRows = W * kR;                  // tokens of a block's window
    constexpr int kTile = kRows * kPitch;          // elements of a tile
    constexpr uint32_t kBytes = kTile * sizeof(T);
    const hm_gated_scan_args &p = f.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int64_t unit = blockIdx.x / cluster, b = unit / f.groups;
    const int64_t c0 = (unit - b * f.groups) * kCols, c = c0 + kFirst * lane;
    const bool in0 = c < p.D, in1 = c + kSecond < p.D;
    const int n = (int)clamped_len(p.lengths, b, p.L);          // L is at most 2^30
    const int window = cluster * kRows;
    const int iters = (int)(((unsigned)n + (unsigned)window - 1u) / (unsigned)window);
    T *stage0 = reinterpret_cast<T *>(smem), *out = stage0 + 2 * kStages * kTile + warp * kR * kCols;
    Exchange x;
    x.agg = reinterpret_cast<Map2 *>(smem + (WIDE ? 2 * kStages + 1 : 2 * kStages) * kBytes);
    x.ctas = x.agg + 2 * W * 32;
    x.low = low;
    x.high = high;
    x.rank = rank;
    x.cluster = cluster;
    x.abort_flag = &abort_flag;
    x.err = err;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < kStages; ++s) tc::mbar_init(&full[s], 1);
        for (int s = 0; s < 2; ++s) tc::mbar_init(&low[s], 1), tc::mbar_init(&high[s], 1);
        tc::mbar_fence_init();
    }
    auto fetch = [&](int it) {
        const int s = it % kStages, t = it * window + rank * kRows;
        T *dst = stage0 + s * 2 * kTile;
        tc::mbar_arrive_expect_tx(&full[s], 2 * kBytes);
        tc::tma_load_3d(dst, &map_dt, &full[s], (int)c0, t, (int)b);
        tc::tma_load_3d(dst + kTile, &map_x, &full[s], (int)c0, t, (int)b);
    };
    if (cluster > 1) cluster_sync();
    else __syncthreads();
    if (WIDE && threadIdx.x == 0)
        for (int s = 0; s < kStages && s < iters; ++s) fetch(s);

    const ChanParams par = chan_params(p.A_log, p.dt_bias, c, c + kSecond, p.D);
    // the state at the start of the window; between windows of a cluster that at this block's runs
    F2 h = splat(0.f);
    if (p.h0) h = pk(in0 ? p.h0[b * p.D + c] : 0.f, in1 ? p.h0[b * p.D + c + kSecond] : 0.f);
    const T *dtp = (const T *)p.dt + b * p.dt_stride_b + c, *xp = (const T *)p.x + b * p.x_stride_b + c;
    T *yp = (T *)p.y + b * p.y_stride_b + c;
    auto fetch_own = [&](int it) {                 // this thread's elements (kOdd: words) of window `it`
        const int t = it * window + rank * kRows + warp * kR, m = in0 || MODE == kOdd ? min(n - t, kR) : 0;
        T *dst = stage0 + (it % kStages) * 2 * kTile + warp * kR * kPitch + (MODE == kOdd ? 0 : kFirst * lane);
        const T *pd = dtp + t * p.dt_stride_t, *px = xp + t * p.x_stride_t;
#pragma unroll 4
        for (int i = 0; i < m; ++i, dst += kPitch, pd += p.dt_stride_t, px += p.x_stride_t) {
            if (MODE == kOdd) {
                own_words(dst, pd - lane, lane, p.D - c0);
                own_words(dst + kTile, px - lane, lane, p.D - c0);
                continue;
            }
            own_pair<T, MODE>(dst, pd, in1);
            own_pair<T, MODE>(dst + kTile, px, in1);
        }
        cp_async_commit();
    };
    if (!WIDE)
        for (int s = 0; s < kStages; ++s) fetch_own(s);
    // kOdd: the half word a row starts in; a run's first token is even
    const int hd = MODE == kOdd ? odd_half(dtp - lane) : 0, hx = MODE == kOdd ? odd_half(xp - lane) : 0;
    const int sd = MODE == kOdd ? (int)p.dt_stride_t & 1 : 0, sx = MODE == kOdd ? (int)p.x_stride_t & 1 : 0;

    int t0 = rank * kRows + warp * kR;             // the run's first token
    for (int it = 0; it < iters; ++it, t0 += window) {
        const int m = min(max(n - t0, 0), kR);     // tokens of this run
        Map2 run[kR];                              // the run's composition up to each token
        Map2 all = {splat(1.f), splat(0.f)};
        if (WIDE) wait_bar<kOwnLoads>(&full[it % kStages], (it / kStages) & 1, &abort_flag, err, 0);
        if (!WIDE) cp_async_wait<kStages - 1>();
        if (MODE == kOdd) __syncwarp();            // the other lanes' words
        if (m > 0) {
            Raw<T> dv[kR], xv[kR];
            const T *sdt = stage0 + (it % kStages) * 2 * kTile + (warp * kR) * kPitch + kFirst * lane;
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                dv[i] = Lanes<T, MODE>::load(sdt + i * kPitch + (hd ^ (i & sd)));
                xv[i] = Lanes<T, MODE>::load(sdt + kTile + i * kPitch + (hx ^ (i & sx)));
            }
            if (m < kR) {        // tokens behind the end change nothing: a step of zero, no input
#pragma unroll
                for (int i = 0; i < kR; ++i)
                    if (i >= m) dv[i].set(-INFINITY, -INFINITY), xv[i].set(0.f, 0.f);
            }
            F2 sum = splat(0.f);
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                const Gate2 g = gates2(dv[i].pair(), par);
                sum = sum + g.la;
                all.B = fma(g.a, all.B, input2<SCALE>(g, xv[i].pair()));
                all.A = all.A * g.a;
                run[i] = all;
            }
            // the whole run's decay from the sum of the exponents: the rounding of the
            // single decays then does not build up over more than a run
            all.A = ex2(sum);
        }
        x.agg[((it & 1) * W + warp) * 32 + lane] = all;
        if (cluster > 1 && it > 0) h = finish_window(x, it, h);
        __syncthreads();         // maps written; this window's tiles, and the window before's maps, read
        if (WIDE && threadIdx.x == 0 && it + kStages < iters) fetch(it + kStages);
        if (!WIDE) fetch_own(it + kStages);
        const F2 hin = enter_run<W>(x, it, warp, h);
        if (m > 0) {
            if (p.states && t0 % kChunk == 0 && in0) {
                float *st = (float *)p.states + (b * f.nchunk + t0 / kChunk) * p.D + c;
                st[0] = un(hin).x;
                if (in1) st[kSecond] = un(hin).y;
            }
            if (WIDE && p.y && m == kR) {
                if (lane == 0) tc::bulk_wait_read_all();         // the last run's results have left
                __syncwarp();
                T *so = out + 2 * lane;
#pragma unroll
                for (int i = 0; i < kR; ++i) st_pair(so + i * kCols, apply(run[i], hin));
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tc::tma_store_3d(&map_y, out, (int)c0, t0, (int)b);
                    tc::bulk_commit();
                }
            } else if (p.y) {
                T *yr = yp + t0 * p.y_stride_t;
#pragma unroll
                for (int i = 0; i < kR; ++i) {
                    if (i < m) {
                        const float2 v = un(apply(run[i], hin));
                        if (MODE == kAsync && kSecond == 1 && in1) {
                            st_pair(yr, pk(v.x, v.y));
                        } else {
                            if (in0) hm_st(yr, 0, v.x);
                            if (in1) hm_st(yr, kSecond, v.y);
                        }
                    }
                    yr += p.y_stride_t;
                }
            }
        }
    }
    if (cluster > 1 && iters > 0) h = finish_window(x, iters, h);
    if (WIDE && lane == 0) tc::bulk_wait_all();
    if (cluster > 1) cluster_sync();               // no block leaves while others may still write to it,
    else __syncthreads();                          // and h_out may be the h0 that all have now read
    if (p.h_out && rank == 0 && warp == 0) {
        if (in0) p.h_out[b * p.D + c] = un(h).x;
        if (in1) p.h_out[b * p.D + c + kSecond] = un(h).y;
    }
}

// ------------------------------------------------------------------ backward

constexpr int kRb = 8;             // tokens of a warp's run
constexpr int kWb = kChunk / kRb;  // a block's window is the chunk behind one stored state
constexpr int kBwdStages = 3;

struct BwdArgs {
    hm_gated_scan_bwd_args p;
    int64_t groups;
    int64_t nchunk;
    float *part;                   // [B * cluster][2][D]: the blocks' shares of dA_log and d_dt_bias
    float *maps;                   // two passes: [3][B, nchunk, D]: A, R and c of every chunk; else NULL
};

__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The forward's scheme with time reversed for the adjoint: c, the gradient
// that reaches h_t from behind token t, goes through a run as c -> A c + R.
// A block's window is one chunk of 64 tokens, entered forward in time from the
// state that the forward stored, so the states need no exchange between
// blocks: the same pass over dt, x and dy gives a run's forward map (A, B) and
// its adjoint map (A, R), both with A = 2^(sum of the exponents).  Then each
// warp walks its run forward for the h_{t-1} and back for the gradients, which
// leave over the tiles of x and dt they came from.
//
// Registers hold a, h_{t-1}, Delta, sigmoid(z) (and beta) of 8 tokens: 16
// warps on an SM; x and dy are read again from shared memory.
//
// A long sequence of few channels does not fill the GPU with clusters.  There
// the backward takes two passes (maps given): gated_adjoint_kernel forms every
// chunk's adjoint map from dt and dy, gated_carry_kernel runs through them to
// the c that enters each chunk, and here every chunk stands for itself; dt and
// dy are read twice.
//
// 4 x 2048 x 2048 bf16: 62 us with the sums below (8 x 4096 x 2048 without a
// cluster 176, 1 x 32768 x 2048 in clusters of 8 264), 110 instructions per channel
// pair and token in half of the issue slots, no pipe above 35 %: bound by latency
// at 16 warps per SM.
template <typename T, int SCALE, int MODE>
__global__ void __launch_bounds__(kWb * 32, 2)
gated_bwd_kernel(const __grid_constant__ CUtensorMap map_dt, const __grid_constant__ CUtensorMap map_x,
                 const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ CUtensorMap map_dx,
                 const __grid_constant__ CUtensorMap map_ddt, BwdArgs f, int splits, DevErr err) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kBwdStages], low[2], high[2];
    __shared__ int abort_flag;
    constexpr bool WIDE = MODE == kTma;
    constexpr int kFirst = Lanes<T, MODE>::kFirst, kSecond = Lanes<T, MODE>::kSecond;
    constexpr int kPitch = Lanes<T, MODE>::kPitch;
    constexpr int kTile = kChunk * kPitch;
    constexpr uint32_t kBytes = kTile * sizeof(T);
    const hm_gated_scan_bwd_args &p = f.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cluster = f.maps ? 1 : splits;       // blocks that exchange
    const int rank = f.maps ? (int)(blockIdx.x % splits) : cluster > 1 ? (int)cluster_rank() : 0;
    const int64_t unit = blockIdx.x / splits, b = unit / f.groups;
    const int64_t c0 = (unit - b * f.groups) * kCols, c = c0 + kFirst * lane;
    const bool in0 = c < p.D, in1 = c + kSecond < p.D;
    const int n = (int)clamped_len(p.lengths, b, p.L);
    const int chunks = (n + kChunk - 1) / kChunk, iters = (chunks + splits - 1) / splits;
    T *stage0 = reinterpret_cast<T *>(smem);
    Exchange x;
    x.agg = reinterpret_cast<Map2 *>(smem + kBwdStages * 3 * kBytes);   // adjoint maps, last warp first
    Map2 *fwd = x.agg + 2 * kWb * 32;                                                // forward maps
    x.ctas = fwd + 2 * kWb * 32;
    x.low = low;
    x.high = high;
    x.rank = rank;
    x.cluster = cluster;
    x.abort_flag = &abort_flag;
    x.err = err;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < kBwdStages; ++s) tc::mbar_init(&full[s], 1);
        for (int s = 0; s < 2; ++s) tc::mbar_init(&low[s], 1), tc::mbar_init(&high[s], 1);
        tc::mbar_fence_init();
    }
    // chunk of window `it`: from the sequence's end; negative: none
    auto chunk_of = [&](int it) { return chunks - 1 - (it * splits + rank); };
    auto fetch = [&](int it) {
        const int s = it % kBwdStages, t = chunk_of(it) * kChunk;
        if (t < 0) return;
        T *dst = stage0 + s * 3 * kTile;
        tc::mbar_arrive_expect_tx(&full[s], 3 * kBytes);
        tc::tma_load_3d(dst, &map_dt, &full[s], (int)c0, t, (int)b);
        tc::tma_load_3d(dst + kTile, &map_x, &full[s], (int)c0, t, (int)b);
        tc::tma_load_3d(dst + 2 * kTile, &map_dy, &full[s], (int)c0, t, (int)b);
    };
    if (cluster > 1) cluster_sync();
    else __syncthreads();
    if (WIDE && threadIdx.x == 0)
        for (int s = 0; s < kBwdStages && s < iters; ++s) fetch(s);

    const ChanParams par = chan_params(p.A_log, p.dt_bias, c, c + kSecond, p.D);
    F2 carry = splat(0.f);         // gradient entering the window from behind (between windows: this block's part)
    if (p.dh_out) carry = pk(in0 ? p.dh_out[b * p.D + c] : 0.f, in1 ? p.dh_out[b * p.D + c + kSecond] : 0.f);
    const T *dtp = (const T *)p.dt + b * p.dt_stride_b + c, *xp = (const T *)p.x + b * p.x_stride_b + c;
    const T *dyp = (const T *)p.dy + b * p.dy_stride_b + c;
    T *dxp = (T *)p.dx + b * p.dx_stride_b + c, *ddtp = (T *)p.ddt + b * p.ddt_stride_b + c;
    auto fetch_own = [&](int it) {
        const int t = chunk_of(it) * kChunk + warp * kRb, m = (in0 || MODE == kOdd) && t >= 0 ? min(n - t, kRb) : 0;
        T *dst = stage0 + it % kBwdStages * 3 * kTile + warp * kRb * kPitch + (MODE == kOdd ? 0 : kFirst * lane);
        const T *pd = dtp + t * p.dt_stride_t, *px = xp + t * p.x_stride_t, *py = dyp + t * p.dy_stride_t;
#pragma unroll 4
        for (int i = 0; i < m; ++i, dst += kPitch) {
            if (MODE == kOdd) {
                own_words(dst, pd - lane + i * p.dt_stride_t, lane, p.D - c0);
                own_words(dst + kTile, px - lane + i * p.x_stride_t, lane, p.D - c0);
                own_words(dst + 2 * kTile, py - lane + i * p.dy_stride_t, lane, p.D - c0);
                continue;
            }
            own_pair<T, MODE>(dst, pd + i * p.dt_stride_t, in1);
            own_pair<T, MODE>(dst + kTile, px + i * p.x_stride_t, in1);
            own_pair<T, MODE>(dst + 2 * kTile, py + i * p.dy_stride_t, in1);
        }
        cp_async_commit();
    };
    if (!WIDE)
        for (int s = 0; s < kBwdStages - 1; ++s) fetch_own(s);
    // kOdd: the half word a row starts in; a run's first token is even
    const int hd = MODE == kOdd ? odd_half(dtp - lane) : 0, sd = MODE == kOdd ? (int)p.dt_stride_t & 1 : 0;
    const int hx = MODE == kOdd ? odd_half(xp - lane) : 0, sx = MODE == kOdd ? (int)p.x_stride_t & 1 : 0;
    const int hy = MODE == kOdd ? odd_half(dyp - lane) : 0, sy = MODE == kOdd ? (int)p.dy_stride_t & 1 : 0;
    // h entering the next window's chunk (with maps also c entering it from behind), a window ahead
    float h0 = 0.f, h1 = 0.f, g0 = 0.f, g1 = 0.f;
    auto fetch_state = [&](int it) {
        const int chunk = chunk_of(it);
        if (chunk < 0) return;
        const float *st = (const float *)p.states + (b * f.nchunk + chunk) * p.D + c;
        if (in0) h0 = st[0];
        if (in1) h1 = st[kSecond];
        if (f.maps) {
            const float *q = f.maps + ((2 * p.B + b) * f.nchunk + chunk) * p.D + c;
            if (in0) g0 = q[0];
            if (in1) g1 = q[kSecond];
        }
    };
    if (iters > 0) fetch_state(0);
    F2 sumA = splat(0.f), sumb = splat(0.f);
    int stage = 0;
    uint32_t phase = 0;

    for (int it = 0; it < iters; ++it) {
        const int chunk = chunk_of(it), t0 = chunk * kChunk + warp * kRb;
        const int m = chunk < 0 ? 0 : min(max(n - t0, 0), kRb);
        T *tile = stage0 + stage * 3 * kTile + (warp * kRb) * kPitch + kFirst * lane;
        F2 a[kRb], h[kRb], step[kRb], sig[kRb], beta[kRb];
        Map2 mf = {splat(1.f), splat(0.f)}, mr = {splat(1.f), splat(0.f)};
        if (WIDE && chunk >= 0) wait_bar<kOwnLoads>(&full[stage], phase, &abort_flag, err, 3);
        if (!WIDE) {
            if (MODE == kOdd) __syncwarp();
            fetch_own(it + kBwdStages - 1);                // over what this thread (kOdd: warp) used one window ago
            cp_async_wait<kBwdStages - 1>();
            if (MODE == kOdd) __syncwarp();                // the other lanes' words
        }
        if (m > 0) {
            auto at_dt = [&](int i) { return tile + i * kPitch + (hd ^ (i & sd)); };
            auto at_x = [&](int i) { return tile + kTile + i * kPitch + (hx ^ (i & sx)); };
            auto at_dy = [&](int i) { return tile + 2 * kTile + i * kPitch + (hy ^ (i & sy)); };
            // tokens behind the end: a step of zero, no input, no gradient of their own
            for (int i = m; i < kRb; ++i) {
                hm_st(at_dt(i), 0, -INFINITY), hm_st(at_dt(i), kSecond, -INFINITY);
                hm_st(at_x(i), 0, 0.f), hm_st(at_x(i), kSecond, 0.f);
                hm_st(at_dy(i), 0, 0.f), hm_st(at_dy(i), kSecond, 0.f);
            }
            Raw<T> dv[kRb], xr[kRb];
#pragma unroll
            for (int i = 0; i < kRb; ++i) {
                dv[i] = Lanes<T, MODE>::load(at_dt(i));
                xr[i] = Lanes<T, MODE>::load(at_x(i));
            }
            F2 sum = splat(0.f);
#pragma unroll
            for (int i = 0; i < kRb; ++i) {
                const Gate2 g = gates2(dv[i].pair(), par);
                const float2 e = un(g.e), z = un(g.z);
                const float r0 = rcp_approx(1.f + e.x), r1 = rcp_approx(1.f + e.y);
                sig[i] = pk(z.x < 0.f ? e.x * r0 : r0, z.y < 0.f ? e.y * r1 : r1);
                a[i] = g.a;
                step[i] = g.step;
                if (SCALE == HM_INPUT_UNIT) {
                    const float2 q = un(unit_sq(g));
                    beta[i] = pk(sqrt_approx(q.x), sqrt_approx(q.y));
                }
                const F2 xv = xr[i].pair();
                const F2 u = SCALE == HM_INPUT_PLAIN ? xv
                             : SCALE == HM_INPUT_STEP ? xv * (g.step * splat(kLn2)) : xv * beta[i];
                sum = sum + g.la;
                h[i] = u;
                mf.B = fma(g.a, mf.B, u);
            }
#pragma unroll
            for (int i = kRb - 1; i >= 0; --i) {
                const Raw<T> dy = Lanes<T, MODE>::load(at_dy(i));
                mr.B = a[i] * (dy.pair() + mr.B);
            }
            mf.A = mr.A = ex2(sum);
        }
        fwd[((it & 1) * kWb + warp) * 32 + lane] = mf;
        x.agg[((it & 1) * kWb + kWb - 1 - warp) * 32 + lane] = mr;
        if (cluster > 1 && it > 0) carry = finish_window(x, it, carry);
        if (WIDE && lane == 0) tc::bulk_wait_read_all();   // this warp's rows of the last window have left
        __syncthreads();           // maps written; the last window's tiles free
        if (WIDE && threadIdx.x == 0 && it > 0 && it - 1 + kBwdStages < iters) fetch(it - 1 + kBwdStages);
        F2 hin = pk(h0, h1);
        if (f.maps) carry = pk(g0, g1);
        F2 cin = enter_run<kWb>(x, it, kWb - 1 - warp, carry);
        if (it + 1 < iters) fetch_state(it + 1);
        if (m > 0) {
            const Map2 *mw = fwd + (it & 1) * kWb * 32 + lane;
            for (int w = 0; w < warp; ++w, mw += 32) hin = apply(*mw, hin);
#pragma unroll
            for (int i = 0; i < kRb; ++i) {                // h[i]: u_t, then h_{t-1}
                const F2 next = fma(a[i], hin, h[i]);
                h[i] = hin;
                hin = next;
            }
#pragma unroll
            for (int i = kRb - 1; i >= 0; --i) {
                const Raw<T> rx = Lanes<T, MODE>::load(tile + kTile + i * kPitch + (hx ^ (i & sx)));
                const Raw<T> rdy = Lanes<T, MODE>::load(tile + 2 * kTile + i * kPitch + (hy ^ (i & sy)));
                const F2 xv = rx.pair(), g = rdy.pair() + cin;
                cin = a[i] * g;
                F2 dla = cin * h[i];
                if (SCALE == HM_INPUT_UNIT) {
                    // g x a^2 / beta; where beta is zero so is what multiplies the quotient below
                    const float2 bt = un(beta[i]);
                    const F2 ib = pk(-rcp_approx(fmaxf(bt.x, 1e-18f)), -rcp_approx(fmaxf(bt.y, 1e-18f)));
                    dla = fma(cin * xv, a[i] * ib, dla);
                }
                F2 dz = dla * par.nrate;
                if (SCALE == HM_INPUT_STEP) dz = fma(g, xv, dz);
                dz = dz * sig[i];
                sumA = fma(dla, step[i], sumA);
                sumb = sumb + dz;
                const F2 dx = SCALE == HM_INPUT_PLAIN ? g
                              : SCALE == HM_INPUT_STEP ? g * (step[i] * splat(kLn2)) : g * beta[i];
                if (WIDE) {
                    st_pair(tile + i * kCols, dz);
                    st_pair(tile + kTile + i * kCols, dx);
                } else if (i < m) {
                    T *oz = ddtp + (int64_t)(t0 + i) * p.ddt_stride_t, *ox = dxp + (int64_t)(t0 + i) * p.dx_stride_t;
                    if (MODE == kAsync && kSecond == 1 && in1) {
                        st_pair(oz, dz);
                        st_pair(ox, dx);
                    } else {
                        if (in0) hm_st(oz, 0, un(dz).x), hm_st(ox, 0, un(dx).x);
                        if (in1) hm_st(oz, kSecond, un(dz).y), hm_st(ox, kSecond, un(dx).y);
                    }
                }
            }
            if (WIDE && m == kRb) {
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    T *row = tile - 2 * lane;
                    tc::tma_store_3d(&map_ddt, row, (int)c0, t0, (int)b);
                    tc::tma_store_3d(&map_dx, row + kTile, (int)c0, t0, (int)b);
                    tc::bulk_commit();
                }
            } else if (WIDE) {   // a thread's own elements, one by one
                tc::fence_proxy_async_smem();              // before a later box lands where they are
#pragma unroll 1
                for (int i = 0; i < m; ++i) {
                    T *oz = ddtp + (int64_t)(t0 + i) * p.ddt_stride_t, *ox = dxp + (int64_t)(t0 + i) * p.dx_stride_t;
                    const T *q = tile + i * kCols;
                    if (in0) oz[0] = q[0], ox[0] = q[kTile];
                    if (in1) oz[1] = q[1], ox[1] = q[kTile + 1];
                }
            }
        }
        if (++stage == kBwdStages) stage = 0, phase ^= 1;
    }
    if (cluster > 1 && iters > 0) carry = finish_window(x, iters, carry);
    // the block's share of the parameter gradients, its warps' in order
    if (WIDE && lane == 0) tc::bulk_wait_all();
    __syncthreads();
    x.agg[warp * 32 + lane] = {sumA, sumb};
    __syncthreads();
    if (warp == 0) {
        for (int w = 1; w < kWb; ++w) {
            const Map2 v = x.agg[w * 32 + lane];
            sumA = sumA + v.A;
            sumb = sumb + v.B;
        }
        sumA = sumA * par.nrate * splat(kLn2); // log a = -rate Delta, Delta from its base-2 exponent
        float *o = f.part + (b * splits + rank) * 2 * p.D + c;
        if (in0) o[0] = un(sumA).x, o[p.D] = un(sumb).x;
        if (in1) o[kSecond] = un(sumA).y, o[p.D + kSecond] = un(sumb).y;
    }
    if (cluster > 1) cluster_sync();                       // all have read dh_out, which dh0 may be
    if (p.dh0 && !f.maps && rank == 0 && warp == 0) {
        if (in0) p.dh0[b * p.D + c] = un(carry).x;
        if (in1) p.dh0[b * p.D + c + kSecond] = un(carry).y;
    }
}

// A warp per chunk and 64 channels: the chunk's adjoint map c -> A c + R, R from
// its last token to its first, A = 2^(sum of the exponents).  Nothing is kept of
// the tokens, so many warps fit: 32768 x 1024 bf16 in about 40 us, bound by the
// latency of 8 rows in flight per warp (16 rows, fewer warps: the same).
template <typename T, int MODE>
__global__ void __launch_bounds__(128, 8) gated_adjoint_kernel(BwdArgs f) {
    constexpr int kFirst = Lanes<T, MODE>::kFirst, kSecond = Lanes<T, MODE>::kSecond, U = 8;
    const hm_gated_scan_bwd_args &p = f.p;
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t at = warp / f.groups, b = at / f.nchunk;      // neighbours in memory: groups of a chunk
    if (b >= p.B) return;
    const int chunk = (int)(at - b * f.nchunk), n = (int)clamped_len(p.lengths, b, p.L);
    const int64_t c = (warp - at * f.groups) * kCols + kFirst * lane;
    const bool in0 = c < p.D, in1 = c + kSecond < p.D;
    const int t0 = chunk * kChunk, t1 = min(n, t0 + kChunk);
    if (t0 >= n) return;                           // the whole warp
    const ChanParams par = chan_params(p.A_log, p.dt_bias, c, c + kSecond, p.D);
    const T *dtp = (const T *)p.dt + b * p.dt_stride_b + c, *dyp = (const T *)p.dy + b * p.dy_stride_b + c;
    F2 R = splat(0.f), sum = splat(0.f);
    auto walk = [&](auto whole) {                  // whole: every lane has both channels, so no load waits for a branch
        auto own = [&](const T *q) {
            if (decltype(whole)::value) return Lanes<T, MODE>::load(q);
            Raw<T> r;
            r.set(in0 ? hm_ld(q, 0) : 0.f, in1 ? hm_ld(q, kSecond) : 0.f);
            return r;
        };
        int t = t1;
        for (; t - t0 >= U; t -= U) {
            Raw<T> d[U], y[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                d[i] = own(dtp + (int64_t)(t - 1 - i) * p.dt_stride_t);
                y[i] = own(dyp + (int64_t)(t - 1 - i) * p.dy_stride_t);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const Gate2 g = gates2(d[i].pair(), par);
                sum = sum + g.la;
                R = g.a * (y[i].pair() + R);
            }
        }
        for (; t > t0; --t) {
            const Gate2 g = gates2(own(dtp + (int64_t)(t - 1) * p.dt_stride_t).pair(), par);
            sum = sum + g.la;
            R = g.a * (own(dyp + (int64_t)(t - 1) * p.dy_stride_t).pair() + R);
        }
    };
    if (__all_sync(0xffffffffu, in1)) walk(std::true_type());
    else walk(std::false_type());
    const float2 A = un(ex2(sum)), r = un(R);
    float *o = f.maps + at * p.D + c;
    const int64_t plane = p.B * f.nchunk * p.D;
    if (in0) o[0] = A.x, o[plane] = r.x;
    if (in1) o[kSecond] = A.y, o[plane + kSecond] = r.y;
}

// c at the end of every chunk (third plane) and before the first (dh0): 64
// segments of a sequence's chunks, each composed, then walked from the c that
// enters it; 16 channels a block, so that there are blocks for half of the SMs
// and a thread's loads are in flight together (512 chunks of 1024: 7.7 us, with 32
// channels and 16 segments 10.6).
__global__ void __launch_bounds__(1024) gated_carry_kernel(BwdArgs f) {
    constexpr int kSegs = 64, kChan = 16;
    __shared__ float2 seg[kSegs][kChan];
    const hm_gated_scan_bwd_args &p = f.p;
    const int x = threadIdx.x % kChan, s = threadIdx.x / kChan;
    const int64_t c = (int64_t)blockIdx.x * kChan + x, b = blockIdx.y, plane = p.B * f.nchunk * p.D;
    const bool on = c < p.D;
    const int n = (int)clamped_len(p.lengths, b, p.L), chunks = (n + kChunk - 1) / kChunk;
    const int S = (chunks + kSegs - 1) / kSegs, lo = min(s * S, chunks), hi = min(lo + S, chunks);
    const float *__restrict__ A = f.maps + b * f.nchunk * p.D + c;
    const float *__restrict__ R = A + plane;
    float *__restrict__ out = f.maps + 2 * plane + b * f.nchunk * p.D + c;
    float a = 1.f, r = 0.f;
    if (on) {
#pragma unroll 8
        for (int k = hi - 1; k >= lo; --k) {
            const float m = A[k * p.D];
            r = fmaf(m, r, R[k * p.D]);
            a *= m;
        }
    }
    seg[s][x] = make_float2(a, r);
    float v = on && p.dh_out ? p.dh_out[b * p.D + c] : 0.f;
    __syncthreads();
#pragma unroll 4
    for (int k = kSegs - 1; k > s; --k) v = fmaf(seg[k][x].x, v, seg[k][x].y);
    if (!on) return;
#pragma unroll 8
    for (int k = hi - 1; k >= lo; --k) {
        out[k * p.D] = v;
        v = fmaf(A[k * p.D], v, R[k * p.D]);
    }
    if (s == 0 && p.dh0) p.dh0[b * p.D + c] = v;
}

// the blocks' shares summed in order: 8 threads per channel, each a stride of
// the rows, then the 8
__global__ void __launch_bounds__(256) gated_sum_kernel(const float *part, int64_t rows, int64_t D, float *dA,
                                                        float *db) {
    __shared__ float s[2][8][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float sA = 0.f, sb = 0.f;
    if (c < D)
        for (int64_t r = threadIdx.y; r < rows; r += 8) {
            sA += part[(r * 2 + 0) * D + c];
            sb += part[(r * 2 + 1) * D + c];
        }
    s[0][threadIdx.y][threadIdx.x] = sA;
    s[1][threadIdx.y][threadIdx.x] = sb;
    __syncthreads();
    if (threadIdx.y == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            sA += s[0][i][threadIdx.x];
            sb += s[1][i][threadIdx.x];
        }
        dA[c] = sA;
        if (db) db[c] = sb;
    }
}

// One token.  N = 16 bytes of x per thread where rows and widths allow (322 x
// 8128 fp32: 20 -> 12 us against single elements), else one element; bytes
// bound it, or with few sequences the launch.
template <typename T, int SCALE, int N>
__global__ void __launch_bounds__(256) gated_step_kernel(hm_gated_step_args p) {
    const int64_t groups = p.D / N, n = p.B * groups;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t b = n < (1LL << 31) ? (int64_t)((uint32_t)i / (uint32_t)groups) : i / groups;
        const int64_t c = (i - b * groups) * N;
        const T *dt = (const T *)p.dt + b * p.dt_stride + c, *x = (const T *)p.x + b * p.x_stride + c;
        T *y = (T *)p.y + b * p.y_stride + c;
        const float *hi = p.h + b * p.D + c;
        float *ho = p.h_out + b * p.D + c;
        if constexpr (N == 1) {
            const ChanParams par = chan_params(p.A_log, p.dt_bias, c, c, p.D);
            const Gate2 g = gates2(splat(hm_ld(dt, 0)), par);
            const float v = un(fma(g.a, splat(hi[0]), input2<SCALE>(g, splat(hm_ld(x, 0))))).x;
            ho[0] = v;
            hm_st(y, 0, v);
        } else {
            union Words {
                uint4 w;
                Raw<T> r[16 / sizeof(Raw<T>)];
                __device__ Words() {}
            } wd, wx, wy;
            wd.w = __ldcs(reinterpret_cast<const uint4 *>(dt));
            wx.w = __ldcs(reinterpret_cast<const uint4 *>(x));
            float4 h[N / 4], A[N / 4], bias[N / 4];
#pragma unroll
            for (int k = 0; k < N / 4; ++k) {
                h[k] = __ldcs(reinterpret_cast<const float4 *>(hi) + k);
                A[k] = __ldg(reinterpret_cast<const float4 *>(p.A_log + c) + k);
                bias[k] = p.dt_bias ? __ldg(reinterpret_cast<const float4 *>(p.dt_bias + c) + k) : float4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int k = 0; k < N / 2; ++k) {
                const float *Ak = &A[k / 2].x + k % 2 * 2, *bk = &bias[k / 2].x + k % 2 * 2;
                float *hk = &h[k / 2].x + k % 2 * 2;
                const Gate2 g = gates2(wd.r[k].pair(), params_of(Ak[0], Ak[1], bk[0], bk[1]));
                const float2 v = un(fma(g.a, pk(hk[0], hk[1]), input2<SCALE>(g, wx.r[k].pair())));
                wy.r[k].set(v.x, v.y);
                hk[0] = v.x, hk[1] = v.y;
            }
            *reinterpret_cast<uint4 *>(y) = wy.w;
#pragma unroll
            for (int k = 0; k < N / 4; ++k) reinterpret_cast<float4 *>(ho)[k] = h[k];
        }
    }
}

// ------------------------------------------------------------------ host

bool aligned_to(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

hm_status check_common(const char *who, int64_t B, int64_t L, int64_t D, hm_dtype t, int scale) {
    if (t != HM_F32 && t != HM_BF16) return fail_args(HM_ERR_INVALID_ARG, "%s: bad io dtype", who);
    if (scale < HM_INPUT_PLAIN || scale > HM_INPUT_UNIT)
        return fail_args(HM_ERR_INVALID_ARG, "%s: bad input scale %d", who, scale);
    if (B < 0 || L < 0 || D < 1)
        return fail_args(HM_ERR_INVALID_ARG, "%s: bad sizes B=%lld L=%lld D=%lld", who, (long long)B, (long long)L,
                         (long long)D);
    if (B > (1LL << 30) || L > (1LL << 30) || D > (1LL << 24) || B * L > (1LL << 40))
        return fail_args(HM_ERR_UNSUPPORTED, "%s: need B, L <= 2^30, B L <= 2^40 and D <= 2^24", who);
    return HM_OK;
}

// rows of one [B, L, D] array: present where needed, aligned, strides in range
hm_status check_rows(const char *who, const char *name, const void *p, size_t esize, int64_t B, int64_t L, int64_t D,
                     int64_t sb, int64_t st) {
    if (B == 0 || L == 0) return HM_OK;
    if (!p) return fail_args(HM_ERR_INVALID_ARG, "%s: null %s", who, name);
    if (!aligned_to(p, esize)) return fail_args(HM_ERR_INVALID_ARG, "%s: %s is not aligned to its type", who, name);
    if ((L > 1 && st < D) || (B > 1 && sb < D) || st < 0 || sb < 0)
        return fail_args(HM_ERR_INVALID_ARG, "%s: strides of %s are below D", who, name);
    if (st > (1LL << 40) || sb > (1LL << 50))
        return fail_args(HM_ERR_UNSUPPORTED, "%s: strides of %s are too large", who, name);
    return HM_OK;
}

hm_status check_f32(const char *who, const char *name, const void *p, bool required) {
    if (!p && required) return fail_args(HM_ERR_INVALID_ARG, "%s: null %s", who, name);
    if (!aligned_to(p, 4)) return fail_args(HM_ERR_INVALID_ARG, "%s: %s is not aligned to its type", who, name);
    return HM_OK;
}

#define HM_TRY(e)                              \
    do {                                       \
        const hm_status st_ = (e);             \
        if (st_ != HM_OK) return st_;          \
    } while (0)

size_t states_bytes(int64_t B, int64_t L, int64_t D) {
    return (size_t)(B * ((L + kChunk - 1) / kChunk) * D) * sizeof(float);
}

size_t esize(hm_dtype t) { return t == HM_BF16 ? 2 : 4; }

hm_status check_fwd(const hm_gated_scan_args *a) {
    const char *w = "gated_scan_fwd";
    if (!a) return fail_args(HM_ERR_INVALID_ARG, "%s: null args", w);
    HM_TRY(check_common(w, a->B, a->L, a->D, a->io_dtype, a->input_scale));
    const size_t es = esize(a->io_dtype);
    HM_TRY(check_rows(w, "x", a->x, es, a->B, a->L, a->D, a->x_stride_b, a->x_stride_t));
    HM_TRY(check_rows(w, "dt", a->dt, es, a->B, a->L, a->D, a->dt_stride_b, a->dt_stride_t));
    if (a->y) HM_TRY(check_rows(w, "y", a->y, es, a->B, a->L, a->D, a->y_stride_b, a->y_stride_t));
    HM_TRY(check_f32(w, "A_log", a->A_log, a->B > 0));
    HM_TRY(check_f32(w, "dt_bias", a->dt_bias, false));
    HM_TRY(check_f32(w, "h0", a->h0, false));
    HM_TRY(check_f32(w, "h_out", a->h_out, false));
    HM_TRY(check_f32(w, "lengths", a->lengths, false));
    if (!a->y && !a->h_out && !a->states && a->B > 0)
        return fail_args(HM_ERR_INVALID_ARG, "%s: y, h_out and states are all NULL", w);
    if (a->y && a->L > 0 && a->B > 0 && (a->y == a->x || a->y == a->dt))
        return fail_args(HM_ERR_INVALID_ARG, "%s: y must not be x or dt", w);
    if (a->states) {
        if (!aligned_to(a->states, 16))
            return fail_args(HM_ERR_INVALID_ARG, "%s: states must be 16-byte aligned", w);
        if (a->states_bytes < states_bytes(a->B, a->L, a->D))
            return fail_args(HM_ERR_INVALID_ARG, "%s: states too small (%zu < %zu bytes)", w, a->states_bytes,
                             states_bytes(a->B, a->L, a->D));
    }
    return HM_OK;
}

struct Split {
    int warps, cluster;       // of a block; blocks of a cluster
};

// Forward.  Four warps a block for sequences up to 2048 and for fp32 (whose
// tiles leave room for two such blocks on an SM), else eight; the tokens are
// split over up to 8 blocks of a cluster until about 14 warps stand on each
// SM, as long as a block keeps 2 windows or the SMs are mostly empty.  Measured
// (bf16, 4 x 2048 x 2048): 4 warps x 1, 2, 4, 8 blocks 39, 33, 30, 36 us, 8 x
// 1, 2, 4: 31, 31, 38; 8 x 4096 x 2048: 8 x 1: 82, 4 x 1: 89, 8 x 2: 100; one of
// 32768: 8 x 8: 129, 4 x 8: 137, 8 x 4: 148, 8 x 16: 162; fp32 2 x 4096 x 2048:
// 4 x 2, 4, 8: 52, 38, 46.  Padded batches count half their tokens (fp32 5 x
// up to 1531 x 1001: 4 x 2, 4, 8: 121, 64, 39).
//
// Clusters are of at most 8 blocks, or 16 where 8 leave SMs idle or half used and
// 16 find room (fp32 1 x 16384 x 512: 57 -> 42 us, 1 x 4096 x 700: 18.9 -> 14.8, but 1 x
// 16384 x 1024: 68 -> 75; bf16 1 x 32768 x 300: 105 -> 60, 1 x 32768 x 1024: 102 -> 97, 1 x
// 2048 x 1024: 12.7 -> 10.6, but 2 x 8192 x 512: 29 -> 31; with more channels,
// 32768 x 2048 above).
int most_blocks(int64_t units, hm_dtype t) { return units * 16 <= (t == HM_BF16 ? 296 : 192) ? 16 : 8; }

Split split_of(int64_t units, int64_t L, hm_dtype t, bool padded) {
    const int64_t runs = (L + kR - 1) / kR, warps = t == HM_BF16 && L > 2048 ? 8 : 4;
    const int64_t most = (t == HM_BF16 ? 148 * 16 : 148 * 12) * (padded ? 2 : 1);
    Split s{(int)warps, 1};
    const int lim = most_blocks(units, t);
    while (s.cluster < lim && units * s.cluster * 2 * warps <= most && warps * s.cluster < runs &&
           (runs >= 2 * warps * s.cluster * 2 || units * s.cluster * 2 <= 148))
        s.cluster *= 2;
    return s;
}

// Backward: 8 warps and a window of 64 tokens a block.  4 x 2048 x 2048 with
// its forward: 1, 2, 4, 8 blocks 95, 91, 98, 109 us; one of 32768: 4, 8, 16:
// 411, 337, 427.  16 as in the forward for bf16 (2 x 1909 x 64: 27 -> 23 us, 1 x
// 4096 x 512: 42 -> 38); fp32 4 x 2885 x 128: 38 -> 42.
Split bwd_split(int64_t units, int64_t L, hm_dtype t) {
    const int64_t chunks = (L + kChunk - 1) / kChunk;
    const int lim = t == HM_BF16 ? most_blocks(units, t) : 8;
    Split s{kWb, 1};
    while (s.cluster < lim && units * s.cluster * 2 <= 148 * 2 && s.cluster < chunks) s.cluster *= 2;
    return s;
}
// Two passes, for long sequences of so few channels that clusters of 8 leave
// SMs idle; a sequence's chunks then go to two blocks on every SM.  Forward and
// backward, one pass and two: fp32 1 x 16384 x 1024: 236, 178 us; bf16 1 x 32768 x
// 1024: 316, 229; 1 x 32768 x 512: 185, 138; 1 x 16384 x 64: 77, 55; but 1 x 4096 x 512:
// 38, 45; 1 x 32768 x 2048: 388, 463 (what is read twice costs more than the waits).
bool two_passes(int64_t units, int64_t L) { return units * 8 <= 148 && L > 8192; }
int bwd_blocks(int64_t units, int64_t L, hm_dtype t) {
    if (!two_passes(units, L)) return bwd_split(units, L, t).cluster;
    const int64_t chunks = (L + kChunk - 1) / kChunk, most = 148 * 2 / units;
    return (int)(most < chunks ? most : chunks);
}

size_t bwd_workspace(const hm_gated_scan_bwd_args *a) {
    const int64_t units = a->B * ((a->D + kCols - 1) / kCols), nchunk = (a->L + kChunk - 1) / kChunk;
    if (units == 0) return 0;
    const int64_t maps = two_passes(units, a->L) ? 3 * a->B * nchunk * a->D : 0;
    return (size_t)(a->B * bwd_blocks(units, a->L, a->io_dtype) * 2 * a->D + maps) * sizeof(float);
}

hm_status check_bwd(const hm_gated_scan_bwd_args *a) {
    const char *w = "gated_scan_bwd";
    if (!a) return fail_args(HM_ERR_INVALID_ARG, "%s: null args", w);
    HM_TRY(check_common(w, a->B, a->L, a->D, a->io_dtype, a->input_scale));
    const size_t es = esize(a->io_dtype);
    HM_TRY(check_rows(w, "x", a->x, es, a->B, a->L, a->D, a->x_stride_b, a->x_stride_t));
    HM_TRY(check_rows(w, "dt", a->dt, es, a->B, a->L, a->D, a->dt_stride_b, a->dt_stride_t));
    HM_TRY(check_rows(w, "dy", a->dy, es, a->B, a->L, a->D, a->dy_stride_b, a->dy_stride_t));
    HM_TRY(check_rows(w, "dx", a->dx, es, a->B, a->L, a->D, a->dx_stride_b, a->dx_stride_t));
    HM_TRY(check_rows(w, "ddt", a->ddt, es, a->B, a->L, a->D, a->ddt_stride_b, a->ddt_stride_t));
    HM_TRY(check_f32(w, "A_log", a->A_log, true));
    HM_TRY(check_f32(w, "dA_log", a->dA_log, true));
    HM_TRY(check_f32(w, "dt_bias", a->dt_bias, false));
    HM_TRY(check_f32(w, "d_dt_bias", a->d_dt_bias, false));
    HM_TRY(check_f32(w, "dh_out", a->dh_out, false));
    HM_TRY(check_f32(w, "dh0", a->dh0, false));
    HM_TRY(check_f32(w, "lengths", a->lengths, false));
    if (a->dA_log == a->d_dt_bias)
        return fail_args(HM_ERR_INVALID_ARG, "%s: dA_log and d_dt_bias are the same array", w);
    if (a->B > 0 && a->L > 0) {
        const void *in[] = {a->x, a->dt, a->dy}, *out[] = {a->dx, a->ddt};
        for (const void *o : out)
            for (const void *i : in)
                if (o == i) return fail_args(HM_ERR_INVALID_ARG, "%s: dx and ddt must not be x, dt or dy", w);
        if (a->dx == a->ddt) return fail_args(HM_ERR_INVALID_ARG, "%s: dx and ddt are the same array", w);
        if (!a->states || !aligned_to(a->states, 16) || a->states_bytes < states_bytes(a->B, a->L, a->D))
            return fail_args(HM_ERR_INVALID_ARG, "%s: states (%zu bytes, 16-byte aligned) of the forward are needed",
                             w, states_bytes(a->B, a->L, a->D));
    }
    return HM_OK;
}

template <typename F>
cudaError_t by_type(hm_dtype t, int scale, F f) {
#define HM_SCALE(T)                                                                           \
    (scale == HM_INPUT_PLAIN ? f((T *)nullptr, std::integral_constant<int, HM_INPUT_PLAIN>()) \
     : scale == HM_INPUT_STEP ? f((T *)nullptr, std::integral_constant<int, HM_INPUT_STEP>()) \
                              : f((T *)nullptr, std::integral_constant<int, HM_INPUT_UNIT>()))
    return t == HM_BF16 ? HM_SCALE(__nv_bfloat16) : HM_SCALE(float);
#undef HM_SCALE
}

}  // namespace

}  // namespace hm

using namespace hm;

extern "C" size_t hm_gated_scan_states_size(const hm_gated_scan_args *a) {
    if (!a || check_common("gated_scan", a->B, a->L, a->D, a->io_dtype, a->input_scale) != HM_OK) return 0;
    return states_bytes(a->B, a->L, a->D);
}

namespace hm {
namespace {

// [B, L, D] as (channel, token, sequence), tiles of 64 channels x `rows` tokens
bool tile_map(CUtensorMap *m, hm_dtype t, const void *base, int64_t B, int64_t L, int64_t D, int64_t sb, int64_t st,
              int rows) {
    const size_t es = esize(t);
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)L, (uint64_t)B};
    const uint64_t strides[2] = {(uint64_t)(L > 1 ? st : (D + 7) / 8 * 8) * es, (uint64_t)(B > 1 ? sb : (D + 7) / 8 * 8) * es};
    const uint32_t box[3] = {kCols, (uint32_t)rows, 1};
    return tc::make_tmap(m, t == HM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, base, 3,
                         dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// rows that TMA can fetch: 16-byte aligned base and strides
bool tma_rows(const void *p, size_t es, int64_t B, int64_t L, int64_t sb, int64_t st) {
    return aligned_to(p, 16) && (L <= 1 || st * (int64_t)es % 16 == 0) && (B <= 1 || sb * (int64_t)es % 16 == 0);
}

// rows whose elements cp.async can fetch: 4-byte words of two bf16, or single fp32 elements
bool word_rows(const void *p, size_t es, int64_t B, int64_t L, int64_t sb, int64_t st) {
    return es == 4 || (aligned_to(p, 4) && (L <= 1 || st % 2 == 0) && (B <= 1 || sb % 2 == 0));
}

struct ClusterLaunch {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at{};
    ClusterLaunch(int64_t units, Split sp, size_t smem, cudaStream_t s) {
        cfg.gridDim = dim3((unsigned)(units * sp.cluster));
        cfg.blockDim = dim3(sp.warps * 32);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = sp.cluster;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
    }
    ClusterLaunch(const ClusterLaunch &) = delete;
};

// Whether the current device has a place for one such cluster (of more blocks
// than every device takes).  Asked once per kernel, device and launch shape.
template <typename K>
bool has_place(K kernel, Split sp, size_t smem) {
    struct Entry {
        const void *kernel;
        int dev, cluster;
        size_t smem;
        bool fits;
    };
    static std::mutex mu;
    static Entry known[64];
    static int n_known = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const void *k = reinterpret_cast<const void *>(kernel);
    std::lock_guard<std::mutex> g(mu);
    for (int i = 0; i < n_known; ++i) {
        const Entry &e = known[i];
        if (e.kernel == k && e.dev == dev && e.cluster == sp.cluster && e.smem == smem) return e.fits;
    }
    const ClusterLaunch l(1, sp, smem, nullptr);
    int n = 0;
    const bool fits = tc::ensure_smem_limit(kernel, (int)smem) == cudaSuccess &&
                      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                      cudaOccupancyMaxActiveClusters(&n, kernel, &l.cfg) == cudaSuccess && n > 0;
    if (!fits) cudaGetLastError();         // a question's error is no launch's
    if (n_known < 64) known[n_known++] = {k, dev, sp.cluster, smem, fits};
    return fits;
}

// sp with a cluster that has a place; smem_of(cluster): shared memory of a block
template <typename K, typename S>
Split placed(K kernel, Split sp, S smem_of) {
    sp.cluster = placeable_cluster(
        sp.cluster, [&](int n) { return has_place(kernel, Split{sp.warps, n}, smem_of(n)); });
    return sp;
}

template <typename K, typename... A>
cudaError_t launch_cluster(K kernel, int64_t units, Split sp, size_t smem, cudaStream_t s, A... args) {
    cudaError_t e = tc::ensure_smem_limit(kernel, (int)smem);
    if (e != cudaSuccess) return e;
    const ClusterLaunch l(units, sp, smem, s);
    e = cudaLaunchKernelEx(&l.cfg, kernel, args...);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace
}  // namespace hm

extern "C" hm_status hm_gated_scan_fwd(const hm_gated_scan_args *a, hm_stream_t stream) {
    set_error_detail("");
    HM_TRY(check_fwd(a));
    if (a->B == 0) return HM_OK;
    FwdArgs f{*a, (a->D + kCols - 1) / kCols, (a->L + kChunk - 1) / kChunk};
    const int64_t units = a->B * f.groups;
    const size_t es = esize(a->io_dtype);
    const Split sp = split_of(units, a->L, a->io_dtype, a->lengths != nullptr);
    if (units * sp.cluster > 0x7fffffffLL)
        return fail_args(HM_ERR_UNSUPPORTED, "gated_scan_fwd: B * D / 64 is too large");
    CUtensorMap mdt{}, mx{}, my{};
    const int rows = sp.warps * kR;
    const bool wide = a->L > 0 && tma_rows(a->x, es, a->B, a->L, a->x_stride_b, a->x_stride_t) &&
                      tma_rows(a->dt, es, a->B, a->L, a->dt_stride_b, a->dt_stride_t) &&
                      (!a->y || (tma_rows(a->y, es, a->B, a->L, a->y_stride_b, a->y_stride_t) &&
                                 tile_map(&my, a->io_dtype, a->y, a->B, a->L, a->D, a->y_stride_b, a->y_stride_t, kR))) &&
                      tile_map(&mdt, a->io_dtype, a->dt, a->B, a->L, a->D, a->dt_stride_b, a->dt_stride_t, rows) &&
                      tile_map(&mx, a->io_dtype, a->x, a->B, a->L, a->D, a->x_stride_b, a->x_stride_t, rows);
    const bool words = word_rows(a->x, es, a->B, a->L, a->x_stride_b, a->x_stride_t) &&
                       word_rows(a->dt, es, a->B, a->L, a->dt_stride_b, a->dt_stride_t) &&
                       (!a->y || word_rows(a->y, es, a->B, a->L, a->y_stride_b, a->y_stride_t));
    const DevErr err{device_error_word()};
    const cudaError_t e = by_type(a->io_dtype, a->input_scale, [&](auto *t, auto sc) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int S = decltype(sc)::value;
        auto go = [&](auto kernel, int tiles, int pitch = kCols) {
            auto smem_of = [&](int cluster) {
                return (size_t)tiles * rows * pitch * sizeof(T) + (size_t)2 * (sp.warps + cluster) * 32 * sizeof(Map2);
            };
            const Split at = placed(kernel, sp, smem_of);
            return launch_cluster(kernel, units, at, smem_of(at.cluster), (cudaStream_t)stream, mdt, mx, my, f,
                                  at.cluster, err);
        };
        auto by_mode = [&](auto w) {
            constexpr int W = decltype(w)::value;
            if (wide) return go(gated_fwd_kernel<T, S, kTma, W>, 2 * kStages + 1);
            if (words) return go(gated_fwd_kernel<T, S, kAsync, W>, 2 * kStages);
            if constexpr (sizeof(T) == 2) return go(gated_fwd_kernel<T, S, kOdd, W>, 2 * kStages, Lanes<T, kOdd>::kPitch);
            return cudaErrorInvalidValue;          // not reached: fp32 rows are words
        };
        if constexpr (sizeof(T) == 2)
            if (sp.warps == 8) return by_mode(std::integral_constant<int, 8>());
        return by_mode(std::integral_constant<int, 4>());
    });
    return e == cudaSuccess ? HM_OK : fail_args(HM_ERR_CUDA, "gated_scan_fwd launch: %s", cudaGetErrorString(e));
}

extern "C" size_t hm_gated_scan_bwd_workspace_size(const hm_gated_scan_bwd_args *a) {
    if (!a || check_common("gated_scan_bwd", a->B, a->L, a->D, a->io_dtype, a->input_scale) != HM_OK) return 0;
    return bwd_workspace(a);
}

extern "C" hm_status hm_gated_scan_bwd(const hm_gated_scan_bwd_args *a, hm_stream_t stream) {
    set_error_detail("");
    HM_TRY(check_bwd(a));
    const size_t need = bwd_workspace(a);
    if (need > 0 && (!a->workspace || a->workspace_bytes < need || !aligned_to(a->workspace, 256)))
        return fail_args(HM_ERR_INVALID_ARG, "gated_scan_bwd: workspace of %zu bytes, 256-byte aligned, is needed",
                         need);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    int64_t shares = 0;
    if (a->B > 0) {
        BwdArgs f{*a, (a->D + kCols - 1) / kCols, (a->L + kChunk - 1) / kChunk, (float *)a->workspace, nullptr};
        const int64_t units = a->B * f.groups;
        const bool two = two_passes(units, a->L);
        const int splits = bwd_blocks(units, a->L, a->io_dtype);
        const Split sp{kWb, two ? 1 : splits};
        if (units * splits > 0x7fffffffLL)
            return fail_args(HM_ERR_UNSUPPORTED, "gated_scan_bwd: B * D / 64 is too large");
        if (two) f.maps = f.part + a->B * splits * 2 * a->D;
        const size_t es = esize(a->io_dtype);
        struct {
            const void *p;
            int64_t sb, st;
            int rows;
            CUtensorMap map;
        } t[5] = {{a->dt, a->dt_stride_b, a->dt_stride_t, kChunk, {}},
                  {a->x, a->x_stride_b, a->x_stride_t, kChunk, {}},
                  {a->dy, a->dy_stride_b, a->dy_stride_t, kChunk, {}},
                  {a->dx, a->dx_stride_b, a->dx_stride_t, kRb, {}},
                  {a->ddt, a->ddt_stride_b, a->ddt_stride_t, kRb, {}}};
        bool wide = a->L > 0, words = true;
        for (auto &r : t) {
            words = words && word_rows(r.p, es, a->B, a->L, r.sb, r.st);
            wide = wide && tma_rows(r.p, es, a->B, a->L, r.sb, r.st) &&
                   tile_map(&r.map, a->io_dtype, r.p, a->B, a->L, a->D, r.sb, r.st, r.rows);
        }
        const DevErr err{device_error_word()};
        e = by_type(a->io_dtype, a->input_scale, [&](auto *tp, auto sc) {
            using T = std::remove_pointer_t<decltype(tp)>;
            constexpr int S = decltype(sc)::value;
            const int pitch = !wide && !words ? Lanes<__nv_bfloat16, kOdd>::kPitch : kCols;
            auto smem_of = [&](int cluster) {
                return (size_t)kBwdStages * 3 * kChunk * pitch * sizeof(T) +
                       (size_t)2 * (2 * kWb + cluster) * 32 * sizeof(Map2);
            };
            auto go = [&](auto kernel, auto adjoint) {
                if (two) {
                    adjoint<<<(unsigned)((units * f.nchunk + 3) / 4), 128, 0, s>>>(f);
                    gated_carry_kernel<<<dim3((unsigned)((a->D + 15) / 16), (unsigned)a->B), 1024, 0, s>>>(f);
                    count_launches(2);
                    const cudaError_t e = cudaGetLastError();
                    if (e != cudaSuccess) return e;
                }
                const Split at = placed(kernel, sp, smem_of);
                const int blocks = two ? splits : at.cluster;      // of a unit; the workspace is for `splits` or fewer
                shares = a->B * blocks;
                return launch_cluster(kernel, units * (two ? splits : 1), at, smem_of(at.cluster), s, t[0].map,
                                      t[1].map, t[2].map, t[3].map, t[4].map, f, blocks, err);
            };
            if (wide) return go(gated_bwd_kernel<T, S, kTma>, gated_adjoint_kernel<T, kTma>);
            if (words) return go(gated_bwd_kernel<T, S, kAsync>, gated_adjoint_kernel<T, kAsync>);
            if constexpr (sizeof(T) == 2) return go(gated_bwd_kernel<T, S, kOdd>, gated_adjoint_kernel<T, kOdd>);
            return cudaErrorInvalidValue;          // not reached: fp32 rows are words
        });
    }
    if (e == cudaSuccess) {
        gated_sum_kernel<<<(unsigned)((a->D + 31) / 32), dim3(32, 8), 0, s>>>((const float *)a->workspace, shares,
                                                                              a->D, a->dA_log, a->d_dt_bias);
        count_launches(1);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? HM_OK : fail_args(HM_ERR_CUDA, "gated_scan_bwd launch: %s", cudaGetErrorString(e));
}

extern "C" hm_status hm_gated_scan_step(const hm_gated_step_args *a, hm_stream_t stream) {
    set_error_detail("");
    const char *w = "gated_scan_step";
    if (!a) return fail_args(HM_ERR_INVALID_ARG, "%s: null args", w);
    HM_TRY(check_common(w, a->B, 1, a->D, a->io_dtype, a->input_scale));
    const size_t es = esize(a->io_dtype);
    HM_TRY(check_rows(w, "x", a->x, es, a->B, 1, a->D, a->x_stride, a->D));
    HM_TRY(check_rows(w, "dt", a->dt, es, a->B, 1, a->D, a->dt_stride, a->D));
    HM_TRY(check_rows(w, "y", a->y, es, a->B, 1, a->D, a->y_stride, a->D));
    HM_TRY(check_f32(w, "A_log", a->A_log, a->B > 0));
    HM_TRY(check_f32(w, "dt_bias", a->dt_bias, false));
    HM_TRY(check_f32(w, "h", a->h, a->B > 0));
    HM_TRY(check_f32(w, "h_out", a->h_out, a->B > 0));
    if (a->B == 0) return HM_OK;
    if (a->y == a->x || a->y == a->dt) return fail_args(HM_ERR_INVALID_ARG, "%s: y must not be x or dt", w);
    const int wide = (int)(16 / es);          // elements of a 16-byte piece
    bool vec = a->D % wide == 0;
    const int64_t strides[] = {a->x_stride, a->dt_stride, a->y_stride};
    for (const int64_t st : strides) vec = vec && (a->B == 1 || st % wide == 0);
    const void *ptrs[] = {a->x, a->dt, a->y, a->h, a->h_out, a->A_log, a->dt_bias};
    for (const void *q : ptrs) vec = vec && aligned_to(q, 16);
    const int64_t blocks = (a->B * (vec ? a->D / wide : a->D) + 255) / 256;
    const unsigned grid = (unsigned)(blocks < 148 * 32 ? blocks : 148 * 32);
    const cudaError_t e = by_type(a->io_dtype, a->input_scale, [&](auto *t, auto sc) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int S = decltype(sc)::value, N = 16 / (int)sizeof(T);
        if (vec) gated_step_kernel<T, S, N><<<grid, 256, 0, (cudaStream_t)stream>>>(*a);
        else gated_step_kernel<T, S, 1><<<grid, 256, 0, (cudaStream_t)stream>>>(*a);
        count_launches(1);
        return cudaGetLastError();
    });
    return e == cudaSuccess ? HM_OK : fail_args(HM_ERR_CUDA, "%s launch: %s", w, cudaGetErrorString(e));
}
