// rotary.cu -- rotary positions on queries and keys (hm_rotary).
//
// Bandwidth-bound: every element read and written once.  A thread takes P
// pairs (P = 8 of bf16, 4 of fp32: two 16-byte loads; fewer where strides or
// the pair count ask for it) of one token and turns them in a run of heads, q's
// and then k's: the angle depends on the token and the pair alone, so its sine
// and cosine are formed once per run.  The loads of four heads are in flight
// together.
//
// Angles are kept as fractions of a turn in 64-bit fixed point: theta / (2 pi)
// mod 1 times 2^64 is an integer (formed in fp64, once per block, in shared
// memory), and its product with the position wraps modulo 2^64, which is the
// reduction modulo whole turns, exactly.
#include <math.h>

#include "hm_internal.h"

namespace hm {

namespace {

struct Side {             // q or k
    const void *in;
    void *out;
    int64_t in_b, in_t, in_h, out_b, out_t, out_h;
};

struct RotArgs {
    Side s[2];
    int Hq, H;            // q's heads, all heads
    int hg;               // heads of a run
    int64_t L;
    unsigned tokens;      // B * L
    int d, rot;
    int ng, nt;           // groups of P pairs; groups of 2 P elements behind rot (0 when left alone)
    int per;              // items of a token: runs * (ng + nt)
    int tb;               // tokens of a block
    const int64_t *positions;
    int64_t pos_b, pos_t, pos0;
    double log2_base;     // of the base in use (HM_ROTARY_NTK has put its factor in)
    double inv_factor;    // frequencies times this (linear), or the by-parts blend's low end
    double turns0;        // by parts: orig_len / (2 pi)
    double slow, inv_span;
    int by_parts;
    float mscale, sign;
};

constexpr int kThreads = 256;
constexpr int kBatch = 4;   // heads whose loads are in flight together

// theta_i / (2 pi) mod 1, in units of 2^-64 of a turn
__device__ __forceinline__ unsigned long long pair_turns(const RotArgs &a, int i) {
    double th = exp2(-(double)(2 * i) / (double)a.rot * a.log2_base);
    if (a.by_parts) {
        const double w = fmin(1.0, fmax(0.0, (a.turns0 * th - a.slow) * a.inv_span));
        th *= (1.0 - w) * a.inv_factor + w;
    } else {
        th *= a.inv_factor;
    }
    const double t = th * 0.15915494309189533577;   // 1 / (2 pi)
    return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
}

__device__ __forceinline__ void turn_of(const RotArgs &a, unsigned long long unit, int64_t pos, float &cs, float &sn) {
    const unsigned long long ph = unit * (unsigned long long)pos;
    // the top 32 bits as a signed fraction of a turn in [-1/2, 1/2)
    const float half_turns = (float)(int)(ph >> 32) * 4.656612873077392578125e-10f;   // 2^-31
    sincospif(half_turns, &sn, &cs);
    cs *= a.mscale;
    sn *= a.mscale * a.sign;
}

// P elements, P * sizeof(T) = 2 .. 16 bytes
template <typename T, int P>
struct alignas(sizeof(T) * P) Vec {
    T v[P];
};
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float &o, float v) { o = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16 &o, float v) { o = __float2bfloat16_rn(v); }

// the head's rows in and out
template <typename T>
__device__ __forceinline__ void head_of(const RotArgs &a, int h, int64_t b, int64_t t, const T *&in, T *&out) {
    const Side &s = h < a.Hq ? a.s[0] : a.s[1];
    const int i = h < a.Hq ? h : h - a.Hq;
    in = (const T *)s.in + b * s.in_b + t * s.in_t + i * s.in_h;
    out = (T *)s.out + b * s.out_b + t * s.out_t + i * s.out_h;
}

template <typename T, int P, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotArgs a) {
    __shared__ unsigned long long unit[512];
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < half; i += kThreads) unit[i] = pair_turns(a, i);
    __syncthreads();
    using V = Vec<T, P>;
    const int groups = a.ng + a.nt;
    for (int i = threadIdx.x; i < a.tb * a.per; i += kThreads) {
        const int local = i / a.per, rest = i - local * a.per, run = rest / groups, grp = rest - run * groups;
        const unsigned tok = blockIdx.x * (unsigned)a.tb + local;
        if (tok >= a.tokens) break;
        const int64_t b = tok / (unsigned)a.L, t = tok - (unsigned)b * (unsigned)a.L;
        const int h0 = run * a.hg, h1 = min(h0 + a.hg, a.H);
        if (grp >= a.ng) {             // elements behind rot
            const int c0 = a.rot + (grp - a.ng) * 2 * P;
            for (int h = h0; h < h1; ++h) {
                const T *in;
                T *out;
                head_of(a, h, b, t, in, out);
                if (c0 + P <= a.d) *reinterpret_cast<V *>(out + c0) = *reinterpret_cast<const V *>(in + c0);
                if (c0 + 2 * P <= a.d)
                    *reinterpret_cast<V *>(out + c0 + P) = *reinterpret_cast<const V *>(in + c0 + P);
            }
            continue;
        }
        const int64_t pos = a.positions ? a.positions[b * a.pos_b + t * a.pos_t] : a.pos0 + t;
        float cs[P], sn[P];
#pragma unroll
        for (int j = 0; j < P; ++j) turn_of(a, unit[grp * P + j], pos, cs[j], sn[j]);
        const int iu = INTER ? grp * 2 * P : grp * P, iv = INTER ? iu + P : iu + half;
        for (int hb = h0; hb < h1; hb += kBatch) {
            V u[kBatch], v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (hb + k < h1) {
                    const T *in;
                    T *out;
                    head_of(a, hb + k, b, t, in, out);
                    u[k] = *reinterpret_cast<const V *>(in + iu);
                    v[k] = *reinterpret_cast<const V *>(in + iv);
                }
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (hb + k < h1) {
                    const T *in;
                    T *out;
                    head_of(a, hb + k, b, t, in, out);
                    V x, y;
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        // interleaved: element 2 j of the 2 P is u_j, 2 j + 1 is v_j
                        const float p = to_f(INTER ? (2 * j < P ? u[k].v[2 * j % P] : v[k].v[2 * j % P]) : u[k].v[j]);
                        const float q = to_f(INTER ? (2 * j + 1 < P ? u[k].v[(2 * j + 1) % P] : v[k].v[(2 * j + 1) % P])
                                                   : v[k].v[j]);
                        const float r = p * cs[j] - q * sn[j], w = p * sn[j] + q * cs[j];
                        if (INTER) {
                            from_f(2 * j < P ? x.v[2 * j % P] : y.v[2 * j % P], r);
                            from_f(2 * j + 1 < P ? x.v[(2 * j + 1) % P] : y.v[(2 * j + 1) % P], w);
                        } else {
                            from_f(x.v[j], r);
                            from_f(y.v[j], w);
                        }
                    }
                    *reinterpret_cast<V *>(out + iu) = x;
                    *reinterpret_cast<V *>(out + iv) = y;
                }
        }
    }
}

size_t esize(hm_dtype t) { return t == HM_BF16 ? 2 : 4; }

hm_status check_side(const char *name, const void *in, const void *out, int H, int64_t B, int64_t L, int d, size_t es,
                     const int64_t *is, const int64_t *os) {
    if (B == 0 || L == 0 || H == 0) return HM_OK;
    if (!in || !out) return fail_args(HM_ERR_INVALID_ARG, "rotary: null %s or %s_out", name, name);
    if ((((uintptr_t)in | (uintptr_t)out) & (es - 1)) != 0)
        return fail_args(HM_ERR_INVALID_ARG, "rotary: %s or %s_out is not aligned to its type", name, name);
    const int64_t n[3] = {B, L, H}, most[3] = {1LL << 50, 1LL << 40, 1LL << 40};
    bool same = true;
    for (int i = 0; i < 3; ++i) {
        if (n[i] > 1 && (is[i] < d || os[i] < d))
            return fail_args(HM_ERR_INVALID_ARG, "rotary: strides of %s or %s_out are below d", name, name);
        if (is[i] < 0 || os[i] < 0 || is[i] > most[i] || os[i] > most[i])
            return fail_args(HM_ERR_UNSUPPORTED, "rotary: strides of %s or %s_out are out of range", name, name);
        same = same && (n[i] == 1 || is[i] == os[i]);
    }
    if (in == out && !same)
        return fail_args(HM_ERR_INVALID_ARG, "rotary: %s_out is %s with other strides", name, name);
    return HM_OK;
}

bool finite_positive(double v) { return v > 0.0 && v - v == 0.0; }

}  // namespace

}  // namespace hm

using namespace hm;

extern "C" hm_status hm_rotary(const hm_rotary_args *a, hm_stream_t stream) {
    set_error_detail("");
    if (!a) return fail_args(HM_ERR_INVALID_ARG, "rotary: null args");
    if (a->io_dtype != HM_F32 && a->io_dtype != HM_BF16) return fail_args(HM_ERR_INVALID_ARG, "rotary: bad io dtype");
    if (a->layout != HM_ROTARY_HALF && a->layout != HM_ROTARY_INTERLEAVED)
        return fail_args(HM_ERR_INVALID_ARG, "rotary: bad layout %d", a->layout);
    if (a->scaling < HM_ROTARY_PLAIN || a->scaling > HM_ROTARY_BY_PARTS)
        return fail_args(HM_ERR_INVALID_ARG, "rotary: bad scaling %d", a->scaling);
    if (a->B < 0 || a->L < 0 || a->Hq < 0 || a->Hk < 0 || a->Hq > (1 << 20) || a->Hk > (1 << 20) || a->d < 1)
        return fail_args(HM_ERR_INVALID_ARG, "rotary: bad sizes");
    if (a->rot < 2 || a->rot % 2 != 0 || a->rot > a->d)
        return fail_args(HM_ERR_INVALID_ARG, "rotary: rot=%d must be even, from 2 to d=%d", a->rot, a->d);
    if (a->d > 1024) return fail_args(HM_ERR_UNSUPPORTED, "rotary: d=%d > 1024", a->d);
    if (a->B > (1LL << 30) || a->L > (1LL << 30) || a->B * a->L > (1LL << 30))
        return fail_args(HM_ERR_UNSUPPORTED, "rotary: need B L <= 2^30");
    if (!finite_positive(a->base)) return fail_args(HM_ERR_INVALID_ARG, "rotary: base must be > 0");
    if (!(a->mscale - a->mscale == 0.0)) return fail_args(HM_ERR_INVALID_ARG, "rotary: mscale must be finite");
    if (a->scaling != HM_ROTARY_PLAIN && !finite_positive(a->factor))
        return fail_args(HM_ERR_INVALID_ARG, "rotary: this scaling needs factor > 0");
    if (a->scaling == HM_ROTARY_NTK && a->rot <= 2)
        return fail_args(HM_ERR_INVALID_ARG, "rotary: NTK scaling needs rot > 2");
    if (a->scaling == HM_ROTARY_BY_PARTS &&
        (!finite_positive(a->orig_len) || !(a->beta_fast > a->beta_slow) ||
         !(a->beta_fast - a->beta_slow < HUGE_VAL)))
        return fail_args(HM_ERR_INVALID_ARG, "rotary: scaling by parts needs orig_len > 0 and beta_fast > beta_slow");
    if (((uintptr_t)a->positions & 7) != 0) return fail_args(HM_ERR_INVALID_ARG, "rotary: misaligned positions");
    const size_t es = esize(a->io_dtype);
    const int64_t is[2][3] = {{a->q_stride_b, a->q_stride_t, a->q_stride_h}, {a->k_stride_b, a->k_stride_t, a->k_stride_h}};
    const int64_t os[2][3] = {{a->q_out_stride_b, a->q_out_stride_t, a->q_out_stride_h},
                              {a->k_out_stride_b, a->k_out_stride_t, a->k_out_stride_h}};
    hm_status st = check_side("q", a->q, a->q_out, a->Hq, a->B, a->L, a->d, es, is[0], os[0]);
    if (st != HM_OK) return st;
    st = check_side("k", a->k, a->k_out, a->Hk, a->B, a->L, a->d, es, is[1], os[1]);
    if (st != HM_OK) return st;
    if (a->B == 0 || a->L == 0 || a->Hq + a->Hk == 0) return HM_OK;

    RotArgs r{};
    r.s[0] = {a->q, a->q_out, is[0][0], is[0][1], is[0][2], os[0][0], os[0][1], os[0][2]};
    r.s[1] = {a->k, a->k_out, is[1][0], is[1][1], is[1][2], os[1][0], os[1][1], os[1][2]};
    r.Hq = a->Hq;
    r.H = a->Hq + a->Hk;
    r.L = a->L;
    r.tokens = (unsigned)(a->B * a->L);
    r.d = a->d;
    r.rot = a->rot;
    r.positions = a->positions;
    r.pos_b = a->pos_stride_b;
    r.pos_t = a->pos_stride_t;
    r.pos0 = a->pos0;
    r.log2_base = log2(a->base);
    if (a->scaling == HM_ROTARY_NTK) r.log2_base += log2(a->factor) * a->rot / (a->rot - 2);
    r.inv_factor = a->scaling == HM_ROTARY_LINEAR || a->scaling == HM_ROTARY_BY_PARTS ? 1.0 / a->factor : 1.0;
    r.by_parts = a->scaling == HM_ROTARY_BY_PARTS;
    if (r.by_parts) {
        r.turns0 = a->orig_len * 0.15915494309189533577;
        r.slow = a->beta_slow;
        r.inv_span = 1.0 / (a->beta_fast - a->beta_slow);
    }
    r.mscale = (float)a->mscale;
    r.sign = a->transpose ? -1.f : 1.f;
    const bool copy = a->rot < a->d && !((a->Hq == 0 || a->q == a->q_out) && (a->Hk == 0 || a->k == a->k_out));
    // the widest pieces that the pair count, the rest of the head and every row start allow
    int P = a->io_dtype == HM_BF16 ? 8 : 4;
    auto fits = [&](int n) {
        if (a->rot / 2 % n || (copy && a->d % n)) return false;
        const void *ptr[2][2] = {{a->q, a->q_out}, {a->k, a->k_out}};
        const int64_t cnt[3] = {a->B, a->L, 0};
        for (int i = 0; i < 2; ++i) {
            const int H = i ? a->Hk : a->Hq;
            if (H == 0) continue;
            for (int j = 0; j < 2; ++j) {
                if ((uintptr_t)ptr[i][j] % (n * es)) return false;
                for (int k = 0; k < 3; ++k)
                    if ((k < 2 ? cnt[k] : H) > 1 && (j ? os : is)[i][k] % n) return false;
            }
        }
        return true;
    };
    while (P > 1 && !fits(P)) P /= 2;
    r.ng = a->rot / 2 / P;
    r.nt = copy ? (a->d - a->rot + 2 * P - 1) / (2 * P) : 0;
    // runs of all heads once that fills the GPU, shorter ones before
    r.hg = r.H;
    while (r.hg > kBatch && (int64_t)r.tokens * r.ng * ((r.H + r.hg - 1) / r.hg) < 148 * 1024) r.hg = (r.hg + 1) / 2;
    const int64_t per = (int64_t)((r.H + r.hg - 1) / r.hg) * (r.ng + r.nt);
    if (per > (1 << 24)) return fail_args(HM_ERR_UNSUPPORTED, "rotary: too many heads");
    r.per = (int)per;
    r.tb = r.per >= kThreads ? 1 : kThreads / r.per;
    const unsigned grid = (r.tokens + r.tb - 1) / r.tb;
    cudaStream_t s = (cudaStream_t)stream;
    const bool inter = a->layout == HM_ROTARY_INTERLEAVED;
#define HM_ROT(T, N)                                                     \
    (inter ? rotary_kernel<T, N, true><<<grid, kThreads, 0, s>>>(r)      \
           : rotary_kernel<T, N, false><<<grid, kThreads, 0, s>>>(r))
    if (a->io_dtype == HM_BF16) P == 8 ? HM_ROT(__nv_bfloat16, 8) : P == 4 ? HM_ROT(__nv_bfloat16, 4) : P == 2 ? HM_ROT(__nv_bfloat16, 2) : HM_ROT(__nv_bfloat16, 1);
    else P == 4 ? HM_ROT(float, 4) : P == 2 ? HM_ROT(float, 2) : HM_ROT(float, 1);
#undef HM_ROT
    count_launches(1);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? HM_OK : fail_args(HM_ERR_CUDA, "rotary launch: %s", cudaGetErrorString(e));
}
