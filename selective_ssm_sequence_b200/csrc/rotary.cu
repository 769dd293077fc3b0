// rotary.cu -- rotary positions on queries and keys (hm_rotary).
//
// Bandwidth-bound: every element read and written once (32768 tokens of 16 heads
// of 256 in bf16, or 16384 in fp32: 87 us, 0.94 of the copy rate).  A thread takes P
// pairs (P = 8 of bf16, 4 of fp32: two 16-byte loads; fewer where strides or
// the pair count ask for it) of one token and turns them in up to four heads,
// q's and then k's, whose loads are in flight together: the angle depends on
// the token and the pair alone, so its sine and cosine are formed once for the
// four.  Its two pieces of a head lie half of rot apart in both layouts: the
// pairs' halves (half layout), or two times P / 2 whole pairs (interleaved), so
// that a warp's accesses are contiguous either way.
//
// Angles are kept as fractions of a turn in 64-bit fixed point: theta / (2 pi)
// mod 1 times 2^64 is an integer (formed in fp64, once per block, in shared
// memory), and its product with the position wraps modulo 2^64, which is the
// reduction modulo whole turns, exactly.
#include <math.h>

#include "packed.cuh"

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
constexpr int kHeads = 4;   // heads of a run

// theta_i / (2 pi) mod 1, in units of 2^-64 of a turn: off by half a unit, and
// theta_i by log2(base) 2^-51.5 + 2^-50 of itself (the exponent's three roundings,
// exp2, and at most five operations behind it), below 2^-47 for bases up to 2^20.
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

// Cosine (times mscale) and sine (times mscale and the direction) of pos times
// the pair's frequency.  The nearest quarter turn goes into signs and an
// exchange, the rest, x in [-pi/4, pi/4], into polynomials of least maximal
// error fitted there, whose coefficients in fp32 give sin x = x + x^3 S(x^2) to
// 8.4e-9 of it and cos x = 1 - x^2 / 2 + x^4 C(x^2) to 7.1e-10.
__device__ __forceinline__ void turn_of(const RotArgs &a, unsigned long long unit, int64_t pos, float &cs, float &sn) {
    const unsigned ph = (unsigned)((unit * (unsigned long long)pos) >> 32);
    const unsigned quarter = (ph + 0x20000000u) >> 30;
    const float x = (float)(int)(ph - (quarter << 30)) * 1.46291807926715968e-09f;   // 2 pi / 2^32
    const float q = x * x;
    float s = fmaf(-1.951528392964974e-04f, q, 8.33216030150652e-03f);
    s = fmaf(s, q, -1.6666655242443085e-01f);
    s = fmaf(s * q, x, x);
    float c = fmaf(2.4438451873720624e-05f, q, -1.388736767694354e-03f);
    c = fmaf(c, q, 4.166664555668831e-02f);
    c = fmaf(c, q, -0.5f);
    c = fmaf(c, q, 1.f);
    const float p = quarter & 1 ? c : s, r = quarter & 1 ? s : c;
    sn = (quarter & 2 ? -p : p) * (a.mscale * a.sign);
    cs = ((quarter + 1) & 2 ? -r : r) * a.mscale;
}

// P elements, P * sizeof(T) = 2 .. 16 bytes, as words (or one half word)
template <typename T, int P>
struct Vec {
    static constexpr int N = P * (int)sizeof(T) / 4;
    uint32_t w[N];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (N == 4) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else if constexpr (N == 2) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x, w[1] = u.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (N == 4) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (N == 2) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t *>(p) = w[0];
    }
    // elements 2 j and 2 j + 1 (P > 1)
    __device__ __forceinline__ F2 pair(int j) const {
        if constexpr (sizeof(T) == 2) return pk_bf16(w[j]);
        else return pk(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    }
    __device__ __forceinline__ void set(int j, F2 v) {
        if constexpr (sizeof(T) == 2) {
            w[j] = bf16_of(v);
        } else {
            w[2 * j] = __float_as_uint(un(v).x);
            w[2 * j + 1] = __float_as_uint(un(v).y);
        }
    }
    __device__ __forceinline__ float one() const { return __uint_as_float(w[0]); }
    __device__ __forceinline__ void one(float v) { w[0] = __float_as_uint(v); }
};
template <>
struct Vec<__nv_bfloat16, 1> {
    __nv_bfloat16 v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = *p; }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *p = v; }
    __device__ __forceinline__ F2 pair(int) const { return splat(0.f); }
    __device__ __forceinline__ void set(int, F2) {}
    __device__ __forceinline__ float one() const { return __bfloat162float(v); }
    __device__ __forceinline__ void one(float f) { v = __float2bfloat16_rn(f); }
};

// the head's rows in and out
template <typename T>
__device__ __forceinline__ void head_of(const RotArgs &a, int h, int64_t b, int64_t t, const T *&in, T *&out) {
    const Side &s = h < a.Hq ? a.s[0] : a.s[1];
    const int i = h < a.Hq ? h : h - a.Hq;
    in = (const T *)s.in + b * s.in_b + t * s.in_t + i * s.in_h;
    out = (T *)s.out + b * s.out_b + t * s.out_t + i * s.out_h;
}

template <typename T, int P, bool INTER>
__global__ void __launch_bounds__(kThreads, 3) rotary_kernel(const __grid_constant__ RotArgs a) {
    __shared__ unsigned long long unit[512];
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < half; i += kThreads) unit[i] = pair_turns(a, i);
    __syncthreads();
    using V = Vec<T, P>;
    const int groups = a.ng + a.nt;
    for (unsigned tok0 = blockIdx.x * (unsigned)a.tb; tok0 < a.tokens; tok0 += gridDim.x * (unsigned)a.tb)
        for (int i = threadIdx.x; i < a.tb * a.per; i += kThreads) {
            const int local = i / a.per, rest = i - local * a.per, run = rest / groups, grp = rest - run * groups;
            const unsigned tok = tok0 + local;
            if (tok >= a.tokens) break;
            const int64_t b = tok / (unsigned)a.L, t = tok - (unsigned)b * (unsigned)a.L;
            const int h0 = run * kHeads;
            // columns of the two pieces: of a rotated group, or of one behind rot
            const bool tail = grp >= a.ng;
            const int iu = tail ? a.rot + (grp - a.ng) * 2 * P : INTER && P == 1 ? 2 * grp : grp * P;
            const int iv = tail ? iu + P : INTER && P == 1 ? iu + 1 : iu + half;
            const bool two = iv + P <= a.d;
            V u[kHeads], v[kHeads];
            T *out[kHeads];
#pragma unroll
            for (int k = 0; k < kHeads; ++k)
                if (h0 + k < a.H) {
                    const T *in;
                    head_of(a, h0 + k, b, t, in, out[k]);
                    u[k].load(in + iu);
                    if (two) v[k].load(in + iv);
                }
            if (!tail) {
                const int64_t pos = a.positions ? a.positions[b * a.pos_b + t * a.pos_t] : a.pos0 + t;
                float cs[P], sn[P];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int pair = !INTER || P == 1 ? grp * P + j
                                     : j < P / 2 ? grp * (P / 2) + j : (half + grp * P) / 2 + j - P / 2;
                    turn_of(a, unit[pair], pos, cs[j], sn[j]);
                }
#pragma unroll
                for (int k = 0; k < kHeads; ++k) {
                    if (P == 1) {
                        const float x = u[k].one(), y = v[k].one();
                        u[k].one(x * cs[0] - y * sn[0]);
                        v[k].one(x * sn[0] + y * cs[0]);
                    } else if (INTER) {
#pragma unroll
                        for (int j = 0; j < P; ++j) {      // pair j is elements 2 j, 2 j + 1 of its piece
                            V &w = j < P / 2 ? u[k] : v[k];
                            const float2 x = un(w.pair(j % (P / 2 > 0 ? P / 2 : 1)));
                            w.set(j % (P / 2 > 0 ? P / 2 : 1),
                                  pk(x.x * cs[j] - x.y * sn[j], x.x * sn[j] + x.y * cs[j]));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < P / 2; ++j) {  // two pairs at once
                            const F2 x = u[k].pair(j), y = v[k].pair(j);
                            const F2 c = pk(cs[2 * j], cs[2 * j + 1]), s = pk(sn[2 * j], sn[2 * j + 1]);
                            u[k].set(j, fma(x, c, y * pk(-sn[2 * j], -sn[2 * j + 1])));
                            v[k].set(j, fma(x, s, y * c));
                        }
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kHeads; ++k)
                if (h0 + k < a.H) {
                    u[k].store(out[k] + iu);
                    if (two) v[k].store(out[k] + iv);
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
    if (a->Hq > 0 && a->Hk > 0 && (a->q_out == a->k_out || a->q_out == a->k || a->k_out == a->q))
        return fail_args(HM_ERR_INVALID_ARG, "rotary: q_out or k_out is the other's array");

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
    const int64_t per = (int64_t)((r.H + kHeads - 1) / kHeads) * (r.ng + r.nt);
    if (per > (1 << 24)) return fail_args(HM_ERR_UNSUPPORTED, "rotary: too many heads");
    r.per = (int)per;
    r.tb = r.per >= kThreads ? 1 : kThreads / r.per;
    // blocks walk the tokens, so that the frequencies are formed once per block
    const unsigned blocks = (r.tokens + r.tb - 1) / r.tb;
    // (one wave where there is little to do, else shorter shares: 8192 tokens, a quarter of 16 heads
    // of 256: 3, 6, 12 blocks per SM 27.4, 29.0, 29.0 us; 32768 whole heads 101, 94, 88)
    const unsigned most = 148 * (blocks < 148 * 32 ? 3 : 12), grid = blocks < most ? blocks : most;
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
