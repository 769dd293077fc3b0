// rotary.cu -- rotary positions on queries and keys (hm_rotary).
//
// A thread takes P pairs (P = 8 bf16, 4 fp32: two 16-byte loads) of one token
// and turns them in a run of heads: the angle depends on the token and the
// pair alone, so its sine and cosine are formed once per run.  Angles are
// kept as fractions of a turn in 64-bit fixed point: theta / (2 pi) mod 1
// times 2^64 is an integer, and the product with the position wraps modulo
// 2^64, which is the reduction modulo whole turns, exactly.
#include <math.h>

#include "hm_internal.h"

namespace hm {

namespace {

struct Side {             // q or k
    const void *in;
    void *out;
    int64_t in_b, in_t, in_h, out_b, out_t, out_h;
    int H;
};

struct RotArgs {
    Side s[2];
    int64_t B, L;
    int d, rot;
    int runs_q, runs;     // runs of kHeads heads of q, of q and k
    bool copy_tail;
    const int64_t *positions;
    int64_t pos_b, pos_t, pos0;
    double log2_base;     // of the base in use (HM_ROTARY_NTK has put its factor in)
    double inv_factor;    // frequencies times this (linear), or the by-parts blend's low end
    double turns0;        // by parts: orig_len / (2 pi)
    double slow, inv_span;
    int by_parts;
    float mscale, sign;
};

constexpr int kHeads = 4;   // heads a thread turns by the same angles

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

template <typename T, int P, bool INTER>
__global__ void __launch_bounds__(256) rotary_kernel(RotArgs a) {
    const int half = a.rot / 2, ng = (half + P - 1) / P;            // groups of P pairs
    const int nt = a.copy_tail ? (a.d - a.rot + 2 * P - 1) / (2 * P) : 0;   // groups behind rot
    const int64_t per = (int64_t)a.runs * (ng + nt);
    const int64_t n = a.B * a.L * per;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t tok = i / per;
        const int rest = (int)(i - tok * per), run = rest / (ng + nt), grp = rest - run * (ng + nt);
        const int64_t b = tok / a.L, t = tok - b * a.L;
        const Side &s = run < a.runs_q ? a.s[0] : a.s[1];
        const int h0 = (run < a.runs_q ? run : run - a.runs_q) * kHeads;
        const T *in = (const T *)s.in + b * s.in_b + t * s.in_t;
        T *out = (T *)s.out + b * s.out_b + t * s.out_t;
        if (grp >= ng) {
            const int c0 = a.rot + (grp - ng) * 2 * P;
            for (int h = h0; h < s.H && h < h0 + kHeads; ++h)
                for (int c = c0; c < c0 + 2 * P && c < a.d; ++c) out[h * s.out_h + c] = in[h * s.in_h + c];
            continue;
        }
        const int64_t pos = a.positions ? a.positions[b * a.pos_b + t * a.pos_t] : a.pos0 + t;
        float cs[P], sn[P];
#pragma unroll
        for (int j = 0; j < P; ++j) turn_of(a, pair_turns(a, grp * P + j), pos, cs[j], sn[j]);
        for (int h = h0; h < s.H && h < h0 + kHeads; ++h)
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int pr = grp * P + j;
                if (pr >= half) break;
                const int iu = INTER ? 2 * pr : pr, iv = INTER ? 2 * pr + 1 : pr + half;
                const float u = hm_ld(in, h * s.in_h + iu), v = hm_ld(in, h * s.in_h + iv);
                hm_st(out, h * s.out_h + iu, u * cs[j] - v * sn[j]);
                hm_st(out, h * s.out_h + iv, u * sn[j] + v * cs[j]);
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
    if (a->B > (1LL << 31) || a->L > (1LL << 31) || a->B * a->L > (1LL << 36))
        return fail_args(HM_ERR_UNSUPPORTED, "rotary: need B, L <= 2^31 and B L <= 2^36");
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
    r.s[0] = {a->q, a->q_out, is[0][0], is[0][1], is[0][2], os[0][0], os[0][1], os[0][2], a->Hq};
    r.s[1] = {a->k, a->k_out, is[1][0], is[1][1], is[1][2], os[1][0], os[1][1], os[1][2], a->Hk};
    r.B = a->B;
    r.L = a->L;
    r.d = a->d;
    r.rot = a->rot;
    r.runs_q = (a->Hq + kHeads - 1) / kHeads;
    r.runs = r.runs_q + (a->Hk + kHeads - 1) / kHeads;
    r.copy_tail = a->rot < a->d && !((a->Hq == 0 || a->q == a->q_out) && (a->Hk == 0 || a->k == a->k_out));
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
    const int P = a->io_dtype == HM_BF16 ? 8 : 4;
    const int64_t per = (int64_t)r.runs * ((a->rot / 2 + P - 1) / P + (r.copy_tail ? (a->d - a->rot + 2 * P - 1) / (2 * P) : 0));
    const int64_t blocks = (a->B * a->L * per + 255) / 256;
    const unsigned grid = (unsigned)(blocks < (1 << 30) ? blocks : (1 << 30));
    cudaStream_t s = (cudaStream_t)stream;
    const bool inter = a->layout == HM_ROTARY_INTERLEAVED;
    if (a->io_dtype == HM_BF16) {
        if (inter) rotary_kernel<__nv_bfloat16, 8, true><<<grid, 256, 0, s>>>(r);
        else rotary_kernel<__nv_bfloat16, 8, false><<<grid, 256, 0, s>>>(r);
    } else {
        if (inter) rotary_kernel<float, 4, true><<<grid, 256, 0, s>>>(r);
        else rotary_kernel<float, 4, false><<<grid, 256, 0, s>>>(r);
    }
    count_launches(1);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? HM_OK : fail_args(HM_ERR_CUDA, "rotary launch: %s", cudaGetErrorString(e));
}
