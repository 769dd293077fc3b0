// gated_scan.cu -- the channel-wise gated recurrence: forward, backward, one
// token (hm_gated_scan_fwd, _bwd, _step).
//
//   z = dt + bias, Delta = softplus(z), a = exp(-Delta exp(A_log))
//   h_t = a_t h_{t-1} + beta_t x_t
//
// A thread per (sequence, channel) walks the tokens.  The forward stores the
// state in front of every 64th token; the backward walks the chunks from the
// end, recomputes the 64 states of each from there and runs the adjoint
// g_t = dy_t + a_{t+1} g_{t+1} back through them.
#include <type_traits>

#include "hm_internal.h"

namespace hm {

namespace {

constexpr int kChunk = 64;   // tokens between two stored states

struct Gate {
    float z, step, la, a, beta;
};

template <int SCALE>
__device__ __forceinline__ Gate gate_of(float dt, float bias, float rate) {
    Gate g;
    g.z = dt + bias;
    g.step = hm_softplus(g.z);
    g.la = rate == 0.f ? 0.f : -g.step * rate;
    g.a = expf(g.la);
    g.beta = SCALE == HM_INPUT_PLAIN ? 1.f : SCALE == HM_INPUT_STEP ? g.step : sqrtf(-expm1f(2.f * g.la));
    return g;
}

__device__ __forceinline__ int64_t clamped_len(const int32_t *lengths, int64_t b, int64_t L) {
    if (!lengths) return L;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n > L ? L : n;
}

template <typename T, int SCALE>
__global__ void __launch_bounds__(128) gated_fwd_kernel(hm_gated_scan_args p) {
    const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= p.D) return;
    const float rate = expf(p.A_log[c]), bias = p.dt_bias ? p.dt_bias[c] : 0.f;
    const int64_t nchunk = (p.L + kChunk - 1) / kChunk;
    for (int64_t b = blockIdx.y; b < p.B; b += gridDim.y) {
        const int64_t n = clamped_len(p.lengths, b, p.L);
        const T *x = (const T *)p.x + b * p.x_stride_b + c;
        const T *dt = (const T *)p.dt + b * p.dt_stride_b + c;
        T *y = (T *)p.y + b * p.y_stride_b + c;
        float h = p.h0 ? p.h0[b * p.D + c] : 0.f;
        for (int64_t t = 0; t < n; ++t) {
            if (p.states && t % kChunk == 0) ((float *)p.states)[(b * nchunk + t / kChunk) * p.D + c] = h;
            const Gate g = gate_of<SCALE>(hm_ld(dt, t * p.dt_stride_t), bias, rate);
            h = fmaf(g.a, h, g.beta * hm_ld(x, t * p.x_stride_t));
            if (p.y) hm_st(y, t * p.y_stride_t, h);
        }
        if (p.h_out) p.h_out[b * p.D + c] = h;
    }
}

// partial sums of dA_log and d_dt_bias: part[(b * 2 + k) * D + c]
template <typename T, int SCALE>
__global__ void __launch_bounds__(128) gated_bwd_kernel(hm_gated_scan_bwd_args p, float *part) {
    const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= p.D) return;
    const float rate = expf(p.A_log[c]), bias = p.dt_bias ? p.dt_bias[c] : 0.f;
    const int64_t nchunk = (p.L + kChunk - 1) / kChunk;
    for (int64_t b = blockIdx.y; b < p.B; b += gridDim.y) {
        const int64_t n = clamped_len(p.lengths, b, p.L);
        const T *x = (const T *)p.x + b * p.x_stride_b + c;
        const T *dt = (const T *)p.dt + b * p.dt_stride_b + c;
        const T *dy = (const T *)p.dy + b * p.dy_stride_b + c;
        T *dx = (T *)p.dx + b * p.dx_stride_b + c;
        T *ddt = (T *)p.ddt + b * p.ddt_stride_b + c;
        float carry = p.dh_out ? p.dh_out[b * p.D + c] : 0.f, sA = 0.f, sb = 0.f;
        float hs[kChunk];
        for (int64_t k = (n + kChunk - 1) / kChunk - 1; k >= 0; --k) {
            const int64_t t0 = k * kChunk;
            const int m = (int)(n - t0 < kChunk ? n - t0 : kChunk);
            float h = ((const float *)p.states)[(b * nchunk + k) * p.D + c];
            for (int i = 0; i < m; ++i) {
                hs[i] = h;
                const Gate g = gate_of<SCALE>(hm_ld(dt, (t0 + i) * p.dt_stride_t), bias, rate);
                h = fmaf(g.a, h, g.beta * hm_ld(x, (t0 + i) * p.x_stride_t));
            }
            float cA = 0.f, cb = 0.f;
            for (int i = m - 1; i >= 0; --i) {
                const int64_t t = t0 + i;
                const Gate q = gate_of<SCALE>(hm_ld(dt, t * p.dt_stride_t), bias, rate);
                const float xv = hm_ld(x, t * p.x_stride_t);
                const float g = hm_ld(dy, t * p.dy_stride_t) + carry;
                carry = q.a * g;
                float dla = carry * hs[i];
                if (SCALE == HM_INPUT_UNIT && q.beta > 0.f) dla -= g * xv * q.a * q.a / q.beta;
                float dstep = -rate * dla;
                if (SCALE == HM_INPUT_STEP) dstep += g * xv;
                const float dz = dstep / (1.f + expf(-q.z));
                hm_st(dx, t * p.dx_stride_t, g * q.beta);
                hm_st(ddt, t * p.ddt_stride_t, dz);
                cA = fmaf(dla, q.la, cA);
                cb += dz;
            }
            sA += cA;
            sb += cb;
        }
        part[(b * 2 + 0) * p.D + c] = sA;
        part[(b * 2 + 1) * p.D + c] = sb;
        if (p.dh0) p.dh0[b * p.D + c] = carry;
    }
}

__global__ void __launch_bounds__(128) gated_sum_kernel(const float *part, int64_t rows, int64_t D, float *dA,
                                                        float *db) {
    const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= D) return;
    float sA = 0.f, sb = 0.f;
    for (int64_t r = 0; r < rows; ++r) {
        sA += part[(r * 2 + 0) * D + c];
        sb += part[(r * 2 + 1) * D + c];
    }
    dA[c] = sA;
    if (db) db[c] = sb;
}

template <typename T, int SCALE>
__global__ void __launch_bounds__(256) gated_step_kernel(hm_gated_step_args p) {
    const int64_t n = p.B * p.D;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t b = i / p.D, c = i - b * p.D;
        const Gate g = gate_of<SCALE>(hm_ld((const T *)p.dt, b * p.dt_stride + c), p.dt_bias ? p.dt_bias[c] : 0.f,
                                      expf(p.A_log[c]));
        const float h = fmaf(g.a, p.h[i], g.beta * hm_ld((const T *)p.x, b * p.x_stride + c));
        p.h_out[i] = h;
        hm_st((T *)p.y, b * p.y_stride + c, h);
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
    if (B > (1LL << 31) || L > (1LL << 31) || D > (1LL << 24) || B * L > (1LL << 40))
        return fail_args(HM_ERR_UNSUPPORTED, "%s: need B, L <= 2^31, B L <= 2^40 and D <= 2^24", who);
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

size_t bwd_workspace(const hm_gated_scan_bwd_args *a) {
    return (size_t)(a->B * 2 * a->D) * sizeof(float);
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

unsigned grid_y(int64_t B) { return (unsigned)(B < 65535 ? B : 65535); }

}  // namespace

}  // namespace hm

using namespace hm;

extern "C" size_t hm_gated_scan_states_size(const hm_gated_scan_args *a) {
    if (!a || check_common("gated_scan", a->B, a->L, a->D, a->io_dtype, a->input_scale) != HM_OK) return 0;
    return states_bytes(a->B, a->L, a->D);
}

extern "C" hm_status hm_gated_scan_fwd(const hm_gated_scan_args *a, hm_stream_t stream) {
    set_error_detail("");
    HM_TRY(check_fwd(a));
    if (a->B == 0) return HM_OK;
    const dim3 grid((unsigned)((a->D + 127) / 128), grid_y(a->B));
    const cudaError_t e = by_type(a->io_dtype, a->input_scale, [&](auto *t, auto sc) {
        using T = std::remove_pointer_t<decltype(t)>;
        gated_fwd_kernel<T, decltype(sc)::value><<<grid, 128, 0, (cudaStream_t)stream>>>(*a);
        count_launches(1);
        return cudaGetLastError();
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
    const unsigned gx = (unsigned)((a->D + 127) / 128);
    cudaError_t e = cudaSuccess;
    if (a->B > 0)
        e = by_type(a->io_dtype, a->input_scale, [&](auto *t, auto sc) {
            using T = std::remove_pointer_t<decltype(t)>;
            gated_bwd_kernel<T, decltype(sc)::value>
                <<<dim3(gx, grid_y(a->B)), 128, 0, s>>>(*a, (float *)a->workspace);
            count_launches(1);
            return cudaGetLastError();
        });
    if (e == cudaSuccess) {
        gated_sum_kernel<<<gx, 128, 0, s>>>((const float *)a->workspace, a->B, a->D, a->dA_log, a->d_dt_bias);
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
    const int64_t blocks = (a->B * a->D + 255) / 256;
    const cudaError_t e = by_type(a->io_dtype, a->input_scale, [&](auto *t, auto sc) {
        using T = std::remove_pointer_t<decltype(t)>;
        gated_step_kernel<T, decltype(sc)::value>
            <<<(unsigned)(blocks < 148 * 32 ? blocks : 148 * 32), 256, 0, (cudaStream_t)stream>>>(*a);
        count_launches(1);
        return cudaGetLastError();
    });
    return e == cudaSuccess ? HM_OK : fail_args(HM_ERR_CUDA, "%s launch: %s", w, cudaGetErrorString(e));
}
