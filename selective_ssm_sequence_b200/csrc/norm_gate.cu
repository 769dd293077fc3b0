// norm_gate.cu -- the seam between two blocks (hm_norm_gate_fwd, _bwd):
// post-norm, SiLU gate, scaled residual sum and the next block's pre-norm.
//
// Bandwidth-bound: five row arrays forward, eight backward, each touched once.
// A block of threads holds a row in registers: statistics come from there
// (mean first, then the centred squares), so nothing is read twice.  In the
// backward each thread keeps its columns' parameter gradients in registers
// over all its rows; the blocks' shares are summed in a second, small kernel
// in a fixed order.
#include "hm_internal.h"

namespace hm {

namespace {

constexpr int kE = 8;   // elements of a thread per piece

// Columns of thread `tid`: with VEC pieces of 8 consecutive elements, else
// single elements a block's width apart (both coalesced).
template <bool VEC>
__device__ __forceinline__ int col_of(int piece, int j, int tid, int nthr) {
    return VEC ? (piece * nthr + tid) * kE + j : (piece * kE + j) * nthr + tid;
}

__device__ __forceinline__ void unpack8(const __nv_bfloat16 *p, float *f) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack8(const float *p, float *f) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void pack8(__nv_bfloat16 *p, const float *f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack8(float *p, const float *f) {
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T *row, int piece, int tid, int nthr, int D, float *f) {
    if (VEC) {
        const int c = col_of<true>(piece, 0, tid, nthr);
        if (c < D) {
            unpack8(row + c, f);
            return;
        }
#pragma unroll
        for (int j = 0; j < kE; ++j) f[j] = 0.f;
    } else {
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            const int c = col_of<false>(piece, j, tid, nthr);
            f[j] = c < D ? hm_ld(row, c) : 0.f;
        }
    }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T *row, int piece, int tid, int nthr, int D, const float *f) {
    if (VEC) {
        const int c = col_of<true>(piece, 0, tid, nthr);
        if (c < D) pack8(row + c, f);
    } else {
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            const int c = col_of<false>(piece, j, tid, nthr);
            if (c < D) hm_st(row, c, f[j]);
        }
    }
}

// fp32 parameters of a thread's columns (any 4-byte alignment), or the default
template <bool VEC>
__device__ __forceinline__ void param8(const float *p, float dflt, int piece, int tid, int nthr, int D, float *f) {
#pragma unroll
    for (int j = 0; j < kE; ++j) {
        const int c = col_of<VEC>(piece, j, tid, nthr);
        f[j] = p && c < D ? p[c] : dflt;
    }
}

// Sum over the block of two values; every thread gets them.  `red` holds 2 x
// 32 floats and alternates, so one barrier per call is enough: a call's reads
// are separated from the next-but-one call's writes by the next call's barrier.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2 (*red)[32], int &turn) {
    a = warp_sum(a);
    b = warp_sum(b);
    const int nw = blockDim.x >> 5;
    if (nw > 1) {
        float2 *r = red[turn & 1];
        ++turn;
        if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const float2 v = (threadIdx.x & 31) < nw ? r[threadIdx.x & 31] : make_float2(0.f, 0.f);
        a = warp_sum(v.x);
        b = warp_sum(v.y);
    }
    return make_float2(a, b);
}

// mean (0 for RMS) and 1 / sqrt(mean square + eps) of up to two rows at once
template <bool VEC, int NV>
__device__ __forceinline__ void stats2(const float (*u)[kE], const float (*v)[kE], bool layer, int D, float eps,
                                       float2 (*red)[32], int &turn, float2 &mean, float2 &rstd) {
    const int tid = threadIdx.x, n = blockDim.x;
    mean = make_float2(0.f, 0.f);
    if (layer) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                a += u[k][j];
                if (v) b += v[k][j];
            }
        mean = block_sum2(a, b, red, turn);
        mean.x /= (float)D;
        mean.y /= (float)D;
    }
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < kE; ++j)
            if (col_of<VEC>(k, j, tid, n) < D) {
                const float d = u[k][j] - mean.x;
                a = fmaf(d, d, a);
                if (v) {
                    const float e = v[k][j] - mean.y;
                    b = fmaf(e, e, b);
                }
            }
    const float2 q = block_sum2(a, b, red, turn);
    rstd.x = rsqrtf(q.x / (float)D + eps);
    rstd.y = rsqrtf(q.y / (float)D + eps);
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

template <typename T, bool VEC, int NV>
__global__ void __launch_bounds__(1024) norm_gate_fwd_kernel(hm_norm_gate_args p) {
    __shared__ float2 red[2][32];
    int turn = 0;
    const int tid = threadIdx.x, nthr = blockDim.x, D = (int)p.D;
    const bool layer = p.norm == HM_NORM_LAYER;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        float u[NV][kE], r[NV][kE], g[NV][kE], w[kE], c[kE];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            load8<VEC>((const T *)p.y + row * p.y_stride, k, tid, nthr, D, u[k]);
            if (p.gate) load8<VEC>((const T *)p.gate + row * p.gate_stride, k, tid, nthr, D, g[k]);
            if (p.r) load8<VEC>((const T *)p.r + row * p.r_stride, k, tid, nthr, D, r[k]);
            else
#pragma unroll
                for (int j = 0; j < kE; ++j) r[k][j] = 0.f;
        }
        float2 mean, rstd;
        if (p.post) {
            stats2<VEC, NV>(u, nullptr, layer, D, p.eps, red, turn, mean, rstd);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                param8<VEC>(p.post_w, 1.f, k, tid, nthr, D, w);
                param8<VEC>(p.post_b, 0.f, k, tid, nthr, D, c);
#pragma unroll
                for (int j = 0; j < kE; ++j) u[k][j] = fmaf((u[k][j] - mean.x) * rstd.x, w[j], c[j]);
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            param8<VEC>(p.scale, 1.f, k, tid, nthr, D, w);
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                const float m = p.gate ? u[k][j] * g[k][j] * sigmoid(g[k][j]) : u[k][j];
                // columns behind D hold zero, for the sums below
                r[k][j] = col_of<VEC>(k, j, tid, nthr) < D ? fmaf(p.alpha * w[j], m, r[k][j]) : 0.f;
            }
            if (p.r_out) store8<VEC>((T *)p.r_out + row * p.r_out_stride, k, tid, nthr, D, r[k]);
        }
        if (p.xn) {
            stats2<VEC, NV>(r, nullptr, layer, D, p.eps, red, turn, mean, rstd);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                param8<VEC>(p.pre_w, 1.f, k, tid, nthr, D, w);
                param8<VEC>(p.pre_b, 0.f, k, tid, nthr, D, c);
#pragma unroll
                for (int j = 0; j < kE; ++j) r[k][j] = fmaf((r[k][j] - mean.x) * rstd.x, w[j], c[j]);
                store8<VEC>((T *)p.xn + row * p.xn_stride, k, tid, nthr, D, r[k]);
            }
        }
    }
}

// part[(blockIdx.x * 5 + i) * D + c]: this block's share of dscale, dpost_w,
// dpost_b, dpre_w, dpre_b
template <typename T, bool VEC, int NV>
__global__ void __launch_bounds__(512) norm_gate_bwd_kernel(hm_norm_gate_bwd_args p, float *part) {
    __shared__ float2 red[2][32];
    int turn = 0;
    const int tid = threadIdx.x, nthr = blockDim.x, D = (int)p.D;
    const bool layer = p.norm == HM_NORM_LAYER;
    float acc[5][NV][kE];
#pragma unroll
    for (int i = 0; i < 5; ++i)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < kE; ++j) acc[i][k][j] = 0.f;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        float y[NV][kE], r[NV][kE], d[NV][kE], e[NV][kE], g[NV][kE], w[kE], c[kE];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            load8<VEC>((const T *)p.y + row * p.y_stride, k, tid, nthr, D, y[k]);
            if (p.gate) load8<VEC>((const T *)p.gate + row * p.gate_stride, k, tid, nthr, D, g[k]);
            if (p.dxn) {
                load8<VEC>((const T *)p.r_out + row * p.r_out_stride, k, tid, nthr, D, r[k]);
                load8<VEC>((const T *)p.dxn + row * p.dxn_stride, k, tid, nthr, D, e[k]);
            }
            if (p.dr_out) load8<VEC>((const T *)p.dr_out + row * p.dr_out_stride, k, tid, nthr, D, d[k]);
            else
#pragma unroll
                for (int j = 0; j < kE; ++j) d[k][j] = 0.f;
        }
        float2 mean = make_float2(0.f, 0.f), rstd = make_float2(1.f, 1.f);
        if (p.dxn) {
            stats2<VEC, NV>(r, p.post ? y : nullptr, layer, D, p.eps, red, turn, mean, rstd);
            // dr = dr_out + rstd (w e - mean(w e) - u mean(w e u)), u = (r - mean) rstd
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                param8<VEC>(p.pre_w, 1.f, k, tid, nthr, D, w);
#pragma unroll
                for (int j = 0; j < kE; ++j) {
                    const float u = (r[k][j] - mean.x) * rstd.x;
                    acc[3][k][j] = fmaf(e[k][j], u, acc[3][k][j]);
                    acc[4][k][j] += e[k][j];
                    r[k][j] = u;
                    e[k][j] *= w[j];      // zero behind D
                    s0 += e[k][j];
                    s1 = fmaf(e[k][j], u, s1);
                }
            }
            const float2 s = block_sum2(s0, s1, red, turn);
            const float m0 = layer ? s.x / (float)D : 0.f, m1 = s.y / (float)D;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < kE; ++j) d[k][j] += rstd.x * (e[k][j] - m0 - r[k][j] * m1);
        } else if (p.post) {
            float2 m1, r1;
            stats2<VEC, NV>(y, nullptr, layer, D, p.eps, red, turn, m1, r1);
            mean.y = m1.x;
            rstd.y = r1.x;
        }
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (p.dr) store8<VEC>((T *)p.dr + row * p.dr_stride, k, tid, nthr, D, d[k]);
            float pw[kE], pb[kE];
            param8<VEC>(p.scale, 1.f, k, tid, nthr, D, c);
            param8<VEC>(p.post_w, 1.f, k, tid, nthr, D, pw);
            param8<VEC>(p.post_b, 0.f, k, tid, nthr, D, pb);
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                const bool in = col_of<VEC>(k, j, tid, nthr) < D;
                const float u = p.post ? (y[k][j] - mean.y) * rstd.y : y[k][j];
                const float n = p.post ? fmaf(u, pw[j], pb[j]) : u;
                const float dm = in ? d[k][j] * (p.alpha * c[j]) : 0.f;
                float m = n, dn = dm;
                if (p.gate) {
                    const float sg = sigmoid(g[k][j]), si = g[k][j] * sg;
                    m = n * si;
                    dn = dm * si;
                    g[k][j] = dm * n * sg * (1.f + g[k][j] * (1.f - sg));
                }
                if (in) acc[0][k][j] = fmaf(d[k][j], p.alpha * m, acc[0][k][j]);
                acc[1][k][j] = fmaf(dn, u, acc[1][k][j]);
                acc[2][k][j] += dn;
                y[k][j] = u;
                d[k][j] = p.post ? dn * pw[j] : dn;
                s0 += d[k][j];
                s1 = fmaf(d[k][j], u, s1);
            }
            if (p.gate) store8<VEC>((T *)p.dgate + row * p.dgate_stride, k, tid, nthr, D, g[k]);
        }
        if (p.post) {
            const float2 s = block_sum2(s0, s1, red, turn);
            const float m0 = layer ? s.x / (float)D : 0.f, m1 = s.y / (float)D;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < kE; ++j) d[k][j] = rstd.y * (d[k][j] - m0 - y[k][j] * m1);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) store8<VEC>((T *)p.dy + row * p.dy_stride, k, tid, nthr, D, d[k]);
    }
#pragma unroll
    for (int i = 0; i < 5; ++i)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                const int c = col_of<VEC>(k, j, tid, nthr);
                if (c < D) part[((int64_t)blockIdx.x * 5 + i) * D + c] = acc[i][k][j];
            }
}

struct GradPtrs {
    float *out[5];
};

// the blocks' shares summed in block order; a block of threads per 32 columns
// and parameter, 8 rows of it walking the shares
__global__ void __launch_bounds__(256) norm_gate_sum_kernel(const float *part, int blocks, int D, GradPtrs g) {
    __shared__ float s[8][33];
    float *out = g.out[blockIdx.y];
    if (!out) return;
    const int c = blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    if (c < D)
        for (int b = threadIdx.y; b < blocks; b += 8) v += part[((int64_t)b * 5 + blockIdx.y) * D + c];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][threadIdx.x];
        out[c] = v;
    }
}

// ------------------------------------------------------------------ host

struct Row {
    const char *name;
    const void *p;
    int64_t stride;
    bool required;
};

constexpr int64_t kMaxD = 16384;
constexpr int64_t kBwdBlocks = 148 * 2;

size_t esize(hm_dtype t) { return t == HM_BF16 ? 2 : 4; }

hm_status check_seam(const char *who, int64_t rows, int64_t D, hm_dtype t, int norm, float eps, float alpha) {
    if (t != HM_F32 && t != HM_BF16) return fail_args(HM_ERR_INVALID_ARG, "%s: bad io dtype", who);
    if (norm != HM_NORM_RMS && norm != HM_NORM_LAYER) return fail_args(HM_ERR_INVALID_ARG, "%s: bad norm %d", who, norm);
    if (rows < 0 || D < 1) return fail_args(HM_ERR_INVALID_ARG, "%s: bad sizes", who);
    if (D > kMaxD) return fail_args(HM_ERR_UNSUPPORTED, "%s: D=%lld > %lld", who, (long long)D, (long long)kMaxD);
    if (rows > (1LL << 40)) return fail_args(HM_ERR_UNSUPPORTED, "%s: rows > 2^40", who);
    if (!(eps > 0.f)) return fail_args(HM_ERR_INVALID_ARG, "%s: eps must be > 0", who);
    if (!(alpha - alpha == 0.f)) return fail_args(HM_ERR_INVALID_ARG, "%s: alpha must be finite", who);
    return HM_OK;
}

hm_status check_row(const char *who, const Row &r, int64_t rows, int64_t D, size_t es) {
    if (rows == 0) return HM_OK;
    if (!r.p) return r.required ? fail_args(HM_ERR_INVALID_ARG, "%s: null %s", who, r.name) : HM_OK;
    if (((uintptr_t)r.p & (es - 1)) != 0)
        return fail_args(HM_ERR_INVALID_ARG, "%s: %s is not aligned to its type", who, r.name);
    if (r.stride < 0 || (rows > 1 && r.stride < D))
        return fail_args(HM_ERR_INVALID_ARG, "%s: stride of %s is below D", who, r.name);
    if (r.stride > (1LL << 40)) return fail_args(HM_ERR_UNSUPPORTED, "%s: stride of %s is too large", who, r.name);
    return HM_OK;
}

bool wide(const Row &r, size_t es) {
    return !r.p || ((((uintptr_t)r.p) & 15) == 0 && (r.stride * (int64_t)es) % 16 == 0);
}

struct Shape {
    int nthr, nv;
};

// the fewest pieces per thread that 1024 threads cover the row with, then
// the fewest whole warps
Shape shape_of(int64_t D, int most) {
    int nv = 1;
    while ((int64_t)nv * kE * most < D) nv *= 2;
    const int thr = (int)((D + (int64_t)nv * kE - 1) / ((int64_t)nv * kE));
    return {(thr + 31) / 32 * 32, nv};
}

}  // namespace

}  // namespace hm

using namespace hm;

#define HM_TRY(e)                     \
    do {                              \
        const hm_status st_ = (e);    \
        if (st_ != HM_OK) return st_; \
    } while (0)

extern "C" hm_status hm_norm_gate_fwd(const hm_norm_gate_args *a, hm_stream_t stream) {
    set_error_detail("");
    const char *w = "norm_gate_fwd";
    if (!a) return fail_args(HM_ERR_INVALID_ARG, "%s: null args", w);
    HM_TRY(check_seam(w, a->rows, a->D, a->io_dtype, a->norm, a->eps, a->alpha));
    const size_t es = esize(a->io_dtype);
    const Row rows[] = {{"y", a->y, a->y_stride, true},
                        {"gate", a->gate, a->gate_stride, false},
                        {"r", a->r, a->r_stride, false},
                        {"r_out", a->r_out, a->r_out_stride, false},
                        {"xn", a->xn, a->xn_stride, false}};
    bool vec = a->D % kE == 0;
    for (const Row &r : rows) {
        HM_TRY(check_row(w, r, a->rows, a->D, es));
        vec = vec && wide(r, es);
    }
    const void *params[] = {a->scale, a->post_w, a->post_b, a->pre_w, a->pre_b};
    for (const void *q : params)
        if (((uintptr_t)q & 3) != 0) return fail_args(HM_ERR_INVALID_ARG, "%s: misaligned parameter", w);
    if (a->rows == 0) return HM_OK;
    if (!a->r_out && !a->xn) return fail_args(HM_ERR_INVALID_ARG, "%s: r_out and xn are both NULL", w);
    if (a->r_out == a->xn) return fail_args(HM_ERR_INVALID_ARG, "%s: r_out and xn are the same array", w);
    const Shape sh = shape_of(a->D, 1024);
    const unsigned grid = (unsigned)(a->rows < (1 << 30) ? a->rows : (1 << 30));
    cudaStream_t s = (cudaStream_t)stream;
#define HM_FWD(T, V, N) norm_gate_fwd_kernel<T, V, N><<<grid, sh.nthr, 0, s>>>(*a)
#define HM_FWD_N(T, V)              \
    do {                            \
        if (sh.nv == 1) HM_FWD(T, V, 1); \
        else HM_FWD(T, V, 2);       \
    } while (0)
    if (a->io_dtype == HM_BF16) {
        if (vec) HM_FWD_N(__nv_bfloat16, true);
        else HM_FWD_N(__nv_bfloat16, false);
    } else {
        if (vec) HM_FWD_N(float, true);
        else HM_FWD_N(float, false);
    }
#undef HM_FWD
#undef HM_FWD_N
    count_launches(1);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? HM_OK : fail_args(HM_ERR_CUDA, "%s launch: %s", w, cudaGetErrorString(e));
}

static int bwd_blocks(int64_t rows) { return (int)(rows < kBwdBlocks ? rows : kBwdBlocks); }

extern "C" size_t hm_norm_gate_bwd_workspace_size(const hm_norm_gate_bwd_args *a) {
    if (!a || check_seam("norm_gate_bwd", a->rows, a->D, a->io_dtype, a->norm, a->eps, a->alpha) != HM_OK) return 0;
    return (size_t)bwd_blocks(a->rows) * 5 * a->D * sizeof(float);
}

extern "C" hm_status hm_norm_gate_bwd(const hm_norm_gate_bwd_args *a, hm_stream_t stream) {
    set_error_detail("");
    const char *w = "norm_gate_bwd";
    if (!a) return fail_args(HM_ERR_INVALID_ARG, "%s: null args", w);
    HM_TRY(check_seam(w, a->rows, a->D, a->io_dtype, a->norm, a->eps, a->alpha));
    const size_t es = esize(a->io_dtype);
    const Row rows[] = {{"y", a->y, a->y_stride, true},
                        {"gate", a->gate, a->gate_stride, false},
                        {"r_out", a->dxn ? a->r_out : nullptr, a->r_out_stride, a->dxn != nullptr},
                        {"dr_out", a->dr_out, a->dr_out_stride, a->dxn == nullptr},
                        {"dxn", a->dxn, a->dxn_stride, false},
                        {"dy", a->dy, a->dy_stride, true},
                        {"dgate", a->gate ? a->dgate : nullptr, a->dgate_stride, a->gate != nullptr},
                        {"dr", a->dr, a->dr_stride, false}};
    bool vec = a->D % kE == 0;
    for (const Row &r : rows) {
        HM_TRY(check_row(w, r, a->rows, a->D, es));
        vec = vec && wide(r, es);
    }
    const void *params[] = {a->scale, a->post_w, a->post_b, a->pre_w, a->dscale, a->dpost_w, a->dpost_b, a->dpre_w,
                            a->dpre_b};
    for (const void *q : params)
        if (((uintptr_t)q & 3) != 0) return fail_args(HM_ERR_INVALID_ARG, "%s: misaligned parameter", w);
    const size_t need = hm_norm_gate_bwd_workspace_size(a);
    if (need > 0 && (!a->workspace || a->workspace_bytes < need || ((uintptr_t)a->workspace & 255) != 0))
        return fail_args(HM_ERR_INVALID_ARG, "%s: workspace of %zu bytes, 256-byte aligned, is needed", w, need);
    const Shape sh = shape_of(a->D, 512);
    const int grid = bwd_blocks(a->rows);
    cudaStream_t s = (cudaStream_t)stream;
    float *part = (float *)a->workspace;
    if (grid > 0) {
#define HM_BWD(T, V, N) norm_gate_bwd_kernel<T, V, N><<<grid, sh.nthr, 0, s>>>(*a, part)
#define HM_BWD_N(T, V)                        \
    do {                                      \
        if (sh.nv == 1) HM_BWD(T, V, 1);      \
        else if (sh.nv == 2) HM_BWD(T, V, 2); \
        else HM_BWD(T, V, 4);                 \
    } while (0)
        if (a->io_dtype == HM_BF16) {
            if (vec) HM_BWD_N(__nv_bfloat16, true);
            else HM_BWD_N(__nv_bfloat16, false);
        } else {
            if (vec) HM_BWD_N(float, true);
            else HM_BWD_N(float, false);
        }
#undef HM_BWD
#undef HM_BWD_N
        count_launches(1);
    }
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) {
        // without dxn the pre-norm's parameters had no part in the loss: their shares are zero
        const GradPtrs g = {{a->dscale, a->dpost_w, a->dpost_b, a->dpre_w, a->dpre_b}};
        norm_gate_sum_kernel<<<dim3((unsigned)((a->D + 31) / 32), 5), dim3(32, 8), 0, s>>>(part, grid, (int)a->D, g);
        count_launches(1);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? HM_OK : fail_args(HM_ERR_CUDA, "%s launch: %s", w, cudaGetErrorString(e));
}
