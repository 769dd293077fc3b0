// norm_gate.cu -- the seam between two blocks (hm_norm_gate_fwd, _bwd):
// post-norm, SiLU gate, scaled residual sum and the next block's pre-norm.
//
// Bandwidth-bound: five row arrays forward, eight backward, each touched once.
// A team of warps holds a row in registers: statistics come from there (mean
// first, then the centred squares), so nothing is read twice.
//
// Forward: a warp takes up to 1024 bf16 (512 fp32) elements of a row, so its
// sums cost five shuffles per 32 elements of a lane and a barrier among few
// warps, and all its loads are in flight at once.  Backward: each
// thread keeps the five parameter gradients of its columns in registers over
// all its rows (40 of them for 8 columns), so there a block shares a row; the
// blocks' shares are summed by a second, small kernel in a fixed order.
#include <type_traits>

#include "packed.cuh"
#include "tc_common.cuh"

namespace hm {

namespace {

// A thread's piece of a row is E elements, 16 bytes (fp32 pieces of 32 bytes
// would leave a warp's loads half of every sector apart), or a pair where rows
// and widths allow no more.  Columns of thread
// `tid` of a team of nthr: with VEC E consecutive elements, else single ones a
// team's width apart (both coalesced).
template <bool VEC, int kE>
__device__ __forceinline__ int col_of(int piece, int j, int tid, int nthr) {
    return VEC ? (piece * nthr + tid) * kE + j : (piece * kE + j) * nthr + tid;
}

// E elements as loaded
template <typename T, int E>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16, 8> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                     : "l"(p));
    }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void set(const F2 *f) {
        w = make_uint4(bf16_of(f[0]), bf16_of(f[1]), bf16_of(f[2]), bf16_of(f[3]));
    }
    __device__ __forceinline__ void get(F2 *f) const {
        f[0] = pk_bf16(w.x);
        f[1] = pk_bf16(w.y);
        f[2] = pk_bf16(w.z);
        f[3] = pk_bf16(w.w);
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { __stcs(reinterpret_cast<uint4 *>(p), w); }
};
template <>
struct Raw8<__nv_bfloat16, 2> {
    uint32_t w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];" : "=r"(w) : "l"(p));
    }
    __device__ __forceinline__ void zero() { w = 0; }
    __device__ __forceinline__ void set(const F2 *f) { w = bf16_of(f[0]); }
    __device__ __forceinline__ void get(F2 *f) const { f[0] = pk_bf16(w); }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { __stcs(reinterpret_cast<unsigned *>(p), w); }
};
template <>
struct Raw8<float, 2> {
    float2 a;
    __device__ __forceinline__ void load(const float *p) {
        asm volatile("ld.global.L1::no_allocate.v2.f32 {%0, %1}, [%2];" : "=f"(a.x), "=f"(a.y) : "l"(p));
    }
    __device__ __forceinline__ void zero() { a = make_float2(0.f, 0.f); }
    __device__ __forceinline__ void set(const F2 *f) { a = un(f[0]); }
    __device__ __forceinline__ void get(F2 *f) const { f[0] = pk(a.x, a.y); }
    __device__ __forceinline__ void store(float *p) const { __stcs(reinterpret_cast<float2 *>(p), a); }
};
template <>
struct Raw8<float, 4> {
    float4 a;
    __device__ __forceinline__ void load(const float *p) {
        asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w)
                     : "l"(p));
    }
    __device__ __forceinline__ void zero() { a = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void set(const F2 *f) {
        const float2 u0 = un(f[0]), u1 = un(f[1]);
        a = make_float4(u0.x, u0.y, u1.x, u1.y);
    }
    __device__ __forceinline__ void get(F2 *f) const {
        f[0] = pk(a.x, a.y);
        f[1] = pk(a.z, a.w);
    }
    __device__ __forceinline__ void store(float *p) const { __stcs(reinterpret_cast<float4 *>(p), a); }
};
template <>
struct Raw8<float, 8> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w)
                     : "l"(p));
        asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(b.x), "=f"(b.y), "=f"(b.z), "=f"(b.w)
                     : "l"(p + 4));
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void set(const F2 *f) {
        const float2 u0 = un(f[0]), u1 = un(f[1]), u2 = un(f[2]), u3 = un(f[3]);
        a = make_float4(u0.x, u0.y, u1.x, u1.y);
        b = make_float4(u2.x, u2.y, u3.x, u3.y);
    }
    __device__ __forceinline__ void get(F2 *f) const {
        f[0] = pk(a.x, a.y);
        f[1] = pk(a.z, a.w);
        f[2] = pk(b.x, b.y);
        f[3] = pk(b.z, b.w);
    }
    __device__ __forceinline__ void store(float *p) const {
        __stcs(reinterpret_cast<float4 *>(p), a);
        __stcs(reinterpret_cast<float4 *>(p + 4), b);
    }
};

// a piece of a row; columns behind D are zero
template <bool VEC, int kE, typename T>
__device__ __forceinline__ Raw8<T, kE> load8(const T *row, int piece, int tid, int nthr, int D) {
    Raw8<T, kE> r;
    if (VEC) {
        const int c = col_of<true, kE>(piece, 0, tid, nthr);
        if (c < D) r.load(row + c);
        else r.zero();
    } else {
        float f[kE];
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            const int c = col_of<false, kE>(piece, j, tid, nthr);
            f[j] = c < D ? hm_ld(row, c) : 0.f;
        }
        F2 g[kE / 2];
#pragma unroll
        for (int j = 0; j < kE / 2; ++j) g[j] = pk(f[2 * j], f[2 * j + 1]);
        r.set(g);
    }
    return r;
}

template <bool VEC, int kE, typename T>
__device__ __forceinline__ void store8(T *row, int piece, int tid, int nthr, int D, const F2 *f) {
    if (VEC) {
        const int c = col_of<true, kE>(piece, 0, tid, nthr);
        if (c < D) {
            Raw8<T, kE> r;
            r.set(f);
            r.store(row + c);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            const int c = col_of<false, kE>(piece, j, tid, nthr);
            if (c < D) hm_st(row, c, j & 1 ? un(f[j / 2]).y : un(f[j / 2]).x);
        }
    }
}

// fp32 parameters of a thread's columns, of a piece that it has().  The same
// for every row, so they stay in L1, which the rows themselves pass by.
template <bool VEC, int kE>
__device__ __forceinline__ void param8(const float *p, int piece, int tid, int nthr, int D, F2 *f) {
    if (VEC) {
        const float *q = p + col_of<true, kE>(piece, 0, tid, nthr);
        if constexpr (kE == 2) {
            const float2 a = __ldg(reinterpret_cast<const float2 *>(q));
            f[0] = pk(a.x, a.y);
        }
#pragma unroll
        for (int j = 0; j < kE / 4; ++j) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(q) + j);
            f[2 * j] = pk(a.x, a.y);
            f[2 * j + 1] = pk(a.z, a.w);
        }
    } else {
        float v[kE];
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            const int c = col_of<false, kE>(piece, j, tid, nthr);
            v[j] = c < D ? __ldg(p + c) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kE / 2; ++j) f[j] = pk(v[2 * j], v[2 * j + 1]);
    }
}

// u * p, u + p; a NULL p leaves u
template <bool VEC, int kE>
__device__ __forceinline__ void times(F2 *u, const float *p, int piece, int tid, int nthr, int D) {
    if (!p) return;
    F2 w[kE / 2];
    param8<VEC, kE>(p, piece, tid, nthr, D, w);
#pragma unroll
    for (int j = 0; j < kE / 2; ++j) u[j] = u[j] * w[j];
}
template <bool VEC, int kE>
__device__ __forceinline__ void plus(F2 *u, const float *p, int piece, int tid, int nthr, int D) {
    if (!p) return;
    F2 w[kE / 2];
    param8<VEC, kE>(p, piece, tid, nthr, D, w);
#pragma unroll
    for (int j = 0; j < kE / 2; ++j) u[j] = u[j] + w[j];
}

// whether a thread has any element of the piece; with VEC (D a multiple of E) all or none
template <bool VEC, int kE>
__device__ __forceinline__ bool has(int piece, int tid, int nthr, int D) {
    return col_of<VEC, kE>(piece, 0, tid, nthr) < D;
}
// f with the elements behind D set to zero (VEC: for a piece that has(); nothing to do)
template <bool VEC, int kE>
__device__ __forceinline__ F2 in_row(F2 f, int piece, int j, int tid, int nthr, int D) {
    if (VEC) return f;
    const float2 u = un(f);
    return pk(col_of<false, kE>(piece, 2 * j, tid, nthr) < D ? u.x : 0.f,
              col_of<false, kE>(piece, 2 * j + 1, tid, nthr) < D ? u.y : 0.f);
}

__device__ __forceinline__ float sum2(F2 f) {
    const float2 u = un(f);
    return u.x + u.y;
}

// Sums over the team (TEAM lanes of a warp: 8, 16 or 32; or with TEAM = 0 the
// whole block of up to 16 warps) of one or of four values; every thread gets them, always added in
// the same order.  `red` alternates between two buffers, so one barrier per
// call is enough: a call's reads are separated from the next-but-one call's
// writes by the next call's barrier.
constexpr int kMaxWarps = 16;
__device__ __forceinline__ float xor_add(float v, int o) { return v + __shfl_xor_sync(0xffffffffu, v, o); }

template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float (*red)[kMaxWarps][4], int &turn) {
#pragma unroll
    for (int o = (TEAM ? TEAM : 32) / 2; o > 0; o /= 2) v = xor_add(v, o);
    if (TEAM) return v;
    float (*r)[4] = red[turn & 1];
    ++turn;
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) r[threadIdx.x >> 5][0] = v;
    __syncthreads();
    v = (lane & 15) < nw ? r[lane & 15][0] : 0.f;
    return xor_add(xor_add(xor_add(xor_add(v, 8), 4), 2), 1);
}

// The four values travel together: each exchange halves what a lane carries,
// so that a quarter of the warp ends with each sum.
template <int TEAM>
__device__ __forceinline__ float4 team_sum4(float4 q, float (*red)[kMaxWarps][4], int &turn) {
    const int lane = threadIdx.x & 31;
    if (TEAM == 8 || TEAM == 16) {
#pragma unroll
        for (int o = TEAM / 2; o > 0; o /= 2)
            q = make_float4(xor_add(q.x, o), xor_add(q.y, o), xor_add(q.z, o), xor_add(q.w, o));
        return q;
    }
    const bool b16 = (lane & 16) != 0, b8 = (lane & 8) != 0;
    const float s0 = b16 ? q.x : q.z, s1 = b16 ? q.y : q.w;
    const float k0 = (b16 ? q.z : q.x) + __shfl_xor_sync(0xffffffffu, s0, 16);
    const float k1 = (b16 ? q.w : q.y) + __shfl_xor_sync(0xffffffffu, s1, 16);
    float v = (b8 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, b8 ? k0 : k1, 8);
    v = xor_add(xor_add(xor_add(v, 4), 2), 1);          // lanes 8 i .. 8 i + 7: the i-th value
    if (TEAM == 0) {
        float (*r)[4] = red[turn & 1];
        ++turn;
        const int nw = blockDim.x >> 5, w = lane & 7, i = lane >> 3;
        if (w == 0) r[threadIdx.x >> 5][i] = v;
        __syncthreads();
        v = w < nw ? r[w][i] : 0.f;
        if (w + 8 < nw) v += r[w + 8][i];
        v = xor_add(xor_add(xor_add(v, 4), 2), 1);
    }
    return make_float4(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 8),
                       __shfl_sync(0xffffffffu, v, 16), __shfl_sync(0xffffffffu, v, 24));
}

// 1 / (1 + e^-x): an e^-x beyond fp32 gives zero
__device__ __forceinline__ F2 sigmoid(F2 x) {
    float2 z = un(x * splat(-1.4426950408889634f));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(z.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(z.y));
    z = un(pk(z.x, z.y) + splat(1.f));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(z.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(z.y));
    return pk(z.x, z.y);
}

// One row per team: a block of 128 threads has several, or is one itself.  Teams
// of less than a warp (D <= 128) stay to the end when they have no row, with no
// columns either, since their warp's shuffles need them.
template <typename T, bool VEC, int NV, int TEAM, bool LAYER, int kE = 16 / (int)sizeof(T)>
__global__ void __launch_bounds__(TEAM ? 128 : 512, 1) norm_gate_fwd_kernel(hm_norm_gate_args p) {
    __shared__ float red[2][kMaxWarps][4];
    int turn = 0;
    constexpr int kP = kE / 2;
    constexpr int kTeam = TEAM ? TEAM : 1;
    const int tid = TEAM ? threadIdx.x % kTeam : threadIdx.x, nthr = TEAM ? TEAM : blockDim.x;
    const float inv = 1.f / (float)p.D;
    const int64_t row = TEAM ? (int64_t)blockIdx.x * (128 / kTeam) + threadIdx.x / kTeam : (int64_t)blockIdx.x;
    if (row >= p.rows && (TEAM == 0 || TEAM == 32)) return;         // whole teams
    const int D = row < p.rows ? (int)p.D : 0;
    Raw8<T, kE> ry[NV], rg[NV], rr[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        ry[k] = load8<VEC, kE>((const T *)p.y + row * p.y_stride, k, tid, nthr, D);
        if (p.gate) rg[k] = load8<VEC, kE>((const T *)p.gate + row * p.gate_stride, k, tid, nthr, D);
        if (p.r) rr[k] = load8<VEC, kE>((const T *)p.r + row * p.r_stride, k, tid, nthr, D);
        else rr[k].zero();
    }
    float mean = 0.f, rstd = 1.f;
    if (p.post) {
        F2 f[kP], v = splat(0.f);
        if (LAYER) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                ry[k].get(f);
#pragma unroll
                for (int j = 0; j < kP; ++j) v = v + f[j];
            }
            mean = team_sum<TEAM>(sum2(v), red, turn) * inv;
            v = splat(0.f);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (LAYER && !has<VEC, kE>(k, tid, nthr, D)) break;
            ry[k].get(f);
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                const F2 d = LAYER ? in_row<VEC, kE>(f[j] + splat(-mean), k, j, tid, nthr, D) : f[j];
                v = fma(d, d, v);
            }
        }
        rstd = rsqrtf(team_sum<TEAM>(sum2(v), red, turn) * inv + p.eps);
    }
    F2 r[NV][kP], v = splat(0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if (!has<VEC, kE>(k, tid, nthr, D)) break;
        F2 u[kP], c[kP];
        ry[k].get(u);
        rr[k].get(r[k]);
        if (p.post) {
#pragma unroll
            for (int j = 0; j < kP; ++j) u[j] = (LAYER ? u[j] + splat(-mean) : u[j]) * splat(rstd);
            times<VEC, kE>(u, p.post_w, k, tid, nthr, D);
            plus<VEC, kE>(u, p.post_b, k, tid, nthr, D);
        }
        if (p.gate) {
            rg[k].get(c);
#pragma unroll
            for (int j = 0; j < kP; ++j) u[j] = u[j] * (c[j] * sigmoid(c[j]));
        }
        times<VEC, kE>(u, p.scale, k, tid, nthr, D);
#pragma unroll
        for (int j = 0; j < kP; ++j) {
            // columns behind D hold zero, for the sums below
            r[k][j] = in_row<VEC, kE>(fma(splat(p.alpha), u[j], r[k][j]), k, j, tid, nthr, D);
            v = LAYER ? v + r[k][j] : fma(r[k][j], r[k][j], v);
        }
        if (p.r_out) store8<VEC, kE>((T *)p.r_out + row * p.r_out_stride, k, tid, nthr, D, r[k]);
    }
    if (!p.xn) return;
    float q = team_sum<TEAM>(sum2(v), red, turn);
    mean = 0.f;
    if (LAYER) {
        mean = q * inv;
        v = splat(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (!has<VEC, kE>(k, tid, nthr, D)) break;
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                const F2 d = in_row<VEC, kE>(r[k][j] + splat(-mean), k, j, tid, nthr, D);
                v = fma(d, d, v);
            }
        }
        q = team_sum<TEAM>(sum2(v), red, turn);
    }
    rstd = rsqrtf(q * inv + p.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if (!has<VEC, kE>(k, tid, nthr, D)) break;
#pragma unroll
        for (int j = 0; j < kP; ++j) r[k][j] = (LAYER ? r[k][j] + splat(-mean) : r[k][j]) * splat(rstd);
        times<VEC, kE>(r[k], p.pre_w, k, tid, nthr, D);
        plus<VEC, kE>(r[k], p.pre_b, k, tid, nthr, D);
        store8<VEC, kE>((T *)p.xn + row * p.xn_stride, k, tid, nthr, D, r[k]);
    }
}

// A team per row: the block, or TEAM lanes of a warp; each team's rows lie
// `stride` apart, the next one's loads under way while one is worked on (the
// teams of a warp go on together; one behind the last row has no columns).
// FULL: the common case that every row array is there and y is normalised,
// known to the compiler.
// part[(w * 5 + i) * D + c]: dscale, dpost_w, dpost_b, dpre_w, dpre_b as the
// w-th block, or warp, has summed them.
template <typename T, bool VEC, int NV, int TEAM, bool LAYER, bool FULL, int THREADS, int kE = 16 / (int)sizeof(T)>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 2 : 1)
norm_gate_bwd_kernel(hm_norm_gate_bwd_args p, float *part) {
    __shared__ float red[2][kMaxWarps][4];
    int turn = 0;
    constexpr int kP = kE / 2;
    constexpr int kTeam = TEAM ? TEAM : 1, kRows = TEAM ? 32 / kTeam : 1;       // rows of a warp, or block
    const bool gate = FULL || p.gate, post = FULL || p.post, pre = FULL || p.dxn;
    const int tid = TEAM ? threadIdx.x % kTeam : threadIdx.x, nthr = TEAM ? TEAM : blockDim.x;
    const float inv = 1.f / (float)p.D;
    const int64_t unit = TEAM ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    const int64_t stride = (TEAM ? (int64_t)gridDim.x * 8 : (int64_t)gridDim.x) * kRows;
    const int64_t first = unit * kRows, mine = TEAM ? threadIdx.x % 32 / kTeam : 0;
    F2 acc[5][NV][kP];
#pragma unroll
    for (int i = 0; i < 5; ++i)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < kP; ++j) acc[i][k][j] = splat(0.f);
    Raw8<T, kE> ry[NV], rg[NV], rr[NV], rd[NV], re[NV];
    auto fetch = [&](int64_t row) {
        const int D = row < p.rows ? (int)p.D : 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            ry[k] = load8<VEC, kE>((const T *)p.y + row * p.y_stride, k, tid, nthr, D);
            if (gate) rg[k] = load8<VEC, kE>((const T *)p.gate + row * p.gate_stride, k, tid, nthr, D);
            if (pre) {
                rr[k] = load8<VEC, kE>((const T *)p.r_out + row * p.r_out_stride, k, tid, nthr, D);
                re[k] = load8<VEC, kE>((const T *)p.dxn + row * p.dxn_stride, k, tid, nthr, D);
            }
            if (FULL || p.dr_out) rd[k] = load8<VEC, kE>((const T *)p.dr_out + row * p.dr_out_stride, k, tid, nthr, D);
            else rd[k].zero();
        }
    };
    if (first < p.rows) fetch(first + mine);
    for (int64_t base = first; base < p.rows; base += stride) {
        const int64_t row = base + mine;
        const int D = row < p.rows ? (int)p.D : 0;
        F2 y[NV][kP], r[NV][kP], d[NV][kP], e[NV][kP], g[NV][kP];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            ry[k].get(y[k]);
            if (gate) rg[k].get(g[k]);
            if (pre) rr[k].get(r[k]), re[k].get(e[k]);
            rd[k].get(d[k]);
        }
        if (base + stride < p.rows) fetch(row + stride);
        // y and r_out less their means
        F2 v0 = splat(0.f), v1 = splat(0.f);
        if (LAYER) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    v0 = v0 + y[k][j];
                    if (pre) v1 = v1 + r[k][j];
                }
            const float4 v = team_sum4<TEAM>(make_float4(sum2(v0), sum2(v1), 0.f, 0.f), red, turn);
            const F2 my = splat(post ? -v.x * inv : 0.f), mr = splat(-v.y * inv);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (!has<VEC, kE>(k, tid, nthr, D)) break;
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    y[k][j] = in_row<VEC, kE>(y[k][j] + my, k, j, tid, nthr, D);
                    if (pre) r[k][j] = in_row<VEC, kE>(r[k][j] + mr, k, j, tid, nthr, D);
                }
            }
        }
        // dr = dr_out + rstd (w e - mean(w e) - u mean(w e u)), u = (r - mean) rstd, e = dxn: the sums
        // over w e and w e (r - mean) go with those over the squares
        F2 v2 = splat(0.f), v3 = splat(0.f);
        v0 = v1 = splat(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (!has<VEC, kE>(k, tid, nthr, D)) break;
            if (pre) {
                F2 we[kP];
#pragma unroll
                for (int j = 0; j < kP; ++j) we[j] = e[k][j];
                times<VEC, kE>(we, p.pre_w, k, tid, nthr, D);        // zero behind D
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    v1 = fma(r[k][j], r[k][j], v1);
                    if (LAYER) v2 = v2 + we[j];
                    v3 = fma(we[j], r[k][j], v3);
                }
            }
#pragma unroll
            for (int j = 0; j < kP; ++j) v0 = fma(y[k][j], y[k][j], v0);
        }
        const float4 v = team_sum4<TEAM>(make_float4(sum2(v0), sum2(v1), sum2(v2), sum2(v3)), red, turn);
        const float rsy = post ? rsqrtf(v.x * inv + p.eps) : 1.f, rsr = rsqrtf(v.y * inv + p.eps);
        const float r0 = -rsr * (v.z * inv), r1 = -rsr * (rsr * (v.w * inv));
        v0 = v1 = splat(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (!has<VEC, kE>(k, tid, nthr, D)) break;
            if (pre) {
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const F2 u = r[k][j] * splat(rsr);
                    acc[3][k][j] = fma(e[k][j], u, acc[3][k][j]);
                    acc[4][k][j] = acc[4][k][j] + e[k][j];
                    d[k][j] = fma(u, splat(r1), LAYER ? d[k][j] + splat(r0) : d[k][j]);
                }
                times<VEC, kE>(e[k], p.pre_w, k, tid, nthr, D);
#pragma unroll
                for (int j = 0; j < kP; ++j) d[k][j] = fma(e[k][j], splat(rsr), d[k][j]);
            }
            if (FULL || p.dr) store8<VEC, kE>((T *)p.dr + row * p.dr_stride, k, tid, nthr, D, d[k]);
            F2 n[kP], dm[kP];
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                if (post) y[k][j] = y[k][j] * splat(rsy);
                n[j] = y[k][j];
                d[k][j] = dm[j] = in_row<VEC, kE>(d[k][j], k, j, tid, nthr, D) * splat(p.alpha);
            }
            if (post) {
                times<VEC, kE>(n, p.post_w, k, tid, nthr, D);
                plus<VEC, kE>(n, p.post_b, k, tid, nthr, D);
            }
            times<VEC, kE>(dm, p.scale, k, tid, nthr, D);
            if (gate) {
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const F2 sg = sigmoid(g[k][j]), si = g[k][j] * sg;
                    acc[0][k][j] = fma(d[k][j], n[j] * si, acc[0][k][j]);
                    // SiLU'(g) = sg + si (1 - sg)
                    g[k][j] = dm[j] * n[j] * fma(si, splat(1.f) - sg, sg);
                    d[k][j] = dm[j] * si;
                }
                store8<VEC, kE>((T *)p.dgate + row * p.dgate_stride, k, tid, nthr, D, g[k]);
            } else {
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    acc[0][k][j] = fma(d[k][j], n[j], acc[0][k][j]);
                    d[k][j] = dm[j];
                }
            }
            // d: gradient of the normalised (or plain) y
            if (post) {
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    acc[1][k][j] = fma(d[k][j], y[k][j], acc[1][k][j]);
                    acc[2][k][j] = acc[2][k][j] + d[k][j];
                }
                times<VEC, kE>(d[k], p.post_w, k, tid, nthr, D);
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    if (LAYER) v0 = v0 + d[k][j];
                    v1 = fma(d[k][j], y[k][j], v1);
                }
            }
        }
        if (post) {
            float y0 = 0.f, y1;
            if (LAYER) {
                const float4 q = team_sum4<TEAM>(make_float4(sum2(v0), sum2(v1), 0.f, 0.f), red, turn);
                y0 = -q.x * inv;
                y1 = -q.y * inv;
            } else {
                y1 = -team_sum<TEAM>(sum2(v1), red, turn) * inv;
            }
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const F2 q = fma(y[k][j], splat(y1), d[k][j]);
                    d[k][j] = splat(rsy) * (LAYER ? q + splat(y0) : q);
                }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) store8<VEC, kE>((T *)p.dy + row * p.dy_stride, k, tid, nthr, D, d[k]);
    }
    const int D = (int)p.D;
#pragma unroll
    for (int i = 0; i < 5; ++i)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                const int c = col_of<VEC, kE>(k, j, tid, nthr);
                float v = j & 1 ? un(acc[i][k][j / 2]).y : un(acc[i][k][j / 2]).x;
                if (TEAM)
#pragma unroll
                    for (int o = 16; o >= kTeam; o /= 2) v = xor_add(v, o);     // the warp's teams
                if (c < D && mine == 0) part[(unit * 5 + i) * D + c] = v;
            }
}

// Sums of N = 2, 4 or 8 values over a block of up to MW warps; every thread gets
// them, always added in the same order.  Each exchange halves what a lane
// carries, so N values cost N + 3 shuffles or so in place of 5 N.  `red` as in
// team_sum.
template <int N, int MW>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*red)[MW][8], int &turn) {
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    constexpr int kLanes = 32 / N;         // lanes that end with the same value
#pragma unroll
    for (int n = N / 2, o = 16; n >= 1; n /= 2, o /= 2) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    float s = v[0];
#pragma unroll
    for (int o = kLanes / 2; o > 0; o /= 2) s = xor_add(s, o);
    float (*r)[8] = red[turn & 1];
    ++turn;
    const int i = lane / kLanes, w = lane % kLanes;
    if (w == 0) r[threadIdx.x >> 5][i] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int k = 0; k < MW; k += kLanes)
        if (k + w < nw) s += r[k + w][i];
#pragma unroll
    for (int o = kLanes / 2; o > 0; o /= 2) s = xor_add(s, o);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __shfl_sync(0xffffffffu, s, k * kLanes);
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src, int bytes) {
    const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
}

// The common case of the backward (every row array there, y normalised, rows on
// 16-byte boundaries), for bf16 rows of 256 to 4096 columns: R rows at a time.
// Their sums share the exchanges and barriers, the rows wait in shared memory
// (each thread's own columns, by cp.async, the next R behind them), which
// leaves the registers to the parameter gradients, and so do the parameters
// (from L1, 8 columns a thread, they cost 91 us in place of 77).  8192 x 2048
// layer norms: 77 us against 95 with a row in registers, RMS 67 against 98, 4096 x
// 4096 68 against 109, 32768 x 512 77 against 83; fp32 rows, with pieces of their
// own half as wide, gained nothing.  What is left is latency at 16 warps per SM
// (52 % of the issue slots, half of what L1 and shared memory can move).
//
// FAR: rows of 4096 to 8192 columns of either type, one at a time over 1024
// threads, whose registers have no room for rows nor sums: the parameter
// gradients lie in shared memory, and a row is read again, from L2, in each of
// the three passes.
template <typename T, bool LAYER, int R, int THREADS, bool FAR>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 2 : 1)
norm_gate_bwd_rows_kernel(hm_norm_gate_bwd_args p, float *part) {
    constexpr int kE = 8, kP = kE / 2, Q = kE * (int)sizeof(T) / 16;
    extern __shared__ __align__(16) uint4 tile[];
    __shared__ float red[2][THREADS / 32][8];
    float4 *sums = reinterpret_cast<float4 *>(tile);       // FAR: [5][2][threads]
    float4 *par = sums + 2 * R * 5 * Q * blockDim.x;    // else, behind the rows: [4][2][threads]
    int turn = 0;
    const int tid = threadIdx.x, nthr = blockDim.x, D = (int)p.D, c = tid * kE;
    const bool live = c < D;
    const float inv = 1.f / (float)D;
    const int64_t groups = (p.rows + R - 1) / R;
    F2 acc[FAR ? 1 : 5][kP];
    if (FAR) {
#pragma unroll
        for (int i = 0; i < 10; ++i) sums[i * nthr + tid] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < 5; ++i)
#pragma unroll
            for (int j = 0; j < kP; ++j) acc[i][j] = splat(0.f);
    }
    // the i-th parameter's gradient += u * w
    auto add = [&](int i, const F2 *u, const F2 *w) {
        if constexpr (FAR) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4 *q = &sums[(i * 2 + h) * nthr + tid];
                const float4 o = *q;
                const float2 a = un(fma(u[2 * h], w[2 * h], pk(o.x, o.y))), b = un(fma(u[2 * h + 1], w[2 * h + 1], pk(o.z, o.w)));
                *q = make_float4(a.x, a.y, b.x, b.y);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kP; ++j) acc[i][j] = fma(u[j], w[j], acc[i][j]);
        }
    };
    const F2 one[kP] = {splat(1.f), splat(1.f), splat(1.f), splat(1.f)};
    // the thread's parameters: pre_w, post_w, post_b, scale.  Not FAR: copied once into shared memory,
    // 16 bytes a lane, since global loads of 8 fp32 columns leave their halves apart
    const float *const params[4] = {p.pre_w, p.post_w, p.post_b, p.scale};
    if (!FAR && live) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float none = i == 2 ? 0.f : 1.f;
                par[(i * 2 + h) * nthr + tid] = params[i] ? __ldg(reinterpret_cast<const float4 *>(params[i] + c) + h)
                                                          : make_float4(none, none, none, none);
            }
    }
    auto get_par = [&](int i, F2 *w) {
        const float4 a = par[i * 2 * nthr + tid], b = par[(i * 2 + 1) * nthr + tid];
        w[0] = pk(a.x, a.y), w[1] = pk(a.z, a.w), w[2] = pk(b.x, b.y), w[3] = pk(b.z, b.w);
    };
    auto by = [&](F2 *u, int i) {                  // u *= the i-th parameter
        if (FAR) {
            times<true, kE>(u, params[i], 0, tid, nthr, D);
            return;
        }
        F2 w[kP];
        get_par(i, w);
#pragma unroll
        for (int j = 0; j < kP; ++j) u[j] = u[j] * w[j];
    };
    const T *const base[5] = {(const T *)p.y, (const T *)p.gate, (const T *)p.r_out, (const T *)p.dr_out, (const T *)p.dxn};
    const int64_t strides[5] = {p.y_stride, p.gate_stride, p.r_out_stride, p.dr_out_stride, p.dxn_stride};
    auto fetch = [&](int64_t g, int s) {
        if (FAR) return;
        if (g < groups) {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int64_t row = g * R + k;
                const bool on = live && row < p.rows;          // else zeros
#pragma unroll
                for (int a = 0; a < 5; ++a) {
                    const T *src = base[a] + (on ? row * strides[a] + c : 0);
#pragma unroll
                    for (int q = 0; q < Q; ++q)
                        cp_async16(&tile[(((s * R + k) * 5 + a) * Q + q) * nthr + tid], src + q * (16 / sizeof(T)),
                                   on ? 16 : 0);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(blockIdx.x, 0);
    fetch((int64_t)blockIdx.x + gridDim.x, 1);
    int s = 0;
    for (int64_t g = blockIdx.x; g < groups; g += gridDim.x, s ^= 1) {
        if (!FAR) asm volatile("cp.async.wait_group 1;" ::: "memory");
        auto get = [&](int k, int a, F2 *f) {
            if (FAR) {
                Raw8<T, kE> r;
                if (live) r.load(base[a] + g * strides[a] + c);
                else r.zero();
                r.get(f);
                return;
            }
            const uint4 *q = &tile[((s * R + k) * 5 + a) * Q * nthr + tid];
            Raw8<T, kE> r;
            if constexpr (Q == 1) {
                r.w = q[0];
            } else {
                r.a = *reinterpret_cast<const float4 *>(q);
                r.b = *reinterpret_cast<const float4 *>(q + nthr);
            }
            r.get(f);
        };
        float my[R] = {}, mr[R] = {};                          // less the means
        if (LAYER) {
            float v[2 * R];
#pragma unroll
            for (int k = 0; k < R; ++k) {
                F2 y[kP], r[kP];
                get(k, 0, y);
                get(k, 2, r);
                v[2 * k] = sum2((y[0] + y[1]) + (y[2] + y[3]));
                v[2 * k + 1] = sum2((r[0] + r[1]) + (r[2] + r[3]));
            }
            block_sums(v, red, turn);
#pragma unroll
            for (int k = 0; k < R; ++k) my[k] = -v[2 * k] * inv, mr[k] = -v[2 * k + 1] * inv;
        }
        float rsy[R], rsr[R], r0[R], r1[R];
        {
            float v[4 * R] = {};
            if (live) {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    F2 y[kP], r[kP], e[kP], v0 = splat(0.f), v1 = v0, v2 = v0, v3 = v0;
                    get(k, 0, y);
                    get(k, 2, r);
                    get(k, 4, e);
                    by(e, 0);
#pragma unroll
                    for (int j = 0; j < kP; ++j) {
                        const F2 yc = LAYER ? y[j] + splat(my[k]) : y[j], rc = LAYER ? r[j] + splat(mr[k]) : r[j];
                        v0 = fma(yc, yc, v0);
                        v1 = fma(rc, rc, v1);
                        if (LAYER) v2 = v2 + e[j];
                        v3 = fma(e[j], rc, v3);
                    }
                    v[4 * k] = sum2(v0), v[4 * k + 1] = sum2(v1), v[4 * k + 2] = sum2(v2), v[4 * k + 3] = sum2(v3);
                }
            }
            block_sums(v, red, turn);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                rsy[k] = rsqrtf(v[4 * k] * inv + p.eps);
                rsr[k] = rsqrtf(v[4 * k + 1] * inv + p.eps);
                r0[k] = -rsr[k] * (v[4 * k + 2] * inv);
                r1[k] = -rsr[k] * (rsr[k] * (v[4 * k + 3] * inv));
            }
        }
        F2 dn[R][kP];
        float v[2 * R] = {};
        if (live) {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int64_t row = g * R + k;
                F2 d[kP], e[kP], u[kP];
                get(k, 2, u);
                get(k, 3, d);
                get(k, 4, e);
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    u[j] = (LAYER ? u[j] + splat(mr[k]) : u[j]) * splat(rsr[k]);
                    d[j] = fma(u[j], splat(r1[k]), LAYER ? d[j] + splat(r0[k]) : d[j]);
                }
                add(3, e, u);
                add(4, e, one);
                by(e, 0);
#pragma unroll
                for (int j = 0; j < kP; ++j) d[j] = fma(e[j], splat(rsr[k]), d[j]);
                if (row < p.rows) store8<true, kE>((T *)p.dr + row * p.dr_stride, 0, tid, nthr, D, d);
                F2 y[kP], n[kP], gt[kP];
                get(k, 0, y);
                get(k, 1, gt);
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    y[j] = (LAYER ? y[j] + splat(my[k]) : y[j]) * splat(rsy[k]);
                    n[j] = y[j];
                    d[j] = d[j] * splat(p.alpha);
                    dn[k][j] = d[j];
                }
                if (FAR) {
                    times<true, kE>(n, p.post_w, 0, tid, nthr, D);
                    plus<true, kE>(n, p.post_b, 0, tid, nthr, D);
                } else {
                    F2 w[kP], b[kP];
                    get_par(1, w);
                    get_par(2, b);
#pragma unroll
                    for (int j = 0; j < kP; ++j) n[j] = fma(n[j], w[j], b[j]);
                }
                by(dn[k], 3);
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const F2 sg = sigmoid(gt[j]), si = gt[j] * sg;
                    gt[j] = dn[k][j] * n[j] * fma(si, splat(1.f) - sg, sg);       // SiLU'(g) = sg + si (1 - sg)
                    n[j] = n[j] * si;
                    dn[k][j] = dn[k][j] * si;
                }
                add(0, d, n);
                add(1, dn[k], y);
                add(2, dn[k], one);
                if (row < p.rows) store8<true, kE>((T *)p.dgate + row * p.dgate_stride, 0, tid, nthr, D, gt);
                by(dn[k], 1);
                F2 v0 = splat(0.f), v1 = v0;
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    if (LAYER) v0 = v0 + dn[k][j];
                    v1 = fma(dn[k][j], y[j], v1);
                }
                v[2 * k] = sum2(v1);
                v[2 * k + 1] = sum2(v0);
            }
        }
        block_sums(v, red, turn);
        if (live) {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int64_t row = g * R + k;
                const F2 y1 = splat(-v[2 * k] * inv), y0 = splat(-v[2 * k + 1] * inv);
                F2 y[kP];
                get(k, 0, y);
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    y[j] = (LAYER ? y[j] + splat(my[k]) : y[j]) * splat(rsy[k]);
                    const F2 q = fma(y[j], y1, dn[k][j]);
                    y[j] = splat(rsy[k]) * (LAYER ? q + y0 : q);
                }
                if (row < p.rows) store8<true, kE>((T *)p.dy + row * p.dy_stride, 0, tid, nthr, D, y);
            }
        }
        fetch(g + 2 * (int64_t)gridDim.x, s);              // over what this thread has read
    }
    if (!FAR) asm volatile("cp.async.wait_all;" ::: "memory");
    if (!live) return;
    if constexpr (FAR) {
#pragma unroll
        for (int i = 0; i < 10; ++i)
            *reinterpret_cast<float4 *>(part + ((int64_t)blockIdx.x * 5 + i / 2) * D + c + i % 2 * 4) = sums[i * nthr + tid];
    } else {
#pragma unroll
        for (int i = 0; i < 5; ++i)
#pragma unroll
            for (int j = 0; j < kP; ++j)
                *reinterpret_cast<float2 *>(part + ((int64_t)blockIdx.x * 5 + i) * D + c + 2 * j) = un(acc[i][j]);
    }
}

struct GradPtrs {
    float *out[5];
};

// the teams' shares summed in a fixed order; a block of threads per 32 columns
// and parameter, ROWS rows of it walking the shares
template <int ROWS>
__global__ void __launch_bounds__(32 * ROWS) norm_gate_sum_kernel(const float *part, int teams, int D, GradPtrs g) {
    __shared__ float s[ROWS][33];
    float *out = g.out[blockIdx.y];
    if (!out) return;
    const int c = blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    if (c < D) {
#pragma unroll 10
        for (int b = threadIdx.y; b < teams; b += ROWS) v += part[((int64_t)b * 5 + blockIdx.y) * D + c];
    }
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < ROWS; ++i) v += s[i][threadIdx.x];
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

size_t esize(hm_dtype t) { return t == HM_BF16 ? 2 : 4; }

// smallest number of lanes, 8, 16 or 32, that have a whole row of one piece each
int lanes_of(int64_t D, size_t es) { return D * es <= 8 * 16 ? 8 : D * es <= 16 * 16 ? 16 : 32; }

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

// What an output may lie over.  An input that a row's thread has read for the
// last time before it writes the output may be the output's array, with the same
// stride: with others one row's output would fall on another's input.
hm_status check_over(const char *who, int64_t rows, const Row &out, const Row &in, bool allowed) {
    if (rows == 0 || !out.p || out.p != in.p) return HM_OK;
    if (!allowed) return fail_args(HM_ERR_INVALID_ARG, "%s: %s must not be %s", who, out.name, in.name);
    if (rows > 1 && out.stride != in.stride)
        return fail_args(HM_ERR_INVALID_ARG, "%s: %s is %s with another stride", who, out.name, in.name);
    return HM_OK;
}

// rows that start on `bytes` boundaries
bool wide(const Row &r, size_t es, size_t bytes = 16) {
    return !r.p || ((((uintptr_t)r.p) & (bytes - 1)) == 0 && (r.stride * (int64_t)es) % (int64_t)bytes == 0);
}

struct Team {
    int nthr, nv;        // threads that share a row (up to 32: of one warp), pieces of 16 bytes per thread
    int blocks;          // backward
};

// Forward: up to 4 pieces a lane: 2048 bf16 columns over 2 warps took 117 us for
// 32768 rows, over 1 warp of 8 pieces 134, over 4 warps 121, over 8 157.  More
// warps for wider rows, and for so few rows that these would leave most of the
// GPU idle.
// Rows of up to 256 bytes share a warp (320719 rows of 64, bf16: 117 -> 37 us).
// Rows that are read element by element get a block with as few pieces as it can.
Team fwd_team(int64_t rows, int64_t D, size_t es, bool vec) {
    const int columns = 32 * 16 / (int)es, pieces = (int)((D + columns - 1) / columns), of8 = es == 2 ? 1 : 2;
    const int most = !vec ? (D > 8192 ? 4 : D > 4096 ? 2 : 1) * of8 : es == 4 && D > 8192 ? 8 : 4;
    int warps = 1;
    if (vec && lanes_of(D, es) < 32) return {lanes_of(D, es), 1, 0};
    while ((pieces + warps - 1) / warps > most) warps *= 2;
    while (warps < 16 && (pieces + warps - 1) / warps > 1 && rows * warps * 2 <= 148 * 16) warps *= 2;
    int nv = 1;
    while (nv * warps < pieces) nv *= 2;
    return {warps * 32, nv, 0};
}

// Rows of pairs: an even width up to `most`, every row on a boundary of two
// elements.  Against element by element: forward, bf16, 60000 x 500 62 us and
// 127, 4000 x 7002 151 and 230 (fp32, 12000 x 1002: 56 and 50, so not there);
// backward 20000 x 1530 334 and 681, fp32 12000 x 1002 120 and 257 (100000 x 170, a warp
// per row: 228 and 214, so only from 256 columns on).
bool pairs(const Row *rows, int n, int64_t D, int64_t most, size_t es, const void *const *params, int np) {
    bool ok = D % 2 == 0 && D <= most;
    for (int i = 0; i < n; ++i) ok = ok && wide(rows[i], es, 2 * es);
    for (int i = 0; i < np; ++i) ok = ok && ((uintptr_t)params[i] & 7) == 0;
    return ok;
}

// Forward of pairs: up to 8 a lane.
Team pair_team(int64_t rows, int64_t D) {
    const int pieces = (int)((D + 63) / 64);
    int warps = 1, nv = 1;
    while ((pieces + warps - 1) / warps > 8) warps *= 2;
    while (warps < 16 && (pieces + warps - 1) / warps > 4 && rows * warps * 2 <= 148 * 16) warps *= 2;
    while (nv * warps < pieces) nv *= 2;
    return {warps * 32, warps > 1 && nv < 4 ? 4 : nv, 0};
}

// Backward: 8 columns a thread (bf16 one piece, fp32 two), up to 512 threads, then
// more; blocks (or warps) to fill the SMs once at 512 threads each.
// Rows of up to 256 bytes share a warp.
Team bwd_team(int64_t rows, int64_t D, size_t es) {
    const int columns = 32 * 16 / (int)es, pieces = (int)((D + columns - 1) / columns);
    int nv = es == 4 && pieces > 1 ? 2 : 1;
    while (nv * 16 < pieces) nv *= 2;
    const int warps = (pieces + nv - 1) / nv, lanes = lanes_of(D, es);
    const int of_block = 8 * 32 / lanes;                               // rows of a block of warps
    const int64_t most = warps == 1 ? 148 * 2 : 148 * (16 / warps);
    const int64_t need = warps == 1 ? (rows + of_block - 1) / of_block : rows;
    return {warps == 1 ? lanes : warps * 32, nv, (int)(need < most ? need : most)};
}

int64_t bwd_shares(const Team &t) { return t.nthr <= 32 ? t.blocks * 8LL : t.blocks; }

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
    bool vec = a->D * es % 16 == 0;
    for (const Row &r : rows) {
        HM_TRY(check_row(w, r, a->rows, a->D, es));
        vec = vec && wide(r, es);
    }
    for (int o = 3; o < 5; ++o)
        for (int i = 0; i < 3; ++i) HM_TRY(check_over(w, a->rows, rows[o], rows[i], true));
    const void *params[] = {a->scale, a->post_w, a->post_b, a->pre_w, a->pre_b};
    for (const void *q : params) {
        if (((uintptr_t)q & 3) != 0) return fail_args(HM_ERR_INVALID_ARG, "%s: misaligned parameter", w);
        vec = vec && ((uintptr_t)q & 15) == 0;
    }
    if (a->rows == 0) return HM_OK;
    if (!a->r_out && !a->xn) return fail_args(HM_ERR_INVALID_ARG, "%s: r_out and xn are both NULL", w);
    if (a->r_out == a->xn) return fail_args(HM_ERR_INVALID_ARG, "%s: r_out and xn are the same array", w);
    const bool two = !vec && es == 2 && pairs(rows, 5, a->D, 8192, es, params, 5);
    const Team t = two ? pair_team(a->rows, a->D) : fwd_team(a->rows, a->D, es, vec);
    const bool block = t.nthr > 32 || !(vec || two);
    const int of_block = block ? 1 : 128 / t.nthr;         // rows
    const int64_t blocks = (a->rows + of_block - 1) / of_block;
    if (blocks > 0x7fffffffLL) return fail_args(HM_ERR_UNSUPPORTED, "%s: too many rows", w);
    cudaStream_t s = (cudaStream_t)stream;
#define HM_FWD(T, V, N, B, Y) norm_gate_fwd_kernel<T, V, N, B, Y><<<(unsigned)blocks, B ? 128 : t.nthr, 0, s>>>(*a)
#define HM_FWD_Y(T, V, N, B) (a->norm == HM_NORM_LAYER ? HM_FWD(T, V, N, B, true) : HM_FWD(T, V, N, B, false))
#define HM_FWD_B(T, N) (block ? HM_FWD_Y(T, true, N, 0) : HM_FWD_Y(T, true, N, 32))
#define HM_FWD_S(T) (t.nv == 1 ? HM_FWD_Y(T, false, 1, 0) : t.nv == 2 ? HM_FWD_Y(T, false, 2, 0) : HM_FWD_Y(T, false, 4, 0))
#define HM_FWD_2(T, N, B)                                                                                            \
    (a->norm == HM_NORM_LAYER                                                                                        \
         ? norm_gate_fwd_kernel<T, true, N, B, true, 2><<<(unsigned)blocks, B ? 128 : t.nthr, 0, s>>>(*a)            \
         : norm_gate_fwd_kernel<T, true, N, B, false, 2><<<(unsigned)blocks, B ? 128 : t.nthr, 0, s>>>(*a))
#define HM_FWD_PAIRS(T)                                                                                              \
    (block ? (t.nv == 4 ? HM_FWD_2(T, 4, 0) : HM_FWD_2(T, 8, 0))                                                     \
     : t.nv == 1 ? HM_FWD_2(T, 1, 32) : t.nv == 2 ? HM_FWD_2(T, 2, 32)                                               \
     : t.nv == 4 ? HM_FWD_2(T, 4, 32) : HM_FWD_2(T, 8, 32))
    if (two) {
        HM_FWD_PAIRS(__nv_bfloat16);
    } else if (a->io_dtype == HM_BF16) {
        if (!vec) HM_FWD_S(__nv_bfloat16);
        else if (t.nthr == 8) HM_FWD_Y(__nv_bfloat16, true, 1, 8);
        else if (t.nthr == 16) HM_FWD_Y(__nv_bfloat16, true, 1, 16);
        else if (t.nv == 1) HM_FWD_B(__nv_bfloat16, 1);
        else if (t.nv == 2) HM_FWD_B(__nv_bfloat16, 2);
        else HM_FWD_B(__nv_bfloat16, 4);
    } else {
        if (!vec && t.nv == 8) HM_FWD_Y(float, false, 8, 0);
        else if (!vec) HM_FWD_S(float);
        else if (t.nthr == 8) HM_FWD_Y(float, true, 1, 8);
        else if (t.nthr == 16) HM_FWD_Y(float, true, 1, 16);
        else if (t.nv == 1) HM_FWD_B(float, 1);
        else if (t.nv == 2) HM_FWD_B(float, 2);
        else if (t.nv == 4) HM_FWD_B(float, 4);
        else HM_FWD_B(float, 8);
    }
#undef HM_FWD
#undef HM_FWD_Y
#undef HM_FWD_B
#undef HM_FWD_S
#undef HM_FWD_2
#undef HM_FWD_PAIRS
    count_launches(1);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? HM_OK : fail_args(HM_ERR_CUDA, "%s launch: %s", w, cudaGetErrorString(e));
}

extern "C" size_t hm_norm_gate_bwd_workspace_size(const hm_norm_gate_bwd_args *a) {
    if (!a || check_seam("norm_gate_bwd", a->rows, a->D, a->io_dtype, a->norm, a->eps, a->alpha) != HM_OK) return 0;
    return (size_t)bwd_shares(bwd_team(a->rows, a->D, esize(a->io_dtype))) * 5 * a->D * sizeof(float);
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
    bool vec = a->D * es % 16 == 0;
    for (const Row &r : rows) {
        HM_TRY(check_row(w, r, a->rows, a->D, es));
        vec = vec && wide(r, es);
    }
    for (int o = 5; o < 8; ++o) {
        // a row's outputs leave in the order dr, dgate, dy, and wide rows are read again in between:
        // gate behind dr, y behind both
        for (int i = 0; i < 5; ++i)
            HM_TRY(check_over(w, a->rows, rows[o], rows[i], o == 5 || (o == 6 ? i > 0 : i > 1)));
        for (int i = 5; i < o; ++i) HM_TRY(check_over(w, a->rows, rows[o], rows[i], false));
    }
    const void *params[] = {a->scale, a->post_w, a->post_b, a->pre_w, a->dscale, a->dpost_w, a->dpost_b, a->dpre_w,
                            a->dpre_b};
    for (const void *q : params)
        if (((uintptr_t)q & 3) != 0) return fail_args(HM_ERR_INVALID_ARG, "%s: misaligned parameter", w);
    for (int i = 0; i < 4; ++i) vec = vec && ((uintptr_t)params[i] & 15) == 0;    // those that are read
    for (int o = 4; o < 9; ++o)
        for (int i = 4; i < o; ++i)
            if (params[o] && params[o] == params[i])
                return fail_args(HM_ERR_INVALID_ARG, "%s: two parameter gradients are the same array", w);
    const size_t need = hm_norm_gate_bwd_workspace_size(a);
    if (need > 0 && (!a->workspace || a->workspace_bytes < need || ((uintptr_t)a->workspace & 255) != 0))
        return fail_args(HM_ERR_INVALID_ARG, "%s: workspace of %zu bytes, 256-byte aligned, is needed", w, need);
    const Team t = bwd_team(a->rows, a->D, es);
    int64_t shares = bwd_shares(t);
    cudaStream_t s = (cudaStream_t)stream;
    float *part = (float *)a->workspace;
    if (t.blocks > 0) {
        const bool full = a->gate && a->post && a->dxn && a->dr_out && a->dr;
        const bool far = vec && full && a->D % 8 == 0 && a->D > 4096 && a->D <= 8192;
        const bool tiled = far || (vec && full && es == 2 && a->D > 256 && t.nv == 1);
        auto rows_kernel = [&](auto kernel, int R) {
            const int nthr = far ? (int)((a->D / 8 + 31) / 32 * 32) : t.nthr;
            const size_t smem = far ? (size_t)10 * sizeof(float4) * nthr : ((size_t)2 * R * 5 + 8) * 16 * nthr;
            const cudaError_t e = tc::ensure_smem_limit(kernel, (int)smem);
            if (e != cudaSuccess) return e;
            // one wave: what an SM's 228 KB hold of these blocks (1.5 KB: the sums, and what a block costs besides)
            const int64_t groups = (a->rows + R - 1) / R, of_sm = (228 << 10) / (smem + 1536), wave = 148 * of_sm;
            shares = groups < t.blocks ? groups : t.blocks;
            if (!far && shares > wave) shares = wave;
            kernel<<<(unsigned)shares, nthr, smem, s>>>(*a, part);
            return cudaGetLastError();
        };
        auto rows_by = [&](auto layer) {
            constexpr bool Y = decltype(layer)::value;
            if (far)
                return es == 2 ? rows_kernel(norm_gate_bwd_rows_kernel<__nv_bfloat16, Y, 1, 1024, true>, 1)
                               : rows_kernel(norm_gate_bwd_rows_kernel<float, Y, 1, 1024, true>, 1);
            return t.nthr <= 256 ? rows_kernel(norm_gate_bwd_rows_kernel<__nv_bfloat16, Y, 2, 256, false>, 2)
                                 : rows_kernel(norm_gate_bwd_rows_kernel<__nv_bfloat16, Y, 2, 512, false>, 2);
        };
#define HM_BWD_F(T, V, N, B, Y, Z)                                                                          \
    (V && full ? norm_gate_bwd_kernel<T, V, N, B, Y, V, Z><<<t.blocks, B ? 256 : t.nthr, 0, s>>>(*a, part)      \
               : norm_gate_bwd_kernel<T, V, N, B, Y, false, Z><<<t.blocks, B ? 256 : t.nthr, 0, s>>>(*a, part))
#define HM_BWD(T, V, N, B, Z) (a->norm == HM_NORM_LAYER ? HM_BWD_F(T, V, N, B, true, Z) : HM_BWD_F(T, V, N, B, false, Z))
#define HM_BWD_WARP(T, V) (t.nthr == 8 ? HM_BWD(T, V, 1, 8, 256) : t.nthr == 16 ? HM_BWD(T, V, 1, 16, 256) : HM_BWD(T, V, 1, 32, 256))
#define HM_BWD_P(T, V, N, B, Z)      /* where the full case has gone to the kernel above */                 \
    (a->norm == HM_NORM_LAYER ? norm_gate_bwd_kernel<T, V, N, B, true, false, Z><<<t.blocks, t.nthr, 0, s>>>(*a, part) \
                              : norm_gate_bwd_kernel<T, V, N, B, false, false, Z><<<t.blocks, t.nthr, 0, s>>>(*a, part))
#define HM_BWD_16(T, V)                                                                                     \
    (t.nthr <= 32 ? HM_BWD_WARP(T, V)                                                                       \
     : t.nv == 1 ? (t.nthr <= 256 ? HM_BWD_P(T, V, 1, 0, 256) : HM_BWD_P(T, V, 1, 0, 512))                  \
     : t.nv == 2 ? HM_BWD_P(T, V, 2, 0, 512) : HM_BWD(T, V, 4, 0, 512))
#define HM_BWD_32(T, V)                                                                                     \
    (t.nthr <= 32 ? (t.nv == 1 ? HM_BWD_WARP(T, V) : HM_BWD(T, V, 2, 32, 256))                              \
     : t.nv == 2 ? (t.nthr <= 256 ? HM_BWD(T, V, 2, 0, 256) : HM_BWD(T, V, 2, 0, 512))                      \
     : t.nv == 4 ? HM_BWD(T, V, 4, 0, 512) : HM_BWD(T, V, 8, 0, 512))
        const bool two = !vec && a->D > 256 && pairs(rows, 8, a->D, 4096, es, params, 4);
#define HM_BWD_2(T, Z)                                                                                               \
    (a->norm == HM_NORM_LAYER ? norm_gate_bwd_kernel<T, true, 4, 0, true, false, Z, 2><<<t.blocks, t.nthr, 0, s>>>(*a, part) \
                              : norm_gate_bwd_kernel<T, true, 4, 0, false, false, Z, 2><<<t.blocks, t.nthr, 0, s>>>(*a, part))
#define HM_BWD_PAIRS(T) (t.nthr > 256 ? HM_BWD_2(T, 512) : HM_BWD_2(T, 256))      /* 8 columns a thread, as bwd_team has them */
        if (two) {
            if (a->io_dtype == HM_BF16) HM_BWD_PAIRS(__nv_bfloat16);
            else HM_BWD_PAIRS(float);
        } else if (tiled) {
            const cudaError_t e = a->norm == HM_NORM_LAYER ? rows_by(std::true_type()) : rows_by(std::false_type());
            if (e != cudaSuccess) return fail_args(HM_ERR_CUDA, "%s launch: %s", w, cudaGetErrorString(e));
        } else if (a->io_dtype == HM_BF16) vec ? HM_BWD_16(__nv_bfloat16, true) : HM_BWD_16(__nv_bfloat16, false);
        else vec ? HM_BWD_32(float, true) : HM_BWD_32(float, false);
#undef HM_BWD
#undef HM_BWD_F
#undef HM_BWD_WARP
#undef HM_BWD_P
#undef HM_BWD_2
#undef HM_BWD_PAIRS
#undef HM_BWD_16
#undef HM_BWD_32
        count_launches(1);
    }
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) {
        // without dxn the pre-norm's parameters had no part in the loss: their shares are zero
        const GradPtrs g = {{a->dscale, a->dpost_w, a->dpost_b, a->dpre_w, a->dpre_b}};
        // more rows of threads for many shares (2368 of 64 columns: 41.8 us a call against 47.7 with 16)
        const dim3 grid((unsigned)((a->D + 31) / 32), 5);
        if (shares > 512) norm_gate_sum_kernel<32><<<grid, dim3(32, 32), 0, s>>>(part, (int)shares, (int)a->D, g);
        else norm_gate_sum_kernel<16><<<grid, dim3(32, 16), 0, s>>>(part, (int)shares, (int)a->D, g);
        count_launches(1);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? HM_OK : fail_args(HM_ERR_CUDA, "%s launch: %s", w, cudaGetErrorString(e));
}
