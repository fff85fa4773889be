// k_group_norm.cu -- group norm with an activation, channels last, forward
// and backward.  Per (sequence, group) with xh = (x - mean) rstd,
// u = xh w + b:
//   y = act(u), or u act(gate) with a gate
//   du = dy act'(u), or dy act(gate);   dgate = dy u act'(gate)
//   dw = sum du xh,  db = sum du,  dn = du w
//   dx = rstd (dn - mean(dn) - xh mean(dn xh))
// Two plans.  `row` (one token a sequence, groups that fit a team of lanes):
// the group stays in registers, one pass over the data.  `seq` (statistics
// over many tokens, or wide groups): a pass for the sums, a pass that applies
// them; the second read of x comes from L2 while the tensors fit there.
#include "group_norm.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace m3 {
namespace {

enum { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU = 2, ACT_RELU = 3, ACT_ANY = -1 };

__device__ __forceinline__ float ex2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// act(u) and act'(u); ACT_ANY takes the activation at run time (the variants
// without vectors).  FAST: the exponentials of 16-bit outputs use the
// hardware approximation (2^-21 relative, against a rounding of 2^-8).
template <int ACT, bool FAST>
__device__ __forceinline__ void act_both(float u, int act, float &f, float &df) {
    const int A = ACT == ACT_ANY ? act : ACT;
    if (A == ACT_SILU) {
        const float s = FAST ? rcp_fast(1.f + ex2_fast(u * -1.4426950408889634f)) : 1.f / (1.f + expf(-u));
        f = u * s;
        df = fmaf(f, 1.f - s, s);
    } else if (A == ACT_GELU) {
        const float p = 0.5f * (1.f + erff(u * 0.70710678118654752f));
        f = u * p;
        df = fmaf(u * 0.39894228040143268f, FAST ? ex2_fast(u * u * -0.72134752044448170f) : expf(-0.5f * u * u), p);
    } else if (A == ACT_RELU) {
        f = u > 0.f ? u : (u == u ? 0.f : u);            // a NaN stays a NaN
        df = u > 0.f ? 1.f : 0.f;
    } else {
        f = u;
        df = 1.f;
    }
}
template <int ACT, bool FAST>
__device__ __forceinline__ float act_only(float u, int act) {
    float f, df;
    act_both<ACT, FAST>(u, act, f, df);
    return f;
}

// fma of two values in one instruction (register pairs)
__device__ __forceinline__ void fma_pair(float &d0, float &d1, float a0, float a1, float b0, float b1, float c0, float c1) {
    ptx::unpair(ptx::fma2(ptx::pair(a0, a1), ptx::pair(b0, b1), ptx::pair(c0, c1)), d0, d1);
}
// o = a * b + c over VEC values; b and c may be one value each
template <int VEC>
__device__ __forceinline__ void fmav(float *o, const float *a, const float *b, const float *c) {
    if (VEC == 1) o[0] = fmaf(a[0], b[0], c[0]);
    else
#pragma unroll
        for (int i = 0; i + 1 < VEC; i += 2) fma_pair(o[i], o[i + 1], a[i], a[i + 1], b[i], b[i + 1], c[i], c[i + 1]);
}
template <int VEC>
__device__ __forceinline__ void fmav(float *o, const float *a, float b, float c) {
    if (VEC == 1) o[0] = fmaf(a[0], b, c);
    else
#pragma unroll
        for (int i = 0; i + 1 < VEC; i += 2) fma_pair(o[i], o[i + 1], a[i], a[i + 1], b, b, c, c);
}

// VEC consecutive elements as they lie in memory: loaded early, unpacked late.
template <typename T, int VEC>
struct Raw {
    T v[VEC];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < VEC; i++) v[i] = p[i];
    }
    __device__ __forceinline__ void get(float *o) const {
#pragma unroll
        for (int i = 0; i < VEC; i++) o[i] = ldf(v, i);
    }
};
template <>
struct Raw<float, 4> {
    float4 v;
    __device__ __forceinline__ void load(const float *p) { v = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void get(float *o) const { o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w; }
};
template <>
struct Raw<__nv_bfloat16, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float *o) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            o[2 * i] = __uint_as_float(w[i] << 16);
            o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

// VEC consecutive elements
template <int VEC>
__device__ __forceinline__ void ldv(const float *p, float *v) {
    if (VEC % 4 == 0)
#pragma unroll
        for (int i = 0; i < VEC; i += 4) *reinterpret_cast<float4 *>(v + i) = *reinterpret_cast<const float4 *>(p + i);
    else
#pragma unroll
        for (int i = 0; i < VEC; i++) v[i] = p[i];
}
template <int VEC>
__device__ __forceinline__ void ldv(const __nv_bfloat16 *p, float *v) {
    if (VEC == 8) {
        const uint4 r = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else
#pragma unroll
        for (int i = 0; i < VEC; i++) v[i] = __bfloat162float(p[i]);
}
template <int VEC>
__device__ __forceinline__ void stv(float *p, const float *v) {
    if (VEC == 4) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
#pragma unroll
        for (int i = 0; i < VEC; i++) p[i] = v[i];
}
template <int VEC>
__device__ __forceinline__ void stv(__nv_bfloat16 *p, const float *v) {
    if (VEC == 8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&t);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else
#pragma unroll
        for (int i = 0; i < VEC; i++) p[i] = __float2bfloat16_rn(v[i]);
}

// Sum over a team of tw lanes (a power of two, 32 at most), every lane
// receives it.
__device__ __forceinline__ float team_sum(float v, int tw) {
    for (int o = tw >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// The same for a team of up to 256 lanes: the warps of a wider team meet in
// shared memory (the whole block takes part; `sh` holds a value per warp).
__device__ __forceinline__ float2 row_sum2(float2 v, int tw, float2 *sh) {
    const int in = tw < 32 ? tw : 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < in) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
    if (tw > 32) {
        const int w = threadIdx.x >> 5, nw = tw >> 5, w0 = w & ~(nw - 1);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sh[w] = v;
        __syncthreads();
        v = make_float2(0.f, 0.f);
        for (int i = 0; i < nw; i++) {
            v.x += sh[w0 + i].x;
            v.y += sh[w0 + i].y;
        }
    }
    return v;
}
__device__ __forceinline__ float row_sum(float v, int tw, float2 *sh) {
    const int in = tw < 32 ? tw : 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < in) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tw > 32) {
        const int w = threadIdx.x >> 5, nw = tw >> 5, w0 = w & ~(nw - 1);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sh[w].x = v;
        __syncthreads();
        v = 0.f;
        for (int i = 0; i < nw; i++) v += sh[w0 + i].x;
    }
    return v;
}

// ------------------------------------------------------------------- row plan
// A team of tw lanes (8 for 64 bf16 channels, a whole block for 4096) takes one
// group's channels of a row; neighbouring teams take neighbouring groups, so a
// row is read as one contiguous piece.  16384 x 1024, 16 groups, gated, bf16:
// 24.6 us, 64 % of the copy rate, bound by issue and by the latency of a team's
// chain of shuffles; the index arithmetic is in 32 bits (a 64-bit division
// costs more than the norm of eight elements does).
constexpr int RT = 256;

// Forward: one team, R rows of one group at once.  Few registers and many
// resident warps hide the latencies; teams that walk rows with the next one on
// its way hold half the warps and were slower (16384 x 1024, gated, 16 groups:
// 32 to 41 us).
template <typename T, int VEC, int NV, int ACT, bool GATE, int R = (VEC > 1 && NV == 1 ? 2 : 1)>
__global__ void __launch_bounds__(RT) k_gn_row_fwd(GnArgs a, int tw) {
    constexpr bool FAST = sizeof(T) == 2;
    __shared__ float2 sh[RT / 32];
    const unsigned tsh = 31 - __clz(tw), G = (unsigned)a.G;
    const unsigned team = blockIdx.x * (RT >> tsh) + (threadIdx.x >> tsh);     // below 2^32, see plan_of
    const int li = threadIdx.x & (tw - 1);
    const unsigned row0 = team / G * R, g = team - team / G * G;
    const int D = (int)((unsigned)a.C / G), nvec = D / VEC;
    const float invD = 1.f / (float)D;
    const int64_t base = (int64_t)row0 * a.C + g * D;
    float x[R][NV][VEC], mean[R], rstd[R];
    Raw<T, VEC> xr[R][NV], z[R][NV];
#pragma unroll
    for (int u = 0; u < R; u++)
#pragma unroll
        for (int m = 0; m < NV; m++) {
            const int v = m * tw + li;
            if (row0 + u < (unsigned)a.Bt && v < nvec) {
                xr[u][m].load(static_cast<const T *>(a.x) + base + u * a.C + v * VEC);
                if (GATE) z[u][m].load(static_cast<const T *>(a.gate) + base + u * a.C + v * VEC);
            }
        }
#pragma unroll
    for (int u = 0; u < R; u++) {
        float s = 0.f;
#pragma unroll
        for (int m = 0; m < NV; m++) {
            if (row0 + u < (unsigned)a.Bt && m * tw + li < nvec) {
                xr[u][m].get(x[u][m]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; e++) x[u][m][e] = 0.f;
            }
            float t[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < VEC; e++) t[e & 1] += x[u][m][e];
            s += t[0] + t[1];
        }
        mean[u] = s;
    }
#pragma unroll
    for (int u = 0; u < R; u++) mean[u] = row_sum(mean[u], tw, sh) * invD;
#pragma unroll
    for (int u = 0; u < R; u++) {
        float q = 0.f;
#pragma unroll
        for (int m = 0; m < NV; m++) {
            fmav<VEC>(x[u][m], x[u][m], 1.f, -mean[u]);
            if (m * tw + li < nvec) {
                if (VEC == 1) {
                    q = fmaf(x[u][m][0], x[u][m][0], q);
                } else {
                    float t0 = 0.f, t1 = 0.f;
#pragma unroll
                    for (int e = 0; e + 1 < VEC; e += 2)
                        fma_pair(t0, t1, x[u][m][e], x[u][m][e + 1], x[u][m][e], x[u][m][e + 1], t0, t1);
                    q += t0 + t1;
                }
            }
        }
        rstd[u] = q;
    }
#pragma unroll
    for (int u = 0; u < R; u++) rstd[u] = rsqrtf(fmaf(row_sum(rstd[u], tw, sh), invD, a.eps));
#pragma unroll
    for (int u = 0; u < R; u++)
        if (row0 + u < (unsigned)a.Bt && li == 0) {
            if (a.mean) a.mean[(int64_t)(row0 + u) * G + g] = mean[u];
            if (a.rstd) a.rstd[(int64_t)(row0 + u) * G + g] = rstd[u];
        }
#pragma unroll
    for (int m = 0; m < NV; m++) {
        const int v = m * tw + li;
        if (v < nvec) {
            float w[VEC], b[VEC], zf[VEC];
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                w[e] = 1.f;
                b[e] = 0.f;
            }
            if (a.w) ldv<VEC>(a.w + g * D + v * VEC, w);
            if (a.b) ldv<VEC>(a.b + g * D + v * VEC, b);
#pragma unroll
            for (int u = 0; u < R; u++) {
                if (row0 + u >= (unsigned)a.Bt) continue;
                if (GATE) z[u][m].get(zf);
                fmav<VEC>(x[u][m], x[u][m], rstd[u], 0.f);
                fmav<VEC>(x[u][m], x[u][m], w, b);
#pragma unroll
                for (int e = 0; e < VEC; e++)
                    x[u][m][e] = GATE ? x[u][m][e] * act_only<ACT, FAST>(zf[e], a.act)
                                      : act_only<ACT, FAST>(x[u][m][e], a.act);
                stv<VEC>(static_cast<T *>(a.y) + base + u * a.C + v * VEC, x[u][m]);
            }
        }
    }
}

// The gradients of w and b are summed in registers over a team's rows, then
// over the block's teams of the same group (in their order, in shared memory),
// and leave as one row of partial sums per block or slot, (row, 2, C);
// k_gn_reduce adds those up in their order.
template <typename T, int VEC, int NV, int ACT, bool GATE>
__global__ void __launch_bounds__(RT) k_gn_row_bwd(GnArgs a, int tw, int fold) {
    constexpr bool FAST = sizeof(T) == 2;
    pdl_trigger();
    extern __shared__ float part[];                       // 2 C sums, when the block folds its slots
    __shared__ float2 sh[RT / 32];
    struct { int slot, g, lane_in, nslots; bool on; } r;
    const unsigned tsh = 31 - __clz(tw), G = (unsigned)a.G;
    {
        const unsigned team = blockIdx.x * (RT >> tsh) + (threadIdx.x >> tsh);
        r.lane_in = threadIdx.x & (tw - 1);
        r.nslots = (int)(gridDim.x * (RT >> tsh) / G);
        r.slot = (int)(team / G);
        r.g = (int)(team % G);
        r.on = r.slot < r.nslots;                         // the rest: lanes past the last whole set of G teams
    }
    const int D = (int)((unsigned)a.C / G), nvec = D / VEC, Bt = (int)a.Bt;
    const float invD = 1.f / (float)D;
    float w[NV][VEC], b[NV][VEC], dw[NV][VEC], db[NV][VEC];
    Raw<T, VEC> nx[NV], ny[NV], nz[NV];
    float nmean = 0.f, nrstd = 0.f;
    const T *xp = static_cast<const T *>(a.x) + r.g * D, *zp = static_cast<const T *>(a.gate) + r.g * D;
    const T *yp = static_cast<const T *>(a.dy) + r.g * D;
    auto fetch = [&](int row) {
        if (r.on && row < Bt) {
            nmean = a.mean_in[(int64_t)row * a.G + r.g];
            nrstd = a.rstd_in[(int64_t)row * a.G + r.g];
#pragma unroll
            for (int m = 0; m < NV; m++) {
                const int v = m * tw + r.lane_in;
                if (v < nvec) {
                    nx[m].load(xp + (int64_t)row * a.C + v * VEC);
                    ny[m].load(yp + (int64_t)row * a.C + v * VEC);
                    if (GATE) nz[m].load(zp + (int64_t)row * a.C + v * VEC);
                }
            }
        }
    };
    fetch(r.slot);
#pragma unroll
    for (int m = 0; m < NV; m++)
#pragma unroll
        for (int e = 0; e < VEC; e++) {
            const int c = (m * tw + r.lane_in) * VEC + e;
            const bool in = r.on && c < D;
            w[m][e] = (in && a.w) ? a.w[r.g * D + c] : 1.f;
            b[m][e] = (in && a.b) ? a.b[r.g * D + c] : 0.f;
            dw[m][e] = db[m][e] = 0.f;
        }
    const int turns = (Bt + r.nslots - 1) / r.nslots;     // the same for every lane: the sums over a team need them all
    for (int k = 0; k < turns; k++) {
        const int row = r.slot + k * r.nslots;
        const bool on = r.on && row < Bt;
        const int64_t base = (int64_t)row * a.C + r.g * D;
        const float mean = nmean, rstd = nrstd;
        float xh[NV][VEC], dn[NV][VEC];
        Raw<T, VEC> z[NV];
        float m1 = 0.f, m2 = 0.f;
#pragma unroll
        for (int m = 0; m < NV; m++) {
            if (on && m * tw + r.lane_in < nvec) {
                nx[m].get(xh[m]);
                ny[m].get(dn[m]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; e++) xh[m][e] = dn[m][e] = 0.f;
            }
            z[m] = nz[m];
        }
        fetch(row + r.nslots);
#pragma unroll
        for (int m = 0; m < NV; m++) {
            const int v = m * tw + r.lane_in;
            if (on && v < nvec) {
                float zf[VEC], dz[VEC];
                if (GATE) z[m].get(zf);
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    float f, df, du;
                    xh[m][e] = (xh[m][e] - mean) * rstd;
                    const float u = fmaf(xh[m][e], w[m][e], b[m][e]);
                    if (GATE) {
                        act_both<ACT, FAST>(zf[e], a.act, f, df);
                        du = dn[m][e] * f;
                        dz[e] = dn[m][e] * u * df;
                    } else {
                        act_both<ACT, FAST>(u, a.act, f, df);
                        du = dn[m][e] * df;
                    }
                    dw[m][e] = fmaf(du, xh[m][e], dw[m][e]);
                    db[m][e] += du;
                    dn[m][e] = du * w[m][e];
                    m1 += dn[m][e];
                    m2 = fmaf(dn[m][e], xh[m][e], m2);
                }
                if (GATE && a.dgate) stv<VEC>(static_cast<T *>(a.dgate) + base + v * VEC, dz);
            }
        }
        const float2 mm = row_sum2(make_float2(m1, m2), tw, sh);
        m1 = mm.x * invD;
        m2 = mm.y * invD;
        if (a.dx) {
#pragma unroll
            for (int m = 0; m < NV; m++) {
                const int v = m * tw + r.lane_in;
                if (on && v < nvec) {
                    float dx[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; e++) dx[e] = (dn[m][e] - m1 - xh[m][e] * m2) * rstd;
                    stv<VEC>(static_cast<T *>(a.dx) + base + v * VEC, dx);
                }
            }
        }
    }
    if (!(a.dw || a.db)) return;
    // fold: every block holds the same number of whole sets of G teams
    const int mine = fold ? (int)(r.slot % fold) : 0;
    for (int f = 0; f < (fold ? fold : 1); f++) {
        if (r.on && mine == f) {
            float *pw = fold ? part + r.g * D : a.ws + (size_t)r.slot * 2 * a.C + r.g * D, *pb = pw + a.C;
#pragma unroll
            for (int m = 0; m < NV; m++)
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    const int c = (m * tw + r.lane_in) * VEC + e;
                    if (c < D) {
                        pw[c] = (f ? pw[c] : 0.f) + dw[m][e];
                        pb[c] = (f ? pb[c] : 0.f) + db[m][e];
                    }
                }
        }
        if (fold) __syncthreads();
    }
    if (fold)
        for (int c = threadIdx.x; c < 2 * a.C; c += RT) a.ws[(size_t)blockIdx.x * 2 * a.C + c] = part[c];
}

// dw, db from partial sums (n rows of 2 C): one block per 32 channels, its
// warps take rows in turn, then add up in a fixed order.
__device__ __forceinline__ void reduce_rows(const float *part, int64_t n, int64_t C, float *dw, float *db, int64_t blk) {
    __shared__ float sh[32][32];
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31, nw = blockDim.x >> 5;
    const int64_t c = blk * 32 + l;                       // of 2 C
    float s0 = 0.f;
    if (c < 2 * C) {
#pragma unroll 8
        for (int64_t r = w; r < n; r += nw) s0 += part[r * 2 * C + c];
    }
    sh[w][l] = s0;
    __syncthreads();
    if (w == 0 && c < 2 * C) {
        float t = 0.f;
        for (int i = 0; i < nw; i++) t += sh[i][l];
        if (c < C) {
            if (dw) dw[c] = t;
        } else if (db) {
            db[c - C] = t;
        }
    }
}

__global__ void __launch_bounds__(1024) k_gn_reduce(const float *part, int64_t n, int64_t C, float *dw, float *db) {
    pdl_wait();
    reduce_rows(part, n, C, dw, db, blockIdx.x);
}

// ------------------------------------------------------------------- seq plan
// The L tokens of a sequence are cut into chunks of `rows` tokens, one CTA
// each, all channels of a token read as one contiguous piece: a thread owns a
// vector of channels (every SQT-th where there are more), and where there are
// fewer vectors than threads, `np` threads share a vector's tokens.  8 x 2048 x
// 1024, 32 groups, bf16: forward 29 us, backward 47 us, bound by the latency of
// each pass (one wave of CTAs; DRAM at 20 to 34 %).
constexpr int SQT = 256;

struct SeqGeo {
    int bi, ch, t0, t1;        // sequence, chunk, its tokens
    int64_t base;              // of the sequence's first element
    int nvec, dvec, np, ph, v0, vstep;
};
__device__ __forceinline__ SeqGeo seq_geo(const GnArgs &a, int vec, int rows, int nch) {
    SeqGeo s;
    const int C = (int)a.C, L = (int)a.L;
    s.bi = (int)(blockIdx.x / (unsigned)nch);
    s.ch = (int)blockIdx.x - s.bi * nch;
    s.base = s.bi * a.L * a.C;
    s.t0 = s.ch * rows;
    s.t1 = min(s.t0 + rows, L);
    s.nvec = C / vec;
    s.dvec = (int)((unsigned)C / (unsigned)a.G) / vec;
    s.np = 1;
    s.ph = 0;
    s.v0 = threadIdx.x;
    s.vstep = SQT;
    if (s.nvec < SQT) {
        s.np = (int)(SQT / (unsigned)s.nvec);
        s.ph = (int)(threadIdx.x / (unsigned)s.nvec);
        s.v0 = s.ph < s.np ? (int)threadIdx.x - s.ph * s.nvec : s.nvec;    // nvec: idle
        s.vstep = s.nvec;
    }
    return s;
}

// A sum of squares that rounding took below zero; a NaN stays one (fmaxf would
// turn it into 0, and the variance of a group with an infinity into eps).
__device__ __forceinline__ float not_below_0(float v) { return v < 0.f ? 0.f : v; }
// What differences are taken from: with an infinity there, the mean would be
// inf - inf and not the infinity that it is.
__device__ __forceinline__ float origin(float v) { return isfinite(v) ? v : 0.f; }

// Per (sequence, chunk, group): the count is known, (mean, M2) are written.  A
// thread sums a vector of channels over its tokens as differences from its
// first value (so a large mean cancels nothing); the threads' (n, mean, M2)
// of a group are merged by the pairwise update of means.
template <typename T, int VEC>
__global__ void __launch_bounds__(SQT, 2) k_gn_seq_stats(GnArgs a, int rows, int nch) {
    pdl_trigger();
    extern __shared__ float2 vstat[];                     // (np, nvec) pairs (mean, M2)
    const SeqGeo s = seq_geo(a, VEC, rows, nch);
    const T *x = static_cast<const T *>(a.x) + s.base;
    for (int v = s.v0; v < s.nvec; v += s.vstep) {
        const int n = (int)((unsigned)(s.t1 - s.t0 - s.ph + s.np - 1) / (unsigned)s.np);   // this thread's tokens
        float K = 0.f, S = 0.f, Q = 0.f;
        if (n > 0) {
            const T *p = x + (int64_t)(s.t0 + s.ph) * a.C + v * VEC;
            const int64_t step = s.np * a.C;
            float sum[VEC], q[VEC];
            K = origin(ldf(p, 0));
#pragma unroll
            for (int e = 0; e < VEC; e++) sum[e] = q[e] = 0.f;
#pragma unroll 8
            for (int t = 0; t < n; t++, p += step) {
                float y[VEC];
                ldv<VEC>(p, y);
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    const float d = y[e] - K;
                    sum[e] += d;
                    q[e] = fmaf(d, d, q[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                S += sum[e];
                Q += q[e];
            }
            const float m = S / (float)(n * VEC);
            K += m;
            Q = not_below_0(Q - S * m);
        }
        vstat[s.ph * s.nvec + v] = make_float2(K, Q);
    }
    __syncthreads();
    // the phases of a vector merged by its first thread (n tokens each, one
    // more in the first phases), then a warp per group: the mean of the
    // vectors' means, and their spread.  Means are averaged as differences from
    // one of them: a sum of 256 of them rounds at its own size each time, which
    // moved means of 100 to 4096 by 12 to 17 half steps (300 x 1000 x 4; now 1)
    const int nt = s.t1 - s.t0;
    if (s.np > 1) {
        if (s.ph == 0) {
            const int q = (int)((unsigned)nt / (unsigned)s.np), more = nt - q * s.np;
            const float inv = 1.f / (float)nt;
            const float K = origin(vstat[s.v0].x);
            float m = 0.f, M2 = 0.f;
            for (int ph = 0; ph < s.np; ph++)
                m = fmaf(vstat[ph * s.nvec + s.v0].x - K, (float)(q + (ph < more)) * inv, m);
            m += K;
            for (int ph = 0; ph < s.np; ph++) {
                const float2 p = vstat[ph * s.nvec + s.v0];
                const float d = p.x - m;
                M2 += fmaf((float)((q + (ph < more)) * VEC) * d, d, p.y);
            }
            vstat[s.v0] = make_float2(m, M2);
        }
        __syncthreads();
    }
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    const float inv = 1.f / (float)s.dvec, n = (float)(nt * VEC);
    float2 *out = reinterpret_cast<float2 *>(a.ws) + (int64_t)blockIdx.x * a.G;
    // lanes of a warp: `per` of one group, so that narrow groups share a warp
    int per = 1;
    while (per < 32 && per < s.dvec) per *= 2;
    const int gs = 32 / per, gi = l / per, li = l & (per - 1);
    for (int g0 = w * gs; g0 < (int)a.G; g0 += SQT / 32 * gs) {
        const int g = g0 + gi;
        const bool on = g < (int)a.G;
        const float K = on ? origin(vstat[g * s.dvec].x) : 0.f;
        float m = 0.f, M2 = 0.f;
        if (on)
            for (int v = li; v < s.dvec; v += per) m += vstat[g * s.dvec + v].x - K;
        m = fmaf(team_sum(m, per), inv, K);
        if (on)
            for (int v = li; v < s.dvec; v += per) {
                const float2 p = vstat[g * s.dvec + v];
                const float d = p.x - m;
                M2 += fmaf(n * d, d, p.y);
            }
        M2 = team_sum(M2, per);
        if (on && li == 0) out[g] = make_float2(m, M2);
    }
}

// Every CTA merges its sequence's chunks itself (a few KB from L2) before it
// applies them: less than a launch of its own costs.
template <typename T, int VEC, int ACT, bool GATE>
__global__ void __launch_bounds__(SQT, 2) k_gn_seq_apply(GnArgs a, int rows, int nch) {
    constexpr bool FAST = sizeof(T) == 2;
    extern __shared__ float2 gstat[];                     // G pairs (mean, rstd)
    const SeqGeo s = seq_geo(a, VEC, rows, nch);
    // U tokens' loads go out together (y may be anywhere: the compiler keeps
    // loads behind stores), the first of them before the merge
    constexpr int U = GATE ? 4 : 8;
    Raw<T, VEC> xr[U], zr[U];
    const int64_t step = s.np * a.C;
    auto fetch = [&](int t, int64_t o) {
#pragma unroll
        for (int u = 0; u < U; u++)
            if (t + u * s.np < s.t1) {
                xr[u].load(static_cast<const T *>(a.x) + o + u * step);
                if (GATE) zr[u].load(static_cast<const T *>(a.gate) + o + u * step);
            }
    };
    const int64_t o0 = s.base + (int64_t)(s.t0 + s.ph) * a.C;
    bool ready = s.v0 < s.nvec;
    if (ready) fetch(s.t0 + s.ph, o0 + s.v0 * VEC);
    {
        // thread = (group of 32, every eighth chunk): sums of n d and of M2 + n d^2,
        // d from the first chunk's mean, so that nothing of size mean^2 cancels
        __shared__ float2 sh[8][32];
        pdl_wait();
        const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
        const float D = (float)(a.C / a.G), n = (float)a.L * D;
        const float nfull = (float)rows * D, nlast = (float)((int)a.L - (nch - 1) * rows) * D;
        for (int g0 = 0; g0 < a.G; g0 += 32) {
            const int g = g0 + l;
            const float2 *p = reinterpret_cast<const float2 *>(a.ws) + (int64_t)s.bi * nch * a.G + g;
            float K = 0.f, s1 = 0.f, s2 = 0.f;
            if (g < a.G) {
                K = origin(p[0].x);
#pragma unroll 8
                for (int c = w; c < nch; c += 8) {
                    const float2 q = p[c * (int)a.G];
                    const float nc = c + 1 < nch ? nfull : nlast, d = q.x - K;
                    s1 = fmaf(nc, d, s1);
                    s2 += fmaf(nc * d, d, q.y);
                }
            }
            __syncthreads();
            sh[w][l] = make_float2(s1, s2);
            __syncthreads();
            if (w == 0 && g < a.G) {
                s1 = s2 = 0.f;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    s1 += sh[i][l].x;
                    s2 += sh[i][l].y;
                }
                const float dm = s1 / n, m = K + dm, rstd = rsqrtf(not_below_0(s2 - s1 * dm) / n + a.eps);
                gstat[g] = make_float2(m, rstd);
                if (s.ch == 0 && a.mean) a.mean[(int64_t)s.bi * a.G + g] = m;
                if (s.ch == 0 && a.rstd) a.rstd[(int64_t)s.bi * a.G + g] = rstd;
            }
        }
        __syncthreads();
    }
    for (int v = s.v0; v < s.nvec; v += s.vstep) {
        const float2 st = gstat[v / s.dvec];
        float w[VEC], b[VEC];
#pragma unroll
        for (int e = 0; e < VEC; e++) {
            w[e] = (a.w ? a.w[v * VEC + e] : 1.f) * st.y;
            b[e] = a.b ? a.b[v * VEC + e] : 0.f;
        }
        int64_t o = o0 + v * VEC;
        for (int t = s.t0 + s.ph; t < s.t1; t += U * s.np, o += U * step) {
            if (!ready) fetch(t, o);
            ready = false;
#pragma unroll
            for (int u = 0; u < U; u++)
                if (t + u * s.np < s.t1) {
                    float x[VEC], z[VEC];
                    xr[u].get(x);
                    if (GATE) zr[u].get(z);
                    fmav<VEC>(x, x, 1.f, -st.x);          // the difference first: a large mean cancels nothing
                    fmav<VEC>(x, x, w, b);
#pragma unroll
                    for (int e = 0; e < VEC; e++)
                        x[e] = GATE ? x[e] * act_only<ACT, FAST>(z[e], a.act) : act_only<ACT, FAST>(x[e], a.act);
                    stv<VEC>(static_cast<T *>(a.y) + o + u * step, x);
                }
        }
    }
}

// du of one element, and xh; dz where there is a gate
template <int ACT, bool GATE, bool FAST>
__device__ __forceinline__ float gn_du(float x, float dy, float z, float2 st, float w, float b, int act, float &xh,
                                       float &dz) {
    float f, df;
    xh = (x - st.x) * st.y;
    const float u = fmaf(xh, w, b);
    if (GATE) {
        act_both<ACT, FAST>(z, act, f, df);
        dz = dy * u * df;
        return dy * f;
    }
    act_both<ACT, FAST>(u, act, f, df);
    return dy * df;
}

// Per (sequence, chunk, channel): sums of du xh and du over the chunk's
// tokens, (sequence, chunk, 2, C); the gate's gradient is written on the way.
template <typename T, int VEC, int ACT, bool GATE>
__global__ void __launch_bounds__(SQT, 2) k_gn_seq_bsums(GnArgs a, int rows, int nch) {
    constexpr bool FAST = sizeof(T) == 2;
    pdl_trigger();
    extern __shared__ float psum[];                       // (np - 1, 2, C): the other phases' sums
    const SeqGeo s = seq_geo(a, VEC, rows, nch);
    float *out = a.ws + (size_t)blockIdx.x * 2 * a.C;
    float s1[VEC], s2[VEC];
    for (int v = s.v0; v < s.nvec; v += s.vstep) {
        const int gi = s.bi * (int)a.G + v / s.dvec;
        const float2 st = make_float2(a.mean_in[gi], a.rstd_in[gi]);
        float w[VEC], b[VEC];
#pragma unroll
        for (int e = 0; e < VEC; e++) {
            w[e] = a.w ? a.w[v * VEC + e] : 1.f;
            b[e] = a.b ? a.b[v * VEC + e] : 0.f;
            s1[e] = s2[e] = 0.f;
        }
        int64_t o = s.base + (int64_t)(s.t0 + s.ph) * a.C + v * VEC;
        const int64_t step = s.np * a.C;
#pragma unroll 4
        for (int t = s.t0 + s.ph; t < s.t1; t += s.np, o += step) {
            float x[VEC], dy[VEC], z[VEC], dz[VEC];
            ldv<VEC>(static_cast<const T *>(a.x) + o, x);
            ldv<VEC>(static_cast<const T *>(a.dy) + o, dy);
            if (GATE) ldv<VEC>(static_cast<const T *>(a.gate) + o, z);
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                float xh;
                const float du = gn_du<ACT, GATE, FAST>(x[e], dy[e], z[e], st, w[e], b[e], a.act, xh, dz[e]);
                s1[e] = fmaf(du, xh, s1[e]);
                s2[e] += du;
            }
            if (GATE && a.dgate) stv<VEC>(static_cast<T *>(a.dgate) + o, dz);
        }
        float *to = s.ph > 0 ? psum + (size_t)(s.ph - 1) * 2 * a.C : out;
        if (s.np == 1 || s.ph > 0) {
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                to[v * VEC + e] = s1[e];
                to[a.C + v * VEC + e] = s2[e];
            }
        }
    }
    if (s.np > 1) {                                       // one vector a thread: the first phase adds the others'
        __syncthreads();
        if (s.ph == 0) {
            const int v = s.v0;
            for (int ph = 1; ph < s.np; ph++) {
                const float *q = psum + (size_t)(ph - 1) * 2 * a.C;
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    s1[e] += q[v * VEC + e];
                    s2[e] += q[a.C + v * VEC + e];
                }
            }
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                out[v * VEC + e] = s1[e];
                out[a.C + v * VEC + e] = s2[e];
            }
        }
    }
}

// Per (sequence, group): the chunks' sums added up into (sequence, 2, C), and
// from them mean(dn xh) and mean(dn).  One block a (sequence, group): warps
// over chunks, lanes over the group's channels.
__global__ void __launch_bounds__(256) k_gn_seq_moments(GnArgs a, int nch, float *sums, float2 *mom) {
    __shared__ float sh[2][8][32];
    __shared__ float red[2];
    pdl_trigger();
    pdl_wait();
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    const int bi = (int)(blockIdx.x / (unsigned)a.G), g = (int)blockIdx.x - bi * (int)a.G;
    const int D = (int)((unsigned)a.C / (unsigned)a.G);
    float m2 = 0.f, m1 = 0.f;
    for (int c0 = 0; c0 < D; c0 += 32) {
        const int c = c0 + l;
        float s1 = 0.f, s2 = 0.f;
        if (c < D) {
            const float *p = a.ws + (size_t)bi * nch * 2 * a.C + g * D + c;
#pragma unroll 4
            for (int k = w; k < nch; k += 8) {
                s1 += p[(int64_t)k * 2 * a.C];
                s2 += p[(int64_t)k * 2 * a.C + a.C];
            }
        }
        __syncthreads();
        sh[0][w][l] = s1;
        sh[1][w][l] = s2;
        __syncthreads();
        if (w < 2) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i++) t += sh[w][i][l];
            if (c < D) {
                sums[(int64_t)bi * 2 * a.C + w * a.C + g * D + c] = t;
                const float wt = a.w ? a.w[g * D + c] : 1.f;
                if (w == 0) m2 = fmaf(t, wt, m2);
                else m1 = fmaf(t, wt, m1);
            }
        }
    }
    if (w < 2) {
        const float t = team_sum(w == 0 ? m2 : m1, 32);
        if (l == 0) red[w] = t / ((float)a.L * (float)D);
    }
    __syncthreads();
    if (threadIdx.x == 0) mom[blockIdx.x] = make_float2(red[0], red[1]);
}

// dx; the last blocks add up dw and db instead
template <typename T, int VEC, int ACT, bool GATE>
__global__ void __launch_bounds__(SQT, 2) k_gn_seq_dx(GnArgs a, int rows, int nch, const float *sums,
                                                   const float2 *mom, unsigned dx_blocks) {
    constexpr bool FAST = sizeof(T) == 2;
    pdl_wait();
    if (blockIdx.x >= dx_blocks) {
        reduce_rows(sums, a.Bt, a.C, a.dw, a.db, blockIdx.x - dx_blocks);
        return;
    }
    const SeqGeo s = seq_geo(a, VEC, rows, nch);
    for (int v = s.v0; v < s.nvec; v += s.vstep) {
        const int gi = s.bi * (int)a.G + v / s.dvec;
        const float2 st = make_float2(a.mean_in[gi], a.rstd_in[gi]), mm = mom[gi];
        float w[VEC], b[VEC];
#pragma unroll
        for (int e = 0; e < VEC; e++) {
            w[e] = a.w ? a.w[v * VEC + e] : 1.f;
            b[e] = a.b ? a.b[v * VEC + e] : 0.f;
        }
        int64_t o = s.base + (int64_t)(s.t0 + s.ph) * a.C + v * VEC;
        const int64_t step = s.np * a.C;
        constexpr int U = GATE ? 2 : 4;                   // tokens whose loads go out together
        for (int t = s.t0 + s.ph; t < s.t1; t += U * s.np, o += U * step) {
            Raw<T, VEC> xr[U], yr[U], zr[U];
#pragma unroll
            for (int u = 0; u < U; u++)
                if (t + u * s.np < s.t1) {
                    xr[u].load(static_cast<const T *>(a.x) + o + u * step);
                    yr[u].load(static_cast<const T *>(a.dy) + o + u * step);
                    if (GATE) zr[u].load(static_cast<const T *>(a.gate) + o + u * step);
                }
#pragma unroll
            for (int u = 0; u < U; u++)
                if (t + u * s.np < s.t1) {
                    float x[VEC], dy[VEC], z[VEC];
                    xr[u].get(x);
                    yr[u].get(dy);
                    if (GATE) zr[u].get(z);
#pragma unroll
                    for (int e = 0; e < VEC; e++) {
                        float xh, dz;
                        const float du = gn_du<ACT, GATE, FAST>(x[e], dy[e], z[e], st, w[e], b[e], a.act, xh, dz);
                        x[e] = (fmaf(du, w[e], -mm.y) - xh * mm.x) * st.y;
                    }
                    stv<VEC>(static_cast<T *>(a.dx) + o + u * step, x);
                }
        }
    }
}

// ---------------------------------------------------------------- host side
struct Plan {
    bool row;
    int vec, nv, tw;           // row plan: vector width, vectors a lane, lanes a team
    unsigned blocks;
    int64_t nslots;            // row plan: rows in flight
    int fold;                  // row plan: slots of a block that the backward adds up in shared memory (0: one at most)
    int64_t parts;             // row plan: rows of partial sums
    int64_t rows, nch;         // seq plan: tokens a chunk, chunks a sequence
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row plan: groups of one token that a block can hold in registers (4096
// bf16, 8192 fp32 channels, 2048 without vectors; the backward of more than 4096
// fp32 channels spills up to 520 bytes a thread).  Otherwise the seq plan.
// Vectors of 16 bytes where the group is a whole number of them (every base
// address is 16-byte aligned), else single elements.
Plan plan_of(int64_t Bt, int64_t L, int64_t C, int64_t G, m3_dtype dt, bool bwd) {
    Plan p{};
    if (L == 0) {
        p.rows = p.nch = 1;
        return p;
    }
    const int64_t D = C / G;
    const int wide = dt == M3_BF16 ? 8 : 4;
    p.vec = D % wide == 0 ? wide : 1;
    const int64_t nvec = D / p.vec;
    const int most = p.vec == 8 ? 2 : 8;                  // vectors a lane: 16 bf16, 32 fp32 or 8 single values
    if (L == 1 && nvec <= RT * most) {
        p.row = true;
        p.tw = 1;
        while (p.tw < 32 && p.tw < nvec) p.tw *= 2;       // a warp first, then more values a lane, then more warps
        while (p.tw < RT && nvec > p.tw * (p.vec > 1 ? most / 2 : 4)) p.tw *= 2;
        const int64_t nv = ceil_div(nvec, p.tw);
        p.nv = 1;
        while (p.nv < nv) p.nv *= 2;
        const int64_t teams_cta = RT / p.tw, need = ceil_div(G, teams_cta);
        const int64_t rows = !bwd && p.vec > 1 && p.nv == 1 ? 2 : 1;   // rows a team takes at once
        int64_t blocks = ceil_div(ceil_div(Bt, rows) * G, teams_cta);
        if (!bwd) {
            p.blocks = (unsigned)blocks;
            return p;
        }
        // backward: at most two CTAs for each SM, at least two rows a team; always
        // enough teams for one of each group.  Two are resident at once up to 128
        // registers a thread; a lane that holds 16 bf16 or from 16 fp32 channels
        // takes 148 to 255, one CTA to an SM, and the blocks come in two turns
        blocks = (blocks + 1) / 2;
        if (blocks > 148 * 2) blocks = 148 * 2;
        if (blocks < need) blocks = need;
        p.blocks = (unsigned)blocks;
        p.nslots = blocks * teams_cta / G;
        p.parts = p.nslots;
        if (teams_cta % G == 0 && teams_cta > G) {
            p.fold = (int)(teams_cta / G);
            p.parts = blocks;
        }
        return p;
    }
    // chunks of tokens: the two CTAs per SM that are resident at once, at
    // least 4 tokens each
    int64_t nch = 148 * 2 / (Bt > 0 ? Bt : 1);
    if (nch > ceil_div(L, 4)) nch = ceil_div(L, 4);
    if (nch < 1) nch = 1;
    p.rows = ceil_div(L, nch);
    p.nch = ceil_div(L, p.rows);
    return p;
}

// the (activation, gate) variant of a kernel template: without vectors the
// activation is a run-time choice (a quarter of the variants)
#define GN_ACTS(CALL, K, T, VEC, NV)                                                  \
    if constexpr (VEC == 1) {                                                         \
        if (a.gate) { CALL((K<T, 1 NV, ACT_ANY, true>)); }                            \
        else { CALL((K<T, 1 NV, ACT_ANY, false>)); }                                  \
    } else {                                                                          \
        constexpr int V = VEC == 1 ? (sizeof(T) == 2 ? 8 : 4) : VEC;                  \
        switch (a.act * 2 + (a.gate ? 1 : 0)) {                                       \
            case 0: CALL((K<T, V NV, ACT_NONE, false>)); break;                       \
            case 1: CALL((K<T, V NV, ACT_NONE, true>)); break;                        \
            case 2: CALL((K<T, V NV, ACT_SILU, false>)); break;                       \
            case 3: CALL((K<T, V NV, ACT_SILU, true>)); break;                        \
            case 4: CALL((K<T, V NV, ACT_GELU, false>)); break;                       \
            case 5: CALL((K<T, V NV, ACT_GELU, true>)); break;                        \
            case 6: CALL((K<T, V NV, ACT_RELU, false>)); break;                       \
            default: CALL((K<T, V NV, ACT_RELU, true>)); break;                       \
        }                                                                             \
    }
#define GN_COMMA_NV(n) , n

template <typename T, int VEC, int NV>
cudaError_t row_launch(const GnArgs &a, const Plan &p, bool bwd, cudaStream_t s) {
    if (bwd) {
        const int smem = p.fold ? (int)(2 * a.C * sizeof(float)) : 0;      // C <= 4096 there
#define GN_CALL(K) K<<<p.blocks, RT, smem, s>>>(a, p.tw, p.fold)
        GN_ACTS(GN_CALL, k_gn_row_bwd, T, VEC, GN_COMMA_NV(NV))
#undef GN_CALL
    } else {
#define GN_CALL(K) K<<<p.blocks, RT, 0, s>>>(a, p.tw)
        GN_ACTS(GN_CALL, k_gn_row_fwd, T, VEC, GN_COMMA_NV(NV))
#undef GN_CALL
    }
    count_launch();
    return cudaGetLastError();
}

template <typename T, int WIDE>
cudaError_t row_dispatch(const GnArgs &a, const Plan &p, bool bwd, cudaStream_t s) {
    if (p.vec == WIDE) {
        if (p.nv == 1) return row_launch<T, WIDE, 1>(a, p, bwd, s);
        if (p.nv == 2) return row_launch<T, WIDE, 2>(a, p, bwd, s);
        if constexpr (WIDE == 4) {
            if (p.nv == 4) return row_launch<T, 4, 4>(a, p, bwd, s);
            return row_launch<T, 4, 8>(a, p, bwd, s);
        }
        return cudaErrorInvalidValue;
    }
    if (p.nv == 1) return row_launch<T, 1, 1>(a, p, bwd, s);
    if (p.nv == 2) return row_launch<T, 1, 2>(a, p, bwd, s);
    if (p.nv == 4) return row_launch<T, 1, 4>(a, p, bwd, s);
    return row_launch<T, 1, 8>(a, p, bwd, s);
}

// phases that share a vector's tokens (as seq_geo)
int seq_phases(int64_t C, int vec) {
    const int64_t nvec = C / vec;
    return nvec < SQT ? (int)(SQT / nvec) : 1;
}

// Dynamic shared memory of the forward over sequences: 8 bytes a vector of
// channels, or a group (16384 of them at most).  A launch gets 48 KB, its static
// part included, without asking; above 40 KB the kernel is allowed the most that
// any call needs, always the same, so that no call takes away from another.
constexpr int SEQ_SMEM = 16384 * (int)sizeof(float2);
template <typename... P>
cudaError_t allow_smem(void (*kernel)(P...), int bytes) {
    return bytes <= 40 * 1024 ? cudaSuccess
                              : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SEQ_SMEM);
}

template <typename T, int VEC>
cudaError_t seq_fwd(const GnArgs &a, const Plan &p, cudaStream_t s) {
    const unsigned blocks = (unsigned)(a.Bt * p.nch);
    const int smem = (int)(seq_phases(a.C, VEC) * (a.C / VEC) * sizeof(float2));
    cudaError_t e;
    if ((e = allow_smem(k_gn_seq_stats<T, VEC>, smem)) != cudaSuccess) return e;
    k_gn_seq_stats<T, VEC><<<blocks, SQT, smem, s>>>(a, (int)p.rows, (int)p.nch);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int gsm = (int)(a.G * sizeof(float2));
#define GN_CALL(K)                                              \
    if ((e = allow_smem(K, gsm)) != cudaSuccess) return e;      \
    e = launch_after(K, dim3(blocks), SQT, gsm, s, a, (int)p.rows, (int)p.nch)
    GN_ACTS(GN_CALL, k_gn_seq_apply, T, VEC, )
#undef GN_CALL
    return e;
}

template <typename T, int VEC>
cudaError_t seq_bwd(const GnArgs &a, const Plan &p, cudaStream_t s) {
    const unsigned blocks = (unsigned)(a.Bt * p.nch);
    const int smem = (int)((seq_phases(a.C, VEC) - 1) * 2 * a.C * sizeof(float));   // below 16 KB: np C / VEC <= 256
    cudaError_t e;
#define GN_CALL(K) K<<<blocks, SQT, smem, s>>>(a, (int)p.rows, (int)p.nch)
    GN_ACTS(GN_CALL, k_gn_seq_bsums, T, VEC, )
#undef GN_CALL
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    float *sums = a.ws + (size_t)a.Bt * p.nch * 2 * a.C;
    float2 *mom = reinterpret_cast<float2 *>(sums + (size_t)a.Bt * 2 * a.C);
    if ((e = launch_after(k_gn_seq_moments, dim3((unsigned)(a.Bt * a.G)), 256, 0, s, a, (int)p.nch, sums, mom)) !=
        cudaSuccess)
        return e;
    const unsigned dxb = a.dx ? blocks : 0, rb = (a.dw || a.db) ? (unsigned)ceil_div(2 * a.C, 32) : 0;
    if (dxb + rb == 0) return cudaSuccess;
#define GN_CALL(K) e = launch_after(K, dim3(dxb + rb), SQT, 0, s, a, (int)p.rows, (int)p.nch, sums, mom, dxb)
    GN_ACTS(GN_CALL, k_gn_seq_dx, T, VEC, )
#undef GN_CALL
    return e;
}

}  // namespace

size_t gn_fwd_workspace_floats(int64_t Bt, int64_t L, int64_t C, int64_t G, m3_dtype dt) {
    const Plan p = plan_of(Bt, L, C, G, dt, false);
    return p.row ? 0 : (size_t)(Bt * p.nch * G) * 2;
}

size_t gn_bwd_workspace_floats(int64_t Bt, int64_t L, int64_t C, int64_t G, m3_dtype dt) {
    const Plan p = plan_of(Bt, L, C, G, dt, true);
    return p.row ? (size_t)p.parts * 2 * C : (size_t)Bt * (p.nch + 1) * 2 * C + (size_t)Bt * G * 2;
}

cudaError_t launch_gn_fwd(const GnArgs &a, m3_dtype dt, cudaStream_t s) {
    const Plan p = plan_of(a.Bt, a.L, a.C, a.G, dt, false);
    if (p.row)
        return dt == M3_BF16 ? row_dispatch<__nv_bfloat16, 8>(a, p, false, s) : row_dispatch<float, 4>(a, p, false, s);
    if (dt == M3_BF16) return p.vec == 8 ? seq_fwd<__nv_bfloat16, 8>(a, p, s) : seq_fwd<__nv_bfloat16, 1>(a, p, s);
    return p.vec == 4 ? seq_fwd<float, 4>(a, p, s) : seq_fwd<float, 1>(a, p, s);
}

cudaError_t launch_gn_bwd(const GnArgs &a, m3_dtype dt, cudaStream_t s) {
    if (a.Bt == 0 || a.L == 0) {                          // nothing was summed: zeros
        if (!(a.dw || a.db)) return cudaSuccess;
        k_gn_reduce<<<(unsigned)ceil_div(2 * a.C, 32), 1024, 0, s>>>(nullptr, 0, a.C, a.dw, a.db);
        count_launch();
        return cudaGetLastError();
    }
    const Plan p = plan_of(a.Bt, a.L, a.C, a.G, dt, true);
    if (p.row) {
        cudaError_t e =
            dt == M3_BF16 ? row_dispatch<__nv_bfloat16, 8>(a, p, true, s) : row_dispatch<float, 4>(a, p, true, s);
        if (e != cudaSuccess || !(a.dw || a.db)) return e;
        return launch_after(k_gn_reduce, dim3((unsigned)ceil_div(2 * a.C, 32)), 1024, 0, s, a.ws, p.parts, a.C, a.dw, a.db);
    }
    if (dt == M3_BF16) return p.vec == 8 ? seq_bwd<__nv_bfloat16, 8>(a, p, s) : seq_bwd<__nv_bfloat16, 1>(a, p, s);
    return p.vec == 4 ? seq_bwd<float, 4>(a, p, s) : seq_bwd<float, 1>(a, p, s);
}

}  // namespace m3
