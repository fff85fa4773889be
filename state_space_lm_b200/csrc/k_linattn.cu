// k_linattn.cu -- linear attention with a decay for each head: the fp32
// kernel for every size and type, the combine of a split time axis, the sum
// of per-head gradients over shared heads, and the single-token step.
#include <algorithm>

#include "launch.cuh"
#include "linattn.cuh"

namespace m3 {
namespace {

// ---------------------------------------------------------------- k_mix_simt
// One CTA owns one lane (or one segment of it) and 32 columns of c, and walks
// the tokens in blocks of 16.  With M the state entering a block, j the place
// in it and L its tokens:
//   y_j = scale_i g^(j+1) M^T a_j + sum_{i <= j} P_ji c_i,  P_ji = scale_p g^(j-i) (a_j . b_i)
//   M  <- M g^L + sum_i b_i (scale_w g^(L-1-i) c_i)^T     (M g^L as in decay_of)
// (walking backwards g^j and g^(L-i)).  A thread holds one column and RS rows
// of M in registers (warp = row slice, lane = column), so a and b rows are
// read from shared memory as broadcasts and the block's own part of M is
// summed before it meets M: a long sum loses no more than one rounding a
// block.  This is the path of fp32 inputs, whose products the tensor cores
// would round, and of sizes that TMA cannot address.  Bound by the chain of a
// lane's blocks at small sizes (3 x 333 tokens, 5 heads of 37 x 29, cut into
// segments: 24 us), by arithmetic and shared-memory reads at large ones (8 x 2048,
// 16 heads of 128 x 64: 680 us forward, 2227 backward).
constexpr int SC = 16, SP = 32, ST = 256;

template <int RS>
struct SimtSmem {
    static constexpr int DA = 8 * RS, LDA = DA + 4;     // row padding: conflict-free 16-byte reads down a column
    float a[SC][LDA], b[SC][LDA], c[SC][SP], p[SC][SC + 4], part[8][SC][SP], sp[8][SC][SC + 4];
    float pw[SC + 1], pm1[SC + 1];
};

// The mixes of a launch (blockIdx.z): the backward's three, or those of them
// that have the same width.  A single one has a variant of its own, whose
// arguments stand at fixed places (3 % of the forward).
template <int NB>
struct MixBatch {
    MixArgs g[NB];
};

template <typename T, int RS, bool SO, int NB>
__global__ void __launch_bounds__(ST, RS <= 4 ? 4 : RS <= 8 ? 3 : RS <= 16 ? 2 : 1) k_mix_simt(const __grid_constant__ MixBatch<NB> P) {
    using Sm = SimtSmem<RS>;
    const MixArgs &g = P.g[NB == 1 ? 0 : blockIdx.z];
    if ((int)blockIdx.y * SP >= g.dc) return;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Sm &sm = *reinterpret_cast<Sm *>(smem_raw);
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31;
    const int nsb = SO ? g.nseg - 1 : g.nseg;
    const int64_t lane = blockIdx.x / nsb, bi = lane / g.H, h = lane % g.H;
    const int seg = (int)(blockIdx.x % nsb);
    const int p0 = blockIdx.y * SP, pc = p0 + l;
    const bool col = pc < g.dc;
    const int64_t len = lane_length(g.lengths, bi, g.T);
    const int64_t t0 = seg_begin(seg, g.nseg, g.seg_len, g.reverse);
    const int64_t n = seg_tokens(seg, g.nseg, g.seg_len, g.reverse, len);
    if (tid <= SC) decay_pow_f32(g.log_decay[h], tid, sm.pw[tid], sm.pm1[tid]);
    const int64_t row0 = bi * g.T;
    const T *A = static_cast<const T *>(g.a) + (int64_t)(h / g.ra) * g.da;
    const T *B = static_cast<const T *>(g.b) + (int64_t)(h / g.rb) * g.da;
    const T *C = static_cast<const T *>(g.c) + (int64_t)(h / g.rc) * g.dc;
    const size_t elems = (size_t)g.da * g.dc;
    float *slots = g.ws + (size_t)lane * (g.nseg - 1) * elems;

    // the state: rows w*RS .. +RS of column pc
    float M[RS];
    {
        const float *src = (SO || (seg == 0 && !g.m0)) ? nullptr : (seg == 0 ? g.m0 + lane * elems : slots + (seg - 1) * elems);
        const bool tr = seg == 0 && g.m_trans;
#pragma unroll
        for (int i = 0; i < RS; i++) {
            const int r = w * RS + i;
            M[i] = (src && col && r < g.da) ? src[tr ? (size_t)pc * g.da + r : (size_t)r * g.dc + pc] : 0.f;
        }
    }

    // a block's rows travel through registers one block ahead: warp w takes
    // its places 2w and 2w+1
    constexpr int NV = RS / 4;                           // 32-wide pieces of a row
    float ra[2][NV], rb[2][NV], rc[2];
    auto fetch = [&](int64_t j0) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const int64_t j = j0 + 2 * w + u;
            const bool on = j < n;
            const int64_t t = row0 + (g.reverse ? t0 + n - 1 - j : t0 + j);
#pragma unroll
            for (int m = 0; m < NV; m++) {
                const int i = l + 32 * m;
                const bool in = on && i < g.da;
                if (!SO) ra[u][m] = in ? ldf(A, t * g.lda + i) : 0.f;
                rb[u][m] = in ? ldf(B, t * g.ldb + i) : 0.f;
            }
            rc[u] = (on && col) ? ldf(C, t * g.ldc + pc) : 0.f;
        }
    };
    if (n > 0) fetch(0);
    for (int64_t j0 = 0; j0 < n; j0 += SC) {
        const int L = (int)(n - j0 < SC ? n - j0 : SC);
        __syncthreads();                                 // the block before is read
#pragma unroll
        for (int u = 0; u < 2; u++) {
#pragma unroll
            for (int m = 0; m < NV; m++) {
                const int i = l + 32 * m;                // rows are 8 RS = 32 NV wide
                if (!SO) sm.a[2 * w + u][i] = ra[u][m];
                sm.b[2 * w + u][i] = rb[u][m];
            }
            sm.c[2 * w + u][l] = rc[u];
        }
        __syncthreads();
        if (j0 + SC < n) fetch(j0 + SC);
        if (!SO) {
            {
                // scores over this warp's rows of the state: a lane takes one row of
                // a against 8 of b, so that most reads are broadcasts
                const int j = l >> 1, i0 = (l & 1) * 8;
                float acc[8];
#pragma unroll
                for (int u = 0; u < 8; u++) acc[u] = 0.f;
#pragma unroll
                for (int k = 0; k < RS; k += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(&sm.a[j][w * RS + k]);
#pragma unroll
                    for (int u = 0; u < 8; u++) {
                        const float4 z = *reinterpret_cast<const float4 *>(&sm.b[i0 + u][w * RS + k]);
                        acc[u] = fmaf(x.x, z.x, acc[u]);
                        acc[u] = fmaf(x.y, z.y, acc[u]);
                        acc[u] = fmaf(x.z, z.z, acc[u]);
                        acc[u] = fmaf(x.w, z.w, acc[u]);
                    }
                }
                *reinterpret_cast<float4 *>(&sm.sp[w][j][i0]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                *reinterpret_cast<float4 *>(&sm.sp[w][j][i0 + 4]) = make_float4(acc[4], acc[5], acc[6], acc[7]);
            }
#pragma unroll 4
            for (int j = 0; j < SC; j++) {
                float acc = 0.f;
#pragma unroll
                for (int i = 0; i < RS; i += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(&sm.a[j][w * RS + i]);
                    acc = fmaf(x.x, M[i], acc);
                    acc = fmaf(x.y, M[i + 1], acc);
                    acc = fmaf(x.z, M[i + 2], acc);
                    acc = fmaf(x.w, M[i + 3], acc);
                }
                sm.part[w][j][l] = acc;
            }
        }
        {
            float own[RS];
#pragma unroll
            for (int i = 0; i < RS; i++) own[i] = 0.f;
#pragma unroll 4
            for (int j = 0; j < SC; j++) {                // rows behind the block's tokens are zeros
                const float cw = sm.c[j][l] * (sm.pw[max(0, g.reverse ? L - j : L - 1 - j)] * g.scale_w);
#pragma unroll
                for (int i = 0; i < RS; i += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(&sm.b[j][w * RS + i]);
                    own[i] = fmaf(x.x, cw, own[i]);
                    own[i + 1] = fmaf(x.y, cw, own[i + 1]);
                    own[i + 2] = fmaf(x.z, cw, own[i + 2]);
                    own[i + 3] = fmaf(x.w, cw, own[i + 3]);
                }
            }
            const Decay d = decay_of(sm.pw[L], sm.pm1[L]);
#pragma unroll
            for (int i = 0; i < RS; i++) M[i] = fmaf(M[i], d.keep, fmaf(M[i], d.f, own[i]));
        }
        if (!SO) {
            __syncthreads();
            {
                const int j = tid >> 4, i = tid & 15;
                float t = 0.f;
#pragma unroll
                for (int k = 0; k < 8; k++) t += sm.sp[k][j][i];
                sm.p[j][i] = t * (sm.pw[max(0, j - i)] * g.scale_p);
            }
            __syncthreads();
            // rows j = w and w + 8 of this thread's column
            float inter[2] = {0.f, 0.f}, intra[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 8; k++) {
                inter[0] += sm.part[k][w][l];
                inter[1] += sm.part[k][w + 8][l];
            }
#pragma unroll
            for (int i = 0; i < SC; i++) {                // later rows are left out, not multiplied by zero
                const float c = sm.c[i][l];
                if (i <= w) intra[0] = fmaf(sm.p[w][i], c, intra[0]);
                if (i <= w + 8) intra[1] = fmaf(sm.p[w + 8][i], c, intra[1]);
            }
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int j = w + 8 * u;
                if (j < L && col && g.y) {
                    const float y = fmaf(inter[u], sm.pw[g.reverse ? j : j + 1] * g.scale_i, intra[u]);
                    const int64_t t = row0 + (g.reverse ? t0 + n - 1 - (j0 + j) : t0 + j0 + j);
                    const int64_t o = (t * g.H + h) * g.dc + pc;
                    if (g.y_f32) stf(static_cast<float *>(g.y), o, y);
                    else stf(static_cast<T *>(g.y), o, y);
                }
            }
        }
    }
    float *dst = SO ? slots + seg * elems : (seg == g.nseg - 1 && g.m_out ? g.m_out + lane * elems : nullptr);
    if (dst && col) {
        const bool tr = !SO && g.m_trans;
#pragma unroll
        for (int i = 0; i < RS; i++) {
            const int r = w * RS + i;
            if (r < g.da) dst[tr ? (size_t)pc * g.da + r : (size_t)r * g.dc + pc] = M[i];
        }
    }
    if (!SO && col && g.y) {
        // rows behind the sequence, inside this segment: zeros
        const int64_t e = t0 + g.seg_len < g.T ? t0 + g.seg_len : g.T;
        const int64_t step = 8 * g.H * g.dc;
        int64_t o = ((row0 + t0 + n + w) * g.H + h) * g.dc + pc;
#pragma unroll 4
        for (int64_t t = t0 + n + w; t < e; t += 8, o += step) {
            if (g.y_f32) stf(static_cast<float *>(g.y), o, 0.f);
            else stf(static_cast<T *>(g.y), o, 0.f);
        }
    }
}

// Between the two passes of a split time axis: slot j holds segment j's own
// state (from zero) and receives the state entering segment j + 1,
//   M_(j+1) = g^n_j M_j + own_j.
// One thread per state element; bound by the slots' bytes, read and written
// once each.
__global__ void __launch_bounds__(256) k_mix_combine(const __grid_constant__ MixBatch<3> P) {
    __shared__ Decay dec[256];
    const MixArgs &g = P.g[blockIdx.z];
    const int64_t lane = blockIdx.x, bi = lane / g.H, h = lane % g.H;
    const int64_t len = lane_length(g.lengths, bi, g.T);
    const double lg = (double)g.log_decay[h];
    for (int j = threadIdx.x; j < g.nseg - 1; j += 256)
        dec[j] = decay_pow_f64(lg, seg_tokens(j, g.nseg, g.seg_len, g.reverse, len));
    __syncthreads();
    const size_t elems = (size_t)g.dar * g.dcr, i = (size_t)blockIdx.y * 256 + threadIdx.x;
    if (i >= elems) return;
    float M = 0.f;
    if (g.m0) {
        const size_t r = i / g.dcr, p = i % g.dcr;
        M = g.m0[lane * elems + (g.m_trans ? p * g.dar + r : i)];
    }
    float *sl = g.ws + (size_t)lane * (g.nseg - 1) * elems + i;
    for (int j = 0; j < g.nseg - 1; j++) {
        M = fmaf(M, dec[j].keep, fmaf(M, dec[j].f, sl[j * elems]));
        sl[j * elems] = M;
    }
}

// Copies into padded rows (PadArgs): a thread takes PAD_U 16-byte pieces 256
// apart, all of its loads before its stores.  Bound by HBM: 8 x 2048 tokens of
// 16 heads of 120 x 60 (q, k and v, 0.28 GB read and written) in 44 us.
constexpr int PAD_U = 4;
__global__ void __launch_bounds__(256) k_pad_rows(PadArgs a) {
    const int k = blockIdx.y;
    const int64_t n = a.n[k], i0 = (int64_t)blockIdx.x * (256 * PAD_U) + threadIdx.x;
    if (i0 >= n) return;
    const int d = a.d[k], w = (d + 7) / 8, heads = a.heads[k], vec = a.vec[k];
    const uint16_t *src = static_cast<const uint16_t *>(a.src[k]);
    uint32_t o[PAD_U][4];
#pragma unroll
    for (int u = 0; u < PAD_U; u++) {
        const int64_t i = i0 + 256 * u;
#pragma unroll
        for (int e = 0; e < 4; e++) o[u][e] = 0u;
        if (i >= n) continue;
        int64_t rh, row;
        if (n < (int64_t)1 << 31) {                       // 64-bit divisions would cost more than the copy
            rh = (unsigned)i / (unsigned)w;
            row = (unsigned)rh / (unsigned)heads;
        } else {
            rh = i / w;
            row = rh / heads;
        }
        const int c = (int)(i - rh * w) * 8, h = (int)(rh - row * heads);
        const uint16_t *p = src + row * a.ld[k] + (int64_t)h * d + c;
        if (vec == 4) {
#pragma unroll
            for (int e = 0; e < 4; e += 2)
                if (c + 2 * e < d) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(p + 2 * e);
                    o[u][e] = v.x;
                    o[u][e + 1] = v.y;
                }
        } else if (vec == 2) {
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (c + 2 * e < d) o[u][e] = *reinterpret_cast<const uint32_t *>(p + 2 * e);
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const uint32_t lo = c + 2 * e < d ? p[2 * e] : 0, hi = c + 2 * e + 1 < d ? p[2 * e + 1] : 0;
                o[u][e] = lo | hi << 16;
            }
        }
    }
    uint4 *dst = static_cast<uint4 *>(a.dst[k]);
#pragma unroll
    for (int u = 0; u < PAD_U; u++)
        if (i0 + 256 * u < n) dst[i0 + 256 * u] = make_uint4(o[u][0], o[u][1], o[u][2], o[u][3]);
}

// out[row, group, :] = sum over the group's heads of in[row, head, :], in
// fp32 and a fixed order, rounded once; one or two tensors (blockIdx.y).  Bound
// by reading `in`: VEC elements a thread, a head's loads in flight together
// (8 x 2048 tokens, 16 heads over 4 groups of 128, two tensors: 59 us, 5.7 TB/s).
struct HeadSum {
    const float *in[2];
    void *out[2];
    int64_t n;                                            // vectors of an output
    int rep, d, wide;                                     // columns of a row, and of a row of `in`
};
template <typename T, int VEC>
__global__ void __launch_bounds__(256) k_head_sum(HeadSum a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    pdl_wait();
    if (i >= a.n) return;
    const int w = a.d / VEC;                              // vectors of a row
    const int64_t rg = a.n < (int64_t)1 << 31 ? (unsigned)i / (unsigned)w : i / w;
    const int e = (int)(i - rg * w) * VEC;
    const float *p = a.in[blockIdx.y] + rg * a.rep * a.wide + e;
    float s[VEC];
#pragma unroll
    for (int k = 0; k < VEC; k++) s[k] = 0.f;
#pragma unroll 4
    for (int r = 0; r < a.rep; r++, p += a.wide) {
        if (VEC == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p);
            s[0] += v.x; s[VEC - 3] += v.y; s[VEC - 2] += v.z; s[VEC - 1] += v.w;
        } else {
            s[0] += p[0];
        }
    }
    T *o = static_cast<T *>(a.out[blockIdx.y]) + i * VEC;
#pragma unroll
    for (int k = 0; k < VEC; k++) stf(o, k, s[k]);
}

// -------------------------------------------------------------- k_lin_step
// One token of every lane: S <- S + (S (g - 1) + k v^T), y = scale S^T q.
// One CTA per lane.  The state is read once and written once in VEC-wide
// pieces: thread = (row of R, piece of a row), so a warp's accesses are
// contiguous; the y sums over rows meet in shared memory.  The first rows of
// the state are on their way before anything else is read (a lane of 128 x 64
// then has its whole 32 KB in flight).  Bound by the state's bytes: 512 x 16
// lanes of 128 x 64 in 86 to 87 us, 95 % of the copy rate.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) k_lin_step(LinStepArgs a) {
    __shared__ float qs[256], ks[256], vs[256];
    __shared__ float red[256 * VEC];
    const int tid = threadIdx.x;
    const unsigned lane = blockIdx.x, H = (unsigned)a.H, b = lane / H, h = lane - b * H;
    const int dk = (int)a.dk, dv = (int)a.dv;
    const int cols = dv / VEC, R = 256 / cols;            // pieces of a row, rows at a time
    const int r0 = (int)((unsigned)tid / (unsigned)cols), c = tid - r0 * cols;
    constexpr int U = 8;
    float *S = a.s + (size_t)lane * dk * dv + VEC * c;
    float x[U][VEC], acc[VEC];
    auto fetch = [&](int rr) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int r = rr + u * R;
            if (r < dk) {
                if (VEC == 4) *reinterpret_cast<float4 *>(x[u]) = *reinterpret_cast<const float4 *>(S + r * dv);
                else x[u][0] = S[r * dv];
            }
        }
    };
    if (r0 < R) fetch(r0);
    const int hg = (int)(h / (unsigned)(a.H / a.G));
    const T *q = static_cast<const T *>(a.q) + b * a.ldq + hg * dk;
    const T *k = static_cast<const T *>(a.k) + b * a.ldk + hg * dk;
    const T *v = static_cast<const T *>(a.v) + b * a.ldv + (int)h * dv;
    if (tid < dk) {
        qs[tid] = ldf(q, tid) * a.scale;
        ks[tid] = ldf(k, tid);
    }
    if (tid < dv) vs[tid] = ldf(v, tid);
    // S keep + (S f + k v): S + (S (g - 1) + k v) for g >= 1/2, S g + k v below.  The
    // first does not inherit the rounding of a g near 1, token after token; but it
    // rounds at the size of the old S, which is too much for the small state that
    // a strong decay leaves (none of the old one at log_decay = -inf)
    const float lg = a.log_decay[h];
    const bool strong = lg < -0.69314718f;
    const float keep = strong ? 0.f : 1.f, f = strong ? expf(lg) : expm1f(lg);
#pragma unroll
    for (int e = 0; e < VEC; e++) acc[e] = 0.f;
    __syncthreads();
    if (r0 < R) {
        for (int rr = r0; rr < dk; rr += U * R) {
            if (rr > r0) fetch(rr);
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int r = rr + u * R;
                if (r < dk) {
                    const float kr = ks[r], qr = qs[r];
#pragma unroll
                    for (int e = 0; e < VEC; e++) {
                        x[u][e] = fmaf(x[u][e], keep, fmaf(x[u][e], f, kr * vs[VEC * c + e]));
                        acc[e] = fmaf(qr, x[u][e], acc[e]);
                    }
                    if (VEC == 4) *reinterpret_cast<float4 *>(S + r * dv) = *reinterpret_cast<float4 *>(x[u]);
                    else S[r * dv] = x[u][0];
                }
            }
        }
#pragma unroll
        for (int e = 0; e < VEC; e++) red[(r0 * cols + c) * VEC + e] = acc[e];
    }
    __syncthreads();
    if (tid < dv) {
        float s = 0.f;
        for (int r = 0; r < R; r++) s += red[r * dv + tid];
        stf(static_cast<T *>(a.y), (int64_t)lane * dv + tid, s);
    }
}

template <typename T, int RS, int NB>
cudaError_t launch_mix_simt_t(const MixArgs *m, int n, cudaStream_t s) {
    constexpr int smem = (int)sizeof(SimtSmem<RS>);
    const int64_t lanes = m[0].Bt * m[0].H;
    const int nseg = m[0].nseg;
    unsigned tiles = 1;
    MixBatch<NB> b;
    for (int i = 0; i < n; i++) {
        b.g[i] = m[i];
        tiles = std::max(tiles, (unsigned)((m[i].dc + SP - 1) / SP));
    }
    cudaError_t e;
    if (nseg > 1) {
        if ((e = cudaFuncSetAttribute(k_mix_simt<T, RS, true, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) !=
            cudaSuccess)
            return e;
        k_mix_simt<T, RS, true, NB><<<dim3((unsigned)(lanes * (nseg - 1)), tiles, n), ST, smem, s>>>(b);
        count_launch();
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = launch_mix_combine(m, n, s)) != cudaSuccess) return e;
    }
    if ((e = cudaFuncSetAttribute(k_mix_simt<T, RS, false, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) !=
        cudaSuccess)
        return e;
    k_mix_simt<T, RS, false, NB><<<dim3((unsigned)(lanes * nseg), tiles, n), ST, smem, s>>>(b);
    count_launch();
    return cudaGetLastError();
}

template <typename T, int NB>
cudaError_t launch_mix_simt_d(const MixArgs *m, int n, cudaStream_t s) {
    switch (m[0].wide) {
        case 32: return launch_mix_simt_t<T, 4, NB>(m, n, s);
        case 64: return launch_mix_simt_t<T, 8, NB>(m, n, s);
        case 128: return launch_mix_simt_t<T, 16, NB>(m, n, s);
        default: return launch_mix_simt_t<T, 32, NB>(m, n, s);
    }
}
template <typename T>
cudaError_t launch_mix_simt_n(const MixArgs *m, int n, cudaStream_t s) {
    return n == 1 ? launch_mix_simt_d<T, 1>(m, n, s) : launch_mix_simt_d<T, 3>(m, n, s);
}

}  // namespace

// Split the time axis where it pays: the second pass repeats 0.4 of the first
// one's work (without answers), but lanes that leave SMs idle fill them.  Costs
// are counted in blocks of 16 tokens, plus 2 to a CTA and 3 to the launches
// between; m CTAs on an SM take 1 + 0.4 (m - 1) of one's time, up to the number
// that its registers hold.  At most 64 segments and 64 MB of states.
// Measured against one piece of each lane: 3 x 333 tokens, 5 heads of 37 x 29:
// 53 us, 24 in seven; 2 x 1000, 4 of 128 x 128: 252 us, 70 in nine (one wave), 95
// in eleven (two); 8 x 2048, 16 of 128 x 64: 712 us, 850 in two.
static void plan_group(MixArgs *m, int n, int wide) {
    int64_t ctas = 0;
    const int64_t lanes = m[0].Bt * m[0].H, T = m[0].T, nb = (T + SC - 1) / SC;
    for (int i = 0; i < n; i++)
        if (m[i].wide == wide) {
            m[i].nseg = 1;
            m[i].seg_len = T > 0 ? T : 1;
            ctas += lanes * ((m[i].dc + SP - 1) / SP);
        }
    if (ctas == 0 || ctas >= 296 || T < 96) return;
    const int most_cta = wide <= 32 ? 4 : wide <= 64 ? 3 : wide <= 128 ? 2 : 1;
    auto cost = [&](int64_t c, double len) {
        const int64_t wave = 148 * most_cta, rest = c % wave;
        double t = (double)(c / wave) * (1 + 0.4 * (most_cta - 1));
        if (rest > 0) t += 1 + 0.4 * (double)((rest + 147) / 148 - 1);
        return t * (len + 2);
    };
    const int64_t most = ((int64_t)64 << 20) / (lanes * m[0].da * m[0].dc * 4) + 1;
    double best = cost(ctas, (double)nb);
    for (int64_t ns = 2; ns <= 64 && ns <= most; ns++) {
        const int64_t len = (nb + ns - 1) / ns, k = (nb + len - 1) / len;
        if (len < 2) break;
        const double c = cost(ctas * k, (double)len) + cost(ctas * (k - 1), 0.4 * (double)len) + 3;
        if (k > 1 && c < best) {
            best = c;
            for (int i = 0; i < n; i++)
                if (m[i].wide == wide) {
                    m[i].nseg = (int)k;
                    m[i].seg_len = len * SC;
                }
        }
    }
}

// Mixes of one width share their launches; all of a call do, at the widest
// one's, where together they are fewer CTAs than SMs (the backward of 3 x 333
// tokens, 5 heads of 37 x 29: 73 us one by one, 47 us together).
void mix_simt_plan(MixArgs *m, int n) {
    int widest = 32;
    int64_t ctas = 0;
    for (int i = 0; i < n; i++) {
        m[i].wide = m[i].da <= 32 ? 32 : m[i].da <= 64 ? 64 : m[i].da <= 128 ? 128 : 256;
        widest = std::max(widest, m[i].wide);
        ctas += m[i].Bt * m[i].H * ((m[i].dc + SP - 1) / SP);
    }
    if (ctas <= 148)
        for (int i = 0; i < n; i++) m[i].wide = widest;
    for (int wide : {32, 64, 128, 256}) plan_group(m, n, wide);
}

cudaError_t launch_mix_simt(const MixArgs *m, int n, m3_dtype dt, cudaStream_t s) {
    for (int wide : {32, 64, 128, 256}) {
        MixArgs g[3];
        int k = 0;
        for (int i = 0; i < n; i++)
            if (m[i].wide == wide) g[k++] = m[i];
        if (k == 0) continue;
        const cudaError_t e = dt == M3_BF16 ? launch_mix_simt_n<__nv_bfloat16>(g, k, s) : launch_mix_simt_n<float>(g, k, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}


cudaError_t launch_mix_combine(const MixArgs *m, int n, cudaStream_t s) {
    MixBatch<3> b;
    int k = 0;
    for (int i = 0; i < n; i++)
        if (m[i].nseg > 1) b.g[k++] = m[i];
    if (k == 0) return cudaSuccess;
    const MixArgs &a = b.g[0];                            // the others' states have as many elements
    k_mix_combine<<<dim3((unsigned)(a.Bt * a.H), (unsigned)((a.dar * a.dcr + 255) / 256), k), 256, 0, s>>>(b);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_head_sum(const float *const in[2], void *const out[2], int count, m3_dtype dt, int64_t rows, int64_t H,
                            int64_t G, int64_t d, int64_t wide, cudaStream_t s) {
    const bool v4 = d % 4 == 0;
    HeadSum a;
    for (int i = 0; i < 2; i++) {
        a.in[i] = in[i];
        a.out[i] = out[i];
    }
    a.n = rows * G * d / (v4 ? 4 : 1);
    a.rep = (int)(H / G);
    a.d = (int)d;
    a.wide = (int)wide;
    if (a.n == 0) return cudaSuccess;
    const dim3 grid((unsigned)((a.n + 255) / 256), count);
    if (dt == M3_BF16)
        return v4 ? launch_after(k_head_sum<__nv_bfloat16, 4>, grid, 256, 0, s, a)
                  : launch_after(k_head_sum<__nv_bfloat16, 1>, grid, 256, 0, s, a);
    return v4 ? launch_after(k_head_sum<float, 4>, grid, 256, 0, s, a) : launch_after(k_head_sum<float, 1>, grid, 256, 0, s, a);
}

cudaError_t launch_pad_rows(const PadArgs &in, cudaStream_t s) {
    PadArgs a = in;
    int64_t most = 0;
    for (int i = 0; i < a.count; i++) {
        if (a.n[i] > most) most = a.n[i];
        const bool four = a.d[i] % 4 == 0 && a.ld[i] % 4 == 0 && (uintptr_t)a.src[i] % 8 == 0;
        const bool two = a.d[i] % 2 == 0 && a.ld[i] % 2 == 0 && (uintptr_t)a.src[i] % 4 == 0;
        a.vec[i] = four ? 4 : two ? 2 : 1;
    }
    if (most == 0) return cudaSuccess;
    k_pad_rows<<<dim3((unsigned)((most + 256 * PAD_U - 1) / (256 * PAD_U)), a.count), 256, 0, s>>>(a);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_linattn_step(const LinStepArgs &a, m3_dtype dt, cudaStream_t s) {
    const unsigned lanes = (unsigned)(a.Bt * a.H);
    const bool v4 = a.dv % 4 == 0;
    if (dt == M3_BF16) {
        if (v4) k_lin_step<__nv_bfloat16, 4><<<lanes, 256, 0, s>>>(a);
        else k_lin_step<__nv_bfloat16, 1><<<lanes, 256, 0, s>>>(a);
    } else {
        if (v4) k_lin_step<float, 4><<<lanes, 256, 0, s>>>(a);
        else k_lin_step<float, 1><<<lanes, 256, 0, s>>>(a);
    }
    count_launch();
    return cudaGetLastError();
}

}  // namespace m3
