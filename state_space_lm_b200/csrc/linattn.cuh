// linattn.cuh -- shared declarations of the linear-attention kernels (not
// part of the ABI).
//
// Forward and backward are one operation, a causal mix of three row
// sequences a_t (width da), b_t (width da), c_t (width dc) of one lane:
//
//   y_t = scale_p sum_{s <= t} g^(t-s) (a_t . b_s) c_s + scale_i g^(t+1) M0^T a_t
//
// with the state M_t = g M_{t-1} + scale_w b_t c_t^T carried along (g the
// lane's decay, t counted in walking order).  The three uses:
//   y  = mix(q, k, v)   forwards,  M = S
//   dq = mix(dy, v, k)  forwards,  M = S^T          (dq_t = scale S_t dy_t)
//   dk = mix(v, dy, q)  backwards, M = Z^T          (dk_t = Z_t v_t)
//   dv = mix(k, q, dy)  backwards, M = Z            (dv_t = Z_t^T k_t)
// where Z_t = scale q_t dy_t^T + g Z_{t+1} is the adjoint of S_t.  Walking
// backwards the carried state is g Z, the adjoint before the walk's next
// token, so its powers are one lower in the answers and one higher in the
// state (`reverse` below).
#pragma once
#include "m3_internal.cuh"

namespace m3 {

struct MixArgs {
    const void *a, *b, *c;
    int64_t lda, ldb, ldc;       // elements between the rows of consecutive tokens
    int ra, rb, rc;              // lanes' heads that share one head of a, b, c
    int da, dc;                  // width of a and b rows, of c rows, in memory
    int dar, dcr;                // the same without padding: widths of the states and of y
    const float *log_decay;      // (H), natural logarithm
    const int32_t *lengths;      // (Bt) tokens of each sequence, or NULL for T
    const float *m0;             // state the walk starts from, or NULL for zero
    float *m_out;                // state after the walk, or NULL
    int m_trans;                 // m0, m_out hold the state transposed, (dcr, dar) instead of (dar, dcr)
    void *y;                     // (Bt, T, H, dcr), or NULL when only m_out is wanted
    int y_f32;                   // y in fp32, rows of dc elements (else the input type, rows of dcr)
    int64_t Bt, T, H;
    int reverse;
    float scale_p, scale_i, scale_w;
    int nseg;                    // segments of the time axis, in walking order
    int64_t seg_len;             // tokens of a segment
    int wide;                    // fp32 kernel: the variant, rows of a and b up to 32, 64, 128 or 256
    float *ws;                   // (nseg - 1) states of dar * dcr floats for each lane
};

struct LinStepArgs {
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;       // elements between the rows of consecutive sequences
    const float *log_decay;
    float *s;
    void *y;
    int64_t Bt, H, G, dk, dv;
    float scale;
};

// Tokens of segment j (walking order) of a sequence of `len` tokens whose
// padded length is T.  Segments are cut at multiples of seg_len from the
// sequence's first token; walking backwards, segment 0 is the last of them.
__host__ __device__ __forceinline__ int64_t seg_begin(int j, int nseg, int64_t seg_len, int reverse) {
    return (int64_t)(reverse ? nseg - 1 - j : j) * seg_len;
}
__device__ __forceinline__ int64_t seg_tokens(int j, int nseg, int64_t seg_len, int reverse, int64_t len) {
    const int64_t t0 = seg_begin(j, nseg, seg_len, reverse);
    const int64_t n = len - t0;
    return n < 0 ? 0 : (n < seg_len ? n : seg_len);
}
__device__ __forceinline__ int64_t lane_length(const int32_t *lengths, int64_t b, int64_t T) {
    if (!lengths) return T;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : (n > T ? T : n);
}
// How a state M is multiplied by p = g^n: as keep M + M f.  For p >= 1/2, M + M
// (p - 1), so that it does not inherit the rounding of a p near 1 from chunk to
// chunk.  Below, M p: p - 1 rounds at 2^-25 whatever p is, which is all there is
// of a small p.  g^0 is 1 for a decay of zero too (log_decay = -inf).
struct Decay {
    float keep, f;
};
__device__ __forceinline__ Decay decay_of(float p, float pm1) {
    return p < 0.5f ? Decay{0.f, p} : Decay{1.f, pm1};
}
// from 64 bits, for any whole n >= 0
__device__ __forceinline__ Decay decay_pow_f64(double lg, int64_t n) {
    const double x = lg * (double)n, m = n == 0 ? 0. : expm1(x);
    return m < -0.5 ? Decay{0.f, (float)exp(x)} : Decay{1.f, (float)m};
}

// g^n and g^n - 1 from fp32 arithmetic for n <= 64, within a few roundings: the
// product's own rounding is put back in (its derivative is the power itself).
// (A double exp is 2 KB of code that every CTA of a short kernel waits for.)
__device__ __forceinline__ void decay_pow_f32(float lg, int n, float &p, float &pm1) {
    const float x = lg * (float)n;
    const float e = isfinite(x) ? fmaf(lg, (float)n, -x) : 0.f;
    const float m = expm1f(x);
    pm1 = n == 0 ? 0.f : fmaf(m + 1.f, e, m);
    p = n == 0 ? 1.f : expf(x) * (1.f + e);
}

// segment plan (nseg, seg_len) and launch of the fp32 kernel: any sizes
// within the limits
void mix_simt_plan(MixArgs *m, int n);
cudaError_t launch_mix_simt(const MixArgs *m, int n, m3_dtype dt, cudaStream_t s);
// The tensor-core kernel: bf16, widths at most 128, widths and row strides
// multiples of 8, 16-byte aligned bases.  Up to three problems of one batch share
// their launches.
bool mix_tc_sizes(const MixArgs &a, m3_dtype dt);
void mix_tc_plan(MixArgs *a, int n);
cudaError_t launch_mix_tc(const MixArgs *a, int n, cudaStream_t s);
int mix_tc_error_and_clear(cudaStream_t s);
// chains the segments' states between the two passes
cudaError_t launch_mix_combine(const MixArgs *m, int n, cudaStream_t s);
// Rows whose width or stride TMA cannot address, copied into rows padded with
// zeros to a multiple of 8 columns: up to four tensors in one launch.
struct PadArgs {
    const void *src[4];          // (rows, heads, d) bf16, ld elements from row to row
    void *dst[4];                // (rows, heads, (d + 7) / 8 * 8), contiguous, 16-byte aligned
    int64_t ld[4], n[4];         // n: 8-column pieces of dst
    int heads[4], d[4];
    int vec[4];                  // elements of a load, as rows and base allow (launch_pad_rows sets it)
    int count;
};
cudaError_t launch_pad_rows(const PadArgs &a, cudaStream_t s);
// sums one or two fp32 (Bt, T, H, wide) tensors over the heads of each of G
// groups; d of the wide columns are real
cudaError_t launch_head_sum(const float *const in[2], void *const out[2], int count, m3_dtype dt, int64_t rows, int64_t H,
                            int64_t G, int64_t d, int64_t wide, cudaStream_t s);
cudaError_t launch_linattn_step(const LinStepArgs &a, m3_dtype dt, cudaStream_t s);

}  // namespace m3
