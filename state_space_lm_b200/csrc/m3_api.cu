// m3_api.cu -- the C ABI declared in include/m3.h: argument validation on
// the host, then kernel launches on the caller's stream.  Nothing here
// allocates, frees or synchronises.
#include <atomic>
#include <cmath>
#include <initializer_list>

#include "group_norm.cuh"
#include "linattn.cuh"
#include "m3_internal.cuh"

namespace m3 {
static std::atomic<uint64_t> g_launches{0};
void count_launch(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }
}  // namespace m3

using namespace m3;

namespace {

constexpr int64_t kMaxDstate = 256, kMaxHeaddim = 256, kMaxStateElems = 16384, kMaxRank = 8;
// Every kernel runs one CTA per (batch, head) lane in a 1-D grid, and no
// tensor may hold more than 2^46 elements (far beyond device memory), so
// that every index product below stays well inside int64.
constexpr int64_t kMaxLanes = 0x7fffffff, kMaxElems = (int64_t)1 << 46;

// Product of non-negative sizes, saturated at kMaxElems + 1.
int64_t sat_product(std::initializer_list<int64_t> f) {
    for (int64_t v : f)
        if (v == 0) return 0;
    int64_t p = 1;
    for (int64_t v : f) {
        if (v > kMaxElems || p > kMaxElems / v) return kMaxElems + 1;
        p *= v;
    }
    return p;
}

// The requested chunk as an int: any request of 2^30 tokens or more behaves
// as 2^30 (longer than any supported sequence).
inline int chunk_request(int64_t c) { return (int)(c < ((int64_t)1 << 30) ? c : ((int64_t)1 << 30)); }

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// required pointer: non-null and 16-byte aligned
#define M3_REQ(p)                                                  \
    do {                                                           \
        if (!(p) || !aligned16(p)) return M3_ERR_INVALID_ARG;      \
    } while (0)
// optional pointer: null, or 16-byte aligned
#define M3_OPT(p)                                                  \
    do {                                                           \
        if ((p) && !aligned16(p)) return M3_ERR_INVALID_ARG;       \
    } while (0)

m3_status check_dtype(m3_dtype t) {
    return (t == M3_F32 || t == M3_BF16) ? M3_OK : M3_ERR_INVALID_ARG;
}

// Sizes shared by the scan, rope and decode entry points.
m3_status check_core_dims(const m3_dims &d, bool need_seq) {
    if (d.batch < 0 || d.nheads < 1 || d.headdim < 1 || d.dstate < 2) return M3_ERR_INVALID_ARG;
    if (need_seq && d.seqlen < 0) return M3_ERR_INVALID_ARG;
    if (d.dstate & 1) return M3_ERR_INVALID_ARG;  // RoPE pairs need an even dstate
    if (d.dstate > kMaxDstate || d.headdim > kMaxHeaddim || d.dstate * d.headdim > kMaxStateElems)
        return M3_ERR_UNSUPPORTED;
    if (d.batch > (int64_t)1 << 24 || d.nheads > 4096 || (need_seq && d.seqlen > ((int64_t)1 << 31)))
        return M3_ERR_UNSUPPORTED;
    if (d.batch * d.nheads > kMaxLanes) return M3_ERR_UNSUPPORTED;
    const int64_t width = d.headdim > d.dstate ? d.headdim : d.dstate;
    if (need_seq && sat_product({d.batch, d.seqlen, d.nheads, width}) > kMaxElems) return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

// B/C groups and rotated pairs, with 0 meaning one group per head and every
// pair (TorchMamba README, "Models": n_groups with H % G == 0; dotLLM pull
// request, real-checkpoint run: num_rope_angles of dstate).
m3_status resolve_groups(const m3_dims &d, int64_t &G, int64_t &K) {
    if (d.ngroups < 0 || d.rope_pairs < 0) return M3_ERR_INVALID_ARG;
    G = d.ngroups ? d.ngroups : d.nheads;
    K = d.rope_pairs ? d.rope_pairs : d.dstate / 2;
    if (d.nheads % G || K > d.dstate / 2) return M3_ERR_INVALID_ARG;
    return M3_OK;
}

m3_status read_norm(const m3_bcnorm *n, NormArgs &o) {
    o = NormArgs{nullptr, nullptr, nullptr, nullptr, 0.f};
    if (!n) return M3_OK;
    M3_OPT(n->normw_B);
    M3_OPT(n->normw_C);
    M3_OPT(n->bias_B);
    M3_OPT(n->bias_C);
    if ((n->normw_B || n->normw_C) && !(n->eps >= 0.f && std::isfinite(n->eps))) return M3_ERR_INVALID_ARG;
    o = NormArgs{n->normw_B, n->normw_C, n->bias_B, n->bias_C, n->eps};
    return M3_OK;
}

inline m3_status launched(cudaError_t e) { return e == cudaSuccess ? M3_OK : M3_ERR_CUDA; }

// Failure-injection hook (m3_debug_fail_next_launches): the next n calls that
// pass validation report a launch failure without launching anything.
std::atomic<int> g_fail_launches{0};
inline bool injected_failure() {
    int n = g_fail_launches.load(std::memory_order_relaxed);
    while (n > 0)
        if (g_fail_launches.compare_exchange_weak(n, n - 1, std::memory_order_relaxed)) return true;
    return false;
}

// Every entry point ends here, after its validation: the launch, or the
// injected failure in its place.
template <typename F>
inline m3_status launch_unless_injected(F &&launch) {
    if (injected_failure()) return M3_ERR_CUDA;
    return launched(launch());
}

m3_status chunked_common(const void *x, const float *dt, const float *A, const float *lam,
                         const float *theta, const void *B, const void *C, const float *D,
                         const float *Wx, const float *Wy, m3_dtype dtype, const m3_bcnorm *norm,
                         const float *h0, const float *prevBx0, const float *angle0, m3_dims d,
                         void *y, float *h_final, float *prevBx_final, float *angle_final,
                         void *workspace, size_t ws_bytes, void *stream, bool mimo) {
    m3_status st;
    if ((st = check_dtype(dtype)) != M3_OK) return st;
    if ((st = check_core_dims(d, true)) != M3_OK) return st;
    if (d.chunk < 1) return M3_ERR_INVALID_ARG;
    int64_t G, K;
    if ((st = resolve_groups(d, G, K)) != M3_OK) return st;
    const int64_t R = mimo ? d.rank : 1;
    if (mimo && d.rank < 1) return M3_ERR_INVALID_ARG;
    if (R > kMaxRank) return M3_ERR_UNSUPPORTED;
    M3_REQ(A);
    M3_REQ(D);
    const bool have_tokens = d.batch > 0 && d.seqlen > 0;
    if (have_tokens) {
        M3_REQ(x); M3_REQ(dt); M3_REQ(lam); M3_REQ(theta); M3_REQ(B); M3_REQ(C); M3_REQ(y);
    } else {
        M3_OPT(x); M3_OPT(dt); M3_OPT(lam); M3_OPT(theta); M3_OPT(B); M3_OPT(C); M3_OPT(y);
    }
    M3_OPT(Wx); M3_OPT(Wy); M3_OPT(h0); M3_OPT(prevBx0); M3_OPT(angle0);
    M3_OPT(h_final); M3_OPT(prevBx_final); M3_OPT(angle_final); M3_OPT(workspace);
    NormArgs nrm;
    if ((st = read_norm(norm, nrm)) != M3_OK) return st;
    const size_t need = m3_workspace_bytes(mimo ? M3_WS_MIMO : M3_WS_SISO, d, dtype);
    if (need > 0 && (!workspace || ws_bytes < need)) return M3_ERR_WORKSPACE;
    const int q = scan_simt_chunk(d.headdim, d.dstate, R, d.chunk);
    if (q < 1) return M3_ERR_UNSUPPORTED;
    if (d.batch == 0) return M3_OK;
    if (d.seqlen > ((int64_t)1 << 30)) return M3_ERR_UNSUPPORTED;

    ScanArgs a;
    a.x = x; a.B = B; a.C = C;
    a.dt = dt; a.A = A; a.lam = lam; a.theta = theta; a.D = D; a.Wx = Wx; a.Wy = Wy;
    a.h0 = h0; a.prevBx0 = prevBx0; a.angle0 = angle0;
    a.nrm = nrm;
    a.y = y; a.h_out = h_final; a.prevBx_out = prevBx_final; a.angle_out = angle_final;
    a.Bt = d.batch; a.T = d.seqlen; a.H = d.nheads; a.P = d.headdim; a.N = d.dstate; a.R = R;
    a.G = G; a.K = K;
    a.mimo_layout = mimo ? 1 : 0;
    a.ws = workspace;
    a.Q = chunk_request(d.chunk);
    if (scan_tc_supported(a, dtype))
        return launch_unless_injected([&] { return launch_scan_tc(a, (cudaStream_t)stream); });
    a.Q = q;
    return launch_unless_injected([&] { return launch_scan_simt(a, dtype, (cudaStream_t)stream); });
}

}  // namespace

extern "C" {

m3_limits m3_get_limits(void) { return m3_limits{kMaxDstate, kMaxHeaddim, kMaxStateElems, kMaxRank}; }

uint64_t m3_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

const char *m3_status_string(m3_status s) {
    switch (s) {
        case M3_OK: return "M3_OK: success";
        case M3_ERR_INVALID_ARG: return "M3_ERR_INVALID_ARG: null, misaligned or inconsistent argument";
        case M3_ERR_UNSUPPORTED: return "M3_ERR_UNSUPPORTED: sizes outside this build's limits";
        case M3_ERR_WORKSPACE: return "M3_ERR_WORKSPACE: workspace missing or too small";
        case M3_ERR_CUDA: return "M3_ERR_CUDA: a kernel launch failed";
        case M3_ERR_TIMEOUT: return "M3_ERR_TIMEOUT: a bounded wait inside a kernel gave up";
    }
    return "unknown m3_status";
}

m3_status m3_device_error(void *stream, int *site) {
    // one error word for the scan's kernels, one for the mixes' (sites from 101)
    int e = scan_tc_error_and_clear((cudaStream_t)stream);
    if (e >= 0) {
        const int e2 = mix_tc_error_and_clear((cudaStream_t)stream);
        if (e2 != 0 && e == 0) e = e2;
    }
    if (site) *site = e > 0 ? e : 0;
    if (e < 0) return M3_ERR_CUDA;
    if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return M3_ERR_CUDA;
    return e ? M3_ERR_TIMEOUT : M3_OK;
}

void m3_debug_fail_next_launches(int n) { g_fail_launches.store(n > 0 ? n : 0, std::memory_order_relaxed); }

m3_status m3_selftest_bounded_wait(void *stream) {
    return launch_unless_injected(
        [&] { return launch_wait_selftest(M3_SELFTEST_SITE, (cudaStream_t)stream); });
}

size_t m3_workspace_bytes(int which, m3_dims d, m3_dtype dtype) {
    if (which == M3_WS_BWD_SISO || which == M3_WS_BWD_MIMO) {
        BwdArgs b{};
        if (check_core_dims(d, true) != M3_OK || d.chunk < 1 || resolve_groups(d, b.G, b.K) != M3_OK) return 0;
        b.Bt = d.batch; b.T = d.seqlen; b.H = d.nheads; b.P = d.headdim; b.N = d.dstate;
        b.R = which == M3_WS_BWD_MIMO ? (d.rank > 1 ? d.rank : 1) : 1;
        b.Q = (int)(d.chunk < 64 ? d.chunk : 64);
        return scan_bwd_workspace_bytes(b);
    }
    // only the tensor-core path uses scratch (long sequences over few lanes)
    if ((which != M3_WS_SISO && which != M3_WS_MIMO) || check_core_dims(d, true) != M3_OK || d.chunk < 1) return 0;
    ScanArgs a{};
    if (resolve_groups(d, a.G, a.K) != M3_OK) return 0;
    a.Bt = d.batch; a.T = d.seqlen; a.H = d.nheads; a.P = d.headdim; a.N = d.dstate;
    a.R = which == M3_WS_MIMO ? d.rank : 1;
    a.Q = chunk_request(d.chunk); a.mimo_layout = which == M3_WS_MIMO ? 1 : 0;
    if (!scan_tc_supported(a, dtype)) return 0;
    return scan_tc_workspace_bytes(d.batch, d.nheads, d.seqlen);
}

m3_status m3_discretize(const float *dt, const float *A, const float *lam, m3_dims d, float *alpha,
                        float *beta, float *gamma, void *stream) {
    if (d.batch < 0 || d.seqlen < 0 || d.nheads < 1) return M3_ERR_INVALID_ARG;
    if (sat_product({d.batch, d.seqlen, d.nheads}) > kMaxElems) return M3_ERR_UNSUPPORTED;
    M3_REQ(A);
    if (d.batch * d.seqlen == 0) return M3_OK;
    M3_REQ(dt); M3_REQ(lam); M3_REQ(alpha); M3_REQ(beta); M3_REQ(gamma);
    return launch_unless_injected([&] {
        return launch_discretize(dt, A, lam, d.batch, d.seqlen, d.nheads, alpha, beta, gamma, (cudaStream_t)stream);
    });
}

m3_status m3_rope_bc(const void *B, const void *C, m3_dtype dtype, const float *theta, const float *dt,
                     const float *angle0, const m3_bcnorm *norm, m3_dims d, void *B_rot, void *C_rot,
                     float *angle_final, void *stream) {
    m3_status st;
    if ((st = check_dtype(dtype)) != M3_OK) return st;
    if ((st = check_core_dims(d, true)) != M3_OK) return st;
    int64_t G, K;
    if ((st = resolve_groups(d, G, K)) != M3_OK) return st;
    const int64_t R = d.rank > 1 ? d.rank : 1;
    if (d.rank < 0) return M3_ERR_INVALID_ARG;
    if (R > kMaxRank) return M3_ERR_UNSUPPORTED;
    if (d.batch > 0 && d.seqlen > 0) {
        M3_REQ(B); M3_REQ(C); M3_REQ(theta); M3_REQ(dt); M3_REQ(B_rot); M3_REQ(C_rot);
    }
    M3_OPT(angle0); M3_OPT(angle_final);
    NormArgs nrm;
    if ((st = read_norm(norm, nrm)) != M3_OK) return st;
    if (d.batch == 0) return M3_OK;
    RopeArgs a;
    a.B = B; a.C = C; a.theta = theta; a.dt = dt; a.angle0 = angle0; a.nrm = nrm;
    a.Bo = B_rot; a.Co = C_rot; a.angle_out = angle_final;
    a.Bt = d.batch; a.T = d.seqlen; a.H = d.nheads; a.R = R; a.N = d.dstate; a.G = G; a.K = K;
    return launch_unless_injected([&] { return launch_rope(a, dtype, (cudaStream_t)stream); });
}

m3_status m3_siso_chunked_fwd(const void *x, const float *dt, const float *A, const float *lam,
                              const float *theta, const void *B, const void *C, const float *D,
                              m3_dtype dtype, const m3_bcnorm *norm, const float *h0,
                              const float *prevBx0, const float *angle0, m3_dims d, void *y,
                              float *h_final, float *prevBx_final, float *angle_final, void *workspace,
                              size_t workspace_bytes, void *stream) {
    return chunked_common(x, dt, A, lam, theta, B, C, D, nullptr, nullptr, dtype, norm, h0, prevBx0,
                          angle0, d, y, h_final, prevBx_final, angle_final, workspace, workspace_bytes,
                          stream, false);
}

m3_status m3_mimo_chunked_fwd(const void *x, const float *dt, const float *A, const float *lam,
                              const float *theta, const void *B, const void *C, const float *D,
                              const float *W_x, const float *W_y, m3_dtype dtype, const m3_bcnorm *norm,
                              const float *h0, const float *prevBx0, const float *angle0, m3_dims d,
                              void *y, float *h_final, float *prevBx_final, float *angle_final,
                              void *workspace, size_t workspace_bytes, void *stream) {
    return chunked_common(x, dt, A, lam, theta, B, C, D, W_x, W_y, dtype, norm, h0, prevBx0, angle0, d, y,
                          h_final, prevBx_final, angle_final, workspace, workspace_bytes, stream, true);
}

m3_status m3_step_decode(const void *x_t, const float *dt_t, const float *A, const float *lam_t,
                         const float *theta_t, const void *B_t, const void *C_t, const float *D,
                         m3_dtype dtype, const m3_bcnorm *norm, m3_dims d, float *h, float *prevBx,
                         float *angle, void *y_t, void *stream) {
    m3_status st;
    if ((st = check_dtype(dtype)) != M3_OK) return st;
    if ((st = check_core_dims(d, false)) != M3_OK) return st;
    int64_t G, K;
    if ((st = resolve_groups(d, G, K)) != M3_OK) return st;
    M3_REQ(A); M3_REQ(D);
    if (d.batch > 0) {
        M3_REQ(x_t); M3_REQ(dt_t); M3_REQ(lam_t); M3_REQ(theta_t); M3_REQ(B_t); M3_REQ(C_t);
        M3_REQ(h); M3_REQ(prevBx); M3_REQ(angle); M3_REQ(y_t);
    }
    NormArgs nrm;
    if ((st = read_norm(norm, nrm)) != M3_OK) return st;
    if (d.batch == 0) return M3_OK;
    DecodeArgs a;
    a.x = x_t; a.B = B_t; a.C = C_t; a.dt = dt_t; a.A = A; a.lam = lam_t; a.theta = theta_t; a.D = D;
    a.nrm = nrm; a.h = h; a.prevBx = prevBx; a.angle = angle; a.y = y_t;
    a.Bt = d.batch; a.H = d.nheads; a.P = d.headdim; a.N = d.dstate; a.G = G; a.K = K;
    return launch_unless_injected([&] { return launch_decode(a, dtype, (cudaStream_t)stream); });
}

namespace {
// Shared validation of the rank-R decode entry points.
m3_status decode_gen(const void *x_t, const float *dt_t, const float *A, const float *lam_t, const float *theta_t,
                     const void *B_t, const void *C_t, const float *D, const float *W_x, const float *W_y,
                     m3_dtype dtype, const m3_bcnorm *norm, m3_dims d, float *h, float *prevBx, float *b_prev,
                     float *x_prev, float *angle, void *y_t, void *stream, bool factored) {
    m3_status st;
    if ((st = check_dtype(dtype)) != M3_OK) return st;
    if ((st = check_core_dims(d, false)) != M3_OK) return st;
    int64_t G, K;
    if ((st = resolve_groups(d, G, K)) != M3_OK) return st;
    if (d.rank < 1) return M3_ERR_INVALID_ARG;
    if (d.rank > kMaxRank || d.headdim % 4) return M3_ERR_UNSUPPORTED;
    M3_REQ(A); M3_REQ(D);
    M3_OPT(W_x); M3_OPT(W_y);
    if (d.batch > 0) {
        M3_REQ(x_t); M3_REQ(dt_t); M3_REQ(lam_t); M3_REQ(theta_t); M3_REQ(B_t); M3_REQ(C_t);
        M3_REQ(h); M3_REQ(angle); M3_REQ(y_t);
        if (factored) { M3_REQ(b_prev); M3_REQ(x_prev); }
        else M3_REQ(prevBx);
    }
    NormArgs nrm;
    if ((st = read_norm(norm, nrm)) != M3_OK) return st;
    if (d.batch == 0) return M3_OK;
    DecodeArgs a;
    a.x = x_t; a.B = B_t; a.C = C_t; a.dt = dt_t; a.A = A; a.lam = lam_t; a.theta = theta_t; a.D = D;
    a.nrm = nrm; a.h = h; a.prevBx = prevBx; a.angle = angle; a.y = y_t;
    a.Bt = d.batch; a.H = d.nheads; a.P = d.headdim; a.N = d.dstate; a.G = G; a.K = K;
    a.Wx = W_x; a.Wy = W_y; a.bprev = b_prev; a.xprev = x_prev; a.R = d.rank;
    return launch_unless_injected([&] { return launch_decode_gen(a, dtype, factored, (cudaStream_t)stream); });
}
}  // namespace

m3_status m3_mimo_step_decode(const void *x_t, const float *dt_t, const float *A, const float *lam_t,
                              const float *theta_t, const void *B_t, const void *C_t, const float *D,
                              const float *W_x, const float *W_y, m3_dtype dtype, const m3_bcnorm *norm,
                              m3_dims d, float *h, float *prevBx, float *angle, void *y_t, void *stream) {
    return decode_gen(x_t, dt_t, A, lam_t, theta_t, B_t, C_t, D, W_x, W_y, dtype, norm, d, h, prevBx, nullptr,
                      nullptr, angle, y_t, stream, false);
}

m3_status m3_step_decode_factored(const void *x_t, const float *dt_t, const float *A, const float *lam_t,
                                  const float *theta_t, const void *B_t, const void *C_t, const float *D,
                                  const float *W_x, const float *W_y, m3_dtype dtype, const m3_bcnorm *norm,
                                  m3_dims d, float *h, float *b_prev, float *x_prev, float *angle, void *y_t,
                                  void *stream) {
    return decode_gen(x_t, dt_t, A, lam_t, theta_t, B_t, C_t, D, W_x, W_y, dtype, norm, d, h, nullptr, b_prev,
                      x_prev, angle, y_t, stream, true);
}

m3_status m3_chunked_bwd(const void *x, const float *dt, const float *A, const float *lam, const float *theta,
                         const void *B, const void *C, const float *D, const float *W_x, const float *W_y,
                         m3_dtype dtype, const m3_bcnorm *norm, const float *h0, const float *prevBx0,
                         const float *angle0, m3_dims d, const void *dy, const float *dh_final,
                         const float *dprevBx_final, const float *dangle_final, const m3_grads *grads,
                         void *workspace, size_t workspace_bytes, void *stream) {
    m3_status st;
    if ((st = check_dtype(dtype)) != M3_OK) return st;
    if ((st = check_core_dims(d, true)) != M3_OK) return st;
    if (d.chunk < 1 || d.rank < 0 || !grads) return M3_ERR_INVALID_ARG;
    int64_t G, K;
    if ((st = resolve_groups(d, G, K)) != M3_OK) return st;
    const bool mimo = d.rank > 1 || W_x || W_y;
    const int64_t R = d.rank > 1 ? d.rank : 1;
    if (R > kMaxRank) return M3_ERR_UNSUPPORTED;
    M3_REQ(A); M3_REQ(D);
    const bool have_tokens = d.batch > 0 && d.seqlen > 0;
    if (have_tokens) {
        M3_REQ(x); M3_REQ(dt); M3_REQ(lam); M3_REQ(theta); M3_REQ(B); M3_REQ(C); M3_REQ(dy);
    } else {
        M3_OPT(x); M3_OPT(dt); M3_OPT(lam); M3_OPT(theta); M3_OPT(B); M3_OPT(C); M3_OPT(dy);
    }
    M3_OPT(W_x); M3_OPT(W_y); M3_OPT(h0); M3_OPT(prevBx0); M3_OPT(angle0);
    M3_OPT(dh_final); M3_OPT(dprevBx_final); M3_OPT(dangle_final); M3_OPT(workspace);
    const m3_grads &g = *grads;
    M3_OPT(g.dx); M3_OPT(g.ddt); M3_OPT(g.dA); M3_OPT(g.dlam); M3_OPT(g.dtheta); M3_OPT(g.dB); M3_OPT(g.dC);
    M3_OPT(g.dD); M3_OPT(g.dW_x); M3_OPT(g.dW_y); M3_OPT(g.dnormw_B); M3_OPT(g.dnormw_C); M3_OPT(g.dbias_B);
    M3_OPT(g.dbias_C); M3_OPT(g.dh0); M3_OPT(g.dprevBx0); M3_OPT(g.dangle0);
    NormArgs nrm;
    if ((st = read_norm(norm, nrm)) != M3_OK) return st;
    BwdArgs a{};
    a.x = x; a.B = B; a.C = C; a.dy = dy;
    a.dt = dt; a.A = A; a.lam = lam; a.theta = theta; a.D = D; a.Wx = W_x; a.Wy = W_y;
    a.h0 = h0; a.prevBx0 = prevBx0; a.angle0 = angle0;
    a.dh = dh_final; a.du = dprevBx_final; a.da = dangle_final;
    a.nrm = nrm;
    a.dx = g.dx; a.ddt = g.ddt; a.dA = g.dA; a.dlam = g.dlam; a.dtheta = g.dtheta; a.dB = g.dB; a.dC = g.dC;
    a.dD = g.dD; a.dWx = g.dW_x; a.dWy = g.dW_y; a.dwB = g.dnormw_B; a.dwC = g.dnormw_C; a.dbB = g.dbias_B;
    a.dbC = g.dbias_C; a.dh0 = g.dh0; a.du0 = g.dprevBx0; a.da0 = g.dangle0;
    a.Bt = d.batch; a.T = d.seqlen; a.H = d.nheads; a.P = d.headdim; a.N = d.dstate; a.R = R; a.G = G; a.K = K;
    const int q = bwd_chunk(a.P, a.N, R, K, d.chunk);
    if (q < 1) return M3_ERR_UNSUPPORTED;
    const size_t need = m3_workspace_bytes(mimo ? M3_WS_BWD_MIMO : M3_WS_BWD_SISO, d, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return M3_ERR_WORKSPACE;
    a.Q = q;
    a.ws = static_cast<float *>(workspace);
    if (d.batch == 0) return M3_OK;
    return launch_unless_injected([&] { return launch_scan_bwd(a, dtype, (cudaStream_t)stream); });
}

// ---- linear attention ------------------------------------------------------
namespace {
struct LinGeo {
    int64_t G, ldq, ldk, ldv;
};
// Sizes and row strides of the linear-attention entry points.
m3_status check_linattn_dims(const m3_linattn_dims &d, bool need_seq, LinGeo &o) {
    if (d.batch < 0 || d.nheads < 1 || d.headdim < 1 || d.dstate < 1 || d.ngroups < 0) return M3_ERR_INVALID_ARG;
    if (need_seq && d.seqlen < 0) return M3_ERR_INVALID_ARG;
    if (d.ld_q < 0 || d.ld_k < 0 || d.ld_v < 0) return M3_ERR_INVALID_ARG;
    if (d.dstate > kMaxDstate || d.headdim > kMaxHeaddim || d.dstate * d.headdim > kMaxStateElems)
        return M3_ERR_UNSUPPORTED;
    if (d.batch > (int64_t)1 << 24 || d.nheads > 4096 || (need_seq && d.seqlen > (int64_t)1 << 30))
        return M3_ERR_UNSUPPORTED;
    if (d.batch * d.nheads > kMaxLanes) return M3_ERR_UNSUPPORTED;
    o.G = d.ngroups ? d.ngroups : d.nheads;
    if (d.nheads % o.G) return M3_ERR_INVALID_ARG;
    o.ldq = d.ld_q ? d.ld_q : o.G * d.dstate;
    o.ldk = d.ld_k ? d.ld_k : o.G * d.dstate;
    o.ldv = d.ld_v ? d.ld_v : d.nheads * d.headdim;
    if (o.ldq < o.G * d.dstate || o.ldk < o.G * d.dstate || o.ldv < d.nheads * d.headdim) return M3_ERR_INVALID_ARG;
    const int64_t T = need_seq ? d.seqlen : 1, wide = d.nheads * (d.headdim > d.dstate ? d.headdim : d.dstate);
    int64_t ld = o.ldq > o.ldk ? o.ldq : o.ldk;
    if (o.ldv > ld) ld = o.ldv;
    if (wide > ld) ld = wide;
    if (sat_product({d.batch, T, ld}) > kMaxElems) return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

// q, k, v: non-null, aligned to their elements (the tensor-core path asks for
// 16 bytes and is chosen only there)
inline bool elem_aligned(const void *p, m3_dtype t) { return ((uintptr_t)p & (t == M3_BF16 ? 1u : 3u)) == 0; }
#define M3_REQ_ELEM(p)                                                          \
    do {                                                                        \
        if (!(p) || !elem_aligned(p, dtype)) return M3_ERR_INVALID_ARG;         \
    } while (0)

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// The mixes of a call (linattn.cuh) and the plan of their launches.
struct LinPlan {
    MixArgs m[3];
    int n;
    bool tc;                   // all of them on the tensor cores (else none)
    size_t states[3], bytes;   // offsets of their segment states, and the end of these
};
void plan_mixes(LinPlan &p, m3_dtype dtype, bool aligned) {
    p.tc = aligned;
    for (int i = 0; i < p.n; i++) p.tc = p.tc && mix_tc_sizes(p.m[i], dtype);
    if (p.tc) mix_tc_plan(p.m, p.n);
    else mix_simt_plan(p.m, p.n);
    p.bytes = 0;
    for (int i = 0; i < p.n; i++) {
        MixArgs &m = p.m[i];
        p.states[i] = p.bytes;
        p.bytes += align256((size_t)(m.Bt * m.H) * (size_t)(m.nseg - 1) * m.dar * m.dcr * sizeof(float));
    }
}
cudaError_t launch_mixes(LinPlan &p, m3_dtype dtype, void *workspace, cudaStream_t s) {
    for (int i = 0; i < p.n; i++)
        p.m[i].ws = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.states[i]);
    if (p.tc) return launch_mix_tc(p.m, p.n, s);
    return launch_mix_simt(p.m, p.n, dtype, s);
}

// bf16 rows that TMA cannot address, for their width or their stride, are
// copied into padded ones first (in the workspace): the tensor cores still pay,
// 8 x 2048 tokens of 16 heads of 120 x 60 take 103 us, 44 of them the copies, and
// took 1.1 ms in fp32 arithmetic.
struct LinPads {
    bool on;
    int64_t dk, dv;            // padded widths
    size_t q, k, v, dy, bytes; // offsets from the first of them, and their end
};
LinPads pads_of(const m3_linattn_dims &d, const LinGeo &o, m3_dtype dtype) {
    LinPads p{};
    p.dk = d.dstate;
    p.dv = d.headdim;
    if (dtype != M3_BF16 || d.dstate > 128 || d.headdim > 128 || d.seqlen < 1) return p;
    if (d.seqlen <= 16 && d.batch * d.nheads <= 256) return p;
    // what the tensor-core path takes (mix_tc_sizes), with room for the padding
    if (d.batch * d.nheads > (int64_t)1 << 28 || sat_product({d.seqlen, d.nheads, 128}) > (int64_t)1 << 37) return p;
    p.on = d.dstate % 8 || d.headdim % 8 || o.ldq % 8 || o.ldk % 8 || o.ldv % 8;
    if (!p.on) return p;
    p.dk = (d.dstate + 7) / 8 * 8;
    p.dv = (d.headdim + 7) / 8 * 8;
    const size_t rows = (size_t)(d.batch * d.seqlen);
    p.k = align256(rows * o.G * p.dk * 2);
    p.v = 2 * p.k;
    p.dy = p.v + align256(rows * d.nheads * p.dv * 2);
    p.bytes = p.dy + align256(rows * d.nheads * p.dv * 2);
    return p;
}

// One mix of the problem, without its pointers.
MixArgs mix_of(const m3_linattn_dims &d, int64_t da, int64_t dc, int64_t dar, int64_t dcr, m3_dtype dtype) {
    MixArgs m{};
    m.Bt = d.batch; m.H = d.nheads; m.T = d.seqlen;
    m.da = (int)da; m.dc = (int)dc;
    m.dar = (int)dar; m.dcr = (int)dcr;
    m.ra = m.rb = m.rc = 1;
    m.y_f32 = dtype == M3_F32;
    return m;
}
LinPlan fwd_mix(const m3_linattn_dims &d, const LinGeo &o, const LinPads &pd, m3_dtype dtype) {
    LinPlan p;
    p.n = 1;
    MixArgs &m = p.m[0] = mix_of(d, pd.dk, pd.dv, d.dstate, d.headdim, dtype);
    m.lda = pd.on ? o.G * pd.dk : o.ldq;
    m.ldb = pd.on ? o.G * pd.dk : o.ldk;
    m.ldc = pd.on ? d.nheads * pd.dv : o.ldv;
    m.ra = m.rb = (int)(d.nheads / o.G);
    return p;
}
// dq = mix(dy, v, k) forwards, dk = mix(v, dy, q) and dv = mix(k, q, dy)
// backwards.
LinPlan bwd_mixes(const m3_linattn_dims &d, const LinGeo &o, const LinPads &pd, m3_dtype dtype) {
    LinPlan p;
    p.n = 3;
    const int rep = (int)(d.nheads / o.G);
    const int64_t ldd = d.nheads * pd.dv, ldq = pd.on ? o.G * pd.dk : o.ldq, ldk = pd.on ? o.G * pd.dk : o.ldk;
    const int64_t ldv = pd.on ? ldd : o.ldv;
    MixArgs &dq = p.m[0] = mix_of(d, pd.dv, pd.dk, d.headdim, d.dstate, dtype);
    dq.lda = ldd; dq.ldb = ldv; dq.ldc = ldk; dq.rc = rep;
    MixArgs &dk = p.m[1] = dq;
    dk.lda = ldv; dk.ldb = ldd; dk.ldc = ldq;
    dk.reverse = 1;
    for (MixArgs *m : {&dq, &dk}) {
        m->m_trans = 1;
        if (rep > 1) m->y_f32 = 1;
    }
    MixArgs &dv = p.m[2] = mix_of(d, pd.dk, pd.dv, d.dstate, d.headdim, dtype);
    dv.lda = ldk; dv.ldb = ldq; dv.ldc = ldd;
    dv.ra = dv.rb = rep;
    dv.reverse = 1;
    return p;
}
// The copies of q, k, v (and dy), and the mixes' pointers turned to them.
PadArgs pad_rows(const m3_linattn_dims &d, const LinGeo &o, const LinPads &pd, char *at, const void *&q, const void *&k,
                 const void *&v, const void **dy) {
    PadArgs a{};
    auto add = [&](const void *&src, size_t off, int64_t ld, int64_t heads, int64_t w, int64_t wp) {
        const int i = a.count++;
        a.src[i] = src;
        a.dst[i] = at + off;
        a.ld[i] = ld;
        a.n[i] = d.batch * d.seqlen * heads * (wp / 8);
        a.heads[i] = (int)heads;
        a.d[i] = (int)w;
        src = at + off;
    };
    add(q, pd.q, o.ldq, o.G, d.dstate, pd.dk);
    add(k, pd.k, o.ldk, o.G, d.dstate, pd.dk);
    add(v, pd.v, o.ldv, d.nheads, d.headdim, pd.dv);
    if (dy) add(*dy, pd.dy, d.nheads * d.headdim, d.nheads, d.headdim, pd.dv);
    return a;
}
// bytes of one gradient of shared heads, per head in fp32, in padded rows
size_t head_bytes(const m3_linattn_dims &d, const LinGeo &o, const LinPads &pd) {
    return o.G == d.nheads ? 0 : align256((size_t)d.batch * d.seqlen * d.nheads * pd.dk * sizeof(float));
}
inline bool tma_aligned(const void *q, const void *k, const void *v) { return aligned16(q) && aligned16(k) && aligned16(v); }
}  // namespace

// Enough for either path (the choice depends on the bases' alignment).  The
// backward's plan is that of all three products, whichever are wanted.
size_t m3_linattn_workspace_bytes(int which, m3_linattn_dims d, m3_dtype dtype) {
    LinGeo o;
    if (check_dtype(dtype) != M3_OK || check_linattn_dims(d, true, o) != M3_OK) return 0;
    if (which != M3_WS_LINATTN_FWD && which != M3_WS_LINATTN_BWD) return 0;
    const bool bwd = which == M3_WS_LINATTN_BWD;
    const LinPads pd = pads_of(d, o, dtype);
    size_t most = 0;
    for (bool aligned : {false, true}) {
        if (pd.on && !aligned) continue;
        LinPlan p = bwd ? bwd_mixes(d, o, pd, dtype) : fwd_mix(d, o, pd, dtype);
        plan_mixes(p, dtype, aligned);
        if (p.bytes > most) most = p.bytes;
    }
    return most + (bwd ? 2 * head_bytes(d, o, pd) + pd.bytes : pd.on ? pd.dy : 0);
}

m3_status m3_linattn_chunked_fwd(const void *q, const void *k, const void *v, m3_dtype dtype, const float *log_decay,
                                 float scale, const float *s0, const int32_t *lengths, m3_linattn_dims d, void *y,
                                 float *s_final, void *workspace, size_t workspace_bytes, void *stream) {
    m3_status st;
    LinGeo o;
    if ((st = check_dtype(dtype)) != M3_OK) return st;
    if ((st = check_linattn_dims(d, true, o)) != M3_OK) return st;
    if (!std::isfinite(scale)) return M3_ERR_INVALID_ARG;
    M3_REQ(log_decay);
    if (d.batch > 0 && d.seqlen > 0) {
        M3_REQ_ELEM(q); M3_REQ_ELEM(k); M3_REQ_ELEM(v); M3_REQ(y);
    }
    M3_OPT(s0); M3_OPT(lengths); M3_OPT(s_final); M3_OPT(workspace);
    const size_t need = m3_linattn_workspace_bytes(M3_WS_LINATTN_FWD, d, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return M3_ERR_WORKSPACE;
    if (d.batch == 0) return M3_OK;
    const LinPads pd = pads_of(d, o, dtype);
    LinPlan p = fwd_mix(d, o, pd, dtype);
    plan_mixes(p, dtype, pd.on || tma_aligned(q, k, v));
    PadArgs pads{};
    if (pd.on && !p.tc) return M3_ERR_UNSUPPORTED;          // does not happen: pads_of has seen to it
    if (pd.on) pads = pad_rows(d, o, pd, static_cast<char *>(workspace) + p.bytes, q, k, v, nullptr);
    MixArgs &m = p.m[0];
    m.a = q; m.b = k; m.c = v;
    m.log_decay = log_decay; m.lengths = lengths;
    m.m0 = s0; m.m_out = s_final;
    m.y = y;
    m.scale_p = m.scale_i = scale;
    m.scale_w = 1.f;
    return launch_unless_injected([&]() -> cudaError_t {
        const cudaError_t e = launch_pad_rows(pads, (cudaStream_t)stream);
        return e != cudaSuccess ? e : launch_mixes(p, dtype, workspace, (cudaStream_t)stream);
    });
}

m3_status m3_linattn_step_decode(const void *q_t, const void *k_t, const void *v_t, m3_dtype dtype,
                                 const float *log_decay, float scale, m3_linattn_dims d, float *s, void *y_t,
                                 void *stream) {
    m3_status st;
    LinGeo o;
    if ((st = check_dtype(dtype)) != M3_OK) return st;
    if ((st = check_linattn_dims(d, false, o)) != M3_OK) return st;
    if (!std::isfinite(scale)) return M3_ERR_INVALID_ARG;
    M3_REQ(log_decay);
    if (d.batch == 0) return M3_OK;
    M3_REQ_ELEM(q_t); M3_REQ_ELEM(k_t); M3_REQ_ELEM(v_t); M3_REQ(s); M3_REQ(y_t);
    LinStepArgs a;
    a.q = q_t; a.k = k_t; a.v = v_t;
    a.ldq = o.ldq; a.ldk = o.ldk; a.ldv = o.ldv;
    a.log_decay = log_decay; a.s = s; a.y = y_t;
    a.Bt = d.batch; a.H = d.nheads; a.G = o.G; a.dk = d.dstate; a.dv = d.headdim;
    a.scale = scale;
    return launch_unless_injected([&] { return launch_linattn_step(a, dtype, (cudaStream_t)stream); });
}

m3_status m3_linattn_chunked_bwd(const void *q, const void *k, const void *v, m3_dtype dtype, const float *log_decay,
                                 float scale, const float *s0, const int32_t *lengths, m3_linattn_dims d,
                                 const void *dy, const float *ds_final, const m3_linattn_grads *grads, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    m3_status st;
    LinGeo o;
    if ((st = check_dtype(dtype)) != M3_OK) return st;
    if ((st = check_linattn_dims(d, true, o)) != M3_OK) return st;
    if (!std::isfinite(scale) || !grads) return M3_ERR_INVALID_ARG;
    M3_REQ(log_decay);
    if (d.batch > 0 && d.seqlen > 0) {
        M3_REQ_ELEM(q); M3_REQ_ELEM(k); M3_REQ_ELEM(v); M3_REQ(dy);
    }
    const m3_linattn_grads &g = *grads;
    M3_OPT(s0); M3_OPT(lengths); M3_OPT(ds_final); M3_OPT(workspace);
    M3_OPT(g.dq); M3_OPT(g.dk); M3_OPT(g.dv); M3_OPT(g.ds0);
    const size_t need = m3_linattn_workspace_bytes(M3_WS_LINATTN_BWD, d, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return M3_ERR_WORKSPACE;
    const bool want[3] = {g.dq != nullptr, g.dk != nullptr, g.dv || g.ds0};
    if (d.batch == 0 || !(want[0] || want[1] || want[2])) return M3_OK;
    const LinPads pd = pads_of(d, o, dtype);
    LinPlan p = bwd_mixes(d, o, pd, dtype);
    plan_mixes(p, dtype, pd.on || tma_aligned(q, k, v));
    const size_t hb = head_bytes(d, o, pd);
    const bool shared = hb > 0;
    char *heads = static_cast<char *>(workspace) + p.bytes;
    PadArgs pads{};
    if (pd.on && !p.tc) return M3_ERR_UNSUPPORTED;          // does not happen: pads_of has seen to it
    if (pd.on) pads = pad_rows(d, o, pd, heads + 2 * hb, q, k, v, &dy);
    const float *sum_in[2] = {};
    void *sum_out[2] = {};
    int ns = 0;
    auto fill = [&](int i, const void *a, const void *b, const void *c, const float *m0, void *y) -> MixArgs & {
        MixArgs &m = p.m[i];
        m.a = a; m.b = b; m.c = c;
        m.m0 = m0;
        m.y = y;
        m.log_decay = log_decay; m.lengths = lengths;
        m.scale_p = scale;
        // the forward walk scales its answers, the walks from the end their state
        m.scale_i = m.reverse ? 1.f : scale;
        m.scale_w = m.reverse ? scale : 1.f;
        return m;
    };
    auto summed = [&](void *out) -> void * {
        if (!shared) return out;
        float *in = reinterpret_cast<float *>(heads + ns * hb);
        sum_in[ns] = in;
        sum_out[ns++] = out;
        return in;
    };
    if (want[0]) fill(0, dy, v, k, s0, summed(g.dq));
    if (want[1]) fill(1, v, dy, q, ds_final, summed(g.dk));
    if (want[2]) fill(2, k, q, dy, ds_final, g.dv).m_out = g.ds0;
    p.n = 0;                                    // those that are wanted, with their places in the workspace
    for (int i = 0; i < 3; i++)
        if (want[i]) {
            p.m[p.n] = p.m[i];
            p.states[p.n++] = p.states[i];
        }
    const cudaStream_t s = (cudaStream_t)stream;
    return launch_unless_injected([&]() -> cudaError_t {
        cudaError_t e = launch_pad_rows(pads, s);
        if (e == cudaSuccess) e = launch_mixes(p, dtype, workspace, s);
        if (e == cudaSuccess && ns > 0)
            e = launch_head_sum(sum_in, sum_out, ns, dtype, d.batch * d.seqlen, d.nheads, o.G, d.dstate, pd.dk, s);
        return e;
    });
}

// ---- group norm --------------------------------------------------------------
namespace {
m3_status check_norm(m3_dtype dtype, m3_act act, const m3_norm_dims &d) {
    m3_status st;
    if ((st = check_dtype(dtype)) != M3_OK) return st;
    if (act < M3_ACT_NONE || act > M3_ACT_RELU) return M3_ERR_INVALID_ARG;
    if (d.batch < 0 || d.seqlen < 0 || d.channels < 1 || d.ngroups < 1 || d.channels % d.ngroups)
        return M3_ERR_INVALID_ARG;
    if (d.channels > 16384 || d.batch > (int64_t)1 << 24 || d.seqlen > (int64_t)1 << 30) return M3_ERR_UNSUPPORTED;
    if (d.batch * d.ngroups > kMaxLanes) return M3_ERR_UNSUPPORTED;
    if (sat_product({d.batch, d.seqlen, d.channels}) > kMaxElems) return M3_ERR_UNSUPPORTED;
    return M3_OK;
}
}  // namespace

size_t m3_group_norm_workspace_bytes(int which, m3_norm_dims d, m3_dtype dtype) {
    if (check_norm(dtype, M3_ACT_NONE, d) != M3_OK || d.batch == 0 || d.seqlen == 0) return 0;
    if (which == M3_WS_NORM_FWD)
        return gn_fwd_workspace_floats(d.batch, d.seqlen, d.channels, d.ngroups, dtype) * sizeof(float);
    if (which == M3_WS_NORM_BWD)
        return gn_bwd_workspace_floats(d.batch, d.seqlen, d.channels, d.ngroups, dtype) * sizeof(float);
    return 0;
}

m3_status m3_group_norm_fwd(const void *x, m3_dtype dtype, const float *weight, const float *bias, const void *gate,
                            m3_act act, float eps, m3_norm_dims d, void *y, float *mean, float *rstd, void *workspace,
                            size_t workspace_bytes, void *stream) {
    m3_status st;
    if ((st = check_norm(dtype, act, d)) != M3_OK) return st;
    if (!(eps >= 0.f && std::isfinite(eps))) return M3_ERR_INVALID_ARG;
    M3_OPT(weight); M3_OPT(bias); M3_OPT(gate); M3_OPT(mean); M3_OPT(rstd); M3_OPT(workspace);
    const size_t need = m3_group_norm_workspace_bytes(M3_WS_NORM_FWD, d, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return M3_ERR_WORKSPACE;
    if (d.batch == 0 || d.seqlen == 0) return M3_OK;
    M3_REQ(x); M3_REQ(y);
    GnArgs a{};
    a.x = x; a.gate = gate; a.w = weight; a.b = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    a.Bt = d.batch; a.L = d.seqlen; a.C = d.channels; a.G = d.ngroups;
    a.act = act; a.eps = eps;
    a.ws = static_cast<float *>(workspace);
    return launch_unless_injected([&] { return launch_gn_fwd(a, dtype, (cudaStream_t)stream); });
}

m3_status m3_group_norm_bwd(const void *x, const void *dy, m3_dtype dtype, const float *weight, const float *bias,
                            const void *gate, m3_act act, const float *mean, const float *rstd, m3_norm_dims d,
                            void *dx, float *dweight, float *dbias, void *dgate, void *workspace,
                            size_t workspace_bytes, void *stream) {
    m3_status st;
    if ((st = check_norm(dtype, act, d)) != M3_OK) return st;
    if (dgate && !gate) return M3_ERR_INVALID_ARG;
    M3_OPT(weight); M3_OPT(bias); M3_OPT(gate); M3_OPT(dx); M3_OPT(dweight); M3_OPT(dbias); M3_OPT(dgate);
    M3_OPT(workspace);
    const size_t need = m3_group_norm_workspace_bytes(M3_WS_NORM_BWD, d, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return M3_ERR_WORKSPACE;
    if (d.batch > 0 && d.seqlen > 0) {
        M3_REQ(x); M3_REQ(dy); M3_REQ(mean); M3_REQ(rstd);
    }
    GnArgs a{};
    a.x = x; a.dy = dy; a.gate = gate; a.w = weight; a.b = bias;
    a.mean_in = mean; a.rstd_in = rstd;
    a.dx = dx; a.dw = dweight; a.db = dbias; a.dgate = dgate;
    a.Bt = d.batch; a.L = d.seqlen; a.C = d.channels; a.G = d.ngroups;
    a.act = act;
    a.ws = static_cast<float *>(workspace);
    return launch_unless_injected([&] { return launch_gn_bwd(a, dtype, (cudaStream_t)stream); });
}

}  // extern "C"
