// group_norm.cuh -- shared declarations of the group-norm kernels (not part
// of the ABI).
#pragma once
#include "m3_internal.cuh"

namespace m3 {

// x, y, gate, dx, dy, dgate: (Bt, L, C), channels last; group = C / G
// consecutive channels; statistics over the L tokens and the group's channels
// of each sequence.
struct GnArgs {
    const void *x, *gate, *dy;
    const float *w, *b;          // (C), NULL for ones / zeros
    const float *mean_in, *rstd_in;
    void *y, *dx, *dgate;
    float *mean, *rstd, *dw, *db;
    int64_t Bt, L, C, G;
    int act;
    float eps;
    float *ws;
};

size_t gn_fwd_workspace_floats(int64_t Bt, int64_t L, int64_t C, int64_t G, m3_dtype dt);
size_t gn_bwd_workspace_floats(int64_t Bt, int64_t L, int64_t C, int64_t G, m3_dtype dt);
cudaError_t launch_gn_fwd(const GnArgs &a, m3_dtype dt, cudaStream_t s);
cudaError_t launch_gn_bwd(const GnArgs &a, m3_dtype dt, cudaStream_t s);

}  // namespace m3
