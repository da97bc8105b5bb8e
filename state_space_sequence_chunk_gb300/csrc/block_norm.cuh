// block_norm.cuh -- shared declarations of the block-norm kernels (not part of the ABI).
#pragma once

#include "ssd_internal.cuh"

namespace ssd {

struct NormParams {
    int64_t T, ys, zs;             // rows; elements from one row of y (z) to the next
    int D, vecs, ngroups, gvecs;   // columns; vectors of eight in a row and in a group
    int grp_floats;                // shared floats for group_sum's general form (0: not used)
    int gate;
    float eps;
    const void *r, *y, *z, *dr_out, *dn;
    const float *w_post, *alpha, *w_pre;
    void *r_out, *n, *dr, *dy, *dz;
    float *rstd_post, *rstd_pre;   // outputs forwards, inputs backwards
    float *partial, *dw_post, *dalpha, *dw_pre;
};

// CTAs of the gradient's kernel, and partial column sums that it leaves.
int block_norm_grid(int64_t T, int vecs, int dtype, int sms);
int block_norm_parts(int64_t T, int vecs, int dtype, int sms);
cudaError_t launch_block_norm_fwd(NormParams& p, int dtype, int rdtype, cudaStream_t stream);
cudaError_t launch_block_norm_bwd(NormParams& p, int dtype, int rdtype, int sms, cudaStream_t stream);

}  // namespace ssd
