// block_norm_api.cu -- the C entry points of the block norms.
#include "block_norm.cuh"

namespace ssd {
namespace {

ssd_status make_norm(const ssd_norm_dims* d, NormParams* p) {
    if (!d) return SSD_ERR_NULL;
    if ((d->dtype != SSD_F32 && d->dtype != SSD_BF16) || (d->rdtype != SSD_F32 && d->rdtype != SSD_BF16))
        return SSD_ERR_DTYPE;
    if (d->dtype == SSD_F32 && d->rdtype != SSD_F32) return SSD_ERR_DTYPE;
    if (d->reserved != 0 || d->tokens < 0 || d->tokens > (1LL << 31) - 1) return SSD_ERR_SHAPE;
    if (d->gate != SSD_GATE_NONE && d->gate != SSD_GATE_SILU && d->gate != SSD_GATE_SIGMOID)
        return SSD_ERR_SHAPE;
    if (d->width < 8 || d->width > 16384 || d->ngroups < 1 || d->width % d->ngroups != 0 ||
        (d->width / d->ngroups) % 8 != 0)
        return SSD_ERR_SHAPE;
    if (!(d->eps >= 0.f) || !(d->eps < 1e30f)) return SSD_ERR_SHAPE;
    const int64_t grain = d->dtype == SSD_BF16 ? 8 : 4;
    NormParams q = {};
    q.T = d->tokens; q.D = (int)d->width; q.vecs = q.D / 8; q.ngroups = (int)d->ngroups;
    q.gvecs = q.vecs / q.ngroups;
    q.ys = d->y_stride ? d->y_stride : q.D;
    q.zs = d->z_stride ? d->z_stride : q.D;
    if (q.ys < q.D || q.zs < q.D || q.ys % grain || q.zs % grain || q.ys > (1LL << 31) || q.zs > (1LL << 31))
        return SSD_ERR_SHAPE;
    const bool shuffled = q.gvecs <= 32 && (q.gvecs & (q.gvecs - 1)) == 0;
    q.grp_floats = q.ngroups == 1 || shuffled ? 0 : q.vecs + q.ngroups;
    q.gate = d->gate;
    q.eps = d->eps;
    *p = q;
    return SSD_OK;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_block_norm_fwd(const ssd_norm_dims* d, const void* r, const void* y, const void* z,
                              const float* w_post, const float* alpha, const float* w_pre,
                              void* r_out, void* n, float* rstd_post, float* rstd_pre, void* stream) {
    NormParams p;
    ssd_status s = make_norm(d, &p);
    if (s != SSD_OK) return s;
    if (p.T == 0) return SSD_OK;
    if (!r || !y || !w_pre || !r_out || !n || (p.gate != SSD_GATE_NONE && !z)) return SSD_ERR_NULL;
    if (!aligned16(r) || !aligned16(y) || !aligned16(z) || !aligned16(w_post) || !aligned16(alpha) ||
        !aligned16(w_pre) || !aligned16(r_out) || !aligned16(n) || !aligned16(rstd_post) ||
        !aligned16(rstd_pre))
        return SSD_ERR_ALIGN;
    const int e = d->dtype == SSD_BF16 ? 2 : 4, er = d->rdtype == SSD_BF16 ? 2 : 4;
    const size_t nb = (size_t)(p.T * p.D), wb = (size_t)p.D * 4;
    const Range in[] = {rng(r, nb * er), rng(y, span(p.T, p.ys, p.D, e)),
                        rng(p.gate != SSD_GATE_NONE ? z : nullptr, span(p.T, p.zs, p.D, e)),
                        rng(w_post, wb), rng(alpha, wb), rng(w_pre, wb)};
    const Range out[] = {rng(r_out, nb * er), rng(n, nb * e),
                         rng(rstd_post, (size_t)(p.T * p.ngroups) * 4), rng(rstd_pre, (size_t)p.T * 4)};
    for (int i = 0; i < 6; ++i)
        for (int j = 0; j < 4; ++j)
            if (overlap(in[i], out[j]) && !(i == 0 && j == 0 && r == r_out)) return SSD_ERR_ALIAS;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SSD_ERR_ALIAS;
    if ((s = pre_launch()) != SSD_OK) return s;
    p.r = r; p.y = y; p.z = z; p.w_post = w_post; p.alpha = alpha; p.w_pre = w_pre;
    p.r_out = r_out; p.n = n; p.rstd_post = rstd_post; p.rstd_pre = rstd_pre;
    return from_cuda(launch_block_norm_fwd(p, d->dtype, d->rdtype, (cudaStream_t)stream));
}

size_t ssd_block_norm_bwd_workspace_bytes(const ssd_norm_dims* d) {
    NormParams p;
    if (make_norm(d, &p) != SSD_OK || p.T == 0) return 0;
    return (size_t)block_norm_parts(p.T, p.vecs, d->dtype, sm_count()) * 2 * p.D * 4;
}

ssd_status ssd_block_norm_bwd(const ssd_norm_dims* d, const void* r, const void* y, const void* z,
                              const float* w_post, const float* alpha, const float* w_pre,
                              const void* dr_out, const void* dn, const float* rstd_post,
                              const float* rstd_pre, void* dr, void* dy, void* dz, float* dw_post,
                              float* dalpha, float* dw_pre, void* workspace, size_t workspace_bytes,
                              void* stream) {
    NormParams p;
    ssd_status s = make_norm(d, &p);
    if (s != SSD_OK) return s;
    const bool gated = p.gate != SSD_GATE_NONE;
    if (!w_pre || !dw_pre) return SSD_ERR_NULL;
    const size_t need = ssd_block_norm_bwd_workspace_bytes(d);
    if (p.T > 0 && (!r || !y || !dr_out || !dn || !rstd_post || !rstd_pre || !dr || !dy ||
                    (gated && (!z || !dz)) || !workspace))
        return SSD_ERR_NULL;
    if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    const void* all[] = {r, y, z, w_post, alpha, w_pre, dr_out, dn, rstd_post, rstd_pre, dr, dy, dz,
                         dw_post, dalpha, dw_pre, workspace};
    for (const void* a : all)
        if (!aligned16(a)) return SSD_ERR_ALIGN;
    const int e = d->dtype == SSD_BF16 ? 2 : 4, er = d->rdtype == SSD_BF16 ? 2 : 4;
    const size_t nb = (size_t)(p.T * p.D), wb = (size_t)p.D * 4;
    const Range in[] = {rng(r, nb * er), rng(y, span(p.T, p.ys, p.D, e)),
                        rng(gated ? z : nullptr, span(p.T, p.zs, p.D, e)), rng(w_post, wb), rng(alpha, wb),
                        rng(w_pre, wb), rng(dr_out, nb * er), rng(dn, nb * e),
                        rng(rstd_post, (size_t)(p.T * p.ngroups) * 4), rng(rstd_pre, (size_t)p.T * 4)};
    const Range out[] = {rng(dr, nb * er), rng(dy, nb * e), rng(gated ? dz : nullptr, nb * e),
                         rng(dw_post, wb), rng(dalpha, wb), rng(dw_pre, wb), rng(workspace, need)};
    for (const Range& a : in)
        for (const Range& b : out)
            if (overlap(a, b)) return SSD_ERR_ALIAS;
    for (int i = 0; i < 7; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SSD_ERR_ALIAS;
    if ((s = pre_launch()) != SSD_OK) return s;
    p.r = r; p.y = y; p.z = z; p.w_post = w_post; p.alpha = alpha; p.w_pre = w_pre;
    p.dr_out = dr_out; p.dn = dn; p.rstd_post = const_cast<float*>(rstd_post);
    p.rstd_pre = const_cast<float*>(rstd_pre); p.dr = dr; p.dy = dy; p.dz = dz;
    p.dw_post = dw_post; p.dalpha = dalpha; p.dw_pre = dw_pre; p.partial = (float*)workspace;
    return from_cuda(launch_block_norm_bwd(p, d->dtype, d->rdtype, sm_count(), (cudaStream_t)stream));
}

}  // extern "C"
