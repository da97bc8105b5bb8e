// short_conv_api.cu -- the C entry points of the short convolution over packed rows.
#include "short_conv.cuh"

namespace ssd {
namespace {

struct Dims {
    ShortConv p;
    int64_t n, T, D, W;
    int es;
    size_t rows, states;     // bytes of [tokens, dim] and of [nseqs, width - 1, dim]
};

ssd_status make(const ssd_short_conv_dims* d, bool packed, Dims* out) {
    if (!d) return SSD_ERR_NULL;
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d->reserved != 0 || d->nseqs < 0 || d->nseqs > (1 << 20) || d->tokens < 0 || d->tokens > (1LL << 30))
        return SSD_ERR_SHAPE;
    if (d->dim < 8 || d->dim > 65536 || d->dim % 8 != 0 || d->width < 2 || d->width > 8) return SSD_ERR_SHAPE;
    if (d->activation != SSD_ACT_NONE && d->activation != SSD_ACT_SILU) return SSD_ERR_SHAPE;
    Dims q = {};
    q.n = d->nseqs; q.T = d->tokens; q.D = d->dim; q.W = d->width;
    q.es = d->dtype == SSD_BF16 ? 2 : 4;
    ShortConv& p = q.p;
    p.xs = d->x_stride ? d->x_stride : q.D;
    if (p.xs < q.D || p.xs % (16 / q.es) || p.xs > (1LL << 31)) return SSD_ERR_SHAPE;
    if (!packed && (q.n > 0 ? q.T % q.n != 0 : q.T > 0)) return SSD_ERR_SHAPE;
    p.nseq = (int)q.n; p.T = (int)q.T; p.D = (int)q.D;
    p.L = packed || q.n == 0 ? 0 : (int)(q.T / q.n);
    p.act = d->activation;
    q.rows = (size_t)(q.T * q.D) * q.es;
    q.states = (size_t)(q.n * (q.W - 1) * q.D) * q.es;
    // a warp for each tile of tokens or sequence and 32 vectors of two channels: their number is an int
    if ((q.T / 8 + 1 + q.n) * ((q.D / 2 + 31) / 32) >= (1LL << 31) - 4) return SSD_ERR_SHAPE;
    *out = q;
    return SSD_OK;
}

size_t part_bytes(const Dims& q, int dtype) {
    if (q.T == 0) return 0;
    const int tile = short_conv_tile(q.T, (int)q.D, (int)q.W, dtype, true, sm_count());
    return (size_t)((q.T + tile - 1) / tile * (q.W + 1) * q.D) * 4;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_short_conv_fwd(const ssd_short_conv_dims* d, const void* x, const float* weight,
                              const float* bias, const int32_t* cu_seqlens, const void* init_state,
                              void* out, void* final_state, void* stream) {
    Dims q;
    ssd_status s = make(d, cu_seqlens != nullptr, &q);
    if (s != SSD_OK) return s;
    if (q.T == 0 && q.n == 0) return SSD_OK;
    if (!weight || (q.T > 0 && (!x || !out))) return SSD_ERR_NULL;
    for (const void* a : {x, (const void*)weight, (const void*)bias, (const void*)cu_seqlens, init_state,
                          (const void*)out, (const void*)final_state})
        if (!aligned16(a)) return SSD_ERR_ALIGN;
    ShortConv& p = q.p;
    const Range in[] = {rng(x, span(q.T, p.xs, q.D, q.es)), rng(weight, (size_t)(q.D * q.W) * 4),
                        rng(bias, (size_t)q.D * 4), rng(cu_seqlens, (size_t)(q.n + 1) * 4),
                        rng(init_state, q.states)};
    const Range o = rng(out, q.rows), f = rng(final_state, q.states);
    for (const Range& a : in)
        if (overlap(a, o) || overlap(a, f)) return SSD_ERR_ALIAS;
    if (overlap(o, f)) return SSD_ERR_ALIAS;
    if ((s = pre_launch()) != SSD_OK) return s;
    p.cu = cu_seqlens; p.x = x; p.w = weight; p.bias = bias; p.init = init_state;
    p.out = out; p.fin = final_state;
    return from_cuda(launch_short_conv_fwd(p, (int)q.W, d->dtype, sm_count(), (cudaStream_t)stream));
}

size_t ssd_short_conv_bwd_workspace_bytes(const ssd_short_conv_dims* d) {
    Dims q;
    return make(d, true, &q) == SSD_OK ? part_bytes(q, d->dtype) : 0;
}

ssd_status ssd_short_conv_bwd(const ssd_short_conv_dims* d, const void* x, const float* weight,
                              const float* bias, const int32_t* cu_seqlens, const void* init_state,
                              const void* dout, const void* dfinal_state, void* dx, float* dweight,
                              float* dbias, void* dinit_state, void* workspace,
                              size_t workspace_bytes, void* stream) {
    Dims q;
    ssd_status s = make(d, cu_seqlens != nullptr, &q);
    if (s != SSD_OK) return s;
    const size_t need = part_bytes(q, d->dtype);
    if (!weight || !dweight || (q.T > 0 && (!x || !dout || !dx || !workspace))) return SSD_ERR_NULL;
    if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    for (const void* a : {x, (const void*)weight, (const void*)bias, (const void*)cu_seqlens, init_state, dout,
                          dfinal_state, (const void*)dx, (const void*)dweight, (const void*)dbias,
                          (const void*)dinit_state, (const void*)workspace})
        if (!aligned16(a)) return SSD_ERR_ALIGN;
    ShortConv& p = q.p;
    const Range in[] = {rng(x, span(q.T, p.xs, q.D, q.es)), rng(weight, (size_t)(q.D * q.W) * 4),
                        rng(bias, (size_t)q.D * 4), rng(cu_seqlens, (size_t)(q.n + 1) * 4),
                        rng(init_state, q.states), rng(dout, q.rows), rng(dfinal_state, q.states)};
    const Range out[] = {rng(dx, q.rows), rng(dweight, (size_t)(q.D * q.W) * 4), rng(dbias, (size_t)q.D * 4),
                         rng(dinit_state, q.states), rng(workspace, need)};
    for (const Range& a : in)
        for (const Range& b : out)
            if (overlap(a, b)) return SSD_ERR_ALIAS;
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SSD_ERR_ALIAS;
    if ((s = pre_launch()) != SSD_OK) return s;
    p.cu = cu_seqlens; p.x = x; p.w = weight; p.bias = bias; p.init = init_state; p.dout = dout;
    p.dfin = dfinal_state; p.dx = dx; p.dw = dweight; p.db = dbias; p.dinit = dinit_state;
    p.part = (float*)workspace;
    return from_cuda(launch_short_conv_bwd(p, (int)q.W, d->dtype, sm_count(), (cudaStream_t)stream));
}

ssd_status ssd_short_conv_step(const ssd_short_conv_dims* d, const void* x, const float* weight,
                               const float* bias, const int32_t* slots, void* cache,
                               int64_t nslots, void* out, void* stream) {
    Dims q;
    ssd_status s = make(d, true, &q);
    if (s != SSD_OK) return s;
    if (q.n != q.T || nslots < 0 || nslots > (1LL << 31) - 1 || (!slots && nslots < q.n)) return SSD_ERR_SHAPE;
    if (q.n == 0) return SSD_OK;
    if (!x || !weight || !out || (!cache && nslots > 0)) return SSD_ERR_NULL;
    for (const void* a : {x, (const void*)weight, (const void*)bias, (const void*)slots, (const void*)cache,
                          (const void*)out})
        if (!aligned16(a)) return SSD_ERR_ALIGN;
    ShortConv& p = q.p;
    const Range in[] = {rng(x, span(q.T, p.xs, q.D, q.es)), rng(weight, (size_t)(q.D * q.W) * 4),
                        rng(bias, (size_t)q.D * 4), rng(slots, (size_t)q.n * 4)};
    const Range c = rng(cache, (size_t)(nslots * (q.W - 1) * q.D) * q.es), o = rng(out, q.rows);
    for (const Range& a : in)
        if (overlap(a, c) || overlap(a, o)) return SSD_ERR_ALIAS;
    if (overlap(c, o)) return SSD_ERR_ALIAS;
    if ((s = pre_launch()) != SSD_OK) return s;
    p.x = x; p.w = weight; p.bias = bias; p.slots = slots; p.cache = cache; p.nslots = nslots;
    p.batch = q.n; p.out = out;
    return from_cuda(launch_short_conv_step(p, (int)q.W, d->dtype, (cudaStream_t)stream));
}

}  // extern "C"
