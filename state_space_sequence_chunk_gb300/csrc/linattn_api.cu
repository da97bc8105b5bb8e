// linattn_api.cu -- the C entry points of linear attention: validation, the
// cut of long sequences into ranges, workspace layout and launches.
#include <math.h>

#include "linattn_internal.cuh"

namespace ssd {
namespace {

struct La {
    int64_t n, T, H, G, K, V, qs, ks, vs, hpg;
    int es;
    LaGeom g;
    size_t agg_bytes;    // one job's range states
};

ssd_status make_la(const ssd_linattn_dims* d, bool packed, bool backward, La* p) {
    if (!d) return SSD_ERR_NULL;
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d->reserved != 0 || d->nseqs < 0 || d->tokens < 0 || d->max_seqlen < 0) return SSD_ERR_SHAPE;
    if (d->nheads < 1 || d->nheads > 4096 || d->ngroups < 1 || d->nheads % d->ngroups != 0)
        return SSD_ERR_SHAPE;
    if (d->kdim < 16 || d->kdim > 128 || d->kdim % 16 != 0) return SSD_ERR_SHAPE;
    if (d->vdim < 16 || d->vdim > 128 || d->vdim % 16 != 0) return SSD_ERR_SHAPE;
    if (d->nseqs > (1 << 20) || d->tokens > (1LL << 30)) return SSD_ERR_SHAPE;
    p->n = d->nseqs; p->T = d->tokens; p->H = d->nheads; p->G = d->ngroups;
    p->K = d->kdim; p->V = d->vdim; p->hpg = p->H / p->G;
    p->es = d->dtype == SSD_BF16 ? 2 : 4;
    const int64_t grain = 16 / p->es;
    p->qs = d->q_stride ? d->q_stride : p->G * p->K;
    p->ks = d->k_stride ? d->k_stride : p->G * p->K;
    p->vs = d->v_stride ? d->v_stride : p->H * p->V;
    if (p->qs < p->G * p->K || p->ks < p->G * p->K || p->vs < p->H * p->V || p->qs % grain ||
        p->ks % grain || p->vs % grain || p->qs > (1LL << 31) || p->ks > (1LL << 31) || p->vs > (1LL << 31))
        return SSD_ERR_SHAPE;
    if (!packed && p->n > 0 && p->T % p->n != 0) return SSD_ERR_SHAPE;
    if (p->n == 0 && p->T > 0 && !packed) return SSD_ERR_SHAPE;

    LaGeom& g = p->g;
    g.cu = nullptr;
    g.nseq = (int)p->n; g.H = (int)p->H; g.T = (int)p->T;
    g.L = packed || p->n == 0 ? 0 : (int)(p->T / p->n);
    g.a = nullptr;
    // A sequence is cut into ranges where a chain of its whole length would keep the
    // other SMs waiting: where it is longer than what an SM gets when the work is spread
    // evenly, by what the cut costs.  That is a second reading of two operands and, with
    // all SMs at work, a slower chunk (together another 9/8 of the share in bf16, 2/5 in
    // fp32, whose chunks are bound by arithmetic), and two launches (some 9 chunks' time
    // in bf16, 1.4 in fp32).  One bf16 sequence, heads of 128 x 64, cut and whole: 2048
    // tokens on 24 heads 35 and 37 us, on 38 42 and 38; 4096 on 38 59 and 66 to 71, on 50
    // 68 to 74 and 67 to 72, on 76 107 and 77; 16384 on 64 195 to 227 and 244 to 257, on
    // 76 330 and 260; gradients: 16384 on 8 161 to 213 and 254 to 318, on 24 390 to 515
    // and 268 to 386.  fp32: 1024 on 76 210 and 260 to 275, on 100 283 to 300 and 260 to
    // 275; 4096 on 100 955 to 985 and 1024 to 1058, on 128 1400 and 1050.
    const int64_t kb = (p->K + kLaCols - 1) / kLaCols, vb = (p->V + kLaCols - 1) / kLaCols;
    const int64_t cols = backward ? 2 * kb + vb : vb;
    const int64_t sms = sm_count(), share = p->T * p->H * cols / sms;
    const int64_t least = d->dtype == SSD_F32 ? 128 : 512;   // fp32 chunks take longer
    int64_t longest = packed ? (d->max_seqlen ? d->max_seqlen : p->T) : g.L;
    if (longest > p->T) longest = p->T;
    int64_t R = (share / 2 + 127) / 128 * 128;
    if (R < least) R = least;
    // (without a sequence there is none to cut: every row's result is 0)
    g.split = p->n > 0 && longest > R &&
              longest > share + (d->dtype == SSD_F32 ? share * 2 / 5 + 176 : share * 9 / 8 + 1152);
    // Half a share, so that the range taken last adds at most half; where the lengths
    // are known, the number of ranges that fills the SMs in the shortest time (a range
    // costs 2 chunks more than its own): one sequence of 65536 tokens on 24 chains in
    // 12.7 ranges of half a share left a third round of 8 items, 293 us instead of 279.
    if (g.split && (p->n == 1 || !packed)) {
        const int64_t L = packed ? p->T : g.L, slots = sms * (d->dtype == SSD_F32 ? 2 : 1);
        int64_t best = INT64_MAX;
        for (int64_t n = 2; n <= 64; ++n) {
            const int64_t r = ((L + n - 1) / n + 127) / 128 * 128;
            if (r < least) break;
            // (ranges end at multiples of r of all rows: one more where r does not divide L)
            const int64_t m = n + (p->n > 1 && L % r != 0);
            const int64_t cost = (p->n * p->H * cols * m + slots - 1) / slots * (r / 128 + 2);
            if (cost < best) {
                best = cost;
                R = r;
            }
        }
    }
    g.R = g.split ? (int)R : (int)(p->T > 0 ? (p->T + 127) / 128 * 128 : 128);
    const int64_t cap = g.split ? p->T / R + p->n + 2 : p->n + 1;
    if (cap > (1LL << 24)) return SSD_ERR_SHAPE;
    g.range_cap = (int)cap;
    p->agg_bytes = g.split ? round_up256((size_t)(la_slots(p->T, R) * p->H * p->K * p->V) * 4) : 0;
    return SSD_OK;
}

// make_la for a whole prompt or its gradient, whose launch has a CTA for each range, head,
// job and 64 columns: their number has to fit a grid (in bf16, where all are in one
// dimension of it).
ssd_status make_prompt(const ssd_linattn_dims* d, bool packed, bool backward, La* p) {
    const ssd_status s = make_la(d, packed, backward, p);
    if (s != SSD_OK || d->dtype != SSD_BF16) return s;
    const int64_t cols = backward && p->K > p->V ? p->K : p->V;
    const int64_t items = p->g.range_cap * p->H * (backward ? 3 : 1) * ((cols + kLaCols - 1) / kLaCols);
    return items < (1LL << 31) ? SSD_OK : SSD_ERR_SHAPE;
}

size_t part_bytes(const La& p) {   // per-head dq and dk, before the sum over a group
    return p.hpg > 1 ? 2 * round_up256((size_t)(p.T * p.H * p.K) * 4) : 0;
}

cudaError_t run_jobs(LaParams& p, int dtype, cudaStream_t st) {
    auto pass = [&](int mode) {
        return dtype == SSD_BF16 ? launch_linattn_tc(p, mode, st)
                                 : launch_linattn_simt(p, mode, st);
    };
    cudaError_t e = cudaSuccess;
    if (p.g.split) {
        e = pass(1);
        if (e == cudaSuccess) e = launch_linattn_scan(p, st);
    }
    return e != cudaSuccess ? e : pass(0);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_linattn_workspace_bytes(const ssd_linattn_dims* d, int backward) {
    // enough for packed and, where the sizes allow them, equal sequences
    size_t need = 0;
    for (int packed = 0; packed < 2; ++packed) {
        La p;
        if (make_prompt(d, packed != 0, backward != 0, &p) != SSD_OK) continue;
        const size_t b = backward ? 3 * p.agg_bytes + part_bytes(p) : p.agg_bytes;
        if (b > need) need = b;
    }
    return need;
}

ssd_status ssd_linattn_fwd(const ssd_linattn_dims* d, const void* q, const void* k, const void* v,
                           const float* log_decay, float scale, const int32_t* cu_seqlens,
                           const float* init_state, void* o, float* final_state, void* workspace,
                           size_t workspace_bytes, void* stream) {
    La p;
    ssd_status s = make_prompt(d, cu_seqlens != nullptr, false, &p);
    if (s != SSD_OK) return s;
    if (p.n == 0 && p.T == 0) return SSD_OK;
    if (!isfinite(scale)) return SSD_ERR_SHAPE;
    if (!log_decay || (p.T > 0 && (!q || !k || !v || !o))) return SSD_ERR_NULL;
    if (p.agg_bytes > 0 && !workspace) return SSD_ERR_NULL;
    if (workspace_bytes < p.agg_bytes) return SSD_ERR_WORKSPACE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(log_decay) ||
        !aligned16(cu_seqlens) || !aligned16(init_state) || !aligned16(final_state) ||
        !aligned16(workspace))
        return SSD_ERR_ALIGN;
    const size_t sb = (size_t)(p.n * p.H * p.V * p.K) * 4, ob = (size_t)(p.T * p.H * p.V) * p.es;
    const Range in[] = {rng(q, span(p.T, p.qs, p.G * p.K, p.es)), rng(k, span(p.T, p.ks, p.G * p.K, p.es)),
                        rng(v, span(p.T, p.vs, p.H * p.V, p.es)), rng(log_decay, (size_t)p.H * 4),
                        rng(cu_seqlens, (size_t)(p.n + 1) * 4), rng(init_state, sb)};
    const Range out[] = {rng(o, ob), rng(workspace, p.agg_bytes), rng(final_state, sb)};
    for (int i = 0; i < 6; ++i)
        for (int j = 0; j < 3; ++j)
            if (overlap(in[i], out[j]) && !(i == 5 && j == 2 && init_state == final_state))
                return SSD_ERR_ALIAS;
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SSD_ERR_ALIAS;
    if ((s = pre_launch()) != SSD_OK) return s;
    LaParams lp;
    lp.g = p.g;
    lp.g.cu = cu_seqlens;
    lp.g.a = log_decay;
    lp.njobs = 1;
    LaJob& j = lp.job[0];
    j = LaJob{q, k, v, p.qs, p.ks, p.vs, (int)p.hpg, (int)p.hpg, 1, (int)p.G, (int)p.G, (int)p.H,
              (int)p.K, (int)p.V, o, 0, 0, 1.f, scale, 1, (int)p.K, init_state, final_state,
              (float*)workspace};
    return from_cuda(run_jobs(lp, d->dtype, (cudaStream_t)stream));
}

ssd_status ssd_linattn_bwd(const ssd_linattn_dims* d, const void* q, const void* k, const void* v,
                           const void* dout, const float* log_decay, float scale,
                           const int32_t* cu_seqlens, const float* init_state,
                           const float* dfinal_state, void* dq, void* dk, void* dv,
                           float* dinit_state, void* workspace, size_t workspace_bytes,
                           void* stream) {
    La p;
    ssd_status s = make_prompt(d, cu_seqlens != nullptr, true, &p);
    if (s != SSD_OK) return s;
    if (p.n == 0 && p.T == 0) return SSD_OK;
    if (!isfinite(scale)) return SSD_ERR_SHAPE;
    if (!log_decay || (p.T > 0 && (!q || !k || !v || !dout || !dq || !dk || !dv))) return SSD_ERR_NULL;
    const size_t need = 3 * p.agg_bytes + part_bytes(p);
    if (need > 0 && !workspace) return SSD_ERR_NULL;
    if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dout) || !aligned16(dq) ||
        !aligned16(dk) || !aligned16(dv) || !aligned16(log_decay) || !aligned16(cu_seqlens) ||
        !aligned16(init_state) || !aligned16(dfinal_state) || !aligned16(dinit_state) ||
        !aligned16(workspace))
        return SSD_ERR_ALIGN;
    const size_t sb = (size_t)(p.n * p.H * p.V * p.K) * 4, vb = (size_t)(p.T * p.H * p.V) * p.es,
                 kb = (size_t)(p.T * p.G * p.K) * p.es;
    const Range in[] = {rng(q, span(p.T, p.qs, p.G * p.K, p.es)), rng(k, span(p.T, p.ks, p.G * p.K, p.es)),
                        rng(v, span(p.T, p.vs, p.H * p.V, p.es)), rng(dout, vb),
                        rng(log_decay, (size_t)p.H * 4), rng(cu_seqlens, (size_t)(p.n + 1) * 4),
                        rng(init_state, sb), rng(dfinal_state, sb)};
    const Range out[] = {rng(dq, kb), rng(dk, kb), rng(dv, vb), rng(dinit_state, sb), rng(workspace, need)};
    for (const Range& a : in)
        for (const Range& b : out)
            if (overlap(a, b)) return SSD_ERR_ALIAS;
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SSD_ERR_ALIAS;
    if ((s = pre_launch()) != SSD_OK) return s;
    char* ws = (char*)workspace;
    float *agg[3], *part[2] = {nullptr, nullptr};
    for (int i = 0; i < 3; ++i) agg[i] = (float*)(ws + i * p.agg_bytes);
    if (p.hpg > 1)
        for (int i = 0; i < 2; ++i) part[i] = (float*)(ws + 3 * p.agg_bytes + i * (part_bytes(p) / 2));
    LaParams lp;
    lp.g = p.g;
    lp.g.cu = cu_seqlens;
    lp.g.a = log_decay;
    lp.njobs = 3;
    const int G = (int)p.G, H = (int)p.H, K = (int)p.K, V = (int)p.V, hpg = (int)p.hpg;
    const int64_t os = p.H * p.V;
    const int shared = hpg > 1;
    // dq = F(do, v; k): X = S^T of the forward pass
    lp.job[0] = LaJob{dout, v, k, os, p.vs, p.ks, 1, 1, hpg, H, H, G, V, K, shared ? (void*)part[0] : dq,
                      shared, 0, 1.f, scale, K, 1, init_state, nullptr, agg[0]};
    // dk = Frev(v, do; q): X = R
    lp.job[1] = LaJob{v, dout, q, p.vs, os, p.qs, 1, 1, hpg, H, H, G, V, K, shared ? (void*)part[1] : dk,
                      shared, 1, scale, 1.f, K, 1, dfinal_state, nullptr, agg[1]};
    // dv = Frev(k, q; do): X = R^T, which ends as dS_0
    lp.job[2] = LaJob{k, q, dout, p.ks, p.qs, os, hpg, hpg, 1, G, G, H, K, V, dv,
                      0, 1, scale, 1.f, 1, K, dfinal_state, dinit_state, agg[2]};
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = run_jobs(lp, d->dtype, st);
    if (e == cudaSuccess && shared && p.T > 0)
        e = launch_linattn_group_sum(part, dq, dk, p.T, G, hpg, K, d->dtype, st);
    return from_cuda(e);
}

ssd_status ssd_linattn_step(const ssd_linattn_dims* d, const void* q, const void* k, const void* v,
                            const float* log_decay, float scale, const int32_t* slots, float* cache,
                            int64_t nslots, void* o, void* stream) {
    La p;
    ssd_status s = make_la(d, true, false, &p);
    if (s != SSD_OK) return s;
    if (p.n != p.T || nslots < 0 || !isfinite(scale)) return SSD_ERR_SHAPE;
    if (!slots && nslots < p.n) return SSD_ERR_SHAPE;
    if (p.n * p.H > (1LL << 31) - 1) return SSD_ERR_SHAPE;
    if (p.n == 0) return SSD_OK;
    if (!q || !k || !v || !log_decay || !o || (!cache && nslots > 0)) return SSD_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(log_decay) ||
        !aligned16(slots) || !aligned16(cache) || !aligned16(o))
        return SSD_ERR_ALIGN;
    const Range in[] = {rng(q, span(p.T, p.qs, p.G * p.K, p.es)), rng(k, span(p.T, p.ks, p.G * p.K, p.es)),
                        rng(v, span(p.T, p.vs, p.H * p.V, p.es)), rng(log_decay, (size_t)p.H * 4),
                        rng(slots, (size_t)p.n * 4)};
    const Range cr = rng(cache, (size_t)(nslots * p.H * p.V * p.K) * 4);
    const Range orr = rng(o, (size_t)(p.T * p.H * p.V) * p.es);
    for (const Range& r : in)
        if (overlap(r, cr) || overlap(r, orr)) return SSD_ERR_ALIAS;
    if (overlap(cr, orr)) return SSD_ERR_ALIAS;
    if ((s = pre_launch()) != SSD_OK) return s;
    return from_cuda(launch_linattn_step(*d, p.qs, p.ks, p.vs, q, k, v, log_decay, scale, slots,
                                         cache, nslots, o, (cudaStream_t)stream));
}

}  // extern "C"
