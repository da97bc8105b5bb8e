// selscan_api.cu -- the C entry points of the selective scan: validation, the cut of
// long sequences into ranges, workspace layout and launches.
#include <limits.h>

#include "selscan.cuh"

namespace ssd {
namespace {

constexpr int64_t kMaxSlots = 512;   // slots of the gradient's terms of dA

struct Scan {
    ScanParams p;
    int64_t n, T, D, N, G;
    int es;
    size_t rows, brows, states, checkpoints;   // bytes of [T, D], [T, G, N], [n, D, N], the stored states
    size_t agg, aggd, part, partA, partD;      // workspace, in this order
};

ssd_status make(const ssd_selscan_dims* d, bool packed, bool backward, Scan* out) {
    if (!d) return SSD_ERR_NULL;
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d->reserved != 0 || d->nseqs < 0 || d->nseqs > (1 << 20) || d->tokens < 0 || d->tokens > (1LL << 30) ||
        d->max_seqlen < 0)
        return SSD_ERR_SHAPE;
    if (d->dim < 8 || d->dim > 65536 || d->dstate < 1 || d->dstate > 64 || d->ngroups < 1 ||
        d->dim % d->ngroups != 0 || (d->dim / d->ngroups) % 8 != 0)
        return SSD_ERR_SHAPE;
    if (d->dt_softplus != 0 && d->dt_softplus != 1) return SSD_ERR_SHAPE;
    Scan q = {};
    q.n = d->nseqs; q.T = d->tokens; q.D = d->dim; q.N = d->dstate; q.G = d->ngroups;
    q.es = d->dtype == SSD_BF16 ? 2 : 4;
    ScanParams& p = q.p;
    p.xs = d->x_stride ? d->x_stride : q.D;
    p.dts = d->dt_stride ? d->dt_stride : q.D;
    p.zs = d->z_stride ? d->z_stride : q.D;
    p.Bs = d->B_stride ? d->B_stride : q.G * q.N;
    p.Cs = d->C_stride ? d->C_stride : q.G * q.N;
    for (int64_t s : {p.xs, p.dts, p.zs})
        if (s < q.D || s % (16 / q.es) || s > (1LL << 31)) return SSD_ERR_SHAPE;
    for (int64_t s : {p.Bs, p.Cs})
        if (s < q.G * q.N || s > (1LL << 31)) return SSD_ERR_SHAPE;
    if (!packed && (q.n > 0 ? q.T % q.n != 0 : q.T > 0)) return SSD_ERR_SHAPE;
    p.D = (int)q.D; p.N = (int)q.N; p.G = (int)q.G; p.cpg = (int)(q.D / q.G);
    p.softplus = d->dt_softplus;
    ScanGeom& g = p.g;
    g.nseq = (int)q.n; g.T = (int)q.T;
    g.L = packed || q.n == 0 ? 0 : (int)(q.T / q.n);
    q.rows = (size_t)(q.T * q.D) * q.es;
    q.brows = (size_t)(q.T * q.G * q.N) * q.es;
    q.states = (size_t)(q.n * q.D * q.N) * 4;
    q.checkpoints = (size_t)((q.T / kScanChunk + q.n) * q.D * q.N) * 4;

    // A sequence is cut where a chain of its whole length would keep the other SMs waiting.  A
    // warp by itself takes 113 ns a token; the cut's two passes take 240 ps for each token
    // and warp when all SMs work, and some 25 us of launches and ramps.  Whole and cut, us, 16
    // states: 256 tokens of 2048 channels (64 warps) 37 and 40, 512 of 5120 63 and 47, 2048 of
    // 2048 in 4 sequences 95 and 61, 8192 of 2048 929 and 152, in 6 sequences 227 and 155;
    // 16384 of 5120 in 12 447 and 627; 16384 of 2048 in 40 207 and 293; 4096 of 768, 64 states, in 8
    // 123 and 158.  Backwards a CTA of 64 (32, 16) channels takes 285 ns a token by itself, and
    // the cut's passes 1.7 ns for each token and CTA: the same sizes 92 and 64, 167 and 113, 265 and
    // 153, 2338 and 462, 672 and 465, -, 799 and 874, 448 and 447.  Where the longest sequence is not
    // known it may be all of the tokens.
    const int64_t bt = selscan_bwd_channels((int)q.N), tiles = (p.cpg + bt - 1) / bt;
    const int64_t warps = q.G * ((p.cpg * (q.N <= 16 ? 1 : q.N <= 32 ? 2 : 4) + 31) / 32);
    const int64_t sms = sm_count(), work = q.T * (backward ? tiles * q.G : warps);
    int64_t longest = packed ? (d->max_seqlen ? d->max_seqlen : q.T) : g.L;
    if (longest > q.T) longest = q.T;
    g.R = INT_MAX;
    if (q.n > 0 && longest > (backward ? work / (sms * 8 / 7) + 136 : work / (3 * sms) + 256)) {
        // several ranges for each warp that is resident, but not too short (2048 tokens of 1536
        // channels: ranges of 32, 64, 96, 128, 256 tokens 52, 49, 49, 57, 65 us, backwards 123, 123,
        // 119, 131, 149; 8192 of 2048: 64, 96, 128 163, 153, 153; 65536 of 1536: 96, 160, 384: 842, 804, 779)
        int64_t R = (work / ((backward ? 13 : 54) * sms) + 16) / 32 * 32;
        const int64_t least = backward ? 64 : 96;
        R = R < least ? least : R > 512 ? 512 : R;
        if (R < longest) g.R = (int)R;
    }
    const bool cut = g.R <= q.T;
    g.items = (int)(cut ? q.T / g.R + q.n : q.n);
    q.agg = cut ? round_up256((size_t)((int64_t)g.items * q.D * q.N) * 4) : 0;
    q.aggd = cut ? round_up256((size_t)((int64_t)g.items * q.D) * 4) : 0;
    if (backward) {
        p.per_slot = (int)((g.items + kMaxSlots - 1) / kMaxSlots);
        if (p.per_slot < 1) p.per_slot = 1;
        p.slots = (g.items + p.per_slot - 1) / p.per_slot;
        q.part = round_up256((size_t)(tiles * q.T * q.G * 2 * q.N) * 4);
        q.partA = round_up256((size_t)(p.slots * q.D * q.N) * 4);
        q.partD = round_up256((size_t)(p.slots * 2 * q.D) * 4);
    }
    // CTAs of a launch: two warps of channels each at least
    if (((int64_t)g.items + 64) * (warps + 1) >= (1LL << 31) || q.T * q.G * 2 * q.N >= (1LL << 38)) return SSD_ERR_SHAPE;
    *out = q;
    return SSD_OK;
}

size_t need(const Scan& q) { return q.agg + q.aggd + q.part + q.partA + q.partD; }

// Where B's and C's rows can be read in vectors of four states.
int vectors(const Scan& q, const void* p, int64_t stride) {
    return q.N % 4 == 0 && stride % 4 == 0 && (uintptr_t)p % (4 * q.es) == 0;
}
bool aligned_to(const void* p, int es) { return (uintptr_t)p % es == 0; }

void operands(Scan& q, const void* x, const void* dt, const float* A, const void* B, const void* C, const float* D,
              const void* z, const float* dt_bias, const int32_t* cu) {
    ScanParams& p = q.p;
    p.x = x; p.dt = dt; p.A = A; p.B = B; p.C = C; p.Dk = D; p.z = z; p.bias = dt_bias; p.g.cu = cu;
    p.vecB = vectors(q, B, p.Bs);
    p.vecC = vectors(q, C, p.Cs);
}

constexpr int kOperands = 9;
void operand_ranges(const Scan& q, const void* x, const void* dt, const float* A, const void* B, const void* C,
                    const float* D, const void* z, const float* dt_bias, const int32_t* cu, Range* r) {
    const ScanParams& p = q.p;
    const Range all[kOperands] = {
        rng(x, span(q.T, p.xs, q.D, q.es)), rng(dt, span(q.T, p.dts, q.D, q.es)), rng(A, (size_t)(q.D * q.N) * 4),
        rng(B, span(q.T, p.Bs, q.G * q.N, q.es)), rng(C, span(q.T, p.Cs, q.G * q.N, q.es)), rng(D, (size_t)q.D * 4),
        rng(z, span(q.T, p.zs, q.D, q.es)), rng(dt_bias, (size_t)q.D * 4), rng(cu, (size_t)(q.n + 1) * 4)};
    for (int i = 0; i < kOperands; ++i) r[i] = all[i];
}

void workspace_at(Scan& q, void* workspace) {
    char* w = (char*)workspace;
    ScanParams& p = q.p;
    p.agg = (float*)w;
    p.aggd = (float*)(w += q.agg);
    p.part = (float*)(w += q.aggd);
    p.partA = (float*)(w += q.part);
    p.partD = (float*)(w += q.partA);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_selscan_workspace_bytes(const ssd_selscan_dims* d, int backward) {
    // enough for packed and, where the sizes allow them, equal sequences
    size_t most = 0;
    for (int packed = 0; packed < 2; ++packed) {
        Scan q;
        if (make(d, packed != 0, backward != 0, &q) == SSD_OK && need(q) > most) most = need(q);
    }
    return most;
}

ssd_status ssd_selscan_fwd(const ssd_selscan_dims* d, const void* x, const void* dt, const float* A,
                           const void* B, const void* C, const float* D, const void* z,
                           const float* dt_bias, const int32_t* cu_seqlens, const float* init_state,
                           void* y, float* final_state, float* states, void* workspace,
                           size_t workspace_bytes, void* stream) {
    Scan q;
    ssd_status s = make(d, cu_seqlens != nullptr, false, &q);
    if (s != SSD_OK) return s;
    if (q.T == 0 && q.n == 0) return SSD_OK;
    if (!A || (q.T > 0 && (!x || !dt || !B || !C || !y))) return SSD_ERR_NULL;
    if (need(q) > 0 && !workspace) return SSD_ERR_NULL;
    if (workspace_bytes < need(q)) return SSD_ERR_WORKSPACE;
    for (const void* a : {x, dt, (const void*)A, (const void*)D, z, (const void*)dt_bias, (const void*)cu_seqlens,
                          (const void*)init_state, (const void*)y, (const void*)final_state, (const void*)states,
                          (const void*)workspace})
        if (!aligned16(a)) return SSD_ERR_ALIGN;
    if (!aligned_to(B, q.es) || !aligned_to(C, q.es)) return SSD_ERR_ALIGN;
    Range in[kOperands + 1];
    operand_ranges(q, x, dt, A, B, C, D, z, dt_bias, cu_seqlens, in);
    in[kOperands] = rng(init_state, q.states);
    const Range out[] = {rng(y, q.rows), rng(states, q.checkpoints), rng(workspace, need(q)),
                         rng(final_state, q.states)};
    for (int i = 0; i <= kOperands; ++i)
        for (int j = 0; j < 4; ++j)
            if (overlap(in[i], out[j]) && !(i == kOperands && j == 3 && init_state == final_state)) return SSD_ERR_ALIAS;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SSD_ERR_ALIAS;
    if ((s = pre_launch()) != SSD_OK) return s;
    operands(q, x, dt, A, B, C, D, z, dt_bias, cu_seqlens);
    ScanParams& p = q.p;
    p.init = init_state; p.y = y; p.fin = final_state; p.states = states;
    workspace_at(q, workspace);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    if (q.agg > 0) {
        e = launch_selscan_fwd(p, d->dtype, kScanSums, st);
        if (e == cudaSuccess) e = launch_selscan_ranges(p, 0, st);
    }
    if (e == cudaSuccess) e = launch_selscan_fwd(p, d->dtype, kScanMain, st);
    return from_cuda(e);
}

ssd_status ssd_selscan_bwd(const ssd_selscan_dims* d, const void* x, const void* dt, const float* A,
                           const void* B, const void* C, const float* D, const void* z,
                           const float* dt_bias, const int32_t* cu_seqlens, const float* states,
                           const void* dout, const float* dfinal_state, void* dx, void* ddt,
                           float* dA, void* dB, void* dC, float* dD, void* dz, float* ddt_bias,
                           float* dinit_state, void* workspace, size_t workspace_bytes,
                           void* stream) {
    Scan q;
    ssd_status s = make(d, cu_seqlens != nullptr, true, &q);
    if (s != SSD_OK) return s;
    if (!A || !dA) return SSD_ERR_NULL;
    if (q.T > 0 && (!x || !dt || !B || !C || !states || !dout || !dx || !ddt || !dB || !dC || (z && !dz)))
        return SSD_ERR_NULL;
    if (need(q) > 0 && !workspace) return SSD_ERR_NULL;
    if (workspace_bytes < need(q)) return SSD_ERR_WORKSPACE;
    for (const void* a : {x, dt, (const void*)A, (const void*)D, z, (const void*)dt_bias, (const void*)cu_seqlens,
                          (const void*)states, dout, (const void*)dfinal_state, (const void*)dx, (const void*)ddt,
                          (const void*)dA, (const void*)dB, (const void*)dC, (const void*)dD, (const void*)dz,
                          (const void*)ddt_bias, (const void*)dinit_state, (const void*)workspace})
        if (!aligned16(a)) return SSD_ERR_ALIGN;
    if (!aligned_to(B, q.es) || !aligned_to(C, q.es)) return SSD_ERR_ALIGN;
    Range in[kOperands + 3];
    operand_ranges(q, x, dt, A, B, C, D, z, dt_bias, cu_seqlens, in);
    in[kOperands] = rng(states, q.checkpoints);
    in[kOperands + 1] = rng(dout, q.rows);
    in[kOperands + 2] = rng(dfinal_state, q.states);
    const Range out[] = {rng(dx, q.rows), rng(ddt, q.rows), rng(dA, (size_t)(q.D * q.N) * 4), rng(dB, q.brows),
                         rng(dC, q.brows), rng(dD, (size_t)q.D * 4), rng(z ? dz : nullptr, q.rows),
                         rng(ddt_bias, (size_t)q.D * 4), rng(dinit_state, q.states), rng(workspace, need(q))};
    for (const Range& a : in)
        for (const Range& b : out)
            if (overlap(a, b)) return SSD_ERR_ALIAS;
    for (int i = 0; i < 10; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SSD_ERR_ALIAS;
    if ((s = pre_launch()) != SSD_OK) return s;
    operands(q, x, dt, A, B, C, D, z, dt_bias, cu_seqlens);
    ScanParams& p = q.p;
    p.states = const_cast<float*>(states); p.dout = dout; p.dfin = dfinal_state; p.dx = dx; p.ddt = ddt; p.dz = dz;
    p.dB = dB; p.dC = dC; p.dA = dA; p.dD = dD; p.dbias = ddt_bias; p.dinit = dinit_state;
    workspace_at(q, workspace);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    if (q.agg > 0) {
        e = launch_selscan_fwd(p, d->dtype, kScanRevSums, st);
        if (e == cudaSuccess) e = launch_selscan_ranges(p, 1, st);
    }
    if (e == cudaSuccess) e = launch_selscan_bwd(p, d->dtype, st);
    return from_cuda(e);
}

ssd_status ssd_selscan_step(const ssd_selscan_dims* d, const void* x, const void* dt, const float* A,
                            const void* B, const void* C, const float* D, const void* z,
                            const float* dt_bias, const int32_t* slots, float* cache,
                            int64_t nslots, void* y, void* stream) {
    Scan q;
    ssd_status s = make(d, true, false, &q);
    if (s != SSD_OK) return s;
    if (q.n != q.T || nslots < 0 || nslots > (1LL << 31) - 1 || (!slots && nslots < q.n)) return SSD_ERR_SHAPE;
    if (q.n * ((q.D + 7) / 8) >= (1LL << 31)) return SSD_ERR_SHAPE;
    if (q.n == 0) return SSD_OK;
    if (!x || !dt || !A || !B || !C || !y || (!cache && nslots > 0)) return SSD_ERR_NULL;
    for (const void* a : {x, dt, (const void*)A, (const void*)D, z, (const void*)dt_bias, (const void*)slots,
                          (const void*)cache, (const void*)y})
        if (!aligned16(a)) return SSD_ERR_ALIGN;
    if (!aligned_to(B, q.es) || !aligned_to(C, q.es)) return SSD_ERR_ALIGN;
    Range in[kOperands + 1];
    operand_ranges(q, x, dt, A, B, C, D, z, dt_bias, nullptr, in);
    in[kOperands] = rng(slots, (size_t)q.n * 4);
    const Range c = rng(cache, (size_t)(nslots * q.D * q.N) * 4), o = rng(y, q.rows);
    for (const Range& a : in)
        if (overlap(a, c) || overlap(a, o)) return SSD_ERR_ALIAS;
    if (overlap(c, o)) return SSD_ERR_ALIAS;
    if ((s = pre_launch()) != SSD_OK) return s;
    const ScanParams& p = q.p;
    ScanStep t = {};
    t.D = p.D; t.N = p.N; t.G = p.G; t.cpg = p.cpg; t.softplus = p.softplus;
    t.vecB = vectors(q, B, p.Bs); t.vecC = vectors(q, C, p.Cs);
    t.batch = q.n; t.nslots = nslots;
    t.x = x; t.dt = dt; t.z = z; t.B = B; t.C = C;
    t.xs = p.xs; t.dts = p.dts; t.zs = p.zs; t.Bs = p.Bs; t.Cs = p.Cs;
    t.A = A; t.Dk = D; t.bias = dt_bias; t.slots = slots; t.cache = cache; t.y = y;
    return from_cuda(launch_selscan_step(t, d->dtype, (cudaStream_t)stream));
}

}  // extern "C"
