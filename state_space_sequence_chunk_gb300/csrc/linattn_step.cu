// linattn_step.cu -- linear attention for single tokens over a cache of states.
//
// For each row of the batch with a slot, per head:
//     S <- lam S + v k^T (V x K, in place at cache[slot]),   o = scale S q.
// Bound by the state's HBM traffic: 8 K V bytes per head, read once and written
// once.  One warp holds four state rows in registers (each lane one float4 of
// each, a row in as few lanes as hold it), so every load of the state is in
// flight before the first is used, and a CTA is four such warps: even one
// stream's 24 heads of 64 x 128 give 96 CTAs.  64 streams, 80 heads of 64 x 128: 59 us
// a call, 83 % of the copy rate; with fp32 rows 61 us.
#include "linattn_internal.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 4;   // state rows per lane

__device__ __forceinline__ float4 load4(const float* p) {
    return __ldg(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
}

struct StepParams {
    const void *q, *k, *v;
    const float* a;
    const int* slots;
    float* cache;
    void* o;
    int64_t qs, ks, vs, nslots;
    int H, hpg, K, V;
    float scale;
};

// LPR lanes hold a row: K <= 4 LPR
template <typename T, int LPR>
__global__ void __launch_bounds__(kWarps * 32, 8) linattn_step(const __grid_constant__ StepParams p) {
    constexpr int kPer = 32 / LPR;                       // rows side by side in a warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int bh = blockIdx.x, b = bh / p.H, h = bh - b * p.H;
    const int row0 = (blockIdx.y * kWarps + warp) * kPer * kRows + lane / LPR;
    const int col = (lane % LPR) * 4;
    const bool in = col < p.K;
    T* o = static_cast<T*>(p.o) + (int64_t)bh * p.V;
    const int64_t slot = p.slots != nullptr ? p.slots[b] : b;
    if (slot < 0 || slot >= p.nslots) {                  // no stream in this row: a zero output
        if (lane % LPR == 0)
            for (int r = 0; r < kRows; ++r)
                if (row0 + r * kPer < p.V) o[row0 + r * kPer] = from_f32<T>(0.f);
        return;
    }
    float* S = p.cache + (slot * p.H + h) * (int64_t)p.V * p.K + col;
    float4 s[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int row = row0 + r * kPer;
        s[r] = in && row < p.V ? *reinterpret_cast<const float4*>(S + (int64_t)row * p.K)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int grp = h / p.hpg;
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 q = in ? load4(static_cast<const T*>(p.q) + b * p.qs + (int64_t)grp * p.K + col) : z;
    const float4 k = in ? load4(static_cast<const T*>(p.k) + b * p.ks + (int64_t)grp * p.K + col) : z;
    const T* v = static_cast<const T*>(p.v) + b * p.vs + (int64_t)h * p.V;
    float hi, lo;
    la_decay_pow(p.a, h, 1, hi, lo);
    float part[kRows], vr[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) vr[r] = row0 + r * kPer < p.V ? to_f32(v[row0 + r * kPer]) : 0.f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int row = row0 + r * kPer;
        s[r].x = fmaf(s[r].x, hi, fmaf(s[r].x, lo, vr[r] * k.x));
        s[r].y = fmaf(s[r].y, hi, fmaf(s[r].y, lo, vr[r] * k.y));
        s[r].z = fmaf(s[r].z, hi, fmaf(s[r].z, lo, vr[r] * k.z));
        s[r].w = fmaf(s[r].w, hi, fmaf(s[r].w, lo, vr[r] * k.w));
        if (in && row < p.V) *reinterpret_cast<float4*>(S + (int64_t)row * p.K) = s[r];
        part[r] = fmaf(s[r].x, q.x, fmaf(s[r].y, q.y, fmaf(s[r].z, q.z, s[r].w * q.w)));
    }
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1)
#pragma unroll
        for (int r = 0; r < kRows; ++r) part[r] += __shfl_xor_sync(0xffffffffu, part[r], off);
    if (lane % LPR == 0) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (row0 + r * kPer < p.V) o[row0 + r * kPer] = from_f32<T>(p.scale * part[r]);
    }
}

template <typename T>
cudaError_t go(const StepParams& p, int64_t batch, cudaStream_t stream) {
    const int lpr = p.K > 64 ? 32 : p.K > 32 ? 16 : p.K > 16 ? 8 : 4;
    const int rows = kWarps * kRows * (32 / lpr);
    const dim3 grid((unsigned)(batch * p.H), (unsigned)((p.V + rows - 1) / rows));
    auto k = lpr == 32 ? linattn_step<T, 32> : lpr == 16 ? linattn_step<T, 16>
           : lpr == 8 ? linattn_step<T, 8> : linattn_step<T, 4>;
    k<<<grid, kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linattn_step(const ssd_linattn_dims& d, int64_t qs, int64_t ks, int64_t vs,
                                const void* q, const void* k, const void* v, const float* a,
                                float scale, const int* slots, float* cache, int64_t nslots,
                                void* o, cudaStream_t stream) {
    StepParams p;
    p.q = q; p.k = k; p.v = v; p.a = a; p.slots = slots; p.cache = cache; p.o = o;
    p.qs = qs; p.ks = ks; p.vs = vs; p.nslots = nslots;
    p.H = (int)d.nheads; p.hpg = (int)(d.nheads / d.ngroups); p.K = (int)d.kdim; p.V = (int)d.vdim;
    p.scale = scale;
    return d.dtype == SSD_BF16 ? go<__nv_bfloat16>(p, d.nseqs, stream) : go<float>(p, d.nseqs, stream);
}

}  // namespace ssd
