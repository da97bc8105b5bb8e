// selscan_step.cu -- the selective scan for single tokens over a cache of states.
//
// For each row of the batch with a slot, per channel with N states:
//     h <- exp(delta A) h + delta x B (in place at cache[slot]),  y = (C.h + D x) silu(z).
// Bound by the states' traffic, 8 N bytes a channel, read once and written once.  A
// lane holds four states of one channel, so that a warp moves 512 contiguous bytes of
// the cache; the channel's own numbers are made by each of its lanes, which costs less
// than handing them round.
#include "selscan.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;

// LPC lanes hold a channel: N <= 4 LPC
template <typename T, int LPC>
__global__ void __launch_bounds__(kThreads) selscan_step(const __grid_constant__ ScanStep p) {
    constexpr int kCh = kThreads / LPC;
    constexpr bool kExact = sizeof(T) == 4;
    const int ctas = (p.D + kCh - 1) / kCh, b = blockIdx.x / ctas;
    const int ch = (blockIdx.x - b * ctas) * kCh + threadIdx.x / LPC, part = threadIdx.x % LPC, n = 4 * part;
    const bool in = ch < p.D;
    const int d = min(ch, p.D - 1);
    const int64_t slot = p.slots != nullptr ? p.slots[b] : b;
    T* y = static_cast<T*>(p.y) + (int64_t)b * p.D + d;
    if (slot < 0 || slot >= p.nslots) {              // no stream in this row: a zero output
        if (in && part == 0) *y = from_f32<T>(0.f);
        return;
    }
    const bool vec = p.N % 4 == 0, mine = in && n < p.N;
    float* at = p.cache + (slot * p.D + d) * p.N + n;
    const float* A = p.A + (int64_t)d * p.N + n;
    float h[4], a[4];
    if (vec) {
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 hv = mine ? *reinterpret_cast<const float4*>(at) : z;
        const float4 av = mine ? __ldg(reinterpret_cast<const float4*>(A)) : z;
        h[0] = hv.x; h[1] = hv.y; h[2] = hv.z; h[3] = hv.w;
        a[0] = av.x; a[1] = av.y; a[2] = av.z; a[3] = av.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool ok = mine && n + i < p.N;
            h[i] = ok ? at[i] : 0.f;
            a[i] = ok ? A[i] : 0.f;
        }
    }
    const int grp = d / p.cpg;
    const float4 Bv = load_states(static_cast<const T*>(p.B) + b * p.Bs + (int64_t)grp * p.N, n, p.N, false);
    const float4 Cv = load_states(static_cast<const T*>(p.C) + b * p.Cs + (int64_t)grp * p.N, n, p.N, false);
    const float B[4] = {Bv.x, Bv.y, Bv.z, Bv.w}, C[4] = {Cv.x, Cv.y, Cv.z, Cv.w};
    const float x = to_f32(static_cast<const T*>(p.x)[b * p.xs + d]);
    const float v = to_f32(static_cast<const T*>(p.dt)[b * p.dts + d]) + (p.bias != nullptr ? p.bias[d] : 0.f);
    const float z = p.z != nullptr ? to_f32(static_cast<const T*>(p.z)[b * p.zs + d]) : 0.f;
    const float skip = p.Dk != nullptr ? p.Dk[d] : 0.f;
    const float delta = p.softplus ? softplus<kExact>(v) : v, u = delta * x;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // h exp(delta A) as h + h (exp(delta A) - 1): thousands of calls multiply a state, one after another
        h[i] = fmaf(u, B[i], fmaf(h[i], expm1f(delta * fmaxf(a[i], -1e37f)), h[i]));
        if (n + i < p.N) s = fmaf(C[i], h[i], s);
    }
    if (vec) {
        if (mine) *reinterpret_cast<float4*>(at) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (mine && n + i < p.N) at[i] = h[i];
    }
#pragma unroll
    for (int off = LPC / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s = fmaf(skip, x, s);
    if (p.z != nullptr) s *= z * sigmoid(z);
    if (in && part == 0) *y = from_f32<T>(s);
}

template <typename T, int LPC> cudaError_t go(const ScanStep& p, cudaStream_t stream) {
    const int64_t ctas = (p.D + kThreads / LPC - 1) / (kThreads / LPC);
    selscan_step<T, LPC><<<(unsigned)(ctas * p.batch), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t by_states(const ScanStep& p, cudaStream_t stream) {
    if (p.N <= 4) return go<T, 1>(p, stream);
    if (p.N <= 8) return go<T, 2>(p, stream);
    if (p.N <= 16) return go<T, 4>(p, stream);
    if (p.N <= 32) return go<T, 8>(p, stream);
    return go<T, 16>(p, stream);
}

}  // namespace

cudaError_t launch_selscan_step(const ScanStep& p, int dtype, cudaStream_t stream) {
    return dtype == SSD_BF16 ? by_states<__nv_bfloat16>(p, stream) : by_states<float>(p, stream);
}

}  // namespace ssd
