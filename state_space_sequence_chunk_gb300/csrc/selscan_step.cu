// selscan_step.cu -- the selective scan for single tokens over a cache of states.
//
// For each row of the batch with a slot, per channel with N states:
//     h <- exp(delta A) h + delta x B (in place at cache[slot]),  y = (C.h + D x) silu(z).
// Bound by the states' traffic, 8 N bytes a channel, read once and written once.  LPC
// lanes hold a channel's states, four each, and V channels one after another: a warp
// moves 512 contiguous bytes of the cache at a time, V of them in flight, B and C are read
// once for V channels, and each of V lanes makes the numbers of one channel for the others.
// 2048 streams of 2048 channels and 16 states: 537 MB of states and 34 of rows in bf16, 91 us, 6.3 TB/s; 67 in
// fp32, 92 us, 6.5 TB/s (a lane with one channel, and expm1f: 221; V = 2: 127; 14 CTAs an SM 94, 10 states by
// vectors of one 113 with 14, 116 with 16); 64 streams 4.1 us, one 2.1 us.
#include "selscan.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 2;

// h exp(e).  Thousands of calls multiply a state, one after another, so near 1 it is h + h (exp(e) - 1),
// by the Taylor polynomial (to e^6: off by 1.2e-8 of h at most), whose errors have no side in
// common; where more goes in a token, by the fast exponential, with what rounds away of e log2(e)
// added back: what is left of a large state keeps its own precision.
__device__ __forceinline__ f32x2 decayed(f32x2 h, f32x2 e) {
    float e0, e1, h0, h1;
    unpair(e, e0, e1);
    e0 = max_nan(e0, -200.f);                // (every power from here on is 0)
    e1 = max_nan(e1, -200.f);
    e = pair(e0, e1);
    const f32x2 x = exp_in_range2(e);
    f32x2 m = fma2(e, both(1.f / 720), both(1.f / 120));
    m = fma2(e, m, both(1.f / 24));
    m = fma2(e, m, both(1.f / 6));
    m = fma2(e, m, both(0.5f));
    m = mul2(e, fma2(e, m, both(1.f)));
    const bool n0 = fabsf(e0) < 0.25f, n1 = fabsf(e1) < 0.25f;
    float m0, m1, x1, x2;
    unpair(m, m0, m1);
    unpair(x, x1, x2);
    unpair(h, h0, h1);
    return fma2(h, pair(n0 ? m0 : x1, n1 ? m1 : x2), pair(n0 ? h0 : 0.f, n1 ? h1 : 0.f));
}

// Four states at p, from the n-th of N on, 0 beyond.
template <bool VEC> __device__ __forceinline__ void load4(f32x2 (&v)[2], const float* p, int n, int N) {
    if (VEC) {
        ulonglong2 w = make_ulonglong2(0ull, 0ull);
        if (n < N) w = *reinterpret_cast<const ulonglong2*>(p);
        v[0] = w.x;
        v[1] = w.y;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = pair(n + 2 * i < N ? p[2 * i] : 0.f, n + 2 * i + 1 < N ? p[2 * i + 1] : 0.f);
    }
}

// LPC lanes hold a channel: N <= 4 LPC.  VEC: N is a multiple of four.
template <typename T, int LPC, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, VEC ? 16 : 14) selscan_step(const __grid_constant__ ScanStep p) {
    constexpr int V = LPC < 4 ? LPC : 4, kWide = 32 / LPC, kTile = V * kWide;   // channels of a lane, abreast, of a warp
    const int lane = threadIdx.x & 31, part = lane % LPC, n = 4 * part;
    const int tpg = (p.cpg + kTile - 1) / kTile, tiles = tpg * p.G;
    const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (item >= p.batch * tiles) return;
    const int b = (int)(item / tiles), tile = (int)(item - (int64_t)b * tiles), grp = tile / tpg;
    const int c0 = (tile - grp * tpg) * kTile + lane / LPC;
    const int own = c0 + part % V * kWide;               // the channel whose numbers this lane makes
    const bool in = own < p.cpg;
    const int d = grp * p.cpg + min(own, p.cpg - 1);
    const int64_t slot = p.slots != nullptr ? p.slots[b] : b;
    T* y = static_cast<T*>(p.y) + (int64_t)b * p.D + d;
    if (slot < 0 || slot >= p.nslots) {                  // no stream in this row: a zero output
        if (in && part < V) *y = from_f32<T>(0.f);
        return;
    }
    float* at = p.cache + (slot * p.D + grp * p.cpg + c0) * p.N + n;
    const float* A = p.A + (int64_t)(grp * p.cpg + c0) * p.N + n;
    const int64_t step = (int64_t)kWide * p.N;           // from one of the lane's channels to the next
    f32x2 h[V][2], a[V][2];
#pragma unroll
    for (int j = 0; j < V; ++j) load4<VEC>(h[j], at + j * step, c0 + j * kWide < p.cpg ? n : p.N, p.N);
#pragma unroll
    for (int j = 0; j < V; ++j) load4<VEC>(a[j], A + j * step, c0 + j * kWide < p.cpg ? n : p.N, p.N);
    // (every load before the first use of one: a conversion in a branch would wait there)
    Raw4<T> Br, Cr;
    fetch(Br, static_cast<const T*>(p.B) + b * p.Bs + (int64_t)grp * p.N, n, p.N, p.vecB != 0);
    fetch(Cr, static_cast<const T*>(p.C) + b * p.Cs + (int64_t)grp * p.N, n, p.N, p.vecC != 0);
    const T xr = static_cast<const T*>(p.x)[b * p.xs + d], tr = static_cast<const T*>(p.dt)[b * p.dts + d];
    const T zr = static_cast<const T*>(p.z != nullptr ? p.z : p.x)[p.z != nullptr ? b * p.zs + d : 0];
    const float bias = p.bias != nullptr ? p.bias[d] : 0.f, skip = p.Dk != nullptr ? p.Dk[d] : 0.f;
    const float4 Bv = widen(Br), Cv = widen(Cr);
    const f32x2 B[2] = {pair(Bv.x, Bv.y), pair(Bv.z, Bv.w)}, C[2] = {pair(Cv.x, Cv.y), pair(Cv.z, Cv.w)};
    const float x = to_f32(xr), v = to_f32(tr) + bias, z = to_f32(zr);
    const float delta = p.softplus ? softplus(v) : v, u = delta * x;
    float s[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int from = (lane & ~(V - 1)) | j;
        const f32x2 dj = both(V > 1 ? __shfl_sync(0xffffffffu, delta, from) : delta);
        const f32x2 uj = both(V > 1 ? __shfl_sync(0xffffffffu, u, from) : u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float a0, a1;
            unpair(a[j][i], a0, a1);
            h[j][i] = fma2(uj, B[i], decayed(h[j][i], mul2(dj, pair(max_nan(a0, -1e37f), max_nan(a1, -1e37f)))));
        }
        float lo, hi;
        unpair(fma2(C[1], h[j][1], mul2(C[0], h[j][0])), lo, hi);    // (C is 0 beyond N, and h finite there)
        s[j] = lo + hi;
        if (c0 + j * kWide < p.cpg) {
            float* to = at + j * step;
            if (VEC) {
                if (n < p.N) *reinterpret_cast<ulonglong2*>(to) = make_ulonglong2(h[j][0], h[j][1]);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    unpair(h[j][i], lo, hi);
                    if (n + 2 * i < p.N) to[2 * i] = lo;
                    if (n + 2 * i + 1 < p.N) to[2 * i + 1] = hi;
                }
            }
        }
    }
    // each lane gets its own channel's sum
    if (V >= 4) halve<V>(s, lane, V / 2);
    if (V >= 2) halve<2>(s, lane, 1);
    float o = s[0];
#pragma unroll
    for (int off = LPC / 2; off >= V; off >>= 1) o += __shfl_xor_sync(0xffffffffu, o, off);
    o = fmaf(skip, x, o);
    if (p.z != nullptr) o *= z * sigmoid<sizeof(T) == 4>(z);
    if (in && part < V) *y = from_f32<T>(o);
}

template <typename T, int LPC> cudaError_t go(const ScanStep& p, cudaStream_t stream) {
    constexpr int kTile = (LPC < 4 ? LPC : 4) * (32 / LPC);
    const int64_t tiles = (int64_t)((p.cpg + kTile - 1) / kTile) * p.G;
    const unsigned grid = (unsigned)((tiles * p.batch + kWarps - 1) / kWarps);
    if (p.N % 4 == 0) selscan_step<T, LPC, true><<<grid, kWarps * 32, 0, stream>>>(p);
    else selscan_step<T, LPC, false><<<grid, kWarps * 32, 0, stream>>>(p);
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
