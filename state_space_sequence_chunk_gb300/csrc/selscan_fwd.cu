// selscan_fwd.cu -- the selective scan over packed prompts.
//
// One warp walks 32 / LPC channels of a sequence (or of a range of it), a lane
// holding S states of one channel in registers: with 16 states a lane is a
// channel, so the sum over the states needs no other lane, and x, dt, z and y go
// straight between its registers and memory (64 bytes a row and warp, whole
// sectors).  Tiles of eight tokens: the next tile's loads are in flight while this
// one is computed; its delta and u = delta x are made first, all eight side by
// side, and the rows of B and C, which every lane reads, pass through shared
// memory as fp32.  The recurrence itself is the packed fp32 instructions' work: per
// pair of states two products, two multiply-adds and two exponentials.
#include "selscan.cuh"

namespace ssd {
namespace {

constexpr int kTok = 8;      // tokens of a tile
constexpr int kWarps = 2;    // warps of a CTA, each on its own
constexpr int kZeroItems = 64;

template <typename T> struct Raw4;                        // four states as loaded
template <> struct Raw4<float> { float4 v; };
template <> struct Raw4<__nv_bfloat16> { uint2 v; };
__device__ __forceinline__ void fetch(Raw4<float>& r, const float* p, int n, int N, bool vec) {
    r.v = load_states(p, n, N, vec);
}
__device__ __forceinline__ void fetch(Raw4<__nv_bfloat16>& r, const __nv_bfloat16* p, int n, int N, bool vec) {
    if (vec) {
        r.v = n < N ? __ldg(reinterpret_cast<const uint2*>(p + n)) : make_uint2(0u, 0u);
    } else {
        const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
        uint32_t e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = n + i < N ? (uint32_t)__ldg(q + n + i) : 0u;
        r.v = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
    }
}
__device__ __forceinline__ float4 widen(const Raw4<float>& r) { return r.v; }
__device__ __forceinline__ float4 widen(const Raw4<__nv_bfloat16>& r) {
    return make_float4(__uint_as_float(r.v.x << 16), __uint_as_float(r.v.x & 0xFFFF0000u),
                       __uint_as_float(r.v.y << 16), __uint_as_float(r.v.y & 0xFFFF0000u));
}

template <int S> __device__ __forceinline__ void load_row(f32x2 (&h)[S / 2], const float* p, int n0, int N, bool in) {
#pragma unroll
    for (int i = 0; i < S / 4; ++i) {
        const int n = n0 + 4 * i;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in) {
            if (N % 4 == 0) {
                if (n < N) v = *reinterpret_cast<const float4*>(p + n);
            } else {
                v = make_float4(n < N ? p[n] : 0.f, n + 1 < N ? p[n + 1] : 0.f, n + 2 < N ? p[n + 2] : 0.f,
                                n + 3 < N ? p[n + 3] : 0.f);
            }
        }
        h[2 * i] = pair(v.x, v.y);
        h[2 * i + 1] = pair(v.z, v.w);
    }
}
template <int S> __device__ __forceinline__ void store_row(const f32x2 (&h)[S / 2], float* p, int n0, int N, bool in) {
    if (!in) return;
#pragma unroll
    for (int i = 0; i < S / 4; ++i) {
        const int n = n0 + 4 * i;
        float4 v;
        unpair(h[2 * i], v.x, v.y);
        unpair(h[2 * i + 1], v.z, v.w);
        if (N % 4 == 0) {
            if (n < N) *reinterpret_cast<float4*>(p + n) = v;
        } else {
            if (n < N) p[n] = v.x;
            if (n + 1 < N) p[n + 1] = v.y;
            if (n + 2 < N) p[n + 2] = v.z;
            if (n + 3 < N) p[n + 3] = v.w;
        }
    }
}

// S states a lane, LPC lanes a channel: N <= S LPC.  The main pass; a range's own end, from
// zero; or, from its last token to its first, what the range adds to the gradient q that
// leaves it at its start: q <- exp(delta A) (q + gy C).
template <typename T, int S, int LPC, int MODE>
__global__ void __launch_bounds__(kWarps * 32) selscan_walk(const __grid_constant__ ScanParams p) {
    constexpr int kCh = 32 / LPC, NP = S * LPC, kVec = kTok * NP / 4, kPer = (kVec + 31) / 32;
    constexpr bool kExact = sizeof(T) == 4, SUMS = MODE != kScanMain, REV = MODE == kScanRevSums;
    __shared__ __align__(16) float sB[kWarps][2][kTok][NP];
    __shared__ __align__(16) float sC[SUMS ? 1 : kWarps][2][kTok][NP];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tpg = (p.cpg + kCh - 1) / kCh, tiles = tpg * p.G, ctas = (tiles + kWarps - 1) / kWarps;
    const int item = blockIdx.x / ctas, tile = (blockIdx.x - item * ctas) * kWarps + warp;
    if (tile >= tiles) return;
    const int grp = tile / tpg, ch = (tile - grp * tpg) * kCh + lane / LPC;
    const bool in = ch < p.cpg;
    const int d = grp * p.cpg + min(ch, p.cpg - 1), n0 = (lane % LPC) * S;
    if (!SUMS && item >= p.g.items) {            // rows of no sequence
        const int end = min(max(p.g.cu[p.g.nseq], 0), p.g.T);
        if (in && lane % LPC == 0)
            for (int64_t t = end + (item - p.g.items); t < p.g.T; t += kZeroItems)
                static_cast<T*>(p.y)[t * p.D + d] = from_f32<T>(0.f);
        return;
    }
    ScanItem it;
    if (!scan_find(p.g, item, it)) return;
    if (SUMS && (REV ? it.first : it.last)) return;   // nothing follows it
    const bool cut = p.g.R <= p.g.T;
    f32x2 h[S / 2], a2[S / 2];
    load_row<S>(a2, p.A + (int64_t)d * p.N, n0, p.N, true);
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
        float u, v;
        unpair(a2[i], u, v);
        a2[i] = pair(scan_rate(u), scan_rate(v));
        h[i] = pair(0.f, 0.f);
    }
    const int64_t row = ((int64_t)it.seq * p.D + d) * p.N;
    if (!SUMS) {
        if (cut && !(it.first && it.last)) load_row<S>(h, p.agg + ((int64_t)item * p.D + d) * p.N, n0, p.N, true);
        else if (p.init != nullptr) load_row<S>(h, p.init + row, n0, p.N, true);
    }
    const float bias = p.bias != nullptr ? p.bias[d] : 0.f, skip = p.Dk != nullptr ? p.Dk[d] : 0.f;
    // backwards, gy = dout silu(z) takes x's place and C takes B's
    const int64_t row0 = REV ? it.t0 + it.len - 1 : it.t0, dir = REV ? -1 : 1;
    const int64_t xs = dir * (REV ? p.D : p.xs), ts = dir * p.dts, zs = dir * p.zs, Bs = dir * (REV ? p.Cs : p.Bs);
    const T* xp = static_cast<const T*>(REV ? p.dout : p.x) + row0 * (REV ? p.D : p.xs) + d;
    const T* tp = static_cast<const T*>(p.dt) + row0 * p.dts + d;
    const bool gated = MODE != kScanSums && p.z != nullptr;
    const T* zp = gated ? static_cast<const T*>(p.z) + row0 * p.zs + d : nullptr;
    const T* Bp = static_cast<const T*>(REV ? p.C : p.B) + row0 * (REV ? p.Cs : p.Bs) + (int64_t)grp * p.N;
    const T* Cp = static_cast<const T*>(p.C) + row0 * p.Cs + (int64_t)grp * p.N;
    const bool vecB = (REV ? p.vecC : p.vecB) != 0;
    T* yp = static_cast<T*>(p.y) + (int64_t)it.t0 * p.D + d;

    T xr[kTok], tr[kTok], zr[kTok];
    Raw4<T> br[kPer], cr[kPer];
    auto prefetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = i * 32 + lane, t = t0 + v / (NP / 4), n = v % (NP / 4) * 4;
            const bool ok = (kVec % 32 == 0 || v < kVec) && t < it.len;
            fetch(br[i], Bp + t * Bs, ok ? n : p.N, p.N, vecB);
            if (!SUMS) fetch(cr[i], Cp + t * p.Cs, ok ? n : p.N, p.N, p.vecC != 0);
        }
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            const bool ok = t0 + t < it.len;
            const T zero = from_f32<T>(0.f);
            tr[t] = ok ? __ldg(tp + (t0 + t) * ts) : zero;
            xr[t] = ok ? __ldg(xp + (t0 + t) * xs) : zero;
            if (gated) zr[t] = ok ? __ldg(zp + (t0 + t) * zs) : zero;
        }
    };
    float total = 0.f;
    prefetch(0);
    for (int t0 = 0; t0 < it.len; t0 += kTok) {
        const int buf = (t0 / kTok) & 1;
        if (!SUMS && p.states != nullptr && (it.done + t0) % kScanChunk == 0)
            store_row<S>(h, p.states + ((int64_t)(it.row0 + (it.done + t0) / kScanChunk) * p.D + d) * p.N, n0, p.N, in);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = i * 32 + lane;
            if (kVec % 32 == 0 || v < kVec) {
                *reinterpret_cast<float4*>(&sB[warp][buf][0][0] + 4 * v) = widen(br[i]);
                if (!SUMS) *reinterpret_cast<float4*>(&sC[SUMS ? 0 : warp][buf][0][0] + 4 * v) = widen(cr[i]);
            }
        }
        __syncwarp();
        float delta[kTok], u[kTok], x[kTok], gate[kTok];
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            const float v = to_f32(tr[t]) + bias;
            // rows past the end multiply the state by 1 and add nothing
            delta[t] = t0 + t < it.len ? (p.softplus ? softplus<kExact>(v) : v) : 0.f;
            x[t] = to_f32(xr[t]);
            if (gated) {
                const float z = to_f32(zr[t]);
                gate[t] = z * sigmoid(z);
            }
            if (REV) u[t] = t0 + t < it.len ? (gated ? x[t] * gate[t] : x[t]) : 0.f;
            else u[t] = delta[t] * x[t];
            if (SUMS) total += delta[t];
        }
        if (t0 + kTok < it.len) prefetch(t0 + kTok);
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            const f32x2 dd = pair(delta[t], delta[t]), uu = pair(u[t], u[t]);
            f32x2 y0 = pair(0.f, 0.f), y1 = y0;
#pragma unroll
            for (int i = 0; i < S / 4; ++i) {
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&sB[warp][buf][t][n0 + 4 * i]);
                const f32x2 a0 = ex2_2(mul2(dd, a2[2 * i])), a1 = ex2_2(mul2(dd, a2[2 * i + 1]));
                if (REV) {
                    h[2 * i] = mul2(a0, fma2(uu, b.x, h[2 * i]));
                    h[2 * i + 1] = mul2(a1, fma2(uu, b.y, h[2 * i + 1]));
                } else {
                    h[2 * i] = fma2(a0, h[2 * i], mul2(uu, b.x));
                    h[2 * i + 1] = fma2(a1, h[2 * i + 1], mul2(uu, b.y));
                }
                if (!SUMS) {
                    const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&sC[SUMS ? 0 : warp][buf][t][n0 + 4 * i]);
                    y0 = fma2(c.x, h[2 * i], y0);
                    y1 = fma2(c.y, h[2 * i + 1], y1);
                }
            }
            if (!SUMS) {
                float lo, hi;
                unpair(add2(y0, y1), lo, hi);
                float y = lo + hi;
#pragma unroll
                for (int off = LPC / 2; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
                y = fmaf(skip, x[t], y);
                if (gated) y *= gate[t];
                if (in && lane % LPC == 0 && t0 + t < it.len) yp[(int64_t)(t0 + t) * p.D] = from_f32<T>(y);
            }
        }
    }
    if (SUMS) {
        store_row<S>(h, p.agg + ((int64_t)item * p.D + d) * p.N, n0, p.N, in);
        if (in && lane % LPC == 0) p.aggd[(int64_t)item * p.D + d] = total;
    } else if (p.fin != nullptr && it.last) {
        store_row<S>(h, p.fin + row, n0, p.N, in);
    }
}

// The states at the starts of a sequence's ranges, in place of the ranges' own ends:
// a thread for each state, the ranges in order, eight of them loaded ahead.  rev: from
// the last range to the first, the gradient that enters each at its end.
__global__ void __launch_bounds__(128) selscan_ranges(const __grid_constant__ ScanParams p, int rev) {
    const int64_t per = (int64_t)p.D * p.N, e = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (e >= per) return;
    const float rate = scan_rate(p.A[e]);
    const float* from = rev ? p.dfin : p.init;
    const int step = rev ? -1 : 1, d = (int)(e / p.N);
    for (int s = blockIdx.y; s < p.g.nseq; s += gridDim.y) {
        int lo, hi;
        scan_bounds(p.g, s, lo, hi);
        const int n = (int)((hi - lo + (int64_t)p.g.R - 1) / p.g.R);
        if (n <= 1) continue;
        float h = from != nullptr ? from[s * per + e] : 0.f;
        const int64_t first = scan_base(p.g, s) + (rev ? n - 1 : 0);
        constexpr int kAhead = 8;
        for (int c0 = 0; c0 < n; c0 += kAhead) {
            float end[kAhead], sum[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int64_t at = first + (int64_t)step * (c0 + i);
                const bool ok = c0 + i < n - 1;      // the last one's own end is not needed (nor made)
                end[i] = ok ? p.agg[at * per + e] : 0.f;
                sum[i] = ok ? p.aggd[at * p.D + d] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (c0 + i >= n) break;
                p.agg[(first + (int64_t)step * (c0 + i)) * per + e] = h;
                h = fmaf(ex2(rate * sum[i]), h, end[i]);
            }
        }
    }
}

template <typename T, int S, int LPC>
cudaError_t go(const ScanParams& p, ScanMode mode, cudaStream_t stream) {
    const int64_t tiles = (int64_t)((p.cpg + 32 / LPC - 1) / (32 / LPC)) * p.G, ctas = (tiles + kWarps - 1) / kWarps;
    const int64_t items = p.g.items + (mode == kScanMain && p.g.cu != nullptr ? kZeroItems : 0);
    if (items == 0) return cudaSuccess;
    auto k = mode == kScanMain ? selscan_walk<T, S, LPC, kScanMain>
           : mode == kScanSums ? selscan_walk<T, S, LPC, kScanSums> : selscan_walk<T, S, LPC, kScanRevSums>;
    k<<<(unsigned)(items * ctas), kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t by_states(const ScanParams& p, ScanMode mode, cudaStream_t stream) {
    if (p.N <= 4) return go<T, 4, 1>(p, mode, stream);
    if (p.N <= 8) return go<T, 8, 1>(p, mode, stream);
    if (p.N <= 16) return go<T, 16, 1>(p, mode, stream);
    if (p.N <= 32) return go<T, 16, 2>(p, mode, stream);
    return go<T, 16, 4>(p, mode, stream);
}

}  // namespace

cudaError_t launch_selscan_fwd(const ScanParams& p, int dtype, ScanMode mode, cudaStream_t stream) {
    return dtype == SSD_BF16 ? by_states<__nv_bfloat16>(p, mode, stream) : by_states<float>(p, mode, stream);
}

cudaError_t launch_selscan_ranges(const ScanParams& p, int rev, cudaStream_t stream) {
    if (p.g.nseq == 0) return cudaSuccess;
    const dim3 grid((unsigned)(((int64_t)p.D * p.N + 127) / 128), (unsigned)(p.g.nseq < 65535 ? p.g.nseq : 65535));
    selscan_ranges<<<grid, 128, 0, stream>>>(p, rev);
    return cudaGetLastError();
}

}  // namespace ssd
