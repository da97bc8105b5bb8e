// selscan_bwd.cu -- the gradient of the selective scan over packed sequences.
//
// With gy = dout silu(z), from the last token to the first:
//     r = q + gy C;  u = sum_n r B;  w = r a h_{t-1};  q = a r          (a = exp(delta A))
//     dx = delta u + D gy    ddelta = x u + sum_n A w    dA += delta w
//     dB = sum over channels of delta x r                dC = sum over channels of gy h
// A range of a sequence is walked backwards in chunks of 32 tokens, from the states that
// the forward pass stored.  In a chunk the states are made forwards once and kept every
// K tokens (in shared memory); then, slab of K tokens by slab from the last one, the
// decays a and the products a h_{t-1} are made again and kept in registers while the
// slab is walked backwards.
//
// A lane holds C channels x S states and a warp 8 C channels x 4 S states, because two
// sums cross lanes: over the states (4 lanes) for dx, ddelta and y, and over the
// channels (8 lanes, then the CTA's warps, then a kernel of its own over the tiles) for
// dB and dC.  Each is a butterfly that halves the values with every step, so that a
// token costs 2 S - 1 shuffles and 3 C / 2 more.
#include <type_traits>

#include "selscan.cuh"

namespace ssd {
namespace {

constexpr int kChunk = kScanChunk;

template <int S> struct Plan {                 // N <= 4 S
    static constexpr int C = S <= 4 ? 2 : 1;   // channels a lane
    static constexpr int K = S <= 8 ? 8 : 4;   // tokens of a slab
    static constexpr int kWarps = S <= 8 ? 4 : 2;
    static constexpr int kCh = 8 * C;          // channels of a warp
    static constexpr int NP = 4 * S;
    static constexpr int kSlabs = kChunk / K;
    // shared memory, in floats
    static constexpr int kBC = 2 * kChunk * NP;                  // B and C, for all warps
    static constexpr int kDu = kChunk * kCh * 2;                 // (delta, u) of each token and channel
    static constexpr int kGy = kChunk * kCh;
    static constexpr int kStart = (kSlabs - 1) * C * S * 32;     // the state before each slab but the first
    static constexpr int kDbc = kChunk * 2 * NP;                 // the warp's terms of dB and dC
    static constexpr int kRed = 3 * K * kCh;                     // u, sum A w and C.h of a slab
    static constexpr int kWarp = kDu + kGy + kStart + kDbc + kRed;
    static constexpr int kBytes = (kBC + kWarps * kWarp) * 4;
};

// Four channels of a row.
__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}
__device__ __forceinline__ void spread(float4 v, float (&o)[4]) { o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w; }

template <int S> __device__ __forceinline__ void load_states_row(f32x2 (&h)[S / 2], const float* p, int n0, int N, bool in) {
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
        const int n = n0 + 2 * i;
        if (N % 2 == 0) {
            h[i] = in && n < N ? *reinterpret_cast<const f32x2*>(p + n) : 0ull;
        } else {
            h[i] = pair(in && n < N ? p[n] : 0.f, in && n + 1 < N ? p[n + 1] : 0.f);
        }
    }
}
template <int S> __device__ __forceinline__ void store_states_row(const f32x2 (&h)[S / 2], float* p, int n0, int N, bool in) {
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
        const int n = n0 + 2 * i;
        if (N % 2 == 0) {
            if (in && n < N) *reinterpret_cast<f32x2*>(p + n) = h[i];
        } else {
            float a, b;
            unpair(h[i], a, b);
            if (in && n < N) p[n] = a;
            if (in && n + 1 < N) p[n + 1] = b;
        }
    }
}
// S consecutive floats of shared memory as pairs
template <int S> __device__ __forceinline__ void lds(f32x2 (&v)[S / 2], const float* p) {
    if (S == 2) {
        v[0] = *reinterpret_cast<const f32x2*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < S / 4; ++i) {
            const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(p + 4 * i);
            v[2 * i] = t.x;
            v[(2 * i + 1) % (S / 2)] = t.y;
        }
    }
}

template <typename T, int S>
__global__ void __launch_bounds__(Plan<S>::kWarps * 32) selscan_bwd(const __grid_constant__ ScanParams p) {
    using P = Plan<S>;
    constexpr int C = P::C, K = P::K, kCh = P::kCh, NP = P::NP, H = S / 2;
    constexpr bool kExact = sizeof(T) == 4;
    extern __shared__ __align__(16) float smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q4 = lane & 3;
    float* sB = smem;                                  // [kChunk][NP]
    float* sC = sB + kChunk * NP;
    float* sDu = smem + P::kBC + warp * P::kWarp;      // [kChunk][kCh][2]
    float* sGy = sDu + P::kDu;                         // [kChunk][kCh]
    float* sStart = sGy + P::kGy;                      // [slab - 1][C S][32]
    float* sDbc = sStart + P::kStart;                  // [kChunk][2][NP]
    float* sRed = sDbc + P::kDbc;                      // u, v, y: [K][kCh] each

    constexpr int kTile = P::kWarps * kCh;
    const int tpg = (p.cpg + kTile - 1) / kTile, tiles = tpg * p.G;
    const int slot = blockIdx.x / tiles, tile = blockIdx.x - slot * tiles;
    const int grp = tile / tpg, tg = tile - grp * tpg;
    const int c0 = tg * kTile + warp * kCh;            // the warp's first channel in the group
    const int n0 = q4 * S;
    // element-wise work: a quad of channels of one row a lane
    constexpr int kQuads = kCh / 4, kRows = 32 / kQuads;
    const int er = lane / kQuads, ec = lane % kQuads * 4;
    const bool ein = c0 + ec < p.cpg;
    const int64_t ed = (int64_t)grp * p.cpg + c0 + ec;

    if (slot >= p.slots) {                             // rows of no sequence
        const int end = min(max(p.g.cu[p.g.nseq], 0), p.g.T), step = gridDim.x / tiles - p.slots;
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        if (ein)
            for (int64_t t = end + (int64_t)(slot - p.slots) * kRows + er; t < p.g.T; t += (int64_t)step * kRows) {
                store4(static_cast<T*>(p.dx) + t * p.D + ed, zero);
                store4(static_cast<T*>(p.ddt) + t * p.D + ed, zero);
                if (p.z != nullptr) store4(static_cast<T*>(p.dz) + t * p.D + ed, zero);
            }
        return;
    }
    int64_t dch[C];
    bool in[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        in[c] = c0 + g * C + c < p.cpg;
        dch[c] = (int64_t)grp * p.cpg + c0 + g * C + c;
    }
    f32x2 dA[C][H], qv[C][H], a2[C][H];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < H; ++i) dA[c][i] = 0ull;
    float dD[4] = {0.f, 0.f, 0.f, 0.f}, db[4] = {0.f, 0.f, 0.f, 0.f};
    float bias[4] = {0.f, 0.f, 0.f, 0.f}, skip[4] = {0.f, 0.f, 0.f, 0.f};
    if (ein) {
        if (p.bias != nullptr) spread(load4(p.bias + ed), bias);
        if (p.Dk != nullptr) spread(load4(p.Dk + ed), skip);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        load_states_row<S>(a2[c], p.A + dch[c] * p.N, n0, p.N, in[c]);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            float a, b;
            unpair(a2[c][i], a, b);
            a2[c][i] = pair(scan_rate(a), scan_rate(b));
        }
    }
    const bool cut = p.g.R <= p.g.T, gated = p.z != nullptr;
    for (int item = slot * p.per_slot; item < min((slot + 1) * p.per_slot, p.g.items); ++item) {
        ScanItem it;
        if (!scan_find(p.g, item, it)) continue;
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int i = 0; i < H; ++i) qv[c][i] = 0ull;
            if (cut && !(it.first && it.last))
                load_states_row<S>(qv[c], p.agg + ((int64_t)item * p.D + dch[c]) * p.N, n0, p.N, in[c]);
            else if (p.dfin != nullptr)
                load_states_row<S>(qv[c], p.dfin + ((int64_t)it.seq * p.D + dch[c]) * p.N, n0, p.N, in[c]);
        }
        const T* x = static_cast<const T*>(p.x) + it.t0 * p.xs + ed;
        const T* dt = static_cast<const T*>(p.dt) + it.t0 * p.dts + ed;
        const T* z = static_cast<const T*>(p.z) + it.t0 * p.zs + ed;
        const T* dout = static_cast<const T*>(p.dout) + (int64_t)it.t0 * p.D + ed;
        for (int chunk = (it.len - 1) / kChunk; chunk >= 0 && it.len > 0; --chunk) {
            const int t0 = chunk * kChunk, nt = min(kChunk, it.len - t0);
            // B and C of the chunk, 0 behind the range's end
            for (int i = threadIdx.x; i < kChunk * NP / 4; i += P::kWarps * 32) {
                const int t = i / (NP / 4), n = i % (NP / 4) * 4;
                const int64_t row = (int64_t)it.t0 + t0 + t;
                const int from = t < nt ? n : p.N;
                *reinterpret_cast<float4*>(sB + 4 * i) =
                    load_states(static_cast<const T*>(p.B) + row * p.Bs + (int64_t)grp * p.N, from, p.N, p.vecB != 0);
                *reinterpret_cast<float4*>(sC + 4 * i) =
                    load_states(static_cast<const T*>(p.C) + row * p.Cs + (int64_t)grp * p.N, from, p.N, p.vecC != 0);
            }
            for (int r0 = 0; r0 < kChunk; r0 += kRows) {
                const int t = r0 + er;
                float du[8], gy[4];
                if (ein && t < nt) {
                    float xv[4], tv[4], gv[4], zv[4];
                    spread(load4(x + (int64_t)(t0 + t) * p.xs), xv);
                    spread(load4(dt + (int64_t)(t0 + t) * p.dts), tv);
                    spread(load4(dout + (int64_t)(t0 + t) * p.D), gv);
                    if (gated) spread(load4(z + (int64_t)(t0 + t) * p.zs), zv);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float v = tv[i] + bias[i], delta = p.softplus ? softplus<kExact>(v) : v;
                        du[2 * i] = delta;
                        du[2 * i + 1] = delta * xv[i];
                        gy[i] = gated ? gv[i] * zv[i] * sigmoid(zv[i]) : gv[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) du[2 * i] = du[2 * i + 1] = gy[i] = 0.f;
                }
                *reinterpret_cast<float4*>(sDu + (t * kCh + ec) * 2) = make_float4(du[0], du[1], du[2], du[3]);
                *reinterpret_cast<float4*>(sDu + (t * kCh + ec) * 2 + 4) = make_float4(du[4], du[5], du[6], du[7]);
                *reinterpret_cast<float4*>(sGy + t * kCh + ec) = make_float4(gy[0], gy[1], gy[2], gy[3]);
            }
            __syncthreads();
            // delta and u (and gy) of the lane's channels for a token
            auto channel = [&](int t, f32x2 (&dd)[C], f32x2 (&uu)[C]) {
                if (C == 2) {
                    const float4 v = *reinterpret_cast<const float4*>(sDu + (t * kCh + g * 2) * 2);
                    dd[0] = pair(v.x, v.x); uu[0] = pair(v.y, v.y);
                    dd[C - 1] = pair(v.z, v.z); uu[C - 1] = pair(v.w, v.w);
                } else {
                    const float2 v = *reinterpret_cast<const float2*>(sDu + (t * kCh + g) * 2);
                    dd[0] = pair(v.x, v.x); uu[0] = pair(v.y, v.y);
                }
            };
            const int slabs = (nt + K - 1) / K;
            f32x2 h[C][H];
            {
                const int64_t at = it.row0 + (it.done + t0) / kChunk;
#pragma unroll
                for (int c = 0; c < C; ++c)
                    load_states_row<S>(h[c], p.states + (at * p.D + dch[c]) * p.N, n0, p.N, in[c]);
            }
            f32x2 first[C][H];
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < H; ++i) first[c][i] = h[c][i];
            for (int sl = 0; sl + 1 < slabs; ++sl) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int t = sl * K + k;
                    f32x2 dd[C], uu[C], B[H];
                    channel(t, dd, uu);
                    lds<S>(B, sB + t * NP + n0);
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int i = 0; i < H; ++i)
                            h[c][i] = fma2(ex2_2(mul2(dd[c], a2[c][i])), h[c][i], mul2(uu[c], B[i]));
                }
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < H; ++i)
                        *reinterpret_cast<f32x2*>(sStart + ((sl * C + c) * H + i) * 64 + lane * 2) = h[c][i];
            }
            for (int sl = slabs - 1; sl >= 0; --sl) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < H; ++i)
                        h[c][i] = sl == 0 ? first[c][i]
                                          : *reinterpret_cast<const f32x2*>(sStart + (((sl - 1) * C + c) * H + i) * 64 + lane * 2);
                f32x2 a[K][C][H], ah[K][C][H];
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int t = sl * K + k;
                    f32x2 dd[C], uu[C], B[H], Cv[H];
                    channel(t, dd, uu);
                    lds<S>(B, sB + t * NP + n0);
                    if (gated) lds<S>(Cv, sC + t * NP + n0);
                    float y[C];
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        f32x2 ys = 0ull;
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            a[k][c][i] = ex2_2(mul2(dd[c], a2[c][i]));
                            ah[k][c][i] = mul2(a[k][c][i], h[c][i]);
                            h[c][i] = fma2(uu[c], B[i], ah[k][c][i]);
                            if (gated) ys = fma2(Cv[i], h[c][i], ys);
                        }
                        float lo, hi;
                        unpair(ys, lo, hi);
                        y[c] = lo + hi;
                    }
                    if (gated) {                       // only dz needs y
                        halve<C>(y, lane, 2);
                        halve<1>(y, lane, 1);
                        if ((lane & 1) == 0 && (C == 2 || q4 == 0))
                            sRed[(2 * K + k) * kCh + g * C + (C == 2 ? q4 >> 1 : 0)] = y[0];
                    }
                }
#pragma unroll
                for (int k = K - 1; k >= 0; --k) {
                    const int t = sl * K + k;
                    f32x2 dd[C], uu[C], B[H], Cv[H];
                    channel(t, dd, uu);
                    lds<S>(B, sB + t * NP + n0);
                    lds<S>(Cv, sC + t * NP + n0);
                    f32x2 dB[H], dC[H];
                    float red[2 * C];
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const float gyv = sGy[t * kCh + g * C + c];
                        const f32x2 gg = pair(gyv, gyv);
                        f32x2 us = 0ull, vs = 0ull;
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            const f32x2 r = fma2(gg, Cv[i], qv[c][i]), hh = fma2(uu[c], B[i], ah[k][c][i]);
                            dC[i] = c == 0 ? mul2(gg, hh) : fma2(gg, hh, dC[i]);
                            dB[i] = c == 0 ? mul2(uu[c], r) : fma2(uu[c], r, dB[i]);
                            us = fma2(r, B[i], us);
                            const f32x2 w = mul2(r, ah[k][c][i]);
                            vs = fma2(w, a2[c][i], vs);
                            dA[c][i] = fma2(dd[c], w, dA[c][i]);
                            qv[c][i] = mul2(a[k][c][i], r);
                        }
                        float lo, hi;
                        unpair(us, lo, hi);
                        red[c] = lo + hi;
                        unpair(vs, lo, hi);
                        red[C + c] = lo + hi;
                    }
                    halve<2 * C>(red, lane, 2);
                    halve<C>(red, lane, 1);            // u of channel 0, 1, sum A w of 0, 1 (C = 1: u, u, ..)
                    if (C == 2 || (lane & 1) == 0)
                        sRed[((q4 >> 1) * K + k) * kCh + g * C + (C == 2 ? q4 & 1 : 0)] = red[0];
                    float bc[2 * S];
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        unpair(dB[i], bc[2 * i], bc[2 * i + 1]);
                        unpair(dC[i], bc[S + 2 * i], bc[S + 2 * i + 1]);
                    }
                    halve<2 * S>(bc, lane, 16);
                    halve<S>(bc, lane, 8);
                    halve<S / 2>(bc, lane, 4);
                    // value g of 2 S / 8 each; with S = 2 lanes differing in bit 2 hold the same
                    constexpr int kLeft = S >= 4 ? S / 4 : 1;
                    if (S >= 4 || (lane & 4) == 0)
#pragma unroll
                        for (int i = 0; i < kLeft; ++i) {
                            const int v = S >= 4 ? g * kLeft + i : g >> 1;     // 0 .. S - 1: dB, then dC
                            sDbc[(t * 2 + v / S) * NP + n0 + v % S] = bc[i];
                        }
                }
                __syncwarp();
                if (er < K && sl * K + er < nt && ein) {
                    const int t = sl * K + er;
                    float xv[4], tv[4], gv[4], zv[4], us[4], vs[4], ys[4], ox[4], ot[4], oz[4];
                    spread(load4(x + (int64_t)(t0 + t) * p.xs), xv);
                    spread(load4(dt + (int64_t)(t0 + t) * p.dts), tv);
                    spread(load4(dout + (int64_t)(t0 + t) * p.D), gv);
                    if (gated) spread(load4(z + (int64_t)(t0 + t) * p.zs), zv);
                    spread(*reinterpret_cast<const float4*>(sRed + er * kCh + ec), us);
                    spread(*reinterpret_cast<const float4*>(sRed + (K + er) * kCh + ec), vs);
                    if (gated) spread(*reinterpret_cast<const float4*>(sRed + (2 * K + er) * kCh + ec), ys);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float delta = sDu[(t * kCh + ec + i) * 2], gy = sGy[t * kCh + ec + i];
                        ox[i] = fmaf(delta, us[i], skip[i] * gy);
                        const float dd = fmaf(xv[i], us[i], vs[i] * 0.69314718055994531f);   // A = a2 ln 2
                        ot[i] = p.softplus ? dd * softplus_grad<kExact>(tv[i] + bias[i]) : dd;
                        if (gated) {
                            const float sg = sigmoid(zv[i]);
                            oz[i] = gv[i] * fmaf(skip[i], xv[i], ys[i]) * sg * fmaf(zv[i], 1.f - sg, 1.f);
                        }
                        dD[i] = fmaf(gy, xv[i], dD[i]);
                        db[i] += ot[i];
                    }
                    const int64_t row = (int64_t)it.t0 + t0 + t;
                    store4(static_cast<T*>(p.dx) + row * p.D + ed, ox);
                    store4(static_cast<T*>(p.ddt) + row * p.D + ed, ot);
                    if (gated) store4(static_cast<T*>(p.dz) + row * p.D + ed, oz);
                }
                __syncwarp();
            }
            __syncthreads();
            // the CTA's terms of dB and dC: its warps' added in order
            for (int i = threadIdx.x; i < nt * 2 * NP; i += P::kWarps * 32) {
                const int t = i / (2 * NP), v = i % (2 * NP), n = v % NP;
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < P::kWarps; ++w) s += smem[P::kBC + w * P::kWarp + P::kDu + P::kGy + P::kStart + i];
                if (n < p.N)
                    p.part[((((int64_t)tg * p.g.T + it.t0 + t0 + t) * p.G + grp) * 2 + v / NP) * p.N + n] = s;
            }
        }
        if (it.first && p.dinit != nullptr)
#pragma unroll
            for (int c = 0; c < C; ++c)
                store_states_row<S>(qv[c], p.dinit + ((int64_t)it.seq * p.D + dch[c]) * p.N, n0, p.N, in[c]);
    }
    // the slot's terms of dA, dD and dbias
#pragma unroll
    for (int c = 0; c < C; ++c)
        store_states_row<S>(dA[c], p.partA + ((int64_t)slot * p.D + dch[c]) * p.N, n0, p.N, in[c]);
#pragma unroll
    for (int bit = kQuads; bit < 32; bit *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dD[i] += __shfl_xor_sync(0xffffffffu, dD[i], bit);
            db[i] += __shfl_xor_sync(0xffffffffu, db[i], bit);
        }
    if (er == 0 && ein) {
        store4(p.partD + (int64_t)slot * 2 * p.D + ed, dD);
        store4(p.partD + ((int64_t)slot * 2 + 1) * p.D + ed, db);
    }
}

// dB and dC: the tiles' terms in order; 0 in rows of no sequence.
template <typename T>
__global__ void __launch_bounds__(256) selscan_sum_bc(const __grid_constant__ ScanParams p, int tpg) {
    const int64_t per = (int64_t)p.g.T * p.G * 2 * p.N, e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= per) return;
    const int n = (int)(e % p.N), kind = (int)(e / p.N % 2);
    const int64_t tg = e / (2 * p.N);                  // t G + g
    const int end = p.g.cu != nullptr ? min(max(p.g.cu[p.g.nseq], 0), p.g.T) : p.g.T;
    float s = 0.f;
    if (tg / p.G < end)
        for (int i = 0; i < tpg; ++i) s += p.part[i * per + e];
    static_cast<T*>(kind == 0 ? p.dB : p.dC)[tg * p.N + n] = from_f32<T>(s);
}

// dA, dD and dbias: the slots' terms in order.
__global__ void __launch_bounds__(128) selscan_sum_a(const __grid_constant__ ScanParams p) {
    const int64_t na = (int64_t)p.D * p.N, e = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (e >= na + 2 * p.D) return;
    const float* at = e < na ? p.partA + e : p.partD + (e - na);
    const int64_t step = e < na ? na : 2 * (int64_t)p.D;
    float s = 0.f;
    int i = 0;
    for (; i + 8 <= p.slots; i += 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = at[(i + j) * step];
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[j];
    }
    for (; i < p.slots; ++i) s += at[i * step];
    if (e < na) p.dA[e] = s;
    else if (e < na + p.D) { if (p.dD != nullptr) p.dD[e - na] = s; }
    else if (p.dbias != nullptr) p.dbias[e - na - p.D] = s;
}

template <typename T, int S> cudaError_t go(const ScanParams& p, cudaStream_t stream) {
    using P = Plan<S>;
    constexpr int kTile = P::kWarps * P::kCh;
    const int tpg = (p.cpg + kTile - 1) / kTile;
    const int64_t slots = p.slots + (p.g.cu != nullptr ? 16 : 0);
    if (slots > 0) {
        const cudaError_t e = cudaFuncSetAttribute(selscan_bwd<T, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kBytes);
        if (e != cudaSuccess) return e;
        selscan_bwd<T, S><<<(unsigned)(slots * tpg * p.G), P::kWarps * 32, P::kBytes, stream>>>(p);
        const cudaError_t l = cudaGetLastError();
        if (l != cudaSuccess) return l;
    }
    const int64_t per = (int64_t)p.g.T * p.G * 2 * p.N;
    if (per > 0) selscan_sum_bc<T><<<(unsigned)((per + 255) / 256), 256, 0, stream>>>(p, tpg);
    selscan_sum_a<<<(unsigned)(((int64_t)p.D * (p.N + 2) + 127) / 128), 128, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t by_states(const ScanParams& p, cudaStream_t stream) {
    if (p.N <= 8) return go<T, 2>(p, stream);
    if (p.N <= 16) return go<T, 4>(p, stream);
    if (p.N <= 32) return go<T, 8>(p, stream);
    return go<T, 16>(p, stream);
}

}  // namespace

int selscan_bwd_channels(int N) { return N <= 16 ? 64 : N <= 32 ? 32 : 16; }

cudaError_t launch_selscan_bwd(const ScanParams& p, int dtype, cudaStream_t stream) {
    return dtype == SSD_BF16 ? by_states<__nv_bfloat16>(p, stream) : by_states<float>(p, stream);
}

}  // namespace ssd
