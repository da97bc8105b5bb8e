// selscan_bwd.cu -- the gradient of the selective scan over packed sequences.
//
// With gy = dout silu(z), from the last token to the first:
//     r = q + gy C;  u = sum_n r B;  w = r a h_{t-1};  q = a r          (a = exp(delta A))
//     dx = delta u + D gy    ddelta = x u + sum_n A w    dA += delta w
//     dB = sum over channels of delta x r                dC = sum over channels of gy h
// A range of a sequence is walked backwards in chunks of 16 tokens, from the states that
// the forward pass stored.  In a chunk the states are made forwards once and kept every
// K tokens (in shared memory); then, slab of K tokens by slab from the last one, the
// decays a and the products a h_{t-1} are made again and kept in registers while the
// slab is walked backwards.  A chunk's rows of x, dt, dout and z and its stored state
// come by cp.async while the chunk behind it is computed.
//
// A lane holds C channels x S states and a warp 8 C channels x 4 S states.  Two sums
// cross lanes, both in fp32 by shuffles that halve the values a lane keeps at each step.  Over the
// states (the 4 lanes of a row, for dx, ddelta and y): of a slab's four tokens each lane ends with
// the sums of one, whose outputs it makes.  Over the channels (for dB and dC): the 8 rows, then the CTA's
// warps, then a kernel of its own over the tiles.  As products of the tensor cores with ones the sums
// over states took 502 us (terms cut to 11 bits, three of each, so that they keep all of theirs) and 493 (two; one for y) instead
// of 457, and leaned to 0, by 4e-8 to 8e-8 of ddt_bias: those sums are not rounded to nearest.  The sums
// over channels on the tensor cores took 6 % less of the call, cut to 11 bits: a token whose
// channels cancel was off by more than the rounding of its sum.
//
// What bounds it: the registers (243 for 16 states) leave two warps a quarter-SM, which issue in half of the
// clocks and wait for their own last results; a token costs a warp of 16 channels 212 instructions.  8192
// tokens of 2048 channels in 6 sequences: 466 us a call, 361 of them this kernel.  Tried with the tensor cores'
// sums over states and channels, against 463 (454 to 511 for the older ones): no cut into ranges 670; rows
// loaded where they are used 617; pairs of channels instead of states, or delta and u stored in
// pairs: 539, 509; slabs of 2 tokens 485, of 8 tokens 646; more warps an SM, which the
// compiler's spills cost more than they bring: CTAs of 3 warps, three an SM 608, of 2 warps, four
// 472, five 607.
#include <type_traits>

#include "selscan.cuh"
#include "sm100_ptx.cuh"

namespace ssd {
namespace {

constexpr int kChunk = kScanChunk;
static_assert(kChunk == kMakeUp, "a chunk is what make_up is for");

template <typename T, int S> struct Plan {     // N <= 4 S
    static constexpr int C = S <= 4 ? 2 : 1;   // channels a lane
    static constexpr int K = S <= 8 ? 4 : 2;   // tokens of a slab
    static constexpr int kWarps = S <= 8 ? 4 : 2;
    static constexpr int kCh = 8 * C;          // channels of a warp
    static constexpr int NP = 4 * S;
    static constexpr int kSlabs = kChunk / K;
    struct Warp {                              // shared memory of a warp
        T raw[2][4][kChunk][kCh];              // x, dt, dout and z of a chunk and the next
        float check[2][C * S * 32];            // the stored states, as the lanes hold them
        float start[kSlabs - 1][C * S * 32];   // the state before each slab but the first
        // (rows padded so that lanes that write different rows meet different banks)
        float du[kChunk][2 * kCh + 8];         // delta and u = delta x of each channel
        float gy[kChunk][kCh + 8];
        float dbc[kChunk][2 * NP + 4];         // the warp's terms of dB and dC
    };
    struct Cta {
        float bc[2][kChunk][NP];               // B and C
        Warp w[kWarps];
    };
};

// The sums over the four lanes of a row of K tokens' values of C channels, in fp32: lane q gets
// those of token q % K, in v[0] (and v[1]).
template <int K, int C> __device__ __forceinline__ void sum_row(float (&v)[K * C], int lane) {
    if (K == 4) {
        halve<K * C>(v, lane, 2);
        halve<K * C / 2>(v, lane, 1);
    } else {
        halve<K * C>(v, lane, 1);
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] += __shfl_xor_sync(0xffffffffu, v[c], 2);
    }
}

// Four channels of a row, zeros.
__device__ __forceinline__ void zero4(float* p) { *reinterpret_cast<float4*>(p) = make_float4(0.f, 0.f, 0.f, 0.f); }
__device__ __forceinline__ void zero4(__nv_bfloat16* p) { *reinterpret_cast<uint2*>(p) = make_uint2(0u, 0u); }
// Two channels of a row.
__device__ __forceinline__ f32x2 load2(const float* p) { return *reinterpret_cast<const unsigned long long*>(p); }
__device__ __forceinline__ f32x2 load2(const __nv_bfloat16* p) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
    return pair(v << 16, v & 0xFFFF0000u);
}
__device__ __forceinline__ void store2(float* p, f32x2 v) { *reinterpret_cast<f32x2*>(p) = v; }
__device__ __forceinline__ void store2(__nv_bfloat16* p, f32x2 v) { *reinterpret_cast<uint32_t*>(p) = pack2(v); }
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_8(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

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
// The S states of lane q of a row of B or C as pairs.  Vector i of four of lane q lies at 4 i + q: so
// the four lanes read other banks (64 states of 8192 tokens and 2048 channels: 1.01 times as fast as each lane's own side by side).
template <int S> __device__ __forceinline__ void lds(f32x2 (&v)[S / 2], const float* row, int q) {
    if (S == 2) {
        v[0] = *reinterpret_cast<const f32x2*>(row + 2 * q);
    } else {
#pragma unroll
        for (int i = 0; i < S / 4; ++i) {
            const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(row + 4 * (4 * i + q));
            v[2 * i] = t.x;
            v[(2 * i + 1) % (S / 2)] = t.y;
        }
    }
}

template <typename T, int S>
__global__ void __launch_bounds__(Plan<T, S>::kWarps * 32, S <= 4 ? 2 : 1) selscan_bwd(const __grid_constant__ ScanParams p) {
    using P = Plan<T, S>;
    constexpr int C = P::C, K = P::K, kCh = P::kCh, NP = P::NP, H = S / 2, kThreads = P::kWarps * 32;
    constexpr bool kExact = sizeof(T) == 4;
    extern __shared__ __align__(16) unsigned char smem[];
    typename P::Cta& sh = *reinterpret_cast<typename P::Cta*>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q4 = lane & 3;
    typename P::Warp& w = sh.w[warp];

    constexpr int kTile = P::kWarps * kCh;
    const int tpg = (p.cpg + kTile - 1) / kTile, tiles = tpg * p.G;
    const int slot = blockIdx.x / tiles, tile = blockIdx.x - slot * tiles;
    const int grp = tile / tpg, tg = tile - grp * tpg;
    const int c0 = tg * kTile + warp * kCh;            // the warp's first channel in the group
    const int n0 = q4 * S;
    if (slot >= p.slots) {                             // rows of no sequence
        constexpr int kQuads = kCh / 4, kRows = 32 / kQuads;
        const int end = min(max(p.g.cu[p.g.nseq], 0), p.g.T), step = gridDim.x / tiles - p.slots, ch = c0 + lane % kQuads * 4;
        if (ch < p.cpg)
            for (int64_t t = end + (int64_t)(slot - p.slots) * kRows + lane / kQuads; t < p.g.T; t += (int64_t)step * kRows) {
                const int64_t at = t * p.D + (int64_t)grp * p.cpg + ch;
                zero4(static_cast<T*>(p.dx) + at);
                zero4(static_cast<T*>(p.ddt) + at);
                if (p.z != nullptr) zero4(static_cast<T*>(p.dz) + at);
            }
        return;
    }
    // A lane's channels are all in the group or none (groups and C are even).
    const bool in = c0 + g * C < p.cpg;
    const int64_t dch = (int64_t)grp * p.cpg + (in ? c0 + g * C : 0);
    f32x2 dA[C][H], qv[C][H], a2[C][H];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        load_states_row<S>(a2[c], p.A + (dch + c) * p.N, n0, p.N, in);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            float a, b;
            unpair(a2[c][i], a, b);
            a2[c][i] = pair(scan_rate(a), scan_rate(b));
            dA[c][i] = 0ull;
        }
    }
    auto per_channel = [&](const float* v) { return v != nullptr ? pair(v[dch], v[dch + C - 1]) : 0ull; };
    const f32x2 bias = per_channel(p.bias), skip = per_channel(p.Dk);
    f32x2 dD = 0ull, db = 0ull;
    const bool cut = p.g.R <= p.g.T, gated = p.z != nullptr;
    for (int item = slot * p.per_slot; item < min((slot + 1) * p.per_slot, p.g.items); ++item) {
        ScanItem it;
        if (!scan_find(p.g, item, it)) continue;
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int i = 0; i < H; ++i) qv[c][i] = 0ull;
            if (cut && !(it.first && it.last))
                load_states_row<S>(qv[c], p.agg + ((int64_t)item * p.D + dch + c) * p.N, n0, p.N, in);
            else if (p.dfin != nullptr)
                load_states_row<S>(qv[c], p.dfin + ((int64_t)it.seq * p.D + dch + c) * p.N, n0, p.N, in);
        }
        // A chunk's rows of x, dt, dout and z and its stored state, zeros behind the range's end.
        auto copy = [&](int chunk, int buf) {
            const int nt = min(kChunk, it.len - chunk * kChunk);
            const int64_t row0 = it.t0 + (int64_t)chunk * kChunk;
            constexpr int kPieces = kCh * (int)sizeof(T), kRow = kPieces / kChunk;     // 16-byte pieces: all, of a row
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const T* base = static_cast<const T*>(k == 0 ? p.x : k == 1 ? p.dt : k == 2 ? p.dout : p.z);
                const int64_t stride = k == 0 ? p.xs : k == 1 ? p.dts : k == 2 ? p.D : p.zs;
                if (k == 3 && !gated) break;
#pragma unroll
                for (int v = 0; v < kPieces; v += 32) {
                    const int r = (v + lane) / kRow, c = (v + lane) % kRow * (16 / (int)sizeof(T));
                    const bool ok = r < nt && c0 + c < p.cpg;
                    const T* from = ok ? base + (row0 + r) * stride + (int64_t)grp * p.cpg + c0 + c : base;
                    if (v + 32 <= kPieces || v + lane < kPieces)
                        cp_async_16(smem_u32(&w.raw[buf][k][0][0]) + 16 * (v + lane), from, ok ? 16u : 0u);
                }
            }
            const float* st = p.states + ((it.row0 + it.done / kChunk + chunk) * (int64_t)p.D + dch) * p.N;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const int n = n0 + 2 * i;
                    const float* from = st + (int64_t)c * p.N + n;
                    const uint32_t to = smem_u32(&w.check[buf][(c * H + i) * 64 + lane * 2]);
                    if (p.N % 2 == 0) {
                        cp_async_8(to, in && n < p.N ? from : p.states, in && n < p.N ? 8u : 0u);
                    } else {
                        cp_async_4(to, in && n < p.N ? from : p.states, in && n < p.N ? 4u : 0u);
                        cp_async_4(to + 4, in && n + 1 < p.N ? from + 1 : p.states, in && n + 1 < p.N ? 4u : 0u);
                    }
                }
        };
        // B's and C's rows of the next chunk wait in registers.
        constexpr int kVec = kChunk * NP / 4, kPer = (2 * kVec + kThreads - 1) / kThreads;
        Raw4<T> bc[kPer];
        auto prefetch = [&](int chunk) {
            const int nt = min(kChunk, it.len - chunk * kChunk);
            const int64_t row0 = it.t0 + (int64_t)chunk * kChunk;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int v = i * kThreads + threadIdx.x, m = v % kVec, t = m / (NP / 4), n = m % (NP / 4) * 4;
                const bool ok = v < 2 * kVec && t < nt;
                if (v < kVec) fetch(bc[i], static_cast<const T*>(p.B) + (row0 + t) * p.Bs + (int64_t)grp * p.N, ok ? n : p.N, p.N, p.vecB != 0);
                else fetch(bc[i], static_cast<const T*>(p.C) + (row0 + t) * p.Cs + (int64_t)grp * p.N, ok ? n : p.N, p.N, p.vecC != 0);
            }
        };
        const int chunks = (it.len + kChunk - 1) / kChunk;
        if (chunks > 0) {
            copy(chunks - 1, 0);
            prefetch(chunks - 1);
        }
        cp_async_commit();
        for (int chunk = chunks - 1, buf = 0; chunk >= 0; --chunk, buf ^= 1) {
            const int t0 = chunk * kChunk, nt = min(kChunk, it.len - t0);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int v = i * kThreads + threadIdx.x;
                constexpr int kOwn = S >= 4 ? S / 4 : 1;      // vectors of a lane
                const int r = v / (NP / 4), e = v % (NP / 4), at = S >= 4 ? e % kOwn * 4 + e / kOwn : e;
                if (2 * kVec % kThreads == 0 || v < 2 * kVec) *reinterpret_cast<float4*>(&sh.bc[0][0][0] + r * NP + 4 * at) = widen(bc[i]);
            }
            cp_async_wait_group<0>();
            __syncwarp();
            if (chunk > 0) {
                copy(chunk - 1, buf ^ 1);
                prefetch(chunk - 1);
            }
            cp_async_commit();
            auto raw = [&](int k, int t) {             // the lane's channels of a row
                const T* r = &w.raw[buf][k][t][g * C];
                return C == 2 ? load2(r) : both(to_f32(*r));
            };
            f32x2 sum = 0ull;                          // of delta over the chunk
#pragma unroll
            for (int e = 0; e < kChunk / 4; ++e) {
                const int t = 4 * e + q4;
                float v0, v1;
                f32x2 dl = add2(raw(1, t), bias);
                if (p.softplus) {
                    unpair(dl, v0, v1);
                    dl = softplus2(v0, v1);
                }
                if (t >= nt) dl = 0ull;                // rows past the end leave the state alone (their x and dout are 0)
                sum = add2(sum, dl);
                const f32x2 u = mul2(dl, raw(0, t)), gy = gated ? mul2(raw(2, t), silu2<kExact>(raw(3, t))) : raw(2, t);
                float u0, u1;
                unpair(dl, v0, v1);
                unpair(u, u0, u1);
                if (C == 2) {
                    *reinterpret_cast<float4*>(&w.du[t][2 * g * C]) = make_float4(v0, u0, v1, u1);
                    *reinterpret_cast<f32x2*>(&w.gy[t][g * C]) = gy;
                } else {
                    *reinterpret_cast<float2*>(&w.du[t][2 * g]) = make_float2(v0, u0);
                    unpair(gy, v0, v1);
                    w.gy[t][g] = v0;
                }
            }
            __syncthreads();
            // delta and u of the lane's channels for a token
            auto channel = [&](int t, f32x2 (&dd)[C], f32x2 (&uu)[C]) {
                if (C == 2) {
                    const float4 v = *reinterpret_cast<const float4*>(&w.du[t][2 * g * C]);
                    dd[0] = both(v.x); uu[0] = both(v.y);
                    dd[C - 1] = both(v.z); uu[C - 1] = both(v.w);
                } else {
                    const float2 v = *reinterpret_cast<const float2*>(&w.du[t][2 * g]);
                    dd[0] = both(v.x); uu[0] = both(v.y);
                }
            };
            const int slabs = (nt + K - 1) / K;
            f32x2 h[C][H];
            auto start_of = [&](int sl) {
                const float* from = sl == 0 ? w.check[buf] : w.start[sl - 1];
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < H; ++i) h[c][i] = *reinterpret_cast<const f32x2*>(from + (c * H + i) * 64 + lane * 2);
            };
            start_of(0);
            for (int sl = 0; sl + 1 < slabs; ++sl) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int t = sl * K + k;
                    f32x2 dd[C], uu[C], B[H];
                    channel(t, dd, uu);
                    lds<S>(B, sh.bc[0][t], q4);
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int i = 0; i < H; ++i)
                            h[c][i] = fma2(ex2_2(mul2(dd[c], a2[c][i])), h[c][i], mul2(uu[c], B[i]));
                }
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < H; ++i) *reinterpret_cast<f32x2*>(&w.start[sl][(c * H + i) * 64 + lane * 2]) = h[c][i];
            }
            for (int sl = slabs - 1; sl >= 0; --sl) {
                start_of(sl);
                float y[K * C], u[K * C], v[K * C];    // C.h, u and sum A w by token and channel
                f32x2 a[K][C][H], ah[K][C][H];
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int t = sl * K + k;
                    f32x2 dd[C], uu[C], B[H], Cv[H];
                    channel(t, dd, uu);
                    lds<S>(B, sh.bc[0][t], q4);
                    lds<S>(Cv, sh.bc[1][t], q4);
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        f32x2 ys = 0ull;
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            a[k][c][i] = ex2_2(mul2(dd[c], a2[c][i]));
                            ah[k][c][i] = mul2(a[k][c][i], h[c][i]);
                            h[c][i] = fma2(uu[c], B[i], ah[k][c][i]);
                            ys = i == 0 ? mul2(Cv[i], h[c][i]) : fma2(Cv[i], h[c][i], ys);
                        }
                        float lo, hi;
                        unpair(ys, lo, hi);
                        y[k * C + c] = lo + hi;
                    }
                }
                sum_row<K, C>(y, lane);
#pragma unroll
                for (int k = K - 1; k >= 0; --k) {
                    const int t = sl * K + k;
                    f32x2 dd[C], uu[C], B[H], Cv[H], gg[C];
                    channel(t, dd, uu);
                    if (C == 2) {
                        const float2 v = *reinterpret_cast<const float2*>(&w.gy[t][g * C]);
                        gg[0] = both(v.x);
                        gg[C - 1] = both(v.y);
                    } else {
                        gg[0] = both(w.gy[t][g]);
                    }
                    lds<S>(B, sh.bc[0][t], q4);
                    lds<S>(Cv, sh.bc[1][t], q4);
                    f32x2 dB[H], dC[H];
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        f32x2 us = 0ull, vs = 0ull;
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            const f32x2 r = fma2(gg[c], Cv[i], qv[c][i]), hh = fma2(uu[c], B[i], ah[k][c][i]);
                            dC[i] = c == 0 ? mul2(gg[c], hh) : fma2(gg[c], hh, dC[i]);
                            dB[i] = c == 0 ? mul2(uu[c], r) : fma2(uu[c], r, dB[i]);
                            us = i == 0 ? mul2(r, B[i]) : fma2(r, B[i], us);
                            const f32x2 rah = mul2(r, ah[k][c][i]);
                            vs = i == 0 ? mul2(rah, a2[c][i]) : fma2(rah, a2[c][i], vs);
                            dA[c][i] = fma2(dd[c], rah, dA[c][i]);
                            qv[c][i] = mul2(a[k][c][i], r);
                        }
                        float lo, hi;
                        unpair(us, lo, hi);
                        u[k * C + c] = lo + hi;
                        unpair(vs, lo, hi);
                        v[k * C + c] = lo + hi;
                    }
                    float part[2 * S];                 // the sums over the warp's channels
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        unpair(dB[i], part[2 * i], part[2 * i + 1]);
                        unpair(dC[i], part[S + 2 * i], part[S + 2 * i + 1]);
                    }
                    halve<2 * S>(part, lane, 16);
                    halve<S>(part, lane, 8);
                    halve<S / 2>(part, lane, 4);
                    // value g of 2 S / 8 each; with S = 2 lanes differing in bit 2 hold the same
                    constexpr int kLeft = S >= 4 ? S / 4 : 1;
                    if (S >= 4 || (lane & 4) == 0)
#pragma unroll
                        for (int i = 0; i < kLeft; ++i) {
                            const int x = S >= 4 ? g * kLeft + i : g >> 1;     // 0 .. S - 1: dB, then dC
                            w.dbc[t][x / S * NP + n0 + x % S] = part[i];
                        }
                }
                sum_row<K, C>(u, lane);
                sum_row<K, C>(v, lane);
                {
                    // a lane's channels, one token of the slab
                    const int t = sl * K + q4 % K;
                    if (t < nt && in && q4 < K) {
                        // (one channel: both halves of a pair are it)
                        const f32x2 x = raw(0, t), dy = raw(2, t), us = pair(u[0], u[C - 1]);
                        f32x2 delta, gy;
                        if (C == 2) {
                            delta = pair(w.du[t][2 * g * C], w.du[t][2 * g * C + 2]);
                            gy = *reinterpret_cast<const f32x2*>(&w.gy[t][g * C]);
                        } else {
                            delta = both(w.du[t][2 * g]);
                            gy = both(w.gy[t][g]);
                        }
                        const f32x2 ox = fma2(delta, us, mul2(skip, gy));
                        f32x2 ot = fma2(x, us, mul2(pair(v[0], v[C - 1]), both(0.69314718055994531f)));   // A = a2 ln 2
                        if (p.softplus) {
                            float a, b;
                            unpair(add2(raw(1, t), bias), a, b);
                            ot = mul2(ot, pair(softplus_grad(a), softplus_grad(b)));
                        }
                        dD = fma2(gy, x, dD);
                        db = add2(db, ot);
                        auto put = [&](void* base, f32x2 o) {
                            T* r = static_cast<T*>(base) + ((int64_t)it.t0 + t0 + t) * p.D + dch;
                            float a, b;
                            unpair(o, a, b);
                            if (C == 2) store2(r, o);
                            else *r = from_f32<T>(a);
                        };
                        put(p.dx, ox);
                        put(p.ddt, ot);
                        if (gated) {
                            // silu'(z) = s + z s (1 - s)
                            const f32x2 z = raw(3, t);
                            const f32x2 s = sigmoid2<kExact>(z), zs = mul2(z, s);
                            const f32x2 slope = fma2(zs, fma2(s, both(-1.f), both(1.f)), s);
                            put(p.dz, mul2(mul2(dy, fma2(skip, x, pair(y[0], y[C - 1]))), slope));
                        }
                    }
                }
            }
            if (nt == kChunk) {
                float of[2];
                unpair(sum, of[0], of[1]);
#pragma unroll
                for (int c = 0; c < C; ++c) {
#pragma unroll
                    for (int bit = 1; bit < 4; bit *= 2) of[c] += __shfl_xor_sync(0xffffffffu, of[c], bit);
                    make_up<H>(qv[c], a2[c], of[c]);
                }
            }
            __syncthreads();
            // the CTA's terms of dB and dC: its warps' added in order
            for (int i = threadIdx.x; i < nt * NP / 2; i += kThreads) {
                const int t = i / (NP / 2), v = i % (NP / 2) * 4, n = v % NP;      // four states of one token and kind
                f32x2 s0 = 0ull, s1 = 0ull;
#pragma unroll
                for (int k = 0; k < P::kWarps; ++k) {
                    const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&sh.w[k].dbc[t][v]);
                    s0 = add2(s0, f.x);
                    s1 = add2(s1, f.y);
                }
                float* to = p.part + ((((int64_t)tg * p.g.T + it.t0 + t0 + t) * p.G + grp) * 2 + v / NP) * p.N + n;
                if (p.N % 4 == 0) {
                    if (n < p.N) *reinterpret_cast<ulonglong2*>(to) = make_ulonglong2(s0, s1);
                } else {
                    float f[4];
                    unpair(s0, f[0], f[1]);
                    unpair(s1, f[2], f[3]);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (n + k < p.N) to[k] = f[k];
                }
            }
        }
        if (it.first && p.dinit != nullptr)
#pragma unroll
            for (int c = 0; c < C; ++c)
                store_states_row<S>(qv[c], p.dinit + ((int64_t)it.seq * p.D + dch + c) * p.N, n0, p.N, in);
    }
    // the slot's terms of dA, dD and dbias
#pragma unroll
    for (int c = 0; c < C; ++c)
        store_states_row<S>(dA[c], p.partA + ((int64_t)slot * p.D + dch + c) * p.N, n0, p.N, in);
    float end[4];
    unpair(dD, end[0], end[1]);
    unpair(db, end[2], end[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int bit = 1; bit < 4; bit *= 2) end[i] += __shfl_xor_sync(0xffffffffu, end[i], bit);
    if (q4 == 0 && in)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            p.partD[(int64_t)slot * 2 * p.D + dch + c] = end[c];
            p.partD[((int64_t)slot * 2 + 1) * p.D + dch + c] = end[2 + c];
        }
}

// dB and dC: the tiles' terms in order; 0 in rows of no sequence.  Bound by the terms' bytes.
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
    using P = Plan<T, S>;
    constexpr auto kernel = selscan_bwd<T, S>;
    constexpr int kTile = P::kWarps * P::kCh;
    const int tpg = (p.cpg + kTile - 1) / kTile;
    const int64_t slots = p.slots + (p.g.cu != nullptr ? 16 : 0);
    if (slots > 0) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(typename P::Cta));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        kernel<<<(unsigned)(slots * tpg * p.G), P::kWarps * 32, (int)sizeof(typename P::Cta), stream>>>(p);
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
