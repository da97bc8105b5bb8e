// selscan_fwd.cu -- the selective scan over packed prompts.
//
// One warp walks 32 / LPC channels of a sequence (or of a range of it), a lane
// holding S states of one channel in registers: with 16 states a lane is a
// channel, so the sum over the states needs no other lane.  Tiles of eight tokens
// of x, dt and z come by cp.async, 16 bytes a lane, three tiles ahead (loaded into
// registers one tile ahead, as in a first version, a warp by itself waited for
// memory at every tile: 121 ns a token instead of 101 at that time); the rows of B and C, which
// every lane reads, wait in registers and pass through shared memory as fp32.  A
// tile's delta and u = delta x are made first, all eight side by side.  The
// recurrence itself is the packed fp32 instructions' work: per pair of states two
// products, two multiply-adds and two exponentials.
//
// What bounds it: for 16 states a token costs a warp 109 instructions (all that are executed, by tokens
// and warps) and 196 clocks of its quarter-SM, in 52 % of which the multiply-add pipe works and in 44 % the
// exponentials'; three warps a quarter-SM (166 registers) issue in 60 %.  16384 tokens of 5120 channels in
// 12 sequences: 445 us (20 of them make_up).  Tried when it took 427 to 432: eight states a lane, two lanes a
// channel (more warps, but every row of B and C is read twice as often for the same work) took
// 1.08 times that, four states 1.41; the next tile's delta made between this one's tokens
// 1.03; the products delta A by scalar instructions, which alone run faster beside the exponential, 1.03;
// pairs of channels instead of states, delta and u through shared memory (fewer moves, more
// shared memory traffic) 1.16; four warps a quarter-SM (128 registers, some spilled) 1.18; y by way of shared memory in
// pieces of 16 bytes 1.01.
#include <type_traits>

#include "selscan.cuh"
#include "sm100_ptx.cuh"

namespace ssd {
namespace {

constexpr int kTok = 8;      // tokens of a tile
constexpr int kWarps = 2;    // warps of a CTA, each on its own
constexpr int kZeroItems = 64;
constexpr int kStages = 4;   // tiles of x, dt and z in shared memory

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
__global__ void __launch_bounds__(kWarps * 32, S == 16 && LPC == 1 ? 6 : 1) selscan_walk(const __grid_constant__ ScanParams p) {
    constexpr int kCh = 32 / LPC, NP = S * LPC, kVec = kTok * NP / 4, kPer = (kVec + 31) / 32, kOwn = kTok / LPC;
    constexpr bool kExact = sizeof(T) == 4, SUMS = MODE != kScanMain, REV = MODE == kScanRevSums;
    constexpr int kPieces = kTok * kCh * sizeof(T) / 16;    // 16-byte pieces of a tile of x, of dt and of z
    constexpr int kRowPieces = kCh * sizeof(T) / 16, kCopies = (3 * kPieces + 31) / 32;
    struct Warp {
        T raw[kStages][3][kTok][kCh];
        float B[2][kTok][NP];
        float C[SUMS ? 1 : 2][kTok][NP];
        float du[LPC > 1 ? 2 : 1][LPC > 1 ? kCh : 1][2 * kTok + 4];
    };
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = lane % LPC;
    const int tpg = (p.cpg + kCh - 1) / kCh, tiles = tpg * p.G, ctas = (tiles + kWarps - 1) / kWarps;
    const int item = blockIdx.x / ctas, tile = (blockIdx.x - item * ctas) * kWarps + warp;
    if (tile >= tiles) return;
    Warp& w = reinterpret_cast<Warp*>(smem)[warp];
    const int grp = tile / tpg, c0 = (tile - grp * tpg) * kCh, cl = lane / LPC, ch = c0 + cl;
    const bool in = ch < p.cpg;
    const int d = grp * p.cpg + min(ch, p.cpg - 1), n0 = part * S;
    if (!SUMS && item >= p.g.items) {            // rows of no sequence
        const int end = min(max(p.g.cu[p.g.nseq], 0), p.g.T);
        if (in && part == 0)
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
    const bool gated = MODE != kScanSums && p.z != nullptr, vecB = (REV ? p.vecC : p.vecB) != 0;
    T* yp = static_cast<T*>(p.y) + (int64_t)it.t0 * p.D + (int64_t)part * p.D + d;
    const int brow = lane / (NP / 4), bcol = lane % (NP / 4) * 4;     // its first vector of a tile's B (C)
    const T* Bp = static_cast<const T*>(REV ? p.C : p.B) + row0 * (REV ? p.Cs : p.Bs) + brow * Bs + (int64_t)grp * p.N;
    const T* Cp = static_cast<const T*>(p.C) + row0 * p.Cs + brow * p.Cs + (int64_t)grp * p.N;
    // the lane's pieces of a tile of x, dt and z: where from, and how far the next tile is
    const T* src[kCopies];
    int64_t step[kCopies];
    int crow[kCopies];                       // row in the tile, or behind all rows: nothing to copy
    uint32_t dst[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int v = i * 32 + lane, k = v / kPieces, r = v % kPieces / kRowPieces, c = v % kRowPieces * (16 / (int)sizeof(T));
        const int64_t stride = k == 0 ? xs : k == 1 ? ts : zs;
        const T* from = static_cast<const T*>(k == 0 ? (REV ? p.dout : p.x) : k == 1 ? p.dt : p.z);
        const int64_t first = row0 * (k == 0 ? (REV ? p.D : p.xs) : k == 1 ? p.dts : p.zs);
        const bool ok = k < (gated ? 3 : 2) && c0 + c < p.cpg;
        crow[i] = ok ? r : 1 << 30;
        src[i] = ok ? from + first + r * stride + (int64_t)grp * p.cpg + c0 + c : reinterpret_cast<const T*>(p.A);   // (x may be NULL)
        step[i] = ok ? kTok * stride : 0;
        dst[i] = k < 3 ? smem_u32(&w.raw[0][0][0][0]) + 16 * v : 0u;
    }
    auto copy = [&](int t0, int stage) {     // the tile at t0; zeros behind the range's end
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            if ((i + 1) * 32 <= 3 * kPieces || i * 32 + lane < 3 * kPieces)
                cp_async_16(dst[i] + stage * (int)sizeof(w.raw[0]), src[i], (int64_t)t0 + crow[i] < it.len ? 16u : 0u);
            src[i] += step[i];
        }
    };
    // B and C of the next tile wait in registers
    Raw4<T> br[kPer], cr[kPer];
    auto prefetch = [&](int t0) {
        constexpr int kStep = 128 / NP;                               // rows from one vector to the next
        static_assert(kPer == 1 || kPer * kStep == kTok, "a lane's vectors are a tile's");
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const bool ok = (kVec % 32 == 0 || lane < kVec) && t0 + brow + i * kStep < it.len;
            fetch(br[i], Bp + i * kStep * Bs, ok ? bcol : p.N, p.N, vecB);
            if (!SUMS) fetch(cr[i], Cp + i * kStep * p.Cs, ok ? bcol : p.N, p.N, p.vecC != 0);
        }
        Bp += kTok * Bs;
        if (!SUMS) Cp += kTok * p.Cs;
    };
    f32x2 total = 0ull, recent = 0ull;      // sums of delta: the range's, the last sixteen tokens'
    struct Own {
        f32x2 x[kOwn / 2], gate[kOwn / 2];   // of its own tokens, in pairs
        float2 du[LPC > 1 ? 1 : kTok];       // a lane with all of a channel: delta and u
    };
    // delta and u of the tile at t0 into shared memory, and B and C; rows behind the range's
    // end multiply the state by 1 and add nothing (their x and dout are zeros)
    auto prepare = [&](int t0, Own& o, auto full) {
        const int at = t0 / kTok, buf = at & 1, stage = at % kStages;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = i * 32 + lane;
            if (kVec % 32 == 0 || v < kVec) {
                // vector k of a row's lane q lies at k LPC + q, so that the lanes of a channel read other
                // banks (8192 tokens of 2048 channels, 64 states: 491 us; each lane's own side by side 756)
                const int r = v / (NP / 4), e = v % (NP / 4), at = e % (S / 4) * LPC + e / (S / 4);
                *reinterpret_cast<float4*>(&w.B[buf][r][4 * at]) = widen(br[i]);
                if (!SUMS) *reinterpret_cast<float4*>(&w.C[SUMS ? 0 : buf][r][4 * at]) = widen(cr[i]);
            }
        }
        auto raw2 = [&](int k, int i) {
            return pair(to_f32(w.raw[stage][k][2 * i * LPC + part][cl]), to_f32(w.raw[stage][k][(2 * i + 1) * LPC + part][cl]));
        };
        f32x2 dl[kOwn / 2];
#pragma unroll
        for (int i = 0; i < kOwn / 2; ++i) {
            dl[i] = add2(raw2(1, i), both(bias));
            o.x[i] = raw2(0, i);
        }
        if (p.softplus)
#pragma unroll
            for (int i = 0; i < kOwn / 2; ++i) {
                float a, b;
                unpair(dl[i], a, b);
                dl[i] = softplus2(a, b);
            }
        if (MODE != kScanSums)
#pragma unroll
            for (int i = 0; i < kOwn / 2; ++i) o.gate[i] = both(1.f);
        if (gated)
#pragma unroll
            for (int i = 0; i < kOwn / 2; ++i) o.gate[i] = silu2<kExact>(raw2(2, i));
        float* row = &w.du[LPC > 1 ? buf : 0][LPC > 1 ? cl : 0][0];
#pragma unroll
        for (int i = 0; i < kOwn / 2; ++i) {
            const int t = t0 + 2 * i * LPC + part;
            float a, b, c, e;
            if (!decltype(full)::value) {
                unpair(dl[i], a, b);
                dl[i] = pair(t < it.len ? a : 0.f, t + LPC < it.len ? b : 0.f);
            }
            recent = add2(recent, dl[i]);
            unpair(dl[i], a, b);
            unpair(REV ? mul2(o.x[i], o.gate[i]) : mul2(dl[i], o.x[i]), c, e);
            if (LPC > 1) {                   // the channel's other lanes need them too
                *reinterpret_cast<float2*>(row + 2 * (2 * i * LPC + part)) = make_float2(a, c);
                *reinterpret_cast<float2*>(row + 2 * ((2 * i + 1) * LPC + part)) = make_float2(b, e);
            } else {
                o.du[(2 * i) % (LPC > 1 ? 1 : kTok)] = make_float2(a, c);
                o.du[(2 * i + 1) % (LPC > 1 ? 1 : kTok)] = make_float2(b, e);
            }
        }
    };
    auto tokens = [&](int t0, const Own& o, auto full) {
        constexpr bool kFull = decltype(full)::value;
        const int buf = (t0 / kTok) & 1;
        auto token = [&](int t, f32x2& delta, f32x2& u) {                  // each twice, for pairs of states
            const float2 v = LPC > 1 ? *reinterpret_cast<const float2*>(&w.du[LPC > 1 ? buf : 0][LPC > 1 ? cl : 0][2 * t])
                                     : o.du[t % (LPC > 1 ? 1 : kTok)];
            delta = both(v.x);
            u = both(v.y);
        };
        // the next token's decays are made while this one's are used
        f32x2 a[S / 2], dn, u, un;
        float y[LPC];
        token(0, dn, un);
#pragma unroll
        for (int i = 0; i < S / 2; ++i) a[i] = ex2_2(mul2(dn, a2[i]));
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            u = un;
            if (t + 1 < kTok) token(t + 1, dn, un);
            f32x2 y0 = 0ull, y1 = 0ull;
#pragma unroll
            for (int i = 0; i < S / 4; ++i) {
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&w.B[buf][t][4 * (i * LPC + part)]);
                f32x2 an0 = 0ull, an1 = 0ull;
                if (t + 1 < kTok) {
                    an0 = ex2_2(mul2(dn, a2[2 * i]));
                    an1 = ex2_2(mul2(dn, a2[2 * i + 1]));
                }
                if (REV) {
                    h[2 * i] = mul2(a[2 * i], fma2(u, b.x, h[2 * i]));
                    h[2 * i + 1] = mul2(a[2 * i + 1], fma2(u, b.y, h[2 * i + 1]));
                } else {
                    h[2 * i] = fma2(a[2 * i], h[2 * i], mul2(u, b.x));
                    h[2 * i + 1] = fma2(a[2 * i + 1], h[2 * i + 1], mul2(u, b.y));
                }
                a[2 * i] = an0;
                a[2 * i + 1] = an1;
                if (!SUMS) {
                    const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&w.C[SUMS ? 0 : buf][t][4 * (i * LPC + part)]);
                    y0 = i == 0 ? mul2(c.x, h[0]) : fma2(c.x, h[2 * i], y0);
                    y1 = i == 0 ? mul2(c.y, h[1]) : fma2(c.y, h[2 * i + 1], y1);
                }
            }
            if (!SUMS) {
                float lo, hi;
                unpair(add2(y0, y1), lo, hi);
                y[t % LPC] = lo + hi;
                if (t % LPC == LPC - 1) {          // of the last LPC tokens a lane gets its own one's sum
                    if (LPC >= 4) halve<LPC>(y, lane, LPC / 2);
                    if (LPC >= 2) halve<2>(y, lane, 1);
                    const int i = t / LPC;
                    float x0, x1, g0, g1;
                    unpair(o.x[i / 2], x0, x1);
                    unpair(o.gate[i / 2], g0, g1);
                    const float v = fmaf(skip, i & 1 ? x1 : x0, y[0]) * (i & 1 ? g1 : g0);
                    if (in && (kFull || t0 + i * LPC + part < it.len)) *yp = from_f32<T>(v);
                    yp += (int64_t)LPC * p.D;
                }
            }
        }
    };
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) {
        copy(i * kTok, i);
        cp_async_commit();
    }
    prefetch(0);
    auto step_of = [&](int t0, auto full) {
        cp_async_wait_group<kStages - 2>();
        __syncwarp();                        // the tile's rows are there; the tile before it is done
        copy(t0 + (kStages - 1) * kTok, (t0 / kTok + kStages - 1) % kStages);
        cp_async_commit();
        if (!SUMS && p.states != nullptr && (it.done + t0) % kScanChunk == 0)
            store_row<S>(h, p.states + ((int64_t)(it.row0 + (it.done + t0) / kScanChunk) * p.D + d) * p.N, n0, p.N, in);
        Own own;
        prepare(t0, own, full);
        prefetch(t0 + kTok);
        __syncwarp();
        tokens(t0, own, full);
        if ((t0 + kTok) % kMakeUp == 0) {
            float sum, odd;
            unpair(recent, sum, odd);
            sum += odd;
#pragma unroll
            for (int bit = LPC / 2; bit > 0; bit /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, bit);
            make_up<S / 2>(h, a2, sum);
            if (SUMS) total = add2(total, recent);
            recent = 0ull;
        }
    };
    int t0 = 0;
    for (; t0 + kTok <= it.len; t0 += kTok) step_of(t0, std::true_type());
    if (t0 < it.len) step_of(t0, std::false_type());
    cp_async_wait_group<0>();
    if (SUMS) {
        store_row<S>(h, p.agg + ((int64_t)item * p.D + d) * p.N, n0, p.N, in);
        float sum, odd;
        unpair(add2(total, recent), sum, odd);
        sum += odd;
#pragma unroll
        for (int bit = LPC / 2; bit > 0; bit /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, bit);
        if (in && part == 0) p.aggd[(int64_t)item * p.D + d] = sum;
    } else if (p.fin != nullptr && it.last) {
        store_row<S>(h, p.fin + row, n0, p.N, in);
    }
}

// The states at the starts of a sequence's ranges, in place of the ranges' own ends:
// a thread for each state, the ranges in order, eight of them loaded ahead.  Bound by the
// latency of those loads where a sequence has many ranges, by the ends' bytes else.  rev: from
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
    constexpr int NP = S * LPC, kCh = 32 / LPC;
    // (shared memory of a warp as the kernel lays it out)
    const int bytes = kWarps * (kStages * 3 * kTok * kCh * (int)sizeof(T) + (mode == kScanMain ? 4 : 3) * kTok * NP * 4 +
                                (LPC > 1 ? 2 * kCh : 1) * (2 * kTok + 4) * 4);
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    k<<<(unsigned)(items * ctas), kWarps * 32, bytes, stream>>>(p);
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
