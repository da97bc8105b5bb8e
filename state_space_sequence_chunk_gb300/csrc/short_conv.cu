// short_conv.cu -- depthwise causal convolution over packed, token-major rows, with
// its activation, its gradient and its form for single tokens.
//
// Per channel and sequence, with W taps and the W - 1 rows before the sequence from
// its initial state (0 without one):
//     p_t = bias + sum_k w_k x_{t-W+1+k},    o_t = a(p_t),  a(p) = p or p sigmoid(p)
//     g_t = do_t a'(p_t),  dx_t = sum_k w_k g_{t+W-1-k},  dw_k = sum_t g_t x_{t-W+1+k}
// Each row is read once and written once.  A thread owns four channels (the gradient:
// two) and walks a tile of tokens with the last W - 1 rows in registers, eight rows'
// loads in flight while eight are computed; the W - 1 rows before a tile are read again
// (from L2, mostly).  Sequences begin and end anywhere in a tile: the walk goes by its
// part of each, with the window loaded anew.
//
// What bounds it: forwards HBM, in bf16 with about half of the issue slots, 49 instructions for a row of four
// channels a thread.  16384 bf16 tokens of 5120 channels, 4 taps: 59 us, 5.7 TB/s (with other tiles: short_conv_tile; of
// tiles of 64, two channels a thread took 1.03 times as long, eight, with checks in the loop instead of
// parts, 1.6 times); the gradient, 46 instructions for two channels, 108 us, 4.7 TB/s (four channels
// 1.08 times; bounds in every group of rows 1.05): neither HBM (62 %) nor the issue (51 %) is full, rows
// come in bursts of eight that are waited for.  fp32, of 2048 channels: 50 us, 5.4 TB/s, and
// 77 us, 5.2 TB/s.  The test for an activation stays in the row: with a kernel of its own for each, the
// compiler mixes more rows, and spills (1.04 to 1.07 times as long, also with fewer CTAs an SM or rows ahead).
#include <type_traits>

#include "approx.cuh"
#include "short_conv.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;        // rows loaded ahead
constexpr int kFwdVec = 4, kBwdVec = 2;   // channels of a thread

// V channels of a row: as loaded, and as pairs of floats.
template <typename T, int V> struct Row;
template <> struct Row<__nv_bfloat16, 4> {
    uint2 r;
    __device__ void load(const __nv_bfloat16* p) { r = __ldg(reinterpret_cast<const uint2*>(p)); }
    __device__ void zero() { r = make_uint2(0u, 0u); }
    __device__ void get(f32x2 (&v)[2]) const {
        v[0] = pair(r.x << 16, r.x & 0xFFFF0000u); v[1] = pair(r.y << 16, r.y & 0xFFFF0000u);
    }
    __device__ static void store(__nv_bfloat16* p, const f32x2 (&v)[2]) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0]), pack2(v[1]));
    }
};
template <> struct Row<__nv_bfloat16, 2> {
    uint32_t r;
    __device__ void load(const __nv_bfloat16* p) { r = __ldg(reinterpret_cast<const uint32_t*>(p)); }
    __device__ void zero() { r = 0u; }
    __device__ void get(f32x2 (&v)[1]) const { v[0] = pair(r << 16, r & 0xFFFF0000u); }
    __device__ static void store(__nv_bfloat16* p, const f32x2 (&v)[1]) { *reinterpret_cast<uint32_t*>(p) = pack2(v[0]); }
};
template <> struct Row<float, 2> {
    f32x2 r;
    __device__ void load(const float* p) { r = __ldg(reinterpret_cast<const f32x2*>(p)); }
    __device__ void zero() { r = 0ull; }
    __device__ void get(f32x2 (&v)[1]) const { v[0] = r; }
    __device__ static void store(float* p, const f32x2 (&v)[1]) { *reinterpret_cast<f32x2*>(p) = v[0]; }
};
template <> struct Row<float, 4> {
    ulonglong2 r;
    __device__ void load(const float* p) { r = __ldg(reinterpret_cast<const ulonglong2*>(p)); }
    __device__ void zero() { r = make_ulonglong2(0ull, 0ull); }
    __device__ void get(f32x2 (&v)[2]) const { v[0] = r.x; v[1] = r.y; }
    __device__ static void store(float* p, const f32x2 (&v)[2]) {
        *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(v[0], v[1]);
    }
};

__device__ __forceinline__ void bounds(const ShortConv& p, int s, int& lo, int& hi) {
    // clamped, so that no content of cu leads out of the tensors
    if (p.cu != nullptr) {
        lo = min(max(p.cu[s], 0), p.T);
        hi = min(max(p.cu[s + 1], lo), p.T);
    } else {
        lo = s * p.L;
        hi = lo + p.L;
    }
}
// The first sequence that ends after row t (nseq: none does).  Executed by a whole warp.
__device__ __forceinline__ int find(const ShortConv& p, int t) {
    if (p.cu == nullptr) return p.L > 0 ? t / p.L : p.nseq;
    const int lane = threadIdx.x & 31;
    int at = 0, n = p.nseq;              // sequences at .. at + n - 1 to look at: those before end at t or before
    while (n > 0) {
        const int step = (n + 31) / 32, o = lane * step;
        const int c = __popc(__ballot_sync(0xffffffffu, o < n && p.cu[at + min(o, n - 1) + 1] <= t));
        if (c == 0) break;
        at += (c - 1) * step + 1;
        n = min(step - 1, n - (c - 1) * step - 1);
    }
    return at;
}

// Row `pos` of sequence s, which begins at lo and may have it before its start.
template <typename T, int V>
__device__ __forceinline__ void row_of(const ShortConv& p, Row<T, V>& r, int W, int s, int lo, int pos, int col) {
    if (pos >= lo) r.load(static_cast<const T*>(p.x) + pos * p.xs + col);
    else if (p.init != nullptr)
        r.load(static_cast<const T*>(p.init) + ((int64_t)s * (W - 1) + max(pos - lo + W - 1, 0)) * p.D + col);
    else r.zero();
}

template <int V, int W> struct Taps {
    f32x2 w[W][V / 2], b[V / 2];
    __device__ void load(const ShortConv& p, int col) {
        float f[V * W];                          // the V channels' taps lie together
        const float* at = p.w + (int64_t)col * W;
        if (V % 4 == 0) {                        // (16-byte vectors: V W is a multiple of four, and so is col W)
#pragma unroll
            for (int i = 0; i < V * W; i += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(at + i));
                f[i] = v.x; f[(i + 1) % (V * W)] = v.y; f[(i + 2) % (V * W)] = v.z; f[(i + 3) % (V * W)] = v.w;
            }
        } else {                                 // (8-byte vectors: both are even)
#pragma unroll
            for (int i = 0; i < V * W; i += 2) {
                const float2 v = __ldg(reinterpret_cast<const float2*>(at + i));
                f[i] = v.x; f[(i + 1) % (V * W)] = v.y;
            }
        }
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][i] = pair(f[2 * i * W + k], f[(2 * i + 1) * W + k]);
            b[i] = p.bias != nullptr ? __ldg(reinterpret_cast<const f32x2*>(p.bias + col) + i) : 0ull;
        }
    }
    // bias + sum of taps: the window's W - 1 rows, then the present one
    __device__ void apply(const f32x2 (&win)[W - 1][V / 2], const f32x2 (&now)[V / 2], f32x2 (&s)[V / 2]) const {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            s[i] = b[i];
#pragma unroll
            for (int k = 0; k < W - 1; ++k) s[i] = fma2(w[k][i], win[k][i], s[i]);
            s[i] = fma2(w[W - 1][i], now[i], s[i]);
        }
    }
};
template <int N2, int M> __device__ __forceinline__ void shift(f32x2 (&win)[M][N2], const f32x2 (&now)[N2]) {
#pragma unroll
    for (int k = 0; k + 1 < M; ++k)
#pragma unroll
        for (int i = 0; i < N2; ++i) win[k][i] = win[k + 1][i];
#pragma unroll
    for (int i = 0; i < N2; ++i) win[M - 1][i] = now[i];
}
template <bool EXACT, int N2> __device__ __forceinline__ void activate(f32x2 (&v)[N2], int act) {
    if (act == SSD_ACT_NONE) return;
#pragma unroll
    for (int i = 0; i < N2; ++i) v[i] = mul2(v[i], sigmoid2<EXACT>(v[i]));
}
// g = do a'(p): silu' = s + p s (1 - s) with s = sigmoid(p)
template <bool EXACT, int N2> __device__ __forceinline__ void back(f32x2 (&g)[N2], const f32x2 (&pre)[N2], int act) {
    if (act == SSD_ACT_NONE) return;
#pragma unroll
    for (int i = 0; i < N2; ++i) {
        const f32x2 s = sigmoid2<EXACT>(pre[i]), ps = mul2(pre[i], s);
        g[i] = mul2(g[i], fma2(ps, fma2(s, pair(-1.f, -1.f), pair(1.f, 1.f)), s));
    }
}

// CTAs that an SM holds (by registers): the tile's length goes by it.
constexpr int ctas_per_sm(int W, int bytes, bool backward) {
    return W > 4 ? 3 : bytes == 2 ? 5 : backward ? 3 : 4;
}
// A warp's item (a tile of tokens, or behind those a sequence) and its lane's vector of the row:
// shared out by warps, so that a row of 386 vectors takes 13 of them and not 4 CTAs.
__device__ __forceinline__ bool warp_item(const ShortConv& p, int vecs, int& item, int& vec) {
    // (the shuffle tells the compiler that all lanes have the same number)
    const int warps = (vecs + 31) / 32, w = blockIdx.x * (kThreads / 32) + __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    item = w / warps;
    vec = (w - item * warps) * 32 + (threadIdx.x & 31);
    return item < p.items;
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(W, sizeof(T), false)) short_conv_fwd(const __grid_constant__ ShortConv p) {
    constexpr int V = kFwdVec, N2 = V / 2;
    int item, vec;
    if (!warp_item(p, p.D / V, item, vec)) return;
    const bool in = vec < p.D / V;
    const int col = in ? vec * V : 0;
    if (item >= p.tiles) {                       // a sequence's final state: its last W - 1 rows
        const int s = item - p.tiles;
        int lo, hi;
        bounds(p, s, lo, hi);
        if (!in) return;
        Row<T, V> r[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) row_of<T, V>(p, r[j], W, s, lo, hi - (W - 1) + j, col);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            f32x2 v[N2];
            r[j].get(v);
            Row<T, V>::store(static_cast<T*>(p.fin) + ((int64_t)s * (W - 1) + j) * p.D + col, v);
        }
        return;
    }
    const int t0 = item * p.TT, t1 = min(t0 + p.TT, p.T);
    int s = find(p, t0);
    if (!in) return;
    const T* x = static_cast<const T*>(p.x) + col;
    T* out = static_cast<T*>(p.out) + col;
    Taps<V, W> taps;
    taps.load(p, col);
    // the tile's part of one sequence after another; rows of none behind the last
    for (int a = t0; a < t1; ++s) {
        int lo = 0, hi = 0;
        for (; s < p.nseq; ++s) {
            bounds(p, s, lo, hi);
            if (hi > a) break;
        }
        if (s >= p.nseq) {
            f32x2 zero[N2];
#pragma unroll
            for (int k = 0; k < N2; ++k) zero[k] = pair(0.f, 0.f);
            for (; a < t1; ++a) Row<T, V>::store(out + (int64_t)a * p.D, zero);
            break;
        }
        const int b = min(hi, t1);
        Row<T, V> ahead[kAhead];
        const T* from = x + a * p.xs;            // the row loaded next
        T* to = out + (int64_t)a * p.D;          // the row stored next
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (a + i < b) ahead[i].load(from);
            from += p.xs;
        }
        f32x2 win[W - 1][N2];
        {
            Row<T, V> r[W - 1];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) row_of<T, V>(p, r[j], W, s, lo, a - (W - 1) + j, col);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) r[j].get(win[j]);
        }
        auto row = [&](const Row<T, V>& r) {
            f32x2 now[N2], o[N2];
            r.get(now);
            taps.apply(win, now, o);
            activate<sizeof(T) == 4>(o, p.act);
            shift(win, now);
            Row<T, V>::store(to, o);
            to += p.D;
        };
        auto rows = [&](int t, auto all) {       // kAhead rows; `all`: as many follow them
            Row<T, V> cur[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                cur[i] = ahead[i];
                if (decltype(all)::value || t + kAhead + i < b) ahead[i].load(from);
                from += p.xs;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) row(cur[i]);
        };
        int t = a;
        for (; t + 2 * kAhead <= b; t += kAhead) rows(t, std::true_type());
        if (t + kAhead <= b) {
            rows(t, std::false_type());
            t += kAhead;
        }
#pragma unroll
        for (int i = 0; i < kAhead - 1; ++i)
            if (t + i < b) row(ahead[i]);
        a = b;
    }
}

// The gradient.  A thread walks a tile's part of each sequence with the last rows of x
// and the unfinished rows of dx in registers (row t - j lacks the terms of g beyond t),
// and W - 1 rows further, whose g the tile's last rows of dx need.  The sums for dw and
// db go into one row of partial sums per tile.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(W, sizeof(T), true)) short_conv_bwd(const __grid_constant__ ShortConv p) {
    constexpr int V = kBwdVec, N2 = V / 2;
    int item, vec;
    if (!warp_item(p, p.D / V, item, vec)) return;
    const bool in = vec < p.D / V;
    const int col = in ? vec * V : 0;
    const T* x = static_cast<const T*>(p.x) + col;
    const T* dout = static_cast<const T*>(p.dout) + col;
    const T* dfin = p.dfin != nullptr ? static_cast<const T*>(p.dfin) + col : nullptr;
    Taps<V, W> taps;
    taps.load(p, col);
    f32x2 win[W - 1][N2];
    if (item >= p.tiles) {                       // the initial state's gradient of one sequence
        const int s = item - p.tiles;
        int lo, hi;
        bounds(p, s, lo, hi);
        if (!in) return;
        const int len = hi - lo;
        f32x2 acc[W - 1][N2];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            Row<T, V> r;
            row_of<T, V>(p, r, W, s, lo, lo - (W - 1) + j, col);
            r.get(win[j]);
            r.zero();
            if (dfin != nullptr && j >= len) r.load(dfin + ((int64_t)s * (W - 1) + j - len) * p.D);
            r.get(acc[j]);
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            if (i < len) {
                Row<T, V> r, q;
                r.load(x + (lo + i) * p.xs);
                q.load(dout + (int64_t)(lo + i) * p.D);
                f32x2 now[N2], g[N2], pre[N2];
                r.get(now);
                q.get(g);
                taps.apply(win, now, pre);
                back<sizeof(T) == 4>(g, pre, p.act);
                shift(win, now);
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    if (j >= i)
#pragma unroll
                        for (int k = 0; k < N2; ++k) acc[j][k] = fma2(taps.w[j - i][k], g[k], acc[j][k]);
            }
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            Row<T, V>::store(static_cast<T*>(p.dinit) + ((int64_t)s * (W - 1) + j) * p.D + col, acc[j]);
        return;
    }
    const int t0 = item * p.TT, t1 = min(t0 + p.TT, p.T);
    int s = find(p, t0);
    if (!in) return;
    T* dx = static_cast<T*>(p.dx) + col;
    const f32x2 z2 = pair(0.f, 0.f);
    f32x2 dw[W][N2], db[N2];
#pragma unroll
    for (int k = 0; k < N2; ++k) {
        db[k] = z2;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][k] = z2;
    }
    int a = t0;
    while (a < t1) {
        int lo = 0, hi = 0;
        for (; s < p.nseq; ++s) {
            bounds(p, s, lo, hi);
            if (hi > a) break;
        }
        if (s >= p.nseq) {                       // rows of no sequence
            f32x2 zero[N2];
#pragma unroll
            for (int k = 0; k < N2; ++k) zero[k] = z2;
            for (; a < t1; ++a) Row<T, V>::store(dx + (int64_t)a * p.D, zero);
            break;
        }
        const int b = min(hi, t1), lim = min(hi, b + W - 1);   // dx of rows a .. b, from g of rows a .. lim
        f32x2 acc[W][N2];
        {
            Row<T, V> r[W - 1];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) row_of<T, V>(p, r[j], W, s, lo, a - (W - 1) + j, col);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) r[j].get(win[j]);
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int k = 0; k < N2; ++k) acc[j][k] = z2;
        Row<T, V> xa[kAhead], da[kAhead];
        const T *xn = x + a * p.xs, *dn = dout + (int64_t)a * p.D;    // the rows loaded next
        T* to = dx + (int64_t)(a - (W - 1)) * p.D;                    // the row finished next
        auto fetch = [&](int t, auto all) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (decltype(all)::value || t + i < lim) {
                    xa[i].load(xn);
                    da[i].load(dn);
                }
                xn += p.xs;
                dn += p.D;
            }
        };
        fetch(a, std::false_type());
        // own: not a row that the next tile adds; inner: a row of the tile is finished
        auto row = [&](const Row<T, V>& xr, const Row<T, V>& dr, int t, auto own, auto inner) {
            f32x2 now[N2], g[N2], pre[N2];
            xr.get(now);
            dr.get(g);
            taps.apply(win, now, pre);
            back<sizeof(T) == 4>(g, pre, p.act);
#pragma unroll
            for (int k = 0; k < N2; ++k) {
                if (decltype(own)::value) {
                    db[k] = add2(db[k], g[k]);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) dw[j][k] = fma2(g[k], win[j][k], dw[j][k]);
                    dw[W - 1][k] = fma2(g[k], now[k], dw[W - 1][k]);
                }
#pragma unroll
                for (int j = W - 1; j > 0; --j) acc[j][k] = fma2(taps.w[W - 1 - j][k], g[k], acc[j - 1][k]);
                acc[0][k] = mul2(taps.w[W - 1][k], g[k]);
            }
            shift(win, now);
            if (decltype(inner)::value || t - (W - 1) >= a) Row<T, V>::store(to, acc[W - 1]);
            to += p.D;
        };
        auto rows = [&](int t, auto all) {       // kAhead rows; `all`: not the first ones, and as many follow
            Row<T, V> xc[kAhead], dc[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                xc[i] = xa[i];
                dc[i] = da[i];
            }
            fetch(t + kAhead, all);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) row(xc[i], dc[i], t + i, std::true_type(), all);
        };
        int t = a;
        if (t + kAhead <= b) {
            rows(t, std::false_type());
            t += kAhead;
        }
        for (; t + kAhead <= b && t + 2 * kAhead <= lim; t += kAhead) rows(t, std::true_type());
        for (; t + kAhead <= b; t += kAhead) rows(t, std::false_type());
        // the rest, fewer than kAhead rows, and up to W - 1 of the next tile
        for (int i = 0; t + i < lim; ++i) {
            Row<T, V> xr, dr;
            xr.load(x + (t + i) * p.xs);
            dr.load(dout + (int64_t)(t + i) * p.D);
            if (t + i < b) row(xr, dr, t + i, std::true_type(), std::false_type());
            else row(xr, dr, t + i, std::false_type(), std::false_type());
        }
        // the sequence's last rows, if it ends here: nothing follows but the final state's gradient
#pragma unroll
        for (int j = W - 2; j >= 0; --j) {
            const int r = lim - 1 - j;
            if (r >= a && r < b) {
                if (dfin != nullptr) {
                    Row<T, V> q;
                    f32x2 v[N2];
                    q.load(dfin + ((int64_t)s * (W - 1) + r - (hi - (W - 1))) * p.D);
                    q.get(v);
#pragma unroll
                    for (int k = 0; k < N2; ++k) acc[j][k] = add2(acc[j][k], v[k]);
                }
                Row<T, V>::store(dx + (int64_t)r * p.D, acc[j]);
            }
        }
        a = b;
        ++s;
    }
    float* part = p.part + (int64_t)item * (W + 1) * p.D + col;
#pragma unroll
    for (int j = 0; j < W; ++j) Row<float, V>::store(part + (int64_t)j * p.D, dw[j]);
    Row<float, V>::store(part + (int64_t)W * p.D, db);
}

// dw and db: the tiles' sums added in the tiles' order, in eight shares, eight loads ahead:
// bound by their latency (128 tiles: two turns).
__global__ void __launch_bounds__(256) short_conv_sum(const __grid_constant__ ShortConv p, int W) {
    __shared__ float sh[8][32];
    const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + lane, k = blockIdx.y;
    const int per = (p.tiles + 7) / 8, from = share * per, to = min(from + per, p.tiles);
    float s = 0.f;
    if (d < p.D) {
        const float* at = p.part + (int64_t)k * p.D + d;
        const int64_t step = (int64_t)(W + 1) * p.D;
        int i = from;
        for (; i + 8 <= to; i += 8) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = at[(i + j) * step];
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[j];
        }
        for (; i < to; ++i) s += at[i * step];
    }
    sh[share][lane] = s;
    __syncthreads();
    if (share == 0 && d < p.D) {
        s = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) s += sh[j][lane];
        if (k < W) p.dw[(int64_t)d * W + k] = s;
        else if (p.db != nullptr) p.db[d] = s;
    }
}

// One more token of each stream: the cache's W - 1 rows move up by one.  All of a thread's
// rows are loaded before the first is stored.  2048 streams of 2048 bf16 channels, 4 taps, 67 MB
// moved: 13 us, 5.1 TB/s (some of it from L2); 64 streams 2.2 us, one 1.6.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) short_conv_step(const __grid_constant__ ShortConv p) {
    constexpr int V = 4, N2 = V / 2;
    const int vecs = p.D / V, blocks = (vecs + kThreads - 1) / kThreads;
    const int b = blockIdx.x / blocks, vec = (blockIdx.x - b * blocks) * kThreads + threadIdx.x;
    if (vec >= vecs) return;
    const int col = vec * V;
    const int64_t slot = p.slots != nullptr ? p.slots[b] : b;
    f32x2 o[N2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
    if (slot >= 0 && slot < p.nslots) {          // otherwise no stream in this row: a zero output
        T* at = static_cast<T*>(p.cache) + slot * (W - 1) * p.D + col;
        Row<T, V> r[W];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) r[j].r = *reinterpret_cast<const decltype(r[j].r)*>(at + (int64_t)j * p.D);
        r[W - 1].load(static_cast<const T*>(p.x) + b * p.xs + col);
        Taps<V, W> taps;
        taps.load(p, col);
        f32x2 win[W - 1][N2], now[N2];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) r[j].get(win[j]);
        r[W - 1].get(now);
        taps.apply(win, now, o);
        activate<sizeof(T) == 4>(o, p.act);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) *reinterpret_cast<decltype(r[j].r)*>(at + (int64_t)j * p.D) = r[j + 1].r;
    }
    Row<T, V>::store(static_cast<T*>(p.out) + (int64_t)b * p.D + col, o);
}

template <typename F> cudaError_t by_width(int W, const F& f) {
    switch (W) {
        case 2: return f(std::integral_constant<int, 2>());
        case 3: return f(std::integral_constant<int, 3>());
        case 4: return f(std::integral_constant<int, 4>());
        case 5: return f(std::integral_constant<int, 5>());
        case 6: return f(std::integral_constant<int, 6>());
        case 7: return f(std::integral_constant<int, 7>());
        default: return f(std::integral_constant<int, 8>());
    }
}

unsigned grid_of(const ShortConv& p, int V) {
    const int64_t warps = (int64_t)p.items * ((p.D / V + 31) / 32);
    return (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
}

}  // namespace

// Tokens of a tile: those of 8 .. 128 (backwards 256) that take the fewest rows of turns of the
// whole GPU, a tile's start counted as 8 rows.  Long tiles re-read fewer rows, short ones share
// few rows out among more SMs, and a last turn that is nearly empty costs as much as a full one: 16384 bf16 tokens of
// 2048 channels, tiles of 64 (1.3 turns), 88 (one): 31.8, 27.2 us; of 5120, 64 (4.2), 72 (3): 63,
// 59; backwards fp32, 128 (2.2), 144 (2): 84, 77.
int short_conv_tile(int64_t T, int D, int W, int dtype, bool backward, int sms) {
    const int64_t warps = (D / (backward ? kBwdVec : kFwdVec) + 31) / 32;
    const int64_t resident = (int64_t)sms * ctas_per_sm(W, dtype == SSD_BF16 ? 2 : 4, backward);
    int best = 8;
    int64_t least = INT64_MAX;
    for (int tile = 8; tile <= (backward ? 256 : 128); tile += 8) {
        const int64_t ctas = ((T + tile - 1) / tile * warps + kThreads / 32 - 1) / (kThreads / 32);
        const int64_t rows = (ctas + resident - 1) / resident * (tile + 8);
        if (rows < least) {
            least = rows;
            best = tile;
        }
    }
    return best;
}

cudaError_t launch_short_conv_fwd(ShortConv& p, int W, int dtype, int sms, cudaStream_t stream) {
    p.TT = short_conv_tile(p.T, p.D, W, dtype, false, sms);
    p.tiles = (p.T + p.TT - 1) / p.TT;
    p.items = p.tiles + (p.fin != nullptr ? p.nseq : 0);
    if (p.items == 0) return cudaSuccess;
    const unsigned grid = grid_of(p, kFwdVec);
    return by_width(W, [&](auto w) {
        if (dtype == SSD_BF16) short_conv_fwd<__nv_bfloat16, decltype(w)::value><<<grid, kThreads, 0, stream>>>(p);
        else short_conv_fwd<float, decltype(w)::value><<<grid, kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

cudaError_t launch_short_conv_bwd(ShortConv& p, int W, int dtype, int sms, cudaStream_t stream) {
    p.TT = short_conv_tile(p.T, p.D, W, dtype, true, sms);
    p.tiles = (p.T + p.TT - 1) / p.TT;
    p.items = p.tiles + (p.dinit != nullptr ? p.nseq : 0);
    if (p.items > 0) {
        const unsigned grid = grid_of(p, kBwdVec);
        const cudaError_t e = by_width(W, [&](auto w) {
            if (dtype == SSD_BF16) short_conv_bwd<__nv_bfloat16, decltype(w)::value><<<grid, kThreads, 0, stream>>>(p);
            else short_conv_bwd<float, decltype(w)::value><<<grid, kThreads, 0, stream>>>(p);
            return cudaGetLastError();
        });
        if (e != cudaSuccess) return e;
    }
    short_conv_sum<<<dim3((unsigned)((p.D + 31) / 32), (unsigned)(W + 1)), 256, 0, stream>>>(p, W);
    return cudaGetLastError();
}

cudaError_t launch_short_conv_step(const ShortConv& p, int W, int dtype, cudaStream_t stream) {
    const unsigned grid = (unsigned)(p.batch * ((p.D / 4 + kThreads - 1) / kThreads));
    return by_width(W, [&](auto w) {
        if (dtype == SSD_BF16) short_conv_step<__nv_bfloat16, decltype(w)::value><<<grid, kThreads, 0, stream>>>(p);
        else short_conv_step<float, decltype(w)::value><<<grid, kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

}  // namespace ssd
