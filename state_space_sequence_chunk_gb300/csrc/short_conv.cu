// short_conv.cu -- depthwise causal convolution over packed, token-major rows, with
// its activation, its gradient and its form for single tokens.
//
// Per channel and sequence, with W taps and the W - 1 rows before the sequence from
// its initial state (0 without one):
//     p_t = bias + sum_k w_k x_{t-W+1+k},    o_t = a(p_t),  a(p) = p or p sigmoid(p)
//     g_t = do_t a'(p_t),  dx_t = sum_k w_k g_{t+W-1-k},  dw_k = sum_t g_t x_{t-W+1+k}
// Bound by HBM: each row read once and written once.  A thread owns a vector of
// channels (a warp 512 or 256 contiguous bytes of a row) and walks a tile of tokens
// with the last W - 1 rows in registers, eight rows' loads in flight while eight are
// computed; the W - 1 rows before a tile are read again (from L2, mostly).  Sequences
// begin and end anywhere in a tile: the walk swaps its window there.
#include <type_traits>

#include "short_conv.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;        // rows loaded ahead

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float sigmoid(float z) { return rcp(1.f + ex2(-z * kLog2e)); }

// V channels of a row: as loaded, and as pairs of floats.
template <typename T, int V> struct Row;
template <> struct Row<__nv_bfloat16, 8> {
    uint4 r;
    __device__ void load(const __nv_bfloat16* p) { r = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ void zero() { r = make_uint4(0u, 0u, 0u, 0u); }
    __device__ void get(f32x2 (&v)[4]) const {
        v[0] = pair(r.x << 16, r.x & 0xFFFF0000u); v[1] = pair(r.y << 16, r.y & 0xFFFF0000u);
        v[2] = pair(r.z << 16, r.z & 0xFFFF0000u); v[3] = pair(r.w << 16, r.w & 0xFFFF0000u);
    }
    __device__ static void store(__nv_bfloat16* p, const f32x2 (&v)[4]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3]));
    }
};
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
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float* at = p.w + (int64_t)(col + 2 * i) * W;
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][i] = pair(__ldg(at + k), __ldg(at + W + k));
            b[i] = p.bias != nullptr ? pair(__ldg(p.bias + col + 2 * i), __ldg(p.bias + col + 2 * i + 1)) : pair(0.f, 0.f);
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
template <int N2> __device__ __forceinline__ void activate(f32x2 (&v)[N2], int act) {
    if (act == SSD_ACT_NONE) return;
#pragma unroll
    for (int i = 0; i < N2; ++i) {
        float a, b;
        unpair(v[i], a, b);
        v[i] = pair(a * sigmoid(a), b * sigmoid(b));
    }
}
// g = do a'(p): silu' = s (1 + p (1 - s)) with s = sigmoid(p)
template <int N2> __device__ __forceinline__ void back(f32x2 (&g)[N2], const f32x2 (&pre)[N2], int act) {
    if (act == SSD_ACT_NONE) return;
#pragma unroll
    for (int i = 0; i < N2; ++i) {
        float a, b, ga, gb;
        unpair(pre[i], a, b);
        unpair(g[i], ga, gb);
        const float sa = sigmoid(a), sb = sigmoid(b);
        g[i] = pair(ga * sa * fmaf(a, 1.f - sa, 1.f), gb * sb * fmaf(b, 1.f - sb, 1.f));
    }
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads) short_conv_fwd(const __grid_constant__ ShortConv p) {
    constexpr int V = 16 / sizeof(T), N2 = V / 2;
    const int vecs = p.D / V, blocks = (vecs + kThreads - 1) / kThreads;
    const int item = blockIdx.x / blocks, vec = (blockIdx.x - item * blocks) * kThreads + threadIdx.x;
    const bool in = vec < vecs;
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
    int s = find(p, t0), lo = 0, hi = p.T;
    if (s < p.nseq) bounds(p, s, lo, hi);
    if (!in) return;
    const T* x = static_cast<const T*>(p.x) + col;
    T* out = static_cast<T*>(p.out) + col;
    Row<T, V> ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (t0 + i < t1) ahead[i].load(x + (t0 + i) * p.xs);
    Taps<V, W> taps;
    taps.load(p, col);
    f32x2 win[W - 1][N2];
    auto enter = [&](int t) {                    // the window before row t of sequence s
        Row<T, V> r[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            if (s < p.nseq) row_of<T, V>(p, r[j], W, s, lo, t - (W - 1) + j, col);
            else r[j].zero();
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) r[j].get(win[j]);
    };
    enter(t0);
    for (int t = t0; t < t1; t += kAhead) {
        Row<T, V> cur[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            cur[i] = ahead[i];
            if (t + kAhead + i < t1) ahead[i].load(x + (t + kAhead + i) * p.xs);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (t + i < t1) {
                if (t + i == hi) {               // the next sequence that has rows, or none
                    while (++s < p.nseq) {
                        bounds(p, s, lo, hi);
                        if (hi > t + i) break;
                    }
                    if (s >= p.nseq) hi = p.T;
                    enter(t + i);
                }
                f32x2 now[N2], o[N2];
                cur[i].get(now);
                if (s < p.nseq) {
                    taps.apply(win, now, o);
                    activate(o, p.act);
                    shift(win, now);
                } else {
#pragma unroll
                    for (int k = 0; k < N2; ++k) o[k] = pair(0.f, 0.f);
                }
                Row<T, V>::store(out + (int64_t)(t + i) * p.D, o);
            }
        }
    }
}

// The gradient.  A thread walks a tile's part of each sequence with the last rows of x
// and the unfinished rows of dx in registers (row t - j lacks the terms of g beyond t),
// and W - 1 rows further, whose g the tile's last rows of dx need.  The sums for dw and
// db go into one row of partial sums per tile.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) short_conv_bwd(const __grid_constant__ ShortConv p) {
    constexpr int V = 4, N2 = 2;
    const int vecs = p.D / V, blocks = (vecs + kThreads - 1) / kThreads;
    const int item = blockIdx.x / blocks, vec = (blockIdx.x - item * blocks) * kThreads + threadIdx.x;
    const bool in = vec < vecs;
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
                back(g, pre, p.act);
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
            const f32x2 zero[N2] = {z2, z2};
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
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (a + i < lim) {
                xa[i].load(x + (a + i) * p.xs);
                da[i].load(dout + (int64_t)(a + i) * p.D);
            }
        for (int t = a; t < lim; t += kAhead) {
            Row<T, V> xc[kAhead], dc[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                xc[i] = xa[i];
                dc[i] = da[i];
                if (t + kAhead + i < lim) {
                    xa[i].load(x + (t + kAhead + i) * p.xs);
                    da[i].load(dout + (int64_t)(t + kAhead + i) * p.D);
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (t + i < lim) {
                    f32x2 now[N2], g[N2], pre[N2];
                    xc[i].get(now);
                    dc[i].get(g);
                    taps.apply(win, now, pre);
                    back(g, pre, p.act);
#pragma unroll
                    for (int k = 0; k < N2; ++k) {
                        if (t + i < b) {
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
                    const int r = t + i - (W - 1);
                    if (r >= a) Row<T, V>::store(dx + (int64_t)r * p.D, acc[W - 1]);
                }
            }
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
    for (int j = 0; j < W; ++j)
        *reinterpret_cast<ulonglong2*>(part + (int64_t)j * p.D) = make_ulonglong2(dw[j][0], dw[j][1]);
    *reinterpret_cast<ulonglong2*>(part + (int64_t)W * p.D) = make_ulonglong2(db[0], db[1]);
}

// dw and db: the tiles' sums added in the tiles' order, in eight shares.
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

// One more token of each stream: the cache's W - 1 rows move up by one.
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
        activate(o, p.act);
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

inline int64_t blocks_of(int D, int V) { return (D / V + kThreads - 1) / kThreads; }

}  // namespace

int short_conv_tile(int64_t T, int D, int dtype, bool backward, int sms) {
    // long tiles re-read fewer rows; short ones where the long ones would leave SMs idle
    const int64_t per = blocks_of(D, backward || dtype == SSD_F32 ? 4 : 8);
    int tile = backward ? 64 : 32;
    while (tile > 8 && (T + tile - 1) / tile * per < 4 * sms) tile /= 2;
    return tile;
}

cudaError_t launch_short_conv_fwd(ShortConv& p, int W, int dtype, int sms, cudaStream_t stream) {
    p.TT = short_conv_tile(p.T, p.D, dtype, false, sms);
    p.tiles = (p.T + p.TT - 1) / p.TT;
    const int64_t items = p.tiles + (p.fin != nullptr ? (int64_t)p.nseq : 0);
    if (items == 0) return cudaSuccess;
    const unsigned grid = (unsigned)(items * blocks_of(p.D, dtype == SSD_BF16 ? 8 : 4));
    return by_width(W, [&](auto w) {
        if (dtype == SSD_BF16) short_conv_fwd<__nv_bfloat16, decltype(w)::value><<<grid, kThreads, 0, stream>>>(p);
        else short_conv_fwd<float, decltype(w)::value><<<grid, kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

cudaError_t launch_short_conv_bwd(ShortConv& p, int W, int dtype, int sms, cudaStream_t stream) {
    p.TT = short_conv_tile(p.T, p.D, dtype, true, sms);
    p.tiles = (p.T + p.TT - 1) / p.TT;
    const int64_t items = p.tiles + (p.dinit != nullptr ? (int64_t)p.nseq : 0);
    if (items > 0) {
        const unsigned grid = (unsigned)(items * blocks_of(p.D, 4));
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
    const unsigned grid = (unsigned)(p.batch * blocks_of(p.D, 4));
    return by_width(W, [&](auto w) {
        if (dtype == SSD_BF16) short_conv_step<__nv_bfloat16, decltype(w)::value><<<grid, kThreads, 0, stream>>>(p);
        else short_conv_step<float, decltype(w)::value><<<grid, kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    });
}

}  // namespace ssd
