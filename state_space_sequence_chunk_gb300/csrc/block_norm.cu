// block_norm.cu -- the norms before and after a block, fused with the block's
// gate and residual scale, and their gradient.
//
// Per row (token) of width D, with a(z) the gate (SiLU, sigmoid or none) and
// the block's output y normalised in `ngroups` groups of its columns:
//     yh = y rsqrt(mean_g(y^2) + eps)
//     r' = r + alpha o w_post o a(z) o yh          (residual stream after the block)
//     n  = w_pre o r' rsqrt(mean(r'^2) + eps)      (input of the next block)
// Gradient, with dr' and dn given, rh = r' rsqrt(...), e = w_pre o dn:
//     g   = dr' + rsqrt(...) (e - rh mean(e o rh))                     = dr
//     u   = g o alpha o w_post o a(z);   dy = rsqrt_g (u - yh mean_g(u o yh))
//     dz  = g o alpha o w_post o yh o a'(z)
//     dw_pre = sum_t dn o rh;   E = sum_t g o a(z) o yh;
//     dw_post = alpha o E;      dalpha = w_post o E
// r' is recomputed from r, y and z in fp32, so that the gradient reads no
// rounded copy of it.
//
// Both directions are bound by HBM: 5 and 8 tensors of the input's size.  A row
// is read once and stays in registers, as it was loaded (bf16 pairs), between
// its reductions; columns are held as vectors of eight.  The weights are read
// where they are used: 12 bytes a column from L1, against 10 to 32 bytes of HBM
// traffic, and the registers they would take hold more rows in flight instead.
// Forwards, a CTA (or, for rows of up to 512 columns, a warp) runs one row.
// Backwards, CTAs are persistent: a thread keeps the same columns for all its
// rows and adds its columns' sums in shared memory; each CTA leaves one partial
// sum, and a second kernel adds those in a fixed order.
//
// Forwards, 16384 rows of 5120 bf16 columns with an fp32 residual stream: 190 us, 92 %
// of the copy rate.  Both directions, 16384 x 2048 bf16: 199 us, 65 %: backwards a row's
// loads are in flight only behind the row before it, and its 3 CTAs an SM do not cover
// that (37 % of the warps, 49 % of the DRAM rate under the profiler).  That is the gradient's
// best form; its share of the copy rate, without the forward pass, is 58 % at 2048
// columns, 47 and 52 % at 4096 and 5120 (one CTA of 512 or 640 threads an SM), 36 to 42 % at
// 6144 and 8192 (two vectors a thread, which spill 172 bytes) and 28 % at 12288 (four
// vectors, 1.5 KB).
#include "block_norm.cuh"
#include "f32x2.cuh"
#include "sm100_ptx.cuh"

namespace ssd {
namespace {

// Eight elements as loaded.
template <typename T> struct Raw;
template <> struct Raw<float> { float4 a, b; };
template <> struct Raw<__nv_bfloat16> { uint4 a; };
__device__ __forceinline__ void zero(Raw<float>& r) { r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f); }
__device__ __forceinline__ void zero(Raw<__nv_bfloat16>& r) { r.a = make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ void load(Raw<float>& r, const float* p) {
    r.a = __ldg(reinterpret_cast<const float4*>(p));
    r.b = __ldg(reinterpret_cast<const float4*>(p) + 1);
}
__device__ __forceinline__ void load(Raw<__nv_bfloat16>& r, const __nv_bfloat16* p) {
    r.a = __ldg(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ f32x2 widen(uint32_t v) { return pair(v << 16, v & 0xFFFF0000u); }
__device__ __forceinline__ void unpack(const Raw<float>& r, f32x2 (&f)[4]) {
    f[0] = pair(r.a.x, r.a.y);
    f[1] = pair(r.a.z, r.a.w);
    f[2] = pair(r.b.x, r.b.y);
    f[3] = pair(r.b.z, r.b.w);
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16>& r, f32x2 (&f)[4]) {
    f[0] = widen(r.a.x);
    f[1] = widen(r.a.y);
    f[2] = widen(r.a.z);
    f[3] = widen(r.a.w);
}
__device__ __forceinline__ void load8(const float* p, f32x2 (&f)[4]) {
    Raw<float> r;
    load(r, p);
    unpack(r, f);
}
__device__ __forceinline__ f32x2 both(float v) { return pair(v, v); }
// alpha o w_post of eight columns
__device__ __forceinline__ void scale8(const NormParams& p, int j, f32x2 (&cw)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) cw[e] = both(1.f);
    if (p.w_post) load8(p.w_post + 8 * j, cw);
    if (p.alpha) {
        f32x2 t[4];
        load8(p.alpha + 8 * j, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) cw[e] = mul2(cw[e], t[e]);
    }
}
__device__ __forceinline__ void store8(float* p, const f32x2 (&f)[4]) {
    reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(f[0], f[1]);
    reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(f[2], f[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const f32x2 (&f)[4]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}
__device__ __forceinline__ float sum2(f32x2 v) {
    float a, b;
    unpair(v, a, b);
    return a + b;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the row's threads.  kWarp: the row is one warp.  Else the CTA; `buf`
// (32 floats) must not be reused until a barrier later than this one.
template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float* buf) {
    v = warp_sum(v);
    if (kWarp) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) buf[warp] = v;
    __syncthreads();
    return warp_sum(lane < nw ? buf[lane] : 0.f);
}

// Per-group sums of part[i] (one per vector of eight columns) for each of this
// thread's vectors.  Three forms: one group (a row sum), groups of 8, 16 .. 256
// columns that lie within a warp's consecutive vectors (shuffles), and any
// other (through shared memory: grp[] holds a float for each vector, then
// behind it one for each group).
template <int NV, bool kWarp>
__device__ __forceinline__ void group_sum(const NormParams& p, float (&part)[NV], float* buf, float* grp,
                                          int first, int stride) {
    if (p.ngroups == 1) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) v += part[i];
        v = row_sum<kWarp>(v, buf);
#pragma unroll
        for (int i = 0; i < NV; ++i) part[i] = v;
        return;
    }
    if (p.gvecs <= 32 && (p.gvecs & (p.gvecs - 1)) == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            for (int o = 1; o < p.gvecs; o <<= 1) part[i] += __shfl_xor_sync(0xffffffffu, part[i], o);
        return;
    }
    const int lane = threadIdx.x & 31, warp = kWarp ? 0 : threadIdx.x >> 5,
              nw = kWarp ? 1 : blockDim.x >> 5;
    float* sums = grp + p.vecs;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (first + i * stride < p.vecs) grp[first + i * stride] = part[i];
    if (kWarp) __syncwarp(); else __syncthreads();
    for (int g = warp; g < p.ngroups; g += nw) {
        float v = 0.f;
        for (int j = lane; j < p.gvecs; j += 32) v += grp[g * p.gvecs + j];
        v = warp_sum(v);
        if (lane == 0) sums[g] = v;
    }
    if (kWarp) __syncwarp(); else __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = first + i * stride;
        if (j < p.vecs) part[i] = sums[j / p.gvecs];
    }
    if (kWarp) __syncwarp(); else __syncthreads();
}

// sigmoid(z).  Beside bf16 inputs the fast exponential and division serve (errors
// of a few 2^-23 of the value, and of z 2^-24 in the exponent); fp32 inputs get
// the exact ones.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
    if (sizeof(T) == 2) return __fdividef(1.f, 1.f + __expf(-z));
    return 1.f / (1.f + expf(-z));
}
// s = sigmoid(z) (1 without a gate), m = z for SiLU and 1 else: the gate is s m,
// its derivative s ([SiLU] + m (1 - s)).
template <typename T>
__device__ __forceinline__ f32x2 sigmoid2(int kind, f32x2 z) {
    if (kind == SSD_GATE_NONE) return both(1.f);
    float a, b;
    unpair(z, a, b);
    return pair(sigmoid<T>(a), sigmoid<T>(b));
}
__device__ __forceinline__ f32x2 factor2(int kind, f32x2 z) { return kind == SSD_GATE_SILU ? z : both(1.f); }

template <typename T, typename R, int NV, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 128 : 512, !kWarp && NV == 2 && sizeof(T) == 2 ? 2 : 1)
block_norm_fwd(const __grid_constant__ NormParams p) {
    extern __shared__ float sm[];
    const int first = kWarp ? threadIdx.x & 31 : threadIdx.x, stride = kWarp ? 32 : blockDim.x;
    const int sub = kWarp ? threadIdx.x >> 5 : 0;
    float* grp = sm + 96 + (kWarp ? sub * p.grp_floats : 0);
    const float inv_gw = 1.f / (float)(8 * p.gvecs), inv_d = 1.f / (float)(8 * p.vecs);
    const int64_t row = kWarp ? (int64_t)blockIdx.x * (blockDim.x >> 5) + sub : (int64_t)blockIdx.x;
    if (row >= p.T) return;   // a whole row's threads
    Raw<T> y[NV], z[NV];
    Raw<R> r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = first + i * stride;
        zero(y[i]);
        zero(z[i]);
        zero(r[i]);
        if (j < p.vecs) {
            load(y[i], static_cast<const T*>(p.y) + row * p.ys + 8 * j);
            if (p.gate != SSD_GATE_NONE) load(z[i], static_cast<const T*>(p.z) + row * p.zs + 8 * j);
            load(r[i], static_cast<const R*>(p.r) + row * p.D + 8 * j);
        }
    }
    float part[NV];
    f32x2 rp[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        f32x2 f[4], v = 0ull;
        unpack(y[i], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) v = fma2(f[e], f[e], v);
        part[i] = sum2(v);
    }
    group_sum<NV, kWarp>(p, part, sm, grp, first, stride);
    f32x2 sq2 = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = first + i * stride;
        if (j < p.vecs) {
            const float rs = rsqrtf(part[i] * inv_gw + p.eps);
            if (p.rstd_post && j % p.gvecs == 0) p.rstd_post[row * p.ngroups + j / p.gvecs] = rs;
            f32x2 cw[4], yf[4], zf[4];
            scale8(p, j, cw);
            unpack(y[i], yf);
            unpack(z[i], zf);
            unpack(r[i], rp[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x2 a = mul2(sigmoid2<T>(p.gate, zf[e]), factor2(p.gate, zf[e]));
                rp[i][e] = fma2(mul2(cw[e], a), mul2(yf[e], both(rs)), rp[i][e]);
                sq2 = fma2(rp[i][e], rp[i][e], sq2);
            }
            store8(static_cast<R*>(p.r_out) + row * p.D + 8 * j, rp[i]);
        }
    }
    const float sq = sum2(sq2);
    const float q = rsqrtf(row_sum<kWarp>(sq, sm + 32) * inv_d + p.eps);
    if (p.rstd_pre && first == 0) p.rstd_pre[row] = q;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = first + i * stride;
        if (j < p.vecs) {
            f32x2 wp[4];
            load8(p.w_pre + 8 * j, wp);
#pragma unroll
            for (int e = 0; e < 4; ++e) rp[i][e] = mul2(rp[i][e], mul2(wp[e], both(q)));
            store8(static_cast<T*>(p.n) + row * p.D + 8 * j, rp[i]);
        }
    }
}

// One row of the gradient's inputs, as loaded.
template <typename T, typename R, int NV>
struct Row {
    Raw<T> y[NV], z[NV], dn[NV];
    Raw<R> r[NV], g[NV];
    float rs[NV], q;
    __device__ __forceinline__ void fetch(const NormParams& p, int64_t row, int first, int stride) {
        q = __ldg(p.rstd_pre + row);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
            if (j < p.vecs) {
                load(y[i], static_cast<const T*>(p.y) + row * p.ys + 8 * j);
                if (p.gate != SSD_GATE_NONE) load(z[i], static_cast<const T*>(p.z) + row * p.zs + 8 * j);
                load(r[i], static_cast<const R*>(p.r) + row * p.D + 8 * j);
                load(dn[i], static_cast<const T*>(p.dn) + row * p.D + 8 * j);
                load(g[i], static_cast<const R*>(p.dr_out) + row * p.D + 8 * j);
                rs[i] = __ldg(p.rstd_post + row * p.ngroups + j / p.gvecs);
            }
        }
    }
    __device__ __forceinline__ void clear() {
        q = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            zero(y[i]); zero(z[i]); zero(dn[i]); zero(r[i]); zero(g[i]);
            rs[i] = 0.f;
        }
    }
};

// The columns' sums lie in shared memory: per vector four pairs of pairs a thread
// (E's eight columns, then w_pre's), strided by the block.  CTAs of up to 256
// threads are bounded to 80 registers, three to an SM (fp32: two).  (Measured at 16384 x 2048
// bf16 and slower: four to an SM, which spills; weights and sums in registers, the
// next row fetched ahead, two to an SM.)
template <typename T, typename R, int NV, bool kWarp, bool kSmall>
__global__ void __launch_bounds__(kWarp ? 128 : kSmall ? 256 : 640, kWarp ? 4 : !kSmall ? 1 : sizeof(T) == 2 ? 3 : 2)
block_norm_bwd(const __grid_constant__ NormParams p) {
    extern __shared__ float sm[];
    grid_launch_dependents();   // the partials' sum may set itself up
    const int first = kWarp ? threadIdx.x & 31 : threadIdx.x, stride = kWarp ? 32 : blockDim.x;
    const int rpb = kWarp ? blockDim.x >> 5 : 1, sub = kWarp ? threadIdx.x >> 5 : 0;
    float* grp = sm + 96 + (kWarp ? sub * p.grp_floats : 0);
    ulonglong2* acc = reinterpret_cast<ulonglong2*>(sm + 96 + ((p.grp_floats * rpb + 3) & ~3)) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) acc[i * blockDim.x] = make_ulonglong2(0ull, 0ull);
    const auto add8 = [&](int at, const f32x2 (&f)[4]) {
        ulonglong2 a = acc[at * blockDim.x], b = acc[(at + 1) * blockDim.x];
        a.x = add2(a.x, f[0]);
        a.y = add2(a.y, f[1]);
        b.x = add2(b.x, f[2]);
        b.y = add2(b.y, f[3]);
        acc[at * blockDim.x] = a;
        acc[(at + 1) * blockDim.x] = b;
    };
    const float inv_gw = 1.f / (float)(8 * p.gvecs), inv_d = 1.f / (float)(8 * p.vecs);
    const int64_t step = (int64_t)gridDim.x * rpb;
    // the last reduction's buffer alternates: a row may have no other barrier
    float* buf = sm + 32;
    Row<T, R, NV> cur;
    cur.clear();
    for (int64_t row = (int64_t)blockIdx.x * rpb + sub; row < p.T; row += step) {
        cur.fetch(p, row, first, stride);
        // rh = r' rsqrt; the mean of e o rh over the row
        f32x2 dot2 = 0ull, u[NV][4], sg[NV][4];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
            if (j < p.vecs) {
                f32x2 cw[4], wp[4], yf[4], zf[4], dnf[4], t[4];
                scale8(p, j, cw);
                load8(p.w_pre + 8 * j, wp);
                unpack(cur.y[i], yf);
                unpack(cur.z[i], zf);
                unpack(cur.r[i], u[i]);
                unpack(cur.dn[i], dnf);
                const f32x2 rs2 = both(cur.rs[i]), q2 = both(cur.q);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sg[i][e] = sigmoid2<T>(p.gate, zf[e]);
                    const f32x2 a = mul2(sg[i][e], factor2(p.gate, zf[e]));
                    u[i][e] = mul2(fma2(mul2(cw[e], a), mul2(yf[e], rs2), u[i][e]), q2);
                    t[e] = mul2(dnf[e], u[i][e]);
                    dot2 = fma2(wp[e], t[e], dot2);
                }
                add8(4 * i + 2, t);
            }
        }
        const float dot = row_sum<kWarp>(sum2(dot2), buf) * inv_d;
        buf = buf == sm + 32 ? sm + 64 : sm + 32;
        float part[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
            part[i] = 0.f;
            if (j < p.vecs) {
                f32x2 cw[4], wp[4], yf[4], zf[4], dnf[4], gf[4], t[4], v = 0ull;
                scale8(p, j, cw);
                load8(p.w_pre + 8 * j, wp);
                unpack(cur.y[i], yf);
                unpack(cur.z[i], zf);
                unpack(cur.dn[i], dnf);
                unpack(cur.g[i], gf);
                const f32x2 rs2 = both(cur.rs[i]), q2 = both(cur.q), ndot2 = both(-dot);
                const f32x2 silu = both(p.gate == SSD_GATE_SILU ? 1.f : 0.f), one = both(1.f), neg = both(-1.f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x2 m = factor2(p.gate, zf[e]), s = sg[i][e];
                    const f32x2 yh = mul2(yf[e], rs2);
                    gf[e] = fma2(q2, fma2(wp[e], dnf[e], mul2(u[i][e], ndot2)), gf[e]);
                    const f32x2 ga = mul2(gf[e], mul2(s, m));
                    t[e] = mul2(ga, yh);
                    u[i][e] = mul2(ga, cw[e]);
                    const f32x2 da = mul2(s, fma2(m, fma2(s, neg, one), silu));
                    zf[e] = mul2(mul2(gf[e], cw[e]), mul2(yh, da));
                    v = fma2(u[i][e], yh, v);
                }
                part[i] = sum2(v);
                add8(4 * i, t);
                store8(static_cast<R*>(p.dr) + row * p.D + 8 * j, gf);
                if (p.gate != SSD_GATE_NONE) store8(static_cast<T*>(p.dz) + row * p.D + 8 * j, zf);
            }
        }
        group_sum<NV, kWarp>(p, part, sm, grp, first, stride);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
            if (j < p.vecs) {
                const f32x2 rs2 = both(cur.rs[i]), nm2 = both(-part[i] * inv_gw);
                f32x2 yf[4];
                unpack(cur.y[i], yf);
#pragma unroll
                for (int e = 0; e < 4; ++e) u[i][e] = mul2(rs2, fma2(mul2(yf[e], rs2), nm2, u[i][e]));
                store8(static_cast<T*>(p.dy) + row * p.D + 8 * j, u[i]);
            }
        }
    }
    float* pe = p.partial + ((int64_t)blockIdx.x * rpb + sub) * 2 * p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = first + i * stride;
        if (j < p.vecs) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                reinterpret_cast<ulonglong2*>(pe + (x >> 1) * p.D + 8 * j)[x & 1] = acc[(4 * i + x) * blockDim.x];
        }
    }
}

// Column sums of the partials: a CTA has 32 columns of E (blockIdx.y 0) or of
// w_pre's sums, and 16 strided runs of the partials, joined in a fixed order.
__global__ void __launch_bounds__(512) block_norm_reduce(const __grid_constant__ NormParams p, int nparts) {
    __shared__ float sh[16][33];
    const int x = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    grid_dependency_wait();
    float v = 0.f;
    if (c < p.D) {
        const float* src = p.partial + (int64_t)blockIdx.y * p.D + c;
#pragma unroll 8
        for (int i = w; i < nparts; i += 16) v += src[(int64_t)i * 2 * p.D];
    }
    sh[w][x] = v;
    __syncthreads();
    if (w != 0 || c >= p.D) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += sh[i][x];
    if (blockIdx.y == 1) {
        p.dw_pre[c] = v;
    } else {
        if (p.dw_post) p.dw_post[c] = (p.alpha ? p.alpha[c] : 1.f) * v;
        if (p.dalpha) p.dalpha[c] = (p.w_post ? p.w_post[c] : 1.f) * v;
    }
}

struct Cut {
    int nv, threads;
    bool warp;
};
// Vectors per thread and threads per row: rows of up to 512 columns take one
// warp each (four to a CTA), longer ones a CTA.  Backwards fewer vectors fit a
// thread's registers.
Cut cut_of(int vecs, bool backward) {
    if (vecs <= 64) return {vecs <= 32 ? 1 : 2, 128, true};
    const int nv = backward ? (vecs <= 640 ? 1 : vecs <= 1280 ? 2 : 4) : vecs <= 128 ? 1 : vecs <= 1024 ? 2 : 4;
    const int per = (vecs + nv - 1) / nv;
    return {nv, (per + 31) / 32 * 32, false};
}

size_t shared_bytes(const NormParams& p, const Cut& c, bool backward) {
    const int rpb = c.warp ? c.threads / 32 : 1;
    const size_t grp = 96 + ((size_t)p.grp_floats * rpb + 3) / 4 * 4;
    return (grp + (backward ? (size_t)16 * c.nv * c.threads : 0)) * 4;
}

template <typename T, typename R>
cudaError_t go(NormParams& p, bool backward, int64_t grid, cudaStream_t stream) {
    const Cut c = cut_of(p.vecs, backward);
    const size_t bytes = shared_bytes(p, c, backward);
    void (*k)(NormParams) = nullptr;
    if (backward)
        k = c.warp ? (c.nv == 1 ? block_norm_bwd<T, R, 1, true, true> : block_norm_bwd<T, R, 2, true, true>)
          : c.nv == 1 ? (c.threads <= 256 ? block_norm_bwd<T, R, 1, false, true> : block_norm_bwd<T, R, 1, false, false>)
          : c.nv == 2 ? block_norm_bwd<T, R, 2, false, false> : block_norm_bwd<T, R, 4, false, false>;
    else
        k = c.warp ? (c.nv == 1 ? block_norm_fwd<T, R, 1, true> : block_norm_fwd<T, R, 2, true>)
          : c.nv == 1 ? block_norm_fwd<T, R, 1, false>
          : c.nv == 2 ? block_norm_fwd<T, R, 2, false> : block_norm_fwd<T, R, 4, false>;
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != cudaSuccess) return e;
    }
    k<<<(unsigned)grid, c.threads, bytes, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t dispatch(NormParams& p, int dtype, int rdtype, bool backward, int64_t grid, cudaStream_t st) {
    if (dtype == SSD_BF16)
        return rdtype == SSD_BF16 ? go<__nv_bfloat16, __nv_bfloat16>(p, backward, grid, st)
                                  : go<__nv_bfloat16, float>(p, backward, grid, st);
    return go<float, float>(p, backward, grid, st);
}

}  // namespace

int block_norm_grid(int64_t T, int vecs, int dtype, int sms) {
    const Cut c = cut_of(vecs, true);
    const int rpb = c.warp ? c.threads / 32 : 1;
    const int per = c.warp ? 4 : c.threads <= 256 ? (dtype == SSD_BF16 ? 3 : 2) * 256 / c.threads : 640 / c.threads;   // by registers
    const int64_t rows = (T + rpb - 1) / rpb, full = (int64_t)sms * per;
    return (int)(rows < full ? rows : full);
}

int block_norm_parts(int64_t T, int vecs, int dtype, int sms) {
    const Cut c = cut_of(vecs, true);
    return block_norm_grid(T, vecs, dtype, sms) * (c.warp ? c.threads / 32 : 1);
}

cudaError_t launch_block_norm_fwd(NormParams& p, int dtype, int rdtype, cudaStream_t st) {
    const Cut c = cut_of(p.vecs, false);
    const int rpb = c.warp ? c.threads / 32 : 1;
    return dispatch(p, dtype, rdtype, false, (p.T + rpb - 1) / rpb, st);
}

cudaError_t launch_block_norm_bwd(NormParams& p, int dtype, int rdtype, int sms, cudaStream_t st) {
    const int grid = p.T > 0 ? block_norm_grid(p.T, p.vecs, dtype, sms) : 0;
    if (grid > 0) {
        const cudaError_t e = dispatch(p, dtype, rdtype, true, grid, st);
        if (e != cudaSuccess) return e;
    }
    const int parts = grid > 0 ? block_norm_parts(p.T, p.vecs, dtype, sms) : 0;
    return launch_chained(block_norm_reduce, dim3((unsigned)(p.D + 31) / 32, 2), dim3(512), 0, st, grid > 0, p, parts);
}

}  // namespace ssd
