// linattn_tc.cu -- linear attention with a decay for each head on the tcgen05
// tensor cores (bf16 operands, fp32 accumulation and state).
//
// One chain is (range of a sequence, head, 64 columns of c), walked in chunks of
// 128 tokens.  With i, j the rows of a chunk (counted from its end when the walk
// is backwards), n its tokens and X the state before it:
//     W   = A B^T                                   128 x 128 x DK
//     P   = s_in W o lam^{-j} [i >= j]              (bf16, tensor memory)
//     out = s_out lam^i o (A (lam X) + P C)         128 x 64 x DK, 128 x 64 x 128
//     U   = B^T (s_in lam^{-j} o C)                 DK x 64 x 128
//     X   <- lam^n X + lam^{n-1} U
// (backwards the decay of X and U is one step longer).  Rows and columns carry
// the decay as separate factors, so that out is one accumulator and P costs one
// product for each element; that is safe while lam^-127 <= 2^40.  For heads that
// forget faster the exact form runs: lam^{i-j} element by element, A X and P C
// in two accumulators, U with weights lam^{n-1-j}.
// Every operand is read once per chain from HBM (a and b once per 64 columns of
// c, from L2 the second time) and no state leaves the chip between chunks.
//
// Precision.  P and the X that multiplies A are rounded to bf16 (as operands of
// a product whose result is rounded to bf16).  X itself must not be: it is kept
// in fp32 registers and U is exact to fp32: C's scaled rows are cut into three
// bf16 terms of 8 bits each, multiplied side by side (N = 192) into separate
// accumulators and added from the smallest up.  X <- lam^n X + U runs on the
// CUDA cores, where it is rounded to nearest (how the tensor core's accumulator
// rounds is not documented, and a chain adds it up over hundreds of chunks).
//
// Persistent CTAs of 22 warps, one per SM:
//   0-3   P: tensor memory -> decay, mask -> tensor memory (bf16, in place)
//   4-7   C's scaled terms (a thread owns token row j); zeroes the rows of a
//         ragged chunk that belong to other tokens, whatever they hold
//   8-15  X in registers (a thread owns 32 columns of a row): bf16 copy for A X,
//         update with U, stored states
//   16-19 out (a thread owns a token row)
//   20    TMA, two stages of A, B and C tiles (80 KB each)
//   21    MMA issue: U(c), A X(c), W(c + 1), P C(c)
// The roles' loops are kept short (packed fp32 arithmetic, little unrolling): six
// codes run side by side on each scheduler, and fully unrolled they spent most of
// their time on instruction fetches.
#include <cuda.h>
#include <string.h>

#include "linattn_internal.cuh"
#include "sm100_ptx.cuh"
#include "tma_host.cuh"

namespace ssd {
namespace {

__device__ unsigned int g_la_error;  // bit 0: a bounded wait gave up

constexpr int kC = 128;                       // tokens per chunk
constexpr int kRow = 128;                     // bytes of a tile row (64 columns)
constexpr int kAtom = kC * kRow;              // 16 KB: 128 rows of 64 columns
constexpr int kThreads = 704;
constexpr int kTmaWarp = 20, kMmaWarp = 21;
constexpr int kStage = 5 * kAtom;             // A (2 atoms), B (2), C (1)
constexpr int kTerms = 3;
constexpr int kSmem = 2 * kStage + kTerms * kAtom + kAtom + 1024 + 1024;
// tensor memory columns
constexpr uint32_t kW = 0;                    // W / P, two buffers of 128
constexpr uint32_t kO = 256, kU = 320;        // out; U's three terms
// A head's decay over a chunk's 127 steps is at most 2^kSpan for the factored form.
constexpr float kSpan = 40.f;

struct TcParams {
    LaParams p;
    int nvb, items;
    unsigned int* host_err;
};
struct TcMaps {
    CUtensorMap m[3][3];   // job, operand (A, B, C)
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
// Pairs of floats in one register pair: the packed fp32 instructions do two
// elements each, rounded as the single ones.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f32x2 pair(uint32_t a, uint32_t b) {
    return pair(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ void unpair(f32x2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint32_t pack2(f32x2 v) {
    float a, b;
    unpair(v, a, b);
    return pack2(a, b);
}
__device__ __forceinline__ void bar_wg(int id) {
    asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}
__device__ __forceinline__ void st_v8(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__device__ __forceinline__ bool factored(float a2) { return a2 * -127.f <= kSpan; }
// 2^(a2 n), with the product's rounding put back: n a2 can be as large as kSpan,
// where a rounding of the exponent would be one of the result's last bits.
__device__ __forceinline__ float la_exp2(float a2, int n) {
    const float p = a2 * (float)n, e = fmaf(a2, (float)n, -p);
    const float r = exp2f(p);
    return fmaf(r, e * 0.6931471805599453f, r);
}

// One item of a CTA's list: the columns of one job, of one head, of one range.
struct Item {
    LaRange rg;
    int job, h, v0, nch;
    bool cut, last, skip;
};
template <bool kAgg>
__device__ __forceinline__ Item item_of(const TcParams& tp, int it) {
    Item r;
    __syncwarp();   // la_find is collective
    const int vb = it % tp.nvb;
    int x = it / tp.nvb;
    r.job = x % tp.p.njobs;
    x /= tp.p.njobs;
    r.h = x % tp.p.g.H;
    r.rg = la_find(tp.p.g, x / tp.p.g.H);
    r.v0 = vb * kLaCols;
    const LaJob& jb = tp.p.job[r.job];
    r.cut = tp.p.g.split && r.rg.n > 1;
    r.last = jb.rev ? r.rg.r == 0 : r.rg.r == r.rg.n - 1;
    r.skip = r.rg.seq < 0 || r.v0 >= jb.DV || (kAgg && (!r.cut || r.last || r.rg.seq == tp.p.g.nseq));
    r.nch = r.skip || r.rg.seq == tp.p.g.nseq ? 0 : (r.rg.len + kC - 1) / kC;
    return r;
}

template <bool kAgg>
__global__ void __launch_bounds__(kThreads, 1)
linattn_tc(const __grid_constant__ TcParams tp, const __grid_constant__ TcMaps maps) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* terms = smem + 2 * kStage;
    uint8_t* xs = terms + kTerms * kAtom;
    uint64_t* bars = reinterpret_cast<uint64_t*>(xs + kAtom);
    uint64_t* b_full = bars;          // [2] stage loaded (tx)
    uint64_t* b_empty = bars + 2;     // [2] stage read by every product (commit)
    uint64_t* b_wdone = bars + 4;     // [2] W computed (commit)
    uint64_t* b_pready = bars + 6;    // [2] P written (128)
    uint64_t* b_udone = bars + 8;     // U computed, terms read (commit)
    uint64_t* b_ufree = bars + 9;     // U read (256)
    uint64_t* b_vready = bars + 10;   // terms written (128)
    uint64_t* b_sready = bars + 11;   // bf16 X written (256)
    uint64_t* b_xdone = bars + 12;    // A X computed: the bf16 X may change (commit)
    uint64_t* b_odone = bars + 13;    // out computed (commit)
    uint64_t* b_ofree = bars + 14;    // out read (128)
    uint32_t* holder = reinterpret_cast<uint32_t*>(bars + 15);
    float* ptab = reinterpret_cast<float*>(bars + 16);   // [128] column factors of P

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(b_full + s), 1);
            mbar_init(smem_u32(b_empty + s), 1);
            mbar_init(smem_u32(b_wdone + s), 1);
            mbar_init(smem_u32(b_pready + s), 128);
        }
        mbar_init(smem_u32(b_udone), 1);
        mbar_init(smem_u32(b_ufree), 256);
        mbar_init(smem_u32(b_vready), 128);
        mbar_init(smem_u32(b_sready), 256);
        mbar_init(smem_u32(b_xdone), 1);
        mbar_init(smem_u32(b_odone), 1);
        mbar_init(smem_u32(b_ofree), 128);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tmem_alloc(smem_u32(holder), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;
    unsigned int* err = &g_la_error;
    const LaGeom& g = tp.p.g;
    // every role walks the same items and counts chunks in c: barrier phases
    // follow from the count alone
    int c = 0;

    if (warp == kTmaWarp) {
        for (int it = blockIdx.x; it < tp.items; it += gridDim.x) {
            const Item im = item_of<kAgg>(tp, it);
            const LaJob& jb = tp.p.job[im.job];
            if (lane == 0) {
                const int ka = (jb.DK + 63) / 64;
                const CUtensorMap* m = maps.m[im.job];
                const int ha = im.h / jb.dA, hb = im.h / jb.dB, hc = im.h / jb.dC;
                for (int x = 0; x < im.nch; ++x, ++c) {
                    const int s = c & 1, t = im.rg.t0 + (jb.rev ? im.nch - 1 - x : x) * kC;
                    mbar_wait(smem_u32(b_empty + s), ((c >> 1) & 1) ^ 1, err, 1u);
                    const uint32_t fb = smem_u32(b_full + s), st = smem_u32(smem + s * kStage);
                    mbar_arrive_expect_tx(fb, ((kAgg ? 1 : 2) * ka + 1) * kAtom);
                    for (int a = 0; a < ka; ++a) {
                        if (!kAgg) tma_load_3d(st + a * kAtom, m + 0, fb, a * 64, ha, t);
                        tma_load_3d(st + (2 + a) * kAtom, m + 1, fb, a * 64, hb, t);
                    }
                    tma_load_3d(st + 4 * kAtom, m + 2, fb, im.v0, hc, t);
                }
            }
            __syncwarp();
        }
    } else if (warp == kMmaWarp) {
        constexpr uint32_t kIdW = make_idesc(1, 128, 128, 0, 0);
        constexpr uint32_t kIdO = make_idesc(1, 128, 64, 0, 1);
        constexpr uint32_t kIdU = make_idesc(1, 128, 64 * kTerms, 1, 1);
        for (int it = blockIdx.x; it < tp.items; it += gridDim.x) {
            const Item im = item_of<kAgg>(tp, it);
            if (lane == 0) {
                const int ks = tp.p.job[im.job].DK / 16;
                const bool fac = factored(la_log2_decay(g.a, im.h));
                auto w_product = [&](int cc) {   // W of chunk cc
                    const int s = cc & 1;
                    mbar_wait(smem_u32(b_full + s), (cc >> 1) & 1, err, 1u);
                    tc_fence_after();
                    const uint32_t st = smem_u32(smem + s * kStage);
                    const uint64_t ad = smem_desc_sw128(st, 16, 8 * kRow);
                    const uint64_t bd = smem_desc_sw128(st + 2 * kAtom, 16, 8 * kRow);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        if (kk < ks) {
                            const uint64_t o = (uint64_t)(((kk / 4) * kAtom + (kk % 4) * 32) >> 4);
                            mma_f16_ss(tmem + kW + s * 128, ad + o, bd + o, kIdW, kk > 0 ? 1u : 0u);
                        }
                    mma_commit(smem_u32(b_wdone + s));
                };
                if (!kAgg && im.nch > 0) w_product(c);
                for (int x = 0; x < im.nch; ++x, ++c) {
                    const int s = c & 1, use = c >> 1;
                    const uint32_t st = smem_u32(smem + s * kStage);
                    if (kAgg) mbar_wait(smem_u32(b_full + s), use & 1, err, 1u);
                    // U = B^T (scaled C), its three terms side by side: B is read once
                    mbar_wait(smem_u32(b_vready), c & 1, err, 1u);
                    mbar_wait(smem_u32(b_ufree), (c & 1) ^ 1, err, 1u);
                    tc_fence_after();
                    {
                        const uint64_t ad = smem_desc_sw128(st + 2 * kAtom, kAtom, 8 * kRow);
                        const uint64_t bd = smem_desc_sw128(smem_u32(terms), kAtom, 8 * kRow);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const uint64_t o = (uint64_t)((kk * 16 * kRow) >> 4);
                            mma_f16_ss(tmem + kU, ad + o, bd + o, kIdU, kk > 0 ? 1u : 0u);
                        }
                    }
                    mma_commit(smem_u32(b_udone));
                    if (kAgg) {
                        mma_commit(smem_u32(b_empty + s));
                        continue;
                    }
                    // out = A X
                    mbar_wait(smem_u32(b_sready), c & 1, err, 1u);
                    mbar_wait(smem_u32(b_ofree), (c & 1) ^ 1, err, 1u);
                    tc_fence_after();
                    {
                        const uint64_t ad = smem_desc_sw128(st, 16, 8 * kRow);
                        const uint64_t bd = smem_desc_sw128(smem_u32(xs), 8 * kRow, 8 * kRow);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            if (kk < ks)
                                mma_f16_ss(tmem + kO, ad + (uint64_t)(((kk / 4) * kAtom + (kk % 4) * 32) >> 4),
                                           bd + (uint64_t)((kk * 16 * kRow) >> 4), kIdO, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(smem_u32(b_xdone));
                    // W of the next chunk before this chunk's last product, if its
                    // tiles are there: P is then built a whole chunk ahead.  Its
                    // buffer's last readers were waited for by the products above.
                    const bool next = x + 1 < im.nch;
                    const bool early = next && mbar_try_wait(smem_u32(b_full + (s ^ 1)), ((c + 1) >> 1) & 1);
                    if (early) w_product(c + 1);
                    // out += P C; in the exact form, beside P's columns in W's buffer
                    mbar_wait(smem_u32(b_pready + s), use & 1, err, 1u);
                    tc_fence_after();
                    {
                        const uint64_t bd = smem_desc_sw128(st + 4 * kAtom, 8 * kRow, 8 * kRow);
                        const uint32_t to = fac ? tmem + kO : tmem + kW + s * 128 + 64;
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            mma_f16_ts(to, tmem + kW + s * 128 + kk * 8,
                                       bd + (uint64_t)((kk * 16 * kRow) >> 4), kIdO, (fac || kk > 0) ? 1u : 0u);
                    }
                    mma_commit(smem_u32(b_odone));
                    mma_commit(smem_u32(b_empty + s));
                    if (next && !early) w_product(c + 1);
                }
            }
            __syncwarp();
        }
    } else if (warp < 4) {
        // ===================== P =====================
        if (!kAgg) {
            const int row = warp * 32 + lane;
            const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
            for (int it = blockIdx.x; it < tp.items; it += gridDim.x) {
                const Item im = item_of<kAgg>(tp, it);
                if (im.nch == 0) continue;
                const LaJob& jb = tp.p.job[im.job];
                const float a2 = la_log2_decay(g.a, im.h);
                const bool fac = factored(a2);
                bar_wg(1);                      // the table's last readers are done
                // factored: lam^{-j'} s_in; exact: lam^j (the first 32 are used) and,
                // from 32 on, lam^{31-j}
                ptab[row] = fac ? la_exp2(-a2, jb.rev ? kC - 1 - row : row) * jb.s_in
                                : exp2f(a2 * (float)(row < 32 ? row : max(63 - row, 0)));
                bar_wg(1);
                const float4* vt = reinterpret_cast<const float4*>(jb.rev ? ptab : ptab + 32);
                for (int x = 0; x < im.nch; ++x, ++c) {
                    const int s = c & 1, ci = jb.rev ? im.nch - 1 - x : x;
                    const int n = min(kC, im.rg.len - ci * kC);
                    mbar_wait(smem_u32(b_wdone + s), (c >> 1) & 1, err, 1u);
                    tc_fence_after();
                    const uint32_t base = tmem + lane_off + kW + s * 128;
                    // in place: block b's 16 packed columns lie within columns that
                    // blocks up to b held
#pragma unroll 1
                    for (int b = 0; b < 4; ++b) {
                        const int rel = jb.rev ? b - warp : warp - b;
                        uint32_t o[16];
                        if (rel < 0) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = 0u;
                        } else {
                            uint32_t v[32];
                            __syncwarp();
                            tmem_ld_x32(base + b * 32, v);
                            tmem_wait_ld();
                            if (fac) {
                                const ulonglong2* ct = reinterpret_cast<const ulonglong2*>(ptab + b * 32);
#pragma unroll
                                for (int e4 = 0; e4 < 8; ++e4) {
                                    const ulonglong2 t = ct[e4];
                                    float x0, x1, x2, x3;
                                    unpair(mul2(pair(v[4 * e4], v[4 * e4 + 1]), t.x), x0, x1);
                                    unpair(mul2(pair(v[4 * e4 + 2], v[4 * e4 + 3]), t.y), x2, x3);
                                    v[4 * e4] = __float_as_uint(x0);
                                    v[4 * e4 + 1] = __float_as_uint(x1);
                                    v[4 * e4 + 2] = __float_as_uint(x2);
                                    v[4 * e4 + 3] = __float_as_uint(x3);
                                }
                                // on the diagonal a select, never a product, drops what
                                // is above it
                                if (rel == 0) {
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        if (jb.rev ? e < lane : e > lane) v[e] = 0u;
                                }
                            } else if (rel == 0) {
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const int d = jb.rev ? e - lane : lane - e;
                                    const float w = ptab[d & 31] * jb.s_in;
                                    v[e] = d >= 0 ? __float_as_uint(__uint_as_float(v[e]) * w) : 0u;
                                }
                            } else {
                                // lam^{i-j} as a row factor times a column factor, both <= 1
                                const float u = exp2f(a2 * (float)(jb.rev ? b * 32 - row : row - b * 32 - 31)) * jb.s_in;
#pragma unroll
                                for (int e4 = 0; e4 < 8; ++e4) {
                                    const float4 t = vt[e4];
                                    v[4 * e4] = __float_as_uint(__uint_as_float(v[4 * e4]) * (u * t.x));
                                    v[4 * e4 + 1] = __float_as_uint(__uint_as_float(v[4 * e4 + 1]) * (u * t.y));
                                    v[4 * e4 + 2] = __float_as_uint(__uint_as_float(v[4 * e4 + 2]) * (u * t.z));
                                    v[4 * e4 + 3] = __float_as_uint(__uint_as_float(v[4 * e4 + 3]) * (u * t.w));
                                }
                            }
                            if (n < kC && jb.rev) {   // later rows than the chunk has
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (b * 32 + e >= n) v[e] = 0u;
                            }
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = pack2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                        }
                        __syncwarp();
                        tmem_st_x16(base + b * 16, o);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(smem_u32(b_pready + s));
                }
            }
        }
    } else if (warp < 8) {
        // ===================== scaled terms of C =====================
        const int row = (warp - 4) * 32 + lane;
        for (int it = blockIdx.x; it < tp.items; it += gridDim.x) {
            const Item im = item_of<kAgg>(tp, it);
            const LaJob& jb = tp.p.job[im.job];
            const float a2 = la_log2_decay(g.a, im.h);
            const bool fac = factored(a2);
            const float wf = la_exp2(-a2, jb.rev ? kC - 1 - row : row) * jb.s_in;
            for (int x = 0; x < im.nch; ++x, ++c) {
                const int s = c & 1, ci = jb.rev ? im.nch - 1 - x : x;
                const int n = min(kC, im.rg.len - ci * kC);
                const float w = fac ? wf : exp2f(a2 * (float)(jb.rev ? row + 1 : n - 1 - row)) * jb.s_in;
                const f32x2 w2 = pair(w, w);
                mbar_wait(smem_u32(b_full + s), (c >> 1) & 1, err, 1u);
                if (c > 0) mbar_wait(smem_u32(b_udone), (c - 1) & 1, err, 1u);
                uint8_t* st = smem + s * kStage;
                if (row < n) {
#pragma unroll 2
                    for (int ch = 0; ch < 8; ++ch) {
                        const int at = row * kRow + ((ch ^ (row & 7)) << 4);
                        const uint4 q = *reinterpret_cast<const uint4*>(st + 4 * kAtom + at);
                        const uint32_t in[4] = {q.x, q.y, q.z, q.w};
                        uint32_t t[kTerms][4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // 24 bits as three times 8, cut off rather than rounded:
                            // the three add up to the product exactly
                            f32x2 r = mul2(pair(lo16(in[e]), hi16(in[e])), w2);
#pragma unroll
                            for (int y = 0; y < kTerms; ++y) {
                                float a, b;
                                unpair(r, a, b);
                                t[y][e] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
                                if (y + 1 < kTerms)
                                    r = add2(r, pair(-hi16(__float_as_uint(a)), -hi16(__float_as_uint(b))));
                            }
                        }
#pragma unroll
                        for (int y = 0; y < kTerms; ++y)
                            *reinterpret_cast<uint4*>(terms + y * kAtom + at) = make_uint4(t[y][0], t[y][1], t[y][2], t[y][3]);
                    }
                } else {
                    // a row of other tokens: nothing of it may reach a product
                    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch) {
                        const int at = row * kRow + (ch << 4);
                        *reinterpret_cast<uint4*>(st + 2 * kAtom + at) = z;
                        *reinterpret_cast<uint4*>(st + 3 * kAtom + at) = z;
                        *reinterpret_cast<uint4*>(st + 4 * kAtom + at) = z;
#pragma unroll
                        for (int q = 0; q < kTerms; ++q)
                            *reinterpret_cast<uint4*>(terms + q * kAtom + at) = z;
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(smem_u32(b_vready));
            }
        }
    } else if (warp < 16) {
        // ===================== X =====================
        const int k = (warp & 3) * 32 + lane;           // X's row = tensor-memory lane
        const int vc = warp < 12 ? 0 : 32;              // X's columns: 32 a thread
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        for (int it = blockIdx.x; it < tp.items; it += gridDim.x) {
            const Item im = item_of<kAgg>(tp, it);
            if (im.skip || im.rg.seq == g.nseq) continue;
            const LaJob& jb = tp.p.job[im.job];
            const int nv = min(kLaCols, jb.DV - im.v0) - vc;
            const int64_t elems = (int64_t)jb.DK * jb.DV;
            const int64_t at = (int64_t)k * jb.sk + (int64_t)(im.v0 + vc) * jb.sv;
            const int64_t so = ((int64_t)im.rg.seq * g.H + im.h) * elems + at;
            // the range's number is the item's: item = ((range H + h) jobs + job) nvb + vb
            const int ridx = it / tp.nvb / tp.p.njobs / g.H;
            float* ag = im.cut ? jb.agg + ((int64_t)ridx * g.H + im.h) * elems + at : nullptr;
            const float* in = kAgg ? nullptr : (im.cut ? ag : (jb.init ? jb.init + so : nullptr));
            f32x2 X[16];
            {
                float x0[32];
#pragma unroll
                for (int v = 0; v < 32; ++v)
                    x0[v] = in != nullptr && k < jb.DK && v < nv ? in[(int64_t)v * jb.sv] : 0.f;
#pragma unroll
                for (int v = 0; v < 16; ++v) X[v] = pair(x0[2 * v], x0[2 * v + 1]);
            }
            const float a2 = la_log2_decay(g.a, im.h);
            const bool fac = factored(a2);
            float f_hi, f_lo;
            la_decay_pow(g.a, im.h, kC, f_hi, f_lo);
            for (int x = 0; x < im.nch; ++x, ++c) {
                const int s = c & 1, ci = jb.rev ? im.nch - 1 - x : x;
                const int n = min(kC, im.rg.len - ci * kC);
                if (!kAgg) {
                    // in the factored form the row factor of out is lam^{i'}
                    const float m = fac ? la_exp2(a2, jb.rev ? n - kC : 1) : 1.f;
                    const f32x2 m2 = pair(m, m);
                    if (c > 0) mbar_wait(smem_u32(b_xdone), (c - 1) & 1, err, 1u);
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch)
                        *reinterpret_cast<uint4*>(xs + k * kRow + (((vc / 8 + ch) ^ (k & 7)) << 4)) =
                            make_uint4(pack2(mul2(X[4 * ch], m2)), pack2(mul2(X[4 * ch + 1], m2)),
                                       pack2(mul2(X[4 * ch + 2], m2)), pack2(mul2(X[4 * ch + 3], m2)));
                    fence_proxy_async_smem();
                    mbar_arrive(smem_u32(b_sready));
                }
                float hi = f_hi, lo = f_lo;
                if (n < kC) la_decay_pow(g.a, im.h, n, hi, lo);
                const float cu = fac ? la_exp2(a2, jb.rev ? kC : n - 1) : 1.f;
                mbar_wait(smem_u32(b_udone), c & 1, err, 1u);
                tc_fence_after();
                const f32x2 hi2 = pair(hi, hi), lo2 = pair(lo, lo), cu2 = pair(cu, cu);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t u[kTerms][16];
                    __syncwarp();
#pragma unroll
                    for (int y = 0; y < kTerms; ++y)
                        tmem_ld_x16(tmem + lane_off + kU + y * 64 + vc + q * 16, u[y]);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const f32x2 u2 = add2(pair(u[0][2 * e], u[0][2 * e + 1]),
                                              add2(pair(u[1][2 * e], u[1][2 * e + 1]), pair(u[2][2 * e], u[2][2 * e + 1])));
                        f32x2& X2 = X[q * 8 + e];
                        X2 = fma2(X2, hi2, fma2(X2, lo2, mul2(cu2, u2)));
                    }
                }
                tc_fence_before();
                mbar_arrive(smem_u32(b_ufree));
            }
            float* outst = kAgg ? ag : (im.last && jb.fin ? jb.fin + so : nullptr);
            if (outst != nullptr && k < jb.DK) {
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    float x0, x1;
                    unpair(X[v], x0, x1);
                    if (2 * v < nv) {   // nv is a multiple of 16
                        outst[(int64_t)(2 * v) * jb.sv] = x0;
                        outst[(int64_t)(2 * v + 1) * jb.sv] = x1;
                    }
                }
            }
            __syncwarp();
        }
    } else if (!kAgg) {
        // ===================== out =====================
        const int i = (warp - 16) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp - 16) * 32) << 16;
        for (int it = blockIdx.x; it < tp.items; it += gridDim.x) {
            const Item im = item_of<kAgg>(tp, it);
            const LaJob& jb = tp.p.job[im.job];
            const int nv = min(kLaCols, jb.DV - im.v0);
            const int64_t os = (int64_t)g.H * jb.DV, oh = (int64_t)im.h * jb.DV + im.v0;
            if (im.rg.seq == g.nseq && !im.skip) {       // tokens of no sequence: zeros
                for (int x = i; x < im.rg.len * (nv / 16); x += 128) {
                    const int64_t e = (int64_t)(im.rg.t0 + x / (nv / 16)) * os + oh + x % (nv / 16) * 16;
                    uint4* d = jb.out_f32 ? reinterpret_cast<uint4*>(static_cast<float*>(jb.out) + e)
                                          : reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(jb.out) + e);
                    for (int q = 0; q < (jb.out_f32 ? 4 : 2); ++q) d[q] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            const float a2 = la_log2_decay(g.a, im.h);
            const bool fac = factored(a2);
            for (int x = 0; x < im.nch; ++x, ++c) {
                const int ci = jb.rev ? im.nch - 1 - x : x;
                const int n = min(kC, im.rg.len - ci * kC);
                const float f = jb.s_out * (fac ? la_exp2(a2, jb.rev ? kC - 1 - i : i)
                                                : exp2f(a2 * (float)(jb.rev ? n - 1 - i : i + 1)));
                const int64_t e0 = (int64_t)(im.rg.t0 + ci * kC + i) * os + oh;
                mbar_wait(smem_u32(b_odone), c & 1, err, 1u);
                tc_fence_after();
                const f32x2 f2 = pair(f, f), s2 = pair(jb.s_out, jb.s_out);
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {   // 16 columns at a time
                    uint32_t p[16];
                    f32x2 r[8];
                    __syncwarp();
                    tmem_ld_x16(tmem + lane_off + kO + b * 16, p);
                    if (fac) {
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e) r[e] = mul2(f2, pair(p[2 * e], p[2 * e + 1]));
                    } else {
                        uint32_t q[16];
                        tmem_ld_x16(tmem + lane_off + kW + (c & 1) * 128 + 64 + b * 16, q);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            r[e] = fma2(f2, pair(p[2 * e], p[2 * e + 1]), mul2(s2, pair(q[2 * e], q[2 * e + 1])));
                    }
                    if (b == 3) {
                        tc_fence_before();
                        mbar_arrive(smem_u32(b_ofree));
                    }
                    if (i < n && b * 16 < nv) {
                        const int64_t e = e0 + b * 16;
                        if (jb.out_f32) {
                            ulonglong2* d = reinterpret_cast<ulonglong2*>(static_cast<float*>(jb.out) + e);
#pragma unroll
                            for (int y = 0; y < 4; ++y) d[y] = make_ulonglong2(r[2 * y], r[2 * y + 1]);
                        } else {
                            uint32_t w[8];
#pragma unroll
                            for (int y = 0; y < 8; ++y) w[y] = pack2(r[y]);
                            __nv_bfloat16* d = static_cast<__nv_bfloat16*>(jb.out) + e;
                            if ((reinterpret_cast<uintptr_t>(d) & 31) == 0) {
                                st_v8(d, w);
                            } else {
                                reinterpret_cast<uint4*>(d)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                                reinterpret_cast<uint4*>(d)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        }
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) report_timeout_to_host(err, tp.host_err);
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

bool encode(CUtensorMap* m, const void* base, int D, int heads, int64_t stride, int T) {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)heads, (uint64_t)T};
    const uint64_t str[2] = {(uint64_t)D * 2, (uint64_t)stride * 2};
    const uint32_t box[3] = {64, 1, kC};
    return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, str, box,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

cudaError_t launch_linattn_tc(const LaParams& p, int mode, int sms, cudaStream_t stream) {
    TcParams tp;
    TcMaps maps;
    tp.p = p;
    tp.nvb = 1;
    memset(&maps, 0, sizeof(maps));
    for (int j = 0; j < p.njobs; ++j) {
        const LaJob& b = p.job[j];
        const int n = (b.DV + kLaCols - 1) / kLaCols;
        tp.nvb = n > tp.nvb ? n : tp.nvb;
        if (p.g.T > 0 && (!encode(&maps.m[j][0], b.A, b.DK, b.hA, b.sA, p.g.T) ||
                          !encode(&maps.m[j][1], b.B, b.DK, b.hB, b.sB, p.g.T) ||
                          !encode(&maps.m[j][2], b.C, b.DV, b.hC, b.sC, p.g.T)))
            return cudaErrorInvalidValue;
    }
    const int64_t items = (int64_t)p.g.range_cap * p.g.H * p.njobs * tp.nvb;
    if (items >= (1LL << 31) - sms) return cudaErrorInvalidValue;
    tp.items = (int)items;
    tp.host_err = host_timeout_word();
    auto k = mode ? linattn_tc<true> : linattn_tc<false>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)(items < sms ? items : sms), kThreads, kSmem, stream>>>(tp, maps);
    return cudaGetLastError();
}

unsigned int take_linattn_error() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_la_error, sizeof(v)) != cudaSuccess) return ~0u;
    cudaMemcpyToSymbol(g_la_error, &zero, sizeof(zero));
    return v;
}

}  // namespace ssd
