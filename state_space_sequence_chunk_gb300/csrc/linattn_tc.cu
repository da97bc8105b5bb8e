// linattn_tc.cu -- linear attention with a decay for each head on the tcgen05
// tensor cores (bf16 operands, fp32 accumulation and state).
//
// One chain is (range of a sequence, head, 64 columns of c), walked in chunks of
// 128 tokens.  With i, j the rows of a chunk of n tokens (forwards; backwards
// the exponents are mirrored) and X the state before it:
//     W   = A B^T                                   128 x 128 x DK
//     P   = s_in W o lam^{i-j} [i >= j]             (bf16, tensor memory)
//     O1  = A X                                     128 x 64 x DK
//     O2  = P C                                     128 x 64 x 128
//     out = s_out (lam^{i+1} o O1 + O2)
//     U   = B^T (s_in lam^{n-1-j} o C)              DK x 64 x 128
//     X   <- lam^n X + U
// Every operand is read once per chain from HBM (a and b once per 64 columns of
// c, from L2 the second time) and no state leaves the chip between chunks.
//
// Precision.  P and the X that multiplies A are rounded to bf16 (as operands of
// a product whose result is rounded to bf16).  X itself must not be: it is kept
// in fp32 registers and U is exact to fp32: C's rows scaled by the decay are
// split into three bf16 terms (8 bits each) whose products are accumulated from
// the smallest up, so that the accumulator's roundings are those of the 8 steps
// of the leading term.  X <- lam^n X + U runs on the CUDA cores, where it is
// rounded to nearest (the accumulator's rounding is not documented, and a chain
// adds it up over hundreds of chunks).
//
// Persistent CTAs of 18 warps, one per SM:
//   0-3   P: tensor memory -> decay, mask -> tensor memory (bf16, in place)
//   4-7   C's scaled terms (a thread owns token row j); zeroes the rows of a
//         ragged chunk that belong to other tokens, whatever they hold
//   8-11  X in registers (a thread owns a row of X, 64 columns): bf16 copy for
//         A X, update with U, stored states
//   12-15 out (a thread owns a token row)
//   16    TMA, two stages of A, B and C tiles (80 KB each)
//   17    MMA issue: U(c), A X(c), P C(c), and W one chunk ahead
// so that per chunk the tensor pipe (about 1800 cycles for DK = 128) runs while
// each warpgroup works on another chunk or product.
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
constexpr int kThreads = 576;
constexpr int kTmaWarp = 16, kMmaWarp = 17;
constexpr int kStage = 5 * kAtom;             // A (2 atoms), B (2), C (1)
constexpr int kTerms = 3;
constexpr int kSmem = 2 * kStage + kTerms * kAtom + kAtom + 1024 + 1024;
// tensor memory columns
constexpr uint32_t kW = 0;                    // W / P, two buffers of 128
constexpr uint32_t kO1 = 256, kO2 = 320, kU = 384;   // U: two buffers of 64

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
__device__ __forceinline__ void bar_wg(int id) {
    asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}
__device__ __forceinline__ void st_v8(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
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
    uint64_t* b_udone = bars + 8;     // [2] U computed, terms read (commit)
    uint64_t* b_ufree = bars + 10;    // [2] U read (128)
    uint64_t* b_vready = bars + 12;   // terms written (128)
    uint64_t* b_sready = bars + 13;   // bf16 X written (128)
    uint64_t* b_xdone = bars + 14;    // A X computed: the bf16 X may change (commit)
    uint64_t* b_odone = bars + 15;    // O1 and O2 computed (commit)
    uint64_t* b_ofree = bars + 16;    // O1 and O2 read (128)
    uint32_t* holder = reinterpret_cast<uint32_t*>(bars + 17);
    float* lamp = reinterpret_cast<float*>(bars + 18);   // lam^0 .. lam^31
    float* lampr = lamp + 32;                            // lam^31 .. lam^0

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(b_full + s), 1);
            mbar_init(smem_u32(b_empty + s), 1);
            mbar_init(smem_u32(b_wdone + s), 1);
            mbar_init(smem_u32(b_pready + s), 128);
            mbar_init(smem_u32(b_udone + s), 1);
            mbar_init(smem_u32(b_ufree + s), 128);
        }
        mbar_init(smem_u32(b_vready), 128);
        mbar_init(smem_u32(b_sready), 128);
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
        constexpr uint32_t kIdU = make_idesc(1, 128, 64, 1, 1);
        for (int it = blockIdx.x; it < tp.items; it += gridDim.x) {
            const Item im = item_of<kAgg>(tp, it);
            if (lane == 0) {
                const int ks = tp.p.job[im.job].DK / 16;
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
                    // W one chunk ahead: its buffer's previous P has been read by an
                    // earlier product of this thread
                    if (!kAgg && x + 1 < im.nch) w_product(c + 1);
                    if (kAgg) mbar_wait(smem_u32(b_full + s), use & 1, err, 1u);
                    // U = B^T (scaled C), smallest term first
                    mbar_wait(smem_u32(b_vready), c & 1, err, 1u);
                    mbar_wait(smem_u32(b_ufree + s), (use & 1) ^ 1, err, 1u);
                    tc_fence_after();
                    {
                        const uint64_t ad = smem_desc_sw128(st + 2 * kAtom, kAtom, 8 * kRow);
#pragma unroll
                        for (int q = kTerms - 1; q >= 0; --q) {
                            const uint64_t bd = smem_desc_sw128(smem_u32(terms) + q * kAtom, 8 * kRow, 8 * kRow);
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) {
                                const uint64_t o = (uint64_t)((kk * 16 * kRow) >> 4);
                                mma_f16_ss(tmem + kU + s * 64, ad + o, bd + o, kIdU,
                                           (q < kTerms - 1 || kk > 0) ? 1u : 0u);
                            }
                        }
                    }
                    mma_commit(smem_u32(b_udone + s));
                    if (kAgg) {
                        mma_commit(smem_u32(b_empty + s));
                        continue;
                    }
                    // O1 = A X
                    mbar_wait(smem_u32(b_sready), c & 1, err, 1u);
                    mbar_wait(smem_u32(b_ofree), (c & 1) ^ 1, err, 1u);
                    tc_fence_after();
                    {
                        const uint64_t ad = smem_desc_sw128(st, 16, 8 * kRow);
                        const uint64_t bd = smem_desc_sw128(smem_u32(xs), 8 * kRow, 8 * kRow);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            if (kk < ks)
                                mma_f16_ss(tmem + kO1, ad + (uint64_t)(((kk / 4) * kAtom + (kk % 4) * 32) >> 4),
                                           bd + (uint64_t)((kk * 16 * kRow) >> 4), kIdO, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(smem_u32(b_xdone));
                    // O2 = P C
                    mbar_wait(smem_u32(b_pready + s), use & 1, err, 1u);
                    tc_fence_after();
                    {
                        const uint64_t bd = smem_desc_sw128(st + 4 * kAtom, 8 * kRow, 8 * kRow);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            mma_f16_ts(tmem + kO2, tmem + kW + s * 128 + kk * 8,
                                       bd + (uint64_t)((kk * 16 * kRow) >> 4), kIdO, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(smem_u32(b_odone));
                    mma_commit(smem_u32(b_empty + s));
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
                bar_wg(1);                      // the tables' last readers are done
                if (warp == 0) {
                    lamp[lane] = exp2f(a2 * (float)lane);
                    lampr[31 - lane] = exp2f(a2 * (float)lane);
                }
                bar_wg(1);
                const float4* vt = reinterpret_cast<const float4*>(jb.rev ? lamp : lampr);
                for (int x = 0; x < im.nch; ++x, ++c) {
                    const int s = c & 1, ci = jb.rev ? im.nch - 1 - x : x;
                    const int n = min(kC, im.rg.len - ci * kC);
                    mbar_wait(smem_u32(b_wdone + s), (c >> 1) & 1, err, 1u);
                    tc_fence_after();
                    const uint32_t base = tmem + lane_off + kW + s * 128;
                    // in place: block b's 16 packed columns lie within columns that
                    // blocks up to b held
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
                            if (rel == 0) {
                                // the block on the diagonal: a select, never a product,
                                // drops what is above it
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const int d = jb.rev ? e - lane : lane - e;
                                    const float w = lamp[d & 31] * jb.s_in;
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
            for (int x = 0; x < im.nch; ++x, ++c) {
                const int s = c & 1, ci = jb.rev ? im.nch - 1 - x : x;
                const int n = min(kC, im.rg.len - ci * kC);
                const float w = exp2f(a2 * (float)(jb.rev ? row + 1 : n - 1 - row)) * jb.s_in;
                mbar_wait(smem_u32(b_full + s), (c >> 1) & 1, err, 1u);
                if (c > 0) mbar_wait(smem_u32(b_udone + ((c - 1) & 1)), ((c - 1) >> 1) & 1, err, 1u);
                uint8_t* st = smem + s * kStage;
                if (row < n) {
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch) {
                        const int at = row * kRow + ((ch ^ (row & 7)) << 4);
                        const uint4 q = *reinterpret_cast<const uint4*>(st + 4 * kAtom + at);
                        const uint32_t in[4] = {q.x, q.y, q.z, q.w};
                        uint32_t t0[4], t1[4], t2[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float a = lo16(in[e]) * w, b = hi16(in[e]) * w;
                            t0[e] = pack2(a, b);
                            a -= lo16(t0[e]);
                            b -= hi16(t0[e]);
                            t1[e] = pack2(a, b);
                            t2[e] = pack2(a - lo16(t1[e]), b - hi16(t1[e]));
                        }
                        *reinterpret_cast<uint4*>(terms + at) = make_uint4(t0[0], t0[1], t0[2], t0[3]);
                        *reinterpret_cast<uint4*>(terms + kAtom + at) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
                        *reinterpret_cast<uint4*>(terms + 2 * kAtom + at) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
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
    } else if (warp < 12) {
        // ===================== X =====================
        const int k = (warp - 8) * 32 + lane;           // X's row = tensor-memory lane
        const uint32_t lane_off = (uint32_t)((warp - 8) * 32) << 16;
        for (int it = blockIdx.x; it < tp.items; it += gridDim.x) {
            const Item im = item_of<kAgg>(tp, it);
            if (im.skip || im.rg.seq == g.nseq) continue;
            const LaJob& jb = tp.p.job[im.job];
            const int nv = min(kLaCols, jb.DV - im.v0);
            const int64_t elems = (int64_t)jb.DK * jb.DV;
            const int64_t at = (int64_t)k * jb.sk + (int64_t)im.v0 * jb.sv;
            const int64_t so = ((int64_t)im.rg.seq * g.H + im.h) * elems + at;
            // the range's number is the item's: item = ((range H + h) jobs + job) nvb + vb
            const int ridx = it / tp.nvb / tp.p.njobs / g.H;
            float* ag = im.cut ? jb.agg + ((int64_t)ridx * g.H + im.h) * elems + at : nullptr;
            const float* in = kAgg ? nullptr : (im.cut ? ag : (jb.init ? jb.init + so : nullptr));
            float X[64];
#pragma unroll
            for (int v = 0; v < 64; ++v)
                X[v] = in != nullptr && k < jb.DK && v < nv ? in[(int64_t)v * jb.sv] : 0.f;
            float f_hi, f_lo;
            la_decay_pow(g.a, im.h, kC, f_hi, f_lo);
            for (int x = 0; x < im.nch; ++x, ++c) {
                const int s = c & 1, ci = jb.rev ? im.nch - 1 - x : x;
                const int n = min(kC, im.rg.len - ci * kC);
                if (!kAgg) {
                    if (c > 0) mbar_wait(smem_u32(b_xdone), (c - 1) & 1, err, 1u);
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch)
                        *reinterpret_cast<uint4*>(xs + k * kRow + ((ch ^ (k & 7)) << 4)) =
                            make_uint4(pack2(X[8 * ch], X[8 * ch + 1]), pack2(X[8 * ch + 2], X[8 * ch + 3]),
                                       pack2(X[8 * ch + 4], X[8 * ch + 5]), pack2(X[8 * ch + 6], X[8 * ch + 7]));
                    fence_proxy_async_smem();
                    mbar_arrive(smem_u32(b_sready));
                }
                float hi = f_hi, lo = f_lo;
                if (n < kC) la_decay_pow(g.a, im.h, n, hi, lo);
                mbar_wait(smem_u32(b_udone + s), (c >> 1) & 1, err, 1u);
                tc_fence_after();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t u[32];
                    __syncwarp();
                    tmem_ld_x32(tmem + lane_off + kU + s * 64 + half * 32, u);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float& X1 = X[half * 32 + e];
                        X1 = fmaf(X1, hi, fmaf(X1, lo, __uint_as_float(u[e])));
                    }
                }
                tc_fence_before();
                mbar_arrive(smem_u32(b_ufree + s));
            }
            float* outst = kAgg ? ag : (im.last && jb.fin ? jb.fin + so : nullptr);
            if (outst != nullptr && k < jb.DK) {
#pragma unroll
                for (int v = 0; v < 64; ++v)
                    if (v < nv) outst[(int64_t)v * jb.sv] = X[v];
            }
            __syncwarp();
        }
    } else if (!kAgg) {
        // ===================== out =====================
        const int i = (warp - 12) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp - 12) * 32) << 16;
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
            for (int x = 0; x < im.nch; ++x, ++c) {
                const int ci = jb.rev ? im.nch - 1 - x : x;
                const int n = min(kC, im.rg.len - ci * kC);
                const float f = exp2f(a2 * (float)(jb.rev ? n - 1 - i : i + 1)) * jb.s_out;
                const int64_t e0 = (int64_t)(im.rg.t0 + ci * kC + i) * os + oh;
                mbar_wait(smem_u32(b_odone), c & 1, err, 1u);
                tc_fence_after();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t p[32], q[32];
                    __syncwarp();
                    tmem_ld_x32(tmem + lane_off + kO1 + half * 32, p);
                    tmem_ld_x32(tmem + lane_off + kO2 + half * 32, q);
                    tmem_wait_ld();
                    if (half == 1) {
                        tc_fence_before();
                        mbar_arrive(smem_u32(b_ofree));
                    }
                    if (i < n) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            p[e] = __float_as_uint(fmaf(f, __uint_as_float(p[e]), jb.s_out * __uint_as_float(q[e])));
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            if (half * 32 + b * 16 >= nv) continue;
                            const int64_t e = e0 + half * 32 + b * 16;
                            if (jb.out_f32) {
                                uint4* d = reinterpret_cast<uint4*>(static_cast<float*>(jb.out) + e);
#pragma unroll
                                for (int y = 0; y < 4; ++y)
                                    d[y] = make_uint4(p[b * 16 + 4 * y], p[b * 16 + 4 * y + 1],
                                                      p[b * 16 + 4 * y + 2], p[b * 16 + 4 * y + 3]);
                            } else {
                                uint32_t w[8];
#pragma unroll
                                for (int y = 0; y < 8; ++y)
                                    w[y] = pack2(__uint_as_float(p[b * 16 + 2 * y]), __uint_as_float(p[b * 16 + 2 * y + 1]));
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
