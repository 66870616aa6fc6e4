// chunk_attention_q8 for batches of a few rows per sequence: plain decoding, chains of drafts.
//
// Up to 8 NT rows (tokens x query heads of a kv head) against their keys: bound by the stream of
// codes, 2 d bytes a key, so what counts is that widening them costs little.  Products by warp:
// S^T = K Q^T and O^T = V^T P^T with the keys, then the columns, in the 16 rows of m16n8k16, so that
// the few rows of the queries are its 8 columns and nothing is padded to 16.  All operands are
// float16: a code becomes one exactly by a conversion of two at a time; a query row is scaled by a
// power of two that brings its largest element to 2^7 .. 2^8 (elements below 2^-21 of it lose
// bits); a weight is at most 2^15 and below 2^-14 subnormal, so those above 2^-27 of a row's largest
// are off by at most 2^-11 of themselves, and the others by 2^-38 of the largest.  The blocks' scales are
// powers of two and stay out of the products: K's multiplies the scores, V's is added to the
// exponent (the running maximum is that of s + log2(scale of V)) and taken out of the sum.
// The order of a head's columns is free in a product, so a lane takes contiguous bytes of a key,
// and of four keys for V, whose bytes are paired by permutations.
//
// Every warp goes through pages of 16 keys for itself (copies into its own ring of stages, its own
// maximum, sum and O^T), the four warps of a CTA through one item's pages in turn; they are
// joined in shared memory at the item's end.  An item is (sequence, kv head, up to 8 NT / G
// tokens); the items of all sequences, laid end to end, are cut into equal runs, one per CTA, as in
// attn_chunk_tc.cuh, and pieces of items that a border cuts are joined by a second kernel.
// Measured (32/8 heads of 128): one row of each of 64 sequences of 512-8,192 keys 63 us = 5.6 TB/s,
// the stream and 41 % of the issue slots; 6 rows of each of 128 sequences of 1,024-4,096 keys 189 us,
// bound by the products (three row tiles of 8: 146 TFLOP/s, about what this GPU gives products by
// warp); one row after 300 keys 11 us, two launches and their start.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "tv_chunk.cuh"
#include "tv_fp8.cuh"
#include "tv_internal.h"
#include "tv_tc.cuh"

namespace tv {

namespace {

constexpr int RQ_WARPS = 4, RQ_THREADS = RQ_WARPS * 32;
constexpr int RQ_JOIN_THREADS = 256;
constexpr float RQ_LOG2E = 1.4426950408889634f;
// The largest weight is 2^(RQ_BIAS + RQ_SLACK): float16's range is used downwards.  The running
// maximum is raised when a score exceeds it by RQ_SLACK.
constexpr float RQ_BIAS = 13.f, RQ_SLACK = 2.f;
// fixed cost of an item, in pages, and a border that is this close to an item's end moves there (the
// cases below, us, with 8: 68 and 204; 16: 63 and 195; 24: 63 and 189; 32: 67 and 187)
constexpr int64_t RQ_C0 = 24;
constexpr int RQ_SNAP = 4;
// cost of a run, in pages, below which cutting further saves nothing: one that begins an item has
// pages of it behind the fixed cost
constexpr int RQ_RUN_MIN = RQ_C0 + RQ_SNAP + 1;

struct RqParams {
    ChunkView c;
    const uint8_t *q, *k, *v;        // q: bfloat16
    const float *k_scale, *v_scale;
    const uint64_t* mask;
    uint8_t* out;
    int64_t q_stride, o_stride;      // elements
    int32_t* status;
    int4* rec;                       // what the slots hold: (first row, tokens, kv head, RQ_*)
    float* part;                     // two slots per CTA
    int Hkv, G, npt, window, sinks;
    float scale_log2;                // scale * log2(e); with a cap: 2 log2(e) scale / cap
    float cap_log2, cap_small, cap_c[3];
    LateWait late;
};
constexpr int RQ_PIECE = 1, RQ_LAST = 2, RQ_LATE = 4;

template <int NT>
struct RqShape {
    static constexpr int ROWS = 8 * NT;
    static constexpr int PER_SM = NT == 1 ? 3 : 2;
    static constexpr int STAGES = NT == 3 ? 5 : 3;
};

// tanh(x) / x for small x, as in attn_chunk_tc.cuh
constexpr double RQ_TANH_SMALL = 0.35;
constexpr double RQ_TANH_C[3] = {0.9999971183259196, -0.3329087359461761, 0.12394375936950675};

// ------------------------------------------------------------ the run space
struct RqSeq {
    int P, n, items;
    int64_t per;       // cost of an item: RQ_C0 + the pages of the one with the most
    bool shape;
};
// Keys of the tokens i0 .. i1 - 1: counted from kbase, the first `front` of them keys 0 .. front - 1
// (as in attn_chunk_tc.cuh), up to hi.
__device__ __forceinline__ void rq_keys(const RqParams& p, int P, int i0, int i1, int& kbase, int& front, int& hi) {
    hi = P + i1;
    kbase = chunk_first_key(P + i0, p.window) & ~15;
    front = (p.sinks + 15) & ~15;
    if (kbase <= front) kbase = front = 0;
    kbase -= front;
}
__device__ __forceinline__ RqSeq rq_seq(const RqParams& p, int P, int n) {
    RqSeq s;
    s.P = P;
    s.n = n;
    s.shape = chunk_shape_ok(p.c, P, n) && (p.mask == nullptr || n <= 64);
    s.items = (n + p.npt - 1) / p.npt;
    int64_t pages = 0;
    if (s.shape && n > 0) {
        // no window: all keys; with one, at most the window, the item's tokens, the first ones and 16
        pages = ((int64_t)P + n + 15) / 16;
        if (p.window > 0) pages = min(pages, ((int64_t)p.window + p.npt + p.sinks + 15 + 15 + 15) / 16);
    }
    s.per = RQ_C0 + pages;
    return s;
}
__device__ __forceinline__ int64_t rq_units(const RqParams& p, int P, int n) {
    const RqSeq s = rq_seq(p, P, n);
    return (int64_t)s.items * p.Hkv * s.per;
}
// Page at which a border y units into an item cuts it (both runs beside it compute it).
__device__ __forceinline__ int rq_cut(int64_t y, int pages) {
    const int64_t t = y - RQ_C0;
    if (t <= RQ_SNAP) return 0;
    return t >= pages - RQ_SNAP ? pages : (int)t;
}
__device__ __forceinline__ void rq_runs(const RqParams& p, int64_t total, int ctas, int64_t& len, int& count) {
    count = (int)min((int64_t)ctas, max(total / RQ_RUN_MIN, (int64_t)1));
    len = (total + count - 1) / count;
}

// ------------------------------------------------------------ instructions
__device__ __forceinline__ void e4m3_halves(uint32_t w, uint32_t& lo, uint32_t& hi) {   // four codes
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {   // an 8 x 8 tile of 16-bit elements
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// l 2^d.  A maximum has the logarithm of V's scale in it, a sum has not: it can be as small as 2^-200 of
// what the maxima say.
__device__ __forceinline__ float times_exp2(float l, float d) {
    const float h = exp2f(0.5f * d);
    return l * h * h;
}

template <int D, int NT, bool CAP>
__global__ void __launch_bounds__(RQ_THREADS, RqShape<NT>::PER_SM)
rows_q8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
               const __grid_constant__ RqParams p) {
    constexpr int ROWS = RqShape<NT>::ROWS, ST = RqShape<NT>::STAGES;
    constexpr int PAGE = 16 * D, STAGE = 2 * PAGE;         // K's page, then V's
    constexpr int KS = D / 16;                             // products over a head's columns, over its rows
    constexpr int CB = D / 8;                              // bytes of a key's V that a lane takes
    extern __shared__ uint8_t rq_raw[];
    __shared__ ChunkLocateTmp<RQ_THREADS> tmp;
    __shared__ __align__(8) uint64_t bars[RQ_WARPS][ST];
    __shared__ float sm_m[RQ_WARPS][ROWS], sm_l[RQ_WARPS][ROWS];
    __shared__ __align__(16) uint4 sq[NT][D / 32][32];     // the queries, as the products take them
    __shared__ int late;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(rq_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q4 = lane & 3, r8 = lane >> 2;
    if (lane < ST) mbar_init(&bars[warp][lane], 1);
    if (tid == 0) late = 0;
    fence_mbar_init();
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    int64_t len = 0, x_lo = 0, x_hi = 0;
    int runs = 0;
    auto where = [&](int64_t total) {
        rq_runs(p, total, gridDim.x, len, runs);
        x_lo = min((int64_t)blockIdx.x * len, total);
        x_hi = min(x_lo + len, total);
        return x_lo;
    };
    auto units = [&](int P, int n) { return rq_units(p, P, n); };
    const ChunkPlace at = p.c.B <= 32 ? chunk_locate_warp(p.c, where, units)
                                      : chunk_locate<RQ_THREADS>(&tmp, p.c, where, units);
    if (blockIdx.x == 0)
        for (int b = tid; b < p.c.B; b += RQ_THREADS)
            if (!at.valid || p.c.q_start[b] == p.c.q_start[b + 1])
                p.status[b] = (at.valid && chunk_shape_ok(p.c, p.c.prefix[b], 0)) ? TV_OK : TV_ERR_OUT_OF_RANGE;
    int4 rec0 = make_int4(0, 0, 0, 0), rec1 = rec0;        // the run's first piece (begun before), its last
    int first_b = 0, last_b = -1;
    uint32_t count = 0;                                    // pages of this warp so far: stage and parity
    bool alive = !(p.late.warp >= 0 && (p.late.cta < 0 || p.late.cta == (int)blockIdx.x));
    if (at.b < p.c.B && x_lo < x_hi) {
        int b = at.b, row = at.row;
        RqSeq s = rq_seq(p, at.P, at.n);
        auto blocks_ok = [&]() -> bool {
            bool ok = s.shape;
            if (ok) {
                const int first = chunk_first_key(s.P, p.window);
                ok = chunk_blocks_ok(p.c, b, first, (int64_t)s.P + s.n, tid, RQ_THREADS);
                ok = chunk_blocks_ok(p.c, b, 0, min(p.sinks, first), tid, RQ_THREADS) && ok;
            }
            return __syncthreads_and(ok ? 1 : 0) != 0;
        };
        bool ok = blocks_ok();
        int64_t idx = (x_lo - at.base) / s.per;            // item of the sequence: kv head, token group
        int64_t start = at.base + idx * s.per;
        int64_t x = x_lo;
        first_b = last_b = b;
#pragma unroll 1
        while (true) {
            const int g = (int)(idx / s.items), k = (int)(idx - (int64_t)g * s.items);
            const int i0 = k * p.npt, ntok = min(p.npt, s.n - i0), rows = ntok * p.G, row0 = row + i0;
            int kbase = 0, front = 0, hi = 0, pages = 0, lo = 0, up = 0;
            if (ok) {
                rq_keys(p, s.P, i0, i0 + ntok, kbase, front, hi);
                pages = (hi - kbase + 15) >> 4;
                lo = rq_cut(x - start, pages);
                up = x_hi - start >= s.per ? pages : rq_cut(x_hi - start, pages);
            }
            // a refused sequence has items without pages: the run with the first unit writes them
            if (pages == 0 ? x == start : lo < up) {
                const bool whole = lo == 0 && up == pages;
                if (g == 0 && i0 == 0 && lo == 0 && tid == 0) p.status[b] = ok ? TV_OK : TV_ERR_OUT_OF_RANGE;
                const int steps = max(0, (up - lo - warp + RQ_WARPS - 1) / RQ_WARPS);
                // ---- queries: row 8 j + r8, its columns q4 D / 4 .. + D / 4 (in shared memory: registers are
                // for O)
                float fac[NT][2];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int rr = 8 * j + r8;
                    const bool in = rr < rows;
                    const int tok = rr / p.G, head = rr - tok * p.G;
                    const uint4* src = reinterpret_cast<const uint4*>(
                        p.q + 2 * ((int64_t)(row0 + (in ? tok : 0)) * p.q_stride + (int64_t)(g * p.G + (in ? head : 0)) * D + q4 * (D / 4)));
                    uint4 x4[D / 32];
                    float top = 0.f;
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) {
                        x4[e] = in ? src[e] : make_uint4(0u, 0u, 0u, 0u);
                        const uint32_t w[4] = {x4[e].x, x4[e].y, x4[e].z, x4[e].w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float a = __uint_as_float(w[y] << 16), c = __uint_as_float(w[y] & 0xffff0000u);
                            top = fmaxf(top, fmaxf(fabsf(fmaf(a, 0.f, a)), fabsf(fmaf(c, 0.f, c))));   // finite ones
                        }
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // 2^(7 - exponent): a normal number whatever the row holds
                    const uint32_t ex = min(max(__float_as_uint(top) >> 23, 20u), 254u);
                    const float up2 = __uint_as_float((261u - ex < 254u ? 261u - ex : 254u) << 23);
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) {
                        const uint32_t w[4] = {x4[e].x, x4[e].y, x4[e].z, x4[e].w};
                        uint32_t h[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            h[y] = half2_of(__uint_as_float(w[y] << 16) * up2, __uint_as_float(w[y] & 0xffff0000u) * up2);
                        if (j % RQ_WARPS == warp) sq[j][e][lane] = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                    const float down = scale_inverse(up2);
                    fac[j][0] = __shfl_sync(0xffffffffu, down, 8 * q4);
                    fac[j][1] = __shfl_sync(0xffffffffu, down, 8 * q4 + 4);
                    if (!CAP) {
                        fac[j][0] *= p.scale_log2;
                        fac[j][1] *= p.scale_log2;
                    }
                }
                __syncthreads();
                const int first_all = p.window > 0 ? max(0, s.P + i0 + ntok - p.window) : 0;   // seen by every row
                // ---- pages: a window of 32 steps, a lane each; the next one's blocks, then scales, ahead
                const int32_t* table = p.c.table + (int64_t)b * p.c.max_blocks;
                auto key_of = [&](int v) -> int { return v < front ? v : kbase + v; };
                struct Win { int row; float ks, ev; };
                int nblk = 0, noff = 0;
                auto ids = [&](int w) {
                    const int i = w * 32 + lane;
                    nblk = noff = 0;
                    if (i < steps) {
                        const int key = key_of((lo + warp + i * RQ_WARPS) * 16);
                        nblk = __ldg(table + key / p.c.bs);
                        noff = key % p.c.bs;
                    }
                };
                auto win = [&]() -> Win {
                    Win w;
                    const int64_t a = (int64_t)nblk * p.Hkv + g;
                    w.row = (nblk * p.Hkv + g) * p.c.bs + noff;
                    w.ks = scale_of(exponent_byte(__ldg(p.k_scale + a)));
                    w.ev = (float)((int)max(exponent_byte(__ldg(p.v_scale + a)), 27u) - 127);   // not below 2^-100
                    return w;
                };
                ids(0);
                Win cur = win(), nxt = cur;
                int wk = 0;
                if (steps > 32) {
                    ids(1);
                    nxt = win();
                }
                const uint64_t policy = ntok == s.n ? l2_policy_evict_first() : l2_policy_evict_normal();
                const uint32_t base = count;
                auto fill = [&](int i) {                   // i < wk * 32 + 64
                    if (i >= steps) return;
                    const int y = __shfl_sync(0xffffffffu, (i >> 5) == wk ? cur.row : nxt.row, i & 31);
                    if (lane == 0) {
                        const uint32_t st = (base + i) % ST;
                        uint8_t* dst = ring + (warp * ST + st) * STAGE;
                        uint64_t* bar = &bars[warp][st];
                        mbar_arrive_expect_tx_relaxed_one(bar, STAGE);
                        if constexpr (D == 128) {
                            tma_load_2d(dst, &kmap, bar, 0, y, policy);
                            tma_load_2d(dst + PAGE, &vmap, bar, 0, y, policy);
                        } else {
                            bulk_load(dst, p.k + (int64_t)y * D, PAGE, bar, policy);
                            bulk_load(dst + PAGE, p.v + (int64_t)y * D, PAGE, bar, policy);
                        }
                    }
                    __syncwarp();
                };
#pragma unroll
                for (int i = 0; i < ST; ++i) fill(i);
                // nb: the bias less the running maximum (of s + log2 of V's scale; none yet: 0); lim: what a
                // score may exceed it by
                float o[NT][KS][4], nb[NT][2], lim[NT][2], l[NT][2];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int t = 0; t < KS; ++t) o[j][t][0] = o[j][t][1] = o[j][t][2] = o[j][t][3] = 0.f;
                    nb[j][0] = nb[j][1] = RQ_BIAS;
                    lim[j][0] = lim[j][1] = -INFINITY;
                    l[j][0] = l[j][1] = 0.f;
                }
                // V's scales of this window lie far below the largest so far, some of them
                int ev_top = -127;
                auto far = [&](const Win& w) -> bool {
                    const bool in = wk * 32 + lane < steps;
                    ev_top = max(ev_top, __reduce_max_sync(0xffffffffu, in ? (int)w.ev : -127));
                    return __reduce_min_sync(0xffffffffu, in ? (int)w.ev : 128) < ev_top - 60;
                };
                bool mixed = far(cur);
                int i = 0;
#pragma unroll 1
                for (; i < steps; ++i) {
                    if ((i & 31) == 0 && i > 0) {
                        cur = nxt;
                        wk = i >> 5;
                        mixed = far(cur);
                        if (steps > (wk + 1) * 32) {
                            ids(wk + 1);
                            nxt = win();
                        }
                    }
                    const uint32_t st = (base + i) % ST;
                    alive = __all_sync(0xffffffffu, alive && mbar_wait(&bars[warp][st], ((base + i) / ST) & 1u));
                    if (!alive) break;
                    const uint8_t* stage = ring + (warp * ST + st) * STAGE;
                    const float ks = __shfl_sync(0xffffffffu, cur.ks, i & 31), ev = __shfl_sync(0xffffffffu, cur.ev, i & 31);
                    // ---- S^T: keys r8 and r8 + 8, rows 8 j + 2 q4 and + 1
                    float sc[NT][4];
#pragma unroll
                    for (int j = 0; j < NT; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
                    for (int hf = 0; hf < D / 64; ++hf) {
                        uint4 k0, k1;
                        if constexpr (D == 128) {
                            const int off = ((2 * q4 + hf) ^ r8) << 4;      // pieces exchanged by the row's number
                            k0 = *reinterpret_cast<const uint4*>(stage + r8 * 128 + off);
                            k1 = *reinterpret_cast<const uint4*>(stage + r8 * 128 + 1024 + off);
                        } else {
                            k0 = *reinterpret_cast<const uint4*>(stage + r8 * 64 + q4 * 16);
                            k1 = *reinterpret_cast<const uint4*>(stage + r8 * 64 + 512 + q4 * 16);
                        }
                        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            uint32_t a[2][4];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                e4m3_halves(w0[2 * z + y], a[y][0], a[y][2]);
                                e4m3_halves(w1[2 * z + y], a[y][1], a[y][3]);
                            }
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                const uint4 b = sq[j][hf * 2 + z][lane];
                                mma_f16(sc[j], a[0][0], a[0][1], a[0][2], a[0][3], b.x, b.y);
                                mma_f16(sc[j], a[1][0], a[1][1], a[1][2], a[1][3], b.z, b.w);
                            }
                        }
                    }
                    // ---- scores in units of log 2, with V's scale, less the running maximum; what a row does
                    // not see is -infinity
                    const int v0 = (lo + warp + i * RQ_WARPS) * 16, key0 = key_of(v0);
                    const bool edge = !(v0 < front ? v0 + 16 <= p.sinks
                                                   : key0 >= first_all && key0 + 15 <= s.P + i0 - (p.mask ? i0 + 1 : 0));
                    bool need = mixed;
                    float lsc = exp2f(-ev - RQ_BIAS);          // V's scale and the bias out of the sum
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const float f0 = ks * fac[j][0], f1 = ks * fac[j][1];
                        const float b0 = ev + nb[j][0], b1 = ev + nb[j][1];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if constexpr (CAP) {
                                const float y = sc[j][e] * (e & 1 ? f1 : f0), u = y * y, w = ex2_approx(y * p.scale_log2);
                                sc[j][e] = (u < p.cap_small ? y * fmaf(fmaf(p.cap_c[2], u, p.cap_c[1]), u, p.cap_c[0])
                                                            : fmaf(-2.f * p.cap_log2, rcp_approx(1.f + w), p.cap_log2)) + (e & 1 ? b1 : b0);
                            } else {
                                sc[j][e] = fmaf(sc[j][e], e & 1 ? f1 : f0, e & 1 ? b1 : b0);
                            }
                        }
                        if (edge) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int key = key0 + r8 + (e >> 1) * 8;
                                const int me = s.P + i0 + min((8 * j + 2 * q4 + (e & 1)) / p.G, ntok - 1);
                                bool seen = key <= me && (p.window <= 0 || key > me - p.window || key < p.sinks);
                                if (p.mask && key >= s.P && seen)
                                    seen = (p.mask[row + me - s.P] >> (key - s.P)) & 1ull;
                                if (!seen) sc[j][e] = -INFINITY;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            need = need || fmaxf(sc[j][e], sc[j][e + 2]) > lim[j][e];
                    }
                    if (__any_sync(0xffffffffu, need)) {
                        // the maxima, over the warp's eight lanes with the same rows
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float mx = fmaxf(sc[j][e], sc[j][e + 2]);
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                                const bool none = lim[j][e] == -INFINITY;      // no maximum yet, and l and O zero
                                const float by = none ? (mx == -INFINITY ? 0.f : mx - RQ_BIAS) : fmaxf(mx - RQ_BIAS, 0.f);
                                const float f = none ? 0.f : exp2f(-by);
                                if (mx != -INFINITY) lim[j][e] = RQ_BIAS + RQ_SLACK;
                                nb[j][e] -= by;
                                sc[j][e] -= by;
                                sc[j][e + 2] -= by;
                                l[j][e] = none ? 0.f : times_exp2(l[j][e], -by);
#pragma unroll
                                for (int t = 0; t < KS; ++t) {
                                    o[j][t][e] *= f;
                                    o[j][t][e + 2] *= f;
                                }
                            }
                        if (mixed && ev < ev_top - 60.f) {
                            // beside a block of much larger values (one of zeros has the smallest scale) the
                            // weights vanish with V's scale in them, but not from the sum
#pragma unroll
                            for (int j = 0; j < NT; ++j)
#pragma unroll
                                for (int e = 0; e < 4; ++e) l[j][e & 1] += ex2_approx(sc[j][e] - (ev + RQ_BIAS));
                            lsc = 0.f;
                        }
                    }
                    uint32_t pb[NT][2];
                    float pw[NT][4];
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) pw[j][e] = ex2_approx(sc[j][e]);
                        l[j][0] = fmaf(pw[j][0] + pw[j][2], lsc, l[j][0]);
                        l[j][1] = fmaf(pw[j][1] + pw[j][3], lsc, l[j][1]);
                        pb[j][0] = transposed(half2_of(pw[j][0], pw[j][1]));
                        pb[j][1] = transposed(half2_of(pw[j][2], pw[j][3]));
                    }
                    // ---- O^T += V^T P^T: columns r8 CB + 2 t and + 1, keys 2 q4, + 1, + 8, + 9
                    constexpr int VW = CB / 4;
                    uint32_t vw[4][VW];
                    const uint8_t* vp = stage + PAGE;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int kr = 2 * q4 + (e & 1) + (e >> 1) * 8;
                        if constexpr (D == 128) {
                            const uint4 w = *reinterpret_cast<const uint4*>(vp + kr * 128 + ((r8 ^ (kr & 7)) << 4));
                            vw[e][0] = w.x, vw[e][1] = w.y, vw[e][2] = w.z, vw[e][3] = w.w;
                        } else {
                            const uint2 w = *reinterpret_cast<const uint2*>(vp + kr * 64 + r8 * 8);
                            vw[e][0] = w.x, vw[e][1] = w.y;
                        }
                    }
                    if (edge) {
                        // NaN among what not every row sees: taken out of the products, and added to the rows
                        // that see it
                        uint32_t odd = 0;                      // keys 2 q4, + 1, + 8, + 9
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t acc = 0;
#pragma unroll
                            for (int y = 0; y < VW; ++y) acc |= (vw[e][y] & 0x7f7f7f7fu) + 0x01010101u;
                            if (acc & 0x80808080u) odd |= 1u << (2 * q4 + (e & 1) + (e >> 1) * 8);
                        }
                        odd = __reduce_or_sync(0xffffffffu, odd);
                        if (odd != 0u) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if ((odd >> (2 * q4 + (e & 1) + (e >> 1) * 8)) & 1u)
#pragma unroll
                                    for (int y = 0; y < VW; ++y) vw[e][y] = 0u;
#pragma unroll 1
                            for (uint32_t left = odd; left != 0u; left &= left - 1u) {
                                const int kk = __ffs(left) - 1, from = (kk & 7) * 4 + q4;
#pragma unroll
                                for (int j = 0; j < NT; ++j)
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        const float w0 = __shfl_sync(0xffffffffu, pw[j][e], from);
                                        const float w1 = __shfl_sync(0xffffffffu, pw[j][e + 2], from);
                                        const float s0 = __shfl_sync(0xffffffffu, sc[j][e], from);
                                        const float s1 = __shfl_sync(0xffffffffu, sc[j][e + 2], from);
                                        const float w = kk < 8 ? w0 : w1;
                                        if ((kk < 8 ? s0 : s1) == -INFINITY) continue;   // not seen
#pragma unroll
                                        for (int t = 0; t < KS; ++t)
#pragma unroll
                                            for (int y = 0; y < 2; ++y) {
                                                const int c = r8 * CB + 2 * t + y;
                                                const uint8_t code = D == 128 ? vp[kk * 128 + ((((c >> 4) ^ (kk & 7)) << 4) | (c & 15))]
                                                                              : vp[kk * 64 + c];
                                                o[j][t][e + 2 * y] = fmaf(w, e4m3_float(code), o[j][t][e + 2 * y]);
                                            }
                                    }
                            }
                        }
                    }
#pragma unroll
                    for (int y = 0; y < VW; ++y)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            // two columns of the word's four: (key 0, key 1) of the first, of the second
                            uint32_t a0, a1, a2, a3;
                            e4m3_halves(__byte_perm(vw[0][y], vw[1][y], z ? 0x7362 : 0x5140), a0, a1);
                            e4m3_halves(__byte_perm(vw[2][y], vw[3][y], z ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                            for (int j = 0; j < NT; ++j) mma_f16(o[j][2 * y + z], a0, a1, a2, a3, pb[j][0], pb[j][1]);
                        }
                    __syncwarp();                              // the stage is read
                    fill(i + ST);
                }
                if (!alive) {
                    // copies under way end before the CTA does
                    for (int y = i; y < min(steps, i + ST); ++y) mbar_wait(&bars[warp][(base + y) % ST], ((base + y) / ST) & 1u);
                    if (lane == 0) late = 1;
                }
                count += steps;
                // ---- the warps' results are joined
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float sum = l[j][e];
                        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                        if (r8 == 0) {
                            sm_m[warp][8 * j + 2 * q4 + e] = lim[j][e] == -INFINITY ? -INFINITY : RQ_BIAS - nb[j][e];
                            sm_l[warp][8 * j + 2 * q4 + e] = sum;
                        }
                    }
                __syncthreads();                               // every warp is done with its stages
                if (late) break;
                float* so = reinterpret_cast<float*>(ring);    // [warp][rows][D]
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int rr = 8 * j + 2 * q4 + e;
                        if (rr < rows)
#pragma unroll
                            for (int t = 0; t < KS; ++t)
                                *reinterpret_cast<float2*>(so + (warp * ROWS + rr) * D + r8 * CB + 2 * t) =
                                    make_float2(o[j][t][e], o[j][t][e + 2]);
                    }
                __syncthreads();
                float* slot = whole ? nullptr : p.part + (int64_t)(2 * blockIdx.x + (lo == 0 ? 1 : 0)) * ROWS * (D + 2);
                for (int e = tid; e < rows * (D / 4); e += RQ_THREADS) {
                    const int rr = e / (D / 4), c = e % (D / 4) * 4;
                    float mx = -INFINITY, den = 0.f;
#pragma unroll
                    for (int w = 0; w < RQ_WARPS; ++w) mx = fmaxf(mx, sm_m[w][rr]);
                    const float bz = mx == -INFINITY ? 0.f : mx;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < RQ_WARPS; ++w) {
                        const float f = exp2f(sm_m[w][rr] - bz), part = times_exp2(sm_l[w][rr], sm_m[w][rr] - bz);
                        const float4 y = *reinterpret_cast<const float4*>(so + (w * ROWS + rr) * D + c);
                        den += part;
                        acc.x = fmaf(f, y.x, acc.x);
                        acc.y = fmaf(f, y.y, acc.y);
                        acc.z = fmaf(f, y.z, acc.z);
                        acc.w = fmaf(f, y.w, acc.w);
                    }
                    if (slot) {
                        *reinterpret_cast<float4*>(slot + rr * D + c) = acc;
                        if (c == 0) {
                            slot[ROWS * D + rr] = mx;
                            slot[ROWS * (D + 1) + rr] = den;
                        }
                    } else {
                        const int tok = rr / p.G, head = rr - tok * p.G;
                        // (no key at all, and refused sequences: zero)
                        bool none = !ok;
                        if (p.mask && s.P == 0 && !none)
                            none = (p.mask[row0 + tok] & (~0ull >> (63 - min(i0 + tok, 63)))) == 0ull;
                        const float inv = none ? 0.f : exp2f(-RQ_BIAS) / den;
                        const uint2 y = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                        *reinterpret_cast<uint2*>(p.out + 2 * ((int64_t)(row0 + tok) * p.o_stride + (int64_t)(g * p.G + head) * D + c)) = y;
                    }
                }
                if (!whole) {
                    const int4 rec = make_int4(row0, ntok, g, RQ_PIECE | (up == pages ? RQ_LAST : 0));
                    if (lo == 0) rec1 = rec;
                    else rec0 = rec;
                }
                fence_proxy_async_smem();                      // the next copies land where so was
                __syncthreads();
            }
            // ---- the next item
            start += s.per;
            x = start;
            if (x >= x_hi) break;
            if (++idx < (int64_t)s.items * p.Hkv) continue;
            idx = 0;
            int n = 0;
            do {
                ++b;
                row = p.c.q_start[b];
                n = p.c.q_start[b + 1] - row;
            } while (n == 0 && b + 1 < p.c.B);
            s = rq_seq(p, p.c.prefix[b], n);
            last_b = b;
            ok = blocks_ok();
        }
    }
    __syncthreads();
    if (tid == 0) {
        if (late) {
            // the sequences with work in this run (those behind where it ended, too)
            int64_t end = at.base;
            for (int b = at.b; b < p.c.B && end < x_hi; ++b) {
                const int n = p.c.q_start[b + 1] - p.c.q_start[b];
                end += rq_units(p, p.c.prefix[b], n);
                if (n > 0) {
                    p.status[b] = TV_ERR_TIMEOUT;
                    last_b = b;
                }
            }
            rec0 = rec1 = make_int4(first_b, last_b, 0, RQ_LATE);
        }
        p.rec[2 * blockIdx.x] = rec0;
        p.rec[2 * blockIdx.x + 1] = rec1;
    }
}

// Joins the pieces of the items that run borders cut, as chunk_tc_join_kernel does: the CTA of
// slot 2 r + 1 takes the item that starts in run r and goes on.
template <int D, int NT>
__global__ void __launch_bounds__(RQ_JOIN_THREADS) rows_q8_join_kernel(const __grid_constant__ RqParams p, int ctas) {
    constexpr int ROWS = RqShape<NT>::ROWS;
    pdl_wait();
    pdl_launch_dependents();
    const int4 rec = __ldcg(&p.rec[2 * blockIdx.x + 1]);
    if (rec.w & RQ_LATE)
        for (int b = rec.x + (int)threadIdx.x; b <= rec.y; b += RQ_JOIN_THREADS)
            if (p.c.q_start[b] != p.c.q_start[b + 1]) p.status[b] = TV_ERR_TIMEOUT;
    if (!(rec.w & RQ_PIECE)) return;
    const int rows = rec.y * p.G;
    for (int e = threadIdx.x; e < rows * (D / 4); e += RQ_JOIN_THREADS) {
        const int rr = e / (D / 4), c = e % (D / 4) * 4;
        float mx = -INFINITY, den = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        int slot = 2 * blockIdx.x + 1;
        int4 r = rec;
        while (true) {
            if (r.w & RQ_LATE) {
                den = 1.f;
                acc = make_float4(0.f, 0.f, 0.f, 0.f);
                break;
            }
            const int ahead = slot + (slot & 1 ? 1 : 2);
            const bool more = !(r.w & RQ_LAST) && ahead < 2 * ctas;
            const int4 nr = more ? __ldcg(&p.rec[ahead]) : r;
            if (r.w & RQ_PIECE) {
                const float* sl = p.part + (int64_t)slot * ROWS * (D + 2);
                const float mk = __ldcg(sl + ROWS * D + rr), lk = __ldcg(sl + ROWS * (D + 1) + rr);
                const float4 y = __ldcg(reinterpret_cast<const float4*>(sl + rr * D + c));
                const float mm = fmaxf(mx, mk), bz = mm == -INFINITY ? 0.f : mm;
                const float f = exp2f(mx - bz), w = exp2f(mk - bz);
                den = times_exp2(lk, mk - bz) + (mx == -INFINITY ? 0.f : times_exp2(den, mx - bz));
                acc.x = fmaf(w, y.x, acc.x * f);
                acc.y = fmaf(w, y.y, acc.y * f);
                acc.z = fmaf(w, y.z, acc.z * f);
                acc.w = fmaf(w, y.w, acc.w * f);
                mx = mm;
            }
            if (!more) break;
            slot = ahead;
            r = nr;
        }
        const float inv = exp2f(-RQ_BIAS) / den;
        const int tok = rr / p.G, head = rr - tok * p.G;
        const uint2 y = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        *reinterpret_cast<uint2*>(p.out + 2 * ((int64_t)(rec.x + tok) * p.o_stride + (int64_t)(rec.z * p.G + head) * D + c)) = y;
    }
}

// n-tiles of 8 rows for the tokens that a sequence has on average; 0: more rows than this is for.
// (128 sequences of 2,500 keys, 32/8 heads of 128, us, here and by attn_chunk_q8.cu: 4 rows 109 and
// 242, 8 rows 111 and 244, 16 rows 152 and 244, 24 rows 195 and 245; 16 sequences: 24 and 44, 26 and
// 45, 34 and 45, 45 and 46.  A fourth tile would cost as much again.)  The lengths of the sequences are not
// known to the host, so a long chunk among decoding sequences is cut into items of a few tokens here, or
// they take tiles of 128 rows there: 64 sequences and a chunk of 300 rows after 8,000 keys 332 us (alone 102 and 72),
// and one of 512 336 (113 and 93).
int rq_tiles(int T, int B, int G) {
    const int64_t per = B > 0 ? ((int64_t)T + B - 1) / B : T;
    const int64_t rows = per * G;
    return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 0;
}
template <int NT>
int rq_ctas() { return RqShape<NT>::PER_SM * device_sm_count(); }
int rq_ctas(int nt) { return nt == 1 ? rq_ctas<1>() : nt == 2 ? rq_ctas<2>() : rq_ctas<3>(); }

template <int D, int NT, bool CAP>
tv_status rq_launch(const ChunkAttnArgs& a, const RqParams& p, const CUtensorMap& km, const CUtensorMap& vm) {
    using S = RqShape<NT>;
    auto fn = rows_q8_kernel<D, NT, CAP>;
    constexpr int SMEM = RQ_WARPS * S::STAGES * 2 * 16 * D + 1024;
    static_assert(RQ_WARPS * S::ROWS * D * 4 <= SMEM - 1024, "the warps' results in the stages' room");
    static std::atomic<bool> set[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TV_ERR_CUDA;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess) {
            cudaGetLastError();
            return TV_ERR_CUDA;
        }
        set[dev] = true;
    }
    const int ctas = rq_ctas<NT>();
    LaunchCfg lc(dim3((unsigned)ctas), dim3(RQ_THREADS), SMEM, a.stream);
    if (cudaLaunchKernelEx(&lc.cfg, fn, km, vm, p) != cudaSuccess) return TV_ERR_CUDA;
    LaunchCfg lj(dim3((unsigned)ctas), dim3(RQ_JOIN_THREADS), 0, a.stream);
    return cudaLaunchKernelEx(&lj.cfg, rows_q8_join_kernel<D, NT>, p, ctas) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

template <int D, bool CAP>
tv_status rq_launch_tiles(const ChunkAttnArgs& a, const RqParams& p, const CUtensorMap& km, const CUtensorMap& vm, int nt) {
    if (nt == 1) return rq_launch<D, 1, CAP>(a, p, km, vm);
    if (nt == 2) return rq_launch<D, 2, CAP>(a, p, km, vm);
    return rq_launch<D, 3, CAP>(a, p, km, vm);
}

}  // namespace

bool rows_q8_applicable(int T, int B, int Hq, int Hkv) { return rq_tiles(T, B, Hq / Hkv) > 0; }

size_t rows_q8_workspace(int T, int B, int Hq, int Hkv, int d) {
    const int nt = rq_tiles(T, B, Hq / Hkv);
    return (size_t)2 * rq_ctas(nt) * ((size_t)8 * nt * (d + 2) * sizeof(float) + sizeof(int4));
}

tv_status launch_rows_q8(const ChunkAttnArgs& a) {
    const int64_t rows = (int64_t)a.num_blocks * a.Hkv * a.bs;
    if (rows >= (1ll << 31)) return TV_ERR_UNSUPPORTED;
    CUtensorMap km{}, vm{};
    if (a.d == 128 && (!make_code_map(&km, a.k_cache, rows) || !make_code_map(&vm, a.v_cache, rows))) return TV_ERR_CUDA;
    const int nt = rq_tiles(a.T, a.B, a.Hq / a.Hkv);
    RqParams p{};
    p.c = ChunkView{a.q_start, a.prefix_lens, a.block_table, a.T, a.B, a.max_blocks, a.bs, a.num_blocks};
    p.q = static_cast<const uint8_t*>(a.q);
    p.k = static_cast<const uint8_t*>(a.k_cache);
    p.v = static_cast<const uint8_t*>(a.v_cache);
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.mask = a.mask;
    p.out = static_cast<uint8_t*>(a.out);
    p.q_stride = a.q_stride;
    p.o_stride = a.out_stride;
    p.status = a.status;
    p.rec = static_cast<int4*>(a.ws);
    p.part = reinterpret_cast<float*>(p.rec + 2 * rq_ctas(nt));
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.npt = 8 * nt / p.G;
    p.window = a.window;
    p.sinks = a.window > 0 ? a.sinks : 0;
    p.late = test_late_wait();
    p.scale_log2 = a.softcap > 0.f ? fminf(2.f * RQ_LOG2E * a.scale / a.softcap, 3e38f) : a.scale * RQ_LOG2E;
    p.cap_log2 = a.softcap * RQ_LOG2E;
    if (a.softcap > 0.f) {
        const double k = (double)a.scale / a.softcap;
        for (int e = 0; e < 3; ++e) p.cap_c[e] = (float)(RQ_TANH_C[e] * a.scale * 1.4426950408889634 * pow(k, 2 * e));
        const double small = k > 1e5 ? 0.0 : std::min((k < 1e-10 ? 0.05 : RQ_TANH_SMALL) / k, 1e18);
        p.cap_small = (float)(small * small);
    }
    if (a.d == 128)
        return a.softcap > 0.f ? rq_launch_tiles<128, true>(a, p, km, vm, nt) : rq_launch_tiles<128, false>(a, p, km, vm, nt);
    return a.softcap > 0.f ? rq_launch_tiles<64, true>(a, p, km, vm, nt) : rq_launch_tiles<64, false>(a, p, km, vm, nt);
}

}  // namespace tv
