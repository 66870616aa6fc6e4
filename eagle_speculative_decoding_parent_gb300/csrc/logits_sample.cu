// logits_sample: the token that a given uniform number draws from a row of logits after
// temperature, top-k, top-p and min-p, and on request the distribution that is left.
//
// With the entries ordered by (logit descending, index ascending), every filter keeps a prefix, so
// a row's filters come down to one cut in that order.  Weights are exp((x - max) / T) in fixed
// point, 2^-42 steps, off by some 2^-39 of themselves: their sums do not depend on an
// order, and a token or a cut differs from the exact one only where the given number is as
// near to a border.
//
// A cluster of CTAs holds a row in shared memory, a slice each:
//   1  the maximum;
//   2  entries counted by (max - x) / T in 2,048 bins of 1/64, over the cluster;
//   3  top-k: the bin that holds the k-th entry, its entries in a list, ranked;
//   4  top-p: the bin where the mass reaches top_p of what top-k left (estimated from the counts,
//      then proved by the exact sums on both sides, or corrected), its entries ranked;
//   5  the mass that is left, by warps in index order: the one in which the draw falls searches;
//   6  the distribution.
// Bins with more entries than the list holds (long runs of equal logits) are cut by bisection
// over the logits' bits and a count of equal ones by index.
#include <cuda_bf16.h>
#include <float.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "tv_device.cuh"
#include "tv_internal.h"

namespace tv {

namespace {

constexpr int LS_THREADS = 512;
constexpr int LS_WARPS = LS_THREADS / 32;
constexpr int LS_STEP = LS_WARPS * 128;      // a slice is a multiple of this
constexpr int LS_CLUSTER_MAX = 16;
constexpr int LS_SLICE = 16384;              // entries per CTA, two CTAs per SM
constexpr int LS_SLICE_MAX = 49152;          // longer rows: one CTA per SM
constexpr int LS_BINS = 2048;
constexpr float LS_BIN = 64.f;               // bins per unit of (max - x) / T
constexpr int LS_LIST = 1024;
constexpr int LS_FRAC = 42;                  // a weight of 1 is 2^42

// 2^(62 - j / 64)
__constant__ uint64_t LS_TABLE[64] = {
    0x4000000000000000ull, 0x3f4f83033d21b05dull, 0x3ea0ecb6dc8a80cfull, 0x3df437dcc2b44eeeull,
    0x3d495f454921b30bull, 0x3ca05dcf167fec4eull, 0x3bf92e66f736bd73ull, 0x3b53cc07b6650ae1ull,
    0x3ab031b9f7490e4cull, 0x3a0e5a940f12f71aull, 0x396e41b9df20d22aull, 0x38cfe25cafa29694ull,
    0x383337bb0aa53844ull, 0x37983d209783a449ull, 0x36feede5f6bc8dd5ull, 0x366745709e2bf5edull,
    0x35d13f32b5a75abdull, 0x353cd6aaf3fb7e88ull, 0x34aa07647c4ab917ull, 0x3418ccf6bbcac965ull,
    0x3389230547e12039ull, 0x32fb053fbc9c9f17ull, 0x326e6f619b8bc9e9ull, 0x31e35d322aee6c57ull,
    0x3159ca845541b6b7ull, 0x30d1b3368925d902ull, 0x304b1332999c2516ull, 0x2fc5e66d9e9cc421ull,
    0x2f4228e7d6030db0ull, 0x2ebfd6ac84cf917full, 0x2e3eebd1d8bee7baull, 0x2dbf6478ca345de4ull,
    0x2d413cccfe779921ull, 0x2cc47104aa444922ull, 0x2c48fd6074ab0964ull, 0x2bcede2b5a4290ddull,
    0x2b560fba90a852b2ull, 0x2ade8e6d6a4fb4ceull, 0x2a6856ad3a9f03beull, 0x29f364ed3a594d5aull,
    0x297fb5aa6c544e3bull, 0x290d456b8279a028ull, 0x289c10c0c3125a06ull, 0x282c1443ee5c53f1ull,
    0x27bd4c982468446bull, 0x274fb669cb3fedd4ull, 0x26e34e6e7553954eull, 0x26781164c82dfe99ull,
    0x260dfc14636e2a5cull, 0x25a50b4dc8061680ull, 0x253d3bea3fbdc258ull, 0x24d68acbc4f9ba4bull,
    0x2470f4dceac470ceull, 0x240c7710c519ac77ull, 0x23a90e62d17354f0ull, 0x2346b7d6df96ea79ull,
    0x22e57078faa2f5baull, 0x2285355d525bbf67ull, 0x222603a024b6a14aull, 0x21c7d865a7a34404ull,
    0x216ab0d9f3121ec5ull, 0x210e8a30eb379012ull, 0x20b361a62b0ae876ull, 0x2059347cef00c1ddull,
};

struct LsParams {
    const void* logits;
    const float* uniform;
    const int32_t* node_counts;
    const float* temp;
    const int32_t* top_k;
    const float *top_p, *min_p;
    int32_t* tokens;
    float* probs;
    int32_t* status;
    int N, V, slice, ctas;   // ctas: of a row
};

// The order of the entries: smaller is better, all different.
__device__ __forceinline__ uint32_t ls_bits(float x) {          // larger numbers, larger bits (no -0)
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t ls_key(float x, int idx) {
    return (uint64_t)(~ls_bits(x)) << 32 | (uint32_t)idx;
}

// exp((x - top) / T) in 2^-42, rounded; (ch, cl): log2(e) / T.  The exponent t = n / 64 + r in two
// floats; 2^-r = 1 - p + p^2 / 2 - p^3 / 6 + p^4 / 24 with p = r ln 2 <= 0.0055 (the next term is
// 2^-44), p in two floats too, and 2^(-n / 64) from a table and a shift.
__device__ __forceinline__ uint64_t ls_weight(float x, float top, float ch, float cl, const uint64_t* table) {
    const float d = top - x, bb = d - top, dl = (top - (d - bb)) - (x + bb);   // top - x = d + dl
    const float t = d * ch;
    if (!(t < (float)(LS_FRAC + 1))) return 0ull;
    const float tl = fmaf(d, cl, fmaf(dl, ch, fmaf(d, ch, -t)));
    const float nf = rintf(t * 64.f), r = fmaf(nf, -0.015625f, t);
    const int n = (int)nf;
    constexpr float LN2H = 0.69314718246459960938f, LN2L = -1.90465429995776804525e-9f;
    const float p = LN2H * r;
    const float e = fmaf(LN2H, tl, fmaf(LN2L, r, fmaf(LN2H, r, -p)));
    const float quad = p * p * fmaf(-p, fmaf(-p, 1.f / 24.f, 1.f / 6.f), 0.5f);
    // -p to 2^-29, what is left of it and the rest to 2^-38
    constexpr float M1 = 1.5f / 64.f, M2 = 1.5f / 32768.f;
    const float a = M1 - p, left = (M1 - a) - p;
    const float b = M2 + ((quad - e) + left);
    const int i = ((__float_as_int(a) - __float_as_int(M1)) << 9) + (__float_as_int(b) - __float_as_int(M2));
    const uint64_t w = table[n & 63];
    const uint64_t v = w + (uint64_t)(((int64_t)(int)(w >> 32) * i) >> 6);
    const int q = n >> 6;
    return (v + (1ull << (61 - LS_FRAC + q))) >> (62 - LS_FRAC + q);
}

__device__ __forceinline__ void remote_st_u64(uint64_t* p, uint32_t rank, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_rank(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t remote_add_u32(uint32_t* p, uint32_t rank, uint32_t v) {
    uint32_t r;
    asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(map_rank(p, rank)), "r"(v) : "memory");
    return r;
}
__device__ __forceinline__ uint32_t remote_ld_u32(const uint32_t* p, uint32_t rank) {
    uint32_t r;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(r) : "r"(map_rank(p, rank)) : "memory");
    return r;
}

template <typename E>
__global__ void __launch_bounds__(LS_THREADS, 2) logits_sample_kernel(const __grid_constant__ LsParams p) {
    extern __shared__ __align__(16) float xs[];            // the slice
    __shared__ uint32_t hist[LS_BINS], tot[LS_BINS];       // the slice's counts, the row's
    __shared__ uint64_t list[LS_LIST], weight[LS_LIST];    // first CTA: entries of one bin
    __shared__ uint64_t table[64];
    __shared__ uint64_t part[3][LS_WARPS];                 // per warp
    __shared__ uint64_t peer[2][3][LS_CLUSTER_MAX];        // per CTA, two exchanges in turn
    __shared__ uint64_t result;                            // of the first CTA
    __shared__ uint32_t list_n[2];
    __shared__ uint32_t pick[2];                           // a bin, entries before it
    __shared__ float fpart[LS_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = p.ctas, me = (int)(blockIdx.x % C);
    const int64_t row = blockIdx.x / C;
    const int b = (int)(row / p.N), node = (int)(row % p.N);
    const int x0 = me * p.slice, n = max(0, min(p.slice, p.V - x0));
    const int chunk = p.slice / LS_WARPS, w0 = warp * chunk;   // a warp's entries
    if (tid < 64) table[tid] = LS_TABLE[tid];
    if (tid < 2) list_n[tid] = 0u;
    if (tid == 0) result = ~0ull;
    for (int i = tid; i < LS_BINS; i += LS_THREADS) hist[i] = 0u;
    pdl_launch_dependents();
    pdl_wait();
    const int cnt = p.node_counts ? p.node_counts[b] : p.N;
    if (cnt >= 1 && cnt <= p.N && node >= cnt) return;         // an absent node (the whole cluster)
    const float T = p.temp ? p.temp[b] : 1.f, top_p = p.top_p ? p.top_p[b] : 1.f;
    const float min_p = p.min_p ? p.min_p[b] : 0.f, u = p.uniform[row];
    const int k = p.top_k ? p.top_k[b] : 0;
    int err = cnt >= 1 && cnt <= p.N ? TV_OK : TV_ERR_OUT_OF_RANGE;
    if (err == TV_OK && !((T == 0.f || (T >= FLT_MIN && T <= FLT_MAX)) && top_p > 0.f && top_p <= 1.f && min_p >= 0.f &&
                          min_p <= 1.f && u >= 0.f && u < 1.f))
        err = TV_ERR_BAD_VALUES;
    float* out = p.probs ? p.probs + row * p.V + x0 : nullptr;
    auto refuse = [&]() {
        if (out)
            for (int i = tid; i < n; i += LS_THREADS) out[i] = 0.f;
        if (me == 0 && tid == 0) {
            p.tokens[row] = -1;
            p.status[row] = err;
        }
    };
    if (err != TV_OK) return refuse();

    // ---- the slice, and its maximum (a NaN wins)
    float mx = -INFINITY;
    auto take = [&](float x) -> float {
        x += 0.f;                                              // -0 is 0
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(mx), "f"(x));
        return x;
    };
    {
        const E* src = static_cast<const E*>(p.logits) + row * p.V + x0;
        if ((reinterpret_cast<uintptr_t>(src) & (4 * sizeof(E) - 1)) == 0) {
            constexpr int U = 4;
            for (int i = tid * 4; i < p.slice; i += LS_THREADS * 4 * U) {
                float4 v[U];
#pragma unroll
                for (int y = 0; y < U; ++y) {
                    const int e = i + y * LS_THREADS * 4;
                    v[y] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                    if (e + 4 <= n) {
                        if constexpr (sizeof(E) == 4) {
                            v[y] = __ldcs(reinterpret_cast<const float4*>(src + e));
                        } else {
                            const uint2 h = __ldcs(reinterpret_cast<const uint2*>(src + e));
                            v[y] = make_float4(__uint_as_float(h.x << 16), __uint_as_float(h.x & 0xffff0000u),
                                               __uint_as_float(h.y << 16), __uint_as_float(h.y & 0xffff0000u));
                        }
                    } else if (e < n) {
                        v[y].x = (float)src[e];
                        if (e + 1 < n) v[y].y = (float)src[e + 1];
                        if (e + 2 < n) v[y].z = (float)src[e + 2];
                    }
                }
#pragma unroll
                for (int y = 0; y < U; ++y) {
                    const int e = i + y * LS_THREADS * 4;
                    if (e < p.slice)
                        *reinterpret_cast<float4*>(xs + e) = make_float4(take(v[y].x), take(v[y].y), take(v[y].z), take(v[y].w));
                }
            }
        } else {
            constexpr int U = 8;
            for (int i = tid; i < p.slice; i += LS_THREADS * U) {
                float v[U];
#pragma unroll
                for (int y = 0; y < U; ++y) v[y] = i + y * LS_THREADS < n ? (float)src[i + y * LS_THREADS] : -INFINITY;
#pragma unroll
                for (int y = 0; y < U; ++y)
                    if (i + y * LS_THREADS < p.slice) xs[i + y * LS_THREADS] = take(v[y]);
            }
        }
    }
    // ---- exchanges over the cluster: what a CTA's threads pass, reduced
    int turn = 0;
    auto exchange = [&](uint64_t v0, uint64_t v1, uint64_t v2) {  // per CTA values into every CTA's peer[turn]
        if (tid < C) {
            remote_st_u64(&peer[turn][0][me], tid, v0);
            remote_st_u64(&peer[turn][1][me], tid, v1);
            remote_st_u64(&peer[turn][2][me], tid, v2);
        }
        cluster_barrier_all();
        turn ^= 1;                                             // (read peer[turn ^ 1])
    };
    auto block_sum = [&](uint64_t (&v)[3], int count) {
        for (int c = 0; c < count; ++c) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v[c] += __shfl_xor_sync(0xffffffffu, v[c], o);
            if (lane == 0) part[c][warp] = v[c];
        }
        __syncthreads();
        for (int c = 0; c < count; ++c) {
            v[c] = 0ull;
            for (int w = 0; w < LS_WARPS; ++w) v[c] += part[c][w];
        }
        __syncthreads();
    };
    auto cluster_sum = [&](uint64_t (&v)[3], int count) {
        block_sum(v, count);
        exchange(v[0], v[1], v[2]);
        for (int c = 0; c < count; ++c) {
            v[c] = 0ull;
            for (int r = 0; r < C; ++r) v[c] += peer[turn ^ 1][c][r];
        }
    };
    // f(entry, its place in the slice) over the warp's entries, four at a time
    auto entries = [&](auto f) {
        for (int i = lane * 4; i < chunk; i += 128) {
            const float4 v = *reinterpret_cast<const float4*>(xs + w0 + i);
            f(v.x, w0 + i);
            f(v.y, w0 + i + 1);
            f(v.z, w0 + i + 2);
            f(v.w, w0 + i + 3);
        }
    };
    float top;
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, mx, o);
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(mx), "f"(y));
        }
        if (lane == 0) fpart[warp] = mx;
        __syncthreads();
        mx = fpart[0];
        for (int w = 1; w < LS_WARPS; ++w) asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(mx), "f"(fpart[w]));
        cluster_barrier_all();                                 // every CTA has started
        exchange(__float_as_uint(mx), 0ull, 0ull);
        top = __uint_as_float((uint32_t)peer[turn ^ 1][0][0]);
        for (int r = 1; r < C; ++r) {
            const float y = __uint_as_float((uint32_t)peer[turn ^ 1][0][r]);
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(top) : "f"(top), "f"(y));
        }
    }
    if (!(fabsf(top) <= FLT_MAX)) {                            // NaN, infinity, or nothing above -infinity
        err = TV_ERR_BAD_VALUES;
        refuse();
        cluster_barrier_all();                                 // (no CTA leaves while others write to it)
        return;
    }
    auto place = [&](int i) -> int { return x0 + i; };
    int token = -1;
    if (T == 0.f) {
        // ---- the best entry, the first of equal ones
        uint32_t best = 0xffffffffu;
        entries([&](float x, int i) {
            if (x == top) best = min(best, (uint32_t)place(i));
        });
        best = __reduce_min_sync(0xffffffffu, best);
        if (lane == 0) part[0][warp] = best;
        __syncthreads();
        for (int w = 0; w < LS_WARPS; ++w) best = min(best, (uint32_t)part[0][w]);
        exchange(best, 0ull, 0ull);
        for (int r = 0; r < C; ++r) best = min(best, (uint32_t)peer[turn ^ 1][0][r]);
        token = (int)best;
        if (me == 0 && tid == 0) {
            p.tokens[row] = token;
            p.status[row] = TV_OK;
        }
        if (out)
            for (int i = tid; i < n; i += LS_THREADS) out[i] = place(i) == token ? 1.f : 0.f;
        return;
    }
    const double c64 = 1.4426950408889634 / (double)T;
    const float ch = (float)c64, cl = (float)(c64 - (double)ch);
    const float bin_scale = fminf(LS_BIN / T, 1e38f);
    auto bin_of = [&](float x) -> int { return (int)fminf((top - x) * bin_scale, (float)(LS_BINS - 1)); };
    auto weigh = [&](float x) -> uint64_t { return ls_weight(x, top, ch, cl, table); };
    const bool use_k = k > 0 && k < p.V, use_p = top_p < 1.f;
    uint64_t cut = ~0ull;                                      // entries up to this key are kept
    // The cut of a run of entries that no list holds, by bisection over the logits' bits: the
    // first key with which count entries, or a mass above before, are kept (`kept` entries count).
    auto bisect = [&](bool mass, uint64_t need, uint64_t limit) -> uint64_t {
        uint32_t lo = 0u, hi = 0xffffffffu;                    // largest bits from which on there are `need`
        uint64_t v[3];
        auto above = [&](uint32_t bits, bool strict) -> uint64_t {
            v[0] = 0ull;
            entries([&](float x, int i) {
                const uint32_t y = ls_bits(x);
                if ((strict ? y > bits : y >= bits) && place(i) < p.V && ls_key(x, place(i)) <= limit) v[0] += mass ? weigh(x) : 1ull;
            });
            cluster_sum(v, 1);
            return v[0];
        };
        while (lo < hi) {
            const uint32_t mid = lo + ((hi - lo) >> 1) + 1u;
            if (above(mid, false) >= need) lo = mid;
            else hi = mid - 1u;
        }
        const uint64_t more = above(lo, true);
        const float x = __uint_as_float((lo & 0x80000000u) ? lo & 0x7fffffffu : ~lo);
        const uint64_t w = mass ? weigh(x) : 1ull;
        // the first `ties` of the entries that equal x
        const uint64_t ties = w == 0ull ? 1ull << 32 : (need > more ? (need - more + w - 1ull) / w : 1ull);
        v[0] = 0ull;
        entries([&](float y, int i) { v[0] += ls_bits(y) == lo && place(i) < p.V ? 1ull : 0ull; });
        uint64_t mine = v[0];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
        block_sum(v, 1);
        exchange(v[0], 0ull, 0ull);
        uint64_t before = 0ull, all = 0ull;
        for (int r = 0; r < C; ++r) {
            if (r < me) before += peer[turn ^ 1][0][r];
            all += peer[turn ^ 1][0][r];
        }
        const uint64_t want = min(ties, all);
        if (want > before && want <= before + v[0]) {
            // in this CTA: its warps in order
            if (lane == 0) part[0][warp] = mine;
            __syncthreads();
            for (int w2 = 0; w2 < warp; ++w2) before += part[0][w2];
            if (want > before && want <= before + mine)
                for (int i = 0; i < chunk; i += 32) {
                    const uint32_t m = __ballot_sync(0xffffffffu, ls_bits(xs[w0 + i + lane]) == lo && place(w0 + i + lane) < p.V);
                    const int here = __popc(m);
                    if (want <= before + here) {
                        const int at = __fns(m, 0, (int)(want - before));
                        if (lane < C) remote_st_u64(&result, lane, ls_key(x, place(w0 + i + at)));
                        break;
                    }
                    before += here;
                }
        }
        cluster_barrier_all();
        const uint64_t found = result;
        cluster_barrier_all();                                 // (read before it is written again)
        return found;
    };
    // The entries of a bin (up to `limit`) in the first CTA's list, ranked there; the key of the
    // one with rank `rank`, or (mass) of the last one that begins below `need`.
    auto cut_in_bin = [&](int which, int bin, bool mass, uint64_t rank, uint64_t base, uint64_t need, uint64_t limit) -> uint64_t {
        entries([&](float x, int i) {
            if (bin_of(x) != bin || place(i) >= p.V) return;
            const uint64_t key = ls_key(x, place(i));
            if (key > limit) return;
            const uint32_t at = remote_add_u32(&list_n[which], 0, 1u);
            if (at < LS_LIST) remote_st_u64(&list[at], 0, key);
        });
        cluster_barrier_all();
        if (me == 0) {
            const int m = min((int)list_n[which], LS_LIST);
            if (mass)
                for (int e = tid; e < m; e += LS_THREADS) {
                    const uint32_t bits = ~(uint32_t)(list[e] >> 32);
                    weight[e] = weigh(__uint_as_float((bits & 0x80000000u) ? bits & 0x7fffffffu : ~bits));
                }
            __syncthreads();
            for (int e = tid; e < m; e += LS_THREADS) {
                const uint64_t key = list[e];
                if (mass) {
                    uint64_t before = base;
                    for (int f = 0; f < m; ++f) before += list[f] < key ? weight[f] : 0ull;
                    // the last one that begins below: the next one does not, or there is none
                    if (before < need && before + weight[e] >= need)
                        for (int r = 0; r < C; ++r) remote_st_u64(&result, r, key);
                } else {
                    uint64_t before = 0ull;
                    for (int f = 0; f < m; ++f) before += list[f] < key ? 1ull : 0ull;
                    if (before == rank)
                        for (int r = 0; r < C; ++r) remote_st_u64(&result, r, key);
                }
            }
        }
        cluster_barrier_all();
        const uint64_t found = result;
        cluster_barrier_all();
        return found;
    };
    if (use_k || use_p) {
        // ---- counts per bin, over the cluster: a CTA sums a part of the bins for all
        entries([&](float x, int) {
            const int bin = bin_of(x);
            if (bin < LS_BINS - 1) atomicAdd(&hist[bin], 1u);
        });
        cluster_barrier_all();
        for (int i = me * LS_THREADS + tid; i < LS_BINS; i += C * LS_THREADS) {
            uint32_t s = 0u;
            for (int r = 0; r < C; ++r) s += remote_ld_u32(&hist[i], r);
            for (int r = 0; r < C; ++r) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(&tot[i], r)), "r"(s) : "memory");
        }
        cluster_barrier_all();
        // four bins per thread; the last one holds what is left
        constexpr int PER = LS_BINS / LS_THREADS;
        uint32_t c[PER], s = 0u;
#pragma unroll
        for (int e = 0; e < PER; ++e) s += c[e] = tot[tid * PER + e];
        uint32_t incl = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) part[0][warp] = incl;
        __syncthreads();
        uint32_t before = incl - s;
        for (int w = 0; w < warp; ++w) before += (uint32_t)part[0][w];
        if (tid == LS_THREADS - 1) c[PER - 1] = tot[LS_BINS - 1] = (uint32_t)p.V - (before + s);
        __syncthreads();
        int k_bin = LS_BINS - 1;
        uint32_t k_rank = (uint32_t)p.V;
        if (use_k) {
            uint32_t at = before;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                if (at < (uint32_t)k && (uint32_t)k <= at + c[e]) {
                    pick[0] = tid * PER + e;
                    pick[1] = at;
                }
                at += c[e];
            }
            __syncthreads();
            k_bin = (int)pick[0];
            k_rank = (uint32_t)k - pick[1];                     // entries of that bin that are kept
            cut = tot[k_bin] <= LS_LIST ? cut_in_bin(0, k_bin, false, k_rank - 1u, 0ull, 0ull, ~0ull)
                                        : bisect(false, (uint64_t)k, ~0ull);
        }
        if (use_p) {
            // ---- the bin where the mass reaches top_p, from the counts at first
            float m[PER], ms = 0.f;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int bin = tid * PER + e;
                const uint32_t in = use_k && bin >= k_bin ? (bin == k_bin ? k_rank : 0u) : c[e];
                m[e] = (float)in * exp2f(-1.44269504f * ((float)bin + 0.5f) / LS_BIN);
                ms += m[e];
            }
            float mi = ms;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float y = __shfl_up_sync(0xffffffffu, mi, o);
                if (lane >= o) mi += y;
            }
            if (lane == 31) fpart[warp] = mi;
            if (tid == 0) pick[0] = (uint32_t)k_bin;
            __syncthreads();
            float at = mi - ms, all = 0.f;
            for (int w = 0; w < LS_WARPS; ++w) {
                if (w < warp) at += fpart[w];
                all += fpart[w];
            }
            const float goal = top_p * all;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                if (at < goal && goal <= at + m[e]) atomicMin(&pick[0], (uint32_t)(tid * PER + e));
                at += m[e];
            }
            __syncthreads();
            int bin = (int)pick[0], lo = 0, hi = k_bin;
            uint64_t v[3], need = 0ull;
            for (int tries = 0;; ++tries) {
                v[0] = v[1] = v[2] = 0ull;
                entries([&](float x, int i) {
                    if (cut != ~0ull && ls_key(x, place(i)) > cut) return;
                    const int y = bin_of(x);
                    const uint64_t w = weigh(x);
                    if (y < bin) v[0] += w;
                    else if (y == bin) v[1] += w;
                    else v[2] += w;
                });
                cluster_sum(v, 3);
                // kept: what begins below top_p of the sum (an integer begins below it when it does below
                // the next one)
                need = (uint64_t)ceil((double)top_p * (double)(v[0] + v[1] + v[2]));
                if (v[0] < need && need <= v[0] + v[1]) break;
                if (need <= v[0]) hi = bin - 1;
                else lo = bin + 1;
                if (lo >= hi) {
                    bin = min(max(lo, 0), LS_BINS - 1);
                    if (tries > 2 * 11) break;
                } else {
                    bin = tries < 2 ? (need <= v[0] ? hi : lo) : (lo + hi) >> 1;
                }
            }
            cut = min(cut, tot[bin] <= LS_LIST ? cut_in_bin(1, bin, true, 0ull, v[0], need, cut) : bisect(true, need, cut));
        }
    }
    // ---- the mass that is left, and where the draw falls
    const uint64_t least = (uint64_t)ceil((double)min_p * (double)(1ull << LS_FRAC));
    auto kept = [&](float x, int i) -> uint64_t {
        if (cut != ~0ull && ls_key(x, place(i)) > cut) return 0ull;
        const uint64_t w = weigh(x);
        return w >= least ? w : 0ull;
    };
    uint64_t v[3] = {0ull, 0ull, 0ull};
    entries([&](float x, int i) { v[0] += kept(x, i); });
    uint64_t mine = v[0];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    block_sum(v, 1);
    exchange(v[0], 0ull, 0ull);
    uint64_t before = 0ull, all = 0ull;
    for (int r = 0; r < C; ++r) {
        if (r < me) before += peer[turn ^ 1][0][r];
        all += peer[turn ^ 1][0][r];
    }
    const uint64_t goal = (uint64_t)((double)u * (double)all);  // the first entry whose sum exceeds it
    if (goal >= before && goal < before + v[0]) {
        if (lane == 0) part[0][warp] = mine;
        __syncthreads();
        for (int w = 0; w < warp; ++w) before += part[0][w];
        if (goal >= before && goal < before + mine)
            for (int i = 0; i < chunk; i += 32) {
                uint64_t s = kept(xs[w0 + i + lane], w0 + i + lane);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t y = __shfl_up_sync(0xffffffffu, s, o);
                    if (lane >= o) s += y;
                }
                const uint32_t over = __ballot_sync(0xffffffffu, before + s > goal);
                if (over != 0u) {
                    if (lane == 0) {
                        p.tokens[row] = place(w0 + i + __ffs(over) - 1);
                        p.status[row] = TV_OK;
                    }
                    break;
                }
                before += __shfl_sync(0xffffffffu, s, 31);
            }
    }
    if (out) {
        // weights again, in float32: 2^-22 of each, with the exponent's rounding
        const float inv = (float)((double)(1ull << LS_FRAC) / (double)all);
        for (int i = tid; i < n; i += LS_THREADS) {
            const float x = xs[i];
            float y = 0.f;
            if (cut == ~0ull || ls_key(x, place(i)) <= cut) {
                y = exp2f((x - top) * ch) * inv;
                if (min_p > 0.f && weigh(x) < least) y = 0.f;
            }
            out[i] = y;
        }
    }
}

template <typename E>
tv_status launch_sample(const LsParams& q, int64_t rows, cudaStream_t stream) {
    LsParams p = q;
    auto fn = logits_sample_kernel<E>;
    const int fewest = (p.V + LS_SLICE - 1) / LS_SLICE;
    int C;
    if (fewest > LS_CLUSTER_MAX) {
        C = LS_CLUSTER_MAX;
    } else {
        // few rows: more CTAs per row, while they have a few thousand entries each
        C = fewest;
        while (C * 2 <= LS_CLUSTER_MAX && rows * C * 2 <= 2 * device_sm_count() && p.V > C * 2 * LS_STEP) C *= 2;
    }
    p.ctas = C;
    p.slice = ((p.V + C - 1) / C + LS_STEP - 1) / LS_STEP * LS_STEP;
    if (p.slice > LS_SLICE_MAX) return TV_ERR_UNSUPPORTED;
    if (rows * C > 0x7fffffff) return TV_ERR_UNSUPPORTED;
    const size_t smem = (size_t)p.slice * sizeof(float);
    static std::atomic<bool> set[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TV_ERR_CUDA;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, LS_SLICE_MAX * (int)sizeof(float)) != cudaSuccess ||
            cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
            cudaGetLastError();
            return TV_ERR_CUDA;
        }
        set[dev] = true;
    }
    LaunchCfg lc(dim3((unsigned)(rows * C)), dim3(LS_THREADS), smem, stream, (unsigned)C);
    return cudaLaunchKernelEx(&lc.cfg, fn, p) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // namespace

tv_status launch_logits_sample(const SampleArgs& a) {
    LsParams p{};
    p.logits = a.logits;
    p.uniform = a.uniform;
    p.node_counts = a.node_counts;
    p.temp = a.temp;
    p.top_k = a.top_k;
    p.top_p = a.top_p;
    p.min_p = a.min_p;
    p.tokens = a.tokens;
    p.probs = a.probs;
    p.status = a.status;
    p.N = a.N;
    p.V = a.V;
    const int64_t rows = (int64_t)a.B * a.N;
    return a.dt == TV_F32 ? launch_sample<float>(p, rows, a.stream) : launch_sample<__nv_bfloat16>(p, rows, a.stream);
}

}  // namespace tv
