// logits_sample: the token that a given uniform number draws from a row of logits after
// temperature, top-k, top-p and min-p, and on request the distribution that is left.
//
// With the entries ordered by (logit descending, index ascending), every filter keeps a prefix, so
// a row's filters come down to one cut in that order.  Weights are exp((x - max) / T) in fixed
// point, 2^-42 steps, off by some 2^-39 of themselves: their sums do not depend on an
// order, and a token or a cut differs from the exact one only where the given number is as
// near to a border.  (The sum that top-p of a whole row is taken of has its far entries in
// float32, off by at most 2^-18 of themselves: up to 2^17 entries with forty instructions each
// would cost more than the rest.)
//
// A cluster of CTAs holds a row in shared memory, a slice each, and nearly always only the entries
// near the maximum matter:
//   1  the maximum;
//   2  the entries within four reaches of it (by (max - x) / T) are counted, and for top-p of a whole
//      row what lies beyond is weighed roughly; the smallest reach that holds all that may be kept is
//      taken, and its entries' places are compacted;
//   3  their counts and exact weights by bins of 1/64; the first CTA sums those of the cluster, finds
//      the bins of the cuts, and ranks these bins' entries, in a list, by counting;
//   4  the mass that is left, CTA by CTA: the one in which the draw falls ranks what it keeps by
//      index (where thousands are kept: by warps in index order);
//   5  the distribution.
// Rows for which no reach does (hardly any filter, or nearly flat) take the same steps over the whole
// row: counts by bins, the bin of the mass estimated from them, then proved by exact sums on both
// sides or corrected.  Bins with more entries than the list holds (long runs of equal logits)
// are cut by bisection over the logits' bits and a count of equal ones by index.
// Distributions of many rows: steps 3 and 4 are a chain of barriers with the row in shared memory,
// and only some 38 rows are on the GPU at once.  So the cluster leaves the near entries in the
// distribution's place, the rest of it zero, and a second kernel settles a row per CTA from them.
// (In one kernel 790 us for the 832 rows below, in two 671 at that time.)
// A weight takes some forty instructions and few entries need theirs, scattered over the row: a
// thread marks them among 32 of its entries, and goes through the marks.
// Measured, rows of 128,256: one row of bfloat16 15-21 us, 64 rows with top-k, top-p and min-p 29
// (latency: launch, the slices, some eight barriers of a cluster; the best entries alone 8); 832
// rows of float32 with distributions: 214 the best entries, 349 min-p, 474 top-p, 470 no filter (of
// that 185 the exact weights of every entry), 856 top-p of flat rows; the bytes take 126.  59 % of the
// issue slots in the first kernel.
#include <cuda_bf16.h>
#include <float.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "tv_device.cuh"
#include "tv_internal.h"

namespace tv {

namespace {

constexpr int LS_THREADS = 512;
constexpr int LS_WARPS = LS_THREADS / 32;
constexpr int LS_STEP = LS_WARPS * 128;      // a slice is a multiple of this
constexpr int LS_CLUSTER_MAX = 16;
constexpr int LS_SLICE_BYTES = 65536;        // of a row per CTA, two CTAs per SM
constexpr int LS_SLICE_MAX = 49152;          // longer rows: one CTA per SM
constexpr int LS_BINS = 2048;
constexpr float LS_BIN = 64.f;               // bins per unit of (max - x) / T
// Reaches of the near entries, in bins: those within 6, 7.5, 9.25 and 10.6 of the maximum (the last
// weigh 2^-15.3 of the first or more).
constexpr int LS_REACHES = 4;
constexpr int LS_NEARER = 592, LS_NEAR = 680;
__device__ constexpr int ls_reach(int j) { return j == 0 ? 384 : j == 1 ? 480 : j == 2 ? LS_NEARER : LS_NEAR; }
static_assert(LS_NEAR % 2 == 0 && LS_NEAR * 12 <= LS_BINS * 4, "counts and masses (of 8 bytes, aligned) of the near bins in a histogram's room");
constexpr float LS_SMALL = 19.f;             // weights below 2^-19 enter the sum of all in float32
constexpr int LS_LIST = 1024;
constexpr int LS_HEAVY = 6144;               // near entries of a CTA (fewer beside the longest slices)
constexpr int LS_STATIC = 34 * 1024, LS_SHARED = 227 * 1024;   // other shared memory, all that there is
constexpr int LS_FEW = 4 * LS_THREADS;       // so many that what is kept of them is put into order
constexpr int LS_TRIES = 4;
// Rows left to logits_sample_rows_kernel, which holds at most so many near entries (more of them are
// read again for each use): dumped behind a header of so many words into the slices' part of the distribution; the status that says so.
// A last slice that is empty or shorter than the header has none, and no near entry.
constexpr int LS_ROW = 8192;
constexpr int LS_HEAD = 8;
constexpr int32_t LS_PENDING = -0x5eed;
constexpr int LS_BUCKETS = 1024;             // of the vocabulary, for the draw
constexpr int LS_FRAC = 42;                  // a weight of 1 is 2^42

// 2^(62 - j / 64)
__device__ const uint64_t LS_TABLE[64] = {
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
    int64_t rows, ahead;     // ahead: rows that the GPU holds at once
    int heavy;               // near entries of a CTA
    bool defer;              // distributions of many rows: the near entries to the second kernel
    __device__ __forceinline__ int cells(int r) const { return min(slice, V - r * slice); }   // of CTA r's slice (0 or less: none)
    __device__ __forceinline__ bool headed(int r) const { return cells(r) >= LS_HEAD; }
};

// The order of the entries: smaller is better, all different.
__device__ __forceinline__ uint32_t ls_bits(float x) {          // larger numbers, larger bits (no -0)
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t ls_key(float x, int idx) {
    return (uint64_t)(~ls_bits(x)) << 32 | (uint32_t)idx;
}

// f times z, f in [0, 1], exactly, rounded down, or (UP) up.
template <bool UP>
__device__ __forceinline__ uint64_t ls_part(float f, uint64_t z) {
    const uint32_t b = __float_as_uint(f), ex = max(b >> 23, 1u);
    const uint64_t mant = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0u);
    const int shift = 150 - (int)ex;                           // f = mant 2^-shift, 23 <= shift <= 149
    const uint64_t hi = __umul64hi(z, mant), lo = z * mant;
    const bool far = shift >= 64;
    const uint64_t whole = far ? (shift - 64 < 64 ? hi >> (shift - 64) : 0ull) : (hi << (64 - shift) | lo >> shift);
    const bool rest = far ? (lo != 0ull || (shift - 64 < 64 ? (hi & ((1ull << (shift - 64)) - 1ull)) != 0ull : hi != 0ull))
                          : (lo & ((1ull << shift) - 1ull)) != 0ull;
    return UP && rest ? whole + 1ull : whole;
}

// exp((x - top) / T) in 2^-42, rounded; (ch, cl): log2(e) / T.  The exponent t = n / 64 + r in two
// floats; 2^-r = 1 - p + p^2 / 2 - p^3 / 6 + p^4 / 24 with p = r ln 2 <= 0.0055 (the next term is
// 2^-44), p in two floats too, and 2^(-n / 64) from a table and a shift.
__device__ __forceinline__ uint64_t ls_weight(float x, float top, float ch, float cl, const uint64_t* table) {
    const float d = top - x, bb = d - top, dl = (top - (d - bb)) - (x + bb);   // top - x = d + dl
    const float t = d * ch;
    if (!(t < (float)(LS_FRAC + 1))) return 0ull;
    const float tl = fmaf(d, cl, fmaf(dl, ch, fmaf(d, ch, -t)));
    // (rounded by adding 1.5 * 2^23: the conversions' unit is slow)
    constexpr float WHOLE = 12582912.f;
    const float near = fmaf(t, 64.f, WHOLE), r = fmaf(near - WHOLE, -0.015625f, t);
    const int n = __float_as_int(near) - __float_as_int(WHOLE);
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

// The cluster's barrier in its two halves and whole.  Its aligned form wants the warp's lanes together,
// and behind stores by some of them, or a loop over a list, nothing else brings them there.
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ void remote_st_u64(uint64_t* p, uint32_t rank, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_rank(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t remote_add_u32(uint32_t* p, uint32_t rank, uint32_t v) {
    uint32_t r;
    asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(map_rank(p, rank)), "r"(v) : "memory");
    return r;
}
__device__ __forceinline__ uint64_t remote_ld_u64(const unsigned long long* p, uint32_t rank) {
    uint64_t r;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(r) : "r"(map_rank(p, rank)) : "memory");
    return r;
}
__device__ __forceinline__ uint32_t remote_ld_u32(const uint32_t* p, uint32_t rank) {
    uint32_t r;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(r) : "r"(map_rank(p, rank)) : "memory");
    return r;
}

template <typename E>
__global__ void __launch_bounds__(LS_THREADS, 2) logits_sample_kernel(const __grid_constant__ LsParams p) {
    extern __shared__ __align__(16) uint8_t ls_smem[];
    E* xs = reinterpret_cast<E*>(ls_smem);                 // the slice
    __shared__ __align__(16) uint32_t hist[LS_BINS];       // the slice's counts (see masses: words of 8 bytes too),
    __shared__ __align__(16) uint32_t tot[LS_BINS];        // the row's
    __shared__ uint64_t lists[2 * LS_LIST];
    uint64_t *list = lists, *weight = lists + LS_LIST;     // first CTA: entries of one bin
    __shared__ uint64_t table[64];
    __shared__ uint64_t part[2][LS_WARPS];                 // per warp
    __shared__ uint64_t peer[2][2][LS_CLUSTER_MAX];        // per CTA, two exchanges in turn
    __shared__ uint32_t held_n, kept_n;
    __shared__ uint64_t result[3];                         // of the first CTA, of a bisection
    __shared__ uint64_t plan[2], before_pick, upto;        // bins that the first CTA looks into
    uint16_t* near_i = reinterpret_cast<uint16_t*>(ls_smem + (size_t)p.slice * sizeof(E));   // places of the near entries
    static_assert(LS_FEW <= 2 * LS_LIST, "what is kept of few entries in the lists' room");
    __shared__ uint32_t list_n[4];
    __shared__ uint32_t pick[2];                           // a bin, entries before it
    __shared__ float fpart[LS_WARPS], est;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = p.ctas, me = (int)(blockIdx.x % C);
    const int64_t row = blockIdx.x / C;
    const int b = (int)(row / p.N), node = (int)(row % p.N);
    const int x0 = me * p.slice, n = max(0, min(p.slice, p.V - x0));
    const int chunk = p.slice / LS_WARPS, w0 = warp * chunk;   // a warp's entries
    if (tid < 64) table[tid] = LS_TABLE[tid];
    if (tid < 4) list_n[tid] = 0u;
    if (tid < 3) result[tid] = ~0ull;
    if (tid == 0) held_n = kept_n = 0u;
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
    if (p.defer && tid == 0) {
        // to L2: this slice of the row that a cluster of the next wave takes
        const int64_t next = row + p.ahead;
        const uintptr_t a = reinterpret_cast<uintptr_t>(static_cast<const E*>(p.logits) + next * p.V + x0);
        const uintptr_t lo = (a + 15) & ~(uintptr_t)15, hi = (a + (uintptr_t)n * sizeof(E)) & ~(uintptr_t)15;
        if (next < p.rows && lo < hi) bulk_prefetch_l2(reinterpret_cast<const void*>(lo), (uint32_t)(hi - lo));
    }
    __syncthreads();
    cluster_arrive();                                          // this CTA has started, its counters are zero

    // ---- the slice, and its maximum (a NaN wins)
    // (read as numbers plus 0: -0 is 0)
    auto at1 = [&](int i) -> float { return (float)xs[i] + 0.f; };
    auto wide = [](const uint2& h) -> float4 {
        return make_float4(__uint_as_float(h.x << 16) + 0.f, __uint_as_float(h.x & 0xffff0000u) + 0.f,
                           __uint_as_float(h.y << 16) + 0.f, __uint_as_float(h.y & 0xffff0000u) + 0.f);
    };
    auto at4 = [&](int i) -> float4 {                          // i a multiple of 4
        if constexpr (sizeof(E) == 4) {
            const float4 v = *reinterpret_cast<const float4*>(xs + i);
            return make_float4(v.x + 0.f, v.y + 0.f, v.z + 0.f, v.w + 0.f);
        } else {
            return wide(*reinterpret_cast<const uint2*>(xs + i));
        }
    };
    float mx = -INFINITY;
    auto take = [&](float x) { asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(mx), "f"(x)); };
    {
        const E* src = static_cast<const E*>(p.logits) + row * p.V + x0;
        if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
            // sixteen bytes at a time, the end by entries
            constexpr int U = 4, VE = 16 / (int)sizeof(E);
            const int full = n & ~(VE - 1);
            for (int i = tid * VE; i < full; i += LS_THREADS * VE * U) {
                uint4 v[U];
#pragma unroll
                for (int y = 0; y < U; ++y)
                    if (i + y * LS_THREADS * VE < full) v[y] = __ldcs(reinterpret_cast<const uint4*>(src + i + y * LS_THREADS * VE));
#pragma unroll
                for (int y = 0; y < U; ++y)
                    if (i + y * LS_THREADS * VE < full) {
                        *reinterpret_cast<uint4*>(xs + i + y * LS_THREADS * VE) = v[y];
                        if constexpr (sizeof(E) == 4) {
                            take(__uint_as_float(v[y].x)), take(__uint_as_float(v[y].y)), take(__uint_as_float(v[y].z)), take(__uint_as_float(v[y].w));
                        } else {
                            const float4 a = wide(make_uint2(v[y].x, v[y].y)), b2 = wide(make_uint2(v[y].z, v[y].w));
                            take(a.x), take(a.y), take(a.z), take(a.w), take(b2.x), take(b2.y), take(b2.z), take(b2.w);
                        }
                    }
            }
            for (int i = full + tid; i < p.slice; i += LS_THREADS) {
                const E x = i < n ? src[i] : (E)(-INFINITY);
                xs[i] = x;
                take((float)x);
            }
        } else {
            constexpr int U = 8;
            for (int i = tid; i < p.slice; i += LS_THREADS * U) {
                E v[U];
#pragma unroll
                for (int y = 0; y < U; ++y) v[y] = i + y * LS_THREADS < n ? src[i + y * LS_THREADS] : (E)(-INFINITY);
#pragma unroll
                for (int y = 0; y < U; ++y)
                    if (i + y * LS_THREADS < p.slice) {
                        xs[i + y * LS_THREADS] = v[y];
                        take((float)v[y]);
                    }
            }
        }
    }
    // ---- exchanges over the cluster: what a CTA's threads pass, reduced
    int turn = 0;
    auto exchange = [&](uint64_t v0, uint64_t v1) {            // per CTA values into every CTA's peer[turn]
        if (tid < C) {
            remote_st_u64(&peer[turn][0][me], tid, v0);
            remote_st_u64(&peer[turn][1][me], tid, v1);
        }
        cluster_sync();
        turn ^= 1;                                             // (read peer[turn ^ 1])
    };
    // Sums over the CTA: true in the first warp, which has them (and passes them on); part is
    // free again after the next barrier.
    auto block_sum = [&](uint64_t (&v)[2], int count) {
        for (int c = 0; c < count; ++c) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v[c] += __shfl_xor_sync(0xffffffffu, v[c], o);
            if (lane == 0) part[c][warp] = v[c];
        }
        __syncthreads();
        if (warp == 0)
            for (int c = 0; c < count; ++c) {
                v[c] = lane < LS_WARPS ? part[c][lane] : 0ull;
#pragma unroll
                for (int o = LS_WARPS / 2; o > 0; o >>= 1) v[c] += __shfl_xor_sync(0xffffffffu, v[c], o);
            }
    };
    auto cluster_sum = [&](uint64_t (&v)[2], int count) {
        block_sum(v, count);
        exchange(v[0], v[1]);
        for (int c = 0; c < count; ++c) {
            v[c] = 0ull;
            for (int r = 0; r < C; ++r) v[c] += peer[turn ^ 1][c][r];
        }
    };
    // f(entry, its place in the slice) over the warp's entries, four at a time
    auto entries = [&](auto f) {
        for (int i = lane * 4; i < chunk; i += 128) {
            const float4 v = at4(w0 + i);
            f(v.x, w0 + i);
            f(v.y, w0 + i + 1);
            f(v.z, w0 + i + 2);
            f(v.w, w0 + i + 3);
        }
    };
    // f(entry, its place) where mark(entry) holds: marks of 32 entries of a thread at a time
    auto marked = [&](auto mark, auto f) {
#pragma unroll 1
        for (int g = 0; g < chunk; g += 1024) {
            uint32_t m = 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (g + e * 128 < chunk) {
                    const float4 v = at4(w0 + g + e * 128 + lane * 4);
                    m |= (mark(v.x) ? 1u : 0u) << (4 * e) | (mark(v.y) ? 2u : 0u) << (4 * e) | (mark(v.z) ? 4u : 0u) << (4 * e) |
                         (mark(v.w) ? 8u : 0u) << (4 * e);
                }
#pragma unroll 1
            while (__any_sync(0xffffffffu, m != 0u)) {
                if (m != 0u) {
                    const int e = __ffs(m) - 1, i = w0 + g + (e >> 2) * 128 + lane * 4 + (e & 3);
                    m &= m - 1u;
                    f(at1(i), i);
                }
                __syncwarp();
            }
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
        cluster_wait();
        exchange(__float_as_uint(mx), 0ull);
        top = __uint_as_float((uint32_t)peer[turn ^ 1][0][0]);
        for (int r = 1; r < C; ++r) {
            const float y = __uint_as_float((uint32_t)peer[turn ^ 1][0][r]);
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(top) : "f"(top), "f"(y));
        }
    }
    top += 0.f;
    if (!(fabsf(top) <= FLT_MAX)) {                            // NaN, infinity, or nothing above -infinity
        err = TV_ERR_BAD_VALUES;
        refuse();
        cluster_sync();                                 // (no CTA leaves while others write to it)
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
        exchange(best, 0ull);
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
    // log2(e) / T in two floats (64-bit arithmetic is slow here)
    constexpr float L2EH = 1.44269502162933349609f, L2EL = 1.92596299112661746887e-8f;
    const float ch = L2EH / T, cl = (fmaf(-ch, T, L2EH) + L2EL) / T;
    const float bin_scale = fminf(LS_BIN / T, 1e38f);
    auto depth = [&](float x) -> float { return fminf((top - x) * bin_scale, (float)(LS_BINS - 1)); };
    auto bin_of = [&](float x) -> int { return (int)depth(x); };
    auto weigh = [&](float x) -> uint64_t { return ls_weight(x, top, ch, cl, table); };
    const bool use_k = k > 0 && k < p.V, use_p = top_p < 1.f;
    uint64_t cut = ~0ull;                                      // entries up to this key are kept
    const uint64_t least = (uint64_t)ceilf(min_p * (float)(1ull << LS_FRAC));
    uint64_t all = 0ull;                                       // the sum of what is kept
    constexpr int PER = LS_BINS / LS_THREADS;                  // bins per thread
    uint32_t c[PER], counted_before = 0u;
    // The row's counts of the bins from .. to - 1 into tot, those below `to` into c; returns their sum.
    // (Between two barriers: the first after every CTA's hist is complete.)
    auto sum_bins = [&](int from, int to) {
        for (int i = me * LS_THREADS + tid; i < LS_BINS; i += C * LS_THREADS)
            if (i >= from && i < to) {
                uint32_t sum = 0u, got[LS_CLUSTER_MAX];
#pragma unroll
                for (int r = 0; r < LS_CLUSTER_MAX; ++r) got[r] = r < C ? remote_ld_u32(&hist[i], r) : 0u;
#pragma unroll
                for (int r = 0; r < LS_CLUSTER_MAX; ++r) sum += got[r];
                for (int r = 0; r < C; ++r) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(&tot[i], r)), "r"(sum) : "memory");
            }
        cluster_sync();
        uint32_t sum = 0u;
#pragma unroll
        for (int e = 0; e < PER; ++e) sum += c[e] = tid * PER + e < to ? tot[tid * PER + e] : 0u;
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) part[0][warp] = incl;
        __syncthreads();
        counted_before = incl - sum;
        uint32_t in_all = 0u;
        for (int w = 0; w < LS_WARPS; ++w) {
            if (w < warp) counted_before += (uint32_t)part[0][w];
            in_all += (uint32_t)part[0][w];
        }
        if (to == LS_BINS - 1 && tid == LS_THREADS - 1) c[PER - 1] = tot[LS_BINS - 1] = (uint32_t)p.V - in_all;
        __syncthreads();
        return in_all;
    };
    // The bin that holds the k-th entry, and the entries before it.
    auto bin_of_rank = [&](uint32_t rank) {
        uint32_t at = counted_before;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            if (at < rank && rank <= at + c[e]) {
                pick[0] = tid * PER + e;
                pick[1] = at;
            }
            at += c[e];
        }
        __syncthreads();
    };
    // The bin in which the mass reaches goal by the counts (up to k_bin, of which k_rank entries count), or
    // LS_BINS; est: the mass before it, by the counts (of all bins, where it is none; every CTA has to
    // come to the same bin, or some would leave while others still write to them).  (The best entry weighs 1, not what its bin's
    // middle does.)
    auto bin_of_mass = [&](float goal, int k_bin, uint32_t k_rank) -> int {
        float m[PER], ms = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int bin = tid * PER + e;
            const uint32_t in = use_k && bin >= k_bin ? (bin == k_bin ? k_rank : 0u) : c[e];
            m[e] = (float)in * ex2_approx(-1.44269504f * ((float)bin + 0.5f) / LS_BIN);
            if (bin == 0) m[e] += 0.5f / LS_BIN;
            ms += m[e];
        }
        float mi = ms;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, mi, o);
            if (lane >= o) mi += y;
        }
        if (lane == 31) fpart[warp] = mi;
        if (tid == 0) pick[0] = (uint32_t)LS_BINS;
        __syncthreads();
        float at = mi - ms;
        for (int w = 0; w < warp; ++w) at += fpart[w];
        const float begin = at;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            if (at < goal && goal <= at + m[e]) atomicMin(&pick[0], (uint32_t)(tid * PER + e));
            at += m[e];
        }
        __syncthreads();
        const int found = (int)pick[0];
        at = begin;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            if (tid * PER + e == found) est = at;
            at += m[e];
        }
        if (found >= LS_BINS && tid == LS_THREADS - 1) est = at;
        __syncthreads();
        return found;
    };
    // The next bin to try when the exact mass before this one is not what the counts say.
    auto next_bin = [&](int bin, float need, float exact_before, bool below, int k_bin, uint32_t k_rank) -> int {
        const int next = bin_of_mass(need + (est - exact_before), k_bin, k_rank);
        return below ? min(next, bin - 1) : (next >= LS_BINS ? bin + 1 : max(next, bin + 1));
    };
    auto value_of = [](uint64_t key) -> float {
        const uint32_t bits = ~(uint32_t)(key >> 32);
        return __uint_as_float((bits & 0x80000000u) ? bits & 0x7fffffffu : ~bits);
    };
    auto to_list = [&](int which, uint64_t key) {              // of the first CTA
        const uint32_t at = remote_add_u32(&list_n[which], 0, 1u);
        if (at < LS_LIST) remote_st_u64(&list[at], 0, key);
    };
    // By the first CTA, for all: the key with rank `rank` in the list, or (mass) of the last one that
    // begins below need, `base` being what comes before the list.
    auto rank_list = [&](int which, int into, bool mass, uint64_t rank, uint64_t base, uint64_t need) {
        const int m = min((int)list_n[which], LS_LIST);
        if (mass)
            for (int e = tid; e < m; e += LS_THREADS) weight[e] = weigh(value_of(list[e]));
        __syncthreads();
        for (int e = tid; e < m; e += LS_THREADS) {
            const uint64_t key = list[e];
            uint64_t before = mass ? base : 0ull;
#pragma unroll 4
            for (int f = 0; f < m; ++f) before += list[f] < key ? (mass ? weight[f] : 1ull) : 0ull;
            // (mass: the last one that begins below; the next one does not, or there is none)
            if (mass ? before < need && before + weight[e] >= need : before == rank)
                for (int r = 0; r < C; ++r) remote_st_u64(&result[into], r, key);
        }
    };

    // ---- The near entries, where they hold all that may be kept: their places in the slice in a list.
    bool deferred = false;
    // Says what is left to do: nothing, the draw, or all of it.
    enum { DONE, DRAW, ALL };
    auto near_path = [&]() -> int {
        if (!(use_k || use_p || min_p > 0.f)) return ALL;
        // The entries within each reach, a byte for each (a thread has at most 96 entries).  For top-p of the
        // whole row also the weights of the entries between the last two and beyond, in 2^-34 and 2^-38
        // of the largest: below 2^23 of them each, so rounded by adding 2^23.  (The exponent t < 32 is off by
        // 2^-24 t for d and three roundings of 2^-20 at most, 3.3e-6 of the weight with ln 2; ex2 by 2^-22;
        // and half a step, of the weights between, 2^-13.3 to 2^-15.3, 2^-19.7: below 2^-18 in all, beyond
        // with 2^-39 for the step.)
        const bool weights = use_p && !use_k;
        uint32_t between = 0u, beyond = 0u, many = 0u;
        if (weights) {
#pragma unroll 1
            for (int g = 0; g < chunk; g += 1024)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (g + e * 128 < chunk) {
                        const float4 q = at4(w0 + g + e * 128 + lane * 4);
                        const float y[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const float d = top - y[z], v = d * bin_scale;
                            const bool is_near = v < (float)LS_NEAR, is_nearer = v < (float)LS_NEARER;
                            many += (is_near ? 1u << 24 : 0u) + (is_nearer ? 1u << 16 : 0u);
                            if (!is_nearer) {
                                const float t = fmaf(d, cl, d * ch), s = is_near ? (float)(LS_FRAC - 8) : (float)(LS_FRAC - 4);
                                const uint32_t w = __float_as_uint(ex2_approx(fmaxf(s - t, -126.f)) + 8388608.f) - __float_as_uint(8388608.f);
                                between += is_near ? w : 0u;
                                beyond += is_near ? 0u : w;
                            }
                        }
                    }
        } else {
            // (most entries are beyond the last: the others are marked and looked at by themselves)
            marked([&](float x) { return (top - x) * bin_scale < (float)LS_NEAR; },
                   [&](float x, int) {
                       const float t = (top - x) * bin_scale;
#pragma unroll
                       for (int j = 0; j < LS_REACHES; ++j) many += t < (float)ls_reach(j) ? 1u << (8 * j) : 0u;
                   });
        }
        // (a CTA has less than 2^16 entries)
        uint64_t v[2] = {(uint64_t)(many & 0xffu) | (uint64_t)(many & 0xff00u) << 8 | (uint64_t)(many & 0xff0000u) << 16 |
                             (uint64_t)(many >> 24) << 48, 0ull};
        block_sum(v, 1);
        exchange(v[0], 0ull);
        // The reach: the smallest with which the near entries hold all that may be kept, if there is room for
        // them; for top-p of the whole row the largest with room.
        int reach = 0;
        bool few = true, enough = false;
        for (int j = weights ? 2 : 0; j < LS_REACHES; ++j) {
            uint32_t sum = 0u;
            bool room = true, small = true;
            for (int r = 0; r < C; ++r) {
                const int a = (int)(peer[turn ^ 1][0][r] >> (16 * j)) & 0xffff;
                // (a dump's header and pairs lie in the slice's own part of the distribution)
                room = room && a <= p.heavy && (!p.defer || a == 0 || LS_HEAD + 2 * a <= p.cells(r));
                small = small && a <= LS_FEW;
                sum += (uint32_t)a;
            }
            if (!room) break;
            reach = ls_reach(j);
            few = small;
            enough = weights || (use_k ? sum >= (uint32_t)k : min_p >= 1.01f * ex2_approx((float)reach * (-1.4427f / LS_BIN)));
            if (enough && !weights) break;
        }
        if (!enough) return ALL;
        const bool fits = reach == LS_NEAR;
#pragma unroll 1
        for (int g = 0; g < chunk; g += 1024) {
            uint32_t marks = 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (g + e * 128 < chunk) {
                    const float4 q = at4(w0 + g + e * 128 + lane * 4);
                    marks |= ((top - q.x) * bin_scale < (float)reach ? 1u : 0u) << (4 * e) | ((top - q.y) * bin_scale < (float)reach ? 2u : 0u) << (4 * e) |
                             ((top - q.z) * bin_scale < (float)reach ? 4u : 0u) << (4 * e) | ((top - q.w) * bin_scale < (float)reach ? 8u : 0u) << (4 * e);
                }
            // places for the warp's entries by one atomic
            const uint32_t own = (uint32_t)__popc(marks);
            uint32_t incl = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            uint32_t to = 0u;
            if (lane == 31) to = atomicAdd(&held_n, incl);
            to = __shfl_sync(0xffffffffu, to, 31) + incl - own;
            for (; marks != 0u; marks &= marks - 1u, ++to) {
                const int e = __ffs(marks) - 1;
                near_i[to] = (uint16_t)(w0 + g + (e >> 2) * 128 + lane * 4 + (e & 3));
            }
        }
        __syncthreads();
        const uint32_t held = held_n;
        auto masses = [](uint32_t* counts) { return reinterpret_cast<unsigned long long*>(counts + LS_NEAR); };
        auto each_near = [&](auto f) {                         // f(entry, its place in the slice)
#pragma unroll 1
            for (int e = tid; e < (int)held; e += LS_THREADS) f(at1(near_i[e]), (int)near_i[e]);
        };
        v[0] = 0ull;
        v[1] = ((uint64_t)beyond << 4) + (fits ? 0ull : (uint64_t)between << 8);
        each_near([&](float x, int) {
            const uint64_t w = weigh(x);
            v[0] += w;
            if (!p.defer && (use_k || use_p)) {
                const int bin = bin_of(x);
                atomicAdd(&hist[bin], 1u);
                atomicAdd(&masses(hist)[bin], (unsigned long long)w);
            }
        });
        // the weights' sums, of these and of the others
        block_sum(v, 2);
        exchange(v[0], v[1]);
        uint64_t mass_near = 0ull, mass_all = 0ull;
        for (int r = 0; r < C; ++r) {
            mass_near += peer[turn ^ 1][0][r];
            mass_all += peer[turn ^ 1][1][r];
        }
        mass_all += mass_near;
        // (not where the near entries do not hold all that may be kept)
        if (weights && ls_part<true>(top_p, mass_all) > mass_near) return ALL;
        if (p.defer) {
            // the second kernel takes it from here (the first slice has a header: in rows shorter than one there is
            // no room for the largest entry)
            uint32_t* dump = reinterpret_cast<uint32_t*>(out);
            const uint64_t others = mass_all - mass_near;
            if (tid == 0 && p.headed(me)) {
                dump[0] = held;
                if (me == 0) {
                    dump[1] = (uint32_t)others;
                    dump[2] = (uint32_t)(others >> 32);
                    dump[3] = __float_as_uint(top);
                    p.status[row] = LS_PENDING;
                }
            }
            for (int e = tid; e < (int)held; e += LS_THREADS) {
                dump[LS_HEAD + 2 * e] = __float_as_uint(at1(near_i[e]));
                dump[LS_HEAD + 2 * e + 1] = (uint32_t)place(near_i[e]);
            }
            const int from = p.headed(me) ? LS_HEAD + 2 * (int)held : 0;
            if ((reinterpret_cast<uintptr_t>(out) & 15) == 0) {
                const int full = min(n, (from + 3) & ~3);
                if (from + tid < full) out[from + tid] = 0.f;
                for (int i = full + tid * 4; i + 4 <= n; i += LS_THREADS * 4) __stcs(reinterpret_cast<float4*>(out + i), make_float4(0.f, 0.f, 0.f, 0.f));
                const int tail = max(full, n & ~3);
                if (tail + tid < n) out[tail + tid] = 0.f;
            } else {
                for (int i = from + tid; i < n; i += LS_THREADS) out[i] = 0.f;
            }
            deferred = true;
            return DONE;
        }
        if (use_k || use_p) {
            // The first CTA sums the counts and masses, says which bin it needs, ranks that bin's entries,
            // and (top-p below the bin that top-k cuts) another one's.
            uint32_t c0 = 0u, c1 = 0u, c_before = 0u;
            uint64_t m0 = 0ull, m1 = 0ull, m_before = 0ull;
            auto pick_mass = [&](uint64_t goal) {              // before <= goal < up to it
                if (m_before <= goal && goal < m_before + m0) {
                    pick[0] = 2 * tid;
                    before_pick = m_before;
                } else if (m_before + m0 <= goal && goal < m_before + m0 + m1) {
                    pick[0] = 2 * tid + 1;
                    before_pick = m_before + m0;
                }
                __syncthreads();
            };
            // the key with rank `rank` among the list's, or (mass) of the last one up to `limit` that begins below
            // need; upto: the list's mass up to it
            auto rank_of = [&](int m, bool by_mass, uint32_t rank, uint64_t base, uint64_t need, uint64_t limit) {
                for (int e = tid; e < m; e += LS_THREADS) {
                    const uint64_t k0 = list[e], w = weight[e];
                    uint32_t nb = 0u;
                    uint64_t before = 0ull;
#pragma unroll 4
                    for (int f = 0; f < m; ++f)
                        if (list[f] < k0) {
                            ++nb;
                            before += weight[f];
                        }
                    if (by_mass ? k0 <= limit && base + before < need && base + before + w >= need : nb == rank) {
                        result[2] = k0;
                        upto = before + w;
                    }
                }
                __syncthreads();
            };
            auto weights_of_list = [&](int which) -> int {
                const int m = (int)list_n[which];
                for (int e = tid; e < m; e += LS_THREADS) weight[e] = weigh(value_of(list[e]));
                __syncthreads();
                return m;
            };
            uint32_t k_rank = 0u;
            uint64_t base = 0ull;
            if (me == 0) {
                for (int i = tid; i < reach; i += LS_THREADS) {
                    uint32_t got[LS_CLUSTER_MAX], sum = 0u;
                    uint64_t more[LS_CLUSTER_MAX], mass = 0ull;
#pragma unroll
                    for (int r = 0; r < LS_CLUSTER_MAX; ++r) {
                        got[r] = r < C ? remote_ld_u32(&hist[i], r) : 0u;
                        more[r] = r < C ? remote_ld_u64(&masses(hist)[i], r) : 0ull;
                    }
#pragma unroll
                    for (int r = 0; r < LS_CLUSTER_MAX; ++r) {
                        sum += got[r];
                        mass += more[r];
                    }
                    tot[i] = sum;
                    masses(tot)[i] = mass;
                }
                __syncthreads();
                // two bins per thread
                if (2 * tid < reach) {
                    c0 = tot[2 * tid], c1 = tot[2 * tid + 1];
                    m0 = masses(tot)[2 * tid], m1 = masses(tot)[2 * tid + 1];
                }
                uint32_t ci = c0 + c1;
                uint64_t mi = m0 + m1;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, ci, o);
                    const uint64_t z = __shfl_up_sync(0xffffffffu, mi, o);
                    if (lane >= o) {
                        ci += y;
                        mi += z;
                    }
                }
                if (lane == 31) {
                    part[0][warp] = mi;
                    part[1][warp] = ci;
                }
                __syncthreads();
                c_before = ci - c0 - c1;
                m_before = mi - m0 - m1;
                for (int w = 0; w < warp; ++w) {
                    m_before += part[0][w];
                    c_before += (uint32_t)part[1][w];
                }
                if (use_k) {
                    const uint32_t want = (uint32_t)k;
                    if (c_before < want && want <= c_before + c0) {
                        pick[0] = 2 * tid;
                        pick[1] = want - c_before - 1u;
                        before_pick = m_before;
                    } else if (c_before + c0 < want && want <= c_before + c0 + c1) {
                        pick[0] = 2 * tid + 1;
                        pick[1] = want - c_before - c0 - 1u;
                        before_pick = m_before + m0;
                    }
                    __syncthreads();
                    k_rank = pick[1];
                } else {
                    pick_mass(ls_part<true>(top_p, mass_all) - 1ull);
                }
                base = before_pick;
                if (tid < C) remote_st_u64(&plan[0], tid, tot[pick[0]] > LS_LIST ? ~0ull : (uint64_t)pick[0]);
            }
            cluster_sync();
            if (plan[0] == ~0ull) return ALL;
            each_near([&](float x, int i) {
                if (bin_of(x) == (int)plan[0]) to_list(2, ls_key(x, place(i)));
            });
            cluster_sync();
            if (me == 0) {
                const int m = weights_of_list(2);
                uint64_t limit = ~0ull, then = ~0ull - 1ull;
                if (use_k) {
                    rank_of(m, false, k_rank, 0ull, 0ull, ~0ull);
                    limit = result[2];
                }
                if (use_p) {
                    const uint64_t need = ls_part<true>(top_p, use_k ? base + upto : mass_all);
                    __syncthreads();
                    if (!use_k || need > base) {
                        rank_of(m, true, 0u, base, need, limit);
                        limit = result[2];
                    } else {
                        pick_mass(need - 1ull);
                        then = tot[pick[0]] > LS_LIST ? ~0ull : (uint64_t)pick[0];
                        upto = need;
                    }
                }
                if (tid < C) {
                    remote_st_u64(&result[0], tid, limit);
                    remote_st_u64(&plan[1], tid, then);
                }
            }
            cluster_sync();
            cut = result[0];
            if (plan[1] == ~0ull) return ALL;
            if (plan[1] != ~0ull - 1ull) {
                each_near([&](float x, int i) {
                    if (bin_of(x) == (int)plan[1]) to_list(3, ls_key(x, place(i)));
                });
                cluster_sync();
                if (me == 0) {
                    const int m = weights_of_list(3);
                    const uint64_t need = upto;
                    __syncthreads();
                    rank_of(m, true, 0u, before_pick, need, ~0ull);
                    if (tid < C) remote_st_u64(&result[1], tid, result[2]);
                }
                cluster_sync();
                cut = min(cut, result[1]);
            }
        }
        if (!few) return DRAW;
        // ---- the mass that is left, and where the draw falls
        auto kept = [&](float x, int i) -> uint64_t {
            if (ls_key(x, place(i)) > cut) return 0ull;
            const uint64_t w = weigh(x);
            return w >= least ? w : 0ull;
        };
        v[0] = 0ull;
        each_near([&](float x, int i) { v[0] += kept(x, i); });
        block_sum(v, 1);
        exchange(v[0], 0ull);
        uint64_t before = 0ull;
        for (int r = 0; r < C; ++r) {
            if (r < me) before += peer[turn ^ 1][0][r];
            all += peer[turn ^ 1][0][r];
        }
        const uint64_t goal = ls_part<false>(u, all);
        if (goal >= before && goal < before + peer[turn ^ 1][0][me]) {
            // in this CTA: what it keeps in a list, (place in the slice, weight) in a word each
            each_near([&](float x, int i) {
                const uint64_t w = kept(x, i);
                if (w != 0ull) lists[atomicAdd(&kept_n, 1u)] = (uint64_t)i << 44 | w;
            });
            __syncthreads();
            const int m = (int)kept_n;
            for (int e = tid; e < m; e += LS_THREADS) {
                const uint64_t mine = lists[e];
                uint64_t at = before;
#pragma unroll 4
                for (int f = 0; f < m; ++f) {
                    const uint64_t other = lists[f];
                    at += (other >> 44) < (mine >> 44) ? other & ((1ull << 44) - 1ull) : 0ull;
                }
                if (goal >= at && goal < at + (mine & ((1ull << 44) - 1ull))) {
                    p.tokens[row] = place((int)(mine >> 44));
                    p.status[row] = TV_OK;
                }
            }
        }
        return DONE;
    };
    // The cut of a run of entries that no list holds, by bisection over the logits' bits: the
    // first key with which count entries, or a mass above before, are kept (`kept` entries count).
    auto bisect = [&](bool mass, uint64_t need, uint64_t limit) -> uint64_t {
        uint32_t lo = 0u, hi = 0xffffffffu;                    // largest bits from which on there are `need`
        uint64_t v[2];
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
        exchange(v[0], 0ull);
        uint64_t before = 0ull, all = 0ull;
        for (int r = 0; r < C; ++r) {
            if (r < me) before += peer[turn ^ 1][0][r];
            all += peer[turn ^ 1][0][r];
        }
        const uint64_t want = min(ties, all);
        if (want > before && want <= before + peer[turn ^ 1][0][me]) {
            // in this CTA: its warps in order
            if (lane == 0) part[0][warp] = mine;
            __syncthreads();
            for (int w2 = 0; w2 < warp; ++w2) before += part[0][w2];
            if (want > before && want <= before + mine)
                for (int i = 0; i < chunk; i += 32) {
                    const uint32_t m = __ballot_sync(0xffffffffu, ls_bits(at1(w0 + i + lane)) == lo && place(w0 + i + lane) < p.V);
                    const int here = __popc(m);
                    if (want <= before + here) {
                        const int at = __fns(m, 0, (int)(want - before));
                        if (lane < C) remote_st_u64(&result[2], lane, ls_key(x, place(w0 + i + at)));
                        break;
                    }
                    before += here;
                }
        }
        cluster_sync();
        const uint64_t found = result[2];
        cluster_sync();                                 // (read before it is written again)
        return found;
    };
    // The entries of a bin (up to `limit`) in the first CTA's list, ranked there.
    auto cut_in_bin = [&](int which, int bin, bool mass, uint64_t rank, uint64_t base, uint64_t need, uint64_t limit) -> uint64_t {
        const float lo_d = (float)bin, up_d = (float)(bin + 1);
        marked([&](float x) { const float d = depth(x); return d >= lo_d && d < up_d; }, [&](float x, int i) {
            if (place(i) >= p.V) return;
            const uint64_t key = ls_key(x, place(i));
            if (key <= limit) to_list(which, key);
        });
        cluster_sync();
        if (me == 0) rank_list(which, which, mass, rank, base, need);
        cluster_sync();
        return result[which];
    };
    // ---- Otherwise: over the whole row.
    auto whole_cut = [&]() {
    __syncthreads();
    for (int i = tid; i < LS_BINS; i += LS_THREADS) hist[i] = 0u;
    if (tid < 3) result[tid] = ~0ull;
    __syncthreads();
    cut = ~0ull;
    if (use_k || use_p) {
        // adds the bins from .. to - 1 of the slice to the row's counts
        auto count = [&](int from, int to) {
            cluster_sync();
            return sum_bins(from, to);
        };
        // the entries that weigh 2^-16 or more; in the same pass, without top-k, the sum of all weights
        uint64_t v[2] = {0ull, 0ull};
        uint32_t small = 0u;                                   // in 2^-42
        marked(
            [&](float x) -> bool {
                const float d = top - x;
                if (!use_k) {
                    const float t = fmaf(d, cl, d * ch);
                    if (t >= LS_SMALL) {
                        // below 2^23 steps: rounded by adding 2^23
                        small += __float_as_uint(ex2_approx(fmaxf((float)LS_FRAC - t, -126.f)) + 8388608.f) - __float_as_uint(8388608.f);
                        return false;
                    }
                    return true;
                }
                return d * bin_scale < (float)LS_NEAR;
            },
            [&](float x, int) {
                if (!use_k) v[0] += weigh(x);
                const int bin = bin_of(x);
                if (bin < LS_NEAR) atomicAdd(&hist[bin], 1u);
            });
        uint64_t mass_all = 0ull;
        if (!use_k) {
            v[0] += small;
            cluster_sum(v, 1);
            mass_all = v[0];
        }
        uint32_t counted = count(0, LS_NEAR);
        auto count_all = [&]() {
            // the others, where those do not reach
            entries([&](float x, int) {
                const int bin = bin_of(x);
                if (bin >= LS_NEAR && bin < LS_BINS - 1) atomicAdd(&hist[bin], 1u);
            });
            counted = count(LS_NEAR, LS_BINS - 1);
            counted = (uint32_t)p.V;
        };
        int k_bin = LS_BINS - 1;
        uint32_t k_rank = (uint32_t)p.V;
        if (use_k) {
            if (counted < (uint32_t)k) count_all();
            bin_of_rank((uint32_t)k);
            k_bin = (int)pick[0];
            k_rank = (uint32_t)k - pick[1];                     // entries of that bin that are kept
            cut = tot[k_bin] <= LS_LIST ? cut_in_bin(0, k_bin, false, k_rank - 1u, 0ull, 0ull, ~0ull)
                                        : bisect(false, (uint64_t)k, ~0ull);
        }
        if (use_p) {
            // ---- the mass that top-k left
            if (use_k) {
                const float up_d = (float)(k_bin + 1);
                v[0] = 0ull;
                marked([&](float x) { return depth(x) < up_d; }, [&](float x, int i) {
                    if (ls_key(x, place(i)) <= cut) v[0] += weigh(x);
                });
                cluster_sum(v, 1);
                mass_all = v[0];
            }
            // kept: what begins below top_p of the sum (an integer begins below it when it does below
            // the next one)
            const uint64_t need = ls_part<true>(top_p, mass_all);
            // ---- the bin where the mass reaches that, from the counts at first
            const float goal = (float)need * 2.2737368e-13f;   // 2^-42
            int guess = bin_of_mass(goal, k_bin, k_rank);
            if (guess >= LS_BINS && counted < (uint32_t)p.V && k_bin >= LS_NEAR) {
                // not reached: among the entries not yet counted
                count_all();
                guess = bin_of_mass(goal, k_bin, k_rank);
            }
            // (or by the estimate's error in the last one)
            if (guess >= LS_BINS) guess = min(k_bin, counted < (uint32_t)p.V ? LS_NEAR - 1 : LS_BINS - 1);
            int bin = guess, lo = 0, hi = k_bin;
            for (int tries = 0;; ++tries) {
                if (bin >= LS_NEAR && counted < (uint32_t)p.V) count_all();
                const float at_d = (float)bin, up_d = (float)(bin + 1);
                v[0] = v[1] = 0ull;
                marked([&](float x) { return depth(x) < up_d; }, [&](float x, int i) {
                    if (ls_key(x, place(i)) > cut) return;
                    const uint64_t w = weigh(x);
                    if (depth(x) < at_d) v[0] += w;
                    else v[1] += w;
                });
                cluster_sum(v, 2);
                if (v[0] < need && need <= v[0] + v[1]) break;
                if (need <= v[0]) hi = bin - 1;
                else lo = bin + 1;
                if (lo >= hi) {
                    bin = min(max(lo, 0), LS_BINS - 1);
                    if (tries > 2 * 11) break;
                } else if (tries < LS_TRIES) {
                    __syncthreads();
                    bin = min(max(next_bin(bin, goal, (float)v[0] * 2.2737368e-13f, need <= v[0], k_bin, k_rank), lo), hi);
                } else {
                    bin = (lo + hi) >> 1;
                }
            }
            cut = min(cut, tot[bin] <= LS_LIST ? cut_in_bin(1, bin, true, 0ull, v[0], need, cut) : bisect(true, need, cut));
        }
    }
    };
    auto draw = [&]() {
    // ---- the mass that is left, and where the draw falls
    auto kept = [&](float x, int i) -> uint64_t {
        if (ls_key(x, place(i)) > cut) return 0ull;
        const uint64_t w = weigh(x);
        return w >= least ? w : 0ull;
    };
    // (the logit of the cut, and the exponent of min_p with room for its rounding: what may be kept)
    const float cut_x = cut == ~0ull ? -INFINITY : value_of(cut);
    const float most_t = min_p > 0.f ? fminf((float)(LS_FRAC + 1), 0.001f - log2f(min_p)) : (float)(LS_FRAC + 1);
    auto maybe = [&](float x) -> bool { return x >= cut_x && (top - x) * ch < most_t; };
    uint64_t v[2] = {0ull, 0ull};
    if (cut == ~0ull && min_p == 0.f) entries([&](float x, int) { v[0] += weigh(x); });
    else marked(maybe, [&](float x, int i) { v[0] += kept(x, i); });
    uint64_t mine = v[0];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    block_sum(v, 1);
    exchange(v[0], 0ull);
    uint64_t before = 0ull;
    for (int r = 0; r < C; ++r) {
        if (r < me) before += peer[turn ^ 1][0][r];
        all += peer[turn ^ 1][0][r];
    }
    const uint64_t goal = ls_part<false>(u, all);              // the first entry whose sum exceeds it
    if (goal >= before && goal < before + peer[turn ^ 1][0][me]) {
        if (lane == 0) part[0][warp] = mine;
        __syncthreads();
        for (int w = 0; w < warp; ++w) before += part[0][w];
        if (goal >= before && goal < before + mine)
#pragma unroll 1
            for (int i = 0; i < chunk; i += 128) {
                // four entries of a lane, in order
                const float4 x = at4(w0 + i + lane * 4);
                const bool some = maybe(x.x) || maybe(x.y) || maybe(x.z) || maybe(x.w);
                if (!__any_sync(0xffffffffu, some)) continue;
                const float y[4] = {x.x, x.y, x.z, x.w};
                uint64_t w[4], sum = 0ull;
#pragma unroll
                for (int e = 0; e < 4; ++e) sum += w[e] = maybe(y[e]) ? kept(y[e], w0 + i + lane * 4 + e) : 0ull;
                uint64_t incl = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t z = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += z;
                }
                const uint32_t over = __ballot_sync(0xffffffffu, before + incl > goal);
                if (over != 0u) {
                    if (lane == __ffs(over) - 1) {
                        uint64_t at = before + incl - sum;
                        int e = 0;
                        while (e < 3 && at + w[e] <= goal) at += w[e++];
                        p.tokens[row] = place(w0 + i + lane * 4 + e);
                        p.status[row] = TV_OK;
                    }
                    break;
                }
                before += __shfl_sync(0xffffffffu, incl, 31);
            }
    }
    };
    const int left = near_path();
    if (left == ALL) whole_cut();
    if (left != DONE) draw();
    if (out && !deferred) {
        const float cut_x = cut == ~0ull ? -INFINITY : value_of(cut);
        // weights again, in float32: 2^-22 of each, with the exponent's rounding
        const float inv = 1.f / ((float)all * 2.2737368e-13f); // 2^-42
        auto prob = [&](float x, int i) -> float {
            if (!(x >= cut_x)) return 0.f;
            const float t = (x - top) * ch, w = ex2_approx(t);
            if (x == cut_x && ls_key(x, place(i)) > cut) return 0.f;
            // (near min_p the exact weight decides)
            if (min_p > 0.f && w < min_p * 1.001f && (w < min_p * 0.999f || weigh(x) < least)) return 0.f;
            return w * inv;
        };
        auto write = [&](auto f) {
            if ((reinterpret_cast<uintptr_t>(out) & 15) == 0) {
#pragma unroll 2
                for (int i = tid * 4; i < n; i += LS_THREADS * 4) {
                    const float4 x = at4(i);
                    const float4 y = make_float4(f(x.x, i), f(x.y, i + 1), f(x.z, i + 2), f(x.w, i + 3));
                    if (i + 4 <= n) {
                        __stcs(reinterpret_cast<float4*>(out + i), y);
                    } else {
                        out[i] = y.x;
                        if (i + 1 < n) out[i + 1] = y.y;
                        if (i + 2 < n) out[i + 2] = y.z;
                    }
                }
            } else {
                for (int i = tid; i < n; i += LS_THREADS) out[i] = f(at1(i), i);
            }
        };
        if (cut == ~0ull && min_p == 0.f) write([&](float x, int) -> float { return ex2_approx((x - top) * ch) * inv; });
        else write(prob);
    }
}

// The rows that the kernel above left: their near entries, by one CTA each.  Counts and exact masses by
// bins give the bins of the cuts, whose entries are ranked (or, if a bin has more than the list
// holds, bisected by key); then what is kept goes where it belongs, and the draw is found by
// buckets of the vocabulary.
constexpr int LR_THREADS = 512, LR_WARPS = LR_THREADS / 32;
static_assert(LS_HEAVY <= LS_ROW, "a CTA's entries at a time");
static_assert(LS_BUCKETS == 2 * LR_THREADS && LS_NEAR <= LS_BUCKETS, "two bins or buckets per thread");

__global__ void __launch_bounds__(LR_THREADS, 2) logits_sample_rows_kernel(const __grid_constant__ LsParams p) {
    extern __shared__ __align__(16) uint2 held[];           // [LS_ROW] (logit, index)
    __shared__ uint32_t count[LS_BUCKETS];                  // entries and mass per bin, then mass per bucket
    __shared__ uint32_t mass[3][LS_BUCKETS];                // (64-bit sums in shared memory are loops)
    __shared__ uint64_t list[LS_LIST], weight[LS_LIST];
    __shared__ uint64_t table[64];
    __shared__ uint64_t part[LR_WARPS];
    __shared__ uint32_t cpart[LR_WARPS];
    __shared__ uint64_t result, upto, others, before_pick;
    __shared__ uint32_t first[LS_CLUSTER_MAX + 1], list_n, pick, pick_rank;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x;
    const int b = (int)(row / p.N), node = (int)(row % p.N);
    if (tid < 64) table[tid] = LS_TABLE[tid];
    for (int i = tid; i < LS_BUCKETS; i += LR_THREADS) {
        count[i] = 0u;
        mass[0][i] = mass[1][i] = mass[2][i] = 0u;
    }
    // less than 2^17 weights of at most 2^42
    auto add = [&](int i, uint64_t w) {
        atomicAdd(&mass[0][i], (uint32_t)w & 0x7fffu);
        atomicAdd(&mass[1][i], (uint32_t)(w >> 15) & 0x7fffu);
        if (w >> 30) atomicAdd(&mass[2][i], (uint32_t)(w >> 30));
    };
    auto mass_of = [&](int i) -> uint64_t { return mass[0][i] + ((uint64_t)mass[1][i] << 15) + ((uint64_t)mass[2][i] << 30); };
    static_assert(LS_CLUSTER_MAX * LS_HEAVY < 1 << 17, "sums of the weights' parts in 32 bits");
    pdl_launch_dependents();
    pdl_wait();
    const int cnt = p.node_counts ? p.node_counts[b] : p.N;
    if ((cnt >= 1 && cnt <= p.N && node >= cnt) || p.status[row] != LS_PENDING) return;
    const float T = p.temp ? p.temp[b] : 1.f, top_p = p.top_p ? p.top_p[b] : 1.f;
    const float min_p = p.min_p ? p.min_p[b] : 0.f, u = p.uniform[row];
    const int k = p.top_k ? p.top_k[b] : 0;
    const bool use_k = k > 0 && k < p.V, use_p = top_p < 1.f;
    const uint64_t least = (uint64_t)ceilf(min_p * (float)(1ull << LS_FRAC));
    float* out = p.probs + row * p.V;
    const uint32_t* dump = reinterpret_cast<const uint32_t*>(out);
    if (warp == 0) {
        const uint32_t mine = lane < p.ctas && p.headed(lane) ? dump[(int64_t)lane * p.slice] : 0u;
        uint32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane <= LS_CLUSTER_MAX) first[lane] = incl - mine;
        if (lane == 0) others = (uint64_t)dump[1] | (uint64_t)dump[2] << 32;
    }
    const float top = __uint_as_float(dump[3]);
    __syncthreads();
    const int total = (int)first[p.ctas];
    // (wide: more entries than are held here, read again each time)
    auto body = [&](auto kind) {
    constexpr bool wide = decltype(kind)::value;
    auto entry = [&](int r, int e) -> uint2 {
        const uint32_t* src = dump + (int64_t)r * p.slice + LS_HEAD;
        return make_uint2(src[2 * e], src[2 * e + 1]);
    };
    // (the dump lies in the distribution)
    auto clear = [&](int r, int id, int count) {
        float* to = out + (int64_t)r * p.slice;
        const int words = p.headed(r) ? LS_HEAD + 2 * (int)(first[r + 1] - first[r]) : 0;
        for (int e = id; e < words; e += count) to[e] = 0.f;
    };
    if constexpr (!wide) {
        for (int r = warp; r < p.ctas; r += LR_WARPS) {
            const int m = (int)(first[r + 1] - first[r]);
#pragma unroll 4
            for (int e = lane; e < m; e += 32) held[first[r] + e] = entry(r, e);
        }
        __syncthreads();
        for (int r = warp; r < p.ctas; r += LR_WARPS) clear(r, lane, 32);
    }
    constexpr float L2EH = 1.44269502162933349609f, L2EL = 1.92596299112661746887e-8f;
    const float ch = L2EH / T, cl = (fmaf(-ch, T, L2EH) + L2EL) / T;
    const float bin_scale = fminf(LS_BIN / T, 1e38f);
    auto bin_of = [&](float x) -> int { return (int)fminf((top - x) * bin_scale, (float)(LS_BUCKETS - 1)); };
    auto weigh = [&](float x) -> uint64_t { return ls_weight(x, top, ch, cl, table); };
    // f(logit, index), by every thread of the CTA; a wide row's entries by the CTA that left them
    auto over = [&](int m, auto f) {
#pragma unroll 1
        for (int e = tid; e < m; e += LR_THREADS) f(__uint_as_float(held[e].x), (int)held[e].y);
    };
    auto each = [&](auto f) {
        if constexpr (!wide) {
            over(total, f);
        } else {
#pragma unroll 1
            for (int r = 0; r < p.ctas; ++r) {
                const int m = (int)(first[r + 1] - first[r]);
                __syncthreads();
#pragma unroll 4
                for (int e = tid; e < m; e += LR_THREADS) held[e] = entry(r, e);
                __syncthreads();
                over(m, f);
            }
        }
    };
    auto sum_of = [&](uint64_t v) -> uint64_t {             // over the CTA, for every thread
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        __syncthreads();
        if (lane == 0) part[warp] = v;
        __syncthreads();
        v = 0ull;
#pragma unroll
        for (int w = 0; w < LR_WARPS; ++w) v += part[w];
        return v;
    };
    // Entries and mass before this thread's two bins (or buckets); the mass of all.
    uint32_t c0 = 0u, c1 = 0u, c_before = 0u;
    uint64_t m0 = 0ull, m1 = 0ull, m_before = 0ull;
    auto scan = [&]() -> uint64_t {
        c0 = count[2 * tid], c1 = count[2 * tid + 1];
        m0 = mass_of(2 * tid), m1 = mass_of(2 * tid + 1);
        uint32_t ci = c0 + c1;
        uint64_t mi = m0 + m1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, ci, o);
            const uint64_t z = __shfl_up_sync(0xffffffffu, mi, o);
            if (lane >= o) {
                ci += y;
                mi += z;
            }
        }
        if (lane == 31) {
            part[warp] = mi;
            cpart[warp] = ci;
        }
        __syncthreads();
        c_before = ci - c0 - c1;
        m_before = mi - m0 - m1;
        uint64_t all = 0ull;
#pragma unroll
        for (int w = 0; w < LR_WARPS; ++w) {
            if (w < warp) {
                c_before += cpart[w];
                m_before += part[w];
            }
            all += part[w];
        }
        return all;
    };
    // The bin in which the mass passes `goal` (before <= goal < up to it): pick, and the mass before it.
    auto pick_mass = [&](uint64_t goal) {
        if (m_before <= goal && goal < m_before + m0) {
            pick = 2 * tid;
            before_pick = m_before;
        } else if (m_before + m0 <= goal && goal < m_before + m0 + m1) {
            pick = 2 * tid + 1;
            before_pick = m_before + m0;
        }
        __syncthreads();
    };
    // Buckets of the vocabulary, for what is kept, in the bins' room once those have been summed.
    int shift = 0;
    while ((p.V - 1) >> shift >= LS_BUCKETS) ++shift;
    auto to_bucket = [&](int i, uint64_t w) {
        if (w >= least) add(i >> shift, w);
    };
    auto clear_buckets = [&]() {
        __syncthreads();
        for (int i = tid; i < LS_BUCKETS; i += LR_THREADS) mass[0][i] = mass[1][i] = mass[2][i] = 0u;
        __syncthreads();
    };
    // (last: what comes before the bin, and what the cut keeps of it, to the buckets)
    // The key in a bin with rank `rank` there (by_rank), or of the last entry (up to `limit`) that begins
    // below need when `base` comes before the bin: result; upto: the bin's mass up to it.
    auto cut_in = [&](int bin, bool by_rank, uint32_t rank, uint64_t base, uint64_t need, uint64_t limit, bool last) {
        if (last) clear_buckets();
        if (count[bin] <= LS_LIST) {
            if (tid == 0) list_n = 0u;
            __syncthreads();
            each([&](float x, int i) {
                const int its = bin_of(x);
                if (its > bin || (!last && its != bin) || ls_key(x, i) > limit) return;
                const uint64_t w = weigh(x);
                if (its < bin) {
                    to_bucket(i, w);
                } else {
                    const uint32_t at = atomicAdd(&list_n, 1u);
                    list[at] = ls_key(x, i);
                    weight[at] = w;
                }
            });
            __syncthreads();
            const int m = (int)list_n;
            for (int e = tid; e < m; e += LR_THREADS) {
                const uint64_t key = list[e], w = weight[e];
                uint32_t n = 0u;
                uint64_t before = 0ull;
#pragma unroll 4
                for (int f = 0; f < m; ++f)
                    if (list[f] < key) {
                        ++n;
                        before += weight[f];
                    }
                if (by_rank ? n == rank : base + before < need && base + before + w >= need) {
                    result = key;
                    upto = before + w;
                }
            }
            __syncthreads();
            if (last)
                for (int e = tid; e < m; e += LR_THREADS)
                    if (list[e] <= result) to_bucket((int)(uint32_t)list[e], weight[e]);
            return;
        }
        // many equal entries: the smallest key up to which there are enough
        uint64_t lo = 0ull, hi = limit, got = 0ull;
        while (lo < hi) {
            const uint64_t mid = lo + ((hi - lo) >> 1);
            uint64_t v = 0ull;
            each([&](float x, int i) {
                if (bin_of(x) == bin && ls_key(x, i) <= mid) v += by_rank ? 1ull : weigh(x);
            });
            v = sum_of(v);
            if (by_rank ? v > rank : base + v >= need) hi = mid;
            else lo = mid + 1ull;
        }
        each([&](float x, int i) {
            if (bin_of(x) == bin && ls_key(x, i) <= hi) got += weigh(x);
        });
        got = sum_of(got);
        if (tid == 0) {
            result = hi;
            upto = got;
        }
        __syncthreads();
        if (last)
            each([&](float x, int i) {
                if (ls_key(x, i) <= hi) to_bucket(i, weigh(x));
            });
    };
    uint64_t cut = ~0ull;
    if (use_k || use_p) {
        each([&](float x, int) {
            const int bin = bin_of(x);
            atomicAdd(&count[bin], 1u);
            add(bin, weigh(x));
        });
        __syncthreads();
        uint64_t left = scan() + others;                    // the mass that top-k leaves
        int k_bin = LS_BUCKETS;
        uint64_t k_before = 0ull;
        if (use_k) {
            const uint32_t want = (uint32_t)k;
            if (c_before < want && want <= c_before + c0) {
                pick = 2 * tid;
                pick_rank = want - c_before - 1u;
                before_pick = m_before;
            } else if (c_before + c0 < want && want <= c_before + c0 + c1) {
                pick = 2 * tid + 1;
                pick_rank = want - c_before - c0 - 1u;
                before_pick = m_before + m0;
            }
            __syncthreads();
            k_bin = (int)pick;
            k_before = before_pick;
            cut_in(k_bin, true, pick_rank, 0ull, 0ull, ~0ull, !use_p);
            cut = result;
            left = k_before + upto;
            __syncthreads();
        }
        if (use_p) {
            const uint64_t need = ls_part<true>(top_p, left);   // (at least 1: the best entry weighs 2^42)
            int bin = k_bin;
            uint64_t base = k_before;
            if (!use_k || need <= k_before) {
                pick_mass(need - 1ull);
                bin = (int)pick;
                base = before_pick;
            }
            cut_in(bin, false, 0u, base, need, cut, true);
            cut = min(cut, result);
        }
    }
    // ---- what is kept: its sum, by buckets of the vocabulary
    if (!(use_k || use_p)) {
        clear_buckets();
        each([&](float x, int i) { to_bucket(i, weigh(x)); });
    }
    __syncthreads();
    const uint64_t all = scan(), goal = ls_part<false>(u, all);
    if (tid == 0) list_n = 0u;
    pick_mass(goal);
    const uint32_t bucket = pick;
    // weights again, in float32, as in the kernel above
    const float inv = 1.f / ((float)all * 2.2737368e-13f);  // 2^-42
    auto give = [&](float x, int i) {
        if (ls_key(x, i) > cut) return;
        const float w = ex2_approx((x - top) * ch);
        if (min_p > 0.f && w < min_p * 1.001f && (w < min_p * 0.999f || weigh(x) < least)) return;
        out[i] = w * inv;
        if ((uint32_t)i >> shift == bucket) {
            const uint32_t at = atomicAdd(&list_n, 1u);     // (a bucket is no larger)
            list[at] = (uint64_t)i;
            weight[at] = weigh(x);
        }
    };
    if constexpr (!wide) {
        each(give);
    } else {
        // a CTA's entries, which lie where some of them go, at a time
        for (int r = 0; r < p.ctas; ++r) {
            const int n = (int)(first[r + 1] - first[r]);
            __syncthreads();
#pragma unroll 4
            for (int e = tid; e < n; e += LR_THREADS) held[e] = entry(r, e);
            __syncthreads();
            clear(r, tid, LR_THREADS);
            __syncthreads();
            over(n, give);
        }
    }
    __syncthreads();
    const int m = (int)list_n;
    for (int e = tid; e < m; e += LR_THREADS) {
        uint64_t at = before_pick;
        for (int f = 0; f < m; ++f) at += list[f] < list[e] ? weight[f] : 0ull;
        if (at <= goal && goal < at + weight[e]) {
            p.tokens[row] = (int)list[e];
            p.status[row] = TV_OK;
        }
    }
    };
    if (total > LS_ROW) body(std::true_type{});
    else body(std::false_type{});
}

template <typename E>
tv_status launch_sample(const LsParams& q, int64_t rows, cudaStream_t stream) {
    LsParams p = q;
    auto fn = logits_sample_kernel<E>;
    constexpr int SLICE = LS_SLICE_BYTES / (int)sizeof(E);
    const int fewest = (p.V + SLICE - 1) / SLICE;
    // few rows: more CTAs per row, while they have a few thousand entries each
    int C = std::min(fewest, LS_CLUSTER_MAX);
    while (C * 2 <= LS_CLUSTER_MAX && rows * C * 2 <= 2 * device_sm_count() && p.V > C * 2 * LS_STEP) C *= 2;
    p.ctas = C;
    p.slice = ((p.V + C - 1) / C + LS_STEP - 1) / LS_STEP * LS_STEP;
    if (p.slice > LS_SLICE_MAX) return TV_ERR_UNSUPPORTED;
    if (rows * C > 0x7fffffff) return TV_ERR_UNSUPPORTED;
    p.heavy = std::min(LS_HEAVY, (LS_SHARED - LS_STATIC - p.slice * (int)sizeof(E)) / 2);
    const size_t smem = (size_t)p.slice * sizeof(E) + (size_t)p.heavy * sizeof(uint16_t);
    static std::atomic<bool> set[64], set_rows[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TV_ERR_CUDA;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, LS_SHARED - LS_STATIC) != cudaSuccess ||
            cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
            cudaGetLastError();
            return TV_ERR_CUDA;
        }
        set[dev] = true;
    }
    // Several waves of clusters, each of which would go through its cuts' barriers with its row in shared
    // memory: the cuts are left to a second kernel, behind the dumps in the distributions.
    p.rows = rows;
    p.ahead = std::max(1, 2 * device_sm_count() / C);
    p.defer = p.probs != nullptr && rows * C > 4 * device_sm_count() && p.slice >= LS_STEP && p.V <= LS_LIST * LS_BUCKETS;
    if (p.defer && !set_rows[dev]) {
        if (cudaFuncSetAttribute(logits_sample_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, LS_ROW * (int)sizeof(uint2)) != cudaSuccess) {
            cudaGetLastError();
            return TV_ERR_CUDA;
        }
        set_rows[dev] = true;
    }
    LaunchCfg lc(dim3((unsigned)(rows * C)), dim3(LS_THREADS), smem, stream, (unsigned)C);
    if (cudaLaunchKernelEx(&lc.cfg, fn, p) != cudaSuccess) return TV_ERR_CUDA;
    if (!p.defer) return TV_OK;
    LaunchCfg lr(dim3((unsigned)rows), dim3(LR_THREADS), LS_ROW * sizeof(uint2), stream);
    return cudaLaunchKernelEx(&lr.cfg, logits_sample_rows_kernel, p) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
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
