// tree_logits_process: the target model's rows of a tree into the logits or
// probabilities that acceptance reads.
//
// Per entry: z = logit + bias; a token that the history or the node's own path
// holds is divided (or multiplied) by the repetition penalty; z -= frequency *
// n + presence * [n > 0]; a token that the grammar forbids becomes -infinity.
// Then z / temperature, or its softmax.
//
// Bound by memory: a row is read once and written once.  A row is cut into slices, one
// CTA each; for the softmax the slices of a row form a cluster, and the maxima and sums
// of their warps are exchanged through distributed shared memory.  The grid is as
// large as the GPU holds at once (two CTAs per SM: one loads or stores while the other
// waits for its cluster), and each group of CTAs takes a contiguous range of rows.
// A slice comes into shared memory by a bulk copy, the next row's while the present
// one is reduced and stored.
// A tree's rows share their sequence's counts and biases, and few tokens have any: when
// the sequence changes the slice's are gathered into a list, and per row only the list's
// entries are changed, in shared memory, one per thread or so, except the tree's own
// tokens (at most 63), whose threads add the path's.  After that an entry costs a read
// into a register, the grammar's bit, the maximum, one exponential and the store.
// The shared memory leaves some 20 KB of L1: a few spilled registers of 1,024 threads do
// not fit and come back from L2 in every row, so the row loop keeps its state in shared
// memory and spills nothing (832 rows of 128,256 float32 probabilities 256 -> 181 us,
// 5.0 TB/s, without history, biases and grammar 137; from bfloat16 199; logits instead of
// probabilities 165; 24 rows of 152,064 bfloat16 logits 12).  Histories and biases with more entries than the list holds (some
// 4,500 per slice) are gone through in every row (both dense: 271 us for the 832 rows).
#include <cuda_bf16.h>
#include <float.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "tv_device.cuh"
#include "tv_internal.h"
#include "tv_tc.cuh"

namespace tv {

namespace {

constexpr int LG_THREADS = 512;
constexpr int LG_NV_MAX = 8;                                // 4-entry vectors per thread
constexpr int LG_SLICE_MAX = LG_THREADS * 4 * LG_NV_MAX - 32;
constexpr int LG_CLUSTER_MAX = 16;
constexpr int LG_PLAIN_SLICE = LG_THREADS * 4 * 4 - 32;     // without a softmax: no cluster
constexpr int LG_SMEM = 103 * 1024;                         // two CTAs per SM
constexpr int LG_WARPS = LG_THREADS / 32;
constexpr float LG_LOG2E = 1.4426950408889634f;

struct LgParams {
    const void* logits;
    const int32_t* node_counts;
    const uint64_t* mask;
    const int32_t* tokens;
    const int32_t* counts;
    const float* bias;
    const uint32_t* grammar;
    const float *rep, *freq, *pres, *temp;
    float* out;
    int32_t* status;
    int N, V, words;
    int64_t rows;
    int groups;     // of CTAs, each with a range of rows
    int slices;     // CTAs per row (the cluster, for the softmax)
    int slice;      // entries per CTA, a multiple of 32
    int list_max;   // entries that the list of counts and biases holds
    bool unscaled;  // the temperature is left to row_softmax_kernel
    LateWait late;  // test-only
};

struct LgRow {
    float rep, inv_rep, freq, pres, inv_temp;
    int cnt, err;                               // nodes, status
};

// The repetition penalty of a token that the history or the path holds, less frequency *
// n + presence [n > 0].
__device__ __forceinline__ float lg_penalty(const LgRow& r, float z, int n) {
    z = z > 0.f ? z * r.inv_rep : z * r.rep;
    return n > 0 ? z - fmaf(r.freq, (float)n, r.pres) : z;
}
// A list entry's word: the entry, and above it 0 (not in the history), 1 (in the prompt
// only), n + 1, or LG_LONG (the count does not fit: read it again).
constexpr uint32_t LG_LONG = 0xffffu;
constexpr uint32_t LG_NODE = 0xffffu;   // the whole word (a slice has fewer entries): skip it
__device__ __forceinline__ uint32_t lg_word(int x, int c) {
    const uint32_t n = (uint32_t)c & 0x7fffffffu;
    return (uint32_t)x | (c == 0 ? 0u : (n + 1u < LG_LONG ? n + 1u : LG_LONG)) << 16;
}
__device__ __forceinline__ float lg_max(float a, float b) {  // NaN wins
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float lg_max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// After a wait ran out, by every thread: the rows from the one that waited to the last of the
// CTA's range take the value of a refused sequence, and their sequences TV_ERR_TIMEOUT.
// (Whole rows: no other slice of them is worth anything.)
__device__ __forceinline__ void lg_fail(const LgParams& p, int64_t row, float value) {
    const int64_t row_hi = p.rows * (blockIdx.x / p.slices + 1) / p.groups;
#pragma unroll 1
    for (; row < row_hi; ++row) {
        const int b = (int)(row / p.N), i = (int)(row % p.N);
        const int cnt = p.node_counts ? p.node_counts[b] : p.N;
        const bool counted = cnt >= 1 && cnt <= p.N;
        if (threadIdx.x == 0) p.status[b] = counted ? TV_ERR_TIMEOUT : TV_ERR_OUT_OF_RANGE;
        if (counted && i >= cnt) continue;
#pragma unroll 1
        for (int x = threadIdx.x; x < p.V; x += LG_THREADS) p.out[row * p.V + x] = value;
    }
}

template <typename E, bool PROBS, int NV>
__global__ void __launch_bounds__(LG_THREADS, 2) tree_logits_kernel(const __grid_constant__ LgParams p) {
    constexpr bool F32 = sizeof(E) == 4;
    constexpr int CAP = LG_THREADS * 4 * NV;             // positions of the slice buffer
    extern __shared__ __align__(128) uint8_t lg_smem[];
    float* zs = reinterpret_cast<float*>(lg_smem);       // [CAP] the slice, entry x at zs[x + shift]
    // the slice as it comes; bfloat16: the buffer's second half and 8 entries more, widened in
    // place through registers
    E* raw = reinterpret_cast<E*>(F32 ? lg_smem : lg_smem + CAP * 2);
    uint32_t* s_gram = reinterpret_cast<uint32_t*>(lg_smem + CAP * 4 + (F32 ? 0 : 16));  // [CAP / 32 + 2]
    uint2* list = reinterpret_cast<uint2*>(s_gram + CAP / 32 + 2);      // (word, bias)
    __shared__ int tok[64];
    // The sequence's state: in shared memory, since registers that hold it would be spilled, and
    // spilled ones do not stay in the little that is left of L1.
    __shared__ uint64_t masks[64], node_same[64];        // node c's path; the nodes with its token
    __shared__ int node_x[64], node_c[64];               // its entry in the slice (or -1), history,
    __shared__ float node_bias[64];                      // bias
    __shared__ LgRow r;
    __shared__ int list_n;
    __shared__ uint32_t nodes[CAP / 32];                 // entries that nodes' threads change
    // [row parity] (maximum, sum) of every warp of the cluster, and their barriers
    __shared__ __align__(16) float2 peer[2][PROBS ? LG_CLUSTER_MAX * LG_WARPS : 1];
    __shared__ __align__(8) uint64_t peer_bar[2];
    __shared__ __align__(8) uint64_t full;               // the slice has landed
    __shared__ int64_t late_row;                         // first row that a wait may have left wrong
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = (int)(blockIdx.x / p.slices), me = (int)(blockIdx.x % p.slices);
    const int64_t row_lo = p.rows * group / p.groups, row_hi = p.rows * (group + 1) / p.groups;
    const int x0 = me * p.slice, n = max(0, min(p.slice, p.V - x0));
    if (tid == 0) {
        mbar_init(&peer_bar[0], 1);
        mbar_init(&peer_bar[1], 1);
        mbar_init(&full, 1);
        fence_mbar_init();
        s_gram[0] = 0u;
        late_row = row_hi - 1;                           // (found out behind the last row)
    }
    if (PROBS && p.slices > 1) cluster_barrier_all();    // every slice's barriers are there
    else __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    // A slice of a row: the 16-byte pieces that lie inside by a bulk copy (issued by thread 0),
    // up to 7 entries at each end and a grammar word by each thread, a row ahead.
    auto ahead = [&](const void* lo, size_t bytes) {     // to L2: the 16-byte pieces inside
        const uintptr_t a = (reinterpret_cast<uintptr_t>(lo) + 15) & ~(uintptr_t)15;
        const uintptr_t z = (reinterpret_cast<uintptr_t>(lo) + bytes) & ~(uintptr_t)15;
        if (a < z) bulk_prefetch_l2(reinterpret_cast<const void*>(a), (uint32_t)(z - a));
    };
    // (of sequence b, or with same_b false of the one after it, whose counts and biases follow)
    auto fetch = [&](int64_t row, int b, bool same_b) {
        if (tid == 0 && !same_b) {
            const int64_t at = (int64_t)(b + 1) * p.V + x0;
            if (p.counts) ahead(p.counts + at, (size_t)n * 4);
            if (p.bias) ahead(p.bias + at, (size_t)n * 4);
        }
        const E* lo = static_cast<const E*>(p.logits) + row * p.V + x0;
        const uintptr_t a = reinterpret_cast<uintptr_t>(lo), al = (a + 15) & ~(uintptr_t)15;
        const uintptr_t ah = max(al, (a + (size_t)n * sizeof(E)) & ~(uintptr_t)15);
        const int head = (int)((al - a) / sizeof(E)), end = (int)((ah - a) / sizeof(E));   // entries [head, end) by the copy
        if (tid == 0) {
            const uint32_t bytes = (uint32_t)(ah - al);
            mbar_arrive_expect_tx_relaxed_one(&full, bytes);
            if (bytes > 0) bulk_load(raw + (a / sizeof(E)) % (16 / sizeof(E)) + head, reinterpret_cast<const void*>(al), bytes, &full, l2_policy_evict_first());
        }
        const int x = tid < head ? tid : end + tid - head;
        if (x < n && tid < 16) {
            E* to = raw + a / sizeof(E) % (16 / sizeof(E)) + x;
            if constexpr (F32) cp_async_4(to, lo + x);
            else *to = lo[x];
        }
        if (p.grammar && tid * 32 < n) cp_async_4(s_gram + 1 + tid, p.grammar + row * p.words + x0 / 32 + tid);
    };
    uint32_t phase = 0, got = 0;
    bool alive = !(p.late.warp >= 0 && (p.late.cta < 0 || p.late.cta == (int)blockIdx.x));   // (test-only)
    int b = (int)(row_lo / p.N), i = (int)(row_lo % p.N) - 1;
    if (row_lo < row_hi) fetch(row_lo, b, true);
#pragma unroll 1
    for (int64_t row = row_lo; row < row_hi; ++row) {
        if (++i == p.N) {
            i = 0;
            ++b;
        }
        float* out = p.out + row * p.V + x0;
        const int64_t at = (int64_t)b * p.V + x0;        // the slice in counts and bias
        if (i == 0 || row == row_lo) {
            // ---- the sequence: parameters, checks, the list of its counts and biases
            const int cnt = p.node_counts ? p.node_counts[b] : p.N;
            const float rep = p.rep ? p.rep[b] : 1.f, freq = p.freq ? p.freq[b] : 0.f;
            const float pres = p.pres ? p.pres[b] : 0.f, temp = p.temp ? p.temp[b] : 1.f;
            int err = (cnt >= 1 && cnt <= p.N) ? TV_OK : TV_ERR_OUT_OF_RANGE;
            const bool tokens = p.mask && err == TV_OK;
            // (1 / x overflows for the smallest positive x)
            if (err == TV_OK && !(isfinite(rep) && rep >= FLT_MIN && isfinite(temp) && temp >= FLT_MIN &&
                                  isfinite(freq) && isfinite(pres)))
                err = TV_ERR_BAD_VALUES;
            int t = 0;                                    // node tid's token, its count and bias
            if (tokens && tid < cnt) t = p.tokens[(int64_t)b * p.N + tid];
            const bool tok_ok = !tokens || tid == 0 || tid >= cnt || (t >= 0 && t < p.V);
            int my_x = -1, my_c = 0;
            float my_bias = 0.f;
            if (tokens && tok_ok && p.counts && tid >= 1 && tid < cnt && t >= x0 && t < x0 + n) {
                my_x = t - x0;
                my_c = p.counts[at + my_x];
                my_bias = p.bias ? p.bias[at + my_x] : 0.f;
            }
            __syncthreads();                              // the sequence before is done with
            if (tid == 0) list_n = 0;
            if (tid < 64) tok[tid] = t;
            if (tid < p.N) masks[tid] = p.mask ? p.mask[(int64_t)b * p.N + tid] & ~1ull : 0ull;
            if (tid < CAP / 32) nodes[tid] = 0u;
            if (__syncthreads_and(tok_ok ? 1 : 0) == 0) err = TV_ERR_OUT_OF_RANGE;
            if (tid == 0) r = LgRow{rep, 1.f / rep, freq, pres, p.unscaled ? 1.f : 1.f / temp, cnt, err};
            if (my_x >= 0) atomicOr(&nodes[my_x >> 5], 1u << (my_x & 31));
            __syncthreads();
            if (p.counts || p.bias) {
                // U groups of four entries per thread and step
                constexpr int U = 2, STEP = LG_THREADS * 4 * U;
                const bool wide = ((reinterpret_cast<uintptr_t>(p.counts) | reinterpret_cast<uintptr_t>(p.bias) |
                                    (uintptr_t)at * 4) & 15) == 0;
                auto get = [&](int base, int (&c)[U][4], float (&f)[U][4]) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int x = base + (u * LG_THREADS + tid) * 4;
                        int4 c4 = make_int4(0, 0, 0, 0);
                        float4 f4 = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (wide && x + 4 <= n) {
                            if (p.counts) c4 = *reinterpret_cast<const int4*>(p.counts + at + x);
                            if (p.bias) f4 = *reinterpret_cast<const float4*>(p.bias + at + x);
                        } else if (x < n) {
                            if (p.counts) {
                                c4.x = p.counts[at + x];
                                if (x + 1 < n) c4.y = p.counts[at + x + 1];
                                if (x + 2 < n) c4.z = p.counts[at + x + 2];
                                if (x + 3 < n) c4.w = p.counts[at + x + 3];
                            }
                            if (p.bias) {
                                f4.x = p.bias[at + x];
                                if (x + 1 < n) f4.y = p.bias[at + x + 1];
                                if (x + 2 < n) f4.z = p.bias[at + x + 2];
                                if (x + 3 < n) f4.w = p.bias[at + x + 3];
                            }
                        }
                        c[u][0] = c4.x, c[u][1] = c4.y, c[u][2] = c4.z, c[u][3] = c4.w;
                        f[u][0] = f4.x, f[u][1] = f4.y, f[u][2] = f4.z, f[u][3] = f4.w;
                    }
                };
                int c[U][4];
                float bs[U][4];
#pragma unroll 1
                for (int base = 0; base < n; base += STEP) {
                    get(base, c, bs);
                    int k = 0;
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e) k += (c[u][e] != 0 || bs[u][e] != 0.f) ? 1 : 0;
                    const int own = k;
                    if (__any_sync(0xffffffffu, own > 0)) {
                        // places for the warp's entries by one atomic
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int y = __shfl_up_sync(0xffffffffu, k, o);
                            if (lane >= o) k += y;
                        }
                        int j = 0;
                        if (lane == 31) j = atomicAdd(&list_n, k);
                        k += __shfl_sync(0xffffffffu, j, 31) - own;
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (c[u][e] != 0 || bs[u][e] != 0.f) {
                                    const int x = base + (u * LG_THREADS + tid) * 4 + e;
                                    if (k < p.list_max)
                                        list[k] = make_uint2((nodes[x >> 5] >> (x & 31)) & 1u ? LG_NODE : lg_word(x, c[u][e]), __float_as_uint(bs[u][e]));
                                    ++k;
                                }
                    }
                }
            }
            if (tid < 64) {
                uint64_t same = 0ull;
                if (my_x >= 0)
                    for (int c = 1; c < cnt; ++c) same |= (uint64_t)(tok[c] == t) << c;
                node_same[tid] = same;
                node_x[tid] = (same & ((1ull << tid) - 1ull)) == 0ull ? my_x : -1;   // once per token
                node_c[tid] = my_c;
                node_bias[tid] = my_bias;
            }
            __syncthreads();
        }
        if (i == 0 && me == 0 && tid == 0) p.status[b] = r.err;
        // ---- the slice has landed; its ends and its grammar words
        // (one warp polls; the others see it through the barrier below)
        if (warp == 0) alive = alive && mbar_wait_sleep(&full, got & 1u);
        ++got;
        const int sh = (int)((reinterpret_cast<uintptr_t>(out) >> 2) & 3);
        const int rsh = (int)((reinterpret_cast<uintptr_t>(static_cast<const E*>(p.logits) + row * p.V + x0) / sizeof(E)) %
                              (16 / sizeof(E)));
        {
            cp_async_wait_all();
            if (tid == 0) s_gram[1 + (n + 31) / 32] = 0u;
            // positions beside the slice weigh nothing
            if constexpr (F32) {
                if (tid < rsh) zs[tid] = -INFINITY;
                for (int q = rsh + n + tid; q < CAP; q += LG_THREADS) zs[q] = -INFINITY;
            }
        }
        const uint64_t m = masks[i];
        auto absent = [&]() -> bool { return r.cnt >= 1 && r.cnt <= p.N && i >= r.cnt; };
        const bool skip = absent() || r.err != TV_OK;
        __syncthreads();
        if constexpr (!F32) {
            // bfloat16: widened, four at a time where both are aligned alike
            uint2 u[NV];
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int q = (k * LG_THREADS + tid) * 4, x = q - sh;
                if (((rsh ^ sh) & 3) == 0) {
                    u[k] = *reinterpret_cast<const uint2*>(raw + q + (rsh - sh));
                } else {
                    const uint16_t* h = reinterpret_cast<const uint16_t*>(raw) + rsh;
                    auto one = [&](int e) -> uint32_t { return x + e >= 0 && x + e < n ? h[x + e] : 0u; };
                    u[k] = make_uint2(one(0) | one(1) << 16, one(2) | one(3) << 16);
                }
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int q = (k * LG_THREADS + tid) * 4, x = q - sh;
                float4 v = make_float4(__uint_as_float(u[k].x << 16), __uint_as_float(u[k].x & 0xffff0000u),
                                       __uint_as_float(u[k].y << 16), __uint_as_float(u[k].y & 0xffff0000u));
                if (x < 0 || x + 4 > n) {
                    // positions beside the slice weigh nothing
                    if (x < 0 || x >= n) v.x = -INFINITY;
                    if (x + 1 < 0 || x + 1 >= n) v.y = -INFINITY;
                    if (x + 2 < 0 || x + 2 >= n) v.z = -INFINITY;
                    if (x + 3 < 0 || x + 3 >= n) v.w = -INFINITY;
                }
                *reinterpret_cast<float4*>(zs + q) = v;
            }
        }
        // (float32: in and out rows may be aligned differently; then the entries move first)
        float* zr = F32 ? reinterpret_cast<float*>(raw) : zs;
        const int zsh = F32 ? rsh : sh;
        // ---- the history and the biases: the list's entries, and (each token once) the nodes'
        const int my_x = tid < 64 ? node_x[tid] : -1;
        const bool mine = my_x >= 0 && !skip;
        if constexpr (!F32) __syncthreads();
        if (!skip && (p.counts || p.bias)) {
            const bool all = list_n > p.list_max;        // (of the whole CTA)
            float my_z = 0.f;
            if (mine) {
                const int on_path = __popcll(node_same[tid] & m), my_c = node_c[tid];
                my_z = zr[my_x + zsh] + node_bias[tid];
                if (my_c != 0 || on_path > 0) my_z = lg_penalty(r, my_z, (my_c & 0x7fffffff) + on_path);
                if (!all) zr[my_x + zsh] = my_z;
            }
            auto change = [&](int x, int c, float bs) {
                float z = zr[x + zsh] + bs;
                if (c != 0) z = lg_penalty(r, z, c & 0x7fffffff);
                zr[x + zsh] = z;
            };
            if (!all) {
                for (int j = tid; j < list_n; j += LG_THREADS) {
                    const uint2 w = list[j];
                    if (w.x == LG_NODE) continue;
                    const int x = (int)(w.x & 0xffffu);
                    const uint32_t k = w.x >> 16;
                    const int c = k == 0u ? 0 : k == LG_LONG ? p.counts[at + x] : (int)(k - 1u) | INT32_MIN;
                    change(x, c, __uint_as_float(w.y));
                }
            } else {
                // more counts and biases than the list holds: all of them, from L2
                __syncthreads();
                const bool wide = ((reinterpret_cast<uintptr_t>(p.counts) | reinterpret_cast<uintptr_t>(p.bias) |
                                    (uintptr_t)at * 4) & 15) == 0;
                const int four = wide ? n & ~3 : 0;
#pragma unroll 1
                for (int x = tid * 4; x < four; x += LG_THREADS * 4) {
                    int4 c = make_int4(0, 0, 0, 0);
                    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (p.counts) c = *reinterpret_cast<const int4*>(p.counts + at + x);
                    if (p.bias) f = *reinterpret_cast<const float4*>(p.bias + at + x);
                    change(x, c.x, f.x);
                    change(x + 1, c.y, f.y);
                    change(x + 2, c.z, f.z);
                    change(x + 3, c.w, f.w);
                }
                for (int x = four + tid; x < n; x += LG_THREADS) {
                    const int c = p.counts ? p.counts[at + x] : 0;
                    const float bs = p.bias ? p.bias[at + x] : 0.f;
                    if (c != 0 || bs != 0.f) change(x, c, bs);
                }
                __syncthreads();
                if (mine) zr[my_x + zsh] = my_z;
            }
            __syncthreads();
        }
        // ---- into registers: positions 4 (k LG_THREADS + tid) of the buffer
        float z[NV][4];
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int q = (k * LG_THREADS + tid) * 4, x = q - zsh;
            const float4 v = *reinterpret_cast<const float4*>(zr + q);
            z[k][0] = v.x;
            z[k][1] = v.y;
            z[k][2] = v.z;
            z[k][3] = v.w;
            if (p.grammar) {                             // (beyond the slice: whatever is there, on -infinity)
                const int w = (x + 32) >> 5;             // (s_gram[0] stands before the slice)
                const uint32_t lo = s_gram[w], hi = zsh != 0 ? s_gram[w + 1] : 0u;
                const uint32_t ok = __funnelshift_r(lo, hi, (x + 32) & 31);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!((ok >> e) & 1u)) z[k][e] = -INFINITY;
            }
            if constexpr (PROBS) mx = lg_max3(lg_max3(mx, z[k][0], z[k][1]), z[k][2], z[k][3]);
        }
        fence_proxy_async_smem();                        // the next copy lands where this row was
        if (__syncthreads_and(alive ? 1 : 0) == 0) {     // a wait ran out, in this row or the last
            if (tid == 0) late_row = max(row_lo, row - 1);
            mbar_wait_sleep(&full, (got - 1u) & 1u);     // (a copy still in flight)
            break;
        }
        if (row + 1 < row_hi) fetch(row + 1, b, i + 1 < p.N);
        const int err = r.err;
        if (absent()) continue;                          // an absent node: nothing is written
        auto store = [&](float scale) {
            // (computed again, rather than kept in registers that there are too few of)
            int64_t at_row = row;
            asm volatile("" : "+l"(at_row));
            float* out = p.out + at_row * p.V + x0;
            const int sh = (int)((reinterpret_cast<uintptr_t>(out) >> 2) & 3);
            const int zsh = F32 ? (int)((reinterpret_cast<uintptr_t>(static_cast<const E*>(p.logits) + at_row * p.V + x0) / sizeof(E)) %
                                        (16 / sizeof(E))) : sh;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int x = (k * LG_THREADS + tid) * 4 - zsh;
                if (x >= 0 && x + 4 <= n && zsh == sh) {
                    __stcs(reinterpret_cast<float4*>(out + x),
                           make_float4(z[k][0] * scale, z[k][1] * scale, z[k][2] * scale, z[k][3] * scale));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (x + e >= 0 && x + e < n) out[x + e] = z[k][e] * scale;
                }
            }
        };
        if (err != TV_OK) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[k][e] = PROBS ? 0.f : -INFINITY;
            store(1.f);
            continue;
        }
        if constexpr (!PROBS) {
            store(r.inv_temp);
        } else {
            // ---- softmax: every warp's maximum and its sum relative to that go to all CTAs of the
            // row, and each warp combines them all, in the same order: weights 2^(m - max).  No
            // barrier of the CTA is needed, nor one of the cluster (which would first wait for the
            // row before to be stored).  Exponents are differences of logits times the scale, not of
            // products: those may be too large for their difference to mean anything.
            const float scale = LG_LOG2E * r.inv_temp;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = lg_max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float base = mx == -INFINITY ? 0.f : -mx;
            const uint64_t base2 = f2_pack(base, base), scale2 = f2_pack(scale, scale);
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    float a, c;
                    f2_unpack(f2_mul(f2_add(f2_pack(z[k][e], z[k][e + 1]), base2), scale2), a, c);
                    z[k][e] = ex2_approx(a);
                    z[k][e + 1] = ex2_approx(c);
                }
                sum += (z[k][0] + z[k][1]) + (z[k][2] + z[k][3]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            // Two barriers in turn: a CTA may be one row ahead of another (for the row after that
            // it needs a pair that the other sends when it has all of this row's).  A CTA ends only
            // with every pair here.
            const uint32_t par = phase & 1u;
            uint64_t* bar = &peer_bar[par];
            if (warp == 0) mbar_arrive_expect_tx_relaxed_elect(bar, (uint32_t)(p.slices * LG_WARPS * 8));
            __syncwarp();
            if (lane < p.slices) remote_st_async(&peer[par][me * LG_WARPS + warp], bar, (uint32_t)lane, mx, sum);
            alive = alive && mbar_wait_sleep(bar, (phase >> 1) & 1u);
            ++phase;
            const volatile float* pairs = reinterpret_cast<const volatile float*>(peer[par]);
            float top = -INFINITY, total = 0.f;
            for (int k = lane; k < p.slices * LG_WARPS; k += 32) top = lg_max(top, pairs[2 * k]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = lg_max(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (top == -INFINITY) top = 0.f;
            for (int k = lane; k < p.slices * LG_WARPS; k += 32) total = fmaf(pairs[2 * k + 1], exp2f((pairs[2 * k] - top) * scale), total);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            const float w = total == 0.f ? 0.f : exp2f((mx - top) * scale) / total;
            store(w);                                    // (NaN stays NaN)
        }
    }
    const bool late = __syncthreads_and(alive ? 1 : 0) == 0;   // (the last row's pairs, too)
    // after a wait that ran out, pairs may still be on their way to this CTA; every CTA gets here,
    // as every wait is bounded
    if (PROBS && p.slices > 1) cluster_barrier_relaxed();
    if (late) lg_fail(p, late_row, PROBS ? 0.f : -INFINITY);
}

template <typename E, bool PROBS, int NV>
tv_status launch_nv(LgParams p, cudaStream_t stream) {
    auto fn = tree_logits_kernel<E, PROBS, NV>;
    constexpr int CAP = LG_THREADS * 4 * NV;
    const size_t fixed = CAP * 4 + (sizeof(E) == 4 ? 0 : 16) + (CAP / 32 + 2) * 4;
    p.list_max = (p.counts || p.bias) ? std::min<int>(p.slice, (int)((LG_SMEM - fixed) / 8)) : 0;
    const size_t smem = fixed + (size_t)p.list_max * 8;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TV_ERR_CUDA;
    static std::atomic<bool> set[64];
    if (!set[dev]) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, LG_SMEM) != cudaSuccess ||
            (PROBS && cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)) {
            cudaGetLastError();
            return TV_ERR_CUDA;
        }
        set[dev] = true;
    }
    // as many groups as the GPU holds at once
    LaunchCfg lc(dim3((unsigned)p.slices), dim3(LG_THREADS), smem, stream, PROBS ? (unsigned)p.slices : 0u);
    // (the last answer is kept: slices, shared memory, what fits)
    static std::atomic<uint64_t> last[64];
    const uint64_t key = ((uint64_t)p.slices << 48) | ((uint64_t)smem << 16);
    const uint64_t known = last[dev].load();
    int fit = (int)(known & 0xffff);
    if ((known & ~0xffffull) != key || fit == 0) {
        const cudaError_t e = PROBS ? cudaOccupancyMaxActiveClusters(&fit, fn, &lc.cfg)
                                    : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, fn, LG_THREADS, smem);
        if (e != cudaSuccess || fit < 1) {
            cudaGetLastError();
            return TV_ERR_CUDA;
        }
        fit = std::min(fit, 0xffff);
        last[dev].store(key | (uint64_t)fit);
    }
    if (!PROBS) fit = std::max(1, fit * device_sm_count() / p.slices);
    p.groups = (int)std::min<int64_t>(p.rows, fit);
    lc.cfg.gridDim = dim3((unsigned)(p.groups * p.slices));
    return cudaLaunchKernelEx(&lc.cfg, fn, p) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

template <typename E, bool PROBS>
tv_status launch_slices(const LgParams& p, cudaStream_t stream) {
    const int per = (p.slice + 3 + LG_THREADS * 4 - 1) / (LG_THREADS * 4);
    if constexpr (!PROBS) {
        return launch_nv<E, PROBS, 4>(p, stream);
    } else {
        if (per <= 2) return launch_nv<E, PROBS, 2>(p, stream);
        if (per <= 5) return launch_nv<E, PROBS, 5>(p, stream);
        return launch_nv<E, PROBS, LG_NV_MAX>(p, stream);
    }
}

// Rows that no cluster holds: the logits are written first, not yet divided by the
// temperature, and this softmax, one CTA per row, reads them again: exponents are
// differences of logits times the scale here, too (208 rows of 262,144: 388 us, where one
// reading and writing of them would be 68 at the copy rate).
__global__ void __launch_bounds__(LG_THREADS) row_softmax_kernel(const LgParams p) {
    __shared__ float red[2][LG_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x;
    const int b = (int)(row / p.N), i = (int)(row % p.N);
    pdl_launch_dependents();
    pdl_wait();
    const int cnt = p.node_counts ? p.node_counts[b] : p.N;
    if (cnt >= 1 && cnt <= p.N && i >= cnt) return;      // an absent node's row
    float* z = p.out + row * p.V;
    auto reduce = [&](float v, bool sum, int where) -> float {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, v, o);
            v = sum ? v + y : lg_max(v, y);
        }
        if (lane == 0) red[where][warp] = v;
        __syncthreads();
        v = sum ? 0.f : -INFINITY;
        for (int w = 0; w < LG_THREADS / 32; ++w) v = sum ? v + red[where][w] : lg_max(v, red[where][w]);
        return v;
    };
    float mx = -INFINITY, sum = 0.f;
    for (int x = tid; x < p.V; x += LG_THREADS) mx = lg_max(mx, z[x]);
    mx = reduce(mx, false, 0);
    if (mx == -INFINITY) {                               // nothing allowed, or a refused sequence
        for (int x = tid; x < p.V; x += LG_THREADS) z[x] = 0.f;
        return;
    }
    const float scale = LG_LOG2E * (p.temp ? 1.f / p.temp[b] : 1.f);
    for (int x = tid; x < p.V; x += LG_THREADS) sum += ex2_approx((z[x] - mx) * scale);
    sum = reduce(sum, true, 1);
    const float inv = 1.f / sum;                         // (the sum is at least 1, or NaN)
    for (int x = tid; x < p.V; x += LG_THREADS) z[x] = ex2_approx((z[x] - mx) * scale) * inv;
}

template <typename E>
tv_status launch_logits(const LogitsArgs& a, LgParams p) {
    const bool cluster = a.probs && a.V <= LG_CLUSTER_MAX * LG_SLICE_MAX;
    p.rows = (int64_t)a.B * a.N;
    if (cluster) {
        // the fewest CTAs that hold the row; up to 8 when that leaves SMs without work
        int cs = (a.V + LG_SLICE_MAX - 1) / LG_SLICE_MAX;
        while (cs <= 4 && p.rows * cs < device_sm_count() && a.V > cs * 4096) cs *= 2;
        p.slices = cs;
    } else {
        p.slices = (a.V + LG_PLAIN_SLICE - 1) / LG_PLAIN_SLICE;
    }
    p.slice = ((a.V + p.slices - 1) / p.slices + 31) & ~31;
    if (cluster) return launch_slices<E, true>(p, a.stream);
    p.unscaled = a.probs;
    const tv_status rc = launch_slices<E, false>(p, a.stream);
    if (rc != TV_OK || !a.probs) return rc;
    if (p.rows > 0x7fffffff) return TV_ERR_UNSUPPORTED;
    LaunchCfg lc(dim3((unsigned)p.rows), dim3(LG_THREADS), 0, a.stream);
    return cudaLaunchKernelEx(&lc.cfg, row_softmax_kernel, p) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // namespace

tv_status launch_tree_logits(const LogitsArgs& a) {
    LgParams p{};
    p.logits = a.logits;
    p.node_counts = a.node_counts;
    p.mask = a.mask;
    p.tokens = a.tokens;
    p.counts = a.counts;
    p.bias = a.bias;
    p.grammar = a.grammar;
    p.rep = a.rep;
    p.freq = a.freq;
    p.pres = a.pres;
    p.temp = a.temp;
    p.out = a.out;
    p.status = a.status;
    p.N = a.N;
    p.V = a.V;
    p.words = (a.V + 31) / 32;
    p.late = test_late_wait();
    return a.dt == TV_F32 ? launch_logits<float>(a, p) : launch_logits<__nv_bfloat16>(a, p);
}

}  // namespace tv
