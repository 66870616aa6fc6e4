// tree_logits_process: the target model's rows of a tree into the logits or
// probabilities that acceptance reads.
//
// Per entry: z = logit + bias; a token that the history or the node's own path
// holds is divided (or multiplied) by the repetition penalty; z -= frequency *
// n + presence * [n > 0]; a token that the grammar forbids becomes -infinity.
// Then z / temperature, or its softmax.
//
// Bound by memory: the row is read once and written once; counts and bias are
// shared by a tree's N rows and come from L2 after the first.  For the softmax
// a cluster of CTAs holds the row's processed logits in shared memory (a row of
// 128,256 tokens is 501 KB), so that the maximum and the sum need no second
// read of the row: each CTA reduces its slice, and the (maximum, then sum) of
// the slices are exchanged through distributed shared memory.
//
// The path's tokens: at most 63 per row.  Those that fall into the CTA's slice
// are marked in a bitmap in shared memory; an entry whose bit is set (a rare
// one) counts its occurrences in the list.
#include <cuda_bf16.h>
#include <math.h>

#include "tv_device.cuh"
#include "tv_internal.h"

namespace tv {

namespace {

constexpr int LG_THREADS = 512;
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
    int slices;     // CTAs per row (the cluster, for the softmax)
    int slice;      // entries per CTA, a multiple of 32
    int staged;     // of them, how many are kept in shared memory (softmax)
};

// What one row needs besides its logits.
struct LgRow {
    float rep, freq, pres, temp;
    const int32_t* counts;     // nullable
    const float* bias;         // nullable
    const uint32_t* grammar;   // nullable
    const uint32_t* marks;     // bitmap of the slice's path tokens, null without any
    const int* path;
    int n_path;
    int x0;                    // the slice's first token
};

// The processed entry x (before the temperature).
__device__ __forceinline__ float lg_entry(const LgRow& r, float z, int x, int word, float bias) {
    z += bias;
    int n = word & 0x7fffffff;
    if (r.marks && ((r.marks[(x - r.x0) >> 5] >> ((x - r.x0) & 31)) & 1u))
        for (int i = 0; i < r.n_path; ++i) n += r.path[i] == x;
    if (word < 0 || n > 0) z = z > 0.f ? z / r.rep : z * r.rep;
    z -= r.freq * (float)n;
    return n > 0 ? z - r.pres : z;
}

template <typename E>
__device__ __forceinline__ float lg_load(const E* p, int64_t i);
template <>
__device__ __forceinline__ float lg_load<float>(const float* p, int64_t i) { return __ldcs(p + i); }
template <>
__device__ __forceinline__ float lg_load<__nv_bfloat16>(const __nv_bfloat16* p, int64_t i) {
    return __bfloat162float(__ldcs(p + i));
}
__device__ __forceinline__ float4 lg_load4(const float* p) {
    return __ldcs(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ float4 lg_load4(const __nv_bfloat16* p) {
    const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

// Row state of (b, i), shared by both kernels.  Returns 0 when the row is to be
// processed, 1 when it is absent, 2 when its sequence has an error.  Called by
// every thread of the CTA (contains barriers).
__device__ __forceinline__ int lg_row_setup(const LgParams& p, int b, int i, int x0, int n,
                                            uint32_t* marks, int* path, int* misc, LgRow& r,
                                            bool report) {
    const int tid = threadIdx.x;
    const int cnt = p.node_counts ? p.node_counts[b] : p.N;
    r.rep = p.rep ? p.rep[b] : 1.f;
    r.freq = p.freq ? p.freq[b] : 0.f;
    r.pres = p.pres ? p.pres[b] : 0.f;
    r.temp = p.temp ? p.temp[b] : 1.f;
    int err = (cnt >= 1 && cnt <= p.N) ? TV_OK : TV_ERR_OUT_OF_RANGE;
    const bool absent = err == TV_OK && i >= cnt;
    if (err == TV_OK && !(isfinite(r.rep) && r.rep > 0.f && isfinite(r.temp) && r.temp > 0.f &&
                          isfinite(r.freq) && isfinite(r.pres)))
        err = TV_ERR_BAD_VALUES;
    if (tid == 0) misc[0] = 0;
    // the tokens of nodes 1 .. cnt-1, one per thread
    bool tok_ok = true;
    int tok = -1;
    if (p.mask && err != TV_ERR_OUT_OF_RANGE && tid >= 1 && tid < cnt) {
        tok = p.tokens[(int64_t)b * p.N + tid];
        tok_ok = tok >= 0 && tok < p.V;
    }
    if (__syncthreads_and(tok_ok ? 1 : 0) == 0) err = TV_ERR_OUT_OF_RANGE;
    if (report && tid == 0) p.status[b] = err;
    if (absent) return 1;
    if (err != TV_OK) return 2;
    r.counts = p.counts ? p.counts + (int64_t)b * p.V : nullptr;
    r.bias = p.bias ? p.bias + (int64_t)b * p.V : nullptr;
    r.grammar = p.grammar ? p.grammar + ((int64_t)b * p.N + i) * p.words : nullptr;
    r.marks = nullptr;
    r.path = path;
    r.x0 = x0;
    r.n_path = 0;
    if (p.mask && p.counts) {
        const uint64_t m = p.mask[(int64_t)b * p.N + i];
        const bool mine = tid >= 1 && tid < cnt && ((m >> (tid & 63)) & 1ull) && tok >= x0 && tok < x0 + n;
        if (mine) path[atomicAdd(&misc[0], 1)] = tok;
        __syncthreads();
        r.n_path = misc[0];
        if (r.n_path > 0) {
            for (int w = tid; w < (n + 31) / 32; w += blockDim.x) marks[w] = 0u;
            __syncthreads();
            if (tid < r.n_path) atomicOr(&marks[(path[tid] - x0) >> 5], 1u << ((path[tid] - x0) & 31));
            __syncthreads();
            r.marks = marks;
        }
    }
    return 0;
}

// Processes entries x .. x + 3 (VEC) or entry x.
template <typename E, bool VEC>
__device__ __forceinline__ void lg_process(const LgRow& r, const E* in, int x, float (&z)[VEC ? 4 : 1]) {
    if constexpr (VEC) {
        const float4 v = lg_load4(in + x);
        int4 c = make_int4(0, 0, 0, 0);
        float4 bs = make_float4(0.f, 0.f, 0.f, 0.f);
        uint32_t ok = 0xfu;
        if (r.counts) c = *reinterpret_cast<const int4*>(r.counts + x);
        if (r.bias) bs = *reinterpret_cast<const float4*>(r.bias + x);
        if (r.grammar) ok = __ldcs(r.grammar + (x >> 5)) >> (x & 31);
        z[0] = (ok & 1u) ? lg_entry(r, v.x, x, c.x, bs.x) : -INFINITY;
        z[1] = (ok & 2u) ? lg_entry(r, v.y, x + 1, c.y, bs.y) : -INFINITY;
        z[2] = (ok & 4u) ? lg_entry(r, v.z, x + 2, c.z, bs.z) : -INFINITY;
        z[3] = (ok & 8u) ? lg_entry(r, v.w, x + 3, c.w, bs.w) : -INFINITY;
    } else {
        const float v = lg_load<E>(in, x);
        const int c = r.counts ? r.counts[x] : 0;
        const float bs = r.bias ? r.bias[x] : 0.f;
        const bool ok = !r.grammar || ((r.grammar[x >> 5] >> (x & 31)) & 1u);
        z[0] = ok ? lg_entry(r, v, x, c, bs) : -INFINITY;
    }
}

template <int W>
__device__ __forceinline__ void lg_store(float* p, const float (&z)[W]) {
    if constexpr (W == 4) __stcs(reinterpret_cast<float4*>(p), make_float4(z[0], z[1], z[2], z[3]));
    else __stcs(p, z[0]);
}

template <int W>
__device__ __forceinline__ void lg_stage(float* p, const float (&z)[W]) {
    if constexpr (W == 4) *reinterpret_cast<float4*>(p) = make_float4(z[0], z[1], z[2], z[3]);
    else *p = z[0];
}
template <int W>
__device__ __forceinline__ void lg_unstage(const float* p, float (&z)[W]) {
    if constexpr (W == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        z[0] = v.x;
        z[1] = v.y;
        z[2] = v.z;
        z[3] = v.w;
    } else {
        z[0] = *p;
    }
}

// Logits out: one CTA per (slice, row).
template <typename E, bool VEC>
__global__ void __launch_bounds__(LG_THREADS) logits_kernel(LgParams p) {
    extern __shared__ uint32_t marks[];
    __shared__ int path[64];
    __shared__ int misc[1];
    const int64_t row = blockIdx.x / p.slices;
    const int part = (int)(blockIdx.x % p.slices);
    const int b = (int)(row / p.N), i = (int)(row % p.N);
    const int x0 = part * p.slice, n = min(p.slice, p.V - x0);
    constexpr int W = VEC ? 4 : 1;
    pdl_launch_dependents();
    pdl_wait();
    LgRow r;
    const int what = lg_row_setup(p, b, i, x0, n, marks, path, misc, r, i == 0 && part == 0);
    if (what == 1) return;
    const E* in = static_cast<const E*>(p.logits) + row * p.V;
    float* out = p.out + row * p.V;
    for (int x = x0 + threadIdx.x * W; x < x0 + n; x += LG_THREADS * W) {
        float z[W];
        if (what == 2) {
#pragma unroll
            for (int e = 0; e < W; ++e) z[e] = -INFINITY;
        } else {
            lg_process<E, VEC>(r, in, x, z);
#pragma unroll
            for (int e = 0; e < W; ++e) z[e] = z[e] / r.temp;
        }
        lg_store(out + x, z);
    }
}

__device__ __forceinline__ float lg_max(float a, float b) {  // NaN wins
    return (a > b || a != a) ? a : b;
}

// Probabilities out: one cluster per row, CTA c of it the slice c.
template <typename E, bool VEC>
__global__ void __launch_bounds__(LG_THREADS) probs_kernel(LgParams p) {
    extern __shared__ __align__(16) float stage[];      // [staged], then the bitmap
    __shared__ int path[64];
    __shared__ int misc[1];
    __shared__ float red[LG_THREADS / 32];
    __shared__ __align__(16) float part[2][4];          // this CTA's maximum, its sum
    const int64_t row = blockIdx.x / p.slices;
    const int b = (int)(row / p.N), i = (int)(row % p.N);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cs = p.slices, me = (int)(blockIdx.x % p.slices);
    const int x0 = me * p.slice, n = max(0, min(p.slice, p.V - x0));
    constexpr int W = VEC ? 4 : 1;
    uint32_t* marks = reinterpret_cast<uint32_t*>(stage + p.staged);
    pdl_launch_dependents();
    pdl_wait();
    LgRow r;
    const int what = lg_row_setup(p, b, i, x0, n, marks, path, misc, r, i == 0 && me == 0);
    if (what == 1) return;                               // the whole cluster returns
    const E* in = static_cast<const E*>(p.logits) + row * p.V;
    float* out = p.out + row * p.V;
    if (what == 2) {
        const float zero[W] = {};
        for (int x = x0 + tid * W; x < x0 + n; x += LG_THREADS * W) lg_store(out + x, zero);
        return;
    }
    // maximum over the cluster
    float mx = -INFINITY;
    for (int e = tid * W; e < n; e += LG_THREADS * W) {
        float z[W];
        lg_process<E, VEC>(r, in, x0 + e, z);
#pragma unroll
        for (int k = 0; k < W; ++k) mx = lg_max(z[k], mx);
        if (e < p.staged) lg_stage(stage + e, z);
    }
    auto reduce = [&](float v, bool sum, int where) -> float {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, v, o);
            v = sum ? v + y : lg_max(v, y);
        }
        if (lane == 0) red[warp] = v;
        __syncthreads();
        v = lane < LG_THREADS / 32 ? red[lane] : (sum ? 0.f : -INFINITY);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, v, o);
            v = sum ? v + y : lg_max(v, y);
        }
        if (tid == 0) part[where][0] = v;
        cluster_barrier_all();
        // every CTA adds the parts in rank order, so all hold the same value
        float all = sum ? 0.f : -INFINITY;
        for (int c = 0; c < cs; ++c) {
            const float u = remote_ld_f4(part[where], (uint32_t)c).x;
            all = sum ? all + u : lg_max(all, u);
        }
        return all;
    };
    mx = reduce(mx, false, 0);
    // exp((z - max) / temperature): the difference first, so the temperature's
    // rounding does not grow with the logits
    const float scale = LG_LOG2E / r.temp;
    const float base = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
    for (int e = tid * W; e < n; e += LG_THREADS * W) {
        float z[W];
        if (e < p.staged) lg_unstage(stage + e, z);
        else lg_process<E, VEC>(r, in, x0 + e, z);
#pragma unroll
        for (int k = 0; k < W; ++k) {
            z[k] = ex2_approx((z[k] - base) * scale);
            sum += z[k];
        }
        if (e < p.staged) lg_stage(stage + e, z);
    }
    sum = reduce(sum, true, 1);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;      // NaN stays NaN
    for (int e = tid * W; e < n; e += LG_THREADS * W) {
        float z[W];
        if (e < p.staged) {
            lg_unstage(stage + e, z);
        } else {
            lg_process<E, VEC>(r, in, x0 + e, z);
#pragma unroll
            for (int k = 0; k < W; ++k) z[k] = ex2_approx((z[k] - base) * scale);
        }
#pragma unroll
        for (int k = 0; k < W; ++k) z[k] *= inv;
        lg_store(out + x0 + e, z);
    }
    cluster_barrier_all();  // no CTA leaves while others read its part
}

template <typename E>
tv_status launch_logits(const LogitsArgs& a, const LgParams& p0, bool vec) {
    LgParams p = p0;
    const int64_t rows = (int64_t)a.B * a.N;
    if (!a.probs) {
        p.slice = 4096;
        p.slices = (a.V + p.slice - 1) / p.slice;
        if (rows * p.slices > 0x7fffffff) return TV_ERR_UNSUPPORTED;
        LaunchCfg lc(dim3((unsigned)(rows * p.slices)), dim3(LG_THREADS), (size_t)p.slice / 8, a.stream);
        const cudaError_t e = vec ? cudaLaunchKernelEx(&lc.cfg, logits_kernel<E, true>, p)
                                  : cudaLaunchKernelEx(&lc.cfg, logits_kernel<E, false>, p);
        return e == cudaSuccess ? TV_OK : TV_ERR_CUDA;
    }
    // cluster size: the fewest CTAs (up to 8) whose slice is at most 64 KB; rows longer
    // than eight such slices take larger ones, and what does not fit into shared
    // memory is read again
    int cs = 1;
    while (cs < 8 && (int64_t)cs * 16384 < a.V) cs *= 2;
    if (rows * cs > 0x7fffffff) return TV_ERR_UNSUPPORTED;
    p.slices = cs;
    p.slice = ((a.V + cs - 1) / cs + 31) & ~31;
    const int room = ((device_smem_optin() - 4096) / 4) & ~31;   // words
    p.staged = p.slice;
    if (p.slice + p.slice / 32 > room) p.staged = max(0, (room - p.slice / 32) & ~31);
    const size_t smem = (size_t)(p.staged + p.slice / 32) * 4;
    if (smem > (size_t)room * 4) return TV_ERR_UNSUPPORTED;
    auto fn = vec ? probs_kernel<E, true> : probs_kernel<E, false>;
    if (smem > 48 * 1024 - 1024 &&
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
        cudaGetLastError();
        return TV_ERR_CUDA;
    }
    LaunchCfg lc(dim3((unsigned)(rows * cs)), dim3(LG_THREADS), smem, a.stream, (unsigned)cs);
    return cudaLaunchKernelEx(&lc.cfg, fn, p) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
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
    const uintptr_t all = reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.counts) |
                          reinterpret_cast<uintptr_t>(a.bias) |
                          (reinterpret_cast<uintptr_t>(a.logits) << (a.dt == TV_BF16 ? 1 : 0));
    const bool vec = a.V % 4 == 0 && (all & 15) == 0;
    return a.dt == TV_F32 ? launch_logits<float>(a, p, vec) : launch_logits<__nv_bfloat16>(a, p, vec);
}

}  // namespace tv
