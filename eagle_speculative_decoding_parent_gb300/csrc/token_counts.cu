// token_counts_update: the token histories that tree_logits_process reads.
//
// With `clear` the whole row is written, so a CTA takes a slice of one row:
// it zeroes the slice in shared memory, goes through all tokens of the
// sequence (they stay in L2) applying those that fall into the slice, and
// writes the slice out once: the row's bytes are the bound.  Without it only a
// few words change: one CTA per sequence checks the tokens, then applies them
// with integer atomics on the row.
#include "tv_device.cuh"
#include "tv_internal.h"

namespace tv {

namespace {

constexpr int TC_THREADS = 256;
constexpr int TC_SLICE = 8192;  // entries per CTA: 32 KB of shared memory, six CTAs per SM

struct TcParams {
    int32_t* counts;
    const int32_t* tokens;
    const int32_t* starts;  // nullable
    int32_t* status;
    int total, B, V, slices;  // slices of a row
    bool prompt;
};

// Token range of sequence b; false when the starts array is out of order or range.
__device__ __forceinline__ bool tc_range(const TcParams& p, int b, int& lo, int& hi) {
    if (!p.starts) {
        const int w = p.total / p.B;
        lo = b * w;
        hi = lo + w;
        return true;
    }
    bool ok = true;
    for (int i = threadIdx.x; i < p.B; i += TC_THREADS) {
        const int s = p.starts[i], e = p.starts[i + 1];
        ok = ok && s >= 0 && s <= e && e <= p.total;
    }
    lo = p.starts[b];
    hi = p.starts[b + 1];
    return __syncthreads_and(ok ? 1 : 0) != 0;
}

__device__ __forceinline__ bool tc_token_ok(const TcParams& p, int x) { return x >= -1 && x < p.V; }

__global__ void __launch_bounds__(TC_THREADS) counts_add_kernel(TcParams p) {
    const int b = blockIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    int lo, hi;
    bool ok = tc_range(p, b, lo, hi);
    if (ok)
        for (int i = lo + threadIdx.x; i < hi; i += TC_THREADS) ok = ok && tc_token_ok(p, p.tokens[i]);
    ok = __syncthreads_and(ok ? 1 : 0) != 0;
    if (threadIdx.x == 0) p.status[b] = ok ? TV_OK : TV_ERR_OUT_OF_RANGE;
    if (!ok) return;
    int32_t* row = p.counts + (int64_t)b * p.V;
    for (int i = lo + threadIdx.x; i < hi; i += TC_THREADS) {
        const int x = p.tokens[i];
        if (x < 0) continue;
        if (p.prompt) atomicOr(row + x, INT32_MIN);
        else atomicAdd(row + x, 1);
    }
}

__global__ void __launch_bounds__(TC_THREADS) counts_clear_kernel(TcParams p) {
    __shared__ __align__(16) int32_t part[TC_SLICE];
    const int b = blockIdx.x / p.slices, x0 = (int)(blockIdx.x % p.slices) * TC_SLICE;
    const int n = min(TC_SLICE, p.V - x0);
    for (int i = threadIdx.x; i < TC_SLICE / 4; i += TC_THREADS)
        reinterpret_cast<int4*>(part)[i] = make_int4(0, 0, 0, 0);
    pdl_launch_dependents();
    pdl_wait();
    int lo, hi;
    bool ok = tc_range(p, b, lo, hi);
    __syncthreads();
    if (ok) {
        for (int i = lo + threadIdx.x; i < hi; i += TC_THREADS) {
            const int x = p.tokens[i], at = x - x0;
            ok = ok && tc_token_ok(p, x);
            if (x < 0 || at < 0 || at >= n) continue;
            if (p.prompt) part[at] = INT32_MIN;   // every writer writes the same word
            else atomicAdd(&part[at], 1);
        }
    }
    ok = __syncthreads_and(ok ? 1 : 0) != 0;
    if (threadIdx.x == 0 && x0 == 0) p.status[b] = ok ? TV_OK : TV_ERR_OUT_OF_RANGE;
    if (!ok) return;
    int32_t* row = p.counts + (int64_t)b * p.V + x0;
    if ((reinterpret_cast<uintptr_t>(row) & 15) == 0) {
        for (int i = threadIdx.x; i < n / 4; i += TC_THREADS)
            reinterpret_cast<int4*>(row)[i] = reinterpret_cast<const int4*>(part)[i];
        if (threadIdx.x < (n & 3)) row[(n & ~3) + threadIdx.x] = part[(n & ~3) + threadIdx.x];
    } else {
        for (int i = threadIdx.x; i < n; i += TC_THREADS) row[i] = part[i];
    }
}

}  // namespace

tv_status launch_token_counts(int32_t* counts, const int32_t* tokens, const int32_t* starts,
                              int total, int B, int V, bool clear, bool prompt, int32_t* status,
                              cudaStream_t stream) {
    TcParams p{counts, tokens, starts, status, total, B, V, (V + TC_SLICE - 1) / TC_SLICE, prompt};
    if (clear) {
        if ((int64_t)B * p.slices > 0x7fffffff) return TV_ERR_UNSUPPORTED;
        LaunchCfg lc(dim3((unsigned)(B * p.slices)), dim3(TC_THREADS), 0, stream);
        return cudaLaunchKernelEx(&lc.cfg, counts_clear_kernel, p) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
    }
    LaunchCfg lc(dim3((unsigned)B), dim3(TC_THREADS), 0, stream);
    return cudaLaunchKernelEx(&lc.cfg, counts_add_kernel, p) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // namespace tv
