// token_counts_update: the token histories that tree_logits_process reads.
//
// With `clear` the whole row is written, so a CTA takes a slice of one row:
// it zeroes the slice in shared memory, goes through all tokens of the
// sequence (they stay in L2) applying those that fall into the slice, and
// writes the slice out once: the row's bytes are the bound.  Without it only a
// few words change: the CTAs of a sequence all check its tokens, and each applies
// its share with integer atomics on the row.  A scan is bound by the latency of
// its loads, so each thread has UNROLL of them in flight.
// Measured: 32 rows of 128,256 with up to 8,192 tokens each 6.4 us (2.6 TB/s; 512 or 1,024
// threads and slices of 4,096 no faster), 128 rows with 1-6 tokens 1.7 us captured, 5.5 from the
// host, which takes that long.
#include <algorithm>

#include "tv_device.cuh"
#include "tv_internal.h"

namespace tv {

namespace {

constexpr int TC_THREADS = 256;
constexpr int UNROLL = 8;
constexpr int TC_SHARE = 4096;  // tokens per CTA without `clear`, on average over the sequences
constexpr int TC_SLICE = 8192;  // entries per CTA: 32 KB of shared memory, six CTAs per SM

struct TcParams {
    int32_t* counts;
    const int32_t* tokens;
    const int32_t* starts;  // nullable
    int32_t* status;
    int total, B, V, slices;  // CTAs per sequence
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
    lo = p.starts[b];       // beside the loads of the check, whose barrier is in between
    hi = p.starts[b + 1];
    bool ok = true;
    for (int i = threadIdx.x; i < p.B; i += TC_THREADS) {
        const int s = p.starts[i], e = p.starts[i + 1];
        ok = ok && s >= 0 && s <= e && e <= p.total;
    }
    return __syncthreads_and(ok ? 1 : 0) != 0;
}

__device__ __forceinline__ bool tc_token_ok(const TcParams& p, int x) { return x >= -1 && x < p.V; }

// each(token) for the tokens lo .. hi, every `step`-th from lo + first on.
template <class Each>
__device__ __forceinline__ void tc_tokens(const TcParams& p, int lo, int hi, int first, int step, Each each) {
    for (int64_t i = (int64_t)lo + first; i < hi; i += (int64_t)UNROLL * step) {
        int x[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int64_t at = i + (int64_t)u * step;
            x[u] = at < hi ? p.tokens[at] : -1;
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) each(x[u]);
    }
}

__global__ void __launch_bounds__(TC_THREADS) counts_add_kernel(TcParams p) {
    const int b = blockIdx.x / p.slices, share = blockIdx.x % p.slices;
    pdl_launch_dependents();
    pdl_wait();
    int lo, hi;
    bool ok = tc_range(p, b, lo, hi);
    if (ok) tc_tokens(p, lo, hi, threadIdx.x, TC_THREADS, [&](int x) { ok = ok && tc_token_ok(p, x); });
    ok = __syncthreads_and(ok ? 1 : 0) != 0;
    if (threadIdx.x == 0 && share == 0) p.status[b] = ok ? TV_OK : TV_ERR_OUT_OF_RANGE;
    if (!ok) return;
    int32_t* row = p.counts + (int64_t)b * p.V;
    tc_tokens(p, lo, hi, share * TC_THREADS + threadIdx.x, p.slices * TC_THREADS, [&](int x) {
        if (x < 0) return;
        if (p.prompt) atomicOr(row + x, INT32_MIN);
        else atomicAdd(row + x, 1);
    });
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
    if (ok)
        tc_tokens(p, lo, hi, threadIdx.x, TC_THREADS, [&](int x) {
            ok = ok && tc_token_ok(p, x);
            if (x < x0 || x >= x0 + n) return;
            if (p.prompt) part[x - x0] = INT32_MIN;   // every writer writes the same word
            else atomicAdd(&part[x - x0], 1);
        });
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
    p.slices = std::max(1, (int)std::min<int64_t>(total / ((int64_t)B * TC_SHARE), 0x7fffffff / B));
    LaunchCfg lc(dim3((unsigned)(B * p.slices)), dim3(TC_THREADS), 0, stream);
    return cudaLaunchKernelEx(&lc.cfg, counts_add_kernel, p) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // namespace tv
