// Device helpers for ragged chunks: the batch's row ranges (q_start), the keys
// a sequence needs, and finding the sequence that holds a given unit of work.
#pragma once

#include "tv_device.cuh"

namespace tv {

struct ChunkView {
    const int32_t* q_start;   // [B + 1]
    const int32_t* prefix;    // [B]
    const int32_t* table;     // [B][max_blocks]
    int T, B, max_blocks, bs, num_blocks;
};

// Whether q_start is non-decreasing within [0, T].  Called by every thread of
// the CTA; contains a barrier.
__device__ __forceinline__ bool chunk_starts_ok(const ChunkView& c) {
    bool ok = true;
    for (int b = threadIdx.x; b < c.B; b += blockDim.x) {
        const int s = c.q_start[b], e = c.q_start[b + 1];
        ok = ok && s >= 0 && s <= e && e <= c.T;
    }
    return __syncthreads_and(ok ? 1 : 0) != 0;
}

// Positions stay below this, so that a tile past the last key still has an int32 position.
constexpr int64_t CHUNK_POS_MAX = 0x7fffffffll - 1023;

// Length part of a sequence's check: its P + n positions fit the block table.
__device__ __forceinline__ bool chunk_shape_ok(const ChunkView& c, int P, int n) {
    return P >= 0 && (int64_t)P + n <= min((int64_t)c.max_blocks * c.bs, CHUNK_POS_MAX);
}

// First key that some row of a sequence attends to (window <= 0: no window).
__device__ __forceinline__ int chunk_first_key(int P, int window) {
    return (window > 0 && P >= window) ? P - window + 1 : 0;
}

// This thread's share of the check of the blocks that hold positions lo .. hi-1
// of sequence b (threads `id` of `count`); lo and hi inside the block table.
__device__ __forceinline__ bool chunk_blocks_ok(const ChunkView& c, int b, int64_t lo, int64_t hi,
                                                int id, int count) {
    const int32_t* row = c.table + (int64_t)b * c.max_blocks;
    const int j1 = (int)((hi + c.bs - 1) / c.bs);
    bool ok = true;
    // independent loads, four in flight
    for (int j = (int)(lo / c.bs) + id; j < j1; j += 4 * count) {
        int blk[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) blk[u] = (j + u * count < j1) ? row[j + u * count] : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) ok = ok && blk[u] >= 0 && blk[u] < c.num_blocks;
    }
    return ok;
}

// Finds the sequence that holds unit x = where(total) when a sequence with prefix
// P and n rows has cost(P, n) units and the sequences are laid end to end; and
// checks q_start.  Called by every thread of the CTA (THREADS of them); each
// thread sums a contiguous run of sequences, then the block scans.  tmp: shared
// memory of its own for the call.
struct ChunkPlace {
    int64_t total;  // units of all sequences
    int64_t base;   // first unit of sequence b
    int b;          // B when x >= total, or when q_start is not valid
    bool valid;     // q_start is non-decreasing within [0, T]
    int row, n, P;  // sequence b's first row, rows, prefix
};

template <int THREADS>
struct ChunkLocateTmp {
    int64_t warp_sum[THREADS / 32];
    int64_t found_base;
    int found_b;
};

template <int THREADS, class Where, class Cost>
__device__ __forceinline__ ChunkPlace chunk_locate(ChunkLocateTmp<THREADS>* tmp, const ChunkView& c,
                                                   Where where, Cost cost) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (c.B + THREADS - 1) / THREADS;
    const int b0 = min(c.B, tid * per), b1 = min(c.B, b0 + per);
    int64_t s = 0;
    bool ok = true;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const int lo = c.q_start[b], hi = c.q_start[b + 1], P = c.prefix[b];
        ok = ok && lo >= 0 && lo <= hi && hi <= c.T;
        s += cost(P, hi - lo);
    }
    int64_t incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) tmp->warp_sum[warp] = incl;
    if (tid == 0) tmp->found_b = c.B;
    ChunkPlace r;
    r.valid = __syncthreads_and(ok ? 1 : 0) != 0;
    int64_t before = 0;
    r.total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += tmp->warp_sum[w];
        r.total += tmp->warp_sum[w];
    }
    const int64_t x = where(r.total);
    int64_t at = before + incl - s;
    if (r.valid && x >= at && x < at + s) {
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const int64_t u = cost(c.prefix[b], c.q_start[b + 1] - c.q_start[b]);
            if (x < at + u) {
                tmp->found_b = b;
                tmp->found_base = at;
                break;
            }
            at += u;
        }
    }
    __syncthreads();
    r.b = tmp->found_b;
    r.base = r.b < c.B ? tmp->found_base : r.total;
    r.row = r.n = r.P = 0;
    if (r.b < c.B) {
        r.row = c.q_start[r.b];
        r.n = c.q_start[r.b + 1] - r.row;
        r.P = c.prefix[r.b];
    }
    return r;
}

// The same for at most 32 sequences, by each warp for itself: one round trip to memory
// and no barrier, for calls whose start is most of their time.
template <class Where, class Cost>
__device__ __forceinline__ ChunkPlace chunk_locate_warp(const ChunkView& c, Where where, Cost cost) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = 0, P = 0;
    bool ok = true;
    if (lane < c.B) {
        const int hi = c.q_start[lane + 1];
        lo = c.q_start[lane];
        P = c.prefix[lane];
        n = hi - lo;
        ok = lo >= 0 && lo <= hi && hi <= c.T;
    }
    ChunkPlace r;
    r.valid = __all_sync(0xffffffffu, ok);
    const int64_t s = lane < c.B && ok ? cost(P, n) : 0;
    int64_t incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    r.total = __shfl_sync(0xffffffffu, incl, 31);
    const int64_t x = where(r.total), at = incl - s;
    const uint32_t here = __ballot_sync(0xffffffffu, r.valid && x >= at && x < incl);
    const int b = here ? __ffs(here) - 1 : 0;
    r.b = here ? b : c.B;
    r.base = __shfl_sync(0xffffffffu, at, b);
    r.row = __shfl_sync(0xffffffffu, lo, b);
    r.n = __shfl_sync(0xffffffffu, n, b);
    r.P = __shfl_sync(0xffffffffu, P, b);
    return r;
}

}  // namespace tv
