// chunk_kv_append: a chunk's keys and values into the paged cache, queries and
// keys rotated by their positions; and rope_table_init.
//
// A rotation moves two columns (x, y) of a pair to (x cos a - y sin a, y cos a +
// x sin a), a = position times the pair's frequency.  The frequency is kept as
// turns per position in 2^-64 of a turn, so position * turn modulo 2^64 is the
// angle's fraction of a turn without rounding (a float32 angle of position
// 100,000 would be off by 0.004 radians); sincospi then needs no range
// reduction, and everything behind it is float32 with one rounding to the
// output type.
//
// Bound by memory: every row is read once and written once.  A CTA takes up to 16
// consecutive rows, a warp finding and checking each; the (cos, sin) of its rows' pairs
// are computed once in shared memory and shared by all heads.  A thread's unit is 16
// bytes of a row (half layout: the two 16-byte vectors that hold a pair's columns), and
// it takes the same unit of several rows, so that finding it is paid once and the rows'
// loads are in flight together.
// Measured (bfloat16): 9,164 rows of 28 + 2 x 4 heads of 128, 169 MB, 40.6 us, where a
// plain copy of those bytes takes 33 (prefetching the rows to L2 first 5 % more, four rows in
// flight per thread 25 %); 832 rows of 32 + 2 x 8 heads 7.8 us captured, most of it the three
// round trips to a row's slot, and 12.7 from the host, which takes that long.  Float32, 6,677
// rows of 32 + 2 x 8 heads, 328 MB: 62 us.  With positions of their own every CTA of a sequence
// reads all of the sequence's: 8,000 rows of 32 + 2 x 8 heads in one, 197 MB, 54 us; 40,000 rows
// of 8 + 2 x 2, 246 MB, the check in a kernel before, 113 us.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "tv_chunk.cuh"
#include "tv_internal.h"

namespace tv {

namespace {

constexpr int CA_THREADS = 256;
constexpr int CA_TT_MAX = 16;  // rows per CTA
constexpr int CA_PER_SM = 4;   // CTAs that an SM holds

struct CaParams {
    ChunkView c;
    const uint8_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, qo_stride;  // bytes
    const int32_t* positions;                         // nullable
    uint8_t *q_out, *k_cache, *v_cache;
    int32_t* status;
    int Hq, Hkv, d, TT;
    bool checked;  // status holds the sequences' checks already
};

// Checks of sequence b: its positions have blocks, its rotary positions are not
// negative.  Threads `id` of `count`, to be combined.
__device__ __forceinline__ bool ca_seq_ok(const CaParams& p, int b, int P, int s, int n, int id,
                                          int count) {
    if (!chunk_shape_ok(p.c, P, n)) return false;
    bool ok = true;
    if (n > 0) ok = chunk_blocks_ok(p.c, b, P, (int64_t)P + n, id, count);
    if (p.positions)
        for (int i = id; i < n; i += count) ok = ok && p.positions[s + i] >= 0;
    return ok;
}

// One CTA per sequence: its status.
__global__ void __launch_bounds__(CA_THREADS) chunk_check_kernel(CaParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const bool valid = chunk_starts_ok(p.c);
    for (int b = blockIdx.x; b < p.c.B; b += gridDim.x) {
        bool ok = valid;
        if (ok) {
            const int s = p.c.q_start[b], n = p.c.q_start[b + 1] - s;
            ok = ca_seq_ok(p, b, p.c.prefix[b], s, n, threadIdx.x, CA_THREADS);
        }
        ok = __syncthreads_and(ok ? 1 : 0) != 0;
        if (threadIdx.x == 0) p.status[b] = ok ? TV_OK : TV_ERR_OUT_OF_RANGE;
    }
}

// VE elements per 16-byte vector.
template <typename E>
struct Vec {
    static constexpr int VE = 16 / (int)sizeof(E);
    float f[VE];
};
__device__ __forceinline__ void unpack(const uint4& u, Vec<float>& x) {
    const float* f = reinterpret_cast<const float*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) x.f[i] = f[i];
}
__device__ __forceinline__ void unpack(const uint4& u, Vec<__nv_bfloat16>& x) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __bfloat1622float2(h[i]);
        x.f[2 * i] = t.x;
        x.f[2 * i + 1] = t.y;
    }
}
__device__ __forceinline__ uint4 pack(const Vec<float>& x) {
    uint4 u;
    float* f = reinterpret_cast<float*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = x.f[i];
    return u;
}
__device__ __forceinline__ uint4 pack(const Vec<__nv_bfloat16>& x) {
    uint4 u;
    u.x = pack_bf16x2(x.f[0], x.f[1]);
    u.y = pack_bf16x2(x.f[2], x.f[3]);
    u.z = pack_bf16x2(x.f[4], x.f[5]);
    u.w = pack_bf16x2(x.f[6], x.f[7]);
    return u;
}

template <typename E>
__global__ void __launch_bounds__(CA_THREADS, CA_PER_SM)
chunk_append_kernel(const CaParams p, const __grid_constant__ tv_rope_table rope) {
    constexpr int VE = Vec<E>::VE;
    extern __shared__ __align__(16) float2 cs[];      // (cos, sin), see cs_at
    __shared__ int64_t slot[CA_TT_MAX];               // first row of the slot's head 0, or -1
    __shared__ int32_t pos[CA_TT_MAX];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const int t0 = blockIdx.x * p.TT, tn = min(p.TT, p.c.T - t0);
    // q_start is checked as a whole; whoever reads a sequence that holds rows of this CTA
    // leaves it with them
    __shared__ int4 owner[CA_TT_MAX];                 // sequence, its first row, rows, prefix
    if (tid < CA_TT_MAX) owner[tid] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    bool valid = true;
    for (int b = tid; b < p.c.B; b += CA_THREADS) {
        const int s = p.c.q_start[b], e = p.c.q_start[b + 1], P = p.c.prefix[b];
        valid = valid && s >= 0 && s <= e && e <= p.c.T;
        for (int t = max(s, t0); t < min(e, t0 + tn); ++t) owner[t - t0] = make_int4(b, s, e - s, P);
    }
    valid = __syncthreads_and(valid ? 1 : 0) != 0;
    if (!p.checked && blockIdx.x == 0) {
        // sequences without rows (and a bad q_start) have no CTA of their own
        for (int b = tid; b < p.c.B; b += CA_THREADS)
            if (!valid || p.c.q_start[b] == p.c.q_start[b + 1])
                p.status[b] = (valid && chunk_shape_ok(p.c, p.c.prefix[b], 0)) ? TV_OK
                                                                               : TV_ERR_OUT_OF_RANGE;
    }
    if (!valid) return;
    // sequences that change within the CTA's rows
    int changes = 0;
    for (int r = 1; r < tn; ++r) changes += owner[r].x != owner[r - 1].x;
    // one sequence, or two: its blocks are checked by every thread at once
    bool whole = false, ok_first = true, ok_last = true;
    if (!p.checked && changes <= 1) {
        whole = true;
        const int4 a = owner[0], z = owner[tn - 1];
        if (a.x >= 0) ok_first = ca_seq_ok(p, a.x, a.w, a.y, a.z, tid, CA_THREADS);
        if (z.x >= 0 && z.x != a.x) ok_last = ca_seq_ok(p, z.x, z.w, z.y, z.z, tid, CA_THREADS);
        ok_first = __syncthreads_and(ok_first ? 1 : 0) != 0;
        ok_last = changes == 0 ? ok_first : __syncthreads_and(ok_last ? 1 : 0) != 0;
    }
    for (int r = warp; r < tn; r += CA_THREADS / 32) {
        // a warp per row: its sequence's check, its slot
        const int t = t0 + r, b = owner[r].x, s = owner[r].y, n = owner[r].z, P = owner[r].w;
        int64_t at = -1;
        if (b >= 0) {
            bool ok;
            if (p.checked) {
                ok = p.status[b] == TV_OK;
            } else {
                ok = whole ? (b == owner[0].x ? ok_first : ok_last)
                           : __all_sync(0xffffffffu, ca_seq_ok(p, b, P, s, n, lane, 32));
                if (lane == 0 && t == s) p.status[b] = ok ? TV_OK : TV_ERR_OUT_OF_RANGE;
            }
            if (ok) {
                const int64_t l = (int64_t)P + (t - s);
                const int64_t blk = p.c.table[(int64_t)b * p.c.max_blocks + l / p.c.bs];
                at = blk * p.Hkv * p.c.bs + l % p.c.bs;
                if (lane == 0) pos[r] = p.positions ? p.positions[t] : (int)l;
            }
        }
        if (lane == 0) slot[r] = at;
    }
    __syncthreads();
    const int half = rope.dim / 2;
    const int vec = p.d / VE;                                   // vectors per head row
    const int rv = rope.dim / VE;                               // rotated vectors
    const int ru = rope.interleaved ? rv : rv / 2;              // rotated units
    const int per = rope.interleaved ? VE / 2 : VE;             // pairs of a unit
    // Pair x of unit c of row r: the 16 bytes of two pairs lie beside the next unit's, so
    // that lanes with consecutive units read consecutive banks.
    auto cs_at = [&](int r, int c, int x) -> int { return ((r * (per / 2) + x / 2) * ru + c) * 2 + (x & 1); };
    for (int e = tid; e < tn * half; e += CA_THREADS) {
        const int r = e / half, j = e - r * half;
        if (slot[r] < 0) continue;
        // the low 64 bits of position * turn: a fraction of a turn in [-1/2, 1/2)
        const int64_t a = (int64_t)((uint64_t)(uint32_t)pos[r] * rope.turn[j]);
        float sn, co;
        sincospif(__ll2float_rn(a) * 1.0842021724855044e-19f, &sn, &co);  // 2^-63: half turns
        cs[cs_at(r, j / per, j % per)] = make_float2(co * rope.amplitude, sn * rope.amplitude);
    }
    __syncthreads();
    // units of a row: for each query and key head its rotated vectors (half layout:
    // pairs of them) and its copied ones, then the value vectors
    const int hu = ru + vec - rv;                               // units per rotated head
    const int uq = (p.q ? p.Hq : 0) * hu, uk = uq + p.Hkv * hu, ut = uk + p.Hkv * vec;
    // few units: the threads also share out the rows
    const int share = max(1, min(p.TT, CA_THREADS / ut)), mine = tid / ut;
    const int r_first = share > 1 ? mine : 0;
    if (share > 1 && mine >= share) return;
    for (int e = share > 1 ? tid - mine * ut : tid; e < ut; e += share > 1 ? ut : CA_THREADS) {
        // the unit's first vector in its head, and where the head is: in the source row, and in
        // the output row or (so many cache rows on) in the slot
        int h, c;
        bool copy = true, cache = true;
        const uint8_t* src = p.v;
        uint8_t* dst = p.v_cache;
        int64_t src_step = p.v_stride, dst_step = 0;
        if (e >= uk) {
            h = (e - uk) / vec;
            c = e - uk - h * vec;
        } else {
            cache = e >= uq;
            h = (cache ? e - uq : e) / hu;
            c = (cache ? e - uq : e) - h * hu;
            copy = c >= ru;
            src = cache ? p.k : p.q;
            dst = cache ? p.k_cache : p.q_out;
            src_step = cache ? p.k_stride : p.q_stride;
            dst_step = p.qo_stride;
            if (copy) c += rv - ru;
        }
        src += (int64_t)t0 * src_step + ((int64_t)h * vec + c) * 16;
        dst += cache ? ((int64_t)h * p.c.bs * vec + c) * 16 : (int64_t)t0 * dst_step + ((int64_t)h * vec + c) * 16;
        const bool two = !copy && !rope.interleaved;            // two vectors
        // the unit of up to ROWS rows at a time, their loads in flight together
        constexpr int ROWS = 2;
        for (int rb = r_first; rb < tn; rb += ROWS * share) {
            uint4 x[ROWS], y[ROWS];
            int64_t at[ROWS];
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                const int r = rb + k * share;
                at[k] = r < tn ? slot[r] : -1;
                if (at[k] < 0) continue;
                x[k] = __ldcs(reinterpret_cast<const uint4*>(src + r * src_step));
                if (two) y[k] = __ldcs(reinterpret_cast<const uint4*>(src + r * src_step + ru * 16));
            }
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                if (at[k] < 0) continue;
                const int r = rb + k * share;
                uint8_t* to = dst + (cache ? at[k] * vec * 16 : r * dst_step);
                if (!copy) {
                    Vec<E> a;
                    unpack(x[k], a);
                    if (two) {
                        Vec<E> b;
                        unpack(y[k], b);
#pragma unroll
                        for (int i = 0; i < VE; i += 2) {
                            const float4 w = *reinterpret_cast<const float4*>(cs + cs_at(r, c, i));
                            const float a0 = a.f[i], b0 = b.f[i], a1 = a.f[i + 1], b1 = b.f[i + 1];
                            a.f[i] = a0 * w.x - b0 * w.y;
                            b.f[i] = b0 * w.x + a0 * w.y;
                            a.f[i + 1] = a1 * w.z - b1 * w.w;
                            b.f[i + 1] = b1 * w.z + a1 * w.w;
                        }
                        *reinterpret_cast<uint4*>(to + ru * 16) = pack(b);
                    } else {
#pragma unroll
                        for (int i = 0; i < VE; i += 4) {
                            const float4 w = *reinterpret_cast<const float4*>(cs + cs_at(r, c, i / 2));
                            const float a0 = a.f[i], b0 = a.f[i + 1], a1 = a.f[i + 2], b1 = a.f[i + 3];
                            a.f[i] = a0 * w.x - b0 * w.y;
                            a.f[i + 1] = b0 * w.x + a0 * w.y;
                            a.f[i + 2] = a1 * w.z - b1 * w.w;
                            a.f[i + 3] = b1 * w.z + a1 * w.w;
                        }
                    }
                    x[k] = pack(a);
                }
                *reinterpret_cast<uint4*>(to) = x[k];
            }
        }
    }
}

}  // namespace

tv_status launch_chunk_append(const ChunkAppendArgs& a) {
    CaParams p{};
    p.c = ChunkView{a.q_start, a.prefix_lens, a.block_table, a.T, a.B, a.max_blocks, a.bs, a.num_blocks};
    p.q = static_cast<const uint8_t*>(a.q);
    p.k = static_cast<const uint8_t*>(a.k);
    p.v = static_cast<const uint8_t*>(a.v);
    p.q_stride = a.q_stride * a.elem;
    p.k_stride = a.k_stride * a.elem;
    p.v_stride = a.v_stride * a.elem;
    p.qo_stride = a.q_out_stride * a.elem;
    p.positions = a.positions;
    p.q_out = static_cast<uint8_t*>(a.q_out);
    p.k_cache = static_cast<uint8_t*>(a.k_cache);
    p.v_cache = static_cast<uint8_t*>(a.v_cache);
    p.status = a.status;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.d = a.d;
    // rows per CTA: one wave of CTAs while they are at most CA_TT_MAX (their start, two round
    // trips to memory, is not repeated then)
    const int wave = CA_PER_SM * device_sm_count();
    p.TT = std::min(CA_TT_MAX, std::max(1, (a.T + wave - 1) / wave));
    const unsigned grid = (unsigned)((a.T + p.TT - 1) / p.TT);
    // Every CTA of a sequence checks all of the sequence's blocks, so that a bad one
    // is left untouched; for long inputs that would be read too often, and a
    // kernel of one CTA per sequence does it first.
    p.checked = a.T > 32768 || grid == 0;
    if (p.checked) {
        LaunchCfg lc(dim3((unsigned)std::min(a.B, 65535)), dim3(CA_THREADS), 0, a.stream);
        if (cudaLaunchKernelEx(&lc.cfg, chunk_check_kernel, p) != cudaSuccess) return TV_ERR_CUDA;
        if (grid == 0) return TV_OK;
    }
    tv_rope_table none{};
    const tv_rope_table& rope = a.rope ? *a.rope : none;
    LaunchCfg lc(dim3(grid), dim3(CA_THREADS), (size_t)p.TT * (rope.dim / 2) * sizeof(float2), a.stream);
    const cudaError_t e = a.elem == 4
        ? cudaLaunchKernelEx(&lc.cfg, chunk_append_kernel<float>, p, rope)
        : cudaLaunchKernelEx(&lc.cfg, chunk_append_kernel<__nv_bfloat16>, p, rope);
    return e == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

tv_status make_rope_table(tv_rope_table* t, int dim, int interleaved, double theta,
                          tv_rope_scaling scaling, double factor, double original_len, double low,
                          double high, double amplitude) {
    const double two_pi = 6.283185307179586;
    if (!t || dim < 2 || dim > TV_ROPE_MAX_DIM || (dim & 1) || !isfinite(theta) || theta <= 1.0)
        return TV_ERR_INVALID_ARG;
    if (scaling != TV_ROPE_NONE && scaling != TV_ROPE_LINEAR && scaling != TV_ROPE_BANDS &&
        scaling != TV_ROPE_RAMP)
        return TV_ERR_INVALID_ARG;
    if (scaling != TV_ROPE_NONE && !(isfinite(factor) && factor >= 1.0)) return TV_ERR_INVALID_ARG;
    if (!isfinite(amplitude)) return TV_ERR_INVALID_ARG;
    if (!(low > 0.0)) low = 1.0;
    if (!(high > 0.0)) high = scaling == TV_ROPE_RAMP ? 32.0 : 4.0;
    if (scaling == TV_ROPE_BANDS || scaling == TV_ROPE_RAMP) {
        if (!isfinite(original_len) || original_len < 1.0 || !isfinite(low) || !isfinite(high) ||
            high <= low)
            return TV_ERR_INVALID_ARG;
    }
    double a = 0.0, z = 0.0;
    if (scaling == TV_ROPE_RAMP) {
        auto edge = [&](double n) { return dim * log(original_len / (two_pi * n)) / (2.0 * log(theta)); };
        a = fmax(0.0, floor(edge(high)));
        z = fmin((double)(dim - 1), ceil(edge(low)));
    }
    memset(t, 0, sizeof(*t));
    t->dim = dim;
    t->interleaved = interleaved ? 1 : 0;
    const double amp = amplitude > 0.0 ? amplitude : (scaling == TV_ROPE_RAMP ? 0.1 * log(factor) + 1.0 : 1.0);
    t->amplitude = (float)amp;
    t->amplitude_rest = isfinite(t->amplitude) ? (float)(amp - t->amplitude) : 0.f;
    for (int j = 0; j < dim / 2; ++j) {
        double f = pow(theta, -2.0 * j / dim);
        if (scaling == TV_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == TV_ROPE_BANDS) {
            const double k = fmin(1.0, fmax(0.0, (original_len * f / two_pi - low) / (high - low)));
            f = f * (k + (1.0 - k) / factor);
        } else if (scaling == TV_ROPE_RAMP) {
            const double s = fmin(1.0, fmax(0.0, (j - a) / fmax(z - a, 0.001)));
            f = f * (1.0 - s) + f / factor * s;
        }
        t->turn[j] = (uint64_t)(f / two_pi * 18446744073709551616.0);  // below 2^62: f <= 1
    }
    return TV_OK;
}

}  // namespace tv
