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
// Bound by memory: every row is read once and written once.  A CTA takes TT
// consecutive rows; the (cos, sin) of its TT x dim/2 pairs are computed once in
// shared memory and shared by all heads, and a thread's unit is 16 bytes of a
// row (half layout: the two 16-byte vectors that hold a pair's columns).
#include <cuda_bf16.h>
#include <math.h>

#include "tv_chunk.cuh"
#include "tv_internal.h"

namespace tv {

namespace {

constexpr int CA_THREADS = 256;
constexpr int CA_TT_MAX = 8;  // rows per CTA

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
__global__ void __launch_bounds__(CA_THREADS)
chunk_append_kernel(const CaParams p, const __grid_constant__ tv_rope_table rope) {
    constexpr int VE = Vec<E>::VE;
    extern __shared__ float2 cs[];                    // [TT][dim / 2] (cos, sin)
    __shared__ int64_t slot[CA_TT_MAX];               // first row of the slot's head 0, or -1
    __shared__ int32_t pos[CA_TT_MAX];
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    const int t0 = blockIdx.x * p.TT, tn = min(p.TT, p.c.T - t0);
    const bool valid = chunk_starts_ok(p.c);
    if (!p.checked && blockIdx.x == 0) {
        // sequences without rows (and a bad q_start) have no CTA of their own
        for (int b = tid; b < p.c.B; b += CA_THREADS)
            if (!valid || p.c.q_start[b] == p.c.q_start[b + 1])
                p.status[b] = (valid && chunk_shape_ok(p.c, p.c.prefix[b], 0)) ? TV_OK
                                                                               : TV_ERR_OUT_OF_RANGE;
    }
    if (!valid) return;
    // the rows' sequences, one after the other (one for all rows of a long chunk)
    int seq = -1, s_lo = 0, s_hi = 0, P = 0;
    bool ok = false;
    for (int r = 0; r < tn; ++r) {
        const int t = t0 + r;
        if (seq < 0 || t >= s_hi) {
            if (t < p.c.q_start[0] || t >= p.c.q_start[p.c.B]) {
                if (tid == 0) slot[r] = -1;
                continue;
            }
            int lo = 0, hi = p.c.B;  // q_start[lo] <= t < q_start[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (p.c.q_start[mid] <= t) lo = mid;
                else hi = mid;
            }
            seq = lo;
            s_lo = p.c.q_start[lo];
            s_hi = p.c.q_start[lo + 1];
            P = p.c.prefix[lo];
            if (p.checked) {
                ok = p.status[lo] == TV_OK;
            } else {
                ok = __syncthreads_and(ca_seq_ok(p, lo, P, s_lo, s_hi - s_lo, tid, CA_THREADS) ? 1 : 0) != 0;
                if (tid == 0 && t == s_lo) p.status[lo] = ok ? TV_OK : TV_ERR_OUT_OF_RANGE;
            }
        }
        if (tid == 0) {
            int64_t at = -1;
            if (ok) {
                const int64_t l = (int64_t)P + (t - s_lo);
                const int64_t blk = p.c.table[(int64_t)seq * p.c.max_blocks + l / p.c.bs];
                at = blk * p.Hkv * p.c.bs + l % p.c.bs;
                pos[r] = p.positions ? p.positions[t] : (int)l;
            }
            slot[r] = at;
        }
    }
    __syncthreads();
    const int half = rope.dim / 2;
    for (int e = tid; e < tn * half; e += CA_THREADS) {
        const int r = e / half, j = e - r * half;
        if (slot[r] < 0) continue;
        // the low 64 bits of position * turn: a fraction of a turn in [-1/2, 1/2)
        const int64_t a = (int64_t)((uint64_t)(uint32_t)pos[r] * rope.turn[j]);
        float sn, co;
        sincospif(__ll2float_rn(a) * 1.0842021724855044e-19f, &sn, &co);  // 2^-63: half turns
        cs[e] = make_float2(co * rope.amplitude, sn * rope.amplitude);
    }
    __syncthreads();
    // units of a row: for each query and key head its rotated vectors (half layout:
    // pairs of them) and its copied ones, then the value vectors
    const int vec = p.d / VE;                                   // vectors per head row
    const int rv = rope.dim / VE;                               // rotated vectors
    const int ru = rope.interleaved ? rv : rv / 2;              // rotated units
    const int hu = ru + vec - rv;                               // units per rotated head
    const int uq = (p.q ? p.Hq : 0) * hu, uk = uq + p.Hkv * hu, ut = uk + p.Hkv * vec;
    for (int e = tid; e < tn * ut; e += CA_THREADS) {
        const int r = e / ut;
        int u = e - r * ut;
        const int64_t at = slot[r];
        if (at < 0) continue;
        const int64_t t = t0 + r;
        if (u >= uk) {
            u -= uk;
            const int g = u / vec, c = u - g * vec;
            const uint4 x = *reinterpret_cast<const uint4*>(p.v + t * p.v_stride + (int64_t)u * 16);
            *reinterpret_cast<uint4*>(p.v_cache + ((at + (int64_t)g * p.c.bs) * vec + c) * 16) = x;
            continue;
        }
        const uint8_t* src;
        uint8_t* dst;
        int c;
        if (u < uq) {
            const int h = u / hu;
            c = u - h * hu;
            src = p.q + t * p.q_stride + (int64_t)h * vec * 16;
            dst = p.q_out + t * p.qo_stride + (int64_t)h * vec * 16;
        } else {
            u -= uq;
            const int g = u / hu;
            c = u - g * hu;
            src = p.k + t * p.k_stride + (int64_t)g * vec * 16;
            dst = p.k_cache + (at + (int64_t)g * p.c.bs) * vec * 16;
        }
        if (c >= ru) {
            c += rv - ru;
            *reinterpret_cast<uint4*>(dst + c * 16) = *reinterpret_cast<const uint4*>(src + c * 16);
            continue;
        }
        const float2* row = cs + r * half;
        if (rope.interleaved) {
            Vec<E> x;
            unpack(*reinterpret_cast<const uint4*>(src + c * 16), x);
#pragma unroll
            for (int i = 0; i < VE; i += 2) {
                const float2 w = row[(c * VE + i) / 2];
                const float a = x.f[i], b = x.f[i + 1];
                x.f[i] = a * w.x - b * w.y;
                x.f[i + 1] = b * w.x + a * w.y;
            }
            *reinterpret_cast<uint4*>(dst + c * 16) = pack(x);
        } else {
            Vec<E> x, y;
            const uint4 ux = *reinterpret_cast<const uint4*>(src + c * 16);
            const uint4 uy = *reinterpret_cast<const uint4*>(src + (c + ru) * 16);
            unpack(ux, x);
            unpack(uy, y);
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                const float2 w = row[c * VE + i];
                const float a = x.f[i], b = y.f[i];
                x.f[i] = a * w.x - b * w.y;
                y.f[i] = b * w.x + a * w.y;
            }
            *reinterpret_cast<uint4*>(dst + c * 16) = pack(x);
            *reinterpret_cast<uint4*>(dst + (c + ru) * 16) = pack(y);
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
    // rows per CTA: as many as still give every SM four CTAs
    p.TT = 1;
    while (p.TT < CA_TT_MAX && (int64_t)a.T >= (int64_t)8 * p.TT * device_sm_count()) p.TT *= 2;
    const unsigned grid = (unsigned)((a.T + p.TT - 1) / p.TT);
    // Every CTA of a sequence checks all of the sequence's blocks, so that a bad one
    // is left untouched; for long inputs that would be read too often, and a
    // kernel of one CTA per sequence does it first.
    p.checked = a.T > 2048 || grid == 0;
    if (p.checked) {
        LaunchCfg lc(dim3((unsigned)min(a.B, 65535)), dim3(CA_THREADS), 0, a.stream);
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
    t->amplitude = (float)(amplitude > 0.0 ? amplitude
                                           : (scaling == TV_ROPE_RAMP ? 0.1 * log(factor) + 1.0 : 1.0));
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
