// chunk_kv_append_q8: a chunk's keys and values, rotated and quantised, into an 8-bit cache.
//
// A block of a kv head has one scale, the smallest power of two with which its largest value
// fits, so the new rows of a block are gone through before any is written: a CTA takes the new
// rows of one block (of a sequence), a warp 16 rows of one head at a time, all of them in
// registers, so that blocks of 16 tokens are read once (longer ones twice, the second time from
// L2).  A lane holds 16-byte pieces of rows; the partner of a rotated column is in the same
// row, so in the same warp, and comes by a shuffle.  The (cos, sin) of a row's pairs are
// computed once per CTA and shared by its heads.  Where the block holds earlier tokens and its
// scale grows, their codes are rounded again.
// Few blocks: their heads are split over several CTAs, so that the GPU is full.
#include <cuda_bf16.h>

#include <algorithm>

#include "tv_chunk.cuh"
#include "tv_fp8.cuh"
#include "tv_internal.h"

namespace tv {

namespace {

constexpr int AQ_THREADS = 256;
constexpr int AQ_WARPS = AQ_THREADS / 32;
constexpr int AQ_PER_SM = 2;   // CTAs that an SM holds
constexpr int AQ_ROWS = 16;    // rows that a warp holds of a head

struct AqParams {
    ChunkView c;
    const uint8_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, qo_stride;  // bytes
    const int32_t* positions;                         // nullable
    uint8_t *q_out, *k_cache, *v_cache;
    float *k_scale, *v_scale;
    int32_t* status;
    int Hq, Hkv;
    int splits;    // CTAs per block
    bool checked;  // status holds the sequences' checks already
};

// Checks of sequence b, as chunk_kv_append: threads `id` of `count`, to be combined.
__device__ __forceinline__ bool aq_seq_ok(const AqParams& p, int b, int P, int s, int n, int id, int count) {
    if (!chunk_shape_ok(p.c, P, n)) return false;
    bool ok = true;
    if (n > 0) ok = chunk_blocks_ok(p.c, b, P, (int64_t)P + n, id, count);
    if (p.positions)
        for (int i = id; i < n; i += count) ok = ok && p.positions[s + i] >= 0;
    return ok;
}

// One CTA per sequence: its status.
__global__ void __launch_bounds__(AQ_THREADS) append_q8_check_kernel(const __grid_constant__ AqParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const bool valid = chunk_starts_ok(p.c);
    for (int b = blockIdx.x; b < p.c.B; b += gridDim.x) {
        bool ok = valid;
        if (ok) {
            const int s = p.c.q_start[b], n = p.c.q_start[b + 1] - s;
            ok = aq_seq_ok(p, b, p.c.prefix[b], s, n, threadIdx.x, AQ_THREADS);
        }
        ok = __syncthreads_and(ok ? 1 : 0) != 0;
        if (threadIdx.x == 0) p.status[b] = ok ? TV_OK : TV_ERR_OUT_OF_RANGE;
    }
}

__device__ __forceinline__ void bf16_floats(const uint4& u, float (&f)[8]) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __bfloat1622float2(h[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}

template <int D>
__global__ void __launch_bounds__(AQ_THREADS, AQ_PER_SM)
append_q8_kernel(const __grid_constant__ AqParams p, const __grid_constant__ tv_rope_table rope) {
    constexpr int VEC = D / 8;           // 16-byte pieces of a row of bfloat16
    constexpr int RPL = 32 / VEC;        // rows that a warp loads at once
    constexpr int NL = AQ_ROWS / RPL;
    extern __shared__ __align__(16) uint8_t aq_smem[];
    float2* cs = reinterpret_cast<float2*>(aq_smem);                        // (cos, sin), see cs_at
    float* top = reinterpret_cast<float*>(cs + AQ_ROWS * (rope.dim / 2));   // [2 Hkv] largest value, then scale
    __shared__ ChunkLocateTmp<AQ_THREADS> tmp;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, bs = p.c.bs;
    pdl_launch_dependents();
    pdl_wait();
    // ---- the block: a sequence's new rows touch the blocks P / bs .. (P + n - 1) / bs
    const int cell = blockIdx.x / p.splits, split = blockIdx.x - cell * p.splits;
    auto cells = [&](int P, int n) -> int64_t {
        return n > 0 && P >= 0 ? (int64_t)(((int64_t)P + n - 1) / bs) - P / bs + 1 : 0;
    };
    auto where = [&](int64_t) { return (int64_t)cell; };
    const ChunkPlace at = p.c.B <= 32 ? chunk_locate_warp(p.c, where, cells)
                                      : chunk_locate<AQ_THREADS>(&tmp, p.c, where, cells);
    if (!p.checked && blockIdx.x == 0)
        // sequences without blocks (and a bad q_start) have no CTA of their own
        for (int b = tid; b < p.c.B; b += AQ_THREADS)
            if (!at.valid || cells(p.c.prefix[b], p.c.q_start[b + 1] - p.c.q_start[b]) == 0)
                p.status[b] = (at.valid && p.c.q_start[b] == p.c.q_start[b + 1] && chunk_shape_ok(p.c, p.c.prefix[b], 0))
                                  ? TV_OK : TV_ERR_OUT_OF_RANGE;
    if (at.b >= p.c.B) return;
    const int P = at.P, n = at.n, lb = P / bs + (int)(cell - at.base);
    bool ok;
    if (p.checked) {
        ok = p.status[at.b] == TV_OK;
    } else {
        ok = __syncthreads_and(aq_seq_ok(p, at.b, P, at.row, n, tid, AQ_THREADS) ? 1 : 0) != 0;
        if (cell == at.base && split == 0 && tid == 0) p.status[at.b] = ok ? TV_OK : TV_ERR_OUT_OF_RANGE;
    }
    if (!ok) return;
    const int64_t blk = p.c.table[(int64_t)at.b * p.c.max_blocks + lb];
    const int64_t first = (int64_t)lb * bs;                       // position of the block's row 0
    const int r0 = (int)max((int64_t)P - first, (int64_t)0);      // new rows of the block: r0 .. r1 - 1
    const int r1 = (int)min((int64_t)P + n - first, (int64_t)bs);
    const int64_t row0 = at.row + first - P;                      // the input's row of the block's row 0
    // ---- this CTA's units: key heads, value heads, query heads
    const int units = 2 * p.Hkv + (p.q ? p.Hq : 0);
    const int u_lo = (int)((int64_t)units * split / p.splits), u_hi = (int)((int64_t)units * (split + 1) / p.splits);
    const int half = rope.dim / 2, rv = rope.dim / 8;             // rotated pairs, rotated pieces
    // A piece's eight columns: 8 pairs' first or second columns, or (interleaved) 4 pairs.  The 16
    // bytes of two pairs lie beside the next piece's, so that lanes read consecutive banks.
    const int per = rope.interleaved ? 4 : 8, ru = half / per;
    auto cs_at = [&](int r, int c, int x) -> int { return ((r * (per / 2) + x / 2) * ru + c) * 2 + (x & 1); };
    const int c = lane % VEC, sub = lane / VEC;                   // the lane's piece, its row of RPL
    const bool turned = c < rv;
    const int hv = rv / 2;                                        // half layout: the partner's distance
    const bool second = !rope.interleaved && c >= hv;
    const int partner = lane - c + (turned ? (second ? c - hv : c + hv) : c);
    const int cc = rope.interleaved ? c : (second ? c - hv : c);  // its pairs in cs
    const int ch0 = r0 / AQ_ROWS, ch1 = (r1 + AQ_ROWS - 1) / AQ_ROWS;
    const bool once = ch1 - ch0 == 1;
    if (!once)
        for (int u = tid; u < 2 * p.Hkv; u += AQ_THREADS) top[u] = 0.f;
#pragma unroll 1
    for (int pass = once ? 1 : 0; pass < 2; ++pass)
#pragma unroll 1
        for (int ch = ch0; ch < ch1; ++ch) {
            const int lo = max(r0, ch * AQ_ROWS), hi = min(r1, (ch + 1) * AQ_ROWS);
            __syncthreads();
            if (u_lo < p.Hkv || u_hi > 2 * p.Hkv)
                for (int e = tid; e < (hi - lo) * half; e += AQ_THREADS) {
                    const int r = lo + e / half, j = e % half;
                    const int64_t pos = p.positions ? p.positions[row0 + r] : first + r;
                    // the low 64 bits of position * turn: a fraction of a turn in [-1/2, 1/2)
                    const int64_t a = (int64_t)((uint64_t)(uint32_t)pos * rope.turn[j]);
                    float sn, co;
                    sincospif(__ll2float_rn(a) * 1.0842021724855044e-19f, &sn, &co);  // 2^-63: half turns
                    cs[cs_at(r - ch * AQ_ROWS, j / per, j % per)] = make_float2(co * rope.amplitude, sn * rope.amplitude);
                }
            __syncthreads();
#pragma unroll 1
            for (int u = u_lo + warp; u < u_hi; u += AQ_WARPS) {
                const int kind = u < p.Hkv ? 0 : (u < 2 * p.Hkv ? 1 : 2);     // key, value, query
                if (pass == 0 && kind == 2) continue;
                const int h = u - (kind == 0 ? 0 : kind == 1 ? p.Hkv : 2 * p.Hkv);
                const uint8_t* src = kind == 0 ? p.k : kind == 1 ? p.v : p.q;
                const int64_t step = kind == 0 ? p.k_stride : kind == 1 ? p.v_stride : p.q_stride;
                uint4 x[NL];
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const int r = ch * AQ_ROWS + i * RPL + sub;
                    x[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (r >= lo && r < hi)
                        x[i] = *reinterpret_cast<const uint4*>(src + (row0 + r) * step + (int64_t)(h * VEC + c) * 16);
                }
                // row i of the lane, rotated: products and sums in float32, each rounded
                auto rotated = [&](int i, float (&f)[8]) {
                    bf16_floats(x[i], f);
                    if (kind == 1 || half == 0) return;
                    float g[8];
                    if (rope.interleaved) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) g[e] = f[e ^ 1];
                    } else {
                        uint4 y;
                        y.x = __shfl_sync(0xffffffffu, x[i].x, partner);
                        y.y = __shfl_sync(0xffffffffu, x[i].y, partner);
                        y.z = __shfl_sync(0xffffffffu, x[i].z, partner);
                        y.w = __shfl_sync(0xffffffffu, x[i].w, partner);
                        bf16_floats(y, g);
                    }
                    const int r = i * RPL + sub;
                    if (!turned || ch * AQ_ROWS + r < lo || ch * AQ_ROWS + r >= hi) return;
                    if (rope.interleaved) {
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float4 w = *reinterpret_cast<const float4*>(cs + cs_at(r, cc, e));
                            f[2 * e] = __fsub_rn(__fmul_rn(f[2 * e], w.x), __fmul_rn(g[2 * e], w.y));
                            f[2 * e + 1] = __fadd_rn(__fmul_rn(f[2 * e + 1], w.x), __fmul_rn(g[2 * e + 1], w.y));
                            f[2 * e + 2] = __fsub_rn(__fmul_rn(f[2 * e + 2], w.z), __fmul_rn(g[2 * e + 2], w.w));
                            f[2 * e + 3] = __fadd_rn(__fmul_rn(f[2 * e + 3], w.z), __fmul_rn(g[2 * e + 3], w.w));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const float4 w = *reinterpret_cast<const float4*>(cs + cs_at(r, cc, e));
                            const float s0 = second ? w.y : -w.y, s1 = second ? w.w : -w.w;
                            f[e] = __fadd_rn(__fmul_rn(f[e], w.x), __fmul_rn(g[e], s0));
                            f[e + 1] = __fadd_rn(__fmul_rn(f[e + 1], w.z), __fmul_rn(g[e + 1], s1));
                        }
                    }
                };
                if (kind == 2) {
#pragma unroll
                    for (int i = 0; i < NL; ++i) {
                        float f[8];
                        rotated(i, f);
                        const int r = ch * AQ_ROWS + i * RPL + sub;
                        uint4 y = x[i];
                        if (turned)
                            y = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                           pack_bf16x2(f[6], f[7]));
                        if (r >= lo && r < hi)
                            *reinterpret_cast<uint4*>(p.q_out + (row0 + r) * p.qo_stride + (int64_t)(h * VEC + c) * 16) = y;
                    }
                    continue;
                }
                float* scale = (kind == 0 ? p.k_scale : p.v_scale) + blk * p.Hkv + h;
                uint8_t* codes = (kind == 0 ? p.k_cache : p.v_cache) + (blk * p.Hkv + h) * bs * D;
                if (once || pass == 0) {
                    // the largest finite value: 0 x + x is NaN for an infinite x, and a NaN is no maximum
                    float m = 0.f;
#pragma unroll
                    for (int i = 0; i < NL; ++i) {
                        float f[8];
                        rotated(i, f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(fmaf(f[e], 0.f, f[e])));
                    }
                    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
                    if (pass == 0) {
                        if (lane == 0) top[u] = fmaxf(top[u], m);
                        __syncwarp();
                        continue;
                    }
                    if (lane == 0) top[u] = m;
                }
                __syncwarp();
                float s = top[u];
                if (ch == ch0) {
                    s = scale_needed(s);
                    if (r0 > 0) {
                        // earlier tokens of the block: their codes for the larger scale
                        const float old = scale_of(exponent_byte(*scale));
                        if (old > s) s = old;
                        else if (old < s) {
                            const float by = old * scale_inverse(s);
                            for (int e = lane; e < r0 * (D / 16); e += 32) {
                                uint4 w = reinterpret_cast<uint4*>(codes)[e];
                                w.x = e4m3_scaled(w.x, by);
                                w.y = e4m3_scaled(w.y, by);
                                w.z = e4m3_scaled(w.z, by);
                                w.w = e4m3_scaled(w.w, by);
                                reinterpret_cast<uint4*>(codes)[e] = w;
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) {
                        *scale = s;
                        top[u] = s;
                    }
                    __syncwarp();
                }
                const float inv = scale_inverse(s);
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    float f[8];
                    rotated(i, f);
                    const int r = ch * AQ_ROWS + i * RPL + sub;
                    // (an infinite value becomes NaN: 0 x is)
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = fmaf(f[e], inv, f[e] * 0.f);
                    const uint2 w = make_uint2(e4m3_pair(f[0], f[1]) | e4m3_pair(f[2], f[3]) << 16,
                                               e4m3_pair(f[4], f[5]) | e4m3_pair(f[6], f[7]) << 16);
                    if (r >= lo && r < hi) *reinterpret_cast<uint2*>(codes + (int64_t)r * D + c * 8) = w;
                }
            }
        }
}

}  // namespace

tv_status launch_chunk_append_q8(const ChunkAppendArgs& a) {
    AqParams p{};
    p.c = ChunkView{a.q_start, a.prefix_lens, a.block_table, a.T, a.B, a.max_blocks, a.bs, a.num_blocks};
    p.q = static_cast<const uint8_t*>(a.q);
    p.k = static_cast<const uint8_t*>(a.k);
    p.v = static_cast<const uint8_t*>(a.v);
    p.q_stride = a.q_stride * 2;
    p.k_stride = a.k_stride * 2;
    p.v_stride = a.v_stride * 2;
    p.qo_stride = a.q_out_stride * 2;
    p.positions = a.positions;
    p.q_out = static_cast<uint8_t*>(a.q_out);
    p.k_cache = static_cast<uint8_t*>(a.k_cache);
    p.v_cache = static_cast<uint8_t*>(a.v_cache);
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.status = a.status;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    // blocks that T rows of B sequences touch at most
    const int64_t cells = (int64_t)a.T / a.bs + 2 * (int64_t)std::min(a.T, a.B);
    // Every CTA of a sequence checks all of the sequence's blocks and positions, so that a bad one is
    // left untouched; for long inputs that would be read too often, and a kernel of one CTA per
    // sequence does it first.
    p.checked = a.T > 32768 || a.T == 0;
    if (p.checked) {
        LaunchCfg lc(dim3((unsigned)std::min(a.B, 65535)), dim3(AQ_THREADS), 0, a.stream);
        if (cudaLaunchKernelEx(&lc.cfg, append_q8_check_kernel, p) != cudaSuccess) return TV_ERR_CUDA;
        if (a.T == 0) return TV_OK;
    }
    const int units = 2 * a.Hkv + (a.q ? a.Hq : 0);
    const int64_t wave = (int64_t)AQ_PER_SM * device_sm_count();
    p.splits = (int)std::clamp<int64_t>(wave / cells, 1, (units + AQ_WARPS - 1) / AQ_WARPS);
    if (cells * p.splits > 0x7fffffff) return TV_ERR_UNSUPPORTED;
    tv_rope_table none{};
    const tv_rope_table& rope = a.rope ? *a.rope : none;
    const size_t smem = (size_t)AQ_ROWS * (rope.dim / 2) * sizeof(float2) + (size_t)2 * a.Hkv * sizeof(float);
    if (smem > 40 * 1024) return TV_ERR_UNSUPPORTED;
    LaunchCfg lc(dim3((unsigned)(cells * p.splits)), dim3(AQ_THREADS), smem, a.stream);
    const cudaError_t e = a.d == 128 ? cudaLaunchKernelEx(&lc.cfg, append_q8_kernel<128>, p, rope)
                                     : cudaLaunchKernelEx(&lc.cfg, append_q8_kernel<64>, p, rope);
    return e == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // namespace tv
