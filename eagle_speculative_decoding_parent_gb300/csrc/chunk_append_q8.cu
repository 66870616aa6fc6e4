// chunk_kv_append_q8: a chunk's keys and values, rotated and quantised, into an 8-bit cache.
//
// A block of a kv head has one scale, the smallest power of two with which its largest value
// fits, so the new rows of a block are gone through before any is written: a CTA takes the new
// rows of one block (of a sequence), a warp 16 rows of one head at a time, all of them in
// registers, so that blocks of 16 tokens are read once (longer ones twice, the second time from
// L2).  A lane holds both columns of the pairs that it rotates.  The (cos, sin) of a row's pairs
// are computed once per CTA and shared by its heads.  Where the block holds earlier tokens and
// its scale grows, their codes are rounded again.
// Short calls are bound by what a CTA waits for in turn: the sequences' starts, then its blocks,
// positions and first rows together, then the block's scales beside the sines (832 rows of 32
// heads on 8, 19 MB with the queries: 10.4 us, 1.8 TB/s).  Long ones by instructions beside the stream (8192
// rows of 28 heads on 4: 32 us, 4.9 TB/s).
#include <cuda_bf16.h>

#include <algorithm>

#include "tv_chunk.cuh"
#include "tv_fp8.cuh"
#include "tv_internal.h"

namespace tv {

namespace {

constexpr int AQ_CHECK = 256;
constexpr int AQ_SM_THREADS = 512;   // that an SM holds, with 128 registers
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

// Checks of sequence b, as chunk_kv_append: threads `id` of `count`, to be combined.  Positions and
// blocks are read independently of each other.
__device__ __forceinline__ bool aq_seq_ok(const AqParams& p, int b, int P, int s, int n, int id, int count) {
    if (!chunk_shape_ok(p.c, P, n)) return false;
    int any = 0;
    if (p.positions)
        for (int i = id; i < n; i += count) any |= p.positions[s + i];
    bool ok = true;
    if (n > 0) {
        const int32_t* row = p.c.table + (int64_t)b * p.c.max_blocks;
        const uint32_t j1 = (uint32_t)(P + n - 1) / (uint32_t)p.c.bs;
        for (uint32_t j = (uint32_t)P / (uint32_t)p.c.bs + id; j <= j1; j += count) ok = ok && row[j] >= 0 && row[j] < p.c.num_blocks;
    }
    return ok && any >= 0;
}

// One CTA per sequence: its status.
__global__ void __launch_bounds__(AQ_CHECK) append_q8_check_kernel(const __grid_constant__ AqParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const bool valid = chunk_starts_ok(p.c);
    for (int b = blockIdx.x; b < p.c.B; b += gridDim.x) {
        bool ok = valid;
        if (ok) {
            const int s = p.c.q_start[b], n = p.c.q_start[b + 1] - s;
            ok = aq_seq_ok(p, b, p.c.prefix[b], s, n, threadIdx.x, AQ_CHECK);
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

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// A pair of columns by an angle: (a, b) to (a cos - b sin, b cos + a sin).
__device__ __forceinline__ void turn(float& a, float& b, float co, float sn) {
    const float x = a;
    a = fmaf(x, co, -(b * sn));
    b = fmaf(b, co, x * sn);
}

template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS, AQ_SM_THREADS / THREADS)
append_q8_kernel(const __grid_constant__ AqParams p, const __grid_constant__ tv_rope_table rope) {
    constexpr int VEC = D / 8;           // 16-byte pieces of a row of bfloat16
    constexpr int LPR = VEC / 2;         // lanes of a row, two pieces each
    constexpr int RPL = 32 / LPR;        // rows that a warp loads at once
    constexpr int NL = AQ_ROWS / RPL;
    extern __shared__ __align__(16) uint8_t aq_smem[];
    float2* cs = reinterpret_cast<float2*>(aq_smem);                        // (cos, sin), see cs_at
    float* top = reinterpret_cast<float*>(cs + AQ_ROWS * (rope.dim / 2));   // [2 Hkv] largest value, then scale
    float* was = top + 2 * p.Hkv;                                           // [2 Hkv] the block's scales before
    __shared__ ChunkLocateTmp<THREADS> tmp;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, bs = p.c.bs;
    pdl_launch_dependents();
    pdl_wait();
    // ---- the block: a sequence's new rows touch the blocks P / bs .. (P + n - 1) / bs
    const int cell = blockIdx.x / p.splits, split = blockIdx.x - cell * p.splits;
    auto cells = [&](int P, int n) -> int64_t {
        return n > 0 && P >= 0 ? (int64_t)((uint32_t)P + (uint32_t)(n - 1)) / (uint32_t)bs - (uint32_t)P / (uint32_t)bs + 1 : 0;
    };
    auto where = [&](int64_t) { return (int64_t)cell; };
    const ChunkPlace at = p.c.B <= 32 ? chunk_locate_warp(p.c, where, cells)
                                      : chunk_locate<THREADS>(&tmp, p.c, where, cells);
    if (!p.checked && blockIdx.x == 0)
        // sequences without blocks (and a bad q_start) have no CTA of their own
        for (int b = tid; b < p.c.B; b += THREADS)
            if (!at.valid || cells(p.c.prefix[b], p.c.q_start[b + 1] - p.c.q_start[b]) == 0)
                p.status[b] = (at.valid && p.c.q_start[b] == p.c.q_start[b + 1] && chunk_shape_ok(p.c, p.c.prefix[b], 0))
                                  ? TV_OK : TV_ERR_OUT_OF_RANGE;
    if (at.b >= p.c.B) return;
    const int P = at.P, n = at.n, lb = (int)((uint32_t)P / (uint32_t)bs) + (int)(cell - at.base);
    // (the sequence's check covers it; looked at here so that its scales can be fetched beside the check)
    const int64_t blk = chunk_shape_ok(p.c, P, n) ? p.c.table[(int64_t)at.b * p.c.max_blocks + lb] : -1;
    const int64_t first = (int64_t)lb * bs;                       // position of the block's row 0
    const int r0 = (int)max((int64_t)P - first, (int64_t)0);      // new rows of the block: r0 .. r1 - 1
    const int r1 = (int)min((int64_t)P + n - first, (int64_t)bs);
    const int64_t row0 = at.row + first - P;                      // the input's row of the block's row 0
    // ---- this CTA's units: key heads, value heads, query heads
    const int units = 2 * p.Hkv + (p.q ? p.Hq : 0);
    const int u_lo = units * split / p.splits, u_hi = units * (split + 1) / p.splits;
    const int half = rope.dim / 2, rv = rope.dim / 8;             // rotated pairs, rotated pieces
    // A piece's eight columns: 8 pairs' first or second columns, or (interleaved) 4 pairs.  The 16
    // bytes of two pairs lie beside the next piece's, so that lanes read consecutive banks.
    const int per = rope.interleaved ? 4 : 8, ru = half / per;
    auto cs_at = [&](int r, int c, int x) -> int { return ((r * (per / 2) + x / 2) * ru + c) * 2 + (x & 1); };
    // The lane's two pieces of a row, and its row of RPL: in the half layout a rotated piece and the one
    // with its pairs' second columns.
    const int l = lane % LPR, sub = lane / LPR;
    const int hv = rope.interleaved ? 0 : rv / 2;
    const int ca = l < hv ? l : l + hv, cb = l < hv ? l + hv : l + LPR;
    const int ch0 = r0 / AQ_ROWS, ch1 = (r1 + AQ_ROWS - 1) / AQ_ROWS;
    const bool once = ch1 - ch0 == 1;
    if (!once)
        for (int u = tid; u < 2 * p.Hkv; u += THREADS) top[u] = 0.f;
    bool fresh = true;
#pragma unroll 1
    for (int pass = once ? 1 : 0; pass < 2; ++pass)
#pragma unroll 1
        for (int ch = ch0; ch < ch1; ++ch) {
            const int lo = max(r0, ch * AQ_ROWS), hi = min(r1, (ch + 1) * AQ_ROWS);
            const int c0 = ch * AQ_ROWS;
            // rows of a piece that none of the new rows is in: the same for the whole warp
            auto idle = [&](int i) { return c0 + (i + 1) * RPL <= lo || c0 + i * RPL >= hi; };
            uint4 x[NL][2];
            auto load = [&](int u) {
                const int kind = u < p.Hkv ? 0 : (u < 2 * p.Hkv ? 1 : 2);     // key, value, query
                const int h = u - (kind == 0 ? 0 : kind == 1 ? p.Hkv : 2 * p.Hkv);
                const uint8_t* src = kind == 0 ? p.k : kind == 1 ? p.v : p.q;
                const int64_t step = kind == 0 ? p.k_stride : kind == 1 ? p.v_stride : p.q_stride;
                src += (row0 + c0 + sub) * step + (int64_t)(h * VEC) * 16;
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const int r = c0 + i * RPL + sub;
                    x[i][0] = x[i][1] = make_uint4(0u, 0u, 0u, 0u);
                    if (r >= lo && r < hi) {
                        x[i][0] = *reinterpret_cast<const uint4*>(src + i * RPL * step + ca * 16);
                        x[i][1] = *reinterpret_cast<const uint4*>(src + i * RPL * step + cb * 16);
                    }
                }
            };
            const int last = pass == 0 ? min(u_hi, 2 * p.Hkv) : u_hi;
            if (u_lo + warp < last) load(u_lo + warp);
            bool ok = true;
            if (fresh) {
                ok = p.checked ? p.status[at.b] == TV_OK : aq_seq_ok(p, at.b, P, at.row, n, tid, THREADS);
                if (r0 > 0 && blk >= 0 && blk < p.c.num_blocks) {
                    // the scales of earlier tokens, and their codes on the way into L2
                    for (int u = tid; u < 2 * p.Hkv; u += THREADS)
                        was[u] = (u < p.Hkv ? p.k_scale : p.v_scale)[blk * p.Hkv + (u < p.Hkv ? u : u - p.Hkv)];
                    for (int u = u_lo + warp; u < min(u_hi, 2 * p.Hkv); u += THREADS / 32)
                        if (lane < (r0 * D + 127) / 128)
                            prefetch_l2((u < p.Hkv ? p.k_cache : p.v_cache) +
                                        ((blk * p.Hkv + (u < p.Hkv ? u : u - p.Hkv)) * bs * D + lane * 128));
                }
            } else {
                __syncthreads();
            }
            // (cos, sin) of the rows' pairs
            if (u_lo < p.Hkv || u_hi > 2 * p.Hkv)
                for (int e = tid; e < (hi - lo) * half; e += THREADS) {
                    const int r = lo + e / half, j = e % half;
                    const int64_t pos = p.positions ? p.positions[row0 + r] : first + r;
                    // the low 64 bits of position * turn: a fraction of a turn in [-1/2, 1/2); in half turns
                    // a float and what it leaves of it, whose sine is pi times as much
                    const int64_t a = (int64_t)((uint64_t)(uint32_t)pos * rope.turn[j]);
                    const float ah = __ll2float_rn(a);
                    const int64_t rest = (int64_t)((uint64_t)a - (fabsf(ah) < 9.2233720368547758e18f ? (uint64_t)(int64_t)ah : 1ull << 63));
                    const float by = __ll2float_rn(rest) * (1.0842021724855044e-19f * 3.14159265f);
                    float sn, co;
                    sincospif(ah * 1.0842021724855044e-19f, &sn, &co);  // 2^-63
                    const float rest_c = fmaf(co, rope.amplitude_rest, -sn * by * rope.amplitude);
                    const float rest_s = fmaf(sn, rope.amplitude_rest, co * by * rope.amplitude);
                    cs[cs_at(r - c0, j / per, j % per)] = make_float2(fmaf(co, rope.amplitude, rest_c), fmaf(sn, rope.amplitude, rest_s));
                }
            ok = __syncthreads_and(ok ? 1 : 0) != 0;
            if (fresh && !p.checked && cell == at.base && split == 0 && tid == 0) p.status[at.b] = ok ? TV_OK : TV_ERR_OUT_OF_RANGE;
            if (!ok) return;
            fresh = false;
#pragma unroll 1
            for (int u = u_lo + warp; u < last; u += THREADS / 32) {
                const int kind = u < p.Hkv ? 0 : (u < 2 * p.Hkv ? 1 : 2);
                const int h = u - (kind == 0 ? 0 : kind == 1 ? p.Hkv : 2 * p.Hkv);
                // the rows, rotated: products and sums in float32
                float f[NL][2][8];
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    bf16_floats(x[i][0], f[i][0]);
                    bf16_floats(x[i][1], f[i][1]);
                }
                if (kind != 1 && half != 0)
#pragma unroll
                    for (int i = 0; i < NL; ++i) {
                        const int r = i * RPL + sub;
                        if (idle(i) || c0 + r < lo || c0 + r >= hi) continue;
                        if (rope.interleaved) {
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int cc = y ? cb : ca;
                                if (cc >= rv) continue;
#pragma unroll
                                for (int e = 0; e < 4; e += 2) {
                                    const float4 w = *reinterpret_cast<const float4*>(cs + cs_at(r, cc, e));
                                    turn(f[i][y][2 * e], f[i][y][2 * e + 1], w.x, w.y);
                                    turn(f[i][y][2 * e + 2], f[i][y][2 * e + 3], w.z, w.w);
                                }
                            }
                        } else if (l < hv) {
#pragma unroll
                            for (int e = 0; e < 8; e += 2) {
                                const float4 w = *reinterpret_cast<const float4*>(cs + cs_at(r, l, e));
                                turn(f[i][0][e], f[i][1][e], w.x, w.y);
                                turn(f[i][0][e + 1], f[i][1][e + 1], w.z, w.w);
                            }
                        }
                    }
                if (kind == 2) {
                    // columns that are not rotated come out as they went in, but for the bits of a NaN
                    uint8_t* dst = p.q_out + (row0 + c0 + sub) * p.qo_stride + (int64_t)(h * VEC) * 16;
#pragma unroll
                    for (int i = 0; i < NL; ++i) {
                        const int r = c0 + i * RPL + sub;
                        if (r >= lo && r < hi)
#pragma unroll
                            for (int y = 0; y < 2; ++y)
                                *reinterpret_cast<uint4*>(dst + i * RPL * p.qo_stride + (y ? cb : ca) * 16) =
                                    make_uint4(pack_bf16x2(f[i][y][0], f[i][y][1]), pack_bf16x2(f[i][y][2], f[i][y][3]),
                                               pack_bf16x2(f[i][y][4], f[i][y][5]), pack_bf16x2(f[i][y][6], f[i][y][7]));
                    }
                }
                if (u + THREADS / 32 < last) load(u + THREADS / 32);
                if (kind == 2) continue;
                float* scale = (kind == 0 ? p.k_scale : p.v_scale) + blk * p.Hkv + h;
                uint8_t* codes = (kind == 0 ? p.k_cache : p.v_cache) + (blk * p.Hkv + h) * bs * D;
                // the largest finite value (a NaN is no maximum); infinities become NaN on the way
                auto largest = [&]() {
                    float m = 0.f;
#pragma unroll
                    for (int i = 0; i < NL; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(f[i][e >> 3][e & 7]));
                    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
                };
                float m = largest();
                if (m == INFINITY) {
#pragma unroll
                    for (int i = 0; i < NL; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e) f[i][e >> 3][e & 7] = fmaf(f[i][e >> 3][e & 7], 0.f, f[i][e >> 3][e & 7]);
                    m = largest();
                }
                if (pass == 0) {
                    if (lane == 0) top[u] = fmaxf(top[u], m);
                    __syncwarp();
                    continue;
                }
                if (!once) m = top[u];
                __syncwarp();
                if (ch == ch0) {
                    m = scale_needed(m);
                    if (r0 > 0) {
                        // earlier tokens of the block: their codes for the larger scale
                        const float old = scale_of(exponent_byte(was[u]));
                        if (old > m) m = old;
                        else if (old < m) {
                            const float by = old * scale_inverse(m);
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
                        *scale = m;
                        if (!once) top[u] = m;
                    }
                    __syncwarp();
                }
                const float inv = scale_inverse(m);
                codes += (int64_t)(c0 + sub) * D;
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    if (idle(i)) continue;
                    const int r = c0 + i * RPL + sub;
                    uint2 w[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float(&g)[8] = f[i][y];
                        w[y] = make_uint2(e4m3_pair(g[0] * inv, g[1] * inv) | e4m3_pair(g[2] * inv, g[3] * inv) << 16,
                                          e4m3_pair(g[4] * inv, g[5] * inv) | e4m3_pair(g[6] * inv, g[7] * inv) << 16);
                    }
                    if (r >= lo && r < hi) {
                        *reinterpret_cast<uint2*>(codes + i * RPL * D + ca * 8) = w[0];
                        *reinterpret_cast<uint2*>(codes + i * RPL * D + cb * 8) = w[1];
                    }
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
        LaunchCfg lc(dim3((unsigned)std::min(a.B, 65535)), dim3(AQ_CHECK), 0, a.stream);
        if (cudaLaunchKernelEx(&lc.cfg, append_q8_check_kernel, p) != cudaSuccess) return TV_ERR_CUDA;
        if (a.T == 0) return TV_OK;
    }
    // Few blocks (a sequence's first and last are half full, say): CTAs of 8 warps, the heads split over as
    // many as the GPU holds, each with a whole number of rounds; the (cos, sin) are computed by each of
    // them.  (832 rows of 32 sequences, 48 heads: 3 CTAs per block 10.5 us, 6 of them 13.8, 6 of 4 warps 11.9.)
    // Many: CTAs of 4 warps, which leave fewer of them idle in the last round (8192 rows, 36 heads: 32 us,
    // with 8 warps 35).
    const int units = 2 * a.Hkv + (a.q ? a.Hq : 0);
    const int64_t likely = (int64_t)a.T / a.bs + std::min(a.T, a.B);
    const int64_t room = (int64_t)device_sm_count() * AQ_SM_THREADS / 256 / likely;
    const bool few = room >= 2;
    p.splits = 1;
    if (few) {
        const int most = (int)std::min<int64_t>(room, (units + 7) / 8);
        const int rounds = (units + 8 * most - 1) / (8 * most);
        p.splits = (units + 8 * rounds - 1) / (8 * rounds);
    }
    if (cells * p.splits > 0x7fffffff) return TV_ERR_UNSUPPORTED;
    tv_rope_table none{};
    const tv_rope_table& rope = a.rope ? *a.rope : none;
    const size_t smem = (size_t)AQ_ROWS * (rope.dim / 2) * sizeof(float2) + (size_t)4 * a.Hkv * sizeof(float);
    if (smem > 40 * 1024) return TV_ERR_UNSUPPORTED;
    LaunchCfg lc(dim3((unsigned)(cells * p.splits)), dim3(few ? 256 : 128), smem, a.stream);
    cudaError_t e;
    if (a.d == 128)
        e = few ? cudaLaunchKernelEx(&lc.cfg, append_q8_kernel<128, 256>, p, rope)
                : cudaLaunchKernelEx(&lc.cfg, append_q8_kernel<128, 128>, p, rope);
    else
        e = few ? cudaLaunchKernelEx(&lc.cfg, append_q8_kernel<64, 256>, p, rope)
                : cudaLaunchKernelEx(&lc.cfg, append_q8_kernel<64, 128>, p, rope);
    return e == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // namespace tv
