// chunk_attention on the CUDA cores: float32 (and bfloat16 when a kv head has
// more query heads than a tensor-core row tile holds).
//
// The online softmax over key tiles, everything in float32: a CTA owns 64 rows
// of one (sequence, kv head) (row r is token r / G, head r % G of the kv head's G
// = Hq / Hkv query heads, so a K/V row is read once for all of them) and walks
// 64-key tiles: S = Q K^T, running maximum and sum, O = O 2^(m - m') + P V.
// Bound by float32 multiply-adds: 4 d per (row, key).  128 threads, each an 8 x 4
// patch of S and an 8 x d/16 patch of O in registers, so that a step of the
// inner loops is 12 shared-memory loads of 16 bytes for 128 multiply-adds, which go two by
// two (packed; sums over even and odd columns apart).  K and V come by one bulk copy per row.
// When the rows are too few to fill the GPU the keys are cut into up to 16
// parts; each part leaves its unnormalised O, maximum and sum in the workspace
// and a second kernel joins them in order.
// Batches of about one token per sequence take a second form, further down.
// Measured: 1,000 rows of 32/8 heads of 128 after 3,000 keys 1.65 ms (35 TFLOP/s; 2.02 with
// single multiply-adds, 2.69 with rows through registers); 316 rows of 2 heads of 64 after up to
// 900 keys 22 us, of which two launches and one item's way through the tiles are nearly all.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "tv_chunk.cuh"
#include "tv_internal.h"
#include "tv_tc.cuh"

namespace tv {

namespace {

constexpr int CF_THREADS = 128;
constexpr int CF_M = 64, CF_N = 64;  // rows, keys per tile
constexpr int CF_SPLITS = 16;        // most parts that the keys are cut into
constexpr float CF_LOG2E = 1.4426950408889634f;

struct CfParams {
    ChunkView c;
    const void *q, *k, *v;
    void* out;
    int64_t q_stride, o_stride;   // elements
    int32_t* status;
    float* part;                  // [tiles][Hkv][splits] x (64 x d, 64 maxima, 64 sums)
    int Hkv, G, d, window, splits, tiles;
    float scale, softcap;
    LateWait late;                // test-only
};

// Test-only: this CTA's waits for data count as run out.
__device__ __forceinline__ bool cf_forced(const LateWait& l) {
    return l.warp >= 0 && (l.cta < 0 || l.cta == (int)blockIdx.x);
}

template <typename E>
__device__ __forceinline__ float4 cf_load4(const E* p);
template <>
__device__ __forceinline__ float4 cf_load4<float>(const float* p) {
    return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 cf_load4<__nv_bfloat16>(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void cf_store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void cf_store4(__nv_bfloat16* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

__device__ __forceinline__ int64_t cf_tiles(const CfParams& p, int n) {
    return ((int64_t)n * p.G + CF_M - 1) / CF_M;
}

// The row tile of this CTA.
struct CfTile {
    int b, s, n, P, tile;   // sequence, first row, rows, prefix, tile within the sequence
    bool ok;                // the sequence passed its check
};

// false: no such tile.  Called by every thread (contains barriers).
__device__ __forceinline__ bool cf_find(const CfParams& p, int tile, CfTile& t, bool& valid) {
    __shared__ ChunkLocateTmp<CF_THREADS> tmp;
    const ChunkPlace at = chunk_locate<CF_THREADS>(&tmp, p.c, [&](int64_t) { return (int64_t)tile; },
                                                   [&](int, int n) { return cf_tiles(p, n); });
    valid = at.valid;
    if (at.b >= p.c.B) return false;
    t.b = at.b;
    t.s = p.c.q_start[at.b];
    t.n = p.c.q_start[at.b + 1] - t.s;
    t.P = p.c.prefix[at.b];
    t.tile = tile - (int)at.base;
    bool ok = chunk_shape_ok(p.c, t.P, t.n);
    if (ok) ok = chunk_blocks_ok(p.c, t.b, chunk_first_key(t.P, p.window), (int64_t)t.P + t.n, threadIdx.x, CF_THREADS);
    t.ok = __syncthreads_and(ok ? 1 : 0) != 0;
    return true;
}

// NC: groups of 64 head columns (columns from d on are zero).
template <typename E, int NC>
__global__ void __launch_bounds__(CF_THREADS) chunk_attn_kernel(CfParams p) {
    constexpr int DP = NC * 64, LD = DP + 4;
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;                    // [64][LD]
    float* sk = sq + CF_M * LD;        // [64][LD]
    float* sv = sk + CF_N * LD;        // [64][DP]
    float* sp = sk;                    // P [64][64 + 4] takes K's place once S is done
    __shared__ __align__(8) uint64_t landed;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    if (tid == 0) {
        mbar_init(&landed, 1);
        fence_mbar_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    const int tile_id = (int)(blockIdx.x / p.splits), split = (int)(blockIdx.x % p.splits);
    const int g = blockIdx.y;
    CfTile t;
    bool valid;
    const bool found = cf_find(p, tile_id, t, valid);
    if (blockIdx.x == 0 && g == 0)
        for (int b = tid; b < p.c.B; b += CF_THREADS)
            if (!valid || p.c.q_start[b] == p.c.q_start[b + 1])
                p.status[b] = (valid && chunk_shape_ok(p.c, p.c.prefix[b], 0)) ? TV_OK
                                                                               : TV_ERR_OUT_OF_RANGE;
    if (!found) return;
    if (t.tile == 0 && g == 0 && split == 0 && tid == 0)
        p.status[t.b] = t.ok ? TV_OK : TV_ERR_OUT_OF_RANGE;
    const int r0 = t.tile * CF_M, rows = min(CF_M, t.n * p.G - r0);
    const int i_lo = r0 / p.G, i_hi = (r0 + rows - 1) / p.G;   // first and last token
    // keys of the tile's rows, from the first row's window to the last row itself
    const int k_lo = t.ok ? chunk_first_key(t.P + i_lo, p.window) : 0;
    const int k_hi = t.ok ? t.P + i_hi + 1 : 0;
    const int nt = (k_hi - k_lo + CF_N - 1) / CF_N;
    const int j0 = (int)((int64_t)nt * split / p.splits), j1 = (int)((int64_t)nt * (split + 1) / p.splits);
    const E* q = static_cast<const E*>(p.q);
    const E* kc = static_cast<const E*>(p.k);
    const E* vc = static_cast<const E*>(p.v);
    const int d4 = p.d / 4;
    for (int e = tid; e < CF_M * (DP / 4); e += CF_THREADS) {
        const int r = e / (DP / 4), c = e % (DP / 4);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows && c < d4)
            x = cf_load4<E>(q + (int64_t)(t.s + (r0 + r) / p.G) * p.q_stride +
                            (int64_t)(g * p.G + (r0 + r) % p.G) * p.d + 4 * c);
        *reinterpret_cast<float4*>(sq + r * LD + 4 * c) = x;
    }
    float o[8][NC][4], m[8], l[8];
    int last[8];                       // the row's own position
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // (a bad sequence has no tiles: 0 / 1.  A row whose every score is -infinity ends as 0 / 0.)
        m[i] = t.ok ? -INFINITY : 0.f;
        l[i] = t.ok ? 0.f : 1.f;
        last[i] = t.P + (r0 + min(ty * 8 + i, rows - 1)) / p.G;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][c][e] = 0.f;
    }
    const uint64_t policy = l2_policy_evict_normal();
    for (int j = j0; j < j1; ++j) {
        const int t0 = k_lo + j * CF_N;
        if constexpr (sizeof(E) == 4) {
            // a row per thread by bulk copies.  (Rows past the last key keep what they held: their
            // scores are masked, and their values are not multiplied.)
            fence_proxy_async_smem();  // P was written where K lands
            __syncthreads();           // the previous tile's P and V are done with
            const int r = tid & (CF_N - 1), nk = min(CF_N, k_hi - t0);
            if (tid == 0) mbar_arrive_expect_tx_relaxed_one(&landed, (uint32_t)(2 * nk * p.d) * 4);
            if (r < nk) {
                const int key = t0 + r;
                const int64_t blk = p.c.table[(int64_t)t.b * p.c.max_blocks + key / p.c.bs];
                const int64_t at = ((blk * p.Hkv + g) * p.c.bs + key % p.c.bs) * p.d;
                if (tid < CF_N) bulk_load(sk + r * LD, kc + at, (uint32_t)p.d * 4, &landed, policy);
                else bulk_load(sv + r * DP, vc + at, (uint32_t)p.d * 4, &landed, policy);
            }
            const bool here = mbar_wait(&landed, (uint32_t)(j - j0) & 1u) && !cf_forced(p.late);
            if (__syncthreads_and(here ? 1 : 0) == 0) {
                mbar_wait(&landed, (uint32_t)(j - j0) & 1u);   // (copies still in flight)
                if (tid == 0) p.status[t.b] = TV_ERR_TIMEOUT;
                break;
            }
        } else {
        __syncthreads();               // the previous tile's P and V are done with
        for (int e = tid; e < CF_N * (DP / 4); e += CF_THREADS) {
            const int r = e / (DP / 4), c = e % (DP / 4);
            const int key = t0 + r;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (key < k_hi && c < d4) {
                const int64_t blk = p.c.table[(int64_t)t.b * p.c.max_blocks + key / p.c.bs];
                const int64_t at = ((blk * p.Hkv + g) * p.c.bs + key % p.c.bs) * p.d + 4 * c;
                x = cf_load4<E>(kc + at);
                y = cf_load4<E>(vc + at);
            }
            *reinterpret_cast<float4*>(sk + r * LD + 4 * c) = x;
            *reinterpret_cast<float4*>(sv + r * DP + 4 * c) = y;
        }
        __syncthreads();
        }
        // S: rows ty * 8 + i, keys tx + 16 u
        float s[8][4];
        uint64_t s2[8][4];             // sums over even and odd columns
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) s2[i][u] = 0ull;
        for (int c = 0; c < p.d; c += 4) {
            float4 b4[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) b4[u] = *reinterpret_cast<const float4*>(sk + (tx + 16 * u) * LD + c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 a4 = *reinterpret_cast<const float4*>(sq + (ty * 8 + i) * LD + c);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    s2[i][u] = f2_fma(f2_pack(a4.x, a4.y), f2_pack(b4[u].x, b4[u].y), s2[i][u]);
                    s2[i][u] = f2_fma(f2_pack(a4.z, a4.w), f2_pack(b4[u].z, b4[u].w), s2[i][u]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float lo, hi;
                f2_unpack(s2[i][u], lo, hi);
                s[i][u] = lo + hi;
            }
        __syncthreads();               // every thread is done with K
        // whether every key of the tile is visible to every row
        const bool full = t0 + CF_N - 1 <= t.P + i_lo &&
                          (p.window <= 0 || t0 > t.P + i_hi - p.window);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int key = t0 + tx + 16 * u;
                float z = s[i][u] * p.scale;
                if (p.softcap > 0.f) z = p.softcap * tanhf(z / p.softcap);
                const bool seen = full || (key <= last[i] && (p.window <= 0 || key > last[i] - p.window));
                s[i][u] = seen ? z * CF_LOG2E : -INFINITY;
                mx = fmaxf(mx, s[i][u]);
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[i] - base);
            m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                s[i][u] = exp2f(s[i][u] - base);
                sum += s[i][u];
                sp[(ty * 8 + i) * (CF_N + 4) + tx + 16 * u] = s[i][u];
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            l[i] = l[i] * f + sum;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][c][e] *= f;
        }
        __syncwarp();                  // a row's P is written and read by one half warp
        // O: columns 64 c + 4 tx + e
        auto add = [&](auto all) {
        for (int k = 0; k < CF_N; k += 4) {
            float4 a4[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                a4[i] = *reinterpret_cast<const float4*>(sp + (ty * 8 + i) * (CF_N + 4) + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float4 v4 = *reinterpret_cast<const float4*>(sv + (k + kk) * DP + 64 * c + 4 * tx);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float w = kk == 0 ? a4[i].x : kk == 1 ? a4[i].y : kk == 2 ? a4[i].z : a4[i].w;
                        // a masked key's value must not reach the row even if it is not finite
                        if (decltype(all)::value || w != 0.f) {
                            f2_unpack(f2_fma(f2_pack(w, w), f2_pack(v4.x, v4.y), f2_pack(o[i][c][0], o[i][c][1])), o[i][c][0], o[i][c][1]);
                            f2_unpack(f2_fma(f2_pack(w, w), f2_pack(v4.z, v4.w), f2_pack(o[i][c][2], o[i][c][3])), o[i][c][2], o[i][c][3]);
                        }
                    }
                }
            }
        }
        };
        if (full) add(std::true_type{});
        else add(std::false_type{});
    }
    if (p.splits > 1) {
        float* slot = p.part + (((int64_t)tile_id * p.Hkv + g) * p.splits + split) * (CF_M * (p.d + 2));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = ty * 8 + i;
            if (r >= rows) continue;
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (64 * c + 4 * tx < p.d)
                    *reinterpret_cast<float4*>(slot + r * p.d + 64 * c + 4 * tx) =
                        make_float4(o[i][c][0], o[i][c][1], o[i][c][2], o[i][c][3]);
            if (tx == 0) {
                slot[CF_M * p.d + r] = m[i];
                slot[CF_M * (p.d + 1) + r] = l[i];
            }
        }
        return;
    }
    E* out = static_cast<E*>(p.out);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = ty * 8 + i;
        if (r >= rows) continue;
        const float inv = 1.f / l[i];
        E* row = out + (int64_t)(t.s + (r0 + r) / p.G) * p.o_stride + (int64_t)(g * p.G + (r0 + r) % p.G) * p.d;
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (64 * c + 4 * tx < p.d)
                cf_store4(row + 64 * c + 4 * tx, make_float4(o[i][c][0] * inv, o[i][c][1] * inv,
                                                             o[i][c][2] * inv, o[i][c][3] * inv));
    }
}

// Joins the parts of a row tile: weights 2^(m_k - max) on the unnormalised rows.  A
// thread per (row, four columns); the parts' maxima and sums are loaded together, then
// the rows, so that a part does not wait for the one before.
template <typename E>
__global__ void __launch_bounds__(CF_THREADS) chunk_join_kernel(CfParams p) {
    __shared__ ChunkLocateTmp<CF_THREADS> tmp;
    pdl_wait();
    pdl_launch_dependents();
    const int g = blockIdx.y;
    const ChunkPlace at = chunk_locate<CF_THREADS>(&tmp, p.c, [&](int64_t) { return (int64_t)blockIdx.x; },
                                                   [&](int, int n) { return cf_tiles(p, n); });
    if (at.b >= p.c.B) return;
    const int s = p.c.q_start[at.b], n = p.c.q_start[at.b + 1] - s;
    const int r0 = ((int)blockIdx.x - (int)at.base) * CF_M, rows = min(CF_M, n * p.G - r0);
    const int64_t step = CF_M * (p.d + 2);
    const float* slot = p.part + ((int64_t)blockIdx.x * p.Hkv + g) * p.splits * step;
    const int d4 = p.d / 4, e = blockIdx.z * CF_THREADS + threadIdx.x;
    if (e >= rows * d4) return;
    const int r = e / d4, c = e % d4;
    float m[CF_SPLITS], w[CF_SPLITS], mx = -INFINITY, den = 0.f;
#pragma unroll
    for (int k = 0; k < CF_SPLITS; ++k) {
        m[k] = k < p.splits ? slot[k * step + CF_M * p.d + r] : -INFINITY;
        w[k] = k < p.splits ? slot[k * step + CF_M * (p.d + 1) + r] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < CF_SPLITS; ++k) mx = fmaxf(mx, m[k]);
    const float base = mx == -INFINITY ? 0.f : mx;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k0 = 0; k0 < CF_SPLITS; k0 += 8) {
        float4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            x[u] = k0 + u < p.splits ? *reinterpret_cast<const float4*>(slot + (k0 + u) * step + r * p.d + 4 * c)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float f = exp2f(m[k0 + u] - base);   // (a part without a key: 0, and zero rows)
            den = fmaf(f, w[k0 + u], den);
            acc.x = fmaf(f, x[u].x, acc.x);
            acc.y = fmaf(f, x[u].y, acc.y);
            acc.z = fmaf(f, x[u].z, acc.z);
            acc.w = fmaf(f, x[u].w, acc.w);
        }
    }
    const float inv = 1.f / den;
    E* out = static_cast<E*>(p.out);
    cf_store4(out + (int64_t)(s + (r0 + r) / p.G) * p.o_stride + (int64_t)(g * p.G + (r0 + r) % p.G) * p.d + 4 * c,
              make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
}

template <typename E, int NC>
tv_status launch_nc(const CfParams& p, cudaStream_t stream) {
    constexpr int DP = NC * 64;
    const size_t smem = (size_t)(2 * CF_M * (DP + 4) + CF_N * DP) * 4;
    static std::atomic<bool> set[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TV_ERR_CUDA;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(chunk_attn_kernel<E, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem) != cudaSuccess) {
            cudaGetLastError();
            return TV_ERR_CUDA;
        }
        set[dev] = true;
    }
    LaunchCfg lc(dim3((unsigned)(p.tiles * p.splits), (unsigned)p.Hkv), dim3(CF_THREADS), smem, stream);
    if (cudaLaunchKernelEx(&lc.cfg, chunk_attn_kernel<E, NC>, p) != cudaSuccess) return TV_ERR_CUDA;
    if (p.splits == 1) return TV_OK;
    LaunchCfg lj(dim3((unsigned)p.tiles, (unsigned)p.Hkv, (unsigned)(CF_M * (p.d / 4) / CF_THREADS)),
                 dim3(CF_THREADS), 0, stream);
    return cudaLaunchKernelEx(&lj.cfg, chunk_join_kernel<E>, p) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

// Upper bound of the row tiles per kv head, whatever q_start says, and the parts
// that the keys are cut into.
int64_t cf_tile_bound(int T, int B, int G) { return (int64_t)T * G / CF_M + std::min(T, B); }
int cf_splits(int T, int B, int Hkv, int G) {
    const int64_t ctas = std::max<int64_t>(1, cf_tile_bound(T, B, G) * Hkv);
    return (int)std::clamp<int64_t>(4 * device_sm_count() / ctas, 1, CF_SPLITS);
}

// ------------------------------------------------------------------ few rows
// Batches with about one token per sequence (plain decoding): a token's G <= 8 rows against
// its keys, bound by the K/V stream.  A CTA takes one (token, kv head, part of the keys);
// 16 lanes hold a key's columns, float2 by float2, and go through four keys at a time.  The
// rows come by bulk copies into two stages of eight keys per warp, one filling while the other
// is read.  The 4 R partial dot products of a group of lanes are
// added up by halving exchanges, which leave lane i with the score of (row i / 4, key i % 4):
// 15 exchanges instead of 64 for R = 4.  Every group keeps its own running maximum, sum and
// O; they are joined at the end, then the parts of the keys by a second kernel.
// Measured: 64 sequences of 512-8,192 keys, 1.4 GB with 32/8 heads of 128: 246 us = 5.7 TB/s
// (rows straight into registers twice that, three stages a fifth more).
constexpr int CR_THREADS = 128;
constexpr int CR_GROUPS = CR_THREADS / 16;
constexpr int CR_KEYS = 4;             // per group and step
constexpr int CR_STAGES = 2;
constexpr int CR_WARP_KEYS = 2 * CR_KEYS;
constexpr int CR_PART = 256;           // keys below which a part is not cut further

struct CrParams {
    ChunkView c;
    const float *q, *k, *v;
    float* out;
    int64_t q_stride, o_stride;
    int32_t* status;
    int32_t* parts;               // [T][Hkv] parts that the join finds (0: none)
    float* part;                  // [T][Hkv][splits] x (G x d, G maxima, G sums)
    int Hkv, G, d, window, splits;
    float scale, softcap;
    LateWait late;                // test-only
};

// What is copied for the values past the last key: weight 0 would not keep out an infinity.
__device__ __align__(16) float cr_zeros[256];

template <int NJ, int R>
__global__ void __launch_bounds__(CR_THREADS) chunk_rows_kernel(CrParams p) {
    __shared__ ChunkLocateTmp<CR_THREADS> tmp;
    __shared__ float so[CR_THREADS / 32][R][NJ * 32];
    __shared__ float sm_m[CR_THREADS / 32][R], sm_l[CR_THREADS / 32][R];
    __shared__ __align__(8) uint64_t bars[CR_THREADS / 32][CR_STAGES];
    extern __shared__ __align__(128) float ring[];        // [warp][stage][K, V][key][d]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l16 = lane & 15;
    const int t = blockIdx.x / p.splits, split = blockIdx.x % p.splits, g = blockIdx.y;
    if (lane < CR_STAGES) mbar_init(&bars[warp][lane], 1);
    fence_mbar_init();
    __syncwarp();
    pdl_launch_dependents();
    pdl_wait();
    const ChunkPlace at = chunk_locate<CR_THREADS>(
        &tmp, p.c, [&](int64_t) { return (int64_t)t - p.c.q_start[0]; }, [&](int, int n) { return (int64_t)n; });
    if (blockIdx.x == 0 && g == 0)
        for (int b = tid; b < p.c.B; b += CR_THREADS)
            if (!at.valid || p.c.q_start[b] == p.c.q_start[b + 1])
                p.status[b] = (at.valid && chunk_shape_ok(p.c, p.c.prefix[b], 0)) ? TV_OK : TV_ERR_OUT_OF_RANGE;
    int32_t* n_parts = p.parts + (int64_t)t * p.Hkv + g;
    if (at.b >= p.c.B) {                                  // a row of no sequence
        if (split == 0 && tid == 0) *n_parts = 0;
        return;
    }
    bool ok = chunk_shape_ok(p.c, at.P, at.n);
    if (ok) ok = chunk_blocks_ok(p.c, at.b, chunk_first_key(at.P, p.window), (int64_t)at.P + at.n, tid, CR_THREADS);
    ok = __syncthreads_and(ok ? 1 : 0) != 0;
    if (t == at.row && g == 0 && split == 0 && tid == 0) p.status[at.b] = ok ? TV_OK : TV_ERR_OUT_OF_RANGE;
    float* out = p.out + (int64_t)t * p.o_stride + (int64_t)g * p.G * p.d;
    if (!ok) {
        if (split == 0) {
            for (int e = tid; e < p.G * p.d; e += CR_THREADS) out[e] = 0.f;
            if (tid == 0) *n_parts = 0;
        }
        return;
    }
    const int pos = at.P + (t - at.row), first = chunk_first_key(pos, p.window), keys = pos - first + 1;
    const int active = min(p.splits, (keys + CR_PART - 1) / CR_PART);
    if (split == 0 && tid == 0) *n_parts = active > 1 ? active : 0;
    if (split >= active) return;
    const int k_lo = first + (int)((int64_t)keys * split / active), k_hi = first + (int)((int64_t)keys * (split + 1) / active);
    float2 q[R][NJ], o[R][NJ];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const bool in = r < p.G && j * 32 < p.d;
            q[r][j] = in ? *reinterpret_cast<const float2*>(p.q + (int64_t)t * p.q_stride + (int64_t)(g * p.G + r) * p.d + j * 32 + 2 * l16)
                         : make_float2(0.f, 0.f);
            o[r][j] = make_float2(0.f, 0.f);
        }
    // lane i of a group: the running statistics of rows i / 4 (and i / 4 + 4)
    constexpr int H = R / 4;
    float m[H], l[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
    }
    const int32_t* table = p.c.table + (int64_t)at.b * p.c.max_blocks;
    const uint64_t policy = l2_policy_evict_first();
    // Lanes 0 - 7 copy the K rows of the warp's keys of a step, 8 - 15 their V rows (past the
    // last key that one's K row again, at weight 0, and zeros); the block is looked up a step ahead.
    constexpr int STEP = CR_THREADS / 32 * CR_WARP_KEYS;
    const int steps = (k_hi - k_lo + STEP - 1) / STEP;
    const int copy_key = k_lo + warp * CR_WARP_KEYS + (lane & (CR_WARP_KEYS - 1));
    auto block = [&](int i) -> int {
        return i < steps && lane < 2 * CR_WARP_KEYS ? table[min(copy_key + i * STEP, k_hi - 1) / p.c.bs] : 0;
    };
    const int stage_floats = 2 * CR_WARP_KEYS * p.d;
    float* mine = ring + (size_t)warp * CR_STAGES * stage_floats;
    auto fill = [&](int i, int blk) {
        if (i >= steps) return;
        uint64_t* bar = &bars[warp][i % CR_STAGES];
        if (lane == 0) mbar_arrive_expect_tx_relaxed_one(bar, (uint32_t)stage_floats * 4);
        __syncwarp();
        if (lane < 2 * CR_WARP_KEYS) {
            const int key = min(copy_key + i * STEP, k_hi - 1);
            const float* src = (lane < CR_WARP_KEYS ? p.k : p.v) + (((int64_t)blk * p.Hkv + g) * p.c.bs + key % p.c.bs) * p.d;
            if (lane >= CR_WARP_KEYS && copy_key + i * STEP >= k_hi) src = cr_zeros;
            bulk_load(mine + (i % CR_STAGES) * stage_floats + lane * p.d, src, (uint32_t)p.d * 4, bar, policy);
        }
    };
#pragma unroll
    for (int i = 0; i < CR_STAGES; ++i) fill(i, block(i));
    int blk = block(CR_STAGES);
    bool alive = true;
    for (int i = 0; i < steps; ++i) {
        alive = __all_sync(0xffffffffu, mbar_wait(&bars[warp][i % CR_STAGES], (i / CR_STAGES) & 1) && !cf_forced(p.late));
        if (!alive) break;
        const float* stage = mine + (i % CR_STAGES) * stage_floats + (lane >> 4) * CR_KEYS * p.d + 2 * l16;
        const int my_key = k_lo + i * STEP + (tid >> 4) * CR_KEYS + (l16 & (CR_KEYS - 1));
        float2 kx[CR_KEYS][NJ];
#pragma unroll
        for (int u = 0; u < CR_KEYS; ++u)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                kx[u][j] = j * 32 < p.d ? *reinterpret_cast<const float2*>(stage + u * p.d + j * 32) : make_float2(0.f, 0.f);
        float f[H], w[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            float s[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = h * 4 + i / 4, u = i % 4;
                float a = 0.f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) a = fmaf(q[r][j].x, kx[u][j].x, fmaf(q[r][j].y, kx[u][j].y, a));
                s[i] = a;
            }
#pragma unroll
            for (int step = 8; step > 0; step >>= 1)
#pragma unroll
                for (int i = 0; i < step; ++i) {
                    const bool up = (l16 & step) != 0;
                    const float y = __shfl_xor_sync(0xffffffffu, up ? s[i] : s[i + step], step);
                    s[i] = (up ? s[i + step] : s[i]) + y;
                }
            float z = s[0] * p.scale;
            if (p.softcap > 0.f) z = p.softcap * tanhf(z / p.softcap);
            z = my_key < k_hi ? z * CF_LOG2E : -INFINITY;
            float mx = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[h], mx), bz = mn == -INFINITY ? 0.f : mn;
            f[h] = exp2f(m[h] - bz);
            w[h] = exp2f(z - bz);
            l[h] = fmaf(l[h], f[h], w[h]);
            m[h] = mn;
        }
        float2 vx[CR_KEYS][NJ];
#pragma unroll
        for (int u = 0; u < CR_KEYS; ++u)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                vx[u][j] = j * 32 < p.d ? *reinterpret_cast<const float2*>(stage + (CR_WARP_KEYS + u) * p.d + j * 32) : make_float2(0.f, 0.f);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float fr = __shfl_sync(0xffffffffu, f[r / 4], r % 4 * 4, 16);
            float wr[CR_KEYS];
#pragma unroll
            for (int u = 0; u < CR_KEYS; ++u) wr[u] = __shfl_sync(0xffffffffu, w[r / 4], r % 4 * 4 + u, 16);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                float x = o[r][j].x * fr, y = o[r][j].y * fr;
#pragma unroll
                for (int u = 0; u < CR_KEYS; ++u) {
                    x = fmaf(wr[u], vx[u][j].x, x);
                    y = fmaf(wr[u], vx[u][j].y, y);
                }
                o[r][j] = make_float2(x, y);
            }
        }
        __syncwarp();                                     // the stage is read
        fill(i + CR_STAGES, blk);
        blk = block(i + CR_STAGES + 1);
    }
    if (!alive) {
        // a copy that did not come: the ones behind it are waited for, too
        for (int x = 0; x < CR_STAGES; ++x)
            for (int y = 0; y < 2; ++y) mbar_wait(&bars[warp][x], y);
        if (lane == 0) p.status[at.b] = TV_ERR_TIMEOUT;
    }
    // ---- join: the two groups of a warp by exchanges, the warps through shared memory
#pragma unroll
    for (int h = 0; h < H; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        const float mo = __shfl_xor_sync(0xffffffffu, m[h], 16), lo = __shfl_xor_sync(0xffffffffu, l[h], 16);
        const float mm = fmaxf(m[h], mo), bz = mm == -INFINITY ? 0.f : mm;
        const float f = exp2f(m[h] - bz);
        l[h] = l[h] * f + lo * exp2f(mo - bz);
        m[h] = mm;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = h * 4 + i;
            const float fr = __shfl_sync(0xffffffffu, f, i * 4, 16);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const float x = o[r][j].x * fr, y = o[r][j].y * fr;
                const float xs = x + __shfl_xor_sync(0xffffffffu, x, 16), ys = y + __shfl_xor_sync(0xffffffffu, y, 16);
                if (lane < 16) *reinterpret_cast<float2*>(&so[warp][r][j * 32 + 2 * l16]) = make_float2(xs, ys);
            }
        }
        if (lane < 16 && (l16 & 3) == 0) {
            sm_m[warp][h * 4 + l16 / 4] = m[h];
            sm_l[warp][h * 4 + l16 / 4] = l[h];
        }
    }
    __syncthreads();
    float* slot = p.part + (((int64_t)t * p.Hkv + g) * p.splits + split) * ((int64_t)p.G * (p.d + 2));
    for (int e = tid; e < p.G * p.d; e += CR_THREADS) {
        const int r = e / p.d, c = e - r * p.d;
        float mm = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
        for (int x = 0; x < CR_THREADS / 32; ++x) mm = fmaxf(mm, sm_m[x][r]);
        const float bz = mm == -INFINITY ? 0.f : mm;
#pragma unroll
        for (int x = 0; x < CR_THREADS / 32; ++x) {
            const float f = exp2f(sm_m[x][r] - bz);
            sum = fmaf(f, sm_l[x][r], sum);
            acc = fmaf(f, so[x][r][c], acc);
        }
        if (active == 1) {
            out[e] = acc / sum;
        } else {
            slot[e] = acc;
            if (c == 0) {
                slot[p.G * p.d + r] = mm;
                slot[p.G * (p.d + 1) + r] = sum;
            }
        }
    }
}

__global__ void __launch_bounds__(CR_THREADS) chunk_rows_join_kernel(CrParams p) {
    const int t = blockIdx.x, g = blockIdx.y;
    pdl_wait();
    pdl_launch_dependents();
    const int n = p.parts[(int64_t)t * p.Hkv + g];
    if (n == 0) return;
    const int64_t step = (int64_t)p.G * (p.d + 2);
    const float* slot = p.part + ((int64_t)t * p.Hkv + g) * p.splits * step;
    float* out = p.out + (int64_t)t * p.o_stride + (int64_t)g * p.G * p.d;
    for (int e = threadIdx.x; e < p.G * p.d; e += CR_THREADS) {
        const int r = e / p.d;
        float m[CF_SPLITS], sums[CF_SPLITS], x[CF_SPLITS], mx = -INFINITY, den = 0.f, acc = 0.f;
#pragma unroll
        for (int k = 0; k < CF_SPLITS; ++k) {
            m[k] = k < n ? slot[k * step + p.G * p.d + r] : -INFINITY;
            sums[k] = k < n ? slot[k * step + p.G * (p.d + 1) + r] : 0.f;
            x[k] = k < n ? slot[k * step + e] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < CF_SPLITS; ++k) mx = fmaxf(mx, m[k]);
        const float bz = mx == -INFINITY ? 0.f : mx;
#pragma unroll
        for (int k = 0; k < CF_SPLITS; ++k) {
            const float f = exp2f(m[k] - bz);
            den = fmaf(f, sums[k], den);
            acc = fmaf(f, x[k], acc);
        }
        out[e] = acc / den;
    }
}

// Each token reads its keys for itself, so at most about one token per sequence; a thread
// holds 3 to 4 x G x d / 16 registers of rows and keys.  Only T and B are known here, not the
// lengths.  Measured against the row tiles (32/8 heads of 128): 64 sequences of 512-8,192 keys with
// one token each 246 us against 1,954, with two 442 against 1,960; 8 of 300-3,000 keys 30 and 48
// against 123 and 129; one of 2,000 keys 19 and 21 against 29.  Where all 2 B rows belong to one
// sequence of 3,000 keys and share them: 128 rows 439 against 710, 16 rows 78 against 102.
bool cr_applies(int T, int B, int Hkv, int G, int d, tv_dtype dt) {
    return dt == TV_F32 && T <= 2 * (int64_t)B && G <= (d <= 128 ? 8 : 4) && Hkv <= 65535;
}
int cr_splits(int T, int Hkv) {
    return (int)std::clamp<int64_t>(32 * (int64_t)device_sm_count() / ((int64_t)T * Hkv), 1, CF_SPLITS);
}
size_t cr_counts_bytes(int T, int Hkv) { return ((size_t)T * Hkv * 4 + 15) & ~(size_t)15; }

template <int NJ, int R>
cudaError_t cr_launch_r(const CrParams& p, cudaStream_t stream) {
    const size_t smem = (size_t)CR_THREADS / 32 * CR_STAGES * 2 * CR_WARP_KEYS * p.d * sizeof(float);
    static std::atomic<bool> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev]) {
        const size_t most = (size_t)CR_THREADS / 32 * CR_STAGES * 2 * CR_WARP_KEYS * NJ * 32 * sizeof(float);
        e = cudaFuncSetAttribute(chunk_rows_kernel<NJ, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return e;
        }
        set[dev] = true;
    }
    LaunchCfg lc(dim3((unsigned)(p.c.T * p.splits), (unsigned)p.Hkv), dim3(CR_THREADS), smem, stream);
    return cudaLaunchKernelEx(&lc.cfg, chunk_rows_kernel<NJ, R>, p);
}
template <int NJ>
cudaError_t cr_launch(const CrParams& p, cudaStream_t stream) {
    if constexpr (NJ < 8)
        if (p.G > 4) return cr_launch_r<NJ, 8>(p, stream);
    return cr_launch_r<NJ, 4>(p, stream);
}

tv_status launch_rows(const ChunkAttnArgs& a) {
    CrParams p{};
    p.c = ChunkView{a.q_start, a.prefix_lens, a.block_table, a.T, a.B, a.max_blocks, a.bs, a.num_blocks};
    p.q = static_cast<const float*>(a.q);
    p.k = static_cast<const float*>(a.k_cache);
    p.v = static_cast<const float*>(a.v_cache);
    p.out = static_cast<float*>(a.out);
    p.q_stride = a.q_stride;
    p.o_stride = a.out_stride;
    p.status = a.status;
    p.parts = static_cast<int32_t*>(a.ws);
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + cr_counts_bytes(a.T, a.Hkv));
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.d = a.d;
    p.window = a.window;
    p.splits = cr_splits(a.T, a.Hkv);
    p.late = test_late_wait();
    p.scale = a.scale;
    p.softcap = a.softcap;
    if ((int64_t)a.T * p.splits > 0x7fffffff) return TV_ERR_UNSUPPORTED;
    const cudaError_t e = a.d <= 64 ? cr_launch<2>(p, a.stream) : a.d <= 128 ? cr_launch<4>(p, a.stream) : cr_launch<8>(p, a.stream);
    if (e != cudaSuccess) return TV_ERR_CUDA;
    if (p.splits == 1) return TV_OK;
    LaunchCfg lj(dim3((unsigned)a.T, (unsigned)a.Hkv), dim3(CR_THREADS), 0, a.stream);
    return cudaLaunchKernelEx(&lj.cfg, chunk_rows_join_kernel, p) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // namespace

size_t chunk_attn_f32_workspace(int T, int B, int Hq, int Hkv, int d, tv_dtype dt) {
    const int G = Hq / Hkv, s = cf_splits(T, B, Hkv, G);
    if (T > 0 && cr_applies(T, B, Hkv, G, d, dt))
        return cr_counts_bytes(T, Hkv) + (size_t)T * Hkv * cr_splits(T, Hkv) * G * (d + 2) * sizeof(float);
    return s == 1 ? 0 : (size_t)(cf_tile_bound(T, B, G) * Hkv) * s * CF_M * (d + 2) * sizeof(float);
}

tv_status launch_chunk_attn_f32(const ChunkAttnArgs& a) {
    if (a.T > 0 && cr_applies(a.T, a.B, a.Hkv, a.Hq / a.Hkv, a.d, a.dt)) return launch_rows(a);
    CfParams p{};
    p.c = ChunkView{a.q_start, a.prefix_lens, a.block_table, a.T, a.B, a.max_blocks, a.bs, a.num_blocks};
    p.q = a.q;
    p.k = a.k_cache;
    p.v = a.v_cache;
    p.out = a.out;
    p.q_stride = a.q_stride;
    p.o_stride = a.out_stride;
    p.status = a.status;
    p.part = static_cast<float*>(a.ws);
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.d = a.d;
    p.window = a.window;
    p.late = test_late_wait();
    p.scale = a.scale;
    p.softcap = a.softcap;
    const int64_t tiles = std::max<int64_t>(1, cf_tile_bound(a.T, a.B, p.G));
    p.splits = cf_splits(a.T, a.B, a.Hkv, p.G);
    if (tiles * p.splits > 0x7fffffff || a.Hkv > 65535) return TV_ERR_UNSUPPORTED;
    p.tiles = (int)tiles;
    const int nc = (a.d + 63) / 64;
    if (a.dt == TV_BF16)
        return nc == 1 ? launch_nc<__nv_bfloat16, 1>(p, a.stream) : launch_nc<__nv_bfloat16, 2>(p, a.stream);
    switch (nc) {
        case 1: return launch_nc<float, 1>(p, a.stream);
        case 2: return launch_nc<float, 2>(p, a.stream);
        case 3: return launch_nc<float, 3>(p, a.stream);
        default: return launch_nc<float, 4>(p, a.stream);
    }
}

}  // namespace tv
