// C-ABI entry points of libtreeverify: argument checks on the host, then one
// launch per call on the caller's stream.  See include/treeverify.h for the
// contract of each call.
#include <math.h>

#include "tv_device.cuh"
#include "tv_internal.h"

namespace tv {

static int cached_attr(cudaDeviceAttr attr, int* cache) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (cache[dev] == 0) {
        int v = 0;
        if (cudaDeviceGetAttribute(&v, attr, dev) == cudaSuccess) cache[dev] = v;
    }
    return cache[dev];
}

int device_sm_count() {
    static int cache[64] = {0};
    const int v = cached_attr(cudaDevAttrMultiProcessorCount, cache);
    return v > 0 ? v : 1;
}

int device_smem_optin() {
    static int cache[64] = {0};
    return cached_attr(cudaDevAttrMaxSharedMemoryPerBlockOptin, cache);
}

LateWait test_late_wait() {
    LateWait l;
    if (const char* e = getenv("TV_TEST_WAITS_RUN_OUT")) {
        char* end = nullptr;
        l.warp = (int)strtol(e, &end, 10);
        if (*end == '@') l.cta = (int)strtol(end + 1, nullptr, 10);
    }
    return l;
}

}  // namespace tv

using namespace tv;

extern "C" {

const char* tv_status_string(int s) {
    switch (s) {
        case TV_OK: return "ok";
        case TV_ERR_INVALID_ARG: return "invalid argument";
        case TV_ERR_BAD_TREE: return "parent array is not a valid topologically ordered tree";
        case TV_ERR_OUT_OF_RANGE: return "block id, position, token id or length out of range";
        case TV_ERR_UNSUPPORTED: return "unsupported shape, dtype or mode";
        case TV_ERR_CUDA: return "CUDA runtime or launch failure";
        case TV_ERR_TIMEOUT: return "bounded device wait ran out";
        case TV_ERR_BAD_VALUES: return "all-NaN logits or zero-mass distribution";
        case TV_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
        default: return "unknown status";
    }
}

int tv_abi_version(void) { return 2; }

tv_status tree_mask_build(const int32_t* parents, int B, int N, const int32_t* node_counts,
                          uint64_t* mask, int32_t* depth, int32_t* status, tv_stream_t stream) {
    if (B < 0 || N < 1 || N > 64) return TV_ERR_INVALID_ARG;
    if (B > 0 && (!parents || !mask || !status)) return TV_ERR_INVALID_ARG;
    return launch_tree_mask(parents, B, N, node_counts, mask, depth, status, (cudaStream_t)stream);
}

static bool attn_shape_ok(int B, int N, int Hq, int Hkv, int d, int max_blocks, int bs,
                          tv_dtype dt) {
    if (B < 0 || N < 1 || N > 64 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return false;
    if (max_blocks < 1 || bs < 1) return false;
    if (dt == TV_BF16) return (d == 64 || d == 128) && bs % 16 == 0;
    if (dt == TV_F32) return d >= 32 && d <= 256 && d % 32 == 0;
    return false;
}

size_t tree_verify_attention_workspace(int B, int N, int Hq, int Hkv, int d,
                                       int max_blocks_per_seq, int block_size, tv_dtype dt) {
    if (!attn_shape_ok(B, N, Hq, Hkv, d, max_blocks_per_seq, block_size, dt)) return 0;
    if (dt != TV_BF16 || B == 0) return 0;
    return attn_bf16_workspace(B, N, Hq, Hkv, d, max_blocks_per_seq, block_size);
}

int tree_verify_attention_kernels(int B, int N, int Hq, int Hkv, int d, int max_blocks_per_seq,
                                  int block_size, tv_dtype dt, size_t workspace_bytes) {
    if (dt != TV_F32 && dt != TV_BF16) return -1;
    if (B < 0 || N < 1 || N > 64 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_blocks_per_seq < 1 ||
        block_size < 1)
        return -1;
    if (!attn_shape_ok(B, N, Hq, Hkv, d, max_blocks_per_seq, block_size, dt)) return -1;
    if (B == 0) return 0;
    if (dt == TV_BF16 && attn_tc_applicable(N, Hq, Hkv, d))
        return attn_tc_kernels(B, N, Hq, Hkv, workspace_bytes);
    return 1;
}

tv_status tree_verify_attention(const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* block_table, int max_blocks_per_seq,
                                const int32_t* prefix_lens, const uint64_t* mask, int B, int N,
                                const int32_t* node_counts, int Hq, int Hkv, int d,
                                int block_size, int num_blocks, tv_dtype dt, float scale,
                                void* out, int32_t* status, void* workspace,
                                size_t workspace_bytes, tv_stream_t stream) {
    if (dt != TV_F32 && dt != TV_BF16) return TV_ERR_INVALID_ARG;
    if (B < 0 || N < 1 || N > 64 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_blocks_per_seq < 1 ||
        block_size < 1 || num_blocks < 1)
        return TV_ERR_INVALID_ARG;
    if (!attn_shape_ok(B, N, Hq, Hkv, d, max_blocks_per_seq, block_size, dt))
        return TV_ERR_UNSUPPORTED;
    if (B == 0) return TV_OK;
    if (!q || !k_cache || !v_cache || !block_table || !prefix_lens || !mask || !out || !status)
        return TV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(k_cache) & 15) || (reinterpret_cast<uintptr_t>(v_cache) & 15) ||
        (reinterpret_cast<uintptr_t>(q) & 15) || (reinterpret_cast<uintptr_t>(out) & 15))
        return TV_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !isfinite(scale)) scale = 1.0f / sqrtf((float)d);
    AttnArgs a;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_table = block_table;
    a.max_blocks = max_blocks_per_seq;
    a.prefix_lens = prefix_lens;
    a.mask = mask;
    a.counts = node_counts;
    a.B = B;
    a.N = N;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.d = d;
    a.bs = block_size;
    a.num_blocks = num_blocks;
    a.scale = scale;
    a.out = out;
    a.status = status;
    a.ws = workspace;
    a.ws_bytes = workspace_bytes;
    a.stream = (cudaStream_t)stream;
    return dt == TV_F32 ? launch_attn_f32(a) : launch_attn_bf16(a);
}

size_t tree_accept_workspace(tv_accept_mode mode, int B, int N, int V) {
    if (B <= 0 || N < 1 || N > 64 || V < 1 || V > (1 << 24)) return 0;
    return accept_workspace(mode, B, N, V);
}

tv_status tree_accept(tv_accept_mode mode, const int32_t* parents, const int32_t* draft_tokens,
                      const float* target, const float* draft_probs, int B, int N,
                      const int32_t* node_counts, int V, uint64_t seed, uint64_t offset,
                      int32_t* accept_len, int32_t* path,
                      int32_t* out_tokens, int max_path, int32_t* status, void* workspace,
                      size_t workspace_bytes, tv_stream_t stream) {
    if (mode != TV_ACCEPT_GREEDY && mode != TV_ACCEPT_STOCHASTIC && mode != TV_ACCEPT_GREEDY_MASKED)
        return TV_ERR_INVALID_ARG;
    if (B < 0 || N < 1 || N > 64 || V < 1 || V > (1 << 24) || max_path < 1)
        return TV_ERR_INVALID_ARG;
    if ((int64_t)B * 16 > 0x7fffffff) return TV_ERR_UNSUPPORTED;
    if (B == 0) return TV_OK;
    if (!parents || !draft_tokens || !target || !accept_len || !path || !out_tokens || !status)
        return TV_ERR_INVALID_ARG;
    if (mode == TV_ACCEPT_STOCHASTIC && !draft_probs) return TV_ERR_INVALID_ARG;
    AcceptArgs a;
    a.mode = mode;
    a.parents = parents;
    a.tokens = draft_tokens;
    a.target = target;
    a.draft = draft_probs;
    a.counts = node_counts;
    a.B = B;
    a.N = N;
    a.V = V;
    a.seed = seed;
    a.offset = offset;
    a.accept_len = accept_len;
    a.path = path;
    a.out_tokens = out_tokens;
    a.max_path = max_path;
    a.status = status;
    a.ws = workspace;
    a.ws_bytes = workspace_bytes;
    a.stream = (cudaStream_t)stream;
    return launch_accept(a);
}

tv_status tree_kv_append(const void* k_new, const void* v_new, const int32_t* depth, int B, int N,
                         const int32_t* node_counts, int Hkv, int d, float rope_theta,
                         void* k_cache, void* v_cache,
                         const int32_t* block_table, int max_blocks_per_seq,
                         const int32_t* prefix_lens, int block_size, int num_blocks, tv_dtype dt,
                         int32_t* status, tv_stream_t stream) {
    if (dt != TV_F32 && dt != TV_BF16) return TV_ERR_INVALID_ARG;
    const int eb = dt == TV_F32 ? 4 : 2;
    if (B < 0 || N < 1 || N > 64 || Hkv < 1 || d < 2 || (d & 1) || block_size < 1 ||
        num_blocks < 1 || max_blocks_per_seq < 1 || !(rope_theta == rope_theta))
        return TV_ERR_INVALID_ARG;
    if ((d * eb) % 16 != 0) return TV_ERR_UNSUPPORTED;
    if (B == 0) return TV_OK;
    if (!k_new || !v_new || !k_cache || !v_cache || !block_table || !prefix_lens || !status ||
        (rope_theta > 0.f && !depth))
        return TV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(k_new) & 15) || (reinterpret_cast<uintptr_t>(v_new) & 15) ||
        (reinterpret_cast<uintptr_t>(k_cache) & 15) || (reinterpret_cast<uintptr_t>(v_cache) & 15))
        return TV_ERR_INVALID_ARG;
    return launch_kv_append(k_new, v_new, depth, B, N, node_counts, Hkv, d, rope_theta, k_cache, v_cache,
                            block_table, max_blocks_per_seq, prefix_lens, block_size, num_blocks,
                            eb, status, (cudaStream_t)stream);
}

tv_status kv_compact(void* k_cache, void* v_cache, int num_layers, int64_t layer_stride,
                     const int32_t* block_table, int max_blocks_per_seq,
                     const int32_t* prefix_lens, const int32_t* path, const int32_t* accept_len,
                     int max_path, int B, int Hkv, int d, int block_size, int num_blocks,
                     tv_dtype dt, int32_t* new_lens, int64_t* src_slots, int64_t* dst_slots,
                     int32_t* status, tv_stream_t stream) {
    if (dt != TV_F32 && dt != TV_BF16) return TV_ERR_INVALID_ARG;
    const int eb = dt == TV_F32 ? 4 : 2;
    if (B < 0 || Hkv < 1 || d < 1 || block_size < 1 || num_blocks < 1 || max_blocks_per_seq < 1 ||
        max_path < 1 || num_layers < 0 || layer_stride < 0)
        return TV_ERR_INVALID_ARG;
    if ((d * eb) % 16 != 0 || d * eb > 1024) return TV_ERR_UNSUPPORTED;
    if (num_layers > 1 && layer_stride < (int64_t)num_blocks * Hkv * block_size * d)
        return TV_ERR_INVALID_ARG;
    if (B == 0 || num_layers == 0) return TV_OK;
    if (!k_cache || !v_cache || !block_table || !prefix_lens || !path || !accept_len ||
        !new_lens || !status)
        return TV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(k_cache) & 15) || (reinterpret_cast<uintptr_t>(v_cache) & 15) ||
        ((layer_stride * eb) & 15))
        return TV_ERR_INVALID_ARG;
    CompactArgs a;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.num_layers = num_layers;
    a.layer_stride = layer_stride;
    a.block_table = block_table;
    a.max_blocks = max_blocks_per_seq;
    a.prefix_lens = prefix_lens;
    a.path = path;
    a.accept_len = accept_len;
    a.max_path = max_path;
    a.B = B;
    a.Hkv = Hkv;
    a.d = d;
    a.bs = block_size;
    a.num_blocks = num_blocks;
    a.elem_bytes = eb;
    a.new_lens = new_lens;
    a.src_slots = src_slots;
    a.dst_slots = dst_slots;
    a.status = status;
    a.stream = (cudaStream_t)stream;
    return launch_compact(a);
}

size_t draft_tree_workspace(int B, int topk, int layers) {
    if (B < 1 || topk < 1 || topk > DT_K_MAX || layers < 1) return 0;
    if (draft_tree_nodes(topk, layers) > DT_NODES_MAX) return 0;
    return draft_tree_ws_bytes(B, topk, layers);
}

tv_status draft_tree_expand(const float* logits, const int32_t* root_tokens, int B, int V, int topk,
                            int layer, int layers, int N, int32_t* front_tokens,
                            int32_t* front_src, int32_t* parents, int32_t* tokens, float* scores,
                            int32_t* status, void* workspace, size_t workspace_bytes,
                            tv_stream_t stream) {
    if (B < 0 || V < 1 || V > (1 << 30) || topk < 1 || topk > DT_K_MAX || topk > V || layers < 1 ||
        layer < 0 || layer >= layers || N < 1 || N > 64)
        return TV_ERR_INVALID_ARG;
    const int64_t nodes = draft_tree_nodes(topk, layers);
    if (nodes > DT_NODES_MAX) return TV_ERR_UNSUPPORTED;
    if (N > nodes) return TV_ERR_INVALID_ARG;
    if (B == 0) return TV_OK;
    const bool last = (layer == layers - 1);
    if (!logits || !status || (layer == 0 && !root_tokens) || (last && (!parents || !tokens)))
        return TV_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) ||
        workspace_bytes < draft_tree_ws_bytes(B, topk, layers))
        return TV_ERR_WORKSPACE;
    // grid: B x F rows x at most DT_CH_MAX chunks
    if ((int64_t)B * topk * DT_CH_MAX > 0x7fffffff) return TV_ERR_UNSUPPORTED;
    DraftArgs a;
    a.logits = logits;
    a.root_tokens = root_tokens;
    a.B = B;
    a.V = V;
    a.k = topk;
    a.layer = layer;
    a.layers = layers;
    a.N = N;
    a.front_tokens = front_tokens;
    a.front_src = front_src;
    a.parents = parents;
    a.tokens = tokens;
    a.scores = scores;
    a.status = status;
    a.ws = workspace;
    a.ws_bytes = workspace_bytes;
    a.stream = (cudaStream_t)stream;
    return launch_draft_expand(a);
}

static bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

tv_status rope_table_init(tv_rope_table* table, int dim, int interleaved, double theta,
                          tv_rope_scaling scaling, double factor, double original_len, double low,
                          double high, double amplitude) {
    return make_rope_table(table, dim, interleaved, theta, scaling, factor, original_len, low, high,
                           amplitude);
}

tv_status chunk_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const int32_t* positions, int T,
                          const int32_t* q_start, const int32_t* prefix_lens, int B, int Hq,
                          int Hkv, int d, const tv_rope_table* rope, void* q_out,
                          int64_t q_out_stride, void* k_cache, void* v_cache,
                          const int32_t* block_table, int max_blocks_per_seq, int block_size,
                          int num_blocks, tv_dtype dt, int32_t* status, tv_stream_t stream) {
    if (dt != TV_F32 && dt != TV_BF16) return TV_ERR_INVALID_ARG;
    const int eb = dt == TV_F32 ? 4 : 2;
    if (T < 0 || B < 0 || Hq < 1 || Hkv < 1 || d < 1 || block_size < 1 || num_blocks < 1 ||
        max_blocks_per_seq < 1)
        return TV_ERR_INVALID_ARG;
    if ((int64_t)Hq * d > 0x7fffffff || (int64_t)Hkv * d > 0x7fffffff) return TV_ERR_UNSUPPORTED;
    if (rope && (rope->dim < 2 || rope->dim > TV_ROPE_MAX_DIM || rope->dim > d))
        return TV_ERR_INVALID_ARG;
    if (((int64_t)d * eb) % 16 != 0 || (rope && (rope->dim * eb) % 32 != 0)) return TV_ERR_UNSUPPORTED;
    if (B == 0) return TV_OK;
    if (!q_start || !prefix_lens || !block_table || !status || !k_cache || !v_cache ||
        (q == nullptr) != (q_out == nullptr))
        return TV_ERR_INVALID_ARG;
    if (T > 0) {
        if (!k || !v || k_stride < (int64_t)Hkv * d || v_stride < (int64_t)Hkv * d ||
            (q && (q_stride < (int64_t)Hq * d || q_out_stride < (int64_t)Hq * d)))
            return TV_ERR_INVALID_ARG;
        if ((k_stride * eb) % 16 || (v_stride * eb) % 16 ||
            (q && ((q_stride * eb) % 16 || (q_out_stride * eb) % 16)))
            return TV_ERR_UNSUPPORTED;
    }
    if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(q_out) ||
        misaligned(k_cache) || misaligned(v_cache))
        return TV_ERR_INVALID_ARG;
    ChunkAppendArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.positions = positions;
    a.T = T;
    a.q_start = q_start;
    a.prefix_lens = prefix_lens;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.d = d;
    a.rope = rope;
    a.q_out = q_out;
    a.q_out_stride = q_out_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_table = block_table;
    a.max_blocks = max_blocks_per_seq;
    a.bs = block_size;
    a.num_blocks = num_blocks;
    a.elem = eb;
    a.status = status;
    a.stream = (cudaStream_t)stream;
    return launch_chunk_append(a);
}

static bool chunk_attn_shape_ok(int Hq, int Hkv, int d, tv_dtype dt) {
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return false;
    if (dt == TV_BF16) return d == 64 || d == 128;
    return dt == TV_F32 && d >= 32 && d <= 256 && d % 32 == 0;
}

size_t chunk_attention_workspace(int T, int B, int Hq, int Hkv, int d, tv_dtype dt) {
    if (T < 1 || B < 1 || !chunk_attn_shape_ok(Hq, Hkv, d, dt)) return 0;
    return chunk_attn_tc_applicable(Hq, Hkv, d, dt) ? chunk_attn_tc_workspace(T, B, Hq, Hkv, d)
                                                    : chunk_attn_f32_workspace(T, B, Hq, Hkv, d, dt);
}

tv_status chunk_attention(const void* q, int64_t q_stride, const void* k_cache,
                          const void* v_cache, const int32_t* block_table,
                          int max_blocks_per_seq, const int32_t* q_start,
                          const int32_t* prefix_lens, int T, int B, int Hq, int Hkv, int d,
                          int block_size, int num_blocks, tv_dtype dt, float scale, float softcap,
                          int window, void* out, int64_t out_stride, int32_t* status,
                          void* workspace, size_t workspace_bytes, tv_stream_t stream) {
    if (dt != TV_F32 && dt != TV_BF16) return TV_ERR_INVALID_ARG;
    if (T < 0 || B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_blocks_per_seq < 1 ||
        block_size < 1 || num_blocks < 1 || !(softcap == softcap) || isinf(softcap))
        return TV_ERR_INVALID_ARG;
    if (!chunk_attn_shape_ok(Hq, Hkv, d, dt) || (dt == TV_BF16 && block_size % 16 != 0))
        return TV_ERR_UNSUPPORTED;
    if (B == 0) return TV_OK;
    if (!q_start || !prefix_lens || !block_table || !status) return TV_ERR_INVALID_ARG;
    const int eb = dt == TV_F32 ? 4 : 2;
    if (T > 0) {
        if (!q || !out || !k_cache || !v_cache || q_stride < (int64_t)Hq * d ||
            out_stride < (int64_t)Hq * d)
            return TV_ERR_INVALID_ARG;
        if ((q_stride * eb) % 16 || (out_stride * eb) % 16) return TV_ERR_UNSUPPORTED;
    }
    if (misaligned(q) || misaligned(out) || misaligned(k_cache) || misaligned(v_cache))
        return TV_ERR_INVALID_ARG;
    const size_t need = chunk_attention_workspace(T, B, Hq, Hkv, d, dt);
    if (need > 0 && (!workspace || misaligned(workspace) || workspace_bytes < need))
        return TV_ERR_WORKSPACE;
    ChunkAttnArgs a;
    a.q = q;
    a.q_stride = q_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_table = block_table;
    a.max_blocks = max_blocks_per_seq;
    a.q_start = q_start;
    a.prefix_lens = prefix_lens;
    a.T = T;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.d = d;
    a.bs = block_size;
    a.num_blocks = num_blocks;
    a.dt = dt;
    a.scale = (scale > 0.f && isfinite(scale)) ? scale : 1.0f / sqrtf((float)d);
    // (a cap of 1e30 changes no score by as much as its rounding, one of 1e-30 leaves nothing of it)
    a.softcap = softcap > 0.f && softcap < 1e30f ? fmaxf(softcap, 1e-30f) : 0.f;
    a.window = window > 0 ? window : 0;
    a.out = out;
    a.out_stride = out_stride;
    a.status = status;
    a.ws = workspace;
    a.stream = (cudaStream_t)stream;
    // without rows there are only statuses to write
    return T > 0 && chunk_attn_tc_applicable(Hq, Hkv, d, dt) ? launch_chunk_attn_tc(a)
                                                             : launch_chunk_attn_f32(a);
}

tv_status token_counts_update(int32_t* counts, const int32_t* tokens, const int32_t* starts,
                              int total, int B, int V, int clear, int prompt, int32_t* status,
                              tv_stream_t stream) {
    if (B < 0 || V < 1 || V > (1 << 24) || total < 0) return TV_ERR_INVALID_ARG;
    if (B == 0) return TV_OK;
    if (!counts || !status || (total > 0 && !tokens) || (!starts && total % B != 0))
        return TV_ERR_INVALID_ARG;
    return launch_token_counts(counts, tokens, starts, total, B, V, clear != 0, prompt != 0, status,
                               (cudaStream_t)stream);
}

tv_status tree_logits_process(const void* logits, tv_dtype dt, int B, int N, int V,
                              const int32_t* node_counts, const uint64_t* mask,
                              const int32_t* draft_tokens, const int32_t* counts,
                              const float* bias, const uint32_t* grammar,
                              const float* repetition, const float* frequency,
                              const float* presence, const float* temperature, int probs,
                              float* out, int32_t* status, tv_stream_t stream) {
    if (dt != TV_F32 && dt != TV_BF16) return TV_ERR_INVALID_ARG;
    if (B < 0 || N < 1 || N > 64 || V < 1 || V > (1 << 24)) return TV_ERR_INVALID_ARG;
    if (B == 0) return TV_OK;
    if (!logits || !out || !status || (mask == nullptr) != (draft_tokens == nullptr))
        return TV_ERR_INVALID_ARG;
    if (!counts && (repetition || frequency || presence)) return TV_ERR_INVALID_ARG;
    LogitsArgs a;
    a.logits = logits;
    a.dt = dt;
    a.B = B;
    a.N = N;
    a.V = V;
    a.node_counts = node_counts;
    a.mask = mask;
    a.tokens = draft_tokens;
    a.counts = counts;
    a.bias = bias;
    a.grammar = grammar;
    a.rep = repetition;
    a.freq = frequency;
    a.pres = presence;
    a.temp = temperature;
    a.probs = probs != 0;
    a.out = out;
    a.status = status;
    a.stream = (cudaStream_t)stream;
    return launch_tree_logits(a);
}

}  // extern "C"
