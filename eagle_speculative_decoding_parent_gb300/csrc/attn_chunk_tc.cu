// chunk_attention over bfloat16 caches: the kernel of attn_chunk_tc.cuh on tiles that TMA brings.
#include "attn_chunk_tc.cuh"

namespace tv {

bool chunk_attn_tc_applicable(int Hq, int Hkv, int d, tv_dtype dt) {
    return dt == TV_BF16 && (d == 64 || d == 128) && Hq / Hkv <= MT;
}

size_t chunk_attn_tc_workspace(int T, int B, int Hq, int Hkv, int d) {
    (void)B;
    return (size_t)2 * device_sm_count() * (partial_rows(T, Hq / Hkv) * (d + 2) * sizeof(float) + sizeof(int4));
}

tv_status launch_chunk_attn_tc(const ChunkAttnArgs& a) { return launch_any<false>(a); }

}  // namespace tv
