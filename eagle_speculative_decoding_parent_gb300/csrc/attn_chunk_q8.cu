// chunk_attention_q8: the kernel of attn_chunk_tc.cuh on tiles of e4m3 codes that four of its warps
// widen to bfloat16.
#include "attn_chunk_tc.cuh"

namespace tv {

tv_status launch_chunk_attn_q8(const ChunkAttnArgs& a) { return launch_any<true>(a); }

}  // namespace tv
