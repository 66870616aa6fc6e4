// chunk_attention_q8 for more than a few rows per sequence: the kernel of attn_chunk_tc.cuh on tiles
// of e4m3 codes (fewer rows: attn_rows_q8.cu).
#include "attn_chunk_tc.cuh"

namespace tv {

tv_status launch_chunk_attn_q8(const ChunkAttnArgs& a) { return launch_any<true>(a); }

}  // namespace tv
