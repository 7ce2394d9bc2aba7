// latent_attn.cu -- attention over the paged latent cache: the choice of the
// kernel, and the one for few rows in bf16.
#include "latent_rows.cuh"

namespace specv {

// Rows of an item, by the most rows that a sequence can have.
int latent_attention_rows(int64_t max_rows) {
  if (max_rows > 64) return 128;
  return max_rows > 48 ? 64 : static_cast<int>((max_rows + 15) / 16 * 16);
}

cudaError_t launch_latent_attention(const LatentAttnArgs& a, int dtype, int rows, const CUtensorMap& map, cudaStream_t st) {
  if (rows == 128) return launch_latent_wide(a, dtype, map, st);
  return dtype == SPEC_BF16 ? launch_type<__nv_bfloat16>(a, rows, map, st) : launch_latent_rows_f16(a, rows, map, st);
}

}  // namespace specv
