// latent_attn_f16.cu -- attention over the paged latent cache for few rows in fp16.
#include "latent_rows.cuh"

namespace specv {

cudaError_t launch_latent_rows_f16(const LatentAttnArgs& a, int rows, const CUtensorMap& map, cudaStream_t st) {
  return launch_type<__half>(a, rows, map, st);
}

}  // namespace specv
