// latent_attn.cu -- attention over the paged latent cache: the choice of the
// kernel, and the one for few rows in bf16.
#include "latent_rows.cuh"

namespace specv {

// Rows of an item, by the most rows that a sequence can have and the latent dimensions; 128: latent_wide.cu. Few rows are
// cheapest with slots as the products' rows. Above 64 a row a thread is cheaper, unless its last tile of 128 would be half
// empty and both halves of the value dimensions compute its scores again: then up to 320 rows.
// B = 64, contexts of 1500 to 6500 tokens, bf16, us:
//   rows of a sequence       16   32   48   64   96  128  144  192  224  256  288  320  384  448
//   512 dimensions, slots    66   71   84   92  132  132  170  181  209  224  258  256  322  361
//   512, a row a thread                         123  125  193  199  197  212  272  271  299  360
//   256, slots               47   50   57   61   93   98  122  129  160  160  190  186  235
//   256, a row a thread                          56   61   80   85   86   90  112  112  121
int latent_attention_rows(int64_t max_rows, int dims) {
  if (max_rows > 64 && !(dims > 256 && max_rows <= 320 && (max_rows - 1) / 64 % 2 == 0)) return 128;
  return max_rows > 48 ? 64 : static_cast<int>((max_rows + 15) / 16 * 16);
}

cudaError_t launch_latent_attention(const LatentAttnArgs& a, int dtype, int rows, const CUtensorMap& map, cudaStream_t st) {
  if (rows == 128) return launch_latent_wide(a, dtype, map, st);
  return dtype == SPEC_BF16 ? launch_type<__nv_bfloat16>(a, rows, map, st) : launch_latent_rows_f16(a, rows, map, st);
}

}  // namespace specv
