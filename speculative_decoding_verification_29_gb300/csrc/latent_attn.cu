// latent_attn.cu -- attention over the paged latent cache: the choice of the
// kernel, and the one for few rows in bf16.
#include "latent_rows.cuh"

namespace specv {

// Rows of an item, by the most rows that a sequence can have and the latent dimensions; 128: latent_wide.cu. Few rows are
// cheapest with slots as the products' rows. Above 64 a row a thread is cheaper, unless its last tile of 128 would be half
// empty and both halves of the value dimensions compute its scores again: then up to 320 rows.
// One token, contexts of 1500 to 6500 tokens, bf16, us:
//   rows of a sequence          16   32   48   64   96  128  144  192  224  256  288  320  384  448
//   B = 64
//   512 dimensions, slots       70   76   89   96  131  137  173  179  219  224  266  271  317  366
//   512, a row a thread        110  112  115  117  123  128  197  203  207  210  283  285  296  364
//   384, slots                  54   58   63   70  103  106  138  143  177  179  214  216  250  294
//   384, a row a thread         95   96   99  101  106  111  169  173  176  180  242  244  251  312
//   256, slots                  41   44   50   52   79   81  107  110  136  138  166  167  195  225
//   256, a row a thread         44   45   47   49   53   59   80   83   83   85  111  112  116  136
//   128, slots                  28   30   34   38   60   61   82   84  105  106  128  128  149  173
//   128, a row a thread         33   34   35   35   37   39   59   60   60   61   80   81   83   99
//   B = 4
//   512, slots                  29   32   35   37   33   34   34   35   37   37   38   39   42   45
//   512, a row a thread         27   29   29   30   33   36   38   38   38   38   45   45   45   50
//   256, slots                  23   26   28   28   25   25   25   25   24   25   27   27   28   29
//   256, a row a thread         25   29   29   30   31   34   29   29   30   30   29   29   30   30
//   B = 1
//   512, slots                  16   19   21   24   25   25   25   26   25   25   25   25   25   25
//   512, a row a thread         19   20   21   22   25   28   28   28   28   28   28   28   29   29
// The rule follows B = 64. What it gives away there: up to 9% with 48 and 64 rows of 256 or 128 dimensions and with 448 of 384;
// with four sequences and fewer up to 7 us, on either side.
int latent_attention_rows(int64_t max_rows, int dims) {
  if (max_rows > 64 && !(dims > 256 && max_rows <= 320 && (max_rows - 1) / 64 % 2 == 0)) return 128;
  return max_rows > 48 ? 64 : static_cast<int>((max_rows + 15) / 16 * 16);
}

cudaError_t launch_latent_attention(const LatentAttnArgs& a, int dtype, int rows, const CUtensorMap& map, cudaStream_t st) {
  if (rows == 128) return launch_latent_wide(a, dtype, map, st);
  return dtype == SPEC_BF16 ? launch_type<__nv_bfloat16>(a, rows, map, st) : launch_latent_rows_f16(a, rows, map, st);
}

}  // namespace specv
