// latent.h -- the paged latent cache and the pages under a cache: records and
// launchers shared by the kernels and the C entry points.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv8.h"

namespace specv {

constexpr int kLatentMaxPath = 256;
constexpr int kMaxPools = 8;

// A pool as the schedule of the attention kernels knows it: c.k the entries, H 1, D the latent dimensions, sb and ss in
// bytes. rot: the shared rotated dimensions behind them.
struct LatentAppendArgs {
  Kv8Pool c;
  int rot;
  const void *x, *r, *q, *w;
  void* qo;
  int64_t xst, rst, qst, qsh, ost, osh;  // strides in elements
  int T, q_heads;
  int vec_x, vec_q, vec_w;  // rows on 16-byte boundaries
  int w_fp32;
  float eps;
  const int32_t* cu;
  const int32_t* pos;
  int32_t* row_status;
  uint64_t freq[32];  // turns per position, as a fraction of 2^64
  int interleaved;
  int tokens;      // a thread block's
  int token_ctas;  // thread blocks of tokens; the rest checks sequences
};
cudaError_t launch_latent_append(const LatentAppendArgs& a, int dtype, int cache_dtype, cudaStream_t st);

struct LatentCompactArgs {
  Kv8Pool c;
  int planes, cols;  // cols: 16-byte columns of an entry
  int64_t sp;        // plane stride in bytes
  const int32_t* path;
  int Dp;
  const int32_t* acc;
  int32_t* new_len;
  int32_t* row_status;
  int what;       // kMoveEntries, kWriteLengths
  bool in_place;  // the lengths are written over those that are read
};
cudaError_t launch_latent_compact(const LatentCompactArgs& a, cudaStream_t st);

// c.H: items that the value dimensions of one row tile are shared out to, item_dims each. gang: thread blocks that walk the
// same tiles, one for each item of a sequence; 0: none do.
struct LatentAttnArgs : Kv8AttnArgs {
  int rot, item_dims, gang;
};
int latent_attention_rows(int64_t max_rows, int dims);
cudaError_t launch_latent_rows_f16(const LatentAttnArgs& a, int rows, const CUtensorMap& pool, cudaStream_t st);
cudaError_t launch_latent_wide(const LatentAttnArgs& a, int dtype, const CUtensorMap& pool, cudaStream_t st);
cudaError_t launch_latent_attention(const LatentAttnArgs& a, int dtype, int rows, const CUtensorMap& pool, cudaStream_t st);

struct PagesPool {
  uint8_t* base;
  int64_t sp, sb;       // strides of plane and block in bytes
  int64_t bytes;        // of a block
  int planes, pieces;   // pieces of kPagesPiece bytes to a block
  int vec;              // everything on 16-byte boundaries
};
constexpr int kPagesPiece = 16384;
struct PagesArgs {
  const int32_t* table;
  int32_t* new_table;
  const int32_t *len, *keep, *source, *need;
  int32_t *refs, *new_len, *row_status;
  int B, M, num_blocks, block;
  int n_pools;
  PagesPool pool[kMaxPools];
  // workspace
  int32_t *sharers, *last_sharer;  // [num_blocks]: sequences that go on writing a partly filled block, the last of them
  int32_t* unsound;                // [B][chunks]: bad ids among a row's kept blocks
  int32_t* free_ids;               // [num_blocks]
  int4* take;                      // [2 B]: rank of the first block taken, blocks, first place in the row, block copied;
                                   // tokens kept, whether unsound, whether it asks for room, whether that passes the table
  int2* copies;                    // [B]: source and destination
  int32_t* n_copies;               // [1]
  int chunks;
};
constexpr int kPagesChunk = 1024;
constexpr int kPagesMaxBlocks = 1 << 30;  // a search that adds 4096 at a time stays below 2^31
cudaError_t launch_pages_update(const PagesArgs& a, cudaStream_t st);

}  // namespace specv
