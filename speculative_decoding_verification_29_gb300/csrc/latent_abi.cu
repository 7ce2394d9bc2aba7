// latent_abi.cu -- the extern "C" entry points of the paged latent cache and of
// the pages: host-side validation and launches. Argument meanings are documented
// in include/specverify.h.
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "latent.h"
#include "paged.h"

using namespace specv;

namespace {

constexpr int64_t kFar = 1LL << 40;

// The pool's checks; fills `c`.
int take_pool(const spec_latent_cache* s, Kv8Pool* c) {
  if (!s || !s->data || !s->block_table || !s->cache_len) return SPEC_ERR_ARG;
  if (s->B < 1 || s->num_blocks < 1 || s->max_blocks < 1 || s->block < 1 || s->latent_dim < 1 || s->rot_dim < 1)
    return SPEC_ERR_ARG;
  if (s->dtype != SPEC_BF16 && s->dtype != SPEC_F16) return SPEC_ERR_ARG;
  if (s->stride_block < 0 || s->stride_slot < 2LL * (static_cast<int64_t>(s->latent_dim) + s->rot_dim)) return SPEC_ERR_ARG;
  if (((s->stride_block | s->stride_slot) & 15) || !on16(s->data)) return SPEC_ERR_ARG;
  if (s->block != 16 && s->block != 32 && s->block != 64 && s->block != 128) return SPEC_ERR_UNSUPPORTED;
  if (s->latent_dim % 128 != 0 || s->latent_dim > 512 || s->rot_dim % 16 != 0 || s->rot_dim > 64) return SPEC_ERR_UNSUPPORTED;
  if (s->B > kMaxB || static_cast<int64_t>(s->max_blocks) * s->block > kMaxTokens) return SPEC_ERR_UNSUPPORTED;
  if (s->stride_block >= kFar || s->stride_slot >= kFar) return SPEC_ERR_UNSUPPORTED;
  *c = Kv8Pool{};
  c->k = static_cast<uint8_t*>(s->data);
  c->table = s->block_table;
  c->len = s->cache_len;
  c->B = s->B;
  c->num_blocks = s->num_blocks;
  c->max_blocks = s->max_blocks;
  c->block = s->block;
  c->H = 1;
  c->D = s->latent_dim;
  c->sb = s->stride_block;
  c->ss = s->stride_slot;
  return SPEC_OK;
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// As the 8-bit cache's attention: a flag and a cut item (with its sequence) per part, then two shares a part.
struct AttnLayout {
  size_t cut, ml, o, total;
};
AttnLayout attn_layout(int rows, int C) {
  const size_t parts = kSms;
  AttnLayout l{};
  l.cut = up256(parts * sizeof(int32_t));
  l.ml = l.cut + up256(2 * parts * sizeof(int4));
  l.o = l.ml + up256(2 * parts * rows * sizeof(float2));
  l.total = l.o + up256(2 * parts * rows * C * sizeof(float));
  return l;
}

// The pool as a tensor of 16-bit elements: 64 of them by `slots` slots of one block a copy. Elements behind an entry's last read
// as zero. Slots and blocks are ordered by their strides; `order` names them.
bool pool_map(const Kv8Pool& c, int rot, int dtype, int slots, CUtensorMap* map, int* order) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  struct Dim {
    cuuint64_t size, stride;
    cuuint32_t box;
    int name;
  } d[2] = {{static_cast<cuuint64_t>(c.block), static_cast<cuuint64_t>(c.ss), static_cast<cuuint32_t>(slots), 0},
            {static_cast<cuuint64_t>(c.num_blocks), static_cast<cuuint64_t>(c.sb), 1, 1}};
  if (d[1].size == 1) d[1].stride = std::max<cuuint64_t>(d[1].stride, d[0].size * d[0].stride);  // never stepped
  if (d[1].stride < d[0].stride) std::swap(d[0], d[1]);
  const cuuint64_t sizes[3] = {static_cast<cuuint64_t>(c.D + rot), d[0].size, d[1].size};
  const cuuint64_t strides[2] = {d[0].stride, d[1].stride};
  const cuuint32_t box[3] = {64, d[0].box, d[1].box}, step[3] = {1, 1, 1};
  *order = d[0].name;
  return encode(map, dtype == SPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, c.k, sizes,
                strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

int spec_latent_append(const spec_latent_cache* cache, const void* latents, int64_t l_stride_token, const void* rope_keys,
                       int64_t r_stride_token, int dtype, int T, const int32_t* cu_tokens, const int32_t* positions,
                       const double* inv_freq, int interleaved, const void* norm_weight, int norm_dtype, float eps,
                       const void* queries, int64_t q_stride_token, int64_t q_stride_head, void* queries_out,
                       int64_t qo_stride_token, int64_t qo_stride_head, int q_heads, int32_t* row_status, void* stream) {
  LatentAppendArgs a{};
  const int rc = take_pool(cache, &a.c);
  if (rc != SPEC_OK) return rc;
  if (T < 0 || (T > 0 && (!latents || !rope_keys)) || !cu_tokens || !row_status || !inv_freq) return SPEC_ERR_ARG;
  if (dtype != SPEC_F32 && dtype != cache->dtype) return SPEC_ERR_ARG;
  if (!strides_ok(l_stride_token, r_stride_token)) return SPEC_ERR_ARG;
  if (norm_weight && ((norm_dtype != SPEC_F32 && norm_dtype != dtype) || !(eps >= 0.f) || !isfinite(eps))) return SPEC_ERR_ARG;
  if (T == 0) queries = queries_out = nullptr;
  if (!queries != !queries_out) return SPEC_ERR_ARG;
  if (queries && (q_heads < 1 || !strides_ok(q_stride_token, q_stride_head) || !strides_ok(qo_stride_token, qo_stride_head)))
    return SPEC_ERR_ARG;
  if (T >= (1 << 26) || (queries && (static_cast<int64_t>(T) * q_heads >= (1LL << 31) || q_heads > 65536)))
    return SPEC_ERR_UNSUPPORTED;
  a.rot = cache->rot_dim;
  for (int i = 0; i < a.rot / 2; ++i) {
    if (!(fabs(inv_freq[i]) <= 1e9)) return SPEC_ERR_ARG;
    a.freq[i] = turn_fraction(inv_freq[i]);
  }
  const int size = dtype == SPEC_F32 ? 4 : 2;
  a.interleaved = interleaved != 0;
  a.x = latents;
  a.xst = l_stride_token;
  a.r = rope_keys;
  a.rst = r_stride_token;
  a.vec_x = vec16(latents, l_stride_token, 0, size);
  a.w = norm_weight;
  a.w_fp32 = norm_dtype == SPEC_F32;
  a.vec_w = on16(norm_weight);
  a.eps = eps;
  a.q = queries;
  a.qst = q_stride_token;
  a.qsh = q_stride_head;
  a.qo = queries_out;
  a.ost = qo_stride_token;
  a.osh = qo_stride_head;
  a.q_heads = queries ? q_heads : 0;
  a.vec_q = queries && vec16(queries, q_stride_token, q_stride_head, size) &&
            vec16(queries_out, qo_stride_token, qo_stride_head, size);
  a.T = T;
  a.cu = cu_tokens;
  a.pos = positions;
  a.row_status = row_status;
  return cuda_status(launch_latent_append(a, dtype, cache->dtype, static_cast<cudaStream_t>(stream)));
}

size_t spec_latent_workspace_bytes(const spec_latent_cache* cache, int q_heads, int max_tokens) {
  Kv8Pool c;
  if (take_pool(cache, &c) != SPEC_OK || q_heads < 1 || max_tokens < 1) return 0;
  const int rows = latent_attention_rows(static_cast<int64_t>(max_tokens) * q_heads, c.D);
  return attn_layout(rows, rows == 128 && c.D > 256 ? c.D / 2 : c.D).total;
}

int spec_latent_attention(const spec_latent_cache* cache, const void* queries, int64_t q_stride_token, int64_t q_stride_head,
                          int T, int q_heads, const int32_t* cu_tokens, int max_tokens, const uint8_t* tree_mask,
                          float sm_scale, void* out, int64_t o_stride_token, int64_t o_stride_head, int32_t* row_status,
                          void* workspace, size_t workspace_bytes, void* stream) {
  LatentAttnArgs a{};
  const int rc = take_pool(cache, &a.c);
  if (rc != SPEC_OK) return rc;
  if (T < 0 || (T > 0 && (!queries || !out)) || !cu_tokens || !row_status || q_heads < 1 || max_tokens < 1)
    return SPEC_ERR_ARG;
  if (!isfinite(sm_scale)) return SPEC_ERR_ARG;
  if (!strides_ok(q_stride_token, q_stride_head) || !strides_ok(o_stride_token, o_stride_head)) return SPEC_ERR_ARG;
  if (q_heads > 1024 || static_cast<int64_t>(T) * q_heads >= (1LL << 31) || (tree_mask && max_tokens > 1024))
    return SPEC_ERR_UNSUPPORTED;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < spec_latent_workspace_bytes(cache, q_heads, max_tokens))
    return SPEC_ERR_WORKSPACE;
  a.rot = cache->rot_dim;
  a.q = queries;
  a.qst = q_stride_token;
  a.qsh = q_stride_head;
  a.out = out;
  a.ost = o_stride_token;
  a.osh = o_stride_head;
  a.T = T;
  a.q_heads = a.group = q_heads;
  a.max_tokens = max_tokens;
  a.cu = cu_tokens;
  a.tree = tree_mask;
  a.scale = static_cast<float>(fabs(sm_scale * 1.4426950408889634));
  a.negate = sm_scale < 0.f;
  if (a.scale == 0.f) a.scale = 1.f, a.negate = 2;  // scores of zeroed queries: a masked -infinity is not multiplied by 0
  a.row_status = row_status;
  const int64_t most = static_cast<int64_t>(std::min(max_tokens, std::max(T, 1))) * q_heads;  // no sequence has more than T
  const int rows = latent_attention_rows(static_cast<int64_t>(max_tokens) * q_heads, a.c.D);
  a.row_tiles = static_cast<int>((most + rows - 1) / rows);
  if (static_cast<int64_t>(a.row_tiles) * a.c.B >= (1LL << 31)) return SPEC_ERR_UNSUPPORTED;
  a.c.H = rows == 128 && a.c.D > 256 ? 2 : 1;
  a.item_dims = a.c.D / a.c.H;
  // In gangs (see latent_attn.cuh) where all sequences have as many items and whole gangs fill 7 of 8 SMs.
  a.gang = 0;
  const int64_t items = static_cast<int64_t>(a.row_tiles) * a.c.H;
  if (items > 1 && items <= kSms && static_cast<int64_t>(a.c.B) * max_tokens == T && kSms / items * items >= kSms * 7 / 8)
    a.gang = static_cast<int>(items);
  a.parts = a.gang ? kSms / a.gang * a.gang : kSms;
  const AttnLayout l = attn_layout(rows, a.item_dims);
  char* ws = static_cast<char*>(workspace);
  a.gave_up = reinterpret_cast<int32_t*>(ws);
  a.cut = reinterpret_cast<int4*>(ws + l.cut);
  a.part_ml = reinterpret_cast<float2*>(ws + l.ml);
  a.part_o = reinterpret_cast<float*>(ws + l.o);
  CUtensorMap map;
  if (!pool_map(a.c, a.rot, cache->dtype, rows == 128 ? std::min(a.c.block, 64) : a.c.block, &map, &a.order))
    return SPEC_ERR_CUDA;
  return cuda_status(launch_latent_attention(a, cache->dtype, rows, map, static_cast<cudaStream_t>(stream)));
}

int spec_latent_compact(const spec_latent_cache* cache, int n_planes, int64_t stride_plane, const int32_t* path, int D,
                        const int32_t* accept_len, int32_t* new_len, int32_t* row_status, void* stream) {
  LatentCompactArgs a{};
  const int rc = take_pool(cache, &a.c);
  if (rc != SPEC_OK) return rc;
  if (!accept_len || !new_len || !row_status || n_planes < 1 || (path && D < 1)) return SPEC_ERR_ARG;
  if (stride_plane < 0 || (stride_plane & 15)) return SPEC_ERR_ARG;
  if (!lengths_in_place(cache->cache_len, accept_len, new_len, row_status, cache->B, &a.in_place)) return SPEC_ERR_ARG;
  if (path && D > kLatentMaxPath) return SPEC_ERR_UNSUPPORTED;
  if (n_planes >= (1 << 24) || stride_plane >= (1LL << 46)) return SPEC_ERR_UNSUPPORTED;
  a.planes = n_planes;
  a.cols = (cache->latent_dim + cache->rot_dim) / 8;
  a.sp = stride_plane;
  a.path = path;
  a.Dp = path ? D : 0;
  a.acc = accept_len;
  a.new_len = new_len;
  a.row_status = row_status;
  return cuda_status(launch_latent_compact(a, static_cast<cudaStream_t>(stream)));
}

size_t spec_pages_workspace_bytes(int B, int max_blocks, int num_blocks) {
  if (B < 1 || max_blocks < 1 || num_blocks < 1 || B > kMaxB || max_blocks > (1 << 27) || num_blocks > kPagesMaxBlocks) return 0;
  const size_t chunks = (max_blocks + kPagesChunk - 1) / kPagesChunk, n = num_blocks;
  return 3 * up256(n * 4) + up256(B * chunks * 4) + up256(2 * B * sizeof(int4)) + up256(B * sizeof(int2)) + 256;
}

int spec_pages_update(const int32_t* block_table, int32_t* new_table, const int32_t* cache_len, const int32_t* keep_len,
                      const int32_t* source, const int32_t* need, int32_t* refs, int B, int max_blocks, int num_blocks,
                      int block, const spec_pages_pool* pools, int n_pools, int32_t* new_len, int32_t* row_status,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (!block_table || !new_table || !cache_len || !refs || !new_len || !row_status) return SPEC_ERR_ARG;
  if (B < 1 || max_blocks < 1 || num_blocks < 1 || block < 1 || n_pools < 0 || (n_pools > 0 && !pools)) return SPEC_ERR_ARG;
  if ((source && new_table == block_table) || new_len == cache_len) return SPEC_ERR_ARG;
  if (B > kMaxB || max_blocks > (1 << 27) || static_cast<int64_t>(max_blocks) * block > kMaxTokens || n_pools > kMaxPools ||
      num_blocks > kPagesMaxBlocks)
    return SPEC_ERR_UNSUPPORTED;
  const uintptr_t rows = 4 * static_cast<uintptr_t>(B) * max_blocks, before = reinterpret_cast<uintptr_t>(block_table),
                  after = reinterpret_cast<uintptr_t>(new_table);
  if (before != after && before < after + rows && after < before + rows) return SPEC_ERR_ARG;
  PagesArgs a{};
  for (int i = 0; i < n_pools; ++i) {
    const spec_pages_pool& p = pools[i];
    if (!p.data || p.n_planes < 1 || p.block_bytes < 1 || p.stride_plane < 0 || p.stride_block < p.block_bytes)
      return SPEC_ERR_ARG;
    if (p.n_planes >= (1 << 24) || p.block_bytes > (1LL << 30) || p.stride_block >= kFar || p.stride_plane >= (1LL << 46))
      return SPEC_ERR_UNSUPPORTED;
    PagesPool& q = a.pool[i];
    q.base = static_cast<uint8_t*>(p.data);
    q.sp = p.stride_plane;
    q.sb = p.stride_block;
    q.bytes = p.block_bytes;
    q.planes = p.n_planes;
    q.pieces = static_cast<int>((p.block_bytes + kPagesPiece - 1) / kPagesPiece);
    q.vec = on16(p.data) && ((p.stride_plane | p.stride_block | p.block_bytes) & 15) == 0;
  }
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < spec_pages_workspace_bytes(B, max_blocks, num_blocks))
    return SPEC_ERR_WORKSPACE;
  a.table = block_table;
  a.new_table = new_table;
  a.len = cache_len;
  a.keep = keep_len;
  a.source = source;
  a.need = need;
  a.refs = refs;
  a.new_len = new_len;
  a.row_status = row_status;
  a.B = B;
  a.M = max_blocks;
  a.num_blocks = num_blocks;
  a.block = block;
  a.n_pools = n_pools;
  a.chunks = (max_blocks + kPagesChunk - 1) / kPagesChunk;
  char* ws = static_cast<char*>(workspace);
  auto room = [&](size_t bytes) {
    char* at = ws;
    ws += up256(bytes);
    return at;
  };
  a.sharers = reinterpret_cast<int32_t*>(room(static_cast<size_t>(num_blocks) * 4));
  a.last_sharer = reinterpret_cast<int32_t*>(room(static_cast<size_t>(num_blocks) * 4));
  a.free_ids = reinterpret_cast<int32_t*>(room(static_cast<size_t>(num_blocks) * 4));
  a.unsound = reinterpret_cast<int32_t*>(room(static_cast<size_t>(B) * a.chunks * 4));
  a.take = reinterpret_cast<int4*>(room(2 * static_cast<size_t>(B) * sizeof(int4)));
  a.copies = reinterpret_cast<int2*>(room(static_cast<size_t>(B) * sizeof(int2)));
  a.n_copies = reinterpret_cast<int32_t*>(room(4));
  return cuda_status(launch_pages_update(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
