// kv8_abi.cu -- the extern "C" entry points of the 8-bit paged KV cache:
// host-side validation and launches. Argument meanings are documented in
// include/specverify.h.
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "kv8.h"
#include "paged.h"

using namespace specv;

namespace {

// The pool's checks; fills `c`.
int take_pool(const spec_kv8_cache* s, Kv8Pool* c) {
  if (!s || !s->k || !s->v || !s->k_scale || !s->v_scale || !s->block_table || !s->cache_len) return SPEC_ERR_ARG;
  if (s->B < 1 || s->num_blocks < 1 || s->max_blocks < 1 || s->kv_heads < 1 || s->head_dim < 1 || s->block < 1)
    return SPEC_ERR_ARG;
  if (s->stride_block < 0 || s->stride_head < 0 || s->stride_slot < s->head_dim) return SPEC_ERR_ARG;
  if ((s->stride_block | s->stride_head | s->stride_slot) & 15) return SPEC_ERR_ARG;
  if (!on16(s->k) || !on16(s->v)) return SPEC_ERR_ARG;
  if (s->block != 16 && s->block != 32 && s->block != 64 && s->block != 128) return SPEC_ERR_UNSUPPORTED;
  if (s->head_dim != 64 && s->head_dim != 128) return SPEC_ERR_UNSUPPORTED;
  if (s->B > kMaxB || s->kv_heads > 1024) return SPEC_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(s->num_blocks) * s->kv_heads > 0x7fffffffLL) return SPEC_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(s->max_blocks) * s->block > kMaxTokens) return SPEC_ERR_UNSUPPORTED;
  if (s->stride_block >= (1LL << 40) || s->stride_head >= (1LL << 40) || s->stride_slot >= (1LL << 40))
    return SPEC_ERR_UNSUPPORTED;
  c->k = static_cast<uint8_t*>(s->k);
  c->v = static_cast<uint8_t*>(s->v);
  c->ks = s->k_scale;
  c->vs = s->v_scale;
  c->table = s->block_table;
  c->len = s->cache_len;
  c->B = s->B;
  c->num_blocks = s->num_blocks;
  c->max_blocks = s->max_blocks;
  c->block = s->block;
  c->H = s->kv_heads;
  c->D = s->head_dim;
  c->sb = s->stride_block;
  c->sh = s->stride_head;
  c->ss = s->stride_slot;
  return SPEC_OK;
}

// The attention's workspace: a flag and a cut item per part, then each part's two shares of
// cut items (exponent references and sums, weighted sums).
struct AttnLayout {
  size_t cut, ml, o, total;
};
AttnLayout attn_layout(int rows, int D) {
  const size_t parts = kv8_attention_parts(rows);
  auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
  AttnLayout l{};
  l.cut = up(parts * sizeof(int32_t));
  l.ml = l.cut + up(parts * sizeof(int4));
  l.o = l.ml + up(2 * parts * rows * sizeof(float2));
  l.total = l.o + up(2 * parts * rows * D * sizeof(float));
  return l;
}

// The pool as a tensor of bytes, one block of one head a copy. Its dimensions
// behind the head's are ordered by their strides; `order` names them.
bool pool_map(const Kv8Pool& c, void* codes, CUtensorMap* map, int* order) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  struct Dim {
    cuuint64_t size, stride;
    cuuint32_t box;
    int name;
  } d[3] = {{static_cast<cuuint64_t>(c.block), static_cast<cuuint64_t>(c.ss), static_cast<cuuint32_t>(c.block), 0},
            {static_cast<cuuint64_t>(c.H), static_cast<cuuint64_t>(c.sh), 1, 1},
            {static_cast<cuuint64_t>(c.num_blocks), static_cast<cuuint64_t>(c.sb), 1, 2}};
  cuuint64_t far = 16;
  for (const Dim& x : d)
    if (x.size > 1) far = std::max(far, x.size * x.stride);
  for (Dim& x : d)
    if (x.size == 1) x.stride = far;  // never stepped
  std::stable_sort(d, d + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
  const cuuint64_t sizes[4] = {static_cast<cuuint64_t>(c.D), d[0].size, d[1].size, d[2].size};
  const cuuint64_t strides[3] = {d[0].stride, d[1].stride, d[2].stride};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(c.D), d[0].box, d[1].box, d[2].box}, step[4] = {1, 1, 1, 1};
  *order = d[0].name | d[1].name << 2 | d[2].name << 4;
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, codes, sizes, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

int spec_kv8_append(const spec_kv8_cache* cache, const void* keys, int64_t k_stride_token, int64_t k_stride_head,
                    const void* values, int64_t v_stride_token, int64_t v_stride_head, int dtype, int T,
                    const int32_t* cu_tokens, const int32_t* positions, const double* inv_freq, int rot_dim,
                    int interleaved, const void* queries, int64_t q_stride_token, int64_t q_stride_head,
                    void* queries_out, int64_t qo_stride_token, int64_t qo_stride_head, int q_heads,
                    int32_t* row_status, void* stream) {
  Kv8AppendArgs a{};
  const int rc = take_pool(cache, &a.c);
  if (rc != SPEC_OK) return rc;
  if (T < 0 || (T > 0 && (!keys || !values)) || !cu_tokens || !row_status) return SPEC_ERR_ARG;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_ARG;
  if (!strides_ok(k_stride_token, k_stride_head) || !strides_ok(v_stride_token, v_stride_head)) return SPEC_ERR_ARG;
  if (T == 0) queries = queries_out = nullptr;
  if (!queries != !queries_out) return SPEC_ERR_ARG;
  if (queries && (q_heads < 1 || !strides_ok(q_stride_token, q_stride_head) ||
                  !strides_ok(qo_stride_token, qo_stride_head)))
    return SPEC_ERR_ARG;
  if (rot_dim < 0 || rot_dim > a.c.D || rot_dim % 16 != 0 || (rot_dim > 0) != (inv_freq != nullptr)) return SPEC_ERR_ARG;
  if (static_cast<int64_t>(T) * a.c.H >= (1LL << 26)) return SPEC_ERR_UNSUPPORTED;
  if (queries && static_cast<int64_t>(T) * q_heads >= (1LL << 31)) return SPEC_ERR_UNSUPPORTED;
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!(fabs(inv_freq[i]) <= 1e9)) return SPEC_ERR_ARG;
    a.rope.freq[i] = turn_fraction(inv_freq[i]);
  }
  a.rope.rot = rot_dim;
  a.rope.interleaved = interleaved != 0;
  const int size = dtype == SPEC_F32 ? 4 : 2;
  a.k = keys;
  a.kst = k_stride_token;
  a.ksh = k_stride_head;
  a.v = values;
  a.vst = v_stride_token;
  a.vsh = v_stride_head;
  a.q = queries;
  a.qst = q_stride_token;
  a.qsh = q_stride_head;
  a.qo = queries_out;
  a.ost = qo_stride_token;
  a.osh = qo_stride_head;
  a.q_heads = queries ? q_heads : 0;
  a.T = T;
  a.vec_k = vec16(keys, k_stride_token, k_stride_head, size);
  a.vec_v = vec16(values, v_stride_token, v_stride_head, size);
  a.vec_q = queries && vec16(queries, q_stride_token, q_stride_head, size) &&
            vec16(queries_out, qo_stride_token, qo_stride_head, size);
  a.cu = cu_tokens;
  a.pos = positions;
  a.row_status = row_status;
  return cuda_status(launch_kv8_append(a, dtype, static_cast<cudaStream_t>(stream)));
}

size_t spec_kv8_workspace_bytes(const spec_kv8_cache* cache, int q_heads, int max_tokens, int dtype) {
  Kv8Pool c;
  if (take_pool(cache, &c) != SPEC_OK || q_heads < 1 || q_heads % c.H != 0 || max_tokens < 1) return 0;
  if (dtype != SPEC_BF16 && dtype != SPEC_F16) return 0;
  return attn_layout(kv8_attention_rows(static_cast<int64_t>(max_tokens) * (q_heads / c.H)), c.D).total;
}

int spec_kv8_attention(const spec_kv8_cache* cache, const void* queries, int64_t q_stride_token,
                       int64_t q_stride_head, int dtype, int T, int q_heads, const int32_t* cu_tokens, int max_tokens,
                       const uint8_t* tree_mask, float sm_scale, void* out, int64_t o_stride_token,
                       int64_t o_stride_head, int32_t* row_status, void* workspace, size_t workspace_bytes,
                       void* stream) {
  Kv8AttnArgs a{};
  const int rc = take_pool(cache, &a.c);
  if (rc != SPEC_OK) return rc;
  if (T < 0 || (T > 0 && (!queries || !out)) || !cu_tokens || !row_status || q_heads < 1 || max_tokens < 1)
    return SPEC_ERR_ARG;
  if (dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_ARG;
  if (q_heads % a.c.H != 0 || !isfinite(sm_scale)) return SPEC_ERR_ARG;
  if (!strides_ok(q_stride_token, q_stride_head) || !strides_ok(o_stride_token, o_stride_head)) return SPEC_ERR_ARG;
  if (q_heads / a.c.H > 64 || static_cast<int64_t>(T) * q_heads >= (1LL << 31) || (tree_mask && max_tokens > 1024))
    return SPEC_ERR_UNSUPPORTED;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < spec_kv8_workspace_bytes(cache, q_heads, max_tokens, dtype))
    return SPEC_ERR_WORKSPACE;
  a.q = queries;
  a.qst = q_stride_token;
  a.qsh = q_stride_head;
  a.out = out;
  a.ost = o_stride_token;
  a.osh = o_stride_head;
  a.T = T;
  a.q_heads = q_heads;
  a.group = q_heads / a.c.H;
  a.max_tokens = max_tokens;
  a.cu = cu_tokens;
  a.tree = tree_mask;
  a.scale = static_cast<float>(fabs(sm_scale * 1.4426950408889634));
  a.negate = sm_scale < 0.f;
  a.row_status = row_status;
  const int64_t most = static_cast<int64_t>(std::min(max_tokens, std::max(T, 1))) * a.group;  // no sequence has more than T
  const int rows = kv8_attention_rows(static_cast<int64_t>(max_tokens) * a.group);
  a.row_tiles = static_cast<int>((most + rows - 1) / rows);
  if (static_cast<int64_t>(a.row_tiles) * a.c.B >= (1LL << 31)) return SPEC_ERR_UNSUPPORTED;
  a.parts = kv8_attention_parts(rows);
  const AttnLayout l = attn_layout(rows, a.c.D);
  char* ws = static_cast<char*>(workspace);
  a.gave_up = reinterpret_cast<int32_t*>(ws);
  a.cut = reinterpret_cast<int4*>(ws + l.cut);
  a.part_ml = reinterpret_cast<float2*>(ws + l.ml);
  a.part_o = reinterpret_cast<float*>(ws + l.o);
  CUtensorMap kmap, vmap;
  if (!pool_map(a.c, a.c.k, &kmap, &a.order) || !pool_map(a.c, a.c.v, &vmap, &a.order)) return SPEC_ERR_CUDA;
  const auto launch = rows >= 128 ? launch_kv8_wide : launch_kv8_attention;
  return cuda_status(launch(a, dtype, rows, kmap, vmap, static_cast<cudaStream_t>(stream)));
}

int spec_kv8_compact(const spec_kv8_cache* cache, int n_planes, int64_t stride_plane, int64_t scale_stride_plane,
                     const int32_t* path, int D, const int32_t* accept_len, int32_t* new_len, int32_t* row_status,
                     void* stream) {
  Kv8CompactArgs a{};
  const int rc = take_pool(cache, &a.c);
  if (rc != SPEC_OK) return rc;
  if (!accept_len || !new_len || !row_status || n_planes < 1 || (path && D < 1)) return SPEC_ERR_ARG;
  if (stride_plane < 0 || scale_stride_plane < 0 || (stride_plane & 15)) return SPEC_ERR_ARG;
  if (!lengths_in_place(cache->cache_len, accept_len, new_len, row_status, cache->B, &a.in_place)) return SPEC_ERR_ARG;
  if (path && D > kKv8MaxPath) return SPEC_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(n_planes) * a.c.B * a.c.H >= (1LL << 30) || stride_plane >= (1LL << 46) ||
      scale_stride_plane >= (1LL << 46))
    return SPEC_ERR_UNSUPPORTED;
  a.planes = n_planes;
  a.sp = stride_plane;
  a.ssp = scale_stride_plane;
  a.path = path;
  a.Dp = path ? D : 0;
  a.acc = accept_len;
  a.new_len = new_len;
  a.row_status = row_status;
  return cuda_status(launch_kv8_compact(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
