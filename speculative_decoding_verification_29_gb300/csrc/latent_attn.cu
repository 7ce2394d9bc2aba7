// latent_attn.cu -- attention whose keys and values all come from one latent
// vector a token, over a paged cache of them.
//
// out = sum_t softmax_t(s q . c_t) c_t[0 .. C): every head reads the same slots,
// the keys' projection has been absorbed into the queries.
//
// A warp owns one row (token and head) and walks its slots.
#include "kv8_attn.cuh"
#include "latent.h"

namespace specv {

namespace {

constexpr int kRowWarps = 8;

template <typename QT>
__global__ void __launch_bounds__(kRowWarps * 32) latent_rows_kernel(const __grid_constant__ LatentAttnArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  if (b == 0)
    for (int i = blockIdx.x * kRowWarps * 32 + threadIdx.x; i < a.parts; i += gridDim.x * kRowWarps * 32)
      a.gave_up[i] = 0, a.cut[i] = make_int4(0, 0, 0, 0);
  const int lo = a.cu[b], hi = a.cu[b + 1], ctx = a.c.len[b];
  if (!kv8_seq_ok(a.c, a.T, lo, hi, ctx) || hi - lo > a.max_tokens) return;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(hi - lo) * a.group) return;
  const int tok = static_cast<int>(row / a.group), h = static_cast<int>(row - static_cast<int64_t>(tok) * a.group);
  const int C = a.c.D, W = C + a.rot;
  const QT* q = static_cast<const QT*>(a.q) + (lo + static_cast<int64_t>(tok)) * a.qst + h * a.qsh;
  float x[18], acc[16] = {}, top = kNegInf, sum = 0.f;
#pragma unroll
  for (int i = 0; i < 18; ++i) x[i] = lane + 32 * i < W ? to_f(q[lane + 32 * i]) * (a.negate ? -a.scale : a.scale) : 0.f;
  for (int t = 0; t < ctx + hi - lo; ++t) {
    if (t >= ctx && !sees(a, b, tok, t - ctx)) continue;
    const int id = a.c.table[static_cast<int64_t>(b) * a.c.max_blocks + t / a.c.block];
    if (id < 0 || id >= a.c.num_blocks) continue;
    const QT* e = reinterpret_cast<const QT*>(a.c.k + id * a.c.sb + (t % a.c.block) * a.c.ss);
    float v[18], y = 0.f;
#pragma unroll
    for (int i = 0; i < 18; ++i) {
      v[i] = lane + 32 * i < W ? to_f(e[lane + 32 * i]) : 0.f;
      y = fmaf(x[i], v[i], y);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    const float m = fmaxf(top, y), by = top == kNegInf ? 0.f : exp2f(top - m), w = m == kNegInf ? 0.f : exp2f(y - m);
    sum = sum * by + w;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = acc[i] * by + w * v[i];
    top = m;
  }
  QT* out = static_cast<QT*>(a.out) + (lo + static_cast<int64_t>(tok)) * a.ost + h * a.osh;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (lane + 32 * i < C) out[lane + 32 * i] = from_f<QT>(sum == 0.f ? 0.f : acc[i] / sum);
}

// -------------------------------------------------------------------- join --
//
// As kv8_join_kernel, for rows of up to 512 dimensions: block x adds the shares of the item that begins in part x and ends
// behind it, a warp one row at a time; the last blocks check sequences, and make the rows NaN that see an entry of a page
// outside the pool.

template <typename QT, int N>
__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(const __grid_constant__ LatentAttnArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, C = a.c.D;
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x >= static_cast<unsigned>(a.parts)) {  // a warp per sequence: row_status
    const int b = (blockIdx.x - a.parts) * (kJoinThreads / 32) + warp;
    if (blockIdx.y > 0 || b >= a.c.B) return;
    bool late = false;
    for (int i = lane; i < a.parts; i += 32) late |= (a.gave_up[i] & kGaveUp) != 0;
    const int lo = a.cu[b], hi = a.cu[b + 1], len = a.c.len[b];
    const bool sound = kv8_seq_ok(a.c, a.T, lo, hi, len) && hi - lo <= a.max_tokens;
    bool bad = !sound;
    if (sound && hi > lo) {
      const int pages = (len + (hi - lo) + a.c.block - 1) / a.c.block;
      for (int j = lane; j < pages; j += 32) {
        const int id = a.c.table[static_cast<int64_t>(b) * a.c.max_blocks + j];
        bad |= id < 0 || id >= a.c.num_blocks;
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    late = __any_sync(0xffffffffu, late);
    if (lane == 0) a.row_status[b] = (bad ? SPEC_ROW_CACHE : 0) | (late ? SPEC_ROW_TIMEOUT : 0);
    if (bad && lo >= 0 && hi > lo && hi <= a.T) {
#pragma unroll 1
      for (int t = lo; t < hi; ++t) {
        if (sound && !sees_outside(a, b, len, hi - lo, t - lo)) continue;
#pragma unroll 1
        for (int h = 0; h < a.q_heads; ++h)
          for (int d = lane; d < C; d += 32)
            static_cast<QT*>(a.out)[t * a.ost + h * a.osh + d] = from_f<QT>(__int_as_float(0x7fffffff));
      }
    }
    return;
  }
  const int4 item = a.cut[blockIdx.x];
  const int n = item.w;
  if (n == 0) return;
  const RowTile r = row_tile<N>(a, item.x, item.y);
  const int64_t first = blockIdx.x;
  bool outside = false;
  for (int i = lane; i < n; i += 32) outside |= (a.gave_up[first + i] & kOutside) != 0;
  outside = __any_sync(0xffffffffu, outside);
#pragma unroll 1
  for (int row = blockIdx.y * (kJoinThreads / 32) + warp; row < r.rows; row += gridDim.y * (kJoinThreads / 32)) {
    auto share = [&](int i) { return (2 * (first + i) + (i == 0 ? 1 : 0)) * N + row; };
    float top = kNegInf;
    for (int i = lane; i < n; i += 32) top = fmaxf(top, a.part_ml[share(i)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float4 acc[4] = {};
    float sum = 0.f;
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const float2 ml = a.part_ml[share(i)];
      const float* p = a.part_o + share(i) * C + 4 * lane;
      const float w = ml.x == top ? 1.f : ex2_fast(ml.x - top);
      sum = fmaf(w, ml.y, sum);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (128 * k >= C) break;
        const float4 u = *reinterpret_cast<const float4*>(p + 128 * k);
        acc[k].x = fmaf(w, u.x, acc[k].x), acc[k].y = fmaf(w, u.y, acc[k].y);
        acc[k].z = fmaf(w, u.z, acc[k].z), acc[k].w = fmaf(w, u.w, acc[k].w);
      }
    }
    const int item_row = item.y * N + row, tok = item_row / a.group;
    QT* out = static_cast<QT*>(a.out) + (r.first + static_cast<int64_t>(tok)) * a.ost + (item_row - tok * a.group) * a.osh + 4 * lane;
    float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (outside && sees_outside(a, item.x, r.ctx, r.n, tok)) inv = __int_as_float(0x7fffffff);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (128 * k >= C) break;
      out[128 * k] = from_f<QT>(acc[k].x * inv), out[128 * k + 1] = from_f<QT>(acc[k].y * inv);
      out[128 * k + 2] = from_f<QT>(acc[k].z * inv), out[128 * k + 3] = from_f<QT>(acc[k].w * inv);
    }
  }
}

template <typename QT, int N>
cudaError_t launch_latent_join(const LatentAttnArgs& a, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.max_tokens) * a.group;
  const int y = static_cast<int>((rows < N ? rows : N) + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  const int checks = (a.c.B + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  return launch_pdl(latent_join_kernel<QT, N>, dim3(static_cast<unsigned>(a.parts + checks), static_cast<unsigned>(y)),
                    dim3(kJoinThreads), st, a);
}

template <typename QT>
cudaError_t launch_rows(const LatentAttnArgs& a, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.max_tokens < a.T ? a.max_tokens : (a.T > 0 ? a.T : 1)) * a.group;
  const cudaError_t e = launch_pdl(latent_rows_kernel<QT>, dim3(static_cast<unsigned>((rows + kRowWarps - 1) / kRowWarps),
                                   static_cast<unsigned>(a.c.B)), dim3(kRowWarps * 32), st, a);
  return e != cudaSuccess ? e : launch_latent_join<QT, 64>(a, st);
}

}  // namespace

int latent_attention_rows(int64_t) { return 64; }

cudaError_t launch_latent_attention(const LatentAttnArgs& a, int dtype, int, const CUtensorMap&, cudaStream_t st) {
  return dtype == SPEC_BF16 ? launch_rows<__nv_bfloat16>(a, st) : launch_rows<__half>(a, st);
}

}  // namespace specv
