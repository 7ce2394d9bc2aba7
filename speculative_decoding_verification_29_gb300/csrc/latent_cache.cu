// latent_cache.cu -- writing the paged latent cache: appending normalised latent
// vectors with their rotated dimensions, and compaction along an accepted path.
//
// Append. y = x / sqrt(mean(x^2) + eps) * w over the latent dimensions (fp32,
// rounded once into the slot), and pairs of the shared dimensions and of the
// queries' last ones turned by position * inv_freq; the angle in turns is an
// integer product modulo 2^64. A thread block owns a run of tokens: it finds
// their sequences with one comparison a sequence, in parallel, makes the
// cosines and sines of its tokens once for all heads, then a warp takes a
// token's latent vector, which stays in registers between the sum of squares
// and the store, and all threads share the query rows.
// What bounds it. Prompts (22,000 tokens, 512 + 64 dimensions, 16 heads, fp16): 39
// us, 3.6 TB/s read and written, 0.54 of a copy; 53% of the issue slots and the
// chain sequence, angle, row of every block. 64 sequences x 9 tokens x 32 heads: 5.2 us,
// that chain.
//
// Compaction. Entries keep their bytes, so a thread owns a 16-byte column of a
// plane and moves it along the whole path by itself: path[t] >= t rises, so a
// destination is never an entry that is still to be read. 32 planes x 16 sequences:
// 2.9 us, one path: 1.8, the chain path, table, entries.
#include "act.cuh"
#include "internal.h"
#include "latent.h"

namespace specv {

namespace {

constexpr int kThreads = 256, kMaxHalf = 32;
// Tokens of a thread block. 22,000 tokens, 16 heads, fp16: 4 47.6 us, 8 39.5, 16 42.8, 32 51.1.
constexpr int kMaxTokensCta = 8;

__device__ __forceinline__ void put4(__nv_bfloat16* p, const float* x) {
  __nv_bfloat162 h[2] = {__floats2bfloat162_rn(x[0], x[1]), __floats2bfloat162_rn(x[2], x[3])};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(h);
}
__device__ __forceinline__ void put4(__half* p, const float* x) {
  __half2 h[2] = {__floats2half2_rn(x[0], x[1]), __floats2half2_rn(x[2], x[3])};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(h);
}
__device__ __forceinline__ void get4(const __nv_bfloat16* p, float* x) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  x[0] = bf16_lo(u.x), x[1] = bf16_hi(u.x), x[2] = bf16_lo(u.y), x[3] = bf16_hi(u.y);
}
__device__ __forceinline__ void get4(const __half* p, float* x) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
__device__ __forceinline__ void get4(const float* p, float* x) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
}

__device__ __forceinline__ float2 angle(const LatentAppendArgs& a, int pair, int64_t pos) {
  const int32_t t = static_cast<int32_t>((static_cast<uint64_t>(pos) * a.freq[pair]) >> 32);  // [-1/2, 1/2) of a turn
  float2 cs;
  sincospif(static_cast<float>(t) * 4.656612873077393e-10f, &cs.y, &cs.x);  // 2 t / 2^32 half turns
  return cs;
}

// T: the inputs' type, CT: the cache's.
template <typename T, typename CT>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const __grid_constant__ LatentAppendArgs a) {
  __shared__ int s_first[kMaxTokensCta], s_count[kMaxTokensCta];
  __shared__ float2 s_cs[kMaxTokensCta][kMaxHalf + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bs = a.c.block, half = a.rot / 2, C = a.c.D;
  griddep_launch_dependents();
  griddep_wait();
  if (static_cast<int>(blockIdx.x) >= a.token_ctas) {  // a warp per sequence: row_status
    const int b = (static_cast<int>(blockIdx.x) - a.token_ctas) * (kThreads / 32) + warp;
    if (b >= a.c.B) return;
    const int lo = a.cu[b], hi = a.cu[b + 1], len = a.c.len[b];
    bool bad = !kv8_seq_ok(a.c, a.T, lo, hi, len);
    if (!bad && hi > lo)
      for (int64_t p = len / bs + lane; p <= (static_cast<int64_t>(len) + hi - lo - 1) / bs; p += 32) {
        const int id = a.c.table[static_cast<int64_t>(b) * a.c.max_blocks + p];
        bad |= id < 0 || id >= a.c.num_blocks;
      }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) a.row_status[b] = bad ? SPEC_ROW_CACHE : 0;
    return;
  }
  const int t0 = blockIdx.x * a.tokens, n = min(a.tokens, a.T - t0);
  // A warp's token is on its way while its sequence is looked up.
  static_assert(kMaxTokensCta <= kThreads / 32, "a warp per token");
  float y[4][4] = {};  // its latent vector, four dimensions every 128
  float u = 0.f, v = 0.f;  // the lane's pair of its shared dimensions
  const int d0 = a.interleaved ? 2 * lane : lane, d1 = a.interleaved ? d0 + 1 : d0 + half;
  if (warp < n) {
    const T* x = static_cast<const T*>(a.x) + (t0 + warp) * a.xst;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = 128 * i + 4 * lane;
      if (d >= C) continue;
      if (a.vec_x) {
        get4(x + d, y[i]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) y[i][k] = Act<T>::get(x + d + k);
      }
    }
    if (lane < half) {
      const T* r = static_cast<const T*>(a.r) + (t0 + warp) * a.rst;
      u = Act<T>::get(r + d0), v = Act<T>::get(r + d1);
    }
  }
  if (tid < n) s_first[tid] = 0x7fffffff, s_count[tid] = 0;
  __syncthreads();
  for (int b = tid; b < a.c.B; b += kThreads) {
    const int lo = a.cu[b], hi = a.cu[b + 1];
    if (hi <= t0 || lo >= t0 + n || !kv8_seq_ok(a.c, a.T, lo, hi, a.c.len[b])) continue;
    for (int t = max(lo, t0); t < min(hi, t0 + n); ++t) {
      atomicMin(&s_first[t - t0], b);
      atomicAdd(&s_count[t - t0], 1);
    }
  }
  __syncthreads();
  for (int i = tid; i < n * half; i += kThreads) {
    const int tok = i / half, pair = i - tok * half, b = s_first[tok], t = t0 + tok;
    if (b == 0x7fffffff) continue;
    s_cs[tok][pair] = angle(a, pair, a.pos ? a.pos[t] : static_cast<int64_t>(a.c.len[b]) + (t - a.cu[b]));
  }
  __syncthreads();

  if (warp < n && s_first[warp] != 0x7fffffff) {
    const int tok = warp, t = t0 + tok;
    int b = s_first[tok];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) sum = fmaf(y[i][k], y[i][k], sum);
    if (a.w) {
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float by = 1.f / sqrtf(sum / static_cast<float>(C) + a.eps);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 128 * i + 4 * lane;
        if (d >= C) continue;
        float w[4];
        if (a.vec_w && a.w_fp32) {
          get4(static_cast<const float*>(a.w) + d, w);
        } else if (a.vec_w) {
          get4(static_cast<const T*>(a.w) + d, w);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = a.w_fp32 ? static_cast<const float*>(a.w)[d + k] : Act<T>::get(static_cast<const T*>(a.w) + d + k);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) y[i][k] *= by * w[k];
      }
    }
    const int64_t pos = a.pos ? a.pos[t] : 0;
#pragma unroll 1
    for (int more = s_count[tok];;) {  // sequences that hold the token: one, but where cu_tokens falls
      const int64_t at = static_cast<int64_t>(a.c.len[b]) + (t - a.cu[b]);
      const int id = a.c.table[static_cast<int64_t>(b) * a.c.max_blocks + at / bs];
      if (id >= 0 && id < a.c.num_blocks) {
        CT* slot = reinterpret_cast<CT*>(a.c.k + id * a.c.sb + (at % bs) * a.c.ss);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (128 * i + 4 * lane < C) put4(slot + 128 * i + 4 * lane, y[i]);
        if (lane < half) {
          const float2 cs = b == s_first[tok] ? s_cs[tok][lane] : angle(a, lane, a.pos ? pos : at);
          Act<CT>::put(slot + C + d0, u * cs.x - v * cs.y);
          Act<CT>::put(slot + C + d1, v * cs.x + u * cs.y);
        }
      }
      if (--more <= 0) break;
      int next = b;
#pragma unroll 1
      for (int base = b + 1; base < a.c.B && next == b; base += 32) {
        const int s = base + lane;
        const bool hit = s < a.c.B && a.cu[s] <= t && t < a.cu[s + 1] && kv8_seq_ok(a.c, a.T, a.cu[s], a.cu[s + 1], a.c.len[s]);
        const uint32_t hits = __ballot_sync(0xffffffffu, hit);
        if (hits) next = base + __ffs(hits) - 1;
      }
      if (next == b) break;
      b = next;
    }
  }

  // queries: eight pairs a thread, always the same ones, of all heads of the block's tokens
  const int nc = half / 8, c = tid % nc, step = kThreads / nc;
  int tok = 0, h = tid / nc;
  if (h >= step) return;
  for (;; h += step) {
    while (h >= a.q_heads && tok < n) h -= a.q_heads, ++tok;
    if (tok >= n) break;
    const int t = t0 + tok;
    if (s_first[tok] == 0x7fffffff) continue;
    const int e0 = a.interleaved ? 16 * c : 8 * c, e1 = a.interleaved ? e0 + 8 : half + 8 * c;
    const T* q = static_cast<const T*>(a.q) + t * a.qst + h * a.qsh;
    T* o = static_cast<T*>(a.qo) + t * a.ost + h * a.osh;
    float x[16];
    load_chunk(q + e0, a.vec_q, x);
    load_chunk(q + e1, a.vec_q, x + 8);
    auto turn = [&](float& u, float& v, int k) {
      const float2 cs = s_cs[tok][8 * c + k];
      const float p = u * cs.x - v * cs.y;
      v = v * cs.x + u * cs.y;
      u = p;
    };
    if (a.interleaved) {
#pragma unroll
      for (int k = 0; k < 8; ++k) turn(x[2 * k], x[2 * k + 1], k);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) turn(x[k], x[k + 8], k);
    }
    if (a.vec_q) {
      Act<T>::store8(o + e0, x);
      Act<T>::store8(o + e1, x + 8);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) Act<T>::put(o + e0 + k, x[k]), Act<T>::put(o + e1 + k, x[8 + k]);
    }
  }
}

template <typename T, typename CT>
cudaError_t launch_append(LatentAppendArgs a, cudaStream_t st) {
  // Fewer tokens to a block while there are SMs without one.
  a.tokens = 1;
  while (a.tokens < kMaxTokensCta && static_cast<int64_t>(a.T) > static_cast<int64_t>(a.tokens) * 4 * kSms) a.tokens *= 2;
  a.token_ctas = (a.T + a.tokens - 1) / a.tokens;
  const unsigned checks = (a.c.B + kThreads / 32 - 1) / (kThreads / 32);
  return launch_pdl(latent_append_kernel<T, CT>, dim3(a.token_ctas + checks), dim3(kThreads), st, a);
}

// ----------------------------------------------------------------- compact --

constexpr int kCompactThreads = 128;

__global__ void __launch_bounds__(kCompactThreads) latent_compact_kernel(const __grid_constant__ LatentCompactArgs a) {
  __shared__ int64_t s_src[kLatentMaxPath], s_dst[kLatentMaxPath];  // offsets of the moves in a plane
  __shared__ int s_state, s_from;
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  griddep_launch_dependents();
  griddep_wait();
  const int L = a.acc[b], base = a.c.len[b], bs = a.c.block;
  const int64_t cap = static_cast<int64_t>(a.c.max_blocks) * bs;
  if (tid < 32) {  // 1: move from entry s_from on, 2: nothing to move, 0: skipped, else the negated status
    int state = 1, from = 0;
    if (L < 0) {
      state = 0;
    } else if (base < 0) {
      state = -SPEC_ROW_CACHE;
    } else if (!a.path) {
      state = static_cast<int64_t>(base) + L >= cap ? -SPEC_ROW_TREE : 2;
    } else if (L >= a.Dp) {
      state = -SPEC_ROW_TREE;
    } else {
      const int32_t* path = a.path + static_cast<int64_t>(b) * a.Dp;
      const int32_t* table = a.c.table + static_cast<int64_t>(b) * a.c.max_blocks;
      bool tree = false, cache = false;
      int moved = 0x7fffffff;
      for (int t = lane; t <= L; t += 32) {
        const int p = path[t], prev = t ? path[t - 1] : -1;
        const bool bad = (t == 0 && p != 0) || p <= prev || static_cast<int64_t>(base) + p >= cap;
        tree |= bad;
        if (bad) continue;
        const int src = table[(base + p) / bs], dst = table[(base + t) / bs];  // t <= p: both in the table
        cache |= src < 0 || src >= a.c.num_blocks || dst < 0 || dst >= a.c.num_blocks;
        s_src[t] = src * a.c.sb + ((base + p) % bs) * a.c.ss;
        s_dst[t] = dst * a.c.sb + ((base + t) % bs) * a.c.ss;
        if (p != t) moved = min(moved, t);
      }
      from = __reduce_min_sync(0xffffffffu, moved);
      if (__any_sync(0xffffffffu, tree)) state = -SPEC_ROW_TREE;
      else if (__any_sync(0xffffffffu, cache)) state = -SPEC_ROW_CACHE;
      else if (from > L) state = 2;
    }
    if (lane == 0) s_state = state, s_from = from;
  }
  __syncthreads();
  const int state = s_state;
  if (blockIdx.x == 0 && tid == 0 && (a.what & kWriteLengths)) {
    a.new_len[b] = state >= 1 ? base + L + 1 : -1;
    a.row_status[b] = state < 0 ? -state : 0;
  }
  if (state != 1 || !(a.what & kMoveEntries)) return;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kCompactThreads + tid;  // plane, column
  const int plane = static_cast<int>(item / a.cols), col = static_cast<int>(item - static_cast<int64_t>(plane) * a.cols);
  if (plane >= a.planes) return;
  uint8_t* p = a.c.k + plane * a.sp + 16 * col;
  for (int t = s_from; t <= L; t += 8) {
    uint4 u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (t + k <= L) u[k] = *reinterpret_cast<const uint4*>(p + s_src[t + k]);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (t + k <= L) *reinterpret_cast<uint4*>(p + s_dst[t + k]) = u[k];
  }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs& a, int dtype, int cache_dtype, cudaStream_t st) {
  if (dtype == SPEC_F32)
    return cache_dtype == SPEC_BF16 ? launch_append<float, __nv_bfloat16>(a, st) : launch_append<float, __half>(a, st);
  return dtype == SPEC_BF16 ? launch_append<__nv_bfloat16, __nv_bfloat16>(a, st) : launch_append<__half, __half>(a, st);
}

cudaError_t launch_latent_compact(const LatentCompactArgs& a, cudaStream_t st) {
  const int64_t items = static_cast<int64_t>(a.planes) * a.cols;
  const dim3 grid(static_cast<unsigned>((items + kCompactThreads - 1) / kCompactThreads), static_cast<unsigned>(a.c.B));
  return launch_compaction(latent_compact_kernel, grid, dim3(kCompactThreads), st, a);
}

}  // namespace specv
