// kv8_attn.cu -- attention over the 8-bit paged KV cache.
//
// One thread block per packed token and KV head, all query heads of the group:
// tiles of 128 cache slots, one slot per thread for the scores, one dimension
// per thread for the weighted sum, a running maximum and sum per row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "kv8.h"

namespace specv {

namespace {

constexpr int kTile = 128;
constexpr int kMaxGroup = 64;

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

template <typename T, int D>
__global__ void __launch_bounds__(kTile) kv8_attention_rows(const __grid_constant__ Kv8AttnArgs a) {
  __shared__ float s_p[kTile], s_v[kTile], s_red[2][4];
  __shared__ int s_id[kTile];
  const int tid = threadIdx.x, t = blockIdx.x, h = blockIdx.y;
  griddep_launch_dependents();
  griddep_wait();
  const bool report = t >= a.T;  // the last B columns of blocks write row_status
  int b = report ? t - a.T : 0;
  for (int hi = report ? b : a.c.B; hi - b > 1;) {
    const int mid = (b + hi) >> 1;
    if (a.cu[mid] <= t) b = mid;
    else hi = mid;
  }
  const int lo = a.cu[b], hi = a.cu[b + 1], len = a.c.len[b], bs = a.c.block;
  bool bad = !kv8_seq_ok(a.c, a.T, lo, hi, len) || hi - lo > a.max_tokens;
  const int i = t - lo, end = len + (a.tree ? hi - lo : i + 1);
  const int32_t* table = a.c.table + static_cast<int64_t>(b) * a.c.max_blocks;
  if (!bad)
    for (int j = tid; j < (len + hi - lo + bs - 1) / bs; j += kTile) bad |= table[j] < 0 || table[j] >= a.c.num_blocks;
  bad = __syncthreads_or(bad);
  if (report) {
    if (tid == 0 && h == 0) a.row_status[b] = bad ? SPEC_ROW_CACHE : 0;
    return;
  }
  if (t < lo || t >= hi) return;
  for (int g = 0; g < a.group; ++g) {
    const int head = h * a.group + g;
    const T* q = static_cast<const T*>(a.q) + t * a.qst + head * a.qsh;
    T* out = static_cast<T*>(a.out) + t * a.ost + head * a.osh;
    if (bad) {
      if (tid < D) out[tid] = from_f<T>(__int_as_float(0x7fffffff));
      continue;
    }
    float top = -__int_as_float(0x7f800000), sum = 0.f, acc = 0.f;
    for (int s0 = 0; s0 < end; s0 += kTile) {
      const int s = s0 + tid;
      float y = -__int_as_float(0x7f800000), vs = 0.f;
      int id = 0;
      if (s < end && (s < len || !a.tree ||
                      a.tree[(static_cast<int64_t>(b) * a.max_tokens + i) * a.max_tokens + (s - len)])) {
        id = table[s / bs];
        const uint8_t* k = a.c.k + id * a.c.sb + h * a.c.sh + (s % bs) * a.c.ss;
        float dot = 0.f;
        for (int d = 0; d < D; d += 4) {
          float x[4];
          kv8_values4(*reinterpret_cast<const uint32_t*>(k + d), x);
#pragma unroll
          for (int u = 0; u < 4; ++u) dot = fmaf(to_f(q[d + u]), x[u], dot);
        }
        y = dot * a.scale * pow2i(kv8_exp(a.c.ks[static_cast<int64_t>(id) * a.c.H + h]));
        vs = pow2i(kv8_exp(a.c.vs[static_cast<int64_t>(id) * a.c.H + h]));
      }
      float m = y;
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      __syncthreads();
      if ((tid & 31) == 0) s_red[0][tid >> 5] = m;
      __syncthreads();
      m = fmaxf(fmaxf(s_red[0][0], s_red[0][1]), fmaxf(s_red[0][2], s_red[0][3]));
      const float now = fmaxf(top, m);
      const float ref = now > -__int_as_float(0x7f800000) ? now : 0.f;
      const float p = exp2f(y - ref), old = exp2f(top - ref);
      float l = p;
      for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if ((tid & 31) == 0) s_red[1][tid >> 5] = l;
      s_p[tid] = p;
      s_v[tid] = vs;
      s_id[tid] = id;
      __syncthreads();
      sum = sum * old + (s_red[1][0] + s_red[1][1] + s_red[1][2] + s_red[1][3]);
      acc *= old;
      top = now;
      if (tid < D)
        for (int u = 0; u < min(kTile, end - s0); ++u) {
          if (s_v[u] == 0.f) continue;  // not seen
          const uint8_t c = a.c.v[s_id[u] * a.c.sb + h * a.c.sh + ((s0 + u) % bs) * a.c.ss + tid];
          float x[4];
          kv8_values4(c, x);
          acc = fmaf(s_p[u] * s_v[u], x[0], acc);
        }
    }
    if (tid < D) out[tid] = from_f<T>(sum > 0.f || sum != sum ? acc / sum : 0.f);
  }
}

template <typename T>
cudaError_t launch_rows(const Kv8AttnArgs& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.T + a.c.B), static_cast<unsigned>(a.c.H)), block(kTile);
  return a.c.D == 128 ? launch_pdl(kv8_attention_rows<T, 128>, grid, block, st, a)
                      : launch_pdl(kv8_attention_rows<T, 64>, grid, block, st, a);
}

}  // namespace

cudaError_t launch_kv8_attention(const Kv8AttnArgs& a, int dtype, cudaStream_t st) {
  return dtype == SPEC_BF16 ? launch_rows<__nv_bfloat16>(a, st) : launch_rows<__half>(a, st);
}

}  // namespace specv
