// kv8.h -- the 8-bit paged KV cache: records and launchers shared by its
// kernels and the C entry points.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "specverify.h"

namespace specv {

constexpr int kKv8ExpLo = -40, kKv8ExpHi = 40;  // the scales' exponents
constexpr float kKv8Max = 448.f;                // the largest e4m3 code
constexpr int kKv8MaxPath = 64;
constexpr int kSms = 152;

struct Kv8Pool {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ks;
  uint8_t* vs;
  const int32_t* table;
  const int32_t* len;
  int B, num_blocks, max_blocks, block, H, D;
  int64_t sb, sh, ss;  // strides of block, head and slot in bytes
};

struct Kv8Rope {
  uint64_t freq[64];  // turns per position, as a fraction of 2^64
  int rot, interleaved;
};

struct Kv8AppendArgs {
  Kv8Pool c;
  const void *k, *v, *q;
  void* qo;
  int64_t kst, ksh, vst, vsh, qst, qsh, ost, osh;  // strides in elements: token, head
  int T, q_heads;
  int vec_k, vec_v, vec_q;  // rows on 16-byte boundaries
  const int32_t* cu;
  const int32_t* pos;
  int32_t* row_status;
  Kv8Rope rope;
  // block indices: row_status, then cache blocks, then query rows
  int status_ctas, item_ctas, heads_per_cta, head_groups;
};
cudaError_t launch_kv8_append(const Kv8AppendArgs& a, int dtype, cudaStream_t st);

struct Kv8CompactArgs {
  Kv8Pool c;
  int planes;
  int64_t sp, ssp;  // plane strides in bytes: codes, scales
  const int32_t* path;
  int Dp;
  const int32_t* acc;
  int32_t* new_len;
  int32_t* row_status;
  int what;       // kMoveEntries, kWriteLengths
  bool in_place;  // the lengths are written over those that are read
};
cudaError_t launch_kv8_compact(const Kv8CompactArgs& a, cudaStream_t st);

struct Kv8AttnArgs {
  Kv8Pool c;
  const void* q;
  void* out;
  int64_t qst, qsh, ost, osh;  // strides in elements: token, head
  int T, q_heads, group, max_tokens;
  const int32_t* cu;
  const uint8_t* tree;  // [B][max_tokens][max_tokens] or NULL
  float scale;          // |sm_scale| * log2(e)
  int negate;           // sm_scale < 0: the queries change sign (2, latent cache only: they are zero)
  int32_t* row_status;
  int row_tiles;        // row tiles a sequence has at most
  int parts;            // thread blocks the cache is split over
  int order;            // tensor maps' dimensions 1..3: 2-bit fields naming slot (0), head (1), block (2)
  int32_t* gave_up;     // workspace [parts]: what a part met (kGaveUp, kOutside)
  int4* cut;            // workspace [parts]: the item that begins in the part and ends behind it: sequence, row tile, KV
                        // head, shares (0: none)
  float2* part_ml;      // workspace [2 parts][rows]: exponent reference, sum of weights
  float* part_o;        // workspace [2 parts][rows][head_dim]: weighted sums
};
// Variant for the most rows (step tokens x group) a sequence can have, and
// thread blocks (parts) of its launch.
int kv8_attention_rows(int64_t max_rows);
int kv8_attention_parts(int rows);
cudaError_t launch_kv8_attention(const Kv8AttnArgs& a, int dtype, int rows, const CUtensorMap& k, const CUtensorMap& v,
                                 cudaStream_t st);
cudaError_t launch_kv8_wide(const Kv8AttnArgs& a, int dtype, int rows, const CUtensorMap& k, const CUtensorMap& v,
                            cudaStream_t st);

// ---------------------------------------------------------------- device --

// Whether sequence b's packed tokens [lo, hi) and positions are in range.
__device__ __forceinline__ bool kv8_seq_ok(const Kv8Pool& c, int T, int lo, int hi, int len) {
  return lo >= 0 && hi >= lo && hi <= T && len >= 0 &&
         static_cast<int64_t>(len) + (hi - lo) <= static_cast<int64_t>(c.max_blocks) * c.block;
}

// Exponent of the least scale in range that holds amax: least e with
// amax <= 448 * 2^e = 1.75 * 2^(8 + e), read off the bits.
__device__ __forceinline__ int kv8_need(float amax, int lo = kKv8ExpLo, int hi = kKv8ExpHi) {
  const uint32_t u = __float_as_uint(amax);
  const int x = static_cast<int>(u >> 23) - 127;
  const int e = (u & 0x7fffffu) <= 0x600000u ? x - 8 : x - 7;
  return min(max(e, lo), hi);  // zero and subnormals: x = -127
}

__device__ __forceinline__ int kv8_exp(uint8_t byte) {
  return min(max(static_cast<int>(byte) - 127, kKv8ExpLo), kKv8ExpHi);
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Four codes of x[0..3] * s: nearest even, clamped to +-448; NaN gives the NaN
// code. No x is infinite.
__device__ __forceinline__ uint32_t kv8_codes4_finite(const float* x, float s) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1] * s), "f"(x[0] * s));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3] * s), "f"(x[2] * s));
  return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}

// The same for any x: an infinite one gives the NaN code.
__device__ __forceinline__ uint32_t kv8_codes4(const float* x, float s) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = fabsf(x[i]) < __int_as_float(0x7f800000) ? x[i] : __int_as_float(0x7fffffff);
  return kv8_codes4_finite(y, s);
}

// Four codes as floats.
__device__ __forceinline__ void kv8_values4(uint32_t w, float* y) {
  uint32_t a, b;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"(static_cast<uint16_t>(w & 0xffff)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"(static_cast<uint16_t>(w >> 16)));
  const __half2 p = *reinterpret_cast<const __half2*>(&a), q = *reinterpret_cast<const __half2*>(&b);
  y[0] = __low2float(p);
  y[1] = __high2float(p);
  y[2] = __low2float(q);
  y[3] = __high2float(q);
}

}  // namespace specv
