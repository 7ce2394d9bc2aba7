// paged.h -- host-side checks and encodings that the entry points of the paged
// caches share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "specverify.h"

namespace specv {

namespace {

constexpr int kMaxB = 65535;
constexpr int64_t kMaxTokens = (1LL << 31) - 128;  // of a sequence: positions rounded up to a tile of 128 stay below 2^31

inline bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Strides of an activation tensor, in elements; a head's row must fit its stride where it has one.
inline bool strides_ok(int64_t token, int64_t head) {
  return token >= 0 && head >= 0 && token < (1LL << 40) && head < (1LL << 40);
}

inline int vec16(const void* p, int64_t token, int64_t head, int size) {
  return on16(p) && (token * size) % 16 == 0 && (head * size) % 16 == 0;
}

// frequency / (2 pi) modulo 1 in units of 2^-64: the quotient as a sum of two
// doubles (1 / (2 pi) itself is given as one), exact to about 2^-100 before
// the rounding.
inline uint64_t turn_fraction(double f) {
  if (f < 0) return 0 - turn_fraction(-f);  // below, floor must not round
  const double hi_c = 0.15915494309189535, lo_c = -9.8393383374256206e-18;  // 1 / (2 pi) = hi_c + lo_c
  double hi = f * hi_c;
  double lo = fma(f, hi_c, -hi) + f * lo_c;
  hi -= floor(hi);  // exact
  const double a = floor(ldexp(hi, 32));
  lo += hi - ldexp(a, -32);
  const double rest = ldexp(lo, 64);  // below 2^32 in magnitude, may be negative
  return (static_cast<uint64_t>(a) << 32) + static_cast<uint64_t>(static_cast<int64_t>(llrint(rest)));
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiled>(nullptr);
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

}  // namespace
}  // namespace specv
