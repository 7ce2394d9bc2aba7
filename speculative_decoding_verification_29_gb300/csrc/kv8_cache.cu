// kv8_cache.cu -- writing the 8-bit paged KV cache: appending rotated keys and
// values, and compaction along an accepted tree path.
//
// Append. One thread block owns one cache block of one head (or of a few
// heads) and either its keys or its values, because the block's scale is a
// maximum over everything the call writes into it: each thread keeps 16
// elements in registers, the largest magnitude goes over
// warps and shared memory, and the codes are stored from the same registers,
// so every input is read once. A cache block that already holds tokens is only
// rewritten when its scale grows.
// Which cache blocks a sequence touches is known on the device alone: sequence
// b gets the candidates cu[b] / block + 2 b .. cu[b + 1] / block + 2 b + 1, at
// least as many as it can touch for any cache_len, and a thread block finds its
// sequence with one comparison per sequence, in parallel. While cu rises a
// candidate is one sequence's; where cu falls it may be several's, which the
// thread block serves one after the other.
// Rotation. position * inv_freq in turns is an integer product modulo 2^64
// (inv_freq / 2 pi as a 64-bit fraction), so the reduced angle loses nothing at
// far positions and takes no 64-bit floating point.
// What bounds it. Prompts (22,000 tokens, 8 KV heads of 128, fp16): 37.6 us, 4.0
// TB/s read and written, 0.59 of a copy; instructions (60% of issue slots) and the
// barrier of each head's maximum share the rest (fp32: 56 us, 4.0 TB/s). 64
// sequences x 9 tokens with queries: 10.5 us, launch and the lookup of each block's
// sequence; 9 tokens: 3.4 us, latency.
//
// Compaction. A warp owns one plane, keys or values and head of a sequence; entries move
// through shared memory in path order, so that a destination is never read
// after it was written. 32 planes x 16 sequences: 7.9 us. A block's room for 64
// entries a warp (33 KB) lets six blocks on an SM, 2.2 rounds of the 2048, and in
// each three warps wait for the one that checks the path (the barrier is the first
// stall); then lengths, path, table, scales and entries are read one after the
// other.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <string.h>

#include <algorithm>

#include "act.cuh"
#include "kv8.h"
#include "internal.h"

namespace specv {

namespace {

constexpr float kInf = __builtin_huge_valf();

// -------------------------------------------------------------- rotation --

// A thread's 16 elements are two chunks of 8. Within the rotated dimensions
// they are the two halves of eight split pairs (chunk at 8 c and at
// rot / 2 + 8 c) or eight interleaved pairs (16 c .. 16 c + 15); behind them,
// two neighbouring chunks.
__device__ __forceinline__ void chunk_dims(const Kv8Rope& r, int c, int* d0, int* d1) {
  const bool split = !r.interleaved && 16 * c < r.rot;
  *d0 = split ? 8 * c : 16 * c;
  *d1 = split ? r.rot / 2 + 8 * c : 16 * c + 8;
}

// cos and sin of pairs 8 c .. 8 c + 7 at a position.
__device__ __forceinline__ void angles(const Kv8Rope& r, int c, int64_t pos, float* cs, float* sn) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t turns = static_cast<uint64_t>(pos) * r.freq[8 * c + i];
    const int32_t t = static_cast<int32_t>(turns >> 32);  // signed: [-1/2, 1/2) of a turn
    sincospif(static_cast<float>(t) * 4.656612873077393e-10f, &sn[i], &cs[i]);  // 2 t / 2^32 half turns
  }
}

__device__ __forceinline__ void turn(const Kv8Rope& r, float* x, const float* cs, const float* sn) {
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = x[2 * i], w = x[2 * i + 1];
      x[2 * i] = u * cs[i] - w * sn[i];
      x[2 * i + 1] = w * cs[i] + u * sn[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = x[i], w = x[8 + i];
      x[i] = u * cs[i] - w * sn[i];
      x[8 + i] = w * cs[i] + u * sn[i];
    }
  }
}

// ------------------------------------------------------------------ append --

template <typename T, int NT>
__device__ __forceinline__ void append_status(const Kv8AppendArgs& a) {  // a warp per sequence
  const int b = blockIdx.x * (NT / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= a.c.B) return;
  const int lo = a.cu[b], hi = a.cu[b + 1], len = a.c.len[b];
  bool bad = !kv8_seq_ok(a.c, a.T, lo, hi, len);
  if (!bad && hi > lo) {
    const int last = (len + (hi - lo) - 1) / a.c.block;
    for (int j = len / a.c.block + lane; j <= last; j += 32) {
      const int id = a.c.table[static_cast<int64_t>(b) * a.c.max_blocks + j];
      bad |= id < 0 || id >= a.c.num_blocks;
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) a.row_status[b] = SPEC_ROW_CACHE;
  else if (lane == 0) a.row_status[b] = 0;
}

template <typename T, int NT>
__device__ __forceinline__ void append_queries(const Kv8AppendArgs& a) {  // a thread: 16 elements of a query row
  const int tpr = a.c.D / 16;
  const int64_t item = static_cast<int64_t>(blockIdx.x - a.status_ctas - a.item_ctas) * NT + threadIdx.x;
  const int64_t row = item / tpr;
  const int c = static_cast<int>(item - row * tpr);
  const int t = static_cast<int>(row / a.q_heads), h = static_cast<int>(row - static_cast<int64_t>(t) * a.q_heads);
  if (t >= a.T) return;
  int64_t pos = 0;
  if (a.pos) {
    pos = a.pos[t];
  } else {  // the token's sequence: the last b with cu[b] <= t
    int lo = 0, hi = a.c.B, from = a.cu[lo], end = a.cu[hi];
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1, at = a.cu[mid];
      if (at <= t) lo = mid, from = at;
      else hi = mid, end = at;
    }
    if (t < from || t >= end) {  // cu falls, or no sequence has the token
      for (int b = 0; b < a.c.B; ++b)
        if (a.cu[b] <= t && t < a.cu[b + 1]) lo = b, from = a.cu[b];
    }
    pos = static_cast<int64_t>(a.c.len[lo]) + (t - from);
  }
  int d0, d1;
  chunk_dims(a.rope, c, &d0, &d1);
  float x[16];
  const T* src = static_cast<const T*>(a.q) + t * a.qst + h * a.qsh;
  load_chunk(src + d0, a.vec_q, x);
  load_chunk(src + d1, a.vec_q, x + 8);
  if (16 * c < a.rope.rot) {
    float cs[8], sn[8];
    angles(a.rope, c, pos, cs, sn);
    turn(a.rope, x, cs, sn);
  }
  T* dst = static_cast<T*>(a.qo) + t * a.ost + h * a.osh;
  if (a.vec_q) {
    Act<T>::store8(dst + d0, x);
    Act<T>::store8(dst + d1, x + 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) Act<T>::put(dst + d0 + i, x[i]), Act<T>::put(dst + d1 + i, x[8 + i]);
  }
}

// 16 elements of a row as they are in memory.
template <typename T>
struct Row16 {
  uint4 u[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Row16<T> load_row(const T* row, int d0, int d1, bool vec) {
  Row16<T> r;
  if (vec) {
    constexpr int kHalf = sizeof(T) / 2;  // vectors of eight elements
#pragma unroll
    for (int k = 0; k < kHalf; ++k) {
      r.u[k] = reinterpret_cast<const uint4*>(row + d0)[k];
      r.u[kHalf + k] = reinterpret_cast<const uint4*>(row + d1)[k];
    }
  } else {
    T e[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = row[d0 + k], e[8 + k] = row[d1 + k];
    memcpy(r.u, e, sizeof(e));
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void row_floats(const Row16<T>& r, float* x) {
  T e[16];
  memcpy(e, r.u, sizeof(e));
#pragma unroll
  for (int k = 0; k < 16; ++k) x[k] = Act<T>::get(&e[k]);
}

// The largest of the block's values (none negative, none NaN), in every thread.
template <int NT>
__device__ __forceinline__ float block_max(float v, uint32_t* s) {
  const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(v));  // magnitudes order as their bits
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = m;
  __syncthreads();
  return __uint_as_float(__reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < NT / 32 ? s[threadIdx.x & 31] : 0u));
}

// The first sequence above found[0] that has this candidate and how many have it, into found[0] and found[1]; of one that
// alone has it, its tokens' range into found[2] and found[3].
template <int NT>
__device__ __forceinline__ void append_find(const Kv8AppendArgs& a, int candidate, int* found) {
  const int bs = a.c.block;
  if (threadIdx.x == 0) found[4] = found[0], found[0] = a.c.B, found[1] = 0;
  __syncthreads();
  const int last = found[4];
  for (int b = threadIdx.x; b < a.c.B; b += NT) {
    const int lo = a.cu[b], hi = a.cu[b + 1];
    if (b > last && lo >= 0 && hi >= lo && hi <= a.T && lo / bs + 2 * b <= candidate && candidate < hi / bs + 2 * b + 2) {
      atomicMin(&found[0], b);
      atomicAdd(&found[1], 1);
      found[2] = lo;
      found[3] = hi;
    }
  }
  __syncthreads();
}

// Sequence b's share of a candidate, tokens [first, first + n). A thread holds 16 elements of one slot (NT >= block *
// head_dim / 16). A thread block takes heads_per_cta heads in turn: the angles and the block's place are found once, and a
// head's rows are loaded while the head before is rotated and stored.
template <typename T, int NT>
__device__ __forceinline__ void append_block(const Kv8AppendArgs& a, int tid, int candidate, bool keys, int h0, int b,
                                             int first, int n, uint32_t (*s_amax)[NT / 32]) {
  const int bs = a.c.block, len = a.c.len[b];
  if (!kv8_seq_ok(a.c, a.T, first, first + n, len)) return;
  const int64_t j = static_cast<int64_t>(len / bs) + (candidate - (first / bs + 2 * b));  // the sequence's block
  const int64_t start = j * bs;
  if (n == 0 || start >= static_cast<int64_t>(len) + n) return;
  const int id = a.c.table[static_cast<int64_t>(b) * a.c.max_blocks + j];
  const int s_lo = max(0, static_cast<int>(len - start));  // slots written: [s_lo, s_hi)
  const int s_hi = static_cast<int>(min(static_cast<int64_t>(bs), static_cast<int64_t>(len) + n - start));

  const int tpr = a.c.D / 16, c = tid % tpr, s = tid / tpr;
  const bool written = s >= s_lo && s < s_hi;
  int d0 = 16 * c, d1 = 16 * c + 8;
  if (keys) chunk_dims(a.rope, c, &d0, &d1);
  const bool rotated = written && keys && 16 * c < a.rope.rot;
  const int64_t sh = keys ? a.ksh : a.vsh, t = first + (start + s - len);
  const bool vec = keys ? a.vec_k : a.vec_v;
  const T* src = static_cast<const T*>(keys ? a.k : a.v) + t * (keys ? a.kst : a.vst) + h0 * sh;
  const int heads = min(a.c.H, h0 + a.heads_per_cta) - h0;
  Row16<T> next = {};
  if (written) next = load_row(src, d0, d1, vec);
  if (id < 0 || id >= a.c.num_blocks) return;
  float cs[8], sn[8];
  if (rotated) angles(a.rope, c, a.pos ? a.pos[t] : start + s, cs, sn);
  uint8_t* dst = (keys ? a.c.k : a.c.v) + id * a.c.sb + h0 * a.c.sh + s * a.c.ss;
  uint8_t* scales = (keys ? a.c.ks : a.c.vs) + static_cast<int64_t>(id) * a.c.H + h0;
#pragma unroll 1
  for (int h = 0; h < heads; ++h, dst += a.c.sh) {
    float x[16];
    float amax = 0.f;
    row_floats(next, x);
    if (h + 1 < heads && written) next = load_row(src + (h + 1) * sh, d0, d1, vec);
    if (rotated) turn(a.rope, x, cs, sn);
    if (written) {  // a maximum passes over NaN
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
    }
    const bool infinite = amax == kInf;
    const uint8_t old_byte = scales[h];
    amax = block_max<NT>(amax, s_amax[h & 1]);
    if (amax == kInf) {  // the whole block: the largest finite magnitude again
      amax = 0.f;
      if (written) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float m = fabsf(x[i]);
          if (m < kInf) amax = fmaxf(amax, m);
        }
      }
      __syncthreads();  // the first maxima have been read
      amax = block_max<NT>(amax, s_amax[h & 1]);
    }
    const int old = kv8_exp(old_byte);
    const int need = kv8_need(amax);
    const int e = s_lo > 0 ? max(old, need) : need;
    if (written) {
      const float down = pow2i(-e);
      if (infinite) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (fabsf(x[i]) == kInf) x[i] = __int_as_float(0x7fffffff);
      }
      *reinterpret_cast<uint2*>(dst + d0) = make_uint2(kv8_codes4_finite(x, down), kv8_codes4_finite(x + 4, down));
      *reinterpret_cast<uint2*>(dst + d1) = make_uint2(kv8_codes4_finite(x + 8, down), kv8_codes4_finite(x + 12, down));
    } else if (s < bs && s_lo > 0 && e > old) {  // codes of the block's other entries, rounded to the grown scale
      const float up = pow2i(old - e);
      uint4 w = *reinterpret_cast<const uint4*>(dst + 16 * c);
      uint32_t* q = &w.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float y[4];
        kv8_values4(q[i], y);
        q[i] = kv8_codes4(y, up);
      }
      *reinterpret_cast<uint4*>(dst + 16 * c) = w;
    }
    // every thread has read the old scale before the barrier above
    if (tid == 0) scales[h] = static_cast<uint8_t>(e + 127);
  }
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT) kv8_append_kernel(const __grid_constant__ Kv8AppendArgs a) {
  __shared__ int s_found[5];
  __shared__ uint32_t s_amax[2][NT / 32];
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x < static_cast<unsigned>(a.status_ctas)) return append_status<T, NT>(a);
  if (static_cast<int>(blockIdx.x) - a.status_ctas >= a.item_ctas) return append_queries<T, NT>(a);
  if (threadIdx.x == 0) s_found[0] = -1;
  // Once, but for a candidate of several sequences. What a round needs is found in it again: kept over the rounds it costs
  // registers (80 instead of 64; prompts 40.3 instead of 37.6 us).
  bool more;
#pragma unroll 1
  do {
    int tid, item;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
    asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(item));
    item -= a.status_ctas;
    const int part = item % (2 * a.head_groups), candidate = item / (2 * a.head_groups);
    const bool keys = part < a.head_groups;
    const int h0 = (keys ? part : part - a.head_groups) * a.heads_per_cta;
    append_find<NT>(a, candidate, s_found);
    const int b = s_found[0];
    if (b == a.c.B) return;
    const bool alone = s_found[1] == 1;
    const int first = alone ? s_found[2] : a.cu[b], end = alone ? s_found[3] : a.cu[b + 1];
    append_block<T, NT>(a, tid, candidate, keys, h0, b, first, end - first, s_amax);
    more = s_found[1] > 1;
    if (more) __syncthreads();
  } while (more);
}

template <typename T, int NT>
cudaError_t launch_append(const Kv8AppendArgs& args, cudaStream_t st) {
  Kv8AppendArgs a = args;
  const int tpr = a.c.D / 16;
  // Heads to a thread block: as many as leave 1024 threads for every other SM, so that what is found once for a block's
  // heads (its sequence, its place, the angles) is shared; a step of few tokens spends most of its time on that.
  // 64 sequences x 9 tokens x 8 heads with queries: 10.5 us, 21.3 us where up to 8 times as many threads were asked for;
  // 22,000 tokens x 8 heads: 37.7 us and 42.4 us, 83 us with one head to a thread block.
  const int64_t candidates = a.T / a.c.block + 2 * static_cast<int64_t>(a.c.B);
  a.heads_per_cta = static_cast<int>(std::min<int64_t>(a.c.H, std::max<int64_t>(1, candidates * 2 * a.c.H / (kSms / 2 * (1024 / NT)))));
  a.head_groups = (a.c.H + a.heads_per_cta - 1) / a.heads_per_cta;
  a.item_ctas = static_cast<int>(candidates * 2 * a.head_groups);
  a.status_ctas = (a.c.B + NT / 32 - 1) / (NT / 32);
  const int64_t q_items = a.q ? static_cast<int64_t>(a.T) * a.q_heads * tpr : 0;
  const int64_t ctas = a.status_ctas + static_cast<int64_t>(a.item_ctas) + (q_items + NT - 1) / NT;
  return launch_pdl(kv8_append_kernel<T, NT>, dim3(static_cast<unsigned>(ctas)), dim3(NT), st, a);
}

template <typename T>
cudaError_t launch_append_type(const Kv8AppendArgs& a, cudaStream_t st) {
  const int threads = a.c.block * a.c.D / 16;  // 64 .. 1024: 16 elements each
  if (threads <= 128) return launch_append<T, 128>(a, st);
  if (threads == 256) return launch_append<T, 256>(a, st);
  if (threads == 512) return launch_append<T, 512>(a, st);
  return launch_append<T, 1024>(a, st);
}

// ----------------------------------------------------------------- compact --
//
// One warp owns one head of one plane of one sequence, keys or values, and its
// whole path: the entries are staged as codes in shared memory first, because
// a destination block whose scale grows is rewritten and may hold sources.

constexpr int kCompWarps = 4;

template <int D>
__global__ void __launch_bounds__(kCompWarps * 32) kv8_compact_kernel(const __grid_constant__ Kv8CompactArgs a) {
  constexpr int kTpr = D / 16, kRows = 32 / kTpr;  // lanes per entry, entries per round
  __shared__ __align__(16) uint8_t s_codes[kCompWarps][kKv8MaxPath * D];
  __shared__ int s_path[kKv8MaxPath];
  __shared__ int s_id[kKv8MaxPath];      // source block of each entry
  __shared__ int s_dst[kKv8MaxPath];     // destination block of each entry
  __shared__ int s_state;
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();
  griddep_wait();
  const int L = a.acc[b], base = a.c.len[b];
  const int bs = a.c.block;
  const int64_t cap = static_cast<int64_t>(a.c.max_blocks) * bs;
  const int32_t* table = a.c.table + static_cast<int64_t>(b) * a.c.max_blocks;
  if (warp == 0) {  // 1: move, 2: nothing to move, 0: skipped, else the negated status
    int state = 1;
    if (L < 0) {
      state = 0;
    } else if (base < 0) {
      state = -SPEC_ROW_CACHE;
    } else if (!a.path) {
      state = static_cast<int64_t>(base) + L >= cap ? -SPEC_ROW_TREE : 2;
    } else if (L >= a.Dp) {
      state = -SPEC_ROW_TREE;
    } else {
      bool tree = false, cache = false;
      for (int t = lane; t <= L; t += 32) {
        const int p = a.path[static_cast<int64_t>(b) * a.Dp + t];
        const int prev = t ? a.path[static_cast<int64_t>(b) * a.Dp + t - 1] : -1;
        const bool bad = (t == 0 && p != 0) || p <= prev || static_cast<int64_t>(base) + p >= cap;
        tree |= bad;
        if (bad) continue;
        s_path[t] = p;
        const int src = table[(base + p) / bs], dst = table[(base + t) / bs];  // t <= p: both in the table
        cache |= src < 0 || src >= a.c.num_blocks || dst < 0 || dst >= a.c.num_blocks;
        s_id[t] = src;
        s_dst[t] = dst;
      }
      if (__any_sync(0xffffffffu, tree)) state = -SPEC_ROW_TREE;
      else if (__any_sync(0xffffffffu, cache)) state = -SPEC_ROW_CACHE;
      __syncwarp();
      if (state == 1 && s_path[L] == L) state = 2;
    }
    if (lane == 0) s_state = state;
  }
  __syncthreads();
  const int state = s_state;
  if (blockIdx.x == 0 && tid == 0 && (a.what & kWriteLengths)) {
    a.new_len[b] = state >= 1 ? base + L + 1 : -1;
    a.row_status[b] = state < 0 ? -state : 0;
  }
  if (state != 1 || !(a.what & kMoveEntries)) return;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kCompWarps + warp;  // plane, keys or values, head
  if (item >= static_cast<int64_t>(a.planes) * 2 * a.c.H) return;
  const int h = static_cast<int>(item % a.c.H);
  const int64_t pk = item / a.c.H, plane = pk >> 1;
  uint8_t* codes = ((pk & 1) ? a.c.v : a.c.k) + plane * a.sp + h * a.c.sh;
  uint8_t* scales = ((pk & 1) ? a.c.vs : a.c.ks) + plane * a.ssp + h;
  uint8_t* stage = s_codes[warp];
  const int c = lane % kTpr, r = lane / kTpr;
  for (int t = r; t <= L; t += kRows) {
    const int p = base + s_path[t];
    *reinterpret_cast<uint4*>(stage + t * D + 16 * c) =
        *reinterpret_cast<const uint4*>(codes + s_id[t] * a.c.sb + (p % bs) * a.c.ss + 16 * c);
  }
  // the scale of a source entry's block, before any is written: lanes hold entries lane and lane + 32
  int src_e[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = lane + 32 * i;
    src_e[i] = t <= L ? kv8_exp(scales[static_cast<int64_t>(s_id[t]) * a.c.H]) : 0;
  }
  __syncwarp();
  for (int t0 = 0; t0 <= L;) {  // entries t0 .. t1 - 1 share a destination block
    const int t1 = min(L + 1, t0 + bs - (base + t0) % bs);
    const int64_t dst = s_dst[t0];
    uint8_t* head = codes + dst * a.c.sb;
    const int old = kv8_exp(scales[dst * a.c.H]);
    int e = old;
    for (int t = t0 + r; __any_sync(0xffffffffu, t < t1); t += kRows) {
      const int e0 = __shfl_sync(0xffffffffu, src_e[0], t & 31), e1 = __shfl_sync(0xffffffffu, src_e[1], t & 31);
      const int es = t < 32 ? e0 : e1;
      if (t >= t1) continue;
      const uint4 w = *reinterpret_cast<const uint4*>(stage + t * D + 16 * c);
      const uint32_t* q = &w.x;
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float y[4];
        kv8_values4(q[i], y);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (fabsf(y[k]) <= kKv8Max) amax = fmaxf(amax, fabsf(y[k]));  // NaN codes do not count
      }
      e = max(e, kv8_need(amax * pow2i(es)));
    }
    e = __reduce_max_sync(0xffffffffu, e);
    if (e > old) {
      const float up = pow2i(old - e);
      for (int s = r; s < bs; s += kRows) {
        uint4 w = *reinterpret_cast<const uint4*>(head + s * a.c.ss + 16 * c);
        uint32_t* q = &w.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float y[4];
          kv8_values4(q[i], y);
          q[i] = kv8_codes4(y, up);
        }
        *reinterpret_cast<uint4*>(head + s * a.c.ss + 16 * c) = w;
      }
      __syncwarp();
      if (lane == 0) scales[dst * a.c.H] = static_cast<uint8_t>(e + 127);
    }
    for (int t = t0 + r; __any_sync(0xffffffffu, t < t1); t += kRows) {
      const int e0 = __shfl_sync(0xffffffffu, src_e[0], t & 31), e1 = __shfl_sync(0xffffffffu, src_e[1], t & 31);
      const int es = t < 32 ? e0 : e1;
      if (t >= t1 || (s_path[t] == t && e == old)) continue;
      uint4 w = *reinterpret_cast<const uint4*>(stage + t * D + 16 * c);
      uint32_t* q = &w.x;
      if (es != e) {
        const float by = pow2i(es - e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float y[4];
          kv8_values4(q[i], y);
          q[i] = kv8_codes4(y, by);
        }
      }
      *reinterpret_cast<uint4*>(head + ((base + t) % bs) * a.c.ss + 16 * c) = w;
    }
    __syncwarp();
    t0 = t1;
  }
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, int dtype, cudaStream_t st) {
  if (dtype == SPEC_F32) return launch_append_type<float>(a, st);
  if (dtype == SPEC_BF16) return launch_append_type<__nv_bfloat16>(a, st);
  return launch_append_type<__half>(a, st);
}

cudaError_t launch_kv8_compact(const Kv8CompactArgs& a, cudaStream_t st) {
  const int64_t items = static_cast<int64_t>(a.planes) * 2 * a.c.H;
  const dim3 grid(static_cast<unsigned>((items + kCompWarps - 1) / kCompWarps), static_cast<unsigned>(a.c.B));
  const dim3 block(kCompWarps * 32);
  return a.c.D == 128 ? launch_compaction(kv8_compact_kernel<128>, grid, block, st, a)
                      : launch_compaction(kv8_compact_kernel<64>, grid, block, st, a);
}

}  // namespace specv
