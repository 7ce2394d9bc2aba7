// pages.cu -- the pages of a paged cache between two steps: every sequence keeps
// the first tokens of its own row or of another one's (a fork), blocks behind
// them are given back, free blocks are taken for the next step, and a partly
// filled block that other sequences hold too is copied before it is written.
//
// Three launches, none of which the host waits for. pages_keep: rows and
// reference counts, by atomics whose order does not matter (whole numbers).
// pages_take: one block of threads counts what each sequence takes, ranks the
// free blocks (lowest first) and hands them out in the sequences' order, so the
// result depends on the inputs alone. pages_copy: the copies of all pools.
//
// Who copies: of the c sequences of a call that go on writing the same partly
// filled block, held by r sequences in all, every one where c < r; where c = r,
// all but the last, which keeps it.
//
// What bounds it. 64 sequences after a step: 8.9 us, the three launches' chain. Four
// prompts forked to 64 sequences, 60 blocks of 74 KB copied in 32 planes: 27.5 us,
// 142 MB of stores (the sources come from L2 after their first reader).
#include <limits.h>

#include "internal.h"
#include "latent.h"

namespace specv {

namespace {

// What a sequence asks for, checked; the same in every kernel.
struct Ask {
  int source, keep, kept, need;  // kept: blocks of the first `keep` tokens
  bool sound;
};

__device__ __forceinline__ Ask ask_of(const PagesArgs& a, int b) {
  Ask k;
  k.source = a.source ? a.source[b] : b;
  k.need = a.need ? a.need[b] : 0;
  k.sound = k.source >= 0 && k.source < a.B && k.need >= 0;
  const int len = k.sound ? a.len[k.source] : 0;
  k.keep = a.keep ? a.keep[b] : len;
  k.sound = k.sound && k.keep >= 0 && k.keep <= len && k.keep <= static_cast<int64_t>(a.M) * a.block;
  if (!k.sound) k.keep = k.need = 0;
  k.kept = static_cast<int>((static_cast<int64_t>(k.keep) + a.block - 1) / a.block);
  return k;
}

constexpr int kKeepThreads = 256;

__global__ void __launch_bounds__(kKeepThreads) pages_keep_kernel(const __grid_constant__ PagesArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int64_t cta = static_cast<int64_t>(b) * gridDim.x + blockIdx.x, all = static_cast<int64_t>(gridDim.x) * gridDim.y;
  for (int64_t i = cta * kKeepThreads + tid; i < a.num_blocks; i += all * kKeepThreads) a.sharers[i] = 0, a.last_sharer[i] = -1;
  const Ask k = ask_of(a, b);
  const int32_t* mine = a.table + static_cast<int64_t>(b) * a.M;
  const int32_t* from = a.table + static_cast<int64_t>(k.sound ? k.source : b) * a.M;
  int32_t* to = a.new_table + static_cast<int64_t>(b) * a.M;
  const bool fork = k.source != b;
  bool bad = false;
  const int end = min(a.M, (static_cast<int>(blockIdx.x) + 1) * kPagesChunk);
  for (int j = blockIdx.x * kPagesChunk + tid; j < end; j += kKeepThreads) {
    const int old = mine[j], id = j < k.kept ? (fork ? from[j] : old) : -1;
    const bool held = old >= 0 && old < a.num_blocks, kept = id >= 0 && id < a.num_blocks;
    if (j < k.kept && !kept) bad = true;
    if (fork || j >= k.kept) {
      if (held) atomicSub(&a.refs[old], 1);
      if (kept) atomicAdd(&a.refs[id], 1);
    }
    if (to != mine || id != old) to[j] = id;
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) a.unsound[static_cast<int64_t>(b) * a.chunks + blockIdx.x] = bad;
}

constexpr int kTakeThreads = 1024;

// Sum of x over the threads before this one, and over all of them.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* total, int64_t* s_warp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[31];
  const int64_t before = (warp ? s_warp[warp - 1] : 0) + v - x;
  __syncthreads();
  return before;
}

__global__ void __launch_bounds__(kTakeThreads) pages_take_kernel(const __grid_constant__ PagesArgs a) {
  __shared__ int64_t s_warp[32];
  __shared__ int s_copies;
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  if (tid == 0) s_copies = 0;
  // The block that b's next token goes into, where that holds tokens already and b asks for room; -1: none. `more`: blocks
  // it needs behind its own; -1: they pass the table.
  auto writes = [&](int b, const Ask& k, int* more) {
    const int64_t blocks = (static_cast<int64_t>(k.keep) + k.need + a.block - 1) / a.block;
    *more = k.need == 0 ? 0 : (blocks > a.M ? -1 : static_cast<int>(blocks - k.kept));
    if (*more < 0 || k.need == 0 || k.keep % a.block == 0) return -1;
    const int id = a.new_table[static_cast<int64_t>(b) * a.M + k.kept - 1];
    return id >= 0 && id < a.num_blocks ? id : -1;
  };
  for (int b = tid; b < a.B; b += kTakeThreads) {
    const Ask k = ask_of(a, b);
    int more;
    const int id = writes(b, k, &more);
    if (id < 0 || a.refs[id] < 2) continue;
    atomicAdd(&a.sharers[id], 1);
    atomicMax(&a.last_sharer[id], b);
  }
  __syncthreads();
  int64_t want = 0;
  for (int base = 0; base < a.B; base += kTakeThreads) {
    const int b = base + tid;
    int n = 0, copy = -1, kept = 0, keep = 0, flags = 0;
    if (b < a.B) {
      const Ask k = ask_of(a, b);
      int more;
      const int id = writes(b, k, &more);
      n = max(more, 0);
      kept = k.kept, keep = k.keep;
      flags = (k.sound ? 0 : 1) | (k.need > 0 ? 2 : 0) | (more < 0 ? 4 : 0);
      if (id >= 0 && a.refs[id] >= 2 && !(a.sharers[id] >= a.refs[id] && a.last_sharer[id] == b)) copy = id, ++n;
    }
    int64_t total;
    const int64_t at = want + block_scan(n, &total, s_warp);
    if (b < a.B) {
      a.take[2 * b] = make_int4(static_cast<int>(min(at, static_cast<int64_t>(INT_MAX))), n, kept - (copy >= 0), copy);
      a.take[2 * b + 1] = make_int4(keep, flags & 1, flags & 2, flags & 4);
    }
    want += total;
  }
  // the free blocks, lowest first, as many as are asked for
  int64_t found = 0;
  for (int base = 0; base < a.num_blocks && found < want; base += 4 * kTakeThreads) {
    const int i = base + 4 * tid;
    int free[4], n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      free[k] = i + k < a.num_blocks && a.refs[i + k] == 0;
      n += free[k];
    }
    int64_t total;
    int64_t at = found + block_scan(n, &total, s_warp);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (free[k]) a.free_ids[at++] = i + k;
    found += total;
  }
  __syncthreads();
  // eight lanes per sequence
  const int sub = tid & 7;
  for (int b = tid >> 3; b < a.B; b += kTakeThreads / 8) {
    const int4 t = a.take[2 * b], k = a.take[2 * b + 1];
    const bool shorts = k.z && (k.w || static_cast<int64_t>(t.x) + t.y > found);
    int32_t* row = a.new_table + static_cast<int64_t>(b) * a.M;
    int dst = -1;
    if (!shorts)
      for (int i = sub; i < t.y; i += 8) {
        const int id = a.free_ids[t.x + i];
        row[t.z + i] = id;
        a.refs[id] = 1;
        if (i == 0) dst = id;
      }
    if (sub == 0) {
      bool bad = k.y || shorts;
      for (int c = 0; c < a.chunks; ++c) bad |= a.unsound[static_cast<int64_t>(b) * a.chunks + c] != 0;
      a.row_status[b] = bad ? SPEC_ROW_CACHE : 0;
      a.new_len[b] = k.x;
      if (t.w >= 0 && !shorts) {
        atomicSub(&a.refs[t.w], 1);
        a.copies[atomicAdd(&s_copies, 1)] = make_int2(t.w, dst);
      }
    }
  }
  __syncthreads();
  if (tid == 0) *a.n_copies = s_copies;
}

constexpr int kCopyThreads = 256;

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ PagesArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int n = *a.n_copies, tid = threadIdx.x;
  for (int p = 0; p < a.n_pools; ++p) {
    const PagesPool& pool = a.pool[p];
    const int64_t all = static_cast<int64_t>(n) * pool.planes * pool.pieces;
    for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
      const int64_t block = i / pool.pieces;  // copy, plane
      const int piece = static_cast<int>(i - block * pool.pieces), c = static_cast<int>(block / pool.planes);
      const int64_t plane = block - static_cast<int64_t>(c) * pool.planes;
      const int2 move = a.copies[c];
      const int64_t off = static_cast<int64_t>(piece) * kPagesPiece;
      const int bytes = static_cast<int>(min(pool.bytes - off, static_cast<int64_t>(kPagesPiece)));
      const uint8_t* src = pool.base + plane * pool.sp + move.x * pool.sb + off;
      uint8_t* dst = pool.base + plane * pool.sp + move.y * pool.sb + off;
      if (pool.vec) {
        uint4 u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (16 * (tid + k * kCopyThreads) < bytes) u[k] = reinterpret_cast<const uint4*>(src)[tid + k * kCopyThreads];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (16 * (tid + k * kCopyThreads) < bytes) reinterpret_cast<uint4*>(dst)[tid + k * kCopyThreads] = u[k];
      } else {
        for (int k = tid; k < bytes; k += kCopyThreads) dst[k] = src[k];
      }
    }
  }
}

}  // namespace

cudaError_t launch_pages_update(const PagesArgs& a, cudaStream_t st) {
  cudaError_t e = launch_pdl(pages_keep_kernel, dim3(a.chunks, a.B), dim3(kKeepThreads), st, a);
  if (e == cudaSuccess) e = launch_pdl(pages_take_kernel, dim3(1), dim3(kTakeThreads), st, a);
  if (e != cudaSuccess || a.n_pools == 0) return e;
  int64_t most = 0;  // pieces when every sequence copies
  for (int p = 0; p < a.n_pools; ++p) most += static_cast<int64_t>(a.B) * a.pool[p].planes * a.pool[p].pieces;
  const unsigned ctas = static_cast<unsigned>(most < 8 * kSms ? most : 8 * kSms);
  return launch_pdl(pages_copy_kernel, dim3(ctas), dim3(kCopyThreads), st, a);
}

}  // namespace specv
