// kv8_attn.cuh -- what the attention kernels over the 8-bit paged cache share:
// the split of the tiles over the thread blocks, and the join of cut items.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "kv8.h"
#include "tc.cuh"

namespace specv {

namespace {

using namespace tc;

constexpr int kTile = 128;
constexpr int kMetaRing = 8;
constexpr int kGaveUp = 1, kOutside = 2;  // of a part: a wait ran out; it met a page outside the pool
constexpr int kMaxPages = kTile / 16;
constexpr float kNegInf = -__builtin_huge_valf();

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

// -------------------------------------------------------------- schedule --

// One row tile of a sequence, all KV heads alike.
struct RowTile {
  int b, rt;
  int first;  // first packed token of the sequence
  int n;      // its step tokens
  int ctx;    // tokens in the cache before the step
  int rows;   // rows of this tile
  int end;    // slots that some row of it may see
  int tiles;  // ceil(end / 128); 0: no such row tile
  int part;   // from this tile on some row does not see every slot
};

template <int N>
__device__ __forceinline__ RowTile row_tile(const Kv8AttnArgs& a, int b, int rt) {
  RowTile r{};
  r.b = b;
  r.rt = rt;
  const int lo = a.cu[b], hi = a.cu[b + 1], len = a.c.len[b];
  if (!kv8_seq_ok(a.c, a.T, lo, hi, len) || hi - lo > a.max_tokens) return r;
  const int rows = (hi - lo) * a.group, r0 = rt * N;  // below 2^31: the host has checked all rows
  if (r0 >= rows) return r;
  r.first = lo;
  r.n = hi - lo;
  r.ctx = len;
  r.rows = min(rows - r0, N);
  r.end = len + (a.tree ? r.n : (r0 + r.rows - 1) / a.group + 1);
  r.tiles = (r.end + kTile - 1) / kTile;
  r.part = (len + (a.tree ? 0 : r0 / a.group + 1)) / kTile;
  return r;
}

// Where a run begins: an item, and a unit of it.
struct Start {
  int b, rt, h, t;
};

// An item has COST units for its queries and results, then one for each tile. Parts are equal runs of the units of all
// items, the first `more` of them one longer; an item begins in the part of its first tile.
struct Runs {
  int64_t all, each;  // units, units of a run
  int parts, more;
  __device__ __forceinline__ int64_t begin(int part) const { return part * each + min(part, more); }
};

// All threads of the block: the runs, and where the part's first unit lies. False
// where it has no tile. s_tmp: 64 words of shared memory.
template <int N, int COST>
__device__ __forceinline__ bool find_run(const Kv8AttnArgs& a, int part, Runs* runs, Start* s, int* s_tmp) {
  const int nthr = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = nthr >> 5;
  const uint32_t cand = static_cast<uint32_t>(a.c.B) * static_cast<uint32_t>(a.row_tiles);  // below 2^31
  // Units of the candidates base .. base + nthr - 1, one a thread, their sums up to this one's, and all.
  auto scan = [&](uint32_t base, int* units, int64_t* upto, int64_t* sum) {
    const uint32_t i = base + tid;
    int v = 0;
    if (i < cand) {
      const uint32_t b = i / static_cast<uint32_t>(a.row_tiles);
      v = row_tile<N>(a, static_cast<int>(b), static_cast<int>(i - b * a.row_tiles)).tiles;
      if (v > 0) v += COST;
    }
    int64_t x = v;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    int64_t* at = reinterpret_cast<int64_t*>(s_tmp);
    if (lane == 31) at[warp] = x;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll 1
    for (int w = 0; w < nw; ++w) {
      if (w < warp) before += at[w];
      total += at[w];
    }
    __syncthreads();
    *units = v;
    *upto = x + before;
    *sum = total;
  };
  int64_t total = 0, want = 0, run = 0;
  bool found = true;
  // the first round's sums serve both the total and the search, as long as there is one round
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (uint32_t base = 0; base < cand; base += nthr) {
      int v;
      int64_t upto, sum;
      scan(base, &v, &upto, &sum);
      if (pass == 0) total += sum;
      if (pass == 0 && cand <= static_cast<uint32_t>(nthr)) pass = 1;
      if (pass == 0) continue;
      if (run == 0 && base == 0) {
        const int64_t all = total * a.c.H;
        runs->all = all;
        runs->parts = static_cast<int>(min(static_cast<int64_t>(a.parts), all));
        if (part >= runs->parts) {
          found = false;
          break;
        }
        runs->each = all / runs->parts;
        runs->more = static_cast<int>(all - runs->each * runs->parts);
        want = runs->begin(part);
      }
      const int64_t from = (run + upto - v) * a.c.H;
      if (v > 0 && want >= from && want < (run + upto) * a.c.H) {
        const uint32_t i = base + tid, b = i / static_cast<uint32_t>(a.row_tiles);
        int64_t off = want - from;
        int h = 0;
        for (; off >= v; off -= v) ++h;  // at most kv_heads steps
        s_tmp[0] = static_cast<int>(b);
        s_tmp[1] = static_cast<int>(i - b * a.row_tiles);
        s_tmp[2] = h;
        s_tmp[3] = static_cast<int>(off);
      }
      run += sum;
      if (run * a.c.H > want) break;  // the same for every thread
    }
    if (cand == 0 || !found) break;
  }
  __syncthreads();
  s->b = s_tmp[0];
  s->rt = s_tmp[1];
  s->h = s_tmp[2];
  s->t = s_tmp[3];
  __syncthreads();
  return found && runs->begin(part + 1) - runs->begin(part) > max(0, COST - s->t);
}

// Walks the items of a run: (r, h) with tiles [t0, t1).
template <int N, int COST>
struct Walk {
  RowTile r;
  int h, t0, t1;
  int64_t left;  // units of the run from t0 on

  __device__ __forceinline__ Walk(const Kv8AttnArgs& a, const Start& s, int64_t count) {
    r = row_tile<N>(a, s.b, s.rt);
    h = s.h;
    t0 = max(0, s.t - COST);
    left = count - max(0, COST - s.t);
    clip();
  }
  __device__ __forceinline__ void clip() { t1 = static_cast<int>(min(static_cast<int64_t>(r.tiles), t0 + left)); }
  // The next item, if any is left.
  __device__ __forceinline__ bool next(const Kv8AttnArgs& a) {
    left -= t1 - t0 + COST;
    if (left <= 0) return false;
    t0 = 0;
    if (++h == a.c.H) {
      h = 0;
      int b = r.b, rt = r.rt;
      do {
        if (++rt == a.row_tiles) {
          rt = 0;
          ++b;
        }
        if (b >= a.c.B) {  // cannot be: the run's units were counted
          left = 0;
          return false;
        }
        r = row_tile<N>(a, b, rt);
        if (r.tiles == 0) rt = a.row_tiles - 1;  // no further row tile in this sequence
      } while (r.tiles == 0);
    }
    clip();
    return true;
  }
};

// Byte offset of element (row, byte) in a tile of rows of ROW bytes, swizzled as bulk tensor copies do.
template <int ROW>
__device__ __forceinline__ uint32_t swz(int row, int byte) {
  const uint32_t o = static_cast<uint32_t>(row * ROW + byte);
  return ROW == 128 ? o ^ ((o >> 3) & 0x70u) : o ^ ((o >> 3) & 0x30u);
}

// 2^d of a whole d <= 127, exact; 0 below -126 and for -inf, NaN for NaN.
__device__ __forceinline__ float exp2_whole(float d) {
  const float p = __int_as_float((static_cast<int>(fmaxf(d, -127.f)) + 127) << 23);
  return d != d ? d : p;
}

// Bit 7 of a byte of the result is set where w holds a NaN code there.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; }

// Whether the step's token i sees its token j.
__device__ __forceinline__ bool sees(const Kv8AttnArgs& a, int b, int i, int j) {
  return a.tree ? a.tree[(static_cast<int64_t>(b) * a.max_tokens + i) * a.max_tokens + j] != 0 : j <= i;
}

// What the join needs to know of a part's last item.
template <int N>
__device__ __forceinline__ int4 cut_item(const Runs& runs, int part, const RowTile& r, int h, int t0, int t1) {
  if (t0 > 0 || t1 == r.tiles) return make_int4(0, 0, 0, 0);
  const int64_t end = runs.begin(part + 1) - t1 + r.tiles;
  int n = 2;
  while (runs.begin(part + n) < end) ++n;
  return make_int4(r.b, r.rt, h, n);
}

// The copying warp: the pages of each tile's keys, then of its values, into a
// ring of NS slots, and of each page of the tile 2^ek, ev and 2^-ev into sm.page (of
// a page outside the pool 1, 0 and 1: its slots hold what was there before, and the
// join finds the rows that see them). Returns the number of ring slots that copies were begun into.
template <int N, int COST, int D, int NS, typename S>
__device__ __forceinline__ uint32_t copy_tiles(const Kv8AttnArgs& a, const Start& start, int64_t count,
                                               const CUtensorMap& kmap, const CUtensorMap& vmap, uint8_t* ring, S& sm,
                                               volatile int* gave_up) {
  const int lane = threadIdx.x & 31;
  Walk<N, COST> it(a, start, count);
  const int bs = a.c.block, ppt = kTile / bs;
  uint32_t fill = 0, begun = 0;
  int i = 0;
  bool ok = true;
  do {
    const int pages = (it.r.end + bs - 1) / bs;
    const int32_t* table = a.c.table + static_cast<int64_t>(it.r.b) * a.c.max_blocks;
    // 32 pages' ids and scales at a time, one a lane; those of the next 32 are on their way meanwhile
    auto page_id = [&](int page) {
      int id = -1;  // behind the sequence
      if (page < pages) {
        id = table[page];
        if (id < 0 || id >= a.c.num_blocks) id = -2;  // outside the pool
      }
      return id;
    };
    auto scale_at = [&](const uint8_t* scales, int id) {
      return id >= 0 ? scales[static_cast<int64_t>(id) * a.c.H + it.h] : static_cast<uint8_t>(127);
    };
    int id = -1, id_next = page_id(it.t0 * ppt + lane);
    uint8_t ke = 127, ve = 127, ke_next = scale_at(a.c.ks, id_next), ve_next = scale_at(a.c.vs, id_next);
#pragma unroll 1
    for (int t = it.t0, g = 0; t < it.t1 && ok; ++t, g += ppt, ++i) {
      if ((g & 31) == 0) {
        id = id_next;
        ke = ke_next;
        ve = ve_next;
        id_next = page_id(t * ppt + 32 + lane);
        if (__any_sync(0xffffffffu, id == -2)) sm.outside = 1;
      }
      if ((g & 31) == 16) {
        ke_next = scale_at(a.c.ks, id_next);
        ve_next = scale_at(a.c.vs, id_next);
      }
      const int from = (g & 31) + (lane & (ppt - 1));
      const int my_id = __shfl_sync(0xffffffffu, id, from);
      const bool mine = lane < ppt && my_id >= 0;
      const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, mine)) * bs * D);
      auto at = [&](int name) { return name == 0 ? 0 : (name == 1 ? it.h : my_id); };
      const int x1 = at(a.order & 3), x2 = at((a.order >> 2) & 3), x3 = at((a.order >> 4) & 3);
#pragma unroll 1
      for (int part = 0; part < 2; ++part, ++fill) {
        const uint32_t slot = fill % NS, bar = smem_addr(&sm.full[slot]);
        if (fill >= NS) ok = bar_wait(smem_addr(&sm.empty[slot]), (fill / NS - 1) & 1, gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;  // no copy is started any more
        begun = fill + 1;
        // the copies begin before the scales are there; the barrier's one arrival comes after both
        if (mine)
          load_4d(smem_addr(ring + slot * (kTile * D) + lane * bs * D), part == 0 ? &kmap : &vmap, bar, 0, x1, x2, x3);
        if (part == 0) {
          const int my_ke = kv8_exp(static_cast<uint8_t>(__shfl_sync(0xffffffffu, static_cast<int>(ke), from))),
                    my_ve = kv8_exp(static_cast<uint8_t>(__shfl_sync(0xffffffffu, static_cast<int>(ve), from)));
          if (lane < ppt)
            sm.page[i % kMetaRing][lane] = make_float4(pow2i(my_ke), static_cast<float>(my_ve), pow2i(-my_ve), 0.f);
        }
        __syncwarp();
        if (lane == 0) bar_expect(bar, bytes);
      }
    }
  } while (ok && it.next(a));
  return begun;
}

// The end of a block in which a wait gave up, all threads: copies and products that are still in flight write this block's
// memory, so the two warps that began them wait for them (with a limit).
template <int NS, typename S>
__device__ __forceinline__ void drain(S& sm, bool copied, uint32_t begun, bool issued) {
  if (copied)
#pragma unroll 1
    for (uint32_t f = begun > NS ? begun - NS : 0; f < begun; ++f)
#pragma unroll 1
      for (int k = 0; k < (1 << 16) && !bar_try(smem_addr(&sm.full[f % NS]), (f / NS) & 1); ++k) {
      }
  if (issued) {
    if (elect()) commit(smem_addr(&sm.drain));
#pragma unroll 1
    for (int k = 0; k < (1 << 16) && !bar_try(smem_addr(&sm.drain), 0); ++k) {
    }
  }
  __syncthreads();
}

// -------------------------------------------------------------------- join --
//
// Adds the shares of items that runs cut. Block x takes the item that begins in
// part x and ends behind it, a warp one row at a time: shares in the order of the
// parts, each times 2^(its reference - the largest). The last blocks check sequences,
// and make the rows NaN that see an entry of a page outside the pool. (A cut item's
// rows are made so by both.)

// Whether step token i of sequence b (ctx tokens before the step, n in it) sees an entry of a page outside the pool; a warp.
__device__ __forceinline__ bool sees_outside(const Kv8AttnArgs& a, int b, int ctx, int n, int i) {
  const int bs = a.c.block, pages = (ctx + n + bs - 1) / bs;
  bool hit = false;
#pragma unroll 1
  for (int p = threadIdx.x & 31; p < pages; p += 32) {
    const int id = a.c.table[static_cast<int64_t>(b) * a.c.max_blocks + p];
    if (id >= 0 && id < a.c.num_blocks) continue;
    hit |= p * bs < ctx;
    for (int j = max(0, p * bs - ctx); j < min(n, (p + 1) * bs - ctx); ++j) hit |= sees(a, b, i, j);
  }
  return __any_sync(0xffffffffu, hit);
}

constexpr int kJoinThreads = 256;

template <typename QT, int D, int N>
__global__ void __launch_bounds__(kJoinThreads) kv8_join_kernel(const __grid_constant__ Kv8AttnArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_launch_dependents();
  if (blockIdx.x >= static_cast<unsigned>(a.parts)) {  // a warp per sequence: row_status
    griddep_wait();
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
          for (int d = lane; d < D; d += 32)
            static_cast<QT*>(a.out)[t * a.ost + h * a.osh + d] = from_f<QT>(__int_as_float(0x7fffffff));
      }
    }
    return;
  }
  griddep_wait();
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
    if (top == kNegInf) top = 0.f;
    constexpr int V = D / 32;
    float acc[V] = {}, sum = 0.f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float2 ml = a.part_ml[share(i)];
      const float* p = a.part_o + share(i) * D + lane * V;
      float x[V];
      if (V == 4) {
        const float4 u = *reinterpret_cast<const float4*>(p);
        x[0] = u.x, x[1] = u.y, x[V - 2] = u.z, x[V - 1] = u.w;
      } else {
        const float2 u = *reinterpret_cast<const float2*>(p);
        x[0] = u.x, x[1] = u.y;
      }
      const float w = exp2_whole(ml.x - top);
      sum = fmaf(w, ml.y, sum);
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] = fmaf(w, x[k], acc[k]);
    }
    const int item_row = item.y * N + row, tok = item_row / a.group;
    QT* out = static_cast<QT*>(a.out) + (r.first + static_cast<int64_t>(tok)) * a.ost +
              (item.z * a.group + (item_row - tok * a.group)) * a.osh + lane * V;
    float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (outside && sees_outside(a, item.x, r.ctx, r.n, tok)) inv = __int_as_float(0x7fffffff);
#pragma unroll
    for (int k = 0; k < V; ++k) out[k] = from_f<QT>(acc[k] * inv);
  }
}


// The join of an attention launch with row tiles of N rows.
template <typename QT, int D, int N>
cudaError_t launch_join(const Kv8AttnArgs& a, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.max_tokens) * a.group;
  const int groups = static_cast<int>((rows < N ? rows : N) + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  const int y = groups < 8 ? groups : 8;
  const int checks = (a.c.B + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  return launch_pdl(kv8_join_kernel<QT, D, N>, dim3(static_cast<unsigned>(a.parts + checks), static_cast<unsigned>(y)),
                    dim3(kJoinThreads), st, a);
}

// One launch of an attention kernel, allowed to start while its predecessor drains.
template <typename K>
cudaError_t launch_tiles(K kernel, const Kv8AttnArgs& a, int threads, int smem, const CUtensorMap& k, const CUtensorMap& v,
                         cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.parts));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, k, v);
}

}  // namespace
}  // namespace specv
