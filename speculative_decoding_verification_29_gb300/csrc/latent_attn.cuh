// latent_attn.cuh -- what the attention kernels over the paged latent cache
// share: elements, copies and the join of cut items.
#pragma once

#include "kv8_attn.cuh"
#include "latent.h"

namespace specv {

namespace {

constexpr float kUnset = -3.0e38f;  // the reference of a row that has seen nothing
constexpr float kPass = 8.f;        // by how much (log2) scores may pass what set a row's reference

// kBelow: how far (log2) a reference is set below the row's largest score. bf16 weights keep their precision at any size. fp16
// weights lose bits below 2^-14 and vanish below 2^-25, and have room up to 2^15. 131,072 entries 25.2 bits below one that leads
// weigh 0.34% together: with references at the largest score all of it is lost, with these 0.15% (in bf16 as well), because the
// tensor cores cut what they add at 2^-25 of the running sum's power of two.
template <typename T>
struct Bits;
template <>
struct Bits<__nv_bfloat16> {
  static constexpr float kBelow = 0.f;
  static constexpr uint32_t kFormat = 1, kExp = 0x7f807f80u, kStep = 0x00800080u;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
};
template <>
struct Bits<__half> {
  static constexpr float kBelow = 7.f;
  static constexpr uint32_t kFormat = 0, kExp = 0x7c007c00u, kStep = 0x04000400u;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
};

// 16 bytes from global to shared memory, asynchronously; zeros where `take` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Four lanes hold four rows' 16-byte units u[0 .. 3]; afterwards lane l of them holds unit l of each row, so that four lanes
// store 64 bytes of a row together.
__device__ __forceinline__ void turn_units(uint4* u, int lane) {
  auto swap = [&](uint4& a, uint4& b, int bit) {  // the lane without the bit gives b for the other's a
    const bool up = lane & bit;
    uint4 v = up ? a : b;
    v.x = __shfl_xor_sync(0xffffffffu, v.x, bit), v.y = __shfl_xor_sync(0xffffffffu, v.y, bit);
    v.z = __shfl_xor_sync(0xffffffffu, v.z, bit), v.w = __shfl_xor_sync(0xffffffffu, v.w, bit);
    if (up) a = v;
    else b = v;
  };
  swap(u[0], u[1], 1);
  swap(u[2], u[3], 1);
  swap(u[0], u[2], 2);
  swap(u[1], u[3], 2);
}

// Clears a slot's chunks of 16 bytes in shared memory where the slot lies behind the rows' last; else only the elements that
// are not finite. True where it met such a one. An exponent of ones carries into the sign's place. Neighbouring slots lie 128
// bytes apart, so each begins at another chunk (`first`): else all would ask the same banks.
template <typename B, int CHUNKS>
__device__ __forceinline__ bool clean_chunks(uint4* row, int first, bool behind) {
  uint32_t hit = 0;
#pragma unroll
  for (int k = 0; k < CHUNKS; ++k) {
    if (behind) {
      row[k ^ first] = make_uint4(0, 0, 0, 0);
    } else {
      const uint4 u = row[k ^ first];
      hit |= ((u.x & B::kExp) + B::kStep) | ((u.y & B::kExp) + B::kStep) | ((u.z & B::kExp) + B::kStep) | ((u.w & B::kExp) + B::kStep);
    }
  }
  if (!(hit & 0x80008000u)) return false;
  uint32_t* w = reinterpret_cast<uint32_t*>(row);
#pragma unroll 1
  for (int k = 0; k < 4 * CHUNKS; ++k) w[k] &= ~__vcmpeq2(w[k] & B::kExp, B::kExp);
  return true;
}

// A descriptor of smem_desc's, its address moved by `bytes`. (Told to be uniform by a shuffle, as the roles' warp is, it costs 1
// to 2% of the kernels' time.)
__device__ __forceinline__ uint64_t moved(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }

// What a tensor memory load has brought is used behind this only (after wait_ld).
template <int C>
__device__ __forceinline__ void settle(uint32_t* r) {
#pragma unroll
  for (int k = 0; k < C; ++k) asm volatile("" : "+r"(r[k]));
}

__device__ __forceinline__ void load_3d(uint32_t dst, const void* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// -------------------------------------------------------------- schedule --
//
// Two orders of the items' tiles over the thread blocks. In a row (Runs of kv8_attn.cuh): every block an equal run of all
// items' tiles. In gangs: `gang` blocks, one for each item of a sequence, walk the same tiles at the same time, so that the
// cache is read from memory once; a gang takes an equal run of the sequences' tiles.
// In a row and in gangs, us: two sequences of 110,001 to 131,072 tokens, 18 items each: 794, 675; 68 items, which leave 16 SMs
// idle: 2673, 2471; 64 sequences of 1500 to 6500, 6 items each: 370, 299; 16 trees of 500 to 3500, 16 items: 143, 142. Where L2
// holds the cache there is less to gain: two of 20,000 to 30,000, 76 items: 554, 539; 68 items: 487, 534; 62 items, whose 28 idle
// SMs are more than an eighth: 448, 530.

constexpr int kWhole = 1 << 30;  // rows of a row tile that is all of a sequence

// Where the block's run begins; false where it has no tile.
template <int N, int COST>
__device__ __forceinline__ bool find_items(const LatentAttnArgs& a, Runs* runs, Start* start, int* s_tmp) {
  if (!a.gang) return find_run<N, COST>(a, blockIdx.x, runs, start, s_tmp);
  Kv8AttnArgs g = a;
  g.row_tiles = g.c.H = 1;
  g.parts = a.parts / a.gang;
  return find_run<kWhole, COST>(g, blockIdx.x / a.gang, runs, start, s_tmp);
}

// Walks the items of a block: (r, h) with tiles [t0, t1), which may be none of them.
template <int N, int COST>
struct Items {
  RowTile r, seq;  // seq: in gangs, the sequence
  int h, t0, t1;
  int from, to;    // the run's tiles of the sequence, or of the item
  int64_t left;    // units of the run from `from` on

  __device__ __forceinline__ Items(const LatentAttnArgs& a, const Start& s, int64_t count) {
    h = s.h;
    from = max(0, s.t - COST);
    left = count - max(0, COST - s.t);
    take(a, s.b, s.rt);
  }
  __device__ __forceinline__ void take(const LatentAttnArgs& a, int b, int rt) {
    if (a.gang) {
      seq = row_tile<kWhole>(a, b, 0);
      const int item = static_cast<int>(blockIdx.x) % a.gang;
      h = item % a.c.H;
      r = row_tile<N>(a, b, item / a.c.H);
    } else {
      r = row_tile<N>(a, b, rt);
      seq = r;
    }
    to = static_cast<int>(min(static_cast<int64_t>(seq.tiles), from + left));
    t0 = min(from, r.tiles);
    t1 = min(to, r.tiles);
  }
  // The next item, if any is left.
  __device__ __forceinline__ bool next(const LatentAttnArgs& a) {
    left -= to - from + COST;
    if (left <= 0) return false;
    from = 0;
    int b = seq.b, rt = seq.rt;
    if (!a.gang && ++h < a.c.H) {
      take(a, b, rt);
      return true;
    }
    if (!a.gang) h = 0;
    do {
      if (a.gang || ++rt == a.row_tiles) {
        rt = 0;
        ++b;
      }
      if (b >= a.c.B) {  // cannot be: the run's units were counted
        left = 0;
        return false;
      }
      take(a, b, rt);
      if (seq.tiles == 0) rt = a.row_tiles - 1;  // no further row tile in this sequence
    } while (seq.tiles == 0);
    return true;
  }
  // What the join needs to know where the item begins in the run and ends behind it.
  __device__ __forceinline__ void cut(const LatentAttnArgs& a, const Runs& runs) const {
    int4* at = a.cut + 2 * blockIdx.x;
    at[0] = make_int4(0, 0, 0, 0);
    if (t0 > 0 || t1 == r.tiles) return;
    const int part = a.gang ? blockIdx.x / a.gang : blockIdx.x;
    const int64_t end = runs.begin(part + 1) - to + r.tiles;
    int n = 2;
    while (runs.begin(part + n) < end) ++n;
    at[0] = make_int4(r.b, r.rt, h, n);
    at[1] = make_int4(r.first, r.rows, r.ctx, r.n);
  }
};

// -------------------------------------------------------------------- join --
//
// As kv8_join_kernel, for items of up to 512 dimensions (item.z of a row's a.c.D): block x adds the shares of the item that begins in part x and ends
// behind it, a warp 128 dimensions of one row at a time; the last blocks check sequences, and make the rows NaN that see an entry of a page
// outside the pool.

template <typename QT, int N>
__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(const __grid_constant__ LatentAttnArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, C = a.c.D, D = a.item_dims;
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
  const int4 item = a.cut[2 * blockIdx.x], seq = a.cut[2 * blockIdx.x + 1];  // seq: first token, rows, context, step tokens
  const int n = item.w;
  if (n == 0) return;
  const int64_t first = blockIdx.x, step = a.gang ? a.gang : 1;  // shares of an item lie `step` parts apart
  const int chunks = (D + 127) / 128, units = seq.y * chunks;
  bool outside = false;
  for (int i = lane; i < n; i += 32) outside |= (a.gave_up[first + i * step] & kOutside) != 0;
  outside = __any_sync(0xffffffffu, outside);
#pragma unroll 1
  for (int unit = blockIdx.y * (kJoinThreads / 32) + warp; unit < units; unit += gridDim.y * (kJoinThreads / 32)) {
    const int row = unit / chunks, d = (unit - row * chunks) * 128 + 4 * lane;
    auto share = [&](int i) { return (2 * (first + i * step) + (i == 0 ? 1 : 0)) * N + row; };
    float top = kNegInf;
    for (int i = lane; i < n; i += 32) top = fmaxf(top, a.part_ml[share(i)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll 1
    for (int base = 0; base < n; base += 32) {  // a share a lane, then all lanes through the shares
      float w = 0.f;
      if (base + lane < n) {
        const float2 ml = a.part_ml[share(base + lane)];
        w = ml.x == top ? 1.f : ex2_fast(ml.x - top);
        sum = fmaf(w, ml.y, sum);
      }
      const int many = min(32, n - base);
#pragma unroll 8
      for (int j = 0; j < many; ++j) {
        const float by = __shfl_sync(0xffffffffu, w, j);
        const float4 u = d < D ? *reinterpret_cast<const float4*>(a.part_o + share(base + j) * D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        acc.x = fmaf(by, u.x, acc.x), acc.y = fmaf(by, u.y, acc.y);
        acc.z = fmaf(by, u.z, acc.z), acc.w = fmaf(by, u.w, acc.w);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int item_row = item.y * N + row, tok = item_row / a.group;
    QT* out = static_cast<QT*>(a.out) + (seq.x + static_cast<int64_t>(tok)) * a.ost + (item_row - tok * a.group) * a.osh +
              item.z * D + d;
    float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (outside && sees_outside(a, item.x, seq.z, seq.w, tok)) inv = __int_as_float(0x7fffffff);
    if (d < D) {
      out[0] = from_f<QT>(acc.x * inv), out[1] = from_f<QT>(acc.y * inv);
      out[2] = from_f<QT>(acc.z * inv), out[3] = from_f<QT>(acc.w * inv);
    }
  }
}

template <typename QT, int N>
cudaError_t launch_latent_join(const LatentAttnArgs& a, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.max_tokens) * a.group;
  const int units = static_cast<int>(rows < N ? rows : N) * ((a.item_dims + 127) / 128);
  const int y = (units + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  const int checks = (a.c.B + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  return launch_pdl(latent_join_kernel<QT, N>, dim3(static_cast<unsigned>(a.parts + checks), static_cast<unsigned>(y)),
                    dim3(kJoinThreads), st, a);
}

// One launch of an attention kernel, allowed to start while its predecessor drains, and the join.
template <typename QT, int N, typename K>
cudaError_t launch_items(K kernel, const LatentAttnArgs& a, int threads, int smem, const CUtensorMap& map, cudaStream_t st) {
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
  e = cudaLaunchKernelEx(&cfg, kernel, a, map);
  return e != cudaSuccess ? e : launch_latent_join<QT, N>(a, st);
}

}  // namespace
}  // namespace specv
