// kv8_attn.cu -- attention over the 8-bit paged KV cache on the tensor cores.
//
// Mathematics. With codes c, block exponents ek and ev, and y_t = sm_scale
// log2(e) 2^ek(t) (q . ck_t) + ev(t), a row's result is
//     sum_t 2^y_t cv_t / sum_t 2^(y_t - ev(t)),
// so neither the keys' nor the values' codes are ever converted: the block
// scales enter as a factor of the score and a summand of the exponent. Over a
// tile of 128 slots a row takes weights w_t = 2^(y_t - E + 8) with E the tile's
// largest y rounded up to a whole number; tiles add up with factors 2^(E - ref),
// exact powers of two, so the accumulators are rescaled only when a tile passes
// the row's reference by 2^60.
// Operands. The products are e4m3 x e4m3 -> fp32. A bf16 query element is the sum
// of two e4m3 terms (4 bits and a sign each), an fp16 one of three, exactly down
// to 2^-17 of the item's largest; a weight is split likewise, its relative error
// about 2^-9 rms for bf16 results and 2^-12 for fp16. Because E is the tile's own
// largest, the codes' floor costs no more than 2^-17 of a weight in the same tile.
//
// Orientation. Slots are the 128 rows of both products' first operand: scores
// are K (128 slots x D) times Q^T (D x N rows), results are V^T (D x 128 slots)
// times the weights (128 slots x N). A thread owns one slot (so block scales and
// masks are scalars of a thread) and one dimension of the result, N is the number
// of rows rounded to 16, and few rows cost little. K, Q enter with their inner
// dimension contiguous, V and the weights with their outer one, as they lie.
//
// Schedule. An item is (sequence, row tile, KV head); its tiles of 128 slots are
// numbered through all items, and every thread block takes an equal run of that
// list, found on the device from the lengths. An item cut by a run's end leaves
// partial sums; a second kernel joins them, in order. One warp copies K and V
// blocks into a ring of tile slots by bulk tensor copies, one issues the
// products, four or eight compute the softmax.
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
constexpr int kMaxPages = kTile / 16;
constexpr int kBadPage = 1 << 20;
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
};

template <int N>
__device__ __forceinline__ RowTile row_tile(const Kv8AttnArgs& a, int b, int rt) {
  RowTile r{};
  r.b = b;
  r.rt = rt;
  const int lo = a.cu[b], hi = a.cu[b + 1], len = a.c.len[b];
  if (!kv8_seq_ok(a.c, a.T, lo, hi, len) || hi - lo > a.max_tokens) return r;
  const int64_t rows = static_cast<int64_t>(hi - lo) * a.group, r0 = static_cast<int64_t>(rt) * N;
  if (r0 >= rows) return r;
  r.first = lo;
  r.n = hi - lo;
  r.ctx = len;
  r.rows = static_cast<int>(min(rows - r0, static_cast<int64_t>(N)));
  r.end = len + (a.tree ? r.n : static_cast<int>((r0 + r.rows - 1) / a.group) + 1);
  r.tiles = (r.end + kTile - 1) / kTile;
  return r;
}

// Where a run of tiles begins.
struct Start {
  int b, rt, h, t;
};

// All threads of the block: the run [lo, hi) of part `part` and its first tile.
// With `last`, the place of tile hi - 1 instead. s_tmp: 34 words of shared memory.
template <int N>
__device__ __forceinline__ bool find_run(const Kv8AttnArgs& a, int part, bool last, int64_t* lo, int64_t* hi, Start* s,
                                         int64_t* all_tiles, int* s_tmp) {
  const int nthr = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = nthr >> 5;
  const int64_t cand = static_cast<int64_t>(a.c.B) * a.row_tiles;
  int64_t total = 0;
  int v0 = 0, incl0 = 0;  // this thread's candidate of the first round
  for (int64_t base = 0; base < cand; base += nthr) {
    const int64_t i = base + tid;
    int v = 0;
    if (i < cand) v = row_tile<N>(a, static_cast<int>(i / a.row_tiles), static_cast<int>(i % a.row_tiles)).tiles;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_tmp[warp] = x;
    __syncthreads();
    int before = 0, sum = 0;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) before += s_tmp[w];
      sum += s_tmp[w];
    }
    __syncthreads();
    if (base == 0) v0 = v, incl0 = x + before;
    total += sum;
  }
  const int64_t all = total * a.c.H;
  const int64_t parts = min(static_cast<int64_t>(a.parts), all);
  *all_tiles = all;
  *lo = part < parts ? all * part / parts : all;
  *hi = part < parts ? all * (part + 1) / parts : all;
  if (*lo >= *hi) return false;
  const int64_t want = last ? *hi - 1 : *lo;
  int64_t run = 0;
  for (int64_t base = 0; base < cand; base += nthr) {
    const int64_t i = base + tid;
    int v = v0, incl = incl0, sum = 0;
    if (base > 0 || cand > nthr) {
      v = 0;
      if (i < cand) v = row_tile<N>(a, static_cast<int>(i / a.row_tiles), static_cast<int>(i % a.row_tiles)).tiles;
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) s_tmp[warp] = x;
      __syncthreads();
      int before = 0;
      for (int w = 0; w < nw; ++w) {
        if (w < warp) before += s_tmp[w];
        sum += s_tmp[w];
      }
      __syncthreads();
      incl = x + before;
    }
    const int64_t from = (run + incl - v) * a.c.H, to = (run + incl) * a.c.H;
    if (v > 0 && want >= from && want < to) {
      const int off = static_cast<int>((want - from) / v);
      s_tmp[0] = static_cast<int>(i / a.row_tiles);
      s_tmp[1] = static_cast<int>(i % a.row_tiles);
      s_tmp[2] = off;
      s_tmp[3] = static_cast<int>((want - from) - static_cast<int64_t>(off) * v);
    }
    run += sum;
    if (cand > nthr && run * a.c.H > want) break;  // the same for every thread
  }
  __syncthreads();
  s->b = s_tmp[0];
  s->rt = s_tmp[1];
  s->h = s_tmp[2];
  s->t = s_tmp[3];
  __syncthreads();
  return true;
}

// Walks the items of a run: (r, h) with tiles [t0, t1).
template <int N>
struct Walk {
  RowTile r;
  int h, t0, t1;
  int64_t left;  // tiles of the run from t0 on

  __device__ __forceinline__ Walk(const Kv8AttnArgs& a, const Start& s, int64_t count) {
    r = row_tile<N>(a, s.b, s.rt);
    h = s.h;
    t0 = s.t;
    left = count;
    clip();
  }
  __device__ __forceinline__ void clip() { t1 = static_cast<int>(min(static_cast<int64_t>(r.tiles), t0 + left)); }
  // The next item, if any is left.
  __device__ __forceinline__ bool next(const Kv8AttnArgs& a) {
    left -= t1 - t0;
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
        if (b >= a.c.B) {  // cannot be: the run's tiles were counted
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

// ---------------------------------------------------------- configuration --

// D: head dimension. RW: rows of one softmax group of four warps, W: groups.
template <int D_, int RW_, int W_, int TERMS_>
struct Cfg {
  static constexpr int D = D_, RW = RW_, W = W_, TERMS = TERMS_;
  static constexpr int N = RW * W;
  static constexpr int kCompute = W * 128, kThreads = kCompute + 64;
  static constexpr int kCtas = N <= 32 ? 2 : 1;  // resident on an SM
  static constexpr int kSlot = kTile * D;
  static constexpr int kQ = TERMS * N * D < 1024 ? 1024 : TERMS * N * D;
  static constexpr int kPanels = (TERMS * N + 127) / 128, kP = kPanels * kTile * 128;
  static constexpr int kCols = 3 * N <= 64 ? 64 : (3 * N <= 128 ? 128 : (3 * N <= 256 ? 256 : 512));
  static constexpr int kGrain = W > 2 ? 4 : 8;  // a group's rows are rounded to this, N to 16
  static __device__ __forceinline__ int group_rows(int rows) {
    constexpr int g = W == 1 ? 16 : kGrain;
    return ((rows + W - 1) / W + g - 1) / g * g;
  }
  static constexpr uint32_t kLayout = D == 128 ? 2 : 4;

  struct Small {
    float smax[2][W][4][RW];
    float e[W * 4][RW];     // of each warp: what the tile's scores are shifted by
    float f[2][W * 4][RW];  // and the tiles' factors
    float red[W * 4];
    int nan[2];
    int kexp[kMetaRing][kMaxPages], vexp[kMetaRing][kMaxPages];
    alignas(8) uint64_t full[12], empty[12], s_full[2], p_ready, o_full, q_ready, drain;
    uint32_t tmem;
    int gave_up;
    int tmp[36];
  };
  static constexpr int kBudget = kCtas == 2 ? 115712 : 231424;
  static constexpr int kFixed = 1024 + kQ + kP + static_cast<int>(sizeof(Small));
  static constexpr int kFit = (kBudget - kFixed) / kSlot;
  static constexpr int kRing = kFit > 12 ? 12 : kFit;
  static constexpr int kSmem = kFixed + kRing * kSlot;
  static_assert(kRing >= 3, "ring of tile slots");
  static_assert(kMetaRing >= (kRing + 1) / 2 + 1, "meta entries live as long as a tile's slots");
};

// Byte offset of element (row, byte) in a tile of rows of ROW bytes, swizzled as bulk tensor copies do.
template <int ROW>
__device__ __forceinline__ uint32_t swz(int row, int byte) {
  const uint32_t o = static_cast<uint32_t>(row * ROW + byte);
  return ROW == 128 ? o ^ ((o >> 3) & 0x70u) : o ^ ((o >> 3) & 0x30u);
}

// The e4m3 terms of eight query elements (already divided by the item's scale).
template <int TERMS>
__device__ __forceinline__ void split8(float* x, uint2* out) {
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    out[t] = make_uint2(kv8_codes4(x, 1.f), kv8_codes4(x + 4, 1.f));
    if (t + 1 < TERMS) {
      float y[8];
      kv8_values4(out[t].x, y);
      kv8_values4(out[t].y, y + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] -= y[i];
    }
  }
}

// 2^d of a whole d <= 127, exact; 0 below -126 and for -inf, NaN for NaN.
__device__ __forceinline__ float exp2_whole(float d) {
  const float p = __int_as_float((static_cast<int>(fmaxf(d, -127.f)) + 127) << 23);
  return d != d ? d : p;
}

// Sums v[0 .. C - 1] over the warp's lanes; lane j (mod C) gets the sum of v[j].
template <int C>
__device__ __forceinline__ float lane_sums(float* v, int lane) {
  if (C == 16) {
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], 16);
  }
#pragma unroll
  for (int o = C / 2; o >= 1; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int k = 0; k < o; ++k) {
      const float send = up ? v[k] : v[k + o], keep = up ? v[k + o] : v[k];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return v[0];
}

// Whether the step's token i sees its token j.
__device__ __forceinline__ bool sees(const Kv8AttnArgs& a, int b, int i, int j) {
  return a.tree ? a.tree[(static_cast<int64_t>(b) * a.max_tokens + i) * a.max_tokens + j] != 0 : j <= i;
}

// ----------------------------------------------------------------- kernel --

template <typename QT, typename C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas)
    kv8_attention_kernel(const __grid_constant__ Kv8AttnArgs a, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t dyn[];
  constexpr int D = C::D, N = C::N, RW = C::RW, NS = C::kRing;
  constexpr int HC = 16, HN = RW / HC;         // columns read from tensor memory at a time
  constexpr int RG = (RW + 31) / 32, RL = RW < 32 ? RW : 32;  // rows as lanes: groups, lanes used
  constexpr int GR = C::kGrain;
  uint8_t* base = dyn + ((1024u - (smem_addr(dyn) & 1023u)) & 1023u);
  uint8_t* ring = base;
  uint8_t* p_smem = ring + NS * C::kSlot;
  uint8_t* q_smem = p_smem + C::kP;
  typename C::Small& sm = *reinterpret_cast<typename C::Small*>(q_smem + C::kQ);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kLoadWarp = C::W * 4, kMmaWarp = C::W * 4 + 1;
  volatile int* gave_up = &sm.gave_up;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      bar_init(smem_addr(&sm.full[i]), 1);
      bar_init(smem_addr(&sm.empty[i]), 1);
    }
    bar_init(smem_addr(&sm.s_full[0]), 1);
    bar_init(smem_addr(&sm.s_full[1]), 1);
    bar_init(smem_addr(&sm.p_ready), C::W * 4);
    bar_init(smem_addr(&sm.o_full), 1);
    bar_init(smem_addr(&sm.q_ready), C::W * 4);
    bar_init(smem_addr(&sm.drain), 1);
    fence_bar_init();
    sm.gave_up = 0;
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&sm.tmem), C::kCols);
  griddep_wait();
  int64_t lo, hi, all;
  Start start;
  fence_before();
  const bool work = find_run<N>(a, blockIdx.x, false, &lo, &hi, &start, &all, sm.tmp);
  __syncthreads();
  fence_after();
  const uint32_t tmem = uniform(sm.tmem);

  if (work && warp == kLoadWarp) {
    // ---- copies: the pages of each tile's keys, then of its values
    Walk<N> it(a, start, hi - lo);
    const int bs = a.c.block, ppt = kTile / bs;
    uint32_t fill = 0, begun = 0;
    int i = 0;
    do {
      const int pages = (it.r.end + bs - 1) / bs;
      const int32_t* table = a.c.table + static_cast<int64_t>(it.r.b) * a.c.max_blocks;
      int id = -1, ke = 0, ve = 0;
      for (int t = it.t0, g = 0; t < it.t1; ++t, g += ppt, ++i) {
        if ((g & 31) == 0) {  // the next 32 pages' ids and scales, one a lane
          const int page = t * ppt + lane;
          id = page < pages ? table[page] : -1;
          if (id >= a.c.num_blocks) id = -1;
          if (id >= 0) {
            const int64_t s = static_cast<int64_t>(id) * a.c.H + it.h;
            ke = kv8_exp(a.c.ks[s]);
            ve = kv8_exp(a.c.vs[s]);
          } else {
            ke = kBadPage;
            ve = 0;
          }
        }
        const int from = (g & 31) + (lane & (ppt - 1));
        const int my_id = __shfl_sync(0xffffffffu, id, from), my_ke = __shfl_sync(0xffffffffu, ke, from),
                  my_ve = __shfl_sync(0xffffffffu, ve, from);
        const bool mine = lane < ppt && my_id >= 0;
        const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, mine)) * bs * D);
        int at[3];
        at[0] = 0;
        at[1] = it.h;
        at[2] = my_id;
        const int x1 = at[a.order & 3], x2 = at[(a.order >> 2) & 3], x3 = at[(a.order >> 4) & 3];
#pragma unroll
        for (int part = 0; part < 2; ++part, ++fill) {
          const uint32_t slot = fill % NS, bar = smem_addr(&sm.full[slot]);
          bool ok = true;
          if (fill >= NS) ok = bar_wait(smem_addr(&sm.empty[slot]), (fill / NS - 1) & 1, gave_up);
          ok = __all_sync(0xffffffffu, ok);
          if (part == 0 && lane < ppt) {
            sm.kexp[i % kMetaRing][lane] = my_ke;
            sm.vexp[i % kMetaRing][lane] = my_ve;
          }
          __syncwarp();
          if (!ok) continue;  // a wait gave up: no copy is started any more
          begun = fill + 1;
          if (lane == 0) bar_expect(bar, bytes);
          __syncwarp();
          if (mine)
            load_4d(smem_addr(ring + slot * C::kSlot + lane * bs * D), part == 0 ? &kmap : &vmap, bar, 0, x1, x2, x3);
        }
      }
    } while (it.next(a));
    if (*gave_up)  // copies that are still in flight write this block's memory
      for (uint32_t f = begun > NS ? begun - NS : 0; f < begun; ++f)
        for (int k = 0; k < (1 << 16) && !bar_try(smem_addr(&sm.full[f % NS]), (f / NS) & 1); ++k) {
        }
  } else if (work && warp == kMmaWarp) {
    // ---- products: the warp waits together, one lane issues
    Walk<N> it(a, start, hi - lo);
    int i = 0, seg = 0;
    constexpr uint32_t kStride = 8 * D;
    const uint32_t ring_at = smem_addr(ring), q_at = smem_addr(q_smem), p_at = smem_addr(p_smem);
    do {
      const uint32_t cols = uniform(C::W * C::group_rows(it.r.rows));
      const uint32_t id_s = instr_desc(kTile, cols, false), id_o = instr_desc(kTile, cols, true);
      auto scores = [&](int j) {  // S[j & 1] = K tile x Q^T
        const uint32_t slot = uniform((2u * j) % NS), to = uniform(tmem + (j & 1) * N);
        bool ok = bar_wait(smem_addr(&sm.full[slot]), ((2u * j) / NS) & 1, gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        fence_after();
        if (elect()) {
          const uint64_t kd = smem_desc(ring_at + slot * C::kSlot, 16, kStride, C::kLayout);
#pragma unroll
          for (int t = 0; t < C::TERMS; ++t) {
            const uint64_t qd = smem_desc(q_at + t * N * D, 16, kStride, C::kLayout);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) mma_f8(to, kd + 2 * k, qd + 2 * k, id_s, t > 0 || k > 0);
          }
          commit(smem_addr(&sm.empty[slot]));
          commit(smem_addr(&sm.s_full[j & 1]));
        }
        __syncwarp();
      };
      bool ok = bar_wait(smem_addr(&sm.q_ready), seg & 1, gave_up);
      ok = __all_sync(0xffffffffu, ok);
      fence_after();
      if (ok) scores(i);
      for (int t = it.t0; t < it.t1; ++t, ++i) {
        if (t + 1 < it.t1) scores(i + 1);
        const uint32_t slot = uniform((2u * i + 1) % NS);
        ok = bar_wait(smem_addr(&sm.full[slot]), ((2u * i + 1) / NS) & 1, gave_up) &&
             bar_wait(smem_addr(&sm.p_ready), i & 1, gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        fence_after();
        if (elect()) {
          // D = 64: the two halves of the 128 rows are the same 64 dimensions (stride 0 between them)
          const uint64_t vd = smem_desc(ring_at + slot * C::kSlot, 0, kStride, C::kLayout);
#pragma unroll
          for (int u = 0; u < C::TERMS; ++u) {
            constexpr uint32_t kPanel = kTile * 128;
            const uint64_t pd = smem_desc(p_at + (u * N / 128) * kPanel + u * N % 128, 1024, 1024, 2);
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k)
              mma_f8(tmem + 2 * N, vd + (k * 32 * D >> 4), pd + (k * 4096 >> 4), id_o, u > 0 || k > 0);
          }
          commit(smem_addr(&sm.empty[slot]));
          commit(smem_addr(&sm.o_full));
        }
        __syncwarp();
      }
      ++seg;
    } while (it.next(a));
    if (*gave_up) {  // products that are still running write this block's tensor memory
      if (elect()) commit(smem_addr(&sm.drain));
      for (int k = 0; k < (1 << 16) && !bar_try(smem_addr(&sm.drain), 0); ++k) {
      }
    }
    __syncwarp();
  } else if (work && warp < kLoadWarp) {
    // ---- softmax: a thread owns a slot of the tile and a dimension of the result
    const int wg = uniform(warp >> 2), quarter = uniform(warp & 3);
    const int own = quarter * 32 + lane;  // slot in the tile; dimension (mod D)
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    Walk<N> it(a, start, hi - lo);

    // Queries of an item into shared memory, as e4m3 terms of q / 2^eq.
    auto load_q = [&](const Walk<N>& w, int item) -> int {
      const int nrw = C::group_rows(w.r.rows);
      const int chunks = C::W * nrw * (D / 8);
      const int64_t r0 = static_cast<int64_t>(w.r.rt) * N;
      const bool vec = ((reinterpret_cast<uintptr_t>(a.q) | (a.qst * 2) | (a.qsh * 2)) & 15) == 0;
      auto chunk = [&](int c, float* x) {
        const int row = c / (D / 8), d = (c % (D / 8)) * 8;
        if (row >= w.r.rows) {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = 0.f;
          return;
        }
        const int64_t r = r0 + row;
        const int64_t tok = r / a.group;
        const int head = w.h * a.group + static_cast<int>(r - tok * a.group);
        const QT* q = static_cast<const QT*>(a.q) + (w.r.first + tok) * a.qst + head * a.qsh + d;
        if (vec) {
          const uint4 u = *reinterpret_cast<const uint4*>(q);
          const QT* e = reinterpret_cast<const QT*>(&u);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = to_f(e[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = to_f(q[k]);
        }
      };
      float amax = 0.f;
      for (int c = tid; c < chunks; c += C::kCompute) {
        float x[8];
        chunk(c, x);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (fabsf(x[k]) < -kNegInf) amax = fmaxf(amax, fabsf(x[k]));
      }
      amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
      if (lane == 0) sm.red[warp] = amax;
      if (tid == 0) sm.nan[item & 1] = 0;
      named_sync(8, C::kCompute);
      amax = 0.f;
#pragma unroll
      for (int k = 0; k < C::W * 4; ++k) amax = fmaxf(amax, sm.red[k]);
      const int eq = kv8_need(amax, -120, 120);
      const float down = pow2i(-eq);
      for (int c = tid; c < chunks; c += C::kCompute) {
        float x[8];
        chunk(c, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= down;
        uint2 codes[C::TERMS];
        split8<C::TERMS>(x, codes);
        const uint32_t o = swz<D>(c / (D / 8), (c % (D / 8)) * 8);
#pragma unroll
        for (int t = 0; t < C::TERMS; ++t) *reinterpret_cast<uint2*>(q_smem + t * N * D + o) = codes[t];
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&sm.q_ready));
      return eq;
    };

    float l[RW], o[RW];
    float ref[RG];  // row 32 g + lane: the exponent its sums are relative to
    int eq = load_q(it, 0);
    int i = 0, seg = 0;  // tiles and items so far
    bool more = true;
    while (more) {
      RowTile r = it.r;
      r.ctx = uniform(r.ctx);
      r.end = uniform(r.end);
      r.rows = uniform(r.rows);
      const int h = uniform(it.h), t0 = uniform(it.t0), t1 = uniform(it.t1);
      const int nrw = uniform(C::group_rows(r.rows));
      const int row_base = wg * nrw;  // first row of this group within the row tile
      const int64_t r0 = static_cast<int64_t>(r.rt) * N;
      const float scale = a.scale * pow2i(eq);
#pragma unroll
      for (int j = 0; j < RW; ++j) l[j] = 0.f, o[j] = 0.f;
#pragma unroll
      for (int g = 0; g < RG; ++g) ref[g] = kNegInf;

      // o += 2^(E - ref) times the product of tile number j
      auto accumulate = [&](int j) {
        bar_wait(smem_addr(&sm.o_full), j & 1, gave_up);
        fence_after();
        const float* f = sm.f[j & 1][warp];
#pragma unroll
        for (int k = 0; k < HN; ++k) {
          if (k * HC >= nrw) break;
          uint32_t x[HC];
          tmem_ld<HC>(lanes + 2 * N + row_base + k * HC, x);
          wait_ld();
#pragma unroll
          for (int q = 0; q < HC; q += 4) {
            const float4 g = *reinterpret_cast<const float4*>(f + k * HC + q);
            float* to = o + k * HC + q;
            const float2 u = fma2(make_float2(__uint_as_float(x[q]), __uint_as_float(x[q + 1])), make_float2(g.x, g.y),
                                  make_float2(to[0], to[1]));
            const float2 v = fma2(make_float2(__uint_as_float(x[q + 2]), __uint_as_float(x[q + 3])), make_float2(g.z, g.w),
                                  make_float2(to[2], to[3]));
            to[0] = u.x, to[1] = u.y, to[2] = v.x, to[3] = v.y;
          }
        }
      };

      for (int t = t0; t < t1; ++t, ++i) {
        const int slot0 = t * kTile, slot = slot0 + own, buf = i & 1;
        bar_wait(smem_addr(&sm.s_full[buf]), (i >> 1) & 1, gave_up);
        fence_after();
        const int page = own / a.c.block;
        const int ke = sm.kexp[i % kMetaRing][page], ve = sm.vexp[i % kMetaRing][page];
        const float cs = ke == kBadPage ? __int_as_float(0x7fffffff) : scale * pow2i(ke);
        const float ev = static_cast<float>(ve), ve_inv = pow2i(-ve);
        const bool masked = slot0 + kTile > r.ctx;  // not every row sees every slot
        if (masked && wg == 0) {
          // Slots behind the sequence hold no values, and a NaN value must not reach the rows that do not see it
          // through a weight of 0: both are cleared here, and the rows that see a NaN get it at the item's end.
          const uint32_t vslot = (2u * i + 1) % NS;
          bar_wait(smem_addr(&sm.full[vslot]), ((2u * i + 1) / NS) & 1, gave_up);
          uint4* vrow = reinterpret_cast<uint4*>(ring + vslot * C::kSlot + own * D);
          bool nan = false;
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k) {
            uint4 u = vrow[k];
            uint32_t any = 0;
            uint32_t* w = &u.x;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const uint32_t m = slot >= r.end ? 0xffffffffu : __vcmpeq4(w[z] & 0x7f7f7f7fu, 0x7f7f7f7fu);
              any |= m;
              w[z] &= ~m;
            }
            if (any) vrow[k] = u;
            nan |= any != 0;
          }
          if (nan && slot < r.end) sm.nan[seg & 1] = 1;
        }

        // the tile's largest exponent of each row
        float y[HC], mine = kNegInf;
        uint32_t vis[HN];
        auto scores = [&](int k) {
          uint32_t x[HC];
          tmem_ld<HC>(lanes + buf * N + row_base + k * HC, x);
          wait_ld();
#pragma unroll
          for (int j = 0; j < HC; j += 2) {
            const float2 z = fma2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), make_float2(cs, cs),
                                  make_float2(ev, ev));
            y[j] = z.x;
            y[j + 1] = z.y;
          }
          if (masked) {
#pragma unroll
            for (int j = 0; j < HC; ++j)
              if (!((vis[k] >> j) & 1)) y[j] = kNegInf;
          }
        };
#pragma unroll
        for (int k = 0; k < HN; ++k) {
          if (k * HC >= nrw) break;
          vis[k] = 0xffffffffu;
          if (masked && slot >= r.ctx) {
            const int64_t row = r0 + row_base + k * HC;  // of the step
            const int j = slot - r.ctx;
            if (slot >= r.end) {
              vis[k] = 0;
            } else if (!a.tree) {
              const int64_t first = static_cast<int64_t>(j) * a.group - row;
              vis[k] = first <= 0 ? 0xffffffffu : (first >= HC ? 0u : 0xffffffffu << first);
            } else {
              uint32_t bits = 0;
              int token = static_cast<int>(row / a.group), sub = static_cast<int>(row - static_cast<int64_t>(token) * a.group);
              bool on = token < r.n && sees(a, r.b, token, j);
              for (int q = 0; q < HC; ++q) {
                if (on) bits |= 1u << q;
                if (++sub == a.group) {
                  sub = 0;
                  ++token;
                  on = token < r.n && sees(a, r.b, token, j);
                }
              }
              vis[k] = bits;
            }
          }
          scores(k);
          if ((k & 1) == 0) mine = kNegInf;
#pragma unroll
          for (int jg = 0; jg < HC; jg += GR) {
            if (k * HC + jg >= nrw) break;
            float m[GR];
#pragma unroll
            for (int j = 0; j < GR; ++j) m[j] = warp_max(y[jg + j]);
#pragma unroll
            for (int j = 0; j < GR; ++j)
              if (lane == (k & 1) * HC + jg + j) mine = m[j];
          }
          if ((k & 1) == 1 || k == HN - 1 || (k + 1) * HC >= nrw) {
            if (RL == 32 || lane < RL) sm.smax[buf][wg][quarter][(k / 2) * 32 + lane] = mine;
          }
        }
        named_sync(1 + wg, 128);
        if (t > t0) accumulate(i - 1);
#pragma unroll
        for (int g = 0; g < RG; ++g) {
          if (g * 32 >= nrw) break;
          const int row = g * 32 + lane % RL;
          const float m = fmaxf(fmaxf(sm.smax[buf][wg][0][row], sm.smax[buf][wg][1][row]),
                                fmaxf(sm.smax[buf][wg][2][row], sm.smax[buf][wg][3][row]));
          const bool none = m == kNegInf;
          const float e = none ? 0.f : ceilf(m);
          const bool far = !none && e - ref[g] > 60.f;
          if (__any_sync(0xffffffffu, far)) {
            const float by = far ? exp2_whole(ref[g] - e) : 1.f;
            if (far) ref[g] = e;
#pragma unroll
            for (int j = 0; j < RL; ++j) {
              const float b = __shfl_sync(0xffffffffu, by, j);
              l[g * 32 + j] *= b;
              o[g * 32 + j] *= b;
            }
          }
          sm.e[warp][row] = 8.f - e;
          sm.f[buf][warp][row] = none ? 0.f : exp2_whole(e - ref[g]);
        }
        __syncwarp();

        // weights, as e4m3 terms, and their sums
#pragma unroll
        for (int k = 0; k < HN; ++k) {
          if (k * HC >= nrw) break;
          scores(k);
#pragma unroll
          for (int jg = 0; jg < HC; jg += GR) {
            if (k * HC + jg >= nrw) break;
            uint32_t code[C::TERMS][GR / 4];
#pragma unroll
            for (int j = 0; j < GR; j += 2) {
              const int q = k * HC + jg + j;
              const float2 e = *reinterpret_cast<const float2*>(&sm.e[warp][q]);
              const float2 f = *reinterpret_cast<const float2*>(&sm.f[buf][warp][q]);
              const float2 z = add2(make_float2(y[jg + j], y[jg + j + 1]), e);
              const float w0 = ex2_fast(z.x), w1 = ex2_fast(z.y);
              const float2 s = fma2(make_float2(w0, w1), mul2(f, make_float2(ve_inv, ve_inv)), make_float2(l[q], l[q + 1]));
              l[q] = s.x;
              l[q + 1] = s.y;
              uint16_t c;
              asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(w1), "f"(w0));
              uint32_t rest;
              asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(rest) : "f"(w1), "f"(w0));
#pragma unroll
              for (int u = 0; u < C::TERMS; ++u) {
                if (u > 0) {
                  uint32_t back;
                  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(c));
                  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(rest) : "r"(back));
                  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(rest));
                }
                if (j % 4 == 0) code[u][j / 4] = c;
                else code[u][j / 4] |= static_cast<uint32_t>(c) << 16;
              }
            }
#pragma unroll
            for (int u = 0; u < C::TERMS; ++u) {
              const int col = u * N + row_base + k * HC + jg;
              uint8_t* to = p_smem + (col / 128) * (kTile * 128) + swz<128>(own, col % 128);
              if (GR == 8) *reinterpret_cast<uint2*>(to) = make_uint2(code[u][0], code[u][GR / 4 - 1]);
              else *reinterpret_cast<uint32_t*>(to) = code[u][0];
            }
          }
        }
        fence_async_shared();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&sm.p_ready));
      }

      more = it.next(a);
      if (more) eq = load_q(it, seg + 1);  // the products that read the last queries are done
      accumulate(i - 1);
      if (sm.nan[seg & 1]) {  // set before the weights of its tile were ready
        for (int slot = max(t0, r.ctx / kTile) * kTile; slot < min(r.end, t1 * kTile); ++slot) {
          const int id = a.c.table[static_cast<int64_t>(r.b) * a.c.max_blocks + slot / a.c.block];
          if (id < 0 || id >= a.c.num_blocks) continue;
          const uint8_t code = a.c.v[id * a.c.sb + h * a.c.sh + (slot % a.c.block) * a.c.ss + own % D];
          if ((code & 0x7f) != 0x7f) continue;
#pragma unroll
          for (int j = 0; j < RW; ++j)
            if (slot < r.ctx || sees(a, r.b, min(r.n - 1, static_cast<int>((r0 + row_base + j) / a.group)), slot - r.ctx))
              o[j] = __int_as_float(0x7fffffff);
        }
      }
      ++seg;

      // ---- the item's results, or its share of them
      const bool whole = t0 == 0 && t1 == r.tiles;
      const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (t0 > 0 ? 0 : 1);
      auto& sums = sm.smax[(i - 1) & 1];  // every warp is past the last tile's maxima, and the next tile's go elsewhere
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        if (g * 32 >= nrw) break;
        const float s = lane_sums<RL>(l + g * 32, lane);
        if (RL == 32 || lane < RL) sums[wg][quarter][g * 32 + lane] = s;
      }
      named_sync(1 + wg, 128);
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        if (g * 32 >= nrw) break;
        const int row = g * 32 + lane % RL;
        const float s = (sums[wg][0][row] + sums[wg][1][row]) + (sums[wg][2][row] + sums[wg][3][row]);
        if (whole) sm.e[warp][row] = s == 0.f ? 0.f : 1.f / s;
        else if (quarter == 0 && lane < RL && row < nrw && row_base + row < r.rows)
          a.part_ml[part * N + row_base + row] = make_float2(ref[g], s);
      }
      __syncwarp();
      if (own < D) {
        int64_t tok = (r0 + row_base) / a.group;
        int sub = static_cast<int>(r0 + row_base - tok * a.group);
        QT* out = static_cast<QT*>(a.out) + own;
#pragma unroll
        for (int j = 0; j < RW; ++j) {
          if (j >= nrw || row_base + j >= r.rows) break;
          if (whole) out[(r.first + tok) * a.ost + (h * a.group + sub) * a.osh] = from_f<QT>(o[j] * sm.e[warp][j]);
          else a.part_o[(part * N + row_base + j) * D + own] = o[j];
          if (++sub == a.group) sub = 0, ++tok;
        }
      }
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp) tmem_free(tmem, C::kCols);
  if (tid == 0) a.gave_up[blockIdx.x] = sm.gave_up;
  griddep_launch_dependents();
}

// -------------------------------------------------------------------- join --
//
// Adds the shares of items that runs cut. Block x takes the item that begins in
// part x and ends behind it, a warp one row: shares in the order of the parts,
// each times 2^(its reference - the largest). The last blocks check sequences.

constexpr int kJoinThreads = 256;

template <typename QT, int D, int N>
__global__ void __launch_bounds__(kJoinThreads) kv8_join_kernel(const __grid_constant__ Kv8AttnArgs a) {
  __shared__ int s_tmp[36];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_launch_dependents();
  if (blockIdx.x >= static_cast<unsigned>(a.parts)) {  // a warp per sequence: row_status
    griddep_wait();
    const int b = (blockIdx.x - a.parts) * (kJoinThreads / 32) + warp;
    if (blockIdx.y > 0 || b >= a.c.B) return;
    bool late = false;
    for (int i = lane; i < a.parts; i += 32) late |= a.gave_up[i] != 0;
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
    if (!sound && lo >= 0 && hi > lo && hi <= a.T) {
      const int64_t rows = static_cast<int64_t>(hi - lo) * a.q_heads;
      for (int64_t i = 0; i < rows; ++i) {
        QT* out = static_cast<QT*>(a.out) + (lo + i / a.q_heads) * a.ost + (i % a.q_heads) * a.osh;
        for (int d = lane; d < D; d += 32) out[d] = from_f<QT>(__int_as_float(0x7fffffff));
      }
    }
    return;
  }
  int64_t lo, hi, all;
  Start s;
  if (!find_run<N>(a, blockIdx.x, true, &lo, &hi, &s, &all, s_tmp)) return;
  const RowTile r = row_tile<N>(a, s.b, s.rt);
  const int64_t begin = hi - 1 - s.t, end = begin + r.tiles;  // the item's tiles
  const int row = blockIdx.y * (kJoinThreads / 32) + warp;
  if (begin < lo || end <= hi || row >= r.rows) return;
  const int64_t parts = min(static_cast<int64_t>(a.parts), all);
  int64_t last = (end - 1) * parts / all;
  while (all * (last + 1) / parts <= end - 1) ++last;
  const int n = static_cast<int>(last - blockIdx.x) + 1;
  griddep_wait();
  const int64_t first = blockIdx.x;
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
  const int64_t item_row = static_cast<int64_t>(s.rt) * N + row, tok = item_row / a.group;
  QT* out = static_cast<QT*>(a.out) + (r.first + tok) * a.ost +
            (s.h * a.group + static_cast<int>(item_row - tok * a.group)) * a.osh + lane * V;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int k = 0; k < V; ++k) out[k] = from_f<QT>(acc[k] * inv);
}

// ------------------------------------------------------------------ launch --

constexpr int kSms = 152;

template <typename QT, int D, int RW, int W, int TERMS>
cudaError_t launch_attention(const Kv8AttnArgs& a, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  using C = Cfg<D, RW, W, TERMS>;
  auto kernel = kv8_attention_kernel<QT, C>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.parts));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a, k, v);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(a.max_tokens) * a.group;
  const int y = static_cast<int>((rows < C::N ? rows : C::N) + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  const int checks = (a.c.B + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  return launch_pdl(kv8_join_kernel<QT, D, C::N>, dim3(static_cast<unsigned>(a.parts + checks), static_cast<unsigned>(y)),
                    dim3(kJoinThreads), st, a);
}

template <typename QT, int D, int TERMS>
cudaError_t launch_rows(const Kv8AttnArgs& a, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  if (rows == 16) return launch_attention<QT, D, 16, 1, TERMS>(a, k, v, st);
  if (rows == 32) return launch_attention<QT, D, 16, 2, TERMS>(a, k, v, st);
  if (rows == 64) return launch_attention<QT, D, 16, 4, TERMS>(a, k, v, st);
  return launch_attention<QT, D, 32, 4, TERMS>(a, k, v, st);
}

}  // namespace

int kv8_attention_rows(int64_t max_rows) { return max_rows <= 16 ? 16 : (max_rows <= 32 ? 32 : (max_rows <= 64 ? 64 : 128)); }

int kv8_attention_parts(int rows) { return rows <= 32 ? 2 * kSms : kSms; }

cudaError_t launch_kv8_attention(const Kv8AttnArgs& a, int dtype, int rows, const CUtensorMap& k, const CUtensorMap& v,
                                 cudaStream_t st) {
  if (dtype == SPEC_BF16)
    return a.c.D == 128 ? launch_rows<__nv_bfloat16, 128, 2>(a, rows, k, v, st)
                        : launch_rows<__nv_bfloat16, 64, 2>(a, rows, k, v, st);
  return a.c.D == 128 ? launch_rows<__half, 128, 3>(a, rows, k, v, st) : launch_rows<__half, 64, 3>(a, rows, k, v, st);
}

}  // namespace specv
