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
// Operands. The products are e4m3 x e5m2 -> fp32 (scores) and e4m3 x e4m3 -> fp32.
// A query element over a power of two is the sum of three e5m2 terms (3 bits and a
// sign each: 8 bits of bf16 and 11 of fp16 leave nothing). The power is one for the
// rows of an item, and e5m2's wide range keeps them apart: elements are exact down
// to 2^-31 of the item's largest, for a row 2^14 times smaller than another still
// 2^-17 of its own. A weight is the sum of two e4m3 terms for bf16 results and three
// for fp16, its relative error about 2^-9 rms and 2^-12. Because E is the tile's own
// largest, the codes' floor costs no more than 2^-17 of a weight in the same tile.
// 64 sequences of 9 tokens, bf16, 140 us. With e4m3 terms, of which bf16 takes two
// (135), a row 2^10 times smaller than another lost 0.6% of its result (fp16: 1%);
// a power of two for each row, as a factor of its scores, costs 12 instructions a
// tile (144); two terms and a third for rows far apart only (138), but 32 and 64
// rows are slower by 2%.
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
// products, groups of four warps turn scores into weights and add the products
// up, each for its share of the rows.
// A step of the softmax group: scores and the product of the tile before last
// leave tensor memory together, each row's maximum crosses lanes by redux and
// warps by shared memory, the weights are written, and the tile's product runs
// while the next tiles are worked on.
//
// What bounds it. One row of 32 heads (decode, 64 sequences of 1500 to 6500
// tokens, 8 KV heads of 128): memory, 547 MB in 92 us, 5.9 TB/s, 0.87 of a
// copy. Nine rows (verification, the same cache): 140 us, 4.0 TB/s, where the
// softmax groups' instructions (61% of issue slots) and the barrier between the
// tile's four maxima and its weights set the step of 2200 clocks a tile; the
// tensor pipe is busy for 21% of them. One sequence of 517 tokens: 11 us, a chain
// of lengths, table, queries, one tile a thread block, and the join.
#include <string.h>

#include "kv8_attn.cuh"

namespace specv {

namespace {

// ---------------------------------------------------------- configuration --

// Units of an item beside its tiles (see Runs). 64 sequences of 500 to 2000 tokens: 36 rows 76 us without, 68 with 2, 65
// with 3 and 4; 16 rows 43, 40, 41.
constexpr int kCost = 3;

// D: head dimension. RW: rows of one softmax group of four warps, W: groups.
template <int D_, int RW_, int W_, int TERMS_, int CTAS_>
struct Cfg {
  static constexpr int D = D_, RW = RW_, W = W_, TERMS = TERMS_;
  static constexpr int N = RW * W;
  static constexpr int EW = (N + 31) / 32;                 // warps that load queries
  static constexpr int kThreads = W * 128 + EW * 32 + 64;  // softmax, queries, copies and products
  static constexpr int kCtas = CTAS_;                  // resident on an SM
  static constexpr int kSlot = kTile * D;
  static constexpr int kQTerms = 3;  // e5m2 terms of a query element
  static constexpr int kQ = kQTerms * N * D;  // one item's queries; two are kept
  static constexpr int kTerm = N == 48 ? 64 : N;  // a term's columns in a row of weights: none crosses a panel of 128
  static constexpr int kPanels = (TERMS * kTerm + 127) / 128, kP = kPanels * kTile * 128;  // one tile's weights; two are kept
  static_assert(128 % kTerm == 0, "terms within panels");
  static constexpr int kCols = N <= 16 ? 64 : (N <= 32 ? 128 : 256);  // scores and products of two tiles: 4 N, a power of two
  static constexpr uint32_t kLayout = D == 128 ? 2 : 4;
  static constexpr int kGrain = RW % 8 == 0 ? 8 : 4;  // weights stored at a time, in bytes
  static_assert(RW % 4 == 0 && N % 16 == 0, "weights four at a time, products 16 columns at a time");

  // One item, as the query warps hand it to the others.
  struct Item {
    int b, first, n, ctx, rows, end, part, r0, h, t0, t1, whole;
  };
  struct Small {
    Item item[2];
    alignas(16) float smax[2][W][4][RW];  // of two tiles: each warp's largest exponents
    alignas(16) float e[W * 4][RW];       // of each warp: what the tile's scores are shifted by, 8 - E
    alignas(16) float f[W * 4][4][RW];    // and the factors 2^(E - ref) of the last four tiles
    float sums[2][W][4][RW];
    float inv[W * 4][RW];
    float red[2];
    int nan[2], eq[2];
    alignas(16) float4 page[kMetaRing][kMaxPages];
    alignas(8) uint64_t full[12], empty[12], s_full[2], p_ready[2], o_full[2], q_ready[2], q_free[2], drain;
    uint32_t tmem;
    int gave_up, outside;
  };
  static_assert(sizeof(Small::smax) >= 64 * sizeof(int), "the search for the run uses these words before the roles begin");
  static constexpr int kBudget = kCtas == 2 ? 115712 : 231424;
  static constexpr int kFixed = 1024 + 2 * kQ + 2 * kP + static_cast<int>(sizeof(Small));
  static constexpr int kFit = (kBudget - kFixed) / kSlot;
  static constexpr int kRing = kFit > 12 ? 12 : kFit;
  static constexpr int kSmem = kFixed + kRing * kSlot;
  static_assert(kRing >= 3, "ring of tile slots");
  static_assert(kMetaRing >= (kRing + 1) / 2 + 1, "meta entries live as long as a tile's slots");
};

// The e5m2 terms of eight query elements (already divided by the item's scale). An infinite one gives NaN, as its scores
// would in any sum.
template <int TERMS>
__device__ __forceinline__ void split8(float* x, uint2* out) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fabsf(x[i]) < -kNegInf ? x[i] : __int_as_float(0x7fffffff);
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    uint16_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(c[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
      uint32_t back;
      asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(back) : "h"(c[i]));
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&back));
      x[2 * i] -= y.x;
      x[2 * i + 1] -= y.y;
    }
    out[t] = make_uint2(c[0] | static_cast<uint32_t>(c[1]) << 16, c[2] | static_cast<uint32_t>(c[3]) << 16);
  }
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

// ----------------------------------------------------------------- kernel --

template <typename QT, typename C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas)
    kv8_attention_kernel(const __grid_constant__ Kv8AttnArgs a, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t dyn[];
  constexpr int D = C::D, N = C::N, RW = C::RW, NS = C::kRing;
  constexpr int GR = C::kGrain;
  uint8_t* q_smem = dyn + ((1024u - (smem_addr(dyn) & 1023u)) & 1023u);
  uint8_t* ring = q_smem + 2 * C::kQ;
  uint8_t* p_smem = ring + NS * C::kSlot;
  typename C::Small& sm = *reinterpret_cast<typename C::Small*>(p_smem + 2 * C::kP);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = uniform(tid >> 5);  // known to be the warp's, so that roles keep their addresses in uniform registers
  constexpr int kQueryWarp = C::W * 4, kLoadWarp = kQueryWarp + C::EW, kMmaWarp = kLoadWarp + 1;
  constexpr uint32_t kO = 2 * N;  // tensor memory: scores at 0 and N, then products
  volatile int* gave_up = &sm.gave_up;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      bar_init(smem_addr(&sm.full[i]), 1);
      bar_init(smem_addr(&sm.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&sm.s_full[i]), 1);
      bar_init(smem_addr(&sm.p_ready[i]), C::W * 4);
      bar_init(smem_addr(&sm.o_full[i]), 1);
      bar_init(smem_addr(&sm.q_ready[i]), C::EW);
      bar_init(smem_addr(&sm.q_free[i]), C::W * 4);
    }
    bar_init(smem_addr(&sm.drain), 1);
    fence_bar_init();
    sm.gave_up = 0;
    sm.outside = 0;
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&sm.tmem), C::kCols);
  griddep_wait();
  Runs runs;
  Start start;
  fence_before();
  const bool work = uniform(find_run<N, kCost>(a, blockIdx.x, &runs, &start, reinterpret_cast<int*>(sm.smax))) != 0;
  const int64_t my_units = work ? runs.begin(blockIdx.x + 1) - runs.begin(blockIdx.x) : 0;
  __syncthreads();
  fence_after();
  const uint32_t tmem = uniform(sm.tmem);

  uint32_t begun = 0;
  if (work && warp == kLoadWarp) {
    begun = copy_tiles<N, kCost, D, NS>(a, start, my_units, kmap, vmap, ring, sm, gave_up);
  } else if (work && warp == kMmaWarp) {
    // ---- products: the warp waits together, one lane issues
    constexpr uint32_t kStride = 8 * D;
    // D = 64: the two halves of the values' 128 rows are the same 64 dimensions (stride 0 between them)
    const uint64_t k_desc = smem_desc(smem_addr(ring), 16, kStride, C::kLayout),
                   v_desc = smem_desc(smem_addr(ring), 0, kStride, C::kLayout),
                   q_desc = smem_desc(smem_addr(q_smem), 16, kStride, C::kLayout),
                   p_desc = smem_desc(smem_addr(p_smem), 1024, 1024, 2);
    for (int i = 0, seg = 0;; ++seg) {
      bool ok = bar_wait(smem_addr(&sm.q_ready[seg & 1]), (seg >> 1) & 1, gave_up);
      ok = __all_sync(0xffffffffu, ok);
      const int t0 = uniform(sm.item[seg & 1].t0), t1 = uniform(sm.item[seg & 1].t1);
      if (!ok || t1 <= t0) break;
      fence_after();
      constexpr uint32_t id_s = instr_desc(kTile, N, false, true), id_o = instr_desc(kTile, N, true, false);
      auto scores = [&](int j) {  // S[j & 1] = K tile x Q^T
        const uint32_t slot = uniform((2u * j) % NS), to = uniform(tmem + (j & 1) * N);
        bool ok = bar_wait(smem_addr(&sm.full[slot]), ((2u * j) / NS) & 1, gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        fence_after();
        if (elect()) {
          const uint64_t kd = k_desc + (slot * C::kSlot >> 4), qd = q_desc + ((seg & 1) * C::kQ >> 4);
#pragma unroll
          for (int t = 0; t < C::kQTerms; ++t)
#pragma unroll
            for (int k = 0; k < D / 32; ++k) mma_f8(to, kd + 2 * k, qd + (2 * k + (t * N * D >> 4)), id_s, t > 0 || k > 0);
          commit(smem_addr(&sm.empty[slot]));
          commit(smem_addr(&sm.s_full[j & 1]));
        }
        __syncwarp();
        return true;
      };
      ok = scores(i);
      for (int t = t0; t < t1 && ok; ++t, ++i) {
        if (t + 1 < t1 && !scores(i + 1)) {
          ok = false;
          break;
        }
        const uint32_t slot = uniform((2u * i + 1) % NS), to = uniform(tmem + kO + (i & 1) * N);
        ok = bar_wait(smem_addr(&sm.full[slot]), ((2u * i + 1) / NS) & 1, gave_up) &&
             bar_wait(smem_addr(&sm.p_ready[i & 1]), (i >> 1) & 1, gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        fence_after();
        if (elect()) {
          const uint64_t vd = v_desc + (slot * C::kSlot >> 4), pd = p_desc + ((i & 1) * C::kP >> 4);
#pragma unroll
          for (int u = 0; u < C::TERMS; ++u) {
            const uint32_t off = (u * C::kTerm / 128) * (kTile * 128) + u * C::kTerm % 128;
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k)
              mma_f8(to, vd + (k * 32 * D >> 4), pd + ((off + k * 4096) >> 4), id_o, u > 0 || k > 0);
          }
          commit(smem_addr(&sm.empty[slot]));
          commit(smem_addr(&sm.o_full[i & 1]));
        }
        __syncwarp();
      }
      if (!ok) break;
    }
  } else if (work && warp >= kQueryWarp && warp < kLoadWarp) {
    // ---- the items' queries, one item ahead: a thread owns a row
    const int own = tid - kQueryWarp * 32, quarter = warp - kQueryWarp;
    Walk<N, kCost> it(a, start, my_units);
    const bool vec = ((reinterpret_cast<uintptr_t>(a.q) | (a.qst * 2) | (a.qsh * 2)) & 15) == 0;
    int seg = 0;
    bool more, ok = true;
    do {
      const RowTile r = it.r;
      const int r0 = r.rt * N;
      // Queries into shared memory, as e5m2 terms of q / 2^eq: kLanes lanes a row. Up to eight loads a lane are in
      // flight at once; an item of more rows is read a second time, from L2, when its scale is known.
      constexpr int kLanes = D / 8, kRows = C::EW * 32 / kLanes, kSteps = (N + kRows - 1) / kRows,
                    kBatch = kSteps <= 8 ? kSteps : kSteps / 2;
      static_assert(kSteps % kBatch == 0 && N % kRows == 0, "whole batches of whole rows");
      const int d = (lane % kLanes) * 8, sub = own / kLanes;
      uint4 u[kBatch];
      auto load = [&](int z0) {
#pragma unroll
        for (int z = 0; z < kBatch; ++z) {
          const uint32_t flat = static_cast<uint32_t>(r0 + min((z0 + z) * kRows + sub, r.rows - 1)),
                         tok = flat / static_cast<uint32_t>(a.group);
          const QT* q = static_cast<const QT*>(a.q) + (r.first + static_cast<int64_t>(tok)) * a.qst +
                        (it.h * a.group + static_cast<int>(flat - tok * a.group)) * a.qsh + d;
          if (vec) {
            u[z] = *reinterpret_cast<const uint4*>(q);
          } else {
            QT e[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) e[k] = q[k];
            memcpy(&u[z], e, 16);
          }
        }
      };
      float amax = 0.f;
#pragma unroll 1
      for (int z0 = 0; z0 < kSteps; z0 += kBatch) {
        load(z0);
#pragma unroll
        for (int z = 0; z < kBatch; ++z) {
          QT e[8];
          memcpy(e, &u[z], 16);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float m = fabsf(to_f(e[k]));
            if (m < -kNegInf) amax = fmaxf(amax, m);
          }
        }
      }
      amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
      if (C::EW > 1) {
        named_sync(2, C::EW * 32);  // the last item's maxima have been read
        if (lane == 0) sm.red[quarter] = amax;
        named_sync(2, C::EW * 32);
        amax = fmaxf(sm.red[0], sm.red[1]);
      }
      const int eq = kv8_need(amax, -113, 120) - 7;  // amax <= 57344 * 2^eq, e5m2's largest
      const float down = a.negate ? -pow2i(-eq) : pow2i(-eq);
      if (seg > 1) {
        ok = bar_wait(smem_addr(&sm.q_free[seg & 1]), ((seg >> 1) - 1) & 1, gave_up);
        ok = C::EW > 1 ? named_all(2, C::EW * 32, ok) : __all_sync(0xffffffffu, ok);
        if (!ok) break;  // the item before the last may still be read
      }
      uint8_t* q_to = q_smem + (seg & 1) * C::kQ;
#pragma unroll 1
      for (int z0 = 0; z0 < kSteps; z0 += kBatch) {
        if (kBatch < kSteps) load(z0);
#pragma unroll
        for (int z = 0; z < kBatch; ++z) {
          const int row = (z0 + z) * kRows + sub;
          QT e[8];
          memcpy(e, &u[z], 16);
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = row < r.rows ? to_f(e[k]) * down : 0.f;
          uint2 codes[C::kQTerms];
          split8<C::kQTerms>(x, codes);
          const uint32_t o = swz<D>(row, d);
#pragma unroll
          for (int t = 0; t < C::kQTerms; ++t) *reinterpret_cast<uint2*>(q_to + t * N * D + o) = codes[t];
        }
      }
      if (own == 0) {
        sm.nan[seg & 1] = 0;
        sm.eq[seg & 1] = eq;
        sm.item[seg & 1] = {r.b, r.first, r.n, r.ctx, r.rows, r.end, r.part, r0, it.h, it.t0, it.t1, it.t0 == 0 && it.t1 == r.tiles};
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&sm.q_ready[seg & 1]));
      ++seg;
      const RowTile last = it.r;
      const int h = it.h, t0 = it.t0, t1 = it.t1;
      more = it.next(a);
      if (!more && own == 0) a.cut[blockIdx.x] = cut_item<N>(runs, blockIdx.x, last, h, t0, t1);
    } while (more);
    if (ok && seg > 1) ok = bar_wait(smem_addr(&sm.q_free[seg & 1]), ((seg >> 1) - 1) & 1, gave_up);
    if (__all_sync(0xffffffffu, ok)) {
      if (own == 0) sm.item[seg & 1].t0 = sm.item[seg & 1].t1 = 0;  // no further item
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&sm.q_ready[seg & 1]));
    }
  } else if (work && warp < kQueryWarp) {
    // ---- weights and sums: a thread owns a slot of the tile and a dimension of the result
    const int wg = uniform(warp >> 2), quarter = uniform(warp & 3);
    const int own = quarter * 32 + lane;  // slot in the tile; dimension (mod D)
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int page = own / a.c.block;
    const int row_base = wg * RW;  // first row of this group within the row tile
    float l[RW], o[RW];
    static_assert(RW <= 16, "a lane holds a row's reference; sums over lanes");
    for (int i = 0, seg = 0;; ++seg) {  // tiles and items so far
      const bool ok = bar_wait(smem_addr(&sm.q_ready[seg & 1]), (seg >> 1) & 1, gave_up);
      if (!named_all(3 + wg, 128, ok)) break;
      const typename C::Item& it = sm.item[seg & 1];
      const int t0 = uniform(it.t0), t1 = uniform(it.t1);
      if (t1 <= t0) break;
      const int first_masked = uniform(it.part);  // from this tile on not every row sees every slot
      const float scale = a.scale * pow2i(sm.eq[seg & 1]);
      float ref = kNegInf;  // of row lane % 16: the exponent its sums are relative to
#pragma unroll
      for (int j = 0; j < RW; ++j) l[j] = 0.f, o[j] = 0.f;

      // o += 2^(E - ref) times the product of tile number j
      auto accumulate = [&](int j) {
        bar_wait(smem_addr(&sm.o_full[j & 1]), (j >> 1) & 1, gave_up);
        fence_after();
        uint32_t x[RW];
        tmem_ld<RW>(lanes + kO + (j & 1) * N + row_base, x);
        const float* f = sm.f[warp][j & 3];
        wait_ld();
#pragma unroll
        for (int q = 0; q < RW; q += 4) {
          const float4 g = *reinterpret_cast<const float4*>(f + q);
          const float2 u = fma2(make_float2(__uint_as_float(x[q]), __uint_as_float(x[q + 1])), make_float2(g.x, g.y),
                                make_float2(o[q], o[q + 1]));
          const float2 v = fma2(make_float2(__uint_as_float(x[q + 2]), __uint_as_float(x[q + 3])), make_float2(g.z, g.w),
                                make_float2(o[q + 2], o[q + 3]));
          o[q] = u.x, o[q + 1] = u.y, o[q + 2] = v.x, o[q + 3] = v.y;
        }
      };

      for (int t = t0; t < t1; ++t, ++i) {
        const int buf = i & 1;
        bar_wait(smem_addr(&sm.s_full[buf]), (i >> 1) & 1, gave_up);
        fence_after();
        uint32_t x[RW];
        tmem_ld<RW>(lanes + buf * N + row_base, x);

        const float4 meta = sm.page[i % kMetaRing][page];
        const float cs = scale * meta.x, ev = meta.y, ve_inv = meta.z;
        const bool masked = t >= first_masked;
        uint32_t vis = 0xffffffffu;
        if (masked) {
          const int slot = t * kTile + own;
          if (wg == 0) {
            // Slots behind the sequence hold no values, and a NaN value must not reach the rows that do not see it
            // through a weight of 0: both are cleared here, and the rows that see a NaN get it at the item's end.
            const uint32_t vslot = (2u * i + 1) % NS;
            bar_wait(smem_addr(&sm.full[vslot]), ((2u * i + 1) / NS) & 1, gave_up);
            uint4* vrow = reinterpret_cast<uint4*>(ring + vslot * C::kSlot + own * D);
            if (slot >= it.end) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k) vrow[k] = make_uint4(0, 0, 0, 0);
            } else {
              uint32_t nan = 0;
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint4 u = vrow[k];
                nan |= nan_codes(u.x) | nan_codes(u.y) | nan_codes(u.z) | nan_codes(u.w);
              }
              if (nan & 0x80808080u) {
                uint32_t* w = reinterpret_cast<uint32_t*>(vrow);
#pragma unroll 1
                for (int k = 0; k < D / 4; ++k) w[k] &= ~__vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                sm.nan[seg & 1] = 1;
              }
            }
          }
          if (slot >= it.ctx) {
            const int row = it.r0 + row_base, j = slot - it.ctx;  // row and token of the step
            if (slot >= it.end) {
              vis = 0;
            } else if (!a.tree) {
              const int64_t first = static_cast<int64_t>(j) * a.group - row;
              vis = first <= 0 ? 0xffffffffu : (first >= RW ? 0u : 0xffffffffu << first);
            } else {
              uint32_t bits = 0;
              int token = row / a.group, sub = row - token * a.group;
              for (int q = 0; q < RW;) {  // the rows of one token see the same
                const bool on = token < it.n && sees(a, it.b, token, j);
                const int many = min(RW - q, a.group - sub);
                if (on) bits |= ((1u << many) - 1u) << q;
                q += many;
                sub = 0;
                ++token;
              }
              vis = bits;
            }
          }
          __syncwarp();
        }
        wait_ld();

        // each row's largest exponent: over the lanes, then over the four warps
        float y[RW];
#pragma unroll
        for (int j = 0; j < RW; j += 2) {
          const float2 z = fma2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), make_float2(cs, cs),
                                make_float2(ev, ev));
          y[j] = z.x;
          y[j + 1] = z.y;
        }
        if (masked) {
#pragma unroll
          for (int j = 0; j < RW; ++j)
            if (!((vis >> j) & 1)) y[j] = kNegInf;
        }
        float mine = kNegInf;
#pragma unroll
        for (int jg = 0; jg < RW; jg += GR) {
          float m[GR];
#pragma unroll
          for (int j = 0; j < GR; ++j) m[j] = warp_max(y[jg + j]);
#pragma unroll
          for (int j = 0; j < GR; ++j)
            if (lane == jg + j) mine = m[j];
        }
        if (lane < RW) sm.smax[buf][wg][quarter][lane] = mine;
        named_sync(3 + wg, 128);
        {
          const int row = lane % RW;
          const float m = fmaxf(fmaxf(sm.smax[buf][wg][0][row], sm.smax[buf][wg][1][row]),
                                fmaxf(sm.smax[buf][wg][2][row], sm.smax[buf][wg][3][row]));
          const bool none = m == kNegInf;
          const float e = none ? 0.f : ceilf(m);
          if (t == t0 && !none) ref = e;
          const bool far = !none && e - ref > 60.f;
          if (__any_sync(0xffffffffu, far)) {
            const float by = far ? exp2_whole(ref - e) : 1.f;
            if (far) ref = e;
            if (lane < RW) sm.f[warp][(i - 1) & 3][row] *= by;  // the product still to come is relative to the old one
#pragma unroll
            for (int j = 0; j < RW; ++j) {
              const float b = __shfl_sync(0xffffffffu, by, j);
              l[j] *= b;
              o[j] *= b;
            }
          }
          if (lane < RW) {
            sm.e[warp][row] = 8.f - e;
            sm.f[warp][i & 3][row] = none ? 0.f : exp2_whole(e - ref);
          }
        }
        __syncwarp();

        // weights, as e4m3 terms, and their sums
        uint32_t turn = static_cast<uint32_t>(own & 7) << 4;  // the swizzle of this slot's row of weights
        asm volatile("" : "+r"(turn));                      // its addresses are not kept over the loop
        uint8_t* p_to = p_smem + buf * C::kP + own * 128;
        const float* e_at = sm.e[warp];
        const float* f_at = sm.f[warp][i & 3];
#pragma unroll
        for (int jg = 0; jg < RW; jg += GR) {
          uint32_t code[C::TERMS][GR / 4];
#pragma unroll
          for (int j4 = 0; j4 < GR; j4 += 4) {
            const float4 e4 = *reinterpret_cast<const float4*>(e_at + jg + j4);
            const float4 f4 = *reinterpret_cast<const float4*>(f_at + jg + j4);
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              const int q = jg + j4 + j;
              const float2 e = j == 0 ? make_float2(e4.x, e4.y) : make_float2(e4.z, e4.w);
              const float2 f = j == 0 ? make_float2(f4.x, f4.y) : make_float2(f4.z, f4.w);
              const float2 z = add2(make_float2(y[q], y[q + 1]), e);
              const float w0 = ex2_fast(z.x), w1 = ex2_fast(z.y);
              const float2 s = fma2(make_float2(w0, w1), mul2(f, make_float2(ve_inv, ve_inv)), make_float2(l[q], l[q + 1]));
              l[q] = s.x;
              l[q + 1] = s.y;
              uint16_t c;
              asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(w1), "f"(w0));
              // Two terms keep 8 bits, so what is left of f16's 11 serves; three keep more, and their rest is taken in fp32.
              uint32_t rest;
              if (C::TERMS == 2) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(rest) : "f"(w1), "f"(w0));
#pragma unroll
              for (int u = 0; u < C::TERMS; ++u) {
                if (u > 0) {
                  uint32_t back;
                  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(c));
                  if (C::TERMS > 2 && u == 1) {
                    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&back));
                    const float2 d = fma2(b, make_float2(-1.f, -1.f), make_float2(w0, w1));
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(rest) : "f"(d.y), "f"(d.x));
                  } else {
                    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(rest) : "r"(back));
                  }
                  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(rest));
                }
                if (j == 0) code[u][j4 / 4] = c;
                else code[u][j4 / 4] |= static_cast<uint32_t>(c) << 16;
              }
            }
          }
#pragma unroll
          for (int u = 0; u < C::TERMS; ++u) {
            const int col = u * C::kTerm + row_base + jg;
            uint8_t* to = p_to + (col / 128) * (kTile * 128) + ((col % 128) ^ turn);
            if (GR == 8) *reinterpret_cast<uint2*>(to) = make_uint2(code[u][0], code[u][GR / 4 - 1]);
            else *reinterpret_cast<uint32_t*>(to) = code[u][0];
          }
        }
        fence_async_shared();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&sm.p_ready[buf]));
        if (t > t0) accumulate(i - 1);
      }
      accumulate(i - 1);
      if (sm.nan[seg & 1]) {  // set before the weights of its tile were ready
        for (int slot = max(t0, it.part) * kTile; slot < min(it.end, t1 * kTile); ++slot) {
          const int id = a.c.table[static_cast<int64_t>(it.b) * a.c.max_blocks + slot / a.c.block];
          if (id < 0 || id >= a.c.num_blocks) continue;
          const uint8_t code = a.c.v[id * a.c.sb + it.h * a.c.sh + (slot % a.c.block) * a.c.ss + own % D];
          if ((code & 0x7f) != 0x7f) continue;
#pragma unroll
          for (int j = 0; j < RW; ++j)
            if (slot < it.ctx || sees(a, it.b, min(it.n - 1, (it.r0 + row_base + j) / a.group), slot - it.ctx))
              o[j] = __int_as_float(0x7fffffff);
        }
      }

      // ---- the item's results, or its share of them
      const bool whole = it.whole;
      const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (t0 > 0 ? 0 : 1);
      {
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = j < RW ? l[j < RW ? j : 0] : 0.f;
        float s = lane_sums<16>(v, lane);
        auto& sums = sm.sums[seg & 1];
        if (lane < RW) sums[wg][quarter][lane] = s;
        named_sync(3 + wg, 128);
        const int row = lane % RW;
        s = (sums[wg][0][row] + sums[wg][1][row]) + (sums[wg][2][row] + sums[wg][3][row]);
        if (whole) sm.inv[warp][row] = s == 0.f ? 0.f : 1.f / s;
        else if (quarter == 0 && lane < RW && row_base + row < it.rows)
          a.part_ml[part * N + row_base + row] = make_float2(ref, s);
      }
      __syncwarp();
      if (own < D) {
        int tok = (it.r0 + row_base) / a.group;
        int sub = it.r0 + row_base - tok * a.group;
        QT* out = static_cast<QT*>(a.out) + own;
#pragma unroll
        for (int j = 0; j < RW; ++j) {
          if (row_base + j >= it.rows) continue;
          if (whole)
            out[(it.first + static_cast<int64_t>(tok)) * a.ost + (it.h * a.group + sub) * a.osh] = from_f<QT>(o[j] * sm.inv[warp][j]);
          else a.part_o[(part * N + row_base + j) * D + own] = o[j];
          if (++sub == a.group) sub = 0, ++tok;
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&sm.q_free[seg & 1]));
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (sm.gave_up) drain<NS>(sm, warp == kLoadWarp, begun, warp == kMmaWarp);
  if (warp == kMmaWarp) tmem_free(tmem, C::kCols);
  if (tid == 0) {
    a.gave_up[blockIdx.x] = (sm.gave_up ? kGaveUp : 0) | (sm.outside ? kOutside : 0);
    if (!work || sm.gave_up) a.cut[blockIdx.x] = make_int4(0, 0, 0, 0);  // what was begun is not to be joined
  }
  griddep_launch_dependents();
}

// ------------------------------------------------------------------ launch --

template <typename QT, int D, int RW, int W, int TERMS, int CTAS>
cudaError_t launch_attention(const Kv8AttnArgs& a, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  using C = Cfg<D, RW, W, TERMS, CTAS>;
  const cudaError_t e = launch_tiles(kv8_attention_kernel<QT, C>, a, C::kThreads, C::kSmem, k, v, st);
  return e != cudaSuccess ? e : launch_join<QT, D, C::N>(a, st);
}

template <typename QT, int D, int TERMS>
cudaError_t launch_rows(const Kv8AttnArgs& a, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  if (rows == 16) return launch_attention<QT, D, 16, 1, TERMS, 2>(a, k, v, st);
  if (rows == 32) return launch_attention<QT, D, 16, 2, TERMS, 1>(a, k, v, st);
  if (rows == 48) return launch_attention<QT, D, 12, 4, TERMS, 1>(a, k, v, st);
  return launch_attention<QT, D, 16, 4, TERMS, 1>(a, k, v, st);
}

}  // namespace

// Rows of an item, by the most rows that a sequence can have. A few rows are cheapest with slots as the products' rows: 16
// rows need so little shared and tensor memory that two thread blocks share an SM and hide each other's waits. From 65 rows
// on a row of scores a lane is cheaper, two row tiles of 128 to an item when there are more than 128.
// B = 64, contexts of 1500 to 6500 tokens, 8 KV heads of 128, bf16, us (16 sequences from 132 rows on):
//   rows of a sequence    4     16     32     36     48     52     64     68    128    132    256
//   as chosen            92     88    123    140    135    160    164    181    190     75     89
//   32 rows an item     114    108    123
//   64                  151    145    161    155    148    160    164
//   128 (kv8_wide)      166    157    172    168    159    172    175    181    190    100    112
//   256 (kv8_wide)      205    193    211    204    191    205    210    212    212     75     89
int kv8_attention_rows(int64_t max_rows) {
  if (max_rows <= 64) return max_rows <= 16 ? 16 : static_cast<int>((max_rows + 15) / 16 * 16);
  return max_rows <= 128 ? 128 : 256;
}

int kv8_attention_parts(int rows) { return rows <= 16 ? 2 * kSms : kSms; }

cudaError_t launch_kv8_attention(const Kv8AttnArgs& a, int dtype, int rows, const CUtensorMap& k, const CUtensorMap& v,
                                 cudaStream_t st) {
  if (dtype == SPEC_BF16)
    return a.c.D == 128 ? launch_rows<__nv_bfloat16, 128, 2>(a, rows, k, v, st)
                        : launch_rows<__nv_bfloat16, 64, 2>(a, rows, k, v, st);
  return a.c.D == 128 ? launch_rows<__half, 128, 3>(a, rows, k, v, st) : launch_rows<__half, 64, 3>(a, rows, k, v, st);
}

}  // namespace specv
