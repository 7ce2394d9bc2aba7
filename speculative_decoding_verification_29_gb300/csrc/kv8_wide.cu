// kv8_wide.cu -- attention over the 8-bit paged KV cache for many rows: the
// target's pass over draft positions, trees and prompts.
//
// Here a row of scores is one thread's. Tiles of keys and values are turned from
// e4m3 into f16 once, exactly, for all the rows of the item (64 conversions a
// thread and tile), which buys products in f16: queries (a power of two times
// bf16 or fp16 values, exact down to 2^-24 of the row's largest) and weights (2^-12
// of their value, down to 2^-32 of the largest) need one term each, and because
// f16 weights keep their precision over 24 powers of two, the output may stay in
// tensor memory across tiles: a row's sums are relative to a reference that
// moves only when a tile passes it by 2^8, and only then the accumulator is read
// and scaled.
// With exponents y_t = sm_scale log2(e) 2^ek(t) (q . ck_t) + ev(t) a row's result
// is sum_t 2^(y_t - ref) cv_t / sum_t 2^(y_t - ref - ev(t)): the blocks' scales
// enter as a factor of the score, a summand of the exponent, and a factor of
// each block's sum of weights.
//
// Two streams, each with four softmax warps, 128 rows of scores that become the
// weights in place, and 128 columns of output in tensor memory, take turns at the
// tensor cores. PAIR: the streams are two row tiles (256 rows of an item) that
// share the tiles. Otherwise they share the rows (128), take every other tile
// and are added up at the item's end: both read each other's accumulator, since a
// row has the same lane in both.
// Four more warps convert tiles and load queries, one copies, one issues.
//
// What bounds it. Prompts (three of 1500 to 4096 tokens behind up to 1000, 32
// heads of 128, fp16): 376 us, 1040 TFLOP/s, 0.54 of a library product's rate
// (bf16: 403).
// Scores and weights of a pair of tiles hold the tensor pipe for 2112 clocks of a
// step of about 3700: a stream's weights must be written before its product, and
// the product issued before its next scores, and two streams do not cover that
// chain; tensor memory has no room for a third. An item's queries and results
// take 13,000 clocks more. Trees of 61 nodes (16 sequences of 500 to 3500): 69 us,
// of which items' ends and the join of cut items are half.
#include <string.h>

#include <type_traits>

#include "kv8_attn.cuh"

namespace specv {

namespace {

constexpr float kFar = 8.f;  // a tile moves the reference when it passes it by 2^8: weights stay below 2^8, far from 65504
// Units of an item beside its tiles (see Runs): its queries and results take 13,000 clocks, a tile 3,700. Prompts whose
// items have 1 to 40 tiles: 592 us without, 381 with 4, 386 with 8.
constexpr int kCost = 4;
constexpr int kItems = 4;    // items in flight between the query loads and the results

template <int D_, bool PAIR_>
struct Wide {
  static constexpr int D = D_, N = PAIR_ ? 256 : 128;
  static constexpr bool PAIR = PAIR_;
  static constexpr int kThreads = 4 * 128;  // two softmax groups, conversions, one of copies and products
  static constexpr int kF8 = kTile * D, kF16 = 2 * kF8;  // a tile of keys or values
  static constexpr int kPanel = kTile * 128;             // 64 columns of f16
  static constexpr int kQ = (PAIR ? 2 : 1) * kF16;
  static constexpr int NF = PAIR ? 3 : 4;  // f16 tiles
  struct Item {
    int b, first, n, ctx, rows, end, part, r0, h, t0, t1, tiles;
  };
  struct Small {
    alignas(16) Item item[kItems];
    float ref[2][2][kTile], sum[2][2][kTile];  // of two items: each stream's rows, exchanged at an item's end
    float qscale[kItems][N];             // 2^eq of the items' rows
    alignas(8) int64_t qrow[N];          // where the item's rows of queries begin
    int nan[kItems];
    alignas(16) float4 page[kMetaRing][kMaxPages];
    alignas(8) uint64_t full[8], empty[8], full16[4], empty16[4], s_full[2], p_ready[2], o_full[2], q_ready[kItems], q_free,
        done, drain;
    uint32_t tmem;
    int gave_up, outside;
    alignas(8) int tmp[64];
  };
  static constexpr int kFixed = 1024 + kQ + NF * kF16 + static_cast<int>(sizeof(Small));
  static constexpr int kFit = (231424 - kFixed) / kF8;
  static constexpr int NS = kFit > 6 ? 6 : kFit;  // e4m3 tiles
  static constexpr int kSmem = kFixed + NS * kF8;
  static_assert(NS >= 3, "ring of e4m3 tiles");
  static_assert(2 * kMetaRing >= NS + NF + 4, "a tile's exponents outlive its weights");
};

__device__ __forceinline__ __half2 abs2(const __half* e) { return __habs2(__half2(e[0], e[1])); }
__device__ __forceinline__ __nv_bfloat162 abs2(const __nv_bfloat16* e) { return __habs2(__nv_bfloat162(e[0], e[1])); }

// u[k] of lane j of four neighbouring lanes becomes u[j] of its lane k.
__device__ __forceinline__ void exchange4(uint4* u, int lane) {
#pragma unroll
  for (int o = 1; o <= 2; o *= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & o) continue;
      const uint4 send = up ? u[k] : u[k + o];
      const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, send.x, o), __shfl_xor_sync(0xffffffffu, send.y, o),
                                   __shfl_xor_sync(0xffffffffu, send.z, o), __shfl_xor_sync(0xffffffffu, send.w, o));
      if (up) u[k] = got;
      else u[k + o] = got;
    }
  }
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename QT, typename C>
__global__ void __launch_bounds__(C::kThreads, 1)
    kv8_wide_kernel(const __grid_constant__ Kv8AttnArgs a, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t dyn[];
  constexpr int D = C::D, N = C::N, NS = C::NS, NF = C::NF;
  constexpr bool PAIR = C::PAIR;
  uint8_t* q_smem = dyn + ((1024u - (smem_addr(dyn) & 1023u)) & 1023u);
  uint8_t* f16 = q_smem + C::kQ;
  uint8_t* ring = f16 + NF * C::kF16;
  typename C::Small& sm = *reinterpret_cast<typename C::Small*>(ring + NS * C::kF8);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = uniform(tid >> 5);  // known to be the warp's, so that roles keep their addresses in uniform registers
  constexpr int kConvWarp = 8, kLoadWarp = 12, kMmaWarp = 13;
  constexpr uint32_t kO = 256;  // tensor memory: scores (and weights) of the streams at 0 and 128, outputs behind
  volatile int* gave_up = &sm.gave_up;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      bar_init(smem_addr(&sm.full[i]), 1);
      bar_init(smem_addr(&sm.empty[i]), 4);
    }
    for (int i = 0; i < NF; ++i) {
      bar_init(smem_addr(&sm.full16[i]), 4);
      bar_init(smem_addr(&sm.empty16[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&sm.s_full[i]), 1);
      bar_init(smem_addr(&sm.p_ready[i]), 4);
      bar_init(smem_addr(&sm.o_full[i]), 1);
    }
    for (int i = 0; i < kItems; ++i) bar_init(smem_addr(&sm.q_ready[i]), 4);
    bar_init(smem_addr(&sm.q_free), 1);
    bar_init(smem_addr(&sm.drain), 1);
    bar_init(smem_addr(&sm.done), 8);
    fence_bar_init();
    sm.gave_up = 0;
    sm.outside = 0;
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&sm.tmem), 512);
  griddep_wait();
  Runs runs;
  Start start;
  fence_before();
  const bool work = uniform(find_run<N, kCost>(a, blockIdx.x, &runs, &start, sm.tmp)) != 0;
  const int64_t my_units = work ? runs.begin(blockIdx.x + 1) - runs.begin(blockIdx.x) : 0;
  __syncthreads();
  fence_after();
  const uint32_t tmem = uniform(sm.tmem);
  // Steps of the two streams for an item of nt tiles.
  auto steps = [](int nt, int rows, int stream) {
    if (PAIR) return stream == 0 || rows > kTile ? nt : 0;
    return (nt + 1 - stream) / 2;
  };

  // ---- products of both streams in turn: the warp waits together, one lane issues
  auto products = [&]() {
    constexpr uint32_t id_s = instr_desc_f16(kTile, kTile, false), id_o = instr_desc_f16(kTile, D, true);
    const uint64_t q_desc = smem_desc(smem_addr(q_smem), 16, 1024, 2), k_desc = smem_desc(smem_addr(f16), 16, 1024, 2),
                   v_desc = smem_desc(smem_addr(f16), C::kPanel, 1024, 2);
    int base = 0, count[2] = {0, 0};  // tiles and steps of earlier items
    for (int seg = 0;; ++seg) {
      bool ok = bar_wait(smem_addr(&sm.q_ready[seg & 3]), (seg >> 2) & 1, gave_up);
      ok = __all_sync(0xffffffffu, ok);
      const int nt = uniform(sm.item[seg & 3].t1 - sm.item[seg & 3].t0), rows = uniform(sm.item[seg & 3].rows);
      if (!ok || nt <= 0) break;
      fence_after();
      const int n[2] = {steps(nt, rows, 0), steps(nt, rows, 1)};
      const bool both = n[1] > 0;  // PAIR: a tile's second user is stream 1
#pragma unroll 1
      for (int s = -1; s < n[0] && ok; ++s) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (s >= 0 && s < n[b]) {  // O += P x V
            const uint32_t j = 2u * (base + (PAIR ? s : 2 * s + b)) + 1, slot = j % NF;
            // the last item's outputs have been read
            if (b == 0 && s == 0 && seg > 0) ok = bar_wait(smem_addr(&sm.done), (seg - 1) & 1, gave_up);
            if (!PAIR || b == 0) ok = bar_wait(smem_addr(&sm.full16[slot]), (j / NF) & 1, gave_up) && ok;
            ok = bar_wait(smem_addr(&sm.p_ready[b]), (count[b] + s) & 1, gave_up) && ok;
            __syncwarp();
            fence_after();
            if (elect() && ok) {
              const uint64_t vd = v_desc + (slot * C::kF16 >> 4);
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k)
                mma_f16_tmem(tmem + kO + b * kTile, tmem + b * kTile + 8 * k, vd + (k * 2048 >> 4), id_o, s > 0 || k > 0);
              commit(smem_addr(&sm.o_full[b]));
              if (!PAIR || b == 1 || !both) commit(smem_addr(&sm.empty16[slot]));
            }
            __syncwarp();
          }
          if (s + 1 < n[b]) {  // the next S = Q x K^T
            const uint32_t j = 2u * (base + (PAIR ? s + 1 : 2 * (s + 1) + b)), slot = j % NF;
            if (!PAIR || b == 0) ok = bar_wait(smem_addr(&sm.full16[slot]), (j / NF) & 1, gave_up) && ok;
            __syncwarp();
            fence_after();
            if (elect() && ok) {
              const uint64_t qd = q_desc + (PAIR ? b * C::kF16 >> 4 : 0), kd = k_desc + (slot * C::kF16 >> 4);
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const int off = ((k / 4) * C::kPanel + (k % 4) * 32) >> 4;
                mma_f16(tmem + b * kTile, qd + off, kd + off, id_s, k > 0);
              }
              commit(smem_addr(&sm.s_full[b]));
              if (!PAIR || b == 1 || !both) commit(smem_addr(&sm.empty16[slot]));
              if (s + 2 == n[b] && (b == 1) == (n[1] == n[0])) commit(smem_addr(&sm.q_free));  // the last with these queries
            }
            __syncwarp();
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) break;
      base += nt;
      count[0] += n[0];
      count[1] += n[1];
    }
  };

  auto convert_tiles = [&]() {
    // ---- an item's queries, then its tiles, into f16: a thread owns a row
    const int own = tid - kConvWarp * 32;
    const bool vec = ((reinterpret_cast<uintptr_t>(a.q) | (a.qst * 2) | (a.qsh * 2)) & 15) == 0;
    const uint32_t turn = static_cast<uint32_t>(own & 7) << 4;  // the swizzle of this row
    Walk<N, kCost> it(a, start, my_units);
    auto row_at = [&](const RowTile& r, int h, int row) {  // where a row's queries begin
      const uint32_t flat = static_cast<uint32_t>(r.rt * N + min(row, r.rows - 1)), tok = flat / static_cast<uint32_t>(a.group);
      return (r.first + static_cast<int64_t>(tok)) * a.qst + (h * a.group + static_cast<int>(flat - tok * a.group)) * a.qsh;
    };
    int seg = 0, i = 0;
    bool more, ok = true;
    do {
      const RowTile r = it.r;
      const int h = it.h, t0 = it.t0, t1 = it.t1, r0 = r.rt * N;
      // Queries as f16, each row over the power of two that leaves its largest element in [2^13, 2^14): kLanes lanes a
      // row, kBatch rows of a lane group in flight. Rows' places and scales are found while the last item's queries are
      // still in use.
      constexpr int kLanes = D / 8, kRows = 128 / kLanes, kBatch = 8;
      static_assert(N % (kRows * kBatch) == 0, "whole batches");
      const int chunk = lane % kLanes, sub = own / kLanes;
      for (int row = own; row < N; row += 128) sm.qrow[row] = row_at(r, h, row);
      ok = named_all(2, 128, ok);
      if (!ok) break;
      auto load = [&](int row, QT* e) {
        const QT* q = static_cast<const QT*>(a.q) + sm.qrow[row] + chunk * 8;
        if (vec) {
          const uint4 u = *reinterpret_cast<const uint4*>(q);
          memcpy(e, &u, 16);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) e[k] = q[k];
        }
      };
#pragma unroll 1
      for (int row0 = 0; row0 < r.rows; row0 += kRows * kBatch) {  // the same for every lane; places behind the rows repeat the last
        QT e[kBatch][8];
#pragma unroll
        for (int z = 0; z < kBatch; ++z) load(row0 + z * kRows + sub, e[z]);
        float amax[kBatch];
#pragma unroll
        for (int z = 0; z < kBatch; ++z) {
          auto m = abs2(e[z]);
#pragma unroll
          for (int k = 2; k < 8; k += 2) m = __hmax2(m, abs2(e[z] + k));
          amax[z] = fmaxf(to_f(m.x), to_f(m.y));
        }
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1)
#pragma unroll
          for (int z = 0; z < kBatch; ++z) amax[z] = fmaxf(amax[z], __shfl_xor_sync(0xffffffffu, amax[z], o));
#pragma unroll
        for (int z = 0; z < kBatch; ++z) {
          const int eq = min(max(static_cast<int>(__float_as_uint(amax[z]) >> 23) - 127 - 13, -110), 110);
          if (chunk == 0) sm.qscale[seg & 3][row0 + z * kRows + sub] = pow2i(eq);
        }
      }
      __syncwarp();
      if (seg > 0) ok = bar_wait(smem_addr(&sm.q_free), (seg - 1) & 1, gave_up);
      ok = __all_sync(0xffffffffu, ok);
#pragma unroll 1
      for (int row0 = 0; row0 < r.rows && ok; row0 += kRows * kBatch) {
        QT e[kBatch][8];
#pragma unroll
        for (int z = 0; z < kBatch; ++z) load(row0 + z * kRows + sub, e[z]);
#pragma unroll
        for (int z = 0; z < kBatch; ++z) {
          const int row = row0 + z * kRows + sub;
          const uint32_t inverse = 0x7f000000u - __float_as_uint(sm.qscale[seg & 3][row]);  // of a power of two
          const float down = __uint_as_float(a.negate ? inverse | 0x80000000u : inverse);
          uint32_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = mul2(make_float2(to_f(e[z][2 * k]), to_f(e[z][2 * k + 1])), make_float2(down, down));
            v[k] = half2_bits(f.x, f.y);
          }
          *reinterpret_cast<uint4*>(q_smem + (row / kTile) * C::kF16 + (chunk / 8) * C::kPanel + (row % kTile) * 128 +
                                    (((chunk % 8) ^ (row & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
      if (own == 0 && ok) {
        sm.nan[seg & 3] = 0;
        sm.item[seg & 3] = {r.b, r.first, r.n, r.ctx, r.rows, r.end, r.part, r0, h, t0, t1, r.tiles};
      }
      fence_async_shared();
      ok = named_all(2, 128, ok);  // and the flag is cleared before a tile of the item sets it
      if (!ok) break;
      if (lane == 0) bar_arrive(smem_addr(&sm.q_ready[seg & 3]));

      more = it.next(a);
      if (!more && own == 0) a.cut[blockIdx.x] = cut_item<N>(runs, blockIdx.x, r, h, t0, t1);
      if (more)  // the next item's queries come from memory by the time they are needed
        for (int row = own; row < it.r.rows; row += 128) {
          const QT* q = static_cast<const QT*>(a.q) + row_at(it.r, it.h, row);
#pragma unroll
          for (int d = 0; d < D; d += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + d));
        }

      for (int t = t0; t < t1 && ok; ++t, ++i) {
        const int slot = t * kTile + own;
        const bool masked = t >= r.part;  // not every row sees every slot
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          const uint32_t j = 2u * i + part, from = j % NS, to = j % NF;
          ok = bar_wait(smem_addr(&sm.full[from]), (j / NS) & 1, gave_up);
          if (j >= NF) ok = bar_wait(smem_addr(&sm.empty16[to]), (j / NF - 1) & 1, gave_up) && ok;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint8_t* src = ring + from * C::kF8 + own * D;
          uint8_t* dst = f16 + to * C::kF16 + own * 128;
          // a row of D bytes is swizzled within 128 bytes, or within 64 by the row's second and third bit
          const uint32_t src_turn = D == 128 ? turn : static_cast<uint32_t>((own >> 1) & 3) << 4;
          bool nan = false;
          auto convert = [&](auto check) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint4 u = *reinterpret_cast<const uint4*>(src + ((16u * c) ^ src_turn));
              if (decltype(check)::value) {
                // Slots behind the sequence hold no values, and a NaN value must not reach the rows that do not see it
                // through a weight of 0: both are cleared here, and the rows that see a NaN get it at the item's end.
                if (slot >= r.end) {
                  u = make_uint4(0, 0, 0, 0);
                } else if ((nan_codes(u.x) | nan_codes(u.y) | nan_codes(u.z) | nan_codes(u.w)) & 0x80808080u) {
                  nan = true;
#pragma unroll 1
                  for (int z = 0; z < 4; ++z) {
                    const uint32_t x = z == 0 ? u.x : (z == 1 ? u.y : (z == 2 ? u.z : u.w));
                    const uint32_t y = x & ~__vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu);
                    if (z == 0) u.x = y;
                    else if (z == 1) u.y = y;
                    else if (z == 2) u.z = y;
                    else u.w = y;
                  }
                }
              }
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
              uint32_t v[8];
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(v[2 * z]) : "h"(static_cast<uint16_t>(w[z] & 0xffff)));
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(v[2 * z + 1]) : "h"(static_cast<uint16_t>(w[z] >> 16)));
              }
              uint8_t* panel = dst + (c / 4) * C::kPanel;
              *reinterpret_cast<uint4*>(panel + ((32u * (c % 4)) ^ turn)) = make_uint4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<uint4*>(panel + ((32u * (c % 4) + 16u) ^ turn)) = make_uint4(v[4], v[5], v[6], v[7]);
            }
          };
          if (part == 1 && masked) convert(std::true_type{});
          else convert(std::false_type{});
          if (nan) sm.nan[seg & 3] = 1;
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            bar_arrive(smem_addr(&sm.empty[from]));
            bar_arrive(smem_addr(&sm.full16[to]));
          }
        }
      }
      ++seg;
    } while (more);
    if (ok) ok = bar_wait(smem_addr(&sm.q_free), (seg - 1) & 1, gave_up);
    if (__all_sync(0xffffffffu, ok)) {
      if (own == 0) sm.item[seg & 3].t0 = sm.item[seg & 3].t1 = 0;  // no further item
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&sm.q_ready[seg & 3]));
    }
  };

  auto softmax = [&]() {
    // ---- weights and sums: a thread owns a row of its stream
    const int b = uniform(warp >> 2), quarter = uniform(warp & 3);
    const int own = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_at = lanes + b * kTile, o_at = lanes + kO + b * kTile;
    const int page_shift = 31 - __clz(a.c.block) - 4;  // sixteen slots g are in page g >> page_shift
    int base = 0, count[2] = {0, 0};
    for (int seg = 0;; ++seg) {
      const bool ok = bar_wait(smem_addr(&sm.q_ready[seg & 3]), (seg >> 2) & 1, gave_up);
      // The eight warps meet once an item (below), and leave together: whoever gets no item says so there.
      if (!__all_sync(0xffffffffu, ok)) {
        named_all(1, 256, false);
        break;
      }
      const typename C::Item& it = sm.item[seg & 3];
      const int t0 = uniform(it.t0), nt = uniform(it.t1) - t0, rows = uniform(it.rows);
      if (nt <= 0) {
        named_all(1, 256, true);
        break;
      }
      const int n[2] = {steps(nt, rows, 0), steps(nt, rows, 1)};
      const int steps_here = b == 0 ? n[0] : n[1], count_here = b == 0 ? count[0] : count[1];
      const int ctx = uniform(it.ctx);
      const int row = PAIR ? b * kTile + own : own;  // within the item
      const bool rows_here = (PAIR ? b * kTile : 0) + quarter * 32 < rows;
      const float scale = a.scale * sm.qscale[seg & 3][min(row, rows - 1)];
      // slots before this are seen by all of the warp's rows
      const int warp_row = it.r0 + (PAIR ? b * kTile : 0) + quarter * 32;
      const int all_seen = uniform(ctx + (a.tree ? 0 : min(it.n - 1, warp_row / a.group) + 1));
      float ref = kNegInf, l = 0.f;
      for (int s = 0; s < steps_here; ++s) {
        const int step = PAIR ? s : 2 * s + b, ti = base + step, slot0 = (t0 + step) * kTile;
        const float4* pages = sm.page[ti % kMetaRing];
        bar_wait(smem_addr(&sm.s_full[b]), (count_here + s) & 1, gave_up);
        fence_after();
        if (rows_here) {
          const bool masked = slot0 + kTile > all_seen;
          uint64_t vis[2] = {~0ull, ~0ull};  // slots of the tile that the row sees
          if (masked) {
            const int token = min(it.n - 1, static_cast<int>(static_cast<uint32_t>(it.r0 + row) / static_cast<uint32_t>(a.group)));
            const int seen = (a.tree ? ctx : ctx + token + 1) - slot0;  // slots before this are seen
#pragma unroll
            for (int k = 0; k < 2; ++k)
              vis[k] = seen >= 64 * k + 64 ? ~0ull : (seen <= 64 * k ? 0ull : (1ull << (seen - 64 * k)) - 1ull);
            if (a.tree) {
              const uint8_t* m8 = a.tree + (static_cast<int64_t>(it.b) * a.max_tokens + token) * a.max_tokens - ctx + slot0;
              const int from = max(0, seen), to = min(kTile, it.end - slot0);
#pragma unroll 4
              for (int c = from; c < to; ++c) {
                const uint64_t bit = static_cast<uint64_t>(m8[c] != 0) << (c & 63);
                vis[0] |= c < 64 ? bit : 0ull;
                vis[1] |= c < 64 ? 0ull : bit;
              }
            }
            __syncwarp();
          }
          auto bits = [&](int g) { return static_cast<uint32_t>((g < 4 ? vis[0] : vis[1]) >> (16 * (g & 3))); };
          // the largest exponent; NaN scores are passed over here
          float m = kNegInf;
          uint32_t x[kTile];
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld<32>(s_at + 32 * k, x + 32 * k);
          wait_ld();
          if (masked) {
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              const uint32_t v = bits(g);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (!((v >> j) & 1)) x[16 * g + j] = 0xff800000u;
            }
          }
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            float top[3] = {__uint_as_float(x[16 * g]), __uint_as_float(x[16 * g + 1]), __uint_as_float(x[16 * g + 2])};
#pragma unroll
            for (int j = 3; j < 15; ++j) top[j % 3] = fmaxf(top[j % 3], __uint_as_float(x[16 * g + j]));
            const float4 meta = pages[g >> page_shift];
            m = fmaxf(m, fmaf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], __uint_as_float(x[16 * g + 15]))), scale * meta.x,
                              meta.y));
          }
          const bool far = m - ref > kFar;  // true from no reference to any; false for m = -inf
          if (__any_sync(0xffffffffu, far)) {
            const float now = far ? ceilf(m) : ref;
            const float by = ref == now ? 1.f : exp2_whole(ref - now);
            ref = now;
            l *= by;
            if (s > 0) {
              bar_wait(smem_addr(&sm.o_full[b]), (count_here + s - 1) & 1, gave_up);
              fence_after();
#pragma unroll 1
              for (int k = 0; k < D / 16; ++k) {
                uint32_t x[16];
                tmem_ld<16>(o_at + 16 * k, x);
                wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * by);
                tmem_st16(o_at + 16 * k, x);
              }
            }
          }
          const float from = ref == kNegInf ? 0.f : ref;
          // weights in place of the scores, and their sum
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const float4 meta = pages[g >> page_shift];
            float cs = scale * meta.x;
            if (cs == 0.f) cs = 1e-37f;  // what is not seen stays at -inf
            const float c0 = meta.y - from;
            float2 sum = make_float2(0.f, 0.f);
            uint32_t p[8];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const int c = 16 * g + j;
              const float2 y = fma2(make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), make_float2(cs, cs),
                                    make_float2(c0, c0));
              const float2 w = make_float2(ex2_fast(y.x), ex2_fast(y.y));
              sum = add2(sum, w);
              p[j / 2] = half2_bits(w.x, w.y);
            }
            l = fmaf(sum.x + sum.y, meta.z, l);
            tmem_st8(s_at + 8 * g, p);
          }
          wait_st();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&sm.p_ready[b]));
      }

      // ---- the item's results, or its share of them
      if (steps_here > 0) bar_wait(smem_addr(&sm.o_full[b]), (count_here + steps_here - 1) & 1, gave_up);
      if (!PAIR) {
        sm.ref[seg & 1][b][own] = ref;
        sm.sum[seg & 1][b][own] = l;
      }
      // both streams' products are done; and a stream without steps does not run ahead
      fence_before();
      if (!named_all(1, 256, true)) break;
      fence_after();
      float a0 = 1.f, a1 = 0.f;  // factors of the own and the other stream's sums
      if (!PAIR) {
        const float other = sm.ref[seg & 1][1 - b][own];
        float top = fmaxf(ref, other);
        if (top == kNegInf) top = 0.f;
        a0 = exp2_whole(ref - top);
        a1 = exp2_whole(other - top);
        l = fmaf(a0, l, a1 * sm.sum[seg & 1][1 - b][own]);
        ref = fmaxf(ref, other);
      }
      const bool whole = t0 == 0 && nt == it.tiles;
      const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (t0 > 0 ? 0 : 1);
      if (rows_here && (!PAIR || steps_here > 0)) {
        const int tok = static_cast<int>(static_cast<uint32_t>(it.r0 + min(row, rows - 1)) / static_cast<uint32_t>(a.group));
        const int head = it.h * a.group + (it.r0 + min(row, rows - 1) - tok * a.group);
        QT* out = static_cast<QT*>(a.out) + (it.first + static_cast<int64_t>(tok)) * a.ost + head * a.osh;
        const bool vec = ((reinterpret_cast<uintptr_t>(a.out) | (a.ost * 2) | (a.osh * 2)) & 15) == 0;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (!whole && row < rows && (PAIR || b == 0)) a.part_ml[part * N + row] = make_float2(ref, l);
        const bool nan = sm.nan[seg & 3] != 0;  // set before the weights of its tile were used
        // the dimensions from d on in which a value that this row sees is NaN
        auto mark_nan = [&](auto& v, int d) {
          const int last = min(it.end, it.t1 * kTile);
          for (int slot = max(t0, it.part) * kTile; slot < last; ++slot) {
            if (slot >= ctx && !sees(a, it.b, tok, slot - ctx)) continue;
            const int id = a.c.table[static_cast<int64_t>(it.b) * a.c.max_blocks + slot / a.c.block];
            if (id < 0 || id >= a.c.num_blocks) continue;
            const uint8_t* code = a.c.v + id * a.c.sb + it.h * a.c.sh + (slot % a.c.block) * a.c.ss + d;
#pragma unroll
            for (int k = 0; k < static_cast<int>(sizeof(v) / sizeof(v[0])); ++k)
              if ((code[k] & 0x7f) == 0x7f) v[k] = __int_as_float(0x7fffffff);
          }
        };
        if constexpr (PAIR) {
          // Four lanes exchange 64 bytes of their rows, so that a store instruction meets eight rows, not 32. Where the
          // streams add each other's sums (below) that costs more than it gives: 128 rows of 64 sequences, 216 against 206 us.
          const int row4 = row & ~3, part4 = lane & 3;
          QT* out4[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            out4[k] = reinterpret_cast<QT*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), (lane & ~3) + k));
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            uint32_t x[32];
            float v[32];
            tmem_ld<32>(o_at + d, x);
            wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(x[k]);
            if (nan) mark_nan(v, d);
            __syncwarp();
            if (!whole) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint4 u[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) memcpy(&u[k], v + 16 * half + 4 * k, 16);
                exchange4(u, lane);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (row4 + k < rows)
                    *reinterpret_cast<uint4*>(a.part_o + (part * N + row4 + k) * D + d + 16 * half + 4 * part4) = u[k];
              }
            } else {
              QT h[32];
#pragma unroll
              for (int k = 0; k < 32; ++k) h[k] = from_f<QT>(v[k] * inv);
              if (vec) {
                uint4 u[4];
                memcpy(u, h, 64);
                exchange4(u, lane);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (row4 + k < rows) *reinterpret_cast<uint4*>(out4[k] + d + 8 * part4) = u[k];
              } else if (row < rows) {
#pragma unroll
                for (int k = 0; k < 32; ++k) out[d + k] = h[k];
              }
            }
            __syncwarp();
          }
        } else {
          // the streams take half of the dimensions each
          const bool both = n[0] > 0 && n[1] > 0;
#pragma unroll 1
          for (int d = b * (D / 2); d < (b + 1) * (D / 2); d += 16) {
            uint32_t x[16], z[16];
            float v[16];
            if (steps_here > 0) tmem_ld<16>(o_at + d, x);
            if (both || steps_here == 0) tmem_ld<16>(lanes + kO + (1 - b) * kTile + d, z);
            wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              v[k] = steps_here > 0 ? a0 * __uint_as_float(x[k]) : 0.f;
              if (both || steps_here == 0) v[k] = fmaf(a1, __uint_as_float(z[k]), v[k]);
            }
            if (nan) mark_nan(v, d);
            if (row >= rows) {
            } else if (!whole) {
              float4* to = reinterpret_cast<float4*>(a.part_o + (part * N + row) * D + d);
#pragma unroll
              for (int k = 0; k < 4; ++k) to[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            } else {
              QT h[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) h[k] = from_f<QT>(v[k] * inv);
              if (vec) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  uint4 u;
                  memcpy(&u, h + 8 * k, 16);
                  *reinterpret_cast<uint4*>(out + d + 8 * k) = u;
                }
              } else {
#pragma unroll
                for (int k = 0; k < 16; ++k) out[d + k] = h[k];
              }
            }
            __syncwarp();
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&sm.done));
      base += nt;
      count[0] += n[0];
      count[1] += n[1];
    }
  };

  // 512 threads of 128 registers; a softmax thread holds a row's 128 scores and takes from the others (176, 80 and 80:
  // prompts 5% slower than with 168, 88 and 88)
  uint32_t begun = 0;
  if (warp < kConvWarp) {
    more_registers<168>();
    if (work) softmax();
  } else if (warp < kLoadWarp) {
    fewer_registers<88>();
    if (work) convert_tiles();
  } else {
    fewer_registers<88>();
    if (work && warp == kLoadWarp) begun = copy_tiles<N, kCost, D, NS>(a, start, my_units, kmap, vmap, ring, sm, gave_up);
    if (work && warp == kMmaWarp) products();
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (sm.gave_up) drain<NS>(sm, warp == kLoadWarp, begun, warp == kMmaWarp);
  if (warp == kMmaWarp) tmem_free(tmem, 512);
  if (tid == 0) {
    a.gave_up[blockIdx.x] = (sm.gave_up ? kGaveUp : 0) | (sm.outside ? kOutside : 0);
    if (!work || sm.gave_up) a.cut[blockIdx.x] = make_int4(0, 0, 0, 0);  // what was begun is not to be joined
  }
  griddep_launch_dependents();
}

template <typename QT, int D, bool PAIR>
cudaError_t launch_wide(const Kv8AttnArgs& a, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  using C = Wide<D, PAIR>;
  const cudaError_t e = launch_tiles(kv8_wide_kernel<QT, C>, a, C::kThreads, C::kSmem, k, v, st);
  return e != cudaSuccess ? e : launch_join<QT, D, C::N>(a, st);
}

template <typename QT>
cudaError_t launch_type(const Kv8AttnArgs& a, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  if (a.c.D == 128) return rows == 128 ? launch_wide<QT, 128, false>(a, k, v, st) : launch_wide<QT, 128, true>(a, k, v, st);
  return rows == 128 ? launch_wide<QT, 64, false>(a, k, v, st) : launch_wide<QT, 64, true>(a, k, v, st);
}

}  // namespace

cudaError_t launch_kv8_wide(const Kv8AttnArgs& a, int dtype, int rows, const CUtensorMap& k, const CUtensorMap& v,
                            cudaStream_t st) {
  return dtype == SPEC_BF16 ? launch_type<__nv_bfloat16>(a, rows, k, v, st) : launch_type<__half>(a, rows, k, v, st);
}

}  // namespace specv
