// latent_wide.cu -- attention over the paged latent cache for many rows: the
// target's pass over draft positions and trees of many heads, and prompts.
//
// Here 128 rows (token, head) are the rows of both products, a thread owns one,
// and the maximum, sum and reference of a row are its registers. Scores of 64
// slots and results of 256 dimensions share tensor memory with half of the
// queries: 2 x 64 columns of scores that become the weights in place, 256 of
// results, 128 of queries. A row's 512 results do not fit beside anything else,
// so a row tile is two items, one for each half of the value dimensions, and
// both compute its scores: (2 (C + R) + C) / (C + R + C) = 1.53 times the products.
// That buys a first operand that lies in tensor memory in three of four
// products: shared memory then only has to deliver the tile, which is what
// bounds few rows on many slots (latent_rows.cuh), and the scores of the next tile
// are computed while the weights of this one are made.
//
// Shared memory: the queries' other dimensions (80 KB) and two tiles of 64
// slots (144 KB) in pieces of the value dimensions of an item, each given back when
// its last product has read it. The piece that holds no values of the item comes
// first in a tile's scores, so that the values, which their own product gives back
// last, are asked for as late as possible (long contexts 966 -> 719 us).
//
// What bounds it. Two sequences of 110,000 to 131,072 tokens x 9 x 128 heads, bf16: 675
// us, 926 TFLOP/s, 0.48 of a library product and 0.73 with the scores counted twice;
// 2700 clocks a tile, of which the products take 1990, then waits for the values'
// piece and those of the issuing warp. 16 trees of 61 tokens x 16 heads, fp16: 142
// us, tensor pipe busy for 40%; an item's queries, first maximum, masked tiles and
// results take a third. 256 dimensions (three prompts of 500 to 1500): 146 us, 885 TFLOP/s.
#include <string.h>

#include "latent_attn.cuh"

namespace specv {

namespace {

// Units of an item beside its tiles (see Runs): its queries and results. Three prompts of 500 to 1500 tokens: 175 us with 0, 156
// with 2, 146 with 4 and 8; 16 trees of 61 tokens: 148, 147, 142, 144.
constexpr int kCost = 4;
constexpr int kRows = 128, kSlots = 64;  // rows of an item, slots of a tile
constexpr int kChunk = kSlots * 128, kQChunk = kRows * 128;  // bytes of 64 dimensions of a tile, of the queries
constexpr int kPieces = 4;  // ring: pieces of two tiles (of four, where a piece is all values); a tile's first one brings the shared dimensions
constexpr uint32_t kQAt = 256, kSAt = 384;  // tensor memory: results at 0, queries, scores
constexpr int kWideThreads = 128 + 128 + 64;  // weights, queries, copies and products
constexpr int kBudget = 232448;

struct Small {
  alignas(8) uint64_t full[kPieces], empty[kPieces];
  alignas(8) uint64_t s_full[2], p_full[2], pv_done[2], q_full, q_free, drain;
  int tmp[64];
  int odd[2];  // item number + 1 where a value that not every row sees is not finite
  uint32_t tmem;
  int gave_up, outside;
};
static_assert(5 * kQChunk + kPieces * 4 * kChunk + 2 * kChunk + sizeof(Small) + 1024 <= kBudget, "shared memory");

// 64 columns of the warp's lanes.
__device__ __forceinline__ void ld64(uint32_t addr, uint32_t* r) {
  tmem_ld<32>(addr, r);
  tmem_ld<32>(addr + 32, r + 32);
}

// An item's tiles of 64 slots.
struct Span {
  int s0, s1, part;
};
__device__ __forceinline__ Span span_of(const LatentAttnArgs& a, const RowTile& r, int t0, int t1) {
  Span s;
  s.s0 = 2 * t0;
  s.s1 = min(2 * t1, (r.end + kSlots - 1) / kSlots);
  s.part = (r.ctx + (a.tree ? 0 : r.rt * kRows / a.group + 1)) / kSlots;  // from here on some row does not see every slot
  return s;
}

// PC: chunks of 64 value dimensions of an item, HALVES: items that a row tile's are shared out to.
template <typename QT, int PC, int HALVES>
__global__ void __launch_bounds__(kWideThreads, 1)
    latent_wide_kernel(const __grid_constant__ LatentAttnArgs a, const __grid_constant__ CUtensorMap map) {
  extern __shared__ uint8_t dyn[];
  using B = Bits<QT>;
  constexpr int pc = PC, vd = 64 * PC, halves = HALVES, dims = vd * HALVES, piece = PC * kChunk;
  uint8_t* q_smem = dyn + ((1024u - (smem_addr(dyn) & 1023u)) & 1023u);  // dimensions that are no values of the item, shared ones
  uint8_t* ring = q_smem + ((halves - 1) * pc + 1) * kQChunk;
  uint8_t* sh = ring + kPieces * piece;
  Small& sm = *reinterpret_cast<Small*>(sh + kPieces / halves * kChunk);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = uniform(tid >> 5);
  constexpr int kQueryWarp = 4, kLoadWarp = 8, kMmaWarp = 9;
  volatile int* gave_up = &sm.gave_up;

  if (tid == 0) {
    for (int i = 0; i < kPieces; ++i) {
      bar_init(smem_addr(&sm.full[i]), 1);
      bar_init(smem_addr(&sm.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&sm.s_full[i]), 1);
      bar_init(smem_addr(&sm.p_full[i]), 4);
      bar_init(smem_addr(&sm.pv_done[i]), 1);
    }
    bar_init(smem_addr(&sm.q_full), 4);
    bar_init(smem_addr(&sm.q_free), 1);
    bar_init(smem_addr(&sm.drain), 1);
    fence_bar_init();
    sm.gave_up = 0;
    sm.outside = 0;
    sm.odd[0] = sm.odd[1] = 0;
    prefetch_map(&map);
  }
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&sm.tmem), 512);
  griddep_wait();
  Runs runs;
  Start start;
  const int part_of_run = a.gang ? blockIdx.x / a.gang : blockIdx.x;
  fence_before();
  const bool work = uniform(find_items<kRows, kCost>(a, &runs, &start, sm.tmp)) != 0;
  const int64_t my_units = work ? runs.begin(part_of_run + 1) - runs.begin(part_of_run) : 0;
  __syncthreads();
  fence_after();
  const uint32_t tmem = uniform(sm.tmem);

  uint32_t fill = 0;  // ring slots that copies were begun into
  if (work && warp == kLoadWarp) {
    // ---- copies: a tile's piece that is no value of the item with its shared dimensions, then its values
    Items<kRows, kCost> it(a, start, my_units);
    const int bs = a.c.block, rows = min(bs, kSlots), ppt = kSlots / rows;  // slots of a copy, copies of 64 dimensions
    bool ok = true;
    do {
      if (it.t0 >= it.t1) continue;
      const Span sp = span_of(a, it.r, it.t0, it.t1);
      const int32_t* table = a.c.table + static_cast<int64_t>(it.r.b) * a.c.max_blocks;
      const int sub = lane & (ppt - 1), c = lane / ppt;
      auto block_of = [&](int s) {  // of the lane's slots of tile s
        const int64_t slot0 = static_cast<int64_t>(s) * kSlots + sub * rows;
        int id = -1;  // behind the sequence
        if (slot0 < it.r.end) {
          id = table[slot0 / bs];
          if (id < 0 || id >= a.c.num_blocks) id = -2;  // outside the pool
        }
        return id;
      };
      int next = block_of(sp.s0);
#pragma unroll 1
      for (int s = sp.s0; s < sp.s1 && ok; ++s) {
        const int id = next, in_block = (s * kSlots + sub * rows) & (bs - 1);
        next = block_of(s + 1);  // on its way meanwhile
        if (__any_sync(0xffffffffu, id == -2)) sm.outside = 1;
        const uint32_t inside = __popc(__ballot_sync(0xffffffffu, id >= 0 && c == 0));
        const int y = a.order ? id : in_block, z = a.order ? in_block : id;
        auto copy_piece = [&](int p, bool shared) {  // value dimensions p * vd on; the shared ones with them
          const uint32_t slot = fill % kPieces, bar = smem_addr(&sm.full[slot]);
          if (fill >= kPieces) ok = bar_wait(smem_addr(&sm.empty[slot]), (fill / kPieces - 1) & 1, gave_up);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) return;
          if (lane == 0) bar_expect(bar, inside * rows * 128 * (shared ? pc + 1 : pc));
          __syncwarp();
          if (id >= 0 && c < pc)
            load_3d(smem_addr(ring + slot * piece + c * kChunk + sub * rows * 128), &map, bar, p * vd + c * 64, y, z);
          if (shared && id >= 0 && c == pc) load_3d(smem_addr(sh + slot / halves * kChunk + sub * rows * 128), &map, bar, dims, y, z);
          ++fill;
        };
        if (halves == 2) copy_piece(1 - it.h, true);
        if (!ok) break;
        copy_piece(it.h, halves == 1);
      }
    } while (ok && it.next(a));
  } else if (work && warp == kMmaWarp) {
    // ---- products: the warp waits together, one lane issues
    constexpr uint32_t format = 1u << 4 | B::kFormat << 7 | B::kFormat << 10 | static_cast<uint32_t>(kRows >> 4) << 24;
    constexpr uint32_t id_s = format | static_cast<uint32_t>(kSlots >> 3) << 17;
    constexpr uint32_t id_o = format | 1u << 16 | static_cast<uint32_t>(vd >> 3) << 17;  // the entries lie with N contiguous
    const uint64_t e_desc = smem_desc(smem_addr(ring), 16, 1024, 2), s_desc = smem_desc(smem_addr(sh), 16, 1024, 2),
                   q_desc = smem_desc(smem_addr(q_smem), 16, 1024, 2),
                   r_desc = moved(q_desc, (halves - 1) * pc * kQChunk),
                   c_desc = smem_desc(smem_addr(ring), kChunk, 1024, 2);
    Items<kRows, kCost> it(a, start, my_units);
    bool ok = true;
    uint32_t f = 0;  // pieces whose scores are begun
    int i = 0, j = 0, seg = 0;  // tiles whose scores, whose results are begun
    do {
      if (it.t0 >= it.t1) continue;
      ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.q_full), seg & 1, gave_up));
      if (!ok) break;
      fence_after();
      const int t0 = uniform(it.t0), t1 = uniform(it.t1);
      const Span sp = span_of(a, it.r, t0, t1);
      const int s0 = uniform(sp.s0), s1 = uniform(sp.s1);
      auto scores = [&](bool last) {  // S[i & 1] = queries x tile, the values last: they are given back last (by the results)
        const uint32_t to = uniform(tmem + kSAt + (i & 1) * kSlots);
        auto ready = [&](uint32_t slot) {
          ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.full[slot]), (f / kPieces) & 1, gave_up));
          if (ok) fence_after();
          return ok;
        };
        uint32_t slot = f % kPieces;
        if (!ready(slot)) return false;
        const uint64_t sd = moved(s_desc, slot / halves * kChunk);
        if (halves == 2) {
          const uint64_t ed = moved(e_desc, slot * piece);
          if (elect()) {
#pragma unroll
            for (int c = 0; c < pc; ++c)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_f16(to, q_desc + (c * kQChunk >> 4) + 2 * k, ed + (c * kChunk >> 4) + 2 * k, id_s, c > 0 || k > 0);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16(to, r_desc + 2 * k, sd + 2 * k, id_s, true);
            commit(smem_addr(&sm.empty[slot]));
          }
          __syncwarp();
          ++f;
          slot = f % kPieces;
          if (!ready(slot)) return false;
        }
        ++f;
        const uint64_t ed = moved(e_desc, slot * piece);
        if (elect()) {
          if (halves == 1)
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16(to, r_desc + 2 * k, sd + 2 * k, id_s, k > 0);
#pragma unroll
          for (int c = 0; c < pc; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16_tmem(to, tmem + kQAt + 32 * c + 8 * k, ed + (c * kChunk >> 4) + 2 * k, id_s, true);
          commit(smem_addr(&sm.s_full[i & 1]));
          if (last) commit(smem_addr(&sm.q_free));
        }
        __syncwarp();
        ++i;
        return true;
      };
      if (!scores(s0 + 1 == s1)) break;
#pragma unroll 1
      for (int s = s0; s < s1; ++s, ++j) {
        if (s + 1 < s1 && !scores(s + 2 == s1)) break;
        ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.p_full[j & 1]), (j >> 1) & 1, gave_up));
        if (!ok) break;
        fence_after();
        const uint32_t slot = uniform((static_cast<uint32_t>(j) * halves + halves - 1) % kPieces);
        const uint64_t cd = moved(c_desc, slot * piece);
        const uint32_t p_at = uniform(tmem + kSAt + (j & 1) * kSlots);
        if (elect()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_tmem(tmem, p_at + 8 * k, cd + 128 * k, id_o, s > s0 || k > 0);
          commit(smem_addr(&sm.empty[slot]));
          commit(smem_addr(&sm.pv_done[j & 1]));
        }
        __syncwarp();
      }
      ++seg;
    } while (ok && it.next(a));
  } else if (work && warp >= kQueryWarp && warp < kLoadWarp) {
    // ---- queries: the item's value dimensions into tensor memory (a lane its row), the rest into shared memory
    const int quarter = uniform(warp & 3), own = quarter * 32 + lane;
    const bool vec = ((reinterpret_cast<uintptr_t>(a.q) | (a.qst * 2) | (a.qsh * 2)) & 15) == 0;
    const int used = (dims + a.rot) / 8;  // 16-byte chunks of an entry
    Items<kRows, kCost> it(a, start, my_units);
    int seg = 0;
    bool ok = true;
    do {
      const RowTile& r = it.r;
      if (it.t0 >= it.t1) continue;
      const uint32_t flat = static_cast<uint32_t>(r.rt * kRows + min(own, r.rows - 1)), tok = flat / static_cast<uint32_t>(a.group);
      const QT* q = static_cast<const QT*>(a.q) + (r.first + static_cast<int64_t>(tok)) * a.qst +
                    static_cast<int>(flat - tok * a.group) * a.qsh;
      const bool mine = own < r.rows && a.negate < 2;
      auto load = [&](int c) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (mine && c < used) {
          if (vec) {
            u = *reinterpret_cast<const uint4*>(q + 8 * c);
          } else {
            QT e[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) e[x] = q[8 * c + x];
            memcpy(&u, e, 16);
          }
        }
        return u;
      };
      // The item's value dimensions are fetched while the last item's queries are still in use, the rest is brought to L2.
      uint32_t w[vd / 2];
#pragma unroll
      for (int k = 0; k < vd / 8; ++k) {
        const uint4 u = load(it.h * (vd / 8) + k);
        w[4 * k] = u.x, w[4 * k + 1] = u.y, w[4 * k + 2] = u.z, w[4 * k + 3] = u.w;
      }
      if (halves == 2 && seg > 0)
#pragma unroll
        for (int k = 0; k < vd; k += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + (1 - it.h) * vd + k));
      if (seg > 0) ok = bar_wait(smem_addr(&sm.q_free), (seg - 1) & 1, gave_up);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      fence_after();
#pragma unroll 1
      for (int c = 0; c < (halves - 1) * pc + 1; ++c) {
        const int from = c < (halves - 1) * pc ? (1 - it.h) * (vd / 8) + 8 * c : dims / 8;
        uint8_t* to = q_smem + c * kQChunk + own * 128;
        if (vec) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const bool take = mine && from + k < used;
            copy16(smem_addr(to + ((k ^ (own & 7)) << 4)), take ? q + 8 * (from + k) : q, take);
          }
        } else {
#pragma unroll 1
          for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(to + ((k ^ (own & 7)) << 4)) = load(from + k);
        }
      }
      const uint32_t q_to = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kQAt;
#pragma unroll
      for (int k = 0; k < vd / 2; k += 16) tmem_st16(q_to + k, w + k);
      copies_done();
      wait_st();
      fence_async_shared();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&sm.q_full));
      ++seg;
    } while (it.next(a));
  } else if (work && warp < kQueryWarp) {
    // ---- weights, sums and results: a thread owns a row
    const int quarter = uniform(warp & 3), own = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const bool vec = ((reinterpret_cast<uintptr_t>(a.out) | (a.ost * 2) | (a.osh * 2)) & 15) == 0;
    Items<kRows, kCost> it(a, start, my_units);
    int i = 0;
    int seg = 0;
    if (tid == 0) a.cut[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    do {
      if (it.t0 >= it.t1) continue;
      const RowTile r = it.r;
      const int t0 = uniform(it.t0), t1 = uniform(it.t1), h = uniform(it.h);
      const Span sp = span_of(a, r, t0, t1);
      const int s0 = uniform(sp.s0), s1 = uniform(sp.s1);
      const int flat = r.rt * kRows + own, tok = flat / a.group, head = flat - tok * a.group;
      float ref = kUnset, sum = 0.f;
      bool ok = true;
#pragma unroll 1
      for (int s = s0; s < s1; ++s, ++i) {
        ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.s_full[i & 1]), (i >> 1) & 1, gave_up));
        if (!ok) break;
        fence_after();
        const uint32_t at = lanes + kSAt + (i & 1) * kSlots;
        uint32_t x[64];
        ld64(at, x);
        const bool masked = s >= sp.part;
        if (masked) {
          // As in latent_rows.cuh: slots behind the rows' last, and values that are not finite, are cleared. Two threads a slot.
          const int in = own & 63, slot = s * kSlots + in;
          const uint32_t value = static_cast<uint32_t>(i) * halves + halves - 1;
          ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.full[value % kPieces]), (value / kPieces) & 1, gave_up));
          if (!ok) break;
          uint8_t* row = ring + (value % kPieces) * piece + in * 128;
          if (slot >= r.ctx) {  // every row sees those before
#pragma unroll 1
            for (int c = own >> 6; c < pc; c += 2)
              if (clean_chunks<B, 8>(reinterpret_cast<uint4*>(row + c * kChunk), in & 7, slot >= r.end)) sm.odd[seg & 1] = seg + 1;
          }
          __syncwarp();
        }
        wait_ld();
        settle<64>(x);
        if (a.negate == 1) {
#pragma unroll
          for (int k = 0; k < 64; ++k) x[k] ^= 0x80000000u;
        }
        if (masked) {
          const int from = s * kSlots - r.ctx;  // token of the step in the tile's first slot
          uint64_t vis;
          if (!a.tree) {
            const int64_t n = static_cast<int64_t>(tok) - from + 1;  // slots from the first on that the row sees
            vis = n >= 64 ? ~0ull : (n <= 0 ? 0ull : (1ull << n) - 1);
          } else {
            vis = 0;
#pragma unroll 1
            for (int k = 0; k < kSlots; ++k) {
              const int j = from + k;
              if (j < 0 || (tok < r.n && j < r.n && sees(a, r.b, tok, j))) vis |= 1ull << k;
            }
          }
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (!((vis >> k) & 1)) x[k] = 0xff800000u;
          __syncwarp();
        }
        float top = kNegInf, top2 = kNegInf;  // of the raw scores; the scale is positive
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
          top = fmaxf(top, __uint_as_float(x[k]));
          top2 = fmaxf(top2, __uint_as_float(x[k + 1]));
        }
        top = fmaxf(top, top2) * a.scale;
        const bool pass = top > ref + (kPass + B::kBelow);
        if (__any_sync(0xffffffffu, pass)) {
          const float now = pass ? top - B::kBelow : ref, by = pass ? ex2_fast(ref - now) : 1.f;
          ref = now;
          sum *= by;
          if (s > s0) {
            ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.pv_done[(i - 1) & 1]), ((i - 1) >> 1) & 1, gave_up));
            if (!ok) break;
            fence_after();
#pragma unroll 1
            for (int c = 0; c < vd; c += 32) {
              uint32_t o[32];
              tmem_ld<32>(lanes + c, o);
              wait_ld();
              settle<32>(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * by);
              tmem_st16(lanes + c, o);
              tmem_st16(lanes + c + 16, o + 16);
            }
          }
        }
        const float2 sc = make_float2(a.scale, a.scale), down = make_float2(-ref, -ref);
        float2 part = make_float2(0.f, 0.f);
#pragma unroll
        for (int g = 0; g < 64; g += 32) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 y = fma2(make_float2(__uint_as_float(x[g + 2 * k]), __uint_as_float(x[g + 2 * k + 1])), sc, down);
            w[k] = B::pack(ex2_fast(y.x), ex2_fast(y.y));
            part = add2(part, B::unpack(w[k]));
          }
          tmem_st16(at + g / 2, w);
        }
        sum += part.x + part.y;
        wait_st();
        if (masked) fence_async_shared();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&sm.p_full[i & 1]));
      }
      ok = ok && bar_wait(smem_addr(&sm.pv_done[(i - 1) & 1]), ((i - 1) >> 1) & 1, gave_up);
      if (!__all_sync(0xffffffffu, ok)) break;
      fence_after();

      // ---- the item's results, or its share of them
      const bool whole = t0 == 0 && t1 == r.tiles;
      const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (t0 > 0 ? 0 : 1);
      if (sm.odd[seg & 1] == seg + 1) {  // set before the weights of its tile were ready: what was cleared, times a weight of 0
#pragma unroll 1
        for (int slot = max(max(s0, sp.part) * kSlots, r.ctx); slot < min(r.end, s1 * kSlots); ++slot) {
          const int id = a.c.table[static_cast<int64_t>(r.b) * a.c.max_blocks + slot / a.c.block];
          if (id < 0 || id >= a.c.num_blocks) continue;
          const uint16_t* e = reinterpret_cast<const uint16_t*>(a.c.k + id * a.c.sb + (slot % a.c.block) * a.c.ss) + h * vd;
          const bool saw = tok < r.n && sees(a, r.b, tok, slot - r.ctx);
#pragma unroll 1
          for (int c = 0; c < vd; c += 32) {
            const uint32_t bad = __ballot_sync(0xffffffffu, (e[c + lane] & (B::kExp & 0xffffu)) == (B::kExp & 0xffffu));
            if (bad == 0) continue;
            uint32_t x[32];
            tmem_ld<32>(lanes + c, x);
            wait_ld();
            settle<32>(x);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (saw && (bad >> k) & 1) x[k] = 0x7fffffffu;
            tmem_st16(lanes + c, x);
            tmem_st16(lanes + c + 16, x + 16);
            wait_st();
          }
        }
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      if (!whole && own < r.rows) a.part_ml[part * kRows + own] = make_float2(ref, sum);
      int64_t at[4];  // of the rows that the lane stores a part of: results, or shares in the workspace
      uint32_t here = 0;
      {
        const int64_t to = whole ? (r.first + static_cast<int64_t>(tok)) * a.ost + head * a.osh + h * vd : (part * kRows + own) * vd;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          at[k] = __shfl_sync(0xffffffffu, to, (lane & ~3) + k);
          here |= ((own & ~3) + k < r.rows ? 1u : 0u) << k;
        }
      }
#pragma unroll 1
      for (int c = 0; c < vd; c += 32) {
        uint32_t x[32];
        tmem_ld<32>(lanes + c, x);
        wait_ld();
        settle<32>(x);
        if (!whole) {
#pragma unroll
          for (int g = 0; g < 32; g += 16) {
            uint4 u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) u[k] = make_uint4(x[g + 4 * k], x[g + 4 * k + 1], x[g + 4 * k + 2], x[g + 4 * k + 3]);
            turn_units(u, lane);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if ((here >> k) & 1) *reinterpret_cast<uint4*>(a.part_o + at[k] + c + g + 4 * (lane & 3)) = u[k];
          }
        } else {
          uint4 u[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int z = 0; z < 4; ++z)
              w[z] = B::pack(__uint_as_float(x[8 * k + 2 * z]) * inv, __uint_as_float(x[8 * k + 2 * z + 1]) * inv);
            u[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          turn_units(u, lane);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (!((here >> k) & 1)) continue;
            QT* o = static_cast<QT*>(a.out) + at[k] + c + 8 * (lane & 3);
            if (vec) {
              *reinterpret_cast<uint4*>(o) = u[k];
            } else {
              QT e[8];
              memcpy(e, &u[k], 16);
#pragma unroll
              for (int z = 0; z < 8; ++z) o[z] = e[z];
            }
          }
        }
        __syncwarp();
      }
      fence_before();
      __syncwarp();
      if (tid == 0) it.cut(a, runs);
      __syncwarp();
      ++seg;
    } while (it.next(a));
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (sm.gave_up) {  // what is in flight writes this block's memory: the warps that began it wait for it, with a limit
    if (warp == kLoadWarp) {
#pragma unroll 1
      for (uint32_t k = fill > kPieces ? fill - kPieces : 0; k < fill; ++k)
#pragma unroll 1
        for (int n = 0; n < (1 << 16) && !bar_try(smem_addr(&sm.full[k % kPieces]), (k / kPieces) & 1); ++n) {
        }
    }
    if (warp == kMmaWarp) {
      if (elect()) commit(smem_addr(&sm.drain));
#pragma unroll 1
      for (int n = 0; n < (1 << 16) && !bar_try(smem_addr(&sm.drain), 0); ++n) {
      }
    }
    __syncthreads();
  }
  if (warp == kMmaWarp) tmem_free(tmem, 512);
  if (tid == 0) {
    a.gave_up[blockIdx.x] = (sm.gave_up ? kGaveUp : 0) | (sm.outside ? kOutside : 0);
    if (!work || sm.gave_up) a.cut[2 * blockIdx.x] = make_int4(0, 0, 0, 0);  // what was begun is not to be joined
  }
  griddep_launch_dependents();
}

template <typename QT>
cudaError_t launch_dims(const LatentAttnArgs& a, const CUtensorMap& map, cudaStream_t st) {
  switch (a.c.D) {
    case 128: return launch_items<QT, kRows>(latent_wide_kernel<QT, 2, 1>, a, kWideThreads, kBudget, map, st);
    case 256: return launch_items<QT, kRows>(latent_wide_kernel<QT, 4, 1>, a, kWideThreads, kBudget, map, st);
    case 384: return launch_items<QT, kRows>(latent_wide_kernel<QT, 3, 2>, a, kWideThreads, kBudget, map, st);
    default: return launch_items<QT, kRows>(latent_wide_kernel<QT, 4, 2>, a, kWideThreads, kBudget, map, st);
  }
}

}  // namespace

cudaError_t launch_latent_wide(const LatentAttnArgs& a, int dtype, const CUtensorMap& map, cudaStream_t st) {
  return dtype == SPEC_BF16 ? launch_dims<__nv_bfloat16>(a, map, st) : launch_dims<__half>(a, map, st);
}

}  // namespace specv
