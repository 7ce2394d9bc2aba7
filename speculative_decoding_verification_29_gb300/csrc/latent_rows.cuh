// latent_rows.cuh -- attention whose keys and values all come from one latent
// vector a token, over a paged cache of them, on the tensor cores.
//
// Mathematics. out = sum_t 2^(y_t - ref) c_t / sum_t 2^(y_t - ref) with y_t = s
// log2(e) (q . e_t), e_t the entry (latent vector c_t and shared dimensions).
// All heads read the same entries, so an item's rows are any 16 to 64 of a
// sequence's rows (token, head). A row's reference is set to its largest y (in
// fp16 7 below it) and moves only when one passes that by more than 2^8; the accumulators are scaled then, and
// otherwise a tile needs no maximum at all, only a vote that none is passed.
//
// Orientation. Slots are the 128 rows of both products' first operand: scores
// are E (128 slots x C + 64) times Q^T, results C^T (dimensions x 128 slots)
// times the weights (128 slots x N), so few rows cost few columns, and the tile
// lies in shared memory once for both: as K x M for the scores and, transposed by
// its descriptor, as M x K for the results. The results of all 512 dimensions stay
// in tensor memory (4 x N columns) over an item's tiles. A thread owns a slot and a group
// of rows; the weights are written 16 bytes at a time, rows contiguous.
//
// Shared memory. A tile of 512 + 64 dimensions is 144 KB, the queries of 64
// rows 72 KB: the tile is held as pieces of 128 dimensions, each given back as soon
// as its product has read it, and the shared dimensions' piece becomes the tile's
// weights once the scores are there.
//
// What bounds it. A product of K = 16 takes 49 clocks at N = 64 (41 at 32), not the
// 32 of its arithmetic: the first operand's 4 KB come from shared memory at 128
// bytes a clock. 64 sequences x 9 tokens x 32 heads (1500 to 6500 tokens, bf16):
// 254 us, 630 TFLOP/s, 0.33 of a library product; of some 5900 clocks a tile 3330 are
// the products', 1400 the softmax step and its hand-overs, which nothing overlaps
// because no second tile fits, the rest waits for pieces; an item of 22 tiles has some
// 20,000 clocks for its queries, first and masked tile and results. 64 x 1 token: 70
// us, 4.1 TB/s, 0.62 of a copy; a tile's pieces are given back one after the other
// during its second product, so that about 2000 clocks a tile go by until the next
// one's are there, and start and join take 15 us.
#pragma once

#include <string.h>

#include "latent_attn.cuh"

namespace specv {

namespace {

// ---------------------------------------------------------- configuration --

// Units of an item beside its tiles (see Runs): its queries, first maximum and results. 64 sequences x 9 tokens x 32 heads: 258 us
// with 0, 256 with 1, 254 with 3, 261 with 6; one token each 71, 70, 70, 74.
constexpr int kCost = 3;
constexpr int kPiece = kTile * 256, kShared = kTile * 128;  // bytes: 128 dimensions of a tile, its shared dimensions
constexpr int kMaxPieces = 6, kMaxShared = 2;

// N: rows of an item. P: pieces of a tile.
template <int N_, int P_>
struct LCfg {
  static constexpr int N = N_, P = P_;
  static constexpr int G = 2, HN = N / G;  // groups of four softmax warps, their rows
  static constexpr int kSoft = G * 128, kThreads = kSoft + 64;  // softmax warps, then copies and products
  static constexpr uint32_t kO = 64;              // tensor memory: scores at 0, results of 128 dimensions every 64 columns
  static constexpr int kBudget = 232448 - 1024;
  struct Small {
    alignas(16) float ref[N], fac[N];  // references, and what sums and results are scaled by when they move
    alignas(16) float smax[G][4][HN];  // each warp's largest scores
    float sums[G][4][HN];
    alignas(16) float inv[4 * G][HN];
    int64_t to[G][HN];  // where an item's rows go (elements; -1: no such row)
    alignas(8) uint64_t full[kMaxPieces], empty[kMaxPieces], sh_full[kMaxShared], sh_empty[kMaxShared];
    alignas(8) uint64_t s_full, p_full, o_full, q_full, drain;
    int tmp[64];
    int odd[2];  // item number + 1 where a value that not every row sees is not finite
    uint32_t tmem;
    int gave_up, outside;
  };
  // Pieces and buffers of shared dimensions that fit beside the queries.
  static constexpr int kQ = (2 * P + 1) * N * 128, kRoom = kBudget - static_cast<int>(sizeof(Small)) - kQ;
  static constexpr int kFit = (kRoom - kShared) / kPiece, kRing = kFit < kMaxPieces ? kFit : kMaxPieces;
  static constexpr int kBuffers = kRoom - kRing * kPiece >= 2 * kShared ? 2 : 1;
  static_assert(kRing >= P, "a tile fits");
};

// HN columns of the warp's lanes: 8, 16, 24 or 32.
template <int HN>
__device__ __forceinline__ void ld_cols(uint32_t addr, uint32_t* r) {
  if constexpr (HN == 24) {
    tmem_ld<16>(addr, r);
    tmem_ld<8>(addr + 16, r + 16);
  } else {
    tmem_ld<HN>(addr, r);
  }
}
template <int HN>
__device__ __forceinline__ void st_cols(uint32_t addr, const uint32_t* r) {
#pragma unroll
  for (int k = 0; k < HN; k += 8) tmem_st8(addr + k, r + k);
}

// Sums of v[j] over the warp's lanes, j < C = 8, 16 or 32: lane j (mod C) gets the j-th. v is not kept.
template <int C>
__device__ __forceinline__ float lane_sum(float* v, int lane) {
#pragma unroll
  for (int o = 16; o >= C; o >>= 1)
#pragma unroll
    for (int k = 0; k < C; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
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
template <int HN>
__device__ __forceinline__ float sums_of(float* v, int lane) {
  if constexpr (HN == 24) {
    const float a = lane_sum<16>(v, lane), b = lane_sum<8>(v + 16, lane);
    return lane < 16 ? a : b;
  } else {
    return lane_sum<HN>(v, lane);
  }
}

// ----------------------------------------------------------------- kernel --

template <typename QT, typename C>
__global__ void __launch_bounds__(C::kThreads, 1)
    latent_attention_kernel(const __grid_constant__ LatentAttnArgs a, const __grid_constant__ CUtensorMap map) {
  extern __shared__ uint8_t dyn[];
  using B = Bits<QT>;
  constexpr int N = C::N, HN = C::HN;
  constexpr int pieces = C::P, dims = 128 * pieces, NP = C::kRing, NS = C::kBuffers;
  uint8_t* q_smem = dyn + ((1024u - (smem_addr(dyn) & 1023u)) & 1023u);
  uint8_t* ring = q_smem + C::kQ;
  uint8_t* sh = ring + NP * kPiece;  // shared dimensions, then weights
  typename C::Small& sm = *reinterpret_cast<typename C::Small*>(sh + NS * kShared);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = uniform(tid >> 5);
  constexpr int kLoadWarp = C::kSoft / 32, kMmaWarp = kLoadWarp + 1;
  volatile int* gave_up = &sm.gave_up;

  if (tid == 0) {
    for (int i = 0; i < kMaxPieces; ++i) {
      bar_init(smem_addr(&sm.full[i]), 1);
      bar_init(smem_addr(&sm.empty[i]), 1);
    }
    for (int i = 0; i < kMaxShared; ++i) {
      bar_init(smem_addr(&sm.sh_full[i]), 1);
      bar_init(smem_addr(&sm.sh_empty[i]), 1);
    }
    bar_init(smem_addr(&sm.s_full), 1);
    bar_init(smem_addr(&sm.p_full), C::kSoft / 32);
    bar_init(smem_addr(&sm.o_full), 1);
    bar_init(smem_addr(&sm.q_full), C::kSoft / 32);
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
  const bool work = uniform(find_items<N, kCost>(a, &runs, &start, sm.tmp)) != 0;
  const int64_t my_units = work ? runs.begin(part_of_run + 1) - runs.begin(part_of_run) : 0;
  __syncthreads();
  fence_after();
  const uint32_t tmem = uniform(sm.tmem);

  uint32_t fill = 0, sh_fill = 0;  // ring slots that copies were begun into
  if (work && warp == kLoadWarp) {
    // ---- copies: a tile's pieces, then its shared dimensions
    Items<N, kCost> it(a, start, my_units);
    const int bs = a.c.block, ppt = kTile / bs;
    bool ok = true;
    do {
      if (it.t0 >= it.t1) continue;
      const int pages = (it.r.end + bs - 1) / bs;
      const int32_t* table = a.c.table + static_cast<int64_t>(it.r.b) * a.c.max_blocks;
      auto page_id = [&](int page) {
        int id = -1;  // behind the sequence
        if (page < pages) {
          id = table[page];
          if (id < 0 || id >= a.c.num_blocks) id = -2;  // outside the pool
        }
        return id;
      };
      int id = -1, id_next = page_id(it.t0 * ppt + lane);
#pragma unroll 1
      for (int t = it.t0, g = 0; t < it.t1 && ok; ++t, g += ppt) {
        if ((g & 31) == 0) {  // 32 pages' ids at a time, one a lane; the next 32 are on their way meanwhile
          id = id_next;
          id_next = page_id(t * ppt + 32 + lane);
          if (__any_sync(0xffffffffu, id == -2)) sm.outside = 1;
        }
        const int page = lane & (ppt - 1), half = lane / ppt;
        const int my_id = __shfl_sync(0xffffffffu, id, (g & 31) + page);
        const uint32_t inside = __popc(__ballot_sync(0xffffffffu, my_id >= 0 && lane < ppt));
        const int y = a.order ? my_id : 0, z = a.order ? 0 : my_id;
#pragma unroll 1
        for (int p = 0; p < pieces; ++p, ++fill) {
          const uint32_t slot = fill % NP, bar = smem_addr(&sm.full[slot]);
          if (fill >= NP) ok = bar_wait(smem_addr(&sm.empty[slot]), (fill / NP - 1) & 1, gave_up);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) bar_expect(bar, inside * bs * 256);
          __syncwarp();
          if (my_id >= 0 && half < 2)
            load_3d(smem_addr(ring + slot * kPiece + half * (kTile * 128) + page * bs * 128), &map, bar, p * 128 + half * 64, y, z);
        }
        if (!ok) break;
        const uint32_t slot = sh_fill % NS, bar = smem_addr(&sm.sh_full[slot]);
        if (sh_fill >= NS) ok = bar_wait(smem_addr(&sm.sh_empty[slot]), (sh_fill / NS - 1) & 1, gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) bar_expect(bar, inside * bs * 128);
        __syncwarp();
        if (my_id >= 0 && half < 1) load_3d(smem_addr(sh + slot * kShared + page * bs * 128), &map, bar, dims, y, z);
        ++sh_fill;
      }
    } while (ok && it.next(a));
  } else if (work && warp == kMmaWarp) {
    // ---- products: the warp waits together, one lane issues
    constexpr uint32_t id_s = 1u << 4 | B::kFormat << 7 | B::kFormat << 10 | static_cast<uint32_t>(N >> 3) << 17 | 8u << 24;
    constexpr uint32_t id_o = id_s | 3u << 15;  // both operands lie with M (N) contiguous
    const uint64_t e_desc = smem_desc(smem_addr(ring), 16, 1024, 2), s_desc = smem_desc(smem_addr(sh), 16, 1024, 2),
                   q_desc = smem_desc(smem_addr(q_smem), 16, 1024, 2),
                   c_desc = smem_desc(smem_addr(ring), kTile * 128, 1024, 2),
                   p_desc = smem_desc(smem_addr(sh), kTile * 128, 1024, 2);
    Items<N, kCost> it(a, start, my_units);
    bool ok = true;
    uint32_t f = 0;  // pieces so far
    int i = 0, seg = 0;
    do {
      if (it.t0 >= it.t1) continue;
      ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.q_full), seg & 1, gave_up));
      if (!ok) break;
      const int t0 = uniform(it.t0), t1 = uniform(it.t1);
#pragma unroll 1
      for (int t = t0; t < t1; ++t, ++i) {
#pragma unroll
        for (int p = 0; p < pieces; ++p) {
          const uint32_t slot = (f + p) % NP;
          ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.full[slot]), ((f + p) / NP) & 1, gave_up));
          if (!ok) break;
          fence_after();
          const uint64_t ed = moved(e_desc, slot * kPiece), qd = q_desc + (2 * p * N * 128 >> 4);
          if (elect()) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_f16(tmem, ed + (k >> 2) * (kTile * 128 >> 4) + 2 * (k & 3), qd + (k >> 2) * (N * 128 >> 4) + 2 * (k & 3), id_s,
                      p > 0 || k > 0);
          }
          __syncwarp();
        }
        if (!ok) break;
        const uint32_t slot = uniform(i % NS);
        ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.sh_full[slot]), (i / NS) & 1, gave_up));
        if (!ok) break;
        fence_after();
        const uint64_t ed = moved(s_desc, slot * kShared), qd = q_desc + (2 * pieces * N * 128 >> 4), pd = moved(p_desc, slot * kShared);
        if (elect()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f16(tmem, ed + 2 * k, qd + 2 * k, id_s, true);
          commit(smem_addr(&sm.s_full));
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.p_full), i & 1, gave_up));
        if (!ok) break;
        fence_after();
#pragma unroll
        for (int p = 0; p < pieces; ++p) {
          const uint32_t from = (f + p) % NP;
          const uint64_t cd = moved(c_desc, from * kPiece);
          const uint32_t to = tmem + C::kO + 64 * p;
          if (elect()) {
#pragma unroll
            for (int k = 0; k < 8; ++k) mma_f16(to, cd + 128 * k, pd + 128 * k, id_o, t > t0 || k > 0);
            commit(smem_addr(&sm.empty[from]));
          }
          __syncwarp();
        }
        f += pieces;
        if (elect()) {
          commit(smem_addr(&sm.sh_empty[slot]));
          if (t + 1 == t1) commit(smem_addr(&sm.o_full));
        }
        __syncwarp();
      }
      ++seg;
    } while (ok && it.next(a));
  } else if (work && warp < kLoadWarp) {
    // ---- weights and sums: a thread owns a slot of the tile and its group's rows; at an item's end a dimension
    const int group = uniform(warp >> 2), quarter = uniform(warp & 3), own = quarter * 32 + lane, bar_id = 3 + group;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + group * HN;
    const bool vec_q = ((reinterpret_cast<uintptr_t>(a.q) | (a.qst * 2) | (a.qsh * 2)) & 15) == 0;
    const bool vec_o = ((reinterpret_cast<uintptr_t>(a.out) | (a.ost * 2) | (a.osh * 2)) & 3) == 0;
    constexpr int chunks = dims / 8 + 8;
    const int used = (dims + a.rot) / 8;  // 16-byte chunks of a row of queries, of an entry
    const float scale = a.negate == 1 ? -a.scale : a.scale;
    Items<N, kCost> it(a, start, my_units);

    // The item's queries into shared memory. The products that read the last item's are over.
    auto load_queries = [&]() {
      const RowTile& r = it.r;
#pragma unroll 1
      for (int c = tid; c < N * chunks; c += C::kSoft) {
        const int row = c / chunks, d = c - row * chunks;
        const uint32_t flat = static_cast<uint32_t>(r.rt * N + row), tok = flat / static_cast<uint32_t>(a.group);
        const QT* q = static_cast<const QT*>(a.q) + (r.first + static_cast<int64_t>(tok)) * a.qst +
                      static_cast<int>(flat - tok * a.group) * a.qsh + 8 * d;
        const bool take = row < r.rows && d < used && a.negate < 2;
        uint8_t* to = q_smem + (d >> 3) * (N * 128) + row * 128 + (((d & 7) ^ (row & 7)) << 4);
        if (vec_q) {
          copy16(smem_addr(to), take ? q : static_cast<const QT*>(a.q), take);
        } else {
          uint4 u = make_uint4(0, 0, 0, 0);
          if (take) {
            QT e[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) e[x] = q[x];
            memcpy(&u, e, 16);
          }
          *reinterpret_cast<uint4*>(to) = u;
        }
      }
      copies_done();
      fence_async_shared();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&sm.q_full));
    };
    auto next_item = [&]() {  // that has a tile
      bool more;
      while ((more = it.next(a)) && it.t0 >= it.t1) {
      }
      return more;
    };
    int i = 0;
    uint32_t f = 0;  // pieces so far
    if (tid == 0) a.cut[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    bool more = it.t0 < it.t1 || next_item();
    if (more) load_queries();
    for (int seg = 0; more; ++seg) {
      const RowTile r = it.r;
      const int t0 = uniform(it.t0), t1 = uniform(it.t1), r0 = r.rt * N + group * HN;  // r0: the thread's first row
      float l[HN];
#pragma unroll
      for (int j = 0; j < HN; ++j) l[j] = 0.f;
      bool ok = true;
#pragma unroll 1
      for (int t = t0; t < t1; ++t, ++i, f += pieces) {
        ok = __all_sync(0xffffffffu, bar_wait(smem_addr(&sm.s_full), i & 1, gave_up));
        fence_after();
        uint32_t x[HN];
        ld_cols<HN>(lanes, x);
        uint32_t vis = 0xffffffffu;
        if (t >= r.part) {
          // Slots behind the rows' last hold no values, and a value that is not finite must not reach the rows that do not see
          // it through a weight of 0: both are cleared here. The scores had it: of the rows that see it, those whose score is
          // NaN or infinity are NaN, and those whose score is -infinity get a NaN in its dimension at the item's end.
          const int slot = t * kTile + own;
#pragma unroll 1
          for (int p = group; p < pieces && ok; p += C::G) {
            const uint32_t at = (f + p) % NP;
            if (!bar_wait(smem_addr(&sm.full[at]), ((f + p) / NP) & 1, gave_up)) break;
            if (slot < r.ctx) continue;  // every row sees it
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint4* row = reinterpret_cast<uint4*>(ring + at * kPiece + c * (kTile * 128) + own * 128);
              if (clean_chunks<B, 8>(row, own & 7, slot >= r.end)) sm.odd[seg & 1] = seg + 1;
            }
          }
          if (slot >= r.ctx) {
            const int j = slot - r.ctx;  // token of the step
            if (slot >= r.end) {
              vis = 0;
            } else if (!a.tree) {
              const int64_t first = static_cast<int64_t>(j) * a.group - r0;
              vis = first <= 0 ? 0xffffffffu : (first >= 32 ? 0u : 0xffffffffu << first);
            } else {
              uint32_t bits = 0;
              int token = r0 / a.group, sub = r0 - token * a.group;
              for (int q = 0; q < HN;) {  // the rows of one token see the same
                const bool on = token < r.n && sees(a, r.b, token, j);
                const int many = min(HN - q, a.group - sub);
                if (on) bits |= (0xffffffffu >> (32 - many)) << q;
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
        settle<HN>(x);
        float y[HN];  // scores over the reference
        bool pass = t == t0;
        float top = kNegInf;
#pragma unroll
        for (int j = 0; j < HN; j += 4) {
          const float4 ref = t == t0 ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(&sm.ref[group * HN + j]);
          const float2 sc = make_float2(scale, scale);
          const float2 u = fma2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), sc, make_float2(-ref.x, -ref.y));
          const float2 v = fma2(make_float2(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])), sc, make_float2(-ref.z, -ref.w));
          y[j] = u.x, y[j + 1] = u.y, y[j + 2] = v.x, y[j + 3] = v.y;
        }
        if (vis != 0xffffffffu) {
#pragma unroll
          for (int j = 0; j < HN; ++j)
            if (!((vis >> j) & 1)) y[j] = kNegInf;
        }
#pragma unroll
        for (int j = 0; j < HN; ++j) top = fmaxf(top, y[j]);
        pass |= top > kPass + B::kBelow;
        if (!named_all(bar_id, 128, ok && !pass)) {
          if (!named_all(bar_id, 128, ok)) {
            ok = false;
            break;
          }
          // the rows' largest scores: over the lanes, then over the four warps; references move, sums and results follow
#pragma unroll
          for (int j = 0; j < HN; ++j) y[j] = (vis >> j) & 1 ? __uint_as_float(x[j]) * scale : kNegInf;
          float mine = kNegInf;
#pragma unroll
          for (int j = 0; j < HN; ++j) {
            const float m = warp_max(y[j]);
            if (lane == j) mine = m;
          }
          if (lane < HN) sm.smax[group][quarter][lane] = mine;
          named_sync(bar_id, 128);
          const int col = lane < HN ? lane : 0;
          const float m = fmaxf(fmaxf(sm.smax[group][0][col], sm.smax[group][1][col]), fmaxf(sm.smax[group][2][col], sm.smax[group][3][col]));
          const float old = t == t0 ? kUnset : sm.ref[group * HN + col], now = fmaxf(old, m - B::kBelow);
          const float by = t == t0 ? 0.f : ex2_fast(old - now);
          named_sync(bar_id, 128);  // references and maxima have been read
          if (quarter == 0 && lane < HN) sm.ref[group * HN + lane] = now, sm.fac[group * HN + lane] = by;
          named_sync(bar_id, 128);
          float fac[HN];
#pragma unroll
          for (int j = 0; j < HN; j += 4) {
            const float4 n4 = *reinterpret_cast<const float4*>(&sm.ref[group * HN + j]),
                         f4 = *reinterpret_cast<const float4*>(&sm.fac[group * HN + j]);
            y[j] -= n4.x, y[j + 1] -= n4.y, y[j + 2] -= n4.z, y[j + 3] -= n4.w;
            fac[j] = f4.x, fac[j + 1] = f4.y, fac[j + 2] = f4.z, fac[j + 3] = f4.w;
            l[j] *= f4.x, l[j + 1] *= f4.y, l[j + 2] *= f4.z, l[j + 3] *= f4.w;
          }
          if (t > t0) {
#pragma unroll 1
            for (int p = 0; p < pieces; ++p) {
              uint32_t o[HN];
              ld_cols<HN>(lanes + C::kO + 64 * p, o);
              wait_ld();
              settle<HN>(o);
#pragma unroll
              for (int j = 0; j < HN; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * fac[j]);
              st_cols<HN>(lanes + C::kO + 64 * p, o);
            }
            wait_st();
          }
        }
        uint8_t* p_row = sh + (i % NS) * kShared + own * 128;
#pragma unroll
        for (int j = 0; j < HN; j += 8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            w[k] = B::pack(ex2_fast(y[j + 2 * k]), ex2_fast(y[j + 2 * k + 1]));
            const float2 s = add2(make_float2(l[j + 2 * k], l[j + 2 * k + 1]), B::unpack(w[k]));
            l[j + 2 * k] = s.x, l[j + 2 * k + 1] = s.y;
          }
          *reinterpret_cast<uint4*>(p_row + ((((group * HN + j) >> 3) ^ (own & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_async_shared();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&sm.p_full));
      }
      if (!ok) break;

      // ---- the next item's queries, then this one's results or its share of them
      const bool whole = t0 == 0 && t1 == r.tiles;
      if (tid == 0) it.cut(a, runs);
      __syncwarp();
      more = next_item();
      if (more) load_queries();
      const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (t0 > 0 ? 0 : 1);
      {
        const float s = sums_of<HN>(l, lane);
        if (lane < HN) sm.sums[group][quarter][lane] = s;
        if (quarter == 3 && lane < HN) {
          const int flat = r0 + lane, tok = flat / a.group;
          sm.to[group][lane] = group * HN + lane < r.rows
                                   ? (r.first + static_cast<int64_t>(tok)) * a.ost + (flat - tok * a.group) * a.osh : -1;
        }
      }
      ok = bar_wait(smem_addr(&sm.o_full), seg & 1, gave_up);
      if (!named_all(bar_id, 128, ok)) break;
      fence_after();
      {
        const int col = lane < HN ? lane : 0;
        const float s = (sm.sums[group][0][col] + sm.sums[group][1][col]) + (sm.sums[group][2][col] + sm.sums[group][3][col]);
        if (lane < HN) {
          sm.inv[warp][lane] = s == 0.f ? 0.f : 1.f / s;
          if (!whole && quarter == 0 && group * HN + lane < r.rows)
            a.part_ml[part * N + group * HN + lane] = make_float2(sm.ref[group * HN + lane], s);
        }
      }
      __syncwarp();
#pragma unroll 1
      for (int p = 0; p < pieces; ++p) {
        __syncwarp();
        uint32_t x[HN];
        ld_cols<HN>(lanes + C::kO + 64 * p, x);
        wait_ld();
        settle<HN>(x);
        if (!whole) {
          float* o = a.part_o + (part * N + group * HN) * dims + 128 * p + own;
#pragma unroll
          for (int j = 0; j < HN; ++j)
            if (group * HN + j < r.rows) o[j * dims] = __uint_as_float(x[j]);
          continue;
        }
#pragma unroll
        for (int j = 0; j < HN; j += 2) {  // neighbours swap: a lane stores two dimensions of every other row
          const float u = __uint_as_float(x[j]) * sm.inv[warp][j], v = __uint_as_float(x[j + 1]) * sm.inv[warp][j + 1];
          const bool odd = lane & 1;
          const float got = __shfl_xor_sync(0xffffffffu, odd ? u : v, 1);
          const int64_t to = sm.to[group][j + (odd ? 1 : 0)];
          if (to < 0) continue;
          QT* o = static_cast<QT*>(a.out) + to + 128 * p + (own & ~1);
          const float lo = odd ? got : u, hi = odd ? v : got;
          if (vec_o) *reinterpret_cast<uint32_t*>(o) = B::pack(lo, hi);
          else o[0] = from_f<QT>(lo), o[1] = from_f<QT>(hi);
        }
      }
      __syncwarp();
      if (sm.odd[seg & 1] == seg + 1) {  // set before the weights of its tile were ready: what was cleared, times a weight of 0
#pragma unroll 1
        for (int slot = max(max(t0, r.part) * kTile, r.ctx); slot < min(r.end, t1 * kTile); ++slot) {
          const int id = a.c.table[static_cast<int64_t>(r.b) * a.c.max_blocks + slot / a.c.block];
          if (id < 0 || id >= a.c.num_blocks) continue;
          const uint16_t* e = reinterpret_cast<const uint16_t*>(a.c.k + id * a.c.sb + (slot % a.c.block) * a.c.ss);
#pragma unroll 1
          for (int d = own; d < dims; d += kTile) {
            if ((e[d] & (B::kExp & 0xffffu)) != (B::kExp & 0xffffu)) continue;
#pragma unroll 1
            for (int j = 0; j < HN && group * HN + j < r.rows; ++j) {
              if (!sees(a, r.b, (r0 + j) / a.group, slot - r.ctx)) continue;
              if (whole) static_cast<QT*>(a.out)[sm.to[group][j] + d] = from_f<QT>(__int_as_float(0x7fffffff));
              else a.part_o[(part * N + group * HN + j) * dims + d] = __int_as_float(0x7fffffff);
            }
          }
        }
        __syncwarp();
      }
      fence_before();
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (sm.gave_up) {  // what is in flight writes this block's memory: the warps that began it wait for it, with a limit
    if (warp == kLoadWarp) {
#pragma unroll 1
      for (uint32_t k = fill > NP ? fill - NP : 0; k < fill; ++k)
#pragma unroll 1
        for (int n = 0; n < (1 << 16) && !bar_try(smem_addr(&sm.full[k % NP]), (k / NP) & 1); ++n) {
        }
#pragma unroll 1
      for (uint32_t k = sh_fill > NS ? sh_fill - NS : 0; k < sh_fill; ++k)
#pragma unroll 1
        for (int n = 0; n < (1 << 16) && !bar_try(smem_addr(&sm.sh_full[k % NS]), (k / NS) & 1); ++n) {
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

// ------------------------------------------------------------------ launch --

template <typename QT, int N, int P>
cudaError_t launch_pieces(const LatentAttnArgs& a, const CUtensorMap& map, cudaStream_t st) {
  using C = LCfg<N, P>;
  return launch_items<QT, N>(latent_attention_kernel<QT, C>, a, C::kThreads, C::kBudget + 1024, map, st);
}

template <typename QT, int N>
cudaError_t launch_rows(const LatentAttnArgs& a, const CUtensorMap& map, cudaStream_t st) {
  switch (a.c.D) {
    case 128: return launch_pieces<QT, N, 1>(a, map, st);
    case 256: return launch_pieces<QT, N, 2>(a, map, st);
    case 384: return launch_pieces<QT, N, 3>(a, map, st);
    default: return launch_pieces<QT, N, 4>(a, map, st);
  }
}

template <typename QT>
cudaError_t launch_type(const LatentAttnArgs& a, int rows, const CUtensorMap& map, cudaStream_t st) {
  if (rows == 16) return launch_rows<QT, 16>(a, map, st);
  if (rows == 32) return launch_rows<QT, 32>(a, map, st);
  if (rows == 48) return launch_rows<QT, 48>(a, map, st);
  return launch_rows<QT, 64>(a, map, st);
}

}  // namespace
}  // namespace specv
