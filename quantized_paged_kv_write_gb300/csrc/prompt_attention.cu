// Causal attention over packed prompts, on the fifth-generation tensor cores.
//
// What it computes: for token t of a sequence and query head h, which reads kv
// head h / G (GQA, "KV Cache Quantization" glossary), over the sequence's
// tokens j <= t:  z_j = q_t k_j / sqrt(d), out = sum softmax(z)_j v_j and
// lse = ln sum exp(z_j).  It is the attention of the prefill whose K and V the
// quantize-write stores ("Use Less Memory: Quantization and Offloading", §2.1).
//
// A unit of work is 2 x 128 rows of one kv head, row = (token, query head of the
// group), against the sequence's keys in tiles of 128: each of two softmax
// warpgroups (thread = row) has 128 rows, both use the tile's K and V.  Scores
// S = Q K^T and outputs O += P V in tensor memory, P as the second product's first
// operand there.  The tensor core alternates between the warpgroups: while one
// takes its exponentials, the other's P V and next S are computed.
//   t = S c - mu, c = log2(e) / sqrt(d); p = 2^t, l += p
// mu, the reference, is the row's maximum in log2 units; it is raised (and O and
// l follow) only when a score passes it by kRaise, so p stays below 2^kRaise.
// p is rounded to BF16, the type of V (the product's operands have one type); l
// sums the unrounded p.  Relative to 64 bits the outputs are off by 0.0018 to
// 0.0021 (2-norm; all in FP32 and rounded once: 0.0015 to 0.0016).
//
// Why this shape.  4 d operations a (row, key) for 2 bytes of K and of V that 128
// rows share: bound by the tensor core.  128 rows are what an instruction of one
// SM takes; two row tiles make one's exponentials hide behind the other's products
// (four would need twice the tensor memory with keys in tiles of 128; in tiles of 64,
// with P over S, four would fit for head dimension 64: not built).  A tile of the group's query heads
// (128 / G tokens of them) instead of one head reads K and V once for all of them.
// Units are handed out one at a time, those with the most keys first, by a counter:
// the causal triangle and mixed lengths make them uneven.
//
// Measured (one GB300, 1906 TFLOP/s for a short product, 1699 for seconds of it; a few
// calls after a rest): head dimension 128, 16384 tokens of 32 heads on 8: 1199 us =
// 1.83 PFLOP/s of the causal half, 23 prompts of up to 2049 tokens 218 us (142 at
// the product's rate), 4 prompts of up to 4097 tokens of 64 on 8 290 us (232); head
// dimension 64, 3 prompts of up to 5003 tokens of 24 on 8 105 us (49).  Calls for
// seconds meet the power limit: 1336 to 1389, 236, 314 to 322 and 104 us.  A step (128
// rows x 128 keys x 2 warpgroups) takes ~2550 cycles where the products alone take
// 2048: the rest is the hand-over between products and softmax.  A unit's first
// scores, last outputs and hand-over cost ~2500 cycles more, which short prompts feel
// (steps and unit ends make ~175 of the 23 prompts' 218 us; where the rest goes, the
// plan, look-ups, the last CTAs, has not been taken apart).
// Head dimension 64 has half the products for the same exponentials (a step's 1024
// and 1150 cycles, each alone); a step takes ~2200: its parts, in a chain for either
// warpgroup, overlap half.
//
// Measured and dropped: waits that spin without suspending (1571 for 1381 us, 16384
// tokens); one warp for both warpgroups' products (1380 for 1324); outputs stored by a
// warpgroup of its own (1235 for 1207); three places for row tiles (no change);
// exponents formed before the exponentials' turn, head dimension 64 (120 for 118);
// P handed over in halves there, so that P V overlaps the next exponentials (117.6
// without turns, 130 with them, for 118).
#include <limits.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kvq_internal.h"
#include "mbar_wait.cuh"
#include "tcgen05.cuh"

namespace kvq {
namespace {

// ---------------------------------------------------------------------------
// plan: the sequences by length, and the list of work
// ---------------------------------------------------------------------------
// A unit is (sequence, tile of `unit` tokens, kv head).  Units are listed by
// tile index from the last to the first, so that those with most keys go
// first: level j holds the tile j of every sequence that has one.
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const PromptArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ int sums[kPlanThreads / 32];
  grid_release();
  // offsets in order and in range, or nothing is computed
  bool order = true;
  for (int s = threadIdx.x; s < a.num_seqs; s += kPlanThreads) {
    const int x = __ldg(a.offsets + s), y = __ldg(a.offsets + s + 1);
    order = order && x >= 0 && y >= x && y <= a.num_tokens;
  }
  for (int j = threadIdx.x; j <= a.levels; j += kPlanThreads) a.ws_level[j] = 0;
  const bool none = __syncthreads_or(!order);
  if (none) {
    if (threadIdx.x == 0) {
      set_error(a.err, KVQ_DEVERR_GROUP_RANGE);
      a.ws_head->units = 0;
      a.ws_head->next = 0;
    }
    return;
  }
  // how many sequences have j tiles (a sequence longer than announced: none)
  auto tiles = [&](int s, int *start, int *len) {
    const int x = __ldg(a.offsets + s), y = __ldg(a.offsets + s + 1);
    *start = x;
    *len = y - x;
    return *len > a.max_seq ? 0 : (*len + a.unit - 1) / a.unit;
  };
  int start, len;
  for (int s = threadIdx.x; s < a.num_seqs; s += kPlanThreads) {
    atomicAdd(a.ws_level + tiles(s, &start, &len), 1);
    if (len > a.max_seq) set_error(a.err, KVQ_DEVERR_CONTEXT_RANGE);
  }
  __syncthreads();
  // from the top: sequences with more than j tiles (where those with j go), and
  // units before level j
  int more = 0, units = 0;
  for (int base = a.levels; base >= 0; base -= kPlanThreads) {
    const int j = base - static_cast<int>(threadIdx.x);
    const int own = j >= 0 ? a.ws_level[j] : 0;
    auto scan = [&](int v, int *total) {  // inclusive, over the CTA
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      if (lane == 31) sums[warp] = v;
      __syncthreads();
      const int w = sums[lane];
      v += __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
      *total = __reduce_add_sync(0xffffffffu, w);
      __syncthreads();
      return v;
    };
    int all;
    int above = more + scan(own, &all) - own;  // sequences with more than j tiles: those that have a tile j
    if (j < 0) above = 0;
    more += all;
    const int before = units + scan(above, &all) - above;
    units += all;
    if (j >= 0) {
      a.ws_level[j] = before * a.H;
      a.ws_place[j] = above;
    }
  }
  if (threadIdx.x == 0) {
    a.ws_head->units = units * a.H;
    a.ws_head->next = 0;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < a.num_seqs; s += kPlanThreads) {
    const int t = tiles(s, &start, &len);
    if (t > 0) a.ws_seq[atomicAdd(a.ws_place + t, 1)] = make_int2(start, len);
  }
}

// Unit x of the list.
struct Unit {
  int start, len, t0, h;
};
__device__ __forceinline__ Unit unit_at(const PromptArgs &a, int x) {
  int lo = 0, hi = a.levels - 1;  // the lowest level whose units begin at or before x
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.ws_level[mid] <= x) hi = mid; else lo = mid + 1;
  }
  const int i = x - a.ws_level[lo], s = i / a.H;
  const int2 q = a.ws_seq[s];
  return {q.x, q.y, lo * a.unit, i - s * a.H};
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
constexpr int kTile = 128;                     // keys of a tile, rows of a row tile
constexpr int kLoadWarp = 0, kMmaWarp = 1, kPlanWarp = 3, kSoftmaxWarp = 4;  // (two warps for the products)
constexpr int kThreads = 12 * 32;
// Registers a thread: 168 at launch; the four single-warp roles give theirs to
// the softmax (128 * 88 + 256 * 208 = 384 * 168).
constexpr int kFewRegs = 88, kManyRegs = 208;
constexpr float kRaise = 6.f;
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D>
struct Smem {
  static constexpr uint32_t HALF = 128 * 128;           // 64 channels of 128 rows
  static constexpr uint32_t TILE = HALF * (D / 64);
  static constexpr int STAGES = D == 128 ? 2 : 4;       // places for tiles of K, and of V
  static constexpr int QS = 2;                          // and for row tiles
  static constexpr uint32_t q = 0;
  static constexpr uint32_t k = q + QS * TILE;
  static constexpr uint32_t v = k + STAGES * TILE;
  static constexpr uint32_t out = v + STAGES * TILE;    // [2] 64 channels of a warpgroup's outputs
  static constexpr uint32_t bars = out + 2 * HALF;
  static constexpr uint32_t tmem = bars + 64 * 8;       // tensor memory address, then the abort flag
  static constexpr uint32_t units = tmem + 16;          // [2] {start, len, t0, h}; start -1: the end
  static constexpr uint32_t bytes = units + 32;
  static_assert(bytes <= 227 * 1024, "shared memory");
};

// Tensor memory: two S, two O; P over S where they fill it, else beside them.
template <int D>
struct Tmem {
  static constexpr bool BESIDE = D == 64;
  static constexpr uint32_t s = 0, p = BESIDE ? 256 : 0, p_step = BESIDE ? 64 : 128, o = BESIDE ? 384 : 256;
};

enum Bar : int {
  B_Q = 0, B_QFREE = 3, B_S = 6, B_TAKEN = 8, B_P = 10, B_PFREE = 12, B_O = 14, B_OFREE = 16, B_UNIT = 18, B_UNITFREE = 20,
  B_KFULL = 22, B_KFREE = 26, B_VFULL = 30, B_VFREE = 34, B_END = 38, B_TURN = 40, B_EXP = 42,
  B_COUNT = 44
};

// What the roles need to know of a unit: tokens t0 .. and the tiles of keys of
// each row tile (the first `step` tokens, and the next).
struct Work {
  int start, len, t0, h;
  int tiles[2], all;
  __device__ __forceinline__ Work(uint4 u, int step) {
    start = static_cast<int>(u.x);
    len = static_cast<int>(u.y);
    t0 = static_cast<int>(u.z);
    h = static_cast<int>(u.w);
    tiles[0] = (min(len, t0 + step) + kTile - 1) / kTile;
    tiles[1] = t0 + step < len ? (min(len, t0 + 2 * step) + kTile - 1) / kTile : 0;
    all = max(tiles[0], tiles[1]);
  }
};

// The units one after the other, as the plan warp hands them out.
struct Units {
  const InlineWaiter &wait;
  uint32_t at;
  int n = 0;
  __device__ __forceinline__ Units(const InlineWaiter &w, uint32_t units) : wait(w), at(units) {}
  __device__ __forceinline__ uint4 next() {
    wait(B_UNIT + (n & 1), (n >> 1) & 1);
    return lds128(at + 16 * (n & 1));
  }
  // (one lane of each warp that has read it)
  __device__ __forceinline__ void done(int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&wait.bars[B_UNITFREE + (n & 1)]);
    ++n;
  }
};

// When a CTA takes its next unit.  Taken two ahead, the look-up is never waited for;
// but where a CTA gets few units, those with the most keys first, some then have more
// to do than others: there it is taken when the one before has kAhead tiles left to be
// loaded (units of up to kShort tiles do not hide the look-up).  3 prompts of up to
// 5003 tokens, head dimension 64, 5 units a CTA: 119 us two ahead, 108 late; 3 of 8000 of
// 8 heads on 1, 5 a CTA: 140 and 102; 4 of up to 4097 of 64 on 8, 16 a CTA: 315 and 321;
// the 23 of up to 2049, 19 a CTA: 216.5 and 219.5.
constexpr int kAhead = 8, kShort = 2, kFewUnits = 12;
__device__ __forceinline__ bool few_units(const PromptArgs &a) {
  return a.ws_head->units <= kFewUnits * static_cast<int>(gridDim.x);
}

__device__ __forceinline__ void plan_role(const PromptArgs &a, uint32_t units, const InlineWaiter &wait, int lane) {
  const int total = a.ws_head->units;
  const bool few = few_units(a);
  int back = 2;
  for (int n = 0;; ++n) {
    // the unit before last has been read, or (few) the last one nears its end
    if (n >= back) wait(B_UNITFREE + ((n - back) & 1), ((n - back) >> 1) & 1);
    int x = 0;
    if (lane == 0) x = atomicAdd(&a.ws_head->next, 1);
    x = __shfl_sync(0xffffffffu, x, 0);
    const bool end = x >= total;
    Unit u = {-1, 0, 0, 0};
    if (!end) u = unit_at(a, x);
    if (lane == 0) {
      sts128(units + 16 * (n & 1), u.start, u.len, u.t0, u.h);
      mbar_arrive(&wait.bars[B_UNIT + (n & 1)]);
    }
    if (end) return;
    back = few && min(u.len, u.t0 + a.unit) > kShort * kTile ? 1 : 2;
  }
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

template <int D>
__device__ __forceinline__ void load_role(const PromptArgs &a, const CUtensorMap *qm, const CUtensorMap *km,
                                          const CUtensorMap *vm, uint32_t base, const InlineWaiter &wait, int lane) {
  using L = Smem<D>;
  const int step = a.unit / 2;
  const uint32_t qbytes = step * a.G * D * 2;
  const int ahead = few_units(a) ? kAhead : INT_MAX;
  Units units(wait, base + L::units);
  int st = 0, qs = 0;             // places for K and V, and for row tiles
  uint32_t ph = 1, qp = 1;        // and their parities
  for (;;) {
    const uint4 u = units.next();
    if (static_cast<int>(u.x) < 0) break;
    const Work w(u, step);
    const int hand_back = max(0, w.all - ahead);
    const bool go = lane == 0 && !*wait.abort;  // (after a wait that ran out nobody reads: no further copies)
    for (int j = 0; j < w.all; ++j) {
      if (j == hand_back) units.done(lane);
      wait(B_KFREE + st, ph);
      if (go) {
        mbar_arrive_expect_tx(&wait.bars[B_KFULL + st], L::TILE);
#pragma unroll
        for (int c = 0; c < D; c += 64)
          tma_load(base + L::k + st * L::TILE + c / 64 * L::HALF, km, c, w.h, w.start + j * kTile, &wait.bars[B_KFULL + st]);
      }
      if (j == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (w.tiles[i] == 0) continue;
          wait(B_QFREE + qs, qp);
          if (go) {
            mbar_arrive_expect_tx(&wait.bars[B_Q + qs], qbytes);
#pragma unroll
            for (int c = 0; c < D; c += 64)
              tma_load(base + L::q + qs * L::TILE + c / 64 * L::HALF, qm, c, w.h * a.G, w.start + w.t0 + i * step,
                       &wait.bars[B_Q + qs]);
          }
          if (++qs == L::QS) {
            qs = 0;
            qp ^= 1;
          }
        }
      }
      wait(B_VFREE + st, ph);
      if (go) {
        mbar_arrive_expect_tx(&wait.bars[B_VFULL + st], L::TILE);
#pragma unroll
        for (int c = 0; c < D; c += 64)
          tma_load(base + L::v + st * L::TILE + c / 64 * L::HALF, vm, c, w.h, w.start + j * kTile, &wait.bars[B_VFULL + st]);
      }
      if (++st == L::STAGES) {
        st = 0;
        ph ^= 1;
      }
    }
  }
  // no copy in flight when the CTA exits: all places are read, or (a wait ran
  // out) a millisecond goes by
  if (*wait.abort) {
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000) {
    }
  }
  for (int i = 0; i < L::STAGES; ++i) {
    wait(B_KFREE + st, ph);
    wait(B_VFREE + st, ph);
    if (++st == L::STAGES) {
      st = 0;
      ph ^= 1;
    }
  }
  for (int i = 0; i < L::QS; ++i) {
    wait(B_QFREE + qs, qp);
    if (++qs == L::QS) {
      qs = 0;
      qp ^= 1;
    }
  }
}

// The products of warpgroup i, a warp for each.  The whole warp walks the steps
// and one elected lane issues, so that what the products take stays in uniform
// registers.  Issuing takes as long as the products themselves, and the waits
// between them several hundred cycles: with one warp for both warpgroups that time
// was lost to the tensor core (16384 tokens: 1380 us; two warps 1324, with all waits
// before the turn 1228).  The tiles of all units are one sequence: the next S follows
// P V, or (P beside S) goes ahead of it, also from one unit to the next, whose first S
// is there when the outputs of the one before are stored.
template <int D>
__device__ __forceinline__ void product_role(const PromptArgs &a, uint32_t base, const InlineWaiter &wait, uint32_t tmem_addr,
                                             const int i, int lane) {
  using L = Smem<D>;
  using M = Tmem<D>;
  constexpr uint32_t id_s = mma_idesc_bf16(128, kTile, false), id_o = mma_idesc_bf16(128, D, true);
  const bool leader = elect_one();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_addr, 0);
  const uint32_t S = tmem + M::s + 128 * i, P = tmem + M::p + M::p_step * i, O = tmem + M::o + D * i;
  const uint64_t dq = mma_desc(base + L::q, 16, 1024), dk = mma_desc(base + L::k, 16, 1024),
                 dv = mma_desc(base + L::v, L::HALF, 1024);
  const int step = a.unit / 2;
  Units units(wait, base + L::units);
  int st = 0, qs = 0;                 // place of the tile of K and V, and of the next row tile,
  uint32_t ph = 0, qp = 0;            // and their parities
  uint32_t ns = 0, np = 0, no = 0;    // steps, P and units so far
  // P V to be issued when P is there
  bool any = false, first = false, last = false;
  int v_st = 0, rows = 0;
  uint32_t v_ph = 0, turns = 0;
  // what it waits for
  auto output_ready = [&]() {
    wait(B_VFULL + v_st, v_ph);
    if (rows < kTile) {
      // what lies behind the sequence may be anything, and 0 times it is not 0
      // (each of the two warps does it: the other one's products read zeros)
      const uint32_t to = base + L::v + v_st * L::TILE;
      for (int x = rows * 8 + lane; x < kTile * 8; x += 32)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) sts128(to + c * L::HALF + 16 * x, 0u, 0u, 0u, 0u);
      fence_proxy_async_shared();
    }
    if (first) wait(B_OFREE + i, (no++ & 1) ^ 1);
    wait(B_P + i, np++ & 1);
  };
  auto issue_output = [&]() {  // (the leader)
    const uint64_t v = dv + v_st * (L::TILE / 16);
#pragma unroll
    for (int e = 0; e < kTile / 16; ++e) mma_f16_ts(O, P + 8 * e, v + e * (2048 / 16), id_o, !first || e > 0);
    mma_commit(&wait.bars[B_VFREE + v_st]);
    if constexpr (M::BESIDE) mma_commit(&wait.bars[B_PFREE + i]);
    if (last) mma_commit(&wait.bars[B_O + i]);
  };
  // P over S: the two warps issue in turns (left alone they fall into step, and the
  // tensor core waits while both warpgroups take exponentials)
  auto take_turn = [&]() {
    if constexpr (!M::BESIDE) wait(B_TURN + i, (turns++ & 1) ^ (i == 0 ? 1 : 0));
  };
  auto pass_turn = [&]() {  // (the leader)
    if constexpr (!M::BESIDE) mbar_arrive(&wait.bars[B_TURN + (i ^ 1)]);
  };
  for (;;) {
    const uint4 u = units.next();
    if (static_cast<int>(u.x) < 0) break;
    const Work w(u, step);
    units.done(lane);
    // the row tiles' places: the first warpgroup's, then the second's
    int place[2];
    uint32_t parity[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      place[k] = qs;
      parity[k] = qp;
      if (w.tiles[k] > 0 && ++qs == L::QS) {
        qs = 0;
        qp ^= 1;
      }
    }
    const int tiles = i ? w.tiles[1] : w.tiles[0], q = i ? place[1] : place[0];
    const uint32_t q_ph = i ? parity[1] : parity[0];
#pragma unroll 1
    for (int j = 0; j < w.all; ++j) {
      const bool mine = j < tiles;  // (else a tile of the other warpgroup alone)
      wait(B_KFULL + st, ph);
      if (mine && j == 0) wait(B_Q + q, q_ph);
      if constexpr (M::BESIDE) {
        if (mine) wait(B_TAKEN + i, (ns++ & 1) ^ 1);
      } else {
        if (any) output_ready();
        take_turn();
      }
      if (!mine) wait(B_VFULL + st, ph);
      __syncwarp();
      tmem_fence_after();
      if (leader) {
        if constexpr (!M::BESIDE)
          if (any) issue_output();
        if (mine) {
          const uint64_t x = dq + q * (L::TILE / 16), k = dk + st * (L::TILE / 16);
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            const uint32_t off = ((e / 4) * L::HALF + (e % 4) * 32) / 16;
            mma_f16_ss(S, x + off, k + off, id_s, e > 0);
          }
          mma_commit(&wait.bars[B_S + i]);
          mma_commit(&wait.bars[B_KFREE + st]);
          if (j + 1 == tiles) mma_commit(&wait.bars[B_QFREE + q]);
        } else {
          mbar_arrive(&wait.bars[B_KFREE + st]);
          mbar_arrive(&wait.bars[B_VFREE + st]);
        }
        pass_turn();
      }
      __syncwarp();
      if constexpr (M::BESIDE) {
        if (any) {
          output_ready();
          __syncwarp();
          tmem_fence_after();
          if (leader) issue_output();
          __syncwarp();
        }
      }
      any = mine;
      first = j == 0;
      last = j + 1 == tiles;
      rows = w.len - j * kTile;
      v_st = st;
      v_ph = ph;
      if (++st == L::STAGES) {
        st = 0;
        ph ^= 1;
      }
    }
  }
  if (any) output_ready();
  take_turn();
  __syncwarp();
  tmem_fence_after();
  if (leader) {
    if (any) issue_output();
    pass_turn();
  }
  __syncwarp();
  // nothing in flight when tensor memory is given back
  if (leader) mma_commit(&wait.bars[B_END + i]);
  __syncwarp();
  wait(B_END + i, 0);
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// 32 bytes of global memory, 32-byte aligned.
__device__ __forceinline__ void store_32(void *to, const uint32_t *r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void tma_store(uint32_t from, const CUtensorMap *map, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(from)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

template <int D>
__device__ __forceinline__ void softmax_role(const PromptArgs &a, const CUtensorMap *om, uint32_t base, const InlineWaiter &wait,
                                             uint32_t tmem) {
  using L = Smem<D>;
  const int wg = (threadIdx.x >> 7) - kSoftmaxWarp / 4, warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
  using M = Tmem<D>;
  const uint32_t S = tmem + lanes + M::s + 128 * wg, P = tmem + lanes + M::p + M::p_step * wg, O = tmem + lanes + M::o + D * wg;
  const int step = a.unit / 2, r = 32 * warp + lane, rt = r / a.G, g = r - rt * a.G;
  const int near = 32 * warp / a.G;  // the warp's first token
  const float c = rsqrtf(static_cast<float>(D)) * kLog2E;
  Units units(wait, base + L::units);
  uint32_t ns = 0, no = 0;  // steps and units of this warpgroup so far
  const bool sender = (threadIdx.x & 127) == 0;  // of the warpgroup's outputs
  // P beside S: the warpgroups take their exponentials in turns, the second half of
  // one's with the first of the other's (left alone both fall into step and the
  // products wait meanwhile: 128 us for 118; a turn that ends with the last
  // exponential 119).  P over S: the products' turns keep them apart.
  uint32_t turns = 0;
  auto take_turn = [&]() {
    wait(B_EXP + wg, (turns++ & 1) ^ (wg == 0 ? 1 : 0));
    __syncwarp();
  };
  auto pass_turn = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&wait.bars[B_EXP + (wg ^ 1)]);
  };
  auto pass_turns = [&](int n) {
    for (int j = 0; M::BESIDE && j < n; ++j) {
      take_turn();
      pass_turn();
    }
  };
  auto meet = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); };
  uint4 u = units.next();
  while (static_cast<int>(u.x) >= 0) {
    const Work w(u, step);
    units.done(lane);
    const int tiles = wg ? w.tiles[1] : w.tiles[0], t = w.t0 + wg * step + rt;
    if (tiles == 0) {
      pass_turns(w.all);
      u = units.next();
      continue;
    }
    const bool live = rt < step && t < w.len;
    const int limit = live ? t + 1 : INT_MAX, nearest = w.t0 + wg * step + near + 1;
    float mu = -INFINITY, l = 0.f;
#pragma unroll 1
    for (int j = 0; j < tiles; ++j) {
      wait(B_S + wg, ns & 1);
      __syncwarp();
      tmem_fence_after();
      uint32_t w0[32], w1[32], w2[32], w3[32];
      float x0, x1, x2, x3;  // the row's largest
      tmem_ld32_max(S, w0, x0);
      tmem_ld32_max(S + 32, w1, x1);
      tmem_ld32_max(S + 64, w2, x2);
      tmem_ld32_max(S + 96, w3, x3);
      tmem_wait_ld(w0, x0);
      tmem_wait_ld(w1, x1);
      tmem_wait_ld(w2, x2);
      tmem_wait_ld(w3, x3);
      if constexpr (M::BESIDE) {
        // in registers: the next S may be written.  The P before it is free, and O
        // is complete, once its product is.
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&wait.bars[B_TAKEN + wg]);
        wait(B_PFREE + wg, (ns & 1) ^ 1);
        __syncwarp();
        tmem_fence_after();
      }
      ++ns;
      if (nearest < (j + 1) * kTile) {  // some row of the warp does not see the whole tile
        const int seen = limit - j * kTile;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          if (e >= seen) w0[e] = 0xFF800000u;
          if (32 + e >= seen) w1[e] = 0xFF800000u;
          if (64 + e >= seen) w2[e] = 0xFF800000u;
          if (96 + e >= seen) w3[e] = 0xFF800000u;
        }
        x0 = x1 = x2 = x3 = -INFINITY;
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          x0 = max3(x0, __uint_as_float(w0[e]), __uint_as_float(w0[e + 1]));
          x1 = max3(x1, __uint_as_float(w1[e]), __uint_as_float(w1[e + 1]));
          x2 = max3(x2, __uint_as_float(w2[e]), __uint_as_float(w2[e + 1]));
          x3 = max3(x3, __uint_as_float(w3[e]), __uint_as_float(w3[e + 1]));
        }
      }
      const float top = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)) * c;
      // (each row for itself: what other rows of the warp hold changes nothing)
      const bool raise = top > mu + kRaise || (mu == -INFINITY && top > mu);
      if (__any_sync(0xffffffffu, raise)) {
        const float keep = raise ? mu == -INFINITY ? 0.f : fast_exp2(mu - top) : 1.f;
        if (raise) mu = top;
        l *= keep;
        if (j > 0) {
#pragma unroll 1
          for (int cc = 0; cc < D / 16; ++cc) {
            uint32_t o[16];
            tmem_ld16(O + 16 * cc, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
            tmem_st16(O + 16 * cc, o);
          }
        }
      }
      const float neg = mu == -INFINITY ? 0.f : -mu;
      float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
      auto exponentials = [&](uint32_t(&x)[32], uint32_t to) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float a0, a1, a2, a3;
          fma_f32x2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]), c, c, neg, neg, a0, a1);
          fma_f32x2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]), c, c, neg, neg, a2, a3);
          a0 = fast_exp2(a0);
          a1 = fast_exp2(a1);
          a2 = fast_exp2(a2);
          a3 = fast_exp2(a3);
          add_f32x2(s0, s1, a0, a1, s0, s1);
          add_f32x2(s2, s3, a2, a3, s2, s3);
          p[e / 2] = f32x2_to_bf16x2(a0, a1);
          p[e / 2 + 1] = f32x2_to_bf16x2(a2, a3);
        }
        tmem_st16(to, p);
      };
      if constexpr (M::BESIDE) take_turn();
      exponentials(w0, P);
      exponentials(w1, P + 16);
      if constexpr (M::BESIDE) pass_turn();
      exponentials(w2, P + 32);
      exponentials(w3, P + 48);
      l += (s0 + s1) + (s2 + s3);
      tmem_wait_st();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&wait.bars[B_P + wg]);
    }
    pass_turns(w.all - tiles);
    // ---- the rows' outputs, 64 channels at a time through shared memory and the copy
    // unit (stores of a lane for each row kept the warpgroup 1500 cycles longer from
    // its next unit); the last rows of a sequence, which are fewer, one by one
    u = units.next();
    wait(B_O + wg, no & 1);
    ++no;
    __syncwarp();
    tmem_fence_after();
    const float inv = 1.f / l;
    const bool run_out = *wait.abort;  // (then the unit may be none)
    const bool whole = w.t0 + (wg + 1) * step <= w.len, store = live && !run_out;
    const int64_t row = static_cast<int64_t>(w.start + t) * a.Hq + w.h * a.G + g;
#pragma unroll
    for (int cc = 0; cc < D / 64; ++cc) {
      uint32_t o[32], x[32];
      tmem_ld32(O + 64 * cc, o);
      tmem_wait_ld(o);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        x[e] = f32x2_to_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
      tmem_ld32(O + 64 * cc + 32, o);
      tmem_wait_ld(o);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        x[16 + e] = f32x2_to_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
      if (cc + 1 == D / 64) {  // O is in registers
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&wait.bars[B_OFREE + wg]);
      }
      if (whole) {
        // (the copy before has read its place)
        if (sender) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        meet();
        const uint32_t to = base + L::out + wg * L::HALF;
#pragma unroll
        for (int e = 0; e < 8; ++e) sts128(to + 128 * r + 16 * (e ^ (r & 7)), x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        fence_proxy_async_shared();
        meet();
        if (sender && !run_out) tma_store(to, om, 64 * cc, w.h * a.G, w.start + w.t0 + wg * step);
      } else if (store) {
#pragma unroll
        for (int e = 0; e < 4; ++e) store_32(a.out + row * D + 64 * cc + 16 * e, x + 8 * e);
      }
    }
    if (store && a.lse != nullptr) a.lse[row] = (mu + log2f(l)) * kLn2;
  }
  if (sender) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attend_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap omap,
                         const __grid_constant__ PromptArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using L = Smem<D>;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::bars);
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t *const tm = reinterpret_cast<uint32_t *>(smem + L::tmem);
  if (warp == kLoadWarp) {
    // arrivals per phase: 4 for a warpgroup's warps, 2 for the products' warps, 11
    // for all that read a unit, else 1
    for (int i = lane; i < B_COUNT; i += 32) {
      const bool four = (i >= B_TAKEN && i < B_TAKEN + 2) || (i >= B_P && i < B_P + 2) || (i >= B_OFREE && i < B_OFREE + 2) ||
                        (i >= B_EXP && i < B_EXP + 2);
      const bool two = (i >= B_KFREE && i < B_KFREE + 4) || (i >= B_VFREE && i < B_VFREE + 4);
      mbar_init(&bars[i], four ? 4 : two ? 2 : i >= B_UNITFREE && i < B_UNITFREE + 2 ? 11 : 1);
    }
    mbar_init_fence();
    if (lane == 0) {
      prefetch_tensormap(&qmap);
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&vmap);
      prefetch_tensormap(&omap);
      *reinterpret_cast<volatile uint32_t *>(tm + 1) = 0;
      for (int i = 0; i < 2; ++i) sts128(base + L::units + 16 * i, 0xFFFFFFFFu, 0u, 0u, 0u);
    }
  }
  __syncwarp();
  if (warp == kMmaWarp) tmem_alloc(smem_u32(tm), 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tm);
  grid_wait();  // the plan
  const InlineWaiter wait = {bars, tm + 1, a.err};
  if (warp >= kSoftmaxWarp) {
    more_registers<kManyRegs>();
    softmax_role<D>(a, &omap, base, wait, tmem);
  } else {
    fewer_registers<kFewRegs>();
    if (warp == kLoadWarp) load_role<D>(a, &qmap, &kmap, &vmap, base, wait, lane);
    else if (warp < kPlanWarp) product_role<D>(a, base, wait, tmem, warp - kMmaWarp, lane);
    else plan_role(a, base + L::units, wait, lane);
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tmem_fence_after();
    tmem_free(tmem, 512);
  }
}

}  // namespace

template <int D>
static cudaError_t attend(const PromptArgs &a, const PromptMaps &m, int sms, cudaStream_t stream) {
  auto kern = prompt_attend_kernel<D>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  static std::atomic<unsigned long long> done{0};  // devices whose limit is raised
  if (!((done.load(std::memory_order_acquire) >> dev) & 1ull)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::bytes)) != cudaSuccess)
      return e;
    done.fetch_or(1ull << dev, std::memory_order_acq_rel);
  }
  return launch_overlapped(kern, sms, kThreads, Smem<D>::bytes, stream, m.q, m.k, m.v, m.out, a);
}

cudaError_t launch_prompt_attention(int head_dim, const PromptArgs &a, const PromptMaps &m, int sms, cudaStream_t stream) {
  prompt_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return head_dim == 128 ? attend<128>(a, m, sms, stream) : attend<64>(a, m, sms, stream);
}

}  // namespace kvq
