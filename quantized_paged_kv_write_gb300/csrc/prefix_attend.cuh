// Prefix attention of a group on the fifth-generation tensor cores (sm_103a):
// the kernel behind kvq_prefix_decode's shared part.
//
// Mathematics.  For the rows of a unit (256 or 128 (sequence, query head)
// pairs of one kv head) and a tile of 128 shared positions:
//   S = Q' K'^T          f16 operands, FP32 accumulators in tensor memory
//   t = S ks, z = t c    ks the position's factor, c the row's (z in log2 units)
//   p = 2^(z - m), l += p, O += (p vs) V'
// Q' = q 2^er in f16 (the row's largest in [2^14, 2^15): a BF16 q is exact
// down to 2^-32 of it).  K' is the codes (exact), ks their scale per token; or,
// with scales per channel, code * s 2^eb rounded once (the tile's largest
// s 2^eb in [2^7, 2^8)), ks = 2^-eb.  V' is the codes (exact) and vs = s_v 2^F;
// or, with scales per 32 channels, code * s 2^F rounded once and vs = 1.  F
// only falls: the largest s 2^F of a tile stays below 2^9, and p <= 2^6 (the
// reference m is raised only when a score passes m + 6), so p vs fits f16; a
// new m or F rescales O in tensor memory.  p vs is rounded to f16 once; l sums
// the unrounded p.
//
// Roles, one CTA per SM: two softmax warpgroups (thread = row), two
// warpgroups that turn codes into f16 tiles in shared memory (one K, one V),
// and a warp each for the products, the TMA loads of codes and the scales.
// Steps alternate between the two softmax warpgroups, so
// the tensor core works for one while the other is in its exponentials:
//   more than 128 rows: warpgroup i owns rows 128 i .. + 127, each tile of
//     codes serves both (steps 2t, 2t + 1 of tile t);
//   at most 128 rows: both own the same rows, warpgroup i the tiles of parity
//     i; each keeps its own (m, l, O), merged later like any other partial.
// P overwrites S in tensor memory and is the A operand of the second product.
#pragma once

#include <limits.h>

#include "paged_decode_impl.cuh"
#include "tcgen05.cuh"

namespace kvq {
namespace prefix {

constexpr int kTile = kPrefixTile;             // positions per tile
constexpr int kTileBlocks = kTile / kBlockSize;
// Warps by role: the single-warp roles, which everybody waits for, come first.
constexpr int kMmaWarp = 0, kLoadWarp = 1, kScaleWarp = 2, kKWarp = 4, kVWarp = 8, kSoftmaxWarp = 12;
constexpr int kThreads = 20 * 32;
constexpr uint32_t kUnit = 4096;               // unit of the rings of codes: a part of a tile
constexpr int kMaxUnits = 8;                   // per ring
constexpr uint32_t kMaxSmem = 227 * 1024;
constexpr int kMeta = 4;                       // ring of per-tile factors
constexpr float kRaise = 6.f;                  // m is raised past m + 6
constexpr int kTopV = 9;                       // s 2^F < 2^9

// Bits per code and the conversion.
enum Code : int { C_INT8, C_FP8, C_INT4, C_INT2 };
template <int KF>
struct KCode {
  static constexpr Code code = KF == K_FP8_TOK ? C_FP8 : KF == K_INT4_TOK ? C_INT4 : KF == K_INT2_CHAN ? C_INT2 : C_INT8;
  static constexpr bool chan = KF == K_INT8_CHAN || KF == K_INT2_CHAN;
};
template <int VF>
struct VCode {
  static constexpr Code code = VF == V_FP8_TOK ? C_FP8 : VF == V_INT4_G32 ? C_INT4 : VF == V_INT2_G32 ? C_INT2 : C_INT8;
  static constexpr bool group = VF == V_INT4_G32 || VF == V_INT2_G32;
};
constexpr int code_bits(Code c) { return c == C_INT4 ? 4 : c == C_INT2 ? 2 : 8; }

// Shared memory: f16 tiles ([64-channel half][row][128 bytes], swizzled), then
// the small arrays, then the ring of codes, as long as there is room.
template <int D>
struct Smem {
  static constexpr uint32_t HALF = 128 * 128;           // 64 channels of 128 rows
  static constexpr uint32_t TILE = HALF * (D / 64);
  static constexpr uint32_t CHAN = kTileBlocks * D * 2; // one part of the channel scales
  static constexpr uint32_t GRP = kTile * (D / 32) * 4; // group scales, f16 pairs (high, low)
  static constexpr uint32_t k = 0;                      // [2] stages
  static constexpr uint32_t v = k + 2 * TILE;           // [2] stages
  static constexpr uint32_t q = v + 2 * TILE;           // [1 or 2] row tiles
  // offsets from the end of q
  static constexpr uint32_t ks = 0;                     // [kMeta][128] FP32
  static constexpr uint32_t vs = ks + kMeta * kTile * 4;
  static constexpr uint32_t info = vs + kMeta * kTile * 4;         // [kMeta] {F, block mask}
  static constexpr uint32_t bars = info + kMeta * 8;    // mbarriers
  static constexpr uint32_t tmem = bars + 56 * 8;       // tensor memory address, then the abort flag
  static constexpr uint32_t factors = tmem + 16;        // [128] row factors
  static constexpr uint32_t scales = factors + 512;     // [2] channel scales (high, low parts) and group scales
  static_assert(scales % 16 == 0 && scales <= 5 * 1024 + 512, "small arrays");
};

// What depends on the formats and on whether any unit has two row tiles.
struct Layout {
  uint32_t small, grp;        // offsets: small arrays, group scales (from `scales`)
  uint32_t ring[2];           // the rings of K and V codes
  int units[2];
  uint32_t bytes;
};
template <int D>
inline Layout layout_of(bool chan, bool group, bool two, int krow, int vrow) {
  using L = Smem<D>;
  Layout y;
  y.small = L::q + (two ? 2 : 1) * L::TILE;
  y.grp = chan ? 4 * L::CHAN : 0;
  y.ring[0] = (y.small + L::scales + y.grp + (group ? 2 * L::GRP : 0) + 1023) & ~1023u;
  // as many units as there is room for, shared out by the bytes of a row
  const int room = static_cast<int>((kMaxSmem - y.ring[0]) / kUnit);
  int k = (room * krow + (krow + vrow) / 2) / (krow + vrow);
  if (k < 1) k = 1;
  if (k > room - 1) k = room - 1;
  y.units[0] = k < kMaxUnits ? k : kMaxUnits;
  y.units[1] = room - k < kMaxUnits ? room - k : kMaxUnits;
  y.ring[1] = y.ring[0] + y.units[0] * kUnit;
  y.bytes = y.ring[1] + y.units[1] * kUnit;
  return y;
}

enum Bar : int {
  B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_S = 8, B_P = 10, B_O = 12, B_Q = 14, B_END = 15, B_META = 16,
  B_FULL = 18 /* [2][kMaxUnits] */, B_EMPTY = B_FULL + 2 * kMaxUnits, B_COUNT = B_EMPTY + 2 * kMaxUnits
};
static_assert(B_COUNT <= 56, "mbarriers");

// The part of a unit that this CTA works on.  Tiles count in 32 bits: with
// batch * max_blocks_per_seq < 2^31 and two sequences or more in a group there
// are fewer than 2^31 of them.  Out of line, like all that runs once a segment:
// the roles of an SM's warps share its instruction caches, and the code of the
// steps has to stay there.
struct Segment {
  PrefixGroup g;
  int u, h, rb, t0, t1;
  bool two;          // two row tiles
};

__device__ __noinline__ void segment_at(const PrefixArgs &a, int x, int x1, Segment *out) {
  int lo = 0, hi = a.groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.ws_groups[mid].tile0 <= x) lo = mid; else hi = mid;
  }
  Segment s;
  s.g = a.ws_groups[lo];
  const int y = x - static_cast<int>(s.g.tile0);
  s.u = y / s.g.tiles;
  s.t0 = y - s.u * s.g.tiles;
  s.t1 = min(s.g.tiles, s.t0 + (x1 - x));
  s.h = s.u % a.H;
  s.rb = s.u / a.H;
  s.two = s.g.rows > kPrefixRows / 2;
  *out = s;
}

// Waits for a phase of an mbarrier.  When a wait runs out, the error is set and
// every later wait of the CTA returns at once: the roles run to their ends (all
// barriers between threads are met, all accesses stay in bounds), and the
// results are void.
// try_wait gets a time for which the hardware may suspend the warp: without it
// the waiting warps' polling takes a large part of the issue slots.
__device__ __forceinline__ bool mbar_suspend_wait(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __noinline__ void mbar_slow_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *abort, unsigned int *err) {
  const long long t0 = clock64();
  while (!mbar_suspend_wait(bar, parity)) {
    if (*abort) return;
    if (clock64() - t0 > kWaitTicks) {
      *abort = 1;
      set_error(err, KVQ_DEVERR_TIMEOUT);
      return;
    }
  }
}

struct Waiter {
  uint64_t *bars;
  volatile uint32_t *abort;
  unsigned int *err;
  __device__ __forceinline__ void operator()(int bar, uint32_t parity) const {
    if (!mbar_suspend_wait(&bars[bar], parity)) mbar_slow_wait(&bars[bar], parity, abort, err);
  }
};

// ---------------------------------------------------------------------------
// codes -> f16 tiles
// ---------------------------------------------------------------------------
// Piece J of 16 bytes of codes: 8 consecutive channels, in channel order.
template <Code C, int J>
__device__ __forceinline__ uint4 decode8(const uint4 &w) {
  uint4 r;
  if constexpr (C == C_INT8 || C == C_FP8) {
    k_word_to_f16<C == C_FP8>(J ? w.z : w.x, r.x, r.y);
    k_word_to_f16<C == C_FP8>(J ? w.w : w.y, r.z, r.w);
  } else if constexpr (C == C_INT4) {
    const uint32_t x = J == 0 ? w.x : J == 1 ? w.y : J == 2 ? w.z : w.w;
    k_nibbles_to_f16(x, r.x, r.y);
    k_nibbles_to_f16(prmt(x, 0u, 0x4432u), r.z, r.w);
  } else {
    const uint32_t x = J / 2 == 0 ? w.x : J / 2 == 1 ? w.y : J / 2 == 2 ? w.z : w.w;
    k_crumbs_to_f16<2 * (J % 2)>(x, r.x, r.y);
    k_crumbs_to_f16<2 * (J % 2) + 1>(x, r.z, r.w);
  }
  return r;
}

// code * (h + l) in one rounding (but for the rounding of code * l).  A 2-bit
// scale is a BF16 absmax (q_max 1), which h holds exactly.
template <Code C>
__device__ __forceinline__ void apply_scales(uint4 &r, const uint4 &h, const uint4 &l) {
  if constexpr (C == C_INT2) {
    r = make_uint4(hmul2_u32(r.x, h.x), hmul2_u32(r.y, h.y), hmul2_u32(r.z, h.z), hmul2_u32(r.w, h.w));
  } else {
    r = make_uint4(hfma2_u32(r.x, h.x, hmul2_u32(r.x, l.x)), hfma2_u32(r.y, h.y, hmul2_u32(r.y, l.y)),
                   hfma2_u32(r.z, h.z, hmul2_u32(r.z, l.z)), hfma2_u32(r.w, h.w, hmul2_u32(r.w, l.w)));
  }
}

// How one thread of 128 covers a tile of codes: chunk c of 16 bytes of rows
// k0 + STEP i.  Pieces of 8 channels go to 16-byte places of the swizzled row;
// threads of one row's two halves would meet in the same banks, so those of
// the upper half take their pieces in another order (the words swapped).
template <int D, Code C>
struct Cover {
  static constexpr int ROW = D * code_bits(C) / 8;
  static constexpr int CH = ROW / 16;              // chunks per row = loads per thread
  static constexpr int NP = 16 * 8 / code_bits(C) / 8;  // pieces per chunk
  static constexpr int STEP = kTile / CH;
  static constexpr int UNITS = kTile * ROW / static_cast<int>(kUnit);  // ring units of a tile
  int c, k0;
  bool swap;
  uint32_t place, row0;  // of piece 0 at row k0
  __device__ __forceinline__ explicit Cover(int tid) {
    c = tid % CH;
    k0 = tid / CH;
    const int piece = c * NP;
    swap = D == 128 && piece >= 8;
    const uint32_t x = (piece & 7) ^ (swap ? NP / 2 : 0) ^ (k0 & 7);
    place = x << 4;
    row0 = (piece >> 3) * Smem<D>::HALF + k0 * 128;
  }
};

// A tile of codes out of its ring into its f16 tile.  `scale(i, j, r)` applies
// scales to piece j (in the thread's order) of load i.  Codes of missing blocks
// (bit clear in mask) read as 0.
template <int D, Code C, typename Scale>
__device__ __forceinline__ void convert_tile(const Cover<D, C> &f, const Waiter &wait, int which, uint32_t ring,
                                             const Layout &y, int &unit, uint32_t &phase, uint32_t tile, uint32_t mask,
                                             int lane, Scale scale) {
  using F = Cover<D, C>;
  constexpr int LPU = F::CH / F::UNITS;  // loads per thread and unit
  static_assert(LPU == 2, "two loads per thread and unit");
  // loads that are unrolled together: enough to overlap their latencies, few
  // enough for the instruction caches that the roles of an SM's warps share
  constexpr int U = C == C_INT2 ? 1 : 2;
#pragma unroll 1
  for (int u = 0; u < F::UNITS; ++u) {
    wait(B_FULL + which * kMaxUnits + unit, phase);
    const uint32_t raw = ring + unit * kUnit;
#pragma unroll 1
    for (int e0 = 0; e0 < LPU; e0 += U) {
      uint4 w[U];
#pragma unroll
      for (int e = 0; e < U; ++e) w[e] = lds128(raw + swz<F::ROW>((f.k0 + F::STEP * (e0 + e)) * F::ROW + 16 * f.c));
      if (mask != 0xFFu) {
#pragma unroll
        for (int e = 0; e < U; ++e)
          if (!((mask >> ((f.k0 + F::STEP * (LPU * u + e0 + e)) / kBlockSize)) & 1u)) w[e] = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int i = LPU * u + e0 + e;
        const uint4 x = f.swap ? make_uint4(w[e].z, w[e].w, w[e].x, w[e].y) : w[e];
        const uint32_t at = tile + f.row0 + i * F::STEP * 128;
        auto piece = [&](auto jj) {
          constexpr int J = decltype(jj)::value;
          if constexpr (J < F::NP) {
            uint4 r = decode8<C, J>(x);
            scale(i, J, r);
            sts128(at + (f.place ^ (16u * J)), r.x, r.y, r.z, r.w);
          }
        };
        piece(std::integral_constant<int, 0>{});
        piece(std::integral_constant<int, 1>{});
        piece(std::integral_constant<int, 2>{});
        piece(std::integral_constant<int, 3>{});
        piece(std::integral_constant<int, 4>{});
        piece(std::integral_constant<int, 5>{});
        piece(std::integral_constant<int, 6>{});
        piece(std::integral_constant<int, 7>{});
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&wait.bars[B_EMPTY + which * kMaxUnits + unit]);
    if (++unit == y.units[which]) {
      unit = 0;
      phase ^= 1;
    }
  }
}

template <int D, int KF>
__device__ __noinline__ void convert_k_role(uint32_t base, const Layout &y, const Waiter &wait, int tiles) {
  using L = Smem<D>;
  using KC = KCode<KF>;
  using F = Cover<D, KC::code>;
  const int tid = threadIdx.x & 127, lane = tid & 31;
  const F f(tid);
  const uint32_t chan = base + y.small + L::scales, ring = base + y.ring[0];
  int unit = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (int n = 0; n < tiles; ++n) {
    const int st = n & 1;
    const uint32_t ph = (n >> 1) & 1;
    wait(B_META + st, ph);
    const uint32_t mask = lds64(base + y.small + L::info + (n % kMeta) * 8).y;
    wait(B_KEMPTY + st, ph ^ 1);
    convert_tile<D, KC::code>(f, wait, 0, ring, y, unit, phase, base + L::k + st * L::TILE, mask, lane,
                              [&](int i, int j, uint4 &r) {
      if constexpr (KC::chan) {
        const int blk = (f.k0 + F::STEP * i) / kBlockSize;
        const int piece = f.c * F::NP + (f.swap ? j ^ (F::NP / 2) : j);
        const uint32_t p = chan + st * 2 * L::CHAN + (blk * D + 8 * piece) * 2;
        const uint4 hi = lds128(p);
        apply_scales<KC::code>(r, hi, KC::code == C_INT2 ? hi : lds128(p + L::CHAN));
      }
    });
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(&wait.bars[B_KFULL + st]);
  }
}

template <int D, int VF>
__device__ __noinline__ void convert_v_role(uint32_t base, const Layout &y, const Waiter &wait, int tiles) {
  using L = Smem<D>;
  using VC = VCode<VF>;
  using F = Cover<D, VC::code>;
  constexpr int NG = D / 32;
  const int tid = threadIdx.x & 127, lane = tid & 31;
  const F f(tid);
  const uint32_t grp = base + y.small + L::scales + y.grp, ring = base + y.ring[1];
  int unit = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (int n = 0; n < tiles; ++n) {
    const int st = n & 1;
    const uint32_t ph = (n >> 1) & 1;
    wait(B_META + st, ph);
    const uint32_t mask = lds64(base + y.small + L::info + (n % kMeta) * 8).y;
    wait(B_VEMPTY + st, ph ^ 1);
    convert_tile<D, VC::code>(f, wait, 1, ring, y, unit, phase, base + L::v + st * L::TILE, mask, lane,
                              [&](int i, int j, uint4 &r) {
      if constexpr (VC::group) {
        const int key = f.k0 + F::STEP * i;
        const int piece = f.c * F::NP + (f.swap ? j ^ (F::NP / 2) : j);
        const uint32_t z = lds32(grp + st * L::GRP + (key * NG + piece / 4) * 4);
        const uint32_t hi = prmt(z, 0u, 0x1010u), lo = prmt(z, 0u, 0x3232u);
        apply_scales<VC::code>(r, make_uint4(hi, hi, hi, hi), make_uint4(lo, lo, lo, lo));
      }
    });
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(&wait.bars[B_VFULL + st]);
  }
}

// ---------------------------------------------------------------------------
// loads
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_tile_load(uint32_t dst, const CUtensorMap *map, int head, int block, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(head), "r"(0), "r"(block), "r"(smem_u32(bar))
      : "memory");
}

// The tiles of the CTA's range one by one, with the ids of the blocks of the
// next two tiles under way: lane j of a warp has block j % 8.
struct TileWalk {
  const PrefixArgs &a;
  const int x1;
  int x;                  // this tile
  const int32_t *row;     // of the next tile: the leader's table, its shared blocks, its segment's end
  int count, t1, end;
  int h, h1, raw, raw1, b;
  bool first, first1;     // first tile of a segment
  __device__ __forceinline__ TileWalk(const PrefixArgs &args, int from, int to)
      : a(args), x1(to), x(from - 2), t1(0), end(0), h1(0), raw1(INT_MIN), b(threadIdx.x & 7), first1(false) {}
  // to the next tile, and the ids of the one after it (twice to reach the first)
  __device__ __forceinline__ void next() {
    ++x;
    h = h1;
    raw = raw1;
    first = first1;
    if (x + 1 >= x1) return;
    first1 = ++t1 >= end;
    if (first1) {
      Segment s;
      segment_at(a, x + 1, x1, &s);
      row = a.tables + static_cast<int64_t>(s.g.lead) * a.max_blocks;
      count = s.g.shared / kBlockSize;
      t1 = s.t0;
      end = s.t1;
      h1 = s.h;
    }
    const int j = t1 * kTileBlocks + b;
    raw1 = j < count ? __ldg(row + j) : INT_MIN;
  }
  // the id, or -1 past the prefix and for ids out of range
  __device__ __forceinline__ int id(bool report) const {
    if (raw >= 0 && raw < a.num_blocks) return raw;
    if (report && raw != INT_MIN) set_error(a.err, KVQ_DEVERR_BLOCK_RANGE);
    return -1;
  }
};

// Codes into the rings, a TMA box (16 rows of one head) per block: lanes 0 .. 7
// have the tile's K blocks, 8 .. 15 its V blocks.  The lanes of a ring poll
// together for its next place, so K and V do not wait for each other.
__device__ __noinline__ void load_role(const PrefixArgs &a, const CUtensorMap *kmap, const CUtensorMap *vmap, int krow,
                                       int vrow, uint32_t base, const Layout &y, const Waiter &wait, int x, int x1) {
  const int lane = threadIdx.x & 31, r = (lane >> 3) & 1;
  const int row = r ? vrow : krow, units = kTile * row / static_cast<int>(kUnit);  // units of a tile
  const int u = (lane & 7) * units / kTileBlocks;  // the unit of this lane's block
  const uint32_t box = kBlockSize * row, place = base + y.ring[r] + ((lane & 7) - u * (kTileBlocks / units)) * box;
  const CUtensorMap *map = r ? vmap : kmap;
  TileWalk w(a, x, x1);
#pragma unroll 1
  for (int k = 0; k < 2; ++k) w.next();
  int id = w.id(lane < 8), slot = 0, turn = 0, used = 0;
  uint32_t phase = 1, used_phase = 0;
  bool left = lane < 16, stopped = false;
  long long last = clock64();
#pragma unroll 1
  while (__any_sync(0xffffffffu, left) && !stopped) {
    const int bar = r * kMaxUnits + slot;
    const bool go = left && mbar_test_wait(&wait.bars[B_EMPTY + bar], phase);
    const bool in = go && u == turn && id >= 0;
    const uint32_t went = __ballot_sync(0xffffffffu, go), boxes = __ballot_sync(0xffffffffu, in) >> (8 * r) & 0xFFu;
    uint64_t *full = &wait.bars[B_FULL + bar];
    if (go && (lane & 7) == 0) {
      if (boxes) mbar_arrive_expect_tx(full, __popc(boxes) * box);
      else mbar_arrive(full);
    }
    __syncwarp();
    if (in) tma_tile_load(place + slot * kUnit, map, w.h, id, full);
    if (go) {
      used = slot;
      used_phase = phase;
      if (++slot == y.units[r]) {
        slot = 0;
        phase ^= 1;
      }
      if (++turn == units) {
        turn = 0;
        w.next();
        left = w.x < x1;
        id = w.id(lane < 8 && left);
      }
    }
    __syncwarp();
    if (went) {
      last = clock64();
    } else {
      // (decided by the whole warp: its lanes leave the loop together)
      const bool late = clock64() - last > kWaitTicks;
      if (late && lane == 0) {
        *wait.abort = 1;
        set_error(a.err, KVQ_DEVERR_TIMEOUT);
      }
      stopped = __any_sync(0xffffffffu, late || *wait.abort != 0);
    }
  }
  // no copy in flight when the CTA exits: the rings' last units, and so all
  // before them, are read, or (a wait ran out, and nobody reads) a millisecond
  // goes by
  if (stopped) {
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000) {
    }
  } else if (lane == 0 || lane == 8) {
    wait(B_EMPTY + r * kMaxUnits + used, used_phase ^ 1);
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------
// scales
// ---------------------------------------------------------------------------
// Per tile: the position factors ks and vs, F and the block mask, and for the
// converters the scaled channel or group scales as f16 pairs.  Lane l has the
// positions 4 l .. 4 l + 3.
template <int D, bool CHAN, bool GROUP>
__device__ __noinline__ void scale_role(const PrefixArgs &a, uint32_t base, const Layout &y, const Waiter &wait, int x,
                                        int x1) {
  using L = Smem<D>;
  constexpr int NG = GROUP ? D / 32 : 1;
  constexpr int NC = CHAN ? kTileBlocks * D / 128 : 1;  // float4 of channel scales
  const int lane = threadIdx.x & 31;
  const uint32_t small = base + y.small, chan = small + L::scales, grp = chan + y.grp;
  TileWalk w(a, x, x1);
  float sk[CHAN ? 1 : 4], sv[4][NG];
  float4 sc[NC];
  uint32_t mask = 0;
  bool first = false;
  int F = kNoScale;
  const int tiles = x1 - x;
  // this lane's places in block 0 of head 0, and the bytes of a block's scales
  const uint8_t *const kp = reinterpret_cast<const uint8_t *>(a.ks) + (CHAN ? 4 * lane % D : 4 * (lane & 3) * a.H) * 4;
  const uint8_t *const vp = reinterpret_cast<const uint8_t *>(a.vs) + 4 * (lane & 3) * a.H * NG * 4;
  const uint32_t kblock = (CHAN ? D : kBlockSize) * a.H * 4, vblock = kBlockSize * a.H * NG * 4;
  // tile n is written while the loads of n + 1 are under way, and the ids of
  // n + 2; one copy of each part
#pragma unroll 1
  for (int n = -2; n < tiles; ++n) {
    if (n >= 0) {
    const int st = n & 1, slot = n % kMeta;
    if (first) F = kNoScale;
    float vmax = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < NG; ++e) vmax = fmaxf(vmax, sv[i][e]);
    vmax = __uint_as_float(warp_max_u32(__float_as_uint(vmax)));
    // F: the tile's largest V scale times 2^F below 2^9, set to [2^7, 2^8)
    if (vmax > 0.f && (F == kNoScale || ilog2f(vmax) + F >= kTopV)) F = min(kTopV - 2 - ilog2f(vmax), kMaxVExp);
    const float pf = F == kNoScale ? 1.f : pow2i(F);
    // tile n - 2 is converted, and so tile n - 4 is out of the products: this
    // tile's places are free
    wait(B_KFULL + st, ((n >> 1) & 1) ^ 1);
    wait(B_VFULL + st, ((n >> 1) & 1) ^ 1);
    const uint32_t at = small + (slot * kTile + 4 * lane) * 4;
    auto store4 = [](uint32_t to, float p, float q, float r, float s) {
      sts128(to, __float_as_uint(p), __float_as_uint(q), __float_as_uint(r), __float_as_uint(s));
    };
    if constexpr (CHAN) {
      float kmax = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) kmax = fmaxf(fmaxf(kmax, fmaxf(sc[i].x, sc[i].y)), fmaxf(sc[i].z, sc[i].w));
      kmax = __uint_as_float(warp_max_u32(__float_as_uint(kmax)));
      const int eb = kmax > 0.f ? min(7 - ilog2f(kmax), kMaxVExp) : 0;
      const float f = pow2i(eb), back = pow2i(-eb);
      store4(at + L::ks, back, back, back, back);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        uint32_t h0, l0, h1, l1;
        split_f16x2(sc[i].x * f, sc[i].y * f, h0, l0);
        split_f16x2(sc[i].z * f, sc[i].w * f, h1, l1);
        const uint32_t p = chan + st * 2 * L::CHAN + 8 * (lane + 32 * i);
        sts64(p, h0, h1);
        sts64(p + L::CHAN, l0, l1);
      }
    } else {
      store4(at + L::ks, sk[0], sk[1], sk[2], sk[3]);
    }
    if constexpr (!GROUP) {
      store4(at + L::vs, sv[0][0] * pf, sv[1][0] * pf, sv[2][0] * pf, sv[3][0] * pf);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t z[NG];
#pragma unroll
        for (int e = 0; e < NG; e += 2) {
          uint32_t hi, lo;
          split_f16x2(sv[i][e] * pf, sv[i][e + 1] * pf, hi, lo);
          z[e] = prmt(hi, lo, 0x5410u);
          z[e + 1] = prmt(hi, lo, 0x7632u);
        }
        const uint32_t p = grp + st * L::GRP + (4 * lane + i) * NG * 4;
        if constexpr (NG == 4) sts128(p, z[0], z[1], z[2], z[3]);
        else sts64(p, z[0], z[1]);
      }
    }
    if (lane == 0) sts64(small + L::info + slot * 8, static_cast<uint32_t>(F), mask);
    __syncwarp();
    if (lane == 0) mbar_arrive(&wait.bars[B_META + st]);
    }
    w.next();
    if (n + 1 < 0 || n + 1 >= tiles) continue;
    const int ids = w.id(false);
    first = w.first;
    mask = __ballot_sync(0xffffffffu, ids >= 0) & 0xFFu;
    const int id = __shfl_sync(0xffffffffu, ids, lane / 4);
    const uint64_t blk = static_cast<uint32_t>(max(id, 0));
    const uint8_t *const vq = vp + blk * vblock + w.h * NG * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (!CHAN) sk[i] = __ldg(reinterpret_cast<const float *>(kp + blk * kblock + (w.h + i * a.H) * 4));
      if constexpr (NG == 4) {
        const float4 f = __ldg(reinterpret_cast<const float4 *>(vq + i * a.H * NG * 4));
        sv[i][0] = f.x; sv[i][1] = f.y; sv[i][2] = f.z; sv[i][3] = f.w;
      } else if constexpr (NG == 2) {
        const float2 f = __ldg(reinterpret_cast<const float2 *>(vq + i * a.H * NG * 4));
        sv[i][0] = f.x; sv[i][1] = f.y;
      } else {
        sv[i][0] = __ldg(reinterpret_cast<const float *>(vq + i * a.H * NG * 4));
      }
    }
    if constexpr (CHAN) {
      // channels 4 (lane + 32 i) .. of the tile's [block][channel] scales
      const uint8_t *const kq = kp + w.h * D * 4;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const uint32_t b = max(__shfl_sync(0xffffffffu, ids, 4 * (lane + 32 * i) / D), 0);
        sc[i] = __ldg(reinterpret_cast<const float4 *>(kq + static_cast<uint64_t>(b) * kblock));
      }
    }
    if (mask != 0xFFu) {  // missing blocks count as scale 0
      if (id < 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (!CHAN) sk[i] = 0.f;
#pragma unroll
          for (int e = 0; e < NG; ++e) sv[i][e] = 0.f;
        }
      if constexpr (CHAN)
#pragma unroll
        for (int i = 0; i < NC; ++i)
          if (!((mask >> (4 * (lane + 32 * i) / D)) & 1u)) sc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
}

// ---------------------------------------------------------------------------
// the products
// ---------------------------------------------------------------------------
// The whole warp walks the steps and one elected lane issues: what the products
// take (descriptors, addresses) then stays in uniform registers.  Issued from a
// branch of one lane, 16 products took 3000 cycles, three times their work.
template <int D>
__device__ __forceinline__ void product_role(const PrefixArgs &a, uint32_t base, const Waiter &wait, uint32_t tmem_addr,
                                             int x, int x1) {
  using L = Smem<D>;
  constexpr uint32_t id_s = mma_idesc_f16(128, kTile, false), id_o = mma_idesc_f16(128, D, true);
  const bool leader = elect_one();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_addr, 0);
  // descriptors of the first operands; addresses count in units of 16 bytes
  const uint64_t dq = mma_desc(base + L::q, 16, 1024), dk = mma_desc(base + L::k, 16, 1024),
                 dv = mma_desc(base + L::v, L::HALF, 1024);
  int nk = 0, nv = 0;          // tiles consumed so far, by S and by O
  uint32_t np = 0;             // bit i: parity of warpgroup i's steps so far
  for (int seg = 0; x < x1; ++seg) {
    Segment s;
    segment_at(a, x, x1, &s);
    const int tiles = __shfl_sync(0xffffffffu, s.t1 - s.t0, 0), two = __shfl_sync(0xffffffffu, s.two ? 1 : 0, 0);
    const int steps = tiles << two;
    wait(B_Q, seg & 1);
    // the scores run two steps ahead of the outputs
#pragma unroll 1
    for (int j = -2; j < steps; ++j) {
      const int i = j & 1;
      if (j >= 0) {
        const int st = nv & 1;
        wait(B_P + i, (np >> i) & 1);
        np ^= 1u << i;
        if (!two || i == 0) wait(B_VFULL + st, (nv >> 1) & 1);
        __syncwarp();
        tmem_fence_after();
        if (leader) {
          const uint64_t v = dv + st * (L::TILE / 16);
          const uint32_t p = tmem + 128 * i;
#pragma unroll
          for (int e = 0; e < kTile / 16; ++e)
            mma_f16_ts(p + 256, p + 8 * e, v + e * (2048 / 16), id_o, j >= 2 || e > 0);
          if (!two || i == 1) mma_commit(&wait.bars[B_VEMPTY + st]);
          if (j + 2 >= steps) mma_commit(&wait.bars[B_O + i]);
        }
        __syncwarp();
        if (!two || i == 1) ++nv;
      }
      if (j + 2 < steps) {
        const int st = nk & 1;
        if (!two || i == 0) wait(B_KFULL + st, (nk >> 1) & 1);
        __syncwarp();
        tmem_fence_after();
        if (leader) {
          const uint64_t q = dq + (two ? i : 0) * (L::TILE / 16), k = dk + st * (L::TILE / 16);
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            const uint32_t off = ((e / 4) * L::HALF + (e % 4) * 32) / 16;
            mma_f16_ss(tmem + 128 * i, q + off, k + off, id_s, e > 0);
          }
          mma_commit(&wait.bars[B_S + i]);
          if (!two || i == 1) mma_commit(&wait.bars[B_KEMPTY + st]);
        }
        __syncwarp();
        if (!two || i == 1) ++nk;
      }
    }
    x += tiles;
  }
  // nothing in flight when tensor memory is given back
  if (leader) mma_commit(&wait.bars[B_END]);
  __syncwarp();
  wait(B_END, 0);
}

// ---------------------------------------------------------------------------
// softmax
// ---------------------------------------------------------------------------
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// H (sigma q) of a row spread over a warp, CPL channels per lane: stages below
// CPL inside the lane, the others across lanes.
template <int D>
__device__ __noinline__ void rotate_row(const PrefixArgs &a, float (&y)[D / 32], int lane) {
  constexpr int CPL = D / 32;
#pragma unroll
  for (int e = 0; e < CPL; ++e) {
    const int ch = lane * CPL + e;
    y[e] = __uint_as_float(__float_as_uint(y[e]) ^ (((a.rot_signs[ch >> 5] >> (ch & 31)) & 1u) << 31));
  }
#pragma unroll
  for (int d = 1; d < CPL; d <<= 1)
#pragma unroll
    for (int e = 0; e < CPL; ++e)
      if (!(e & d)) {
        const float p = y[e], q = y[e + d];
        y[e] = p + q;
        y[e + d] = p - q;
      }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1)
#pragma unroll
    for (int e = 0; e < CPL; ++e) {
      const float p = __shfl_xor_sync(0xffffffffu, y[e], d);
      y[e] = (lane & d) ? p - y[e] : y[e] + p;
    }
}

// The warp's 32 rows of Q' into their tile; `from` is the lane's row of q, -1
// for none.  Returns this lane's row factor c.  The BF16 rows are copied to the
// places of the f16 rows (all copies in flight at once) and converted there.
template <int D>
__device__ __noinline__ float stage_queries(const PrefixArgs &a, int from, uint32_t tile, int row0, int lane) {
  constexpr int CPL = D / 32;  // channels per lane
  const uint16_t *const q = a.q + lane * CPL;
  const int ch = lane * CPL;
  const uint32_t at = tile + (ch >> 6) * Smem<D>::HALF + (ch & 7) * 2 + row0 * 128;
  const uint32_t chunk = (ch & 63) >> 3;
  float c = 0.f;
#pragma unroll 1
  for (int r = 0; r < 32; ++r) {
    const int row = __shfl_sync(0xffffffffu, from, r);
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(at + r * 128 + ((chunk ^ (r & 7)) << 4)),
                 "l"(q + static_cast<int64_t>(max(row, 0)) * D), "n"(CPL * 2), "r"(row < 0 ? 0 : CPL * 2)
                 : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
#pragma unroll 4
  for (int r = 0; r < 32; ++r) {
    const uint32_t to = at + r * 128 + ((chunk ^ (r & 7)) << 4);
    float y[CPL];
    if constexpr (CPL == 4) {
      const uint2 w = lds64(to);
      y[0] = bf16lo_to_f32(w.x); y[1] = bf16hi_to_f32(w.x); y[2] = bf16lo_to_f32(w.y); y[3] = bf16hi_to_f32(w.y);
    } else {
      const uint32_t w = lds32(to);
      y[0] = bf16lo_to_f32(w); y[1] = bf16hi_to_f32(w);
    }
    if (a.rot) rotate_row<D>(a, y, lane);
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < CPL; ++e) m = fmaxf(m, fabsf(y[e]));
    m = __uint_as_float(warp_max_u32(__float_as_uint(m)));
    // 2^er brings m into [2^14, 2^15).  Below 2^-86 the scores vanish anyway:
    // er <= 100 keeps 2^er and c normal floats.
    const int er = m > 0.f ? min(14 - ilog2f(m), 100) : 0;
    const float f = pow2i(er);
    if (lane == r) c = pow2i(-er);
    uint32_t h[CPL / 2];
#pragma unroll
    for (int e = 0; e < CPL / 2; ++e) h[e] = f32x2_to_f16x2(y[2 * e] * f, y[2 * e + 1] * f);
    if constexpr (CPL == 4) sts64(to, h[0], h[1]);
    else sts32(to, h[0]);
  }
  return c * rsqrtf(static_cast<float>(D)) * kLog2e * (a.rot ? 1.f / D : 1.f);
}

// KS, VS: factors per position of K and V (else the K factor is one number per
// tile, and the V factors are 1).
template <int D, bool KS, bool VS>
__device__ __noinline__ void softmax_role(const PrefixArgs &a, uint8_t *smem, const Layout &y0, const Waiter &wait,
                                             uint32_t tmem, int x, int x1) {
  using L = Smem<D>;
  const uint32_t base = smem_u32(smem);
  const int wg = (threadIdx.x >> 7) - kSoftmaxWarp / 4, warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
  const uint32_t S = tmem + lanes + 128 * wg, O = tmem + lanes + 256 + 128 * wg;
  int n0 = 0;                  // tiles of earlier segments
  uint32_t ns = 0, no = 0;     // steps and segments of this warpgroup so far
  for (int seg = 0; x < x1; ++seg) {
    Segment s;
    segment_at(a, x, x1, &s);
    const int tiles = s.t1 - s.t0, R = s.g.nseq * a.G;
    const int r0 = s.two ? 128 * wg : 0, r = r0 + 32 * warp + lane, row = s.rb * s.g.rows + r;
    const bool live = r < s.g.rows && row < R;
    // ---- queries
    const int b = s.g.start + row / a.G;
    float c = 0.f;
    if (s.two || wg == 0) {
      c = stage_queries<D>(a, live ? b * a.Hq + s.h * a.G + row % a.G : -1, base + L::q + (s.two ? wg : 0) * L::TILE,
                           32 * warp, lane);
      fence_proxy_async_shared();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&wait.bars[B_Q]);
    if (!s.two) {
      // both warpgroups have the same rows: the factors go through shared memory
      float *const f = reinterpret_cast<float *>(smem + y0.small + L::factors);
      if (wg == 0) f[32 * warp + lane] = c;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      c = f[32 * warp + lane];
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    const int limit = live ? __ldg(a.ws_limit + b) : s.g.shared;
    const int nearest = __reduce_min_sync(0xffffffffu, limit);

    float m = -INFINITY, l = 0.f;  // m as a value of t
    int F = kNoScale;
    bool begun = false, huge = false;
    for (int k = s.two ? 0 : wg; k < tiles; k += s.two ? 1 : 2) {
      const int slot = (n0 + k) % kMeta;
      wait(B_S + wg, ns & 1);
      __syncwarp();
      ++ns;
      tmem_fence_after();
      const uint2 info = lds64(base + y0.small + L::info + slot * 8);
      const int Ft = static_cast<int>(info.x);
      // plain loads, which the compiler may place ahead of their uses
      const float4 *ks = reinterpret_cast<const float4 *>(smem + y0.small + L::ks) + slot * (kTile / 4);
      const float4 *vs = reinterpret_cast<const float4 *>(smem + y0.small + L::vs) + slot * (kTile / 4);
      const int seen = limit - (s.t0 + k) * kTile;  // positions of the tile that the row attends to
      const bool masked = nearest < (s.t0 + k + 1) * kTile || info.y != 0xFFu;
      // The loops over the tile's four pieces of 32 positions stay rolled: fully
      // unrolled, the roles' code does not fit the instruction caches, and
      // fetching it bounds the kernel.
      //
      // ---- the row's largest t = S ks; with factors per position, t replaces S
      // (-inf where the row does not attend)
      float top = -INFINITY;
      const float k0 = KS ? 1.f : ks[0].x;
      auto largest = [&](auto tag) {
        constexpr bool MASK = decltype(tag)::value;
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll 1
        for (int cc = 0; cc < kTile / 32; ++cc) {
          uint32_t w[32];
          tmem_ld32(S + 32 * cc, w);
          const float4 *const f = ks + 8 * cc;
          tmem_wait_ld(w);
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            if constexpr (KS) {
              const float4 g = f[e / 4];
              mul_f32x2(__uint_as_float(w[e]), __uint_as_float(w[e + 1]), g.x, g.y, y[e], y[e + 1]);
              mul_f32x2(__uint_as_float(w[e + 2]), __uint_as_float(w[e + 3]), g.z, g.w, y[e + 2], y[e + 3]);
            } else {
#pragma unroll
              for (int d = 0; d < 4; ++d) y[e + d] = __uint_as_float(w[e + d]);
            }
          }
          if constexpr (MASK) {
            const uint32_t in = info.y >> (2 * cc);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * cc + e >= seen || !((in >> (e / kBlockSize)) & 1u)) y[e] = -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            t0 = max3(t0, y[e], y[e + 1]);
            t1 = max3(t1, y[e + 2], y[e + 3]);
          }
          if constexpr (KS || MASK) {
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(y[e]);
            tmem_st32(S + 32 * cc, w);
          }
        }
        if constexpr (KS || MASK) tmem_wait_st();
        top = fmaxf(t0, t1) * k0;
      };
      if (masked) largest(std::true_type{}); else largest(std::false_type{});
      // ---- m and F: O follows
      const bool raise = top != -INFINITY && (m == -INFINITY || (top - m) * c > kRaise);
      if (__any_sync(0xffffffffu, raise) || Ft != F) {
        const float mn = fmaxf(m, top);
        const float keep = m == -INFINITY ? 0.f : fast_exp2((m - mn) * c);
        m = mn;
        l *= keep;
        if (begun) {
          const float ko = F == kNoScale ? keep : keep * scale_pow2(1.f, Ft - F);
#pragma unroll 1
          for (int cc = 0; cc < D / 16; ++cc) {
            uint32_t w[16];
            tmem_ld16(O + 16 * cc, w);
            tmem_wait_ld(w);
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * ko);
            tmem_st16(O + 16 * cc, w);
          }
          tmem_wait_st();
        }
        F = Ft;
        huge = __any_sync(0xffffffffu, m != -INFINITY && fabsf(m * c) > 0x1p10f);
      }
      begun = true;
      // ---- p = 2^(z - m): plainly t c - RN(m c) in one FMA; beyond |m c| = 2^10
      // the rounding of m c would show in the exponent, so the careful form
      // takes (t - m) c
      auto exponentials = [&](auto tag) {
        constexpr bool careful = decltype(tag)::value;
        const float ref = m == -INFINITY ? 0.f : m, mu = -ref * c, ck = c * k0;
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll 1
        for (int cc = 0; cc < kTile / 32; ++cc) {
          uint32_t w[32];
          tmem_ld32(S + 32 * cc, w);
          const float4 *const f = vs + 8 * cc;
          tmem_wait_ld(w);
          uint32_t P[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float a0 = __uint_as_float(w[e]), a1 = __uint_as_float(w[e + 1]), a2 = __uint_as_float(w[e + 2]),
                  a3 = __uint_as_float(w[e + 3]);
            if constexpr (careful) {
              a0 = (a0 * k0 - ref) * c;
              a1 = (a1 * k0 - ref) * c;
              a2 = (a2 * k0 - ref) * c;
              a3 = (a3 * k0 - ref) * c;
            } else {
              fma_f32x2(a0, a1, ck, ck, mu, mu, a0, a1);
              fma_f32x2(a2, a3, ck, ck, mu, mu, a2, a3);
            }
            a0 = fast_exp2(a0);
            a1 = fast_exp2(a1);
            a2 = fast_exp2(a2);
            a3 = fast_exp2(a3);
            add_f32x2(s0, s1, a0, a1, s0, s1);
            add_f32x2(s2, s3, a2, a3, s2, s3);
            if constexpr (VS) {
              const float4 g = f[e / 4];
              mul_f32x2(a0, a1, g.x, g.y, a0, a1);
              mul_f32x2(a2, a3, g.z, g.w, a2, a3);
            }
            P[e / 2] = f32x2_to_f16x2(a0, a1);
            P[e / 2 + 1] = f32x2_to_f16x2(a2, a3);
          }
          // over scores that are in registers by now: 16 columns of P per 32 of S
          tmem_st16(S + 16 * cc, P);
        }
        l += (s0 + s1) + (s2 + s3);
      };
      if (huge) exponentials(std::true_type{}); else exponentials(std::false_type{});
      tmem_wait_st();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&wait.bars[B_P + wg]);
    }
    // ---- the unit's partial state: ml by row, O as [D / 4][rows][4], so that the
    // lanes' 16-byte stores are consecutive
    const int64_t slot0 = s.g.row0 + static_cast<int64_t>(s.u) * s.g.slots + static_cast<int64_t>(blockIdx.x) * kPrefixRows +
                          (s.two ? 0 : wg * s.g.rows);
    if (begun) {
      wait(B_O + wg, no & 1);
      __syncwarp();
      ++no;
      tmem_fence_after();
      const float back = F == kNoScale ? 1.f : pow2i(-F);
#pragma unroll 1
      for (int cc = 0; cc < D / 16; ++cc) {
        uint32_t w[16];
        __syncwarp();
        tmem_ld16(O + 16 * cc, w);
        tmem_wait_ld(w);
        if (live) {
          float4 *o = reinterpret_cast<float4 *>(a.ws_o + slot0 * D) + 4 * cc * s.g.rows + r;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e * s.g.rows] = make_float4(__uint_as_float(w[4 * e]) * back, __uint_as_float(w[4 * e + 1]) * back,
                               __uint_as_float(w[4 * e + 2]) * back, __uint_as_float(w[4 * e + 3]) * back);
        }
      }
      tmem_fence_before();
    } else {
      // one tile for two warpgroups: the other one has it.  Its end is awaited,
      // so that no warpgroup runs a segment ahead.
      wait(B_O, seg & 1);
      __syncwarp();
    }
    if (live) *reinterpret_cast<float2 *>(a.ws_ml + (slot0 + r) * 2) = make_float2(m == -INFINITY ? m : m * c, l);
    x += tiles;
    n0 += tiles;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_attend_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const __grid_constant__ PrefixArgs a, const __grid_constant__ Layout y, const int kf,
                         const int vf, const int krow, const int vrow) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using L = Smem<D>;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + y.small + L::bars);
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int64_t T = a.ws_groups[a.groups].tile0;
  const int P = a.ws_groups[a.groups].tiles, cta = blockIdx.x;
  if (cta >= P) return;
  const int x = static_cast<int>(cta * T / P), x1 = static_cast<int>((cta + 1) * T / P);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[B_KFULL + i], 4);
      mbar_init(&bars[B_KEMPTY + i], 1);
      mbar_init(&bars[B_VFULL + i], 4);
      mbar_init(&bars[B_VEMPTY + i], 1);
      mbar_init(&bars[B_S + i], 1);
      mbar_init(&bars[B_P + i], 4);
      mbar_init(&bars[B_O + i], 1);
      mbar_init(&bars[B_META + i], 1);
    }
    mbar_init(&bars[B_Q], 8);
    mbar_init(&bars[B_END], 1);
    for (int i = 0; i < 2 * kMaxUnits; ++i) {
      mbar_init(&bars[B_FULL + i], 1);
      mbar_init(&bars[B_EMPTY + i], 4);
    }
    mbar_init_fence();
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  uint32_t *const tm = reinterpret_cast<uint32_t *>(smem + y.small + L::tmem);
  if (threadIdx.x == 32) *reinterpret_cast<volatile uint32_t *>(tm + 1) = 0;
  __syncwarp();
  if (warp == kMmaWarp) tmem_alloc(smem_u32(tm), 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tm);

  const Waiter wait = {bars, tm + 1, a.err};
  const int tiles = x1 - x;
  const bool chan = kf == K_INT8_CHAN || kf == K_INT2_CHAN, group = vf == V_INT4_G32 || vf == V_INT2_G32;
  if (warp >= kSoftmaxWarp) {
    if (!chan && !group) softmax_role<D, true, true>(a, smem, y, wait, tmem, x, x1);
    else if (!chan) softmax_role<D, true, false>(a, smem, y, wait, tmem, x, x1);
    else if (!group) softmax_role<D, false, true>(a, smem, y, wait, tmem, x, x1);
    else softmax_role<D, false, false>(a, smem, y, wait, tmem, x, x1);
  } else if (warp >= kVWarp) {
    if (vf == V_INT8_TOK) convert_v_role<D, V_INT8_TOK>(base, y, wait, tiles);
    else if (vf == V_FP8_TOK) convert_v_role<D, V_FP8_TOK>(base, y, wait, tiles);
    else if (vf == V_INT4_G32) convert_v_role<D, V_INT4_G32>(base, y, wait, tiles);
    else if constexpr (D == 128) convert_v_role<D, V_INT2_G32>(base, y, wait, tiles);  // 2-bit rows: head_dim 128
  } else if (warp >= kKWarp) {
    if (kf == K_INT8_TOK) convert_k_role<D, K_INT8_TOK>(base, y, wait, tiles);
    else if (kf == K_FP8_TOK) convert_k_role<D, K_FP8_TOK>(base, y, wait, tiles);
    else if (kf == K_INT8_CHAN) convert_k_role<D, K_INT8_CHAN>(base, y, wait, tiles);
    else if (kf == K_INT4_TOK) convert_k_role<D, K_INT4_TOK>(base, y, wait, tiles);
    else if constexpr (D == 128) convert_k_role<D, K_INT2_CHAN>(base, y, wait, tiles);
  } else if (warp == kMmaWarp) {
    product_role<D>(a, base, wait, tmem, x, x1);
  } else if (warp == kLoadWarp) {
    load_role(a, &kmap, &vmap, krow, vrow, base, y, wait, x, x1);
  } else if (warp == kScaleWarp) {
    if (chan && group) scale_role<D, true, true>(a, base, y, wait, x, x1);
    else if (chan) scale_role<D, true, false>(a, base, y, wait, x, x1);
    else if (group) scale_role<D, false, true>(a, base, y, wait, x, x1);
    else scale_role<D, false, false>(a, base, y, wait, x, x1);
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tmem_fence_after();
    tmem_free(tmem, 512);
  }
}

}  // namespace prefix
}  // namespace kvq
