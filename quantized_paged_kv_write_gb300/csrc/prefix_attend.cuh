// Prefix attention of a group on the fifth-generation tensor cores (sm_103a):
// the kernel behind kvq_prefix_decode's shared part.
//
// Mathematics.  For the rows of a unit (256 or 128 (sequence, query head)
// pairs of one kv head) and a tile of 128 shared positions:
//   S = Q' K'^T          f16 operands, FP32 accumulators in tensor memory
//   t = S s 2^eb         scales per position; scales per channel are in K'
//   z = t 2^-eb c        c the row's factor (z in log2 units)
//   p = 2^(z - m + 8), l += p, O += p V'
// Q' = q 2^er in f16 (the row's largest in [2^14, 2^15): a BF16 q is exact
// down to 2^-32 of it; a rotated one is rounded once).  K' is the codes themselves
// where a position has one scale: it multiplies the score in FP32, and t goes back
// to where S was.  A rounding of K' would move a score by up to 2^-11 of sum |q k|,
// which the softmax raises: with K outliers, whole tenths of an output (K' = code *
// s in f16 was 2 % slower for 27 sequences, FP8, 2 to 10 % faster for 256 and 64
// sequences, whose softmax is the longer chain).  With scales per channel K' = code
// * s 2^eb, and V' = code * s 2^F, are rounded to f16 once.  Powers of two keep t
// in range and K' and V' below 2^15: eb by tile; F falls when a tile's scales need
// it and O follows, as it does when m is raised (only past m + 6, so p <= 2^14).
// p is rounded to f16 once; l sums the unrounded p.
//
// Roles, one CTA per SM: two softmax warpgroups (thread = row), two
// warpgroups that turn codes into f16 tiles in shared memory (one K, one V),
// and a warp each for the products, for the TMA loads of K and of V codes, and
// for the scales of K and of V.  Steps alternate between the two softmax
// warpgroups, so the tensor core works for one while the other is in its
// exponentials:
//   more than 128 rows: warpgroup i owns rows 128 i .. + 127, each tile of
//     codes serves both (steps 2t, 2t + 1 of tile t);
//   at most 128 rows: both own the same rows, warpgroup i the tiles of parity
//     i; each keeps its own (m, l, O), joined in tensor memory at the end.
// P overwrites S in tensor memory and is the A operand of the second product.
//
// What bounds it.  27 sequences, 32 query heads on 8, FP8 K and V, 32003 shared
// positions: 35 us, 66 MB of codes and scales at 1.9 TB/s.  A tile takes ~3500
// cycles of an SM, most of them the converters' chains (load, decode, V: scale,
// store); twice the converter warps at fewer registers gained nothing.  100
// sequences, 64 query heads on 8, INT2 K and V, 65536 positions: 254 us, 0.85
// PFLOP/s, a two-row-tile step in ~4280 cycles, 2080 of them products; the rest is
// the chain S - softmax - P V of a warpgroup, whose single S buffer (tensor memory
// is full: two S, two O) keeps its next S waiting for its P V.  Halves of S to
// overlap them made products of 64 columns, which shared memory's bandwidth slows
// (9 % more time).  Measured on the way: out-of-line roles, which reload their
// parameters after every barrier, 46 instead of 41 us (first shape); one load warp
// for both rings 41 instead of 34 us; scales read again for the exponentials
// instead of t stored 64.0 instead of 61.9 us for the whole call.
#pragma once

#include <limits.h>

#include "mbar_wait.cuh"
#include "paged_decode_impl.cuh"
#include "tcgen05.cuh"

namespace kvq {
namespace prefix {

constexpr int kTile = kPrefixTile;             // positions per tile
constexpr int kTileBlocks = kTile / kBlockSize;
// Warps by role: the single-warp roles, which everybody waits for, come first.
constexpr int kMmaWarp = 0, kLoadWarp = 1, kScaleWarp = 2, kKWarp = 4, kVWarp = 8, kSoftmaxWarp = 12, kLoadVWarp = 20;
constexpr int kThreads = 21 * 32;
constexpr uint32_t kPair = 4096;               // codes that a converter warpgroup takes in one turn
constexpr int kMaxUnits = 8;                   // per ring
constexpr uint32_t kMaxSmem = 227 * 1024;
constexpr int kMeta = 4;                       // ring of per-tile factors
constexpr float kRaise = 6.f;                  // m is raised past m + 6
constexpr float kBias = 8.f;                   // p's factor 2^8: small p stay normal f16 numbers

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
// Scales below 2^top keep code * scale below 2^15 (codes up to 448, 127, 7, 1).
constexpr int top_exponent(Code c) { return c == C_FP8 ? 6 : 8; }

// Shared memory: f16 tiles ([64-channel half][row][128 bytes], swizzled), then
// the small arrays, then the ring of codes, as long as there is room.
template <int D>
struct Smem {
  static constexpr uint32_t HALF = 128 * 128;           // 64 channels of 128 rows
  static constexpr uint32_t TILE = HALF * (D / 64);
  static constexpr uint32_t CHAN = kTileBlocks * D * 2; // one part (high or low) of the channel scales
  static constexpr uint32_t POS = kTile * 4;            // scales per position, f16 pairs (high, low) or FP32
  static constexpr uint32_t GRP = POS * (D / 32);       // and per position and group
  static constexpr uint32_t k = 0;                      // [2] stages
  static constexpr uint32_t v = k + 2 * TILE;           // [2] stages
  static constexpr uint32_t q = v + 2 * TILE;           // [1 or 2] row tiles
  // offsets from the end of q
  static constexpr uint32_t info = 0;                   // [kMeta] {F, block mask, 2^-eb, -}
  static constexpr uint32_t bars = info + kMeta * 16;   // mbarriers
  static constexpr uint32_t tmem = bars + 56 * 8;       // tensor memory address, then the abort flag
  static constexpr uint32_t factors = tmem + 16;        // [128] row factors
  static constexpr uint32_t segment = factors + 512;    // the CTA's first segment
  // scales of K: [2] f16 pairs per channel, or [kMeta] FP32 per position; then
  // [2] of V, f16 pairs
  static constexpr uint32_t scales = segment + 96;
  static_assert(scales % 16 == 0, "small arrays");
};

// What depends on the formats and on whether any unit has two row tiles.
struct Layout {
  uint32_t small, vscales;    // offsets: small arrays, scales of V (from `scales`)
  uint32_t ring[2];           // the rings of K and V codes
  int units[2];               // places in the rings,
  uint32_t unit[2];           // and their bytes: a tile of codes or a part of one
  uint32_t bytes;
};
template <int D>
inline Layout layout_of(bool chan, bool group, bool two, int krow, int vrow) {
  using L = Smem<D>;
  Layout y;
  y.small = L::q + (two ? 2 : 1) * L::TILE;
  y.vscales = chan ? 4 * L::CHAN : kMeta * L::POS;
  y.ring[0] = (y.small + L::scales + y.vscales + 2 * (group ? L::GRP : L::POS) + 1023) & ~1023u;
  // Units of up to 8 KB, fewer to wait for; of 4 KB where two row tiles leave
  // little room.  As many as fit, shared out by the bytes of a row.
  const uint32_t room = kMaxSmem - y.ring[0], most = two ? kPair : 2 * kPair;
  const int row[2] = {krow, vrow};
  for (int i = 0; i < 2; ++i) y.unit[i] = kTile * row[i] < static_cast<int>(most) ? kTile * row[i] : most;
  int k = static_cast<int>((room * krow / (krow + vrow) + y.unit[0] / 2) / y.unit[0]);
  if (k < 1) k = 1;
  while (k > 1 && k * y.unit[0] + y.unit[1] > room) --k;
  const int v = static_cast<int>((room - k * y.unit[0]) / y.unit[1]);
  y.units[0] = k < kMaxUnits ? k : kMaxUnits;
  y.units[1] = v < kMaxUnits ? v : kMaxUnits;
  y.ring[1] = y.ring[0] + y.units[0] * y.unit[0];
  y.bytes = y.ring[1] + y.units[1] * y.unit[1];
  return y;
}

enum Bar : int {
  B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_S = 8, B_P = 10, B_O = 12, B_Q = 14, B_END = 15, B_META = 16,
  B_FULL = 18 /* [2][kMaxUnits] */, B_EMPTY = B_FULL + 2 * kMaxUnits, B_COUNT = B_EMPTY + 2 * kMaxUnits
};
static_assert(B_COUNT <= 56, "mbarriers");

// The part of a unit that this CTA works on.  Out of line, like all that runs
// once a segment: the roles of an SM's warps share its instruction caches, and
// the code of the steps has to stay there.
struct Segment {
  PrefixGroup g;
  int u, h, rb, t0, t1;
  bool two;          // two row tiles
};

__device__ __noinline__ void find_segment(const PrefixArgs &a, int x, int x1, Segment *out) {
  int lo = 0, hi = a.groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.ws_groups[mid].tile0 <= x) lo = mid; else hi = mid;
  }
  Segment s;
  s.g = a.ws_groups[lo];
  const int y = x - s.g.tile0;
  s.u = y / s.g.tiles;
  s.t0 = y - s.u * s.g.tiles;
  s.t1 = min(s.g.tiles, s.t0 + (x1 - x));
  s.h = s.u % a.H;
  s.rb = s.u / a.H;
  s.two = s.g.rows > kPrefixRows / 2;
  *out = s;
}

// The CTA's first segment is found once and kept in shared memory.
struct Segments {
  const Segment *first;
  int x0;
};
__device__ __forceinline__ void segment_at(const PrefixArgs &a, const Segments &f, int x, int x1, Segment *out) {
  if (x == f.x0) *out = *f.first;
  else find_segment(a, x, x1, out);
}

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
  static constexpr int PAIRS = CH / 2;             // turns of two loads, kPair bytes of codes
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
  // loads that are unrolled together: enough to overlap their latencies, few
  // enough for the instruction caches that the roles of an SM's warps share
  constexpr int U = C == C_INT2 ? 1 : 2;
  const uint32_t end = y.unit[which];
  uint32_t done = 0;  // bytes of the unit
#pragma unroll 1
  for (int u = 0; u < F::PAIRS; ++u) {
    if (done == 0) wait(B_FULL + which * kMaxUnits + unit, phase);
    const uint32_t raw = ring + unit * end + done;
#pragma unroll 1
    for (int e0 = 0; e0 < 2; e0 += U) {
      uint4 w[U];
#pragma unroll
      for (int e = 0; e < U; ++e) w[e] = lds128(raw + swz<F::ROW>((f.k0 + F::STEP * (e0 + e)) * F::ROW + 16 * f.c));
      if (mask != 0xFFu) {
#pragma unroll
        for (int e = 0; e < U; ++e)
          if (!((mask >> ((f.k0 + F::STEP * (2 * u + e0 + e)) / kBlockSize)) & 1u)) w[e] = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int i = 2 * u + e0 + e;
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
    done += kPair;
    if (done < end) continue;
    done = 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(&wait.bars[B_EMPTY + which * kMaxUnits + unit]);
    if (++unit == y.units[which]) {
      unit = 0;
      phase ^= 1;
    }
  }
}

// The f16 pair (high, low) of one scale, each part in both halves.
struct ScalePair {
  uint4 hi, lo;
  __device__ __forceinline__ explicit ScalePair(uint32_t z) {
    const uint32_t h = prmt(z, 0u, 0x1010u), l = prmt(z, 0u, 0x3232u);
    hi = make_uint4(h, h, h, h);
    lo = make_uint4(l, l, l, l);
  }
};

template <int D, int KF>
__device__ __forceinline__ void convert_k_role(uint32_t base, const Layout &y, const Waiter &wait, int tiles) {
  using L = Smem<D>;
  using KC = KCode<KF>;
  using F = Cover<D, KC::code>;
  const int tid = threadIdx.x & 127, lane = tid & 31;
  const F f(tid);
  const uint32_t scales = base + y.small + L::scales, ring = base + y.ring[0];
  int unit = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (int n = 0; n < tiles; ++n) {
    const int st = n & 1;
    const uint32_t ph = (n >> 1) & 1;
    wait(B_META + st, ph);
    const uint32_t mask = lds32(base + y.small + L::info + (n % kMeta) * 16 + 4);
    wait(B_KEMPTY + st, ph ^ 1);
    convert_tile<D, KC::code>(f, wait, 0, ring, y, unit, phase, base + L::k + st * L::TILE, mask, lane,
                              [&](int i, int j, uint4 &r) {
      if constexpr (KC::chan) {
        const int blk = (f.k0 + F::STEP * i) / kBlockSize;
        const int piece = f.c * F::NP + (f.swap ? j ^ (F::NP / 2) : j);
        const uint32_t p = scales + st * 2 * L::CHAN + (blk * D + 8 * piece) * 2;
        const uint4 hi = lds128(p);
        apply_scales<KC::code>(r, hi, KC::code == C_INT2 ? hi : lds128(p + L::CHAN));
      }  // (scales per position: the softmax has them)
    });
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(&wait.bars[B_KFULL + st]);
  }
}

template <int D, int VF>
__device__ __forceinline__ void convert_v_role(uint32_t base, const Layout &y, const Waiter &wait, int tiles) {
  using L = Smem<D>;
  using VC = VCode<VF>;
  using F = Cover<D, VC::code>;
  constexpr int NG = VC::group ? D / 32 : 1;
  const int tid = threadIdx.x & 127, lane = tid & 31;
  const F f(tid);
  const uint32_t scales = base + y.small + L::scales + y.vscales, ring = base + y.ring[1];
  int unit = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (int n = 0; n < tiles; ++n) {
    const int st = n & 1;
    const uint32_t ph = (n >> 1) & 1;
    wait(B_META + st, ph);
    const uint32_t mask = lds32(base + y.small + L::info + (n % kMeta) * 16 + 4);
    wait(B_VEMPTY + st, ph ^ 1);
    convert_tile<D, VC::code>(f, wait, 1, ring, y, unit, phase, base + L::v + st * L::TILE, mask, lane,
                              [&](int i, int j, uint4 &r) {
      const int key = f.k0 + F::STEP * i;
      const int piece = f.c * F::NP + (f.swap ? j ^ (F::NP / 2) : j);
      const ScalePair z(lds32(scales + st * L::POS * NG + (key * NG + (VC::group ? piece / 4 : 0)) * 4));
      apply_scales<VC::code>(r, z.hi, z.lo);
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
  const Segments &seg;
  const int x1;
  int x;                  // this tile
  const int32_t *row;     // of the next tile: the leader's table, its shared blocks, its segment's end
  int count, t1, end;
  int h, h1, raw, raw1, b;
  bool first, first1;     // first tile of a segment
  __device__ __forceinline__ TileWalk(const PrefixArgs &args, const Segments &segments, int from, int to)
      : a(args), seg(segments), x1(to), x(from - 2), t1(0), end(0), h1(0), raw1(INT_MIN), b(threadIdx.x & 7), first1(false) {}
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
      segment_at(a, seg, x + 1, x1, &s);
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

// Codes into a ring (r = 0: of K, 1: of V), a TMA box (16 rows of one head) per
// block.  A warp's box takes it ~175 cycles (its lanes issue one by one; one
// lane for all boxes took twice as long), which bounds the kernel with one warp
// for both rings.
__device__ __forceinline__ void load_role(const PrefixArgs &a, const CUtensorMap *map, int row, int r, uint32_t base,
                                          const Layout &y, const Waiter &wait, const Segments &seg, int x, int x1) {
  const int lane = threadIdx.x & 31, tiles = x1 - x, places = y.units[r];
  const uint32_t box = kBlockSize * row, bytes = y.unit[r], ring = base + y.ring[r];
  const int per = static_cast<int>(bytes / box);  // blocks of a unit
  TileWalk w(a, seg, x, x1);
  int at = 0;
  uint32_t ph = 1;
  w.next();
#pragma unroll 1
  for (int n = 0; n < tiles; ++n) {
    w.next();
    const int id = w.id(lane < 8 && r == 0);
#pragma unroll 1
    for (int b = 0; b < kTileBlocks; b += per) {
      const int bar = r * kMaxUnits + at;
      wait(B_EMPTY + bar, ph);
      const bool in = static_cast<unsigned>(lane - b) < static_cast<unsigned>(per) && id >= 0;
      const int boxes = __popc(__ballot_sync(0xffffffffu, in));
      uint64_t *full = &wait.bars[B_FULL + bar];
      if (lane == 0) {
        if (boxes) mbar_arrive_expect_tx(full, boxes * box);
        else mbar_arrive(full);
      }
      __syncwarp();
      // (after a wait that ran out nobody reads: no further copies)
      if (in && !*wait.abort) tma_tile_load(ring + at * bytes + (lane - b) * box, map, w.h, id, full);
      if (++at == places) {
        at = 0;
        ph ^= 1;
      }
    }
  }
  // no copy in flight when the CTA exits: all units are read, or (a wait ran
  // out) a millisecond goes by
  if (*wait.abort) {
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000) {
    }
  }
#pragma unroll 1
  for (int k = 0; k < places; ++k) {
    wait(B_EMPTY + r * kMaxUnits + at, ph);
    if (++at == places) {
      at = 0;
      ph ^= 1;
    }
  }
}

// ---------------------------------------------------------------------------
// scales
// ---------------------------------------------------------------------------
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// Two warps: the scales of K 2^eb, per position in FP32 for the softmax or per
// channel, and of V 2^F as pairs of f16 (high and low part), for the converters; F,
// the block mask and 2^-eb, for the softmax.  Lane
// l has the positions 4 l .. 4 l + 3.  Tile n is written while the loads of n + 1
// are under way, and the ids of n + 2; one copy of each part.

// Tile n - 2 is converted, and so tile n - 4 is out of the products: tile n's
// places are free.
__device__ __forceinline__ void wait_places(const Waiter &wait, int n) {
  wait(B_KFULL + (n & 1), ((n >> 1) & 1) ^ 1);
  wait(B_VFULL + (n & 1), ((n >> 1) & 1) ^ 1);
}

// x f and y f as two f16 pairs, high and (LOW) low parts.
template <bool LOW>
__device__ __forceinline__ void scaled_pair(float x, float y, float f, uint32_t &hi, uint32_t &lo) {
  mul_f32x2(x, y, f, f, x, y);
  if constexpr (LOW) {
    split_f16x2(x, y, hi, lo);
  } else {
    hi = f32x2_to_f16x2(x, y);
    lo = 0u;
  }
}

// Pairs of N scales (N even) times f, as (high, low) words.
template <bool LOW, int N>
__device__ __forceinline__ void pair_scales(const float (&s)[N], float f, uint32_t (&z)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    uint32_t hi, lo;
    scaled_pair<LOW>(s[e], s[e + 1], f, hi, lo);
    z[e] = prmt(hi, lo, 0x5410u);
    z[e + 1] = prmt(hi, lo, 0x7632u);
  }
}

// LOW false: 2-bit codes, whose scales are BF16 numbers (q_max 1).
template <int D, bool CHAN, bool LOW>
__device__ __forceinline__ void scale_k_role(const PrefixArgs &a, uint32_t base, const Layout &y,
                                          const Waiter &wait, const Segments &seg, int top, int x, int x1) {
  using L = Smem<D>;
  constexpr int NC = CHAN ? kTileBlocks * D / 128 : 1;  // float4 of scales
  const int lane = threadIdx.x & 31, tiles = x1 - x;
  const uint32_t small = base + y.small, to = small + L::scales;
  TileWalk w(a, seg, x, x1);
  float sk[NC][4];
  // this lane's place in block 0 of head 0, and the bytes of a block's scales
  const uint8_t *const kp = reinterpret_cast<const uint8_t *>(a.ks) + (CHAN ? 4 * lane % D : 4 * (lane & 3) * a.H) * 4;
  const uint32_t kblock = (CHAN ? D : kBlockSize) * a.H * 4;
#pragma unroll 1
  for (int n = -2; n < tiles; ++n) {
    if (n >= 0) {
      const int st = n & 1;
      float kmax = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) kmax = max3(max3(kmax, sk[i][0], sk[i][1]), sk[i][2], sk[i][3]);
      kmax = __uint_as_float(warp_max_u32(__float_as_uint(kmax)));
      const int eb = kmax > 0.f ? min(top - 1 - ilog2f(kmax), kMaxVExp) : 0;
      const float f = pow2i(eb);
      wait_places(wait, n);
      if constexpr (CHAN) {
        const uint32_t p = to + st * 2 * L::CHAN + 8 * lane;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          uint32_t h0, l0, h1, l1;
          scaled_pair<LOW>(sk[i][0], sk[i][1], f, h0, l0);
          scaled_pair<LOW>(sk[i][2], sk[i][3], f, h1, l1);
          sts64(p + 256 * i, h0, h1);
          if constexpr (LOW) sts64(p + 256 * i + L::CHAN, l0, l1);
        }
      } else {
        sts128(to + n % kMeta * L::POS + 16 * lane, __float_as_uint(sk[0][0] * f), __float_as_uint(sk[0][1] * f),
               __float_as_uint(sk[0][2] * f), __float_as_uint(sk[0][3] * f));
      }
      if (lane == 0) sts32(small + L::info + (n % kMeta) * 16 + 8, __float_as_uint(pow2i(-eb)));
      __syncwarp();
      if (lane == 0) mbar_arrive(&wait.bars[B_META + st]);
    }
    w.next();
    if (n + 1 < 0 || n + 1 >= tiles) continue;
    const int ids = w.id(false);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      // channels 4 (lane + 32 i) .. of the tile's [block][channel] scales, or positions
      const int b = __shfl_sync(0xffffffffu, ids, CHAN ? 4 * (lane + 32 * i) / D : lane / 4);
      const uint8_t *const kq = kp + static_cast<uint64_t>(static_cast<uint32_t>(max(b, 0))) * kblock + w.h * (CHAN ? D * 4 : 4);
      if constexpr (CHAN) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(kq));
        sk[i][0] = v.x; sk[i][1] = v.y; sk[i][2] = v.z; sk[i][3] = v.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) sk[i][e] = __ldg(reinterpret_cast<const float *>(kq + e * a.H * 4));
      }
    }
    if (__any_sync(0xffffffffu, ids < 0)) {  // missing blocks count as scale 0
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (__shfl_sync(0xffffffffu, ids, CHAN ? 4 * (lane + 32 * i) / D : lane / 4) < 0)
          sk[i][0] = sk[i][1] = sk[i][2] = sk[i][3] = 0.f;
    }
  }
}

template <int D, bool GROUP, bool LOW>
__device__ __forceinline__ void scale_v_role(const PrefixArgs &a, uint32_t base, const Layout &y,
                                          const Waiter &wait, const Segments &seg, int top, int x, int x1) {
  using L = Smem<D>;
  constexpr int NG = GROUP ? D / 32 : 1;
  const int lane = threadIdx.x & 31, tiles = x1 - x;
  const uint32_t small = base + y.small, to = small + L::scales + y.vscales;
  TileWalk w(a, seg, x, x1);
  float sv[4 * NG];
  uint32_t mask = 0;
  bool first = false;
  int F = kNoScale;
  const uint8_t *const vp = reinterpret_cast<const uint8_t *>(a.vs) + 4 * (lane & 3) * a.H * NG * 4;
  const uint32_t vblock = kBlockSize * a.H * NG * 4;
#pragma unroll 1
  for (int n = -2; n < tiles; ++n) {
    if (n >= 0) {
      const int st = n & 1;
      if (first) F = kNoScale;
      float vmax = 0.f;
#pragma unroll
      for (int e = 0; e < 4 * NG; ++e) vmax = fmaxf(vmax, sv[e]);
      vmax = __uint_as_float(warp_max_u32(__float_as_uint(vmax)));
      // F: the tile's largest V scale times 2^F below 2^top, set two below
      if (vmax > 0.f && (F == kNoScale || ilog2f(vmax) + F >= top)) F = min(top - 2 - ilog2f(vmax), kMaxVExp);
      wait_places(wait, n);
      uint32_t z[4 * NG];
      pair_scales<LOW>(sv, F == kNoScale ? 1.f : pow2i(F), z);
#pragma unroll
      for (int e = 0; e < 4 * NG; e += 4)
        sts128(to + (st * L::POS + 16 * lane) * NG + 4 * e, z[e], z[e + 1], z[e + 2], z[e + 3]);
      if (lane == 0) sts64(small + L::info + (n % kMeta) * 16, static_cast<uint32_t>(F), mask);
      __syncwarp();
      if (lane == 0) mbar_arrive(&wait.bars[B_META + st]);
    }
    w.next();
    if (n + 1 < 0 || n + 1 >= tiles) continue;
    const int ids = w.id(false);
    first = w.first;
    mask = __ballot_sync(0xffffffffu, ids >= 0) & 0xFFu;
    const int id = __shfl_sync(0xffffffffu, ids, lane / 4);
    const uint8_t *const vq = vp + static_cast<uint64_t>(static_cast<uint32_t>(max(id, 0))) * vblock + w.h * NG * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (NG == 4) {
        const float4 f = __ldg(reinterpret_cast<const float4 *>(vq + i * a.H * NG * 4));
        sv[4 * i] = f.x; sv[4 * i + 1] = f.y; sv[4 * i + 2] = f.z; sv[4 * i + 3] = f.w;
      } else if constexpr (NG == 2) {
        const float2 f = __ldg(reinterpret_cast<const float2 *>(vq + i * a.H * NG * 4));
        sv[2 * i] = f.x; sv[2 * i + 1] = f.y;
      } else {
        sv[i] = __ldg(reinterpret_cast<const float *>(vq + i * a.H * NG * 4));
      }
    }
    if (id < 0)  // missing blocks count as scale 0
#pragma unroll
      for (int e = 0; e < 4 * NG; ++e) sv[e] = 0.f;
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
                                             const Segments &sg, int x, int x1) {
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
    segment_at(a, sg, x, x1, &s);
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
// H (sigma q) of a row spread over a warp, CPL channels per lane: stages below
// CPL inside the lane, the others across lanes.
template <int D>
__device__ __forceinline__ void rotate_row(const PrefixArgs &a, float (&y)[D / 32], int lane) {
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
template <int D, bool ROT>
__device__ __noinline__ float stage_queries(const PrefixArgs &a, int from, uint32_t tile, int row0, int lane) {
  constexpr int CPL = D / 32;  // channels per lane
  const uint16_t *const q = a.q + lane * CPL;
  const int ch = lane * CPL;
  const uint32_t at = tile + (ch >> 6) * Smem<D>::HALF + (ch & 7) * 2 + row0 * 128;
  const uint32_t chunk = ((ch & 63) >> 3) << 4;
  float c = 0.f;
#pragma unroll 4
  for (int r = 0; r < 32; ++r) {
    const int row = __shfl_sync(0xffffffffu, from, r);
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(at + r * 128 + (chunk ^ ((r & 7) << 4))),
                 "l"(q + static_cast<uint64_t>(static_cast<uint32_t>(max(row, 0))) * D), "n"(CPL * 2),
                 "r"(row < 0 ? 0 : CPL * 2)
                 : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
#pragma unroll(ROT ? 1 : 4)
  for (int r = 0; r < 32; ++r) {
    const uint32_t to = at + r * 128 + (chunk ^ ((r & 7) << 4));
    float y[CPL];
    if constexpr (CPL == 4) {
      const uint2 w = lds64(to);
      y[0] = bf16lo_to_f32(w.x); y[1] = bf16hi_to_f32(w.x); y[2] = bf16lo_to_f32(w.y); y[3] = bf16hi_to_f32(w.y);
    } else {
      const uint32_t w = lds32(to);
      y[0] = bf16lo_to_f32(w); y[1] = bf16hi_to_f32(w);
    }
    if constexpr (ROT) rotate_row<D>(a, y, lane);
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < CPL; ++e) m = fmaxf(m, fabsf(y[e]));
    const uint32_t mb = warp_max_u32(__float_as_uint(m));
    // 2^er brings m into [2^14, 2^15) (a subnormal m counts as 2^-127).  Below
    // 2^-86 the scores vanish anyway: er <= 100 keeps 2^er and c normal floats.
    const int er = min(14 + 127 - static_cast<int>(mb >> 23), 100);
    const float f = mb < 0x7F800000u ? pow2i(er) : NAN;  // (an infinite row: no score is a number)
    if (lane == r) c = pow2i(-er);
    uint32_t h[CPL / 2];
#pragma unroll
    for (int e = 0; e < CPL / 2; ++e) h[e] = f32x2_to_f16x2(y[2 * e] * f, y[2 * e + 1] * f);
    if constexpr (CPL == 4) sts64(to, h[0], h[1]);
    else sts32(to, h[0]);
  }
  return c * rsqrtf(static_cast<float>(D)) * kLog2e * (ROT ? 1.f / D : 1.f);
}

// The unit's partial state: ml by row, O as [D / 4][rows][4], so that the lanes'
// 16-byte stores are consecutive.  Two warpgroups with the same rows (one row
// tile) join their streams here: both see both outputs in tensor memory and
// take half of the channels each, which halves what the merge has to read.
template <int D>
__device__ __noinline__ void store_partial(const PrefixArgs &a, const Segment &s, uint8_t *exchange, uint32_t O, int wg, bool live,
                                           int r, float m, float l, float back) {
  const int rows = s.g.rows;
  const int64_t slot = s.g.row0 + s.u * rows + static_cast<int>(blockIdx.x) * kPrefixRows;
  float w0 = back, w1 = 0.f;  // of O and of the other stream's
  uint32_t other = O;
  if (s.two) {
    O += 128 * wg;
    other = O;
  } else {
    float4 *const x = reinterpret_cast<float4 *>(exchange);
    x[128 * wg + r] = make_float4(m, l, back, 0.f);
    // each warpgroup has waited for its own products: the barrier passes on that
    // they are complete
    tmem_fence_before();
    asm volatile("bar.sync 1, 256;" ::: "memory");
    tmem_fence_after();
    const float4 y0 = x[r], y1 = x[128 + r];
    m = fmaxf(y0.x, y1.x);
    // (a stream without weight, -inf, may have left anything in its O)
    w0 = y0.x == -INFINITY ? 0.f : fast_exp2(y0.x - m);
    w1 = y1.x == -INFINITY ? 0.f : fast_exp2(y1.x - m);
    l = w0 * y0.y + w1 * y1.y;
    w0 *= y0.z;
    w1 *= y1.z;
    other = O + 128;
  }
  const int n = s.two ? D / 16 : D / 32, c0 = s.two ? 0 : wg * (D / 32);
#pragma unroll 1
  for (int cc = c0; cc < c0 + n; ++cc) {
    uint32_t u[16], v[16];
    __syncwarp();
    tmem_ld16(O + 16 * cc, u);
    tmem_ld16(other + 16 * cc, v);
    tmem_wait_ld(u);
    tmem_wait_ld(v);
    if (live) {
      float4 *o = reinterpret_cast<float4 *>(a.ws_o + slot * D) + 4 * cc * rows + r;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float z[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float p = __uint_as_float(u[4 * e + k]), q = __uint_as_float(v[4 * e + k]);
          z[k] = (w0 != 0.f ? w0 * p : 0.f) + (w1 != 0.f ? w1 * q : 0.f);
        }
        o[e * rows] = make_float4(z[0], z[1], z[2], z[3]);
      }
    }
  }
  if (live && (s.two || wg == 0)) *reinterpret_cast<float2 *>(a.ws_ml + (slot + r) * 2) = make_float2(m, l);
}

// SCALED: a scale per position, which the scores take; else K' has them.
template <int D, bool SCALED>
__device__ __forceinline__ void softmax_role(const PrefixArgs &a, uint8_t *smem, const Layout &y0, const Waiter &wait,
                                             uint32_t tmem, const Segments &sg, int x, int x1) {
  using L = Smem<D>;
  const uint32_t base = smem_u32(smem);
  const int wg = (threadIdx.x >> 7) - kSoftmaxWarp / 4, warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
  const uint32_t S = tmem + lanes + 128 * wg, O = tmem + lanes + 256 + 128 * wg;
  int n0 = 0;                  // tiles of earlier segments
  uint32_t ns = 0, no = 0;     // steps and segments of this warpgroup so far
  for (int seg = 0; x < x1; ++seg) {
    Segment s;
    segment_at(a, sg, x, x1, &s);
    const int tiles = s.t1 - s.t0, R = s.g.nseq * a.G;
    const int r0 = s.two ? 128 * wg : 0, r = r0 + 32 * warp + lane, row = s.rb * s.g.rows + r;
    const bool live = r < s.g.rows && row < R;
    // ---- queries
    const int b = s.g.start + row / a.G;
    float c = 0.f;
    if (s.two || wg == 0) {
      const int from = live ? b * a.Hq + s.h * a.G + row - (b - s.g.start) * a.G : -1;
      const uint32_t tile = base + L::q + (s.two ? wg : 0) * L::TILE;
      c = a.rot ? stage_queries<D, true>(a, from, tile, 32 * warp, lane) : stage_queries<D, false>(a, from, tile, 32 * warp, lane);
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
    const int limit = live ? __ldcg(a.ws_limit + b) : s.g.shared;
    const int nearest = __reduce_min_sync(0xffffffffu, limit);

    float m = -INFINITY, l = 0.f;  // m as a value of t 2^-eb
    int F = kNoScale;
    bool begun = false, huge = false;
    for (int k = s.two ? 0 : wg; k < tiles; k += s.two ? 1 : 2) {
      const int slot = (n0 + k) % kMeta;
      wait(B_S + wg, ns & 1);
      __syncwarp();
      ++ns;
      tmem_fence_after();
      const uint4 info = lds128(base + y0.small + L::info + slot * 16);
      const uint32_t scales = base + y0.small + L::scales + slot * L::POS;
      const int Ft = static_cast<int>(info.x);
      const float k0 = __uint_as_float(info.z);
      const int seen = limit - (s.t0 + k) * kTile;  // positions of the tile that the row attends to
      const bool masked = nearest < (s.t0 + k + 1) * kTile || info.y != 0xFFu;
      // The loops over the tile's four pieces of 32 positions stay rolled: fully
      // unrolled, the roles' code does not fit the instruction caches, and
      // fetching it bounds the kernel.
      //
      // ---- t in place of S (masked: -inf), and the row's largest t 2^-eb
      float top = -INFINITY;
      auto largest = [&](auto tag) {
        constexpr bool MASK = decltype(tag)::value;
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll 1
        for (int cc = 0; cc < kTile / 32; ++cc) {
          uint32_t w[32];
          tmem_ld32(S + 32 * cc, w);
          tmem_wait_ld(w);
          if constexpr (SCALED) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const uint4 z = lds128(scales + 4 * (32 * cc + e));
              float a0, a1, a2, a3;
              mul_f32x2(__uint_as_float(w[e]), __uint_as_float(w[e + 1]), __uint_as_float(z.x), __uint_as_float(z.y), a0, a1);
              mul_f32x2(__uint_as_float(w[e + 2]), __uint_as_float(w[e + 3]), __uint_as_float(z.z), __uint_as_float(z.w), a2, a3);
              w[e] = __float_as_uint(a0);
              w[e + 1] = __float_as_uint(a1);
              w[e + 2] = __float_as_uint(a2);
              w[e + 3] = __float_as_uint(a3);
            }
          }
          if constexpr (MASK) {
            const uint32_t in = info.y >> (2 * cc);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * cc + e >= seen || !((in >> (e / kBlockSize)) & 1u)) w[e] = 0xFF800000u;
          }
          if constexpr (MASK || SCALED) tmem_st32(S + 32 * cc, w);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            t0 = max3(t0, __uint_as_float(w[e]), __uint_as_float(w[e + 1]));
            t1 = max3(t1, __uint_as_float(w[e + 2]), __uint_as_float(w[e + 3]));
          }
        }
        if constexpr (MASK || SCALED) tmem_wait_st();
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
      // ---- p = 2^(z - m + 8): plainly t c - RN(m c - 8) in one FMA; beyond
      // |m c| = 2^10 the rounding of m c would show in the exponent, so the
      // careful form takes (t - m) c + 8.  c 2^-eb underflows for tiny queries
      // against tiny scales, and a masked -inf times 0 would be NaN: there 2^-126
      // stands for it (|t| < 2^38, so all that z loses is below 2^-88).
      auto exponentials = [&](auto tag) {
        constexpr bool careful = decltype(tag)::value;
        const float ref = m == -INFINITY ? 0.f : m, mu = kBias - ref * c, ck = fmaxf(c * k0, 0x1p-126f);
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll 1
        for (int cc = 0; cc < kTile / 32; ++cc) {
          uint32_t w[32];
          tmem_ld32(S + 32 * cc, w);
          tmem_wait_ld(w);
          uint32_t P[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float a0 = __uint_as_float(w[e]), a1 = __uint_as_float(w[e + 1]), a2 = __uint_as_float(w[e + 2]),
                  a3 = __uint_as_float(w[e + 3]);
            if constexpr (careful) {
              a0 = (a0 * k0 - ref) * c + kBias;
              a1 = (a1 * k0 - ref) * c + kBias;
              a2 = (a2 * k0 - ref) * c + kBias;
              a3 = (a3 * k0 - ref) * c + kBias;
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
    if (begun) {
      wait(B_O + wg, no & 1);
      ++no;
    } else {
      // one tile for two warpgroups: the other one has it
      wait(B_O, seg & 1);
    }
    __syncwarp();
    tmem_fence_after();
    // Scores that are no numbers make l NaN and leave m alone: a state of any finite
    // m carries it through the merge.
    const float mz = l != l ? 0.f : m == -INFINITY ? m : m * c - kBias;
    // The scores' products are behind either B_O too, so Q is free to be written.
    store_partial<D>(a, s, smem + L::q, tmem + lanes + 256, wg, live, r, mz, l, F == kNoScale ? 0.f : pow2i(-F));
    tmem_fence_before();
    // no warpgroup goes on while the other one reads O, or Q's place
    if (!s.two) {
      asm volatile("bar.sync 1, 256;" ::: "memory");
      tmem_fence_after();
    }
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
  grid_wait();  // the plan
  grid_release();
  const int T = a.ws_groups[a.groups].tile0, P = a.ws_groups[a.groups].tiles, cta = blockIdx.x;
  if (cta >= P) return;
  // c T / P in 32 bits
  const int whole = T / P, rest = T - whole * P;
  const int x = cta * whole + cta * rest / P, x1 = (cta + 1) * whole + (cta + 1) * rest / P;

  uint32_t *const tm = reinterpret_cast<uint32_t *>(smem + y.small + L::tmem);
  Segment *const first = reinterpret_cast<Segment *>(smem + y.small + L::segment);
  if (warp == kLoadWarp) {
    // arrivals per phase: 4 for a warpgroup's warps, 8 for B_Q, 2 for B_META, else 1
    for (int i = threadIdx.x & 31; i < B_COUNT; i += 32) {
      const bool four = (i >= B_KFULL && i < B_KFULL + 2) || (i >= B_VFULL && i < B_VFULL + 2) || (i >= B_P && i < B_P + 2) ||
                        i >= B_EMPTY;
      const bool two = i >= B_META && i < B_META + 2;
      mbar_init(&bars[i], i == B_Q ? 8 : four ? 4 : two ? 2 : 1);
    }
    mbar_init_fence();
    if (threadIdx.x % 32 == 0) {
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&vmap);
      *reinterpret_cast<volatile uint32_t *>(tm + 1) = 0;
    }
  }
  if (threadIdx.x == 32 * kScaleWarp) {
    Segment s;
    find_segment(a, x, x1, &s);
    *first = s;
  }
  __syncwarp();
  if (warp == kMmaWarp) tmem_alloc(smem_u32(tm), 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tm);

  const Waiter wait = {bars, tm + 1, a.err};
  const Segments sg = {first, x};
  const int tiles = x1 - x;
  const bool chan = kf == K_INT8_CHAN || kf == K_INT2_CHAN, group = vf == V_INT4_G32 || vf == V_INT2_G32;
  if (warp == kLoadWarp || warp == kLoadVWarp) {
    const int r = warp == kLoadWarp ? 0 : 1;
    load_role(a, r ? &vmap : &kmap, r ? vrow : krow, r, base, y, wait, sg, x, x1);
  } else if (warp >= kSoftmaxWarp) {
    if (chan) softmax_role<D, false>(a, smem, y, wait, tmem, sg, x, x1);
    else softmax_role<D, true>(a, smem, y, wait, tmem, sg, x, x1);
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
    product_role<D>(a, base, wait, tmem, sg, x, x1);
  } else if (warp == kScaleWarp) {
    const int top = top_exponent(kf == K_FP8_TOK ? C_FP8 : C_INT8);
    if (kf == K_INT2_CHAN) scale_k_role<D, true, false>(a, base, y, wait, sg, top, x, x1);
    else if (chan) scale_k_role<D, true, true>(a, base, y, wait, sg, top, x, x1);
    else scale_k_role<D, false, true>(a, base, y, wait, sg, top, x, x1);
  } else {
    const int top = top_exponent(vf == V_FP8_TOK ? C_FP8 : C_INT8);
    if (vf == V_INT2_G32) scale_v_role<D, true, false>(a, base, y, wait, sg, top, x, x1);
    else if (group) scale_v_role<D, true, true>(a, base, y, wait, sg, top, x, x1);
    else scale_v_role<D, false, true>(a, base, y, wait, sg, top, x, x1);
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
