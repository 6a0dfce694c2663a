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
// Roles, one CTA per SM: two softmax warpgroups (thread = row), one
// warpgroup that turns codes into f16 tiles in shared memory, one warp that
// issues the products.  Steps alternate between the two softmax warpgroups, so
// the tensor core works for one while the other is in its exponentials:
//   more than 128 rows: warpgroup i owns rows 128 i .. + 127, each tile of
//     codes serves both (steps 2t, 2t + 1 of tile t);
//   at most 128 rows: both own the same rows, warpgroup i the tiles of parity
//     i; each keeps its own (m, l, O), merged later like any other partial.
// P overwrites S in tensor memory and is the A operand of the second product.
#pragma once

#include "paged_decode_impl.cuh"
#include "tcgen05.cuh"

namespace kvq {
namespace prefix {

constexpr int kTile = kPrefixTile;             // positions per tile
constexpr int kTileBlocks = kTile / kBlockSize;
constexpr int kThreads = 13 * 32;
constexpr int kMmaWarp = 12;
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

// Shared memory.  Tiles are [64-channel half][row][128 bytes], swizzled.
template <int D>
struct Smem {
  static constexpr uint32_t HALF = 128 * 128;           // 64 channels of 128 rows
  static constexpr uint32_t TILE = HALF * (D / 64);
  static constexpr uint32_t q = 0;                      // [2] row tiles
  static constexpr uint32_t k = q + 2 * TILE;           // [2] stages
  static constexpr uint32_t v = k + 2 * TILE;           // [2] stages
  static constexpr uint32_t ks = v + 2 * TILE;          // [kMeta][128] FP32
  static constexpr uint32_t vs = ks + kMeta * kTile * 4;
  static constexpr uint32_t chan = vs + kMeta * kTile * 4;   // [2][8][D] f16: channel scales, high and low parts
  static constexpr uint32_t grp = chan + 2 * kTileBlocks * D * 2;  // [128][D / 32] f16 pairs (high, low)
  static constexpr uint32_t info = grp + kTile * (D / 32) * 4;     // [kMeta] {F, block mask}
  static constexpr uint32_t red = info + kMeta * 8;     // [2][2][4] warp maxima
  static constexpr uint32_t bars = red + 16 * 4;        // mbarriers
  static constexpr uint32_t tmem = bars + 16 * 8;       // tensor memory address, then the abort flag
  static constexpr uint32_t bytes = tmem + 16;
};

enum Bar : int { B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_S = 8, B_P = 10, B_O = 12, B_Q = 14, B_END = 15 };

// The part of a unit that this CTA works on.
struct Segment {
  PrefixGroup g;
  int u, h, rb, t0, t1;
  bool two;          // two row tiles
};

__device__ __forceinline__ Segment segment_at(const PrefixArgs &a, int64_t x, int64_t x1) {
  int lo = 0, hi = a.groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.ws_groups[mid].tile0 <= x) lo = mid; else hi = mid;
  }
  Segment s;
  s.g = a.ws_groups[lo];
  const int64_t y = x - s.g.tile0;
  s.u = static_cast<int>(y / s.g.tiles);
  s.t0 = static_cast<int>(y - static_cast<int64_t>(s.u) * s.g.tiles);
  s.t1 = static_cast<int>(min(static_cast<int64_t>(s.g.tiles), s.t0 + (x1 - x)));
  s.h = s.u % a.H;
  s.rb = s.u / a.H;
  s.two = s.g.rows > kPrefixRows / 2;
  return s;
}

// Waits for a phase of an mbarrier.  When a wait runs out, the error is set and
// every later wait of the CTA returns at once: the roles run to their ends (all
// barriers between threads are met, all accesses stay in bounds), and the
// results are void.
struct Waiter {
  uint64_t *bars;
  volatile uint32_t *abort;
  unsigned int *err;
  __device__ __forceinline__ void operator()(int bar, uint32_t parity) const {
    if (mbar_try_wait(&bars[bar], parity)) return;
    const long long t0 = clock64();
    while (!mbar_try_wait(&bars[bar], parity)) {
      if (*abort) return;
      if (clock64() - t0 > kWaitTicks) {
        *abort = 1;
        set_error(err, KVQ_DEVERR_TIMEOUT);
        return;
      }
    }
  }
};

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---------------------------------------------------------------------------
// codes -> f16 tiles
// ---------------------------------------------------------------------------
// 8 consecutive channels out of 16 bytes of codes, in channel order.
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

// code * (h + l) in one rounding (but for the rounding of code * l).
__device__ __forceinline__ uint32_t scaled(uint32_t c, uint32_t h, uint32_t l) {
  return hfma2_u32(c, h, hmul2_u32(c, l));
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

template <int D, Code C>
__device__ __forceinline__ void load_codes(const Cover<D, C> &f, const uint8_t *codes, int H, int h, int ids,
                                           uint4 (&w)[Cover<D, C>::CH]) {
  using F = Cover<D, C>;
#pragma unroll
  for (int i = 0; i < F::CH; ++i) {
    const int key = f.k0 + F::STEP * i;
    const int id = __shfl_sync(0xffffffffu, ids, key / kBlockSize);
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (id >= 0)
      w[i] = __ldg(reinterpret_cast<const uint4 *>(
          codes + ((static_cast<int64_t>(id) * kBlockSize + key % kBlockSize) * H + h) * F::ROW + 16 * f.c));
  }
}

// Converts and stores; `scale(i, j, r)` applies scales to piece j (in the
// thread's order) of load i.
template <int D, Code C, typename Scale>
__device__ __forceinline__ void store_codes(const Cover<D, C> &f, uint32_t tile, uint4 (&w)[Cover<D, C>::CH],
                                            Scale scale) {
  using F = Cover<D, C>;
#pragma unroll
  for (int i = 0; i < F::CH; ++i) {
    uint4 x = w[i];
    if (f.swap) x = make_uint4(x.z, x.w, x.x, x.y);
    const uint32_t at = tile + f.row0 + i * F::STEP * 128;
    auto piece = [&](auto j) {
      constexpr int J = decltype(j)::value;
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

// Maximum over the converter warpgroup of non-negative floats.  Its barrier
// also keeps the scratch of one tile from being written before the last one's
// has been read; `red` alternates between two places.
__device__ __forceinline__ float group_max(float x, uint32_t red, int warp, int lane) {
  const uint32_t m = warp_max_u32(__float_as_uint(x));
  if (lane == 0) sts32(red + 4 * warp, m);
  bar_sync(1, 128);
  const uint4 v = lds128(red);
  return __uint_as_float(max(max(v.x, v.y), max(v.z, v.w)));
}

template <int D, int KF, int VF>
__device__ __noinline__ void convert_role(const PrefixArgs &a, uint8_t *smem, const Waiter &wait, int64_t x, int64_t x1) {
  using L = Smem<D>;
  using KC = KCode<KF>;
  using VC = VCode<VF>;
  constexpr int NG = D / 32;
  constexpr int NCS = kTileBlocks * D / 128;  // channel scales per thread
  const int tid = threadIdx.x - 256, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_u32(smem);
  const Cover<D, KC::code> fk(tid);
  const Cover<D, VC::code> fv(tid);

  uint4 kw[Cover<D, KC::code>::CH], vw[Cover<D, VC::code>::CH];
  float sk[KC::chan ? NCS : 1], sv[VC::group ? NG : 1];
  Segment s = segment_at(a, x, x1);
  int t = s.t0;

  // lane j < 8: the id of block j of the tile, -1 past the prefix or invalid
  auto ids_of = [&](const Segment &sg, int tile) {
    const int j = tile * kTileBlocks + (lane & 7);
    if (j >= sg.g.shared / kBlockSize) return -1;
    const int id = __ldg(a.tables + static_cast<int64_t>(sg.g.lead) * a.max_blocks + j);
    if (id >= 0 && id < a.num_blocks) return id;
    if (warp == 0 && lane < 8) set_error(a.err, KVQ_DEVERR_BLOCK_RANGE);
    return -1;
  };
  auto load_k = [&](int h, int ids) {
    load_codes<D, KC::code>(fk, a.kc, a.H, h, ids, kw);
    const int id = __shfl_sync(0xffffffffu, ids, tid >> 4);
    if constexpr (KC::chan) {
#pragma unroll
      for (int e = 0; e < NCS; ++e) sk[e] = 0.f;
      if (id >= 0) {
        const float4 *p = reinterpret_cast<const float4 *>(a.ks + (static_cast<int64_t>(id) * a.H + h) * D + (tid & 15) * NCS);
#pragma unroll
        for (int e = 0; e < NCS; e += 4) {
          const float4 y = __ldg(p + e / 4);
          sk[e] = y.x; sk[e + 1] = y.y; sk[e + 2] = y.z; sk[e + 3] = y.w;
        }
      }
    } else {
      sk[0] = id >= 0 ? __ldg(a.ks + (static_cast<int64_t>(id) * kBlockSize + (tid & 15)) * a.H + h) : 0.f;
    }
    // the V scales go with K: the tile's factors are complete when K is
    const int64_t tok = (static_cast<int64_t>(id) * kBlockSize + (tid & 15)) * a.H + h;
#pragma unroll
    for (int e = 0; e < (VC::group ? NG : 1); ++e) sv[e] = id >= 0 ? __ldg(a.vs + tok * (VC::group ? NG : 1) + e) : 0.f;
  };

  int ids = ids_of(s, t);
  load_k(s.h, ids);
  load_codes<D, VC::code>(fv, a.vc, a.H, s.h, ids, vw);
  int F = kNoScale;
  for (int n = 0; x < x1; ++n) {
    // the next tile, in this unit or the next one
    Segment nx = s;
    int nt = t + 1, nids = -1;
    if (x + 1 < x1) {
      if (nt == s.t1) {
        nx = segment_at(a, x + 1, x1);
        nt = nx.t0;
      }
      nids = ids_of(nx, nt);
    }
    if (t == s.t0) F = kNoScale;
    const int st = n & 1, slot = n % kMeta;
    const uint32_t ph = ((n >> 1) & 1) ^ 1;
    // ---- K and the tile's factors
    wait(B_KEMPTY + st, ph);
    float kmax = 0.f, vmax = 0.f;
    if constexpr (KC::chan)
#pragma unroll
      for (int e = 0; e < NCS; ++e) kmax = fmaxf(kmax, sk[e]);
#pragma unroll
    for (int e = 0; e < (VC::group ? NG : 1); ++e) vmax = fmaxf(vmax, sv[e]);
    if constexpr (KC::chan) kmax = group_max(kmax, base + L::red + 32 * (n & 1), warp, lane);
    vmax = group_max(vmax, base + L::red + 32 * (n & 1) + 16, warp, lane);
    // F: the tile's largest V scale times 2^F below 2^9, set to [2^7, 2^8)
    if (vmax > 0.f && (F == kNoScale || ilog2f(vmax) + F >= kTopV)) F = min(kTopV - 2 - ilog2f(vmax), kMaxVExp);
    const float pf = F == kNoScale ? 1.f : pow2i(F);
    if constexpr (KC::chan) {
      const int eb = kmax > 0.f ? min(7 - ilog2f(kmax), kMaxVExp) : 0;
      const float f = pow2i(eb);
      sts32(base + L::ks + (slot * kTile + tid) * 4, __float_as_uint(pow2i(-eb)));
      uint32_t hi[NCS / 2], lo[NCS / 2];
#pragma unroll
      for (int e = 0; e < NCS; e += 2) split_f16x2(sk[e] * f, sk[e + 1] * f, hi[e / 2], lo[e / 2]);
      const uint32_t p = base + L::chan + tid * NCS * 2;
      if constexpr (NCS == 8) {
        sts128(p, hi[0], hi[1], hi[2], hi[3]);
        sts128(p + kTileBlocks * D * 2, lo[0], lo[1], lo[2], lo[3]);
      } else {
        sts64(p, hi[0], hi[1]);
        sts64(p + kTileBlocks * D * 2, lo[0], lo[1]);
      }
    } else {
      sts32(base + L::ks + (slot * kTile + tid) * 4, __float_as_uint(sk[0]));
    }
    sts32(base + L::vs + (slot * kTile + tid) * 4, __float_as_uint(VC::group ? 1.f : sv[0] * pf));
    if constexpr (VC::group) {
#pragma unroll
      for (int e = 0; e < NG; ++e) {
        const float y = sv[e] * pf;
        uint32_t hi, lo;
        split_f16x2(y, y, hi, lo);
        sts32(base + L::grp + (tid * NG + e) * 4, prmt(hi, lo, 0x5410u));
      }
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, ids >= 0) & 0xFFu;
    if (tid == 0) sts64(base + L::info + slot * 8, static_cast<uint32_t>(F), mask);
    if constexpr (KC::chan || VC::group) bar_sync(1, 128);
    store_codes<D, KC::code>(fk, base + L::k + st * L::TILE, kw, [&](int i, int j, uint4 &r) {
      if constexpr (KC::chan) {
        const int blk = (fk.k0 + Cover<D, KC::code>::STEP * i) / kBlockSize;
        const int piece = fk.c * Cover<D, KC::code>::NP + (fk.swap ? j ^ (Cover<D, KC::code>::NP / 2) : j);
        const uint32_t p = base + L::chan + (blk * D + 8 * piece) * 2;
        const uint4 hi = lds128(p), lo = lds128(p + kTileBlocks * D * 2);
        r.x = scaled(r.x, hi.x, lo.x);
        r.y = scaled(r.y, hi.y, lo.y);
        r.z = scaled(r.z, hi.z, lo.z);
        r.w = scaled(r.w, hi.w, lo.w);
      }
    });
    fence_proxy_async_shared();
    mbar_arrive(&wait.bars[B_KFULL + st]);
    if (x + 1 < x1) load_k(nx.h, nids);
    // ---- V
    wait(B_VEMPTY + st, ph);
    store_codes<D, VC::code>(fv, base + L::v + st * L::TILE, vw, [&](int i, int j, uint4 &r) {
      if constexpr (VC::group) {
        const int key = fv.k0 + Cover<D, VC::code>::STEP * i;
        const int piece = fv.c * Cover<D, VC::code>::NP + (fv.swap ? j ^ (Cover<D, VC::code>::NP / 2) : j);
        const uint32_t y = lds32(base + L::grp + (key * NG + piece / 4) * 4);
        const uint32_t hi = prmt(y, 0u, 0x1010u), lo = prmt(y, 0u, 0x3232u);
        r.x = scaled(r.x, hi, lo);
        r.y = scaled(r.y, hi, lo);
        r.z = scaled(r.z, hi, lo);
        r.w = scaled(r.w, hi, lo);
      }
    });
    fence_proxy_async_shared();
    mbar_arrive(&wait.bars[B_VFULL + st]);
    if (x + 1 < x1) load_codes<D, VC::code>(fv, a.vc, a.H, nx.h, nids, vw);
    s = nx;
    t = nt;
    ids = nids;
    ++x;
  }
}

// ---------------------------------------------------------------------------
// the products
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void product_role(const PrefixArgs &a, uint8_t *smem, const Waiter &wait, uint32_t tmem, int64_t x,
                                             int64_t x1) {
  using L = Smem<D>;
  const uint32_t base = smem_u32(smem);
  constexpr uint32_t id_s = mma_idesc_f16(128, kTile, false), id_o = mma_idesc_f16(128, D, true);
  int nk = 0, nv = 0;          // tiles consumed so far, by S and by O
  uint32_t np[2] = {0, 0};     // steps of each warpgroup so far
  for (int seg = 0; x < x1; ++seg) {
    const Segment s = segment_at(a, x, x1);
    const int tiles = s.t1 - s.t0, steps = s.two ? 2 * tiles : tiles;
    wait(B_Q, seg & 1);
    tmem_fence_after();
    auto scores = [&](int j) {
      const int i = j & 1, st = nk & 1;
      if (!s.two || i == 0) wait(B_KFULL + st, (nk >> 1) & 1);
      tmem_fence_after();
      const uint32_t q = base + L::q + (s.two ? i : 0) * L::TILE, k = base + L::k + st * L::TILE;
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        const uint32_t off = (e / 4) * L::HALF + (e % 4) * 32;
        mma_f16_ss(tmem + 128 * i, mma_desc(q + off, 16, 1024), mma_desc(k + off, 16, 1024), id_s, e > 0);
      }
      mma_commit(&wait.bars[B_S + i]);
      if (!s.two || i == 1) {
        mma_commit(&wait.bars[B_KEMPTY + st]);
        ++nk;
      }
    };
    scores(0);
    if (steps > 1) scores(1);
    for (int j = 0; j < steps; ++j) {
      const int i = j & 1, st = nv & 1;
      wait(B_P + i, np[i] & 1);
      ++np[i];
      if (!s.two || i == 0) wait(B_VFULL + st, (nv >> 1) & 1);
      tmem_fence_after();
      const uint32_t v = base + L::v + st * L::TILE;
#pragma unroll
      for (int e = 0; e < kTile / 16; ++e)
        mma_f16_ts(tmem + 256 + 128 * i, tmem + 128 * i + 8 * e, mma_desc(v + e * 2048, L::HALF, 1024), id_o,
                   j >= 2 || e > 0);
      if (!s.two || i == 1) {
        mma_commit(&wait.bars[B_VEMPTY + st]);
        ++nv;
      }
      if (j + 2 < steps) scores(j + 2);
      else mma_commit(&wait.bars[B_O + i]);
    }
    x += tiles;
  }
  // nothing in flight when tensor memory is given back
  mma_commit(&wait.bars[B_END]);
  wait(B_END, 0);
}

// ---------------------------------------------------------------------------
// softmax
// ---------------------------------------------------------------------------
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// The warp's 32 rows of Q' into their tile; returns this lane's row factor c.
template <int D>
__device__ __forceinline__ float stage_queries(const PrefixArgs &a, const Segment &s, uint32_t tile, int row0, int lane,
                                               bool store) {
  constexpr int CPL = D / 32;  // channels per lane
  const int R = s.g.nseq * a.G;
  float c = 0.f;
  constexpr int U = 8;
  for (int r0 = 0; r0 < 32; r0 += U) {
    uint32_t w[U][CPL / 2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row0 + r0 + u, row = s.rb * s.g.rows + r;
#pragma unroll
      for (int e = 0; e < CPL / 2; ++e) w[u][e] = 0u;
      if (r < s.g.rows && row < R) {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(
            a.q + (static_cast<int64_t>(s.g.start + row / a.G) * a.Hq + s.h * a.G + row % a.G) * D + lane * CPL);
#pragma unroll
        for (int e = 0; e < CPL / 2; ++e) w[u][e] = __ldg(p + e);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[CPL];
#pragma unroll
      for (int e = 0; e < CPL / 2; ++e) {
        y[2 * e] = bf16lo_to_f32(w[u][e]);
        y[2 * e + 1] = bf16hi_to_f32(w[u][e]);
      }
      if (a.rot) {
        // H (sigma q): stages below CPL inside the lane, the others across
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
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < CPL; ++e) m = fmaxf(m, fabsf(y[e]));
      m = __uint_as_float(warp_max_u32(__float_as_uint(m)));
      // below 2^-86 the scores vanish anyway: er <= 100 keeps c a normal float
      const int er = m > 0.f ? min(14 - ilog2f(m), 100) : 0;
      if (lane == r0 + u) c = scale_pow2(rsqrtf(static_cast<float>(D)) * kLog2e, -(er + (a.rot ? (D == 128 ? 7 : 6) : 0)));
      uint32_t f[CPL / 2];
#pragma unroll
      for (int e = 0; e < CPL / 2; ++e) f[e] = f32x2_to_f16x2(scale_pow2(y[2 * e], er), scale_pow2(y[2 * e + 1], er));
      const int rr = row0 % 128 + r0 + u, ch = lane * CPL;
      const uint32_t at = tile + (ch >> 6) * Smem<D>::HALF + rr * 128 + ((((ch & 63) >> 3) ^ (rr & 7)) << 4) + (ch & 7) * 2;
      if (store) {
        if constexpr (CPL == 4) sts64(at, f[0], f[1]);
        else sts32(at, f[0]);
      }
    }
  }
  return c;
}

template <int D>
__device__ __forceinline__ void softmax_role(const PrefixArgs &a, uint8_t *smem, const Waiter &wait, uint32_t tmem, int64_t x,
                                             int64_t x1) {
  using L = Smem<D>;
  const uint32_t base = smem_u32(smem);
  const int wg = threadIdx.x >> 7, warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
  const uint32_t S = tmem + lanes + 128 * wg, O = tmem + lanes + 256 + 128 * wg;
  int n0 = 0;                  // tiles of earlier segments
  uint32_t ns = 0, no = 0;     // steps and segments of this warpgroup so far
  for (int seg = 0; x < x1; ++seg) {
    const Segment s = segment_at(a, x, x1);
    const int tiles = s.t1 - s.t0, R = s.g.nseq * a.G;
    const int r0 = s.two ? 128 * wg : 0, r = r0 + 32 * warp + lane, row = s.rb * s.g.rows + r;
    const bool live = r < s.g.rows && row < R;
    // ---- queries
    const float c = stage_queries<D>(a, s, base + L::q + (s.two ? wg : 0) * L::TILE, r0 + 32 * warp, lane, s.two || wg == 0);
    fence_proxy_async_shared();
    mbar_arrive(&wait.bars[B_Q]);
    const int limit = live ? __ldg(a.ws_limit + s.g.start + row / a.G) : s.g.shared;
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
      const uint2 info = lds64(base + L::info + slot * 8);
      const int Ft = static_cast<int>(info.x);
      const uint32_t ks = base + L::ks + slot * kTile * 4, vs = base + L::vs + slot * kTile * 4;
      const int seen = limit - (s.t0 + k) * kTile;  // positions of the tile that the row attends to
      // The plain pass forms z - m as t c - RN(m c) in one FMA.  The careful one
      // masks and forms (t - m) c: beyond |m c| = 2^10 the rounding of m c
      // would show in the exponent (below, it is at most 2^-15).
      const bool masked = nearest < (s.t0 + k + 1) * kTile || info.y != 0xFFu;
      uint32_t P[kTile / 2];
      float top, sum;
      auto pass = [&](auto tag) {
        constexpr bool MASK = decltype(tag)::value;
        const float ref = m == -INFINITY ? 0.f : m, mu = -ref * c;
        float t0 = -INFINITY, t1 = -INFINITY, s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
        uint32_t w[16];
        tmem_ld16(S, w);
#pragma unroll
        for (int cc = 0; cc < kTile / 16; ++cc) {
          float y[16];
          tmem_wait_ld(w);
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = __uint_as_float(w[e]);
          if (cc + 1 < kTile / 16) tmem_ld16(S + 16 * (cc + 1), w);
          const bool gone = MASK && !((info.y >> cc) & 1u);
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const uint4 kf = lds128(ks + (16 * cc + e) * 4), vf = lds128(vs + (16 * cc + e) * 4);
            float a0, a1, a2, a3;
            mul_f32x2(y[e], y[e + 1], __uint_as_float(kf.x), __uint_as_float(kf.y), a0, a1);
            mul_f32x2(y[e + 2], y[e + 3], __uint_as_float(kf.z), __uint_as_float(kf.w), a2, a3);
            if constexpr (MASK) {
              const int p = 16 * cc + e;
              a0 = gone || p >= seen ? -INFINITY : a0;
              a1 = gone || p + 1 >= seen ? -INFINITY : a1;
              a2 = gone || p + 2 >= seen ? -INFINITY : a2;
              a3 = gone || p + 3 >= seen ? -INFINITY : a3;
            }
            t0 = max3(t0, a0, a1);
            t1 = max3(t1, a2, a3);
            if constexpr (MASK) {
              sub_f32x2(a0, a1, ref, ref, a0, a1);
              sub_f32x2(a2, a3, ref, ref, a2, a3);
              mul_f32x2(a0, a1, c, c, a0, a1);
              mul_f32x2(a2, a3, c, c, a2, a3);
            } else {
              fma_f32x2(a0, a1, c, c, mu, mu, a0, a1);
              fma_f32x2(a2, a3, c, c, mu, mu, a2, a3);
            }
            a0 = fast_exp2(a0);
            a1 = fast_exp2(a1);
            a2 = fast_exp2(a2);
            a3 = fast_exp2(a3);
            add_f32x2(s0, s1, a0, a1, s0, s1);
            add_f32x2(s2, s3, a2, a3, s2, s3);
            mul_f32x2(a0, a1, __uint_as_float(vf.x), __uint_as_float(vf.y), a0, a1);
            mul_f32x2(a2, a3, __uint_as_float(vf.z), __uint_as_float(vf.w), a2, a3);
            P[8 * cc + e / 2] = f32x2_to_f16x2(a0, a1);
            P[8 * cc + e / 2 + 1] = f32x2_to_f16x2(a2, a3);
          }
        }
        top = fmaxf(t0, t1);
        sum = (s0 + s1) + (s2 + s3);
      };
      // with the old m first: it is rarely raised after the first tiles
      if (masked || huge) pass(std::true_type{}); else pass(std::false_type{});
      const bool raise = top != -INFINITY && (m == -INFINITY || (top - m) * c > kRaise);
      if (__any_sync(0xffffffffu, raise) || Ft != F) {
        const float mn = fmaxf(m, top);
        const float keep = m == -INFINITY ? 0.f : fast_exp2((m - mn) * c);
        const bool again = __any_sync(0xffffffffu, mn != m);
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
        if (again) {
          huge = __any_sync(0xffffffffu, m != -INFINITY && fabsf(m * c) > 0x1p10f);
          if (masked || huge) pass(std::true_type{}); else pass(std::false_type{});
        }
      }
      l += sum;
      begun = true;
#pragma unroll
      for (int cc = 0; cc < kTile / 32; ++cc) tmem_st16(S + 16 * cc, P + 16 * cc);
      tmem_wait_st();
      tmem_fence_before();
      mbar_arrive(&wait.bars[B_P + wg]);
    }
    // ---- the unit's partial state
    const int64_t at = s.g.row0 + static_cast<int64_t>(s.u) * s.g.slots + static_cast<int64_t>(blockIdx.x) * kPrefixRows +
                       (s.two ? r : wg * s.g.rows + r);
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
          float4 *o = reinterpret_cast<float4 *>(a.ws_o + at * D + 16 * cc);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = make_float4(__uint_as_float(w[4 * e]) * back, __uint_as_float(w[4 * e + 1]) * back,
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
    if (live) *reinterpret_cast<float2 *>(a.ws_ml + at * 2) = make_float2(m == -INFINITY ? m : m * c, l);
    x += tiles;
    n0 += tiles;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefix_attend_kernel(const __grid_constant__ PrefixArgs a, const int kf,
                                                                    const int vf) {
  extern __shared__ __align__(1024) uint8_t raw[];
  using L = Smem<D>;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::bars);
  const int warp = threadIdx.x >> 5;
  const int64_t T = a.ws_groups[a.groups].tile0;
  const int P = a.ws_groups[a.groups].tiles, cta = blockIdx.x;
  if (cta >= P) return;
  const int64_t x = cta * T / P, x1 = (cta + 1) * T / P;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[B_KFULL + i], 128);
      mbar_init(&bars[B_KEMPTY + i], 1);
      mbar_init(&bars[B_VFULL + i], 128);
      mbar_init(&bars[B_VEMPTY + i], 1);
      mbar_init(&bars[B_S + i], 1);
      mbar_init(&bars[B_P + i], 128);
      mbar_init(&bars[B_O + i], 1);
    }
    mbar_init(&bars[B_Q], 256);
    mbar_init(&bars[B_END], 1);
    mbar_init_fence();
  }
  if (threadIdx.x == 32) *reinterpret_cast<volatile uint32_t *>(smem + L::tmem + 4) = 0;
  if (warp == kMmaWarp) tmem_alloc(smem_u32(smem + L::tmem), 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::tmem);

  const Waiter wait = {bars, reinterpret_cast<volatile uint32_t *>(smem + L::tmem + 4), a.err};
  if (warp < 8) {
    softmax_role<D>(a, smem, wait, tmem, x, x1);
  } else if (warp < kMmaWarp) {
    switch (kf * 4 + vf) {
#define KVQ_CASE(K, V) \
  case K * 4 + V: convert_role<D, K, V>(a, smem, wait, x, x1); break;
#define KVQ_CASES(K) KVQ_CASE(K, V_INT8_TOK) KVQ_CASE(K, V_FP8_TOK) KVQ_CASE(K, V_INT4_G32)
      KVQ_CASES(K_INT8_TOK)
      KVQ_CASES(K_FP8_TOK)
      KVQ_CASES(K_INT8_CHAN)
      KVQ_CASES(K_INT4_TOK)
      default:
        if constexpr (D == 128) {  // INT2 rows: head_dim 128
          switch (kf * 4 + vf) {
            KVQ_CASE(K_INT8_TOK, V_INT2_G32)
            KVQ_CASE(K_FP8_TOK, V_INT2_G32)
            KVQ_CASE(K_INT8_CHAN, V_INT2_G32)
            KVQ_CASE(K_INT4_TOK, V_INT2_G32)
            KVQ_CASES(K_INT2_CHAN)
            KVQ_CASE(K_INT2_CHAN, V_INT2_G32)
          }
        }
#undef KVQ_CASES
#undef KVQ_CASE
    }
  } else if ((threadIdx.x & 31) == 0) {
    product_role<D>(a, smem, wait, tmem, x, x1);
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
