// Eviction of the cached tokens with the least accumulated attention weight.
//
// What it computes, for every row and kv head: of n cached tokens k stay, namely
// the first p (attention sinks, a shared prompt), the last w, and the k - w - p
// heaviest of the others (ties: the lower position).  Kept tokens below k - w
// stay where they are; those in [k - w, n - w) move, in order, to the places
// that evicted tokens leave in [p, k - w); the last w become [k - w, k).  The
// cache is read by softmax sums over all positions, so the order of the older
// tokens does not matter, and moving only what has to move is the least
// traffic; the last w keep their order, so that the next eviction finds them.
// Codes and scales move byte for byte ("PidokuInfra 12 KV Cache Quantization",
// §5 Where the scales live: a scale for each token and head), so a head's token
// keeps its values.  The pages have no eviction: it is this library's.
//
// Three kernels, since a place may be written only when what lies there has been
// read: selection, the moves of the older tokens (into places that evicted ones
// left), the shift of the last w (into places that moved ones left).  One kernel that
// did all three for a (row, head) in turn took 298, 132 and 124 us where these take
// 241, 110 and 65 (the three cases below): its passes wait for one another's latency
// with the whole SM.
// 27 x 8 heads, 32768 tokens to 16384 (FP8): select 35 us, move 179, shift 17.  The
// moves are of 256 bytes a token in two places, its scales and its weight 4 bytes each
// in sectors of 32: 352 bytes of traffic for 268, near the memory's rate.
// 256 x 8 heads, ~4160 tokens to 4096 (INT8), the last 256 shifted: 35, 10 and 53 us
// (the shift's bytes alone: 42).  8 x 8 heads, 65536 to 8192 (INT4): 24, 27 and 9; of
// the moves' 27 the sectors alone take ~15, of the shift's 9 the bytes 2.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

// Weights as unsigned numbers in the same order; -0 counts as 0, NaN as the
// largest (adding 0 leaves one NaN, 0x7FFFFFFF).  None is 0, which stands for a
// position that is no candidate.
__device__ __forceinline__ unsigned order_of(float x) {
  const unsigned b = __float_as_uint(x + 0.f);
  return b ^ (static_cast<unsigned>(static_cast<int>(b) >> 31) | 0x80000000u);
}

// ---------------------------------------------------------------------------
// which tokens stay
// ---------------------------------------------------------------------------
// One cluster of CTAs per (row, kv head), each with an even part of the
// candidates, each warp with an even part of that: the threshold by three passes
// over their weights (11, 11 and 10 bits, from the top; the CTAs add up their
// histograms), then what every warp has of larger and equal ones, then the lists
// of places and of tokens to go there.  The weights are read from memory once (the
// keys stay in shared memory); after that it is latency: of ~45000 cycles (32768
// tokens a head, clusters of two) the reading pass takes 9000, a search of a
// histogram 3000 to 3800 (three), the other two counts 3000 each, the lists 8500.
constexpr int kBins = 2048;
constexpr int kHeld = 16384;  // keys that 512 threads hold at most: 64 KB, three CTAs an SM (1024: twice that)

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned x;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(x));
  return x;
}
template <bool CLUSTER>
__device__ __forceinline__ void sync_all() {
  if constexpr (CLUSTER) {
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
}
// Shared memory of CTA `rank` of the cluster, at this CTA's address `at`.
__device__ __forceinline__ uint4 remote128(uint32_t at, unsigned rank) {
  uint32_t to;
  uint4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(to));
  return v;
}

// hist[k >> SHIFT & (2^BITS - 1)] += 1 if (k & mask) == want (SHIFT 21: if k is not
// 0), without a branch; `base` is the address of hist.
template <int SHIFT, int BITS>
__device__ __forceinline__ void count_key(uint32_t base, unsigned k, unsigned mask, unsigned want) {
  constexpr unsigned DIGIT = ((1u << BITS) - 1u) << 2;
  const uint32_t at = ((SHIFT >= 2 ? k >> (SHIFT - 2) : k << (2 - SHIFT)) & DIGIT) + base;
  if constexpr (SHIFT == 21)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t@p red.shared.add.u32 [%0], 1;\n\t}" ::"r"(at), "r"(k) : "memory");
  else
    asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %1, %2;\n\t@p red.shared.add.u32 [%0], 1;\n\t}" ::"r"(at), "r"(k & mask),
                 "r"(want)
                 : "memory");
}

// A lane has bits of four consecutive positions, the warp of 128: the number set
// before this lane's.
__device__ __forceinline__ unsigned lanes_before(unsigned bits) {
  unsigned below, n = 0;
  asm("mov.u32 %0, %%lanemask_lt;" : "=r"(below));
#pragma unroll
  for (int e = 0; e < 4; ++e) n += __popc(__ballot_sync(0xffffffffu, bits >> e & 1u) & below);
  return n;
}

// What a warp or a CTA has: larger and equal keys below `end`, and from there on.
struct Counts {
  unsigned larger_low, equal_low, larger, equal;
};

// HELD: the keys stay in shared memory; else each pass makes them from the weights
// again (in L2 after the first).  CLUSTER: more than one CTA.
template <int T, bool HELD, bool CLUSTER>
__global__ void __launch_bounds__(T, 1536 / T) evict_select_kernel(const EvictArgs a, const int ctas) {
  constexpr int W = T / 32;
  extern __shared__ uint4 held[];
  __shared__ __align__(16) unsigned hist[kBins];
  __shared__ unsigned sums[W];
  __shared__ __align__(16) Counts counts[W + 1];  // the warps', and the CTA's
  __shared__ unsigned chosen, left;
  const int x = CLUSTER ? blockIdx.x / ctas : blockIdx.x, rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
  const int r = x / a.H, h = x - r * a.H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool reports = tid == 0 && rank == 0;
  const int n = __ldg(a.ctx + r), keep = __ldg(a.keep + r), recent = __ldg(a.recent + r);
  const int pinned = a.pinned != nullptr ? __ldg(a.pinned + r) : 0;
  EvictMeta *meta = a.ws_meta + x;
  const bool range = n < 0 || n > a.max_len || keep < 0 || recent < 0 || pinned < 0;
  if (range || n <= keep) {  // (the same for all CTAs of a cluster, as below)
    if (reports) *meta = {0, 0, 0, 0};
    if (reports && range) set_error(a.err, KVQ_DEVERR_CONTEXT_RANGE);
    if (reports && h == 0) a.kept[r] = n;
    return;
  }
  const int w = min(recent, keep), p = min(pinned, keep - w), end = keep - w;
  const float *weights = a.weights + static_cast<int64_t>(x) * a.stride;
  const int last = n - w;  // candidates are [p, last)
  // Vectors of four weights on 16-byte boundaries: vector v holds the positions
  // 4 v - skew .. + 3; those outside the candidates are masked.
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(weights) >> 2) & 3);
  const int all0 = (p + skew) / 4, all1 = (last + skew + 3) / 4, part = (all1 - all0 + ctas - 1) / ctas;
  const int v0 = min(all1, all0 + rank * part), v1 = min(all1, v0 + part);
  const int share = ((v1 - v0 + W - 1) / W + 31) / 32 * 32;  // whole rounds of a warp
  const int w0 = min(v1, v0 + warp * share), w1 = min(v1, w0 + share);
  auto load = [&](int v) {
    const int i = 4 * v - skew;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i >= p && i + 4 <= last) {
      y = *reinterpret_cast<const float4 *>(weights + i);
    } else {
      if (i >= p && i < last) y.x = weights[i];
      if (i + 1 >= p && i + 1 < last) y.y = weights[i + 1];
      if (i + 2 >= p && i + 2 < last) y.z = weights[i + 2];
      if (i + 3 >= p && i + 3 < last) y.w = weights[i + 3];
    }
    return y;
  };
  auto keys_of = [&](int v, const float4 &y) {
    const int i = 4 * v - skew;
    uint4 k = make_uint4(order_of(y.x), order_of(y.y), order_of(y.z), order_of(y.w));
    if (i < p || i + 4 > last) {
      if (i < p || i >= last) k.x = 0u;
      if (i + 1 < p || i + 1 >= last) k.y = 0u;
      if (i + 2 < p || i + 2 >= last) k.z = 0u;
      if (i + 3 < p || i + 3 >= last) k.w = 0u;
    }
    return k;
  };
  // f(vector, its keys) for this warp's vectors in rounds of 32, four of a lane
  // in flight; lanes past the end have keys 0
  constexpr int U = 4;
  auto each = [&](auto from, auto f) {
#pragma unroll 1
    for (int v = w0; v < w1; v += 32 * U) {
      uint4 k[U];
      from(v, k);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v + 32 * u < w1) f(v + 32 * u + lane, k[u]);
    }
  };
  auto of_weights = [&](int v, uint4(&k)[U]) {
    float4 y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) y[u] = v + 32 * u + lane < w1 ? load(v + 32 * u + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < U; ++u)
      k[u] = v + 32 * u + lane < w1 ? keys_of(v + 32 * u + lane, y[u]) : make_uint4(0u, 0u, 0u, 0u);
  };
  auto of_held = [&](int v, uint4(&k)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      k[u] = v + 32 * u + lane < w1 ? held[v + 32 * u + lane - v0] : make_uint4(0u, 0u, 0u, 0u);
  };
  auto walk = [&](auto f) {
    if constexpr (HELD) each(of_held, f);
    else each(of_weights, f);
  };
  for (int i = tid; i < kBins; i += T) hist[i] = 0;
  // every block of the row, and nobody else's among those to be written (none where
  // all that stays is pinned)
  const int written = p < keep ? keep : 0;
  const int32_t *table = a.tables + static_cast<int64_t>(r) * a.max_blocks;
  bool bad = false, shared = false;
  // (eight of a thread in flight: one by one they took longer than the passes below)
  constexpr int C = 8;
  const int blocks = (n + kBlockSize - 1) / kBlockSize;
#pragma unroll 1
  for (int base = tid; base < blocks; base += C * T) {
    int id[C];
#pragma unroll
    for (int c = 0; c < C; ++c) id[c] = base + c * T < blocks ? __ldg(table + base + c * T) : 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = base + c * T;
      if (i >= blocks) break;
      if (id[c] < 0 || id[c] >= a.num_blocks) bad = true;
      else if (a.refs != nullptr && i >= p / kBlockSize && i * kBlockSize < written) shared = shared || __ldg(a.refs + id[c]) != 1;
    }
  }
  bad = __syncthreads_or(bad);
  shared = __syncthreads_or(shared);
  if (bad || shared) {
    if (reports) *meta = {0, 0, 0, 0};
    if (reports) set_error(a.err, bad ? KVQ_DEVERR_BLOCK_RANGE : KVQ_DEVERR_POOL_STATE);
    if (reports && h == 0) a.kept[r] = n;
    return;
  }
  if (reports && h == 0) a.kept[r] = keep;
  if (end == p) {  // none of the candidates stays: no places between what stays anyway
    if (reports) *meta = {0, 1, keep, w};
    return;
  }
  // ---- the need-th largest key, and how many of its equals are kept
  unsigned prefix = 0, need = end - p;
  {
    unsigned mask = 0;
    const uint32_t bins = smem_u32(hist);
    auto digit = [&](auto shift_tag, auto bits_tag) {
      constexpr int SHIFT = decltype(shift_tag)::value, BITS = decltype(bits_tag)::value;
      auto count = [&](const uint4 &k) {
        count_key<SHIFT, BITS>(bins, k.x, mask, prefix);
        count_key<SHIFT, BITS>(bins, k.y, mask, prefix);
        count_key<SHIFT, BITS>(bins, k.z, mask, prefix);
        count_key<SHIFT, BITS>(bins, k.w, mask, prefix);
      };
      if constexpr (SHIFT == 21) {
        each(of_weights, [&](int v, const uint4 &k) {
          if constexpr (HELD)
            if (v < w1) held[v - v0] = k;
          count(k);
        });
      } else {
        walk([&](int, const uint4 &k) { count(k); });
      }
      sync_all<CLUSTER>();
      // digits from the largest: the one in which the need-th lies
      constexpr int SEARCH = T < 512 ? T : 512, PER = kBins / SEARCH;  // (by the first 512 threads)
      static_assert(PER % 4 == 0, "whole vectors of bins");
      const int b0 = kBins - (tid + 1) * PER;
      unsigned bin[PER], own = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k) bin[k] = 0;
      for (int j = 0; j < (tid < SEARCH ? CLUSTER ? ctas : 1 : 0); ++j)
#pragma unroll
        for (int k = 0; k < PER; k += 4) {
          const uint4 y = CLUSTER ? remote128(smem_u32(hist + b0 + k), j) : *reinterpret_cast<const uint4 *>(hist + b0 + k);
          bin[k] += y.x;
          bin[k + 1] += y.y;
          bin[k + 2] += y.z;
          bin[k + 3] += y.w;
        }
#pragma unroll
      for (int k = 0; k < PER; ++k) own += bin[k];
      unsigned before = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      if (lane == 31) sums[warp] = before;
      __syncthreads();
      before += __reduce_add_sync(0xffffffffu, lane < warp ? sums[min(lane, W - 1)] : 0u) - own;
      if (before < need && need <= before + own) {
        bool found = false;
#pragma unroll
        for (int k = PER - 1; k >= 0; --k) {
          if (!found && before + bin[k] >= need) {
            found = true;
            chosen = b0 + k;
            left = need - before;
          }
          before += bin[k];
        }
      }
      sync_all<CLUSTER>();  // (and all CTAs have read the histograms)
      prefix |= chosen << SHIFT;
      mask |= ((1u << BITS) - 1u) << SHIFT;
      need = left;
      if constexpr (SHIFT > 0) {
        for (int i = tid; i < kBins; i += T) hist[i] = 0;
        __syncthreads();
      }
    };
    digit(std::integral_constant<int, 21>{}, std::integral_constant<int, 11>{});
    digit(std::integral_constant<int, 10>{}, std::integral_constant<int, 11>{});
    digit(std::integral_constant<int, 0>{}, std::integral_constant<int, 10>{});
  }
  // ---- what the warps before this one have
  Counts own = {0u, 0u, 0u, 0u};
  walk([&](int v, const uint4 &k) {
    const int low = end - (4 * v - skew);  // of the vector, below `end`
    if (low >= 4 || low <= 0) {
      const unsigned g = (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix),
                     q = (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
      if (low > 0) {
        own.larger_low += g;
        own.equal_low += q;
      } else {
        own.larger += g;
        own.equal += q;
      }
    } else {
      const unsigned key[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (key[e] > prefix) (e < low ? own.larger_low : own.larger) += 1u;
        if (key[e] == prefix) (e < low ? own.equal_low : own.equal) += 1u;
      }
    }
  });
  own.larger_low = __reduce_add_sync(0xffffffffu, own.larger_low);
  own.equal_low = __reduce_add_sync(0xffffffffu, own.equal_low);
  own.larger = __reduce_add_sync(0xffffffffu, own.larger);
  own.equal = __reduce_add_sync(0xffffffffu, own.equal);
  if (lane == 0) counts[warp] = own;
  __syncthreads();
  unsigned ties = 0;        // equals before this warp,
  int holes = 0, late = 0;  // places and tokens
  // takes one more part, the vectors [from, to)
  auto pass = [&](const Counts &c, int from, int to) {
    const unsigned stay = min(ties < need ? need - ties : 0u, c.equal_low + c.equal), low = min(stay, c.equal_low);
    holes += max(0, min(end, 4 * to - skew) - max(p, 4 * from - skew)) - static_cast<int>(c.larger_low + low);
    late += static_cast<int>(c.larger + stay - low);
    ties += c.equal_low + c.equal;
  };
  if constexpr (CLUSTER) {
    if (tid < 4) {
      const unsigned *c = reinterpret_cast<const unsigned *>(counts) + tid;
      unsigned s = 0;
      for (int k = 0; k < W; ++k) s += c[4 * k];
      reinterpret_cast<unsigned *>(counts + W)[tid] = s;
    }
    sync_all<true>();
    for (int j = 0; j < rank; ++j) {
      const uint4 y = remote128(smem_u32(counts + W), j);
      pass({y.x, y.y, y.z, y.w}, min(all1, all0 + j * part), min(all1, all0 + (j + 1) * part));
    }
    sync_all<true>();  // nobody leaves while its counts are read
  }
#pragma unroll 1
  for (int j = 0; j < warp; ++j) pass(counts[j], min(v1, v0 + j * share), min(v1, v0 + (j + 1) * share));
  // ---- the lists
  int *places = a.ws_list + static_cast<int64_t>(x) * 2 * a.cap, *tokens = places + a.cap;
  walk([&](int v, const uint4 &k) {
    const int i = 4 * v - skew;
    const unsigned key[4] = {k.x, k.y, k.z, k.w};
    unsigned stay = 0, same = 0, in = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (key[e] > prefix) stay |= 1u << e;
      if (key[e] == prefix) same |= 1u << e;
      if (key[e] != 0u) in |= 1u << e;
    }
    if (__any_sync(0xffffffffu, same != 0u)) {  // equals up to the need-th
      unsigned y = ties + lanes_before(same);
      ties += __reduce_add_sync(0xffffffffu, __popc(same));
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (same >> e & 1u)
          if (y++ < need) stay |= 1u << e;
    }
    const unsigned below = (1u << max(0, min(4, end - i))) - 1u, hole = in & ~stay & below, goes = stay & ~below;
    if (__any_sync(0xffffffffu, hole != 0u)) {
      int *to = places + holes + lanes_before(hole);
      holes += __reduce_add_sync(0xffffffffu, __popc(hole));
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (hole >> e & 1u) *to++ = i + e;
    }
    if (__any_sync(0xffffffffu, goes != 0u)) {
      int *to = tokens + late + lanes_before(goes);
      late += __reduce_add_sync(0xffffffffu, __popc(goes));
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (goes >> e & 1u) *to++ = i + e;
    }
  });
  if (tid == T - 1 && rank == ctas - 1) *meta = {late, 1, keep, w};
}

// ---------------------------------------------------------------------------
// moving them
// ---------------------------------------------------------------------------
// A token's codes are pieces of 16 bytes, first K's, then V's; LANES lanes (4, 8
// or 16, at least as many as there are pieces) have one token's.
__device__ __forceinline__ uint4 *piece_of(const EvictArgs &a, int64_t slot, int piece) {
  const int kp = a.krow / 16;
  return piece < kp ? reinterpret_cast<uint4 *>(a.kc + slot * a.krow) + piece
                    : reinterpret_cast<uint4 *>(a.vc + slot * a.vrow) + (piece - kp);
}
// The (token, head) row of position i of a cache row.
__device__ __forceinline__ int64_t slot_of(const EvictArgs &a, const int32_t *table, int h, int i) {
  return (static_cast<int64_t>(__ldg(table + i / kBlockSize)) * kBlockSize + i % kBlockSize) * a.H + h;
}
// A token's scales and weight.
struct Rest {
  float k, v[4], w;
};
__device__ __forceinline__ Rest load_rest(const EvictArgs &a, const float *weights, int64_t slot, int i) {
  Rest x;
  x.k = a.ks[slot];
  const float *v = a.vs + slot * a.vgroups;
#pragma unroll
  for (int g = 0; g < 4; ++g) x.v[g] = g < a.vgroups ? v[g] : 0.f;
  x.w = weights[i];
  return x;
}
__device__ __forceinline__ void store_rest(const EvictArgs &a, float *weights, int64_t slot, int i, const Rest &x) {
  a.ks[slot] = x.k;
  float *v = a.vs + slot * a.vgroups;
#pragma unroll
  for (int g = 0; g < 4; ++g)
    if (g < a.vgroups) v[g] = x.v[g];
  weights[i] = x.w;
}

// A warp takes 32 tokens of a (row, head): each lane looks one up, then all lanes
// copy, LANES of them a token, eight loads of a lane in flight.
template <int LANES>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
  constexpr int AT_ONCE = 32 / LANES, U = LANES < 8 ? LANES : 8;
  const int lane = threadIdx.x & 31, piece = lane % LANES, heads = a.rows * a.H;
  const bool has = piece < (a.krow + a.vrow) / 16;
  // the warps that share a (row, head), 32 tokens each in turn
  const int warps = gridDim.x * 8, per = max(1, warps / heads);
  grid_wait();  // the lists
  for (int it = blockIdx.x * 8 + (threadIdx.x >> 5); it < heads * per; it += warps) {
    const int x = it % heads, moves = a.ws_meta[x].moves;
    const int32_t *table = a.tables + static_cast<int64_t>(x / a.H) * a.max_blocks;
    const int *places = a.ws_list + static_cast<int64_t>(x) * 2 * a.cap, *tokens = places + a.cap;
    float *weights = a.weights + static_cast<int64_t>(x) * a.stride;
    for (int c = 32 * (it / heads); c < moves; c += 32 * per) {
      const int left = moves - c, me = c + min(lane, left - 1), to = places[me], from = tokens[me];
      const int64_t sf = slot_of(a, table, x % a.H, from), st = slot_of(a, table, x % a.H, to);
      const Rest rest = load_rest(a, weights, sf, from);
#pragma unroll 1
      for (int s = 0; s < LANES; s += U) {
        if (s * AT_ONCE >= left) break;
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t f = __shfl_sync(0xffffffffu, sf, (s + u) * AT_ONCE + lane / LANES);
          if (has) v[u] = *piece_of(a, f, piece);  // (past the last token: its own again)
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = (s + u) * AT_ONCE + lane / LANES;
          const int64_t t = __shfl_sync(0xffffffffu, st, k);
          if (has && k < left) *piece_of(a, t, piece) = v[u];
        }
      }
      if (lane < left) store_rest(a, weights, st, to, rest);
    }
  }
}

// The last w tokens of a (row, head) move down by s = n - k places.  A place is
// written by the token s behind it and no other, so the tokens of one residue of s
// are a chain of their own: the CTAs share the residues, and each takes its tokens
// in ascending order, as many at a time as its registers hold (all are read before
// any is written).  Weights past k become 0.
// A CTA that has all residues, or whose residues have one token each, has
// neighbouring tokens and needs no division (NEAR).
constexpr int kShiftThreads = 256, kShiftPieces = 8;
template <int LANES, bool NEAR>
__device__ __forceinline__ void shift_tokens(const EvictArgs &a, const int32_t *table, float *weights, int h, int n, int k, int w,
                                             int c0, int r) {
  constexpr int TOKENS = kShiftThreads * kShiftPieces / LANES, SCALARS = (TOKENS + kShiftThreads - 1) / kShiftThreads;
  const int tid = threadIdx.x, piece = tid % LANES, s = n - k;
  const bool has = piece < (a.krow + a.vrow) / 16;
  const int first = n - w, to = k - w;
  // element e of this CTA's; those past its last get w
  const int mine = NEAR ? (w <= s ? r : w) : (w - c0 + s - 1) / s * r;
  auto token = [&](int e) {
    if (e >= mine) return w;
    if (NEAR) return c0 + e;
    const int m = e / r;
    const int64_t i = static_cast<int64_t>(m) * s + c0 + (e - m * r);
    return i < w ? static_cast<int>(i) : w;
  };
#pragma unroll 1
  for (int base = 0; base < mine; base += TOKENS) {
    uint4 v[kShiftPieces];
    Rest rest[SCALARS];
#pragma unroll
    for (int u = 0; u < kShiftPieces; ++u) {
      const int i = token(base + (u * kShiftThreads + tid) / LANES);
      if (has && i < w) v[u] = *piece_of(a, slot_of(a, table, h, first + i), piece);
    }
#pragma unroll
    for (int u = 0; u < SCALARS; ++u) {
      const int i = token(base + u * kShiftThreads + tid);
      if (u * kShiftThreads + tid < TOKENS && i < w) rest[u] = load_rest(a, weights, slot_of(a, table, h, first + i), first + i);
    }
    if (w > s) __syncthreads();
#pragma unroll
    for (int u = 0; u < kShiftPieces; ++u) {
      const int i = token(base + (u * kShiftThreads + tid) / LANES);
      if (has && i < w) *piece_of(a, slot_of(a, table, h, to + i), piece) = v[u];
    }
#pragma unroll
    for (int u = 0; u < SCALARS; ++u) {
      const int i = token(base + u * kShiftThreads + tid);
      if (u * kShiftThreads + tid >= TOKENS || i >= w) continue;
      store_rest(a, weights, slot_of(a, table, h, to + i), to + i, rest[u]);
      if (first + i >= k) weights[first + i] = 0.f;  // (its reader clears it)
    }
    if (w > s) __syncthreads();
  }
}

template <int LANES>
__global__ void __launch_bounds__(kShiftThreads, 3) evict_shift_kernel(const EvictArgs a) {
  const int x = blockIdx.x, y = blockIdx.y;
  grid_wait();  // the moves have read what is written here
  const EvictMeta meta = a.ws_meta[x];
  if (!meta.active) return;
  const int32_t *table = a.tables + static_cast<int64_t>(x / a.H) * a.max_blocks;
  const int n = __ldg(a.ctx + x / a.H), w = meta.recent, k = meta.keep, h = x % a.H;
  float *weights = a.weights + static_cast<int64_t>(x) * a.stride;
  // residues [c0, c0 + r) of the chains, of which there are no more than tokens
  const int chains = min(n - k, w);
  const int c0 = static_cast<int>(static_cast<int64_t>(chains) * y / gridDim.y);
  const int r = static_cast<int>(static_cast<int64_t>(chains) * (y + 1) / gridDim.y) - c0;
  if (r == n - k || w <= n - k) shift_tokens<LANES, true>(a, table, weights, h, n, k, w, c0, r);
  else if (r > 0) shift_tokens<LANES, false>(a, table, weights, h, n, k, w, c0, r);
  for (int64_t i = k + static_cast<int64_t>(y) * kShiftThreads + threadIdx.x; i < n - w; i += gridDim.y * kShiftThreads) weights[i] = 0.f;
}

template <int LANES>
cudaError_t move(const EvictArgs &a, int sms, cudaStream_t stream) {
  // (no more warps than there can be lists of 32)
  const int64_t heads = a.rows * a.H, ctas = (heads * ((a.cap + 31) / 32) + 7) / 8;
  cudaError_t e = launch_overlapped(evict_move_kernel<LANES>, static_cast<int>(ctas < 1 ? 1 : ctas < 8 * sms ? ctas : 8 * sms),
                                    256, 0, stream, a);
  if (e != cudaSuccess) return e;
  // CTAs for a (row, head): enough for all SMs
  const int share = static_cast<int>(4 * sms / heads);
  return launch_overlapped(evict_shift_kernel<LANES>, dim3(static_cast<unsigned>(heads), share < 1 ? 1 : share > 64 ? 64 : share),
                           kShiftThreads, 0, stream, a);
}

template <int T, bool HELD, bool CLUSTER>
cudaError_t select_with(const EvictArgs &a, int ctas, size_t bytes, cudaStream_t stream) {
  auto kern = evict_select_kernel<T, HELD, CLUSTER>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  static std::atomic<unsigned long long> done{0};  // devices whose limit is raised
  if (HELD && !((done.load(std::memory_order_acquire) >> dev) & 1ull)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  16 * ((T > 512 ? 2 : 1) * kHeld / 4 + 2))) != cudaSuccess)
      return e;
    done.fetch_or(1ull << dev, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.rows * a.H * ctas);
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CLUSTER ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a, ctas);
}

cudaError_t select(const EvictArgs &a, int sms, cudaStream_t stream) {
  // CTAs that hold the keys of a row as long as the weights are wide (the host does not
  // see the rows' lengths), and no more: where few rows leave SMs without work, more of
  // them for a (row, head) still take longer (8 heads of 16384 positions: one 13 us,
  // four 26; 32 heads of 32768: two 18, eight 54).  Weights much wider than the rows
  // cost the same surplus (256 x 8 heads of ~4160 tokens, the three kernels: 103 us
  // with 4160 positions, 104 with 8192, 117 with 16384, 188 with 32768, 1260 with 131072)
  int ctas = 1;
  while (ctas < 8 && a.stride > static_cast<int64_t>(ctas) * kHeld) ctas *= 2;
  // Where SMs would hold two or three of a cluster's CTAs, half as many of twice the
  // threads and keys, if that is one an SM (64 heads of 65536: 31 and 25 us, 144 of 32768
  // 26 and 21, 32 of 120000 48 and 27; not where there is an SM for each as it is:
  // 32 of 60000 21 and 24)
  const int64_t heads = static_cast<int64_t>(a.rows) * a.H;
  const int half = ctas / 2;
  if (half > 0 && a.stride <= int64_t{2} * half * kHeld && heads * ctas > sms && heads * half <= sms) {
    const size_t bytes = 16 * (static_cast<size_t>(a.stride / 4 + 2 + half - 1) / half);
    return half == 1 ? select_with<1024, true, false>(a, 1, bytes, stream) : select_with<1024, true, true>(a, half, bytes, stream);
  }
  const int64_t keys = (a.stride + ctas - 1) / ctas;
  if (keys > kHeld) return select_with<512, false, true>(a, ctas, 0, stream);
  const size_t bytes = 16 * (static_cast<size_t>(a.stride / 4 + 2 + ctas - 1) / ctas);  // vectors of any alignment
  // Half as many threads for short rows, or where there are more of them than SMs hold
  // (512 rows of 8192: 20.8 for 23.9 us, 400 of 4000 11.8 for 13.6; 8 of 8192 11.1 for 8.9)
  if (keys <= 4096 || (keys <= 8192 && heads > 3 * sms))
    return select_with<256, true, false>(a, 1, bytes, stream);
  return ctas == 1 ? select_with<512, true, false>(a, 1, bytes, stream) : select_with<512, true, true>(a, ctas, bytes, stream);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t stream) {
  const cudaError_t e = select(a, sms, stream);
  if (e != cudaSuccess) return e;
  const int pieces = (a.krow + a.vrow) / 16;
  return pieces <= 4 ? move<4>(a, sms, stream) : pieces <= 8 ? move<8>(a, sms, stream) : move<16>(a, sms, stream);
}

}  // namespace kvq
