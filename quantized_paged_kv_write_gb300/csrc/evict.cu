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
#include "common.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

// Weights as unsigned numbers in the same order; -0 counts as 0, NaN as the
// largest.  None is 0, which stands for a position that is no candidate.
__device__ __forceinline__ unsigned order_of(float x) {
  const unsigned b = __float_as_uint(x + 0.f);
  return x != x ? 0xFFFFFFFFu : b ^ (static_cast<unsigned>(static_cast<int>(b) >> 31) | 0x80000000u);
}

// ---------------------------------------------------------------------------
// which tokens stay
// ---------------------------------------------------------------------------
// One cluster of CTAs per (row, kv head), each with an even part of the
// candidates: the threshold by three passes over their weights (11, 11 and 10
// bits, from the top; the CTAs add up their histograms), then the lists of places
// and of tokens to go there.
constexpr int kBins = 2048;

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

// The sum of a warp's `own` over the warps before this one; *all over all.
template <int T>
__device__ __forceinline__ unsigned warps_before(unsigned own, unsigned *sums, unsigned *all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sums[warp] = own;
  __syncthreads();
  const unsigned s = lane < T / 32 ? sums[lane] : 0u;
  *all = __reduce_add_sync(0xffffffffu, s);
  const unsigned before = __reduce_add_sync(0xffffffffu, lane < warp ? s : 0u);
  __syncthreads();
  return before;
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

// A step is up to T KV vectors of four weights, a warp's in one piece: vector u of
// a lane is 32 behind its vector u - 1.  ONE: a step holds all candidates, which
// stay in registers; else each pass reads them again (from L2, after the first).
// CLUSTER: more than one CTA.
template <int T, int KV, bool ONE, bool CLUSTER>
__global__ void __launch_bounds__(T, 768 / T) evict_select_kernel(const EvictArgs a, const int ctas) {
  static_assert(!(ONE && CLUSTER), "one step of one CTA");
  static_assert(4 * KV <= 32, "a bit for each of a lane's weights");
  __shared__ __align__(16) unsigned hist[kBins];
  __shared__ unsigned sums[32];
  __shared__ __align__(16) unsigned counts[4];
  __shared__ unsigned chosen, left, equals;
  grid_release();
  const int x = CLUSTER ? blockIdx.x / ctas : blockIdx.x, rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
  const int r = x / a.H, h = x - r * a.H, tid = threadIdx.x;
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
  int v0 = (p + skew) / 4, v1 = (last + skew + 3) / 4;
  if constexpr (CLUSTER) {
    const int per = (v1 - v0 + ctas - 1) / ctas;
    v0 = min(v1, v0 + rank * per);
    v1 = min(v1, v0 + per);
  }
  // the keys of a step, 0 where there is no candidate
  unsigned key[KV][4];
  int su = 0, first = 0;  // vectors of a lane, and its first one
  auto load = [&](int base) {
    su = (min(v1 - base, T * KV) + T - 1) / T;
    first = base + (tid >> 5) * 32 * su + (tid & 31);
    float4 y[KV];
#pragma unroll
    for (int u = 0; u < KV; ++u) {
      if (u >= su) break;
      const int v = first + 32 * u, i = 4 * v - skew;
      y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (v < v1 && i >= p && i + 4 <= last) {
        y[u] = *reinterpret_cast<const float4 *>(weights + i);
      } else if (v < v1) {
        if (i >= p && i < last) y[u].x = weights[i];
        if (i + 1 >= p && i + 1 < last) y[u].y = weights[i + 1];
        if (i + 2 >= p && i + 2 < last) y[u].z = weights[i + 2];
        if (i + 3 >= p && i + 3 < last) y[u].w = weights[i + 3];
      }
    }
#pragma unroll
    for (int u = 0; u < KV; ++u) {
      if (u >= su) break;
      const int v = first + 32 * u, i = 4 * v - skew;
      key[u][0] = order_of(y[u].x);
      key[u][1] = order_of(y[u].y);
      key[u][2] = order_of(y[u].z);
      key[u][3] = order_of(y[u].w);
      if (v >= v1 || i < p || i + 4 > last)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (v >= v1 || i + e < p || i + e >= last) key[u][e] = 0u;
    }
  };
  if constexpr (ONE) load(v0);
  // (while they are under way) every block of the row, and nobody else's among
  // those to be written
  const int32_t *table = a.tables + static_cast<int64_t>(r) * a.max_blocks;
  bool bad = false, shared = false;
  for (int i = tid; i < (n + kBlockSize - 1) / kBlockSize; i += T) {
    const int id = __ldg(table + i);
    if (id < 0 || id >= a.num_blocks) bad = true;
    else if (a.refs != nullptr && i >= p / kBlockSize && i * kBlockSize < keep && __ldg(a.refs + id) != 1) shared = true;
  }
  for (int i = tid; i < kBins; i += T) hist[i] = 0;
  bad = __syncthreads_or(bad);
  shared = __syncthreads_or(shared);
  if (bad || shared) {
    if (reports) *meta = {0, 0, 0, 0};
    if (reports) set_error(a.err, bad ? KVQ_DEVERR_BLOCK_RANGE : KVQ_DEVERR_POOL_STATE);
    if (reports && h == 0) a.kept[r] = n;
    return;
  }
  if (reports && h == 0) a.kept[r] = keep;
  // ---- the need-th largest key, and how many of its equals are kept
  unsigned prefix = 0xFFFFFFFFu, need = end - p;  // (nothing needed: nothing is above)
  bool partial = need == 0;                       // of the equals some stay and some go
  if (need > 0) {
    unsigned mask = 0;
    prefix = 0;
#pragma unroll 1
    for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift == 10 ? 0 : -1) {
      const unsigned digit = shift == 0 ? 1023u : 2047u;
#pragma unroll 1
      for (int base = v0; base < v1; base += T * KV) {
        if constexpr (!ONE) load(base);
#pragma unroll
        for (int u = 0; u < KV; ++u) {
          if (u >= su) break;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key[u][e] != 0u && (key[u][e] & mask) == prefix) atomicAdd(&hist[(key[u][e] >> shift) & digit], 1u);
        }
      }
      sync_all<CLUSTER>();
      // digits from the largest: the one in which the need-th lies
      constexpr int PER = kBins / T;
      static_assert(PER % 4 == 0, "whole vectors of bins");
      const int b0 = kBins - (tid + 1) * PER;
      unsigned bin[PER], own = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k) bin[k] = 0;
      if constexpr (CLUSTER) {
#pragma unroll 1
        for (int j = 0; j < ctas; ++j)
#pragma unroll
          for (int k = 0; k < PER; k += 4) {
            const uint4 y = remote128(smem_u32(hist + b0 + k), j);
            bin[k] += y.x;
            bin[k + 1] += y.y;
            bin[k + 2] += y.z;
            bin[k + 3] += y.w;
          }
      } else {
#pragma unroll
        for (int k = 0; k < PER; k += 4) {
          const uint4 y = *reinterpret_cast<const uint4 *>(hist + b0 + k);
          bin[k] = y.x;
          bin[k + 1] = y.y;
          bin[k + 2] = y.z;
          bin[k + 3] = y.w;
        }
      }
#pragma unroll
      for (int k = 0; k < PER; ++k) own += bin[k];
      unsigned before = own, all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, before, o);
        if ((tid & 31) >= o) before += y;
      }
      before += warps_before<T>(__shfl_sync(0xffffffffu, before, 31), sums, &all) - own;
      if (before < need && need <= before + own) {
        bool found = false;
#pragma unroll
        for (int k = PER - 1; k >= 0; --k) {
          if (!found && before + bin[k] >= need) {
            found = true;
            chosen = b0 + k;
            left = need - before;
            equals = bin[k];
          }
          before += bin[k];
        }
      }
      sync_all<CLUSTER>();  // (and all CTAs have read the histograms)
      prefix |= chosen << shift;
      mask |= digit << shift;
      need = left;
      partial = need < equals;
      if (shift > 0) {
        for (int i = tid; i < kBins; i += T) hist[i] = 0;
        __syncthreads();
      }
    }
  }
  // ---- what the CTAs before this one have
  unsigned ties = 0;        // equals,
  int holes = 0, late = 0;  // places and tokens
  if constexpr (CLUSTER) {
    if (tid < 4) counts[tid] = 0;
    __syncthreads();
    // larger and equal keys below `end`, and from there on
    unsigned c[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
    for (int base = v0; base < v1; base += T * KV) {
      load(base);
#pragma unroll
      for (int u = 0; u < KV; ++u) {
        if (u >= su) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool low = 4 * (first + 32 * u) - skew + e < end;
          c[0] += key[u][e] > prefix && low;
          c[1] += key[u][e] == prefix && low;
          c[2] += key[u][e] > prefix && !low;
          c[3] += key[u][e] == prefix && !low;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const unsigned s = __reduce_add_sync(0xffffffffu, c[k]);
      if ((tid & 31) == 0) atomicAdd(&counts[k], s);
    }
    sync_all<CLUSTER>();
    const int per = ((last + skew + 3) / 4 - (p + skew) / 4 + ctas - 1) / ctas;
#pragma unroll 1
    for (int j = 0; j < rank; ++j) {
      const uint4 y = remote128(smem_u32(counts), j);
      const unsigned stay = min(ties < need ? need - ties : 0u, y.y + y.w), low = min(stay, y.y);
      // the candidates below `end` of CTA j
      const int from = max(p, 4 * ((p + skew) / 4 + j * per) - skew), to = min(end, 4 * ((p + skew) / 4 + (j + 1) * per) - skew);
      holes += max(0, to - from) - static_cast<int>(y.x + low);
      late += static_cast<int>(y.z + stay - low);
      ties += y.y + y.w;
    }
    sync_all<CLUSTER>();  // nobody leaves while its counts are read
  }
  // ---- the lists
  int *places = a.ws_list + static_cast<int64_t>(x) * 2 * a.cap, *tokens = places + a.cap;
#pragma unroll 1
  for (int base = v0; base < v1; base += T * KV) {
    if constexpr (!ONE) load(base);
    // bit 4 u + e: a candidate that stays
    unsigned stay = 0, same = 0, in = 0, all;
#pragma unroll
    for (int u = 0; u < KV; ++u) {
      if (u >= su) break;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (key[u][e] >= prefix) stay |= 1u << (4 * u + e);
        if (key[u][e] == prefix) same |= 1u << (4 * u + e);
        if (key[u][e] != 0u) in |= 1u << (4 * u + e);
      }
    }
    if (partial) {  // (uniform) equals past the need-th go
      unsigned y = ties + warps_before<T>(__reduce_add_sync(0xffffffffu, __popc(same)), sums, &all);
      ties += all;
#pragma unroll
      for (int u = 0; u < KV; ++u) {
        const unsigned bits = same >> (4 * u) & 15u;
        if (u >= su) break;
        if (!__any_sync(0xffffffffu, bits != 0u)) continue;
        unsigned z = y + lanes_before(bits);
        y += __reduce_add_sync(0xffffffffu, __popc(bits));
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (bits >> e & 1u)
            if (z++ >= need) stay &= ~(1u << (4 * u + e));
      }
    }
    unsigned hole = 0, goes = 0;
#pragma unroll
    for (int u = 0; u < KV; ++u) {
      if (u >= su) break;
      const int low = max(0, min(4, end - (4 * (first + 32 * u) - skew)));  // of the vector, below `end`
      const unsigned below = ((1u << low) - 1u) << (4 * u), above = (15u << (4 * u)) & ~below;
      hole |= in & ~stay & below;
      goes |= stay & above;
    }
    // places (low half) and tokens (high half), at most 4 T KV <= 2^13 of each in a step
    const unsigned before =
        warps_before<T>(__reduce_add_sync(0xffffffffu, __popc(hole) | __popc(goes) << 16), sums, &all);
    int y = holes + static_cast<int>(before & 0xFFFFu), z = late + static_cast<int>(before >> 16);
#pragma unroll
    for (int u = 0; u < KV; ++u) {
      if (u >= su) break;
      const int i = 4 * (first + 32 * u) - skew;
      const unsigned b = hole >> (4 * u) & 15u, c = goes >> (4 * u) & 15u;
      if (__any_sync(0xffffffffu, b != 0u)) {
        int *to = places + y + lanes_before(b);
        y += __reduce_add_sync(0xffffffffu, __popc(b));
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (b >> e & 1u) *to++ = i + e;
      }
      if (__any_sync(0xffffffffu, c != 0u)) {
        int *to = tokens + z + lanes_before(c);
        z += __reduce_add_sync(0xffffffffu, __popc(c));
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c >> e & 1u) *to++ = i + e;
      }
    }
    holes += static_cast<int>(all & 0xFFFFu);
    late += static_cast<int>(all >> 16);
  }
  if (tid == 0 && rank == ctas - 1) *meta = {late, 1, keep, w};
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
  grid_release();
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

// The last w tokens of a (row, head), which may overlap their new places: one
// CTA, in ascending order (a place is below its token), as many tokens at a time
// as its registers hold.  Then weights past k.
constexpr int kShiftThreads = 256, kShiftPieces = 8;
template <int LANES>
__global__ void __launch_bounds__(kShiftThreads, 3) evict_shift_kernel(const EvictArgs a) {
  constexpr int TOKENS = kShiftThreads * kShiftPieces / LANES, SCALARS = (TOKENS + kShiftThreads - 1) / kShiftThreads;
  const int x = blockIdx.x, tid = threadIdx.x, piece = tid % LANES;
  const bool has = piece < (a.krow + a.vrow) / 16;
  grid_wait();  // the moves have read what is written here
  const EvictMeta meta = a.ws_meta[x];
  if (!meta.active) return;
  const int32_t *table = a.tables + static_cast<int64_t>(x / a.H) * a.max_blocks;
  const int n = __ldg(a.ctx + x / a.H), w = meta.recent, k = meta.keep, h = x % a.H;
  float *weights = a.weights + static_cast<int64_t>(x) * a.stride;
#pragma unroll 1
  for (int base = 0; base < w; base += TOKENS) {
    uint4 v[kShiftPieces];
    Rest rest[SCALARS];
#pragma unroll
    for (int u = 0; u < kShiftPieces; ++u) {
      const int i = base + (u * kShiftThreads + tid) / LANES;
      if (has && i < w) v[u] = *piece_of(a, slot_of(a, table, h, n - w + i), piece);
    }
#pragma unroll
    for (int u = 0; u < SCALARS; ++u) {
      const int i = base + u * kShiftThreads + tid;
      if (u * kShiftThreads + tid < TOKENS && i < w) rest[u] = load_rest(a, weights, slot_of(a, table, h, n - w + i), n - w + i);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kShiftPieces; ++u) {
      const int i = base + (u * kShiftThreads + tid) / LANES;
      if (has && i < w) *piece_of(a, slot_of(a, table, h, k - w + i), piece) = v[u];
    }
#pragma unroll
    for (int u = 0; u < SCALARS; ++u) {
      const int i = base + u * kShiftThreads + tid;
      if (u * kShiftThreads + tid < TOKENS && i < w) store_rest(a, weights, slot_of(a, table, h, k - w + i), k - w + i, rest[u]);
    }
    __syncthreads();
  }
  for (int i = k + tid; i < n; i += kShiftThreads) weights[i] = 0.f;
}

template <int LANES>
cudaError_t move(const EvictArgs &a, int sms, cudaStream_t stream) {
  // (no more warps than there can be lists of 32)
  const int64_t heads = a.rows * a.H, ctas = (heads * ((a.cap + 31) / 32) + 7) / 8;
  cudaError_t e = launch_overlapped(evict_move_kernel<LANES>, static_cast<int>(ctas < 1 ? 1 : ctas < 8 * sms ? ctas : 8 * sms),
                                    256, 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_overlapped(evict_shift_kernel<LANES>, static_cast<int>(heads), kShiftThreads, 0, stream, a);
}

cudaError_t select(const EvictArgs &a, int sms, cudaStream_t stream) {
  const int heads = a.rows * a.H;
  // (4 KV T positions from any of four alignments)
  if (a.stride <= 8192 - 4) {
    evict_select_kernel<256, 8, true, false><<<heads, 256, 0, stream>>>(a, 1);
    return cudaGetLastError();
  }
  // few rows: a cluster for each, as long as two CTAs an SM hold them all
  int ctas = 1;
  while (ctas < 8 && 2 * ctas * heads <= 2 * sms) ctas *= 2;
  if (ctas == 1) {
    evict_select_kernel<256, 8, false, false><<<heads, 256, 0, stream>>>(a, 1);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(heads * ctas);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<256, 8, false, true>, a, ctas);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t stream) {
  const cudaError_t e = select(a, sms, stream);
  if (e != cudaSuccess) return e;
  const int pieces = (a.krow + a.vrow) / 16;
  return pieces <= 4 ? move<4>(a, sms, stream) : pieces <= 8 ? move<8>(a, sms, stream) : move<16>(a, sms, stream);
}

}  // namespace kvq
