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

// Weights as unsigned numbers in the same order; -0 counts as 0, NaN as the largest.
__device__ __forceinline__ unsigned order_of(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const unsigned b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// ---------------------------------------------------------------------------
// which tokens stay
// ---------------------------------------------------------------------------
// One CTA per (row, kv head): the threshold by three passes over the candidates'
// weights (11, 11 and 10 bits, from the top), then the lists of places and of
// tokens to go there.  The weights are read again in each pass (they are in L2
// after the first), four vectors of a thread in flight.
constexpr int kBins = 2048, kVectors = 4;

// c[u]: own counts; becomes the counts before this thread's, in the order (u,
// thread).  Returns the sum of all.
template <int T>
__device__ __forceinline__ unsigned scan_before(unsigned (&c)[kVectors], unsigned (*sums)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned x[kVectors];
#pragma unroll
  for (int u = 0; u < kVectors; ++u) {
    x[u] = c[u];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, x[u], o);
      if (lane >= o) x[u] += y;
    }
    if (lane == 31) sums[u][warp] = x[u];
  }
  __syncthreads();
  unsigned all = 0;
#pragma unroll
  for (int u = 0; u < kVectors; ++u) {
    const unsigned s = lane < T / 32 ? sums[u][lane] : 0u;
    c[u] = all + __reduce_add_sync(0xffffffffu, lane < warp ? s : 0u) + x[u] - c[u];
    all += __reduce_add_sync(0xffffffffu, s);
  }
  __syncthreads();
  return all;
}

template <int T>
__global__ void __launch_bounds__(T, 1024 / T) evict_select_kernel(const EvictArgs a) {
  __shared__ unsigned hist[kBins], sums[kVectors][32];
  __shared__ unsigned chosen, left, equals;
  grid_release();
  const int r = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x;
  const int n = __ldg(a.ctx + r), keep = __ldg(a.keep + r), recent = __ldg(a.recent + r);
  const int pinned = a.pinned != nullptr ? __ldg(a.pinned + r) : 0;
  EvictMeta *meta = a.ws_meta + blockIdx.x;
  const bool range = n < 0 || n > a.max_len || keep < 0 || recent < 0 || pinned < 0;
  if (range || n <= keep) {
    if (tid == 0) *meta = {0, 0, 0, 0};
    if (tid == 0 && range) set_error(a.err, KVQ_DEVERR_CONTEXT_RANGE);
    if (tid == 0 && h == 0) a.kept[r] = n;
    return;
  }
  const int w = min(recent, keep), p = min(pinned, keep - w), end = keep - w;
  // every block of the row, and nobody else's among those to be written
  const int32_t *table = a.tables + static_cast<int64_t>(r) * a.max_blocks;
  bool bad = false, shared = false;
  for (int i = tid; i < (n + kBlockSize - 1) / kBlockSize; i += T) {
    const int id = __ldg(table + i);
    if (id < 0 || id >= a.num_blocks) bad = true;
    else if (a.refs != nullptr && i >= p / kBlockSize && i * kBlockSize < keep && __ldg(a.refs + id) != 1) shared = true;
  }
  bad = __syncthreads_or(bad);
  shared = __syncthreads_or(shared);
  if (bad || shared) {
    if (tid == 0) *meta = {0, 0, 0, 0};
    if (tid == 0) set_error(a.err, bad ? KVQ_DEVERR_BLOCK_RANGE : KVQ_DEVERR_POOL_STATE);
    if (tid == 0 && h == 0) a.kept[r] = n;
    return;
  }
  if (tid == 0 && h == 0) a.kept[r] = keep;
  const float *weights = a.weights + static_cast<int64_t>(blockIdx.x) * a.stride;
  const int last = n - w;  // candidates are [p, last)
  // Vectors of four weights on 16-byte boundaries: vector v holds the positions
  // 4 v - skew .. + 3; those outside the candidates are masked.
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(weights) >> 2) & 3);
  const int v0 = (p + skew) / 4, v1 = (last + skew + 3) / 4;
  auto load = [&](int v) {
    const int i = 4 * v - skew;
    if (v < v1 && i >= p && i + 4 <= last) return *reinterpret_cast<const float4 *>(weights + i);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (v < v1) {
      if (i >= p && i < last) x.x = weights[i];
      if (i + 1 >= p && i + 1 < last) x.y = weights[i + 1];
      if (i + 2 >= p && i + 2 < last) x.z = weights[i + 2];
      if (i + 3 >= p && i + 3 < last) x.w = weights[i + 3];
    }
    return x;
  };
  // f(u, position, key) for the candidates of this thread's vectors from `base` on
  auto each = [&](int base, auto f) {
    float4 x[kVectors];
#pragma unroll
    for (int u = 0; u < kVectors; ++u) x[u] = load(base + u * T + tid);
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      const int i = 4 * (base + u * T + tid) - skew;
      const float y[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e >= p && i + e < last) f(u, i + e, order_of(y[e]));
    }
  };
  // ---- the need-th largest weight, and how many of its equals are kept
  unsigned prefix = 0, mask = 0, need = end - p;
  bool partial = false;  // of the equals some stay and some go
  if (need > 0) {
#pragma unroll 1
    for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift == 10 ? 0 : -1) {
      // (digits of 11, 11 and 10 bits: shifts 21, 10 and 0)
      const unsigned digit = shift == 0 ? 1023u : 2047u;
      for (int i = tid; i < kBins; i += T) hist[i] = 0;
      __syncthreads();
#pragma unroll 1
      for (int base = v0; base < v1; base += T * kVectors)
        each(base, [&](int, int, unsigned key) {
          if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & digit], 1u);
        });
      __syncthreads();
      // digits from the largest: the one in which the need-th lies
      constexpr int PER = kBins / T;
      unsigned own = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k) own += hist[kBins - 1 - (tid * PER + k)];
      unsigned c[kVectors] = {own, 0u, 0u, 0u};
      scan_before<T>(c, sums);
      if (c[0] < need && need <= c[0] + own) {
        unsigned before = c[0];
        int b = kBins - 1 - tid * PER;
        while (before + hist[b] < need) before += hist[b--];
        chosen = b;
        left = need - before;
        equals = hist[b];
      }
      __syncthreads();
      prefix |= chosen << shift;
      mask |= digit << shift;
      need = left;
      partial = need < equals;
      __syncthreads();
    }
  }
  // ---- the lists
  int *places = a.ws_list + static_cast<int64_t>(blockIdx.x) * 2 * a.cap, *tokens = places + a.cap;
  const bool some = end > p;
  unsigned ties = 0, lists = 0;  // places (low half) and tokens (high half) so far: below 2^15 in a step
  int holes = 0, late = 0;
#pragma unroll 1
  for (int base = v0; base < v1; base += T * kVectors) {
    unsigned stay = 0, same = 0;  // bit 4 u + e: kept, and equal to the threshold
    const int first = 4 * (base + tid) - skew;
    each(base, [&](int u, int i, unsigned key) {
      const int bit = 4 * u + (i - first - 4 * T * u);
      if (some && key > prefix) stay |= 1u << bit;
      if (some && key == prefix) same |= 1u << bit;
    });
    if (partial) {  // (uniform)
      unsigned c[kVectors];
#pragma unroll
      for (int u = 0; u < kVectors; ++u) c[u] = __popc(same >> (4 * u) & 15u);
      const unsigned all = scan_before<T>(c, sums);
#pragma unroll
      for (int u = 0; u < kVectors; ++u) {
        unsigned rank = ties + c[u];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (same >> (4 * u + e) & 1u)
            if (rank++ < need) stay |= 1u << (4 * u + e);
      }
      ties += all;
    } else {
      stay |= same;
    }
    unsigned c[kVectors], goes = 0, hole = 0;
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = first + 4 * T * u + e, bit = 4 * u + e;
        const bool in = i >= p && i < last, kept = stay >> bit & 1u;
        if (in && i < end && !kept) hole |= 1u << bit;
        if (in && i >= end && kept) goes |= 1u << bit;
      }
      c[u] = __popc(hole >> (4 * u) & 15u) | __popc(goes >> (4 * u) & 15u) << 16;
    }
    lists = scan_before<T>(c, sums);
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      int x = holes + static_cast<int>(c[u] & 0xFFFFu), y = late + static_cast<int>(c[u] >> 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = first + 4 * T * u + e, bit = 4 * u + e;
        if (hole >> bit & 1u) places[x++] = i;
        if (goes >> bit & 1u) tokens[y++] = i;
      }
    }
    holes += static_cast<int>(lists & 0xFFFFu);
    late += static_cast<int>(lists >> 16);
  }
  if (tid == 0) *meta = {late, 1, keep, w};
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
  const int64_t items = static_cast<int64_t>((a.cap + 31) / 32) * heads;
  grid_wait();  // the lists
  grid_release();
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items; it += gridDim.x * 8) {
    const int c = static_cast<int>(it / heads), x = static_cast<int>(it - static_cast<int64_t>(c) * heads);
    const int left = a.ws_meta[x].moves - 32 * c;
    if (left <= 0) continue;
    const int32_t *table = a.tables + static_cast<int64_t>(x / a.H) * a.max_blocks;
    const int *places = a.ws_list + static_cast<int64_t>(x) * 2 * a.cap + 32 * c, *tokens = places + a.cap;
    float *weights = a.weights + static_cast<int64_t>(x) * a.stride;
    const int me = min(lane, left - 1), to = places[me], from = tokens[me];
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
  const int heads = a.rows * a.H;
  const int64_t items = static_cast<int64_t>((a.cap + 31) / 32) * heads, ctas = (items + 7) / 8;
  cudaError_t e = launch_overlapped(evict_move_kernel<LANES>, static_cast<int>(ctas < 8 * sms ? (ctas < 1 ? 1 : ctas) : 8 * sms),
                                    256, 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_overlapped(evict_shift_kernel<LANES>, heads, kShiftThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t stream) {
  const int heads = a.rows * a.H;
  // short rows: more CTAs an SM, whose barriers are cheaper
  if (a.stride <= 8192) evict_select_kernel<256><<<heads, 256, 0, stream>>>(a);
  else evict_select_kernel<512><<<heads, 512, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int pieces = (a.krow + a.vrow) / 16;
  return pieces <= 4 ? move<4>(a, sms, stream) : pieces <= 8 ? move<8>(a, sms, stream) : move<16>(a, sms, stream);
}

}  // namespace kvq
