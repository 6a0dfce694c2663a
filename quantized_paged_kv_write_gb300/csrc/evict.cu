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

constexpr int kSelectThreads = 1024;

struct RowPlan {
  int n, k, w, p;
};

// Sums v over the CTA's threads before this one; *total over all.
__device__ __forceinline__ unsigned scan_before(unsigned v, unsigned *sums, unsigned *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  const unsigned s = sums[lane];
  const unsigned before = __reduce_add_sync(0xffffffffu, lane < warp ? s : 0u);
  *total = __reduce_add_sync(0xffffffffu, s);
  __syncthreads();
  return before + x - v;
}

// Weights as unsigned numbers in the same order; -0 counts as 0, NaN as the largest.
__device__ __forceinline__ unsigned order_of(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const unsigned b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One CTA per (row, kv head): the threshold by four passes of eight bits over
// the candidates' weights, then the lists of places and of tokens to go there.
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ unsigned hist[256], sums[32];
  __shared__ unsigned chosen, left;
  const int r = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x;
  const int n = __ldg(a.ctx + r), keep = __ldg(a.keep + r), recent = __ldg(a.recent + r);
  const int pinned = a.pinned != nullptr ? __ldg(a.pinned + r) : 0;
  EvictMeta *meta = a.ws_meta + blockIdx.x;
  if (tid == 0) *meta = {0, 0, 0, 0};
  const bool range = n < 0 || n > a.max_len || keep < 0 || recent < 0 || pinned < 0;
  if (range || n <= keep) {
    if (tid == 0 && range) set_error(a.err, KVQ_DEVERR_CONTEXT_RANGE);
    if (tid == 0 && h == 0) a.kept[r] = n;
    return;
  }
  const int w = min(recent, keep), p = min(pinned, keep - w), end = keep - w;
  // every block of the row, and nobody else's among those to be written
  const int32_t *table = a.tables + static_cast<int64_t>(r) * a.max_blocks;
  bool bad = false, shared = false;
  for (int i = tid; i < (n + kBlockSize - 1) / kBlockSize; i += kSelectThreads) {
    const int id = __ldg(table + i);
    if (id < 0 || id >= a.num_blocks) bad = true;
    else if (a.refs != nullptr && i >= p / kBlockSize && i * kBlockSize < keep && __ldg(a.refs + id) != 1) shared = true;
  }
  bad = __syncthreads_or(bad);
  shared = __syncthreads_or(shared);
  if (bad || shared) {
    if (tid == 0) set_error(a.err, bad ? KVQ_DEVERR_BLOCK_RANGE : KVQ_DEVERR_POOL_STATE);
    if (tid == 0 && h == 0) a.kept[r] = n;
    return;
  }
  if (tid == 0 && h == 0) a.kept[r] = keep;
  const float *weights = a.weights + static_cast<int64_t>(blockIdx.x) * a.stride;
  const int last = n - w;  // candidates are [p, last)
  // ---- the need-th largest weight, and how many of its equals are kept
  unsigned prefix = 0, mask = 0, need = end - p;
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i = p + tid; i < last; i += kSelectThreads) {
        const unsigned key = order_of(weights[i]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      // digits from the largest: the one in which the need-th lies
      unsigned total;
      const unsigned own = tid < 256 ? hist[255 - tid] : 0u;
      const unsigned before = scan_before(own, sums, &total);
      if (own > 0 && before < need && need <= before + own) {
        chosen = 255 - tid;
        left = need - before;
      }
      __syncthreads();
      prefix |= chosen << shift;
      mask |= 255u << shift;
      need = left;
      __syncthreads();
    }
  }
  // ---- the lists
  int *places = a.ws_list + static_cast<int64_t>(blockIdx.x) * 2 * a.cap, *tokens = places + a.cap;
  unsigned ties = 0, holes = 0, late = 0;
  for (int base = p; base < last; base += kSelectThreads) {
    const int i = base + tid;
    const unsigned key = i < last ? order_of(weights[i]) : 0u;
    const bool equal = i < last && end > p && key == prefix;
    unsigned total;
    const unsigned rank = ties + scan_before(equal ? 1u : 0u, sums, &total);
    ties += total;
    const bool kept = i < last && end > p && (key > prefix || (equal && rank < need));
    const bool hole = i < end && !kept, goes = i >= end && kept;
    const unsigned at = scan_before((hole ? 1u : 0u) | (goes ? 0x10000u : 0u), sums, &total);
    if (hole) places[holes + (at & 0xFFFFu)] = i;
    if (goes) tokens[late + (at >> 16)] = i;
    holes += total & 0xFFFFu;
    late += total >> 16;
  }
  if (tid == 0) *meta = {static_cast<int>(late), 1, keep, w};
}

// The codes, scales and weight of one (row, head)'s token.
struct Mover {
  const EvictArgs &a;
  const int32_t *table;
  int h;
  __device__ __forceinline__ int64_t slot(int i) const {
    return (static_cast<int64_t>(__ldg(table + i / kBlockSize)) * kBlockSize + i % kBlockSize) * a.H + h;
  }
  // `part` of the token's pieces: 16-byte pieces of K's and V's codes, K's scale, V's scales
  __device__ __forceinline__ uint32_t *piece(int64_t s, int part, int *words) const {
    const int kp = a.krow / 16, vp = a.vrow / 16;
    *words = 4;
    if (part < kp) return reinterpret_cast<uint32_t *>(a.kc + s * a.krow) + 4 * part;
    part -= kp;
    if (part < vp) return reinterpret_cast<uint32_t *>(a.vc + s * a.vrow) + 4 * part;
    part -= vp;
    *words = 1;
    if (part == 0) return reinterpret_cast<uint32_t *>(a.ks + s);
    return reinterpret_cast<uint32_t *>(a.vs + s * a.vgroups) + part - 1;
  }
  __device__ __forceinline__ int parts() const { return a.krow / 16 + a.vrow / 16 + 1 + a.vgroups; }
};

// A warp's lanes have the pieces of one token.
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
  const int x = blockIdx.x, lane = threadIdx.x & 31;
  const EvictMeta meta = a.ws_meta[x];
  const Mover mv = {a, a.tables + static_cast<int64_t>(x / a.H) * a.max_blocks, x % a.H};
  const int *places = a.ws_list + static_cast<int64_t>(x) * 2 * a.cap, *tokens = places + a.cap;
  float *weights = a.weights + static_cast<int64_t>(x) * a.stride;
  for (int i = blockIdx.y * 8 + (threadIdx.x >> 5); i < meta.moves; i += gridDim.y * 8) {
    const int to = places[i], from = tokens[i];
    const int64_t st = mv.slot(to), sf = mv.slot(from);
    if (lane < mv.parts()) {
      int n;
      uint32_t *d = mv.piece(st, lane, &n);
      const uint32_t *s = mv.piece(sf, lane, &n);
      if (n == 4) *reinterpret_cast<uint4 *>(d) = *reinterpret_cast<const uint4 *>(s);
      else *d = *s;
    } else if (lane == 31) {
      weights[to] = weights[from];
    }
  }
}

// The last w tokens of a (row, head), which may overlap their new places: one
// CTA, in ascending order (a place is below its token).  Then weights past k.
__global__ void __launch_bounds__(1024) evict_shift_kernel(const EvictArgs a) {
  const int x = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const EvictMeta meta = a.ws_meta[x];
  if (!meta.active) return;
  const Mover mv = {a, a.tables + static_cast<int64_t>(x / a.H) * a.max_blocks, x % a.H};
  const int n = __ldg(a.ctx + x / a.H), w = meta.recent, k = meta.keep;
  float *weights = a.weights + static_cast<int64_t>(x) * a.stride;
  for (int base = 0; base < w; base += 32) {
    const int i = base + warp;
    const bool in = i < w;
    uint32_t *d = nullptr;
    int c = 0;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    float z = 0.f;
    if (in && lane < mv.parts()) {
      const uint32_t *s = mv.piece(mv.slot(n - w + i), lane, &c);
      d = mv.piece(mv.slot(k - w + i), lane, &c);
      if (c == 4) v = *reinterpret_cast<const uint4 *>(s);
      else v.x = *s;
    } else if (in && lane == 31) {
      z = weights[n - w + i];
    }
    __syncthreads();
    if (in && lane < mv.parts()) {
      if (c == 4) *reinterpret_cast<uint4 *>(d) = v;
      else *d = v.x;
    } else if (in && lane == 31) {
      weights[k - w + i] = z;
    }
    __syncthreads();
  }
  for (int i = k + static_cast<int>(threadIdx.x); i < n; i += 1024) weights[i] = 0.f;
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t stream) {
  const int heads = a.rows * a.H;
  evict_select_kernel<<<heads, kSelectThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // (rows <= 8192 and 8 heads: x holds what y cannot)
  evict_move_kernel<<<dim3(heads, (8 * sms + heads - 1) / heads), 256, 0, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  evict_shift_kernel<<<heads, 1024, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
