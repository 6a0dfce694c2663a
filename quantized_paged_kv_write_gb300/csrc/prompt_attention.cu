// Causal attention over packed prompts.
//
// What it computes: for token t of a sequence and query head h, which reads kv
// head h / G (GQA, "KV Cache Quantization" glossary), over the sequence's
// tokens j <= t:  z_j = q_t k_j / sqrt(d), out = sum softmax(z)_j v_j and
// lse = ln sum exp(z_j).  It is the attention of the prefill whose K and V the
// quantize-write stores ("Use Less Memory: Quantization and Offloading", §2.1).
#include "common.cuh"
#include "kvq_internal.h"

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
  // offsets in order and in range, or nothing is computed
  bool order = true;
  for (int s = threadIdx.x; s < a.num_seqs; s += kPlanThreads) {
    const int x = __ldg(a.offsets + s), y = __ldg(a.offsets + s + 1);
    order = order && x >= 0 && y >= x && y <= a.num_tokens;
    if (y >= x && y - x > a.max_seq) set_error(a.err, KVQ_DEVERR_CONTEXT_RANGE);
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
  // how many sequences have j tiles
  auto tiles = [&](int s, int *start, int *len) {
    const int x = __ldg(a.offsets + s), y = __ldg(a.offsets + s + 1);
    *start = x;
    *len = y - x > a.max_seq ? 0 : y - x;
    return (*len + a.unit - 1) / a.unit;
  };
  int start, len;
  for (int s = threadIdx.x; s < a.num_seqs; s += kPlanThreads) atomicAdd(a.ws_level + tiles(s, &start, &len), 1);
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
// attention: one warp per row (token, query head)
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) prompt_attend_kernel(const PromptArgs a) {
  constexpr int CPL = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float c = rsqrtf(static_cast<float>(D));
  for (int x = blockIdx.x; x < a.ws_head->units; x += gridDim.x) {
    const Unit u = unit_at(a, x);
    const int rows = min(a.unit, u.len - u.t0) * a.G;
    for (int r = warp; r < rows; r += 8) {
      const int t = u.t0 + r / a.G, hq = u.h * a.G + r % a.G;
      const int64_t row = u.start + t;
      float q[CPL], o[CPL], m = -INFINITY, l = 0.f;
      for (int e = 0; e < CPL; ++e) {
        q[e] = c * __uint_as_float(static_cast<uint32_t>(a.q[row * a.q_stride + hq * D + lane * CPL + e]) << 16);
        o[e] = 0.f;
      }
      for (int j = 0; j <= t; ++j) {
        const uint16_t *k = a.k + (static_cast<int64_t>(u.start) + j) * a.k_stride + u.h * D + lane * CPL;
        const uint16_t *v = a.v + (static_cast<int64_t>(u.start) + j) * a.v_stride + u.h * D + lane * CPL;
        float z = 0.f;
        for (int e = 0; e < CPL; ++e) z += q[e] * __uint_as_float(static_cast<uint32_t>(k[e]) << 16);
        for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
        const float mn = fmaxf(m, z), keep = expf(m - mn), p = expf(z - mn);
        l = l * keep + p;
        for (int e = 0; e < CPL; ++e) o[e] = o[e] * keep + p * __uint_as_float(static_cast<uint32_t>(v[e]) << 16);
        m = mn;
      }
      for (int e = 0; e < CPL; ++e) {
        uint32_t w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(0.f), "f"(o[e] / l));
        a.out[(row * a.Hq + hq) * D + lane * CPL + e] = static_cast<uint16_t>(w);
      }
      if (a.lse != nullptr && lane == 0) a.lse[row * a.Hq + hq] = m + logf(l);
    }
  }
}

}  // namespace

cudaError_t launch_prompt_attention(int head_dim, const PromptArgs &a, int sms, cudaStream_t stream) {
  prompt_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (head_dim == 128) prompt_attend_kernel<128><<<8 * sms, 256, 0, stream>>>(a);
  else prompt_attend_kernel<64><<<8 * sms, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
