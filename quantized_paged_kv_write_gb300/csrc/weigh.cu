// Attention weights of the cached tokens, out of the scores that the paged
// decode's split kernel leaves behind.
//
// What it computes: weights[b, h, t] += sum over the query heads of kv head h of
// softmax(q k^T / sqrt(d))_t for every cached token t of sequence b.  The split
// writes its scores z (log2 units, FP32), the reduce each row's maximum m and
// 1 / sum; a weight is 2^(z - m) / sum, formed and summed in FP32.
//
// Why the scores and not K again: a token and kv head has 4 G bytes of scores,
// written once and read once, against d bytes of codes and all of the decode's
// products.  27 sequences of 32768 tokens, 32 heads on 8, FP8: the split takes
// 309 us with the scores (278 without: 113 MB more), the weights 26 us (170 MB,
// 6.4 TB/s) and the reduce 7.  What the decode reads bounds the call: 343 us where
// its bytes and the weights' take 285.  The split with scores is a kernel of its
// own: a run-time branch slowed the plain decode by up to 4.5 %.
#include "common.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kWarps = 8;

// The last sequence that begins at or before block g of the list, by 32 samples
// at a time.
__device__ __forceinline__ int sequence_of(const int *cum, int B, int g, int lane) {
  int lo = 0, n = B;  // in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const unsigned in = __ballot_sync(0xffffffffu, lane * step < n && cum[at] <= g);
    const int k = 31 - __clz(in);  // (lane 0's is)
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// w[k] of lane i (of four) to w[i] of lane k.
__device__ __forceinline__ void transpose4(float (&w)[4], int i) {
#pragma unroll
  for (int s = 1; s < 4; s <<= 1) {
    const bool up = i & s;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & s) continue;
      const float give = up ? w[k] : w[k + s], got = __shfl_xor_sync(0xffffffffu, give, s);
      if (up) w[k] = got; else w[k + s] = got;
    }
  }
}

// A warp takes an even, contiguous part of the blocks, N of them at a time (8 / H
// side by side, the rest in turn); four lanes have one head of a block, first
// four tokens i, i + 4, .. each, as the scores lie, then four in a row, as the
// weights do.  G query heads in registers: their maxima and sums change with the
// sequence alone.  Bound by memory: scores once, weights read and written.
// VEC: rows of weights on 16-byte boundaries.
template <int G, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) weigh_kernel(const WeighArgs a) {
  constexpr int U = G <= 2 ? 4 : G <= 4 ? 2 : 1;  // blocks of a lane in flight
  const int lane = threadIdx.x & 31, i = lane & 3;
  const int side = 8 / a.H, sub = lane / (4 * a.H), h = lane / 4 % a.H;
  const bool mine = sub < side;
  grid_wait();  // maxima and sums
  const int total = a.cum[a.B];
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), W = static_cast<int64_t>(gridDim.x) * kWarps;
  const int g0 = static_cast<int>(w * total / W), g1 = static_cast<int>((w + 1) * total / W);
  if (g0 >= g1) return;
  int b = sequence_of(a.cum, a.B, g0, lane);
  for (int g = g0; g < g1;) {
    const int begin = a.cum[b], end = min(a.cum[b + 1], g1);
    if (end <= g) {  // an empty sequence
      ++b;
      continue;
    }
    const int n = a.ctx[b];
    float2 s[G];
#pragma unroll
    for (int q = 0; q < G; ++q) s[q] = a.norm[(static_cast<int64_t>(b) * a.H + h) * G + q];
    const int32_t *table = a.tables + static_cast<int64_t>(b) * a.max_blocks;
    float *row = a.weights + (static_cast<int64_t>(b) * a.H + h) * a.stride;
    for (; g < end; g += side * U) {
      float4 z[U][G], old[U];
      bool go[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int x = g + u * side + sub, t = (x - begin) * kBlockSize + 4 * i;
        go[u] = mine && x < end;
        if (!go[u]) continue;
        const int id = table[x - begin];
        const float4 *from = reinterpret_cast<const float4 *>(a.z + (static_cast<int64_t>(x) * a.H + h) * (G * kBlockSize)) + i;
#pragma unroll
        for (int q = 0; q < G; ++q) z[u][q] = __ldcs(from + 4 * q);
        if (VEC && t + 4 <= n) {
          old[u] = *reinterpret_cast<const float4 *>(row + t);
        } else {
          if (t < n) old[u].x = row[t];
          if (t + 1 < n) old[u].y = row[t + 1];
          if (t + 2 < n) old[u].z = row[t + 2];
          if (t + 3 < n) old[u].w = row[t + 3];
        }
        go[u] = id >= 0 && id < a.num_blocks;  // (else the decode left no scores)
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float p[4] = {0.f, 0.f, 0.f, 0.f};
        if (go[u]) {
#pragma unroll
          for (int q = 0; q < G; ++q) {
            p[0] = fmaf(fast_exp2(z[u][q].x - s[q].x), s[q].y, p[0]);
            p[1] = fmaf(fast_exp2(z[u][q].y - s[q].x), s[q].y, p[1]);
            p[2] = fmaf(fast_exp2(z[u][q].z - s[q].x), s[q].y, p[2]);
            p[3] = fmaf(fast_exp2(z[u][q].w - s[q].x), s[q].y, p[3]);
          }
        }
        transpose4(p, i);
        const int t = (g + u * side + sub - begin) * kBlockSize + 4 * i;
        if (!go[u]) continue;
        if (VEC && t + 4 <= n) {
          *reinterpret_cast<float4 *>(row + t) = make_float4(old[u].x + p[0], old[u].y + p[1], old[u].z + p[2], old[u].w + p[3]);
        } else {
          if (t < n) row[t] = old[u].x + p[0];
          if (t + 1 < n) row[t + 1] = old[u].y + p[1];
          if (t + 2 < n) row[t + 2] = old[u].z + p[2];
          if (t + 3 < n) row[t + 3] = old[u].w + p[3];
        }
      }
    }
    g = end;
    ++b;
  }
}

template <int G>
cudaError_t launch_g(const WeighArgs &a, int sms, cudaStream_t stream) {
  const bool vec = a.stride % 4 == 0 && (reinterpret_cast<uintptr_t>(a.weights) & 15u) == 0;
  const int64_t ctas = (a.most_blocks + kWarps - 1) / kWarps;  // a block for each warp
  return launch_overlapped(vec ? weigh_kernel<G, true> : weigh_kernel<G, false>,
                           dim3(static_cast<unsigned>(ctas < 1 ? 1 : ctas < 8 * sms ? ctas : 8 * sms)), 32 * kWarps, 0, stream, a);
}

}  // namespace

cudaError_t launch_weigh(const WeighArgs &a, int sms, cudaStream_t stream) {
  switch (a.G) {
    case 1: return launch_g<1>(a, sms, stream);
    case 2: return launch_g<2>(a, sms, stream);
    case 3: return launch_g<3>(a, sms, stream);
    case 4: return launch_g<4>(a, sms, stream);
    case 5: return launch_g<5>(a, sms, stream);
    case 6: return launch_g<6>(a, sms, stream);
    case 7: return launch_g<7>(a, sms, stream);
    case 8: return launch_g<8>(a, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
