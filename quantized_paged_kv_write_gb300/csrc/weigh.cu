// Attention weights of the cached tokens, out of the scores that the paged
// decode's split kernel leaves behind.
//
// What it computes: weights[b, h, t] += sum over the query heads of kv head h of
// softmax(q k^T / sqrt(d))_t for every cached token t of sequence b.  The split
// writes its scores z (log2 units, 4 bytes for each query head, where reading K
// again would take d code bytes), the reduce each row's maximum m and 1 / sum;
// a weight is 2^(z - m) / sum.
#include "common.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

// One warp per block of the list; a lane has tokens i, i + 4, .. of a head.
__global__ void __launch_bounds__(256) weigh_kernel(const WeighArgs a) {
  const int lane = threadIdx.x & 31;
  const int total = a.cum[a.B], step = gridDim.x * 8;
  for (int g = blockIdx.x * 8 + (threadIdx.x >> 5); g < total; g += step) {
    int lo = 0, hi = a.B;  // the last sequence that begins at or before g
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cum[mid] <= g) lo = mid; else hi = mid;
    }
    const int b = lo, j = g - a.cum[b], n = a.ctx[b];
    const int id = a.tables[static_cast<int64_t>(b) * a.max_blocks + j];
    if (id < 0 || id >= a.num_blocks) continue;  // (no scores)
    for (int x = lane; x < 4 * a.H; x += 32) {
      const int h = x / 4, i = x % 4;
      float w[4] = {0.f, 0.f, 0.f, 0.f};
      for (int q = 0; q < a.G; ++q) {
        const float4 z = *reinterpret_cast<const float4 *>(
            a.z + ((static_cast<int64_t>(g) * a.H + h) * a.G + q) * kBlockSize + 4 * i);
        const float2 s = a.norm[(b * a.H + h) * a.G + q];
        w[0] += exp2f(z.x - s.x) * s.y;
        w[1] += exp2f(z.y - s.x) * s.y;
        w[2] += exp2f(z.z - s.x) * s.y;
        w[3] += exp2f(z.w - s.x) * s.y;
      }
      float *to = a.weights + (static_cast<int64_t>(b) * a.H + h) * a.stride;
      for (int k = 0; k < 4; ++k) {
        const int t = j * kBlockSize + i + 4 * k;
        if (t < n) to[t] += w[k];
      }
    }
  }
}

}  // namespace

cudaError_t launch_weigh(const WeighArgs &a, int sms, cudaStream_t stream) {
  weigh_kernel<<<8 * sms, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
