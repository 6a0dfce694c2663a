// Decode attention over a prefix that the sequences of a group share.
//
// What it computes: out[b, hq] = softmax(q k^T / sqrt(d)) V over the positions
// [0, context_len) of sequence b, as the paged decode does ("PidokuInfra 12 KV
// Cache Quantization", §5 The kernel side), where the first S positions of all
// sequences of a group lie in the same physical blocks (shared blocks:
// "Quantized KV caches in production", PagedAttention).  The softmax over the
// prefix of all (sequence, query head) rows that read one kv head is one
// matrix product, so the prefix is read once per group, not once per sequence.
// Prefix and suffix give partial states (m, l, O = sum 2^(z - m) v) in FP32,
// merged as sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i.
//
// Three steps around the suffix's split decode: the plan (what is shared, and
// the list of work), the prefix attention, and the merge.
#include <atomic>

#include "prefix_attend.cuh"

namespace kvq {
namespace {

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

// A sequence's context if it is valid, else 0 (the split decode's rule).
__device__ __forceinline__ int valid_ctx(const PrefixArgs &a, int b, bool &bad) {
  const int c = __ldg(a.ctx + b);
  const int64_t cap = static_cast<int64_t>(a.max_blocks) * kBlockSize + (a.res_k != nullptr ? kBlockSize - 1 : 0);
  bad = c < 0 || c > cap || c > a.max_ctx;
  return bad ? 0 : c;
}

__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PrefixArgs a) {
  __shared__ long long wt[kPlanThreads / 32], wr[kPlanThreads / 32];
  __shared__ int wn[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // ---- per group: how far its sequences share, and who holds the blocks
  for (int g = warp; g < a.groups; g += kPlanThreads / 32) {
    const int st = __ldg(a.group_starts + g), en = __ldg(a.group_starts + g + 1);
    const int pl = __ldg(a.prefix_lens + g);
    const bool range = st >= 0 && en >= st && en <= a.B;
    const bool len = pl >= 0 && pl <= a.max_prefix;
    int best = -1, lead = 0;
    if (range) {
      for (int b = st + lane; b < en; b += 32) {
        bool bad;
        const int c = valid_ctx(a, b, bad);
        if (c > best) {
          best = c;
          lead = b;
        }
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      const int c = __shfl_xor_sync(0xffffffffu, best, o), l = __shfl_xor_sync(0xffffffffu, lead, o);
      if (c > best || (c == best && l < lead)) {
        best = c;
        lead = l;
      }
    }
    if (lane == 0) {
      if (!range) set_error(a.err, KVQ_DEVERR_GROUP_RANGE);
      if (!len) set_error(a.err, KVQ_DEVERR_CONTEXT_RANGE);
      PrefixGroup r;
      r.start = st;
      r.nseq = range ? en - st : 0;
      // no further than the longest sequence: past it nothing was written
      r.shared = range && len ? max(0, min(pl, best)) / kBlockSize * kBlockSize : 0;
      r.lead = lead;
      a.ws_groups[g] = r;
    }
  }
  __syncthreads();
  // ---- the list of work
  long long t0 = 0, r0 = 0;
  int n0 = 0;
  for (int base = 0; base < a.groups; base += kPlanThreads) {
    const int g = base + threadIdx.x;
    PrefixGroup r = {};
    if (g < a.groups) r = a.ws_groups[g];
    // groups that overlap earlier ones (starts out of order) share nothing:
    // the sequences counted so far never exceed the batch
    int in = r.nseq;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += x;
    }
    if (lane == 31) wn[warp] = in;
    __syncthreads();
    int nb = n0;
    for (int w = 0; w < warp; ++w) nb = min(a.B + 1, nb + wn[w]);
    if (static_cast<long long>(nb) + in > a.B) {
      if (r.nseq > 0) set_error(a.err, KVQ_DEVERR_GROUP_RANGE);
      r.nseq = 0;
    }
    // a prefix of one sequence is that sequence's own
    if (r.nseq < 2 || r.shared == 0) r.nseq = r.shared = 0;
    const int R = r.nseq * a.G;
    r.row_blocks = (R + kPrefixRows - 1) / kPrefixRows;
    r.rows = R > 0 ? (R + r.row_blocks - 1) / r.row_blocks : 0;
    r.tiles = (r.shared + kPrefixTile - 1) / kPrefixTile;
    r.slots = r.rows > kPrefixRows / 2 ? r.rows : 2 * r.rows;
    const long long units = static_cast<long long>(r.row_blocks) * a.H;
    long long it = units * r.tiles, ir = units * r.slots;
    const long long t = it, rr = ir;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, it, o), y = __shfl_up_sync(0xffffffffu, ir, o);
      if (lane >= o) {
        it += x;
        ir += y;
      }
    }
    if (lane == 31) {
      wt[warp] = it;
      wr[warp] = ir;
    }
    __syncthreads();
    long long bt = t0, br = r0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w == warp) {
        bt = t0;
        br = r0;
      }
      t0 += wt[w];
      r0 += wr[w];
      n0 = min(a.B + 1, n0 + wn[w]);
    }
    r.tile0 = bt + it - t;
    r.row0 = br + ir - rr;
    if (g < a.groups) a.ws_groups[g] = r;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    PrefixGroup r = {};
    r.tile0 = t0;
    r.tiles = static_cast<int>(min(static_cast<long long>(a.nctas), t0));
    a.ws_groups[a.groups] = r;
  }
  __syncthreads();
  // ---- per sequence: where the prefix ends and the suffix begins
  for (int b = threadIdx.x; b < a.B; b += kPlanThreads) {
    int lo = 0, hi = a.groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.group_starts + mid) <= b) lo = mid; else hi = mid;
    }
    int g = -1, S = 0;
    if (a.groups > 0) {
      const PrefixGroup &r = a.ws_groups[lo];
      if (r.nseq > 0 && b >= r.start && b < r.start + r.nseq) {
        g = lo;
        S = r.shared;
      }
    }
    bool bad;
    const int c = valid_ctx(a, b, bad);
    if (bad) set_error(a.err, KVQ_DEVERR_CONTEXT_RANGE);
    const int cached = a.res_k != nullptr ? c / kBlockSize * kBlockSize : c;
    a.ws_group[b] = g;
    a.ws_limit[b] = min(cached, S);
    // a sequence that ends inside the prefix has no suffix but its tail
    a.ws_ctx[b] = c >= S ? c - S : c - cached;
    a.ws_off[b] = c >= S ? S / kBlockSize : 0;
  }
}

// ---------------------------------------------------------------------------
// merge: one warp per (sequence, query head)
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) prefix_merge_kernel(const PrefixArgs a) {
  constexpr int CPL = D / 32;  // channels per lane
  const int id = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (id >= a.B * a.Hq) return;
  const int b = id / a.Hq, hq = id % a.Hq, h = hq / a.G, gq = hq % a.G;
  float acc[CPL], L = 0.f, mx = -INFINITY;
#pragma unroll
  for (int k = 0; k < CPL; ++k) acc[k] = 0.f;

  // one more partial state with its output in o[0 .. CPL)
  auto add = [&](float m, float l, const float (&o)[CPL]) {
    if (m == -INFINITY) return;
    const float mn = fmaxf(mx, m);
    const float keep = exp2f(mx - mn), w = exp2f(m - mn);
    L = L * keep + w * l;
#pragma unroll
    for (int k = 0; k < CPL; ++k) acc[k] = acc[k] * keep + w * o[k];
    mx = mn;
  };
  auto load = [&](const float *p, float (&o)[CPL]) {
#pragma unroll
    for (int k = 0; k < CPL; ++k) o[k] = p[lane * CPL + k];
  };

  // ---- prefix
  const int gi = a.ws_group[b];
  if (gi >= 0) {
    const PrefixGroup g = a.ws_groups[gi];
    const int row = (b - g.start) * a.G + gq;
    const int rb = row / g.rows, r = row % g.rows, u = rb * a.H + h;
    const int64_t T = a.ws_groups[a.groups].tile0;
    const int64_t x0 = g.tile0 + static_cast<int64_t>(u) * g.tiles;
    // the CTA that holds tile x of the list
    const int P = a.ws_groups[a.groups].tiles;
    auto cta_of = [&](int64_t x) { return static_cast<int>(min(static_cast<int64_t>(P - 1), ((x + 1) * P - 1) / T)); };
    const int c0 = cta_of(x0), c1 = cta_of(x0 + g.tiles - 1);
    for (int c = c0; c <= c1; ++c) {
      for (int s = 0; s < (g.slots > g.rows ? 2 : 1); ++s) {
        const int64_t at = g.row0 + static_cast<int64_t>(u) * g.slots + static_cast<int64_t>(c) * kPrefixRows + s * g.rows + r;
        const float2 ml = *reinterpret_cast<const float2 *>(a.ws_ml + at * 2);
        if (ml.x == -INFINITY) continue;
        float o[CPL];
        load(a.ws_o + at * D, o);
        add(ml.x, ml.y, o);
      }
    }
  }
  // ---- suffix: the split decode's partials
  const int s0 = a.sfx_cum[b], s1 = a.sfx_cum[b + 1];
  if (s1 > s0) {
    const int total = a.sfx_cum[a.B];
    const int P = min(a.sfx_nctas, max(1, (total + a.sfx_blocks_per_cta - 1) / a.sfx_blocks_per_cta));
    auto cta_of = [&](int x) {
      const int64_t v = ((static_cast<int64_t>(x) + 1) * P - 1) / total;
      return static_cast<int>(v < P - 1 ? v : P - 1);
    };
    const bool packed = 2 * a.G <= 8;  // columns g (high) and g + G (low)
    for (int c = cta_of(s0); c <= cta_of(s1 - 1); ++c) {
      const int64_t rec = (static_cast<int64_t>(b) + c) * a.H + h;
      const float2 ml = *reinterpret_cast<const float2 *>(a.sfx_ml + (rec * 8 + gq) * 2);
      if (ml.x == -INFINITY) continue;
      float o[CPL];
      load(a.sfx_o + (rec * 8 + gq) * D, o);
      if (packed) {
        float y[CPL];
        load(a.sfx_o + (rec * 8 + gq + a.G) * D, y);
#pragma unroll
        for (int k = 0; k < CPL; ++k) o[k] += y[k];
      }
      add(ml.x, ml.y, o);
    }
  }
  // ---- the full-precision tail of a per-channel K cache
  if (a.res_k != nullptr) {
    const int nt = a.ws_ctx[b] % kBlockSize;
    const uint16_t *q = a.q + static_cast<int64_t>(id) * D + lane * CPL;
    const float zs = rsqrtf(static_cast<float>(D)) * kLog2e;
    for (int t = 0; t < nt; ++t) {
      const int64_t at = ((static_cast<int64_t>(b) * kBlockSize + t) * a.H + h) * D + lane * CPL;
      float dot = 0.f, o[CPL];
#pragma unroll
      for (int k = 0; k < CPL; ++k) {
        dot += bf16lo_to_f32(q[k]) * bf16lo_to_f32(a.res_k[at + k]);
        o[k] = bf16lo_to_f32(a.res_v[at + k]);
      }
#pragma unroll
      for (int s = 16; s >= 1; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
      add(dot * zs, 1.f, o);
    }
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
  for (int k = 0; k < CPL; ++k) acc[k] *= inv;
  if (a.rot) {
    // back from the rotated basis: sigma * (H o) / d, stages below CPL inside
    // the lane, the others across lanes
#pragma unroll
    for (int s = 1; s < CPL; s <<= 1)
#pragma unroll
      for (int k = 0; k < CPL; ++k)
        if (!(k & s)) {
          const float x = acc[k], y = acc[k + s];
          acc[k] = x + y;
          acc[k + s] = x - y;
        }
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
#pragma unroll
      for (int k = 0; k < CPL; ++k) {
        const float p = __shfl_xor_sync(0xffffffffu, acc[k], s);
        acc[k] = (lane & s) ? p - acc[k] : acc[k] + p;
      }
    }
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
      const int ch = lane * CPL + k;
      const float x = acc[k] * (1.f / D);
      acc[k] = (a.rot_signs[ch >> 5] >> (ch & 31)) & 1u ? -x : x;
    }
  }
  // BF16 out, rounded once: what the output projection reads
  uint32_t *out = reinterpret_cast<uint32_t *>(a.out + static_cast<int64_t>(id) * D + lane * CPL);
#pragma unroll
  for (int k = 0; k < CPL; k += 2) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(acc[k + 1]), "f"(acc[k]));
    out[k / 2] = w;
  }
}

}  // namespace

cudaError_t launch_prefix_plan(const PrefixArgs &a, cudaStream_t stream) {
  prefix_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D>
static cudaError_t attend(int kf, int vf, const PrefixArgs &a, const DecodeMaps &m, cudaStream_t stream) {
  auto kern = prefix::prefix_attend_kernel<D>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  static std::atomic<unsigned long long> done{0};  // devices whose limit is raised
  if (!((done.load(std::memory_order_acquire) >> dev) & 1ull)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, prefix::kMaxSmem)) != cudaSuccess)
      return e;
    done.fetch_or(1ull << dev, std::memory_order_acq_rel);
  }
  // a batch that cannot fill more than one row tile gives the other one's
  // place to the ring of codes
  const int krow = kf == K_INT4_TOK ? D / 2 : kf == K_INT2_CHAN ? D / 4 : D;
  const int vrow = vf == V_INT4_G32 ? D / 2 : vf == V_INT2_G32 ? D / 4 : D;
  const prefix::Layout y = prefix::layout_of<D>(kf == K_INT8_CHAN || kf == K_INT2_CHAN, vf == V_INT4_G32 || vf == V_INT2_G32,
                                                a.B * a.G > kPrefixRows / 2, krow, vrow);
  kern<<<a.nctas, prefix::kThreads, y.bytes, stream>>>(m.k, m.v, a, y, kf, vf, krow, vrow);
  return cudaGetLastError();
}

cudaError_t launch_prefix_attend(int head_dim, int kf, int vf, const PrefixArgs &a, const DecodeMaps &m,
                                 cudaStream_t stream) {
  return head_dim == 128 ? attend<128>(kf, vf, a, m, stream) : attend<64>(kf, vf, a, m, stream);
}

cudaError_t launch_prefix_merge(int head_dim, const PrefixArgs &a, cudaStream_t stream) {
  const int n = (a.B * a.Hq + 7) / 8;
  if (head_dim == 128) prefix_merge_kernel<128><<<n, 256, 0, stream>>>(a);
  else prefix_merge_kernel<64><<<n, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
