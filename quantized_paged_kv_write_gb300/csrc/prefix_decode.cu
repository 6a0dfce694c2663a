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
// merge
// ---------------------------------------------------------------------------
// A CTA merges kMergeRows rows of one kv head (row = sequence * G + query head
// of the group, as the units count them); a thread has 4 channels of a row, so
// the rows' 16-byte pieces of a partial are consecutive in memory.  Bound by the
// latency of the partials in L2 (up to ~40 of them for a row): eight are in
// flight at a time.
constexpr int kMergeRows = 8;

template <int D>
__global__ void __launch_bounds__(kMergeRows *D / 4) prefix_merge_kernel(const PrefixArgs a) {
  constexpr int CG = D / 4;  // channel groups
  constexpr int U = 8;
  __shared__ float sh[kMergeRows][D + 4];
  const int rl = threadIdx.x % kMergeRows, cg = threadIdx.x / kMergeRows;
  const int h = blockIdx.x % a.H, row = blockIdx.x / a.H * kMergeRows + rl;
  const bool live = row < a.B * a.G;
  const int b = live ? row / a.G : 0, gq = live ? row % a.G : 0;

  // ---- where the row's partials are: prefix (CTA c of its unit, one or two
  // streams), then suffix (the split decode's)
  int n0 = 0, streams = 1, prows = 0, n1 = 0;
  int64_t pslot = 0, srec = 0;
  const int gi = live ? a.ws_group[b] : -1;
  if (gi >= 0) {
    const PrefixGroup g = a.ws_groups[gi];
    const int r = (b - g.start) * a.G + gq, rb = r / g.rows, u = rb * a.H + h;
    const int T = static_cast<int>(a.ws_groups[a.groups].tile0), P = a.ws_groups[a.groups].tiles;
    const int x0 = static_cast<int>(g.tile0) + u * g.tiles;
    // the CTA that holds tile x of the list
    auto cta_of = [&](int x) { return min(P - 1, static_cast<int>(((static_cast<int64_t>(x) + 1) * P - 1) / T)); };
    const int c0 = cta_of(x0), c1 = cta_of(x0 + g.tiles - 1);
    streams = g.slots > g.rows ? 2 : 1;
    prows = g.rows;
    n0 = (c1 - c0 + 1) * streams;
    pslot = g.row0 + static_cast<int64_t>(u) * g.slots + static_cast<int64_t>(c0) * kPrefixRows;
    srec = r % g.rows;  // (the row in its block, for now)
  }
  const int prow = static_cast<int>(srec);
  const bool packed = 2 * a.G <= 8;  // suffix columns g (high) and g + G (low)
  if (live) {
    const int s0 = a.sfx_cum[b], s1 = a.sfx_cum[b + 1];
    if (s1 > s0) {
      const int total = a.sfx_cum[a.B];
      const int P = min(a.sfx_nctas, max(1, (total + a.sfx_blocks_per_cta - 1) / a.sfx_blocks_per_cta));
      auto cta_of = [&](int x) { return min(P - 1, static_cast<int>(((static_cast<int64_t>(x) + 1) * P - 1) / total)); };
      const int c0 = cta_of(s0);
      n1 = cta_of(s1 - 1) - c0 + 1;
      srec = ((static_cast<int64_t>(b) + c0) * a.H + h) * 8 + gq;
    }
  }
  auto ml_of = [&](int i) -> float2 {
    if (i < n0) {
      const int64_t at = pslot + static_cast<int64_t>(i / streams) * kPrefixRows + (i % streams) * prows + prow;
      return *reinterpret_cast<const float2 *>(a.ws_ml + at * 2);
    }
    return *reinterpret_cast<const float2 *>(a.sfx_ml + (srec + static_cast<int64_t>(i - n0) * a.H * 8) * 2);
  };
  auto o_of = [&](int i) -> float4 {
    if (i < n0) {
      const int64_t at = pslot + static_cast<int64_t>(i / streams) * kPrefixRows + (i % streams) * prows;
      return reinterpret_cast<const float4 *>(a.ws_o + at * D)[cg * prows + prow];
    }
    const float *p = a.sfx_o + (srec + static_cast<int64_t>(i - n0) * a.H * 8) * D + 4 * cg;
    float4 v = *reinterpret_cast<const float4 *>(p);
    if (packed) {
      const float4 y = *reinterpret_cast<const float4 *>(p + a.G * D);
      v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
    }
    return v;
  };
  const int n = n0 + n1;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float L = 0.f, mx = -INFINITY;
  for (int i = 0; i < n; i += U) {
    // a batch's largest m, then its weighted sum; partials without weight (a
    // warpgroup that had no tile, a row masked there) hold no O
    float2 ml[U];
#pragma unroll
    for (int k = 0; k < U; ++k) ml[k] = i + k < n ? ml_of(i + k) : make_float2(-INFINITY, 0.f);
    float4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) v[k] = i + k < n ? o_of(i + k) : make_float4(0.f, 0.f, 0.f, 0.f);
    float mn = mx;
#pragma unroll
    for (int k = 0; k < U; ++k) mn = fmaxf(mn, ml[k].x);
    if (mn == -INFINITY) continue;
    const float keep = exp2f(mx - mn);
    mx = mn;
    L *= keep;
    acc.x *= keep; acc.y *= keep; acc.z *= keep; acc.w *= keep;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (ml[k].x == -INFINITY) continue;
      const float w = exp2f(ml[k].x - mn);
      L = fmaf(w, ml[k].y, L);
      acc.x = fmaf(w, v[k].x, acc.x);
      acc.y = fmaf(w, v[k].y, acc.y);
      acc.z = fmaf(w, v[k].z, acc.z);
      acc.w = fmaf(w, v[k].w, acc.w);
    }
  }
  // ---- the full-precision tail of a per-channel K cache (products summed over
  // the row's threads in shared memory)
  if (a.res_k != nullptr) {
    const int nt = live ? a.ws_ctx[b] % kBlockSize : 0;
    const uint2 qw = live ? *reinterpret_cast<const uint2 *>(a.q + (static_cast<int64_t>(b) * a.Hq + h * a.G + gq) * D + 4 * cg)
                          : make_uint2(0u, 0u);
    const float zs = rsqrtf(static_cast<float>(D)) * kLog2e;
    for (int t = 0; t < kBlockSize; ++t) {
      const bool in = t < nt;
      const int64_t at = ((static_cast<int64_t>(b) * kBlockSize + t) * a.H + h) * D + 4 * cg;
      float dot = 0.f;
      if (in) {
        const uint2 k = *reinterpret_cast<const uint2 *>(a.res_k + at);
        dot = bf16lo_to_f32(qw.x) * bf16lo_to_f32(k.x) + bf16hi_to_f32(qw.x) * bf16hi_to_f32(k.x) +
              bf16lo_to_f32(qw.y) * bf16lo_to_f32(k.y) + bf16hi_to_f32(qw.y) * bf16hi_to_f32(k.y);
      }
      // lanes rl, rl + 8, .. of a warp share a row; then the warps
#pragma unroll
      for (int o = kMergeRows; o < 32; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      __syncthreads();
      if ((threadIdx.x & 31) < kMergeRows) sh[rl][threadIdx.x >> 5] = dot;
      __syncthreads();
      if (in) {
        float z = 0.f;
        for (int w = 0; w < kMergeRows * CG / 32; ++w) z += sh[rl][w];
        z *= zs;
        const uint2 v = *reinterpret_cast<const uint2 *>(a.res_v + at);
        const float mn = fmaxf(mx, z), keep = exp2f(mx - mn), p = exp2f(z - mn);
        mx = mn;
        L = L * keep + p;
        acc.x = acc.x * keep + p * bf16lo_to_f32(v.x);
        acc.y = acc.y * keep + p * bf16hi_to_f32(v.x);
        acc.z = acc.z * keep + p * bf16lo_to_f32(v.y);
        acc.w = acc.w * keep + p * bf16hi_to_f32(v.y);
      }
    }
    __syncthreads();
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
  if (a.rot) {
    // back from the rotated basis, sigma * (H o) / d: stages 1 and 2 in the
    // thread, the others between threads through shared memory
    float t0 = acc.x + acc.y, t1 = acc.x - acc.y, t2 = acc.z + acc.w, t3 = acc.z - acc.w;
    float4 y = make_float4(t0 + t2, t1 + t3, t0 - t2, t1 - t3);
#pragma unroll
    for (int s = 1; s < CG; s <<= 1) {
      *reinterpret_cast<float4 *>(&sh[rl][4 * cg]) = y;
      __syncthreads();
      const float4 p = *reinterpret_cast<const float4 *>(&sh[rl][4 * (cg ^ s)]);
      const float f = (cg & s) ? -1.f : 1.f;
      y = make_float4(fmaf(f, y.x, p.x), fmaf(f, y.y, p.y), fmaf(f, y.z, p.z), fmaf(f, y.w, p.w));
      __syncthreads();
    }
    const uint32_t neg = a.rot_signs[cg >> 3] >> (4 * (cg & 7));
    constexpr float kInvD = 1.f / D;
    acc.x = y.x * (neg & 1u ? -kInvD : kInvD);
    acc.y = y.y * (neg & 2u ? -kInvD : kInvD);
    acc.z = y.z * (neg & 4u ? -kInvD : kInvD);
    acc.w = y.w * (neg & 8u ? -kInvD : kInvD);
  }
  // BF16 out, rounded once: what the output projection reads
  if (live) {
    uint2 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(acc.y), "f"(acc.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(acc.w), "f"(acc.z));
    *reinterpret_cast<uint2 *>(a.out + (static_cast<int64_t>(b) * a.Hq + h * a.G + gq) * D + 4 * cg) = w;
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
  const int n = (a.B * a.G + kMergeRows - 1) / kMergeRows * a.H;
  if (head_dim == 128) prefix_merge_kernel<128><<<n, kMergeRows * 32, 0, stream>>>(a);
  else prefix_merge_kernel<64><<<n, kMergeRows * 16, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
