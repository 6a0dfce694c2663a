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
// the list of work), the prefix attention, and the merge.  Each kernel is
// launched while the one before runs; one after the other they took 7 to 12 us
// more.  27 sequences, 32 query heads on 8, FP8, 32003 shared positions and
// 1000 of each one's own: plan 4 us, attention 35, then 14 for the suffixes
// (55 MB) and 12 for the merge, 66 in all.
#include <limits.h>

#include <atomic>

#include "prefix_attend.cuh"

namespace kvq {
namespace {

// The plan and the merge run once a call, in microseconds.  What they cost is
// first of all fetching their code (it left the instruction caches while the
// prefix kernel ran): loops stay rolled, sums are in 32 bits, divisions few.

// The CTA of P that holds item x of T shared out as [c T / P, (c + 1) T / P):
// floor(((x + 1) P - 1) / T) by a reciprocal that is off by less than one.
__device__ __noinline__ int cta_of(int x, int T, int P) {
  const unsigned long long n = (static_cast<unsigned long long>(x) + 1) * static_cast<unsigned>(P) - 1;
  unsigned q = static_cast<unsigned>(static_cast<float>(n) * __frcp_rn(static_cast<float>(T)));
  if (static_cast<unsigned long long>(q) * static_cast<unsigned>(T) > n) --q;
  if (static_cast<unsigned long long>(q + 1) * static_cast<unsigned>(T) <= n) ++q;
  return min(static_cast<int>(q), P - 1);
}

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kMaxShared = INT_MAX - 255;  // so that the last tile's end counts in 32 bits, too

// One CTA: a chain of dependent loads and a few barriers.  The records of up to
// kPlanGroups groups stay in shared memory between the steps.
constexpr int kPlanGroups = 256;
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PrefixArgs a) {
  __shared__ PrefixGroup sh[kPlanGroups];
  __shared__ int2 sums[kPlanThreads / 32];
  grid_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  PrefixGroup *const rec = a.groups <= kPlanGroups ? sh : a.ws_groups;
  // a sequence's context if it is valid, else 0 (the split decode's rule)
  auto context = [&](int b) {
    const int c = __ldg(a.ctx + b);
    return c < 0 || c > a.ctx_cap ? 0 : c;
  };
  // ---- per group: how far its sequences share, and who holds the blocks
  bool order = true;
#pragma unroll 1
  for (int g = warp; g < a.groups; g += kPlanThreads / 32) {
    const int st = __ldg(a.group_starts + g), en = __ldg(a.group_starts + g + 1), pl = __ldg(a.prefix_lens + g);
    const bool range = st >= 0 && en >= st && en <= a.B, len = pl >= 0 && pl <= a.max_prefix;
    order = order && range;
    if (!len && lane == 0) set_error(a.err, KVQ_DEVERR_CONTEXT_RANGE);
    // the longest context, and the first sequence that has it
    int best = 0, lead = st;
    if (range)
#pragma unroll 1
      for (int b = st + lane; b < en; b += 32) {
        const int c = context(b);
        if (c > best) {
          best = c;
          lead = b;
        }
      }
    const int most = __reduce_max_sync(0xffffffffu, best);
    lead = __reduce_min_sync(0xffffffffu, best == most ? lead : INT_MAX);
    if (lane == 0) {
      // no further than the longest sequence: past it nothing was written; a
      // prefix of one sequence is that sequence's own
      const int S = range && len && en - st >= 2 ? min(min(pl, most), kMaxShared) / kBlockSize * kBlockSize : 0;
      const int R = S > 0 ? (en - st) * a.G : 0;
      PrefixGroup r;
      r.start = st;
      r.nseq = S > 0 ? en - st : 0;
      r.shared = S;
      r.lead = lead;
      r.row_blocks = (R + kPrefixRows - 1) / kPrefixRows;
      r.rows = R > kPrefixRows ? (R + r.row_blocks - 1) / r.row_blocks : R;
      r.tiles = (S + kPrefixTile - 1) / kPrefixTile;
      r.tile0 = r.row0 = 0;
      rec[g] = r;
    }
  }
  // groups out of order or range may overlap: then nothing is shared
  const bool none = __syncthreads_or(!order);
  if (none && threadIdx.x == 0) set_error(a.err, KVQ_DEVERR_GROUP_RANGE);
  // ---- the list of work
  int t0 = 0, r0 = 0;
#pragma unroll 1
  for (int base = 0; base < a.groups; base += kPlanThreads) {
    const int g = base + threadIdx.x;
    PrefixGroup r = {};
    if (g < a.groups) r = rec[g];
    if (none) r.nseq = r.shared = r.row_blocks = r.tiles = 0;
    const int t = r.row_blocks * a.H * r.tiles, s = r.row_blocks * a.H * r.rows;
    int it = t, is = s;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, it, o), y = __shfl_up_sync(0xffffffffu, is, o);
      if (lane >= o) {
        it += x;
        is += y;
      }
    }
    if (lane == 31) sums[warp] = make_int2(it, is);
    __syncthreads();
    const int2 w = sums[lane];  // every warp sums the warps' totals for itself
    const bool before = lane < warp;
    r.tile0 = t0 + it - t + __reduce_add_sync(0xffffffffu, before ? w.x : 0);
    r.row0 = r0 + is - s + __reduce_add_sync(0xffffffffu, before ? w.y : 0);
    t0 += __reduce_add_sync(0xffffffffu, w.x);
    r0 += __reduce_add_sync(0xffffffffu, w.y);
    if (g < a.groups) {
      rec[g] = r;
      if (rec == sh) a.ws_groups[g] = r;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    PrefixGroup r = {};
    r.tile0 = t0;
    r.tiles = min(a.nctas, t0);
    a.ws_groups[a.groups] = r;
  }
  // ---- per sequence: where the prefix ends and the suffix begins
#pragma unroll 1
  for (int b = threadIdx.x; b < a.B; b += kPlanThreads) {
    // the last group that starts at or before b
    int lo = 0, hi = a.groups;
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (rec[mid].start <= b) lo = mid; else hi = mid;
    }
    int g = -1, S = 0;
    if (a.groups > 0 && b >= rec[lo].start && b < rec[lo].start + rec[lo].nseq) {
      g = lo;
      S = rec[lo].shared;
    }
    const int raw = __ldg(a.ctx + b), c = context(b);
    if (raw != c) set_error(a.err, KVQ_DEVERR_CONTEXT_RANGE);
    const int cached = a.res_k != nullptr ? c / kBlockSize * kBlockSize : c;
    a.ws_group[b] = g;
    a.ws_limit[b] = min(cached, S);
    // a sequence that ends inside the prefix has no suffix but its tail
    a.ws_ctx[b] = c >= S ? c - S : c - cached;
    a.ws_off[b] = c >= S ? S / kBlockSize : 0;
  }
  __syncthreads();
  if (threadIdx.x == 0) release_token(a.ready, a.token);
}

// ---------------------------------------------------------------------------
// merge
// ---------------------------------------------------------------------------
// A CTA merges kMergeRows rows of one kv head (row = sequence * G + query head
// of the group, as the units count them); a thread has 4 channels of a row, so
// the rows' 16-byte pieces of a partial are consecutive in memory, and every
// SPLIT-th partial.  Bound by the latency of the partials in L2 (up to ~46 of
// them for a row), so U are in flight in each thread, nothing branches around a
// load (that would end in a wait for it), and few rows are split further.
constexpr int kMergeRows = 8;

// A row's running state, four channels of it.
struct RowState {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void raise(float mn) {  // mn >= m, finite
    const float keep = fast_exp2(m - mn);
    m = mn;
    l *= keep;
    o.x *= keep; o.y *= keep; o.z *= keep; o.w *= keep;
  }
  // a state with reference mp <= m; one without weight (-inf: a warpgroup that
  // had no tile, a row masked there) holds no output
  __device__ __forceinline__ void add(float mp, float lp, float4 v) {
    const float w = fast_exp2(mp - m);
    if (mp == -INFINITY) v = make_float4(lp = 0.f, 0.f, 0.f, 0.f);
    l = fmaf(w, lp, l);
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
};

// The full-precision tail of a per-channel K cache: every SPLIT-th of its nt
// tokens, dot products summed over the row's threads.
template <int D, int SPLIT>
__device__ __noinline__ RowState add_tail(const PrefixArgs &a, RowState s, int b, int h, int gq, int rl, int cg, int sp, int nt) {
  constexpr int WARPS = kMergeRows * D / 128, NT = kBlockSize / SPLIT;
  __shared__ float sd[kBlockSize][kMergeRows][WARPS];
  const uint2 q = *reinterpret_cast<const uint2 *>(a.q + (static_cast<int64_t>(b) * a.Hq + h * a.G + gq) * D + 4 * cg);
  const int64_t at = (static_cast<int64_t>(b) * kBlockSize + sp) * a.H * D + h * D + 4 * cg;
  const int step = SPLIT * a.H * D;
#pragma unroll 4
  for (int k = 0; k < NT; ++k) {
    const uint2 w = *reinterpret_cast<const uint2 *>(a.res_k + at + k * step);
    float z = bf16lo_to_f32(q.x) * bf16lo_to_f32(w.x) + bf16hi_to_f32(q.x) * bf16hi_to_f32(w.x) +
              bf16lo_to_f32(q.y) * bf16lo_to_f32(w.y) + bf16hi_to_f32(q.y) * bf16hi_to_f32(w.y);
    // lanes rl, rl + 8, .. of a warp share a row; then the split's warps
    z += __shfl_xor_sync(0xffffffffu, z, 8);
    z += __shfl_xor_sync(0xffffffffu, z, 16);
    if ((threadIdx.x & 31) < kMergeRows) sd[k * SPLIT + sp][rl][threadIdx.x / 32 % WARPS] = z;
  }
  __syncthreads();
  const float zs = rsqrtf(static_cast<float>(D)) * kLog2e;
#pragma unroll 1
  for (int k = 0; k < NT; ++k) {
    float z = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) z += sd[k * SPLIT + sp][rl][w];
    const uint2 v = *reinterpret_cast<const uint2 *>(a.res_v + at + k * step);
    if (k * SPLIT + sp < nt) {  // (rows past the tail hold anything)
      z *= zs;
      s.raise(fmaxf(s.m, z));
      s.add(z, 1.f, make_float4(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x), bf16lo_to_f32(v.y), bf16hi_to_f32(v.y)));
    }
  }
  return s;
}

// Back from the rotated basis, sigma * (H o) / d: stages 1 and 2 in the thread,
// the others between threads through shared memory (every thread of the CTA
// comes here; split 0 has the rows).
template <int D>
__device__ __noinline__ float4 rotate_back(const PrefixArgs &a, float4 o, int rl, int cg, bool writes) {
  __shared__ float4 sh[D / 4][kMergeRows];
  float4 y = make_float4((o.x + o.y) + (o.z + o.w), (o.x - o.y) + (o.z - o.w), (o.x + o.y) - (o.z + o.w), (o.x - o.y) - (o.z - o.w));
#pragma unroll 1
  for (int s = 1; s < D / 4; s <<= 1) {
    if (writes) sh[cg][rl] = y;
    __syncthreads();
    const float4 p = sh[cg ^ s][rl];
    const float f = (cg & s) ? -1.f : 1.f;
    y = make_float4(fmaf(f, y.x, p.x), fmaf(f, y.y, p.y), fmaf(f, y.z, p.z), fmaf(f, y.w, p.w));
    __syncthreads();
  }
  const uint32_t neg = a.rot_signs[cg >> 3] >> (4 * (cg & 7));
  constexpr float kInvD = 1.f / D;
  return make_float4(y.x * (neg & 1u ? -kInvD : kInvD), y.y * (neg & 2u ? -kInvD : kInvD), y.z * (neg & 4u ? -kInvD : kInvD),
                     y.w * (neg & 8u ? -kInvD : kInvD));
}

template <int D, int SPLIT>
__global__ void __launch_bounds__(kMergeRows *SPLIT *D / 4, 1024 / (kMergeRows * SPLIT * D / 4))
    prefix_merge_kernel(const __grid_constant__ PrefixArgs a) {
  constexpr int CG = D / 4;  // channel groups
  constexpr int U = 4, V = 3;
  __shared__ float4 so[SPLIT][CG][kMergeRows];
  __shared__ float2 sm[SPLIT][kMergeRows];
  const int rl = threadIdx.x % kMergeRows, cg = threadIdx.x / kMergeRows % CG, sp = threadIdx.x / (kMergeRows * CG);
  const int h = blockIdx.x % a.H, row = blockIdx.x / a.H * kMergeRows + rl;
  const bool live = row < a.B * a.G;
  const int b = live ? row / a.G : 0, gq = live ? row - b * a.G : 0;

  // ---- the row's partials.  What the plan says is read after the wait too: that
  // it has ended by the time this kernel can start does not make it visible here
  // (reading it before the wait took 1 us off a call).
  grid_wait();
  // the suffix's CTAs have read the token: none is left to the workspace's next call
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ready = 0;
  const int gi = live ? a.ws_group[b] : -1;
  const int total = a.sfx_cum[a.B], s0 = a.sfx_cum[b], s1 = live ? a.sfx_cum[b + 1] : 0;
  int n0 = 0, n1 = 0;
  const float2 *pml = reinterpret_cast<const float2 *>(a.ws_ml), *sml = reinterpret_cast<const float2 *>(a.sfx_ml);
  const float4 *po = reinterpret_cast<const float4 *>(a.ws_o), *qo = reinterpret_cast<const float4 *>(a.sfx_o);
  if (gi >= 0) {
    // (through L1: all CTAs read few records, which would wait in line at L2)
    const PrefixGroup g = a.ws_groups[gi];
    const int T = a.ws_groups[a.groups].tile0, P = a.ws_groups[a.groups].tiles;
    const int r = (b - g.start) * a.G + gq, rb = r / g.rows, u = rb * a.H + h, x0 = g.tile0 + u * g.tiles;
    const int c0 = cta_of(x0, T, P);
    n0 = cta_of(x0 + g.tiles - 1, T, P) - c0 + 1;
    const int slot = g.row0 + u * g.rows + c0 * kPrefixRows, prow = r - rb * g.rows;
    pml += slot + prow;
    po += static_cast<int64_t>(slot) * CG + cg * g.rows + prow;
  }
  RowState s;
#pragma unroll 1
  for (int i = sp; i < n0; i += U * SPLIT) {
    float2 w[U];
    float4 v[U];
    float mn = s.m;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int e = i + k * SPLIT;
      const int64_t at = static_cast<int64_t>(min(e, n0 - 1)) * kPrefixRows;
      w[k] = pml[at];
      v[k] = po[at * CG];
      if (e >= n0) w[k].x = -INFINITY;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) mn = fmaxf(mn, w[k].x);
    if (mn == -INFINITY) continue;
    s.raise(mn);
#pragma unroll
    for (int k = 0; k < U; ++k) s.add(w[k].x, w[k].y, v[k]);
  }
  if (s1 > s0) {
    const int Ps = min(a.sfx_nctas, max(1, (total + a.sfx_blocks_per_cta - 1) / a.sfx_blocks_per_cta));
    const int c0 = cta_of(s0, total, Ps);
    n1 = cta_of(s1 - 1, total, Ps) - c0 + 1;
    const int64_t rec = (static_cast<int64_t>(b + c0) * a.H + h) * 8 + gq;
    sml += rec;
    qo += rec * CG + cg;
  }
  // the suffix's high and (packed: columns g and g + G) low parts; both have the
  // high parts' m and l
  const bool packed = 2 * a.G <= 8;
#pragma unroll 1
  for (int i = sp; i < n1; i += V * SPLIT) {
    float2 w[V];
    float4 v[V], lo[V];
    float mn = s.m;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int e = i + k * SPLIT;
      const int64_t at = static_cast<int64_t>(min(e, n1 - 1)) * a.H * 8;
      w[k] = sml[at];
      v[k] = qo[at * CG];
      lo[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (e >= n1) w[k].x = -INFINITY;
    }
    if (packed) {
#pragma unroll
      for (int k = 0; k < V; ++k)
        lo[k] = qo[(static_cast<int64_t>(min(i + k * SPLIT, n1 - 1)) * a.H * 8 + a.G) * CG];
    }
#pragma unroll
    for (int k = 0; k < V; ++k) mn = fmaxf(mn, w[k].x);
    if (mn == -INFINITY) continue;
    s.raise(mn);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      v[k].x += lo[k].x;
      v[k].y += lo[k].y;
      v[k].z += lo[k].z;
      v[k].w += lo[k].w;
      s.add(w[k].x, w[k].y, v[k]);
    }
  }
  if (a.res_k != nullptr) s = add_tail<D, SPLIT>(a, s, b, h, gq, rl, cg, sp, live ? a.ws_ctx[b] % kBlockSize : 0);
  // ---- the splits' sums
  if constexpr (SPLIT > 1) {
    if (cg == 0) sm[sp][rl] = make_float2(s.m, s.l);
    so[sp][cg][rl] = s.o;
    __syncthreads();
    if (sp == 0) {
      float mn = s.m;
#pragma unroll 1
      for (int k = 1; k < SPLIT; ++k) mn = fmaxf(mn, sm[k][rl].x);
      if (mn != -INFINITY) {
        s.raise(mn);
#pragma unroll 1
        for (int k = 1; k < SPLIT; ++k) s.add(sm[k][rl].x, sm[k][rl].y, so[k][cg][rl]);
      }
    }
  }
  const float inv = s.l > 0.f ? __frcp_rn(s.l) : 0.f;
  float4 o = make_float4(s.o.x * inv, s.o.y * inv, s.o.z * inv, s.o.w * inv);
  if (a.rot) o = rotate_back<D>(a, o, rl, cg, sp == 0);
  // BF16 out, rounded once: what the output projection reads
  if (live && sp == 0) {
    uint2 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(o.y), "f"(o.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(o.w), "f"(o.z));
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
  return launch_overlapped(kern, a.nctas, prefix::kThreads, y.bytes, stream, m.k, m.v, a, y, kf, vf, krow, vrow);
}

cudaError_t launch_prefix_attend(int head_dim, int kf, int vf, const PrefixArgs &a, const DecodeMaps &m,
                                 cudaStream_t stream) {
  return head_dim == 128 ? attend<128>(kf, vf, a, m, stream) : attend<64>(kf, vf, a, m, stream);
}

template <int D>
static cudaError_t merge(const PrefixArgs &a, cudaStream_t stream) {
  const int n = (a.B * a.G + kMergeRows - 1) / kMergeRows * a.H;
  // threads for one wave of half-full SMs (64 registers): as many splits as that
  // allows
  const int64_t threads = static_cast<int64_t>(n) * kMergeRows * (D / 4), wave = static_cast<int64_t>(a.nctas) * 1024;
  constexpr int kOne = kMergeRows * D / 4;
  if (4 * threads <= wave) return launch_overlapped(prefix_merge_kernel<D, 4>, n, 4 * kOne, 0, stream, a);
  if (2 * threads <= wave) return launch_overlapped(prefix_merge_kernel<D, 2>, n, 2 * kOne, 0, stream, a);
  return launch_overlapped(prefix_merge_kernel<D, 1>, n, kOne, 0, stream, a);
}

cudaError_t launch_prefix_merge(int head_dim, const PrefixArgs &a, cudaStream_t stream) {
  return head_dim == 128 ? merge<128>(a, stream) : merge<64>(a, stream);
}

}  // namespace kvq
