// Block tables and slot mappings made on the GPU, and blocks given back.
//
// What it computes: the paged cache's bookkeeping ("Quantized KV caches in
// production", PagedAttention: fixed-size blocks found through a per-sequence
// table) from the requests' lengths.  The order is that of a loop over the
// rows (assign: row 0 first; release: the last row first, its last block
// first), so results do not depend on scheduling and a release that undoes an
// assign leaves the free list as it was.
//
// What bounds it: latency.  A decode step of 256 rows moves 7 KB.  So each
// call is one launch of one thread-block cluster: every CTA scans all rows
// into its own shared memory (two running sums), the CTAs share the rest of the
// checks and the writing, and a cluster barrier orders the in-place updates after
// everybody's reads, where a second launch or a counter in memory would cost more
// than the work.  Measured: 6.4 us for one token of 256 rows, 11.8 us for 64 x
// 4097 tokens (3.1 MB written), 12 us for giving back 256 rows' drafts, 12.6 and
// 35 us for taking up and giving back 64 rows behind 2048 shared blocks.  Of this
// the look at all blocks to be shared or taken before the first write is 0.5, 2
// and 4 us of the three assignments.
#include <limits.h>

#include "common.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;
constexpr int kFlight = 4;  // loads of a thread that are under way together
constexpr int kStrip = 8;   // rows that a thread takes together where they may share blocks

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();  // the aligned forms want the warp together
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();  // (there may be loops of different lengths since the arrival)
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_cluster_s32(const int *smem, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(smem)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ int blocks_of(int tokens) { return (tokens + kBlockSize - 1) / kBlockSize; }

// Exclusive sums over the CTA's threads of x (64-bit) and y; the totals go to
// tx and ty.  wsum holds two values per warp; the caller may call again at
// once.
__device__ __forceinline__ void scan2(long long x, int y, long long *wx, int *wy, long long &ex, int &ey,
                                      long long &tx, int &ty) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ix = x;
  int iy = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, ix, o);
    const int b = __shfl_up_sync(0xffffffffu, iy, o);
    if (lane >= o) {
      ix += a;
      iy += b;
    }
  }
  if (lane == 31) {
    wx[warp] = ix;
    wy[warp] = iy;
  }
  __syncthreads();
  long long bx = 0, sx = 0;
  int by = 0, sy = 0;
  for (int w = 0; w < kPoolWarps; ++w) {
    if (w == warp) {
      bx = sx;
      by = sy;
    }
    sx += wx[w];
    sy += wy[w];
  }
  __syncthreads();
  ex = bx + ix - x;
  ey = by + iy - y;
  tx = sx;
  ty = sy;
}

// Last row r with off[r] <= i (off non-decreasing, off[0] = 0, i < off[rows]).
__device__ __forceinline__ int row_of(const int *off, int rows, int i) {
  int lo = 0, hi = rows;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// assign
// ---------------------------------------------------------------------------
// visit(first row of a strip, column, ids) for this CTA's part of the blocks that
// rows share.  A thread has one column of kStrip rows: rows behind the same prefix
// read its entry once.  INT_MIN: the row shares nothing there.  A unit is every
// other 1024 columns of a strip.
template <typename Visit>
__device__ __forceinline__ void shared_columns(const AssignArgs &a, const int *ctx, uint32_t rank, uint32_t nct, Visit visit) {
  const int B = a.rows, M = a.max_blocks;
#pragma unroll 1
  for (int unit = rank; unit / 2 * kStrip < B; unit += nct) {
    const int b0 = unit / 2 * kStrip;
    int from[kStrip], k[kStrip], most = 0;
#pragma unroll
    for (int u = 0; u < kStrip; ++u) {
      const int b = min(b0 + u, B - 1);
      from[u] = __ldg(a.prefix_rows + b);
      k[u] = b0 + u < B && from[u] >= 0 ? ctx[b] / kBlockSize : 0;
      most = max(most, k[u]);
    }
#pragma unroll 1
    for (int i = (unit & 1) * kPoolThreads + threadIdx.x; i < most; i += 2 * kPoolThreads) {
      int id[kStrip];
#pragma unroll
      for (int u = 0; u < kStrip; ++u)
        id[u] = i < k[u] ? max(__ldcg(a.tables + static_cast<int64_t>(from[u]) * M + i), INT_MIN + 1) : INT_MIN;
      visit(b0, i, id);
    }
  }
}

// Shared: tok[rows + 1], blk[rows + 1], ctx[rows] (contexts after sharing).
__global__ void __launch_bounds__(kPoolThreads) assign_blocks_kernel(const AssignArgs a) {
  extern __shared__ int sm[];
  __shared__ long long wx[kPoolWarps];
  __shared__ int wy[kPoolWarps];
  __shared__ int refused;
  const int B = a.rows, M = a.max_blocks;
  int *tok = sm, *blk = sm + B + 1, *ctx = sm + 2 * (B + 1);
  const uint32_t rank = cluster_rank(), nct = cluster_size();
  const int f = __ldcg(a.free_count);  // (written at the end: not through the read-only path)

  // ---- check the rows and sum tokens and blocks
  unsigned int bad = 0;
  long long ctok = 0;  // running totals of the rows so far
  int cblk = 0;
  for (int base = 0; base < B; base += kPoolThreads) {
    const int b = base + threadIdx.x;
    int n = 0, c = 0, need = 0;
    if (b < B) {
      n = __ldg(a.new_lens + b);
      c = __ldcg(a.ctx + b);
      if (n < 0 || c < 0) bad |= KVQ_DEVERR_CONTEXT_RANGE;
      if (a.prefix_rows != nullptr) {
        const int s = __ldg(a.prefix_rows + b);
        if (s >= 0) {
          const int k = __ldg(a.prefix_blocks + b);
          // the source row must hold the shared blocks already, all full
          if (s >= B || s == b || c != 0 || k < 0 || k > M ||
              static_cast<long long>(k) * kBlockSize > __ldcg(a.ctx + (s < B ? s : 0)))
            bad |= KVQ_DEVERR_CONTEXT_RANGE;
          else
            c = k * kBlockSize;
        }
      }
      if (!bad && static_cast<long long>(c) + n > static_cast<long long>(M) * kBlockSize) bad |= KVQ_DEVERR_CONTEXT_RANGE;
      if (!bad && n > 0 && c % kBlockSize != 0) {
        // the row continues a block of its own: never one that others read
        const int id = __ldcg(a.tables + static_cast<int64_t>(b) * M + c / kBlockSize);
        if (id < 0 || id >= a.num_blocks) bad |= KVQ_DEVERR_BLOCK_RANGE;
        else if (__ldcg(a.ref_counts + id) != 1) bad |= KVQ_DEVERR_POOL_STATE;
      }
      if (bad) n = 0;
      need = bad ? 0 : blocks_of(c + n) - blocks_of(c);
    }
    long long et, tt;
    int eb, tb;
    scan2(n, need, wx, wy, et, eb, tt, tb);
    if (b < B) {
      const long long t = ctok + et;
      tok[b] = t > INT_MAX ? INT_MAX : static_cast<int>(t);
      blk[b] = cblk + eb;
      ctx[b] = c;
    }
    ctok += tt;
    cblk += tb;
  }
  if (f < 0 || f > a.num_blocks) bad |= KVQ_DEVERR_POOL_STATE;
  else if (cblk > f || ctok > a.max_tokens) bad |= KVQ_DEVERR_CAPACITY;
  const int tid = rank * kPoolThreads + threadIdx.x, nth = nct * kPoolThreads;
  if (!__syncthreads_or(bad != 0)) {
    // ---- the blocks that the call would share and take, the CTAs each a part
    if (a.prefix_rows != nullptr)
      shared_columns(a, ctx, rank, nct, [&](int, int, const int (&id)[kStrip]) {
#pragma unroll
        for (int u = 0; u < kStrip; ++u)
          if (id[u] != INT_MIN && (id[u] < 0 || id[u] >= a.num_blocks)) bad |= KVQ_DEVERR_BLOCK_RANGE;
      });
#pragma unroll 4
    for (int i = tid; i < cblk; i += nth) {
      const int id = __ldg(a.free_list + (f - 1 - i));
      if (id < 0 || id >= a.num_blocks) bad |= KVQ_DEVERR_POOL_STATE;
    }
  }
  if (bad) set_error(a.err, bad);
  // No CTA writes anything before every CTA has checked, and one that has found
  // something holds all of them back.
  const bool any = __syncthreads_or(bad != 0);
  if (threadIdx.x == 0) {
    refused = any;
    tok[B] = static_cast<int>(ctok);
    blk[B] = cblk;
  }
  cluster_arrive();
  cluster_wait();
  const int lane = threadIdx.x & 31;
  const bool ok = !__any_sync(0xffffffffu, lane < static_cast<int>(nct) && ld_cluster_s32(&refused, lane) != 0);
  cluster_arrive();  // no CTA exits while another may still read its word
  const int ntok = ok ? static_cast<int>(ctok) : 0, nblk = ok ? cblk : 0;

  // ---- offsets, slots and positions
  for (int b = tid; b <= B; b += nth) a.token_offsets[b] = ok ? tok[b] : 0;
#pragma unroll 1
  for (unsigned int t0 = tid; t0 < static_cast<unsigned int>(a.max_tokens); t0 += kFlight * nth) {
    int pos[kFlight], id[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const unsigned int at = t0 + u * nth;
      pos[u] = id[u] = -1;
      if (at >= static_cast<unsigned int>(ntok)) continue;
      const int t = static_cast<int>(at), b = row_of(tok, B, t);
      const int c = ctx[b], have = blocks_of(c);
      pos[u] = c + t - tok[b];
      const int j = pos[u] / kBlockSize;
      id[u] = __ldcg(j < have ? a.tables + static_cast<int64_t>(b) * M + j : a.free_list + (f - 1 - (blk[b] + j - have)));
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const unsigned int t = t0 + u * nth;
      if (t >= static_cast<unsigned int>(a.max_tokens)) break;
      a.slots[t] = id[u] >= 0 ? static_cast<int64_t>(id[u]) * kBlockSize + pos[u] % kBlockSize : -1;
      if (a.positions != nullptr) a.positions[t] = pos[u];
    }
  }
  if (ok) {
    // ---- shared blocks (rows behind the same prefix raise its count once), then
    // new ones
    if (a.prefix_rows != nullptr)
      shared_columns(a, ctx, rank, nct, [&](int b0, int i, const int (&id)[kStrip]) {
        int run = 0;
#pragma unroll
        for (int u = 0; u < kStrip; ++u) {
          ++run;
          if (id[u] != INT_MIN) a.tables[static_cast<int64_t>(b0 + u) * M + i] = id[u];
          if (u + 1 < kStrip && id[u + 1] == id[u]) continue;
          if (id[u] != INT_MIN) atomicAdd(a.ref_counts + id[u], run);
          run = 0;
        }
      });
    for (int i = tid; i < nblk; i += nth) {
      const int b = row_of(blk, B, i);
      const int id = __ldg(a.free_list + (f - 1 - i));
      a.tables[static_cast<int64_t>(b) * M + blocks_of(ctx[b]) + i - blk[b]] = id;
      a.ref_counts[id] = 1;
    }
    for (int b = tid; b < B; b += nth) a.ctx[b] = ctx[b] + tok[b + 1] - tok[b];
    if (tid == 0) *a.free_count = f - nblk;
  }
  cluster_wait();
}

// ---------------------------------------------------------------------------
// release
// ---------------------------------------------------------------------------
// Items are the released table entries in (row, block) order.  A block that
// several rows give back in one call is pushed by the first of its items (the
// last one of the descending loop): after all counts are taken down, every
// item of a block whose count is 0 offers INT_MIN + item to an atomic minimum
// on the count itself, and the item that finds its own code pushes.
__global__ void __launch_bounds__(kPoolThreads) release_blocks_kernel(const ReleaseArgs a) {
  extern __shared__ int sm[];
  __shared__ long long wx[kPoolWarps];
  __shared__ int wy[kPoolWarps];
  __shared__ int pushes;
  const int B = a.rows, M = a.max_blocks;
  int *off = sm, *first = sm + B + 1;  // first released block of the row
  const uint32_t rank = cluster_rank(), nct = cluster_size();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int f = __ldcg(a.free_count);  // (written at the end: not through the read-only path)
  const bool pool_ok = f >= 0 && f <= a.num_blocks;
  if (!pool_ok && rank == 0 && threadIdx.x == 0) set_error(a.err, KVQ_DEVERR_POOL_STATE);

  int n = 0;
  for (int base = 0; base < B; base += kPoolThreads) {
    const int b = base + threadIdx.x;
    int cnt = 0, i0 = 0;
    if (b < B) {
      const int c = __ldcg(a.ctx + b), keep = __ldg(a.keep + b);
      if (c < 0 || static_cast<long long>(c) > static_cast<long long>(M) * kBlockSize || keep < 0) {
        if (rank == 0) set_error(a.err, KVQ_DEVERR_CONTEXT_RANGE);
        i0 = -1;  // the row stays as it is
      } else {
        i0 = blocks_of(keep < c ? keep : c);
        cnt = pool_ok ? blocks_of(c) - i0 : 0;
      }
    }
    long long e0, t0;
    int eb, tb;
    scan2(0, cnt, wx, wy, e0, eb, t0, tb);
    if (b < B) {
      off[b] = n + eb;
      first[b] = i0;
    }
    n += tb;
  }
  if (threadIdx.x == 0) {
    off[B] = n;
    pushes = 0;
  }
  __syncthreads();

  // each warp owns a contiguous run of items
  const unsigned int items = n, each = (items + nct * kPoolWarps - 1) / (nct * kPoolWarps);
  const int lo = min(items, (rank * kPoolWarps + warp) * each), hi = min(items, lo + each);
  auto entry = [&](int i) -> int32_t * {
    const int b = row_of(off, B, i);
    return a.tables + static_cast<int64_t>(b) * M + first[b] + (i - off[b]);
  };
  // Long rows may share most of their blocks: a lane then has one column of
  // kStrip rows, whose runs of one id give it back, and offer for it, once.
  const bool strips = n / 32 >= B;
  const int gw = rank * kPoolWarps + warp, warps = nct * kPoolWarps;
  // visit(row of the strip's first entry, column) for this warp's columns
  auto each_column = [&](auto visit) {
    int skip = gw;  // the warp's first group of 32 columns in the strip
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += kStrip) {
      const int b = min(b0 + lane % kStrip, B - 1), cnt = off[b + 1] - off[b];
      const int j0 = __reduce_min_sync(0xffffffffu, cnt > 0 ? first[b] : INT_MAX);
      const int j1 = __reduce_max_sync(0xffffffffu, cnt > 0 ? first[b] + cnt : 0);
      const int groups = j1 > j0 ? (j1 - j0 + 31) / 32 : 0;
#pragma unroll 1
      for (; skip < groups; skip += warps) visit(b0, j0 + 32 * skip + lane);
      skip -= groups;  // the next strip's groups go on with the next warp
    }
  };
  // the column's ids: INT_MIN where the row gives nothing back there
  auto column = [&](int b0, int j, int (&id)[kStrip]) {
#pragma unroll
    for (int u = 0; u < kStrip; ++u) {
      const int b = min(b0 + u, B - 1);
      const bool in = b0 + u < B && off[b + 1] > off[b] && j >= first[b] && j - first[b] < off[b + 1] - off[b];
      id[u] = in ? max(__ldcg(a.tables + static_cast<int64_t>(b) * M + j), INT_MIN + 1) : INT_MIN;
    }
  };
  if (strips) {
    each_column([&](int b0, int j) {
      int id[kStrip], run = 0;
      column(b0, j, id);
#pragma unroll
      for (int u = 0; u < kStrip; ++u) {
        ++run;
        if (u + 1 < kStrip && id[u + 1] == id[u]) continue;
        if (id[u] != INT_MIN) {
          const bool in = id[u] >= 0 && id[u] < a.num_blocks;
          const int held = in ? atomicSub(a.ref_counts + id[u], run) : 0;
          if (held < run) {  // no block, or given back more often than held
            set_error(a.err, in ? KVQ_DEVERR_POOL_STATE : KVQ_DEVERR_BLOCK_RANGE);
            if (in) atomicAdd(a.ref_counts + id[u], run - max(held, 0));
            if (held <= 0)
              for (int v = u - run + 1; v <= u; ++v) a.tables[static_cast<int64_t>(b0 + v) * M + j] = -1;
          }
        }
        run = 0;
      }
    });
  } else {
#pragma unroll 1
    for (int i = lo + lane; i < hi; i += 32) {
      int32_t *e = entry(i);
      const int id = __ldcg(e);
      const bool in = id >= 0 && id < a.num_blocks;
      if (in && atomicSub(a.ref_counts + id, 1) > 0) continue;
      if (in) atomicAdd(a.ref_counts + id, 1);  // given back more often than held
      set_error(a.err, in ? KVQ_DEVERR_POOL_STATE : KVQ_DEVERR_BLOCK_RANGE);
      *e = -1;
    }
  }
  cluster_arrive();
  cluster_wait();
  if (strips) {
    each_column([&](int b0, int j) {
      int id[kStrip];
      column(b0, j, id);
#pragma unroll
      for (int u = kStrip - 1; u >= 0; --u) {  // (the first row of a run has its first item)
        const bool lead = u == 0 || id[u - 1] != id[u];
        if (id[u] < 0) continue;
        if (lead && __ldcg(a.ref_counts + id[u]) <= 0)
          atomicMin(a.ref_counts + id[u], INT_MIN + off[b0 + u] + (j - first[b0 + u]));
        else
          a.tables[static_cast<int64_t>(b0 + u) * M + j] = -1;  // does not push
      }
    });
  } else {
#pragma unroll 1
    for (int i = lo + lane; i < hi; i += 32) {
      const int id = __ldcg(entry(i));
      if (id >= 0 && __ldcg(a.ref_counts + id) <= 0) atomicMin(a.ref_counts + id, INT_MIN + i);
    }
  }
  cluster_arrive();
  cluster_wait();
  // Which items push; the others are done.  kFlight of them are searched for and
  // loaded together; `which` has the first 64 turns, so that the last pass takes
  // only those that push.
  int mine = 0;  // pushes of this warp
  unsigned long long which = 0;
  int top = 1;
  while (2 * top < B) top *= 2;
#pragma unroll 1
  for (int i = lo + lane, k = 0; i < hi; i += 32 * kFlight, k += kFlight) {
    int b[kFlight], id[kFlight], code[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) b[u] = 0;
#pragma unroll 1
    for (int step = top; step > 0; step >>= 1)
#pragma unroll
      for (int u = 0; u < kFlight; ++u)
        if (b[u] + step < B && off[b[u] + step] <= min(i + 32 * u, hi - 1)) b[u] += step;
    int32_t *e[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      e[u] = a.tables + static_cast<int64_t>(b[u]) * M + first[b[u]] + (min(i + 32 * u, hi - 1) - off[b[u]]);
      id[u] = __ldcg(e[u]);
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) code[u] = id[u] >= 0 ? __ldcg(a.ref_counts + id[u]) : 0;
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      if (i + 32 * u >= hi) break;
      const bool push = id[u] >= 0 && code[u] == INT_MIN + i + 32 * u;
      mine += push;
      if (push && k + u < 64) which |= 1ull << (k + u);
      if (!push && id[u] != -1) *e[u] = -1;
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) wy[warp] = mine;
  __syncthreads();
  int before = 0;  // pushes of the CTA's earlier warps
  for (int k = 0; k < warp; ++k) before += wy[k];
  if (threadIdx.x == kPoolThreads - 1) pushes = before + mine;
  cluster_arrive();
  cluster_wait();
  int total = 0;
  for (uint32_t r = 0; r < nct; ++r) {
    const int p = ld_cluster_s32(&pushes, r);
    if (r < rank) before += p;
    total += p;
  }
  // the descending loop pushes the last item first
  int done = before;
  for (int base = lo, k = 0; base < hi; base += 32, ++k) {
    const int i = base + lane;
    bool push = k < 64 && (which >> k & 1);
    if (k < 64 && !__any_sync(0xffffffffu, push)) continue;
    int id = -1;
    if (i < hi && (push || k >= 64)) {
      int32_t *e = entry(i);
      id = __ldcg(e);
      if (k >= 64) push = id >= 0 && __ldcg(a.ref_counts + id) == INT_MIN + i;
      *e = -1;
    }
    const unsigned int votes = __ballot_sync(0xffffffffu, push);
    if (push) {
      const int64_t at = static_cast<int64_t>(f) + total - 1 - (done + __popc(votes & ((1u << lane) - 1)));
      if (at < a.num_blocks) a.free_list[at] = id;
      else set_error(a.err, KVQ_DEVERR_POOL_STATE);
      a.ref_counts[id] = 0;
    }
    done += __popc(votes);
  }
  const int tid = rank * kPoolThreads + threadIdx.x, nth = nct * kPoolThreads;
  for (int b = tid; b < B; b += nth) {
    if (!pool_ok || first[b] < 0) continue;
    const int c = a.ctx[b], keep = __ldg(a.keep + b);
    if (keep < c) a.ctx[b] = keep;
  }
  if (tid == 0 && total > 0) {
    const int64_t v = static_cast<int64_t>(f) + total;
    *a.free_count = v < a.num_blocks ? static_cast<int>(v) : static_cast<int>(a.num_blocks);
  }
  cluster_arrive();  // no CTA exits while another may still read its pushes
  cluster_wait();
}

template <typename Args>
cudaError_t launch_cluster(void (*kern)(const Args), const Args &a, int ctas, size_t smem, cudaStream_t stream) {
  // Above the default 48 KB only with many rows, and sixteen CTAs only with much
  // work; the attributes are per device and idempotent.
  cudaError_t e;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024)) != cudaSuccess)
    return e;
  if (ctas > 8 && (e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) {
    cudaGetLastError();
    ctas = 8;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPoolThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

// One CTA per 4096 items of work, up to the largest cluster: scattered accesses
// to the counts bound large calls, and so the SMs that make them (release of 64
// rows behind 2048 shared blocks, all of them given back: 8 CTAs 73 us, 16 CTAs
// 41 us).  What a release gives back is known on the device only: the host counts
// the tables' width, so that a rollback in a wide table takes the large form too.
int cluster_for(int64_t items) {
  int c = 1;
  while (c < 16 && static_cast<int64_t>(c) * 4096 < items) c *= 2;
  return c;
}

}  // namespace

cudaError_t launch_assign_blocks(const AssignArgs &a, cudaStream_t stream) {
  int64_t items = a.max_tokens;
  if (a.prefix_rows != nullptr) items += static_cast<int64_t>(a.rows) * a.max_blocks;
  const size_t smem = (3 * static_cast<size_t>(a.rows) + 2) * sizeof(int);
  return launch_cluster(assign_blocks_kernel, a, cluster_for(items), smem, stream);
}

cudaError_t launch_release_blocks(const ReleaseArgs &a, cudaStream_t stream) {
  const size_t smem = (2 * static_cast<size_t>(a.rows) + 1) * sizeof(int);
  return launch_cluster(release_blocks_kernel, a, cluster_for(static_cast<int64_t>(a.rows) * a.max_blocks), smem,
                        stream);
}

}  // namespace kvq
