// Internal interfaces between the C-ABI layer (kvq_api.cu) and the kernel
// translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace kvq {

struct QuantizeArgs {
  const void *k;          // BF16 [ntok, H, D]
  const void *v;          // BF16 [ntok, H, D]
  const int64_t *slots;   // [ntok]
  int64_t ntok;
  int H;
  int64_t nslots;         // num_blocks * block_size
  uint8_t *kc, *vc;       // code caches
  float *ks, *vs;         // scale arrays
  unsigned int *err;      // sticky error word of this device
  int rot = 0;            // 1: Walsh-Hadamard rotation of every row (include/kvq.h)
  uint32_t rot_signs[4] = {0u, 0u, 0u, 0u};
};

cudaError_t launch_quantize_write(int head_dim, int kf, int vf, const QuantizeArgs &a, int sms,
                                  cudaStream_t stream);

struct DecodeArgs {
  const uint16_t *q;           // BF16 [B, Hq, D]
  const float *ks;             // K scales (layout by granularity)
  const float *vs;             // V scales
  const int32_t *tables;       // [B, max_blocks]
  const int32_t *ctx;          // [B]
  float *ws_o;                 // partial O^T, column-major: [slots, H, 8, D]
  float *ws_ml;                // partial (m, l): [slots, H, 8, 2]
  int *ws_cum;                 // block-count prefix sums [B + 1]
  float *out;                  // [B, Hq, D]
  unsigned int *err;
  int64_t num_blocks;
  int B, Hq, H, G;
  int max_blocks;
  int max_ctx;
  int nctas;                   // P: CTAs of the split kernel
  int rot = 0;                 // 1: rotated cache (include/kvq.h): rotate q, rotate the output back
  uint32_t rot_signs[4] = {0u, 0u, 0u, 0u};
  // Fused write (kvq_write_decode): the step's new K and V, one token per
  // sequence at position ctx - 1, BF16 [B, H, D]; null for a plain decode.
  const uint16_t *knew = nullptr, *vnew = nullptr;
  // Per-channel K with a full-precision tail (kvq_kivi_decode): the split
  // covers the complete blocks only; the reduce adds the residual rows
  // [16 floor(n / 16), n), BF16 [B, 16, H, D]; null otherwise.
  const uint16_t *res_k = nullptr, *res_v = nullptr;
  uint8_t *kc_w = nullptr, *vc_w = nullptr;  // code caches (written)
  float *ks_w = nullptr, *vs_w = nullptr;    // scales (written)
  // Suffix of a shared-prefix decode (kvq_prefix_decode): ctx then holds the
  // suffix lengths, sequence b's blocks start at entry tab_off[b] of its table
  // row, fewer than blocks_per_cta blocks per CTA leave CTAs idle (the host
  // does not know the suffix lengths), and the caller merges the partials.
  const int32_t *tab_off = nullptr;
  int blocks_per_cta = 0;
  bool split_only = false;
  // In what order it is launched: 0 plainly; 1 while the kernel before it, which
  // writes ctx and tab_off, may still run; 2 while the kernel before it may still
  // run, and ctx and tab_off are from an earlier one that has ended and left
  // `token` in `ready`.
  int overlap = 0;
  const unsigned long long *ready = nullptr;
  unsigned long long token = 0;
  // Decode that adds up attention weights (kvq_weigh_decode): the split leaves
  // every score (log2 units) here, [block of the list][H][G][16] with token
  // i + 4 k at 4 i + k, and the reduce each row's maximum and 1 / sum; else null.
  float *ws_z = nullptr;
  float2 *ws_norm = nullptr;   // [B, Hq]
};

// Launches kern so that it may start while the stream's kernel before it still
// runs (that one says when, and kern waits for its results itself).
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kern)(Params...), dim3 ctas, int threads, size_t smem, cudaStream_t stream,
                              const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = ctas;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Launch plan of the split kernel for one shape on the current device.
struct DecodePlan {
  int nstages = 0;       // pipeline depth
  size_t smem = 0;       // dynamic shared memory bytes
  int threads = 0;       // 32 * (H + 1)
  int ctas_per_sm = 0;   // occupancy
  int max_ctas = 0;      // SMs * ctas_per_sm: bound of P, sizes the workspace
};

// TMA descriptors of one decode call: K and V code caches (one (block, head)
// tile per load) and, for INT4 V with four group scales per row, the V scale
// array (one (block, head) [16 tokens][4] tile per load; otherwise a copy of
// v, unused).
struct DecodeMaps {
  CUtensorMap k, v, vs;
};


// Block prefetch from the host pool (prefetch.cu).  Piece sizes are in
// 16-byte vectors per block; host pointers are device-accessible addresses of
// pinned host memory.
struct PrefetchArgs {
  const int32_t *src, *dst;  // [n] host block, device block slot
  int64_t n;
  int64_t host_nb, dev_nb;
  const uint4 *hk, *hv, *hks, *hvs;
  uint4 *dk, *dv, *dks, *dvs;
  int64_t kb16, vb16, ksb16, vsb16;
  unsigned int *err;
};
cudaError_t launch_prefetch(const PrefetchArgs &a, int sms, cudaStream_t stream);

// Append to a per-channel K cache with a full-precision tail (kivi.cu).
struct KiviAppendArgs {
  const uint16_t *knew, *vnew;   // BF16 [B, H, D]: one token per sequence
  uint16_t *res_k, *res_v;       // BF16 [B, 16, H, D] residual rows
  const int32_t *tables;         // [B, max_blocks]
  const int32_t *ctx;            // [B] lengths after the append (0: none)
  uint8_t *kc, *vc;
  float *ks, *vs;
  unsigned int *err;
  int64_t num_blocks;
  int B, H, max_blocks;
};
cudaError_t launch_kivi_append(int head_dim, int kf, int vf, const KiviAppendArgs &a, cudaStream_t stream);

// (dispatch lives in kvq_api.cu)

// Block bookkeeping on the device (block_pool.cu).
struct AssignArgs {
  const int32_t *new_lens;                     // [rows]
  int32_t *ctx;                                // [rows], updated
  int32_t *tables;                             // [rows, max_blocks], updated
  const int32_t *free_list;                    // [num_blocks] stack
  int32_t *free_count, *ref_counts;            // [1], [num_blocks], updated
  const int32_t *prefix_rows, *prefix_blocks;  // [rows] or null
  int32_t *token_offsets;                      // [rows + 1]
  int64_t *slots;                              // [max_tokens]
  int32_t *positions;                          // [max_tokens] or null
  unsigned int *err;
  int64_t num_blocks;
  int rows, max_blocks, max_tokens;
};
struct ReleaseArgs {
  const int32_t *keep;                         // [rows]
  int32_t *ctx, *tables, *free_list, *free_count, *ref_counts;
  unsigned int *err;
  int64_t num_blocks;
  int rows, max_blocks;
};
cudaError_t launch_assign_blocks(const AssignArgs &a, cudaStream_t stream);
cudaError_t launch_release_blocks(const ReleaseArgs &a, cudaStream_t stream);

// Attention weights out of a decode's scores (weigh.cu).
struct WeighArgs {
  const float *z;              // DecodeArgs::ws_z
  const float2 *norm;          // DecodeArgs::ws_norm
  const int *cum;              // DecodeArgs::ws_cum
  const int32_t *tables, *ctx; // [B, max_blocks], [B]
  float *weights;              // [B, H, stride]
  int64_t stride, num_blocks;
  int64_t most_blocks;         // that the contexts can have
  int B, H, G, max_blocks;
};
cudaError_t launch_weigh(const WeighArgs &a, int sms, cudaStream_t stream);

// Eviction by attention weight (evict.cu).
struct EvictMeta {
  int moves;                   // tokens that go to the places of evicted ones
  int active;                  // 0: the row stays as it is
  int keep, recent;
};
struct EvictArgs {
  const int32_t *keep, *recent, *pinned;  // [rows]; pinned or null
  const int32_t *ctx, *tables;            // [rows], [rows, max_blocks]
  const int32_t *refs;                    // [num_blocks] or null
  float *weights;                         // [rows, H, stride]
  int32_t *kept;                          // [rows]
  uint8_t *kc, *vc;
  float *ks, *vs;
  EvictMeta *ws_meta;                     // [rows * H]
  int *ws_list;                           // [rows * H][2][cap]: places, then tokens
  unsigned int *err;
  int64_t num_blocks, stride;
  int rows, H, max_blocks;
  int max_len;                            // largest valid context
  int cap;                                // moves of a (row, head) at most
  int krow, vrow, vgroups;                // bytes of a row of codes; V scales of a row
};
cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t stream);

// Causal attention over packed prompts (prompt_attention.cu).
struct PromptHead {
  int units;                   // units of work
  int next;                    // the first one that no CTA has taken
};
struct PromptArgs {
  const int32_t *offsets;      // [num_seqs + 1]
  uint16_t *out;               // BF16 [num_tokens, Hq, D]
  float *lse;                  // [num_tokens, Hq] or null
  PromptHead *ws_head;
  int2 *ws_seq;                // [num_seqs] start and length, by tiles, most first
  int *ws_level, *ws_place;    // [levels + 1] units before the tile index; places in ws_seq
  unsigned int *err;
  int num_tokens, num_seqs, max_seq;
  int Hq, H, G;
  int unit, levels;            // tokens of a unit, tiles of max_seq
};
// Boxes of 64 channels: of a row tile's tokens and a kv head's query heads (q,
// out), and of one head's tile of keys.
struct PromptMaps {
  CUtensorMap q, k, v, out;
};
cudaError_t launch_prompt_attention(int head_dim, const PromptArgs &a, const PromptMaps &maps, int sms,
                                    cudaStream_t stream);

// Decode over a prefix that the sequences of a group share (prefix_decode.cu).
//
// Work: a unit is (group, row block, kv head); its rows are the (sequence,
// query head) pairs of the group that read the kv head, cut evenly into row
// blocks of at most kPrefixRows; it has ceil(shared / kPrefixTile) tiles.  The
// units' tiles form one list, of which CTA c of P = min(nctas, T) takes
// [c T / P, (c + 1) T / P), at least one tile.  Unit u's partial softmax state in CTA c lies at row
// (row slots of the units before u) + kPrefixRows c of ws_o and ws_ml, which
// never collides: from one (unit, CTA) pair to the next in order, either the
// CTA grows by one or the unit does.
constexpr int kPrefixRows = 256;
constexpr int kPrefixTile = 128;
struct PrefixGroup {
  int start, nseq;       // sequences [start, start + nseq); nseq 0: no sharing
  int shared;            // shared positions, a multiple of the block size
  int lead;              // the sequence whose table holds all shared blocks
  int row_blocks, rows;  // row blocks, and rows in each (the last may have fewer)
  int tiles;             // tiles of a unit
  int tile0;             // tiles of the groups before (< 2^31 in all, the host has checked)
  int row0;              // row slots of the groups before (a unit has `rows`; <= 2 batch * num_q_heads in all)
};
struct PrefixArgs {
  const uint16_t *q;             // BF16 [B, Hq, D]
  const uint8_t *kc, *vc;        // codes
  const float *ks, *vs;          // scales
  const int32_t *tables, *ctx;   // [B, max_blocks], [B]
  const int32_t *group_starts, *prefix_lens;  // [groups + 1], [groups]
  const uint16_t *res_k, *res_v; // full-precision tail or null
  PrefixGroup *ws_groups;        // [groups + 1]; entry `groups` holds tile0 = T and tiles = P
  int *ws_limit;                 // [B] shared positions that the sequence attends to
  int *ws_ctx, *ws_off;          // [B] suffix length, first suffix block
  int *ws_group;                 // [B] group or -1
  unsigned long long *ready, token;  // the plan leaves the call's token here, the merge takes it out
  float *ws_o, *ws_ml;           // prefix partials: by (unit, CTA, stream) [D / 4][rows][4], and [rows, 2]
  const float *sfx_o, *sfx_ml;   // suffix partials (DecodeArgs::ws_o, ws_ml)
  const int *sfx_cum;            // suffix block counts, prefix sums
  uint16_t *out;                 // BF16 [B, Hq, D]
  unsigned int *err;
  int64_t num_blocks;
  int B, Hq, H, G, groups, max_blocks, max_prefix;
  int ctx_cap;                   // largest valid context
  int nctas;                     // CTAs of the prefix kernel
  int sfx_nctas, sfx_blocks_per_cta;
  int rot;
  uint32_t rot_signs[4];
};
cudaError_t launch_prefix_plan(const PrefixArgs &a, cudaStream_t stream);
cudaError_t launch_prefix_attend(int head_dim, int kf, int vf, const PrefixArgs &a, const DecodeMaps &maps,
                                 cudaStream_t stream);
cudaError_t launch_prefix_merge(int head_dim, const PrefixArgs &a, cudaStream_t stream);

// Per-format entry points defined in the decode_k*.cu translation units, and in
// decode_s*.cu for a decode that leaves its scores (per-token K).
template <int KF, bool SCORES = false>
cudaError_t plan_decode_kf(int head_dim, int vf, int H, int G, int B, bool rot, DecodePlan *plan);
template <int KF, bool SCORES = false>
cudaError_t launch_decode_kf(int head_dim, int vf, const DecodeArgs &a, const DecodePlan &plan,
                             const DecodeMaps &maps, cudaStream_t stream);

}  // namespace kvq
