// The C ABI of libkvq (declared in include/kvq.h): argument checks, format
// decoding, tensor-map encoding and kernel launches.  Nothing here computes
// on the host; every step of the path runs in the kernels.
#include <algorithm>
#include <atomic>
#include <chrono>
#include <mutex>
#include <unordered_map>

#include "common.cuh"
#include "kvq_internal.h"

namespace {

using namespace kvq;

// The sticky device error word, one per device (kernels receive its address).
__device__ unsigned int g_kvq_errors = 0;

constexpr int kMaxDevices = 64;
unsigned int *g_err_addr[kMaxDevices] = {};
std::mutex g_err_mu;

cudaError_t error_word(unsigned int **out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_err_mu);
  if (!g_err_addr[dev]) {
    void *p = nullptr;
    e = cudaGetSymbolAddress(&p, g_kvq_errors);
    if (e != cudaSuccess) return e;
    g_err_addr[dev] = static_cast<unsigned int *>(p);
  }
  *out = g_err_addr[dev];
  return cudaSuccess;
}

int sm_count(int *sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVQ_ERR_CUDA;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return KVQ_ERR_CUDA;
  return KVQ_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Decodes and checks a format; on success sets the kernel format codes.
int decode_format(const kvq_format *f, int *kf, int *vf) {
  if (!f) return KVQ_ERR_INVALID_ARG;
  if (f->rotation != KVQ_ROT_NONE && f->rotation != KVQ_ROT_HADAMARD) return KVQ_ERR_INVALID_ARG;
  if (f->num_blocks < 0 || f->num_kv_heads < 1) return KVQ_ERR_INVALID_ARG;
  if (f->block_size != kBlockSize) return KVQ_ERR_UNSUPPORTED;
  if (f->head_dim != 64 && f->head_dim != 128) return KVQ_ERR_UNSUPPORTED;
  if (f->num_kv_heads > 8) return KVQ_ERR_UNSUPPORTED;
  if (f->k_gran == KVQ_PER_TOKEN_HEAD && f->k_dtype == KVQ_INT8) *kf = K_INT8_TOK;
  else if (f->k_gran == KVQ_PER_TOKEN_HEAD && f->k_dtype == KVQ_FP8_E4M3FN) *kf = K_FP8_TOK;
  else if (f->k_gran == KVQ_PER_BLOCK_CHANNEL && f->k_dtype == KVQ_INT8) *kf = K_INT8_CHAN;
  else if (f->k_gran == KVQ_PER_TOKEN_HEAD && f->k_dtype == KVQ_INT4) *kf = K_INT4_TOK;
  else if (f->k_gran == KVQ_PER_BLOCK_CHANNEL && f->k_dtype == KVQ_INT2 && f->head_dim == 128) *kf = K_INT2_CHAN;
  else return KVQ_ERR_UNSUPPORTED;
  if (f->v_gran == KVQ_PER_TOKEN_HEAD && f->v_dtype == KVQ_INT8) *vf = V_INT8_TOK;
  else if (f->v_gran == KVQ_PER_TOKEN_HEAD && f->v_dtype == KVQ_FP8_E4M3FN) *vf = V_FP8_TOK;
  else if (f->v_gran == KVQ_PER_TOKEN_GROUP && f->v_dtype == KVQ_INT4 && f->v_group == 32) *vf = V_INT4_G32;
  else if (f->v_gran == KVQ_PER_TOKEN_GROUP && f->v_dtype == KVQ_INT2 && f->v_group == 32 && f->head_dim == 128)
    *vf = V_INT2_G32;
  else return KVQ_ERR_UNSUPPORTED;
  if (f->rotation == KVQ_ROT_HADAMARD && (*kf == K_INT8_CHAN || *kf == K_INT2_CHAN)) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

cudaError_t plan_decode_uncached(int D, int kf, int vf, int H, int G, int B, bool rot, bool scores, DecodePlan *plan) {
  if (scores) {
    if (kf == K_INT8_TOK) return plan_decode_kf<K_INT8_TOK, true>(D, vf, H, G, B, rot, plan);
    if (kf == K_FP8_TOK) return plan_decode_kf<K_FP8_TOK, true>(D, vf, H, G, B, rot, plan);
    if (kf == K_INT4_TOK) return plan_decode_kf<K_INT4_TOK, true>(D, vf, H, G, B, rot, plan);
    return cudaErrorInvalidValue;
  }
  if (kf == K_INT8_TOK) return plan_decode_kf<K_INT8_TOK>(D, vf, H, G, B, rot, plan);
  if (kf == K_FP8_TOK) return plan_decode_kf<K_FP8_TOK>(D, vf, H, G, B, rot, plan);
  if (kf == K_INT8_CHAN) return plan_decode_kf<K_INT8_CHAN>(D, vf, H, G, B, rot, plan);
  if (kf == K_INT4_TOK) return plan_decode_kf<K_INT4_TOK>(D, vf, H, G, B, rot, plan);
  if (kf == K_INT2_CHAN) return plan_decode_kf<K_INT2_CHAN>(D, vf, H, G, B, rot, plan);
  return cudaErrorInvalidValue;
}

// Launch plans are computed once per (device, kernel instance, batch): the
// kernel attributes, the SM count and the occupancy query stay off the
// per-call path.  The map is bounded (cleared when full).
struct PlanKey {
  int dev, D, kf, vf, H, G, B, rot, scores;
  bool operator==(const PlanKey &o) const {
    return dev == o.dev && D == o.D && kf == o.kf && vf == o.vf && H == o.H && G == o.G && B == o.B && rot == o.rot &&
           scores == o.scores;
  }
};
struct PlanKeyHash {
  size_t operator()(const PlanKey &k) const {
    size_t h = 1469598103934665603ull;
    for (int x : {k.dev, k.D, k.kf, k.vf, k.H, k.G, k.B, k.rot, k.scores})
      h = (h ^ static_cast<uint32_t>(x)) * 1099511628211ull;
    return h;
  }
};
constexpr size_t kMaxPlans = 1024;
std::unordered_map<PlanKey, DecodePlan, PlanKeyHash> g_plans;
std::mutex g_plan_mu;

cudaError_t plan_decode(int D, int kf, int vf, int H, int G, int B, bool rot, DecodePlan *plan, bool scores = false) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const PlanKey key{dev, D, kf, vf, H, G, B, rot ? 1 : 0, scores ? 1 : 0};
  {
    std::lock_guard<std::mutex> lk(g_plan_mu);
    auto it = g_plans.find(key);
    if (it != g_plans.end()) {
      *plan = it->second;
      return cudaSuccess;
    }
  }
  DecodePlan p;
  if ((e = plan_decode_uncached(D, kf, vf, H, G, B, rot, scores, &p)) != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(g_plan_mu);
  if (g_plans.size() >= kMaxPlans) g_plans.clear();
  g_plans.emplace(key, p);
  *plan = p;
  return cudaSuccess;
}

cudaError_t launch_decode(int D, int kf, int vf, const DecodeArgs &a, const DecodePlan &plan,
                          const DecodeMaps &m, cudaStream_t s) {
  if (a.ws_z != nullptr) {
    if (kf == K_INT8_TOK) return launch_decode_kf<K_INT8_TOK, true>(D, vf, a, plan, m, s);
    if (kf == K_FP8_TOK) return launch_decode_kf<K_FP8_TOK, true>(D, vf, a, plan, m, s);
    if (kf == K_INT4_TOK) return launch_decode_kf<K_INT4_TOK, true>(D, vf, a, plan, m, s);
    return cudaErrorInvalidValue;
  }
  if (kf == K_INT8_TOK) return launch_decode_kf<K_INT8_TOK>(D, vf, a, plan, m, s);
  if (kf == K_FP8_TOK) return launch_decode_kf<K_FP8_TOK>(D, vf, a, plan, m, s);
  if (kf == K_INT8_CHAN) return launch_decode_kf<K_INT8_CHAN>(D, vf, a, plan, m, s);
  if (kf == K_INT4_TOK) return launch_decode_kf<K_INT4_TOK>(D, vf, a, plan, m, s);
  if (kf == K_INT2_CHAN) return launch_decode_kf<K_INT2_CHAN>(D, vf, a, plan, m, s);
  return cudaErrorInvalidValue;
}

// Workspace layout: [partial O^T][partial (m, l)][prefix sums], 256-aligned.
struct WsLayout {
  size_t o_off, ml_off, cum_off, total;
};

WsLayout ws_layout(int B, int H, int D, int max_ctas) {
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t slots = static_cast<size_t>(B) + static_cast<size_t>(max_ctas);
  WsLayout w;
  w.o_off = 0;
  w.ml_off = al(slots * H * D * 8 * sizeof(float));
  w.cum_off = w.ml_off + al(slots * H * 8 * 2 * sizeof(float));
  w.total = w.cum_off + al((static_cast<size_t>(B) + 1) * sizeof(int));
  return w;
}

// A decode that adds up attention weights needs the scores of every block that
// max_context_len allows, and each row's maximum and sum, behind that.
struct WeighWs {
  size_t z_off, norm_off, total;
};

WeighWs weigh_ws(const WsLayout &wl, int B, int Hq, int max_context) {
  const size_t blocks = static_cast<size_t>(B) * ((static_cast<size_t>(max_context) + kBlockSize - 1) / kBlockSize);
  WeighWs w;
  w.z_off = wl.total;
  w.norm_off = w.z_off + blocks * Hq * kBlockSize * sizeof(float);
  w.total = w.norm_off + ((static_cast<size_t>(B) * Hq * sizeof(float2) + 255) & ~size_t(255));
  return w;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 4-D map over a code cache [num_blocks, bs, H, row_bytes] (uint8) with a
// box of one (block, head) tile: 16 rows of row_bytes.
int encode_cache_map(CUtensorMap *map, const void *base, int64_t nb, int H, int row_bytes) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return KVQ_ERR_CUDA;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(kBlockSize), static_cast<cuuint64_t>(nb)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(row_bytes),
                                 static_cast<cuuint64_t>(row_bytes) * H,
                                 static_cast<cuuint64_t>(row_bytes) * H * kBlockSize};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(row_bytes), 1, static_cast<cuuint32_t>(kBlockSize), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle sw = row_bytes >= 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                : (row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box,
                        estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? KVQ_OK : KVQ_ERR_CUDA;
}

// 4-D map over INT4 V group scales [num_blocks, bs, H, 4] (float32) with a
// box of one (block, head) tile: 16 tokens x 4 groups (256 bytes).
int encode_vscale_map(CUtensorMap *map, const float *base, int64_t nb, int H) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return KVQ_ERR_CUDA;
  const cuuint64_t dims[4] = {4, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(kBlockSize),
                              static_cast<cuuint64_t>(nb)};
  const cuuint64_t strides[3] = {16, static_cast<cuuint64_t>(16) * H,
                                 static_cast<cuuint64_t>(16) * H * kBlockSize};
  const cuuint32_t box[4] = {4, 1, static_cast<cuuint32_t>(kBlockSize), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<float *>(base), dims, strides, box,
                        estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? KVQ_OK : KVQ_ERR_CUDA;
}

// 3-D map over BF16 rows [tokens, heads, D], tokens `stride` elements apart, with
// a box of 64 channels of `h` heads of `t` tokens.
int encode_rows_map(CUtensorMap *map, const void *base, int64_t tokens, int heads, int D, int64_t stride, int h, int t) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return KVQ_ERR_CUDA;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(h), static_cast<cuuint32_t>(t)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? KVQ_OK : KVQ_ERR_CUDA;
}

// The descriptors of one decode call.
int encode_decode_maps_uncached(DecodeMaps *m, const kvq_caches &caches, const kvq_scales &scales, int64_t nb,
                                int H, int D, int kf, int vf) {
  const int krow = (kf == K_INT4_TOK) ? D / 2 : (kf == K_INT2_CHAN ? D / 4 : D);
  const int vrow = (vf == V_INT4_G32) ? D / 2 : (vf == V_INT2_G32 ? D / 4 : D);
  int st;
  if ((st = encode_cache_map(&m->k, caches.k_cache, nb, H, krow)) != KVQ_OK) return st;
  if ((st = encode_cache_map(&m->v, caches.v_cache, nb, H, vrow)) != KVQ_OK) return st;
  if ((vf == V_INT4_G32 || vf == V_INT2_G32) && D / 32 == 4) return encode_vscale_map(&m->vs, scales.v_scale, nb, H);
  m->vs = m->v;
  return KVQ_OK;
}

// The tensor maps of the last few caches, so that a serving loop over the
// same cache encodes them once: keyed by the cache and scale pointers and
// the shape and format they were encoded for.
struct MapEntry {
  bool used = false;
  int dev = 0, H = 0, D = 0, kf = 0, vf = 0;
  int64_t nb = 0;
  const void *kc = nullptr, *vc = nullptr;
  const float *vs = nullptr;
  DecodeMaps maps;
};
constexpr int kMapSlots = 16;
MapEntry g_maps[kMapSlots];
int g_map_next = 0;
std::mutex g_map_mu;

int encode_decode_maps(DecodeMaps *m, const kvq_caches &caches, const kvq_scales &scales, int64_t nb, int H, int D,
                       int kf, int vf) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVQ_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lk(g_map_mu);
    for (const MapEntry &e : g_maps) {
      if (e.used && e.dev == dev && e.kc == caches.k_cache && e.vc == caches.v_cache && e.vs == scales.v_scale &&
          e.nb == nb && e.H == H && e.D == D && e.kf == kf && e.vf == vf) {
        *m = e.maps;
        return KVQ_OK;
      }
    }
  }
  DecodeMaps fresh;
  const int st = encode_decode_maps_uncached(&fresh, caches, scales, nb, H, D, kf, vf);
  if (st != KVQ_OK) return st;
  std::lock_guard<std::mutex> lk(g_map_mu);
  MapEntry &e = g_maps[g_map_next];
  g_map_next = (g_map_next + 1) % kMapSlots;
  e.used = true;
  e.dev = dev;
  e.H = H;
  e.D = D;
  e.kf = kf;
  e.vf = vf;
  e.nb = nb;
  e.kc = caches.k_cache;
  e.vc = caches.v_cache;
  e.vs = scales.v_scale;
  e.maps = fresh;
  *m = fresh;
  return KVQ_OK;
}

}  // namespace

extern "C" {

int32_t kvq_version(void) { return 110; }

#ifndef KVQ_BUILD_ID
#define KVQ_BUILD_ID "unknown"
#endif
const char *kvq_build_id(void) { return KVQ_BUILD_ID; }

const char *kvq_status_string(int32_t status) {
  switch (status) {
    case KVQ_OK: return "ok";
    case KVQ_ERR_INVALID_ARG: return "invalid argument";
    case KVQ_ERR_UNSUPPORTED: return "unsupported format or shape";
    case KVQ_ERR_WORKSPACE: return "workspace too small";
    case KVQ_ERR_CUDA: return "CUDA error";
    default: return "unknown status";
  }
}

int kvq_quantize_write(const void *k_bf16, const void *v_bf16, const int64_t *slot_mapping,
                       int64_t num_tokens, const kvq_format *fmt, kvq_caches caches, kvq_scales scales,
                       kvq_stream_t stream) {
  int kf = 0, vf = 0;
  int st = decode_format(fmt, &kf, &vf);
  if (st != KVQ_OK) return st;
  if (num_tokens < 0) return KVQ_ERR_INVALID_ARG;
  if (num_tokens == 0) return KVQ_OK;
  if (!k_bf16 || !v_bf16 || !slot_mapping || !caches.k_cache || !caches.v_cache || !scales.k_scale ||
      !scales.v_scale)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(k_bf16) || !aligned16(v_bf16) || !aligned16(caches.k_cache) || !aligned16(caches.v_cache) ||
      !aligned16(scales.k_scale) || !aligned16(scales.v_scale) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return KVQ_ERR_INVALID_ARG;
  unsigned int *err = nullptr;
  if (error_word(&err) != cudaSuccess) return KVQ_ERR_CUDA;
  int sms = 0;
  if ((st = sm_count(&sms)) != KVQ_OK) return st;
  QuantizeArgs a;
  a.k = k_bf16;
  a.v = v_bf16;
  a.slots = slot_mapping;
  a.ntok = num_tokens;
  a.H = fmt->num_kv_heads;
  a.nslots = fmt->num_blocks * fmt->block_size;
  a.kc = static_cast<uint8_t *>(caches.k_cache);
  a.vc = static_cast<uint8_t *>(caches.v_cache);
  a.ks = scales.k_scale;
  a.vs = scales.v_scale;
  a.err = err;
  a.rot = fmt->rotation;
  for (int w = 0; w < 4; ++w) a.rot_signs[w] = fmt->rotation_signs[w];
  return launch_quantize_write(fmt->head_dim, kf, vf, a, sms, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? KVQ_OK
             : KVQ_ERR_CUDA;
}

static int check_decode_shape(const kvq_format *fmt, int32_t batch, int32_t num_q_heads, int *kf, int *vf) {
  int st = decode_format(fmt, kf, vf);
  if (st != KVQ_OK) return st;
  if (batch < 0 || num_q_heads < 1) return KVQ_ERR_INVALID_ARG;
  if (num_q_heads % fmt->num_kv_heads != 0) return KVQ_ERR_INVALID_ARG;
  const int G = num_q_heads / fmt->num_kv_heads;
  if (G > 8) return KVQ_ERR_UNSUPPORTED;
  if (batch > 8192) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

int kvq_decode_workspace_size(const kvq_format *fmt, int32_t batch, int32_t num_q_heads,
                              int32_t max_context_len, size_t *bytes) {
  int kf = 0, vf = 0;
  int st = check_decode_shape(fmt, batch, num_q_heads, &kf, &vf);
  if (st != KVQ_OK) return st;
  if (!bytes || max_context_len < 0) return KVQ_ERR_INVALID_ARG;
  DecodePlan plan;
  if (plan_decode(fmt->head_dim, kf, vf, fmt->num_kv_heads, num_q_heads / fmt->num_kv_heads, batch,
                  fmt->rotation != 0, &plan) !=
      cudaSuccess)
    return KVQ_ERR_CUDA;
  *bytes = ws_layout(batch, fmt->num_kv_heads, fmt->head_dim, plan.max_ctas).total;
  return KVQ_OK;
}

// The kernels count a sequence's positions in 32 bits.
constexpr int32_t kMaxRowBlocks = 1 << 27;

// The decode entry points with a caller workspace; k_new / v_new non-null
// fuse the write of each sequence's new token (kvq_write_decode).
// `weights_stride` >= 0 adds up attention weights (kvq_weigh_decode).
static int run_decode(const void *q_bf16, int32_t batch, int32_t num_q_heads, const kvq_format *fmt,
                      kvq_caches caches, kvq_scales scales, const int32_t *block_tables,
                      int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t max_context_len,
                      float *out, void *workspace, size_t workspace_bytes, kvq_stream_t stream,
                      const void *k_new, const void *v_new, const void *res_k = nullptr,
                      const void *res_v = nullptr, float *weights = nullptr, int64_t weights_stride = -1) {
  int kf = 0, vf = 0;
  int st = check_decode_shape(fmt, batch, num_q_heads, &kf, &vf);
  if (st != KVQ_OK) return st;
  const bool tail = res_k != nullptr || res_v != nullptr;
  if (tail) {
    if (kf != K_INT8_CHAN && kf != K_INT2_CHAN) return KVQ_ERR_UNSUPPORTED;  // the tail belongs to per-channel K
    if (!res_k || !res_v || !aligned16(res_k) || !aligned16(res_v)) return KVQ_ERR_INVALID_ARG;
  }
  const bool weigh = weights_stride >= 0;
  if (weigh && (kf == K_INT8_CHAN || kf == K_INT2_CHAN)) return KVQ_ERR_UNSUPPORTED;
  const bool fused = k_new != nullptr || v_new != nullptr;
  if (fused) {
    if (kf == K_INT8_CHAN || kf == K_INT2_CHAN) return KVQ_ERR_UNSUPPORTED;  // per-channel K blocks take no appends
    if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)) return KVQ_ERR_INVALID_ARG;
  }
  if (batch == 0) return KVQ_OK;
  if (!q_bf16 || !caches.k_cache || !caches.v_cache || !scales.k_scale || !scales.v_scale || !block_tables ||
      !context_lens || !out || !workspace)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(q_bf16) || !aligned16(caches.k_cache) || !aligned16(caches.v_cache) ||
      !aligned16(scales.k_scale) || !aligned16(scales.v_scale) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) || (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
      (reinterpret_cast<uintptr_t>(context_lens) & 3u))
    return KVQ_ERR_INVALID_ARG;
  if (max_blocks_per_seq < 1 || max_context_len < 0) return KVQ_ERR_INVALID_ARG;
  if (max_blocks_per_seq >= kMaxRowBlocks || static_cast<int64_t>(batch) * max_blocks_per_seq >= (int64_t(1) << 31))
    return KVQ_ERR_UNSUPPORTED;
  if (fmt->num_blocks < 1 || fmt->num_blocks >= (int64_t(1) << 31)) return KVQ_ERR_UNSUPPORTED;
  const int H = fmt->num_kv_heads, D = fmt->head_dim, G = num_q_heads / H;
  DecodePlan plan;
  if (plan_decode(D, kf, vf, H, G, batch, fmt->rotation != 0, &plan) != cudaSuccess) return KVQ_ERR_CUDA;
  if (weigh) {
    // the same split as the plain decode's, on kernels of their own
    DecodePlan own;
    if (plan_decode(D, kf, vf, H, G, batch, fmt->rotation != 0, &own, true) != cudaSuccess) return KVQ_ERR_CUDA;
    own.max_ctas = plan.max_ctas;
    plan = own;
  }
  const WsLayout wl = ws_layout(batch, H, D, plan.max_ctas);
  const WeighWs ww = weigh_ws(wl, batch, num_q_heads, max_context_len);
  if (workspace_bytes < (weigh ? ww.total : wl.total)) return KVQ_ERR_WORKSPACE;
  unsigned int *err = nullptr;
  if (error_word(&err) != cudaSuccess) return KVQ_ERR_CUDA;

  DecodeMaps maps;
  if ((st = encode_decode_maps(&maps, caches, scales, fmt->num_blocks, H, D, kf, vf)) != KVQ_OK) return st;

  // CTAs: one resident wave, but no more than one per 4 blocks of the
  // largest possible batch
  const int64_t ctx_cap = max_context_len < max_blocks_per_seq * kBlockSize ? max_context_len
                                                                             : max_blocks_per_seq * kBlockSize;
  const int64_t blocks_ub = static_cast<int64_t>(batch) * ((ctx_cap + kBlockSize - 1) / kBlockSize);
  int64_t P = (blocks_ub + 3) / 4;
  if (P > plan.max_ctas) P = plan.max_ctas;
  if (P < 1) P = 1;

  uint8_t *ws = static_cast<uint8_t *>(workspace);
  DecodeArgs a;
  a.q = static_cast<const uint16_t *>(q_bf16);
  a.ks = scales.k_scale;
  a.vs = scales.v_scale;
  a.tables = block_tables;
  a.ctx = context_lens;
  a.ws_o = reinterpret_cast<float *>(ws + wl.o_off);
  a.ws_ml = reinterpret_cast<float *>(ws + wl.ml_off);
  a.ws_cum = reinterpret_cast<int *>(ws + wl.cum_off);
  a.out = out;
  a.err = err;
  a.num_blocks = fmt->num_blocks;
  a.B = batch;
  a.Hq = num_q_heads;
  a.H = H;
  a.G = G;
  a.max_blocks = max_blocks_per_seq;
  a.max_ctx = max_context_len;
  a.nctas = static_cast<int>(P);
  a.rot = fmt->rotation;
  for (int w = 0; w < 4; ++w) a.rot_signs[w] = fmt->rotation_signs[w];
  if (tail) {
    a.res_k = static_cast<const uint16_t *>(res_k);
    a.res_v = static_cast<const uint16_t *>(res_v);
  }
  if (fused) {
    a.knew = static_cast<const uint16_t *>(k_new);
    a.vnew = static_cast<const uint16_t *>(v_new);
    a.kc_w = static_cast<uint8_t *>(caches.k_cache);
    a.vc_w = static_cast<uint8_t *>(caches.v_cache);
    a.ks_w = scales.k_scale;
    a.vs_w = scales.v_scale;
  }
  if (weigh) {
    a.ws_z = reinterpret_cast<float *>(ws + ww.z_off);
    a.ws_norm = reinterpret_cast<float2 *>(ws + ww.norm_off);
  }
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (launch_decode(D, kf, vf, a, plan, maps, s) != cudaSuccess) return KVQ_ERR_CUDA;
  if (!weigh) return KVQ_OK;
  WeighArgs w;
  w.z = a.ws_z;
  w.norm = a.ws_norm;
  w.cum = a.ws_cum;
  w.tables = block_tables;
  w.ctx = context_lens;
  w.weights = weights;
  w.stride = weights_stride;
  w.num_blocks = fmt->num_blocks;
  w.most_blocks = blocks_ub;
  w.B = batch;
  w.H = H;
  w.G = G;
  w.max_blocks = max_blocks_per_seq;
  int sms = 0;
  if ((st = sm_count(&sms)) != KVQ_OK) return st;
  return launch_weigh(w, sms, s) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

int kvq_paged_decode(const void *q_bf16, int32_t batch, int32_t num_q_heads, const kvq_format *fmt,
                     kvq_caches caches, kvq_scales scales, const int32_t *block_tables,
                     int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t max_context_len,
                     float *out, void *workspace, size_t workspace_bytes, kvq_stream_t stream) {
  return run_decode(q_bf16, batch, num_q_heads, fmt, caches, scales, block_tables, max_blocks_per_seq,
                    context_lens, max_context_len, out, workspace, workspace_bytes, stream, nullptr, nullptr);
}

int kvq_write_decode(const void *q_bf16, const void *k_new_bf16, const void *v_new_bf16, int32_t batch,
                     int32_t num_q_heads, const kvq_format *fmt, kvq_caches caches, kvq_scales scales,
                     const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *context_lens,
                     int32_t max_context_len, float *out, void *workspace, size_t workspace_bytes,
                     kvq_stream_t stream) {
  if (!k_new_bf16 || !v_new_bf16) return KVQ_ERR_INVALID_ARG;
  return run_decode(q_bf16, batch, num_q_heads, fmt, caches, scales, block_tables, max_blocks_per_seq,
                    context_lens, max_context_len, out, workspace, workspace_bytes, stream, k_new_bf16,
                    v_new_bf16);
}

int kvq_kivi_decode(const void *q_bf16, int32_t batch, int32_t num_q_heads, const kvq_format *fmt,
                    kvq_caches caches, kvq_scales scales, const int32_t *block_tables,
                    int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t max_context_len,
                    const void *res_k_bf16, const void *res_v_bf16, float *out, void *workspace,
                    size_t workspace_bytes, kvq_stream_t stream) {
  if (!res_k_bf16 || !res_v_bf16) return KVQ_ERR_INVALID_ARG;
  return run_decode(q_bf16, batch, num_q_heads, fmt, caches, scales, block_tables, max_blocks_per_seq,
                    context_lens, max_context_len, out, workspace, workspace_bytes, stream, nullptr, nullptr,
                    res_k_bf16, res_v_bf16);
}

int kvq_weigh_decode_workspace_size(const kvq_format *fmt, int32_t batch, int32_t num_q_heads,
                                    int32_t max_context_len, size_t *bytes) {
  const int st = kvq_decode_workspace_size(fmt, batch, num_q_heads, max_context_len, bytes);
  if (st != KVQ_OK) return st;
  WsLayout wl = {};
  wl.total = *bytes;
  *bytes = weigh_ws(wl, batch, num_q_heads, max_context_len).total;
  return KVQ_OK;
}

int kvq_weigh_decode(const void *q_bf16, int32_t batch, int32_t num_q_heads, const kvq_format *fmt,
                     kvq_caches caches, kvq_scales scales, const int32_t *block_tables,
                     int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t max_context_len,
                     float *weights, int64_t weights_stride, float *out, void *workspace, size_t workspace_bytes,
                     kvq_stream_t stream) {
  // (arrays without entries may be null)
  if (weights_stride < 0 || weights_stride < max_context_len || (reinterpret_cast<uintptr_t>(weights) & 3u) ||
      (!weights && batch > 0 && weights_stride > 0))
    return KVQ_ERR_INVALID_ARG;
  return run_decode(q_bf16, batch, num_q_heads, fmt, caches, scales, block_tables, max_blocks_per_seq,
                    context_lens, max_context_len, out, workspace, workspace_bytes, stream, nullptr, nullptr,
                    nullptr, nullptr, weights, weights_stride);
}

int kvq_kivi_append(const void *k_new_bf16, const void *v_new_bf16, int32_t batch, const kvq_format *fmt,
                    kvq_caches caches, kvq_scales scales, const int32_t *block_tables,
                    int32_t max_blocks_per_seq, const int32_t *context_lens, void *res_k_bf16,
                    void *res_v_bf16, kvq_stream_t stream) {
  int kf = 0, vf = 0;
  int st = decode_format(fmt, &kf, &vf);
  if (st != KVQ_OK) return st;
  if (kf != K_INT8_CHAN && kf != K_INT2_CHAN) return KVQ_ERR_UNSUPPORTED;
  if (batch < 0 || max_blocks_per_seq < 1) return KVQ_ERR_INVALID_ARG;
  if (batch == 0) return KVQ_OK;
  if (!k_new_bf16 || !v_new_bf16 || !res_k_bf16 || !res_v_bf16 || !block_tables || !context_lens ||
      !caches.k_cache || !caches.v_cache || !scales.k_scale || !scales.v_scale)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(k_new_bf16) || !aligned16(v_new_bf16) || !aligned16(res_k_bf16) || !aligned16(res_v_bf16) ||
      !aligned16(caches.k_cache) || !aligned16(caches.v_cache) || !aligned16(scales.k_scale) ||
      !aligned16(scales.v_scale) || (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
      (reinterpret_cast<uintptr_t>(context_lens) & 3u))
    return KVQ_ERR_INVALID_ARG;
  if (max_blocks_per_seq >= kMaxRowBlocks || static_cast<int64_t>(batch) * max_blocks_per_seq >= (int64_t(1) << 31))
    return KVQ_ERR_UNSUPPORTED;
  unsigned int *err = nullptr;
  if (error_word(&err) != cudaSuccess) return KVQ_ERR_CUDA;
  KiviAppendArgs a;
  a.knew = static_cast<const uint16_t *>(k_new_bf16);
  a.vnew = static_cast<const uint16_t *>(v_new_bf16);
  a.res_k = static_cast<uint16_t *>(res_k_bf16);
  a.res_v = static_cast<uint16_t *>(res_v_bf16);
  a.tables = block_tables;
  a.ctx = context_lens;
  a.kc = static_cast<uint8_t *>(caches.k_cache);
  a.vc = static_cast<uint8_t *>(caches.v_cache);
  a.ks = scales.k_scale;
  a.vs = scales.v_scale;
  a.err = err;
  a.num_blocks = fmt->num_blocks;
  a.B = batch;
  a.H = fmt->num_kv_heads;
  a.max_blocks = max_blocks_per_seq;
  return launch_kivi_append(fmt->head_dim, kf, vf, a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KVQ_OK
             : KVQ_ERR_CUDA;
}

// Device-accessible address of pinned host memory, or null.
static const void *host_device_ptr(const void *p) {
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  if (at.type != cudaMemoryTypeHost || !at.devicePointer) return nullptr;
  return at.devicePointer;
}

// bytes of one block's scales for a granularity
static int64_t block_scale_bytes(int gran, int group, int H, int D) {
  if (gran == KVQ_PER_TOKEN_HEAD) return int64_t(kBlockSize) * H * 4;
  if (gran == KVQ_PER_TOKEN_GROUP) return int64_t(kBlockSize) * H * (D / group) * 4;
  return int64_t(H) * D * 4;
}

int kvq_prefetch_blocks(const kvq_format *fmt, kvq_caches host_caches, kvq_scales host_scales,
                        int64_t host_num_blocks, const int32_t *src_blocks, const int32_t *dst_blocks,
                        int32_t num_pairs, kvq_caches caches, kvq_scales scales, kvq_stream_t stream) {
  int kf = 0, vf = 0;
  int st = decode_format(fmt, &kf, &vf);
  if (st != KVQ_OK) return st;
  if (num_pairs < 0 || host_num_blocks < 0) return KVQ_ERR_INVALID_ARG;
  if (num_pairs == 0) return KVQ_OK;
  if (!src_blocks || !dst_blocks || !caches.k_cache || !caches.v_cache || !scales.k_scale || !scales.v_scale ||
      !host_caches.k_cache || !host_caches.v_cache || !host_scales.k_scale || !host_scales.v_scale)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(caches.k_cache) || !aligned16(caches.v_cache) || !aligned16(scales.k_scale) ||
      !aligned16(scales.v_scale) || !aligned16(host_caches.k_cache) || !aligned16(host_caches.v_cache) ||
      !aligned16(host_scales.k_scale) || !aligned16(host_scales.v_scale) ||
      (reinterpret_cast<uintptr_t>(src_blocks) & 3u) || (reinterpret_cast<uintptr_t>(dst_blocks) & 3u))
    return KVQ_ERR_INVALID_ARG;
  const void *hk = host_device_ptr(host_caches.k_cache), *hv = host_device_ptr(host_caches.v_cache);
  const void *hks = host_device_ptr(host_scales.k_scale), *hvs = host_device_ptr(host_scales.v_scale);
  if (!hk || !hv || !hks || !hvs) return KVQ_ERR_INVALID_ARG;  // not pinned host memory
  unsigned int *err = nullptr;
  if (error_word(&err) != cudaSuccess) return KVQ_ERR_CUDA;
  const int H = fmt->num_kv_heads, D = fmt->head_dim;
  auto row_bytes = [D](int dt) -> int64_t { return dt == KVQ_INT4 ? D / 2 : (dt == KVQ_INT2 ? D / 4 : D); };
  const int64_t krow = row_bytes(fmt->k_dtype), vrow = row_bytes(fmt->v_dtype);
  PrefetchArgs a;
  a.src = src_blocks;
  a.dst = dst_blocks;
  a.n = num_pairs;
  a.host_nb = host_num_blocks;
  a.dev_nb = fmt->num_blocks;
  a.hk = static_cast<const uint4 *>(hk);
  a.hv = static_cast<const uint4 *>(hv);
  a.hks = static_cast<const uint4 *>(hks);
  a.hvs = static_cast<const uint4 *>(hvs);
  a.dk = static_cast<uint4 *>(caches.k_cache);
  a.dv = static_cast<uint4 *>(caches.v_cache);
  a.dks = reinterpret_cast<uint4 *>(scales.k_scale);
  a.dvs = reinterpret_cast<uint4 *>(scales.v_scale);
  a.kb16 = int64_t(kBlockSize) * H * krow / 16;
  a.vb16 = int64_t(kBlockSize) * H * vrow / 16;
  a.ksb16 = block_scale_bytes(fmt->k_gran, fmt->k_group, H, D) / 16;
  a.vsb16 = block_scale_bytes(fmt->v_gran, fmt->v_group, H, D) / 16;
  a.err = err;
  int sms = 0;
  if ((st = sm_count(&sms)) != KVQ_OK) return st;
  return launch_prefetch(a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

// ... and step past a pool table's last entry by less than 2^16.
static bool table_fits(int32_t rows, int32_t max_blocks) {
  return max_blocks < kMaxRowBlocks && static_cast<int64_t>(rows) * max_blocks <= (int64_t(1) << 31) - (1 << 16);
}

static bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

static int check_pool(int32_t num_rows, const int32_t *lens, const int32_t *context_lens, const int32_t *block_tables,
                      int32_t max_blocks, const kvq_block_pool &pool) {
  if (num_rows < 0 || max_blocks < 1 || pool.num_blocks < 0) return KVQ_ERR_INVALID_ARG;
  if (num_rows > 8192 || !table_fits(num_rows, max_blocks) || pool.num_blocks >= (int64_t(1) << 31))
    return KVQ_ERR_UNSUPPORTED;
  if (num_rows > 0 && (!lens || !context_lens || !block_tables)) return KVQ_ERR_INVALID_ARG;
  if (!pool.free_count || (pool.num_blocks > 0 && (!pool.free_list || !pool.ref_counts))) return KVQ_ERR_INVALID_ARG;
  if (!aligned4(lens) || !aligned4(context_lens) || !aligned4(block_tables) || !aligned4(pool.free_list) ||
      !aligned4(pool.free_count) || !aligned4(pool.ref_counts))
    return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

int kvq_assign_blocks(const int32_t *new_lens, int32_t num_rows, int32_t *context_lens, int32_t *block_tables,
                      int32_t max_blocks_per_seq, kvq_block_pool pool, const int32_t *prefix_rows,
                      const int32_t *prefix_blocks, int32_t max_tokens, int32_t *token_offsets,
                      int64_t *slot_mapping, int32_t *positions, kvq_stream_t stream) {
  const int st = check_pool(num_rows, new_lens, context_lens, block_tables, max_blocks_per_seq, pool);
  if (st != KVQ_OK) return st;
  if (max_tokens < 0 || !token_offsets || (max_tokens > 0 && !slot_mapping)) return KVQ_ERR_INVALID_ARG;
  if ((prefix_rows == nullptr) != (prefix_blocks == nullptr)) return KVQ_ERR_INVALID_ARG;
  if (!aligned4(prefix_rows) || !aligned4(prefix_blocks) || !aligned4(token_offsets) || !aligned4(positions) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return KVQ_ERR_INVALID_ARG;
  AssignArgs a;
  if (error_word(&a.err) != cudaSuccess) return KVQ_ERR_CUDA;
  a.new_lens = new_lens;
  a.ctx = context_lens;
  a.tables = block_tables;
  a.free_list = pool.free_list;
  a.free_count = pool.free_count;
  a.ref_counts = pool.ref_counts;
  a.prefix_rows = prefix_rows;
  a.prefix_blocks = prefix_blocks;
  a.token_offsets = token_offsets;
  a.slots = slot_mapping;
  a.positions = positions;
  a.num_blocks = pool.num_blocks;
  a.rows = num_rows;
  a.max_blocks = max_blocks_per_seq;
  a.max_tokens = max_tokens;
  return launch_assign_blocks(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

int kvq_release_blocks(const int32_t *keep_lens, int32_t num_rows, int32_t *context_lens, int32_t *block_tables,
                       int32_t max_blocks_per_seq, kvq_block_pool pool, kvq_stream_t stream) {
  const int st = check_pool(num_rows, keep_lens, context_lens, block_tables, max_blocks_per_seq, pool);
  if (st != KVQ_OK) return st;
  if (num_rows == 0) return KVQ_OK;
  ReleaseArgs a;
  if (error_word(&a.err) != cudaSuccess) return KVQ_ERR_CUDA;
  a.keep = keep_lens;
  a.ctx = context_lens;
  a.tables = block_tables;
  a.free_list = pool.free_list;
  a.free_count = pool.free_count;
  a.ref_counts = pool.ref_counts;
  a.num_blocks = pool.num_blocks;
  a.rows = num_rows;
  a.max_blocks = max_blocks_per_seq;
  return launch_release_blocks(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

// Workspace of an eviction: a record and two lists for each (row, kv head).  A
// token moves into a place that another one leaves: at most half of them do.
static size_t evict_ws(int rows, int heads, int64_t max_positions, size_t *list) {
  const size_t n = static_cast<size_t>(rows) * heads;
  *list = (n * sizeof(EvictMeta) + 255) & ~size_t(255);
  return *list + n * 2 * (max_positions / 2) * sizeof(int);
}

static int check_evict(int32_t num_rows, int32_t num_kv_heads, int32_t max_positions) {
  if (num_rows < 0 || num_kv_heads < 1 || max_positions < 0) return KVQ_ERR_INVALID_ARG;
  return num_rows > 8192 || num_kv_heads > 8 || max_positions > (1 << 30) ? KVQ_ERR_UNSUPPORTED : KVQ_OK;
}

// Whether two arrays of n entries share some.
static bool overlap(const int32_t *a, const int32_t *b, int32_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b), bytes = 4 * static_cast<uintptr_t>(n);
  return a != nullptr && b != nullptr && x < y + bytes && y < x + bytes;
}

int kvq_evict_workspace_size(int32_t num_rows, int32_t num_kv_heads, int32_t max_positions, size_t *bytes) {
  const int st = check_evict(num_rows, num_kv_heads, max_positions);
  if (st != KVQ_OK) return st;
  if (!bytes) return KVQ_ERR_INVALID_ARG;
  size_t list;
  *bytes = evict_ws(num_rows, num_kv_heads, max_positions, &list);
  return KVQ_OK;
}

int kvq_evict_tokens(const int32_t *keep_lens, const int32_t *recent_lens, const int32_t *pinned_lens,
                     int32_t num_rows, const int32_t *context_lens, const int32_t *block_tables,
                     int32_t max_blocks_per_seq, const kvq_format *fmt, kvq_caches caches, kvq_scales scales,
                     const int32_t *ref_counts, float *weights, int32_t max_positions, int32_t *kept_lens,
                     void *workspace, size_t workspace_bytes, kvq_stream_t stream) {
  int kf = 0, vf = 0;
  int st = decode_format(fmt, &kf, &vf);
  if (st != KVQ_OK) return st;
  if (kf == K_INT8_CHAN || kf == K_INT2_CHAN) return KVQ_ERR_UNSUPPORTED;  // a token's codes depend on its block
  if ((st = check_evict(num_rows, fmt->num_kv_heads, max_positions)) != KVQ_OK) return st;
  if (max_blocks_per_seq < 1) return KVQ_ERR_INVALID_ARG;
  if (!table_fits(num_rows, max_blocks_per_seq) || fmt->num_blocks >= (int64_t(1) << 31)) return KVQ_ERR_UNSUPPORTED;
  if (num_rows == 0) return KVQ_OK;
  if (!keep_lens || !recent_lens || !context_lens || !block_tables || (!weights && max_positions > 0) || !kept_lens || !workspace ||
      !caches.k_cache || !caches.v_cache || !scales.k_scale || !scales.v_scale)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned4(keep_lens) || !aligned4(recent_lens) || !aligned4(pinned_lens) || !aligned4(context_lens) ||
      !aligned4(block_tables) || !aligned4(ref_counts) || !aligned4(weights) || !aligned4(kept_lens) ||
      !aligned16(caches.k_cache) || !aligned16(caches.v_cache) || !aligned16(scales.k_scale) ||
      !aligned16(scales.v_scale) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return KVQ_ERR_INVALID_ARG;
  size_t list;
  // written while other CTAs still read theirs
  if (overlap(kept_lens, keep_lens, num_rows) || overlap(kept_lens, recent_lens, num_rows) ||
      overlap(kept_lens, pinned_lens, num_rows) || overlap(kept_lens, context_lens, num_rows))
    return KVQ_ERR_INVALID_ARG;
  if (workspace_bytes < evict_ws(num_rows, fmt->num_kv_heads, max_positions, &list)) return KVQ_ERR_WORKSPACE;
  EvictArgs a;
  if (error_word(&a.err) != cudaSuccess) return KVQ_ERR_CUDA;
  a.keep = keep_lens;
  a.recent = recent_lens;
  a.pinned = pinned_lens;
  a.ctx = context_lens;
  a.tables = block_tables;
  a.refs = ref_counts;
  a.weights = weights;
  a.kept = kept_lens;
  a.kc = static_cast<uint8_t *>(caches.k_cache);
  a.vc = static_cast<uint8_t *>(caches.v_cache);
  a.ks = scales.k_scale;
  a.vs = scales.v_scale;
  a.ws_meta = static_cast<EvictMeta *>(workspace);
  a.ws_list = reinterpret_cast<int *>(static_cast<uint8_t *>(workspace) + list);
  a.num_blocks = fmt->num_blocks;
  a.stride = max_positions;
  a.rows = num_rows;
  a.H = fmt->num_kv_heads;
  a.max_blocks = max_blocks_per_seq;
  a.max_len = static_cast<int>(std::min<int64_t>(max_positions, static_cast<int64_t>(max_blocks_per_seq) * kBlockSize));
  a.cap = max_positions / 2;
  a.krow = kf == K_INT4_TOK ? fmt->head_dim / 2 : fmt->head_dim;
  a.vrow = vf == V_INT4_G32 ? fmt->head_dim / 2 : vf == V_INT2_G32 ? fmt->head_dim / 4 : fmt->head_dim;
  a.vgroups = vf == V_INT4_G32 || vf == V_INT2_G32 ? fmt->head_dim / 32 : 1;
  int sms = 0;
  if ((st = sm_count(&sms)) != KVQ_OK) return st;
  return launch_evict(a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

// Work of a prompt attention: units of so many tokens, and the places of the plan.
struct PromptWs {
  int unit, levels;
  size_t seq, level, place, total;
};

static PromptWs prompt_ws(int seqs, int max_seq, int G) {
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  PromptWs w;
  w.unit = 2 * (128 / G);
  w.levels = std::max(1, static_cast<int>((static_cast<int64_t>(max_seq) + w.unit - 1) / w.unit));
  w.seq = al(sizeof(PromptHead));
  w.level = w.seq + al(static_cast<size_t>(seqs) * sizeof(int2));
  w.place = w.level + al((static_cast<size_t>(w.levels) + 1) * sizeof(int));
  w.total = w.place + al((static_cast<size_t>(w.levels) + 1) * sizeof(int));
  return w;
}

static int check_prompt(int32_t num_seqs, int32_t max_seq_len, int32_t num_q_heads, int32_t num_kv_heads) {
  if (num_seqs < 0 || max_seq_len < 0 || num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0)
    return KVQ_ERR_INVALID_ARG;
  return num_kv_heads > 8 || num_q_heads / num_kv_heads > 8 || num_seqs > 8192 || max_seq_len > (1 << 24)
             ? KVQ_ERR_UNSUPPORTED
             : KVQ_OK;
}

int kvq_prompt_attention_workspace_size(int32_t num_seqs, int32_t max_seq_len, int32_t num_q_heads,
                                        int32_t num_kv_heads, size_t *bytes) {
  const int st = check_prompt(num_seqs, max_seq_len, num_q_heads, num_kv_heads);
  if (st != KVQ_OK) return st;
  if (!bytes) return KVQ_ERR_INVALID_ARG;
  *bytes = prompt_ws(num_seqs, max_seq_len, num_q_heads / num_kv_heads).total;
  return KVQ_OK;
}

int kvq_prompt_attention(const void *q_bf16, int64_t q_stride, const void *k_bf16, int64_t k_stride,
                         const void *v_bf16, int64_t v_stride, const int32_t *seq_offsets, int32_t num_seqs,
                         int64_t num_tokens, int32_t max_seq_len, int32_t num_q_heads, int32_t num_kv_heads,
                         int32_t head_dim, void *out_bf16, float *lse, void *workspace, size_t workspace_bytes,
                         kvq_stream_t stream) {
  int st = check_prompt(num_seqs, max_seq_len, num_q_heads, num_kv_heads);
  if (st != KVQ_OK) return st;
  if (head_dim != 64 && head_dim != 128) return KVQ_ERR_UNSUPPORTED;
  if (num_tokens < 0) return KVQ_ERR_INVALID_ARG;
  const int64_t qrow = static_cast<int64_t>(num_q_heads) * head_dim, krow = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (q_stride < qrow || k_stride < krow || v_stride < krow || q_stride % 8 || k_stride % 8 || v_stride % 8)
    return KVQ_ERR_INVALID_ARG;
  if (num_tokens > (1 << 24) || q_stride > (1 << 24) || k_stride > (1 << 24) || v_stride > (1 << 24))
    return KVQ_ERR_UNSUPPORTED;
  if (num_seqs == 0 || num_tokens == 0 || max_seq_len == 0) return KVQ_OK;
  if (!q_bf16 || !k_bf16 || !v_bf16 || !seq_offsets || !out_bf16 || !workspace) return KVQ_ERR_INVALID_ARG;
  if (!aligned16(q_bf16) || !aligned16(k_bf16) || !aligned16(v_bf16) ||
      (reinterpret_cast<uintptr_t>(out_bf16) & 31u) || !aligned4(seq_offsets) || !aligned4(lse) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return KVQ_ERR_INVALID_ARG;
  const int G = num_q_heads / num_kv_heads;
  // (no sequence is longer than the tokens: a loose bound costs nothing)
  max_seq_len = static_cast<int32_t>(std::min<int64_t>(max_seq_len, num_tokens));
  const PromptWs wl = prompt_ws(num_seqs, max_seq_len, G);
  if (workspace_bytes < wl.total) return KVQ_ERR_WORKSPACE;
  PromptArgs a;
  if (error_word(&a.err) != cudaSuccess) return KVQ_ERR_CUDA;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.offsets = seq_offsets;
  a.out = static_cast<uint16_t *>(out_bf16);
  a.lse = lse;
  a.ws_head = reinterpret_cast<PromptHead *>(ws);
  a.ws_seq = reinterpret_cast<int2 *>(ws + wl.seq);
  a.ws_level = reinterpret_cast<int *>(ws + wl.level);
  a.ws_place = reinterpret_cast<int *>(ws + wl.place);
  a.num_tokens = static_cast<int>(num_tokens);
  a.num_seqs = num_seqs;
  a.max_seq = max_seq_len;
  a.Hq = num_q_heads;
  a.H = num_kv_heads;
  a.G = G;
  a.unit = wl.unit;
  a.levels = wl.levels;
  PromptMaps m;
  if ((st = encode_rows_map(&m.q, q_bf16, num_tokens, num_q_heads, head_dim, q_stride, G, wl.unit / 2)) != KVQ_OK ||
      (st = encode_rows_map(&m.k, k_bf16, num_tokens, num_kv_heads, head_dim, k_stride, 1, 128)) != KVQ_OK ||
      (st = encode_rows_map(&m.v, v_bf16, num_tokens, num_kv_heads, head_dim, v_stride, 1, 128)) != KVQ_OK ||
      (st = encode_rows_map(&m.out, out_bf16, num_tokens, num_q_heads, head_dim, qrow, G, wl.unit / 2)) != KVQ_OK)
    return st;
  int sms = 0;
  if ((st = sm_count(&sms)) != KVQ_OK) return st;
  return launch_prompt_attention(head_dim, a, m, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KVQ_OK
             : KVQ_ERR_CUDA;
}

// Workspace of the shared-prefix decode: the suffix's split decode, then the
// plan and the prefix partials, each 256-aligned.
struct PrefixWs {
  WsLayout sfx;
  size_t groups, seqs, ready, o, ml, total;
};

static PrefixWs prefix_ws(int B, int Hq, int H, int D, int groups, int sfx_ctas, int ctas) {
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  PrefixWs w;
  w.sfx = ws_layout(B, H, D, sfx_ctas);
  const size_t rows = 2 * static_cast<size_t>(B) * Hq + static_cast<size_t>(kPrefixRows) * ctas;
  w.groups = al(w.sfx.total);
  w.seqs = w.groups + al((static_cast<size_t>(groups) + 1) * sizeof(PrefixGroup));
  w.ready = w.seqs + al(4 * static_cast<size_t>(B) * sizeof(int));
  w.o = w.ready + al(sizeof(unsigned long long));
  w.ml = w.o + al(rows * D * sizeof(float));
  w.total = w.ml + al(rows * 2 * sizeof(float));
  return w;
}

// A word that no other call has and that a fresh workspace does not hold by
// chance: a counter from the clock on, its bits mixed (xor-shifts and products by
// odd numbers, which lose nothing).
static unsigned long long call_token() {
  static std::atomic<unsigned long long> next{
      static_cast<unsigned long long>(std::chrono::system_clock::now().time_since_epoch().count())};
  unsigned long long x = next.fetch_add(1, std::memory_order_relaxed);
  for (int i = 0; i < 3; ++i) x = (x ^ (x >> 31)) * 0x9E3779B97F4A7C15ull;
  return x ^ (x >> 31);
}

// CTAs of the prefix kernel: one per SM.
static int prefix_plan(const kvq_format *fmt, int32_t batch, int32_t num_q_heads, int32_t num_groups, int *kf, int *vf,
                       DecodePlan *plan, int *sms) {
  int st = check_decode_shape(fmt, batch, num_q_heads, kf, vf);
  if (st != KVQ_OK) return st;
  if (num_groups < 0) return KVQ_ERR_INVALID_ARG;
  if (num_groups > 8192) return KVQ_ERR_UNSUPPORTED;
  if (batch == 0) return KVQ_OK;
  if (plan_decode(fmt->head_dim, *kf, *vf, fmt->num_kv_heads, num_q_heads / fmt->num_kv_heads, batch,
                  fmt->rotation != 0, plan) != cudaSuccess)
    return KVQ_ERR_CUDA;
  return sm_count(sms);
}

int kvq_prefix_decode_workspace_size(const kvq_format *fmt, int32_t batch, int32_t num_q_heads,
                                     int32_t max_context_len, int32_t num_groups, size_t *bytes) {
  int kf = 0, vf = 0, sms = 0;
  DecodePlan plan;
  const int st = prefix_plan(fmt, batch, num_q_heads, num_groups, &kf, &vf, &plan, &sms);
  if (st != KVQ_OK) return st;
  if (!bytes || max_context_len < 0) return KVQ_ERR_INVALID_ARG;
  *bytes = prefix_ws(batch, num_q_heads, fmt->num_kv_heads, fmt->head_dim, num_groups, plan.max_ctas, sms).total;
  return KVQ_OK;
}

int kvq_prefix_decode(const void *q_bf16, int32_t batch, int32_t num_q_heads, const kvq_format *fmt,
                      kvq_caches caches, kvq_scales scales, const int32_t *block_tables, int32_t max_blocks_per_seq,
                      const int32_t *context_lens, int32_t max_context_len, const int32_t *group_starts,
                      const int32_t *prefix_lens, int32_t num_groups, int32_t max_prefix_len, const void *res_k_bf16,
                      const void *res_v_bf16, void *out_bf16, void *workspace, size_t workspace_bytes,
                      kvq_stream_t stream) {
  if (max_blocks_per_seq >= kMaxRowBlocks) return KVQ_ERR_UNSUPPORTED;
  int kf = 0, vf = 0, sms = 0;
  DecodePlan plan;
  int st = prefix_plan(fmt, batch, num_q_heads, num_groups, &kf, &vf, &plan, &sms);
  if (st != KVQ_OK) return st;
  const bool tail = res_k_bf16 != nullptr || res_v_bf16 != nullptr;
  if (tail) {
    if (kf != K_INT8_CHAN && kf != K_INT2_CHAN) return KVQ_ERR_UNSUPPORTED;  // the tail belongs to per-channel K
    if (!res_k_bf16 || !res_v_bf16 || !aligned16(res_k_bf16) || !aligned16(res_v_bf16)) return KVQ_ERR_INVALID_ARG;
  }
  if (max_blocks_per_seq < 1 || max_context_len < 0 || max_prefix_len < 0) return KVQ_ERR_INVALID_ARG;
  if (batch == 0) return KVQ_OK;
  if (!q_bf16 || !caches.k_cache || !caches.v_cache || !scales.k_scale || !scales.v_scale || !block_tables ||
      !context_lens || !out_bf16 || !workspace || (num_groups > 0 && (!group_starts || !prefix_lens)))
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(q_bf16) || !aligned16(caches.k_cache) || !aligned16(caches.v_cache) || !aligned16(scales.k_scale) ||
      !aligned16(scales.v_scale) || !aligned16(out_bf16) || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      !aligned4(block_tables) || !aligned4(context_lens) || !aligned4(group_starts) || !aligned4(prefix_lens))
    return KVQ_ERR_INVALID_ARG;
  if (static_cast<int64_t>(batch) * max_blocks_per_seq >= (int64_t(1) << 31)) return KVQ_ERR_UNSUPPORTED;
  if (fmt->num_blocks < 1 || fmt->num_blocks >= (int64_t(1) << 31)) return KVQ_ERR_UNSUPPORTED;
  const int H = fmt->num_kv_heads, D = fmt->head_dim, G = num_q_heads / H;
  // Tiles count in 32 bits: a group has nseq * G / 256 row blocks, rounded up,
  // for each kv head, so with two sequences or more in it fewer than nseq.
  const int64_t prefix_blocks = std::min<int64_t>(max_blocks_per_seq, max_prefix_len / kBlockSize);
  if (static_cast<int64_t>(batch) * H * ((prefix_blocks + 7) / 8) >= (int64_t(1) << 31)) return KVQ_ERR_UNSUPPORTED;
  const PrefixWs wl = prefix_ws(batch, num_q_heads, H, D, num_groups, plan.max_ctas, sms);
  if (workspace_bytes < wl.total) return KVQ_ERR_WORKSPACE;
  unsigned int *err = nullptr;
  if (error_word(&err) != cudaSuccess) return KVQ_ERR_CUDA;
  DecodeMaps maps;
  if ((st = encode_decode_maps(&maps, caches, scales, fmt->num_blocks, H, D, kf, vf)) != KVQ_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t *ws = static_cast<uint8_t *>(workspace);

  PrefixArgs p;
  p.q = static_cast<const uint16_t *>(q_bf16);
  p.kc = static_cast<const uint8_t *>(caches.k_cache);
  p.vc = static_cast<const uint8_t *>(caches.v_cache);
  p.ks = scales.k_scale;
  p.vs = scales.v_scale;
  p.tables = block_tables;
  p.ctx = context_lens;
  p.group_starts = group_starts;
  p.prefix_lens = prefix_lens;
  p.res_k = static_cast<const uint16_t *>(res_k_bf16);
  p.res_v = static_cast<const uint16_t *>(res_v_bf16);
  p.ws_groups = reinterpret_cast<PrefixGroup *>(ws + wl.groups);
  p.ws_limit = reinterpret_cast<int *>(ws + wl.seqs);
  p.ws_ctx = p.ws_limit + batch;
  p.ws_off = p.ws_ctx + batch;
  p.ws_group = p.ws_off + batch;
  p.ready = reinterpret_cast<unsigned long long *>(ws + wl.ready);
  p.token = call_token();
  p.ws_o = reinterpret_cast<float *>(ws + wl.o);
  p.ws_ml = reinterpret_cast<float *>(ws + wl.ml);
  p.sfx_o = reinterpret_cast<float *>(ws + wl.sfx.o_off);
  p.sfx_ml = reinterpret_cast<float *>(ws + wl.sfx.ml_off);
  p.sfx_cum = reinterpret_cast<int *>(ws + wl.sfx.cum_off);
  p.out = static_cast<uint16_t *>(out_bf16);
  p.err = err;
  p.num_blocks = fmt->num_blocks;
  p.B = batch;
  p.Hq = num_q_heads;
  p.H = H;
  p.G = G;
  p.groups = num_groups;
  p.max_blocks = max_blocks_per_seq;
  const int64_t held = static_cast<int64_t>(max_blocks_per_seq) * kBlockSize + (tail ? kBlockSize - 1 : 0);
  p.ctx_cap = held < max_context_len ? static_cast<int>(held) : max_context_len;
  p.max_prefix = max_prefix_len;
  p.nctas = sms;
  p.sfx_nctas = plan.max_ctas;
  p.sfx_blocks_per_cta = 1;
  p.rot = fmt->rotation;
  for (int w = 0; w < 4; ++w) p.rot_signs[w] = fmt->rotation_signs[w];

  DecodeArgs a;
  a.q = p.q;
  a.ks = scales.k_scale;
  a.vs = scales.v_scale;
  a.tables = block_tables;
  a.ctx = p.ws_ctx;
  a.ws_o = reinterpret_cast<float *>(ws + wl.sfx.o_off);
  a.ws_ml = reinterpret_cast<float *>(ws + wl.sfx.ml_off);
  a.ws_cum = reinterpret_cast<int *>(ws + wl.sfx.cum_off);
  a.out = nullptr;
  a.err = err;
  a.num_blocks = fmt->num_blocks;
  a.B = batch;
  a.Hq = num_q_heads;
  a.H = H;
  a.G = G;
  a.max_blocks = max_blocks_per_seq;
  a.max_ctx = max_context_len;
  a.nctas = plan.max_ctas;
  a.rot = fmt->rotation;
  for (int w = 0; w < 4; ++w) a.rot_signs[w] = fmt->rotation_signs[w];
  a.res_k = p.res_k;
  a.res_v = p.res_v;
  a.tab_off = p.ws_off;
  a.blocks_per_cta = p.sfx_blocks_per_cta;
  a.split_only = true;

  const bool prefix = num_groups > 0 && max_prefix_len >= kBlockSize;
  a.overlap = prefix ? 2 : 1;
  a.ready = p.ready;
  a.token = p.token;
  if (launch_prefix_plan(p, s) != cudaSuccess) return KVQ_ERR_CUDA;
  if (prefix && launch_prefix_attend(D, kf, vf, p, maps, s) != cudaSuccess) return KVQ_ERR_CUDA;
  if (launch_decode(D, kf, vf, a, plan, maps, s) != cudaSuccess) return KVQ_ERR_CUDA;
  return launch_prefix_merge(D, p, s) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

int kvq_device_errors(uint32_t *bits_out, int32_t clear, kvq_stream_t stream) {
  if (!bits_out) return KVQ_ERR_INVALID_ARG;
  unsigned int *err = nullptr;
  if (error_word(&err) != cudaSuccess) return KVQ_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned int v = 0;
  if (cudaMemcpyAsync(&v, err, sizeof(v), cudaMemcpyDeviceToHost, s) != cudaSuccess) return KVQ_ERR_CUDA;
  if (clear && cudaMemsetAsync(err, 0, sizeof(unsigned int), s) != cudaSuccess) return KVQ_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return KVQ_ERR_CUDA;
  *bits_out = v;
  return KVQ_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Decode without a caller-provided workspace.
//
// Some callers cannot allocate device memory when they call the decode: code
// that runs under an engine or plugin host that owns all device memory and
// forbids allocation on the serving path, or latency-critical loops that
// must not take the allocator's locks or synchronizations.  For them the
// split-K scratch lives in one static device array, allocated when the
// library's module is loaded and held by every GPU that loads the library
// until the process exits.  The array is shared by every call: calls whose
// work overlaps on the GPU (for example on two streams at once) race on it,
// so such callers must order their calls.  Nothing in it has to start at
// zero (every partial the merge reads is written by the same call).
// ---------------------------------------------------------------------------
namespace {

__device__ __align__(256) static unsigned char g_noalloc_scratch[KVQ_NOALLOC_SCRATCH_BYTES];

void *g_noalloc_addr[kMaxDevices] = {};
std::mutex g_noalloc_mu;

// Set-up, once per device with that device current: the device address of
// the array.  (In host code the array's name is only a host-side stand-in.)
cudaError_t noalloc_scratch(void **out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_noalloc_mu);
  if (!g_noalloc_addr[dev]) {
    void *p = nullptr;
    e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (e != cudaSuccess) return e;
    g_noalloc_addr[dev] = p;
  }
  *out = g_noalloc_addr[dev];
  return cudaSuccess;
}

}  // namespace

extern "C" int kvq_paged_decode_noalloc(const void *q_bf16, int32_t batch, int32_t num_q_heads,
                                        const kvq_format *fmt, kvq_caches caches, kvq_scales scales,
                                        const int32_t *block_tables, int32_t max_blocks_per_seq,
                                        const int32_t *context_lens, int32_t max_context_len, float *out,
                                        kvq_stream_t stream) {
  void *scratch = nullptr;
  if (noalloc_scratch(&scratch) != cudaSuccess) return KVQ_ERR_CUDA;
  // the decode with a workspace, on the static array; a shape that needs
  // more than the array holds is refused there with KVQ_ERR_WORKSPACE
  return run_decode(q_bf16, batch, num_q_heads, fmt, caches, scales, block_tables, max_blocks_per_seq,
                    context_lens, max_context_len, out, scratch, KVQ_NOALLOC_SCRATCH_BYTES, stream, nullptr,
                    nullptr);
}
