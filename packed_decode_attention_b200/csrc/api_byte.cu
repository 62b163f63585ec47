// The C ABI of the 8-bit cache (include/bgtq.h): argument checks, buffer
// carving and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <new>

#include "pages.h"
#include "state.h"

using bgtq::aligned16;
using bgtq::as_stream;
using bgtq::check_device;
using bgtq::layer_range_ok;

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct ByteLayout {
  size_t codes[2], scales[2], cache_total;
  size_t err, partials, parts, ws_total;
};

int64_t blocks_of(int64_t capacity) { return (capacity + bgtq::kByteBlock - 1) / bgtq::kByteBlock; }

// Slots of the cache, estimated in floating point (no overflow for any config).
double slots_estimate(const bgtq_byte_config* c) {
  const double lh = double(c->n_layers) * c->n_kv_heads;
  return c->page_pool_tiles > 0 ? lh * c->page_pool_tiles : lh * c->max_batch * double(blocks_of(c->capacity_tokens));
}

int validate(const bgtq_byte_config* c) {
  if (!c) return BGTQ_ERR_NULL;
  if (c->n_layers < 1 || c->n_layers > 65535 || c->n_kv_heads < 1 || c->n_q_heads < 1 || c->max_batch < 1)
    return BGTQ_ERR_INVALID_ARG;
  if (c->n_q_heads % c->n_kv_heads != 0 || c->n_q_heads / c->n_kv_heads > 16) return BGTQ_ERR_INVALID_ARG;
  if (c->head_dim != bgtq::kD) return BGTQ_ERR_INVALID_ARG;
  if (c->code != BGTQ_CODE_E4M3 && c->code != BGTQ_CODE_INT) return BGTQ_ERR_INVALID_ARG;
  if (c->dtype != BGTQ_DTYPE_HALF && c->dtype != BGTQ_DTYPE_BFLOAT) return BGTQ_ERR_INVALID_ARG;
  if (c->max_q_tokens < 1 || c->max_q_tokens > bgtq::kByteMaxQTokens) return BGTQ_ERR_INVALID_ARG;
  if (c->page_pool_tiles < 0 || c->reserved != 0) return BGTQ_ERR_INVALID_ARG;
  if (c->capacity_tokens < 1 || c->capacity_tokens > (int64_t(1) << 30)) return BGTQ_ERR_INVALID_ARG;
  // the codes' rows of 128 bytes are addressed by an int32 coordinate
  if (slots_estimate(c) * bgtq::kByteBlock > 2147483648.0 - bgtq::kByteBlock) return BGTQ_ERR_INVALID_ARG;
  // a sequence's query and output elements are addressed by an int32 offset
  if (double(c->n_q_heads) * c->max_q_tokens * bgtq::kD > 2147483648.0) return BGTQ_ERR_INVALID_ARG;
  // the workspace's places for each unit of a call
  if (double(c->n_layers) * c->n_q_heads * c->max_q_tokens * double(c->max_batch) > 1125899906842624.0)  // 2^50
    return BGTQ_ERR_INVALID_ARG;
  return BGTQ_OK;
}

size_t slots_of(const bgtq_byte_config* c) {
  const size_t lh = size_t(c->n_layers) * c->n_kv_heads;
  return c->page_pool_tiles > 0 ? lh * size_t(c->page_pool_tiles)
                                : lh * c->max_batch * size_t(blocks_of(c->capacity_tokens));
}

// SMs the workspace's partials are sized for when no device is asked (the
// size must not depend on the current device): the most a split pass uses.
constexpr int kMaxSplitCtas = 160;

ByteLayout plan(const bgtq_byte_config* c) {
  ByteLayout p{};
  const size_t slots = slots_of(c);
  p.codes[0] = 0;
  p.scales[0] = align_up(p.codes[0] + slots * bgtq::kByteTileBytes);
  p.codes[1] = align_up(p.scales[0] + slots * sizeof(float));
  p.scales[1] = align_up(p.codes[1] + slots * bgtq::kByteTileBytes);
  p.cache_total = align_up(p.scales[1] + slots * sizeof(float));
  p.err = 0;
  p.partials = kAlign;
  p.parts = align_up(p.partials + bgtq::byte_partial_bytes(kMaxSplitCtas));
  p.ws_total = align_up(p.parts + bgtq::byte_parts_bytes(c->n_layers, c->n_kv_heads, c->n_q_heads / c->n_kv_heads,
                                                         c->max_batch, c->max_q_tokens));
  return p;
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The map of a codes array: rows of 128 bytes, boxes of half a block's rows.
int code_map(CUtensorMap* map, void* base, size_t slots) {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &found) != cudaSuccess || !fn)
    return BGTQ_ERR_CUDA;
  const cuuint64_t dims[2] = {128, slots * bgtq::kByteBlock};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, bgtq::kByteBlock / 2}, step[2] = {1, 1};
  return reinterpret_cast<EncodeTiled>(fn)(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, step,
                                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? BGTQ_OK
             : BGTQ_ERR_CUDA;
}

// The checks every call on the cache shares.
int check_byte_call(const bgtq_state* st, int32_t layer, int32_t layer_count, int32_t batch) {
  if (!st->byte) return BGTQ_ERR_INVALID_ARG;
  if (st->cache.n_pages > 0 && !st->cache.block_table) return BGTQ_ERR_NOT_READY;
  if (const int dv = check_device(st)) return dv;
  if (!layer_range_ok(st->cfg, layer, layer_count)) return BGTQ_ERR_INVALID_ARG;
  if (batch < 1 || batch > st->cfg.max_batch) return BGTQ_ERR_INVALID_ARG;
  return BGTQ_OK;
}

int status_of(cudaError_t e) {
  if (e == cudaSuccess) return BGTQ_OK;
  return e == cudaErrorInvalidConfiguration ? BGTQ_ERR_INVALID_ARG : BGTQ_ERR_CUDA;
}

}  // namespace

extern "C" {

int bgtq_byte_required_bytes(const bgtq_byte_config* cfg, size_t* cache_bytes, size_t* workspace_bytes) {
  const int v = validate(cfg);
  if (v != BGTQ_OK) return v;
  if (!cache_bytes || !workspace_bytes) return BGTQ_ERR_NULL;
  const ByteLayout p = plan(cfg);
  *cache_bytes = p.cache_total;
  *workspace_bytes = p.ws_total;
  return BGTQ_OK;
}

int bgtq_byte_create(const bgtq_byte_config* cfg, void* d_cache, size_t cache_bytes, void* d_workspace,
                     size_t workspace_bytes, void* stream, bgtq_state** out) {
  const int v = validate(cfg);
  if (v != BGTQ_OK) return v;
  if (!d_cache || !d_workspace || !out) return BGTQ_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(d_cache) | reinterpret_cast<uintptr_t>(d_workspace)) % kAlign) return BGTQ_ERR_ALIGNMENT;
  const ByteLayout p = plan(cfg);
  if (cache_bytes < p.cache_total || workspace_bytes < p.ws_total) return BGTQ_ERR_BUFFER_SIZE;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return BGTQ_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return BGTQ_ERR_CUDA;
  if (bgtq::byte_decode_setup() != cudaSuccess) return BGTQ_ERR_CUDA;
  if (cfg->page_pool_tiles > 0 && bgtq::page_setup() != cudaSuccess) return BGTQ_ERR_CUDA;
  bgtq_state* st = new (std::nothrow) bgtq_state();
  if (!st) return BGTQ_ERR_HOST_ALLOC;
  st->byte = true;
  st->device = dev;
  st->num_sms = sms < kMaxSplitCtas ? sms : kMaxSplitCtas;
  std::memset(&st->cfg, 0, sizeof(st->cfg));
  st->cfg.n_layers = cfg->n_layers;
  st->cfg.n_kv_heads = cfg->n_kv_heads;
  st->cfg.n_q_heads = cfg->n_q_heads;
  st->cfg.head_dim = cfg->head_dim;
  st->cfg.max_batch = cfg->max_batch;
  st->cfg.page_pool_tiles = cfg->page_pool_tiles;
  st->cfg.capacity_tokens = cfg->capacity_tokens;
  std::memset(&st->shape, 0, sizeof(st->shape));
  st->shape.drop_tile = -1;
  std::memset(&st->ws, 0, sizeof(st->ws));
  std::memset(&st->cache, 0, sizeof(st->cache));
  st->cache.n_pages = cfg->page_pool_tiles;
  uint8_t* c8 = static_cast<uint8_t*>(d_cache);
  uint8_t* w8 = static_cast<uint8_t*>(d_workspace);
  for (int i = 0; i < 2; ++i) {
    st->byte_cache.codes[i] = c8 + p.codes[i];
    st->byte_cache.scales[i] = reinterpret_cast<float*>(c8 + p.scales[i]);
    st->cache_off[2 * i] = p.codes[i];
    st->cache_off[2 * i + 1] = p.scales[i];
  }
  st->cache_bytes = p.cache_total;
  st->ws_bytes = p.ws_total;
  st->ws.err = reinterpret_cast<uint32_t*>(w8 + p.err);
  st->byte_partials = reinterpret_cast<float*>(w8 + p.partials);
  st->byte_parts = reinterpret_cast<int2*>(w8 + p.parts);
  bgtq::ByteShape& s = st->byte_shape;
  s.n_layers = cfg->n_layers;
  s.n_kv_heads = cfg->n_kv_heads;
  s.n_q_heads = cfg->n_q_heads;
  s.group = cfg->n_q_heads / cfg->n_kv_heads;
  s.max_batch = cfg->max_batch;
  s.code = cfg->code;
  s.bf16 = cfg->dtype;
  s.max_q_tokens = cfg->max_q_tokens;
  s.capacity = cfg->capacity_tokens;
  s.ntiles = blocks_of(cfg->capacity_tokens);
  s.n_pages = cfg->page_pool_tiles;
  s.n_sms = st->num_sms;
  const size_t slots = slots_of(cfg);
  int r = code_map(&st->byte_map[0], st->byte_cache.codes[0], slots);
  if (r == BGTQ_OK) r = code_map(&st->byte_map[1], st->byte_cache.codes[1], slots);
  cudaStream_t cs = as_stream(stream);
  if (r == BGTQ_OK && (cudaMemsetAsync(st->ws.err, 0, sizeof(uint32_t), cs) != cudaSuccess ||
                       cudaStreamSynchronize(cs) != cudaSuccess))
    r = BGTQ_ERR_CUDA;
  if (r != BGTQ_OK) {
    delete st;
    return r;
  }
  *out = st;
  return BGTQ_OK;
}

int bgtq_byte_append(bgtq_state* st, int32_t layer, int32_t layer_count, const void* d_k, const void* d_v,
                     const int32_t* d_start, const int32_t* d_count, int32_t batch, int32_t n, void* stream) {
  if (!st || (n != 0 && (!d_k || !d_v)) || !d_start || !d_count) return BGTQ_ERR_NULL;
  const int v = check_byte_call(st, layer, layer_count, batch);
  if (v != BGTQ_OK) return v;
  if (n < 0 || n > (1 << 30) / 64) return BGTQ_ERR_INVALID_ARG;
  if (!aligned16(d_k) || !aligned16(d_v) || !aligned16(d_start) || !aligned16(d_count)) return BGTQ_ERR_ALIGNMENT;
  if (n == 0) return BGTQ_OK;
  return status_of(bgtq::launch_byte_append(st->byte_shape, st->byte_cache, st->cache.block_table, st->ws.err, layer,
                                            layer_count, d_k, d_v, d_start, d_count, batch, n, as_stream(stream)));
}

int bgtq_byte_decode_attn(bgtq_state* st, int32_t layer, int32_t layer_count, const void* d_q,
                          const int32_t* d_seq_lens, int32_t batch, int32_t n_q, const bgtq_score* score, void* d_out,
                          void* stream) {
  if (!st || !d_q || !d_seq_lens || !d_out) return BGTQ_ERR_NULL;
  const int v = check_byte_call(st, layer, layer_count, batch);
  if (v != BGTQ_OK) return v;
  if (n_q < 1 || n_q > st->byte_shape.max_q_tokens) return BGTQ_ERR_INVALID_ARG;
  if (!aligned16(d_q) || !aligned16(d_seq_lens) || !aligned16(d_out)) return BGTQ_ERR_ALIGNMENT;
  bgtq::ByteAttnArgs a;
  std::memset(&a, 0, sizeof(a));
  double scale = 0.0;
  if (score) {
    scale = score->scale;
    if (!std::isfinite(scale) || scale < 0.0 || scale > 16384.0) return BGTQ_ERR_INVALID_ARG;
    if (!std::isfinite(score->softcap) || score->softcap < 0.0 || score->softcap > 1e30) return BGTQ_ERR_INVALID_ARG;
    if (score->window < 0) return BGTQ_ERR_INVALID_ARG;
    if (!aligned16(score->d_slopes) || !aligned16(score->d_prefix) || !aligned16(score->d_doc_start))
      return BGTQ_ERR_ALIGNMENT;
    a.cap = static_cast<float>(score->softcap);
    if (score->softcap > 0.0 && a.cap < 1e-30f) return BGTQ_ERR_INVALID_ARG;
    // past the capacity a window hides nothing (and p - window + 1 stays in an int32)
    a.window = score->window >= st->byte_shape.capacity ? 0 : score->window;
    a.slopes = score->d_slopes;
    a.prefix = score->d_prefix;
    a.doc_start = score->d_doc_start;
  }
  a.scale = scale > 0.0 ? static_cast<float>(scale) : 0.08838834764831845f;  // 1 / sqrt(128)
  const bgtq::ByteShape& s = st->byte_shape;
  for (int i = 0; i < 2; ++i) {
    a.map[i] = st->byte_map[i];
    a.scales[i] = st->byte_cache.scales[i];
  }
  a.block_table = st->cache.block_table;
  a.q = d_q;
  a.out = d_out;
  a.seq_lens = d_seq_lens;
  a.partials = st->byte_partials;
  a.parts = st->byte_parts;
  a.err = st->ws.err;
  a.capacity = s.capacity;
  a.ntiles = s.ntiles;
  a.n_pages = s.n_pages;
  a.max_batch = s.max_batch;
  a.hkv = s.n_kv_heads;
  a.hq = s.n_q_heads;
  a.group = s.group;
  a.n_q = n_q;
  a.layer0 = layer;
  a.layer_count = layer_count;
  a.batch = batch;
  a.bf16 = s.bf16;
  a.drop_tile = st->shape.drop_tile;
  return status_of(bgtq::launch_byte_attn(s, a, as_stream(stream)));
}

}  // extern "C"
