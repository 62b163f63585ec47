// The library's state object, shared by the entry points of the packed cache
// (api.cu), of the 8-bit cache (api_byte.cu) and of the pages (api_pages.cu).
#pragma once
#include <stddef.h>

#include <vector>

#include "../../include/bgtq.h"
#include "byte_cache.h"
#include "device_tables.h"
#include "host_tables.h"

struct bgtq_state {
  bgtq_config cfg;
  bgtq::Shape shape;
  bgtq::Workspace ws;
  bgtq::CacheDev cache;
  size_t cache_off[4];
  size_t cache_bytes, ws_bytes;
  int split_tokens = 0;  // 0 = automatic
  int ctas_per_sm = 0;   // resident decode CTAs per SM (looked up on first use)
  int fused_clusters = -1;  // co-resident clusters of the fused decode (looked up on first use; 0: not usable)
  int fused_cluster_size = 8;
  int decode_mode = 0;      // 1: the fused decode where the GPU can run it; 0: rotation + split + combine
  int num_sms = 148;
  int device = -1;       // the CUDA device current at bgtq_create: its buffers live there
  bool ready = false;
  bool have_energy = false;
  std::vector<int8_t> widths;                    // [L][Hkv][64]
  std::vector<bgtq::GroupLayout> layouts;        // [L][Hkv]
  std::vector<float> krot;                       // [L][Hkv][4][128*128] per group, row-major d x d
  std::vector<float> vrot;                       // [L][Hkv][128*128]
  std::vector<uint64_t> energy_q, energy_k;      // [L][Hkv][64][2]
  // an 8-bit cache (bgtq_byte_create): cfg holds the sizes, cache.n_pages and
  // cache.block_table the paging; `ready` stays false, so the packed cache's
  // calls answer BGTQ_ERR_NOT_READY
  bool byte = false;
  bgtq::ByteShape byte_shape;
  bgtq::ByteCacheDev byte_cache;
  CUtensorMap byte_map[2];
  float* byte_partials = nullptr;
  int2* byte_parts = nullptr;
};

namespace bgtq {

// A call that launches or copies runs on the device the state was created
// on: its cache, workspace and tables live there, and a launch on another
// device would read them through the wrong context.
inline int check_device(const bgtq_state* st) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BGTQ_ERR_CUDA;
  return dev == st->device ? BGTQ_OK : BGTQ_ERR_INVALID_ARG;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

// layers [layer, layer + layer_count) of the config (no overflow for any int32 inputs)
inline bool layer_range_ok(const bgtq_config& c, int32_t layer, int32_t layer_count) {
  return layer >= 0 && layer < c.n_layers && layer_count >= 1 && layer_count <= c.n_layers - layer;
}

}  // namespace bgtq
