// Launch parameters of the 8-bit cache (byte_append.cu, byte_decode.cu),
// shared by the kernels and the C ABI (api_byte.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace bgtq {

constexpr int kByteBlock = 64;                  // positions of a block (one scale for K, one for V)
constexpr int kByteTileBytes = kByteBlock * 128;
constexpr int kByteMaxQTokens = 16;             // query tokens of a sequence in one call
constexpr int kBytePartStride = 132;            // floats of a row's partial: m, l, pad, pad, acc[128]
constexpr int kByteMaxRows = 16;                // query rows a split CTA attends at once
constexpr int kByteMinExp = -100;               // a block's scale is 2^e with e >= this

struct ByteShape {
  int32_t n_layers, n_kv_heads, n_q_heads, group, max_batch;
  int32_t code;         // 0: e4m3, 1: int8
  int32_t bf16;         // rows, queries and outputs: 0 fp16, 1 bf16
  int32_t max_q_tokens;
  int64_t capacity, ntiles;
  int32_t n_pages;      // pages per (layer, KV head); 0: contiguous
  int32_t n_sms;
};

// Slots (blocks) as in the packed cache: contiguous [L][B][H][T], paged [L][H][P].
struct ByteCacheDev {
  uint8_t* codes[2];    // K, V: [slots][64][128]
  float* scales[2];     // K, V: [slots]
};

struct ByteAttnArgs {
  CUtensorMap map[2];             // K, V codes: rows of 128 bytes, boxes of 32 rows, 128-byte swizzle
  const float* scales[2];
  const int32_t* block_table;
  const void* q;
  void* out;
  const int32_t* seq_lens;
  const int32_t* prefix;          // null: 0
  const int32_t* doc_start;       // [batch][n_q]; null: 0
  const float* slopes;            // [n_q_heads]; null: no bias
  float* partials;
  int2* parts;                    // of each unit with steps: the place of the first, and how many
  uint32_t* err;
  int64_t capacity, ntiles;
  int32_t n_pages, max_batch, hkv, hq, group, n_q, layer0, layer_count, batch;
  int32_t window;                 // 0: none
  int32_t bf16, row_blocks, drop_tile;
  float scale;                    // of q . k
  float cap;                      // 0: none
};

// Bytes of the units' parts, and of the split pass's partials (two a CTA).
size_t byte_parts_bytes(int n_layers, int n_kv_heads, int group, int max_batch, int max_q_tokens);
size_t byte_partial_bytes(int n_sms);
// Sets the kernels' shared-memory limits on the current device.
cudaError_t byte_decode_setup();
cudaError_t launch_byte_attn(const ByteShape& s, ByteAttnArgs& a, cudaStream_t stream);
cudaError_t launch_byte_append(const ByteShape& s, const ByteCacheDev& c, const int32_t* block_table, uint32_t* err,
                               int layer0, int layer_count, const void* k, const void* v, const int32_t* start,
                               const int32_t* count, int batch, int n, cudaStream_t stream);

}  // namespace bgtq
