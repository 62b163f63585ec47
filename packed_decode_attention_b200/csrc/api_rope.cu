// The C ABI of the rotary positions over several axes (include/bgtq.h):
// argument checks and the launch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "rope.h"
#include "state.h"

using bgtq::aligned16;

namespace {

// `tokens` rows of `width` bytes, one every `stride` bytes.
struct Rows {
  uintptr_t at;
  int64_t stride, width;
};

// Whether no byte belongs to rows of both.
bool disjoint(const Rows& a, const Rows& b, int64_t tokens) {
  if (a.width == 0 || b.width == 0) return true;
  const uintptr_t a_end = a.at + uintptr_t((tokens - 1) * a.stride + a.width);
  const uintptr_t b_end = b.at + uintptr_t((tokens - 1) * b.stride + b.width);
  if (a_end <= b.at || b_end <= a.at) return true;
  if (a.stride != b.stride) return false;
  // slices of one buffer's rows
  const Rows &lo = a.at <= b.at ? a : b, &hi = a.at <= b.at ? b : a;
  const int64_t off = int64_t((hi.at - lo.at) % uintptr_t(lo.stride));
  return off >= lo.width && off + hi.width <= lo.stride;
}

bool same(const Rows& a, const Rows& b) { return a.at == b.at && a.stride == b.stride; }

}  // namespace

extern "C" int bgtq_rope_axes(const bgtq_rope_config* cfg, const void* d_q, int32_t q_stride, const void* d_k,
                              int32_t k_stride, const int32_t* d_pos, int32_t tokens, void* d_q_out,
                              int32_t q_out_stride, void* d_k_out, int32_t k_out_stride, void* stream) {
  if (!cfg || !d_pos) return BGTQ_ERR_NULL;
  if (cfg->n_q_heads < 0 || cfg->n_kv_heads < 0 || cfg->n_q_heads > 65536 || cfg->n_kv_heads > 65536 ||
      cfg->n_q_heads + cfg->n_kv_heads < 1 || cfg->head_dim != bgtq::kD)
    return BGTQ_ERR_INVALID_ARG;
  if ((cfg->n_q_heads > 0 && (!d_q || !d_q_out)) || (cfg->n_kv_heads > 0 && (!d_k || !d_k_out))) return BGTQ_ERR_NULL;
  if (cfg->pairing != 0 && cfg->pairing != 1) return BGTQ_ERR_INVALID_ARG;
  if (cfg->dtype != BGTQ_DTYPE_HALF && cfg->dtype != BGTQ_DTYPE_BFLOAT) return BGTQ_ERR_INVALID_ARG;
  if (!std::isfinite(cfg->base) || !(cfg->base > 1.0)) return BGTQ_ERR_INVALID_ARG;
  if (cfg->n_axes < 1 || cfg->n_axes > 64) return BGTQ_ERR_INVALID_ARG;
  for (int j = 0; j < 64; ++j)
    if (cfg->axis[j] >= cfg->n_axes) return BGTQ_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > (1 << 30)) return BGTQ_ERR_INVALID_ARG;
  const int64_t wq = int64_t(cfg->n_q_heads) * bgtq::kD, wk = int64_t(cfg->n_kv_heads) * bgtq::kD;
  const int64_t strides[4] = {q_stride, q_out_stride, k_stride, k_out_stride};
  for (int i = 0; i < 4; ++i) {
    const int64_t w = i < 2 ? wq : wk;
    if (w > 0 && (strides[i] < w || strides[i] > (int64_t(1) << 30) || strides[i] % 8 != 0)) return BGTQ_ERR_INVALID_ARG;
  }
  if ((wq > 0 && (!aligned16(d_q) || !aligned16(d_q_out))) || (wk > 0 && (!aligned16(d_k) || !aligned16(d_k_out))) ||
      reinterpret_cast<uintptr_t>(d_pos) % 4 != 0)
    return BGTQ_ERR_ALIGNMENT;
  if (tokens == 0) return BGTQ_OK;
  const Rows q{reinterpret_cast<uintptr_t>(d_q), 2 * int64_t(q_stride), 2 * wq};
  const Rows k{reinterpret_cast<uintptr_t>(d_k), 2 * int64_t(k_stride), 2 * wk};
  const Rows qo{reinterpret_cast<uintptr_t>(d_q_out), 2 * int64_t(q_out_stride), 2 * wq};
  const Rows ko{reinterpret_cast<uintptr_t>(d_k_out), 2 * int64_t(k_out_stride), 2 * wk};
  const Rows pos{reinterpret_cast<uintptr_t>(d_pos), 4 * cfg->n_axes, 4 * cfg->n_axes};
  if (!(same(q, qo) || disjoint(q, qo, tokens)) || !(same(k, ko) || disjoint(k, ko, tokens)) ||
      !disjoint(q, ko, tokens) || !disjoint(k, qo, tokens) || !disjoint(qo, ko, tokens) || !disjoint(pos, qo, tokens) ||
      !disjoint(pos, ko, tokens))
    return BGTQ_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return BGTQ_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return BGTQ_ERR_CUDA;
  bgtq::RopeAxesArgs a;
  std::memset(&a, 0, sizeof(a));
  // base^(-j/64) = base^(-(j/8)/8) base^(-(j%8)/64)
  double hi[8], lo[8];
  for (int i = 0; i < 8; ++i) {
    hi[i] = std::pow(cfg->base, -i / 8.0) / 6.283185307179586477;
    lo[i] = std::pow(cfg->base, -i / 64.0);
  }
  for (int j = 0; j < 64; ++j) {
    a.turns[j] = hi[j >> 3] * lo[j & 7];
    a.axis[j] = cfg->axis[j];
  }
  a.pos = d_pos;
  a.q = d_q;
  a.k = d_k;
  a.q_out = d_q_out;
  a.k_out = d_k_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.tokens = tokens;
  a.hq = cfg->n_q_heads;
  a.hkv = cfg->n_kv_heads;
  a.pairing = cfg->pairing;
  const cudaError_t e = bgtq::launch_rope_axes(a, cfg->dtype, sms, bgtq::as_stream(stream));
  return e == cudaSuccess ? BGTQ_OK : e == cudaErrorInvalidConfiguration ? BGTQ_ERR_INVALID_ARG : BGTQ_ERR_CUDA;
}
