// Rotary positions over several axes (time, height, width of images and
// video; one axis: plain RoPE).
//
// Block j of the 64 pairs of dimensions turns by the angle
// pos[axis(j)][token] base^(-2j/128).  Angles are taken in turns: the product
// of position and frequency / (2 pi) in fp64, whose fraction is exact, then
// sine and cosine of it in fp32.  The products with the row are fp32, rounded
// once to the row's type.
#include <cuda_bf16.h>

#include "common.cuh"
#include "rope.h"

namespace bgtq {

namespace {

constexpr int kRopeWarps = 4;
constexpr int kRopeHeads = 4;         // heads a warp takes at once: 8 lanes each
constexpr int kRopeAhead = 2;         // (1: 108.0 us, 3: 107.0)

template <bool BF16>
__device__ __forceinline__ float2 wide2(uint32_t w) {
  if constexpr (BF16) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}

template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float x, float y) {
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  return pack_half2(x, y);
}

// A warp per (token, part of the heads).  Lane l computes the sines of blocks
// 2 l and 2 l + 1 once for all heads; lane (h, c) = (l / 8, l % 8) turns
// blocks 8 c .. 8 c + 7 of head h, 16 bytes of each half of the row (pairing
// 0) or 32 in a row (pairing 1).  Bound by HBM: 32768 tokens of 40 heads take
// 107.6 us, 95 % of the copy rate.
template <bool BF16>
__global__ __launch_bounds__(32 * kRopeWarps) void rope_axes_kernel(const __grid_constant__ RopeAxesArgs a) {
  const int lane = threadIdx.x & 31, h = lane >> 3, c = lane & 7;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
  const int64_t token = id / a.parts;
  if (token >= a.tokens) return;
  const int part = static_cast<int>(id - token * a.parts);
  const int heads = a.hq + a.hkv;
  const int first = part * a.part_heads, last = min(heads, first + a.part_heads);
  float s[2], co[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = 2 * lane + i;
    const double turns = a.turns[j] * static_cast<double>(__ldg(a.pos + a.axis[j] * a.tokens + token));
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &s[i], &co[i]);
  }
  float sn[8], cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sn[i] = __shfl_sync(0xffffffffu, s[i & 1], 4 * c + (i >> 1));
    cs[i] = __shfl_sync(0xffffffffu, co[i & 1], 4 * c + (i >> 1));
  }
  const int lo = a.pairing == 0 ? 8 * c : 16 * c, hi = a.pairing == 0 ? 64 + 8 * c : 16 * c + 8;
  // kRopeAhead heads' loads before the first store (which may be to the same
  // rows, so the compiler keeps the order)
#pragma unroll 1
  for (int h0 = first + h; h0 < last; h0 += kRopeAhead * kRopeHeads) {
    uint4 u[kRopeAhead], w[kRopeAhead];
#pragma unroll
    for (int n = 0; n < kRopeAhead; ++n) {
      const int hd = h0 + n * kRopeHeads;
      if (hd >= last) break;
      const uint16_t* x = hd < a.hq ? static_cast<const uint16_t*>(a.q) + token * a.q_stride + 128 * hd
                                    : static_cast<const uint16_t*>(a.k) + token * a.k_stride + 128 * (hd - a.hq);
      u[n] = *reinterpret_cast<const uint4*>(x + lo);
      w[n] = *reinterpret_cast<const uint4*>(x + hi);
    }
#pragma unroll
    for (int n = 0; n < kRopeAhead; ++n) {
      const int hd = h0 + n * kRopeHeads;
      if (hd >= last) break;
      const uint32_t uw[4] = {u[n].x, u[n].y, u[n].z, u[n].w}, ww[4] = {w[n].x, w[n].y, w[n].z, w[n].w};
      uint32_t ou[4], ow[4];
      if (a.pairing == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = wide2<BF16>(uw[i]), r = wide2<BF16>(ww[i]);
          ou[i] = narrow2<BF16>(p.x * cs[2 * i] - r.x * sn[2 * i], p.y * cs[2 * i + 1] - r.y * sn[2 * i + 1]);
          ow[i] = narrow2<BF16>(p.x * sn[2 * i] + r.x * cs[2 * i], p.y * sn[2 * i + 1] + r.y * cs[2 * i + 1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = wide2<BF16>(uw[i]), r = wide2<BF16>(ww[i]);
          ou[i] = narrow2<BF16>(p.x * cs[i] - p.y * sn[i], p.x * sn[i] + p.y * cs[i]);
          ow[i] = narrow2<BF16>(r.x * cs[4 + i] - r.y * sn[4 + i], r.x * sn[4 + i] + r.y * cs[4 + i]);
        }
      }
      uint16_t* y = hd < a.hq ? static_cast<uint16_t*>(a.q_out) + token * a.q_out_stride + 128 * hd
                              : static_cast<uint16_t*>(a.k_out) + token * a.k_out_stride + 128 * (hd - a.hq);
      *reinterpret_cast<uint4*>(y + lo) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
      *reinterpret_cast<uint4*>(y + hi) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
    }
  }
}

}  // namespace

cudaError_t launch_rope_axes(RopeAxesArgs& a, int bf16, int n_sms, cudaStream_t stream) {
  // all heads of a token in one warp, so that the sines are computed once;
  // with few tokens the heads are split until every SM has 16 warps
  const int heads = a.hq + a.hkv, most = (heads + kRopeHeads - 1) / kRopeHeads;
  int64_t parts = (16 * static_cast<int64_t>(n_sms) + a.tokens - 1) / a.tokens;
  if (parts > most) parts = most;
  a.part_heads = (most + static_cast<int>(parts) - 1) / static_cast<int>(parts) * kRopeHeads;
  a.parts = (heads + a.part_heads - 1) / a.part_heads;
  const int64_t ctas = (a.tokens * a.parts + kRopeWarps - 1) / kRopeWarps;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (bf16)
    rope_axes_kernel<true><<<static_cast<unsigned>(ctas), 32 * kRopeWarps, 0, stream>>>(a);
  else
    rope_axes_kernel<false><<<static_cast<unsigned>(ctas), 32 * kRopeWarps, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace bgtq
