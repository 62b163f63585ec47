// Append to the 8-bit cache: rows of K and V are quantised to e4m3 or int8
// codes with one power-of-two scale per (layer, page, KV head, K or V) block
// of 64 positions.
//
//   a = max |x| over the block's new rows, e = the least integer with
//   a <= Qmax 2^e (Qmax 448 or 127), code = round(x 2^-e) to nearest even.
//
// A power-of-two scale makes x 2^-e exact, so a code is rounded once, and a
// block whose scale grows with a later row (a call that starts inside it)
// rescales its old codes by a power of two: exact in e4m3 down to its
// subnormals, one more rounding in int8.  The price is at most one bit of
// int8's range against a scale of a / 127.
#include <cuda_bf16.h>

#include "byte_cache.h"
#include "common.cuh"

namespace bgtq {

namespace {

constexpr int kAppThreads = 256;

// The least e >= kByteMinExp with a <= Qmax 2^e, from a's bits (finite, >= 0).
__device__ __forceinline__ int block_exp(float a, int code) {
  // a = (1 + f 2^-23) 2^(x - 127); subnormals fall under the least exponent
  const uint32_t u = __float_as_uint(a);
  const int x = static_cast<int>(u >> 23) - 126;
  const uint32_t f = u & 0x7FFFFFu;
  const int e = code == 0 ? x - 9 + (f > 0x600000u) : x - 7 + (f > 0x7E0000u);
  return e < kByteMinExp ? kByteMinExp : e;
}

// 2^e, e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Two values (already scaled) to two codes; NaN to 0, values past the range to the largest code.
__device__ __forceinline__ uint32_t encode2(float x, float y, int code) {
  if (code == 0) {
    x = x == x ? x : 0.f;
    y = y == y ? y : 0.f;
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
    return r;
  }
  const int a = max(-127, min(127, __float2int_rn(x))), b = max(-127, min(127, __float2int_rn(y)));
  return (a & 255) | ((b & 255) << 8);
}

// Two codes as values.
__device__ __forceinline__ float2 decode2(uint32_t w, int code) {
  if (code == 0) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
  }
  return make_float2(static_cast<float>(static_cast<int8_t>(w & 255)), static_cast<float>(static_cast<int8_t>(w >> 8 & 255)));
}

// Two finite elements of a row, scaled by 2^-e, to two e4m3 codes.  Products
// by a power of two are exact in fp16 (INV: its pair, -15 <= e <= 15) and in
// bf16 but for what lies far under e4m3's least step of 2^-9, which is 0
// either way.
template <bool BF16>
__device__ __forceinline__ uint32_t scale2_e4m3(uint32_t w, uint32_t inv) {
  uint16_t r;
  if constexpr (BF16) {
    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&w), *reinterpret_cast<__nv_bfloat162*>(&inv));
    const uint32_t y = *reinterpret_cast<const uint32_t*>(&x);
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(r)
        : "f"(__uint_as_float(y & 0xFFFF0000u)), "f"(__uint_as_float(y << 16)));
  } else {
    const __half2 x = __hmul2(*reinterpret_cast<__half2*>(&w), *reinterpret_cast<__half2*>(&inv));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  }
  return r;
}

// Four finite elements to four int8 codes: adding 1.5 times the number whose
// last place is 1 rounds to an integer, to nearest even, in the low bits
// (|x 2^-e| <= 127, and the product is exact inside the fused operation).
template <bool BF16>
__device__ __forceinline__ uint32_t scale4_int8(uint32_t w0, uint32_t w1, float inv, uint32_t inv2) {
  if constexpr (BF16) {
    const float m = 12582912.f;  // 1.5 2^23
    const uint32_t a = __float_as_uint(fmaf(__uint_as_float(w0 << 16), inv, m));
    const uint32_t b = __float_as_uint(fmaf(__uint_as_float(w0 & 0xFFFF0000u), inv, m));
    const uint32_t c = __float_as_uint(fmaf(__uint_as_float(w1 << 16), inv, m));
    const uint32_t d = __float_as_uint(fmaf(__uint_as_float(w1 & 0xFFFF0000u), inv, m));
    return prmt(prmt(a, b, 0x0040u), prmt(c, d, 0x0040u), 0x5410u);
  } else {
    const __half2 m = __half2half2(__ushort_as_half(0x6600));  // 1.5 2^10
    const __half2 k = *reinterpret_cast<__half2*>(&inv2);
    const __half2 a = __hfma2(*reinterpret_cast<__half2*>(&w0), k, m), b = __hfma2(*reinterpret_cast<__half2*>(&w1), k, m);
    return prmt(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b), 0x6420u);
  }
}

template <bool BF16>
__device__ __forceinline__ float2 row2(uint32_t w) {
  if constexpr (BF16) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}

// Division by a number the host knows: n / d = n ceil(2^(31 + s) / d) 2^-(31 +
// s) rounded down for n < 2^31, s the least with 2^s >= d (the factor's
// excess over 2^(31 + s) / d is under 1, n times it under 2^(31 + s) / d).
struct Divisor {
  uint32_t d, mul, shift;
  explicit Divisor(uint32_t x) : d(x), shift(31) {
    uint32_t s = 0;
    while ((uint64_t(1) << s) < x) ++s;
    shift += s;
    mul = static_cast<uint32_t>(((uint64_t(1) << shift) + x - 1) / x);
  }
  __device__ __forceinline__ uint32_t split(uint32_t& n) const {  // n becomes the remainder
    const uint32_t q = static_cast<uint32_t>(static_cast<uint64_t>(n) * mul >> shift);
    n -= q * d;
    return q;
  }
};

// A CTA per (layer, sequence, block, KV head, K or V), heads next to one
// another in the grid so that neighbouring CTAs read a row's neighbouring
// heads.  Thread (r, c) of the 16 x 16 holds dimensions 8 c .. 8 c + 7 of
// rows r, r + 16, r + 32, r + 48: 64 bytes in flight a thread, and a row's
// 256 bytes are one warp half's load.  Magnitudes are compared as packed
// 16-bit integers, and finite rows of an ordinary size are converted two
// elements at a time; other rows take the path through fp32, element by
// element (all rows that way: 52 us where this takes 33.5).  Bound by HBM, 2
// bytes read and 1 written an element: 32768 rows of 8 heads take 33.5 us, 92 %
// of the copy rate, at 6 CTAs an SM (4: 36.4).
template <bool BF16, int CODE>
__global__ __launch_bounds__(kAppThreads, 6) void byte_append_kernel(ByteShape sh, ByteCacheDev cache,
                                                                  const int32_t* __restrict__ table, uint32_t* err,
                                                                  int layer0, const uint16_t* __restrict__ k,
                                                                  const uint16_t* __restrict__ v,
                                                                  const int32_t* __restrict__ start_v,
                                                                  const int32_t* __restrict__ count_v, int batch, int n,
                                                                  Divisor kinds, Divisor per_seq, Divisor seqs) {
  const int tid = threadIdx.x;
  // (layer, sequence, block, K or V, head)
  uint32_t h = blockIdx.x;
  uint32_t tb = kinds.split(h), b = per_seq.split(tb), li = seqs.split(b);
  const int kind = h >= static_cast<uint32_t>(sh.n_kv_heads);
  if (kind) h -= sh.n_kv_heads;
  const int layer = layer0 + li;
  const int start = start_v[b], count = count_v[b];
  if (start < 0 || count < 0 || count > n) {
    if (tid == 0) atomicOr(err, kErrArg);
    return;
  }
  if (count == 0) return;  // wherever the sequence stands
  const int64_t past = static_cast<int64_t>(start) + count;
  if (past > sh.capacity && tid == 0) atomicOr(err, kErrCapacity);
  const int end = static_cast<int>(min(past, sh.capacity));  // at most 2^30; slots are fewer than 2^25
  const int t = start / kByteBlock + static_cast<int>(tb);
  if (end <= start || t > (end - 1) / kByteBlock) return;
  int slot;
  if (sh.n_pages == 0) {
    slot = ((layer * sh.max_batch + static_cast<int>(b)) * sh.n_kv_heads + static_cast<int>(h)) * static_cast<int>(sh.ntiles) + t;
  } else {
    const int32_t page = __ldcg(table + static_cast<int64_t>(b) * sh.ntiles + t);
    if (page < 0 || page >= sh.n_pages) {
      if (tid == 0) atomicOr(err, kErrPage);
      return;
    }
    slot = (layer * sh.n_kv_heads + static_cast<int>(h)) * sh.n_pages + page;
  }
  uint8_t* codes = cache.codes[kind] + static_cast<int64_t>(slot) * kByteTileBytes;
  float* scale = cache.scales[kind] + slot;
  const int r = tid >> 4, c = tid & 15;
  const int lo = max(start - t * kByteBlock, 0), hi = min(end - t * kByteBlock, kByteBlock);  // written: [lo, hi)
  const float old_scale = lo > 0 ? __ldcg(scale) : 0.f;

  // the new rows' elements, and their largest finite magnitude
  const int64_t stride = static_cast<int64_t>(sh.n_kv_heads) * 128;
  const uint16_t* x = (kind == 0 ? k : v) +
                      ((static_cast<int64_t>(li) * batch + b) * n + (t * kByteBlock - start + r)) * stride + h * 128 + 8 * c;
  uint4 w[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int p = r + 16 * s;
    w[s] = p >= lo && p < hi ? __ldcs(reinterpret_cast<const uint4*>(x + 16 * s * stride))
                             : make_uint4(0u, 0u, 0u, 0u);
  }
  // the magnitudes' bits order as the magnitudes do; kInf and above: not finite
  constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;
  __shared__ uint32_t red[kAppThreads / 32];
  auto largest = [&](uint32_t x) {
    const uint32_t wm = __reduce_max_sync(0xffffffffu, x);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = wm;
    __syncthreads();
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kAppThreads / 32; ++i) m = max(m, red[i]);
    return m;
  };
  uint32_t pair = 0;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const uint32_t u[4] = {w[s].x, w[s].y, w[s].z, w[s].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) pair = __vmaxu2(pair, u[j] & 0x7FFF7FFFu);
  }
  uint32_t m = largest(max(pair & 0xFFFFu, pair >> 16));
  const bool finite = m < kInf;
  if (!finite) {
    // the largest finite one
    uint32_t x = 0;
    bool bad = false;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t u[4] = {w[s].x, w[s].y, w[s].z, w[s].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = u[j] & 0x7FFFu, d = u[j] >> 16 & 0x7FFFu;
        if (a < kInf) x = max(x, a); else bad = true;
        if (d < kInf) x = max(x, d); else bad = true;
      }
    }
    if (bad) atomicOr(err, kErrNonFinite);
    m = largest(x);
  }
  m = __float_as_uint(row2<BF16>(m).x);
  int e = block_exp(__uint_as_float(m), CODE);
  int grow = 0;  // e - e_old where the block's other codes are to be rescaled
  if (lo > 0) {
    // a block nothing was written to has no power of two in its place: as the least scale
    const uint32_t bits = __float_as_uint(old_scale);
    int e_old = static_cast<int>(bits >> 23 & 255) - 127;
    if ((bits & 0x807FFFFFu) != 0 || e_old < kByteMinExp || e_old > 127) e_old = kByteMinExp;
    if (e > e_old) grow = e - e_old;
    else e = e_old;
  }
  const float inv = pow2(-e);
  // 2^-e as a pair of the rows' type; fp16 has it for -15 <= e <= 15
  const bool packed = finite && (BF16 || (e >= -15 && e <= 15));
  uint32_t inv2;
  if constexpr (BF16)
    inv2 = (__float_as_uint(inv) & 0xFFFF0000u) | __float_as_uint(inv) >> 16;
  else
    inv2 = pack_half2(inv, inv);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int p = r + 16 * s;
    uint2* at = reinterpret_cast<uint2*>(codes + p * 128 + 8 * c);
    uint32_t out[4];
    if (p >= lo && p < hi && packed) {
      if constexpr (CODE == 0)
        *at = make_uint2(scale2_e4m3<BF16>(w[s].x, inv2) | scale2_e4m3<BF16>(w[s].y, inv2) << 16,
                         scale2_e4m3<BF16>(w[s].z, inv2) | scale2_e4m3<BF16>(w[s].w, inv2) << 16);
      else
        *at = make_uint2(scale4_int8<BF16>(w[s].x, w[s].y, inv, inv2), scale4_int8<BF16>(w[s].z, w[s].w, inv, inv2));
      continue;
    } else if (p >= lo && p < hi) {
      const uint32_t u[4] = {w[s].x, w[s].y, w[s].z, w[s].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = row2<BF16>(u[j]);
        out[j] = encode2(f.x * inv, f.y * inv, CODE);
      }
    } else if (grow > 0) {
      const uint2 was = *at;
      const float down = grow > 126 ? 0.f : pow2(-grow);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = decode2((j < 2 ? was.x : was.y) >> (16 * (j & 1)) & 0xFFFFu, CODE);
        out[j] = encode2(f.x * down, f.y * down, CODE);
      }
    } else {
      continue;
    }
    *at = make_uint2(out[0] | out[1] << 16, out[2] | out[3] << 16);
  }
  if (tid == 0) *scale = pow2(e);
}

}  // namespace

cudaError_t launch_byte_append(const ByteShape& s, const ByteCacheDev& c, const int32_t* block_table, uint32_t* err,
                               int layer0, int layer_count, const void* k, const void* v, const int32_t* start,
                               const int32_t* count, int batch, int n, cudaStream_t stream) {
  // n rows touch at most this many blocks, wherever they start
  const int per_seq = (n - 1) / kByteBlock + (n > 1 ? 2 : 1);
  const int64_t ctas = static_cast<int64_t>(layer_count) * batch * per_seq * 2 * s.n_kv_heads;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const uint16_t* kp = static_cast<const uint16_t*>(k);
  const uint16_t* vp = static_cast<const uint16_t*>(v);
  auto launch = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(ctas), kAppThreads, 0, stream>>>(s, c, block_table, err, layer0, kp, vp, start, count,
                                                                    batch, n, Divisor(2 * s.n_kv_heads), Divisor(per_seq), Divisor(batch));
  };
  if (s.code == 0)
    s.bf16 ? launch(byte_append_kernel<true, 0>) : launch(byte_append_kernel<false, 0>);
  else
    s.bf16 ? launch(byte_append_kernel<true, 1>) : launch(byte_append_kernel<false, 1>);
  return cudaGetLastError();
}

}  // namespace bgtq
