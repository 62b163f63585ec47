// Decode attention over the 8-bit cache (byte_append.cu), with capped,
// biased and masked scores.
//
//   x = scale q . k;  x <- c tanh(x / c);  x <- x - slope_h (p_i - t)
//   out = sum_t softmax(x)_t v_t over the positions t visible to query i,
//
// which stands at p_i = len - n_q + i: t < min(prefix, len), or
// max(doc_start_i, p_i - window + 1) <= t <= p_i.
//
// byte_split_kernel: one pass over the codes with the running maximum and
// sum of a softmax, split over the GPU's CTAs; byte_combine_kernel joins
// the parts of units that more than one CTA attended.
#include <cuda_bf16.h>

#include "byte_cache.h"
#include "common.cuh"

namespace bgtq {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRing = 3;                 // 8 KB buffers a warp: K, V and the next K
constexpr int kByteWaitLimit = 1 << 20;  // polls of up to a microsecond each: about a second
constexpr float kPShift = 14.f;          // softmax weights are held as 2^14 p (see the weights' comment)

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  for (int i = 0; i < kByteWaitLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "n"(1000)
        : "memory");
    if (ok) return true;
  }
  return false;
}

// One block's 64 x 128 codes into shared memory: 16-byte piece c of position
// p lands at piece c ^ (p & 7) (the map's 128-byte swizzle).
__device__ __forceinline__ void copy_block(uint32_t dst, const CUtensorMap* map, int32_t row, uint32_t bar) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "n"(kByteTileBytes) : "memory");
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(0), "r"(row), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Four codes (the bytes of w) as two fp16 pairs: bytes 0, 1 and bytes 2, 3.
// Both formats are exact in fp16.  int8: c + 128 in the low mantissa bits
// of 1024 (0x6400), less 1152.
template <int CODE>
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (CODE == 0) {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = prmt(u, 0x64646464u, 0x4140u), b = prmt(u, 0x64646464u, 0x4342u);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// ---- which blocks a sequence's queries see -----------------------------------

struct SeqBlocks {
  int32_t len;    // 0 where the given length is out of range
  int32_t pre;    // prefix positions, min(prefix, len)
  int32_t n_pre;  // blocks 0 .. n_pre - 1 are seen for the prefix alone
  int32_t t0;     // then blocks t0, t0 + 1, ...
  int32_t n;      // blocks in all
  bool bad;
};

__device__ __forceinline__ int32_t query_lo(const ByteAttnArgs& a, int b, int i, int p) {
  int32_t lo = a.doc_start ? max(0, __ldcg(a.doc_start + static_cast<int64_t>(b) * a.n_q + i)) : 0;
  if (a.window > 0) lo = max(lo, p - a.window + 1);
  return lo;
}

__device__ __forceinline__ SeqBlocks seq_blocks(const ByteAttnArgs& a, int b) {
  SeqBlocks s;
  const int32_t len = __ldcg(a.seq_lens + b);
  s.bad = len < 0 || len > a.capacity;
  s.len = s.bad ? 0 : len;
  s.pre = a.prefix ? min(max(0, __ldcg(a.prefix + b)), s.len) : 0;
  int32_t lo = INT32_MAX;
  if (a.doc_start == nullptr && a.window <= 0) {
    if (s.len > 0) lo = 0;
  } else {
    for (int i = 0; i < a.n_q; ++i) {
      const int p = s.len - a.n_q + i;
      if (p < 0) continue;
      const int32_t l = query_lo(a, b, i, p);
      if (l <= p) lo = min(lo, l);
    }
  }
  const int pre_blocks = (s.pre + kByteBlock - 1) / kByteBlock;
  if (lo == INT32_MAX) {
    s.n_pre = s.n = pre_blocks;
    s.t0 = 0;
  } else {
    s.t0 = lo / kByteBlock;
    s.n_pre = min(pre_blocks, s.t0);
    s.n = s.n_pre + (s.len - 1) / kByteBlock - s.t0 + 1;
  }
  return s;
}

// The work is the blocks of all units (layer, KV head, row block) of all
// sequences, in the order sequence, unit, block; CTA c of `ctas` takes
// blocks [c N / ctas, (c + 1) N / ctas) whatever units they belong to, so
// ragged batches are shared evenly.
__device__ __forceinline__ int active_ctas(int64_t total, int grid) {
  const int64_t c = (total + kWarps - 1) / kWarps;  // at least a block for each warp
  return static_cast<int>(c < grid ? (c < 1 ? 1 : c) : grid);
}

// The CTA that attends block g.
__device__ __forceinline__ int cta_of(int64_t g, int64_t total, int ctas) {
  return static_cast<int>(((g + 1) * ctas - 1) / total);
}

// Sum over the NT threads; red: NT / 32 places.
template <int NT>
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t* red) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((tid & 31) == 0) red[tid >> 5] = x;
  __syncthreads();
  int64_t s = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) s += red[w];
  return s;
}

// ---- the split pass ------------------------------------------------------------

struct Cursor {
  int b, u, j;
  SeqBlocks s;
};

// Moves k blocks on; the caller knows that they exist.
__device__ __forceinline__ void advance(const ByteAttnArgs& a, Cursor& c, int units, int k) {
  c.j += k;
  while (c.j >= c.s.n) {
    c.j -= c.s.n;
    if (++c.u == units) {
      c.u = 0;
      do {
        if (++c.b >= a.batch) { c.b = a.batch - 1; c.j = 0; return; }
        c.s = seq_blocks(a, c.b);
      } while (c.s.n == 0);
    }
  }
}

struct Place {
  int32_t tile;
  int64_t slot;
};

__device__ __forceinline__ Place place_of(const ByteAttnArgs& a, const Cursor& c) {
  Place r;
  r.tile = c.j < c.s.n_pre ? c.j : c.s.t0 + c.j - c.s.n_pre;
  const int lh = c.u / a.row_blocks, li = lh / a.hkv, h = lh - li * a.hkv, layer = a.layer0 + li;
  if (a.n_pages == 0) {
    r.slot = ((static_cast<int64_t>(layer) * a.max_batch + c.b) * a.hkv + h) * a.ntiles + r.tile;
  } else {
    int32_t page = __ldcg(a.block_table + static_cast<int64_t>(c.b) * a.ntiles + r.tile);
    if (page < 0 || page >= a.n_pages) {
      if ((threadIdx.x & 31) == 0) atomicOr(a.err, kErrPage);
      page = 0;
    }
    r.slot = (static_cast<int64_t>(layer) * a.hkv + h) * a.n_pages + page;
  }
  return r;
}

// Shared memory: the warps' rings, then the merge's places.
template <int NB>
struct SplitSmem {
  static constexpr int kRingBytes = kWarps * kRing * kByteTileBytes;
  static constexpr int kMergeFloats = NB * (1024 + 16);      // a warp's acc [32][32 lanes] and (m, l) of 8 NB rows
  static constexpr int kMergeBytes = kWarps / 2 * kMergeFloats * 4;
  static constexpr int kTotal = 1024 + kRingBytes + kMergeBytes;  // 1024: the swizzle's alignment
};

// NB blocks of 8 query rows against one KV head.  The tensor cores take the
// codes as the 16-row operand (m16n8k16): positions for q . k, dimensions
// for p . v, the query rows as the 8 columns, so 8 rows waste nothing and a
// row block's second 8 rows reuse the widened codes.
//
// A warp's lane (g, t) = (lane / 4, lane % 4).  K: row g of an M-tile stands
// for position pi(g) = g / 2 + 4 (g % 2) of its 8, and its K index runs over
// dimensions so that a lane's 16 consecutive codes (one 16-byte load, piece
// t + 4 i of the position) are the words of 4 chunks.  V: lane g holds the 16
// dimensions of piece sigma(g) = g / 2 + 4 (g % 2) and positions t, t + 4,
// t + 8, t + 12 of each 16, which is the order pi gives p.  With the 128-byte
// swizzle both loads touch all 32 banks in every 8-lane phase.
//
// The scores of a lane belong to columns (rows of q) 2 t and 2 t + 1; p is
// turned into the second product's operand by movmatrix.
//
// HBM bound: 16.4 KB a block and KV head.  At the copy rate a block may take
// about 730 cycles of an SM; its instructions take about 300 (NB = 1).
template <int CODE, int NB>
__global__ __launch_bounds__(kThreads, 1) void byte_split_kernel(const __grid_constant__ ByteAttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[kWarps * kRing];
  __shared__ int64_t red[kWarps];
  __shared__ int64_t found_base;
  __shared__ int found_b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  float* merge = reinterpret_cast<float*>(smem_raw + (ring0 - smem_u32(smem_raw)) + SplitSmem<NB>::kRingBytes);
  const uint32_t ring = ring0 + warp * kRing * kByteTileBytes;
  const uint32_t bar0 = smem_u32(&bars[warp * kRing]);
  if (tid < kWarps * kRing) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&bars[tid])) : "memory");
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // this CTA's blocks [r0, r1) of the call's
  const int units = a.layer_count * a.hkv * a.row_blocks;
  SeqBlocks mine{};
  int64_t sum = 0;
  for (int b = tid; b < a.batch; b += kThreads) {
    const SeqBlocks s = seq_blocks(a, b);
    if (b == tid) mine = s;
    if (s.bad && blockIdx.x == 0) atomicOr(a.err, kErrSeqLen);
    sum += s.n;
  }
  const int64_t total = units * block_sum<kThreads>(sum, red);
  if (total == 0) return;
  const int ctas = active_ctas(total, gridDim.x);
  if (static_cast<int>(blockIdx.x) >= ctas) return;
  const int64_t r0 = blockIdx.x * total / ctas, r1 = (blockIdx.x + 1) * total / ctas;
  {
    int64_t before = 0;  // blocks of the sequences before this chunk of 256
    for (int base = 0; base < a.batch; base += kThreads) {
      const int b = base + tid;
      const int n = b < a.batch ? (base == 0 ? mine.n : seq_blocks(a, b).n) : 0;
      int64_t incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      __syncthreads();
      if (lane == 31) red[warp] = incl;
      __syncthreads();
      int64_t all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) incl += red[w];
        all += red[w];
      }
      const int64_t first = (before + incl - n) * units;
      if (n > 0 && first <= r0 && r0 < first + static_cast<int64_t>(n) * units) {
        found_b = b;
        found_base = first;
      }
      before += all;
      if (before * units > r0) break;
    }
    __syncthreads();
  }
  Cursor seg;  // the start of the segment (a unit's blocks in this CTA's range)
  seg.b = found_b;
  seg.s = seq_blocks(a, seg.b);
  {
    const int64_t off = r0 - found_base;
    seg.u = static_cast<int>(off / seg.s.n);
    seg.j = static_cast<int>(off - static_cast<int64_t>(seg.u) * seg.s.n);
  }
  const int mine_total = static_cast<int>(r1 - r0);

  // this warp's blocks: warp, warp + 8, ... of the CTA's; copies run one and
  // a half blocks ahead (K, V, next K)
  const int nt = mine_total > warp ? (mine_total - warp + kWarps - 1) / kWarps : 0;
  Cursor cur = seg;
  float ks = 0.f, vs = 0.f, ks_next = 0.f, vs_next = 0.f;
  uint32_t pending = 0;    // bit i: a copy into buffer i is on its way
  auto issue = [&](int kind, const Place& pl, int buf) {
    if (pl.tile == a.drop_tile) return;
    pending |= 1u << buf;
    if (lane == 0)
      copy_block(ring + buf * kByteTileBytes, &a.map[kind], static_cast<int32_t>(pl.slot * kByteBlock), bar0 + 8 * buf);
  };
  Place ahead{};
  if (nt > 0) {
    advance(a, cur, units, warp);
    const Place p0 = place_of(a, cur);
    issue(0, p0, 0);
    issue(1, p0, 1);
    ks = __ldcg(a.scales[0] + p0.slot);
    vs = __ldcg(a.scales[1] + p0.slot);
  }
  if (nt > 1) {
    advance(a, cur, units, kWarps);
    ahead = place_of(a, cur);
    issue(0, ahead, 2);
    ks_next = __ldcg(a.scales[0] + ahead.slot);
    vs_next = __ldcg(a.scales[1] + ahead.slot);
  }
  int it = 0;              // the warp's next block
  int buf = 0;             // its K buffer; its V buffer is the next one
  uint32_t phases = 0;     // bit i: parity of buffer i's next completion
  bool dead = false;
  auto wait = [&](int i) {
    if (__all_sync(0xffffffffu, bar_wait(bar0 + 8 * i, phases >> i & 1))) {
      phases ^= 1u << i;
      pending &= ~(1u << i);
    } else {
      dead = true;
    }
  };
  int f0 = 0;              // blocks of the CTA's range before this segment
  const int pig = (g >> 1) | ((g & 1) << 2);

  while (f0 < mine_total) {
    const int len_seg = min(seg.s.n - seg.j, mine_total - f0);
    const int lh = seg.u / a.row_blocks, rb = seg.u - lh * a.row_blocks;
    const int li = lh / a.hkv, h = lh - li * a.hkv;
    const int rows = a.group * a.n_q, row0 = rb * 8 * NB;
    const int len = seg.s.len, pre = seg.s.pre;

    // q as the products' 8-column operand, scaled by a power of two a row so
    // that its largest element lies in [2^14, 2^15): fp16 and bf16 queries
    // are then both exact in fp16 but for elements under 2^-29 of the
    // largest
    uint32_t qf[NB][16];
    float colf[NB][2], slope[NB][2];
    int lo[NB][2], hi[NB][2], rpre[NB][2], tref[NB][2];
    int lo_max = 0, hi_min = INT32_MAX;
    if (it < nt && warp + kWarps * it < f0 + len_seg) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int row = row0 + nb * 8 + g;
        float x[32];
        if (row < rows) {
          const int i = row / a.group, hg = row - i * a.group;
          const uint16_t* qp = static_cast<const uint16_t*>(a.q) +
                               (((static_cast<int64_t>(li) * a.batch + seg.b) * a.n_q + i) * a.hq + h * a.group + hg) * 128;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const uint4 w = *reinterpret_cast<const uint4*>(qp + 16 * (t + 4 * (p >> 1)) + 8 * (p & 1));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = a.bf16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[e]))
                                      : __half22float2(*reinterpret_cast<const __half2*>(&u[e]));
              x[8 * p + 2 * e] = f.x;
              x[8 * p + 2 * e + 1] = f.y;
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = 0.f;
        }
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) m = fmaxf(m, fabsf(x[e]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        // 2^up m in [2^14, 2^15); zero and non-finite rows as they are
        const int ex = static_cast<int>(__float_as_uint(m) >> 23);
        const int up = ex == 0 || ex == 255 ? 0 : max(-113, min(113, 141 - ex));
        const float fac = __int_as_float((up + 127) << 23);
#pragma unroll
        for (int e = 0; e < 16; ++e) qf[nb][e] = pack_half2(x[2 * e] * fac, x[2 * e + 1] * fac);
        const float back = __int_as_float((127 - up) << 23) * a.scale;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          colf[nb][c] = __shfl_sync(0xffffffffu, back, 4 * (2 * t + c));
          const int r = row0 + nb * 8 + 2 * t + c;
          if (r < rows) {
            const int i = r / a.group, hg = r - i * a.group, p = len - a.n_q + i;
            lo[nb][c] = query_lo(a, seg.b, i, p);
            hi[nb][c] = p;
            rpre[nb][c] = pre;
            lo_max = max(lo_max, lo[nb][c]);
            hi_min = min(hi_min, p);
            slope[nb][c] = a.slopes ? __ldg(a.slopes + h * a.group + hg) * kLog2e : 0.f;
            // distances count from the row's last visible position: its
            // weights do not change, and the near ones stay exact
            tref[nb][c] = max(lo[nb][c] <= p ? p : -1, pre - 1);
          } else {
            lo[nb][c] = 1;
            hi[nb][c] = 0;
            rpre[nb][c] = 0;
            slope[nb][c] = 0.f;
            tref[nb][c] = 0;
          }
        }
      }
      lo_max = __reduce_max_sync(0xffffffffu, lo_max);
      hi_min = __reduce_min_sync(0xffffffffu, hi_min);
    }

    float m[NB][2], l[NB][2], acc[NB][8][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m[nb][0] = m[nb][1] = -CUDART_INF_F;
      l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nb][u][e] = 0.f;
    }

    for (; it < nt && warp + kWarps * it < f0 + len_seg; ++it) {
      const int j = seg.j + warp + kWarps * it - f0;
      const int p0 = kByteBlock * (j < seg.s.n_pre ? j : seg.s.t0 + j - seg.s.n_pre);
      const int vbuf = buf == kRing - 1 ? 0 : buf + 1;
      const int nbuf = vbuf == kRing - 1 ? 0 : vbuf + 1;  // the next block's K
      Place after{};
      const bool more = it + 2 < nt && !dead;
      if (more) {
        advance(a, cur, units, kWarps);
        after = place_of(a, cur);
      }
      if (!dead) wait(buf);
      float S[NB][4][4];
      if (!dead) {
        const uint32_t kb = ring + buf * kByteTileBytes + pig * 128;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t piece = ((t + 4 * i) ^ pig) * 16;
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            const uint4 x = lds128(kb + mt * 2048 + piece), y = lds128(kb + mt * 2048 + 1024 + piece);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t a0, a1, a2, a3;
              widen<CODE>(xw[w], a0, a2);
              widen<CODE>(yw[w], a1, a3);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                if (i == 0 && w == 0)
                  mma16816_zero(S[nb][mt], a0, a1, a2, a3, qf[nb][0], qf[nb][1]);
                else
                  mma16816(S[nb][mt], a0, a1, a2, a3, qf[nb][8 * i + 2 * w], qf[nb][8 * i + 2 * w + 1]);
              }
            }
          }
        }
      }
      __syncwarp();
      if (it + 1 < nt && !dead) issue(1, ahead, buf);  // the K buffer is free: the next block's V
      uint32_t pf[NB][4][2];
      if (!dead) {
        const bool full = (p0 >= lo_max && p0 + kByteBlock - 1 <= hi_min) || p0 + kByteBlock <= pre;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          // scores in log2 units
          const float f0c = colf[nb][0] * ks, f1c = colf[nb][1] * ks;
          if (a.cap > 0.f) {
            const float ic = 1.f / a.cap, oc = a.cap * kLog2e;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // tanh u = 1 - 2 / (1 + e^2u); the series' first terms where
                // that cancels, so that the error stays relative
                const float u = S[nb][mt][e] * ((e & 1) ? f1c : f0c) * ic, s = u * u;
                const float far = 1.f - __fdividef(2.f, 1.f + ex2(2.f * kLog2e * u));
                const float near = u * (1.f + s * (-1.f / 3 + s * (2.f / 15 + s * (-17.f / 315))));
                S[nb][mt][e] = (fabsf(u) < 0.2f ? near : far) * oc;
              }
          } else {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) S[nb][mt][e] *= ((e & 1) ? f1c : f0c) * kLog2e;
          }
          if (a.slopes) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                S[nb][mt][e] += slope[nb][e & 1] * static_cast<float>(p0 + 16 * mt + 8 * (e >> 1) + pig - tref[nb][e & 1]);
          }
          if (!full) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int p = p0 + 16 * mt + 8 * (e >> 1) + pig;
                const bool see = p < rpre[nb][e & 1] || (p >= lo[nb][e & 1] && p <= hi[nb][e & 1]);
                if (!see) S[nb][mt][e] = -CUDART_INF_F;
              }
          }
          float mx[2] = {m[nb][0], m[nb][1]};
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e & 1] = fmaxf(mx[e & 1], S[nb][mt][e]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
          }
          if (__any_sync(0xffffffffu, mx[0] != m[nb][0] || mx[1] != m[nb][1])) {
            // a row nothing of which was visible has m = -inf and acc = l = 0
            const float al[2] = {mx[0] == m[nb][0] ? 1.f : ex2(m[nb][0] - mx[0]),
                                 mx[1] == m[nb][1] ? 1.f : ex2(m[nb][1] - mx[1])};
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[nb][u][e] *= al[e & 1];
            l[nb][0] *= al[0];
            l[nb][1] *= al[1];
            m[nb][0] = mx[0];
            m[nb][1] = mx[1];
          }
          // weights 2^14 2^(x - m) in fp16: the tensor cores' type, rounded
          // once (2^-11 relative); the factor keeps weights down to 2^-28 of
          // the largest out of fp16's subnormals, and cancels in acc / l
          const float s0 = mx[0] == -CUDART_INF_F ? 0.f : kPShift - mx[0];
          const float s1 = mx[1] == -CUDART_INF_F ? 0.f : kPShift - mx[1];
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            pf[nb][mt][0] = transpose8x8(pack_half2(ex2(S[nb][mt][0] + s0), ex2(S[nb][mt][1] + s1)));
            pf[nb][mt][1] = transpose8x8(pack_half2(ex2(S[nb][mt][2] + s0), ex2(S[nb][mt][3] + s1)));
          }
          // l: the columns' sums of the rounded weights, by ones on the tensor cores
          float lt[4];
          mma16816_zero(lt, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, pf[nb][0][0], pf[nb][0][1]);
#pragma unroll
          for (int mt = 1; mt < 4; ++mt)
            mma16816(lt, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, pf[nb][mt][0], pf[nb][mt][1]);
          l[nb][0] += lt[0];
          l[nb][1] += lt[1];
        }
      }
      if (!dead) wait(vbuf);
      if (!dead) {
        const uint32_t vb = ring + vbuf * kByteTileBytes;
        if (CODE == 0 && p0 + kByteBlock > len) {
          // positions behind the sequence may hold anything, and a NaN code
          // times a zero weight is NaN
          for (int p = len - p0; p < kByteBlock; ++p)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(vb + p * 128 + lane * 4), "r"(0) : "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        // 4 of the 8 M-tiles (dimension pairs) at a time: half of each 16-byte piece
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float T[NB][4][4];
          const uint32_t at0 = vb + t * 128 + ((pig ^ t) * 16) + half * 8;
          const uint32_t at1 = vb + t * 128 + ((pig ^ t ^ 4) * 16) + half * 8;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint2 x = lds64(at0 + kk * 2048), y = lds64(at1 + kk * 2048 + 512);
            const uint2 z = lds64(at0 + kk * 2048 + 1024), w = lds64(at1 + kk * 2048 + 1536);
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              const uint32_t xd = d ? x.y : x.x, yd = d ? y.y : y.x, zd = d ? z.y : z.x, wd = d ? w.y : w.x;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t sel = e ? 0x7362u : 0x5140u;
                uint32_t a0, a1, a2, a3;
                widen<CODE>(prmt(xd, yd, sel), a0, a1);
                widen<CODE>(prmt(zd, wd, sel), a2, a3);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                  if (kk == 0)
                    mma16816_zero(T[nb][2 * d + e], a0, a1, a2, a3, pf[nb][kk][0], pf[nb][kk][1]);
                  else
                    mma16816(T[nb][2 * d + e], a0, a1, a2, a3, pf[nb][kk][0], pf[nb][kk][1]);
                }
              }
            }
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[nb][4 * half + u][e] = fmaf(T[nb][u][e], vs, acc[nb][4 * half + u][e]);
        }
      }
      __syncwarp();
      ks = ks_next;
      vs = vs_next;
      ahead = after;
      if (more && !dead) {
        issue(0, after, vbuf);  // the V buffer is free: K of the block after the next
        ks_next = __ldcg(a.scales[0] + after.slot);
        vs_next = __ldcg(a.scales[1] + after.slot);
      }
      buf = nbuf;
    }

    // merge of the 8 warps: a tree through shared memory, in a fixed order
#pragma unroll 1
    for (int s = kWarps / 2; s > 0; s >>= 1) {
      float* at = merge + (warp >= s ? warp - s : warp) * SplitSmem<NB>::kMergeFloats;
      if (warp >= s && warp < 2 * s) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) at[(nb * 32 + u * 4 + e) * 32 + lane] = acc[nb][u][e];
          if (g == 0) {
            float* ml = at + NB * 1024 + nb * 16 + t * 4;
            ml[0] = m[nb][0];
            ml[1] = m[nb][1];
            ml[2] = l[nb][0];
            ml[3] = l[nb][1];
          }
        }
      }
      __syncthreads();
      if (warp < s) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float* ml = at + NB * 1024 + nb * 16 + t * 4;
          float ca[2], cb[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float mo = ml[c], mn = fmaxf(m[nb][c], mo);
            ca[c] = m[nb][c] == mn ? 1.f : ex2(m[nb][c] - mn);
            cb[c] = mo == mn ? 1.f : ex2(mo - mn);
            m[nb][c] = mn;
            l[nb][c] = l[nb][c] * ca[c] + ml[2 + c] * cb[c];
          }
#pragma unroll
          for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[nb][u][e] = acc[nb][u][e] * ca[e & 1] + at[(nb * 32 + u * 4 + e) * 32 + lane] * cb[e & 1];
        }
      }
      __syncthreads();
    }
    if (warp == 0) {
      const bool whole = seg.j == 0 && len_seg == seg.s.n;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int rl = nb * 8 + 2 * t + c, row = row0 + rl;
          if (row >= rows) continue;
          if (whole) {
            const int i = row / a.group, hg = row - i * a.group;
            uint16_t* op = static_cast<uint16_t*>(a.out) +
                           (((static_cast<int64_t>(li) * a.batch + seg.b) * a.n_q + i) * a.hq + h * a.group + hg) * 128 +
                           16 * pig;
            const float inv = l[nb][c] == 0.f ? 0.f : 1.f / l[nb][c];
            uint32_t o[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const float x = acc[nb][u][c] * inv, y = acc[nb][u][2 + c] * inv;
              if (a.bf16) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
                o[u] = *reinterpret_cast<const uint32_t*>(&v);
              } else {
                o[u] = pack_half2(x, y);
              }
            }
            reinterpret_cast<uint4*>(op)[0] = make_uint4(o[0], o[1], o[2], o[3]);
            reinterpret_cast<uint4*>(op)[1] = make_uint4(o[4], o[5], o[6], o[7]);
          } else {
            // place 0: the segment that opens this CTA's range; 1: a later one
            float* pp = a.partials + ((static_cast<int64_t>(blockIdx.x) * 2 + (f0 > 0)) * kByteMaxRows + rl) * kBytePartStride;
            if (g == 0) {
              pp[0] = m[nb][c];
              pp[1] = l[nb][c];
            }
#pragma unroll
            for (int u = 0; u < 8; u += 2)
              *reinterpret_cast<float4*>(pp + 4 + 16 * pig + 2 * u) =
                  make_float4(acc[nb][u][c], acc[nb][u][2 + c], acc[nb][u + 1][c], acc[nb][u + 1][2 + c]);
          }
        }
    }
    f0 += len_seg;
    if (f0 < mine_total) advance(a, seg, units, len_seg);
  }
  if (dead) {
    if (lane == 0) atomicOr(a.err, kErrTimeout);
    // copies on their way land (bounded) before the shared memory goes
    for (int i = 0; i < kRing; ++i)
      if (pending >> i & 1) bar_wait(bar0 + 8 * i, phases >> i & 1);
  }
}

// ---- the join ------------------------------------------------------------------

constexpr int kCombThreads = 128;
constexpr int kCombMaxParts = 1024;  // CTAs of a split pass

// A CTA per (sequence, unit, row): the unit's parts, in the order of their
// CTAs, joined by their maxima and sums.  Rows of units that one CTA attended
// whole are done; rows that see nothing become 0.
__global__ __launch_bounds__(kCombThreads) void byte_combine_kernel(const __grid_constant__ ByteAttnArgs a, int split_grid,
                                                                    int rows_per_unit) {
  __shared__ int64_t red[kCombThreads / 32];
  __shared__ float wgt[kCombMaxParts];
  __shared__ float accs[kCombThreads / 32][128];
  __shared__ float fred[kCombThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int units = a.layer_count * a.hkv * a.row_blocks;
  int id = blockIdx.x;
  const int rl = id % rows_per_unit;
  id /= rows_per_unit;
  const int u = id % units, b = id / units;
  const int lh = u / a.row_blocks, rb = u - lh * a.row_blocks, li = lh / a.hkv, h = lh - li * a.hkv;
  const int row = rb * rows_per_unit + rl;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= a.group * a.n_q) return;
  int64_t sum = 0, before = 0;
  for (int i = tid; i < a.batch; i += kCombThreads) {
    const int n = seq_blocks(a, i).n;
    sum += n;
    if (i < b) before += n;
  }
  const int64_t total = units * block_sum<kCombThreads>(sum, red);
  before = block_sum<kCombThreads>(before, red);
  const int n = seq_blocks(a, b).n;
  const int i = row / a.group, hg = row - i * a.group;
  uint16_t* op = static_cast<uint16_t*>(a.out) +
                 (((static_cast<int64_t>(li) * a.batch + b) * a.n_q + i) * a.hq + h * a.group + hg) * 128;
  if (n == 0) {
    op[tid] = 0;
    return;
  }
  const int ctas = active_ctas(total, split_grid);
  const int64_t s = before * units + static_cast<int64_t>(u) * n;
  const int c0 = cta_of(s, total, ctas), c1 = cta_of(s + n - 1, total, ctas);
  if (c0 == c1) return;
  const int parts = c1 - c0 + 1;
  const int first = static_cast<int64_t>(c0) * total / ctas == s ? 0 : 1;  // the unit's place in CTA c0
  auto part = [&](int k) {
    return a.partials + ((static_cast<int64_t>(c0 + k) * 2 + (k == 0 ? first : 0)) * kByteMaxRows + rl) * kBytePartStride;
  };
  float mx = -CUDART_INF_F;
  for (int k = tid; k < parts; k += kCombThreads) {
    const float m = __ldcg(part(k));
    wgt[k] = m;
    mx = fmaxf(mx, m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) fred[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kCombThreads / 32; ++w) mx = fmaxf(mx, fred[w]);
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = warp; k < parts; k += kCombThreads / 32) {
    const float* pp = part(k);
    const float m = wgt[k], w = m == mx ? 1.f : ex2(m - mx);
    const float4 x = __ldcg(reinterpret_cast<const float4*>(pp + 4) + lane);
    l += w * __ldcg(pp + 1);
    acc.x += w * x.x;
    acc.y += w * x.y;
    acc.z += w * x.z;
    acc.w += w * x.w;
  }
  reinterpret_cast<float4*>(accs[warp])[lane] = acc;
  __syncthreads();
  if (lane == 0) fred[warp] = l;
  __syncthreads();
  float o = 0.f, lt = 0.f;
#pragma unroll
  for (int w = 0; w < kCombThreads / 32; ++w) {
    o += accs[w][tid];
    lt += fred[w];
  }
  o = lt == 0.f ? 0.f : o / lt;
  if (a.bf16) {
    const __nv_bfloat16 v = __float2bfloat16_rn(o);
    op[tid] = *reinterpret_cast<const uint16_t*>(&v);
  } else {
    const __half v = __float2half_rn(o);
    op[tid] = *reinterpret_cast<const uint16_t*>(&v);
  }
}

template <int CODE, int NB>
cudaError_t launch_split(const ByteAttnArgs& a, int grid, cudaStream_t stream) {
  byte_split_kernel<CODE, NB><<<grid, kThreads, SplitSmem<NB>::kTotal, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t byte_partial_bytes(int n_sms) {
  return static_cast<size_t>(n_sms) * 2 * kByteMaxRows * kBytePartStride * sizeof(float);
}

cudaError_t byte_decode_setup() {
  cudaError_t e = set_smem(byte_split_kernel<0, 1>, SplitSmem<1>::kTotal);
  if (e == cudaSuccess) e = set_smem(byte_split_kernel<1, 1>, SplitSmem<1>::kTotal);
  if (e == cudaSuccess) e = set_smem(byte_split_kernel<0, 2>, SplitSmem<2>::kTotal);
  if (e == cudaSuccess) e = set_smem(byte_split_kernel<1, 2>, SplitSmem<2>::kTotal);
  return e;
}

cudaError_t launch_byte_attn(const ByteShape& s, ByteAttnArgs& a, cudaStream_t stream) {
  const int rows = s.group * a.n_q;
  const int nb = rows <= 8 ? 1 : 2;
  a.row_blocks = (rows + 8 * nb - 1) / (8 * nb);
  const int64_t units = static_cast<int64_t>(a.layer_count) * a.hkv * a.row_blocks;
  const int64_t comb = units * a.batch * 8 * nb;
  if (units > INT32_MAX || comb > INT32_MAX) return cudaErrorInvalidConfiguration;
  const int64_t most = (units * a.batch * s.ntiles + kWarps - 1) / kWarps;
  const int grid = static_cast<int>(most < s.n_sms ? most : s.n_sms);
  cudaError_t e;
  if (s.code == 0)
    e = nb == 1 ? launch_split<0, 1>(a, grid, stream) : launch_split<0, 2>(a, grid, stream);
  else
    e = nb == 1 ? launch_split<1, 1>(a, grid, stream) : launch_split<1, 2>(a, grid, stream);
  if (e != cudaSuccess) return e;
  return launch_dependent(byte_combine_kernel, dim3(static_cast<unsigned>(comb)), dim3(kCombThreads), 0, stream, a, grid,
                          8 * nb);
}

}  // namespace bgtq
