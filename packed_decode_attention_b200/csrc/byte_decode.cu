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
//
// Bound by HBM where there is enough to read: a ragged batch of 16 x 16K to 32K
// positions, 4 KV heads (429 MB) takes 83 us, 79 % of the copy rate, of which
// about 10 us are not the pass over the codes: a call with nothing to attend
// takes 2.4 to 3.3 us, the way to the first codes 4, the merge 2, the join 3.
// One layer of 8 KV heads at 32K takes 23.3 us (67 MB, 44 %): there those count.
//
// The products run on mma.sync, not tcgen05: its 128-row operand would be filled
// by 1 to 16 query rows or, with the codes as that operand, leave a row's
// scores across 128 lanes, and the pass is not bound by the products (8.6
// cycles of an SM quarter each, 32 for 32 positions, where HBM gives 360 cycles).
#include <cuda_bf16.h>

#include <cfloat>

#include "byte_cache.h"
#include "common.cuh"

namespace bgtq {

namespace {

constexpr int kStep = 32;                // positions a warp takes at once: half a block
constexpr int kStepBytes = kStep * 128;
constexpr int kByteWaitLimit = 1 << 20;  // polls of up to a microsecond each: about a second
constexpr float kPShift = 14.f;          // softmax weights are held as 2^14 p (see the weights' comment)
// Sums of p v are held as 2^-16 of them (2^14 in the weight, 2^-30 with V's
// scale): they overflow only where more than 2^16 positions share the weight
// of values near bf16's largest, and the least code of the least scale, 2^-109,
// stays a normal number.
constexpr float kVDown = 0x1p-30f, kVUp = 0x1p30f;
// A unit (one KV head's rows of one sequence) costs a CTA its queries and a
// merge besides its steps: about as long as this many steps.  Counted when
// the work is shared out, so that a CTA gets few short sequences.
constexpr int kUnitCost = 18;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What is added to a score before ex2: kPShift - m for the running maximum m
// (0 where nothing was seen: the scores are -inf), rounded down, so that the
// largest weight is at most 2^14.  To nearest it would be 2^16 and more, past
// fp16, for m of 2^25 to 2^28, where fp32 does not hold kPShift - m.
__device__ __forceinline__ float weight_shift(float m) {
  return m == -CUDART_INF_F ? 0.f : __fadd_rd(kPShift, -m);
}

// Products q . codes stay under 2^31 (128 of 2^15 by 448).  Their factor is cut
// to kMaxFactor and slopes to kMaxSlope (distances are at most 2^30), so that a
// score, in log2 units and with its bias, stays in fp32.  A product that is not
// 0 is at least 2^-33 (fp16's least times e4m3's), so what is cut is a score
// past 2^57, and it stays one: a softmax that steep takes its largest score
// whichever way.  (Cutting the scores themselves: 5 % slower for short sequences.)
constexpr float kMaxFactor = 0x1p90f;
constexpr float kMaxSlope = 0x1p96f;

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

// 32 x 128 codes into shared memory, 16-byte piece c of position p at piece
// c ^ (p & 7) (the map's 128-byte swizzle).
__device__ __forceinline__ void copy_step(uint32_t dst, const CUtensorMap* map, int32_t row, uint32_t bar) {
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

// ---- which steps a sequence's queries see -----------------------------------

struct SeqSteps {
  int32_t len;    // 0 where the given length is out of range
  int32_t pre;    // prefix positions, min(prefix, len)
  int32_t n_pre;  // steps 0 .. n_pre - 1 are seen for the prefix alone
  int32_t t0;     // then steps t0, t0 + 1, ...
  int32_t n;      // steps in all
  bool bad;
};

__device__ __forceinline__ int32_t query_lo(const ByteAttnArgs& a, int b, int i, int p) {
  int32_t lo = a.doc_start ? max(0, __ldg(a.doc_start + static_cast<int64_t>(b) * a.n_q + i)) : 0;
  if (a.window > 0) lo = max(lo, p - a.window + 1);
  return lo;
}

// Loads through L1: a CTA asks again for the sequences that it works on.
__device__ __forceinline__ SeqSteps seq_steps(const ByteAttnArgs& a, int b) {
  SeqSteps s;
  const int32_t len = __ldg(a.seq_lens + b);
  s.bad = len < 0 || len > a.capacity;
  s.len = s.bad ? 0 : len;
  s.pre = a.prefix ? min(max(0, __ldg(a.prefix + b)), s.len) : 0;
  int32_t lo = INT32_MAX;
  if (a.doc_start == nullptr && a.window <= 0) {
    if (s.len > 0) lo = 0;
  } else {
#pragma unroll 4
    for (int i = 0; i < a.n_q; ++i) {
      const int p = s.len - a.n_q + i;
      const int32_t l = query_lo(a, b, i, p);
      if (p >= 0 && l <= p) lo = min(lo, l);
    }
  }
  const int pre_steps = (s.pre + kStep - 1) / kStep;
  if (lo == INT32_MAX) {
    s.n_pre = s.n = pre_steps;
    s.t0 = 0;
  } else {
    s.t0 = lo / kStep;
    s.n_pre = min(pre_steps, s.t0);
    s.n = s.n_pre + (s.len - 1) / kStep - s.t0 + 1;
  }
  return s;
}

// The work is the steps of all units (layer, KV head, row block) of all
// sequences, in the order sequence, unit, step; each unit is preceded by
// `pad` places that stand for its own cost.  CTA c of `ctas` takes the places
// [c V / ctas, (c + 1) V / ctas) of V, whatever units they belong to, so
// ragged batches are shared evenly.
struct Sums {
  int64_t v, r;   // places, steps
  int32_t k;      // sequences that have any
};

__device__ __forceinline__ int unit_pad(const ByteAttnArgs& a) { return a.batch > 1 ? kUnitCost : 0; }
__device__ __forceinline__ int places(int n, int pad) { return n > 0 ? n + pad : 0; }

// Quotients whose operands hardly ever need 64 bits.
__device__ __forceinline__ int64_t quot(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// CTA c has places [begin(c), begin(c + 1)): equal shares, or, with per > 0,
// each unit's steps in `per` equal shares (one sequence: units alike).
struct Shares {
  int64_t each;
  int32_t rem, ctas, per, n;
  __device__ int64_t begin(int c) const {
    if (per > 0) {
      const int u = c / per;
      return static_cast<int64_t>(u) * n + static_cast<int>(quot(static_cast<int64_t>(c - u * per) * n, per));
    }
    return c * each + min(c, rem);
  }
  __device__ int of(int64_t g) const {
    if (per > 0) {
      const int u = static_cast<int>(quot(g, n));
      return u * per + static_cast<int>(quot((g - static_cast<int64_t>(u) * n + 1) * per - 1, n));
    }
    const int64_t head = rem * (each + 1);
    return static_cast<int>(g < head ? quot(g, each + 1) : rem + quot(g - head, each));
  }
};

// At most a CTA for each `warps` steps or for each unit, whichever are more:
// a unit's steps are spread over the warps of a CTA first.
__device__ __forceinline__ Shares shares(const Sums& s, int units, int grid, int warps) {
  const int64_t c = max(quot(units * s.r + warps - 1, warps), static_cast<int64_t>(units) * s.k);
  Shares r;
  r.ctas = static_cast<int>(min(c, static_cast<int64_t>(grid)));
  r.each = quot(units * s.v, r.ctas);
  r.rem = static_cast<int32_t>(units * s.v - r.each * r.ctas);
  r.per = 0;
  r.n = static_cast<int32_t>(s.r);
  if (s.v == s.r && units <= r.ctas) {
    // one sequence: no CTA has steps of two units where the larger shares
    // cost less than a second unit
    const int per = r.ctas / units;
    if (r.n <= per * (r.each + kUnitCost)) {
      r.per = per;
      r.ctas = per * units;
    }
  }
  return r;
}

// Sums over the NT threads; red: NT / 32 places.
template <int NT>
__device__ __forceinline__ Sums block_sum(Sums x, Sums* red) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    x.v += __shfl_xor_sync(0xffffffffu, x.v, o);
    x.r += __shfl_xor_sync(0xffffffffu, x.r, o);
    x.k += __shfl_xor_sync(0xffffffffu, x.k, o);
  }
  __syncthreads();
  if ((tid & 31) == 0) red[tid >> 5] = x;
  __syncthreads();
  Sums s{0, 0, 0};
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    s.v += red[w].v;
    s.r += red[w].r;
    s.k += red[w].k;
  }
  return s;
}

// ---- the split pass ------------------------------------------------------------

struct Cursor {
  int b, u, j;
  int base;       // the unit's first slot (its pool's, where paged)
  SeqSteps s;
};

struct Unit {
  int li, h, rb;  // layer of the call, KV head, row block
};

__device__ __forceinline__ Unit unit_of(const ByteAttnArgs& a, int u) {
  Unit r{0, u, 0};
  if (a.row_blocks > 1) {
    r.h = u / a.row_blocks;
    r.rb = u - r.h * a.row_blocks;
  }
  if (a.layer_count > 1) {
    r.li = r.h / a.hkv;
    r.h -= r.li * a.hkv;
  }
  return r;
}

// Slots are fewer than 2^25 (the codes' rows have int32 numbers).
__device__ __forceinline__ int base_of(const ByteAttnArgs& a, int b, int u) {
  const Unit x = unit_of(a, u);
  const int layer = a.layer0 + x.li;
  return a.n_pages == 0 ? ((layer * a.max_batch + b) * a.hkv + x.h) * static_cast<int>(a.ntiles)
                        : (layer * a.hkv + x.h) * a.n_pages;
}

// Moves k steps on; the caller knows that they exist.
__device__ __forceinline__ void advance(const ByteAttnArgs& a, Cursor& c, int units, int k) {
  c.j += k;
  if (c.j < c.s.n) return;
  do {
    c.j -= c.s.n;
    if (++c.u == units) {
      c.u = 0;
      do {
        if (++c.b >= a.batch) { c.b = a.batch - 1; c.j = 0; return; }
        c.s = seq_steps(a, c.b);
      } while (c.s.n == 0);
    }
  } while (c.j >= c.s.n);
  c.base = base_of(a, c.b, c.u);
}

__device__ __forceinline__ int tile_of(const SeqSteps& s, int j) { return j < s.n_pre ? j : s.t0 + j - s.n_pre; }

// The slot of a step's block.
__device__ __forceinline__ int slot_of(const ByteAttnArgs& a, const Cursor& c, int tile) {
  const int block = tile / (kByteBlock / kStep);
  if (a.n_pages == 0) return c.base + block;
  int32_t page = __ldg(a.block_table + static_cast<int64_t>(c.b) * a.ntiles + block);
  if (page < 0 || page >= a.n_pages) {
    if ((threadIdx.x & 31) == 0) atomicOr(a.err, kErrPage);
    page = 0;
  }
  return c.base + page;
}

// The end r1 of a CTA's places, in the sequence whose places start at v0 and
// whose steps start at number s0, n of them a unit: the number of the first
// step behind the end, and in how many CTAs the unit is that the end cuts
// (1: none).
__device__ __forceinline__ void tail_of(const Shares& sh, int64_t v0, int64_t s0, int64_t r1, int n, int pad, int64_t& end,
                                        int& tail) {
  const int np = places(n, pad);
  const int64_t u = quot(r1 - v0, np), at = v0 + u * np;
  end = s0 + u * n + max(static_cast<int64_t>(0), r1 - at - pad);
  tail = r1 > at + pad ? sh.of(at + np - 1) - static_cast<int>(blockIdx.x) + 1 : 1;
}

// The first step of a CTA, `off` places into its first sequence, and the
// number of its steps; `left`: from the sequence's first step to the CTA's end.
__device__ __forceinline__ void start_of(int64_t off, int64_t left, int pad, Cursor& seg, int& total) {
  const int np = places(seg.s.n, pad);
  seg.u = static_cast<int>(quot(off, np));
  seg.j = max(0, static_cast<int>(off - static_cast<int64_t>(seg.u) * np) - pad);
  total = static_cast<int>(left - static_cast<int64_t>(seg.u) * seg.s.n - seg.j);
}

// NB blocks of 8 query rows.  One: 12 warps of 168 registers; two, with twice
// the accumulators: 8 warps of 255 (12 of 168 spill: 39 us where these take 28.5).
// More than 16 rows take several passes.  (One block, the ragged batch: 16
// warps of 128 registers spill, 99 us; 8 of 221 in steps of 64 positions, 86; 12
// are 83.)  Two pairs of buffers a warp (a step's K and V) keep 192 or 128 KB an
// SM on their way, where 64 reach the read rate (three pairs for two blocks
// were 5 % slower).
template <int NB>
struct Split {
  static constexpr int kWarps = NB == 1 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRing = 2;                         // pairs of buffers
  static constexpr int kRows = 8 * NB;
  static constexpr int kQPitch = 136;                   // halves: rows 4 banks apart
  static constexpr int kUStride = 129;                  // merge: floats from a dimension pair to the next
  static constexpr int kMergeU = 4;                     // of the 8 pairs of a lane
  static constexpr int kMergeFloats = kMergeU * kUStride;
  // shared memory, from a 1024-byte boundary
  static constexpr int kMergeAt = kWarps * kRing * 2 * kStepBytes;
  static constexpr int kTotal = 1024 + kMergeAt + kWarps * kMergeFloats * 4;
};

struct Row {
  float back;     // undoes the query's scaling, times the scores' scale (at most 2^113 2^14)
  float slope;    // in log2 units
  int32_t lo, hi; // sees lo .. hi
  int32_t pre;    // and positions below
  int32_t tref;   // distances count from here
  int32_t out;    // its output's place among the sequence's
};

// The tensor cores take the codes as the 16-row operand (m16n8k16): positions
// for q . k, dimensions for p . v, the query rows as the 8 columns, so 8 rows
// waste nothing and a row block's second 8 rows reuse the widened codes.
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
template <int CODE, int NB>
__global__ __launch_bounds__(Split<NB>::kThreads, 1) void byte_split_kernel(const __grid_constant__ ByteAttnArgs a) {
  using C = Split<NB>;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads, kRing = C::kRing;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[kWarps * kRing];
  __shared__ __align__(16) uint16_t qs[C::kRows * C::kQPitch];
  __shared__ Row row_info[C::kRows];
  __shared__ float ms[kWarps * C::kRows], ls[kWarps * C::kRows], m_all[C::kRows], l_all[C::kRows];
  __shared__ Sums red[kWarps];
  __shared__ int tail_parts;
  __shared__ int64_t found[4];     // the first sequence, its first place, its first step's number; the end's step
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (tid < 2) asm volatile("prefetch.tensormap [%0];" ::"l"(&a.map[tid]) : "memory");
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  float* merge = reinterpret_cast<float*>(smem_raw + (smem0 - smem_u32(smem_raw)) + C::kMergeAt);
  const uint32_t ring = smem0 + warp * kRing * 2 * kStepBytes;
  const uint32_t bar0 = smem_u32(&bars[warp * kRing]);
  if (lane < kRing) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar0 + 8 * lane) : "memory");
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // this CTA's places [r0, r1), and the steps among them; and for the join, in
  // how many CTAs the unit is that the CTA ends in
  const int units = a.layer_count * a.hkv * a.row_blocks, pad = unit_pad(a);
  Cursor seg;      // the start of the segment (a unit's steps in this CTA)
  int mine_total;
  if (a.batch == 1) {
    seg.b = 0;
    seg.s = seq_steps(a, 0);
    const int n = seg.s.n;
    if (seg.s.bad && blockIdx.x == 0 && tid == 0) atomicOr(a.err, kErrSeqLen);
    if (n == 0) return;
    const Shares sh = shares(Sums{n, n, 1}, units, gridDim.x, kWarps);
    if (static_cast<int>(blockIdx.x) >= sh.ctas) return;
    const int64_t r0 = sh.begin(blockIdx.x), r1 = sh.begin(blockIdx.x + 1);
    seg.u = static_cast<int>(quot(r0, n));
    seg.j = static_cast<int>(r0 - static_cast<int64_t>(seg.u) * n);
    mine_total = static_cast<int>(r1 - r0);
    if (tid == 0) tail_parts = sh.per > 0 ? sh.per : sh.of((quot(r1 - 1, n) + 1) * n - 1) - static_cast<int>(blockIdx.x) + 1;
  } else if (a.batch <= 32) {
    // a lane a sequence, every warp for itself; sums of 32 fit an int32 (a
    // sequence has fewer than 2^26 places)
    SeqSteps s{};
    if (lane < a.batch) s = seq_steps(a, lane);
    if (s.bad && blockIdx.x == 0 && warp == 0) atomicOr(a.err, kErrSeqLen);
    const int np = places(s.n, pad);
    int iv = np, ir = s.n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, iv, o), z = __shfl_up_sync(0xffffffffu, ir, o);
      if (lane >= o) {
        iv += y;
        ir += z;
      }
    }
    const Sums sum{__shfl_sync(0xffffffffu, iv, a.batch - 1), __shfl_sync(0xffffffffu, ir, a.batch - 1),
                   __popc(__ballot_sync(0xffffffffu, s.n > 0))};
    if (sum.r == 0) return;
    const Shares sh = shares(sum, units, gridDim.x, kWarps);
    if (static_cast<int>(blockIdx.x) >= sh.ctas) return;
    const int64_t r0 = sh.begin(blockIdx.x), r1 = sh.begin(blockIdx.x + 1);
    const int64_t v0 = static_cast<int64_t>(iv - np) * units, v1 = static_cast<int64_t>(iv) * units;
    const int64_t s0 = static_cast<int64_t>(ir - s.n) * units;
    int64_t end = units * sum.r;
    int tail = 1;
    const int last = __ffs(__ballot_sync(0xffffffffu, v0 <= r1 && r1 < v1)) - 1;
    if (lane == last) tail_of(sh, v0, s0, r1, s.n, pad, end, tail);
    if (last >= 0) {
      end = __shfl_sync(0xffffffffu, end, last);
      tail = __shfl_sync(0xffffffffu, tail, last);
    }
    if (tid == 0) tail_parts = tail;
    seg.b = __ffs(__ballot_sync(0xffffffffu, v0 <= r0 && r0 < v1)) - 1;
    seg.s.len = __shfl_sync(0xffffffffu, s.len, seg.b);
    seg.s.pre = __shfl_sync(0xffffffffu, s.pre, seg.b);
    seg.s.n_pre = __shfl_sync(0xffffffffu, s.n_pre, seg.b);
    seg.s.t0 = __shfl_sync(0xffffffffu, s.t0, seg.b);
    seg.s.n = __shfl_sync(0xffffffffu, s.n, seg.b);
    start_of(r0 - __shfl_sync(0xffffffffu, v0, seg.b), end - __shfl_sync(0xffffffffu, s0, seg.b), pad, seg, mine_total);
  } else {
    int n0 = 0;
    Sums sum{0, 0, 0};
    for (int b = tid; b < a.batch; b += kThreads) {
      const SeqSteps s = seq_steps(a, b);
      const int n = s.n;
      if (b == tid) n0 = n;
      if (s.bad && blockIdx.x == 0) atomicOr(a.err, kErrSeqLen);
      sum.v += places(n, pad);
      sum.r += n;
      sum.k += n > 0;
    }
    sum = block_sum<kThreads>(sum, red);
    if (sum.r == 0) return;
    const Shares sh = shares(sum, units, gridDim.x, kWarps);
    if (static_cast<int>(blockIdx.x) >= sh.ctas) return;
    const int64_t r0 = sh.begin(blockIdx.x), r1 = sh.begin(blockIdx.x + 1);
    Sums before{0, 0, 0};  // of the sequences before this chunk
    if (tid == 0) {
      found[3] = units * sum.r;
      tail_parts = 1;
    }
    for (int base = 0; base < a.batch; base += kThreads) {
      const int b = base + tid;
      const int n = b < a.batch ? (base == 0 ? n0 : seq_steps(a, b).n) : 0, np = places(n, pad);
      int iv = np, ir = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, iv, o), z = __shfl_up_sync(0xffffffffu, ir, o);
        if (lane >= o) {
          iv += y;
          ir += z;
        }
      }
      __syncthreads();
      if (lane == 31) red[warp] = Sums{iv, ir, 0};
      __syncthreads();
      Sums incl{before.v + iv, before.r + ir, 0};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
          incl.v += red[w].v;
          incl.r += red[w].r;
        }
        before.v += red[w].v;
        before.r += red[w].r;
      }
      const int64_t v0 = (incl.v - np) * units, v1 = incl.v * units, s0 = (incl.r - n) * units;
      if (v0 <= r0 && r0 < v1) {
        found[0] = b;
        found[1] = v0;
        found[2] = s0;
      }
      if (v0 <= r1 && r1 < v1) {
        int64_t end;
        int tail;
        tail_of(sh, v0, s0, r1, n, pad, end, tail);
        found[3] = end;
        tail_parts = tail;
      }
      if (before.v * units > r1) break;
    }
    __syncthreads();
    seg.b = static_cast<int>(found[0]);
    seg.s = seq_steps(a, seg.b);
    start_of(r0 - found[1], found[3] - found[2], pad, seg, mine_total);
  }
  if (mine_total <= 0) return;
  seg.base = base_of(a, seg.b, seg.u);

  // this warp's steps: warp, warp + kWarps, ... of the CTA's, kRing of them on
  // their way
  const int nt = mine_total > warp ? (mine_total - warp + kWarps - 1) / kWarps : 0;
  Cursor cur = seg;
  int issued = 0, ibuf = 0;
  float ks[kRing], vs[kRing];   // the blocks' scales, the oldest step's first
  uint32_t pending = 0;         // bit i: copies into pair i are on their way
  auto issue = [&](float& k, float& v) {
    if (issued >= nt) return;
    advance(a, cur, units, issued == 0 ? warp : kWarps);
    const int tile = tile_of(cur.s, cur.j), slot = slot_of(a, cur, tile);
    k = __ldg(a.scales[0] + slot);
    v = __ldg(a.scales[1] + slot);
    if (tile / (kByteBlock / kStep) != a.drop_tile) {
      pending |= 1u << ibuf;
      if (lane == 0) {
        const uint32_t bar = bar0 + 8 * ibuf, dst = ring + ibuf * 2 * kStepBytes;
        const int32_t row = slot * kByteBlock + tile % (kByteBlock / kStep) * kStep;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "n"(2 * kStepBytes) : "memory");
        copy_step(dst, &a.map[0], row, bar);
        copy_step(dst + kStepBytes, &a.map[1], row, bar);
      }
    }
    ++issued;
    ibuf = ibuf == kRing - 1 ? 0 : ibuf + 1;
  };
#pragma unroll
  for (int i = 0; i < kRing; ++i) {
    ks[i] = vs[i] = 0.f;
    issue(ks[i], vs[i]);
  }
  int it = 0;              // the warp's next step
  int buf = 0;             // its pair
  uint32_t phases = 0;     // bit i: parity of pair i's next completion
  bool dead = false;
  int f0 = 0;              // steps of the CTA before this segment
  const int pig = (g >> 1) | ((g & 1) << 2);
  const int rows = a.group * a.n_q;

  // A segment's queries, half a warp a row: asked for before the merge of the
  // segment before it, everything a row needs at once.
  struct Asked {
    uint4 q;
    float slope;
    int32_t lo, p, out;
    bool real;
  };
  auto ask = [&](const Cursor& c) {
    Asked r{make_uint4(0u, 0u, 0u, 0u), 0.f, 1, 0, 0, false};
    if (warp < C::kRows / 2) {
      const Unit un = unit_of(a, c.u);
      const int row = un.rb * C::kRows + 2 * warp + (lane >> 4), i = row / a.group, hg = row - i * a.group;
      r.real = row < rows;
      r.p = c.s.len - a.n_q + i;
      r.out = (i * a.hq + un.h * a.group + hg) * 128;
      if (r.real) {
        r.q = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                   (static_cast<int64_t>(un.li) * a.batch + c.b) * a.n_q * a.hq * 128 +
                                                   r.out + 8 * (lane & 15)));
        if (a.slopes) r.slope = __ldg(a.slopes + un.h * a.group + hg);
        r.lo = query_lo(a, c.b, i, r.p);
      }
    }
    return r;
  };
  Asked asked = ask(seg);

  while (f0 < mine_total) {
    const int len_seg = min(seg.s.n - seg.j, mine_total - f0);
    const int pre = seg.s.pre;

    // q as the products' 8-column operand, scaled by a power of two a row so
    // that its largest element lies in [2^14, 2^15): fp16 and bf16 queries
    // are then both exact in fp16 but for elements under 2^-29 of the
    // largest
    if (warp < C::kRows / 2) {
      const int rl = 2 * warp + (lane >> 4);
      const uint4 w = asked.q;
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      float2 x[4];
      float big = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = a.bf16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[e]))
                      : __half22float2(*reinterpret_cast<const __half2*>(&u[e]));
        big = fmaxf(big, fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      // 2^up m in [2^14, 2^15); zero and non-finite rows as they are
      const int ex = static_cast<int>(__float_as_uint(big) >> 23);
      const int up = ex == 0 || ex >= 255 ? 0 : max(-113, min(113, 141 - ex));
      const float fac = __int_as_float((up + 127) << 23);
      *reinterpret_cast<uint4*>(qs + rl * C::kQPitch + 8 * (lane & 15)) =
          make_uint4(pack_half2(x[0].x * fac, x[0].y * fac), pack_half2(x[1].x * fac, x[1].y * fac),
                     pack_half2(x[2].x * fac, x[2].y * fac), pack_half2(x[3].x * fac, x[3].y * fac));
      if ((lane & 15) == 0) {
        Row r{0.f, 0.f, 1, 0, 0, 0, -1};
        if (asked.real) {
          r.back = __int_as_float((127 - up) << 23) * a.scale;
          r.lo = asked.lo;
          r.hi = asked.p;
          r.pre = pre;
          r.slope = fminf(fmaxf(asked.slope * kLog2e, -kMaxSlope), kMaxSlope);
          // distances count from the row's last visible position, or with a
          // negative slope its first: its weights do not change, and the
          // positions that the bias favours keep theirs exact
          if (asked.slope < 0.f)
            r.tref = pre > 0 ? 0 : asked.lo;
          else
            r.tref = max(asked.lo <= asked.p ? asked.p : -1, pre - 1);
          r.out = asked.out;
        }
        row_info[rl] = r;
      }
    }
    __syncthreads();
    float colf[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      colf[nb][0] = row_info[nb * 8 + 2 * t].back;
      colf[nb][1] = row_info[nb * 8 + 2 * t + 1].back;
    }
    const bool real = lane < C::kRows && row_info[lane % C::kRows].out >= 0;
    const int lo_max = __reduce_max_sync(0xffffffffu, real ? row_info[lane].lo : 0);
    const int hi_min = __reduce_min_sync(0xffffffffu, real ? row_info[lane].hi : INT32_MAX);

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

#pragma unroll 1
    for (; it < nt && warp + kWarps * it < f0 + len_seg; ++it) {
      const int p0 = kStep * tile_of(seg.s, seg.j + warp + kWarps * it - f0);
      if (!dead) {
        if (__all_sync(0xffffffffu, bar_wait(bar0 + 8 * buf, phases >> buf & 1))) {
          phases ^= 1u << buf;
          pending &= ~(1u << buf);
        } else {
          // copies on their way land (bounded) before their places are used otherwise
          dead = true;
          for (int i = 0; i < kRing; ++i)
            if (pending >> i & 1) bar_wait(bar0 + 8 * i, phases >> i & 1);
        }
      }
      if (!dead) {
        float S[NB][2][4];
        const uint32_t kb = ring + buf * 2 * kStepBytes + pig * 128, vb = ring + buf * 2 * kStepBytes + kStepBytes;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t piece = ((t + 4 * i) ^ pig) * 16;
          uint32_t qf[NB][8];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint32_t qa = smem_u32(qs) + ((nb * 8 + g) * C::kQPitch + 64 * i + 16 * t) * 2;
            const uint4 x = lds128(qa), y = lds128(qa + 16);
            qf[nb][0] = x.x, qf[nb][1] = x.y, qf[nb][2] = x.z, qf[nb][3] = x.w;
            qf[nb][4] = y.x, qf[nb][5] = y.y, qf[nb][6] = y.z, qf[nb][7] = y.w;
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
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
                  mma16816(S[nb][mt], a0, a1, a2, a3, qf[nb][2 * w], qf[nb][2 * w + 1]);
              }
            }
          }
        }
        uint32_t pf[NB][2][2];
        uint32_t seen = 0;     // bit i: some row sees position 8 i + pig of a step that is not full
        const bool full = (p0 >= lo_max && p0 + kStep - 1 <= hi_min) || p0 + kStep <= pre;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          // scores in log2 units
          const float f0c = fminf(colf[nb][0] * ks[0], kMaxFactor), f1c = fminf(colf[nb][1] * ks[0], kMaxFactor);
          if (a.cap > 0.f) {
            const float ic = 1.f / a.cap, oc = a.cap * kLog2e;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
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
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) S[nb][mt][e] *= ((e & 1) ? f1c : f0c) * kLog2e;
          }
          if (a.slopes) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float sl = row_info[nb * 8 + 2 * t + c].slope;
              const int d0 = p0 + pig - row_info[nb * 8 + 2 * t + c].tref;
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int e = c; e < 4; e += 2) S[nb][mt][e] += sl * static_cast<float>(d0 + 16 * mt + 8 * (e >> 1));
            }
          }
          if (!full) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const Row r = row_info[nb * 8 + 2 * t + c];
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int e = c; e < 4; e += 2) {
                  const int p = p0 + 16 * mt + 8 * (e >> 1) + pig;
                  if (p < r.pre || (p >= r.lo && p <= r.hi))
                    seen |= 1u << (2 * mt + (e >> 1));
                  else
                    S[nb][mt][e] = -CUDART_INF_F;
                }
            }
            // positions that no row sees (behind the sequence, before a
            // document or the window) may never have been written, and a NaN
            // code times a zero weight is NaN: their V rows are cleared
            if (CODE == 0 && nb == NB - 1) {
              seen |= __shfl_xor_sync(0xffffffffu, seen, 1);
              seen |= __shfl_xor_sync(0xffffffffu, seen, 2);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (!(seen >> i & 1)) {
                  const uint32_t at = vb + (8 * i + pig) * 128 + t * 32;
                  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + 16), "r"(0) : "memory");
                }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
            }
          }
          float mx[2] = {m[nb][0], m[nb][1]};
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e & 1] = fmaxf(mx[e & 1], S[nb][mt][e]);
          // past the first steps a new maximum is rare: only then do the lanes
          // agree on it
          if (__any_sync(0xffffffffu, mx[0] != m[nb][0] || mx[1] != m[nb][1])) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
              mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
            }
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
          const float s0 = weight_shift(m[nb][0]), s1 = weight_shift(m[nb][1]);
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t w = pack_half2(ex2(S[nb][mt][2 * e] + s0), ex2(S[nb][mt][2 * e + 1] + s1));
              pf[nb][mt][e] = transpose8x8(w);
              // the sum is that of the rounded weights; a lane's own positions until the merge
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
              l[nb][0] += f.x;
              l[nb][1] += f.y;
            }
        }
        // a block that no row sees any of may have any scale, and 0 times it is to be 0
        vs[0] = fminf(fmaxf(vs[0], 0.f), FLT_MAX) * kVDown;
        // 4 of the 8 M-tiles (dimension pairs) at a time: half of each 16-byte piece
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float T[NB][4][4];
          const uint32_t at0 = vb + t * 128 + ((pig ^ t) * 16) + half * 8;
          const uint32_t at1 = vb + t * 128 + ((pig ^ t ^ 4) * 16) + half * 8;
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
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
              for (int e = 0; e < 4; ++e) acc[nb][4 * half + u][e] = fmaf(T[nb][u][e], vs[0], acc[nb][4 * half + u][e]);
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i + 1 < kRing; ++i) {
        ks[i] = ks[i + 1];
        vs[i] = vs[i + 1];
      }
      if (!dead) issue(ks[kRing - 1], vs[kRing - 1]);  // the pair is free
      buf = buf == kRing - 1 ? 0 : buf + 1;
    }

    const bool whole = seg.j == 0 && len_seg == seg.s.n;
    // place 0: the segment that opens this CTA's range; 1: a later one
    const int place = 2 * blockIdx.x + (f0 > 0);
    if (seg.j == 0 && tid == 0)
      a.parts[static_cast<int64_t>(seg.b) * units + seg.u] = make_int2(place, whole ? 1 : tail_parts);
    uint16_t* const out = static_cast<uint16_t*>(a.out) +
                          (static_cast<int64_t>(unit_of(a, seg.u).li) * a.batch + seg.b) * a.n_q * a.hq * 128;
    f0 += len_seg;
    const bool more = f0 < mine_total;
    if (more) {
      advance(a, seg, units, len_seg);
      asked = ask(seg);
    }

    // merge of the warps: their maxima and sums, then the accumulators
    // through shared memory, half a row block at a time, a thread summing its
    // elements over the warps in order
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nb][c] += __shfl_xor_sync(0xffffffffu, l[nb][c], o);
        if (g == 0) {
          ms[warp * C::kRows + nb * 8 + 2 * t + c] = m[nb][c];
          ls[warp * C::kRows + nb * 8 + 2 * t + c] = l[nb][c];
        }
      }
    __syncthreads();
    {
      const int rl = lane % C::kRows;
      float mw[kWarps], mx = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mw[w] = ms[w * C::kRows + rl];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, mw[w]);
      const float own = ms[warp * C::kRows + rl], f = own == mx ? 1.f : ex2(own - mx);
      if (warp == 0 && lane < C::kRows) {
        float sum_l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum_l += ls[w * C::kRows + rl] * (mw[w] == mx ? 1.f : ex2(mw[w] - mx));
        m_all[rl] = mx;
        l_all[rl] = !whole ? sum_l : sum_l == 0.f ? 0.f : kVUp / sum_l;
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float al[2] = {__shfl_sync(0xffffffffu, f, nb * 8 + 2 * t), __shfl_sync(0xffffffffu, f, nb * 8 + 2 * t + 1)};
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nb][u][e] *= al[e & 1];
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int u0 = 0; u0 < 8; u0 += C::kMergeU) {
        if (nb + u0 > 0) __syncthreads();
#pragma unroll
        for (int u = 0; u < C::kMergeU; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            merge[warp * C::kMergeFloats + u * C::kUStride + e * 32 + lane] = acc[nb][u0 + u][e];
        __syncthreads();
        // element i: row, 16-dimension piece and place in the piece's part
        constexpr int kDims = 2 * C::kMergeU;
#pragma unroll
        for (int i = tid; i < 64 * kDims; i += kThreads) {
          const int r = i / (8 * kDims), piece = i / kDims % 8, d = i % kDims, rl = nb * 8 + r;
          const int row_out = row_info[rl].out;
          if (row_out < 0) continue;
          const int gg = (piece & 3) << 1 | piece >> 2;
          const float* at = merge + (d >> 1) * C::kUStride + ((r & 1) + 2 * (d & 1)) * 32 + 4 * gg + (r >> 1);
          float x = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) x += at[w * C::kMergeFloats];
          const int dim = 16 * piece + 2 * u0 + d;
          if (whole) {
            x *= l_all[rl];
            if (a.bf16) {
              const __nv_bfloat16 v = __float2bfloat16_rn(x);
              out[row_out + dim] = *reinterpret_cast<const uint16_t*>(&v);
            } else {
              out[row_out + dim] = __half_as_ushort(__float2half_rn(x));
            }
          } else {
            float* pp = a.partials + (static_cast<int64_t>(place) * kByteMaxRows + rl) * kBytePartStride;
            pp[4 + dim] = x;
            if (dim == 0) *reinterpret_cast<float2*>(pp) = make_float2(m_all[rl], l_all[rl]);
          }
        }
      }
    if (!more) break;
    __syncthreads();  // row_info and the sums are the next segment's now
  }
  if (dead && lane == 0) atomicOr(a.err, kErrTimeout);
}

// ---- the join ------------------------------------------------------------------

constexpr int kCombAhead = 6;       // parts a warp has on their way at once

__device__ __forceinline__ void store2(const ByteAttnArgs& a, uint16_t* p, float x, float y) {
  uint32_t w;
  if (a.bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    w = *reinterpret_cast<const uint32_t*>(&v);
  } else {
    w = pack_half2(x, y);
  }
  *reinterpret_cast<uint32_t*>(p) = w;
}

// The parts of units that more than one CTA attended, joined by their maxima
// and sums in the order of the CTAs; rows that see nothing become 0.  WARPS
// warps share a row's parts (1: units are in few parts, and a CTA's 8 warps
// take 8 rows; 16: a CTA a row).
template <int WARPS>
__global__ __launch_bounds__(WARPS == 1 ? 256 : 32 * WARPS) void byte_combine_kernel(const __grid_constant__ ByteAttnArgs a,
                                                                                      int rows_per_unit) {
  constexpr int kRowsCta = WARPS == 1 ? 8 : 1;
  __shared__ float accs[WARPS][128];
  __shared__ float2 ml[WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int units = a.layer_count * a.hkv * a.row_blocks;
  int id = blockIdx.x;
  const int row_ctas = rows_per_unit / kRowsCta;
  const int rl = id % row_ctas * kRowsCta + (WARPS == 1 ? warp : 0), slice = WARPS == 1 ? 0 : warp;
  id /= row_ctas;
  const int u = id % units, b = id / units;
  const Unit un = unit_of(a, u);
  const int row = un.rb * rows_per_unit + rl;
  const int i = row / a.group, hg = row - i * a.group;
  uint16_t* op = static_cast<uint16_t*>(a.out) +
                 (((static_cast<int64_t>(un.li) * a.batch + b) * a.n_q + i) * a.hq + un.h * a.group + hg) * 128 + 4 * lane;
  const bool work = row < a.group * a.n_q;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // where the unit's first part lies, and how many there are
  const int2 where = __ldcg(a.parts + static_cast<int64_t>(b) * units + u);
  const int parts = seq_steps(a, b).n == 0 ? 0 : where.y;
  if (parts == 0 && work && slice == 0) *reinterpret_cast<uint2*>(op) = make_uint2(0u, 0u);
  if (parts <= 1 || (WARPS > 1 && !work)) return;
  // a warp's parts: slice, slice + WARPS, ..., with the running maximum
  // (part k > 0 opens its CTA's range)
  constexpr int64_t kPart = 2 * kByteMaxRows * kBytePartStride;
  const float* const part0 = a.partials + (where.x >> 1) * kPart + rl * kBytePartStride;
  float m = -CUDART_INF_F, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (work) {
#pragma unroll 1
    for (int k0 = slice; k0 < parts; k0 += kCombAhead * WARPS) {
      float4 x[kCombAhead];
      float2 s[kCombAhead];
#pragma unroll
      for (int j = 0; j < kCombAhead; ++j) {
        const int k = k0 + j * WARPS;
        s[j] = make_float2(-CUDART_INF_F, 0.f);
        x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < parts) {
          const float* p = part0 + k * kPart + (k == 0 ? (where.x & 1) * kByteMaxRows * kBytePartStride : 0);
          s[j] = __ldcg(reinterpret_cast<const float2*>(p));
          x[j] = __ldcg(reinterpret_cast<const float4*>(p + 4) + lane);
        }
      }
      float mx = m;
#pragma unroll
      for (int j = 0; j < kCombAhead; ++j) mx = fmaxf(mx, s[j].x);
      const float w0 = m == mx ? 1.f : ex2(m - mx);
      l *= w0;
      acc = make_float4(acc.x * w0, acc.y * w0, acc.z * w0, acc.w * w0);
#pragma unroll
      for (int j = 0; j < kCombAhead; ++j) {
        const float w = s[j].x == mx ? 1.f : ex2(s[j].x - mx);
        l = fmaf(w, s[j].y, l);
        acc = make_float4(fmaf(w, x[j].x, acc.x), fmaf(w, x[j].y, acc.y), fmaf(w, x[j].z, acc.z), fmaf(w, x[j].w, acc.w));
      }
      m = mx;
    }
  }
  if constexpr (WARPS == 1) {
    if (!work) return;
    const float inv = l == 0.f ? 0.f : kVUp / l;
    store2(a, op, acc.x * inv, acc.y * inv);
    store2(a, op + 2, acc.z * inv, acc.w * inv);
  } else {
    reinterpret_cast<float4*>(accs[warp])[lane] = acc;
    if (lane == 0) ml[warp] = make_float2(m, l);
    __syncthreads();
    if (tid >= 128) return;
    float mx = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, ml[w].x);
    float o = 0.f, lt = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = ml[w].x == mx ? 1.f : ex2(ml[w].x - mx);
      o = fmaf(f, accs[w][tid], o);
      lt = fmaf(f, ml[w].y, lt);
    }
    o = lt == 0.f ? 0.f : o / lt * kVUp;
    op += tid - 4 * lane;
    if (a.bf16) {
      const __nv_bfloat16 v = __float2bfloat16_rn(o);
      *op = *reinterpret_cast<const uint16_t*>(&v);
    } else {
      *op = __half_as_ushort(__float2half_rn(o));
    }
  }
}

template <int CODE, int NB>
cudaError_t launch_split(const ByteAttnArgs& a, int grid, cudaStream_t stream) {
  byte_split_kernel<CODE, NB><<<grid, Split<NB>::kThreads, Split<NB>::kTotal, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t byte_parts_bytes(int n_layers, int n_kv_heads, int group, int max_batch, int max_q_tokens) {
  return static_cast<size_t>(n_layers) * n_kv_heads * ((group * max_q_tokens + 7) / 8) * max_batch * sizeof(int2);
}

size_t byte_partial_bytes(int n_sms) {
  return static_cast<size_t>(n_sms) * 2 * kByteMaxRows * kBytePartStride * sizeof(float);
}

cudaError_t byte_decode_setup() {
  cudaError_t e = set_smem(byte_split_kernel<0, 1>, Split<1>::kTotal);
  if (e == cudaSuccess) e = set_smem(byte_split_kernel<1, 1>, Split<1>::kTotal);
  if (e == cudaSuccess) e = set_smem(byte_split_kernel<0, 2>, Split<2>::kTotal);
  if (e == cudaSuccess) e = set_smem(byte_split_kernel<1, 2>, Split<2>::kTotal);
  return e;
}

cudaError_t launch_byte_attn(const ByteShape& s, ByteAttnArgs& a, cudaStream_t stream) {
  const int rows = s.group * a.n_q;
  const int nb = rows <= 8 ? 1 : 2;
  a.row_blocks = (rows + 8 * nb - 1) / (8 * nb);
  const int64_t units = static_cast<int64_t>(a.layer_count) * a.hkv * a.row_blocks;
  const int64_t comb = units * a.batch * 8 * nb;
  if (units > INT32_MAX || comb > INT32_MAX) return cudaErrorInvalidConfiguration;
  // a CTA for each `warps` steps or for each unit (shares())
  const int warps = nb == 1 ? Split<1>::kWarps : Split<2>::kWarps;
  const int64_t steps = (s.ntiles * (kByteBlock / kStep) + warps - 1) / warps;
  const int64_t most = units * a.batch * steps;
  const int grid = static_cast<int>(most < s.n_sms ? most : s.n_sms);
  cudaError_t e;
  if (s.code == 0)
    e = nb == 1 ? launch_split<0, 1>(a, grid, stream) : launch_split<0, 2>(a, grid, stream);
  else
    e = nb == 1 ? launch_split<1, 1>(a, grid, stream) : launch_split<1, 2>(a, grid, stream);
  if (e != cudaSuccess) return e;
  // few units: many parts each, a CTA a row; else a warp a row
  if (units * a.batch * 8 <= grid)
    return launch_dependent(byte_combine_kernel<16>, dim3(static_cast<unsigned>(comb)), dim3(512), 0, stream, a, 8 * nb);
  return launch_dependent(byte_combine_kernel<1>, dim3(static_cast<unsigned>(comb / 8)), dim3(256), 0, stream, a, 8 * nb);
}

}  // namespace bgtq
