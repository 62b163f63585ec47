// Pages of a paged cache, packed or 8-bit: copying, forking, resizing and
// compacting.
//
// A page id names the same page of every layer and KV head; refs[p] counts
// who holds page p (rows of the block table and other owners), 0: free.
//
//   plan kernels  one CTA, or for large pools a cluster of 8, turns parents,
//                 lengths and counts into a new table, new counts and a list
//                 of page pairs
//   copy kernel   moves the pairs' bytes, for every layer and head
//
// The plans touch a few words a table entry and are bound by latency: each
// step between two cluster barriers is a few trips to L2.  The copy is bound
// by HBM: every byte of a copied page is read once and written once (256 MB
// each way in 78 us, the copy rate).
#include "common.cuh"
#include "pages.h"

namespace bgtq {

namespace {

constexpr int kPlanCtas = 8;          // the largest portable cluster
constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanAll = kPlanCtas * kPlanThreads;
constexpr int kPlanChunk = 128;       // table entries a warp takes at once
constexpr uint32_t kErrPool = 64;

// All CTAs of the plan's cluster, with their global writes.
__device__ __forceinline__ void plan_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ int pages_for(int len) { return len / kTile + (len % kTile != 0); }

// Exclusive sum of x over the CTA's NT threads, and the total.
template <int NT = kPlanThreads, typename T>
__device__ __forceinline__ T plan_scan(T x, T* red, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) red[warp] = incl;
  __syncthreads();
  T sums = lane < NT / 32 ? red[lane] : T(0);
#pragma unroll
  for (int o = 1; o < NT / 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += y;
  }
  total = __shfl_sync(0xffffffffu, sums, NT / 32 - 1);
  const T before = __shfl_sync(0xffffffffu, sums, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : T(0)) + incl - x;
}

// Calls f(p, k) for each page p of [lo, hi) with pred(p), k its rank among
// them plus base, in ascending order, until `most` are found; returns base
// plus their number.
template <int NT = kPlanThreads, typename P, typename F>
__device__ __forceinline__ int plan_select(int lo, int hi, int base, int* red, P pred, F f, int most = INT32_MAX) {
  for (int64_t c = lo; c < hi && base < most; c += 4 * NT) {
    const int64_t p = c + 4 * threadIdx.x;
    bool in[4];
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      in[i] = p + i < hi && pred(static_cast<int>(p + i));
      n += in[i];
    }
    int total;
    int k = base + plan_scan<NT>(n, red, total);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (in[i]) f(static_cast<int>(p + i), k++);
    base += total;
  }
  return base;
}

__device__ __forceinline__ int plan_count(int lo, int hi, int* red, const int32_t* refs, bool live) {
  int n = 0;
  for (int64_t p = lo + threadIdx.x; p < hi; p += kPlanThreads) {
    const int r = __ldcg(refs + p);
    n += live ? r > 0 : r == 0;
  }
  int total;
  plan_scan(n, red, total);
  return total;
}

__device__ __forceinline__ int checked_len(const PagePlanArgs& a, int len) {
  if (len >= 0 && len <= a.capacity) return len;
  atomicOr(a.err, kErrSeqLen);
  return 0;
}

__device__ __forceinline__ bool page_ok(const PagePlanArgs& a, int id) {
  if (id >= 0 && id < a.n_pages) return true;
  atomicOr(a.err, kErrPage);
  return false;
}

// fork:   row b becomes row parent[b]; the last page, where the row fills it
//         partly, is shared by nobody afterwards
// resize: rows give back pages or get new ones; a partly filled page that a
//         growing row shares is copied for it
// Both end the same way: rows that need pages get the free ones in ascending
// order of the pages, in the order of the rows.
template <int OP>
__global__ __launch_bounds__(kPlanThreads, 1) void plan_kernel(const __grid_constant__ PagePlanArgs a) {
  __shared__ int red[kPlanWarps];
  __shared__ int64_t wide[kPlanWarps];
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = blockIdx.x, gid = rank * kPlanThreads + tid, gwarp = gid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // the rows' new lengths, and the partly filled page each would write
  if (a.refs_out != a.refs)
    for (int p = gid; p < a.n_pages; p += kPlanAll) a.refs_out[p] = __ldg(a.refs + p);
  for (int b = gid; b < a.batch; b += kPlanAll) {
    int row = b, len, part;
    if constexpr (OP == kPageFork) {
      row = __ldg(a.parent + b);
      if (row < -1 || row >= a.batch) {
        atomicOr(a.err, kErrArg);
        row = -1;
      }
      len = row < 0 ? 0 : checked_len(a, a.lens[row]);
      if (row != b) checked_len(a, a.lens[b]);  // for its flag
      part = len;
    } else {
      part = checked_len(a, a.lens[b]);
      len = __ldg(a.new_lens + b);
      if (len < 0 || len > a.capacity) {
        atomicOr(a.err, kErrSeqLen);
        len = part;
      }
      if (len <= part) part = 0;  // nothing will be written behind it
    }
    int page = -1;
    if (part % kTile != 0) {
      page = a.table[row * a.ntiles + part / kTile];
      if (!page_ok(a, page)) page = -1;
    }
    a.ws.page[b] = page;
    a.ws.len[b] = len;
  }
  plan_sync();

  // who holds what now
  const int64_t chunks = (a.ntiles + kPlanChunk - 1) / kPlanChunk;
  for (int64_t it = gwarp; it < a.batch * chunks; it += kPlanAll / 32) {
    const int b = static_cast<int>(it / chunks);
    const int64_t t0 = (it - b * chunks) * kPlanChunk;
    const int have = a.lens[b] >= 0 && a.lens[b] <= a.capacity ? pages_for(a.lens[b]) : 0;
    const int want = pages_for(__ldcg(a.ws.len + b));
    int row = b;
    if constexpr (OP == kPageFork) {
      row = __ldg(a.parent + b);
      if (row < -1 || row >= a.batch) row = -1;
    }
#pragma unroll
    for (int i = 0; i < kPlanChunk / 32; ++i) {
      const int64_t t = t0 + 32 * i + lane;
      if constexpr (OP == kPageFork) {
        if (t < want) {
          const int id = __ldg(a.table + row * a.ntiles + t);
          a.table_out[b * a.ntiles + t] = id;
          if (page_ok(a, id) && row != b) atomicAdd(a.refs_out + id, 1);
        }
        if (t < have && row != b) {
          const int id = __ldg(a.table + b * a.ntiles + t);
          if (page_ok(a, id)) atomicSub(a.refs_out + id, 1);
        }
      } else if (t >= want && t < have) {
        const int id = a.table[b * a.ntiles + t];
        a.table_out[b * a.ntiles + t] = -1;
        if (page_ok(a, id)) atomicSub(a.refs_out + id, 1);
      }
    }
  }
  plan_sync();

  // a shared partly filled page stays with its first row, unless somebody
  // else holds it too; the other rows take a page for a copy
  for (int b = gwarp; b < a.batch; b += kPlanAll / 32) {
    const int page = __ldcg(a.ws.page + b);
    int take = 0;
    if (page >= 0) {
      int users = 0, before = 0;
      for (int o = lane; o < a.batch; o += 32) {
        const bool same = __ldcg(a.ws.page + o) == page;
        users += same;
        before += same && o < b;
      }
      users = __reduce_add_sync(0xffffffffu, users);
      before = __reduce_add_sync(0xffffffffu, before);
      take = before > 0 || __ldcg(a.refs_out + page) > users;
    }
    if constexpr (OP == kPageResize) {
      const int len = __ldcg(a.ws.len + b);
      const int have = a.lens[b] >= 0 && a.lens[b] <= a.capacity ? pages_for(a.lens[b]) : 0;
      take |= max(0, pages_for(len) - have) << 1;  // bit 0: the copy; above: new pages
    }
    if (lane == 0) a.ws.need[b] = take;
  }
  const int per = (a.n_pages + kPlanCtas - 1) / kPlanCtas;
  const int lo = min(a.n_pages, rank * per), hi = min(a.n_pages, lo + per);
  {
    const int n = plan_count(lo, hi, red, a.refs_out, false);
    if (tid == 0) a.ws.head[8 + rank] = n;
  }
  plan_sync();

  int first = 0, n_free = 0;
#pragma unroll
  for (int r = 0; r < kPlanCtas; ++r) {
    const int n = __ldcg(a.ws.head + 8 + r);
    first += r < rank ? n : 0;
    n_free += n;
  }
  plan_select(
      lo, hi, first, red, [&](int p) { return __ldcg(a.refs_out + p) == 0; },
      [&](int p, int k) { a.ws.list[k] = p; });
  if (rank == 0) {
    int64_t off = 0;
    for (int c = 0; c < a.batch; c += kPlanThreads) {
      const int b = c + tid;
      const int need = b < a.batch ? __ldcg(a.ws.need + b) : 0;
      int64_t total;
      const int64_t at = off + plan_scan(static_cast<int64_t>((need & 1) + (need >> 1)), wide, total);
      if (b < a.batch) a.ws.off[b] = static_cast<int>(min(at, static_cast<int64_t>(n_free)));
      off += total;
    }
    if (tid == 0) a.ws.head[0] = 0;
  }
  plan_sync();

  for (int b = gwarp; b < a.batch; b += kPlanAll / 32) {
    const int need = __ldcg(a.ws.need + b), off = __ldcg(a.ws.off + b), len = __ldcg(a.ws.len + b);
    const int take = need & 1, grow = need >> 1;
    int got = len;
    if constexpr (OP == kPageFork) {
      if (take) {
        const int page = __ldcg(a.ws.page + b), t = len / kTile;
        const int to = off < n_free ? __ldcg(a.ws.list + off) : -1;
        if (to < 0) got = t * kTile;
        if (lane == 0) {
          a.table_out[b * a.ntiles + t] = to;
          atomicSub(a.refs_out + page, 1);
          if (to >= 0) {
            a.refs_out[to] = 1;
            const int k = atomicAdd(a.ws.head, 1);
            a.ws.src[k] = page;
            a.ws.dst[k] = to;
          } else {
            atomicOr(a.err, kErrPool);
          }
        }
      }
    } else {
      const int was = a.lens[b] >= 0 && a.lens[b] <= a.capacity ? a.lens[b] : 0;
      bool full = true;
      if (take) {
        const int page = __ldcg(a.ws.page + b);
        full = off < n_free;
        if (!full) {
          got = was;  // the shared page stays as it is
        } else if (lane == 0) {
          const int to = __ldcg(a.ws.list + off);
          a.table_out[b * a.ntiles + was / kTile] = to;
          atomicSub(a.refs_out + page, 1);
          a.refs_out[to] = 1;
          const int k = atomicAdd(a.ws.head, 1);
          a.ws.src[k] = page;
          a.ws.dst[k] = to;
        }
      }
      if (grow > 0) {
        const int have = pages_for(was), can = min(grow, max(0, n_free - off - take));
        for (int i = lane; i < can; i += 32) {
          const int to = __ldcg(a.ws.list + off + take + i);
          a.table_out[b * a.ntiles + have + i] = to;
          a.refs_out[to] = 1;
        }
        if (can < grow) {
          if (full) got = (have + can) * kTile;
          full = false;
        }
      }
      if (!full && lane == 0) atomicOr(a.err, kErrPool);
    }
    __syncwarp();  // lens_out may be lens
    if (lane == 0) a.lens_out[b] = got;
  }
}

// Live pages move to [0, n_live): the k-th live page at or above n_live takes
// the k-th hole below it.
__global__ __launch_bounds__(kPlanThreads, 1) void compact_kernel(const __grid_constant__ PagePlanArgs a) {
  __shared__ int red[kPlanWarps];
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = blockIdx.x, gid = rank * kPlanThreads + tid, gwarp = gid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int per = (a.n_pages + kPlanCtas - 1) / kPlanCtas;
  const int lo = min(a.n_pages, rank * per), hi = min(a.n_pages, lo + per);
  {
    const int n = plan_count(lo, hi, red, a.refs, true);
    if (tid == 0) a.ws.head[8 + rank] = n;
  }
  plan_sync();
  int first = 0, n_live = 0;
#pragma unroll
  for (int r = 0; r < kPlanCtas; ++r) {
    const int n = __ldcg(a.ws.head + 8 + r);
    first += r < rank ? n : 0;
    n_live += n;
  }
  // holes below n_live by their ranks; live pages from n_live on by their
  // ranks among all live ones, counted from the end: both lists then need no
  // further count.  The j-th live page from the end takes the
  // (moves - 1 - j)-th hole.
  const int lo_end = min(hi, n_live), hi_begin = max(lo, n_live);
  plan_select(
      lo, lo_end, lo - first, red, [&](int p) { return __ldcg(a.refs + p) <= 0; },
      [&](int p, int k) { a.ws.dst[k] = p; });
  {
    const int mine = lo_end > lo ? plan_count(lo, lo_end, red, a.refs, true) : 0;  // live pages below n_live
    plan_select(
        hi_begin, hi, first + mine, red, [&](int p) { return __ldcg(a.refs + p) > 0; },
        [&](int p, int k) { a.ws.list[n_live - 1 - k] = p; });
    if (tid == 0) a.ws.head[16 + rank] = mine;
  }
  plan_sync();
  int moves = n_live;
#pragma unroll
  for (int r = 0; r < kPlanCtas; ++r) moves -= __ldcg(a.ws.head + 16 + r);
  if (gid == 0) {
    a.ws.head[0] = moves;
    a.n_live[0] = n_live;
  }
  // where each page goes, and its count there; a count is read before the
  // barrier and written behind it, so that refs_out may be refs
  for (int p = gid; p < a.n_pages; p += kPlanAll) a.map[p] = __ldcg(a.refs + p) > 0 && p < n_live ? p : -1;
  for (int k = gid; k < moves; k += kPlanAll) {
    const int src = __ldcg(a.ws.list + moves - 1 - k);
    a.ws.src[k] = src;
  }
  plan_sync();
  for (int k = gid; k < moves; k += kPlanAll) {
    const int src = __ldcg(a.ws.src + k), dst = __ldcg(a.ws.dst + k);
    a.map[src] = dst;
    a.refs_out[dst] = __ldcg(a.refs + src);
    if (a.refs_out == a.refs) a.refs_out[src] = 0;
  }
  if (a.refs_out != a.refs)
    for (int p = gid; p < a.n_pages; p += kPlanAll) {
      const int r = __ldcg(a.refs + p);
      if (p >= n_live)
        a.refs_out[p] = min(r, 0);
      else if (r > 0)
        a.refs_out[p] = r;
    }
  plan_sync();
  const int64_t chunks = (a.ntiles + kPlanChunk - 1) / kPlanChunk;
  for (int64_t it = gwarp; it < a.batch * chunks; it += kPlanAll / 32) {
    const int b = static_cast<int>(it / chunks);
    const int64_t t0 = (it - b * chunks) * kPlanChunk;
    const int len = a.lens[b];
    const bool ok = len >= 0 && len <= a.capacity;
    if (!ok && lane == 0 && t0 == 0) atomicOr(a.err, kErrSeqLen);
    const int held = ok ? pages_for(len) : 0;
#pragma unroll
    for (int i = 0; i < kPlanChunk / 32; ++i) {
      const int64_t t = t0 + 32 * i + lane;
      if (t >= held) continue;
      const int id = a.table[b * a.ntiles + t];
      const int to = page_ok(a, id) ? __ldcg(a.map + id) : -1;
      if (to < 0 && id >= 0 && id < a.n_pages) atomicOr(a.err, kErrPage);  // a free page in the table
      a.table_out[b * a.ntiles + t] = to;
    }
  }
}

// ---- the plans of a pool that fits one CTA's shared memory ---------------------
//
// The same steps with the counts in shared memory: two trips to global memory
// (counts and lengths, then the table) instead of one or two a step.  With the
// copy, one layer and head: a fork of 16 rows over 1024 pages takes 5.6 us
// instead of 9.7, a compaction of 4096 pages 12.4 instead of 16.7; at 8192
// pages both take as long, at 16384 this way 19.4 and the cluster 17.1 (1024
// rows: 97 and 38).

constexpr int kSmallThreads = 1024;
constexpr int kSmallPages = 8192;      // at most 65536: the lists' numbers have 16 bits
constexpr int kSmallRows = 256;

__host__ __device__ constexpr size_t small_smem(int n_pages, int batch) {
  return 4 * static_cast<size_t>(n_pages) + 20 * static_cast<size_t>(batch) + 4 * static_cast<size_t>(n_pages);
}

__device__ __forceinline__ void load_counts(const PagePlanArgs& a, int* refs) {
#pragma unroll 4
  for (int p = threadIdx.x; p < a.n_pages; p += kSmallThreads) refs[p] = __ldcg(a.refs + p);
}

template <int OP>
__global__ __launch_bounds__(kSmallThreads, 1) void small_plan_kernel(const __grid_constant__ PagePlanArgs a) {
  extern __shared__ int smem_int[];
  __shared__ int red[kSmallThreads / 32];
  __shared__ int64_t wide[kSmallThreads / 32];
  __shared__ int n_pairs;
  int* refs = smem_int;
  int *was = refs + a.n_pages, *row_v = was + a.batch, *len_v = row_v + a.batch, *page_v = len_v + a.batch,
      *off_v = page_v + a.batch;
  uint16_t* list = reinterpret_cast<uint16_t*>(off_v + a.batch);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) n_pairs = 0;
  load_counts(a, refs);
  for (int b = tid; b < a.batch; b += kSmallThreads) {
    was[b] = a.lens[b];
    row_v[b] = OP == kPageFork ? __ldg(a.parent + b) : __ldg(a.new_lens + b);
  }
  __syncthreads();

  // the rows' new lengths, and (resize) the partly filled page each would write
  for (int b = tid; b < a.batch; b += kSmallThreads) {
    int row = row_v[b], len, page = -1;
    if constexpr (OP == kPageFork) {
      if (row < -1 || row >= a.batch) {
        atomicOr(a.err, kErrArg);
        row = -1;
      }
      len = row < 0 ? 0 : checked_len(a, was[row]);
      if (row != b) checked_len(a, was[b]);  // for its flag
      row_v[b] = row;
    } else {
      const int part = checked_len(a, was[b]);
      len = row;
      if (len < 0 || len > a.capacity) {
        atomicOr(a.err, kErrSeqLen);
        len = part;
      }
      if (len > part && part % kTile != 0) {
        page = a.table[b * a.ntiles + part / kTile];
        if (!page_ok(a, page)) page = -1;
      }
    }
    len_v[b] = len;
    page_v[b] = page;
  }
  __syncthreads();

  // who holds what now
  const int64_t chunks = (a.ntiles + kPlanChunk - 1) / kPlanChunk;
  for (int64_t it = warp; it < a.batch * chunks; it += kSmallThreads / 32) {
    const int b = static_cast<int>(it / chunks);
    const int64_t t0 = (it - b * chunks) * kPlanChunk;
    const int have = was[b] >= 0 && was[b] <= a.capacity ? pages_for(was[b]) : 0;
    const int len = len_v[b], want = pages_for(len), row = OP == kPageFork ? row_v[b] : b;
    if (t0 >= max(have, want)) continue;
    int to[kPlanChunk / 32], from[kPlanChunk / 32];
#pragma unroll
    for (int i = 0; i < kPlanChunk / 32; ++i) {
      const int64_t t = t0 + 32 * i + lane;
      if (OP == kPageFork && t < want) to[i] = __ldg(a.table + row * a.ntiles + t);
      if (OP == kPageFork ? t < have && row != b : t >= want && t < have) from[i] = a.table[b * a.ntiles + t];
    }
#pragma unroll
    for (int i = 0; i < kPlanChunk / 32; ++i) {
      const int64_t t = t0 + 32 * i + lane;
      if (OP == kPageFork && t < want) {
        a.table_out[b * a.ntiles + t] = to[i];
        if (page_ok(a, to[i])) {
          if (row != b) atomicAdd(refs + to[i], 1);
          if (t == len / kTile) page_v[b] = to[i];
        }
      }
      if (OP == kPageFork ? t < have && row != b : t >= want && t < have) {
        if (OP == kPageResize) a.table_out[b * a.ntiles + t] = -1;
        if (page_ok(a, from[i])) atomicSub(refs + from[i], 1);
      }
    }
  }
  __syncthreads();

  // a shared partly filled page stays with its first row, unless somebody
  // else holds it too; the other rows take a page for a copy.  (row_v: bit
  // 0: the copy; above: new pages)
  for (int b = warp; b < a.batch; b += kSmallThreads / 32) {
    const int page = page_v[b];
    int take = 0;
    if (page >= 0) {
      int users = 0, before = 0;
      for (int o = lane; o < a.batch; o += 32) {
        const bool same = page_v[o] == page;
        users += same;
        before += same && o < b;
      }
      users = __reduce_add_sync(0xffffffffu, users);
      before = __reduce_add_sync(0xffffffffu, before);
      take = before > 0 || refs[page] > users;
    }
    if constexpr (OP == kPageResize) {
      const int have = was[b] >= 0 && was[b] <= a.capacity ? pages_for(was[b]) : 0;
      take |= max(0, pages_for(len_v[b]) - have) << 1;
    }
    if (lane == 0) row_v[b] = take;
  }
  __syncthreads();
  int64_t total = 0;
  for (int c = 0; c < a.batch; c += kSmallThreads) {
    const int b = c + tid, need = b < a.batch ? row_v[b] : 0;
    int64_t sum;
    const int64_t at = total + plan_scan<kSmallThreads>(static_cast<int64_t>((need & 1) + (need >> 1)), wide, sum);
    if (b < a.batch) off_v[b] = static_cast<int>(min(at, static_cast<int64_t>(a.n_pages)));
    total += sum;
  }
  const int found = plan_select<kSmallThreads>(
      0, a.n_pages, 0, red, [&](int p) { return refs[p] == 0; }, [&](int p, int k) { list[k] = static_cast<uint16_t>(p); },
      static_cast<int>(min(total, static_cast<int64_t>(a.n_pages))));
  __syncthreads();

  for (int b = warp; b < a.batch; b += kSmallThreads / 32) {
    const int take = row_v[b] & 1, grow = row_v[b] >> 1, off = off_v[b], len = len_v[b];
    const int old = was[b] >= 0 && was[b] <= a.capacity ? was[b] : 0;
    int got = len;
    bool full = true;
    if (take) {
      const int t = (OP == kPageFork ? len : old) / kTile;
      const int to = off < found ? list[off] : -1;
      full = to >= 0;
      if (!full) got = OP == kPageFork ? t * kTile : old;
      // a resize that finds no page leaves the shared one as it is
      if (lane == 0 && (full || OP == kPageFork)) {
        a.table_out[b * a.ntiles + t] = to;
        atomicSub(refs + page_v[b], 1);
        if (full) {
          refs[to] = 1;
          const int k = atomicAdd(&n_pairs, 1);
          a.ws.src[k] = page_v[b];
          a.ws.dst[k] = to;
        }
      }
    }
    if (OP == kPageResize && grow > 0) {
      const int have = pages_for(old), can = min(grow, max(0, found - off - take));
      for (int i = lane; i < can; i += 32) {
        const int to = list[off + take + i];
        a.table_out[b * a.ntiles + have + i] = to;
        refs[to] = 1;
      }
      if (can < grow) {
        if (full) got = (have + can) * kTile;
        full = false;
      }
    }
    if (lane == 0) {
      if (!full) atomicOr(a.err, kErrPool);
      a.lens_out[b] = got;
    }
  }
  __syncthreads();
  for (int p = tid; p < a.n_pages; p += kSmallThreads) a.refs_out[p] = refs[p];
  if (tid == 0) a.ws.head[0] = n_pairs;
}

__global__ __launch_bounds__(kSmallThreads, 1) void small_compact_kernel(const __grid_constant__ PagePlanArgs a) {
  extern __shared__ int smem_int[];
  __shared__ int red[kSmallThreads / 32];
  int* refs = smem_int;
  int* lens = refs + a.n_pages;
  uint16_t *srcs = reinterpret_cast<uint16_t*>(lens + a.batch), *holes = srcs + a.n_pages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  load_counts(a, refs);
  for (int b = tid; b < a.batch; b += kSmallThreads) lens[b] = a.lens[b];
  __syncthreads();
  int n = 0, n_live;
  for (int p = tid; p < a.n_pages; p += kSmallThreads) n += refs[p] > 0;
  plan_scan<kSmallThreads>(n, red, n_live);
  plan_select<kSmallThreads>(
      0, n_live, 0, red, [&](int p) { return refs[p] <= 0; }, [&](int p, int k) { holes[k] = static_cast<uint16_t>(p); });
  const int moves = plan_select<kSmallThreads>(
      n_live, a.n_pages, 0, red, [&](int p) { return refs[p] > 0; },
      [&](int p, int k) { srcs[k] = static_cast<uint16_t>(p); });
  __syncthreads();
  // a moved page's count goes with it
  for (int k = tid; k < moves; k += kSmallThreads) {
    const int src = srcs[k], dst = holes[k];
    a.ws.src[k] = src;
    a.ws.dst[k] = dst;
    a.refs_out[dst] = refs[src];
  }
  __syncthreads();
  for (int p = tid; p < a.n_pages; p += kSmallThreads) {
    const int r = refs[p];
    if (p >= n_live)
      a.refs_out[p] = min(r, 0);
    else if (r > 0)
      a.refs_out[p] = r;
    a.map[p] = refs[p] = r > 0 && p < n_live ? p : -1;  // from here on the map
  }
  __syncthreads();
  for (int k = tid; k < moves; k += kSmallThreads) a.map[srcs[k]] = refs[srcs[k]] = holes[k];
  if (tid == 0) {
    a.ws.head[0] = moves;
    a.n_live[0] = n_live;
  }
  __syncthreads();
  const int64_t chunks = (a.ntiles + kPlanChunk - 1) / kPlanChunk;
  for (int64_t it = warp; it < a.batch * chunks; it += kSmallThreads / 32) {
    const int b = static_cast<int>(it / chunks);
    const int64_t t0 = (it - b * chunks) * kPlanChunk;
    const int len = lens[b];
    const bool ok = len >= 0 && len <= a.capacity;
    if (!ok && lane == 0 && t0 == 0) atomicOr(a.err, kErrSeqLen);
    const int held = ok ? pages_for(len) : 0;
    if (t0 >= held) continue;
    int id[kPlanChunk / 32];
#pragma unroll
    for (int i = 0; i < kPlanChunk / 32; ++i) {
      const int64_t t = t0 + 32 * i + lane;
      if (t < held) id[i] = a.table[b * a.ntiles + t];
    }
#pragma unroll
    for (int i = 0; i < kPlanChunk / 32; ++i) {
      const int64_t t = t0 + 32 * i + lane;
      if (t >= held) continue;
      const int to = page_ok(a, id[i]) ? refs[id[i]] : -1;
      if (to < 0 && id[i] >= 0 && id[i] < a.n_pages) atomicOr(a.err, kErrPage);  // a free page in the table
      a.table_out[b * a.ntiles + t] = to;
    }
  }
}

// ---- the copy ----------------------------------------------------------------

constexpr int kCopyStages = 3;
constexpr int kCopyWarps = 8;              // most per CTA, one CTA an SM
constexpr int kCopySmem = 100 * 1024;
constexpr int kCopyWaitLimit = 1 << 20;    // polls of up to a microsecond each: about a second

__device__ __forceinline__ bool copy_wait(uint32_t bar, uint32_t parity) {
  for (int i = 0; i < kCopyWaitLimit; ++i) {
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

// An item is one (pair, layer, head): a slot of each array.  A warp takes
// items through its own ring of stages in shared memory by bulk copies: two
// items on their way in while one is on its way out, so an SM has up to 100
// KB in flight (200 were 3 % slower); its lanes look up 32 items at once.
// One value a slot (a scale) moves by a lane's load and store.
__global__ __launch_bounds__(32 * kCopyWarps, 1) void page_copy_kernel(const __grid_constant__ PageArrays c,
                                                                       const int32_t* __restrict__ src_v,
                                                                       const int32_t* __restrict__ dst_v, int n_pairs,
                                                                       const int32_t* n_pairs_dev, int stage,
                                                                       uint32_t* err) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kCopyWarps * kCopyStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const uint32_t bar0 = smem_u32(&bars[warp * kCopyStages]), buf0 = smem_u32(smem) + warp * kCopyStages * stage;
  if (lane < kCopyStages) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar0 + 8 * lane) : "memory");
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();
  if (n_pairs_dev != nullptr) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    n_pairs = min(n_pairs, __ldcg(n_pairs_dev));
  }
  const int64_t items = n_pairs * c.lh, step = static_cast<int64_t>(gridDim.x) * warps;
  const int64_t first = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
  if (first >= items) return;
  const int64_t mine = (items - first + step - 1) / step;
  int bytes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) bytes += c.bytes[i] >= 16 ? c.bytes[i] : 0;

  // lane's item among the 32 from `base` on: its slots, or -1 to skip it
  int64_t from = -1, to = -1;
  auto look_up = [&](int64_t base) {
    from = to = -1;
    if (base + lane >= mine) return;
    const int64_t it = first + (base + lane) * step, lh = it / n_pairs;
    const int pair = static_cast<int>(it - lh * n_pairs);
    const int src = __ldcg(src_v + pair), dst = __ldcg(dst_v + pair);
    if (src < 0 || src >= c.n_pages || dst < 0 || dst >= c.n_pages) {
      atomicOr(err, kErrPage);
      return;
    }
    if (src == dst) return;
    from = lh * c.n_pages + src;
    to = lh * c.n_pages + dst;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c.bytes[i] == 4)
        reinterpret_cast<uint32_t*>(c.base[i])[to] = __ldcg(reinterpret_cast<const uint32_t*>(c.base[i]) + from);
  };
  uint32_t phases = 0, pending = 0;       // bit i: parity of stage i's next completion; copies into it under way
  // copies of a slot into a stage; lane 0 issues
  auto load = [&](int st, int64_t slot) {
    if (slot < 0) return;
    pending |= 1u << st;
    if (lane != 0) return;
    uint32_t at = buf0 + st * stage;
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar0 + 8 * st), "r"(bytes) : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c.bytes[i] >= 16) {
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(at),
                     "l"(__cvta_generic_to_global(c.base[i] + slot * c.bytes[i])), "r"(c.bytes[i]), "r"(bar0 + 8 * st)
                     : "memory");
        at += c.bytes[i];
      }
  };
  int64_t next_from = -1, next_to = -1;   // of the 32 items after this one's
  look_up(0);
  {
    const int64_t f0 = __shfl_sync(0xffffffffu, from, 0), f1 = __shfl_sync(0xffffffffu, from, 1);
    load(0, f0);
    load(1, f1);
  }
  bool dead = false;
  int st = 0;
  for (int64_t k = 0; k < mine && !dead; ++k) {
    const int j = static_cast<int>(k & 31);
    if (j == 0 && k > 0) {
      from = next_from;
      to = next_to;
    }
    if (j == 16) {
      // ask for the next 32 while this half goes on; two of them are loaded ahead
      const int64_t f = from, t = to;
      look_up(k + 16);
      next_from = from;
      next_to = to;
      from = f;
      to = t;
    }
    const int64_t slot = __shfl_sync(0xffffffffu, to, j);
    if (slot >= 0) {
      if (__all_sync(0xffffffffu, copy_wait(bar0 + 8 * st, phases >> st & 1))) {
        phases ^= 1u << st;
        pending &= ~(1u << st);
        if (lane == 0) {
          uint32_t at = buf0 + st * stage;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c.bytes[i] >= 16) {
              asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                               __cvta_generic_to_global(c.base[i] + slot * c.bytes[i])),
                           "r"(at), "r"(c.bytes[i])
                           : "memory");
              at += c.bytes[i];
            }
        }
      } else {
        dead = true;
      }
    }
    // the stage two items on was last read by the stores of the item before
    // this one (an empty group where there were none)
    asm volatile("cp.async.bulk.commit_group;\n cp.async.bulk.wait_group.read 1;" ::: "memory");
    const int64_t f2 = j < 30 ? __shfl_sync(0xffffffffu, from, (j + 2) & 31)
                              : __shfl_sync(0xffffffffu, next_from, (j + 2) & 31);
    if (!dead && k + 2 < mine) load(st == 0 ? kCopyStages - 1 : st - 1, f2);
    st = st == kCopyStages - 1 ? 0 : st + 1;
  }
  if (dead) {
    if (lane == 0) atomicOr(err, kErrTimeout);
    // copies on their way land (bounded) before the shared memory goes
    for (int i = 0; i < kCopyStages; ++i)
      if (pending >> i & 1) copy_wait(bar0 + 8 * i, phases >> i & 1);
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

}  // namespace

cudaError_t launch_page_copy(const PageArrays& c, const int32_t* src, const int32_t* dst, int n_pairs,
                             const int32_t* n_pairs_dev, uint32_t* err, int n_sms, cudaStream_t stream) {
  int stage = 0;
  for (int i = 0; i < 4; ++i) stage += c.bytes[i] >= 16 ? c.bytes[i] : 0;
  stage = (stage + 127) / 128 * 128;
  int warps = kCopySmem / (kCopyStages * stage);
  warps = warps < kCopyWarps ? warps : kCopyWarps;
  const size_t smem = static_cast<size_t>(warps) * kCopyStages * stage;
  const int64_t items = n_pairs * c.lh;
  const unsigned grid = static_cast<unsigned>(items < n_sms ? items : n_sms);
  if (n_pairs_dev != nullptr)
    return launch_dependent(page_copy_kernel, dim3(grid), dim3(32 * warps), smem, stream, c, src, dst, n_pairs,
                            n_pairs_dev, stage, err);
  page_copy_kernel<<<grid, 32 * warps, smem, stream>>>(c, src, dst, n_pairs, nullptr, stage, err);
  return cudaGetLastError();
}

cudaError_t page_setup() {
  cudaError_t e = set_smem(page_copy_kernel, kCopySmem);
  const size_t most = small_smem(kSmallPages, kSmallRows);
  if (e == cudaSuccess) e = set_smem(small_plan_kernel<kPageFork>, most);
  if (e == cudaSuccess) e = set_smem(small_plan_kernel<kPageResize>, most);
  if (e == cudaSuccess) e = set_smem(small_compact_kernel, most);
  return e;
}

cudaError_t launch_page_plan(PageOp op, const PagePlanArgs& a, cudaStream_t stream) {
  if (a.n_pages <= kSmallPages && a.batch <= kSmallRows) {
    const size_t smem = small_smem(a.n_pages, a.batch);
    if (op == kPageFork)
      small_plan_kernel<kPageFork><<<1, kSmallThreads, smem, stream>>>(a);
    else if (op == kPageResize)
      small_plan_kernel<kPageResize><<<1, kSmallThreads, smem, stream>>>(a);
    else
      small_compact_kernel<<<1, kSmallThreads, smem, stream>>>(a);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPlanCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (op == kPageFork) return cudaLaunchKernelEx(&cfg, plan_kernel<kPageFork>, a);
  if (op == kPageResize) return cudaLaunchKernelEx(&cfg, plan_kernel<kPageResize>, a);
  return cudaLaunchKernelEx(&cfg, compact_kernel, a);
}

}  // namespace bgtq
