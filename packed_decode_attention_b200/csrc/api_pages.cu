// The C ABI of the page operations (include/bgtq.h): argument checks and
// launches, for packed and 8-bit paged caches.
#include <cuda_runtime.h>

#include <cstring>

#include "pages.h"
#include "state.h"

using bgtq::as_stream;
using bgtq::check_device;

namespace {

struct Range {
  const void* p;
  int64_t bytes;
};

bool aligned4(const Range& r) { return reinterpret_cast<uintptr_t>(r.p) % 4 == 0; }

bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + uintptr_t(b.bytes) && y < x + uintptr_t(a.bytes);
}

// Outputs lie apart from one another and from the inputs, except that
// output i may be input twin[i] itself (-1: none).
int check_ranges(const Range* in, int n_in, const Range* out, int n_out, const int* twin) {
  for (int i = 0; i < n_in; ++i)
    if (!aligned4(in[i])) return BGTQ_ERR_ALIGNMENT;
  for (int i = 0; i < n_out; ++i) {
    if (!aligned4(out[i])) return BGTQ_ERR_ALIGNMENT;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return BGTQ_ERR_INVALID_ARG;
    for (int j = 0; j < n_in; ++j)
      if (overlap(out[i], in[j]) && !(twin[i] == j && out[i].p == in[j].p)) return BGTQ_ERR_INVALID_ARG;
  }
  return BGTQ_OK;
}

int check_paged(const bgtq_state* st, int32_t batch) {
  if (st->cache.n_pages == 0) return BGTQ_ERR_INVALID_ARG;
  if (const int dv = check_device(st)) return dv;
  return batch < 1 || batch > st->cfg.max_batch ? BGTQ_ERR_INVALID_ARG : BGTQ_OK;
}

bgtq::PageArrays arrays(const bgtq_state* st) {
  bgtq::PageArrays c;
  if (st->byte) {
    for (int i = 0; i < 2; ++i) {
      c.base[2 * i] = st->byte_cache.codes[i];
      c.bytes[2 * i] = bgtq::kByteTileBytes;
      c.base[2 * i + 1] = reinterpret_cast<uint8_t*>(st->byte_cache.scales[i]);
      c.bytes[2 * i + 1] = 4;
    }
  } else {
    c.base[0] = reinterpret_cast<uint8_t*>(st->cache.ktile);
    c.bytes[0] = 1024 * st->shape.kbits;
    c.base[1] = reinterpret_cast<uint8_t*>(st->cache.knorm);
    c.bytes[1] = bgtq::kTile * 8;
    c.base[2] = reinterpret_cast<uint8_t*>(st->cache.vtile);
    c.bytes[2] = 1024 * st->shape.vbits;
    c.base[3] = reinterpret_cast<uint8_t*>(st->cache.vnorm);
    c.bytes[3] = bgtq::kTile * 2;
  }
  c.n_pages = st->cache.n_pages;
  c.lh = int64_t(st->cfg.n_layers) * st->cfg.n_kv_heads;
  return c;
}

bgtq::PagePlanArgs plan_args(const bgtq_state* st, int32_t batch, void* scratch) {
  bgtq::PagePlanArgs a;
  std::memset(&a, 0, sizeof(a));
  a.ws = bgtq::page_scratch(static_cast<int32_t*>(scratch), st->cfg.max_batch, st->cache.n_pages);
  a.err = st->ws.err;
  a.capacity = st->cfg.capacity_tokens;
  a.ntiles = (st->cfg.capacity_tokens + bgtq::kTile - 1) / bgtq::kTile;
  a.n_pages = st->cache.n_pages;
  a.batch = batch;
  return a;
}

// The plan, then the copy of at most `most` pairs.
int plan_and_copy(const bgtq_state* st, bgtq::PageOp op, const bgtq::PagePlanArgs& a, int most, void* stream) {
  if (bgtq::launch_page_plan(op, a, as_stream(stream)) != cudaSuccess) return BGTQ_ERR_CUDA;
  if (bgtq::launch_page_copy(arrays(st), a.ws.src, a.ws.dst, most < a.n_pages ? most : a.n_pages, a.ws.head, st->ws.err,
                             st->num_sms, as_stream(stream)) != cudaSuccess)
    return BGTQ_ERR_CUDA;
  return BGTQ_OK;
}

int64_t table_bytes(const bgtq_state* st, int32_t batch) {
  return 4 * int64_t(batch) * ((st->cfg.capacity_tokens + bgtq::kTile - 1) / bgtq::kTile);
}

size_t scratch_bytes(const bgtq_state* st) {
  return 4 * bgtq::page_scratch_ints(st->cfg.max_batch, st->cache.n_pages);
}

Range scratch_range(const bgtq_state* st, const void* p) { return Range{p, int64_t(scratch_bytes(st))}; }

}  // namespace

extern "C" {

int bgtq_page_scratch_bytes(const bgtq_state* st, size_t* bytes) {
  if (!st || !bytes) return BGTQ_ERR_NULL;
  if (st->cache.n_pages == 0) return BGTQ_ERR_INVALID_ARG;
  *bytes = scratch_bytes(st);
  return BGTQ_OK;
}

int bgtq_copy_pages(bgtq_state* st, const int32_t* d_src, const int32_t* d_dst, int32_t n, void* stream) {
  if (!st || !d_src || !d_dst) return BGTQ_ERR_NULL;
  if (const int v = check_paged(st, 1)) return v;
  if (n < 0) return BGTQ_ERR_INVALID_ARG;
  if (!aligned4(Range{d_src, 0}) || !aligned4(Range{d_dst, 0})) return BGTQ_ERR_ALIGNMENT;
  if (n == 0) return BGTQ_OK;
  return bgtq::launch_page_copy(arrays(st), d_src, d_dst, n, nullptr, st->ws.err, st->num_sms, as_stream(stream)) ==
                 cudaSuccess
             ? BGTQ_OK
             : BGTQ_ERR_CUDA;
}

int bgtq_fork_sequences(bgtq_state* st, const int32_t* d_parent, const int32_t* d_table, const int32_t* d_refs,
                        const int32_t* d_lens, int32_t batch, int32_t* d_table_out, int32_t* d_refs_out,
                        int32_t* d_lens_out, void* d_scratch, void* stream) {
  if (!st || !d_parent || !d_table || !d_refs || !d_lens || !d_table_out || !d_refs_out || !d_lens_out || !d_scratch)
    return BGTQ_ERR_NULL;
  if (const int v = check_paged(st, batch)) return v;
  const int64_t pool = 4 * int64_t(st->cache.n_pages), rows = 4 * int64_t(batch), tb = table_bytes(st, batch);
  const Range in[4] = {{d_parent, rows}, {d_table, tb}, {d_refs, pool}, {d_lens, rows}};
  const Range out[4] = {{d_table_out, tb}, {d_refs_out, pool}, {d_lens_out, rows}, scratch_range(st, d_scratch)};
  const int twin[4] = {-1, 2, 3, -1};
  if (const int v = check_ranges(in, 4, out, 4, twin)) return v;
  bgtq::PagePlanArgs a = plan_args(st, batch, d_scratch);
  a.parent = d_parent;
  a.table = d_table;
  a.refs = d_refs;
  a.lens = d_lens;
  a.table_out = d_table_out;
  a.refs_out = d_refs_out;
  a.lens_out = d_lens_out;
  return plan_and_copy(st, bgtq::kPageFork, a, batch, stream);
}

int bgtq_resize_sequences(bgtq_state* st, int32_t* d_table, int32_t* d_refs, const int32_t* d_lens,
                          const int32_t* d_new_lens, int32_t batch, int32_t* d_lens_out, void* d_scratch, void* stream) {
  if (!st || !d_table || !d_refs || !d_lens || !d_new_lens || !d_lens_out || !d_scratch) return BGTQ_ERR_NULL;
  if (const int v = check_paged(st, batch)) return v;
  const int64_t pool = 4 * int64_t(st->cache.n_pages), rows = 4 * int64_t(batch), tb = table_bytes(st, batch);
  // lens_out may be either of the lengths, or both where they are one
  const bool is_new = d_lens_out == d_new_lens;
  const Range in[2] = {{is_new ? d_new_lens : d_lens, rows}, {is_new ? d_lens : d_new_lens, rows}};
  const Range out[4] = {{d_table, tb}, {d_refs, pool}, {d_lens_out, rows}, scratch_range(st, d_scratch)};
  const int twin[4] = {-1, -1, 0, -1};
  if (const int v = check_ranges(in, d_lens == d_new_lens ? 1 : 2, out, 4, twin)) return v;
  bgtq::PagePlanArgs a = plan_args(st, batch, d_scratch);
  a.table = d_table;
  a.refs = d_refs;
  a.lens = d_lens;
  a.new_lens = d_new_lens;
  a.table_out = d_table;
  a.refs_out = d_refs;
  a.lens_out = d_lens_out;
  return plan_and_copy(st, bgtq::kPageResize, a, batch, stream);
}

int bgtq_compact_pages(bgtq_state* st, const int32_t* d_table, const int32_t* d_refs, const int32_t* d_lens,
                       int32_t batch, int32_t* d_table_out, int32_t* d_refs_out, int32_t* d_map, int32_t* d_n_live,
                       void* d_scratch, void* stream) {
  if (!st || !d_table || !d_refs || !d_lens || !d_table_out || !d_refs_out || !d_map || !d_n_live || !d_scratch)
    return BGTQ_ERR_NULL;
  if (const int v = check_paged(st, batch)) return v;
  const int64_t pool = 4 * int64_t(st->cache.n_pages), rows = 4 * int64_t(batch), tb = table_bytes(st, batch);
  const Range in[3] = {{d_table, tb}, {d_refs, pool}, {d_lens, rows}};
  const Range out[5] = {{d_table_out, tb}, {d_refs_out, pool}, {d_map, pool}, {d_n_live, 4}, scratch_range(st, d_scratch)};
  const int twin[5] = {0, 1, -1, -1, -1};
  if (const int v = check_ranges(in, 3, out, 5, twin)) return v;
  bgtq::PagePlanArgs a = plan_args(st, batch, d_scratch);
  a.table = d_table;
  a.refs = d_refs;
  a.lens = d_lens;
  a.table_out = d_table_out;
  a.refs_out = d_refs_out;
  a.map = d_map;
  a.n_live = d_n_live;
  return plan_and_copy(st, bgtq::kPageCompact, a, st->cache.n_pages, stream);
}

}  // extern "C"
