// Launch parameters of the page operations (pages.cu), shared by the kernels
// and the C ABI (api_pages.cu).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bgtq {

// The four arrays of a paged cache, packed or 8-bit: bytes[i] a slot (a
// multiple of 16, or 4), slots [L][H][P].
struct PageArrays {
  uint8_t* base[4];
  int32_t bytes[4];
  int32_t n_pages;
  int64_t lh;             // layers x KV heads
};

enum PageOp { kPageFork, kPageResize, kPageCompact };

// int32 places in the workspace that a plan leaves for the copy.
struct PageScratch {
  int32_t* head;          // [0] pairs to copy, [8 ..] a plan's partial counts
  int32_t* page;          // [max_batch] the partly filled page a row shares, or -1
  int32_t* len;           // [max_batch] a row's new length
  int32_t* need;          // [max_batch] pages it takes
  int32_t* off;           // [max_batch] pages taken by the rows before it
  int32_t* list;          // [n_pages] free pages, ascending
  int32_t* src;           // [n_pages] pairs
  int32_t* dst;           // [n_pages]
};

constexpr int kPageHead = 64;

inline size_t page_scratch_ints(int max_batch, int n_pages) {
  return kPageHead + 4 * static_cast<size_t>(max_batch) + 3 * static_cast<size_t>(n_pages);
}

inline PageScratch page_scratch(int32_t* p, int max_batch, int n_pages) {
  PageScratch s;
  s.head = p;
  s.page = p + kPageHead;
  s.len = s.page + max_batch;
  s.need = s.len + max_batch;
  s.off = s.need + max_batch;
  s.list = s.off + max_batch;
  s.src = s.list + n_pages;
  s.dst = s.src + n_pages;
  return s;
}

struct PagePlanArgs {
  PageScratch ws;
  const int32_t* parent;    // fork
  const int32_t* table;
  const int32_t* refs;
  const int32_t* lens;
  const int32_t* new_lens;  // resize
  int32_t* table_out;
  int32_t* refs_out;
  int32_t* lens_out;
  int32_t* map;             // compact
  int32_t* n_live;          // compact
  uint32_t* err;
  int64_t capacity, ntiles;
  int32_t n_pages, batch;
};

// Sets the kernels' shared-memory limits on the current device.
cudaError_t page_setup();
// Copies pages src[i] to dst[i], i < n_pairs (n_pairs_dev null) or, after the
// plan that the stream holds, i < *n_pairs_dev <= n_pairs.
cudaError_t launch_page_copy(const PageArrays& c, const int32_t* src, const int32_t* dst, int n_pairs,
                             const int32_t* n_pairs_dev, uint32_t* err, int n_sms, cudaStream_t stream);
cudaError_t launch_page_plan(PageOp op, const PagePlanArgs& a, cudaStream_t stream);

}  // namespace bgtq
