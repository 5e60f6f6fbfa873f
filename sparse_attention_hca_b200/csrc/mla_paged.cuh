// mla_paged.cuh -- what the paged-cache kernels of the full-context (MLA) layers share: the
// description of a ragged batch over pages, read from device memory, and its checks.
//
// A batch of B sequences is given by cu_q (sequence b's new tokens are the rows cu_q[b] ..
// cu_q[b+1]-1 of the packed new rows), kv_len (rows in b's cache, its new tokens included) and
// a page table: row i of b's cache lies in page table[b * max_pages + i / page] at i % page.
// The host never sees these values, so every kernel clamps what it reads to the sizes it was
// given and records HCADSA_ERR_DEVICE_BOUNDS where a value was out of range: no entry of a
// table or length array can make a kernel touch memory outside the tensors.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace hcadsa {

constexpr int kMlaD = 256;  // head width of the full-context layers

struct PagedBatch {
  const int32_t* table;   // [B, max_pages]
  const int32_t* cu_q;    // [B + 1]
  const int32_t* kv_len;  // [B]
  int* err;
  int B, T, n_pages, max_pages, page_log2;
};

struct PagedSeq {
  int q0;    // first packed row of the new tokens
  int n;     // new tokens
  int len;   // rows in the cache
  int base;  // rows before the new tokens: new token i sees the rows <= base + i
};

// Rows of sequence b, clamped to the capacity of its table row.
__device__ __forceinline__ int paged_len(const PagedBatch& s, int b, bool report) {
  const int cap = s.max_pages << s.page_log2;
  const int len = s.kv_len[b];
  if (len >= 0 && len <= cap) return len;
  if (report) raise_device_error(s.err, kErrDeviceBounds);
  return len < 0 ? 0 : cap;
}

__device__ __forceinline__ PagedSeq paged_seq(const PagedBatch& s, int b, bool report) {
  const int a = s.cu_q[b], z = s.cu_q[b + 1];
  PagedSeq r;
  r.len = paged_len(s, b, report);
  r.q0 = a < 0 ? 0 : (a > s.T ? s.T : a);
  const int e = z < r.q0 ? r.q0 : (z > s.T ? s.T : z);
  if (report && (r.q0 != a || e != z)) raise_device_error(s.err, kErrDeviceBounds);
  r.n = e - r.q0;
  r.base = r.len - r.n;
  return r;
}

// Page of row i (i < max_pages * page) of sequence b, or -1 (recorded) if the table's entry is
// not a page of the pool.
__device__ __forceinline__ int paged_page(const PagedBatch& s, int b, int i) {
  const int pg = s.table[(size_t)b * s.max_pages + (i >> s.page_log2)];
  if (pg >= 0 && pg < s.n_pages) return pg;
  raise_device_error(s.err, kErrDeviceBounds);
  return -1;
}

}  // namespace hcadsa
