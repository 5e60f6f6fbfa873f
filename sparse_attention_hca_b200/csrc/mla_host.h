// mla_host.h -- host-side checks shared by the paged-cache entry points of the full-context
// (MLA) layers.
#pragma once
#include "host_common.h"
#include "mla_paged.cuh"

namespace hcadsa {

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

// Sizes of a pool of pages and of a batch over it.  A page is a power of two between 16 rows
// (the narrowest box the attention kernels load) and 1024.
inline hcadsa_status check_paged_sizes(int B, int n_pages, int page, int max_pages, int Hkv) {
  if (B < 0 || n_pages <= 0 || max_pages <= 0 || Hkv <= 0) return HCADSA_ERR_SHAPE;
  if (page < 16 || page > 1024 || (page & (page - 1))) return HCADSA_ERR_UNSUPPORTED;
  if ((long long)max_pages * page > (1LL << 30) || (long long)n_pages * page * Hkv > (1LL << 40) || Hkv > 65535 ||
      B > (1 << 24))
    return HCADSA_ERR_UNSUPPORTED;
  return HCADSA_OK;
}

// A page stride (elements): pages may not overlap and rows stay 16-byte aligned.
inline hcadsa_status check_page_stride(long long stride, int page, int Hkv) {
  if (stride < (long long)page * Hkv * kMlaD) return HCADSA_ERR_SHAPE;
  return stride % 8 ? HCADSA_ERR_ALIGN : HCADSA_OK;
}

// A row stride (elements) of packed new rows [T, H, 256].
inline hcadsa_status check_row_stride(long long stride, int H) {
  if (stride < (long long)H * kMlaD) return HCADSA_ERR_SHAPE;
  return stride % 8 ? HCADSA_ERR_ALIGN : HCADSA_OK;
}

// Query sizes: whole groups of query heads per K/V head, a power of two up to 128, so that a tile
// of 128 rows holds whole tokens.
inline hcadsa_status check_query_sizes(int T, int Hq, int Hkv, int d, float scale) {
  if (T < 0 || Hq <= 0 || Hq % Hkv || !(scale > 0.0f)) return HCADSA_ERR_SHAPE;
  const int g = Hq / Hkv;
  if (d != kMlaD || g > 128 || (g & (g - 1)) || T > (1 << 23)) return HCADSA_ERR_UNSUPPORTED;
  return HCADSA_OK;
}

inline PagedBatch paged_batch(const int32_t* table, const int32_t* cu_q, const int32_t* kv_len, int B, int T,
                              int n_pages, int page, int max_pages) {
  PagedBatch s;
  s.table = table;
  s.cu_q = cu_q;
  s.kv_len = kv_len;
  s.err = device_error_ptr();
  s.B = B;
  s.T = T;
  s.n_pages = n_pages;
  s.max_pages = max_pages;
  s.page_log2 = log2_of(page);
  return s;
}

// Launches a kernel that follows one on the same stream and calls wait_for_primary() before it reads
// what that one wrote: its launch overlaps the end of the first.
template <typename... Params, typename... Args>
hcadsa_status launch_after(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, Params(args)...) != cudaSuccess) return launch_status();
  return launch_status();
}

#define HCADSA_TRY(expr)                             \
  do {                                               \
    const hcadsa_status try_st_ = (expr);            \
    if (try_st_ != HCADSA_OK) return try_st_;        \
  } while (0)

}  // namespace hcadsa
