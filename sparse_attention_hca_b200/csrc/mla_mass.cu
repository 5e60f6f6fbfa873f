// mla_mass.cu -- the attention weight that every row of the paged cache of the full-context
// (MLA) layers received from a chunk of new tokens (mla_paged_attn_mass).
//
// Method: eviction keeps the rows that queries attended to, so each row accumulates
//     mass[s] += sum over the chunk's tokens t that see s, and the query heads of the K/V head,
//                of exp(scale <q[t], k_s> - lse[t])
// with the log-sum-exp of the attention call.
//
// One warp per (row, K/V head), lane l holding channels 8 l .. 8 l + 7 of the key.
#include "mla_host.h"

namespace hcadsa {
namespace {

struct Params {
  PagedBatch s;
  const uint16_t* Q;
  const uint16_t* K_pool;
  const float* lse;
  float* mass;
  long long q_row, k_page;
  int Hq, Hkv;
  float scale;
};

__device__ __forceinline__ void unpack8(const uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__global__ void __launch_bounds__(256) mass_kernel(const Params p) {
  const int b = blockIdx.y, hk = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PagedSeq q = paged_seq(p.s, b, blockIdx.x == 0 && hk == 0);
  const int g = p.Hq / p.Hkv, page_mask = (1 << p.s.page_log2) - 1;
  for (int i = blockIdx.x * 8 + warp; i < q.len; i += gridDim.x * 8) {
    const int pg = paged_page(p.s, b, i);
    if (pg < 0) continue;
    const size_t row = (size_t)(i & page_mask) * p.Hkv + hk;
    float kf[8];
    unpack8(reinterpret_cast<const uint4*>(p.K_pool + (size_t)pg * p.k_page + row * kMlaD)[lane], kf);
    float sum = 0.0f;
    for (int t = max(0, i - q.base); t < q.n; ++t)
      for (int h = hk * g; h < hk * g + g; ++h) {
        float qf[8], x = 0.0f;
        unpack8(reinterpret_cast<const uint4*>(p.Q + (size_t)(q.q0 + t) * p.q_row + (size_t)h * kMlaD)[lane], qf);
#pragma unroll
        for (int c = 0; c < 8; ++c) x = fmaf(qf[c], kf[c], x);
#pragma unroll
        for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
        sum += expf(x * p.scale - p.lse[(size_t)(q.q0 + t) * p.Hq + h]);
      }
    if (lane == 0) atomicAdd(p.mass + (((size_t)pg << p.s.page_log2) * p.Hkv) + row, sum);
  }
}

}  // namespace
}  // namespace hcadsa

extern "C" size_t mla_paged_attn_mass_workspace_size(int B, int T, int Hq, int Hkv) {
  (void)B;
  (void)T;
  (void)Hq;
  (void)Hkv;
  return 0;
}

extern "C" hcadsa_status mla_paged_attn_mass(const hcadsa_bf16* Q, long long q_row_stride, const hcadsa_bf16* K_pool,
                                             long long k_page_stride, const int32_t* table, const int32_t* cu_q,
                                             const int32_t* kv_len, const float* lse, float* mass, int B, int T,
                                             int n_pages, int page, int max_pages, int Hq, int Hkv, int d,
                                             float scale, void* workspace, size_t workspace_bytes,
                                             hcadsa_stream stream) {
  using namespace hcadsa;
  if (B > 0 && T > 0 && (!Q || !K_pool || !table || !cu_q || !kv_len || !lse || !mass)) return HCADSA_ERR_NULL;
  HCADSA_TRY(check_paged_sizes(B, n_pages, page, max_pages, Hkv));
  HCADSA_TRY(check_query_sizes(T, Hq, Hkv, d, scale));
  HCADSA_TRY(check_row_stride(q_row_stride, Hq));
  HCADSA_TRY(check_page_stride(k_page_stride, page, Hkv));
  if (!aligned16(Q) || !aligned16(K_pool) || !aligned4(table) || !aligned4(cu_q) || !aligned4(kv_len) ||
      !aligned4(lse) || !aligned4(mass))
    return HCADSA_ERR_ALIGN;
  if (B == 0 || T == 0) return HCADSA_OK;
  Params p;
  p.s = paged_batch(table, cu_q, kv_len, B, T, n_pages, page, max_pages);
  p.Q = Q;
  p.K_pool = K_pool;
  p.lse = lse;
  p.mass = mass;
  p.q_row = q_row_stride;
  p.k_page = k_page_stride;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.scale = scale;
  const long long cap = (long long)max_pages * page;
  mass_kernel<<<dim3((unsigned)(cap / 8 < 4096 ? cap / 8 : 4096), B, Hkv), 256, 0, as_stream(stream)>>>(p);
  return launch_status();
}
