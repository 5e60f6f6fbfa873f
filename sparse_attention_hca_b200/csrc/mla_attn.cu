// mla_attn.cu -- attention of a chunk of new tokens over the paged cache of the full-context
// (MLA) layers (mla_paged_attn_fwd).
//
// Method: the mirrorspeed page, section "Hybrid sparse attention, 1/7 full context access": the
// MLA layers see every token; heads are 256 wide.  New token i of a sequence sees the rows
// <= base + i of its cache (base: rows before the chunk):
//     O = sum_s p_s v_s,  p = softmax_s(scale <q, k_s>),  lse = log sum_s exp(scale <q, k_s>)
//
// One warp per (token, query head), lane l holding channels 8 l .. 8 l + 7: one pass over the
// visible rows with a running maximum and sum.
#include "mla_host.h"

namespace hcadsa {
namespace {

struct Params {
  PagedBatch s;
  const uint16_t* Q;
  const uint16_t* K_pool;
  const uint16_t* V_pool;
  uint16_t* O;
  float* lse;
  long long q_row, k_page, v_page;
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

__global__ void __launch_bounds__(256) attn_kernel(const Params p) {
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ int owner;
  if (threadIdx.x == 0) owner = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < p.s.B; b += blockDim.x) {
    const PagedSeq q = paged_seq(p.s, b, t == 0);
    if (t >= q.q0 && t < q.q0 + q.n) owner = b;
  }
  __syncthreads();
  const int b = owner;
  if (b < 0) return;
  const PagedSeq q = paged_seq(p.s, b, false);
  const int n_vis = min(q.len, q.base + (t - q.q0) + 1);
  const int page_mask = (1 << p.s.page_log2) - 1;
  for (int h = blockIdx.y * 8 + warp; h < p.Hq; h += 8 * gridDim.y) {
    const int hk = h / (p.Hq / p.Hkv);
    float qf[8], o[8] = {};
    unpack8(reinterpret_cast<const uint4*>(p.Q + (size_t)t * p.q_row + (size_t)h * kMlaD)[lane], qf);
    float m = -INFINITY, l = 0.0f;
    for (int i = 0; i < n_vis; ++i) {
      const int pg = paged_page(p.s, b, i);
      float kf[8] = {}, vf[8] = {};
      if (pg >= 0) {
        const size_t row = ((size_t)(i & page_mask) * p.Hkv + hk) * kMlaD;
        unpack8(reinterpret_cast<const uint4*>(p.K_pool + (size_t)pg * p.k_page + row)[lane], kf);
        unpack8(reinterpret_cast<const uint4*>(p.V_pool + (size_t)pg * p.v_page + row)[lane], vf);
      }
      float x = 0.0f;
#pragma unroll
      for (int c = 0; c < 8; ++c) x = fmaf(qf[c], kf[c], x);
#pragma unroll
      for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
      x *= p.scale;
      const float mn = fmaxf(m, x), a = expf(m - mn), w = expf(x - mn);
      m = mn;
      l = fmaf(l, a, w);
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = fmaf(o[c], a, w * vf[c]);
    }
    const float inv = n_vis > 0 ? 1.0f / l : 0.0f;
    const size_t row = (size_t)t * p.Hq + h;
    uint4 w;
    w.x = pack_bf16x2(o[0] * inv, o[1] * inv);
    w.y = pack_bf16x2(o[2] * inv, o[3] * inv);
    w.z = pack_bf16x2(o[4] * inv, o[5] * inv);
    w.w = pack_bf16x2(o[6] * inv, o[7] * inv);
    reinterpret_cast<uint4*>(p.O + row * kMlaD)[lane] = w;
    if (p.lse && lane == 0) p.lse[row] = n_vis > 0 ? m + logf(l) : -INFINITY;
  }
}

}  // namespace
}  // namespace hcadsa

extern "C" size_t mla_paged_attn_fwd_workspace_size(int B, int T, int Hq, int Hkv) {
  (void)B;
  (void)T;
  (void)Hq;
  (void)Hkv;
  return 0;
}

extern "C" hcadsa_status mla_paged_attn_fwd(const hcadsa_bf16* Q, long long q_row_stride, const hcadsa_bf16* K_pool,
                                            const hcadsa_bf16* V_pool, long long k_page_stride,
                                            long long v_page_stride, const int32_t* table, const int32_t* cu_q,
                                            const int32_t* kv_len, hcadsa_bf16* O, float* lse, int B, int T,
                                            int n_pages, int page, int max_pages, int Hq, int Hkv, int d,
                                            float scale, void* workspace, size_t workspace_bytes,
                                            hcadsa_stream stream) {
  using namespace hcadsa;
  if (B > 0 && T > 0 && (!Q || !K_pool || !V_pool || !table || !cu_q || !kv_len || !O)) return HCADSA_ERR_NULL;
  HCADSA_TRY(check_paged_sizes(B, n_pages, page, max_pages, Hkv));
  HCADSA_TRY(check_query_sizes(T, Hq, Hkv, d, scale));
  HCADSA_TRY(check_row_stride(q_row_stride, Hq));
  HCADSA_TRY(check_page_stride(k_page_stride, page, Hkv));
  HCADSA_TRY(check_page_stride(v_page_stride, page, Hkv));
  if (!aligned16(Q) || !aligned16(K_pool) || !aligned16(V_pool) || !aligned16(O) || !aligned4(table) ||
      !aligned4(cu_q) || !aligned4(kv_len) || !aligned4(lse))
    return HCADSA_ERR_ALIGN;
  if (B == 0 || T == 0) return HCADSA_OK;
  Params p;
  p.s = paged_batch(table, cu_q, kv_len, B, T, n_pages, page, max_pages);
  p.Q = Q;
  p.K_pool = K_pool;
  p.V_pool = V_pool;
  p.O = O;
  p.lse = lse;
  p.q_row = q_row_stride;
  p.k_page = k_page_stride;
  p.v_page = v_page_stride;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.scale = scale;
  attn_kernel<<<dim3(T, (Hq + 7) / 8 < 8 ? (Hq + 7) / 8 : 8), 256, 0, as_stream(stream)>>>(p);
  return launch_status();
}
