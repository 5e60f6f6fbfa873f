// mla_evict.cu -- which rows of a paged cache stay when it is cut to a budget (mla_evict_select).
//
// Method: eviction by accumulated attention weight.  A row stays if its position is one of the
// first n_sink or of the last n_recent of its sequence; the rest of the budget goes to the rows
// with the most weight, equal weights to the lower row.  Rows that stay below the budget are not
// touched; the i-th row that stays beyond it moves to the i-th freed place below it, so a cut of
// m rows moves at most m rows, whatever the budget.
//
// One cluster of 1 to 8 CTAs per (sequence, K/V head); a CTA owns a contiguous slice of the rows.
//   * Weights become 32-bit keys whose order is that of the weights (protected rows on top) and
//     stay in shared memory.  The budget-th largest key is found with a radix select of 11, 11
//     and 10 bits: a histogram per CTA, summed over the cluster through distributed shared
//     memory, so all CTAs follow the same bin.
//   * Ties at the threshold are taken in row order: every warp owns a contiguous run of its
//     CTA's slice, and prefix counts over warps and CTAs give each row its rank, with no atomics:
//     the result does not depend on timing.
// Slices that do not fit in shared memory (caches of more than 8 * 48K rows) are read from
// global memory again in every pass.
#include "mla_host.h"
#include "pair.cuh"

namespace hcadsa {
namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kSliceTarget = 4096;     // rows per CTA below which a list gets no further CTA
constexpr int kMaxSmemRows = 48 * 1024;

struct Params {
  PagedBatch s;
  const float* mass;
  const int32_t* pos;
  const int32_t* seen;
  int2* moves;
  int32_t* new_len;
  int Hkv, budget, n_sink, n_recent, n_moves;
  int smem_rows;  // rows of a slice that fit the dynamic shared memory; 0: keys are recomputed
};

struct Shared {
  uint32_t hist[kBins];    // this CTA's counts (read by the cluster)
  uint32_t warp_sum[32];
  uint32_t digit, above;   // found by one thread of every CTA
  uint32_t total[2];       // this CTA's counts of a pass (read by the cluster)
};

// Keys in the order of the weights: protected rows over everything, NaN over +inf, -0 equal to 0.
__device__ __forceinline__ uint32_t key_of(float m, bool safe) {
  if (safe) return 0xffffffffu;
  if (m != m) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(m + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t warp_incl_scan(uint32_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

__global__ void __launch_bounds__(kThreads, 1) select_kernel(const Params p) {
  extern __shared__ uint32_t keys[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t n_cta;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n_cta));
  const uint32_t rank = cluster_rank();
  const int list = blockIdx.x / n_cta;
  const int b = list / p.Hkv, h = list - b * p.Hkv;
  const int len = paged_len(p.s, b, h == 0 && rank == 0 && tid == 0);
  int2* out = p.moves + (size_t)list * p.n_moves;
  if (h == 0 && rank == 0 && tid == 0) p.new_len[b] = min(len, p.budget);
  if (len <= p.budget) {  // nothing to evict
    for (int i = rank * kThreads + tid; i < p.n_moves; i += n_cta * kThreads) out[i] = make_int2(-1, -1);
    return;
  }
  // rows [lo, hi) of this CTA; warp w owns rows [lo + w * per_warp, ...)
  const int per_cta = ((len + (int)n_cta - 1) / (int)n_cta + kThreads - 1) / kThreads * kThreads;
  const int lo = min(len, (int)rank * per_cta), hi = min(len, lo + per_cta);
  const int per_warp = per_cta / 32;
  const int w_lo = min(hi, lo + warp * per_warp), w_hi = min(hi, w_lo + per_warp);
  const bool in_smem = per_cta <= p.smem_rows;
  const long long seen = p.seen ? p.seen[b] : len;
  const int page_mask = (1 << p.s.page_log2) - 1;

  auto load_key = [&](int i) -> uint32_t {
    const int pg = paged_page(p.s, b, i);
    if (pg < 0) return key_of(0.0f, false);
    const size_t slot = (((size_t)pg << p.s.page_log2) + (i & page_mask)) * p.Hkv + h;
    const int ps = p.pos[slot];
    return key_of(p.mass[slot], ps < p.n_sink || ps >= seen - p.n_recent);
  };
  if (in_smem) {
#pragma unroll 4
    for (int i = lo + tid; i < hi; i += kThreads) keys[i - lo] = load_key(i);
  }
  auto key_at = [&](int i) -> uint32_t { return in_smem ? keys[i - lo] : load_key(i); };
  __syncthreads();

  // ---- the budget-th largest key: `prefix` holds its bits found so far, `need` its rank among
  // the rows that share them
  uint32_t prefix = 0, need = p.budget;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bits = pass == 2 ? 10 : 11;
    const uint32_t mask = (1u << bits) - 1;
    for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
    __syncthreads();
    for (int i0 = lo + (tid & ~31); i0 < hi; i0 += kThreads) {
      const int i = i0 + lane;
      const uint32_t k = i < hi ? key_at(i) : 0;
      const bool in = i < hi && (pass == 0 || (k >> (shift + bits)) == prefix);
      const uint32_t d = (k >> shift) & mask;
      // rows of one bin in a whole warp (protected runs, ties) cost one atomic instead of 32
      const uint32_t live = __ballot_sync(0xffffffffu, in);
      if (!live) continue;
      const uint32_t d0 = __shfl_sync(0xffffffffu, d, __ffs(live) - 1);
      if (__all_sync(0xffffffffu, !in || d == d0)) {
        if (lane == 0) atomicAdd(&sh.hist[d0], __popc(live));
      } else if (in) {
        atomicAdd(&sh.hist[d], 1u);
      }
    }
    __syncthreads();
    if (n_cta > 1) cluster_sync();
    // bins from the top: thread t holds bins 2047 - 2t and 2046 - 2t
    uint32_t c0 = 0, c1 = 0;
    for (uint32_t r = 0; r < n_cta; ++r) {
      const uint32_t a = cluster_addr(&sh.hist[kBins - 2 - 2 * tid], r);
      c1 += ld_cluster_u32(a);
      c0 += ld_cluster_u32(a + 4);
    }
    const uint32_t incl = warp_incl_scan(c0 + c1, lane);
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    if (warp == 0) sh.warp_sum[lane] = warp_incl_scan(sh.warp_sum[lane], lane);
    __syncthreads();
    const uint32_t upto = incl + (warp ? sh.warp_sum[warp - 1] : 0), before = upto - c0 - c1;
    if (before < need && need <= upto) {
      const bool first = need <= before + c0;
      sh.digit = kBins - 1 - 2 * tid - (first ? 0 : 1);
      sh.above = before + (first ? 0 : c0);
    }
    __syncthreads();
    prefix = (prefix << bits) | sh.digit;
    need -= sh.above;
    if (n_cta > 1) cluster_sync();  // the histograms have been read
    else __syncthreads();
  }
  const uint32_t thr = prefix;  // keys above it stay, and the first `need` rows that equal it

  // ---- ties before this warp: counts of equal keys per warp, then over warps and CTAs
  auto cta_prefix = [&](uint32_t mine, uint32_t& total) -> uint32_t {  // all warps; mine: uniform in a warp
    if (lane == 0) sh.warp_sum[warp] = mine;
    __syncthreads();
    uint32_t x = sh.warp_sum[lane];
    const uint32_t s = warp_incl_scan(x, lane);
    total = __shfl_sync(0xffffffffu, s, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, s - x, warp);
    __syncthreads();
    return before;
  };
  uint32_t eq = 0;
  for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
    const int i = i0 + lane;
    eq += __popc(__ballot_sync(0xffffffffu, i < w_hi && key_at(i) == thr));
  }
  uint32_t total;
  uint32_t eq_before = cta_prefix(eq, total);
  if (n_cta > 1) {
    if (tid == 0) sh.total[0] = total;
    cluster_sync();
    for (uint32_t r = 0; r < rank; ++r) eq_before += ld_cluster_u32(cluster_addr(&sh.total[0], r));
    cluster_sync();
  }
  // ---- rows that stay beyond the budget and places freed below it, counted, then written
  uint32_t late = 0, freed = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t e = eq_before;
    uint32_t n_late = late, n_free = freed;  // pass 1: ranks of this warp's first rows
    for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t k = i < w_hi ? key_at(i) : 0;
      const bool is_eq = i < w_hi && k == thr;
      const uint32_t eqs = __ballot_sync(0xffffffffu, is_eq);
      const uint32_t below = (1u << lane) - 1;
      const bool keep = i < w_hi && (k > thr || (is_eq && e + __popc(eqs & below) < need));
      e += __popc(eqs);
      const uint32_t ls = __ballot_sync(0xffffffffu, keep && i >= p.budget);
      const uint32_t fs = __ballot_sync(0xffffffffu, i < w_hi && !keep && i < p.budget);
      if (pass) {
        if ((ls >> lane) & 1u) {
          const uint32_t at = n_late + __popc(ls & below);
          if (at < (uint32_t)p.n_moves) out[at].x = i;
        }
        if ((fs >> lane) & 1u) {
          const uint32_t at = n_free + __popc(fs & below);
          if (at < (uint32_t)p.n_moves) out[at].y = i;
        }
      }
      n_late += __popc(ls);
      n_free += __popc(fs);
    }
    if (pass) break;
    uint32_t t_late, t_free;
    late = cta_prefix(n_late, t_late);
    freed = cta_prefix(n_free, t_free);
    if (n_cta > 1) {
      if (tid == 0) {
        sh.total[0] = t_late;
        sh.total[1] = t_free;
      }
      cluster_sync();
      t_late = 0;
      for (uint32_t r = 0; r < n_cta; ++r) {
        const uint32_t l = ld_cluster_u32(cluster_addr(&sh.total[0], r));
        if (r < rank) {
          late += l;
          freed += ld_cluster_u32(cluster_addr(&sh.total[1], r));
        }
        t_late += l;
      }
      cluster_sync();  // no CTA ends while another reads its counts
    }
    for (int i = t_late + rank * kThreads + tid; i < p.n_moves; i += n_cta * kThreads) out[i] = make_int2(-1, -1);
  }
}

}  // namespace
}  // namespace hcadsa

extern "C" hcadsa_status mla_evict_select(const float* mass, const int32_t* pos, const int32_t* table,
                                          const int32_t* kv_len, const int32_t* seen, int32_t* moves,
                                          int32_t* new_len, int B, int n_pages, int page, int max_pages, int Hkv,
                                          int budget, int n_sink, int n_recent, int n_moves, hcadsa_stream stream) {
  using namespace hcadsa;
  if (B > 0 && (!mass || !pos || !table || !kv_len || (n_moves > 0 && !moves) || !new_len)) return HCADSA_ERR_NULL;
  HCADSA_TRY(check_paged_sizes(B, n_pages, page, max_pages, Hkv));
  const long long cap = (long long)max_pages * page;
  if (budget < 1 || n_sink < 0 || n_recent < 0 || (long long)n_sink + n_recent > budget) return HCADSA_ERR_SHAPE;
  const long long most = cap <= budget ? 0 : (budget < cap - budget ? budget : cap - budget);
  if (n_moves < most) return HCADSA_ERR_SHAPE;
  if (!aligned4(mass) || !aligned4(pos) || !aligned4(table) || !aligned4(kv_len) || !aligned4(seen) ||
      (reinterpret_cast<uintptr_t>(moves) & 7u) || !aligned4(new_len))
    return HCADSA_ERR_ALIGN;
  if (B == 0) return HCADSA_OK;
  int cluster = 1;
  while (cluster < kMaxCluster && cap > (long long)cluster * kSliceTarget) cluster *= 2;
  const long long blocks = (long long)B * Hkv * cluster;
  if (blocks > 2147483647LL) return HCADSA_ERR_UNSUPPORTED;
  const long long slice = ((cap + cluster - 1) / cluster + kThreads - 1) / kThreads * kThreads;
  Params p;
  p.s = paged_batch(table, nullptr, kv_len, B, 0, n_pages, page, max_pages);
  p.mass = mass;
  p.pos = pos;
  p.seen = seen;
  p.moves = reinterpret_cast<int2*>(moves);
  p.new_len = new_len;
  p.Hkv = Hkv;
  p.budget = budget;
  p.n_sink = n_sink;
  p.n_recent = n_recent;
  p.n_moves = n_moves;
  p.smem_rows = slice <= kMaxSmemRows ? (int)slice : 0;
  const size_t smem = (size_t)p.smem_rows * 4;
  if (smem > 32 * 1024 && cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMaxSmemRows * 4) != cudaSuccess)
    return launch_status();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = as_stream(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, select_kernel, p) != cudaSuccess) return launch_status();
  return launch_status();
}
