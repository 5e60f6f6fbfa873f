// mla_evict.cu -- which rows of a paged cache stay when it is cut to a budget (mla_evict_select).
//
// Method: eviction by accumulated attention weight.  A row stays if its position is one of the
// first n_sink or of the last n_recent of its sequence; the rest of the budget goes to the rows
// with the most weight, equal weights to the lower row.  Rows that stay below the budget are not
// touched; the i-th row that stays beyond it moves to the i-th freed place below it, so a cut of
// m rows moves at most m rows, whatever the budget.
//
// One cluster of 2 to 8 CTAs per (sequence, K/V head).  The first CTAs share the rows below the
// budget, the others those beyond it, in contiguous slices, so every CTA counts either freed places
// or rows that move.
//   * Weights become 32-bit keys whose order is that of the weights (protected rows on top) and stay
//     in shared memory.  The budget-th largest key is found with a radix select of 11, 11 and 10
//     bits: a histogram per CTA and pass, read by all CTAs of the cluster through distributed shared
//     memory, so all follow the same bin, with one cluster barrier per pass.
//   * The same histograms say how many rows of every CTA lie above the threshold and how many equal
//     it.  Ties are taken in row order: from those counts, and counts per warp (a warp owns a
//     contiguous run of its CTA's slice), every row knows its rank.  No atomics decide anything that
//     is written: the result does not depend on timing.
// What bounds it is latency: two dependent loads per row, three passes over the keys, four cluster
// barriers.  A thread takes four consecutive rows at a time (a page holds at least 16).  Slices that
// do not fit in shared memory are read from global memory again in every pass.
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
  int smem_rows;  // rows of a slice that fit the dynamic shared memory
  bool vec;       // four rows are 16 aligned bytes of mass and pos
};

struct Shared {
  uint32_t hist[3][kBins];       // this CTA's counts of each pass (read by the cluster)
  uint32_t warp_sum[32];
  uint32_t digit, above;         // the bin of a pass, and the rows above it, found by one thread
  uint32_t gt[kMaxCluster];      // rows above the threshold, by CTA
  uint32_t eq[kMaxCluster];      // rows that equal it
  uint32_t warp_gt[32], warp_eq[32];
};

// Keys in the order of the weights: protected rows over everything, NaN over +inf, -0 equal to 0.  No
// key is 0, which stands for a row that is not there.
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
  extern __shared__ uint4 keys[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t n_cta_;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n_cta_));
  const int n_cta = (int)n_cta_, rank = (int)cluster_rank();
  const int list = blockIdx.x / n_cta;
  const int b = list / p.Hkv, h = list - b * p.Hkv;
  const int budget = p.budget;
  const int len = paged_len(p.s, b, h == 0 && rank == 0 && tid == 0);
  int2* out = p.moves + (size_t)list * p.n_moves;
  if (h == 0 && rank == 0 && tid == 0) p.new_len[b] = min(len, budget);
  if (len <= budget) {  // nothing to evict
    for (int i = rank * kThreads + tid; i < p.n_moves; i += n_cta * kThreads) out[i] = make_int2(-1, -1);
    return;
  }
  // CTAs [0, c1) share the rows [0, budget), the others [budget, len); slices start at multiples of 4
  // from the start of their side, the second side's start rounded down (row_of).
  int c1 = (int)(((long long)n_cta * budget + len / 2) / len);
  c1 = c1 < 1 ? 1 : (c1 > n_cta - 1 ? n_cta - 1 : c1);
  const int a0 = budget & ~3;
  const int per1 = ((budget + c1 - 1) / c1 + 3) & ~3, per2 = ((len - a0 + n_cta - c1 - 1) / (n_cta - c1) + 3) & ~3;
  auto slice = [&](int r, int& start, int& lo, int& hi) {  // start: multiple of 4; rows [lo, hi)
    start = r < c1 ? r * per1 : a0 + (r - c1) * per2;
    lo = r < c1 ? min(start, budget) : min(max(start, budget), len);
    hi = r < c1 ? min(start + per1, budget) : min(start + per2, len);
    if (hi < lo) hi = lo;
  };
  int start, lo, hi;
  slice(rank, start, lo, hi);
  const bool late_side = rank >= c1;
  const int quads = hi > lo ? (hi - start + 3) / 4 : 0;  // groups of four rows of this CTA
  const bool in_smem = 4 * quads <= p.smem_rows;
  const long long seen = p.seen ? p.seen[b] : len;
  const int page_mask = (1 << p.s.page_log2) - 1;

  // four keys from four consecutive rows of page pg (-1: recorded as bad; its rows count as weightless)
  auto load_keys = [&](int q, int pg) -> uint4 {
    const int i = start + 4 * q;
    uint32_t k[4];
    float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int ps[4];
    const bool ok = pg >= 0;
    if (ok) {
      const size_t slot = (((size_t)pg << p.s.page_log2) + (i & page_mask)) * p.Hkv + h;
      if (p.vec) {
        const float4 m4 = *reinterpret_cast<const float4*>(p.mass + slot);
        const int4 p4 = *reinterpret_cast<const int4*>(p.pos + slot);
        m[0] = m4.x, m[1] = m4.y, m[2] = m4.z, m[3] = m4.w;
        ps[0] = p4.x, ps[1] = p4.y, ps[2] = p4.z, ps[3] = p4.w;
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          m[x] = p.mass[slot + (size_t)x * p.Hkv];
          ps[x] = p.pos[slot + (size_t)x * p.Hkv];
        }
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
      k[x] = i + x < lo || i + x >= hi ? 0u : key_of(m[x], ok && (ps[x] < p.n_sink || ps[x] >= seen - p.n_recent));
    return make_uint4(k[0], k[1], k[2], k[3]);
  };
  auto page_at = [&](int q) { return paged_page(p.s, b, start + 4 * q); };
  if (in_smem) {
    constexpr int kAhead = 4;  // page lookups, then row loads, in flight per thread
    for (int q0 = tid; q0 < quads; q0 += kAhead * kThreads) {
      int pg[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) pg[x] = q0 + x * kThreads < quads ? page_at(q0 + x * kThreads) : -1;
      uint4 k[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x)
        if (q0 + x * kThreads < quads) k[x] = load_keys(q0 + x * kThreads, pg[x]);
#pragma unroll
      for (int x = 0; x < kAhead; ++x)
        if (q0 + x * kThreads < quads) keys[q0 + x * kThreads] = k[x];
    }
  }
  auto keys_at = [&](int q) -> uint4 { return in_smem ? keys[q] : load_keys(q, page_at(q)); };
  for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
  if (tid < kMaxCluster) sh.gt[tid] = sh.eq[tid] = 0;
  __syncthreads();

  // ---- the budget-th largest key: `prefix` holds its bits found so far, `need` its rank among
  // the rows that share them
  uint32_t prefix = 0, need = (uint32_t)budget;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bits = pass == 2 ? 10 : 11;
    const uint32_t mask = (1u << bits) - 1;
    uint32_t* hist = sh.hist[pass];
    for (int q0 = tid & ~31; q0 < quads; q0 += kThreads) {
      const int q = q0 + lane;
      const uint4 k4 = q < quads ? keys_at(q) : make_uint4(0, 0, 0, 0);
      const uint32_t kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bool in = kk[x] != 0 && (pass == 0 || (kk[x] >> (shift + bits)) == prefix);
        const uint32_t d = (kk[x] >> shift) & mask;
        // rows of one bin in a whole warp (protected runs, ties) cost one atomic instead of 32
        const uint32_t live = __ballot_sync(0xffffffffu, in);
        if (!live) continue;
        const uint32_t d0 = __shfl_sync(0xffffffffu, d, __ffs(live) - 1);
        if (__all_sync(0xffffffffu, !in || d == d0)) {
          if (lane == 0) atomicAdd(&hist[d0], __popc(live));
        } else if (in) {
          atomicAdd(&hist[d], 1u);
        }
      }
    }
    __syncthreads();
    cluster_sync();
    // bins from the top: thread t holds bins 2047 - 2t and 2046 - 2t, of every CTA
    uint32_t c0[kMaxCluster], c1_[kMaxCluster], s0 = 0, s1 = 0;
    const int bin0 = kBins - 1 - 2 * tid;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      c0[r] = c1_[r] = 0;
      if (r < n_cta) {
        const uint32_t a = cluster_addr(&hist[bin0 - 1], r);
        c1_[r] = ld_cluster_u32(a);
        c0[r] = ld_cluster_u32(a + 4);
      }
    }
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) s0 += c0[r], s1 += c1_[r];
    const uint32_t incl = warp_incl_scan(s0 + s1, lane);
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    const uint32_t sums = sh.warp_sum[lane];
    const uint32_t sums_incl = warp_incl_scan(sums, lane);
    const uint32_t upto = incl + __shfl_sync(0xffffffffu, sums_incl - sums, warp), before = upto - s0 - s1;
    if (before < need && need <= upto) {
      const bool first = need <= before + s0;
      sh.digit = (uint32_t)(first ? bin0 : bin0 - 1);
      sh.above = before + (first ? 0 : s0);
    }
    __syncthreads();
    const int digit = (int)sh.digit;
    prefix = (prefix << bits) | (uint32_t)digit;
    need -= sh.above;
    // per CTA: its rows above the bin, and in the last pass those in it
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      if (r >= n_cta) break;
      const uint32_t g = __reduce_add_sync(0xffffffffu, (bin0 > digit ? c0[r] : 0) + (bin0 - 1 > digit ? c1_[r] : 0));
      if (lane == 0 && g) atomicAdd(&sh.gt[r], g);
      if (pass == 2) {
        if (bin0 == digit) sh.eq[r] = c0[r];
        else if (bin0 - 1 == digit) sh.eq[r] = c1_[r];
      }
    }
  }
  const uint32_t thr = prefix;  // keys above it stay, and the first `need` rows that equal it
  // ---- counts per warp: warp w owns the groups [w * per_warp, ...) of the CTA
  const int per_warp = ((quads + 31) / 32 + 31) / 32 * 32;
  const int w_lo = min(quads, warp * per_warp), w_hi = min(quads, w_lo + per_warp);
  uint32_t n_gt = 0, n_eq = 0;
  for (int q0 = w_lo; q0 < w_hi; q0 += 32) {
    const int q = q0 + lane;
    const uint4 k4 = q < w_hi ? keys_at(q) : make_uint4(0, 0, 0, 0);
    n_gt += (k4.x > thr) + (k4.y > thr) + (k4.z > thr) + (k4.w > thr);
    n_eq += (k4.x == thr) + (k4.y == thr) + (k4.z == thr) + (k4.w == thr);
  }
  n_gt = __reduce_add_sync(0xffffffffu, n_gt);
  n_eq = __reduce_add_sync(0xffffffffu, n_eq);
  if (lane == 0) {
    sh.warp_gt[warp] = n_gt;
    sh.warp_eq[warp] = n_eq;
  }
  __syncthreads();
  // ---- ranks: entries and ties before this CTA, then before this warp
  uint32_t before_cta = 0, eq_run = 0, at = 0, total = 0;
  for (int r = 0; r < n_cta; ++r) {
    int s_, l_, h_;
    slice(r, s_, l_, h_);
    const uint32_t kept = sh.gt[r] + min(need, eq_run + sh.eq[r]) - min(need, eq_run);
    const uint32_t entries = r >= c1 ? kept : (uint32_t)(h_ - l_) - kept;
    if (r >= c1) total += entries;
    if (r < rank && (r >= c1) == late_side) at += entries;
    if (r == rank) before_cta = eq_run;
    eq_run += sh.eq[r];
  }
  {
    const uint32_t g = sh.warp_gt[lane], e = sh.warp_eq[lane];
    const uint32_t g_before = __shfl_sync(0xffffffffu, warp_incl_scan(g, lane) - g, warp);
    const uint32_t e_before = before_cta + __shfl_sync(0xffffffffu, warp_incl_scan(e, lane) - e, warp);
    const uint32_t taken = min(need, e_before) - min(need, before_cta);
    uint32_t kept = g_before + taken;  // staying rows of this CTA before the position reached
    uint32_t ties = e_before;          // rows that equal the threshold before it, over the whole list
    int32_t* dst = reinterpret_cast<int32_t*>(out) + (late_side ? 0 : 1);
    for (int q0 = w_lo; q0 < w_hi; q0 += 32) {
      const int q = q0 + lane;
      const uint4 k4 = q < w_hi ? keys_at(q) : make_uint4(0, 0, 0, 0);
      const uint32_t kk[4] = {k4.x, k4.y, k4.z, k4.w};
      uint32_t mine = 0;  // rows above the threshold, and from bit 16 on those that equal it
#pragma unroll
      for (int x = 0; x < 4; ++x) mine += (kk[x] > thr ? 1u : 0u) + (kk[x] == thr ? 0x10000u : 0u);
      const uint32_t incl = warp_incl_scan(mine, lane), excl = incl - mine;
      uint32_t e = ties + (excl >> 16);
      uint32_t k = kept + (excl & 0xffffu) + min(need, e) - min(need, ties);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = start + 4 * q + x;
        const bool is_eq = kk[x] == thr, keep = kk[x] > thr || (is_eq && e < need);
        const uint32_t entry = at + (late_side ? k : (uint32_t)(i - lo) - k);
        if (kk[x] != 0 && keep == late_side && entry < (uint32_t)p.n_moves) dst[2 * (size_t)entry] = i;
        e += is_eq;
        k += keep;
      }
      const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
      kept += (all & 0xffffu) + min(need, ties + (all >> 16)) - min(need, ties);
      ties += all >> 16;
    }
  }
  for (int i = (int)total + rank * kThreads + tid; i < p.n_moves; i += n_cta * kThreads) out[i] = make_int2(-1, -1);
  cluster_sync();  // no CTA ends while another reads its histograms
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
  int cluster = 2;
  while (cluster < kMaxCluster && cap > (long long)cluster * kSliceTarget) cluster *= 2;
  const long long blocks = (long long)B * Hkv * cluster;
  if (blocks > 2147483647LL) return HCADSA_ERR_UNSUPPORTED;
  // a side's share of the CTAs is rounded, so a slice may be half as long again as the average
  const long long slice = (cap * 3 / 2 / cluster + 64 + 3) / 4 * 4;
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
  p.smem_rows = (int)(slice < kMaxSmemRows ? slice : kMaxSmemRows);
  p.vec = Hkv == 1 && aligned16(mass) && aligned16(pos);
  const size_t smem = (size_t)p.smem_rows * 4;
  if (smem > 16 * 1024 && cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
