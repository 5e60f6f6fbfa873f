// mla_evict.cu -- which rows of a paged cache stay when it is cut to a budget (mla_evict_select).
//
// Method: eviction by accumulated attention weight.  A row stays if its position is one of the
// first n_sink or of the last n_recent of its sequence; the rest of the budget goes to the rows
// with the most weight, equal weights to the lower row.  Rows that stay below the budget are not
// touched; the i-th row that stays beyond it moves to the i-th freed place below it, so a cut of
// m rows moves at most m rows, whatever the budget.
//
// One cluster of 2 to 16 CTAs per (sequence, K/V head).  The first CTAs share the rows below the
// budget, the others those beyond it, in contiguous slices, so every CTA counts either freed places
// or rows that move.
//   * Weights become 32-bit keys whose order is that of the weights (protected rows on top) and stay
//     in shared memory.  The budget-th largest key is found with a radix select of 11, 11 and 10
//     bits: a histogram per CTA and pass, with one cluster barrier per pass.  One warp of every CTA
//     then reads, through distributed shared memory, 64 sums of 32 bins from each CTA, and the 32
//     bins of the group that holds the rank: all CTAs follow the same bin.  The loops run to the largest
//     cluster of the variant, so a pass reads 8 x 96 words (16 x 96 for clusters of 16) per CTA instead of
//     whole histograms (8 x 2048 words took 9000 cycles).
//   * Ties at the threshold are taken in row order: from counts per warp (a warp owns a contiguous run
//     of its CTA's slice) and per CTA every row knows its rank.  No atomics decide anything that is
//     written: the result does not depend on timing.
//   * Entries are gathered in shared memory, 128 rows of a warp at a time, and written side by side.
// What bounds it is latency: two dependent loads per row, three passes over the keys with a
// cluster barrier each, and two more for the counts and the end.  A thread takes four consecutive rows at a time (a page holds at least 16).  Slices that
// do not fit in shared memory are read from global memory again in every pass.
// Measured (B200): 32 lists of 4224 rows cut to 4096 in 12.4 us, 4 lists of 131072 cut to 32768 in 23.
#include <mutex>

#include "mla_host.h"
#include "pair.cuh"

namespace hcadsa {
namespace {

constexpr int kBins = 2048;
constexpr int kPortable = 8, kLargest = 16;  // CTAs of a cluster
constexpr int kGroupBins = 32, kBinGroups = kBins / kGroupBins;
constexpr int kMaxSmemRows = 44 * 1024;
constexpr uint32_t kSafe = 0xffffffffu;  // the key of a protected row

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

template <int kWarps>
struct Shared {
  uint32_t hist[3][kBins];        // this CTA's counts of each pass (read by the cluster)
  uint32_t group[3][kBinGroups];  // and of every 32 bins (read by the cluster)
  uint32_t protected_rows;        // (read by the cluster)
  uint32_t total[2];              // rows above the threshold, rows that equal it (read by the cluster)
  uint32_t digit, need;           // the bin of a pass, and the rank left among its rows
  uint32_t warp_gt[kWarps], warp_eq[kWarps];
  int32_t entry[kWarps][128];     // a warp's next entries of the list
};

// Keys in the order of the weights: protected rows over everything, NaN over +inf, -0 equal to 0.  No
// key is 0, which stands for a row that is not there.
__device__ __forceinline__ uint32_t key_of(float m, bool safe) {
  if (safe) return kSafe;
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

template <int kThreads, int kMaxCluster>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 4 : 1) select_kernel(const Params p) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint4 keys[];
  __shared__ Shared<kWarps> sh;
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
  // from the start of their side, the second side's start rounded down.
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
  if (tid == 0) sh.protected_rows = 0;
  __syncthreads();

  // ---- the budget-th largest key: `prefix` holds its bits found so far, `need` its rank among the
  // rows that share them.  Protected rows, which come in runs, are counted without the histogram.
  uint32_t prefix = 0, need = (uint32_t)budget;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bits = pass == 2 ? 10 : 11;
    uint32_t* hist = sh.hist[pass];
    uint32_t safe = 0;
    for (int q = tid; q < quads; q += kThreads) {
      const uint4 k4 = keys_at(q);
      const uint32_t kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (pass == 0) {
          if (kk[x] == kSafe) ++safe;
          else if (kk[x] != 0) atomicAdd(&hist[kk[x] >> 21], 1u);
        } else if ((kk[x] >> (shift + bits)) == prefix && kk[x] != kSafe) {
          atomicAdd(&hist[(kk[x] >> shift) & ((1u << bits) - 1)], 1u);
        }
      }
    }
    if (pass == 0) {
      safe = __reduce_add_sync(0xffffffffu, safe);
      if (lane == 0) atomicAdd(&sh.protected_rows, safe);
    }
    __syncthreads();
    for (int g = warp; g < kBinGroups; g += kWarps) {
      const uint32_t sum = __reduce_add_sync(0xffffffffu, hist[g * kGroupBins + lane]);
      if (lane == 0) sh.group[pass][g] = sum;
    }
    __syncthreads();
    cluster_sync();
    if (warp == 0) {
      if (pass == 0) {
        const uint32_t mine = ld_cluster_u32(cluster_addr(&sh.protected_rows, lane < n_cta ? lane : rank));
        const uint32_t all = __reduce_add_sync(0xffffffffu, lane < n_cta ? mine : 0);
        need = all < need ? need - all : 0;  // 0: the budget goes to protected rows alone
      }
      // from the top: lane l holds the groups 63 - 2 l and 62 - 2 l, then the bin 31 - l of the group that
      // holds the rank (unconditional loads from every CTA, all in flight at once)
      const int g0 = kBinGroups - 1 - 2 * lane;
      uint32_t s0 = 0, s1 = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        const uint32_t a = cluster_addr(&sh.group[pass][g0 - 1], r < n_cta ? r : rank);
        const uint32_t c_lo = ld_cluster_u32(a), c_hi = ld_cluster_u32(a + 4);
        s1 += r < n_cta ? c_lo : 0;
        s0 += r < n_cta ? c_hi : 0;
      }
      const uint32_t upto = warp_incl_scan(s0 + s1, lane), before = upto - s0 - s1;
      const int at = __ffs(__ballot_sync(0xffffffffu, upto >= need)) - 1;  // the lane of the rank's group
      const bool first = need <= before + s0;
      const uint32_t above0 = __shfl_sync(0xffffffffu, before + (first ? 0 : s0), at);
      const int group = __shfl_sync(0xffffffffu, first ? g0 : g0 - 1, at);
      uint32_t sum = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        const uint32_t c = ld_cluster_u32(cluster_addr(&hist[group * kGroupBins + 31 - lane], r < n_cta ? r : rank));
        sum += r < n_cta ? c : 0;
      }
      const uint32_t incl = above0 + warp_incl_scan(sum, lane);
      const int in_group = __ffs(__ballot_sync(0xffffffffu, incl >= need)) - 1;
      const uint32_t above = __shfl_sync(0xffffffffu, incl - sum, in_group);
      if (lane == 0) {
        sh.digit = (uint32_t)(group * kGroupBins + 31 - in_group);
        sh.need = need - (need ? above : 0);
      }
    }
    __syncthreads();
    prefix = (prefix << bits) | sh.digit;
    need = sh.need;
    if (need == 0) break;  // (in the first pass only: every later rank is at least 1)
  }
  if (need == 0) {
    prefix = kSafe;
    need = (uint32_t)budget;
  }
  const uint32_t thr = prefix;  // keys above it stay, and the first `need` rows that equal it
  // ---- counts per warp: warp w owns the groups [w * per_warp, ...) of the CTA
  const int per_warp = ((quads + kWarps - 1) / kWarps + 31) / 32 * 32;
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
  if (warp == 0) {
    const uint32_t g = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.warp_gt[lane] : 0);
    const uint32_t e = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.warp_eq[lane] : 0);
    if (lane == 0) {
      sh.total[0] = g;
      sh.total[1] = e;
    }
  }
  __syncthreads();
  cluster_sync();
  // ---- ranks: entries and ties before this CTA (lane r reads CTA r's counts), then before this warp
  uint32_t before_cta, at, total;
  {
    const int r = lane < n_cta ? lane : rank;
    const uint32_t a = cluster_addr(&sh.total[0], r);
    const uint32_t g = lane < n_cta ? ld_cluster_u32(a) : 0, e = lane < n_cta ? ld_cluster_u32(a + 4) : 0;
    const uint32_t e_to = warp_incl_scan(e, lane), e_from = e_to - e;
    const uint32_t kept = g + min(need, e_to) - min(need, e_from);
    int s_, l_, h_;
    slice(r, s_, l_, h_);
    const uint32_t entries = lane >= n_cta ? 0 : (lane >= c1 ? kept : (uint32_t)(h_ - l_) - kept);
    before_cta = __shfl_sync(0xffffffffu, e_from, rank);
    at = __reduce_add_sync(0xffffffffu, lane < rank && (lane >= c1) == late_side ? entries : 0);
    total = __reduce_add_sync(0xffffffffu, lane >= c1 ? entries : 0);
  }
  {
    const uint32_t g = lane < kWarps ? sh.warp_gt[lane] : 0, e = lane < kWarps ? sh.warp_eq[lane] : 0;
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
      // entries before this step of the warp: staying rows, or freed places
      const int row0 = max(start + 4 * q0, lo);
      const uint32_t first = late_side ? kept : (uint32_t)(row0 - lo) - kept;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = start + 4 * q + x;
        const bool is_eq = kk[x] == thr, keep = kk[x] > thr || (is_eq && e < need);
        if (kk[x] != 0 && keep == late_side) sh.entry[warp][(late_side ? k : (uint32_t)(i - lo) - k) - first] = i;
        e += is_eq;
        k += keep;
      }
      const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
      kept += (all & 0xffffu) + min(need, ties + (all >> 16)) - min(need, ties);
      ties += all >> 16;
      const int row1 = min(start + 4 * q0 + 128, hi);
      const uint32_t n = (late_side ? kept : (uint32_t)(row1 - lo) - kept) - first;
      __syncwarp();
      for (uint32_t o = lane; o < n; o += 32)
        if (at + first + o < (uint32_t)p.n_moves) dst[2 * (size_t)(at + first + o)] = sh.entry[warp][o];
      __syncwarp();
    }
  }
  for (int i = (int)total + rank * kThreads + tid; i < p.n_moves; i += n_cta * kThreads) out[i] = make_int2(-1, -1);
  cluster_sync();  // no CTA ends while another reads its histograms
}

// The current device: its SMs, and how many clusters of 16 CTAs run on it at once.
struct Device {
  int sms, large;
};

template <int kThreads, int kMaxCluster>
bool set_up() {
  return cudaFuncSetAttribute(select_kernel<kThreads, kMaxCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kMaxSmemRows * 4) == cudaSuccess &&
         (kMaxCluster <= kPortable ||
          cudaFuncSetAttribute(select_kernel<kThreads, kMaxCluster>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                               1) == cudaSuccess);
}

// `attr` has to live as long as the configuration.
cudaLaunchConfig_t config_of(unsigned blocks, int cluster, int threads, size_t smem, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = cluster;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// The kernels' attributes are set on the first call.
Device this_device() {
  static std::mutex mu;
  static Device cache[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return {};
  std::lock_guard<std::mutex> lock(mu);
  if (!cache[dev].sms) {
    int sms = 0, large = 0;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config_of(kLargest, kLargest, 1024, kMaxSmemRows * 4, &attr);
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        !set_up<256, kPortable>() || !set_up<512, kPortable>() || !set_up<1024, kPortable>() ||
        !set_up<512, kLargest>() || !set_up<1024, kLargest>() ||
        cudaOccupancyMaxActiveClusters(&large, select_kernel<1024, kLargest>, &cfg) != cudaSuccess) {
      launch_status();
      return {};
    }
    cache[dev] = {sms, large};
  }
  return cache[dev];
}

// A list of 4096 rows takes 12.4 us on four CTAs and 18.5 on two (32 lists at once); CTAs beyond one
// per SM would wait for the first (35 us on eight), so beyond that a CTA gets 4096 rows (80 lists of 32768
// rows of 8 K/V heads 77 us, 119 on two CTAs each).  Long lists go to 16 CTAs, as many as find room
// for all of them at once: 131072 rows 23.4 us against 26.7 on eight, 65536 rows 18.8 against 20.5 (7
// lists; 8 lists, for which there is no room, 35.4), but 32768 rows 17.9 against 16.4.
// The host knows the table's width and not the lengths, so `cap` is the former: 32 lists of 4224 rows in a
// table for 32768 rows take as long as in one that just fits (12.6 and 11.0 us, replayed), in one for 131072
// rows they get eight CTAs of 1024 threads each, twice what the SMs hold at once, and take 38 us.
int cluster_of(long long lists, long long cap, const Device& dev) {
  if (cap >= 65536 && lists <= dev.large) return kLargest;
  int cluster = 2;
  while (cluster < kPortable && cap > 1024LL * cluster &&
         (2 * cluster * lists <= dev.sms || cap > 4096LL * cluster))
    cluster *= 2;
  return cluster;
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
  // new_len is written by one CTA of a sequence while others still read its lengths
  const auto overlap = [&](const int32_t* x) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), n = reinterpret_cast<uintptr_t>(new_len);
    return x && (a < n ? n - a : a - n) < 4 * (uintptr_t)B;
  };
  if (overlap(kv_len) || overlap(seen)) return HCADSA_ERR_SHAPE;
  if (B == 0) return HCADSA_OK;
  const Device dev = this_device();
  if (dev.sms <= 0) return HCADSA_ERR_CUDA;
  const int cluster = cluster_of((long long)B * Hkv, cap, dev);
  const long long blocks = (long long)B * Hkv * cluster;
  if (blocks > 2147483647LL) return HCADSA_ERR_UNSUPPORTED;
  // a side's share of the CTAs is rounded, so a slice may be half as long again as the average, and of two
  // CTAs one may get nearly all (80 lists of 32768 rows, cut to 4096 on two CTAs each and
  // read again in every pass, took 334 us instead of 119)
  const long long slice = ((cluster == 2 ? cap : cap * 3 / 2 / cluster) + 64 + 3) / 4 * 4;
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
  // rows per CTA and list: 4096, 512 threads 12.4 us, 1024 threads 14.4; 8192, 23.4 and 24.6; 16384,
  // 28.7 and 26.8.  More CTAs than SMs: blocks of 256 threads, four to an SM (256 lists of 2048 rows 19.5 us
  // against 45 with 512 threads).
  const bool wide = cap > 8192LL * cluster, many = blocks > dev.sms;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = config_of((unsigned)blocks, cluster, wide ? 1024 : many ? 256 : 512, smem, &attr);
  cfg.stream = as_stream(stream);
  void (*kernel)(Params);
  if (cluster > kPortable) kernel = wide ? select_kernel<1024, kLargest> : select_kernel<512, kLargest>;
  else if (many && !wide) kernel = select_kernel<256, kPortable>;
  else kernel = wide ? select_kernel<1024, kPortable> : select_kernel<512, kPortable>;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return launch_status();
  return launch_status();
}
