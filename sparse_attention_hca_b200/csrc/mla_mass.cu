// mla_mass.cu -- the attention weight that every row of the paged cache of the full-context
// (MLA) layers received from a chunk of new tokens (mla_paged_attn_mass), on sm_100a.
//
// Method: eviction keeps the rows that queries attended to, so each row accumulates
//     mass[s] += sum over the chunk's tokens t that see s, and the query heads of the K/V head,
//                of exp(scale <q[t], k_s> - lse[t])
// with the log-sum-exp of the attention call.
//
// Tiles: keys are the M of the products.  A CTA pair holds a block of 256 cache rows (CTA r the rows
// 128 r .. +127, its TMEM lanes) and streams the chunk's (token, head) rows past them, 128 per tile
// (64 loaded by each CTA): S^T = K (A) * Q^T (B), tcgen05 cta_group::2, M = 256, N = 128.  A thread
// owns a cache row and sums exp2 over its TMEM lane's 128 columns, so the sum over tokens and heads
// needs no exchange between threads, but one at the end of a block, and no atomics.  Four S buffers
// (all of TMEM), one warpgroup for each: a TMEM load takes about 600 cycles next to the MMAs, and
// four warps per scheduler hide it.  The sums are fp32, over the tiles with Kahan's compensation.
// A decode step has few rows per sequence: the same Q tile stays in its slot from one block of cache
// rows to the next, and the kernel streams K.
//
// Schedule: as the attention kernel's, one list of (256-row block, 128-row Q tile) products over the
// batch -- sequence, K/V head, block, Q tile, those that see some row of the block -- cut evenly over
// the pairs (see kBlockCost).  A block that several pairs share leaves partial sums in the workspace, which
// add_kernel adds up in list order; every row's mass gets exactly one addition per call.
//
// Measured (B200, 64 heads on one K/V head): 1021 tokens over 16381 rows 380 us in a short run (1.40
// PFLOP/s), 446 us when repeated (power limit); the MMAs and loads alone, without the sums, take 313.
// Products of 256 columns (two S buffers) took 412 us, K held in TMEM as the A operand 417.  A decode
// step of 32 sequences of 1K-32K rows: 55 us for the kernel (5.2 TB/s), 61 with zeroing and adding up.
#include <mutex>

#include "mla_host.h"
#include "pair.cuh"

namespace hcadsa {
namespace {

constexpr int kKeys = 256;                  // cache rows of a block (128 per CTA)
constexpr int kCols = 128;                  // (token, head) rows of a Q tile (64 loaded per CTA)
constexpr int kKBytes = 64 * 1024;
constexpr int kQSlots = 3, kQBytes = 32 * 1024, kQChunk = 8 * 1024;
constexpr int kSmemBytes = 2 * kKBytes + kQSlots * kQBytes;
constexpr int kGroups = 4;                  // warpgroups that sum, one per S buffer
constexpr int kThreads = 128 + 128 * kGroups;  // warp 0 TMA, warp 1 MMA, warps 4-19 sums
constexpr int kMetaInts = 8;
constexpr int kMaxPairs = 80;

struct Params {
  PagedBatch s;
  const float* lse;
  float* mass;
  float* ws_sum;  // [2 G][256]: pair c's block that began before its range (2 c) or in it (2 c + 1)
  int* ws_meta;   // [G][kMetaInts]
  int Hq, Hkv, g_log2;
  int box_log2, k_group, k_chunk;  // K rows of a box; bytes from 8 rows to the next, from 64 columns to the next
  float scale_log2;
};

struct __align__(8) Barriers {
  uint64_t k_full[2], k_empty[2];
  uint64_t q_full[kQSlots], q_empty[kQSlots];
  uint64_t s_full[kGroups], s_empty[kGroups];
  uint64_t sum_ready, sum_free;
};

// ------------------------------------------------------------------ the list of products

// A block's K tile takes as long to arrive as about one more product, so a block takes one place in the
// list besides its products; the place comes first.  (3 chunks of 435 tokens over 1.3K-4.8K rows next to 22
// single tokens, whose blocks are one product each: 113 us against 153; two of 433 next to 21, 128 heads,
// 55 against 73.)
constexpr int kBlockCost = 1;

// One sequence's part of the list (of one K/V head).
struct SeqBlocks {
  int base, n, len, s_log2;  // s_log2: tokens of a Q tile
  __host__ __device__ int q_tiles() const { return n > 0 ? ((n - 1) >> s_log2) + 1 : 0; }
  __host__ __device__ int blocks() const { return n > 0 ? (len + kKeys - 1) / kKeys : 0; }
  // the first Q tile with a token that sees row 256 k: token 256 k - base, if that is not before 0
  __host__ __device__ int first_tile(int k) const {
    const int t = k * kKeys - base;
    return t <= 0 ? 0 : t >> s_log2;
  }
  // products of the blocks before k: the first kf blocks take every Q tile, and from there on the first
  // tile grows by 256 / tokens per block
  __host__ __device__ long long before(int k) const {
    const int kf = base < 0 ? 0 : base / kKeys + 1;
    const long long q = q_tiles();
    if (k <= kf) return k * q;
    const long long cb = (base + (1 << s_log2) - 1) >> s_log2;  // ceil(base / tokens)
    const long long c = k - kf, sum = ((long long)kf + k - 1) * c / 2;
    return kf * q + c * (q + cb) - (sum << (8 - s_log2));
  }
  // where block k begins in the list
  __host__ __device__ long long start(int k) const { return before(k) + (long long)k * kBlockCost; }
  __host__ __device__ int find(long long w) const {
    int lo = 0, hi = blocks();
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start(mid) <= w) lo = mid;
      else hi = mid;
    }
    return lo;
  }
};

struct Start {
  long long count;
  int b, h, k, at;  // where it begins: `at` places into block k
  PagedSeq q;  // sequence b
};

// Walks a pair's pieces: runs of Q tiles against one block.
struct Walk {
  const Params& p;
  long long left;
  int b, h, k, at, t0, t1, first, last;  // Q tiles [t0, t1) of the block's [first, last)
  PagedSeq q;
  SeqBlocks s;
  __device__ Walk(const Params& p_, const Start& st) : p(p_) {
    left = st.count;
    b = st.b;
    h = st.h;
    k = st.k;
    if (left > 0) {
      load(st.q);
      cut(st.at);
    }
  }
  __device__ bool done() const { return left <= 0; }
  __device__ bool whole() const { return t0 == first && t1 == last; }
  // whether the product after this piece's last one uses the same Q tile
  __device__ bool same_tile_next() const {
    return left - places() > kBlockCost && t1 == last && k + 1 < s.blocks() && s.first_tile(k + 1) == last - 1;
  }
  __device__ void next() {
    left -= places();
    if (left <= 0) return;
    if (++k == s.blocks()) {
      k = 0;
      if (++h == p.Hkv) {
        h = 0;
        do {
          if (++b >= p.s.B) {  // cannot happen unless the lengths change under the kernel
            left = 0;
            return;
          }
          load(paged_seq(p.s, b, false));
        } while (s.blocks() == 0);
      }
    }
    cut(0);
  }

 private:
  __device__ void load(const PagedSeq& seq) {
    q = seq;
    s.base = q.base;
    s.n = q.n;
    s.len = q.len;
    s.s_log2 = 7 - p.g_log2;
  }
  __device__ int places() const { return t1 - first + kBlockCost - at; }  // this piece's part of the share
  __device__ void cut(int from) {  // places [0, kBlockCost) of a block hold no product
    at = from;
    first = s.first_tile(k);
    last = s.q_tiles();
    t0 = first + (at > kBlockCost ? at - kBlockCost : 0);
    const long long e = first + at + left - kBlockCost;
    t1 = e < last ? (int)e : last;
    if (t1 <= t0) left = 0;  // the share ends before the block's first product
  }
};

// Every thread of the CTA: this pair's share of the list.
__device__ __forceinline__ void find_start(const Params& p, int worker, int n_workers, Start* out) {
  __shared__ long long sums[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto blocks_of = [&](const PagedSeq& q) -> SeqBlocks {
    SeqBlocks s;
    s.base = q.base;
    s.n = q.n;
    s.len = q.len;
    s.s_log2 = 7 - p.g_log2;
    return s;
  };
  auto work_of = [&](int b, bool report) -> long long {
    if (b >= p.s.B) return 0;
    const SeqBlocks s = blocks_of(paged_seq(p.s, b, report));
    return s.start(s.blocks()) * p.Hkv;
  };
  auto scan = [&](long long x, long long& total) -> long long {  // inclusive prefix over the threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    long long before = 0;
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    __syncthreads();
    return before + x;
  };
  long long mine = 0, all;
  for (int b = tid; b < p.s.B; b += kThreads) mine += work_of(b, blockIdx.x == 0);
  const long long mine_to = scan(mine, all);
  const int n = all < n_workers ? (int)all : n_workers;
  const long long lo = worker < n ? all * worker / n : 0, hi = worker < n ? all * (worker + 1) / n : 0;
  if (tid == 0) out->count = hi - lo;
  if (hi <= lo) return;
  auto find = [&](int b, long long from, long long upto) {  // sequence b's products are [from, upto)
    if (lo < from || lo >= upto) return;
    out->q = paged_seq(p.s, b, false);
    const SeqBlocks s = blocks_of(out->q);
    const long long per_head = (upto - from) / p.Hkv, r = lo - from;
    out->b = b;
    out->h = (int)(r / per_head);
    const long long in = r - out->h * per_head;
    out->k = s.find(in);
    out->at = (int)(in - s.start(out->k));
  };
  if (p.s.B <= kThreads) {  // known from the first pass
    find(tid, mine_to - mine, mine_to);
    return;
  }
  long long done = 0;
  for (int b0 = 0; b0 < p.s.B && done <= lo; b0 += kThreads) {
    long long total;
    const long long w = work_of(b0 + tid, false), upto = done + scan(w, total);
    find(b0 + tid, upto - w, upto);
    done += total;
  }
}

// ------------------------------------------------------------------ the kernel

__device__ __forceinline__ void group_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mass_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Barriers bar;
  __shared__ Start start;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  // by warpgroup: a tile's lse in log2 units, negated; at the end of a piece, its sums
  __shared__ __align__(16) float s_col[kGroups][kCols];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();  // 0: the leader, which issues the MMAs
  const int worker = (int)blockIdx.x >> 1, n_workers = (int)gridDim.x >> 1;
  uint8_t* sK = smem;
  uint8_t* sQ = smem + 2 * kKBytes;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.k_full[s], 1);
      mbar_init(&bar.k_empty[s], 1);
    }
    for (int s = 0; s < kQSlots; ++s) {
      mbar_init(&bar.q_full[s], 1);
      mbar_init(&bar.q_empty[s], 1);
    }
    for (int s = 0; s < kGroups; ++s) {
      mbar_init(&bar.s_full[s], 1);
      mbar_init(&bar.s_empty[s], 8);  // a warpgroup's four warps in both CTAs
    }
    mbar_init(&bar.sum_ready, 4 * (kGroups - 1));
    mbar_init(&bar.sum_free, 4);
    abort_flag = 0;
    fence_mbarrier_init();
  }
  if (threadIdx.x == 32 * 2) {
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
  }
  if (warp == 1) tmem_alloc_pair(&tmem_base_sh, 512);
  __syncwarp();
  cluster_arrive();
  find_start(p, worker, n_workers, &start);
  // the tiles need every byte there is, so their 1024-byte alignment is the declaration's; placed
  // elsewhere, no pair takes any work, and all record that
  if (threadIdx.x == 0 && (smem_u32(smem) & 1023u)) {
    raise_device_error(p.s.err, HCADSA_ERR_CUDA);
    start.count = 0;
  }
  tc_fence_before();
  __syncthreads();
  cluster_wait();  // barriers and TMEM of both CTAs exist before any cross-CTA operation
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const int page_mask = (1 << p.s.page_log2) - 1;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (all lanes)
    // boxes of 128 K rows, one per lane: 8 rows x 4 chunks, or 128 / box rows x 1 chunk.  (Pages of 16 rows
    // would take boxes of 2 KB, and a TMA copy costs some 95 cycles however small: 181 + 10 tokens over
    // 4K-12K rows of such pages 80 us against 99.  With pages of 64 rows the larger boxes win, 72 against 78.)
    const bool groups = p.box_log2 == 3;
    const int krow = groups ? 8 * lane : (lane >> 2) << p.box_log2, kchunk = groups ? 0 : lane & 3;
    const int kboxes = groups ? 16 : 512 >> p.box_log2, kdst = krow * (p.k_group >> 3) + kchunk * p.k_chunk;
    const int g64 = p.g_log2 < 6 ? p.g_log2 : 6;  // heads of a Q box; a group of 128 is two boxes, one per CTA
    uint32_t piece = 0, u = 0;                    // u: Q tiles loaded
    bool ok = true, loaded = false;
    for (Walk w(p, start); !w.done() && ok; w.next(), ++piece) {
      const uint32_t kb = piece & 1;
      const int row = w.k * kKeys + 128 * (int)rank + krow;
      int pg = p.s.n_pages;  // a page that is not there: zeros (outside the tensor map)
      if (lane < kboxes && row < w.q.len) {
        pg = paged_page(p.s, w.b, row);
        if (pg < 0) pg = p.s.n_pages;
      }
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.k_empty[kb], ((piece >> 1) & 1) ^ 1, &abort_flag, p.s.err));
      if (!ok) break;
      if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&bar.k_full[kb], 2 * kKBytes);
      __syncwarp();
      if (lane < kboxes)
        tma_load_5d_pair(sK + kb * kKBytes + kdst, &map_k, cluster_addr(&bar.k_full[kb], 0), 0, row & page_mask,
                         kchunk, w.h, pg);
      for (int t = w.t0; t < w.t1 && ok; ++t) {
        if (!loaded) {
          const uint32_t s = u % kQSlots;
          ok = __all_sync(0xffffffffu,
                          mbar_wait(&bar.q_empty[s], ((u / kQSlots) & 1) ^ 1, &abort_flag, p.s.err));
          if (!ok) break;
          if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&bar.q_full[s], 2 * kQBytes);
          __syncwarp();
          if (lane < 4) {
            const int tok = w.q.q0 + (t << (7 - p.g_log2)) + ((int)rank << (6 - g64));
            const int head = (w.h << p.g_log2) + (p.g_log2 == 7 ? 64 * (int)rank : 0);
            tma_load_3d_pair(sQ + s * kQBytes + lane * kQChunk, &map_q, cluster_addr(&bar.q_full[s], 0), lane * 64,
                             head, p.g_log2 == 7 ? w.q.q0 + t : tok);
          }
          ++u;
        }
        loaded = t + 1 == w.t1 && w.same_tile_next();  // the next product's Q tile is this one
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader CTA)
    // The whole warp walks and waits, one elected lane issues: the descriptors stay warp-uniform values.
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(kKeys, kCols, false, false);
      const uint32_t sKa = smem_u32(sK), sQa = smem_u32(sQ);
      auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(b, parity, &abort_flag, p.s.err));
      };
      uint32_t piece = 0, u = 0, n = 0;  // n: products so far (S buffer n & 3)
      bool ok = true;
      for (Walk w(p, start); !w.done() && ok; w.next(), ++piece) {
        const uint32_t kb = piece & 1;
        ok = wait(&bar.k_full[kb], (piece >> 1) & 1);
        const uint64_t da = smem_desc_sw128(sKa + kb * kKBytes, 16, p.k_group);
        for (int t = w.t0; t < w.t1 && ok; ++t, ++n) {
          const uint32_t s = u % kQSlots, sb = n & 3;
          const bool last = t + 1 == w.t1, keep = last && w.same_tile_next();
          ok = wait(&bar.q_full[s], (u / kQSlots) & 1) && wait(&bar.s_empty[sb], ((n >> 2) & 1) ^ 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t db = smem_desc_sw128(sQa + s * kQBytes, 16, 1024);
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)  // start addresses in 16-byte units
                mma_ss_pair(tmem + sb * kCols, da + (uint64_t)((c * p.k_chunk + kk * 32) >> 4),
                            db + (uint64_t)((c * kQChunk + kk * 32) >> 4), idesc, (c | kk) != 0);
            mma_commit_pair(&bar.s_full[sb]);
            if (!keep) mma_commit_pair(&bar.q_empty[s]);
            if (last) mma_commit_pair(&bar.k_empty[kb]);
          }
          __syncwarp();
          if (!keep) ++u;
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ sums (one thread per cache row)
    // Warpgroup w takes the products whose S buffer is w.
    const int wg = (warp - 4) >> 2, quarter = warp & 3;
    const int in_cta = quarter * 32 + lane;  // TMEM lane; also the column whose lse this thread fetches
    const uint32_t t_lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int group_mask = (1 << p.g_log2) - 1;
    const size_t lse_step = (size_t)((kGroups * kCols) >> p.g_log2) * p.Hq;  // to this group's next tile
    float* col = s_col[wg];
    const uint32_t empty_addr = cluster_addr(&bar.s_empty[wg], 0);
    uint32_t n = 0, shared_pieces = 0;
    bool ok = true, handed = false;  // handed: s_col holds sums that the finishing group has not read yet
    int head_flag = 0, tail_flag = 0, tail_b = 0, tail_h = 0, tail_k = 0;  // for ws_meta
    for (Walk w(p, start); !w.done(); w.next()) {
      const int key = w.k * kKeys + 128 * (int)rank + in_cta;
      const int n_rows = w.q.n << p.g_log2;  // (token, head) rows of the chunk; column c of tile t is 128 t + c
      const int mine = (int)((wg - n) & (kGroups - 1));  // this warpgroup's first tile of the piece
      int r = (w.t0 + mine) * kCols + in_cta;  // the row whose lse this thread fetches next
      const float* lse_at = p.lse + (size_t)(w.q.q0 + (r >> p.g_log2)) * p.Hq + (w.h << p.g_log2) + (r & group_mask);
      auto fetch = [&]() -> float {
        const float v = r < n_rows ? *lse_at : 0.0f;  // scaled when it is used, so that nothing waits here
        r += kGroups * kCols;
        lse_at += lse_step;
        return v;
      };
      // the warpgroup of the piece's last tile finishes the piece
      const int tiles = w.t1 - w.t0, finisher = (int)((n + (uint32_t)tiles - 1) & (kGroups - 1));
      const bool finish = finisher == wg;
      // this row's page, looked up now and looked at when the piece is done
      const bool mine_to_add = finish && key < w.q.len;
      int pg = 0;
      if (mine_to_add) pg = p.s.table[(size_t)w.b * p.s.max_pages + (key >> p.s.page_log2)];
      // tokens from here on see this row
      const int lo_row = min(max(key - w.q.base, 0), w.q.n) << p.g_log2;
      float sum = 0.0f, low = 0.0f;  // compensated: sum + low
      float next = w.t0 + mine < w.t1 ? fetch() : 0.0f;
      auto wait_free = [&]() {
        if (handed) ok = mbar_wait(&bar.sum_free, (shared_pieces - 1) & 1, &abort_flag, p.s.err) && ok;
        handed = false;
      };
      for (int t = w.t0 + mine; t < w.t1; t += kGroups) {
        const uint32_t at = n + (uint32_t)(t - w.t0), sb = (uint32_t)wg;
        wait_free();
        group_bar(1 + wg, 128);  // the tile before has been summed
        col[in_cta] = next * -1.4426950408889634f;
        if (t + kGroups < w.t1) next = fetch();
        group_bar(1 + wg, 128);
        ok = mbar_wait(&bar.s_full[sb], (at >> 2) & 1, &abort_flag, p.s.err) && ok;
        tc_fence_after();
        const int c_hi = min(kCols, n_rows - t * kCols);                                // uniform
        const int c_lo = max(0, min(kCols, lo_row - t * kCols));                              // this row's
        const bool all = c_hi == kCols && __all_sync(0xffffffffu, c_lo == 0);
        const int c_end = __all_sync(0xffffffffu, c_lo >= c_hi) ? 0 : c_hi;  // 0: no row of the warp is seen
        float a4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c * 32 >= c_end) break;
          uint32_t v[32];
          tmem_ld32_nowait(t_lanes + sb * kCols + c * 32, v);
          tmem_wait_ld_regs(v);
          if (all) {
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const float4 l = *reinterpret_cast<const float4*>(col + c * 32 + x);
              a4[0] += fast_exp2(fmaf(__uint_as_float(v[x]), p.scale_log2, l.x));
              a4[1] += fast_exp2(fmaf(__uint_as_float(v[x + 1]), p.scale_log2, l.y));
              a4[2] += fast_exp2(fmaf(__uint_as_float(v[x + 2]), p.scale_log2, l.z));
              a4[3] += fast_exp2(fmaf(__uint_as_float(v[x + 3]), p.scale_log2, l.w));
            }
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const int cc = c * 32 + x;
              const float e = fast_exp2(fmaf(__uint_as_float(v[x]), p.scale_log2, col[cc]));
              a4[x & 3] += cc >= c_lo && cc < c_hi ? e : 0.0f;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster_relaxed(empty_addr);
        const float y = ((a4[0] + a4[1]) + (a4[2] + a4[3])) - low, z = sum + y;  // Kahan's sum over the tiles
        low = (z - sum) - y;
        sum = z;
      }
      // ---- the piece's sum: the other warpgroups hand theirs to the one of the last tile
      if (tiles > 1) {
        wait_free();
        if (!finish) {
          group_bar(1 + wg, 128);
          col[in_cta] = sum;  // (without `low`: one fp32 rounding per warpgroup and piece)
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.sum_ready);
          handed = true;
        } else {
          ok = mbar_wait(&bar.sum_ready, shared_pieces & 1, &abort_flag, p.s.err) && ok;
#pragma unroll
          for (int o = 1; o < kGroups; ++o) {
            const int from = (wg + o) & (kGroups - 1);
            if ((int)((from - n) & (kGroups - 1)) < tiles) sum += s_col[from][in_cta];  // it had a tile
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.sum_free);
        }
        ++shared_pieces;
      }
      n += (uint32_t)tiles;
      if (finish) {
        if (w.whole()) {
          if (mine_to_add) {
            if (pg >= 0 && pg < p.s.n_pages)
              atomicAdd(p.mass + (((size_t)pg << p.s.page_log2) + (key & page_mask)) * p.Hkv + w.h, sum);
            else
              raise_device_error(p.s.err, kErrDeviceBounds);
          }
        } else {
          const int rec = 2 * worker + (w.t0 == w.first ? 1 : 0);
          p.ws_sum[(size_t)rec * kKeys + 128 * (int)rank + in_cta] = sum;
        }
      }
      if (!w.whole()) {
        if (w.t0 > w.first) {
          head_flag = w.t1 == w.last ? 2 : 1;
        } else {
          tail_flag = 1;
          tail_b = w.b;
          tail_h = w.h;
          tail_k = w.k;
        }
      }
    }
    if (rank == 0 && threadIdx.x == 128) {
      int* m = p.ws_meta + worker * kMetaInts;
      m[0] = head_flag;
      m[1] = tail_flag;
      m[2] = tail_b;
      m[3] = tail_h;
      m[4] = tail_k;
    }
  }

  launch_dependents();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no MMA of the pair and no cross-CTA arrival is pending any more
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// Adds up the partial sums of a block that began in pair c's range and went on in pairs c+1, c+2, ...,
// in that order, one thread per cache row.
__global__ void __launch_bounds__(kKeys) add_kernel(const Params p, int n_workers) {
  wait_for_primary();
  const int c = blockIdx.x;
  const int* meta = p.ws_meta + c * kMetaInts;
  if (!meta[1]) return;
  int n = 1;  // pieces: up to the one that ends the block (the lanes read the records side by side)
  for (int k0 = c + 1; k0 < n_workers; k0 += 32) {
    const int lane = threadIdx.x & 31;
    const int flag = k0 + lane < n_workers ? p.ws_meta[(k0 + lane) * kMetaInts] : 2;
    const uint32_t last = __ballot_sync(0xffffffffu, flag != 1);
    n += last ? __ffs(last) : 32;
    if (last) break;
  }
  n = min(n, n_workers - c);
  const int b = meta[2], h = meta[3], key = meta[4] * kKeys + threadIdx.x;
  if (key >= paged_len(p.s, b, false)) return;
  float sum = p.ws_sum[(size_t)(2 * c + 1) * kKeys + threadIdx.x];
#pragma unroll 8
  for (int k = 1; k < n; ++k) sum += p.ws_sum[(size_t)(2 * (c + k)) * kKeys + threadIdx.x];
  const int pg = paged_page(p.s, b, key);
  if (pg < 0) return;
  const int in = key & ((1 << p.s.page_log2) - 1);
  atomicAdd(p.mass + (((size_t)pg << p.s.page_log2) + in) * p.Hkv + h, sum);
}

// Pairs of a launch: one per two SMs of the current device.
int pairs_of_device() {
  static std::mutex mu;
  static int cache[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (!cache[dev]) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 2 ||
        cudaFuncSetAttribute(mass_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess) {
      launch_status();
      return 0;
    }
    cache[dev] = sms / 2 < kMaxPairs ? sms / 2 : kMaxPairs;
  }
  return cache[dev];
}

size_t workspace_bytes_of(int pairs) { return (size_t)pairs * (2 * kKeys * 4 + kMetaInts * 4); }

}  // namespace
}  // namespace hcadsa

extern "C" size_t mla_paged_attn_mass_workspace_size(int B, int T, int Hq, int Hkv) {
  using namespace hcadsa;
  if (B <= 0 || T <= 0 || Hkv <= 0 || check_query_sizes(T, Hq, Hkv, kMlaD, 1.0f) != HCADSA_OK) return 0;
  return workspace_bytes_of(pairs_of_device());
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
  const int pairs = pairs_of_device();
  if (pairs <= 0) return HCADSA_ERR_CUDA;
  if (!workspace || workspace_bytes < workspace_bytes_of(pairs)) return HCADSA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return HCADSA_ERR_ALIGN;
  Params p;
  p.s = paged_batch(table, cu_q, kv_len, B, T, n_pages, page, max_pages);
  p.lse = lse;
  p.mass = mass;
  p.ws_sum = static_cast<float*>(workspace);
  p.ws_meta = reinterpret_cast<int*>(p.ws_sum + (size_t)2 * pairs * kKeys);
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.g_log2 = log2_of(Hq / Hkv);
  const bool groups = page < 32;
  p.box_log2 = groups ? 3 : page < 64 ? log2_of(page) : 6;
  p.k_group = groups ? 4096 : 1024;
  p.k_chunk = groups ? 1024 : kKBytes / 4;
  p.scale_log2 = scale * 1.4426950408889634f;
  CUtensorMap mq, mk;
  {
    const int g = p.g_log2 < 6 ? 1 << p.g_log2 : 64;
    const uint64_t dims[3] = {(uint64_t)kMlaD, (uint64_t)Hq, (uint64_t)T};
    const uint64_t strides[2] = {(uint64_t)kMlaD * 2, (uint64_t)q_row_stride * 2};
    const uint32_t box[3] = {64, (uint32_t)g, (uint32_t)(64 / g)};
    if (!encode_tmap_bf16(&mq, 3, const_cast<hcadsa_bf16*>(Q), dims, strides, box, true)) return HCADSA_ERR_CUDA;
  }
  {
    const uint64_t dims[5] = {64, (uint64_t)page, kMlaD / 64, (uint64_t)Hkv, (uint64_t)n_pages};
    const uint64_t strides[4] = {(uint64_t)Hkv * kMlaD * 2, 64 * 2, (uint64_t)kMlaD * 2, (uint64_t)k_page_stride * 2};
    const uint32_t box[5] = {64, 1u << p.box_log2, groups ? kMlaD / 64u : 1u, 1, 1};
    if (!encode_tmap_bf16(&mk, 5, const_cast<hcadsa_bf16*>(K_pool), dims, strides, box, true)) return HCADSA_ERR_CUDA;
  }
  mass_kernel<<<2 * pairs, kThreads, kSmemBytes, as_stream(stream)>>>(mq, mk, p);
  HCADSA_TRY(launch_status());
  return launch_after(add_kernel, dim3(pairs), kKeys, as_stream(stream), p, pairs);
}
