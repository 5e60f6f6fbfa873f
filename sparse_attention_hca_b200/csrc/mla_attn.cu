// mla_attn.cu -- attention of a chunk of new tokens over the paged cache of the full-context
// (MLA) layers on sm_100a (mla_paged_attn_fwd): TMA page loads, tcgen05 MMA on CTA pairs, TMEM.
//
// Method: the mirrorspeed page, section "Hybrid sparse attention, 1/7 full context access": the
// MLA layers see every token; heads are 256 wide.  New token i of a sequence sees the rows
// <= base + i of its cache (base: rows before the chunk):
//     O = sum_s p_s v_s,  p = softmax_s(scale <q, k_s>),  lse = log sum_s exp(scale <q, k_s>)
//
// Tiles: the g query heads of a K/V head share its rows, so a row tile is 256 (token, head) rows
// = 256 / g tokens; a key tile is 128 cache rows.  A CTA pair computes a row tile against a run of
// key tiles: CTA r holds rows 128 r .. 128 r + 127 (its TMEM lanes), and loads half of every K and
// V tile -- K rows 64 r .. +63, V columns 128 r .. +127 -- which the pair's MMAs (cta_group::2,
// M = 256) read from both.  One CTA alone (M = 128) would need 64 bytes of K and V per SM cycle at
// the full MMA rate, the limit of the L2; the pair needs 32.  Batches of short chunks (decode steps)
// run on single CTAs with row tiles of 128 rows instead: see use_pairs.
//   S  = Q (A, smem) * K^T (B, smem, K-major)        128 columns of TMEM, two buffers
//   O += P (A, TMEM, bf16 over its own S) * V (B, smem, MN-major)   256 columns of TMEM
// S and O together are all 512 columns.  Roles per CTA: warp 0 TMA (both CTAs; the lanes issue a
// tile's page boxes side by side), warp 1 the MMA thread (leader CTA), warps 4-11 softmax, two
// threads per row.  The reference maximum moves only when it is exceeded by 2^8 (lazy rescale of
// O).  P is rounded to bf16, the type the tensor cores take, after its sum was taken in fp32.
//
// Schedule: the (row tile, key tile) products of the whole batch form one list -- sequence, K/V
// head, row tile, key tile -- whose length follows in closed form from the lengths (in long lists a
// row tile also takes some places for its output, see kTileCost).  Worker c of G takes the places
// [c N / G, (c+1) N / G): equal work for prompts, chunks and single tokens alike, decided on the device
// (the host never sees the lengths).  A row tile that several workers share
// leaves unnormalised fp32 rows and (max, sum) in the workspace -- at most two such pieces per
// worker -- and combine_kernel merges them in list order: the result does not depend on timing.
//
// Measured (B200, 64 heads on one K/V head): 2048 tokens over 32768 rows 2.8 ms in a short run
// (1.52 PFLOP/s), 2.95 ms when repeated (1.44 PFLOP/s; the power limit holds the clock at 1.45 GHz).
// A product takes about 2300 cycles of 2048 for its MMAs (the tensor pipe is busy 89 % of the active
// cycles): the S MMAs read A and B from shared memory at 128 bytes per cycle, its limit, next to the
// incoming tiles.  32 sequences of 1K-32K rows, one token each: 106 us on the device, 5.4 TB/s (113
// repeated).
//
// Rows behind the end of a sequence in its last page may hold anything.  Their scores are replaced
// before the softmax, and since 0 * NaN is NaN, the V rows of such a tile are cleared in shared
// memory by the softmax warps before the PV product: that tile's V completes on a barrier of its
// own CTA (v_tail) instead of the leader's.
#include <mutex>

#include "mla_host.h"
#include "pair.cuh"

namespace hcadsa {
namespace {

constexpr int kKeyTile = 128;
constexpr int kCtaRows = 128;              // (token, head) rows of a CTA: TMEM lanes
constexpr int kSlots = 5;                  // ring of half tiles of K and V
constexpr int kSlotBytes = 32 * 1024;
constexpr int kQBytes = 64 * 1024;         // 128 rows x 256
constexpr int kQChunk = 16 * 1024;         // 64 columns of 128 rows
constexpr int kSmemBytes = kQBytes + kSlots * kSlotBytes + 1024;
constexpr int kSoftmaxWarps = 8;           // two per TMEM lane quarter: each takes half of a row
constexpr int kThreads = 128 + 32 * kSoftmaxWarps;
constexpr uint32_t kTmemS = 256;           // S buffers at columns 256 and 384; O at 0
constexpr float kLazyRescale = 8.0f;
constexpr int kMetaInts = 8;

// How the page boxes of K or V lie in a slot: boxes of 2^rows_log2 rows x 2^chunks_log2 chunks of 64
// columns; `step` bytes from 8 rows of K (16 of V) to the next, `chunk` from a chunk to the next.
struct BoxLayout {
  int rows_log2, chunks_log2, step, chunk;
};

struct Params {
  PagedBatch s;
  uint16_t* O;
  float* lse;
  float* ws_O;   // [2 G][rows][256]: worker c's piece that began before its range (2 c) or in it (2 c + 1)
  float* ws_ml;  // [2 G][2][rows]: reference maximum (log2 units), sum
  int* ws_meta;  // [G][kMetaInts]
  int Hq, Hkv, g_log2;
  int piece_rows;  // rows of an average row tile where the batch has more rows than the merge has blocks, or 0
  BoxLayout k_box, v_box;
  float scale_log2;
  bool wide_stores;  // O is 32-byte aligned
};

// A worker is a CTA pair or a single CTA.
//   pair   : row tile 256 rows; a slot is CTA r's half of a tile for the pair's MMAs: K rows 64 r .. +63
//            (4 chunks of 64 columns), V columns 128 r .. +127 (2 chunks of 128 rows)
//   single : row tile 128 rows; a tile is two slots: K columns 128 half .. +127 (2 chunks of 128 rows),
//            V rows 64 half .. +63 (4 chunks of 64 rows)
template <bool kPair>
struct Shape {
  static constexpr int kRows = kPair ? 2 * kCtaRows : kCtaRows;
  static constexpr int kRowsLog2 = kPair ? 8 : 7;
  static constexpr int kParts = kPair ? 1 : 2;                           // slots of a tile
  static constexpr int kKChunksLog2 = kPair ? 2 : 1, kVChunksLog2 = kPair ? 1 : 2;  // chunks of a slot
  static constexpr int kReady = (kPair ? 2 : 1) * kSoftmaxWarps;
};

struct __align__(8) Barriers {
  uint64_t q_full, q_empty;
  uint64_t full[kSlots], empty[kSlots];
  uint64_t s_full[2], p_ready[2];
  uint64_t pv_done, o_full;  // a tile's PV, a piece's last PV
  uint64_t v_tail[2];  // alternating: a piece's tail may land while the piece before waits for its own
};

// ------------------------------------------------------------------ the list of products

// One sequence's part of the list (of one K/V head).
struct SeqTiles {
  int base, n, len, tq_log2;
  int extra;  // what a row tile weighs in the list besides its products
  __host__ __device__ int row_tiles() const { return (n + (1 << tq_log2) - 1) >> tq_log2; }
  // key tiles of row tile i: up to the last row its last token sees.  A sequence declared shorter
  // than its chunk (base < 0) has rows that see nothing; its row tiles take every key tile, at
  // least one, and the mask does the rest.
  __host__ __device__ int key_tiles(int i) const {
    if (base < 0) return len > 0 ? (len + kKeyTile - 1) / kKeyTile : 1;
    const long long last = (long long)(i + 1) << tq_log2;
    return (int)((base + (last < n ? last : n) + kKeyTile - 1) / kKeyTile);
  }
  // key tiles of the row tiles before i, in closed form: sum over k = 1 .. i of
  // ceil((base + k tq) / 128), whose terms grow by one every 128 / tq row tiles
  __host__ __device__ long long before(int i) const {
    if (base < 0) return (long long)i * key_tiles(0);
    const int rem = base % kKeyTile;
    long long sum = (long long)i * (base / kKeyTile);
    if (tq_log2 >= 8) {
      sum += (long long)i * (i + 1) + (rem > 0 ? i : 0);
    } else {
      const int p_log2 = 7 - tq_log2, p = 1 << p_log2;
      const long long a = i >> p_log2, r = i & (p - 1);
      const int ones = (kKeyTile - rem) >> tq_log2;  // terms of the first 128 / tq that are 1, not 2
      const auto part = [&](long long x) { return x + (x > ones ? x - ones : 0); };
      sum += a * part(p) + p * (a * (a - 1) / 2) + a * r + part(r);
    }
    if (i > 0 && i == row_tiles()) {  // the last row tile ends with the cache
      const long long full = base + ((long long)i << tq_log2);
      sum -= (full + kKeyTile - 1) / kKeyTile - key_tiles(i - 1);
    }
    return sum;
  }
  // where row tile i begins in the list
  __host__ __device__ long long start(int i) const { return before(i) + (long long)extra * i; }
  // the row tile that holds place w of the list
  __host__ __device__ int find(long long w) const {
    int lo = 0, hi = row_tiles();
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start(mid) <= w) lo = mid;
      else hi = mid;
    }
    return lo;
  }
};

// A pair's row tile costs its output (3-4 us) besides its products (1.3 us each), so in lists that give
// every pair 2 products or more a tile weighs as much as this many more, which come first in it.  (3
// sequences of 844 tokens over up to 1749 rows next to 26 single tokens, 16 heads: 59 us against 84; 361
// tokens over 10164 rows, 16 heads, 61 against 62; 512 tokens from nothing, 64 heads, 33 against 37; a
// weight of 2 is 2-4 % slower in the first two, 6 10 %.)  Not the tile of a
// sequence with at most 32 rows to write (weighed as well, 2 chunks next to 22 single tokens of 8 rows took
// 1 % longer; with single tokens of 64 rows not weighed, 29 sequences took 90 us against 82).
constexpr int kTileCost = 3;

__device__ __forceinline__ SeqTiles seq_tiles(const PagedSeq& q, int tq_log2, bool weigh) {
  SeqTiles t;
  t.extra = weigh && 8 * q.n > (1 << tq_log2) ? kTileCost : 0;
  t.base = q.base;
  t.n = q.n;
  t.len = q.len;
  t.tq_log2 = tq_log2;
  return t;
}

struct Start {
  long long count;  // this worker's share of the list
  int b, h, i, at;  // where it begins: `at` places into row tile i
  bool weigh;       // whether row tiles weigh more than their products
  PagedSeq q;       // sequence b
};

// Walks a worker's pieces: runs of key tiles of one row tile.
template <int kRowsLog2>
struct Walk {
  const Params& p;
  long long left;
  int b, h, i, at, j0, j1, n_keys, tq_log2;
  bool weigh;
  PagedSeq q;
  SeqTiles t;
  __device__ Walk(const Params& p_, const Start& s) : p(p_) {
    tq_log2 = kRowsLog2 - p.g_log2;
    left = s.count;
    b = s.b;
    h = s.h;
    i = s.i;
    at = s.at;
    weigh = s.weigh;
    if (left > 0) {
      q = s.q;
      t = seq_tiles(q, tq_log2, weigh);
      cut();
    }
  }
  __device__ bool done() const { return left <= 0; }
  __device__ int tiles() const { return j1 - j0; }
  __device__ int first_token() const { return i << tq_log2; }
  __device__ void next() {
    left -= j1 + t.extra - at;
    if (left <= 0) return;
    at = 0;
    if (++i == t.row_tiles()) {
      i = 0;
      if (++h == p.Hkv) {
        h = 0;
        do {
          if (++b >= p.s.B) {  // cannot happen unless the lengths change under the kernel
            left = 0;
            return;
          }
          load();
        } while (t.n == 0);
      }
    }
    cut();
  }

 private:
  __device__ void load() {
    q = paged_seq(p.s, b, false);
    t = seq_tiles(q, tq_log2, weigh);
  }
  __device__ void cut() {  // places [0, t.extra) of a row tile hold no product
    n_keys = t.key_tiles(i);
    const long long e = at + left - t.extra;
    j0 = at > t.extra ? at - t.extra : 0;
    j1 = e < n_keys ? (int)e : n_keys;
    if (j1 <= j0) left = 0;  // the share ends before the tile's first product
  }
};

// Where a worker's share begins: product x of the list, or the start or end of the row tile that
// holds it, whichever is nearer, if that tile is short: a cut costs its partial rows, written and
// merged, about as much as 8 products, and moving it at most half the tile's length in balance.
// Shares of one or two products are cut all the same: there the time is that of the longest one.
// Nor are single CTAs' (a few rows a sequence) moved: their partial rows are few.
// (256 tokens on 1024 rows, 64 heads: 27.1 us against 41.0; but 32 sequences of one token on up to
// 4000 rows 36.3 against 33.1 when single CTAs did the same.)
constexpr int kShortTile = 12;

__device__ __forceinline__ long long snap(const SeqTiles& t, long long from, long long per_head, long long x,
                                          long long share) {
  if (t.base >= kShortTile * kKeyTile) return x;  // (every tile of the sequence is long)
  const long long in = (x - from) % per_head;
  const int i = t.find(in), n = t.key_tiles(i);
  if (n > kShortTile || n > 2 * share) return x;
  const long long j = in - t.start(i);
  return x - j + (2 * j >= n + t.extra ? n + t.extra : 0);
}

// Every thread of the CTA: this worker's share of the list.
template <bool kPair>
__device__ __forceinline__ void find_start(const Params& p, int tq_log2, int worker, int n_workers, Start* out) {
  __shared__ long long sums[kThreads / 32];
  __shared__ long long cut[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool weigh = false;
  auto work_of = [&](int b, bool report) -> long long {
    if (b >= p.s.B) return 0;
    const SeqTiles t = seq_tiles(paged_seq(p.s, b, report), tq_log2, weigh);
    return t.n > 0 ? t.start(t.row_tiles()) * p.Hkv : 0;
  };
  // inclusive prefix over the CTA's threads, and its total
  auto scan = [&](long long x, long long& total) -> long long {
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
  long long mine_to = scan(mine, all);
  if (kPair && all >= 2LL * n_workers) {
    weigh = true;
    mine = 0;
    for (int b = tid; b < p.s.B; b += kThreads) mine += work_of(b, false);
    mine_to = scan(mine, all);
  }
  // A short list goes to as many workers as it has products, so that consecutive pieces of a row
  // tile always lie with consecutive workers; where merging costs more, to fewer.  A piece costs the
  // merge about 1/12 of a product, so a tile of k products is best cut into pieces of sqrt(k / 12).  (One
  // token over 16K, 32K, 128K rows: 20.5, 24.6, 41.2 us against 23.3, 30.0, 45.1 on all workers; a constant
  // of 8 or 16 is up to 2 us slower.)  Where many rows are merged it also costs their bytes, 1/6000 of a
  // product per row of every piece (124 tokens over 1747 rows, 16 K/V heads: 26 us against 33; 18 tokens of
  // 128 heads over up to 2245 rows 30.5 against 33; 1500 and 700 cost other batches 3 and 7 %).
  const long long tiles = (long long)p.Hkv * max(p.s.B, (int)(((long long)p.s.T << p.g_log2) >> (kPair ? 8 : 7)));
  long long most = all;
  if (all >= 48 * tiles || p.piece_rows > 0) {
    const float share2 = (float)all * (1.0f / (float)(12 * tiles) + (float)p.piece_rows * (1.0f / 6000.0f));
    const int least = max(1, (int)sqrtf(share2));
    most = (all + least - 1) / least;
  }
  const int n = most < n_workers ? (int)most : n_workers;
  if (tid == 0) out->count = 0;
  if (worker >= n) return;
  const long long x0 = all * worker / n, x1 = all * (worker + 1) / n;
  const long long share = all / n;  // (the same for all workers, so that neighbours agree on a cut)
  // f(sequence, its products [from, upto)) for every sequence, all threads side by side
  auto each = [&](auto&& f) {
    long long done = 0;
    for (int b0 = 0; b0 < p.s.B; b0 += kThreads) {
      const int b = b0 + tid;
      if (p.s.B <= kThreads) {  // known from the first pass
        if (mine > 0) f(b, mine_to - mine, mine_to);
      } else {
        long long total;
        const long long w = work_of(b, false), upto = done + scan(w, total);
        if (w > 0) f(b, upto - w, upto);
        done += total;
      }
    }
  };
  if (tid < 2) cut[tid] = tid ? x1 : x0;
  __syncthreads();
  if (kPair && share >= 3) {
    each([&](int b, long long from, long long upto) {
#pragma unroll 1
      for (int e = 0; e < 2; ++e) {
        const long long x = e ? x1 : x0;
        if (from <= x && x < upto)
          cut[e] = snap(seq_tiles(paged_seq(p.s, b, false), tq_log2, weigh), from,
                        (upto - from) / p.Hkv, x, share);
      }
    });
    __syncthreads();
  }
  const long long lo = cut[0], hi = cut[1];
  if (tid == 0) out->count = hi - lo;
  each([&](int b, long long from, long long upto) {
    if (from <= lo && lo < upto) {
      out->q = paged_seq(p.s, b, false);
      const SeqTiles t = seq_tiles(out->q, tq_log2, weigh);
      const long long per_head = (upto - from) / p.Hkv, r = lo - from;
      out->b = b;
      out->h = (int)(r / per_head);
      const long long in = r - out->h * per_head;
      out->i = t.find(in);
      out->at = (int)(in - t.start(out->i));
      out->weigh = weigh;
    }
  });
}

__device__ __forceinline__ void store_32(void* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Lanes 4 q .. 4 q + 3 hold four rows of 32 columns; afterwards lane 4 q + i holds columns 8 i .. 8 i + 7 of
// all four, row k in v[8 k .. 8 k + 7].
__device__ __forceinline__ void transpose_4(uint32_t (&v)[32], int lane) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a & bit) continue;
      const int b = a | bit;
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v[8 * a + y] : v[8 * b + y], bit);
        if (up) v[8 * a + y] = got;
        else v[8 * b + y] = got;
      }
    }
  }
}

// ------------------------------------------------------------------ the kernel

template <bool kPair>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (kPair) mma_commit_pair(bar);
  else mma_commit(bar);
}
// A page box into this CTA's shared memory, completing on the leader's copy of `bar`.
template <bool kPair>
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, uint64_t* bar, int row, int chunk, int head,
                                         int page) {
  if constexpr (kPair) tma_load_5d_pair(dst, map, cluster_addr(bar, 0), 0, row, chunk, head, page);
  else tma_load_5d(dst, map, bar, 0, row, chunk, head, page);
}

template <bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + kQBytes;
  __shared__ Barriers bar;
  __shared__ Start start;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  using Sh = Shape<kPair>;
  using Pieces = Walk<Sh::kRowsLog2>;
  const uint32_t rank = kPair ? cluster_rank() : 0;  // 0: the leader, which issues the MMAs
  const int worker = kPair ? (int)blockIdx.x >> 1 : (int)blockIdx.x;
  const int n_workers = kPair ? (int)gridDim.x >> 1 : (int)gridDim.x;
  if (threadIdx.x == 0) {
    mbar_init(&bar.q_full, 1);
    mbar_init(&bar.q_empty, 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&bar.full[s], 1);
      mbar_init(&bar.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.s_full[s], 1);
      mbar_init(&bar.p_ready[s], Sh::kReady);  // the worker's softmax warps
    }
    mbar_init(&bar.pv_done, 1);
    mbar_init(&bar.o_full, 1);
    for (int s = 0; s < 2; ++s) mbar_init(&bar.v_tail[s], 1);
    abort_flag = 0;
    fence_mbarrier_init();
  }
  if (threadIdx.x == 32 * 2) {
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(&tmem_base_sh, 512);
    } else {
      tmem_alloc(&tmem_base_sh, 512);
      tmem_relinquish();
    }
  }
  __syncwarp();
  if constexpr (kPair) cluster_arrive();
  find_start<kPair>(p, Sh::kRowsLog2 - p.g_log2, worker, n_workers, &start);
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_wait();  // barriers and TMEM of both CTAs exist before any cross-CTA operation
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const int box_rows = 1 << p.v_box.rows_log2;
  // whether key tile j holds rows behind the sequence's end that a page box brings in
  auto is_tail = [&](int len, int j) { return (len & (box_rows - 1)) != 0 && len / kKeyTile == j; };
  // the half of such a tile (64 rows) that holds them: a box lies in one half
  auto tail_part = [](int len) { return (len & (kKeyTile - 1)) >> 6; };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (all lanes)
    // A slot's page boxes, one per lane, each of `rows` rows and some of the slot's chunks.
    struct Box {
      int row, chunk, to;  // this lane's first row and chunk, and where in the slot they go
      bool on;
    };
    auto box_of = [&](int rows_log2, int chunks_log2, int slot_chunks_log2, int step_log2, int step, int chunk_bytes) {
      const int across = slot_chunks_log2 - chunks_log2;  // log2 of the boxes side by side
      Box x;
      x.row = (lane >> across) << rows_log2;
      x.chunk = (lane & ((1 << across) - 1)) << chunks_log2;
      x.to = (x.row >> step_log2) * step + x.chunk * chunk_bytes;
      x.on = x.row < (256 >> slot_chunks_log2);
      return x;
    };
    const Box kb = box_of(p.k_box.rows_log2, p.k_box.chunks_log2, Sh::kKChunksLog2, 3, p.k_box.step, p.k_box.chunk);
    const Box vb = box_of(p.v_box.rows_log2, p.v_box.chunks_log2, Sh::kVChunksLog2, 4, p.v_box.step, p.v_box.chunk);
    const int k_row = kb.row + (kPair ? 64 * (int)rank : 0);  // this lane's row of a K tile
    const int v_row = vb.row;                                 // and of a V tile (single: + 64 per part)
    const int page_mask = (1 << p.s.page_log2) - 1;
    uint32_t u = 0;  // slots issued: slot u % kSlots
    uint32_t it = 0, tails = 0;
    bool ok = true;
    for (Pieces w(p, start); !w.done() && ok; w.next(), ++it) {
      const int J = w.tiles();
      auto page_of = [&](int row, bool on) -> int {  // a page that is not there: zeros (outside the tensor map)
        if (!on || row >= w.q.len) return p.s.n_pages;
        const int pg = paged_page(p.s, w.b, row);
        return pg < 0 ? p.s.n_pages : pg;
      };
      auto wait_slot = [&]() -> bool {
        return __all_sync(0xffffffffu,
                          mbar_wait(&bar.empty[u % kSlots], ((u / kSlots) & 1) ^ 1, &abort_flag, p.s.err));
      };
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.q_empty, (it & 1) ^ 1, &abort_flag, p.s.err));
      if (!ok) break;
      if (lane == 0) {
        if (rank == 0) mbar_arrive_expect_tx(&bar.q_full, (kPair ? 2 : 1) * kQBytes);
        const int tok = w.q.q0 + w.first_token() + (int)(rank << (7 - p.g_log2));
        for (int c = 0; c < 4; ++c) {
          if constexpr (kPair)
            tma_load_3d_pair(sQ + c * kQChunk, &map_q, cluster_addr(&bar.q_full, 0), c * 64, w.h << p.g_log2, tok);
          else
            tma_load_3d(sQ + c * kQChunk, &map_q, &bar.q_full, c * 64, w.h << p.g_log2, tok);
        }
      }
      __syncwarp();
      // the pages of the next K tile, and of a K tile's V (used a step later), are looked up once this
      // step's loads are on their way
      int pk = page_of(w.j0 * kKeyTile + k_row, kb.on), pv[Sh::kParts] = {};
      for (int step = 0; step <= J && ok; ++step) {
        const int j = w.j0 + step;
        if (step < J) {
#pragma unroll
          for (int part = 0; part < Sh::kParts && ok; ++part) {
            ok = wait_slot();
            if (!ok) break;
            const uint32_t s = u % kSlots;
            if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&bar.full[s], (kPair ? 2 : 1) * kSlotBytes);
            __syncwarp();
            if (kb.on)
              load_box<kPair>(sRing + s * kSlotBytes + kb.to, &map_k, &bar.full[s], (j * kKeyTile + k_row) & page_mask,
                              kPair ? kb.chunk : 2 * part + kb.chunk, w.h, pk);
            ++u;
          }
        }
        if (step >= 1) {
          const bool tail_tile = is_tail(w.q.len, j - 1);
#pragma unroll
          for (int part = 0; part < Sh::kParts && ok; ++part) {
            ok = wait_slot();
            if (!ok) break;
            const uint32_t s = u % kSlots;
            const int in = ((j - 1) * kKeyTile + v_row + 64 * part) & page_mask;
            uint8_t* dst = sRing + s * kSlotBytes + vb.to;
            const int chunk = kPair ? 2 * (int)rank + vb.chunk : vb.chunk;
            if (tail_tile && (kPair || part == tail_part(w.q.len))) {
              uint64_t* tail = &bar.v_tail[tails++ & 1];
              if (lane == 0) {
                mbar_arrive_expect_tx(tail, kSlotBytes);
                if (rank == 0) mbar_arrive(&bar.full[s]);
              }
              __syncwarp();
              if (vb.on) tma_load_5d(dst, &map_v, tail, 0, in, chunk, w.h, pv[part]);
            } else {
              if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&bar.full[s], (kPair ? 2 : 1) * kSlotBytes);
              __syncwarp();
              if (vb.on) load_box<kPair>(dst, &map_v, &bar.full[s], in, chunk, w.h, pv[part]);
            }
            ++u;
          }
        }
        if (step + 1 < J) pk = page_of((j + 1) * kKeyTile + k_row, kb.on);
        if (step < J) {
#pragma unroll
          for (int part = 0; part < Sh::kParts; ++part) pv[part] = page_of(j * kKeyTile + v_row + 64 * part, vb.on);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader CTA)
    // The whole warp walks and waits, one elected lane issues: the descriptors stay warp-uniform values.
    if (rank == 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(Sh::kRows, kKeyTile, false, false);
      constexpr uint32_t idesc_o = idesc_bf16_f32(Sh::kRows, kMlaD, false, true);
      const uint32_t sRa = smem_u32(sRing);
      const uint64_t dq = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(b, parity, &abort_flag, p.s.err));
      };
      uint32_t u = 0, it = 0, g = 0;  // g: key tiles so far (S buffer and barrier phases)
      bool ok = true;
      for (Pieces w(p, start); !w.done() && ok; w.next(), ++it) {
        const int J = w.tiles();
        ok = wait(&bar.q_full, it & 1);
        for (int step = 0; step <= J && ok; ++step) {
          if (step < J) {
            const uint32_t gs = g + step, tS = tmem + kTmemS + (gs & 1) * kKeyTile;
#pragma unroll
            for (int part = 0; part < Sh::kParts && ok; ++part) {
              const uint32_t s = u % kSlots;
              ok = wait(&bar.full[s], (u / kSlots) & 1);
              if (!ok) break;
              tc_fence_after();
              const uint64_t dk = smem_desc_sw128(sRa + s * kSlotBytes, 16, p.k_box.step);
              if (elect_one()) {
#pragma unroll
                for (int c = 0; c < 4 / Sh::kParts; ++c)
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk) {  // start addresses in 16-byte units
                    const uint64_t a = dq + (uint64_t)(((part * 2 + c) * kQChunk + kk * 32) >> 4);
                    const uint64_t b = dk + (uint64_t)((c * p.k_box.chunk + kk * 32) >> 4);
                    if constexpr (kPair) mma_ss_pair(tS, a, b, idesc_s, (part | c | kk) != 0);
                    else mma_ss(tS, a, b, idesc_s, (part | c | kk) != 0);
                  }
                commit<kPair>(&bar.empty[s]);
                if (part == Sh::kParts - 1) {
                  commit<kPair>(&bar.s_full[gs & 1]);
                  if (step == J - 1) commit<kPair>(&bar.q_empty);
                }
              }
              __syncwarp();
              ++u;
            }
          }
          if (step >= 1 && ok) {
            const uint32_t gj = g + step - 1;
            const uint32_t tP = tmem + kTmemS + (gj & 1) * kKeyTile;  // bf16 pairs: 64 columns
#pragma unroll
            for (int part = 0; part < Sh::kParts && ok; ++part) {
              const uint32_t s = u % kSlots;
              ok = wait(&bar.full[s], (u / kSlots) & 1);
              if (ok && part == 0)
                ok = kPair && is_tail(w.q.len, w.j0 + step - 1)
                         ? __all_sync(0xffffffffu,
                                      mbar_wait_cluster(&bar.p_ready[gj & 1], (gj >> 1) & 1, &abort_flag, p.s.err))
                         : wait(&bar.p_ready[gj & 1], (gj >> 1) & 1);
              if (!ok) break;
              tc_fence_after();
              const uint64_t dv = smem_desc_sw128(sRa + s * kSlotBytes, p.v_box.chunk, 1024);
              if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kKeyTile / 16 / Sh::kParts; ++kk) {
                  const uint32_t a = tP + (part * 4 + kk) * 8;
                  const uint64_t b = dv + (uint64_t)((kk * p.v_box.step) >> 4);
                  const uint32_t acc = (step > 1 || part > 0 || kk > 0) ? 1u : 0u;
                  if constexpr (kPair) mma_ts_pair(tmem, a, b, idesc_o, acc);
                  else mma_ts(tmem, a, b, idesc_o, acc);
                }
                commit<kPair>(&bar.empty[s]);
                if (part == Sh::kParts - 1) {
                  commit<kPair>(&bar.pv_done);
                  if (step == J) commit<kPair>(&bar.o_full);
                }
              }
              __syncwarp();
              ++u;
            }
          }
        }
        g += J;
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax and output
    // Two threads per row, lanes t and t + 16 of one warp (16 TMEM lanes of its quarter): half hf
    // takes keys 64 hf .. +63 of a tile and columns 128 hf .. +127 of the output.
    const int lane0 = (warp & 3) * 32 + ((warp - 4) >> 2) * 16, hf = lane >> 4;
    const int row = (int)rank * 128 + lane0 + (lane & 15);  // row of the row tile
    const int my_tok = row >> p.g_log2, my_head = row & ((1 << p.g_log2) - 1);
    const uint32_t t_lanes = tmem + (static_cast<uint32_t>(lane0) << 16);
    const int tid = threadIdx.x - 128;
    const uint32_t ready0 = cluster_addr(&bar.p_ready[0], 0);
    uint32_t g = 0, u = 0, tails = 0, pieces = 0;
    bool ok = true;
    int head_flag = 0, tail_flag = 0, tail_tok = 0, tail_n = 0, tail_h = 0;  // for ws_meta
    for (Pieces w(p, start); !w.done(); w.next()) {
      const int J = w.tiles();
      const int tok = w.first_token() + my_tok;  // token of the sequence
      const bool valid = tok < w.q.n;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      const int n_vis = min(w.q.base + tok + 1, w.q.len) - 64 * hf;  // rows this row sees (may be <= 0)
      float m_run = -INFINITY, l_run = 0.0f;
      for (int jj = 0; jj < J; ++jj, ++g) {
        const int j = w.j0 + jj;
        ok = mbar_wait(&bar.s_full[g & 1], (g >> 1) & 1, &abort_flag, p.s.err) && ok;
        tc_fence_after();
        if (warp_valid) {
          const uint32_t tS = t_lanes + kTmemS + (g & 1) * kKeyTile;
          uint32_t s[2][32];
          tmem_ld_half32<64>(tS, s[0]);
          tmem_ld_half32<64>(tS + 32, s[1]);
          tmem_wait_ld_regs2(s[0], s[1]);
          const int vis = n_vis - j * kKeyTile;
          if (!__all_sync(0xffffffffu, vis >= 64)) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (c * 32 + x >= vis) s[c][x] = 0xff800000u;
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int x = 0; x < 16; ++x)
#pragma unroll
            for (int c = 0; c < 4; ++c) m4[c] = fmaxf(m4[c], __uint_as_float(s[c >> 1][2 * x + (c & 1)]));
          const float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          const float xt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16)) * p.scale_log2;
          bool resc = false;
          float alpha = 1.0f;
          if (m_run == -INFINITY) {
            m_run = xt;  // nothing visible so far: O is all zeros, or not yet written
          } else if (xt > m_run + kLazyRescale) {
            alpha = fast_exp2(m_run - xt);
            m_run = xt;
            resc = true;
          }
          const float m_ref = m_run == -INFINITY ? 0.0f : m_run;
          l_run *= alpha;
          float l4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pw[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float p0 = fast_exp2(fmaf(__uint_as_float(s[c][2 * x]), p.scale_log2, -m_ref));
              const float p1 = fast_exp2(fmaf(__uint_as_float(s[c][2 * x + 1]), p.scale_log2, -m_ref));
              l4[(2 * x) & 3] += p0;
              l4[(2 * x + 1) & 3] += p1;
              pw[x] = pack_bf16x2(p0, p1);
            }
            tmem_st_half16<32>(tS + c * 16, pw);
          }
          l_run += (l4[0] + l4[1]) + (l4[2] + l4[3]);
          if (__any_sync(0xffffffffu, resc)) {
            // O holds every PV of this piece up to the previous tile; this tile's waits for p_ready
            ok = mbar_wait(&bar.pv_done, (g - 1) & 1, &abort_flag, p.s.err) && ok;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tmem_ld_half32<128>(t_lanes + c * 32, o);
              tmem_wait_ld_regs(o);
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
              tmem_st_half32<128>(t_lanes + c * 32, o);
            }
          }
          tmem_wait_st();
        }
        const bool tail = is_tail(w.q.len, j);
        if (tail) {
          // V of the piece's last tile: clear the rows behind the sequence's end, up to the box's end
          ok = mbar_wait(&bar.v_tail[tails & 1], (tails >> 1) & 1, &abort_flag, p.s.err) && ok;
          ++tails;
          const int r0 = w.q.len & (kKeyTile - 1), r1 = (r0 + box_rows - 1) & ~(box_rows - 1);
          const int part = kPair ? 0 : tail_part(w.q.len);
          constexpr int kRowPieces = kPair ? 16 : 32;  // 16-byte pieces of a row in the slot
          uint8_t* slot = sRing + ((u + (2 * J - 1) * Sh::kParts + part) % kSlots) * kSlotBytes;
          for (int e = tid; e < (r1 - r0) * kRowPieces; e += 32 * kSoftmaxWarps) {
            const int r = r0 + e / kRowPieces - 64 * part, x = e % kRowPieces;
            *reinterpret_cast<uint4*>(slot + (x >> 3) * p.v_box.chunk + (r >> 4) * p.v_box.step + (r & 15) * 128 +
                                      (x & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair) {
            const uint32_t ready = ready0 + (g & 1) * 8;
            if (tail) arrive_cluster(ready);  // shared memory was written
            else arrive_cluster_relaxed(ready);
          } else {
            mbar_arrive(&bar.p_ready[g & 1]);
          }
        }
      }
      u += 2 * J * Sh::kParts;
      // ---- output of the piece, once its last PV is done.  (Not on pv_done: a phase of a barrier may only
      // be waited for by its parity if the one before it is known to be complete.)
      ok = mbar_wait(&bar.o_full, pieces & 1, &abort_flag, p.s.err) && ok;
      ++pieces;
      tc_fence_after();
      const bool whole = w.j0 == 0 && w.j1 == w.n_keys;
      if (warp_valid) {
        const float l = l_run + __shfl_xor_sync(0xffffffffu, l_run, 16);
        const size_t orow = (size_t)(w.q.q0 + tok) * p.Hq + (w.h << p.g_log2) + my_head;
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // (a NaN stays one: O and lse show it)
        const int slot = 2 * worker + (w.j0 == 0 ? 1 : 0);
        if (valid && hf == 0) {
          if (whole) {
            if (p.lse) p.lse[orow] = l != 0.0f ? (m_run + __log2f(l)) * 0.69314718055994531f : -INFINITY;
          } else {
            p.ws_ml[(size_t)slot * 2 * Sh::kRows + row] = m_run;
            p.ws_ml[(size_t)slot * 2 * Sh::kRows + Sh::kRows + row] = l;
          }
        }
#pragma unroll 1
        for (int c0 = 0; c0 < 4; c0 += 2) {  // 64 columns in flight: a TMEM load takes about 600 cycles
          uint32_t o[2][32];
          tmem_ld_half32<128>(t_lanes + c0 * 32, o[0]);
          tmem_ld_half32<128>(t_lanes + c0 * 32 + 32, o[1]);
          tmem_wait_ld_regs2(o[0], o[1]);
          // Four lanes exchange their 32-byte pieces, so that each store fills lines of 128 bytes (18 tokens of
          // 128 heads over up to 2245 rows 26.8 us against 30.8, two short conversations 14.4 against 16.4).
          const int n_valid = (w.q.n - w.first_token()) << p.g_log2, row4 = row & ~3, quarter = lane & 3;
          if (whole) {
            uint32_t v[32];
#pragma unroll
            for (int y = 0; y < 32; ++y) {
              const uint32_t* q = &o[y >> 4][2 * (y & 15)];
              v[y] = pack_bf16x2(__uint_as_float(q[0]) * inv, __uint_as_float(q[1]) * inv);
            }
            transpose_4(v, lane);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = row4 + k;
              if (r >= n_valid) break;
              const size_t at = (size_t)(w.q.q0 + w.first_token() + (r >> p.g_log2)) * p.Hq + (w.h << p.g_log2) +
                                (r & ((1 << p.g_log2) - 1));
              uint16_t* dst = p.O + at * kMlaD + hf * 128 + c0 * 32 + 16 * quarter;
              if (p.wide_stores) {
                store_32(dst, &v[8 * k]);
              } else {
                reinterpret_cast<uint4*>(dst)[0] = make_uint4(v[8 * k], v[8 * k + 1], v[8 * k + 2], v[8 * k + 3]);
                reinterpret_cast<uint4*>(dst)[1] = make_uint4(v[8 * k + 4], v[8 * k + 5], v[8 * k + 6], v[8 * k + 7]);
              }
            }
          } else {
            float* dst = p.ws_O + ((size_t)slot * Sh::kRows + row4) * kMlaD + hf * 128 + c0 * 32 + 8 * quarter;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              transpose_4(o[x], lane);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (row4 + k < n_valid) store_32(dst + k * kMlaD + 32 * x, &o[x][8 * k]);
            }
          }
          __syncwarp();
        }
      }
      if (!whole) {
        if (w.j0 > 0) {
          head_flag = w.j1 == w.n_keys ? 2 : 1;
        } else {
          tail_flag = 1;
          tail_tok = w.q.q0 + w.first_token();
          tail_n = min(1 << w.tq_log2, w.q.n - w.first_token());
          tail_h = w.h;
        }
      }
    }
    if (rank == 0 && tid == 0) {
      int* m = p.ws_meta + worker * kMetaInts;
      m[0] = head_flag;
      m[1] = tail_flag;
      m[2] = tail_tok;
      m[3] = tail_n;
      m[4] = tail_h;
    }
  }

  launch_dependents();
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // no MMA of the pair and no cross-CTA arrival is pending any more
  tc_fence_after();
  if (warp == 1) {
    if constexpr (kPair) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
}

// Merges the pieces of a row tile that began in worker c's range and went on in those of workers
// c+1, c+2, ... (piece k >= 1 is the one worker c + k began with), in that order: with M the largest
// of the maxima,
//     O = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k.
// A piece that sees no row has l_k = 0 and no weight; one with a NaN among its scores has l_k = NaN, which
// reaches the row's O and lse through the denominator.
// Every block lists the row tiles to merge from the workers' records and takes its share of the work
// items: with up to `few` pieces an item is 8 rows, one warp each; with more (a long cache cut over
// many workers) it is one row, whose pieces the 8 warps divide among themselves and add up through
// shared memory, in warp order.  `few` is 8, or 32 where there are twice as many rows as blocks,
// which one warp per row keeps busy (124 tokens over 1747 rows, 16 K/V heads: 33.5 us against 43; but 5
// tokens of 128 heads over up to 7209 rows 31.7 against 28.7, with 640 rows for 592 blocks).  Lane l holds
// columns 8 l .. 8 l + 7; the lanes read the pieces' (max, sum) side by side, so the loads of the rows
// do not wait on one another.
// (One sequence of 32768 rows cut into 148 pieces of 64 rows: one warp per row took 30 us of the call's 47.)
constexpr int kCombineWarps = 8;
constexpr int kMaxWorkers = 160;

// Columns 8 l .. 8 l + 7 of piece k's row, added to acc with weight w.
__device__ __forceinline__ void add_piece(const float4& a, const float4& b, float w, float (&acc)[8]) {
  if (w > 0.0f) {  // a piece without weight may hold anything
    acc[0] = fmaf(w, a.x, acc[0]);
    acc[1] = fmaf(w, a.y, acc[1]);
    acc[2] = fmaf(w, a.z, acc[2]);
    acc[3] = fmaf(w, a.w, acc[3]);
    acc[4] = fmaf(w, b.x, acc[4]);
    acc[5] = fmaf(w, b.y, acc[5]);
    acc[6] = fmaf(w, b.z, acc[6]);
    acc[7] = fmaf(w, b.w, acc[7]);
  }
}

__global__ void __launch_bounds__(32 * kCombineWarps, 4)
    combine_kernel(const Params p, int n_workers, int n_rows, int few_pieces) {
  __shared__ int pieces_of[kMaxWorkers], first_item[kMaxWorkers + 1];
  __shared__ int4 tile_of[kMaxWorkers];  // first packed token, tokens, K/V head
  __shared__ uint32_t ends[kMaxWorkers / 32];  // bit c: worker c's first piece, if any, is the last of its row tile
  __shared__ float weight[kMaxWorkers], red[2][kCombineWarps], part[kCombineWarps][kMlaD];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  wait_for_primary();
  // ---- row tiles to merge: their pieces and work items, and the prefix of the items
  const int* mine = p.ws_meta + tid * kMetaInts;
  const int head = tid < n_workers ? mine[0] : 2, tail = tid < n_workers ? mine[1] : 0;
  const int rows = tail ? mine[3] << p.g_log2 : 0;
  const uint32_t end_bits = __ballot_sync(0xffffffffu, head != 1);
  if (lane == 0 && warp < kMaxWorkers / 32) ends[warp] = end_bits;
  __syncthreads();
  if (tid < kMaxWorkers) {
    int items = 0;
    if (tail) {
      int c = tid + 1;  // the first worker from here on whose first piece ends the tile
      while (c < n_workers) {
        const uint32_t left = ends[c >> 5] >> (c & 31);
        if (left) {
          c += __ffs(left) - 1;
          break;
        }
        c = (c | 31) + 1;
      }
      const int n = min(c, n_workers - 1) - tid + 1;
      pieces_of[tid] = n;
      tile_of[tid] = make_int4(mine[2], mine[3], mine[4], 0);
      items = n <= few_pieces ? (rows + kCombineWarps - 1) / kCombineWarps : rows;
    }
    first_item[tid + 1] = items;
    if (tid == 0) first_item[0] = 0;
  }
  __syncthreads();
  if (warp == 0) {
    int run = 0;
#pragma unroll
    for (int w0 = 0; w0 < kMaxWorkers; w0 += 32) {
      int x = first_item[w0 + lane + 1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      first_item[w0 + lane + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  const int total = first_item[kMaxWorkers];
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    int c = 0, hi = kMaxWorkers;  // the last worker whose items begin at or before this one
    while (hi - c > 1) {
      const int mid = (c + hi) >> 1;
      if (first_item[mid] <= item) c = mid;
      else hi = mid;
    }
    const int4 tile = tile_of[c];
    const int n = pieces_of[c];
    const bool few = n <= few_pieces;
    const int row = few ? (item - first_item[c]) * kCombineWarps + warp : item - first_item[c];
    const int tok = row >> p.g_log2;
    auto slot = [&](int k) { return (size_t)(k ? 2 * (c + k) : 2 * c + 1); };
    auto row_of = [&](int k) {
      return reinterpret_cast<const float4*>(p.ws_O + (slot(k) * n_rows + row) * kMlaD + lane * 8);
    };
    float M, den, acc[8] = {};
    if (few) {
      if (tok >= tile.y) continue;
      float m = -INFINITY, l = 0.0f;
      if (lane < n) {
        const float* ml = p.ws_ml + slot(lane) * 2 * n_rows + row;
        m = ml[0];
        l = ml[n_rows];
      }
      M = l != 0.0f ? m : -INFINITY;
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float w_mine = l != 0.0f ? exp2f(m - M) : 0.0f;
      den = 0.0f;
#pragma unroll 4
      for (int k = 0; k < n; ++k) {
        const float w = __shfl_sync(0xffffffffu, w_mine, k), lk = __shfl_sync(0xffffffffu, l, k);
        const float4 a = row_of(k)[0], b = row_of(k)[1];
        den = fmaf(w, lk, den);
        add_piece(a, b, w, acc);
      }
    } else {
      // thread k: piece k's maximum and sum, then its weight
      float m = -INFINITY, l = 0.0f;
      if (tid < n) {
        const float* ml = p.ws_ml + slot(tid) * 2 * n_rows + row;
        m = ml[0];
        l = ml[n_rows];
      }
      M = l != 0.0f ? m : -INFINITY;
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      __syncthreads();  // the item before has been read
      if (lane == 0) red[0][warp] = M;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kCombineWarps; ++w) M = fmaxf(M, red[0][w]);
      const float w_mine = l != 0.0f ? exp2f(m - M) : 0.0f;
      if (tid < n) weight[tid] = w_mine;
      den = w_mine * l;
#pragma unroll
      for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
      if (lane == 0) red[1][warp] = den;
      __syncthreads();
#pragma unroll 8
      for (int k = warp; k < n; k += kCombineWarps) {
        const float4 a = row_of(k)[0], b = row_of(k)[1];
        add_piece(a, b, weight[k], acc);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) part[warp][lane * 8 + x] = acc[x];
      __syncthreads();
      if (warp != 0) continue;
      den = 0.0f;
#pragma unroll
      for (int w = 0; w < kCombineWarps; ++w) den += red[1][w];
#pragma unroll
      for (int w = 1; w < kCombineWarps; ++w)
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[x] += part[w][lane * 8 + x];
    }
    const float inv = den != 0.0f ? 1.0f / den : 0.0f;
    const size_t orow = (size_t)(tile.x + tok) * p.Hq + (tile.z << p.g_log2) + (row & ((1 << p.g_log2) - 1));
    uint4 v;
    v.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    v.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
    v.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
    v.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
    reinterpret_cast<uint4*>(p.O + orow * kMlaD)[lane] = v;
    if (p.lse && lane == 0) p.lse[orow] = den != 0.0f ? (M + __log2f(den)) * 0.69314718055994531f : -INFINITY;
  }
}

// SMs of the current device, its kernels' shared memory set up.
int sms_of_device() {
  static std::mutex mu;
  static int cache[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (!cache[dev]) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 2 ||
        cudaFuncSetAttribute(attn_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) !=
            cudaSuccess ||
        cudaFuncSetAttribute(attn_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) !=
            cudaSuccess) {
      launch_status();
      return 0;
    }
    cache[dev] = sms < kMaxWorkers ? sms : kMaxWorkers;
  }
  return cache[dev];
}

// The same for both kernels: half as many pairs, each with twice the rows.
size_t workspace_bytes_of(int sms) {
  return (size_t)sms * (2 * ((size_t)kCtaRows * kMlaD * 4 + 2 * kCtaRows * 4) + kMetaInts * 4);
}

// Pairs take row tiles of 256 rows and load half the K and V per product; single CTAs take row tiles
// of 128 rows, so a sequence that has no more rows than that (a decode step) costs half the MMA time.
// Both give right results for every batch; the host only knows the averages.  Measured, pairs and
// single CTAs: 32 decode steps over 1K-32K rows 116 and 106 us; two 389-token chunks next to 22
// decode steps (266 rows per sequence on average) 211 and 233 us; 2048 tokens over 32768 rows 2.8 and
// 3.6 ms.
bool use_pairs(int B, int T, int g) { return (long long)T * g > (long long)kCtaRows * B; }

// A box holds 64 rows of one chunk of 64 columns, or a page's.  A TMA copy costs some 95 cycles however
// small, so that 2 KB boxes of 16-row pages would take longer than a pair's MMAs: there a box is 8 rows of
// all of a pair's K chunks, which keeps the groups of 8 rows evenly apart, as the MMA's descriptor wants
// them, or a page's V rows of all chunks, which are the keys of one MMA step.
// (512 tokens over 8192 rows of 16-row pages 194 us against 236, one token of 16 sequences over 16384
// rows each 68 against 72; larger pages gain nothing from it.)
template <bool kPair>
void box_layouts(int page, BoxLayout* k, BoxLayout* v) {
  const bool small = page < 32;
  const int rows = page < 64 ? log2_of(page) : 6, kc = Shape<kPair>::kKChunksLog2, vc = Shape<kPair>::kVChunksLog2;
  *k = small && kPair ? BoxLayout{3, kc, 1024 << kc, 1024} : BoxLayout{rows, 0, 1024, kSlotBytes >> kc};
  *v = small ? BoxLayout{4, vc, 2048 << vc, 2048} : BoxLayout{rows, 0, 2048, kSlotBytes >> vc};
}

template <bool kPair>
hcadsa_status launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, Params p, int sms,
                     cudaStream_t stream) {
  const int workers = kPair ? sms / 2 : sms, blocks = 4 * sms;  // (of the merge)
  const long long all_rows = (long long)p.s.T * p.Hq;
  const long long rows = ((long long)p.s.T << p.g_log2) / p.s.B;
  p.piece_rows = all_rows <= blocks ? 0 : (int)(rows < Shape<kPair>::kRows ? rows : Shape<kPair>::kRows);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPair ? 2 * workers : workers, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kPair ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, attn_kernel<kPair>, mq, mk, mv, p) != cudaSuccess) return launch_status();
  return launch_after(combine_kernel, dim3(blocks), 32 * kCombineWarps, stream, p, workers, (int)Shape<kPair>::kRows,
                      all_rows > 2 * blocks ? 32 : 8);
}

}  // namespace
}  // namespace hcadsa

extern "C" size_t mla_paged_attn_fwd_workspace_size(int B, int T, int Hq, int Hkv) {
  using namespace hcadsa;
  if (B <= 0 || T <= 0 || Hkv <= 0 || check_query_sizes(T, Hq, Hkv, kMlaD, 1.0f) != HCADSA_OK) return 0;
  return workspace_bytes_of(sms_of_device());
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
  const int sms = sms_of_device();
  if (sms <= 0) return HCADSA_ERR_CUDA;
  if (!workspace || workspace_bytes < workspace_bytes_of(sms)) return HCADSA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 31u) return HCADSA_ERR_ALIGN;
  Params p;
  p.s = paged_batch(table, cu_q, kv_len, B, T, n_pages, page, max_pages);
  p.O = O;
  p.lse = lse;
  p.ws_O = static_cast<float*>(workspace);
  p.ws_ml = p.ws_O + (size_t)2 * sms * kCtaRows * kMlaD;
  p.ws_meta = reinterpret_cast<int*>(p.ws_ml + (size_t)2 * sms * 2 * kCtaRows);
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.g_log2 = log2_of(Hq / Hkv);
  const bool pairs = use_pairs(B, T, Hq / Hkv);
  if (pairs) box_layouts<true>(page, &p.k_box, &p.v_box);
  else box_layouts<false>(page, &p.k_box, &p.v_box);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wide_stores = (reinterpret_cast<uintptr_t>(O) & 31u) == 0;
  CUtensorMap mq, mk, mv;
  {
    const int g = 1 << p.g_log2;
    const uint64_t dims[3] = {(uint64_t)kMlaD, (uint64_t)Hq, (uint64_t)T};
    const uint64_t strides[2] = {(uint64_t)kMlaD * 2, (uint64_t)q_row_stride * 2};
    const uint32_t box[3] = {64, (uint32_t)g, (uint32_t)(128 / g)};
    if (!encode_tmap_bf16(&mq, 3, const_cast<hcadsa_bf16*>(Q), dims, strides, box, true)) return HCADSA_ERR_CUDA;
  }
  for (int v = 0; v < 2; ++v) {
    const BoxLayout& x = v ? p.v_box : p.k_box;
    const uint64_t dims[5] = {64, (uint64_t)page, kMlaD / 64, (uint64_t)Hkv, (uint64_t)n_pages};
    const uint64_t strides[4] = {(uint64_t)Hkv * kMlaD * 2, 64 * 2, (uint64_t)kMlaD * 2,
                                 (uint64_t)(v ? v_page_stride : k_page_stride) * 2};
    const uint32_t box[5] = {64, 1u << x.rows_log2, 1u << x.chunks_log2, 1, 1};
    if (!encode_tmap_bf16(v ? &mv : &mk, 5, const_cast<hcadsa_bf16*>(v ? V_pool : K_pool), dims, strides, box, true))
      return HCADSA_ERR_CUDA;
  }
  return pairs ? launch<true>(mq, mk, mv, p, sms, as_stream(stream))
               : launch<false>(mq, mk, mv, p, sms, as_stream(stream));
}
