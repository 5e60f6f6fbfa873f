// mla_cache.cu -- writes to the paged cache of the full-context (MLA) layers: a chunk's new rows
// (mla_cache_append) and the moves that close the gaps an eviction left (mla_cache_move).
//
// Method: the mirrorspeed page, section "Hybrid sparse attention, 1/7 full context access": the
// MLA layers keep every token's K and V.  A cache row is 256 bf16 per K/V head in each pool.
//
// Both kernels only copy 512-byte rows (one warp instruction: lane l moves bytes 16 l .. 16 l + 15),
// so their bound is HBM: 1 KB read and 1 KB written per pair of K and V rows.  Measured (B200): 16384 tokens of
// 4 K/V heads appended in 27 us (5.0 TB/s of the 135 MB), 98284 moves in 41 us (5.0 TB/s); 4, 8 and
// 16 moves per warp 43, 41 and 51 us; 4, 8 and 16 tokens per block 29, 27 and 29 us.
#include "mla_host.h"

namespace hcadsa {
namespace {

constexpr int kWarps = 8;
constexpr int kTokens = 8;  // new tokens of a block

struct AppendParams {
  PagedBatch s;
  const uint16_t* K;
  const uint16_t* V;
  uint16_t* K_pool;
  uint16_t* V_pool;
  const int32_t* seen;
  int32_t* pos;
  float* mass;
  long long k_row, v_row, k_page, v_page;  // strides in elements
  int Hkv;
};

// A block owns kTokens packed tokens: all its threads look for the sequences that own them (one
// pass over cu_q, no search chain) while the first K and V rows are on their way, one thread per
// token looks up where it goes, and the warps copy one (token, head) after the other, kAhead rows
// of each pool in flight.
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const AppendParams p) {
  __shared__ int owner[kTokens];
  __shared__ int page_of[kTokens], place_of[kTokens];  // where the token's row goes; page -1: nowhere
  const int t0 = blockIdx.x * kTokens, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int units = min(kTokens, p.s.T - t0) * p.Hkv;
  constexpr int kAhead = 4;
  uint4 k[kAhead], v[kAhead];
  auto load = [&](int u0) {
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int u = u0 + x * kWarps;
      if (u >= units) continue;
      const int i = u / p.Hkv, h = u - i * p.Hkv;
      k[x] = reinterpret_cast<const uint4*>(p.K + (size_t)(t0 + i) * p.k_row + (size_t)h * kMlaD)[lane];
      v[x] = reinterpret_cast<const uint4*>(p.V + (size_t)(t0 + i) * p.v_row + (size_t)h * kMlaD)[lane];
    }
  };
  load(warp);
  if (threadIdx.x < kTokens) owner[threadIdx.x] = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < p.s.B; b += blockDim.x) {
    const PagedSeq q = paged_seq(p.s, b, blockIdx.x == 0);
    const int a = max(q.q0, t0), z = min(q.q0 + q.n, t0 + kTokens);
    for (int t = a; t < z; ++t) owner[t - t0] = b;
  }
  __syncthreads();
  const int page_mask = (1 << p.s.page_log2) - 1;
  if (threadIdx.x < kTokens) {
    const int b = owner[threadIdx.x];
    int pg = -1, r = 0;
    if (b >= 0) {  // otherwise a packed row behind the last sequence
      // from the declared end, not the clamped one: a row without a place in the table may not take
      // the place of another
      const long long back = (long long)p.s.cu_q[b + 1] - (t0 + (int)threadIdx.x);  // rows from this one to the end
      const long long at = p.s.kv_len[b] - back;
      if (at >= 0 && at < (long long)p.s.max_pages << p.s.page_log2) {
        r = (int)at;
        pg = paged_page(p.s, b, r);
      } else {
        raise_device_error(p.s.err, kErrDeviceBounds);
      }
      if (pg >= 0) {
        const size_t slot = (((size_t)pg << p.s.page_log2) + (r & page_mask)) * p.Hkv;
        const int ps = p.seen ? (int)(p.seen[b] - back) : r;
        for (int h = 0; h < p.Hkv; ++h) {
          if (p.pos) p.pos[slot + h] = ps;
          if (p.mass) p.mass[slot + h] = 0.0f;
        }
      }
    }
    page_of[threadIdx.x] = pg;
    place_of[threadIdx.x] = r & page_mask;
  }
  __syncthreads();
  for (int u0 = warp; u0 < units; u0 += kAhead * kWarps) {
    if (u0 != warp) load(u0);
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int u = u0 + x * kWarps;
      if (u >= units) continue;
      const int i = u / p.Hkv, h = u - i * p.Hkv, pg = page_of[i];
      if (pg < 0) continue;
      const size_t row = ((size_t)place_of[i] * p.Hkv + h) * kMlaD;
      reinterpret_cast<uint4*>(p.K_pool + (size_t)pg * p.k_page + row)[lane] = k[x];
      reinterpret_cast<uint4*>(p.V_pool + (size_t)pg * p.v_page + row)[lane] = v[x];
    }
  }
}

struct MoveParams {
  PagedBatch s;
  const int2* moves;  // [B, Hkv, n_moves] (from, to)
  uint16_t* K_pool;
  uint16_t* V_pool;
  int32_t* pos;
  float* mass;
  long long k_page, v_page;
  int Hkv, n_moves, blocks_per_list;
};

constexpr int kMovesPerWarp = 8;

// A warp takes 8 consecutive entries of one list: lane i < 8 reads entry i and looks both rows'
// pages up, then all 16 row loads are in flight before the first store.
__global__ void __launch_bounds__(32 * kWarps) move_kernel(const MoveParams p) {
  const int list = blockIdx.x / p.blocks_per_list, part = blockIdx.x - list * p.blocks_per_list;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i0 = (part * kWarps + warp) * kMovesPerWarp;
  if (i0 >= p.n_moves) return;
  const int b = list / p.Hkv, h = list - b * p.Hkv;
  const int cap = p.s.max_pages << p.s.page_log2, page_mask = (1 << p.s.page_log2) - 1;
  // pool row numbers (page << page_log2 | place) of this lane's entry; -1: nothing to move
  long long from = -1, to = -1;
  if (lane < kMovesPerWarp && i0 + lane < p.n_moves) {
    const int2 m = p.moves[(size_t)list * p.n_moves + i0 + lane];
    if (m.x >= 0 && m.y >= 0) {
      if (m.x < cap && m.y < cap) {
        const int pf = paged_page(p.s, b, m.x), pt = paged_page(p.s, b, m.y);
        if (pf >= 0 && pt >= 0) {
          from = ((long long)pf << p.s.page_log2) + (m.x & page_mask);
          to = ((long long)pt << p.s.page_log2) + (m.y & page_mask);
        }
      } else {
        raise_device_error(p.s.err, kErrDeviceBounds);
      }
    }
  }
  if (!__any_sync(0xffffffffu, from >= 0)) return;
  if (from >= 0) {
    const size_t sf = (size_t)from * p.Hkv + h, st = (size_t)to * p.Hkv + h;
    if (p.pos) p.pos[st] = p.pos[sf];
    if (p.mass) p.mass[st] = p.mass[sf];
  }
  uint4 k[kMovesPerWarp], v[kMovesPerWarp];
#pragma unroll
  for (int i = 0; i < kMovesPerWarp; ++i) {
    const long long f = __shfl_sync(0xffffffffu, from, i);
    if (f < 0) continue;
    const size_t pg = (size_t)(f >> p.s.page_log2), row = (size_t)((int)f & page_mask) * p.Hkv + h;
    k[i] = reinterpret_cast<const uint4*>(p.K_pool + pg * p.k_page + row * kMlaD)[lane];
    v[i] = reinterpret_cast<const uint4*>(p.V_pool + pg * p.v_page + row * kMlaD)[lane];
  }
#pragma unroll
  for (int i = 0; i < kMovesPerWarp; ++i) {
    const long long f = __shfl_sync(0xffffffffu, from, i), t = __shfl_sync(0xffffffffu, to, i);
    if (f < 0) continue;
    const size_t pg = (size_t)(t >> p.s.page_log2), row = (size_t)((int)t & page_mask) * p.Hkv + h;
    reinterpret_cast<uint4*>(p.K_pool + pg * p.k_page + row * kMlaD)[lane] = k[i];
    reinterpret_cast<uint4*>(p.V_pool + pg * p.v_page + row * kMlaD)[lane] = v[i];
  }
}

}  // namespace
}  // namespace hcadsa

extern "C" hcadsa_status mla_cache_append(const hcadsa_bf16* K, const hcadsa_bf16* V, long long k_row_stride,
                                          long long v_row_stride, hcadsa_bf16* K_pool, hcadsa_bf16* V_pool,
                                          long long k_page_stride, long long v_page_stride, const int32_t* table,
                                          const int32_t* cu_q, const int32_t* kv_len, const int32_t* seen,
                                          int32_t* pos, float* mass, int B, int T, int n_pages, int page,
                                          int max_pages, int Hkv, int d, hcadsa_stream stream) {
  using namespace hcadsa;
  if (T < 0) return HCADSA_ERR_SHAPE;
  if (B > 0 && T > 0 && (!K || !V || !K_pool || !V_pool || !table || !cu_q || !kv_len)) return HCADSA_ERR_NULL;
  HCADSA_TRY(check_paged_sizes(B, n_pages, page, max_pages, Hkv));
  if (d != kMlaD) return HCADSA_ERR_UNSUPPORTED;
  HCADSA_TRY(check_row_stride(k_row_stride, Hkv));
  HCADSA_TRY(check_row_stride(v_row_stride, Hkv));
  HCADSA_TRY(check_page_stride(k_page_stride, page, Hkv));
  HCADSA_TRY(check_page_stride(v_page_stride, page, Hkv));
  if (!aligned16(K) || !aligned16(V) || !aligned16(K_pool) || !aligned16(V_pool) || !aligned4(table) ||
      !aligned4(cu_q) || !aligned4(kv_len) || !aligned4(seen) || !aligned4(pos) || !aligned4(mass))
    return HCADSA_ERR_ALIGN;
  if (B == 0 || T == 0) return HCADSA_OK;
  AppendParams p;
  p.s = paged_batch(table, cu_q, kv_len, B, T, n_pages, page, max_pages);
  p.K = K;
  p.V = V;
  p.K_pool = K_pool;
  p.V_pool = V_pool;
  p.seen = seen;
  p.pos = pos;
  p.mass = mass;
  p.k_row = k_row_stride;
  p.v_row = v_row_stride;
  p.k_page = k_page_stride;
  p.v_page = v_page_stride;
  p.Hkv = Hkv;
  append_kernel<<<(T + kTokens - 1) / kTokens, 32 * kWarps, 0, as_stream(stream)>>>(p);
  return launch_status();
}

extern "C" hcadsa_status mla_cache_move(const int32_t* moves, const int32_t* table, hcadsa_bf16* K_pool,
                                        hcadsa_bf16* V_pool, long long k_page_stride, long long v_page_stride,
                                        int32_t* pos, float* mass, int B, int n_moves, int n_pages, int page,
                                        int max_pages, int Hkv, int d, hcadsa_stream stream) {
  using namespace hcadsa;
  if (n_moves < 0) return HCADSA_ERR_SHAPE;
  if (B > 0 && n_moves > 0 && (!moves || !table || !K_pool || !V_pool)) return HCADSA_ERR_NULL;
  HCADSA_TRY(check_paged_sizes(B, n_pages, page, max_pages, Hkv));
  if (d != kMlaD) return HCADSA_ERR_UNSUPPORTED;
  HCADSA_TRY(check_page_stride(k_page_stride, page, Hkv));
  HCADSA_TRY(check_page_stride(v_page_stride, page, Hkv));
  if (!aligned16(K_pool) || !aligned16(V_pool) || (reinterpret_cast<uintptr_t>(moves) & 7u) || !aligned4(table) ||
      !aligned4(pos) || !aligned4(mass))
    return HCADSA_ERR_ALIGN;
  if (B == 0 || n_moves == 0) return HCADSA_OK;
  MoveParams p;
  p.s = paged_batch(table, nullptr, nullptr, B, 0, n_pages, page, max_pages);
  p.moves = reinterpret_cast<const int2*>(moves);
  p.K_pool = K_pool;
  p.V_pool = V_pool;
  p.pos = pos;
  p.mass = mass;
  p.k_page = k_page_stride;
  p.v_page = v_page_stride;
  p.Hkv = Hkv;
  p.n_moves = n_moves;
  p.blocks_per_list = (n_moves - 1) / (kWarps * kMovesPerWarp) + 1;
  const long long blocks = (long long)B * Hkv * p.blocks_per_list;
  if (blocks > 2147483647LL) return HCADSA_ERR_UNSUPPORTED;
  move_kernel<<<(unsigned)blocks, 32 * kWarps, 0, as_stream(stream)>>>(p);
  return launch_status();
}
