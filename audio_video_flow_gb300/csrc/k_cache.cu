// The paged cache of keys and values: append of new rows, the attention weight
// that each cached row collects, and eviction by that weight.
//   pages    [n_pages][n_kv_heads][page_size][128] bf16, one array each for K
//            and V; a head's rows of a page are contiguous
//   weights  [n_pages][n_kv_heads][page_size] fp32
#include "attention_device.cuh"
#include "h3_internal.h"

#include <cmath>

namespace h3 {

namespace {
// Element offset of a slot's row in the pages (of 128 channels; of 1 in the
// weights).
__device__ __forceinline__ int64_t page_row(const CacheArgs& c, int page, int head, int slot) {
  return ((int64_t)page * c.n_kv_heads + head) * c.page_size + slot % c.page_size;
}
__device__ __forceinline__ int page_of(const CacheArgs& c, int seq, int slot) {
  return c.table[(int64_t)seq * c.table_width + slot / c.page_size];
}
__device__ __forceinline__ int64_t cache_slots(const CacheArgs& c) { return (int64_t)c.table_width * c.page_size; }
}  // namespace

// ---------------------------------------------------------------------------
// Append: row i of sequence s, the rows-before-it-in-s'th of its new ones, goes
// to slot length[s] - new + that.  A warp copies one row of one head: K by the
// lower, V by the upper half of its lanes.  Bound by HBM (or by its launch).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) cache_append_kernel(const AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t units = (int64_t)a.n_rows * a.c.n_kv_heads;
  const int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (u >= units) return;
  const int row = (int)(u / a.c.n_kv_heads), head = (int)(u - (int64_t)row * a.c.n_kv_heads);
  int s = -1;
  for (int lo = 0, hi = a.c.n_seqs - 1; lo <= hi;) {   // the last sequence that starts at or before the row
    const int mid = (lo + hi) >> 1;
    if (a.c.start[mid] <= row) { s = mid; lo = mid + 1; } else { hi = mid - 1; }
  }
  if (s < 0) return;
  const int b = a.c.start[s], e = a.c.start[s + 1], len = a.c.length[s];
  if (row >= e && e >= b && s == a.c.n_seqs - 1) return;   // behind the last sequence
  if (b < 0 || e < b || row >= e || e > a.n_rows || len < e - b || len > cache_slots(a.c)) {
    if (lane == 0) record_error(a.err, DEVERR_INDEX);
    return;
  }
  const int slot = len - (e - b) + (row - b), page = page_of(a.c, s, slot);
  if (page < 0 || page >= a.c.n_pages) {
    if (lane == 0) record_error(a.err, DEVERR_INDEX);
    return;
  }
  const int64_t to = page_row(a.c, page, head, slot);
  const __nv_bfloat16* src = (lane < 16 ? a.k : a.v) + (int64_t)row * a.row_stride + (int64_t)head * a.head_stride;
  __nv_bfloat16* dst = (lane < 16 ? a.k_pages : a.v_pages) + to * 128;
  if (in_bounds<__nv_bfloat16>(lane < 16 ? a.k_pages : a.v_pages, a.page_elems, dst, 128, a.err, 60) &&
      in_bounds<__nv_bfloat16>(lane < 16 ? a.k : a.v, a.src_elems, src, 128, a.err, 61))
    reinterpret_cast<uint4*>(dst)[lane & 15] = reinterpret_cast<const uint4*>(src)[lane & 15];
  if (lane == 0 && a.weights != nullptr && in_bounds<float>(a.weights, a.page_elems / 128, a.weights + to, 1, a.err, 62))
    a.weights[to] = 0.0f;
}

// ---------------------------------------------------------------------------
// Collected weights: w_j += sum over the new rows i and the heads that share
// the KV head of P_ij = exp(q_i . k_j / sqrt(128) - lse_i).  Keys are the rows
// of the score tiles (S = K Q^T), so that each key's sum stays in one thread,
// in an order that nothing but the row count fixes: no atomics.
//   A unit is up to four 128-key tiles of one KV head and sequence, each owned
//   by one warpgroup; the tiles of 128 (row, head) pairs that see any of them
//   stream past, each used by all four.  CTA c takes units c, c + grid, ...
//   warp 0 TMA producer, warp 1 MMA issuer, warp 2 the rows' log-sum-exp,
//   warps 4-19 exponentials and sums.
// TMEM: S of key tile w at [128 w, 128 w + 128).
// Many rows are bound by the exponentials (16 a clock and SM: 1024 cycles a
// tile, its product 512), single rows by reading K.
// ---------------------------------------------------------------------------
namespace {
constexpr int CW_THREADS = 32 * 20;
constexpr int CW_KT = 4, CW_QST = 2;
constexpr int CW_TILE = 128 * 128 * 2, CW_BOX = 128 * 64 * 2;
constexpr int CW_SMEM = CW_TILE * (CW_KT + CW_QST) + 8 * kCacheMaxSeqs + CW_QST * 512 + 256;

struct CwUnit {
  int head, seq, key0, tiles;    // key tiles of the unit, from key0
  int row0, pos0, keys, rows;    // the sequence: first new row, its position, keys, new rows
  int q0, nq;                    // tiles of rows that see any of the keys
};
__device__ __forceinline__ bool cw_seq_ok(const CacheArgs& c, int n_rows, int s) {
  const int b = c.start[s], e = c.start[s + 1], len = c.length[s];
  return b >= 0 && e >= b && e <= n_rows && len >= e - b && (int64_t)len <= cache_slots(c);
}
__device__ __forceinline__ CwUnit cw_unit(const CacheWeightsArgs& a, const int64_t* pre, int64_t per_head, int64_t u) {
  CwUnit x;
  x.head = (int)(u / per_head);
  const int64_t y = u - (int64_t)x.head * per_head;
  int s = 0;
  for (int lo = 0, hi = a.c.n_seqs - 1; lo <= hi;) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= y) { s = mid; lo = mid + 1; } else { hi = mid - 1; }
  }
  x.seq = s;
  x.key0 = (int)(y - pre[s]) * a.tiles * 128;
  x.row0 = a.c.start[s];
  x.rows = a.c.start[s + 1] - x.row0;
  x.keys = a.c.length[s];
  x.pos0 = x.keys - x.rows;
  x.tiles = min(a.tiles, (x.keys - x.key0 + 127) >> 7);
  const int last = min(x.keys, x.key0 + x.tiles * 128) - 1;
  const int lo = max(win_row_lo(a.w, x.key0, x.keys), x.pos0) - x.pos0;
  const int hi = max(win_row_hi(a.w, x.key0, x.keys), win_row_hi(a.w, last, x.keys)) - x.pos0;
  x.q0 = lo / a.R;
  x.nq = hi > lo ? (hi + a.R - 1) / a.R - x.q0 : 0;
  return x;
}
}  // namespace

__global__ void __launch_bounds__(CW_THREADS, 1)
    cache_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const CacheWeightsArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sk = smem_raw;
  uint8_t* sq = sk + CW_KT * CW_TILE;
  int64_t* pre = reinterpret_cast<int64_t*>(sq + CW_QST * CW_TILE);
  float* sl = reinterpret_cast<float*>(pre + kCacheMaxSeqs);   // [CW_QST][128] log-sum-exp, base 2
  uint64_t* bars = reinterpret_cast<uint64_t*>(sl + CW_QST * 128);
  uint64_t* k_full = bars;
  uint64_t* k_empty = k_full + CW_KT;
  uint64_t* q_full = k_empty + CW_KT;
  uint64_t* q_empty = q_full + CW_QST;
  uint64_t* l_full = q_empty + CW_QST;
  uint64_t* l_empty = l_full + CW_QST;
  uint64_t* s_full = l_empty + CW_QST;
  uint64_t* s_empty = s_full + CW_KT;
  uint64_t* drain = s_empty + CW_KT;
  int64_t* total = reinterpret_cast<int64_t*>(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(total + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  static_assert((4 * CW_KT + 4 * CW_QST + 2) * 8 + 8 <= 256, "barriers fit");

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int w = 0; w < CW_KT; ++w) {
      mbar_init(&k_full[w], 1);
      mbar_init(&k_empty[w], 1);
      mbar_init(&s_full[w], 1);
      mbar_init(&s_empty[w], 4);
    }
    for (int s = 0; s < CW_QST; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
      mbar_init(&l_full[s], 1);
      mbar_init(&l_empty[s], 16);
    }
    mbar_init(drain, 1);
    *abort_flag = timeout_recorded(a.err) ? 1 : 0;   // sticky timeout of an earlier launch
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  griddep_wait();
  if (warp == 2) {   // groups of key tiles before each sequence
    int64_t carry = 0;
    for (int s0 = 0; s0 < a.c.n_seqs; s0 += 32) {
      const int s = s0 + lane;
      int64_t mine = 0;
      if (s < a.c.n_seqs) {
        if (cw_seq_ok(a.c, a.n_rows, s)) mine = (a.c.length[s] + a.tiles * 128 - 1) / (a.tiles * 128);
        else if (blockIdx.x == 0) record_error(a.err, DEVERR_INDEX);
      }
      int64_t sum = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += t;
      }
      if (s < a.c.n_seqs) pre[s] = carry + sum - mine;
      carry += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) *total = carry;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl ctl{abort_flag, a.err, KID_CACHE_WEIGHTS};
  const int64_t per_head = *total, units = per_head * a.c.n_kv_heads;

  if (*ctl.flag != 0) {
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    uint32_t kph[CW_KT] = {0, 0, 0, 0}, st = 0, ph = 0, issued = 0, loaded = 0;
    for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const CwUnit x = cw_unit(a, pre, per_head, u);
      if (x.nq == 0) continue;
      const int ps = a.c.page_size, rows = min(ps, 128);
#pragma unroll
      for (int w = 0; w < CW_KT; ++w) {
        if (w >= x.tiles || !ok) continue;
        if (!at_wait(&k_empty[w], kph[w] ^ 1u, ctl)) { ok = false; continue; }
        kph[w] ^= 1u;
        loaded |= 1u << w;
        if (lane == 0) mbar_arrive_expect_tx(&k_full[w], CW_TILE);
        __syncwarp();
        if (lane < 256 / rows) {
          const int box = lane >> 1, slot = x.key0 + w * 128 + box * rows;
          int page = a.c.n_pages;   // out of range: zeros
          if (slot < x.keys) {
            const int id = page_of(a.c, x.seq, slot);
            if (id >= 0 && id < a.c.n_pages) page = id;
          }
          tma_load_4d(sk + w * CW_TILE + (lane & 1) * CW_BOX + box * rows * 128, &tmK, &k_full[w], (lane & 1) * 64,
                      slot % ps, x.head, page);
        }
      }
      for (int i = 0; i < x.nq && ok; ++i) {
        if (!at_wait(&q_empty[st], ph ^ 1u, ctl)) { ok = false; break; }
        if (lane == 0) mbar_arrive_expect_tx(&q_full[st], (uint32_t)(a.R * a.G * 256));
        __syncwarp();
        if (lane < 2)
          tma_load_4d(sq + st * CW_TILE + lane * CW_BOX, &tmQ, &q_full[st], lane * 64, 0, x.head,
                      x.row0 + (x.q0 + i) * a.R);
        ++issued;
        if (++st == CW_QST) { st = 0; ph ^= 1u; }
      }
    }
    if (!ok && lane == 0) {   // let issued loads land before the CTA exits
      for (uint32_t j = issued > CW_QST ? issued - CW_QST : 0; j < issued; ++j)
        at_drain(&q_full[j % CW_QST], (j / CW_QST) & 1u);
#pragma unroll
      for (int w = 0; w < CW_KT; ++w)
        if ((loaded >> w) & 1u) at_drain(&k_full[w], kph[w] ^ 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc = idesc_bf16(128, 128, false, false);
    constexpr uint64_t kTile = CW_TILE >> 4, kBox = CW_BOX >> 4;
    const uint32_t one = at_elect();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem_base, 0);
    const uint64_t kd = sdesc_kmajor(smem_u32(sk)), qd = sdesc_kmajor(smem_u32(sq));
    uint32_t kph = 0, sph = 0, st = 0, ph = 0;   // one phase bit per key tile
    bool ok = true;
    for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const CwUnit x = cw_unit(a, pre, per_head, u);
      for (int i = 0; i < x.nq && ok; ++i) {
        if (!at_wait(&q_full[st], ph, ctl)) { ok = false; break; }
        for (int w = 0; w < x.tiles; ++w) {
          if (i == 0) {
            if (!at_wait(&k_full[w], (kph >> w) & 1u, ctl)) { ok = false; break; }
            kph ^= 1u << w;
          }
          if (!at_wait(&s_empty[w], ((sph >> w) & 1u) ^ 1u, ctl)) { ok = false; break; }
          sph ^= 1u << w;
          tc_fence_after();
          at_mma4_ss<2, 2>(tm + (uint32_t)(w * 128), kd + w * kTile, qd + st * kTile, idesc, 0u, one);
          at_mma4_ss<2, 2>(tm + (uint32_t)(w * 128), kd + w * kTile + kBox, qd + st * kTile + kBox, idesc, 1u, one);
          at_commit(&s_full[w], one);
          if (i == x.nq - 1) at_commit(&k_empty[w], one);
        }
        at_commit(&q_empty[st], one);
        if (++st == CW_QST) { st = 0; ph ^= 1u; }
      }
    }
    if (!ok) {
      at_commit(drain, one);
      if (one) at_drain(drain, 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ log-sum-exp of the rows
    uint32_t st = 0, ph = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const CwUnit x = cw_unit(a, pre, per_head, u);
      for (int i = 0; i < x.nq; ++i) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = e * 32 + lane, r = c / a.G, row = (x.q0 + i) * a.R + r;
          v[e] = INFINITY;
          if (r < a.R && row < x.rows) {
            const float* at = a.lse + (int64_t)(x.head * a.G + c - r * a.G) * a.n_rows + x.row0 + row;
            if (in_bounds<float>(a.lse, a.lse_elems, at, 1, a.err, 63)) v[e] = *at * 1.44269504088896340736f;
            if (v[e] == -INFINITY) v[e] = INFINITY;   // a row that saw nothing adds nothing
          }
        }
        if (!at_wait(&l_empty[st], ph ^ 1u, ctl)) { ok = false; break; }
#pragma unroll
        for (int e = 0; e < 4; ++e) sl[st * 128 + e * 32 + lane] = v[e];
        __syncwarp();
        if (lane == 0) mbar_arrive(&l_full[st]);
        if (++st == CW_QST) { st = 0; ph ^= 1u; }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ exponentials and sums
    const int w = (warp - 4) >> 2, qq = warp & 3;
    const uint32_t s_base = tmem_addr(tmem_base, (uint32_t)(qq * 32), (uint32_t)(w * 128));
    const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
    uint32_t st = 0, ph = 0, sph = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const CwUnit x = cw_unit(a, pre, per_head, u);
      const int key = x.key0 + w * 128 + qq * 32 + lane;
      const bool mine = w < x.tiles && key < x.keys;
      // rows of the sequence that see the key
      const int see_lo = max(win_row_lo(a.w, min(key, x.keys - 1), x.keys) - x.pos0, 0);
      const int see_hi = win_row_hi(a.w, min(key, x.keys - 1), x.keys) - x.pos0;
      float sum = 0.0f;
      for (int i = 0; i < x.nq; ++i) {
        if (!at_wait(&l_full[st], ph, ctl)) { ok = false; break; }
        if (w < x.tiles) {
          if (!at_wait(&s_full[w], sph, ctl)) { ok = false; break; }
          sph ^= 1u;
          tc_fence_after();
          const int at = (x.q0 + i) * a.R;            // the tile's first row
          const int ncol = min(a.R, x.rows - at) * a.G;
          // columns that see the key
          const int ca = min(max(see_lo - at, 0), a.R) * a.G, cb = min(max(see_hi - at, 0) * a.G, ncol);
          float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
          for (int q4 = 0; q4 * 32 < ncol; ++q4) {
            uint32_t s[32];
            tmem_ld32(s_base + (uint32_t)(q4 * 32), s);
            tmem_ld_wait(s);
            const uint32_t see = win_bits(cb - q4 * 32) & ~win_bits(ca - q4 * 32);
            if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!((see >> c) & 1u)) s[c] = __float_as_uint(-INFINITY);
            }
            const float4* l4 = reinterpret_cast<const float4*>(sl + st * 128 + q4 * 32);
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 l = l4[c >> 2];
              const float2 z0 = __ffma2_rn(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sl2,
                                           make_float2(-l.x, -l.y));
              const float2 z1 = __ffma2_rn(make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), sl2,
                                           make_float2(-l.z, -l.w));
              acc[0] = __fadd2_rn(acc[0], make_float2(at_ex2(z0.x), at_ex2(z0.y)));
              acc[1] = __fadd2_rn(acc[1], make_float2(at_ex2(z1.x), at_ex2(z1.y)));
            }
          }
          sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[w]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&l_empty[st]);
        if (++st == CW_QST) { st = 0; ph ^= 1u; }
      }
      if (ok && mine) {
        const int page = page_of(a.c, x.seq, key);
        if (page >= 0 && page < a.c.n_pages) {
          const int64_t at = page_row(a.c, page, x.head, key);
          if (in_bounds<float>(a.out, a.page_rows, a.out + at, 1, a.err, 64))
            a.out[at] = (a.in != nullptr ? a.in[at] : 0.0f) + sum;
        } else if (see_lo < min(see_hi, x.rows)) {
          record_error(a.err, DEVERR_INDEX);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *ctl.flag) record_error(a.err, DEVERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// ---------------------------------------------------------------------------
// Eviction.  evict_select_kernel, one CTA per sequence and head: which of n
// slots stay.  The weights become 32-bit keys that order as they do (NaN lowest);
// three passes of 11, 11 and 10 bits find the key that the last kept slot has,
// and one ordered pass writes the slots above it and the earliest of those equal
// to it.  Counts are integers: the result is exact and repeatable.
// ---------------------------------------------------------------------------
namespace {
constexpr int EV_THREADS = 1024, EV_BINS = 2048;
constexpr int EV_KEYS = 48 * 1024;               // keys held in shared memory; further ones are read again
constexpr int EV_SMEM = EV_BINS * 4 + 256;

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w == 0.0f ? 0.0f : w);   // -0 as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
}  // namespace

__global__ void __launch_bounds__(EV_THREADS) evict_select_kernel(const EvictArgs a, int held) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint32_t* hist = reinterpret_cast<uint32_t*>(smem_raw);
  uint32_t* misc = hist + EV_BINS;                 // [0, 32) warp sums, [32] the bin, [33] what is still to keep in it
  uint32_t* keys = misc + 64;
  griddep_launch_dependents();
  griddep_wait();
  const int head = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = a.from.length[s];
  int32_t* kept = a.kept + ((int64_t)s * a.from.n_kv_heads + head) * a.budget;
  const bool bad = n < 0 || (int64_t)n > cache_slots(a.from) || (int64_t)min(n, a.budget) > cache_slots(a.to);
  if (bad) {   // nothing of this sequence is moved
    if (tid == 0) {
      record_error(a.err, DEVERR_INDEX);
      if (head == 0) a.length[s] = 0;
    }
    for (int i = tid; i < a.budget; i += EV_THREADS) kept[i] = -1;
    return;
  }
  if (tid == 0 && head == 0) a.length[s] = min(n, a.budget);
  if (n <= a.budget) {
    for (int i = tid; i < a.budget; i += EV_THREADS) kept[i] = i < n ? i : -1;
    return;
  }
  const int m0 = a.first, m1 = n - a.recent;       // slots that go by weight
  uint32_t want = (uint32_t)(a.budget - a.first - a.recent);
  auto weight_at = [&](int slot) -> uint32_t {
    const int page = page_of(a.from, s, slot);
    if (page < 0 || page >= a.from.n_pages) {
      record_error(a.err, DEVERR_INDEX);
      return 0u;
    }
    const float* w = a.weights + page_row(a.from, page, head, slot);
    return in_bounds<float>(a.weights, a.from_rows, w, 1, a.err, 65) ? weight_key(*w) : 0u;
  };
  for (int i = m0 + tid; i < min(m1, m0 + held); i += EV_THREADS) keys[i - m0] = weight_at(i);
  __syncthreads();
  auto key_at = [&](int slot) -> uint32_t { return slot - m0 < held ? keys[slot - m0] : weight_at(slot); };
  uint32_t prefix = 0, mask = 0;
  if (want > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      for (int b = tid; b < EV_BINS; b += EV_THREADS) hist[b] = 0;
      __syncthreads();
      const uint32_t digit = pass == 2 ? 1023u : 2047u;
      for (int i0 = m0; i0 < m1; i0 += EV_THREADS) {
        const int i = i0 + tid;
        const uint32_t key = i < m1 ? key_at(i) : 0u;
        if (i < m1 && (key & mask) == prefix) atomicAdd(&hist[(key >> shift) & digit], 1u);
      }
      __syncthreads();
      // from the highest bin down: thread t holds bins 2047 - 2t and 2046 - 2t
      const uint32_t h0 = hist[EV_BINS - 1 - 2 * tid], h1 = hist[EV_BINS - 2 - 2 * tid];
      uint32_t sum = h0 + h1;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += t;
      }
      if (lane == 31) misc[warp] = sum;
      __syncthreads();
      uint32_t before = sum - h0 - h1;
      for (int w = 0; w < warp; ++w) before += misc[w];
      if (before < want && want <= before + h0) {
        misc[32] = (uint32_t)(EV_BINS - 1 - 2 * tid);
        misc[33] = want - before;
      } else if (before + h0 < want && want <= before + h0 + h1) {
        misc[32] = (uint32_t)(EV_BINS - 2 - 2 * tid);
        misc[33] = want - before - h0;
      }
      __syncthreads();
      prefix |= misc[32] << shift;
      mask |= digit << shift;
      want = misc[33];
      __syncthreads();
    }
  }
  // In order: warp w takes an equal run of the slots, counts what it keeps and
  // how many equal the last key, and then writes from the sum of those before.
  const int run = ((n + 31) / 32 + 31) & ~31, r0 = min(n, warp * run), r1 = min(n, r0 + run);
  auto classify = [&](int i) -> int {              // 2: stays, 1: as the last key, 0: goes
    if (i >= r1) return 0;
    if (i < m0 || i >= m1) return 2;
    if (mask == 0u) return 0;
    const uint32_t k = key_at(i);
    return k > prefix ? 2 : (k == prefix ? 1 : 0);
  };
  uint32_t above = 0, equal = 0;
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const int c = classify(i0 + lane);
    above += __popc(__ballot_sync(0xffffffffu, c == 2));
    equal += __popc(__ballot_sync(0xffffffffu, c == 1));
  }
  if (lane == 0) {
    hist[warp] = above;
    hist[32 + warp] = equal;
  }
  __syncthreads();
  uint32_t out = 0, seen = 0;
  for (int w = 0; w < warp; ++w) {
    out += hist[w];
    seen += hist[32 + w];
  }
  out += min(seen, want);
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const int i = i0 + lane, c = classify(i);
    const unsigned eq = __ballot_sync(0xffffffffu, c == 1), below = (1u << lane) - 1u;
    const bool stays = c == 2 || (c == 1 && seen + __popc(eq & below) < want);
    const unsigned st = __ballot_sync(0xffffffffu, stays);
    if (stays) kept[out + __popc(st & below)] = i;
    out += __popc(st);
    seen += __popc(eq);
  }
}

// Moves the kept rows: a warp a row, K by the lower and V by the upper half of
// its lanes, eight rows in flight.  Bound by HBM.
namespace {
constexpr int EM_ROWS = 8;   // rows of a warp
}
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int head = blockIdx.y, s = blockIdx.z, lane = threadIdx.x & 31;
  const int d0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * EM_ROWS;
  const int32_t* kept = a.kept + ((int64_t)s * a.from.n_kv_heads + head) * a.budget;
  const __nv_bfloat16* src = lane < 16 ? a.k_from : a.v_from;
  __nv_bfloat16* dst = lane < 16 ? a.k_to : a.v_to;
  int64_t from[EM_ROWS], to[EM_ROWS];
  uint4 row[EM_ROWS];
  float w[EM_ROWS];
#pragma unroll
  for (int e = 0; e < EM_ROWS; ++e) {
    const int d = d0 + e, slot = d < a.budget ? kept[d] : -1;
    from[e] = to[e] = -1;
    if (slot < 0) continue;
    const int pf = page_of(a.from, s, slot), pt = page_of(a.to, s, d);
    if (pf < 0 || pf >= a.from.n_pages || pt < 0 || pt >= a.to.n_pages) {
      if (lane == 0) record_error(a.err, DEVERR_INDEX);
      continue;
    }
    from[e] = page_row(a.from, pf, head, slot);
    to[e] = page_row(a.to, pt, head, d);
    if (!in_bounds<__nv_bfloat16>(src, a.from_rows * 128, src + from[e] * 128, 128, a.err, 66) ||
        !in_bounds<__nv_bfloat16>(dst, a.to_rows * 128, dst + to[e] * 128, 128, a.err, 67))
      to[e] = -1;
  }
#pragma unroll
  for (int e = 0; e < EM_ROWS; ++e) {
    if (to[e] < 0) continue;
    row[e] = reinterpret_cast<const uint4*>(src + from[e] * 128)[lane & 15];
    if (lane == 0 && a.weights_to != nullptr) w[e] = a.weights[from[e]];
  }
#pragma unroll
  for (int e = 0; e < EM_ROWS; ++e) {
    if (to[e] < 0) continue;
    reinterpret_cast<uint4*>(dst + to[e] * 128)[lane & 15] = row[e];
    if (lane == 0 && a.weights_to != nullptr) a.weights_to[to[e]] = w[e];
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream) {
  const int64_t units = (int64_t)a.n_rows * a.c.n_kv_heads;
  const cudaError_t e = launch_kernel(cache_append_kernel, dim3((unsigned)((units + 7) / 8)), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  set_kernel_info("cache_append_kernel rows=%d heads=%d", a.n_rows, a.c.n_kv_heads);
  return cudaGetLastError();
}

cudaError_t launch_cache_weights(const CUtensorMap& tmQ, const CUtensorMap& tmK, CacheWeightsArgs a,
                                 cudaStream_t stream) {
  static_assert(tmem_footprint_exclusive(CW_SMEM), "an attention CTA must hold its SM's TMEM alone");
  if (!tmem_exclusive(CW_SMEM)) return cudaErrorNotSupported;
  cudaError_t e = cudaFuncSetAttribute(cache_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CW_SMEM);
  if (e != cudaSuccess) return e;
  // units of four key tiles where they fill the SMs at the tables' width
  const int64_t tiles = ((int64_t)a.c.table_width * a.c.page_size + 127) / 128;
  const int64_t lists = (int64_t)a.c.n_kv_heads * a.c.n_seqs;
  a.tiles = CW_KT;
  while (a.tiles > 1 && lists * ((tiles + a.tiles - 1) / a.tiles) < num_sms()) a.tiles >>= 1;
  const int64_t units = lists * ((tiles + a.tiles - 1) / a.tiles);
  const int grid = (int)(units < num_sms() ? units : num_sms());
  e = launch_kernel(cache_weights_kernel, dim3((unsigned)grid), dim3(CW_THREADS), CW_SMEM, stream, tmQ, tmK, a);
  if (e != cudaSuccess) return e;
  set_kernel_info("cache_weights_kernel tcgen05.mma.cta_group::1.kind::f16 key_tiles=%dx128 rows/tile=%d shared=%d acc=f32 "
                  "grid=%d", a.tiles, a.R, a.G, grid);
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t stream) {
  const int64_t slots = (int64_t)a.from.table_width * a.from.page_size;
  const int held = (int)(slots < EV_KEYS ? slots : EV_KEYS);
  const size_t smem = EV_SMEM + (size_t)held * 4;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       EV_SMEM + EV_KEYS * 4);
  if (e != cudaSuccess) return e;
  e = launch_kernel(evict_select_kernel, dim3((unsigned)a.from.n_kv_heads, (unsigned)a.from.n_seqs), dim3(EV_THREADS),
                    smem, stream, a, held);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((a.budget + 8 * EM_ROWS - 1) / (8 * EM_ROWS)), (unsigned)a.from.n_kv_heads,
                  (unsigned)a.from.n_seqs);
  e = launch_kernel(evict_move_kernel, grid, dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  set_kernel_info("evict_select_kernel + evict_move_kernel heads=%d sequences=%d budget=%d held=%d", a.from.n_kv_heads,
                  a.from.n_seqs, a.budget, held);
  return cudaGetLastError();
}

}  // namespace h3
