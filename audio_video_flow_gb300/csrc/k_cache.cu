// The paged cache of keys and values: append of new rows, the attention weight
// that each cached row collects, and eviction by that weight.
//   pages    [n_pages][n_kv_heads][page_size][128] bf16, one array each for K
//            and V; a head's rows of a page are contiguous
//   weights  [n_pages][n_kv_heads][page_size] fp32
#include "attention_device.cuh"
#include "h3_internal.h"

#include <algorithm>
#include <cmath>

namespace h3 {

namespace {
// Element offset of a slot's row in the pages (of 128 channels; of 1 in the
// weights).
__device__ __forceinline__ int64_t page_row(const CacheArgs& c, int page, int head, int slot) {
  return (((int64_t)page * c.n_kv_heads + head) << c.page_shift) + (slot & (c.page_size - 1));
}
__device__ __forceinline__ int page_of(const CacheArgs& c, int seq, int slot) {
  return c.table[(int64_t)seq * c.table_width + (slot >> c.page_shift)];
}
}  // namespace

// ---------------------------------------------------------------------------
// Append: row i of sequence s, the rows-before-it-in-s'th of its new ones, goes
// to slot length[s] - new + that.  A warp copies up to eight heads of one row, all
// in flight: K by the lower, V by the upper half of its lanes.  The last CTA copies
// nothing: it looks at the sequences, which the others meet only by their rows.  Bound
// by HBM, or by its launch.
// ---------------------------------------------------------------------------
namespace {
constexpr int CA_HEADS = 8;
}
__global__ void __launch_bounds__(256) cache_append_kernel(const AppendArgs a, int warps_per_row) {
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x == gridDim.x - 1) {
    for (int s = threadIdx.x; s < a.c.n_seqs; s += 256)
      if (!cache_seq_ok(a.c, a.n_rows, s)) record_error(a.err, DEVERR_INDEX);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (u >= (int64_t)a.n_rows * warps_per_row) return;
  const int row = (int)(u / warps_per_row), head0 = (int)(u - (int64_t)row * warps_per_row) * CA_HEADS;
  int s = -1;
  for (int lo = 0, hi = a.c.n_seqs - 1; lo <= hi;) {   // the last sequence that starts at or before the row
    const int mid = (lo + hi) >> 1;
    if (a.c.start[mid] <= row) { s = mid; lo = mid + 1; } else { hi = mid - 1; }
  }
  if (s < 0) return;
  const int b = a.c.start[s], e = a.c.start[s + 1], len = a.c.length[s];
  // behind the last sequence, or of one that the last CTA reports
  if (row >= e || !cache_seq_ok(a.c, a.n_rows, s)) return;
  const int slot = len - (e - b) + (row - b), page = page_of(a.c, s, slot);
  if (page < 0 || page >= a.c.n_pages) {
    if (lane == 0) record_error(a.err, DEVERR_INDEX);
    return;
  }
  const __nv_bfloat16* src = lane < 16 ? a.k : a.v;
  __nv_bfloat16* dst = lane < 16 ? a.k_pages : a.v_pages;
  uint4 x[CA_HEADS];
#pragma unroll
  for (int h = 0; h < CA_HEADS; ++h) {
    const __nv_bfloat16* from = src + (int64_t)row * a.row_stride + (int64_t)(head0 + h) * a.head_stride;
    if (head0 + h < a.c.n_kv_heads && in_bounds<__nv_bfloat16>(src, a.src_elems, from, 128, a.err, 61))
      x[h] = reinterpret_cast<const uint4*>(from)[lane & 15];
  }
#pragma unroll
  for (int h = 0; h < CA_HEADS; ++h) {
    if (head0 + h >= a.c.n_kv_heads) break;
    const int64_t to = page_row(a.c, page, head0 + h, slot);
    if (in_bounds<__nv_bfloat16>(dst, a.page_elems, dst + to * 128, 128, a.err, 60))
      reinterpret_cast<uint4*>(dst + to * 128)[lane & 15] = x[h];
    if (lane == h && a.weights != nullptr && in_bounds<float>(a.weights, a.page_elems / 128, a.weights + to, 1, a.err, 62))
      a.weights[to] = 0.0f;
  }
}

// ---------------------------------------------------------------------------
// Collected weights: w_j += sum over the new rows i and the heads that share
// the KV head of P_ij = exp(q_i . k_j / sqrt(128) - lse_i).  Keys are the rows
// of the score tiles (S = K Q^T), so that each key's sum stays in one thread,
// in an order that nothing but the row count fixes: no atomics.
//   A unit is a few 128-key tiles of one KV head and sequence; CTA c takes units
// c, c + grid, ...  The tiles of 128 (row, head) pairs that see any of its keys
// are held in shared memory, up to four at a time (a pass), and the key tiles
// stream past them, each half (64 channels) a stage of the ring.  Two tiles of rows
// make a product of 256 columns (tile by tile, its issue and waits took 940 cycles
// where the tensor core had 580 to do, and K was read twice: 117 -> 109 us of a call
// of 405 rows).  Of a pass,
// pair i lies in half (h + i) % 2, h where the pass before ended, so that the next
// pass's rows load while this one's last are used.
//   warp 0 TMA producer, warp 1 MMA issuer, warp 2 the rows' log-sum-exp,
//   warps 4-7 exponentials and sums of the pairs' first tiles, 8-11 of their second
//   (a key per thread),
//   warp 3 adds the two groups' sums of a key tile to the weights (one sum per group,
//   not per tile of rows, and no window arithmetic where all rows see a unit: 109 ->
//   105 us).
// TMEM: S of every second product at 0, of the others at 256.  A product has as
// many columns as its tiles have pairs, rounded up to 16: single rows cost little
// beside reading K.
// Shared memory is what the products themselves fill, so the rows' log-sum-exp is
// not read from it column by column by every thread (16 KB a product and warp, as
// much as the operands: 124 us of a call of 405 rows) but comes with the product,
// as a K step of its own: ones times -lse sqrt(128) in three bf16 parts, 2^-26 of
// it off.
// Measured (56 heads, 405 rows over 14,836 keys): 97 us, 886 TFLOP/s; a key tile
// takes about 3300 cycles, of which the tensor core has 1950 and the exponentials
// 1660 to do, the rest is waits between the two, and a CTA's first product starts
// after 9500.  Single rows (8 sequences of up to 4096 keys): 22 us, by the start and
// the latency of a few key tiles.
// ---------------------------------------------------------------------------
namespace {
constexpr int CW_THREADS = 32 * 12;
constexpr int CW_SLOTS = 4, CW_PAIRS = 2, CW_KST = 4, CW_RED = 2;
constexpr int CW_TILE = 128 * 128 * 2, CW_BOX = 128 * 64 * 2;
constexpr int CW_STEP = 128 * 16 * 2;   // an operand of one K step
constexpr int CW_SMEM =
    CW_TILE * CW_SLOTS + CW_BOX * CW_KST + CW_STEP * (CW_SLOTS + 1) + 4 * kCacheMaxSeqs + 2 * CW_RED * 512 + 512;

struct CwUnit {
  int head, seq, key0, tiles;    // key tiles of the unit, from key0
  int row0, pos0, keys, rows;    // the sequence: first new row, its position, keys, new rows
  int q0, nq;                    // tiles of rows that see any of the keys
  bool whole;                    // all rows see all of them
};
// Not inlined: every role calls it once per unit, and fetching the code is what a
// first call costs.
__device__ __noinline__ CwUnit cw_unit(const CacheWeightsArgs& a, const int* pre, int per_head, int u) {
  CwUnit x;
  x.head = u / per_head;
  const int y = u - x.head * per_head;
  int s = 0;
  for (int lo = 0, hi = a.c.n_seqs - 1; lo <= hi;) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= y) { s = mid; lo = mid + 1; } else { hi = mid - 1; }
  }
  x.seq = s;
  x.key0 = (y - pre[s]) * a.tiles * 128;
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
  // a key's first row never falls from key to key, its last one only behind the first keys
  x.whole = win_row_lo(a.w, last, x.keys) <= x.pos0 &&
            win_row_hi(a.w, min(max(x.key0, a.w.first), last), x.keys) >= x.keys;
  return x;
}
// Which of the keys key, key + 32, ... some new row, from position pos0 on, sees: bit e
// for key + 32 e.
__device__ __noinline__ unsigned cw_seen(WindowArgs w, int key, int keys, int pos0) {
  unsigned seen = 0;
#pragma unroll 1
  for (int e = 0; e < 4; ++e, key += 32)
    if (key < keys && max(win_row_lo(w, key, keys), pos0) < win_row_hi(w, key, keys)) seen |= 1u << e;
  return seen;
}
// exp2(s scale) over the columns [ca, cb) of 32 Q, added to acc; s_empty is
// arrived at once the scores are in registers.
template <int Q>
__device__ __forceinline__ void cw_sums(uint32_t s_at, int ca, int cb, float2 scale, float2 (&acc)[4], uint64_t* s_empty) {
  uint32_t s[Q][32];
#pragma unroll
  for (int q = 0; q < Q; ++q) tmem_ld32(s_at + (uint32_t)(q * 32), s[q]);
  tmem_ld_wait(s);
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(s_empty);
  if (!__all_sync(0xffffffffu, ca <= 0 && cb >= 32 * Q)) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const uint32_t see = win_bits(cb - q * 32) & ~win_bits(ca - q * 32);
      if (__all_sync(0xffffffffu, see == 0xffffffffu)) continue;
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (!((see >> c) & 1u)) s[q][c] = __float_as_uint(-INFINITY);
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const float2 z = __fmul2_rn(make_float2(__uint_as_float(s[q][2 * c]), __uint_as_float(s[q][2 * c + 1])), scale);
      acc[c & 3] = __fadd2_rn(acc[c & 3], make_float2(at_ex2(z.x), at_ex2(z.y)));
    }
}
}  // namespace

__global__ void __launch_bounds__(CW_THREADS, 1)
    cache_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CacheWeightsArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sq = smem_raw;
  uint8_t* sk = sq + CW_SLOTS * CW_TILE;
  uint8_t* sl = sk + CW_KST * CW_BOX;                          // [slot] the rows' part of the last K step, then the ones
  int* pre = reinterpret_cast<int*>(sl + (CW_SLOTS + 1) * CW_STEP);
  float* red = reinterpret_cast<float*>(pre + kCacheMaxSeqs);  // [group][CW_RED][128] sums of a key tile
  uint64_t* k_full = reinterpret_cast<uint64_t*>(red + 2 * CW_RED * 128);
  uint64_t* k_empty = k_full + CW_KST;
  uint64_t* q_full = k_empty + CW_KST;
  uint64_t* q_empty = q_full + CW_PAIRS;
  uint64_t* l_full = q_empty + CW_PAIRS;
  uint64_t* l_empty = l_full + CW_PAIRS;
  uint64_t* s_full = l_empty + CW_PAIRS;
  uint64_t* s_empty = s_full + CW_PAIRS;
  uint64_t* r_full = s_empty + CW_PAIRS;                       // [group][CW_RED]
  uint64_t* r_empty = r_full + 2 * CW_RED;
  uint64_t* drain = r_empty + 2 * CW_RED;
  int* total = reinterpret_cast<int*>(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(total + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  static_assert((2 * CW_KST + 6 * CW_PAIRS + 4 * CW_RED + 1) * 8 + 12 <= 512, "barriers fit");

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < CW_KST; ++s) { mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], 1); }
    for (int i = 0; i < CW_PAIRS; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&l_full[i], 1);
      mbar_init(&l_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 8);
    }
    for (int b = 0; b < 2 * CW_RED; ++b) {
      mbar_init(&r_full[b], 4);
      mbar_init(&r_empty[b], 1);
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
  // ones for every key in the first three channels of the last K step; its second
  // eight channels are zero on both sides
  for (int i = threadIdx.x; i < (CW_SLOTS + 1) * 256; i += CW_THREADS) {
    const bool ones = i >= CW_SLOTS * 256 && ((i >> 3) & 1) == 0;
    reinterpret_cast<uint4*>(sl)[i] = make_uint4(ones ? 0x3F803F80u : 0u, ones ? 0x3F80u : 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  griddep_wait();
  if (warp == 2) {   // units before each sequence
    int carry = 0;
    for (int s0 = 0; s0 < a.c.n_seqs; s0 += 32) {
      const int s = s0 + lane;
      int mine = 0;
      if (s < a.c.n_seqs) {
        if (cache_seq_ok(a.c, a.n_rows, s)) mine = (a.c.length[s] + a.tiles * 128 - 1) / (a.tiles * 128);
        else if (blockIdx.x == 0) record_error(a.err, DEVERR_INDEX);
      }
      int sum = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, sum, d);
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
  const int per_head = *total, units = per_head * a.c.n_kv_heads;

  if (*ctl.flag != 0) {
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    uint32_t qph = 0, pair = 0, st = 0, ph = 0, issued = 0, loaded = 0;   // qph: a phase bit per pair
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const CwUnit x = cw_unit(a, pre, per_head, u);
      const int rows = min(a.c.page_size, 128);
      for (int p = 0; p < x.nq && ok; p += CW_SLOTS) {
        const int n = min(CW_SLOTS, x.nq - p);
        int page = 0;
        auto page_at = [&](int k) -> int {   // this lane's page of key tile k, n_pages: zeros
          const int key = x.key0 + k * 128 + lane * rows;
          if (lane >= 128 / rows || key >= x.keys) return a.c.n_pages;
          const int id = page_of(a.c, x.seq, key);
          return id >= 0 && id < a.c.n_pages ? id : a.c.n_pages;
        };
        page = page_at(0);
        for (int k = 0; k < x.tiles && ok; ++k) {
          const int next = k + 1 < x.tiles ? page_at(k + 1) : 0;   // arrives during the waits
          for (int h = 0; h < 2; ++h) {
            if (!at_wait(&k_empty[st], ph ^ 1u, ctl)) { ok = false; break; }
            if (lane == 0) mbar_arrive_expect_tx(&k_full[st], CW_BOX);
            __syncwarp();
            if (lane < 128 / rows)
              tma_load_4d(sk + st * CW_BOX + lane * rows * 128, &tmK, &k_full[st], h * 64,
                          (x.key0 + k * 128 + lane * rows) & (a.c.page_size - 1), x.head, page);
            ++issued;
            if (++st == CW_KST) { st = 0; ph ^= 1u; }
          }
          page = next;
          if (k > 0) continue;
          for (int i = 0; i < n && ok; i += 2) {                   // the pass's rows, after its first keys
            if (!at_wait(&q_empty[pair], ((qph >> pair) & 1u) ^ 1u, ctl)) { ok = false; break; }
            qph ^= 1u << pair;
            loaded |= 1u << pair;
            const int both = min(2, n - i);
            if (lane == 0) mbar_arrive_expect_tx(&q_full[pair], (uint32_t)(both * a.R * a.G * 256));
            __syncwarp();
            if (lane < 2 * both)   // lane: half of the channels, and tile in bit 1
              tma_load_4d(sq + pair * 2 * CW_TILE + (lane & 1) * CW_TILE + (lane >> 1) * CW_BOX, &tmQ, &q_full[pair],
                          (lane & 1) * 64, 0, x.head, x.row0 + (x.q0 + p + i + (lane >> 1)) * a.R);
            pair ^= 1u;
          }
        }
      }
    }
    if (*ctl.flag && lane == 0) {   // a wait ran out: let issued loads land before the CTA exits
      for (uint32_t j = issued > CW_KST ? issued - CW_KST : 0; j < issued; ++j)
        at_drain(&k_full[j % CW_KST], (j / CW_KST) & 1u);
      for (uint32_t i = 0; i < CW_PAIRS; ++i)
        if ((loaded >> i) & 1u) at_drain(&q_full[i], ((qph >> i) & 1u) ^ 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc0 = idesc_bf16(128, 0, false, false);
    constexpr uint64_t kTile = CW_TILE >> 4, kBox = CW_BOX >> 4, kStep = CW_STEP >> 4;
    const uint32_t one = at_elect();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem_base, 0);
    const uint64_t kd = sdesc_kmajor(smem_u32(sk)), qd = sdesc_kmajor(smem_u32(sq));
    const uint64_t ld = at_sdesc_plain16(smem_u32(sl)), ones = ld + CW_SLOTS * kStep;
    uint32_t qph = 0, prod = 0, pair0 = 0, st = 0, ph = 0;   // qph: a phase bit per pair; prod: products issued
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const CwUnit x = cw_unit(a, pre, per_head, u);
      for (int p = 0; p < x.nq && ok; p += CW_SLOTS) {
        const int n = min(CW_SLOTS, x.nq - p);
        for (int k = 0; k < x.tiles && ok; ++k) {
          uint32_t s[2];
          for (int h = 0; h < 2 && ok; ++h) {
            s[h] = st;
            ok = at_wait(&k_full[st], ph, ctl);
            if (++st == CW_KST) { st = 0; ph ^= 1u; }
          }
          uint32_t pair = pair0;
          for (int i = 0; i < n && ok; i += 2, pair ^= 1u) {
            if (k == 0) {
              if (!at_wait(&q_full[pair], (qph >> pair) & 1u, ctl) || !at_wait(&l_full[pair], (qph >> pair) & 1u, ctl)) {
                ok = false;
                break;
              }
              qph ^= 1u << pair;
            }
            const uint32_t sb = prod & 1u;
            if (!at_wait(&s_empty[sb], ((prod >> 1) & 1u) ^ 1u, ctl)) { ok = false; break; }
            ++prod;
            tc_fence_after();
            const int tile = min(i + 1, n - 1);   // the pair's last
            const int cols = (tile - i) * 128 + min(a.R, x.rows - (x.q0 + p + tile) * a.R) * a.G;
            const uint32_t idesc = idesc0 | (uint32_t)((cols + 15) >> 4) << 18;   // columns / 8 at bit 17
            const uint32_t d = tm + sb * 256u;
            const uint64_t q = qd + pair * 2 * kTile;
            at_mma4_ss<2, 2>(d, kd + s[0] * kBox, q, idesc, 0u, one);
            at_mma4_ss<2, 2>(d, kd + s[1] * kBox, q + kTile, idesc, 1u, one);
            at_mma1_ss(d, ones, ld + pair * 2 * kStep, idesc, 1u, one);
            at_commit(&s_full[sb], one);
            if (k == x.tiles - 1) {
              at_commit(&q_empty[pair], one);
              at_commit(&l_empty[pair], one);
            }
          }
          at_commit(&k_empty[s[0]], one);
          at_commit(&k_empty[s[1]], one);
        }
        pair0 ^= (uint32_t)((n + 1) >> 1) & 1u;
      }
    }
    if (*ctl.flag) {   // a wait ran out: let issued products end
      at_commit(drain, one);
      if (one) at_drain(drain, 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ log-sum-exp of the rows
    // One copy of the loads, its divisions before the loop: fetching the code is what
    // the first tiles wait for.
    uint32_t lph = 0, pair = 0;
    bool ok = true;
    int r[4], head_of[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = e * 32 + lane;
      r[e] = c / a.G;
      head_of[e] = c - r[e] * a.G;
    }
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const CwUnit x = cw_unit(a, pre, per_head, u);
      float v[4], next[4] = {};
#pragma unroll 1
      for (int i = -1; i < x.nq; ++i) {                   // the next tile's values arrive during the wait
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = (x.q0 + i + 1) * a.R + r[e];
          v[e] = next[e];
          next[e] = INFINITY;
          if (i + 1 < x.nq && r[e] < a.R && row < x.rows) {
            const float* at = a.lse + (int64_t)(x.head * a.G + head_of[e]) * a.n_rows + x.row0 + row;
            if (in_bounds<float>(a.lse, a.lse_elems, at, 1, a.err, 63)) next[e] = *at;
          }
        }
        if (i < 0) continue;
        if ((i & 1) == 0) {
          if (!at_wait(&l_empty[pair], ((lph >> pair) & 1u) ^ 1u, ctl)) { ok = false; break; }
          lph ^= 1u << pair;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = e * 32 + lane;
          // -lse sqrt(128); a row that saw nothing (lse -inf) adds nothing, and so does none
          float l = v[e] * -11.313708498984761f;
          if (fabsf(l) == INFINITY) l = -1e30f;
          const float hi = bf16_round(l), mid = bf16_round(l - hi), lo = l - hi - mid;
          *reinterpret_cast<uint4*>(sl + (2 * pair + (i & 1)) * CW_STEP + (c >> 3) * 256 + (c & 7) * 16) =
              make_uint4(pack_bf16x2(hi, mid), pack_bf16x2(lo, 0.0f), 0u, 0u);
        }
        if ((i & 1) == 0 && i + 1 < x.nq) continue;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&l_full[pair]);
        pair ^= 1u;
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ sums to weights
    uint32_t turn[2] = {0, 0};               // sums taken of each group
    // Added in place, what no row sees is neither read nor written: its page may have
    // been given back and be another sequence's now, whose sums a rewrite would lose
    // (405 rows in a window of 3000: 134 us, 132.5 with the rewrite).
    const bool in_place = a.in == a.out;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const CwUnit x = cw_unit(a, pre, per_head, u);
      for (int p = 0; p < max(x.nq, in_place ? 0 : 1) && ok; p += CW_SLOTS) {
        const int n = min(CW_SLOTS, x.nq - p);   // 0: no row sees the unit, its weights stay
        // this lane's four keys of key tile k: their places (-1: none) and weights
        auto weights_of = [&](int k, int64_t (&at)[4], float (&w)[4]) {
          int mine[4];                           // keys whose weights are this call's
#pragma unroll
          for (int e = 0; e < 4; ++e) mine[e] = x.key0 + k * 128 + e * 32 + lane;
          if (in_place && !x.whole) {
            const unsigned seen = cw_seen(a.w, mine[0], x.keys, x.pos0);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((seen >> e) & 1u)) mine[e] = x.keys;
          }
          int page[4];                           // all in flight
#pragma unroll
          for (int e = 0; e < 4; ++e) page[e] = mine[e] < x.keys ? page_of(a.c, x.seq, mine[e]) : -1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = mine[e];
            at[e] = -1;
            w[e] = 0.0f;
            if (key < x.keys) {
              if (page[e] >= 0 && page[e] < a.c.n_pages) {
                at[e] = page_row(a.c, page[e], x.head, key);
                if (!in_bounds<float>(a.out, a.page_rows, a.out + at[e], 1, a.err, 64)) at[e] = -1;
              } else if (p == 0 && max(win_row_lo(a.w, key, x.keys), x.pos0) < win_row_hi(a.w, key, x.keys)) {
                record_error(a.err, DEVERR_INDEX);   // a page that some row sees
              }
              // later passes add to what the first one wrote
              if (at[e] >= 0) w[e] = p > 0 ? a.out[at[e]] : (a.in != nullptr ? a.in[at[e]] : 0.0f);
            }
          }
        };
        int64_t at[4], next_at[4] = {};
        float w[4], next_w[4] = {};
#pragma unroll 1
        for (int k = -1; k < x.tiles && ok; ++k) {       // one copy of the loads, as above
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            at[e] = next_at[e];
            w[e] = next_w[e];
          }
          if (k + 1 < x.tiles) weights_of(k + 1, next_at, next_w);   // arrive during the waits
          if (k < 0) continue;
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (g >= n) break;
            const uint32_t b = g * CW_RED + (turn[g] & (CW_RED - 1));
            if (!at_wait(&r_full[b], (turn[g] / CW_RED) & 1u, ctl)) { ok = false; break; }
            ++turn[g];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += red[b * 128 + e * 32 + lane];
            __syncwarp();
            if (lane == 0) mbar_arrive(&r_empty[b]);
          }
          if (!ok) break;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (at[e] >= 0) a.out[at[e]] = w[e] + sum[e];
        }
      }
    }
  } else {
    // ------------------------------------------------------------ exponentials and sums
    const int group = (warp - 4) >> 2;                // the pair's tile
    const int qq = warp & 3;
    const uint32_t s_base = tmem_addr(tmem_base, (uint32_t)(qq * 32), 0);
    const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
    uint32_t prod = 0, turn = 0;                      // products seen, sums written
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const CwUnit x = cw_unit(a, pre, per_head, u);
      for (int p = 0; p < x.nq && ok; p += CW_SLOTS) {
        const int n = min(CW_SLOTS, x.nq - p);
        for (int k = 0; k < x.tiles && ok; ++k) {
          int see_lo = 0, see_hi = x.rows;                  // rows that see the key
          if (!x.whole) {
            const int key = min(x.key0 + k * 128 + qq * 32 + lane, x.keys - 1), unit = win_unit(a.w, key);
            see_lo = win_row_lo_of(a.w, unit, x.keys) - x.pos0;
            see_hi = win_row_hi_of(a.w, unit, key, x.keys) - x.pos0;
          }
          float2 acc[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = make_float2(0.0f, 0.0f);
          for (int i = group; i < n + group; i += 2) {
            const int at = (x.q0 + p + i) * a.R;            // the tile's first row
            const int ncol = min(a.R, x.rows - at) * a.G;
            // columns that see the key
            const int ca = min(max(see_lo - at, 0), a.R) * a.G, cb = min(min(max(see_hi - at, 0), a.R) * a.G, ncol);
            const uint32_t sb = prod & 1u;
            if (!at_wait(&s_full[sb], (prod >> 1) & 1u, ctl)) { ok = false; break; }
            ++prod;
            if (i >= n) {                                   // a pass's last tile stands alone
              if (lane == 0) mbar_arrive(&s_empty[sb]);
              continue;
            }
            tc_fence_after();
            const uint32_t s_at = s_base + sb * 256u + (uint32_t)group * 128u;
            if (ncol <= 32) cw_sums<1>(s_at, ca, cb, sl2, acc, &s_empty[sb]);
            else cw_sums<4>(s_at, ca, cb, sl2, acc, &s_empty[sb]);
          }
          if (!ok) break;
          if (group < n) {
            const uint32_t b = turn & (CW_RED - 1);
            if (!at_wait(&r_empty[group * CW_RED + b], ((turn / CW_RED) & 1u) ^ 1u, ctl)) { ok = false; break; }
            ++turn;
            const float2 sum = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
            red[(group * CW_RED + b) * 128 + qq * 32 + lane] = sum.x + sum.y;
            __syncwarp();
            if (lane == 0) mbar_arrive(&r_full[group * CW_RED + b]);
          }
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
// up to three passes of 11, 11 and 10 bits find the key that the last kept slot
// has, or a border between keys, and one ordered pass writes the slots above it and
// the earliest of those equal to it.  Counts are integers: the result is exact and
// repeatable.  Bound by instructions (issue slots 65 % busy), so each pass over the
// keys does little: 56 x 15,860 slots, 20 us and the call 84, with classes of slots
// in each pass and always three; now the call is 81.
// ---------------------------------------------------------------------------
namespace {
constexpr int EV_THREADS = 1024, EV_BINS = 2048;
constexpr int EV_KEYS = 48 * 1024;               // keys held in shared memory; further ones are read again
constexpr int EV_BATCH = 4;                      // slots of a thread in flight (8: 80.2 us of 80.8, short caches 10.1 of 9.4)
constexpr int EV_SMEM = EV_BINS * 4 + 256;

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w == 0.0f ? 0.0f : w);   // -0 as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ bool evict_bad(const EvictArgs& a, int n) {
  return n < 0 || (int64_t)n > cache_slots(a.from) || (int64_t)min(n, a.budget) > cache_slots(a.to);
}
}  // namespace

// HELD: shared memory holds all keys; otherwise the first `held`.
template <bool HELD>
__global__ void __launch_bounds__(EV_THREADS) evict_select_kernel(const EvictArgs a, int held) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint32_t* hist = reinterpret_cast<uint32_t*>(smem_raw);
  uint32_t* misc = hist + EV_BINS;                 // [0, 32) warp sums, [32] the bin, [33] what is still to keep in it, [34] its keys
  uint32_t* keys = misc + 64;
  griddep_wait();
  griddep_launch_dependents();   // after the wait: the move begins with what earlier kernels left
  const int head = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = a.from.length[s];
  int32_t* kept = a.kept + ((int64_t)s * a.from.n_kv_heads + head) * a.budget;
  if (evict_bad(a, n)) {   // nothing of this sequence is moved
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
  const int m0 = a.first, m = n - a.recent - m0;   // slots [m0, m0 + m) go by weight
  for (int i = tid; i < m0; i += EV_THREADS) kept[i] = i;
  for (int i = tid; i < a.recent; i += EV_THREADS) kept[a.budget - a.recent + i] = m0 + m + i;
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
  // a few slots a thread at a time: table entries, then weights, in flight together
  // (one by one: 25 us of a call of 15,860 slots)
  const int in_smem = min(m, held);
  for (int i0 = tid; i0 < in_smem; i0 += EV_BATCH * EV_THREADS) {
    int page[EV_BATCH];
    float w[EV_BATCH];
#pragma unroll
    for (int e = 0; e < EV_BATCH; ++e) {
      const int i = i0 + e * EV_THREADS;
      page[e] = i < in_smem ? page_of(a.from, s, m0 + i) : -1;
    }
#pragma unroll
    for (int e = 0; e < EV_BATCH; ++e) {
      const int i = i0 + e * EV_THREADS;
      w[e] = NAN;
      if (page[e] < 0 || page[e] >= a.from.n_pages) {
        if (i < in_smem) record_error(a.err, DEVERR_INDEX);
        continue;
      }
      const float* at = a.weights + page_row(a.from, page[e], head, m0 + i);
      if (in_bounds<float>(a.weights, a.from_rows, at, 1, a.err, 65)) w[e] = *at;
    }
#pragma unroll
    for (int e = 0; e < EV_BATCH; ++e)
      if (i0 + e * EV_THREADS < in_smem) keys[i0 + e * EV_THREADS] = weight_key(w[e]);
  }
  __syncthreads();
  auto key_at = [&](int i) -> uint32_t { return HELD || i < held ? keys[i] : weight_at(m0 + i); };
  // Slots with a key above `last` stay, and the first `want` of those equal to it.
  uint32_t last = 0xffffffffu, mask = 0;           // no weight has that key
  if (want > 0) {
    last = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      for (int b = tid; b < EV_BINS; b += EV_THREADS) hist[b] = 0;
      __syncthreads();
      const uint32_t digit = pass == 2 ? 1023u : 2047u;
#pragma unroll 4
      for (int i = tid; i < m; i += EV_THREADS) {
        const uint32_t key = key_at(i);
        if ((key & mask) == last) atomicAdd(&hist[(key >> shift) & digit], 1u);
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
      const uint32_t warps = __reduce_add_sync(0xffffffffu, lane < warp ? misc[lane] : 0u);
      const uint32_t before = warps + sum - h0 - h1;
      if (before < want && want <= before + h0) {
        misc[32] = (uint32_t)(EV_BINS - 1 - 2 * tid);
        misc[33] = want - before;
        misc[34] = h0;
      } else if (before + h0 < want && want <= before + h0 + h1) {
        misc[32] = (uint32_t)(EV_BINS - 2 - 2 * tid);
        misc[33] = want - before - h0;
        misc[34] = h1;
      }
      __syncthreads();
      last |= misc[32] << shift;
      mask |= digit << shift;
      want = misc[33];
      const bool whole = want == misc[34] && last > 0;
      __syncthreads();
      if (whole) {                                 // all of the bin stay: distinct weights seldom need the third pass
        --last;
        want = 0;
        break;
      }
    }
  }
  // In order: warp w takes an equal run of the slots, counts what it keeps and
  // how many equal the last key, and then writes from the sum of those before.
  const int run = ((m + 31) / 32 + 31) & ~31, r0 = min(m, warp * run), r1 = min(m, r0 + run);
  uint32_t above = 0, equal = 0;
#pragma unroll 4
  for (int i = r0 + lane; i < r1; i += 32) {
    const uint32_t key = key_at(i);
    above += key > last;
    equal += key == last;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    hist[warp] = above;
    hist[32 + warp] = equal;
  }
  __syncthreads();
  uint32_t out = (uint32_t)m0 + __reduce_add_sync(0xffffffffu, lane < warp ? hist[lane] : 0u);
  uint32_t seen = __reduce_add_sync(0xffffffffu, lane < warp ? hist[32 + lane] : 0u);
  out += min(seen, want);
  const unsigned below = (1u << lane) - 1u;
#pragma unroll 4
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < r1 ? key_at(i) : 0u;
    bool stays = i < r1 && key > last;
    const unsigned eq = want > 0 ? __ballot_sync(0xffffffffu, i < r1 && key == last) : 0u;
    if (eq != 0u) {
      stays = stays || (((eq >> lane) & 1u) && seen + __popc(eq & below) < want);
      seen += __popc(eq);
    }
    const unsigned st = __ballot_sync(0xffffffffu, stays);
    if (stays) kept[out + __popc(st & below)] = m0 + i;
    out += __popc(st);
  }
}

// Moves the kept rows: a warp a row, K by the lower and V by the upper half of
// its lanes, eight rows in flight.  The first and the recent rows, and sequences
// that fit the budget, move whatever the selection says, so their tiles come first
// and do not wait for it: it has let this grid start once it had itself waited for
// all before it, and it neither reads nor writes what they touch (a tenth of the rows
// of a call of 56 heads x 15,860 slots: 90 -> 87 us as a graph).  Bound by HBM:
// that call moves 7930 of each, 464 MB, in 81 us, 5.7 TB/s with the selection, 12 us
// of which nothing overlaps.
namespace {
constexpr int EM_ROWS = 8, EM_TILE = 8 * EM_ROWS;   // rows of a warp and of a CTA
}
// Grid: tiles x heads, sequences; first_tile, that of the first recent row, is first.
// The next kernel starts with the last of its CTAs, not earlier: one that comes to
// select for another call would take places of these (95 us for 84).
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a, int tiles, int first_tile) {
  const int y = (int)(blockIdx.x / (unsigned)a.from.n_kv_heads), head = (int)blockIdx.x - y * a.from.n_kv_heads;
  const int s = blockIdx.y, lane = threadIdx.x & 31;
  const int tile = first_tile + y - (y >= tiles - first_tile ? tiles : 0);
  const int d0 = tile * EM_TILE + (int)(threadIdx.x >> 5) * EM_ROWS, n = a.from.length[s];
  const int32_t* kept = a.kept + ((int64_t)s * a.from.n_kv_heads + head) * a.budget;
  const bool sure = !evict_bad(a, n) && (n <= a.budget || d0 + EM_ROWS <= a.first || d0 >= a.budget - a.recent);
  if (!sure) griddep_wait();
  auto slot_of = [&](int d) { return !sure ? kept[d] : (n > a.budget && d >= a.first ? n - a.budget + d : (d < n ? d : -1)); };
  const __nv_bfloat16* src = lane < 16 ? a.k_from : a.v_from;
  __nv_bfloat16* dst = lane < 16 ? a.k_to : a.v_to;
  // lane e % 8 finds row e's places
  int64_t from_row = -1, to_row = -1;
  {
    const int d = d0 + (lane & (EM_ROWS - 1)), slot = d < a.budget ? slot_of(d) : -1;
    if (slot >= 0) {
      const int pf = page_of(a.from, s, slot), pt = page_of(a.to, s, d);
      if (pf >= 0 && pf < a.from.n_pages && pt >= 0 && pt < a.to.n_pages) {
        from_row = page_row(a.from, pf, head, slot);
        to_row = page_row(a.to, pt, head, d);
      } else if (lane < EM_ROWS) {
        record_error(a.err, DEVERR_INDEX);
      }
    }
  }
  const bool moves = to_row >= 0 && in_bounds<__nv_bfloat16>(src, a.from_rows * 128, src + from_row * 128, 128, a.err, 66) &&
                     in_bounds<__nv_bfloat16>(dst, a.to_rows * 128, dst + to_row * 128, 128, a.err, 67);
  const unsigned rows = __ballot_sync(0xffffffffu, moves);
  uint4 row[EM_ROWS];
#pragma unroll
  for (int e = 0; e < EM_ROWS; ++e) {
    const int64_t at = __shfl_sync(0xffffffffu, from_row, e);
    if ((rows >> e) & 1u) row[e] = __ldcs(reinterpret_cast<const uint4*>(src + at * 128) + (lane & 15));
  }
  if (moves && lane < EM_ROWS && a.weights_to != nullptr) a.weights_to[to_row] = a.weights[from_row];
#pragma unroll
  for (int e = 0; e < EM_ROWS; ++e) {
    const int64_t at = __shfl_sync(0xffffffffu, to_row, e);
    if ((rows >> e) & 1u) reinterpret_cast<uint4*>(dst + at * 128)[lane & 15] = row[e];
  }
  if (sure) griddep_wait();   // this grid ends after the selection's
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream) {
  const int warps_per_row = (a.c.n_kv_heads + CA_HEADS - 1) / CA_HEADS;
  const int64_t units = (int64_t)a.n_rows * warps_per_row;
  const cudaError_t e = launch_kernel(cache_append_kernel, dim3((unsigned)((units + 7) / 8 + 1)), dim3(256), 0, stream, a,
                                      warps_per_row);
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
  // Units of one to sixteen key tiles: against the rounds of the grid (between full
  // ones at the tables' width and a last one half full: the lengths are on the
  // device) stands what each unit costs beside its products, one product's time for
  // each of its tiles of rows (at the sequences' average) and two for its start
  // (405 rows: 15 key tiles 101 us, 8 of them 126, 4 116).
  const int64_t tiles = ((int64_t)a.c.table_width * a.c.page_size + 127) / 128;
  const int64_t lists = (int64_t)a.c.n_kv_heads * a.c.n_seqs;
  const int64_t per_seq = (a.n_rows + a.c.n_seqs - 1) / a.c.n_seqs;
  const double nq = (double)((per_seq + a.R - 1) / a.R);
  double best = 0.0;
  int64_t units = 0;
  for (int t = 1; t <= 16; ++t) {
    const int64_t n = lists * ((tiles + t - 1) / t), rounds = (n + num_sms() - 1) / num_sms();
    const double cost = ((double)rounds + (double)n / num_sms() + 0.5) * ((double)t * nq + nq + 2.0);
    if (t == 1 || cost < best) {
      best = cost;
      a.tiles = t;
      units = n;
    }
  }
  const int grid = (int)(units < num_sms() ? units : num_sms());
  e = launch_kernel(cache_weights_kernel, dim3((unsigned)grid), dim3(CW_THREADS), CW_SMEM, stream, tmQ, tmK, a);
  if (e != cudaSuccess) return e;
  set_kernel_info("cache_weights_kernel tcgen05.mma.cta_group::1.kind::f16 unit=%dx128 keys rows/tile=%d shared=%d acc=f32 "
                  "grid=%d", a.tiles, a.R, a.G, grid);
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t stream) {
  const int64_t slots = (int64_t)a.from.table_width * a.from.page_size;
  const int held = (int)(slots < EV_KEYS ? slots : EV_KEYS);
  const size_t smem = EV_SMEM + (size_t)held * 4;
  const auto kernel = held == slots ? evict_select_kernel<true> : evict_select_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, EV_SMEM + EV_KEYS * 4);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kernel, dim3((unsigned)a.from.n_kv_heads, (unsigned)a.from.n_seqs), dim3(EV_THREADS),
                    smem, stream, a, held);
  if (e != cudaSuccess) return e;
  const int tiles = (a.budget + EM_TILE - 1) / EM_TILE;
  const dim3 grid((unsigned)tiles * (unsigned)a.from.n_kv_heads, (unsigned)a.from.n_seqs);
  e = launch_kernel(evict_move_kernel, grid, dim3(256), 0, stream, a, tiles,
                    std::min(tiles - 1, (a.budget - a.recent) / EM_TILE));
  if (e != cudaSuccess) return e;
  set_kernel_info("evict_select_kernel + evict_move_kernel heads=%d sequences=%d budget=%d held=%d", a.from.n_kv_heads,
                  a.from.n_seqs, a.budget, held);
  return cudaGetLastError();
}

}  // namespace h3
