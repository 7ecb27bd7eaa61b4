// Attention with a window (h3_window: units before and after the row's own,
// first keys that stay visible), 128-wide heads, query heads that may share a
// KV head, over one document or over the pages of a cache; fp32 online
// softmax, on the 5th-generation tensor cores.
//
// A tile is 128 (row, head) pairs: R rows of the G query heads that share a KV
// head, so that single rows of shared heads fill a tile and K and V are read
// once for all of them.  A unit of work is two such tiles (slots A and B, 2R
// rows) of one KV head over the 128-key tiles that any of its rows sees: the
// tiles of the first keys, then those of the window.  The CTAs (one per SM)
// share the key tiles of all units out in equal runs, KV head by KV head, so
// documents of any lengths balance and a single row over a long cache uses
// every SM.  A unit that a run's end cuts leaves partial results (maximum, sum,
// unnormalised output), which attention_window_combine_kernel joins in order;
// ends less than kSnap tiles from a unit's own are moved there.
//   warp 0       TMA producer of Q and K;
//   warp 1       MMA issuer: S_t = Q_t K_j^T, O_t += P_t V_j;
//   warp 2       TMA producer of V;
//   warps 4-7    softmax of slot A, 8-11 of slot B, one row per thread.
// TMEM: S_A [0,128), S_B [128,256), O_A [256,384), O_B [384,512); P (bf16) over
// its S.  A unit of one tile (single rows, short documents) uses both slots for
// the same rows, A for its even and B for its odd key tiles, so that the tensor
// core works for one while the other's softmax runs; A joins the two.
// The next unit's S products run while the last one's results leave.
//
// Tiles that all of a warp's rows see whole take no mask; a masked score becomes
// -inf by selection, so whatever a hidden key holds takes no part in maximum or
// sum.  Rows of V past a sequence's last slot are zeroed in shared memory, and
// pages that no row of the unit sees are not read (zeros in their place): P is 0
// there, and 0 times an infinity or NaN of a stale page would be NaN.
//
// P is rounded to bf16 for its product, as in the unmasked kernel (its bound and
// its reason apply); maxima, sums and accumulators are fp32.
#include "attention_device.cuh"
#include "h3_internal.h"

#include <cmath>

namespace h3 {

namespace {
constexpr int AW_THREADS = 384;
constexpr int AW_KST = 3, AW_VST = 2;
constexpr int AW_TILE = 128 * 128 * 2;   // 32 KB: two 64-channel boxes
constexpr int AW_BOX = 128 * 64 * 2;
constexpr int AW_SMEM = AW_TILE * (2 + AW_KST + AW_VST) + 512;
constexpr int kSnap = 2;                 // tiles
constexpr float kLazyRescale = 8.0f;     // see the unmasked kernel

// What a CTA leaves for the combine kernel: x bit 0: its first unit began in an
// earlier CTA (partial tile 0), bit 1: and ends here; bit 2: its last unit
// begins here and goes on (partial tile 1), being pair w of sequence z, head y.
enum : int { AW_HEAD = 1, AW_HEAD_ENDS = 2, AW_TAIL = 4 };

// New rows [row0, row0 + rows) of a sequence and its keys; rows 0 for a
// sequence whose metadata is out of range.
struct AwSeq { int row0, rows, keys; };
template <bool PAGED>
__device__ __forceinline__ AwSeq aw_seq(const AttnWinArgs& a, int s) {
  if (!PAGED) return {0, a.n_rows, a.n_rows};
  const int b = a.c.start[s], e = a.c.start[s + 1], len = a.c.length[s];
  if (b < 0 || e < b || e > a.n_rows || len < e - b || (int64_t)len > (int64_t)a.c.table_width * a.c.page_size)
    return {0, 0, -1};
  return {b, e - b, len};
}
// Key tiles of a pair of tiles: [0, nsink) and [wbeg, wbeg + n - nsink).
struct AwPair { int rows, pos0, lo, hi, first, nsink, wbeg, n; };
__device__ __forceinline__ AwPair aw_pair(const AttnWinArgs& a, const AwSeq& q, int pair) {
  AwPair p;
  const int at = pair * 2 * a.R;
  p.rows = min(2 * a.R, q.rows - at);
  p.pos0 = q.keys - q.rows + at;
  const int last = p.pos0 + p.rows - 1;
  p.lo = win_lo(a.w, p.pos0, q.keys);
  p.hi = win_hi(a.w, last, q.keys);
  p.first = min(a.w.first, win_lo(a.w, last, q.keys));   // first keys that only they make visible
  p.wbeg = p.lo >> 7;
  p.nsink = min((p.first + 127) >> 7, p.wbeg);
  p.n = p.nsink + ((p.hi + 127) >> 7) - p.wbeg;
  return p;
}
__device__ __forceinline__ int aw_pairs(const AttnWinArgs& a, int rows) { return (rows + 2 * a.R - 1) / (2 * a.R); }

// Where a run begins: key tile `off` of n of pair `pair` of sequence `seq`, head
// `head`; off = n: at the end of that pair.
struct AwLoc { int head, seq, pair, off, n; int64_t x; };
struct AwShared {
  AwLoc loc[2];
  int64_t total;
};

// A whole warp: the key tiles before sequence s are pre[s] (of one head), all
// of them `per_head`.
template <bool PAGED>
__device__ __forceinline__ AwLoc aw_locate(const AttnWinArgs& a, const int64_t* pre, int64_t per_head, int64_t x) {
  AwLoc l;
  const int lane = threadIdx.x & 31;
  l.x = x;
  l.head = (int)(x / per_head);
  l.seq = l.pair = l.off = l.n = 0;
  if (l.head >= a.c.n_kv_heads) return l;
  int64_t y = x - (int64_t)l.head * per_head;
  int s = 0;
  for (int lo = 0, hi = a.c.n_seqs - 1; lo <= hi;) {   // the last sequence that begins at or before y
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= y) { s = mid; lo = mid + 1; } else { hi = mid - 1; }
  }
  y -= pre[s];
  const AwSeq q = aw_seq<PAGED>(a, s);
  const int np = aw_pairs(a, q.rows);
  l.seq = s;
  for (int p0 = 0; p0 < np; p0 += 32) {
    const int n = p0 + lane < np ? aw_pair(a, q, p0 + lane).n : 0;
    int64_t sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += t;
    }
    const unsigned over = __ballot_sync(0xffffffffu, sum > y);
    if (over) {
      const int w = __ffs(over) - 1;
      l.pair = p0 + w;
      l.n = __shfl_sync(0xffffffffu, n, w);
      l.off = (int)(y - (__shfl_sync(0xffffffffu, sum, w) - l.n));
      break;
    }
    y -= __shfl_sync(0xffffffffu, sum, 31);
  }
  if (l.off <= kSnap) {
    l.x -= l.off;
    l.off = 0;
  } else if (l.n - l.off <= kSnap) {
    l.x += l.n - l.off;
    l.off = l.n;
  }
  return l;
}

// The segments of a CTA's run, one after the other (the same in every warp).
template <bool PAGED>
struct AwIter {
  int head, seq, pair, off, np;
  int64_t rem;
  AwSeq q;
  AwPair p;
  int cnt;                       // key tiles of this segment: [off, off + cnt)
  __device__ __forceinline__ AwIter(const AttnWinArgs& a, const AwShared& sh) {
    const AwLoc& l = sh.loc[0];
    head = l.head;
    seq = l.seq;
    pair = l.pair;
    off = l.off;
    rem = sh.loc[1].x - l.x;
    if (rem <= 0) return;
    q = aw_seq<PAGED>(a, seq);
    np = aw_pairs(a, q.rows);
    if (off >= l.n) advance(a);
    else p = aw_pair(a, q, pair);
    cnt = rem < p.n - off ? (int)rem : p.n - off;
  }
  __device__ __forceinline__ void advance(const AttnWinArgs& a) {
    off = 0;
    if (++pair >= np) {
      pair = 0;
      do {
        if (++seq == a.c.n_seqs) {
          seq = 0;
          if (++head == a.c.n_kv_heads) { rem = 0; return; }
        }
        if (PAGED) q = aw_seq<PAGED>(a, seq);
      } while (q.rows == 0);
      np = aw_pairs(a, q.rows);
    }
    p = aw_pair(a, q, pair);
  }
  __device__ __forceinline__ bool more() const { return rem > 0; }
  __device__ __forceinline__ void next(const AttnWinArgs& a) {
    rem -= cnt;
    if (rem <= 0) return;
    advance(a);
    cnt = rem < p.n ? (int)rem : p.n;
  }
  __device__ __forceinline__ int key_tile(int j) const {   // j counts from the segment's first
    const int t = off + j;
    return t < p.nsink ? t : p.wbeg + t - p.nsink;
  }
  __device__ __forceinline__ bool dual(const AttnWinArgs& a) const { return p.rows > a.R; }
};

// One 128-key tile: two 64-channel boxes of a document's rows, or the boxes of
// the pages it spans, one lane each.  Slots of no row of the unit, and pages
// whose table entry is out of range, read as zeros.
template <bool PAGED>
__device__ __forceinline__ void aw_load_kv(uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, const AttnWinArgs& a,
                                           const AwIter<PAGED>& it, int tile, int lane) {
  if (!PAGED) {
    if (lane < 2) tma_load_3d(dst + lane * AW_BOX, tm, bar, lane * 64, it.head, tile * 128);
    return;
  }
  const int ps = a.c.page_size, rows = min(ps, 128);
  if (lane >= 256 / rows) return;
  const int box = lane >> 1, half = lane & 1, slot = tile * 128 + box * rows;
  int page = a.c.n_pages;
  if (slot < it.q.keys && (slot < it.p.first || (slot + rows > it.p.lo && slot < it.p.hi))) {
    const int at = slot / ps;
    const int id = a.c.table[(int64_t)it.seq * a.c.table_width + at];
    if (id < 0 || id >= a.c.n_pages) record_error(a.err, DEVERR_INDEX);
    else page = id;
  }
  tma_load_4d(dst + half * AW_BOX + box * rows * 128, tm, bar, half * 64, slot % ps, it.head, page);
}

struct AwSmem {
  uint8_t *q, *k, *v;
  uint64_t *q_full, *q_empty, *k_full, *k_empty, *v_full, *v_empty, *s_full, *p_full, *o_final, *b_ready, *drain;
};
}  // namespace

template <bool PAGED>
__global__ void __launch_bounds__(AW_THREADS, 1)
    attention_window_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const AttnWinArgs a) {
  // no static shared memory: the dynamic part starts at a multiple of 1024
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  AwSmem sm;
  sm.q = smem_raw;
  sm.k = sm.q + 2 * AW_TILE;
  sm.v = sm.k + AW_KST * AW_TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm.v + AW_VST * AW_TILE);
  sm.q_full = bars;
  sm.q_empty = bars + 1;
  sm.k_full = bars + 2;
  sm.k_empty = sm.k_full + AW_KST;
  sm.v_full = sm.k_empty + AW_KST;
  sm.v_empty = sm.v_full + AW_VST;
  sm.s_full = sm.v_empty + AW_VST;
  sm.p_full = sm.s_full + 2;
  sm.o_final = sm.p_full + 2;
  sm.b_ready = sm.o_final + 2;
  sm.drain = sm.b_ready + 1;
  AwShared* sh = reinterpret_cast<AwShared*>(sm.drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sh + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  static_assert((2 + 2 * AW_KST + 2 * AW_VST + 8) * 8 + sizeof(AwShared) + 8 <= 512, "barriers and setup fit");

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(sm.q_full, 1);
    mbar_init(sm.q_empty, 1);
    for (int s = 0; s < AW_KST; ++s) { mbar_init(&sm.k_full[s], 1); mbar_init(&sm.k_empty[s], 1); }
    for (int s = 0; s < AW_VST; ++s) { mbar_init(&sm.v_full[s], 1); mbar_init(&sm.v_empty[s], 1); }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.p_full[t], 4);
      mbar_init(&sm.o_final[t], 1);
    }
    mbar_init(sm.b_ready, 4);
    mbar_init(sm.drain, 1);
    *abort_flag = timeout_recorded(a.err) ? 1 : 0;   // sticky timeout of an earlier launch
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  griddep_wait();

  // ---- the run of this CTA: key tiles of each sequence, their prefix sums (in
  // the K ring, before its first load), both ends of the run
  int64_t* pre = reinterpret_cast<int64_t*>(sm.k);
  const int ns = a.c.n_seqs;
  for (int s = threadIdx.x; s < ns; s += AW_THREADS) {
    const AwSeq q = aw_seq<PAGED>(a, s);
    if (PAGED && q.keys < 0 && blockIdx.x == 0) record_error(a.err, DEVERR_INDEX);
    const int np = aw_pairs(a, q.rows);
    int64_t n = np > 4 ? -1 : 0;
    for (int p = 0; p < np && n >= 0; ++p) n += aw_pair(a, q, p).n;
    pre[s] = n;
  }
  __syncthreads();
  for (int s = warp; s < ns; s += AW_THREADS / 32) {
    if (pre[s] >= 0) continue;
    const AwSeq q = aw_seq<PAGED>(a, s);
    int64_t n = 0;
    for (int p = lane, np = aw_pairs(a, q.rows); p < np; p += 32) n += aw_pair(a, q, p).n;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
    __syncwarp();
    if (lane == 0) pre[s] = n;
  }
  __syncthreads();
  if (warp < 2) {   // both warps scan: each needs the sums (warp 0 writes them)
    int64_t carry = 0;
    if (warp == 0) {
      for (int s0 = 0; s0 < ns; s0 += 32) {
        const int64_t mine = s0 + lane < ns ? pre[s0 + lane] : 0;
        int64_t sum = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int64_t t = __shfl_up_sync(0xffffffffu, sum, d);
          if (lane >= d) sum += t;
        }
        if (s0 + lane < ns) pre[s0 + lane] = carry + sum - mine;
        carry += __shfl_sync(0xffffffffu, sum, 31);
      }
      if (lane == 0) sh->total = carry;
    }
  }
  __syncthreads();
  const int64_t per_head = sh->total, all = per_head * a.c.n_kv_heads;
  if (warp < 2 && all > 0) {
    const int64_t c = (int64_t)blockIdx.x + warp;
    const AwLoc l = aw_locate<PAGED>(a, pre, per_head, all / gridDim.x * c + all % gridDim.x * c / gridDim.x);
    if (lane == 0) sh->loc[warp] = l;
  }
  fence_proxy_async_smem();   // the sums were read; the ring's loads may overwrite them
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl ctl{abort_flag, a.err, KID_ATTN_WIN};
  const bool skip = *ctl.flag != 0 || all <= 0 || sh->loc[1].x <= sh->loc[0].x;

  if (threadIdx.x == 0) {
    int4 d = make_int4(0, 0, 0, 0);
    if (!skip) {
      const AwLoc &b = sh->loc[0], &e = sh->loc[1];
      const bool head = b.off > 0 && b.off < b.n;
      const bool inside = e.off > 0 && e.off < e.n;
      const bool same = head && inside && b.head == e.head && b.seq == e.seq && b.pair == e.pair;
      d = make_int4((head ? AW_HEAD | (same ? 0 : AW_HEAD_ENDS) : 0) | (inside && !same ? AW_TAIL : 0), e.head, e.seq,
                    e.pair);
    }
    a.desc[blockIdx.x] = d;
  }

  if (skip) {
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer of Q and K
    bool ok = true;
    uint32_t items = 0, st = 0, ph = 0, issued = 0;
    for (AwIter<PAGED> it(a, *sh); it.more() && ok; it.next(a)) {
      if (!at_wait(sm.q_empty, (items & 1u) ^ 1u, ctl)) { ok = false; break; }
      const int slots = it.dual(a) ? 2 : 1;
      if (lane == 0) mbar_arrive_expect_tx(sm.q_full, (uint32_t)(slots * a.R * a.G * 256));
      __syncwarp();
      if (lane < 2 * slots)
        tma_load_4d(sm.q + (lane >> 1) * AW_TILE + (lane & 1) * AW_BOX, &tmQ, sm.q_full, (lane & 1) * 64, 0, it.head,
                    it.q.row0 + (it.pair * 2 + (lane >> 1)) * a.R);
      ++items;
      for (int j = 0; j < it.cnt; ++j) {
        if (!at_wait(&sm.k_empty[st], ph ^ 1u, ctl)) { ok = false; break; }
        if (lane == 0) mbar_arrive_expect_tx(&sm.k_full[st], AW_TILE);
        __syncwarp();
        aw_load_kv<PAGED>(sm.k + st * AW_TILE, &tmK, &sm.k_full[st], a, it, it.key_tile(j), lane);
        ++issued;
        if (++st == AW_KST) { st = 0; ph ^= 1u; }
      }
    }
    if (!ok && lane == 0) {   // let issued loads land before the CTA exits
      if (items > 0) at_drain(sm.q_full, (items - 1) & 1u);
      for (uint32_t j = issued > AW_KST ? issued - AW_KST : 0; j < issued; ++j)
        at_drain(&sm.k_full[j % AW_KST], (j / AW_KST) & 1u);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ producer of V
    bool ok = true;
    uint32_t st = 0, ph = 0, issued = 0;
    for (AwIter<PAGED> it(a, *sh); it.more() && ok; it.next(a)) {
      for (int j = 0; j < it.cnt; ++j) {
        if (!at_wait(&sm.v_empty[st], ph ^ 1u, ctl)) { ok = false; break; }
        if (lane == 0) mbar_arrive_expect_tx(&sm.v_full[st], AW_TILE);
        __syncwarp();
        aw_load_kv<PAGED>(sm.v + st * AW_TILE, &tmV, &sm.v_full[st], a, it, it.key_tile(j), lane);
        ++issued;
        if (++st == AW_VST) { st = 0; ph ^= 1u; }
      }
    }
    if (!ok && lane == 0)
      for (uint32_t j = issued > AW_VST ? issued - AW_VST : 0; j < issued; ++j)
        at_drain(&sm.v_full[j % AW_VST], (j / AW_VST) & 1u);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = idesc_bf16(128, 128, false, false);
    constexpr uint32_t idesc_o = idesc_bf16(128, 128, false, true);   // V is MN-major
    constexpr uint64_t kTile = AW_TILE >> 4, kBox = AW_BOX >> 4;      // descriptor address steps
    const uint32_t one = at_elect();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem_base, 0);
    const uint64_t qd = sdesc_kmajor(smem_u32(sm.q)), kd = sdesc_kmajor(smem_u32(sm.k));
    const uint64_t vd = sdesc_sw128(smem_u32(sm.v), AW_BOX, 1024);
    uint32_t items = 0, ks = 0, kp = 0, vs = 0, vp = 0, pp[2] = {0, 0};
    bool ok = true;
    for (AwIter<PAGED> it(a, *sh); it.more() && ok; it.next(a)) {
      const bool dual = it.dual(a);
      const int na = dual ? it.cnt : (it.cnt + 1) >> 1, nb = dual ? it.cnt : it.cnt >> 1;
      int left = na + nb;                       // S products of this segment still to issue
      ok = at_wait(sm.q_full, items & 1u, ctl);
      ++items;
      // S_t of the slot's next tile; with two tiles of rows both slots read the
      // same K tile, A first
      auto issue_s = [&](int t) -> bool {
        if ((!dual || t == 0) && !at_wait(&sm.k_full[ks], kp, ctl)) return false;
        tc_fence_after();
        const uint64_t q = qd + (dual && t ? kTile : 0), k = kd + ks * kTile;
        at_mma4_ss<2, 2>(tm + (uint32_t)(t * 128), q, k, idesc_s, 0u, one);
        at_mma4_ss<2, 2>(tm + (uint32_t)(t * 128), q + kBox, k + kBox, idesc_s, 1u, one);
        if (!dual || t == 1) {
          at_commit(&sm.k_empty[ks], one);
          if (++ks == AW_KST) { ks = 0; kp ^= 1u; }
        }
        at_commit(&sm.s_full[t], one);
        if (--left == 0) at_commit(sm.q_empty, one);
        return true;
      };
      if (ok) ok = issue_s(0) && (nb == 0 || issue_s(1));
      for (int j = 0; j < na && ok; ++j) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int nt = t ? nb : na;
          if (j >= nt) break;
          if (!dual || t == 0) {
            if (!at_wait(&sm.v_full[vs], vp, ctl)) { ok = false; break; }
            if (PAGED) {
              const int valid = it.q.keys - it.key_tile(dual ? j : 2 * j + t) * 128;
              if (valid < 128) {   // slots past the sequence's last: zeros
                uint8_t* v = sm.v + vs * AW_TILE;
                for (int u = lane; u < (128 - valid) * 16; u += 32)
                  *reinterpret_cast<uint4*>(v + ((u >> 3) & 1) * AW_BOX + (valid + (u >> 4)) * 128 + (u & 7) * 16) =
                      make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                __syncwarp();
              }
            }
          }
          if (!at_wait(&sm.p_full[t], pp[t], ctl)) { ok = false; break; }
          pp[t] ^= 1u;
          tc_fence_after();
          const uint64_t v = vd + vs * kTile;
          const uint32_t o = tm + 256u + (uint32_t)(t * 128), p = tm + (uint32_t)(t * 128);
          at_mma4_ts<8, 128>(o, p, v, idesc_o, j != 0 ? 1u : 0u, one);
          at_mma4_ts<8, 128>(o, p + 32u, v + 512u, idesc_o, 1u, one);
          if (!dual || t == 1) {
            at_commit(&sm.v_empty[vs], one);
            if (++vs == AW_VST) { vs = 0; vp ^= 1u; }
          }
          if (j + 1 < nt) {
            if (!issue_s(t)) { ok = false; break; }
          } else {
            at_commit(&sm.o_final[t], one);
          }
        }
      }
    }
    if (!ok) {
      at_commit(sm.drain, one);
      if (one) at_drain(sm.drain, 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    const int t = (warp - 4) >> 2;
    const int qq = warp & 3;
    const int row = qq * 32 + lane;            // (row, head) pair of the tile
    const int r = row / a.G, g = row - r * a.G;
    const uint32_t s_base = tmem_addr(tmem_base, (uint32_t)(qq * 32), (uint32_t)(t * 128));
    const uint32_t o_base = s_base + 256u;
    const float sl2 = a.scale_log2;
    uint32_t sph = 0, oph = 0, jph = 0;
    bool ok = true;
    float* part = a.part + (int64_t)blockIdx.x * a.part_slots * a.part_rows * 130;
    for (AwIter<PAGED> it(a, *sh); it.more() && ok; it.next(a)) {
      const bool dual = it.dual(a);
      const int nt = dual ? it.cnt : (t == 0 ? (it.cnt + 1) >> 1 : it.cnt >> 1);
      if (nt == 0) continue;                   // one key tile: slot A alone
      const int rbase = dual && t ? a.R : 0;   // first row of the slot in the pair
      const int nrows = dual && t ? it.p.rows - a.R : min(it.p.rows, a.R);
      const bool active = qq * 32 < nrows * a.G;
      const bool valid = row < nrows * a.G;
      const int pos = it.p.pos0 + rbase + min(r, nrows - 1);
      const int lo = win_lo(a.w, pos, it.q.keys), hi = win_hi(a.w, pos, it.q.keys), first = min(a.w.first, hi);
      float m_used = -INFINITY, l_run = 0.0f;
      for (int j = 0; j < nt; ++j) {
        if (!at_wait(&sm.s_full[t], sph, ctl)) { ok = false; break; }
        sph ^= 1u;
        if (active) {
          tc_fence_after();
          const int k0 = it.key_tile(dual ? j : 2 * j + t) * 128;
          uint32_t s[4][32];
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) tmem_ld32(s_base + (uint32_t)(q4 * 32), s[q4]);
          tmem_ld_wait(s[0]);
          if (!__all_sync(0xffffffffu, (k0 >= lo && k0 + 128 <= hi) || k0 + 128 <= first)) {
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              const int at = k0 + q4 * 32;
              const uint32_t see = (win_bits(hi - at) & ~win_bits(lo - at)) | win_bits(first - at);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!((see >> c) & 1u)) s[q4][c] = __float_as_uint(-INFINITY);
            }
          }
          float mp[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) mp[e] = -INFINITY;
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
            for (int c = 0; c < 32; ++c) mp[c & 7] = fmaxf(mp[c & 7], __uint_as_float(s[q4][c]));
          const float mx = fmaxf(fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])),
                                 fmaxf(fmaxf(mp[4], mp[5]), fmaxf(mp[6], mp[7])));
          const float m_tile = mx * sl2;
          const bool need = m_tile > m_used + kLazyRescale;
          if (__any_sync(0xffffffffu, need)) {
            const float m_new = need ? m_tile : m_used;
            const float alpha = need ? at_ex2(m_used - m_new) : 1.0f;   // 0 when m_used = -inf
            l_run *= alpha;
            if (j > 0) {
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint32_t o[16];
                tmem_ld16(o_base + (uint32_t)(c * 16), o);
                at_tmem_ld_wait16(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                at_tmem_st16(o_base + (uint32_t)(c * 16), o);
              }
            }
            m_used = m_new;
          }
          // nothing seen so far: every score is -inf, and 2^(-inf - 0) = 0
          const float m_ref = m_used == -INFINITY ? 0.0f : m_used;
          const float2 sl2x2 = make_float2(sl2, sl2), negm = make_float2(-m_ref, -m_ref);
          float2 sp[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) sp[e] = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float2 z = __ffma2_rn(
                  make_float2(__uint_as_float(s[q4][2 * c]), __uint_as_float(s[q4][2 * c + 1])), sl2x2, negm);
              const float e0 = at_ex2(z.x), e1 = at_ex2(z.y);
              sp[c & 3] = __fadd2_rn(sp[c & 3], make_float2(e0, e1));
              pk[c] = pack_bf16x2(e0, e1);
            }
            at_tmem_st16(s_base + (uint32_t)(q4 * 16), pk);
          }
          l_run += ((sp[0].x + sp[0].y) + (sp[1].x + sp[1].y)) + ((sp[2].x + sp[2].y) + (sp[3].x + sp[3].y));
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[t]);
      }
      if (!ok || !at_wait(&sm.o_final[t], oph, ctl)) { ok = false; break; }
      oph ^= 1u;
      tc_fence_after();

      // ---- results.  One tile of rows: slot B's go to slot A through the
      // workspace (the CTA's own partial tile 2).
      const bool joint = !dual && it.cnt > 1;
      const bool begins = it.off == 0, ends = it.off + it.cnt == it.p.n;
      const int slot = joint && t == 1 ? 2 * (a.part_slots / 2) : (begins ? 1 : 0) * (a.part_slots / 2) + (dual ? t : 0);
      float* to = part + (int64_t)slot * a.part_rows * 130;
      const bool whole = begins && ends && !(joint && t == 1);
      float fa = 1.0f, fb = 0.0f, l = l_run, m = m_used;
      const float* other = part + (int64_t)(2 * (a.part_slots / 2)) * a.part_rows * 130;
      if (joint && t == 0) {
        if (!at_wait(sm.b_ready, jph, ctl)) { ok = false; break; }
        jph ^= 1u;
        if (valid) {
          const float mb = other[(int64_t)a.part_rows * 128 + row * 2], lb = other[(int64_t)a.part_rows * 128 + row * 2 + 1];
          m = fmaxf(m_used, mb);
          const float m_ref = m == -INFINITY ? 0.0f : m;
          fa = at_ex2(m_used - m_ref);
          fb = at_ex2(mb - m_ref);
          l = l_run * fa + lb * fb;
        }
      }
      const int grow = it.q.row0 + it.pair * 2 * a.R + rbase + r, qhead = it.head * a.G + g;
      if (whole) {
        const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // a NaN stays one
        fa *= inv;
        fb *= inv;
      }
      if (active) {
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t o[16];
          tmem_ld16(o_base + (uint32_t)(c * 16), o);
          at_tmem_ld_wait16(o);
          if (valid) {
            float f[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(o[e]) * fa;
            if (joint && t == 0) {
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 b = *reinterpret_cast<const float4*>(other + (int64_t)row * 128 + c * 16 + e);
                f[e] = __fmaf_rn(b.x, fb, f[e]);
                f[e + 1] = __fmaf_rn(b.y, fb, f[e + 1]);
                f[e + 2] = __fmaf_rn(b.z, fb, f[e + 2]);
                f[e + 3] = __fmaf_rn(b.w, fb, f[e + 3]);
              }
            }
            if (whole) {
              __nv_bfloat16* dst = a.o + ((int64_t)grow * a.H + qhead) * 128 + c * 16;
              if (in_bounds<__nv_bfloat16>(a.o, a.o_elems, dst, 16, a.err, 50)) {
                uint4* d = reinterpret_cast<uint4*>(dst);
                d[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                  pack_bf16x2(f[6], f[7]));
                d[1] = make_uint4(pack_bf16x2(f[8], f[9]), pack_bf16x2(f[10], f[11]), pack_bf16x2(f[12], f[13]),
                                  pack_bf16x2(f[14], f[15]));
              }
            } else {
              float* dst = to + (int64_t)row * 128 + c * 16;
              if (in_bounds<float>(a.part, a.part_elems, dst, 16, a.err, 51)) {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                  *reinterpret_cast<float4*>(dst + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
              }
            }
          }
        }
        if (valid) {
          if (whole) {
            if (a.lse != nullptr) {
              float* dst = a.lse + (int64_t)qhead * a.n_rows + grow;
              if (in_bounds<float>(a.lse, a.lse_elems, dst, 1, a.err, 52))
                *dst = (m + log2f(l)) * 0.69314718055994530942f;
            }
          } else {
            float* dst = to + (int64_t)a.part_rows * 128 + row * 2;
            if (in_bounds<float>(a.part, a.part_elems, dst, 2, a.err, 53))
              *reinterpret_cast<float2*>(dst) = make_float2(m, l);
          }
        }
        tc_fence_before();
      }
      if (joint && t == 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.b_ready);
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
// Joins the partial results of the units that the runs' ends cut, in the order
// of their key tiles: block (c, slot and quarter) the rows of the unit that CTA
// c began and did not finish.  With m the largest of the segments' maxima,
//   l = sum_s l_s 2^(m_s - m),   o = sum_s O_s 2^(m_s - m) / l.
// ---------------------------------------------------------------------------
template <bool PAGED>
__global__ void __launch_bounds__(256) attention_window_combine_kernel(const AttnWinArgs a, int ctas) {
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x, t = blockIdx.y >> 2;
  const int4 d = a.desc[c];
  if (!(d.x & AW_TAIL)) return;
  const AwSeq q = aw_seq<PAGED>(a, d.z);
  const AwPair p = aw_pair(a, q, d.w);
  const int row = (blockIdx.y & 3) * 32 + (threadIdx.x >> 3), ch = (threadIdx.x & 7) * 16;
  const int nrows = t == 0 ? min(p.rows, a.R) : p.rows - a.R;
  if (row >= nrows * a.G) return;
  const int64_t tile = (int64_t)a.part_rows * 130;
  const int ts = a.part_slots / 2;
  float m = -INFINITY, l = 0.0f, o[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) o[e] = 0.0f;
  for (int s = c; s < ctas; ++s) {
    int x = AW_TAIL;
    if (s > c) {
      x = a.desc[s].x;
      if (!(x & AW_HEAD)) continue;
    }
    const float* from = a.part + ((int64_t)s * a.part_slots + (s == c ? ts : 0) + t) * tile;
    const float2 ml = *reinterpret_cast<const float2*>(from + (int64_t)a.part_rows * 128 + row * 2);
    const float m_new = fmaxf(m, ml.x), m_ref = m_new == -INFINITY ? 0.0f : m_new;
    const float f0 = at_ex2(m - m_ref), f1 = at_ex2(ml.x - m_ref);
    l = l * f0 + ml.y * f1;
    m = m_new;
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const float4 v = *reinterpret_cast<const float4*>(from + (int64_t)row * 128 + ch + e);
      o[e] = o[e] * f0 + v.x * f1;
      o[e + 1] = o[e + 1] * f0 + v.y * f1;
      o[e + 2] = o[e + 2] * f0 + v.z * f1;
      o[e + 3] = o[e + 3] * f0 + v.w * f1;
    }
    if (s > c && (x & AW_HEAD_ENDS)) break;
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  const int r = row / a.G, qhead = d.y * a.G + row - r * a.G;
  const int grow = q.row0 + (d.w * 2 + t) * a.R + r;
  __nv_bfloat16* dst = a.o + ((int64_t)grow * a.H + qhead) * 128 + ch;
  if (in_bounds<__nv_bfloat16>(a.o, a.o_elems, dst, 16, a.err, 54)) {
    uint4* w = reinterpret_cast<uint4*>(dst);
    w[0] = make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                      pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
    w[1] = make_uint4(pack_bf16x2(o[8] * inv, o[9] * inv), pack_bf16x2(o[10] * inv, o[11] * inv),
                      pack_bf16x2(o[12] * inv, o[13] * inv), pack_bf16x2(o[14] * inv, o[15] * inv));
  }
  if (ch == 0 && a.lse != nullptr) {
    float* at = a.lse + (int64_t)qhead * a.n_rows + grow;
    if (in_bounds<float>(a.lse, a.lse_elems, at, 1, a.err, 55)) *at = (m + log2f(l)) * 0.69314718055994530942f;
  }
}

// CTAs of a call: one per SM, or as many as there are key tiles at most.
int attn_win_ctas(int64_t n_rows, int64_t kv_heads, int64_t n_seqs, int G, int64_t max_keys) {
  const int64_t rows = 2 * (128 / G);
  const int64_t units = (n_rows + rows - 1) / rows + (n_seqs - 1), tiles = (max_keys + 127) / 128;
  const int64_t most = (__int128)units * tiles * kv_heads > 4096 ? 4096 : units * tiles * kv_heads;
  const int64_t sms = num_sms();
  return (int)(most < 1 ? 1 : (most < sms ? most : sms));
}
size_t attn_win_desc_bytes(int ctas) { return ((size_t)ctas * sizeof(int4) + 255) & ~size_t(255); }
void attn_win_part(int64_t n_rows, int G, int* part_rows, int* part_slots) {
  const int R = 128 / G;
  *part_rows = ((int)(n_rows < R ? n_rows : R) * G + 7) & ~7;   // tiles of 130 floats a row stay 16-byte aligned
  *part_slots = n_rows > R ? 5 : 3;
}

cudaError_t launch_attention_window(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                    const AttnWinArgs& a, int ctas, cudaStream_t stream) {
  static_assert(tmem_footprint_exclusive(AW_SMEM), "an attention CTA must hold its SM's TMEM alone");
  if (!tmem_exclusive(AW_SMEM)) return cudaErrorNotSupported;
  const bool paged = a.c.start != nullptr;
  const auto kernel = paged ? attention_window_kernel<true> : attention_window_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, AW_SMEM);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kernel, dim3((unsigned)ctas), dim3(AW_THREADS), AW_SMEM, stream, tmQ, tmK, tmV, a);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)ctas, a.part_slots == 5 ? 8u : 4u);
  e = paged ? launch_kernel(attention_window_combine_kernel<true>, grid, dim3(256), 0, stream, a, ctas)
            : launch_kernel(attention_window_combine_kernel<false>, grid, dim3(256), 0, stream, a, ctas);
  if (e != cudaSuccess) return e;
  set_kernel_info("attention_window_kernel tcgen05.mma.cta_group::1.kind::f16 q_tiles=2x128 kv_tile=128 rows/tile=%d "
                  "shared=%d k_stages=%d v_stages=%d acc=f32 P-in-TMEM lazy-rescale=%g %s grid=%d",
                  a.R, a.G, AW_KST, AW_VST, (double)kLazyRescale, paged ? "paged" : "document", ctas);
  return cudaGetLastError();
}

}  // namespace h3
