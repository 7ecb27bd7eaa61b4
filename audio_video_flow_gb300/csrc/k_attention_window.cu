// Attention with a window (h3_window: units before and after the row's own,
// first keys that stay visible), 128-wide heads, query heads that may share a
// KV head, over one document or over the pages of a cache; fp32 online
// softmax, on the 5th-generation tensor cores.
//
// A tile is 128 (row, head) pairs: R rows of the G query heads that share a KV
// head, so that single rows of shared heads fill a tile and K and V are read
// once for all of them.  A unit of work is two such tiles (slots A and B, 2R
// rows) of one KV head over the 128-key tiles that any of its rows sees: the
// tiles of the first keys, then those of the window.
//   The CTAs (one per SM) form gangs of M.  A gang takes M units that follow one
// another in a sequence, one each, so that its CTAs read the same K and V tiles
// at about the same time, once from HBM and M - 1 times from L2 (gangs of one read
// 27 bytes a clock and SM at full rate, more than HBM's 23).  The gangs share the
// key tiles of all such groups out in equal runs, KV head by KV head, so documents
// of any lengths balance and a single row over a long cache uses every SM.  A unit
// that a run's end cuts leaves partial results (maximum, sum, unnormalised
// output) in the workspace, but for the last of its CTAs to count itself in: that
// one joins the others' with its own, still in TMEM, in the order of their key
// tiles whoever it is.  It may find a part counted in and not yet written, which
// its CTA does without waiting for anything.  Units of more than kFew parts are
// joined by the last CTA's warps together, once its run is done.  The counters are
// zeroed by a kernel before this one.  (A kernel after this one that joins all
// parts: 20 us of a call with one row over 15,860, 8 of them its launch, and 35 us
// of one with 405.)  Ends less than kSnap tiles from a group's own are moved there.
//   warp 0       TMA producer of Q and K;
//   warp 1       MMA issuer: S_t = Q_t K_j^T, O_t += P_t V_j;
//   warp 2       TMA producer of V;
//   warp 3       walks the CTA's run and hands its segments (a unit, or the part
//                of one that lies in the run) to the others through a small ring;
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

#include <algorithm>
#include <cmath>

namespace h3 {

namespace {
constexpr int AW_THREADS = 384;
constexpr int AW_REGS = 168, AW_REGS_FEW = 88, AW_REGS_MANY = 208;   // registers a thread: at launch, and split
constexpr int AW_SEGS = 4;               // segments handed out ahead
constexpr int AW_TILE = 128 * 128 * 2;   // 32 KB: two 64-channel boxes
constexpr int AW_BOX = 128 * 64 * 2;
// What the shared memory holds.  A document's units end in whole tiles of results,
// which leave through a stage of 32 rows x 64 channels per softmax warp.  Chunks
// over a cache have few of those.  Single rows (units of one tile) are bound by
// reading K and V and hold one Q tile, so a third V tile takes the place of the
// other.
enum AwMode : int { AW_DOC = 0, AW_CHUNK = 1, AW_ROWS = 2 };
template <int MODE>
struct AwPlan {
  static constexpr int q = MODE == AW_ROWS ? 1 : 2, k = MODE == AW_DOC ? 2 : 3, v = MODE == AW_ROWS ? 3 : 2;
  static constexpr int stage = MODE == AW_DOC ? 32 * 128 : 0;
  static constexpr int tail = 2560;      // segments, slot B's statistics, barriers, setup
  static constexpr int smem = AW_TILE * (q + k + v) + 8 * stage + tail;
};
constexpr int kSnap = 2;                 // tiles
constexpr float kLazyRescale = 8.0f;     // see the unmasked kernel

// Partial tiles: [row][channel] fp32, then the row's maximum and sum.  A CTA has
// two places (times the tiles of a unit): for the unit that began in an earlier
// gang, and for the one that goes on in a later.  Its control words: per softmax
// warp a counter for the units that begin with it, and the key tiles that it did
// for either.
// Units of at most kFew parts that are chunks: [channel][row] instead, a warp's
// rows side by side.
constexpr int kPartRow = 132;
constexpr int kCtrl = 24, kCtrlHead = 8, kCtrlTail = 16;
constexpr int kFew = 4;

// New rows [row0, row0 + rows) of a sequence and its keys; rows 0 for a
// sequence whose metadata is out of range.
struct AwSeq { int row0, rows, keys; };
template <bool PAGED>
__device__ __forceinline__ AwSeq aw_seq(const AttnWinArgs& a, int s) {
  if (!PAGED) return {0, a.n_rows, a.n_rows};
  if (!cache_seq_ok(a.c, a.n_rows, s)) return {0, 0, -1};
  const int b = a.c.start[s], e = a.c.start[s + 1], len = a.c.length[s];
  return {b, e - b, len};
}
// The setup and the segments are straight-line code that each CTA runs a few
// times, so their time is that of fetching it: divisions and the key tiles of a
// unit are functions that are not inlined (405 rows over a cache: 101 -> 95 us).
__device__ __noinline__ uint32_t aw_div(uint32_t a, uint32_t b) { return a / b; }
__device__ __forceinline__ int aw_unit_of(const WindowArgs& w, int i) {   // win_unit
  return w.unit == 1 ? i : (int)aw_div((uint32_t)(i - w.origin + w.unit), (uint32_t)w.unit) - 1;
}
// Key tiles of a unit (U rows): [0, nsink) and [wbeg, wbeg + n - nsink).
struct AwUnit { int rows, pos0, lo, hi, first, nsink, wbeg, n; };
__device__ __forceinline__ AwUnit aw_unit(const WindowArgs& w, int U, int rows, int keys, int unit) {
  AwUnit p;
  const int at = unit * U;
  p.rows = min(U, rows - at);
  p.pos0 = keys - rows + at;
  const int u0 = aw_unit_of(w, p.pos0), u1 = aw_unit_of(w, p.pos0 + p.rows - 1);
  p.lo = win_lo_of(w, u0, keys);
  p.hi = win_hi_of(w, u1, keys);
  p.first = min(w.first, win_lo_of(w, u1, keys));   // first keys that only they make visible
  p.wbeg = p.lo >> 7;
  p.nsink = min((p.first + 127) >> 7, p.wbeg);
  p.n = p.nsink + ((p.hi + 127) >> 7) - p.wbeg;
  return p;
}
__device__ __forceinline__ int aw_units(const AttnWinArgs& a, int rows) { return aw_div(rows + a.U - 1, a.U); }
__device__ __forceinline__ int aw_groups(const AttnWinArgs& a, int rows) { return aw_div(rows + a.U * a.M - 1, a.U * a.M); }
// The weight of a group of M units: its key tiles over M, from its first and last
// unit's.
__device__ __noinline__ int aw_weight(WindowArgs w, int U, int M, int rows, int keys, int group) {
  const int p0 = group * M, n0 = aw_unit(w, U, rows, keys, p0).n;
  if (M == 1) return n0;
  const int p1 = min(p0 + M, (int)aw_div(rows + U - 1, U)) - 1;
  return aw_div((n0 + aw_unit(w, U, rows, keys, p1).n) * (p1 - p0 + 1) + 2 * M - 1, 2 * M);
}
__device__ __forceinline__ int aw_group(const AttnWinArgs& a, const AwSeq& q, int group) {
  return aw_weight(a.w, a.U, a.M, q.rows, q.keys, group);
}

// Where gang g's run begins, before the move to a near border: all g / gangs.
struct AwBorder {
  int each, rest;
  uint64_t inv;                  // 2^32 / gangs + 1; rest g is below 2^16
  __host__ __device__ __forceinline__ AwBorder(int all, int gangs, uint64_t gangs_inv)
      : each(all / gangs), rest(all - each * gangs), inv(gangs_inv) {}
  __host__ __device__ __forceinline__ int at(int g) const { return each * g + (int)(((uint32_t)(rest * g) * inv) >> 32); }
};
// Where a run begins: `off` of the weight n of group `group` of sequence `seq`,
// head `head`; off = n: at the end of that group.
struct AwLoc { int head, seq, group, off, n, x; };
struct AwShared {
  AwLoc loc[2];
  int total;
};
// A document's runs are known to the host, which passes where they begin (the
// device's own setup: 3 us of a call).
constexpr int kMaxGangs = 160;
template <int MODE>
struct AwRuns {};
template <>
struct AwRuns<0> {
  CUtensorMap o;      // the results: boxes of a softmax warp's 32 (row, head) pairs x 64 channels
  int all;
  struct { int head, group, off, n, x; } begin[kMaxGangs + 1];
};
// The move of a run's end to a group's that is near.
__host__ __device__ __forceinline__ void aw_snap(int& off, int n, int& x) {
  if (off <= kSnap) {
    x -= off;
    off = 0;
  } else if (n - off <= kSnap) {
    x += n - off;
    off = n;
  }
}

__device__ __forceinline__ int warp_prefix(int v) {   // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, d);
    if ((int)(threadIdx.x & 31) >= d) v += t;
  }
  return v;
}

// A whole warp: the weights before sequence s sum to pre[s] (of one head), all
// of them to `per_head`.
template <bool PAGED>
__device__ __forceinline__ AwLoc aw_locate(const AttnWinArgs& a, const int* pre, int per_head, int x) {
  AwLoc l;
  const int lane = threadIdx.x & 31;
  l.x = x;
  l.head = (int)aw_div(x, per_head);
  l.seq = l.group = l.off = l.n = 0;
  if (l.head >= a.c.n_kv_heads) return l;
  int y = x - l.head * per_head;
  int s = 0;
  for (int lo = 0, hi = a.c.n_seqs - 1; lo <= hi;) {   // the last sequence that begins at or before y
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= y) { s = mid; lo = mid + 1; } else { hi = mid - 1; }
  }
  y -= pre[s];
  const AwSeq q = aw_seq<PAGED>(a, s);
  const int ng = aw_groups(a, q.rows);
  l.seq = s;
  for (int p0 = 0; p0 < ng; p0 += 32) {
    const int n = p0 + lane < ng ? aw_group(a, q, p0 + lane) : 0, sum = warp_prefix(n);
    const unsigned over = __ballot_sync(0xffffffffu, sum > y);
    if (over) {
      const int w = __ffs(over) - 1;
      l.group = p0 + w;
      l.n = __shfl_sync(0xffffffffu, n, w);
      l.off = y - (__shfl_sync(0xffffffffu, sum, w) - l.n);
      break;
    }
    y -= __shfl_sync(0xffffffffu, sum, 31);
  }
  aw_snap(l.off, l.n, l.x);
  return l;
}

// A segment: key tiles [off, off + cnt) of a unit (cnt 0: the run's end).
struct AwSeg {
  int head, seq, row0, rows;     // KV head, sequence, the unit's first row and its rows
  int pos0, keys;                // its position, keys of the sequence
  int lo, hi, first;             // slots that some row of the unit sees: [lo, hi), [0, first)
  int nsink, wbeg, off, cnt, n;  // n: all key tiles of the unit
  int owner, parts;              // the CTA that the unit's parts count in at; 2 x their number at most + tail()
  // whether the gang's run holds the unit's beginning
  __device__ __forceinline__ int tail() const { return parts & 1; }
  __device__ __forceinline__ int key_tile(int j) const {   // j counts from the segment's first
    const int t = off + j;
    return t < nsink ? t : wbeg + t - nsink;
  }
};
static_assert(sizeof(AwSeg) == 64, "a segment is 64 bytes");

// One 128-key tile: two 64-channel boxes of a document's rows, or the boxes of
// the pages it spans, one lane each.  aw_page: this lane's page, n_pages (out of
// range: reads as zeros) for slots of no row of the unit and for table entries
// out of range.
__device__ __forceinline__ int aw_page(const AttnWinArgs& a, const AwSeg& g, int tile, int lane) {
  const int rows = min(a.c.page_size, 128);
  if (lane >= 256 / rows) return 0;
  const int slot = tile * 128 + (lane >> 1) * rows;
  if (slot >= g.keys || !(slot < g.first || (slot + rows > g.lo && slot < g.hi))) return a.c.n_pages;
  const int id = a.c.table[(int64_t)g.seq * a.c.table_width + (slot >> a.c.page_shift)];
  if (id >= 0 && id < a.c.n_pages) return id;
  record_error(a.err, DEVERR_INDEX);
  return a.c.n_pages;
}
template <bool PAGED>
__device__ __forceinline__ void aw_load_kv(uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, const AttnWinArgs& a,
                                           int head, int tile, int page, int lane) {
  if (!PAGED) {
    if (lane < 2) tma_load_3d(dst + lane * AW_BOX, tm, bar, lane * 64, head, tile * 128);
    return;
  }
  const int ps = a.c.page_size, rows = min(ps, 128);
  if (lane >= 256 / rows) return;
  const int box = lane >> 1, half = lane & 1;
  tma_load_4d(dst + half * AW_BOX + box * rows * 128, tm, bar, half * 64, (tile * 128 + box * rows) & (ps - 1), head,
              page);
}

struct AwSmem {
  uint8_t *q, *k, *v, *stage;
  float2* stats;   // slot B's maxima and sums, for slot A
  AwSeg *seg, *cut;   // the ring; the units that the run's ends cut
  int* joins;         // [2][8] which of these this CTA completed, per softmax warp
  uint64_t *seg_full, *seg_empty, *q_full, *q_empty, *k_full, *k_empty, *v_full, *v_empty, *s_full, *p_full, *o_final,
      *b_ready, *a_done, *drain;
};
}  // namespace

namespace {
// A whole warp takes the next segment (its n'th) out of the ring, null at the
// end of the run or when a wait ran out; and gives it back.
__device__ __forceinline__ const AwSeg* aw_take(const AwSmem& sm, uint32_t n, const WaitCtl& ctl) {
  if (!at_wait(&sm.seg_full[n % AW_SEGS], (n / AW_SEGS) & 1u, ctl)) return nullptr;
  const AwSeg* g = &sm.seg[n % AW_SEGS];
  return g->cnt > 0 ? g : nullptr;
}
__device__ __forceinline__ void aw_give(const AwSmem& sm, uint32_t n) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.seg_empty[n % AW_SEGS]);
}
// Eight rows of a unit's results out of its parts, in the order of their key
// tiles: rows 32 q + r0 and on of a slot, who = 4 slot + q the softmax warp they
// were counted in by.
__device__ __forceinline__ void aw_join(const AttnWinArgs& a, const AwSeg& g, int who, int r0) {
  const int lane = threadIdx.x & 31, t = who >> 2, ts = a.part_slots / 2;
  const int row0 = (who & 3) * 32 + r0, rbase = t * a.R, nrows = min(g.rows - rbase, a.R), rows = min(nrows * a.G - row0, 8);
  if (rows <= 0) return;
  const int row = row0 + min(lane & 7, rows - 1), r = row / a.G, qhead = g.head * a.G + row - r * a.G;   // lane's row
  const int64_t at = ((int64_t)(g.row0 + rbase + r) * a.H + qhead) * 128;   // in o
  const int64_t tile_elems = (int64_t)a.part_rows * kPartRow, next = (int64_t)a.M * a.part_slots * tile_elems;
  const float* from = a.part + ((int64_t)g.owner * a.part_slots + t) * tile_elems + (int64_t)row0 * kPartRow;
  // The unit's parts, 32 CTAs at a time: bit s for the k + s'th from its owner.
  auto parts_at = [&](int k) -> unsigned {
    const int cta = g.owner + (k + lane) * a.M;
    const int n = k + lane < (g.parts >> 1) ? __ldcg(a.ctrl + cta * kCtrl + (k + lane == 0 ? kCtrlTail : kCtrlHead) + who) : 0;
    return __ballot_sync(0xffffffffu, n > 0);
  };
  auto part_at = [&](int s) -> const float* { return from + s * next + (s == 0 ? ts * tile_elems : 0); };
  float m = -INFINITY, l = 0.0f;      // of lane's row
  float4 acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int k = 0; k < (g.parts >> 1); k += 32)
    for (unsigned have = parts_at(k); have;) {
      // two parts at a time: their loads are in flight together
      const float* p[2];
      float2 ml[2];
      float4 v[2][8];
      int n = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!have) break;
        p[i] = part_at(k + __ffs(have) - 1);
        have &= have - 1;
        ml[i] = __ldcg(reinterpret_cast<const float2*>(p[i] + (int64_t)(row - row0) * kPartRow + 128));
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[i][e] = __ldcg(reinterpret_cast<const float4*>(p[i] + (int64_t)min(e, rows - 1) * kPartRow + lane * 4));
        n = i + 1;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i >= n) break;
        const float top = fmaxf(m, ml[i].x), ref = top == -INFINITY ? 0.0f : top;
        const float f0 = at_ex2(m - ref), f1 = at_ex2(ml[i].x - ref);
        l = l * f0 + ml[i].y * f1;
        m = top;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float e0 = __shfl_sync(0xffffffffu, f0, e), e1 = __shfl_sync(0xffffffffu, f1, e);
          acc[e].x = acc[e].x * e0 + v[i][e].x * e1;
          acc[e].y = acc[e].y * e0 + v[i][e].y * e1;
          acc[e].z = acc[e].z * e0 + v[i][e].z * e1;
          acc[e].w = acc[e].w * e0 + v[i][e].w * e1;
        }
      }
    }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  if (lane < rows && a.lse != nullptr) {
    float* to = a.lse + (int64_t)qhead * a.n_rows + g.row0 + rbase + r;
    if (in_bounds<float>(a.lse, a.lse_elems, to, 1, a.err, 52)) *to = (m + log2f(l)) * 0.69314718055994530942f;
  }
  const unsigned fits = __ballot_sync(0xffffffffu, lane < rows && in_bounds<__nv_bfloat16>(a.o, a.o_elems, a.o + at, 128, a.err, 50));
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float f = __shfl_sync(0xffffffffu, inv, e);
    const int64_t to = __shfl_sync(0xffffffffu, at, e) + lane * 4;
    if ((fits >> e) & 1u)
      *reinterpret_cast<uint2*>(a.o + to) =
          make_uint2(pack_bf16x2(acc[e].x * f, acc[e].y * f), pack_bf16x2(acc[e].z * f, acc[e].w * f));
  }
}
// Largest of 32 scores (a NaN is not one).
__device__ __forceinline__ float aw_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float aw_max(const uint32_t (&s)[32]) {
  float m0 = __uint_as_float(s[0]), m1 = __uint_as_float(s[1]);
#pragma unroll
  for (int c = 2; c < 30; c += 4) {
    m0 = aw_max3(m0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
    m1 = aw_max3(m1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
  }
  return fmaxf(aw_max3(m0, __uint_as_float(s[30]), __uint_as_float(s[31])), m1);
}
}  // namespace

template <int MODE>
__global__ void __launch_bounds__(AW_THREADS, 1)
    attention_window_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AttnWinArgs a,
                            const __grid_constant__ AwRuns<MODE> runs) {
  // no static shared memory: the dynamic part starts at a multiple of 1024
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  AwSmem sm;
  sm.q = smem_raw;
  constexpr bool PAGED = MODE != AW_DOC;
  constexpr int AW_KST = AwPlan<MODE>::k, AW_VST = AwPlan<MODE>::v, AW_STAGE = AwPlan<MODE>::stage;
  sm.k = sm.q + AwPlan<MODE>::q * AW_TILE;
  sm.v = sm.k + AW_KST * AW_TILE;
  sm.stage = sm.v + AW_VST * AW_TILE;
  sm.stats = reinterpret_cast<float2*>(sm.stage + 8 * AW_STAGE);
  sm.seg = reinterpret_cast<AwSeg*>(sm.stats + 128);
  sm.cut = sm.seg + AW_SEGS;
  sm.joins = reinterpret_cast<int*>(sm.cut + 2);
  sm.seg_full = reinterpret_cast<uint64_t*>(sm.joins + 16);
  sm.seg_empty = sm.seg_full + AW_SEGS;
  sm.q_full = sm.seg_empty + AW_SEGS;
  sm.q_empty = sm.q_full + 1;
  sm.k_full = sm.q_empty + 1;
  sm.k_empty = sm.k_full + AW_KST;
  sm.v_full = sm.k_empty + AW_KST;
  sm.v_empty = sm.v_full + AW_VST;
  sm.s_full = sm.v_empty + AW_VST;
  sm.p_full = sm.s_full + 2;
  sm.o_final = sm.p_full + 2;
  sm.b_ready = sm.o_final + 2;
  sm.a_done = sm.b_ready + 1;
  sm.drain = sm.a_done + 1;
  AwShared* sh = reinterpret_cast<AwShared*>(sm.drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sh + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  static_assert(128 * 8 + (AW_SEGS + 2) * sizeof(AwSeg) + 64 + (11 + 2 * AW_SEGS + 2 * AW_KST + 2 * AW_VST) * 8 + sizeof(AwShared) + 8 <=
                    AwPlan<MODE>::tail,
                "segments, barriers and setup fit");

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < AW_SEGS; ++s) { mbar_init(&sm.seg_full[s], 1); mbar_init(&sm.seg_empty[s], 11); }
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
    mbar_init(sm.a_done, 4);
    mbar_init(sm.drain, 1);
    for (int e = 0; e < 16; ++e) sm.joins[e] = 0;
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

  // ---- the run of this CTA.  A cache: weights of each sequence, their prefix sums (in the
  // K ring, before its first load), both ends of the run
  int all = 0;
  const int gang = (int)aw_div(blockIdx.x, a.M);
  if constexpr (MODE == AW_DOC) {
    all = runs.all;
    if (threadIdx.x < 2) {
      const auto& r = runs.begin[gang + threadIdx.x];
      sh->loc[threadIdx.x] = {r.head, 0, r.group, r.off, r.n, r.x};
    }
  } else {
    int* pre = reinterpret_cast<int*>(sm.k);
    const int ns = a.c.n_seqs;
    constexpr int kWarps = AW_THREADS / 32;
    if (ns == 1) {   // the whole CTA sums one sequence
      const AwSeq q = aw_seq<PAGED>(a, 0);
      if (PAGED && q.keys < 0 && blockIdx.x == 0 && threadIdx.x == 0) record_error(a.err, DEVERR_INDEX);
      int n = 0;
      for (int p = threadIdx.x, ng = aw_groups(a, q.rows); p < ng; p += AW_THREADS) n += aw_group(a, q, p);
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) pre[1 + warp] = n;
      __syncthreads();
      n = lane < kWarps ? pre[1 + lane] : 0;
      n = __reduce_add_sync(0xffffffffu, n);
      if (threadIdx.x == 0) {
        pre[0] = 0;
        sh->total = n;
      }
    } else {
      for (int s = threadIdx.x; s < ns; s += AW_THREADS) {
        const AwSeq q = aw_seq<PAGED>(a, s);
        if (PAGED && q.keys < 0 && blockIdx.x == 0) record_error(a.err, DEVERR_INDEX);
        const int ng = aw_groups(a, q.rows);
        pre[s] = ng > 2 ? -1 : (ng > 0 ? aw_group(a, q, 0) : 0) + (ng > 1 ? aw_group(a, q, 1) : 0);
      }
      __syncthreads();
      for (int s = warp; s < ns; s += kWarps) {
        if (pre[s] >= 0) continue;
        const AwSeq q = aw_seq<PAGED>(a, s);
        int n = 0;
        for (int p = lane, ng = aw_groups(a, q.rows); p < ng; p += 32) n += aw_group(a, q, p);
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) pre[s] = n;
      }
      __syncthreads();
      if (warp == 0) {
        int carry = 0;
        for (int s0 = 0; s0 < ns; s0 += 32) {
          const int mine = s0 + lane < ns ? pre[s0 + lane] : 0, sum = warp_prefix(mine);
          if (s0 + lane < ns) pre[s0 + lane] = carry + sum - mine;
          carry += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane == 0) sh->total = carry;
      }
    }
    __syncthreads();
    const int per_head = sh->total;
    all = per_head * a.c.n_kv_heads;
    if (warp < 2 && all > 0) {
      const AwLoc l = aw_locate<PAGED>(a, pre, per_head, AwBorder(all, a.gangs, a.gangs_inv).at(gang + warp));
      if (lane == 0) sh->loc[warp] = l;
    }
  }
  fence_proxy_async_smem();   // the sums were read; the ring's loads may overwrite them
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl ctl{abort_flag, a.err, KID_ATTN_WIN};
  const bool skip = *ctl.flag != 0 || all <= 0 || sh->loc[1].x <= sh->loc[0].x;

  // The softmax warps get registers of the others' (their
  // share at launch is AW_REGS each, where the scores spill; the build checks that it is).
  static_assert(128 * AW_REGS_FEW + 256 * AW_REGS_MANY <= AW_THREADS * AW_REGS, "the split is within the launch's registers");
  if (skip) {
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(AW_REGS_FEW));
    if (warp == 3) {
      // ------------------------------------------------------------ the run's segments
      const AwLoc b = sh->loc[0];
      int rem = sh->loc[1].x - b.x;
      int head = b.head, seq = b.seq, group = b.group, off = b.off;
      AwSeq q = aw_seq<PAGED>(a, seq);
      int ng = aw_groups(a, q.rows);
      bool here = off < b.n, first_group = here; // else the run begins with the group after this one
      const int member = blockIdx.x - gang * a.M;
      int x0 = b.x - (here ? off : 0), w0 = 0;   // where the group begins, its weight
      for (uint32_t n = 0;;) {
        if (!here && rem > 0) {
          off = 0;
          x0 += w0;
          if (++group >= ng) {
            group = 0;
            do {
              if (++seq == a.c.n_seqs) {
                seq = 0;
                if (++head == a.c.n_kv_heads) break;
              }
              if (PAGED) q = aw_seq<PAGED>(a, seq);
            } while (q.rows == 0);
            ng = aw_groups(a, q.rows);
          }
          if (head == a.c.n_kv_heads) rem = 0;   // not reached while the metadata stay as they are
        }
        here = false;
        AwSeg g;
        g.cnt = 0;
        if (rem > 0) {
          // the gang's part of the group's weight, in proportion of this CTA's unit.
          // The members take turns, so that units of growing windows even out.
          const int weight = first_group ? b.n : aw_group(a, q, group), part = min(rem, weight - off);
          int turn = member + group + head + seq;
          turn -= (int)aw_div(turn, a.M) * a.M;
          const int unit = group * a.M + turn;
          first_group = false;
          w0 = weight;
          rem -= part;
          if (unit >= aw_units(a, q.rows)) continue;
          const AwUnit p = aw_unit(a.w, a.U, q.rows, q.keys, unit);
          const float ratio = __fdividef((float)p.n, (float)weight);
          const int done = off + part;
          g.off = min((int)((float)off * ratio), p.n);
          g.cnt = (done == weight ? p.n : min((int)((float)done * ratio), p.n)) - g.off;
          if (g.cnt == 0) continue;
          g.head = head;
          g.seq = seq;
          g.row0 = q.row0 + unit * a.U;
          g.rows = p.rows;
          g.pos0 = p.pos0;
          g.keys = q.keys;
          g.lo = p.lo;
          g.hi = p.hi;
          g.first = p.first;
          g.nsink = p.nsink;
          g.wbeg = p.wbeg;
          g.n = p.n;
          g.owner = g.parts = 0;
          if (g.cnt < p.n) {
            // the gangs whose runs hold the group's beginning and its end: the last
            // whose border, as it is after the move, is no later
            const AwBorder border(all, a.gangs, a.gangs_inv);
            int first = gang, last = gang;
            while (off > 0 && border.at(first) > x0 + kSnap) --first;
            while (last + 1 < a.gangs && border.at(last + 1) < x0 + weight - kSnap) ++last;
            g.owner = first * a.M + member;
            g.parts = 2 * (last - first + 1) + (off == 0 ? 1 : 0);
          }
        }
        if (!at_wait(&sm.seg_empty[n % AW_SEGS], ((n / AW_SEGS) & 1u) ^ 1u, ctl)) break;
        if (lane == 0) {
          sm.seg[n % AW_SEGS] = g;
          if (g.cnt > 0 && g.cnt < g.n) sm.cut[g.tail()] = g;
          mbar_arrive(&sm.seg_full[n % AW_SEGS]);
        }
        __syncwarp();
        if (g.cnt == 0) break;
        ++n;
      }
    } else if (warp == 0) {
      // ------------------------------------------------------------ producer of Q and K
      bool ok = true;
      uint32_t items = 0, st = 0, ph = 0, issued = 0;
      for (const AwSeg* g; ok && (g = aw_take(sm, items, ctl)) != nullptr;) {
        if (!at_wait(sm.q_empty, (items & 1u) ^ 1u, ctl)) { ok = false; break; }
        const int slots = MODE != AW_ROWS && g->rows > a.R ? 2 : 1;
        if (lane == 0) mbar_arrive_expect_tx(sm.q_full, (uint32_t)(slots * a.R * a.G * 256));
        __syncwarp();
        if (lane < 2 * slots)
          tma_load_4d(sm.q + (lane >> 1) * AW_TILE + (lane & 1) * AW_BOX, &tmQ, sm.q_full, (lane & 1) * 64, 0, g->head,
                      g->row0 + (lane >> 1) * a.R);
        int page = PAGED ? aw_page(a, *g, g->key_tile(0), lane) : 0;
        for (int j = 0; j < g->cnt; ++j) {
          // the next tile's table entry arrives during the wait
          const int next = PAGED && j + 1 < g->cnt ? aw_page(a, *g, g->key_tile(j + 1), lane) : 0;
          if (!at_wait(&sm.k_empty[st], ph ^ 1u, ctl)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&sm.k_full[st], AW_TILE);
          __syncwarp();
          aw_load_kv<PAGED>(sm.k + st * AW_TILE, &tmK, &sm.k_full[st], a, g->head, g->key_tile(j), page, lane);
          page = next;
          ++issued;
          if (++st == AW_KST) { st = 0; ph ^= 1u; }
        }
        aw_give(sm, items);
        ++items;
      }
      // a wait that ran out, here or elsewhere: let issued loads land before the CTA exits
      if (*ctl.flag && lane == 0) {
        if (items > 0) at_drain(sm.q_full, (items - 1) & 1u);
        for (uint32_t j = issued > AW_KST ? issued - AW_KST : 0; j < issued; ++j)
          at_drain(&sm.k_full[j % AW_KST], (j / AW_KST) & 1u);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------------------ producer of V
      bool ok = true;
      uint32_t items = 0, st = 0, ph = 0, issued = 0;
      for (const AwSeg* g; ok && (g = aw_take(sm, items, ctl)) != nullptr; ++items) {
        int page = PAGED ? aw_page(a, *g, g->key_tile(0), lane) : 0;
        for (int j = 0; j < g->cnt; ++j) {
          const int next = PAGED && j + 1 < g->cnt ? aw_page(a, *g, g->key_tile(j + 1), lane) : 0;
          if (!at_wait(&sm.v_empty[st], ph ^ 1u, ctl)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&sm.v_full[st], AW_TILE);
          __syncwarp();
          aw_load_kv<PAGED>(sm.v + st * AW_TILE, &tmV, &sm.v_full[st], a, g->head, g->key_tile(j), page, lane);
          page = next;
          ++issued;
          if (++st == AW_VST) { st = 0; ph ^= 1u; }
        }
        aw_give(sm, items);
      }
      if (*ctl.flag && lane == 0)
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
      for (const AwSeg* g; ok && (g = aw_take(sm, items, ctl)) != nullptr;) {
        const bool dual = MODE != AW_ROWS && g->rows > a.R;
        const int cnt = g->cnt, na = dual ? cnt : (cnt + 1) >> 1, nb = dual ? cnt : cnt >> 1;
        int left = na + nb;                       // S products of this segment still to issue
        ok = at_wait(sm.q_full, items & 1u, ctl);
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
                const int valid = g->keys - g->key_tile(dual ? j : 2 * j + t) * 128;
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
        aw_give(sm, items);
        ++items;
      }
      if (*ctl.flag) {   // a wait ran out: let issued products end
        at_commit(sm.drain, one);
        if (one) at_drain(sm.drain, 0);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(AW_REGS_MANY));
    const int t = (warp - 4) >> 2;
    const int qq = warp & 3;
    const int row = qq * 32 + lane, row_r = (int)aw_div(row, a.G);   // (row, head) pair of the tile, its row
    const uint32_t s_base = tmem_addr(tmem_base, (uint32_t)(qq * 32), (uint32_t)(t * 128));
    const uint32_t o_base = s_base + 256u;
    const float sl2 = a.scale_log2;
    uint32_t sph = 0, oph = 0, jph = 0;
    bool given = false;                        // slot B: A may still read the last segment's results
    bool ok = true;
    uint32_t items = 0;
    for (const AwSeg* g; ok && (g = aw_take(sm, items, ctl)) != nullptr; aw_give(sm, items), ++items) {
      const bool dual = MODE != AW_ROWS && g->rows > a.R;
      const int cnt = g->cnt, nt = dual ? cnt : (t == 0 ? (cnt + 1) >> 1 : cnt >> 1);
      if (nt == 0) continue;                   // one key tile: slot A alone
      if (given) {                             // before its first product may overwrite them
        if (!at_wait(sm.a_done, jph, ctl)) { ok = false; break; }
        jph ^= 1u;
        given = false;
      }
      const int rbase = dual && t ? a.R : 0;   // first row of the slot in the unit
      const int nrows = dual && t ? g->rows - a.R : min(g->rows, a.R);
      const bool active = qq * 32 < nrows * a.G;
      int lo, hi, first;
      {
        const int pos = g->pos0 + rbase + min(row_r, nrows - 1), keys = g->keys;
        const int u = aw_unit_of(a.w, pos);
        lo = win_lo_of(a.w, u, keys);
        hi = win_hi_of(a.w, u, keys);
        first = min(a.w.first, hi);
      }
      const int step = dual ? 1 : 2, off = g->off + (dual ? 0 : t), nsink = g->nsink, wshift = g->wbeg - nsink;
      float m_used = -INFINITY, l_run = 0.0f;
      for (int j = 0; j < nt; ++j) {
        if (!at_wait(&sm.s_full[t], sph, ctl)) { ok = false; break; }
        sph ^= 1u;
        if (active) {
          tc_fence_after();
          const int tile = off + j * step, k0 = (tile < nsink ? tile : tile + wshift) * 128;
          if (__all_sync(0xffffffffu, k0 >= first && (k0 >= hi || k0 + 128 <= lo))) {
            // nothing of the tile is visible to this warp's rows
            const uint32_t zero[16] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) at_tmem_st16(s_base + (uint32_t)(q4 * 16), zero);
          } else {
            uint32_t s[4][32];
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) tmem_ld32(s_base + (uint32_t)(q4 * 32), s[q4]);
            tmem_ld_wait(s);
            if (!__all_sync(0xffffffffu, (k0 >= lo && k0 + 128 <= hi) || k0 + 128 <= first)) {
#pragma unroll
              for (int q4 = 0; q4 < 4; ++q4) {
                const int at = k0 + q4 * 32;
                const uint32_t see = (win_bits(hi - at) & ~win_bits(lo - at)) | win_bits(first - at);
                if (__all_sync(0xffffffffu, see == 0xffffffffu)) continue;
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (!((see >> c) & 1u)) s[q4][c] = __float_as_uint(-INFINITY);
              }
            }
            const float m_tile = fmaxf(fmaxf(aw_max(s[0]), aw_max(s[1])), fmaxf(aw_max(s[2]), aw_max(s[3]))) * sl2;
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
          }
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[t]);
      }
      if (!ok || !at_wait(&sm.o_final[t], oph, ctl)) { ok = false; break; }
      oph ^= 1u;
      tc_fence_after();

      // ---- results.  One tile of rows: slot B leaves its maxima and sums in
      // shared memory, and slot A reads both accumulators.
      const bool valid = row < nrows * a.G;
      const bool joint = !dual && cnt > 1;
      if (joint && t == 1) {
        if (active) sm.stats[row] = make_float2(m_used, l_run);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.b_ready);
        given = true;
        continue;
      }
      const int64_t tile_elems = (int64_t)a.part_rows * kPartRow;
      const int ts = a.part_slots / 2;
      const bool whole = g->cnt == g->n;
      float fa = 1.0f, fb = 0.0f, l = l_run, m = m_used, f_own = 1.0f;
      if (joint) {
        if (!at_wait(sm.b_ready, jph, ctl)) { ok = false; break; }
        jph ^= 1u;
        tc_fence_after();
        if (active) {
          const float2 b = sm.stats[row];
          m = fmaxf(m_used, b.x);
          const float m_ref = m == -INFINITY ? 0.0f : m;
          fa = at_ex2(m_used - m_ref);
          fb = at_ex2(b.x - m_ref);
          l = l_run * fa + b.y * fb;
        }
      }
      const int r = row_r, qhead = g->head * a.G + row - r * a.G;
      const int64_t at = ((int64_t)(g->row0 + rbase + r) * a.H + qhead) * 128;   // the row in o
      const int who = (dual ? t : 0) * 4 + qq;
      const bool few = MODE != AW_ROWS && g->parts <= 2 * kFew + 1;
      // A part of a unit.  Few parts: counted in now; who completes the count
      // goes on, with the others' parts (have: those, by the order of the gangs).
      bool last = whole;
      unsigned have = 0, own = 0;
      float* to = a.part + ((int64_t)blockIdx.x * a.part_slots + (g->tail() ? ts : 0) + (dual ? t : 0)) * tile_elems;
      const float* from = nullptr;
      const int64_t next = (int64_t)a.M * a.part_slots * tile_elems;
      if (few && active && !whole) {
        int done = 0;
        if (lane == 0) done = atomicAdd(a.ctrl + g->owner * kCtrl + who, g->cnt) + g->cnt;
        last = __shfl_sync(0xffffffffu, done, 0) == g->n;
        if (last) {
          from = a.part + (int64_t)g->owner * a.part_slots * tile_elems + (dual ? t : 0) * tile_elems;
          own = 1u << ((blockIdx.x - g->owner) / a.M);
          const volatile int* flag = a.ctrl + (g->owner + lane * a.M) * kCtrl + (lane == 0 ? kCtrlTail : kCtrlHead) + who;
          const bool look = lane < (g->parts >> 1) && !((own >> lane) & 1u);
          const uint64_t t0 = globaltimer();
          for (uint32_t i = 1;; ++i) {
            const int n = look ? *flag : 0;
            have = __ballot_sync(0xffffffffu, n > 0);
            if (__reduce_add_sync(0xffffffffu, n) + g->cnt == g->n) break;
            if (__any_sync(0xffffffffu, (i & 31u) == 0 && wait_gives_up(ctl, t0, kSiteStreamKFlag))) { ok = false; break; }
          }
          if (!ok) break;
          __threadfence();
          // maximum and sum of all parts, in their order
          const float mo = m, lo_ = l;
          float mt = -INFINITY, lt = 0.0f;
          for (unsigned h = have | own; h; h &= h - 1) {
            const int k = __ffs(h) - 1;
            float mk = mo, lk = lo_;
            if (!((own >> k) & 1u)) {
              const float* p = from + k * next + (k == 0 ? ts * tile_elems : 0);
              const int64_t rr = min(row, nrows * a.G - 1);
              mk = __ldcg(p + 128 * (int64_t)a.part_rows + rr);
              lk = __ldcg(p + 129 * (int64_t)a.part_rows + rr);
            }
            const float top = fmaxf(mt, mk), ref = top == -INFINITY ? 0.0f : top;
            lt = __fadd_rn(__fmul_rn(lt, at_ex2(mt - ref)), __fmul_rn(lk, at_ex2(mk - ref)));
            mt = top;
          }
          m = mt;
          l = lt;
          f_own = at_ex2(mo - (mt == -INFINITY ? 0.0f : mt));
        }
      }
      float inv = 1.0f;
      if (last) inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // a NaN stays one
      if (whole) {
        fa *= inv;
        fb *= inv;
      }
      uint8_t* stg = sm.stage + (warp - 4) * AW_STAGE;
      const unsigned rows_out = __ballot_sync(
          0xffffffffu, last && valid && in_bounds<__nv_bfloat16>(a.o, a.o_elems, a.o + at, 128, a.err, 50));
      if (active) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {          // 32 channels at a time
          uint32_t o[32];
          tmem_ld32(o_base + (uint32_t)(c * 32), o);
          tmem_ld_wait(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fa);
          if (joint) {
            uint32_t ob[32];
            tmem_ld32(o_base + 128u + (uint32_t)(c * 32), ob);
            tmem_ld_wait(ob);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(__fmaf_rn(__uint_as_float(ob[e]), fb, __uint_as_float(o[e])));
          }
          if (few && last && !whole) {   // (few: never of single rows)
            // the parts in their order, each scaled to the common maximum as it would be
            // out of the workspace (both slots' accumulators joined, then one rounded
            // product), so that the sums do not depend on which part is the own one
            float sum[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) sum[e] = 0.0f;
            const float m_ref = m == -INFINITY ? 0.0f : m;
            for (unsigned h = have | own; h; h &= h - 1) {
              const int k = __ffs(h) - 1;
              if ((own >> k) & 1u) {
#pragma unroll
                for (int e = 0; e < 32; ++e) sum[e] = __fadd_rn(sum[e], __fmul_rn(__uint_as_float(o[e]), f_own));
                continue;
              }
              const float* p = from + k * next + (k == 0 ? ts * tile_elems : 0);
              const int64_t rr = min(row, nrows * a.G - 1);
              float v[32];
              const float mk = __ldcg(p + 128 * (int64_t)a.part_rows + rr);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __ldcg(p + (int64_t)(c * 32 + e) * a.part_rows + rr);
              const float f = at_ex2(mk - m_ref);
#pragma unroll
              for (int e = 0; e < 32; ++e) sum[e] = __fadd_rn(sum[e], __fmul_rn(v[e], f));
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(sum[e] * inv);
          }
          if (last) {
            uint4 w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              w[u] = make_uint4(pack_bf16x2(__uint_as_float(o[u * 8]), __uint_as_float(o[u * 8 + 1])),
                                pack_bf16x2(__uint_as_float(o[u * 8 + 2]), __uint_as_float(o[u * 8 + 3])),
                                pack_bf16x2(__uint_as_float(o[u * 8 + 4]), __uint_as_float(o[u * 8 + 5])),
                                pack_bf16x2(__uint_as_float(o[u * 8 + 6]), __uint_as_float(o[u * 8 + 7])));
            if (AW_STAGE == 0) {
              if ((rows_out >> lane) & 1u) {
#pragma unroll
                for (int u = 0; u < 4; ++u) *reinterpret_cast<uint4*>(a.o + at + c * 32 + u * 8) = w[u];
              }
            } else {
              // through the warp's stage (16-byte unit u of a row at u ^ (row & 7)),
              // so that 64 channels of a row leave as one line
#pragma unroll
              for (int u = 0; u < 4; ++u)
                *reinterpret_cast<uint4*>(stg + lane * 128 + ((((c & 1) * 4 + u) ^ (lane & 7)) << 4)) = w[u];
              if ((c & 1) && a.o_tma) {
                // rows past the document are outside the map and not written
                fence_proxy_async_smem();
                __syncwarp();
                if constexpr (MODE == AW_DOC)
                  if (lane == 0) {
                    at_tma_store_4d(&runs.o, stg, (c >> 1) * 64, 0, g->head, g->row0 + rbase + row_r);
                    at_tma_store_read();   // before the stage is written again
                  }
                __syncwarp();
              } else if (c & 1) {
                __syncwarp();
#pragma unroll
                for (int it = 0; it < 8; ++it) {
                  const int rr = it * 4 + (lane >> 3), u = lane & 7;
                  const int64_t dst = __shfl_sync(0xffffffffu, at, rr) + (c >> 1) * 64 + u * 8;
                  if ((rows_out >> rr) & 1u)
                    *reinterpret_cast<uint4*>(a.o + dst) =
                        *reinterpret_cast<const uint4*>(stg + rr * 128 + ((u ^ (rr & 7)) << 4));
                }
                __syncwarp();
              }
            }
          } else if (valid && in_bounds<float>(a.part, a.part_elems, to, (size_t)tile_elems, a.err, 51)) {
            if (!few) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<uint4*>(to + (int64_t)row * kPartRow + c * 32 + e) =
                    make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) to[(int64_t)(c * 32 + e) * a.part_rows + row] = __uint_as_float(o[e]);
            }
          }
        }
        tc_fence_before();
      }
      if (joint) {
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.a_done);
      }
      if (!active) continue;
      if (last) {
        float* lse_at = a.lse + (int64_t)qhead * a.n_rows + g->row0 + rbase + r;
        if (valid && a.lse != nullptr && in_bounds<float>(a.lse, a.lse_elems, lse_at, 1, a.err, 52))
          *lse_at = (m + log2f(l)) * 0.69314718055994530942f;
        continue;
      }
      if (valid && in_bounds<float>(a.part, a.part_elems, to, (size_t)tile_elems, a.err, 53)) {
        to[few ? 128 * (int64_t)a.part_rows + row : (int64_t)row * kPartRow + 128] = m;
        to[few ? 129 * (int64_t)a.part_rows + row : (int64_t)row * kPartRow + 129] = l;
      }
      __threadfence();
      __syncwarp();
      if (lane == 0) {
        volatile int* flag = a.ctrl + blockIdx.x * kCtrl + (g->tail() ? kCtrlTail : kCtrlHead) + who;
        *flag = g->cnt;
        if (!few) {   // many parts: counted in now; joined after the run (here, the registers are the softmax loop's)
          __threadfence();
          if (atomicAdd(a.ctrl + g->owner * kCtrl + who, g->cnt) + g->cnt == g->n) sm.joins[(g->tail() ? 8 : 0) + who] = 1;
        }
      }
    }
    // ---- units of many parts that this CTA's completed, all softmax warps (which
    // come here from wherever a wait ran out, too)
    asm volatile("bar.sync 1, 256;" ::: "memory");
    __threadfence();
    for (int job = warp - 4; job < 64; job += 8)
      if (sm.joins[job >> 2]) aw_join(a, sm.cut[job >> 5], (job >> 2) & 7, (job & 3) * 8);
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *ctl.flag) record_error(a.err, DEVERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Zeroes the control words of a call whose units may be cut.
__global__ void __launch_bounds__(256) attention_window_start_kernel(int* ctrl, int words) {
  griddep_launch_dependents();
  griddep_wait();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < words) ctrl[i] = 0;
}

// How a call runs.  Units of one tile where the sequences have no more rows than
// that on average, of two otherwise; one CTA per SM, or as many as there are key
// tiles; gangs of M.  What speaks against a larger M: SMs that no gang fits on and,
// where a gang gets few groups, members without a unit in a sequence's last one;
// against a smaller: K and V read from HBM that many times less often shared
// (16,384 rows x 56 heads: 5770 us in gangs of one, 4874 in gangs of eight), taken
// to cost 0.12 / M^2.
size_t attn_win_ctrl_bytes(int ctas) { return ((size_t)ctas * kCtrl * 4 + 255) & ~size_t(255); }
size_t attn_win_part_bytes(int ctas, int rows) { return (size_t)ctas * 4 * rows * kPartRow * 4; }
namespace {
// Where the runs of a document's gangs begin.
void aw_doc_runs(const AttnWinArgs& a, const AttnWinPlan& p, AwRuns<AW_DOC>* runs) {
  const int units = (a.n_rows + a.U - 1) / a.U, groups = (units + a.M - 1) / a.M;
  auto tiles = [&](int unit) -> int {   // aw_unit's n
    const int pos0 = unit * a.U, last = std::min(pos0 + a.U, a.n_rows) - 1;
    const int lo = win_lo(a.w, pos0, a.n_rows), first = std::min(a.w.first, win_lo(a.w, last, a.n_rows));
    return std::min((first + 127) >> 7, lo >> 7) + ((win_hi(a.w, last, a.n_rows) + 127) >> 7) - (lo >> 7);
  };
  auto weight = [&](int g) -> int {     // aw_weight
    const int p0 = g * a.M, p1 = std::min(p0 + a.M, units) - 1;
    return a.M == 1 ? tiles(p0) : ((tiles(p0) + tiles(p1)) * (p1 - p0 + 1) + 2 * a.M - 1) / (2 * a.M);
  };
  int64_t per_head = 0;
  for (int g = 0; g < groups; ++g) per_head += weight(g);
  runs->all = (int)(per_head * a.c.n_kv_heads);
  const AwBorder border(runs->all, a.gangs, a.gangs_inv);
  int g = 0, at = 0, n = weight(0), head = 0;         // the group that holds a border, its beginning in the head
  for (int i = 0; i <= p.gangs; ++i) {
    auto& r = runs->begin[i];
    r = {a.c.n_kv_heads, 0, 0, 0, border.at(i)};
    for (; head < r.x / per_head && head < a.c.n_kv_heads; ++head) {
      g = at = 0;
      n = weight(0);
    }
    if (head == a.c.n_kv_heads) continue;
    const int y = r.x - (int)(head * per_head);
    while (at + n <= y) {
      at += n;
      n = weight(++g);
    }
    r.head = head;
    r.group = g;
    r.n = n;
    r.off = y - at;
    aw_snap(r.off, r.n, r.x);
  }
}
}  // namespace

bool attn_win_plan(AttnWinPlan* p, int64_t n_rows, int64_t kv_heads, int64_t n_seqs, int G, int64_t max_keys, bool paged,
                   const WindowArgs& w) {
  const int64_t R = 128 / G;
  p->mode = !paged ? AW_DOC : (n_rows <= n_seqs * R ? AW_ROWS : AW_CHUNK);
  p->U = (int)(p->mode == AW_ROWS ? R : 2 * R);
  // key tiles of a unit at most: the window of all its rows and the first keys
  int64_t tiles = (max_keys + 127) / 128;
  if (w.left >= 0 && w.right >= 0) {
    const __int128 span = (__int128)((int64_t)w.left + w.right + 2) * w.unit + p->U;
    const __int128 most = span / 128 + 2 + ((int64_t)w.first + 127) / 128;
    if (most < tiles) tiles = (int64_t)most;
  }
  const int64_t units = (n_rows + p->U - 1) / p->U + (n_seqs - 1);
  const __int128 all = (__int128)units * (tiles + 1) * kv_heads;
  if (all >= (__int128)1 << 31) return false;        // the runs are counted in 32 bits
  const int64_t sms = num_sms(), work = units * (tiles > 0 ? tiles : 1) * kv_heads;
  const int ctas = (int)std::min<int64_t>(std::min(work, sms), kMaxGangs);
  const int64_t per_seq = ((n_rows + n_seqs - 1) / n_seqs + p->U - 1) / p->U;   // units of a sequence, on average
  double best = 0.0;
  p->M = 1;
  for (int m = 1; m <= 16 && m <= per_seq && m <= ctas; ++m) {
    const int64_t groups = (per_seq + m - 1) / m, gangs = ctas / m;
    double cost = (double)ctas / (double)(gangs * m) * (1.0 + 0.12 / (m * m));
    if (groups * n_seqs * kv_heads < 8 * gangs) cost *= (double)(groups * m) / (double)per_seq;
    if (m == 1 || cost < best) {
      best = cost;
      p->M = m;
    }
  }
  p->ctas = ctas / p->M * p->M;
  p->gangs = ctas / p->M;
  p->split = tiles > 2 * kSnap + 1;                  // else every end moves to a unit's
  p->part_rows = (int)(n_rows < R ? n_rows : R) * G;
  p->part_slots = p->mode != AW_ROWS && n_rows > R ? 4 : 2;
  p->ctrl_bytes = attn_win_ctrl_bytes(p->ctas);
  p->part_elems = (size_t)p->ctas * p->part_slots * p->part_rows * kPartRow;
  return true;
}

template <int MODE>
static cudaError_t launch_mode(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV, const AttnWinArgs& a,
                               const AwRuns<MODE>& runs, int ctas, cudaStream_t stream) {
  const auto kernel = attention_window_kernel<MODE>;
  constexpr int smem = AwPlan<MODE>::smem;
  static_assert(tmem_footprint_exclusive(smem), "an attention CTA must hold its SM's TMEM alone");
  if (!tmem_exclusive(smem)) return cudaErrorNotSupported;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kernel, dim3((unsigned)ctas), dim3(AW_THREADS), (size_t)smem, stream, tmQ, tmK, tmV, a, runs);
}

cudaError_t launch_attention_window(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                    const CUtensorMap* tmO, const AttnWinArgs& a, const AttnWinPlan& p, cudaStream_t stream) {
  if (p.split) {
    const int words = p.ctas * kCtrl;
    const cudaError_t e = launch_kernel(attention_window_start_kernel, dim3((unsigned)((words + 255) / 256)), dim3(256), 0,
                                        stream, a.ctrl, words);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e;
  if (p.mode == AW_DOC) {
    AwRuns<AW_DOC> runs;
    aw_doc_runs(a, p, &runs);
    runs.o = *tmO;
    e = launch_mode<AW_DOC>(tmQ, tmK, tmV, a, runs, p.ctas, stream);
  } else if (p.mode == AW_CHUNK) {
    e = launch_mode<AW_CHUNK>(tmQ, tmK, tmV, a, {}, p.ctas, stream);
  } else {
    e = launch_mode<AW_ROWS>(tmQ, tmK, tmV, a, {}, p.ctas, stream);
  }
  if (e != cudaSuccess) return e;
  set_kernel_info("attention_window_kernel<%s> tcgen05.mma.cta_group::1.kind::f16 unit=%d rows kv_tile=128 shared=%d "
                  "acc=f32 P-in-TMEM lazy-rescale=%g grid=%d gang=%d%s",
                  p.mode == AW_DOC ? "document" : (p.mode == AW_CHUNK ? "cache, chunks" : "cache, rows"), a.U, a.G,
                  (double)kLazyRescale, p.ctas, a.M, p.split ? " split" : "");
  return cudaGetLastError();
}

}  // namespace h3
