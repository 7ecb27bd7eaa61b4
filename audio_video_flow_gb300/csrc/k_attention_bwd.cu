// Gradient of the full non-causal attention of one packed document (128-wide
// heads, no mask), with the probabilities recomputed from the forward pass's
// log-sum-exp, on the 5th-generation tensor cores.  With
//   P = exp(q k^T / sqrt(128) - lse),  D = rowsum(dO o O),
//   dS = P o (dO V^T - D):
//   dV = P^T dO,   dK = dS^T Q / sqrt(128),   dQ = dS K / sqrt(128).
//
// Every output element is one fixed chain of MMAs over the row tiles in order,
// without atomics: dK and dV are computed by CTAs that own 128 key rows of a
// head and stream the query tiles, dQ by CTAs that own 128 query rows and
// stream the key tiles.  The probabilities are recomputed on both sides, so
// the tensor cores do 7 products of 128 x 128 x 128 per tile pair where the
// gradient alone needs 5; the alternative, adding dQ from the key side, would
// either depend on the order of atomics or serialise the key tiles.
//
// Both sides are one program.  With (F1, F2) the owned tiles and (G1, G2) the
// streamed ones, (K, V) and (Q, dO) on the key side or (Q, dO) and (K, V) on
// the query side, a step computes
//   S = F1 G1^T,  dP = F2 G2^T,  A1 += dS G1,  and on the key side A2 += P G2
// (S and dP are transposed there: rows are keys, columns queries).
//   warp 0       TMA producer: F1, F2 once, then G1 and G2 tiles into rings of
//                three and two stages;
//   warp 1       MMA issuer; G1 and G2 are read K-major for S and dP and
//                MN-major for A1 and A2 from the same tile;
//   warp 2       on the key side, the query rows' log-sum-exp and D (where few
//                CTAs run, the softmax warps compute them instead);
//   warps 4-19   softmax: warpgroup w takes columns [32 w, 32 w + 32), one row
//                per thread: P from S, then dS from dP and the P still in
//                registers, both to TMEM as bf16, where they are left operands.
// P and dS are rounded to bf16 for their products, as the forward kernel's P
// is: tf32 operands have half the rate and twice the bytes.  Each result so
// carries the error of one such rounding (2^-8 of each term, independent ones)
// beside that of its own; statistics, dS before the rounding and the
// accumulators are fp32.  Nothing else is lost: against the formulas in 64 bits
// with those two roundings put in, 99.2 % (4099 rows) to 99.9 % (72 rows) of the
// results have the same bits.
// On the key side each warp hands P and dS over in two halves of its columns,
// so that the products that read them begin while the second half is computed
// (8192 rows x 56 heads, that side alone: 1994 -> 1946 us).
// TMEM: S [0,128), dP [128,256), A1 [256,384); on the key side A2 [384,512), P
// over S and dS over dP; on the query side Q [384,448) as the left operand of S
// and dS [448,512), so that the next S and dP can be computed as soon as the
// softmax holds this step's (4096 rows x 56 heads, that side alone: 446 us;
// without the early dP 460, with Q from shared memory 466).
//
// Bound by the tensor pipe: 83 % active at 4096 rows x 16 heads; 3.43 ms at 8192
// rows x 56 heads is 1.40 PFLOP/s of the gradient's five products and 1.96 of
// the seven computed, the rate of a large cuBLAS product.  At 15,860 rows a
// single call takes 12.5 ms, repeated ones 14.5 at the 1.4 kW power limit.  The
// rest is each CTA's start and end (about 4 us, 10 % at 4096 rows, half at 505).
// Tried and slower: G tiles multicast to a pair of CTAs (3.69 ms at 8192 rows:
// the two then wait for each other), persistent CTAs (3.6 to 3.8), 8 softmax
// warps of 64 columns (the same).
#include "attention_device.cuh"
#include "h3_internal.h"

#include <algorithm>
#include <cmath>

namespace h3 {

namespace {
constexpr int AB_WARPS = 16;                 // softmax warps: 4 per 32 columns of a tile
constexpr int AB_THREADS = 32 * (4 + AB_WARPS);
constexpr int AB_ST1 = 3, AB_ST2 = 2;        // stages of the G1 and G2 rings
constexpr int AB_TILE = 128 * 128 * 2;       // 32 KB: two 64-channel boxes of 16 KB
constexpr int AB_BOX = 128 * 64 * 2;
constexpr int AB_ROWVALS = 2 * 128 * 4;      // a tile's log-sum-exp (base 2) and D
constexpr uint32_t TM_S = 0, TM_DP = 128, TM_A1 = 256, TM_A2 = 384, TM_Q = 384, TM_DS = 448;   // TMEM columns
constexpr int AB_SMEM = AB_TILE * (2 + AB_ST1 + AB_ST2) + 2 * AB_ROWVALS + 256;

// Eight packed columns to TMEM, then this warp's arrival at the barrier that the
// MMA warp waits on.
__device__ __forceinline__ void ab_hand_over(uint32_t taddr, const uint32_t* r, uint64_t* bar, int lane) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
  tmem_st_wait();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void ab_bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Sum over 128 channels of a product: 16 lanes with 8 channels each.
__device__ __forceinline__ float ab_row_dot(const uint4& x, const uint4& y) {
  const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    s = __fmaf_rn(bf16_lo(xw[e]), bf16_lo(yw[e]), s);
    s = __fmaf_rn(bf16_hi(xw[e]), bf16_hi(yw[e]), s);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
}  // namespace

// ---------------------------------------------------------------------------
// Row values: for each head and 128-row tile, 128 log-sum-exps in base 2
// followed by 128 sums D = sum_c dO[c] O[c] (fp32).  Rows past the end get
// +inf and 0, so their probabilities and dS are 0.  Bound by reading o and dO
// (4 us of a call at 505 rows x 56 heads).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) attention_bwd_rows_kernel(const AttnBwdArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int tile = blockIdx.x, head = blockIdx.y;
  const int sub = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  uint4 ov[8], dv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = tile * 128 + i * 16 + r0;
    ov[i] = dv[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row < a.S) {
      const size_t off = ((size_t)row * a.H + head) * 128 + sub * 8;
      if (in_bounds<__nv_bfloat16>(a.o, a.o_elems, a.o + off, 8, a.err, 40))
        ov[i] = *reinterpret_cast<const uint4*>(a.o + off);
      if (in_bounds<__nv_bfloat16>(a.d_o, a.o_elems, a.d_o + off, 8, a.err, 41))
        dv[i] = *reinterpret_cast<const uint4*>(a.d_o + off);
    }
  }
  float* out = a.rowvals + ((size_t)head * a.tiles + tile) * 256;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = ab_row_dot(ov[i], dv[i]);
    if (sub == 0) {
      const int r = i * 16 + r0, row = tile * 128 + r;
      float l2 = INFINITY;
      if (row < a.S && in_bounds<float>(a.lse, a.lse_elems, a.lse + (size_t)head * a.S + row, 1, a.err, 42))
        l2 = a.lse[(size_t)head * a.S + row] * 1.44269504088896340736f;
      if (in_bounds<float>(a.rowvals, a.rowval_elems, out + r, 129, a.err, 43)) {
        out[r] = l2;
        out[128 + r] = s;
      }
    }
  }
}

namespace {
// Places for pieces of split key tiles, per KV head.
__host__ __device__ inline int ab_part_slots(const AttnBwdArgs& a) {
  return (a.first_pieces > 1 ? a.first_tiles * a.first_pieces : 0) +
         (a.other_pieces > 1 ? (a.tiles - a.first_tiles) * a.other_pieces : 0);
}

struct AbSmem {
  uint8_t *f1, *f2, *g1, *g2, *rowvals;
  uint64_t *f1_full, *f2_full, *g1_full, *g1_empty, *g2_full, *g2_empty, *rv_full, *rv_empty;
  uint64_t *s_full, *s_empty, *p_full, *dp_full, *dp_empty, *ds_full, *ds_empty, *f_full, *acc_full, *drain;
};

// Rows [row0, row0 + 32) of one warp, NC columns of an accumulator, scaled and
// rounded to bf16: staged in shared memory (16-byte unit u of a row at unit
// u ^ (row & 7)), then written as whole lines.
template <int NC>
__device__ __forceinline__ void ab_store(uint32_t taddr, float scale, uint8_t* stg, int lane, int row0, int S,
                                         __nv_bfloat16* out, int64_t row_stride, const __nv_bfloat16* base,
                                         size_t elems, uint32_t* err) {
  constexpr int U = NC / 8;
  uint32_t all[NC / 32][32];
#pragma unroll
  for (int c = 0; c < NC / 32; ++c) tmem_ld32(taddr + (uint32_t)(c * 32), all[c]);
#pragma unroll
  for (int c = 0; c < NC / 32; ++c) {
    uint32_t(&o)[32] = all[c];
    tmem_ld_wait(o);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int u = c * 4 + g;
      *reinterpret_cast<uint4*>(stg + lane * (U * 16) + ((u ^ (lane & (U < 8 ? U - 1 : 7))) << 4)) =
          make_uint4(pack_bf16x2(__uint_as_float(o[g * 8 + 0]) * scale, __uint_as_float(o[g * 8 + 1]) * scale),
                     pack_bf16x2(__uint_as_float(o[g * 8 + 2]) * scale, __uint_as_float(o[g * 8 + 3]) * scale),
                     pack_bf16x2(__uint_as_float(o[g * 8 + 4]) * scale, __uint_as_float(o[g * 8 + 5]) * scale),
                     pack_bf16x2(__uint_as_float(o[g * 8 + 6]) * scale, __uint_as_float(o[g * 8 + 7]) * scale));
    }
  }
  __syncwarp();
#pragma unroll
  for (int it = 0; it < U; ++it) {
    const int r = it * (32 / U) + lane / U, u = lane % U;
    __nv_bfloat16* p = out + (int64_t)(row0 + r) * row_stride + u * 8;
    if (row0 + r < S && in_bounds<__nv_bfloat16>(base, elems, p, 8, err, 44))
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(stg + r * (U * 16) + ((u ^ (r & (U < 8 ? U - 1 : 7))) << 4));
  }
}

// The same rows and columns as they are, one row per lane.
template <int NC>
__device__ __forceinline__ void ab_store_part(uint32_t taddr, float* to, const AttnBwdArgs& a) {
#pragma unroll
  for (int c = 0; c < NC; c += 32) {
    uint32_t o[32];
    tmem_ld32(taddr + (uint32_t)c, o);
    tmem_ld_wait(o);
    if (in_bounds<float>(a.part, a.part_elems, to + (c + 31) * 128, 1, a.err, 46)) {
#pragma unroll
      for (int e = 0; e < 32; ++e) to[(c + e) * 128] = __uint_as_float(o[e]);
    }
  }
}

// The row values of tile t into slot `slot` of shared memory, by the softmax
// warps themselves (the same sums as attention_bwd_rows_kernel's).
__device__ __forceinline__ void ab_own_rows(const AttnBwdArgs& a, const AbSmem& sm, int t, int slot, int head) {
  const int tid = threadIdx.x - 128, sub = tid & 15, r0 = tid >> 4;
  constexpr int kStep = AB_WARPS * 2;            // rows at once
  float* out = reinterpret_cast<float*>(sm.rowvals + slot * AB_ROWVALS);
  uint4 ov[128 / kStep], dv[128 / kStep];
  float l2[128 / kStep];
#pragma unroll
  for (int i = 0; i < 128 / kStep; ++i) {
    const int row = t * 128 + i * kStep + r0;
    ov[i] = dv[i] = make_uint4(0u, 0u, 0u, 0u);
    l2[i] = INFINITY;
    if (row < a.S) {
      const size_t off = ((size_t)row * a.H + head) * 128 + sub * 8;
      if (in_bounds<__nv_bfloat16>(a.o, a.o_elems, a.o + off, 8, a.err, 40))
        ov[i] = *reinterpret_cast<const uint4*>(a.o + off);
      if (in_bounds<__nv_bfloat16>(a.d_o, a.o_elems, a.d_o + off, 8, a.err, 41))
        dv[i] = *reinterpret_cast<const uint4*>(a.d_o + off);
      if (sub == 0 && in_bounds<float>(a.lse, a.lse_elems, a.lse + (size_t)head * a.S + row, 1, a.err, 42))
        l2[i] = a.lse[(size_t)head * a.S + row] * 1.44269504088896340736f;
    }
  }
#pragma unroll
  for (int i = 0; i < 128 / kStep; ++i) {
    const float s = ab_row_dot(ov[i], dv[i]);
    if (sub == 0) {
      out[i * kStep + r0] = l2[i];
      out[128 + i * kStep + r0] = s;
    }
  }
}

// The streamed tiles of a CTA's steps.  Without a window all tiles of its head,
// in order.  With one, the key side takes the query tiles [lo, lo + per) that see
// its keys, of each head that shares them (or piece `piece` of `pieces` of these
// steps); the query side the first `sink` key tiles, then those from lo on.
template <bool KEYS, bool WIN>
struct AbSteps {
  int n, lo, per, sink, head0, from;
  __device__ __forceinline__ AbSteps(const AttnBwdArgs& a, int tile, int head, int piece, int pieces) {
    n = a.tiles;
    lo = sink = from = 0;
    per = n;
    head0 = head;
    if (!WIN) return;
    const int first = tile * 128, last = min(first + 128, a.S) - 1;
    if (KEYS) {
      lo = win_row_lo(a.w, first, a.S) >> 7;
      per = ((max(win_row_hi(a.w, first, a.S), win_row_hi(a.w, last, a.S)) + 127) >> 7) - lo;
      head0 = head * a.G;
      n = per * a.G;
      from = (int)((int64_t)n * piece / pieces);
      n = (int)((int64_t)n * (piece + 1) / pieces) - from;
    } else {
      lo = win_lo(a.w, first, a.S) >> 7;
      sink = min((min(a.w.first, win_lo(a.w, last, a.S)) + 127) >> 7, lo);
      n = sink + ((win_hi(a.w, last, a.S) + 127) >> 7) - lo;
      head0 = head / a.G;
    }
  }
  __device__ __forceinline__ int tile(int j) const {
    if (!WIN) return j;
    if (KEYS) return lo + (from + j) % per;
    return j < sink ? j : lo + j - sink;
  }
  __device__ __forceinline__ int head(int j) const { return WIN && KEYS ? head0 + (from + j) / per : head0; }
};

// One CTA's work: KEYS = true computes dK and dV of key tile `tile` of (KV) head
// `head`, false dQ of query tile `tile`.  OWN = true: at most two tiles, and the
// CTA computes their row values itself.  WIN = true: with a window and, where
// query heads share a KV head, over all of them on the key side.
template <bool KEYS, bool OWN, bool WIN>
__device__ __forceinline__ void ab_tile(const CUtensorMap* tmF1, const CUtensorMap* tmF2, const CUtensorMap* tmG1,
                                        const CUtensorMap* tmG2, const AttnBwdArgs& a, const AbSmem& sm,
                                        uint32_t tmem_base, int tile, int head, const WaitCtl& ctl, int piece = 0,
                                        int pieces = 1, int slot = 0) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AbSteps<KEYS, WIN> steps(a, tile, head, piece, pieces);
  const int n = steps.n;
  if (WIN && KEYS && n == 0) {   // a tile of fewer steps than pieces: this one adds nothing
    float* to = a.part + (int64_t)slot * 2 * 128 * 128;
    if (in_bounds<float>(a.part, a.part_elems, to, 2 * 128 * 128, a.err, 46))
      for (int i = threadIdx.x; i < 2 * 128 * 128; i += AB_THREADS) to[i] = 0.0f;
    return;
  }
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      bool ok = true;
      int i1 = 0, i2 = 0;
      auto load = [&](uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, int h, int t) {
        tma_load_3d(dst, tm, bar, 0, h, t * 128);
        tma_load_3d(dst + AB_BOX, tm, bar, 64, h, t * 128);
      };
      mbar_arrive_expect_tx(sm.f1_full, AB_TILE);
      load(sm.f1, tmF1, sm.f1_full, head, tile);
      for (int j = 0; j < n && ok; ++j) {
        const int s1 = j % AB_ST1, s2 = j % AB_ST2;
        if (!mbar_wait(&sm.g1_empty[s1], ((uint32_t)(j / AB_ST1) & 1u) ^ 1u, ctl)) { ok = false; break; }
        mbar_arrive_expect_tx(&sm.g1_full[s1], AB_TILE);
        load(sm.g1 + s1 * AB_TILE, tmG1, &sm.g1_full[s1], steps.head(j), steps.tile(j));
        ++i1;
        if (j == 0) {
          mbar_arrive_expect_tx(sm.f2_full, AB_TILE);
          load(sm.f2, tmF2, sm.f2_full, head, tile);
        }
        if (!mbar_wait(&sm.g2_empty[s2], ((uint32_t)(j / AB_ST2) & 1u) ^ 1u, ctl)) { ok = false; break; }
        mbar_arrive_expect_tx(&sm.g2_full[s2], AB_TILE);
        load(sm.g2 + s2 * AB_TILE, tmG2, &sm.g2_full[s2], steps.head(j), steps.tile(j));
        ++i2;
      }
      if (!ok) {  // let issued loads land before the CTA exits
        at_drain(sm.f1_full, 0);
        if (i1 > 0) at_drain(sm.f2_full, 0);
        for (int j = (i1 > AB_ST1 ? i1 - AB_ST1 : 0); j < i1; ++j)
          at_drain(&sm.g1_full[j % AB_ST1], (uint32_t)(j / AB_ST1) & 1u);
        for (int j = (i2 > AB_ST2 ? i2 - AB_ST2 : 0); j < i2; ++j)
          at_drain(&sm.g2_full[j % AB_ST2], (uint32_t)(j / AB_ST2) & 1u);
      }
    }
    __syncwarp();
  } else if (KEYS && !OWN && warp == 2) {
    // ------------------------------------------------------------ producer of the query rows' values
    if (lane == 0) {
      int i = 0;
      bool ok = true;
      for (int j = 0; j < n; ++j) {
        if (!mbar_wait(&sm.rv_empty[j & 1], ((uint32_t)(j >> 1) & 1u) ^ 1u, ctl)) { ok = false; break; }
        mbar_arrive_expect_tx(&sm.rv_full[j & 1], AB_ROWVALS);
        ab_bulk_load(sm.rowvals + (j & 1) * AB_ROWVALS, a.rowvals + ((size_t)steps.head(j) * a.tiles + steps.tile(j)) * 256, AB_ROWVALS,
                     &sm.rv_full[j & 1]);
        ++i;
      }
      if (!ok)
        for (int j = (i > 2 ? i - 2 : 0); j < i; ++j) at_drain(&sm.rv_full[j & 1], (uint32_t)(j >> 1) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = idesc_bf16(128, 128, false, false);
    constexpr uint32_t idesc_a = idesc_bf16(128, 128, false, true);   // G1, G2 MN-major
    constexpr uint64_t kTile = AB_TILE >> 4, kBox = AB_BOX >> 4;      // descriptor address steps
    const uint32_t one = at_elect();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem_base, 0);
    const uint64_t f1 = sdesc_kmajor(smem_u32(sm.f1)), f2 = sdesc_kmajor(smem_u32(sm.f2));
    const uint64_t g1k = sdesc_kmajor(smem_u32(sm.g1)), g2k = sdesc_kmajor(smem_u32(sm.g2));
    const uint64_t g1m = sdesc_sw128(smem_u32(sm.g1), AB_BOX, 1024), g2m = sdesc_sw128(smem_u32(sm.g2), AB_BOX, 1024);
    auto issue_ss = [&](uint32_t d, uint64_t f, uint64_t g) {   // F G^T: two 64-channel boxes
      at_mma4_ss<2, 2>(tm + d, f, g, idesc_s, 0u, one);
      at_mma4_ss<2, 2>(tm + d, f + kBox, g + kBox, idesc_s, 1u, one);
    };
    auto issue_q = [&](uint32_t d, uint64_t g) {                // Q in TMEM times G^T
      at_mma4_ts<8, 2>(tm + d, tm + TM_Q, g, idesc_s, 0u, one);
      at_mma4_ts<8, 2>(tm + d, tm + TM_Q + 32u, g + kBox, idesc_s, 1u, one);
    };
    // accumulator += A G, A bf16 in TMEM.  Key side, half h: the first or
    // second 16 of each warpgroup's 32 columns, 8 packed ones at 32 w + 8 h.
    auto issue_half = [&](uint32_t d, uint32_t s, uint64_t g, int h, uint32_t accumulate) {
      at_mma4_ts<32, 256>(tm + d, tm + s + (uint32_t)(8 * h), g + (uint64_t)(128 * h), idesc_a, accumulate, one);
    };
    auto issue_ds = [&](uint64_t g, uint32_t accumulate) {      // query side: 64 packed columns in a row
      at_mma4_ts<8, 128>(tm + TM_A1, tm + TM_DS, g, idesc_a, accumulate, one);
      at_mma4_ts<8, 128>(tm + TM_A1, tm + TM_DS + 32u, g + 512u, idesc_a, 1u, one);
    };
    // S and dP of the next tile: stages and phases of the rings go round here
    uint32_t s1 = 0, p1 = 0, s2 = 0, p2 = 0;   // the next tile's stage and phase in each ring
    auto issue_s = [&]() -> bool {
      if (!at_wait(&sm.g1_full[s1], p1, ctl)) return false;
      tc_fence_after();
      if (KEYS) issue_ss(TM_S, f1, g1k + s1 * kTile);
      else issue_q(TM_S, g1k + s1 * kTile);
      at_commit(sm.s_full, one);
      if (++s1 == AB_ST1) { s1 = 0; p1 ^= 1u; }
      return true;
    };
    auto issue_dp = [&]() -> bool {
      if (!at_wait(&sm.g2_full[s2], p2, ctl)) return false;
      tc_fence_after();
      issue_ss(TM_DP, f2, g2k + s2 * kTile);
      if (!KEYS) at_commit(&sm.g2_empty[s2], one);
      at_commit(sm.dp_full, one);
      if (++s2 == AB_ST2) { s2 = 0; p2 ^= 1u; }
      return true;
    };
    bool ok = at_wait(KEYS ? sm.f1_full : sm.f_full, 0, ctl);
    if (ok) ok = issue_s() && at_wait(sm.f2_full, 0, ctl) && issue_dp();
    uint32_t c1 = 0, c2 = 0;                   // this tile's stages
    for (int j = 0; j < n && ok; ++j) {
      const bool more = j + 1 < n;
      const uint32_t ph = (uint32_t)j & 1u, accumulate = j != 0 ? 1u : 0u;
      if (KEYS) {
        // A2 += P G2 in the halves that the softmax hands over, then the next
        // S over P
        if (!at_wait(&sm.p_full[0], ph, ctl)) { ok = false; break; }
        tc_fence_after();
        issue_half(TM_A2, TM_S, g2m + c2 * kTile, 0, accumulate);
        if (!at_wait(&sm.p_full[1], ph, ctl)) { ok = false; break; }
        tc_fence_after();
        issue_half(TM_A2, TM_S, g2m + c2 * kTile, 1, 1u);
        at_commit(&sm.g2_empty[c2], one);
        if (more && !issue_s()) { ok = false; break; }
      } else if (more) {
        // S (and dP) of the next tile as soon as the softmax holds this one's
        if (!at_wait(sm.s_empty, ph, ctl) || !issue_s()) { ok = false; break; }
        if (!at_wait(sm.dp_empty, ph, ctl) || !issue_dp()) { ok = false; break; }
      }
      if (!at_wait(&sm.ds_full[0], ph, ctl)) { ok = false; break; }
      tc_fence_after();
      if (KEYS) {
        issue_half(TM_A1, TM_DP, g1m + c1 * kTile, 0, accumulate);
        if (!at_wait(&sm.ds_full[1], ph, ctl)) { ok = false; break; }
        tc_fence_after();
        issue_half(TM_A1, TM_DP, g1m + c1 * kTile, 1, 1u);
      } else {
        issue_ds(g1m + c1 * kTile, accumulate);
      }
      at_commit(&sm.g1_empty[c1], one);
      if (!KEYS) at_commit(sm.ds_empty, one);
      if (KEYS && more && !issue_dp()) { ok = false; break; }
      if (!more) at_commit(sm.acc_full, one);
      if (++c1 == AB_ST1) c1 = 0;
      if (++c2 == AB_ST2) c2 = 0;
    }
    if (!ok) {
      at_commit(sm.drain, one);
      if (one) at_drain(sm.drain, 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    const int wg = (warp - 4) >> 2;
    const int qq = warp & 3;
    const int row = qq * 32 + lane;
    const uint32_t s_base = tmem_addr(tmem_base, (uint32_t)(qq * 32), TM_S + (uint32_t)(wg * 32));
    const uint32_t dp_base = tmem_addr(tmem_base, (uint32_t)(qq * 32), TM_DP + (uint32_t)(wg * 32));
    // where the packed dS goes: over the thread's own dP on the key side
    const uint32_t ds_base =
        KEYS ? dp_base : tmem_addr(tmem_base, (uint32_t)(qq * 32), TM_DS + (uint32_t)(wg * 16));
    const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
    float my_l2 = 0.0f, my_d = 0.0f;
    bool ok = true;
    if (OWN) {   // every softmax warp comes here, before any wait that can run out
      for (int t = KEYS ? 0 : tile; t < (KEYS ? n : tile + 1); ++t) ab_own_rows(a, sm, t, KEYS ? t : 0, head);
      asm volatile("bar.sync 1, %0;" ::"n"(32 * AB_WARPS) : "memory");
    }
    if (!KEYS) {
      const float* rv = a.rowvals + ((size_t)head * a.tiles + tile) * 256 + row;
      if (OWN) {
        my_l2 = reinterpret_cast<const float*>(sm.rowvals)[row];
        my_d = reinterpret_cast<const float*>(sm.rowvals)[128 + row];
      } else if (in_bounds<float>(a.rowvals, a.rowval_elems, rv, 129, a.err, 45)) {
        my_l2 = rv[0];
        my_d = rv[128];
      }
      // Q from its tile into TMEM, where it is the left operand of every S:
      // warpgroup w takes channels [32 w, 32 w + 32) of the row
      ok = at_wait(sm.f1_full, 0, ctl);
      if (ok) {
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(
              sm.f1 + (wg >> 1) * AB_BOX + sw128_offset((uint32_t)row, (uint32_t)((wg & 1) * 4 + c)));
          pk[4 * c] = v.x;
          pk[4 * c + 1] = v.y;
          pk[4 * c + 2] = v.z;
          pk[4 * c + 3] = v.w;
        }
        at_tmem_st16(tmem_addr(tmem_base, (uint32_t)(qq * 32), TM_Q + (uint32_t)(wg * 16)), pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.f_full);
      }
    }
    // what this thread's key (or query) sees: [see_lo, see_hi) and [0, see_first)
    int see_lo = 0, see_hi = 0, see_first = 0;
    if (WIN) {
      const int at = min(tile * 128 + row, a.S - 1);
      see_lo = KEYS ? win_row_lo(a.w, at, a.S) : win_lo(a.w, at, a.S);
      see_hi = KEYS ? win_row_hi(a.w, at, a.S) : win_hi(a.w, at, a.S);
      if (!KEYS) see_first = min(a.w.first, see_hi);
    }
    int at_tile = steps.tile(0);   // the tile of step j, without a division each
    for (int j = 0; j < n && ok; ++j) {
      const uint32_t ph = (uint32_t)j & 1u;
      const float* rv = reinterpret_cast<const float*>(sm.rowvals + (j & 1) * AB_ROWVALS) + wg * 32;
      if (KEYS && !OWN && !at_wait(&sm.rv_full[j & 1], (uint32_t)(j >> 1) & 1u, ctl)) { ok = false; break; }
      if (!at_wait(sm.s_full, ph, ctl)) { ok = false; break; }
      tc_fence_after();
      uint32_t p[32], pk[16];
      tmem_ld32(s_base, p);
      tmem_ld_wait(p);
      if (WIN) {
        const int c0 = at_tile * 128 + wg * 32;
        const uint32_t see = (win_bits(see_hi - c0) & ~win_bits(see_lo - c0)) | win_bits(see_first - c0);
        if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!((see >> c) & 1u)) p[c] = __float_as_uint(-INFINITY);
        }
        ++at_tile;
        if (KEYS) {
          if (at_tile == steps.lo + steps.per) at_tile = steps.lo;
        } else if (j + 1 == steps.sink) {
          at_tile = steps.lo;
        }
      }
      if (!KEYS) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.s_empty);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 16 * h; c < 16 * h + 16; c += 4) {
          const float4 l =
              KEYS ? *reinterpret_cast<const float4*>(rv + c) : make_float4(my_l2, my_l2, my_l2, my_l2);
          const float2 z0 = __ffma2_rn(make_float2(__uint_as_float(p[c]), __uint_as_float(p[c + 1])), sl2,
                                       make_float2(-l.x, -l.y));
          const float2 z1 = __ffma2_rn(make_float2(__uint_as_float(p[c + 2]), __uint_as_float(p[c + 3])), sl2,
                                       make_float2(-l.z, -l.w));
          const float e0 = at_ex2(z0.x), e1 = at_ex2(z0.y), e2 = at_ex2(z1.x), e3 = at_ex2(z1.y);
          p[c] = __float_as_uint(e0);
          p[c + 1] = __float_as_uint(e1);
          p[c + 2] = __float_as_uint(e2);
          p[c + 3] = __float_as_uint(e3);
          if (KEYS) {
            pk[c >> 1] = pack_bf16x2(e0, e1);
            pk[(c >> 1) + 1] = pack_bf16x2(e2, e3);
          }
        }
        if (KEYS) ab_hand_over(s_base + (uint32_t)(8 * h), &pk[8 * h], &sm.p_full[h], lane);
      }
      if (!KEYS && !WIN && j == n - 1) {
        // keys past the end: their K rows are zero, but exp(-lse) times 0
        // must not become NaN where lse is far below 0
        const int valid = a.S - j * 128 - wg * 32;
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c >= valid) p[c] = 0u;
      }
      if (!at_wait(sm.dp_full, ph, ctl)) { ok = false; break; }
      tc_fence_after();
      uint32_t d[32];
      tmem_ld32(dp_base, d);
      tmem_ld_wait(d);
      if (!KEYS) {   // the next dP may follow
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.dp_empty);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 16 * h; c < 16 * h + 16; c += 4) {
          const float4 dd =
              KEYS ? *reinterpret_cast<const float4*>(rv + 128 + c) : make_float4(my_d, my_d, my_d, my_d);
          const float2 t0 = __fadd2_rn(make_float2(__uint_as_float(d[c]), __uint_as_float(d[c + 1])),
                                       make_float2(-dd.x, -dd.y));
          const float2 t1 = __fadd2_rn(make_float2(__uint_as_float(d[c + 2]), __uint_as_float(d[c + 3])),
                                       make_float2(-dd.z, -dd.w));
          const float2 u0 = __fmul2_rn(t0, make_float2(__uint_as_float(p[c]), __uint_as_float(p[c + 1])));
          const float2 u1 = __fmul2_rn(t1, make_float2(__uint_as_float(p[c + 2]), __uint_as_float(p[c + 3])));
          pk[c >> 1] = pack_bf16x2(u0.x, u0.y);
          pk[(c >> 1) + 1] = pack_bf16x2(u1.x, u1.y);
        }
        if (KEYS) ab_hand_over(ds_base + (uint32_t)(8 * h), &pk[8 * h], &sm.ds_full[h], lane);
      }
      if (KEYS) {
        if (lane == 0) mbar_arrive(&sm.rv_empty[j & 1]);
      } else {   // once the previous dS has been read
        if (!at_wait(sm.ds_empty, ph ^ 1u, ctl)) { ok = false; break; }
        tc_fence_after();
        at_tmem_st16(ds_base, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ds_full[0]);
      }
    }
    if (ok && at_wait(sm.acc_full, 0, ctl)) {
      tc_fence_after();
      // the accumulators leave through the G rings, idle now (acc_full covers
      // every MMA, and every load has been consumed by one)
      uint8_t* stg = sm.g1 + (warp - 4) * 4096;
      const int row0 = tile * 128 + qq * 32;
      const uint32_t acc = tmem_addr(tmem_base, (uint32_t)(qq * 32), TM_A1);
      const int64_t at_head = head * (KEYS ? a.dkv_head_stride : a.d_head_stride);
      if (KEYS) {
        const int half = (wg & 1) * 64;
        if (WIN && pieces > 1)   // one of several pieces: fp32, [channel][row], dV then dK
          ab_store_part<64>(acc + (wg < 2 ? TM_A2 - TM_A1 : 0u) + (uint32_t)half,
                            a.part + ((int64_t)slot * 2 + (wg < 2 ? 0 : 1)) * 128 * 128 + half * 128 + qq * 32 + lane, a);
        else if (wg < 2)
          ab_store<64>(acc + (TM_A2 - TM_A1) + (uint32_t)half, 1.0f, stg, lane, row0, a.S, a.dv + at_head + half,
                       a.dkv_row_stride, a.dv, a.dkv_elems, a.err);
        else
          ab_store<64>(acc + (uint32_t)half, a.scale, stg, lane, row0, a.S, a.dk + at_head + half, a.dkv_row_stride,
                       a.dk, a.dkv_elems, a.err);
      } else {
        ab_store<32>(acc + (uint32_t)(wg * 32), a.scale, stg, lane, row0, a.S, a.dq + at_head + wg * 32,
                     a.d_row_stride, a.dq, a.d_elems, a.err);
      }
    }
  }
}
}  // namespace

// blockIdx.x: 128-row tile, blockIdx.y: head; z = 0 the key side, z = 1 the
// query side (the longer key-side CTAs are scheduled first).  WIN: a line of
// CTAs, for each KV head the pieces of its key tiles (first_pieces for each of the
// first_tiles ones, which all rows may see, then other_pieces), then for each
// query head its tiles.
template <bool OWN, bool WIN>
__global__ void __launch_bounds__(AB_THREADS, 1)
    attention_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                         const AttnBwdArgs args) {
  // no static shared memory: the dynamic part starts at a multiple of 1024,
  // as the swizzled tiles need
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  AbSmem sm;
  sm.f1 = smem_raw;
  sm.f2 = sm.f1 + AB_TILE;
  sm.g1 = sm.f2 + AB_TILE;
  sm.g2 = sm.g1 + AB_ST1 * AB_TILE;
  sm.rowvals = sm.g2 + AB_ST2 * AB_TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm.rowvals + 2 * AB_ROWVALS);
  sm.f1_full = bars;
  sm.f2_full = bars + 1;
  sm.g1_full = bars + 2;
  sm.g1_empty = sm.g1_full + AB_ST1;
  sm.g2_full = sm.g1_empty + AB_ST1;
  sm.g2_empty = sm.g2_full + AB_ST2;
  sm.rv_full = sm.g2_empty + AB_ST2;
  sm.rv_empty = sm.rv_full + 2;
  sm.s_full = sm.rv_empty + 2;
  sm.s_empty = sm.s_full + 1;
  sm.p_full = sm.s_empty + 1;     // [2]
  sm.dp_full = sm.p_full + 2;
  sm.dp_empty = sm.dp_full + 1;
  sm.ds_full = sm.dp_empty + 1;   // [2]
  sm.ds_empty = sm.ds_full + 2;
  sm.f_full = sm.ds_empty + 1;
  sm.acc_full = sm.f_full + 1;
  sm.drain = sm.acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm.drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int skip = 0;
  if (threadIdx.x == 0) {
    mbar_init(sm.f1_full, 1);
    mbar_init(sm.f2_full, 1);
    for (int s = 0; s < AB_ST1; ++s) {
      mbar_init(&sm.g1_full[s], 1);
      mbar_init(&sm.g1_empty[s], 1);
    }
    for (int s = 0; s < AB_ST2; ++s) {
      mbar_init(&sm.g2_full[s], 1);
      mbar_init(&sm.g2_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.rv_full[s], 1);
      mbar_init(&sm.rv_empty[s], AB_WARPS);
    }
    mbar_init(sm.s_full, 1);
    mbar_init(sm.s_empty, AB_WARPS);
    mbar_init(sm.dp_full, 1);
    mbar_init(sm.dp_empty, AB_WARPS);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&sm.p_full[h], AB_WARPS);
      mbar_init(&sm.ds_full[h], AB_WARPS);
    }
    mbar_init(sm.ds_empty, 1);
    mbar_init(sm.f_full, AB_WARPS);
    mbar_init(sm.acc_full, 1);
    mbar_init(sm.drain, 1);
    skip = timeout_recorded(args.err) ? 1 : 0;   // sticky timeout of an earlier launch
    *abort_flag = skip;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmO);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  if (OWN) skip = __syncthreads_or(skip);   // one answer for all warps: they meet at a barrier in ab_tile
  else __syncthreads();
  tc_fence_after();
  griddep_wait();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl ctl{abort_flag, args.err, KID_ATTN_BWD};

  // a wait of an earlier launch ran out: this launch skips its work, before
  // any copy or MMA is issued
  if (OWN ? skip == 0 : *ctl.flag == 0) {
    if (!WIN) {
      if (blockIdx.z == 0)
        ab_tile<true, OWN, WIN>(&tmK, &tmV, &tmQ, &tmO, args, sm, tmem_base, blockIdx.x, blockIdx.y, ctl);
      else
        ab_tile<false, OWN, WIN>(&tmQ, &tmO, &tmK, &tmV, args, sm, tmem_base, blockIdx.x, blockIdx.y, ctl);
    } else {
      const int firsts = args.first_tiles * args.first_pieces;
      const int per_head = firsts + (args.tiles - args.first_tiles) * args.other_pieces;
      const int id = (int)blockIdx.x, key_ctas = args.H / args.G * per_head;
      if (id < key_ctas) {
        const int head = id / per_head, x = id - head * per_head;
        const bool first = x < firsts;
        const int pieces = first ? args.first_pieces : args.other_pieces, y = first ? x : x - firsts;
        const int tile = y / pieces + (first ? 0 : args.first_tiles);
        // a piece's place among those of split tiles
        const int slot = head * ab_part_slots(args) + (first || args.first_pieces == 1 ? y : firsts + y);
        ab_tile<true, OWN, WIN>(&tmK, &tmV, &tmQ, &tmO, args, sm, tmem_base, tile, head, ctl, y % pieces, pieces, slot);
      } else {
        const int y = id - key_ctas, head = y / args.tiles;
        ab_tile<false, OWN, WIN>(&tmQ, &tmO, &tmK, &tmV, args, sm, tmem_base, y - head * args.tiles, head, ctl);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *ctl.flag) record_error(args.err, DEVERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

cudaError_t launch_attention_bwd(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                 const CUtensorMap& tmO, const AttnBwdArgs& a, cudaStream_t stream) {
  static_assert(tmem_footprint_exclusive(AB_SMEM), "an attention CTA must hold its SM's TMEM alone");
  if (!tmem_exclusive(AB_SMEM)) return cudaErrorNotSupported;
  const dim3 rows_grid((unsigned)a.tiles, (unsigned)a.H), grid((unsigned)a.tiles, (unsigned)a.H, 2);
  // Up to two tiles and two CTAs per SM, every CTA computes its row values
  // itself beside its first loads: one launch instead of two (72 rows x 4
  // heads 9.4 -> 7.9 us, 128 x 152 18.1 -> 13.0, 256 x 56 16.6 -> 15.1).  With
  // more CTAs that work, which each then repeats before its first step, costs
  // more than the launch (256 x 600 136 -> 175 us, 100 x 600 59.5 -> 62.8).
  const bool own = a.tiles <= 2 && (int64_t)a.tiles * a.H <= num_sms();
  cudaError_t e = cudaSuccess;
  if (!own) e = launch_kernel(attention_bwd_rows_kernel, rows_grid, dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  const auto kernel = own ? attention_bwd_kernel<true, false> : attention_bwd_kernel<false, false>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, AB_SMEM);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kernel, grid, dim3(AB_THREADS), AB_SMEM, stream, tmQ, tmK, tmV, tmO, a);
  if (e != cudaSuccess) return e;
  set_kernel_info("attention_bwd_kernel tcgen05.mma.cta_group::1.kind::f16 tile=128x128 stages=%d,%d acc=f32 "
                  "P,dS-in-TMEM grid=%ux%ux2%s",
                  AB_ST1, AB_ST2, grid.x, grid.y, own ? " own-row-values" : "");
  return cudaGetLastError();
}

// dV and dK of the key tiles that several pieces computed: their sums, in order.
// Block: 32 rows of a split tile (x), KV head (y), dV or dK (z).
__global__ void __launch_bounds__(256) attention_bwd_join_kernel(const AttnBwdArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int x = blockIdx.x >> 2, lane = threadIdx.x & 31, row = (blockIdx.x & 3) * 32 + lane, ch = (threadIdx.x >> 5) * 16;
  const int firsts = a.first_pieces > 1 ? a.first_tiles : 0;    // split ones among the first tiles
  const bool first = x < firsts;
  const int tile = first ? x : x - firsts + a.first_tiles, pieces = first ? a.first_pieces : a.other_pieces;
  const int slot = blockIdx.y * ab_part_slots(a) + (first ? x * pieces : firsts * a.first_pieces + (x - firsts) * pieces);
  const float* from = a.part + ((int64_t)slot * 2 + blockIdx.z) * 128 * 128 + ch * 128 + row;
  float sum[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) sum[e] = 0.0f;
  for (int p = 0; p < pieces; ++p, from += 2 * 128 * 128) {
    if (!in_bounds<float>(a.part, a.part_elems, from + 15 * 128, 1, a.err, 47)) continue;
#pragma unroll
    for (int e = 0; e < 16; ++e) sum[e] += from[e * 128];
  }
  const int grow = tile * 128 + row;
  if (grow >= a.S) return;
  const float scale = blockIdx.z == 0 ? 1.0f : a.scale;
  __nv_bfloat16* base = blockIdx.z == 0 ? a.dv : a.dk;
  __nv_bfloat16* to = base + (int64_t)grow * a.dkv_row_stride + (int64_t)blockIdx.y * a.dkv_head_stride + ch;
  if (!in_bounds<__nv_bfloat16>(base, a.dkv_elems, to, 16, a.err, 48)) return;
#pragma unroll
  for (int e = 0; e < 16; e += 8)
    *reinterpret_cast<uint4*>(to + e) =
        make_uint4(pack_bf16x2(sum[e] * scale, sum[e + 1] * scale), pack_bf16x2(sum[e + 2] * scale, sum[e + 3] * scale),
                   pack_bf16x2(sum[e + 4] * scale, sum[e + 5] * scale), pack_bf16x2(sum[e + 6] * scale, sum[e + 7] * scale));
}

// How the key side is split.  Key tiles that all rows see (the first ones), or of
// heads that many share, take many more steps than a query tile; one of more steps
// than an SM's share of all the work (a key step counts 4 products, a query step
// 3) would run alone at the end, and is cut into pieces of half that share, at
// least kPieceSteps (4099 rows, 24 heads over 4, 640 keys and 3 first: one CTA of
// 198 steps, 281 us; in pieces 135 us).
constexpr int kPieceSteps = 16, kMaxPieces = 520;
void attn_bwd_split(AttnBwdArgs* a) {
  a->first_tiles = a->w.left < 0 ? 0 : (int)std::min<int64_t>(a->tiles, ((int64_t)a->w.first + 127) / 128);
  a->first_pieces = a->other_pieces = 1;
  int64_t steps = 0;
  int most[2] = {0, 0};
  for (int t = 0; t < a->tiles; ++t) {
    const int j0 = t * 128, j1 = std::min(j0 + 128, a->S) - 1;
    const int lo = win_row_lo(a->w, j0, a->S) >> 7;
    const int hi = std::max(win_row_hi(a->w, j0, a->S), win_row_hi(a->w, j1, a->S));
    const int n = (((hi + 127) >> 7) - lo) * a->G;
    steps += n;
    int& m = most[t < a->first_tiles ? 0 : 1];
    m = std::max(m, n);
  }
  const int heads = a->H / a->G;
  const int64_t share = steps * heads * 7 / 4 / num_sms();
  auto pieces = [&](int n) -> int {
    if (n <= share || n <= kPieceSteps) return 1;
    const int64_t each = std::max<int64_t>(kPieceSteps, share / 2);
    return (int)((n + each - 1) / each);
  };
  a->first_pieces = pieces(most[0]);
  a->other_pieces = pieces(most[1]);
  if ((int64_t)heads * ab_part_slots(*a) > kMaxPieces) a->other_pieces = 1;
  if ((int64_t)heads * ab_part_slots(*a) > kMaxPieces) a->first_pieces = 1;
  a->part_elems = (size_t)heads * ab_part_slots(*a) * 2 * 128 * 128;
}
// Bytes of pieces, for every window.
size_t attn_bwd_part_bytes(int64_t S, int64_t H, int64_t Hk) {
  const int64_t tiles = (S + 127) / 128, n = tiles * (H / Hk);
  if (n <= kPieceSteps) return 0;
  const int64_t most = std::min<int64_t>(kMaxPieces, Hk * tiles * ((n + kPieceSteps - 1) / kPieceSteps));
  return (size_t)most * 2 * 128 * 128 * 4;
}

cudaError_t launch_attention_window_bwd(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                        const CUtensorMap& tmO, const AttnBwdArgs& a, cudaStream_t stream) {
  if (!tmem_exclusive(AB_SMEM)) return cudaErrorNotSupported;
  const int heads = a.H / a.G;
  const int64_t key_ctas = (int64_t)heads * (a.first_tiles * a.first_pieces + (a.tiles - a.first_tiles) * a.other_pieces);
  const dim3 rows_grid((unsigned)a.tiles, (unsigned)a.H), grid((unsigned)(key_ctas + (int64_t)a.H * a.tiles));
  cudaError_t e = launch_kernel(attention_bwd_rows_kernel, rows_grid, dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  const auto kernel = attention_bwd_kernel<false, true>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, AB_SMEM);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kernel, grid, dim3(AB_THREADS), AB_SMEM, stream, tmQ, tmK, tmV, tmO, a);
  if (e != cudaSuccess) return e;
  const int split = (a.first_pieces > 1 ? a.first_tiles : 0) + (a.other_pieces > 1 ? a.tiles - a.first_tiles : 0);
  if (split > 0) {
    e = launch_kernel(attention_bwd_join_kernel, dim3((unsigned)(split * 4), (unsigned)heads, 2), dim3(256), 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  set_kernel_info("attention_bwd_kernel<window> tcgen05.mma.cta_group::1.kind::f16 tile=128x128 stages=%d,%d acc=f32 "
                  "P,dS-in-TMEM shared=%d grid=%u pieces=%d,%d",
                  AB_ST1, AB_ST2, a.G, grid.x, a.first_pieces, a.other_pieces);
  return cudaGetLastError();
}

}  // namespace h3
