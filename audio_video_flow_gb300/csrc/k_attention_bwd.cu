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
//   warp 0       TMA producer: F1, F2 once, then G1 and G2 tiles (and on the
//                key side their rows' log-sum-exp and D) into two-deep rings;
//   warp 1       MMA issuer (one thread); G1 and G2 are read K-major for S
//                and dP and MN-major for A1 and A2 from the same tile;
//   warps 4-11   softmax: warpgroup w takes columns [64 w, 64 w + 64), one
//                row per thread: P from S into bf16 over the thread's own S
//                columns, then dS from dP and the P still in registers.
// TMEM: S [0,128), dP [128,256), A1 [256,384), A2 [384,512).
#include "h3_device.cuh"
#include "h3_internal.h"

#include <cmath>

namespace h3 {

namespace {
constexpr int AB_THREADS = 384;
constexpr int AB_STAGES = 2;
constexpr int AB_TILE = 128 * 128 * 2;       // 32 KB: two 64-channel boxes of 16 KB
constexpr int AB_BOX = 128 * 64 * 2;
constexpr int AB_ROWVALS = 2 * 128 * 4;      // a tile's log-sum-exp (base 2) and D
constexpr int AB_SMEM = 1024 + AB_TILE * (2 + 2 * AB_STAGES) + AB_STAGES * AB_ROWVALS + 256;

__device__ __forceinline__ float ab_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ab_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void ab_tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void ab_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer() - t0 > kWaitLimitNs) return;
  }
}
__device__ __forceinline__ void ab_bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
}  // namespace

// ---------------------------------------------------------------------------
// Row values: for each head and 128-row tile, 128 log-sum-exps in base 2
// followed by 128 sums D = sum_c dO[c] O[c] (fp32).  Rows past the end get
// +inf and 0, so their probabilities and dS are 0.  Bound by reading o and dO.
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
    const uint32_t ow[4] = {ov[i].x, ov[i].y, ov[i].z, ov[i].w}, dw[4] = {dv[i].x, dv[i].y, dv[i].z, dv[i].w};
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = __fmaf_rn(bf16_lo(ow[e]), bf16_lo(dw[e]), s);
      s = __fmaf_rn(bf16_hi(ow[e]), bf16_hi(dw[e]), s);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
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
struct AbSmem {
  uint8_t *f1, *f2, *g1, *g2, *rowvals;
  uint64_t *f1_full, *f2_full, *g1_full, *g1_empty, *g2_full, *g2_empty;
  uint64_t *s_full, *p_full, *dp_full, *ds_full, *acc_full, *drain;
};

// Rows [row0, row0 + 32) of one warp, NC columns of an accumulator, scaled and
// rounded to bf16: staged in shared memory (16-byte unit u of a row at unit
// u ^ (row & 7)), then written as whole lines.
template <int NC>
__device__ __forceinline__ void ab_store(uint32_t taddr, float scale, uint8_t* stg, int lane, int row0, int S,
                                         __nv_bfloat16* out, int64_t row_stride, const __nv_bfloat16* base,
                                         size_t elems, uint32_t* err) {
  constexpr int U = NC / 8;
#pragma unroll 1
  for (int c = 0; c < NC / 32; ++c) {
    uint32_t o[32];
    tmem_ld32(taddr + (uint32_t)(c * 32), o);
    tmem_ld_wait(o);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int u = c * 4 + g;
      *reinterpret_cast<uint4*>(stg + lane * (U * 16) + ((u ^ (lane & 7)) << 4)) =
          make_uint4(pack_bf16x2(__uint_as_float(o[g * 8 + 0]) * scale, __uint_as_float(o[g * 8 + 1]) * scale),
                     pack_bf16x2(__uint_as_float(o[g * 8 + 2]) * scale, __uint_as_float(o[g * 8 + 3]) * scale),
                     pack_bf16x2(__uint_as_float(o[g * 8 + 4]) * scale, __uint_as_float(o[g * 8 + 5]) * scale),
                     pack_bf16x2(__uint_as_float(o[g * 8 + 6]) * scale, __uint_as_float(o[g * 8 + 7]) * scale));
    }
  }
  __syncwarp();
#pragma unroll 4
  for (int it = 0; it < U; ++it) {
    const int r = it * (32 / U) + lane / U, u = lane % U;
    __nv_bfloat16* p = out + (int64_t)(row0 + r) * row_stride + u * 8;
    if (row0 + r < S && in_bounds<__nv_bfloat16>(base, elems, p, 8, err, 44))
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(stg + r * (U * 16) + ((u ^ (r & 7)) << 4));
  }
}

// One CTA's work: KEYS = true computes dK and dV of key tile `tile`, false dQ
// of query tile `tile`.
template <bool KEYS>
__device__ __forceinline__ void ab_tile(const CUtensorMap* tmF1, const CUtensorMap* tmF2, const CUtensorMap* tmG1,
                                        const CUtensorMap* tmG2, const AttnBwdArgs& a, const AbSmem& sm,
                                        uint32_t tmem_base, int tile, int head, const WaitCtl& ctl) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = a.tiles;
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      bool ok = true;
      int i1 = 0, i2 = 0;
      auto load = [&](uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, int t) {
        tma_load_3d(dst, tm, bar, 0, head, t * 128);
        tma_load_3d(dst + AB_BOX, tm, bar, 64, head, t * 128);
      };
      mbar_arrive_expect_tx(sm.f1_full, AB_TILE);
      load(sm.f1, tmF1, sm.f1_full, tile);
      for (int j = 0; j < n && ok; ++j) {
        const int st = j % AB_STAGES;
        const uint32_t ph = (uint32_t)(j / AB_STAGES) & 1u;
        if (!mbar_wait(&sm.g1_empty[st], ph ^ 1u, ctl)) { ok = false; break; }
        mbar_arrive_expect_tx(&sm.g1_full[st], AB_TILE + (KEYS ? AB_ROWVALS : 0));
        load(sm.g1 + st * AB_TILE, tmG1, &sm.g1_full[st], j);
        if (KEYS)
          ab_bulk_load(sm.rowvals + st * AB_ROWVALS, a.rowvals + ((size_t)head * n + j) * 256, AB_ROWVALS,
                       &sm.g1_full[st]);
        ++i1;
        if (j == 0) {
          mbar_arrive_expect_tx(sm.f2_full, AB_TILE);
          load(sm.f2, tmF2, sm.f2_full, tile);
        }
        if (!mbar_wait(&sm.g2_empty[st], ph ^ 1u, ctl)) { ok = false; break; }
        mbar_arrive_expect_tx(&sm.g2_full[st], AB_TILE);
        load(sm.g2 + st * AB_TILE, tmG2, &sm.g2_full[st], j);
        ++i2;
      }
      if (!ok) {  // let issued loads land before the CTA exits
        ab_drain(sm.f1_full, 0);
        if (i1 > 0) ab_drain(sm.f2_full, 0);
        for (int j = (i1 > AB_STAGES ? i1 - AB_STAGES : 0); j < i1; ++j)
          ab_drain(&sm.g1_full[j % AB_STAGES], (uint32_t)(j / AB_STAGES) & 1u);
        for (int j = (i2 > AB_STAGES ? i2 - AB_STAGES : 0); j < i2; ++j)
          ab_drain(&sm.g2_full[j % AB_STAGES], (uint32_t)(j / AB_STAGES) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idesc_a = idesc_bf16(128, 128, false, true);   // G1, G2 MN-major
      const uint32_t f1 = smem_u32(sm.f1), f2 = smem_u32(sm.f2), g1 = smem_u32(sm.g1), g2 = smem_u32(sm.g2);
      // columns [0,128) or [128,256) = F G^T
      auto issue_ss = [&](uint32_t d, uint32_t f, uint32_t g) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = (uint32_t)((k >> 2) * AB_BOX + (k & 3) * 32);
          mma_bf16_ss(tmem_base + d, sdesc_kmajor(f + off), sdesc_kmajor(g + off), idesc_s, k != 0 ? 1u : 0u);
        }
      };
      // accumulator += A G, A bf16 in TMEM: each warpgroup's 64 columns are
      // 32 packed ones at the start of its own half
      auto issue_ts = [&](uint32_t d, uint32_t s, uint32_t g, bool first) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t b = sdesc_sw128(g + (uint32_t)(k * 2048), AB_BOX, 1024);
          ab_mma_ts(tmem_base + d, tmem_base + s + (uint32_t)((k >> 2) * 64 + (k & 3) * 8), b, idesc_a,
                    first && k == 0 ? 0u : 1u);
        }
      };
      bool ok = mbar_wait(sm.f1_full, 0, ctl) && mbar_wait(&sm.g1_full[0], 0, ctl);
      if (ok) {
        tc_fence_after();
        issue_ss(0, f1, g1);
        mma_commit(sm.s_full);
        ok = mbar_wait(sm.f2_full, 0, ctl) && mbar_wait(&sm.g2_full[0], 0, ctl);
      }
      if (ok) {
        tc_fence_after();
        issue_ss(128, f2, g2);
        if (!KEYS) mma_commit(&sm.g2_empty[0]);
        mma_commit(sm.dp_full);
      }
      for (int j = 0; j < n && ok; ++j) {
        const bool more = j + 1 < n;
        const int st = j % AB_STAGES, nx = (j + 1) % AB_STAGES;
        const uint32_t nph = (uint32_t)((j + 1) / AB_STAGES) & 1u;
        // the softmax has read S (and on the key side written P over it)
        if (!mbar_wait(sm.p_full, (uint32_t)j & 1u, ctl)) { ok = false; break; }
        if (KEYS) {
          tc_fence_after();
          issue_ts(384, 0, g2 + st * AB_TILE, j == 0);
          mma_commit(&sm.g2_empty[st]);
        }
        if (more) {
          if (!mbar_wait(&sm.g1_full[nx], nph, ctl)) { ok = false; break; }
          tc_fence_after();
          issue_ss(0, f1, g1 + nx * AB_TILE);
          mma_commit(sm.s_full);
        }
        if (!mbar_wait(sm.ds_full, (uint32_t)j & 1u, ctl)) { ok = false; break; }
        tc_fence_after();
        issue_ts(256, 128, g1 + st * AB_TILE, j == 0);
        mma_commit(&sm.g1_empty[st]);
        if (more) {
          if (!mbar_wait(&sm.g2_full[nx], nph, ctl)) { ok = false; break; }
          tc_fence_after();
          issue_ss(128, f2, g2 + nx * AB_TILE);
          if (!KEYS) mma_commit(&sm.g2_empty[nx]);
          mma_commit(sm.dp_full);
        } else {
          mma_commit(sm.acc_full);
        }
      }
      if (!ok) {
        mma_commit(sm.drain);
        ab_drain(sm.drain, 0);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    const int wg = (warp - 4) >> 2;
    const int qq = warp & 3;
    const int row = qq * 32 + lane;
    const uint32_t s_base = tmem_addr(tmem_base, (uint32_t)(qq * 32), (uint32_t)(wg * 64));
    const uint32_t dp_base = s_base + 128u;
    const float sl2 = a.scale_log2;
    float my_l2 = 0.0f, my_d = 0.0f;
    if (!KEYS) {
      const float* rv = a.rowvals + ((size_t)head * n + tile) * 256 + row;
      if (in_bounds<float>(a.rowvals, a.rowval_elems, rv, 129, a.err, 45)) {
        my_l2 = rv[0];
        my_d = rv[128];
      }
    }
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int st = j % AB_STAGES;
      const float* rv = reinterpret_cast<const float*>(sm.rowvals + st * AB_ROWVALS) + wg * 64;
      if (KEYS && !mbar_wait(&sm.g1_full[st], (uint32_t)(j / AB_STAGES) & 1u, ctl)) { ok = false; break; }
      if (!mbar_wait(sm.s_full, (uint32_t)j & 1u, ctl)) { ok = false; break; }
      tc_fence_after();
      uint32_t p[2][32];
      tmem_ld32(s_base, p[0]);
      tmem_ld32(s_base + 32u, p[1]);
      tmem_ld_wait(p[0]);
      tmem_ld_wait(p[1]);
      const float2 sl2x2 = make_float2(sl2, sl2);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          const float4 l = KEYS ? *reinterpret_cast<const float4*>(rv + h * 32 + c * 2)
                                : make_float4(my_l2, my_l2, my_l2, my_l2);
          const float2 z0 = __ffma2_rn(make_float2(__uint_as_float(p[h][2 * c]), __uint_as_float(p[h][2 * c + 1])),
                                       sl2x2, make_float2(-l.x, -l.y));
          const float2 z1 = __ffma2_rn(make_float2(__uint_as_float(p[h][2 * c + 2]), __uint_as_float(p[h][2 * c + 3])),
                                       sl2x2, make_float2(-l.z, -l.w));
          const float e0 = ab_ex2(z0.x), e1 = ab_ex2(z0.y), e2 = ab_ex2(z1.x), e3 = ab_ex2(z1.y);
          p[h][2 * c] = __float_as_uint(e0);
          p[h][2 * c + 1] = __float_as_uint(e1);
          p[h][2 * c + 2] = __float_as_uint(e2);
          p[h][2 * c + 3] = __float_as_uint(e3);
          pk[c] = pack_bf16x2(e0, e1);
          pk[c + 1] = pack_bf16x2(e2, e3);
        }
        if (KEYS) ab_tmem_st16(s_base + (uint32_t)(h * 16), pk);
      }
      if (KEYS) tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.p_full);
      if (!KEYS && j == n - 1) {
        // keys past the end: their K rows are zero, but exp(-lse) times 0
        // must not become NaN where lse is far below 0
        const int valid = a.S - j * 128 - wg * 64;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (h * 32 + c >= valid) p[h][c] = 0u;
      }
      if (!mbar_wait(sm.dp_full, (uint32_t)j & 1u, ctl)) { ok = false; break; }
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t d[32], pk[16];
        tmem_ld32(dp_base + (uint32_t)(h * 32), d);
        tmem_ld_wait(d);
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          const float4 dd = KEYS ? *reinterpret_cast<const float4*>(rv + 128 + h * 32 + c * 2)
                                 : make_float4(my_d, my_d, my_d, my_d);
          const float2 t0 = __fadd2_rn(make_float2(__uint_as_float(d[2 * c]), __uint_as_float(d[2 * c + 1])),
                                       make_float2(-dd.x, -dd.y));
          const float2 t1 = __fadd2_rn(make_float2(__uint_as_float(d[2 * c + 2]), __uint_as_float(d[2 * c + 3])),
                                       make_float2(-dd.z, -dd.w));
          const float2 u0 = __fmul2_rn(t0, make_float2(__uint_as_float(p[h][2 * c]), __uint_as_float(p[h][2 * c + 1])));
          const float2 u1 =
              __fmul2_rn(t1, make_float2(__uint_as_float(p[h][2 * c + 2]), __uint_as_float(p[h][2 * c + 3])));
          pk[c] = pack_bf16x2(u0.x, u0.y);
          pk[c + 1] = pack_bf16x2(u1.x, u1.y);
        }
        ab_tmem_st16(dp_base + (uint32_t)(h * 16), pk);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.ds_full);
    }
    if (ok && mbar_wait(sm.acc_full, 0, ctl)) {
      tc_fence_after();
      // the accumulators leave through the G rings, idle now (acc_full covers
      // every MMA, and every load has been consumed by one)
      uint8_t* stg = sm.g1 + (warp - 4) * 8192;
      const int row0 = tile * 128 + qq * 32;
      const uint32_t acc = tmem_addr(tmem_base, (uint32_t)(qq * 32), 256);
      if (KEYS) {
        if (wg == 0)
          ab_store<128>(acc + 128u, 1.0f, stg, lane, row0, a.S, a.dv + head * a.d_head_stride, a.d_row_stride, a.dv,
                        a.d_elems, a.err);
        else
          ab_store<128>(acc, a.scale, stg, lane, row0, a.S, a.dk + head * a.d_head_stride, a.d_row_stride, a.dk,
                        a.d_elems, a.err);
      } else {
        ab_store<64>(acc + (uint32_t)(wg * 64), a.scale, stg, lane, row0, a.S,
                     a.dq + head * a.d_head_stride + wg * 64, a.d_row_stride, a.dq, a.d_elems, a.err);
      }
    }
  }
}
}  // namespace

// blockIdx.x: 128-row tile, blockIdx.y: head; z = 0 the key side, z = 1 the
// query side (the longer key-side CTAs are scheduled first).
__global__ void __launch_bounds__(AB_THREADS, 1)
    attention_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                         const AttnBwdArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  AbSmem sm;
  sm.f1 = smem;
  sm.f2 = sm.f1 + AB_TILE;
  sm.g1 = sm.f2 + AB_TILE;
  sm.g2 = sm.g1 + AB_STAGES * AB_TILE;
  sm.rowvals = sm.g2 + AB_STAGES * AB_TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm.rowvals + AB_STAGES * AB_ROWVALS);
  sm.f1_full = bars;
  sm.f2_full = bars + 1;
  sm.g1_full = bars + 2;
  sm.g1_empty = sm.g1_full + AB_STAGES;
  sm.g2_full = sm.g1_empty + AB_STAGES;
  sm.g2_empty = sm.g2_full + AB_STAGES;
  sm.s_full = sm.g2_empty + AB_STAGES;
  sm.p_full = sm.s_full + 1;
  sm.dp_full = sm.p_full + 1;
  sm.ds_full = sm.dp_full + 1;
  sm.acc_full = sm.ds_full + 1;
  sm.drain = sm.acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm.drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(sm.f1_full, 1);
    mbar_init(sm.f2_full, 1);
    for (int s = 0; s < AB_STAGES; ++s) {
      mbar_init(&sm.g1_full[s], 1);
      mbar_init(&sm.g1_empty[s], 1);
      mbar_init(&sm.g2_full[s], 1);
      mbar_init(&sm.g2_empty[s], 1);
    }
    mbar_init(sm.s_full, 1);
    mbar_init(sm.p_full, 8);
    mbar_init(sm.dp_full, 1);
    mbar_init(sm.ds_full, 8);
    mbar_init(sm.acc_full, 1);
    mbar_init(sm.drain, 1);
    *abort_flag = timeout_recorded(args.err) ? 1 : 0;   // sticky timeout of an earlier launch
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
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl ctl{abort_flag, args.err, KID_ATTN_BWD};

  // a wait of an earlier launch ran out: this launch skips its work, before
  // any copy or MMA is issued
  if (*ctl.flag == 0) {
    if (blockIdx.z == 0)
      ab_tile<true>(&tmK, &tmV, &tmQ, &tmO, args, sm, tmem_base, blockIdx.x, blockIdx.y, ctl);
    else
      ab_tile<false>(&tmQ, &tmO, &tmK, &tmV, args, sm, tmem_base, blockIdx.x, blockIdx.y, ctl);
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
  cudaError_t e = launch_kernel(attention_bwd_rows_kernel, rows_grid, dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(attention_bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, AB_SMEM);
  if (e != cudaSuccess) return e;
  e = launch_kernel(attention_bwd_kernel, grid, dim3(AB_THREADS), AB_SMEM, stream, tmQ, tmK, tmV, tmO, a);
  if (e != cudaSuccess) return e;
  set_kernel_info("attention_bwd_kernel tcgen05.mma.cta_group::1.kind::f16 tile=128x128 stages=%d acc=f32 "
                  "tmem=S,dP,A1,A2 P,dS-in-TMEM grid=%ux%ux2",
                  AB_STAGES, grid.x, grid.y);
  return cudaGetLastError();
}

}  // namespace h3
