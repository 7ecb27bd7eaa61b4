// Device helpers shared by the attention kernels whose MMA warp runs converged
// (the gradient and the windowed and cached forms): MMAs issued four at a time
// by one elected lane, whole-warp waits, packed TMEM stores, and the visible
// ranges of a window.
#pragma once
#include "h3_device.cuh"
#include "h3_internal.h"

namespace h3 {

__device__ __forceinline__ float at_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The MMA warp runs its loop converged, and one lane (`one` != 0) issues.  With
// one lane's branch around the loop instead, a product took about 800 cycles, not
// 600-640, and 8192 rows x 56 heads 4.5 ms, not 3.5.
// Four K steps of 16.  Operand steps are immediate: SA, SB in descriptor units
// of 16 bytes (shared memory) or TMEM columns.
template <int SA, int SB>
__device__ __forceinline__ void at_mma4_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "add.s64 a1, %1, %6;\n\tadd.s64 b1, %2, %7;\n\t"
      "add.s64 a2, a1, %6;\n\tadd.s64 b2, b1, %7;\n\t"
      "add.s64 a3, a2, %6;\n\tadd.s64 b3, b2, %7;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(one), "n"(SA), "n"(SB)
      : "memory");
}
template <int SA, int SB>
__device__ __forceinline__ void at_mma4_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "add.s32 a1, %1, %6;\n\tadd.s64 b1, %2, %7;\n\t"
      "add.s32 a2, a1, %6;\n\tadd.s64 b2, b1, %7;\n\t"
      "add.s32 a3, a2, %6;\n\tadd.s64 b3, b2, %7;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(one), "n"(SA), "n"(SB)
      : "memory");
}
// One K step of 16.
__device__ __forceinline__ void at_mma1_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
// Shared-memory descriptor of a K-major operand without swizzle, K = 16: cores of
// 8 rows x 16 bytes, the two of a row group side by side (row r, channel k at
// (r / 8) 256 + (k / 8) 128 + (r % 8) 16 + (k % 8) 2 bytes).
__device__ __forceinline__ uint64_t at_sdesc_plain16(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128u >> 4) << 16 | (uint64_t)(256u >> 4) << 32 | (uint64_t)1 << 46;
}
__device__ __forceinline__ void at_commit(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
      "r"(one)
      : "memory");
}
__device__ __forceinline__ uint32_t at_elect() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(one));
  return one;
}
__device__ __forceinline__ void at_tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void at_tmem_ld_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void at_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer() - t0 > kWaitLimitNs) return;
  }
}
// A whole warp's wait: one outcome for all lanes, so that a wait that runs out
// leaves no lane behind.
__device__ __forceinline__ bool at_wait(uint64_t* bar, uint32_t parity, const WaitCtl& c) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, c));
}

// TMA loads of four-dimensional boxes
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* tm, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, "
      "%6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

__device__ __forceinline__ void at_tma_store_4d(const CUtensorMap* tm, const void* src, int32_t x, int32_t y, int32_t z,
                                                int32_t w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tm)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Waits until this thread's stores have read their source.
__device__ __forceinline__ void at_tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// ---------------------------------------------------------------------------
// Windows (see h3_window): unit(i) = floor((i - origin) / unit).  Row i sees
// the keys [win_lo, win_hi) and, of the first ones, [0, min(first, win_hi)).
// Key j is seen by the rows [win_row_lo, win_row_hi).  Both ends grow with the
// row or key, so a tile's range runs from its first row's to its last row's.
// ---------------------------------------------------------------------------
__host__ __device__ inline int win_unit(const WindowArgs& w, int i) {   // -1 for rows before the origin
  return w.unit == 1 ? i : (int)((uint32_t)(i - w.origin + w.unit) / (uint32_t)w.unit) - 1;
}
__host__ __device__ inline int win_edge(const WindowArgs& w, int unit, int n) {   // where a unit begins, within [0, n]
  const int64_t x = w.origin + (int64_t)unit * w.unit;
  return x < 0 ? 0 : (x > n ? n : (int)x);
}
// of a row in unit u
__host__ __device__ inline int win_lo_of(const WindowArgs& w, int u, int keys) {
  return w.left < 0 ? 0 : win_edge(w, u - w.left, keys);
}
__host__ __device__ inline int win_hi_of(const WindowArgs& w, int u, int keys) {
  return w.right < 0 ? keys : win_edge(w, u + w.right + 1, keys);
}
__host__ __device__ inline int win_lo(const WindowArgs& w, int i, int keys) { return win_lo_of(w, win_unit(w, i), keys); }
__host__ __device__ inline int win_hi(const WindowArgs& w, int i, int keys) { return win_hi_of(w, win_unit(w, i), keys); }
// of a key in unit u
__host__ __device__ inline int win_row_lo_of(const WindowArgs& w, int u, int rows) {
  return w.right < 0 ? 0 : win_edge(w, u - w.right, rows);
}
__host__ __device__ inline int win_row_hi_of(const WindowArgs& w, int u, int j, int rows) {
  return w.left < 0 || j < w.first ? rows : win_edge(w, u + w.left + 1, rows);
}
__host__ __device__ inline int win_row_lo(const WindowArgs& w, int j, int rows) {
  return win_row_lo_of(w, win_unit(w, j), rows);
}
__host__ __device__ inline int win_row_hi(const WindowArgs& w, int j, int rows) {
  return win_row_hi_of(w, win_unit(w, j), j, rows);
}
// bits [0, x) of a word
__device__ __forceinline__ uint32_t win_bits(int x) {
  return x <= 0 ? 0u : (x >= 32 ? 0xffffffffu : (1u << x) - 1u);
}

// ---------------------------------------------------------------------------
// Sequences of a cache
// ---------------------------------------------------------------------------
__device__ __forceinline__ int64_t cache_slots(const CacheArgs& c) { return (int64_t)c.table_width * c.page_size; }
// Whether a sequence's new rows and length are in range: rows that begin where no
// earlier sequence's do and end within n_rows, and slots for all of them.
__device__ __forceinline__ bool cache_seq_ok(const CacheArgs& c, int n_rows, int s) {
  const int before = s > 0 ? c.start[s - 1] : 0, b = c.start[s], e = c.start[s + 1], len = c.length[s];
  return b >= before && b >= 0 && e >= b && e <= n_rows && len >= e - b && (int64_t)len <= cache_slots(c);
}

}  // namespace h3
