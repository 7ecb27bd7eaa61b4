// Layer norm and RMS norm over rows of `width` channels, forward and backward.
// A row is (packed row i, head h) at i*row_stride + h*head_stride, so that the
// same kernels serve a residual stream (one head) and the per-head Q/K norms
// in place of a packed [S][H][3][128] tensor.  With
//   c = x - mean(x) (layer) or x (RMS),  r = 1/sqrt(mean(c^2) + eps),
//   xhat = c r,  y = xhat gain + bias:
// backward, with w = dy gain,
//   dx = r (w - xhat mean(w xhat) - mean(w))      (mean(w) for the layer norm)
//   dgain = sum over rows of dy xhat,  dbias = sum over rows of dy.
//
// All statistics and sums are fp32, each result is rounded once.  The mean is
// subtracted before squaring, from values already on chip (a variance from
// sums of squares would lose a row whose mean is large).  Every reduction has
// a fixed order, so results repeat bit for bit.
//
// Channels are handled in chunks of 8: thread t of a row's `tpr` threads owns
// chunks t, t + tpr, ...; only the last chunk of a row may be partial.  Narrow
// rows (up to 1024 channels forward, up to 512 backward) belong to a group of up
// to 32 threads, which reduces by shuffles alone, several groups to a CTA; wider
// rows to a whole CTA.
#include "h3_device.cuh"
#include "h3_internal.h"

#include <mutex>
#include <type_traits>

namespace h3 {

namespace {
constexpr int NORM_GROUP_THREADS = 256;   // forward: CTA of rows of at most 1024 channels
constexpr int NORM_BWD_GROUP_THREADS = 256, NORM_BWD_GROUP_CTAS = 2;   // backward: of at most 512
constexpr int NORM_GROUP_CHUNKS = 128;    // forward: the widest such row
constexpr int NORM_MAX_WARPS = 8;

// Eight channels as they lie in memory.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void load_part(const __nv_bfloat16* p, int valid) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = 2 * e < valid ? reinterpret_cast<const uint16_t*>(p)[2 * e] : 0u;
      const uint32_t hi = 2 * e + 1 < valid ? reinterpret_cast<const uint16_t*>(p)[2 * e + 1] : 0u;
      w[e] = lo | (hi << 16);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    v[0] = make_float2(bf16_lo(r.x), bf16_hi(r.x));
    v[1] = make_float2(bf16_lo(r.y), bf16_hi(r.y));
    v[2] = make_float2(bf16_lo(r.z), bf16_hi(r.z));
    v[3] = make_float2(bf16_lo(r.w), bf16_hi(r.w));
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void load_part(const float* p, int valid) {
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = e < valid ? p[e] : 0.0f;
    a = make_float4(w[0], w[1], w[2], w[3]);
    b = make_float4(w[4], w[5], w[6], w[7]);
  }
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
  }
};
// the first `valid` of eight results, each rounded once
__device__ __forceinline__ void put8(__nv_bfloat16* p, int valid, const float2 (&v)[4]) {
  if (valid >= 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                              pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) p[e] = __float2bfloat16_rn((e & 1) ? v[e >> 1].y : v[e >> 1].x);
  }
}
__device__ __forceinline__ void put8(float* p, int valid, const float2 (&v)[4]) {
  if (valid >= 8) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) p[e] = (e & 1) ? v[e >> 1].y : v[e >> 1].x;
  }
}
// 8 channels of gain or bias (either type; null reads as `none`)
__device__ __forceinline__ void param8(const void* p, int is_fp32, int at, int valid, float none, float2 (&v)[4]) {
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = make_float2(none, none);
  } else if (is_fp32) {
    Chunk<float> c;
    if (valid >= 8) c.load(static_cast<const float*>(p) + at);
    else c.load_part(static_cast<const float*>(p) + at, valid);
    c.get(v);
  } else {
    Chunk<__nv_bfloat16> c;
    if (valid >= 8) c.load(static_cast<const __nv_bfloat16*>(p) + at);
    else c.load_part(static_cast<const __nv_bfloat16*>(p) + at, valid);
    c.get(v);
  }
}
__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }
__device__ __forceinline__ void zero_past(float2 (&v)[4], int valid) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (2 * e >= valid) v[e].x = 0.0f;
    if (2 * e + 1 >= valid) v[e].y = 0.0f;
  }
}

// NV sums over a row's threads, the same value in all of them: a butterfly
// inside the group (or warp), then one over the CTA's warps.  slot: scratch of
// NORM_MAX_WARPS * NV floats; two calls in a row need different ones.
template <bool BLOCK, int NV>
__device__ __forceinline__ void row_sum(float (&s)[NV], int tpr, float* slot) {
  if (BLOCK) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < NV; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < NV; ++k) slot[warp * NV + k] = s[k];
    __syncthreads();
    // lane l takes warp (l mod 8)'s sums, 0 past the last warp
#pragma unroll
    for (int k = 0; k < NV; ++k) s[k] = (lane & 7) * 32 < tpr ? slot[(lane & 7) * NV + k] : 0.0f;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < NV; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
  } else {
    for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < NV; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
  }
}
}  // namespace

// ---------------------------------------------------------------------------
// Forward: R rows per thread group at a time, NC chunks of each row per
// thread, kept in registers as read; every row is read and written once.
// Bound by memory.  Few threads with many chunks each keep more rows, and so
// more bytes, in flight on an SM than many threads with few (15,860 x 5376 bf16
// RMS: 56 us, 6.1 TB/s; with three chunks of 256 threads unpacked on loading 94
// us).  A layer norm waits for two reductions, one after the other: 76 us there,
// in fp32 125 us against the RMS norm's 106 (the copy rate: 50 and 101).
// ---------------------------------------------------------------------------
template <typename T, int NC, int R, bool LAYER, bool BLOCK>
__global__ void __launch_bounds__(NORM_GROUP_THREADS) norm_fwd_kernel(const NormArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float red[2][NORM_MAX_WARPS * R];
  const int tpr = a.tpr;
  const int t = BLOCK ? threadIdx.x : threadIdx.x & (tpr - 1);
  const int g = BLOCK ? 0 : threadIdx.x / tpr;
  const int groups = BLOCK ? 1 : NORM_GROUP_THREADS / tpr;
  const int width = a.width;
  const float inv_width = 1.0f / (float)width;
  Chunk<T> raw[R][NC];
  T* y[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const long long u = ((long long)blockIdx.x * R + k) * groups + g;
    y[k] = nullptr;
    if (u < a.units) {
      const int64_t i = a.heads == 1 ? u : u / a.heads, h = a.heads == 1 ? 0 : u - i * a.heads;
      const T* x = static_cast<const T*>(a.x) + i * a.x_row + h * a.x_head;
      y[k] = static_cast<T*>(a.y) + i * a.y_row + h * a.y_head;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (t + c * tpr) * 8, valid = min(width - at, 8);
        if (valid <= 0 || !in_bounds<T>(static_cast<const T*>(a.x), a.x_elems, x + at, valid, a.err, 50)) continue;
        if (valid == 8) raw[k][c].load(x + at);
        else raw[k][c].load_part(x + at, valid);
      }
    }
  }
  float mean[R], s[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    mean[k] = 0.0f;
    if (LAYER) {
      float2 acc = splat(0.0f);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (y[k] == nullptr || (t + c * tpr) * 8 >= width) continue;
        float2 v[4];
        raw[k][c].get(v);
        acc = __fadd2_rn(acc, __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3])));
      }
      s[k] = acc.x + acc.y;
    }
  }
  if (LAYER) {
    row_sum<BLOCK>(s, tpr, red[0]);
#pragma unroll
    for (int k = 0; k < R; ++k) mean[k] = s[k] * inv_width;
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    float2 acc = splat(0.0f);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (t + c * tpr) * 8;
      if (y[k] == nullptr || at >= width) continue;
      float2 v[4];
      raw[k][c].get(v);
      if (LAYER) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __fadd2_rn(v[e], splat(-mean[k]));
        if (width - at < 8) zero_past(v, width - at);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc = __ffma2_rn(v[e], v[e], acc);
    }
    s[k] = acc.x + acc.y;
  }
  row_sum<BLOCK>(s, tpr, red[1]);
  float r[R];
#pragma unroll
  for (int k = 0; k < R; ++k) r[k] = rsqrtf(s[k] * inv_width + a.eps);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int at = (t + c * tpr) * 8, valid = min(width - at, 8);
    if (valid <= 0) continue;
    float2 gn[4], bs[4];
    param8(a.gain, a.param_fp32, at, valid, 1.0f, gn);
    param8(a.bias, a.param_fp32, at, valid, 0.0f, bs);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (y[k] == nullptr) continue;
      float2 v[4];
      raw[k][c].get(v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (LAYER) v[e] = __fadd2_rn(v[e], splat(-mean[k]));
        v[e] = __ffma2_rn(__fmul2_rn(v[e], splat(r[k])), gn[e], bs[e]);
      }
      if (in_bounds<T>(static_cast<const T*>(a.y), a.y_elems, y[k] + at, valid, a.err, 51)) put8(y[k] + at, valid, v);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  Persistent CTAs take R rows per thread group and step.  The x and
// dy of a step are copied asynchronously into a ring of ST stages ahead of
// their use (each thread copies and later reads its own chunks, so a stage
// needs no barrier) and then, with HOLD, kept in registers as fp32: unpacking
// them again for each pass costs about as many instructions as the
// arithmetic.  The gain is kept in shared memory as fp32; every thread
// accumulates dgain (and, with BIAS, dbias) of its own channels in registers
// over all the CTA's rows.  The CTAs' sums go to the workspace, where
// norm_param_kernel adds them in CTA order.
// Measured, with both launches: 15,860 x 5376 bf16 RMS 86 us (5.9 TB/s), layer norm with
// bias 115 us (4.4 TB/s: its two reductions and the accumulators of both
// parameters, 48 registers of a thread, leave 14 warps to an SM), in fp32 153 and
// 209 us (6.7 and 4.9 TB/s); 1824 x 56 rows of 128 20 us, 15,860 x 56 of them 116
// us (5.9 TB/s), layer norms 128.
// ---------------------------------------------------------------------------
namespace {
__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 8 channels of which the first `valid` (1..8) exist: the others become 0
template <typename T>
__device__ __forceinline__ void copy8(T* dst, const T* src, int valid) {
  constexpr int PER = 16 / (int)sizeof(T);
#pragma unroll
  for (int k = 0; k < 8 / PER; ++k) {
    const int n = max(0, min(valid - k * PER, PER));
    cp_async16(dst + k * PER, n > 0 ? src + k * PER : src, n * (int)sizeof(T));
  }
}
}  // namespace

template <typename T, int NC, int R, int ST, bool HOLD, bool LAYER, bool BIAS, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 32 * NORM_MAX_WARPS : NORM_BWD_GROUP_THREADS, BLOCK ? (NC == 4 ? 1 : 2) : NORM_BWD_GROUP_CTAS)
    norm_bwd_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ float red[2][NORM_MAX_WARPS * 2 * R];
  const int tpr = a.tpr;
  const int t = BLOCK ? threadIdx.x : threadIdx.x & (tpr - 1);
  const int g = BLOCK ? 0 : threadIdx.x / tpr;
  const int groups = BLOCK ? 1 : NORM_BWD_GROUP_THREADS / tpr;
  const int row = NC * tpr * 8;                   // channels of a row, padded
  // ring: [stage][R][x|dy][group][row]
  T* ring = reinterpret_cast<T*>(norm_smem) + (size_t)g * row + t * 8;
  const int which_step = groups * row, stage_step = R * 2 * which_step;
  float* sgain = reinterpret_cast<float*>(norm_smem + (size_t)ST * stage_step * sizeof(T));
  griddep_launch_dependents();
  griddep_wait();
  const int width = a.width;
  const float inv_width = 1.0f / (float)width;
  const long long step = (long long)gridDim.x * groups * R;
  // only a thread's last chunk may be partial or missing: layout_of() leaves
  // no more than that to a width
  const int last = max(0, min(width - (t + (NC - 1) * tpr) * 8, 8));
  auto valid = [&](int c) { return c < NC - 1 ? 8 : last; };

  // The rows of a step are base + g + k groups, k < R.  Pointers to x and dy of
  // the next step to fetch and to dx of the current one advance by a step's
  // packed rows and heads, and by one more row where the heads wrap round.
  const int64_t di = step / a.heads;
  const int dh = (int)(step - di * a.heads);
  const int64_t adv_x = di * a.x_row + dh * a.x_head, wrap_x = a.x_row - a.heads * a.x_head;
  const int64_t adv_dy = di * a.dy_row + dh * a.dy_head, wrap_dy = a.dy_row - a.heads * a.dy_head;
  const int64_t adv_dx = di * a.dx_row + dh * a.dx_head, wrap_dx = a.dx_row - a.heads * a.dx_head;
  long long base = (long long)blockIdx.x * groups * R;
  const T *px[R], *pdy[R];
  T* pdx[R];
  int nh[R], ch[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const long long u = base + g + k * groups;
    const int64_t i = u / a.heads;
    nh[k] = ch[k] = (int)(u - i * a.heads);
    px[k] = static_cast<const T*>(a.x) + i * a.x_row + nh[k] * a.x_head + t * 8;
    pdy[k] = static_cast<const T*>(a.dy) + i * a.dy_row + nh[k] * a.dy_head + t * 8;
    pdx[k] = static_cast<T*>(a.dx) + i * a.dx_row + nh[k] * a.dx_head + t * 8;
  }
  // rows of the CTA's step that begins at `from` (uniform), as an int
  auto rows_left = [&](long long from) { return (int)min(max(a.units - from, 0LL), (long long)(1 << 30)); };
  auto fetch = [&](long long from, T* to) {
    const int left = rows_left(from);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (g + k * groups < left) {
        T* to_x = to + k * 2 * which_step;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int at = c * tpr * 8;
          if (valid(c) <= 0) continue;
          if (in_bounds<T>(static_cast<const T*>(a.x), a.x_elems, px[k] + at, valid(c), a.err, 52))
            copy8(to_x + at, px[k] + at, valid(c));
          if (in_bounds<T>(static_cast<const T*>(a.dy), a.dy_elems, pdy[k] + at, valid(c), a.err, 53))
            copy8(to_x + which_step + at, pdy[k] + at, valid(c));
        }
        nh[k] += dh;
        const bool wrap = nh[k] >= a.heads;
        if (wrap) nh[k] -= a.heads;
        px[k] += adv_x + (wrap ? wrap_x : 0);
        pdy[k] += adv_dy + (wrap ? wrap_dy : 0);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) fetch(base + s * step, ring + s * stage_step);
  for (int at = threadIdx.x * 8; at < row; at += blockDim.x * 8) {
    float2 v[4];
    param8(at < width ? a.gain : nullptr, a.param_fp32, at, width - at, 1.0f, v);
    zero_past(v, width - at);
    put8(sgain + at, 8, v);
  }
  __syncthreads();

  float2 ag[NC][4], ab[BIAS ? NC : 1][4];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ag[c][e] = splat(0.0f);
      if (BIAS) ab[c][e] = splat(0.0f);
    }
  auto gain8 = [&](int at, float2 (&v)[4]) {
    Chunk<float> c;
    c.load(sgain + at);
    c.get(v);
  };

  // every group of the CTA runs the same number of steps: wide rows meet at
  // the reductions' barrier, and half-warp groups at their warp's shuffles
  const T* from = ring;
  T* to = ring + (ST - 1) * stage_step;
  T* const ring_end = ring + ST * stage_step;
  int parity = 0;
  for (; base < a.units; base += step) {
    fetch(base + (ST - 1) * step, to);
    cp_async_wait<ST - 1>();
    const int left = rows_left(base);
    // x and dy of a row's chunk: unpacked once (HOLD), or again for each pass
    float2 xv[HOLD ? R : 1][HOLD ? NC : 1][4], dv[HOLD ? R : 1][HOLD ? NC : 1][4];
    auto unpack = [&](int k, int c, float2 (&x)[4], float2 (&d)[4]) {
      if (valid(c) > 0 && g + k * groups < left) {
        const T* p = from + k * 2 * which_step + c * tpr * 8;
        Chunk<T> xc, dc;
        xc.load(p);
        dc.load(p + which_step);
        xc.get(x);
        dc.get(d);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = d[e] = splat(0.0f);
      }
    };
    auto row_of = [&](int k, int c, float2 (&x)[4], float2 (&d)[4]) {
      if (HOLD) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = xv[HOLD ? k : 0][HOLD ? c : 0][e];
          d[e] = dv[HOLD ? k : 0][HOLD ? c : 0][e];
        }
      } else {
        unpack(k, c, x, d);
      }
    };
    if (HOLD) {
#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int c = 0; c < NC; ++c) unpack(k, c, xv[HOLD ? k : 0][HOLD ? c : 0], dv[HOLD ? k : 0][HOLD ? c : 0]);
    }
    float mean[R], mean_w[R], s[2 * R];
#pragma unroll
    for (int k = 0; k < R; ++k) mean[k] = mean_w[k] = 0.0f;
    if (LAYER) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        float2 sx = splat(0.0f), sw = splat(0.0f);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          float2 gv[4], x[4], d[4];
          row_of(k, c, x, d);
          gain8((t + c * tpr) * 8, gv);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sx = __fadd2_rn(sx, x[e]);
            sw = __ffma2_rn(d[e], gv[e], sw);
          }
        }
        s[2 * k] = sx.x + sx.y;
        s[2 * k + 1] = sw.x + sw.y;
      }
      row_sum<BLOCK>(s, tpr, red[0]);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        mean[k] = s[2 * k] * inv_width;
        mean_w[k] = s[2 * k + 1] * inv_width;
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float2 sc = splat(0.0f), sw = splat(0.0f);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float2 gv[4], x[4], d[4];
        row_of(k, c, x, d);
        gain8((t + c * tpr) * 8, gv);
        if (LAYER) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = __fadd2_rn(x[e], splat(-mean[k]));
          if (valid(c) < 8) zero_past(x, valid(c));
          if (HOLD) {
#pragma unroll
            for (int e = 0; e < 4; ++e) xv[HOLD ? k : 0][HOLD ? c : 0][e] = x[e];
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc = __ffma2_rn(x[e], x[e], sc);
          sw = __ffma2_rn(__fmul2_rn(d[e], gv[e]), x[e], sw);
        }
      }
      s[2 * k] = sc.x + sc.y;
      s[2 * k + 1] = sw.x + sw.y;
    }
    // (the RMS norm's one sum per step alternates the scratch slots)
    row_sum<BLOCK>(s, tpr, red[LAYER ? 1 : parity]);
    parity ^= 1;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float r = rsqrtf(s[2 * k] * inv_width + a.eps);
      const float m = s[2 * k + 1] * r * inv_width;          // mean(w xhat)
      const bool have = g + k * groups < left;
      T* dx = pdx[k];
      ch[k] += dh;
      const bool wrap = ch[k] >= a.heads;
      if (wrap) ch[k] -= a.heads;
      pdx[k] += adv_dx + (wrap ? wrap_dx : 0);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float2 gv[4], x[4], d[4];
        row_of(k, c, x, d);
        gain8((t + c * tpr) * 8, gv);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 cx = LAYER && !HOLD ? __fadd2_rn(x[e], splat(-mean[k])) : x[e];
          const float2 xhat = __fmul2_rn(cx, splat(r));
          ag[c][e] = __ffma2_rn(d[e], xhat, ag[c][e]);
          if (BIAS) ab[c][e] = __fadd2_rn(ab[c][e], d[e]);
          const float2 w = LAYER ? __ffma2_rn(d[e], gv[e], splat(-mean_w[k])) : __fmul2_rn(d[e], gv[e]);
          gv[e] = __fmul2_rn(__ffma2_rn(xhat, splat(-m), w), splat(r));
        }
        dx += c == 0 ? 0 : tpr * 8;
        if (have && valid(c) > 0 &&
            in_bounds<T>(static_cast<const T*>(a.dx), a.dx_elems, dx, valid(c), a.err, 54))
          put8(dx, valid(c), gv);
      }
    }
    from = from + stage_step == ring_end ? ring : from + stage_step;
    to = to + stage_step == ring_end ? ring : to + stage_step;
  }
  cp_async_wait<0>();

  if (a.part == nullptr) return;
  // the CTA's sums: each group's channels, the groups added in order
  const int n_which = BIAS ? 2 : 1;
  float* part = a.part + (size_t)blockIdx.x * n_which * a.part_width;
  float* comb = reinterpret_cast<float*>(norm_smem);
#pragma unroll
  for (int which = 0; which < n_which; ++which) {
    if (BLOCK) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (t + c * tpr) * 8;
        float* p = part + which * a.part_width + at;
        if (at < width && in_bounds<float>(a.part, a.part_elems, p, 8, a.err, 55))
          put8(p, 8, which == 0 ? ag[c] : ab[BIAS ? c : 0]);
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < NC; ++c)
        put8(comb + (size_t)g * row + (t + c * tpr) * 8, 8, which == 0 ? ag[c] : ab[BIAS ? c : 0]);
      __syncthreads();
      for (int at = threadIdx.x; at < width; at += NORM_BWD_GROUP_THREADS) {
        float v = 0.0f;
        for (int k = 0; k < groups; ++k) v += comb[(size_t)k * row + at];
        float* p = part + which * a.part_width + at;
        if (in_bounds<float>(a.part, a.part_elems, p, 1, a.err, 55)) *p = v;
      }
    }
  }
}

// dgain and dbias: the CTAs' sums added in a fixed order (32 interleaved runs
// over the CTAs, then the 32 in order).  A CTA handles 32 channels of one of
// the two (blockIdx.y: 0 gain, 1 bias).
__global__ void __launch_bounds__(256) norm_param_kernel(const float* part, int n_parts, int n_which, int part_width,
                                                         int width, float* dgain, float* dbias) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float4 red[32][8];
  float* out = blockIdx.y == 0 ? dgain : dbias;
  if (out == nullptr) return;
  const int seg = threadIdx.x >> 3, q = threadIdx.x & 7;
  const int col = blockIdx.x * 32 + q * 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (col < width) {   // part_width is a multiple of 8: whole vectors
    const float* p = part + (size_t)blockIdx.y * part_width + col;
#pragma unroll 8
    for (int k = seg; k < n_parts; k += 32) {
      const float4 v = *reinterpret_cast<const float4*>(p + (size_t)k * n_which * part_width);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  red[seg][q] = s;
  __syncthreads();
  if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < (unsigned)width) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += reinterpret_cast<const float*>(red[k])[threadIdx.x];
    out[blockIdx.x * 32 + threadIdx.x] = v;
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
namespace {
constexpr int kNormSmemMax = 227 * 1024;
constexpr int kNormBwdCtasPerSm = 4;

// Thread layout of a width: chunks per thread nc, threads per row tpr (a power
// of two up to 32 for a thread group, whole warps for a CTA).
struct NormLayout {
  int nc, tpr;
  bool block;
};
// Every thread's chunks but the last exist: (nc - 1) tpr chunks are no more than
// the row's n.
NormLayout group_layout(int n) {
  NormLayout l;
  l.block = false;
  l.nc = n <= 32 ? 1 : (n <= 64 ? 2 : 4);
  l.tpr = 4;
  while (l.tpr * l.nc < n) l.tpr *= 2;
  return l;
}
NormLayout block_layout(int n, int nc) {
  NormLayout l;
  l.block = true;
  l.nc = nc;
  l.tpr = (n + 32 * nc - 1) / (32 * nc) * 32;
  return l;
}
// Forward, wide rows: 8 chunks per thread (here any chunk may be missing).
NormLayout fwd_layout(int width) {
  const int n = (width + 7) / 8;
  return n > NORM_GROUP_CHUNKS ? block_layout(n, 8) : group_layout(n);
}
// Backward: a thread group while two chunks of 32 threads reach, then one chunk
// of up to 8 warps, then three of them, then four (the accumulators are 16
// registers a chunk).  Both sides of each limit, 2^25 channels in all, RMS bf16 /
// layer fp32, us: group against CTA at 400 channels 39 / 70 against 82 / 98, at 512
// 34 / 67 against 66 / 82; CTA of one chunk against a group of four at 1000 43 / 83
// against 61 / 148; one chunk against three at 1536 41 / 76 against 57 / 127, at
// 2048 39 / 77 against 40 / 85.
NormLayout bwd_layout(int width) {
  const int n = (width + 7) / 8;
  if (n <= 64) return group_layout(n);
  return block_layout(n, n <= 32 * NORM_MAX_WARPS ? 1 : (n <= 3 * 32 * NORM_MAX_WARPS ? 3 : 4));
}

// Rows per group and step, ring stages, and whether rows are held as fp32.
// Wide bf16 layer norms take two rows at a time and unpack them for every pass:
// their second reduction costs more than the unpacking (8192 channels: 112 us
// against 123 held; RMS norms measure the same either way).  fp32 rows are held:
// two at a time do not fit in shared memory at four chunks, and one at a time read
// again measures 102, 100 and 106 us at 2688, 5376 and 8192 channels (2^25 in all)
// against 89, 94 and 92 held.
struct NormBwdShape {
  int rows, stages;
  bool hold;
};
constexpr NormBwdShape bwd_shape(int nc, bool fp32, bool layer) {
  if (layer && !fp32 && nc >= 3) return {2, 2, false};
  return {nc == 1 ? 2 : 1, fp32 ? 2 : 4, true};
}
struct NormBwdPlan {
  NormLayout l;
  int rows, threads, groups;
  size_t smem;
  int ctas;
};
NormBwdPlan bwd_plan(long long units, int width, bool fp32, bool layer) {
  NormBwdPlan p;
  p.l = bwd_layout(width);
  p.threads = p.l.block ? p.l.tpr : NORM_BWD_GROUP_THREADS;
  p.groups = p.threads / p.l.tpr;
  const NormBwdShape sh = bwd_shape(p.l.nc, fp32, layer);
  p.rows = sh.rows;
  const size_t row = (size_t)p.l.nc * p.l.tpr * 8;
  p.smem = (size_t)sh.stages * p.rows * 2 * p.groups * row * (fp32 ? 4 : 2) + row * 4;
  if (!p.l.block && p.smem < (size_t)p.groups * row * 4) p.smem = (size_t)p.groups * row * 4;
  // at most what fits by shared memory and four: the workspace is sized for
  // these, the launch takes as many as the kernel's registers let be resident
  const int per_sm = (int)(kNormSmemMax / (p.smem + 1024));
  const long long most = (long long)(per_sm < 1 ? 1 : (per_sm > kNormBwdCtasPerSm ? kNormBwdCtasPerSm : per_sm)) * num_sms();
  const long long steps = (units + p.groups * p.rows - 1) / (p.groups * p.rows);
  p.ctas = (int)(steps < most ? steps : most);
  return p;
}
// CTAs of a kernel that fit on one SM; asked once per kernel, device and shape
// (when the table is full, every time).
int resident_ctas(const void* kernel, int threads, size_t smem) {
  struct Entry {
    const void* kernel;
    int device, threads;
    size_t smem;
    int ctas;
  };
  static std::mutex mu;
  static Entry known[256];
  static int n_known = 0;
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lk(mu);
  for (int i = 0; i < n_known; ++i) {
    const Entry& e = known[i];
    if (e.kernel == kernel && e.device == dev && e.threads == threads && e.smem == smem) return e.ctas;
  }
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 1;
  }
  if (n_known < (int)(sizeof(known) / sizeof(known[0]))) known[n_known++] = {kernel, dev, threads, smem, n};
  return n;
}

template <typename F>
cudaError_t with_flag(bool b, F&& f) {
  return b ? f(std::true_type{}) : f(std::false_type{});
}

template <typename T, int NC, int R, bool BLOCK>
cudaError_t launch_fwd(const NormArgs& a, int threads, cudaStream_t st) {
  const long long per = (long long)R * (BLOCK ? 1 : threads / a.tpr);
  const long long blocks = (a.units + per - 1) / per;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return with_flag(a.layer != 0, [&](auto layer) {
    return launch_kernel(norm_fwd_kernel<T, NC, R, decltype(layer)::value, BLOCK>, dim3((unsigned)blocks),
                         dim3((unsigned)threads), 0, st, a);
  });
}
template <typename T>
cudaError_t launch_fwd_t(NormArgs& a, cudaStream_t st) {
  const NormLayout l = fwd_layout(a.width);
  a.tpr = l.tpr;
  if (l.block) return launch_fwd<T, 8, 1, true>(a, l.tpr, st);
  if (l.nc == 1) return launch_fwd<T, 1, 4, false>(a, NORM_GROUP_THREADS, st);
  if (l.nc == 2) return launch_fwd<T, 2, 2, false>(a, NORM_GROUP_THREADS, st);
  return launch_fwd<T, 4, 1, false>(a, NORM_GROUP_THREADS, st);
}

template <typename T, int NC, bool BLOCK>
cudaError_t launch_bwd(const NormArgs& a, NormBwdPlan& p, bool bias, cudaStream_t st) {
  return with_flag(a.layer != 0, [&](auto layer) {
    return with_flag(bias, [&](auto with_bias) {
      constexpr bool LAYER = decltype(layer)::value;
      constexpr NormBwdShape sh = bwd_shape(NC, sizeof(T) == 4, LAYER);
      auto kernel =
          norm_bwd_kernel<T, NC, sh.rows, sh.stages, sh.hold, LAYER, decltype(with_bias)::value, BLOCK>;
      if (p.smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem);
        if (e != cudaSuccess) return e;
      }
      const long long fit =
          (long long)resident_ctas(reinterpret_cast<const void*>(kernel), p.threads, p.smem) * num_sms();
      if (p.ctas > fit) p.ctas = (int)fit;
      return launch_kernel(kernel, dim3((unsigned)p.ctas), dim3((unsigned)p.threads), p.smem, st, a);
    });
  });
}
template <typename T>
cudaError_t launch_bwd_t(const NormArgs& a, NormBwdPlan& p, bool bias, cudaStream_t st) {
  if (!p.l.block) return p.l.nc == 1 ? launch_bwd<T, 1, false>(a, p, bias, st) : launch_bwd<T, 2, false>(a, p, bias, st);
  if (p.l.nc == 1) return launch_bwd<T, 1, true>(a, p, bias, st);
  return p.l.nc == 3 ? launch_bwd<T, 3, true>(a, p, bias, st) : launch_bwd<T, 4, true>(a, p, bias, st);
}
}  // namespace

int norm_bwd_ctas(long long units, int width, bool fp32, bool layer) {
  return bwd_plan(units, width, fp32, layer).ctas;
}

cudaError_t launch_norm_fwd(NormArgs a, cudaStream_t st) {
  cudaError_t e = a.fp32 ? launch_fwd_t<float>(a, st) : launch_fwd_t<__nv_bfloat16>(a, st);
  if (e != cudaSuccess) return e;
  set_kernel_info("norm_fwd_kernel %s %s rows=%lld width=%d threads/row=%d", a.layer ? "layer" : "rms",
                  a.fp32 ? "fp32" : "bf16", a.units, a.width, a.tpr);
  return cudaGetLastError();
}

cudaError_t launch_norm_bwd(NormArgs a, float* dgain, float* dbias, cudaStream_t st) {
  NormBwdPlan p = bwd_plan(a.units, a.width, a.fp32, a.layer);
  a.tpr = p.l.tpr;
  const bool bias = dbias != nullptr;
  cudaError_t e = a.fp32 ? launch_bwd_t<float>(a, p, bias, st) : launch_bwd_t<__nv_bfloat16>(a, p, bias, st);
  if (e != cudaSuccess) return e;
  if (dgain || dbias) {
    e = launch_kernel(norm_param_kernel, dim3((unsigned)((a.width + 31) / 32), bias ? 2 : 1), dim3(256), 0, st,
                      (const float*)a.part, p.ctas, bias ? 2 : 1, a.part_width, a.width, dgain, dbias);
    if (e != cudaSuccess) return e;
  }
  set_kernel_info("norm_bwd_kernel %s %s rows=%lld width=%d threads/row=%d rows/step=%d ctas=%d",
                  a.layer ? "layer" : "rms", a.fp32 ? "fp32" : "bf16", a.units, a.width, a.tpr, p.rows * p.groups,
                  p.ctas);
  return cudaGetLastError();
}

}  // namespace h3
