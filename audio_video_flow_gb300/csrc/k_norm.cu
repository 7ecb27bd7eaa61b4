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
// Channels are handled in chunks of 8: thread t of a row's TPR threads owns
// chunks t, t + TPR, ...; only the last chunk of a row may be partial.
#include "h3_device.cuh"
#include "h3_internal.h"

#include <type_traits>

namespace h3 {

namespace {
constexpr int NORM_FWD_BATCH_THREADS = 256;

// 8 values at p, of which the first `valid` exist (the others read as 0).
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int valid, float (&v)[8]) {
  if (valid >= 8) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = bf16_lo(w[e]);
      v[2 * e + 1] = bf16_hi(w[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < valid ? __bfloat162float(p[e]) : 0.0f;
  }
}
__device__ __forceinline__ void load8(const float* p, int valid, float (&v)[8]) {
  if (valid >= 8) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < valid ? p[e] : 0.0f;
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int valid, const float (&v)[8]) {
  if (valid >= 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) p[e] = __float2bfloat16_rn(v[e]);
  }
}
__device__ __forceinline__ void store8(float* p, int valid, const float (&v)[8]) {
  if (valid >= 8) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) p[e] = v[e];
  }
}
// gain or bias (either type; null reads as `none`)
__device__ __forceinline__ void load_param8(const void* p, int is_fp32, int at, int valid, float none, float (&v)[8]) {
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = none;
  } else if (is_fp32) {
    load8(static_cast<const float*>(p) + at, valid, v);
  } else {
    load8(static_cast<const __nv_bfloat16*>(p) + at, valid, v);
  }
}

// Sum over the row's TPR threads, the same value in all of them: a butterfly
// inside a warp, then the warps' sums in order.  slot: the group's scratch,
// not read since the last __syncthreads before the previous use of the other
// slot (callers alternate two).
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(float (&s)[NV], float* slot) {
  constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < NV; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
  if (TPR > 32) {
    constexpr int NW = TPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < NV; ++k) slot[warp * NV + k] = s[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) t += slot[w * NV + k];
      s[k] = t;
    }
  }
}
}  // namespace

// ---------------------------------------------------------------------------
// Forward: TPR threads per row, NC chunks per thread, the row read once into
// registers and written once.
// ---------------------------------------------------------------------------
template <typename T, int TPR, int NC, bool LAYER>
__global__ void __launch_bounds__(TPR < NORM_FWD_BATCH_THREADS && TPR <= 32 ? NORM_FWD_BATCH_THREADS : TPR)
    norm_fwd_kernel(const NormArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int RPB = TPR <= 32 ? NORM_FWD_BATCH_THREADS / TPR : 1;    // rows per block
  __shared__ float red[2][32];
  const int t = threadIdx.x % TPR;
  const long long unit = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool have = unit < a.units;
  const long long u = have ? unit : 0;
  const int64_t i = u / a.heads, h = u % a.heads;
  const T* x = static_cast<const T*>(a.x) + i * a.x_row + h * a.x_head;
  T* y = static_cast<T*>(a.y) + i * a.y_row + h * a.y_head;
  const int width = a.width;
  float v[NC][8];
  float s[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int at = (t + c * TPR) * 8;
    const int valid = min(width - at, 8);
    if (have && valid > 0 && in_bounds<T>(static_cast<const T*>(a.x), a.x_elems, x + at, valid, a.err, 50)) {
      load8(x + at, valid, v[c]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = 0.0f;
    }
  }
  const float inv_width = 1.0f / (float)width;
  if (LAYER) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[c][e];
    row_sum<TPR>(s, red[0]);
    const float mean = s[0] * inv_width;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int valid = width - (t + c * TPR) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = e < valid ? v[c][e] - mean : 0.0f;
    }
    s[0] = 0.0f;
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] = __fmaf_rn(v[c][e], v[c][e], s[0]);
  row_sum<TPR>(s, red[1]);
  const float r = 1.0f / sqrtf(s[0] * inv_width + a.eps);
  if (!have) return;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int at = (t + c * TPR) * 8;
    const int valid = min(width - at, 8);
    if (valid <= 0) continue;
    float g[8], b[8];
    load_param8(a.gain, a.param_fp32, at, valid, 1.0f, g);
    load_param8(a.bias, a.param_fp32, at, valid, 0.0f, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = __fmaf_rn(v[c][e] * r, g[e], b[e]);
    if (in_bounds<T>(static_cast<const T*>(a.y), a.y_elems, y + at, valid, a.err, 51)) store8(y + at, valid, g);
  }
}

// ---------------------------------------------------------------------------
// Backward.  Persistent CTAs; each row's x and dy are copied asynchronously
// into a ring of NORM_STAGES stages (each thread copies and later reads its
// own chunks, so a stage needs no barrier), the gain is kept in shared memory
// as fp32, and every thread accumulates dgain and dbias of its own channels
// in registers over all the CTA's rows.  The CTA's sums go to the workspace
// and norm_param_kernel adds them in CTA order.
// ---------------------------------------------------------------------------
namespace {
constexpr int NORM_STAGES = 2;

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

template <typename T, int TPR, int NC, bool LAYER>
__global__ void __launch_bounds__(TPR <= 32 ? 256 : TPR) norm_bwd_kernel(const NormArgs a) {
  constexpr int NT = TPR <= 32 ? 256 : TPR;
  constexpr int RPB = NT / TPR;                   // rows a CTA works on at once
  constexpr int ROW = NC * TPR * 8;               // channels of a row, padded
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ float red[2][2 * 32];
  T* ring = reinterpret_cast<T*>(norm_smem);      // [stage][x|dy][RPB][ROW]
  float* sgain = reinterpret_cast<float*>(norm_smem + (size_t)NORM_STAGES * 2 * RPB * ROW * sizeof(T));
  griddep_launch_dependents();
  griddep_wait();
  const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
  const int width = a.width;
  const float inv_width = 1.0f / (float)width;

  auto row_at = [&](long long u, int64_t row, int64_t head) { return (u / a.heads) * row + (u % a.heads) * head; };
  const long long step = (long long)gridDim.x * RPB;
  auto fetch = [&](long long u, int st) {
    if (u < a.units) {
      const T* x = static_cast<const T*>(a.x) + row_at(u, a.x_row, a.x_head);
      const T* dy = static_cast<const T*>(a.dy) + row_at(u, a.dy_row, a.dy_head);
      T* to = ring + (size_t)(st * 2 * RPB + g) * ROW;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (t + c * TPR) * 8;
        const int valid = min(width - at, 8);
        if (valid <= 0) continue;
        if (in_bounds<T>(static_cast<const T*>(a.x), a.x_elems, x + at, valid, a.err, 52)) copy8(to + at, x + at, valid);
        if (in_bounds<T>(static_cast<const T*>(a.dy), a.dy_elems, dy + at, valid, a.err, 53))
          copy8(to + RPB * ROW + at, dy + at, valid);
      }
    }
    cp_async_commit();
  };

  long long u = (long long)blockIdx.x * RPB + g;
  for (int st = 0; st < NORM_STAGES - 1; ++st) fetch(u + st * step, st);
  for (int at = threadIdx.x * 8; at < ROW; at += NT * 8) {
    float v[8];
    const int valid = min(width - at, 8);
    load_param8(valid > 0 ? a.gain : nullptr, a.param_fp32, at, valid, 1.0f, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < valid ? v[e] : 0.0f;
    store8(sgain + at, 8, v);
  }
  __syncthreads();

  float ag[NC][8], ab[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) ag[c][e] = ab[c][e] = 0.0f;

  // every group of the CTA runs the same number of steps (the row sums of
  // TPR > 32 hold a block barrier; narrower groups only shuffle)
  const long long first = (long long)blockIdx.x * RPB;
  int st = 0, parity = 0;   // the RMS norm's one sum per row alternates the scratch slots
  for (long long base = first; base < a.units; base += step, u += step) {
    const bool have = u < a.units;
    fetch(u + (NORM_STAGES - 1) * step, (st + NORM_STAGES - 1) % NORM_STAGES);
    cp_async_wait<NORM_STAGES - 1>();
    const T* xs = ring + (size_t)(st * 2 * RPB + g) * ROW;
    const T* ds = xs + RPB * ROW;
    float mean = 0.0f, mean_w = 0.0f;
    float s[2] = {0.0f, 0.0f};
    if (LAYER) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (t + c * TPR) * 8;
        if (!have || at >= width) continue;
        float x[8], dy[8], gn[8];
        load8(xs + at, 8, x);
        load8(ds + at, 8, dy);
        load8(sgain + at, 8, gn);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[0] += x[e];
          s[1] = __fmaf_rn(dy[e], gn[e], s[1]);
        }
      }
      row_sum<TPR>(s, red[0]);
      mean = s[0] * inv_width;
      mean_w = s[1] * inv_width;
      s[0] = s[1] = 0.0f;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (t + c * TPR) * 8;
      if (!have || at >= width) continue;
      float x[8], dy[8], gn[8];
      load8(xs + at, 8, x);
      load8(ds + at, 8, dy);
      load8(sgain + at, 8, gn);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float cx = !LAYER ? x[e] : (at + e < width ? x[e] - mean : 0.0f);
        s[0] = __fmaf_rn(cx, cx, s[0]);
        s[1] = __fmaf_rn(dy[e] * gn[e], cx, s[1]);
      }
    }
    row_sum<TPR>(s, red[LAYER ? 1 : parity]);
    parity ^= 1;
    const float r = 1.0f / sqrtf(s[0] * inv_width + a.eps);
    const float k = s[1] * r * inv_width;          // mean(w xhat)
    if (have) {
      T* dx = static_cast<T*>(a.dx) + row_at(u, a.dx_row, a.dx_head);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (t + c * TPR) * 8;
        const int valid = min(width - at, 8);
        if (valid <= 0) continue;
        float x[8], dy[8], gn[8], out[8];
        load8(xs + at, 8, x);
        load8(ds + at, 8, dy);
        load8(sgain + at, 8, gn);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xhat = (x[e] - mean) * r;
          out[e] = (__fmaf_rn(dy[e], gn[e], -mean_w) - xhat * k) * r;
          ag[c][e] = __fmaf_rn(dy[e], xhat, ag[c][e]);
          ab[c][e] += dy[e];
        }
        if (in_bounds<T>(static_cast<const T*>(a.dx), a.dx_elems, dx + at, valid, a.err, 54))
          store8(dx + at, valid, out);
      }
    }
    st = (st + 1) % NORM_STAGES;
  }
  cp_async_wait<0>();

  if (a.part == nullptr) return;
  // the CTA's sums: group 0's channels, the other groups added in order
  __syncthreads();
  float* comb = reinterpret_cast<float*>(norm_smem);
  float* part = a.part + (size_t)blockIdx.x * 2 * a.part_width;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (RPB > 1) {
#pragma unroll
      for (int c = 0; c < NC; ++c) store8(comb + (size_t)g * ROW + (t + c * TPR) * 8, 8, which == 0 ? ag[c] : ab[c]);
      __syncthreads();
      for (int at = threadIdx.x; at < width; at += NT) {
        float v = 0.0f;
        for (int k = 0; k < RPB; ++k) v += comb[(size_t)k * ROW + at];
        if (in_bounds<float>(a.part, a.part_elems, part + which * a.part_width + at, 1, a.err, 55))
          part[which * a.part_width + at] = v;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (t + c * TPR) * 8;
        if (at < width && in_bounds<float>(a.part, a.part_elems, part + which * a.part_width + at, 8, a.err, 55))
          store8(part + which * a.part_width + at, 8, which == 0 ? ag[c] : ab[c]);
      }
    }
  }
}

// dgain and dbias: the CTAs' sums added in a fixed order (eight interleaved
// runs over the CTAs, then the eight in order).  blockIdx.y: 0 gain, 1 bias.
__global__ void __launch_bounds__(256) norm_param_kernel(const float* part, int n_parts, int part_width, int width,
                                                         float* dgain, float* dbias) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float red[8][32];
  float* out = blockIdx.y == 0 ? dgain : dbias;
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), seg = threadIdx.x >> 5;
  float s = 0.0f;
  if (out != nullptr && col < width) {
    const float* p = part + (size_t)blockIdx.y * part_width + col;
#pragma unroll 8
    for (int k = seg; k < n_parts; k += 8) s += p[(size_t)k * 2 * part_width];
  }
  red[seg][threadIdx.x & 31] = s;
  __syncthreads();
  if (seg == 0 && out != nullptr && col < width) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += red[k][threadIdx.x];
    out[col] = v;
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
namespace {
// The thread layout of a width: TPR threads per row, NC chunks of 8 channels
// per thread.
template <typename F>
cudaError_t norm_layout(int width, F&& f) {
  const int n = (width + 7) / 8;
#define H3_NORM_CASE(tpr, nc) return f(std::integral_constant<int, tpr>{}, std::integral_constant<int, nc>{})
  if (n <= 16) H3_NORM_CASE(16, 1);
  if (n <= 32) H3_NORM_CASE(32, 1);
  if (n <= 64) H3_NORM_CASE(32, 2);
  if (n <= 128) H3_NORM_CASE(32, 4);
  if (n <= 256) H3_NORM_CASE(128, 2);
  if (n <= 384) H3_NORM_CASE(128, 3);
  if (n <= 512) H3_NORM_CASE(128, 4);
  if (n <= 768) H3_NORM_CASE(256, 3);
  H3_NORM_CASE(256, 4);
#undef H3_NORM_CASE
}
int norm_rows_at_once(int width) {
  int r = 1;
  norm_layout(width, [&](auto tpr, auto) {
    r = tpr() <= 32 ? 256 / tpr() : 1;
    return cudaSuccess;
  });
  return r;
}

template <typename T>
cudaError_t launch_norm_fwd_t(const NormArgs& a, cudaStream_t st) {
  return norm_layout(a.width, [&](auto tpr, auto nc) {
    constexpr int TPR = decltype(tpr)::value, NC = decltype(nc)::value;
    constexpr int RPB = TPR <= 32 ? NORM_FWD_BATCH_THREADS / TPR : 1;
    const long long blocks = (a.units + RPB - 1) / RPB;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(TPR <= 32 ? NORM_FWD_BATCH_THREADS : TPR);
    return a.layer ? launch_kernel(norm_fwd_kernel<T, TPR, NC, true>, grid, block, 0, st, a)
                   : launch_kernel(norm_fwd_kernel<T, TPR, NC, false>, grid, block, 0, st, a);
  });
}

template <typename T>
cudaError_t launch_norm_bwd_t(const NormArgs& a, cudaStream_t st) {
  return norm_layout(a.width, [&](auto tpr, auto nc) {
    constexpr int TPR = decltype(tpr)::value, NC = decltype(nc)::value;
    constexpr int NT = TPR <= 32 ? 256 : TPR, RPB = NT / TPR, ROW = NC * TPR * 8;
    constexpr size_t ring = (size_t)NORM_STAGES * 2 * RPB * ROW * sizeof(T) + (size_t)ROW * 4;
    constexpr size_t comb = RPB > 1 ? (size_t)RPB * ROW * 4 : 0;
    constexpr size_t smem = ring > comb ? ring : comb;
    auto kernel = a.layer ? norm_bwd_kernel<T, TPR, NC, true> : norm_bwd_kernel<T, TPR, NC, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, dim3((unsigned)norm_bwd_ctas(a.units, a.width)), dim3(NT), smem, st, a);
  });
}
}  // namespace

int norm_bwd_ctas(long long units, int width) {
  const long long most = 2LL * num_sms(), blocks = (units + norm_rows_at_once(width) - 1) / norm_rows_at_once(width);
  return (int)(blocks < most ? blocks : most);
}

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st) {
  cudaError_t e = a.fp32 ? launch_norm_fwd_t<float>(a, st) : launch_norm_fwd_t<__nv_bfloat16>(a, st);
  if (e != cudaSuccess) return e;
  set_kernel_info("norm_fwd_kernel %s %s rows=%lld width=%d", a.layer ? "layer" : "rms", a.fp32 ? "fp32" : "bf16",
                  a.units, a.width);
  return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormArgs& a, float* dgain, float* dbias, cudaStream_t st) {
  cudaError_t e = a.fp32 ? launch_norm_bwd_t<float>(a, st) : launch_norm_bwd_t<__nv_bfloat16>(a, st);
  if (e != cudaSuccess) return e;
  const int ctas = norm_bwd_ctas(a.units, a.width);
  if (dgain || dbias) {
    e = launch_kernel(norm_param_kernel, dim3((unsigned)((a.width + 31) / 32), dbias ? 2 : 1), dim3(256), 0, st,
                      (const float*)a.part, ctas, a.part_width, a.width, dgain, dbias);
    if (e != cudaSuccess) return e;
  }
  set_kernel_info("norm_bwd_kernel %s %s rows=%lld width=%d ctas=%d stages=%d", a.layer ? "layer" : "rms",
                  a.fp32 ? "fp32" : "bf16", a.units, a.width, ctas, NORM_STAGES);
  return cudaGetLastError();
}

}  // namespace h3
