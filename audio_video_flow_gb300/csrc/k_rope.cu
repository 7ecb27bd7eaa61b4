// Rotary positions on the channels of every head of q and k: the pair of
// channels of (axis a, frequency f), j = a F + f, is turned by the angle
// pos[i][a] * omega[a][f] and scaled by the magnitude.  Pairs lie half a
// rotated width apart (j, j + A F) or side by side (2j, 2j + 1); channels past
// the 2 A F rotated ones pass through.  The gradient is the turn by the
// opposite angle.
//
// Angles: omega is held as turns per position in 64-bit fixed point (2^64 = one
// turn), so that the low 64 bits of pos * omega are the angle's fraction of a
// turn, within 2^-32 turns for every 32-bit position (an fp32 product is
// wrong by 0.06 radians at position 10^6).  The sine and cosine are of what
// that fraction is off the nearest quarter turn, in units of 2^-34 turns; of
// its 32 bits fp32 holds 24, and the rest is brought in as a first-order
// change (the whole fraction rounded to fp32 would be off by 2^-26 turns, and
// a sine near the half turn by many of its own units).
//
// Bound by memory: q and k are read and written once.  A CTA handles one
// packed row (of few rows: a range of its heads; of many rows with few heads:
// several rows).  A thread owns a pair of
// 16-byte vectors of a head (the first channels and the second ones of its
// pairs, or two vectors of whole pairs, or two of passed-through channels) and
// walks over the heads; it asks for the vectors of RO_BATCH heads before the
// row's sines and cosines are computed (once per CTA, into shared memory).
#include "h3_device.cuh"
#include "h3_internal.h"

namespace h3 {

namespace {
// 128 threads with 4 heads' loads each, five CTAs per SM (15,860 rows of 112
// heads x 128 bf16: 130 us, 7.0 TB/s; 256 threads, two CTAs: 162 us; two heads'
// loads, eight CTAs: 141 us).
constexpr int RO_THREADS = 128, RO_CTAS = 5;
constexpr int RO_BATCH = 4;              // heads whose loads a thread issues before their use
constexpr int RO_STAGE_BYTES = 16384;    // the staged form's heads of one CTA
constexpr int RO_ANGLES = 512;           // rows x pairs of a CTA that handles several rows

// 16 bytes of channels, as they lie in memory and as fp32.
template <typename T>
__device__ __forceinline__ void ro_unpack(const uint4& r, float (&v)[16 / sizeof(T)]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (sizeof(T) == 2) {
      v[2 * e] = bf16_lo(w[e]);
      v[2 * e + 1] = bf16_hi(w[e]);
    } else {
      v[e] = __uint_as_float(w[e]);
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 ro_pack(const float (&v)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 2)
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  else
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ float ro_get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ro_get(const float* p) { return *p; }
__device__ __forceinline__ void ro_put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void ro_put(float* p, float v) { *p = v; }

// two neighbouring channels, the first at an even place
__device__ __forceinline__ float2 ro_get2(const __nv_bfloat16* p) {
  const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(bf16_lo(v), bf16_hi(v));
}
__device__ __forceinline__ float2 ro_get2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ void ro_put2(__nv_bfloat16* p, float2 v) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v.x, v.y);
}
__device__ __forceinline__ void ro_put2(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }

// sines and cosines of `rows` rows, times the magnitude: [row][pair]
__device__ __forceinline__ void ro_angles(const RopePosArgs& a, int64_t row, int rows, float* cs, float* sn) {
  const int P = a.axes * a.freqs;
  for (int i = threadIdx.x; i < rows * P; i += blockDim.x) {
    const int r = i / P, p = i - r * P;
    const int32_t* pp = a.pos + (row + r) * a.axes + p / a.freqs;
    const int32_t pos = in_bounds<int32_t>(a.pos, a.pos_elems, pp, 1, a.err, 60) ? *pp : 0;
    const uint64_t turn = (uint64_t)(int64_t)pos * a.turns[p];
    const uint32_t quarter = ((uint32_t)(turn >> 32) + 0x20000000u) >> 30;   // the nearest one, 0..3
    const int32_t off = (int32_t)(uint32_t)(turn >> 30);                     // from it, 2^-34 turns each
    const float f = (float)off;
    const float low = (float)(off - __float2int_rn(f)) * 3.6572953e-10f;     // 2 pi 2^-34: radians
    float s0, c0;
    sincospif(f * 1.16415321826934814453e-10f, &s0, &c0);                    // 2^-33: half turns in [-1/4, 1/4]
    const float s1 = __fmaf_rn(c0, low, s0), c1 = __fmaf_rn(-s0, low, c0);
    const bool odd = quarter & 1u, back = quarter & 2u;
    const float s = back ? -(odd ? c1 : s1) : (odd ? c1 : s1);
    const float c = back != odd ? -(odd ? s1 : c1) : (odd ? s1 : c1);
    cs[i] = c * a.magnitude;
    sn[i] = s * a.sin_scale;
  }
}

// The heads of a CTA's rows, numbered through: `n` of each row, the q heads and
// then the k heads from number `first` on.  MULTI: several rows.
template <typename T, bool MULTI>
struct RoHeads {
  const T *q_in, *k_in;
  T *q_out, *k_out;
  int first, n;
  __device__ __forceinline__ RoHeads(const RopePosArgs& a, int64_t row, int first_, int n_) : first(first_), n(n_) {
    q_in = static_cast<const T*>(a.q_in) + row * a.in_row;
    k_in = static_cast<const T*>(a.k_in) + row * a.in_row - a.q_heads * a.in_head;
    q_out = static_cast<T*>(a.q_out) + row * a.out_row;
    k_out = static_cast<T*>(a.k_out) + row * a.out_row - a.q_heads * a.out_head;
  }
  __device__ __forceinline__ int row_of(int i) const { return MULTI ? i / n : 0; }
  __device__ __forceinline__ int head_of(int i) const { return first + (MULTI ? i - i / n * n : i); }
  __device__ __forceinline__ const T* src(const RopePosArgs& a, int i) const {
    const int h = head_of(i);
    return (h < a.q_heads ? q_in : k_in) + h * a.in_head + row_of(i) * a.in_row;
  }
  __device__ __forceinline__ T* dst(const RopePosArgs& a, int i) const {
    const int h = head_of(i);
    return (h < a.q_heads ? q_out : k_out) + h * a.out_head + row_of(i) * a.out_row;
  }
};
template <typename T>
__device__ __forceinline__ bool ro_in_ok(const RopePosArgs& a, int h, const T* p, int n) {
  return h < a.q_heads ? in_bounds<T>(static_cast<const T*>(a.q_in), a.q_in_elems, p, n, a.err, 61)
                       : in_bounds<T>(static_cast<const T*>(a.k_in), a.k_in_elems, p, n, a.err, 62);
}
template <typename T>
__device__ __forceinline__ bool ro_out_ok(const RopePosArgs& a, int h, const T* p, int n) {
  return h < a.q_heads ? in_bounds<T>(static_cast<const T*>(a.q_out), a.q_out_elems, p, n, a.err, 63)
                       : in_bounds<T>(static_cast<const T*>(a.k_out), a.k_out_elems, p, n, a.err, 64);
}
}  // namespace

// Heads whose rotated channels are whole 16-byte vectors.
template <typename T, bool HALF, bool MULTI>
__global__ void __launch_bounds__(RO_THREADS, RO_CTAS) rope_kernel(const RopePosArgs a) {
  __shared__ float cs[MULTI ? RO_ANGLES : kRopeMaxPairs], sn[MULTI ? RO_ANGLES : kRopeMaxPairs];
  griddep_launch_dependents();
  griddep_wait();
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t row = (int64_t)blockIdx.x * (MULTI ? a.rows_per_cta : 1);
  const int rows = MULTI ? (int)min((int64_t)a.rows_per_cta, a.rows - row) : 1;
  const int n_heads = min(a.heads_per_cta, a.q_heads + a.k_heads - (int)blockIdx.y * a.heads_per_cta);
  const RoHeads<T, MULTI> hd(a, row, (int)blockIdx.y * a.heads_per_cta, n_heads);
  const int P = a.axes * a.freqs;
  const int rot_vecs = 2 * P / V;
  const int n_rot = (rot_vecs + 1) / 2;                       // units of rotated channels
  const int upl = a.units;                                    // all units of a head
  const int at_once = RO_THREADS / upl;                       // heads the CTA handles at once
  const int u = threadIdx.x % upl, hg = threadIdx.x / upl;
  const int h_hi = hg < at_once ? rows * n_heads : 0;
  // the unit's two vectors: channel offsets and channels (0: no vector)
  int at0, at1, n0 = V, n1 = V;
  if (u < n_rot) {
    at0 = HALF ? u * V : 2 * u * V;
    at1 = HALF ? P + u * V : at0 + V;
    if (!HALF && 2 * u + 1 >= rot_vecs) n1 = 0;
  } else {
    at0 = 2 * P + 2 * (u - n_rot) * V;
    at1 = at0 + V;
    n0 = min(V, a.width - at0);
    n1 = max(0, min(V, a.width - at1));
  }
  bool angles = false;
  float c[V], s[V];
  // half: vector 0 holds the first channels of V pairs, vector 1 the second
  // ones; interleaved: each vector holds V / 2 pairs
  auto turn_of = [&](int r) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const bool have = e < V / 2 || HALF || n1 == V;
      c[e] = have ? cs[r * P + u * V + e] : 0.0f;
      s[e] = have ? sn[r * P + u * V + e] : 0.0f;
    }
  };
  int h0 = hg;
  do {
    uint4 x[RO_BATCH], y[RO_BATCH];
#pragma unroll
    for (int b = 0; b < RO_BATCH; ++b) {
      const int h = h0 + b * at_once;
      if (h < h_hi) {
        const T* p = hd.src(a, h);
        if (n0 == V && ro_in_ok(a, hd.head_of(h), p + at0, V)) x[b] = *reinterpret_cast<const uint4*>(p + at0);
        if (n1 == V && ro_in_ok(a, hd.head_of(h), p + at1, V)) y[b] = *reinterpret_cast<const uint4*>(p + at1);
      }
    }
    if (!angles) {   // (every thread comes here once, in its first pass)
      ro_angles(a, row, rows, cs, sn);
      __syncthreads();
      angles = true;
      if (!MULTI && u < n_rot) turn_of(0);
    }
#pragma unroll
    for (int b = 0; b < RO_BATCH; ++b) {
      const int h = h0 + b * at_once;
      if (h >= h_hi) break;
      T* p = hd.dst(a, h);
      if (u < n_rot) {
        if (MULTI) turn_of(hd.row_of(h));
        float v[V], w[V];
        ro_unpack<T>(x[b], v);
        ro_unpack<T>(y[b], w);
        if (HALF) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float x0 = v[e], x1 = w[e];
            v[e] = __fmaf_rn(x0, c[e], -(x1 * s[e]));
            w[e] = __fmaf_rn(x0, s[e], x1 * c[e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            const float x0 = v[2 * e], x1 = v[2 * e + 1], y0 = w[2 * e], y1 = w[2 * e + 1];
            v[2 * e] = __fmaf_rn(x0, c[e], -(x1 * s[e]));
            v[2 * e + 1] = __fmaf_rn(x0, s[e], x1 * c[e]);
            w[2 * e] = __fmaf_rn(y0, c[V / 2 + e], -(y1 * s[V / 2 + e]));
            w[2 * e + 1] = __fmaf_rn(y0, s[V / 2 + e], y1 * c[V / 2 + e]);
          }
        }
        x[b] = ro_pack<T>(v);
        y[b] = ro_pack<T>(w);
      }
      const int hn = hd.head_of(h);
      if (n0 == V && ro_out_ok(a, hn, p + at0, V)) *reinterpret_cast<uint4*>(p + at0) = x[b];
      if (n1 == V && ro_out_ok(a, hn, p + at1, V)) *reinterpret_cast<uint4*>(p + at1) = y[b];
      // the last passed-through channels of a width that is no whole vector
      const int tail = n0 < V ? n0 : (n1 < V ? n1 : 0);
      if (tail > 0 && u >= n_rot) {
        const int at = n0 < V ? at0 : at1;
        const T* q = hd.src(a, h) + at;
        if (ro_in_ok(a, hn, q, tail) && ro_out_ok(a, hn, p + at, tail))
          for (int e = 0; e < tail; ++e) p[at + e] = q[e];
      }
    }
    h0 += RO_BATCH * at_once;
  } while (h0 < h_hi);
}

// Any other head: its second channels do not begin a 16-byte vector, or a
// vector holds rotated and passed-through channels.  A CTA brings whole vectors
// of a group of heads into shared memory, turns the pairs there, and writes
// whole vectors back (in place, of a vector that is rotated only in part, the
// rotated channels alone).
template <typename T, bool HALF, bool MULTI>
__global__ void __launch_bounds__(RO_THREADS) rope_staged_kernel(const RopePosArgs a) {
  __shared__ float cs[MULTI ? RO_ANGLES : kRopeMaxPairs], sn[MULTI ? RO_ANGLES : kRopeMaxPairs];
  __shared__ __align__(16) T tile[RO_STAGE_BYTES / sizeof(T)];
  griddep_launch_dependents();
  griddep_wait();
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t row = (int64_t)blockIdx.x * (MULTI ? a.rows_per_cta : 1);
  const int rows = MULTI ? (int)min((int64_t)a.rows_per_cta, a.rows - row) : 1;
  const int n_heads = min(a.heads_per_cta, a.q_heads + a.k_heads - (int)blockIdx.y * a.heads_per_cta);
  const RoHeads<T, MULTI> hd(a, row, (int)blockIdx.y * a.heads_per_cta, n_heads);
  const int P = a.axes * a.freqs;
  const int heads = rows * n_heads;
  const int span = a.in_place ? 2 * P : a.width;               // channels that are written
  const int vecs = (span + V - 1) / V;                         // = a.units
  // a thread's vectors: (head, place) advanced by RO_THREADS without divisions
  const int adv_h = RO_THREADS / vecs, adv_v = RO_THREADS - adv_h * vecs;
  const int first_h = threadIdx.x / vecs, first_v = threadIdx.x - first_h * vecs;
  const int total = heads * vecs;
  for (int u = threadIdx.x, h = first_h, v = first_v; u < total; u += RO_THREADS) {
    const T* p = hd.src(a, h) + v * V;
    const int n = min(V, a.width - v * V);   // (the bytes past a partial vector's become 0)
    if (ro_in_ok(a, hd.head_of(h), p, n))
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(tile + u * V)), "l"(p),
                   "r"(n * (int)sizeof(T))
                   : "memory");
    h += adv_h;
    v += adv_v;
    if (v >= vecs) {
      v -= vecs;
      ++h;
    }
  }
  ro_angles(a, row, rows, cs, sn);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  // two pairs at a time (of an odd number, the last alone)
  const int twos = (P + 1) / 2, stride = vecs * V;
  const int dh = RO_THREADS / twos, dt = RO_THREADS - dh * twos;
  int h = threadIdx.x / twos, two = threadIdx.x - h * twos;
  while (h < heads) {
    const int pair = 2 * two;
    const bool both = pair + 1 < P;
    T* x = tile + h * stride + (HALF ? pair : 2 * pair);
    const int at = hd.row_of(h) * P + pair;
    const float2 c = make_float2(cs[at], both ? cs[at + 1] : 0.0f), sv = make_float2(sn[at], both ? sn[at + 1] : 0.0f);
    if (HALF) {
      T* y = x + P;
      const bool even = (P & 1) == 0;
      float2 x0, x1;
      if (both) {
        x0 = ro_get2(x);
        if (even) x1 = ro_get2(y);
        else x1 = make_float2(ro_get(y), ro_get(y + 1));
      } else {
        x0 = make_float2(ro_get(x), 0.0f);
        x1 = make_float2(ro_get(y), 0.0f);
      }
      const float2 r0 = make_float2(__fmaf_rn(x0.x, c.x, -(x1.x * sv.x)), __fmaf_rn(x0.y, c.y, -(x1.y * sv.y)));
      const float2 r1 = make_float2(__fmaf_rn(x0.x, sv.x, x1.x * c.x), __fmaf_rn(x0.y, sv.y, x1.y * c.y));
      if (both) {
        ro_put2(x, r0);
        if (even) {
          ro_put2(y, r1);
        } else {
          ro_put(y, r1.x);
          ro_put(y + 1, r1.y);
        }
      } else {
        ro_put(x, r0.x);
        ro_put(y, r1.x);
      }
    } else {
      const float2 u = ro_get2(x);
      ro_put2(x, make_float2(__fmaf_rn(u.x, c.x, -(u.y * sv.x)), __fmaf_rn(u.x, sv.x, u.y * c.x)));
      if (both) {
        const float2 w = ro_get2(x + 2);
        ro_put2(x + 2, make_float2(__fmaf_rn(w.x, c.y, -(w.y * sv.y)), __fmaf_rn(w.x, sv.y, w.y * c.y)));
      }
    }
    h += dh;
    two += dt;
    if (two >= twos) {
      two -= twos;
      ++h;
    }
  }
  __syncthreads();
  for (int u = threadIdx.x, hh = first_h, v = first_v; u < total; u += RO_THREADS) {
    T* p = hd.dst(a, hh) + v * V;
    const int n = span - v * V;
    const T* from = tile + u * V;
    if (n >= V) {
      if (ro_out_ok(a, hd.head_of(hh), p, V)) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(from);
    } else if (ro_out_ok(a, hd.head_of(hh), p, n)) {
      for (int e = 0; e < n; ++e) p[e] = from[e];
    }
    hh += adv_h;
    v += adv_v;
    if (v >= vecs) {
      v -= vecs;
      ++hh;
    }
  }
}

namespace {
template <typename T>
cudaError_t launch_rope_t(RopePosArgs& a, cudaStream_t st, bool* vec) {
  constexpr int V = 16 / (int)sizeof(T);
  const int P = a.axes * a.freqs;
  // whole 16-byte vectors: the half layout needs its second channels aligned
  // too, the interleaved one whole vectors of pairs
  *vec = a.half ? P % V == 0 : 2 * P % V == 0;
  const int pass = a.in_place ? 0 : a.width - 2 * P;
  a.units = *vec ? (2 * P / V + 1) / 2 + (pass + 2 * V - 1) / (2 * V) : (2 * P + pass + V - 1) / V;
  const int heads = a.q_heads + a.k_heads;
  // heads of one pass over a CTA's threads, or of its shared memory
  const int at_once = *vec ? RO_THREADS / a.units : RO_STAGE_BYTES / 16 / a.units;
  const long long passes = (heads + at_once - 1) / at_once;
  // of few rows, several CTAs per row: as many as fit on the GPU at once; with
  // vectors each has at least one pass, the staged form at most one
  const long long room = (long long)RO_CTAS * num_sms();
  long long split = (room + a.rows - 1) / a.rows;
  if (*vec ? split > passes : split < passes) split = passes;
  if (split > heads) split = heads;
  a.heads_per_cta = (int)((heads + split - 1) / split);
  // of many rows whose units do not fill a CTA's threads, several rows per CTA:
  // as many as fill its threads' loads or its shared memory, while every SM keeps
  // its CTAs (15,000 rows of 2 + 1 heads of 128: 11 us)
  a.rows_per_cta = 1;
  if (split == 1 && heads * a.units <= RO_THREADS) {
    long long more = (*vec ? RO_BATCH : 1) * (long long)at_once / heads;
    if (more > RO_ANGLES / P) more = RO_ANGLES / P;
    if (more > a.rows / room) more = a.rows / room;
    if (more > 1) a.rows_per_cta = (int)more;
  }
  const bool multi = a.rows_per_cta > 1;
  const dim3 grid((unsigned)((a.rows + (long long)a.rows_per_cta - 1) / a.rows_per_cta),
                  (unsigned)((heads + a.heads_per_cta - 1) / a.heads_per_cta));
  void (*kernel)(RopePosArgs);
  if (*vec)
    kernel = a.half ? (multi ? rope_kernel<T, true, true> : rope_kernel<T, true, false>)
                    : (multi ? rope_kernel<T, false, true> : rope_kernel<T, false, false>);
  else
    kernel = a.half ? (multi ? rope_staged_kernel<T, true, true> : rope_staged_kernel<T, true, false>)
                    : (multi ? rope_staged_kernel<T, false, true> : rope_staged_kernel<T, false, false>);
  return launch_kernel(kernel, grid, dim3(RO_THREADS), 0, st, a);
}
}  // namespace

cudaError_t launch_rope(RopePosArgs a, cudaStream_t st) {
  bool vec = false;
  cudaError_t e = a.fp32 ? launch_rope_t<float>(a, st, &vec) : launch_rope_t<__nv_bfloat16>(a, st, &vec);
  if (e != cudaSuccess) return e;
  set_kernel_info("rope_kernel %s %s rows=%d heads=%d pairs=%d %s heads/cta=%d rows/cta=%d", a.half ? "half" : "interleaved",
                  a.fp32 ? "fp32" : "bf16", a.rows, a.q_heads + a.k_heads, a.axes * a.freqs,
                  vec ? "vectors" : "staged", a.heads_per_cta, a.rows_per_cta);
  return cudaGetLastError();
}

}  // namespace h3
