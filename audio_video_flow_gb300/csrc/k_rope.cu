// Rotary positions on the channels of every head of q and k: the pair of
// channels of (axis a, frequency f), j = a F + f, is turned by the angle
// pos[i][a] * omega[a][f] and scaled by the magnitude.  Pairs lie half a
// rotated width apart (j, j + A F) or side by side (2j, 2j + 1); channels past
// the 2 A F rotated ones pass through.  The gradient is the turn by the
// opposite angle.
//
// Angles: omega is held as turns per position in 64-bit fixed point (2^64 = one
// turn), so that the low 64 bits of pos * omega are the angle's fraction of a
// turn, exact to 2^-33 turns for every 32-bit position (an fp32 product is
// wrong by 0.06 radians at position 10^6).  The sine and cosine are of that
// fraction, in half turns.
//
// Bound by memory: q and k are read and written once.  A CTA handles one
// packed row (of few rows: a range of its heads); it computes the row's A F
// sines and cosines once into shared memory, and each thread keeps those of
// its own 16-byte unit of a head in registers while it walks over the heads.
#include "h3_device.cuh"
#include "h3_internal.h"

namespace h3 {

namespace {
constexpr int RO_THREADS = 256;
constexpr int RO_BATCH = 4;      // heads whose loads a thread issues before their use

template <typename T>
struct Vec16 {
  static constexpr int N = 16 / (int)sizeof(T);
  float v[N];
  __device__ __forceinline__ void load(const T* p) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = bf16_lo(w[e]);
        v[2 * e + 1] = bf16_hi(w[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(w[e]);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
};
__device__ __forceinline__ float ro_get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ro_get(const float* p) { return *p; }
__device__ __forceinline__ void ro_put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void ro_put(float* p, float v) { *p = v; }
}  // namespace

// VEC: 16-byte units (half layout: a unit of first channels with its unit of
// second ones; interleaved: one unit holding whole pairs); otherwise one pair
// or one passed-through channel at a time.
template <typename T, bool HALF, bool VEC>
__global__ void __launch_bounds__(RO_THREADS) rope_kernel(const RopePosArgs a) {
  __shared__ float cs[kRopeMaxPairs], sn[kRopeMaxPairs];
  griddep_launch_dependents();
  griddep_wait();
  constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;
  const int64_t row = blockIdx.x;
  const int P = a.axes * a.freqs;
  for (int p = threadIdx.x; p < P; p += RO_THREADS) {
    const int32_t* pp = a.pos + row * a.axes + p / a.freqs;
    const int32_t pos = in_bounds<int32_t>(a.pos, a.pos_elems, pp, 1, a.err, 60) ? *pp : 0;
    const uint64_t turn = (uint64_t)(int64_t)pos * a.turns[p];
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns in [-1, 1)
    cs[p] = c * a.magnitude;
    sn[p] = s * a.sin_scale;
  }
  __syncthreads();

  // units of a head: rotated ones first, then the passed-through channels
  // (in place: none)
  const int per_rot = HALF ? V : (VEC ? V / 2 : 1);            // pairs per rotated unit
  const int n_rot = P / per_rot;
  const int pass = a.in_place ? 0 : a.width - 2 * P;
  const int upl = n_rot + (pass + V - 1) / V;
  const int at_once = RO_THREADS / upl;                         // heads the CTA handles at once
  const int u = threadIdx.x % upl, hg = threadIdx.x / upl;
  if (hg >= at_once) return;
  const int h_lo = (int)blockIdx.y * a.heads_per_cta;
  const int h_hi = min(h_lo + a.heads_per_cta, a.q_heads + a.k_heads);

  auto src = [&](int h) {
    return (h < a.q_heads ? static_cast<const T*>(a.q_in) + (int64_t)h * a.in_head
                          : static_cast<const T*>(a.k_in) + (int64_t)(h - a.q_heads) * a.in_head) +
           row * a.in_row;
  };
  auto dst = [&](int h) {
    return (h < a.q_heads ? static_cast<T*>(a.q_out) + (int64_t)h * a.out_head
                          : static_cast<T*>(a.k_out) + (int64_t)(h - a.q_heads) * a.out_head) +
           row * a.out_row;
  };
  auto in_ok = [&](int h, const T* p, int n) {
    return h < a.q_heads ? in_bounds<T>(static_cast<const T*>(a.q_in), a.q_in_elems, p, n, a.err, 61)
                         : in_bounds<T>(static_cast<const T*>(a.k_in), a.k_in_elems, p, n, a.err, 62);
  };
  auto out_ok = [&](int h, const T* p, int n) {
    return h < a.q_heads ? in_bounds<T>(static_cast<const T*>(a.q_out), a.q_out_elems, p, n, a.err, 63)
                         : in_bounds<T>(static_cast<const T*>(a.k_out), a.k_out_elems, p, n, a.err, 64);
  };

  if (u >= n_rot) {
    // passed-through channels
    const int at = 2 * P + (u - n_rot) * V;
    const int n = min(V, a.width - at);
    for (int h = h_lo + hg; h < h_hi; h += at_once) {
      const T* s = src(h) + at;
      T* d = dst(h) + at;
      if (!in_ok(h, s, n) || !out_ok(h, d, n)) continue;
      if (VEC && n == V) {
        *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(s);
      } else {
        for (int e = 0; e < n; ++e) d[e] = s[e];
      }
    }
    return;
  }

  if constexpr (VEC) {
    constexpr int NP = HALF ? V : V / 2;
    float c[NP], s[NP];
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      c[e] = cs[u * NP + e];
      s[e] = sn[u * NP + e];
    }
    const int at0 = u * V, at1 = HALF ? P + u * V : 0;
    for (int h0 = h_lo + hg; h0 < h_hi; h0 += RO_BATCH * at_once) {
      Vec16<T> x[RO_BATCH], y[HALF ? RO_BATCH : 1];
#pragma unroll
      for (int b = 0; b < RO_BATCH; ++b) {
        const int h = h0 + b * at_once;
        if (h < h_hi) {
          const T* p = src(h);
          if (in_ok(h, p + at0, V)) x[b].load(p + at0);
          if (HALF && in_ok(h, p + at1, V)) y[b].load(p + at1);
        }
      }
#pragma unroll
      for (int b = 0; b < RO_BATCH; ++b) {
        const int h = h0 + b * at_once;
        if (h >= h_hi) break;
        T* p = dst(h);
        if constexpr (HALF) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float x0 = x[b].v[e], x1 = y[b].v[e];
            x[b].v[e] = __fmaf_rn(x0, c[e], -(x1 * s[e]));
            y[b].v[e] = __fmaf_rn(x0, s[e], x1 * c[e]);
          }
          if (out_ok(h, p + at0, V)) x[b].store(p + at0);
          if (out_ok(h, p + at1, V)) y[b].store(p + at1);
        } else {
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            const float x0 = x[b].v[2 * e], x1 = x[b].v[2 * e + 1];
            x[b].v[2 * e] = __fmaf_rn(x0, c[e], -(x1 * s[e]));
            x[b].v[2 * e + 1] = __fmaf_rn(x0, s[e], x1 * c[e]);
          }
          if (out_ok(h, p + at0, V)) x[b].store(p + at0);
        }
      }
    }
  } else {
    const float c = cs[u], s = sn[u];
    const int at0 = HALF ? u : 2 * u, at1 = HALF ? P + u : 2 * u + 1;
    for (int h = h_lo + hg; h < h_hi; h += at_once) {
      const T* p = src(h);
      T* d = dst(h);
      if (!in_ok(h, p + at0, 1) || !in_ok(h, p + at1, 1) || !out_ok(h, d + at0, 1) || !out_ok(h, d + at1, 1)) continue;
      const float x0 = ro_get(p + at0), x1 = ro_get(p + at1);
      ro_put(d + at0, __fmaf_rn(x0, c, -(x1 * s)));
      ro_put(d + at1, __fmaf_rn(x0, s, x1 * c));
    }
  }
}

namespace {
template <typename T>
cudaError_t launch_rope_t(RopePosArgs& a, cudaStream_t st, bool* vec) {
  constexpr int V = 16 / (int)sizeof(T);
  const int P = a.axes * a.freqs;
  // whole 16-byte units: the half layout needs its second channels aligned
  // too, the interleaved one whole units of pairs
  *vec = a.half ? P % V == 0 : 2 * P % V == 0;
  const int units = *vec ? (a.half ? P / V : 2 * P / V) : P;
  const int pass = a.in_place ? 0 : a.width - 2 * P;
  const int at_once = RO_THREADS / (units + (*vec ? (pass + V - 1) / V : pass));
  const int heads = a.q_heads + a.k_heads;
  // of few rows, several CTAs per row: at least two per SM in all, each with
  // at least one pass over its threads
  long long split = (2LL * num_sms() + a.rows - 1) / a.rows;
  const long long most = (heads + at_once - 1) / at_once;
  if (split > most) split = most;
  a.heads_per_cta = (int)((heads + split - 1) / split);
  const dim3 grid((unsigned)a.rows, (unsigned)((heads + a.heads_per_cta - 1) / a.heads_per_cta));
  auto kernel = a.half ? (*vec ? rope_kernel<T, true, true> : rope_kernel<T, true, false>)
                       : (*vec ? rope_kernel<T, false, true> : rope_kernel<T, false, false>);
  return launch_kernel(kernel, grid, dim3(RO_THREADS), 0, st, a);
}
}  // namespace

cudaError_t launch_rope(RopePosArgs a, cudaStream_t st) {
  bool vec = false;
  cudaError_t e = a.fp32 ? launch_rope_t<float>(a, st, &vec) : launch_rope_t<__nv_bfloat16>(a, st, &vec);
  if (e != cudaSuccess) return e;
  set_kernel_info("rope_kernel %s %s rows=%d heads=%d pairs=%d vec=%dB heads/cta=%d", a.half ? "half" : "interleaved",
                  a.fp32 ? "fp32" : "bf16", a.rows, a.q_heads + a.k_heads, a.axes * a.freqs,
                  vec ? 16 : (a.fp32 ? 4 : 2), a.heads_per_cta);
  return cudaGetLastError();
}

}  // namespace h3
