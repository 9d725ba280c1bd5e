// Root-mean-square norm of token rows, with the residual's addition.
//
//   h = x + residual                         (h = x without a residual)
//   rstd = (mean_d h_d^2 + eps)^(-1/2)       (0 for a row of zeros without an eps)
//   y_d = h_d rstd weight_d
//
// y in the input's type, or in 8 bits: with top = max_d |y_d|, scale = top / 448
// (448 is e4m3's largest number) and q_d = e4m3(y_d 448 / top), so that
// q_d scale ~ y_d; a row of zeros has scale 0 and codes 0. The norm is taken of
// the fp32 sum; the residual stream h that is written out is rounded once, to the
// input's type. Statistics are fp32; rows whose squares leave fp32's range are scaled by
// a power of two first.
//
// Backward, with xh = h rstd and g = dy weight:
//   dx_d = rstd (g_d - xh_d mean_d(g xh)) + dh_d      dweight_d = sum_rows dy_d xh_d
// dx is the gradient of x and of the residual alike; dh is the cotangent of the
// written residual stream.
//
// Memory bound: every row is read once, kept in registers across its reduction
// and written once. Rows up to 1024 wide take a warp each (eight rows per CTA, no
// barrier); wider rows take one CTA. Measured: 32768 x 2048 bf16 with the residual
// 83 us (6.5 TB/s, the copy rate), to 8 bits of 131072 x 512 73 us; backward of 8191 x 2048
// bf16 28 us and 4 us for the column sums (4.2 TB/s together; 42 us before the next row's
// loads were issued ahead of a row's reduction).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace muir {

struct NormParams {
  const void *x, *residual;
  const float* weight;
  void *y, *h;
  uint8_t* q;
  float *scale, *rstd;
  int64_t n;
  int d;
  float eps;
};

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// The reductions of one row over its NT threads: a warp, or a CTA of NT threads
// (slot: shared array of 32 floats per call, so that one barrier is enough).
template <int NT>
__device__ __forceinline__ float row_sum(float x, float* slot) {
  x = warp_sum(x);
  if constexpr (NT > 32) {
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = x;
    __syncthreads();
    x = warp_sum((threadIdx.x & 31) < NT / 32 ? slot[threadIdx.x & 31] : 0.f);
  }
  return x;
}
template <int NT>
__device__ __forceinline__ float row_max(float x, float* slot) {
  x = warp_max_nan(x);
  if constexpr (NT > 32) {
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = x;
    __syncthreads();
    x = warp_max_nan((threadIdx.x & 31) < NT / 32 ? slot[threadIdx.x & 31] : 0.f);
  }
  return x;
}

// NT threads per row, V pieces of 8 elements per thread: piece (v, thread) holds
// elements 8 (v NT + thread) .. + 7, absent past d. (Two CTAs asked for where 32 floats
// a thread otherwise spill for a third one: 32768 x 1024 fp32, 85 us against 89; elsewhere the compiler's choice.)
template <typename T, int NT, int V, bool QUANT>
__global__ void __launch_bounds__(NT > 32 ? NT : 256, NT == 32 && V == 4 && sizeof(T) == 4 ? 2 : 0) rms_norm_kernel(NormParams p) {
  __shared__ float slot[3][32];  // sums, the largest y, the largest x: a reduction's slot is only written behind a later one's barrier
  constexpr int ROWS = NT > 32 ? 1 : 8;
  const int lane = NT > 32 ? threadIdx.x : threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * ROWS + (NT > 32 ? 0 : threadIdx.x >> 5);
  if (row >= p.n) return;  // whole warps (NT = 32) or no one
  const int64_t off = row * p.d;
  // every load of the row first: a store of h in between would hold back those after it
  Pack8<T> px[V], pr[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = (v * NT + lane) * 8;
    if (e < p.d) {
      px[v].ld(static_cast<const T*>(p.x) + off + e);
      if (p.residual) pr[v].ld(static_cast<const T*>(p.residual) + off + e);
    }
  }
  float x[V][8];
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = (v * NT + lane) * 8;
    if (e < p.d) {
      px[v].get(x[v]);
      if (p.residual) {
        float r[8];
        pr[v].get(r);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] += r[i];
        Elt<T>::st8(static_cast<T*>(p.h) + off + e, x[v]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[v][i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[v][i], x[v][i], ss);
  }
  ss = row_sum<NT>(ss, slot[0]);
  float ms = ss / (float)p.d + p.eps, up = 1.f;
  if (isinf(ss) || (ss < 0x1p-86f && p.eps < 0x1p-100f)) {
    // squares outside fp32's range (the whole row comes here or no thread of it): once
    // more with the row brought near 1 by a power of two. eps counts for the size as well,
    // so that neither term overflows. An infinity in the row stays one.
    float big = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(x[v][i]));
    big = row_max<NT>(big, slot[2]);
    if (!isinf(big)) {
      // exponents by their bits (0 for zeros and subnormal numbers), of eps that of its root
      const int e = (int)(__float_as_uint(big) >> 23), er = p.eps > 0.f ? ((int)(__float_as_uint(p.eps) >> 23) + 127) >> 1 : 0;
      up = __uint_as_float((uint32_t)(254 - max(1, min(253, max(e, er)))) << 23);
      ss = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[v][i] *= up;
          ss = fmaf(x[v][i], x[v][i], ss);
        }
      ms = row_sum<NT>(ss, slot[0]) / (float)p.d + p.eps * up * up;
    }
  }
  const float rs = ms == 0.f ? 0.f : 1.f / sqrtf(ms);  // rstd = rs up; y = x rs w, x being up times the row's
  if (lane == 0 && p.rstd) p.rstd[row] = rs * up;
  float top = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = (v * NT + lane) * 8;
    if (e < p.d) {
      float w[8];
      Elt<float>::ld8(p.weight + e, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[v][i] = x[v][i] * rs * w[i];
        top = max_nan(top, fabsf(x[v][i]));
      }
      if constexpr (!QUANT) Elt<T>::st8(static_cast<T*>(p.y) + off + e, x[v]);
    }
  }
  if constexpr (QUANT) {
    top = row_max<NT>(top, slot[1]);
    if (lane == 0) p.scale[row] = top / 448.f;
    // 448 / top overflows below 1.4e-36: such a row is brought up by 2^100 first
    const float up = top < 1e-30f ? 0x1p100f : 1.f;
    const float inv = top == 0.f ? 0.f : 448.f / (top * up);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = (v * NT + lane) * 8;
      if (e < p.d) {
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float s[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] = x[v][4 * k + i] * up * inv;
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(s[0], s[1]), __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(s[2], s[3]), __NV_SATFINITE, __NV_E4M3);
          w[k] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2*>(p.q + off + e) = make_uint2(w[0], w[1]);
      }
    }
  }
}

struct NormBwdParams {
  const void *dy, *h, *dh;
  const float *weight, *rstd;
  void* dx;
  float *dweight, *part;  // part: [gridDim.x][d]
  int64_t n;
  int d;
};

// Each CTA walks rows blockIdx.x, + gridDim.x, .. and keeps its threads' share of
// dweight in registers; the partial sums go to the workspace and are added in a
// fixed order by rms_norm_dw_kernel, so that a repeated call gives the same bits.
template <typename T, int NT, int V>
__global__ void __launch_bounds__(NT, NT <= 512 ? 1024 / NT : 1) rms_norm_bwd_kernel(NormBwdParams p) {
  __shared__ float slot[2][32];
  const int lane = threadIdx.x;
  float dw[V][8], w[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = (v * NT + lane) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) { dw[v][i] = 0.f; w[v][i] = 0.f; }
    if (e < p.d) Elt<float>::ld8(p.weight + e, w[v]);
  }
  // the next row is on its way while this one is reduced
  Pack8<T> nh[V], ng[V], nr[V];
  float nrstd = 0.f;
  auto fetch = [&](int64_t row) {
    if (row >= p.n) return;
    nrstd = __ldg(p.rstd + row);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = (v * NT + lane) * 8;
      if (e < p.d) {
        nh[v].ld(static_cast<const T*>(p.h) + row * p.d + e);
        ng[v].ld(static_cast<const T*>(p.dy) + row * p.d + e);
        if (p.dh) nr[v].ld(static_cast<const T*>(p.dh) + row * p.d + e);
      }
    }
  };
  fetch(blockIdx.x);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.n; row += gridDim.x, turn ^= 1) {
    const int64_t off = row * p.d;
    const float rstd = nrstd;
    float xh[V][8], g[V][8];
    Pack8<T> r[V];
    float dot = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = (v * NT + lane) * 8;
      if (e < p.d) {
        nh[v].get(xh[v]);
        ng[v].get(g[v]);
        r[v] = nr[v];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xh[v][i] *= rstd;
          dw[v][i] = fmaf(g[v][i], xh[v][i], dw[v][i]);
          g[v][i] *= w[v][i];
          dot = fmaf(g[v][i], xh[v][i], dot);
        }
      }
    }
    fetch(row + gridDim.x);
    dot = row_sum<NT>(dot, slot[turn]) / (float)p.d;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = (v * NT + lane) * 8;
      if (e < p.d) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = rstd * fmaf(-xh[v][i], dot, g[v][i]);
        if (p.dh) {
          float x[8];
          r[v].get(x);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += x[i];
        }
        Elt<T>::st8(static_cast<T*>(p.dx) + off + e, o);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = (v * NT + lane) * 8;
    if (e < p.d) Elt<float>::st8(p.part + (int64_t)blockIdx.x * p.d + e, dw[v]);
  }
}

// dweight = the column sums of part [m][d]: 32 columns per CTA, 32 x 32 threads, each
// thread's rows and then the threads' sums in a fixed order.
__global__ void __launch_bounds__(1024) rms_norm_dw_kernel(const float* __restrict__ part, float* __restrict__ dweight, int m,
                                                           int d) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  float a = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int i = r; i < m; i += 32) a += part[(int64_t)i * d + c];
  }
  s[threadIdx.x & 31][r] = a;
  __syncthreads();
  a = warp_sum(s[r][threadIdx.x & 31]);  // warp r: column r of the CTA
  if ((threadIdx.x & 31) == 0 && blockIdx.x * 32 + r < (unsigned)d) dweight[blockIdx.x * 32 + r] = a;
}

}  // namespace muir
