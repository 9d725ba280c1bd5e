// Product of a few rows with 4-bit weights and group scales.
//
//   y[n][o] = x_scale[n] sum_k x[n][k] scale[o][k / group] (code[o][k] - 8)
//
// Weights are read once per 32 rows of x, which bounds the product for the few
// rows of a decode step: O K / 2 bytes and 2 O K / group bytes of scales. Measured
// (K = 2048): 50257 outputs, eight e4m3 rows, groups of 64: 17.4 us, 3.2 TB/s; 6144
// outputs, one bf16 row: 3.8 us a call in a graph. The wide product is half as fast as
// its bytes: a warp executes 21 instructions for each word of eight codes, of which 9
// turn the codes into numbers and 12 are the inputs (fetched and converted again by every
// CTA), two-byte scales, products and addresses, and no loads of the next block are in
// flight while a block is multiplied.
//
// Layout. Tiles of 16 outputs x 128 inputs, 1024 bytes each, so that a warp
// reads a tile as two coalesced 16-byte loads per lane and finds in its registers
// the operand of m16n8k16 matrix instructions: lane (g, t) = (lane / 4, lane % 4)
// holds 32 bytes, for the outputs g and g + 8 four 4-byte words j = 0..3, word j
// with the inputs 32 j + 8 t .. + 7, lowest nibble first. Every group of 32 or more
// inputs is then a run of whole words of all four lanes t, so each group's products
// can be summed by themselves and scaled once. Scales (bf16): [tile][block of 128
// inputs][group in the block][16 outputs]. Outputs past O hold code 8 and scale 0.
//
// Codes become numbers exactly (128 + code is the bf16 pattern 0x4300 | code, 1024 +
// code the fp16 pattern 0x6400 | code). Products of bf16 rows are bf16, of e4m3 rows
// fp16 (both exact, and one instruction converts a pair of e4m3 numbers), and fp32
// rows are cut into three bf16 parts whose sum has all 24 bits. The matrix instruction
// (mma.sync: eight columns are enough, and the weights come out of registers, not
// shared memory) accumulates in fp32 within a group; the scaled sums are fp32.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace muir {

struct W4Params {
  const void* x;
  const float* x_scale;
  const uint8_t* wq;
  const __nv_bfloat16* ws;
  void* y;
  int64_t n;
  int K, O;
};

// d = a b + (FIRST ? 0 : d)
template <bool HALF, bool FIRST>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
#define MUIR_MMA(TYPE)                                                                                                   \
  if constexpr (FIRST)                                                                                                   \
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32." TYPE "." TYPE                                                  \
                 ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"                                        \
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])                                                        \
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));                              \
  else                                                                                                                   \
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32." TYPE "." TYPE                                                  \
                 ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"                                            \
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                                        \
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1))
  if constexpr (HALF) {
    MUIR_MMA("f16");
  } else {
    MUIR_MMA("bf16");
  }
#undef MUIR_MMA
}

// The eight nibbles of a word as four pairs (nibbles i and i + 4) of numbers
// (code - 8) 2^-10, exactly: the code beside a constant's exponent, less 8 and the
// constant. A group's sum of up to 128 products then stays below its largest input,
// so that no input overflows before its scale is applied. fp16 has room for a code
// in bits 4 .. 7 as well (1024 + 16 code), which saves two of three shifts.
constexpr float kW4Up = 1024.f;
template <bool HALF>
__device__ __forceinline__ void w4_pairs(uint32_t w, uint32_t (&o)[4]) {
  if constexpr (HALF) {
    const auto number = [](uint32_t u, uint32_t m, uint32_t c) {
      const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&m),
                                *reinterpret_cast<const __half2*>(&c));
      return *reinterpret_cast<const uint32_t*>(&r);
    };
    const uint32_t v = w >> 8;
    o[0] = number((w & 0x000F000Fu) | 0x64006400u, 0x14001400u, 0xBC08BC08u);  // 2^-10, -1032 2^-10
    o[1] = number((w & 0x00F000F0u) | 0x64006400u, 0x04000400u, 0xAC80AC80u);  // 2^-14, -(1024 + 128) 2^-14
    o[2] = number((v & 0x000F000Fu) | 0x64006400u, 0x14001400u, 0xBC08BC08u);
    o[3] = number((v & 0x00F000F0u) | 0x64006400u, 0x04000400u, 0xAC80AC80u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
      const uint32_t m = 0x3A803A80u, c = 0xBE08BE08u;  // 2^-10, -136 2^-10
      const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                       *reinterpret_cast<const __nv_bfloat162*>(&m),
                                       *reinterpret_cast<const __nv_bfloat162*>(&c));
      o[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
}

// 8 consecutive inputs of one row as matrix operands: part p, pairs (0,4), (1,5), (2,6), (3,7).
template <typename X> struct W4X;
template <> struct W4X<__nv_bfloat16> {
  static constexpr int PARTS = 1;
  static constexpr bool HALF = false;
  static __device__ __forceinline__ void get(const __nv_bfloat16* p, uint32_t (&o)[1][4]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    o[0][0] = __byte_perm(u.x, u.z, 0x5410);
    o[0][1] = __byte_perm(u.x, u.z, 0x7632);
    o[0][2] = __byte_perm(u.y, u.w, 0x5410);
    o[0][3] = __byte_perm(u.y, u.w, 0x7632);
  }
};
template <> struct W4X<__nv_fp8_e4m3> {
  static constexpr int PARTS = 1;
  static constexpr bool HALF = true;
  static __device__ __forceinline__ void get(const __nv_fp8_e4m3* p, uint32_t (&o)[1][4]) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // elements i (of u.x) and i + 4 (of u.y)
      const uint32_t two = __byte_perm(u.x, u.y, i | ((i + 4) << 4));
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
      o[0][i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};
template <> struct W4X<float> {
  static constexpr int PARTS = 3;
  static constexpr bool HALF = false;
  static __device__ __forceinline__ void get(const float* p, uint32_t (&o)[3][4]) {
    float f[8];
    Elt<float>::ld8(p, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = f[i], b = f[i + 4];
#pragma unroll
      for (int m = 0; m < 3; ++m) {  // the upper 16 bits, exactly; an infinity has no remainder
        o[m][i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
        a = isinf(a) ? 0.f : a - __uint_as_float(__float_as_uint(a) & 0xFFFF0000u);
        b = isinf(b) ? 0.f : b - __uint_as_float(__float_as_uint(b) & 0xFFFF0000u);
      }
    }
  }
};

constexpr int kW4Warps = 4;

// One CTA per RT tiles of 16 outputs and 8 NB rows of x; the warps share the inputs,
// so each piece of x is fetched and converted once per RT tiles. GPB: groups per
// block of 128 inputs (1, 2 or 4).
template <typename X, typename Y, int NB, int GPB, int RT>
__global__ void __launch_bounds__(32 * kW4Warps, NB == 1 ? 6 : 3) w4_matvec_kernel(W4Params p) {
  using XL = W4X<X>;
  __shared__ float red[kW4Warps][NB][32][4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int blocks = p.K >> 7;
  const int64_t tiles = (p.O + 15) >> 4, tile0 = (int64_t)blockIdx.x * RT;
  const int64_t n0 = (int64_t)blockIdx.y * (8 * NB);
  const X* x = static_cast<const X*>(p.x);
  float acc[RT][NB][4];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[rt][b][i] = 0.f;
  // this lane's first weights, scales and inputs; a block of inputs further on each turn
  const uint4* wt[RT];
  const __nv_bfloat16* st[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    // tiles past the last repeat it; their sums are not stored
    const int64_t at = (tile0 + rt < tiles ? tile0 + rt : tiles - 1) * blocks + warp;
    wt[rt] = reinterpret_cast<const uint4*>(p.wq + at * 1024) + lane * 2;
    st[rt] = p.ws + at * (GPB * 16) + g;
  }
  const X* xt[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    // rows past the last repeat it; their results are not stored
    const int64_t r = n0 + 8 * b + g < p.n ? n0 + 8 * b + g : p.n - 1;
    xt[b] = x + r * p.K + warp * 128 + 8 * t;
  }
  for (int kb = warp; kb < blocks; kb += kW4Warps) {
    uint4 w[RT][2];
    __nv_bfloat16 sc[RT][GPB][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      w[rt][0] = __ldg(wt[rt]);
      w[rt][1] = __ldg(wt[rt] + 1);
      wt[rt] += 64 * kW4Warps;
#pragma unroll
      for (int gr = 0; gr < GPB; ++gr) {
        sc[rt][gr][0] = __ldg(st[rt] + gr * 16);
        sc[rt][gr][1] = __ldg(st[rt] + gr * 16 + 8);
      }
      st[rt] += GPB * 16 * kW4Warps;
    }
#pragma unroll
    for (int gr = 0; gr < GPB; ++gr) {
      float part[RT][NB][4];
#pragma unroll
      for (int jj = 0; jj < 4 / GPB; ++jj) {
        const int j = gr * (4 / GPB) + jj;
        uint32_t xb[NB][XL::PARTS][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) XL::get(xt[b] + 32 * j, xb[b]);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const uint32_t u0 = reinterpret_cast<const uint32_t*>(&w[rt][0])[j], u1 = reinterpret_cast<const uint32_t*>(&w[rt][1])[j];
          uint32_t n0[4], n1[4];
          w4_pairs<XL::HALF>(u0, n0);
          w4_pairs<XL::HALF>(u1, n1);
          const uint32_t a0[4] = {n0[0], n1[0], n0[1], n1[1]}, a1[4] = {n0[2], n1[2], n0[3], n1[3]};
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int m = 0; m < XL::PARTS; ++m) {
              if (jj == 0 && m == 0) mma_16816<XL::HALF, true>(part[rt][b], a0, xb[b][m][0], xb[b][m][1]);
              else mma_16816<XL::HALF, false>(part[rt][b], a0, xb[b][m][0], xb[b][m][1]);
              mma_16816<XL::HALF, false>(part[rt][b], a1, xb[b][m][2], xb[b][m][3]);
            }
        }
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float s0 = __bfloat162float(sc[rt][gr][0]), s1 = __bfloat162float(sc[rt][gr][1]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          acc[rt][b][0] = fmaf(s0, part[rt][b][0], acc[rt][b][0]);
          acc[rt][b][1] = fmaf(s0, part[rt][b][1], acc[rt][b][1]);
          acc[rt][b][2] = fmaf(s1, part[rt][b][2], acc[rt][b][2]);
          acc[rt][b][3] = fmaf(s1, part[rt][b][3], acc[rt][b][3]);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) xt[b] += 128 * kW4Warps;
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if (rt > 0) __syncthreads();
#pragma unroll
    for (int b = 0; b < NB; ++b)
      *reinterpret_cast<float4*>(red[warp][b][lane]) = make_float4(acc[rt][b][0], acc[rt][b][1], acc[rt][b][2], acc[rt][b][3]);
    __syncthreads();
    // 16 outputs x 8 NB rows; output o of row r is element (o / 8) * 2 + r % 2 of lane (o % 8) * 4 + (r % 8) / 2
    for (int i = threadIdx.x; i < 128 * NB; i += 32 * kW4Warps) {
      const int o = i & 15, r = i >> 4;
      const int l = (o & 7) * 4 + ((r & 7) >> 1), e = (o >> 3) * 2 + (r & 1);
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kW4Warps; ++k) s += red[k][r >> 3][l][e];
      s *= kW4Up;
      const int64_t row = n0 + r, col = (tile0 + rt) * 16 + o;
      if (row < p.n && col < p.O) {
        if (p.x_scale) s *= __ldg(p.x_scale + row);
        Elt<Y>::st(static_cast<Y*>(p.y) + row * p.O + col, s);
      }
    }
  }
}

// ---- laying the weights out -----------------------------------------------------

// Codes [O][K] (0..15; only the low four bits count) and scales [O][K / group] into
// the layout above: one thread per 4-byte word and per scale.
__global__ void __launch_bounds__(256) w4_pack_kernel(const uint8_t* __restrict__ codes, const __nv_bfloat16* __restrict__ scales,
                                                      uint32_t* __restrict__ wq, __nv_bfloat16* __restrict__ ws, int K, int O,
                                                      int gpb, int64_t words, int64_t nscales) {
  const int blocks = K >> 7;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < words + nscales; i += gridDim.x * 256ll) {
    if (i < words) {
      const int j = (int)(i & 3), half = (int)(i >> 2) & 1, t = (int)(i >> 3) & 3, g = (int)(i >> 5) & 7;
      const int64_t kb = (i >> 8) % blocks, o = (i >> 8) / blocks * 16 + half * 8 + g;
      uint32_t w = 0x88888888u;
      if (o < O) {
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(codes + o * K + kb * 128 + 32 * j + 8 * t));
        w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w |= ((c.x >> (8 * e)) & 15u) << (4 * e);
          w |= ((c.y >> (8 * e)) & 15u) << (4 * e + 16);
        }
      }
      wq[i] = w;
    } else {
      const int64_t s = i - words;
      const int o16 = (int)(s & 15), gr = (int)((s >> 4) % gpb);
      const int64_t kb = (s >> 4) / gpb % blocks, o = (s >> 4) / gpb / blocks * 16 + o16;
      ws[s] = o < O ? scales[o * blocks * gpb + kb * gpb + gr] : __float2bfloat16_rn(0.f);
    }
  }
}

// Weights [O][K] to codes and scales: scale = bf16(max |w| / 7) of each group and
// code = 8 + w / scale rounded to the nearest, held to 0..15; a group of zeros has
// scale 0 and codes 8. One warp per output and group.
template <typename T>
__global__ void __launch_bounds__(256) w4_quantize_kernel(const T* __restrict__ w, uint8_t* __restrict__ codes,
                                                          __nv_bfloat16* __restrict__ scales, int64_t groups, int group) {
  const int lane = threadIdx.x & 31;
  for (int64_t i = blockIdx.x * 8ll + (threadIdx.x >> 5); i < groups; i += gridDim.x * 8ll) {
    const T* src = w + i * group;
    float top = 0.f;
    for (int e = lane; e < group; e += 32) top = fmaxf(top, fabsf(Elt<T>::ld(src + e)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const __nv_bfloat16 s = __float2bfloat16_rn(top / 7.f);
    const float sf = __bfloat162float(s);
    if (lane == 0) scales[i] = s;
    for (int e = lane; e < group; e += 32) {
      const float q = sf > 0.f ? rintf(Elt<T>::ld(src + e) / sf) : 0.f;
      codes[i * group + e] = (uint8_t)(8 + (int)fminf(fmaxf(q, -8.f), 7.f));
    }
  }
}

}  // namespace muir
