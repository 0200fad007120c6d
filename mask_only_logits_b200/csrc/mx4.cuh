// mx4.cuh - microscaled 4-bit floating point (MXFP4, OCP Microscaling Formats v1.0): blocks of
// 32 consecutive elements of a row share one power-of-two scale (E8M0: byte s = 2^(s - 127),
// 0xFF = NaN), each element an E2M1 code (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives).
//
//   e    = max(floor(log2 max|x|) - 2, -127)      (2 = exponent of E2M1's largest power of two)
//   code = the E2M1 value nearest to x * 2^-e, ties to the even code, at most 6 in size
// A block that holds a NaN or an infinity gets scale 0xFF: all of it stands for NaN.  All steps
// before the rounding to E2M1 are exact in fp32.
//
// Storage of an [R, K] matrix (K a multiple of 32):
//   codes   [R, K/2] bytes, row-major, element 2i in the low nibble of byte i
//   scales  in tiles of 128 rows x 4 blocks (512 bytes), the order in which the tensor cores'
//           scale memory takes them: tile (r / 128, k / 128) at ((r/128) * ceil(K/128) + k/128)
//           * 512, in it byte (r % 32) * 16 + ((r / 32) % 4) * 4 + (k / 32) % 4.  Rows and
//           blocks past the matrix hold 0.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace dllm {
namespace mx4 {

constexpr int kThreads = 256;

__host__ __device__ inline long long scale_bytes(long long rows, int cols) {
  return (rows + 127) / 128 * ((cols + 127) / 128) * 512;
}

// Index (in 32-bit words, one per 4 blocks of a row) of row r, 128-column group g.
__device__ __forceinline__ long long scale_word(long long r, int g, int groups) {
  return ((r >> 7) * groups + g) * 128 + (r & 31) * 4 + ((r >> 5) & 3);
}

// Two fp32 values to E2M1 codes (round to nearest even, saturating): lo in the low nibble.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint16_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
      "cvt.u16.u8 %0, b;\n\t}"
      : "=h"(r)
      : "f"(lo), "f"(hi));
  return r;
}

// One block: 32 values to 16 bytes of codes and the scale byte.
__device__ __forceinline__ uint32_t quantize_block(const float (&x)[32], uint32_t (&q)[4]) {
  uint32_t top = 0;                                    // |x| compares as its bit pattern
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
    top = b > top ? b : top;
  }
  if (top >= 0x7f800000u) {                            // infinity or NaN
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = 0;
    return 0xffu;
  }
  int e = static_cast<int>(top >> 23) - 129;
  e = e < -127 ? -127 : e;
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    q[w] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[w] |= e2m1x2(x[8 * w + 2 * i] * inv, x[8 * w + 2 * i + 1] * inv) << (8 * i);
  }
  return static_cast<uint32_t>(e + 127);
}

__device__ __forceinline__ void load_block(const __nv_bfloat16* p, float (&x)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void load_block(const __half* p, float (&x)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 h = *reinterpret_cast<const __half2*>(&w[j]);
      x[8 * i + 2 * j] = __low2float(h);
      x[8 * i + 2 * j + 1] = __high2float(h);
    }
  }
}
__device__ __forceinline__ void load_block(const float* p, float (&x)[32]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
    x[4 * i] = v.x;
    x[4 * i + 1] = v.y;
    x[4 * i + 2] = v.z;
    x[4 * i + 3] = v.w;
  }
}

// Quantise block `blk` (of 4 * groups, those past K / 32 empty) of a row into codes row r and
// scale row r; the four lanes of a 128-column group write their scale bytes as one word.
// src: the row's first element, null for a row past the matrix (scales 0, no codes).
template <typename T>
__device__ __forceinline__ void quantize_to(const T* src, int blk, int K, int groups, long long r,
                                            uint8_t* __restrict__ q, uint32_t* __restrict__ s) {
  uint32_t scale = 0;
  if (src != nullptr && blk * 32 < K) {
    float x[32];
    uint32_t c[4];
    load_block(src + blk * 32, x);
    scale = quantize_block(x, c);
    *reinterpret_cast<uint4*>(q + r * (K / 2) + blk * 16) = make_uint4(c[0], c[1], c[2], c[3]);
  }
  const unsigned quad = 0xfu << (threadIdx.x & 28);    // the four lanes of this group
  scale <<= 8 * (threadIdx.x & 3);
  scale |= __shfl_xor_sync(quad, scale, 1);
  scale |= __shfl_xor_sync(quad, scale, 2);
  if ((threadIdx.x & 3) == 0) s[scale_word(r, blk >> 2, groups)] = scale;
}

// X [rows, K] (row stride ld elements) to MXFP4: one thread per block of 32.
template <typename T>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const T* __restrict__ X, long long rows, int K, long long ld, uint8_t* __restrict__ q,
                uint32_t* __restrict__ s) {
  pdl_wait();
  pdl_launch_dependents();
  const int groups = (K + 127) / 128, per_row = groups * 4;
  const long long total = (rows + 127) / 128 * 128 * per_row;      // a multiple of 4
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const long long r = i / per_row;
    const int blk = static_cast<int>(i - r * per_row);
    quantize_to(r < rows ? X + r * ld : static_cast<const T*>(nullptr), blk, K, groups, r, q, s);
  }
}

// The masked rows H[row_idx[r]] (r < count) to MXFP4 rows r of q and s, and n_zero ints at
// `zero` cleared: gather_rows_kernel (compact.cuh) with the quantisation in the copy.
__global__ void __launch_bounds__(kThreads)
gather_quantize_kernel(const uint16_t* __restrict__ H, const int* __restrict__ row_idx,
                       const int* __restrict__ count, long long n_pos, long long n_cap, int d,
                       uint8_t* __restrict__ q, uint32_t* __restrict__ s, int* __restrict__ zero,
                       int n_zero, int* __restrict__ status) {
  pdl_wait();
  pdl_launch_dependents();
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < n_zero; i += gridDim.x * kThreads) zero[i] = 0;
  int n = *count;
  if (n < 0 || n > n_pos) {                          // cannot happen: bad compaction
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(status, kStatusBounds);
    n = 0;
  } else if (n > n_cap) {                            // workspace sized for fewer rows
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(status, kStatusCapacity);
    n = static_cast<int>(n_cap);
  }
  const int groups = (d + 127) / 128, per_row = groups * 4;
  const long long total = static_cast<long long>(n) * per_row;
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const long long r = i / per_row;
    const int blk = static_cast<int>(i - r * per_row);
    const int p = row_idx[r];
    const bool bad = p < 0 || p >= n_pos;
    if (bad && blk == 0) atomicOr(status, kStatusBounds);
    quantize_to(bad ? static_cast<const __nv_bfloat16*>(nullptr)
                    : reinterpret_cast<const __nv_bfloat16*>(H) + static_cast<size_t>(p) * d,
                blk, d, groups, r, q, s);
  }
}

// The value of an E2M1 code (4 bits).
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t mag = c & 7u;
  // 0 and .5, then 1 + mantissa / 2 scaled by 2^(exponent - 1)
  const float v = mag < 2u ? 0.5f * static_cast<float>(mag)
                           : __uint_as_float(((mag >> 1) + 126u) << 23 | (mag & 1u) << 22);
  return (c & 8u) ? -v : v;
}

// 2^(s - 127), NaN for 0xFF (2^-127 is subnormal).
__device__ __forceinline__ float e8m0_value(uint32_t s) {
  return s == 0xffu ? __uint_as_float(0x7fc00000u) : s == 0u ? __uint_as_float(0x00400000u)
                                                             : __uint_as_float(s << 23);
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {     // exact: two significant bits, bf16 has fp32's exponents
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// The values an MXFP4 matrix stands for (bf16 or fp32: both exact): one thread per 8 elements.
template <typename T>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, long long rows, int K,
                  T* __restrict__ X, long long ld) {
  pdl_wait();
  pdl_launch_dependents();
  const int groups = (K + 127) / 128, per_row = K / 8;
  const long long total = rows * per_row;
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const long long r = i / per_row;
    const int c8 = static_cast<int>(i - r * per_row);
    const uint32_t codes = __ldg(reinterpret_cast<const uint32_t*>(q) + i);
    const int blk = c8 >> 2;
    const float scale = e8m0_value(__ldg(s + 4 * scale_word(r, blk >> 2, groups) + (blk & 3)));
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e2m1_value((codes >> (4 * j)) & 15u) * scale;
    store8(X + r * ld + c8 * 8, v);
  }
}

}  // namespace mx4
}  // namespace dllm
