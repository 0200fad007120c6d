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
constexpr int kGridPerSm = 64;          // quantize / dequantize: CTAs per SM, a warp per row

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

// Eight neighbouring elements of a row, and what the quantisation asks of them: the bit pattern
// of their largest size as fp32 (sizes compare as their bit patterns, two 16-bit ones at a time;
// infinity and NaN come out as the largest), and their values.
struct Eight16 {
  uint4 v;
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ uint32_t top16() const {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t t = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
    return max(t & 0xffffu, t >> 16);
  }
};
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> : Eight16 {
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ uint32_t top() const { return top16() << 16; }
  __device__ __forceinline__ float2 pair(int i) const {
    const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
};
template <> struct Eight<__half> : Eight16 {
  __device__ __forceinline__ void load(const __half* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ uint32_t top() const {
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top16())))) & 0x7fffffffu;
  }
  __device__ __forceinline__ float2 pair(int i) const {
    const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
};
template <> struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ uint32_t top() const {
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(x[i]) & 0x7fffffffu);
    return t;
  }
  __device__ __forceinline__ float2 pair(int i) const {
    return i == 0 ? make_float2(a.x, a.y) : i == 1 ? make_float2(a.z, a.w)
         : i == 2 ? make_float2(b.x, b.y) : make_float2(b.z, b.w);
  }
};

// A warp's piece of a row: kPiece elements in kSteps steps of 256, eight neighbouring elements
// per lane (16 bytes of bf16, so that a warp's loads and stores are whole lines) and a block in
// four lanes.  All loads are issued before the first is used.
constexpr int kSteps = 4;
constexpr int kPiece = 256 * kSteps;

// Quantise columns k0 .. k0 + kPiece - 1 of a row (src: its first element, null for a row past
// the matrix: scales 0, no codes) into codes row r and scale row r.  Called by whole warps.
template <typename T>
__device__ __forceinline__ void quantize_piece(const T* src, int k0, int K, int groups, long long r,
                                               uint8_t* __restrict__ q, uint32_t* __restrict__ s) {
  const int lane = threadIdx.x & 31;
  Eight<T> x[kSteps];
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const int k = k0 + 256 * j + 8 * lane;
    if (src != nullptr && k < K) x[j].load(src + k);
    else x[j].zero();
  }
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    if (k0 + 256 * j >= groups * 128) break;           // uniform: nothing of the row is left
    const int k = k0 + 256 * j + 8 * lane;
    uint32_t top = x[j].top();
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const bool bad = top >= 0x7f800000u;               // infinity or NaN in the block
    const int e = max(static_cast<int>(top >> 23) - 129, -127);
    const float inv = bad ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = x[j].pair(i);
      codes |= e2m1x2(y.x * inv, y.y * inv) << (8 * i);
    }
    const bool here = src != nullptr && k < K;
    if (here) *reinterpret_cast<uint32_t*>(q + r * (K / 2) + k / 2) = bad ? 0u : codes;
    // the scale bytes of four blocks (16 lanes) as one word
    uint32_t w = here ? (bad ? 0xffu : static_cast<uint32_t>(e + 127)) << (8 * ((lane >> 2) & 3)) : 0u;
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    w |= __shfl_xor_sync(0xffffffffu, w, 8);
    const int g = (k0 >> 7) + 2 * j + (lane >> 4);
    if ((lane & 15) == 0 && g < groups) s[scale_word(r, g, groups)] = w;
  }
}

// X [rows, K] (row stride ld elements) to MXFP4: a warp per row, piece by piece.  Bound by HBM:
// 2.53 bytes move per bf16 element (126464 x 4096: 211 us, 6.2 TB/s).  kGridPerSm CTAs per SM: a
// grid of the 4 to 8 that are resident at once, each with many rows, took 12% longer.
template <typename T>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const T* __restrict__ X, long long rows, int K, long long ld, uint8_t* __restrict__ q,
                uint32_t* __restrict__ s) {
  pdl_wait();
  pdl_launch_dependents();
  const int groups = (K + 127) / 128;
  const long long padded = (rows + 127) / 128 * 128;
  const long long warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
  for (long long r = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < padded; r += warps)
    for (int k0 = 0; k0 < groups * 128; k0 += kPiece)
      quantize_piece(r < rows ? X + r * ld : static_cast<const T*>(nullptr), k0, K, groups, r, q, s);
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
  // pieces of a row go to neighbouring warps, so that few rows still spread over the SMs
  const int groups = (d + 127) / 128, pieces = (groups * 128 + kPiece - 1) / kPiece;
  const long long items = static_cast<long long>(n) * pieces;
  const long long warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
  for (long long i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < items; i += warps) {
    const int r = static_cast<int>(i / pieces), piece = static_cast<int>(i - static_cast<long long>(r) * pieces);
    const int p = row_idx[r];
    const bool bad = p < 0 || p >= n_pos;
    if (bad && (threadIdx.x & 31) == 0) atomicOr(status, kStatusBounds);
    quantize_piece(bad ? static_cast<const __nv_bfloat16*>(nullptr)
                       : reinterpret_cast<const __nv_bfloat16*>(H) + static_cast<size_t>(p) * d,
                   piece * kPiece, d, groups, r, q, s);
  }
}

// The values of two E2M1 codes (a byte, low nibble first).
__device__ __forceinline__ float2 e2m1x2_values(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 b, x;\n\t"
      "cvt.u8.u32 b, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
      : "=r"(h)
      : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
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
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}

// The values an MXFP4 matrix stands for (bf16 or fp32: both exact): a warp per row, eight
// elements per lane and step.
template <typename T>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint8_t* __restrict__ q, const uint32_t* __restrict__ s, long long rows, int K,
                  T* __restrict__ X, long long ld) {
  pdl_wait();
  pdl_launch_dependents();
  const int groups = (K + 127) / 128, lane = threadIdx.x & 31;
  const long long warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
  for (long long r = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < rows; r += warps) {
    for (int k0 = 8 * lane; k0 < K; k0 += kPiece) {
      uint32_t codes[kSteps], words[kSteps];
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int k = k0 + 256 * j;
        if (k < K) {
          codes[j] = __ldcs(reinterpret_cast<const uint32_t*>(q + r * (K / 2) + k / 2));
          words[j] = __ldg(s + scale_word(r, k >> 7, groups));
        }
      }
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int k = k0 + 256 * j;
        if (k < K) {
          const float scale = e8m0_value((words[j] >> (8 * ((k >> 5) & 3))) & 0xffu);
          float v[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 y = e2m1x2_values((codes[j] >> (8 * i)) & 0xffu);
            v[2 * i] = y.x * scale;
            v[2 * i + 1] = y.y * scale;
          }
          store8(X + r * ld + k, v);
        }
      }
    }
  }
}

}  // namespace mx4
}  // namespace dllm
