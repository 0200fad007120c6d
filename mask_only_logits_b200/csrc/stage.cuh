// stage.cuh - compaction and gather of a small mask in one launch, for the LM head of
// shaped.cuh: the masked rows of H as dense rows (bf16, or quantised to MXFP4), with the
// compaction's own outputs (row_idx, seq_off, count).
//
// Every CTA scans the whole mask, 16 bytes a thread, and so knows its share of the masked rows
// without a word from the others; it writes those rows and their positions.  One launch fewer is
// 2.3 us of the host's 11 us in a call, which a small step waits for.  Up to kMaxPositions: there
// the GPU takes as long as with the two kernels of compact.cuh and mx4.cuh (20.8 against 20.5 us
// a step at 655 positions); at 4096 positions the step is 1 to 2 us longer, the scan being every
// CTA's first work.
#pragma once
#include "compact.cuh"
#include "mx4.cuh"

namespace dllm {
namespace stage {

constexpr int kThreads = 256;
constexpr int kMaxPositions = 2048;                  // at most kThreads * kCompactVec
constexpr int kCtas = 64;

template <bool kMx4>
__global__ void __launch_bounds__(kThreads)
stage_rows_kernel(const uint8_t* __restrict__ M, int B, int L, const int* __restrict__ win_lo,
                  const int* __restrict__ win_hi, const uint16_t* __restrict__ H, int d, long long n_cap,
                  int* __restrict__ row_idx, int* __restrict__ seq_off, int* __restrict__ count,
                  uint8_t* __restrict__ rows_out, uint32_t* __restrict__ scales_out,
                  int* __restrict__ zero, int n_zero, int* __restrict__ status) {
  __shared__ int warp_sum[kThreads / 32];
  __shared__ int pos[kMaxPositions / kCtas];         // this CTA's rows
  pdl_wait();
  pdl_launch_dependents();
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < n_zero; i += gridDim.x * kThreads) zero[i] = 0;
  const int n = B * L;                               // <= kMaxPositions
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int p0 = threadIdx.x * kCompactVec;
  const uint32_t bits = p0 < n ? window_filter(load_mask16(M, p0, n), p0, L, win_lo, win_hi) : 0u;
  const int c = __popc(bits);
  int incl = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int base = incl - c, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += warp_sum[w];
    total += warp_sum[w];
  }
  // this CTA's rows [r0, r1): at most kMaxPositions / kCtas
  const int per = (total + kCtas - 1) / kCtas;
  const int r0 = min(static_cast<int>(blockIdx.x) * per, total), r1 = min(r0 + per, total);
  int r = base;
  for (uint32_t b = bits; b != 0; b &= b - 1, ++r)
    if (r >= r0 && r < r1) pos[r - r0] = p0 + __ffs(b) - 1;
  if (blockIdx.x == 0) {
    if (p0 < n) {                                    // sequences that begin in this vector
      const int lim = min(p0 + kCompactVec, n);
      for (int s = (p0 + L - 1) / L; s < B && s * L < lim; ++s)
        seq_off[s] = base + __popc(bits & ((1u << (s * L - p0)) - 1u));
    }
    if (threadIdx.x == 0) {
      seq_off[B] = total;
      *count = total;
      if (total > n_cap) atomicOr(status, kStatusCapacity);   // workspace sized for fewer rows
    }
  }
  __syncthreads();
  for (int i = r0 + threadIdx.x; i < r1; i += kThreads) row_idx[i] = pos[i - r0];
  // the rows that fit, in pieces a warp takes at a time
  const int mine = (n_cap < r1 ? static_cast<int>(n_cap) : r1) - r0;
  if constexpr (kMx4) {
    const int groups = (d + 127) / 128, pieces = (groups * 128 + mx4::kPiece - 1) / mx4::kPiece;
    for (int i = warp; i < mine * pieces; i += kThreads / 32) {
      const int j = i / pieces;
      mx4::quantize_piece(reinterpret_cast<const __nv_bfloat16*>(H) + static_cast<size_t>(pos[j]) * d,
                          (i - j * pieces) * mx4::kPiece, d, groups, r0 + j, rows_out, scales_out);
    }
  } else {
    const int vec_per_row = d / 8, pieces = (vec_per_row + 127) / 128;        // 128 vectors of 16 bytes
    for (int i = warp; i < mine * pieces; i += kThreads / 32) {
      const int j = i / pieces, w0 = (i - j * pieces) * 128 + lane;
      const uint4* src = reinterpret_cast<const uint4*>(H + static_cast<size_t>(pos[j]) * d);
      uint4* dst = reinterpret_cast<uint4*>(rows_out) + static_cast<size_t>(r0 + j) * vec_per_row;
      uint4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (w0 + 32 * k < vec_per_row) x[k] = __ldg(src + w0 + 32 * k);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (w0 + 32 * k < vec_per_row) dst[w0 + 32 * k] = x[k];
    }
  }
}

}  // namespace stage
}  // namespace dllm
