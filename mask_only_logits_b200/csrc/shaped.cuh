// shaped.cuh - the masked LM head with rules on its logits, with bf16 or MXFP4 operands.
//
// Plain tiles on the CUDA cores: a CTA owns 64 masked rows and a contiguous range of the
// vocabulary, forms 64 x 64 logits at a time in registers (fp32), and folds them row by row
// into the running statistics; shaped_merge_kernel merges the ranges' partials in order.
#pragma once
#include "mx4.cuh"
#include "rules.cuh"

namespace dllm {
namespace shaped {

constexpr int kThreads = 256;
constexpr int BM = 64, BN = 64, BK = 32;

struct Operands {
  const uint16_t* Hm; const uint16_t* W;                       // bf16
  const uint8_t* Hq; const uint8_t* Hs; const uint8_t* Wq; const uint8_t* Ws;   // MXFP4
};

template <bool kMx4>
__device__ __forceinline__ float element(const Operands& o, bool a, long long r, int k, int d) {
  if constexpr (!kMx4) {
    const uint16_t b = (a ? o.Hm : o.W)[r * d + k];
    return __uint_as_float(static_cast<uint32_t>(b) << 16);
  } else {
    const uint8_t c = (a ? o.Hq : o.Wq)[r * (d / 2) + k / 2];
    const uint8_t s = (a ? o.Hs : o.Ws)[4 * mx4::scale_word(r, k >> 7, (d + 127) / 128) + ((k >> 5) & 3)];
    return mx4::e2m1_value(k & 1 ? c >> 4 : c & 15) * mx4::e8m0_value(s);
  }
}

template <bool kMx4, bool kExt>
__global__ void __launch_bounds__(kThreads)
shaped_kernel(const Operands o, const int* __restrict__ count_ptr, int n_cap, int V, int d, int L,
              const dllm_logit_rules r, const int* __restrict__ row_idx, const lm::Partials part,
              int n_split, int* __restrict__ status) {
  __shared__ float a[BK][BM + 1], b[BK][BN + 1];
  __shared__ float z[BM][BN + 1];
  pdl_wait();
  pdl_launch_dependents();
  int n = *count_ptr;
  n = n < 0 ? 0 : (n > n_cap ? n_cap : n);
  const int r0 = blockIdx.x * BM;
  if (r0 >= n) return;
  const int tiles = (V + BN - 1) / BN;
  const int t0 = static_cast<int>(static_cast<long long>(blockIdx.y) * tiles / n_split);
  const int t1 = static_cast<int>(static_cast<long long>(blockIdx.y + 1) * tiles / n_split);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int row = r0 + threadIdx.x;                        // threads 0..63: one row each
  rules::RowRules rr = rules::no_rules();
  if (threadIdx.x < BM && row < n) rr = rules::row_rules(r, row_idx[row], L, status);
  lm::RowState st;
  st.reset();
  for (int t = t0; t < t1; ++t) {
    float acc[4][4] = {};
    for (int k0 = 0; k0 < d; k0 += BK) {
      for (int i = threadIdx.x; i < BM * BK; i += kThreads) {
        const int rr_ = i / BK, k = i % BK;
        a[k][rr_] = r0 + rr_ < n ? element<kMx4>(o, true, r0 + rr_, k0 + k, d) : 0.f;
        b[k][rr_] = t * BN + rr_ < V ? element<kMx4>(o, false, t * BN + rr_, k0 + k, d) : 0.f;
      }
      __syncthreads();
      for (int k = 0; k < BK; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[k][ty * 4 + i], b[k][tx * 4 + j], acc[i][j]);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) z[ty * 4 + i][tx * 4 + j] = acc[i][j];
    __syncthreads();
    if (threadIdx.x < BM) {
      for (int c = 0; c < BN; c += 32) {
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = z[threadIdx.x][c + j];
        rules::shape_chunk(v, t * BN + c, V, rr);
        rules::fold<kExt>(v, t * BN + c, st);
      }
    }
    __syncthreads();
  }
  if (threadIdx.x < BM && row < n) {
    const long long e = static_cast<long long>(blockIdx.y) * n_cap + row;
    part.m[e] = st.m;
    part.s[e] = st.s;
    part.a[e] = st.a;
    if constexpr (kExt) {
      part.t[e] = st.t;
      part.m2[e] = st.m2;
    }
  }
}

template <bool kExt>
__global__ void __launch_bounds__(kThreads)
shaped_merge_kernel(const lm::Partials part, const int* __restrict__ count_ptr, int n_cap, int n_split,
                    const lm::Outputs out) {
  pdl_wait();
  pdl_launch_dependents();
  int n = *count_ptr;
  n = n < 0 ? 0 : (n > n_cap ? n_cap : n);
  for (int row = blockIdx.x * kThreads + threadIdx.x; row < n; row += gridDim.x * kThreads) {
    lm::RowState st;
    st.reset();
    for (int j = 0; j < n_split; ++j) {
      const long long e = static_cast<long long>(j) * n_cap + row;
      rules::merge<kExt>(st, part.m[e], part.s[e], part.a[e], kExt ? part.t[e] : 0.f,
                         kExt ? part.m2[e] : 0.f);
    }
    int t;
    float c, l, en, mg;
    rules::finish(st, t, c, l, en, mg);
    out.tok[row] = t;
    out.conf[row] = c;
    out.lse[row] = l;
    if constexpr (kExt) {
      if (out.entropy) out.entropy[row] = en;
      if (out.margin) out.margin[row] = mg;
    }
  }
}

}  // namespace shaped
}  // namespace dllm
