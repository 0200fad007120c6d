// rules.cuh - rules on the logits of a masked row (dllm_logit_rules): penalties for tokens the
// sequence already holds, a bias, and a bitmap of the tokens allowed; and the token counts the
// penalties read.
//
// With z0 the row's raw logit of token v, c how often v stands in the row's sequence b:
//   z1 = c > 0 ? (z0 > 0 ? z0 / theta_b : z0 * theta_b) - presence_b - frequency_b * c : z0
//   z2 = z1 + bias[b, v]
//   z  = allowed(row, v) ? z2 : -inf
// The rules act on the accumulator chunk of 32 columns that the LM head's epilogue holds in
// registers, so a shaped logit is never stored either.  Every step is rounded to fp32 on its
// own (no contraction), the same as the formula evaluated step by step in fp32.
//
// The row states here differ from lmhead.cuh's in what rules make possible: a row, a split or
// a chunk with nothing allowed (max = -inf), and logits at the lowest finite value (a bias of
// -FLT_MAX is a number, not a ban).  Differences to the maximum are taken before the scaling
// by log2 e, so that neither overflows, and a factor exp(m_old - m_new) of 0 drops what it
// multiplies.
#pragma once
#include "dllm.h"
#include "lmhead.cuh"

namespace dllm {
namespace rules {

// The rules of one row: pointers into its sequence's and its bitmap's rows (null = no such rule).
struct RowRules {
  const float* bias;
  const int* counts;
  const uint32_t* seen;
  const uint32_t* allow;
  float theta, presence, frequency;
};

__device__ __forceinline__ RowRules no_rules() {
  return RowRules{nullptr, nullptr, nullptr, nullptr, 1.f, 0.f, 0.f};
}

// The rules of the row at flat position pos (= b * L + l).  A bitmap number past the table is
// recorded and the row left unrestricted.
__device__ __forceinline__ RowRules row_rules(const dllm_logit_rules& r, int pos, int L, int* status) {
  RowRules o = no_rules();
  const long long b = pos / L;
  if (r.bias) o.bias = r.bias + b * r.bias_stride;
  if (r.counts) {
    o.counts = r.counts + b * r.counts_stride;
    o.seen = r.seen + b * r.seen_stride;
    if (r.repetition) o.theta = r.repetition[b];
    if (r.presence) o.presence = r.presence[b];
    if (r.frequency) o.frequency = r.frequency[b];
  }
  if (r.allow) {
    const int id = r.allow_id ? r.allow_id[pos] : (r.allow_rows == 1 ? 0 : static_cast<int>(b));
    if (id >= r.allow_rows) atomicOr(status, kStatusBounds);
    else if (id >= 0) o.allow = r.allow + static_cast<long long>(id) * r.allow_stride;
  }
  return o;
}

__device__ __forceinline__ float penalise(float z, int c, const RowRules& r) {
  z = z > 0.f ? __fdiv_rn(z, r.theta) : __fmul_rn(z, r.theta);
  return __fsub_rn(__fsub_rn(z, r.presence), __fmul_rn(r.frequency, static_cast<float>(c)));
}

// Shape the 32 logits of columns col0 .. col0+31 (col0 a multiple of 32) of each lane's row;
// columns at and past V become -inf.  Called by all 32 lanes of a warp together: the tests
// that skip a rule are taken for the warp, whose rows mostly share a sequence.
__device__ __forceinline__ void shape_chunk(float (&v)[32], int col0, int V, const RowRules& r) {
  const int left = V - col0;
  const uint32_t in = left >= 32 ? 0xffffffffu : (left > 0 ? (1u << left) - 1u : 0u);
  const uint32_t seen = r.seen && in ? __ldg(r.seen + (col0 >> 5)) & in : 0u;
  const uint32_t ok = r.allow && in ? __ldg(r.allow + (col0 >> 5)) & in : in;
  const uint32_t any_seen = __reduce_or_sync(0xffffffffu, seen);
  if (any_seen != 0u) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if ((any_seen >> j) & 1u) {
        if ((seen >> j) & 1u) v[j] = penalise(v[j], __ldg(r.counts + col0 + j), r);
      }
  }
  if (__any_sync(0xffffffffu, r.bias != nullptr)) {
    if (r.bias != nullptr) {
      if (left >= 32) {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 b = __ldg(reinterpret_cast<const float4*>(r.bias + col0 + j));
          v[j + 0] = __fadd_rn(v[j + 0], b.x);
          v[j + 1] = __fadd_rn(v[j + 1], b.y);
          v[j + 2] = __fadd_rn(v[j + 2], b.z);
          v[j + 3] = __fadd_rn(v[j + 3], b.w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < left) v[j] = __fadd_rn(v[j], __ldg(r.bias + col0 + j));
      }
    }
  }
  if (!__all_sync(0xffffffffu, ok == 0xffffffffu)) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (!((ok >> j) & 1u)) v[j] = -INFINITY;
  }
}

// Fold 32 logits (columns col0 ..) into a row's state (see above for how this differs from
// lm::fold_chunk).
template <bool kExt>
__device__ __forceinline__ void fold(const float (&v)[32], int col0, lm::RowState& st) {
  float mx = v[0];
#pragma unroll
  for (int j = 1; j < 32; ++j) mx = fmaxf(mx, v[j]);
  if (mx == -INFINITY) return;                 // nothing allowed in this chunk
  float c2 = -INFINITY;                        // chunk's second largest (= mx on a tie)
  if constexpr (kExt) {
    int n_at_max = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      n_at_max += v[j] == mx ? 1 : 0;
      c2 = v[j] == mx ? c2 : fmaxf(c2, v[j]);
    }
    if (n_at_max > 1) c2 = mx;
  }
  if (mx > st.m) {                             // strict: earlier (lower) index wins ties
    int j0 = 31;
#pragma unroll
    for (int j = 31; j >= 0; --j)
      if (v[j] == mx) j0 = j;
    const float sc = ex2_approx((st.m - mx) * lm::kLog2e);
    if constexpr (kExt) {
      st.t = sc > 0.f ? sc * (st.t + (st.m - mx) * st.s) : 0.f;
      st.m2 = fmaxf(st.m, c2);
    }
    st.s *= sc;
    st.m = mx;
    st.a = col0 + j0;
  } else if constexpr (kExt) {
    st.m2 = fmaxf(st.m2, mx);
  }
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f, t0 = 0.f, t1 = 0.f;
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const float x0 = v[j] - st.m, x1 = v[j + 1] - st.m, x2 = v[j + 2] - st.m, x3 = v[j + 3] - st.m;
    const float e0 = ex2_approx(x0 * lm::kLog2e), e1 = ex2_approx(x1 * lm::kLog2e);
    const float e2 = ex2_approx(x2 * lm::kLog2e), e3 = ex2_approx(x3 * lm::kLog2e);
    s0 += e0;
    s1 += e1;
    s2 += e2;
    s3 += e3;
    if constexpr (kExt) {
      t0 += e0 > 0.f ? e0 * x0 : 0.f;
      t1 += e1 > 0.f ? e1 * x1 : 0.f;
      t0 += e2 > 0.f ? e2 * x2 : 0.f;
      t1 += e3 > 0.f ? e3 * x3 : 0.f;
    }
  }
  st.s += (s0 + s1) + (s2 + s3);
  if constexpr (kExt) st.t += t0 + t1;
}

// Merge a later split's state into st (lm::merge_state with the factor guarded).
template <bool kExt>
__device__ __forceinline__ void merge(lm::RowState& st, float m, float s, int a, float t, float m2) {
  if (m == -INFINITY) return;
  if (m > st.m) {                              // strict: the earlier split keeps a tie
    const float sc = ex2_approx((st.m - m) * lm::kLog2e);
    if constexpr (kExt) {
      st.t = (sc > 0.f ? sc * (st.t + (st.m - m) * st.s) : 0.f) + t;
      st.m2 = fmaxf(st.m, m2);
    }
    st.s = st.s * sc + s;
    st.m = m;
    st.a = a;
  } else {
    const float sc = ex2_approx((m - st.m) * lm::kLog2e);
    if constexpr (kExt) {
      st.t += sc > 0.f ? sc * (t + (m - st.m) * s) : 0.f;
      st.m2 = fmaxf(st.m2, m);
    }
    st.s += s * sc;
  }
}

// Final values of a row.  Nothing allowed: no token, no confidence, and the worst of each
// score, so that a selection takes such a row last.
__device__ __forceinline__ void finish(const lm::RowState& st, int& tok, float& conf, float& lse,
                                       float& ent, float& margin) {
  if (st.m == -INFINITY) {
    tok = -1;
    conf = 0.f;
    lse = -INFINITY;
    ent = INFINITY;
    margin = 0.f;
    return;
  }
  const float ls = logf(st.s);
  tok = st.a;
  lse = st.m + ls;
  conf = 1.0f / st.s;
  ent = ls - st.t / st.s;
  margin = (1.0f - ex2_approx((st.m2 - st.m) * lm::kLog2e)) / st.s;
}

// ---------------------------------------------------------------------------------------
// token counts
// ---------------------------------------------------------------------------------------
constexpr int kCountThreads = 512;
constexpr int kCountMaxSlice = 32768;          // columns of one CTA: 128 KB of shared memory

// counts[b, v] = how often v stands among sequence b's first n_valid[b] of n tokens, at
// positions whose mask byte is zero; seen: the bitmap of counts > 0.  One CTA per (slice of
// the vocabulary, sequence) reads all of the sequence's tokens and counts those of its slice
// in shared memory: the counts are written once, in order, and no count depends on an order.
__global__ void __launch_bounds__(kCountThreads)
token_count_kernel(const int* __restrict__ tokens, const uint8_t* __restrict__ M,
                   const int* __restrict__ n_valid, int n, int V, int slice,
                   int* __restrict__ counts, uint32_t* __restrict__ seen) {
  extern __shared__ int hist[];
  const int b = blockIdx.y, v0 = blockIdx.x * slice;
  for (int i = threadIdx.x; i < slice; i += kCountThreads) hist[i] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  int valid = n;
  if (n_valid) {
    valid = n_valid[b];
    valid = valid < 0 ? 0 : (valid > n ? n : valid);
  }
  const long long row = static_cast<long long>(b) * n;
  const int v1 = v0 + slice < V ? v0 + slice : V;
  for (int j = threadIdx.x; j < valid; j += kCountThreads) {
    if (M && M[row + j] != 0) continue;
    const int t = tokens[row + j];
    if (t >= v0 && t < v1) atomicAdd(&hist[t - v0], 1);
  }
  __syncthreads();
  const int words = (V + 31) / 32;
  for (int i = threadIdx.x; i < slice; i += kCountThreads) {     // slice: a multiple of 32
    const int c = hist[i];
    const uint32_t bits = __ballot_sync(0xffffffffu, c > 0);
    if (v0 + i < V) counts[static_cast<long long>(b) * V + v0 + i] = c;
    if ((threadIdx.x & 31) == 0 && v0 + i < V)
      seen[static_cast<long long>(b) * words + ((v0 + i) >> 5)] = bits;
  }
}

// The same tokens added to counts and seen that are there already (one thread per token).
__global__ void __launch_bounds__(kCountThreads)
token_add_kernel(const int* __restrict__ tokens, const uint8_t* __restrict__ M,
                 const int* __restrict__ n_valid, int n, int V, int* __restrict__ counts,
                 uint32_t* __restrict__ seen) {
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y;
  const int valid = n_valid ? (n_valid[b] < n ? n_valid[b] : n) : n;
  const long long row = static_cast<long long>(b) * n;
  const int words = (V + 31) / 32;
  for (int j = blockIdx.x * kCountThreads + threadIdx.x; j < valid; j += gridDim.x * kCountThreads) {
    if (M && M[row + j] != 0) continue;
    const int t = tokens[row + j];
    if (t < 0 || t >= V) continue;
    atomicAdd(counts + static_cast<long long>(b) * V + t, 1);
    atomicOr(seen + static_cast<long long>(b) * words + (t >> 5), 1u << (t & 31));
  }
}

}  // namespace rules
}  // namespace dllm
