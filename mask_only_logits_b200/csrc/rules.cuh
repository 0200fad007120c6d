// rules.cuh - rules on the logits of a masked row (dllm_logit_rules): penalties for tokens the
// sequence already holds, a bias, and a bitmap of the tokens allowed; and the token counts the
// penalties read.
//
// With z0 the row's raw logit of token v, c how often v stands in the row's sequence b:
//   z1 = c > 0 ? (z0 > 0 ? z0 / theta_b : z0 * theta_b) - presence_b - frequency_b * c : z0
//   z2 = z1 + bias[b, v]
//   z  = allowed(row, v) ? z2 : -inf
// theta's reciprocal is rounded once per row: z * (1 / theta) is within one unit in the last
// place of z / theta, and the 32 columns of a chunk stay free of the division's branches (with
// them a chunk of penalised columns took 5000 cycles).
//
// The rules act on the accumulator chunk of 32 columns that the LM head's epilogue holds in
// registers, so a shaped logit is never stored either; they are evaluated in fp32.
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

// Two fp32 operations in one instruction (packed, each rounded as on its own).
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// The rules of one row: pointers into its sequence's and its bitmap's rows (null = no such rule).
struct RowRules {
  const float* bias;
  const int* counts;
  const uint32_t* seen;
  const uint32_t* allow;
  float theta, inverse, presence, frequency;     // inverse = 1 / theta
};

__device__ __forceinline__ RowRules no_rules() {
  return RowRules{nullptr, nullptr, nullptr, nullptr, 1.f, 1.f, 0.f, 0.f};
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
    o.inverse = 1.0f / o.theta;
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

// A read-only load that stays where it is written (the compiler would move one whose value is
// needed much later down to its use).
__device__ __forceinline__ uint32_t load_now(const void* p) {
  uint32_t x;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}

// The words of a row's two bitmaps that cover columns col0 .. col0+31 (col0 a multiple of 32;
// bits at and past V cleared): which of them the sequence holds, and which are allowed.
struct Words {
  uint32_t seen, ok;
};
__device__ __forceinline__ Words load_words(int col0, int V, const RowRules& r) {
  const int left = V - col0;
  const uint32_t in = left >= 32 ? 0xffffffffu : (left > 0 ? (1u << left) - 1u : 0u);
  Words w{0u, in};
  if (r.seen && in) w.seen = load_now(r.seen + (col0 >> 5)) & in;
  if (r.allow && in) w.ok = load_now(r.allow + (col0 >> 5)) & in;
  return w;
}

__device__ __forceinline__ void ban(float (&v)[32], uint32_t ok) {
  if (!__all_sync(0xffffffffu, ok == 0xffffffffu)) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (!((ok >> j) & 1u)) v[j] = -INFINITY;
  }
}

// Shape the 32 logits of columns col0 .. col0+31 of each lane's row; what is not allowed, and
// columns at and past V, become -inf.  Called by all 32 lanes of a warp together.
//
// shape_same: all rows of the warp have the same bias row and the same sequence's counts.  Then
// column j's additive part (bias - presence - frequency * count, see additive) was fetched by
// lane j ahead of time, one coalesced word per chunk, and stands in shared memory at `add`
// (null: neither rule), from where every lane reads all 32.
__device__ __forceinline__ void shape_same(float (&v)[32], const RowRules& r, const Words& w, const float* add) {
  if (w.seen != 0u) {                          // the same word in every lane
#pragma unroll
    for (int g = 0; g < 32; g += 8) {
      if (((w.seen >> g) & 0xffu) == 0u) continue;
#pragma unroll
      for (int j = g; j < g + 8; ++j) {
        const float y = v[j] * (v[j] > 0.f ? r.inverse : r.theta);
        v[j] = (w.seen >> j) & 1u ? y : v[j];
      }
    }
  }
  if (add != nullptr) {
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 b = *reinterpret_cast<const float4*>(add + j);
      const float2 lo = add2(make_float2(v[j], v[j + 1]), make_float2(b.x, b.y));
      const float2 hi = add2(make_float2(v[j + 2], v[j + 3]), make_float2(b.z, b.w));
      v[j + 0] = lo.x;
      v[j + 1] = lo.y;
      v[j + 2] = hi.x;
      v[j + 3] = hi.y;
    }
  }
  ban(v, w.ok);
}

// The additive part of a column, of a bias and a count that were read for it.
__device__ __forceinline__ float additive(float bias, int c, bool seen, const RowRules& r) {
  return seen ? fmaf(-r.frequency, static_cast<float>(c), bias - r.presence) : bias;
}

// shape_mixed: the rows belong to several sequences; each lane reads its own.
__device__ __forceinline__ void shape_mixed(float (&v)[32], int col0, int V, const RowRules& r, const Words& w) {
  const uint32_t any_seen = __reduce_or_sync(0xffffffffu, w.seen);
  if (any_seen != 0u) {
    // eight columns at a time, without branches: all their counts are asked for before the
    // first is used
#pragma unroll
    for (int g = 0; g < 32; g += 8) {
      if (((any_seen >> g) & 0xffu) == 0u) continue;
      int c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        c[j] = 0;
        if ((w.seen >> (g + j)) & 1u) c[j] = __ldg(r.counts + col0 + g + j);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float z = v[g + j];
        const float y = z * (z > 0.f ? r.inverse : r.theta) + additive(0.f, c[j], true, r);
        v[g + j] = (w.seen >> (g + j)) & 1u ? y : z;
      }
    }
  }
  if (r.bias != nullptr) {
    if (col0 + 32 <= V) {
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 b = __ldg(reinterpret_cast<const float4*>(r.bias + col0 + j));
        v[j + 0] += b.x;
        v[j + 1] += b.y;
        v[j + 2] += b.z;
        v[j + 3] += b.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (col0 + j < V) v[j] += __ldg(r.bias + col0 + j);
    }
  }
  ban(v, w.ok);
}

// Running statistics of one row, as lm::RowState, with the rounding errors of s and t carried
// along (Kahan): a row's sum grows by thousands of chunks, each small against it, and adding
// them plainly lost up to 6e-6 of it.
struct State {
  float m, s, t, m2;
  int a;
  float sc, tc;                                // what s and t hold too much
  __device__ __forceinline__ void reset() {
    m = m2 = -INFINITY;
    s = t = sc = tc = 0.f;
    a = 0;
  }
  __device__ __forceinline__ lm::RowState value() const {
    lm::RowState r;
    r.m = m;
    r.s = s - sc;
    r.t = t - tc;
    r.m2 = m2;
    r.a = a;
    return r;
  }
};

// The largest of three, NaN if one of them is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void kahan(float& sum, float& over, float x) {
  const float y = x - over;
  const float n = sum + y;
  over = (n - sum) - y;
  sum = n;
}

// Fold 32 logits (columns col0 ..) into a row's state (see above for how this differs from
// lm::fold_chunk).
template <bool kExt>
__device__ __forceinline__ void fold(const float (&v)[32], int col0, State& st) {
  float mx = v[0];
#pragma unroll
  for (int j = 1; j < 31; j += 2) mx = max3(mx, v[j], v[j + 1]);
  mx = max3(mx, v[31], v[31]);
  if (mx == -INFINITY) return;                 // nothing allowed in this chunk
  if (mx != mx) {                              // a NaN: so are the row's statistics
    st.s = mx;
    if constexpr (kExt) st.t = mx;
    return;
  }
  // of equal maxima the lower token wins; chunks come in any order
  const bool above = mx > st.m;
  if (above || (mx == st.m && col0 < st.a)) {
    uint32_t at = 0;                           // columns at the maximum
    float c2 = -INFINITY;                      // the largest of the others
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (v[j] == mx) at |= 1u << j;
      else if constexpr (kExt) c2 = fmaxf(c2, v[j]);
    }
    st.a = col0 + __ffs(at) - 1;
    if (above) {
      const float f = ex2_approx((st.m - mx) * lm::kLog2e);
      if constexpr (kExt) {
        st.t = f > 0.f ? f * ((st.t - st.tc) + (st.m - mx) * (st.s - st.sc)) : 0.f;
        st.tc = 0.f;
        st.m2 = (at & (at - 1u)) != 0u ? mx : fmaxf(st.m, c2);
      }
      st.s *= f;
      st.sc *= f;
      st.m = mx;
    }
  }
  if constexpr (kExt) {
    if (!above) st.m2 = fmaxf(st.m2, mx);
  }
  const float2 shift = make_float2(-st.m, -st.m), log2e = make_float2(lm::kLog2e, lm::kLog2e);
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  float2 dev[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float2 x = add2(make_float2(v[2 * j], v[2 * j + 1]), shift);
    const float2 y = mul2(x, log2e);
    const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
    sum[j & 1] = add2(sum[j & 1], e);
    if constexpr (kExt) {                      // e is 0 long before x reaches the bound
      x = make_float2(fmaxf(x.x, -1e4f), fmaxf(x.y, -1e4f));
      dev[j & 1] = fma2(e, x, dev[j & 1]);
    }
  }
  kahan(st.s, st.sc, (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
  if constexpr (kExt) kahan(st.t, st.tc, (dev[0].x + dev[0].y) + (dev[1].x + dev[1].y));
}

// Merge another part of the vocabulary's statistics into st; of equal maxima the lower token
// wins, so the parts may come in any order.
template <bool kExt>
__device__ __forceinline__ void merge(lm::RowState& st, float m, float s, int a, float t, float m2) {
  if (m == -INFINITY && s == 0.f) return;      // nothing allowed (a sum that is NaN goes on)
  if (m > st.m) {
    const float f = ex2_approx((st.m - m) * lm::kLog2e);
    if constexpr (kExt) {
      st.t = (f > 0.f ? f * (st.t + (st.m - m) * st.s) : 0.f) + t;
      st.m2 = fmaxf(st.m, m2);
    }
    st.s = st.s * f + s;
    st.m = m;
    st.a = a;
  } else {
    const float f = ex2_approx((m - st.m) * lm::kLog2e);
    if constexpr (kExt) {
      st.t += f > 0.f ? f * (t + (m - st.m) * s) : 0.f;
      st.m2 = fmaxf(st.m2, m);
    }
    st.s += s * f;
    if (m == st.m && a < st.a) st.a = a;
  }
}

// Final values of a row.  Nothing allowed: no token, no confidence, and the worst of each
// score, so that a selection takes such a row last; the margin is a negative zero, behind the zero
// of a row whose two best logits are equal.  A row whose every logit is NaN has NaN statistics and
// token 0.
__device__ __forceinline__ void finish(const lm::RowState& st, int& tok, float& conf, float& lse,
                                       float& ent, float& margin) {
  if (st.m == -INFINITY && st.s == 0.f) {
    tok = -1;
    conf = 0.f;
    lse = -INFINITY;
    ent = INFINITY;
    margin = -0.f;
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
  // unsigned: n may be 2^31 - 1, and j goes a stride past it
  for (unsigned j = threadIdx.x; j < static_cast<unsigned>(valid); j += kCountThreads) {
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
  const unsigned valid = n_valid ? min(max(n_valid[b], 0), n) : n;
  const long long row = static_cast<long long>(b) * n;
  const int words = (V + 31) / 32;
  for (unsigned j = blockIdx.x * kCountThreads + threadIdx.x; j < valid; j += gridDim.x * kCountThreads) {
    if (M && M[row + j] != 0) continue;
    const int t = tokens[row + j];
    if (t < 0 || t >= V) continue;
    atomicAdd(counts + static_cast<long long>(b) * V + t, 1);
    atomicOr(seen + static_cast<long long>(b) * words + (t >> 5), 1u << (t & 31));
  }
}

}  // namespace rules
}  // namespace dllm
