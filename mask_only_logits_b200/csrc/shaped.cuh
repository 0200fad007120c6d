// shaped.cuh - the masked LM head with rules on its logits, with bf16 or MXFP4 operands, on the
// 5th-generation tensor cores.
//
// The persistent, warp-specialised structure, the work schedule (Plan) and the split merge are
// those of lmhead.cuh: per CTA one TMA warp, one MMA warp, and epilogue warps; single CTAs or
// CTA pairs chosen on the device from the masked count.  What differs:
//   operands  Bf16: kind::f16, 256 vocabulary columns a tile.
//             Mx4:  kind::mxf4 with one power-of-two scale per 32 elements of K.  256 elements
//             of K are 128 bytes, so a stage holds four times the K of a bf16 stage.  The
//             scales of a stage are copied from shared memory to TMEM (tcgen05.cp, each 512-byte
//             tile to 4 columns, replicated over the four lane quadrants) ahead of its MMAs.
//             TMEM holds two accumulators and the scales of five stages; with 192 columns a
//             tile that is 2 x 192 + 5 x 24 = 504 of 512 columns.  Scale columns are rewritten
//             only after the MMAs that read them have released their stage.  A tile of 192
//             columns starts on a scale tile (128 rows of W) or in the middle of one: it takes
//             two scale tiles and, if odd, starts two columns in.
//   issue     four MMAs of a stage take 0.2 us, so the issuing warp runs converged, with
//             warp-uniform operands, and elects a lane per instruction: from a lone lane the
//             operands pass through vector registers and a stage took 0.53 us to issue.
//   ring      as many stages as fit: what bounds the staging is the bytes in flight (a stage
//             comes 2 us after it is asked for when every SM loads).
//   A rows    single CTAs load their rows of Hm in boxes of 32, only as many as are masked; the
//             rest of the operand's 128 rows is zeroed once: the tensor cores' power depends on
//             what they multiply, and streaming W for one row runs at the power cap (one row
//             d4096 V126464, back to back: bf16, K in pieces of 512, 195.3 -> 191.8 us, MXFP4
//             65.4 -> 64.4 us).
//   order     the schedule's vocabulary tile i is tile i * step mod (tiles), step coprime to the
//             tiles and about 0.62 of them: frequent tokens sit at the low ids of a vocabulary,
//             so a stream of consecutive tiles would get all the penalised columns (99 us where
//             the others took 65, 256 rows of d2048 V151936).
//   sums      The tensor cores drop what does not fit fp32 beside the running sum, always
//             towards zero: over d = 4096 a large bf16 logit came out 5e-6 too small.  An
//             accumulator therefore holds a piece of K; the epilogue adds the pieces up in
//             registers (128 a thread, dealt to the epilogue's warpgroups by setmaxnreg).  Of a
//             normal row's statistics that leaves an fp32 sum's error (d up to 4096: 0.1e-6 to
//             1.5e-6).  Where a few channels make most of a sum and the rest add to it with one
//             sign, the piece that holds them loses about 1.4 last places per step of K = 16:
//             with the largest 2^10 times the others, d = 4096, pairs are 9e-6 off, single CTAs
//             0.8e-6, a rounded fp32 sum 0.7e-6.
//             MXFP4 products are a few bits wide: their sums are exact while the scales of the
//             blocks that matter lie close together.  With scales drawn from 2^-12 to 2^12 the
//             d / 64 steps truncate too: 0.8e-6 at d = 2048, 1.5e-6 at 4096, 2.7e-6 at 8192 (a
//             rounded fp32 sum 0.9e-6, 1.1e-6, 2.1e-6), so a tile's K stays in one accumulator.
//   epilogue  eight warps: two per TMEM lane quadrant, each with half of a tile's columns (the
//             rules and scores cost more instructions than the plain statistics, and four MXFP4
//             tiles take the time of one bf16 tile).  rules on each 32 logits, then
//             the fold and merge of rules.cuh.  Warps without a masked row only release the
//             accumulator.  Rows of one warp mostly share a sequence: what its rules read for a
//             tile then comes as one coalesced word per chunk and array, fetched during the
//             tile before; loaded where it is used it held each chunk up by 2 us.
//   merge     of at most 32 rows: a warp per row, its lanes over the splits (a row's partials
//             then come in one or two rounds of loads instead of one per eight splits).
#pragma once
#include "mx4.cuh"
#include "rules.cuh"

namespace dllm {
namespace shaped {

constexpr int kEpiWarps = 8;
using lm::Outputs;
using lm::Plan;
using lm::RowState;
using lm::Unit;

struct Bf16 {
  static constexpr bool kMx4 = false;
  static constexpr int BN = 256;        // vocabulary entries per tile
  static constexpr int BK = 64;         // K per stage: 128 bytes
  static constexpr int UK = 16;         // K per tcgen05.mma
  static constexpr int SFA = 0, SFB = 0, kSfCols = 0, kSfRing = 0;
};
struct Mx4 {
  static constexpr bool kMx4 = true;
  static constexpr int BN = 192;
  static constexpr int BK = 256;
  static constexpr int UK = 64;
  static constexpr int SFA = 1024;      // scale bytes per stage: 128 rows of Hm, 8 blocks
  static constexpr int SFB = 2048;      // 256 rows of W
  static constexpr int kSfCols = 24;    // TMEM columns of one stage's scales
  static constexpr int kSfRing = 5;     // stages whose scales TMEM holds
};

// Warps: TMA, MMA, two idle (an epilogue warp's number gives its TMEM lane quadrant), epilogue.
constexpr int kEpiFirst = 4;
constexpr int kThreads = 32 * (kEpiFirst + kEpiWarps);

// Shared memory: barriers and flags, two blocks of row states (the halves of a tile meet there),
// per epilogue warp the additive rules of its half of a tile, then the ring.
constexpr int kMaxStages = 8;
constexpr int kHeadBytes = 512;
constexpr int kCombBytes = 2 * 128 * 20;
constexpr int kSmemBytes = 232448;                   // all of a CTA's 227 KB
template <class Op>
constexpr int ring_offset() {
  return (kHeadBytes + kCombBytes + kEpiWarps * (Op::BN / 2) * 4 + 1023) / 1024 * 1024;
}

template <int CG, class Op>
struct Cfg {
  static constexpr int BM_CTA = 128;                 // rows per CTA (TMEM lanes)
  static constexpr int BM = BM_CTA * CG;             // rows per m-tile
  static constexpr int B_ROWS = Op::BN / CG;         // W rows staged per CTA per stage
  static constexpr int A_BOX = 32 * 128;             // 32 rows of Hm
  static constexpr int B_BYTES = B_ROWS * 128;
  static_assert(B_BYTES % 1024 == 0, "B tiles start on swizzle atoms");
  static_assert(2 * Op::BN + Op::kSfRing * Op::kSfCols <= 512, "exceeds TMEM");
  static constexpr int kGroupM = CG == 1 ? DLLM_GROUP_M1 : DLLM_GROUP_M2;
  // Instruction descriptors.  kind::f16: fp32 accumulator (bits 4-5 = 1), A and B bf16 (bits
  // 7-9, 10-12 = 1).  kind::mxf4: A and B E2M1 (bits 7-9, 10-11 = 1), E8M0 scales (bit 23), the
  // scale bytes used of each TMEM word (bits 4-5 for B, 29-30 for A: 0 or 2).  Both K-major, N >> 3
  // at bits 17-22, M >> 4 at bits 24-28.
  static constexpr uint32_t kIdesc =
      (Op::kMx4 ? (1u << 7) | (1u << 10) | (1u << 23) : (1u << 4) | (1u << 7) | (1u << 10)) |
      (static_cast<uint32_t>(Op::BN >> 3) << 17) | (static_cast<uint32_t>(BM >> 4) << 24);
};

// lm::Plan counts vocabulary tiles of lm::BN columns; a V that has as many of those as the real
// one has tiles of Op::BN.
template <class Op>
__host__ __device__ inline int plan_v(int V) {
  return (V + Op::BN - 1) / Op::BN * lm::BN;
}

// The step of the walk over the vocabulary tiles: coprime to their number, about 0.62 of it.
inline int tile_step(int tiles) {
  int step = static_cast<int>(0.6180339887 * tiles);
  for (step = step < 1 ? 1 : step;; ++step) {
    int a = step, b = tiles;
    while (b != 0) {
      const int t = a % b;
      a = b;
      b = t;
    }
    if (a == 1) return step;
  }
}

// ---- MXFP4 tensor-core wrappers ---------------------------------------------------------
// D (+)= (A * scales) * (B * scales)^T, block scaled, 32 elements per scale.
template <int CG>
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// One scale tile (512 bytes: 32 rows of 16) from shared memory to 4 TMEM columns, in each lane
// quadrant; with CG = 2 in both CTAs of the pair, each from its own shared memory.
template <int CG>
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Shared-memory descriptor of a scale tile: no swizzle, 8 rows of 16 bytes contiguous, 128
// bytes from one such group to the next.
__device__ __forceinline__ uint64_t scale_desc(uint32_t smem_addr) {
  return static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128u >> 4) << 32) |
         (static_cast<uint64_t>(1u) << 46);
}

// Registers of a thread, moved between the warpgroups of a CTA (bf16): 384 threads start with
// kLaunchRegs each (the host checks that the build has them).
#ifndef DLLM_SHAPED_LAUNCH_REGS
#define DLLM_SHAPED_LAUNCH_REGS 168                  // other values: a test of the host's check
#endif
constexpr int kLaunchRegs = DLLM_SHAPED_LAUNCH_REGS, kProducerRegs = 72, kEpilogueRegs = 216;
static_assert(kProducerRegs + 2 * kEpilogueRegs <= 3 * kLaunchRegs, "more registers than the launch has");
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Addresses in shared memory.  A stage: [Hm rows | W rows | scales of Hm | scales of W].
template <int CG, class Op>
struct Smem {
  using C = Cfg<CG, Op>;
  uint64_t *full, *empty;                            // per stage
  uint64_t *tfull, *tempty, *drain, *epi_bar, *tready;
  uint32_t* tmem_slot;
  int* abort_flag;
  volatile int* last_flag;
  struct RowStateRaw { float m, s, t, m2; int a; };
  RowStateRaw* comb;
  float* add;
  uint8_t* ring;
  static constexpr uint32_t kA = 4 * C::A_BOX, kStageBytes = kA + C::B_BYTES + Op::SFA + Op::SFB;
  static constexpr int kFit = (kSmemBytes - 1024 - ring_offset<Op>()) / static_cast<int>(kStageBytes);
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;

  __device__ __forceinline__ explicit Smem(uint8_t* raw) {
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    full = reinterpret_cast<uint64_t*>(base);
    empty = full + kMaxStages;
    tfull = empty + kMaxStages;
    tempty = tfull + 2;
    drain = tfull + 4;
    epi_bar = tfull + 5;
    tready = tfull + 6;
    tmem_slot = reinterpret_cast<uint32_t*>(tfull + 7);
    abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
    last_flag = abort_flag + 1;
    comb = reinterpret_cast<RowStateRaw*>(base + kHeadBytes);
    add = reinterpret_cast<float*>(base + kHeadBytes + kCombBytes);
    ring = base + ring_offset<Op>();
  }
  __device__ __forceinline__ uint32_t a(int s) const { return smem_u32(ring) + s * kStageBytes; }
  __device__ __forceinline__ uint32_t b(int s) const { return a(s) + kA; }
  __device__ __forceinline__ uint32_t sfa(int s) const { return b(s) + C::B_BYTES; }
  __device__ __forceinline__ uint32_t sfb(int s) const { return sfa(s) + Op::SFA; }
};

// The MMA warp waits for the release of the stage whose scale columns it is about to rewrite; with
// fewer stages than that the barrier could be a whole turn ahead.
static_assert(Smem<1, Mx4>::kStages >= Mx4::kSfRing && Smem<2, Mx4>::kStages >= Mx4::kSfRing,
              "the ring is shorter than the scales' ring");

// Position in the ring: stage, and the parity of its current use.
struct Turn {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      ph ^= 1u;
    }
  }
};

struct Maps {
  const CUtensorMap* a;      // Hm (or its codes): box of 32 rows (CG = 1) or 128 (CG = 2)
  const CUtensorMap* b;      // W (or its codes): box of Op::BN / CG rows
  const CUtensorMap* sa;     // scales of Hm: box of one tile row, 1024 bytes
  const CUtensorMap* sb;     // scales of W: box of two tile rows, 1024 bytes
};

struct Problem {
  int n_cap, V, d, L;
  int tile_step;             // order of the vocabulary tiles
  const int* row_idx;
  float4* part;              // per (split, row): m, s, t, m2
  int* part_a;               // and the argmax
  long long part_cap;
  int* unit_ctr;
  Outputs out;
  int* status;
};

// Add one to a counter with release and acquire order.
__device__ __forceinline__ int count_unit(int* ctr) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(ctr) : "memory");
  return old;
}

// The partials of one row in slots i0, i0 + step, .. below i1 (streams 0 .. P - 1, then remainder
// holders from j_lo), merged four at a time: the next four are on their way meanwhile, and the
// four's sums are taken against their maximum, so that no partial waits for another.  A short
// loop, out of line: it runs once at the end of a launch, from a cold instruction cache (unrolled
// to 8 or 18 partials the merge of 72 x 128 took 12 and 10 us).
template <bool kExt>
__device__ __noinline__ RowState merge_slots(const float4* part, const int* part_a, long long base,
                                             long long stride, int i0, int i1, int step, int P, int j_lo) {
  constexpr int kRound = 4;
  RowState acc;
  acc.reset();
  float4 v[kRound], next[kRound];                // m, s, t, m2
  int a[kRound], next_a[kRound];
#pragma unroll
  for (int k = 0; k < kRound; ++k) {
    v[k] = make_float4(-INFINITY, 0.f, 0.f, -INFINITY);
    a[k] = 0;
  }
#pragma unroll 1
  for (int i = i0; i < i1 + kRound * step; i += kRound * step) {     // the last turn merges the rest
#pragma unroll
    for (int k = 0; k < kRound; ++k) {
      const int slot = i + k * step;
      const long long e = base + (slot < P ? slot : slot + j_lo) * stride;
      next[k] = make_float4(-INFINITY, 0.f, 0.f, -INFINITY);
      next_a[k] = 0;
      if (slot < i1) {
        next[k] = __ldcg(part + e);
        next_a[k] = __ldcg(part_a + e);
      }
    }
    float m = acc.m;
#pragma unroll
    for (int k = 0; k < kRound; ++k) {
      if constexpr (kExt) acc.m2 = fmaxf(fmaxf(acc.m2, v[k].w), fminf(m, v[k].x));
      m = fmaxf(m, v[k].x);
    }
    // nothing allowed anywhere yet: the sums are 0 (or NaN, which stays)
    const float shift = m == -INFINITY ? 0.f : m;
    const float f = ex2_approx((acc.m - shift) * lm::kLog2e);
    if constexpr (kExt) acc.t = f > 0.f ? f * (acc.t + (acc.m - shift) * acc.s) : 0.f;
    acc.s *= f;
    if (acc.m != m) acc.a = 0x7fffffff;
    acc.m = m;
#pragma unroll
    for (int k = 0; k < kRound; ++k) {
      const float d = v[k].x - shift, g = ex2_approx(d * lm::kLog2e);
      acc.s += v[k].x == -INFINITY ? v[k].y : v[k].y * g;
      if constexpr (kExt) acc.t += g > 0.f ? g * (v[k].z + d * v[k].y) : 0.f;
      if (v[k].x == m) acc.a = min(acc.a, a[k]);   // of equal maxima the lower token
      v[k] = next[k];
      a[k] = next_a[k];
    }
  }
  return acc;
}

template <int CG, class Op, bool kRules, bool kExt>
__device__ __forceinline__ void run(uint8_t* smem_raw, const Maps& tm, int count_raw, const Problem& p,
                                    const dllm_logit_rules& rule_set) {
  using C = Cfg<CG, Op>;
  constexpr int BN = Op::BN;
  count_raw = __shfl_sync(0xffffffffu, count_raw, 0);              // warp-uniform, and known to be
  const int count = count_raw < 0 ? 0 : (count_raw > p.n_cap ? p.n_cap : count_raw);
  const Smem<CG, Op> sm(smem_raw);
  constexpr int kStages = Smem<CG, Op>::kStages;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform
  const uint32_t rank = CG == 1 ? 0u : cluster_ctarank();
  const bool leader = rank == 0;
  int* const status = p.status;

  // TMEM, while the first loads are on their way; tready: both CTAs of a pair have theirs
  if (warp == 1) {
    if constexpr (CG == 1) {
      tmem_alloc(smem_u32(sm.tmem_slot), 512);
      tmem_relinquish();
      tc_fence_before();
      if (lane < 2) mbar_arrive(smem_u32(sm.tready));
    } else {
      tmem_alloc_pair(smem_u32(sm.tmem_slot), 512);
      tmem_relinquish_pair();
      tc_fence_before();
      if (lane < 2) mbar_arrive_cluster(smem_u32(sm.tready), lane);
    }
    __syncwarp();
  }
  volatile int* abort_flag = sm.abort_flag;

  const Plan pl = Plan::make(count, plan_v<Op>(p.V), static_cast<int>(gridDim.x) / CG, C::kGroupM, C::BM);
  const int holder = static_cast<int>(blockIdx.x) / CG;
  const int KB = (p.d + Op::BK - 1) / Op::BK;
  // Stages summed in one accumulator (bf16; MXFP4 a tile's whole K).  Single CTAs: 128 of K; W's
  // way from HBM hides most of the epilogue's extra reads (one row d4096 V126464: 192 us, with 256
  // of K 185, with 512 178, unsplit 173), and a call on few rows has no others for its error to
  // average with: of 40 random calls of 1 to 128 rows 5 came out more than 1e-6 off (256: 8, 512:
  // 13), as many as with plain fp32 sums.
  // Pairs: a quarter of K, at least 512: with it a normal row's error stays by that of an fp32 sum,
  // which grows with K too (d = 1024, 2048, 4096, 8192: 0.7, 0.7, 1.2, 2.7e-6; fp32 0.7, 0.7, 1.8,
  // 2.3e-6).  256 rows d2048 V151936 with all rules: 512 219 us, 768 209, 1024 188, unsplit 173;
  // 1024 rows d4096 V126464: 907, 876, 832, 800 us (both under the power cap).
  int piece_stages = KB;
  if (!Op::kMx4) {
    const int quarter = (KB + 3) / 4;
    const int most = CG == 1 ? 2 : (quarter < 8 ? 8 : quarter);
    const int pieces = (KB + most - 1) / most;
    piece_stages = (KB + pieces - 1) / pieces;
  }
  // the schedule's vocabulary tile i, in the order of the walk
  auto tile_at = [&](int i) {
    const unsigned n = static_cast<unsigned>(pl.numN), u = static_cast<unsigned>(i), v = static_cast<unsigned>(p.tile_step);
    return static_cast<int>(n < 65536u ? u * v % n : static_cast<unsigned>(static_cast<unsigned long long>(u) * v % n));
  };
  uint32_t armed_mask = 0, armed_parity = 0;      // as in lm::lmhead_run
  // TMEM's base address once it is allocated; false if the CTA is aborting
  uint32_t tmem_base = 0;
  auto wait_tmem = [&]() -> bool {
    const bool got = __all_sync(0xffffffffu, mbar_wait(smem_u32(sm.tready), 0u, abort_flag, status));
    tc_fence_after();
    tmem_base = __shfl_sync(0xffffffffu, *sm.tmem_slot, 0);
    return got;
  };

  if (warp < kEpiFirst) {
    if constexpr (!Op::kMx4) give_registers<kProducerRegs>();
    if (warp == 0 && lane == 0) {
      // ------------------------------ TMA producer ------------------------------
      Turn at;
#ifdef DLLM_FAULT_SKIP_STAGE
      uint32_t it = 0;
#endif
      constexpr int kPace = CG == 2 ? DLLM_PAIR_PACE : 0;      // see lm::lmhead_run
      constexpr int kMates = C::kGroupM;
      int* const progress = p.unit_ctr + ((p.n_cap + 127) / 128 + 2);
      int started = 0;
      int seen[kMates];
#pragma unroll
      for (int j = 0; j < kMates; ++j) seen[j] = 0;
      auto pace = [&](int m_tile) -> bool {
        if (kPace <= 0 || pl.ngroups < 2 || pl.rem || pl.gmax > kMates) return true;
        const int g = m_tile / pl.gmax;
        if (pl.group_size(g) != pl.gmax) return true;
        if (rank == 0) st_relaxed_gpu(progress + holder, started);
        const int first = (holder / pl.gmax) * pl.gmax;
        const int need = started - kPace;
        bool behind = false;
#pragma unroll
        for (int j = 0; j < kMates; ++j) behind |= j < pl.gmax && seen[j] < need;
        if (behind) {
          const unsigned long long t0 = globaltimer_ns();
          for (;;) {
            bool lag = false;
            for (int j = 0; j < pl.gmax; ++j) lag |= ld_relaxed_gpu(progress + first + j) < need;
            if (!lag) break;
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
              atomicOr(status, kStatusTimeout);
              *abort_flag = 1;
              return false;
            }
            __nanosleep(128);
          }
        }
#pragma unroll
        for (int j = 0; j < kMates; ++j)
          if (j < pl.gmax) seen[j] = ld_relaxed_gpu(progress + first + j);
        return true;
      };
      auto load_tile = [&](int m_tile, int i) -> bool {
        if (!pace(m_tile)) return false;
        const int n = tile_at(i);
        ++started;
        const int a_row = m_tile * C::BM + static_cast<int>(rank) * C::BM_CTA;
        const int b_row = n * BN + static_cast<int>(rank) * C::B_ROWS;
        const int valid = count - a_row;
        const int boxes = valid >= C::BM_CTA ? 4 : (valid + 31) / 32;          // CG = 1: valid >= 1
        for (int kb = 0; kb < KB; ++kb, at.next(kStages)) {
          const int s = at.s;
          const uint32_t ph = at.ph;
          if (!mbar_wait(smem_u32(&sm.empty[s]), ph ^ 1u, abort_flag, status)) return false;
#ifdef DLLM_FAULT_SKIP_STAGE
          // Failure-detection test builds only: this stage is never armed or loaded.
          if (it++ == DLLM_FAULT_SKIP_STAGE) continue;
#endif
          const uint32_t fb = smem_u32(&sm.full[s]);
          armed_mask |= 1u << s;
          armed_parity = (armed_parity & ~(1u << s)) | (ph << s);
          // x: elements of the map's type (bf16, bytes of codes, 8-byte words of scales)
          const int x = kb * (Op::kMx4 ? 128 : 64);
          const uint32_t da = sm.a(s), db = sm.b(s);
          if constexpr (CG == 1) {
            mbar_arrive_expect_tx(fb, boxes * C::A_BOX + C::B_BYTES + Op::SFA + Op::SFB);
            for (int j = 0; j < boxes; ++j)
              tma_load_2d(da + j * C::A_BOX, tm.a, fb, x, a_row + 32 * j);
            tma_load_2d(db, tm.b, fb, x, b_row);
            if constexpr (Op::kMx4) {
              tma_load_2d(sm.sfa(s), tm.sa, fb, x, a_row / 128);
              tma_load_2d(sm.sfb(s), tm.sb, fb, x, n * BN / 128);
            }
          } else {
            if (leader) mbar_arrive_expect_tx(fb, CG * (4 * C::A_BOX + C::B_BYTES + Op::SFA + Op::SFB));
            const uint32_t fl = fb & kPeerBitMask;
            tma_load_2d_pair(da, tm.a, fl, x, a_row);
            tma_load_2d_pair(db, tm.b, fl, x, b_row);
            if constexpr (Op::kMx4) {          // both CTAs of a pair need all of the tile's scales
              tma_load_2d_pair(sm.sfa(s), tm.sa, fl, x, a_row / 128);
              tma_load_2d_pair(sm.sfb(s), tm.sb, fl, x, n * BN / 128);
            }
          }
        }
        return true;
      };
      lm::for_each_tile(pl, holder, load_tile);
    } else if (warp == 1 && leader) {
      // ------------------------------ MMA issuer --------------------------------
      Turn at, sat, old;          // places in the ring and the scales' ring; the stage whose scale
      int ahead = 0;              // columns come next
      uint32_t piece = 0;
      auto mma_tile = [&](int, int i) -> bool {
        const int n = tile_at(i);
        for (int kb = 0, kp = 0; kb < KB; ++kb) {                // kp: stage within its accumulator
          const uint32_t buf = piece & 1u;
          const uint32_t d_tmem = tmem_base + buf * BN;
          if (kp == 0) {
            const uint32_t ph = (piece >> 1) & 1u;
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.tempty[buf]), ph ^ 1u, abort_flag, status)))
              return false;
            tc_fence_after();
          }
          bool got = mbar_wait(smem_u32(&sm.full[at.s]), at.ph, abort_flag, status);
          if constexpr (Op::kMx4) {
            if (ahead < Op::kSfRing) {
              ++ahead;
            } else {              // the MMAs that read these scale columns are done
              got = got && mbar_wait(smem_u32(&sm.empty[old.s]), old.ph, abort_flag, status);
              old.next(kStages);
            }
          }
          if (!__all_sync(0xffffffffu, got)) return false;
          tc_fence_after();
          const uint64_t adesc = sw128_kmajor_desc(sm.a(at.s));
          const uint64_t bdesc = sw128_kmajor_desc(sm.b(at.s));
          const uint32_t empty = smem_u32(&sm.empty[at.s]);
          if constexpr (!Op::kMx4) {
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < Op::BK / Op::UK; ++k)
                lm::mma_issue<CG>(d_tmem, adesc + 2 * k, bdesc + 2 * k, C::kIdesc, (kp | k) != 0 ? 1u : 0u);
              lm::mma_commit_all<CG>(empty);            // stage free once these MMAs retire
            }
          } else {
            // d is a multiple of 64, so the last stage holds 1 to 4 steps of K = 64; a scale tile
            // covers two of them (bytes 0, 1 and 2, 3 of its words)
            const int left = (p.d - kb * Op::BK) / Op::UK;
            const uint32_t sf = tmem_base + 2 * BN + sat.s * Op::kSfCols;
            const uint32_t sfb = sf + 8 + ((n * BN) % 128 != 0 ? 2 : 0);
            const uint64_t sa = scale_desc(sm.sfa(at.s)), sb = scale_desc(sm.sfb(at.s));
            if (elect_one()) {
              auto copy = [&](int g) {
                tmem_cp_scales<CG>(sf + 4 * g, sa + 32 * g);                  // 512 bytes apart
                tmem_cp_scales<CG>(sf + 8 + 8 * g, sb + 32 * g);
                tmem_cp_scales<CG>(sf + 8 + 8 * g + 4, sb + 64 + 32 * g);
              };
              auto mma = [&](int k) {
                umma_mxf4<CG>(d_tmem, adesc + 2 * k, bdesc + 2 * k,
                              C::kIdesc | ((k & 1) ? (2u << 4) | (2u << 29) : 0u), sf + 4 * (k >> 1),
                              sfb + 8 * (k >> 1), (kb | k) != 0 ? 1u : 0u);
              };
              if (left >= 4) {
                copy(0);
                copy(1);
#pragma unroll
                for (int k = 0; k < 4; ++k) mma(k);
              } else {
                copy(0);
                mma(0);
                if (left > 1) mma(1);
                if (left > 2) {
                  copy(1);
                  mma(2);
                }
              }
              lm::mma_commit_all<CG>(empty);
            }
            sat.next(Op::kSfRing);
          }
          __syncwarp();
          at.next(kStages);
          if (++kp == piece_stages || kb == KB - 1) {
            if (elect_one()) lm::mma_commit_all<CG>(smem_u32(&sm.tfull[buf]));   // accumulator ready
            __syncwarp();
            ++piece;
            kp = 0;
          }
        }
        return true;
      };
      if (!wait_tmem() || !lm::for_each_tile(pl, holder, mma_tile)) {
        if (elect_one()) {
          lm::mma_commit_all<CG>(smem_u32(sm.drain));       // no MMA may outlive TMEM
          mbar_wait_drain(smem_u32(sm.drain), 0u, status);
        }
        __syncwarp();
      }
    }
  } else {
    if constexpr (!Op::kMx4) take_registers<kEpilogueRegs>();
    // -------------------------------- epilogue ---------------------------------
    const int q = warp & 3;                      // TMEM lane quadrant of this warp
    const int half = (warp - kEpiFirst) >> 2;            // which half of a tile's columns
    constexpr int kChunks = BN / 64;             // 32-column chunks of a half
    const int row_in_cta = q * 32 + lane;
    const int row_in_tile = static_cast<int>(rank) * C::BM_CTA + row_in_cta;
    bool ok = wait_tmem();
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + half * (BN / 2);
    uint32_t piece = 0, epi_phase = 0, units_done = 0;
    bool live = false;                // live: this warp holds a masked row of the m-tile
    rules::RowRules rr = rules::no_rules();
    // rules: whether all of the warp's rows share them (rules::shape_same), and the additive part
    // of this warp's columns of the current tile
    bool same = false;
    float* const add = sm.add + (warp - kEpiFirst) * (BN / 2);
    const bool has_add = kRules && (rule_set.bias != nullptr || rule_set.counts != nullptr);
    auto enter_m_tile = [&](int m_tile) {
      const int row = m_tile * C::BM + row_in_tile;
      live = row - lane < count;
      if constexpr (kRules) {
        if (live) {                              // lanes past the last row take its rules
          rr = rules::row_rules(rule_set, p.row_idx[row < count ? row : count - 1], p.L, status);
          const float* b0 = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(rr.bias), 0));
          const int* c0 = reinterpret_cast<const int*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(rr.counts), 0));
          same = __all_sync(0xffffffffu, rr.bias == b0 && rr.counts == c0);
        }
      }
    };
    // What the rules of a tile read, fetched while the tile before it is worked on: the bitmap
    // words, and (rows alike) lane j's bias and count of column j of each chunk.
    struct Fetched {
      rules::Words w[kChunks];
      float bias[kChunks];
      int c[kChunks];
    };
    auto fetch = [&](int n, Fetched& f) {
      if constexpr (kRules) {
        const int first = n * BN + half * (BN / 2);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const int col = first + 32 * c + lane;
          f.w[c] = rules::load_words(first + 32 * c, p.V, rr);
          f.bias[c] = 0.f;
          f.c[c] = 0;
          if (same && col < p.V) {
            if (rr.bias) f.bias[c] = __uint_as_float(rules::load_now(rr.bias + col));
            if (rr.counts) f.c[c] = static_cast<int>(rules::load_now(rr.counts + col));
          }
        }
      }
    };
    // ... becomes the current tile's: words in registers, the additive parts in shared memory
    rules::Words words[kChunks] = {};
    auto settle = [&](const Fetched& f) {
      if constexpr (kRules) {
        __syncwarp();                            // no lane still reads the tile before
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          words[c] = f.w[c];
          if (same && has_add)
            add[32 * c + lane] = rules::additive(f.bias[c], f.c[c], (f.w[c].seen >> lane) & 1u, rr);
        }
        __syncwarp();
      }
    };
    // all epilogue warps meet; false (warp-uniform) if the CTA is aborting
    auto epi_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(sm.epi_bar));
      const bool got = mbar_wait(smem_u32(sm.epi_bar), epi_phase, abort_flag, status);
      epi_phase ^= 1u;
      return __all_sync(0xffffffffu, got);
    };
    // the next accumulator; false (warp-uniform) if the CTA is aborting
    auto wait_piece = [&]() -> bool {
      const bool got = mbar_wait(smem_u32(&sm.tfull[piece & 1u]), (piece >> 1) & 1u, abort_flag, status);
      if (!__all_sync(0xffffffffu, got)) return false;
      tc_fence_after();
      return true;
    };
    // release it: the leader's MMA waits for the epilogues of both CTAs
    auto release_piece = [&]() {
      tc_fence_before();
      __syncwarp();
      const uint32_t bar = smem_u32(&sm.tempty[piece & 1u]);
      if constexpr (CG == 2) {
        if (lane == 0) mbar_arrive_cluster(bar, 0u);
      } else {
        if (lane < 2) mbar_arrive(bar);          // twice: the barrier counts both CTAs of a pair
      }
      ++piece;
    };
    // shape 32 logits (chunk c of the tile, columns col0 ..) and fold them into st
    auto take = [&](float (&v)[32], int c, int col0, const rules::Words& w, rules::State& st) {
      if constexpr (kRules) {
        if (__reduce_or_sync(0xffffffffu, w.ok) == 0u) return;
        if (same) rules::shape_same(v, rr, w, has_add ? add + 32 * c : nullptr);
        else rules::shape_mixed(v, col0, p.V, rr, w);
      } else if (col0 + 32 > p.V) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (col0 + j >= p.V) v[j] = -INFINITY;
      }
      rules::fold<kExt>(v, col0, st);
    };
    // fold this warp's half of vocabulary tile n into st; the unit's next tile is `next` (-1: none)
    auto consume = [&](int n, int next, rules::State& st) -> bool {
      const int first = n * BN + half * (BN / 2);
      Fetched f;
      if constexpr (Op::kMx4) {
        if (!wait_piece()) return false;
        if (live) {
          if (next >= 0) fetch(next, f);
          const uint32_t taddr = lane_base + (piece & 1u) * BN;
#pragma unroll 1
          for (int c = 0; c < kChunks; ++c) {
            float v[32];
            tmem_ld32(taddr + c * 32, v);
            const rules::Words w = words[0];
#pragma unroll
            for (int k = 1; k < kChunks; ++k) words[k - 1] = words[k];   // the next chunk's
            tmem_ld_wait();
            take(v, c, first + 32 * c, w, st);
          }
        }
        release_piece();
      } else {
        float acc[kChunks][32];
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c][j] = 0.f;
#pragma unroll 1
        for (int kb = 0; kb < KB; kb += piece_stages) {
          if (!wait_piece()) return false;
          if (live) {
            const uint32_t taddr = lane_base + (piece & 1u) * BN;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              float v[32];
              tmem_ld32(taddr + c * 32, v);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                const float2 y = rules::add2(make_float2(acc[c][j], acc[c][j + 1]), make_float2(v[j], v[j + 1]));
                acc[c][j] = y.x;
                acc[c][j + 1] = y.y;
              }
            }
          }
          release_piece();
        }
        if (live) {
          if (next >= 0) fetch(next, f);
#pragma unroll 1
          for (int c = 0; c < kChunks; ++c) {
            take(acc[0], c, first + 32 * c, words[0], st);
#pragma unroll
            for (int k = 1; k < kChunks; ++k) {                          // the next chunk's
              words[k - 1] = words[k];
#pragma unroll
              for (int j = 0; j < 32; ++j) acc[k - 1][j] = acc[k][j];
            }
          }
        }
      }
      if (live && next >= 0) settle(f);
      return true;
    };
    auto write_result = [&](int row, const RowState& st) {
      int t;
      float c, l, e, mg;
      rules::finish(st, t, c, l, e, mg);
      p.out.tok[row] = t;
      p.out.conf[row] = c;
      p.out.lse[row] = l;
      if constexpr (kExt) {
        if (p.out.entropy) p.out.entropy[row] = e;
        if (p.out.margin) p.out.margin[row] = mg;
      }
    };
    auto put = [&](int block, int r, const RowState& st) {
      auto& c = sm.comb[block * C::BM_CTA + r];
      c.m = st.m;
      c.s = st.s;
      c.t = st.t;
      c.m2 = st.m2;
      c.a = st.a;
    };
    auto join = [&](int block, int r, RowState& st) {
      const auto& c = sm.comb[block * C::BM_CTA + r];
      rules::merge<kExt>(st, c.m, c.s, c.a, c.t, c.m2);
    };
    // A finished (m-tile, slot): the two halves' states are joined; the result itself when the
    // m-tile has a single unit, else a partial; the last of the m-tile's units to finish merges
    // its rows.
    auto finish = [&](int g, const Unit& u, int m_local, int slot, const rules::State& part_st) -> bool {
      const int m_tile = g * pl.gmax + m_local;
      const int row = m_tile * C::BM + row_in_tile;
      const bool valid = row < count;
      int j_lo = 0, j_hi = -1;
      if (pl.rem) pl.leftovers_of(m_local, u.G, j_lo, j_hi);
      const int units = u.P + (j_hi >= j_lo ? j_hi - j_lo + 1 : 0);
      RowState st = part_st.value();
      // two blocks in turn: the next unit's states may be written while these are still read
      const int block = units_done++ & 1;
      if (half == 1) put(block, row_in_cta, st);
      if (!epi_sync()) return false;
      if (half == 0) join(block, row_in_cta, st);
      if (units == 1) {
        if (half == 0 && valid) write_result(row, st);
        return true;
      }
      if (half == 0 && valid) {
        const long long e = pl.part_index(g, u.G, slot, m_local * C::BM + row_in_tile);
        if (e < p.part_cap) {
          p.part[e] = make_float4(st.m, st.s, st.t, st.m2);
          p.part_a[e] = st.a;
        } else {
          atomicOr(status, kStatusBounds);             // cannot happen: workspace sized for it
        }
      }
      // Once all partials are written, one thread counts the unit (releasing the whole CTA's writes,
      // which the meeting put before it); the last unit's CTA reads them through L2.
      if (!epi_sync()) return false;
      if (threadIdx.x == kEpiFirst * 32) {
        const int old = count_unit(&p.unit_ctr[m_tile * CG + static_cast<int>(rank)]);
        *sm.last_flag = old == units - 1 ? 1 : 0;
      }
      if (!epi_sync()) return false;
      if (!*sm.last_flag) return true;
      const int row0 = m_tile * C::BM + static_cast<int>(rank) * C::BM_CTA;   // CTA's first row
      const int n_valid = count - row0 < C::BM_CTA ? count - row0 : C::BM_CTA;
      const long long base0 = pl.part_index(g, u.G, 0, m_local * C::BM + static_cast<int>(rank) * C::BM_CTA);
      const long long stride = static_cast<long long>(u.G) * C::BM;
      if (n_valid <= 32) {
        for (int r = warp - kEpiFirst; r < n_valid; r += kEpiWarps) {
          RowState acc = merge_slots<kExt>(p.part, p.part_a, base0 + r, stride, lane, units, 32, u.P, j_lo);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const float m = __shfl_xor_sync(0xffffffffu, acc.m, o), s = __shfl_xor_sync(0xffffffffu, acc.s, o);
            const int a = __shfl_xor_sync(0xffffffffu, acc.a, o);
            const float t = kExt ? __shfl_xor_sync(0xffffffffu, acc.t, o) : 0.f;
            const float m2 = kExt ? __shfl_xor_sync(0xffffffffu, acc.m2, o) : 0.f;
            rules::merge<kExt>(acc, m, s, a, t, m2);
          }
          if (lane == 0) write_result(row0 + r, acc);
        }
      } else {
        // each warp takes half of the slots, of its own quadrant's rows; the halves meet as above
        const int mid = units / 2, next_block = units_done++ & 1;
        RowState acc;
        acc.reset();
        if (valid)
          acc = merge_slots<kExt>(p.part, p.part_a, base0 + row_in_cta, stride, half ? mid : 0,
                                  half ? units : mid, 1, u.P, j_lo);
        if (half == 1) put(next_block, row_in_cta, acc);
        if (!epi_sync()) return false;
        if (half == 0 && valid) {
          join(next_block, row_in_cta, acc);
          write_result(row, acc);
        }
      }
      return true;
    };

    for (int g = 0; g < pl.ngroups && ok; ++g) {
      Unit u;
      if (!lm::unit_of(pl, g, holder, u)) continue;
      // a stream's tiles, or remainder tiles in m-major order: one running state, finished where
      // the m-tile changes
      const int n_tiles = u.leftover ? static_cast<int>(u.i1 - u.i0) : u.n1 - u.n0;
      rules::State st;
      int m_local = u.leftover ? static_cast<int>(u.i0 / pl.rr) : u.m_local;
      bool fresh = true;
      for (int j = 0; j < n_tiles && ok; ++j) {
        int i = u.n0 + j, i_next = i + 1, next_m = m_local;
        if (u.leftover) {
          i = u.P * pl.rb + static_cast<int>((u.i0 + j) % pl.rr);
          i_next = u.P * pl.rb + static_cast<int>((u.i0 + j + 1) % pl.rr);
          next_m = static_cast<int>((u.i0 + j + 1) / pl.rr);
        }
        const int n = tile_at(i);
        const bool last = j + 1 == n_tiles || next_m != m_local;
        if (fresh) {
          st.reset();
          enter_m_tile(g * pl.gmax + m_local);
          if (live) {
            Fetched f;
            fetch(n, f);
            settle(f);
          }
          fresh = false;
        }
        ok = consume(n, last ? -1 : tile_at(i_next), st);
        if (ok && last) {
          ok = finish(g, u, m_local, u.p, st);
          m_local = next_m;
          fresh = true;
        }
      }
    }
  }

  tc_fence_before();
  if constexpr (CG == 1) __syncthreads();
  else cluster_sync();          // neither CTA leaves while its peer may still touch its smem
  bool aborted = *abort_flag != 0;
  if constexpr (CG == 2) {
    aborted = aborted || ld_shared_cluster_s32(smem_u32(sm.abort_flag), rank ^ 1u) != 0;
    cluster_sync();             // the peer's shared memory stays alive until both have read
  }
  if (aborted) {                // loads already issued land before shared memory is released
    if (warp == 0 && lane == 0 && leader) {
      const unsigned long long deadline = globaltimer_ns() + kWaitLimitNs;
      for (int s = 0; s < kStages; ++s)
        if (armed_mask & (1u << s))
          if (!mbar_wait_until(smem_u32(&sm.full[s]), (armed_parity >> s) & 1u, deadline, status)) break;
    }
    if constexpr (CG == 1) __syncthreads();
    else cluster_sync();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_base = __shfl_sync(0xffffffffu, *sm.tmem_slot, 0);
    if constexpr (CG == 1) tmem_dealloc(tmem_base, 512);
    else tmem_dealloc_pair(tmem_base, 512);
  }
}

// Launched in clusters of two CTAs; variant 0 chooses the body from the masked count as
// lm::lmhead_auto_kernel does, 1 and 2 force it (test hook).
template <class Op, bool kRules, bool kExt>
__global__ void __launch_bounds__(kThreads, 1)
shaped_kernel(const __grid_constant__ CUtensorMap tmA1, const __grid_constant__ CUtensorMap tmA2,
              const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ CUtensorMap tmB2,
              const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
              const int* __restrict__ count_ptr, int variant, const Problem p,
              const __grid_constant__ dllm_logit_rules rule_set) {
  extern __shared__ uint8_t smem_raw[];
  // What no variant changes is set up while the staging kernel still runs.
  const Smem<1, Op> sm(smem_raw);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sm.tfull[b]), 1);
      mbar_init(smem_u32(&sm.tempty[b]), 2 * kEpiWarps);
    }
    mbar_init(smem_u32(sm.drain), 1);
    mbar_init(smem_u32(sm.epi_bar), kEpiWarps);
    mbar_init(smem_u32(sm.tready), 2);
    *sm.abort_flag = 0;
    fence_mbar_init();
  } else if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmA1);
    tma_prefetch_desc(&tmA2);
    tma_prefetch_desc(&tmB1);
    tma_prefetch_desc(&tmB2);
    if constexpr (Op::kMx4) {
      tma_prefetch_desc(&tmSA);
      tma_prefetch_desc(&tmSB);
    }
  }
  // rows of Hm that single CTAs do not load count as zero; the loads (asynchronous proxy) come after
  for (int s = 0; s < sm.kStages; ++s)
    for (uint32_t i = threadIdx.x; i < sm.kA / 16; i += kThreads)
      reinterpret_cast<uint4*>(sm.ring + s * sm.kStageBytes)[i] = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  cluster_sync();               // barriers of both CTAs initialised before any remote use
  pdl_wait();
  pdl_launch_dependents();
  const int c = *count_ptr;
  if ((variant == 0 ? lm::auto_variant(c) : variant) == 2)
    run<2, Op, kRules, kExt>(smem_raw, Maps{&tmA2, &tmB2, &tmSA, &tmSB}, c, p, rule_set);
  else
    run<1, Op, kRules, kExt>(smem_raw, Maps{&tmA1, &tmB1, &tmSA, &tmSB}, c, p, rule_set);
}

}  // namespace shaped
}  // namespace dllm
