// dllm_api.cu - the C ABI (include/dllm.h): argument validation, workspace layout, TMA
// tensor maps, launches on the caller's stream, device status word and kernel timing.
//
// All kernels are compiled in this one translation unit so that they share the device
// status word without relocatable device code.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstdio>
#include <mutex>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "dllm.h"
#include "ptx.cuh"
#include "compact.cuh"
#include "lmhead.cuh"
#include "merge.cuh"
#include "select.cuh"
#include "arena.cuh"
#include "mx4.cuh"
#include "rules.cuh"
#include "shaped.cuh"
#include "stage.cuh"

#ifndef DLLM_GATHER_HOST_CTAS
#define DLLM_GATHER_HOST_CTAS 1   // gather CTAs per SM when the rows come from host memory
#endif

namespace dllm {

// An NVTX range around each entry point of the ABI, named after it, so that a timeline
// profiler groups the kernels of one library call (header-only NVTX v3: without a tool
// attached a range costs a null-pointer check).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// Device-side error bits (kStatusTimeout, kStatusBounds, kStatusCapacity); one word per device.
__device__ int g_status;

namespace {

constexpr int kMaxDevices = 64;

struct DeviceState {
  bool ready = false;
  dllm_status err = DLLM_OK;
  int sms = 0;
  int pairs = 0;                // co-resident CTA pairs of the cta_group::2 GEMM
  bool shaped_bf16 = false;     // the bf16 kernels of shaped.cuh may run (see device_state)
  int* status = nullptr;        // device address of g_status on this device
};

// GEMM variant: 2 = CTA pairs (cta_group::2, 256x256 tiles), 1 = single CTAs
// (cta_group::1, 128x256 tiles), both forced (test hook).  0 = default: chosen on the
// device from the masked count (lm::auto_variant): single CTAs for one m-tile of at most
// 128 rows (a pair would compute 128 empty rows), CTA pairs above (per SM a third fewer
// bytes staged from L2 per flop, which sets the clock under the 1 kW power cap).
std::atomic<int> g_gemm_variant{0};

std::mutex g_mu;
DeviceState g_dev[kMaxDevices];

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

// Kernel-time accounting (dllm_prof_begin / dllm_prof_end).
struct Prof {
  bool on = false;
  std::vector<cudaEvent_t> ev;  // pairs: start, stop
  size_t used = 0;
  int gemm_launches = 0;
  std::atomic<int> kernel_launches{0};
};
Prof g_prof;

inline void count_launch(int n = 1) {
  if (g_prof.on) g_prof.kernel_launches += n;
}

// The event pair around a GEMM launch: records the first and hands out the second.
bool prof_gemm_start(cudaStream_t s, cudaEvent_t* stop) {
  if (!g_prof.on) return true;
  if (g_prof.used + 2 > g_prof.ev.size()) {
    for (int i = 0; i < 64; ++i) {
      cudaEvent_t e;
      if (cudaEventCreate(&e) != cudaSuccess) return false;
      g_prof.ev.push_back(e);
    }
  }
  cudaEventRecord(g_prof.ev[g_prof.used], s);
  *stop = g_prof.ev[g_prof.used + 1];
  g_prof.used += 2;
  return true;
}
void prof_gemm_stop(cudaStream_t s, cudaEvent_t stop) {
  if (!g_prof.on) return;
  cudaEventRecord(stop, s);
  g_prof.gemm_launches++;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Launch with programmatic stream serialization: the kernel may start while the previous
// kernel on the stream finishes; every kernel of this library waits for its predecessors
// (griddepcontrol.wait) before it touches global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Per-device setup, once: check the architecture, find g_status, raise the GEMM's shared
// memory limit, resolve the tensor-map encoder.
dllm_status device_state(DeviceState** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DLLM_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return DLLM_ERR_DEVICE;
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState& st = g_dev[dev];
  if (!st.ready) {
    st.err = DLLM_OK;
    cudaDeviceProp prop;
    if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) {
      st.err = DLLM_ERR_CUDA;
    } else if (prop.major != 10 || prop.minor != 0) {
      st.err = DLLM_ERR_DEVICE;
    } else {
      st.sms = prop.multiProcessorCount;
      void* p = nullptr;
      if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess) st.err = DLLM_ERR_CUDA;
      st.status = static_cast<int*>(p);
      const auto smem_attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
      if (st.err == DLLM_OK &&
          (cudaFuncSetAttribute(lm::lmhead_kernel<1, lm::kModeStats>, smem_attr, lm::Cfg<1>::SMEM_BYTES) ||
           cudaFuncSetAttribute(lm::lmhead_kernel<1, lm::kModeStatsExt>, smem_attr, lm::Cfg<1>::SMEM_BYTES) ||
           cudaFuncSetAttribute(lm::lmhead_kernel<1, lm::kModeDebugStore>, smem_attr, lm::Cfg<1>::SMEM_BYTES) ||
           cudaFuncSetAttribute(lm::lmhead_kernel<2, lm::kModeStats>, smem_attr, lm::Cfg<2>::SMEM_BYTES) ||
           cudaFuncSetAttribute(lm::lmhead_kernel<2, lm::kModeStatsExt>, smem_attr, lm::Cfg<2>::SMEM_BYTES) ||
           cudaFuncSetAttribute(lm::lmhead_kernel<2, lm::kModeDebugStore>, smem_attr, lm::Cfg<2>::SMEM_BYTES) ||
           cudaFuncSetAttribute(lm::lmhead_auto_kernel<lm::kModeStats>, smem_attr, lm::kAutoSmemBytes) ||
           cudaFuncSetAttribute(lm::lmhead_auto_kernel<lm::kModeStatsExt>, smem_attr, lm::kAutoSmemBytes) ||
           cudaFuncSetAttribute(lm::lmhead_auto_kernel<lm::kModeDebugStore>, smem_attr, lm::kAutoSmemBytes) ||
           cudaFuncSetAttribute(shaped::shaped_kernel<shaped::Bf16, true, false>, smem_attr, shaped::kSmemBytes) ||
           cudaFuncSetAttribute(shaped::shaped_kernel<shaped::Bf16, true, true>, smem_attr, shaped::kSmemBytes) ||
           cudaFuncSetAttribute(shaped::shaped_kernel<shaped::Mx4, true, false>, smem_attr, shaped::kSmemBytes) ||
           cudaFuncSetAttribute(shaped::shaped_kernel<shaped::Mx4, true, true>, smem_attr, shaped::kSmemBytes) ||
           cudaFuncSetAttribute(shaped::shaped_kernel<shaped::Mx4, false, false>, smem_attr, shaped::kSmemBytes) ||
           cudaFuncSetAttribute(shaped::shaped_kernel<shaped::Mx4, false, true>, smem_attr, shaped::kSmemBytes) ||
           cudaFuncSetAttribute(rules::token_count_kernel, smem_attr, rules::kCountMaxSlice * 4)))
        st.err = DLLM_ERR_CUDA;
      // the bf16 kernels of shaped.cuh deal their registers out anew: what the warpgroups take must be
      // what the launch gave them, or they would wait for the rest.  In a build that gives them
      // another number the calls that launch them are refused, and no others.
      cudaFuncAttributes fa0, fa1;
      if (st.err == DLLM_OK &&
          (cudaFuncGetAttributes(&fa0, shaped::shaped_kernel<shaped::Bf16, true, false>) ||
           cudaFuncGetAttributes(&fa1, shaped::shaped_kernel<shaped::Bf16, true, true>)))
        st.err = DLLM_ERR_CUDA;
      st.shaped_bf16 = st.err == DLLM_OK && fa0.numRegs == shaped::kLaunchRegs && fa1.numRegs == shaped::kLaunchRegs;
      if (st.err == DLLM_OK) {
        // how many CTA pairs of the paired GEMM can be resident at once (a persistent grid
        // larger than that would serialise)
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(2 * (st.sms / 2), 1, 1);
        cfg.blockDim = dim3(lm::kThreads, 1, 1);
        cfg.dynamicSmemBytes = lm::Cfg<2>::SMEM_BYTES;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, lm::lmhead_kernel<2, lm::kModeStats>, &cfg) != cudaSuccess)
          clusters = 0;
        st.pairs = clusters < lm::kMaxCtas / 2 ? clusters : lm::kMaxCtas / 2;
      }
      if (st.err == DLLM_OK && g_encode == nullptr) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || fn == nullptr)
          st.err = DLLM_ERR_CUDA;
        else
          g_encode = reinterpret_cast<EncodeTiledFn>(fn);
      }
    }
    st.ready = true;
  }
  if (st.err != DLLM_OK) return st.err;
  *out = &st;
  return DLLM_OK;
}

// Workspace layout for at most `rows` masked rows (rows = B*L: any mask):
// [tile counts | unit counters | gathered rows Hm | part_m | part_s | part_a | part_t | part_m2];
// with MXFP4 operands Hm holds the rows' codes, and their scales (hs_off) follow it.
struct WsLayout {
  size_t tiles_off, ctr_off, hm_off, hs_off, pm_off, ps_off, pa_off, pt_off, pm2_off, total;
  long long part_cap;
  long long rows;          // masked-row capacity: rows of Hm, and the GEMM's row bound
  int n_ctr;
};

WsLayout ws_layout(int B, int L, int d, int V, long long rows, bool mx4 = false) {
  WsLayout w{};
  const long long n = static_cast<long long>(B) * L;
  const long long ntiles = (n + kCompactTile - 1) / kCompactTile;
  if (rows > n) rows = n;
  if (rows < 1) rows = 1;
  w.rows = rows;
  // partial entries: worst case over the masked count (up to `rows`), the largest number of
  // work holders and either GEMM variant; fewer masked rows never need more.
  const lm::Plan w1 = lm::Plan::make(static_cast<int>(rows), V, lm::kMaxCtas, lm::Cfg<1>::kGroupM,
                                     lm::Cfg<1>::BM);
  const lm::Plan w2 = lm::Plan::make(static_cast<int>(rows), V, lm::kMaxCtas / 2, lm::Cfg<2>::kGroupM,
                                     lm::Cfg<2>::BM);
  const long long cap1 = w1.ngroups * static_cast<long long>(lm::kMaxCtas) * lm::Cfg<1>::BM;
  const long long cap2 = w2.ngroups * static_cast<long long>(lm::kMaxCtas / 2) * lm::Cfg<2>::BM;
  long long cap = cap1 > cap2 ? cap1 : cap2;
  // a masked count that fits one group may use remainder holders: (P + R) slots of G m-tiles,
  // with P * G + R <= holders and R < G <= gmax, so fewer than (holders + gmax^2) m-tile rows
  const long long r1 = (static_cast<long long>(lm::kMaxCtas) + lm::Cfg<1>::kGroupM * lm::Cfg<1>::kGroupM) *
                       lm::Cfg<1>::BM;
  const long long r2 = (static_cast<long long>(lm::kMaxCtas / 2) + lm::Cfg<2>::kGroupM * lm::Cfg<2>::kGroupM) *
                       lm::Cfg<2>::BM;
  if (r1 > cap) cap = r1;
  if (r2 > cap) cap = r2;
  if (cap < 1) cap = 1;
  w.part_cap = cap;
  // one counter per (m-tile, CTA of the pair): ceil(rows / 128) + 2 covers both variants;
  // then one progress word per work holder (the pair body's pacing), zeroed with them
  w.n_ctr = static_cast<int>((rows + 127) / 128 + 2 + lm::kMaxCtas);
  size_t off = 0;
  w.tiles_off = off; off = round_up(off + sizeof(int) * ntiles, 256);
  w.ctr_off = off;   off = round_up(off + sizeof(int) * static_cast<size_t>(w.n_ctr), 256);
  w.hm_off = off;    off = round_up(off + (mx4 ? static_cast<size_t>(rows) * d / 2
                                               : static_cast<size_t>(rows) * d * 2), 256);
  w.hs_off = off;    if (mx4) off = round_up(off + static_cast<size_t>(mx4::scale_bytes(rows, d)), 256);
  w.pm_off = off;    off = round_up(off + sizeof(float) * cap, 256);
  w.ps_off = off;    off = round_up(off + sizeof(float) * cap, 256);
  w.pa_off = off;    off = round_up(off + sizeof(int) * cap, 256);
  w.pt_off = off;    off = round_up(off + sizeof(float) * cap, 256);
  w.pm2_off = off;   off = round_up(off + sizeof(float) * cap, 256);
  w.total = off;
  return w;
}

// The layout a workspace of ws_bytes can hold: all B*L rows when it is at least the full
// layout, else the largest masked-row capacity whose layout fits (the total grows with the
// capacity), or rows = 0 when not even one row fits.
WsLayout ws_layout_for(int B, int L, int d, int V, size_t ws_bytes, bool mx4 = false) {
  const long long n = static_cast<long long>(B) * L;
  WsLayout full = ws_layout(B, L, d, V, n, mx4);
  if (ws_bytes >= full.total) return full;
  WsLayout one = ws_layout(B, L, d, V, 1, mx4);
  if (ws_bytes < one.total) {
    one.rows = 0;
    return one;
  }
  long long lo = 1, hi = n;                   // layout(lo) fits, layout(hi) does not
  while (hi - lo > 1) {
    const long long mid = lo + (hi - lo) / 2;
    if (ws_layout(B, L, d, V, mid, mx4).total <= ws_bytes) lo = mid;
    else hi = mid;
  }
  return ws_layout(B, L, d, V, lo, mx4);
}

// A step input (H or M) may live in device memory or in page-locked host memory that the
// device can read over PCIe (zero-copy: only the bytes the kernels touch cross the bus,
// e.g. just the masked rows of H).  Resolves the pointer the kernels use; pageable host
// memory is rejected (DLLM_ERR_MEMORY) because the device cannot read it.
dllm_status resolve_input(const void* p, const void** dev, bool* on_host = nullptr) {
  cudaPointerAttributes at{};
  if (on_host) *on_host = false;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();                       // clear the sticky-free error of the query
    return DLLM_ERR_MEMORY;
  }
  if (at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged) {
    *dev = p;
    return DLLM_OK;
  }
  if (at.type == cudaMemoryTypeHost && at.devicePointer != nullptr) {
    *dev = at.devicePointer;
    if (on_host) *on_host = true;
    return aligned16(*dev) ? DLLM_OK : DLLM_ERR_ALIGN;
  }
  return DLLM_ERR_MEMORY;
}

bool shapes_ok(int B, int L) {
  return B >= 1 && L >= 1 && static_cast<long long>(B) * L < (1ll << 31);
}

dllm_status launch_compact(const uint8_t* M, int B, int L, const int* win_lo, const int* win_hi,
                           int* row_idx, int* seq_off, int* count, int* tiles, int* status,
                           cudaStream_t s) {
  const long long n = static_cast<long long>(B) * L;
  const unsigned ntiles = static_cast<unsigned>((n + kCompactTile - 1) / kCompactTile);
  // a single tile needs no per-tile counts: its offset is 0
  if (ntiles > 1) {
    if (launch_pdl(compact_count_kernel, dim3(ntiles), dim3(kCompactThreads), 0, s, M, n, L, win_lo,
                   win_hi, tiles) != cudaSuccess)
      return DLLM_ERR_CUDA;
    count_launch();
  }
  const bool offsets = ntiles > static_cast<unsigned>(kCompactDirectTiles);
  if (offsets) {
    if (launch_pdl(compact_scan_kernel, dim3(1), dim3(kScanThreads), 0, s, tiles,
                   static_cast<int>(ntiles)) != cudaSuccess)
      return DLLM_ERR_CUDA;
    count_launch();
  }
  if (launch_pdl(compact_scatter_kernel, dim3(ntiles), dim3(kCompactThreads), 0, s, M, B, L, win_lo,
                 win_hi, (const int*)tiles, offsets, row_idx, seq_off, count, status) != cudaSuccess)
    return DLLM_ERR_CUDA;
  count_launch();
  return DLLM_OK;
}

dllm_status make_tmap(CUtensorMap* tm, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(lm::BK), box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = g_encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DLLM_OK : DLLM_ERR_CUDA;
}

struct LogitsArgs {
  const uint16_t* H; const uint8_t* M; const uint16_t* W;
  int B, L, d, V;
  const int* win_lo; const int* win_hi;          // rows restricted to windows, or both NULL
  uint32_t stats; float* entropy; float* margin;
  int* tok; float* conf; float* lse; float* dbg;
  int* row_idx; int* seq_off; int* count;
  void* ws; size_t ws_bytes; cudaStream_t s;
  lm::Partials raw = {nullptr, nullptr, nullptr, nullptr, nullptr};   // vocabulary-shard mode
  int a_offset = 0;
};

dllm_status validate_logits(const LogitsArgs& a, bool debug, bool prepared = false) {
  if ((!prepared && (!a.H || !a.M || !a.row_idx || !a.seq_off)) || !a.W || !a.count || !a.ws)
    return DLLM_ERR_NULL;
  const bool shard = a.raw.m != nullptr;
  if (shard) {
    if (!a.raw.s || !a.raw.a) return DLLM_ERR_NULL;
    if ((a.stats != 0) != (a.raw.t != nullptr) || (a.stats != 0) != (a.raw.m2 != nullptr))
      return DLLM_ERR_NULL;
    if (a.a_offset < 0 || static_cast<long long>(a.a_offset) + a.V >= (1ll << 31)) return DLLM_ERR_SHAPE;
  } else if (!debug && (!a.tok || !a.conf || !a.lse)) {
    return DLLM_ERR_NULL;
  }
  if (debug && !a.dbg) return DLLM_ERR_NULL;
  if ((a.win_lo == nullptr) != (a.win_hi == nullptr)) return DLLM_ERR_NULL;
  if ((a.stats & ~(DLLM_STAT_ENTROPY | DLLM_STAT_MARGIN)) != 0) return DLLM_ERR_SHAPE;
  if (!shard && ((a.stats & DLLM_STAT_ENTROPY) != 0) != (a.entropy != nullptr)) return DLLM_ERR_NULL;
  if (!shard && ((a.stats & DLLM_STAT_MARGIN) != 0) != (a.margin != nullptr)) return DLLM_ERR_NULL;
  if (!shapes_ok(a.B, a.L) || a.V < 1 || a.d < DLLM_D_MULTIPLE || a.d % DLLM_D_MULTIPLE != 0)
    return DLLM_ERR_SHAPE;
  const void* ptrs[] = {a.H, a.M, a.W, a.row_idx, a.seq_off, a.count, a.ws, a.tok, a.conf, a.lse,
                        a.dbg, a.entropy, a.margin, a.win_lo, a.win_hi, a.raw.m, a.raw.s,
                        a.raw.a, a.raw.t, a.raw.m2};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return DLLM_ERR_ALIGN;
  if (ws_layout_for(a.B, a.L, a.d, a.V, a.ws_bytes).rows < 1) return DLLM_ERR_WORKSPACE;
  return DLLM_OK;
}

// a1 + gather: compaction of the mask (in the windows, if any) and the copy of the masked
// rows of H into the workspace's dense Hm; H and M may be page-locked host memory.
dllm_status prepare_rows(const LogitsArgs& a, const DeviceState& ds, const WsLayout& w) {
  const void* Hd = nullptr;
  const void* Md = nullptr;
  bool host_rows = false;
  dllm_status st = resolve_input(a.H, &Hd, &host_rows);
  if (st != DLLM_OK) return st;
  if ((st = resolve_input(a.M, &Md)) != DLLM_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  int* tiles = reinterpret_cast<int*>(ws + w.tiles_off);
  uint16_t* Hm = reinterpret_cast<uint16_t*>(ws + w.hm_off);
  int* ctr = reinterpret_cast<int*>(ws + w.ctr_off);
  const long long n = static_cast<long long>(a.B) * a.L;
  if ((st = launch_compact(static_cast<const uint8_t*>(Md), a.B, a.L, a.win_lo, a.win_hi, a.row_idx,
                           a.seq_off, a.count, tiles, ds.status, a.s)) != DLLM_OK)
    return st;
  // Rows read from device memory: 4 CTAs per SM.  Rows read over the bus from page-locked
  // host memory: the bus, not the SMs, bounds the copy (about 20 ms for cfg3's 0.97 GB), and
  // one CTA per SM keeps enough reads in flight while leaving each SM room for the next
  // GEMM's persistent CTA, which this staging overlaps.
  if (launch_pdl(gather_rows_kernel, dim3(ds.sms * (host_rows ? DLLM_GATHER_HOST_CTAS : 4)),
                 dim3(kGatherThreads), 0, a.s,
                 static_cast<const uint16_t*>(Hd), (const int*)a.row_idx, (const int*)a.count, n,
                 w.rows, a.d, Hm, ctr, w.n_ctr, ds.status) != cudaSuccess)
    return DLLM_ERR_CUDA;
  count_launch();
  return DLLM_OK;
}

// skip_prepare: the rows were prepared by an earlier dllm_prepare_rows into the same
// workspace (H and M are then not read).
dllm_status run_logits(const LogitsArgs& a, bool debug, bool skip_prepare = false) {
  dllm_status st = validate_logits(a, debug, skip_prepare);
  if (st != DLLM_OK) return st;
  DeviceState* ds = nullptr;
  if ((st = device_state(&ds)) != DLLM_OK) return st;
  const WsLayout w = ws_layout_for(a.B, a.L, a.d, a.V, a.ws_bytes);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  uint16_t* Hm = reinterpret_cast<uint16_t*>(ws + w.hm_off);
  float* pm = reinterpret_cast<float*>(ws + w.pm_off);
  float* ps = reinterpret_cast<float*>(ws + w.ps_off);
  int* pa = reinterpret_cast<int*>(ws + w.pa_off);
  float* pt = reinterpret_cast<float*>(ws + w.pt_off);
  float* pm2 = reinterpret_cast<float*>(ws + w.pm2_off);
  int* ctr = reinterpret_cast<int*>(ws + w.ctr_off);
  const lm::Partials part{pm, ps, pa, pt, pm2};
  const lm::Outputs outs{a.tok, a.conf, a.lse, a.entropy, a.margin, a.raw, a.a_offset};
  const long long n = w.rows;        // masked-row capacity of this workspace (B*L when full)

  // GEMM variant: 0 = chosen on the device from the masked count (lm::auto_variant, one
  // launch in clusters of two CTAs), 1 / 2 = forced single CTAs / CTA pairs (test hook)
  int cg = g_gemm_variant.load();
  if (ds->pairs < 1) cg = 1;                                   // no CTA pairs on this device
  const int single_holders = cg == 0 ? 2 * ds->pairs : (ds->sms < lm::kMaxCtas ? ds->sms : lm::kMaxCtas);
  for (int v = 1; v <= 2; ++v) {
    if (cg != 0 && cg != v) continue;
    // largest partial footprint over every masked count this variant may run: all
    // positions masked, or any count that fits one group of m-tiles (remainder holders)
    const int holders = v == 2 ? ds->pairs : single_holders;
    const int bm = v == 2 ? lm::Cfg<2>::BM : lm::Cfg<1>::BM;
    const int gmax = v == 2 ? lm::Cfg<2>::kGroupM : lm::Cfg<1>::kGroupM;
    long long need = lm::Plan::make(static_cast<int>(n), a.V, holders, gmax, bm).part_entries();
    const long long mt = (n + bm - 1) / bm;
    for (long long m = 1; m <= mt && m <= gmax; ++m) {
      const long long c = m * bm < n ? m * bm : n;
      const long long e = lm::Plan::make(static_cast<int>(c), a.V, holders, gmax, bm).part_entries();
      if (e > need) need = e;
    }
    if (need > w.part_cap) return DLLM_ERR_WORKSPACE;                  // cannot happen on B200
  }

  if (!skip_prepare) {
    if ((st = prepare_rows(a, *ds, w)) != DLLM_OK) return st;
  }

  // W is staged 256 rows per CTA by single CTAs and 128 rows per CTA by pairs
  CUtensorMap tmA, tmB1, tmB2;
  if (make_tmap(&tmA, Hm, static_cast<uint64_t>(n), a.d, 128) != DLLM_OK) return DLLM_ERR_CUDA;
  if (cg != 2 && make_tmap(&tmB1, a.W, static_cast<uint64_t>(a.V), a.d, lm::BN) != DLLM_OK)
    return DLLM_ERR_CUDA;
  if (cg != 1 && make_tmap(&tmB2, a.W, static_cast<uint64_t>(a.V), a.d, lm::BN / 2) != DLLM_OK)
    return DLLM_ERR_CUDA;

  cudaEvent_t e1 = nullptr;
  if (!prof_gemm_start(a.s, &e1)) return DLLM_ERR_CUDA;
  {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.blockDim = dim3(lm::kThreads, 1, 1);
    cfg.stream = a.s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cg != 1) {
      attr[1].id = cudaLaunchAttributeClusterDimension;
      attr[1].val.clusterDim.x = 2;
      attr[1].val.clusterDim.y = 1;
      attr[1].val.clusterDim.z = 1;
      cfg.numAttrs = 2;
      cfg.gridDim = dim3(2 * ds->pairs, 1, 1);
      cfg.dynamicSmemBytes = cg == 0 ? lm::kAutoSmemBytes : lm::Cfg<2>::SMEM_BYTES;
    } else {
      cfg.gridDim = dim3(single_holders, 1, 1);
      cfg.dynamicSmemBytes = lm::Cfg<1>::SMEM_BYTES;
    }
    const int n_cap = static_cast<int>(n);
    float* dbg = debug ? a.dbg : nullptr;
    const int mode = debug ? lm::kModeDebugStore : (a.stats ? lm::kModeStatsExt : lm::kModeStats);
    const int* cnt = a.count;
    cudaError_t e;
#define DLLM_LAUNCH_GEMM(CGV, MODE, TMB)                                                      \
  cudaLaunchKernelEx(&cfg, lm::lmhead_kernel<CGV, MODE>, tmA, TMB, cnt, n_cap, a.V, a.d,      \
                     lm::Cfg<CGV>::kGroupM, part, w.part_cap, ctr, outs, dbg, ds->status)
#define DLLM_LAUNCH_AUTO(MODE)                                                                 \
  cudaLaunchKernelEx(&cfg, lm::lmhead_auto_kernel<MODE>, tmA, tmB1, tmB2, cnt, n_cap, a.V, a.d, \
                     part, w.part_cap, ctr, outs, dbg, ds->status)
    if (cg == 0)
      e = mode == lm::kModeStats ? DLLM_LAUNCH_AUTO(lm::kModeStats)
        : mode == lm::kModeStatsExt ? DLLM_LAUNCH_AUTO(lm::kModeStatsExt)
        : DLLM_LAUNCH_AUTO(lm::kModeDebugStore);
    else if (cg == 2)
      e = mode == lm::kModeStats ? DLLM_LAUNCH_GEMM(2, lm::kModeStats, tmB2)
        : mode == lm::kModeStatsExt ? DLLM_LAUNCH_GEMM(2, lm::kModeStatsExt, tmB2)
        : DLLM_LAUNCH_GEMM(2, lm::kModeDebugStore, tmB2);
    else
      e = mode == lm::kModeStats ? DLLM_LAUNCH_GEMM(1, lm::kModeStats, tmB1)
        : mode == lm::kModeStatsExt ? DLLM_LAUNCH_GEMM(1, lm::kModeStatsExt, tmB1)
        : DLLM_LAUNCH_GEMM(1, lm::kModeDebugStore, tmB1);
#undef DLLM_LAUNCH_GEMM
#undef DLLM_LAUNCH_AUTO
    if (e != cudaSuccess) return DLLM_ERR_CUDA;
  }
  count_launch();
  prof_gemm_stop(a.s, e1);
  return cudaPeekAtLastError() == cudaSuccess ? DLLM_OK : DLLM_ERR_CUDA;
}

// ---------------------------------------------------------------------------------------
// Rules on the logits, and MXFP4 operands (dllm_masked_logits_rules, dllm_masked_logits_mx4)
// ---------------------------------------------------------------------------------------
constexpr int kMaxColumns = 1 << 30;             // vocabulary tiles and columns stay in 32 bits
bool logits_shape_ok(int B, int L, int d, int V) {
  return shapes_ok(B, L) && V >= 1 && V <= kMaxColumns && d >= DLLM_D_MULTIPLE && d % DLLM_D_MULTIPLE == 0;
}

dllm_status validate_rules(const dllm_logit_rules& r, int B, int V) {
  const long long words = (static_cast<long long>(V) + 31) / 32;
  if ((r.counts == nullptr) != (r.seen == nullptr)) return DLLM_ERR_NULL;
  if (!r.counts && (r.repetition || r.presence || r.frequency)) return DLLM_ERR_NULL;
  if (r.allow_id && !r.allow) return DLLM_ERR_NULL;
  const void* ptrs[] = {r.bias, r.counts, r.seen, r.repetition, r.presence, r.frequency, r.allow, r.allow_id};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return DLLM_ERR_ALIGN;
  if (r.bias && r.bias_stride != 0 && (r.bias_stride < V || r.bias_stride % 4 != 0)) return DLLM_ERR_SHAPE;
  if (r.counts && (r.counts_stride < V || r.seen_stride < words)) return DLLM_ERR_SHAPE;
  if (r.allow && (r.allow_stride < words || r.allow_rows < 1)) return DLLM_ERR_SHAPE;
  if (r.allow && !r.allow_id && r.allow_rows != 1 && r.allow_rows != B) return DLLM_ERR_SHAPE;
  return DLLM_OK;
}

struct ShapedArgs {
  LogitsArgs a;                                  // a.W is null with MXFP4 operands
  const uint8_t* Wq; const uint8_t* Ws;          // MXFP4 codes and scales of W, or both null
  const dllm_logit_rules* rules;                 // null: no rules (MXFP4 only)
};

// A 2-D map of rows of `cols` elements (row pitch cols * bytes), boxes of box_cols x box_rows.
dllm_status make_map(CUtensorMap* tm, CUtensorMapDataType type, int bytes, const void* base, uint64_t rows,
                     uint64_t cols, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols * bytes};
  const cuuint32_t box[2] = {box_cols, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = g_encode(tm, type, 2, const_cast<void*>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DLLM_OK : DLLM_ERR_CUDA;
}

// The GEMM on prepared rows: one launch in clusters of two CTAs.
template <class Op>
dllm_status launch_shaped(const ShapedArgs& x, const DeviceState& ds, const WsLayout& w,
                          const lm::Outputs& outs) {
  const LogitsArgs& a = x.a;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  const void* Hm = ws + w.hm_off;
  const uint64_t n = static_cast<uint64_t>(w.rows), V = static_cast<uint64_t>(a.V);
  CUtensorMap tmA1, tmA2, tmB1, tmB2, tmSA, tmSB;
  const auto sw128 = CU_TENSOR_MAP_SWIZZLE_128B;
  dllm_status st = DLLM_OK;
  auto map = [&](CUtensorMap* tm, const void* base, uint64_t rows, uint32_t box_rows) {
    if (st != DLLM_OK) return;
    st = Op::kMx4 ? make_map(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, rows, a.d / 2, 128, box_rows, sw128)
                  : make_map(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, rows, a.d, 64, box_rows, sw128);
  };
  const void* W = Op::kMx4 ? static_cast<const void*>(x.Wq) : static_cast<const void*>(a.W);
  map(&tmA1, Hm, n, 32);
  map(&tmA2, Hm, n, 128);
  map(&tmB1, W, V, Op::BN);
  map(&tmB2, W, V, Op::BN / 2);
  if (Op::kMx4 && st == DLLM_OK) {
    // scale tiles as rows of ceil(d / 128) * 512 bytes, in 8-byte words: 1024 bytes a stage
    const uint64_t words = static_cast<uint64_t>((a.d + 127) / 128) * 64;
    st = make_map(&tmSA, CU_TENSOR_MAP_DATA_TYPE_UINT64, 8, ws + w.hs_off, (n + 127) / 128, words, 128, 1,
                  CU_TENSOR_MAP_SWIZZLE_NONE);
    if (st == DLLM_OK)
      st = make_map(&tmSB, CU_TENSOR_MAP_DATA_TYPE_UINT64, 8, x.Ws, (V + 127) / 128, words, 128, 2,
                    CU_TENSOR_MAP_SWIZZLE_NONE);
  } else {
    tmSA = tmSB = tmA1;                                                // not used
  }
  if (st != DLLM_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(2 * ds.pairs, 1, 1);
  cfg.blockDim = dim3(shaped::kThreads, 1, 1);
  cfg.dynamicSmemBytes = shaped::kSmemBytes;
  cfg.stream = a.s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // partials: 16 bytes each in the first four of the workspace's partial arrays (which are one
  // piece), the argmax in the fifth
  const int tiles = (a.V + Op::BN - 1) / Op::BN;
  const shaped::Problem p{static_cast<int>(w.rows), a.V, a.d, a.L, shaped::tile_step(tiles), a.row_idx,
                          reinterpret_cast<float4*>(ws + w.pm_off), reinterpret_cast<int*>(ws + w.pm2_off),
                          w.part_cap,
                          reinterpret_cast<int*>(ws + w.ctr_off), outs, ds.status};
  const dllm_logit_rules rules = x.rules ? *x.rules : dllm_logit_rules{};
  const int* count = a.count;
  const int variant = g_gemm_variant.load();
  cudaEvent_t stop = nullptr;
  if (!prof_gemm_start(a.s, &stop)) return DLLM_ERR_CUDA;
#define DLLM_LAUNCH_SHAPED(RULES, EXT)                                                            \
  cudaLaunchKernelEx(&cfg, shaped::shaped_kernel<Op, RULES, EXT>, tmA1, tmA2, tmB1, tmB2, tmSA,    \
                     tmSB, count, variant, p, rules)
  cudaError_t e;
  if constexpr (Op::kMx4) {
    if (!x.rules)
      e = a.stats ? DLLM_LAUNCH_SHAPED(false, true) : DLLM_LAUNCH_SHAPED(false, false);
    else
      e = a.stats ? DLLM_LAUNCH_SHAPED(true, true) : DLLM_LAUNCH_SHAPED(true, false);
  } else {
    e = a.stats ? DLLM_LAUNCH_SHAPED(true, true) : DLLM_LAUNCH_SHAPED(true, false);
  }
#undef DLLM_LAUNCH_SHAPED
  if (e != cudaSuccess) return DLLM_ERR_CUDA;
  count_launch();
  prof_gemm_stop(a.s, stop);
  return cudaPeekAtLastError() == cudaSuccess ? DLLM_OK : DLLM_ERR_CUDA;
}

// Compaction, and the masked rows of H into the workspace: in MXFP4, or as they are.
dllm_status stage_shaped(const LogitsArgs& a, const DeviceState& ds, const WsLayout& w, bool mx4) {
  const void* Hd = nullptr;
  const void* Md = nullptr;
  bool h_host = false, m_host = false;
  dllm_status st = resolve_input(a.H, &Hd, &h_host);
  if (st != DLLM_OK) return st;
  if ((st = resolve_input(a.M, &Md, &m_host)) != DLLM_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  const uint8_t* M = static_cast<const uint8_t*>(Md);
  const uint16_t* H = static_cast<const uint16_t*>(Hd);
  uint8_t* rows = ws + w.hm_off;
  uint32_t* scales = reinterpret_cast<uint32_t*>(ws + w.hs_off);
  int* ctr = reinterpret_cast<int*>(ws + w.ctr_off);
  const long long n = static_cast<long long>(a.B) * a.L;
  cudaError_t e;
  if (n <= stage::kMaxPositions && !m_host) {          // a mask in host memory is read once, not by every CTA
    const dim3 grid(stage::kCtas), thr(stage::kThreads);
    e = mx4 ? launch_pdl(stage::stage_rows_kernel<true>, grid, thr, 0, a.s, M, a.B, a.L, a.win_lo, a.win_hi, H,
                         a.d, w.rows, a.row_idx, a.seq_off, a.count, rows, scales, ctr, w.n_ctr, ds.status)
            : launch_pdl(stage::stage_rows_kernel<false>, grid, thr, 0, a.s, M, a.B, a.L, a.win_lo, a.win_hi, H,
                         a.d, w.rows, a.row_idx, a.seq_off, a.count, rows, scales, ctr, w.n_ctr, ds.status);
  } else {
    if (!mx4) return prepare_rows(a, ds, w);
    if ((st = launch_compact(M, a.B, a.L, a.win_lo, a.win_hi, a.row_idx, a.seq_off, a.count,
                             reinterpret_cast<int*>(ws + w.tiles_off), ds.status, a.s)) != DLLM_OK)
      return st;
    e = launch_pdl(mx4::gather_quantize_kernel, dim3(ds.sms * (h_host ? DLLM_GATHER_HOST_CTAS : 4)),
                   dim3(mx4::kThreads), 0, a.s, H, (const int*)a.row_idx, (const int*)a.count, n, w.rows, a.d,
                   rows, scales, ctr, w.n_ctr, ds.status);
  }
  if (e != cudaSuccess) return DLLM_ERR_CUDA;
  count_launch();
  return DLLM_OK;
}

dllm_status run_shaped(const ShapedArgs& x) {
  const LogitsArgs& a = x.a;
  const bool mx4 = x.Wq != nullptr;
  if (!a.H || !a.M || !a.row_idx || !a.seq_off || !a.count || !a.ws || !a.tok || !a.conf || !a.lse)
    return DLLM_ERR_NULL;
  if ((a.win_lo == nullptr) != (a.win_hi == nullptr)) return DLLM_ERR_NULL;
  if ((a.stats & ~(DLLM_STAT_ENTROPY | DLLM_STAT_MARGIN)) != 0) return DLLM_ERR_SHAPE;
  if (((a.stats & DLLM_STAT_ENTROPY) != 0) != (a.entropy != nullptr)) return DLLM_ERR_NULL;
  if (((a.stats & DLLM_STAT_MARGIN) != 0) != (a.margin != nullptr)) return DLLM_ERR_NULL;
  if (!logits_shape_ok(a.B, a.L, a.d, a.V)) return DLLM_ERR_SHAPE;
  const void* ptrs[] = {a.H, a.M, a.W, x.Wq, x.Ws, a.row_idx, a.seq_off, a.count, a.ws, a.tok, a.conf,
                        a.lse, a.entropy, a.margin, a.win_lo, a.win_hi};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return DLLM_ERR_ALIGN;
  dllm_status st = DLLM_OK;
  if (x.rules && (st = validate_rules(*x.rules, a.B, a.V)) != DLLM_OK) return st;
  const WsLayout w = ws_layout_for(a.B, a.L, a.d, a.V, a.ws_bytes, mx4);
  if (w.rows < 1) return DLLM_ERR_WORKSPACE;
  DeviceState* ds = nullptr;
  if ((st = device_state(&ds)) != DLLM_OK) return st;
  if (ds->pairs < 1 || (!mx4 && !ds->shaped_bf16)) return DLLM_ERR_DEVICE;
  if ((st = stage_shaped(a, *ds, w, mx4)) != DLLM_OK) return st;
  const lm::Outputs outs{a.tok, a.conf, a.lse, a.entropy, a.margin, a.raw, 0};
  return mx4 ? launch_shaped<shaped::Mx4>(x, *ds, w, outs) : launch_shaped<shaped::Bf16>(x, *ds, w, outs);
}

dllm_status mx4_checks(const void* X, int dtype, bool f16_ok, int64_t rows, int32_t cols, int64_t ld,
                       const void* q, const void* s) {
  if (!X || !q || !s) return DLLM_ERR_NULL;
  if (rows < 1 || rows >= (1ll << 31) || cols < 32 || cols % 32 != 0 || cols > kMaxColumns || ld < cols)
    return DLLM_ERR_SHAPE;
  if (dtype != DLLM_BF16 && dtype != DLLM_F32 && !(f16_ok && dtype == DLLM_F16)) return DLLM_ERR_SHAPE;
  if (!aligned16(X) || !aligned16(q) || !aligned16(s) || ld % (dtype == DLLM_F32 ? 4 : 8) != 0)
    return DLLM_ERR_ALIGN;
  return DLLM_OK;
}

// Blocks of a grid-stride kernel: one per `per` items, at most `most`.
unsigned grid_for(long long items, int per, long long most) {
  const long long g = (items + per - 1) / per;
  return static_cast<unsigned>(g < 1 ? 1 : (g > most ? most : g));
}

}  // namespace
}  // namespace dllm

// ---------------------------------------------------------------------------------------
// Allocation-free compaction (dllm_mask_compact_noalloc): the per-tile counts live in this
// fixed static device array instead of the caller's workspace.  In host code the array's
// name is only a host-side stand-in; its device address comes from cudaGetSymbolAddress,
// looked up once per device.
// ---------------------------------------------------------------------------------------
static __device__ __align__(256) int g_noalloc_tile_counts[DLLM_NOALLOC_MAX_TILES];

static_assert(static_cast<long long>(DLLM_NOALLOC_MAX_TILES) * dllm::kCompactTile ==
                  DLLM_NOALLOC_MAX_POSITIONS,
              "scratch limit and compaction tile size disagree");

namespace {
struct NoAllocScratch {
  bool ready = false;
  dllm_status err = DLLM_OK;
  int* tiles = nullptr;           // device address of g_noalloc_tile_counts on this device
};
std::mutex g_noalloc_mu;
NoAllocScratch g_noalloc[64];

dllm_status noalloc_scratch(int** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DLLM_ERR_CUDA;
  if (dev < 0 || dev >= 64) return DLLM_ERR_DEVICE;
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  NoAllocScratch& st = g_noalloc[dev];
  if (!st.ready) {
    void* p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_noalloc_tile_counts);
    st.err = (e == cudaSuccess && p != nullptr) ? DLLM_OK : DLLM_ERR_CUDA;
    st.tiles = static_cast<int*>(p);
    st.ready = true;
  }
  if (st.err != DLLM_OK) return st.err;
  *out = st.tiles;
  return DLLM_OK;
}
}  // namespace

using namespace dllm;

extern "C" {

dllm_status dllm_mask_compact_noalloc(const uint8_t* M, int32_t B, int32_t L, int32_t* row_idx,
                                      int32_t* seq_off, int32_t* count, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_mask_compact_noalloc");
  if (!M || !row_idx || !seq_off || !count) return DLLM_ERR_NULL;
  if (!shapes_ok(B, L)) return DLLM_ERR_SHAPE;
  if (static_cast<long long>(B) * L > DLLM_NOALLOC_MAX_POSITIONS) return DLLM_ERR_SCRATCH;
  if (!aligned16(M) || !aligned16(row_idx) || !aligned16(seq_off) || !aligned16(count))
    return DLLM_ERR_ALIGN;
  DeviceState* ds = nullptr;
  dllm_status st = device_state(&ds);
  if (st != DLLM_OK) return st;
  int* tiles = nullptr;
  if ((st = noalloc_scratch(&tiles)) != DLLM_OK) return st;
  return launch_compact(M, B, L, nullptr, nullptr, row_idx, seq_off, count, tiles, ds->status,
                        static_cast<cudaStream_t>(stream));
}

int32_t dllm_version(void) { return 10200; }

const char* dllm_status_string(dllm_status s) {
  switch (s) {
    case DLLM_OK: return "ok";
    case DLLM_ERR_NULL: return "a required pointer is NULL";
    case DLLM_ERR_ALIGN: return "a device pointer is not 16-byte aligned";
    case DLLM_ERR_SHAPE: return "shape out of range";
    case DLLM_ERR_WORKSPACE: return "workspace too small";
    case DLLM_ERR_CUDA: return "CUDA error";
    case DLLM_ERR_TIMEOUT: return "a device-side wait timed out";
    case DLLM_ERR_DEVICE: return "device is not an sm_100 GPU, or the library was not built for it";
    case DLLM_ERR_BOUNDS: return "a device-side bound check failed";
    case DLLM_ERR_SCRATCH: return "B*L exceeds the fixed scratch of the allocation-free entry point";
    case DLLM_ERR_MEMORY: return "an input is neither device memory nor page-locked host memory";
    case DLLM_ERR_CAPACITY: return "more masked rows than the workspace was sized for";
    default: return "unknown status";
  }
}

size_t dllm_workspace_bytes(int32_t B, int32_t L, int32_t d, int32_t V) {
  if (!shapes_ok(B, L) || V < 1 || d < DLLM_D_MULTIPLE || d % DLLM_D_MULTIPLE != 0) return 0;
  return ws_layout(B, L, d, V, static_cast<long long>(B) * L).total;
}

size_t dllm_workspace_bytes_rows(int32_t B, int32_t L, int32_t d, int32_t V, int64_t max_rows) {
  if (!shapes_ok(B, L) || V < 1 || d < DLLM_D_MULTIPLE || d % DLLM_D_MULTIPLE != 0 || max_rows < 1)
    return 0;
  return ws_layout(B, L, d, V, max_rows).total;
}

int64_t dllm_workspace_rows(int32_t B, int32_t L, int32_t d, int32_t V, size_t ws_bytes) {
  if (!shapes_ok(B, L) || V < 1 || d < DLLM_D_MULTIPLE || d % DLLM_D_MULTIPLE != 0) return 0;
  return ws_layout_for(B, L, d, V, ws_bytes).rows;
}

dllm_status dllm_mask_compact_window(const uint8_t* M, int32_t B, int32_t L, const int32_t* win_lo,
                                     const int32_t* win_hi, int32_t* row_idx, int32_t* seq_off,
                                     int32_t* count, void* ws, size_t ws_bytes, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_mask_compact_window");
  if (!M || !row_idx || !seq_off || !count || !ws) return DLLM_ERR_NULL;
  if ((win_lo == nullptr) != (win_hi == nullptr)) return DLLM_ERR_NULL;
  if (!shapes_ok(B, L)) return DLLM_ERR_SHAPE;
  if (!aligned16(M) || !aligned16(row_idx) || !aligned16(seq_off) || !aligned16(count) || !aligned16(ws))
    return DLLM_ERR_ALIGN;
  if ((win_lo && !aligned16(win_lo)) || (win_hi && !aligned16(win_hi))) return DLLM_ERR_ALIGN;
  const long long n = static_cast<long long>(B) * L;
  const size_t need = sizeof(int) * static_cast<size_t>((n + kCompactTile - 1) / kCompactTile);
  if (ws_bytes < need) return DLLM_ERR_WORKSPACE;
  DeviceState* ds = nullptr;
  dllm_status st = device_state(&ds);
  if (st != DLLM_OK) return st;
  return launch_compact(M, B, L, win_lo, win_hi, row_idx, seq_off, count, static_cast<int*>(ws),
                        ds->status, static_cast<cudaStream_t>(stream));
}

dllm_status dllm_mask_compact(const uint8_t* M, int32_t B, int32_t L, int32_t* row_idx,
                              int32_t* seq_off, int32_t* count, void* ws, size_t ws_bytes,
                              void* stream) {
  return dllm_mask_compact_window(M, B, L, nullptr, nullptr, row_idx, seq_off, count, ws, ws_bytes,
                                  stream);
}

dllm_status dllm_masked_logits(const uint16_t* H, const uint8_t* M, const uint16_t* W, int32_t B,
                               int32_t L, int32_t d, int32_t V, int32_t* tok, float* conf,
                               float* lse, int32_t* row_idx, int32_t* seq_off, int32_t* count,
                               void* ws, size_t ws_bytes, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_masked_logits");
  LogitsArgs a{H, M, W, B, L, d, V, nullptr, nullptr, 0u, nullptr, nullptr, tok, conf, lse, nullptr,
               row_idx, seq_off, count, ws, ws_bytes, static_cast<cudaStream_t>(stream)};
  return run_logits(a, false);
}

dllm_status dllm_masked_logits_ex(const uint16_t* H, const uint8_t* M, const uint16_t* W, int32_t B,
                                  int32_t L, int32_t d, int32_t V, uint32_t stats, int32_t* tok,
                                  float* conf, float* lse, float* entropy, float* margin,
                                  int32_t* row_idx, int32_t* seq_off, int32_t* count, void* ws,
                                  size_t ws_bytes, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_masked_logits_ex");
  LogitsArgs a{H, M, W, B, L, d, V, nullptr, nullptr, stats, entropy, margin, tok, conf, lse, nullptr,
               row_idx, seq_off, count, ws, ws_bytes, static_cast<cudaStream_t>(stream)};
  return run_logits(a, false);
}

dllm_status dllm_masked_logits_window(const uint16_t* H, const uint8_t* M, const uint16_t* W,
                                      int32_t B, int32_t L, int32_t d, int32_t V,
                                      const int32_t* win_lo, const int32_t* win_hi, uint32_t stats,
                                      int32_t* tok, float* conf, float* lse, float* entropy,
                                      float* margin, int32_t* row_idx, int32_t* seq_off,
                                      int32_t* count, void* ws, size_t ws_bytes, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_masked_logits_window");
  if (!win_lo || !win_hi) return DLLM_ERR_NULL;
  LogitsArgs a{H, M, W, B, L, d, V, win_lo, win_hi, stats, entropy, margin, tok, conf, lse, nullptr,
               row_idx, seq_off, count, ws, ws_bytes, static_cast<cudaStream_t>(stream)};
  return run_logits(a, false);
}

dllm_status dllm_masked_partials(const uint16_t* H, const uint8_t* M, const uint16_t* W_shard,
                                 int32_t B, int32_t L, int32_t d, int32_t V_shard, int32_t v_offset,
                                 const int32_t* win_lo, const int32_t* win_hi, uint32_t stats,
                                 float* part_m, float* part_s, int32_t* part_a, float* part_t,
                                 float* part_m2, int32_t* row_idx, int32_t* seq_off, int32_t* count,
                                 void* ws, size_t ws_bytes, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_masked_partials");
  if (!part_m) return DLLM_ERR_NULL;
  LogitsArgs a{H, M, W_shard, B, L, d, V_shard, win_lo, win_hi, stats, nullptr, nullptr, nullptr,
               nullptr, nullptr, nullptr, row_idx, seq_off, count, ws, ws_bytes,
               static_cast<cudaStream_t>(stream)};
  a.raw = lm::Partials{part_m, part_s, part_a, part_t, part_m2};
  a.a_offset = v_offset;
  return run_logits(a, false);
}

dllm_status dllm_lse_merge(const float* part_m, const float* part_s, const int32_t* part_a,
                           const float* part_t, const float* part_m2, int64_t split_stride,
                           int32_t n_split, const int32_t* count, int32_t n_cap, uint32_t stats,
                           int32_t* tok, float* conf, float* lse, float* entropy, float* margin,
                           void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_lse_merge");
  if (!part_m || !part_s || !part_a || !count || !tok || !conf || !lse) return DLLM_ERR_NULL;
  if ((stats & ~(DLLM_STAT_ENTROPY | DLLM_STAT_MARGIN)) != 0) return DLLM_ERR_SHAPE;
  if ((stats != 0) != (part_t != nullptr) || (stats != 0) != (part_m2 != nullptr)) return DLLM_ERR_NULL;
  if (((stats & DLLM_STAT_ENTROPY) != 0) != (entropy != nullptr)) return DLLM_ERR_NULL;
  if (((stats & DLLM_STAT_MARGIN) != 0) != (margin != nullptr)) return DLLM_ERR_NULL;
  if (n_split < 1 || n_cap < 1 || split_stride < n_cap) return DLLM_ERR_SHAPE;
  const void* ptrs[] = {part_m, part_s, part_a, part_t, part_m2, count, tok, conf, lse, entropy, margin};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return DLLM_ERR_ALIGN;
  DeviceState* ds = nullptr;
  dllm_status st = device_state(&ds);
  if (st != DLLM_OK) return st;
  int blocks = (n_cap + kMergeThreads - 1) / kMergeThreads;
  if (blocks > ds->sms * 8) blocks = ds->sms * 8;
  const lm::Partials part{const_cast<float*>(part_m), const_cast<float*>(part_s),
                          const_cast<int*>(part_a), const_cast<float*>(part_t),
                          const_cast<float*>(part_m2)};
  const lm::Outputs outs{tok, conf, lse, entropy, margin, lm::Partials{nullptr, nullptr, nullptr, nullptr, nullptr}, 0};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = stats != 0
      ? launch_pdl(lse_merge_kernel<true>, dim3(blocks), dim3(kMergeThreads), 0, s, part,
                   static_cast<long long>(split_stride), static_cast<int>(n_split), count,
                   static_cast<int>(n_cap), outs)
      : launch_pdl(lse_merge_kernel<false>, dim3(blocks), dim3(kMergeThreads), 0, s, part,
                   static_cast<long long>(split_stride), static_cast<int>(n_split), count,
                   static_cast<int>(n_cap), outs);
  if (e != cudaSuccess) return DLLM_ERR_CUDA;
  count_launch();
  return DLLM_OK;
}

dllm_status dllm_prepare_rows(const uint16_t* H, const uint8_t* M, int32_t B, int32_t L, int32_t d,
                              int32_t V, const int32_t* win_lo, const int32_t* win_hi,
                              int32_t* row_idx, int32_t* seq_off, int32_t* count, void* ws,
                              size_t ws_bytes, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_prepare_rows");
  if (!H || !M || !row_idx || !seq_off || !count || !ws) return DLLM_ERR_NULL;
  if ((win_lo == nullptr) != (win_hi == nullptr)) return DLLM_ERR_NULL;
  if (!shapes_ok(B, L) || V < 1 || d < DLLM_D_MULTIPLE || d % DLLM_D_MULTIPLE != 0) return DLLM_ERR_SHAPE;
  const void* ptrs[] = {H, M, row_idx, seq_off, count, ws, win_lo, win_hi};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return DLLM_ERR_ALIGN;
  const WsLayout w = ws_layout_for(B, L, d, V, ws_bytes);
  if (w.rows < 1) return DLLM_ERR_WORKSPACE;
  DeviceState* ds = nullptr;
  dllm_status st = device_state(&ds);
  if (st != DLLM_OK) return st;
  LogitsArgs a{H, M, nullptr, B, L, d, V, win_lo, win_hi, 0u, nullptr, nullptr, nullptr, nullptr, nullptr,
               nullptr, row_idx, seq_off, count, ws, ws_bytes, static_cast<cudaStream_t>(stream)};
  return prepare_rows(a, *ds, w);
}

dllm_status dllm_masked_logits_prepared(const uint16_t* W, int32_t B, int32_t L, int32_t d, int32_t V,
                                        uint32_t stats, int32_t* tok, float* conf, float* lse,
                                        float* entropy, float* margin, const int32_t* count,
                                        void* ws, size_t ws_bytes, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_masked_logits_prepared");
  LogitsArgs a{nullptr, nullptr, W, B, L, d, V, nullptr, nullptr, stats, entropy, margin, tok, conf,
               lse, nullptr, nullptr, nullptr, const_cast<int32_t*>(count), ws, ws_bytes,
               static_cast<cudaStream_t>(stream)};
  return run_logits(a, false, true);
}

dllm_status dllm_debug_lmhead_logits(const uint16_t* H, const uint8_t* M, const uint16_t* W,
                                     int32_t B, int32_t L, int32_t d, int32_t V, float* logits_out,
                                     int32_t* row_idx, int32_t* seq_off, int32_t* count, void* ws,
                                     size_t ws_bytes, void* stream) {
  LogitsArgs a{H, M, W, B, L, d, V, nullptr, nullptr, 0u, nullptr, nullptr, nullptr, nullptr, nullptr,
               logits_out, row_idx, seq_off, count, ws, ws_bytes, static_cast<cudaStream_t>(stream)};
  return run_logits(a, true);
}

}  // extern "C"

namespace {
dllm_status run_select(const float* conf, const int32_t* row_idx, const int32_t* seq_off,
                       int32_t B, int32_t L, int32_t k, bool use_threshold, float threshold,
                       int32_t min_sel, bool ascending, const int32_t* win_lo, const int32_t* win_hi,
                       const int32_t* tok, int32_t* idx, int32_t* n_sel, int32_t* tok_sel,
                       float* conf_sel, void* stream) {
  if (!conf || !row_idx || !seq_off || !idx || !n_sel) return DLLM_ERR_NULL;
  if (use_threshold && (min_sel < 0 || threshold != threshold)) return DLLM_ERR_SHAPE;
  if ((win_lo == nullptr) != (win_hi == nullptr)) return DLLM_ERR_NULL;
  if (tok_sel && !tok) return DLLM_ERR_NULL;
  if (!shapes_ok(B, L) || k < 1 || k > DLLM_MAX_K) return DLLM_ERR_SHAPE;
  const void* ptrs[] = {conf, row_idx, seq_off, win_lo, win_hi, tok, idx, n_sel, tok_sel, conf_sel};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return DLLM_ERR_ALIGN;
  DeviceState* ds = nullptr;
  dllm_status st = device_state(&ds);
  if (st != DLLM_OK) return st;
  if (launch_pdl(select_unmask_kernel, dim3(B), dim3(kSelThreads), 0, static_cast<cudaStream_t>(stream),
                 conf, row_idx, seq_off, B * L, L, k, use_threshold, threshold, min_sel, ascending,
                 win_lo, win_hi, tok, idx, n_sel, tok_sel, conf_sel) != cudaSuccess)
    return DLLM_ERR_CUDA;
  count_launch();
  return DLLM_OK;
}
}  // namespace

extern "C" {

dllm_status dllm_select_unmask(const float* conf, const int32_t* row_idx, const int32_t* seq_off,
                               int32_t B, int32_t L, int32_t k, const int32_t* win_lo,
                               const int32_t* win_hi, const int32_t* tok, int32_t* idx,
                               int32_t* n_sel, int32_t* tok_sel, float* conf_sel, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_select_unmask");
  return run_select(conf, row_idx, seq_off, B, L, k, false, 0.f, 0, false, win_lo, win_hi, tok, idx,
                    n_sel, tok_sel, conf_sel, stream);
}

dllm_status dllm_select_unmask_ex(const float* score, const int32_t* row_idx, const int32_t* seq_off,
                                  int32_t B, int32_t L, int32_t k, float threshold, int32_t min_sel,
                                  int32_t ascending, const int32_t* win_lo, const int32_t* win_hi,
                                  const int32_t* tok, int32_t* idx, int32_t* n_sel, int32_t* tok_sel,
                                  float* score_sel, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_select_unmask_ex");
  if (ascending != 0 && ascending != 1) return DLLM_ERR_SHAPE;
  return run_select(score, row_idx, seq_off, B, L, k, true, threshold, min_sel, ascending != 0,
                    win_lo, win_hi, tok, idx, n_sel, tok_sel, score_sel, stream);
}

dllm_status dllm_decode_step(const uint16_t* H, const uint8_t* M, const uint16_t* W, int32_t B,
                             int32_t L, int32_t d, int32_t V, int32_t k, const int32_t* win_lo,
                             const int32_t* win_hi, int32_t* tok, float* conf, float* lse,
                             int32_t* row_idx, int32_t* seq_off, int32_t* count, int32_t* idx,
                             int32_t* n_sel, int32_t* tok_sel, float* conf_sel, void* ws,
                             size_t ws_bytes, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_decode_step");
  // validate the selection's own arguments first so that nothing is launched on error
  if (!idx || !n_sel) return DLLM_ERR_NULL;
  if ((win_lo == nullptr) != (win_hi == nullptr)) return DLLM_ERR_NULL;
  if (k < 1 || k > DLLM_MAX_K) return DLLM_ERR_SHAPE;
  const void* ptrs[] = {win_lo, win_hi, idx, n_sel, tok_sel, conf_sel};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return DLLM_ERR_ALIGN;
  dllm_status st = dllm_masked_logits(H, M, W, B, L, d, V, tok, conf, lse, row_idx, seq_off, count,
                                      ws, ws_bytes, stream);
  if (st != DLLM_OK) return st;
  return dllm_select_unmask(conf, row_idx, seq_off, B, L, k, win_lo, win_hi, tok, idx, n_sel,
                            tok_sel, conf_sel, stream);
}

dllm_status dllm_decode_block_step(const uint16_t* H, const uint8_t* M, const uint16_t* W, int32_t B,
                                   int32_t L, int32_t d, int32_t V, int32_t k, const int32_t* win_lo,
                                   const int32_t* win_hi, int32_t* tok, float* conf, float* lse,
                                   int32_t* row_idx, int32_t* seq_off, int32_t* count, int32_t* idx,
                                   int32_t* n_sel, int32_t* tok_sel, float* conf_sel, void* ws,
                                   size_t ws_bytes, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_decode_block_step");
  if (!idx || !n_sel || !win_lo || !win_hi) return DLLM_ERR_NULL;
  if (k < 1 || k > DLLM_MAX_K) return DLLM_ERR_SHAPE;
  const void* ptrs[] = {idx, n_sel, tok_sel, conf_sel};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return DLLM_ERR_ALIGN;
  dllm_status st = dllm_masked_logits_window(H, M, W, B, L, d, V, win_lo, win_hi, 0u, tok, conf, lse,
                                             nullptr, nullptr, row_idx, seq_off, count, ws, ws_bytes,
                                             stream);
  if (st != DLLM_OK) return st;
  // every compacted row already lies in its window: no window test is needed in the selection
  return dllm_select_unmask(conf, row_idx, seq_off, B, L, k, nullptr, nullptr, tok, idx, n_sel,
                            tok_sel, conf_sel, stream);
}

dllm_status dllm_debug_lse_merge(const float* part_m, const float* part_s, const int32_t* part_a,
                                 int32_t n_rows, int32_t n_split, int32_t* tok, float* conf,
                                 float* lse, void* stream) {
  if (!part_m || !part_s || !part_a || !tok || !conf || !lse) return DLLM_ERR_NULL;
  if (n_rows < 1 || n_split < 1) return DLLM_ERR_SHAPE;
  const void* ptrs[] = {part_m, part_s, part_a, tok, conf, lse};
  for (const void* p : ptrs)
    if (!aligned16(p)) return DLLM_ERR_ALIGN;
  DeviceState* ds = nullptr;
  dllm_status st = device_state(&ds);
  if (st != DLLM_OK) return st;
  int blocks = (n_rows + kMergeThreads - 1) / kMergeThreads;
  if (blocks > ds->sms * 8) blocks = ds->sms * 8;
  lse_merge_plain_kernel<<<blocks, kMergeThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      part_m, part_s, part_a, n_rows, n_split, tok, conf, lse);
  count_launch();
  return cudaPeekAtLastError() == cudaSuccess ? DLLM_OK : DLLM_ERR_CUDA;
}

dllm_status dllm_debug_set_gemm_variant(int32_t cta_group) {
  if (cta_group != 0 && cta_group != 1 && cta_group != 2) return DLLM_ERR_SHAPE;
  g_gemm_variant.store(cta_group);
  return DLLM_OK;
}

dllm_status dllm_get_status(void* stream) {
  DeviceState* ds = nullptr;
  dllm_status st = device_state(&ds);
  if (st != DLLM_OK) return st;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return DLLM_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return DLLM_ERR_CUDA;
  const int zero = 0;
  if (v != 0 && cudaMemcpyToSymbol(g_status, &zero, sizeof(int)) != cudaSuccess) return DLLM_ERR_CUDA;
  if (v & kStatusTimeout) return DLLM_ERR_TIMEOUT;
  if (v & kStatusBounds) return DLLM_ERR_BOUNDS;
  if (v & kStatusCapacity) return DLLM_ERR_CAPACITY;
  return DLLM_OK;
}

dllm_status dllm_prof_begin(void) {
  g_prof.on = true;
  g_prof.used = 0;
  g_prof.gemm_launches = 0;
  g_prof.kernel_launches = 0;
  return DLLM_OK;
}

dllm_status dllm_prof_end(double* gemm_ms, int32_t* gemm_launches, int32_t* kernel_launches) {
  double total = 0.0;
  dllm_status st = DLLM_OK;
  for (size_t i = 0; i + 1 < g_prof.used; i += 2) {
    if (cudaEventSynchronize(g_prof.ev[i + 1]) != cudaSuccess) { st = DLLM_ERR_CUDA; break; }
    float ms = 0.f;
    if (cudaEventElapsedTime(&ms, g_prof.ev[i], g_prof.ev[i + 1]) != cudaSuccess) { st = DLLM_ERR_CUDA; break; }
    total += ms;
  }
  if (gemm_ms) *gemm_ms = total;
  if (gemm_launches) *gemm_launches = g_prof.gemm_launches;
  if (kernel_launches) *kernel_launches = g_prof.kernel_launches;
  g_prof.on = false;
  g_prof.used = 0;
  return st;
}

dllm_status dllm_masked_logits_rules(const uint16_t* H, const uint8_t* M, const uint16_t* W, int32_t B,
                                     int32_t L, int32_t d, int32_t V, const int32_t* win_lo,
                                     const int32_t* win_hi, const dllm_logit_rules* rules, uint32_t stats,
                                     int32_t* tok, float* conf, float* lse, float* entropy, float* margin,
                                     int32_t* row_idx, int32_t* seq_off, int32_t* count, void* ws,
                                     size_t ws_bytes, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_masked_logits_rules");
  if (!W || !rules) return DLLM_ERR_NULL;
  ShapedArgs x{{H, M, W, B, L, d, V, win_lo, win_hi, stats, entropy, margin, tok, conf, lse, nullptr,
                row_idx, seq_off, count, ws, ws_bytes, static_cast<cudaStream_t>(stream)},
               nullptr, nullptr, rules};
  return run_shaped(x);
}

dllm_status dllm_token_counts(const int32_t* tokens, const uint8_t* M, const int32_t* n_valid, int32_t B,
                              int32_t n, int32_t V, int32_t accumulate, int32_t* counts, uint32_t* seen,
                              void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_token_counts");
  if ((!tokens && n != 0) || !counts || !seen) return DLLM_ERR_NULL;
  if (B < 1 || B > 65535 || n < 0 || V < 1 || V > kMaxColumns || (accumulate != 0 && accumulate != 1)) return DLLM_ERR_SHAPE;
  const void* ptrs[] = {tokens, M, n_valid, counts, seen};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return DLLM_ERR_ALIGN;
  if (accumulate && n == 0) return DLLM_OK;
  DeviceState* ds = nullptr;
  dllm_status st = device_state(&ds);
  if (st != DLLM_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (accumulate) {
    if (launch_pdl(rules::token_add_kernel, dim3(grid_for(n, rules::kCountThreads, ds->sms), B),
                   dim3(rules::kCountThreads), 0, s, tokens, M, n_valid, n, V, counts, seen) != cudaSuccess)
      return DLLM_ERR_CUDA;
  } else {
    // slices of the vocabulary: enough CTAs for every SM, at most what shared memory holds
    const long long per_seq = B < ds->sms ? ds->sms / B : 1;
    long long slice = ((V + per_seq - 1) / per_seq + 31) / 32 * 32;
    if (slice > rules::kCountMaxSlice) slice = rules::kCountMaxSlice;
    if (launch_pdl(rules::token_count_kernel, dim3(grid_for(V, static_cast<int>(slice), 1ll << 30), B),
                   dim3(rules::kCountThreads), static_cast<size_t>(slice) * 4, s, tokens, M, n_valid, n, V,
                   static_cast<int>(slice), counts, seen) != cudaSuccess)
      return DLLM_ERR_CUDA;
  }
  count_launch();
  return DLLM_OK;
}

size_t dllm_mx4_scale_bytes(int64_t rows, int32_t cols) {
  if (rows < 1 || rows >= (1ll << 31) || cols < 32 || cols % 32 != 0 || cols > kMaxColumns) return 0;
  return static_cast<size_t>(mx4::scale_bytes(rows, cols));
}

dllm_status dllm_mx4_quantize(const void* X, int32_t dtype, int64_t rows, int32_t cols, int64_t ld,
                              uint8_t* q, uint8_t* s, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_mx4_quantize");
  dllm_status st = mx4_checks(X, dtype, true, rows, cols, ld, q, s);
  if (st != DLLM_OK) return st;
  DeviceState* ds = nullptr;
  if ((st = device_state(&ds)) != DLLM_OK) return st;
  const dim3 grid(grid_for((rows + 127) / 128 * 128, mx4::kThreads / 32, static_cast<long long>(ds->sms) * mx4::kGridPerSm)), thr(mx4::kThreads);
  uint32_t* sw = reinterpret_cast<uint32_t*>(s);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == DLLM_BF16)
    e = launch_pdl(mx4::quantize_kernel<__nv_bfloat16>, grid, thr, 0, cs, static_cast<const __nv_bfloat16*>(X),
                   (long long)rows, cols, (long long)ld, q, sw);
  else if (dtype == DLLM_F16)
    e = launch_pdl(mx4::quantize_kernel<__half>, grid, thr, 0, cs, static_cast<const __half*>(X),
                   (long long)rows, cols, (long long)ld, q, sw);
  else
    e = launch_pdl(mx4::quantize_kernel<float>, grid, thr, 0, cs, static_cast<const float*>(X),
                   (long long)rows, cols, (long long)ld, q, sw);
  if (e != cudaSuccess) return DLLM_ERR_CUDA;
  count_launch();
  return DLLM_OK;
}

dllm_status dllm_mx4_dequantize(const uint8_t* q, const uint8_t* s, int64_t rows, int32_t cols, int32_t dtype,
                                void* X, int64_t ld, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_mx4_dequantize");
  dllm_status st = mx4_checks(X, dtype, false, rows, cols, ld, q, s);
  if (st != DLLM_OK) return st;
  DeviceState* ds = nullptr;
  if ((st = device_state(&ds)) != DLLM_OK) return st;
  const dim3 grid(grid_for(rows, mx4::kThreads / 32, static_cast<long long>(ds->sms) * mx4::kGridPerSm)), thr(mx4::kThreads);
  const uint32_t* sw = reinterpret_cast<const uint32_t*>(s);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DLLM_BF16
      ? launch_pdl(mx4::dequantize_kernel<__nv_bfloat16>, grid, thr, 0, cs, q, sw, (long long)rows, cols,
                   static_cast<__nv_bfloat16*>(X), (long long)ld)
      : launch_pdl(mx4::dequantize_kernel<float>, grid, thr, 0, cs, q, sw, (long long)rows, cols,
                   static_cast<float*>(X), (long long)ld);
  if (e != cudaSuccess) return DLLM_ERR_CUDA;
  count_launch();
  return DLLM_OK;
}

size_t dllm_workspace_bytes_mx4(int32_t B, int32_t L, int32_t d, int32_t V, int64_t max_rows) {
  if (!logits_shape_ok(B, L, d, V) || max_rows < 1) return 0;
  return ws_layout(B, L, d, V, max_rows, true).total;
}

int64_t dllm_workspace_rows_mx4(int32_t B, int32_t L, int32_t d, int32_t V, size_t ws_bytes) {
  if (!logits_shape_ok(B, L, d, V)) return 0;
  return ws_layout_for(B, L, d, V, ws_bytes, true).rows;
}

dllm_status dllm_masked_logits_mx4(const uint16_t* H, const uint8_t* M, const uint8_t* Wq, const uint8_t* Ws,
                                   int32_t B, int32_t L, int32_t d, int32_t V, const int32_t* win_lo,
                                   const int32_t* win_hi, const dllm_logit_rules* rules, uint32_t stats,
                                   int32_t* tok, float* conf, float* lse, float* entropy, float* margin,
                                   int32_t* row_idx, int32_t* seq_off, int32_t* count, void* ws,
                                   size_t ws_bytes, void* stream) {
  const dllm::NvtxRange nvtx_range("dllm_masked_logits_mx4");
  if (!Wq || !Ws) return DLLM_ERR_NULL;
  ShapedArgs x{{H, M, nullptr, B, L, d, V, win_lo, win_hi, stats, entropy, margin, tok, conf, lse, nullptr,
                row_idx, seq_off, count, ws, ws_bytes, static_cast<cudaStream_t>(stream)},
               Wq, Ws, rules};
  return run_shaped(x);
}

}  // extern "C"
