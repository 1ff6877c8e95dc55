// A1 -- placement plan: histogram of local (token, k) pairs, padded exclusive
// scan into expert offsets, stable rank of every pair inside its expert.
//
// StreamEP README, "How it works" (pool-layout dispatch): pairs land in an
// expert-major, tile-padded pool. Reading taken here: inside a segment pairs
// keep the order of q = t*K + k, a segment is ceil(count/tile)*tile rows, and
// ids outside [expert_begin, expert_begin + E_local) are not local.
//
// Scheme (no global atomics on counts, so every result is deterministic):
//   column c = a run of ppw consecutive pairs (1024; 256 for small batches), shared by W waves of a
//           block in order, so that a wave has 512 pairs at most.
//   pass 1  each wave counts its pairs per expert in its LDS row (LDS atomics); the column's sums
//           go to hist[c][e]. The last block to finish (a device-scope counter) reduces hist over
//           columns into counts, scans the padded counts into offsets (DPP wave scan) and turns
//           hist into per-column bases, several threads to an expert.
//   pass 2  each wave counts again, takes its bases from hist and the column's earlier waves, and
//           ranks its pairs: per 64 pairs, lanes with the same expert are matched with one
//           ballot per key bit, and a pair's row is the base plus its rank in the lane mask. Writes
//           pos and src; the plan's other arrays are filled by all blocks.
// With a single block both passes run in one launch and the columns' counts stay in LDS. It is latency
// alone: 128 experts, 65536 pairs 9.5 + 6.3 us (count and place), 8192 pairs 10.1, 1024 pairs 6.0; with one wave
// a column, a serial scan and fills a thread an expert 19.9 + 9.8, 15.0 + 7.9 and 14.7.
#include <algorithm>
#include <mutex>

#include "common.h"
#include "kernels.h"

namespace moe {

constexpr int kMaxExperts = 1024;

struct PlanArgs {
  const int32_t* topk_idx;
  int32_t pairs;          // T*K
  int32_t expert_begin;
  int32_t E;
  int32_t tile;
  int32_t tile_shift;     // log2(tile)
  int32_t key_bits;       // bits to tell local experts apart
  int32_t rows_cap;
  int32_t ntiles_cap;     // entries of tile_expert / tile_ready (rows_cap / tile)
  int32_t nfill;          // entries of the workspace's fill counters
  int32_t ncols;
  int32_t ppw;            // pairs per column
  int32_t col_waves;      // W: waves a column
  int32_t lanes_log2;     // scan: log2 of the threads side by side, which have the experts
  int32_t* counts;
  int32_t* offsets;
  int32_t* pos;
  int32_t* src;
  int32_t* tile_expert;
  int32_t* num_tiles;
  uint32_t* tile_ready;
  uint32_t* tile_fill;
  int32_t* hist;
  uint32_t* done;
  uint32_t* tiles_done;   // dispatch's count of raised ready flags
};

constexpr int kScanThreads = 64 * kPlanWaves;
constexpr int kWaveIters = 8;   // of 64 pairs a wave
constexpr int kScanKeep = 32;   // columns a scan thread keeps in registers

// A wave's pairs [begin, end): the local experts, -1 for none. Loaded up front, all in flight.
struct WavePairs {
  int begin, end;
  int e[kWaveIters];
  __device__ void load(const PlanArgs& a, int col, int part) {
    const int lane = lane_id();
    const int per_wave = a.ppw / a.col_waves;
    const int stop = min(a.pairs, (int)min((int64_t)a.pairs, ((int64_t)col + 1) * a.ppw));
    begin = (int)min((int64_t)stop, (int64_t)col * a.ppw + (int64_t)part * per_wave);
    end = min(stop, begin + per_wave);
    const __amdgpu_buffer_rsrc_t r = make_rsrc(a.topk_idx + begin, (uint32_t)(end - begin) * 4u);
#pragma unroll
    for (int i = 0; i < kWaveIters; ++i) {
      const int id = (int)__builtin_amdgcn_raw_buffer_load_b32(r, (uint32_t)(i * kWave + lane) * 4u, 0, 0);
      const int x = id - a.expert_begin;
      e[i] = begin + i * kWave + lane < end && id >= a.expert_begin && x < a.E ? x : -1;
    }
  }
  // whether all lanes have the same local expert
  __device__ static bool all_one(int x) {
    const int first = __builtin_amdgcn_readfirstlane(x);
    return first >= 0 && ballot(x != first) == 0;
  }
  // run[e] = the wave's pairs of e. RUNS: neighbouring pairs may well be of one expert (K = 1: rows of adapters, one request
  // behind another), and 64 additions to one word are 64 steps: 8192 rows in 16 runs 13.0 us so, 7.8 by one addition. A wave looks
  // for runs at its first and last pairs; a top-1 router's mixed ids pay for that (1024 of 128 experts 6.31 us without, 6.44 with, 7.01 with
  // every 64 pairs looked at; 8192 of 16 7.35, 7.48 and 7.76).
  template <bool RUNS>
  __device__ void count(const PlanArgs& a, int* run) const {
    for (int x = lane_id(); x < a.E; x += kWave) run[x] = 0;
    wave_sync();
    if (RUNS && __builtin_expect(all_one(e[0]) || all_one(e[kWaveIters - 1]), 0)) {
#pragma unroll
      for (int i = 0; i < kWaveIters; ++i) {
        const int first = __builtin_amdgcn_readfirstlane(e[i]);
        const bool one = ballot(e[i] != first) == 0;
        if (one ? (lane_id() == 0 && first >= 0) : e[i] >= 0) atomicAdd(&run[e[i]], one ? kWave : 1);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < kWaveIters; ++i)
      if (e[i] >= 0) atomicAdd(&run[e[i]], 1);
  }
  // run[e] = the row of the wave's first pair of e
  __device__ void place(const PlanArgs& a, int* run) const {
    const int lane = lane_id();
#pragma unroll
    for (int i = 0; i < kWaveIters; ++i) {
      const int q = begin + i * kWave + lane;
      if (begin + i * kWave >= end) break;
      const bool local = e[i] >= 0;
      const uint64_t peers = match_key(local ? (uint32_t)e[i] : 0u, local, a.key_bits);
      const int rank = mask_rank(peers);
      int row = -1;
      if (local) {
        const int b = run[e[i]];
        row = b + rank;
        if (rank == 0) run[e[i]] = b + __popcll(peers);
      }
      if (q < end) a.pos[q] = row;
      if (local) a.src[row] = q;
    }
  }
};

// Counts of the column's waves to bases, from the column's in hist: the lanes of its waves share the experts.
__device__ inline void wave_bases(const PlanArgs& a, int col, int part, int first_base, int (*rows)[kMaxExperts]) {
  for (int e = part * kWave + lane_id(); e < a.E; e += kWave * a.col_waves) {
    int run = e < kWave * a.col_waves ? first_base : a.hist[(int64_t)col * a.E + e];
    for (int v = 0; v < a.col_waves; ++v) {
      const int c = rows[v][e];
      rows[v][e] = run;
      run += c;
    }
  }
}

// What the plan holds beside pos and the real rows of src, by `waves` waves: padding rows, tile
// owners, and a fresh start for the dispatch that follows.
__device__ void plan_fill(const PlanArgs& a, const int* counts, const int* offsets, int wave, int waves) {
  const int lane = lane_id();
  for (int e = wave; e < a.E; e += waves) {
    const int seg = offsets[e], seg_end = offsets[e + 1];
    for (int r = seg + counts[e] + lane; r < seg_end; r += kWave) a.src[r] = -1;
    for (int t = (seg >> a.tile_shift) + lane; t < (seg_end >> a.tile_shift); t += kWave) a.tile_expert[t] = e;
  }
  const int P = offsets[a.E];
  const int64_t first = wave * kWave + lane, step = waves * kWave;   // rows_cap + step may pass 2^31
  for (int64_t t = (P >> a.tile_shift) + first; t < a.ntiles_cap; t += step) a.tile_expert[t] = -1;
  for (int64_t r = P + first; r < a.rows_cap; r += step) a.src[r] = -1;
  for (int64_t t = first; t < a.ntiles_cap; t += step) a.tile_ready[t] = 0u;
  for (int64_t t = first; t < a.nfill; t += step) a.tile_fill[t] = 0u;
  if (first == 0) *a.tiles_done = 0u;
}

struct ScanMem {
  int cnt[kMaxExperts], off[kMaxExperts + 1], part[kScanThreads], wave[kPlanWaves];
};

// counts and offsets, in memory and in `m`, from thread e's count of expert e; by a whole block
__device__ inline void plan_offsets(const PlanArgs& a, ScanMem& m, int count) {
  const int tid = threadIdx.x;
  const int E = a.E;
  const int padded = tid < E ? ((count + a.tile - 1) >> a.tile_shift) << a.tile_shift : 0;
  const int upto = wave_inclusive_scan(padded);
  if (lane_id() == 63) m.wave[tid >> 6] = upto;
  __syncthreads();
  int before = upto - padded, P = 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    const int t = m.wave[w];
    if (w < (tid >> 6)) before += t;
    P += t;
  }
  if (tid < E) {
    m.cnt[tid] = count;
    m.off[tid] = before;
    a.counts[tid] = count;
    a.offsets[tid] = before;
  }
  if (tid == 0) {
    m.off[E] = P;
    a.offsets[E] = P;
    a.num_tiles[0] = P >> a.tile_shift;
  }
  __syncthreads();
}

// The scan step, run by the last block of pass 1 (all its threads): thread (part, e) has a run of
// the columns of expert e.
__device__ void plan_scan(const PlanArgs& a, ScanMem& m) {
  const int tid = threadIdx.x;
  const int E = a.E;
  const int parts = kScanThreads >> a.lanes_log2;
  const int e = tid & ((1 << a.lanes_log2) - 1), part = tid >> a.lanes_log2;
  const int each = (a.ncols + parts - 1) / parts;
  const int c0 = min(a.ncols, part * each), c1 = e < E ? min(a.ncols, c0 + each) : c0;
  int32_t* h = a.hist + min(e, E - 1);
  // the first columns stay in registers; loads past the last read it again
  int v[kScanKeep];
#pragma unroll
  for (int i = 0; i < kScanKeep; ++i) v[i] = h[(int64_t)min(c0 + i, a.ncols - 1) * E];
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kScanKeep; ++i) {
    v[i] = c0 + i < c1 ? v[i] : 0;
    sum += v[i];
  }
#pragma unroll 16
  for (int col = c0 + kScanKeep; col < c1; ++col) sum += h[(int64_t)col * E];
  m.part[tid] = sum;
  __syncthreads();
  // an expert's count, and the pairs before each part
  int count = 0;
  if (tid < E) {
#pragma unroll 8
    for (int p = 0; p < parts; ++p) {
      const int c = m.part[(p << a.lanes_log2) + tid];
      m.part[(p << a.lanes_log2) + tid] = count;
      count += c;
    }
  }
  plan_offsets(a, m, count);
  // per-column bases
  int run = e < E ? m.off[e] + m.part[tid] : 0;
#pragma unroll
  for (int i = 0; i < kScanKeep; ++i) {
    if (c0 + i < c1) h[(int64_t)(c0 + i) * E] = run;
    run += v[i];
  }
#pragma unroll 16
  for (int col = c0 + kScanKeep; col < c1; ++col) {
    const int c = h[(int64_t)col * E];
    h[(int64_t)col * E] = run;
    run += c;
  }
}

template <bool RUNS>
__global__ __launch_bounds__(kScanThreads) void plan_count_kernel(PlanArgs a) {
  __shared__ int s_run[kPlanWaves][kMaxExperts];
  __shared__ ScanMem s_scan;
  __shared__ int s_last;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane_id();
  const int part = w % a.col_waves;
  const int col = blockIdx.x * (kPlanWaves / a.col_waves) + w / a.col_waves;
  WavePairs pairs;
  pairs.load(a, min(col, a.ncols - 1), part);
  if (col < a.ncols) pairs.count<RUNS>(a, s_run[w]);
  __syncthreads();
  if (gridDim.x == 1) {
    // single block: the waves' counts are all there is, and the pairs are placed right away
    int count = 0;
    if (threadIdx.x < a.E) {
#pragma unroll 4
      for (int v = 0; v < a.ncols * a.col_waves; ++v) {
        const int c = s_run[v][threadIdx.x];
        s_run[v][threadIdx.x] = count;
        count += c;
      }
    }
    plan_offsets(a, s_scan, count);
    if (col < a.ncols) {
      for (int e = lane; e < a.E; e += kWave) s_run[w][e] += s_scan.off[e];
      wave_sync();
      pairs.place(a, s_run[w]);
    }
    plan_fill(a, s_scan.cnt, s_scan.off, w, kPlanWaves);
    return;
  }
  if (col < a.ncols) {
    for (int e = part * kWave + lane; e < a.E; e += kWave * a.col_waves) {
      int c = 0;
      for (int v = w - part; v < w - part + a.col_waves; ++v) c += s_run[v][e];
      a.hist[(int64_t)col * a.E + e] = c;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
    const uint32_t prev = __hip_atomic_fetch_add(a.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    s_last = prev == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  plan_scan(a, s_scan);
  if (threadIdx.x == 0) __hip_atomic_store(a.done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <bool RUNS>
__global__ __launch_bounds__(kScanThreads) void plan_place_kernel(PlanArgs a) {
  __shared__ int s_run[kPlanWaves][kMaxExperts];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = w % a.col_waves;
  const int col = blockIdx.x * (kPlanWaves / a.col_waves) + w / a.col_waves;
  const int e = part * kWave + lane_id();
  WavePairs pairs;
  pairs.load(a, min(col, a.ncols - 1), part);
  const int first_base = a.hist[(int64_t)min(col, a.ncols - 1) * a.E + min(e, a.E - 1)];
  if (col < a.ncols) pairs.count<RUNS>(a, s_run[w]);
  __syncthreads();
  if (col < a.ncols) wave_bases(a, col, part, first_base, s_run + (w - part));
  __syncthreads();
  if (col < a.ncols) pairs.place(a, s_run[w]);
  plan_fill(a, a.counts, a.offsets, blockIdx.x * kPlanWaves + w, gridDim.x * kPlanWaves);
}

int launch_plan(const int32_t* topk_idx, const moe_plan_t& p, const WsLayout& L, char* ws,
                hipStream_t stream) {
  PlanArgs a;
  a.topk_idx = topk_idx;
  a.pairs = p.T * p.K;
  a.expert_begin = p.expert_begin;
  a.E = p.E_local;
  a.tile = p.tile;
  a.tile_shift = __builtin_ctz((unsigned)p.tile);
  int bits = 0;
  while ((1 << bits) < p.E_local) ++bits;
  a.key_bits = bits;
  a.rows_cap = p.rows_cap;
  a.ntiles_cap = p.rows_cap / p.tile;
  a.nfill = 2 * L.ntiles_cap;   // dispatch's and combine backward's counters (adjacent)
  a.ncols = L.ncols;
  a.ppw = L.ppw;
  // Four waves a column of 1024 pairs, one a column of 256; two and four where a block then still has
  // all columns: 8168 pairs in one launch of one block 8.5 us, in two of two blocks 9.3 + 5.4 (16384 pairs,
  // one wave a column: 15.3 and 8.2 + 6.5)
  a.col_waves = L.ncols <= kPlanWaves / 4 ? 4 : L.ppw == kPairsPerWave ? 1 : L.ncols <= kPlanWaves / 2 ? 2 : 4;
  a.lanes_log2 = bits < 5 ? 5 : bits;   // 32 parts at most
  a.counts = p.counts;
  a.offsets = p.offsets;
  a.pos = p.pos;
  a.src = p.src;
  a.tile_expert = p.tile_expert;
  a.num_tiles = p.num_tiles;
  a.tile_ready = p.tile_ready;
  a.tile_fill = reinterpret_cast<uint32_t*>(ws + L.fill);
  a.hist = reinterpret_cast<int32_t*>(ws + L.hist);
  a.done = reinterpret_cast<uint32_t*>(ws + L.done);
  a.tiles_done = reinterpret_cast<uint32_t*>(ws + L.tiles_done);
  const int cols = kPlanWaves / a.col_waves;   // a block's
  const int blocks = (L.ncols + cols - 1) / cols;
  const bool runs = p.K == 1;
  hipLaunchKernelGGL(runs ? plan_count_kernel<true> : plan_count_kernel<false>, dim3(blocks), dim3(kScanThreads), 0, stream, a);
  if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
  if (blocks > 1) {
    // blocks past the columns' only fill; 4 rows a thread (8192 pairs on 1024 experts: 18 us by two blocks)
    const int filling = std::min(256, p.rows_cap / (4 * kScanThreads) + 1);
    hipLaunchKernelGGL(runs ? plan_place_kernel<true> : plan_place_kernel<false>, dim3(std::max(blocks, filling)), dim3(kScanThreads), 0, stream, a);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
  }
  return MOE_OK;
}

// ----------------------------------------------------------------------------
// moe_plan_noalloc: moe_plan with its scratch (the per-column histogram and the blocks'
// completion counter) in a file-scope device array instead of a caller's workspace.
// Every call on a device shares that device's array.
// ----------------------------------------------------------------------------
constexpr size_t kPlanScratchBytes = (size_t)4 << 20;
static __device__ __align__(256) uint8_t scratch[kPlanScratchBytes];

// the array's device address, looked up once per device with that device current
static std::mutex g_scratch_mu;
static void* g_scratch_ptr[1024];

static void* plan_scratch_ptr() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 1024) return nullptr;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_ptr[dev] == nullptr) {
    void* ptr = nullptr;
    if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) != hipSuccess || ptr == nullptr) return nullptr;
    g_scratch_ptr[dev] = ptr;
  }
  return g_scratch_ptr[dev];
}

// the completion counter starts at zero (a kernel, not a memset, so the call can be captured
// in a graph)
__global__ void zero_word_kernel(uint32_t* w) { *w = 0u; }

}  // namespace moe

extern "C" MOE355_API int moe_plan_noalloc(const int32_t* topk_idx, const moe_plan_t* plan, void* stream) {
  using namespace moe;
  int rc = check_plan(plan);
  if (rc != MOE_OK) return rc;
  if (!topk_idx) return MOE_ERR_INVALID;
  WsLayout L = ws_layout(plan->T, plan->K, plan->E_local, plan->tile, 0, 0, MOE_BF16);
  if (L.hist + (size_t)L.ncols * plan->E_local * 4 > kPlanScratchBytes) return MOE_ERR_UNSUPPORTED;
  char* base = static_cast<char*>(plan_scratch_ptr());
  if (base == nullptr) return MOE_ERR_HIP;
  // no layer workspace: nothing is prepared for moe_dispatch (no fill counters to clear)
  L.ntiles_cap = 0;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(zero_word_kernel, dim3(1), dim3(1), 0, s, reinterpret_cast<uint32_t*>(base + L.done));
  if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
  return launch_plan(topk_idx, *plan, L, base, s);
}
