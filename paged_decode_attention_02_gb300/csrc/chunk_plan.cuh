// chunk_plan.cuh -- the device side of chunk_plan.h, shared by the chunk-attention kernels: the
// plan every block makes of the batch's work, the partial results of cut items, their merge.
#pragma once

#include <algorithm>

#include "chunk_internal.h"
#include "chunk_plan.h"
#include "pda_device.cuh"

namespace pda {

// How a kernel cuts its work: log2 of an item's rows, the fewest key tiles of a cut item's
// piece, and the fewest units of a worker's range.
template <int rows_log2, int piece_tiles, int worker_units>
struct Cuts {
  static constexpr int kRowsLog2 = rows_log2, kPieceTiles = piece_tiles,
                       kWorkerUnits = worker_units;
};

// ---------------------------------------------------------------- plan
// Units of the requests [0, c * per) for every c, built by all threads of the block.
constexpr int kPlanChunks = 256;

struct Req {
  int row0;  // first row of q and out
  ChunkReq r;
};

struct PlanMemory {
  int prefix[kPlanChunks + 1];
  int3 req[kPlanChunks];  // (row0, n, L) of each request, where there are no more than this
};

struct Plan {
  PlanMemory* mem;
  int per, workers, units;
  bool ok;  // query_start never decreases and stays within [0, T]; otherwise there is no work
};

struct Where {
  int b, kh, i, start;  // start: a unit
  Req q;
};

// A request with work to do; n = 0 for one without (empty, padded or in error).
__device__ __forceinline__ Req chunk_req(const ChunkParams& p, int b, int lt) {
  const int q0 = p.query_start[b], q1 = p.query_start[b + 1], L = p.context_lens[b];
  const bool ok = q0 >= 0 && q1 <= p.T && q0 < q1 && L >= q1 - q0 && L <= p.max_context_len &&
                  L <= static_cast<long long>(p.max_blocks) * p.block_size;
  return Req{q0, ChunkReq{ok ? q1 - q0 : 0, ok ? L : 0, lt}};
}

// Called by all threads of a block of at least 256.
template <typename C>
__device__ __forceinline__ Plan make_plan(const ChunkParams& p, int lt, int workers,
                                          PlanMemory* mem) {
  Plan pl;
  pl.mem = mem;
  pl.per = (p.B + kPlanChunks - 1) / kPlanChunks;
  const int c = threadIdx.x, lane = c & 31;
  int x = 0;
  bool bad = false;
  if (c < kPlanChunks)
    for (int b = c * pl.per; b < min(p.B, (c + 1) * pl.per); ++b) {
      const Req q = chunk_req(p, b, lt);
      bad |= q.row0 < 0 || q.row0 > p.query_start[b + 1] || p.query_start[b + 1] > p.T;
      x += q.r.units();
      if (pl.per == 1) mem->req[b] = make_int3(q.row0, q.r.n, q.r.L);
    }
  x *= p.H_kv;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFullMask, x, o);
    if (lane >= o) x += y;
  }
  if (c < kPlanChunks) mem->prefix[c + 1] = x;
  // overlapping requests could be any amount of work, so there is none at all
  pl.ok = !__syncthreads_or(bad);
  int before = 0;
  if (c < kPlanChunks)
    for (int w = 0; w < (c >> 5); ++w) before += mem->prefix[32 * w + 32];
  __syncthreads();
  if (c < kPlanChunks) mem->prefix[c + 1] = x + before;
  if (c == 0) mem->prefix[0] = 0;
  __syncthreads();
  pl.units = pl.ok ? mem->prefix[kPlanChunks] : 0;
  pl.workers = chunk_workers(pl.units, workers, C::kWorkerUnits);
  return pl;
}

// The item that holds unit u < units. Valid while the plan's memory is.
__device__ __forceinline__ Where locate(const ChunkParams& p, const Plan& pl, int lt, int u) {
  int lo = 0, hi = kPlanChunks - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pl.mem->prefix[mid + 1] > u)
      hi = mid;
    else
      lo = mid + 1;
  }
  int at = pl.mem->prefix[lo];
  int b = lo * pl.per;
  Req q;
  if (pl.per == 1) {
    const int3 v = pl.mem->req[b];
    q = Req{v.x, ChunkReq{v.y, v.z, lt}};
  } else {
    q = chunk_req(p, b, lt);
  }
  int one = q.r.units();
  while (at + one * p.H_kv <= u) {
    at += one * p.H_kv;
    q = chunk_req(p, ++b, lt);
    one = q.r.units();
  }
  const int kh = static_cast<unsigned>(u - at) / static_cast<unsigned>(one);
  at += kh * one;
  const int i = q.r.item_of(u - at);
  return Where{b, kh, i, at + q.r.units_before(i), q};
}

// Moves on to the item behind, of a batch that has one.
__device__ __forceinline__ void next_item(const ChunkParams& p, int lt, Where* w) {
  w->start += w->q.r.tiles(w->i) + kItemUnits;
  if (++w->i < w->q.r.items()) return;
  w->i = 0;
  if (++w->kh < p.H_kv) return;
  w->kh = 0;
  do {
    w->q = chunk_req(p, ++w->b, lt);
  } while (w->q.r.n == 0 && w->b + 1 < p.B);
}

// The cut before worker c, snapped; *w: the item it falls into (for a cut below `units`).
template <typename C>
__device__ __forceinline__ int cut_of(const ChunkParams& p, const Plan& pl, int lt, int c,
                                      Where* w) {
  const int u = chunk_cut(pl.units, pl.workers, c);
  if (u >= pl.units) return pl.units;
  *w = locate(p, pl, lt, u);
  return chunk_snap(u, w->start, w->q.r.tiles(w->i), C::kPieceTiles);
}

// ---------------------------------------------------------------- partial results
// A cut item's: per slot (m, l) of 256 rows, then O as [D / 4][256] float4.
__host__ __device__ constexpr size_t part_floats(int D) { return 256 * (D + 2); }
__device__ __forceinline__ float2* part_ml(float* partial, int slot, int D) {
  return reinterpret_cast<float2*>(partial + slot * part_floats(D));
}
__device__ __forceinline__ float4* part_o(float* partial, int slot, int D) {
  return reinterpret_cast<float4*>(partial + slot * part_floats(D) + 512);
}

// Two values rounded to a pair of bf16 or fp16.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (kBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void store4(__nv_bfloat16* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2<true>(a, b), pack2<true>(c, d));
}
__device__ __forceinline__ void store4(__half* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2<false>(a, b), pack2<false>(c, d));
}
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}

// ---------------------------------------------------------------- merge of cut items
// Block x handles the item that cut x + 1 falls into, if that is the first cut inside it:
// piece i of a row holds (m_i, l_i, O_i); with M = max m_i the row is
// sum O_i 2^(m_i - M) / sum l_i 2^(m_i - M). A lane takes a row, a warp 32 rows and every
// eighth group of four columns. Eight warps share 32 rows; an item's rows are spread over the
// grid's y or, in a capped call, over the warps of one block a cut and a loop, so that there are
// no more blocks than the cap has SMs.
constexpr int kMergeRows = 32;
constexpr int kMergeThreads = 256;  // of 32 rows

template <int D, typename Out, typename C>
__global__ void __launch_bounds__(1024)
    chunk_merge_kernel(const ChunkParams p, int g_shift, float* partial, int grid) {
  __shared__ PlanMemory mem;
  const int lt = C::kRowsLog2 - g_shift;
  const Plan pl = make_plan<C>(p, lt, grid, &mem);
  const int c = blockIdx.x + 1;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 7;
  const int sets = static_cast<int>(blockDim.x) / kMergeThreads;
  const int first = (blockIdx.y * sets + threadIdx.x / kMergeThreads) * kMergeRows;
  int pieces = 0, rows = 0;
  Where w{};
  if (c < pl.workers) {
    // the cut and, on the odd lanes, the one before it
    const int s = cut_of<C>(p, pl, lt, c - (lane & 1), &w);
    const int tiles = w.q.r.tiles(w.i);
    const int end = w.start + tiles + kItemUnits;
    const int before = __shfl_sync(kFullMask, s, 1);
    if (lane == 0 && s > w.start && s < end && before <= w.start) {
      pieces = 2;  // worker c - 1's, and one for each cut inside the item
      for (; c + pieces - 1 < pl.workers; ++pieces) {
        const int u = chunk_cut(pl.units, pl.workers, c + pieces - 1);
        if (u >= end || chunk_snap(u, w.start, tiles, C::kPieceTiles) >= end) break;
      }
      rows = min(1 << lt, w.q.r.n - (w.i << lt)) << g_shift;
    }
    pieces = __shfl_sync(kFullMask, pieces, 0);
    rows = __shfl_sync(kFullMask, rows, 0);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are written
  if (first >= rows) return;
  const int row0 = __shfl_sync(kFullMask, w.q.row0 + (w.i << lt), 0);
  const int kh = __shfl_sync(kFullMask, w.kh, 0);
  auto slot = [&](int i) { return i == 0 ? 2 * (c - 1) + 1 : 2 * (c + i - 1); };
  for (int r = first + lane; r < rows; r += gridDim.y * sets * kMergeRows) {
    float M = -INFINITY;
#pragma unroll 4
    for (int i = 0; i < pieces; ++i) M = fmaxf(M, part_ml(partial, slot(i), D)[r].x);
    constexpr int V = D / 32;  // groups of four columns of a warp
    float l = 0.f;
    float4 acc[V] = {};
#pragma unroll 2
    for (int i = 0; i < pieces; ++i) {
      const float2 ml = part_ml(partial, slot(i), D)[r];
      if (ml.x == -INFINITY && !isnan(ml.y)) continue;  // the row sees none of the piece's keys
      const float wgt = ex2(ml.x - M);
      l = fmaf(wgt, ml.y, l);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float4 o = part_o(partial, slot(i), D)[(warp + 8 * e) * 256 + r];
        acc[e].x = fmaf(wgt, o.x, acc[e].x);
        acc[e].y = fmaf(wgt, o.y, acc[e].y);
        acc[e].z = fmaf(wgt, o.z, acc[e].z);
        acc[e].w = fmaf(wgt, o.w, acc[e].w);
      }
    }
    const float inv = p.v_scale / l;
    Out* out = static_cast<Out*>(p.out) +
               ((static_cast<size_t>(row0) + (r >> g_shift)) * p.H + (kh << g_shift) +
                (r & ((1 << g_shift) - 1))) * D;
#pragma unroll
    for (int e = 0; e < V; ++e)
      store4(out + 4 * (warp + 8 * e), acc[e].x * inv, acc[e].y * inv, acc[e].z * inv,
             acc[e].w * inv);
  }
}

// ---------------------------------------------------------------- host side
// Most key tiles of an item, by the host's bound on the lengths.
inline int chunk_tiles(const ChunkParams& p) {
  const long long cap = static_cast<long long>(p.max_blocks) * p.block_size;
  const long long keys = std::min<long long>(p.max_context_len, cap);
  return static_cast<int>((keys + kChunkKeys - 1) / kChunkKeys);
}
// Blocks of a launch: no more than that bound can keep busy.
template <typename C>
long long chunk_units(const ChunkParams& p, int g_shift) {
  const long long items =
      ((static_cast<long long>(p.T) >> (C::kRowsLog2 - g_shift)) + p.B) * p.H_kv;
  return items * (chunk_tiles(p) + kItemUnits);
}
template <typename C>
int chunk_grid(const ChunkParams& p, int g_shift, int sms) {
  return chunk_workers(chunk_units<C>(p, g_shift), sms, C::kWorkerUnits);
}

// Merges what the kernel before it on the stream has cut, where anything can have been. Without
// a cap the merge starts early and looks its items up beside that kernel's last blocks; with one
// (`capped`) it waits for its end, and its grid - 1 blocks fit the cap that `grid` keeps to.
template <int D, typename Out, typename C>
pda_status launch_merge(const ChunkParams& p, int g_shift, float* partial, int grid, bool capped,
                        cudaStream_t stream) {
  if (grid == 1 || chunk_tiles(p) < 2 * C::kPieceTiles) return PDA_OK;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  constexpr int kSets = (1 << C::kRowsLog2) / kMergeRows;
  cfg.gridDim = dim3(static_cast<unsigned>(grid - 1), capped ? 1 : kSets);
  cfg.blockDim = dim3((capped ? std::min(kSets, 4) : 1) * kMergeThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = capped ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, chunk_merge_kernel<D, Out, C>, p, g_shift, partial, grid) ==
                 cudaSuccess
             ? PDA_OK
             : PDA_ERR_CUDA;
}

}  // namespace pda
