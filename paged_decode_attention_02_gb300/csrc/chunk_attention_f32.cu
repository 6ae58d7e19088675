// chunk_attention_f32.cu -- chunk attention over fp32 caches, in fp32 throughout (the tensor
// cores' 32-bit kind keeps 11 significant bits of its operands).
//
// A block of 256 threads walks its range of the batch's units as in the tensor-core kernel,
// with items of 64 rows. Thread (y, x) of 16 x 16 owns rows 4 y .. + 3: of the scores the keys
// x + 16 j of a 64-key step, of the output the columns 4 x + 64 j. Q, two K and V steps
// (cp.async, one in flight) and the probabilities lie in shared memory; a row's maximum and
// sum are reduced over the 16 threads that share it.
// Two 256-token chunks on 1024 of 32/8 heads run at 28.6 TFLOP/s (338 us), 38 % of the fp32
// lanes' rate. Bound by shared-memory loads (69 % of their rate while an SM works, the multiply-
// adds 51 %: a 4 x 4 tile loads eight 16-byte pieces for 64 of them), by SMs that end early (a
// quarter of their time) and, in short batches, by rows padded to 64.
#include <atomic>

#include "chunk_plan.cuh"

namespace pda {
namespace {

using CutsOf = Cuts<6, 4, 6>;  // 64-row items
constexpr int kRows = 64, kKeys = 64;

template <int D>
struct Smem {
  float q[kRows][D + 4];
  float k[2][kKeys][D + 4];  // padded: eight keys' 16-byte pieces lie in different banks
  float v[2][kKeys][D];
  float p[kKeys][kRows + 4];  // key-major, so a thread's four rows are one piece
  PlanMemory plan;
  Where first;
  int range[2];
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool there) {
  // a piece that is not there is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(there ? 16 : 0)
               : "memory");
}
template <int n>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

template <int D>
__global__ void __launch_bounds__(256, 1)
    chunk_f32_kernel(const ChunkParams p, int g_shift, float* partial) {
  constexpr int kCols = D / 16;  // output columns of a thread, four side by side
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int x = tid & 15, y = tid >> 4;
  const int lt = CutsOf::kRowsLog2 - g_shift;
  const Plan pl = make_plan<CutsOf>(p, lt, gridDim.x, &sm.plan);

  // requests without work whose rows are written all the same: padded (zeros) or in error (NaN)
  if (!pl.ok && blockIdx.x == 0 && tid == 0) atomic_or_error(p.error_word, PDA_DEVERR_QUERY);
  for (int b = pl.ok ? blockIdx.x : p.B; b < p.B; b += gridDim.x) {
    const int q0 = p.query_start[b], q1 = p.query_start[b + 1], L = p.context_lens[b];
    if (q0 == q1 || chunk_req(p, b, lt).r.n > 0) continue;
    if (L != 0 && tid == 0) atomic_or_error(p.error_word, PDA_DEVERR_CONTEXT_LEN);
    const float f = L == 0 ? 0.f : NAN;
    float4* rows = reinterpret_cast<float4*>(p.out) + static_cast<size_t>(q0) * p.H * (D / 4);
    const long long vecs = static_cast<long long>(q1 - q0) * p.H * (D / 4);
    for (long long i = tid; i < vecs; i += 256) rows[i] = make_float4(f, f, f, f);
  }

  if (warp == 0) {
    Where w{};
    int u = 0, u_end = 0;
    if (static_cast<int>(blockIdx.x) < pl.workers && pl.units > 0) {
      u = cut_of<CutsOf>(p, pl, lt, blockIdx.x + (lane & 1), &w);
      u_end = __shfl_sync(kFullMask, u, 1);
      u = __shfl_sync(kFullMask, u, 0);
      // lane 0's item is the block's; the others' are not
      if (lane == 0 && u < u_end && u >= w.start + w.q.r.tiles(w.i) + kItemUnits)
        next_item(p, lt, &w);
    }
    if (lane == 0) {
      sm.first = w;
      sm.range[0] = u;
      sm.range[1] = u_end;
    }
  }
  __syncthreads();
  Where w = sm.first;
  int u = sm.range[0];
  const int u_end = sm.range[1];
  const float* k_cache = static_cast<const float*>(p.k_cache);
  const float* v_cache = static_cast<const float*>(p.v_cache);

  while (u < u_end) {
    const ChunkReq r = w.q.r;
    const int tiles = r.tiles(w.i);
    const int end = w.start + tiles + kItemUnits;
    const int tok0 = w.i << lt, tokens = min(1 << lt, r.n - tok0);
    const int ja = u == w.start ? 0 : u - w.start - kItemUnits;
    const int jb = u_end >= end ? tiles : u_end - w.start - kItemUnits;
    const int pos0 = r.L - r.n + tok0, kv_end = pos0 + tokens;
    const int32_t* table = p.block_tables + static_cast<size_t>(w.b) * p.max_blocks;
    const int first_key = ja * kChunkKeys, last_key = min(kv_end, jb * kChunkKeys);
    const int steps = (last_key - first_key + kKeys - 1) / kKeys;
    int bad_from = 0x7fffffff;  // first key of a block with an id out of range

    // a warp loads every eighth row; ids are the same for all its lanes
    auto load = [&](int s) {
      const int buf = s & 1, key0 = first_key + s * kKeys;
      for (int i = warp; i < kKeys; i += 8) {
        const int key = key0 + i;
        bool there = key < last_key;
        int id = there ? table[key / p.block_size] : 0;
        if (id < 0 || id >= p.num_blocks) {
          bad_from = min(bad_from, max(key / p.block_size * p.block_size, first_key));
          if (lane == 0) atomic_or_error(p.error_word, PDA_DEVERR_BLOCK_ID);
          there = false;
          id = 0;
        }
        const size_t at =
            ((static_cast<size_t>(id) * p.block_size + key % p.block_size) * p.H_kv + w.kh) * D;
        if (4 * lane < D) {
          cp_async16(&sm.k[buf][i][4 * lane], k_cache + at + 4 * lane, there);
          cp_async16(&sm.v[buf][i][4 * lane], v_cache + at + 4 * lane, there);
        }
      }
      cp_async_commit();
    };
    __syncthreads();  // the item before is done with the buffers
    for (int i = tid; i < kRows * (D / 4); i += 256) {
      const int row = i / (D / 4), c = 4 * (i % (D / 4)), tok = row >> g_shift;
      const bool there = tok < tokens;
      const size_t at = ((static_cast<size_t>(w.q.row0 + tok0) + (there ? tok : 0)) * p.H +
                         (w.kh << g_shift) + (row & ((1 << g_shift) - 1))) * D + c;
      cp_async16(&sm.q[row][c], static_cast<const float*>(p.q) + at, there);
    }
    load(0);
    float m[4], l[4], o[4][kCols];
    int pos[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      m[a] = -INFINITY;
      l[a] = 0.f;
      pos[a] = pos0 + min((4 * y + a) >> g_shift, tokens - 1);
#pragma unroll
      for (int e = 0; e < kCols; ++e) o[a][e] = 0.f;
    }
    for (int s = 0; s < steps; ++s) {
      const int buf = s & 1, key0 = first_key + s * kKeys;
      if (s + 1 < steps) {
        load(s + 1);
        cp_async_wait<1>();
      } else {
        cp_async_wait<0>();
      }
      __syncthreads();
      float sc[4][4] = {};
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 qa[4], kb[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) qa[a] = *reinterpret_cast<const float4*>(&sm.q[4 * y + a][d]);
#pragma unroll
        for (int b = 0; b < 4; ++b)
          kb[b] = *reinterpret_cast<const float4*>(&sm.k[buf][x + 16 * b][d]);
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            sc[a][b] = fmaf(qa[a].x, kb[b].x, sc[a][b]);
            sc[a][b] = fmaf(qa[a].y, kb[b].y, sc[a][b]);
            sc[a][b] = fmaf(qa[a].z, kb[b].z, sc[a][b]);
            sc[a][b] = fmaf(qa[a].w, kb[b].w, sc[a][b]);
          }
      }
      // some row does not see the whole step: its V may not even be multiplied by zero
      const bool edge = key0 + kKeys - 1 > pos0;
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        float top = m[a];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          sc[a][b] = key0 + x + 16 * b <= pos[a] ? sc[a][b] * p.scale_log2 : -INFINITY;
          top = fmaxf(top, sc[a][b]);
        }
#pragma unroll
        for (int i = 1; i < 16; i <<= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, i));
        const float ref = top == -INFINITY ? 0.f : top;
        const float c = ex2(m[a] - ref);
        m[a] = top;
        l[a] *= c;
#pragma unroll
        for (int e = 0; e < kCols; ++e) o[a][e] *= c;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          sc[a][b] = ex2(sc[a][b] - ref);
          l[a] += sc[a][b];
        }
      }
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *reinterpret_cast<float4*>(&sm.p[x + 16 * b][4 * y]) =
            make_float4(sc[0][b], sc[1][b], sc[2][b], sc[3][b]);
      __syncwarp();  // a warp reads back its own rows only
      const int keys = min(kKeys, last_key - key0);
      auto accumulate = [&](int j, bool masked) {
        const float4 pr = *reinterpret_cast<const float4*>(&sm.p[j][4 * y]);
        const float pa[4] = {pr.x, pr.y, pr.z, pr.w};
#pragma unroll
        for (int e = 0; e < kCols; e += 4) {
          const float4 v = *reinterpret_cast<const float4*>(&sm.v[buf][j][16 * e + 4 * x]);
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            if (masked && key0 + j > pos[a]) continue;
            o[a][e] = fmaf(pa[a], v.x, o[a][e]);
            o[a][e + 1] = fmaf(pa[a], v.y, o[a][e + 1]);
            o[a][e + 2] = fmaf(pa[a], v.z, o[a][e + 2]);
            o[a][e + 3] = fmaf(pa[a], v.w, o[a][e + 3]);
          }
        }
      };
      if (edge || keys < kKeys) {
        for (int j = 0; j < keys; ++j) accumulate(j, true);
      } else {
#pragma unroll 8
        for (int j = 0; j < kKeys; ++j) accumulate(j, false);
      }
      __syncthreads();  // the step's buffers are free
    }
    // the smallest bad_from of the block's warps (rarely any)
    if (__syncthreads_or(bad_from != 0x7fffffff)) {
      int* all = reinterpret_cast<int*>(&sm.p[0][0]);
      if (lane == 0) all[warp] = bad_from;
      __syncthreads();
      for (int i = 0; i < 8; ++i) bad_from = min(bad_from, all[i]);
      __syncthreads();
    }
    const int part =
        ja == 0 && jb == tiles ? -1 : static_cast<int>(blockIdx.x) * 2 + (ja == 0 ? 1 : 0);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
#pragma unroll
      for (int i = 1; i < 16; i <<= 1) l[a] += __shfl_xor_sync(kFullMask, l[a], i);
      const int row = 4 * y + a, tok = row >> g_shift;
      if (tok >= tokens) continue;
      const bool dead = pos[a] >= bad_from;
      if (part >= 0) {
        if (x == 0) part_ml(partial, part, D)[row] = make_float2(m[a], dead ? NAN : l[a]);
#pragma unroll
        for (int e = 0; e < kCols; e += 4)
          part_o(partial, part, D)[(4 * e + x) * 256 + row] =
              make_float4(o[a][e], o[a][e + 1], o[a][e + 2], o[a][e + 3]);
      } else {
        const float inv = dead ? NAN : p.v_scale / l[a];
        float* out = static_cast<float*>(p.out) +
                     ((static_cast<size_t>(w.q.row0 + tok0) + tok) * p.H + (w.kh << g_shift) +
                      (row & ((1 << g_shift) - 1))) * D;
#pragma unroll
        for (int e = 0; e < kCols; e += 4)
          store4(out + 16 * e + 4 * x, o[a][e] * inv, o[a][e + 1] * inv, o[a][e + 2] * inv,
                 o[a][e + 3] * inv);
      }
    }
    // the next item
    u = end;
    if (u < u_end) next_item(p, lt, &w);
  }
}

template <int D>
pda_status launch(const ChunkParams& p, int dev, int sms, bool capped, float* partial,
                  cudaStream_t stream) {
  constexpr int smem = static_cast<int>(sizeof(Smem<D>));
  static_assert(smem <= 232448, "227 KB a block");
  static std::atomic<bool> raised[64];
  if (dev >= 64 || !raised[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(chunk_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem) != cudaSuccess)
      return PDA_ERR_CUDA;
    if (dev < 64) raised[dev].store(true, std::memory_order_release);
  }
  int g_shift = 0;
  while ((1 << g_shift) < p.G) ++g_shift;
  const int grid = chunk_grid<CutsOf>(p, g_shift, sms);
  chunk_f32_kernel<D><<<grid, 256, smem, stream>>>(p, g_shift, partial);
  if (cudaGetLastError() != cudaSuccess) return PDA_ERR_CUDA;
  return launch_merge<D, float, CutsOf>(p, g_shift, partial, grid, capped, stream);
}

}  // namespace

pda_status launch_chunk_f32(const ChunkParams& p, int D, int dev, int sms, bool capped,
                            void* workspace, cudaStream_t stream) {
  float* partial = static_cast<float*>(workspace);
  return D == 128 ? launch<128>(p, dev, sms, capped, partial, stream)
                  : launch<64>(p, dev, sms, capped, partial, stream);
}

}  // namespace pda
