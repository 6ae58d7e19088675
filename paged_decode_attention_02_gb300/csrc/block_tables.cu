// block_tables.cu -- the paged cache's bookkeeping of one step, on the GPU: block tables
// grown and shrunk to the requests' lengths, and the slot of every new token.
//
// Both are integer prefix sums over the requests followed by one gather or scatter per block
// entry or token. The bytes are few (a step of 512 requests moves half a megabyte), so what
// bounds them is latency: one launch each, the prefix sums repeated in every thread block
// (8192 lengths are 32 KB of L2 reads) rather than passed through memory from a first kernel.
#include <cooperative_groups.h>

#include <atomic>

#include "pda_device.cuh"
#include "pda_internal.h"

namespace pda {

constexpr int kTableMaxBatch = 8192;  // requests a call takes (as the attention's)

// Exclusive prefix sum of one value per thread over the block; *total is the block's sum.
// `warp_sums` holds 32 values of shared memory; ends with the block synchronised.
template <typename T>
__device__ __forceinline__ T block_exclusive_scan(T v, T* warp_sums, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nwarps = static_cast<int>(blockDim.x) >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kFullMask, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T s = lane < nwarps ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(kFullMask, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const T before = warp == 0 ? 0 : warp_sums[warp - 1];
  *total = warp_sums[31];
  __syncthreads();
  return before + x - v;
}

// The first b with end[b] > i, for a non-decreasing `end` whose last element is above i.
__device__ __forceinline__ int owner_of(const int* end, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > i)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// ---------------------------------------------------------------- block assignment
// need_b = ceil(L_b / block_size). Rows that shrink push entries [max(need, shared), held)
// onto the stack free_list[0, F); rows that grow pop need - held entries off its top, first
// come first served in row order. A row that grows from inside its shared prefix owns what it
// gets there, so the prefix ends at held from then on.
//
// One cluster of 8 blocks does the whole call: every block reads the lengths, the held
// counts and F and computes both prefix sums; the cluster's barrier then separates the pushes
// (and every other block's read of `held`, `shared_blocks` and F) from the pops and from the
// writes of the new counts, so the outputs may be the inputs' own buffers and no workspace or
// second launch is needed.
constexpr int kAssignCluster = 8;
constexpr int kAssignThreads = 1024;

__global__ void __cluster_dims__(kAssignCluster, 1, 1) __launch_bounds__(kAssignThreads)
    kv_assign_kernel(int32_t* tables, const int32_t* held, int32_t* held_out, int32_t* free_list,
                     const int32_t* free_count, int32_t* free_count_out, const int32_t* lens,
                     int32_t* shared_blocks, int B, int max_blocks, int block_size,
                     int num_blocks, int32_t* error_word) {
  extern __shared__ int smem_ints[];
  __shared__ int warp_sums[32];
  __shared__ int granted_sh;
  int* back_end = smem_ints;    // prefix ends of the blocks given back
  int* grow_end = back_end + B; // prefix ends of the blocks asked for
  int* base = grow_end + B;     // first table column the row gives back or fills
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x;
  const int F = free_count[0];

  // this thread's rows [b0, b1)
  const int per = (B + kAssignThreads - 1) / kAssignThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  int back = 0, grow = 0;
  bool bad_len = false;
  for (int b = b0; b < b1; ++b) {
    const int h = held[b], L = lens[b];
    int r = 0, g = 0, at = 0;
    if (h < 0 || h > max_blocks || L < 0 ||
        L > static_cast<long long>(max_blocks) * block_size) {
      bad_len = true;
    } else {
      const int need = static_cast<int>((static_cast<long long>(L) + block_size - 1) / block_size);
      if (need > h) {
        g = need - h;
        at = h;
      } else {
        const int keep = shared_blocks != nullptr ? max(need, shared_blocks[b]) : need;
        r = max(h - keep, 0);
        at = keep;
      }
    }
    back += r;
    grow += g;
    back_end[b] = back;
    grow_end[b] = grow;
    base[b] = at;
  }
  if (tid == 0) granted_sh = 0;
  int R, A;
  const int back0 = block_exclusive_scan<int>(back, warp_sums, &R);
  const int grow0 = block_exclusive_scan<int>(grow, warp_sums, &A);
  // an unusable stack (a count out of range, or more given back than it can hold) leaves
  // everything as it was
  const bool stack_ok = F >= 0 && F <= num_blocks;
  const bool room_ok = stack_ok && R <= num_blocks - F;
  const int top = room_ok ? F + R : 0;
  int granted = 0;
  for (int b = b0; b < b1; ++b) {
    back_end[b] += back0;
    grow_end[b] += grow0;
    if (grow_end[b] <= top) granted = grow_end[b];
  }
  granted = __reduce_max_sync(kFullMask, granted);
  if ((tid & 31) == 0 && granted > 0) atomicMax(&granted_sh, granted);
  __syncthreads();
  granted = granted_sh;
  if (rank == 0) {
    if (bad_len) atomic_or_error(error_word, PDA_DEVERR_CONTEXT_LEN);
    if (tid == 0 && (!stack_ok || (room_ok && granted < A)))
      atomic_or_error(error_word, PDA_DEVERR_NO_BLOCKS);
    if (tid == 0 && stack_ok && !room_ok) atomic_or_error(error_word, PDA_DEVERR_BLOCK_ID);
  }

  const int first = rank * kAssignThreads + tid;
  bool bad_id = false;
  if (room_ok) {
    for (int i = first; i < R; i += kAssignCluster * kAssignThreads) {
      const int b = owner_of(back_end, B, i);
      const int j = base[b] + i - (b > 0 ? back_end[b - 1] : 0);
      const int id = tables[static_cast<size_t>(b) * max_blocks + j];
      bad_id |= id < 0 || id >= num_blocks;
      free_list[F + i] = id;
    }
  }
  cluster.sync();
  if (room_ok) {
    for (int i = first; i < granted; i += kAssignCluster * kAssignThreads) {
      const int b = owner_of(grow_end, B, i);
      const int j = base[b] + i - (b > 0 ? grow_end[b - 1] : 0);
      const int id = free_list[top - 1 - i];
      bad_id |= id < 0 || id >= num_blocks;
      tables[static_cast<size_t>(b) * max_blocks + j] = id;
    }
  }
  if (bad_id) atomic_or_error(error_word, PDA_DEVERR_BLOCK_ID);
  for (int b = first; b < B; b += kAssignCluster * kAssignThreads) {
    const int h = held[b], L = lens[b];  // held[b] is written by this thread alone
    const bool bad = h < 0 || h > max_blocks || L < 0 ||
                     L > static_cast<long long>(max_blocks) * block_size;
    int now = h;
    if (!bad && room_ok) {
      const int need = static_cast<int>((static_cast<long long>(L) + block_size - 1) / block_size);
      if (need <= h || grow_end[b] <= granted) {
        now = need;
        if (need > h && shared_blocks != nullptr && shared_blocks[b] > h) shared_blocks[b] = h;
      }
    }
    held_out[b] = now;
  }
  if (rank == 0 && tid == 0) free_count_out[0] = room_ok ? top - granted : F;
}

// ---------------------------------------------------------------- slots of new tokens
// Token i of request b (n_b new tokens of L_b) is at position p = L_b - n_b + i, in slot
// table[b][p / block_size] * block_size + p % block_size. Each block scans the lengths,
// then its threads find their tokens' requests in the prefix ends (in shared memory).
constexpr int kSlotThreads = 256;
constexpr int kSlotPerThread = 4;

__global__ void __launch_bounds__(kSlotThreads)
    kv_slots_kernel(int32_t* __restrict__ slots, int32_t* __restrict__ query_start,
                    const int32_t* __restrict__ query_lens, const int32_t* __restrict__ lens,
                    const int32_t* __restrict__ tables, int N, int B, int max_blocks,
                    int block_size, int num_blocks, int32_t* error_word) {
  extern __shared__ int smem_ints[];
  __shared__ long long warp_sums[32];
  int* end = smem_ints;  // prefix ends, clipped at N
  const int tid = threadIdx.x;
  const int per = (B + kSlotThreads - 1) / kSlotThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  // each thread's sum saturates at N + 1 and the block's is taken in 64 bits, so no list of
  // lengths overflows
  int sum = 0;
  bool bad_query = false;
  for (int b = b0; b < b1; ++b) {
    const int n = query_lens[b];
    bad_query |= n < 0;
    sum = n > N - sum ? N + 1 : sum + max(n, 0);
    end[b] = sum;
  }
  long long total;
  const long long before = block_exclusive_scan<long long>(sum, warp_sums, &total);
  for (int b = b0; b < b1; ++b)
    end[b] = static_cast<int>(min(static_cast<long long>(N), before + end[b]));
  if (blockIdx.x == 0) {
    if (bad_query || (tid == 0 && total > N)) atomic_or_error(error_word, PDA_DEVERR_QUERY);
    if (tid == 0) query_start[0] = 0;
    for (int b = b0; b < b1; ++b) {
      query_start[b + 1] = end[b];
      const int L = lens[b], n = query_lens[b];
      if (L < 0 || L > static_cast<long long>(max_blocks) * block_size || (L > 0 && L < n))
        atomic_or_error(error_word, PDA_DEVERR_CONTEXT_LEN);
    }
  }
  __syncthreads();
  const int used = B > 0 ? end[B - 1] : 0;
  for (int k = 0; k < kSlotPerThread; ++k) {
    const long long at =
        (static_cast<long long>(blockIdx.x) * kSlotPerThread + k) * kSlotThreads + tid;
    if (at >= N) break;
    const int t = static_cast<int>(at);
    int slot = -1;
    if (t < used) {
      const int b = owner_of(end, B, t);
      const int L = lens[b], n = query_lens[b];
      if (L >= n && L <= static_cast<long long>(max_blocks) * block_size) {
        const int p = L - n + t - (b > 0 ? end[b - 1] : 0);
        const int id = tables[static_cast<size_t>(b) * max_blocks + p / block_size];
        if (id < 0 || id >= num_blocks)
          atomic_or_error(error_word, PDA_DEVERR_BLOCK_ID);
        else
          slot = id * block_size + p % block_size;
      }
    }
    slots[t] = slot;
  }
}

namespace {

// Shared memory of an assignment, 12 bytes a row. Together with the kernel's own it passes the
// default 48 KB from 4085 rows on, so the limit is raised, once a device, to what the largest
// batch takes: a limit of each call's own size could be lowered by one host thread between
// another's raise and its launch. (Slots take 4 bytes a row: 32 KB at most.)
constexpr size_t assign_smem(int B) { return static_cast<size_t>(B) * 3 * sizeof(int); }

bool raise_assign_smem() {
  static std::atomic<bool> raised[64];
  int dev;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < 64 && raised[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kv_assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(assign_smem(kTableMaxBatch))) != cudaSuccess)
    return false;
  if (dev < 64) raised[dev].store(true, std::memory_order_release);
  return true;
}

pda_status check_tables(int B, int max_blocks, int block_size, int num_blocks) {
  if (B < 0 || max_blocks < 0 || block_size <= 0 || num_blocks <= 0) return PDA_ERR_INVALID_ARG;
  if (B > kTableMaxBatch || static_cast<long long>(B) * max_blocks >= (1ll << 31) ||
      static_cast<long long>(num_blocks) * block_size >= (1ll << 31))
    return PDA_ERR_UNSUPPORTED;
  return PDA_OK;
}

}  // namespace
}  // namespace pda

using namespace pda;

extern "C" pda_status pda_kv_assign_blocks(int32_t* block_tables, const int32_t* blocks_held,
                                           int32_t* blocks_held_out, int32_t* free_list,
                                           const int32_t* free_count, int32_t* free_count_out,
                                           const int32_t* context_lens,
                                           int32_t* shared_blocks, int B,
                                           int max_blocks_per_seq, int block_size,
                                           int num_blocks, int32_t* error_word,
                                           cudaStream_t stream) {
  const pda_status st = check_tables(B, max_blocks_per_seq, block_size, num_blocks);
  if (st != PDA_OK) return st;
  if (free_list == nullptr || free_count == nullptr || free_count_out == nullptr)
    return PDA_ERR_INVALID_ARG;
  if (B > 0 && (block_tables == nullptr || blocks_held == nullptr || blocks_held_out == nullptr ||
                context_lens == nullptr))
    return PDA_ERR_INVALID_ARG;
  if (!raise_assign_smem()) return PDA_ERR_CUDA;
  kv_assign_kernel<<<kAssignCluster, kAssignThreads, assign_smem(B), stream>>>(
      block_tables, blocks_held, blocks_held_out, free_list, free_count, free_count_out,
      context_lens, shared_blocks, B, max_blocks_per_seq, block_size, num_blocks, error_word);
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}

extern "C" pda_status pda_kv_build_slots(int32_t* slot_mapping, int32_t* query_start,
                                         const int32_t* query_lens, const int32_t* context_lens,
                                         const int32_t* block_tables, int N, int B,
                                         int max_blocks_per_seq, int block_size, int num_blocks,
                                         int32_t* error_word, cudaStream_t stream) {
  if (N < 0) return PDA_ERR_INVALID_ARG;
  if (N > (1 << 30)) return PDA_ERR_UNSUPPORTED;
  const pda_status st = check_tables(B, max_blocks_per_seq, block_size, num_blocks);
  if (st != PDA_OK) return st;
  if (query_start == nullptr || (N > 0 && slot_mapping == nullptr)) return PDA_ERR_INVALID_ARG;
  if (B > 0 && (query_lens == nullptr || context_lens == nullptr || block_tables == nullptr))
    return PDA_ERR_INVALID_ARG;
  const long long per = static_cast<long long>(kSlotThreads) * kSlotPerThread;
  const long long blocks = (static_cast<long long>(N) + per - 1) / per;
  const size_t smem = static_cast<size_t>(B) * sizeof(int);
  kv_slots_kernel<<<static_cast<unsigned>(blocks > 0 ? blocks : 1), kSlotThreads, smem, stream>>>(
      slot_mapping, query_start, query_lens, context_lens, block_tables, N, B,
      max_blocks_per_seq, block_size, num_blocks, error_word);
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}
