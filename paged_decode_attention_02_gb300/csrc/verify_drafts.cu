// verify_drafts.cu -- which of each request's drafted tokens the target model keeps, and the token
// that comes after them, from given random numbers.
//
// Mathematics. Row i of a request (i = 0 .. d, d drafts) holds the target's probabilities p_i of
// the token behind its token i; draft i + 1 was drawn from q_i. With uniforms u_i, w in [0, 1):
//   accepted a = number of leading i < d with u_i q_i(x_{i+1}) < p_i(x_{i+1});
//   weights  r = max(p_a - q_a, 0) if a < d (p_a where all are zero), p_d if a = d;
//   token    = the first t with sum_{s <= t} r_s > w sum r.
// The tokens so produced are distributed as the target's own (the published accept-and-resample
// argument of speculative sampling). A draft without probabilities was certain: q = 1 at x, 0
// elsewhere.
//
// Sums. The answer is a whole number that depends on sums over the whole vocabulary, so a sum is
// kept to about 2^-46: a lane adds its eight values in 32 bits with the error of every addition
// kept (the two-sum of Knuth), everything above that in 64 bits.
//
// What bounds it: the two rows that a request draws from, read once (the accepted drafts cost a
// few loads each). A cluster of blocks shares a request's vocabulary; each keeps the sums of its
// own tiles of 256 tokens in shared memory, their totals meet over the cluster's shared memory,
// and the one warp whose tile holds the answer reads that tile again: one launch, no workspace.
#include <cooperative_groups.h>

#include <atomic>

#include "pda_device.cuh"
#include "pda_internal.h"

namespace pda {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kLaneTokens = 8;                  // consecutive tokens of a lane
constexpr int kTileTokens = 32 * kLaneTokens;   // of a warp's step
constexpr int kVerifyCluster = 8;               // blocks of a request
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxTiles = kMaxVocab / kTileTokens / kVerifyCluster;  // of a block

struct VerifyParams {
  int32_t* accepted;
  int32_t* next_tokens;
  const void* target;
  const void* draft;  // nullptr: certain drafts
  long long target_stride, draft_stride;
  const int32_t* tokens;
  const int32_t* query_start;
  const float* accept_u;
  const float* sample_u;
  int32_t* error_word;
  int T, V, tiles;  // tiles: of a block
};

template <typename E>
__device__ __forceinline__ float widen1(E v) {
  return static_cast<float>(v);
}

// Eight probabilities from token v on (zeros behind V). kWide: rows are 16-byte aligned.
template <typename E, bool kWide>
__device__ __forceinline__ void load_row(const E* row, int v, int V, float* x) {
  if (kWide && v + kLaneTokens <= V) {
    load_elems<E, kLaneTokens>(row + v, x);
    return;
  }
#pragma unroll
  for (int e = 0; e < kLaneTokens; ++e) x[e] = v + e < V ? widen1(row[v + e]) : 0.f;
}

// The weight of each of a lane's eight tokens; a weight that is no positive number counts as zero.
template <typename E, bool kWide>
__device__ __forceinline__ void weights(const E* p_row, const E* q_row, int without, int v, int V,
                                        float* r) {
  load_row<E, kWide>(p_row, v, V, r);
  if (q_row != nullptr) {
    float q[kLaneTokens];
    load_row<E, kWide>(q_row, v, V, q);
#pragma unroll
    for (int e = 0; e < kLaneTokens; ++e) r[e] -= q[e];
  }
#pragma unroll
  for (int e = 0; e < kLaneTokens; ++e) {
    if (v + e == without) r[e] = 0.f;
    r[e] = fmaxf(r[e], 0.f);  // NaN gives 0
  }
}

// The sum of eight values and what its additions lost, in 64 bits.
__device__ __forceinline__ double sum8(const float* r) {
  float s = r[0], lost = 0.f;
#pragma unroll
  for (int e = 1; e < kLaneTokens; ++e) {
    const float t = s + r[e], back = t - s;
    lost += (s - (t - back)) + (r[e] - back);
    s = t;
  }
  return static_cast<double>(s) + static_cast<double>(lost);
}

template <typename E, bool kWide>
__global__ void __cluster_dims__(kVerifyCluster, 1, 1) __launch_bounds__(kVerifyThreads)
    verify_kernel(const VerifyParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ double tile_sum[kMaxTiles];
  __shared__ double total[2][kVerifyCluster];  // of each block of the cluster, in each pass
  __shared__ int first_rejected;
  const int rank = static_cast<int>(cluster.block_rank());
  const int b = static_cast<int>(blockIdx.x) / kVerifyCluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  const int q0 = p.query_start[b], q1 = p.query_start[b + 1];
  const bool in_range = q0 >= 0 && q1 <= p.T && q0 <= q1;
  if (!in_range || q0 == q1) {  // all of the cluster's blocks leave here
    if (rank == 0 && tid == 0) {
      p.accepted[b] = 0;
      p.next_tokens[b] = -1;
      if (!in_range) atomic_or_error(p.error_word, PDA_DEVERR_QUERY);
    }
    return;
  }
  const int drafts = q1 - q0 - 1;
  // the others' shared memory exists once they have arrived here (waited for below)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  // ---- the drafts: a thread each, the first that is turned down wins
  if (tid == 0) first_rejected = drafts;
  __syncthreads();
  bool bad_token = false;
  for (int i = tid; i < drafts; i += kVerifyThreads) {
    const int x = p.tokens[q0 + i + 1];
    bool ok = false;
    if (x < 0 || x >= p.V) {
      bad_token = true;
    } else {
      const size_t row = static_cast<size_t>(q0) + i;
      const float pt = widen1(static_cast<const E*>(p.target)[row * p.target_stride + x]);
      const float qt = p.draft != nullptr
                           ? widen1(static_cast<const E*>(p.draft)[row * p.draft_stride + x])
                           : 1.f;
      ok = p.accept_u[row] * qt < pt;
    }
    if (!ok) {
      atomicMin(&first_rejected, i);
      break;  // this thread's later drafts come behind it
    }
  }
  __syncthreads();
  const int a = first_rejected;
  const size_t row = static_cast<size_t>(q0) + a;
  const E* p_row = static_cast<const E*>(p.target) + row * p.target_stride;
  const int rejected = a < drafts ? p.tokens[q0 + a + 1] : -1;
  if (bad_token && rank == 0) atomic_or_error(p.error_word, PDA_DEVERR_TOKEN);

  // ---- the weights' sums; once more over p alone where nothing is left of p - q
  const int tile0 = rank * p.tiles;
  int pass = 0;
  const E* q_row = nullptr;
  int without = -1;
  double all = 0.0, before = 0.0;
  for (;; ++pass) {
    const bool rest = pass == 0 && a < drafts;
    q_row = rest && p.draft != nullptr
                ? static_cast<const E*>(p.draft) + row * p.draft_stride
                : nullptr;
    without = rest && p.draft == nullptr ? rejected : -1;
    for (int t = warp; t < p.tiles; t += kVerifyWarps) {
      const int v = (tile0 + t) * kTileTokens + lane * kLaneTokens;
      float r[kLaneTokens];
      weights<E, kWide>(p_row, q_row, without, v, p.V, r);
      double s = sum8(r);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
      if (lane == 0) tile_sum[t] = s;
    }
    __syncthreads();
    if (pass == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (warp == 0) {
      double s = 0.0;
      for (int t = lane; t < p.tiles; t += 32) s += tile_sum[t];
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
      if (lane < kVerifyCluster) *cluster.map_shared_rank(&total[pass][rank], lane) = s;
    }
    cluster.sync();
    all = before = 0.0;
    for (int k = 0; k < kVerifyCluster; ++k) {
      if (k == rank) before = all;
      all += total[pass][k];
    }
    if (all > 0.0 || !rest) break;  // the second pass is never `rest`
  }
  if (rank == 0 && tid == 0) {
    p.accepted[b] = a;
    if (!(all > 0.0 && isfinite(all))) {
      p.next_tokens[b] = -1;
      atomic_or_error(p.error_word, PDA_DEVERR_PROBS);
    }
  }
  if (!(all > 0.0 && isfinite(all))) return;
  // ---- the block, the tile and the lane that the answer lies in
  const double u = fmin(fmax(static_cast<double>(p.sample_u[b]), 0.0), 1.0);
  double goal = u * all;
  // u = 1, or sums in another order: the last token with a weight
  int last_block = 0;
  {
    double run = 0.0;
    int found = -1;
    for (int k = 0; k < kVerifyCluster; ++k) {
      const double s = total[pass][k];
      if (s > 0.0) last_block = k;
      run += s;
      if (found < 0 && run > goal) found = k;
    }
    const bool none = found < 0;
    if (none) found = last_block;
    if (found != rank || warp != 0) return;
    goal = none ? INFINITY : goal - before;
  }
  double run = 0.0;
  int tile = -1, last_tile = 0;
  double tile_goal = INFINITY;
  for (int t0 = 0; t0 < p.tiles && tile < 0; t0 += 32) {
    const double s = t0 + lane < p.tiles ? tile_sum[t0 + lane] : 0.0;
    double end = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(kFullMask, end, o);
      if (lane >= o) end += y;
    }
    const unsigned over = __ballot_sync(kFullMask, run + end > goal);
    const unsigned some = __ballot_sync(kFullMask, s > 0.0);
    if (over != 0) {
      const int l = __ffs(over) - 1;
      tile = t0 + l;
      tile_goal = goal - (run + __shfl_sync(kFullMask, end - s, l));
    } else if (some != 0) {
      last_tile = t0 + 31 - __clz(some);
    }
    run += __shfl_sync(kFullMask, end, 31);
  }
  if (tile < 0) tile = last_tile;
  const int v = (tile0 + tile) * kTileTokens + lane * kLaneTokens;
  float r[kLaneTokens];
  weights<E, kWide>(p_row, q_row, without, v, p.V, r);
  const double s = sum8(r);
  double end = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(kFullMask, end, o);
    if (lane >= o) end += y;
  }
  // this lane's first token past the goal, and its last with a weight
  double at = end - s;
  int hit = -1, last = -1;
#pragma unroll
  for (int e = 0; e < kLaneTokens; ++e) {
    at += static_cast<double>(r[e]);
    if (r[e] > 0.f) {
      last = v + e;
      if (hit < 0 && at > tile_goal) hit = v + e;
    }
  }
  const unsigned hits = __ballot_sync(kFullMask, hit >= 0);
  const unsigned lasts = __ballot_sync(kFullMask, last >= 0);
  const int from = hits != 0 ? __ffs(hits) - 1 : lasts != 0 ? 31 - __clz(lasts) : 0;
  const int token = __shfl_sync(kFullMask, hits != 0 ? hit : last, from);
  if (lane == 0) p.next_tokens[b] = token;
}

template <typename E>
void launch_verify(const VerifyParams& p, int B, bool wide, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(B) * kVerifyCluster);
  if (wide)
    verify_kernel<E, true><<<grid, kVerifyThreads, 0, stream>>>(p);
  else
    verify_kernel<E, false><<<grid, kVerifyThreads, 0, stream>>>(p);
}

}  // namespace
}  // namespace pda

using namespace pda;

extern "C" pda_status pda_verify_drafts(int32_t* accepted, int32_t* next_tokens,
                                        const void* target_probs, const void* draft_probs,
                                        long long target_stride, long long draft_stride,
                                        const int32_t* tokens, const int32_t* query_start,
                                        const float* accept_u, const float* sample_u, int T, int B,
                                        int V, pda_dtype dtype, int32_t* error_word,
                                        cudaStream_t stream) {
  if (T < 0 || B < 0 || V <= 0 || !float_dtype_ok(dtype) || target_stride < V ||
      (draft_probs != nullptr && draft_stride < V))
    return PDA_ERR_INVALID_ARG;
  if (V > kMaxVocab || B > 8192) return PDA_ERR_UNSUPPORTED;
  if (B == 0) return PDA_OK;
  if (accepted == nullptr || next_tokens == nullptr || query_start == nullptr ||
      sample_u == nullptr ||
      (T > 0 && (target_probs == nullptr || tokens == nullptr || accept_u == nullptr)))
    return PDA_ERR_INVALID_ARG;
  const int e = static_cast<int>(dtype_bytes(dtype));
  auto whole = [&](const void* x) { return (reinterpret_cast<uintptr_t>(x) % e) == 0; };
  if (!whole(target_probs) || !whole(draft_probs)) return PDA_ERR_INVALID_ARG;
  const bool wide = aligned16(target_probs) && aligned16(draft_probs) &&
                    target_stride * e % 16 == 0 &&
                    (draft_probs == nullptr || draft_stride * e % 16 == 0);
  const int tiles = (V + kTileTokens - 1) / kTileTokens;
  const VerifyParams p{accepted, next_tokens, target_probs, draft_probs, target_stride,
                       draft_stride, tokens, query_start, accept_u, sample_u, error_word, T, V,
                       (tiles + kVerifyCluster - 1) / kVerifyCluster};
  if (dtype == PDA_F32)
    launch_verify<float>(p, B, wide, stream);
  else if (dtype == PDA_BF16)
    launch_verify<__nv_bfloat16>(p, B, wide, stream);
  else
    launch_verify<__half>(p, B, wide, stream);
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}
