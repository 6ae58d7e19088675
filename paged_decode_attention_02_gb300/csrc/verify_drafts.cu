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
// kept to about 2^-44, as a 32-bit value and what its additions lost (the two-sum of Knuth). An SM
// does two 64-bit additions a cycle, each a long wait for the next: sums of that type took 36 us
// for 64 requests of 131072 tokens.
//
// What bounds it: the two rows that a request draws from, read once (the accepted drafts cost a
// few loads each), after a chain of three loads that finds them. A cluster of blocks shares a
// request's vocabulary; each keeps the sums of its own tiles in shared memory, their totals meet
// over the cluster's shared memory, and the one warp whose tile holds the answer reads that tile
// again: one launch, no workspace. 64 requests of 131072 tokens in fp32 take 18 us (the stream 10,
// the loads before it 2, the search behind it 3), one of 32000 in bf16 5.7 us.
#include <cooperative_groups.h>

#include <atomic>

#include "pda_device.cuh"
#include "pda_internal.h"

namespace pda {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kLaneTokens = 8;                  // consecutive tokens of a lane
constexpr int kStepTokens = 32 * kLaneTokens;   // of a warp's step; a tile is 1, 2 or 4 of them
constexpr int kVerifyCluster = 8;               // blocks of a request
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxTiles = kMaxVocab / kStepTokens / kVerifyCluster;  // of a block

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

// Eight probabilities, of tokens v, v + kApart, ... (zeros behind V). kWide: rows are 16-byte
// aligned.
template <typename E, bool kWide, int kApart>
__device__ __forceinline__ void load_row(const E* row, int v, int V, float* x) {
  if (kWide && kApart == 1 && v + kLaneTokens <= V) {
    load_elems<E, kLaneTokens>(row + v, x);
    return;
  }
#pragma unroll
  for (int e = 0; e < kLaneTokens; ++e)
    x[e] = v + e * kApart < V ? widen1(row[v + e * kApart]) : 0.f;
}

// The weights of a lane's eight tokens; one that is no positive number counts as zero.
template <typename E, bool kWide, int kApart>
__device__ __forceinline__ void weights(const E* p_row, const E* q_row, int without, int v, int V,
                                        float* r) {
  load_row<E, kWide, kApart>(p_row, v, V, r);
  if (q_row != nullptr) {
    float q[kLaneTokens];
    load_row<E, kWide, kApart>(q_row, v, V, q);
#pragma unroll
    for (int e = 0; e < kLaneTokens; ++e) r[e] -= q[e];
  }
#pragma unroll
  for (int e = 0; e < kLaneTokens; ++e) {
    if (v + e * kApart == without) r[e] = 0.f;
    r[e] = fmaxf(r[e], 0.f);  // NaN gives 0
  }
}

// A sum and what its additions lost.
struct Sum {
  float s, lost;
  __device__ __forceinline__ void add(float x) {
    const float t = s + x, back = t - s;
    lost += (s - (t - back)) + (x - back);
    s = t;
  }
  __device__ __forceinline__ void add(Sum o) {
    lost += o.lost;
    add(o.s);
  }
  __device__ __forceinline__ Sum minus(Sum o) const {
    Sum d = *this;
    d.add(Sum{-o.s, -o.lost});
    return d;
  }
  __device__ __forceinline__ bool above(Sum o) const { return (s - o.s) + (lost - o.lost) > 0.f; }
  __device__ __forceinline__ bool positive() const { return s + lost > 0.f; }
};

// The sum of eight values, in two chains.
__device__ __forceinline__ Sum sum8(const float* r) {
  Sum a{r[0], 0.f}, b{r[1], 0.f};
#pragma unroll
  for (int e = 2; e < kLaneTokens; e += 2) {
    a.add(r[e]);
    b.add(r[e + 1]);
  }
  a.add(b);
  return a;
}

__device__ __forceinline__ Sum from_lane(Sum x, int lane) {
  return Sum{__shfl_sync(kFullMask, x.s, lane), __shfl_sync(kFullMask, x.lost, lane)};
}

// On every lane, the sum over the lanes.
__device__ __forceinline__ Sum over_lanes(Sum x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1)
    x.add(Sum{__shfl_xor_sync(kFullMask, x.s, o), __shfl_xor_sync(kFullMask, x.lost, o)});
  return x;
}

// The sum over this lane and those below.
__device__ __forceinline__ Sum up_to_lane(Sum x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sum y{__shfl_up_sync(kFullMask, x.s, o), __shfl_up_sync(kFullMask, x.lost, o)};
    if (lane >= o) x.add(y);
  }
  return x;
}

// Lanes hold consecutive stretches of sum x. Finds the first past `goal` (else the last positive
// one; -1: there is none) and takes what lies before it off the goal.
struct Found {
  int lane;
  bool past;
};
__device__ __forceinline__ Found find(Sum x, Sum* goal) {
  const Sum end = up_to_lane(x);
  const unsigned over = __ballot_sync(kFullMask, x.positive() && end.above(*goal));
  const unsigned some = __ballot_sync(kFullMask, x.positive());
  const int lane = over != 0 ? __ffs(over) - 1 : 31 - __clz(some);
  const Sum before = from_lane(end, lane > 0 ? lane - 1 : 0);
  if (lane > 0) *goal = goal->minus(before);
  return Found{lane, over != 0};
}

template <typename E, bool kWide, int kSteps>
__global__ void __cluster_dims__(kVerifyCluster, 1, 1) __launch_bounds__(kVerifyThreads, 4)
    verify_kernel(const VerifyParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ Sum tile_sum[kMaxTiles];
  __shared__ Sum total[2][kVerifyCluster];  // of each block of the cluster, in each pass
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
  Sum mine, all;  // lane k: block k's total; every lane: the cluster's
  for (;; ++pass) {
    const bool rest = pass == 0 && a < drafts;
    q_row = rest && p.draft != nullptr
                ? static_cast<const E*>(p.draft) + row * p.draft_stride
                : nullptr;
    without = rest && p.draft == nullptr ? rejected : -1;
    // rows of odd alignment are read a token a lane
    constexpr int kApart = kWide ? 1 : 32;
    for (int t = warp; t < p.tiles; t += kVerifyWarps) {
      Sum sum{0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int v = ((tile0 + t) * kSteps + k) * kStepTokens + lane * (kWide ? kLaneTokens : 1);
        float r[kLaneTokens];
        weights<E, kWide, kApart>(p_row, q_row, without, v, p.V, r);
        sum.add(sum8(r));
      }
      sum = over_lanes(sum);
      if (lane == 0) tile_sum[t] = sum;
    }
    __syncthreads();
    if (pass == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (warp == 0) {
      Sum s{0.f, 0.f};
      for (int t = lane; t < p.tiles; t += 32) s.add(tile_sum[t]);
      s = over_lanes(s);
      if (lane < kVerifyCluster) *cluster.map_shared_rank(&total[pass][rank], lane) = s;
    }
    cluster.sync();
    mine = lane < kVerifyCluster ? total[pass][lane] : Sum{0.f, 0.f};
    all = over_lanes(mine);
    if (all.positive() || !rest) break;  // the second pass is never `rest`
  }
  if (warp != 0) return;

  const bool usable = all.positive() && isfinite(all.s) && isfinite(all.lost);
  if (rank == 0 && lane == 0) {
    p.accepted[b] = a;
    if (!usable) {
      p.next_tokens[b] = -1;
      atomic_or_error(p.error_word, PDA_DEVERR_PROBS);
    }
  }
  if (!usable) return;
  // ---- the block, the tile, the step and the lane that the answer lies in; where sums in another
  // order leave none past the goal (or u = 1), the last with a weight
  const float u = fminf(fmaxf(p.sample_u[b], 0.f), 1.f);
  Sum goal{u * all.s, 0.f};
  goal.lost = fmaf(u, all.s, -goal.s) + u * all.lost;
  const Found block = find(mine, &goal);
  if (block.lane != rank) return;
  bool past = block.past;
  if (!past) goal.s = INFINITY;
  int tile = -1;
  for (int t0 = 0; t0 < p.tiles; t0 += 32) {
    const Sum s = t0 + lane < p.tiles ? tile_sum[t0 + lane] : Sum{0.f, 0.f};
    Sum left = goal;
    const Found f = find(s, &left);
    if (f.lane >= 0) tile = t0 + f.lane;
    if (f.past) {
      goal = left;
      break;
    }
    past = past && t0 + 32 < p.tiles;
    goal = goal.minus(over_lanes(s));
  }
  if (!past) goal.s = INFINITY;
  float r[kSteps][kLaneTokens];
  Sum step[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k)
    weights<E, kWide, 1>(p_row, q_row, without,
                         ((tile0 + tile) * kSteps + k) * kStepTokens + lane * kLaneTokens, p.V,
                         r[k]);
#pragma unroll
  for (int k = 0; k < kSteps; ++k) step[k] = sum8(r[k]);
  int at = 0;  // the step
  if (kSteps > 1) {
    Sum whole{0.f, 0.f};  // lane k: step k's
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const Sum s = over_lanes(step[k]);
      if (lane == k) whole = s;
    }
    const Found f = find(whole, &goal);
    at = f.lane;
    if (!f.past) goal.s = INFINITY;
  }
#pragma unroll
  for (int k = 1; k < kSteps; ++k)
    if (k == at) {
      step[0] = step[k];
#pragma unroll
      for (int e = 0; e < kLaneTokens; ++e) r[0][e] = r[k][e];
    }
  const Found f = find(step[0], &goal);
  if (!f.past) goal.s = INFINITY;
  if (lane != f.lane) return;
  Sum end{0.f, 0.f};
  int hit = -1, last = 0;
#pragma unroll
  for (int e = 0; e < kLaneTokens; ++e) {
    end.add(r[0][e]);
    if (r[0][e] > 0.f) {
      last = e;
      if (hit < 0 && end.above(goal)) hit = e;
    }
  }
  p.next_tokens[b] = ((tile0 + tile) * kSteps + at) * kStepTokens + lane * kLaneTokens +
                     (hit >= 0 ? hit : last);
}

template <typename E, bool kWide>
void launch_steps(VerifyParams p, int B, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(B) * kVerifyCluster);
  const int steps = (p.V + kStepTokens - 1) / kStepTokens;
  auto tiles = [&](int of) {
    return ((steps + of - 1) / of + kVerifyCluster - 1) / kVerifyCluster;
  };
  // the longest tile that still gives every warp of the cluster one: a tile's sum over the lanes
  // costs about as much as a step of it
  if (steps >= 4 * kVerifyCluster * kVerifyWarps) {
    p.tiles = tiles(4);
    verify_kernel<E, kWide, 4><<<grid, kVerifyThreads, 0, stream>>>(p);
  } else if (steps >= kVerifyCluster * kVerifyWarps) {
    p.tiles = tiles(2);
    verify_kernel<E, kWide, 2><<<grid, kVerifyThreads, 0, stream>>>(p);
  } else {
    p.tiles = tiles(1);
    verify_kernel<E, kWide, 1><<<grid, kVerifyThreads, 0, stream>>>(p);
  }
}

template <typename E>
void launch_verify(const VerifyParams& p, int B, bool wide, cudaStream_t stream) {
  if (wide)
    launch_steps<E, true>(p, B, stream);
  else
    launch_steps<E, false>(p, B, stream);
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
  const VerifyParams p{accepted, next_tokens, target_probs, draft_probs, target_stride,
                       draft_stride, tokens, query_start, accept_u, sample_u, error_word, T, V, 0};
  if (dtype == PDA_F32)
    launch_verify<float>(p, B, wide, stream);
  else if (dtype == PDA_BF16)
    launch_verify<__nv_bfloat16>(p, B, wide, stream);
  else
    launch_verify<__half>(p, B, wide, stream);
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}
