// decode_kernel.cuh -- the kernel of batched single-query attention over a paged KV cache, sm_103a
// (launched by decode_attention.cu).
//
// What it computes: for each request b and query head h (kv-head k = h / G, G = H / H_kv),
//   out[b,h] = sum_t softmax_t(scale * q[b,h] . K_t[k]) V_t[k],  t < context_lens[b],
// with token t in physical block block_tables[b][t / 16], row t % 16. Decode reads the
// whole cached history each step (page "Disaggregated LLM Serving: from PD disaggregation
// to attention offload", sec. 1 and sec. 6.1); the history is paged (page "From
// PagedAttention to Prefill-Decode disaggregation", sec. 2.2).
//
// How (GB300 design):
//  * Unit of work = one tile = one physical block (16 tokens) of one kv-head: 16 rows of
//    D elements for K and for V. Tiles are numbered request-major, then kv-head, then
//    block, so the tiles of one (request, kv-head) "segment" are consecutive.
//  * The total tile count is split evenly over all warps of a persistent grid (one block
//    per SM, at most sm_cap SMs). Each warp is an independent worker: it streams its tile
//    range through its own ring of shared-memory stages filled by TMA (3-D tiled
//    cp.async.bulk.tensor for the K and V rows, a 1-D bulk copy for the segment's q rows),
//    each stage guarded by an mbarrier. There is no block-wide synchronisation in the loop.
//  * The G query heads that share a kv-head are processed together, so each K/V byte is
//    read from HBM once (GQA).
//  * Scores use fp32 FMAs; the partial dot products of a lane group are summed with a
//    shuffle reduce-scatter, which leaves each lane owning a few complete (head, token)
//    scores. Softmax is online, in base 2 (q is pre-scaled by scale * log2 e).
//  * A segment that lies wholly inside one worker's range is normalised and written
//    directly. A segment cut by a range boundary leaves (m, l, o) pieces in the workspace
//    (at most two per worker); the warp that registers a segment's last piece merges them
//    with a log-sum-exp combine, so no second kernel is needed. This is the split and merge
//    of Orca's iteration-level batching (page "Disaggregated LLM Serving", sec. 2.1),
//    applied along the sequence.
//  * bf16 and fp32 caches run on the CUDA cores: per kv-head and token this is G dot
//    products of length D against 2 * D * sizeof(elem) bytes, and the bf16 path already
//    streams at the HBM rate. Quantised caches (FP8, NVFP4) at D = 128 carry two to four
//    times as many tokens per byte, so their dot products go to the tensor cores
//    (warp_attn_tc.cuh), mostly on units of two adjacent kv-heads (one TMA box for both);
//    the pipeline, scheduling and merge below are shared and see a pair as one unit with
//    2 G query heads.
//  * With a sliding window (kWindow), a request's tiles are those of its first `sinks` tokens
//    and, behind them, those that hold its last `window` tokens: tile blk of a segment is block
//    blk, or blk + skip from the window on. Everything but that step, and the mask of rows of
//    the tiles at the borders, works on these tiles as on a shorter history; blocks between are
//    neither read nor looked up. So the work, and the time, is that of a history of
//    sinks + window tokens: 256 requests over 4096 + 4 keys of 8 kv-heads in bf16 take 622 us
//    (6.5 TB/s, 97 % of the copy rate).
#pragma once

#include <math.h>

#include <type_traits>

#include "pda_device.cuh"
#include "pda_internal.h"
#include "warp_attn_tc.cuh"
#include "work_units.h"

namespace pda {

#ifndef PDA_ATTN_WARPS
#define PDA_ATTN_WARPS 12     // preferred warps (workers) per block
#endif
#ifndef PDA_ATTN_MAX_STAGES
#define PDA_ATTN_MAX_STAGES 4  // most pipeline stages per warp
#endif

// A launch uses no more warps than give each at least this many tiles. With fewer, a small
// batch spreads over thousands of warps and every (request, kv-head) segment is cut into
// dozens of pieces for its merge to read back: one 13B-shape request ran 51 us over 1824
// warps and 31 us at 8 tiles per warp (4 and 16 measured slower).
#ifndef PDA_MIN_TILES_PER_WARP
#define PDA_MIN_TILES_PER_WARP 8
#endif

// With a window, whose launches are short, a warp takes as few as two tiles, and more where a
// segment has many: with T tiles over n warps, the tiles take T / n and the merge n, so n follows
// sqrt(T). 16 requests of 16/2 heads of 64 in bf16: 128 keys 17 us at two tiles and 19 at four,
// 1024 keys 25 and 23, 4096 keys (one request) 46 and 31.
constexpr int kWindowMinTiles = 2;
__device__ __forceinline__ int window_tiles_per_warp(int tiles, int segments) {
  const float mean = static_cast<float>(tiles) / static_cast<float>(max(segments, 1));
  return max(kWindowMinTiles, static_cast<int>(sqrtf(mean) * 0.25f));
}

#ifndef PDA_TC_WARPS
#define PDA_TC_WARPS 12        // warps (workers) per block of the tensor-core tile step
#endif

constexpr int kBS = 16;             // tokens per physical block (box height of the TMA)
constexpr int kMaxWarps = PDA_ATTN_WARPS > PDA_TC_WARPS ? PDA_ATTN_WARPS : PDA_TC_WARPS;
// Warps per block for a GQA group of G: on the CUDA cores the group of 8 keeps 8 warps so
// its 8 heads of q and o stay in registers (up to 255 per thread); the tensor-core tile
// step holds q and o in mma fragments and keeps all warps.
__host__ __device__ constexpr int warps_for_group(int G, bool tc) {
  return tc ? PDA_TC_WARPS : (G >= 8 ? 8 : PDA_ATTN_WARPS);
}
// The two-head tensor-core step holds both heads' q fragments and running state (about 230
// registers). A scheduler's register file (16K) holds three warps only below 171 registers
// each. FP8 runs it with 8 warps (two per scheduler, no spills); NVFP4, whose longer
// dequantisation chains need more warps to hide, with 12 and a few spilled registers
// (measured 9-10 % faster for NVFP4 and 2 % slower for FP8 than the other choice).
#ifndef PDA_TC_PAIR_WARPS_FP8
#define PDA_TC_PAIR_WARPS_FP8 8
#endif
#ifndef PDA_TC_PAIR_WARPS_NVFP4
#define PDA_TC_PAIR_WARPS_NVFP4 12
#endif
static_assert(PDA_TC_PAIR_WARPS_FP8 <= kMaxWarps && PDA_TC_PAIR_WARPS_NVFP4 <= kMaxWarps,
              "per-warp shared arrays are sized for kMaxWarps");
__host__ __device__ constexpr int warps_for_mode(int G, int mode, bool fp4) {
  return mode == 2 ? (fp4 ? PDA_TC_PAIR_WARPS_NVFP4 : PDA_TC_PAIR_WARPS_FP8)
                   : warps_for_group(G, mode != 0);
}
// Stage alignment: the tensor-core step reads TMA tiles written with the 128-byte (FP8) or
// 64-byte (NVFP4) swizzle, whose pattern repeats every 1024 (512) bytes.
__host__ __device__ constexpr int stage_align(bool tc) { return tc ? 1024 : 128; }

// Tile steps (see attn_partial_kernel).
constexpr int kModeCuda = 0;
constexpr int kModeTc = 1;
constexpr int kModeTcPair = 2;
// What the lane that issues a tile leaves for the warp: which rows count, and whether the block's
// id was out of range.
constexpr int kBadTile = 0x10000;
constexpr int kMetaBytesPerWarp = 2 * 32 * 8;  // two groups of 32 (block id, length) pairs
constexpr int kMaxBatch = 8192;     // prefix table size bound (shared memory)
constexpr int kSmemBudget = 226 * 1024;  // dynamic bytes; static shared memory sits on top
constexpr int kMinResidentSmem = 116 * 1024;  // > half an SM: never two blocks per SM

struct AttnParams {
  void* out;
  const void* q;
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* ws_o;                    // [2 * units][G][D]   piece outputs (two slots per unit)
  float* ws_ml;                   // [2 * units][G][2]   piece (max, sum)
  unsigned long long* ws_arrive;  // [B * H_kv] piece arrivals (tagged counters, see arrive)
  unsigned long long* ws_claim;   // pool chunks claimed so far (tagged counter)
  unsigned long long call;        // this call's number (48 bits)
  int pool_k;                     // most pool chunks per warp the workspace holds pieces for
  int32_t* error_word;
  float v_scale;                  // value of a stored V element = code * v_scale (1 if plain)
  const uint8_t* k_bscales;       // NVFP4: [blocks, H_kv, 16, D/16] E4M3 block scales
  const uint8_t* v_bscales;
  int B, H, H_kv, num_blocks, max_blocks, max_context_len;
  int window, sinks;              // kWindow: the last `window` tokens and the first `sinks`
  int block_size;                 // tokens per physical block: 16 << bs_shift
  int bs_shift;                   // log2 of the 16-row tiles per physical block
  int out_kind;                   // output type: 0 fp32, 1 bf16, 2 fp16
  float scale_log2;
  int num_workers;
  int stages;
  uint32_t stage_bytes;   // one stage: K tile, V tile, q slot
  uint32_t prefix_bytes;  // shared bytes reserved for the prefix table
};

// Reduce-scatter over the lanes of one row group: n values per lane, xor masks from
// `mask` down to 1. While n > 1 every lane keeps the lower half of its values and adds the
// partner's upper half; once one value is left the remaining steps are plain butterflies.
// This leaves each lane with complete sums only because every lane stores its values in a
// lane-dependent order (see WarpAttn::init): local index u holds real index u ^ idx0, so a
// lane's lower half is exactly the half its partner sends it.
template <int n, int mask>
struct ReduceScatter {
  static __device__ __forceinline__ void run(float* v) {
    if constexpr (mask == 0) {
      return;
    } else if constexpr (n > 1) {
#pragma unroll
      for (int i = 0; i < n / 2; ++i) v[i] += __shfl_xor_sync(kFullMask, v[i + n / 2], mask);
      ReduceScatter<n / 2, mask / 2>::run(v);
    } else {
      v[0] += __shfl_xor_sync(kFullMask, v[0], mask);
      ReduceScatter<1, mask / 2>::run(v);
    }
  }
};

template <typename KV, typename QT, int D, int G>
struct Geometry {
  using E = Elem<KV>;
  static constexpr int VEC = E::kVec;               // elements per lane per row (16 bytes)
  static constexpr int LPR = D / VEC;               // lanes covering one row
  static constexpr int RPW = 32 / LPR;              // rows a warp covers per step
  static constexpr int TPL = kBS / RPW;             // token slots per lane per tile
  static constexpr int N = G * TPL;                 // partial dots per lane per tile
  static constexpr int C = N >= LPR ? N / LPR : 1;  // complete scores per lane
  static constexpr int DUP = N >= LPR ? 1 : LPR / N;  // lanes holding the same score
  static constexpr int LPH = N >= LPR ? LPR / G : LPR;  // lanes of a row group per head
  // Scores of two token slots share one packed fp32x2 FMA when q fits twice in registers.
  static constexpr bool PAIR_QK = G * VEC <= 32 && TPL % 2 == 0;
  // NVFP4: every row of a tile comes with one E4M3 scale per 16 elements
  static constexpr bool SCALED = std::is_same<KV, nvfp4>::value;
  static constexpr int ROW_SCALES = D / 16;  // scale bytes per row (NVFP4)
  static constexpr uint32_t TILE_BYTES = kBS * D * E::kBits / 8;
  static constexpr uint32_t SCALE_BYTES = SCALED ? kBS * ROW_SCALES : 0;  // per K or V tile
  static constexpr uint32_t Q_BYTES = G * D * sizeof(QT);
  static_assert(32 % LPR == 0 && kBS % RPW == 0, "row geometry");
  static_assert(LPR >= G, "one head per lane after the reduce-scatter");
  static_assert(VEC % 2 == 0, "packed fp32x2 accumulation");
  static_assert(TILE_BYTES % 128 == 0 && Q_BYTES % 16 == 0, "smem alignment");
  static_assert(!SCALED || (VEC <= 16 && 16 % VEC == 0), "a lane's dims share one scale");
};

// Per-warp online-softmax state and tile arithmetic.
//
// Lane layout: lane = rw * LPR + cl; the lane covers dims [cl*VEC, cl*VEC + VEC) of the
// rows rw, rw + RPW, ... (token slot i is row rw + RPW * i of the 16-row tile). Each lane
// forms N = G * TPL partial dot products (head j, slot i; real index j * TPL + i), sums
// them with the other lanes of its row group by a reduce-scatter, and is left with C
// complete scores of one head: real indices idx0 .. idx0 + C - 1.
template <typename KV, typename QT, int D, int G>
struct WarpAttn {
  using Geo = Geometry<KV, QT, D, G>;
  using E = typename Geo::E;
  static constexpr int VEC = Geo::VEC, LPR = Geo::LPR, RPW = Geo::RPW, TPL = Geo::TPL;
  static constexpr int N = Geo::N, C = Geo::C, DUP = Geo::DUP, LPH = Geo::LPH;
  static constexpr bool PAIR_QK = Geo::PAIR_QK;
  static constexpr bool SCALED = Geo::SCALED;
  static constexpr int ROW_SCALES = Geo::ROW_SCALES;

  int lane, rw, cl, idx0;
  int sblk;                      // NVFP4: index of this lane's 16-element block in a row
  int srow[SCALED ? TPL : 1];    // NVFP4: scale offset of the K row behind local slot il
  int hp;             // local head jl holds real head jl ^ hp
  int krow[TPL];      // element offset of the K row behind local slot il (real slot il ^ tp)
  float2 q2[PAIR_QK ? G : 1][PAIR_QK ? VEC : 1];  // q (scaled), duplicated, local head order
  float qs[PAIR_QK ? 1 : G][PAIR_QK ? 1 : VEC];   // q (scaled), local head order
  float2 o2[G][VEC / 2];  // unnormalised output, real head order, dims pairs
  float m_own;  // running max of this lane's head (log2 domain)
  float l_own;  // this lane's share of the running sum of its head

  __device__ __forceinline__ void init(int lane_) {
    lane = lane_;
    rw = lane / LPR;
    cl = lane % LPR;
    idx0 = (cl / DUP) * C;
    hp = idx0 / TPL;
    const int tp = idx0 % TPL;
#pragma unroll
    for (int il = 0; il < TPL; ++il) krow[il] = (rw + RPW * (il ^ tp)) * D + cl * VEC;
    sblk = (cl * VEC) / 16;
    if constexpr (SCALED) {
#pragma unroll
      for (int il = 0; il < TPL; ++il) srow[il] = (rw + RPW * (il ^ tp)) * ROW_SCALES + sblk;
    }
  }

  __device__ __forceinline__ void reset(const QT* q_smem, float scale_log2) {
#pragma unroll
    for (int jl = 0; jl < G; ++jl) {
      float t[VEC];
      load_elems<QT, VEC>(q_smem + (jl ^ hp) * D + cl * VEC, t);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float qv = t[e] * scale_log2;
        if constexpr (PAIR_QK)
          q2[jl][e] = make_float2(qv, qv);
        else
          qs[jl][e] = qv;
      }
    }
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) o2[j][e] = make_float2(0.f, 0.f);
    m_own = -INFINITY;
    l_own = 0.f;
  }

  // ksc/vsc: the tile's NVFP4 block scales ([16 rows][D/16] E4M3 bytes), unused otherwise.
  // valid(t): row t of the tile counts (asked where kPartial).
  template <bool kPartial, typename Valid>
  __device__ __forceinline__ void tile(const KV* ks, const KV* vs, const uint8_t* ksc,
                                       const uint8_t* vsc, Valid valid) {
    // ---- scores: part[jl * TPL + il] = q(real head jl ^ hp) . K(real slot il ^ tp)
    float part[N];
    if constexpr (PAIR_QK) {
#pragma unroll
      for (int m = 0; m < TPL / 2; ++m) {
        float k0[VEC], k1[VEC];
        E::load(elem_ptr<KV>(ks, krow[2 * m]), k0);
        E::load(elem_ptr<KV>(ks, krow[2 * m + 1]), k1);
        float2 sk = make_float2(1.f, 1.f);
        if constexpr (SCALED)
          sk = make_float2(e4m3_to_f32(ksc[srow[2 * m]]), e4m3_to_f32(ksc[srow[2 * m + 1]]));
#pragma unroll
        for (int jl = 0; jl < G; ++jl) {
          float2 acc = __fmul2_rn(q2[jl][0], make_float2(k0[0], k1[0]));
#pragma unroll
          for (int e = 1; e < VEC; ++e)
            acc = __ffma2_rn(q2[jl][e], make_float2(k0[e], k1[e]), acc);
          if constexpr (SCALED) acc = __fmul2_rn(acc, sk);
          part[jl * TPL + 2 * m] = acc.x;
          part[jl * TPL + 2 * m + 1] = acc.y;
        }
      }
    } else {
#pragma unroll
      for (int il = 0; il < TPL; ++il) {
        float k[VEC];
        E::load(elem_ptr<KV>(ks, krow[il]), k);
        float sk = 1.f;
        if constexpr (SCALED) sk = e4m3_to_f32(ksc[srow[il]]);
#pragma unroll
        for (int jl = 0; jl < G; ++jl) {
          float acc = qs[jl][0] * k[0];
#pragma unroll
          for (int e = 1; e < VEC; ++e) acc = fmaf(qs[jl][e], k[e], acc);
          part[jl * TPL + il] = SCALED ? acc * sk : acc;
        }
      }
    }
    ReduceScatter<N, LPR / 2>::run(part);

    // part[0..C) are now complete scores of real index idx0 + r: head (idx0 + r) / TPL,
    // slot (idx0 + r) % TPL.
    float tmax = -INFINITY;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      if (kPartial) {
        const int t = rw + RPW * ((idx0 + r) % TPL);
        if (!valid(t)) part[r] = -INFINITY;
      }
      tmax = fmaxf(tmax, part[r]);
    }
    // lanes cl and cl ^ m for m < DUP hold the same scores, so the max skips those masks
#pragma unroll
    for (int mask = LPH / 2; mask >= DUP; mask >>= 1)
      tmax = fmaxf(tmax, __shfl_xor_sync(kFullMask, tmax, mask));
#pragma unroll
    for (int mask = LPR; mask < 32; mask <<= 1)
      tmax = fmaxf(tmax, __shfl_xor_sync(kFullMask, tmax, mask));

    const float m_new = fmaxf(m_own, tmax);
    const float alpha = ex2(m_own - m_new);
    m_own = m_new;
    float psum = 0.f;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      part[r] = ex2(part[r] - m_new);
      psum += part[r];
    }
    l_own = l_own * alpha + ((cl % DUP) == 0 ? psum : 0.f);
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const float a = (G == 1) ? alpha : __shfl_sync(kFullMask, alpha, j * LPH);
      const float2 a2 = make_float2(a, a);
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) o2[j][e] = __fmul2_rn(o2[j][e], a2);
    }

    // ---- o[j] += p(j, slot i) * V(row of slot i), real order
#pragma unroll
    for (int i = 0; i < TPL; ++i) {
      const int t = rw + RPW * i;
      float v[VEC];
      E::load(elem_ptr<KV>(vs, t * D + cl * VEC), v);
      float sv = 1.f;  // NVFP4: this lane's block scale of row t, folded into p
      if constexpr (SCALED) sv = e4m3_to_f32(vsc[t * ROW_SCALES + sblk]);
      if constexpr (kPartial) valid.template keep<VEC>(t, v, sv);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int idx = j * TPL + i;
        const int src = rw * LPR + (idx / C) * DUP;
        float p = __shfl_sync(kFullMask, part[idx % C], src);
        if constexpr (SCALED) p *= sv;
        const float2 p2 = make_float2(p, p);
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e)
          o2[j][e] = __ffma2_rn(p2, make_float2(v[2 * e], v[2 * e + 1]), o2[j][e]);
      }
    }
  }

  // Sums the state over lanes; afterwards lanes of row group 0 hold, for every head j,
  // o[j] over their dims, and lj[j], mj[j] on every lane.
  __device__ __forceinline__ void reduce(float* lj, float* mj) {
    float l = l_own;
#pragma unroll
    for (int mask = LPH / 2; mask >= 1; mask >>= 1) l += __shfl_xor_sync(kFullMask, l, mask);
#pragma unroll
    for (int mask = LPR; mask < 32; mask <<= 1) l += __shfl_xor_sync(kFullMask, l, mask);
#pragma unroll
    for (int j = 0; j < G; ++j) {
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e)
#pragma unroll
        for (int mask = LPR; mask < 32; mask <<= 1) {
          o2[j][e].x += __shfl_xor_sync(kFullMask, o2[j][e].x, mask);
          o2[j][e].y += __shfl_xor_sync(kFullMask, o2[j][e].y, mask);
        }
      lj[j] = __shfl_sync(kFullMask, l, j * LPH);
      mj[j] = __shfl_sync(kFullMask, m_own, j * LPH);
    }
  }

  __device__ __forceinline__ float o(int j, int e) const {
    return (e & 1) ? o2[j][e >> 1].y : o2[j][e >> 1].x;
  }

  // Calls f(head, d, values, VEC, l of the head) for each run of output elements this lane
  // writes (lanes of row group 0 hold the reduced state); lj as filled by reduce().
  template <typename F>
  __device__ __forceinline__ void for_each_out(const float* lj, F&& f) const {
    if (rw != 0) return;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      float v[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = o(j, e);
      f(j, cl * VEC, v, VEC, lj[j]);
    }
  }
  __device__ __forceinline__ bool writes_ml(int lane_) const { return lane_ == 0; }
};

// n fp32 values (n = 2 or a multiple of 4, p aligned to n * 4 bytes up to 16).
__device__ __forceinline__ void store_f32(float* p, const float* v, int n) {
  if (n == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    return;
  }
  for (int e = 0; e < n; e += 4)
    *reinterpret_cast<float4*>(p + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
}

// Output kinds (AttnParams::out_kind).
constexpr int kOutF32 = 0;
constexpr int kOutBF16 = 1;
constexpr int kOutF16 = 2;

__device__ __forceinline__ void store_one(void* out, size_t off, float v, int kind) {
  if (kind == kOutBF16)
    reinterpret_cast<__nv_bfloat16*>(out)[off] = __float2bfloat16_rn(v);
  else if (kind == kOutF16)
    reinterpret_cast<__half*>(out)[off] = __float2half_rn(v);
  else
    reinterpret_cast<float*>(out)[off] = v;
}

__device__ __forceinline__ void store_out(void* out, size_t off, const float* v, int n,
                                          int kind) {
  if (kind == kOutF16) {
    __half* p = reinterpret_cast<__half*>(out) + off;
    if (n % 2 == 0) {
      for (int e = 0; e < n; e += 2)
        *reinterpret_cast<__half2*>(p + e) = __floats2half2_rn(v[e], v[e + 1]);
    } else {
      for (int e = 0; e < n; ++e) p[e] = __float2half_rn(v[e]);
    }
  } else if (kind == kOutBF16) {
    __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(out) + off;
    if (n == 2) {
      *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v[0], v[1]);
    } else if (n == 8) {
      uint4 w;
      __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]);
      __nv_bfloat162 b = __floats2bfloat162_rn(v[2], v[3]);
      __nv_bfloat162 c = __floats2bfloat162_rn(v[4], v[5]);
      __nv_bfloat162 d = __floats2bfloat162_rn(v[6], v[7]);
      w.x = *reinterpret_cast<uint32_t*>(&a);
      w.y = *reinterpret_cast<uint32_t*>(&b);
      w.z = *reinterpret_cast<uint32_t*>(&c);
      w.w = *reinterpret_cast<uint32_t*>(&d);
      *reinterpret_cast<uint4*>(p) = w;
    } else {
      for (int e = 0; e < n; ++e) p[e] = __float2bfloat16_rn(v[e]);
    }
  } else {
    store_f32(reinterpret_cast<float*>(out) + off, v, n);
  }
}

// Arrival counters hold ((call number << 16) | count) ^ kTagMix. A counter written by an
// earlier call (or one that was aborted) carries another call number and counts as 0. The
// mix keeps other data from passing for a live counter: a workspace reused for calls of
// other shapes holds fp32 partial results where this call's counters lie, and zeros or
// small values there would otherwise read as the tag of one of the first calls.
constexpr unsigned long long kTagMix = 0xa5c396e17b2d0000ull;

__device__ __forceinline__ unsigned long long arrival_reset(unsigned long long call) {
  return (call << 16) ^ kTagMix;
}

// Registers one more piece of a segment and returns how many pieces of it this call has
// registered so far.
__device__ __forceinline__ unsigned arrive(unsigned long long* counter,
                                           unsigned long long call) {
  unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(counter);
  while (true) {
    const unsigned long long cur = old ^ kTagMix;
    const unsigned long long next = ((cur >> 16) == call) ? cur + 1 : ((call << 16) | 1ull);
    const unsigned long long seen = atomicCAS(counter, old, next ^ kTagMix);
    if (seen == old) return static_cast<unsigned>(next & 0xffffull);
    old = seen;
  }
}

// Makes the pool's claim counter this call's, with nothing claimed yet, unless it already is
// (a counter of another call, or one never written, is replaced). Each warp does this once,
// before its first claim.
__device__ __forceinline__ void register_claims(unsigned long long* c, unsigned long long call) {
  unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(c);
  while (((old ^ kTagMix) >> 16) != call) {
    const unsigned long long seen = atomicCAS(c, old, arrival_reset(call));
    if (seen == old) return;
    old = seen;
  }
}

// The same for a window, whose segments' pieces arrive together: the counter is made this call's
// first, then counted up by additions. (Exchanges that fail and start again take an L2 round trip
// a piece.)
__device__ __forceinline__ unsigned arrive_add(unsigned long long* counter,
                                               unsigned long long call) {
  register_claims(counter, call);
  return (static_cast<unsigned>(atomicAdd(counter, 1ull)) & 0xffffu) + 1u;
}

// Claims the next pool chunk and returns its index (NW k or more once the pool is used up).
// The tag mix leaves the low 16 bits alone, so the count adds without unmixing; a call makes
// NW k + NW claims, below 2^16, and its last one resets the counter.
__device__ __forceinline__ unsigned claim_chunk(unsigned long long* c) {
  return static_cast<unsigned>(atomicAdd(c, 1ull) & 0xffffull);
}

// Log-sum-exp merge of the pieces of one segment (request b, kv-head h) into out, done by
// the warp that registered the segment's last piece. Pieces come from units w0..w1 (the
// first may hold it as its tail piece); empty units hold none. For each head j:
//   M = max m_i,  L = sum l_i 2^(m_i - M),  out = sum o_i 2^(m_i - M) / L.
// All heads are merged together so the loads of one pass are in flight at once: lane i
// reads piece i's (m, l) of every head, then lanes stream the pieces' o rows. Pieces are
// read from L2 (ld.cg): other SMs wrote them during this launch.
template <int D, int G, int HP>
__device__ __forceinline__ void merge_heads(const AttnParams& p, int b, int h, int j0, int w0,
                                            int w1, bool w0_tail, const Units un, int lane) {
  constexpr int PER = D / 32;
  auto slot_of = [&](int w) { return 2 * w + ((w == w0 && w0_tail) ? 1 : 0); };
  const float* ml = p.ws_ml;
  // pass 1: M[j] over all pieces (lane i looks at unit w0 + i, w0 + i + 32, ...)
  float M[HP];
#pragma unroll
  for (int j = 0; j < HP; ++j) M[j] = -INFINITY;
  for (int w = w0 + lane; w <= w1; w += 32) {
    if (!un.live(w)) continue;
    const float2* mlw =
        reinterpret_cast<const float2*>(ml) + static_cast<size_t>(slot_of(w)) * G + j0;
#pragma unroll
    for (int j = 0; j < HP; ++j) M[j] = fmaxf(M[j], __ldcg(mlw + j).x);
  }
#pragma unroll
  for (int j = 0; j < HP; ++j)
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) M[j] = fmaxf(M[j], __shfl_xor_sync(kFullMask, M[j], m));

  // pass 2: weights, L[j], and the weighted o rows
  float acc[HP][PER], Lsum[HP];
#pragma unroll
  for (int j = 0; j < HP; ++j) {
    Lsum[j] = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[j][e] = 0.f;
  }
  for (int base = w0; base <= w1; base += 32) {
    const int w = base + lane;
    float f[HP];
#pragma unroll
    for (int j = 0; j < HP; ++j) f[j] = 0.f;
    const bool mine = w <= w1 && un.live(w);
    const unsigned live_mask = __ballot_sync(kFullMask, mine);  // bit i: unit base + i
    if (mine) {
      const float2* mlw =
          reinterpret_cast<const float2*>(ml) + static_cast<size_t>(slot_of(w)) * G + j0;
#pragma unroll
      for (int j = 0; j < HP; ++j) {
        const float2 v = __ldcg(mlw + j);
        f[j] = ex2(v.x - M[j]);
        Lsum[j] += v.y * f[j];
      }
    }
    // The live pieces of this group of 32 units, U rows in flight at once (each load is an L2
    // round trip), in increasing unit order. Empty units are skipped outright: a launch with
    // fewer tiles than warps leaves most units empty, and a segment's range of units can
    // hold hundreds of them. A missing slot of the last batch reads piece w0's row (always
    // written: w0 holds the segment's first tile) and is left out of the sum by its flag, not
    // by a zero weight (its row may hold NaN).
    constexpr int U = HP * PER <= 4 ? 4 : 1;  // wider would spill in the kernels with G >= 2
    unsigned rest = live_mask;  // the same on every lane
    while (rest != 0u) {
      float v[U][HP][PER];
      float fu[U][HP];
      bool use[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        use[u] = rest != 0u;
        const int i = use[u] ? __ffs(rest) - 1 : 0;
        rest &= rest - 1u;  // no-op once empty
        const float* row =
            p.ws_o + (static_cast<size_t>(slot_of(use[u] ? base + i : w0)) * G + j0) * D;
#pragma unroll
        for (int j = 0; j < HP; ++j) {
          fu[u][j] = __shfl_sync(kFullMask, f[j], i);
#pragma unroll
          for (int e = 0; e < PER; ++e) v[u][j][e] = __ldcg(row + j * D + lane + 32 * e);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!use[u]) continue;
#pragma unroll
        for (int j = 0; j < HP; ++j)
#pragma unroll
          for (int e = 0; e < PER; ++e) acc[j][e] = fmaf(v[u][j][e], fu[u][j], acc[j][e]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < HP; ++j) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) Lsum[j] += __shfl_xor_sync(kFullMask, Lsum[j], m);
    const size_t row = (static_cast<size_t>(b) * p.H + static_cast<size_t>(h) * G + j0 + j) * D;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const float v = acc[j][e] * (p.v_scale / Lsum[j]);
      store_one(p.out, row + lane + 32 * e, v, p.out_kind);
    }
  }
}

// Merges all G heads of a segment, at most four heads per pass (register budget).
template <int D, int G>
__device__ void merge_segment(const AttnParams& p, int b, int h, int w0, int w1, bool w0_tail,
                              const Units un, int lane) {
  constexpr int HP = G < 4 ? G : 4;
#pragma unroll 1
  for (int j0 = 0; j0 < G; j0 += HP)
    merge_heads<D, G, HP>(p, b, h, j0, w0, w1, w0_tail, un, lane);
}

// The same merge for a window, most of whose launches are short and a good part of their time the
// merge's: a lane takes four columns of a head, and eight loads of a lane are in flight at once
// (with a piece's after the other's, each an L2 round trip, 33 pieces of 8 heads took 50 us).
// Windows against the merge and the arrivals above: 4 requests of 16/2 heads of 64 over 250 + 4 keys
// 20.5 us for 30.8, 2 of 32/8 over 8192 + 4 56 for 117, one over 30000 + 4 87 for 188, 8 of them
// 196 for 233, 256 over 4096 + 4 418 for 414. The kernels without a window keep theirs: with this
// one a single request of 30000 tokens takes 93 us for 240 and short launches up to 4 us less, 64
// requests of 64/8 heads over 4096 312 for 305, and sums are added in another order.
template <int D, int G>
__device__ __forceinline__ void merge_segment_wide(const AttnParams& p, int b, int h, int w0,
                                                   int w1, bool w0_tail, const Units un,
                                                   int lane) {
  constexpr int kHeads = 128 / D;                               // heads of a warp's load
  constexpr int kSets = (G + kHeads - 1) / kHeads;              // loads of a piece
  constexpr int kHere = kSets < 4 ? kSets : 4;                  // of them at once
  constexpr int kBatch = 8 / kHere;                             // pieces at once
  const int sub = lane / (D / 4);                               // this lane's head of a load
  auto slot_of = [&](int w) { return 2 * w + ((w == w0 && w0_tail) ? 1 : 0); };
  const float2* ml = reinterpret_cast<const float2*>(p.ws_ml);
  // lane i looks at unit w0 + i, w0 + i + 32, ...
  float M[G], L[G];
#pragma unroll
  for (int j = 0; j < G; ++j) {
    M[j] = -INFINITY;
    L[j] = 0.f;
  }
  for (int w = w0 + lane; w <= w1; w += 32)
    if (un.live(w))
#pragma unroll
      for (int j = 0; j < G; ++j)
        M[j] = fmaxf(M[j], __ldcg(ml + static_cast<size_t>(slot_of(w)) * G + j).x);
#pragma unroll
  for (int j = 0; j < G; ++j)
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) M[j] = fmaxf(M[j], __shfl_xor_sync(kFullMask, M[j], m));
  float4 acc[kSets];
#pragma unroll
  for (int s = 0; s < kSets; ++s) acc[s] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int base = w0; base <= w1; base += 32) {
    const int w = base + lane;
    const bool mine = w <= w1 && un.live(w);
    const unsigned live_mask = __ballot_sync(kFullMask, mine);
    float f[G];
#pragma unroll
    for (int j = 0; j < G; ++j) {
      f[j] = 0.f;
      if (mine) {
        const float2 v = __ldcg(ml + static_cast<size_t>(slot_of(w)) * G + j);
        f[j] = ex2(v.x - M[j]);
        L[j] = fmaf(v.y, f[j], L[j]);
      }
    }
#pragma unroll
    for (int s0 = 0; s0 < kSets; s0 += kHere) {
      unsigned rest = live_mask;  // the same on every lane
#pragma unroll 1
      while (rest != 0u) {
        float4 o[kBatch][kHere];
        int from[kBatch];
        unsigned todo = rest;
        // a missing piece of the last batch reads one that is there, and counts nothing
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          from[u] = todo != 0u ? __ffs(todo) - 1 : -1;
          todo &= todo - 1u;
          const size_t row = static_cast<size_t>(slot_of(from[u] >= 0 ? base + from[u] : w0)) * G;
#pragma unroll
          for (int s = 0; s < kHere; ++s) {
            const int j = min((s0 + s) * kHeads + sub, G - 1);
            o[u][s] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + (row + j) * D) +
                             lane % (D / 4));
          }
        }
        rest = todo;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (from[u] < 0) continue;
#pragma unroll
          for (int s = 0; s < kHere; ++s) {
            const int j = (s0 + s) * kHeads;
            float g = __shfl_sync(kFullMask, f[j], from[u]);
            if (kHeads == 2 && j + 1 < G) {
              const float g1 = __shfl_sync(kFullMask, f[j + 1 < G ? j + 1 : j], from[u]);
              if (sub == 1) g = g1;
            }
            float4& to = acc[s0 + s];
            to.x = fmaf(o[u][s].x, g, to.x);
            to.y = fmaf(o[u][s].y, g, to.y);
            to.z = fmaf(o[u][s].z, g, to.z);
            to.w = fmaf(o[u][s].w, g, to.w);
          }
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < G; ++j)
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) L[j] += __shfl_xor_sync(kFullMask, L[j], m);
#pragma unroll
  for (int s = 0; s < kSets; ++s) {
    const int j = s * kHeads + sub;
    const float l = kHeads == 2 && sub == 1 ? L[s * kHeads + 1 < G ? s * kHeads + 1 : 0]
                                            : L[s * kHeads];
    if (j >= G) continue;
    const float inv = p.v_scale / l;
    const float v[4] = {acc[s].x * inv, acc[s].y * inv, acc[s].z * inv, acc[s].w * inv};
    const size_t at = (static_cast<size_t>(b) * p.H + static_cast<size_t>(h) * G + j) * D +
                      4 * (lane % (D / 4));
    store_out(p.out, at, v, 2, p.out_kind);
    store_out(p.out, at + 2, v + 2, 2, p.out_kind);
  }
}

// Tiles of the first n >= 0 tokens.
__device__ __forceinline__ int tiles_of(int n) { return (n >> 4) + ((n & 15) != 0); }

// MODE selects the tile step: kModeCuda (CUDA cores), kModeTc (tensor cores, one kv-head
// per tile) or kModeTcPair (tensor cores, two adjacent kv-heads per tile, loaded by one
// 4-D TMA box). G is the unit's query heads: the kv-head's G, or 2 G for a pair; p.H_kv
// counts units (kv-heads, or pairs).
template <typename KV, typename QT, int D, int G, int MODE, bool kWindow>
__global__ void __launch_bounds__(warps_for_mode(G, MODE, std::is_same<KV, nvfp4>::value) * 32,
                                  1)
    attn_partial_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const AttnParams p) {
  constexpr bool TC = MODE != kModeCuda;
  using Geo = Geometry<KV, QT, D, G>;
  using W = std::conditional_t<
      MODE == kModeCuda, WarpAttn<KV, QT, D, G>,
      std::conditional_t<MODE == kModeTc, WarpAttnTC<KV, D, G>, WarpAttnTCPair<KV, D, G / 2>>>;
  // a unit's tile: one head tile, or a pair's two head tiles back to back
  constexpr int kHeads = MODE == kModeTcPair ? 2 : 1;
  constexpr uint32_t kTile = kHeads * Geo::TILE_BYTES;
  constexpr uint32_t kScales = kHeads * Geo::SCALE_BYTES;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  // The host reserves stage_align(TC) - 128 spare bytes; the layout starts at the first
  // aligned address (swizzled TMA tiles need the swizzle period's alignment).
  constexpr uint32_t kAlign = stage_align(TC);
  unsigned char* smem =
      smem_raw + ((kAlign - (smem_addr(smem_raw) & (kAlign - 1))) & (kAlign - 1));
  if ((smem_addr(smem_raw) & 127u) != 0) {  // TMA destinations assume 128-byte alignment
    if (threadIdx.x == 0) atomic_or_error(p.error_word, PDA_DEVERR_TIMEOUT);
    return;
  }

  const int tid = threadIdx.x;
  const int lane = tid & 31;
  const int warp = tid >> 5;
  const int nwarps = blockDim.x >> 5;
  const int B = p.B;

  // ---- shared layout: prefix table (kWindow: and the tiles each request skips) | stage buffers |
  // barriers | stage info words
  int32_t* s_pre = reinterpret_cast<int32_t*>(smem);
  int32_t* s_skip = s_pre + B + 1;
  unsigned char* s_stage = smem + p.prefix_bytes;
  const size_t stage_region = static_cast<size_t>(nwarps) * p.stages * p.stage_bytes;
  uint64_t* s_bar = reinterpret_cast<uint64_t*>(s_stage + stage_region);
  int32_t* s_info = reinterpret_cast<int32_t*>(s_bar + nwarps * p.stages);
  int2* s_meta = reinterpret_cast<int2*>(
      (reinterpret_cast<uintptr_t>(s_info + nwarps * p.stages) + 7) & ~uintptr_t(7));

  // The tensor maps' descriptors are fetched while the prologue below reads the lengths.
  if (tid == 0) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }

  // ---- 1. block prefix sums of per-request tile counts (every block computes its own)
  const int cap_tokens = min(p.max_blocks * p.block_size, p.max_context_len);
  // tiles between the first tokens' and the window's, of a request of L tokens
  auto skipped = [&](int L) {
    return kWindow ? max(0, (max(0, L - p.window) >> 4) - tiles_of(p.sinks)) : 0;
  };
  {
    const int per = (B + blockDim.x - 1) / blockDim.x;
    const int lo = min(B, tid * per), hi = min(B, lo + per);
    int local = 0;
    for (int b = lo; b < hi; ++b) {
      const int L = p.context_lens[b];
      const bool ok = L >= 0 && L <= cap_tokens;
      local += ok ? (L + kBS - 1) / kBS - skipped(L) : 0;
    }
    // block-wide exclusive scan of `local`
    int incl = local;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(kFullMask, incl, d);
      if (lane >= d) incl += y;
    }
    __shared__ int warp_tot[kMaxWarps];
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += warp_tot[w];
    int run = base + incl - local;
    for (int b = lo; b < hi; ++b) {
      s_pre[b] = run;
      const int L = p.context_lens[b];
      const bool ok = L >= 0 && L <= cap_tokens;
      if constexpr (kWindow) s_skip[b] = ok ? skipped(L) : 0;
      run += ok ? (L + kBS - 1) / kBS - skipped(L) : 0;
    }
    if (tid == blockDim.x - 1) s_pre[B] = run;
  }
  // barrier init (one lane per warp, its own stages)
  if (lane == 0) {
    // one arrive carries the byte count of the stage's copies
    for (int s = 0; s < p.stages; ++s) mbar_init(&s_bar[warp * p.stages + s], 1);
    fence_mbar_init();
  }
  __syncthreads();

  // ---- 2. rows that get no tiles: empty histories (zeros) and invalid lengths (NaN)
  for (int b = blockIdx.x; b < B; b += gridDim.x) {
    if (s_pre[b + 1] != s_pre[b]) continue;
    const int L = p.context_lens[b];
    const bool bad = !(L >= 0 && L <= cap_tokens);
    if (bad && tid == 0) atomic_or_error(p.error_word, PDA_DEVERR_CONTEXT_LEN);
    const float val = bad ? __int_as_float(0x7fc00000) : 0.f;
    for (int i = tid; i < p.H * D; i += blockDim.x) {
      const size_t off = static_cast<size_t>(b) * p.H * D + i;
      store_one(p.out, off, val, p.out_kind);
    }
  }

  // ---- 3. this warp's work: its static unit, then pool chunks while any are left
  const int H_kv = p.H_kv;
  const int W_tiles = s_pre[B] * H_kv;
  // Workers: the grid's warps, but no more than give each PDA_MIN_TILES_PER_WARP tiles of
  // this launch (the host sized the grid by its bound on the lengths; the lengths on the
  // device may be shorter). The others leave here. Only the CUDA-core step leaves a pool
  // (see make_plan); the tensor-core steps compile without it.
  const int least = kWindow ? window_tiles_per_warp(W_tiles, B * H_kv) : PDA_MIN_TILES_PER_WARP;
  const int nw = max(1, min(p.num_workers, (W_tiles + least - 1) / least));
  const int wi = blockIdx.x * nwarps + warp;
  if (wi >= nw) return;
  const Units un = make_units(W_tiles, nw, MODE == kModeCuda ? p.pool_k : 0);
  const int w = wi * (un.k + 1);  // this warp's static unit
  if (un.k == 0 && !un.live(w)) return;

  unsigned char* my_stage = s_stage + static_cast<size_t>(warp) * p.stages * p.stage_bytes;
  uint64_t* my_bar = s_bar + warp * p.stages;
  int32_t* my_info = s_info + warp * p.stages;
  auto k_buf = [&](int s) { return reinterpret_cast<KV*>(my_stage + s * p.stage_bytes); };
  auto v_buf = [&](int s) {
    return reinterpret_cast<KV*>(my_stage + s * p.stage_bytes + kTile);
  };
  auto ks_buf = [&](int s) {  // NVFP4 block scales of the K tile, [kHeads][16][D/16]
    return reinterpret_cast<uint8_t*>(my_stage + s * p.stage_bytes + 2 * kTile);
  };
  auto vs_buf = [&](int s) {
    return reinterpret_cast<uint8_t*>(my_stage + s * p.stage_bytes + 2 * kTile + kScales);
  };
  auto q_buf = [&](int s) {
    return reinterpret_cast<QT*>(my_stage + s * p.stage_bytes + 2 * kTile + 2 * kScales);
  };

  // (request, kv-head, block) of tile y
  auto locate = [&](int y, int& b, int& h, int& blk, int& nb) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_pre[mid] * H_kv <= y) lo = mid; else hi = mid;
    }
    b = lo;
    nb = s_pre[b + 1] - s_pre[b];
    const int rem = y - s_pre[b] * H_kv;
    h = rem / nb;
    blk = rem - h * nb;
  };

  const uint64_t policy = l2_policy_evict_first();
  int2* my_meta = s_meta + warp * 64;
  const int S = p.stages;
  // The stage ring persists across units: every tile a unit loads is consumed within it, so
  // the next unit starts on the stage (and phase) after the last one used.
  int stage = 0;
  uint32_t phase = 0;
  W st;
  st.init(lane);
  bool registered = false;

  // Runs tiles [t_begin, t_end) as unit `unit`. When claim_next is set, lane 0 claims the
  // next pool chunk as soon as the range has no more tiles to load (the atomic's latency
  // hides behind the range's last tiles); the claimed index is returned through `claimed`.
  // Returns false after a wait that timed out (the error bit is set).
  auto run = [&](int t_begin, int t_end, int unit, bool claim_next, unsigned& claimed) -> bool {
    // Issue-side metadata, one group of 32 tiles at a time: lane i describes tile
    // g_base + i. The block id and context length of the next group are fetched with
    // cp.async a whole group ahead into this warp's two-slot ring, so the lane that issues a
    // tile never waits on a global load. Each lane reads only the slot it filled itself.
    int g_base = t_begin, g_buf = 0;
    int cur_b = 0, cur_h = 0, cur_blk = 0, cur_pid = 0, cur_len = 0;
    int nxt_b = 0, nxt_h = 0, nxt_blk = 0;
    bool cur_first = false, nxt_first = false;  // the segment's first tile
    auto prefetch = [&](int base, int buf) {
      const int y = base + lane;
      if (y < t_end) {
        int nb;
        locate(y, nxt_b, nxt_h, nxt_blk, nb);
        if constexpr (kWindow) {
          nxt_first = nxt_blk == 0;
          if (nxt_blk >= tiles_of(p.sinks)) nxt_blk += s_skip[nxt_b];
        }
        cp_async4(&my_meta[buf * 32 + lane].x, p.block_tables +
                                                       static_cast<size_t>(nxt_b) * p.max_blocks +
                                                       (nxt_blk >> p.bs_shift));
        cp_async4(&my_meta[buf * 32 + lane].y, p.context_lens + nxt_b);
      }
      cp_async_commit();
    };
    auto enter = [&](int base, int buf) {  // the group starting at `base` becomes current
      cp_async_wait_all();
      g_base = base;
      g_buf = buf;
      cur_b = nxt_b;
      cur_h = nxt_h;
      cur_blk = nxt_blk;
      cur_first = nxt_first;
      const int2 m = my_meta[buf * 32 + lane];
      cur_pid = m.x;
      cur_len = m.y;
      if (base + 32 < t_end) prefetch(base + 32, buf ^ 1);
    };
    prefetch(t_begin, 0);
    enter(t_begin, 0);
    auto issue = [&](int x, int s) {
      if (x >= g_base + 32) enter(g_base + 32, g_buf ^ 1);
      if (lane == x - g_base) {
        const bool bad = cur_pid < 0 || cur_pid >= p.num_blocks;
        const bool need_q = (kWindow ? cur_first : cur_blk == 0) || (x == t_begin);
        if constexpr (kWindow) {
          // a bit per row of the tile that counts
          auto below = [&](int n) { return (1u << min(max(n - cur_blk * kBS, 0), kBS)) - 1u; };
          const uint32_t rows =
              below(cur_len) & (~below(cur_len - p.window) | below(p.sinks));
          my_info[s] = static_cast<int32_t>(rows | (bad ? kBadTile : 0));
        } else {
          const int n_valid = min(kBS, cur_len - cur_blk * kBS);
          my_info[s] = n_valid | (bad ? kBadTile : 0);
        }
        if (bad) atomic_or_error(p.error_word, PDA_DEVERR_BLOCK_ID);
        const uint32_t bytes = 2 * kTile + 2 * kScales + (need_q ? Geo::Q_BYTES : 0);
        mbar_arrive_expect_tx(&my_bar[s], bytes);
        // the tile is rows sub * 16 .. + 15 of its physical block
        const int sub = cur_blk & ((1 << p.bs_shift) - 1);
        const int row = (bad ? 0 : cur_pid) * p.block_size + sub * kBS;
        if constexpr (Geo::SCALED) {
          // scales [blocks][heads][block_size][D/16]: each head's 16 rows are one run; with
          // 16-token blocks a pair's two runs are adjacent (one copy)
          constexpr uint32_t kRun = Geo::SCALE_BYTES;  // one head's 16 rows
          const size_t head0 = static_cast<size_t>(bad ? 0 : cur_pid) * H_kv * kHeads +
                               static_cast<size_t>(cur_h) * kHeads;
          const size_t off = (head0 * p.block_size + static_cast<size_t>(sub) * kBS) *
                             Geo::ROW_SCALES;
          if (kHeads == 1 || p.bs_shift == 0) {
            bulk_load(ks_buf(s), p.k_bscales + off, kScales, &my_bar[s]);
            bulk_load(vs_buf(s), p.v_bscales + off, kScales, &my_bar[s]);
          } else {
            const size_t step = static_cast<size_t>(p.block_size) * Geo::ROW_SCALES;
#pragma unroll
            for (int u = 0; u < kHeads; ++u) {
              bulk_load(ks_buf(s) + u * kRun, p.k_bscales + off + u * step, kRun, &my_bar[s]);
              bulk_load(vs_buf(s) + u * kRun, p.v_bscales + off + u * step, kRun, &my_bar[s]);
            }
          }
        }
        if constexpr (MODE == kModeTcPair) {  // both heads of pair cur_h in one box
          tma_load_4d(k_buf(s), &tmK, 0, row, 0, cur_h, &my_bar[s], policy);
          tma_load_4d(v_buf(s), &tmV, 0, row, 0, cur_h, &my_bar[s], policy);
        } else {
          tma_load_3d(k_buf(s), &tmK, 0, cur_h, row, &my_bar[s], policy);
          tma_load_3d(v_buf(s), &tmV, 0, cur_h, row, &my_bar[s], policy);
        }
        if (need_q) {
          const QT* src = reinterpret_cast<const QT*>(p.q) +
                          (static_cast<size_t>(cur_b) * p.H + static_cast<size_t>(cur_h) * G) * D;
          bulk_load(q_buf(s), src, Geo::Q_BYTES, &my_bar[s]);
        }
      }
    };

    const int n_tiles = t_end - t_begin;
    for (int i = 0; i < S && i < n_tiles; ++i) issue(t_begin + i, (stage + i) % S);
    if (claim_next && !registered) {  // overlaps the first loads
      if (lane == 0) register_claims(p.ws_claim, p.call);
      registered = true;
    }
    unsigned next_claim = 0;
    if (claim_next && n_tiles < S && lane == 0) next_claim = claim_chunk(p.ws_claim);

    // Consumer-side sequential position.
    int cb, ch, cblk, cnb;
    locate(t_begin, cb, ch, cblk, cnb);
    bool seg_bad = false;
    int head_seg = -1, tail_seg = -1;  // segments to merge

    for (int x = t_begin; x < t_end; ++x) {
      const bool ready = __all_sync(kFullMask, mbar_wait_bounded(&my_bar[stage], phase));
      if (!ready) {
        atomic_or_error(p.error_word, PDA_DEVERR_TIMEOUT);
        cp_async_wait_all();
        // Give copies still in flight a bounded chance to land before leaving.
        for (int y = x; y < min(t_end, x + S); ++y) {
          const int s2 = (stage + (y - x)) % S;
          const uint32_t ph2 = phase ^ (((stage + (y - x)) / S) & 1);
          mbar_wait_bounded(&my_bar[s2], ph2);
        }
        return false;
      }
      const int info = my_info[stage];
      if (cblk == 0 || x == t_begin) {
        st.reset(q_buf(stage), p.scale_log2);
        seg_bad = false;
      }
      seg_bad |= (info & kBadTile) != 0;
      const std::conditional_t<kWindow, RowMask, FirstRows> valid{info & (kBadTile - 1)};
      if (valid.all())
        st.template tile<false>(k_buf(stage), v_buf(stage), ks_buf(stage), vs_buf(stage), valid);
      else
        st.template tile<true>(k_buf(stage), v_buf(stage), ks_buf(stage), vs_buf(stage), valid);

      // hand the stage back to the TMA engine
      __syncwarp();
      fence_proxy_async_smem();
      if (x + S < t_end)
        issue(x + S, stage);
      else if (claim_next && x + S == t_end && lane == 0)  // nothing left to load
        next_claim = claim_chunk(p.ws_claim);
      if (++stage == S) {
        stage = 0;
        phase ^= 1;
      }

      // segment end?
      const bool last_of_seg = (cblk + 1 == cnb);
      if (last_of_seg || x + 1 == t_end) {
        float lj[G], mj[G];
        st.reduce(lj, mj);
        const int seg_start = s_pre[cb] * H_kv + ch * cnb;
        const int seg_end = seg_start + cnb;
        const bool complete = seg_start >= t_begin && seg_end <= t_end;
        if (complete) {
          st.for_each_out(lj, [&](int j, int d, const float* o, int n, float l) {
            float v[8];
            const float inv = seg_bad ? __int_as_float(0x7fc00000) : p.v_scale / l;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e < n) v[e] = o[e] * inv;
            const size_t off =
                (static_cast<size_t>(cb) * p.H + static_cast<size_t>(ch) * G + j) * D + d;
            store_out(p.out, off, v, n, p.out_kind);
          });
        } else {
          // A piece of a segment cut by a unit boundary: store (m, l, o), register it, and
          // merge the segment if this was its last piece.
          const int slot = 2 * unit + (seg_start <= t_begin ? 0 : 1);
          st.for_each_out(lj, [&](int j, int d, const float* o, int n, float) {
            store_f32(p.ws_o + (static_cast<size_t>(slot) * G + j) * D + d, o, n);
          });
          if (st.writes_ml(lane)) {
#pragma unroll
            for (int j = 0; j < G; ++j) {
              p.ws_ml[(static_cast<size_t>(slot) * G + j) * 2 + 0] = mj[j];
              p.ws_ml[(static_cast<size_t>(slot) * G + j) * 2 + 1] =
                  seg_bad ? __int_as_float(0x7fc00000) : lj[j];
            }
          }
          __threadfence();  // this lane's piece stores before the arrival below
          __syncwarp();
          const int seg = cb * H_kv + ch;
          unsigned arrived = 0;
          if (lane == 0)
            arrived = kWindow ? arrive_add(p.ws_arrive + seg, p.call)
                              : arrive(p.ws_arrive + seg, p.call);
          arrived = __shfl_sync(kFullMask, arrived, 0);
          const int w0 = un.owner(seg_start);
          const int w1 = un.owner(seg_end - 1);
          unsigned pieces = 0;
          for (int wb = w0; wb <= w1; wb += 32) {
            const int ww = wb + lane;
            pieces += __popc(__ballot_sync(kFullMask, ww <= w1 && un.live(ww)));
          }
          if (arrived == pieces) {
            if constexpr (kWindow) {  // merged behind the unit's tiles
              if (seg_start <= t_begin)
                head_seg = seg;
              else
                tail_seg = seg;
            } else {
              __threadfence();  // see the other pieces' stores
              merge_segment<D, G>(p, cb, ch, w0, w1, seg_start != un.start(w0), un, lane);
              if (lane == 0) atomicExch(p.ws_arrive + seg, arrival_reset(p.call));
            }
          }
        }
      }
      // advance the consumer position
      if (++cblk == cnb) {
        cblk = 0;
        if (++ch == H_kv) {
          ch = 0;
          do {
            ++cb;
          } while (cb < B && s_pre[cb + 1] == s_pre[cb]);
        }
        if (cb < B) cnb = s_pre[cb + 1] - s_pre[cb];
      }
    }
    if constexpr (kWindow) {
      // Segments whose last piece this unit brought: at most its first and its last. Behind the
      // loop, so that the merge's registers are not held beside the tiles' (within it, it spilled
      // them: 690 us for 633 on 256 requests over 4100 keys).
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        const int seg = k == 0 ? head_seg : tail_seg;
        if (seg < 0) continue;
        const int mb = seg / H_kv, mh = seg - mb * H_kv, nb = s_pre[mb + 1] - s_pre[mb];
        const int seg_start = s_pre[mb] * H_kv + mh * nb;
        const int w0 = un.owner(seg_start), w1 = un.owner(seg_start + nb - 1);
        __threadfence();  // see the other pieces' stores
        merge_segment_wide<D, G>(p, mb, mh, w0, w1, seg_start != un.start(w0), un, lane);
        if (lane == 0) atomicExch(p.ws_arrive + seg, arrival_reset(p.call));
      }
    }
    claimed = __shfl_sync(kFullMask, next_claim, 0);
    return true;
  };

  const bool pool = un.k > 0;
  const unsigned n_chunks = static_cast<unsigned>(un.NW) * un.k;
  unsigned c = 0;
  if (un.live(w)) {
    if (!run(un.start(w), un.start(w + 1), w, pool, c)) return;
  } else if (pool) {
    if (lane == 0) {
      register_claims(p.ws_claim, p.call);
      c = claim_chunk(p.ws_claim);
    }
    registered = true;
    c = __shfl_sync(kFullMask, c, 0);
  }
  // pool chunks, each the next one nobody has taken yet
  while (pool && c < n_chunks) {
    const int u = un.chunk_unit(static_cast<int>(c));
    if (un.live(u)) {
      if (!run(un.start(u), un.start(u + 1), u, true, c)) return;
    } else {
      if (lane == 0) c = claim_chunk(p.ws_claim);
      c = __shfl_sync(kFullMask, c, 0);
    }
  }
  // Every warp ends with one claim past the pool, so NW k + NW claims are made, as many as there
  // are units, and whoever makes the last leaves the counter with nothing claimed: a captured call
  // keeps its number, and its next replay would find the pool used up.
  if (pool && lane == 0 && static_cast<int>(c) + 1 == un.units())
    atomicExch(p.ws_claim, arrival_reset(p.call));
}

// ------------------------------------------------------------------ the launch's choice of kernel
using KernelFn = void (*)(const CUtensorMap, const CUtensorMap, const AttnParams);

// The kernel for a unit of G_u query heads in the given mode.
template <typename KV, typename QT, int D, bool kWindow>
KernelFn pick_g(int G_u, int mode) {
  if constexpr (std::is_same<KV, fp8e4m3>::value || std::is_same<KV, nvfp4>::value) {
    if constexpr (D == 128) {
      if (mode == kModeTcPair) {
        switch (G_u) {
          case 2: return attn_partial_kernel<KV, QT, D, 2, kModeTcPair, kWindow>;
          case 4: return attn_partial_kernel<KV, QT, D, 4, kModeTcPair, kWindow>;
          case 8: return attn_partial_kernel<KV, QT, D, 8, kModeTcPair, kWindow>;
          default: return nullptr;
        }
      }
      if (mode == kModeTc) {
        switch (G_u) {
          case 2: return attn_partial_kernel<KV, QT, D, 2, kModeTc, kWindow>;
          case 4: return attn_partial_kernel<KV, QT, D, 4, kModeTc, kWindow>;
          case 8: return attn_partial_kernel<KV, QT, D, 8, kModeTc, kWindow>;
          default: return nullptr;
        }
      }
    }
  }
  if (mode != kModeCuda) return nullptr;
  switch (G_u) {
    case 1: return attn_partial_kernel<KV, QT, D, 1, kModeCuda, kWindow>;
    case 2: return attn_partial_kernel<KV, QT, D, 2, kModeCuda, kWindow>;
    case 4: return attn_partial_kernel<KV, QT, D, 4, kModeCuda, kWindow>;
    case 8: return attn_partial_kernel<KV, QT, D, 8, kModeCuda, kWindow>;
    default: return nullptr;
  }
}

template <typename KV, typename QT, bool kWindow>
KernelFn pick_d(int D, int G_u, int mode) {
  if (D == 128) return pick_g<KV, QT, 128, kWindow>(G_u, mode);
  if (D == 64) return pick_g<KV, QT, 64, kWindow>(G_u, mode);
  return nullptr;
}

// The windowed kernels, compiled in units of their own.
KernelFn pick_window_kernel(pda_dtype kv, int D, int G_u, int mode);
KernelFn pick_window_codes_kernel(pda_dtype kv, int D, int G_u, int mode);

}  // namespace pda
