// decode_attention.cu -- the host side of decode attention: tiling, launch plan, workspace and the
// C entry points (the kernel is in decode_kernel.cuh).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>
#include <utility>
#include <vector>

#include "decode_kernel.cuh"

namespace pda {

// ------------------------------------------------------------------ host side
namespace {

struct LaunchPlan {
  int nwarps, stages, grid;
  int pool_k;  // pool chunks per warp the workspace has piece slots for (0: all static)
  uint32_t stage_bytes, prefix_bytes;
  size_t smem_bytes;
  size_t ws_arrive, ws_claim, ws_ml, ws_o, ws_total;  // byte offsets / total
};

// q is bf16 beside a quantised cache, otherwise of the cache's own type.
size_t q_bytes_for(pda_dtype kv) {
  return (kv == PDA_FP8_E4M3 || kv == PDA_NVFP4) ? 2u : dtype_bytes(kv);
}

// How a launch tiles the work: the tile step and the unit (one kv-head, or a pair).
struct Tiling {
  int mode;   // kModeCuda, kModeTc or kModeTcPair
  int H_u;    // units per request (kv-heads, or pairs)
  int G_u;    // query heads per unit
};

// Quantised caches at D = 128 run on the tensor cores. Where H_kv is even and G <= 4, two
// adjacent kv-heads share a tile (one TMA box and one pipeline step for both): per byte
// that halves the TMA operations, which bound small quantised tiles (about one per 120 SM
// cycles, whatever their size), and the per-tile pipeline work. Otherwise a quantised tile
// is one kv-head on the tensor cores for G >= 2, and on the CUDA cores for G = 1 (a plain
// GEMV, where they keep up: measured equal to the single-head tensor-core step).
Tiling tiling_for(pda_dtype kv, int D, int H_kv, int G) {
  const bool quantised = kv == PDA_FP8_E4M3 || kv == PDA_NVFP4;
  if (quantised && D == 128 && G <= 4 && H_kv % 2 == 0) return {kModeTcPair, H_kv / 2, 2 * G};
  if (quantised && D == 128 && G >= 2) return {kModeTc, H_kv, G};
  return {kModeCuda, H_kv, G};
}

// One pipeline stage: the K and V tiles, (NVFP4) their block scales, the q rows, for a unit.
uint32_t stage_bytes_for(pda_dtype kv, int D, const Tiling& t) {
  const size_t heads = t.mode == kModeTcPair ? 2 : 1;
  const size_t tile = heads * (kv == PDA_NVFP4 ? kBS * D / 2 : kBS * D * dtype_bytes(kv));
  const size_t scales = heads * (kv == PDA_NVFP4 ? 2 * kBS * D / 16 : 0);
  const size_t q = static_cast<size_t>(t.G_u) * D * q_bytes_for(kv);
  return static_cast<uint32_t>(
      round_up(2 * tile + scales + q, stage_align(t.mode != kModeCuda)));
}

// pool: leave a share of the tiles to chunks claimed at run time (see Units); the
// workspace then holds piece slots for them as well.
bool make_plan(int B, int H_kv, int G, int D, pda_dtype kv, int sm_cap, int num_sms, bool pool,
               bool windowed, LaunchPlan* pl) {
  const Tiling t = tiling_for(kv, D, H_kv, G);
  const bool tc = t.mode != kModeCuda;
  const size_t align = stage_align(tc);
  pl->stage_bytes = stage_bytes_for(kv, D, t);
  pl->prefix_bytes = static_cast<uint32_t>(
      round_up(static_cast<size_t>(windowed ? 2 * B + 1 : B + 1) * 4, align));
  // + alignment of the metadata ring, + room to align the layout's start
  const size_t fixed = pl->prefix_bytes + 8 + (align - 128);
  if (fixed >= static_cast<size_t>(kSmemBudget)) return false;
  pl->nwarps = 0;
  // The most warps that still get two stages each; then as many stages as fit.
  for (int nw = warps_for_mode(t.G_u, t.mode, kv == PDA_NVFP4); nw >= 2; --nw) {
    const size_t per_stage = static_cast<size_t>(nw) * (pl->stage_bytes + 8 + 4);
    const size_t meta = static_cast<size_t>(nw) * kMetaBytesPerWarp;
    if (fixed + meta >= static_cast<size_t>(kSmemBudget)) continue;
    const int stages = static_cast<int>((kSmemBudget - fixed - meta) / per_stage);
    if (stages >= 2) {
      pl->nwarps = nw;
      pl->stages = stages > PDA_ATTN_MAX_STAGES ? PDA_ATTN_MAX_STAGES : stages;
      break;
    }
  }
  if (pl->nwarps == 0) return false;
  size_t smem = fixed + static_cast<size_t>(pl->nwarps) * kMetaBytesPerWarp +
                static_cast<size_t>(pl->nwarps) * pl->stages * (pl->stage_bytes + 8 + 4);
  smem = round_up(smem, 128);
  if (smem < static_cast<size_t>(kMinResidentSmem)) smem = kMinResidentSmem;
  pl->smem_bytes = smem;
  int grid = num_sms;
  if (sm_cap > 0 && sm_cap < grid) grid = sm_cap;
  pl->grid = grid;
  const size_t nw_total = static_cast<size_t>(grid) * pl->nwarps;
  // Pool chunks pay off where the grid covers the whole chip: there SMs stream at unequal
  // rates (measured: whole runs of SMs about 10 % slower than the rest, at every workload),
  // while a capped grid leaves room around its SMs and runs evenly, so the chunks' extra
  // pieces and pipeline refills would cost more than they balance. The tensor-core steps
  // (quantised caches) process a tile in a fraction of the time and pay relatively more for
  // both; they keep the static split. A call claims at most NW k chunks plus one failed claim
  // per warp, within 16 bits.
  pl->pool_k = pool && t.mode == kModeCuda && grid == num_sms &&
                       nw_total * (PDA_POOL_CHUNKS_PER_WARP + 1) < 65536
                   ? PDA_POOL_CHUNKS_PER_WARP
                   : 0;
  const size_t units = nw_total * (1 + pl->pool_k);
  pl->ws_arrive = 0;
  pl->ws_claim = static_cast<size_t>(B) * t.H_u * 8;
  pl->ws_ml = round_up(pl->ws_claim + 8, 256);
  pl->ws_o = pl->ws_ml + round_up(2 * units * t.G_u * 2 * 4, 256);
  pl->ws_total = pl->ws_o + round_up(2 * units * t.G_u * static_cast<size_t>(D) * 4, 256);
  return true;
}

KernelFn pick_kernel(pda_dtype kv, int D, const Tiling& t, bool windowed) {
  if (windowed)
    return kv == PDA_FP8_E4M3 || kv == PDA_NVFP4 ? pick_window_codes_kernel(kv, D, t.G_u, t.mode)
                                                 : pick_window_kernel(kv, D, t.G_u, t.mode);
  switch (kv) {
    case PDA_F16: return pick_d<__half, __half, false>(D, t.G_u, t.mode);
    case PDA_BF16: return pick_d<__nv_bfloat16, __nv_bfloat16, false>(D, t.G_u, t.mode);
    case PDA_FP8_E4M3: return pick_d<fp8e4m3, __nv_bfloat16, false>(D, t.G_u, t.mode);
    case PDA_NVFP4: return pick_d<nvfp4, __nv_bfloat16, false>(D, t.G_u, t.mode);
    default: return pick_d<float, float, false>(D, t.G_u, t.mode);
  }
}

bool supported_g(int G) { return G == 1 || G == 2 || G == 4 || G == 8; }
// Physical blocks of 16, 32, ..., 256 tokens (a tile is 16 rows of one block).
bool supported_block_size(int bs) {
  return bs >= kBS && bs <= 16 * kBS && (bs & (bs - 1)) == 0;
}

// Numbers the calls, so a call recognises arrival counters left by earlier ones.
std::atomic<unsigned long long> g_call{1};

// Raises a kernel's dynamic shared-memory limit to the full budget once per device, so
// later calls (and calls made while a stream is being captured) skip the runtime call.
std::mutex g_attr_mu;
std::vector<std::pair<const void*, int>> g_attr_done;

pda_status allow_max_smem(const void* fn, int dev) {
  std::lock_guard<std::mutex> lock(g_attr_mu);
  for (const auto& e : g_attr_done)
    if (e.first == fn && e.second == dev) return PDA_OK;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget) !=
      cudaSuccess)
    return PDA_ERR_CUDA;
  g_attr_done.emplace_back(fn, dev);
  return PDA_OK;
}

// The last few encoded KV tensor maps, keyed by everything the encoding depends on.
struct MapKey {
  const void* base;
  int num_blocks, block_size, H_kv, D, dtype, swizzle;
  bool pair;
  bool operator==(const MapKey& o) const {
    return base == o.base && num_blocks == o.num_blocks && block_size == o.block_size &&
           H_kv == o.H_kv && D == o.D && dtype == o.dtype && swizzle == o.swizzle &&
           pair == o.pair;
  }
};
constexpr int kMapCache = 8;
std::mutex g_map_mu;
MapKey g_map_key[kMapCache];
CUtensorMap g_map_val[kMapCache];
int g_map_used = 0, g_map_next = 0;

// pair: the two-head map of encode_kv_pair_tensor_map (byte caches; D = row bytes).
pda_status cached_kv_tensor_map(CUtensorMap* tm, const void* base, int num_blocks,
                                int block_size, int H_kv, int D, pda_dtype dtype,
                                int swizzle_bytes, bool pair) {
  const MapKey key{base, num_blocks, block_size, H_kv, D, static_cast<int>(dtype),
                   swizzle_bytes, pair};
  {
    std::lock_guard<std::mutex> lock(g_map_mu);
    for (int i = 0; i < g_map_used; ++i)
      if (g_map_key[i] == key) {
        *tm = g_map_val[i];
        return PDA_OK;
      }
  }
  // boxes are one tile: kBS rows of one physical block (block_size is a multiple of kBS)
  const pda_status st =
      pair ? encode_kv_pair_tensor_map(tm, base, num_blocks, block_size, H_kv, D, swizzle_bytes,
                                       kBS)
           : encode_kv_tensor_map(tm, base, num_blocks, block_size, H_kv, D, dtype,
                                  swizzle_bytes, kBS);
  if (st != PDA_OK) return st;
  std::lock_guard<std::mutex> lock(g_map_mu);
  g_map_key[g_map_next] = key;
  g_map_val[g_map_next] = *tm;
  g_map_next = (g_map_next + 1) % kMapCache;
  if (g_map_used < kMapCache) ++g_map_used;
  return PDA_OK;
}

}  // namespace
}  // namespace pda

using namespace pda;

extern "C" pda_status pda_attention_workspace_size(int B, int H, int H_kv, int D, int block_size,
                                                   pda_dtype kv_dtype, int sm_cap,
                                                   size_t* bytes) {
  if (bytes == nullptr || B < 0 || H <= 0 || H_kv <= 0 || H % H_kv != 0 || D <= 0 ||
      block_size <= 0 || sm_cap < 0 || !(dtype_ok(kv_dtype) || kv_dtype == PDA_NVFP4))
    return PDA_ERR_INVALID_ARG;
  if (!supported_block_size(block_size) || (D != 64 && D != 128) || !supported_g(H / H_kv) ||
      B > kMaxBatch)
    return PDA_ERR_UNSUPPORTED;
  int dev, sms;
  const pda_status st = current_device_sms(&dev, &sms);
  if (st != PDA_OK) return st;
  LaunchPlan pl;
  if (!make_plan(B, H_kv, H / H_kv, D, kv_dtype, sm_cap, sms, true, false, &pl))
    return PDA_ERR_UNSUPPORTED;
  *bytes = pl.ws_total;
  return PDA_OK;
}

namespace pda {
namespace {

// The attention launch behind every public entry point. kv_dtype selects the cache format;
// k_scale and v_scale are the values of one stored unit of K and V (1 for plain caches).
pda_status launch_attention(void* out, const void* q, const void* k_cache, const void* v_cache,
                            const void* k_bscales, const void* v_bscales,
                            const int32_t* block_tables, int max_blocks_per_seq,
                            const int32_t* context_lens, int max_context_len, int B, int H,
                            int H_kv, int D, int block_size, int num_blocks, float scale,
                            float k_scale, float v_scale, pda_dtype q_dtype,
                            pda_dtype kv_dtype, pda_dtype out_dtype, int sm_cap,
                            void* workspace, size_t workspace_bytes, int32_t* error_word,
                            cudaStream_t stream, bool pool = true, bool clear_arrivals = false,
                            int window = 0, int sinks = 0) {
  // ---- host-side validation, before any CUDA call
  if (B < 0 || H <= 0 || H_kv <= 0 || H % H_kv != 0 || D <= 0 || block_size <= 0 ||
      num_blocks <= 0 || max_blocks_per_seq < 0 || max_context_len < 0 || sm_cap < 0 ||
      !float_dtype_ok(q_dtype) || !(dtype_ok(kv_dtype) || kv_dtype == PDA_NVFP4) ||
      !float_dtype_ok(out_dtype) ||
      !isfinite(scale) || !isfinite(k_scale) || !isfinite(v_scale))
    return PDA_ERR_INVALID_ARG;
  if (B == 0) return PDA_OK;
  if (out == nullptr || q == nullptr || k_cache == nullptr || v_cache == nullptr ||
      block_tables == nullptr || context_lens == nullptr)
    return PDA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PDA_ERR_INVALID_ARG;
  if (kv_dtype == PDA_NVFP4 && (k_bscales == nullptr || v_bscales == nullptr ||
                                !aligned16(k_bscales) || !aligned16(v_bscales)))
    return PDA_ERR_INVALID_ARG;
  const int G = H / H_kv;
  const bool quantised = kv_dtype == PDA_FP8_E4M3 || kv_dtype == PDA_NVFP4;
  const bool q_ok = quantised ? q_dtype == PDA_BF16 : q_dtype == kv_dtype;
  if (!supported_block_size(block_size) || (D != 64 && D != 128) || !supported_g(G) || !q_ok ||
      B > kMaxBatch)
    return PDA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_blocks) * block_size >= (1ll << 31) ||
      static_cast<long long>(B) * max_blocks_per_seq * H_kv >= (1ll << 31))
    return PDA_ERR_UNSUPPORTED;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return PDA_ERR_WORKSPACE;

  int dev, sms;
  pda_status st = current_device_sms(&dev, &sms);
  if (st != PDA_OK) return st;
  LaunchPlan pl;
  // a window no shorter than any history is none
  const long long capacity = static_cast<long long>(max_blocks_per_seq) * block_size;
  const bool windowed = window > 0 && window < std::min<long long>(max_context_len, capacity);
  if (!make_plan(B, H_kv, G, D, kv_dtype, sm_cap, sms, pool, windowed, &pl))
    return PDA_ERR_UNSUPPORTED;
  if (workspace_bytes < pl.ws_total) return PDA_ERR_WORKSPACE;

  const Tiling tiling = tiling_for(kv_dtype, D, H_kv, G);
  // No more blocks than give every warp PDA_MIN_TILES_PER_WARP tiles at the host's bound on
  // the lengths (every request at max_context_len); the kernel applies the same rule to the
  // lengths it reads. The workspace, sized for the full grid, is large enough for fewer
  // workers.
  {
    const long long max_len = std::min<long long>(max_context_len, capacity);
    long long per_row = (max_len + kBS - 1) / kBS;
    // a window that starts inside a tile takes one more
    if (windowed)
      per_row = std::min(per_row, (static_cast<long long>(sinks) + kBS - 1) / kBS +
                                      (static_cast<long long>(window) + kBS - 1) / kBS + 1);
    const long long tiles = static_cast<long long>(B) * tiling.H_u * per_row;
    const long long per_block = static_cast<long long>(pl.nwarps) *
                                (windowed ? kWindowMinTiles : PDA_MIN_TILES_PER_WARP);
    const long long blocks = (tiles + per_block - 1) / per_block;
    if (blocks < pl.grid) {
      pl.grid = static_cast<int>(std::max<long long>(1, blocks));
      pl.pool_k = 0;  // the pool is for the whole chip's grid
    }
  }
  KernelFn fn = pick_kernel(kv_dtype, D, tiling, windowed);
  if (fn == nullptr) return PDA_ERR_UNSUPPORTED;
  st = allow_max_smem(reinterpret_cast<const void*>(fn), dev);
  if (st != PDA_OK) return st;

  // the TMA sees an NVFP4 row as D/2 bytes; the tensor-core step reads swizzled tiles whose
  // swizzle span is one whole row (128 bytes FP8, 64 bytes NVFP4)
  const int row_elems = kv_dtype == PDA_NVFP4 ? D / 2 : D;
  const pda_dtype map_type = kv_dtype == PDA_NVFP4 ? PDA_FP8_E4M3 : kv_dtype;
  const int swizzle = tiling.mode != kModeCuda ? row_elems : 0;
  const bool pair = tiling.mode == kModeTcPair;
  CUtensorMap tmK, tmV;
  st = cached_kv_tensor_map(&tmK, k_cache, num_blocks, block_size, H_kv, row_elems, map_type,
                            swizzle, pair);
  if (st != PDA_OK) return st;
  st = cached_kv_tensor_map(&tmV, v_cache, num_blocks, block_size, H_kv, row_elems, map_type,
                            swizzle, pair);
  if (st != PDA_OK) return st;

  unsigned char* ws = static_cast<unsigned char*>(workspace);
  AttnParams ap;
  ap.out = out;
  ap.q = q;
  ap.block_tables = block_tables;
  ap.context_lens = context_lens;
  ap.ws_arrive = reinterpret_cast<unsigned long long*>(ws + pl.ws_arrive);
  ap.ws_claim = reinterpret_cast<unsigned long long*>(ws + pl.ws_claim);
  ap.pool_k = pl.pool_k;
  ap.call = g_call.fetch_add(1, std::memory_order_relaxed) & ((1ull << 48) - 1);
  ap.ws_ml = reinterpret_cast<float*>(ws + pl.ws_ml);
  ap.ws_o = reinterpret_cast<float*>(ws + pl.ws_o);
  ap.error_word = error_word;
  ap.v_scale = v_scale;
  ap.k_bscales = static_cast<const uint8_t*>(k_bscales);
  ap.v_bscales = static_cast<const uint8_t*>(v_bscales);
  ap.B = B;
  ap.H = H;
  ap.H_kv = tiling.H_u;  // units: kv-heads, or pairs of them
  ap.num_blocks = num_blocks;
  ap.max_blocks = max_blocks_per_seq;
  ap.max_context_len = max_context_len;
  ap.window = window;
  ap.sinks = sinks;
  ap.block_size = block_size;
  ap.bs_shift = 0;
  while ((kBS << ap.bs_shift) < block_size) ++ap.bs_shift;
  ap.out_kind = out_dtype == PDA_BF16 ? kOutBF16 : out_dtype == PDA_F16 ? kOutF16 : kOutF32;
  // the K scale folds into q's pre-scale: s = scale * (k_scale * code) . q
  ap.scale_log2 = scale * k_scale * 1.4426950408889634f;
  ap.num_workers = pl.grid * pl.nwarps;
  ap.stages = pl.stages;
  ap.stage_bytes = pl.stage_bytes;
  ap.prefix_bytes = pl.prefix_bytes;

  // clear_arrivals: zero the arrival counters first (a memset on the same stream), so no
  // counter left in the workspace by an earlier call can pass for one of this call's
  if (clear_arrivals && cudaMemsetAsync(ap.ws_arrive, 0, pl.ws_claim + 8, stream) != cudaSuccess)
    return PDA_ERR_CUDA;
  fn<<<pl.grid, pl.nwarps * 32, pl.smem_bytes, stream>>>(tmK, tmV, ap);
  if (cudaGetLastError() != cudaSuccess) return PDA_ERR_CUDA;
  return PDA_OK;
}

}  // namespace
}  // namespace pda

extern "C" pda_status pda_paged_decode_attention(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
    int max_context_len, int B, int H, int H_kv, int D, int block_size, int num_blocks,
    float scale, pda_dtype q_dtype, pda_dtype kv_dtype, pda_dtype out_dtype, int sm_cap,
    void* workspace, size_t workspace_bytes, int32_t* error_word, cudaStream_t stream) {
  if (kv_dtype == PDA_FP8_E4M3) return PDA_ERR_UNSUPPORTED;  // needs its scales: _fp8 entry
  return launch_attention(out, q, k_cache, v_cache, nullptr, nullptr, block_tables,
                          max_blocks_per_seq, context_lens, max_context_len, B, H, H_kv, D,
                          block_size, num_blocks, scale, 1.f, 1.f, q_dtype, kv_dtype, out_dtype,
                          sm_cap, workspace, workspace_bytes, error_word, stream);
}

extern "C" pda_status pda_paged_decode_attention_fp8(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
    int max_context_len, int B, int H, int H_kv, int D, int block_size, int num_blocks,
    float scale, float k_scale, float v_scale, pda_dtype q_dtype, pda_dtype out_dtype,
    int sm_cap, void* workspace, size_t workspace_bytes, int32_t* error_word,
    cudaStream_t stream) {
  return launch_attention(out, q, k_cache, v_cache, nullptr, nullptr, block_tables,
                          max_blocks_per_seq, context_lens, max_context_len, B, H, H_kv, D,
                          block_size, num_blocks, scale, k_scale, v_scale, q_dtype,
                          PDA_FP8_E4M3, out_dtype, sm_cap, workspace, workspace_bytes,
                          error_word, stream);
}

extern "C" pda_status pda_paged_decode_attention_nvfp4(
    void* out, const void* q, const void* k_data, const void* v_data,
    const void* k_block_scales, const void* v_block_scales, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* context_lens, int max_context_len, int B, int H,
    int H_kv, int D, int block_size, int num_blocks, float scale, float k_scale, float v_scale,
    pda_dtype q_dtype, pda_dtype out_dtype, int sm_cap, void* workspace,
    size_t workspace_bytes, int32_t* error_word, cudaStream_t stream) {
  return launch_attention(out, q, k_data, v_data, k_block_scales, v_block_scales,
                          block_tables, max_blocks_per_seq, context_lens, max_context_len, B, H,
                          H_kv, D, block_size, num_blocks, scale, k_scale, v_scale, q_dtype,
                          PDA_NVFP4, out_dtype, sm_cap, workspace, workspace_bytes, error_word,
                          stream);
}

extern "C" pda_status pda_paged_window_attention(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const void* k_block_scales, const void* v_block_scales, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* context_lens, int max_context_len, int window,
    int sinks, int B, int H, int H_kv, int D, int block_size, int num_blocks, float scale,
    float k_scale, float v_scale, pda_dtype q_dtype, pda_dtype kv_dtype, pda_dtype out_dtype,
    int sm_cap, void* workspace, size_t workspace_bytes, int32_t* error_word,
    cudaStream_t stream) {
  if (window < 1 || sinks < 0) return PDA_ERR_INVALID_ARG;
  return launch_attention(out, q, k_cache, v_cache, k_block_scales, v_block_scales, block_tables,
                          max_blocks_per_seq, context_lens, max_context_len, B, H, H_kv, D,
                          block_size, num_blocks, scale, k_scale, v_scale, q_dtype, kv_dtype,
                          out_dtype, sm_cap, workspace, workspace_bytes, error_word, stream,
                          /*pool=*/true, /*clear_arrivals=*/false, window, sinks);
}

// ------------------------------------------------------------------ no-allocation variant
// Scratch for pda_paged_decode_attention_noalloc: a fixed device array in this module, for
// callers that may not allocate device memory while they run: a plugin whose host
// framework owns all device memory and hands it only inputs and outputs, or a serving loop
// that forbids allocation once it has started. Host code must not pass `g_noalloc_scratch`
// itself to a kernel (on the host it names a host-side shadow, not device memory); it
// passes the address cudaGetSymbolAddress returns for the current device.
static __device__ __align__(256) unsigned char g_noalloc_scratch[PDA_NOALLOC_SCRATCH_BYTES];

namespace {
constexpr int kNoallocMaxDevices = 64;
std::atomic<void*> g_noalloc_ptr[kNoallocMaxDevices];
std::mutex g_noalloc_mu;

// Device address of the scratch array on `dev` (the current device), looked up once.
pda_status noalloc_scratch(int dev, void** ptr) {
  if (dev < 0 || dev >= kNoallocMaxDevices) return PDA_ERR_UNSUPPORTED;
  void* p = g_noalloc_ptr[dev].load(std::memory_order_acquire);
  if (p == nullptr) {
    std::lock_guard<std::mutex> lock(g_noalloc_mu);
    p = g_noalloc_ptr[dev].load(std::memory_order_acquire);
    if (p == nullptr) {
      if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || p == nullptr)
        return PDA_ERR_CUDA;
      g_noalloc_ptr[dev].store(p, std::memory_order_release);
    }
  }
  *ptr = p;
  return PDA_OK;
}
}  // namespace

extern "C" pda_status pda_paged_decode_attention_noalloc(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
    int max_context_len, int B, int H, int H_kv, int D, int block_size, int num_blocks,
    float scale, pda_dtype q_dtype, pda_dtype kv_dtype, pda_dtype out_dtype, int sm_cap,
    int32_t* error_word, cudaStream_t stream) {
  if (kv_dtype == PDA_FP8_E4M3) return PDA_ERR_UNSUPPORTED;  // as pda_paged_decode_attention
  // The same checks as pda_attention_workspace_size, for the all-static split (no pool of
  // claimed chunks, whose piece slots would not fit the fixed array).
  if (B < 0 || H <= 0 || H_kv <= 0 || H % H_kv != 0 || D <= 0 || block_size <= 0 ||
      sm_cap < 0 || !(dtype_ok(kv_dtype) || kv_dtype == PDA_NVFP4))
    return PDA_ERR_INVALID_ARG;
  if (!supported_block_size(block_size) || (D != 64 && D != 128) || !supported_g(H / H_kv) ||
      B > kMaxBatch)
    return PDA_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  pda_status st = current_device_sms(&dev, &sms);
  if (st != PDA_OK) return st;
  LaunchPlan pl;
  if (!make_plan(B, H_kv, H / H_kv, D, kv_dtype, sm_cap, sms, false, false, &pl))
    return PDA_ERR_UNSUPPORTED;
  if (pl.ws_total > PDA_NOALLOC_SCRATCH_BYTES) return PDA_ERR_TOO_LARGE;
  void* scratch = nullptr;
  st = noalloc_scratch(dev, &scratch);
  if (st != PDA_OK) return st;
  // The shared array keeps whatever the previous call left, which may be a call of another
  // shape or one that timed out: its counters are cleared before the kernel runs.
  return launch_attention(out, q, k_cache, v_cache, nullptr, nullptr, block_tables,
                          max_blocks_per_seq, context_lens, max_context_len, B, H, H_kv, D,
                          block_size, num_blocks, scale, 1.f, 1.f, q_dtype, kv_dtype, out_dtype,
                          sm_cap, scratch, PDA_NOALLOC_SCRATCH_BYTES, error_word, stream,
                          /*pool=*/false, /*clear_arrivals=*/true);
}
