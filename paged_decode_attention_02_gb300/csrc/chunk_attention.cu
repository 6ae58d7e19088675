// chunk_attention.cu -- the C entry points of chunk attention: attention of a chunk of new
// tokens over the paged cache, every new token of a request attending to the request's whole
// history up to and including itself.
//
// Row (token i of request b, head h) at position p = L_b - n_b + i, kv-head k = h / G:
//   s_t = scale q . K_t[k],  out = sum_{t <= p} softmax(s)_t V_t[k],
// with a sliding window over t > p - window or t < sinks alone.
// Checks the arguments and hands over to the kernel of the cache's type.
#include <math.h>

#include "chunk_internal.h"
#include "chunk_plan.cuh"

namespace pda {

size_t chunk_workspace(int sms, int D) {
  return static_cast<size_t>(sms) * 2 * part_floats(D) * sizeof(float);
}

namespace {

constexpr int kChunkMaxBatch = 8192;

bool chunk_block_size_ok(int bs) { return bs >= 16 && bs <= 256 && (bs & (bs - 1)) == 0; }
bool chunk_group_ok(int G) { return G == 1 || G == 2 || G == 4 || G == 8; }

pda_status check_shape(int B, int T, int H, int H_kv, int D, int block_size, pda_dtype kv_dtype,
                       int sm_cap) {
  if (B < 0 || T < 0 || H <= 0 || H_kv <= 0 || H % H_kv != 0 || D <= 0 || block_size <= 0 ||
      sm_cap < 0 || !dtype_ok(kv_dtype))
    return PDA_ERR_INVALID_ARG;
  if (!chunk_block_size_ok(block_size) || (D != 64 && D != 128) || !chunk_group_ok(H / H_kv) ||
      B > kChunkMaxBatch || static_cast<long long>(T) * H >= (1ll << 31))
    return PDA_ERR_UNSUPPORTED;
  return PDA_OK;
}

// The launch behind the public entry points.
pda_status launch_chunk(void* out, const void* q, const void* k_cache, const void* v_cache,
                        const int32_t* block_tables, int max_blocks_per_seq,
                        const int32_t* context_lens, const int32_t* query_start,
                        int max_context_len, int B, int T, int H, int H_kv, int D, int block_size,
                        int num_blocks, float scale, float k_scale, float v_scale,
                        pda_dtype q_dtype, pda_dtype kv_dtype, int sm_cap, void* workspace,
                        size_t workspace_bytes, int32_t* error_word, cudaStream_t stream,
                        int window = 0, int sinks = 0) {
  const pda_status st = check_shape(B, T, H, H_kv, D, block_size, kv_dtype, sm_cap);
  if (st == PDA_ERR_INVALID_ARG || num_blocks <= 0 || max_blocks_per_seq < 0 ||
      max_context_len < 0 || !float_dtype_ok(q_dtype) || !isfinite(scale) || !isfinite(k_scale) ||
      !isfinite(v_scale))
    return PDA_ERR_INVALID_ARG;
  if (st != PDA_OK) return st;
  if (B == 0 || T == 0) return PDA_OK;
  if (out == nullptr || q == nullptr || k_cache == nullptr || v_cache == nullptr ||
      block_tables == nullptr || context_lens == nullptr || query_start == nullptr)
    return PDA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PDA_ERR_INVALID_ARG;
  if (q_dtype != (kv_dtype == PDA_FP8_E4M3 ? PDA_BF16 : kv_dtype)) return PDA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_blocks) * block_size >= (1ll << 31) ||
      static_cast<long long>(B) * max_blocks_per_seq >= (1ll << 31))
    return PDA_ERR_UNSUPPORTED;
  ChunkParams p{out,          q,            k_cache,     v_cache,
                block_tables, context_lens, query_start, error_word,
                scale * k_scale * 1.4426950408889634f,
                v_scale,      B,            T,           H,
                H_kv,         H / H_kv,     max_blocks_per_seq, max_context_len,
                block_size,   num_blocks,   0,           0,
                0};
  // a window no shorter than any history is none
  if (window > 0 && window < std::min<long long>(max_context_len, static_cast<long long>(
                                                     max_blocks_per_seq) * block_size)) {
    p.window = window;
    p.sinks = sinks;
    p.sink_tiles = std::min(sinks / kChunkKeys + (sinks % kChunkKeys != 0), chunk_tiles(p));
  }
  // the kernels number keys in 31 bits with a tile to spare, and their work, items by key
  // tiles, in 31 bits
  if (chunk_tiles(p) > (1 << 23)) return PDA_ERR_UNSUPPORTED;
  int g_shift = 0;
  while ((1 << g_shift) < p.G) ++g_shift;
  const long long units = kv_dtype == PDA_F32 ? chunk_units<Cuts<6, 1, 1>>(p, g_shift)
                                              : chunk_units<Cuts<8, 1, 1>>(p, g_shift);
  if (units >= (1ll << 31)) return PDA_ERR_UNSUPPORTED;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return PDA_ERR_WORKSPACE;
  int dev, sms;
  const pda_status dst = current_device_sms(&dev, &sms);
  if (dst != PDA_OK) return dst;
  const bool capped = sm_cap > 0 && sm_cap < sms;
  if (capped) sms = sm_cap;
  if (workspace_bytes < chunk_workspace(sms, D)) return PDA_ERR_WORKSPACE;
  if (kv_dtype == PDA_F32) return launch_chunk_f32(p, D, dev, sms, capped, workspace, stream);
  return (p.window > 0 ? launch_chunk_window_tc : launch_chunk_tc)(p, D, kv_dtype, dev, sms, capped,
                                                                   workspace, stream);
}

}  // namespace
}  // namespace pda

using namespace pda;

extern "C" pda_status pda_chunk_attention_workspace_size(int B, int T, int H, int H_kv, int D,
                                                         int block_size, pda_dtype kv_dtype,
                                                         int sm_cap, size_t* bytes) {
  if (bytes == nullptr) return PDA_ERR_INVALID_ARG;
  const pda_status st = check_shape(B, T, H, H_kv, D, block_size, kv_dtype, sm_cap);
  if (st != PDA_OK) return st;
  int dev, sms;
  const pda_status dst = current_device_sms(&dev, &sms);
  if (dst != PDA_OK) return dst;
  *bytes = chunk_workspace(sm_cap > 0 && sm_cap < sms ? sm_cap : sms, D);
  return PDA_OK;
}

extern "C" pda_status pda_paged_chunk_attention(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
    const int32_t* query_start, int max_context_len, int B, int T, int H, int H_kv, int D,
    int block_size, int num_blocks, float scale, pda_dtype q_dtype, pda_dtype kv_dtype,
    int sm_cap, void* workspace, size_t workspace_bytes, int32_t* error_word,
    cudaStream_t stream) {
  if (kv_dtype == PDA_FP8_E4M3) return PDA_ERR_UNSUPPORTED;  // needs its scales: _fp8 entry
  return launch_chunk(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                      query_start, max_context_len, B, T, H, H_kv, D, block_size, num_blocks,
                      scale, 1.f, 1.f, q_dtype, kv_dtype, sm_cap, workspace, workspace_bytes,
                      error_word, stream);
}

extern "C" pda_status pda_paged_chunk_attention_fp8(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
    const int32_t* query_start, int max_context_len, int B, int T, int H, int H_kv, int D,
    int block_size, int num_blocks, float scale, float k_scale, float v_scale, pda_dtype q_dtype,
    int sm_cap, void* workspace, size_t workspace_bytes, int32_t* error_word,
    cudaStream_t stream) {
  return launch_chunk(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                      query_start, max_context_len, B, T, H, H_kv, D, block_size, num_blocks,
                      scale, k_scale, v_scale, q_dtype, PDA_FP8_E4M3, sm_cap, workspace,
                      workspace_bytes, error_word, stream);
}

extern "C" pda_status pda_paged_window_chunk_attention(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
    const int32_t* query_start, int max_context_len, int window, int sinks, int B, int T, int H,
    int H_kv, int D, int block_size, int num_blocks, float scale, float k_scale, float v_scale,
    pda_dtype q_dtype, pda_dtype kv_dtype, int sm_cap, void* workspace, size_t workspace_bytes,
    int32_t* error_word, cudaStream_t stream) {
  if (window < 1 || sinks < 0) return PDA_ERR_INVALID_ARG;
  return launch_chunk(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                      query_start, max_context_len, B, T, H, H_kv, D, block_size, num_blocks,
                      scale, k_scale, v_scale, q_dtype, kv_dtype, sm_cap, workspace,
                      workspace_bytes, error_word, stream, window, sinks);
}
