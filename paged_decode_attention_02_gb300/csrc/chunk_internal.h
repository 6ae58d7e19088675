// chunk_internal.h -- what the translation units of chunk attention share.
#pragma once

#include "pda_internal.h"

namespace pda {

struct ChunkParams {
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  int32_t* error_word;
  float scale_log2;  // softmax scale times log2 e (and the cache's K scale)
  float v_scale;
  int B, T, H, H_kv, G, max_blocks, max_context_len, block_size, num_blocks;
  // sliding window (window 0: none): a token sees the last `window` keys up to itself and the
  // first `sinks`, which lie in sink_tiles key tiles
  int window, sinks, sink_tiles;
};

// Workspace bytes on `sms` SMs: two cut items' partial results a block.
size_t chunk_workspace(int sms, int D);

// 16-bit and FP8 caches, on the tensor cores. No kernel of the call has more than `sms` blocks
// where it is `capped` to them.
pda_status launch_chunk_tc(const ChunkParams& p, int D, pda_dtype kv_dtype, int dev, int sms,
                           bool capped, void* workspace, cudaStream_t stream);
// The same with a sliding window, compiled in a unit of its own.
pda_status launch_chunk_window_tc(const ChunkParams& p, int D, pda_dtype kv_dtype, int dev,
                                  int sms, bool capped, void* workspace, cudaStream_t stream);
// fp32 caches.
pda_status launch_chunk_f32(const ChunkParams& p, int D, int dev, int sms, bool capped,
                            void* workspace, cudaStream_t stream);

}  // namespace pda
