// chunk_attention.cu -- attention of a chunk of new tokens over the paged cache: every new
// token of a request attends to the request's whole history up to and including itself.
//
// Row (token i of request b, head h) at position p = L_b - n_b + i, kv-head k = h / G:
//   s_t = scale q . K_t[k],  out = sum_{t <= p} softmax(s)_t V_t[k].
// One warp per row: lanes own D / 32 dims, keys stream past one at a time with a running
// maximum and sum in fp32.
#include <math.h>

#include "chunk_internal.h"
#include "pda_device.cuh"

namespace pda {
namespace {

constexpr int kChunkMaxBatch = 8192;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(fp8e4m3 x) { return e4m3_to_f32(x.bits); }
__device__ __forceinline__ void from_f32(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename KV, typename Q, int D>
__global__ void __launch_bounds__(256) chunk_rows_kernel(const ChunkParams p) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = blockIdx.x * 8ll + (threadIdx.x >> 5);
  if (w >= static_cast<long long>(p.T) * p.H) return;
  const int tok = static_cast<int>(w / p.H), h = static_cast<int>(w % p.H), kh = h / p.G;
  // the request whose rows hold tok: the last b with query_start[b] <= tok
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.query_start[mid] <= tok)
      lo = mid;
    else
      hi = mid;
  }
  const int q0 = p.query_start[lo], q1 = p.query_start[lo + 1];
  if (q0 < 0 || q1 > p.T || q0 > q1) {
    if (lane == 0) atomic_or_error(p.error_word, PDA_DEVERR_QUERY);
    return;
  }
  if (tok < q0 || tok >= q1) return;
  const int L = p.context_lens[lo], n = q1 - q0;
  const bool bad_len = L < 0 || L > p.max_context_len ||
                       L > static_cast<long long>(p.max_blocks) * p.block_size ||
                       (L > 0 && L < n);
  if (bad_len && lane == 0) atomic_or_error(p.error_word, PDA_DEVERR_CONTEXT_LEN);
  const size_t row = (static_cast<size_t>(tok) * p.H + h) * D + lane * V;
  float q[V], o[V], m = -INFINITY, l = 0.f;
  for (int i = 0; i < V; ++i) {
    q[i] = to_f32(static_cast<const Q*>(p.q)[row + i]) * p.scale_log2;
    o[i] = 0.f;
  }
  const int keys = bad_len || L == 0 ? 0 : L - n + (tok - q0) + 1;
  bool bad_block = false;
  const int32_t* table = p.block_tables + static_cast<size_t>(lo) * p.max_blocks;
  for (int t = 0; t < keys; ++t) {
    const int id = table[t / p.block_size];
    if (id < 0 || id >= p.num_blocks) {
      bad_block = true;
      break;
    }
    const size_t at =
        ((static_cast<size_t>(id) * p.block_size + t % p.block_size) * p.H_kv + kh) * D + lane * V;
    float s = 0.f;
    for (int i = 0; i < V; ++i) s = fmaf(q[i], to_f32(static_cast<const KV*>(p.k_cache)[at + i]), s);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(kFullMask, s, x);
    const float m1 = fmaxf(m, s);
    const float c = ex2(m - m1), e = ex2(s - m1);
    l = l * c + e;
    for (int i = 0; i < V; ++i)
      o[i] = fmaf(e, to_f32(static_cast<const KV*>(p.v_cache)[at + i]), o[i] * c);
    m = m1;
  }
  if (bad_block && lane == 0) atomic_or_error(p.error_word, PDA_DEVERR_BLOCK_ID);
  const float inv = bad_len || bad_block ? NAN : keys == 0 ? 0.f : p.v_scale / l;
  for (int i = 0; i < V; ++i) from_f32(static_cast<Q*>(p.out) + row + i, o[i] * inv);
}

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

template <typename KV, typename Q>
void launch_rows(const ChunkParams& p, int D, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.T) * p.H + 7) / 8);
  if (D == 128)
    chunk_rows_kernel<KV, Q, 128><<<grid, 256, 0, stream>>>(p);
  else
    chunk_rows_kernel<KV, Q, 64><<<grid, 256, 0, stream>>>(p);
}

size_t workspace_for(pda_dtype kv_dtype, int D, int sms) {
  const size_t n = kv_dtype != PDA_F32 ? chunk_tc_workspace(sms, D) : 0;
  return n < 256 ? 256 : n;
}

// The launch behind both public entry points.
pda_status launch_chunk(void* out, const void* q, const void* k_cache, const void* v_cache,
                        const int32_t* block_tables, int max_blocks_per_seq,
                        const int32_t* context_lens, const int32_t* query_start,
                        int max_context_len, int B, int T, int H, int H_kv, int D, int block_size,
                        int num_blocks, float scale, float k_scale, float v_scale,
                        pda_dtype q_dtype, pda_dtype kv_dtype, int sm_cap, void* workspace,
                        size_t workspace_bytes, int32_t* error_word, cudaStream_t stream) {
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
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return PDA_ERR_WORKSPACE;
  int dev, sms;
  const pda_status dst = current_device_sms(&dev, &sms);
  if (dst != PDA_OK) return dst;
  if (sm_cap > 0 && sm_cap < sms) sms = sm_cap;
  if (workspace_bytes < workspace_for(kv_dtype, D, sms)) return PDA_ERR_WORKSPACE;
  const ChunkParams p{out,     q,      k_cache,   v_cache,
                      block_tables, context_lens, query_start, error_word,
                      scale * k_scale * 1.4426950408889634f,
                      v_scale, B,      T,         H,
                      H_kv,    H / H_kv, max_blocks_per_seq, max_context_len,
                      block_size, num_blocks};
  if (kv_dtype != PDA_F32) return launch_chunk_tc(p, D, kv_dtype, dev, sms, workspace, stream);
  launch_rows<float, float>(p, D, stream);
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
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
  *bytes = workspace_for(kv_dtype, D, sm_cap > 0 && sm_cap < sms ? sm_cap : sms);
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
