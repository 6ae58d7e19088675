/*
 * pda.h -- C ABI of the paged decode-attention library for GB300 (sm_103a).
 *
 * The library implements the data-parallel hot path of one decode step over a paged KV
 * cache: the append of each request's new K/V, the attention of each request's single
 * query token over its whole cached history, and the gather of one request's scattered
 * KV blocks into a contiguous buffer for transfer. For the step that comes before it, the
 * new tokens of prompts, prompt chunks or drafts, it holds the attention of a chunk over the
 * same cache and the block tables and slots built on the GPU from the requests' lengths; for
 * windowed models and drafted tokens, the same attention with a sliding window, the norm and
 * rotation of queries and keys on their way into the cache, and the verification of drafts.
 *
 * Conventions shared by every entry point:
 *  - Every pointer argument is a DEVICE pointer unless its comment says "host". The caller
 *    owns all memory; the library allocates nothing. Apart from the fixed scratch array of
 *    pda_paged_decode_attention_noalloc it keeps no state between calls.
 *  - Tensors are dense and row-major with exactly the shapes given; strides only where a call
 *    takes them.
 *  - KV caches are [num_blocks, block_size, H_kv, D]: physical block p holds block_size
 *    consecutive tokens, token row r of block p is at ((p * block_size + r) * H_kv) * D.
 *    (Page "From PagedAttention to Prefill-Decode disaggregation", sec. 2.2 step 1: the
 *    cache is cut into fixed-size physical blocks, each holding the K and V of a fixed
 *    number of tokens.)
 *  - block_tables is [B, max_blocks_per_seq] int32: logical block i of request b is
 *    physical block block_tables[b * max_blocks_per_seq + i]; blocks need not be
 *    contiguous or ordered, and several requests may share blocks (same page, sec. 2.2
 *    step 2 and sec. 2.3). Entries past a request's last block are never read.
 *  - Query head h reads kv-head h / (H / H_kv) (grouped-query attention, contiguous groups).
 *  - Every call is asynchronous on `stream`, never synchronises the host and allocates no
 *    device memory. A sequence of the calls other than pda_paged_decode_attention_noalloc
 *    can be captured in a CUDA graph once each kernel has been launched outside capture.
 *  - Host-checkable errors (null pointers, bad sizes, unsupported dtypes or shapes,
 *    misaligned pointers) return a status before anything is launched. Errors in device
 *    data (a block id or slot out of range, a context length beyond capacity) cannot be
 *    seen on the host without a sync; kernels OR a PDA_DEVERR_* bit into *error_word
 *    (when error_word is not NULL) and never trap. The caller zeroes the error word and
 *    reads it back whenever it chooses to synchronise.
 */
#ifndef PDA_H
#define PDA_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PDA_OK = 0,
  PDA_ERR_INVALID_ARG = 1, /* null pointer, negative or inconsistent size, misalignment */
  PDA_ERR_UNSUPPORTED = 2, /* a valid request the library does not implement */
  PDA_ERR_CUDA = 3,        /* a CUDA runtime call failed; see cudaGetLastError */
  PDA_ERR_WORKSPACE = 4,   /* workspace missing or smaller than required */
  PDA_ERR_TOO_LARGE = 5    /* needs more scratch than pda_paged_decode_attention_noalloc has */
} pda_status;

/* Element types. PDA_F32, PDA_BF16 and PDA_F16 (IEEE binary16, the precision the pages'
 * decode kernels were measured in) are q, output and KV-cache types. PDA_FP8_E4M3 (the OCP
 * 8-bit format without infinities) is a KV-cache type only: append, pack and unpack copy
 * its bytes, and pda_paged_decode_attention_fp8 reads it with per-tensor scales. PDA_NVFP4
 * names the 4-bit cache read by pda_paged_decode_attention_nvfp4 (and sizes its workspace);
 * its data tensors are moved as 1-byte rows by append, pack and unpack, its block scales by
 * the *_block_scales calls. */
typedef enum {
  PDA_F32 = 0,
  PDA_BF16 = 1,
  PDA_FP8_E4M3 = 2,
  PDA_NVFP4 = 3,
  PDA_F16 = 4
} pda_dtype;

/* Bits OR-ed into *error_word by the kernels. */
#define PDA_DEVERR_CONTEXT_LEN 0x1 /* context_lens[b] < 0, > max_context_len or > table capacity */
#define PDA_DEVERR_BLOCK_ID 0x2    /* a block id needed by a request is outside [0, num_blocks) */
#define PDA_DEVERR_SLOT 0x4        /* slot_mapping[b] >= num_blocks * block_size */
#define PDA_DEVERR_TIMEOUT 0x8     /* a pipeline wait passed its time limit; results invalid */
#define PDA_DEVERR_QUERY 0x10      /* query_lens / query_start negative, decreasing or beyond T */
#define PDA_DEVERR_NO_BLOCKS 0x20  /* free_count out of range, or too few free blocks */
#define PDA_DEVERR_TOKEN 0x40      /* a drafted token outside [0, V) */
#define PDA_DEVERR_PROBS 0x80      /* a row to draw from has no positive, finite weight */

/* Bytes of the fixed device scratch behind pda_paged_decode_attention_noalloc. */
#define PDA_NOALLOC_SCRATCH_BYTES (8u << 20)

/* Most requests one batched pack or unpack call takes. */
#define PDA_PACK_MAX_BATCH 64

/* Most layers one pda_kv_pack_layers / pda_kv_unpack_layers call takes. */
#define PDA_PACK_MAX_LAYERS 256

/* Human-readable name of a status. Never NULL. */
const char* pda_status_string(pda_status status);

/* ABI version of this library (incremented on incompatible change). */
int pda_version(void);

/* Number of SMs of the current device, written to *num_sms (host). */
pda_status pda_device_sm_count(int* num_sms);

/*
 * pda_kv_append -- write each request's new token into the paged cache.
 *
 * Defined by the decode step of page "Disaggregated LLM Serving: from PD disaggregation to
 * attention offload", sec. 1 (second list, item 2): every decode step reads the cached
 * history and appends the new token's K/V; the slot comes from the block table (page "From
 * PagedAttention to Prefill-Decode disaggregation", sec. 2.2 step 3: blocks are handed out
 * as tokens arrive).
 *
 *  k_new, v_new   [B, H_kv, D] in kv_dtype: this step's K and V of each request.
 *  k_cache,v_cache [num_blocks, block_size, H_kv, D] in kv_dtype, updated in place.
 *  slot_mapping   [B] int32: flat slot s = block * block_size + row for request b. s < 0
 *                 means "no token" (padding) and is skipped; s >= num_blocks * block_size
 *                 sets PDA_DEVERR_SLOT and is skipped.
 *  The copy is bitwise. Two requests given the same slot race; the caller must not do so.
 *  Requires H_kv * D * sizeof(kv_dtype) to be a multiple of 16 bytes and 16-byte aligned
 *  pointers. B == 0 is a no-op.
 */
pda_status pda_kv_append(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                         const int32_t* slot_mapping, int B, int H_kv, int D, int block_size,
                         int num_blocks, pda_dtype kv_dtype, int32_t* error_word,
                         cudaStream_t stream);

/*
 * pda_attention_workspace_size -- bytes of device workspace pda_paged_decode_attention
 * needs on the current device for these sizes. The bound does not depend on the context
 * lengths. Written to *bytes (host).
 */
pda_status pda_attention_workspace_size(int B, int H, int H_kv, int D, int block_size,
                                        pda_dtype kv_dtype, int sm_cap, size_t* bytes);

/*
 * pda_paged_decode_attention -- one query token per head attends over its request's whole
 * cached history, read through the block table.
 *
 * Defined by: decode reads the request's whole KV history each step (page "Disaggregated
 * LLM Serving", sec. 1, and sec. 6.1 on why this is memory-bound); the history lives in
 * fixed-size blocks reached through a per-request table (page "From PagedAttention to
 * Prefill-Decode disaggregation", sec. 2.2). For each request b and query head h with
 * kv-head k = h / (H / H_kv) and L = context_lens[b]:
 *      s_t = scale * q[b,h,:] . K_t[k,:],   t < L
 *      out[b,h,:] = sum_t softmax(s)_t * V_t[k,:]
 * The work is split per request and kv-head and, for long histories, along the sequence;
 * the pieces are merged with a log-sum-exp combine (the per-request split and merge of
 * Orca's iteration-level batching, page "Disaggregated LLM Serving", sec. 2.1, applied
 * also along the sequence). Accumulation is fp32.
 *
 *  out            [B, H, D] in out_dtype (PDA_F32, PDA_BF16 or PDA_F16).
 *  q              [B, H, D] in q_dtype; q_dtype must equal kv_dtype.
 *  k_cache,v_cache [num_blocks, block_size, H_kv, D] in kv_dtype (PDA_F32, PDA_BF16 or
 *                 PDA_F16; an FP8 cache goes through pda_paged_decode_attention_fp8); read
 *                 only.
 *  block_tables   [B, max_blocks_per_seq] int32.
 *  context_lens   [B] int32 (device): tokens of history including this step's token.
 *                 L == 0 gives a zero row. L < 0, L > max_context_len or
 *                 L > max_blocks_per_seq * block_size gives NaN rows and
 *                 PDA_DEVERR_CONTEXT_LEN. A block id out of range gives NaN rows for
 *                 that (request, kv-head group) and PDA_DEVERR_BLOCK_ID.
 *  max_context_len host upper bound of context_lens (validation only).
 *  scale          softmax scale, usually 1/sqrt(D).
 *  sm_cap         0 runs on every SM; n > 0 confines the kernel to at most n SMs (one
 *                 resident block per SM, a persistent grid walks the work). This models
 *                 attention sharing the GPU with other work on a fraction of its SMs
 *                 (review of "Injecting Adrenaline into LLM Serving", sec. 3.3).
 *  workspace      device scratch of at least pda_attention_workspace_size(...) bytes,
 *                 256-byte aligned; not shared by calls that may run concurrently. No
 *                 initialisation is needed: its arrival counters are tagged with a number
 *                 the library gives each call, mixed with a fixed 48-bit pattern so that
 *                 what another call left there (zeros, or the fp32 partial results of a call
 *                 of another shape) is not taken for a live counter. (A call captured in a
 *                 CUDA graph keeps its number on every replay; if a replay ever reports
 *                 PDA_DEVERR_TIMEOUT, zero the workspace before the next replay.)
 *  Supported: D in {64, 128}; block_size in {16, 32, 64, 128, 256} (the kernel works in
 *  tiles of 16 rows of one physical block); H / H_kv in {1, 2, 4, 8}; B <= 8192;
 *  kv_dtype in {PDA_F32, PDA_BF16, PDA_F16}. Pointers 16-byte aligned. Other sizes return
 *  PDA_ERR_UNSUPPORTED.
 */
pda_status pda_paged_decode_attention(void* out, const void* q, const void* k_cache,
                                      const void* v_cache, const int32_t* block_tables,
                                      int max_blocks_per_seq, const int32_t* context_lens,
                                      int max_context_len, int B, int H, int H_kv, int D,
                                      int block_size, int num_blocks, float scale,
                                      pda_dtype q_dtype, pda_dtype kv_dtype, pda_dtype out_dtype,
                                      int sm_cap, void* workspace, size_t workspace_bytes,
                                      int32_t* error_word, cudaStream_t stream);

/*
 * pda_paged_decode_attention_fp8 -- pda_paged_decode_attention over an FP8 E4M3 KV cache.
 *
 * A quantised KV cache cuts the bytes each decode step must read (page "From
 * PagedAttention to Prefill-Decode disaggregation", sec. 6.2: a low-precision KV cache,
 * dequantised to FP8 before attention, raises memory bandwidth and throughput). Each
 * stored K code means decode(code) * k_scale and each V code decode(code) * v_scale
 * (per-tensor scales); the result is softmax(scale * q K^T) V over those values, exactly as
 * pda_paged_decode_attention computes it. Codes are widened exactly in registers. At D = 128
 * the products run on the tensor cores: K, V (exact in fp16) and q (exact in fp16 after a
 * power-of-two rescale) as fp16 operands, fp32 accumulation, probabilities entering P V as
 * two fp16 parts (relative error about 2^-22); softmax in fp32. At D = 64 all arithmetic is
 * fp32.
 *
 *  k_cache, v_cache [num_blocks, block_size, H_kv, D] bytes (E4M3 codes).
 *  q               [B, H, D] in q_dtype, which must be PDA_BF16.
 *  k_scale, v_scale finite per-tensor scales.
 *  Every other argument, the workspace (pda_attention_workspace_size with PDA_FP8_E4M3),
 *  the supported sizes and the errors are those of pda_paged_decode_attention.
 */
pda_status pda_paged_decode_attention_fp8(void* out, const void* q, const void* k_cache,
                                          const void* v_cache, const int32_t* block_tables,
                                          int max_blocks_per_seq, const int32_t* context_lens,
                                          int max_context_len, int B, int H, int H_kv, int D,
                                          int block_size, int num_blocks, float scale,
                                          float k_scale, float v_scale, pda_dtype q_dtype,
                                          pda_dtype out_dtype, int sm_cap, void* workspace,
                                          size_t workspace_bytes, int32_t* error_word,
                                          cudaStream_t stream);

/*
 * pda_paged_decode_attention_nvfp4 -- pda_paged_decode_attention over an NVFP4 KV cache.
 *
 * The 4-bit KV format with fine-grained block scaling in E4M3 (page "From PagedAttention to
 * Prefill-Decode disaggregation", sec. 6.2: NVFP4 KV stores 4-bit values with fine-grained
 * block scales and E4M3 scale factors). Element d of the K row of (token row r, kv-head h)
 * means  e2m1(code) * e4m3(block scale) * k_scale,  with
 *   code        = nibble d % 2 (0: low, 1: high) of k_data[r][h][d / 2],
 *   block scale = k_block_scales[r / block_size][h][r % block_size][d / 16]
 *                 (one per 16 consecutive elements),
 * and the same for V. E2M1 is the 4-bit float with 2 exponent bits (bias 1) and 1 mantissa
 * bit: magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6. Values are dequantised exactly in registers
 * (the pages describe a dequantisation to FP8 before attention; fp16 and fp32 hold every
 * product e2m1 * e4m3 exactly, so nothing is rounded before the attention arithmetic),
 * which at D = 128 runs on the tensor cores as for pda_paged_decode_attention_fp8.
 *
 *  k_data, v_data   [num_blocks, block_size, H_kv, D / 2] bytes.
 *  k_block_scales, v_block_scales [num_blocks, H_kv, block_size, D / 16] E4M3 bytes,
 *                   16-byte aligned: per block and head-major, so the scales of the 16
 *                   rows of one kv-head that a tile covers are one contiguous run of D
 *                   bytes (the pages give no layout; this is the one the kernel reads in
 *                   one bulk copy per tile and head).
 *  q                [B, H, D] in q_dtype, which must be PDA_BF16.
 *  k_scale, v_scale finite per-tensor scales.
 *  Every other argument, the workspace (pda_attention_workspace_size with PDA_NVFP4), the
 *  supported sizes and the errors are those of pda_paged_decode_attention.
 *  Append, pack and unpack: the data tensors are token-major byte caches, moved by
 *  pda_kv_append, pda_kv_pack_blocks[_batched] and pda_kv_unpack_blocks[_batched] with
 *  kv_dtype PDA_FP8_E4M3 (any 1-byte type) and D / 2 as the row length (H_kv * D / 2 a
 *  multiple of 16 bytes); the block scales by pda_kv_append_block_scales,
 *  pda_kv_pack_block_scales_batched and pda_kv_unpack_block_scales_batched.
 */
pda_status pda_paged_decode_attention_nvfp4(void* out, const void* q, const void* k_data,
                                            const void* v_data, const void* k_block_scales,
                                            const void* v_block_scales,
                                            const int32_t* block_tables, int max_blocks_per_seq,
                                            const int32_t* context_lens, int max_context_len,
                                            int B, int H, int H_kv, int D, int block_size,
                                            int num_blocks, float scale, float k_scale,
                                            float v_scale, pda_dtype q_dtype,
                                            pda_dtype out_dtype, int sm_cap, void* workspace,
                                            size_t workspace_bytes, int32_t* error_word,
                                            cudaStream_t stream);

/*
 * pda_paged_window_attention -- decode attention with a sliding window: each request's query token
 * attends over the last `window` tokens of its history (itself among them) and the first `sinks`,
 * which stay visible:
 *      s_t = scale * q[b,h,:] . K_t[k,:],   t < L and (t >= L - window or t < sinks).
 * The pages describe no windowed model; this is what its layers need beside
 * pda_paged_decode_attention (page "Disaggregated LLM Serving", sec. 1), of which everything else
 * holds. Blocks that hold no visible token are not looked up or read: their table entries may be
 * anything (pda_kv_assign_blocks wants them negative once their blocks are given back), and their
 * memory another request's. What blocks hold in rows that are not visible does
 * not reach the output.
 *
 *  window         >= 1; sinks >= 0. A window as long as the history is none.
 *  kv_dtype       any of pda_paged_decode_attention, _fp8 and _nvfp4; q_dtype, the caches, the
 *                 block scales (NULL but for PDA_NVFP4) and k_scale, v_scale (1 for the plain
 *                 types) are as there.
 *  workspace      of pda_attention_workspace_size for the same sizes.
 *  The other sizes and the errors are those calls'.
 */
pda_status pda_paged_window_attention(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const void* k_block_scales, const void* v_block_scales, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* context_lens, int max_context_len, int window,
    int sinks, int B, int H, int H_kv, int D, int block_size, int num_blocks, float scale,
    float k_scale, float v_scale, pda_dtype q_dtype, pda_dtype kv_dtype, pda_dtype out_dtype,
    int sm_cap, void* workspace, size_t workspace_bytes, int32_t* error_word,
    cudaStream_t stream);

/*
 * pda_paged_decode_attention_noalloc -- pda_paged_decode_attention without a workspace
 * argument, for callers that cannot allocate device memory.
 *
 * The pages describe no such call; it exists for code that may not call cudaMalloc or any
 * allocator when it runs: a plugin inside a host framework that owns all device memory and
 * hands out only inputs and outputs, or a serving loop that forbids allocation once it has
 * started. Such a caller still provides q, the caches, the tables, the lengths and out
 * exactly as for pda_paged_decode_attention (same meaning, layout and errors); the scratch
 * the kernels need comes from one fixed array of PDA_NOALLOC_SCRATCH_BYTES bytes compiled
 * into the library as a device global. Every GPU that loads the library holds that array
 * until the process exits. The call itself never calls cudaMalloc, cudaFree or any
 * allocating routine.
 *
 *  - Sizes whose scratch need exceeds PDA_NOALLOC_SCRATCH_BYTES (see
 *    pda_attention_workspace_size) are rejected with PDA_ERR_TOO_LARGE before any launch.
 *    On a 152-SM GB300 this admits every supported shape with H / H_kv <= 4 at D = 128
 *    (about 5 MB) and rejects H / H_kv = 8 at D = 128 (about 10 MB).
 *  - The first call on a device looks up the array's device address (cudaGetSymbolAddress,
 *    with that device current) and caches it for later calls.
 *  - Every call shares the one array, which keeps the previous call's contents: those of a
 *    call of another shape, or of one that stopped early with PDA_DEVERR_TIMEOUT. Partial
 *    results are written before they are read. The per-segment arrival counters at the
 *    head of the array must not carry counts from an earlier call, so every call first
 *    clears them (B * H_kv * 8 bytes or less, one cudaMemsetAsync on `stream`, which
 *    allocates nothing) and then launches the kernel.
 *    Calls that overlap on the GPU (on different streams, or from different host threads)
 *    race on the array and produce wrong results; serialise them.
 */
pda_status pda_paged_decode_attention_noalloc(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
    int max_context_len, int B, int H, int H_kv, int D, int block_size, int num_blocks,
    float scale, pda_dtype q_dtype, pda_dtype kv_dtype, pda_dtype out_dtype, int sm_cap,
    int32_t* error_word, cudaStream_t stream);

/*
 * pda_kv_pack_blocks -- gather one request's KV into one contiguous buffer.
 *
 * Defined by the request-level KV transfer of PD disaggregation (page on goodput and PD
 * disaggregation, 0539edu.com, sec. 5.4: after prefill, a request's whole KV is sent in
 * one transfer) over the paged layout above: for t < context_len,
 *      out[t, 0, :, :] = K of token t,   out[t, 1, :, :] = V of token t,
 * token t being row t % block_size of physical block block_table_row[t / block_size].
 *
 *  out            [context_len, 2, H_kv, D] in kv_dtype, dense.
 *  block_table_row device pointer to the request's table row (int32).
 *  context_len    host int, tokens to pack; 0 is a no-op.
 *  A block id out of range sets PDA_DEVERR_BLOCK_ID and fills that token's output with
 *  0xFF bytes (a NaN pattern). The copy is bitwise. Needs H_kv * D * sizeof(kv_dtype) to be
 *  a multiple of 16 bytes and 16-byte aligned pointers.
 */
pda_status pda_kv_pack_blocks(void* out, const void* k_cache, const void* v_cache,
                              const int32_t* block_table_row, int context_len, int H_kv, int D,
                              int block_size, int num_blocks, pda_dtype kv_dtype,
                              int32_t* error_word, cudaStream_t stream);

/*
 * pda_kv_pack_blocks_batched -- pda_kv_pack_blocks for n requests in one launch.
 *
 *  outs, block_table_rows, context_lens: HOST arrays of n entries; outs[i] and
 *  block_table_rows[i] are device pointers, context_lens[i] a host count. The arrays are
 *  copied into the launch, so the caller may reuse them when the call returns.
 *  n <= PDA_PACK_MAX_BATCH. Same semantics per request as pda_kv_pack_blocks.
 */
pda_status pda_kv_pack_blocks_batched(void* const* outs, const int32_t* const* block_table_rows,
                                      const int32_t* context_lens, int n, const void* k_cache,
                                      const void* v_cache, int H_kv, int D, int block_size,
                                      int num_blocks, pda_dtype kv_dtype, int32_t* error_word,
                                      cudaStream_t stream);

/*
 * pda_kv_unpack_blocks -- the receiving side of a request-level KV transfer: scatter one
 * request's contiguous KV buffer into the blocks allocated for it.
 *
 * Defined by the KV migration of PD disaggregation (page on goodput and PD disaggregation,
 * 0539edu.com, sec. 3: after prefill the request's KV moves to a decode worker; sec. 5.4:
 * request-level transfer sends it in one piece) into the paged layout, whose blocks are
 * allocated on demand (page "From PagedAttention to Prefill-Decode disaggregation", sec. 2.2
 * step 3). The inverse of pda_kv_pack_blocks: for t < context_len, the K row of token t
 * (row t % block_size of block block_table_row[t / block_size]) = in[t, 0, :, :] and the V
 * row = in[t, 1, :, :].
 *
 *  in             [context_len, 2, H_kv, D] in kv_dtype, dense; read only.
 *  k_cache,v_cache [num_blocks, block_size, H_kv, D], updated in place; rows of other
 *                 tokens are not touched.
 *  A block id out of range sets PDA_DEVERR_BLOCK_ID and that token is not written. Tokens
 *  that map to the same row race (the caller must not do that). Bitwise copy; 16-byte rows
 *  and alignment as for pack.
 */
pda_status pda_kv_unpack_blocks(const void* in, void* k_cache, void* v_cache,
                                const int32_t* block_table_row, int context_len, int H_kv,
                                int D, int block_size, int num_blocks, pda_dtype kv_dtype,
                                int32_t* error_word, cudaStream_t stream);

/*
 * pda_kv_unpack_blocks_batched -- pda_kv_unpack_blocks for n requests in one launch.
 *  ins, block_table_rows, context_lens: HOST arrays of n entries (device pointers and host
 *  counts), copied into the launch. n <= PDA_PACK_MAX_BATCH.
 */
pda_status pda_kv_unpack_blocks_batched(const void* const* ins,
                                        const int32_t* const* block_table_rows,
                                        const int32_t* context_lens, int n, void* k_cache,
                                        void* v_cache, int H_kv, int D, int block_size,
                                        int num_blocks, pda_dtype kv_dtype, int32_t* error_word,
                                        cudaStream_t stream);

/*
 * pda_kv_pack_layers -- pda_kv_pack_blocks of one request over n_layers layers' caches, in
 * one launch.
 *
 * A model keeps one K and one V cache per layer, and a request's blocks have the same ids in
 * every layer (one block table per request). Request-level transfer sends all layers once
 * prefill ends (page on goodput and PD disaggregation, 0539edu.com, sec. 5.4, request
 * granularity); layer-level transfer sends layer N as soon as its prefill is done, hidden
 * behind the computation of the later layers (same page and section, layer granularity;
 * page "Disaggregated LLM Serving: from PD disaggregation to attention offload", sec. 5.6),
 * which is one pda_kv_pack_blocks per layer on a transfer stream. This call is the
 * whole-model form: for layer i < n_layers and t < context_len,
 *      outs[i][t, 0, :, :] = K of token t in k_caches[i],  outs[i][t, 1, :, :] = V.
 *
 *  outs, k_caches, v_caches: HOST arrays of n_layers device pointers, copied into the
 *                 launch; outs[i] is [context_len, 2, H_kv, D] in kv_dtype, dense; every
 *                 layer's caches are [num_blocks, block_size, H_kv, D].
 *  block_table_row device pointer to the request's table row (int32), shared by all layers.
 *  n_layers <= PDA_PACK_MAX_LAYERS (more: PDA_ERR_UNSUPPORTED); 0 or context_len 0 is a
 *  no-op. Errors, bitwise copy and alignment as for pda_kv_pack_blocks.
 */
pda_status pda_kv_pack_layers(void* const* outs, const void* const* k_caches,
                              const void* const* v_caches, int n_layers,
                              const int32_t* block_table_row, int context_len, int H_kv, int D,
                              int block_size, int num_blocks, pda_dtype kv_dtype,
                              int32_t* error_word, cudaStream_t stream);

/*
 * pda_kv_unpack_layers -- the receiving side of pda_kv_pack_layers: for layer i and
 * t < context_len, the K row of token t in k_caches[i] = ins[i][t, 0, :, :] and the V row =
 * ins[i][t, 1, :, :]. HOST arrays of n_layers device pointers, copied into the launch;
 * semantics per layer as for pda_kv_unpack_blocks (a bad block id sets
 * PDA_DEVERR_BLOCK_ID and that token is not written in any layer).
 */
pda_status pda_kv_unpack_layers(const void* const* ins, void* const* k_caches,
                                void* const* v_caches, int n_layers,
                                const int32_t* block_table_row, int context_len, int H_kv,
                                int D, int block_size, int num_blocks, pda_dtype kv_dtype,
                                int32_t* error_word, cudaStream_t stream);

/*
 * pda_kv_append_block_scales -- pda_kv_append for the E4M3 block scales of an NVFP4 cache.
 *
 * Each decode step's new token brings one scale per 16 elements of its K and V rows (page
 * "From PagedAttention to Prefill-Decode disaggregation", sec. 6.2, NVFP4 KV with block
 * scales); the token of request b goes to slot s = slot_mapping[b], i.e. row s % block_size of
 * block s / block_size (page "Disaggregated LLM Serving: from PD disaggregation to attention
 * offload", sec. 1, the per-step KV write). For b < B and h < H_kv:
 *      k_scales[s / block_size][h][s % block_size][:] = k_new[b][h][:]   (D / 16 bytes)
 * and the same for V.
 *
 *  k_new, v_new     [B, H_kv, D / 16] E4M3 bytes, 4-byte aligned; read only.
 *  k_scales, v_scales [num_blocks, H_kv, block_size, D / 16] (the layout of
 *                   pda_paged_decode_attention_nvfp4), 4-byte aligned; updated in place.
 *  slot_mapping     [B] int32, device; negative = padding (skipped).
 *  D a multiple of 64 (rows move as 4-byte words), else PDA_ERR_UNSUPPORTED. A slot at or
 *  beyond num_blocks * block_size sets PDA_DEVERR_SLOT and is skipped. B = 0 is a no-op.
 */
pda_status pda_kv_append_block_scales(const void* k_new, const void* v_new, void* k_scales,
                                      void* v_scales, const int32_t* slot_mapping, int B,
                                      int H_kv, int D, int block_size, int num_blocks,
                                      int32_t* error_word, cudaStream_t stream);

/*
 * pda_kv_pack_block_scales_batched -- pda_kv_pack_blocks_batched for the block scales of an
 * NVFP4 cache: for request i and t < context_lens[i], with block = block_table_rows[i][t /
 * block_size] and offset = t % block_size,
 *      outs[i][t, 0, h, :] = k_scales[block][h][offset][:],
 *      outs[i][t, 1, h, :] = v_scales[block][h][offset][:].
 *
 *  outs[i]          [context_lens[i], 2, H_kv, D / 16] bytes, dense, 4-byte aligned.
 *  outs, block_table_rows, context_lens: HOST arrays of n entries (device pointers and host
 *  counts), copied into the launch. n <= PDA_PACK_MAX_BATCH. A block id out of range sets
 *  PDA_DEVERR_BLOCK_ID and fills that token's scales with 0xFF bytes (an E4M3 NaN).
 *  D a multiple of 64. Bitwise copy.
 */
pda_status pda_kv_pack_block_scales_batched(void* const* outs,
                                            const int32_t* const* block_table_rows,
                                            const int32_t* context_lens, int n,
                                            const void* k_scales, const void* v_scales,
                                            int H_kv, int D, int block_size, int num_blocks,
                                            int32_t* error_word, cudaStream_t stream);

/*
 * pda_kv_unpack_block_scales_batched -- the inverse of pda_kv_pack_block_scales_batched:
 * k_scales[block][h][offset][:] = ins[i][t, 0, h, :] and v_scales[...] = ins[i][t, 1, h, :].
 * A block id out of range sets PDA_DEVERR_BLOCK_ID and that token is not written; other
 * rows are not touched. Arrays, limits and alignment as for the pack.
 */
pda_status pda_kv_unpack_block_scales_batched(const void* const* ins,
                                              const int32_t* const* block_table_rows,
                                              const int32_t* context_lens, int n,
                                              void* k_scales, void* v_scales, int H_kv, int D,
                                              int block_size, int num_blocks,
                                              int32_t* error_word, cudaStream_t stream);

/*
 * pda_kv_assign_blocks -- grow and shrink every request's block table to its length, taking
 * blocks from a free list and giving them back, on the GPU.
 *
 * Blocks are handed out as tokens arrive (page "From PagedAttention to Prefill-Decode
 * disaggregation", sec. 2.2 step 3); the pages give no free list. Here it is a stack:
 * free_list[0 .. free_count) holds the ids of the free blocks, the last one on top. With
 * need_b = ceil(context_lens[b] / block_size):
 *  - a row that holds more than it needs gives back entries [need_b, blocks_held[b]) of its
 *    table; all rows' entries are pushed in order of b, then of the entry. A negative entry holds
 *    no block and is passed over;
 *  - after that, a row that holds fewer gets entries [blocks_held[b], need_b), popped one at
 *    a time in the same order. The first row whose blocks are not all there, and every later
 *    row that grows, get none (PDA_DEVERR_NO_BLOCKS); their counts stay.
 *
 *  block_tables   [B, max_blocks_per_seq] int32, updated in place. Entries given back are
 *                 left in the table, behind the row's new end.
 *  blocks_held    [B] int32: entries of each row in use; blocks_held_out [B] receives the
 *                 new counts. The two may be the same buffer.
 *  free_list      [num_blocks] int32, updated in place; entries above the new count are
 *                 unspecified but in place (popped entries are not cleared).
 *  free_count     [1] int32; free_count_out [1] receives the new count; may be the same.
 *  context_lens   [B] int32: the length each row must cover; 0 gives every block back.
 *  shared_blocks  [B] int32 or NULL: the row's first shared_blocks[b] entries belong to
 *                 somebody else (a prefix that several rows share) and are never given back.
 *                 No other block may be in two rows, or it is given back twice. Updated in
 *                 place: a row that shrinks into its prefix and grows again gets blocks of
 *                 its own from blocks_held[b] on, not the shared ones, which it may not
 *                 write; its shared_blocks[b] falls to blocks_held[b], so that they are
 *                 given back. It is set anew, with the entries and blocks_held[b], when the
 *                 row takes its next request.
 *  Blocks that the caller gives back itself out of a row's middle, as those that have left a
 *  sliding window: it puts their ids on the stack, and makes their entries negative before the
 *  next call. An entry that keeps such an id is given back a second time with its row, and two
 *  rows then share the block, which this call cannot see.
 *  A row with context_lens < 0 or beyond max_blocks_per_seq * block_size, or with blocks_held
 *  outside [0, max_blocks_per_seq], is left as it is (PDA_DEVERR_CONTEXT_LEN). free_count
 *  outside [0, num_blocks] (PDA_DEVERR_NO_BLOCKS), or more blocks given back than the list
 *  holds (PDA_DEVERR_BLOCK_ID), leaves everything as it is. An entry of num_blocks or more that
 *  would be given back is passed over, and an id out of range that is popped goes into the table;
 *  both set PDA_DEVERR_BLOCK_ID. Buffers not named as shareable must not overlap.
 *  B <= 8192 and B * max_blocks_per_seq < 2^31, else PDA_ERR_UNSUPPORTED. B == 0 copies the
 *  count.
 */
pda_status pda_kv_assign_blocks(int32_t* block_tables, const int32_t* blocks_held,
                                int32_t* blocks_held_out, int32_t* free_list,
                                const int32_t* free_count, int32_t* free_count_out,
                                const int32_t* context_lens, int32_t* shared_blocks, int B,
                                int max_blocks_per_seq, int block_size, int num_blocks,
                                int32_t* error_word, cudaStream_t stream);

/*
 * pda_kv_build_slots -- the cache slot of every new token, and where each request's tokens
 * start, from the requests' lengths, on the GPU.
 *
 * The slot that pda_kv_append takes comes from the block table (page "From PagedAttention to
 * Prefill-Decode disaggregation", sec. 2.2 step 3). Request b brings n = query_lens[b] new
 * tokens, the last of its L = context_lens[b]; they are rows query_start[b] ..
 * query_start[b + 1) of the step's tokens. Token i is at position p = L - n + i:
 *      slot_mapping[query_start[b] + i] = block_tables[b][p / block_size] * block_size
 *                                         + p % block_size.
 *
 *  slot_mapping   [N] int32, written whole: rows behind the last token get -1 (padding).
 *  query_start    [B + 1] int32, written: exclusive prefix sum of query_lens, clipped at N.
 *  query_lens     [B] int32; context_lens [B] int32; block_tables [B, max_blocks_per_seq].
 *  More than N tokens, or a negative query_lens (taken as 0), sets PDA_DEVERR_QUERY.
 *  L < 0, L beyond the table, or 0 < L < n gives the request's tokens -1 and sets
 *  PDA_DEVERR_CONTEXT_LEN; L == 0 gives -1 without an error (a padded row). A block id out
 *  of range gives -1 and PDA_DEVERR_BLOCK_ID. Outputs must not overlap inputs.
 *  B <= 8192, N <= 2^30, B * max_blocks_per_seq < 2^31, else PDA_ERR_UNSUPPORTED.
 */
pda_status pda_kv_build_slots(int32_t* slot_mapping, int32_t* query_start,
                              const int32_t* query_lens, const int32_t* context_lens,
                              const int32_t* block_tables, int N, int B, int max_blocks_per_seq,
                              int block_size, int num_blocks, int32_t* error_word,
                              cudaStream_t stream);

/*
 * pda_kv_build_slots_positions -- pda_kv_build_slots, and the position p of every new token in
 * its request (what pda_qk_norm_rope_append turns its queries and keys by).
 *
 *  positions      [N] int32, written whole: 0 for rows behind the last token and for the tokens
 *                 of a request whose length is in error or 0 (padded). A token whose block id is
 *                 out of range has no slot, but its position all the same.
 *                 Everything else as pda_kv_build_slots.
 */
pda_status pda_kv_build_slots_positions(int32_t* slot_mapping, int32_t* positions,
                                        int32_t* query_start, const int32_t* query_lens,
                                        const int32_t* context_lens, const int32_t* block_tables,
                                        int N, int B, int max_blocks_per_seq, int block_size,
                                        int num_blocks, int32_t* error_word,
                                        cudaStream_t stream);

/*
 * pda_qk_norm_rope_append -- the queries and keys of a step's new tokens, normed per head and
 * turned by their positions, and the keys and values written into their cache slots, in one pass:
 * what comes between a layer's projections and its attention, with pda_kv_append's write.
 *
 * The pages give no position encoding; the shapes and slots are pda_kv_append's (page
 * "Disaggregated LLM Serving: from PD disaggregation to attention offload", sec. 1). Each head row
 * x [D] of q and k, in fp32 and rounded once at the end:
 *  - with a weight w [D]:  x = x / sqrt(mean(x^2) + eps) * w   (q_weight for q, k_weight for k);
 *  - the first R = rope_dim elements turn in pairs by the angle of the token's position p:
 *      (a, b) -> (a c - b s, b c + a s),  c, s = attention_factor * cos, sin (2 pi p F_i / 2^64),
 *    pair i < R / 2 being elements (i, i + R / 2), or (2 i, 2 i + 1) where `interleaved` is not 0.
 * v is copied (a 16-bit NaN as the type's usual one). k and v of token t go to slot_mapping[t] as
 * by pda_kv_append (< 0: not written; too large: PDA_DEVERR_SLOT, not written; no slot twice);
 * q_out is written for every token.
 *
 *  q_out          [T, H, D] in dtype, dense. May be q itself where q is dense.
 *  q, k, v        [T, H, D], [T, H_kv, D], [T, H_kv, D] in dtype; a token's heads are dense, and
 *                 tokens are q_stride, k_stride, v_stride elements apart (slices of one
 *                 projection's output need no copy). Strides a multiple of 16 bytes, no smaller
 *                 than a token.
 *  k_cache,v_cache [num_blocks, block_size, H_kv, D] in kv_dtype, updated in place; kv_dtype is
 *                 dtype (PDA_F32, PDA_BF16, PDA_F16), or PDA_FP8_E4M3 with dtype PDA_BF16: then
 *                 the code nearest to x * (1 / k_scale) (v: 1 / v_scale) in fp32, no larger than
 *                 448, is stored.
 *  positions      [T] int32, any value.
 *  freqs          [rope_dim / 2] uint64: F_i, turns per position as a fraction of 2^64.
 *                 p F_i modulo 2^64 is exact, so far positions lose nothing.
 *  q_weight, k_weight [D] in dtype, each may be NULL (no norm).
 *  Supported: D a multiple of 8 up to 256; rope_dim a multiple of 16 up to D (0: no rotation);
 *  H, H_kv <= 16384. Pointers 16-byte aligned. Scales and their
 *  reciprocals finite. Inputs and outputs do not
 *  overlap otherwise. T == 0 is a no-op.
 */
pda_status pda_qk_norm_rope_append(void* q_out, const void* q, const void* k, const void* v,
                                   long long q_stride, long long k_stride, long long v_stride,
                                   void* k_cache, void* v_cache, const int32_t* slot_mapping,
                                   const int32_t* positions, const uint64_t* freqs, int rope_dim,
                                   int interleaved, float attention_factor, const void* q_weight,
                                   const void* k_weight, float eps, int T, int H, int H_kv, int D,
                                   int block_size, int num_blocks, float k_scale, float v_scale,
                                   pda_dtype dtype, pda_dtype kv_dtype, int32_t* error_word,
                                   cudaStream_t stream);

/*
 * pda_qk_norm_rope -- the same norm and rotation into dense rows, without a cache (for keys that
 * are quantised further before they are appended).
 *
 *  q_out, k_out   [T, H, D], [T, H_kv, D] in dtype, dense; may be q and k themselves where those
 *                 are dense. Everything else as pda_qk_norm_rope_append.
 */
pda_status pda_qk_norm_rope(void* q_out, void* k_out, const void* q, const void* k,
                            long long q_stride, long long k_stride, const int32_t* positions,
                            const uint64_t* freqs, int rope_dim, int interleaved,
                            float attention_factor, const void* q_weight, const void* k_weight,
                            float eps, int T, int H, int H_kv, int D, pda_dtype dtype,
                            cudaStream_t stream);

/*
 * pda_chunk_attention_workspace_size -- bytes of device workspace pda_paged_chunk_attention
 * (or _fp8, with PDA_FP8_E4M3) needs on the current device for these sizes. The bound does
 * not depend on the lengths. Written to *bytes (host).
 */
pda_status pda_chunk_attention_workspace_size(int B, int T, int H, int H_kv, int D,
                                              int block_size, pda_dtype kv_dtype, int sm_cap,
                                              size_t* bytes);

/*
 * pda_paged_chunk_attention -- every new token of each request attends over the request's
 * cached history up to and including itself.
 *
 * The attention of a prompt, of a chunk of a long prompt (the pages' chunked prefill), of
 * the rest of a prompt behind a shared prefix (page "From PagedAttention to Prefill-Decode
 * disaggregation", sec. 2.3) or of drafted tokens, after their K and V have been appended
 * (pda_kv_append takes any number of tokens). Request b has n = query_start[b + 1] -
 * query_start[b] new tokens, the last of its L = context_lens[b]. For token i, at position
 * p = L - n + i, and head h with kv-head k = h / (H / H_kv):
 *      s_t = scale * q . K_t[k],  t <= p
 *      out = sum_t softmax(s)_t * V_t[k].
 * n == 1 is pda_paged_decode_attention's row.
 *
 *  out, q         [T, H, D], both in q_dtype: the step's tokens, request after request. Rows
 *                 outside [query_start[0], query_start[B]) are neither computed nor written.
 *  query_start    [B + 1] int32 (device), non-decreasing, within [0, T].
 *  context_lens   [B] int32 (device). L == 0 gives zero rows (a padded request). L < 0,
 *                 L > max_context_len, L > max_blocks_per_seq * block_size or 0 < L < n
 *                 gives NaN rows and PDA_DEVERR_CONTEXT_LEN.
 *  A query_start that decreases or leaves [0, T] anywhere sets PDA_DEVERR_QUERY, and the
 *  call computes and writes nothing. A block id out of range gives NaN in the rows that see the block and
 *  PDA_DEVERR_BLOCK_ID.
 *  What the cache holds behind a row's position (later tokens, rows behind L, unused blocks)
 *  does not reach that row's output, NaN and infinities included.
 *  q_dtype must equal kv_dtype (PDA_F32, PDA_BF16 or PDA_F16); out has the same type.
 *  fp32 is computed in fp32; bf16 and fp16 on the tensor cores with fp32 accumulation and
 *  softmax, the probabilities rounded to the cache's type.
 *  workspace      device scratch of at least pda_chunk_attention_workspace_size(...) bytes,
 *                 256-byte aligned, not shared by calls that may run concurrently; its
 *                 content before and after a call means nothing.
 *  The other arguments, the supported sizes (D, block_size, H / H_kv, B) and alignment are
 *  those of pda_paged_decode_attention; T * H < 2^31, the smaller of max_context_len and
 *  max_blocks_per_seq * block_size at most 2^30, and (T / t + B) * H_kv *
 *  (max_context_len / 128 + 5) < 2^31 with t = 256 * H_kv / H tokens (fp32: 64 * H_kv / H).
 */
pda_status pda_paged_chunk_attention(void* out, const void* q, const void* k_cache,
                                     const void* v_cache, const int32_t* block_tables,
                                     int max_blocks_per_seq, const int32_t* context_lens,
                                     const int32_t* query_start, int max_context_len, int B,
                                     int T, int H, int H_kv, int D, int block_size,
                                     int num_blocks, float scale, pda_dtype q_dtype,
                                     pda_dtype kv_dtype, int sm_cap, void* workspace,
                                     size_t workspace_bytes, int32_t* error_word,
                                     cudaStream_t stream);

/*
 * pda_paged_chunk_attention_fp8 -- pda_paged_chunk_attention over an FP8 E4M3 cache: stored
 * code c of K means decode(c) * k_scale, of V decode(c) * v_scale (finite per-tensor scales).
 * q and out are PDA_BF16. Both products run with fp16 operands and fp32 accumulation: the codes
 * are widened exactly, each row of q (of a token and head) is scaled by a power of two that puts
 * its largest element at 2^14 and rounded to fp16 (elements below 2^-28 of that largest lose
 * bits, those below 2^-38 of it count as zero), and the probabilities are rounded to fp16.
 */
pda_status pda_paged_chunk_attention_fp8(void* out, const void* q, const void* k_cache,
                                         const void* v_cache, const int32_t* block_tables,
                                         int max_blocks_per_seq, const int32_t* context_lens,
                                         const int32_t* query_start, int max_context_len, int B,
                                         int T, int H, int H_kv, int D, int block_size,
                                         int num_blocks, float scale, float k_scale,
                                         float v_scale, pda_dtype q_dtype, int sm_cap,
                                         void* workspace, size_t workspace_bytes,
                                         int32_t* error_word, cudaStream_t stream);

/*
 * pda_paged_window_chunk_attention -- chunk attention with a sliding window: token i of request b,
 * at position p = L - n + i, attends over the last `window` tokens up to itself and the request's
 * first `sinks`:  t <= p and (t > p - window or t < sinks).
 * n == 1 is pda_paged_window_attention's row.
 *
 * Everything else is pda_paged_chunk_attention's (pda_paged_chunk_attention_fp8's with kv_dtype
 * PDA_FP8_E4M3; k_scale and v_scale are 1 for the plain types), the workspace too. Blocks that no
 * new token of the request sees are not looked up or read, whatever their table entries. A block
 * id out of range gives NaN in the rows that see the block, and PDA_DEVERR_BLOCK_ID. What the cache holds in
 * rows that a token does not see does not reach its output, NaN and infinities included.
 *  window >= 1, sinks >= 0. A window as long as the history is none.
 */
pda_status pda_paged_window_chunk_attention(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
    const int32_t* query_start, int max_context_len, int window, int sinks, int B, int T, int H,
    int H_kv, int D, int block_size, int num_blocks, float scale, float k_scale, float v_scale,
    pda_dtype q_dtype, pda_dtype kv_dtype, int sm_cap, void* workspace, size_t workspace_bytes,
    int32_t* error_word, cudaStream_t stream);

/*
 * pda_verify_drafts -- how many of each request's drafted tokens the target model keeps, and the
 * token that comes after them: what follows the chunk attention of drafted tokens.
 *
 * The pages describe no drafting; the rule is the published one of speculative sampling (accept a
 * draft x of probability q(x) with probability min(1, p(x) / q(x)); at the first one turned down,
 * draw from what p has over q), whose tokens are distributed as the target's own. Request b has
 * the step's rows query_start[b] .. query_start[b + 1): its last token, then d drafts. Row r
 * holds the target's probabilities p_r of the token behind row r's, and judges row r + 1's:
 *  - accepted[b] = a, the number of leading drafts with
 *      accept_u[r] * q_r(tokens[r + 1]) < p_r(tokens[r + 1])     (in fp32);
 *  - next_tokens[b]: with weights max(p_r - q_r, 0) at the row r that turned its draft down (p_r
 *    if none of them is positive), or p_r at the request's last row, the first token t whose
 *    sum of weights up to t exceeds sample_u[b] times their sum.
 * So the request goes on with its first a drafts and next_tokens[b], and its length falls by
 * d - a. (A request without rows has no d: its length stays.)
 *
 *  accepted, next_tokens [B] int32, written.
 *  target_probs   [T, V] in dtype (PDA_F32, PDA_BF16, PDA_F16), rows target_stride elements apart
 *                 (>= V). They need not sum to one. A weight that is not positive counts as zero.
 *  draft_probs    [T, V] in dtype, row r: what the token of row r + 1 was drawn from; rows
 *                 draft_stride apart; a request's last row is not read. NULL: the drafts were
 *                 certain (q = 1 at the draft, 0 elsewhere).
 *  tokens         [T] int32, the step's tokens; a request's first is not read.
 *  query_start    [B + 1] int32, non-decreasing, within [0, T].
 *  accept_u       [T] fp32, sample_u [B] fp32: uniform in [0, 1); a request's last accept_u is not
 *                 read.
 *  A request without rows gets accepted 0 and token -1; so does one whose query_start decreases or
 *  leaves [0, T], with PDA_DEVERR_QUERY. A draft outside [0, V) is turned down
 *  (PDA_DEVERR_TOKEN). Where no weight is positive, or their sum is not finite, next_tokens[b] is
 *  -1 (PDA_DEVERR_PROBS). Probabilities aligned to their type; rows aligned to 16 bytes are read
 *  faster. V <= 2^20, B <= 8192, else PDA_ERR_UNSUPPORTED. B == 0 is a no-op.
 */
pda_status pda_verify_drafts(int32_t* accepted, int32_t* next_tokens, const void* target_probs,
                             const void* draft_probs, long long target_stride,
                             long long draft_stride, const int32_t* tokens,
                             const int32_t* query_start, const float* accept_u,
                             const float* sample_u, int T, int B, int V, pda_dtype dtype,
                             int32_t* error_word, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PDA_H */
