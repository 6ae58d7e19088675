// chunk_tc_kernel.cuh -- chunk attention over 16-bit and FP8 caches on the tcgen05 tensor
// cores, and its launch.
//
// Mathematics. With packed rows R = token * G + head (the G query heads of a kv-head share its
// keys), S = Q K^T per 128 rows x 128 keys, softmax with a running maximum m and sum l,
// O += P V. m is a reference, not the exact maximum: it only moves when a row's scores pass
// it by 2^8, and then O and l are rescaled; the result O / l does not depend on it. Scores,
// m, l and O stay in fp32; the probabilities are rounded to the operands' 16-bit type for the
// P V product (the matrix instruction takes no wider operand with 16-bit V).
//
// What bounds it: 4096 tokens on 12288 of 32/8 heads run at 1592 TFLOP/s under the power cap (604
// us, 90 % of the measured sustained GEMM rate) and 570 us before it sets in (86 % of the burst
// rate), the tensor pipe 73 % busy: Q K's two operands come from shared memory, 128 bytes a cycle,
// and one warp hands the pipe from group to group. 32 requests of 1 to 8 tokens over up to 8192
// stream 5.7 TB/s (120 us, 85 % of the copy peak). Eight warps of softmax with a thread per row
// need no shuffles; with score tiles of 128 keys more do not fit TMEM's 512 columns.
//
// One block per SM walks a contiguous range of the launch's units (chunk_plan.h). Warps:
//   0-3, 4-7  softmax of row group 0 and 1 (a thread per row: TMEM lane = row)
//   8         plans the block's pieces, publishes them, and loads Q and K with TMA
//   9         issues the matrix instructions
//   10        loads V with TMA
//   11        writes the rows of requests without work
//   12-15     clean the V tiles at the diagonal and the end (see below), or, over an FP8
//             cache, widen every K and V tile: the TMA brings the codes, these warps write
//             them as fp16 (exact, and one instruction for two codes, where bf16 took four:
//             365 -> 341 us on three chunks of up to 2048 tokens; 311 with K and V through
//             one copy of the loop) where the products read them. The softmax warps then
//             bring Q, each row scaled by a power of two that puts its largest value at
//             2^14: elements below 2^-28 of that value are subnormal and lose bits, and
//             what falls under fp16's smallest step is below 2^-38 of it.
// The softmax warps take the registers that the others give back (setmaxnreg).
// An item of more than 128 rows gives each group 128 rows; both read every K and V tile. An
// item of fewer gives both groups the same rows and alternate tiles, merged at the end, so
// that one group's softmax still runs under the other's products.
// TMEM: S0 | S1 | O0 | O1, 128 columns each; P overwrites the first 64 columns of its S. The next
// Q K then overwrites P, with nothing but the order of issue between it and the P V that reads P:
// the kernel relies on matrix instructions of one thread running in that order, which PTX states
// for equal accumulators and shapes only. A commit and a wait between them took 634 us for 562 on
// the large chunk, 142 for 136 on ragged prompts.
//
// V tiles that reach past what some row may see (the diagonal ones) multiply zero
// probabilities with later tokens' V, or with whatever lies behind the last token; 0 * NaN
// would reach the output. Warps 12 to 15 zero the rows behind the end, replace non-finite
// values by zeros and note their rows, and the epilogue adds those values back to the rows
// that do see them.
//
// With a sliding window (kWindow) an item's tiles are those of the first `sinks` tokens and, from
// its first token's window on, the rest: `skip` key tiles between them are left out, and nothing
// but the key a tile starts at (key_tile) knows of the gap. Tiles at the window's lower border
// and the end of the first tokens are masked per row and cleaned as the diagonal's are, and their
// blocks that no row of the item sees are not looked up: block 0 stands in, whose values are
// masked and cleaned too. 4096 tokens over 4096 + 64 keys of 32/8 heads run at 1313 TFLOP/s of
// visible pairs (213 us), ragged prompts over 513 keys take 162 us: item borders, with five of an
// item's seven tiles masked (5 % of the time) and cleaned (5-8 %).
#pragma once

#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>
#include <type_traits>

#include "chunk_plan.cuh"
#include "tcgen05.cuh"

namespace pda {
namespace {

constexpr int kThreads = 512;
constexpr int kSoftmaxRegs = 176, kOtherRegs = 80;  // 2 x 128 of each: what 512 x 128 give
constexpr int kCleaners = 4;
// with a window a piece's description is longer, and the last kilobytes hold three
template <bool kWindow>
constexpr int kDescsOf = kWindow ? 3 : 4;
template <bool kWindow>
using CutsOf = Cuts<8, 4, 6, kWindow>;  // 256-row items
constexpr float kRaise = 8.f;       // the reference maximum moves by at least 2^8

template <bool kWindow>
struct DescWindow {};
template <>
struct DescWindow<true> {
  int skip;    // key tiles left out behind the first tokens'
  int lowest;  // first key of the first token's window; the last token's starts at
  int last_lowest;
};

// Tiles that some row does not see whole: the diagonal's three, and with a window the last of the
// first tokens' (before the others) and three at the window's lower border.
template <bool kWindow>
constexpr int kEdgesOf = kWindow ? 7 : 3;

// One piece of work: key tiles [ja, jb) of an item.
template <bool kWindow>
struct Desc : DescWindow<kWindow> {
  int valid;
  int row0;     // the item's first token: row of q and out
  int tokens;   // tokens of the item
  int pos0;     // position of the first
  int kh;
  int ja, jb;
  int tiles0, tiles1;  // key tiles of row groups 0 and 1
  int single;   // both groups hold the same 128 rows
  int jc;       // first tile that some row does not see whole
  int end;      // keys any row sees
  int slot;     // partial-result slot, -1: the whole item
  int bad_from; // position of the first block with an id out of range
  long long table;  // the request's row in block_tables
  unsigned nonfinite[kEdgesOf<kWindow>][4];  // V rows of those tiles that hold a NaN or infinity

  // the key tile behind tile j of the item
  __device__ __forceinline__ int key_tile(const ChunkParams& p, int j) const {
    if constexpr (kWindow) return j + (j >= p.sink_tiles ? this->skip : 0);
    return j;
  }
  // key tile r's number among those that some row does not see whole, -1: every row does
  __device__ __forceinline__ int edge(const ChunkParams& p, int r) const {
    if constexpr (!kWindow) return r < jc ? -1 : r - jc;
    if constexpr (kWindow) {
      if (r >= jc) return 4 + r - jc;
      if (r * kChunkKeys >= this->last_lowest || r * kChunkKeys + kChunkKeys - 1 < p.sinks)
        return -1;
      const int low = r - (this->lowest >> 7);
      return low < 0 ? 0 : 1 + low;
    }
  }
  // and the key tile of such a number
  __device__ __forceinline__ int edge_tile(const ChunkParams& p, int e) const {
    if constexpr (kWindow)
      return e == 0 ? p.sink_tiles - 1 : e < 4 ? (this->lowest >> 7) + e - 1 : jc + e - 4;
    return jc + e;
  }
};

template <int D, bool kFp8>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kChunkKeys * D * 2;  // bytes of a K, V or Q tile
  static constexpr int kHalf = kChunkKeys * 128;    // of its 64-element half
  // K and V ring apart: every V tile passes through the cleaning warps, K tiles do not
  static constexpr int kK = D == 64 ? 5 : kFp8 ? 2 : 3;
  static constexpr int kV = D == 64 ? 5 : 2;
  static constexpr int kRaw = kFp8 ? kChunkKeys * D : 0;  // bytes of a tile of codes
};

// One box of a tensor map into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* tm, int c0, int c1, int c2,
                                        uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tma_box4(void* dst, const CUtensorMap* tm, int c0, int c1, int c2,
                                         int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "r"(smem_addr(bar))
      : "memory");
}

template <bool kWindow>
struct Misc {
  static constexpr int kDescs = kDescsOf<kWindow>;
  uint64_t k_full[5], k_empty[5], v_full[5], v_empty[5], clean[5];
  uint64_t raw_full[2], raw_empty[2];  // codes of a K and of a V tile
  uint64_t q_full, q_full1, q_empty,  // q_full1: group 1's, where the softmax warps bring Q
           s_full[2], p_full[2], o_full[2], merge_ready, merge_done, done;
  uint64_t desc_full[kDescs], desc_empty[kDescs];
  Desc<kWindow> desc[kDescs];
  float2 ml[128];
  uint32_t tmem;
};

template <int D, bool kFp8, bool kWindow>
constexpr size_t smem_bytes() {
  using C = Cfg<D, kFp8>;
  return 1024 + static_cast<size_t>(C::kK + C::kV + 2) * C::kTile + 2 * C::kRaw +
         sizeof(Misc<kWindow>);
}
template <bool kWindow>
constexpr bool kFits =
    smem_bytes<128, false, kWindow>() <= 232448 && smem_bytes<64, false, kWindow>() <= 232448 &&
    smem_bytes<128, true, kWindow>() <= 232448 && smem_bytes<64, true, kWindow>() <= 232448;
static_assert(kFits<false> && kFits<true>, "227 KB a block");

// ---------------------------------------------------------------- the block's pipeline
// The ids of a piece's blocks, 32 at a time: lane l holds that of block l % nbt of tile
// l / nbt of the current group of tiles, the next group's already under way.
struct BlockIds {
  const int32_t* table;
  int bs, nbt, per_group;  // block size, blocks of a tile, tiles of a group
  int ja, nt, end, num_blocks;
  int group, ids, next;

  __device__ __forceinline__ int block_of(int gr, bool* used) const {
    const int lane = threadIdx.x & 31, t = gr * per_group + lane / nbt;
    const long long key = static_cast<long long>(ja + t) * kChunkKeys + (lane % nbt) * bs;
    *used = t < nt && key < end;
    return *used ? static_cast<int>(key / bs) : 0;
  }
  __device__ __forceinline__ int fetch(int gr) const {
    bool used;
    const int blk = block_of(gr, &used);
    return used ? table[blk] : 0;
  }
  __device__ __forceinline__ void start(const ChunkParams& p, const Desc<false>& d) {
    bs = p.block_size;
    nbt = bs >= kChunkKeys ? 1 : kChunkKeys / bs;
    per_group = 32 / nbt;
    table = p.block_tables + d.table;
    ja = d.ja;
    nt = d.jb - d.ja;
    end = d.end;
    num_blocks = p.num_blocks;
    group = -1;
    next = fetch(0);
  }
  // Makes tile t's group current; *bad_from falls to the first key of a block whose id is out
  // of range (any block stands in: the rows that see it become NaN).
  __device__ __forceinline__ void advance(int t, int* bad_from, int32_t* error_word) {
    if (t / per_group == group) return;
    group = t / per_group;
    ids = next;
    if (ids < 0 || ids >= num_blocks) {
      if (bad_from != nullptr) {
        bool used;
        const int blk = block_of(group, &used);
        const int tile = ja + group * per_group + (threadIdx.x & 31) / nbt;
        atomicMin(bad_from, max(blk * bs, tile * kChunkKeys));
        atomic_or_error(error_word, PDA_DEVERR_BLOCK_ID);
        __threadfence_block();
      }
      ids = 0;
    }
    __syncwarp();
    next = fetch(group + 1);
  }
  // Tiles of the piece; the key tile behind tile t, its blocks, and the keys from its first on
  // that some row may see.
  __device__ __forceinline__ int tiles() const { return nt; }
  __device__ __forceinline__ int blocks() const { return nbt; }
  __device__ __forceinline__ int keys(int t) const { return end - (ja + t) * kChunkKeys; }
  // Cache row of block `blk` of tile t (all lanes call).
  __device__ __forceinline__ int row(int t, int blk) const {
    const int id = __shfl_sync(kFullMask, ids, ((t - group * per_group) * nbt + blk) & 31);
    return id * bs + (bs > kChunkKeys ? ((ja + t) * kChunkKeys) % bs : 0);
  }
};

// The same with a window: tiles behind the first tokens' are `skip` key tiles further, and blocks
// that no row of the item sees are not looked up (block 0 stands in). *bad_from falls to 0 where
// an id is out of range: the rows look for themselves. Few registers: what the plan gives is read
// where it is used (with it in registers of their own, the loading warps spilled, and every tile
// took a seventh longer).
struct WindowIds {
  const ChunkParams& p;
  const Desc<true>* d;
  int group, ids, next;

  __device__ __forceinline__ int bs_log2() const { return __ffs(p.block_size) - 1; }
  __device__ __forceinline__ int nbt_log2() const { return max(0, 7 - bs_log2()); }
  __device__ __forceinline__ int group_log2() const { return 5 - nbt_log2(); }
  __device__ __forceinline__ int fetch(int gr) const {
    const int lane = threadIdx.x & 31, n = nbt_log2();
    const int t = (gr << (5 - n)) + (lane >> n), j = d->ja + t;
    if (j >= d->jb) return 0;
    const int key = d->key_tile(p, j) * kChunkKeys + ((lane & ((1 << n) - 1)) << bs_log2());
    const bool used = key < d->end && (key < p.sinks || key + p.block_size > d->lowest);
    return used ? p.block_tables[d->table + (key >> bs_log2())] : 0;
  }
  __device__ __forceinline__ void start(const ChunkParams&, const Desc<true>& piece) {
    d = &piece;
    group = -1;
    next = fetch(0);
  }
  __device__ __forceinline__ void advance(int t, int* bad_from, int32_t* error_word) {
    const int g = t >> group_log2();
    if (g == group) return;
    group = g;
    ids = next;
    if (ids < 0 || ids >= p.num_blocks) {
      if (bad_from != nullptr) {
        atomicMin(bad_from, 0);
        atomic_or_error(error_word, PDA_DEVERR_BLOCK_ID);
        __threadfence_block();
      }
      ids = 0;
    }
    __syncwarp();
    next = fetch(g + 1);
  }
  __device__ __forceinline__ int tiles() const { return d->jb - d->ja; }
  __device__ __forceinline__ int blocks() const { return 1 << nbt_log2(); }
  __device__ __forceinline__ int keys(int t) const {
    return d->end - d->key_tile(p, d->ja + t) * kChunkKeys;
  }
  __device__ __forceinline__ int row(int t, int blk) const {
    const int id = __shfl_sync(
        kFullMask, ids, (((t - (group << group_log2())) << nbt_log2()) + blk) & 31);
    const int r = id << bs_log2();
    return p.block_size > kChunkKeys && (d->key_tile(p, d->ja + t) & 1) != 0 ? r + kChunkKeys : r;
  }
};

struct Groups {
  int n0, n1;  // steps of each group
};
template <bool kWindow>
__device__ __forceinline__ Groups groups_of(const Desc<kWindow>& d) {
  const int nt = d.jb - d.ja;
  if (d.single) return Groups{(nt + 1) >> 1, nt >> 1};
  return Groups{max(0, min(d.jb, d.tiles0) - d.ja), max(0, min(d.jb, d.tiles1) - d.ja)};
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// This warp's quarter of a tile of E4M3 codes, [128][D] bytes: NaN codes of the first `keys` rows
// become zeros, and their rows' bits are set in `nonfinite`.
template <int D>
__device__ __forceinline__ void clean_codes(unsigned char* codes, int part, int keys,
                                            unsigned* nonfinite) {
  constexpr int kLanes = D / 16;  // lanes of a row, 16 codes each
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int i = 0; i < kLanes; ++i) {
    const int r = 32 * part + i * (32 / kLanes) + lane / kLanes;
    uint4* at = reinterpret_cast<uint4*>(codes + r * D) + lane % kLanes;
    uint4 v = *at;
    uint32_t* w = &v.x;
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t hit = ((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
      w[k] &= ~((hit >> 7) * 0xffu);
      any |= hit;
    }
    if (any != 0 && r < keys) {
      *at = v;
      atomicOr(&nonfinite[r >> 5], 1u << (r & 31));
    }
  }
  __syncwarp();
}

// Widens this warp's quarter of a tile of E4M3 codes to fp16 in the products' layout (64-element
// halves, 128-byte swizzle). Rows from `keys` on become zeros.
template <int D>
__device__ __forceinline__ void widen(unsigned char* dst, const unsigned char* codes, int part,
                                      int keys) {
  constexpr int kLanes = D / 16, kBatch = 4;
  const int lane = threadIdx.x & 31, c = 2 * (lane % kLanes);
  // lanes of the second half take their pieces the other way round: no bank conflicts
  const bool swap = c >= 8;
#pragma unroll 1
  for (int i0 = 0; i0 < kLanes; i0 += kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = 32 * part + (i0 + i) * (32 / kLanes) + lane / kLanes;
      v[i] = r < keys ? *reinterpret_cast<const uint4*>(codes + r * D + 8 * c)
                      : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = 32 * part + (i0 + i) * (32 / kLanes) + lane / kLanes;
      uint4 o[2];
      e4m3x4_to_f16x2(v[i].x, o[0].x, o[0].y);
      e4m3x4_to_f16x2(v[i].y, o[0].z, o[0].w);
      e4m3x4_to_f16x2(v[i].z, o[1].x, o[1].y);
      e4m3x4_to_f16x2(v[i].w, o[1].z, o[1].w);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int piece = c + (swap ? 1 - k : k);
        *reinterpret_cast<uint4*>(dst + (piece >> 3) * (kChunkKeys * 128) + r * 128 +
                                  (((piece & 7) ^ (r & 7)) << 4)) = swap == (k == 0) ? o[1] : o[0];
      }
    }
  }
}

// One row of Q, D bf16 values, into row r of a tile in the products' layout as fp16, scaled by a
// power of two that puts its largest value into [2^14, 2^15). Returns the factor that undoes it.
// `store`: false only finds the factor.
template <int D>
__device__ __forceinline__ float scale_q_row(const uint4* row, unsigned char* tile, int r,
                                             bool store) {
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    const uint4 v = row[c];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7fffu, w[k] >> 16 & 0x7fffu));
  }
  // the largest value's exponent field; 15 keeps the factor's own exponent in range
  const int e = max(static_cast<int>(top >> 7), 15);
  const float up = __uint_as_float(static_cast<uint32_t>(min(268 - e, 253)) << 23);
  if (store) {
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
      const uint4 v = row[c];
      const uint4 o = make_uint4(pack2<false>(bf16_lo(v.x) * up, bf16_hi(v.x) * up),
                                 pack2<false>(bf16_lo(v.y) * up, bf16_hi(v.y) * up),
                                 pack2<false>(bf16_lo(v.z) * up, bf16_hi(v.z) * up),
                                 pack2<false>(bf16_lo(v.w) * up, bf16_hi(v.w) * up));
      *reinterpret_cast<uint4*>(tile + (c >> 3) * (kChunkKeys * 128) + r * 128 +
                                (((c & 7) ^ (r & 7)) << 4)) = o;
    }
  }
  return 1.f / up;
}

// Cleans this warp's quarter of a V tile of `keys` rows, in boxes of `box_rows` rows: zeroes what
// the products read behind them, and replaces non-finite values by zeros, setting their rows'
// bits in `nonfinite`.
template <int D, bool kBf16>
__device__ __forceinline__ void clean_tile(unsigned char* tile, int part, int keys, int box_rows,
                                           unsigned* nonfinite) {
  constexpr uint32_t kMask = kBf16 ? 0x7f807f80u : 0x7c007c00u;
  constexpr uint32_t kOne = kBf16 ? 0x00800080u : 0x04000400u;
  const int lane = threadIdx.x & 31;
  const int rows = (keys + 15) & ~15;
  // a lane takes one 16-byte chunk of each 128-byte half of every fourth row
  auto chunk = [&](int i) {
    const int h = D == 128 ? i & 1 : 0, r = 32 * part + 4 * (D == 128 ? i >> 1 : i) + (lane >> 3);
    return reinterpret_cast<uint4*>(tile + (r & ~(box_rows - 1)) * (D * 2) +
                                    (h * box_rows + (r & (box_rows - 1))) * 128) + (lane & 7);
  };
  auto row = [&](int i) { return 32 * part + 4 * (D == 128 ? i >> 1 : i) + (lane >> 3); };
  // exponents of all ones carry into the sign's place when one is added
  auto hits = [&](uint32_t w) { return ((w & kMask) + kOne) & 0x80008000u; };
  uint32_t any = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < D / 8; i0 += 4) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *chunk(i0 + i);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row(i0 + i) < keys) any |= hits(v[i].x) | hits(v[i].y) | hits(v[i].z) | hits(v[i].w);
  }
  if (keys < kChunkKeys)
#pragma unroll 1
    for (int i = 0; i < D / 8; ++i)
      if (row(i) >= keys && row(i) < rows) *chunk(i) = make_uint4(0, 0, 0, 0);
  if (!__any_sync(kFullMask, any != 0)) return;
#pragma unroll 1
  for (int i = 0; i < D / 8; ++i) {
    if (row(i) >= keys) continue;
    uint4 v = *chunk(i);
    uint32_t* e = &v.x;
    uint32_t all = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t hit = hits(e[k]);
      e[k] &= ~((hit >> 15) * 0xffffu);
      all |= hit;
    }
    if (all != 0) {
      *chunk(i) = v;
      atomicOr(&nonfinite[row(i) >> 5], 1u << (row(i) & 31));
    }
  }
}

// A mask of the n lowest bits (none where n < 0, 32 at most).
__device__ __forceinline__ uint32_t low_bits(int n) {
  uint32_t r;
  asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(r) : "r"(max(n, 0)));
  return r;
}

// Lane q of each quad gives v[c] = its 16 bytes number c and gets v[r] = bytes number q of
// the quad's lane r.
__device__ __forceinline__ void quad_transpose(uint4* v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int step = 1; step < 4; step <<= 1) {
    const bool up = lane & step;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c & step) continue;
      uint4& lo = v[c];
      uint4& hi = v[c + step];
      const uint4 give = up ? lo : hi;
      uint4 take;
      take.x = __shfl_xor_sync(kFullMask, give.x, step);
      take.y = __shfl_xor_sync(kFullMask, give.y, step);
      take.z = __shfl_xor_sync(kFullMask, give.z, step);
      take.w = __shfl_xor_sync(kFullMask, give.w, step);
      if (up)
        lo = take;
      else
        hi = take;
    }
  }
}

template <int D, bool kBf16, bool kFp8, bool kWindow>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const ChunkParams p, int g_shift,
                    float* partial) {
  static_assert(kBf16 || !kFp8, "q and out are bf16 over a cache of codes");
  constexpr bool kOpBf16 = kBf16 && !kFp8;  // the products' operands
  using C = Cfg<D, kFp8>;
  using Cuts = CutsOf<kWindow>;
  using Piece = Desc<kWindow>;
  using Ids = std::conditional_t<kWindow, WindowIds, BlockIds>;
  auto new_ids = [&] {
    if constexpr (kWindow)
      return WindowIds{p};
    else
      return BlockIds{};
  };
  constexpr int kDescs = kDescsOf<kWindow>, kEdges = kEdgesOf<kWindow>;
  constexpr int NK = C::kK, NV = C::kV;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* ks = smem;
  unsigned char* vs = ks + NK * C::kTile;
  unsigned char* qs = vs + NV * C::kTile;
  unsigned char* raw = qs + 2 * C::kTile;  // codes: a K tile, then a V tile
  Misc<kWindow>& ms = *reinterpret_cast<Misc<kWindow>*>(raw + 2 * C::kRaw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lt = Cuts::kRowsLog2 - g_shift;

  // the merge kernel may start its own prologue as soon as blocks leave
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < 5; ++i) {
      mbar_init(&ms.k_full[i], kFp8 ? kCleaners : 1);
      mbar_init(&ms.k_empty[i], 1);
      mbar_init(&ms.v_full[i], 1);
      mbar_init(&ms.v_empty[i], 1);
      mbar_init(&ms.clean[i], kCleaners);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.raw_full[i], 1);
      mbar_init(&ms.raw_empty[i], kCleaners);
    }
    mbar_init(&ms.q_full, kFp8 ? 4 : 1);  // a group's softmax warps, or the copy
    mbar_init(&ms.q_full1, 4);
    mbar_init(&ms.q_empty, 1);
    for (int g = 0; g < 2; ++g) {
      mbar_init(&ms.s_full[g], 1);
      mbar_init(&ms.p_full[g], 128);
      mbar_init(&ms.o_full[g], 1);
    }
    mbar_init(&ms.merge_ready, 128);
    mbar_init(&ms.merge_done, 128);
    mbar_init(&ms.done, 1);
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(&ms.desc_full[i], 1);
      mbar_init(&ms.desc_empty[i], 1 + 1 + kCleaners + 8);  // all that read it
    }
    fence_mbar_init();
  }
  if (tid == 32) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == 9) {
    tmem_alloc(&ms.tmem, 512);
    tmem_relinquish();
  }
  const Plan pl = make_plan<Cuts>(p, lt, gridDim.x, reinterpret_cast<PlanMemory*>(ks));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;

  bool timed_out = false;
  if (warp < 8) {
    reg_inc<kSoftmaxRegs>();
    // ================================================================ softmax and output
    const int g = warp >> 2;
    const int row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // lane 32 (warp % 4) << 16
    const uint32_t tS = tmem + lanes + g * 128, tO = tmem + lanes + 256 + g * 128;
    // never 0: masked scores are -inf times this
    const float least = __uint_as_float(1), sl_all = fmaxf(fabsf(p.scale_log2), least);
    // fp16 probabilities are kept 2^4 higher (the factor cancels in O / l): with the
    // reference up to 2^8 below the maximum they stay below 2^13, and only those under 2^-18 of
    // the reference are subnormal
    const float lift = kOpBf16 ? 0.f : 4.f;
    unsigned s_phase = 0, o_phase = 0, m_phase = 0;
    for (int item = 0; !timed_out; ++item) {
      const int slot = item % kDescs;
      if (!warp_wait(&ms.desc_full[slot], (item / kDescs) & 1)) {
        timed_out = true;
        break;
      }
      const Piece& d = ms.desc[slot];
      if (!d.valid) break;
      const Groups gr = groups_of(d);
      const int steps = g == 0 ? gr.n0 : gr.n1;
      const bool single = d.single != 0;
      const int ja = d.ja;
      const int packed = single ? row : g * 128 + row;
      const int tok = packed >> g_shift;
      const int pos = d.pos0 + min(tok, d.tokens - 1);  // this row's position
      const int first_pos = d.pos0 + ((single ? 0 : g * 128) >> g_shift);
      float sl = sl_all;  // of a score, in log2 units
      if (kFp8) {
        // this row of Q; where the groups share their rows, group 0's warps store it
        if (!warp_wait(&ms.q_empty, (item & 1) ^ 1)) {
          timed_out = true;
          break;
        }
        const int there = min(tok, d.tokens - 1);
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(p.q) +
            ((static_cast<size_t>(d.row0) + there) * p.H + (d.kh << g_shift) +
             (packed & ((1 << g_shift) - 1))) * D);
        const float back = scale_q_row<D>(src, qs + (single ? 0 : g * C::kTile), row,
                                          g == 0 || !single);
        // times the row's factor, up to 2^113, the floor of a scale of zero would count
        sl = p.scale_log2 == 0.f ? least : fmaxf(least, sl * back);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(g == 0 ? &ms.q_full : &ms.q_full1);
      }
      float m = -INFINITY, l = 0.f;
      for (int s = 0; s < steps; ++s) {
        const int key0 = d.key_tile(p, ja + (single ? 2 * s + g : s)) * kChunkKeys;
        if (!warp_wait(&ms.s_full[g], s_phase)) {
          timed_out = true;
          break;
        }
        s_phase ^= 1;
        tc_fence_after();
        float x[kChunkKeys];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32(x + 32 * k, tS + 32 * k);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < kChunkKeys; k += 32) tmem_arrived32(x + k);
        if constexpr (kWindow) {
          // masked where some row of this warp does not see the whole tile, by a bit per key
          const int warp_pos = __shfl_sync(kFullMask, pos, 0);
          const int warp_end = __shfl_sync(kFullMask, pos, 31);
          if (key0 + kChunkKeys - 1 > warp_pos ||
              (key0 <= warp_end - p.window && key0 + kChunkKeys > p.sinks)) {
#pragma unroll
            for (int k0 = 0; k0 < kChunkKeys; k0 += 32) {
              const int at = key0 + k0;
              const uint32_t seen = low_bits(pos + 1 - at) &
                                    (~low_bits(pos - p.window + 1 - at) | low_bits(p.sinks - at));
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(seen >> k & 1)) x[k0 + k] = -INFINITY;
            }
          }
        } else if (key0 + kChunkKeys - 1 > first_pos) {
          const int seen = pos - key0;
#pragma unroll
          for (int k = 0; k < kChunkKeys; ++k)
            if (k > seen) x[k] = -INFINITY;
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int k = 4; k + 4 < kChunkKeys; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[k + 2 * e], x[k + 2 * e + 1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[kChunkKeys - 4 + e]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (s == 0) {
          m = top;
        } else {
          const bool raise = top > m && (top - m) * sl > kRaise;
          if (__any_sync(kFullMask, raise)) {
            const float c = raise ? ex2((m - top) * sl) : 1.f;
            if (raise) m = top;
            l *= c;
            // the product of the step before is complete: its successor's scores are
#pragma unroll 1
            for (int k = 0; k < D; k += 16) {
              float o[16];
              tmem_ld16(o, tO + k);
              tmem_wait_ld();
              tmem_arrived16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= c;
              tmem_st16(tO + k, reinterpret_cast<const uint32_t*>(o));
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : lift - m * sl;
        const float2 sl2 = make_float2(sl, sl), ref2 = make_float2(ref, ref);
        float2 sum[2] = {};
#pragma unroll
        for (int k = 0; k < kChunkKeys; k += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float2 a = __ffma2_rn(make_float2(x[k + e], x[k + e + 1]), sl2, ref2);
            a.x = ex2(a.x);
            a.y = ex2(a.y);
            sum[(e >> 1) & 1] = __fadd2_rn(sum[(e >> 1) & 1], a);
            pk[e / 2] = pack2<kOpBf16>(a.x, a.y);
          }
          tmem_st16(tS + k / 2, pk);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&ms.p_full[g]);
      }
      if (timed_out) break;
      // ---- the piece's rows
      if (steps > 0) {
        if (!warp_wait(&ms.o_full[g], o_phase)) {
          timed_out = true;
          break;
        }
        o_phase ^= 1;
        tc_fence_after();
      }
      float m1 = -INFINITY, l1 = 0.f;  // group 1's, where the groups share their rows
      const bool other = single && gr.n1 > 0;
      if (other) {
        if (g == 1) {
          ms.ml[row] = make_float2(m, l);
          tc_fence_before();
          mbar_arrive(&ms.merge_ready);
          if (!warp_wait(&ms.merge_done, m_phase)) {
            timed_out = true;
            break;
          }
        } else {
          if (!warp_wait(&ms.merge_ready, m_phase)) {
            timed_out = true;
            break;
          }
          tc_fence_after();
          const float2 v = ms.ml[row];
          m1 = v.x;
          l1 = v.y;
        }
        m_phase ^= 1;
      }
      if (g == 0 || !single) {
        const float top = fmaxf(m, m1);
        const float c0 = m == -INFINITY ? 0.f : ex2((m - top) * sl);
        const float c1 = m1 == -INFINITY ? 0.f : ex2((m1 - top) * sl);
        l = l * c0 + (other ? l1 * c1 : 0.f);
        bool dead = pos >= d.bad_from;
        if constexpr (kWindow)
          if (dead) dead = sees_bad_block(p, p.block_tables + d.table, pos);
        const bool write = tok < d.tokens;
        const int part = d.slot;
        bool odd = false;
        if (kWindow || d.jb > d.jc)
          for (int k = 0; k < 4 * kEdges; ++k) odd |= d.nonfinite[k >> 2][k & 3] != 0;
        const float inv = dead ? NAN : part >= 0 ? 1.f : p.v_scale / l;
        if (part >= 0 && write)
          part_ml(partial, part, D)[packed] =
              make_float2(steps > 0 && top != -INFINITY ? top * sl : -INFINITY, dead ? NAN : l);
        // rows of this lane's quad: the first one's place in the output, the steps to the other
        // three, and how many of them are the item's
        const int quad = packed & ~3, HD = p.H * D;
        const int step1 = g_shift == 0 ? HD : D;
        const int step2 = g_shift == 0 ? 2 * HD : g_shift == 1 ? HD : 2 * D;
        const int in_quad = (d.tokens << g_shift) - quad;
        uint16_t* out = static_cast<uint16_t*>(p.out) +
                        (static_cast<size_t>(d.row0 + (quad >> g_shift)) * p.H + (d.kh << g_shift) +
                         (quad & ((1 << g_shift) - 1))) * D + 8 * (lane & 3);
        const float f0 = c0 * inv, f1 = c1 * inv;
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
          float o[32];
          if (steps > 0) {
            tmem_ld32(o, tO + k);
            tmem_wait_ld();
            tmem_arrived32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f0;
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
          }
          if (other) {
            float o1[32];
            tmem_ld32(o1, tO + 128 + k);
            tmem_wait_ld();
            tmem_arrived32(o1);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(o1[e], f1, o[e]);
          }
          if (part >= 0) {
            // four columns of a row, rows side by side: a warp writes 512 bytes at a time
            if (write) {
              float4* dst = part_o(partial, part, D) + (k / 4) * 256 + packed;
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                dst[(e / 4) * 256] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          } else {
            // a lane holds 64 bytes of its row; exchanged within quads, four lanes store the
            // 64 bytes of one row together (a row per lane would take four times the passes)
            uint4 v[4];
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              v[e / 8] =
                  make_uint4(pack2<kBf16>(o[e], o[e + 1]), pack2<kBf16>(o[e + 2], o[e + 3]),
                             pack2<kBf16>(o[e + 4], o[e + 5]), pack2<kBf16>(o[e + 6], o[e + 7]));
            quad_transpose(v);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (r < in_quad)
                *reinterpret_cast<uint4*>(out + (r & 1) * step1 + (r >> 1) * step2 + k) = v[r];
          }
          __syncwarp();
        }
        if (odd && write) {  // non-finite V values, for the rows that see them (__syncwarp: the
                             // row's values, stored by its quad, are this thread's to change)
#pragma unroll 1
          for (int y = 0; y < 128 * kEdges; ++y) {
            if (!((d.nonfinite[y >> 7][(y >> 5) & 3] >> (y & 31)) & 1)) continue;
            const int key = d.edge_tile(p, y >> 7) * kChunkKeys + (y & 127);
            if (key > pos) continue;
            if (kWindow && key >= p.sinks && key <= pos - p.window) continue;
            const int id = p.block_tables[d.table + key / p.block_size];
            if (id < 0 || id >= p.num_blocks) continue;
            const size_t first =
                ((static_cast<size_t>(id) * p.block_size + key % p.block_size) * p.H_kv + d.kh) * D;
#pragma unroll 1
            for (int k = 0; k < D; ++k) {
              float f;
              if (kFp8) {
                f = e4m3_to_f32(static_cast<const uint8_t*>(p.v_cache)[first + k]);
              } else {
                const uint16_t u = static_cast<const uint16_t*>(p.v_cache)[first + k];
                f = kBf16 ? __uint_as_float(static_cast<uint32_t>(u) << 16)
                          : __half2float(__ushort_as_half(u));
              }
              if (isfinite(f)) continue;
              if (part >= 0) {
                float* at =
                    reinterpret_cast<float*>(part_o(partial, part, D) + (k / 4) * 256 + packed) +
                    (k & 3);
                *at = fmaf(f, inv, *at);
              } else {
                using Out = std::conditional_t<kBf16, __nv_bfloat16, __half>;
                Out* at = static_cast<Out*>(p.out) +
                          ((static_cast<size_t>(d.row0) + tok) * p.H + (d.kh << g_shift) +
                           (packed & ((1 << g_shift) - 1))) * D + k;
                *at = static_cast<Out>(fmaf(f, inv, static_cast<float>(*at)));
              }
            }
          }
        }
        if (other) {
          tc_fence_before();
          mbar_arrive(&ms.merge_done);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.desc_empty[slot]);
    }
  } else {
    reg_dec<kOtherRegs>();
    if (warp == 8) {
      // ================================================================ plan, load Q and K
      Where<Cuts> w{};
      int u = 0, u_end = 0;
      if (static_cast<int>(blockIdx.x) < pl.workers && pl.units > 0) {
        // both ends of the range at once: the odd lanes find the upper one
        u = cut_of<Cuts>(p, pl, lt, blockIdx.x + (lane & 1), &w);
        u_end = __shfl_sync(kFullMask, u, 1);
        u = __shfl_sync(kFullMask, u, 0);
        w.b = __shfl_sync(kFullMask, w.b, 0);
        w.kh = __shfl_sync(kFullMask, w.kh, 0);
        w.i = __shfl_sync(kFullMask, w.i, 0);
        w.start = __shfl_sync(kFullMask, w.start, 0);
        w.q.row0 = __shfl_sync(kFullMask, w.q.row0, 0);
        w.q.r.n = __shfl_sync(kFullMask, w.q.r.n, 0);
        w.q.r.L = __shfl_sync(kFullMask, w.q.r.L, 0);
        w.q.r = request<Cuts>(p, w.q.r.n, w.q.r.L, lt);
        if (u < u_end && u >= w.start + w.q.r.tiles(w.i) + kItemUnits) next_item(p, lt, &w);
      }
      __syncwarp();
      fence_proxy_async_smem();  // the plan's shared memory becomes load stages
      int item = 0;
      int k_at = 0, k_turn = 0;
      while (u < u_end && !timed_out) {
        const typename Cuts::Request r = w.q.r;
        const int tiles = r.tiles(w.i);
        const int end = w.start + tiles + kItemUnits;
        const int tok0 = w.i << lt, tokens = min(1 << lt, r.n - tok0);
        const int ja = u == w.start ? 0 : u - w.start - kItemUnits;
        const int jb = u_end >= end ? tiles : u_end - w.start - kItemUnits;
        const int slot = item % kDescs;
        Piece& d = ms.desc[slot];
        if (!warp_wait(&ms.desc_empty[slot], ((item / kDescs) & 1) ^ 1)) {
          timed_out = true;
          break;
        }
        const int pos0 = r.L - r.n + tok0;
        const int half = 128 >> g_shift;  // tokens of a row group
        const bool single = tokens <= half;
        const int kv_end = pos0 + tokens;
        const long long table = static_cast<long long>(w.b) * p.max_blocks;
        const int row0 = w.q.row0 + tok0;
        if (lane == 0) {
          d.valid = 1;
          d.row0 = row0;
          d.tokens = tokens;
          d.pos0 = pos0;
          d.kh = w.kh;
          d.ja = ja;
          d.jb = jb;
          d.tiles0 = single ? tiles : ((pos0 + half - 1) >> 7) + 1;
          if constexpr (kWindow) {
            d.skip = r.skipped(w.i);
            d.lowest = r.lowest(w.i);
            d.last_lowest = max(0, kv_end - p.window);
            if (!single) d.tiles0 -= d.skip;
          }
          d.tiles1 = tiles;
          d.single = single;
          d.jc = (pos0 + 1) >> 7;
          d.end = kv_end;
          d.slot =
              ja == 0 && jb == tiles ? -1 : static_cast<int>(blockIdx.x) * 2 + (ja == 0 ? 1 : 0);
          d.bad_from = 0x7fffffff;
          d.table = table;
          for (int k = 0; k < 4 * kEdges; ++k) d.nonfinite[k >> 2][k & 3] = 0;
          mbar_arrive(&ms.desc_full[slot]);
        }
        __syncwarp();
        // Q (over codes the softmax warps bring it)
        if (!kFp8) {
          if (!warp_wait(&ms.q_empty, (item & 1) ^ 1)) {
            timed_out = true;
            break;
          }
          const int q_tiles = single ? 1 : 2;
          if (lane == 0) mbar_arrive_expect_tx(&ms.q_full, q_tiles * C::kTile);
          __syncwarp();
          if (lane < q_tiles * C::kHalves) {
            const int g = lane / C::kHalves, h = lane % C::kHalves;
            tma_box(qs + g * C::kTile + h * C::kHalf, &tm_q, 64 * h, w.kh << g_shift,
                    row0 + g * half, &ms.q_full);
          }
        }
        // K: a box of a block's rows (128 at most), for each 64-element half of a row, or of codes
        const int nt = jb - ja;
        const int box_rows = min(p.block_size, kChunkKeys);
        Ids ids = new_ids();
        ids.start(p, d);
        for (int t = 0; t < nt; ++t) {
          ids.advance(t, &d.bad_from, p.error_word);
          uint64_t* full = kFp8 ? &ms.raw_full[0] : &ms.k_full[k_at];
          if (!warp_wait(kFp8 ? &ms.raw_empty[0] : &ms.k_empty[k_at], k_turn ^ 1)) {
            timed_out = true;
            break;
          }
          const int keys = ids.keys(t);
          const int boxes = min(ids.blocks(), (keys + box_rows - 1) / box_rows);
          if (lane == 0)
            mbar_arrive_expect_tx(full, boxes * box_rows * (kFp8 ? D : 2 * D));
          __syncwarp();
          constexpr int kParts = kFp8 ? 1 : C::kHalves;
          const int blk = lane / kParts, h = lane % kParts;
          const int row = ids.row(t, blk);
          if (blk < boxes)
            tma_box(kFp8 ? raw + blk * box_rows * D
                         : ks + k_at * C::kTile + h * C::kHalf + blk * box_rows * 128,
                    &tm_k, 64 * h, w.kh, row, full);
          if (++k_at == (kFp8 ? 1 : NK)) {
            k_at = 0;
            k_turn ^= 1;
          }
        }
        ++item;
        // the next item
        u = end;
        if (u < u_end) next_item(p, lt, &w);
      }
      if (!timed_out) {
        const int slot = item % kDescs;
        if (warp_wait(&ms.desc_empty[slot], ((item / kDescs) & 1) ^ 1)) {
          if (lane == 0) {
            ms.desc[slot].valid = 0;
            mbar_arrive(&ms.desc_full[slot]);
          }
        } else {
          timed_out = true;
        }
      }
      if (timed_out) {
        // copies in flight land before the block may leave
        for (int st = 0; st < (kFp8 ? 1 : 5); ++st)
          for (int turn = 0; turn < 2; ++turn)
            warp_wait(kFp8 ? &ms.raw_full[0] : &ms.k_full[st], turn);
        if (!kFp8) {
          warp_wait(&ms.q_full, 0);
          warp_wait(&ms.q_full, 1);
        }
      }
    } else if (warp == 9) {
      // ================================================================ matrix instructions
      // The whole warp walks the steps, so that descriptors stay in uniform registers; one
      // elected lane issues.
      const bool leader = elect_one();
      const bool negate = p.scale_log2 < 0.f;  // S is compared and scaled by |scale|
      const uint32_t id_qk = mma_idesc(kOpBf16, kChunkKeys, negate, false);
      const uint32_t id_pv = mma_idesc(kOpBf16, D, false, true);
      // descriptors as (address, rest) words: moving along a tile changes the address alone
      const uint64_t dk = smem_desc_sw128(smem_addr(ks), 16, 1024);
      const uint64_t dq = smem_desc_sw128(smem_addr(qs), 16, 1024);
      const uint32_t dk0 = static_cast<uint32_t>(dk), dq0 = static_cast<uint32_t>(dq);
      const uint32_t hi_qk = static_cast<uint32_t>(dk >> 32);
      auto desc = [](uint32_t lo, uint32_t hi) { return static_cast<uint64_t>(hi) << 32 | lo; };
      const int box_rows = kFp8 ? kChunkKeys : min(p.block_size, kChunkKeys);
      const uint64_t dv = smem_desc_sw128(smem_addr(vs), box_rows * 128, 1024);
      const uint32_t dv0 = static_cast<uint32_t>(dv), hi_v = static_cast<uint32_t>(dv >> 32);
      // 16, 32 and 64 rows further down: in the same box, or past the boxes in between
      auto rows_down = [&](int n) {
        return static_cast<uint32_t>(n < box_rows ? n * 128 : n * D * 2) >> 4;
      };
      const uint32_t v_step1 = rows_down(16), v_step2 = rows_down(32), v_step4 = rows_down(64);
      int k_at = 0, k_turn = 0, v_at = 0, v_turn = 0;  // stage and parity of the next K, V tile
      unsigned p_phase = 0;
      for (int item = 0; !timed_out; ++item) {
        const int slot = item % kDescs;
        if (!warp_wait(&ms.desc_full[slot], (item / kDescs) & 1)) {
          timed_out = true;
          break;
        }
        const Piece& d = ms.desc[slot];
        if (!__shfl_sync(kFullMask, d.valid, 0)) break;
        const Groups grp = groups_of(d);
        const int n0 = __shfl_sync(kFullMask, grp.n0, 0), n1 = __shfl_sync(kFullMask, grp.n1, 0);
        const bool single = __shfl_sync(kFullMask, d.single, 0) != 0;
        // keys the rows may see from the piece's first tile on
        const int keys = __shfl_sync(kFullMask, d.end - d.ja * kChunkKeys, 0);
        int piece_sinks = 0, skip_keys = 0;  // the piece's tiles before the gap, and its keys
        if constexpr (kWindow) {
          piece_sinks = __shfl_sync(kFullMask, p.sink_tiles - d.ja, 0);
          skip_keys = __shfl_sync(kFullMask, d.skip * kChunkKeys, 0);
        }
        const int steps = max(n0, n1), last_g = n1 >= n0 ? 1 : 0;
        if (!warp_wait(&ms.q_full, item & 1)) {
          timed_out = true;
          break;
        }
        tc_fence_after();
        // A tile is used by both groups, the second releasing it, or (single) by one.
        auto qk = [&](int g, int s) {
          if (leader) {
            const uint32_t a = dq0 + (single ? 0 : g * (C::kTile >> 4));
            const uint32_t b = dk0 + k_at * (C::kTile >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = ((k >> 2) * C::kHalf + (k & 3) * 32) >> 4;
              mma_f16_ss(tmem + g * 128, desc(a + off, hi_qk), desc(b + off, hi_qk), id_qk, k > 0);
            }
            mma_commit(&ms.s_full[g]);
            if (single || g == 1) mma_commit(&ms.k_empty[k_at]);
            if (g == last_g && s == steps - 1) mma_commit(&ms.q_empty);
          }
          if (single || g == 1) {
            if (++k_at == NK) {
              k_at = 0;
              k_turn ^= 1;
            }
          }
        };
        // Group g's P V of step s and its Q K of the next, issued back to back and run in that
        // order (see TMEM above: the second writes where the first reads). Their three
        // barriers are polled at once, a lane each: one wait after the other left the tensor
        // core idle for a fifth of the time.
        auto step = [&](int g, int s, int n) {
          const bool more = s + 1 < n;
          uint64_t* bar = &ms.p_full[g];
          uint32_t turn = (p_phase >> g) & 1;
          if (lane == 1) {
            bar = &ms.clean[v_at];
            turn = v_turn;
          } else if (lane == 2 && more) {
            bar = &ms.k_full[k_at];
            turn = k_turn;
          }
          if (!warp_wait(bar, turn)) return false;
          p_phase ^= 1u << g;
          tc_fence_after();
          int left = keys - (single ? 2 * s + g : s) * kChunkKeys;
          if constexpr (kWindow)
            if ((single ? 2 * s + g : s) >= piece_sinks) left -= skip_keys;
          if (leader) {
            const uint32_t b = dv0 + v_at * (C::kTile >> 4);
#pragma unroll
            for (int k = 0; k < kChunkKeys / 16; ++k)
              if (16 * k < left)
                mma_f16_ts(
                    tmem + 256 + g * 128, tmem + g * 128 + 8 * k,
                    desc(b + (k & 1) * v_step1 + (k >> 1 & 1) * v_step2 + (k >> 2) * v_step4, hi_v),
                    id_pv, s > 0 || k > 0);
            if (single || g == 1) mma_commit(&ms.v_empty[v_at]);
            if (!more) mma_commit(&ms.o_full[g]);
          }
          if (single || g == 1) {
            if (++v_at == NV) {
              v_at = 0;
              v_turn ^= 1;
            }
          }
          if (more) qk(g, s + 1);
          __syncwarp();
          return true;
        };
        bool ok = true;
        // group 1's warps bring their Q at their own pace; an item without steps of theirs waits
        // for them all the same, so that they see every turn of q_empty
        if (kFp8 && n1 == 0) ok = warp_wait(&ms.q_full1, item & 1);
        if (ok && n0 > 0) {
          ok = warp_wait(&ms.k_full[k_at], k_turn);
          tc_fence_after();
          if (ok) qk(0, 0);
        }
        if (kFp8 && ok && n1 > 0) ok = warp_wait(&ms.q_full1, item & 1);
        if (ok && n1 > 0) {
          ok = warp_wait(&ms.k_full[k_at], k_turn);
          tc_fence_after();
          if (ok) qk(1, 0);
        }
        for (int s = 0; ok && s < steps; ++s) {
          if (s < n0) ok = step(0, s, n0);
          if (ok && s < n1) ok = step(1, s, n1);
        }
        if (!ok) {
          timed_out = true;
          break;
        }
        if (lane == 0) mbar_arrive(&ms.desc_empty[slot]);
      }
      // nothing of this warp's is in flight when the block gives its TMEM back
      if (leader) mma_commit(&ms.done);
      if (!warp_wait(&ms.done, 0)) timed_out = true;
    } else if (warp == 10) {
      // ================================================================ load V
      // A block's rows (128 at most) come as one box, both halves of its rows one behind the
      // other: the P V product takes 16 rows of one block at a time, so blocks need not join.
      int v_at = 0, v_turn = 0;
      for (int item = 0; !timed_out; ++item) {
        const int slot = item % kDescs;
        if (!warp_wait(&ms.desc_full[slot], (item / kDescs) & 1)) {
          timed_out = true;
          break;
        }
        const Piece& d = ms.desc[slot];
        if (!d.valid) break;
        const int box_rows = min(p.block_size, kChunkKeys);
        const int kh = d.kh;
        Ids ids = new_ids();
        ids.start(p, d);
        for (int t = 0; t < ids.tiles(); ++t) {
          ids.advance(t, nullptr, nullptr);
          uint64_t* full = kFp8 ? &ms.raw_full[1] : &ms.v_full[v_at];
          if (!warp_wait(kFp8 ? &ms.raw_empty[1] : &ms.v_empty[v_at], v_turn ^ 1)) {
            timed_out = true;
            break;
          }
          const int keys = ids.keys(t);
          const int boxes = min(ids.blocks(), (keys + box_rows - 1) / box_rows);
          if (lane == 0) mbar_arrive_expect_tx(full, boxes * box_rows * (kFp8 ? D : 2 * D));
          __syncwarp();
          const int row = ids.row(t, lane);
          if (lane < boxes) {
            if (kFp8)
              tma_box(raw + C::kRaw + lane * box_rows * D, &tm_v, 0, kh, row, full);
            else
              tma_box4(vs + v_at * C::kTile + lane * box_rows * D * 2, &tm_v, 0, row, 0, kh, full);
          }
          if (++v_at == (kFp8 ? 1 : NV)) {
            v_at = 0;
            v_turn ^= 1;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.desc_empty[slot]);
      }
      if (timed_out)
        for (int st = 0; st < (kFp8 ? 1 : 5); ++st)
          for (int turn = 0; turn < 2; ++turn)
            warp_wait(kFp8 ? &ms.raw_full[1] : &ms.v_full[st], turn);
    } else if (warp == 11) {
      // ================================================================ rows without work
      // requests whose rows are written all the same: padded (zeros) or in error (NaN)
      if (!pl.ok && blockIdx.x == 0 && lane == 0) atomic_or_error(p.error_word, PDA_DEVERR_QUERY);
      for (int first = pl.ok ? blockIdx.x : p.B; first < p.B; first += 32 * gridDim.x) {
        const int b = first + lane * gridDim.x;
        int q0 = 0, q1 = 0, L = 0;
        if (b < p.B && chunk_req<Cuts>(p, b, lt).r.n == 0) {
          q0 = p.query_start[b];
          q1 = p.query_start[b + 1];
          L = p.context_lens[b];
          if (q0 < q1 && L != 0) atomic_or_error(p.error_word, PDA_DEVERR_CONTEXT_LEN);
        }
        for (unsigned todo = __ballot_sync(kFullMask, q0 < q1); todo != 0; todo &= todo - 1) {
          const int from = __ffs(todo) - 1;
          const int r0 = __shfl_sync(kFullMask, q0, from), r1 = __shfl_sync(kFullMask, q1, from);
          // 0x7fff is a NaN in either type
          const uint32_t v = __shfl_sync(kFullMask, L, from) == 0 ? 0u : 0x7fff7fffu;
          uint4* rows = reinterpret_cast<uint4*>(p.out) + static_cast<size_t>(r0) * p.H * (D / 8);
          const long long vecs = static_cast<long long>(r1 - r0) * p.H * (D / 8);
          for (long long i = lane; i < vecs; i += 32) rows[i] = make_uint4(v, v, v, v);
        }
      }
    } else if (warp >= 12) {
      // ================================================================ clean V tiles
      const int part = warp - 12;
      const int box_rows = min(p.block_size, kChunkKeys);
      unsigned loads = 0;
      for (int item = 0; !timed_out; ++item) {
        const int slot = item % kDescs;
        if (!warp_wait(&ms.desc_full[slot], (item / kDescs) & 1)) {
          timed_out = true;
          break;
        }
        Piece& d = ms.desc[slot];
        if (!d.valid) break;
        const int ja = d.ja, nt = d.jb - ja, kv_end = d.end;
        for (int t = 0; t < nt; ++t) {
          const unsigned at = loads + t;
          const int st = at % NV;
          const int tile = d.key_tile(p, ja + t), edge = d.edge(p, tile);
          if (kFp8) {
            const int keys = min(kChunkKeys, kv_end - tile * kChunkKeys);
            const int kst = at % NK;
            bool ok = true;
#pragma unroll 1
            for (int v = 0; ok && v < 2; ++v) {  // K, then V
              ok = warp_wait(&ms.raw_full[v], at & 1) &&
                   warp_wait(v == 0 ? &ms.k_empty[kst] : &ms.v_empty[st],
                             ((v == 0 ? at / NK : at / NV) & 1) ^ 1);
              if (!ok) break;
              unsigned char* codes = raw + v * C::kRaw;
              if (v == 1 && edge >= 0) clean_codes<D>(codes, part, keys, d.nonfinite[edge]);
              widen<D>(v == 0 ? ks + kst * C::kTile : vs + st * C::kTile, codes, part, keys);
              fence_proxy_async_smem();
              __threadfence_block();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive(v == 0 ? &ms.k_full[kst] : &ms.clean[st]);
                mbar_arrive(&ms.raw_empty[v]);
              }
            }
            if (!ok) {
              timed_out = true;
              break;
            }
            continue;
          }
          if (!warp_wait(&ms.v_full[st], (at / NV) & 1)) {
            timed_out = true;
            break;
          }
          if (edge < 0) {  // every row sees every key
            if (lane == 0) mbar_arrive(&ms.clean[st]);
            continue;
          }
          const int keys = min(kChunkKeys, kv_end - tile * kChunkKeys);
          clean_tile<D, kBf16>(vs + st * C::kTile, part, keys, box_rows, d.nonfinite[edge]);
          fence_proxy_async_smem();
          __threadfence_block();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.clean[st]);
        }
        loads += nt;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.desc_empty[slot]);
      }
    }
  }
  if (timed_out) atomic_or_error(p.error_word, PDA_DEVERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

// A map over rows [rows, heads, D] whose boxes are `box_rows` rows of `box_heads` heads: of
// 64 16-bit elements, written with the 128-byte swizzle, or of whole rows of codes.
pda_status encode_heads(CUtensorMap* tm, const void* base, long long rows, int heads, int D,
                        pda_dtype type, int box_heads, int box_rows) {
  const bool codes = type == PDA_FP8_E4M3;
  const cuuint64_t e = dtype_bytes(type);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {D * e, heads * D * e};
  const cuuint32_t box[3] = {codes ? static_cast<cuuint32_t>(D) : 64u,
                             static_cast<cuuint32_t>(box_heads),
                             static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t one[3] = {1u, 1u, 1u};
  const CUresult r = g_encode(
      tm,
      codes              ? CU_TENSOR_MAP_DATA_TYPE_UINT8
      : type == PDA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
      3, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
      codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
      D * e >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
      : D * e >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                     : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PDA_OK : PDA_ERR_INVALID_ARG;
}

// The V cache with a row's 64-element halves as a dimension of their own: boxes of `box_rows`
// rows of both halves of one head, half after half.
pda_status encode_v(CUtensorMap* tm, const void* base, long long rows, int heads, int D, bool bf16,
                    int box_rows) {
  const cuuint64_t dims[4] = {64u, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(D / 64),
                              static_cast<cuuint64_t>(heads)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(heads) * D * 2, 128u,
                                 static_cast<cuuint64_t>(D) * 2};
  const cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(box_rows),
                             static_cast<cuuint32_t>(D / 64), 1u};
  const cuuint32_t one[4] = {1u, 1u, 1u, 1u};
  const CUresult r = g_encode(
      tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
      const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B,
      D == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PDA_OK : PDA_ERR_INVALID_ARG;
}

template <int D, bool kBf16, bool kFp8, bool kWindow>
pda_status launch(const ChunkParams& p, int dev, int sms, bool capped, float* partial,
                  cudaStream_t stream) {
  constexpr size_t smem = smem_bytes<D, kFp8, kWindow>();
  static std::atomic<bool> raised[64];
  if (dev >= 64 || !raised[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(chunk_tc_kernel<D, kBf16, kFp8, kWindow>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
      return PDA_ERR_CUDA;
    if (dev < 64) raised[dev].store(true, std::memory_order_release);
  }
  int g_shift = 0;
  while ((1 << g_shift) < p.G) ++g_shift;
  CUtensorMap tq, tk, tv;
  const long long rows = static_cast<long long>(p.num_blocks) * p.block_size;
  const int box = p.block_size < kChunkKeys ? p.block_size : kChunkKeys;
  const pda_dtype q_type = kBf16 ? PDA_BF16 : PDA_F16, kv_type = kFp8 ? PDA_FP8_E4M3 : q_type;
  pda_status st = encode_heads(&tq, p.q, p.T, p.H, D, q_type, p.G, 128 >> g_shift);
  if (st == PDA_OK) st = encode_heads(&tk, p.k_cache, rows, p.H_kv, D, kv_type, 1, box);
  if (st == PDA_OK)
    st = kFp8 ? encode_heads(&tv, p.v_cache, rows, p.H_kv, D, kv_type, 1, box)
              : encode_v(&tv, p.v_cache, rows, p.H_kv, D, kBf16, box);
  if (st != PDA_OK) return st;
  const int grid = chunk_grid<CutsOf<kWindow>>(p, g_shift, sms);
  chunk_tc_kernel<D, kBf16, kFp8, kWindow><<<grid, kThreads, smem, stream>>>(tq, tk, tv, p, g_shift,
                                                                    partial);
  if (cudaGetLastError() != cudaSuccess) return PDA_ERR_CUDA;
  using Out = std::conditional_t<kBf16, __nv_bfloat16, __half>;
  return launch_merge<D, Out, CutsOf<kWindow>>(p, g_shift, partial, grid, capped, stream);
}

template <bool kWindow>
pda_status launch_tc(const ChunkParams& p, int D, pda_dtype kv_dtype, int dev, int sms,
                           bool capped, void* workspace, cudaStream_t stream) {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (g_encode == nullptr) return PDA_ERR_CUDA;
  float* partial = static_cast<float*>(workspace);
  const bool wide = D == 128;
  if (kv_dtype == PDA_BF16)
    return wide ? launch<128, true, false, kWindow>(p, dev, sms, capped, partial, stream)
                : launch<64, true, false, kWindow>(p, dev, sms, capped, partial, stream);
  if (kv_dtype == PDA_F16)
    return wide ? launch<128, false, false, kWindow>(p, dev, sms, capped, partial, stream)
                : launch<64, false, false, kWindow>(p, dev, sms, capped, partial, stream);
  return wide ? launch<128, true, true, kWindow>(p, dev, sms, capped, partial, stream)
              : launch<64, true, true, kWindow>(p, dev, sms, capped, partial, stream);
}

}  // namespace
}  // namespace pda
