// qk_rope.cu -- norm and position rotation of a step's queries and keys, in one pass that writes
// the keys and values into their cache slots.
//
// Mathematics. A head's row x [D]: y = x rsqrt(mean x^2 + eps) w where it has a norm weight w;
// then the first R elements turn in pairs (a, b), by the angle of the token's position p:
//   (a, b) -> (a c - b s, b c + a s),  (c, s) = f (cos, sin)(2 pi p F_i),
// pair i being elements (i, i + R / 2), or (2 i, 2 i + 1) interleaved. All in 32 bits, rounded
// once. F_i, turns per position, comes as a 64-bit fraction of a turn, so p F_i modulo 2^64 is the
// angle's exact remainder however far the position: the product's wrap is the range reduction.
// Its top 32 bits are what cos and sin see (2^-25 of a half turn off at most, 1e-7).
//
// What bounds it: memory, each byte read and written once; a step of few tokens is bound by
// latency. 16384 tokens of 32/8 heads of 128 in bf16, with norms: 71 us, 5.7 TB/s (84 % of the
// copy rate); 256 tokens into an FP8 cache 4.4 us, 8 tokens 2.7 us. A warp takes a whole token, so
// that its angles are computed once and its weights folded into them once per kind of row; a block
// a token with a barrier took 232 us, a warp that found each step's row by itself 94.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "pda_device.cuh"
#include "pda_internal.h"

namespace pda {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeVec = 8;        // elements of a lane
constexpr int kRopeMaxHead = 256;  // largest D
// few tokens are spread over this many warps of an SM: 256 tokens 4.4 us, 6.0 over 32, 4.9 over 8
constexpr int kRopeWarpsPerSm = 16;
constexpr int kRopeSteps = 4;      // rows of a lane in flight

struct RopeParams {
  void* q_out;
  const void* q;
  const void* k;
  const void* v;  // nullptr: none
  long long q_stride, k_stride, v_stride;  // elements from token to token
  void* k_out;  // cache, or (slots == nullptr) dense rows
  void* v_out;
  const int32_t* slots;
  const int32_t* positions;
  const unsigned long long* freqs;
  const void* q_weight;  // nullptr: no norm
  const void* k_weight;
  int32_t* error_word;
  int T, H, H_kv, D, R;
  int group_rows, groups_per_warp, parts;  // parts: warps of a token
  long long num_slots;
  float eps, factor, per_k, per_v;  // codes: 1 / scale
};

// Eight elements as they lie in memory.
template <typename E>
struct Raw {
  static constexpr int kWords = kRopeVec * sizeof(E) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const E* p) {
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
      const uint4 v = *(reinterpret_cast<const uint4*>(p) + i / 4);
      w[i] = v.x;
      w[i + 1] = v.y;
      w[i + 2] = v.z;
      w[i + 3] = v.w;
    }
  }
  __device__ __forceinline__ void widen(float* x) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (std::is_same<E, float>::value) {
        x[i] = __uint_as_float(w[i]);
      } else if constexpr (std::is_same<E, __nv_bfloat16>::value) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
      } else {
        const float2 f = __half22float2(as_half2(w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
};

__device__ __forceinline__ void store8(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// E4M3 codes, saturating at 448; NaN stays NaN.
__device__ __forceinline__ void store8(fp8e4m3* p, const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %1, %2;\n\t"
        "cvt.u32.u16 %0, h;\n\t}"
        : "=r"(w[i])
        : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// A step is 32 / LPR head rows of one kind (queries, then keys, then values), LPR lanes sharing a
// row, eight elements each (kWhole: D = 8 LPR; otherwise those behind D idle); up to kRopeSteps
// steps of a kind make a group, whose loads are in flight together and under the group before. A
// warp takes one token's groups [part * groups_per_warp, + 1). With y the pair's other element, the
// weights folded into the angle:
//   out = rsqrt(mean x^2 + eps) (x (w c) + y (+- w_y s)).
template <typename E, typename KV, int LPR, bool kHalf, bool kWhole>
__global__ void __launch_bounds__(kRopeThreads, 5) qk_rope_kernel(const RopeParams p) {
  constexpr int kRows = 32 / LPR;                                  // rows of a step
  __shared__ float2 trig[kRopeThreads / 32][kRopeMaxHead / 2];     // (cos, sin) of the pairs
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cl = lane % LPR, d0 = cl * kRopeVec, sub = lane / LPR;
  const unsigned task = blockIdx.x * (kRopeThreads / 32) + warp;
  const unsigned t = task / static_cast<unsigned>(p.parts);
  if (t >= static_cast<unsigned>(p.T)) return;
  const int part = static_cast<int>(task - t * p.parts);
  const int D = kWhole ? LPR * kRopeVec : p.D;
  const int half_lanes = p.R / (2 * kRopeVec);
  const bool live = kWhole || d0 < D, turns = d0 < p.R, first_half = cl < half_lanes;
  const int partner = turns ? (first_half ? lane + half_lanes : lane - half_lanes) : lane;
  const int q_groups = (p.H + p.group_rows - 1) / p.group_rows;
  const int k_groups = (p.H_kv + p.group_rows - 1) / p.group_rows;
  const int all = q_groups + (p.v != nullptr ? 2 : 1) * k_groups;
  const int g0 = part * p.groups_per_warp, g1 = min(all, g0 + p.groups_per_warp);
  if (g0 >= g1) return;

  // group g's kind (0 queries, 1 keys, 2 values), this lane's first row and the end of its rows
  struct Group {
    int kind, row, end;
  };
  auto group = [&](int g) {
    Group r;
    r.kind = g < q_groups ? 0 : g < q_groups + k_groups ? 1 : 2;
    const int first = (g - (r.kind == 0 ? 0 : q_groups) - (r.kind == 2 ? k_groups : 0)) *
                      p.group_rows;
    r.row = first + sub;
    r.end = min(first + p.group_rows, r.kind == 0 ? p.H : p.H_kv);
    return r;
  };
  Raw<E> x[kRopeSteps];
  auto load = [&](const Group& g) {
    const E* base = static_cast<const E*>(g.kind == 0 ? p.q : g.kind == 1 ? p.k : p.v) +
                    static_cast<long long>(t) *
                        (g.kind == 0 ? p.q_stride : g.kind == 1 ? p.k_stride : p.v_stride) +
                    g.row * D + d0;
#pragma unroll
    for (int u = 0; u < kRopeSteps; ++u) {
      if (live && g.row + u * kRows < g.end)
        x[u].load(base + u * kRows * D);
      else
#pragma unroll
        for (int i = 0; i < Raw<E>::kWords; ++i) x[u].w[i] = 0;
    }
  };
  Group next = group(g0);
  load(next);
  const long long slot = p.slots != nullptr ? p.slots[t] : static_cast<long long>(t);
  const unsigned long long pos =
      static_cast<unsigned long long>(static_cast<long long>(p.positions[t]));
  for (int i = lane; i < p.R / 2; i += 32) {
    const unsigned long long turn = pos * p.freqs[i];
    float sn, cs;
    sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &sn, &cs);
    trig[warp][i] = make_float2(cs * p.factor, sn * p.factor);
  }
  __syncwarp();
  const float inv_d = 1.f / static_cast<float>(D);
  float c[kRopeVec], s[kRopeVec];
  // c, s of a kind's rows
  auto angles = [&](const void* weight) {
    float w[kRopeVec], wy[kRopeVec];
#pragma unroll
    for (int e = 0; e < kRopeVec; ++e) w[e] = wy[e] = 1.f;
    if (weight != nullptr && live) {
      load_elems<E, kRopeVec>(static_cast<const E*>(weight) + d0, w);
      if (kHalf && turns)
        load_elems<E, kRopeVec>(
            static_cast<const E*>(weight) + d0 + (first_half ? p.R / 2 : -p.R / 2), wy);
    }
#pragma unroll
    for (int e = 0; e < kRopeVec; ++e) {
      float2 v = make_float2(1.f, 0.f);
      if (turns)
        v = trig[warp][kHalf ? d0 + e - (first_half ? 0 : p.R / 2) : (d0 + e) / 2];
      c[e] = w[e] * v.x;
      if (kHalf)
        s[e] = first_half ? -(wy[e] * v.y) : wy[e] * v.y;
      else
        s[e] = (e & 1) == 0 ? -(w[e + 1] * v.y) : w[e - 1] * v.y;
    }
  };
  int kind = -1;  // of c and s
  for (int g = g0; g < g1; ++g) {
    const Group now = next;
    Raw<E> in[kRopeSteps];
#pragma unroll
    for (int u = 0; u < kRopeSteps; ++u) in[u] = x[u];
    if (g + 1 < g1) {
      next = group(g + 1);
      load(next);
    }
    const void* weight = now.kind == 0 ? p.q_weight : p.k_weight;
    if (now.kind != 2 && now.kind != kind) {
      kind = now.kind;
      angles(weight);
    }
    // where the group's rows go; nothing is written where a slot is not one
    const bool write = now.kind == 0 || (slot >= 0 && slot < p.num_slots);
    const size_t to = (now.kind == 0 ? static_cast<size_t>(t) * p.H
                                     : static_cast<size_t>(write ? slot : 0) * p.H_kv) * D +
                      now.row * D + d0;
#pragma unroll
    for (int u = 0; u < kRopeSteps; ++u) {
      if (now.row - sub + u * kRows >= now.end) break;
      float o[kRopeVec];
      in[u].widen(o);
      if (now.kind != 2) {
        float y[kRopeVec];
        if (kHalf) {
          Raw<E> other;
#pragma unroll
          for (int i = 0; i < Raw<E>::kWords; ++i) {
            other.w[i] = __shfl_sync(kFullMask, in[u].w[i], partner);
            if (!turns) other.w[i] = 0;
          }
          other.widen(y);
        } else {
#pragma unroll
          for (int e = 0; e < kRopeVec; ++e) y[e] = turns ? o[e ^ 1] : 0.f;
        }
        float rs = 1.f;
        if (weight != nullptr) {
          float2 sq = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < kRopeVec; e += 2) {
            const float2 v = make_float2(o[e], o[e + 1]);
            sq = __ffma2_rn(v, v, sq);
          }
          float ss = sq.x + sq.y;
#pragma unroll
          for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor_sync(kFullMask, ss, m);
          rs = rsqrtf(fmaf(ss, inv_d, p.eps));
        }
        const float2 rs2 = make_float2(rs, rs);
#pragma unroll
        for (int e = 0; e < kRopeVec; e += 2) {
          float2 v = __fmul2_rn(make_float2(o[e], o[e + 1]), make_float2(c[e], c[e + 1]));
          v = __ffma2_rn(make_float2(y[e], y[e + 1]), make_float2(s[e], s[e + 1]), v);
          v = __fmul2_rn(v, rs2);
          o[e] = v.x;
          o[e + 1] = v.y;
        }
      }
      if (!write || !live || now.row + u * kRows >= now.end) continue;
      const size_t at = to + u * kRows * D;
      if (now.kind == 0) {
        store8(static_cast<E*>(p.q_out) + at, o);
      } else {
        if constexpr (std::is_same<KV, fp8e4m3>::value) {
          const float per = now.kind == 2 ? p.per_v : p.per_k;
#pragma unroll
          for (int e = 0; e < kRopeVec; ++e) o[e] *= per;
        }
        store8(static_cast<KV*>(now.kind == 2 ? p.v_out : p.k_out) + at, o);
      }
    }
  }
  if (slot >= p.num_slots && lane == 0) atomic_or_error(p.error_word, PDA_DEVERR_SLOT);
}

template <typename E, typename KV, int LPR>
void launch_layout(const RopeParams& p, bool interleaved, dim3 grid, cudaStream_t stream) {
  const bool whole = p.D == LPR * kRopeVec;
  if (interleaved)
    (whole ? qk_rope_kernel<E, KV, LPR, false, true> : qk_rope_kernel<E, KV, LPR, false, false>)
        <<<grid, kRopeThreads, 0, stream>>>(p);
  else
    (whole ? qk_rope_kernel<E, KV, LPR, true, true> : qk_rope_kernel<E, KV, LPR, true, false>)
        <<<grid, kRopeThreads, 0, stream>>>(p);
}

template <typename E, typename KV>
void launch_width(const RopeParams& p, bool interleaved, dim3 grid, cudaStream_t stream) {
  if (p.D <= 64)
    launch_layout<E, KV, 8>(p, interleaved, grid, stream);
  else if (p.D <= 128)
    launch_layout<E, KV, 16>(p, interleaved, grid, stream);
  else
    launch_layout<E, KV, 32>(p, interleaved, grid, stream);
}

pda_status check_rope(const RopeParams& p, pda_dtype dtype) {
  if (p.T < 0 || p.H <= 0 || p.H_kv <= 0 || p.D <= 0 || p.R < 0 || p.R > p.D ||
      !float_dtype_ok(dtype) || !isfinite(p.eps) || p.eps < 0.f || !isfinite(p.factor))
    return PDA_ERR_INVALID_ARG;
  if (p.D % kRopeVec != 0 || p.D > kRopeMaxHead || p.R % 16 != 0 || p.H > (1 << 14) ||
      p.H_kv > (1 << 14))
    return PDA_ERR_UNSUPPORTED;
  const long long per_vec = dtype == PDA_F32 ? 4 : 8;  // elements of 16 bytes
  const long long q_row = static_cast<long long>(p.H) * p.D;
  const long long k_row = static_cast<long long>(p.H_kv) * p.D;
  if (p.q_stride < q_row || p.k_stride < k_row || (p.v != nullptr && p.v_stride < k_row) ||
      p.q_stride % per_vec != 0 || p.k_stride % per_vec != 0 ||
      (p.v != nullptr && p.v_stride % per_vec != 0))
    return PDA_ERR_INVALID_ARG;
  return PDA_OK;
}

pda_status launch_rope(RopeParams p, pda_dtype dtype, pda_dtype kv_dtype, bool interleaved,
                       cudaStream_t stream) {
  if (p.q_out == nullptr || p.q == nullptr || p.k == nullptr || p.k_out == nullptr ||
      p.positions == nullptr || (p.R > 0 && p.freqs == nullptr))
    return PDA_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(p.q_out), p.q, p.k, p.v,
                        static_cast<const void*>(p.k_out), static_cast<const void*>(p.v_out),
                        p.q_weight, p.k_weight})
    if (!aligned16(x)) return PDA_ERR_INVALID_ARG;
  int dev, sms;
  const pda_status st = current_device_sms(&dev, &sms);
  if (st != PDA_OK) return st;
  // A warp takes a token; with few tokens their groups are spread over several warps, down to
  // groups of one step each.
  const int rows = p.D <= 64 ? 4 : p.D <= 128 ? 2 : 1;  // of a step
  const long long want = static_cast<long long>(sms) * kRopeWarpsPerSm / p.T;  // warps of a token
  int groups = 0;
  for (int steps = kRopeSteps; steps >= 1; steps >>= 1) {
    p.group_rows = rows * steps;
    groups = (p.H + p.group_rows - 1) / p.group_rows +
             (p.H_kv + p.group_rows - 1) / p.group_rows * (p.v != nullptr ? 2 : 1);
    if (groups >= want) break;
  }
  const long long parts = std::min<long long>(groups, std::max<long long>(1, want));
  p.groups_per_warp = static_cast<int>((groups + parts - 1) / parts);
  p.parts = (groups + p.groups_per_warp - 1) / p.groups_per_warp;
  const long long blocks =
      (static_cast<long long>(p.T) * p.parts + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  const dim3 grid(static_cast<unsigned>(blocks));
  if (dtype == PDA_F32)
    launch_width<float, float>(p, interleaved, grid, stream);
  else if (dtype == PDA_F16)
    launch_width<__half, __half>(p, interleaved, grid, stream);
  else if (kv_dtype == PDA_FP8_E4M3)
    launch_width<__nv_bfloat16, fp8e4m3>(p, interleaved, grid, stream);
  else
    launch_width<__nv_bfloat16, __nv_bfloat16>(p, interleaved, grid, stream);
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}

}  // namespace
}  // namespace pda

using namespace pda;

extern "C" pda_status pda_qk_norm_rope_append(
    void* q_out, const void* q, const void* k, const void* v, long long q_stride,
    long long k_stride, long long v_stride, void* k_cache, void* v_cache,
    const int32_t* slot_mapping, const int32_t* positions, const uint64_t* freqs, int rope_dim,
    int interleaved, float attention_factor, const void* q_weight, const void* k_weight,
    float eps, int T, int H, int H_kv, int D, int block_size, int num_blocks, float k_scale,
    float v_scale, pda_dtype dtype, pda_dtype kv_dtype, int32_t* error_word,
    cudaStream_t stream) {
  RopeParams p{q_out, q, k, v, q_stride, k_stride, v_stride, k_cache, v_cache, slot_mapping,
               positions, reinterpret_cast<const unsigned long long*>(freqs), q_weight, k_weight,
               error_word, T, H, H_kv, D, rope_dim, 0, 0, 0,
               static_cast<long long>(num_blocks) * block_size, eps, attention_factor,
               1.f / k_scale, 1.f / v_scale};
  if (block_size <= 0 || num_blocks <= 0 || !dtype_ok(kv_dtype) || !isfinite(k_scale) ||
      !isfinite(v_scale) || !isfinite(p.per_k) || !isfinite(p.per_v) || (v == nullptr && T > 0))
    return PDA_ERR_INVALID_ARG;
  const pda_status st = check_rope(p, dtype);
  if (st != PDA_OK) return st;
  if (kv_dtype == PDA_FP8_E4M3 ? dtype != PDA_BF16 : dtype != kv_dtype)
    return PDA_ERR_UNSUPPORTED;
  if (p.num_slots >= (1ll << 31)) return PDA_ERR_UNSUPPORTED;
  if (T == 0) return PDA_OK;
  if (v_cache == nullptr || slot_mapping == nullptr) return PDA_ERR_INVALID_ARG;
  return launch_rope(p, dtype, kv_dtype, interleaved != 0, stream);
}

extern "C" pda_status pda_qk_norm_rope(void* q_out, void* k_out, const void* q, const void* k,
                                       long long q_stride, long long k_stride,
                                       const int32_t* positions, const uint64_t* freqs,
                                       int rope_dim, int interleaved, float attention_factor,
                                       const void* q_weight, const void* k_weight, float eps,
                                       int T, int H, int H_kv, int D, pda_dtype dtype,
                                       cudaStream_t stream) {
  const RopeParams p{q_out, q, k, nullptr, q_stride, k_stride, 0, k_out, nullptr, nullptr,
                     positions, reinterpret_cast<const unsigned long long*>(freqs), q_weight,
                     k_weight, nullptr, T, H, H_kv, D, rope_dim, 0, 0, 0, T, eps, attention_factor,
                     1.f, 1.f};
  const pda_status st = check_rope(p, dtype);
  if (st != PDA_OK) return st;
  if (T == 0) return PDA_OK;
  return launch_rope(p, dtype, dtype, interleaved != 0, stream);
}
