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
// latency.
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
constexpr int kRopeWarpsPerSm = 32;  // spread few tokens over this many
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
  int parts, steps_per_warp;  // warps of a token
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
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i / 4);
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

// A warp takes one token's steps [part * steps_per_warp, + 1): a step is 32 / LPR head rows of
// one kind, queries first, then keys, then values. LPR lanes share a row, eight elements each
// (those behind D idle). With y the pair's other element, the weights folded into the angle:
//   out = rsqrt(mean x^2 + eps) (x (w c) + y (+- w_y s)).
template <typename E, typename KV, int LPR, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(const RopeParams p) {
  constexpr int kRows = 32 / LPR;                                  // rows of a step
  __shared__ float2 trig[kRopeThreads / 32][kRopeMaxHead / 2];     // (cos, sin) of the pairs
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cl = lane % LPR, d0 = cl * kRopeVec, sub = lane / LPR;
  const unsigned task = blockIdx.x * (kRopeThreads / 32) + warp;
  const unsigned t = task / static_cast<unsigned>(p.parts);
  if (t >= static_cast<unsigned>(p.T)) return;
  const int part = static_cast<int>(task - t * p.parts);
  const size_t token = t;
  const int half_lanes = p.R / (2 * kRopeVec);
  const bool live = d0 < p.D, turns = d0 < p.R, first_half = cl < half_lanes;
  const int partner = turns ? (first_half ? lane + half_lanes : lane - half_lanes) : lane;
  const int q_steps = (p.H + kRows - 1) / kRows, k_steps = (p.H_kv + kRows - 1) / kRows;
  const int all = q_steps + (p.v != nullptr ? 2 : 1) * k_steps;
  const int s0 = part * p.steps_per_warp, s1 = min(all, s0 + p.steps_per_warp);
  if (s0 >= s1) return;

  // this lane's place in step s's row (nullptr: none), and the row's head
  auto source = [&](int s, int* head) -> const E* {
    const int h_k = s - q_steps, h_v = h_k - k_steps;
    const E* base;
    long long stride;
    int h, n;
    if (h_k < 0) {
      base = static_cast<const E*>(p.q), stride = p.q_stride, h = s * kRows + sub, n = p.H;
    } else if (h_v < 0) {
      base = static_cast<const E*>(p.k), stride = p.k_stride, h = h_k * kRows + sub, n = p.H_kv;
    } else {
      base = static_cast<const E*>(p.v), stride = p.v_stride, h = h_v * kRows + sub, n = p.H_kv;
    }
    *head = h;
    return live && h < n ? base + token * stride + h * p.D + d0 : nullptr;
  };
  Raw<E> x[kRopeSteps];
  auto load = [&](int s) {
#pragma unroll
    for (int u = 0; u < kRopeSteps; ++u) {
      int h;
      const E* at = s + u < s1 ? source(s + u, &h) : nullptr;
      if (at != nullptr)
        x[u].load(at);
      else
#pragma unroll
        for (int i = 0; i < Raw<E>::kWords; ++i) x[u].w[i] = 0;
    }
  };
  load(s0);
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
  const float inv_d = 1.f / static_cast<float>(p.D);
  float c[kRopeVec], s_[kRopeVec];
  // c, s_ of a kind's rows
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
        s_[e] = first_half ? -(wy[e] * v.y) : wy[e] * v.y;
      else
        s_[e] = (e & 1) == 0 ? -(w[e + 1] * v.y) : w[e - 1] * v.y;
    }
  };
  int kind = -1;  // of c and s_: 0 queries, 1 keys
  bool bad_slot = false;
  for (int s = s0; s < s1; s += kRopeSteps) {
    Raw<E> now[kRopeSteps];
#pragma unroll
    for (int u = 0; u < kRopeSteps; ++u) now[u] = x[u];
    if (s + kRopeSteps < s1) load(s + kRopeSteps);
#pragma unroll
    for (int u = 0; u < kRopeSteps; ++u) {
      if (s + u >= s1) break;
      int h;
      const bool there = source(s + u, &h) != nullptr;
      const bool is_q = s + u < q_steps, is_v = s + u >= q_steps + k_steps;
      float o[kRopeVec];
      now[u].widen(o);
      if (!is_v) {
        const void* weight = is_q ? p.q_weight : p.k_weight;
        if (kind != (is_q ? 0 : 1)) {
          kind = is_q ? 0 : 1;
          angles(weight);
        }
        float y[kRopeVec];
        if (kHalf) {
          Raw<E> other;
#pragma unroll
          for (int i = 0; i < Raw<E>::kWords; ++i) {
            other.w[i] = __shfl_sync(kFullMask, now[u].w[i], partner);
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
          v = __ffma2_rn(make_float2(y[e], y[e + 1]), make_float2(s_[e], s_[e + 1]), v);
          v = __fmul2_rn(v, rs2);
          o[e] = v.x;
          o[e + 1] = v.y;
        }
      }
      if (!there) continue;
      if (is_q) {
        store8(static_cast<E*>(p.q_out) + (token * p.H + h) * p.D + d0, o);
      } else if (slot >= p.num_slots) {
        bad_slot = true;
      } else if (slot >= 0) {
        if constexpr (std::is_same<KV, fp8e4m3>::value) {
          const float per = is_v ? p.per_v : p.per_k;
#pragma unroll
          for (int e = 0; e < kRopeVec; ++e) o[e] *= per;
        }
        store8(static_cast<KV*>(is_v ? p.v_out : p.k_out) +
                   (static_cast<size_t>(slot) * p.H_kv + h) * p.D + d0,
               o);
      }
    }
  }
  if (bad_slot) atomic_or_error(p.error_word, PDA_DEVERR_SLOT);
}

template <typename E, typename KV, int LPR>
void launch_layout(const RopeParams& p, bool interleaved, dim3 grid, cudaStream_t stream) {
  if (interleaved)
    qk_rope_kernel<E, KV, LPR, false><<<grid, kRopeThreads, 0, stream>>>(p);
  else
    qk_rope_kernel<E, KV, LPR, true><<<grid, kRopeThreads, 0, stream>>>(p);
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
  // A warp takes a token; with few tokens their steps are spread over several, down to one each.
  const int rows = p.D <= 64 ? 4 : p.D <= 128 ? 2 : 1;  // of a step
  const int steps = (p.H + rows - 1) / rows + (p.H_kv + rows - 1) / rows * (p.v != nullptr ? 2 : 1);
  const long long want = static_cast<long long>(sms) * kRopeWarpsPerSm;
  const long long parts = std::min<long long>(steps, std::max<long long>(1, want / p.T));
  p.steps_per_warp = static_cast<int>((steps + parts - 1) / parts);
  p.parts = (steps + p.steps_per_warp - 1) / p.steps_per_warp;
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
               error_word, T, H, H_kv, D, rope_dim, 0, 0,
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
                     k_weight, nullptr, T, H, H_kv, D, rope_dim, 0, 0, T, eps, attention_factor,
                     1.f, 1.f};
  const pda_status st = check_rope(p, dtype);
  if (st != PDA_OK) return st;
  if (T == 0) return PDA_OK;
  return launch_rope(p, dtype, dtype, interleaved != 0, stream);
}
