// Gradients of the combine and of the routing weights.
//
// Combine:  out[t] = sum_j w[t, j] y[p],  p = dst_pos[t*k + j]
//   d_y[p]    = w[t, j] d_out[t]          (rounded once to y's type)
//   d_w[t, j] = sum_i d_out[t, i] y[p, i]
// Routing weights, S = sum_j w_j d_j over a token's slots (d = d_topk_w):
//   renormalised over the selected experts: d_logits[idx_j] = w_j (d_j - S), else 0
//   full softmax p:  d_logits[e] = sum_{j: idx_j = e} w_j d_j - p_e S
// The dispatch's gradient is the combine with unit weights (combine.hip).
#include "device_common.hpp"
#include "launch.hpp"

namespace moe {

namespace {

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / kWave;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Sum over the wave, the same in every lane (a fixed order of additions).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {   // rounds to nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

template <bool NT, typename V>
__device__ __forceinline__ V load_as(const void* p) {
  return NT ? __builtin_nontemporal_load(static_cast<const V*>(p)) : *static_cast<const V*>(p);
}

// G consecutive elements of a row in registers as loaded.
template <typename T, int G> struct Raw;
template <> struct Raw<uint16_t, 8> {
  u32x4 v;
  template <bool NT> __device__ void load(const uint16_t* p) { v = load_as<NT, u32x4>(p); }
  __device__ void to_f32(float (&o)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack_bf16x2(v[i], o[2 * i], o[2 * i + 1]);
  }
  __device__ static void store(uint16_t* p, const float (&o)[8]) {
    __builtin_nontemporal_store(u32x4{pack2(o[0], o[1]), pack2(o[2], o[3]), pack2(o[4], o[5]),
                                      pack2(o[6], o[7])}, reinterpret_cast<u32x4*>(p));
  }
};
template <> struct Raw<uint16_t, 4> {
  u32x2 v;
  template <bool NT> __device__ void load(const uint16_t* p) { v = load_as<NT, u32x2>(p); }
  __device__ void to_f32(float (&o)[4]) const {
    unpack_bf16x2(v.x, o[0], o[1]); unpack_bf16x2(v.y, o[2], o[3]);
  }
  __device__ static void store(uint16_t* p, const float (&o)[4]) {
    __builtin_nontemporal_store(u32x2{pack2(o[0], o[1]), pack2(o[2], o[3])}, reinterpret_cast<u32x2*>(p));
  }
};
template <> struct Raw<uint16_t, 1> {
  uint16_t v;
  template <bool NT> __device__ void load(const uint16_t* p) { v = load_as<NT, uint16_t>(p); }
  __device__ void to_f32(float (&o)[1]) const { o[0] = bf16_to_f32(v); }
  __device__ static void store(uint16_t* p, const float (&o)[1]) { *p = f32_to_bf16_rne(o[0]); }
};
template <int G> struct Raw<float, G> {       // 4 or 8
  u32x4 v[G / 4];
  template <bool NT> __device__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < G / 4; ++i) v[i] = load_as<NT, u32x4>(p + 4 * i);
  }
  __device__ void to_f32(float (&o)[G]) const {
#pragma unroll
    for (int i = 0; i < G; ++i) o[i] = __uint_as_float(v[i / 4][i % 4]);
  }
  __device__ static void store(float* p, const float (&o)[G]) {
#pragma unroll
    for (int i = 0; i < G / 4; ++i)
      __builtin_nontemporal_store(u32x4{__float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]),
                                        __float_as_uint(o[4 * i + 2]), __float_as_uint(o[4 * i + 3])},
                                  reinterpret_cast<u32x4*>(p + 4 * i));
  }
};
template <> struct Raw<float, 1> {
  float v;
  template <bool NT> __device__ void load(const float* p) { v = load_as<NT, float>(p); }
  __device__ void to_f32(float (&o)[1]) const { o[0] = v; }
  __device__ static void store(float* p, const float (&o)[1]) { *p = o[0]; }
};

// One wave per pair q = t*k + j: it reads row dst_pos[q] of y and row t of
// d_out once, writes row dst_pos[q] of d_y, and keeps the dot product in fp32
// registers, so d_w needs no second pass, no atomics and no workspace.  The k
// waves of a token sit side by side, so d_out comes from the caches after the
// first.  y and d_y are touched once and bypass them (non-temporal).  Bound by
// memory: 4096 tokens x 7168, top-8, bf16 move 1 GB in 183 us, 5.5 TB/s (a
// device copy reaches 4.8 here).
// Lanes take G consecutive elements at a time, U groups in flight.  WPP: waves
// per pair, which share its row and add their partial sums in wave order.
template <typename TG, typename TY, int G, int U, int WPP>
__global__ __launch_bounds__(kBlock) void combine_backward_kernel(
    const TG* __restrict__ d_out, const TY* __restrict__ y, int64_t nk, int64_t hidden, int k,
    const int32_t* __restrict__ dst_pos, const float* __restrict__ topk_w, TY* __restrict__ d_y,
    float* __restrict__ d_w) {
  static_assert(WPP == 1 || WPP == kWaves, "a wave or a workgroup per pair");
  __shared__ float s_part[kWaves];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x / kWave));
  const int64_t q = WPP == 1 ? block_id() * kWaves + wave : block_id();
  if (q >= nk) return;
  const int p = __builtin_amdgcn_readfirstlane(dst_pos[q]);
  const bool writes = lane == 0 && (WPP == 1 || wave == 0);
  if (unsigned(p) >= uint64_t(nk)) {            // a pair that holds no row
    if (writes) d_w[q] = 0.f;
    return;
  }
  const float w = topk_w[q];
  const TG* g = d_out + q / k * hidden;
  const TY* yr = y + int64_t(p) * hidden;
  TY* dr = d_y + int64_t(p) * hidden;
  float dot = 0.f;
  const int64_t ngroups = hidden / G;
  for (int64_t g0 = (WPP == 1 ? 0 : wave * U * kWave) + lane; g0 < ngroups; g0 += WPP * U * kWave) {
    Raw<TG, G> rg[U];
    Raw<TY, G> ry[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // past the row's end: its last group again, not used
      const int64_t gi = g0 + u * kWave < ngroups ? g0 + u * kWave : ngroups - 1;
      ry[u].template load<true>(yr + gi * G);
      rg[u].template load<false>(g + gi * G);
    }
    __builtin_amdgcn_sched_barrier(0);          // all loads go out before the first is used
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (g0 + u * kWave >= ngroups) break;
      float a[G], b[G];
      rg[u].to_f32(a);
      ry[u].to_f32(b);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        dot = __builtin_fmaf(a[i], b[i], dot);
        a[i] *= w;
      }
      Raw<TY, G>::store(dr + (g0 + u * kWave) * G, a);
    }
  }
  dot = wave_sum(dot);
  if (WPP > 1) {
    if (lane == 0) s_part[wave] = dot;
    __syncthreads();
    dot = s_part[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) dot += s_part[i];
  }
  if (writes) d_w[q] = dot;
}

template <typename TG, typename TY>
hipError_t launch_combine_backward_typed(const void* d_out, const void* y, int64_t n_tokens,
                                         int64_t hidden, int k, const int32_t* dst_pos,
                                         const float* topk_w, void* d_y, float* d_w,
                                         hipStream_t stream) {
  const int64_t nk = n_tokens * k;
  const TG* g = static_cast<const TG*>(d_out);
  const TY* yy = static_cast<const TY*>(y);
  TY* dy = static_cast<TY*>(d_y);
  // groups of G start on the alignment of their widest load (16 bytes at most)
  auto fits = [&](int64_t n) {
    auto ok = [&](const void* p, size_t elem) {
      const size_t a = n * elem < 16 ? n * elem : 16;
      return reinterpret_cast<uintptr_t>(p) % a == 0;
    };
    return hidden % n == 0 && ok(g, sizeof(TG)) && ok(yy, sizeof(TY)) && ok(dy, sizeof(TY));
  };
  auto run = [&](auto kernel, int per_block) {
    kernel<<<grid_of((nk + per_block - 1) / per_block), kBlock, 0, stream>>>(g, yy, nk, hidden, k, dst_pos, topk_w, dy, d_w);
  };
  // a workgroup per pair where a wave per pair would leave the card idle and
  // rows are long enough to share.  Measured, wave against workgroup per pair:
  // 1024 pairs of 7168 bf16 14.8 and 8.8 us, 2048 of 4096 12.5 and 9.8; 4096 of
  // 7168 25.6 and 28.6, 2800 of 1001 5.3 and 6.0.
  const bool few = nk < 4096 && hidden >= 2048;
  if (fits(8)) few ? run(combine_backward_kernel<TG, TY, 8, 4, kWaves>, 1) : run(combine_backward_kernel<TG, TY, 8, 4, 1>, kWaves);
  else if (fits(4)) few ? run(combine_backward_kernel<TG, TY, 4, 4, kWaves>, 1) : run(combine_backward_kernel<TG, TY, 4, 4, 1>, kWaves);
  else few ? run(combine_backward_kernel<TG, TY, 1, 8, kWaves>, 1) : run(combine_backward_kernel<TG, TY, 1, 8, 1>, kWaves);
  return hipGetLastError();
}

// v of the lane that DPP control CTRL names; v itself where that lane or this
// one's row takes no part.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp_or_self(float v) {
  const int b = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, ROW_MASK, 0xF, false));
}
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp_or_zero(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROW_MASK, 0xF, true));
}
__device__ __forceinline__ float lane63(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
// Maximum and sum over the wave by DPP row operations (within quads, halves and
// rows of 16 lanes, then across the rows), the same in every lane.
__device__ __forceinline__ float wave_max_dpp(float v) {
  v = fmaxf(v, dpp_or_self<0xB1, 0xF>(v));      // lanes 1 0 3 2
  v = fmaxf(v, dpp_or_self<0x4E, 0xF>(v));      // lanes 2 3 0 1
  v = fmaxf(v, dpp_or_self<0x141, 0xF>(v));     // row_half_mirror
  v = fmaxf(v, dpp_or_self<0x140, 0xF>(v));     // row_mirror
  v = fmaxf(v, dpp_or_self<0x142, 0xA>(v));     // row_bcast:15
  v = fmaxf(v, dpp_or_self<0x143, 0xC>(v));     // row_bcast:31
  return lane63(v);
}
__device__ __forceinline__ float wave_sum_dpp(float v) {
  v += dpp_or_zero<0xB1, 0xF>(v);
  v += dpp_or_zero<0x4E, 0xF>(v);
  v += dpp_or_zero<0x141, 0xF>(v);
  v += dpp_or_zero<0x140, 0xF>(v);
  v += dpp_or_zero<0x142, 0xA>(v);
  v += dpp_or_zero<0x143, 0xC>(v);
  return lane63(v);
}

// One wave per token; lane l holds experts l, l + 64, ..., so a row is written
// in whole 256-byte runs.  The slots are added in order j = 0..k-1, also where
// two of them name the same expert.  RENORM false computes the softmax of the
// row's logits again, p_e = exp(l_e - max) / sum exp(l - max), from registers.
// The first slot's logit serves as the maximum where none is larger; that
// expert may have been dropped, though, or the slots come in another order, and
// then the lanes exchange theirs (doing that always: 15.0 -> 16.2 us for 32768 x 256).
template <int SLOTS, bool RENORM>
__global__ __launch_bounds__(kBlock) void route_backward_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const float* __restrict__ topk_w, const float* __restrict__ d_w, int64_t n_tokens,
    int n_experts, int k, float* __restrict__ d_logits) {
  const int lane = lane_id();
  const int64_t t = block_id() * kWaves + __builtin_amdgcn_readfirstlane(int(threadIdx.x / kWave));
  if (t >= n_tokens) return;
  const bool has = lane < k;
  const int my_e = has ? topk_idx[t * k + lane] : -1;
  const bool ok = unsigned(my_e) < unsigned(n_experts);
  const float w = ok ? topk_w[t * k + lane] : 0.f;
  const float wd = ok ? w * d_w[t * k + lane] : 0.f;
  float p[SLOTS];
  if (!RENORM) {
    const int e_r = __builtin_amdgcn_readfirstlane(my_e);
    float mine_top = -__builtin_inff(), top = 0.f, total = 0.f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int e = s * kWave + lane;
      p[s] = e < n_experts ? logits[t * n_experts + e] : -__builtin_inff();
      mine_top = fmaxf(mine_top, p[s]);
      top = e_r / kWave == s ? p[s] : top;
    }
    top = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(top), e_r & (kWave - 1)));
    if (unsigned(e_r) >= unsigned(n_experts) || ballot(mine_top > top)) top = wave_max_dpp(mine_top);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      p[s] = expf(p[s] - top);
      total += p[s];
    }
    const float inv = 1.f / wave_sum_dpp(total);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) p[s] *= inv;
  }
  float sum = 0.f;
  for (int j = 0; j < k; ++j) sum += __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wd), j));
  const float mine = RENORM ? wd - w * sum : wd;
  float d[SLOTS];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) d[s] = RENORM ? 0.f : -p[s] * sum;
  for (int j = 0; j < k; ++j) {
    const int e = __builtin_amdgcn_readlane(my_e, j);
    const float v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine), j));
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) d[s] += e == s * kWave + lane ? v : 0.f;
  }
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    const int e = s * kWave + lane;
    if (e < n_experts) d_logits[t * n_experts + e] = d[s];
  }
}

template <bool RENORM>
void launch_route_backward_slots(const float* logits, const int32_t* idx, const float* w,
                                 const float* d_w, int64_t n, int e, int k, float* d_logits,
                                 hipStream_t stream) {
  const dim3 blocks = grid_of((n + kWaves - 1) / kWaves);
  if (e <= 64)
    route_backward_kernel<1, RENORM><<<blocks, kBlock, 0, stream>>>(logits, idx, w, d_w, n, e, k, d_logits);
  else if (e <= 128)
    route_backward_kernel<2, RENORM><<<blocks, kBlock, 0, stream>>>(logits, idx, w, d_w, n, e, k, d_logits);
  else if (e <= 256)
    route_backward_kernel<4, RENORM><<<blocks, kBlock, 0, stream>>>(logits, idx, w, d_w, n, e, k, d_logits);
  else if (e <= 512)
    route_backward_kernel<8, RENORM><<<blocks, kBlock, 0, stream>>>(logits, idx, w, d_w, n, e, k, d_logits);
  else
    route_backward_kernel<16, RENORM><<<blocks, kBlock, 0, stream>>>(logits, idx, w, d_w, n, e, k, d_logits);
}

}  // namespace

hipError_t launch_combine_backward(const void* d_out, int g_bf16, const void* y, int y_bf16,
                                   int64_t n_tokens, int64_t hidden, int k, const int32_t* dst_pos,
                                   const float* topk_w, void* d_y, float* d_topk_w,
                                   hipStream_t stream) {
  if (g_bf16 && y_bf16)
    return launch_combine_backward_typed<uint16_t, uint16_t>(d_out, y, n_tokens, hidden, k, dst_pos, topk_w, d_y, d_topk_w, stream);
  if (g_bf16)
    return launch_combine_backward_typed<uint16_t, float>(d_out, y, n_tokens, hidden, k, dst_pos, topk_w, d_y, d_topk_w, stream);
  if (y_bf16)
    return launch_combine_backward_typed<float, uint16_t>(d_out, y, n_tokens, hidden, k, dst_pos, topk_w, d_y, d_topk_w, stream);
  return launch_combine_backward_typed<float, float>(d_out, y, n_tokens, hidden, k, dst_pos, topk_w, d_y, d_topk_w, stream);
}

hipError_t launch_route_topk_backward(const float* logits, const int32_t* topk_idx,
                                      const float* topk_w, const float* d_topk_w,
                                      int64_t n_tokens, int n_experts, int k, int renormalize,
                                      float* d_logits, hipStream_t stream) {
  if (renormalize)
    launch_route_backward_slots<true>(logits, topk_idx, topk_w, d_topk_w, n_tokens, n_experts, k, d_logits, stream);
  else
    launch_route_backward_slots<false>(logits, topk_idx, topk_w, d_topk_w, n_tokens, n_experts, k, d_logits, stream);
  return hipGetLastError();
}

}  // namespace moe
