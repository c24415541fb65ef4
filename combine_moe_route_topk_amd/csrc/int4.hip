// Weights as 4-bit integers with group scales: codes two to a byte (the even
// element in the low nibble), one scale, and in the affine form one bias, per
// group of 32, 64 or 128 consecutive elements of a row.
//   symmetric:  s = T(max |x| * (1/7)),      q = clamp(rne(x / s) + 8, 0, 15),    x ~ s (q - 8)
//   affine:     s = T((max - min) * (1/15)), b = T(min),
//               q = clamp(rne((x - b) / s), 0, 15),                               x ~ s q + b
// T rounds to the scales' type (bf16 or fp32), the difference, the constants and
// the products before it are fp32, and the quotients are rounded as exact numbers,
// ties to even: from v = x * (1 / s) where v is clear of a half, else from the exact
// remainder x - q s.  s = 0 gives q = 0 before the offset of 8.  A group that
// holds a NaN or an infinity, or whose range or rounded bias is infinite, gets
// s = NaN (b = NaN).
//
// Rows are whole groups, so a matrix is one flat run of them.  Both kernels only
// stream: 8 elements per lane, 4, 8 or 16 lanes to a group, always within a row
// of 16 lanes.
#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"

namespace moe {

namespace {

constexpr int kBlock = 256;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const u32x4 a = *reinterpret_cast<const u32x4*>(p);
  const u32x4 b = *reinterpret_cast<const u32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) { v[i] = __uint_as_float(a[i]); v[4 + i] = __uint_as_float(b[i]); }
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack_bf16x2(a[i], v[2 * i], v[2 * i + 1]);
}
// Values are stored past the caches, as those of the MXFP4 kernels.
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  u32x4 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) { a[i] = __float_as_uint(v[i]); b[i] = __float_as_uint(v[4 + i]); }
  __builtin_nontemporal_store(a, reinterpret_cast<u32x4*>(p));
  __builtin_nontemporal_store(b, reinterpret_cast<u32x4*>(p + 4));
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  u32x4 a;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * i], v[2 * i + 1]}, bf16x2));
  __builtin_nontemporal_store(a, reinterpret_cast<u32x4*>(p));
}

__device__ __forceinline__ float scale_value(const float* s, int64_t i) { return s[i]; }
__device__ __forceinline__ float scale_value(const uint16_t* s, int64_t i) { return bf16_to_f32(s[i]); }
// v rounded to the scales' type, stored by the lanes that `put` names
__device__ __forceinline__ float round_scale(float v, float*) { return v; }
__device__ __forceinline__ float round_scale(float v, uint16_t*) { return bf16_to_f32(f32_to_bf16_rne(v)); }
__device__ __forceinline__ void put_scale(float* s, int64_t i, float v) { s[i] = v; }
__device__ __forceinline__ void put_scale(uint16_t* s, int64_t i, float v) { s[i] = f32_to_bf16_rne(v); }

template <int CTRL>
__device__ __forceinline__ float row_step(float v) {
  const int b = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, false));
}
// Maximum over the GROUP / 8 lanes of a group, in each of them.
template <int GROUP>
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, row_step<0xB1>(v));                     // lanes 1 0 3 2
  v = fmaxf(v, row_step<0x4E>(v));                     // lanes 2 3 0 1
  if (GROUP >= 64) v = fmaxf(v, row_step<0x141>(v));   // row_half_mirror
  if (GROUP >= 128) v = fmaxf(v, row_step<0x140>(v));  // row_mirror
  return v;
}

// 8 codes of 0 .. 15, held as floats, the first in the lowest nibble.
__device__ __forceinline__ uint32_t pack8(const float (&q)[8]) {
  const float lo = fmaf(q[3], 4096.f, fmaf(q[2], 256.f, fmaf(q[1], 16.f, q[0])));
  const float hi = fmaf(q[7], 4096.f, fmaf(q[6], 256.f, fmaf(q[5], 16.f, q[4])));
  return uint32_t(lo) | (uint32_t(hi) << 16);
}

// Past this distance from the nearest integer, x (1 / s) may be on the other side
// of a half than x / s: the quotient is within 16 in magnitude, the reciprocal,
// the product and the difference x - b err by 2^-24 or so each, relatively.
constexpr float kNearHalf = 0.5f - 0x1p-16f;

template <int GROUP, bool AFFINE, typename T, typename S>
__global__ __launch_bounds__(kBlock) void quantize_kernel(const T* __restrict__ x, int64_t n_octets,
                                                          uint32_t* __restrict__ codes,
                                                          S* __restrict__ scales, S* __restrict__ biases) {
  const int64_t g = block_id() * kBlock + threadIdx.x;
  if (g >= n_octets) return;             // groups are whole: every lane of one is here
  float v[8];
  load8(x + g * 8, v);
  // fmaxf drops a NaN: whether there is one, or an infinity, is carried beside it
  float hi = v[0], lo = -v[0], odd = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi = fmaxf(hi, AFFINE ? v[i] : fabsf(v[i]));
    if (AFFINE) lo = fmaxf(lo, -v[i]);
    odd = fmaf(v[i], 0.f, odd);          // NaN once some value is not finite
  }
  if (!AFFINE) hi = fmaxf(hi, fabsf(v[0]));
  hi = group_max<GROUP>(hi);
  if (AFFINE) lo = -group_max<GROUP>(lo);
  float bad = group_max<GROUP>(odd == 0.f ? 0.f : 1.f);
  const float b = AFFINE ? round_scale(lo, scales) : 0.f;
  const float range = AFFINE ? hi - lo : hi;
  float s = round_scale(range * (AFFINE ? 1.f / 15.f : 1.f / 7.f), scales);
  if (!(range < __builtin_inff()) || (AFFINE && !(fabsf(b) < __builtin_inff()))) bad = 1.f;

  // a scale near the smallest numbers has no finite reciprocal: scale all up, exactly
  const float up = s < 0x1p-100f ? 0x1p+64f : 1.f;
  const float su = s * up;
  const float inv = s > 0.f ? 1.f / su : 0.f;
  float q[8], far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float w = (AFFINE ? v[i] - b : v[i]) * up * inv;
    q[i] = rintf(w);
    far = fmaxf(far, fabsf(w - q[i]));
  }
  if (s > 0.f && far > kNearHalf) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!(fabsf(q[i]) <= 32.f)) continue;            // clamped whichever side it is on
      // x - b = d + e exactly (two-sum); the remainder d + e - q s against half a
      // step: near a half the fused product leaves it exact, else its sign stands
      const float xu = v[i] * up, bu = b * up;
      const float d = AFFINE ? xu - bu : xu;
      const float t = d - xu;
      const float e = AFFINE ? (xu - (d - t)) - (bu + t) : 0.f;
      const float above = fmaf(-(q[i] + 0.5f), su, d) + e;     // over q + 1/2
      const float below = fmaf(-(q[i] - 0.5f), su, d) + e;     // under q - 1/2
      const bool odd_q = int(q[i]) & 1;
      if (above > 0.f || (above == 0.f && odd_q)) q[i] += 1.f;
      else if (below < 0.f || (below == 0.f && odd_q)) q[i] -= 1.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf(AFFINE ? q[i] : q[i] + 8.f, 0.f), 15.f);
  const bool is_bad = bad != 0.f;
  codes[g] = is_bad ? (AFFINE ? 0u : 0x88888888u) : pack8(q);
  if (g % (GROUP / 8) == 0) {
    const float nan = __uint_as_float(0x7fc00000u);
    put_scale(scales, g / (GROUP / 8), is_bad ? nan : s);
    if (AFFINE) put_scale(biases, g / (GROUP / 8), is_bad ? nan : b);
  }
}

template <int GROUP, bool AFFINE, typename T, typename S>
__global__ __launch_bounds__(kBlock) void dequant_kernel(const uint32_t* __restrict__ codes,
                                                         const S* __restrict__ scales,
                                                         const S* __restrict__ biases, int64_t n_octets,
                                                         T* __restrict__ out) {
  const int64_t g = block_id() * kBlock + threadIdx.x;
  if (g >= n_octets) return;
  const uint32_t c = codes[g];
  const float s = scale_value(scales, g / (GROUP / 8));
  const float b = AFFINE ? scale_value(biases, g / (GROUP / 8)) : 0.f;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int q = int((c >> (4 * i)) & 15u);
    v[i] = AFFINE ? fmaf(s, float(q), b) : s * float(q - 8);
  }
  store8(out + g * 8, v);
}

template <typename F>
void by_group(int group, bool affine, F f) {
  using std::integral_constant;
  const auto go = [&](auto g) {
    if (affine) f(g, std::true_type());
    else f(g, std::false_type());
  };
  if (group == 32) go(integral_constant<int, 32>());
  else if (group == 64) go(integral_constant<int, 64>());
  else go(integral_constant<int, 128>());
}

}  // namespace

hipError_t launch_quantize_int4(const void* x, int x_bf16, int64_t n_elems, int group, void* codes,
                                void* scales, void* biases, int scales_bf16, hipStream_t stream) {
  const int64_t octets = n_elems / 8;
  const dim3 blocks = grid_of((octets + kBlock - 1) / kBlock);
  by_group(group, biases != nullptr, [&](auto g, auto affine) {
    const auto run = [&](auto* p, auto* s) {
      using T = std::remove_reference_t<decltype(*p)>;
      using S = std::remove_reference_t<decltype(*s)>;
      quantize_kernel<decltype(g)::value, decltype(affine)::value, std::remove_const_t<T>, S>
          <<<blocks, kBlock, 0, stream>>>(p, octets, static_cast<uint32_t*>(codes), s, static_cast<S*>(biases));
    };
    const auto with_x = [&](auto* p) {
      if (scales_bf16) run(p, static_cast<uint16_t*>(scales));
      else run(p, static_cast<float*>(scales));
    };
    if (x_bf16) with_x(static_cast<const uint16_t*>(x));
    else with_x(static_cast<const float*>(x));
  });
  return hipGetLastError();
}

hipError_t launch_dequant_int4(const void* codes, const void* scales, const void* biases, int scales_bf16,
                               int64_t n_elems, int group, void* out, int out_bf16, hipStream_t stream) {
  const int64_t octets = n_elems / 8;
  const dim3 blocks = grid_of((octets + kBlock - 1) / kBlock);
  by_group(group, biases != nullptr, [&](auto g, auto affine) {
    const auto run = [&](auto* o, auto* s) {
      using T = std::remove_reference_t<decltype(*o)>;
      using S = std::remove_const_t<std::remove_reference_t<decltype(*s)>>;
      dequant_kernel<decltype(g)::value, decltype(affine)::value, T, S><<<blocks, kBlock, 0, stream>>>(
          static_cast<const uint32_t*>(codes), s, static_cast<const S*>(biases), octets, o);
    };
    const auto to = [&](auto* o) {
      if (scales_bf16) run(o, static_cast<const uint16_t*>(scales));
      else run(o, static_cast<const float*>(scales));
    };
    if (out_bf16) to(static_cast<uint16_t*>(out));
    else to(static_cast<float*>(out));
  });
  return hipGetLastError();
}

}  // namespace moe
