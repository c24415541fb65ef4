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
// Octets per thread, and the size from which x is loaded past the last-level cache
// (256 MB).  Measured on 114688 x 4096 bf16, groups of 128, quantising with 1, 2 and
// 4 octets: 237, 189 and 193 us (1.18 GB, 6.2 TB/s); back to bf16 with 1, 2, 4 and 8:
// 226, 161, 165 and 166 (7.2 TB/s).  With ordinary loads quantising took 222 us.  (The
// rounding below then took more instructions; with 2 octets it is 177 us now, 6.7 TB/s.)
// 2113 x 7168 fp32 with biases per 32: 13.5 and 7.8 us (the launches and the groups'
// exchanges; 71 MB of x would take 9).
constexpr int kQuant = 2, kDequant = 4;
constexpr int64_t kCacheBytes = int64_t(256) << 20;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// 8 consecutive elements as loaded, NT past the last-level cache, and as fp32.
template <typename T>
struct Octet;
template <>
struct Octet<float> {
  u32x4 a[2];
  template <bool NT>
  __device__ __forceinline__ void load(const float* p) {
    const u32x4* q = reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 2; ++i) a[i] = NT ? __builtin_nontemporal_load(q + i) : q[i];
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(a[i / 4][i % 4]);
  }
  // largest magnitude, as fp32 bits: a NaN or an infinity is above all numbers
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, a[i / 4][i % 4] & 0x7fffffffu);
    return m;
  }
};
template <>
struct Octet<uint16_t> {
  u32x4 a;
  template <bool NT>
  __device__ __forceinline__ void load(const uint16_t* p) {
    const u32x4* q = reinterpret_cast<const u32x4*>(p);
    a = NT ? __builtin_nontemporal_load(q) : *q;
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack_bf16x2(a[i], v[2 * i], v[2 * i + 1]);
  }
  __device__ __forceinline__ uint32_t top() const {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, a[i] & 0x7fff7fffu));
    return uint32_t(max(m.x, m.y)) << 16;
  }
};
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
// v rounded to the scales' type
__device__ __forceinline__ float round_scale(float v, float*) { return v; }
__device__ __forceinline__ float round_scale(float v, uint16_t*) { return float(__bf16(v)); }
__device__ __forceinline__ void put_scale(float* s, int64_t i, float v) { s[i] = v; }
__device__ __forceinline__ void put_scale(uint16_t* s, int64_t i, float v) { s[i] = uint16_t(__float_as_uint(v) >> 16); }   // rounded already

template <int CTRL>
__device__ __forceinline__ float row_step(float v) {
  const int b = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
template <int CTRL>
__device__ __forceinline__ uint32_t row_step(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(int(v), int(v), CTRL, 0xF, 0xF, false));
}
// Maximum over the GROUP / 8 lanes of a group, in each of them.
template <int GROUP, typename V>
__device__ __forceinline__ V group_max(V v) {
  v = larger(v, row_step<0xB1>(v));                     // lanes 1 0 3 2
  v = larger(v, row_step<0x4E>(v));                     // lanes 2 3 0 1
  if (GROUP >= 64) v = larger(v, row_step<0x141>(v));   // row_half_mirror
  if (GROUP >= 128) v = larger(v, row_step<0x140>(v));  // row_mirror
  return v;
}

// 8 codes of 0 .. 15, held as floats, the first in the lowest nibble.
__device__ __forceinline__ uint32_t pack8(const float (&q)[8]) {
  const float lo = fmaf(q[3], 4096.f, fmaf(q[2], 256.f, fmaf(q[1], 16.f, q[0])));
  const float hi = fmaf(q[7], 4096.f, fmaf(q[6], 256.f, fmaf(q[5], 16.f, q[4])));
  return uint32_t(lo) | (uint32_t(hi) << 16);
}

// Past this distance from the nearest integer, x (1 / s) may be on the other side
// of a half than x / s: for a quotient within 16 in magnitude, since the reciprocal,
// the product and the difference x - b err by 2^-24 or so each, relatively.  Larger
// ones, of either sign, come up where a bf16 bias is far from the group's minimum for
// its range; they are clamped to 0 or 15 whichever way they are rounded.
constexpr float kNearHalf = 0.5f - 0x1p-16f;

// Of bf16 x and s no slow path is needed: with mantissas of 8 bits a quotient of at
// least 1/4 that is no half is 2^-11 or more away from every half, so x (1 / s)
// rounded to multiples of 2^-12, which the sum with 2^11 does, is a half when x / s is
// one and on the same side of it when not.  2^23 more rounds that to a whole number,
// ties to even, in the sum's low bits, which are added up as integers.  Ties are common
// there (3 waves of 8 held one): 114688 x 4096 bf16 takes 181 us so, 188 with the
// codes taken from floats and 265 with the remainders.
constexpr float kGrid = 0x1p+11f, kWhole = 0x1p+23f;
constexpr uint32_t kWholeBits = 0x4b000800u;   // of 2^23 + 2^11

// The codes and, in the first lane of each group, the scale (and bias) of an octet.
template <int GROUP, bool AFFINE, typename T, typename S>
__device__ __forceinline__ void quantize_octet(const Octet<T>& x, int64_t g, uint32_t* __restrict__ codes,
                                               S* __restrict__ scales, S* __restrict__ biases) {
  constexpr float kZero = AFFINE ? 0.f : 8.f;
  float v[8], b = 0.f, range;
  x.values(v);
  const uint32_t top = group_max<GROUP>(x.top());
  bool bad = top >= 0x7f800000u;
  if (AFFINE) {
    float hi = v[0], lo = -v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) { hi = fmaxf(hi, v[i]); lo = fmaxf(lo, -v[i]); }
    lo = -group_max<GROUP>(lo);
    range = group_max<GROUP>(hi) - lo;
    b = round_scale(lo, scales);
    bad = bad || !(range < __builtin_inff()) || !(fabsf(b) < __builtin_inff());
  } else {
    range = __uint_as_float(top);
  }
  const float s = round_scale(range * (AFFINE ? 1.f / 15.f : 1.f / 7.f), scales);

  // a scale near the smallest numbers has no finite reciprocal: scale all up, exactly
  float su = s, bu = b;
  if (s < 0x1p-100f) {
    su *= 0x1p+64f;
    bu *= 0x1p+64f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= 0x1p+64f;
    // elsewhere a symmetric quotient is at most 7 (1 + 2^-8); one whose scale is below
    // the normal numbers may be larger, and is clamped here, off every half
    if (!AFFINE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], -8.25f * su), 7.25f * su);
    }
  }
  const float inv = su > 0.f ? __builtin_amdgcn_rcpf(su) : 0.f;
  uint32_t packed;
  if constexpr (!AFFINE && sizeof(T) == 2 && sizeof(S) == 2) {
    packed = 0u - kWholeBits * 0x11111111u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      packed += __float_as_uint(fmaf(v[i], inv, kZero + kGrid) + kWhole) << (4 * i);
  } else {
    float q[8], far = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = fmaf(AFFINE ? v[i] - bu : v[i], inv, kZero);
      q[i] = rintf(w);
      far = fmaxf(far, fabsf(w - q[i]));
    }
    if (su > 0.f && far > kNearHalf) {
      const float half = 0.5f * su;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // v - b = d + e exactly (two-sum).  The remainder d + e - q s is exact where it
        // is near half a step, and otherwise on its side of that.
        const float p = q[i] - kZero;
        const float d = AFFINE ? v[i] - bu : v[i];
        const float t = d - v[i];
        const float e = AFFINE ? (v[i] - (d - t)) - (bu + t) : 0.f;
        const float rest = fmaf(-p, su, d);
        const float up = copysignf(1.f, rest);
        const float over = AFFINE ? fmaf(up, e, fabsf(rest) - half) : fabsf(rest) - half;   // past half a step
        const bool odd = rintf(0.5f * p) != 0.5f * p;
        q[i] += (over > 0.f) | ((over == 0.f) & odd) ? up : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf(q[i], 0.f), 15.f);
    packed = pack8(q);
  }
  codes[g] = bad ? (AFFINE ? 0u : 0x88888888u) : packed;
  if (g % (GROUP / 8) == 0) {
    const float nan = __uint_as_float(0x7fc00000u);
    put_scale(scales, g / (GROUP / 8), bad ? nan : s);
    if (AFFINE) put_scale(biases, g / (GROUP / 8), bad ? nan : b);
  }
}

template <int GROUP, bool AFFINE, bool NT, typename T, typename S>
__global__ __launch_bounds__(kBlock) void quantize_kernel(const T* __restrict__ x, int64_t n_octets,
                                                          uint32_t* __restrict__ codes,
                                                          S* __restrict__ scales, S* __restrict__ biases) {
  const int64_t g0 = block_id() * (kBlock * kQuant) + threadIdx.x;
  Octet<T> o[kQuant];
#pragma unroll
  for (int u = 0; u < kQuant; ++u)
    if (g0 + u * kBlock < n_octets) o[u].template load<NT>(x + (g0 + u * kBlock) * 8);
#pragma unroll
  for (int u = 0; u < kQuant; ++u) {
    if (g0 + u * kBlock >= n_octets) break;            // groups are whole: every lane of one is here
    quantize_octet<GROUP, AFFINE>(o[u], g0 + u * kBlock, codes, scales, biases);
  }
}

template <int GROUP, bool AFFINE, typename T, typename S>
__global__ __launch_bounds__(kBlock) void dequant_kernel(const uint32_t* __restrict__ codes,
                                                         const S* __restrict__ scales,
                                                         const S* __restrict__ biases, int64_t n_octets,
                                                         T* __restrict__ out) {
  const int64_t g0 = block_id() * (kBlock * kDequant) + threadIdx.x;
  uint32_t c[kDequant];
  float s[kDequant], b[kDequant];
#pragma unroll
  for (int u = 0; u < kDequant; ++u) {
    const int64_t g = g0 + u * kBlock;
    if (g >= n_octets) break;
    c[u] = codes[g];
    s[u] = scale_value(scales, g / (GROUP / 8));
    b[u] = AFFINE ? scale_value(biases, g / (GROUP / 8)) : 0.f;
  }
#pragma unroll
  for (int u = 0; u < kDequant; ++u) {
    const int64_t g = g0 + u * kBlock;
    if (g >= n_octets) break;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = int((c[u] >> (4 * i)) & 15u);
      v[i] = AFFINE ? fmaf(s[u], float(q), b[u]) : s[u] * float(q - 8);
    }
    store8(out + g * 8, v);
  }
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
  const dim3 blocks = grid_of((octets + kBlock * kQuant - 1) / (kBlock * kQuant));
  by_group(group, biases != nullptr, [&](auto g, auto affine) {
    const auto run = [&](auto* p, auto* s) {
      using T = std::remove_reference_t<decltype(*p)>;
      using S = std::remove_reference_t<decltype(*s)>;
      constexpr int kG = decltype(g)::value;
      constexpr bool kA = decltype(affine)::value;
      const bool past = n_elems * int64_t(sizeof(T)) > kCacheBytes;
      const auto launch = [&](auto kernel) {
        kernel<<<blocks, kBlock, 0, stream>>>(p, octets, static_cast<uint32_t*>(codes), s, static_cast<S*>(biases));
      };
      if (past) launch(quantize_kernel<kG, kA, true, std::remove_const_t<T>, S>);
      else launch(quantize_kernel<kG, kA, false, std::remove_const_t<T>, S>);
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
  const dim3 blocks = grid_of((octets + kBlock * kDequant - 1) / (kBlock * kDequant));
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
