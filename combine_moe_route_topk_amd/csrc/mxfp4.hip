// MXFP4 (OCP microscaling): E2M1 elements, two per byte (even element in the
// low nibble), one E8M0 scale per 32 consecutive elements of a row.
//
// Quantise, per block of 32 with largest magnitude m and E = its fp32 exponent
// field:  scale byte X = max(E - 2, 0)  (2^(X-127) = 2^(floor(log2 m) - 2), 2
// being the exponent of the largest E2M1 value 6),  code = round to nearest
// even of x / 2^(X-127) on the E2M1 grid {0, .5, 1, 1.5, 2, 3, 4, 6},
// magnitudes above 6 saturating.  The division is exact.  A block that holds a
// NaN or an infinity gets scale 255 (NaN) and codes 0.
// Dequantise: value * 2^(X-127), exact in fp32 before one rounding; X = 255
// gives NaN.
//
// Rows are multiples of 32 elements, so a matrix is one flat run of blocks.
// Both kernels only stream: 8 elements per lane per step, four lanes to a
// block, so loads and stores are whole lines per wave and the block maximum is
// two lane exchanges within a quad.
#include "device_common.hpp"
#include "launch.hpp"

namespace moe {

namespace {

constexpr int kBlock = 256;
// Groups of 8 per thread.  Measured on 16384 x 14336 bf16, quantising: 1, 2, 4
// and 8 groups 98, 96, 107 and 106 us (2 also best at 4096 x 7168); back to
// bf16, with ordinary stores: 113, 105, 100 and 106 us.
constexpr int kQuant = 2, kDequant = 4;

// bf16 x beyond the last-level cache (256 MB) is loaded past it: 98 -> 90 us at
// 470 MB (6.6 TB/s); at 59 MB, which the cache holds, that costs 17% (11.9 ->
// 13.9).  fp32 x of 940 MB takes 190 us either way.
constexpr int64_t kCacheBytes = int64_t(256) << 20;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// 8 consecutive elements as fp32.
template <bool NT>
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const u32x4 a = *reinterpret_cast<const u32x4*>(p);
  const u32x4 b = *reinterpret_cast<const u32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) { v[i] = __uint_as_float(a[i]); v[4 + i] = __uint_as_float(b[i]); }
}
template <bool NT>
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const u32x4* q = reinterpret_cast<const u32x4*>(p);
  const u32x4 a = NT ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack_bf16x2(a[i], v[2 * i], v[2 * i + 1]);
}
// Values are stored past the caches: 100 -> 84 us for 16384 x 14336 bf16 (7.1
// TB/s), 11.9 -> 9.9 for 4096 x 7168.
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

// Maximum over the four lanes of a quad (DPP quad permutes).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = __builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xF, 0xF, true);   // lanes 1 0 3 2
  v = o > v ? o : v;
  o = __builtin_amdgcn_update_dpp(0, int(v), 0x4E, 0xF, 0xF, true);            // lanes 2 3 0 1
  return o > v ? o : v;
}

template <typename T, bool NT>
__global__ __launch_bounds__(kBlock) void quantize_kernel(const T* __restrict__ x, int64_t n_groups,
                                                          uint32_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  const int64_t g0 = block_id() * (kBlock * kQuant) + threadIdx.x;
  float v[kQuant][8];
#pragma unroll
  for (int u = 0; u < kQuant; ++u) {
    const int64_t g = g0 + u * kBlock;
    if (g < n_groups) load8<NT>(x + g * 8, v[u]);   // quads are whole: n_groups is a multiple of 4
  }
#pragma unroll
  for (int u = 0; u < kQuant; ++u) {
    const int64_t g = g0 + u * kBlock;
    if (g >= n_groups) break;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = __float_as_uint(v[u][i]) & 0x7fffffffu;
      m = b > m ? b : m;
    }
    const int e = int(quad_max(m) >> 23);
    const bool bad = e == 255;
    const int byte = e > 2 ? e - 2 : 0;
    // 2^(byte - 127) as the instruction's scale operand, of which it takes the
    // exponent field; a field of 0 would be a subnormal: scale the block up instead
    uint32_t q = 0;
    if (byte == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] *= 0x1p+64f;
    }
    const float s = __uint_as_float(uint32_t(byte == 0 ? 64 : byte) << 23);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[u][0], v[u][1], s, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[u][2], v[u][3], s, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[u][4], v[u][5], s, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[u][6], v[u][7], s, 3);
    codes[g] = bad ? 0u : q;
    if ((threadIdx.x & 3) == 0) scales[g >> 2] = uint8_t(bad ? 255 : byte);
  }
}

template <typename T>
__global__ __launch_bounds__(kBlock) void dequant_kernel(const uint32_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales,
                                                         int64_t n_groups, T* __restrict__ out) {
  const int64_t g0 = block_id() * (kBlock * kDequant) + threadIdx.x;
  uint32_t q[kDequant];
  int byte[kDequant];
#pragma unroll
  for (int u = 0; u < kDequant; ++u) {
    const int64_t g = g0 + u * kBlock;
    if (g < n_groups) { q[u] = codes[g]; byte[u] = scales[g >> 2]; }
  }
#pragma unroll
  for (int u = 0; u < kDequant; ++u) {
    const int64_t g = g0 + u * kBlock;
    if (g >= n_groups) break;
    const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.f, 0),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.f, 2),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.f, 3)};
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = __builtin_ldexpf(p[i >> 1][i & 1], byte[u] - 127);
      v[i] = byte[u] == 255 ? __uint_as_float(0x7fc00000u) : r;
    }
    store8(out + g * 8, v);
  }
}

}  // namespace

hipError_t launch_quantize_mxfp4(const void* x, int x_bf16, int64_t n_elems, void* codes,
                                 uint8_t* scales, hipStream_t stream) {
  const int64_t groups = n_elems / 8;
  const dim3 blocks = grid_of((groups + kBlock * kQuant - 1) / (kBlock * kQuant));
  auto run = [&](auto kernel, auto* p) {
    kernel<<<blocks, kBlock, 0, stream>>>(p, groups, static_cast<uint32_t*>(codes), scales);
  };
  if (!x_bf16)
    run(quantize_kernel<float, false>, static_cast<const float*>(x));
  else if (n_elems * 2 > kCacheBytes)
    run(quantize_kernel<uint16_t, true>, static_cast<const uint16_t*>(x));
  else
    run(quantize_kernel<uint16_t, false>, static_cast<const uint16_t*>(x));
  return hipGetLastError();
}

hipError_t launch_dequant_mxfp4(const void* codes, const uint8_t* scales, int64_t n_elems, void* out,
                                int out_bf16, hipStream_t stream) {
  const int64_t groups = n_elems / 8;
  const dim3 blocks = grid_of((groups + kBlock * kDequant - 1) / (kBlock * kDequant));
  if (out_bf16)
    dequant_kernel<uint16_t><<<blocks, kBlock, 0, stream>>>(static_cast<const uint32_t*>(codes), scales,
                                                            groups, static_cast<uint16_t*>(out));
  else
    dequant_kernel<float><<<blocks, kBlock, 0, stream>>>(static_cast<const uint32_t*>(codes), scales,
                                                         groups, static_cast<float*>(out));
  return hipGetLastError();
}

}  // namespace moe
