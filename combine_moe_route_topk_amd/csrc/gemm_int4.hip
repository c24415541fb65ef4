// Expert products with 4-bit integer weights: bf16 rows x, row r taking expert
// e_r, weights w = s (q - 8) or s q + b with one s (and b) per G of K,
//   y[r, n] = sum_groups s[n, grp] (sum_{k in grp} q[n, k] x[r, k]) + (b or -8 s) X[r, grp],
// X[r, grp] the sum of x over the group; or silu(.) * (the same with w_up).
//
// Few rows per expert: the weights are most of the bytes, and each is read once
// per tile of 16 NB rows, straight from memory into registers.  A code becomes a
// bf16 number without rounding: a byte 0 .. 15 is q 2^-9 as an fp8 number (its
// subnormals and the binade above go on in equal steps), which one instruction
// per two codes turns into bf16 times 2^9.  v_mfma_f32_16x16x32_bf16 multiplies:
// rows of x are its A operand, 16 weight rows the B operand, so a lane holds
// results of the one weight row whose codes and scales it reads, and a group's
// fp32 sum is scaled in fp32.  X comes from the same instruction with a constant
// for B (-8 where there are no biases, which makes it the sum's start).
#include <type_traits>

#include "device_common.hpp"
#include "expert_tiles.hpp"
#include "launch.hpp"

namespace moe {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;              // of a workgroup, each a quarter of K
constexpr int kT = 4;                  // 16-column tiles of a wave: 64 columns
constexpr int kStep = 128;             // elements of K that one 16-byte load per lane covers

struct Product {
  const uint16_t* rows;
  int n_rows, K;
  const int32_t* index;                // expert offsets, or with direct the expert of each row
  const int32_t* order;                // row of each grouped position, or null
  int n_experts, N;
  const uint8_t* w[2];                 // w and w_up
  const void* s[2];
  const void* b[2];
  void* y;
  int y_bf16, glu, direct, n_groups;
};

// Two codes as bf16, from bytes 0 and 1 of v, or 2 and 3.
template <bool HI>
__device__ __forceinline__ uint32_t codes2(uint32_t v) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.f, HI));
}
// 8 codes (a dword) as the B operand: elements 0 2 4 6 1 3 5 7.
__device__ __forceinline__ bf16x8 codes8(uint32_t v) {
  const uint32_t even = v & 0x0f0f0f0fu, odd = (v >> 4) & 0x0f0f0f0fu;
  return __builtin_bit_cast(bf16x8, u32x4{codes2<false>(even), codes2<true>(even), codes2<false>(odd), codes2<true>(odd)});
}
// 8 elements of x in the order of codes8.
__device__ __forceinline__ bf16x8 evens_odds(u32x4 v) {
  return __builtin_bit_cast(bf16x8, u32x4{__builtin_amdgcn_perm(v.y, v.x, 0x05040100u), __builtin_amdgcn_perm(v.w, v.z, 0x05040100u),
                                          __builtin_amdgcn_perm(v.y, v.x, 0x07060302u), __builtin_amdgcn_perm(v.w, v.z, 0x07060302u)});
}
// Lane (n, g) = (l % 16, l / 16) holds dwords 0 .. 3 of 16-byte piece g; after it
// the dwords g of pieces 0 .. 3.
__device__ __forceinline__ u32x4 transpose4(u32x4 v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ float scale_at(const float* s, int i) { return s[i]; }
__device__ __forceinline__ float scale_at(const uint16_t* s, int i) { return bf16_to_f32(s[i]); }

// 1 / (1 + e^-a) a from expf and a division, for fp32 results.
__device__ __forceinline__ float silu_f32(float a) { return a / (1.f + expf(-a)); }

// G: elements per scale; S: their type; BIAS: affine; NB: 16-row blocks of a tile.
// K % G == 0, so K is a multiple of 32; past K, x is zero and the last codes and
// scales are read again.
template <int G, typename S, bool BIAS, int NB>
__global__ __launch_bounds__(kWaves * kWave) void stream_kernel(Product p) {
  constexpr int kTM = 16 * NB;
  constexpr int kPer = kStep / G;      // groups in a step
  constexpr bool kSplit = G < kStep;   // the four lanes of a weight row are in different groups
  constexpr int kPitch = 16 * kT + 4;
  __shared__ float s_sum[kWaves][kTM][kPitch];
  __shared__ int s_rows[kTM];

  // workgroup b runs on XCD b % 8; XCD x takes row tiles x, x + 8, ..., all
  // column groups of one back to back
  const int slot = blockIdx.x / kXcds;
  const int m_idx = (slot / p.n_groups) * kXcds + blockIdx.x % kXcds, grp = slot % p.n_groups;
  const int tid = threadIdx.x, lane = lane_id();
  const Tile tile = p.direct ? direct_tile(m_idx, p.index, p.n_rows, p.n_experts, s_rows)
                             : find_tile<kTM>(m_idx, p.index, p.n_experts, p.n_rows);
  if (!tile.valid) return;             // whole workgroup
  if (!p.direct && tid < kTM && tile.row0 + tid < tile.row_end)   // live rows
    s_rows[tid] = p.order ? p.order[tile.row0 + tid] : tile.row0 + tid;
  __syncthreads();
  // rows of the tile (row_end is the expert's); past them its first is read, and never stored
  const int live = tile.row_end - tile.row0 < kTM ? tile.row_end - tile.row0 : kTM;

  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int n = lane & 15, g = lane >> 4;
  const int cols = p.glu ? 8 * kT : 16 * kT;   // output columns of the workgroup
  const int col0 = grp * cols;
  const int n_scales = p.K / G;

  const uint16_t* x_ptr[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) x_ptr[i] = p.rows + int64_t(s_rows[16 * i + n < live ? 16 * i + n : 0]) * p.K;
  const uint8_t* w_ptr[kT];
  const S *s_ptr[kT], *b_ptr[kT];
#pragma unroll
  for (int t = 0; t < kT; ++t) {
    const int up = p.glu && t >= kT / 2;
    int c = col0 + 16 * (up ? t - kT / 2 : t) + n;
    if (c >= p.N) c = p.N - 1;                 // partial last group; never stored
    const int64_t row = int64_t(tile.expert) * p.N + c;
    w_ptr[t] = (up ? p.w[1] : p.w[0]) + row * (p.K / 2);
    s_ptr[t] = static_cast<const S*>(up ? p.s[1] : p.s[0]) + row * n_scales;
    b_ptr[t] = BIAS ? static_cast<const S*>(up ? p.b[1] : p.b[0]) + row * n_scales : nullptr;
  }

  f32x4 acc[NB][kT];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int t = 0; t < kT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  // one step: codes q, scales and biases of its groups, x as four A operands
  const uint32_t c1 = BIAS ? 0x3f803f80u : 0xc100c100u;        // 1, or -8, twice in bf16
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{c1, c1, c1, c1});
  auto multiply = [&](const u32x4 (&q)[kT], const float (&sc)[kT][kPer], const float (&bi)[kT][kPer],
                      const u32x4 (&x)[NB][4]) {
    bf16x8 a[NB][4];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) a[i][j] = evens_odds(x[i][j]);
    f32x4 sum[NB][kPer];                       // X, or -8 X
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int h = 0; h < kPer; ++h) {
        sum[i][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4 / kPer; ++j)
          sum[i][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i][h * (4 / kPer) + j], ones, sum[i][h], 0, 0, 0);
      }
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      const u32x4 v = kSplit ? transpose4(q[t]) : q[t];
      bf16x8 b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = codes8(v[j]);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int h = 0; h < kPer; ++h) {
          f32x4 d = BIAS ? f32x4{0.f, 0.f, 0.f, 0.f} : sum[i][h];
#pragma unroll
          for (int j = 0; j < 4 / kPer; ++j)
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i][h * (4 / kPer) + j], b[h * (4 / kPer) + j], d, 0, 0, 0);
#pragma unroll
          for (int v4 = 0; v4 < 4; ++v4) {
            acc[i][t][v4] = fmaf(sc[t][h], d[v4], acc[i][t][v4]);
            if (BIAS) acc[i][t][v4] = fmaf(bi[t][h], sum[i][h][v4], acc[i][t][v4]);
          }
        }
    }
  };

  const int pieces = p.K / 32;
  auto load = [&](int step, u32x4 (&q)[kT], float (&sc)[kT][kPer], float (&bi)[kT][kPer], u32x4 (&x)[NB][4]) {
    const int piece = 4 * step + g;
    const int at = piece < pieces ? piece : pieces - 1;
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      q[t] = *reinterpret_cast<const u32x4*>(w_ptr[t] + 16 * at);
#pragma unroll
      for (int h = 0; h < kPer; ++h) {
        const int k = step * kPer + h < n_scales ? step * kPer + h : n_scales - 1;
        sc[t][h] = scale_at(s_ptr[t], k);
        bi[t][h] = BIAS ? scale_at(b_ptr[t], k) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = kSplit ? kStep * step + 32 * j + 8 * g : kStep * step + 32 * g + 8 * j;
        x[i][j] = k < p.K ? *reinterpret_cast<const u32x4*>(x_ptr[i] + k) : u32x4{0, 0, 0, 0};
      }
  };

  const int n_steps = (p.K + kStep - 1) / kStep;
  const int first = int(int64_t(n_steps) * wave / kWaves), last = int(int64_t(n_steps) * (wave + 1) / kWaves);
  for (int step = first; step < last; ++step) {
    u32x4 q[kT], x[NB][4];
    float sc[kT][kPer], bi[kT][kPer];
    load(step, q, sc, bi, x);
    multiply(q, sc, bi, x);
  }

  // the four quarters of K, added in order: lane (n, g) holds rows 4 g .. 4 g + 3
  // of column n of each 16 x 16 tile
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) s_sum[wave][16 * i + 4 * g + v][16 * t + n] = acc[i][t][v];
  __syncthreads();
  const int quads = cols / 4;
  for (int at = tid; at < live * quads; at += kWaves * kWave) {
    const int r = at / quads, c = at % quads * 4;
    float o[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float a = 0.f, u = 0.f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        a += s_sum[k][r][c + v];
        if (p.glu) u += s_sum[k][r][8 * kT + c + v];
      }
      o[v] = p.glu ? (p.y_bf16 ? silu(a) : silu_f32(a)) * u : a;
    }
    const int64_t row = int64_t(s_rows[r]) * p.N;
    if (p.y_bf16) {
      store4(static_cast<uint16_t*>(p.y) + row, col0 + c, p.N, p.N % 4 == 0, o);
    } else {
      float* out = static_cast<float*>(p.y) + row;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (col0 + c + v < p.N) out[col0 + c + v] = o[v];
    }
  }
}

// Mean rows per expert from which a tile holds 32 rows.
constexpr int64_t kNarrowRows = 10;

struct Shape {
  bool direct;
  int nb, col_groups;
  int64_t blocks;
};
Shape shape_of(const Int4Product& g) {
  Shape s{};
  s.nb = g.n_rows < kNarrowRows * g.n_experts ? 1 : 2;
  s.direct = s.nb == 1 && g.n_rows <= kDirectRows;
  const int cols = g.w_up ? 8 * kT : 16 * kT;
  s.col_groups = int((g.n_dim + cols - 1) / cols);
  s.blocks = (most_tiles(g.n_rows, g.n_experts, 16 * s.nb) + kXcds - 1) / kXcds * kXcds * s.col_groups;
  return s;
}

template <int G>
void launch_group(const Product& p, const Shape& s, bool scales_bf16, hipStream_t stream) {
  const auto go = [&](auto* type, auto bias, auto nb) {
    using S = std::remove_pointer_t<decltype(type)>;
    stream_kernel<G, S, decltype(bias)::value, decltype(nb)::value>
        <<<unsigned(s.blocks), kWaves * kWave, 0, stream>>>(p);
  };
  const auto rows = [&](auto* type, auto bias) {
    if (s.nb == 1) go(type, bias, std::integral_constant<int, 1>());
    else go(type, bias, std::integral_constant<int, 2>());
  };
  const auto form = [&](auto* type) {
    if (p.b[0]) rows(type, std::true_type());
    else rows(type, std::false_type());
  };
  if (scales_bf16) form(static_cast<uint16_t*>(nullptr));
  else form(static_cast<float*>(nullptr));
}

}  // namespace

int64_t gemm_int4_blocks(const Int4Product& g) { return shape_of(g).blocks; }

size_t gather_gemm_int4_workspace_bytes(int64_t n_rows, int n_experts) {
  return gather_layout(n_rows, n_experts).total;
}

hipError_t launch_gather_gemm_int4(const Int4Product& g, const int32_t* row_expert, void* workspace,
                                   hipStream_t stream) {
  const Shape s = shape_of(g);
  const int32_t *index = row_expert, *order = nullptr;
  if (!s.direct) {
    const hipError_t err = launch_grouping(row_expert, g.n_rows, g.n_experts, workspace, &index, &order, stream);
    if (err != hipSuccess) return err;
  }
  const auto u8 = [](const void* v) { return static_cast<const uint8_t*>(v); };
  const Product p{static_cast<const uint16_t*>(g.rows), int(g.n_rows), int(g.k_dim), index, order, g.n_experts,
                  int(g.n_dim), {u8(g.w), u8(g.w_up)}, {g.w_scales, g.w_up_scales}, {g.w_biases, g.w_up_biases},
                  g.y, g.y_bf16, g.w_up != nullptr, s.direct, s.col_groups};
  if (g.group == 32) launch_group<32>(p, s, g.scales_bf16, stream);
  else if (g.group == 64) launch_group<64>(p, s, g.scales_bf16, stream);
  else launch_group<128>(p, s, g.scales_bf16, stream);
  return hipGetLastError();
}

}  // namespace moe
