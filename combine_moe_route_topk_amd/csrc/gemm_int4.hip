// Expert products with 4-bit integer weights: bf16 rows x, row r taking expert
// e_r, weights w = s (q - 8) or s q + b with one s (and b) per G of K,
//   y[r, n] = sum_groups s[n, grp] (sum_{k in grp} q[n, k] x[r, k]) + (b or -8 s) X[r, grp],
// X[r, grp] the sum of x over the group; or silu(.) * (the same with w_up).
//
// Few rows per expert: the weights are most of the bytes, and each is read once
// per tile of 16 NB rows, in whole lines, and brought into the operands' order by
// LDS.  Two kernels, both below: stream_kernel splits K over the waves of a
// workgroup, wide_kernel the columns.  A code becomes a bf16 number without rounding: a byte 0 .. 15 is q 2^-9 as an fp8 number (its
// subnormals and the binade above go on in equal steps), which one instruction
// per two codes turns into bf16 times 2^9.  v_mfma_f32_16x16x32_bf16 multiplies:
// rows of x are its A operand, 16 weight rows the B operand, so a lane holds
// results of the one weight row whose codes and scales it reads, and a group's
// fp32 sum is scaled in fp32.  X comes from the same instruction with a constant
// for B (-8 where there are no biases, which makes it the sum's start).
//
// Measured, bytes of codes, scales and biases over the time:
//   1024 rows, 256 experts, K 7168, F 2048 SwiGLU, per 128:   654 us, 5.8 TB/s
//   128 rows, 8 experts, K 4096, F 14336 SwiGLU, per 32 + b:  154 us, 3.8 TB/s
//   48 rows, 8 experts, K 14336, N 4096, per 64, all fp32:     50 us, 5.3 TB/s
//   8 rows, 8 of 256 experts, K 2048, N 7168, per 128:         15 us, 4.1 TB/s
//   1 row, 1 expert, K 7168, N 2113, per 64 + b:               11 us, 0.8 TB/s
// The first runs at the rate of memory (with the clocks that its power allows: 636 to
// 728 us), the second at that of the vector units and LDS, which turn 4
// bits into bf16, scale every 32 elements and serve two row blocks; the last two are
// one start, a chain of loads and one end, with 29 and 9 KB to read for a workgroup.
#include <type_traits>

#include "device_common.hpp"
#include "expert_tiles.hpp"
#include "launch.hpp"

namespace moe {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;             // elements of K that one 16-byte load per lane covers
constexpr int kUnit = 256;             // elements of K asked for together: whole lines of a weight row

// Bytes of scales and biases of a weight row in a unit.  They share the registers
// with the codes: past 16, a SIMD holds one wave of a kernel whose tiles have 16 rows.
// Two waves keep at most 24 registers in memory at 16 bytes (4 to 24, and none below),
// and 72 to 212 past them.  One wave and two, 1024 rows over 128 experts, K 1408, N 2048:
// at 16 bytes (per 64 with bf16 biases) 161 and 103 us, at 32 (per 64, fp32 with biases)
// 163 and 219; 16 rows over 16 experts, K 4096, N 1024: 13.9 and 14.5, 14.9 and 34 us.
template <int G, typename S, bool BIAS>
constexpr int kScaleBytes = (BIAS ? 2 : 1) * int(sizeof(S)) * kUnit / G;

struct Product {
  const uint16_t* rows;
  int n_rows, K;
  const int32_t* index;                // expert offsets, or with direct the expert of each row
  const int32_t* order;                // row of each grouped position (null with direct)
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
// The N scales of a unit, as loaded, and the i-th of them.  They may begin at any
// element.
template <typename S, int N>
struct Scales {
  static constexpr int kWords = N * int(sizeof(S)) / 4;
  typedef uint32_t Words __attribute__((ext_vector_type(kWords)));
  typedef Words AnyWords __attribute__((aligned(sizeof(S))));
  Words v;
  __device__ __forceinline__ void load(const S* p) { v = *reinterpret_cast<const AnyWords*>(p); }
  __device__ __forceinline__ void set(int i, S x) {
    if constexpr (sizeof(S) == 4) v[i] = __builtin_bit_cast(uint32_t, x);
    else v[i / 2] = i % 2 ? (v[i / 2] & 0xffffu) | (uint32_t(x) << 16) : uint32_t(x);
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(S) == 4) return __uint_as_float(v[i]);
    else return __uint_as_float(i % 2 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
  }
};

template <int CTRL>
__device__ __forceinline__ float row_step(float v) {
  const int b = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, false));
}
// Sum of 8 elements of x.
__device__ __forceinline__ float piece_sum(u32x4 x) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = x[i];           // a copy: of an element itself the cast takes element 0
    sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, v), __builtin_bit_cast(bf16x2, 0x3f803f80u), sum, false);
  }
  return sum;
}

// 1 / (1 + e^-a) a from expf and a division, for fp32 results.
__device__ __forceinline__ float silu_f32(float a) { return a / (1.f + expf(-a)); }

// How the term (b or -8 s) X is added.
//   kSym: a constant operand of -8 makes it the start of a group's sum.
//   kFma: X by a constant operand of 1, then a multiply-add per group and result.
//   kMfma (bf16 biases, wide_kernel): the matrix cores add it for 16 groups at a time
//     from X as three bf16 terms, which hold all its 24 bits.
enum class Bias { kSym, kFma, kMfma };

// One step of 16 rows: a their A operands, b the codes of the KT tiles as B operands,
// us and ub the scales and biases of the unit's groups, ST the step of it.
template <int G, typename S, Bias HOW, int KT, int ST>
__device__ __forceinline__ void multiply(f32x4 (&acc)[KT], const bf16x8 (&a)[4], const bf16x8 (&b)[KT][4],
                                         const Scales<S, kUnit / G> (&us)[KT], const Scales<S, kUnit / G> (&ub)[KT]) {
  constexpr int kPer = kStep / G, kChain = 4 / kPer;           // groups of a step, MFMAs of a group
  constexpr uint32_t c = HOW == Bias::kSym ? 0xc100c100u : 0x3f803f80u;   // -8, or 1, twice in bf16
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{c, c, c, c});
#pragma unroll
  for (int h = 0; h < kPer; ++h) {
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};          // X, or -8 X
    if (HOW != Bias::kMfma) {
#pragma unroll
      for (int j = 0; j < kChain; ++j)
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[h * kChain + j], ones, sum, 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      f32x4 d = HOW == Bias::kSym ? sum : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kChain; ++j)
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[h * kChain + j], b[t][h * kChain + j], d, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        acc[t][r] = fmaf(us[t].at(ST * kPer + h), d[r], acc[t][r]);
        if (HOW == Bias::kFma) acc[t][r] = fmaf(ub[t].at(ST * kPer + h), sum[r], acc[t][r]);
      }
    }
  }
}

typedef __attribute__((address_space(3))) void* lds_ptr;

// 16 bytes per lane straight into LDS, lane l's at `to` + 16 l.
__device__ __forceinline__ void load_lds(const void* from, u32x4* to) {
  __builtin_amdgcn_global_load_lds(from, (lds_ptr)to, 16, 0, 0);
}
// G: elements per scale; S: their type; BIAS: affine; NB: 16-row blocks of a tile;
// KT: 16-column tiles of a wave (SwiGLU: half of them of w_up); WAVES of a
// workgroup, each with its part of K: no wave waits for another before the end.
//
// K advances in units of two steps.  Loads are made in whole lines by consecutive
// lanes (an L1 lookup serves 64 bytes of neighbouring lanes; in the operands' order,
// 16 rows apart, each lane cost one), and LDS puts them in the operands' order: x
// takes direct loads into it, 16 lanes a row and step; codes go to registers, 8 lanes
// a row, and from there to LDS when their unit's turn comes.  A turn waits for all
// that is on its way, takes both operands of its unit from LDS, asks for the next
// unit, and multiplies meanwhile.
// The 16-byte pieces of a row are swizzled by it (on the side of the global
// addresses), so that 16 lanes that read the same piece of 16 rows meet 64 banks.
// K % G == 0, so K is a multiple of 32; in a last, partial unit x is taken as zero
// past K and the last codes and scales are read again.
template <int G, typename S, bool BIAS, int NB, int KT, int WAVES>
__global__ __launch_bounds__(WAVES * kWave, (NB == 1 && (kScaleBytes<G, S, BIAS> <= 16 || KT == 2) ? 2 : 1)) void stream_kernel(Product p) {
  constexpr int kTM = 16 * NB;
  constexpr int kPer = kStep / G;      // groups in a step
  constexpr int kSteps = kUnit / kStep;
  constexpr bool kSplit = G < kStep;   // the four 32-element pieces of a step are in different groups
  constexpr int kSlot = NB * 4 * kWave;        // 16-byte pieces of a step of x
  constexpr int kCodes = KT * 2 * kWave;       // 16-byte pieces of a unit's codes
  constexpr int kPitch = 16 * KT;              // floats of a row of partial sums, kept in s_x at the end
  static_assert(kTM * kPitch * 4 <= kSteps * kSlot * 16, "the sums fit in s_x");
  __shared__ u32x4 s_x[WAVES][kSteps][kSlot];
  __shared__ u32x4 s_codes[WAVES][kCodes];
  __shared__ int s_rows[kTM];

  const int m_idx = blockIdx.x / p.n_groups, grp = blockIdx.x % p.n_groups;
  const int tid = threadIdx.x, lane = lane_id();
  const Tile tile = p.direct ? direct_tile(m_idx, p.index, p.n_rows, p.n_experts, s_rows)
                             : find_tile<kTM>(m_idx, p.index, p.n_experts, p.n_rows);
  if (!tile.valid) return;             // whole workgroup
  // rows of the tile (row_end is the expert's); past them its first is read, and never stored
  const int live = tile.row_end - tile.row0 < kTM ? tile.row_end - tile.row0 : kTM;
  if (!p.direct && tid < live) s_rows[tid] = p.order[tile.row0 + tid];
  __syncthreads();

  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int n = lane & 15, g = lane >> 4;
  const int cols = p.glu ? 8 * KT : 16 * KT;   // output columns of the workgroup
  const int col0 = grp * cols;
  const int n_scales = p.K / G;
  const int units = p.K / kUnit;               // whole ones
  const int first = int(int64_t(units) * wave / WAVES), last = int(int64_t(units) * (wave + 1) / WAVES);

  // weight row of row i of tile t, counted from the expert's first
  auto row_of = [&](int t, int i) {
    const int c = col0 + 16 * (p.glu && t >= KT / 2 ? t - KT / 2 : t) + i;
    return c < p.N ? c : p.N - 1;              // partial last group; never stored
  };
  auto of_up = [&](int t) { return p.glu && t >= KT / 2; };
  const int64_t row0 = int64_t(tile.expert) * p.N;
  const S *s_ptr[KT], *b_ptr[KT];
  uint32_t w_off[KT][2];                       // from the workgroup's first row, below 2^28
  const uint8_t* w_base[2] = {p.w[0] + (row0 + col0) * (p.K / 2), p.glu ? p.w[1] + (row0 + col0) * (p.K / 2) : nullptr};
#pragma unroll
  for (int t = 0; t < KT; ++t) {
    const int64_t row = row0 + row_of(t, n);
    s_ptr[t] = static_cast<const S*>(of_up(t) ? p.s[1] : p.s[0]) + row * n_scales;
    b_ptr[t] = BIAS ? static_cast<const S*>(of_up(t) ? p.b[1] : p.b[0]) + row * n_scales : nullptr;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 8 * h + lane / 8;          // its row of the tile, piece lane % 8 ^ i / 2
      w_off[t][h] = uint32_t(row_of(t, i) - col0) * uint32_t(p.K / 2) + 16 * ((lane % 8) ^ (i / 2));
    }
  }
  const uint16_t* x_ptr[NB][4];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 4 * j + lane / 16;         // row of the block, piece lane % 16 ^ r
      x_ptr[i][j] = p.rows + int64_t(s_rows[16 * i + r < live ? 16 * i + r : 0]) * p.K + 8 * ((lane % 16) ^ r);
    }

  f32x4 acc[NB][KT];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int t = 0; t < KT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Unit {
    u32x4 q[KT][2];                            // rows 8 h + l / 8 of tile t
    Scales<S, kUnit / G> s[KT], b[KT];
  };
  auto load_x = [&](int unit) {
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          load_lds(x_ptr[i][j] + (int64_t(unit) * kUnit + kStep * st), &s_x[wave][st][(4 * i + j) * kWave]);
  };
  auto load_w = [&](int unit, Unit& u) {
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      u.s[t].load(s_ptr[t] + int64_t(unit) * (kUnit / G));
      if (BIAS) u.b[t].load(b_ptr[t] + int64_t(unit) * (kUnit / G));
    }
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        u.q[t][h] = *reinterpret_cast<const u32x4*>((of_up(t) ? w_base[1] : w_base[0]) + int64_t(unit) * (kUnit / 2) + w_off[t][h]);
  };
  struct Operands {
    u32x4 x[kSteps][NB][4], q[kSteps][KT];
  };
  auto take = [&](const Unit& u, Operands& o) {
    u32x4* codes = s_codes[wave];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) codes[(2 * t + h) * kWave + lane] = u.q[t][h];
    // MFMA j takes from lane (n, g) the 8 elements of piece 4 j + g of x, or 4 g + j,
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o.x[st][i][j] = s_x[wave][st][4 * i * kWave + 16 * n + ((kSplit ? 4 * j + g : 4 * g + j) ^ n)];
    // and the codes in dword g of piece 4 st + j, or dword j of piece 4 st + g
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const u32x4* row = codes + 2 * t * kWave + 8 * n;
        if constexpr (kSplit) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o.q[st][t][j] = reinterpret_cast<const uint32_t*>(row + ((4 * st + j) ^ (n / 2)))[g];
        } else {
          o.q[st][t] = row[(4 * st + g) ^ (n / 2)];
        }
      }
  };

  auto step = [&](const Operands& o, const Scales<S, kUnit / G> (&us)[KT], const Scales<S, kUnit / G> (&ub)[KT], auto which) __attribute__((always_inline)) {
    constexpr int st = decltype(which)::value;
    bf16x8 b[KT][4];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) b[t][j] = codes8(o.q[st][t][j]);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      bf16x8 a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = evens_odds(o.x[st][i][j]);
      multiply<G, S, BIAS ? Bias::kFma : Bias::kSym, KT, st>(acc[i], a, b, us, ub);
    }
  };
  auto both_steps = [&](const Operands& o, const Scales<S, kUnit / G> (&us)[KT], const Scales<S, kUnit / G> (&ub)[KT]) __attribute__((always_inline)) {
    step(o, us, ub, std::integral_constant<int, 0>());
    step(o, us, ub, std::integral_constant<int, 1>());
  };
  if (first < last) {
    Unit u;
    Operands o;
    load_w(first, u);
    load_x(first);
    for (int at = first; at < last; ++at) {
      __builtin_amdgcn_s_waitcnt(0x0f70);      // every load has landed
      take(u, o);
      Scales<S, kUnit / G> us[KT], ub[KT];
#pragma unroll
      for (int t = 0; t < KT; ++t) { us[t] = u.s[t]; ub[t] = u.b[t]; }
      __builtin_amdgcn_s_waitcnt(0xc07f);      // and is read from LDS before more is asked for
      __builtin_amdgcn_sched_barrier(0);
      if (at + 1 < last) {
        load_w(at + 1, u);
        load_x(at + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
      both_steps(o, us, ub);
    }
  }
  if (p.K % kUnit != 0 && wave == WAVES - 1) {
    // the operands in place: lane (n, g) loads its own
    Scales<S, kUnit / G> us[KT], ub[KT];
    Operands o;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      const int k0 = units * kUnit + st * kStep;
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const uint8_t* row = (of_up(t) ? p.w[1] : p.w[0]) + (row0 + row_of(t, n)) * (p.K / 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = k0 + (kSplit ? 32 * j + 8 * g : 32 * g + 8 * j);
          o.q[st][t][j] = *reinterpret_cast<const uint32_t*>(row + (k < p.K ? k : 0) / 2);
        }
#pragma unroll
        for (int h = 0; h < kPer; ++h) {
          const int k = k0 / G + h < n_scales ? k0 / G + h : n_scales - 1;
          us[t].set(st * kPer + h, s_ptr[t][k]);
          if (BIAS) ub[t].set(st * kPer + h, b_ptr[t][k]);
        }
      }
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const uint16_t* row = p.rows + int64_t(s_rows[16 * i + n < live ? 16 * i + n : 0]) * p.K;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = k0 + (kSplit ? 32 * j + 8 * g : 32 * g + 8 * j);
          o.x[st][i][j] = k < p.K ? *reinterpret_cast<const u32x4*>(row + k) : u32x4{0, 0, 0, 0};
        }
      }
    }
    both_steps(o, us, ub);
  }

  // the parts of K, added in order: lane (n, g) holds rows 4 g .. 4 g + 3 of column
  // n of each 16 x 16 tile; columns are swizzled by the row's g, which keeps the
  // four of them in different banks
  auto swizzled = [](int row, int col) { return row * kPitch + (col ^ (16 * (row / 4 % KT))); };
  float* mine = reinterpret_cast<float*>(s_x[wave]);
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) mine[swizzled(16 * i + 4 * g + v, 16 * t + n)] = acc[i][t][v];
  __syncthreads();
  const int quads = cols / 4;
  for (int at = tid; at < live * quads; at += WAVES * kWave) {
    const int r = at / quads, c = at % quads * 4;
    f32x4 a = {0.f, 0.f, 0.f, 0.f}, u = a;
    for (int k = 0; k < WAVES; ++k) {
      const float* part = reinterpret_cast<const float*>(s_x[k]);
      a += *reinterpret_cast<const f32x4*>(part + swizzled(r, c));
      if (p.glu) u += *reinterpret_cast<const f32x4*>(part + swizzled(r, 8 * KT + c));
    }
    float o[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) o[v] = p.glu ? (p.y_bf16 ? silu(a[v]) : silu_f32(a[v])) * u[v] : a[v];
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

// Many tiles: the waves of a workgroup take 16 KT columns each over the whole K and
// share x, double-buffered in LDS, one barrier a unit.  Codes go to registers two
// units ahead and through the wave's own LDS into the operands' order, as above; x
// one unit ahead, its elements brought into the codes' order on the way.
// Scales are asked for 32 bytes of a row at a time, for up to 8 units: unit by unit
// the same lines came from L2 again each time, as much as the codes themselves (1024
// rows, 256 experts, K 7168, F 2048: 807 us, 713 without these loads).
// K is whole units and a row's scales whole 16 bytes (whole_rows below), so no load in
// the loop has another form for the end of a row: the branch between two forms made
// the compiler wait for every load there.
template <int G, typename S, bool BIAS, int NB, int KT>
__global__ __launch_bounds__(256, 2) void wide_kernel(Product p) {
  constexpr int kWaves = 4, kThreads = kWaves * kWave;
  constexpr int kTM = 16 * NB;
  constexpr bool kSplit = G < kStep;
  constexpr Bias kHow = !BIAS ? Bias::kSym : sizeof(S) == 2 ? Bias::kMfma : Bias::kFma;
  constexpr int kPieces = kUnit / 8;           // 16-byte pieces of a row of x in a unit
  constexpr int kLoads = kTM * kPieces / kThreads;
  __shared__ u32x4 s_x[2][kTM * kPieces];
  __shared__ u32x4 s_codes[kWaves][KT * 2 * kWave];
  constexpr int kRowBytes = 32;                // of a row's scales in a chunk, two lanes a row
  constexpr int kPerChunk = kRowBytes / int(sizeof(S)), kPerUnit = kUnit / G;
  constexpr int kChunkUnits = kPerChunk / kPerUnit;
  static_assert(KT * 16 * kRowBytes == kWave * 16, "16 bytes per lane");
  __shared__ u32x4 s_scales[kWaves][kHow == Bias::kFma ? 2 : 1][kWave];
  // kMfma: X of 16 groups, by row, in three bf16 terms; one block of groups is added
  // while the next one's X are written
  constexpr int kBlockUnits = 16 * G / kUnit;
  __shared__ uint16_t s_sums[kHow == Bias::kMfma ? 2 : 1][3][kHow == Bias::kMfma ? kTM : 1][16];
  __shared__ int s_rows[kTM];

  const int m_idx = blockIdx.x / p.n_groups, grp = blockIdx.x % p.n_groups;
  const int tid = threadIdx.x, lane = lane_id();
  const Tile tile = p.direct ? direct_tile(m_idx, p.index, p.n_rows, p.n_experts, s_rows)
                             : find_tile<kTM>(m_idx, p.index, p.n_experts, p.n_rows);
  if (!tile.valid) return;             // whole workgroup
  // rows of the tile (row_end is the expert's); past them its first is read, and never stored
  const int live = tile.row_end - tile.row0 < kTM ? tile.row_end - tile.row0 : kTM;
  if (!p.direct && tid < live) s_rows[tid] = p.order[tile.row0 + tid];
  if constexpr (kHow == Bias::kMfma) {         // groups past K are multiplied by 0
    uint16_t* sums = &s_sums[0][0][0][0];
    for (int i = tid; i < 2 * 3 * kTM * 16; i += kThreads) sums[i] = 0;
  }
  __syncthreads();

  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int n = lane & 15, g = lane >> 4;
  const int cols = p.glu ? 8 * KT : 16 * KT;   // output columns of the wave
  const int col0 = (grp * kWaves + wave) * cols;
  const int n_scales = p.K / G;
  const int units = p.K / kUnit;

  // weight row of row i of tile t, counted from the expert's first
  auto row_of = [&](int t, int i) {
    const int c = col0 + 16 * (p.glu && t >= KT / 2 ? t - KT / 2 : t) + i;
    return c < p.N ? c : p.N - 1;              // partial last group; never stored
  };
  auto of_up = [&](int t) { return p.glu && t >= KT / 2; };
  const int64_t row0 = int64_t(tile.expert) * p.N;
  const int base = row_of(0, 0);
  // its row of the KT tiles' scales, 16-byte piece lane % 2 of a chunk
  const int64_t s_row = (row0 + row_of(lane / 32, lane / 2 % 16)) * n_scales;
  const S* s_ptr = static_cast<const S*>(of_up(lane / 32) ? p.s[1] : p.s[0]) + s_row;
  const S* b_ptr = kHow == Bias::kFma ? static_cast<const S*>(of_up(lane / 32) ? p.b[1] : p.b[0]) + s_row : nullptr;
  uint32_t w_off[KT][2];                       // from the wave's first row, below 2^28
  const uint8_t* w_base[2] = {p.w[0] + (row0 + base) * (p.K / 2), p.glu ? p.w[1] + (row0 + base) * (p.K / 2) : nullptr};
#pragma unroll
  for (int t = 0; t < KT; ++t) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 8 * h + lane / 8;          // its row of the tile, piece lane % 8 ^ i / 2
      w_off[t][h] = uint32_t(row_of(t, i) - base) * uint32_t(p.K / 2) + 16 * ((lane % 8) ^ (i / 2));
    }
  }
  // row tid / 32 + 8 j of the tile, piece tid % 32
  const uint16_t* x_ptr[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int r = tid / kPieces + 8 * j;
    x_ptr[j] = p.rows + int64_t(s_rows[r < live ? r : 0]) * p.K + 8 * (tid % kPieces);
  }

  f32x4 acc[NB][KT];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int t = 0; t < KT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  using Codes = u32x4[KT][2];                  // rows 8 h + l / 8 of tile t
  using UnitScales = Scales<S, kPerUnit>;
  auto load_x = [&](int unit, u32x4 (&x)[kLoads]) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) x[j] = *reinterpret_cast<const u32x4*>(x_ptr[j] + int64_t(unit) * kUnit);
  };
  auto put_x = [&](int unit, const u32x4 (&x)[kLoads]) {
    const int buf = unit & 1;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int r = tid / kPieces + 8 * j, piece = tid % kPieces;
      s_x[buf][r * kPieces + (piece & 16) + ((piece ^ r) & 15)] = __builtin_bit_cast(u32x4, evens_odds(x[j]));
      if constexpr (kHow == Bias::kMfma) {     // the piece's sum, and its group's, G / 8 lanes side by side
        float sum = piece_sum(x[j]);
        sum += row_step<0xB1>(sum);            // lanes 1 0 3 2
        sum += row_step<0x4E>(sum);            // lanes 2 3 0 1
        if (G >= 64) sum += row_step<0x141>(sum);    // row_half_mirror
        if (G >= 128) sum += row_step<0x140>(sum);   // row_mirror
        if (piece % (G / 8) == 0) {
          const int at = unit % kBlockUnits * (kUnit / G) + piece / (G / 8);
#pragma unroll
          for (int term = 0; term < 3; ++term) {
            const uint32_t v = pack2(sum, 0.f);
            s_sums[unit / kBlockUnits & 1][term][r][at] = uint16_t(v);
            sum -= __uint_as_float(v << 16);
          }
        }
      }
    }
  };
  auto load_w = [&](int unit, Codes& q) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        q[t][h] = *reinterpret_cast<const u32x4*>((of_up(t) ? w_base[1] : w_base[0]) + int64_t(unit) * (kUnit / 2) + w_off[t][h]);
  };
  // this lane's 16 bytes of a chunk; of a last, partial chunk some lie behind the row
  // and are not used: the row's first in their place
  auto load_piece = [&](const S* row, int chunk) {
    const int first = chunk * kPerChunk + 16 / int(sizeof(S)) * (lane % 2);
    return *reinterpret_cast<const u32x4*>(row + (first < n_scales ? first : 0));
  };
  auto load_scales = [&](int chunk, u32x4 (&c)[2]) {
    c[0] = load_piece(s_ptr, chunk);
    if (kHow == Bias::kFma) c[1] = load_piece(b_ptr, chunk);
  };
  // kMfma: the biases of 16 groups, groups 4 g .. 4 g + 3 of row n of each tile, 0 past
  // the row's end; and their products with these groups' X
  uint2 biases[KT];
  const uint16_t* bias_ptr[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t)
    bias_ptr[t] = kHow == Bias::kMfma ? static_cast<const uint16_t*>(of_up(t) ? p.b[1] : p.b[0]) + (row0 + row_of(t, n)) * n_scales : nullptr;
  auto get_biases = [&](int unit) __attribute__((always_inline)) {
    const int first = unit * kPerUnit + 4 * g;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const uint2 v = *reinterpret_cast<const uint2*>(bias_ptr[t] + (first < n_scales ? first : 0));
      biases[t] = first < n_scales ? v : make_uint2(0u, 0u);
    }
  };
  auto use_biases = [&](int unit) __attribute__((always_inline)) {
    typedef short short4v __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        const short4v v = *reinterpret_cast<const short4v*>(&s_sums[unit / kBlockUnits & 1][term][16 * i + n][4 * g]);
#pragma unroll
        for (int t = 0; t < KT; ++t)
          acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(v, __builtin_bit_cast(short4v, biases[t]), acc[i][t], 0, 0, 0);
      }
  };
  auto put_scales = [&](const u32x4 (&c)[2]) {
#pragma unroll
    for (int i = 0; i < (kHow == Bias::kFma ? 2 : 1); ++i) s_scales[wave][i][lane] = c[i];
  };
  auto take_scales = [&](int unit, UnitScales (&us)[KT], UnitScales (&ub)[KT]) {
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int at = (16 * t + n) * kPerChunk + unit % kChunkUnits * kPerUnit;
      us[t].load(reinterpret_cast<const S*>(s_scales[wave][0]) + at);
      if (kHow == Bias::kFma) ub[t].load(reinterpret_cast<const S*>(s_scales[wave][1]) + at);
    }
  };
  u32x4* codes = s_codes[wave];
  auto put_w = [&](const Codes& q) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) codes[(2 * t + h) * kWave + lane] = q[t][h];
  };
  auto step = [&](int buf, const UnitScales (&us)[KT], const UnitScales (&ub)[KT], auto which) __attribute__((always_inline)) {
    constexpr int st = decltype(which)::value;
    // MFMA j takes from lane (n, g) the codes in dword g of piece 4 st + j, or dword j
    // of piece 4 st + g, and the 8 elements of piece 4 j + g of x, or 4 g + j
    bf16x8 b[KT][4];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const u32x4* row = codes + 2 * t * kWave + 8 * n;
      u32x4 v;
      if constexpr (kSplit) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = reinterpret_cast<const uint32_t*>(row + ((4 * st + j) ^ (n / 2)))[g];
      } else {
        v = row[(4 * st + g) ^ (n / 2)];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) b[t][j] = codes8(v[j]);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if (i > 0 && 16 * i >= live) break;      // whole workgroup
      bf16x8 a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a[j] = __builtin_bit_cast(bf16x8, s_x[buf][(16 * i + n) * kPieces + 16 * st + ((kSplit ? 4 * j + g : 4 * g + j) ^ n)]);
      multiply<G, S, kHow, KT, st>(acc[i], a, b, us, ub);
    }
    // the products stay in their step: moved out of it they keep its operands alive
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int t = 0; t < KT; ++t) asm volatile("" : "+v"(acc[i][t])::"memory");
  };
  auto both_steps = [&](int buf, const UnitScales (&us)[KT], const UnitScales (&ub)[KT]) __attribute__((always_inline)) {
    step(buf, us, ub, std::integral_constant<int, 0>());
    step(buf, us, ub, std::integral_constant<int, 1>());
  };

  u32x4 x[kLoads], chunk[2];
  UnitScales us[KT], ub[KT];
  load_scales(0, chunk);
  if (kHow == Bias::kMfma) get_biases(0);
  __builtin_amdgcn_sched_barrier(0);
  Codes q0, q1;
  load_x(0, x);
  load_w(0, q0);
  __builtin_amdgcn_sched_barrier(0);
  load_w(units > 1 ? 1 : 0, q1);
  __builtin_amdgcn_sched_barrier(0);
  put_x(0, x);
  __syncthreads();
  // units past the last one are the last one again, and are not used
  auto turn = [&](int at, int buf, Codes& q) __attribute__((always_inline)) {
    load_x(at + 1 < units ? at + 1 : units - 1, x);
    __builtin_amdgcn_sched_barrier(0);
    if (at % kChunkUnits == 0) {
      put_scales(chunk);
      load_scales(at / kChunkUnits + 1, chunk);
    }
    put_w(q);
    take_scales(at, us, ub);
    __builtin_amdgcn_sched_barrier(0);
    load_w(at + 2 < units ? at + 2 : units - 1, q);
    __builtin_amdgcn_sched_barrier(0);
    both_steps(buf, us, ub);
    if (kHow == Bias::kMfma && (at % kBlockUnits == kBlockUnits - 1 || at + 1 == units)) {
      use_biases(at);
      get_biases(at + 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    // the buffer was last read a unit ago, which every wave has left
    if (at + 1 < units) put_x(at + 1, x);
    __syncthreads();
  };
  int at = 0;
#pragma clang loop unroll(disable)
  for (; at + 1 < units; at += 2) {
    turn(at, 0, q0);
    turn(at + 1, 1, q1);
  }
  if (at < units) turn(at, 0, q0);
  // lane (n, g) holds rows 4 g .. 4 g + 3 of column n of each 16 x 16 tile
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int at = 16 * i + 4 * g + r;
      if (at >= live) continue;
      const int64_t row = int64_t(s_rows[at]) * p.N;
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const int c = col0 + 16 * t + n;
        if (c >= p.N || (p.glu && t >= KT / 2)) continue;
        const float a = acc[i][t][r], up = acc[i][(t + KT / 2) % KT][r];
        const float o = p.glu ? (p.y_bf16 ? silu(a) : silu_f32(a)) * up : a;
        if (p.y_bf16) static_cast<uint16_t*>(p.y)[row + c] = uint16_t(pack2(o, 0.f));
        else static_cast<float*>(p.y)[row + c] = o;
      }
    }
}

// Mean rows per expert from which a tile holds 32 rows, if there are kManyBlocks such
// tiles: 8 and 64 experts, K = N = 4096, with tiles of 16 and of 32 rows
//   16 rows each, at most: 21 and 22 us, 124 and 128 us (of 4: 18 and 35 us)
//   20 rows each:          28 and 27 us, 171 and 152 us (64: 48 and 40, 317 and 273)
// and between, where 10 rows are the mean, some experts have more than 16.  One expert
// of 64, 256 and 512 rows: 11 and 19, 29 and 33 us; K 7168: 75 and 62 us.
constexpr int64_t kNarrowRows = 10;
// Workgroups of 64 columns up to which a workgroup has half of them and splits K over
// 8 waves instead of 4: up to a workgroup per CU.  One row, K 7168, 128 and 144 of
// them: 10.6 and 15.7, 17.4 and 16.0 us; K 2048, 64 and 144: 5.6 and 7.1, 9.6 and 7.4.
constexpr int64_t kFewBlocks = 128;
// Workgroups of 128 columns from which the waves split the columns.  One row per expert,
// splitting columns and splitting K: 256 (16 experts, K 4096, N 2048) 16.8 and 17.6 us,
// 256 (8, K 7168, N 4096) 26.1 and 24.8, 448 (8, K 2048, N 7168) 14.6 and 18.5, 1024
// (64, K 4096, N 2048) 49.5 and 55.3 us.
constexpr int64_t kManyBlocks = 300;
constexpr int kWideT = 2;

enum class Form { kDeep, kSplitK, kWide };
struct Shape {
  bool direct;
  Form form;
  int nb, col_groups;
  int64_t blocks;
};
Shape shape_of(const Int4Product& g) {
  Shape s{};
  const auto groups = [&](int kt, int waves) { return (g.n_dim + (g.w_up ? 8 : 16) * kt * waves - 1) / ((g.w_up ? 8 : 16) * kt * waves); };
  s.nb = g.n_rows < kNarrowRows * g.n_experts ||
         most_tiles(g.n_rows, g.n_experts, 32) * groups(kWideT, 4) < kManyBlocks ? 1 : 2;
  s.direct = s.nb == 1 && g.n_rows <= kDirectRows;
  const int64_t tiles = most_tiles(g.n_rows, g.n_experts, 16 * s.nb);
  const bool whole_rows = g.k_dim % kUnit == 0 && g.k_dim / g.group * (g.scales_bf16 ? 2 : 4) % 16 == 0 &&
                          !((reinterpret_cast<uintptr_t>(g.w_scales) | reinterpret_cast<uintptr_t>(g.w_biases) |
                             reinterpret_cast<uintptr_t>(g.w_up_scales) | reinterpret_cast<uintptr_t>(g.w_up_biases)) & 15);
  s.form = whole_rows && tiles * groups(kWideT, 4) >= kManyBlocks ? Form::kWide
           : s.nb == 1 && tiles * groups(4, 1) <= kFewBlocks ? Form::kDeep : Form::kSplitK;
  s.col_groups = int(s.form == Form::kWide ? groups(kWideT, 4) : groups(s.form == Form::kDeep ? 2 : 4, 1));
  s.blocks = tiles * s.col_groups;
  return s;
}

template <int G>
void launch_group(const Product& p, const Shape& s, bool scales_bf16, hipStream_t stream) {
  const auto form = [&](auto* type, auto bias) {
    using S = std::remove_pointer_t<decltype(type)>;
    constexpr bool B = decltype(bias)::value;
    const unsigned blocks = unsigned(s.blocks);
    if (s.form == Form::kDeep) stream_kernel<G, S, B, 1, 2, 8><<<blocks, 8 * kWave, 0, stream>>>(p);
    else if (s.form == Form::kSplitK && s.nb == 1) stream_kernel<G, S, B, 1, 4, 4><<<blocks, 4 * kWave, 0, stream>>>(p);
    else if (s.form == Form::kSplitK) stream_kernel<G, S, B, 2, 4, 4><<<blocks, 4 * kWave, 0, stream>>>(p);
    else if (s.nb == 1) wide_kernel<G, S, B, 1, kWideT><<<blocks, 4 * kWave, 0, stream>>>(p);
    else wide_kernel<G, S, B, 2, kWideT><<<blocks, 4 * kWave, 0, stream>>>(p);
  };
  const auto type = [&](auto* t) {
    if (p.b[0]) form(t, std::true_type());
    else form(t, std::false_type());
  };
  if (scales_bf16) type(static_cast<uint16_t*>(nullptr));
  else type(static_cast<float*>(nullptr));
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
