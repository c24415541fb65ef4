// What the expert products share: rows grouped by expert, tiles of them, and how
// outputs are activated and stored.
#pragma once

#include "device_common.hpp"
#include "launch.hpp"

namespace moe {
namespace {

constexpr int kXcds = 8;

struct Tile {
  int expert;
  int row0, row_end;
  bool valid;
};

// Row ranges of experts 4 l .. 4 l + 3 past e0 in lane l, clamped into
// [0, n_rows], so no row outside the buffer is read whatever the offsets hold,
// and the tiles they take.
template <int TM>
struct Experts {
  static constexpr int kPer = 4;
  int lo[kPer], hi[kPer], nt[kPer], sum;
  __device__ Experts(int e0, const int32_t* __restrict__ offs, int n_experts, int n_rows) {
    int at[kPer + 1];
#pragma unroll
    for (int i = 0; i <= kPer; ++i) {
      const int e = e0 + kPer * lane_id() + i;
      at[i] = offs[e < n_experts ? e : n_experts];             // past the last: no rows
    }
    sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int a = at[i], b = at[i + 1];
      lo[i] = a < 0 ? 0 : (a > n_rows ? n_rows : a);
      hi[i] = b < lo[i] ? lo[i] : (b > n_rows ? n_rows : b);
      nt[i] = (hi[i] - lo[i]) / TM + ((hi[i] - lo[i]) % TM != 0);
      sum += nt[i];
    }
  }
};

// m-tile index -> expert and row range: a wave prefix sum over each 256 experts
// finds the lane, and the lane the expert.
template <int TM>
__device__ Tile find_tile(int m_idx, const int32_t* __restrict__ offs, int n_experts, int n_rows) {
  Tile t{};
  using X = Experts<TM>;
  int base = 0;
  for (int c = 0; c < n_experts; c += X::kPer * kWave) {
    const X x(c, offs, n_experts, n_rows);
    const int incl = wave_inclusive_scan(x.sum);
    int at = m_idx - (base + incl - x.sum);                    // tile number within the lane's four
    const uint64_t own = ballot(at >= 0 && at < x.sum);
    if (own) {
      const int src = __ffsll((unsigned long long)own) - 1;
      int i = 0, lo = x.lo[0], hi = x.hi[0];
#pragma unroll
      for (int j = 0; j + 1 < X::kPer; ++j)
        if (i == j && at >= x.nt[j]) { at -= x.nt[j]; i = j + 1; lo = x.lo[j + 1]; hi = x.hi[j + 1]; }
      t.expert = __builtin_amdgcn_readfirstlane(c + X::kPer * src + lane_value(i, src));
      t.row0 = lane_value(lo, src) + lane_value(at, src) * TM;
      t.row_end = lane_value(hi, src);
      t.valid = true;
      return t;
    }
    base += lane_value(incl, kWave - 1);
  }
  return t;
}

// silu(a) = a / (1 + e^-a) from the exponential and reciprocal instructions (1
// ulp each), beside the 2^-8 of the bf16 rounding that follows.  The exponent is
// rounded once, which a negative gate carries into the result: within 2^-21 +
// |a| 2^-23.6, 2^-17 at a = -87.  Below -87.3 the reciprocal would be subnormal,
// and the result is 0 in place of a e^a, under 2^-119; -inf gives NaN, as
// a / (1 + e^-a) does.  Measured, 16384 rows over 8 experts, K 4096, F 14336: 1064
// us; 1088 with a scaled denominator that keeps those values, 1180 with expf and
// the division.
__device__ __forceinline__ float silu(float a) {
  return a * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(a * -1.44269504f));
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {   // rounds to nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// Columns c .. c + 3 of a row of n (c a multiple of 4): 8 bytes where rows are
// multiples of 8 bytes, else element by element.
__device__ __forceinline__ void store4(uint16_t* row, int c, int n, bool whole, const float (&o)[4]) {
  const uint32_t lo = pack2(o[0], o[1]), hi = pack2(o[2], o[3]);
  if (whole) {
    if (c < n) *reinterpret_cast<uint2*>(row + c) = make_uint2(lo, hi);
  } else {
    if (c < n) row[c] = uint16_t(lo);
    if (c + 1 < n) row[c + 1] = uint16_t(lo >> 16);
    if (c + 2 < n) row[c + 2] = uint16_t(hi);
    if (c + 3 < n) row[c + 3] = uint16_t(hi >> 16);
  }
}

// Up to 64 rows in any order: tile m of 16 rows of one expert, found in every
// wave without a grouping pass before the product.  Lane q holds row q's
// expert; the lanes with the same one come from a ballot per bit of the ids, a
// tile begins at every 16th of them, and tiles are numbered by where they
// begin.  Row i of the tile goes to s_rows[i], the tile's row_end is their
// number.  Every lane calls it.
__device__ __forceinline__ Tile direct_tile(int m, const int32_t* __restrict__ row_expert, int n_rows,
                                            int n_experts, int* s_rows) {
  const int lane = lane_id();
  const int mine = lane < n_rows ? row_expert[lane] : -1;
  const bool ok = unsigned(mine) < unsigned(n_experts);        // ids below 2^10
  uint64_t same = ballot(ok);
#pragma unroll
  for (int bit = 1; bit < kMaxExperts; bit <<= 1) {
    const uint64_t on = ballot(mine & bit);
    same &= mine & bit ? on : ~on;
  }
  const int rank = __popcll(same & lanemask_lt());
  const uint64_t begins = ballot(ok && rank % 16 == 0);
  Tile t{};
  const uint64_t at = ballot(((begins >> lane) & 1) && __popcll(begins & lanemask_lt()) == m);
  if (!at) return t;                                           // fewer tiles
  const int q = __ffsll((unsigned long long)at) - 1;
  t.expert = lane_value(mine, q);
  const int i = rank - lane_value(rank, q);
  const bool in = ok && mine == t.expert && unsigned(i) < 16u;
  if (in) s_rows[i] = lane;
  t.row_end = __popcll(ballot(in));
  t.valid = true;
  return t;
}

// Workspace of the gather form: the maps of a sorted dispatch of the ids.  It grows
// with rows and experts, so that one made for the most rows holds every smaller call.
struct GatherLayout {
  size_t counts, offsets, seg_offsets, dst_pos, order, dispatch_ws, total;
};
// The most that the dispatch of up to n_pairs pairs takes: fewer can take more chunks,
// since a chunk's length jumps.  At most 64 of 256 pairs or more up to 65536 pairs, then
// 1024 pairs each up to 2^20, then at most 1024 chunks.
size_t most_dispatch_workspace(int64_t n_pairs, int n_experts) {
  const int64_t even = (n_pairs + 255) / 256 < 64 ? (n_pairs + 255) / 256 : 64;
  const int64_t longer = (n_pairs + 1023) / 1024 < 1024 ? (n_pairs + 1023) / 1024 : 1024;
  const int64_t chunks = even > longer ? even : longer;
  const size_t most = size_t(chunks) * size_t(n_experts) * 4 + 256;
  const size_t own = dispatch_workspace_bytes(n_pairs, n_experts, 1, 1);
  return most > own ? most : own;
}
size_t round256(size_t v) { return (v + 255) / 256 * 256; }
GatherLayout gather_layout(int64_t n_rows, int n_experts) {
  GatherLayout L{};
  size_t o = 0;
  L.counts = o;      o += round256(size_t(n_experts) * 4);
  L.offsets = o;     o += round256(size_t(n_experts + 1) * 4);
  L.seg_offsets = o; o += round256(2 * 4);
  L.dst_pos = o;     o += round256(size_t(n_rows) * 4);
  L.order = o;       o += round256(size_t(n_rows) * 4);
  L.dispatch_ws = o; o += round256(most_dispatch_workspace(n_rows, n_experts));
  L.total = o;
  return L;
}

// The maps of rows in any order, made by a sorted dispatch of their experts'
// ids: *offsets the experts' offsets, *order the row of each grouped position.
hipError_t launch_grouping(const int32_t* row_expert, int64_t n_rows, int n_experts, void* workspace,
                           const int32_t** offsets, const int32_t** order, hipStream_t stream) {
  const GatherLayout L = gather_layout(n_rows, n_experts);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  DispatchArgs d{};
  d.n_tokens = n_rows;
  d.topk_idx = row_expert;
  d.n_experts = n_experts;
  d.k = 1;
  d.n_segments = 1;
  d.sorted = 1;
  d.expert_counts = reinterpret_cast<int32_t*>(ws + L.counts);
  d.expert_offsets = reinterpret_cast<int32_t*>(ws + L.offsets);
  d.segment_offsets = reinterpret_cast<int32_t*>(ws + L.seg_offsets);
  d.dst_pos = reinterpret_cast<int32_t*>(ws + L.dst_pos);
  d.src_pair = reinterpret_cast<int32_t*>(ws + L.order);
  d.workspace = ws + L.dispatch_ws;
  *offsets = d.expert_offsets;
  *order = d.src_pair;
  return launch_dispatch(d, stream);
}

// Row tiles at most: every expert can end in a partial one, and each holds a row.
int64_t most_tiles(int64_t n_rows, int n_experts, int tm) {
  const int64_t m = (n_rows + tm - 1) / tm + n_experts;
  return m < n_rows ? m : n_rows;
}

// Rows up to which the gather form groups them inside the product's launch.
constexpr int kDirectRows = 64;

}  // namespace
}  // namespace moe
