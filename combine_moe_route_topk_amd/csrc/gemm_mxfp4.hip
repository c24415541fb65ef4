// MXFP4 expert products: y[p] = W[e] x[p] for every row p of expert e, rows
// and weights as E2M1 codes (two per byte) with one E8M0 scale per 32 elements
// of K, or, with an up projection, y[p] = silu(W[e] x[p]) * (W_up[e] x[p]).
//   y[p, n] = bf16( sum_b 2^(sx[p,b] + sw[e,n,b] - 254) sum_{k in block b} q(x[p,k]) q(w[e,n,k]) )
//
// The matrix cores take the format as it is: v_mfma_scale_f32_32x32x64_f8f6f4
// reads 32 codes (16 bytes) and their scale byte per lane and operand, lane l
// holding row l % 32 and the block of 32 that l / 32 names.
#include "device_common.hpp"
#include "launch.hpp"

namespace moe {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kTM = 32;           // rows per tile
constexpr int kTN = 128;          // columns per workgroup: 32 per wave
constexpr int kXcds = 8;

struct Tile {
  int expert;
  int row0, row_end;
  bool valid;
};

// m-tile index -> expert and row range.  Lane j of each 64-expert chunk counts
// the tiles of expert c + j; a wave prefix sum finds the owner.  Row ranges are
// clamped into [0, n_rows], so no row outside the buffer is read whatever the
// offsets hold.
template <int TM>
__device__ Tile find_tile(int m_idx, const int32_t* __restrict__ offs, int n_experts, int n_rows) {
  Tile t{};
  const int lane = lane_id();
  int base = 0;
  for (int c = 0; c < n_experts; c += kWave) {
    const int e = c + lane;
    int lo = 0, hi = 0, nt = 0;
    if (e < n_experts) {
      const int a = offs[e], b = offs[e + 1];
      lo = a < 0 ? 0 : (a > n_rows ? n_rows : a);
      hi = b < lo ? lo : (b > n_rows ? n_rows : b);
      nt = (hi - lo) / TM + ((hi - lo) % TM != 0);
    }
    const int incl = wave_inclusive_scan(nt);
    const int excl = incl - nt;
    const uint64_t own = ballot(nt > 0 && m_idx >= base + excl && m_idx < base + incl);
    if (own) {
      const int src = __ffsll((unsigned long long)own) - 1;
      t.expert = __builtin_amdgcn_readfirstlane(c + src);
      t.row0 = lane_value(lo, src) + (m_idx - base - lane_value(excl, src)) * TM;
      t.row_end = lane_value(hi, src);
      t.valid = true;
      return t;
    }
    base += lane_value(incl, kWave - 1);
  }
  return t;
}

__device__ __forceinline__ i32x8 codes16(const uint8_t* p) {
  const i32x4 q = *reinterpret_cast<const i32x4*>(p);
  return i32x8{q.x, q.y, q.z, q.w, 0, 0, 0, 0};
}

__device__ __forceinline__ f32x16 mfma4(i32x8 a, i32x8 b, f32x16 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, 0, sa, 0, sb);
}

__device__ __forceinline__ float silu(float a) { return a / (1.f + expf(-a)); }

// order: row p of the grouped order is row order[p] of rows and of y (null: p itself)
template <bool GLU>
__global__ __launch_bounds__(kThreads) void gemm_mxfp4_kernel(
    const uint8_t* __restrict__ rows, const uint8_t* __restrict__ row_scales, int n_rows, int K,
    const int32_t* __restrict__ offs, int n_experts, const int32_t* __restrict__ order,
    const uint8_t* __restrict__ w, const uint8_t* __restrict__ w_scales,
    const uint8_t* __restrict__ w_up, const uint8_t* __restrict__ w_up_scales, int N,
    uint16_t* __restrict__ y, int n_tiles) {
  const int b = blockIdx.x;
  const int slot = b / kXcds;
  const int m_idx = (slot / n_tiles) * kXcds + b % kXcds, n_tile = slot % n_tiles;
  const Tile t = find_tile<kTM>(m_idx, offs, n_experts, n_rows);
  if (!t.valid) return;
  const int lane = lane_id(), r = lane & 31, half = lane >> 5;
  const int64_t col0 = int64_t(n_tile) * kTN + __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave) * 32;
  int p = t.row0 + r < t.row_end ? t.row0 + r : t.row_end - 1;    // clamped rows are never stored
  if (order) p = order[p];
  const int64_t n = col0 + r < N ? col0 + r : N - 1;
  const int64_t wr = int64_t(t.expert) * N + n;
  const int kb = K / 32;
  f32x16 acc = {}, up = {};
  for (int i = half; i < kb; i += 2) {                            // K is a multiple of 64
    const i32x8 a = codes16(rows + int64_t(p) * (K / 2) + i * 16);
    const int sa = row_scales[int64_t(p) * kb + i];
    acc = mfma4(a, codes16(w + wr * (K / 2) + i * 16), acc, sa, w_scales[wr * kb + i]);
    if (GLU) up = mfma4(a, codes16(w_up + wr * (K / 2) + i * 16), up, sa, w_up_scales[wr * kb + i]);
  }
  // lane holds C[8*(v/4) + 4*half + v%4][lane % 32]
  if (col0 + r >= N) return;
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    int g = t.row0 + 8 * (v >> 2) + 4 * half + (v & 3);
    if (g >= t.row_end) continue;
    if (order) g = order[g];
    const float o = GLU ? silu(acc[v]) * up[v] : acc[v];
    y[int64_t(g) * N + col0 + r] = f32_to_bf16_rne(o);
  }
}

// Workspace of the gather form: the maps of a sorted dispatch of the ids.
struct GatherLayout {
  size_t counts, offsets, seg_offsets, dst_pos, order, dispatch_ws, total;
};
size_t round256(size_t v) { return (v + 255) / 256 * 256; }
GatherLayout gather_layout(int64_t n_rows, int n_experts) {
  GatherLayout L{};
  size_t o = 0;
  L.counts = o;      o += round256(size_t(n_experts) * 4);
  L.offsets = o;     o += round256(size_t(n_experts + 1) * 4);
  L.seg_offsets = o; o += round256(2 * 4);
  L.dst_pos = o;     o += round256(size_t(n_rows) * 4);
  L.order = o;       o += round256(size_t(n_rows) * 4);
  L.dispatch_ws = o; o += round256(dispatch_workspace_bytes(n_rows, n_experts, 1, 1));
  L.total = o;
  return L;
}

hipError_t launch_product(const Mxfp4Product& g, const int32_t* offs, const int32_t* order,
                          hipStream_t stream) {
  const int n_tiles = int((g.n_dim + kTN - 1) / kTN);
  const int64_t m = (g.n_rows + kTM - 1) / kTM + g.n_experts;
  const unsigned grid = unsigned((m + kXcds - 1) / kXcds * kXcds * n_tiles);
  const uint8_t *x = static_cast<const uint8_t*>(g.rows), *w = static_cast<const uint8_t*>(g.w),
                *u = static_cast<const uint8_t*>(g.w_up);
  uint16_t* y = static_cast<uint16_t*>(g.y);
  if (u)
    gemm_mxfp4_kernel<true><<<grid, kThreads, 0, stream>>>(x, g.row_scales, int(g.n_rows), int(g.k_dim), offs, g.n_experts, order, w, g.w_scales, u, g.w_up_scales, int(g.n_dim), y, n_tiles);
  else
    gemm_mxfp4_kernel<false><<<grid, kThreads, 0, stream>>>(x, g.row_scales, int(g.n_rows), int(g.k_dim), offs, g.n_experts, order, w, g.w_scales, u, g.w_up_scales, int(g.n_dim), y, n_tiles);
  return hipGetLastError();
}

}  // namespace

int64_t gemm_mxfp4_tiles(int64_t n_rows, int n_experts, int64_t n_dim) {
  return ((n_rows + kTM - 1) / kTM + n_experts + kXcds) * ((n_dim + kTN - 1) / kTN);
}

size_t gather_gemm_mxfp4_workspace_bytes(int64_t n_rows, int n_experts) {
  return gather_layout(n_rows, n_experts).total;
}

hipError_t launch_grouped_gemm_mxfp4(const Mxfp4Product& g, const int32_t* expert_offsets,
                                     hipStream_t stream) {
  return launch_product(g, expert_offsets, nullptr, stream);
}

hipError_t launch_gather_gemm_mxfp4(const Mxfp4Product& g, const int32_t* row_expert,
                                    void* workspace, hipStream_t stream) {
  const GatherLayout L = gather_layout(g.n_rows, g.n_experts);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  DispatchArgs d{};
  d.n_tokens = g.n_rows;
  d.topk_idx = row_expert;
  d.n_experts = g.n_experts;
  d.k = 1;
  d.n_segments = 1;
  d.sorted = 1;
  d.expert_counts = reinterpret_cast<int32_t*>(ws + L.counts);
  d.expert_offsets = reinterpret_cast<int32_t*>(ws + L.offsets);
  d.segment_offsets = reinterpret_cast<int32_t*>(ws + L.seg_offsets);
  d.dst_pos = reinterpret_cast<int32_t*>(ws + L.dst_pos);
  d.src_pair = reinterpret_cast<int32_t*>(ws + L.order);
  d.workspace = ws + L.dispatch_ws;
  const hipError_t err = launch_dispatch(d, stream);
  if (err != hipSuccess) return err;
  return launch_product(g, d.expert_offsets, d.src_pair, stream);
}

}  // namespace moe
