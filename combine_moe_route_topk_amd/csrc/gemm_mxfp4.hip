// MXFP4 expert products: y[p] = W[e] x[p] for every row p of expert e, rows
// and weights as E2M1 codes (two per byte) with one E8M0 scale per 32 elements
// of K, or, with an up projection, y[p] = silu(W[e] x[p]) * (W_up[e] x[p]).
//   y[p, n] = bf16( sum_b 2^(sx[p,b] + sw[e,n,b] - 254) sum_{k in block b} q(x[p,k]) q(w[e,n,k]) )
//
// The matrix cores take the format as it is: v_mfma_scale_f32_32x32x64_f8f6f4
// reads 32 codes (16 bytes) and their scale byte per lane and operand, lane l
// holding row l % 32 and the block of 32 that l / 32 names.
#include <type_traits>

#include "device_common.hpp"
#include "expert_tiles.hpp"
#include "launch.hpp"
#include "mxfp4_tiles.hpp"

namespace moe {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------- few rows per expert
// The weights are most of the bytes: each is read once per tile of 16 NB rows,
// straight from memory into registers, 1024 elements of K of every weight row
// in flight.  A workgroup of 4 waves takes one tile; a wave owns 32 weight rows
// (SwiGLU: 16 of w and the same 16 of w_up, so silu(g) * u is lane-local) over
// the whole K, as the A operand of v_mfma_scale_f32_16x16x128: lane (n, g) =
// (l % 16, l / 16) holds row n and block 4 s + g of step s, so one load
// instruction reads 64 consecutive bytes of 16 weight rows.  The tile's rows
// are the B operand, staged through LDS 1024 elements at a time,
// double-buffered, one barrier a stage, which leaves the memory queues to the
// weights.  A lane ends with 4 consecutive columns of one row: 8-byte stores.
namespace stream {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4a __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kWT = 2;                   // 16-row weight tiles per wave
constexpr int kCh = 4;                   // K steps of 128 per refill
constexpr int kSt = 8;                   // K steps per LDS stage (1024 elements), all in flight
constexpr int kPitch = kSt * 64 + 16;    // code bytes of a staged row: rows land 4 banks apart
constexpr int kScPitch = kSt * 4 + 16;   // scale bytes of a staged row

// order: row p of the grouped order is row order[p] of rows and of y (null: p
// itself).  DIRECT (up to 64 rows, NB 1): offs holds the expert of each row.
// X4: K is a multiple of 512, so a row's scales are read four steps at a time.
// The loop over K has no other branches: past K the last step is read again
// and multiplied by zero codes (loads under a branch made the compiler move
// the products away from them and keep copies of what they multiply).
template <bool GLU, int NB, int WAVES, bool X4, bool DIRECT>
__global__ __launch_bounds__(WAVES * kWave) void stream_kernel(
    const uint8_t* __restrict__ rows, const uint8_t* __restrict__ row_scales, int n_rows, int K,
    const int32_t* __restrict__ offs, int n_experts, const int32_t* __restrict__ order,
    const uint8_t* __restrict__ w, const uint8_t* __restrict__ w_scales,
    const uint8_t* __restrict__ w_up, const uint8_t* __restrict__ w_up_scales, int N,
    uint16_t* __restrict__ y, int n_groups) {
  constexpr int kTM = 16 * NB;
  constexpr int kThreads = WAVES * kWave;
  constexpr int kPieces = kTM * kSt * 4 / kThreads;            // 16-byte staging loads per thread
  constexpr int kScPieces = (kTM * kSt + kThreads - 1) / kThreads;   // and scale dwords
  static_assert(kPieces * kThreads == kTM * kSt * 4, "whole staging loads");
  __shared__ __align__(16) unsigned char s_q[2][kTM * kPitch];
  __shared__ __align__(16) unsigned char s_sc[2][kTM * kScPitch];

  // workgroup b runs on XCD b % 8; XCD x takes row tiles x, x + 8, ..., all
  // column groups of one back to back (its rows stay in that XCD's L2); the
  // unused tail of the worst-case grid is spread evenly.  (Row tiles of one
  // expert on one XCD, side by side, measured 0-16% slower: the last-level cache
  // already serves their second reading of its weights.)
  const int b = blockIdx.x;
  const int slot = b / kXcds;
  const int m_idx = (slot / n_groups) * kXcds + b % kXcds, grp = slot % n_groups;
  const int tid = threadIdx.x, lane = lane_id();
  __shared__ int s_rows[DIRECT ? kTM : 1];
  Tile tile{};
  if constexpr (DIRECT) {
    static_assert(kTM == 16 && kMaxExperts <= 1024, "tiles of 16 rows, ids of 10 bits");
    tile = direct_tile(m_idx, offs, n_rows, n_experts, s_rows);
  } else {
    tile = find_tile<kTM>(m_idx, offs, n_experts, n_rows);
  }
  if (!tile.valid) return;                                     // whole workgroup
  if (DIRECT) __syncthreads();
  // row i of the tile in rows and y; past the last one its first
  auto row_at = [&](int i) {
    const int p = tile.row0 + (tile.row0 + i < tile.row_end ? i : 0);
    return DIRECT ? s_rows[p] : (order ? order[p] : p);
  };

  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int n = lane & 15, g = lane >> 4;
  constexpr int kCols = GLU ? 16 : 16 * kWT;                   // output columns per wave
  const int col0 = (grp * WAVES + wave) * kCols;
  const int n_steps = K / 128, kb = K / 32;

  // staging: piece tid + threads * j is row p / 32 and 16-byte column p % 32 of
  // the stage; rows past the end of the tile repeat its first (never stored)
  const uint8_t* a_src[kPieces];
  int a_lds[kPieces];
  const int a_step = tid % (kSt * 4) / 4;
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int p = tid + kThreads * j;
    const int row = p / (kSt * 4);
    a_src[j] = rows + int64_t(row_at(row)) * (K / 2) + 16 * (tid % 4);
    a_lds[j] = row * kPitch + (p % (kSt * 4)) * 16;
  }
  const uint8_t* sc_src[kScPieces];
  int sc_lds[kScPieces];
  const int sc_step = tid % kSt;
#pragma unroll
  for (int j = 0; j < kScPieces; ++j) {
    const int row = (tid + kThreads * j) / kSt % kTM;          // the spare threads repeat rows
    sc_src[j] = row_scales + int64_t(row_at(row)) * kb;
    sc_lds[j] = row * kScPitch + 4 * sc_step;
  }

  const uint8_t *w_ptr[kWT], *ws_ptr[kWT];
#pragma unroll
  for (int t = 0; t < kWT; ++t) {
    int c = GLU ? col0 + n : col0 + 16 * t + n;
    if (c >= N) c = N - 1;                                     // partial last group; never stored
    const int64_t wr = int64_t(tile.expert) * N + c;
    w_ptr[t] = (GLU && t ? w_up : w) + wr * (K / 2) + 16 * g;
    ws_ptr[t] = (GLU && t ? w_up_scales : w_scales) + wr * kb;
  }

  f32x4 acc[kWT][NB];
#pragma unroll
  for (int t = 0; t < kWT; ++t)
#pragma unroll
    for (int i = 0; i < NB; ++i) acc[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  // step k of a stage lives in q[.][k], refilled for the next stage four steps
  // at a time: whole lines of a weight row are asked for together (refilled
  // step by step, as soon as each is multiplied, was 13-22% slower)
  i32x4 q[kWT][kSt];
  int sc[kWT][kSt];
  auto clamp = [&](int step) { return step < n_steps ? step : n_steps - 1; };
  auto refill = [&](int k, int step) {     // q[.][k .. k + 3] from `step`
#pragma unroll
    for (int t = 0; t < kWT; ++t) {
      if (X4) {
        const u32x4a v = *reinterpret_cast<const u32x4a*>(ws_ptr[t] + 4 * (clamp(step) / kCh * kCh));
#pragma unroll
        for (int i = 0; i < kCh; ++i) sc[t][k + i] = v[i];
      }
#pragma unroll
      for (int i = 0; i < kCh; ++i) {
        q[t][k + i] = *reinterpret_cast<const i32x4*>(w_ptr[t] + 64 * clamp(step + i));
        if (!X4) sc[t][k + i] = *reinterpret_cast<const int*>(ws_ptr[t] + 4 * clamp(step + i));
      }
    }
  };
#pragma unroll
  for (int k = 0; k < kSt; k += kCh) refill(k, k);

  i32x4 stg[kPieces];
  int stg_sc[kScPieces];
  auto fetch = [&](int step) {                                 // the stage that begins at `step`
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int s = a_step + step;
      stg[j] = *reinterpret_cast<const i32x4*>(a_src[j] + 64 * clamp(s));
      stg[j] = s < n_steps ? stg[j] : i32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int j = 0; j < kScPieces; ++j)
      stg_sc[j] = *reinterpret_cast<const int*>(sc_src[j] + 4 * clamp(sc_step + step));
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) *reinterpret_cast<i32x4*>(&s_q[buf][a_lds[j]]) = stg[j];
#pragma unroll
    for (int j = 0; j < kScPieces; ++j) *reinterpret_cast<int*>(&s_sc[buf][sc_lds[j]]) = stg_sc[j];
  };
  fetch(0);
  put(0);
  __syncthreads();

  // the stage that begins at step st; MORE: there is another one
  auto stage = [&](int st, auto more) {
    constexpr bool MORE = decltype(more)::value;
    const int buf = (st / kSt) & 1;
    if constexpr (MORE) fetch(st + kSt);
    const unsigned char* bq_base = s_q[buf] + n * kPitch + 16 * g;
    const unsigned char* bs_base = s_sc[buf] + n * kScPitch + g;
#pragma unroll
    for (int k = 0; k < kSt; ++k) {
      i32x8 bq[NB];
      int bs[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const i32x4 v = *reinterpret_cast<const i32x4*>(bq_base + i * 16 * kPitch + 64 * k);
        bq[i] = i32x8{v.x, v.y, v.z, v.w, 0, 0, 0, 0};
        bs[i] = bs_base[i * 16 * kScPitch + 4 * k];
      }
#pragma unroll
      for (int t = 0; t < kWT; ++t) {
        i32x4 v = q[t][k];
        asm volatile("" : "+v"(v));        // keeps the loop's copies four registers wide
        const i32x8 a = {v.x, v.y, v.z, v.w, 0, 0, 0, 0};
        const int as = int(uint32_t(sc[t][k]) >> (8 * g));
#pragma unroll
        for (int i = 0; i < NB; ++i)
          acc[t][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, bq[i], acc[t][i], 4, 4, 0, as, 0, bs[i]);
      }
      if (MORE && k % kCh == kCh - 1) {
        __builtin_amdgcn_sched_barrier(0); // the refills stay where they are
        refill(k + 1 - kCh, st + kSt + k + 1 - kCh);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (MORE) {
      // the other buffer was last read in the stage before, which every wave has left
      put(buf ^ 1);
      __syncthreads();
    }
  };
  int st = 0;
  for (; st + kSt < n_steps; st += kSt) stage(st, std::true_type());
  stage(st, std::false_type());
  // the products end here, with every lane on: moved into the divergent stores
  // below, the shifts of their scales would skip the lanes that store nothing
#pragma unroll
  for (int t = 0; t < kWT; ++t)
#pragma unroll
    for (int i = 0; i < NB; ++i) asm volatile("" : "+v"(acc[t][i]));
  if (col0 >= N) return;

  // lane holds columns 4 g .. 4 g + 3 of row n of each 16 x 16 tile
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    if (tile.row0 + 16 * i + n >= tile.row_end) continue;
    uint16_t* out = y + int64_t(row_at(16 * i + n)) * N;
#pragma unroll
    for (int t = 0; t < (GLU ? 1 : kWT); ++t) {
      const int c = col0 + 16 * t + 4 * g;
      float o[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) o[v] = GLU ? silu(acc[0][i][v]) * acc[1][i][v] : acc[t][i][v];
      store4(out, c, N, N % 4 == 0, o);
    }
  }
}

}  // namespace stream

// ---------------------------------------------------------------- many rows per expert
// 256 x 256 tiles (SwiGLU: 128 columns of w and the same 128 of w_up), one
// workgroup of 4 waves (2 x 2) per CU, a wave owning 128 x 128 as 4 x 4 MFMA
// tiles whose 256 accumulators stay in registers: each operand byte read from
// LDS feeds four MFMAs, half the LDS rate.  A tile that holds at most 192 or 128
// rows (an expert's last) loads and multiplies only those: 3 or 2 row tiles a
// wave (256 experts, K 7168, N 4096: 64 rows each 1012 -> 897 us; SwiGLU of N
// 2048, 128 rows each 1087 -> 990).  Where the tiles are no more than half the
// CUs, they have half the columns (8 experts of 64 rows, K = N = 4096: 22.0 ->
// 17.2 us; 128 rows 27.1 -> 21.4; past half, 192 tiles, 37 -> 44, so not there).
//   * K advances in stages of 256, so a stage row is 128 bytes of codes, one
//     line.  Direct global->LDS loads fill two 64 KB slots: stage d is
//     multiplied from slot d % 2 while stage d + 1 lands in the other; the one
//     barrier per stage publishes stage d + 1 and frees slot d % 2.
//   * Lane half h multiplies 16-byte chunks 4h..4h+3 of its row, one per MFMA
//     slice, so its four blocks of 32 have consecutive scale bytes: one dword
//     per row and stage, the slice number picking the byte.
//   * Scales skip LDS: 32 bytes of a row's scales cover four stages; lane half
//     h loads 16 of them, and two swaps between the halves leave one register
//     per stage in each lane.
//   * Past K the scale bytes are 0 on both sides: whatever codes are there add
//     36 * 2^-254, less than the smallest fp32.
// LDS rows are XOR-swizzled in 16-byte chunks by (row >> 1) & 7: the rows that
// a 16-lane phase of a ds_read_b128 reads fall in distinct bank groups.
namespace big {

constexpr int kThreads = 256;
constexpr int kRowBytes = 128;                 // 256 codes
constexpr int kTileBytes = kBM * kRowBytes;    // 32 KB per operand and stage
constexpr int kSlotBytes = 2 * kTileBytes;
constexpr int kLd = kTileBytes / (kThreads * 16);   // direct loads per lane, operand and stage at most (8)
// A wave has MT x NT MFMA tiles of 32 x 32: MT 4, 3 or 2; NT 4, or 2 where tiles
// are few.
constexpr int kT = 4;
constexpr int kGroupM = 8;                     // row tiles per group of the tile order

typedef __attribute__((address_space(3))) void* lds_ptr;
typedef unsigned int u32x4a __attribute__((ext_vector_type(4), aligned(4)));

// at most n vector-memory operations outstanding, LDS operations all returned
constexpr unsigned wait_vm_lgkm0(int n) {
  return unsigned(n & 15) | (unsigned((n >> 4) & 3) << 14) | (0x7u << 4);
}
constexpr unsigned wait_vm(int n) { return wait_vm_lgkm0(n) | (0xFu << 8); }

// Sources of this lane's direct loads.  Run r = 4 i + wave of an operand tile
// is its rows 8 r .. 8 r + 7; lane l fills row 8 r + l / 8, LDS chunk l % 8,
// and so reads global chunk (l % 8) ^ ((row >> 1) & 7), the same for every i.
struct Src {
  const uint8_t* base[3];          // the tile's rows, w and w_up columns, at K = 0
  uint32_t a_off[kLd], b_off[kLd]; // from those bases
  uint32_t back;                   // taken off in the last stage where K ends inside it
  int n_stages;
};

template <bool GLU, int MT, int NT, int LO, int HI>   // runs 0 .. 2 MT - 1: rows, the 2 NT after: columns
__device__ __forceinline__ void load_runs(unsigned char* slot, const Src& s, int wave, int d) {
  constexpr int kRows = 2 * MT;
  const bool last = d >= s.n_stages - 1;        // stages past the end repeat the last one
  const int64_t k = int64_t(last ? s.n_stages - 1 : d) * kRowBytes;
  const uint32_t back = last ? s.back : 0u;
#pragma unroll
  for (int i = LO; i < HI; ++i) {
    const int run = ((i < kRows ? i : i - kRows) * 4 + wave) * 1024;
    const uint8_t* base = (i < kRows ? s.base[0] : s.base[GLU && i - kRows >= NT ? 2 : 1]) + k;
    const uint32_t o = (i < kRows ? s.a_off[i] : s.b_off[i - kRows]) - back;
    __builtin_amdgcn_global_load_lds(base + o, (lds_ptr)(slot + (i < kRows ? 0 : kTileBytes) + run), 16, 0, 0);
  }
}

template <int MT, int NT>
struct Frag {
  i32x4 a[MT], b[NT];
};
struct Lds {
  int a_row, b_row[kT], chunk[4];
};
template <int MT, int NT>
__device__ __forceinline__ void read_frag(const unsigned char* slot, const Lds& l, int kk, Frag<MT, NT>& f) {
#pragma unroll
  for (int i = 0; i < MT; ++i)
    f.a[i] = *reinterpret_cast<const i32x4*>(slot + l.a_row + i * 32 * kRowBytes + l.chunk[kk]);
#pragma unroll
  for (int j = 0; j < NT; ++j)
    f.b[j] = *reinterpret_cast<const i32x4*>(slot + kTileBytes + l.b_row[j] + l.chunk[kk]);
}

template <int KK, int MT, int NT>
__device__ __forceinline__ void mma(f32x16 (&acc)[MT][NT], const Frag<MT, NT>& f, const int (&sa)[MT], const int (&sb)[NT]) {
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const i32x8 a = {f.a[i].x, f.a[i].y, f.a[i].z, f.a[i].w, 0, 0, 0, 0};
      const i32x8 b = {f.b[j].x, f.b[j].y, f.b[j].z, f.b[j].w, 0, 0, 0, 0};
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc[i][j], 4, 4, KK, sb[j], KK, sa[i]);
    }
}

// Issue order of one slice: its M MFMAs, the first R each followed by an LDS
// read, N direct loads spread between them.
template <int M, int R, int N>
__device__ __forceinline__ void slice_order() {
  static_assert(R <= M && N <= M, "at most one of each per MFMA");
#pragma unroll
  for (int q = 0; q < M; ++q) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                     // MFMA
    if (q < R) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);          // LDS read
    if ((q * N) / M != ((q + 1) * N) / M) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
  }
}

// Scale dwords of four stages for MT rows and NT columns: [stage][row].
template <int MT, int NT>
struct Scales {
  int a[4][MT], b[4][NT];
};
struct ScaleSrc {
  const uint8_t* base[3];
  uint32_t a_off[kT], b_off[kT];
  int n_bytes;                     // K / 32
};
template <bool GLU, bool FULL, int MT, int NT>   // FULL: the four stages are all within K
__device__ __forceinline__ void load_scales(const ScaleSrc& s, int super, int half, int (&raw)[MT + NT][4]) {
  const uint32_t first = 32 * super + 16 * half;
  if (FULL || 32 * super + 32 <= s.n_bytes) {
#pragma unroll
    for (int i = 0; i < MT + NT; ++i) {
      const uint8_t* base = s.base[i < MT ? 0 : (GLU && i - MT >= NT / 2 ? 2 : 1)];
      const u32x4a q = *reinterpret_cast<const u32x4a*>(base + ((i < MT ? s.a_off[i] : s.b_off[i - MT]) + first));
      raw[i][0] = q.x; raw[i][1] = q.y; raw[i][2] = q.z; raw[i][3] = q.w;
    }
  } else {                                       // K ends in these four stages
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const bool in = int(first) + 4 * t < s.n_bytes;
      const uint32_t o = in ? first + 4 * t : 0u;
#pragma unroll
      for (int i = 0; i < MT + NT; ++i) {
        const uint8_t* base = s.base[i < MT ? 0 : (GLU && i - MT >= NT / 2 ? 2 : 1)];
        const int v = *reinterpret_cast<const int*>(base + ((i < MT ? s.a_off[i] : s.b_off[i - MT]) + o));
        raw[i][t] = in ? v : 0;
      }
    }
  }
}
// raw: lane half h holds dwords 4h..4h+3 of the 8; stage t wants dword 2t + h
template <int MT, int NT>
__device__ __forceinline__ void spread_scales(const int (&raw)[MT + NT][4], Scales<MT, NT>& s) {
#pragma unroll
  for (int i = 0; i < MT + NT; ++i) {
    const auto x = __builtin_amdgcn_permlane32_swap(raw[i][0], raw[i][1], false, false);
    const auto y = __builtin_amdgcn_permlane32_swap(raw[i][2], raw[i][3], false, false);
    const int d[4] = {int(x[0]), int(y[0]), int(x[1]), int(y[1])};
#pragma unroll
    for (int t = 0; t < 4; ++t) (i < MT ? s.a[t][i < MT ? i : 0] : s.b[t][i < MT ? 0 : i - MT]) = d[t];
  }
}

// Barrier that publishes the direct loads every wave has waited for; KEEP
// younger vector-memory operations may still be in flight.
template <int KEEP = 0>
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(KEEP));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Stage d from `cur`; on entry f0 holds its slice 0 and the row half of stage
// d + 1, if there is one, is on its way into `nxt`.  LEFT: stages after this
// one (2 for more than that); unless it is the last, f0 ends as slice 0 of the next.
// SCALES: the scales of the next four stages are asked for in slice 1, younger
// than all that this stage's barrier waits for, so that they have until the next
// one (16384 rows, K 14336, N 4096: 544 -> 526 us).
template <bool GLU, int T, int LEFT, bool SCALES, int MT, int NT>
__device__ __forceinline__ void stage(f32x16 (&acc)[MT][NT], Frag<MT, NT>& f0, Frag<MT, NT>& f1, unsigned char* cur,
                                      unsigned char* nxt, const Src& src, const Lds& l,
                                      const Scales<MT, NT>& sc, int wave, int d, const ScaleSrc& ss, int half,
                                      int (&raw)[MT + NT][4]) {
  constexpr int kRows = 2 * MT, kColumns = 2 * NT, kReads = MT + NT, kM = MT * NT;
  __builtin_amdgcn_sched_barrier(0);
  if (LEFT > 0) load_runs<GLU, MT, NT, kRows, kRows + kColumns>(nxt, src, wave, d + 1);
  read_frag(cur, l, 1, f1);
  mma<0>(acc, f0, sc.a[T], sc.b[T]);
  slice_order<kM, kReads, (LEFT > 0 ? kColumns : 0)>();
  __builtin_amdgcn_sched_barrier(0);
  if (SCALES) load_scales<GLU, true, MT, NT>(ss, (d >> 2) + 1, half, raw);
  read_frag(cur, l, 2, f0);
  mma<1>(acc, f1, sc.a[T], sc.b[T]);
  slice_order<kM, kReads, (SCALES ? kReads : 0)>();
  __builtin_amdgcn_sched_barrier(0);
  read_frag(cur, l, 3, f1);
  mma<2>(acc, f0, sc.a[T], sc.b[T]);
  slice_order<kM, kReads, 0>();
  __builtin_amdgcn_sched_barrier(0);
  if (LEFT > 0) {
    stage_barrier<SCALES ? kReads : 0>();   // stage d + 1 landed everywhere; cur is free
    __builtin_amdgcn_sched_barrier(0);
    if (LEFT > 1) load_runs<GLU, MT, NT, 0, kRows>(cur, src, wave, d + 2);
    read_frag(nxt, l, 0, f0);
  }
  mma<3>(acc, f1, sc.a[T], sc.b[T]);
  slice_order<kM, (LEFT > 0 ? kReads : 0), (LEFT > 1 ? kRows : 0)>();
  __builtin_amdgcn_sched_barrier(0);
}

// Real row tiles of all experts, under find_tile's clamping.
__device__ int count_tiles(const int32_t* __restrict__ offs, int n_experts, int n_rows) {
  int total = 0;
  for (int c = 0; c < n_experts; c += Experts<kBM>::kPer * kWave)
    total += lane_value(wave_inclusive_scan(Experts<kBM>(c, offs, n_experts, n_rows).sum), kWave - 1);
  return __builtin_amdgcn_readfirstlane(total);
}

template <bool GLU, int TAIL, bool FULL, int MT, int NT>
__device__ __forceinline__ void tile(const uint8_t* __restrict__ rows, const uint8_t* __restrict__ row_scales,
                                     int K, const uint8_t* __restrict__ w, const uint8_t* __restrict__ w_scales,
                                     const uint8_t* __restrict__ w_up, const uint8_t* __restrict__ w_up_scales,
                                     int N, uint16_t* __restrict__ y, const int32_t* __restrict__ order,
                                     const Tile& t, int n_tile, unsigned char* slot0, unsigned char* slot1) {
  constexpr int kCols = GLU ? 32 * NT : 64 * NT;   // output columns of a tile
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int wm = wave >> 1, wn = wave & 1, r32 = lane & 31, half = lane >> 5;
  const int64_t col0 = int64_t(n_tile) * kCols;
  const int64_t w_row0 = int64_t(t.expert) * N + col0;
  const int cols = N - int(col0);                // columns left, at least 1
  const int left = t.row_end - t.row0;           // rows left, at least 1
  // row i of the tile, from row `first` of rows and of row_scales
  const int first = order ? 0 : t.row0;
  auto row_at = [&](int i) { return order ? order[t.row0 + i] : i; };

  Src src;
  src.n_stages = (K + 255) / 256;
  src.base[0] = rows + int64_t(first) * (K / 2);
  src.base[1] = w + w_row0 * (K / 2);
  src.base[2] = GLU ? w_up + w_row0 * (K / 2) : nullptr;
  const int q8 = lane >> 3;
  const int chunk = (lane & 7) ^ ((4 * wave + (q8 >> 1)) & 7);
  src.back = K % 256 != 0 && chunk >= 4 ? 64u : 0u;
#pragma unroll
  for (int i = 0; i < kLd; ++i) {
    const int row = (4 * i + wave) * 8 + q8;
    const int ar = row < left ? row : left - 1;            // clamped rows are never stored
    const int bc = GLU ? row & (kCols - 1) : row;
    const int br = bc < cols ? bc : cols - 1;
    src.a_off[i] = uint32_t(row_at(ar)) * uint32_t(K / 2) + chunk * 16;
    src.b_off[i] = uint32_t(br) * uint32_t(K / 2) + chunk * 16;
  }
  // B tile rows of fragment j: columns wn*128 + 32 j, or with SwiGLU columns
  // wn*64 + 32 (j % 2) of w (j < 2) and of w_up
  Lds l;
  ScaleSrc ss;
  ss.n_bytes = K / 32;
  ss.base[0] = row_scales + int64_t(first) * ss.n_bytes;
  ss.base[1] = w_scales + w_row0 * ss.n_bytes;
  ss.base[2] = GLU ? w_up_scales + w_row0 * ss.n_bytes : nullptr;
  l.a_row = (wm * 32 * MT + r32) * kRowBytes;
#pragma unroll
  for (int i = 0; i < kT; ++i) {
    const int ar = wm * 32 * MT + 32 * i + r32;
    const int bc = (GLU ? wn * 16 * NT + 32 * (i % (NT / 2)) : wn * 32 * NT + 32 * i) + r32;
    l.b_row[i] = ((GLU && i >= NT / 2 ? kCols : 0) + bc) * kRowBytes;
    ss.a_off[i] = uint32_t(row_at(ar < left ? ar : left - 1)) * uint32_t(ss.n_bytes);
    ss.b_off[i] = uint32_t(bc < cols ? bc : cols - 1) * uint32_t(ss.n_bytes);
  }
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) l.chunk[kk] = ((4 * half + kk) ^ ((r32 >> 1) & 7)) << 4;

  f32x16 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  Frag<MT, NT> f0, f1;
  Scales<MT, NT> sc;
  int raw[MT + NT][4];
  load_runs<GLU, MT, NT, 0, 2 * MT + 2 * NT>(slot0, src, wave, 0);
  load_scales<GLU, FULL, MT, NT>(ss, 0, half, raw);
  stage_barrier();                               // stage 0 landed
  const int n_stages = src.n_stages;
  if (n_stages > 1) load_runs<GLU, MT, NT, 0, 2 * MT>(slot1, src, wave, 1);
  read_frag(slot0, l, 0, f0);
  int d = 0;
  for (; d + TAIL < n_stages; d += 4) {
    spread_scales(raw, sc);
    if (!FULL) load_scales<GLU, false, MT, NT>(ss, (d >> 2) + 1, half, raw);
    stage<GLU, 0, 2, FULL, MT, NT>(acc, f0, f1, slot0, slot1, src, l, sc, wave, d, ss, half, raw);
    stage<GLU, 1, 2, false, MT, NT>(acc, f0, f1, slot1, slot0, src, l, sc, wave, d + 1, ss, half, raw);
    stage<GLU, 2, 2, false, MT, NT>(acc, f0, f1, slot0, slot1, src, l, sc, wave, d + 2, ss, half, raw);
    stage<GLU, 3, 2, false, MT, NT>(acc, f0, f1, slot1, slot0, src, l, sc, wave, d + 3, ss, half, raw);
  }
  spread_scales(raw, sc);
  stage<GLU, 0, TAIL - 1, false, MT, NT>(acc, f0, f1, slot0, slot1, src, l, sc, wave, d, ss, half, raw);
  if constexpr (TAIL > 1) stage<GLU, 1, TAIL - 2, false, MT, NT>(acc, f0, f1, slot1, slot0, src, l, sc, wave, d + 1, ss, half, raw);
  if constexpr (TAIL > 2) stage<GLU, 2, TAIL - 3, false, MT, NT>(acc, f0, f1, slot0, slot1, src, l, sc, wave, d + 2, ss, half, raw);
  if constexpr (TAIL > 3) stage<GLU, 3, 0, false, MT, NT>(acc, f0, f1, slot1, slot0, src, l, sc, wave, d + 3, ss, half, raw);
  __builtin_amdgcn_s_waitcnt(wait_vm(0));        // no direct load may outlive the workgroup
  // the products end here, with every lane on, not in the divergent stores below
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) asm volatile("" : "+a"(acc[i][j]));

  // lane holds columns 8*(v/4) + 4*half + v%4 of row lane % 32 of each 32 x 32 tile
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = wm * 32 * MT + 32 * i + r32;
    if (r >= left) continue;
    uint16_t* out = y + int64_t(order ? order[t.row0 + r] : t.row0 + r) * N + col0;
#pragma unroll
    for (int j = 0; j < (GLU ? NT / 2 : NT); ++j)
#pragma unroll
      for (int v = 0; v < 16; v += 4) {
        const int c = (GLU ? wn * 16 * NT : wn * 32 * NT) + 32 * j + 2 * v + 4 * half;
        float o[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          o[u] = GLU ? silu(acc[i][j][v + u]) * acc[i][j + (GLU ? NT / 2 : 0)][v + u] : acc[i][j][v + u];
        store4(out, c, cols, N % 4 == 0, o);
      }
  }
}

// order: as in stream_kernel (rows * K / 2 below 2^32 then; only with ANY).
// 16384 rows in any order over 8 experts, K = N = 4096: 205 us, 399 by 64-row tiles.
// TAIL: the stages of the last group of up to four, each count its own straight
// line (exits in the middle of the four-stage loop made the compiler move the
// accumulators).  FULL: K is a multiple of 1024, so scales are always read four
// stages at a time (a branch for it inside a stage made the compiler spill).
// ANY: the tiles can be few, or rows be in any order (in every kernel these cost
// SwiGLU 1% and 2% where neither is so).
// Measured: 16384 rows over 8 experts, K 4096, F 14336 with SwiGLU, 3.85 TFLOP
// in 1.06 ms, 3.63 PFLOP/s; K 14336, N 4096 3.6 PFLOP/s.  The card's clock falls
// to 1.6-1.8 GHz under it, and MFMAs take 47-48% of the cycles at that clock;
// waves wait for 17-20% of theirs.  With all codes zero, which draws less power,
// the same calls run 11-16% faster, without the loads into LDS 17-21%.
template <bool GLU, int TAIL, bool FULL, bool ANY>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void tile_kernel(const uint8_t* __restrict__ rows, const uint8_t* __restrict__ row_scales, int n_rows,
                 int K, const int32_t* __restrict__ offs, int n_experts, const int32_t* __restrict__ order,
                 const uint8_t* __restrict__ w, const uint8_t* __restrict__ w_scales,
                 const uint8_t* __restrict__ w_up, const uint8_t* __restrict__ w_up_scales, int N,
                 uint16_t* __restrict__ y) {
  // two arrays, so the compiler can tell the slot being loaded from the slot
  // being read and adds no wait between them
  __shared__ __align__(1024) unsigned char slot0[kSlotBytes];
  __shared__ __align__(1024) unsigned char slot1[kSlotBytes];

  // XCD x (workgroup b runs on XCD b % 8) takes a contiguous range of the
  // grouped order: 8 row tiles x all column tiles, row tiles fastest
  const int m_real = count_tiles(offs, n_experts, n_rows);
  const bool few = few_tiles(m_real, N, GLU, ANY);
  const int n_tiles = int(col_tiles(N, GLU, few));
  const int64_t tiles = int64_t(m_real) * n_tiles;
  const int64_t per_xcd = (tiles + kXcds - 1) / kXcds;
  const int64_t in_xcd = blockIdx.x / kXcds;
  const int64_t tt = int64_t(blockIdx.x % kXcds) * per_xcd + in_xcd;
  if (in_xcd >= per_xcd || tt >= tiles) return;
  const int g = int(tt / (int64_t(kGroupM) * n_tiles));
  const int gm = m_real - g * kGroupM < kGroupM ? m_real - g * kGroupM : kGroupM;
  const int in_group = int(tt - int64_t(g) * kGroupM * n_tiles);
  const Tile t = find_tile<kBM>(g * kGroupM + in_group % gm, offs, n_experts, n_rows);
  if (!t.valid) return;
  const int n_tile = in_group / gm;
  const auto run = [&](auto mt, auto nt) {
    tile<GLU, TAIL, FULL, decltype(mt)::value, decltype(nt)::value>(
        rows, row_scales, K, w, w_scales, w_up, w_up_scales, N, y, ANY ? order : nullptr, t, n_tile, slot0, slot1);
  };
  const auto rows_of = [&](auto nt) {
    const int left = t.row_end - t.row0;
    if (left > 192) run(std::integral_constant<int, 4>(), nt);
    else if (left > 128) run(std::integral_constant<int, 3>(), nt);
    else run(std::integral_constant<int, 2>(), nt);
  };
  if constexpr (ANY) {
    if (few) return rows_of(std::integral_constant<int, 2>());
  }
  rows_of(std::integral_constant<int, 4>());
}

}  // namespace big

// Mean rows per expert from which tiles of 32 rows are taken, of 64 rows, and
// the tile kernel.  The rows are the call's, also those without an expert, which
// the launch cannot know.  Measured with equally popular experts (rows per
// expert: times in us of 16-, 32-, 64-row tiles and the tile kernel; 64 experts,
// K = N = 4096): 8: 104, 108, 114, -; 16: 138, 120, 116, -; 32: 212, 148, 121,
// 128; 48: 288, 186, 138, 136; 64: 366, 225, 163, 141; 128: 678, 393, 255, 166.
// 256 experts, K 7168, N 4096: 40 rows 847 and 846, 56 rows 912 and 872.  With 8
// experts 32-row tiles lead up to 24: 14.7 against 23.4 and 16.1; 64-row tiles
// and the tile kernel take 17.0 and 16.7 at 48, 26.3 and 16.9 at 56.
constexpr int64_t kNarrowRows = 10, kMiddleRows = 24, kManyRows = 48;

constexpr int kStreamWaves = 4;    // 8 measured the same where rows are many, 2-8% slower where few

// The kernel that takes a product, and its grid.
struct Shape {
  bool big, direct;
  bool any;                        // big: the tiles can turn out to be few, or rows are in any order
  int nb;                          // stream: 16-row groups per tile
  int col_tiles;                   // stream: column groups
  int64_t blocks;
};
Shape shape_of(const Mxfp4Product& g, bool gather) {
  Shape s{};
  const int64_t rows = g.n_rows, e = g.n_experts;
  // rows in any order are 32-bit offsets from the first in the tile kernel
  s.big = rows >= kManyRows * e && (!gather || rows * (g.k_dim / 2) < int64_t(1) << 32);
  if (s.big) {
    s.any = gather || big::few_tiles((rows + big::kBM - 1) / big::kBM, g.n_dim, g.w_up, true);
    s.blocks = big::blocks_for(most_tiles(rows, g.n_experts, big::kBM), g.n_dim, g.w_up, s.any);
    s.blocks = (s.blocks + kXcds - 1) / kXcds * kXcds;   // every XCD as many
    return s;
  }
  s.nb = rows < kNarrowRows * e ? 1 : (rows < kMiddleRows * e ? 2 : 4);
  s.direct = gather && s.nb == 1 && rows <= kDirectRows;
  const int cols = kStreamWaves * (g.w_up ? 16 : 32);
  s.col_tiles = int((g.n_dim + cols - 1) / cols);
  s.blocks = (most_tiles(rows, g.n_experts, 16 * s.nb) + kXcds - 1) / kXcds * kXcds * s.col_tiles;
  return s;
}

// index: expert offsets, or with s.direct the expert of each row.
hipError_t launch_product(const Mxfp4Product& g, const Shape& s, const int32_t* index,
                          const int32_t* order, hipStream_t stream) {
  const uint8_t *x = static_cast<const uint8_t*>(g.rows), *w = static_cast<const uint8_t*>(g.w),
                *u = static_cast<const uint8_t*>(g.w_up);
  uint16_t* y = static_cast<uint16_t*>(g.y);
  const int n_rows = int(g.n_rows), k = int(g.k_dim), n = int(g.n_dim);
  const unsigned blocks = unsigned(s.blocks);
  auto big_kernel = [&](auto kernel) {
    kernel<<<blocks, big::kThreads, 0, stream>>>(x, g.row_scales, n_rows, k, index, g.n_experts, order, w, g.w_scales, u, g.w_up_scales, n, y);
  };
  auto stream_kernel = [&](auto kernel) {
    kernel<<<blocks, kStreamWaves * kWave, 0, stream>>>(x, g.row_scales, n_rows, k, index, g.n_experts, order, w, g.w_scales, u, g.w_up_scales, n, y, s.col_tiles);
  };
  auto pick = [&](auto glu, auto x4) {
    constexpr bool G = decltype(glu)::value, X4 = decltype(x4)::value;
    constexpr int W = kStreamWaves;
    if (s.direct) stream_kernel(stream::stream_kernel<G, 1, W, X4, true>);
    else if (s.nb == 1) stream_kernel(stream::stream_kernel<G, 1, W, X4, false>);
    else if (s.nb == 2) stream_kernel(stream::stream_kernel<G, 2, W, X4, false>);
    else stream_kernel(stream::stream_kernel<G, 4, W, X4, false>);
  };
  auto go = [&](auto glu) {
    constexpr bool G = decltype(glu)::value;
    auto tiles = [&](auto any) {
      constexpr bool A = decltype(any)::value;
      if (k % 1024 == 0) return big_kernel(big::tile_kernel<G, 4, true, A>);
      switch ((k + 255) / 256 % 4) {
        case 1: return big_kernel(big::tile_kernel<G, 1, false, A>);
        case 2: return big_kernel(big::tile_kernel<G, 2, false, A>);
        case 3: return big_kernel(big::tile_kernel<G, 3, false, A>);
        default: return big_kernel(big::tile_kernel<G, 4, false, A>);
      }
    };
    if (s.big) return s.any ? tiles(std::true_type()) : tiles(std::false_type());
    if (k % 512 == 0) pick(glu, std::true_type());
    else pick(glu, std::false_type());
  };
  if (u) go(std::true_type());
  else go(std::false_type());
  return hipGetLastError();
}

}  // namespace

int64_t gemm_mxfp4_blocks(const Mxfp4Product& g, bool gather) { return shape_of(g, gather).blocks; }

size_t gather_gemm_mxfp4_workspace_bytes(int64_t n_rows, int n_experts) {
  return gather_layout(n_rows, n_experts).total;
}

hipError_t launch_grouped_gemm_mxfp4(const Mxfp4Product& g, const int32_t* expert_offsets,
                                     hipStream_t stream) {
  return launch_product(g, shape_of(g, false), expert_offsets, nullptr, stream);
}

hipError_t launch_gather_gemm_mxfp4(const Mxfp4Product& g, const int32_t* row_expert,
                                    void* workspace, hipStream_t stream) {
  const Shape s = shape_of(g, true);
  if (s.direct) return launch_product(g, s, row_expert, nullptr, stream);
  const int32_t *offsets = nullptr, *order = nullptr;
  const hipError_t err = launch_grouping(row_expert, g.n_rows, g.n_experts, workspace, &offsets, &order, stream);
  if (err != hipSuccess) return err;
  return launch_product(g, s, offsets, order, stream);
}

}  // namespace moe
