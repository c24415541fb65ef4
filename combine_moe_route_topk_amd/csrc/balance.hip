// Load-balance and z losses of a softmax top-k router, per sequence of tokens,
// with the per-expert counts they rest on, and their gradient.
//   p_t = softmax(l_t),  lse_t = log sum_e exp(l_te)
//   c_e = pairs of the sequence's n counted tokens routed to e,  P_e = sum_t p_te / n
//   loss = E / (k n) sum_e c_e P_e,   z = sum_t lse_t^2 / n
//   d l_te = p_te (u_e - sum_i p_ti u_i + 2 d_z lse_t / n),
//   u_e = d_loss (E c_e - k n) / (k n^2)
// c is piecewise constant and has no gradient.  u is the count less its mean,
// taken in integers: the mean would fall out of u_e - sum_i p_ti u_i anyway, and
// without it that difference loses no digits where the experts are nearly even.
//
// Both kernels read the logits once.  16 lanes hold a token of up to 256 experts
// (a wave four tokens), so the row's maximum and sum are four exchanges within a
// row of lanes; more experts take a whole wave per token.  A token's logits are
// asked for while the one before it is worked on.  32768 tokens of 256 experts in 37
// sequences: 13.1 us forward (34.6 MB, 2.6 TB/s) and 8.7 us for the sums, 18.1 us backward
// (67 MB, 3.7 TB/s; a large copy reaches 4.95), with 28 vector instructions to a logit
// forward and 32 backward, two thirds of them the exponential's, which take some 7 us by
// themselves.  4096 tokens: 4.1, 5.6 and 5.1 us, little more than launches and first loads.
#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"

namespace moe {

namespace {

constexpr int kBlock = 256;
constexpr int kSliceExperts = 32;      // experts per workgroup of the second launch

// Tokens per workgroup, usually a multiple of the 16 that its waves hold at once, so that
// about kChunks workgroups share them; up to kOneChunk tokens are one workgroup's,
// which then finishes the sums itself.  512, 1024 and 2048 for 32768 tokens of 256
// experts in 37 sequences: 13.9, 13.5 and 13.7 us, backward (its counts still loaded
// one by one) 24.7, 22.1 and 24.8.
// Sequences follow one another within a chunk, each with its own chain of loads, so
// a chunk holds no more tokens than a sequence does on average, and one workgroup
// takes all tokens of at most kOneSeqs sequences.  256 experts, 12 tokens in 44
// sequences 29 -> 13 us and backward 28 -> 5, 51 in 16: 31 -> 14 and 13 -> 9; 64 tokens
// in 3 and 4, one workgroup or two launches: 10.5 and 10.8, 12.6 and 11.0 us.
constexpr int kChunks = 1024, kOneChunk = 64, kOneSeqs = 3;
int64_t chunk_tokens(int64_t n_tokens, int64_t n_seqs) {
  const int64_t c = (n_tokens + kChunks - 1) / kChunks, mean = n_tokens / n_seqs;
  const int64_t most = c < 16 ? 16 : (c + 15) / 16 * 16;
  return mean < 1 ? 1 : (mean < most ? mean : most);
}

// Sums of one sequence within one chunk of tokens.  Chunk c and sequence b meet
// in slot c + b: along the tokens either c or b grows, so no two pairs share a
// slot, and a sequence's slots follow one another.
struct Partials {
  float* probs;        // [slots, E]
  int32_t* counts;     // [slots, E]
  int32_t* tokens;     // [slots]
  float* z;            // [slots]
  int32_t* tickets;    // [B]
  float* slices;       // [B, slices]: parts of a sequence's loss
};
// Slots of a call, or more: the most that n <= n_tokens tokens in b <= n_seqs sequences
// take, so that a workspace made for the largest batch holds every smaller one.  Fewer
// tokens can take more chunks, since a chunk's length jumps.  Where it is the 16 ceil(n /
// 16384) tokens of chunk_tokens there are at most n / 16 chunks and at most 1024; where it
// is the mean m = n / b >= 1, ceil(n / m) <= b + ceil((b - 1) / m) <= 2 b - 1; with m < 1
// they are n < b; and n at most in every case.
int64_t most_slots(int64_t n_tokens, int64_t n_seqs) {
  const int64_t even = (n_tokens + 15) / 16 < kChunks ? (n_tokens + 15) / 16 : kChunks;
  const int64_t by_mean = n_tokens < 2 * n_seqs - 1 ? n_tokens : 2 * n_seqs - 1;
  return (even > by_mean ? even : by_mean) + n_seqs;
}
struct Layout {
  int64_t chunk, chunks;
  int slices;
  size_t counts, tokens, z, tickets, slice_sums, total;
};
Layout layout_of(int64_t n_tokens, int n_experts, int64_t n_seqs) {
  Layout L{};
  L.chunk = chunk_tokens(n_tokens, n_seqs);
  L.chunks = (n_tokens + L.chunk - 1) / L.chunk;
  const int64_t slots = most_slots(n_tokens, n_seqs);
  L.slices = (n_experts + kSliceExperts - 1) / kSliceExperts;
  const auto after = [](size_t o, size_t n) { return (o + n * 4 + 255) / 256 * 256; };
  L.counts = after(0, size_t(slots) * n_experts);
  L.tokens = after(L.counts, size_t(slots) * n_experts);
  L.z = after(L.tokens, size_t(slots));
  L.tickets = after(L.z, size_t(slots));
  L.slice_sums = after(L.tickets, size_t(n_seqs));
  L.total = after(L.slice_sums, size_t(n_seqs) * L.slices);
  return L;
}

template <int CTRL>
__device__ __forceinline__ float row_step(float v) {
  const int b = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, false));
}
// Maximum and sum over the LANES lanes of a token, the same in each of them:
// quads, half rows, rows of 16, then halves of the wave.
template <int LANES, typename Op>
__device__ __forceinline__ float reduce_lanes(float v, Op op) {
  v = op(v, row_step<0xB1>(v));        // lanes 1 0 3 2
  v = op(v, row_step<0x4E>(v));        // lanes 2 3 0 1
  v = op(v, row_step<0x141>(v));       // row_half_mirror
  v = op(v, row_step<0x140>(v));       // row_mirror
  if constexpr (LANES == 64) {
    v = op(v, __shfl_xor(v, 16));
    v = op(v, __shfl_xor(v, 32));
  }
  return v;
}
struct Max { __device__ float operator()(float a, float b) const { return fmaxf(a, b); } };
struct Add { __device__ float operator()(float a, float b) const { return a + b; } };

// Expert of slot r of lane i of a token.
template <int LANES>
__device__ __forceinline__ int expert_of(int i, int r) { return 4 * (i + LANES * (r / 4)) + r % 4; }

// A token's logits, -inf past the last expert.
template <int LANES, int R, bool VEC>
__device__ __forceinline__ void load_token(const float* __restrict__ row, int n_experts, int i, float (&v)[R]) {
#pragma unroll
  for (int r = 0; r < R; r += 4) {
    const int e = expert_of<LANES>(i, r);
    if (VEC) {
      float4 w = make_float4(-__builtin_inff(), -__builtin_inff(), -__builtin_inff(), -__builtin_inff());
      if (e < n_experts) w = *reinterpret_cast<const float4*>(row + e);
      v[r] = w.x; v[r + 1] = w.y; v[r + 2] = w.z; v[r + 3] = w.w;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[r + q] = e + q < n_experts ? row[e + q] : -__builtin_inff();
    }
  }
}

// A token's logits to its probabilities; p ends as 0 past the last expert.  live:
// some logit is above -inf (a NaN is none of these: it is carried on).
template <int LANES, int R>
__device__ __forceinline__ void token_softmax(float (&p)[R], float& lse, bool& live) {
  float top = p[0];
#pragma unroll
  for (int r = 1; r < R; ++r) top = fmaxf(top, p[r]);
  top = reduce_lanes<LANES>(top, Max());
  if (top == -__builtin_inff()) top = 0.f;       // no finite logit: every term is 0 (or NaN)
  float sum = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    p[r] = expf(p[r] - top);
    sum += p[r];
  }
  sum = reduce_lanes<LANES>(sum, Add());
  live = sum != 0.f;
  const float inv = live ? 1.f / sum : 0.f;
  lse = top + logf(sum);
#pragma unroll
  for (int r = 0; r < R; ++r) p[r] *= inv;
}

// Runs f(t, v) over the tokens lo + team, + TEAMS, ... before hi that the mask keeps
// (and g(t) over the others), the next token's logits asked for before f.  No sum
// passes hi, which may be the largest int.
template <int LANES, int R, bool VEC, int TEAMS, typename F, typename G>
__device__ __forceinline__ void for_tokens(const float* __restrict__ logits, const uint8_t* __restrict__ mask,
                                           int n_experts, int i, int team, int lo, int hi, F f, G g) {
  if (hi - lo <= team) return;
  float next[R];
  bool keep = false;
  const auto ask = [&](int t) __attribute__((always_inline)) {
    keep = !mask || mask[t];
    load_token<LANES, R, VEC>(logits + int64_t(t) * n_experts, n_experts, i, next);
  };
  ask(lo + team);
  for (int t = lo + team;; t += TEAMS) {
    float v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = next[r];
    const bool kept = keep, more = hi - t > TEAMS;
    if (more) ask(t + TEAMS);
    if (kept) f(t, v);
    else g(t);
    if (!more) break;
  }
}

// First sequence that ends behind token t: the number of ends offs[1 .. n] at or
// before it, 64 of them looked at in each step.  Every lane calls it.
__device__ int first_sequence(const int32_t* __restrict__ offs, int n_seqs, int t) {
  int lo = 0, hi = n_seqs;               // the answer lies in [lo, hi]
  while (hi > lo) {
    const int step = (hi - lo + kWave - 1) / kWave;
    const int at = lo + (lane_id() + 1) * step;       // the end of sequence at - 1
    const int k = __popcll(ballot(at <= hi && offs[at <= hi ? at : hi] <= t));
    const int base = lo + k * step;
    hi = step == 1 ? base : (base + step - 1 < hi ? base + step - 1 : hi);
    lo = base;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Walks the tokens [t0, t1) sequence by sequence: f(b, lo, hi), b = -1 for tokens
// of no sequence.  Offsets are clamped into the tokens, whatever they hold.
template <typename F>
__device__ __forceinline__ void for_sequences(const int32_t* __restrict__ offs, int n_seqs, int t0,
                                              int t1, F f) {
  if (!offs) return f(0, t0, t1);
  int t = t0;
  for (int b = first_sequence(offs, n_seqs, t0); b < n_seqs && t < t1; ++b) {
    int lo = offs[b], hi = offs[b + 1];
    lo = lo < t ? t : (lo > t1 ? t1 : lo);
    hi = hi < lo ? lo : (hi > t1 ? t1 : hi);
    if (lo > t) f(-1, t, lo);
    if (hi > lo) f(b, lo, hi);
    t = hi;
  }
  if (t < t1) f(-1, t, t1);
}

struct ForwardArgs {
  const float* logits;
  const int32_t* idx;
  const int32_t* offs;
  const uint8_t* mask;
  int n_tokens, n_experts, k, n_seqs, chunk;
  float *loss, *z_loss;
  int32_t* counts;
  float* probs;
  int32_t* tokens;
  Partials part;
};

__device__ __forceinline__ float mean_loss(float sum, int n_experts, int k, int n) {
  return n > 0 ? sum * (float(n_experts) / (float(k) * (float(n) * float(n)))) : 0.f;
}

// One workgroup per chunk of tokens.  ONE: a single chunk, whose sums are the
// results; else they go to the chunk's slots.
template <int LANES, int R, bool VEC, bool ONE>
__global__ __launch_bounds__(kBlock) void balance_kernel(ForwardArgs a) {
  constexpr int kTeams = kBlock / LANES, kPadded = LANES * R;
  __shared__ float s_p[kTeams][kPadded];
  __shared__ int s_c[kPadded];
  __shared__ float s_z[kTeams], s_sum[kBlock / kWave];
  __shared__ int s_n[kTeams];
  const int tid = threadIdx.x, team = tid / LANES, i = tid % LANES;
  if (ONE) {
    for (int q = tid; q < a.n_seqs * a.n_experts; q += kBlock) { a.counts[q] = 0; a.probs[q] = 0.f; }
    for (int q = tid; q < a.n_seqs; q += kBlock) { a.loss[q] = 0.f; a.z_loss[q] = 0.f; a.tokens[q] = 0; }
  } else {
    for (int q = blockIdx.x * kBlock + tid; q < a.n_seqs; q += gridDim.x * kBlock) a.part.tickets[q] = 0;
  }
  for (int q = tid; q < kPadded; q += kBlock) s_c[q] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * a.chunk;
  const int t1 = a.n_tokens - t0 < a.chunk ? a.n_tokens : t0 + a.chunk;
  for_sequences(a.offs, a.n_seqs, t0, t1, [&](int b, int lo, int hi) {
    if (b < 0) return;
    float acc[R], z = 0.f;
    int n = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = 0.f;
    const auto add = [&](int t, float (&p)[R]) __attribute__((always_inline)) {
      float lse;
      bool live;
      int e = i < a.k ? a.idx[int64_t(t) * a.k + i] : -1;
      token_softmax<LANES, R>(p, lse, live);
      if (!live) return;
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] += p[r];
      z += lse * lse;
      ++n;
      if (unsigned(e) < unsigned(a.n_experts)) atomicAdd(&s_c[e], 1);
      for (int j = i + LANES; j < a.k; j += LANES) {
        e = a.idx[int64_t(t) * a.k + j];
        if (unsigned(e) < unsigned(a.n_experts)) atomicAdd(&s_c[e], 1);
      }
    };
    for_tokens<LANES, R, VEC, kTeams>(a.logits, a.mask, a.n_experts, i, team, lo, hi, add, [](int) {});
#pragma unroll
    for (int r = 0; r < R; ++r) s_p[team][expert_of<LANES>(i, r)] = acc[r];
    if (i == 0) { s_z[team] = z; s_n[team] = n; }
    __syncthreads();
    const int64_t slot = ONE ? b : int64_t(blockIdx.x) + b;
    float zs = 0.f, dot = 0.f;
    int ns = 0;
    for (int g = 0; g < kTeams; ++g) { zs += s_z[g]; ns += s_n[g]; }
    for (int e = tid; e < a.n_experts; e += kBlock) {
      float sum = 0.f;
#pragma unroll
      for (int g = 0; g < kTeams; ++g) sum += s_p[g][e];
      const int c = s_c[e];
      s_c[e] = 0;
      if (ONE) {
        a.counts[slot * a.n_experts + e] = c;
        a.probs[slot * a.n_experts + e] = ns > 0 ? sum / float(ns) : 0.f;
        dot += float(c) * sum;
      } else {
        a.part.counts[slot * a.n_experts + e] = c;
        a.part.probs[slot * a.n_experts + e] = sum;
      }
    }
    if (ONE) {
      dot = reduce_lanes<kWave>(dot, Add());
      if (lane_id() == 0) s_sum[tid / kWave] = dot;
    }
    __syncthreads();
    if (tid == 0) {
      if (ONE) {
        float sum = 0.f;
        for (int w = 0; w < kBlock / kWave; ++w) sum += s_sum[w];
        a.loss[slot] = mean_loss(sum, a.n_experts, a.k, ns);
        a.z_loss[slot] = ns > 0 ? zs / float(ns) : 0.f;
        a.tokens[slot] = ns;
      } else {
        a.part.z[slot] = zs;
        a.part.tokens[slot] = ns;
      }
    }
  });
}

// Second launch: a workgroup per sequence and 32 experts adds the slots of the
// sequence, 32 rows at a time and always in the same order, and the last
// workgroup of a sequence adds the 32-expert parts of its loss.  kDeep rows of a
// thread are in flight, and the last workgroup asks for all parts at once: 256 slots
// of 256 experts 10.5 -> 5.4 us, of which the ticket and its visibility are about 3.
constexpr int kDeep = 8;
// LOOP: a workgroup per sequence takes all its experts, 32 after 32, and draws no
// ticket, from kLoopBlocks workgroups of the other form on (each ticket makes a cache
// visible to the other XCDs).  The whole loss of 4096 tokens of 256 experts in 64, 128
// and 512 sequences, with tickets 21, 30 and 86 us, without 24, 25 and 27.  All of these
// sequences are alike; the slots of one long sequence among many short ones are one
// workgroup's too (32768 tokens in 128 sequences: 25 us, with one of 30000 tokens 61).
constexpr int64_t kLoopBlocks = 768;
template <bool VEC, bool LOOP>
__global__ __launch_bounds__(kBlock) void balance_sum_kernel(ForwardArgs a, int n_slices) {
  constexpr int kQuads = kSliceExperts / 4, kRows = kBlock / kQuads;
  __shared__ float s_p[kRows][kSliceExperts + 1];
  __shared__ int s_c[kRows][kSliceExperts + 1];
  __shared__ float s_z[kBlock];
  __shared__ int s_n[kBlock];
  const int b = LOOP ? blockIdx.x : blockIdx.x / n_slices;
  int slice = LOOP ? 0 : blockIdx.x % n_slices;
  const int tid = threadIdx.x, q = tid % kQuads, row = tid / kQuads;
  int lo = a.offs ? a.offs[b] : 0, hi = a.offs ? a.offs[b + 1] : a.n_tokens;
  lo = lo < 0 ? 0 : (lo > a.n_tokens ? a.n_tokens : lo);
  hi = hi < lo ? lo : (hi > a.n_tokens ? a.n_tokens : hi);
  const int64_t first = int64_t(lo / a.chunk) + b;
  const int count = hi > lo ? (hi - 1) / a.chunk - lo / a.chunk + 1 : 0;

  float z = 0.f, dot = 0.f, part = 0.f;          // part: in lane s, of slice s
  int n = 0;
  for (int s = tid; s < count; s += kBlock) { z += a.part.z[first + s]; n += a.part.tokens[first + s]; }
  s_z[tid] = z;
  s_n[tid] = n;
  for (;; ++slice) {
    const int e0 = slice * kSliceExperts + 4 * q;
    float p[4] = {0.f, 0.f, 0.f, 0.f};
    int c[4] = {0, 0, 0, 0};
    for (int s = row; s < count; s += kDeep * kRows) {
      float pr[kDeep][4];
      int cr[kDeep][4];
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        const int at_row = s + d * kRows;
        const int64_t at = (first + (at_row < count ? at_row : s)) * a.n_experts + e0;
        if (VEC) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          int4 y = make_int4(0, 0, 0, 0);
          if (e0 < a.n_experts) {
            x = *reinterpret_cast<const float4*>(a.part.probs + at);
            y = *reinterpret_cast<const int4*>(a.part.counts + at);
          }
          pr[d][0] = x.x; pr[d][1] = x.y; pr[d][2] = x.z; pr[d][3] = x.w;
          cr[d][0] = y.x; cr[d][1] = y.y; cr[d][2] = y.z; cr[d][3] = y.w;
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            pr[d][v] = e0 + v < a.n_experts ? a.part.probs[at + v] : 0.f;
            cr[d][v] = e0 + v < a.n_experts ? a.part.counts[at + v] : 0;
          }
        }
      }
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        if (s + d * kRows >= count) break;
#pragma unroll
        for (int v = 0; v < 4; ++v) { p[v] += pr[d][v]; c[v] += cr[d][v]; }
      }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) { s_p[row][4 * q + v] = p[v]; s_c[row][4 * q + v] = c[v]; }
    __syncthreads();
    if (tid < kWave) {
      // its lanes add the tokens, and 32 of them an expert each
      z = 0.f;
      n = 0;
      for (int w = 0; w < kBlock; w += kWave) { z += s_z[w + tid]; n += s_n[w + tid]; }
      z = reduce_lanes<kWave>(z, Add());
      for (int d = 1; d < kWave; d <<= 1) n += __shfl_xor(n, d);
      dot = 0.f;
      const int e = slice * kSliceExperts + tid;
      if (tid < kSliceExperts && e < a.n_experts) {
        float sum = 0.f;
        int cs = 0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) { sum += s_p[r][tid]; cs += s_c[r][tid]; }
        a.counts[int64_t(b) * a.n_experts + e] = cs;
        a.probs[int64_t(b) * a.n_experts + e] = n > 0 ? sum / float(n) : 0.f;
        dot = float(cs) * sum;
      }
      dot = reduce_lanes<kWave>(dot, Add());
      if (LOOP && tid == slice) part = dot;
    }
    if (!LOOP || slice + 1 == n_slices) break;
    __syncthreads();                             // s_p and s_c are read
  }
  if (tid >= kWave) return;
  if (LOOP) {
    dot = reduce_lanes<kWave>(part, Add());
  } else if (n_slices > 1) {
    float* parts = a.part.slices + int64_t(b) * n_slices;
    int last = 0;
    if (tid == 0) {
      // made visible to the other XCDs before the ticket is drawn
      __hip_atomic_store(parts + slice, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(&a.part.tickets[b], 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == n_slices - 1;
    }
    if (!__builtin_amdgcn_readfirstlane(last)) return;
    // at most 32 parts (1024 experts), one to a lane
    dot = tid < n_slices ? __hip_atomic_load(parts + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.f;
    dot = reduce_lanes<kWave>(dot, Add());
  }
  if (tid == 0) {
    a.loss[b] = mean_loss(dot, a.n_experts, a.k, n);
    a.z_loss[b] = n > 0 ? z / float(n) : 0.f;
    a.tokens[b] = n;
  }
}

struct BackwardArgs {
  const float* logits;
  const int32_t* offs;
  const uint8_t* mask;
  const int32_t* counts;
  const int32_t* tokens;
  const float *d_loss, *d_z;
  int n_tokens, n_experts, k, n_seqs, chunk;
  float* d_logits;
};

// One workgroup per chunk of tokens, the lanes as in balance_kernel; a lane keeps
// the u of its experts while the sequence lasts.
template <int LANES, int R, bool VEC, bool ADD>
__global__ __launch_bounds__(kBlock) void balance_backward_kernel(BackwardArgs a) {
  constexpr int kTeams = kBlock / LANES;
  const int team = threadIdx.x / LANES, i = threadIdx.x % LANES;
  const int t0 = blockIdx.x * a.chunk;
  const int t1 = a.n_tokens - t0 < a.chunk ? a.n_tokens : t0 + a.chunk;
  for_sequences(a.offs, a.n_seqs, t0, t1, [&](int b, int lo, int hi) {
    const int n = b < 0 ? 0 : a.tokens[b];
    float u[R], zf = 0.f;
    if (n > 0) {
      const float f = a.d_loss[b] / (float(a.k) * (float(n) * float(n)));
      zf = a.d_z ? 2.f * a.d_z[b] / float(n) : 0.f;
      const double mean = -double(a.k) * double(n);
      const int32_t* counts = a.counts + int64_t(b) * a.n_experts;
      // whole numbers below 2^53
      const auto centred = [&](int c) __attribute__((always_inline)) { return f * float(fma(double(c), double(a.n_experts), mean)); };
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const int e = expert_of<LANES>(i, r);
        if (VEC) {
          const int4 c = e < a.n_experts ? *reinterpret_cast<const int4*>(counts + e) : make_int4(0, 0, 0, 0);
          u[r] = u[r + 1] = u[r + 2] = u[r + 3] = 0.f;
          if (e < a.n_experts) { u[r] = centred(c.x); u[r + 1] = centred(c.y); u[r + 2] = centred(c.z); u[r + 3] = centred(c.w); }
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) u[r + q] = e + q < a.n_experts ? centred(counts[e + q]) : 0.f;
        }
      }
    }
    const auto put = [&](int t, const float (&p)[R]) __attribute__((always_inline)) {
      float* out = a.d_logits + int64_t(t) * a.n_experts;
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        // the gradient is rounded before it is added: the same bits as two calls and a sum
#pragma clang fp contract(off)
        const int e = expert_of<LANES>(i, r);
        if (VEC) {
          if (e < a.n_experts) {
            float4* o = reinterpret_cast<float4*>(out + e);
            float4 v = make_float4(p[r], p[r + 1], p[r + 2], p[r + 3]);
            if (ADD) { const float4 w = *o; v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w; }
            *o = v;
          }
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (e + q < a.n_experts) out[e + q] = p[r + q] + (ADD ? out[e + q] : 0.f);
        }
      }
    };
    const auto none = [&](int t) __attribute__((always_inline)) {
      if (ADD) return;
      float p[R];
#pragma unroll
      for (int r = 0; r < R; ++r) p[r] = 0.f;
      put(t, p);
    };
    if (n <= 0) {
      for (int left = hi - lo - team; left > 0; left -= kTeams) none(hi - left);
      return;
    }
    for_tokens<LANES, R, VEC, kTeams>(a.logits, a.mask, a.n_experts, i, team, lo, hi,
                                      [&](int t, float (&p)[R]) __attribute__((always_inline)) {
      float lse, dot = 0.f;
      bool live;
      token_softmax<LANES, R>(p, lse, live);
      if (!live) return none(t);
#pragma unroll
      for (int r = 0; r < R; ++r) dot += p[r] * u[r];
      dot = reduce_lanes<LANES>(dot, Add());
      const float shift = zf * lse - dot;
#pragma unroll
      for (int r = 0; r < R; ++r) p[r] *= u[r] + shift;
      put(t, p);
    }, none);
  });
}

// Lanes and slots per token by the number of experts: f(lanes, slots, vec).
template <typename F>
void by_experts(int n_experts, bool vec, F f) {
  const auto go = [&](auto lanes, auto slots) {
    if (vec) f(lanes, slots, std::true_type());
    else f(lanes, slots, std::false_type());
  };
  using std::integral_constant;
  if (n_experts <= 64) go(integral_constant<int, 16>(), integral_constant<int, 4>());
  else if (n_experts <= 128) go(integral_constant<int, 16>(), integral_constant<int, 8>());
  else if (n_experts <= 256) go(integral_constant<int, 16>(), integral_constant<int, 16>());
  else if (n_experts <= 512) go(integral_constant<int, 64>(), integral_constant<int, 8>());
  else go(integral_constant<int, 64>(), integral_constant<int, 16>());
}

bool rows_of_16_bytes(const void* p, int n_experts) {
  return n_experts % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

}  // namespace

size_t balance_workspace_bytes(int64_t n_tokens, int n_experts, int64_t n_seqs) {
  return layout_of(n_tokens, n_experts, n_seqs).total;
}

hipError_t launch_balance_loss(const BalanceForward& g, void* workspace, hipStream_t stream) {
  const Layout L = layout_of(g.n_tokens, g.n_experts, g.n_seqs);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const Partials part{reinterpret_cast<float*>(ws), reinterpret_cast<int32_t*>(ws + L.counts),
                      reinterpret_cast<int32_t*>(ws + L.tokens), reinterpret_cast<float*>(ws + L.z),
                      reinterpret_cast<int32_t*>(ws + L.tickets), reinterpret_cast<float*>(ws + L.slice_sums)};
  const bool one = g.n_tokens <= kOneChunk && g.n_seqs <= kOneSeqs;
  const ForwardArgs a{g.logits, g.topk_idx, g.seq_offsets, g.token_mask, int(g.n_tokens), g.n_experts, g.k,
                      g.n_seqs, one ? kOneChunk : int(L.chunk), g.loss, g.z_loss, g.counts, g.probs, g.tokens, part};
  by_experts(g.n_experts, rows_of_16_bytes(g.logits, g.n_experts), [&](auto lanes, auto slots, auto vec) {
    constexpr int kL = decltype(lanes)::value, kR = decltype(slots)::value;
    constexpr bool kV = decltype(vec)::value;
    if (one) balance_kernel<kL, kR, kV, true><<<1, kBlock, 0, stream>>>(a);
    // without a token there is still a workgroup, which clears the tickets
    else balance_kernel<kL, kR, kV, false><<<L.chunks > 0 ? unsigned(L.chunks) : 1u, kBlock, 0, stream>>>(a);
  });
  if (!one) {
    const bool loop = int64_t(g.n_seqs) * L.slices >= kLoopBlocks;
    const unsigned blocks = unsigned(g.n_seqs) * unsigned(loop ? 1 : L.slices);
    const auto sum = [&](auto vec) {
      constexpr bool kV = decltype(vec)::value;
      if (loop) balance_sum_kernel<kV, true><<<blocks, kBlock, 0, stream>>>(a, L.slices);
      else balance_sum_kernel<kV, false><<<blocks, kBlock, 0, stream>>>(a, L.slices);
    };
    if (g.n_experts % 4 == 0) sum(std::true_type());
    else sum(std::false_type());
  }
  return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const BalanceBackward& g, hipStream_t stream) {
  const int64_t chunk = chunk_tokens(g.n_tokens, g.n_seqs);
  const BackwardArgs a{g.logits, g.seq_offsets, g.token_mask, g.counts, g.tokens, g.d_loss, g.d_z_loss,
                       int(g.n_tokens), g.n_experts, g.k, g.n_seqs, int(chunk), g.d_logits};
  const unsigned blocks = unsigned((g.n_tokens + chunk - 1) / chunk);
  const bool vec = rows_of_16_bytes(g.logits, g.n_experts) && rows_of_16_bytes(g.d_logits, g.n_experts) &&
                   rows_of_16_bytes(g.counts, g.n_experts);
  by_experts(g.n_experts, vec, [&](auto lanes, auto slots, auto v) {
    constexpr int kL = decltype(lanes)::value, kR = decltype(slots)::value;
    constexpr bool kV = decltype(v)::value;
    if (g.accumulate) balance_backward_kernel<kL, kR, kV, true><<<blocks, kBlock, 0, stream>>>(a);
    else balance_backward_kernel<kL, kR, kV, false><<<blocks, kBlock, 0, stream>>>(a);
  });
  return hipGetLastError();
}

}  // namespace moe
