// C ABI of libmoe_dc: argument checking, mode resolution, workspace sizing and
// error reporting.  Every check runs on the host before any HIP call, so a
// rejected call touches no device state.
#include "../../include/moe_dc.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>

#include "launch.hpp"

namespace {

thread_local std::string g_last_error;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

int ok() {
  g_last_error.clear();
  return MOE_OK;
}

int hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

bool validate_mode() {
  const char* v = std::getenv("MOE_DC_VALIDATE");
  return v && v[0] == '1';
}

// Test hook: MOE_DC_SPIN_LIMIT=<n> caps the polls of a copy wave that waits for
// positions of its own launch (so tests can force the give-up path); unset or
// malformed: the library default.
int spin_limit() {
  const char* v = std::getenv("MOE_DC_SPIN_LIMIT");
  if (!v || !*v) return -1;
  char* end = nullptr;
  const long n = std::strtol(v, &end, 10);
  return (end && *end == '\0' && n >= 0 && n < (1L << 30)) ? int(n) : -1;
}

int check_routing_sizes(const char* fn, int64_t n_tokens, int32_t n_experts, int32_t k) {
  if (n_tokens < 0) return fail(MOE_ERR_ARG, "%s: n_tokens < 0", fn);
  if (n_experts < 1) return fail(MOE_ERR_ARG, "%s: n_experts < 1", fn);
  if (k < 1 || k > n_experts) return fail(MOE_ERR_ARG, "%s: need 1 <= k <= n_experts (k=%d, E=%d)", fn, k, n_experts);
  if (n_experts > MOE_MAX_EXPERTS) return fail(MOE_ERR_UNSUPPORTED, "%s: n_experts > %d", fn, MOE_MAX_EXPERTS);
  if (k > MOE_MAX_TOPK) return fail(MOE_ERR_UNSUPPORTED, "%s: k > %d", fn, MOE_MAX_TOPK);
  if (n_tokens > 0 && n_tokens * int64_t(k) > INT32_MAX)
    return fail(MOE_ERR_UNSUPPORTED, "%s: n_tokens * k exceeds the int32 index range", fn);
  return MOE_OK;
}

int resolve_sorted(int32_t sort, int64_t n_tokens, int32_t cutoff, int32_t* out) {
  if (sort == MOE_SORT_ON) { *out = 1; return MOE_OK; }
  if (sort == MOE_SORT_OFF) { *out = 0; return MOE_OK; }
  if (sort != MOE_SORT_AUTO) return fail(MOE_ERR_ARG, "sort must be -1, 0 or 1 (got %d)", sort);
  if (cutoff <= 0) { *out = 1; return MOE_OK; }
  // (M - 1) // cutoff >= 1  <=>  M > cutoff, for M >= 1
  *out = n_tokens > cutoff ? 1 : 0;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_abi_version(void) { return MOE_DC_ABI_VERSION; }

const char* moe_last_error(void) { return g_last_error.c_str(); }

int moe_resolve_sorted(int32_t sort, int64_t n_tokens, int32_t sort_cutoff, int32_t* sorted_out) {
  if (!sorted_out) return fail(MOE_ERR_ARG, "moe_resolve_sorted: sorted_out is null");
  if (n_tokens < 0) return fail(MOE_ERR_ARG, "moe_resolve_sorted: n_tokens < 0");
  const int rc = resolve_sorted(sort, n_tokens, sort_cutoff, sorted_out);
  return rc == MOE_OK ? ok() : rc;
}

int moe_route_topk(const float* logits, int64_t n_tokens, int32_t n_experts, int32_t k,
                   int32_t renormalize, int32_t* topk_idx, float* topk_w, void* stream) {
  const char* fn = "moe_route_topk";
  int rc = check_routing_sizes(fn, n_tokens, n_experts, k);
  if (rc) return rc;
  if (n_tokens == 0) return ok();
  if (!logits || !topk_idx || !topk_w) return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  return hip_status(moe::launch_route_topk(logits, n_tokens, n_experts, k, renormalize ? 1 : 0,
                                           topk_idx, topk_w, static_cast<hipStream_t>(stream)),
                    fn);
}

size_t moe_dispatch_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t k,
                                    int32_t n_segments) {
  if (n_tokens < 0 || n_experts < 1 || n_experts > MOE_MAX_EXPERTS || k < 1 || k > n_experts ||
      k > MOE_MAX_TOPK || n_segments < 1 || n_experts % n_segments != 0 ||
      n_tokens * int64_t(k) > INT32_MAX)
    return 0;
  return moe::dispatch_workspace_bytes(n_tokens, n_experts, k, n_segments);
}

}  // extern "C"

namespace {

// Shared argument checking and packing of moe_dispatch / moe_route_dispatch.
// Returns MOE_OK and fills `a` (and `sorted`) or returns the error status.
int prepare_dispatch(const char* fn, const void* x, const float* x_scales, int32_t dtype,
                     int64_t n_tokens, int64_t hidden, const int32_t* topk_idx, int32_t n_experts,
                     int32_t k, int32_t n_segments, int32_t sort, int32_t sort_cutoff, void* rows,
                     float* row_scales, int32_t* expert_counts, int32_t* expert_offsets,
                     int32_t* segment_offsets, int32_t* src_pair, int32_t* dst_pos,
                     int32_t* row_expert, void* workspace, size_t workspace_bytes, size_t need,
                     moe::DispatchArgs& a) {
  int rc = check_routing_sizes(fn, n_tokens, n_experts, k);
  if (rc) return rc;
  if (hidden < 1) return fail(MOE_ERR_ARG, "%s: hidden < 1", fn);
  if (n_segments < 1 || n_experts % n_segments != 0)
    return fail(MOE_ERR_ARG, "%s: n_segments must divide n_experts (E=%d, G=%d)", fn, n_experts, n_segments);
  int64_t elem = 0;
  switch (dtype) {
    case MOE_F32: elem = 4; break;
    case MOE_BF16: elem = 2; break;
    case MOE_F8E4M3: elem = 1; break;
    default: return fail(MOE_ERR_ARG, "%s: unknown dtype %d", fn, dtype);
  }
  if ((x == nullptr) != (rows == nullptr))
    return fail(MOE_ERR_ARG, "%s: x and rows must both be given or both be null", fn);
  if (dtype == MOE_F8E4M3) {
    if (hidden % 128 != 0) return fail(MOE_ERR_ARG, "%s: F8 payload needs hidden %% 128 == 0", fn);
    if (x && (!x_scales || !row_scales))
      return fail(MOE_ERR_ARG, "%s: F8 payload needs x_scales and row_scales", fn);
  } else if (x_scales || row_scales) {
    return fail(MOE_ERR_ARG, "%s: block scales are only for the F8 payload", fn);
  }
  if (!x && (x_scales || row_scales))
    return fail(MOE_ERR_ARG, "%s: scales given without a payload", fn);
  if (!expert_counts || !expert_offsets || !segment_offsets)
    return fail(MOE_ERR_ARG, "%s: null offsets/counts output", fn);
  if (n_tokens > 0 && (!topk_idx || !src_pair || !dst_pos))
    return fail(MOE_ERR_ARG, "%s: null index input or map output", fn);
  int32_t sorted = 0;
  rc = resolve_sorted(sort, n_tokens, sort_cutoff, &sorted);
  if (rc) return rc;
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? workspace_bytes : size_t(0));
  if (reinterpret_cast<uintptr_t>(workspace) & 15)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace must be 16-byte aligned", fn);
  a = moe::DispatchArgs{};
  a.x = x;
  a.x_scales = x_scales;
  a.row_bytes = hidden * elem;
  a.scale_bytes = dtype == MOE_F8E4M3 ? hidden / 128 * 4 : 0;
  a.n_tokens = n_tokens;
  a.topk_idx = topk_idx;
  a.n_experts = n_experts;
  a.k = k;
  a.n_segments = n_segments;
  a.sorted = sorted;
  a.rows = rows;
  a.row_scales = row_scales;
  a.expert_counts = expert_counts;
  a.expert_offsets = expert_offsets;
  a.segment_offsets = segment_offsets;
  a.src_pair = src_pair;
  a.dst_pos = dst_pos;
  a.row_expert = row_expert;
  a.workspace = workspace;
  a.spin_limit = spin_limit();
  return MOE_OK;
}

// Validate mode: clear the status word before the launches, then wait and
// report out-of-range expert ids.
int32_t* validate_begin(void* workspace, size_t need, hipStream_t s, int* rc, const char* fn) {
  int32_t* status = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + need - 16);
  hipError_t e = hipMemsetAsync(status, 0, sizeof(int32_t), s);
  *rc = e == hipSuccess ? MOE_OK : hip_status(e, fn);
  return status;
}

int validate_end(int32_t* status, hipStream_t s, int32_t n_experts, const char* fn) {
  int32_t host_status = 0;
  hipError_t e = hipMemcpyAsync(&host_status, status, sizeof(int32_t), hipMemcpyDeviceToHost, s);
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  if (e != hipSuccess) return hip_status(e, fn);
  if (host_status & 1) return fail(MOE_ERR_ARG, "%s: topk_idx holds expert ids outside [0, %d)", fn, n_experts);
  if (host_status & 2)
    return fail(MOE_ERR_HIP, "%s: the row copy gave up waiting for positions of its own launch", fn);
  return ok();
}

}  // namespace

extern "C" {

int moe_dispatch(const void* x, const float* x_scales, int32_t dtype, int64_t n_tokens,
                 int64_t hidden, const int32_t* topk_idx, int32_t n_experts, int32_t k,
                 int32_t n_segments, int32_t sort, int32_t sort_cutoff, int32_t* sorted_used,
                 void* rows, float* row_scales, int32_t* expert_counts, int32_t* expert_offsets,
                 int32_t* segment_offsets, int32_t* src_pair, int32_t* dst_pos,
                 int32_t* row_expert, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "moe_dispatch";
  const int early = check_routing_sizes(fn, n_tokens, n_experts, k);
  if (early) return early;
  const size_t need = moe::dispatch_workspace_bytes(n_tokens, n_experts, k, n_segments > 0 ? n_segments : 1);
  moe::DispatchArgs a;
  int rc = prepare_dispatch(fn, x, x_scales, dtype, n_tokens, hidden, topk_idx, n_experts, k,
                            n_segments, sort, sort_cutoff, rows, row_scales, expert_counts,
                            expert_offsets, segment_offsets, src_pair, dst_pos, row_expert,
                            workspace, workspace_bytes, need, a);
  if (rc) return rc;
  if (sorted_used) *sorted_used = a.sorted;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool validate = validate_mode();
  if (validate) {
    a.status = validate_begin(workspace, need, s, &rc, fn);
    if (rc) return rc;
  }
  rc = hip_status(moe::launch_dispatch(a, s), fn);
  if (rc || !validate) return rc;
  return validate_end(a.status, s, n_experts, fn);
}

size_t moe_route_dispatch_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t k,
                                          int32_t n_segments) {
  if (moe_dispatch_workspace_bytes(n_tokens, n_experts, k, n_segments) == 0) return 0;
  return moe::route_dispatch_workspace_bytes(n_tokens, n_experts, k, n_segments);
}

}  // extern "C"

namespace {

// moe_route_dispatch and its allocation-free variant: the same checks and
// launches; `workspace` is the caller's buffer or the static scratch.
int route_dispatch_impl(const char* fn, const float* logits, int32_t renormalize,
                        int32_t* topk_idx, float* topk_w, const void* x, const float* x_scales,
                        int32_t dtype, int64_t n_tokens, int64_t hidden, int32_t n_experts,
                        int32_t k, int32_t n_segments, int32_t sort, int32_t sort_cutoff,
                        int32_t* sorted_used, void* rows, float* row_scales,
                        int32_t* expert_counts, int32_t* expert_offsets,
                        int32_t* segment_offsets, int32_t* src_pair, int32_t* dst_pos,
                        int32_t* row_expert, void* workspace, size_t workspace_bytes,
                        void* stream, bool static_scratch) {
  const int early = check_routing_sizes(fn, n_tokens, n_experts, k);
  if (early) return early;
  if (n_tokens > 0 && (!logits || !topk_idx || !topk_w))
    return fail(MOE_ERR_ARG, "%s: null routing pointer", fn);
  const size_t need = moe::route_dispatch_workspace_bytes(n_tokens, n_experts, k, n_segments > 0 ? n_segments : 1);
  if (static_scratch && need > MOE_NOALLOC_SCRATCH_BYTES)
    return fail(MOE_ERR_UNSUPPORTED,
                "%s: these sizes need %zu bytes of scratch, more than the %zu-byte static array "
                "(use moe_route_dispatch with a workspace)",
                fn, need, size_t(MOE_NOALLOC_SCRATCH_BYTES));
  // every argument is checked before the scratch is looked up, so a rejected
  // call touches no device state (a placeholder address stands in for it)
  moe::DispatchArgs a;
  int rc = prepare_dispatch(fn, x, x_scales, dtype, n_tokens, hidden, topk_idx, n_experts, k,
                            n_segments, sort, sort_cutoff, rows, row_scales, expert_counts,
                            expert_offsets, segment_offsets, src_pair, dst_pos, row_expert,
                            static_scratch ? reinterpret_cast<void*>(uintptr_t(256)) : workspace,
                            static_scratch ? size_t(MOE_NOALLOC_SCRATCH_BYTES) : workspace_bytes,
                            need, a);
  if (rc) return rc;
  if (static_scratch) {
    const hipError_t e = moe::noalloc_scratch(static_cast<hipStream_t>(stream), &a.workspace);
    if (e != hipSuccess) return hip_status(e, fn);
  }
  if (sorted_used) *sorted_used = a.sorted;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  // validate mode: moe_route_dispatch only (its host copy and wait have no
  // place in the allocation-free variant)
  const bool validate = !static_scratch && validate_mode();
  if (validate) {
    a.status = validate_begin(workspace, need, s, &rc, fn);
    if (rc) return rc;
  }
  moe::RouteArgs r{logits, renormalize ? 1 : 0, topk_w};
  rc = hip_status(moe::launch_route_dispatch(r, a, s), fn);
  if (rc || !validate) return rc;
  return validate_end(a.status, s, n_experts, fn);
}

}  // namespace

extern "C" {

int moe_route_dispatch(const float* logits, int32_t renormalize, int32_t* topk_idx, float* topk_w,
                       const void* x, const float* x_scales, int32_t dtype, int64_t n_tokens,
                       int64_t hidden, int32_t n_experts, int32_t k, int32_t n_segments,
                       int32_t sort, int32_t sort_cutoff, int32_t* sorted_used, void* rows,
                       float* row_scales, int32_t* expert_counts, int32_t* expert_offsets,
                       int32_t* segment_offsets, int32_t* src_pair, int32_t* dst_pos,
                       int32_t* row_expert, void* workspace, size_t workspace_bytes,
                       void* stream) {
  return route_dispatch_impl("moe_route_dispatch", logits, renormalize, topk_idx, topk_w, x,
                             x_scales, dtype, n_tokens, hidden, n_experts, k, n_segments, sort,
                             sort_cutoff, sorted_used, rows, row_scales, expert_counts,
                             expert_offsets, segment_offsets, src_pair, dst_pos, row_expert,
                             workspace, workspace_bytes, stream, false);
}

int moe_route_dispatch_noalloc(const float* logits, int32_t renormalize, int32_t* topk_idx,
                               float* topk_w, const void* x, const float* x_scales, int32_t dtype,
                               int64_t n_tokens, int64_t hidden, int32_t n_experts, int32_t k,
                               int32_t n_segments, int32_t sort, int32_t sort_cutoff,
                               int32_t* sorted_used, void* rows, float* row_scales,
                               int32_t* expert_counts, int32_t* expert_offsets,
                               int32_t* segment_offsets, int32_t* src_pair, int32_t* dst_pos,
                               int32_t* row_expert, void* stream) {
  return route_dispatch_impl("moe_route_dispatch_noalloc", logits, renormalize, topk_idx, topk_w,
                             x, x_scales, dtype, n_tokens, hidden, n_experts, k, n_segments, sort,
                             sort_cutoff, sorted_used, rows, row_scales, expert_counts,
                             expert_offsets, segment_offsets, src_pair, dst_pos, row_expert,
                             nullptr, 0, stream, true);
}

int moe_scatter_rows(const void* x, int64_t n_tokens, int64_t row_bytes, int32_t k,
                     const int32_t* dst_pos, void* rows, void* stream) {
  const char* fn = "moe_scatter_rows";
  if (n_tokens < 0 || row_bytes < 1 || k < 1) return fail(MOE_ERR_ARG, "%s: need n_tokens >= 0, row_bytes >= 1, k >= 1", fn);
  // one lane of a wave holds each of a token's k destinations
  if (k > MOE_MAX_TOPK) return fail(MOE_ERR_UNSUPPORTED, "%s: k > %d", fn, MOE_MAX_TOPK);
  if (n_tokens * int64_t(k) > INT32_MAX)
    return fail(MOE_ERR_UNSUPPORTED, "%s: n_tokens * k exceeds the int32 index range", fn);
  if (n_tokens == 0) return ok();
  if (!x || !dst_pos || !rows) return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  return hip_status(moe::launch_scatter_rows(x, n_tokens, row_bytes, k, dst_pos, rows,
                                             static_cast<hipStream_t>(stream)),
                    fn);
}

int moe_gather_rows(const void* x, int64_t n_tokens, int64_t row_bytes, int32_t k,
                    const int32_t* src_pair, int64_t n_rows, void* rows, void* stream) {
  const char* fn = "moe_gather_rows";
  if (n_tokens < 0 || n_rows < 0 || row_bytes < 1 || k < 1)
    return fail(MOE_ERR_ARG, "%s: need n_tokens, n_rows >= 0, row_bytes >= 1, k >= 1", fn);
  if (n_tokens * int64_t(k) > INT32_MAX || n_rows > INT32_MAX)
    return fail(MOE_ERR_UNSUPPORTED, "%s: sizes exceed the int32 index range", fn);
  if (n_rows == 0) return ok();
  if (!x || !src_pair || !rows) return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  return hip_status(moe::launch_gather_rows(x, n_tokens, row_bytes, k, src_pair, n_rows, rows,
                                            static_cast<hipStream_t>(stream)),
                    fn);
}

int moe_combine(const void* y, int32_t y_dtype, int64_t n_tokens, int64_t hidden, int32_t k,
                const int32_t* dst_pos, const float* topk_w, void* out, int32_t out_dtype,
                void* stream) {
  const char* fn = "moe_combine";
  if (n_tokens < 0) return fail(MOE_ERR_ARG, "%s: n_tokens < 0", fn);
  if (hidden < 1) return fail(MOE_ERR_ARG, "%s: hidden < 1", fn);
  if (k < 1) return fail(MOE_ERR_ARG, "%s: k < 1", fn);
  if (k > MOE_MAX_TOPK) return fail(MOE_ERR_UNSUPPORTED, "%s: k > %d", fn, MOE_MAX_TOPK);
  if ((y_dtype != MOE_F32 && y_dtype != MOE_BF16) || (out_dtype != MOE_F32 && out_dtype != MOE_BF16))
    return fail(MOE_ERR_ARG, "%s: y and out must be MOE_F32 or MOE_BF16", fn);
  if (n_tokens * int64_t(k) > INT32_MAX)
    return fail(MOE_ERR_UNSUPPORTED, "%s: n_tokens * k exceeds the int32 index range", fn);
  if (n_tokens == 0) return ok();
  if (!y || !dst_pos || !topk_w || !out) return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  return hip_status(moe::launch_combine(y, y_dtype == MOE_BF16, n_tokens, hidden, k, dst_pos,
                                        topk_w, out, out_dtype == MOE_BF16,
                                        static_cast<hipStream_t>(stream)),
                    fn);
}

namespace {
// sizes of the [NK, D] row gradients and the alignment of their elements
int check_row_gradient(const char* fn, int64_t n_tokens, int64_t hidden, int32_t k, int32_t dt_a,
                       int32_t dt_b) {
  if (n_tokens < 0) return fail(MOE_ERR_ARG, "%s: n_tokens < 0", fn);
  if (hidden < 1) return fail(MOE_ERR_ARG, "%s: hidden < 1", fn);
  if (k < 1) return fail(MOE_ERR_ARG, "%s: k < 1", fn);
  if ((dt_a != MOE_F32 && dt_a != MOE_BF16) || (dt_b != MOE_F32 && dt_b != MOE_BF16))
    return fail(MOE_ERR_ARG, "%s: dtypes must be MOE_F32 or MOE_BF16", fn);
  if (k > MOE_MAX_TOPK) return fail(MOE_ERR_UNSUPPORTED, "%s: k > %d", fn, MOE_MAX_TOPK);
  if (n_tokens > INT32_MAX / k)
    return fail(MOE_ERR_UNSUPPORTED, "%s: n_tokens * k exceeds the int32 index range", fn);
  return MOE_OK;
}
bool misaligned(const void* p, int32_t dtype) {
  return reinterpret_cast<uintptr_t>(p) & (dtype == MOE_F32 ? 3 : 1);
}
bool misaligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) & 3; }
}  // namespace

int moe_combine_backward(const void* d_out, int32_t g_dtype, const void* y, int32_t y_dtype,
                         int64_t n_tokens, int64_t hidden, int32_t k, const int32_t* dst_pos,
                         const float* topk_w, void* d_y, float* d_topk_w, void* stream) {
  const char* fn = "moe_combine_backward";
  const int rc = check_row_gradient(fn, n_tokens, hidden, k, g_dtype, y_dtype);
  if (rc) return rc;
  if (n_tokens == 0) return ok();
  if (!d_out || !y || !dst_pos || !topk_w || !d_y || !d_topk_w)
    return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  if (misaligned(d_out, g_dtype) || misaligned(y, y_dtype) || misaligned(d_y, y_dtype) ||
      misaligned4(dst_pos) || misaligned4(topk_w) || misaligned4(d_topk_w))
    return fail(MOE_ERR_ARG, "%s: pointers must be aligned to their elements", fn);
  return hip_status(moe::launch_combine_backward(d_out, g_dtype == MOE_BF16, y, y_dtype == MOE_BF16,
                                                 n_tokens, hidden, k, dst_pos, topk_w, d_y,
                                                 d_topk_w, static_cast<hipStream_t>(stream)),
                    fn);
}

int moe_dispatch_backward(const void* d_rows, int32_t rows_dtype, int64_t n_tokens, int64_t hidden,
                          int32_t k, const int32_t* dst_pos, void* d_x, int32_t x_dtype,
                          void* stream) {
  const char* fn = "moe_dispatch_backward";
  const int rc = check_row_gradient(fn, n_tokens, hidden, k, rows_dtype, x_dtype);
  if (rc) return rc;
  if (n_tokens == 0) return ok();
  if (!d_rows || !dst_pos || !d_x) return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  if (misaligned(d_rows, rows_dtype) || misaligned(d_x, x_dtype) || misaligned4(dst_pos))
    return fail(MOE_ERR_ARG, "%s: pointers must be aligned to their elements", fn);
  return hip_status(moe::launch_dispatch_backward(d_rows, rows_dtype == MOE_BF16, n_tokens, hidden,
                                                  k, dst_pos, d_x, x_dtype == MOE_BF16,
                                                  static_cast<hipStream_t>(stream)),
                    fn);
}

int moe_route_topk_backward(const float* logits, const int32_t* topk_idx, const float* topk_w,
                            const float* d_topk_w, int64_t n_tokens, int32_t n_experts, int32_t k,
                            int32_t renormalize, float* d_logits, void* stream) {
  const char* fn = "moe_route_topk_backward";
  const int rc = check_routing_sizes(fn, n_tokens, n_experts, k);
  if (rc) return rc;
  if (n_tokens == 0) return ok();
  if (!topk_idx || !topk_w || !d_topk_w || !d_logits || (!renormalize && !logits))
    return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  if (misaligned4(logits) || misaligned4(topk_idx) || misaligned4(topk_w) ||
      misaligned4(d_topk_w) || misaligned4(d_logits))
    return fail(MOE_ERR_ARG, "%s: pointers must be aligned to their elements", fn);
  return hip_status(moe::launch_route_topk_backward(logits, topk_idx, topk_w, d_topk_w, n_tokens,
                                                    n_experts, k, renormalize ? 1 : 0, d_logits,
                                                    static_cast<hipStream_t>(stream)),
                    fn);
}

int moe_dequant_rows(const uint8_t* rows, const float* row_scales, int64_t n_rows, int64_t hidden,
                     uint16_t* y, void* stream) {
  const char* fn = "moe_dequant_rows";
  if (n_rows < 0) return fail(MOE_ERR_ARG, "%s: n_rows < 0", fn);
  if (hidden < 1 || hidden % 128 != 0) return fail(MOE_ERR_ARG, "%s: hidden must be a positive multiple of 128", fn);
  if (n_rows == 0) return ok();
  if (!rows || !row_scales || !y) return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  if ((reinterpret_cast<uintptr_t>(rows) | reinterpret_cast<uintptr_t>(y)) & 15)
    return fail(MOE_ERR_ARG, "%s: rows and y must be 16-byte aligned", fn);
  return hip_status(moe::launch_dequant_rows(rows, row_scales, n_rows, hidden, y,
                                             static_cast<hipStream_t>(stream)),
                    fn);
}

size_t moe_grouped_swiglu_workspace_bytes(int64_t n_rows, int32_t n_experts, int64_t hidden,
                                          int64_t ffn) {
  if (n_rows < 0 || n_experts < 1 || hidden < 1 || ffn < 1) return 0;
  return moe::grouped_swiglu_workspace_bytes(n_rows, n_experts, hidden, ffn);
}

int moe_grouped_swiglu(const void* rows, int64_t n_rows, int64_t hidden,
                       const int32_t* expert_offsets, int32_t n_experts, const void* w_gate,
                       const void* w_up, const void* w_down, int64_t ffn, void* y,
                       void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "moe_grouped_swiglu";
  if (n_rows < 0) return fail(MOE_ERR_ARG, "%s: n_rows < 0", fn);
  if (hidden < 1 || ffn < 1 || n_experts < 1) return fail(MOE_ERR_ARG, "%s: sizes must be >= 1", fn);
  if (n_experts > MOE_MAX_EXPERTS) return fail(MOE_ERR_UNSUPPORTED, "%s: n_experts > %d", fn, MOE_MAX_EXPERTS);
  if (hidden % 64 != 0 || ffn % 64 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: hidden and ffn must be multiples of 64", fn);
  if (n_rows > INT32_MAX) return fail(MOE_ERR_UNSUPPORTED, "%s: n_rows exceeds the int32 range", fn);
  // per-lane load offsets within a 256-row tile are 32-bit
  if (hidden > (int64_t(1) << 22) || ffn > (int64_t(1) << 22))
    return fail(MOE_ERR_UNSUPPORTED, "%s: hidden and ffn must be at most %d", fn, 1 << 22);
  // the grid also holds up to 256 extra workgroups for the split parts of the last round
  if (moe::grouped_swiglu_tiles(n_rows, n_experts, hidden, ffn) > INT32_MAX - 8 - 256)
    return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles", fn);
  if (n_rows == 0) return ok();
  if (!rows || !expert_offsets || !w_gate || !w_up || !w_down || !y)
    return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  // the operands are read in 16-byte runs straight into LDS
  if ((reinterpret_cast<uintptr_t>(rows) | reinterpret_cast<uintptr_t>(w_gate) |
       reinterpret_cast<uintptr_t>(w_up) | reinterpret_cast<uintptr_t>(w_down) |
       reinterpret_cast<uintptr_t>(y)) & 15)
    return fail(MOE_ERR_UNSUPPORTED, "%s: rows, weights and y must be 16-byte aligned", fn);
  const size_t need = moe::grouped_swiglu_workspace_bytes(n_rows, n_experts, hidden, ffn);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? workspace_bytes : size_t(0));
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", fn);
  return hip_status(moe::launch_grouped_swiglu(rows, n_rows, hidden, expert_offsets, n_experts,
                                               w_gate, w_up, w_down, ffn, y, workspace,
                                               static_cast<hipStream_t>(stream)),
                    fn);
}

size_t moe_gather_swiglu_workspace_bytes(int64_t n_rows, int32_t n_experts, int64_t hidden,
                                         int64_t ffn) {
  if (n_rows < 0 || n_rows > INT32_MAX || n_experts < 1 || n_experts > MOE_MAX_EXPERTS ||
      hidden < 1 || ffn < 1)
    return 0;
  return moe::gather_swiglu_workspace_bytes(n_rows, n_experts, hidden, ffn);
}

int moe_gather_swiglu(const void* rows, int64_t n_rows, int64_t hidden,
                      const int32_t* row_expert, int32_t n_experts, const void* w_gate,
                      const void* w_up, const void* w_down, int64_t ffn, void* y,
                      void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "moe_gather_swiglu";
  if (n_rows < 0) return fail(MOE_ERR_ARG, "%s: n_rows < 0", fn);
  if (hidden < 1 || ffn < 1 || n_experts < 1) return fail(MOE_ERR_ARG, "%s: sizes must be >= 1", fn);
  if (n_experts > MOE_MAX_EXPERTS) return fail(MOE_ERR_UNSUPPORTED, "%s: n_experts > %d", fn, MOE_MAX_EXPERTS);
  if (hidden % 128 != 0 || ffn % 128 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: hidden and ffn must be multiples of 128", fn);
  if (n_rows > INT32_MAX || hidden > INT32_MAX || ffn > INT32_MAX)
    return fail(MOE_ERR_UNSUPPORTED, "%s: sizes exceed the int32 range", fn);
  if (moe::gather_swiglu_tiles(n_rows, n_experts, hidden, ffn) > INT32_MAX - 8)
    return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles", fn);
  if (n_rows == 0) return ok();
  if (!rows || !row_expert || !w_gate || !w_up || !w_down || !y)
    return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  // rows and weights are read in 16-byte runs; y is written element by element
  if ((reinterpret_cast<uintptr_t>(rows) | reinterpret_cast<uintptr_t>(w_gate) |
       reinterpret_cast<uintptr_t>(w_up) | reinterpret_cast<uintptr_t>(w_down)) & 15)
    return fail(MOE_ERR_UNSUPPORTED, "%s: rows and weights must be 16-byte aligned", fn);
  if (reinterpret_cast<uintptr_t>(y) & 1)
    return fail(MOE_ERR_UNSUPPORTED, "%s: y must be 2-byte aligned", fn);
  const size_t need = moe::gather_swiglu_workspace_bytes(n_rows, n_experts, hidden, ffn);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? workspace_bytes : size_t(0));
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", fn);
  return hip_status(moe::launch_gather_swiglu(rows, n_rows, hidden, row_expert, n_experts,
                                              w_gate, w_up, w_down, ffn, y, workspace,
                                              static_cast<hipStream_t>(stream)),
                    fn);
}

int moe_gather_swiglu_combine(const void* rows, int64_t n_rows, int64_t hidden,
                              const int32_t* row_expert, const int32_t* row_pair,
                              const float* topk_w, int64_t n_tokens, int32_t k, int32_t n_experts,
                              const void* w_gate, const void* w_up, const void* w_down,
                              int64_t ffn, float* out, void* workspace, size_t workspace_bytes,
                              void* stream) {
  const char* fn = "moe_gather_swiglu_combine";
  if (n_rows < 0 || n_tokens < 0) return fail(MOE_ERR_ARG, "%s: n_rows and n_tokens must be >= 0", fn);
  if (hidden < 1 || ffn < 1 || n_experts < 1) return fail(MOE_ERR_ARG, "%s: sizes must be >= 1", fn);
  if (k < 1 || k > moe::kMaxTopK) return fail(MOE_ERR_ARG, "%s: k must be in [1, %d]", fn, moe::kMaxTopK);
  if (n_experts > MOE_MAX_EXPERTS) return fail(MOE_ERR_UNSUPPORTED, "%s: n_experts > %d", fn, MOE_MAX_EXPERTS);
  if (hidden % 128 != 0 || ffn % 128 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: hidden and ffn must be multiples of 128", fn);
  if (n_rows > INT32_MAX || hidden > INT32_MAX || ffn > INT32_MAX || n_tokens * k > INT32_MAX)
    return fail(MOE_ERR_UNSUPPORTED, "%s: sizes exceed the int32 range", fn);
  if (moe::gather_swiglu_tiles(n_rows, n_experts, hidden, ffn) > INT32_MAX - 8)
    return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles", fn);
  if (n_rows == 0 || n_tokens == 0) return ok();
  if (!rows || !row_expert || !topk_w || !w_gate || !w_up || !w_down || !out)
    return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  if ((reinterpret_cast<uintptr_t>(rows) | reinterpret_cast<uintptr_t>(w_gate) |
       reinterpret_cast<uintptr_t>(w_up) | reinterpret_cast<uintptr_t>(w_down)) & 15)
    return fail(MOE_ERR_UNSUPPORTED, "%s: rows and weights must be 16-byte aligned", fn);
  if ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(topk_w)) & 3)
    return fail(MOE_ERR_UNSUPPORTED, "%s: out and topk_w must be 4-byte aligned", fn);
  const size_t need = moe::gather_swiglu_workspace_bytes(n_rows, n_experts, hidden, ffn);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? workspace_bytes : size_t(0));
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", fn);
  const moe::FusedCombine fc{row_pair, topk_w, out, int(k), int(n_tokens * k)};
  return hip_status(moe::launch_gather_swiglu(rows, n_rows, hidden, row_expert, n_experts,
                                              w_gate, w_up, w_down, ffn, nullptr, workspace,
                                              static_cast<hipStream_t>(stream), &fc),
                    fn);
}

int moe_grouped_gemm_fp8(const void* rows, const float* row_scales, int64_t n_rows,
                         int64_t k_dim, const int32_t* expert_offsets, int32_t n_experts,
                         const void* w, const float* w_scales, int64_t n_dim, void* y,
                         void* stream) {
  const char* fn = "moe_grouped_gemm_fp8";
  if (n_rows < 0) return fail(MOE_ERR_ARG, "%s: n_rows < 0", fn);
  if (k_dim < 1 || n_dim < 1 || n_experts < 1) return fail(MOE_ERR_ARG, "%s: sizes must be >= 1", fn);
  if (n_experts > MOE_MAX_EXPERTS) return fail(MOE_ERR_UNSUPPORTED, "%s: n_experts > %d", fn, MOE_MAX_EXPERTS);
  if (k_dim % 128 != 0 || n_dim % 128 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: k_dim and n_dim must be multiples of 128", fn);
  if (n_rows > INT32_MAX || n_dim > INT32_MAX || k_dim > INT32_MAX)
    return fail(MOE_ERR_UNSUPPORTED, "%s: sizes exceed the int32 range", fn);
  const int64_t tiles = ((n_rows + 63) / 64 + n_experts + 7) / 8 * 8 * (n_dim / 128);
  if (tiles > INT32_MAX - 8) return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles", fn);
  if (n_rows == 0) return ok();
  if (!rows || !row_scales || !expert_offsets || !w || !w_scales || !y)
    return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  // operands are read in 16-byte runs; scales as 4-byte words
  if ((reinterpret_cast<uintptr_t>(rows) | reinterpret_cast<uintptr_t>(w) |
       reinterpret_cast<uintptr_t>(y)) & 15)
    return fail(MOE_ERR_UNSUPPORTED, "%s: rows, w and y must be 16-byte aligned", fn);
  if ((reinterpret_cast<uintptr_t>(row_scales) | reinterpret_cast<uintptr_t>(w_scales)) & 3)
    return fail(MOE_ERR_ARG, "%s: scales must be 4-byte aligned", fn);
  return hip_status(moe::launch_grouped_gemm_fp8(rows, row_scales, n_rows, k_dim, expert_offsets,
                                                 n_experts, w, w_scales, n_dim, y,
                                                 static_cast<hipStream_t>(stream)),
                    fn);
}

namespace {
bool off(const void* p, unsigned align) { return reinterpret_cast<uintptr_t>(p) & (align - 1); }

int check_mxfp4_rows(const char* fn, int32_t dtype, int64_t n_rows, int64_t k_dim) {
  if (n_rows < 0) return fail(MOE_ERR_ARG, "%s: n_rows < 0", fn);
  if (k_dim < 1) return fail(MOE_ERR_ARG, "%s: k_dim < 1", fn);
  if (dtype != MOE_F32 && dtype != MOE_BF16)
    return fail(MOE_ERR_ARG, "%s: dtype must be MOE_F32 or MOE_BF16", fn);
  if (k_dim % 32 != 0) return fail(MOE_ERR_UNSUPPORTED, "%s: k_dim must be a multiple of 32", fn);
  if (n_rows > (int64_t(1) << 40) / k_dim)
    return fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^40 elements", fn);
  return MOE_OK;
}

int check_mxfp4_product(const char* fn, const moe::Mxfp4Product& g, const void* index, bool gather) {
  if (g.n_rows < 0) return fail(MOE_ERR_ARG, "%s: n_rows < 0", fn);
  if (g.k_dim < 1 || g.n_dim < 1 || g.n_experts < 1) return fail(MOE_ERR_ARG, "%s: sizes must be >= 1", fn);
  if (!g.w_up != !g.w_up_scales)
    return fail(MOE_ERR_ARG, "%s: w_up and w_up_scales go together", fn);
  if (g.n_experts > MOE_MAX_EXPERTS) return fail(MOE_ERR_UNSUPPORTED, "%s: n_experts > %d", fn, MOE_MAX_EXPERTS);
  if (g.k_dim % 128 != 0) return fail(MOE_ERR_UNSUPPORTED, "%s: k_dim must be a multiple of 128", fn);
  // per-lane load offsets within a tile are 32-bit
  if (g.k_dim > (int64_t(1) << 22) || g.n_dim > (int64_t(1) << 22))
    return fail(MOE_ERR_UNSUPPORTED, "%s: k_dim and n_dim must be at most %d", fn, 1 << 22);
  if (g.n_rows > INT32_MAX) return fail(MOE_ERR_UNSUPPORTED, "%s: n_rows exceeds the int32 range", fn);
  if (g.n_rows > 0 && moe::gemm_mxfp4_blocks(g, gather) > moe::kMaxMxfp4Blocks)
    return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles", fn);
  if (g.n_rows == 0) return MOE_OK;
  if (!g.rows || !g.row_scales || !index || !g.w || !g.w_scales || !g.y)
    return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  if (off(g.rows, 16) || off(g.w, 16) || off(g.w_up, 16) || off(g.y, 16))
    return fail(MOE_ERR_UNSUPPORTED, "%s: rows, weights and y must be 16-byte aligned", fn);
  if (off(g.row_scales, 4) || off(g.w_scales, 4) || off(g.w_up_scales, 4) || off(index, 4))
    return fail(MOE_ERR_UNSUPPORTED, "%s: scales and indices must be 4-byte aligned", fn);
  return MOE_OK;
}
}  // namespace

int moe_quantize_mxfp4(const void* x, int32_t x_dtype, int64_t n_rows, int64_t k_dim,
                       uint8_t* codes, uint8_t* scales, void* stream) {
  const char* fn = "moe_quantize_mxfp4";
  const int rc = check_mxfp4_rows(fn, x_dtype, n_rows, k_dim);
  if (rc) return rc;
  if (n_rows == 0) return ok();
  if (!x || !codes || !scales) return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  if (off(x, 16) || off(codes, 4))
    return fail(MOE_ERR_UNSUPPORTED, "%s: x must be 16-byte and codes 4-byte aligned", fn);
  return hip_status(moe::launch_quantize_mxfp4(x, x_dtype == MOE_BF16, n_rows * k_dim, codes, scales,
                                               static_cast<hipStream_t>(stream)),
                    fn);
}

int moe_dequant_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t n_rows, int64_t k_dim,
                      void* out, int32_t out_dtype, void* stream) {
  const char* fn = "moe_dequant_mxfp4";
  const int rc = check_mxfp4_rows(fn, out_dtype, n_rows, k_dim);
  if (rc) return rc;
  if (n_rows == 0) return ok();
  if (!codes || !scales || !out) return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  if (off(out, 16) || off(codes, 4))
    return fail(MOE_ERR_UNSUPPORTED, "%s: out must be 16-byte and codes 4-byte aligned", fn);
  return hip_status(moe::launch_dequant_mxfp4(codes, scales, n_rows * k_dim, out,
                                              out_dtype == MOE_BF16, static_cast<hipStream_t>(stream)),
                    fn);
}

int moe_grouped_gemm_mxfp4(const uint8_t* rows, const uint8_t* row_scales, int64_t n_rows,
                           int64_t k_dim, const int32_t* expert_offsets, int32_t n_experts,
                           const uint8_t* w, const uint8_t* w_scales, const uint8_t* w_up,
                           const uint8_t* w_up_scales, int64_t n_dim, void* y, void* stream) {
  const char* fn = "moe_grouped_gemm_mxfp4";
  const moe::Mxfp4Product g{rows, row_scales, n_rows, k_dim, n_experts, w, w_scales,
                            w_up, w_up_scales, n_dim, y};
  const int rc = check_mxfp4_product(fn, g, expert_offsets, false);
  if (rc) return rc;
  if (n_rows == 0) return ok();
  return hip_status(moe::launch_grouped_gemm_mxfp4(g, expert_offsets, static_cast<hipStream_t>(stream)),
                    fn);
}

size_t moe_gather_gemm_mxfp4_workspace_bytes(int64_t n_rows, int32_t n_experts) {
  if (n_rows < 0 || n_rows > INT32_MAX || n_experts < 1 || n_experts > MOE_MAX_EXPERTS) return 0;
  return moe::gather_gemm_mxfp4_workspace_bytes(n_rows, n_experts);
}

int moe_gather_gemm_mxfp4(const uint8_t* rows, const uint8_t* row_scales, int64_t n_rows,
                          int64_t k_dim, const int32_t* row_expert, int32_t n_experts,
                          const uint8_t* w, const uint8_t* w_scales, const uint8_t* w_up,
                          const uint8_t* w_up_scales, int64_t n_dim, void* y, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const char* fn = "moe_gather_gemm_mxfp4";
  const moe::Mxfp4Product g{rows, row_scales, n_rows, k_dim, n_experts, w, w_scales,
                            w_up, w_up_scales, n_dim, y};
  const int rc = check_mxfp4_product(fn, g, row_expert, true);
  if (rc) return rc;
  if (n_rows == 0) return ok();
  const size_t need = moe::gather_gemm_mxfp4_workspace_bytes(n_rows, n_experts);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? workspace_bytes : size_t(0));
  if (off(workspace, 256))
    return fail(MOE_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", fn);
  return hip_status(moe::launch_gather_gemm_mxfp4(g, row_expert, workspace, static_cast<hipStream_t>(stream)),
                    fn);
}

size_t moe_balance_loss_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t n_sequences) {
  if (n_tokens < 0 || n_tokens > INT32_MAX || n_experts < 1 || n_experts > MOE_MAX_EXPERTS ||
      n_sequences < 1 || n_sequences > MOE_MAX_SEQUENCES)
    return 0;
  return moe::balance_workspace_bytes(n_tokens, n_experts, n_sequences);
}

namespace {
int check_balance(const char* fn, int64_t n_tokens, int32_t n_experts, int32_t k,
                  const int32_t* seq_offsets, int32_t n_sequences) {
  const int rc = check_routing_sizes(fn, n_tokens, n_experts, k);
  if (rc) return rc;
  if (n_sequences < 1) return fail(MOE_ERR_ARG, "%s: n_sequences < 1", fn);
  if (n_sequences > MOE_MAX_SEQUENCES)
    return fail(MOE_ERR_UNSUPPORTED, "%s: n_sequences > %d", fn, MOE_MAX_SEQUENCES);
  if (!seq_offsets && n_sequences != 1)
    return fail(MOE_ERR_ARG, "%s: %d sequences need seq_offsets", fn, n_sequences);
  return MOE_OK;
}
}  // namespace

int moe_balance_loss(const float* logits, const int32_t* topk_idx, int64_t n_tokens,
                     int32_t n_experts, int32_t k, const int32_t* seq_offsets, int32_t n_sequences,
                     const uint8_t* token_mask, float* loss, float* z_loss, int32_t* counts,
                     float* probs, int32_t* tokens, void* workspace, size_t workspace_bytes,
                     void* stream) {
  const char* fn = "moe_balance_loss";
  const int rc = check_balance(fn, n_tokens, n_experts, k, seq_offsets, n_sequences);
  if (rc) return rc;
  if (((!logits || !topk_idx) && n_tokens > 0) || !loss || !z_loss || !counts || !probs || !tokens)
    return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  if (off(logits, 4) || off(topk_idx, 4) || off(seq_offsets, 4) || off(loss, 4) || off(z_loss, 4) ||
      off(counts, 4) || off(probs, 4) || off(tokens, 4))
    return fail(MOE_ERR_ARG, "%s: pointers must be aligned to their elements", fn);
  const size_t need = moe::balance_workspace_bytes(n_tokens, n_experts, n_sequences);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? workspace_bytes : size_t(0));
  if (off(workspace, 256))
    return fail(MOE_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", fn);
  const moe::BalanceForward g{logits, topk_idx, n_tokens, n_experts, k, seq_offsets, n_sequences,
                              token_mask, loss, z_loss, counts, probs, tokens};
  return hip_status(moe::launch_balance_loss(g, workspace, static_cast<hipStream_t>(stream)), fn);
}

int moe_balance_loss_backward(const float* logits, int64_t n_tokens, int32_t n_experts, int32_t k,
                              const int32_t* seq_offsets, int32_t n_sequences,
                              const uint8_t* token_mask, const int32_t* counts,
                              const int32_t* tokens, const float* d_loss, const float* d_z_loss,
                              float* d_logits, int32_t accumulate, void* stream) {
  const char* fn = "moe_balance_loss_backward";
  const int rc = check_balance(fn, n_tokens, n_experts, k, seq_offsets, n_sequences);
  if (rc) return rc;
  if (n_tokens == 0) return ok();
  if (!logits || !counts || !tokens || !d_loss || !d_logits)
    return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  if (off(logits, 4) || off(seq_offsets, 4) || off(counts, 4) || off(tokens, 4) || off(d_loss, 4) ||
      off(d_z_loss, 4) || off(d_logits, 4))
    return fail(MOE_ERR_ARG, "%s: pointers must be aligned to their elements", fn);
  const moe::BalanceBackward g{logits, n_tokens, n_experts, k, seq_offsets, n_sequences, token_mask,
                               counts, tokens, d_loss, d_z_loss, d_logits, accumulate ? 1 : 0};
  return hip_status(moe::launch_balance_loss_backward(g, static_cast<hipStream_t>(stream)), fn);
}

namespace {
bool float_type(int32_t dtype) { return dtype == MOE_F32 || dtype == MOE_BF16; }

int check_int4_rows(const char* fn, int32_t dtype, int32_t scale_dtype, int64_t n_rows, int64_t k_dim,
                    int32_t group) {
  if (n_rows < 0) return fail(MOE_ERR_ARG, "%s: n_rows < 0", fn);
  if (k_dim < 1) return fail(MOE_ERR_ARG, "%s: k_dim < 1", fn);
  if (!float_type(dtype) || !float_type(scale_dtype))
    return fail(MOE_ERR_ARG, "%s: types must be MOE_F32 or MOE_BF16", fn);
  if (group != 32 && group != 64 && group != 128)
    return fail(MOE_ERR_UNSUPPORTED, "%s: group must be 32, 64 or 128 (got %d)", fn, group);
  if (k_dim % group != 0) return fail(MOE_ERR_UNSUPPORTED, "%s: k_dim must be a multiple of the group", fn);
  if (n_rows > (int64_t(1) << 40) / k_dim)
    return fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^40 elements", fn);
  return MOE_OK;
}
}  // namespace

int moe_quantize_int4(const void* x, int32_t x_dtype, int64_t n_rows, int64_t k_dim, int32_t group,
                      uint8_t* codes, void* scales, void* biases, int32_t scale_dtype, void* stream) {
  const char* fn = "moe_quantize_int4";
  const int rc = check_int4_rows(fn, x_dtype, scale_dtype, n_rows, k_dim, group);
  if (rc) return rc;
  if (n_rows == 0) return ok();
  if (!x || !codes || !scales) return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  if (off(x, 16) || off(codes, 4) || off(scales, 4) || off(biases, 4))
    return fail(MOE_ERR_UNSUPPORTED, "%s: x must be 16-byte, codes, scales and biases 4-byte aligned", fn);
  return hip_status(moe::launch_quantize_int4(x, x_dtype == MOE_BF16, n_rows * k_dim, group, codes, scales,
                                              biases, scale_dtype == MOE_BF16,
                                              static_cast<hipStream_t>(stream)),
                    fn);
}

int moe_dequant_int4(const uint8_t* codes, const void* scales, const void* biases, int32_t scale_dtype,
                     int64_t n_rows, int64_t k_dim, int32_t group, void* out, int32_t out_dtype,
                     void* stream) {
  const char* fn = "moe_dequant_int4";
  const int rc = check_int4_rows(fn, out_dtype, scale_dtype, n_rows, k_dim, group);
  if (rc) return rc;
  if (n_rows == 0) return ok();
  if (!codes || !scales || !out) return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  if (off(out, 16) || off(codes, 4) || off(scales, 4) || off(biases, 4))
    return fail(MOE_ERR_UNSUPPORTED, "%s: out must be 16-byte, codes, scales and biases 4-byte aligned", fn);
  return hip_status(moe::launch_dequant_int4(codes, scales, biases, scale_dtype == MOE_BF16, n_rows * k_dim,
                                             group, out, out_dtype == MOE_BF16,
                                             static_cast<hipStream_t>(stream)),
                    fn);
}

size_t moe_gather_gemm_int4_workspace_bytes(int64_t n_rows, int32_t n_experts) {
  if (n_rows < 0 || n_rows > INT32_MAX || n_experts < 1 || n_experts > MOE_MAX_EXPERTS) return 0;
  return moe::gather_gemm_int4_workspace_bytes(n_rows, n_experts);
}

int moe_gather_gemm_int4(const void* rows, int64_t n_rows, int64_t k_dim, const int32_t* row_expert,
                         int32_t n_experts, const uint8_t* w, const void* w_scales,
                         const void* w_biases, const uint8_t* w_up, const void* w_up_scales,
                         const void* w_up_biases, int32_t scale_dtype, int32_t group, int64_t n_dim,
                         void* y, int32_t y_dtype, void* workspace, size_t workspace_bytes,
                         void* stream) {
  const char* fn = "moe_gather_gemm_int4";
  if (n_rows < 0) return fail(MOE_ERR_ARG, "%s: n_rows < 0", fn);
  if (k_dim < 1 || n_dim < 1 || n_experts < 1) return fail(MOE_ERR_ARG, "%s: sizes must be >= 1", fn);
  if (!float_type(scale_dtype) || !float_type(y_dtype))
    return fail(MOE_ERR_ARG, "%s: scale and output types must be MOE_F32 or MOE_BF16", fn);
  if (!w_up != !w_up_scales) return fail(MOE_ERR_ARG, "%s: w_up and w_up_scales go together", fn);
  if (w_up ? !w_biases != !w_up_biases : w_up_biases != nullptr)
    return fail(MOE_ERR_ARG, "%s: w_biases and w_up_biases go together", fn);
  if (n_experts > MOE_MAX_EXPERTS) return fail(MOE_ERR_UNSUPPORTED, "%s: n_experts > %d", fn, MOE_MAX_EXPERTS);
  if (group != 32 && group != 64 && group != 128)
    return fail(MOE_ERR_UNSUPPORTED, "%s: group must be 32, 64 or 128 (got %d)", fn, group);
  if (k_dim % group != 0) return fail(MOE_ERR_UNSUPPORTED, "%s: k_dim must be a multiple of the group", fn);
  if (k_dim > (int64_t(1) << 22) || n_dim > (int64_t(1) << 22))
    return fail(MOE_ERR_UNSUPPORTED, "%s: k_dim and n_dim must be at most %d", fn, 1 << 22);
  if (n_rows > INT32_MAX) return fail(MOE_ERR_UNSUPPORTED, "%s: n_rows exceeds the int32 range", fn);
  const moe::Int4Product g{rows, n_rows, k_dim, n_experts, w, w_scales, w_biases, w_up, w_up_scales, w_up_biases,
                           scale_dtype == MOE_BF16, group, n_dim, y, y_dtype == MOE_BF16};
  if (n_rows > 0 && moe::gemm_int4_blocks(g) > moe::kMaxInt4Blocks)
    return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles", fn);
  if (n_rows == 0) return ok();
  if (!rows || !row_expert || !w || !w_scales || !y) return fail(MOE_ERR_ARG, "%s: null pointer argument", fn);
  if (off(rows, 16) || off(w, 16) || off(w_up, 16) || off(y, 16))
    return fail(MOE_ERR_UNSUPPORTED, "%s: rows, weights and y must be 16-byte aligned", fn);
  if (off(w_scales, 4) || off(w_biases, 4) || off(w_up_scales, 4) || off(w_up_biases, 4) || off(row_expert, 4))
    return fail(MOE_ERR_UNSUPPORTED, "%s: scales, biases and indices must be 4-byte aligned", fn);
  const size_t need = moe::gather_gemm_int4_workspace_bytes(n_rows, n_experts);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? workspace_bytes : size_t(0));
  if (off(workspace, 256))
    return fail(MOE_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", fn);
  return hip_status(moe::launch_gather_gemm_int4(g, row_expert, workspace, static_cast<hipStream_t>(stream)), fn);
}

}  // extern "C"
