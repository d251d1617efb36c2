// The C-ABI entry points: argument validation, plan lifetime, launches.
// Every function returns a status and never throws; a failing call leaves a
// message in a thread-local buffer (h3attn_last_error).
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>
#include <new>

#include "h3attn_internal.h"

namespace h3 {

static thread_local std::string g_last_error;

h3attn_status fail(h3attn_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

void clear_error() { g_last_error.clear(); }

void clear_runtime_error() { cudaGetLastError(); }

}  // namespace h3

using namespace h3;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Byte extent of a bf16 [S, H, 128] tensor with the given row stride (elements).
struct Extent {
  uintptr_t lo, hi;
};
Extent extent_of(const void* p, int64_t S, int32_t H, int64_t stride) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + (uintptr_t)(((S - 1) * stride + (int64_t)H * kHeadDim) * 2)};
}

// True when two bf16 [S, H, 128] strided tensors can share an element.  With
// equal strides the rows interleave, so compare the column windows modulo the
// stride; with different strides, any byte overlap counts.
bool may_overlap(const void* a, int64_t sa, const void* b, int64_t sb, int64_t S, int32_t H) {
  const Extent ea = extent_of(a, S, H, sa), eb = extent_of(b, S, H, sb);
  if (ea.hi <= eb.lo || eb.hi <= ea.lo) return false;
  if (sa != sb) return true;
  const int64_t width = (int64_t)H * kHeadDim;
  const int64_t delta = ((int64_t)eb.lo - (int64_t)ea.lo) / 2;  // both 16-byte aligned
  int64_t r = delta % sa;
  if (r < 0) r += sa;
  return r < width || r + width > sa;
}

struct DeviceGuard {
  int prev = -1;
  bool switched = false;
  cudaError_t enter(int dev) {
    clear_runtime_error();
    cudaError_t e = cudaGetDevice(&prev);
    if (e != cudaSuccess) return e;
    if (prev != dev) {
      e = cudaSetDevice(dev);
      switched = (e == cudaSuccess);
    }
    return e;
  }
  ~DeviceGuard() {
    if (switched) cudaSetDevice(prev);
  }
};

h3attn_status cuda_fail(cudaError_t e, const char* what) {
  return fail(H3ATTN_ECUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

void free_walk(WalkPlan* w) {
  if (w->d_units) cudaFree(w->d_units);
  if (w->d_own) cudaFree(w->d_own);
  if (w->d_joins) cudaFree(w->d_joins);
  if (w->d_part_o) cudaFree(w->d_part_o);
  if (w->d_part_ml) cudaFree(w->d_part_ml);
  w->d_units = nullptr;
  w->d_own = nullptr;
  w->d_joins = nullptr;
  w->d_part_o = nullptr;
  w->d_part_ml = nullptr;
}

void free_tree(TreePlan* t) {
  if (t->d_rows) cudaFree(t->d_rows);
  if (t->d_item0) cudaFree(t->d_item0);
  if (t->d_joins) cudaFree(t->d_joins);
  if (t->d_part_o) cudaFree(t->d_part_o);
  if (t->d_part_ml) cudaFree(t->d_part_ml);
  *t = TreePlan();
}

// Device copies of a walk's lists, and its partial buffers (enqueued; the caller
// synchronises the stream before the host lists change).
cudaError_t upload_walk(WalkPlan* w, cudaStream_t st) {
  const size_t units = w->units.size() * sizeof(WalkUnit), off = w->unit_off.size() * sizeof(int32_t);
  const size_t joins = w->joins.size() * sizeof(JoinRec), own = w->own.size() * sizeof(OwnTile);
  cudaError_t e = cudaMalloc(&w->d_units, units + off);
  if (e == cudaSuccess && joins > 0) e = cudaMalloc(&w->d_joins, joins);
  if (e == cudaSuccess && own > 0) e = cudaMalloc(&w->d_own, own);
  if (e == cudaSuccess && w->part_rows > 0) {
    e = cudaMalloc(&w->d_part_o, (size_t)w->part_rows * kHeadDim * sizeof(float));
    if (e == cudaSuccess) e = cudaMalloc(&w->d_part_ml, (size_t)w->part_rows * sizeof(float2));
  }
  if (e == cudaSuccess) e = cudaMemcpyAsync(w->d_units, w->units.data(), units, cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(w->d_units + w->units.size(), w->unit_off.data(), off, cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess && own > 0) e = cudaMemcpyAsync(w->d_own, w->own.data(), own, cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess && joins > 0)
    e = cudaMemcpyAsync(w->d_joins, w->joins.data(), joins, cudaMemcpyHostToDevice, st);
  return e;
}

void free_plan_device(Plan* p) {
  if (p->d_cu) cudaFree(p->d_cu);
  if (p->d_rope) cudaFree(p->d_rope);
  if (p->d_units) cudaFree(p->d_units);
  if (p->d_err) cudaFree(p->d_err);
  if (p->d_merges) cudaFree(p->d_merges);
  if (p->d_part_o) cudaFree(p->d_part_o);
  if (p->d_part_ml) cudaFree(p->d_part_ml);
  if (p->d_ktiles) cudaFree(p->d_ktiles);
  p->d_ktiles = nullptr;
  p->d_merges = nullptr;
  p->d_part_o = nullptr;
  p->d_part_ml = nullptr;
  p->d_cu = nullptr;
  p->d_rope = nullptr;
  p->d_units = nullptr;
  p->d_err = nullptr;
  free_walk(&p->sparse.walk);
  free_walk(&p->prefix.walk);
  free_walk(&p->causal.walk);
  free_tree(&p->tree);
  if (p->sparse.d_groups) cudaFree(p->sparse.d_groups);
  if (p->sparse.d_q_sum) cudaFree(p->sparse.d_q_sum);
  if (p->sparse.d_k_mean) cudaFree(p->sparse.d_k_mean);
  p->sparse.d_groups = nullptr;
  p->sparse.d_q_sum = nullptr;
  p->sparse.d_k_mean = nullptr;
}

// Device copy of the plan's unit_off (stored after the segment list).
const int32_t* unit_offsets(const Plan* p) {
  return reinterpret_cast<const int32_t*>(p->d_units + p->units_host.size());
}

// Uploads a walk's lists; `more` allocates and uploads what belongs with them.
template <class More>
h3attn_status attach_walk(WalkPlan* w, const char* what, void* cuda_stream, More more) {
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = upload_walk(w, st);
  if (e == cudaSuccess) e = more(st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess) {
    w->set = true;
    return H3ATTN_OK;
  }
  free_walk(w);
  return e == cudaErrorMemoryAllocation ? fail(H3ATTN_ENOMEM, "cudaMalloc failed for the plan's %s list", what)
                                        : cuda_fail(e, what);
}

h3attn_status check_plan(h3attn_plan_t plan) {
  if (plan == nullptr) return fail(H3ATTN_EINVAL, "plan is NULL");
  return H3ATTN_OK;
}

// True when byte ranges [a, a + na) and [b, b + nb) share a byte.
bool ranges_overlap(const void* a, uintptr_t na, const void* b, uintptr_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Checks of the forward's tensors shared by h3attn_forward and the forwards
// over other key walks.
h3attn_status check_forward_io(const Plan* plan, const void* q, const void* k, const void* v, int64_t qkv_row_stride,
                               const void* o, int64_t o_row_stride, float softmax_scale, const float* lse_out) {
  if (!q || !k || !v || !o) return fail(H3ATTN_EINVAL, "NULL q/k/v/o pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o))
    return fail(H3ATTN_EINVAL, "q/k/v/o must be 16-byte aligned");
  if (lse_out && !aligned4(lse_out)) return fail(H3ATTN_EINVAL, "lse_out must be 4-byte aligned");
  const int64_t width = (int64_t)plan->num_heads * kHeadDim;
  if (qkv_row_stride < width || o_row_stride < width || (qkv_row_stride % 8) || (o_row_stride % 8))
    return fail(H3ATTN_EINVAL, "row strides must be >= H*128 = %lld and multiples of 8 (got %lld, %lld)",
                (long long)width, (long long)qkv_row_stride, (long long)o_row_stride);
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f))
    return fail(H3ATTN_EINVAL, "softmax_scale must be finite and > 0");
  const int64_t S = plan->S;
  const int32_t H = plan->num_heads;
  const void* ins[3] = {q, k, v};
  for (int i = 0; i < 3; ++i)
    if (may_overlap(o, o_row_stride, ins[i], qkv_row_stride, S, H))
      return fail(H3ATTN_EINVAL, "o overlaps %c", "qkv"[i]);
  if (lse_out) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(lse_out), hi = lo + (uintptr_t)S * H * 4;
    const Extent eo = extent_of(o, S, H, o_row_stride);
    if (!(hi <= eo.lo || eo.hi <= lo)) return fail(H3ATTN_EINVAL, "lse_out overlaps o");
  }
  return H3ATTN_OK;
}

// lse_out against the inputs that the other walks read while they write it.
h3attn_status check_lse_inputs(const Plan* plan, const void* q, const void* k, const void* v, int64_t qkv_row_stride,
                               const float* lse_out) {
  if (!lse_out) return H3ATTN_OK;
  const void* ins[3] = {q, k, v};
  for (int i = 0; i < 3; ++i) {
    const Extent e = extent_of(ins[i], plan->S, plan->num_heads, qkv_row_stride);
    if (ranges_overlap(lse_out, (uintptr_t)plan->S * plan->num_heads * 4, ins[i], e.hi - e.lo))
      return fail(H3ATTN_EINVAL, "lse_out overlaps %c", "qkv"[i]);
  }
  return H3ATTN_OK;
}

// A packed layout given on the host, for the host listings of work.
h3attn_status check_layout(const int32_t* cu_seqlens, int32_t n_docs, int32_t num_heads, int32_t n_pairs) {
  if (n_docs < 1) return fail(H3ATTN_EINVAL, "n_docs must be >= 1 (got %d)", n_docs);
  if (num_heads < 1) return fail(H3ATTN_EINVAL, "num_heads must be >= 1 (got %d)", num_heads);
  if (n_pairs < 1 || n_pairs > 1024) return fail(H3ATTN_EINVAL, "n_pairs must be in [1, 1024] (got %d)", n_pairs);
  if (cu_seqlens[0] != 0) return fail(H3ATTN_EINVAL, "cu_seqlens[0] must be 0");
  for (int32_t d = 0; d < n_docs; ++d)
    if (cu_seqlens[d + 1] <= cu_seqlens[d])
      return fail(H3ATTN_EINVAL, "document %d is empty or cu_seqlens is not increasing", d);
  return H3ATTN_OK;
}

h3attn_status check_wait_limit(uint64_t timeout_ns) {
  if (timeout_ns < 1000ull || timeout_ns > 10000000000ull)
    return fail(H3ATTN_EINVAL, "timeout_ns must be in [1e3, 1e10]");
  return H3ATTN_OK;
}

// Sizes shared by the calls that set a list and the host listing.
h3attn_status check_list_sizes(int32_t q_block, int32_t max_blocks) {
  if (q_block != 256 && q_block != 512) return fail(H3ATTN_EINVAL, "q_block must be 256 or 512 (got %d)", q_block);
  if (max_blocks < 1 || max_blocks > (1 << 20))
    return fail(H3ATTN_EINVAL, "max_blocks must be in [1, 2^20] (got %d)", max_blocks);
  return H3ATTN_OK;
}
h3attn_status check_kv_heads(int32_t num_heads, int32_t num_kv_heads) {
  if (num_kv_heads < 1 || num_heads % num_kv_heads)
    return fail(H3ATTN_EINVAL, "num_kv_heads must be a divisor of num_heads = %d (got %d)", num_heads, num_kv_heads);
  return H3ATTN_OK;
}
h3attn_status check_prefix_len(int32_t prefix_len) {
  if (prefix_len < 1) return fail(H3ATTN_EINVAL, "prefix_len must be >= 1 (got %d)", prefix_len);
  return H3ATTN_OK;
}

}  // namespace

struct h3attn_plan : public h3::Plan {};

extern "C" {

const char* h3attn_last_error(void) { return g_last_error.c_str(); }

h3attn_status h3attn_plan_create(const h3attn_doc* docs, int32_t n_docs,
                                 const h3attn_plan_opts* opts, void* cuda_stream,
                                 h3attn_plan_t* out) {
  clear_error();
  if (out == nullptr) return fail(H3ATTN_EINVAL, "out is NULL");
  *out = nullptr;
  if (docs == nullptr) return fail(H3ATTN_EINVAL, "docs is NULL");
  if (opts == nullptr) return fail(H3ATTN_EINVAL, "opts is NULL");
  if (n_docs < 1) return fail(H3ATTN_EINVAL, "n_docs must be >= 1 (got %d)", n_docs);
  if (opts->num_heads < 1) return fail(H3ATTN_EINVAL, "num_heads must be >= 1 (got %d)", opts->num_heads);
  if (opts->head_dim != kHeadDim)
    return fail(H3ATTN_EUNSUPPORTED, "head_dim must be 128 (got %d)", opts->head_dim);
  if (opts->rope_dims != kRopeDims)
    return fail(H3ATTN_EUNSUPPORTED, "rope_dims must be 96 (got %d)", opts->rope_dims);
  if (!std::isfinite(opts->rope_base) || !(opts->rope_base > 1.0))
    return fail(H3ATTN_EINVAL, "rope_base must be finite and > 1");

  // Validate the layout on the host first (no device needed for EINVAL).
  {
    h3attn_plan probe;
    std::string why;
    try {
      why = build_plan_host(docs, n_docs, *opts, 1, probe, /*validate_only=*/true);
    } catch (const std::bad_alloc&) {
      return fail(H3ATTN_ENOMEM, "host allocation failed while building the plan");
    }
    if (!why.empty()) return fail(H3ATTN_EINVAL, "%s", why.c_str());
  }
  h3attn_plan* p = new (std::nothrow) h3attn_plan();
  if (p == nullptr) return fail(H3ATTN_ENOMEM, "host allocation failed");

  clear_runtime_error();
  cudaError_t e = cudaGetDevice(&p->device);
  if (e != cudaSuccess) {
    delete p;
    return cuda_fail(e, "cudaGetDevice");
  }
  int major = 0, minor = 0;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, p->device);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, p->device);
  cudaDeviceGetAttribute(&p->num_sms, cudaDevAttrMultiProcessorCount, p->device);
  if (major != 10 || minor != 3) {
    const int dev = p->device;
    delete p;
    return fail(H3ATTN_EUNSUPPORTED, "device %d is sm_%d%d; this library is built for sm_103a",
                dev, major, minor);
  }
  // the work list is balanced for the forward's persistent CTA pairs
  try {
    build_plan_host(docs, n_docs, *opts, forward_slots(p->device, p->num_sms), *p);
  } catch (const std::bad_alloc&) {
    delete p;
    return fail(H3ATTN_ENOMEM, "host allocation failed while building the plan");
  }

  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const size_t n_cu = p->cu_host.size(), n_rope = (size_t)p->S * kRopeHalf;
  const size_t units_bytes = p->units_host.size() * sizeof(WorkUnit),
               off_bytes = p->unit_off_host.size() * sizeof(int32_t);
  if ((e = cudaMalloc(&p->d_cu, n_cu * sizeof(int32_t))) != cudaSuccess ||
      (e = cudaMalloc(&p->d_rope, n_rope * sizeof(float2))) != cudaSuccess ||
      (e = cudaMalloc(&p->d_units, units_bytes + off_bytes)) != cudaSuccess ||
      (e = cudaMalloc(&p->d_err, 16)) != cudaSuccess ||
      (e = cudaMalloc(&p->d_ktiles, p->ktiles_host.size() * sizeof(int4))) != cudaSuccess ||
      (p->n_parts > 0 &&
       ((e = cudaMalloc(&p->d_merges, p->merges_host.size() * sizeof(MergeUnit))) != cudaSuccess ||
        (e = cudaMalloc(&p->d_part_o, (size_t)p->n_parts * kUnitRows * kHeadDim * sizeof(float))) != cudaSuccess ||
        (e = cudaMalloc(&p->d_part_ml, (size_t)p->n_parts * kUnitRows * sizeof(float2))) != cudaSuccess))) {
    free_plan_device(p);
    delete p;
    return e == cudaErrorMemoryAllocation ? fail(H3ATTN_ENOMEM, "cudaMalloc failed for the plan")
                                          : cuda_fail(e, "cudaMalloc");
  }
  if ((e = cudaMemcpyAsync(p->d_cu, p->cu_host.data(), n_cu * sizeof(int32_t),
                           cudaMemcpyHostToDevice, st)) != cudaSuccess ||
      (e = cudaMemcpyAsync(p->d_rope, p->rope_host.data(), n_rope * sizeof(float2),
                           cudaMemcpyHostToDevice, st)) != cudaSuccess ||
      (e = cudaMemcpyAsync(p->d_units, p->units_host.data(), units_bytes, cudaMemcpyHostToDevice, st)) !=
          cudaSuccess ||
      (e = cudaMemcpyAsync(p->d_units + p->units_host.size(), p->unit_off_host.data(), off_bytes,
                           cudaMemcpyHostToDevice, st)) != cudaSuccess ||
      (p->n_parts > 0 &&
       (e = cudaMemcpyAsync(p->d_merges, p->merges_host.data(), p->merges_host.size() * sizeof(MergeUnit),
                            cudaMemcpyHostToDevice, st)) != cudaSuccess) ||
      (e = cudaMemsetAsync(p->d_err, 0, 16, st)) != cudaSuccess ||
      (e = cudaMemcpyAsync(p->d_ktiles, p->ktiles_host.data(), p->ktiles_host.size() * sizeof(int4),
                           cudaMemcpyHostToDevice, st)) != cudaSuccess ||
      (e = cudaStreamSynchronize(st)) != cudaSuccess) {
    free_plan_device(p);
    delete p;
    return cuda_fail(e, "plan upload");
  }
  *out = p;
  return H3ATTN_OK;
}

h3attn_status h3attn_plan_destroy(h3attn_plan_t plan) {
  clear_error();
  if (plan == nullptr) return H3ATTN_OK;
  DeviceGuard g;
  g.enter(plan->device);
  cudaDeviceSynchronize();
  free_plan_device(plan);
  delete plan;
  return H3ATTN_OK;
}

h3attn_status h3attn_plan_info(h3attn_plan_t plan, int64_t* total_tokens, int32_t* n_docs,
                               int32_t* max_seqlen, int32_t* num_heads) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (total_tokens) *total_tokens = plan->S;
  if (n_docs) *n_docs = plan->n_docs;
  if (max_seqlen) *max_seqlen = plan->max_seqlen;
  if (num_heads) *num_heads = plan->num_heads;
  return H3ATTN_OK;
}

h3attn_status h3attn_plan_copy_cu_seqlens(h3attn_plan_t plan, int32_t* host_out) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (host_out == nullptr) return fail(H3ATTN_EINVAL, "host_out is NULL");
  // copy back from the device so the check covers the uploaded layout
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e == cudaSuccess)
    e = cudaMemcpy(host_out, plan->d_cu, plan->cu_host.size() * sizeof(int32_t), cudaMemcpyDeviceToHost);
  return e == cudaSuccess ? H3ATTN_OK : cuda_fail(e, "copy cu_seqlens");
}

h3attn_status h3attn_plan_copy_positions(h3attn_plan_t plan, double* host_out) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (host_out == nullptr) return fail(H3ATTN_EINVAL, "host_out is NULL");
  std::memcpy(host_out, plan->pos_host.data(), plan->pos_host.size() * sizeof(double));
  return H3ATTN_OK;
}

h3attn_status h3attn_plan_copy_rope_table(h3attn_plan_t plan, float* host_out) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (host_out == nullptr) return fail(H3ATTN_EINVAL, "host_out is NULL");
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e == cudaSuccess)
    e = cudaMemcpy(host_out, plan->d_rope, (size_t)plan->S * kRopeHalf * sizeof(float2),
                   cudaMemcpyDeviceToHost);
  return e == cudaSuccess ? H3ATTN_OK : cuda_fail(e, "copy rope table");
}

h3attn_status h3attn_qk_prologue(h3attn_plan_t plan, const void* q_in, const void* k_in,
                                 int64_t in_row_stride, void* q_out, void* k_out,
                                 int64_t out_row_stride, const float* gain_q,
                                 const float* gain_k, int64_t gain_head_stride, float eps,
                                 void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  // q_in and q_out both NULL: k only (the queries go to h3attn_forward_fused_q)
  const bool with_q = q_in != nullptr || q_out != nullptr;
  if (with_q && (!q_in || !q_out)) return fail(H3ATTN_EINVAL, "q_in and q_out must both be set or both NULL");
  if (!k_in || !k_out || !gain_k || (with_q && !gain_q))
    return fail(H3ATTN_EINVAL, "NULL tensor or gain pointer");
  if (!aligned16(k_in) || !aligned16(k_out) || !aligned16(gain_k) ||
      (with_q && (!aligned16(q_in) || !aligned16(q_out) || !aligned16(gain_q))))
    return fail(H3ATTN_EINVAL, "tensors and gains must be 16-byte aligned");
  const int64_t width = (int64_t)plan->num_heads * kHeadDim;
  if (in_row_stride < width || out_row_stride < width || (in_row_stride % 8) || (out_row_stride % 8))
    return fail(H3ATTN_EINVAL, "row strides must be >= H*128 = %lld and multiples of 8 (got %lld, %lld)",
                (long long)width, (long long)in_row_stride, (long long)out_row_stride);
  if (gain_head_stride != 0 && (gain_head_stride < kHeadDim || (gain_head_stride % 4)))
    return fail(H3ATTN_EINVAL, "gain_head_stride must be 0 or >= 128 and a multiple of 4");
  if (!std::isfinite(eps) || eps < 0.f) return fail(H3ATTN_EINVAL, "eps must be finite and >= 0");
  const int64_t S = plan->S;
  const int32_t H = plan->num_heads;
  // Outputs may alias their own input exactly (in place); no other overlap.
  struct T { const void* p; int64_t s; };
  const T ins[2] = {{q_in, in_row_stride}, {k_in, in_row_stride}};
  const T outs[2] = {{q_out, out_row_stride}, {k_out, out_row_stride}};
  if (with_q && may_overlap(q_out, out_row_stride, k_out, out_row_stride, S, H))
    return fail(H3ATTN_EINVAL, "q_out and k_out overlap");
  for (int o = with_q ? 0 : 1; o < 2; ++o)
    for (int i = with_q ? 0 : 1; i < 2; ++i) {
      const bool same = (outs[o].p == ins[i].p && outs[o].s == ins[i].s && o == i);
      if (!same && may_overlap(outs[o].p, outs[o].s, ins[i].p, ins[i].s, S, H))
        return fail(H3ATTN_EINVAL, "%s_out overlaps %s_in other than exactly in place",
                    o ? "k" : "q", i ? "k" : "q");
    }
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  PrologueArgs a{with_q ? q_in : nullptr, k_in, with_q ? q_out : nullptr, k_out, in_row_stride, out_row_stride,
                 gain_q, gain_k, gain_head_stride, plan->d_rope, S, H, eps};
  e = launch_qk_prologue(a, plan->num_sms, static_cast<cudaStream_t>(cuda_stream));
  return e == cudaSuccess ? H3ATTN_OK : cuda_fail(e, "qk_prologue launch");
}

static h3attn_status forward_impl(h3attn_plan_t plan, const void* q, const void* k, const void* v,
                                  int64_t qkv_row_stride, void* o, int64_t o_row_stride, float softmax_scale,
                                  float* lse_out, const float* gain_q, int64_t gain_head_stride, float eps,
                                  void* cuda_stream) {
  if (h3attn_status st = check_forward_io(plan, q, k, v, qkv_row_stride, o, o_row_stride, softmax_scale, lse_out))
    return st;
  const int64_t S = plan->S;
  const int32_t H = plan->num_heads;
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  ForwardArgs a{q, k, v, o, lse_out, qkv_row_stride, o_row_stride, S, H,
                softmax_scale * 1.4426950408889634f, plan->d_units, plan->n_units, unit_offsets(plan),
                plan->n_pairs, plan->d_err,
                plan->d_merges, (int32_t)plan->merges_host.size(), plan->d_part_o, plan->d_part_ml,
                gain_q, gain_head_stride, eps, plan->d_rope};
  std::string why;
  e = launch_forward(a, plan->device, plan->num_sms, static_cast<cudaStream_t>(cuda_stream), &why);
  if (e != cudaSuccess) {
    if (!why.empty()) return fail(H3ATTN_ECUDA, "forward: %s", why.c_str());
    return cuda_fail(e, "forward launch");
  }
  return H3ATTN_OK;
}

h3attn_status h3attn_forward(h3attn_plan_t plan, const void* q, const void* k, const void* v,
                             int64_t qkv_row_stride, void* o, int64_t o_row_stride,
                             float softmax_scale, float* lse_out, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  return forward_impl(plan, q, k, v, qkv_row_stride, o, o_row_stride, softmax_scale, lse_out, nullptr, 0, 0.f,
                      cuda_stream);
}

h3attn_status h3attn_forward_fused_q(h3attn_plan_t plan, const void* q_raw, const void* k, const void* v,
                                     int64_t qkv_row_stride, void* o, int64_t o_row_stride,
                                     const float* gain_q, int64_t gain_head_stride, float eps,
                                     float softmax_scale, float* lse_out, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (!gain_q) return fail(H3ATTN_EINVAL, "NULL gain_q");
  if (!aligned16(gain_q)) return fail(H3ATTN_EINVAL, "gain_q must be 16-byte aligned");
  if (gain_head_stride != 0 && (gain_head_stride < kHeadDim || (gain_head_stride % 4)))
    return fail(H3ATTN_EINVAL, "gain_head_stride must be 0 or >= 128 and a multiple of 4");
  if (!std::isfinite(eps) || eps < 0.f) return fail(H3ATTN_EINVAL, "eps must be finite and >= 0");
  return forward_impl(plan, q_raw, k, v, qkv_row_stride, o, o_row_stride, softmax_scale, lse_out, gain_q,
                      gain_head_stride, eps, cuda_stream);
}

// Checks shared by the FP8 quantisation calls: the three bf16 inputs (row
// stride qkv_row_stride) and the six outputs are non-NULL and 16-byte
// aligned, and no output shares bytes with an input or another output.
static h3attn_status check_fp8_io(const Plan* plan, const void* const (&in)[3], int64_t qkv_row_stride, void* q8,
                                  void* k8, void* v8t, float* sq, float* sk, float* sv) {
  if (!in[0] || !in[1] || !in[2] || !q8 || !k8 || !v8t || !sq || !sk || !sv)
    return fail(H3ATTN_EINVAL, "NULL tensor or scale pointer");
  if (!aligned16(in[0]) || !aligned16(in[1]) || !aligned16(in[2]) || !aligned16(q8) || !aligned16(k8) ||
      !aligned16(v8t) || !aligned16(sq) || !aligned16(sk) || !aligned16(sv))
    return fail(H3ATTN_EINVAL, "tensors and scales must be 16-byte aligned");
  const int64_t width = (int64_t)plan->num_heads * kHeadDim;
  if (qkv_row_stride < width || (qkv_row_stride % 8))
    return fail(H3ATTN_EINVAL, "row stride must be >= H*128 = %lld and a multiple of 8", (long long)width);
  const int64_t S = plan->S;
  const int32_t H = plan->num_heads;
  const int64_t v_pad = plan->v_pad;
  const uintptr_t in_lo[3] = {reinterpret_cast<uintptr_t>(in[0]), reinterpret_cast<uintptr_t>(in[1]),
                              reinterpret_cast<uintptr_t>(in[2])};
  const uintptr_t in_len = (uintptr_t)(((S - 1) * qkv_row_stride + width) * 2);
  const uintptr_t out_lo[6] = {reinterpret_cast<uintptr_t>(q8), reinterpret_cast<uintptr_t>(k8),
                               reinterpret_cast<uintptr_t>(v8t), reinterpret_cast<uintptr_t>(sq),
                               reinterpret_cast<uintptr_t>(sk), reinterpret_cast<uintptr_t>(sv)};
  const uintptr_t out_len[6] = {(uintptr_t)(S * width), (uintptr_t)(S * width), (uintptr_t)(H * kHeadDim * v_pad),
                                (uintptr_t)(H * S * 4), (uintptr_t)(H * S * 4), (uintptr_t)(H * kHeadDim * 4)};
  for (int o = 0; o < 6; ++o) {
    for (int i = 0; i < 3; ++i)
      if (out_lo[o] < in_lo[i] + in_len && in_lo[i] < out_lo[o] + out_len[o])
        return fail(H3ATTN_EINVAL, "an output overlaps an input");
    for (int o2 = o + 1; o2 < 6; ++o2)
      if (out_lo[o] < out_lo[o2] + out_len[o2] && out_lo[o2] < out_lo[o] + out_len[o])
        return fail(H3ATTN_EINVAL, "two outputs overlap");
  }
  return H3ATTN_OK;
}

h3attn_status h3attn_fp8_quantize(h3attn_plan_t plan, const void* q_hat, const void* k_hat, const void* v,
                                  int64_t qkv_row_stride, void* q8, void* k8, void* v8t, float* sq, float* sk,
                                  float* sv, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  const void* const in[3] = {q_hat, k_hat, v};
  if (h3attn_status s = check_fp8_io(plan, in, qkv_row_stride, q8, k8, v8t, sq, sk, sv)) return s;
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  Fp8QuantArgs a{q_hat, k_hat, v, qkv_row_stride, plan->S, plan->num_heads, plan->d_ktiles,
                 (int32_t)plan->ktiles_host.size(), q8, k8, v8t, plan->v_pad, sq, sk, sv};
  e = launch_fp8_quantize(a, plan->num_sms, static_cast<cudaStream_t>(cuda_stream));
  return e == cudaSuccess ? H3ATTN_OK : cuda_fail(e, "fp8 quantise launch");
}

h3attn_status h3attn_qk_prologue_fp8(h3attn_plan_t plan, const void* q_in, const void* k_in, const void* v,
                                     int64_t qkv_row_stride, const float* gain_q, const float* gain_k,
                                     int64_t gain_head_stride, float eps, void* q8, void* k8, void* v8t, float* sq,
                                     float* sk, float* sv, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (!gain_q || !gain_k) return fail(H3ATTN_EINVAL, "NULL gain pointer");
  if (!aligned16(gain_q) || !aligned16(gain_k)) return fail(H3ATTN_EINVAL, "gains must be 16-byte aligned");
  if (gain_head_stride != 0 && (gain_head_stride < kHeadDim || (gain_head_stride % 4)))
    return fail(H3ATTN_EINVAL, "gain_head_stride must be 0 or >= 128 and a multiple of 4");
  if (!std::isfinite(eps) || eps < 0.f) return fail(H3ATTN_EINVAL, "eps must be finite and >= 0");
  const void* const in[3] = {q_in, k_in, v};
  if (h3attn_status s = check_fp8_io(plan, in, qkv_row_stride, q8, k8, v8t, sq, sk, sv)) return s;
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  const PrologueArgs p{q_in, k_in, nullptr, nullptr, qkv_row_stride, 0, gain_q, gain_k, gain_head_stride,
                       plan->d_rope, plan->S, plan->num_heads, eps};
  const Fp8QuantArgs a{nullptr, nullptr, v, qkv_row_stride, plan->S, plan->num_heads, plan->d_ktiles,
                       (int32_t)plan->ktiles_host.size(), q8, k8, v8t, plan->v_pad, sq, sk, sv};
  e = launch_prologue_fp8(p, a, static_cast<cudaStream_t>(cuda_stream));
  return e == cudaSuccess ? H3ATTN_OK : cuda_fail(e, "fp8 prologue launch");
}

h3attn_status h3attn_plan_forward_kernels(h3attn_plan_t plan, int32_t* n_kernels) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (!n_kernels) return fail(H3ATTN_EINVAL, "NULL output pointer");
  *n_kernels = plan->merges_host.empty() ? 1 : 2;
  return H3ATTN_OK;
}

h3attn_status h3attn_work_list_host(const int32_t* cu_seqlens, int32_t n_docs, int32_t num_heads,
                                    int32_t n_pairs, int32_t* units, int64_t units_cap, int32_t* unit_off,
                                    int64_t* n_units, int32_t* n_pairs_used) {
  clear_error();
  if (!cu_seqlens || !n_units || !n_pairs_used) return fail(H3ATTN_EINVAL, "NULL cu_seqlens or output count");
  if (h3attn_status s = check_layout(cu_seqlens, n_docs, num_heads, n_pairs)) return s;
  try {
    std::vector<WorkUnit> all, segs;
    std::vector<int32_t> v_off, off;
    std::vector<MergeUnit> merges;
    int64_t v_pad = 0;
    int32_t pairs = 0, parts = 0;
    const std::string why = build_units(cu_seqlens, n_docs, num_heads, all, v_off, &v_pad);
    if (!why.empty()) return fail(H3ATTN_EINVAL, "%s", why.c_str());
    build_segments(all, n_pairs, segs, off, &pairs, merges, &parts);
    *n_units = (int64_t)segs.size();
    *n_pairs_used = pairs;
    if (units == nullptr) return H3ATTN_OK;
    if (units_cap < (int64_t)segs.size())
      return fail(H3ATTN_EINVAL, "units_cap %lld < %lld segments", (long long)units_cap, (long long)segs.size());
    std::memcpy(units, segs.data(), segs.size() * sizeof(WorkUnit));
    if (unit_off) std::memcpy(unit_off, off.data(), off.size() * sizeof(int32_t));
  } catch (const std::bad_alloc&) {
    return fail(H3ATTN_ENOMEM, "host allocation failed while building the work list");
  }
  return H3ATTN_OK;
}

h3attn_status h3attn_plan_fp8_v_keys(h3attn_plan_t plan, int64_t* v_keys) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (!v_keys) return fail(H3ATTN_EINVAL, "NULL output pointer");
  *v_keys = plan->v_pad;
  return H3ATTN_OK;
}

h3attn_status h3attn_forward_fp8(h3attn_plan_t plan, const void* q8, const void* k8, const void* v8t,
                                 const float* sq, const float* sk, const float* sv, void* o, int64_t o_row_stride,
                                 float softmax_scale, float* lse_out, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (!q8 || !k8 || !v8t || !sq || !sk || !sv || !o) return fail(H3ATTN_EINVAL, "NULL tensor or scale pointer");
  if (!aligned16(q8) || !aligned16(k8) || !aligned16(v8t) || !aligned16(sq) || !aligned16(sk) || !aligned16(sv) ||
      !aligned16(o))
    return fail(H3ATTN_EINVAL, "tensors and scales must be 16-byte aligned");
  if (lse_out && (reinterpret_cast<uintptr_t>(lse_out) & 3u))
    return fail(H3ATTN_EINVAL, "lse_out must be 4-byte aligned");
  const int64_t width = (int64_t)plan->num_heads * kHeadDim;
  if (o_row_stride < width || (o_row_stride % 8))
    return fail(H3ATTN_EINVAL, "o_row_stride must be >= H*128 = %lld and a multiple of 8", (long long)width);
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f))
    return fail(H3ATTN_EINVAL, "softmax_scale must be finite and > 0");
  const int64_t S = plan->S;
  const int32_t H = plan->num_heads;
  const Extent eo = extent_of(o, S, H, o_row_stride);
  const uintptr_t in_lo[3] = {reinterpret_cast<uintptr_t>(q8), reinterpret_cast<uintptr_t>(k8),
                              reinterpret_cast<uintptr_t>(v8t)};
  const uintptr_t in_len[3] = {(uintptr_t)(S * width), (uintptr_t)(S * width),
                               (uintptr_t)(H * kHeadDim * plan->v_pad)};
  for (int i = 0; i < 3; ++i)
    if (in_lo[i] < eo.hi && eo.lo < in_lo[i] + in_len[i]) return fail(H3ATTN_EINVAL, "o overlaps an input");
  if (lse_out) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(lse_out), hi = lo + (uintptr_t)S * H * 4;
    if (!(hi <= eo.lo || eo.hi <= lo)) return fail(H3ATTN_EINVAL, "lse_out overlaps o");
  }
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  ForwardArgs a{q8, k8, v8t, o, lse_out, width, o_row_stride, S, H,
                softmax_scale * 1.4426950408889634f, plan->d_units, plan->n_units, unit_offsets(plan),
                plan->n_pairs, plan->d_err,
                plan->d_merges, (int32_t)plan->merges_host.size(), plan->d_part_o, plan->d_part_ml,
                nullptr, 0, 0.f, nullptr, sq, sk, sv, plan->v_pad};
  std::string why;
  e = launch_forward_fp8(a, plan->device, plan->num_sms, static_cast<cudaStream_t>(cuda_stream), &why);
  if (e != cudaSuccess) {
    if (!why.empty()) return fail(H3ATTN_ECUDA, "forward: %s", why.c_str());
    return cuda_fail(e, "forward launch");
  }
  return H3ATTN_OK;
}

h3attn_status h3attn_plan_set_sparse(h3attn_plan_t plan, int32_t q_block, int32_t max_blocks, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (h3attn_status s = check_list_sizes(q_block, max_blocks)) return s;
  SparsePlan& sp = plan->sparse;
  if (sp.walk.set) return fail(H3ATTN_EINVAL, "the plan's sparse lists are already set");
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  try {
    const int32_t* cu = plan->cu_host.data();
    sp.walk = WalkPlan();
    const std::string why = build_list_walk(cu, plan->n_docs, plan->num_heads, q_block, max_blocks,
                                            forward_slots(plan->device, plan->num_sms), sp.walk);
    if (!why.empty()) return fail(H3ATTN_EINVAL, "%s", why.c_str());
    sp.q_block = q_block;
    sp.max_blocks = max_blocks;
    sp.n_q_blocks = 0;
    sp.max_tiles = 0;
    sp.groups.clear();
    for (int32_t d = 0; d < plan->n_docs; ++d)
      sp.max_tiles = std::max(sp.max_tiles, (cu[d + 1] - cu[d] + kKeyTile - 1) / kKeyTile);
    const int32_t warps = select_warps(sp.max_tiles);
    int32_t tile0 = 0;
    for (int32_t d = 0; d < plan->n_docs; ++d) {
      const int32_t L = cu[d + 1] - cu[d], blocks = (L + q_block - 1) / q_block, tiles = (L + kKeyTile - 1) / kKeyTile;
      for (int32_t i = 0; i < blocks; i += warps)
        sp.groups.push_back(SelectGroup{sp.n_q_blocks + i, std::min(warps, blocks - i), tile0, tiles, i, L, {0, 0}});
      sp.n_q_blocks += blocks;
      tile0 += tiles;
    }
  } catch (const std::exception&) {
    return fail(H3ATTN_ENOMEM, "host allocation failed while building the sparse lists");
  }
  const size_t words = (size_t)plan->num_heads * plan->ktiles_host.size() * kHeadDim;
  const size_t group_bytes = sp.groups.size() * sizeof(SelectGroup);
  const h3attn_status s = attach_walk(&sp.walk, "sparse", cuda_stream, [&](cudaStream_t st) {
    cudaError_t m = cudaMalloc(&sp.d_groups, group_bytes);
    if (m == cudaSuccess) m = cudaMalloc(&sp.d_q_sum, words * sizeof(float2));
    if (m == cudaSuccess) m = cudaMalloc(&sp.d_k_mean, words / 2 * sizeof(float2));
    if (m == cudaSuccess) m = cudaMemcpyAsync(sp.d_groups, sp.groups.data(), group_bytes, cudaMemcpyHostToDevice, st);
    return m;
  });
  if (s != H3ATTN_OK) {
    if (sp.d_groups) cudaFree(sp.d_groups);
    if (sp.d_q_sum) cudaFree(sp.d_q_sum);
    if (sp.d_k_mean) cudaFree(sp.d_k_mean);
    sp = SparsePlan();
  }
  return s;
}

static h3attn_status check_sparse(h3attn_plan_t plan) {
  if (h3attn_status s = check_plan(plan)) return s;
  if (!plan->sparse.walk.set) return fail(H3ATTN_EINVAL, "h3attn_plan_set_sparse has not been called on this plan");
  return H3ATTN_OK;
}

// The lists' pointers against a tensor of `bytes` bytes at p.
static bool lists_overlap(const Plan* plan, const int32_t* idx, const int32_t* cnt, const void* p, uintptr_t bytes) {
  const uintptr_t n = (uintptr_t)plan->num_heads * plan->sparse.n_q_blocks * 4;
  return ranges_overlap(idx, n * plan->sparse.max_blocks, p, bytes) || ranges_overlap(cnt, n, p, bytes);
}

h3attn_status h3attn_plan_sparse_info(h3attn_plan_t plan, int32_t* q_block, int32_t* max_blocks, int32_t* n_q_blocks) {
  clear_error();
  if (h3attn_status s = check_sparse(plan)) return s;
  if (q_block) *q_block = plan->sparse.q_block;
  if (max_blocks) *max_blocks = plan->sparse.max_blocks;
  if (n_q_blocks) *n_q_blocks = plan->sparse.n_q_blocks;
  return H3ATTN_OK;
}

h3attn_status h3attn_block_select(h3attn_plan_t plan, const void* q_hat, const void* k_hat, int64_t qkv_row_stride,
                                  int32_t keep, int32_t keep_own, int32_t* block_idx, int32_t* block_cnt,
                                  void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_sparse(plan)) return s;
  const SparsePlan& sp = plan->sparse;
  if (!q_hat || !k_hat || !block_idx || !block_cnt) return fail(H3ATTN_EINVAL, "NULL tensor or list pointer");
  if (!aligned16(q_hat) || !aligned16(k_hat)) return fail(H3ATTN_EINVAL, "q_hat and k_hat must be 16-byte aligned");
  if (!aligned4(block_idx) || !aligned4(block_cnt)) return fail(H3ATTN_EINVAL, "lists must be 4-byte aligned");
  const int64_t width = (int64_t)plan->num_heads * kHeadDim;
  if (qkv_row_stride < width || (qkv_row_stride % 8))
    return fail(H3ATTN_EINVAL, "row stride must be >= H*128 = %lld and a multiple of 8", (long long)width);
  if (keep < 1 || keep > sp.max_blocks)
    return fail(H3ATTN_EINVAL, "keep must be in [1, max_blocks = %d] (got %d)", sp.max_blocks, keep);
  if (plan->num_heads > 65535 || 2 * (int64_t)plan->ktiles_host.size() * plan->num_heads >= (int64_t(1) << 31))
    return fail(H3ATTN_EUNSUPPORTED, "too many heads or tokens to score");
  if (sp.max_tiles > kSelectMaxTiles)
    return fail(H3ATTN_EUNSUPPORTED, "a document of more than %d tokens cannot be scored", kSelectMaxTiles * kKeyTile);
  const uintptr_t n = (uintptr_t)plan->num_heads * sp.n_q_blocks * 4;
  const void* ins[2] = {q_hat, k_hat};
  for (const void* p : ins) {
    const Extent e = extent_of(p, plan->S, plan->num_heads, qkv_row_stride);
    if (lists_overlap(plan, block_idx, block_cnt, p, e.hi - e.lo))
      return fail(H3ATTN_EINVAL, "a list overlaps q_hat or k_hat");
  }
  if (ranges_overlap(block_idx, n * sp.max_blocks, block_cnt, n))
    return fail(H3ATTN_EINVAL, "block_idx and block_cnt overlap");
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  const SelectArgs a{q_hat, k_hat, qkv_row_stride, plan->num_heads, plan->d_ktiles, (int32_t)plan->ktiles_host.size(),
                     sp.d_groups, (int32_t)sp.groups.size(), sp.max_tiles, sp.n_q_blocks, sp.q_block / kKeyTile,
                     sp.d_q_sum, sp.d_k_mean, keep, keep_own, sp.max_blocks, block_idx, block_cnt, plan->num_sms};
  e = launch_block_select(a, static_cast<cudaStream_t>(cuda_stream));
  return e == cudaSuccess ? H3ATTN_OK : cuda_fail(e, "block select launch");
}

// Arguments of the forward over a walk's work list.
static ForwardArgs walk_forward_args(const Plan* plan, const WalkPlan& w, const void* q, const void* k, const void* v,
                                     int64_t qkv_row_stride, void* o, int64_t o_row_stride, float softmax_scale,
                                     float* lse_out) {
  return ForwardArgs{q, k, v, o, lse_out, qkv_row_stride, o_row_stride, plan->S, plan->num_heads,
                     softmax_scale * 1.4426950408889634f, reinterpret_cast<const WorkUnit*>(w.d_units),
                     (int32_t)w.units.size(), reinterpret_cast<const int32_t*>(w.d_units + w.units.size()), w.n_pairs,
                     plan->d_err, nullptr, 0, w.d_part_o, w.d_part_ml, nullptr, 0, 0.f, nullptr};
}
static WalkArgs walk_args(const WalkPlan& w) {
  WalkArgs x{};
  x.joins = w.d_joins;
  x.n_joins = (int32_t)w.joins.size();
  x.join_warps = w.join_warps;
  x.pair = w.streams == 2;
  x.pieces = w.pieces;
  return x;
}

h3attn_status h3attn_forward_sparse(h3attn_plan_t plan, const void* q, const void* k, const void* v,
                                    int64_t qkv_row_stride, const int32_t* block_idx, const int32_t* block_cnt,
                                    void* o, int64_t o_row_stride, float softmax_scale, float* lse_out,
                                    void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_sparse(plan)) return s;
  if (h3attn_status s = check_forward_io(plan, q, k, v, qkv_row_stride, o, o_row_stride, softmax_scale, lse_out))
    return s;
  if (h3attn_status s = check_lse_inputs(plan, q, k, v, qkv_row_stride, lse_out)) return s;
  const SparsePlan& sp = plan->sparse;
  if (!block_idx || !block_cnt) return fail(H3ATTN_EINVAL, "NULL block_idx or block_cnt");
  if (!aligned4(block_idx) || !aligned4(block_cnt)) return fail(H3ATTN_EINVAL, "lists must be 4-byte aligned");
  const Extent eo = extent_of(o, plan->S, plan->num_heads, o_row_stride);
  if (lists_overlap(plan, block_idx, block_cnt, o, eo.hi - eo.lo)) return fail(H3ATTN_EINVAL, "o overlaps a list");
  if (lse_out && lists_overlap(plan, block_idx, block_cnt, lse_out, (uintptr_t)plan->S * plan->num_heads * 4))
    return fail(H3ATTN_EINVAL, "lse_out overlaps a list");
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  const ForwardArgs a =
      walk_forward_args(plan, sp.walk, q, k, v, qkv_row_stride, o, o_row_stride, softmax_scale, lse_out);
  WalkArgs w = walk_args(sp.walk);
  w.block_idx = block_idx;
  w.block_cnt = block_cnt;
  w.n_q_blocks = sp.n_q_blocks;
  w.max_blocks = sp.max_blocks;
  std::string why;
  e = launch_forward_list(a, w, static_cast<cudaStream_t>(cuda_stream), &why);
  if (e != cudaSuccess) {
    if (!why.empty()) return fail(H3ATTN_ECUDA, "sparse forward: %s", why.c_str());
    return cuda_fail(e, "sparse forward launch");
  }
  return H3ATTN_OK;
}

h3attn_status h3attn_plan_set_prefix(h3attn_plan_t plan, int32_t prefix_len, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (h3attn_status s = check_prefix_len(prefix_len)) return s;
  PrefixPlan& pp = plan->prefix;
  if (pp.walk.set) return fail(H3ATTN_EINVAL, "the plan's prefix is already set");
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  try {
    pp.walk = WalkPlan();
    const std::string why = build_prefix_walk(plan->cu_host.data(), plan->n_docs, plan->num_heads, prefix_len,
                                              forward_slots(plan->device, plan->num_sms), pp.walk);
    if (!why.empty()) return fail(H3ATTN_EINVAL, "%s", why.c_str());
    pp.len = prefix_len;
  } catch (const std::exception&) {
    return fail(H3ATTN_ENOMEM, "host allocation failed while building the prefix list");
  }
  return attach_walk(&pp.walk, "prefix", cuda_stream, [](cudaStream_t) { return cudaSuccess; });
}

h3attn_status h3attn_forward_prefix(h3attn_plan_t plan, const void* q, const void* k, const void* v,
                                    int64_t qkv_row_stride, const void* k_prefix, const void* v_prefix,
                                    int64_t prefix_row_stride, void* o, int64_t o_row_stride, float softmax_scale,
                                    float* lse_out, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  const PrefixPlan& pp = plan->prefix;
  if (!pp.walk.set) return fail(H3ATTN_EINVAL, "h3attn_plan_set_prefix has not been called on this plan");
  if (h3attn_status s = check_forward_io(plan, q, k, v, qkv_row_stride, o, o_row_stride, softmax_scale, lse_out))
    return s;
  if (h3attn_status s = check_lse_inputs(plan, q, k, v, qkv_row_stride, lse_out)) return s;
  if (!k_prefix || !v_prefix) return fail(H3ATTN_EINVAL, "NULL k_prefix or v_prefix");
  if (!aligned16(k_prefix) || !aligned16(v_prefix))
    return fail(H3ATTN_EINVAL, "k_prefix and v_prefix must be 16-byte aligned");
  const int64_t width = (int64_t)plan->num_heads * kHeadDim;
  if (prefix_row_stride < width || (prefix_row_stride % 8))
    return fail(H3ATTN_EINVAL, "the prefix's row stride must be >= H*128 = %lld and a multiple of 8 (got %lld)",
                (long long)width, (long long)prefix_row_stride);
  const Extent eo = extent_of(o, plan->S, plan->num_heads, o_row_stride);
  const void* pre[2] = {k_prefix, v_prefix};
  for (const void* p : pre) {
    const Extent ep = extent_of(p, pp.len, plan->num_heads, prefix_row_stride);
    if (ranges_overlap(o, eo.hi - eo.lo, p, ep.hi - ep.lo)) return fail(H3ATTN_EINVAL, "o overlaps the prefix");
    if (lse_out && ranges_overlap(lse_out, (uintptr_t)plan->S * plan->num_heads * 4, p, ep.hi - ep.lo))
      return fail(H3ATTN_EINVAL, "lse_out overlaps the prefix");
  }
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  const ForwardArgs a =
      walk_forward_args(plan, pp.walk, q, k, v, qkv_row_stride, o, o_row_stride, softmax_scale, lse_out);
  WalkArgs w = walk_args(pp.walk);
  w.k_prefix = k_prefix;
  w.v_prefix = v_prefix;
  w.prefix_stride = prefix_row_stride;
  w.prefix_len = pp.len;
  w.own = pp.walk.d_own;
  std::string why;
  e = launch_forward_prefix(a, w, static_cast<cudaStream_t>(cuda_stream), &why);
  if (e != cudaSuccess) {
    if (!why.empty()) return fail(H3ATTN_ECUDA, "prefix forward: %s", why.c_str());
    return cuda_fail(e, "prefix forward launch");
  }
  return H3ATTN_OK;
}

h3attn_status h3attn_walk_list_host(int32_t kind, const int32_t* cu_seqlens, int32_t n_docs, int32_t num_heads,
                                    int32_t p0, int32_t p1, int32_t n_pairs, int32_t* units, int64_t units_cap,
                                    int32_t* unit_off, int32_t* joins, int64_t joins_cap, int32_t* own,
                                    int64_t own_cap, int64_t* n_units, int32_t* n_pairs_used, int64_t* n_joins,
                                    int64_t* n_own, int64_t* n_part_rows) {
  clear_error();
  if (!cu_seqlens || !n_units || !n_pairs_used || !n_joins || !n_own || !n_part_rows)
    return fail(H3ATTN_EINVAL, "NULL cu_seqlens or output count");
  if (h3attn_status s = check_layout(cu_seqlens, n_docs, num_heads, n_pairs)) return s;
  if (kind < 0 || kind > 2) return fail(H3ATTN_EINVAL, "kind must be 0, 1 or 2 (got %d)", kind);
  if (h3attn_status s = kind == 0 ? check_list_sizes(p0, p1) : kind == 1 ? check_prefix_len(p0) : check_kv_heads(num_heads, p0))
    return s;
  try {
    WalkPlan w;
    const std::string why = kind == 0   ? build_list_walk(cu_seqlens, n_docs, num_heads, p0, p1, n_pairs, w)
                            : kind == 1 ? build_prefix_walk(cu_seqlens, n_docs, num_heads, p0, n_pairs, w)
                                        : build_causal_walk(cu_seqlens, n_docs, num_heads, p0, n_pairs, w);
    if (!why.empty()) return fail(H3ATTN_EINVAL, "%s", why.c_str());
    // pair by pair (of two streams, the first one's segments before the second's)
    std::vector<WalkUnit> segs;
    std::vector<int32_t> off(1, 0);
    for (int32_t p = 0; p < w.n_pairs; ++p) {
      for (int x = 0; x < w.streams; ++x) {
        const int32_t* r = w.streams == 1 ? &w.unit_off[p] : &w.unit_off[4 * p + 2 * x];
        segs.insert(segs.end(), w.units.begin() + r[0], w.units.begin() + r[1]);
      }
      off.push_back((int32_t)segs.size());
    }
    *n_units = (int64_t)segs.size();
    *n_pairs_used = w.n_pairs;
    *n_joins = (int64_t)w.joins.size();
    *n_own = (int64_t)w.own.size();
    *n_part_rows = w.part_rows;
    if (units == nullptr) return H3ATTN_OK;
    if (units_cap < *n_units || (joins && joins_cap < *n_joins) || (own && own_cap < *n_own))
      return fail(H3ATTN_EINVAL, "capacities %lld, %lld, %lld < %lld segments, %lld joins, %lld own tiles",
                  (long long)units_cap, (long long)joins_cap, (long long)own_cap, (long long)*n_units,
                  (long long)*n_joins, (long long)*n_own);
    std::memcpy(units, segs.data(), segs.size() * sizeof(WalkUnit));
    if (unit_off) std::memcpy(unit_off, off.data(), off.size() * sizeof(int32_t));
    if (joins && !w.joins.empty()) std::memcpy(joins, w.joins.data(), w.joins.size() * sizeof(JoinRec));
    if (own && !w.own.empty()) std::memcpy(own, w.own.data(), w.own.size() * sizeof(OwnTile));
  } catch (const std::exception&) {
    return fail(H3ATTN_ENOMEM, "host allocation failed while building the work list");
  }
  return H3ATTN_OK;
}

// ------------------------------------------- rotary positions, the cache ----

h3attn_status h3attn_rope_init(const h3attn_rope_opts* opts, h3attn_rope* out) {
  clear_error();
  if (opts == nullptr || out == nullptr) return fail(H3ATTN_EINVAL, "opts or out is NULL");
  const int32_t d = opts->rope_dims;
  if (d < 16 || d > kHeadDim || d % 16)
    return fail(H3ATTN_EUNSUPPORTED, "rope_dims must be a multiple of 16 in [16, 128] (got %d)", d);
  if (opts->interleaved != 0 && opts->interleaved != 1) return fail(H3ATTN_EINVAL, "interleaved must be 0 or 1");
  if (!std::isfinite(opts->base) || !(opts->base > 1.0)) return fail(H3ATTN_EINVAL, "base must be finite and > 1");
  if (opts->scaling < H3ATTN_ROPE_PLAIN || opts->scaling > H3ATTN_ROPE_BY_PARTS)
    return fail(H3ATTN_EINVAL, "scaling must be a h3attn_rope_scaling (got %d)", opts->scaling);
  const double s = opts->scaling == H3ATTN_ROPE_PLAIN ? 1.0 : opts->factor;
  if (!std::isfinite(s) || !(s >= 1.0)) return fail(H3ATTN_EINVAL, "factor must be finite and >= 1");
  const bool parts = opts->scaling == H3ATTN_ROPE_BY_PARTS;
  if (parts && (!std::isfinite(opts->original_len) || !(opts->original_len > 0.0) || !std::isfinite(opts->beta_fast) ||
                !(opts->beta_slow >= 0.0) || !(opts->beta_fast > opts->beta_slow)))
    return fail(H3ATTN_EINVAL, "scaling by parts needs original_len > 0 and beta_fast > beta_slow >= 0");
  if (!std::isfinite(opts->amplitude) || opts->amplitude < 0.0 || opts->amplitude > 1e30)
    return fail(H3ATTN_EINVAL, "amplitude must be 0 (the default) or in (0, 1e30]");
  if (opts->n_axes < 1 || opts->n_axes > 3) return fail(H3ATTN_EINVAL, "n_axes must be in [1, 3] (got %d)", opts->n_axes);
  for (int32_t j = 0; opts->axis != nullptr && j < d / 2; ++j)
    if (opts->axis[j] >= opts->n_axes) return fail(H3ATTN_EINVAL, "axis[%d] = %d is no axis", j, (int)opts->axis[j]);
  const double two_pi = 6.283185307179586476925;
  const double base = opts->scaling == H3ATTN_ROPE_NTK ? opts->base * std::pow(s, (double)d / (d - 2)) : opts->base;
  if (!std::isfinite(base)) return fail(H3ATTN_EINVAL, "base and factor are too large");
  h3attn_rope r;
  std::memset(&r, 0, sizeof(r));
  r.rope_dims = d;
  r.interleaved = opts->interleaved;
  r.n_axes = opts->n_axes;
  r.amplitude = (float)(opts->amplitude != 0.0 ? opts->amplitude : parts ? 0.1 * std::log(s) + 1.0 : 1.0);
  for (int32_t j = 0; j < d / 2; ++j) {
    double f = std::pow(base, -2.0 * j / d);
    if (opts->scaling == H3ATTN_ROPE_LINEAR) f /= s;
    if (parts) {
      double g = (opts->original_len * f / two_pi - opts->beta_slow) / (opts->beta_fast - opts->beta_slow);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f *= g + (1.0 - g) / s;
    }
    r.turns[j] = (uint64_t)std::ldexp(f / two_pi, 64);  // (f <= 1: below 2^62)
    r.axis[j] = opts->axis != nullptr ? opts->axis[j] : 0;
  }
  *out = r;
  return H3ATTN_OK;
}

namespace {

h3attn_status check_rope(const h3attn_rope* rope, const int32_t* positions, int64_t n_tokens) {
  if (!rope || (!positions && n_tokens != 0)) return fail(H3ATTN_EINVAL, "NULL rope or positions");
  bool good = rope->rope_dims >= 16 && rope->rope_dims <= kHeadDim && rope->rope_dims % 16 == 0 &&
              (rope->interleaved == 0 || rope->interleaved == 1) && rope->n_axes >= 1 && rope->n_axes <= 3;
  for (int j = 0; good && j < 64; ++j) good = rope->axis[j] < rope->n_axes;
  if (!good) return fail(H3ATTN_EINVAL, "rope was not filled by h3attn_rope_init");
  if (!aligned4(positions)) return fail(H3ATTN_EINVAL, "positions must be 4-byte aligned");
  if (n_tokens < 0 || n_tokens > INT32_MAX) return fail(H3ATTN_EINVAL, "n_tokens must be in [0, 2^31) (got %lld)", (long long)n_tokens);
  return H3ATTN_OK;
}

// Rows of a call without a plan: bf16 [n, heads, 128].
struct Rows {
  const char* name;
  const void* p;
  int64_t stride;
  int32_t heads;
  int64_t width() const { return (int64_t)heads * kHeadDim; }
  uintptr_t bytes(int64_t n) const { return n > 0 ? (uintptr_t)((n - 1) * stride + width()) * 2 : 0; }
};

h3attn_status check_rows(const Rows& r, int64_t n) {
  if (!r.p) return fail(H3ATTN_EINVAL, "NULL %s", r.name);
  if (!aligned16(r.p)) return fail(H3ATTN_EINVAL, "%s must be 16-byte aligned", r.name);
  if (r.heads < 1 || r.heads > (1 << 20)) return fail(H3ATTN_EINVAL, "%s: heads must be in [1, 2^20] (got %d)", r.name, r.heads);
  if (r.stride < r.width() || r.stride % 8 || (n > 1 && r.stride > (int64_t(1) << 60) / n))
    return fail(H3ATTN_EINVAL, "%s: its row stride must be >= %lld and a multiple of 8 (got %lld)", r.name,
                (long long)r.width(), (long long)r.stride);
  return H3ATTN_OK;
}

// True when two tensors of n rows can share an element: with equal strides their
// column windows are compared, otherwise any byte counts.
bool rows_overlap(const Rows& a, const Rows& b, int64_t n) {
  if (!ranges_overlap(a.p, a.bytes(n), b.p, b.bytes(n))) return false;
  if (a.stride != b.stride) return true;
  const int64_t delta = ((int64_t)reinterpret_cast<uintptr_t>(b.p) - (int64_t)reinterpret_cast<uintptr_t>(a.p)) / 2;
  int64_t r = delta % a.stride;
  if (r < 0) r += a.stride;
  return r < a.width() || r + b.width() > a.stride;
}

// A dimension of the cache's rows.
struct CacheDim {
  int64_t n, stride;
};

// Whether a row of the cache `delta` elements on meets a row: d[0 .. dims) sorted by stride, each stride past what the
// smaller ones span, so that only the two multiples of a stride around delta come near it.
bool rows_meet(const CacheDim* d, int dims, int64_t delta) {
  if (dims == 0) return delta > -kHeadDim && delta < kHeadDim;
  const CacheDim& x = d[dims - 1];
  if (x.n == 1) return rows_meet(d, dims - 1, delta);
  int64_t i = delta / x.stride;
  if (delta % x.stride < 0) --i;
  for (int64_t at = i; at <= i + 1; ++at)
    if (at > -x.n && at < x.n && rows_meet(d, dims - 1, delta - at * x.stride)) return true;
  return false;
}

h3attn_status check_cache(const h3attn_cache* c) {
  if (!c || !c->k || !c->v) return fail(H3ATTN_EINVAL, "NULL cache or cache tensor");
  if (!aligned16(c->k) || !aligned16(c->v)) return fail(H3ATTN_EINVAL, "the cache's tensors must be 16-byte aligned");
  if (c->n_pages < 1 || c->page_size < 1 || c->num_kv_heads < 1)
    return fail(H3ATTN_EINVAL, "the cache's sizes must be >= 1 (got %d pages of %d, %d heads)", c->n_pages, c->page_size,
                c->num_kv_heads);
  if ((int64_t)c->n_pages * c->page_size > INT32_MAX) return fail(H3ATTN_EINVAL, "the cache has 2^31 or more slots");
  // rows share no element where every stride reaches past what the smaller ones span
  CacheDim d[3] = {{c->n_pages, c->page_stride}, {c->page_size, c->token_stride}, {c->num_kv_heads, c->head_stride}};
  std::sort(d, d + 3, [](const CacheDim& x, const CacheDim& y) { return x.stride < y.stride; });
  int64_t span = kHeadDim;
  for (const CacheDim& x : d) {
    if (x.stride < 0 || x.stride % 8) return fail(H3ATTN_EINVAL, "the cache's strides must be multiples of 8 (got %lld)", (long long)x.stride);
    if (x.n == 1) continue;
    if (x.stride < span || x.stride > (int64_t(1) << 38) || x.stride > (int64_t(1) << 60) / x.n)
      return fail(H3ATTN_EINVAL, "the cache's rows share elements, or lie too far apart (stride %lld)", (long long)x.stride);
    span += (x.n - 1) * x.stride;
  }
  // (v's rows may lie between k's; the distance of addresses below 2^63 in elements)
  const int64_t delta = ((int64_t)reinterpret_cast<uintptr_t>(c->v) - (int64_t)reinterpret_cast<uintptr_t>(c->k)) / 2;
  if (rows_meet(d, 3, delta)) return fail(H3ATTN_EINVAL, "the cache's k and v share elements");
  return H3ATTN_OK;
}

// Bytes that the cache's k (or v) spans.
uintptr_t cache_bytes(const h3attn_cache* c) {
  return (uintptr_t)((c->n_pages - 1) * c->page_stride + (c->page_size - 1) * c->token_stride +
                     (c->num_kv_heads - 1) * c->head_stride + kHeadDim) * 2;
}
bool overlaps_cache(const h3attn_cache* c, const void* p, uintptr_t bytes) {
  const uintptr_t n = cache_bytes(c);
  return ranges_overlap(c->k, n, p, bytes) || ranges_overlap(c->v, n, p, bytes);
}

cudaError_t current_sms(int* sms) {
  clear_runtime_error();
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

h3attn_status launch_rotary_args(const RotaryArgs& a, void* cuda_stream) {
  int sms = 0;
  cudaError_t e = current_sms(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  e = launch_rotary(a, sms, static_cast<cudaStream_t>(cuda_stream));
  return e == cudaSuccess ? H3ATTN_OK : cuda_fail(e, "rotary launch");
}

}  // namespace

h3attn_status h3attn_rotary(const h3attn_rope* rope, const int32_t* positions, int64_t n_tokens, const void* q_in,
                            int64_t q_in_stride, void* q_out, int64_t q_out_stride, int32_t num_heads, const void* k_in,
                            int64_t k_in_stride, void* k_out, int64_t k_out_stride, int32_t num_kv_heads,
                            int32_t inverse, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_rope(rope, positions, n_tokens)) return s;
  if (n_tokens == 0) return H3ATTN_OK;
  const bool with_q = q_in || q_out, with_k = k_in || k_out;
  if (!with_q && !with_k) return fail(H3ATTN_EINVAL, "NULL q and k");
  const Rows in[2] = {{"q_in", q_in, q_in_stride, num_heads}, {"k_in", k_in, k_in_stride, num_kv_heads}};
  const Rows out[2] = {{"q_out", q_out, q_out_stride, num_heads}, {"k_out", k_out, k_out_stride, num_kv_heads}};
  const bool with[2] = {with_q, with_k};
  for (int i = 0; i < 2; ++i)
    if (with[i]) {
      if (h3attn_status s = check_rows(in[i], n_tokens)) return s;
      if (h3attn_status s = check_rows(out[i], n_tokens)) return s;
    }
  for (int i = 0; i < 2; ++i) {
    if (!with[i]) continue;
    if (ranges_overlap(out[i].p, out[i].bytes(n_tokens), positions, (uintptr_t)n_tokens * rope->n_axes * 4))
      return fail(H3ATTN_EINVAL, "%s overlaps positions", out[i].name);
    for (int j = 0; j < 2; ++j) {
      if (!with[j]) continue;
      const bool in_place = i == j && in[j].p == out[i].p && in[j].stride == out[i].stride;
      if (!in_place && rows_overlap(out[i], in[j], n_tokens))
        return fail(H3ATTN_EINVAL, "%s overlaps %s other than exactly in place", out[i].name, in[j].name);
    }
  }
  if (with_q && with_k && rows_overlap(out[0], out[1], n_tokens)) return fail(H3ATTN_EINVAL, "q_out and k_out overlap");
  RotaryArgs a{};
  a.rope = *rope;
  a.positions = positions;
  a.n = n_tokens;
  a.q_in = static_cast<const __nv_bfloat16*>(q_in);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.q_in_stride = q_in_stride;
  a.q_out_stride = q_out_stride;
  a.k_in = static_cast<const __nv_bfloat16*>(k_in);
  a.k_in_stride = k_in_stride;
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.k_out_stride = k_out_stride;
  a.k_out_head_stride = kHeadDim;
  a.H = with_q ? num_heads : 0;
  a.Hk = with_k ? num_kv_heads : 0;
  a.inverse = inverse != 0;
  return launch_rotary_args(a, cuda_stream);
}

h3attn_status h3attn_rotary_store(const h3attn_rope* rope, const int32_t* positions, int64_t n_tokens, const void* q_in,
                                  int64_t q_in_stride, void* q_out, int64_t q_out_stride, int32_t num_heads,
                                  const void* k_in, const void* v_in, int64_t kv_row_stride, const h3attn_cache* cache,
                                  const int32_t* slots, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_rope(rope, positions, n_tokens)) return s;
  if (h3attn_status s = check_cache(cache)) return s;
  if (n_tokens == 0) return H3ATTN_OK;
  if (!slots || !aligned4(slots)) return fail(H3ATTN_EINVAL, "slots must be a 4-byte aligned list");
  const bool with_q = q_in || q_out;
  const Rows q[2] = {{"q_in", q_in, q_in_stride, num_heads}, {"q_out", q_out, q_out_stride, num_heads}};
  const Rows kv[2] = {{"k_in", k_in, kv_row_stride, cache->num_kv_heads}, {"v_in", v_in, kv_row_stride, cache->num_kv_heads}};
  const uintptr_t n = (uintptr_t)n_tokens;
  for (int i = 0; i < 2; ++i) {
    if (h3attn_status s = check_rows(kv[i], n_tokens)) return s;
    if (overlaps_cache(cache, kv[i].p, kv[i].bytes(n_tokens))) return fail(H3ATTN_EINVAL, "%s overlaps the cache", kv[i].name);
    if (!with_q) continue;
    if (h3attn_status s = check_rows(q[i], n_tokens)) return s;
    if (overlaps_cache(cache, q[i].p, q[i].bytes(n_tokens))) return fail(H3ATTN_EINVAL, "%s overlaps the cache", q[i].name);
  }
  if (overlaps_cache(cache, positions, n * rope->n_axes * 4) || overlaps_cache(cache, slots, n * 4))
    return fail(H3ATTN_EINVAL, "positions or slots overlap the cache");
  if (with_q) {
    if (ranges_overlap(q_out, q[1].bytes(n_tokens), positions, n * rope->n_axes * 4) ||
        ranges_overlap(q_out, q[1].bytes(n_tokens), slots, n * 4))
      return fail(H3ATTN_EINVAL, "q_out overlaps positions or slots");
    if (!(q_in == q_out && q_in_stride == q_out_stride) && rows_overlap(q[1], q[0], n_tokens))
      return fail(H3ATTN_EINVAL, "q_out overlaps q_in other than exactly in place");
    for (const Rows& r : kv)
      if (rows_overlap(q[1], r, n_tokens)) return fail(H3ATTN_EINVAL, "q_out overlaps %s", r.name);
  }
  RotaryArgs a{};
  a.rope = *rope;
  a.positions = positions;
  a.n = n_tokens;
  a.q_in = static_cast<const __nv_bfloat16*>(q_in);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.q_in_stride = q_in_stride;
  a.q_out_stride = q_out_stride;
  a.k_in = static_cast<const __nv_bfloat16*>(k_in);
  a.v_in = static_cast<const __nv_bfloat16*>(v_in);
  a.k_in_stride = kv_row_stride;
  a.k_out = static_cast<__nv_bfloat16*>(cache->k);
  a.v_out = static_cast<__nv_bfloat16*>(cache->v);
  a.k_out_stride = cache->token_stride;
  a.k_out_head_stride = cache->head_stride;
  a.slots = slots;
  a.page_stride = cache->page_stride;
  a.page_size = cache->page_size;
  a.n_slots = cache->n_pages * cache->page_size;
  a.H = with_q ? num_heads : 0;
  a.Hk = a.Hv = cache->num_kv_heads;
  return launch_rotary_args(a, cuda_stream);
}

h3attn_status h3attn_cache_move(const h3attn_cache* cache, const int32_t* src, const int32_t* dst, int64_t n_groups,
                                int32_t width, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_cache(cache)) return s;
  if (n_groups == 0) return H3ATTN_OK;
  if (!src || !dst || !aligned4(src) || !aligned4(dst)) return fail(H3ATTN_EINVAL, "src and dst must be 4-byte aligned lists");
  if (n_groups < 0 || n_groups > INT32_MAX) return fail(H3ATTN_EINVAL, "n_groups must be in [0, 2^31) (got %lld)", (long long)n_groups);
  if (width < 1 || width > 256) return fail(H3ATTN_EUNSUPPORTED, "width must be in [1, 256] (got %d)", width);
  if (cache->num_kv_heads > 32767) return fail(H3ATTN_EUNSUPPORTED, "more than 32767 key heads");
  const uintptr_t bytes = (uintptr_t)n_groups * width * 4;
  if (overlaps_cache(cache, src, bytes) || overlaps_cache(cache, dst, bytes))
    return fail(H3ATTN_EINVAL, "a list overlaps the cache");
  int sms = 0;
  cudaError_t e = current_sms(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const CacheMoveArgs a{static_cast<__nv_bfloat16*>(cache->k), static_cast<__nv_bfloat16*>(cache->v), src, dst, n_groups,
                        width, cache->page_size, cache->n_pages * cache->page_size, cache->page_stride,
                        cache->token_stride, cache->head_stride};
  e = launch_cache_move(a, cache->num_kv_heads, static_cast<cudaStream_t>(cuda_stream));
  return e == cudaSuccess ? H3ATTN_OK : cuda_fail(e, "cache move launch");
}

// ------------------------------------------------------ causal attention ----

h3attn_status h3attn_plan_set_causal(h3attn_plan_t plan, int32_t num_kv_heads, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (h3attn_status s = check_kv_heads(plan->num_heads, num_kv_heads)) return s;
  CausalPlan& cp = plan->causal;
  if (cp.walk.set) return fail(H3ATTN_EINVAL, "the plan's causal list is already set");
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  try {
    cp.walk = WalkPlan();
    const std::string why = build_causal_walk(plan->cu_host.data(), plan->n_docs, plan->num_heads, num_kv_heads,
                                              forward_slots(plan->device, plan->num_sms), cp.walk);
    if (!why.empty()) return fail(H3ATTN_EINVAL, "%s", why.c_str());
    cp.kv_heads = num_kv_heads;
  } catch (const std::exception&) {
    return fail(H3ATTN_ENOMEM, "host allocation failed while building the causal list");
  }
  return attach_walk(&cp.walk, "causal", cuda_stream, [](cudaStream_t) { return cudaSuccess; });
}

namespace {

// Checks of q, o, softmax_scale and lse_out where k and v have heads of their own.
h3attn_status check_grouped_io(const Plan* plan, const void* q, int64_t q_row_stride, const void* o, int64_t o_row_stride,
                               float softmax_scale, const float* lse_out) {
  const int64_t S = plan->S;
  const Rows rq{"q", q, q_row_stride, plan->num_heads}, ro{"o", o, o_row_stride, plan->num_heads};
  if (h3attn_status s = check_rows(rq, S)) return s;
  if (h3attn_status s = check_rows(ro, S)) return s;
  if (lse_out && !aligned4(lse_out)) return fail(H3ATTN_EINVAL, "lse_out must be 4-byte aligned");
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f))
    return fail(H3ATTN_EINVAL, "softmax_scale must be finite and > 0");
  if (rows_overlap(ro, rq, S)) return fail(H3ATTN_EINVAL, "o overlaps q");
  if (lse_out) {
    const uintptr_t n = (uintptr_t)S * plan->num_heads * 4;
    if (ranges_overlap(lse_out, n, o, ro.bytes(S))) return fail(H3ATTN_EINVAL, "lse_out overlaps o");
    if (ranges_overlap(lse_out, n, q, rq.bytes(S))) return fail(H3ATTN_EINVAL, "lse_out overlaps q");
  }
  return H3ATTN_OK;
}

}  // namespace

h3attn_status h3attn_forward_causal(h3attn_plan_t plan, const void* q, int64_t q_row_stride, const void* k, const void* v,
                                    int64_t kv_row_stride, void* o, int64_t o_row_stride, float softmax_scale,
                                    float* lse_out, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  const CausalPlan& cp = plan->causal;
  if (!cp.walk.set) return fail(H3ATTN_EINVAL, "h3attn_plan_set_causal has not been called on this plan");
  if (h3attn_status s = check_grouped_io(plan, q, q_row_stride, o, o_row_stride, softmax_scale, lse_out)) return s;
  const int64_t S = plan->S;
  const Rows ro{"o", o, o_row_stride, plan->num_heads};
  for (const Rows& r : {Rows{"k", k, kv_row_stride, cp.kv_heads}, Rows{"v", v, kv_row_stride, cp.kv_heads}}) {
    if (h3attn_status s = check_rows(r, S)) return s;
    if (rows_overlap(ro, r, S)) return fail(H3ATTN_EINVAL, "o overlaps %s", r.name);
    if (lse_out && ranges_overlap(lse_out, (uintptr_t)S * plan->num_heads * 4, r.p, r.bytes(S)))
      return fail(H3ATTN_EINVAL, "lse_out overlaps %s", r.name);
  }
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  const ForwardArgs a = walk_forward_args(plan, cp.walk, q, k, v, q_row_stride, o, o_row_stride, softmax_scale, lse_out);
  WalkArgs w = walk_args(cp.walk);
  w.kv_heads = cp.kv_heads;
  w.kv_stride = kv_row_stride;
  w.pack = causal_pack(plan->num_heads / cp.kv_heads);
  std::string why;
  e = launch_forward_causal(a, w, static_cast<cudaStream_t>(cuda_stream), &why);
  if (e != cudaSuccess) {
    if (!why.empty()) return fail(H3ATTN_ECUDA, "causal forward: %s", why.c_str());
    return cuda_fail(e, "causal forward launch");
  }
  return H3ATTN_OK;
}

// ------------------------------------------------------- tree attention ----

h3attn_status h3attn_plan_set_tree(h3attn_plan_t plan, int32_t num_kv_heads, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (h3attn_status s = check_kv_heads(plan->num_heads, num_kv_heads)) return s;
  TreePlan& tp = plan->tree;
  if (tp.set) return fail(H3ATTN_EINVAL, "the plan's tree workspace is already set");
  if (plan->max_seqlen > kTreeMax)
    return fail(H3ATTN_EUNSUPPORTED, "a document of more than %d drafted tokens (%d)", kTreeMax, plan->max_seqlen);
  if (plan->n_docs > kTreeDocs) return fail(H3ATTN_EUNSUPPORTED, "more than %d documents (%d)", kTreeDocs, plan->n_docs);
  if (plan->S * plan->num_heads >= (int64_t(1) << 31)) return fail(H3ATTN_EUNSUPPORTED, "2^31 or more rows");
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  TreePlan t;
  t.kv_heads = num_kv_heads;
  const int32_t group = plan->num_heads / num_kv_heads;
  for (int32_t p = 1; p <= kKeyTile; ++p)
    if (group % p == 0) t.pack = p;
  t.toks = std::min(kKeyTile / t.pack, plan->max_seqlen);
  t.max_len = plan->max_seqlen;
  const int32_t qtiles = group / t.pack * ((plan->max_seqlen + t.toks - 1) / t.toks);
  t.slot_rows = qtiles > 1 ? 2 * kKeyTile : kKeyTile;
  int64_t items = 0;
  for (int32_t d = 0; d < plan->n_docs; ++d) {
    const int32_t T = plan->cu_host[d + 1] - plan->cu_host[d];
    items += ((int64_t)(group / t.pack) * ((T + t.toks - 1) / t.toks) + 1) / 2 * num_kv_heads;
  }
  if (items >= (int64_t(1) << 24)) return fail(H3ATTN_EUNSUPPORTED, "2^24 or more items (sequences times key heads times row tiles)");
  t.items = (int32_t)items;
  t.grid = plan->num_sms;
  const size_t rows = (size_t)4 * t.grid * kKeyTile;  // (two slots of two tiles a block, or of one tile a stream)
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  std::vector<TreeRow> token;
  std::vector<int32_t> item0;
  try {
    token.resize((size_t)plan->S);
    item0.resize((size_t)plan->n_docs);
  } catch (const std::exception&) {
    return fail(H3ATTN_ENOMEM, "host allocation failed for the tree workspace");
  }
  const int32_t packs = group / t.pack;
  for (int32_t d = 0, item = 0; d < plan->n_docs; ++d) {
    const int32_t b = plan->cu_host[d], T = plan->cu_host[d + 1] - b, units = (packs * ((T + t.toks - 1) / t.toks) + 1) / 2;
    for (int32_t i = 0; i < T; ++i) token[(size_t)(b + i)] = TreeRow{item, i / t.toks * packs, i % t.toks, units};
    item0[d] = item;
    item += units * num_kv_heads;
  }
  e = cudaMalloc(&t.d_rows, token.size() * sizeof(TreeRow));
  if (e == cudaSuccess) e = cudaMalloc(&t.d_item0, item0.size() * sizeof(int32_t));
  if (e == cudaSuccess) e = cudaMalloc(&t.d_joins, (size_t)t.items * sizeof(int2));
  if (e == cudaSuccess) e = cudaMalloc(&t.d_part_o, rows * kHeadDim * sizeof(float));
  if (e == cudaSuccess) e = cudaMalloc(&t.d_part_ml, rows * sizeof(float2));
  // (no pieces: a forward whose wait runs out leaves the entries of the items that it did not reach)
  if (e == cudaSuccess) e = cudaMemsetAsync(t.d_joins, 0, (size_t)t.items * sizeof(int2), st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(t.d_item0, item0.data(), item0.size() * sizeof(int32_t), cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(t.d_rows, token.data(), token.size() * sizeof(TreeRow), cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) {
    free_tree(&t);
    return e == cudaErrorMemoryAllocation ? fail(H3ATTN_ENOMEM, "cudaMalloc failed for the plan's tree workspace")
                                          : cuda_fail(e, "tree");
  }
  t.set = true;
  tp = t;
  return H3ATTN_OK;
}

namespace {

// What the tree forward and its join have of the plan and the outputs.
TreeArgs tree_args(const Plan* plan, void* o, int64_t o_row_stride, float* lse_out) {
  const TreePlan& tp = plan->tree;
  TreeArgs a{};
  a.cu = plan->d_cu;
  a.rows = tp.d_rows;
  a.S = plan->S;
  a.n_docs = plan->n_docs;
  a.H = plan->num_heads;
  a.kv_heads = tp.kv_heads;
  a.group = plan->num_heads / tp.kv_heads;
  a.pack = tp.pack;
  a.toks = tp.toks;
  a.packs = a.group / tp.pack;
  a.slot_rows = tp.slot_rows;
  a.grid = tp.grid;
  a.items = tp.items;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.o_stride = o_row_stride;
  a.lse = lse_out;
  a.item0 = tp.d_item0;
  a.joins = tp.d_joins;
  a.part_o = tp.d_part_o;
  a.part_ml = tp.d_part_ml;
  a.err = plan->d_err;
  return a;
}

}  // namespace

h3attn_status h3attn_forward_tree(h3attn_plan_t plan, const void* q, int64_t q_row_stride, const h3attn_cache* cache,
                                  const int32_t* page_table, int32_t table_width, const int32_t* ctx_lens,
                                  const uint64_t* tree_mask, void* o, int64_t o_row_stride, float softmax_scale,
                                  float* lse_out, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  const TreePlan& tp = plan->tree;
  if (!tp.set) return fail(H3ATTN_EINVAL, "h3attn_plan_set_tree has not been called on this plan");
  if (h3attn_status s = check_grouped_io(plan, q, q_row_stride, o, o_row_stride, softmax_scale, lse_out)) return s;
  if (h3attn_status s = check_cache(cache)) return s;
  if (cache->num_kv_heads != tp.kv_heads)
    return fail(H3ATTN_EINVAL, "the cache has %d key heads, the plan %d", cache->num_kv_heads, tp.kv_heads);
  if (!page_table || !ctx_lens || !aligned4(page_table) || !aligned4(ctx_lens) ||
      (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
    return fail(H3ATTN_EINVAL, "page_table and ctx_lens must be 4-byte aligned, tree_mask 8-byte aligned lists");
  if (table_width < 1 || (int64_t)table_width * cache->page_size > INT32_MAX - kKeyTile ||
      (int64_t)table_width * cache->page_size < tp.max_len)
    return fail(H3ATTN_EINVAL, "table_width must hold the drafts and less than 2^31 - 128 rows (got %d pages of %d)", table_width,
                cache->page_size);
  const int64_t S = plan->S;
  const uintptr_t o_bytes = Rows{"o", o, o_row_stride, plan->num_heads}.bytes(S), lse_bytes = (uintptr_t)S * plan->num_heads * 4;
  struct List {
    const void* p;
    uintptr_t bytes;
  };
  for (const List& x : {List{page_table, (uintptr_t)plan->n_docs * table_width * 4}, List{ctx_lens, (uintptr_t)plan->n_docs * 4},
                        List{tree_mask, tree_mask ? (uintptr_t)S * 8 : 0}})
    if (x.p && (ranges_overlap(o, o_bytes, x.p, x.bytes) || (lse_out && ranges_overlap(lse_out, lse_bytes, x.p, x.bytes))))
      return fail(H3ATTN_EINVAL, "o or lse_out overlaps a list");
  if (overlaps_cache(cache, o, o_bytes) || (lse_out && overlaps_cache(cache, lse_out, lse_bytes)))
    return fail(H3ATTN_EINVAL, "o or lse_out overlaps the cache");
  if (cache->page_size % 8) return fail(H3ATTN_EUNSUPPORTED, "page_size must be a multiple of 8 (got %d)", cache->page_size);
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  TreeArgs a = tree_args(plan, o, o_row_stride, lse_out);
  a.ctx_lens = ctx_lens;
  a.page_table = page_table;
  a.tree_mask = tree_mask;
  a.table_width = table_width;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  std::string why;
  e = launch_attn_tree(a, q, q_row_stride, *cache, static_cast<cudaStream_t>(cuda_stream), &why);
  if (e != cudaSuccess) {
    if (!why.empty()) return fail(H3ATTN_ECUDA, "tree forward: %s", why.c_str());
    return cuda_fail(e, "tree forward launch");
  }
  return H3ATTN_OK;
}

h3attn_status h3attn_get_device_error(h3attn_plan_t plan, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if ((e = cudaStreamSynchronize(st)) != cudaSuccess) return cuda_fail(e, "stream synchronize");
  uint32_t word = 0;
  if ((e = cudaMemcpy(&word, plan->d_err, sizeof(word), cudaMemcpyDeviceToHost)) != cudaSuccess)
    return cuda_fail(e, "read device error word");
  if (word == kErrNone) return H3ATTN_OK;
  cudaMemset(plan->d_err, 0, sizeof(word));
  if (word == kErrTimeout)
    return fail(H3ATTN_ETIMEOUT, "a bounded device wait ran out; the outputs of that call are invalid");
  if (word == kErrPage)
    return fail(H3ATTN_EINVAL, "a sequence of the tree forward names a page outside the cache, or a length outside its table");
  if (word == kErrBlockIndex)
    return fail(H3ATTN_EINVAL, "a list of the sparse forward names a key tile outside its document (skipped)");
  return fail(H3ATTN_ECUDA, "device error word 0x%x", word);
}

h3attn_status h3attn_selftest_bounded_wait(uint64_t timeout_ns, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_wait_limit(timeout_ns)) return s;
  clear_runtime_error();
  uint32_t* d_flag = nullptr;
  cudaError_t e = cudaMalloc(&d_flag, sizeof(uint32_t));
  if (e != cudaSuccess) return cuda_fail(e, "cudaMalloc");
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  uint32_t word = 0;
  if ((e = cudaMemsetAsync(d_flag, 0, sizeof(uint32_t), st)) == cudaSuccess &&
      (e = launch_selftest_bounded_wait(timeout_ns, d_flag, st)) == cudaSuccess &&
      (e = cudaStreamSynchronize(st)) == cudaSuccess)
    e = cudaMemcpy(&word, d_flag, sizeof(word), cudaMemcpyDeviceToHost);
  cudaFree(d_flag);
  if (e != cudaSuccess) return cuda_fail(e, "selftest");
  if (word == kErrTimeout) return fail(H3ATTN_ETIMEOUT, "bounded wait ran out (expected)");
  return fail(H3ATTN_ECUDA, "bounded wait did not report a timeout (word 0x%x)", word);
}

h3attn_status h3attn_selftest_plan_wait(h3attn_plan_t plan, uint64_t timeout_ns, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (h3attn_status s = check_wait_limit(timeout_ns)) return s;
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  e = launch_selftest_bounded_wait(timeout_ns, plan->d_err, static_cast<cudaStream_t>(cuda_stream));
  return e == cudaSuccess ? H3ATTN_OK : cuda_fail(e, "selftest launch");
}

h3attn_status h3attn_selftest_tree_join(h3attn_plan_t plan, const int32_t* joins, int64_t n_joins, void* o, int64_t o_row_stride,
                                        float* lse_out, void* cuda_stream) {
  clear_error();
  if (h3attn_status s = check_plan(plan)) return s;
  if (!plan->tree.set) return fail(H3ATTN_EINVAL, "h3attn_plan_set_tree has not been called on this plan");
  const Rows ro{"o", o, o_row_stride, plan->num_heads};
  if (h3attn_status s = check_rows(ro, plan->S)) return s;
  if (!aligned4(lse_out) || (reinterpret_cast<uintptr_t>(joins) & 7u))
    return fail(H3ATTN_EINVAL, "lse_out must be 4-byte and joins 8-byte aligned");
  if (joins && n_joins != plan->tree.items)
    return fail(H3ATTN_EINVAL, "joins must have an entry for each of the %d items (got %lld)", plan->tree.items, (long long)n_joins);
  DeviceGuard g;
  cudaError_t e = g.enter(plan->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  TreeArgs a = tree_args(plan, o, o_row_stride, lse_out);
  if (joins) a.joins = reinterpret_cast<int2*>(const_cast<int32_t*>(joins));  // (the join reads it)
  std::string why;
  e = launch_tree_join(a, static_cast<cudaStream_t>(cuda_stream), &why);
  return e == cudaSuccess ? H3ATTN_OK : cuda_fail(e, "selftest launch");
}

}  // extern "C"
