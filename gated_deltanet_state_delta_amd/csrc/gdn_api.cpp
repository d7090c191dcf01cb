// gdn_api.cpp -- the C ABI of libgdn: argument validation and dispatch.
//
// Everything checked here is host-visible metadata (pointers, sizes, strides,
// dtypes).  No device memory is read and nothing is synchronised, so every
// entry point can be captured in a HIP graph.  Data-dependent conditions
// (cu_seqlens contents, slot indices) are handled on the device as the pages
// prescribe: clamping and skipping, never faulting.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/libgdn.h"
#include "gdn_kernels.hpp"
#include "gdn_paged.hpp"

namespace {

thread_local char g_err[512] = "";

gdn_status fail(gdn_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return s;
}

gdn_status from_hip(hipError_t e, const char* what) {
  if (e == hipSuccess) return GDN_OK;
  return fail(GDN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// Static device scratch of gdn_prefill_noalloc: one copy per device, held
// until the process ends.  In host code `scratch` names a host-side stand-in,
// not device memory: only the address hipGetSymbolAddress returns for the
// current device is ever passed to a kernel.
static __device__ __align__(256) unsigned char scratch[GDN_NOALLOC_SCRATCH_BYTES];

// The current device's address of `scratch`, looked up once per device (with
// that device current) and kept.
hipError_t noalloc_scratch(void** out) {
  constexpr int kMaxDevices = 64;
  static std::atomic<void*> cache[kMaxDevices];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  void* ptr = cache[dev].load(std::memory_order_acquire);
  if (!ptr) {
    e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return e;
    if (!ptr) return hipErrorInvalidSymbol;
    cache[dev].store(ptr, std::memory_order_release);
  }
  *out = ptr;
  return hipSuccess;
}

bool head_size_ok(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p % n) == 0; }
size_t elem_size(int32_t dt) { return dt == GDN_BF16 ? 2 : 4; }
size_t cache_elem(int32_t dt) { return dt == GDN_E4M3 || dt == GDN_I8 ? 1 : elem_size(dt); }

}  // namespace

extern "C" {

const char* gdn_last_error(void) { return g_err; }

const char* gdn_version(void) { return "0.1.0"; }

const char* gdn_header_digest(void) { return GDN_HEADER_DIGEST; }  // (the build defines it)

gdn_status gdn_gate(const float* A_log, const float* dt_bias, const void* a, const void* b,
                    int32_t ab_dtype, int64_t n_tokens, int32_t hv, float* log_decay_out,
                    float* gamma_out, float* beta_out, void* stream) {
  g_err[0] = 0;
  if (ab_dtype != GDN_F32 && ab_dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "gdn_gate: ab_dtype %d", ab_dtype);
  if (n_tokens < 0 || hv <= 0) return fail(GDN_ERR_SHAPE, "gdn_gate: n_tokens=%lld hv=%d", (long long)n_tokens, hv);
  if ((log_decay_out || gamma_out) && !a) return fail(GDN_ERR_NULL, "gdn_gate: decay output requested without a");
  if (beta_out && !b) return fail(GDN_ERR_NULL, "gdn_gate: beta output requested without b");
  if (a && (!A_log || !dt_bias)) return fail(GDN_ERR_NULL, "gdn_gate: a given without A_log / dt_bias");
  if (n_tokens == 0) return GDN_OK;
  // an input whose outputs are all absent is ignored
  const void* ua = (log_decay_out || gamma_out) ? a : nullptr;
  const void* ub = beta_out ? b : nullptr;
  if (!ua && !ub) return GDN_OK;
  return from_hip(gdn::launch_gate(A_log, dt_bias, ua, ub, ab_dtype, n_tokens, hv, log_decay_out,
                                   gamma_out, beta_out, (hipStream_t)stream),
                  "gdn_gate launch");
}

gdn_status gdn_wait_timeouts(uint32_t* count, int32_t clear) {
  g_err[0] = 0;
  if (!count) return fail(GDN_ERR_NULL, "gdn_wait_timeouts: count is NULL");
  return from_hip(gdn::wait_timeouts(count, clear != 0), "gdn_wait_timeouts");
}

size_t gdn_prefill_workspace_size(const gdn_prefill_args* args) {
  return args ? gdn::prefill_workspace_bytes(*args) : 0;
}

// Every host-visible check of a gdn_prefill call, in order; *noop is set
// when the call is valid and has nothing to do (n_seqs == 0).
static gdn_status prefill_check(const gdn_prefill_args& a, bool* noop) {
  *noop = false;
  if (a.io_dtype != GDN_F32 && a.io_dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "gdn_prefill: io_dtype %d", a.io_dtype);
  if (a.decay_kind != GDN_DECAY_LOG && a.decay_kind != GDN_DECAY_GAMMA)
    return fail(GDN_ERR_DTYPE, "gdn_prefill: decay_kind %d", a.decay_kind);
  if (a.n_seqs < 0 || a.total_tokens < 0 || a.hq <= 0 || a.hv <= 0 || a.dk <= 0 || a.dv <= 0)
    return fail(GDN_ERR_SHAPE, "gdn_prefill: bad sizes n_seqs=%d T=%lld hq=%d hv=%d dk=%d dv=%d", a.n_seqs,
                (long long)a.total_tokens, a.hq, a.hv, a.dk, a.dv);
  if (a.hv % a.hq != 0) return fail(GDN_ERR_SHAPE, "gdn_prefill: hv=%d is not a multiple of hq=%d", a.hv, a.hq);
  if (!head_size_ok(a.dk) || !head_size_ok(a.dv))
    return fail(GDN_ERR_UNSUPPORTED, "gdn_prefill: dk=%d dv=%d (supported: 16, 32, 64, 128)", a.dk, a.dv);
  if (a.chunk_size != 0 && a.chunk_size != 16 && a.chunk_size != 32 && a.chunk_size != 64)
    return fail(GDN_ERR_UNSUPPORTED, "gdn_prefill: chunk_size=%d (supported: 0, 16, 32, 64)", a.chunk_size);
  if (!a.cu_seqlens && (a.seq_len < 0 || (int64_t)a.n_seqs * a.seq_len != a.total_tokens))
    return fail(GDN_ERR_SHAPE, "gdn_prefill: without cu_seqlens n_seqs*seq_len (%d*%d) must equal total_tokens %lld",
                a.n_seqs, a.seq_len, (long long)a.total_tokens);
  if (a.qk_l2norm && !(a.qk_l2norm_eps >= 0.f && a.qk_l2norm_eps <= 3.0e38f))
    return fail(GDN_ERR_SHAPE, "gdn_prefill: qk_l2norm_eps must be finite and >= 0");
  if (a.update_rule < GDN_RULE_GATED_DELTA || a.update_rule > GDN_RULE_LINEAR)
    return fail(GDN_ERR_DTYPE, "gdn_prefill: update_rule %d", a.update_rule);
  if ((int64_t)a.total_tokens * a.hv >= (int64_t(1) << 31))
    return fail(GDN_ERR_SHAPE, "gdn_prefill: total_tokens * hv must be below 2^31");
  if (a.total_tokens > 0) {
    // gate sources: present exactly for the rules that use them (not read
    // at all when there are no tokens)
    const bool uses_decay = a.update_rule == GDN_RULE_GATED_DELTA || a.update_rule == GDN_RULE_GATED;
    const bool uses_beta = a.update_rule == GDN_RULE_GATED_DELTA || a.update_rule == GDN_RULE_DELTA;
    const bool has_decay = a.decay || a.gate_a, has_beta = a.beta || a.gate_b;
    if (a.decay && a.gate_a) return fail(GDN_ERR_SHAPE, "gdn_prefill: decay and gate_a are both given");
    if (a.beta && a.gate_b) return fail(GDN_ERR_SHAPE, "gdn_prefill: beta and gate_b are both given");
    if (has_decay != uses_decay)
      return fail(uses_decay ? GDN_ERR_NULL : GDN_ERR_SHAPE, "gdn_prefill: update_rule %d %s a decay input",
                  a.update_rule, uses_decay ? "needs" : "takes no");
    if (has_beta != uses_beta)
      return fail(uses_beta ? GDN_ERR_NULL : GDN_ERR_SHAPE, "gdn_prefill: update_rule %d %s a beta input",
                  a.update_rule, uses_beta ? "needs" : "takes no");
  }
  if (a.gate_a && (!a.A_log || !a.dt_bias)) return fail(GDN_ERR_NULL, "gdn_prefill: gate_a needs A_log and dt_bias");
  if (a.decay_per_key && a.gate_a)
    return fail(GDN_ERR_UNSUPPORTED, "gdn_prefill: decay_per_key takes the decay as a given input (not gate_a)");
  if (a.decay_per_key && a.update_rule != GDN_RULE_GATED_DELTA && a.update_rule != GDN_RULE_GATED)
    return fail(GDN_ERR_SHAPE, "gdn_prefill: decay_per_key needs an update_rule with a decay (gated_delta, gated)");
  if (a.state_pool) {
    if (a.initial_state || a.final_state)
      return fail(GDN_ERR_SHAPE, "gdn_prefill: state_pool replaces initial_state and final_state (pass NULL)");
    if (a.pool_size < 0) return fail(GDN_ERR_SHAPE, "gdn_prefill: pool_size=%d", a.pool_size);
    if (!aligned(a.state_pool, 16) || a.pool_slot_stride % 4 != 0 || a.pool_head_stride % 4 != 0 ||
        a.pool_slot_stride < 0 || a.pool_head_stride < 0)
      return fail(GDN_ERR_LAYOUT, "gdn_prefill: state_pool must be 16-byte aligned with strides multiple of 4 elements");
    if (a.pool_head_stride < (int64_t)a.dv * a.dk ||
        a.pool_slot_stride < (int64_t)(a.hv - 1) * a.pool_head_stride + (int64_t)a.dv * a.dk)
      return fail(GDN_ERR_LAYOUT, "gdn_prefill: pool strides smaller than the dense extents");
  } else if (a.read_slot || a.write_slot) {
    return fail(GDN_ERR_SHAPE, "gdn_prefill: read_slot / write_slot need state_pool");
  }
  if (a.n_seqs == 0) {
    *noop = true;
    return GDN_OK;
  }
  if (!a.final_state && !a.state_pool) return fail(GDN_ERR_NULL, "gdn_prefill: final_state is NULL");
  if (a.total_tokens > 0 && (!a.q || !a.k || !a.v || !a.out))
    return fail(GDN_ERR_NULL, "gdn_prefill: q, k, v and out are required");
  const void* ptrs[] = {a.q, a.k, a.v, a.out, a.decay, a.beta, a.initial_state, a.final_state, a.cu_seqlens,
                        a.state_pool};
  for (const void* q : ptrs)
    if (q && !aligned(q, 16)) return fail(GDN_ERR_LAYOUT, "gdn_prefill: pointers must be 16-byte aligned");
  const int64_t strides[] = {a.q_stride_token, a.q_stride_head, a.k_stride_token, a.k_stride_head,
                             a.v_stride_token, a.v_stride_head, a.out_stride_token, a.out_stride_head};
  // The kernels form in-chunk row offsets (up to 63 rows of a stride, in bytes
  // of fp32 at most) in 32-bit arithmetic: strides below 2^23 elements keep
  // 63 * stride * 4 plus a row's extent below 2^31.
  for (int64_t s : strides)
    if (s < 0 || s % 8 != 0 || s >= (int64_t(1) << 23))
      return fail(GDN_ERR_LAYOUT, "gdn_prefill: strides must be non-negative multiples of 8 elements below 2^23");
  if (a.total_tokens > 0) {
    if (a.q_stride_head < a.dk || a.k_stride_head < a.dk || a.v_stride_head < a.dv || a.out_stride_head < a.dv ||
        a.q_stride_token < (int64_t)a.hq * a.dk || a.k_stride_token < (int64_t)a.hq * a.dk ||
        a.v_stride_token < (int64_t)a.hv * a.dv || a.out_stride_token < (int64_t)a.hv * a.dv)
      return fail(GDN_ERR_LAYOUT, "gdn_prefill: strides smaller than the dense extents");
  }
  if (a.initial_state && a.initial_state != a.final_state) {
    const char* i0 = (const char*)a.initial_state;
    const char* f0 = (const char*)a.final_state;
    const size_t bytes = (size_t)a.n_seqs * a.hv * a.dv * a.dk * sizeof(float);
    if (i0 < f0 + bytes && f0 < i0 + bytes)
      return fail(GDN_ERR_LAYOUT, "gdn_prefill: initial_state and final_state partially overlap");
  }
  return GDN_OK;
}

gdn_status gdn_prefill(const gdn_prefill_args* p, void* stream) {
  g_err[0] = 0;
  if (!p) return fail(GDN_ERR_NULL, "gdn_prefill: args is NULL");
  bool noop = false;
  const gdn_status st = prefill_check(*p, &noop);
  if (st != GDN_OK || noop) return st;
  return from_hip(gdn::launch_prefill(*p, (hipStream_t)stream), "gdn_prefill launch");
}

gdn_status gdn_prefill_noalloc(const gdn_prefill_args* p, void* stream) {
  g_err[0] = 0;
  if (!p) return fail(GDN_ERR_NULL, "gdn_prefill_noalloc: args is NULL");
  bool noop = false;
  const gdn_status st = prefill_check(*p, &noop);
  if (st != GDN_OK || noop) return st;
  const size_t need = gdn::prefill_workspace_bytes(*p);
  if (need > (size_t)GDN_NOALLOC_SCRATCH_BYTES)
    return fail(GDN_ERR_UNSUPPORTED,
                "gdn_prefill_noalloc: the call needs %zu bytes of scratch, more than the %zu of the static array "
                "(use gdn_prefill with a workspace)",
                need, (size_t)GDN_NOALLOC_SCRATCH_BYTES);
  gdn_prefill_args a = *p;
  a.workspace = nullptr;
  a.workspace_bytes = 0;
  if (need > 0) {
    void* ptr = nullptr;
    const hipError_t e = noalloc_scratch(&ptr);
    if (e != hipSuccess) return from_hip(e, "gdn_prefill_noalloc: static scratch address");
    a.workspace = ptr;
    a.workspace_bytes = GDN_NOALLOC_SCRATCH_BYTES;
  }
  return from_hip(gdn::launch_prefill(a, (hipStream_t)stream), "gdn_prefill_noalloc launch");
}

gdn_status gdn_decode(const gdn_decode_args* p, void* stream) {
  g_err[0] = 0;
  if (!p) return fail(GDN_ERR_NULL, "gdn_decode: args is NULL");
  const gdn_decode_args& a = *p;
  if (a.io_dtype != GDN_F32 && a.io_dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "gdn_decode: io_dtype %d", a.io_dtype);
  if (a.batch < 0 || a.T <= 0 || a.hq <= 0 || a.hv <= 0 || a.dk <= 0 || a.dv <= 0 || a.pool_size < 0)
    return fail(GDN_ERR_SHAPE, "gdn_decode: bad sizes batch=%d T=%d hq=%d hv=%d dk=%d dv=%d pool_size=%d", a.batch,
                a.T, a.hq, a.hv, a.dk, a.dv, a.pool_size);
  if (a.T > 64) return fail(GDN_ERR_UNSUPPORTED, "gdn_decode: T=%d (supported 1..64)", a.T);
  if (a.n_householder < 1 || a.n_householder > 4)
    return fail(GDN_ERR_UNSUPPORTED, "gdn_decode: n_householder=%d (supported 1..4)", a.n_householder);
  if (a.hv % a.hq != 0) return fail(GDN_ERR_SHAPE, "gdn_decode: hv=%d is not a multiple of hq=%d", a.hv, a.hq);
  if (a.hv > 65536) return fail(GDN_ERR_UNSUPPORTED, "gdn_decode: hv=%d (supported up to 65536)", a.hv);
  if (a.qk_l2norm && !(a.qk_l2norm_eps >= 0.f && a.qk_l2norm_eps <= 3.0e38f))
    return fail(GDN_ERR_SHAPE, "gdn_decode: qk_l2norm_eps must be finite and >= 0");
  if (!head_size_ok(a.dk) || !head_size_ok(a.dv))
    return fail(GDN_ERR_UNSUPPORTED, "gdn_decode: dk=%d dv=%d (supported: 16, 32, 64, 128)", a.dk, a.dv);
  if (a.scatter_idx && a.disable_state_update)
    return fail(GDN_ERR_UNSUPPORTED, "gdn_decode: scatter_idx requires disable_state_update == 0");
  if (a.batch == 0) return GDN_OK;
  if (!a.q || !a.k || !a.v || !a.b || !a.pool || !a.read_idx || !a.out)
    return fail(GDN_ERR_NULL, "gdn_decode: q, k, v, b, pool, read_idx and out are required");
  if (!a.decay_per_key && (!a.A_log || !a.dt_bias || !a.a))
    return fail(GDN_ERR_NULL, "gdn_decode: A_log, dt_bias and a are required (or decay_per_key)");
  if (a.decay_per_key && !aligned(a.decay_per_key, 16))
    return fail(GDN_ERR_LAYOUT, "gdn_decode: decay_per_key must be 16-byte aligned");
  if (!aligned(a.pool, 16) || a.pool_slot_stride % 4 != 0 || a.pool_head_stride % 4 != 0 ||
      a.pool_slot_stride < 0 || a.pool_head_stride < 0)
    return fail(GDN_ERR_LAYOUT, "gdn_decode: pool must be 16-byte aligned with strides multiple of 4 elements");
  if (a.pool_head_stride < (int64_t)a.dv * a.dk || a.pool_slot_stride < (int64_t)(a.hv - 1) * a.pool_head_stride + (int64_t)a.dv * a.dk)
    return fail(GDN_ERR_LAYOUT, "gdn_decode: pool strides smaller than the dense extents");
  const size_t es = elem_size(a.io_dtype);
  const void* act[] = {a.q, a.k, a.v, a.out};
  for (const void* q : act)
    if (!aligned(q, es == 2 ? 8 : 16)) return fail(GDN_ERR_LAYOUT, "gdn_decode: q, k, v, out must be aligned to 4 elements");
  return from_hip(gdn::launch_decode(a, (hipStream_t)stream), "gdn_decode launch");
}

gdn_status gdn_conv1d(const gdn_conv1d_args* p, void* stream) {
  g_err[0] = 0;
  if (!p) return fail(GDN_ERR_NULL, "gdn_conv1d: args is NULL");
  const gdn_conv1d_args& a = *p;
  if (a.io_dtype != GDN_F32 && a.io_dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "gdn_conv1d: io_dtype %d", a.io_dtype);
  if (a.total_tokens < 0 || a.conv_dim <= 0 || a.n_seqs < 0 || a.max_slots < 0)
    return fail(GDN_ERR_SHAPE, "gdn_conv1d: bad sizes T=%lld conv_dim=%d n_seqs=%d max_slots=%d",
                (long long)a.total_tokens, a.conv_dim, a.n_seqs, a.max_slots);
  if (a.kernel_size < 1 || a.kernel_size > 8)
    return fail(GDN_ERR_UNSUPPORTED, "gdn_conv1d: kernel_size=%d (supported 1..8)", a.kernel_size);
  const int64_t ve = a.io_dtype == GDN_BF16 ? 8 : 4;
  if (a.conv_dim % ve != 0)
    return fail(GDN_ERR_LAYOUT, "gdn_conv1d: conv_dim=%d is not a multiple of %lld elements", a.conv_dim, (long long)ve);
  if (a.n_seqs == 0 || a.total_tokens == 0) return GDN_OK;
  if (!a.x || !a.weight || !a.slot_idx || !a.row_offsets || !a.out || (a.kernel_size > 1 && !a.conv_state))
    return fail(GDN_ERR_NULL, "gdn_conv1d: x, weight, slot_idx, row_offsets, out (and conv_state for kernel_size > 1) are required");
  if (a.x_stride_token < a.conv_dim || a.out_stride_token < a.conv_dim || a.x_stride_token % ve != 0 ||
      a.out_stride_token % ve != 0)
    return fail(GDN_ERR_LAYOUT, "gdn_conv1d: row strides must be >= conv_dim and multiples of %lld elements", (long long)ve);
  if (!aligned(a.x, 16) || !aligned(a.out, 16) || !aligned(a.conv_state, 16))
    return fail(GDN_ERR_LAYOUT, "gdn_conv1d: x, out and conv_state must be 16-byte aligned");
  {
    const size_t es = elem_size(a.io_dtype);
    const uintptr_t x0 = (uintptr_t)a.x, o0 = (uintptr_t)a.out;
    const uintptr_t x1 = x0 + ((size_t)(a.total_tokens - 1) * a.x_stride_token + a.conv_dim) * es;
    const uintptr_t o1 = o0 + ((size_t)(a.total_tokens - 1) * a.out_stride_token + a.conv_dim) * es;
    if (x0 < o1 && o0 < x1) return fail(GDN_ERR_LAYOUT, "gdn_conv1d: out overlaps x");
  }
  return from_hip(gdn::launch_conv1d(a, (hipStream_t)stream), "gdn_conv1d launch");
}

// What the calls over a paged cache share: types and sizes.
static gdn_status cache_sizes(const char* f, int32_t batch, int32_t hkv, int32_t d, int32_t io_dtype,
                              int32_t cache_dtype, int32_t n_pages, int32_t page_size, int32_t max_pages) {
  if (io_dtype != GDN_F32 && io_dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "%s: io_dtype %d", f, io_dtype);
  if (cache_dtype != io_dtype && cache_dtype != GDN_E4M3 && cache_dtype != GDN_I8)
    return fail(GDN_ERR_DTYPE, "%s: cache_dtype %d (io_dtype's type, GDN_E4M3 or GDN_I8)", f, cache_dtype);
  if (batch < 0 || hkv <= 0 || d <= 0 || n_pages < 0 || page_size <= 0 || max_pages < 0)
    return fail(GDN_ERR_SHAPE, "%s: bad sizes batch=%d hkv=%d d=%d n_pages=%d page_size=%d max_pages=%d", f, batch,
                hkv, d, n_pages, page_size, max_pages);
  if (d != 32 && d != 64 && d != 128 && d != 256)
    return fail(GDN_ERR_UNSUPPORTED, "%s: d=%d (supported: 32, 64, 128, 256)", f, d);
  // page_size by itself too: max_pages may be 0
  if (page_size > (1 << 30) || (int64_t)max_pages * page_size > (int64_t(1) << 30))
    return fail(GDN_ERR_UNSUPPORTED, "%s: page_size and max_pages * page_size must be at most 2^30", f);
  return GDN_OK;
}

// The tokens of a block of block scales, 0 without them.
static gdn_status block_size(const char* f, int32_t cache_dtype, int32_t page_size, int32_t block) {
  if (block < 0) return fail(GDN_ERR_SHAPE, "%s: scale_block=%d", f, block);
  if (block == 0) return GDN_OK;
  if (cache_dtype != GDN_E4M3 && cache_dtype != GDN_I8)
    return fail(GDN_ERR_SHAPE, "%s: block scales are for 8-bit caches", f);
  if (block > page_size || page_size % block != 0)
    return fail(GDN_ERR_SHAPE, "%s: scale_block=%d does not divide page_size=%d", f, block, page_size);
  if (block > 65536) return fail(GDN_ERR_UNSUPPORTED, "%s: scale_block=%d (supported up to 65536)", f, block);
  return GDN_OK;
}

// The scales of a cache: a factor a head, or block scales.
static gdn_status scales_check(const char* f, int32_t cache_dtype, int32_t n_pages, int32_t page_size, const float* k_scale,
                               const float* v_scale, int32_t block, const float* k_blocks, const float* v_blocks) {
  const gdn_status st = block_size(f, cache_dtype, page_size, block);
  if (st != GDN_OK) return st;
  if (block == 0) {
    if (k_blocks || v_blocks) return fail(GDN_ERR_SHAPE, "%s: block scales need scale_block", f);
    if (cache_dtype == GDN_I8) return fail(GDN_ERR_NULL, "%s: an int8 cache needs block scales", f);
    if (cache_dtype == GDN_E4M3 && (!k_scale || !v_scale))
      return fail(GDN_ERR_NULL, "%s: an e4m3 cache needs k_scale and v_scale", f);
    if (cache_dtype != GDN_E4M3 && (k_scale || v_scale))
      return fail(GDN_ERR_SHAPE, "%s: k_scale and v_scale are for e4m3 caches", f);
    return GDN_OK;
  }
  if (k_scale || v_scale) return fail(GDN_ERR_SHAPE, "%s: k_scale and v_scale with block scales", f);
  if (n_pages > 0 && (!k_blocks || !v_blocks)) return fail(GDN_ERR_NULL, "%s: k_block_scale and v_block_scale are required", f);
  if (!aligned(k_blocks, 4) || !aligned(v_blocks, 4))
    return fail(GDN_ERR_LAYOUT, "%s: block scales must be 4-byte aligned", f);
  return GDN_OK;
}

// What the calls over a paged cache share with its page table and scales (A: one of their argument structs).
extern "C++" template <typename A>
static gdn_status cache_check(const char* f, const A& a) {
  const gdn_status st = cache_sizes(f, a.batch, a.hkv, a.d, a.io_dtype, a.cache_dtype, a.n_pages, a.page_size, a.max_pages);
  if (st != GDN_OK) return st;
  if (a.page_table_stride < a.max_pages) return fail(GDN_ERR_LAYOUT, "%s: page_table_stride smaller than max_pages", f);
  return scales_check(f, a.cache_dtype, a.n_pages, a.page_size, a.k_scale, a.v_scale, a.scale_block, a.k_block_scale, a.v_block_scale);
}

// Strides of a [page, token, head, d] cache (es bytes an element): either
// order of tokens and heads inside a page, nothing smaller than dense.
static gdn_status cache_layout(const char* f, const void* base, int64_t page, int64_t token, int64_t head,
                               int32_t page_size, int32_t hkv, int32_t d, size_t es) {
  // the kernels' offsets inside a page are 32 bits over 16 tokens, 64 bits over heads and pages
  const int64_t unit = 16 / (int64_t)es, token_lim = int64_t(1) << 23, head_lim = int64_t(1) << 40;
  if (!aligned(base, 16) || page < 0 || page % unit != 0 || token % unit != 0 || head % unit != 0)
    return fail(GDN_ERR_LAYOUT, "%s: caches and their strides must be 16-byte aligned", f);
  if (token < d || head < d || token >= token_lim || head >= head_lim)
    return fail(GDN_ERR_LAYOUT, "%s: cache token strides must be in [d, 2^23), head strides must be in [d, 2^40)", f);
  // one of the two orders must keep every row apart
  if (token < (int64_t)(hkv - 1) * head + d && head < (int64_t)(page_size - 1) * token + d)
    return fail(GDN_ERR_LAYOUT, "%s: cache rows overlap", f);
  if (page < (int64_t)(page_size - 1) * token + (int64_t)(hkv - 1) * head + d)
    return fail(GDN_ERR_LAYOUT, "%s: cache page stride smaller than a page", f);
  return GDN_OK;
}

// The sizes that gdn_attn_decode takes beyond those of the caches.
static gdn_status attn_sizes(const char* f, const gdn_attn_decode_args& a) {
  if (a.T <= 0 || a.hq <= 0) return fail(GDN_ERR_SHAPE, "%s: bad sizes T=%d hq=%d", f, a.T, a.hq);
  if (a.T > 64) return fail(GDN_ERR_UNSUPPORTED, "%s: T=%d (supported 1..64)", f, a.T);
  if (a.hq % a.hkv != 0) return fail(GDN_ERR_SHAPE, "%s: hq=%d is not a multiple of hkv=%d", f, a.hq, a.hkv);
  if (a.hq > 65536) return fail(GDN_ERR_UNSUPPORTED, "%s: hq=%d (supported up to 65536)", f, a.hq);
  // Each size is below 2^31 and hq at most 2^16: in this order no product overflows 64 bits.
  if ((int64_t)a.batch * a.hq >= (int64_t(1) << 31) || (int64_t)a.batch * a.hq * a.T >= (int64_t(1) << 31))
    return fail(GDN_ERR_UNSUPPORTED, "%s: batch * hq * T must be below 2^31", f);
  // A wave takes 16 query rows or more of a row and key-value head, or a share of several rows; a workgroup's four
  // waves hold row tiles padded to less than twice their number.  So fewer than 2^22 workgroups (and 8 for the last
  // of the 8 XCDs), where a grid ends at 2^24 of 256 threads.
  if ((int64_t)a.batch * a.hkv * (((int64_t)a.T * (a.hq / a.hkv) + 15) / 16) > (int64_t(1) << 23))
    return fail(GDN_ERR_UNSUPPORTED, "%s: batch * hkv * ceil(T * hq / hkv / 16) must be at most 2^23", f);
  // the rows' tiles of 16 keys and more are counted in 32 bits
  if ((int64_t)a.batch * (((int64_t)a.max_pages * a.page_size + 15) / 16 + 1) >= (int64_t(1) << 31))
    return fail(GDN_ERR_UNSUPPORTED, "%s: batch * (max_pages * page_size / 16 + 1) must be below 2^31", f);
  return GDN_OK;
}

size_t gdn_attn_decode_workspace_size(const gdn_attn_decode_args* args) {
  static const char* f = "gdn_attn_decode_workspace_size";
  g_err[0] = 0;
  if (!args) return 0;
  const gdn_attn_decode_args& a = *args;
  // the split's arithmetic holds for sizes that the call takes
  if (cache_sizes(f, a.batch, a.hkv, a.d, a.io_dtype, a.cache_dtype, a.n_pages, a.page_size, a.max_pages) != GDN_OK ||
      block_size(f, a.cache_dtype, a.page_size, a.scale_block) != GDN_OK || attn_sizes(f, a) != GDN_OK)
    return 0;
  return gdn::attn_workspace_bytes(a);
}

gdn_status gdn_attn_decode(const gdn_attn_decode_args* p, void* stream) {
  static const char* f = "gdn_attn_decode";
  g_err[0] = 0;
  if (!p) return fail(GDN_ERR_NULL, "%s: args is NULL", f);
  const gdn_attn_decode_args& a = *p;
  gdn_status st = cache_check(f, a);
  if (st != GDN_OK) return st;
  st = attn_sizes(f, a);
  if (st != GDN_OK || a.batch == 0) return st;
  if (!a.q || !a.out || !a.lens || (a.max_pages > 0 && !a.page_table) || (a.n_pages > 0 && (!a.k_cache || !a.v_cache)))
    return fail(GDN_ERR_NULL, "%s: q, caches, page_table, lens and out are required", f);
  const size_t es = elem_size(a.io_dtype), ce = cache_elem(a.cache_dtype);
  if (!aligned(a.q, 16) || !aligned(a.out, 16)) return fail(GDN_ERR_LAYOUT, "%s: q and out must be 16-byte aligned", f);
  const int64_t unit = 16 / (int64_t)es;
  if (a.q_stride_row < 0 || a.q_stride_token < 0 || a.q_stride_head < 0 || a.q_stride_row % unit != 0 ||
      a.q_stride_token % unit != 0 || a.q_stride_head % unit != 0)
    return fail(GDN_ERR_LAYOUT, "%s: q strides must be non-negative multiples of 16 bytes", f);
  {
    const uintptr_t q0 = (uintptr_t)a.q, o0 = (uintptr_t)a.out;
    const uintptr_t q1 = q0 + ((size_t)(a.batch - 1) * a.q_stride_row + (size_t)(a.T - 1) * a.q_stride_token +
                               (size_t)(a.hq - 1) * a.q_stride_head + a.d) * es;
    if (q0 < o0 + (size_t)a.batch * a.T * a.hq * a.d * es && o0 < q1) return fail(GDN_ERR_LAYOUT, "%s: out overlaps q", f);
  }
  if (a.n_pages > 0) {
    st = cache_layout(f, a.k_cache, a.k_stride_page, a.k_stride_token, a.k_stride_head, a.page_size, a.hkv, a.d, ce);
    if (st != GDN_OK) return st;
    st = cache_layout(f, a.v_cache, a.v_stride_page, a.v_stride_token, a.v_stride_head, a.page_size, a.hkv, a.d, ce);
    if (st != GDN_OK) return st;
  }
  if (a.workspace && !aligned(a.workspace, 256)) return fail(GDN_ERR_LAYOUT, "%s: workspace must be 256-byte aligned", f);
  return from_hip(gdn::launch_attn_decode(a, (hipStream_t)stream), "gdn_attn_decode launch");
}

// What gdn_kv_append and gdn_kv_read check alike.  done: there is nothing to do.
extern "C++" template <typename A>
static gdn_status tokens_check(const char* f, const A& a, bool& done) {
  gdn_status st = cache_check(f, a);
  if (st != GDN_OK) return st;
  if (a.total_tokens < 0) return fail(GDN_ERR_SHAPE, "%s: total_tokens=%lld", f, (long long)a.total_tokens);
  if (a.hkv > 65536) return fail(GDN_ERR_UNSUPPORTED, "%s: hkv=%d (supported up to 65536)", f, a.hkv);
  if (a.total_tokens > (int64_t(1) << 28)) return fail(GDN_ERR_UNSUPPORTED, "%s: total_tokens must be at most 2^28", f);
  done = a.batch == 0 || a.total_tokens == 0;
  if (!done && !a.cu_seqlens && a.total_tokens % a.batch != 0)
    return fail(GDN_ERR_SHAPE, "%s: without cu_seqlens total_tokens %lld must be a multiple of batch %d", f,
                (long long)a.total_tokens, a.batch);
  return GDN_OK;
}
extern "C++" template <typename A>
static gdn_status tokens_layout(const char* f, const A& a) {
  const size_t es = elem_size(a.io_dtype), ce = cache_elem(a.cache_dtype);
  const int64_t unit = 16 / (int64_t)es;
  const int64_t strides[] = {a.k_stride_token, a.k_stride_head, a.v_stride_token, a.v_stride_head};
  if (!aligned(a.k, 16) || !aligned(a.v, 16)) return fail(GDN_ERR_LAYOUT, "%s: k and v must be 16-byte aligned", f);
  for (int64_t s : strides)
    if (s < 0 || s % unit != 0) return fail(GDN_ERR_LAYOUT, "%s: k and v strides must be non-negative multiples of 16 bytes", f);
  if (a.n_pages == 0) return GDN_OK;
  const gdn_status st =
      cache_layout(f, a.k_cache, a.kc_stride_page, a.kc_stride_token, a.kc_stride_head, a.page_size, a.hkv, a.d, ce);
  if (st != GDN_OK) return st;
  return cache_layout(f, a.v_cache, a.vc_stride_page, a.vc_stride_token, a.vc_stride_head, a.page_size, a.hkv, a.d, ce);
}

gdn_status gdn_kv_append(const gdn_kv_append_args* p, void* stream) {
  static const char* f = "gdn_kv_append";
  g_err[0] = 0;
  if (!p) return fail(GDN_ERR_NULL, "%s: args is NULL", f);
  const gdn_kv_append_args& a = *p;
  bool done = false;
  gdn_status st = tokens_check(f, a, done);
  if (st != GDN_OK || done) return st;
  if (a.n_pages == 0 || a.max_pages == 0) return GDN_OK;  // no page to write to
  if (!a.k || !a.v || !a.k_cache || !a.v_cache || !a.page_table || !a.lens)
    return fail(GDN_ERR_NULL, "%s: k, v, caches, page_table and lens are required", f);
  st = tokens_layout(f, a);
  if (st != GDN_OK) return st;
  if (a.scale_block == 0) return from_hip(gdn::launch_kv_append(a, (hipStream_t)stream), "gdn_kv_append launch");
  // its blocks are counted in 32 bits, 64 to a workgroup
  if (a.total_tokens / a.scale_block + 2 * (int64_t)a.batch >= (int64_t(1) << 29))
    return fail(GDN_ERR_UNSUPPORTED, "%s: total_tokens / scale_block + 2 * batch must be below 2^29", f);
  if (a.k_cache == a.v_cache || a.k_block_scale == a.v_block_scale)
    return fail(GDN_ERR_LAYOUT, "%s: one cache, or its block scales, for keys and values", f);
  return from_hip(gdn::launch_kv_quantise(a, (hipStream_t)stream), "gdn_kv_append launch");
}

// Whether rows of d elements, of so many tokens and heads, keep apart: one of the two strides holds all of the other's.
static bool rows_apart(int64_t tokens, int64_t token, int64_t heads, int64_t head, int64_t d) {
  typedef __int128 wide;  // strides are any int64
  const bool heads_inside = (heads == 1 || head >= d) && (tokens == 1 || token >= (wide)(heads - 1) * head + d);
  const bool tokens_inside = (tokens == 1 || token >= d) && (heads == 1 || head >= (wide)(tokens - 1) * token + d);
  return heads_inside || tokens_inside;
}

gdn_status gdn_kv_read(const gdn_kv_read_args* p, void* stream) {
  static const char* f = "gdn_kv_read";
  g_err[0] = 0;
  if (!p) return fail(GDN_ERR_NULL, "%s: args is NULL", f);
  const gdn_kv_read_args& a = *p;
  bool done = false;
  gdn_status st = tokens_check(f, a, done);
  if (st != GDN_OK || done) return st;
  if (!a.k || !a.v || !a.lens || (a.max_pages > 0 && !a.page_table) || (a.n_pages > 0 && (!a.k_cache || !a.v_cache)))
    return fail(GDN_ERR_NULL, "%s: k, v, caches, page_table and lens are required", f);
  st = tokens_layout(f, a);
  if (st != GDN_OK) return st;
  if (!rows_apart(a.total_tokens, a.k_stride_token, a.hkv, a.k_stride_head, a.d) ||
      !rows_apart(a.total_tokens, a.v_stride_token, a.hkv, a.v_stride_head, a.d))
    return fail(GDN_ERR_LAYOUT, "%s: rows of k or v overlap", f);
  return from_hip(gdn::launch_kv_read(a, (hipStream_t)stream), "gdn_kv_read launch");
}

// One input and output of gdn_rope.
static gdn_status rope_layout(const char* f, const char* name, const gdn_rope_args& a, int32_t heads, const void* in,
                              int64_t st, int64_t sh, const void* out, int64_t ot, int64_t oh) {
  const size_t es = elem_size(a.io_dtype);
  if (!aligned(in, es) || !aligned(out, es)) return fail(GDN_ERR_LAYOUT, "%s: %s is not aligned to its elements", f, name);
  const int64_t lim = int64_t(1) << 40;
  if (st < 0 || sh < 0 || ot < 0 || oh < 0 || st >= lim || sh >= lim || ot >= lim || oh >= lim)
    return fail(GDN_ERR_LAYOUT, "%s: strides of %s must be in [0, 2^40)", f, name);
  if (!rows_apart(a.total_tokens, ot, heads, oh, a.d)) return fail(GDN_ERR_LAYOUT, "%s: rows of the output of %s overlap", f, name);
  if (in == out) {
    if ((a.total_tokens > 1 && st != ot) || (heads > 1 && sh != oh))
      return fail(GDN_ERR_LAYOUT, "%s: %s in place needs equal strides", f, name);
    return GDN_OK;
  }
  auto span = [&](int64_t t, int64_t h) { return ((size_t)(a.total_tokens - 1) * t + (size_t)(heads - 1) * h + a.d) * es; };
  const uintptr_t i0 = (uintptr_t)in, o0 = (uintptr_t)out;
  if (i0 >= o0 + span(ot, oh) || o0 >= i0 + span(st, sh)) return GDN_OK;
  // slices of one buffer: tokens the same stride apart, the output's heads in the gaps between the input's
  const int64_t gap = ot * (int64_t)es;
  if (st == ot && gap > 0) {
    const int64_t in_heads = ((heads - 1) * sh + a.d) * (int64_t)es, out_heads = ((heads - 1) * oh + a.d) * (int64_t)es;
    const int64_t behind = ((int64_t)(o0 - i0) % gap + gap) % gap;  // from an input's token to the next output's
    if (behind >= in_heads && behind + out_heads <= gap) return GDN_OK;
  }
  return fail(GDN_ERR_LAYOUT, "%s: the output of %s overlaps it", f, name);
}

gdn_status gdn_rope(const gdn_rope_args* p, void* stream) {
  static const char* f = "gdn_rope";
  g_err[0] = 0;
  if (!p) return fail(GDN_ERR_NULL, "%s: args is NULL", f);
  const gdn_rope_args& a = *p;
  if (a.io_dtype != GDN_F32 && a.io_dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "%s: io_dtype %d", f, a.io_dtype);
  if (a.total_tokens < 0 || a.batch < 0 || a.hq <= 0 || a.hkv < 0 || a.d <= 0 || a.rot <= 0)
    return fail(GDN_ERR_SHAPE, "%s: bad sizes total_tokens=%lld batch=%d hq=%d hkv=%d d=%d rot=%d", f,
                (long long)a.total_tokens, a.batch, a.hq, a.hkv, a.d, a.rot);
  if (a.rot % 2 != 0 || a.rot > a.d) return fail(GDN_ERR_SHAPE, "%s: rot=%d must be even and at most d=%d", f, a.rot, a.d);
  if (a.d > 1024) return fail(GDN_ERR_UNSUPPORTED, "%s: d=%d (supported up to 1024)", f, a.d);
  if ((int64_t)a.hq + a.hkv > 65536) return fail(GDN_ERR_UNSUPPORTED, "%s: hq + hkv must be at most 65536", f);
  if (a.total_tokens > (1 << 24)) return fail(GDN_ERR_UNSUPPORTED, "%s: total_tokens must be at most 2^24", f);
  if (a.total_tokens == 0 || (a.batch == 0 && !a.positions)) return GDN_OK;
  if (!a.positions && !a.cu_seqlens && a.total_tokens % a.batch != 0)
    return fail(GDN_ERR_SHAPE, "%s: without cu_seqlens total_tokens %lld must be a multiple of batch %d", f,
                (long long)a.total_tokens, a.batch);
  if (!a.q || !a.q_out || !a.inv_freq || (!a.positions && !a.lens))
    return fail(GDN_ERR_NULL, "%s: q, q_out, inv_freq and positions or lens are required", f);
  if ((a.hkv > 0) != (a.k != nullptr) || (a.k != nullptr) != (a.k_out != nullptr))
    return fail(GDN_ERR_NULL, "%s: k, k_out and hkv go together", f);
  if (a.k && (a.q_out == a.k || a.k_out == a.q || a.q_out == a.k_out))
    return fail(GDN_ERR_LAYOUT, "%s: one input's output is the other, or its output", f);
  if (!aligned(a.inv_freq, 8) || (a.positions && !aligned(a.positions, a.positions_i64 ? 8 : 4)))
    return fail(GDN_ERR_LAYOUT, "%s: inv_freq and positions must be aligned to their elements", f);
  gdn_status st = rope_layout(f, "q", a, a.hq, a.q, a.q_stride_token, a.q_stride_head, a.q_out, a.qo_stride_token, a.qo_stride_head);
  if (st == GDN_OK && a.k)
    st = rope_layout(f, "k", a, a.hkv, a.k, a.k_stride_token, a.k_stride_head, a.k_out, a.ko_stride_token, a.ko_stride_head);
  if (st != GDN_OK) return st;
  return from_hip(gdn::launch_rope(a, (hipStream_t)stream), "gdn_rope launch");
}

gdn_status gdn_pages_copy(void* pool, int64_t page_bytes, int64_t page_stride, int32_t n_pages, const int32_t* src,
                          const int32_t* dst, int64_t n, void* stream) {
  static const char* f = "gdn_pages_copy";
  g_err[0] = 0;
  if (page_bytes < 0 || n_pages < 0 || n < 0)
    return fail(GDN_ERR_SHAPE, "%s: page_bytes=%lld n_pages=%d n=%lld", f, (long long)page_bytes, n_pages, (long long)n);
  if (page_stride < page_bytes) return fail(GDN_ERR_LAYOUT, "%s: page_stride smaller than page_bytes", f);
  if (n >= (int64_t(1) << 31) || page_bytes >= (int64_t(1) << 40))
    return fail(GDN_ERR_UNSUPPORTED, "%s: n must be below 2^31 and page_bytes below 2^40", f);
  if (n == 0 || page_bytes == 0 || n_pages == 0) return GDN_OK;
  if (!pool || !src || !dst) return fail(GDN_ERR_NULL, "%s: pool, src and dst are required", f);
  return from_hip(gdn::launch_pages_copy(pool, page_bytes, page_stride, n_pages, src, dst, n, (hipStream_t)stream),
                  "gdn_pages_copy launch");
}

size_t gdn_pages_workspace_size(int32_t rows, int32_t n_pages) {
  return rows < 0 || n_pages <= 0 ? 0 : gdn::pages_workspace_bytes(rows, n_pages);
}

// The checks that the page-table calls share; lens: whether the call has row lengths.
static gdn_status pages_check(const char* f, const gdn_pages_args* p, bool lens, bool workspace) {
  g_err[0] = 0;
  if (!p) return fail(GDN_ERR_NULL, "%s: args is NULL", f);
  const gdn_pages_args& a = *p;
  if (a.rows < 0 || a.max_pages <= 0 || a.n_pages <= 0 || a.page_size <= 0)
    return fail(GDN_ERR_SHAPE, "%s: bad sizes rows=%d max_pages=%d n_pages=%d page_size=%d", f, a.rows, a.max_pages,
                a.n_pages, a.page_size);
  if (a.n_pages > (1 << 22)) return fail(GDN_ERR_UNSUPPORTED, "%s: n_pages=%d (supported up to 2^22)", f, a.n_pages);
  if (a.rows > (1 << 20)) return fail(GDN_ERR_UNSUPPORTED, "%s: rows=%d (supported up to 2^20)", f, a.rows);
  if ((int64_t)a.max_pages * a.page_size > (int64_t(1) << 30))
    return fail(GDN_ERR_UNSUPPORTED, "%s: max_pages * page_size must be at most 2^30", f);
  if (a.page_table_stride < a.max_pages || a.page_table_out_stride < a.max_pages)
    return fail(GDN_ERR_LAYOUT, "%s: row strides smaller than max_pages", f);
  if (!a.refs || !a.refs_out || (a.rows > 0 && (!a.page_table || !a.page_table_out)) ||
      (lens && a.rows > 0 && (!a.lens || !a.lens_out)))
    return fail(GDN_ERR_NULL, "%s: page_table, refs%s and their outputs are required", f, lens ? ", lens" : "");
  if (a.page_table == a.page_table_out && a.rows > 1 && a.page_table_stride != a.page_table_out_stride)
    return fail(GDN_ERR_LAYOUT, "%s: page_table in place needs equal strides", f);
  if (workspace) {
    if (!a.workspace) return fail(GDN_ERR_NULL, "%s: workspace is required", f);
    if (!aligned(a.workspace, 256)) return fail(GDN_ERR_LAYOUT, "%s: workspace must be 256-byte aligned", f);
    if (a.workspace_bytes < gdn::pages_workspace_bytes(a.rows, a.n_pages))
      return fail(GDN_ERR_SHAPE, "%s: workspace of %zu bytes (%zu needed)", f, a.workspace_bytes,
                  gdn::pages_workspace_bytes(a.rows, a.n_pages));
  }
  return GDN_OK;
}

gdn_status gdn_pages_extend(const gdn_pages_args* p, const int32_t* add, int32_t* ok, void* stream) {
  const gdn_status st = pages_check("gdn_pages_extend", p, true, true);
  if (st != GDN_OK) return st;
  if (p->rows > 0 && (!add || !ok)) return fail(GDN_ERR_NULL, "gdn_pages_extend: add and ok are required");
  return from_hip(gdn::launch_pages_extend(*p, add, ok, (hipStream_t)stream), "gdn_pages_extend launch");
}

gdn_status gdn_pages_fork(const gdn_pages_args* p, const int32_t* parent, int32_t* src, int32_t* dst, void* stream) {
  const gdn_status st = pages_check("gdn_pages_fork", p, true, true);
  if (st != GDN_OK) return st;
  if (p->rows > 0) {
    if (!parent || !src || !dst) return fail(GDN_ERR_NULL, "gdn_pages_fork: parent, src and dst are required");
    const char* i0 = (const char*)p->page_table;
    const char* o0 = (const char*)p->page_table_out;
    const size_t in = ((size_t)(p->rows - 1) * p->page_table_stride + p->max_pages) * 4;
    const size_t out = ((size_t)(p->rows - 1) * p->page_table_out_stride + p->max_pages) * 4;
    const char* l0 = (const char*)p->lens;
    const char* m0 = (const char*)p->lens_out;
    const size_t ln = (size_t)p->rows * 4;
    if ((i0 < o0 + out && o0 < i0 + in) || (l0 < m0 + ln && m0 < l0 + ln))
      return fail(GDN_ERR_LAYOUT, "gdn_pages_fork: page_table_out and lens_out must be apart from the inputs");
  }
  return from_hip(gdn::launch_pages_fork(*p, parent, src, dst, (hipStream_t)stream), "gdn_pages_fork launch");
}

gdn_status gdn_pages_free(const gdn_pages_args* p, const uint8_t* mask, void* stream) {
  const gdn_status st = pages_check("gdn_pages_free", p, true, false);
  if (st != GDN_OK) return st;
  if (p->rows > 0 && !mask) return fail(GDN_ERR_NULL, "gdn_pages_free: mask is required");
  return from_hip(gdn::launch_pages_free(*p, mask, (hipStream_t)stream), "gdn_pages_free launch");
}

gdn_status gdn_pages_compact(const gdn_pages_args* p, int32_t* src, int32_t* dst, int32_t* n_live, void* stream) {
  const gdn_status st = pages_check("gdn_pages_compact", p, false, true);
  if (st != GDN_OK) return st;
  if (!n_live || (p->n_pages > 1 && (!src || !dst)))
    return fail(GDN_ERR_NULL, "gdn_pages_compact: src, dst and n_live are required");
  return from_hip(gdn::launch_pages_compact(*p, src, dst, n_live, (hipStream_t)stream), "gdn_pages_compact launch");
}

}  // extern "C"
