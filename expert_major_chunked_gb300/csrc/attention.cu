// C entries of the attention operators (include/moe_attention.h): argument checks, then the launches of
// attn_prefill.cu, attn_decode.cu and kv_cache.cu. Nothing here throws past the C boundary.
#include "attn.h"
#include "internal.h"

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>

using namespace moe;

moe::EncodeTiledFn moe::tensor_map_encoder() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

namespace {

moe_status fail(moe_status st, const char* fmt, ...) noexcept {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  try {
    set_last_error(buf);
  } catch (...) {  // no memory for the message: the status stands without it
  }
  return st;
}

#define REQUIRE(cond, ...) \
  do {                     \
    if (!(cond)) return fail(MOE_ERR_INVALID_ARG, __VA_ARGS__); \
  } while (0)

constexpr int32_t kPrefillMax = 1 << 30;  // row numbers and tile numbers stay within int32 in the kernel

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

moe_status cuda_failed(cudaError_t e, const char* what) noexcept {
  cudaGetLastError();  // reported here, so not left for another call of the thread to find
  return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

moe_status launched(cudaError_t e, const char* what) noexcept { return e == cudaSuccess ? MOE_OK : cuda_failed(e, what); }

moe_status check_device() noexcept {
  // the answer for a device does not change, so it is looked up once for each
  static int major[kMaxDevices], minor[kMaxDevices];
  static bool known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_failed(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices)
    return fail(MOE_ERR_UNSUPPORTED, "device %d: only 0..%d are supported", dev, kMaxDevices - 1);
  if (!__atomic_load_n(&known[dev], __ATOMIC_ACQUIRE)) {
    int ma = 0, mi = 0;
    e = cudaDeviceGetAttribute(&ma, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&mi, cudaDevAttrComputeCapabilityMinor, dev);
    if (e != cudaSuccess) return cuda_failed(e, "cudaDeviceGetAttribute");
    __atomic_store_n(&major[dev], ma, __ATOMIC_RELAXED);
    __atomic_store_n(&minor[dev], mi, __ATOMIC_RELAXED);
    __atomic_store_n(&known[dev], true, __ATOMIC_RELEASE);
  }
  if (major[dev] != 10 || minor[dev] != 3)
    return fail(MOE_ERR_ARCH, "device %d is sm_%d%d; the kernels are built for sm_103a", dev, major[dev], minor[dev]);
  return MOE_OK;
}

moe_status check_heads(int n_heads, int n_kv_heads, int head_dim, int dtype) noexcept {
  REQUIRE(n_heads > 0 && n_kv_heads > 0 && n_heads % n_kv_heads == 0,
          "n_heads (%d) must be a positive multiple of n_kv_heads (%d)", n_heads, n_kv_heads);
  if (n_heads > 65535) return fail(MOE_ERR_UNSUPPORTED, "n_heads %d: at most 65535", n_heads);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(MOE_ERR_UNSUPPORTED, "head_dim %d: 64, 128 and 256 are supported", head_dim);
  if (dtype != MOE_ATTN_BF16 && dtype != MOE_ATTN_F16)
    return fail(MOE_ERR_UNSUPPORTED, "dtype %d: MOE_ATTN_BF16 and MOE_ATTN_F16 are supported", dtype);
  return MOE_OK;
}

moe_status check_rows(const char* name, const void* p, int64_t token, int64_t head) noexcept {
  REQUIRE(p, "%s is NULL", name);
  REQUIRE(aligned(p, 16) && token >= 0 && head >= 0 && token % 8 == 0 && head % 8 == 0,
          "%s: rows must start on 16-byte boundaries (pointer aligned, strides multiples of 8 elements)", name);
  return MOE_OK;
}

// A tensor map walks rows by their stride, which must then be positive and below 2^40 bytes.
moe_status check_walk(const char* name, int64_t stride, int64_t count) noexcept {
  REQUIRE(count <= 1 || (stride > 0 && stride < (int64_t{1} << 39)), "%s: rows must be apart, by less than 2^39 elements",
          name);
  return MOE_OK;
}

// Rows that are written lie apart.
moe_status check_out(const void* p, int64_t token, int64_t tokens, int64_t head, int64_t heads, int dim) noexcept {
  const moe_status st = check_rows("out", p, token, head);
  if (st != MOE_OK) return st;
  REQUIRE((tokens <= 1 || token >= dim) && (heads <= 1 || head >= dim), "out: rows must be at least head_dim apart");
  return MOE_OK;
}

moe_status check_block(int block_size, int num_blocks) noexcept {
  if (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128)
    return fail(MOE_ERR_UNSUPPORTED, "block_size %d: 16, 32, 64 and 128 are supported", block_size);
  REQUIRE(num_blocks >= 0, "num_blocks %d is negative", num_blocks);
  return MOE_OK;
}

#define TRY(expr)                          \
  do {                                     \
    const moe_status st_ = (expr);         \
    if (st_ != MOE_OK) return st_;         \
  } while (0)

}  // namespace

extern "C" {

moe_status moe_attn_prefill(const moe_attn_prefill_args* p, void* stream) {
  REQUIRE(p, "args is NULL");
  const moe_attn_prefill_args& a = *p;
  TRY(check_heads(a.n_heads, a.n_kv_heads, a.head_dim, a.dtype));
  REQUIRE(a.n_seqs >= 0 && a.total_q >= 0 && a.total_k >= 0, "n_seqs, total_q and total_k must not be negative");
  REQUIRE(std::isfinite(a.scale) && a.scale > 0.0f, "scale must be positive and finite");
  if (a.n_seqs > kPrefillMax || a.total_q > kPrefillMax || a.total_k > kPrefillMax ||
      (int64_t{a.total_q} + a.n_seqs) * a.n_heads > INT32_MAX)
    return fail(MOE_ERR_UNSUPPORTED, "n_seqs, total_q and total_k: at most 2^30, (total_q + n_seqs) * n_heads below 2^31");
  if (a.total_q == 0 || a.n_seqs == 0) return MOE_OK;
  REQUIRE(a.cu_q && a.cu_k && aligned(a.cu_q, 4) && aligned(a.cu_k, 4), "cu_q and cu_k must be int32 arrays");
  TRY(check_rows("q", a.q, a.q_token, a.q_head));
  TRY(check_walk("q", a.q_token, a.total_q));
  TRY(check_walk("q", a.q_head, a.n_heads));
  TRY(check_out(a.out, a.out_token, a.total_q, a.out_head, a.n_heads, a.head_dim));
  if (a.total_k > 0) {
    TRY(check_rows("k", a.k, a.k_token, a.k_head));
    TRY(check_walk("k", a.k_token, a.total_k));
    TRY(check_walk("k", a.k_head, a.k_head ? a.n_kv_heads : 1));
    TRY(check_rows("v", a.v, a.v_token, a.v_head));
    TRY(check_walk("v", a.v_token, a.total_k));
    TRY(check_walk("v", a.v_head, a.v_head ? a.n_kv_heads : 1));
  }
  REQUIRE(aligned(a.lse, 4), "lse must be 4-byte aligned");
  TRY(check_device());
  return launched(launch_attn_prefill(a, static_cast<cudaStream_t>(stream)), "moe_attn_prefill");
}

moe_status moe_attn_check(void* stream) {
  TRY(check_device());
  int site = 0;
  TRY(launched(attn_prefill_take_error(&site, static_cast<cudaStream_t>(stream)), "moe_attn_check"));
  if (site) return fail(MOE_ERR_DEVICE_TIMEOUT, "moe_attn_prefill: a wait on the device gave up (site %d)", site);
  return MOE_OK;
}

moe_status moe_kv_assign(const moe_kv_assign_args* p, void* stream) {
  REQUIRE(p, "args is NULL");
  const moe_kv_assign_args& a = *p;
  REQUIRE(a.n_requests >= 0 && a.n_free >= 0 && a.max_blocks >= 0 && a.max_tokens >= 0,
          "n_requests, n_free, max_blocks and max_tokens must not be negative");
  if (a.n_requests > kAssignMaxRequests)
    return fail(MOE_ERR_UNSUPPORTED, "n_requests %d: at most %d", a.n_requests, kAssignMaxRequests);
  REQUIRE(a.block_size > 0, "block_size must be positive");
  REQUIRE(a.cu_new && a.used, "cu_new and used must not be NULL");
  REQUIRE(a.n_requests == 0 || (a.ctx_lens && a.new_lens && a.kv_lens), "ctx_lens, new_lens and kv_lens must not be NULL");
  REQUIRE(a.n_requests == 0 || a.max_blocks == 0 || (a.block_table && a.table_stride >= a.max_blocks),
          "block_table must have rows of at least max_blocks entries");
  REQUIRE(a.n_free == 0 || a.free_blocks, "free_blocks is NULL");
  REQUIRE(a.max_tokens == 0 || (a.slot_map && a.positions), "slot_map and positions must not be NULL");
  REQUIRE(aligned(a.slot_map, 8) && aligned(a.positions, 4) && aligned(a.block_table, 4),
          "slot_map, positions and block_table must be aligned to their elements");
  TRY(check_device());
  return launched(launch_kv_assign(a, static_cast<cudaStream_t>(stream)), "moe_kv_assign");
}

moe_status moe_kv_append(const moe_kv_append_args* p, void* stream) {
  REQUIRE(p, "args is NULL");
  const moe_kv_append_args& a = *p;
  TRY(check_heads(a.n_kv_heads, a.n_kv_heads, a.head_dim, a.dtype));
  TRY(check_block(a.block_size, a.num_blocks));
  REQUIRE(a.n_tokens >= 0, "n_tokens %d is negative", a.n_tokens);
  if (a.n_tokens == 0) return MOE_OK;
  TRY(check_rows("k", a.k, a.k_token, a.k_head));
  TRY(check_rows("v", a.v, a.v_token, a.v_head));
  REQUIRE(a.slot_map && aligned(a.slot_map, 8), "slot_map must be an int64 array");
  REQUIRE(a.num_blocks == 0 || (a.k_codes && a.v_codes && a.k_scale && a.v_scale), "a part of the cache is NULL");
  REQUIRE(aligned(a.k_codes, 16) && aligned(a.v_codes, 16) && aligned(a.k_scale, 4) && aligned(a.v_scale, 4),
          "the codes must be 16-byte aligned, the scales 4-byte aligned");
  TRY(check_device());
  return launched(launch_kv_append(a, static_cast<cudaStream_t>(stream)), "moe_kv_append");
}

size_t moe_attn_decode_workspace(int32_t n_requests, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (n_requests < 0 || check_heads(n_heads, n_kv_heads, head_dim, MOE_ATTN_BF16) != MOE_OK) return 0;
  return attn_decode_workspace(n_requests, n_heads, n_kv_heads, head_dim);
}

moe_status moe_attn_decode(const moe_attn_decode_args* p, void* stream) {
  REQUIRE(p, "args is NULL");
  const moe_attn_decode_args& a = *p;
  TRY(check_heads(a.n_heads, a.n_kv_heads, a.head_dim, a.dtype));
  TRY(check_block(a.block_size, a.num_blocks));
  REQUIRE(a.n_requests >= 0 && a.max_blocks >= 0, "n_requests and max_blocks must not be negative");
  if (a.n_requests > 65535) return fail(MOE_ERR_UNSUPPORTED, "n_requests %d: at most 65535", a.n_requests);
  REQUIRE(std::isfinite(a.scale) && a.scale > 0.0f, "scale must be positive and finite");
  if (a.n_requests == 0) return MOE_OK;
  TRY(check_rows("q", a.q, a.q_token, a.q_head));
  TRY(check_out(a.out, a.out_token, a.n_requests, a.out_head, a.n_heads, a.head_dim));
  REQUIRE(a.kv_lens && aligned(a.kv_lens, 4), "kv_lens must be an int32 array");
  REQUIRE(a.max_blocks == 0 || (a.block_table && aligned(a.block_table, 4) && a.table_stride >= a.max_blocks),
          "block_table must have int32 rows of at least max_blocks entries");
  REQUIRE(a.num_blocks == 0 || (a.k_codes && a.v_codes && a.k_scale && a.v_scale), "a part of the cache is NULL");
  REQUIRE(aligned(a.k_codes, 16) && aligned(a.v_codes, 16) && aligned(a.k_scale, 4) && aligned(a.v_scale, 4),
          "the codes must be 16-byte aligned, the scales 4-byte aligned");
  REQUIRE(aligned(a.lse, 4), "lse must be 4-byte aligned");
  REQUIRE(a.workspace && aligned(a.workspace, 16), "workspace must be 16-byte aligned");
  const size_t need = attn_decode_workspace(a.n_requests, a.n_heads, a.n_kv_heads, a.head_dim);
  if (a.workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes: %zu are needed", a.workspace_bytes, need);
  TRY(check_device());
  return launched(launch_attn_decode(a, static_cast<cudaStream_t>(stream)), "moe_attn_decode");
}

}  // extern "C"
