// Entry points of decode attention and of the decode steps; the kernels are
// in decode_kernels.cuh.

#include <atomic>
#include <chrono>
#include <random>

#include "decode_kernels.cuh"

namespace pagedkv {

// Tag of one stream-K call: a per-process random base plus a call counter,
// so a ready flag left by any other call (or uninitialised workspace) does
// not match.
uint64_t next_epoch() {
  static std::atomic<uint64_t> counter{0};
  static const uint64_t base = [] {
    std::random_device rd;
    uint64_t x = (static_cast<uint64_t>(rd()) << 32) ^ rd();
    x ^= static_cast<uint64_t>(std::chrono::steady_clock::now().time_since_epoch().count()) * 0x9E3779B97F4A7C15ull;
    return x;
  }();
  return base + 2 * (counter.fetch_add(1) + 1);
}

namespace {

// Stream-K test controls (kv_debug_set), read at each launch; the
// shared-prefix and prefill kernels read skip_tile too.
struct SkControls {
  std::atomic<int64_t> wait_limit_ns{static_cast<int64_t>(kWaitLimitNs)};
  std::atomic<int64_t> skip_tile{-1};
};
SkControls& sk_controls() {
  static SkControls c;
  return c;
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" int pagedkv_internal_reshape_error(int reset, int* code);
extern "C" int pagedkv_internal_prefill_error(int reset, int* code);
extern "C" int pagedkv_internal_rope_error(int reset, int* code);
extern "C" int pagedkv_internal_shared_error(int reset, int* code);
extern "C" int pagedkv_internal_decode_rules_error(int reset, int* code);
extern "C" int pagedkv_internal_decode_rules_cap_error(int reset, int* code);
extern "C" int pagedkv_internal_prefill_rules_error(int reset, int* code);
extern "C" int paged_reshape_and_cache(const void* k, const void* v, void* k_cache, void* v_cache,
                                       const int32_t* slot_mapping, int64_t num_tokens, int32_t num_kv_heads,
                                       int32_t head_dim, int32_t block_size, int64_t num_blocks,
                                       int64_t k_token_stride, int64_t v_token_stride, int dtype, void* stream);

extern "C" int paged_decode_plan(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t block_size, int64_t max_seq_len, int32_t blocks_per_split, int dtype,
                                 int32_t* kernel_out, int32_t* blocks_per_split_out, int32_t* num_splits_out,
                                 size_t* workspace_bytes_out) {
  int st = check_shapes(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_seq_len, dtype);
  if (st != KV_OK) return st;
  if (blocks_per_split < 0) return KV_ERR_INVALID_ARG;
  Plan pl = make_plan(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_seq_len, blocks_per_split, dtype);
  if (kernel_out) *kernel_out = pl.kind;
  if (blocks_per_split_out) *blocks_per_split_out = pl.bps;
  if (num_splits_out) *num_splits_out = pl.num_splits;
  if (workspace_bytes_out) *workspace_bytes_out = pl.ws_bytes;
  return KV_OK;
}

extern "C" int paged_decode_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                           int32_t head_dim, int32_t block_size, int64_t max_seq_len,
                                           int32_t blocks_per_split, int dtype, size_t* bytes_out) {
  if (!bytes_out) return KV_ERR_INVALID_ARG;
  return paged_decode_plan(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_seq_len, blocks_per_split,
                           dtype, nullptr, nullptr, nullptr, bytes_out);
}

extern "C" int paged_decode_attention(void* out, const void* q, const void* k_cache, const void* v_cache,
                                      const int32_t* block_tables, const int32_t* seq_lens, int32_t num_seqs,
                                      int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                      int32_t block_size, int64_t num_blocks, int32_t max_blocks_per_seq,
                                      int64_t max_seq_len, float scale, int32_t blocks_per_split, int dtype,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  return decode_impl(out, q, k_cache, v_cache, block_tables, seq_lens, num_seqs, num_heads, num_kv_heads, head_dim,
                     block_size, num_blocks, max_blocks_per_seq, max_seq_len, scale, blocks_per_split, dtype,
                     workspace, workspace_bytes, stream, nullptr);
}

extern "C" int paged_decode_step(void* out, const void* q, const void* k, const void* v,
                                 const int32_t* slot_mapping, int64_t num_tokens, int64_t k_token_stride,
                                 int64_t v_token_stride, const int32_t* new_token_row, void* k_cache,
                                 void* v_cache, const int32_t* block_tables, const int32_t* seq_lens,
                                 int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t block_size, int64_t num_blocks, int32_t max_blocks_per_seq,
                                 int64_t max_seq_len, float scale, int dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (num_tokens < 0) return KV_ERR_INVALID_ARG;
  if (num_tokens > 0) {
    const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (!k || !v || !slot_mapping || k_token_stride < row || v_token_stride < row) return KV_ERR_INVALID_ARG;
    if (num_seqs > 0 && !new_token_row) return KV_ERR_INVALID_ARG;
  }
  const StepArgs step{k, v, slot_mapping, new_token_row, num_tokens, k_token_stride, v_token_stride};
  if (num_seqs == 0) {  // nothing to attend: the cache write alone
    return paged_reshape_and_cache(k, v, k_cache, v_cache, slot_mapping, num_tokens, num_kv_heads, head_dim,
                                   block_size, num_blocks, k_token_stride, v_token_stride, dtype, stream);
  }
  return decode_impl(out, q, k_cache, v_cache, block_tables, seq_lens, num_seqs, num_heads, num_kv_heads, head_dim,
                     block_size, num_blocks, max_blocks_per_seq, max_seq_len, scale, 0, dtype, workspace,
                     workspace_bytes, stream, &step);
}

// ---------------------------------------------------------------------------
// Decode attention over fp8 (E4M3) caches with per-token scales.

extern "C" int paged_decode_attention_fp8(void* out, const void* q, const void* k_cache, const void* v_cache,
                                          const float* k_scales, const float* v_scales, const int32_t* block_tables,
                                          const int32_t* seq_lens, int32_t num_seqs, int32_t num_heads,
                                          int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                          int64_t num_blocks, int32_t max_blocks_per_seq, int64_t max_seq_len,
                                          float scale, int dtype, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  return decode_fp8_impl(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens, num_seqs, num_heads,
                         num_kv_heads, head_dim, block_size, num_blocks, max_blocks_per_seq, max_seq_len, scale, dtype,
                         workspace, workspace_bytes, stream, nullptr);
}

extern "C" int paged_decode_step_fp8(void* out, const void* q, const void* k, const void* v,
                                     const int32_t* slot_mapping, int64_t num_tokens, int64_t k_token_stride,
                                     int64_t v_token_stride, const int32_t* new_token_row, void* k_cache,
                                     void* v_cache, float* k_scales, float* v_scales, const int32_t* block_tables,
                                     const int32_t* seq_lens, int32_t num_seqs, int32_t num_heads,
                                     int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int64_t num_blocks,
                                     int32_t max_blocks_per_seq, int64_t max_seq_len, float scale, int dtype,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  if (num_tokens < 0) return KV_ERR_INVALID_ARG;
  if (num_tokens > 0) {
    const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (!k || !v || !slot_mapping || k_token_stride < row || v_token_stride < row) return KV_ERR_INVALID_ARG;
    if (num_seqs > 0 && !new_token_row) return KV_ERR_INVALID_ARG;
  }
  if (num_seqs == 0)  // nothing to attend: the cache write alone
    return paged_reshape_and_cache_fp8(k, v, k_cache, v_cache, k_scales, v_scales, slot_mapping, num_tokens,
                                       num_kv_heads, head_dim, block_size, num_blocks, k_token_stride, v_token_stride,
                                       dtype, stream);
  const StepArgs step{k, v, slot_mapping, new_token_row, num_tokens, k_token_stride, v_token_stride};
  return decode_fp8_impl(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens, num_seqs, num_heads,
                         num_kv_heads, head_dim, block_size, num_blocks, max_blocks_per_seq, max_seq_len, scale, dtype,
                         workspace, workspace_bytes, stream, &step);
}

// ---------------------------------------------------------------------------
// Decode attention for callers that cannot allocate device memory.
//
// Some callers may not call cudaMalloc at all: a host process whose GPU memory
// is owned by another allocator (a framework caching allocator or a serving
// runtime that reserves nearly all HBM up front), a plugin interface that
// forbids allocation while it executes, or a latency-critical loop where an
// allocation could synchronise the device.  paged_decode_attention needs a
// caller-provided workspace; this variant instead uses one fixed scratch array
// in device memory that the library defines at file scope, so the call itself
// allocates nothing.
//
// The array is a static __device__ object of kStaticScratchBytes: every GPU
// that loads this library holds it until the process exits.  In host code its
// name is only a host-side stand-in, so the device address is looked up once
// per device (cudaGetSymbolAddress, with that device current) on the first
// call made on it.  All calls on a device share the array and it keeps the
// last call's contents; the kernels write every scratch value they read in the
// same call (the stream-K ready flags carry a per-call tag), so nothing needs
// clearing between calls, but calls that overlap on the GPU race on it.
constexpr size_t kStaticScratchBytes = size_t(8) << 20;  // 8 MiB
static __device__ __align__(256) unsigned char g_decode_scratch[kStaticScratchBytes];

namespace {
void* static_scratch_address(int dev, cudaError_t* err) {
  static std::mutex mu;
  static void* addr[64] = {nullptr};
  std::lock_guard<std::mutex> lock(mu);
  if (!addr[dev]) {
    void* ptr = nullptr;
    *err = cudaGetSymbolAddress(&ptr, g_decode_scratch);
    if (*err != cudaSuccess) return nullptr;
    addr[dev] = ptr;
  }
  *err = cudaSuccess;
  return addr[dev];
}
}  // namespace

extern "C" int paged_decode_attention_static_scratch(
    void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
    const int32_t* seq_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t block_size, int64_t num_blocks, int32_t max_blocks_per_seq, int64_t max_seq_len, float scale,
    int32_t blocks_per_split, int dtype, void* stream) {
  size_t need = 0;
  int st = paged_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_seq_len,
                                       blocks_per_split, dtype, &need);
  if (st != KV_OK) return st;
  if (need > kStaticScratchBytes) return KV_ERR_WORKSPACE;  // beyond the fixed scratch: use the workspace call
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e);
  if (dev < 0 || dev >= 64) return KV_ERR_INVALID_ARG;
  void* scratch = static_scratch_address(dev, &e);
  if (!scratch) return cuda_status(e, "cudaGetSymbolAddress of the decode scratch failed");
  return paged_decode_attention(out, q, k_cache, v_cache, block_tables, seq_lens, num_seqs, num_heads, num_kv_heads,
                                head_dim, block_size, num_blocks, max_blocks_per_seq, max_seq_len, scale,
                                blocks_per_split, dtype, scratch, kStaticScratchBytes, stream);
}

extern "C" size_t paged_decode_static_scratch_bytes(void) { return kStaticScratchBytes; }

extern "C" int kv_device_error(int reset, int* status_out) {
  if (!status_out) return KV_ERR_INVALID_ARG;
  if (cudaDeviceSynchronize() != cudaSuccess) return KV_ERR_CUDA;
  int a = 0;
  if (cudaMemcpyFromSymbol(&a, g_device_error, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  if (reset) {
    int zero = 0;
    if (cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  }
  // the other translation units' words; the first that holds an error, in this order
  int (*const others[])(int, int*) = {pagedkv_internal_reshape_error, pagedkv_internal_prefill_error,
                                      pagedkv_internal_rope_error, pagedkv_internal_shared_error,
                                      pagedkv_internal_decode_rules_error, pagedkv_internal_decode_rules_cap_error,
                                      pagedkv_internal_prefill_rules_error};
  for (auto read : others) {
    int c = 0;
    const int r = read(reset, &c);
    if (r != KV_OK) return r;
    if (!a) a = c;
  }
  *status_out = a;
  return KV_OK;
}

extern "C" int kv_debug_set(int key, int64_t value) {
  SkControls& c = sk_controls();
  switch (key) {
    case KV_DEBUG_WAIT_LIMIT_NS:
      c.wait_limit_ns = value > 0 ? value : static_cast<int64_t>(kWaitLimitNs);
      return KV_OK;
    case KV_DEBUG_SKIP_TILE:
      c.skip_tile = value >= 0 ? value : -1;
      return KV_OK;
    default:
      return KV_ERR_INVALID_ARG;
  }
}

extern "C" const char* kv_version(void) { return "pagedkv-gb300 0.1 (sm_103a)"; }

namespace pagedkv {
int64_t debug_wait_limit_ns() { return sk_controls().wait_limit_ns.load(); }

int32_t debug_skip_tile() { return static_cast<int32_t>(sk_controls().skip_tile.load()); }

const char*& last_cuda_error_text() {
  static thread_local const char* text = "no error";
  return text;
}
}  // namespace pagedkv

extern "C" const char* kv_last_cuda_error(void) { return last_cuda_error_text(); }
