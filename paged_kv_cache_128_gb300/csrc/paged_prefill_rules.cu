// Chunked-prefill attention under score rules (score_rules.cuh): capped
// scores, a bias that falls with the distance, windows, documents and spans
// seen both ways, each query row over its own interval of keys.

#include "prefill_common.cuh"

using namespace pagedkv;

extern "C" int paged_prefill_attention_rules(
    void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
    const int32_t* seq_lens, const int32_t* query_start_loc, int64_t num_query_tokens, int32_t num_seqs,
    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int64_t num_blocks,
    int32_t max_blocks_per_seq, int32_t max_query_len, float scale, float softcap, const float* slopes, int32_t window,
    const int32_t* key_begin, const int32_t* key_end, int dtype, void* stream) {
  RulesPrefillParams p{};
  int s = make_rules(scale, softcap, slopes, window, key_begin, key_end, &p.rules);
  if (s != KV_OK) return s;
  s = prefill_params(out, q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, num_query_tokens, num_seqs,
                     num_heads, num_kv_heads, head_dim, block_size, num_blocks, max_blocks_per_seq, max_query_len,
                     scale, dtype, &p);
  if (s != KV_OK || p.num_seqs == 0) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == KV_DTYPE_F16 ? launch_prefill<__half>(p, head_dim, max_query_len, st)
                                              : launch_prefill<__nv_bfloat16>(p, head_dim, max_query_len, st);
  return cuda_status(e);
}

// Read (and optionally clear) this translation unit's device error word.
extern "C" int pagedkv_internal_prefill_rules_error(int reset, int* code) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  if (reset) {
    int zero = 0;
    if (cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  }
  *code = v;
  return KV_OK;
}
