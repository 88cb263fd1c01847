// Decode attention under score rules (score_rules.cuh): the decode kernels of
// decode_kernels.cuh compiled with them.  What they add there: a sequence's
// tiles start with the one that holds the first key its query sees, so a window
// of W tokens costs what W tokens cost whatever the length, and blocks that end
// before that key are not looked up; scores pass through the cap and the
// distance bias before the online softmax.  What bounds it: memory, as the plain
// calls; fp8 caches their consumers' instructions.  Measured: 64 sequences to
// 16384 tokens, window 4096, cap 30, 32/8 heads of 128: 176 us, 1075 MB (0.92 of
// the copy rate); 32 to 8192, cap 50, 16/8 heads of 256: 209 us, 1308 MB (0.94);
// fp8, 121 sequences, stretches of 8192, 28/4 heads: 123 us, 536 MB (0.65; a
// copy of the kernel that only loads takes 103).  Here without a cap; with one in
// paged_decode_rules_cap.cu.

#include "decode_kernels.cuh"

using namespace pagedkv;

extern "C" int paged_decode_attention_rules(void* out, const void* q, const void* k_cache, const void* v_cache,
                                            const int32_t* block_tables, const int32_t* seq_lens, int32_t num_seqs,
                                            int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                            int32_t block_size, int64_t num_blocks, int32_t max_blocks_per_seq,
                                            int64_t max_seq_len, float scale, float softcap, const float* slopes,
                                            int32_t window, const int32_t* key_begin, int dtype, void* workspace,
                                            size_t workspace_bytes, void* stream) {
  ScoreRules rules;
  const int st = make_rules(scale, softcap, slopes, window, key_begin, nullptr, &rules);
  if (st != KV_OK) return st;
  return (rules.cap_log2 > 0.f ? decode_rules_cap() : &decode_impl<RulesParams<false>>)(
      out, q, k_cache, v_cache, block_tables, seq_lens, num_seqs, num_heads, num_kv_heads, head_dim, block_size,
      num_blocks, max_blocks_per_seq, max_seq_len, scale, 0, dtype, workspace, workspace_bytes, stream, nullptr, &rules);
}

extern "C" int paged_decode_attention_rules_fp8(
    void* out, const void* q, const void* k_cache, const void* v_cache, const float* k_scales, const float* v_scales,
    const int32_t* block_tables, const int32_t* seq_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int64_t num_blocks, int32_t max_blocks_per_seq, int64_t max_seq_len,
    float scale, float softcap, const float* slopes, int32_t window, const int32_t* key_begin, int dtype,
    void* workspace, size_t workspace_bytes, void* stream) {
  ScoreRules rules;
  const int st = make_rules(scale, softcap, slopes, window, key_begin, nullptr, &rules);
  if (st != KV_OK) return st;
  return (rules.cap_log2 > 0.f ? decode_rules_cap_fp8() : &decode_fp8_impl<RulesParams<false>>)(
      out, q, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens, num_seqs, num_heads, num_kv_heads, head_dim,
      block_size, num_blocks, max_blocks_per_seq, max_seq_len, scale, dtype, workspace, workspace_bytes, stream, nullptr,
      &rules);
}

// Read (and optionally clear) this translation unit's device error word.
extern "C" int pagedkv_internal_decode_rules_error(int reset, int* code) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  if (reset) {
    int zero = 0;
    if (cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  }
  *code = v;
  return KV_OK;
}
