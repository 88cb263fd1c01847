// Decode attention under score rules with a cap: the kernels of
// decode_kernels.cuh that paged_decode_rules.cu calls for one.

#include "decode_kernels.cuh"

namespace pagedkv {
DecodeCall decode_rules_cap() { return &decode_impl<RulesParams<true>>; }
DecodeFp8Call decode_rules_cap_fp8() { return &decode_fp8_impl<RulesParams<true>>; }
}  // namespace pagedkv

using namespace pagedkv;

// Read (and optionally clear) this translation unit's device error word.
extern "C" int pagedkv_internal_decode_rules_cap_error(int reset, int* code) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  if (reset) {
    int zero = 0;
    if (cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  }
  *code = v;
  return KV_OK;
}
