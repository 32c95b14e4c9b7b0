// Dense attention over the paged 4-bit K/V cache for requests of many rows: paged_prompt.cu's kernel compiled for it.
#define DSA_PAGED_KERNEL_ONLY
#include "paged_prompt.cu"

namespace dsa {

cudaError_t launch_kv4_prompt(const PagedAttnArgs& a, const PagedAttnArgs& few, int few_y, const CUtensorMap& k_map, const uint8_t* v_codes,
                              int ctas, cudaStream_t s) {
  const cudaError_t e = launch_prompt<true>(a, k_map, v_codes, ctas, s);
  return e != cudaSuccess ? e : launch_prompt_join(a, few, few_y, ctas, s);
}

}  // namespace dsa
