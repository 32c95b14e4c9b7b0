// Dense grouped-head attention over the paged 4-bit K/V cache: paged_attention.cu's kernel compiled for it, and its launch.
#define DSA_PAGED_KERNEL_ONLY
#include "paged_attention.cu"

namespace dsa {

cudaError_t launch_kv4_attention(PagedAttnArgs a, const uint8_t* k_codes, const uint8_t* v_codes, int max_seq_len, void* workspace,
                                 const PagedAttnPlan& plan, cudaStream_t s) {
  const int ctas = device_sm_count();
  pa_layout(a, workspace, plan, ctas, max_seq_len);
  const uint64_t rows = (uint64_t)a.num_pages * a.kv_heads << a.log2_page;
  CUtensorMap k_map, v_map;
  if (!encode_2d(&k_map, k_codes, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 1, kKvDim, rows, kKvDim / 2, kKvDim, 1u << a.log2_page) ||
      !encode_2d(&v_map, v_codes, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 1, kKvDim, rows, kKvDim / 2, kKvDim, 1u << a.log2_page))
    return cudaErrorInvalidValue;
  a.k_codes4 = k_codes;
  cudaError_t e = launch_few_rows<true>(a, k_map, v_map, ctas, !plan.prompt, s);
  if (e == cudaSuccess && plan.prompt)
    e = launch_kv4_prompt(pa_prompt_args(a, workspace, plan, ctas), a, kPagedAttnColumns / 8, k_map, v_codes, ctas, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dsa
