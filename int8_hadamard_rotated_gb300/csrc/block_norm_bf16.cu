// block_norm_bf16.cu -- the block norms of bf16 residual streams (block_norm.cuh).
#include "block_norm.cuh"

namespace convrot {
namespace fp8 {

template int launch_block_norm_as<__nv_bfloat16>(const convrot_block_norm_args& a, cudaStream_t stream,
                                                 NormTimeoutTest test);
template cudaError_t norm_error_word<__nv_bfloat16>(int** p);

}  // namespace fp8
}  // namespace convrot
