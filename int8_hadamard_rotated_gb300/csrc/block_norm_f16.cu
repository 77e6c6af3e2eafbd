// block_norm_f16.cu -- the block norms of fp16 residual streams (block_norm.cuh).
#include "block_norm.cuh"

namespace convrot {
namespace fp8 {

template int launch_block_norm_as<__half>(const convrot_block_norm_args& a, cudaStream_t stream,
                                          NormTimeoutTest test);
template cudaError_t norm_error_word<__half>(int** p);

}  // namespace fp8
}  // namespace convrot
