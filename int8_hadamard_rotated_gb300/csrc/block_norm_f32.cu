// block_norm_f32.cu -- the block norms of fp32 residual streams (block_norm.cuh).
#include "block_norm.cuh"

namespace convrot {
namespace fp8 {

template int launch_block_norm_as<float>(const convrot_block_norm_args& a, cudaStream_t stream,
                                         NormTimeoutTest test);
template cudaError_t norm_error_word<float>(int** p);

}  // namespace fp8
}  // namespace convrot
