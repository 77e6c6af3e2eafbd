// moe_common.cuh -- what the experts' operators share: the launchers behind
// their entry points (moe_api.cu) and the limits that the kernels count on.
#pragma once

#include "fp8_common.cuh"

namespace convrot {
namespace moe {

constexpr int MAX_EXPERTS = CONVROT_MOE_MAX_EXPERTS;
constexpr int MAX_TOP_K = CONVROT_MOE_MAX_TOP_K;

// 1 / (1 + exp(-l)) from the hardware's base-2 exponential and reciprocal
// (ex2.approx, rcp.approx, within 2^-22 and one ulp): the exponential of -|l|, so
// that nothing overflows and the reciprocal of 1 to 2 is not flushed to zero,
// and not its .ftz form, so that neither is the result.
__device__ __forceinline__ float sigmoid_fast(float l) {
  float e;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * fabsf(l)));
  return rcp_approx(1.0f + e) * (l >= 0.0f ? 1.0f : e);
}

// Rows sorted by expert, as moe_plan leaves them.
struct Rows {
  const int32_t* order;    // [n] the choice (token * top_k + slot) of a row, or null: row i of the activation
  const int32_t* offsets;  // [E + 1] an expert's first row
  int64_t n, T;            // rows; rows of the activation
  int E, top_k;
};

// moe_route.cu: arguments already checked; T > 0 (n > 0).
int launch_route(const convrot_moe_route_args& a, cudaStream_t stream);
size_t plan_workspace(int64_t n, int E);
int launch_plan(const int32_t* experts, int64_t n, int E, int32_t* order, int32_t* place, int32_t* offsets, void* workspace,
                cudaStream_t stream);
struct CombineArgs {
  const void* rows;  // [n,N] of r_dtype
  int r_dtype;
  int64_t ldr, n;
  const int32_t* place;  // [T,top_k]
  const float* weights;  // [T,top_k]
  int64_t T;
  int top_k;
  int64_t N;
  const void* residual;  // [T,N] of y_dtype, or null
  int64_t ld_res;
  void* Y;
  int64_t ldy;
  int y_dtype;
  const float* r_scale;  // [n, r_blocks] a factor per row and 128 features of rows, or null
  int64_t r_blocks;
};
int launch_combine(const CombineArgs& a, cudaStream_t stream);
cudaError_t route_error_word(int** p);

// Codes and scales by token, or X itself, to codes and scales in the plan's order.
int launch_gather(const uint8_t* Q, const float* s, int64_t K, const Rows& r, uint8_t* Q_out, float* s_out,
                  cudaStream_t stream);
int launch_pack_sorted(const void* X, int x_dtype, int64_t T, int64_t K, int64_t ldx, const int32_t* place, int top_k,
                       uint8_t* Q, float* s, cudaStream_t stream);

// launch_plan, and X packed by token; in one launch where the choices are few.
int launch_plan_pack(const int32_t* experts, int64_t n, int E, int32_t* order, int32_t* place, int32_t* offsets,
                     void* workspace, const void* X, int x_dtype, int64_t T, int64_t K, int64_t ldx, int top_k, uint8_t* Q,
                     float* s, cudaStream_t stream);

// Whether n rows of E experts are taken by the kernel for many rows per expert,
// which wants them in the plan's order (r.order null).
bool many_rows(int64_t n, int E);
// expert_gemm.cu: n, T > 0, every width > 0. With `powers` [n, ceil(N/128)], Y
// (binary16) is stored divided by a power of two per row and 128 features, to
// be read with it by launch_combine (its r_scale).
int launch_expert_swiglu(const uint8_t* Q, const float* s, int64_t K, const Rows& r, const convrot_experts& gate,
                         const convrot_experts& up, uint8_t* Q_h, float* s_h, cudaStream_t stream,
                         uint64_t test_wait_ns = 0);
int launch_expert_linear(const uint8_t* Q, const float* s, int64_t K, const Rows& r, const convrot_experts& w, void* Y,
                         int64_t ldy, int y_dtype, float* powers, cudaStream_t stream, uint64_t test_wait_ns = 0);
// expert_pair.cu, expert_few.cu
cudaError_t pair_error_word(int** p);
cudaError_t few_error_word(int** p);

}  // namespace moe
}  // namespace convrot
