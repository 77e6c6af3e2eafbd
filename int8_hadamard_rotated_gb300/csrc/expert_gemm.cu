// expert_gemm.cu -- the block-scaled 8-bit floating-point linears over rows
// sorted by expert: rows of one expert go through that expert's matrix.
//
//   y[i,n] = sum_b s_x[m,b] s_w[e,n/128,b] (sum_{k in b} q_x[m,k] q_w[e,n,k]) + bias[e,n],
//   m = the activation row of sorted row i, e = its expert,
//
// and, for a gate and an up matrix, h = silu(g) u, quantized over 128 features
// as it leaves. Which kernel takes them.
#include "expert_common.cuh"

namespace convrot {
namespace moe {

// By the rows that an expert has on average. 64 experts of 3 x 1024 x 2048 (16 of
// 3 x 1536 x 4096), gate and up plus down: 48 rows each take 121 us (85) with
// the few-row kernel and 124 us (96) with the other, 64 rows 126 us (95) and 124
// us (96), 80 rows 149 us (129) and 125 us (96).
bool many_rows(int64_t n, int E) { return n / E > 64; }

int launch_expert_swiglu(const uint8_t* Q, const float* s, int64_t K, const Rows& r, const convrot_experts& gate,
                         const convrot_experts& up, uint8_t* Q_h, float* s_h, cudaStream_t stream,
                         uint64_t test_wait_ns) {
  const ExpertCall c{Q, s, K, r, &gate, &up, Q_h, s_h, gate.N, 0, test_wait_ns};
  return many_rows(r.n, r.E) ? launch_expert_pair(c, stream) : launch_expert_few(c, stream);
}

int launch_expert_linear(const uint8_t* Q, const float* s, int64_t K, const Rows& r, const convrot_experts& w, void* Y,
                         int64_t ldy, int y_dtype, float* powers, cudaStream_t stream, uint64_t test_wait_ns) {
  const ExpertCall c{Q, s, K, r, &w, nullptr, Y, powers, ldy, y_dtype, test_wait_ns};
  return many_rows(r.n, r.E) ? launch_expert_pair(c, stream) : launch_expert_few(c, stream);
}

}  // namespace moe
}  // namespace convrot
