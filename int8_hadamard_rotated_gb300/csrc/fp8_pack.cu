// fp8_pack.cu -- activations and weights to 8-bit floating point (e4m3) with
// one fp32 scale per block: 1 x 128 features of an activation row, 128 x 128
// of a weight.
//
//   s = max |x| / 448 over the block,   q = e4m3(x / s)
//
// (448 is the largest e4m3 value; rounding to nearest even; an all-zero block
// has scale 0 and codes 0; a block that holds an infinity or a NaN has that
// as its scale, so the products it enters are not finite either.)
#include "fp8_common.cuh"

namespace convrot {
namespace fp8 {
namespace {

constexpr int PACK_THREADS = 256;

// Eight lanes per block of 128 features, 16 features per lane, one block per
// lane group: reads b_in and writes one byte per feature (and 4 bytes per
// 128), so bound by HBM, and what keeps enough loads in flight is how many
// warps fit an SM. bf16 [4608, 12288]: 26.7 us = 6.43 TB/s at 32 registers;
// 28.6 us without the bound on registers, 34.4 us with two blocks per group
// loaded ahead, 51.8 us with four.
template <typename T>
__global__ void __launch_bounds__(PACK_THREADS, sizeof(T) == 2 ? 8 : 6)
fp8_pack_kernel(const T* __restrict__ X, int64_t ldx, uint32_t n_qblocks, uint32_t KB, uint32_t K, bool vec,
                uint8_t* __restrict__ Q, float* __restrict__ s) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const uint32_t sub = threadIdx.x & 7, b = blockIdx.x * (PACK_THREADS / 8) + (threadIdx.x >> 3);
  const uint32_t row = b / KB, col = (b - row * KB) * QBLOCK + sub * 16;
  const bool on = b < n_qblocks && col < K;
  Pair x[8];
  if (on) {
    load16(X + row * ldx + col, vec, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0ull;
  }
  float m = max_magnitude(x);
#pragma unroll
  for (int d = 1; d < 8; d *= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float sc = e4m3_scale(m);
  uint32_t c[4];
  e4m3_codes(x, sc, e4m3_factor(sc), c);
  if (on) {
    *reinterpret_cast<uint4*>(Q + static_cast<int64_t>(row) * K + col) = make_uint4(c[0], c[1], c[2], c[3]);
    if (sub == 0) s[b] = sc;
  }
}

// One CTA per 128 x 128 block of a weight: 16 threads per 8 rows hold 64
// elements each. Offline; not on a hot path.
template <typename T>
__global__ void __launch_bounds__(256)
fp8_weight_kernel(const T* __restrict__ W, int64_t N, int64_t K, bool vec, uint8_t* __restrict__ Q,
                  float* __restrict__ s) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  __shared__ float part[8];
  const int64_t KB = (K + QBLOCK - 1) / QBLOCK;
  const int64_t nb = blockIdx.x / KB, kb = blockIdx.x - nb * KB;
  Pair x[4][8];
  float m = 0.0f;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int unit = threadIdx.x + 256 * u;
    const int64_t row = nb * QBLOCK + unit / 8, col = kb * QBLOCK + (unit & 7) * 16;
    if (row < N && col < K) {
      load16(W + row * K + col, vec, x[u]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u][i] = 0ull;
    }
    m = max_nan(m, max_magnitude(x[u]));
  }
#pragma unroll
  for (int d = 1; d < 32; d *= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max_nan(m, part[w]);
  const float sc = e4m3_scale(m), nr = e4m3_factor(sc);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int unit = threadIdx.x + 256 * u;
    const int64_t row = nb * QBLOCK + unit / 8, col = kb * QBLOCK + (unit & 7) * 16;
    uint32_t c[4];
    e4m3_codes(x[u], sc, nr, c);
    if (row < N && col < K) *reinterpret_cast<uint4*>(Q + row * K + col) = make_uint4(c[0], c[1], c[2], c[3]);
  }
  if (threadIdx.x == 0) s[blockIdx.x] = sc;
}

template <typename T>
int pack_as(const void* X, int64_t M, int64_t K, int64_t ldx, uint8_t* Q, float* s, cudaStream_t stream) {
  const int64_t KB = n_blocks(K), blocks = M * KB;
  const bool vec = aligned16(X) && (ldx * sizeof(T)) % 16 == 0;
  const int64_t per = PACK_THREADS / 8;
  Launch l(static_cast<unsigned>((blocks + per - 1) / per), PACK_THREADS, 0, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, fp8_pack_kernel<T>, static_cast<const T*>(X), ldx,
                                           static_cast<uint32_t>(blocks), static_cast<uint32_t>(KB),
                                           static_cast<uint32_t>(K), vec, Q, s);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

template <typename T>
int weight_as(const void* W, int64_t N, int64_t K, uint8_t* Q, float* s, cudaStream_t stream) {
  Launch l(static_cast<unsigned>(n_blocks(N) * n_blocks(K)), 256, 0, stream);
  const cudaError_t e =
      cudaLaunchKernelEx(&l.cfg, fp8_weight_kernel<T>, static_cast<const T*>(W), N, K, aligned16(W), Q, s);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

}  // namespace

int launch_fp8_pack(const void* X, int x_dtype, int64_t M, int64_t K, int64_t ldx, uint8_t* Q, float* s,
                    cudaStream_t stream) {
  if (x_dtype == CONVROT_F32) return pack_as<float>(X, M, K, ldx, Q, s, stream);
  if (x_dtype == CONVROT_F16) return pack_as<__half>(X, M, K, ldx, Q, s, stream);
  return pack_as<__nv_bfloat16>(X, M, K, ldx, Q, s, stream);
}

int launch_fp8_weight(const void* W, int w_dtype, int64_t N, int64_t K, uint8_t* Q, float* s, cudaStream_t stream) {
  if (w_dtype == CONVROT_F32) return weight_as<float>(W, N, K, Q, s, stream);
  if (w_dtype == CONVROT_F16) return weight_as<__half>(W, N, K, Q, s, stream);
  return weight_as<__nv_bfloat16>(W, N, K, Q, s, stream);
}

}  // namespace fp8
}  // namespace convrot
