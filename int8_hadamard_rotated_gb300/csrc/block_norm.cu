// block_norm.cu -- the norms before and after a transformer block fused with
// the block's gate and its residual, in one pass over the rows:
//
//   v  = block_scale * post(y)                  y: the block's output
//   h' = residual_scale * h + gate[s] * v       h: the residual stream
//   u  = pre(h');  u = u + u * scale[s] + shift[s]
//
// with s the row's sample, and post and pre each the identity, an RMS norm
// x / sqrt(mean(x^2) + eps) or a LayerNorm (x - mean) / sqrt(var + eps), times
// a weight and plus a bias where given. h' is rounded once to h's type; u is
// formed from the unrounded fp32 h' and either stored in a type of its own or
// quantized to e4m3 codes with one scale per 128 features (what fp8_linear
// reads). Statistics are fp32 sums in a fixed order: a thread's elements, the
// warp's lanes, the warps; the variance is taken around the warp's own mean
// first and corrected by the warps' distances from the row's mean, so that a
// large common offset does not cancel.
//
// Bound by HBM: per row h and y in, h' and u out, once each.
#include "fp8_common.cuh"

#include <algorithm>
#include <mutex>

namespace convrot {
namespace fp8 {

// Sticky device error word of the block norms: a bounded wait that gave up
// (CONVROT_ERR_TIMEOUT) or a row's sample outside [0, n_samples)
// (CONVROT_ERR_ARG).
__device__ int g_norm_error = 0;

namespace {

struct NormParams {
  const void* H;
  const void* Y;      // null: no block output
  void* H_out;        // null: not stored
  void* U;            // null: not stored
  uint8_t* Q;         // codes instead of U
  float* s;
  const float *post_weight, *post_bias, *pre_weight, *pre_bias, *gate, *scale, *shift;
  const int32_t* row_sample;
  int64_t ldh, ldy, ldho, ldu, ld_gate, ld_mod;
  int M, K, KB;
  int rows_per_sample, n_samples;
  int post, pre;
  float post_eps, pre_eps, residual_scale, block_scale;
  int stages;
  uint32_t row_smem;  // bytes of one staged row, a multiple of 128
};

// The sample whose gate, scale and shift apply to a row; -1 (none: gate 0, no
// modulation) after recording the error where row_sample is out of range.
__device__ __forceinline__ int sample_of(const NormParams& p, int row) {
  if (p.row_sample) {
    const int s = __ldg(p.row_sample + row);
    if (s >= 0 && s < p.n_samples) return s;
    if (threadIdx.x == 0) record_error(&g_norm_error, CONVROT_ERR_ARG);
    return -1;
  }
  return p.rows_per_sample > 0 ? row / p.rows_per_sample : 0;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// The affine forms that the two halves of a row apply: v = n_y * a + b on the
// normalized block output (gate and block_scale folded in), u = n_h * a + b
// on the normalized h' (modulation folded in: w (1 + scale), bias (1 + scale)
// + shift; 1 + scale is exact where it cancels).
struct Coef {
  float a, b;
};
__device__ __forceinline__ Coef post_coef(const NormParams& p, int s, int e) {
  Coef c{p.block_scale, 0.0f};
  if (p.gate) c.a *= s < 0 ? 0.0f : __ldg(p.gate + s * p.ld_gate + e);
  if (p.post_bias) c.b = c.a * __ldg(p.post_bias + e);
  if (p.post_weight) c.a *= __ldg(p.post_weight + e);
  return c;
}
__device__ __forceinline__ Coef pre_coef(const NormParams& p, int s, int e) {
  Coef c{p.pre_weight ? __ldg(p.pre_weight + e) : 1.0f, p.pre_bias ? __ldg(p.pre_bias + e) : 0.0f};
  if (p.scale && s >= 0) {
    const float f = 1.0f + __ldg(p.scale + s * p.ld_mod + e);
    c.a *= f;
    c.b *= f;
  }
  if (p.shift && s >= 0) c.b += __ldg(p.shift + s * p.ld_mod + e);
  return c;
}

__device__ __forceinline__ void load8_vec(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
// The same for eight consecutive features at a 16-byte aligned place.
__device__ __forceinline__ void post_coef8(const NormParams& p, int s, int e, float (&a)[8], float (&b)[8]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) { a[i] = p.block_scale; b[i] = 0.0f; }
  if (p.gate) {
    if (s >= 0) load8_vec(p.gate + s * p.ld_gate + e, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] *= s < 0 ? 0.0f : v[i];
  }
  if (p.post_bias) {
    load8_vec(p.post_bias + e, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = a[i] * v[i];
  }
  if (p.post_weight) {
    load8_vec(p.post_weight + e, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] *= v[i];
  }
}
__device__ __forceinline__ void pre_coef8(const NormParams& p, int s, int e, float (&a)[8], float (&b)[8]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) { a[i] = 1.0f; b[i] = 0.0f; }
  if (p.pre_weight) load8_vec(p.pre_weight + e, a);
  if (p.pre_bias) load8_vec(p.pre_bias + e, b);
  if (p.scale && s >= 0) {
    load8_vec(p.scale + s * p.ld_mod + e, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] *= 1.0f + v[i];
      b[i] *= 1.0f + v[i];
    }
  }
  if (p.shift && s >= 0) {
    load8_vec(p.shift + s * p.ld_mod + e, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] += v[i];
  }
}

// What a norm does to a row: x -> (x - mean) * rstd.
struct Stats {
  float mean, rstd;
};

// Statistics of a row of K elements spread over the CTA, V * 8 per thread
// (units of eight, `on` where the unit lies inside the row). One barrier;
// `red` holds 2 x 32 floats and alternates between two such buffers from one
// call to the next, so that the reads after one barrier are over before the
// next but one call writes.
template <int V>
__device__ __forceinline__ Stats row_stats(const float (&x)[V][8], const bool (&on)[V], int kind, float eps, int K,
                                           int n_warp, float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_warps = blockDim.x >> 5;
  Stats st{0.0f, 1.0f};
  float acc = 0.0f;
  if (kind == CONVROT_NORM_RMS) {
#pragma unroll
    for (int u = 0; u < V; ++u)
      if (on[u]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc = fmaf(x[u][i], x[u][i], acc);
      }
    acc = warp_sum(acc);
    if (lane == 0) red[warp] = acc;
    __syncthreads();
    const float total = warp_sum(lane < n_warps ? red[lane] : 0.0f);
    st.rstd = 1.0f / sqrtf(total / static_cast<float>(K) + eps);
    return st;
  }
#pragma unroll
  for (int u = 0; u < V; ++u)
    if (on[u]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc += x[u][i];
    }
  const float sum = warp_sum(acc);
  const float mean_w = n_warp > 0 ? sum / static_cast<float>(n_warp) : 0.0f;
  acc = 0.0f;
#pragma unroll
  for (int u = 0; u < V; ++u)
    if (on[u]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = x[u][i] - mean_w;
        acc = fmaf(d, d, acc);
      }
    }
  const float m2 = warp_sum(acc);
  if (lane == 0) {
    red[warp] = sum;
    red[32 + warp] = m2;
  }
  __syncthreads();
  // lane w recomputes warp w's count and mean
  int n_l = 0;
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int lo = (u * n_warps + lane) * 32 * 8;
    if (lane < n_warps) n_l += min(max(K - lo, 0), 32 * 8);
  }
  const float sum_l = lane < n_warps ? red[lane] : 0.0f;
  const float m2_l = lane < n_warps ? red[32 + lane] : 0.0f;
  st.mean = warp_sum(sum_l) / static_cast<float>(K);
  const float d = n_l > 0 ? sum_l / static_cast<float>(n_l) - st.mean : 0.0f;
  const float var = warp_sum(fmaf(static_cast<float>(n_l) * d, d, m2_l)) / static_cast<float>(K);
  st.rstd = 1.0f / sqrtf(var + eps);
  return st;
}

// Rows whose every part is a whole number of aligned 16-byte units.
//
// Persistent CTAs, each over a contiguous range of rows, one row at a time
// with V units of eight features per thread (unit u * blockDim + thread), the
// row in registers from its arrival to its last store. The rows of h and y
// come through a ring of shared-memory stages, filled by bulk copies that one
// thread issues several rows ahead, so that enough bytes are in flight
// whatever the reductions wait for; a stage is refilled after the row's first
// barrier, when every thread holds its part. With V = 1 a thread's
// coefficients (norm weights, gate, modulation) stay in registers and are
// read again only when the sample changes.
template <typename T, typename TU, int V, bool FP8>
__global__ void __launch_bounds__(512, 1)
block_norm_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[8];
  __shared__ float red[2][64];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, n_warps = blockDim.x >> 5;
  const uint32_t row_bytes = static_cast<uint32_t>(p.K) * sizeof(T);
  const uint32_t stage_bytes = p.row_smem * (p.Y ? 2u : 1u);
  const int r0 = static_cast<int>(static_cast<int64_t>(p.M) * blockIdx.x / gridDim.x);
  const int r1 = static_cast<int>(static_cast<int64_t>(p.M) * (blockIdx.x + 1) / gridDim.x);
  const T* H = static_cast<const T*>(p.H);
  const T* Y = static_cast<const T*>(p.Y);
  auto fetch = [&](int row, int st) {
    uint8_t* dst = smem + st * stage_bytes;
    mbar_arrive_expect_tx(&full[st], row_bytes * (Y ? 2u : 1u));
    bulk_load(dst, H + row * p.ldh, row_bytes, &full[st]);
    if (Y) bulk_load(dst + p.row_smem, Y + row * p.ldy, row_bytes, &full[st]);
  };
  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) mbar_init(&full[i], 1);
    abort_flag = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  if (tid == 0)
    for (int i = 0; i < p.stages && r0 + i < r1; ++i) fetch(r0 + i, i);

  bool on[V];
  int n_warp = 0;  // elements of the row that this warp holds
#pragma unroll
  for (int u = 0; u < V; ++u) {
    on[u] = (u * static_cast<int>(blockDim.x) + tid) * 8 < p.K;
    n_warp += min(max(p.K - (u * n_warps + (tid >> 5)) * 32 * 8, 0), 32 * 8);
  }
  float pa[8], pb[8], qa[8], qb[8];  // V = 1: the thread's coefficients of sample `cur`
  int cur = -2;
  int st = 0, phase = 0, flip = 0;
  for (int row = r0; row < r1; ++row) {
    const int s = sample_of(p, row);
    if (V == 1 && s != cur) {
      cur = s;
      if (on[0]) {
        if (Y) post_coef8(p, s, tid * 8, pa, pb);
        pre_coef8(p, s, tid * 8, qa, qb);
      }
    }
    float h[V][8], y[V][8];
    mbar_wait(&full[st], phase, &abort_flag, &g_norm_error);
    const T* sh = reinterpret_cast<const T*>(smem + st * stage_bytes);
    const T* sy = reinterpret_cast<const T*>(smem + st * stage_bytes + p.row_smem);
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int e = (u * blockDim.x + tid) * 8;
      if (on[u]) {
        load8(sh + e, h[u]);
        if (Y) load8(sy + e, y[u]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[u][i] = y[u][i] = 0.0f;
      }
    }
    // the next row of this stage, once a barrier has passed that follows every read above
    auto refill = [&] {
      if (tid == 0 && row + p.stages < r1) fetch(row + p.stages, st);
    };
    bool refilled = false;
    if (Y) {
      Stats ps{0.0f, 1.0f};
      if (p.post != CONVROT_NORM_NONE) {
        ps = row_stats<V>(y, on, p.post, p.post_eps, p.K, n_warp, red[flip]);
        flip ^= 1;
        refill();
        refilled = true;
      }
#pragma unroll
      for (int u = 0; u < V; ++u)
        if (on[u]) {
          if (V > 1) post_coef8(p, s, (u * blockDim.x + tid) * 8, pa, pb);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            h[u][i] = fmaf((y[u][i] - ps.mean) * ps.rstd, pa[i], fmaf(p.residual_scale, h[u][i], pb[i]));
        }
    } else {
#pragma unroll
      for (int u = 0; u < V; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) h[u][i] *= p.residual_scale;
    }
    if (p.H_out) {
      T* out = static_cast<T*>(p.H_out) + row * p.ldho;
#pragma unroll
      for (int u = 0; u < V; ++u)
        if (on[u]) store8(out + (u * blockDim.x + tid) * 8, h[u]);
    }
    Stats us{0.0f, 1.0f};
    if (p.pre != CONVROT_NORM_NONE) {
      us = row_stats<V>(h, on, p.pre, p.pre_eps, p.K, n_warp, red[flip]);
      flip ^= 1;
      if (!refilled) refill();
    } else if (!refilled) {
      __syncthreads();
      refill();
    }
    if (FP8 || p.U) {
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const int e = (u * blockDim.x + tid) * 8;
        float o[8];
        if (on[u]) {
          if (V > 1) pre_coef8(p, s, e, qa, qb);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = fmaf((h[u][i] - us.mean) * us.rstd, qa[i], qb[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = 0.0f;
        }
        if (FP8) {
          // sixteen lanes hold a block of 128
          float m = fabsf(o[0]);
#pragma unroll
          for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(o[i]));
#pragma unroll
          for (int d = 1; d < 16; d *= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
          const float sc = e4m3_scale(m);
          uint32_t c[2];
          e4m3_codes(o, sc, c);
          if (on[u]) {
            *reinterpret_cast<uint2*>(p.Q + static_cast<int64_t>(row) * p.K + e) = make_uint2(c[0], c[1]);
            if ((tid & 15) == 0) p.s[static_cast<int64_t>(row) * p.KB + e / QBLOCK] = sc;
          }
        } else if (on[u]) {
          store8(static_cast<TU*>(p.U) + row * p.ldu + e, o);
        }
      }
    }
    if (++st == p.stages) {
      st = 0;
      phase ^= 1;
    }
  }
}

// Rows of any width, alignment and stride: one row per CTA at a time, kept
// as fp32 in shared memory, elements taken one by one (thread t owns the
// elements t, t + blockDim, ...).
__device__ float block_sum(float v, float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_warps = blockDim.x >> 5;
  v = warp_sum(v);
  __syncthreads();  // the reads of the call before
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return warp_sum(lane < n_warps ? red[lane] : 0.0f);
}
__device__ Stats row_stats_any(const float* x, int kind, float eps, int K, float* red) {
  Stats st{0.0f, 1.0f};
  if (kind == CONVROT_NORM_NONE) return st;
  float acc = 0.0f;
  if (kind == CONVROT_NORM_LAYER) {
    for (int e = threadIdx.x; e < K; e += blockDim.x) acc += x[e];
    st.mean = block_sum(acc, red) / static_cast<float>(K);
    acc = 0.0f;
  }
  for (int e = threadIdx.x; e < K; e += blockDim.x) {
    const float d = x[e] - st.mean;
    acc = fmaf(d, d, acc);
  }
  st.rstd = 1.0f / sqrtf(block_sum(acc, red) / static_cast<float>(K) + eps);
  return st;
}

template <typename T, typename TU, bool FP8>
__global__ void __launch_bounds__(1024, 1)
block_norm_any_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ float x[];
  __shared__ float red[32];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const int s = sample_of(p, static_cast<int>(row));
    const T* h = static_cast<const T*>(p.H) + row * p.ldh;
    T* ho = p.H_out ? static_cast<T*>(p.H_out) + row * p.ldho : nullptr;
    Stats ps{0.0f, 1.0f};
    if (p.Y) {
      const T* y = static_cast<const T*>(p.Y) + row * p.ldy;
      for (int e = threadIdx.x; e < p.K; e += blockDim.x) x[e] = to_f32(y[e]);
      ps = row_stats_any(x, p.post, p.post_eps, p.K, red);
    }
    for (int e = threadIdx.x; e < p.K; e += blockDim.x) {
      float v = p.residual_scale * to_f32(h[e]);
      if (p.Y) {
        const Coef c = post_coef(p, s, e);
        v = fmaf((x[e] - ps.mean) * ps.rstd, c.a, v + c.b);
      }
      x[e] = v;
      if (ho) ho[e] = from_f32<T>(v);
    }
    if (FP8 || p.U) {
      const Stats us = row_stats_any(x, p.pre, p.pre_eps, p.K, red);
      for (int e = threadIdx.x; e < p.K; e += blockDim.x) {
        const Coef c = pre_coef(p, s, e);
        const float o = fmaf((x[e] - us.mean) * us.rstd, c.a, c.b);
        if (FP8) x[e] = o;
        else static_cast<TU*>(p.U)[row * p.ldu + e] = from_f32<TU>(o);
      }
      if (FP8) {
        __syncthreads();
        const int lane = threadIdx.x & 31;
        for (int kb = threadIdx.x >> 5; kb < p.KB; kb += blockDim.x >> 5) {
          const int e = kb * QBLOCK + lane * 4;  // K is a multiple of 16: whole groups of four
          float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          if (e < p.K) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = x[e + i];
          }
          float m = fabsf(o[0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) m = max_nan(m, fabsf(o[i]));
#pragma unroll
          for (int d = 1; d < 32; d *= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
          const float sc = e4m3_scale(m);
          uint32_t c[1];
          e4m3_codes(o, sc, c);
          if (e < p.K) *reinterpret_cast<uint32_t*>(p.Q + row * p.K + e) = c[0];
          if (lane == 0) p.s[row * p.KB + kb] = sc;
        }
      }
    }
    __syncthreads();  // the row's last reads, before the next row is written
  }
}

constexpr int MAX_SMEM = 227 * 1024 - 2048;
constexpr size_t RING_BYTES = 48 * 1024;  // of staged rows that a CTA keeps in flight, where they fit

// Shared memory beyond 48 KB, once per kernel and device.
template <typename F>
int allow_smem(F* kernel, uint64_t& done, std::mutex& mu) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return set_cuda_error(e);
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 64 || !((done >> dev) & 1u)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
    if (e != cudaSuccess) return set_cuda_error(e);
    if (dev < 64) done |= 1ull << dev;
  }
  return CONVROT_OK;
}

template <typename F>
int launch_rows(F* kernel, const NormParams& p, unsigned grid, unsigned threads, size_t smem, cudaStream_t stream) {
  Launch l(grid, threads, smem, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kernel, p);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

template <typename T, typename TU, int V, bool FP8>
int launch_vec(NormParams& p, int threads, cudaStream_t stream) {
  static std::mutex mu;
  static uint64_t done = 0;
  auto kernel = block_norm_kernel<T, TU, V, FP8>;
  if (int st = allow_smem(kernel, done, mu)) return st;
  const size_t stage = static_cast<size_t>(p.row_smem) * (p.Y ? 2 : 1);
  p.stages = static_cast<int>(std::min<size_t>(8, std::max<size_t>(2, RING_BYTES / stage)));
  while (p.stages > 1 && p.stages * stage > MAX_SMEM) --p.stages;
  const size_t smem = p.stages * stage;
  const int sms = device_sm_count();
  int per_sm = 1;
  if (p.M > sms) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
    if (e != cudaSuccess) return set_cuda_error(e);
  }
  const int grid = std::min(p.M, std::max(1, per_sm) * sms);
  return launch_rows(kernel, p, grid, threads, smem, stream);
}

template <typename T, typename TU, bool FP8>
int launch_typed(NormParams& p, bool vec, cudaStream_t stream) {
  const int units = (p.K + 7) / 8;
  const size_t stage = static_cast<size_t>(p.row_smem) * (p.Y ? 2 : 1);
  if (vec && units <= 4 * 512 && stage <= MAX_SMEM) {
    const int v = (units + 511) / 512;
    const int threads = ((units + v - 1) / v + 31) / 32 * 32;
    if (v == 1) return launch_vec<T, TU, 1, FP8>(p, threads, stream);
    if (v == 2) return launch_vec<T, TU, 2, FP8>(p, threads, stream);
    if (v == 3) return launch_vec<T, TU, 3, FP8>(p, threads, stream);
    return launch_vec<T, TU, 4, FP8>(p, threads, stream);
  }
  static std::mutex mu;
  static uint64_t done = 0;
  auto kernel = block_norm_any_kernel<T, TU, FP8>;
  if (int st = allow_smem(kernel, done, mu)) return st;
  const int threads = std::min(1024, (std::max(32, p.K / 4) + 31) / 32 * 32);
  const unsigned grid = std::min(p.M, device_sm_count() * std::max(1, 2048 / threads));
  return launch_rows(kernel, p, grid, threads, static_cast<size_t>(p.K) * 4, stream);
}

template <typename T>
int launch_from(NormParams& p, int u_dtype, bool fp8, bool vec, cudaStream_t stream) {
  if (fp8) return launch_typed<T, T, true>(p, vec, stream);
  if (u_dtype == CONVROT_F32) return launch_typed<T, float, false>(p, vec, stream);
  if (u_dtype == CONVROT_F16) return launch_typed<T, __half, false>(p, vec, stream);
  return launch_typed<T, __nv_bfloat16, false>(p, vec, stream);
}

}  // namespace

int launch_block_norm(const convrot_block_norm_args& a, cudaStream_t stream) {
  NormParams p{};
  p.H = a.H;
  p.Y = a.Y;
  p.H_out = a.H_out;
  p.U = a.U;
  p.Q = a.Q;
  p.s = a.s;
  p.post_weight = a.post_weight;
  p.post_bias = a.post_bias;
  p.pre_weight = a.pre_weight;
  p.pre_bias = a.pre_bias;
  p.gate = a.gate;
  p.scale = a.scale;
  p.shift = a.shift;
  p.row_sample = a.row_sample;
  p.ldh = a.ldh;
  p.ldy = a.ldy;
  p.ldho = a.ldho;
  p.ldu = a.ldu;
  p.ld_gate = a.ld_gate;
  p.ld_mod = a.ld_mod;
  p.M = static_cast<int>(a.M);
  p.K = static_cast<int>(a.K);
  p.KB = static_cast<int>(n_blocks(a.K));
  p.rows_per_sample = static_cast<int>(std::min<int64_t>(a.rows_per_sample, 0x7fffffff));
  p.n_samples = static_cast<int>(a.n_samples);
  p.post = a.Y ? a.post_norm : CONVROT_NORM_NONE;
  p.pre = a.pre_norm;
  p.post_eps = a.post_eps;
  p.pre_eps = a.pre_eps;
  p.residual_scale = a.residual_scale;
  p.block_scale = a.block_scale;
  const size_t sz = dtype_size(a.dtype), usz = dtype_size(a.u_dtype);
  p.row_smem = static_cast<uint32_t>((a.K * sz + 127) / 128 * 128);
  auto row_ok = [](const void* ptr, int64_t ld, size_t size) { return !ptr || (aligned16(ptr) && ld * size % 16 == 0); };
  const bool vec = a.K % 8 == 0 && row_ok(a.H, a.ldh, sz) && row_ok(a.Y, a.ldy, sz) && row_ok(a.H_out, a.ldho, sz) &&
                   row_ok(a.U, a.ldu, usz) && row_ok(a.gate, a.ld_gate, 4) && row_ok(a.scale, a.ld_mod, 4) &&
                   row_ok(a.shift, a.ld_mod, 4) && row_ok(a.post_weight, 0, 4) && row_ok(a.post_bias, 0, 4) &&
                   row_ok(a.pre_weight, 0, 4) && row_ok(a.pre_bias, 0, 4);
  const bool fp8 = a.Q != nullptr;
  if (a.dtype == CONVROT_F32) return launch_from<float>(p, a.u_dtype, fp8, vec, stream);
  if (a.dtype == CONVROT_F16) return launch_from<__half>(p, a.u_dtype, fp8, vec, stream);
  return launch_from<__nv_bfloat16>(p, a.u_dtype, fp8, vec, stream);
}

int read_and_clear_norm_error() {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_norm_error, sizeof(int));
  if (e != cudaSuccess) return set_cuda_error(e);
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_norm_error, &zero, sizeof(int));
    if (e != cudaSuccess) return set_cuda_error(e);
  }
  return v;
}

}  // namespace fp8
}  // namespace convrot
