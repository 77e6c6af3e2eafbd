// fp8_common.cuh -- helpers shared by the block norms (block_norm.cuh), the
// 8-bit floating-point pack (fp8_pack.cu) and the block-scaled GEMM
// (fp8_gemm.cu): element conversion, the e4m3 block quantizer, bulk loads and
// the host-side launchers.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace convrot {
namespace fp8 {

constexpr int QBLOCK = CONVROT_FP8_BLOCK;  // features that share one scale (128)
constexpr float kE4M3Max = 448.0f;

// ---------------------------------------------------------------------------
// element types
// ---------------------------------------------------------------------------

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two values as the bits of two consecutive 16-bit elements (round to nearest
// even; a's at the lower address).
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
template <typename T> __device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b);
template <> __device__ __forceinline__ void unpack2<__half>(uint32_t w, float& a, float& b) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  a = f.x;
  b = f.y;
}
template <> __device__ __forceinline__ void unpack2<__nv_bfloat16>(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}

// Lane-wise pairs, and four or eight consecutive elements as pairs, at an
// address (global or shared) aligned to their size, at most 16 bytes.
typedef unsigned long long Pair;
__device__ __forceinline__ void load4(const float* p, Pair& a, Pair& b) {
  const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
  a = v.x;
  b = v.y;
}
template <typename T>
__device__ __forceinline__ Pair widen2(uint32_t w) {
  float a, b;
  unpack2<T>(w, a, b);
  return f32x2_pack(a, b);
}
__device__ __forceinline__ void load8(const float* p, Pair (&x)[4]) {
  load4(p, x[0], x[1]);
  load4(p + 4, x[2], x[3]);
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, Pair (&x)[4]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  x[0] = widen2<T>(v.x);
  x[1] = widen2<T>(v.y);
  x[2] = widen2<T>(v.z);
  x[3] = widen2<T>(v.w);
}
template <typename T>
__device__ __forceinline__ uint32_t narrow2(Pair x) {
  float a, b;
  f32x2_unpack(x, a, b);
  return pack2<T>(a, b);
}
__device__ __forceinline__ void store4(float* p, Pair a, Pair b) {
  *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(a, b);
}
template <typename T>
__device__ __forceinline__ void store4(T* p, Pair a, Pair b) {
  *reinterpret_cast<uint2*>(p) = make_uint2(narrow2<T>(a), narrow2<T>(b));
}
__device__ __forceinline__ void store8(float* p, const Pair (&x)[4]) {
  store4(p, x[0], x[1]);
  store4(p + 4, x[2], x[3]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Pair (&x)[4]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(narrow2<T>(x[0]), narrow2<T>(x[1]), narrow2<T>(x[2]), narrow2<T>(x[3]));
}

// Sixteen consecutive elements as pairs; `vec`: the address is 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load16(const T* p, bool vec, Pair (&x)[8]) {
  if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      Pair v[4];
      load8(p + 8 * h, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * h + i] = v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = f32x2_pack(to_f32(p[2 * i]), to_f32(p[2 * i + 1]));
  }
}

// ---------------------------------------------------------------------------
// the e4m3 block quantizer
// ---------------------------------------------------------------------------

// The larger of two values; NaN if either is one, so that a block that holds
// a NaN gets a NaN scale instead of a finite one that hides it.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The codes of two values (a's in the low byte): round to nearest even,
// saturating at +-448; NaN becomes the NaN code.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// The codes of four values that are quotients already.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) { return e4m3x2(a, b) | (e4m3x2(c, d) << 16); }

// RN(x / s) without a division: a correction step after Markstein ("IA-64 and
// Elementary Functions", 2000). With r = RN(1 / s) and q0 = RN(x r), the result
// is RN(q0 + RN(x - q0 s) r), as long as everything stays normal.
//
// Markstein's proof asks for a q0 within one ulp of x / s, whose remainder is
// exact; here r's rounding and the product's put q0 up to 1.5 ulp away. So the
// step is not proven to give RN(x / s) for every x, and the codes do not need
// it: the result is within an ulp, which another code can come of only next to
// a rounding border of e4m3. There it was compared with the IEEE quotient on
// the CPU, for every significand of s, every significand of a border (16) and
// the eleven x around their product: 1.48e9 quotients, all equal (q0 up to
// 1.467 ulp off). Powers of two change nothing in the normal range. For the
// scale, s = 448, every significand of x was compared: all equal.

// The scale of a block, RN(amax / 448).
static __device__ __noinline__ float e4m3_scale_divided(float amax) { return __fdiv_rn(amax, kE4M3Max); }
__device__ __forceinline__ float e4m3_scale(float amax) {
  if (amax >= 0x1p-90f && amax <= 3.0e38f) {
    constexpr float r = 1.0f / kE4M3Max;
    const float q0 = __fmul_rn(amax, r);
    return __fmaf_rn(__fmaf_rn(-q0, kE4M3Max, amax), r, q0);
  }
  return e4m3_scale_divided(amax);  // 0, tiny, infinite, NaN
}

// Codes of four values with the scale s of their block by division: scales
// outside the correction step's range. Out of line, so that unrolled code
// does not carry a division per element.
static __device__ __noinline__ uint32_t e4m3_codes_divided(float a, float b, float c, float d, float s) {
  if (s == 0.0f) return 0u;
  return e4m3x4(__fdiv_rn(a, s), __fdiv_rn(b, s), __fdiv_rn(c, s), __fdiv_rn(d, s));
}

// Codes of 2 * NP values, as lane-wise pairs, with the scale s of their block:
// e4m3 of the IEEE quotient RN(x / s), and 0 where s is 0.
//
// The correction step is taken where s and 1 / s are normal and every x whose
// code is not 0 (|x| >= 2^-10 s) leaves the remainder normal: s >= 2^-90. It
// runs on the negated values, so that zeros keep their sign; the codes' sign
// bits are flipped at the end. Three packed operations and a conversion per
// two elements. (Two products that enclose the quotient, and the division
// where their codes differ, cost the same without ties, but 16-bit inputs are
// full of exact ties: the pack of bf16 [4608, 12288] took 51 us with them and
// 35 us with the correction step, everything else the same.)
// `nr` is -RN(1 / s) in that range.
__device__ __forceinline__ bool e4m3_corrected(float s) { return s >= 0x1p-90f && s <= 3.0e38f; }
__device__ __forceinline__ float e4m3_factor(float s) { return e4m3_corrected(s) ? -__frcp_rn(s) : 0.0f; }
template <int NP>
__device__ __forceinline__ void e4m3_codes(const unsigned long long (&x)[NP], float s, float nr,
                                           uint32_t (&out)[NP / 2]) {
  if (e4m3_corrected(s)) {
    const unsigned long long nr2 = f32x2_pack(nr, nr), s2 = f32x2_pack(s, s);
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) {
      float q[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const unsigned long long nq0 = f32x2_mul(x[2 * i + k], nr2);
        f32x2_unpack(f32x2_fma(f32x2_fma(nq0, s2, x[2 * i + k]), nr2, nq0), q[2 * k], q[2 * k + 1]);
      }
      out[i] = e4m3x4(q[0], q[1], q[2], q[3]) ^ 0x80808080u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) {
      float q[4];
      f32x2_unpack(x[2 * i], q[0], q[1]);
      f32x2_unpack(x[2 * i + 1], q[2], q[3]);
      out[i] = e4m3_codes_divided(q[0], q[1], q[2], q[3], s);
    }
  }
}

// The largest magnitude of 2 * NP values (NaN if one is).
template <int NP>
__device__ __forceinline__ float max_magnitude(const unsigned long long (&x)[NP]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    float a, b;
    f32x2_unpack(x[i], a, b);
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(a), "f"(b));
  }
  return m;
}

// ---------------------------------------------------------------------------
// untiled bulk loads
// ---------------------------------------------------------------------------

// Global -> shared, 16-byte aligned on both sides, bytes % 16 == 0, counted
// on `bar`.
__device__ __forceinline__ void bulk_load(void* sdst, const void* gsrc, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_u32(sdst)), "l"(gsrc), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

inline size_t dtype_size(int dtype) { return dtype == CONVROT_F32 ? 4 : 2; }
inline bool known_dtype(int dtype) { return dtype == CONVROT_F32 || dtype == CONVROT_F16 || dtype == CONVROT_BF16; }
inline int64_t n_blocks(int64_t n) { return (n + QBLOCK - 1) / QBLOCK; }

// A launch that may set itself up while the kernel before it in the stream
// ends. Every kernel here waits for that one before it reads or writes global
// memory; the one that streams weights (fp8_gemm.cu) asks for them in L2 before,
// which only moves them: what the kernel before still writes is seen.
struct Launch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  Launch(unsigned grid, unsigned block, size_t smem, cudaStream_t stream, unsigned cluster = 1) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
  }
};

// fp8_pack.cu
int launch_fp8_pack(const void* X, int x_dtype, int64_t M, int64_t K, int64_t ldx, uint8_t* Q, float* s,
                    cudaStream_t stream);
int launch_fp8_weight(const void* W, int w_dtype, int64_t N, int64_t K, uint8_t* Q, float* s, cudaStream_t stream);

// Test of the block norms' timeout (convrot_test_block_norm_timeout): a limit
// for the launch's waits (0: none of this) and the row from which on no row is
// copied in.
struct NormTimeoutTest {
  uint64_t wait_ns = 0;
  int64_t row = -1;
};

// block_norm_*.cu, one per type T of H, Y and H_out: arguments already checked;
// M > 0. The second gives the address of the kernels' error word.
template <typename T>
int launch_block_norm_as(const convrot_block_norm_args& a, cudaStream_t stream, NormTimeoutTest test);
template <typename T>
cudaError_t norm_error_word(int** p);

// fp8_gemm.cu: every linear has N > 0; M > 0. launch_fp8_packing packs X
// itself, for few rows; *launched says whether the call is of that kind.
// test_wait_ns: a limit for the waits of a test of the timeout
// (fp8_test_linear_timeout), whose last tile is not loaded to its end; else 0.
int launch_fp8_packing(const void* X, int x_dtype, int64_t M, int64_t K, int64_t ldx, const convrot_fp8_weight* weights,
                       int n_weights, int y_dtype, cudaStream_t stream, bool* launched);
int launch_fp8_gemm(const uint8_t* Qx, const float* s_x, int64_t M, int64_t K, const convrot_fp8_weight* weights,
                    int n_weights, int y_dtype, cudaStream_t stream, uint64_t test_wait_ns = 0);

cudaError_t linear_error_word(int** p);  // the address of their error word

}  // namespace fp8
}  // namespace convrot
