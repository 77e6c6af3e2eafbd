// expert_common.cuh -- what the experts' GEMM kernels share: an expert's rows,
// the work list that the kernels derive from the plan, gathered tile loads and
// the experts' tensor maps.
#pragma once

#include "fp8_gemm.cuh"
#include "moe_common.cuh"

namespace convrot {
namespace moe {

using namespace fp8;

// One expert's first and last row, within [0, n] whatever the plan says.
__device__ __forceinline__ int2 rows_of(const Rows& r, int e) {
  const int n = static_cast<int>(r.n);
  const int a = min(max(__ldg(r.offsets + e), 0), n), b = min(max(__ldg(r.offsets + e + 1), a), n);
  return make_int2(a, b);
}
// The activation row of sorted row i.
__device__ __forceinline__ int source_row(const Rows& r, int i) {
  if (!r.order) return i;
  const int t = __ldg(r.order + i) / r.top_k;
  return min(max(t, 0), static_cast<int>(r.T) - 1);
}

// The row tiles of all experts, as a prefix sum over the experts in shared
// memory: first[e] is expert e's first tile of `tile` rows, first[E] their
// number. By one warp.
__device__ __forceinline__ void count_tiles(const Rows& r, int tile, int* first) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  for (int e0 = 0; e0 < r.E; e0 += 32) {
    const int e = e0 + lane;
    int tiles = 0;
    if (e < r.E) {
      const int2 c = rows_of(r, e);
      tiles = (c.y - c.x + tile - 1) / tile;
    }
    int scan = tiles;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, scan, d);
      if (lane >= d) scan += v;
    }
    if (e < r.E) first[e] = carry + scan - tiles;
    carry += __shfl_sync(0xffffffffu, scan, 31);
  }
  if (lane == 0) first[r.E] = carry;
}

// Work item w of n_cols columns of tiles for every expert: its expert, column
// and row tile. An expert's items are taken column by column, the row tiles of
// one column next to each other, so that those who share a weight tile run at
// the same time.
struct Item {
  int expert, col, tile;
};
__device__ __forceinline__ Item find_item(const int* first, int E, int n_cols, int w) {
  int lo = 0, hi = E - 1;  // the last expert whose items start at or before w
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] * n_cols <= w) lo = mid;
    else hi = mid - 1;
  }
  const int tiles = first[lo + 1] - first[lo], at = w - first[lo] * n_cols;
  Item i;
  i.expert = lo;
  i.col = at / tiles;
  i.tile = at - i.col * tiles;
  return i;
}

// The same where shared memory is short: a prefix sum over groups of eight
// experts, whose own tiles are counted again when an item is looked up. Both by
// one warp; the item's rows [x, y) of the expert come with it.
constexpr int GROUP = 8;
__device__ __forceinline__ int tiles_of(const Rows& r, int e, int tile, int2& c) {
  c = e < r.E ? rows_of(r, e) : make_int2(0, 0);
  return (c.y - c.x + tile - 1) / tile;
}
__device__ __forceinline__ void count_tiles_grouped(const Rows& r, int tile, int* first) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  for (int e0 = 0; e0 < r.E; e0 += 32) {
    int2 c;
    int scan = tiles_of(r, e0 + lane, tile, c);
    const int tiles = scan;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, scan, d);
      if (lane >= d) scan += v;
    }
    if (lane % GROUP == 0 && e0 + lane < r.E) first[(e0 + lane) / GROUP] = carry + scan - tiles;
    carry += __shfl_sync(0xffffffffu, scan, 31);
  }
  if (lane == 0) first[(r.E + GROUP - 1) / GROUP] = carry;
}
__device__ __forceinline__ Item find_item_grouped(const Rows& r, int tile, const int* first, int n_cols, int w, int2& range) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = (r.E + GROUP - 1) / GROUP - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] * n_cols <= w) lo = mid;
    else hi = mid - 1;
  }
  int2 c = make_int2(0, 0);
  const int tiles = lane < GROUP ? tiles_of(r, lo * GROUP + lane, tile, c) : 0;
  int start = tiles;
#pragma unroll
  for (int d = 1; d < GROUP; d *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, start, d);
    if (lane >= d) start += v;
  }
  start = (first[lo] + start - tiles) * n_cols;
  const uint32_t here = __ballot_sync(0xffffffffu, w >= start && w < start + tiles * n_cols);
  const int src = __ffs(here) - 1, of = __shfl_sync(0xffffffffu, tiles, src);
  const int at = w - __shfl_sync(0xffffffffu, start, src);
  range = make_int2(__shfl_sync(0xffffffffu, c.x, src), __shfl_sync(0xffffffffu, c.y, src));
  Item i;
  i.expert = lo * GROUP + src;
  i.col = at / of;
  i.tile = at - i.col * of;
  return i;
}

__device__ __forceinline__ unsigned long long f32x2_add(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// silu(g) u = g u sigmoid(g): a relative error of a few 1e-7 and |g| 2^-24 from
// the exponent's rounding while the sigmoid is a normal number (g > -87.3);
// below, it is off by up to 2^-149.
__device__ __forceinline__ float silu_mul(float g, float u) { return g * sigmoid_fast(g) * u; }

// Rows that only moe_combine reads, on the way to a bf16 output: binary16
// with a power of two per row and 128 features that brings the largest
// magnitude just below 2^15, so that every value within 2^-29 of it keeps 11
// bits (a row's rounding is an eighth of bf16's) and none overflows; smaller
// ones are subnormal, off by up to 2^-39 of the largest.
struct ScaledHalf {};
template <typename TY> constexpr bool SCALED = false;
template <> inline constexpr bool SCALED<ScaledHalf> = true;
template <typename TY> struct StoredAs { using type = TY; };
template <> struct StoredAs<ScaledHalf> { using type = __half; };
template <typename TY> using Stored = typename StoredAs<TY>::type;

// What a value has to do with the choice of the power: infinities and NaN stay
// what they are under any, and must not push their finite neighbours out.
__device__ __forceinline__ float finite_magnitude(float v) { return fabsf(v) <= 3.402823466e38f ? fabsf(v) : 0.0f; }
// 2^-14 of the power of two at or below a finite `top` >= 0, at least 2^-126.
__device__ __forceinline__ float power_of(float top) {
  const uint32_t e = __float_as_uint(top) >> 23;
  return e < 15u ? 0x1p-126f : __uint_as_float((e - 14u) << 23);
}

// Four rows of a matrix (box one row high) to four consecutive rows of a tile.
__device__ __forceinline__ void tma_gather4(void* smem_dst, const void* tmap, uint64_t* bar, int32_t x, int4 rows,
                                            uint64_t cache_hint) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;"
      ::"r"(smem_u32(smem_dst)), "l"(tmap), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w),
      "r"(smem_u32(bar)), "l"(cache_hint)
      : "memory");
}
// Whether the phase with the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}

// A box of a three-dimensional map (an expert's matrix), counted on an mbarrier
// of either CTA of the pair.
__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const void* tmap, uint32_t bar_cluster_addr, int32_t x,
                                                 int32_t y, int32_t z, uint64_t cache_hint) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;"
      ::"r"(smem_u32(smem_dst)), "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar_cluster_addr), "l"(cache_hint)
      : "memory");
}

// The codes [N,K] of E experts, box box_rows x 128 codes of one expert: rows
// past N are zeros, not the next expert's.
inline int make_tmap_experts(CUtensorMap* m, const convrot_experts& w, int64_t E, int64_t K, int box_rows) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return set_cuda_error(cudaErrorNotSupported);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(w.N), static_cast<cuuint64_t>(E)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(K),
                                 static_cast<cuuint64_t>(E > 1 ? w.q_stride : (w.N * K + 15) / 16 * 16)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(BK), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(w.q), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? CONVROT_OK : set_cuda_error(cudaErrorInvalidValue);
}

// expert_pair.cu: many rows per expert. Both operators: `up` null for a linear,
// whose Y has the type y_dtype; else out are codes and s_out their scales.
struct ExpertCall {
  const uint8_t* Q;
  const float* s;
  int64_t K;
  Rows rows;
  const convrot_experts* w;
  const convrot_experts* up;
  void* out;
  float* s_out;
  int64_t ldy;
  int y_dtype;
  uint64_t test_wait_ns;
};
// A linear with s_out stores ScaledHalf rows, s_out [n, ceil(N/128)] their powers.
int launch_expert_pair(const ExpertCall& c, cudaStream_t stream);
// expert_few.cu: few rows per expert.
int launch_expert_few(const ExpertCall& c, cudaStream_t stream);

}  // namespace moe
}  // namespace convrot
