// fp8_gemm.cuh -- what the block-scaled 8-bit floating-point GEMMs share (the
// dense linears of fp8_gemm.cu, the experts' of expert_gemm.cu): the MMA and its
// tensor-memory accumulators, their promotion with the block scales, stores,
// waits by whole warps, and the tensor maps.
#pragma once

#include "fp8_common.cuh"

namespace convrot {
namespace fp8 {

constexpr int BK = QBLOCK;      // K per stage: 128 codes = 128 bytes
constexpr int UMMA_K = 32;      // K of one kind::f8f6f4 MMA
constexpr int LANES = 128;      // TMEM lanes: rows of the MMA's first operand per CTA

// Instruction descriptor, kind::f8f6f4: e4m3 A and B (format 0, K-major),
// fp32 D.
//   bits 4-5 D format (1 = f32)   bits 7-9 A format   bits 10-12 B format
//   bits 17-22 N >> 3             bits 24-28 M >> 4
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

template <int CG>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// The MMAs of one block of K on the operand tiles at `sa` and `sb`.
template <int CG>
__device__ __forceinline__ void mma_block(uint32_t d_tmem, uint32_t sa, uint32_t sb, uint32_t idesc) {
  const uint64_t a = smem_desc_sw128(sa), b = smem_desc_sw128(sb);
#pragma unroll
  for (int k = 0; k < BK / UMMA_K; ++k) {
    const uint64_t off = static_cast<uint64_t>((k * UMMA_K) >> 4);
    mma_f8<CG>(d_tmem, a + off, b + off, idesc, k > 0 ? 1u : 0u);
  }
}

// 16 columns of the warp's 32 lanes, and the wait that hands them over (the
// registers pass through the wait, so no use can be moved before it).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :: "memory");
}
__device__ __forceinline__ unsigned long long pair_bits(uint32_t a, uint32_t b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}

// Loads that stay where they are written (the compiler would move plain ones
// down to their first use, next to it in time).
__device__ __forceinline__ float ldg_now(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float4 ldg_now4(const float* p) {
  float4 v;
  asm volatile("ld.global.nc.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}

// Four block scales of one row, from block kb on (0 past the last one).
__device__ __forceinline__ void load_scales(const float* row, int kb, int KB, bool vec, float (&v)[4]) {
  if (vec) {
    const float4 t = ldg_now4(row + kb);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = kb + i < KB ? ldg_now(row + kb + i) : 0.0f;
  }
}

// 16 bytes of consecutive outputs, each rounded once.
template <typename TY, int E>
__device__ __forceinline__ uint4 pack16(const float (&v)[E]) {
  static_assert(E * sizeof(TY) == 16, "sixteen bytes");
  if constexpr (E == 4)
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  else
    return make_uint4(pack2<TY>(v[0], v[1]), pack2<TY>(v[2], v[3]), pack2<TY>(v[4], v[5]), pack2<TY>(v[6], v[7]));
}
// Four consecutive outputs, each rounded once, at an address aligned to them.
template <typename TY>
__device__ __forceinline__ void store4(TY* p, const float (&v)[4]) {
  if constexpr (sizeof(TY) == 4)
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<TY>(v[0], v[1]), pack2<TY>(v[2], v[3]));
}

constexpr int STORE_ROW = 128;                 // bytes of a row that one store takes

// Where the store's 128-byte swizzle puts 16-byte piece `ch` of row `row`.
__device__ __forceinline__ int swizzled(int ch, int row) { return ch ^ (row & 7); }

// A staged block to rows of Y that no tensor map covers, element by element.
// Out of line: the unrolled epilogue carries one call of it per block.
template <typename TY>
static __device__ __noinline__ void store_rows(const uint8_t* sb, TY* y, int64_t ldy, int rows, int cols) {
  const int lane = threadIdx.x & 31;
  constexpr int PER = STORE_ROW / sizeof(TY);
  for (int r = 0; r < rows; ++r, y += ldy)
    for (int k = lane; k < PER && k < cols; k += 32) {
      const int byte = k * static_cast<int>(sizeof(TY));
      y[k] = *reinterpret_cast<const TY*>(sb + r * STORE_ROW + ((swizzled(byte >> 4, r) << 4) | (byte & 15)));
    }
}

// mbar_wait by a whole warp, with one outcome for all its lanes: each waits by
// itself, and one may give up just before the phase completes for another,
// while what follows (tcgen05 loads, warp barriers) wants the warp together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err,
                                          uint64_t limit_ns) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, err, limit_ns));
}

// warp_wait by a warp that is in no hurry: one lane looks, now and then.
__device__ __forceinline__ bool wait_slowly(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err,
                                            uint64_t limit_ns) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
      __nanosleep(400);
      if (*abort_flag || global_timer_ns() - t0 > limit_ns) {
        if (!*abort_flag) record_error(err, CONVROT_ERR_TIMEOUT);
        *abort_flag = 1;
        ok = 0;
        break;
      }
    }
  }
  ok = __shfl_sync(0xffffffffu, ok, 0);
  return __all_sync(0xffffffffu, ok != 0 && mbar_try_wait(bar, parity));
}

// Adds f times the accumulator at `ta` (COLS columns of the warp's lanes) to acc.
template <int COLS>
__device__ __forceinline__ void drain(unsigned long long (&acc)[COLS / 2], uint32_t ta, unsigned long long f2) {
  uint32_t r[2][16];
  tmem_ld16(ta, r[0]);
#pragma unroll
  for (int q = 0; q < COLS / 16; ++q) {
    tmem_wait16(r[q & 1]);
    if (q + 1 < COLS / 16) tmem_ld16(ta + (q + 1) * 16, r[(q + 1) & 1]);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      acc[q * 8 + k] = f32x2_fma(pair_bits(r[q & 1][2 * k], r[q & 1][2 * k + 1]), f2, acc[q * 8 + k]);
  }
}

// The same for n <= KG accumulators of COLS columns side by side (KG * COLS
// <= 64), each with a factor per column, read from shared memory at f + its
// index * COLS. One wait for all of them.
template <int COLS, int KG>
__device__ __forceinline__ void drain_scaled(unsigned long long (&acc)[COLS / 2], uint32_t ta, const float* f, int n) {
  constexpr int PER = COLS / 16;  // loads per accumulator
  uint32_t r[KG * PER][16];
#pragma unroll
  for (int q = 0; q < KG * PER; ++q) tmem_ld16(ta + q * 16, r[q]);
#pragma unroll
  for (int q = 0; q < KG * PER; ++q) tmem_wait16(r[q]);
#pragma unroll
  for (int g = 0; g < KG; ++g) {
    if (g >= n) break;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const uint32_t(&v)[16] = r[g * PER + q];
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float4 s = *reinterpret_cast<const float4*>(f + g * COLS + q * 16 + 2 * k);
        acc[q * 8 + k] = f32x2_fma(pair_bits(v[2 * k], v[2 * k + 1]), f32x2_pack(s.x, s.y), acc[q * 8 + k]);
        acc[q * 8 + k + 1] =
            f32x2_fma(pair_bits(v[2 * k + 2], v[2 * k + 3]), f32x2_pack(s.z, s.w), acc[q * 8 + k + 1]);
      }
    }
  }
}

// Arrive on an mbarrier of either CTA of the pair with a CTA-scope release.
// What is handed over is an accumulator that this thread has read (the wait
// for the tcgen05 loads came before), no memory that another CTA would have to
// see: a cluster-scope release, which orders every earlier access of the
// thread at the cluster, costs about 0.5 us for each block here.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Four outputs of a row from feature n on, each rounded once; `vec`: all of them
// exist and the address is aligned to them.
template <typename TY>
__device__ __forceinline__ void store_outputs(TY* yr, bool vec, int n, int N, const float (&v)[4]) {
  if (vec) {
    store4(yr, v);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n + k < N) yr[k] = from_f32<TY>(v[k]);
  }
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// d += a b for 16 weight rows and 8 activation rows over 32 places of K.
__device__ __forceinline__ void mma_sync_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// e4m3 codes [rows,K] (dense), box box_rows x 128 codes, 128-byte swizzle.
inline int make_tmap_codes(CUtensorMap* m, const void* base, int64_t rows, int64_t K, int box_rows) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return set_cuda_error(cudaErrorNotSupported);
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(BK), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? CONVROT_OK : set_cuda_error(cudaErrorInvalidValue);
}

// Y [rows,cols], box 32 rows x 128 bytes, 128-byte swizzle.
inline int make_tmap_out(CUtensorMap* m, void* base, int y_dtype, int64_t rows, int64_t cols, int64_t ldy) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return set_cuda_error(cudaErrorNotSupported);
  const cuuint64_t size = dtype_size(y_dtype);
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ldy) * size};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(STORE_ROW / size), 32};
  const cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType type = y_dtype == CONVROT_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : y_dtype == CONVROT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                            : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUresult r = enc(m, type, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? CONVROT_OK : set_cuda_error(cudaErrorInvalidValue);
}

}  // namespace fp8
}  // namespace convrot
