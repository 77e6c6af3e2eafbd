// fp8_gemm.cu -- the block-scaled 8-bit floating-point GEMM on the sm_103a
// tensor cores (tcgen05 kind::f8f6f4 + TMA + TMEM).
//
//   Y[m,n] = sum_b s_x[m,b] s_w[n/128,b] P_b[m,n] + bias[n],
//   P_b[m,n] = sum of q_x[m,k] q_w[n,k] over the 128 features k of block b.
//
// The tensor cores sum one block, P_b, in an fp32 TMEM accumulator (the
// instruction has no room for a factor per block); the epilogue warps read
// it, multiply it by the two scales and add it to fp32 registers, which stay
// for the whole tile. So every block costs the MMA a commit and the epilogue
// one TMEM read and one multiply-add per output, and two or more accumulators
// alternate so that the MMA of a block overlaps the reading of the one before.
//
// Both operands are K-major rows of e4m3 codes; one block of K is one 128-byte
// swizzled row per operand row, so a pipeline stage is exactly one block. K
// past the end is filled with zero codes by the tensor maps.
#include "fp8_common.cuh"

#include <algorithm>
#include <mutex>

namespace convrot {
namespace fp8 {

// Sticky device error word of these kernels (timeouts of bounded waits).
__device__ int g_fp8_error = 0;

namespace {

constexpr int MAX_LIN = CONVROT_MAX_LINEARS;
constexpr int BK = QBLOCK;      // K per stage: 128 codes = 128 bytes
constexpr int UMMA_K = 32;      // K of one kind::f8f6f4 MMA
constexpr int LANES = 128;      // TMEM lanes: rows of the MMA's first operand per CTA

struct GemmParams {
  CUtensorMap tmap_x;             // codes [M,K]
  CUtensorMap tmap_w[MAX_LIN];    // codes [N_j,K]
  CUtensorMap tmap_y[MAX_LIN];    // Y_j [M,N_j], where tma_y
  const float* s_x;               // [M,KB]
  const float* s_w[MAX_LIN];      // [ceil(N_j/128),KB]
  const float* bias[MAX_LIN];
  void* out[MAX_LIN];
  int64_t ldy[MAX_LIN];
  int N[MAX_LIN];
  int tile_start[MAX_LIN + 1];    // prefix sums of column tiles per linear
  int M, KB;
  int n_mtiles, n_lin, total_tiles;
  int raster_mtiles;              // row tiles per raster group
  int split;                      // CTAs (one cluster) that share a tile's K
  bool tma_y;                     // every Y_j can be stored through its tensor map
  bool vec_scales;                // the scales of a row can be read four at a time
  uint64_t wait_ns;               // limit of every wait
  int withheld_tile;              // test of the timeout: the last block of K of this tile is not loaded; -1
};

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

struct Tile {
  int lin, nt, mt;
};
// Tiles are taken in groups of raster_mtiles row tiles, and inside a group
// column tile by column tile, so that the group's activation codes stay in L2
// while the weights stream through.
__device__ __forceinline__ Tile decode(const GemmParams& p, int t) {
  const int n_cols = p.tile_start[p.n_lin];
  const int per_group = p.raster_mtiles * n_cols;
  const int g = t / per_group, idx = t - g * per_group;
  const int gm = min(p.raster_mtiles, p.n_mtiles - g * p.raster_mtiles);
  const int col = idx / gm;
  Tile c;
  c.mt = g * p.raster_mtiles + (idx - col * gm);
  c.lin = 0;
#pragma unroll 1
  while (c.lin + 1 < p.n_lin && col >= p.tile_start[c.lin + 1]) ++c.lin;
  c.nt = col - p.tile_start[c.lin];
  return c;
}

// ---------------------------------------------------------------------------
// many rows: CTA pairs, activation rows on the TMEM lanes
// ---------------------------------------------------------------------------
//
// Persistent clusters of two CTAs; a tile is 256 activation rows x 256 output
// features, M = 256 MMAs issued by the even CTA, each CTA holding its 128 rows
// x 256 features. Activations take the lanes because a lane's row scale is then
// one register, and the 128 features of a warp's half tile share one weight
// scale: the promotion of a block is a single packed multiply-add per two
// outputs with one factor. Twelve warps: 0-7 promote and store (quarter = warp
// & 3 of the lanes, half = warp >> 2 of the features), 8 loads, 9 issues MMAs,
// 10 looks up each tile's place, scales and bias ahead of the epilogue, 11
// only completes the control warpgroup.
// Y leaves per warp through its own 4 KB of shared memory, 32 rows x 128
// bytes at a time in the 128-byte swizzle (no barrier between warps), by
// tensor-map stores where the rows of Y are 16-byte aligned, else by
// coalesced element stores.
//
// [4608, 3072] through three [3072, 3072] weights to bf16: 112 us = 2.3
// PFLOP/s; [4608, 12288] through [3072, 12288] to fp32: 138 us = 2.5 PFLOP/s
// (152 us under sustained load). Two chains bound it about equally. In copies
// of the kernel with parts left out, taken when the whole took 113 us, the MMAs
// with no loads and no promotion take 82 us on the first shape; with the loads
// 116 us, since a pair's operands (64 KB per block of K, all from L2) arrive at
// some 12 TB/s over the GPU; with the promotion and no loads 117 us: reading
// an accumulator out of TMEM and handing it back takes as long as a block's
// MMAs, and only two fit beside each other. The last tile's promotion and
// stores, and 648 tiles over 76 pairs (8.5 waves), cost another 10 %.

constexpr int EPI_WARPS = 8;
constexpr int PAIR_THREADS = (EPI_WARPS + 4) * 32;  // three warpgroups
// Registers: 168 a thread at launch; the control warpgroup gives up what the
// two epilogue warpgroups, which hold 128 accumulators a thread, take.
constexpr int LAUNCH_REGS = 168, CONTROL_REGS = 56, EPI_REGS = 224;
static_assert(2 * EPI_REGS + CONTROL_REGS <= 3 * LAUNCH_REGS, "within what the block was launched with");
constexpr int STORE_ROW = 128;                 // bytes of a row that one store takes
constexpr int STORE_BLOCK = 32 * STORE_ROW;    // one store: 32 rows
constexpr int STORE_BYTES = 2 * STORE_BLOCK;   // one warp's two store buffers

// What the epilogue needs to know of a tile, prepared by a warp of its own.
struct __align__(16) TileInfo {
  int lin, row, col, N;  // the linear, the tile's first row and feature, the linear's features
  const float* ws;       // the weight scales of the tile's first block of features
};
static_assert(sizeof(TileInfo) == 32, "as laid out in shared memory");

struct PairGeom {
  static constexpr int BN = 256;  // features of a tile
  static constexpr int X_BYTES = LANES * BK;
  static constexpr int W_BYTES = BN / 2 * BK;
  static constexpr int STAGE_BYTES = X_BYTES + W_BYTES;
  static constexpr int STAGES = 5;
  static constexpr int BUFS = 512 / BN;  // TMEM accumulators
  static constexpr uint32_t IDESC = idesc_e4m3_f32(256, BN);
  static constexpr int SMEM_OUT = STAGES * STAGE_BYTES;
  static constexpr int SMEM_BIAS = SMEM_OUT + EPI_WARPS * STORE_BYTES;  // [BN] fp32
  static constexpr int SMEM_INFO = SMEM_BIAS + BN * 4;                  // [2] TileInfo
  static constexpr int SMEM_BARS = SMEM_INFO + 2 * 32;
  static constexpr int SMEM_ALLOC = SMEM_BARS + (2 * STAGES + 2 * BUFS + 7) * 8 + 16 + 1024;
};
static_assert(PairGeom::SMEM_ALLOC <= 227 * 1024, "shared memory");

// Where the store's 128-byte swizzle puts 16-byte piece `ch` of row `row`.
__device__ __forceinline__ int swizzled(int ch, int row) { return ch ^ (row & 7); }

// A staged block to rows of Y that no tensor map covers, element by element.
// Out of line: the unrolled epilogue carries one call of it per block.
template <typename TY>
__device__ __noinline__ void store_rows(const uint8_t* sb, TY* y, int64_t ldy, int rows, int cols) {
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

template <typename TY>
__global__ void __launch_bounds__(PAIR_THREADS, 1)
fp8_pair_kernel(const __grid_constant__ GemmParams p) {
  using G = PairGeom;
  constexpr int BN = G::BN;
  constexpr int COLS = BN / 2;  // features per epilogue thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::SMEM_BARS);
  uint64_t* empty = full + G::STAGES;
  uint64_t* tfull = empty + G::STAGES;
  uint64_t* tempty = tfull + G::BUFS;
  uint64_t* done = tempty + G::BUFS;
  uint64_t* ifull = done + 1;    // [2] a tile's info is in shared memory
  uint64_t* iempty = ifull + 2;   // [2] and has been read
  uint64_t* bfull = iempty + 2;   // the same for its bias
  uint64_t* bempty = bfull + 1;
  TileInfo* info = reinterpret_cast<TileInfo*>(smem + G::SMEM_INFO);
  float* sbias = reinterpret_cast<float*>(smem + G::SMEM_BIAS);
  uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(bempty + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_smem + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int unit = static_cast<int>(cluster_id_x()), n_units = static_cast<int>(cluster_count_x());
  int* err = &g_fp8_error;

  if (threadIdx.x == EPI_WARPS * 32) {
    for (int s = 0; s < G::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < G::BUFS; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], EPI_WARPS * 2);
    }
    mbar_init(done, 1);
    for (int e = 0; e < 2; ++e) {
      mbar_init(&ifull[e], 1);
      mbar_init(&iempty[e], EPI_WARPS);
    }
    mbar_init(bfull, 1);
    mbar_init(bempty, EPI_WARPS);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&p.tmap_x);
    for (int j = 0; j < p.n_lin; ++j) tma_prefetch_desc(&p.tmap_w[j]);
  }
  if (warp == EPI_WARPS + 1) {
    tmem_alloc_pair(tmem_base_smem, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_base_smem;
  pdl_wait_prerequisites();
  pdl_launch_dependents();

  if (warp >= EPI_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CONTROL_REGS));
    if (warp == EPI_WARPS && lane == 0) {
      const uint64_t pol = l2_policy_evict_normal();
      const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
      uint32_t stage = 0, phase = 0, n_issued = 0;
      bool ok = true;
      for (int t = unit; ok && t < p.total_tiles; t += n_units) {
        const Tile c = decode(p, t);
        const int w_row = c.nt * BN + static_cast<int>(rank) * (BN / 2);
        const int x_row = c.mt * 256 + static_cast<int>(rank) * LANES;
        for (int kb = 0; kb < p.KB; ++kb) {
          if (t == p.withheld_tile && kb == p.KB - 1) break;
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, err, p.wait_ns)) { ok = false; break; }
          uint8_t* sx = smem + stage * G::STAGE_BYTES;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * G::STAGE_BYTES);
          const uint32_t fb = full_leader + stage * 8u;
          tma_load_2d_pair(sx, &p.tmap_x, fb, kb * BK, x_row, pol);
          tma_load_2d_pair(sx + G::X_BYTES, &p.tmap_w[c.lin], fb, kb * BK, w_row, pol);
          ++n_issued;
          if (++stage == G::STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // No copy may land after the CTAs exit. The even CTA's barriers count both
      // CTAs' bytes; where the odd one's wait gave up, it may have issued copies
      // that the even one does not wait for, and gives them 1 ms, a thousand
      // times what a copy takes.
      if (rank == 1 && !ok)
        for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < 1000000;) __nanosleep(10000);
      if (rank == 0)
        for (uint32_t s = 0; s < G::STAGES; ++s)
          if (n_issued > s) mbar_wait(&full[s], ((n_issued - 1 - s) / G::STAGES) & 1u, nullptr, err, p.wait_ns);
    }
    if (warp == EPI_WARPS + 1 && lane == 0 && rank == 0) {
      uint32_t stage = 0, phase = 0, buf = 0, bphase = 0;
      bool ok = true;
      for (int t = unit; ok && t < p.total_tiles; t += n_units) {
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort_flag, err, p.wait_ns) ||
              !mbar_wait(&tempty[buf], bphase ^ 1u, abort_flag, err, p.wait_ns)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sx = smem_u32(smem + stage * G::STAGE_BYTES);
          mma_block<2>(tmem_base + buf * BN, sx, sx + G::X_BYTES, G::IDESC);
          mma_commit_pair(&tfull[buf], 0x3u);
          mma_commit_pair(&empty[stage], 0x3u);
          if (++stage == G::STAGES) { stage = 0; phase ^= 1u; }
          if (++buf == G::BUFS) { buf = 0; bphase ^= 1u; }
        }
      }
      // all issued MMAs complete before TMEM is released
      mma_commit_pair(done, 0x1u);
      mbar_wait(done, 0, nullptr, err, p.wait_ns);
    }
    if (warp == EPI_WARPS + 2) {
      int i = 0;
      for (int t = unit; t < p.total_tiles; t += n_units, ++i) {
        const Tile c = decode(p, t);
        const int N = p.N[c.lin], n0 = c.nt * BN;
        const float* b = p.bias[c.lin];
        float v[BN / 32];
#pragma unroll
        for (int k = 0; k < BN / 32; ++k) v[k] = b && n0 + 32 * k + lane < N ? __ldg(b + n0 + 32 * k + lane) : 0.0f;
        if (!wait_slowly(&iempty[i & 1], ((i >> 1) & 1) ^ 1u, abort_flag, err, p.wait_ns)) break;
        if (lane == 0) {
          info[i & 1] = TileInfo{c.lin, c.mt * 256 + static_cast<int>(rank) * LANES, n0, N,
                                 p.s_w[c.lin] + static_cast<int64_t>(n0 / QBLOCK) * p.KB};
          mbar_arrive(&ifull[i & 1]);
        }
        __syncwarp();
        if (!wait_slowly(bempty, (i & 1) ^ 1u, abort_flag, err, p.wait_ns)) break;
#pragma unroll
        for (int k = 0; k < BN / 32; ++k) sbias[32 * k + lane] = v[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(bfull);
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t t_addr = tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) + half * COLS;
    const uint32_t tempty_leader = mapa_shared(smem_u32(tempty), 0);
    uint8_t* sout = smem + G::SMEM_OUT + warp * STORE_BYTES;
    uint32_t buf = 0, bphase = 0;
    bool ok = true;
    // a tile's info is read, and its first scales are loaded, before the
    // stores of the tile before it
    TileInfo c{};
    const float *xs = nullptr, *ws = nullptr;
    float nx[4], nw[4];
    auto start = [&](int i) {  // the CTA's tile i
      if (!warp_wait(&ifull[i & 1], (i >> 1) & 1u, abort_flag, err, p.wait_ns)) return false;
      c = info[i & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&iempty[i & 1]);
      c.row += 32 * quarter;  // the warp's first row
      c.col += half * COLS;   // and first feature
      // rows and features past the end read the last one's scales; their
      // outputs are not stored
      xs = p.s_x + static_cast<int64_t>(min(c.row + lane, p.M - 1)) * p.KB;
      ws = c.ws + (half && c.col < c.N ? p.KB : 0);
      load_scales(xs, 0, p.KB, p.vec_scales, nx);
      load_scales(ws, 0, p.KB, p.vec_scales, nw);
      return true;
    };
    int seq = 0;
    if (unit < p.total_tiles) ok = start(0);
    for (int t = unit; ok && t < p.total_tiles; t += n_units, ++seq) {
      unsigned long long acc[COLS / 2];
#pragma unroll
      for (int i = 0; i < COLS / 2; ++i) acc[i] = 0ull;
      // One block of K a turn, not unrolled: the loop stays small enough for
      // the instruction caches that it shares with the other warps.
      float f[4];  // the factors of this block and the next three at most
#pragma unroll 1
      for (int kb = 0; kb < p.KB; ++kb) {
        if (!warp_wait(&tfull[buf], bphase, abort_flag, err, p.wait_ns)) { ok = false; break; }
        tc_fence_after();
        if ((kb & 3) == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = nx[i] * nw[i];
          if (kb + 4 < p.KB) {
            load_scales(xs, kb + 4, p.KB, p.vec_scales, nx);
            load_scales(ws, kb + 4, p.KB, p.vec_scales, nw);
          }
        }
        drain<COLS>(acc, t_addr + buf * BN, f32x2_pack(f[0], f[0]));
        f[0] = f[1];
        f[1] = f[2];
        f[2] = f[3];
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty_leader + buf * 8u);
        if (++buf == G::BUFS) { buf = 0; bphase ^= 1u; }
      }
      if (!ok) break;
      const int lin = c.lin, N = c.N, y_row = c.row, y_col = c.col;
      if (t + n_units < p.total_tiles) ok = start(seq + 1);
      if (!warp_wait(bfull, seq & 1u, abort_flag, err, p.wait_ns)) break;
      // store: PER features of a row at a time
      constexpr int PER = STORE_ROW / sizeof(TY);
      constexpr int E = 16 / sizeof(TY);  // of them in 16 bytes
      static_assert((COLS / PER) % 2 == 0, "both store buffers equally often");
#pragma unroll
      for (int b = 0; b < COLS / PER; ++b) {
        // the two buffers in turn (an even number of blocks per tile): the
        // store before the last has been read
        uint8_t* sb = sout + (b & 1) * STORE_BLOCK;
        if (lane == 0) bulk_wait_read<1>();
        __syncwarp();
#pragma unroll
        for (int ch = 0; ch < PER / E; ++ch) {
          float v[E];
#pragma unroll
          for (int k = 0; k < E; k += 2) f32x2_unpack(acc[(b * PER + ch * E + k) / 2], v[k], v[k + 1]);
#pragma unroll
          for (int k = 0; k < E; k += 4) {
            const float4 bb = *reinterpret_cast<const float4*>(sbias + half * COLS + b * PER + ch * E + k);
            v[k] += bb.x;
            v[k + 1] += bb.y;
            v[k + 2] += bb.z;
            v[k + 3] += bb.w;
          }
          *reinterpret_cast<uint4*>(sb + lane * STORE_ROW + (swizzled(ch, lane) << 4)) = pack16<TY>(v);
        }
        const int n = y_col + b * PER;
        if (p.tma_y) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (n < N && y_row < p.M) tma_store_2d(&p.tmap_y[lin], sb, n, y_row);
            bulk_commit();
          }
        } else {
          __syncwarp();
          store_rows<TY>(sb, static_cast<TY*>(p.out[lin]) + y_row * p.ldy[lin] + n, p.ldy[lin], min(32, p.M - y_row), N - n);
          __syncwarp();
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bempty);
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  cluster_sync();
  if (warp == EPI_WARPS + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ---------------------------------------------------------------------------
// few rows: single CTAs, K split over a cluster
// ---------------------------------------------------------------------------
//
// One tile per cluster: 128 output features x BN activation rows (SWAP: the
// weight rows take the TMEM lanes, the activations the columns, down to 16 of
// them), or 128 activation rows x 128 features. The CTAs of a cluster take
// contiguous shares of K, so that with few tiles every SM still streams
// weights; each leaves its fp32 partial tile in its own shared memory (the
// stages are free by then) and, after a cluster barrier, sums a part of the
// rows over all CTAs in rank order through distributed shared memory: no
// workspace, no atomics, the same order every time.
// Bound by the chain of a CTA's blocks, about 0.3 us each from the last load to
// the promoted sums, against the time its weights take from HBM: 24 rows
// through [3072, 12288] take 12.9 us = 2.98 TB/s. With few blocks it is the
// fixed costs that count (setting up tensor memory, the cluster's barriers and
// sums): 331 rows through [1283, 1280], 33 tiles of ten blocks of K, take 6.3 us
// with K split in four, 7.4 us in two, 7.5 us unsplit, and 8.6 us with their
// pack, which alone takes 1.8 us. (Asking for the weights in L2 before the wait
// for the kernel ahead: 7.1 us instead of 6.6 us for 16 rows through three
// 3072 x 3072 linears.)
// Six warps: 0-3 promote (32 lanes each), 4 loads, 5 issues MMAs.

constexpr int SOLO_THREADS = 6 * 32;
constexpr int MAX_SPLIT = 4;  // CTAs of a cluster

template <int BN, bool SWAP>
struct SoloGeom {
  static constexpr int X_ROWS = SWAP ? BN : LANES;
  static constexpr int W_ROWS = QBLOCK;
  static constexpr int X_BYTES = X_ROWS * BK;
  static constexpr int W_BYTES = W_ROWS * BK;
  static constexpr int STAGE_BYTES = X_BYTES + W_BYTES;
  static constexpr int SCALE_BYTES = SWAP ? 4 * 2 * 4 * BN * 4 : 0;  // [warp][2][4 blocks][BN]
  // Few columns: two CTAs per SM, so that one's set-up and sums overlap the
  // other's loads (16 rows through three 3072 x 3072 linears, K split in four:
  // 6.7 us against 7.7 us with one CTA per SM and K split in two).
  static constexpr int STAGES = ((SWAP ? 96 : 200) * 1024) / STAGE_BYTES;
  // With few columns, KG blocks of K, each in an accumulator of its own, are
  // handed over together, which saves hand-overs: 12 rows through [3072, 12288]
  // 11.6 us, one block at a time 12.2 us. At more columns or shorter K it makes
  // little difference (24 rows 12.9 and 12.6 us, 16 rows through three 3072 x
  // 3072 linears 6.7 us both ways).
  static constexpr int KG = SWAP ? 64 / BN : 1;
  static constexpr int BUF_COLS = KG * BN;
  static constexpr int BUFS = SWAP ? 4 : 2;
  static constexpr int TMEM_COLS = BUFS * BUF_COLS;  // 256
  static constexpr uint32_t IDESC = idesc_e4m3_f32(LANES, BN);
  static constexpr int TILE_ROWS = X_ROWS;             // activation rows of a tile
  static constexpr int PITCH = SWAP ? QBLOCK : QBLOCK + 4;  // of the partial tile, floats
  static constexpr int SMEM_SCALES = STAGES * STAGE_BYTES;
  static constexpr int SMEM_BARS = SMEM_SCALES + SCALE_BYTES;
  static constexpr int SMEM_ALLOC = SMEM_BARS + (2 * STAGES + 2 * BUFS + 1) * 8 + 16 + 1024;
  static_assert(TILE_ROWS * PITCH * 4 <= STAGES * STAGE_BYTES, "the partial tile fits the stages");
  static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// What a warp leaves in place of its sums where a wait gave up: a NaN that no
// arithmetic forms (fp32 operations give 0x7fffffff). The CTA that adds the
// sums up has them in hand anyway, while a flag of each CTA beside them, read
// through distributed shared memory, costs 0.2 us.
constexpr uint32_t GAVE_UP = 0x7fc0dead;

// GAVE_UP for what a warp holds of a partial tile: `rows` rows from `part` on,
// one feature per lane. Out of line, off the path of every tile.
__device__ __noinline__ void mark_rows(float* part, int rows, int pitch) {
  for (int r = 0; r < rows; ++r) part[r * pitch + (threadIdx.x & 31)] = __uint_as_float(GAVE_UP);
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

// Sums the partial tiles that the cluster's CTAs hold at `smem` (ROWS
// activation rows x 128 features, PITCH floats apart) in rank order, adds the
// bias bv of the lane's four features (from feature n on) and stores: one row
// per warp at a time, the rows shared out over the CTAs. Every thread of the
// cluster comes here after a barrier that follows the last write. Nothing is
// stored where a wait gave up: the abort flag of a CTA alone, outputs whose sums
// are GAVE_UP in one of several CTAs (four neighbours are one warp's, so the
// first of them speaks for all).
template <typename TY, int ROWS, int PITCH>
__device__ __forceinline__ void finish_tile(const GemmParams& p, const Tile& c, int m0, int n, int rank,
                                            const uint8_t* smem, volatile int* abort_flag, const float (&bv)[4]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = min(ROWS, p.M - m0), N = p.N[c.lin];
  TY* Y = static_cast<TY*>(p.out[c.lin]) + static_cast<int64_t>(m0) * p.ldy[c.lin] + n;
  const int64_t ldy = p.ldy[c.lin];
  const bool vec_out = n + 4 <= N && ldy % 4 == 0 && (reinterpret_cast<uintptr_t>(Y) & (4 * sizeof(TY) - 1)) == 0;
  if (p.split == 1) {
    if (*abort_flag) return;
    for (int r = warp; r < rows; r += SOLO_THREADS / 32) {
      const float4 s = *reinterpret_cast<const float4*>(smem + (r * PITCH + lane * 4) * 4);
      store_outputs(Y + r * ldy, vec_out, n, N, {s.x + bv[0], s.y + bv[1], s.z + bv[2], s.w + bv[3]});
    }
    return;
  }
  for (int r = warp * p.split + rank; r < rows; r += (SOLO_THREADS / 32) * p.split) {
    const int off = (r * PITCH + lane * 4) * 4;
    float4 s[MAX_SPLIT];
#pragma unroll
    for (int j = 0; j < MAX_SPLIT; ++j)
      if (j < p.split) s[j] = ld_cluster_v4(mapa_shared(smem_u32(smem) + off, j));
    float v[4] = {s[0].x, s[0].y, s[0].z, s[0].w};
    bool whole = __float_as_uint(s[0].x) != GAVE_UP;
#pragma unroll
    for (int j = 1; j < MAX_SPLIT; ++j)
      if (j < p.split) {
        whole = whole && __float_as_uint(s[j].x) != GAVE_UP;
        v[0] += s[j].x;
        v[1] += s[j].y;
        v[2] += s[j].z;
        v[3] += s[j].w;
      }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] += bv[k];
    if (whole) store_outputs(Y + r * ldy, vec_out, n, N, v);
  }
  cluster_sync();  // the others' reads of this CTA's partial sums
}

template <typename TY, int BN, bool SWAP>
__global__ void __launch_bounds__(SOLO_THREADS, SWAP ? 2 : 1)
fp8_solo_kernel(const __grid_constant__ GemmParams p) {
  using G = SoloGeom<BN, SWAP>;
  extern __shared__ uint8_t smem_raw[];
  // the offset to the next 1024-byte boundary is the same in every CTA of a cluster
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::SMEM_BARS);
  uint64_t* empty = full + G::STAGES;
  uint64_t* tfull = empty + G::STAGES;
  uint64_t* tempty = tfull + G::BUFS;
  uint64_t* done = tempty + G::BUFS;
  uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_smem + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* err = &g_fp8_error;
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / p.split;
  const Tile c = decode(p, tile);
  const int N = p.N[c.lin];
  const int m0 = c.mt * G::TILE_ROWS, n0 = c.nt * QBLOCK;
  const int kb_begin = p.KB * rank / p.split, kb_end = p.KB * (rank + 1) / p.split;

  if (threadIdx.x == 4 * 32) {
    for (int s = 0; s < G::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < G::BUFS; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&p.tmap_x);
    tma_prefetch_desc(&p.tmap_w[c.lin]);
  }
  if (warp == 5) {
    tmem_alloc(tmem_base_smem, G::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_base_smem;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  // the bias of this lane's four features, for the end
  const int n = n0 + lane * 4;
  const float* bias = p.bias[c.lin];
  float bv[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) bv[k] = (bias && n + k < N) ? ldg_now(bias + n + k) : 0.0f;

  if (warp == 4) {
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_normal();
      uint32_t stage = 0, phase = 0, n_issued = 0;
      for (int kb = kb_begin; kb < kb_end; ++kb) {
        if (tile == p.withheld_tile && rank == p.split - 1 && kb == kb_end - 1) break;
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, err, p.wait_ns)) break;
        uint8_t* sx = smem + stage * G::STAGE_BYTES;
        mbar_arrive_expect_tx(&full[stage], G::STAGE_BYTES);
        tma_load_2d(sx + G::X_BYTES, &p.tmap_w[c.lin], &full[stage], kb * BK, n0, pol);
        tma_load_2d(sx, &p.tmap_x, &full[stage], kb * BK, m0, pol);
        ++n_issued;
        if (++stage == G::STAGES) { stage = 0; phase ^= 1u; }
      }
      // no copy may land once the stages hold partial sums, or after the exit
      for (uint32_t s = 0; s < G::STAGES; ++s)
        if (n_issued > s) mbar_wait(&full[s], ((n_issued - 1 - s) / G::STAGES) & 1u, nullptr, err, p.wait_ns);
    }
    __syncwarp();
  } else if (warp == 5) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, buf = 0, bphase = 0;
      bool ok = true;
      for (int kb0 = kb_begin; ok && kb0 < kb_end; kb0 += G::KG) {
        if (!mbar_wait(&tempty[buf], bphase ^ 1u, abort_flag, err, p.wait_ns)) break;
        for (int kb = kb0; kb < min(kb0 + G::KG, kb_end); ++kb) {
          if (!mbar_wait(&full[stage], phase, abort_flag, err, p.wait_ns)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sx = smem_u32(smem + stage * G::STAGE_BYTES), sw = sx + G::X_BYTES;
          mma_block<1>(tmem_base + buf * G::BUF_COLS + (kb - kb0) * BN, SWAP ? sw : sx, SWAP ? sx : sw, G::IDESC);
          mma_commit(&empty[stage]);
          if (++stage == G::STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        mma_commit(&tfull[buf]);
        if (++buf == G::BUFS) { buf = 0; bphase ^= 1u; }
      }
      mma_commit(done);
      mbar_wait(done, 0, nullptr, err, p.wait_ns);
    }
    __syncwarp();
  } else {
    const uint32_t t_addr = tmem_base + (static_cast<uint32_t>(32 * warp) << 16);
    const float* ws = p.s_w[c.lin] + static_cast<int64_t>(c.nt) * p.KB;
    // SWAP: lane l scales the activation rows (columns) l and l + 32; else
    // its own row
    constexpr int XR = SWAP ? (BN + 31) / 32 : 1;
    const float* xs[XR];
#pragma unroll
    for (int i = 0; i < XR; ++i) {
      const int r = SWAP ? m0 + (32 * i + lane) % BN : m0 + 32 * warp + lane;
      xs[i] = p.s_x + static_cast<int64_t>(min(r, p.M - 1)) * p.KB;
    }
    float* sc = reinterpret_cast<float*>(smem + G::SMEM_SCALES) + warp * (2 * 4 * BN);
    unsigned long long acc[BN / 2];
#pragma unroll
    for (int i = 0; i < BN / 2; ++i) acc[i] = 0ull;
    uint32_t buf = 0, bphase = 0;
    const bool vec = p.vec_scales && kb_begin % 4 == 0;
    float nx[XR][4], nw[4];
#pragma unroll
    for (int i = 0; i < XR; ++i) load_scales(xs[i], kb_begin, p.KB, vec, nx[i]);
    load_scales(ws, kb_begin, p.KB, vec, nw);
    float f[4];
    int flip = 1;
    bool ok = true;
#pragma unroll 1
    for (int kb = kb_begin, i = 0; kb < kb_end; kb += G::KG, i = (i + G::KG) & 3) {
      if (i == 0) {  // the factors of four blocks; the next four's scales are on their way meanwhile
        flip ^= 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[j] = nx[0][j] * nw[j];
          if (SWAP) {
#pragma unroll
            for (int k = 0; k < XR; ++k)
              if (BN >= 32 || lane < BN) sc[(flip * 4 + j) * BN + 32 * k + lane] = nx[k][j] * nw[j];
          }
        }
        if (SWAP) __syncwarp();
        if (kb + 4 < kb_end) {
#pragma unroll
          for (int k = 0; k < XR; ++k) load_scales(xs[k], kb + 4, p.KB, vec, nx[k]);
          load_scales(ws, kb + 4, p.KB, vec, nw);
        }
      }
      ok = warp_wait(&tfull[buf], bphase, abort_flag, err, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      const uint32_t ta = t_addr + buf * G::BUF_COLS;
      if constexpr (SWAP) drain_scaled<BN, G::KG>(acc, ta, sc + (flip * 4 + i) * BN, kb_end - kb);
      else drain<BN>(acc, ta, f32x2_pack(f[0], f[0]));
      f[0] = f[1];
      f[1] = f[2];
      f[2] = f[3];
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[buf]);
      if (++buf == G::BUFS) { buf = 0; bphase ^= 1u; }
    }
    // The partial tile, activation row by activation row. Every MMA of this
    // CTA has completed (the last block's commit was seen), so no stage is
    // read or filled any more.
    float* part = reinterpret_cast<float*>(smem);
    if (SWAP) {
#pragma unroll
      for (int i = 0; i < BN / 2; ++i) {
        float a, b;
        f32x2_unpack(acc[i], a, b);
        part[(2 * i) * G::PITCH + 32 * warp + lane] = a;
        part[(2 * i + 1) * G::PITCH + 32 * warp + lane] = b;
      }
    } else {
#pragma unroll
      for (int i = 0; i < BN / 4; ++i) {
        float4 v;
        f32x2_unpack(acc[2 * i], v.x, v.y);
        f32x2_unpack(acc[2 * i + 1], v.z, v.w);
        *reinterpret_cast<float4*>(part + (32 * warp + lane) * G::PITCH + 4 * i) = v;
      }
    }
    if (!ok) {
      __syncwarp();
      if (SWAP) mark_rows(part + 32 * warp, BN, G::PITCH);
      else
        for (int i = 0; i < 4; ++i) mark_rows(part + 32 * warp * G::PITCH + 32 * i, 32, G::PITCH);
    }
  }
  tc_fence_before();
  if (p.split > 1) cluster_sync(); else __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem_base, G::TMEM_COLS);
  }
  finish_tile<TY, G::TILE_ROWS, G::PITCH>(p, c, m0, n, rank, smem, abort_flag, bv);
}

// ---------------------------------------------------------------------------
// at most 8 rows: weights streamed to registers
// ---------------------------------------------------------------------------
//
// Bound by reading the weights once, so nothing stands between memory and the
// multiply: a CTA takes 16 output features, its NW warps every NW-th block of K
// each, and every lane loads its operands of mma.sync (m16n8k32, weights
// first) straight to registers, 16 bytes at a time. The instruction wants
// four codes of each of two places of K per thread; which four does not matter
// as long as both operands agree, so a lane takes 16 consecutive codes of a
// row and spends them on two instructions. The block's fp32 sums are scaled
// into the warp's accumulators, and the warps' sums meet in shared memory, in
// warp order. (The instruction's own sums are fp32: outputs of 1 to 8 rows at
// K = 3072 and 12288 are 1e-7 of the 64-bit result away, root mean square.)
// Several CTAs per SM keep enough bytes in flight, and there is no tensor
// memory, barrier or cluster to set up. One token through three 3072 x 3072
// linears, packed here too: 6.7 us = 4.2 TB/s against 8.8 us on tcgen05 with K
// split over clusters; from 9 rows on that one is faster (16 rows: 9.4 against
// 6.7 us).
//
// TX: the activations come as codes and scales (uint8_t), or as they are, up
// to PACK_ROWS rows; then every CTA packs them all into shared memory (the
// quantizer of fp8_pack.cu, so the same codes), which saves a launch.

constexpr int STREAM_FEATURES = 16;
constexpr int STREAM_ROWS = 8;                   // most rows
constexpr int PACK_ROWS = 4;                     // most rows packed inside
constexpr int64_t PACK_MAX_K = 12288;            // and their longest K
static_assert(PACK_ROWS * PACK_MAX_K + PACK_ROWS * (PACK_MAX_K / QBLOCK) * 4 <= 56 * 1024, "several CTAs per SM");

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

struct StreamParams {
  const void* X;                // codes [M,K], or activations
  const float* s_x;             // with codes
  int64_t ldx;
  const uint8_t* q[MAX_LIN];
  const float* s_w[MAX_LIN];
  const float* bias[MAX_LIN];
  void* out[MAX_LIN];
  int64_t ldy[MAX_LIN];
  int N[MAX_LIN];
  int tile_start[MAX_LIN + 1];
  int M, K, KB, n_lin;
  bool vec_x;
};

template <typename TX, typename TY, int NW>
__global__ void __launch_bounds__(NW * 32, 32 / NW)
fp8_stream_kernel(const __grid_constant__ StreamParams p) {
  constexpr bool PACK = sizeof(TX) > 1;
  extern __shared__ __align__(16) uint8_t sx[];  // PACK: codes [M][K rounded up to blocks], scales [M][KB]
  __shared__ float part[NW][STREAM_ROWS][STREAM_FEATURES + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  int lin = 0;
#pragma unroll 1
  while (lin + 1 < p.n_lin && static_cast<int>(blockIdx.x) >= p.tile_start[lin + 1]) ++lin;
  const int N = p.N[lin], n0 = (static_cast<int>(blockIdx.x) - p.tile_start[lin]) * STREAM_FEATURES;
  // this lane's two weight rows (past the last one: the last one again, not stored)
  const uint8_t* w0 = p.q[lin] + static_cast<int64_t>(min(n0 + g, N - 1)) * p.K;
  const uint8_t* w1 = p.q[lin] + static_cast<int64_t>(min(n0 + g + 8, N - 1)) * p.K;
  pdl_launch_dependents();
  // ask for the weights while the launch before this one ends (into L2 only:
  // what it may still write is seen)
  for (int k = (warp * 4 + t) * 128; k < p.K; k += NW * 4 * 128) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(w0 + k));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(w1 + k));
  }
  pdl_wait_prerequisites();

  // The weights of one block: [half of 64 codes][row]; zeros past K.
  auto load_w = [&](int kb, uint4 (&a)[2][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = kb * BK + h * 64 + t * 16;
      const bool on = k < p.K;
      a[h][0] = on ? ldg_stream(w0 + k) : make_uint4(0, 0, 0, 0);
      a[h][1] = on ? ldg_stream(w1 + k) : make_uint4(0, 0, 0, 0);
    }
  };
  uint4 a[2][2], next[2][2];
  if (warp < p.KB) load_w(warp, a);
  // PACK (whose K is short): the packed rows' length, and where their scales lie
  const int Kp = PACK ? p.KB * BK : 0;
  float* ssx = reinterpret_cast<float*>(sx + p.M * Kp);
  if constexpr (PACK) {
    // eight lanes per block of 128 features, 16 features per lane; a warp's
    // lanes all take the same turns
    const int sub = lane & 7, items = p.KB * p.M;
    for (int i0 = warp * 4; i0 < items; i0 += NW * 4) {
      const int i = i0 + (lane >> 3), kb = i / p.M, r = i - kb * p.M, col = kb * BK + sub * 16;
      Pair x[8];
      if (i < items && col < p.K) {
        load16(static_cast<const TX*>(p.X) + r * p.ldx + col, p.vec_x, x);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = 0ull;
      }
      float m = max_magnitude(x);
#pragma unroll
      for (int d = 1; d < 8; d *= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
      const float sc = e4m3_scale(m);
      uint32_t q[4];
      e4m3_codes(x, sc, e4m3_factor(sc), q);
      if (i < items) {
        *reinterpret_cast<uint4*>(sx + r * Kp + col) = make_uint4(q[0], q[1], q[2], q[3]);
        if (sub == 0) ssx[r * p.KB + kb] = sc;
      }
    }
    __syncthreads();
  }

  const float* ws = p.s_w[lin] + static_cast<int64_t>(n0 / QBLOCK) * p.KB;
  // the activation row that this lane holds, and the scales of the two whose
  // results it has (past the last row: the last one again, not stored)
  const int r = min(g, p.M - 1), r0 = min(2 * t, p.M - 1), r1 = min(2 * t + 1, p.M - 1);
  const uint8_t* xr = static_cast<const uint8_t*>(p.X) + static_cast<int64_t>(r) * p.K;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb = warp; kb < p.KB; kb += NW) {
    if (kb + NW < p.KB) load_w(kb + NW, next);
    uint4 b[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = kb * BK + h * 64 + t * 16;
      if (PACK) b[h] = *reinterpret_cast<const uint4*>(sx + r * Kp + k);
      else b[h] = k < p.K ? __ldg(reinterpret_cast<const uint4*>(xr + k)) : make_uint4(0, 0, 0, 0);
    }
    const float sw = __ldg(ws + kb);
    const float f0 = sw * (PACK ? ssx[r0 * p.KB + kb] : __ldg(p.s_x + static_cast<int64_t>(r0) * p.KB + kb));
    const float f1 = sw * (PACK ? ssx[r1 * p.KB + kb] : __ldg(p.s_x + static_cast<int64_t>(r1) * p.KB + kb));
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mma_sync_e4m3(d, a[h][0].x, a[h][1].x, a[h][0].y, a[h][1].y, b[h].x, b[h].y);
      mma_sync_e4m3(d, a[h][0].z, a[h][1].z, a[h][0].w, a[h][1].w, b[h].z, b[h].w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(d[i], i & 1 ? f1 : f0, acc[i]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      a[h][0] = next[h][0];
      a[h][1] = next[h][1];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[warp][2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[i];
  __syncthreads();
  const float* bias = p.bias[lin];
  for (int i = threadIdx.x; i < p.M * STREAM_FEATURES; i += NW * 32) {
    const int m = i / STREAM_FEATURES, n = i % STREAM_FEATURES;
    if (n0 + n >= N) continue;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) y += part[w][m][n];
    if (bias) y += __ldg(bias + n0 + n);
    static_cast<TY*>(p.out[lin])[m * p.ldy[lin] + n0 + n] = from_f32<TY>(y);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// e4m3 codes [rows,K] (dense), box box_rows x 128 codes, 128-byte swizzle.
int make_tmap_codes(CUtensorMap* m, const void* base, int64_t rows, int64_t K, int box_rows) {
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
int make_tmap_out(CUtensorMap* m, void* base, int y_dtype, int64_t rows, int64_t cols, int64_t ldy) {
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

// Raises the kernel's shared-memory limit, once per device. `regs`: the
// registers a thread that the kernel's own redistribution counts on (it would
// wait forever for more than the launch has).
template <typename F>
int allow_smem(F* kernel, int bytes, uint64_t& done, std::mutex& mu, int regs = 0) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return set_cuda_error(e);
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 64 || !((done >> dev) & 1u)) {
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e != cudaSuccess) return set_cuda_error(e);
    if (attr.numRegs < regs) return CONVROT_ERR_UNSUPPORTED;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return set_cuda_error(e);
    if (dev < 64) done |= 1ull << dev;
  }
  return CONVROT_OK;
}

constexpr int64_t RASTER_L2_BYTES = 48ll << 20;  // activation codes a raster group keeps in L2

// Everything of a launch but the tensor maps of Y: tiles of tile_rows
// activation rows x tile_cols features, operand boxes x_box and w_box rows.
int fill(GemmParams& p, const uint8_t* Qx, const float* s_x, int64_t M, int64_t K, const convrot_fp8_weight* w, int n,
         int tile_rows, int tile_cols, int x_box, int w_box, uint64_t test_wait_ns) {
  if (int st = make_tmap_codes(&p.tmap_x, Qx, M, K, x_box)) return st;
  int64_t cols = 0;
  const int64_t KB = n_blocks(K);
  p.vec_scales = KB % 4 == 0 && aligned16(s_x);
  for (int j = 0; j < n; ++j) {
    if (int st = make_tmap_codes(&p.tmap_w[j], w[j].q, w[j].N, K, w_box)) return st;
    p.s_w[j] = w[j].scale;
    p.bias[j] = w[j].bias;
    p.out[j] = w[j].Y;
    p.ldy[j] = w[j].ldy;
    p.N[j] = static_cast<int>(w[j].N);
    p.tile_start[j] = static_cast<int>(cols);
    cols += (w[j].N + tile_cols - 1) / tile_cols;
    p.vec_scales = p.vec_scales && aligned16(w[j].scale);
  }
  p.n_mtiles = static_cast<int>((M + tile_rows - 1) / tile_rows);
  if (cols * p.n_mtiles > 0x7fffffff / 8) return CONVROT_ERR_UNSUPPORTED;
  p.tile_start[n] = static_cast<int>(cols);
  p.total_tiles = static_cast<int>(cols * p.n_mtiles);
  p.raster_mtiles =
      static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(p.n_mtiles, RASTER_L2_BYTES / (tile_rows * K))));
  p.s_x = s_x;
  p.M = static_cast<int>(M);
  p.KB = static_cast<int>(KB);
  p.n_lin = n;
  p.split = 1;
  p.tma_y = false;
  p.wait_ns = test_wait_ns ? test_wait_ns : kWaitLimitNs;
  p.withheld_tile = test_wait_ns ? p.total_tiles - 1 : -1;
  return CONVROT_OK;
}

template <typename TY>
int launch_pair(const uint8_t* Qx, const float* s_x, int64_t M, int64_t K, const convrot_fp8_weight* w, int n,
                int y_dtype, uint64_t test_wait_ns, cudaStream_t stream) {
  using G = PairGeom;
  GemmParams p;
  if (int st = fill(p, Qx, s_x, M, K, w, n, 256, G::BN, LANES, G::BN / 2, test_wait_ns)) return st;
  p.tma_y = true;
  for (int j = 0; j < n; ++j) {
    const uint64_t pitch = static_cast<uint64_t>(w[j].ldy) * sizeof(TY);
    p.tma_y = p.tma_y && aligned16(w[j].Y) && pitch % 16 == 0 && pitch < (1ull << 40);
  }
  if (p.tma_y)
    for (int j = 0; j < n; ++j)
      if (int st = make_tmap_out(&p.tmap_y[j], w[j].Y, y_dtype, M, w[j].N, w[j].ldy)) return st;
  static std::mutex mu;
  static uint64_t done = 0;
  auto kernel = fp8_pair_kernel<TY>;
  if (int st = allow_smem(kernel, G::SMEM_ALLOC, done, mu, LAUNCH_REGS)) return st;
  const int pairs = std::min(p.total_tiles, device_sm_count() / 2);
  Launch l(2 * pairs, PAIR_THREADS, G::SMEM_ALLOC, stream, 2);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kernel, p);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

template <typename TY, int BN, bool SWAP>
int launch_solo(const uint8_t* Qx, const float* s_x, int64_t M, int64_t K, const convrot_fp8_weight* w, int n,
                int split, uint64_t test_wait_ns, cudaStream_t stream) {
  using G = SoloGeom<BN, SWAP>;
  GemmParams p;
  if (int st = fill(p, Qx, s_x, M, K, w, n, G::TILE_ROWS, QBLOCK, G::X_ROWS, G::W_ROWS, test_wait_ns)) return st;
  p.split = split;
  static std::mutex mu;
  static uint64_t done = 0;
  auto kernel = fp8_solo_kernel<TY, BN, SWAP>;
  if (int st = allow_smem(kernel, G::SMEM_ALLOC, done, mu)) return st;
  Launch l(p.total_tiles * split, SOLO_THREADS, G::SMEM_ALLOC, stream, split);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kernel, p);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

// CTAs per tile (a cluster of 1, 2, 4 or at most `most`): as many as keep all
// tiles within one wave of `slots` CTAs and leave every CTA a block of K.
// Clusters of six and eight measured slower than four on [24, 12288] x [3072,
// 12288] although they use more SMs: 19 and 17 us against 13 us.
int pick_split(int64_t tiles, int64_t KB, int64_t slots, int most) {
  int s = 1;
  while (s < most && tiles * (2 * s) <= slots && 2 * s <= KB) s *= 2;
  return s;
}

template <typename TX, typename TY, int NW>
int launch_stream_of(const StreamParams& p, size_t smem, cudaStream_t stream) {
  static std::mutex mu;
  static uint64_t done = 0;
  auto kernel = fp8_stream_kernel<TX, TY, NW>;
  if (int st = allow_smem(kernel, 64 * 1024, done, mu)) return st;
  Launch l(p.tile_start[p.n_lin], NW * 32, smem, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kernel, p);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

// Sixteen warps per CTA where the tiles alone would leave the SMs few, and K
// is long enough for them.
template <typename TX, typename TY>
int launch_stream_as(const StreamParams& p, size_t smem, cudaStream_t stream) {
  if (p.tile_start[p.n_lin] <= 2 * device_sm_count() && p.KB >= 16)
    return launch_stream_of<TX, TY, 16>(p, smem, stream);
  return launch_stream_of<TX, TY, 8>(p, smem, stream);
}

StreamParams stream_params(const void* X, const float* s_x, int64_t M, int64_t K, int64_t ldx,
                           const convrot_fp8_weight* w, int n) {
  StreamParams p{};
  p.X = X;
  p.s_x = s_x;
  p.ldx = ldx;
  p.M = static_cast<int>(M);
  p.K = static_cast<int>(K);
  p.KB = static_cast<int>(n_blocks(K));
  p.n_lin = n;
  for (int j = 0; j < n; ++j) {
    p.q[j] = w[j].q;
    p.s_w[j] = w[j].scale;
    p.bias[j] = w[j].bias;
    p.out[j] = w[j].Y;
    p.ldy[j] = w[j].ldy;
    p.N[j] = static_cast<int>(w[j].N);
    p.tile_start[j + 1] = p.tile_start[j] + static_cast<int>((w[j].N + STREAM_FEATURES - 1) / STREAM_FEATURES);
  }
  return p;
}

template <typename TX>
int launch_packing_stream(const void* X, int64_t M, int64_t K, int64_t ldx, const convrot_fp8_weight* w, int n,
                          int y_dtype, cudaStream_t stream) {
  StreamParams p = stream_params(X, nullptr, M, K, ldx, w, n);
  p.vec_x = aligned16(X) && (ldx * sizeof(TX)) % 16 == 0;
  const size_t smem = static_cast<size_t>(M) * p.KB * (BK + 4);
  if (y_dtype == CONVROT_F32) return launch_stream_as<TX, float>(p, smem, stream);
  if (y_dtype == CONVROT_F16) return launch_stream_as<TX, __half>(p, smem, stream);
  return launch_stream_as<TX, __nv_bfloat16>(p, smem, stream);
}

template <typename TY>
int launch_as(const uint8_t* Qx, const float* s_x, int64_t M, int64_t K, const convrot_fp8_weight* w, int n,
              int y_dtype, uint64_t test_wait_ns, cudaStream_t stream) {
  const int sms = device_sm_count();
  const int64_t KB = n_blocks(K);
  int64_t cols = 0;  // tiles of 128 features
  for (int j = 0; j < n; ++j) cols += n_blocks(w[j].N);
  if (M <= STREAM_ROWS) {
    if (test_wait_ns) return CONVROT_ERR_UNSUPPORTED;  // a kernel without waits
    return launch_stream_as<uint8_t, TY>(stream_params(Qx, s_x, M, K, K, w, n), 0, stream);
  }
  if (M <= 64) {
    const int split = pick_split(cols, KB, 2 * sms, 4);
    if (M <= 16) return launch_solo<TY, 16, true>(Qx, s_x, M, K, w, n, split, test_wait_ns, stream);
    if (M <= 32) return launch_solo<TY, 32, true>(Qx, s_x, M, K, w, n, split, test_wait_ns, stream);
    return launch_solo<TY, 64, true>(Qx, s_x, M, K, w, n, split, test_wait_ns, stream);
  }
  const int64_t solo = (M + 127) / 128 * cols;
  // Whole waves of single-CTA tiles while one wave holds them all: measured at
  // 65 to 2304 rows on five weight shapes, within 2 % of the faster of the two
  // kernels everywhere (1024 rows, 3072 x 3072: 26 us here, 16 us in pairs;
  // 700 rows: 12.6 us here, 15.2 us in pairs).
  if (solo <= sms)
    return launch_solo<TY, 128, false>(Qx, s_x, M, K, w, n, pick_split(solo, KB, sms, 4), test_wait_ns, stream);
  return launch_pair<TY>(Qx, s_x, M, K, w, n, y_dtype, test_wait_ns, stream);
}

}  // namespace

int launch_fp8_gemm(const uint8_t* Qx, const float* s_x, int64_t M, int64_t K, const convrot_fp8_weight* weights,
                    int n_weights, int y_dtype, cudaStream_t stream, uint64_t test_wait_ns) {
  if (y_dtype == CONVROT_F32) return launch_as<float>(Qx, s_x, M, K, weights, n_weights, y_dtype, test_wait_ns, stream);
  if (y_dtype == CONVROT_F16) return launch_as<__half>(Qx, s_x, M, K, weights, n_weights, y_dtype, test_wait_ns, stream);
  return launch_as<__nv_bfloat16>(Qx, s_x, M, K, weights, n_weights, y_dtype, test_wait_ns, stream);
}

int launch_fp8_packing(const void* X, int x_dtype, int64_t M, int64_t K, int64_t ldx, const convrot_fp8_weight* weights,
                       int n_weights, int y_dtype, cudaStream_t stream, bool* launched) {
  *launched = M <= PACK_ROWS && K <= PACK_MAX_K;
  if (!*launched) return CONVROT_OK;
  if (x_dtype == CONVROT_F32) return launch_packing_stream<float>(X, M, K, ldx, weights, n_weights, y_dtype, stream);
  if (x_dtype == CONVROT_F16) return launch_packing_stream<__half>(X, M, K, ldx, weights, n_weights, y_dtype, stream);
  return launch_packing_stream<__nv_bfloat16>(X, M, K, ldx, weights, n_weights, y_dtype, stream);
}

cudaError_t linear_error_word(int** p) { return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_fp8_error); }

}  // namespace fp8
}  // namespace convrot
