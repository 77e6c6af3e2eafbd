// expert_pair.cu -- the experts' linears with many rows per expert: CTA pairs,
// activation rows on the TMEM lanes.
//
// As the many-row kernel of the dense linears (fp8_gemm.cu): persistent
// clusters of two CTAs; a tile is 256 rows of one expert x 256 rows of its
// weights, M = 256 MMAs of the even CTA, one TMEM accumulator per block of K,
// promoted with the block's scales into fp32 registers that stay for the tile.
// What differs: which tiles there are is known on the device alone (every CTA
// sums the experts' row tiles up when it starts); a tile's last rows may be the
// next expert's, and are not stored; and with SwiGLU a tile's weight rows are 128
// of the gate and the same 128 of the up matrix, dealt out in runs of 64 so
// that every epilogue thread has gate and up of the same 64 features of its
// row. It forms h there; the two threads of a row exchange their maxima through
// shared memory, and codes and scale leave from registers.
//
// 8192 rows of eight experts, 4096 -> 2 x 2432: 148 us = 2.2 PFLOP/s; a linear of
// as many products 139 us, the dense kernel 129 us. A tile costs 0.47 us for each
// block of K (operand delivery and the accumulator's hand-over, as there), and 2
// to 3 us for the epilogue beyond the two blocks that the MMAs run ahead (SwiGLU:
// 64 exponentials and as many reciprocals a thread among it). Experts of 512
// uneven rows leave a fifth of the tiles' rows empty.
#include "expert_common.cuh"

#include <algorithm>

namespace convrot {
namespace moe {

// Sticky device error word of this kernel (timeouts of bounded waits).
__device__ int g_pair_error = 0;

namespace {

constexpr int EPI_WARPS = 8;
constexpr int PAIR_THREADS = (EPI_WARPS + 4) * 32;  // three warpgroups
constexpr int LAUNCH_REGS = 168, CONTROL_REGS = 56, EPI_REGS = 224;
static_assert(2 * EPI_REGS + CONTROL_REGS <= 3 * LAUNCH_REGS, "within what the block was launched with");
constexpr int STORE_BLOCK = 32 * STORE_ROW;  // one store: 32 rows
constexpr int STORE_BYTES = 2 * STORE_BLOCK;  // one warp's two store buffers
constexpr int ROWS = 256;                     // of a tile

struct PairParams {
  CUtensorMap tmap_x;     // codes [n,K] in the plan's order
  CUtensorMap tmap_w[2];  // codes [E][N,K]: the matrix, or gate and up
  CUtensorMap tmap_y;     // Y [n,N], where tma_y
  Rows rows;
  convrot_experts w[2];
  const float* s_x;  // [n,KB]
  void* out;         // Y, or the codes of h
  float* s_out;      // their scales
  int64_t ldy;
  int N, KB, n_cols;
  bool tma_y, vec_scales;
  uint64_t wait_ns;
  bool withhold;  // test of the timeout: the last block of K of the last tile is not loaded
};

// What the epilogue needs to know of a tile, prepared by a warp of its own.
struct __align__(16) TileInfo {
  int row, end;         // this CTA's first row, and the end of the expert's
  int col, pad;         // the tile's first feature
  const float* ws[2];   // the weight scales of the tile's two blocks of weight rows
};
static_assert(sizeof(TileInfo) == 32, "as laid out in shared memory");

struct Geom {
  static constexpr int BN = 256;  // weight rows of a tile
  static constexpr int X_BYTES = LANES * BK;
  static constexpr int W_BYTES = BN / 2 * BK;
  static constexpr int STAGE_BYTES = X_BYTES + W_BYTES;
  static constexpr int STAGES = 5;
  static constexpr int BUFS = 512 / BN;
  static constexpr uint32_t IDESC = idesc_e4m3_f32(256, BN);
  static constexpr int SMEM_OUT = STAGES * STAGE_BYTES;
  // the stores' buffers; with SwiGLU the rows' maxima [2 tiles][2 halves][LANES]
  static constexpr int SMEM_BIAS = SMEM_OUT + (EPI_WARPS * STORE_BYTES);  // [BN] fp32
  static constexpr int SMEM_INFO = SMEM_BIAS + BN * 4;
  static constexpr int SMEM_BARS = SMEM_INFO + 2 * 32;
  static constexpr int SMEM_FIRST = SMEM_BARS + (2 * STAGES + 2 * BUFS + 11) * 8 + 16;  // [groups of experts + 1]
  static constexpr int SMEM_ALLOC = SMEM_FIRST + (MAX_EXPERTS / GROUP + 1) * 4 + 1024;
};
static_assert(Geom::SMEM_ALLOC <= 227 * 1024, "shared memory");

// Adds f0 times the first half and f1 times the second half of the accumulator
// at `ta` (128 columns of the warp's lanes) to acc.
__device__ __forceinline__ void drain2(unsigned long long (&acc)[64], uint32_t ta, float f0, float f1) {
  uint32_t r[2][16];
  tmem_ld16(ta, r[0]);
  const unsigned long long a = f32x2_pack(f0, f0), b = f32x2_pack(f1, f1);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    tmem_wait16(r[q & 1]);
    if (q + 1 < 8) tmem_ld16(ta + (q + 1) * 16, r[(q + 1) & 1]);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      acc[q * 8 + k] = f32x2_fma(pair_bits(r[q & 1][2 * k], r[q & 1][2 * k + 1]), q < 4 ? a : b, acc[q * 8 + k]);
  }
}

// The first `rows` rows of a staged block, 16 bytes per lane: rows of Y start on
// 16-byte boundaries.
template <typename TS>
static __device__ __noinline__ void store_part(const uint8_t* sb, TS* y, int64_t ldy, int rows, int cols) {
  const int lane = threadIdx.x & 31, ch = lane & 7;
  constexpr int E = 16 / sizeof(TS);
#pragma unroll 1
  for (int r = lane >> 3; r < min(rows, 32); r += 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(sb + r * STORE_ROW + (swizzled(ch, r) << 4));
    TS* to = y + r * ldy + ch * E;
    if ((ch + 1) * E <= cols) {
      *reinterpret_cast<uint4*>(to) = v;
    } else {
      const TS* from = reinterpret_cast<const TS*>(&v);
      for (int k = 0; ch * E + k < cols; ++k) to[k] = from[k];
    }
  }
}

template <typename TY, bool SWIGLU>
__global__ void __launch_bounds__(PAIR_THREADS, 1) expert_pair_kernel(const __grid_constant__ PairParams p) {
  using G = Geom;
  constexpr int BN = G::BN;
  constexpr int COLS = BN / 2;                     // accumulator columns per epilogue thread
  constexpr int FEATURES = SWIGLU ? BN / 2 : BN;  // of a tile
  constexpr bool EARLY = SWIGLU || SCALED<TY>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::SMEM_BARS);
  uint64_t* empty = full + G::STAGES;
  uint64_t* tfull = empty + G::STAGES;
  uint64_t* tempty = tfull + G::BUFS;
  uint64_t* done = tempty + G::BUFS;
  uint64_t* ifull = done + 1;    // [2] a tile's info is in shared memory
  uint64_t* iempty = ifull + 2;  // [2] and has been read
  uint64_t* bfull = iempty + 2;  // the same for its bias
  uint64_t* bempty = bfull + 1;
  uint64_t* xbar = bempty + 1;   // [4] both halves' maxima of a quarter's rows
  TileInfo* info = reinterpret_cast<TileInfo*>(smem + G::SMEM_INFO);
  float* sbias = reinterpret_cast<float*>(smem + G::SMEM_BIAS);
  int* first = reinterpret_cast<int*>(smem + G::SMEM_FIRST);
  uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(xbar + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_smem + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int unit = static_cast<int>(cluster_id_x()), n_units = static_cast<int>(cluster_count_x());
  int* err = &g_pair_error;

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
    for (int q = 0; q < 4; ++q) mbar_init(&xbar[q], 2);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&p.tmap_x);
    tma_prefetch_desc(&p.tmap_w[0]);
    if (SWIGLU) tma_prefetch_desc(&p.tmap_w[1]);
  }
  if (warp == EPI_WARPS + 1) {
    tmem_alloc_pair(tmem_base_smem, 512);
    tmem_relinquish_pair();
  }
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  if (warp == EPI_WARPS + 3) count_tiles_grouped(p.rows, ROWS, first);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_base_smem;
  const int total = first[(p.rows.E + GROUP - 1) / GROUP] * p.n_cols;

  if (warp >= EPI_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CONTROL_REGS));
    if (warp == EPI_WARPS) {
      const uint64_t pol = l2_policy_evict_normal();
      const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
      uint32_t stage = 0, phase = 0, n_issued = 0;
      bool ok = true;
      for (int t = unit; ok && t < total; t += n_units) {
        int2 range;
        const Item c = find_item_grouped(p.rows, ROWS, first, p.n_cols, t, range);
        const int row = range.x + c.tile * ROWS + static_cast<int>(rank) * LANES;
        for (int kb = 0; kb < p.KB; ++kb) {
          if (p.withhold && t == total - 1 && kb == p.KB - 1) break;
          ok = warp_wait(&empty[stage], phase ^ 1u, abort_flag, err, p.wait_ns);
          if (!ok) break;
          uint8_t* sx = smem + stage * G::STAGE_BYTES;
          uint8_t* sw = sx + G::X_BYTES;
          const uint32_t fb = full_leader + stage * 8u;
          if (lane == 0) {
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * G::STAGE_BYTES);
            if (SWIGLU) {
              const int f = c.col * FEATURES + static_cast<int>(rank) * 64;
              tma_load_3d_pair(sw, &p.tmap_w[0], fb, kb * BK, f, c.expert, pol);
              tma_load_3d_pair(sw + 64 * BK, &p.tmap_w[1], fb, kb * BK, f, c.expert, pol);
            } else {
              tma_load_3d_pair(sw, &p.tmap_w[0], fb, kb * BK, c.col * FEATURES + static_cast<int>(rank) * LANES, c.expert, pol);
            }
            tma_load_2d_pair(sx, &p.tmap_x, fb, kb * BK, row, pol);
          }
          __syncwarp();
          ++n_issued;
          if (++stage == G::STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // No copy may land after the CTAs exit: see fp8_pair_kernel.
      if (rank == 1 && !ok && lane == 0)
        for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < 1000000;) __nanosleep(10000);
      if (rank == 0 && lane == 0)
        for (uint32_t s = 0; s < G::STAGES; ++s)
          if (n_issued > s) mbar_wait(&full[s], ((n_issued - 1 - s) / G::STAGES) & 1u, nullptr, err, p.wait_ns);
    }
    if (warp == EPI_WARPS + 1 && lane == 0 && rank == 0) {
      uint32_t stage = 0, phase = 0, buf = 0, bphase = 0;
      bool ok = true;
      for (int t = unit; ok && t < total; t += n_units) {
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
      for (int t = unit; t < total; t += n_units, ++i) {
        int2 range;
        const Item c = find_item_grouped(p.rows, ROWS, first, p.n_cols, t, range);
        const int n0 = c.col * FEATURES;
        // the bias in the order of the accumulator's columns
        float v[BN / 32];
#pragma unroll
        for (int k = 0; k < BN / 32; ++k) {
          const int j = SWIGLU ? (k >> 1) & 1 : 0;
          const int n = n0 + (SWIGLU ? 64 * (k >> 2) + 32 * (k & 1) : 32 * k) + lane;
          v[k] = p.w[j].bias && n < p.N ? __ldg(p.w[j].bias + c.expert * p.w[j].bias_stride + n) : 0.0f;
        }
        if (!wait_slowly(&iempty[i & 1], ((i >> 1) & 1) ^ 1u, abort_flag, err, p.wait_ns)) break;
        if (lane == 0) {
          TileInfo ti;
          ti.row = range.x + c.tile * ROWS + static_cast<int>(rank) * LANES;
          ti.end = range.y;
          ti.col = n0;
          ti.pad = 0;
          const int64_t block = static_cast<int64_t>(n0 / QBLOCK) * p.KB;
          ti.ws[0] = p.w[0].scale + c.expert * p.w[0].scale_stride + block;
          // past the features the first block's again; nothing of it is stored
          ti.ws[1] = SWIGLU ? p.w[1].scale + c.expert * p.w[1].scale_stride + block
                            : ti.ws[0] + (n0 + QBLOCK < p.N ? p.KB : 0);
          info[i & 1] = ti;
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
    TileInfo c{};
    const float *xs = nullptr, *ws0 = nullptr, *ws1 = nullptr;
    float nx[4], nw0[4], nw1[4];
    auto load_weight_scales = [&](int kb) {
      load_scales(ws0, kb, p.KB, p.vec_scales, nw0);
      if (SWIGLU) load_scales(ws1, kb, p.KB, p.vec_scales, nw1);
    };
    auto start = [&](int i) {  // the CTA's tile i
      if (!warp_wait(&ifull[i & 1], (i >> 1) & 1u, abort_flag, err, p.wait_ns)) return false;
      c = info[i & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&iempty[i & 1]);
      c.row += 32 * quarter;  // the warp's first row
      // rows past the expert's last read the last one's scales; their outputs
      // are not stored
      xs = p.s_x + static_cast<int64_t>(min(c.row + lane, c.end - 1)) * p.KB;
      ws0 = SWIGLU || half == 0 ? c.ws[0] : c.ws[1];
      ws1 = c.ws[1];
      load_scales(xs, 0, p.KB, p.vec_scales, nx);
      load_weight_scales(0);
      return true;
    };
    int seq = 0;
    if (unit < total) ok = start(0);
    for (int t = unit; ok && t < total; t += n_units, ++seq) {
      const int row = c.row, end = c.end, col = c.col;
      unsigned long long acc[COLS / 2];
#pragma unroll
      for (int i = 0; i < COLS / 2; ++i) acc[i] = 0ull;
      float f[4], h[4];
#pragma unroll 1
      for (int kb = 0; kb < p.KB; ++kb) {
        if ((kb & 3) == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[i] = nx[i] * nw0[i];
            if (SWIGLU) h[i] = nx[i] * nw1[i];
          }
          if (kb + 4 < p.KB) {
            load_scales(xs, kb + 4, p.KB, p.vec_scales, nx);
            load_weight_scales(kb + 4);
          }
        }
        // the next tile's info and first scales, while the last block's MMAs run
        // (in the linears that store their sums as they are, the loop would
        // spill more registers for it than the epilogue does now, 32 bytes and
        // 84 in fp32: 54 us instead of 49 us for eight-block tiles)
        if (EARLY && kb == p.KB - 1 && t + n_units < total && !start(seq + 1)) { ok = false; break; }
        if (!warp_wait(&tfull[buf], bphase, abort_flag, err, p.wait_ns)) { ok = false; break; }
        tc_fence_after();
        if (SWIGLU) drain2(acc, t_addr + buf * BN, f[0], h[0]);
        else drain<COLS>(acc, t_addr + buf * BN, f32x2_pack(f[0], f[0]));
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          f[i] = f[i + 1];
          if (SWIGLU) h[i] = h[i + 1];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty_leader + buf * 8u);
        if (++buf == G::BUFS) { buf = 0; bphase ^= 1u; }
      }
      if (!ok) break;
      if (!EARLY && t + n_units < total) ok = start(seq + 1);
      if (!warp_wait(bfull, seq & 1u, abort_flag, err, p.wait_ns)) break;
      const float* bias = sbias + half * COLS;
      if constexpr (SWIGLU) {
        // h in place of the gate's sums
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < COLS / 4; ++k) {
          float g0, g1, u0, u1;
          f32x2_unpack(acc[k], g0, g1);
          f32x2_unpack(acc[COLS / 4 + k], u0, u1);
          const float2 bg = *reinterpret_cast<const float2*>(bias + 2 * k);
          const float2 bu = *reinterpret_cast<const float2*>(bias + COLS / 2 + 2 * k);
          g0 = silu_mul(g0 + bg.x, u0 + bu.x);
          g1 = silu_mul(g1 + bg.y, u1 + bu.y);
          asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(top) : "f"(top), "f"(g0), "f"(g1));
          acc[k] = f32x2_pack(g0, g1);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bempty);
        // the other 64 features' maximum, through shared memory; the buffers
        // alternate, so that one hand-over per tile is enough
        float* top_of = reinterpret_cast<float*>(smem + G::SMEM_OUT) + (seq & 1) * 2 * LANES + 32 * quarter + lane;
        top_of[half * LANES] = top;
        __syncwarp();
        if (lane == 0) mbar_arrive(&xbar[quarter]);
        if (!warp_wait(&xbar[quarter], seq & 1u, abort_flag, err, p.wait_ns)) break;
        top = max_nan(top, top_of[(half ^ 1) * LANES]);
        const float sc = e4m3_scale(top);
        uint32_t q[COLS / 8];
        const unsigned long long(&x)[COLS / 4] = reinterpret_cast<const unsigned long long(&)[COLS / 4]>(acc);
        e4m3_codes(x, sc, e4m3_factor(sc), q);
        const int i = row + lane, n = col + half * 64;
        if (i < end) {
          uint8_t* out = static_cast<uint8_t*>(p.out) + i * p.ldy + n;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (n + 16 * k < p.N)
              *reinterpret_cast<uint4*>(out + 16 * k) = make_uint4(q[4 * k], q[4 * k + 1], q[4 * k + 2], q[4 * k + 3]);
          if (half == 0) p.s_out[static_cast<int64_t>(i) * ((p.N + QBLOCK - 1) / QBLOCK) + col / QBLOCK] = sc;
        }
      } else {
        using TS = Stored<TY>;
        const unsigned long long* add = reinterpret_cast<const unsigned long long*>(bias);
#pragma unroll
        for (int k = 0; k < COLS / 2; k += 2) {
          const ulonglong2 bb = *reinterpret_cast<const ulonglong2*>(add + k);
          acc[k] = f32x2_add(acc[k], bb.x);
          acc[k + 1] = f32x2_add(acc[k + 1], bb.y);
        }
        if constexpr (SCALED<TY>) {
          // a thread's columns are the 128 features of one power
          float top = 0.0f;
#pragma unroll
          for (int k = 0; k < COLS / 2; ++k) {
            float a, b;
            f32x2_unpack(acc[k], a, b);
            top = fmaxf(top, fmaxf(finite_magnitude(a), finite_magnitude(b)));
          }
          const float power = power_of(top), inv = __frcp_rn(power);
          const unsigned long long inv2 = f32x2_pack(inv, inv);
#pragma unroll
          for (int k = 0; k < COLS / 2; ++k) acc[k] = f32x2_mul(acc[k], inv2);
          const int n = col + half * COLS;
          if (row + lane < end && n < p.N)
            p.s_out[static_cast<int64_t>(row + lane) * ((p.N + QBLOCK - 1) / QBLOCK) + n / QBLOCK] = power;
        }
        // store: PER features of a row at a time
        constexpr int PER = STORE_ROW / sizeof(TS);
        constexpr int E = 16 / sizeof(TS);  // of them in 16 bytes
        static_assert((COLS / PER) % 2 == 0, "both store buffers equally often");
        const bool whole = p.tma_y && row + 32 <= end;  // else the next expert's rows are in the block
#pragma unroll
        for (int b = 0; b < COLS / PER; ++b) {
          uint8_t* sb = sout + (b & 1) * STORE_BLOCK;
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
#pragma unroll
          for (int ch = 0; ch < PER / E; ++ch) {
            float v[E];
#pragma unroll
            for (int k = 0; k < E; k += 2) f32x2_unpack(acc[(b * PER + ch * E + k) / 2], v[k], v[k + 1]);
            *reinterpret_cast<uint4*>(sb + lane * STORE_ROW + (swizzled(ch, lane) << 4)) = pack16<TS>(v);
          }
          const int n = col + half * COLS + b * PER;
          if (whole) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (n < p.N) tma_store_2d(&p.tmap_y, sb, n, row);
              bulk_commit();
            }
          } else {
            __syncwarp();
            TS* y = static_cast<TS*>(p.out) + row * p.ldy + n;
            if (p.tma_y) store_part<TS>(sb, y, p.ldy, end - row, p.N - n);
            else store_rows<TS>(sb, y, p.ldy, min(32, end - row), p.N - n);
            // (an empty group, so that the next store into this buffer waits
            // for the right one)
            if (lane == 0) bulk_commit();
            __syncwarp();
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bempty);
      }
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

template <typename TY, bool SWIGLU>
int launch_as(const ExpertCall& c, cudaStream_t stream) {
  using G = Geom;
  const int64_t N = c.w->N, KB = n_blocks(c.K);
  PairParams p;
  if (int st = make_tmap_codes(&p.tmap_x, c.Q, c.rows.n, c.K, LANES)) return st;
  for (int j = 0; j < (SWIGLU ? 2 : 1); ++j) {
    p.w[j] = j ? *c.up : *c.w;
    if (int st = make_tmap_experts(&p.tmap_w[j], p.w[j], c.rows.E, c.K, SWIGLU ? 64 : LANES)) return st;
  }
  p.rows = c.rows;
  p.s_x = c.s;
  p.out = c.out;
  p.s_out = c.s_out;
  p.ldy = c.ldy;
  p.N = static_cast<int>(N);
  p.KB = static_cast<int>(KB);
  const int64_t cols = (N + (SWIGLU ? G::BN / 2 : G::BN) - 1) / (SWIGLU ? G::BN / 2 : G::BN);
  const int64_t tiles = c.rows.n / ROWS + std::min<int64_t>(c.rows.E, c.rows.n);  // of rows, at most
  if (cols * tiles > 0x7fffffff / 8) return CONVROT_ERR_UNSUPPORTED;
  p.n_cols = static_cast<int>(cols);
  p.vec_scales = KB % 4 == 0 && aligned16(c.s);
  for (int j = 0; j < (SWIGLU ? 2 : 1); ++j)
    p.vec_scales = p.vec_scales && aligned16(p.w[j].scale) && p.w[j].scale_stride % 4 == 0;
  const uint64_t pitch = static_cast<uint64_t>(c.ldy) * sizeof(Stored<TY>);
  p.tma_y = !SWIGLU && aligned16(c.out) && pitch % 16 == 0 && pitch < (1ull << 40);
  if (p.tma_y)
    if (int st = make_tmap_out(&p.tmap_y, c.out, c.y_dtype, c.rows.n, N, c.ldy)) return st;
  p.wait_ns = c.test_wait_ns ? c.test_wait_ns : kWaitLimitNs;
  p.withhold = c.test_wait_ns != 0;
  static std::mutex mu;
  static uint64_t done = 0;
  auto kernel = expert_pair_kernel<TY, SWIGLU>;
  if (int st = allow_smem(kernel, G::SMEM_ALLOC, done, mu, LAUNCH_REGS)) return st;
  const int64_t pairs = std::min<int64_t>(cols * tiles, device_sm_count() / 2);
  Launch l(static_cast<unsigned>(2 * pairs), PAIR_THREADS, G::SMEM_ALLOC, stream, 2);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kernel, p);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

}  // namespace

int launch_expert_pair(const ExpertCall& c, cudaStream_t stream) {
  if (c.up) return launch_as<uint8_t, true>(c, stream);
  if (c.s_out) return launch_as<ScaledHalf, false>(c, stream);
  if (c.y_dtype == CONVROT_F32) return launch_as<float, false>(c, stream);
  if (c.y_dtype == CONVROT_F16) return launch_as<__half, false>(c, stream);
  return launch_as<__nv_bfloat16, false>(c, stream);
}

cudaError_t pair_error_word(int** p) { return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_pair_error); }

}  // namespace moe
}  // namespace convrot
