// expert_few.cu -- the experts' linears with few rows per expert: weights on
// the TMEM lanes, activation rows as columns.
//
// Bound by reading the weights of the experts that have rows, once. Persistent
// CTAs; a work item is up to BN rows of one expert x 256 of its weight rows
// (SwiGLU: 128 of the gate and the same 128 of the up matrix, a scale's whole
// block). The loads run ahead over the items' borders, so that a CTA streams
// weights all the time. Where there are few items the CTAs of a cluster take
// shares of K and add their partial tiles up through distributed shared memory,
// in rank order.
//
// 256 rows over 128 experts, 2048 -> 2 x 768: 50 us for the 83 experts that are
// reached, 261 MB = 5.2 TB/s; 144 items of 256 weight rows of 4096, one for each
// CTA, 30 us = 5.0 TB/s. A CTA streams a block of K (34 KB) in 0.45 us at best:
// its eight MMAs take 0.32 us (75 cycles each, whatever their width), and issuing
// the copies about as long; so the last round of items counts, and 5 us for
// setting up, the first loads and the last sums.
//
// The MMAs' width is the item's rows, rounded up to 16, so that a tile that an
// expert does not fill costs no more than its rows.
//
// Twelve warps: 0-3 promote the first matrix' accumulators (32 lanes each), 4-7
// the second's, 8 loads weights and 10 activation rows (in the plan's order, or
// gathered by the plan, four to a copy), 9 issues MMAs, 11 only completes the
// warpgroup. The promoted sums meet in shared
// memory as [row][weight row], 32 rows at a time, where a warp takes a row: a
// lane has four features, and the largest magnitude of 128 is a warp's.
#include "expert_common.cuh"

#include <algorithm>
#include <cmath>

namespace convrot {
namespace moe {

// Sticky device error word of this kernel (timeouts of bounded waits).
__device__ int g_few_error = 0;

namespace {

constexpr int EPI_WARPS = 8;
constexpr int FEW_THREADS = (EPI_WARPS + 4) * 32;  // three warpgroups
// The control warpgroup gives up registers for the epilogue's accumulators.
constexpr int LAUNCH_REGS = 168, CONTROL_REGS = 56, EPI_REGS = 224;
static_assert(2 * EPI_REGS + CONTROL_REGS <= 3 * LAUNCH_REGS, "within what the block was launched with");
constexpr int MAX_SPLIT = 4;
constexpr int W_ROWS = 2 * QBLOCK;  // weight rows of an item

struct FewParams {
  CUtensorMap tmap_x;     // codes [T,K], box one row (gathered) or 16 rows
  CUtensorMap tmap_w[2];  // codes [E][N,K]: the matrix, or gate and up; box 128 rows
  Rows rows;
  convrot_experts w[2];
  const float* s_x;  // [T,KB]
  void* out;         // Y, or the codes of h
  float* s_out;      // their scales
  int64_t ldy;
  int N, KB, n_cols, split;
  bool vec_scales;
  uint64_t wait_ns;
  bool withhold;  // test of the timeout: the last block of K of the last item is not loaded
};

template <int BN>
struct FewGeom {
  static constexpr int W_BYTES = QBLOCK * BK;  // of one matrix
  static constexpr int X_BYTES = BN * BK;
  static constexpr int STAGE_BYTES = 2 * W_BYTES + X_BYTES;
  static constexpr int STAGES = BN == 64 ? 4 : 5;
  static constexpr int KG = 64 / BN;  // blocks of K handed over together
  static constexpr int BUF_COLS = 2 * KG * BN;
  static constexpr int TMEM_COLS = 512;
  static constexpr int BUFS = TMEM_COLS / BUF_COLS;
  static constexpr int PART_ROWS = BN < 32 ? BN : 32;
  static constexpr int SMEM_PART = STAGES * STAGE_BYTES;                  // [PART_ROWS][W_ROWS] fp32
  static constexpr int SMEM_SCALES = SMEM_PART + PART_ROWS * W_ROWS * 4;  // [warp][2][4 blocks][BN] fp32
  static constexpr int SMEM_BARS = SMEM_SCALES + EPI_WARPS * 2 * 4 * BN * 4;
  static constexpr int SMEM_WIDTH = SMEM_BARS + (2 * STAGES + 2 * BUFS + 3) * 8 + 16;  // [STAGES] columns of a stage
  static constexpr int SMEM_FIRST = SMEM_WIDTH + STAGES * 4;                           // [E + 1]
  static constexpr int smem(int E) { return SMEM_FIRST + (E + 1) * 4 + 1024; }
  static_assert(smem(MAX_EXPERTS) <= 227 * 1024, "shared memory");
  static_assert(BN % 16 == 0 && 64 % BN == 0, "columns");
};

// Adds n <= KG accumulators of `width` <= BN columns (2 * BN apart), each with a
// factor per column at f + its index * BN, to acc; 16 columns at a time, the
// next ones on their way.
template <int BN, int KG>
__device__ __forceinline__ void drain_columns(unsigned long long (&acc)[BN / 2], uint32_t ta, const float* f, int n, int width) {
  constexpr int PER = BN / 16;
  uint32_t r[2][16];
  tmem_ld16(ta, r[0]);
#pragma unroll
  for (int i = 0; i < KG * PER; ++i) {
    const int g = i / PER, q = i % PER;
    if (g < n && (KG > 1 || 16 * q < width)) {
      tmem_wait16(r[i & 1]);
      const int h = (i + 1) / PER, p = (i + 1) % PER;
      if (i + 1 < KG * PER) tmem_ld16(ta + h * 2 * BN + p * 16, r[(i + 1) & 1]);
      const uint32_t(&v)[16] = r[i & 1];
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float4 s = *reinterpret_cast<const float4*>(f + g * BN + q * 16 + 2 * k);
        acc[q * 8 + k] = f32x2_fma(pair_bits(v[2 * k], v[2 * k + 1]), f32x2_pack(s.x, s.y), acc[q * 8 + k]);
        acc[q * 8 + k + 1] =
            f32x2_fma(pair_bits(v[2 * k + 2], v[2 * k + 3]), f32x2_pack(s.z, s.w), acc[q * 8 + k + 1]);
      }
    }
  }
  tmem_ld_wait();  // a load past the width may still be on its way
}

// Where an item's walk over the blocks of K starts: not at the first one for
// all. Rows of K = 4096 codes lie 4 KB apart, and CTAs that read the same block
// of their rows at the same time meet in a few of the memory's channels: 144
// items, one per CTA, were read at 3.7 TB/s. By the matrix' place and the CTA's
// blocks alone, not by where the arrays lie in memory: in fours (the scales'
// wide loads) wherever the blocks are, also for scales that are loaded singly.
__device__ __forceinline__ int first_block(int expert, int col, int n_cols, int blocks, bool fours) {
  const int at = expert * n_cols + col;
  return fours ? at % (blocks / 4) * 4 : at * 5 % blocks;
}

// warp_wait for what the CTAs of a cluster (or this CTA's warps alone) have
// handed over: what they wrote before is seen.
__device__ __forceinline__ bool cluster_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err,
                                             uint64_t limit_ns, int ctas) {
  const bool ok = warp_wait(bar, parity, abort_flag, err, limit_ns);
  if (ctas > 1) asm volatile("fence.acq_rel.cluster;" ::: "memory");
  return ok;
}

template <int BN, bool SWIGLU, typename TY>
__global__ void __launch_bounds__(FEW_THREADS, 1) expert_few_kernel(const __grid_constant__ FewParams p) {
  using G = FewGeom<BN>;
  constexpr int FEATURES = SWIGLU ? QBLOCK : W_ROWS;  // of an item
  extern __shared__ uint8_t smem_raw[];
  // the offset to the next 1024-byte boundary is the same in every CTA of a cluster
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::SMEM_BARS);
  uint64_t* empty = full + G::STAGES;
  uint64_t* tfull = empty + G::STAGES;
  uint64_t* tempty = tfull + G::BUFS;
  uint64_t* done = tempty + G::BUFS;
  uint64_t* pfull = done + 1;    // all CTAs' partial tiles are in shared memory
  uint64_t* pempty = pfull + 1;  // and have been read
  uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(pempty + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_smem + 1);
  volatile int* stage_width = reinterpret_cast<volatile int*>(smem + G::SMEM_WIDTH);
  int* first = reinterpret_cast<int*>(smem + G::SMEM_FIRST);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* err = &g_few_error;
  const int split = p.split, rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = static_cast<int>(blockIdx.x) / split, n_units = static_cast<int>(gridDim.x) / split;
  const int kb_begin = p.KB * rank / split, kb_end = p.KB * (rank + 1) / split;  // this CTA's blocks of K
  const int blocks = kb_end - kb_begin;
  const bool fours = p.KB % 4 == 0 && kb_begin % 4 == 0 && blocks % 4 == 0;
  const bool vec = p.vec_scales && fours;  // their scales are loaded together

  if (threadIdx.x == EPI_WARPS * 32) {
    for (int s = 0; s < G::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < G::BUFS; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], EPI_WARPS);
    }
    mbar_init(done, 1);
    mbar_init(pfull, EPI_WARPS * split);
    mbar_init(pempty, EPI_WARPS * split);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&p.tmap_x);
    tma_prefetch_desc(&p.tmap_w[0]);
    if (SWIGLU) tma_prefetch_desc(&p.tmap_w[1]);
  }
  if (warp == EPI_WARPS + 1) {
    tmem_alloc(tmem_base_smem, G::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  if (warp == 0) count_tiles(p.rows, BN, first);
  tc_fence_before();
  if (split > 1) cluster_sync(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_base_smem;
  const int total = first[p.rows.E] * p.n_cols;

  if (warp >= EPI_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CONTROL_REGS));
    const uint64_t pol = l2_policy_evict_normal();
    if (warp == EPI_WARPS) {
      if (lane == 0) {
        uint32_t stage = 0, phase = 0, n_issued = 0;
        bool ok = true;
        // an item is looked up while the one before it is loaded
        struct Source {
          int col, expert, width;
        };
        auto look_up = [&](int t) {
          const Item c = find_item(first, p.rows.E, p.n_cols, t);
          const int2 range = rows_of(p.rows, c.expert);
          return Source{c.col, c.expert, (min(BN, range.y - range.x - c.tile * BN) + 15) & ~15};
        };
        Source next{};
        if (unit < total) next = look_up(unit);
        for (int t = unit; ok && t < total; t += n_units) {
          const Source c = next;
          const int f = c.col * FEATURES;
          int kb = kb_begin + first_block(c.expert, c.col, p.n_cols, blocks, fours);
          for (int i = 0; i < blocks; ++i) {
            if (i == min(blocks, G::STAGES) - 1 && t + n_units < total) next = look_up(t + n_units);
            if (p.withhold && t == total - 1 && rank == split - 1 && i == blocks - 1) break;
            ok = mbar_wait(&empty[stage], phase ^ 1u, abort_flag, err, p.wait_ns);
            if (!ok) break;
            uint8_t* sw = smem + stage * G::STAGE_BYTES;
            stage_width[stage] = c.width;
            mbar_arrive_expect_tx(&full[stage], 2 * G::W_BYTES + c.width * BK);
            tma_load_3d(sw, &p.tmap_w[0], &full[stage], kb * BK, f, c.expert, pol);
            if (SWIGLU) tma_load_3d(sw + G::W_BYTES, &p.tmap_w[1], &full[stage], kb * BK, f, c.expert, pol);
            else tma_load_3d(sw + G::W_BYTES, &p.tmap_w[0], &full[stage], kb * BK, f + QBLOCK, c.expert, pol);
            ++n_issued;
            if (++kb == kb_end) kb = kb_begin;
            if (++stage == G::STAGES) { stage = 0; phase ^= 1u; }
          }
        }
        // no copy may land after the exit
        for (uint32_t s = 0; s < G::STAGES; ++s)
          if (n_issued > s) mbar_wait(&full[s], ((n_issued - 1 - s) / G::STAGES) & 1u, nullptr, err, p.wait_ns);
      }
      __syncwarp();
    } else if (warp == EPI_WARPS + 2) {
      const bool gather = p.rows.order != nullptr;
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      struct Source {
        int row, width, kb;
        int4 rows;  // gathered: the four rows that this lane's copy takes (past the expert's last: that one again)
      };
      auto look_up = [&](int t) {
        const Item c = find_item(first, p.rows.E, p.n_cols, t);
        const int2 range = rows_of(p.rows, c.expert);
        Source s;
        s.row = range.x + c.tile * BN;
        s.width = (min(BN, range.y - s.row) + 15) & ~15;
        s.kb = kb_begin + first_block(c.expert, c.col, p.n_cols, blocks, fours);
        s.rows = make_int4(0, 0, 0, 0);
        if (gather && lane < BN / 4) {
          const int i = s.row + 4 * lane, last = range.y - 1;
          s.rows.x = source_row(p.rows, min(i, last));
          s.rows.y = source_row(p.rows, min(i + 1, last));
          s.rows.z = source_row(p.rows, min(i + 2, last));
          s.rows.w = source_row(p.rows, min(i + 3, last));
        }
        return s;
      };
      Source next{};
      if (unit < total) next = look_up(unit);
      for (int t = unit; ok && t < total; t += n_units) {
        const Source c = next;
        int kb = c.kb;
        for (int i = 0; i < blocks; ++i) {
          if (i == min(blocks, G::STAGES) - 1 && t + n_units < total) next = look_up(t + n_units);
          if (p.withhold && t == total - 1 && rank == split - 1 && i == blocks - 1) break;
          ok = warp_wait(&empty[stage], phase ^ 1u, abort_flag, err, p.wait_ns);
          if (!ok) break;
          uint8_t* sx = smem + stage * G::STAGE_BYTES + 2 * G::W_BYTES;
          if (gather) {
            if (4 * lane < c.width) tma_gather4(sx + lane * 4 * BK, &p.tmap_x, &full[stage], kb * BK, c.rows, pol);
          } else if (16 * lane < c.width) {
            tma_load_2d(sx + lane * 16 * BK, &p.tmap_x, &full[stage], kb * BK, c.row + 16 * lane, pol);
          }
          __syncwarp();
          if (++kb == kb_end) kb = kb_begin;
          if (++stage == G::STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // Copies that the other loading warp, whose wait gave up first, does not
      // wait for have 1 ms to land, a thousand times what a copy takes.
      if (!ok && lane == 0)
        for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < 1000000;) __nanosleep(10000);
      __syncwarp();
    } else if (warp == EPI_WARPS + 1) {
      if (lane == 0) {
        uint32_t stage = 0, phase = 0, buf = 0, bphase = 0;
        bool ok = true, there = false;  // there: the stage has been seen to be full
        for (int t = unit; ok && t < total; t += n_units) {
          for (int i0 = 0; ok && i0 < blocks; i0 += G::KG) {
            ok = mbar_wait(&tempty[buf], bphase ^ 1u, abort_flag, err, p.wait_ns);
            for (int i = i0; ok && i < min(i0 + G::KG, blocks); ++i) {
              ok = there || mbar_wait(&full[stage], phase, abort_flag, err, p.wait_ns);
              if (!ok) break;
              tc_fence_after();
              const uint32_t sw = smem_u32(smem + stage * G::STAGE_BYTES), sx = sw + 2 * G::W_BYTES;
              const uint32_t idesc = idesc_e4m3_f32(LANES, stage_width[stage]);
              const uint32_t d = tmem_base + buf * G::BUF_COLS + (i - i0) * 2 * BN;
              mma_block<1>(d, sw, sx, idesc);
              // a look at the next stage while the tensor cores are busy
              const uint32_t after = stage + 1 == G::STAGES ? 0 : stage + 1;
              there = mbar_test_wait(&full[after], after ? phase : phase ^ 1u);
              mma_block<1>(d + BN, sw + G::W_BYTES, sx, idesc);
              mma_commit(&empty[stage]);
              stage = after;
              if (!after) phase ^= 1u;
            }
            if (!ok) break;
            mma_commit(&tfull[buf]);
            if (++buf == G::BUFS) { buf = 0; bphase ^= 1u; }
          }
        }
        mma_commit(done);
        mbar_wait(done, 0, nullptr, err, p.wait_ns);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    const int quarter = warp & 3, m = warp >> 2;  // of the lanes; the matrix, or half of the features
    const uint32_t t_addr = tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) + m * BN;
    float* sc = reinterpret_cast<float*>(smem + G::SMEM_SCALES) + warp * (2 * 4 * BN);
    float* part = reinterpret_cast<float*>(smem + G::SMEM_PART);
    constexpr int XR = (BN + 31) / 32;  // columns whose scales this lane fetches
    uint32_t buf = 0, bphase = 0;
    int flip = 1;
    uint32_t seq = 0;  // partial tiles that have been handed over
    const int N = p.N;
    auto arrive_everywhere = [&](uint64_t* bar) {
      __syncwarp();
      if (split == 1) {
        if (lane == 0) mbar_arrive(bar);
      } else if (lane < split) {
        mbar_arrive_cluster(mapa_shared(smem_u32(bar), lane));
      }
    };
    // An item's place is looked up, and its first scales are loaded, while the
    // one before it is finished.
    struct Info {
      int row, valid, col, expert, kb;  // kb: the first block of K
      const float* xs[XR];
      const float* ws;
    };
    auto look_up = [&](int t) {
      const Item c = find_item(first, p.rows.E, p.n_cols, t);
      const int2 range = rows_of(p.rows, c.expert);
      Info i;
      i.row = range.x + c.tile * BN;
      i.valid = min(BN, range.y - i.row);
      i.col = c.col;
      i.expert = c.expert;
      i.kb = kb_begin + first_block(c.expert, c.col, p.n_cols, blocks, fours);
#pragma unroll
      for (int k = 0; k < XR; ++k)
        i.xs[k] = p.s_x + static_cast<int64_t>(source_row(p.rows, min(i.row + (32 * k + lane) % BN, range.y - 1))) * p.KB;
      // (a half past the features reads the first one's scales; it is not stored)
      const convrot_experts& w = p.w[SWIGLU ? m : 0];
      const int n0 = c.col * FEATURES, block = n0 / QBLOCK + (!SWIGLU && m && n0 + QBLOCK < N ? 1 : 0);
      i.ws = w.scale + c.expert * w.scale_stride + static_cast<int64_t>(block) * p.KB;
      return i;
    };
    float nx[XR][4], nw[4];
    // Four blocks' scales from kb on (past the CTA's last one: its first ones),
    // `count` of them in use.
    auto load_four = [&](const float* s, int kb, int count, float (&v)[4]) {
      if (vec) {
        const float4 f = ldg_now4(s + kb);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < count ? ldg_now(s + (kb + i < kb_end ? kb + i : kb + i - blocks)) : 0.0f;
      }
    };
    auto load_factors = [&](const Info& i, int kb, int count) {
#pragma unroll
      for (int k = 0; k < XR; ++k) load_four(i.xs[k], kb, count, nx[k]);
      load_four(i.ws, kb, count, nw);
    };
    Info info{};
    if (unit < total) {
      info = look_up(unit);
      load_factors(info, info.kb, blocks);
    }
    for (int t = unit; t < total; t += n_units) {
      const int row = info.row, valid = info.valid, width = (valid + 15) & ~15, n0 = info.col * FEATURES;
      float bv[2][4];  // of this lane's four features of either half
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const convrot_experts& wj = p.w[SWIGLU ? j : 0];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int n = n0 + (SWIGLU ? 0 : j * QBLOCK) + 4 * lane + k;
          bv[j][k] = wj.bias && n < N ? __ldg(wj.bias + info.expert * wj.bias_stride + n) : 0.0f;
        }
      }
      unsigned long long acc[BN / 2];
#pragma unroll
      for (int i = 0; i < BN / 2; ++i) acc[i] = 0ull;
      bool ok = true;
#pragma unroll 1
      for (int done_blocks = 0, kb = info.kb, i = 0; done_blocks < blocks; done_blocks += G::KG, i = (i + G::KG) & 3) {
        if (i == 0) {  // the factors of four blocks; the next four's scales are on their way meanwhile
          flip ^= 1;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < XR; ++k)
              if (BN >= 32 || lane < BN) sc[(flip * 4 + j) * BN + 32 * k + lane] = nx[k][j] * nw[j];
          __syncwarp();
          kb = kb + 4 < kb_end ? kb + 4 : kb + 4 - blocks;
          if (done_blocks + 4 < blocks) load_factors(info, kb, blocks - done_blocks - 4);
        }
        ok = warp_wait(&tfull[buf], bphase, abort_flag, err, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        drain_columns<BN, G::KG>(acc, t_addr + buf * G::BUF_COLS, sc + (flip * 4 + i) * BN, blocks - done_blocks, width);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[buf]);
        if (++buf == G::BUFS) { buf = 0; bphase ^= 1u; }
      }
      if (!ok) break;
      const int col = info.col;
      if (t + n_units < total) {
        info = look_up(t + n_units);
        load_factors(info, info.kb, blocks);
      }
#pragma unroll
      for (int part_row = 0; part_row < BN; part_row += G::PART_ROWS) {
        if (part_row >= valid) break;
        // the partial tile, once the one before it has been read everywhere
        ok = cluster_wait(pempty, (seq & 1u) ^ 1u, abort_flag, err, p.wait_ns, split);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < G::PART_ROWS / 2; ++i) {
          float a, b;
          f32x2_unpack(acc[part_row / 2 + i], a, b);
          part[2 * i * W_ROWS + 32 * warp + lane] = a;
          part[(2 * i + 1) * W_ROWS + 32 * warp + lane] = b;
        }
        arrive_everywhere(pfull);
        ok = cluster_wait(pfull, seq & 1u, abort_flag, err, p.wait_ns, split);
        if (!ok) break;
        ++seq;
        const int rows = min(G::PART_ROWS, valid - part_row);
        for (int r = warp * split + rank; r < rows; r += EPI_WARPS * split) {
          float v[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float* at = part + r * W_ROWS + j * QBLOCK + 4 * lane;
            if (split == 1) {
              const float4 s = *reinterpret_cast<const float4*>(at);
              v[j][0] = s.x; v[j][1] = s.y; v[j][2] = s.z; v[j][3] = s.w;
            } else {
              float4 s[MAX_SPLIT];
#pragma unroll
              for (int k = 0; k < MAX_SPLIT; ++k)
                if (k < split) s[k] = ld_cluster_v4(mapa_shared(smem_u32(at), k));
              v[j][0] = s[0].x; v[j][1] = s[0].y; v[j][2] = s[0].z; v[j][3] = s[0].w;
#pragma unroll
              for (int k = 1; k < MAX_SPLIT; ++k)
                if (k < split) {
                  v[j][0] += s[k].x;
                  v[j][1] += s[k].y;
                  v[j][2] += s[k].z;
                  v[j][3] += s[k].w;
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) v[j][k] += bv[j][k];
          }
          const int64_t i = row + part_row + r;
          if constexpr (SWIGLU) {
            Pair h[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
              h[k] = f32x2_pack(silu_mul(v[0][2 * k], v[1][2 * k]), silu_mul(v[0][2 * k + 1], v[1][2 * k + 1]));
            float top = max_magnitude(h);
#pragma unroll
            for (int d = 1; d < 32; d *= 2) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float scale = e4m3_scale(top);
            uint32_t q[1];
            e4m3_codes(h, scale, e4m3_factor(scale), q);
            const int n = n0 + 4 * lane;
            if (n < N) *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + i * p.ldy + n) = q[0];
            if (lane == 0) p.s_out[i * ((N + QBLOCK - 1) / QBLOCK) + col] = scale;
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int n = n0 + j * QBLOCK + 4 * lane;
              if constexpr (SCALED<TY>) {
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) top = fmaxf(top, finite_magnitude(v[j][k]));
                // (bits of positive floats order as integers)
                top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
                const float factor = power_of(top);
                if (lane == 0 && n0 + j * QBLOCK < N) p.s_out[i * ((N + QBLOCK - 1) / QBLOCK) + 2 * col + j] = factor;
                const float inv = __frcp_rn(factor);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[j][k] *= inv;
              }
              using TS = Stored<TY>;
              TS* y = static_cast<TS*>(p.out) + i * p.ldy + n;
              const bool whole = n + 4 <= N && (reinterpret_cast<uintptr_t>(y) & (4 * sizeof(TS) - 1)) == 0;
              store_outputs(y, whole, n, N, v[j]);
            }
          }
        }
        arrive_everywhere(pempty);
      }
      if (!ok) break;
    }
  }
  tc_fence_before();
  if (split > 1) cluster_sync(); else __syncthreads();
  if (warp == EPI_WARPS + 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, G::TMEM_COLS);
  }
}

// Clusters of `split` CTAs that run at the same time: looked up once per device
// (every instance of the kernel takes an SM to itself).
template <typename F>
int resident_clusters(F* kernel, int smem, int split, int& n) {
  static std::mutex mu;
  static int known[64][MAX_SPLIT + 1] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return set_cuda_error(e);
  std::lock_guard<std::mutex> lock(mu);
  n = dev < 64 ? known[dev][split] : 0;
  if (n == 0) {
    Launch l(split, FEW_THREADS, smem, nullptr, split);
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &l.cfg);
    if (e != cudaSuccess) return set_cuda_error(e);
    if (dev < 64) known[dev][split] = n;
  }
  return CONVROT_OK;
}

template <int BN, bool SWIGLU, typename TY>
int launch_as(const ExpertCall& c, cudaStream_t stream) {
  using G = FewGeom<BN>;
  const int64_t N = c.w->N, KB = n_blocks(c.K), E = c.rows.E, n = c.rows.n;
  FewParams p;
  if (int st = make_tmap_codes(&p.tmap_x, c.Q, c.rows.T, c.K, c.rows.order ? 1 : 16)) return st;
  for (int j = 0; j < (SWIGLU ? 2 : 1); ++j) {
    p.w[j] = j ? *c.up : *c.w;
    if (int st = make_tmap_experts(&p.tmap_w[j], p.w[j], E, c.K, QBLOCK)) return st;
  }
  p.rows = c.rows;
  p.s_x = c.s;
  p.out = c.out;
  p.s_out = c.s_out;
  p.ldy = c.ldy;
  p.N = static_cast<int>(N);
  p.KB = static_cast<int>(KB);
  const int features = SWIGLU ? QBLOCK : W_ROWS;
  const int64_t cols = (N + features - 1) / features, tiles = n / BN + std::min(E, n);  // of rows, at most
  if (cols * tiles > 0x7fffffff / 8) return CONVROT_ERR_UNSUPPORTED;
  p.n_cols = static_cast<int>(cols);
  p.vec_scales = KB % 4 == 0 && aligned16(c.s);
  for (int j = 0; j < (SWIGLU ? 2 : 1); ++j)
    p.vec_scales = p.vec_scales && aligned16(p.w[j].scale) && p.w[j].scale_stride % 4 == 0;
  p.wait_ns = c.test_wait_ns ? c.test_wait_ns : kWaitLimitNs;
  p.withhold = c.test_wait_ns != 0;
  static std::mutex mu;
  static uint64_t done = 0;
  auto kernel = expert_few_kernel<BN, SWIGLU, TY>;
  if (int st = allow_smem(kernel, G::smem(MAX_EXPERTS), done, mu, LAUNCH_REGS)) return st;
  // K is split over as many CTAs as give each item of evenly spread choices a
  // cluster of its own at the same time: one CTA streams 75 GB/s at most (a
  // block of 34 KB in 0.45 us), but a second round of a cluster's exchange costs more
  // than it gains. SwiGLU of 2 x 1536 x 4096 matrices: 36 items (three experts)
  // take 22.2, 15.7 and 14.1 us unsplit, in two and in four, 72 items 22.6, 19.7
  // and 20.5 us, 96 items 23.5, 28.2 and 27.5 us.
  const double reached = static_cast<double>(E) * (1.0 - std::pow(1.0 - 1.0 / static_cast<double>(E), static_cast<double>(n)));
  const double items = std::max(reached, static_cast<double>(n) / BN) * static_cast<double>(cols);
  const int sms = device_sm_count();
  int split = 1, units = sms;
  for (int s : {4, 2}) {
    if (items > sms / s || KB < s) continue;
    int n = 0;
    if (int st = resident_clusters(kernel, G::smem(MAX_EXPERTS), s, n)) return st;
    if (items <= n) {
      split = s;
      units = n;
      break;
    }
  }
  units = static_cast<int>(std::min<int64_t>(units, cols * tiles));
  p.split = split;
  Launch l(static_cast<unsigned>(units * split), FEW_THREADS, G::smem(c.rows.E), stream, split);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kernel, p);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

template <int BN>
int launch_columns(const ExpertCall& c, cudaStream_t stream) {
  if (c.up) return launch_as<BN, true, uint8_t>(c, stream);
  if (c.s_out) return launch_as<BN, false, ScaledHalf>(c, stream);
  if (c.y_dtype == CONVROT_F32) return launch_as<BN, false, float>(c, stream);
  if (c.y_dtype == CONVROT_F16) return launch_as<BN, false, __half>(c, stream);
  return launch_as<BN, false, __nv_bfloat16>(c, stream);
}

}  // namespace

int launch_expert_few(const ExpertCall& c, cudaStream_t stream) {
  // Items of the rows that an expert has on average: narrower ones cost less
  // while the expert's rows are one item, and read its weights once more for
  // every further item. 64 experts of 3 x 1024 x 2048 (16 of 3 x 1536 x 4096),
  // gate, up and down: 16 rows each 80, 80 and 87 us (67, 70 and 80) with 16, 32
  // and 64 columns; 24 rows 100, 89 and 92 us (85, 68 and 79); 32 rows 125, 100 and
  // 98 us (106, 88 and 83). By the average alone, since the counts are on the
  // device: where a few experts have most of the rows, a tile that reads weights
  // again costs little less than one that reads new ones (1024 choices of 128
  // experts, 2048 -> 2 x 768: evenly 72 us for 129 tiles, with 47 experts reached
  // and up to 121 rows each 41 us for 93).
  const int64_t per = c.rows.n / c.rows.E;
  if (per <= 16) return launch_columns<16>(c, stream);
  if (per <= 24) return launch_columns<32>(c, stream);
  return launch_columns<64>(c, stream);
}

cudaError_t few_error_word(int** p) { return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_few_error); }

}  // namespace moe
}  // namespace convrot
