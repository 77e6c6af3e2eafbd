// expert_gemm.cu -- the block-scaled 8-bit floating-point linears over rows
// sorted by expert: rows of one expert go through that expert's matrix.
//
//   y[i,n] = sum_b s_x[m,b] s_w[e,n/128,b] (sum_{k in b} q_x[m,k] q_w[e,n,k]) + bias[e,n],
//   m = the activation row of sorted row i, e = its expert,
//
// and, for a gate and an up matrix, h = silu(g) u, quantized over 128 features
// as it leaves.
#include "expert_common.cuh"

#include <algorithm>
#include <cstdlib>

namespace convrot {
namespace moe {

namespace {

// ---------------------------------------------------------------------------
// few rows per expert: weights streamed to registers
// ---------------------------------------------------------------------------
//
// As the few-row kernel of the dense linears: a CTA takes 16 output features
// of one expert (for SwiGLU 16 of the gate and the same 16 of the up matrix),
// its warps every NW-th block of K each, on mma.sync (m16n8k32, weights first)
// with operands loaded straight to registers; an expert's rows are taken eight
// at a time. SwiGLU: eight CTAs (a cluster) have the 128 features of a scale
// between them; their row maxima meet through distributed shared memory.

constexpr int FEATURES = 16;
constexpr int CHUNK = 8;  // rows at a time
constexpr int STREAM_WARPS = 8;
constexpr int BLOCK_CTAS = QBLOCK / FEATURES;  // CTAs that share a block's scale

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

struct StreamParams {
  const uint8_t* X;  // codes [T,K]
  const float* s_x;  // [T,KB]
  Rows rows;
  convrot_experts w[2];  // the matrix, or gate and up
  void* out;             // Y [n,N], or the codes of h [n,N]
  float* s_out;          // their scales [n, ceil(N/128)]
  int64_t ldy;
  int N, K, KB, tiles;   // tiles: CTAs along the features
};

template <bool SWIGLU, typename TY>
__global__ void __launch_bounds__(STREAM_WARPS * 32) expert_stream_kernel(const __grid_constant__ StreamParams p) {
  constexpr int NW = STREAM_WARPS, W = SWIGLU ? 2 : 1;
  __shared__ float part[W][NW][CHUNK][FEATURES + 1];
  __shared__ float row_max[2][BLOCK_CTAS][CHUNK];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int slot = static_cast<int>(blockIdx.x) / p.tiles, n0 = (static_cast<int>(blockIdx.x) - slot * p.tiles) * FEATURES;
  // the slot-th expert that has rows (the same search in every warp)
  int expert = -1, left = slot;
  for (int e0 = 0; e0 < p.rows.E; e0 += 32) {
    const int e = e0 + lane;
    const int2 r = e < p.rows.E ? rows_of(p.rows, e) : make_int2(0, 0);
    const uint32_t some = __ballot_sync(0xffffffffu, r.y > r.x);
    const int count = __popc(some);
    if (left < count) {
      const bool here = (some >> lane & 1u) && __popc(some & ((1u << lane) - 1u)) == left;
      expert = e0 + __ffs(__ballot_sync(0xffffffffu, here)) - 1;
      break;
    }
    left -= count;
  }
  if (expert < 0) return;  // the whole cluster: its CTAs have one slot
  // that every CTA of the cluster runs is known before one writes to another
  if (SWIGLU) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int2 range = rows_of(p.rows, expert);
  const int N = p.N;
  const uint8_t* w[W][2];
  const float* ws[W];
#pragma unroll
  for (int j = 0; j < W; ++j) {
    const uint8_t* q = p.w[j].q + expert * p.w[j].q_stride;
    w[j][0] = q + static_cast<int64_t>(min(n0 + g, N - 1)) * p.K;
    w[j][1] = q + static_cast<int64_t>(min(n0 + g + 8, N - 1)) * p.K;
    ws[j] = p.w[j].scale + expert * p.w[j].scale_stride + static_cast<int64_t>(min(n0, N - 1) / QBLOCK) * p.KB;
  }
  auto load_w = [&](int kb, uint4 (&a)[W][2][2]) {
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = kb * BK + h * 64 + t * 16;
        const bool on = k < p.K;
        a[j][h][0] = on ? ldg_stream(w[j][0] + k) : make_uint4(0, 0, 0, 0);
        a[j][h][1] = on ? ldg_stream(w[j][1] + k) : make_uint4(0, 0, 0, 0);
      }
  };
  int turn = 0;
  for (int i0 = range.x; i0 < range.y; i0 += CHUNK, ++turn) {
    const int last = range.y - 1, rows = min(CHUNK, range.y - i0);
    uint4 a[W][2][2], next[W][2][2];
    if (warp < p.KB) load_w(warp, a);
    // the row whose codes this lane holds and the two whose results it has
    // (past the last one: the last one again, not stored)
    const uint8_t* xr = p.X + static_cast<int64_t>(source_row(p.rows, min(i0 + g, last))) * p.K;
    const float* s0 = p.s_x + static_cast<int64_t>(source_row(p.rows, min(i0 + 2 * t, last))) * p.KB;
    const float* s1 = p.s_x + static_cast<int64_t>(source_row(p.rows, min(i0 + 2 * t + 1, last))) * p.KB;
    float acc[W][4] = {};
    for (int kb = warp; kb < p.KB; kb += NW) {
      if (kb + NW < p.KB) load_w(kb + NW, next);
      uint4 b[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = kb * BK + h * 64 + t * 16;
        b[h] = k < p.K ? __ldg(reinterpret_cast<const uint4*>(xr + k)) : make_uint4(0, 0, 0, 0);
      }
      const float x0 = __ldg(s0 + kb), x1 = __ldg(s1 + kb);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float sw = __ldg(ws[j] + kb);
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mma_sync_e4m3(d, a[j][h][0].x, a[j][h][1].x, a[j][h][0].y, a[j][h][1].y, b[h].x, b[h].y);
          mma_sync_e4m3(d, a[j][h][0].z, a[j][h][1].z, a[j][h][0].w, a[j][h][1].w, b[h].z, b[h].w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(d[i], sw * (i & 1 ? x1 : x0), acc[j][i]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          a[j][h][0] = next[j][h][0];
          a[j][h][1] = next[j][h][1];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[j][warp][2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[j][i];
    __syncthreads();
    // 16 lanes per row
    const int m = threadIdx.x / FEATURES, n = threadIdx.x % FEATURES;
    const bool on = m < rows && n0 + n < N;
    float y[W] = {};
    if (m < CHUNK) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
#pragma unroll
        for (int v = 0; v < NW; ++v) y[j] += part[j][v][m][n];
        if (p.w[j].bias && on) y[j] += __ldg(p.w[j].bias + expert * p.w[j].bias_stride + n0 + n);
      }
    }
    if constexpr (SWIGLU) {
      const uint32_t rank = cluster_ctarank();
      const float h = on ? silu_mul_fast(y[0], y[1]) : 0.0f;
      float top = fabsf(h);
#pragma unroll
      for (int d = 1; d < FEATURES; d *= 2) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
      // to every CTA of the block; the buffers alternate, so that this turn's
      // maxima cannot meet the reads of the turn before
      if (turn == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      if (m < CHUNK && n < BLOCK_CTAS)
        st_cluster_f32(mapa_shared(smem_u32(&row_max[turn & 1][rank][m]), n), top);
      cluster_sync();
      if (on) {
        top = 0.0f;
#pragma unroll
        for (int c = 0; c < BLOCK_CTAS; ++c) top = max_nan(top, row_max[turn & 1][c][m]);
        const float sc = e4m3_scale(top);
        Pair x[2] = {f32x2_pack(h, 0.0f), 0ull};
        uint32_t q[1];
        e4m3_codes(x, sc, e4m3_factor(sc), q);
        static_cast<uint8_t*>(p.out)[(i0 + m) * p.ldy + n0 + n] = static_cast<uint8_t>(q[0]);
        if (rank == 0 && n == 0) p.s_out[static_cast<int64_t>(i0 + m) * ((N + QBLOCK - 1) / QBLOCK) + n0 / QBLOCK] = sc;
      }
    } else {
      if (on) static_cast<TY*>(p.out)[(i0 + m) * p.ldy + n0 + n] = from_f32<TY>(y[0]);
    }
    __syncthreads();  // the sums have been read
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

StreamParams stream_params(const uint8_t* Q, const float* s, int64_t K, const Rows& r, int64_t N) {
  StreamParams p{};
  p.X = Q;
  p.s_x = s;
  p.rows = r;
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.KB = static_cast<int>(n_blocks(K));
  return p;
}

template <bool SWIGLU, typename TY>
int launch_stream(StreamParams& p, cudaStream_t stream) {
  const int64_t slots = std::min<int64_t>(p.rows.E, p.rows.n);
  p.tiles = SWIGLU ? static_cast<int>(n_blocks(p.N)) * BLOCK_CTAS : (p.N + FEATURES - 1) / FEATURES;
  if (slots * p.tiles > 0x7fffffff) return CONVROT_ERR_UNSUPPORTED;
  Launch l(static_cast<unsigned>(slots * p.tiles), STREAM_WARPS * 32, 0, stream, SWIGLU ? BLOCK_CTAS : 1);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, expert_stream_kernel<SWIGLU, TY>, p);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

int pick(const Rows& r) {
  if (const char* v = getenv("EXPERT_KERNEL")) return atoi(v);
  return r.n / r.E > 64 ? 2 : 1;
}

}  // namespace

int launch_expert_swiglu(const uint8_t* Q, const float* s, int64_t K, const Rows& r, const convrot_experts& gate,
                         const convrot_experts& up, uint8_t* Q_h, float* s_h, cudaStream_t stream,
                         uint64_t test_wait_ns) {
  const ExpertCall c{Q, s, K, r, &gate, &up, Q_h, s_h, gate.N, 0, test_wait_ns};
  const int which = pick(r);
  if (which == 2) return launch_expert_pair(c, stream);
  if (which == 1) return launch_expert_few(c, stream);
  StreamParams p = stream_params(Q, s, K, r, gate.N);
  p.w[0] = gate;
  p.w[1] = up;
  p.out = Q_h;
  p.s_out = s_h;
  p.ldy = gate.N;
  return launch_stream<true, uint8_t>(p, stream);
}

int launch_expert_linear(const uint8_t* Q, const float* s, int64_t K, const Rows& r, const convrot_experts& w, void* Y,
                         int64_t ldy, int y_dtype, cudaStream_t stream, uint64_t test_wait_ns) {
  const ExpertCall c{Q, s, K, r, &w, nullptr, Y, nullptr, ldy, y_dtype, test_wait_ns};
  const int which = pick(r);
  if (which == 2) return launch_expert_pair(c, stream);
  if (which == 1) return launch_expert_few(c, stream);
  StreamParams p = stream_params(Q, s, K, r, w.N);
  p.w[0] = w;
  p.out = Y;
  p.ldy = ldy;
  if (y_dtype == CONVROT_F32) return launch_stream<false, float>(p, stream);
  if (y_dtype == CONVROT_F16) return launch_stream<false, __half>(p, stream);
  return launch_stream<false, __nv_bfloat16>(p, stream);
}

}  // namespace moe
}  // namespace convrot
