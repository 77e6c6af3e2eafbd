// block_norm.cuh -- the norms before and after a transformer block fused with
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
//
// Compiled once per type of the residual stream (block_norm_*.cu).
#pragma once

#include "fp8_common.cuh"

#include <algorithm>
#include <mutex>

namespace convrot {
namespace fp8 {

namespace {

// Sticky device error word of this type's kernels: a bounded wait that gave up
// (CONVROT_ERR_TIMEOUT) or a row's sample outside [0, n_samples)
// (CONVROT_ERR_ARG).
__device__ int g_norm_error = 0;

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
  float post_eps, pre_eps, residual_scale, block_scale, inv_k;
  // of the kernels for aligned rows
  int warps_per_row, stages;
  uint32_t coef_smem;  // bytes of the coefficients, a multiple of 128
  uint32_t row_smem;  // bytes of one staged row, a multiple of 128
  uint64_t wait_ns;   // limit of every wait
  int withheld_row;   // test of the timeout: rows from here on are not copied in
};

// The sample whose gate, scale and shift apply to a row; -1 (none: gate 0, no
// modulation) after recording the error where row_sample is out of range.
__device__ __forceinline__ int sample_of(const NormParams& p, int row) {
  if (p.row_sample) {
    const int s = __ldg(p.row_sample + row);
    if (s >= 0 && s < p.n_samples) return s;
    record_error(&g_norm_error, CONVROT_ERR_ARG);
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

__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair both(float v) { return f32x2_pack(v, v); }

// The same for four consecutive features at a 16-byte aligned place, in two
// steps: first every vector's values, so that all loads of a thread's places
// are on their way together, then the arithmetic, with 1 and 0 for what is
// absent. (With a wait after every load, at the start of a kernel and at every
// change of sample: bf16 [4608, 3072] to codes with seven samples 36.8 us
// instead of 34.1 us, fp32 [4608, 12288] between weighted RMS norms with a gate
// 169 us instead of 161 us. All loads of eight features together spill: 167 us
// instead of 135 us for bf16 [4608, 16384] with gate and modulation.)
struct PostVectors {
  Pair gate[2], weight[2], bias[2];
};
__device__ __forceinline__ void load_or(const float* v, bool has, int64_t at, float otherwise, Pair (&x)[2]) {
  x[0] = x[1] = both(otherwise);
  if (has) load4(v + at, x[0], x[1]);
}
__device__ __forceinline__ PostVectors post_vectors(const NormParams& p, int s, int e) {
  PostVectors v;
  load_or(p.gate, p.gate && s >= 0, s * p.ld_gate + e, p.gate ? 0.0f : 1.0f, v.gate);
  load_or(p.post_weight, p.post_weight, e, 1.0f, v.weight);
  load_or(p.post_bias, p.post_bias, e, 0.0f, v.bias);
  return v;
}
__device__ __forceinline__ void fold(const NormParams& p, const PostVectors& v, Pair (&a)[2], Pair (&b)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const Pair g = f32x2_mul(both(p.block_scale), v.gate[i]);
    b[i] = f32x2_mul(g, v.bias[i]);
    a[i] = f32x2_mul(g, v.weight[i]);
  }
}
struct PreVectors {
  Pair weight[2], bias[2], scale[2], shift[2];
};
__device__ __forceinline__ PreVectors pre_vectors(const NormParams& p, int s, int e) {
  PreVectors v;
  load_or(p.pre_weight, p.pre_weight, e, 1.0f, v.weight);
  load_or(p.pre_bias, p.pre_bias, e, 0.0f, v.bias);
  load_or(p.scale, p.scale && s >= 0, s * p.ld_mod + e, 0.0f, v.scale);
  load_or(p.shift, p.shift && s >= 0, s * p.ld_mod + e, 0.0f, v.shift);
  return v;
}
__device__ __forceinline__ void fold(const NormParams&, const PreVectors& v, Pair (&a)[2], Pair (&b)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const Pair f = add2(v.scale[i], both(1.0f));
    a[i] = f32x2_mul(v.weight[i], f);
    b[i] = add2(f32x2_mul(v.bias[i], f), v.shift[i]);
  }
}

// What a norm does to a row: x -> (x - mean) * rstd.
struct Stats {
  float mean, rstd;
};

// Barrier of the W warps that share a row (one warp: only itself).
__device__ __forceinline__ void group_sync(int W, int group) {
  if (W == 1) __syncwarp();
  else named_bar_sync(1 + group, W * 32);
}

// The sum of v over W neighbouring lanes (W a power of two up to 16), the same
// in all of them.
__device__ __forceinline__ float lanes_sum(float v, int W) {
  if (W > 1) v += __shfl_xor_sync(0xffffffffu, v, 1);
  if (W > 2) v += __shfl_xor_sync(0xffffffffu, v, 2);
  if (W > 4) v += __shfl_xor_sync(0xffffffffu, v, 4);
  if (W > 8) v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v;
}

// What each warp of the group has put into its place of `red`, one warp's per
// lane. `red` alternates between two such arrays from one call to the next, so
// that the reads after one barrier are over before the next but one call
// writes.
__device__ __forceinline__ float2 exchange(float2 mine, int W, int group, int warp_in_group, float2* red) {
  if (W == 1) return mine;
  if ((threadIdx.x & 31) == 0) red[warp_in_group] = mine;
  group_sync(W, group);
  return red[threadIdx.x & (W - 1)];
}

// s / n by the hardware's reciprocal r of n (or a better one) and a correction
// step, within an ulp; 0 where n is 0.
__device__ __forceinline__ float quotient(float s, float n, float r) {
  const float q = s * r;
  return n > 0.0f ? fmaf(fmaf(-q, n, s), r, q) : 0.0f;
}
__device__ __forceinline__ float quotient(float s, float n) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(n));
  return quotient(s, n, r);
}

// 1 / sqrt(v): the hardware's approximation (relative error under 2^-22) and
// one Newton step, which squares it; 0 and infinity are kept as they are.
__device__ __forceinline__ float inverse_root(float v) {
  float r;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  const float better = fmaf(fmaf(-v * r, r, 1.0f), 0.5f * r, r);
  return (r > 0.0f && r < INFINITY) ? better : r;
}

// Statistics of a row of K elements spread over a group of W warps; `get(u,
// x)` yields a thread's unit u (four pairs, zeros past the end) and returns its
// place, `count(w)` the elements that warp w of the group holds.
template <int V, typename Get, typename Count>
__device__ __forceinline__ Stats row_stats(Get get, Count count, int kind, float eps, int K, float inv_k, int W, int group,
                                           int warp_in_group, float2* red) {
  Stats st{0.0f, 1.0f};
  auto total = [](const Pair (&acc)[2]) {
    float a, b;
    f32x2_unpack(add2(acc[0], acc[1]), a, b);
    return warp_sum(a + b);
  };
  Pair acc[2] = {0ull, 0ull};
  if (kind == CONVROT_NORM_RMS) {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      Pair x[4];
      get(u, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i & 1] = f32x2_fma(x[i], x[i], acc[i & 1]);
    }
    const float sum = lanes_sum(exchange(make_float2(total(acc), 0.0f), W, group, warp_in_group, red).x, W);
    st.rstd = inverse_root(fmaf(sum, inv_k, eps));
    return st;
  }
#pragma unroll
  for (int u = 0; u < V; ++u) {
    Pair x[4];
    get(u, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i & 1] = add2(acc[i & 1], x[i]);
  }
  // around the warp's own mean, then that mean's distance from the row's
  const float mean_w = quotient(total(acc), static_cast<float>(count(warp_in_group)));
  const Pair minus = both(-mean_w);
  acc[0] = acc[1] = 0ull;
#pragma unroll
  for (int u = 0; u < V; ++u) {
    Pair x[4];
    const auto unit = get(u, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Pair d = unit.inside(i, add2(x[i], minus));
      acc[i & 1] = f32x2_fma(d, d, acc[i & 1]);
    }
  }
  float m2 = total(acc);
  st.mean = mean_w;
  if (W > 1) {
    const float2 of_warp = exchange(make_float2(mean_w, m2), W, group, warp_in_group, red);
    const float n = static_cast<float>(count(threadIdx.x & (W - 1)));
    st.mean = quotient(lanes_sum(n * of_warp.x, W), static_cast<float>(K), inv_k);
    const float d = of_warp.x - st.mean;
    m2 = lanes_sum(fmaf(n * d, d, of_warp.y), W);
  }
  st.rstd = inverse_root(fmaf(m2, inv_k, eps));
  return st;
}

// How a warp takes 256 consecutive features, a unit of eight per lane in two
// halves of four: 16-bit elements are one 16-byte piece per lane, 32-bit ones
// two, 128 features apart, so that a warp's accesses are always contiguous.
template <typename T>
struct Unit {
  int lo, hi;  // first features of the two halves
  bool on[2];  // which lie inside the row
  // `whole`: the chunk is known to lie inside (every unit of a thread but its
  // last, which spares them the tests)
  __device__ __forceinline__ Unit(int chunk, int K, bool whole = false) {
    const int lane = threadIdx.x & 31;
    lo = chunk * 256 + lane * (sizeof(T) == 4 ? 4 : 8);
    hi = lo + (sizeof(T) == 4 ? 128 : 4);
    on[0] = whole || lo < K;
    on[1] = sizeof(T) == 4 ? whole || hi < K : on[0];
  }
  __device__ __forceinline__ void load(const T* row, Pair (&x)[4]) const {
    if constexpr (sizeof(T) == 4) {
      if (on[0]) load4(row + lo, x[0], x[1]);
      if (on[1]) load4(row + hi, x[2], x[3]);
    } else {
      if (on[0]) load8(row + lo, x);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!on[i / 2]) x[i] = 0ull;
  }
  // pair i with what lies past the end replaced by zeros
  __device__ __forceinline__ Pair inside(int i, Pair x) const { return on[i / 2] ? x : 0ull; }
  template <typename TU>
  __device__ __forceinline__ void store(TU* row, const Pair (&x)[4]) const {
    if constexpr (sizeof(T) == 4) {
      if (on[0]) store4(row + lo, x[0], x[1]);
      if (on[1]) store4(row + hi, x[2], x[3]);
    } else {
      if (on[0]) store8(row + lo, x);
    }
  }
  // Blocks of 128 of the unit's features: the same half of all lanes (32-bit
  // elements) or both halves of sixteen lanes.
  static constexpr int BLOCKS = sizeof(T) == 4 ? 2 : 1, SPAN = sizeof(T) == 4 ? 32 : 16;
  __device__ __forceinline__ void maxima(const Pair (&x)[4], float* m) const {
    if constexpr (BLOCKS == 2) {
      m[0] = max_magnitude({x[0], x[1]});
      m[1] = max_magnitude({x[2], x[3]});
    } else {
      m[0] = max_magnitude(x);
    }
  }
  // `sc`, `nr`: the blocks' scales and factors
  __device__ __forceinline__ void store_codes(uint8_t* q, float* s, const Pair (&x)[4], const float (&sc)[BLOCKS],
                                              const float (&nr)[BLOCKS]) const {
    if constexpr (BLOCKS == 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t c[1];
        e4m3_codes({x[2 * h], x[2 * h + 1]}, sc[h], nr[h], c);
        if (on[h]) {
          *reinterpret_cast<uint32_t*>(q + (h ? hi : lo)) = c[0];
          if ((threadIdx.x & 31) == 0) s[(h ? hi : lo) / QBLOCK] = sc[h];
        }
      }
    } else {
      uint32_t c[2];
      e4m3_codes(x, sc[0], nr[0], c);
      if (on[0]) {
        *reinterpret_cast<uint2*>(q + lo) = make_uint2(c[0], c[1]);
        if ((threadIdx.x & 15) == 0) s[lo / QBLOCK] = sc[0];
      }
    }
  }
};

// The maxima of N values over SPAN neighbouring lanes, value j in lane j of
// them: while several are left, each step hands half of them to the other lane.
template <int N, int SPAN, int D = 1>
__device__ __forceinline__ float spread_max(const float (&m)[N]) {
  if constexpr (D == SPAN) {
    static_assert(N == 1, "at most a value per lane");
    return m[0];
  } else {
    const bool odd = threadIdx.x & D;
    float next[(N + 1) / 2];
#pragma unroll
    for (int i = 0; i < (N + 1) / 2; ++i) {
      if (2 * i + 1 < N)
        next[i] = max_nan(odd ? m[2 * i + 1] : m[2 * i],
                          __shfl_xor_sync(0xffffffffu, odd ? m[2 * i] : m[2 * i + 1], D));
      else
        next[i] = max_nan(m[2 * i], __shfl_xor_sync(0xffffffffu, m[2 * i], D));
    }
    return spread_max<(N + 1) / 2, SPAN, 2 * D>(next);
  }
}

// The codes of a thread's V units, with the scales of their blocks: each scale
// is computed in one lane and handed round.
template <int V, typename Place, typename At>
__device__ __forceinline__ void quantize_row(At at, uint8_t* q, float* s, const Pair (&x)[V][4]) {
  constexpr int B = Place::BLOCKS;
  float m[V * B];
#pragma unroll
  for (int u = 0; u < V; ++u) at(u).maxima(x[u], m + u * B);
  const float scale = e4m3_scale(spread_max<V * B, Place::SPAN>(m)), factor = e4m3_factor(scale);
#pragma unroll
  for (int u = 0; u < V; ++u) {
    float sc[B], nr[B];
#pragma unroll
    for (int h = 0; h < B; ++h) {
      sc[h] = __shfl_sync(0xffffffffu, scale, u * B + h, Place::SPAN);
      nr[h] = __shfl_sync(0xffffffffu, factor, u * B + h, Place::SPAN);
    }
    at(u).store_codes(q, s, x[u], sc, nr);
  }
}

// The thread's part of a row, V units (unit u of chunk u * W + wg), from its
// arrival in shared memory to its last store: see the two kernels that use it.
// The coefficients come from `post(u, unit, a, b)` and `pre(u, unit, a, b)`;
// `loaded()` is called once the staged row has been read; it passes a barrier
// of the group and says, alike in all its threads, whether the row had arrived.
// If not, nothing is stored and do_row returns false.
template <typename T, typename TU, int V, bool FP8, typename Place, typename Post, typename Pre, typename Loaded>
__device__ __forceinline__ bool do_row(const NormParams& p, int row, const T* sh, const T* sy, int W, int group, int wg,
                                       float2* red_post, float2* red_pre, Post post, Pre pre, Loaded loaded) {
  auto count = [&](int w) {  // features of the row that warp w of the group holds
    int n = 0;
#pragma unroll
    for (int u = 0; u < V; ++u) n += min(max(p.K - (u * W + w) * 256, 0), 256);
    return n;
  };
  auto normalized = [](Pair x, const Stats& st) { return f32x2_mul(add2(x, both(-st.mean)), both(st.rstd)); };
  Pair x[V][4];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    Place(u * W + wg, p.K, u < V - 1).load(sh, x[u]);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[u][i] = f32x2_mul(x[u][i], both(p.residual_scale));
  }
  if (p.Y) {
    Stats ps{0.0f, 1.0f};
    if (p.post != CONVROT_NORM_NONE) {
      auto get = [&](int u, Pair (&v)[4]) {
        const Place unit(u * W + wg, p.K, u < V - 1);
        unit.load(sy, v);
        return unit;
      };
      ps = row_stats<V>(get, count, p.post, p.post_eps, p.K, p.inv_k, W, group, wg, red_post);
    }
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const Place unit(u * W + wg, p.K, u < V - 1);
      Pair y[4], a[4], b[4];
      unit.load(sy, y);
      post(u, unit, a, b);
      if (p.post_bias) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[u][i] = add2(x[u][i], b[i]);
      }
      if (p.post != CONVROT_NORM_NONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = normalized(y[i], ps);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[u][i] = unit.inside(i, f32x2_fma(y[i], a[i], x[u][i]));
    }
  }
  if (!loaded()) return false;
  if (p.H_out) {
    T* out = static_cast<T*>(p.H_out) + row * p.ldho;
#pragma unroll
    for (int u = 0; u < V; ++u) Place(u * W + wg, p.K, u < V - 1).store(out, x[u]);
  }
  if (!FP8 && !p.U) return true;
  Stats us{0.0f, 1.0f};
  if (p.pre != CONVROT_NORM_NONE) {
    auto get = [&](int u, Pair (&v)[4]) {
      const Place unit(u * W + wg, p.K, u < V - 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = x[u][i];
      return unit;
    };
    us = row_stats<V>(get, count, p.pre, p.pre_eps, p.K, p.inv_k, W, group, wg, red_pre);
  }
  uint8_t* q = FP8 ? p.Q + static_cast<int64_t>(row) * p.K : nullptr;
  float* s = FP8 ? p.s + static_cast<int64_t>(row) * p.KB : nullptr;
  TU* out = FP8 ? nullptr : static_cast<TU*>(p.U) + row * p.ldu;
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const Place unit(u * W + wg, p.K, u < V - 1);
    Pair a[4], b[4];
    pre(u, unit, a, b);
    if (p.pre != CONVROT_NORM_NONE) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[u][i] = normalized(x[u][i], us);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[u][i] = unit.inside(i, f32x2_fma(x[u][i], a[i], b[i]));
    if (!FP8) unit.store(out, x[u]);
  }
  if constexpr (FP8) quantize_row<V, Place>([&](int u) { return Place(u * W + wg, p.K, u < V - 1); }, q, s, x);
  return true;
}

constexpr int MAX_STAGES = 8;

// What the threads of a ring share: a stage has arrived; the row at which a
// wait gave up.
struct RingState {
  uint64_t full[MAX_STAGES];
  int gave_up;
};

// A ring of staged rows of h and y: one lane issues bulk copies a few rows
// ahead, so that enough bytes are in flight whatever the sums wait for.
//
// Threads wait one by one, and some may give up where others do not. The group
// decides together: after the barrier that follows its last reading of a row,
// `arrived` says the same to all its threads (one that waits for the next row
// already can only leave a later row there), and nothing of the row is stored
// before. The vote in it adds nothing but that the compiler sees a branch that
// a warp takes as one: without it bf16 [4608, 8192] takes 81 us, with it 76 us;
// a vote in a barrier before the row costs bf16 [4608, 3072] 26.3 us instead of
// 24.9 us.
template <typename T>
struct Ring {
  const NormParams& p;
  uint8_t* smem;
  RingState* state;
  int st = 0, phase = 0;
  __device__ uint32_t stage_bytes() const { return p.row_smem * (p.Y ? 2u : 1u); }
  __device__ void fetch(int row, int stage) {
    if (row >= p.withheld_row) return;
    const uint32_t bytes = static_cast<uint32_t>(p.K) * sizeof(T);
    uint8_t* dst = smem + stage * stage_bytes();
    uint64_t* full = &state->full[stage];
    mbar_arrive_expect_tx(full, bytes * (p.Y ? 2u : 1u));
    bulk_load(dst, static_cast<const T*>(p.H) + row * p.ldh, bytes, full);
    if (p.Y) bulk_load(dst + p.row_smem, static_cast<const T*>(p.Y) + row * p.ldy, bytes, full);
  }
  __device__ const T* h() const { return reinterpret_cast<const T*>(smem + st * stage_bytes()); }
  __device__ const T* y() const { return reinterpret_cast<const T*>(smem + st * stage_bytes() + p.row_smem); }
  __device__ void wait(int row, int* abort_flag) const {
    if (!mbar_wait(&state->full[st], phase, abort_flag, &g_norm_error, p.wait_ns)) state->gave_up = row;
  }
  __device__ bool arrived(int row) const {
    return __all_sync(0xffffffffu, *const_cast<volatile int*>(&state->gave_up) > row);
  }
  // No copy may land after the CTA has gone: the lane that fetched waits for
  // those of the row that did not arrive and of the rows ahead of it (`step`
  // apart, before `end`).
  __device__ void drain(int row, int step, int end) {
    for (int i = 0; i < p.stages && row < min(end, p.withheld_row); ++i, row += step) {
      mbar_wait(&state->full[st], phase, nullptr, &g_norm_error, p.wait_ns);
      next();
    }
  }
  __device__ void next() {
    if (++st == p.stages) {
      st = 0;
      phase ^= 1;
    }
  }
};

constexpr int WARPS = 8;  // per CTA of the grouped kernel

// Rows whose every part is a whole number of aligned 16-byte units, and whose
// coefficients fit in shared memory.
//
// W warps share a row (1, 2, 4 or 8; a CTA has 8 / W such groups), so that a
// lane has up to 96 features to spread the per-row work (sums over lanes and
// warps, square roots) over. CTAs are persistent, each over a contiguous range
// of rows, its groups taking them in turn; the affine coefficients of the
// current sample (norm weights, gate and modulation folded, only those that
// are not 0 or 1) lie in shared memory and are formed again when it changes.
//
// bf16 [4608, 3072] with gate, LayerNorm and modulation, two samples: 24.8 us
// = 4.57 TB/s (a copy with as many bytes 5.7 TB/s); RMS norms on both sides to
// codes, seven samples: 33.9 us. What is left is the chain from a row's arrival
// over two sums to its last store with 16 warps per SM to cover it (registers
// and the coefficients take the SM), issuing in 38 % of the cycles.
// (One thread block per row with one unit per thread and its coefficients in
// registers: 49 us, 53 instructions per feature, most of them per row and
// thread; coefficients read through L1 for every row: 60 us; three CTAs per SM
// at three units: 12 % slower, spilling, and the rows divide worse.)
template <typename T, typename TU, int V, bool FP8>
__global__ void __launch_bounds__(WARPS * 32, V <= 2 ? 3 : V <= 4 ? 2 : 1)
block_norm_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ RingState state[WARPS];
  __shared__ float2 red[2][WARPS];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = p.warps_per_row, G = WARPS / W, group = warp / W, wg = warp - group * W;
  const int c0 = static_cast<int>(static_cast<int64_t>(p.M) * blockIdx.x / gridDim.x);
  const int c1 = static_cast<int>(static_cast<int64_t>(p.M) * (blockIdx.x + 1) / gridDim.x);
  const int n_coef = (p.K + 255) / 256 * 256;  // floats of a coefficient vector
  const bool has_pa = p.Y && (p.gate || p.post_weight), has_pb = p.Y && p.post_bias;
  const bool has_qa = p.pre_weight || p.scale, has_qb = p.pre_bias || p.shift;
  float* cpa = reinterpret_cast<float*>(smem);
  float* cpb = cpa + (has_pa ? n_coef : 0);
  float* cqa = cpb + (has_pb ? n_coef : 0);
  float* cqb = cqa + (has_qa ? n_coef : 0);
  Ring<T> ring{p, smem + p.coef_smem, state + group};
  ring.smem += group * p.stages * ring.stage_bytes();
  const bool leader = wg == 0 && lane == 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < WARPS * MAX_STAGES; ++i) mbar_init(&state[i / MAX_STAGES].full[i % MAX_STAGES], 1);
    abort_flag = 0;
    fence_mbarrier_init();
  }
  if (threadIdx.x < WARPS) state[threadIdx.x].gave_up = 0x7fffffff;
  __syncthreads();
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  int row = c0 + group;  // the group's next row
  if (leader)
    for (int i = 0; i < p.stages && row + i * G < c1; ++i) ring.fetch(row + i * G, i);

  // A unit's coefficients: in every 256 floats the first halves of the lanes,
  // then the second ones, so that a warp reads them without bank conflicts.
  const int n_chunks = (p.K + 255) / 256;
  auto take = [&](const float* c, bool has, int u, float otherwise, Pair (&v)[4]) {
    const int chunk = u * W + wg;
    if (has && (u < V - 1 || chunk < n_chunks)) {
      load4(c + chunk * 256 + lane * 4, v[0], v[1]);
      load4(c + chunk * 256 + 128 + lane * 4, v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = both(otherwise);
    }
  };
  // A group whose wait gave up leaves its rows, and goes on meeting the others
  // where the sample changes.
  for (int start = c0; start < c1;) {
    // the rows from `start` on that share its sample
    int s = 0, end = c1;
    if (p.row_sample) {
      for (end = start; end < c1; end += 32) {
        const int mine = sample_of(p, min(end + lane, c1 - 1));
        if (end == start) s = __shfl_sync(0xffffffffu, mine, 0);
        const unsigned other = __ballot_sync(0xffffffffu, mine != s);
        if (other) {
          end = min(c1, end + __ffs(other) - 1);
          break;
        }
      }
      end = min(end, c1);
    } else if (p.rows_per_sample > 0) {
      s = start / p.rows_per_sample;
      end = static_cast<int>(min(static_cast<int64_t>(c1), (static_cast<int64_t>(s) + 1) * p.rows_per_sample));
    }
    if (has_pa || has_pb || has_qa || has_qb) {
      __syncthreads();  // the rows before may still read theirs
      // pieces of four features per lane, one half of a unit; one at a time, for
      // the registers' sake
#pragma unroll 1
      for (int piece = warp; piece < 2 * n_chunks; piece += WARPS) {
        const Unit<T> unit(piece / 2, p.K);
        const bool second = piece & 1;
        if (!(second ? unit.on[1] : unit.on[0])) continue;
        const int e = second ? unit.hi : unit.lo, at = piece * 128 + lane * 4;
        PostVectors post;
        if (has_pa || has_pb) post = post_vectors(p, s, e);
        const PreVectors pre = pre_vectors(p, s, e);
        Pair a[2], b[2];
        if (has_pa || has_pb) {
          fold(p, post, a, b);
          if (has_pa) store4(cpa + at, a[0], a[1]);
          if (has_pb) store4(cpb + at, b[0], b[1]);
        }
        fold(p, pre, a, b);
        if (has_qa) store4(cqa + at, a[0], a[1]);
        if (has_qb) store4(cqb + at, b[0], b[1]);
      }
      __syncthreads();
    }
    for (; row < end; row += G) {
      ring.wait(row, &abort_flag);
      const bool alive = do_row<T, TU, V, FP8, Unit<T>>(
          p, row, ring.h(), ring.y(), W, group, wg, red[0] + group * W, red[1] + group * W,
          [&](int u, const Unit<T>&, Pair (&a)[4], Pair (&b)[4]) {
            take(cpa, has_pa, u, p.block_scale, a);
            take(cpb, has_pb, u, 0.0f, b);
          },
          [&](int u, const Unit<T>&, Pair (&a)[4], Pair (&b)[4]) {
            take(cqa, has_qa, u, 1.0f, a);
            take(cqb, has_qb, u, 0.0f, b);
          },
          [&] {
            group_sync(W, group);
            if (!ring.arrived(row)) return false;
            if (leader && row + p.stages * G < c1) ring.fetch(row + p.stages * G, ring.st);
            return true;
          });
      if (!alive) {
        if (leader) ring.drain(row, G, c1);
        row = c1;
        break;
      }
      ring.next();
    }
    start = end;
  }
}

// The same for rows whose coefficients do not fit beside the staged rows: one
// row per CTA; a thread's factors stay in registers while the sample stays,
// what is added (a bias of the first norm; bias and shift of the second) in
// shared memory where that fits (p.coef_smem) and else read again for every
// row. Eight warps with up to six units per thread: fp32 [4608, 12288] between
// two weighted RMS norms with a gate 161 us = 5.63 TB/s, with 24 warps of two
// units 214 us.
template <typename T, typename TU, int V, bool FP8, int NW>
__global__ void __launch_bounds__(NW * 32, 1)
block_norm_wide_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ RingState state;
  __shared__ float2 red[2][NW];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = static_cast<int>(static_cast<int64_t>(p.M) * blockIdx.x / gridDim.x);
  const int c1 = static_cast<int>(static_cast<int64_t>(p.M) * (blockIdx.x + 1) / gridDim.x);
  const bool has_pb = p.Y && p.post_bias, has_qb = p.pre_bias || p.shift, staged = p.coef_smem > 0;
  float* cpb = reinterpret_cast<float*>(smem);
  float* cqb = cpb + (has_pb ? (p.K + 255) / 256 * 256 : 0);
  Ring<T> ring{p, smem + p.coef_smem, &state};
  if (threadIdx.x == 0) {
    for (int i = 0; i < MAX_STAGES; ++i) mbar_init(&state.full[i], 1);
    abort_flag = 0;
    fence_mbarrier_init();
  }
  if (threadIdx.x == 32) state.gave_up = 0x7fffffff;
  __syncthreads();
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  if (threadIdx.x == 0)
    for (int i = 0; i < p.stages && c0 + i < c1; ++i) ring.fetch(c0 + i, i);
  Pair pa[V][4], qa[V][4];
  auto coefs = [&](int s, const Unit<T>& unit, bool pre, Pair (&a)[4], Pair (&b)[4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      Pair va[2] = {0ull, 0ull}, vb[2] = {0ull, 0ull};
      if (unit.on[h]) {
        if (pre) fold(p, pre_vectors(p, s, h ? unit.hi : unit.lo), va, vb);
        else fold(p, post_vectors(p, s, h ? unit.hi : unit.lo), va, vb);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[2 * h + i] = va[i];
        b[2 * h + i] = vb[i];
      }
    }
  };
  // a thread reads back what it wrote itself: no barrier
  auto put = [&](float* c, int u, const Pair (&v)[4]) {
    float* at = c + (u * NW + warp) * 256 + lane * 4;
    if (u < V - 1 || (u * NW + warp) * 256 < p.K) {
      store4(at, v[0], v[1]);
      store4(at + 128, v[2], v[3]);
    }
  };
  auto take = [&](const float* c, int u, Pair (&v)[4]) {
    const float* at = c + (u * NW + warp) * 256 + lane * 4;
    if (u < V - 1 || (u * NW + warp) * 256 < p.K) {
      load4(at, v[0], v[1]);
      load4(at + 128, v[2], v[3]);
    } else {
      v[0] = v[1] = v[2] = v[3] = 0ull;
    }
  };
  int cur = -2;
  for (int row = c0; row < c1; ++row) {
    const int s = sample_of(p, row);
    if (s != cur) {
      cur = s;
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const Unit<T> unit(u * NW + warp, p.K, u < V - 1);
        Pair b[4];
        if (p.Y) {
          coefs(s, unit, false, pa[u], b);
          if (staged && has_pb) put(cpb, u, b);
        }
        coefs(s, unit, true, qa[u], b);
        if (staged && has_qb) put(cqb, u, b);
      }
    }
    ring.wait(row, &abort_flag);
    const bool alive = do_row<T, TU, V, FP8, Unit<T>>(
        p, row, ring.h(), ring.y(), NW, 0, warp, red[0], red[1],
        [&](int u, const Unit<T>& unit, Pair (&a)[4], Pair (&b)[4]) {
          if (has_pb) {
            if (staged) take(cpb, u, b);
            else coefs(s, unit, false, a, b);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = pa[u][i];
        },
        [&](int u, const Unit<T>& unit, Pair (&a)[4], Pair (&b)[4]) {
          if (has_qb) {
            if (staged) take(cqb, u, b);
            else coefs(s, unit, true, a, b);
          } else {
            b[0] = b[1] = b[2] = b[3] = 0ull;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = qa[u][i];
        },
        [&] {
          group_sync(NW, 0);
          if (!ring.arrived(row)) return false;
          if (threadIdx.x == 0 && row + p.stages < c1) ring.fetch(row + p.stages, ring.st);
          return true;
        });
    if (!alive) {
      if (threadIdx.x == 0) ring.drain(row, 1, c1);
      break;
    }
    ring.next();
  }
}

// Rows of any width, alignment and stride up to 12288 features: the same with
// the elements of 256 features dealt out one by one (element i of a lane is
// feature 32 i + lane), so that a warp's accesses are contiguous however the
// row starts; everything is read from global memory, the coefficients and the
// second reading of y through L1. Bound by issuing element-wise accesses: bf16
// [4000, 3071] with gate and modulation 56 us = 1.75 TB/s, fp16 [1003, 1283]
// 8.6 us; loading the coefficients element by element as they are used, not one
// vector at a time, more than doubled it.
template <typename T>
struct Scattered {
  int e0, K;
  __device__ __forceinline__ Scattered(int chunk, int K_, bool) : e0(chunk * 256 + (threadIdx.x & 31)), K(K_) {}
  template <typename TV>
  __device__ __forceinline__ void load(const TV* row, Pair (&x)[4]) const {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = e0 + 32 * i < K ? to_f32(row[e0 + 32 * i]) : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f32x2_pack(v[2 * i], v[2 * i + 1]);
  }
  __device__ __forceinline__ Pair inside(int i, Pair x) const {
    float a, b;
    f32x2_unpack(x, a, b);
    return f32x2_pack(e0 + 64 * i < K ? a : 0.0f, e0 + 64 * i + 32 < K ? b : 0.0f);
  }
  template <typename TU>
  __device__ __forceinline__ void store(TU* row, const Pair (&x)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      f32x2_unpack(x[i], a, b);
      if (e0 + 64 * i < K) row[e0 + 64 * i] = from_f32<TU>(a);
      if (e0 + 64 * i + 32 < K) row[e0 + 64 * i + 32] = from_f32<TU>(b);
    }
  }
  // a block of 128 is half of every lane's elements
  static constexpr int BLOCKS = 2, SPAN = 32;
  __device__ __forceinline__ void maxima(const Pair (&x)[4], float* m) const {
    m[0] = max_magnitude({x[0], x[1]});
    m[1] = max_magnitude({x[2], x[3]});
  }
  __device__ __forceinline__ void store_codes(uint8_t* q, float* s, const Pair (&x)[4], const float (&sc)[2],
                                              const float (&nr)[2]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t c[1];
      e4m3_codes({x[2 * h], x[2 * h + 1]}, sc[h], nr[h], c);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + 128 * h + 32 * i < K) q[e0 + 128 * h + 32 * i] = static_cast<uint8_t>(c[0] >> (8 * i));
      if ((threadIdx.x & 31) == 0 && e0 + 128 * h < K) s[(e0 + 128 * h) / QBLOCK] = sc[h];
    }
  }
};

template <typename T, typename TU, int V, bool FP8>
__global__ void __launch_bounds__(WARPS * 32, V <= 2 ? 3 : 1)
block_norm_scattered_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 red[2][WARPS];
  const int warp = threadIdx.x >> 5;
  const int W = p.warps_per_row, G = WARPS / W, group = warp / W, wg = warp - group * W;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * G + group; row < p.M; row += static_cast<int64_t>(gridDim.x) * G) {
    const int s = sample_of(p, static_cast<int>(row));
    // one vector at a time, so that its loads are on their way together
    auto fold = [](Pair (&a)[4], const Pair (&v)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = f32x2_mul(a[i], v[i]);
    };
    auto post = [&](int, const Scattered<T>& unit, Pair (&a)[4], Pair (&b)[4]) {
      Pair v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = both(p.gate && s < 0 ? 0.0f : p.block_scale);
        b[i] = 0ull;
      }
      if (p.gate && s >= 0) {
        unit.load(p.gate + s * p.ld_gate, v);
        fold(a, v);
      }
      if (p.post_bias) {
        unit.load(p.post_bias, b);
        fold(b, a);
      }
      if (p.post_weight) {
        unit.load(p.post_weight, v);
        fold(a, v);
      }
    };
    auto pre = [&](int, const Scattered<T>& unit, Pair (&a)[4], Pair (&b)[4]) {
      Pair v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = both(1.0f);
        b[i] = 0ull;
      }
      if (p.pre_weight) unit.load(p.pre_weight, a);
      if (p.pre_bias) unit.load(p.pre_bias, b);
      if (p.scale && s >= 0) {
        unit.load(p.scale + s * p.ld_mod, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = add2(v[i], both(1.0f));
        fold(a, v);
        fold(b, v);
      }
      if (p.shift && s >= 0) {
        unit.load(p.shift + s * p.ld_mod, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = add2(b[i], v[i]);
      }
    };
    do_row<T, TU, V, FP8, Scattered<T>>(
        p, static_cast<int>(row), static_cast<const T*>(p.H) + row * p.ldh,
        p.Y ? static_cast<const T*>(p.Y) + row * p.ldy : nullptr, W, group, wg, red[0] + group * W, red[1] + group * W,
        post, pre, [&] {
          group_sync(W, group);
          return true;
        });
  }
}

// Rows longer than the kernels above hold in registers: one row per CTA at a
// time, kept as fp32 in shared memory, elements taken one by one (thread t
// owns the elements t, t + blockDim, ...). Bound by the latency of its loads:
// with gate and modulation bf16 [512, 32768] 251 us, [512, 24001] 102 us; four
// loads of each array together need 59 registers, which leaves one CTA per SM:
// 236 and 173 us.
constexpr int ANY_THREADS = 1024;
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
__global__ void __launch_bounds__(ANY_THREADS, 1)
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
          Pair o[2] = {0ull, 0ull};
          if (e < p.K) {
            o[0] = f32x2_pack(x[e], x[e + 1]);
            o[1] = f32x2_pack(x[e + 2], x[e + 3]);
          }
          float m = max_magnitude(o);
#pragma unroll
          for (int d = 1; d < 32; d *= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
          const float sc = e4m3_scale(m);
          uint32_t c[1];
          e4m3_codes(o, sc, e4m3_factor(sc), c);
          if (e < p.K) *reinterpret_cast<uint32_t*>(p.Q + row * p.K + e) = c[0];
          if (lane == 0) p.s[row * p.KB + kb] = sc;
        }
      }
    }
    __syncthreads();  // the row's last reads, before the next row is written
  }
}

constexpr int MAX_SMEM = 227 * 1024 - 2048;
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

size_t stage_bytes(const NormParams& p) { return static_cast<size_t>(p.row_smem) * (p.Y ? 2 : 1); }

template <typename T, typename TU, int V, bool FP8>
int launch_grouped(NormParams& p, cudaStream_t stream) {
  static std::mutex mu;
  static uint64_t done = 0;
  auto kernel = block_norm_kernel<T, TU, V, FP8>;
  if (int st = allow_smem(kernel, done, mu)) return st;
  const int groups = WARPS / p.warps_per_row, sms = device_sm_count();
  const size_t stage = stage_bytes(p) * groups;
  // as many CTAs per SM as the registers allow while each keeps two rows per
  // group in flight; then as many rows as fit
  int per_sm = V <= 2 ? 3 : V <= 4 ? 2 : 1;
  auto room = [&](int n) { return static_cast<size_t>(MAX_SMEM) / n - (n > 1 ? 2048 : 0); };
  while (per_sm > 1 && p.coef_smem + 2 * stage > room(per_sm)) --per_sm;
  p.stages = static_cast<int>(std::min<size_t>(MAX_STAGES, (room(per_sm) - p.coef_smem) / stage));
  const int64_t ctas = (static_cast<int64_t>(p.M) + groups - 1) / groups;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(ctas, static_cast<int64_t>(per_sm) * sms));
  return launch_rows(kernel, p, grid, WARPS * 32, p.coef_smem + p.stages * stage, stream);
}

template <typename T, typename TU, int V, bool FP8, int NW>
int launch_wide(NormParams& p, cudaStream_t stream) {
  static std::mutex mu;
  static uint64_t done = 0;
  auto kernel = block_norm_wide_kernel<T, TU, V, FP8, NW>;
  if (int st = allow_smem(kernel, done, mu)) return st;
  const size_t added = static_cast<size_t>((p.Y && p.post_bias) + (p.pre_bias || p.shift)) * ((p.K + 255) / 256) * 1024;
  p.coef_smem = added + 2 * stage_bytes(p) <= MAX_SMEM ? static_cast<uint32_t>(added) : 0;
  p.stages = static_cast<int>(std::min<size_t>(MAX_STAGES, (MAX_SMEM - p.coef_smem) / stage_bytes(p)));
  const unsigned grid = static_cast<unsigned>(std::min(p.M, device_sm_count()));
  return launch_rows(kernel, p, grid, NW * 32, p.coef_smem + p.stages * stage_bytes(p), stream);
}

// Warps per row of the grouped kernel: enough that a lane has at most four
// units (two CTAs per SM; six with all eight warps) and that two rows of every
// group fit beside the coefficients, and more while there are fewer rows than
// groups on the GPU. 0: nothing fits. More warps per row cost more than the
// warps per SM that two units allow (24 instead of 16) give: bf16 with gate,
// LayerNorm and modulation, [4608, 3072] 24.7 us with four warps and three
// units, 33.1 us with eight and two (to codes 28.9 and 39.6 us); [4608, 2048]
// 17.2 us with two and four, 21.1 us with four and two; [8192, 1280] 20.9 us
// with two and three, 21.2 us with one and five, 27.1 us with four and two.
int pick_warps(const NormParams& p) {
  const int chunks = (p.K + 255) / 256;
  const int64_t sms = device_sm_count();
  for (int W = 1; W <= WARPS; W *= 2) {
    if (chunks > (W == WARPS ? 6 : 4) * W || p.coef_smem + 2 * stage_bytes(p) * (WARPS / W) > MAX_SMEM) continue;
    if (W < WARPS && chunks > W && p.M * static_cast<int64_t>(W) * 2 <= sms * WARPS) continue;
    return W;
  }
  return 0;
}

template <typename T, typename TU, int V, bool FP8>
int launch_scattered(NormParams& p, int chunks, cudaStream_t stream) {
  const int64_t sms = device_sm_count();
  int W = 1;
  while (W < WARPS && (chunks > V * W || (chunks > W && p.M * static_cast<int64_t>(W) * 2 <= sms * WARPS))) W *= 2;
  p.warps_per_row = W;
  const int64_t ctas = (p.M + static_cast<int64_t>(WARPS / W) - 1) / (WARPS / W);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(ctas, (V <= 2 ? 3 : 1) * sms));
  return launch_rows(block_norm_scattered_kernel<T, TU, V, FP8>, p, grid, WARPS * 32, 0, stream);
}

// `test`: the call is the timeout's test, which only kernels that wait can take.
template <typename T, typename TU, bool FP8>
int launch_typed(NormParams& p, bool vec, bool test, cudaStream_t stream) {
  const int chunks = (p.K + 255) / 256;
  if (const int W = vec ? pick_warps(p) : 0) {
    p.warps_per_row = W;
    const int v = (chunks + W - 1) / W;
    if (v == 1) return launch_grouped<T, TU, 1, FP8>(p, stream);
    if (v == 2) return launch_grouped<T, TU, 2, FP8>(p, stream);
    if (v == 3) return launch_grouped<T, TU, 3, FP8>(p, stream);
    if (v == 4) return launch_grouped<T, TU, 4, FP8>(p, stream);
    if (v == 5) return launch_grouped<T, TU, 5, FP8>(p, stream);
    return launch_grouped<T, TU, 6, FP8>(p, stream);
  }
  if (vec && chunks > 3 * WARPS && stage_bytes(p) <= MAX_SMEM) {
    if (chunks <= 4 * WARPS) return launch_wide<T, TU, 4, FP8, WARPS>(p, stream);
    if (chunks <= 5 * WARPS) return launch_wide<T, TU, 5, FP8, WARPS>(p, stream);
    if (chunks <= 6 * WARPS) return launch_wide<T, TU, 6, FP8, WARPS>(p, stream);
    if (chunks <= 8 * WARPS) return launch_wide<T, TU, 4, FP8, 2 * WARPS>(p, stream);
  }
  if (test) return CONVROT_ERR_UNSUPPORTED;
  if (chunks <= 6 * WARPS) return chunks <= 2 * WARPS ? launch_scattered<T, TU, 2, FP8>(p, chunks, stream)
                                                       : launch_scattered<T, TU, 6, FP8>(p, chunks, stream);
  static std::mutex mu;
  static uint64_t done = 0;
  auto kernel = block_norm_any_kernel<T, TU, FP8>;
  if (int st = allow_smem(kernel, done, mu)) return st;
  const unsigned grid = std::min(p.M, 2 * device_sm_count());
  return launch_rows(kernel, p, grid, ANY_THREADS, static_cast<size_t>(p.K) * 4, stream);
}

}  // namespace

template <typename T>
int launch_block_norm_as(const convrot_block_norm_args& a, cudaStream_t stream, NormTimeoutTest test) {
  NormParams p{};
  p.wait_ns = test.wait_ns ? test.wait_ns : kWaitLimitNs;
  p.withheld_row = test.wait_ns ? static_cast<int>(test.row) : 0x7fffffff;
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
  const bool sampled = a.gate || a.scale || a.shift;
  p.row_sample = sampled ? a.row_sample : nullptr;
  p.ldh = a.ldh;
  p.ldy = a.ldy;
  p.ldho = a.ldho;
  p.ldu = a.ldu;
  p.ld_gate = a.ld_gate;
  p.ld_mod = a.ld_mod;
  p.M = static_cast<int>(a.M);
  p.K = static_cast<int>(a.K);
  p.KB = static_cast<int>(n_blocks(a.K));
  p.rows_per_sample = sampled ? static_cast<int>(std::min<int64_t>(a.rows_per_sample, 0x7fffffff)) : 0;
  p.n_samples = static_cast<int>(a.n_samples);
  p.post = a.Y ? a.post_norm : CONVROT_NORM_NONE;
  p.pre = a.pre_norm;
  p.post_eps = a.post_eps;
  p.pre_eps = a.pre_eps;
  p.residual_scale = a.residual_scale;
  p.block_scale = a.block_scale;
  p.inv_k = 1.0f / static_cast<float>(a.K);
  const size_t sz = sizeof(T), usz = dtype_size(a.u_dtype);
  p.row_smem = static_cast<uint32_t>((a.K * sz + 127) / 128 * 128);
  const int n_coef = (a.Y && (a.gate || a.post_weight)) + (a.Y && a.post_bias) + (a.pre_weight || a.scale) +
                     (a.pre_bias || a.shift);
  p.coef_smem = static_cast<uint32_t>(n_coef * ((a.K + 255) / 256 * 256) * 4);
  auto row_ok = [](const void* ptr, int64_t ld, size_t size) { return !ptr || (aligned16(ptr) && ld * size % 16 == 0); };
  const bool vec = a.K % 8 == 0 && row_ok(a.H, a.ldh, sz) && row_ok(a.Y, a.ldy, sz) && row_ok(a.H_out, a.ldho, sz) &&
                   row_ok(a.U, a.ldu, usz) && row_ok(a.gate, a.ld_gate, 4) && row_ok(a.scale, a.ld_mod, 4) &&
                   row_ok(a.shift, a.ld_mod, 4) && row_ok(a.post_weight, 0, 4) && row_ok(a.post_bias, 0, 4) &&
                   row_ok(a.pre_weight, 0, 4) && row_ok(a.pre_bias, 0, 4);
  if (a.Q) return launch_typed<T, T, true>(p, vec, test.wait_ns != 0, stream);
  if (a.u_dtype == CONVROT_F32) return launch_typed<T, float, false>(p, vec, test.wait_ns != 0, stream);
  if (a.u_dtype == CONVROT_F16) return launch_typed<T, __half, false>(p, vec, test.wait_ns != 0, stream);
  return launch_typed<T, __nv_bfloat16, false>(p, vec, test.wait_ns != 0, stream);
}

template <typename T>
cudaError_t norm_error_word(int** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_norm_error);
}

}  // namespace fp8
}  // namespace convrot
