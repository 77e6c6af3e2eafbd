// moe_route.cu -- what stands around the experts' linears: the router's choice
// of experts, the plan that sorts the choices by expert, and the weighted sum
// of the experts' rows.
#include "moe_common.cuh"

#include <algorithm>
#include <climits>

namespace convrot {
namespace moe {

using fp8::from_f32;
using fp8::Launch;
using fp8::to_f32;

// Sticky device error word of these kernels (experts out of range).
__device__ int g_moe_error = 0;

namespace {

// ---------------------------------------------------------------------------
// the router
// ---------------------------------------------------------------------------
//
//   s = softmax(l) or 1 / (1 + exp(-l)),   v = s + bias (l itself without one),
// the top_k largest v of the best groups, ties to the lowest index.
//
// One token per warp, its logits read once; expert i is on lane i % 32. The
// work is a chain of warp-wide maxima over order-preserving 32-bit keys
// (redux), so a token costs instructions and latency, not bandwidth: 4096 x 256
// logits, eight of four groups by sigmoid and bias, 1860 instructions a warp,
// 14 us; one token 3.7 us, most of it a launch.
//
// Which of two values is larger must not hang on the rounding of exp: values
// are formed in fp32 with a bound on their error (a group's: the bounds of its
// summands), and where more than one may be the largest by it (about one token
// in a few hundred), those alone are formed again in 64 bits and compared there.
// So the choice is that of 64-bit arithmetic at the price of fp32. (All values
// in 64 bits would take some 50 us for 4096 x 256 logits at this GPU's fp64
// rate.)

constexpr int ROUTE_WARPS = 4;
// Eight CTAs an SM leave 64 registers a thread, for which the kernel of up to
// 256 experts spills 36 bytes.

struct RouteParams {
  const void* logits;
  int64_t ld, T;
  const float* bias;
  int32_t* experts;
  float* weights;
  float scale;
  int E, top_k, n_groups, per_group, top_groups, group_top, lanes_per_group;
  uint32_t group_factor;  // e / per_group = e * group_factor >> 20 for e < 1024
  bool sigmoid, renormalise;
};

// Order-preserving keys: a < b as floats <=> key(a) < key(b); 0 is below every
// value's key and says "not to be chosen".
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 to +0: they are equal
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
// The index (any lane's `i`) of the largest `v`, the lowest among equal ones;
// lanes without a candidate give i = INT_MAX.
__device__ __forceinline__ int warp_argmax(double v, int i) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const double w = __shfl_xor_sync(0xffffffffu, v, d);
    const int j = __shfl_xor_sync(0xffffffffu, i, d);
    if (j != INT_MAX && (i == INT_MAX || w > v || (w == v && j < i))) {
      v = w;
      i = j;
    }
  }
  return i;
}

// Scores in 64 bits. Out of line: inlined, the compiler moves them out of the
// loops that rarely need them (160 us for 4096 x 256 logits).
__device__ __noinline__ double exp64(float l, float m) { return exp(static_cast<double>(l) - static_cast<double>(m)); }
__device__ __noinline__ double score64(float l, float m, double total, bool sigmoid) {
  return sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l))) : exp64(l, m) / total;
}

// exp(-c) / (1 + exp(-l)) for c = 0, or l <= c < 0: without underflow in the
// latter case where l is near c.
__device__ __forceinline__ float sigmoid_from(float l, float c) {
  const float e = expf(-fabsf(l));
  return __fdiv_rn(l >= 0.0f ? 1.0f : c == 0.0f ? e : expf(l - c), 1.0f + e);
}

template <typename T, int EPL>
__global__ void __launch_bounds__(ROUTE_WARPS * 32, EPL <= 8 ? 8 : 1) moe_route_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ float route_smem[];  // grouped: [warp][E + padding] logits, then values
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  constexpr uint32_t ALL = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * ROUTE_WARPS + warp;
  if (token >= p.T) return;
  const T* row = static_cast<const T*>(p.logits) + token * p.ld;
  const bool biased = p.bias != nullptr;

  float l[EPL], s[EPL];
  bool bad = false;  // the row has no scores
  float m = -INFINITY;
#pragma unroll
  for (int r = 0; r < EPL; ++r) {
    const int e = lane + 32 * r;
    l[r] = e < p.E ? to_f32(row[e]) : -INFINITY;
    bad |= l[r] != l[r] || (!p.sigmoid && l[r] == INFINITY);
    m = fmaxf(m, l[r]);
  }
  float total = 1.0f;
  if (p.sigmoid) {
#pragma unroll
    for (int r = 0; r < EPL; ++r) s[r] = sigmoid_fast(l[r]);
  } else {
    m = value_of(__reduce_max_sync(ALL, key_of(m)));
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < EPL; ++r) {
      s[r] = l[r] == -INFINITY ? 0.0f : expf(l[r] - m);
      sum += s[r];
    }
    total = warp_sum(sum);
    const float inv = total > 0.0f ? __fdiv_rn(1.0f, total) : 0.0f;
#pragma unroll
    for (int r = 0; r < EPL; ++r) s[r] *= inv;
  }
  // what is compared; an expert whose logit or bias is -inf is not chosen
  uint32_t key[EPL];
#pragma unroll
  for (int r = 0; r < EPL; ++r) {
    const int e = lane + 32 * r;
    const float b = biased && e < p.E ? __ldg(p.bias + e) : 0.0f;
    bad |= b != b;
    const float v = biased ? s[r] + b : l[r];
    key[r] = l[r] == -INFINITY || v == -INFINITY ? 0u : key_of(v);
  }
  if (__any_sync(ALL, bad)) {  // a NaN stays visible: in the weights
    if (lane < p.top_k) {
      p.experts[token * p.top_k + lane] = lane;
      p.weights[token * p.top_k + lane] = __uint_as_float(0x7fffffffu);
    }
    return;
  }

  // Bound on the error of an fp32 value against its 64-bit one. Sigmoid: the
  // exponential is within 2^-22 and, from its argument's rounding, |x| 2^-23,
  // both times s (1 - s) (|x| s (1 - s) <= 0.23); the sum, the reciprocal (one
  // ulp) and the product make 4 x 2^-24 s: 3.3e-7 in all. Softmax: exp within 2
  // ulp, the rounding of its argument (x exp(-x) 2^-24 <= 2^-25), a sum of at
  // most EPL + 5 steps, a division and a product: 44 x 2^-24 / total at most.
  // The bias adds 2^-24 |v|.
  const float score_error = p.sigmoid ? 0x1p-21f : 0x1p-18f * __fdiv_rn(1.0f, fmaxf(total, 1.0f));
  auto error_at = [&](float v) { return score_error + 0x1p-23f * fabsf(v); };
  double total64 = 0.0;  // softmax: formed when first needed
  auto need_total64 = [&]() {  // by the whole warp
    if (p.sigmoid || total64 != 0.0) return;
#pragma unroll 1
    for (int r = 0; r < EPL; ++r) {
      float x = -INFINITY;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i == r) x = l[i];
      total64 += x == -INFINITY ? 0.0 : exp64(x, m);
    }
    total64 = warp_sum(total64);
  };
  auto value64 = [&](float logit, int e) {
    return score64(logit, m, total64, p.sigmoid) + (biased ? static_cast<double>(__ldg(p.bias + e)) : 0.0);
  };

  if (p.n_groups > 1) {
    // The groups' values: lanes_per_group lanes look through a group each, from
    // shared memory, where a group starts lanes_per_group words further than
    // the one before it ends (another bank for each).
    const int P = p.lanes_per_group, pitch = p.per_group + P;
    float* sl = route_smem + warp * 2 * p.n_groups * pitch;
    float* sv = sl + p.n_groups * pitch;
    const bool exact = p.group_top == 1 && !biased;
#pragma unroll
    for (int r = 0; r < EPL; ++r) {
      const int e = lane + 32 * r;
      if (e < p.E) {
        const int at = e + static_cast<int>(e * p.group_factor >> 20) * P;
        sl[at] = l[r];
        sv[at] = key[r] == 0u ? -INFINITY : exact ? l[r] : biased ? value_of(key[r]) : s[r];
      }
    }
    __syncwarp();
    const int g = lane / P, sub = lane - g * P;
    const bool mine = g < p.n_groups;
    float a = -INFINITY, b = -INFINITY;  // the two largest
    if (mine)
      for (int i = sub; i < p.per_group; i += P) {
        const float v = sv[g * pitch + i];
        b = fmaxf(b, fminf(a, v));
        a = fmaxf(a, v);
      }
    for (int d = 1; d < P; d *= 2) {
      const float oa = __shfl_xor_sync(ALL, a, d), ob = __shfl_xor_sync(ALL, b, d);
      b = fmaxf(fmaxf(b, ob), fminf(a, oa));
      a = fmaxf(a, oa);
    }
    const bool two = p.group_top == 2 && b > -INFINITY;
    // (half of the value where it is not exact: a sum of two need not fit fp32)
    const float value = exact ? a : two ? fmaf(0.5f, a, 0.5f * b) : 0.5f * a;
    // What it may be off by is what its summands are, whose sum may cancel; and
    // the roundings of the sum and of the bounds.
    const float off = exact || value == INFINITY
                          ? 0.0f
                          : fmaf(0x1p-22f, fabsf(value), 0.5f * (error_at(a) + (two ? error_at(b) : 0.0f)));
    const float least_value = value - off, most_value = value + off;
    uint32_t gkey = mine && a > -INFINITY ? key_of(value) : 0u;
    uint32_t open = 0;  // the chosen groups
    for (int j = 0; j < p.top_groups; ++j) {
      const uint32_t top = __reduce_max_sync(ALL, gkey);
      if (top == 0u) break;
      int best = static_cast<int>(__reduce_min_sync(ALL, gkey == top ? static_cast<uint32_t>(g) : 0xffffu));
      if (!exact) {
        const float least = __shfl_sync(ALL, least_value, best * P);
        const bool near = gkey != 0u && most_value >= least;
        if (__popc(__ballot_sync(ALL, near && sub == 0)) > 1) {
          need_total64();
          double a64 = -INFINITY, b64 = -INFINITY;
          if (near) {
            const float last = two ? b : a;
            const float from = last - 2.5f * error_at(last);
            for (int i = sub; i < p.per_group; i += P) {
              const float w = sv[g * pitch + i];
              if (w == -INFINITY || !(w >= from || w == a)) continue;
              const double x = value64(sl[g * pitch + i], g * p.per_group + i);
              b64 = fmax(b64, fmin(a64, x));
              a64 = fmax(a64, x);
            }
          }
          for (int d = 1; d < P; d *= 2) {
            const double oa = __shfl_xor_sync(ALL, a64, d), ob = __shfl_xor_sync(ALL, b64, d);
            b64 = fmax(fmax(b64, ob), fmin(a64, oa));
            a64 = fmax(a64, oa);
          }
          best = warp_argmax(two ? a64 + b64 : a64, near ? g : INT_MAX);
        }
      }
      open |= 1u << best;
      if (g == best) gkey = 0u;
    }
#pragma unroll
    for (int r = 0; r < EPL; ++r) {
      const int e = lane + 32 * r;
      if (e < p.E && !(open >> (e * p.group_factor >> 20) & 1u)) key[r] = 0u;
    }
  }

  // The choice. A first turn goes by the fp32 values and takes one more than
  // top_k; where two neighbours of that list are near, a second one compares
  // what is near the largest in 64 bits.
  int chosen;          // lane j: the j-th expert
  uint32_t place_key;  // and its value's key
  auto choose = [&](bool exact, int count) {
    chosen = -1;
    place_key = 0u;
    uint32_t left[EPL], most = 0u;  // what is left, and the lane's largest of it
#pragma unroll
    for (int r = 0; r < EPL; ++r) {
      left[r] = key[r];
      most = max(most, key[r]);
    }
    for (int j = 0; j < count; ++j) {
      const uint32_t top = __reduce_max_sync(ALL, most);
      if (top == 0u) break;
      uint32_t e = 0xffffu;
      if (most == top) {
#pragma unroll
        for (int r = EPL - 1; r >= 0; --r)
          if (left[r] == top) e = lane + 32 * r;
      }
      e = __reduce_min_sync(ALL, e);
      if (exact) {
        const float v = value_of(top), lo = v - 2.5f * error_at(v);
        uint32_t near = 0u;
#pragma unroll
        for (int r = 0; r < EPL; ++r)
          if (left[r] != 0u && (left[r] == top || value_of(left[r]) >= lo)) near |= 1u << r;
        if (__reduce_add_sync(ALL, __popc(near)) > 1) {
          need_total64();
          double best = -INFINITY;
          int at = INT_MAX;
          for (; near; near &= near - 1) {
            const int r = __ffs(near) - 1;
            float x = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
              if (i == r) x = l[i];
            const double y = value64(x, lane + 32 * r);
            if (at == INT_MAX || y > best) {
              best = y;
              at = lane + 32 * r;
            }
          }
          e = warp_argmax(best, at);
        }
      }
      if ((e & 31u) == static_cast<uint32_t>(lane)) {
        most = 0u;
#pragma unroll
        for (int r = 0; r < EPL; ++r) {
          if (e >> 5 == static_cast<uint32_t>(r)) left[r] = 0u;
          most = max(most, left[r]);
        }
      }
      if (lane == j) {
        chosen = static_cast<int>(e);
        place_key = top;
      }
    }
  };
  // (of 32 choices the 33rd has no lane to compare with)
  choose(biased && p.top_k == 32, min(p.top_k + (biased ? 1 : 0), 32));
  if (biased && p.top_k < 32) {
    const uint32_t next = __shfl_down_sync(ALL, place_key, 1);
    const float v = value_of(place_key);
    const bool near = lane < p.top_k && next != 0u && !(value_of(next) < v - 2.5f * error_at(v));
    if (__any_sync(ALL, near)) choose(true, p.top_k);
    if (lane >= p.top_k) chosen = -1;
  }
  const float logit = chosen < 0 ? -INFINITY : to_f32(row[chosen]);
  // The weights from the logits: where they are renormalised, relative to the
  // largest chosen one, so that scores too small for fp32 keep their ratios.
  const float most = p.renormalise ? value_of(__reduce_max_sync(ALL, key_of(logit))) : 0.0f;
  float weight = 0.0f;
  if (chosen >= 0)
    weight = p.sigmoid         ? sigmoid_from(logit, fminf(most, 0.0f))
             : p.renormalise ? expf(logit - most)
                             : __fdiv_rn(expf(logit - m), total);
  if (p.renormalise) {
    const float sum = warp_sum(weight);
    weight = sum > 0.0f ? __fdiv_rn(weight, sum) : 0.0f;
  }
  if (lane < p.top_k) {
    p.experts[token * p.top_k + lane] = chosen;
    p.weights[token * p.top_k + lane] = weight * p.scale;
  }
}

// ---------------------------------------------------------------------------
// the plan
// ---------------------------------------------------------------------------
//
// A stable counting sort of n choices by expert. No atomics decide an order:
// it is the choices' own. Choices outside [0, E) count as expert E, behind all
// others.
//
// Few choices: one launch. Every CTA places the choices of W experts and looks
// through all choices for them, twice: every warp has a contiguous part; the
// first turn counts its choices of each of the CTA's experts and those of lower
// ones, the second hands the places out, by ballots. Nothing passes between
// CTAs, but every SM looks at every choice: 512 of 128 experts take 3.2 us, 12288
// of 64, 256 and 1024 experts 5.7, 6.2 and 9.5 us (in two launches 6.3, 6.9 and 9.8
// us), 16384 of 64 experts 7.0 us (6.4 us), 65536 of 256 experts 33 us (9.8 us).
//
// Many: two launches. The choices are dealt out in contiguous parts; the first
// launch counts a part's choices of every expert, the second sums the parts
// before its own up and ranks its choices (32 at a time: the lanes that hold the
// same expert find each other by match).

constexpr int PLAN_WARPS = 32;
constexpr int PLAN_STEP = 4;          // choices per lane and turn
constexpr int64_t PLAN_ONE = 12288;   // most choices of the one launch
constexpr int PART_WARPS = 16;        // the two launches: warps of a CTA
constexpr int64_t PLAN_PARTS = 32;    // most parts
constexpr int64_t PART_LEAST = 1024;  // fewest choices of a part

__device__ __forceinline__ int bucket_of(int e, int E, bool& bad) {
  if (e >= 0 && e < E) return e;
  bad |= e != -1;
  return E;
}

template <int W>
__device__ __forceinline__ void plan_experts(const int32_t* __restrict__ experts, int64_t n, int E,
                                             int32_t* __restrict__ order, int32_t* __restrict__ place,
                                             int32_t* __restrict__ offsets) {
  __shared__ int counts[PLAN_WARPS][W + 1];  // of the CTA's experts; of lower ones
  constexpr uint32_t ALL = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = static_cast<int>(blockIdx.x) * W;
  constexpr int TURN = 32 * PLAN_STEP;
  const int64_t turns = (n + TURN - 1) / TURN;
  const int64_t t0 = turns * warp / PLAN_WARPS, t1 = turns * (warp + 1) / PLAN_WARPS;
  // a turn's choices, as places among the CTA's experts: negative for lower ones
  auto load = [&](int64_t t, int (&b)[PLAN_STEP]) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < PLAN_STEP; ++j) {
      const int64_t i = t * TURN + 32 * j + lane;
      b[j] = i < n ? bucket_of(__ldg(experts + i), E, bad) - e0 : INT_MAX;
    }
    if (bad) record_error(&g_moe_error, CONVROT_ERR_ARG);
  };
  int mine[W] = {}, lower = 0;
  for (int64_t t = t0; t < t1; ++t) {
    int b[PLAN_STEP];
    load(t, b);
#pragma unroll
    for (int j = 0; j < PLAN_STEP; ++j) {
      lower += b[j] < 0;
#pragma unroll
      for (int w = 0; w < W; ++w) mine[w] += b[j] == w;
    }
  }
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const int c = __reduce_add_sync(ALL, mine[w]);
    if (lane == 0) counts[warp][w] = c;
  }
  lower = __reduce_add_sync(ALL, lower);
  if (lane == 0) counts[warp][W] = lower;
  __syncthreads();
  // lane v has warp v's counts
  int at[W], first = __reduce_add_sync(ALL, counts[lane][W]);
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const int c = counts[lane][w];
    at[w] = first + __reduce_add_sync(ALL, lane < warp ? c : 0);
    if (threadIdx.x == 0 && e0 + w <= E) offsets[e0 + w] = first;
    first += __reduce_add_sync(ALL, c);
  }
  const uint32_t before = (1u << lane) - 1u;
  for (int64_t t = t0; t < t1; ++t) {
    int b[PLAN_STEP];
    load(t, b);
#pragma unroll
    for (int j = 0; j < PLAN_STEP; ++j) {
      const bool here = b[j] >= 0 && b[j] < W;
      if (!__any_sync(ALL, here)) continue;
      int to = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const uint32_t same = __ballot_sync(ALL, b[j] == w);
        if (b[j] == w) to = at[w] + __popc(same & before);
        at[w] += __popc(same);
      }
      if (here) {
        const int64_t i = t * TURN + 32 * j + lane;
        const bool some = e0 + b[j] < E;
        order[to] = some ? static_cast<int32_t>(i) : -1;
        place[i] = some ? to : -1;
      }
    }
  }
}

template <int W>
__global__ void __launch_bounds__(PLAN_WARPS * 32)
moe_plan_kernel(const int32_t* __restrict__ experts, int64_t n, int E, int32_t* __restrict__ order,
                int32_t* __restrict__ place, int32_t* __restrict__ offsets) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  plan_experts<W>(experts, n, E, order, place, offsets);
}

// Part p of `parts`: choices [part_start(p), part_start(p + 1)), whole groups of 32.
__device__ __forceinline__ int64_t part_start(int64_t n, int64_t parts, int64_t p) {
  const int64_t at = (n + 31) / 32 * p / parts * 32;
  return at < n ? at : n;
}

// counts [part][E + 1]
__global__ void __launch_bounds__(PART_WARPS * 32)
moe_count_kernel(const int32_t* __restrict__ experts, int64_t n, int E, int32_t* __restrict__ counts) {
  __shared__ int count[MAX_EXPERTS + 1];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  for (int e = threadIdx.x; e <= E; e += PART_WARPS * 32) count[e] = 0;
  __syncthreads();
  const int64_t i0 = part_start(n, gridDim.x, blockIdx.x), i1 = part_start(n, gridDim.x, blockIdx.x + 1);
  bool bad = false;
#pragma unroll 4
  for (int64_t i = i0 + threadIdx.x; i < i1; i += PART_WARPS * 32)
    atomicAdd(&count[bucket_of(__ldg(experts + i), E, bad)], 1);  // a sum: any order gives the same
  if (bad) record_error(&g_moe_error, CONVROT_ERR_ARG);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += PART_WARPS * 32) counts[static_cast<int64_t>(blockIdx.x) * (E + 1) + e] = count[e];
}

__global__ void __launch_bounds__(PART_WARPS * 32)
moe_place_kernel(const int32_t* __restrict__ experts, int64_t n, int E, const int32_t* __restrict__ counts,
                 int32_t* __restrict__ order, int32_t* __restrict__ place, int32_t* __restrict__ offsets) {
  extern __shared__ int place_smem[];  // next place [PART_WARPS][E + 1]
  __shared__ int warp_sums[PART_WARPS];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  constexpr uint32_t ALL = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, B = E + 1;
  const int part = static_cast<int>(blockIdx.x), parts = static_cast<int>(gridDim.x);
  int* next = place_smem + warp * B;
  for (int e = lane; e < B; e += 32) next[e] = 0;
  __syncwarp();
  const int64_t i0 = part_start(n, parts, part), i1 = part_start(n, parts, part + 1);
  const int64_t groups = (i1 - i0 + 31) / 32, g0 = groups * warp / PART_WARPS, g1 = groups * (warp + 1) / PART_WARPS;
  bool bad = false;
  auto bucket_at = [&](int64_t i) { return i < i1 ? bucket_of(__ldg(experts + i), E, bad) : -1; };
  for (int64_t g = g0; g < g1; ++g) {
    const int b = bucket_at(i0 + g * 32 + lane);
    const uint32_t same = __match_any_sync(ALL, b);
    if (b >= 0 && (same >> lane) == 1u) next[b] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  int carry = 0;  // choices of the experts before this turn's
  for (int e0 = 0; e0 < B; e0 += PART_WARPS * 32) {
    const int e = e0 + threadIdx.x;
    int before = 0, all = 0;
    if (e < B) {
      int v[PLAN_PARTS];  // on their way together
#pragma unroll
      for (int c = 0; c < PLAN_PARTS; ++c) v[c] = c < parts ? __ldg(counts + static_cast<int64_t>(c) * B + e) : 0;
#pragma unroll
      for (int c = 0; c < PLAN_PARTS; ++c) {
        before += c < part ? v[c] : 0;
        all += v[c];
      }
    }
    int scan = all;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(ALL, scan, d);
      if (lane >= d) scan += v;
    }
    if (lane == 31) warp_sums[warp] = scan;
    __syncthreads();
    int first = carry + scan - all;
#pragma unroll
    for (int w = 0; w < PART_WARPS; ++w) {
      if (w < warp) first += warp_sums[w];
      carry += warp_sums[w];
    }
    if (e < B) {
      if (part == 0) offsets[e] = first;
      int at = first + before;
#pragma unroll
      for (int w = 0; w < PART_WARPS; ++w) {
        const int c = place_smem[w * B + e];
        place_smem[w * B + e] = at;
        at += c;
      }
    }
    __syncthreads();
  }
  for (int64_t g = g0; g < g1; ++g) {
    const int64_t i = i0 + g * 32 + lane;
    const int b = bucket_at(i);
    const uint32_t same = __match_any_sync(ALL, b);
    const int to = b >= 0 ? next[b] + __popc(same & ((1u << lane) - 1u)) : 0;
    __syncwarp();
    if (b >= 0 && (same >> lane) == 1u) next[b] += __popc(same);
    __syncwarp();
    if (b >= 0) {
      order[to] = b < E ? static_cast<int32_t>(i) : -1;
      place[i] = b < E ? to : -1;
    }
  }
}

// ---------------------------------------------------------------------------
// rows in the plan's order
// ---------------------------------------------------------------------------
//
// The many-row kernel reads the rows of a tile once for every column of tiles,
// and gathering them each time costs it more than this one pass (bound by
// writing n K bytes): copies of four rows by index take the copy engine 43 ns
// each, 1.1 ms for 4096 tokens' 32768 rows of 4096 codes against 0.5 ms.

constexpr int ROW_THREADS = 256;

// Codes and scales of X by token to rows in the plan's order: a warp per row.
__global__ void __launch_bounds__(ROW_THREADS)
moe_gather_kernel(const uint8_t* __restrict__ Q, const float* __restrict__ s, int64_t K, int KB, const __grid_constant__ Rows r,
                  uint8_t* __restrict__ Q_out, float* __restrict__ s_out) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (ROW_THREADS / 32) + (threadIdx.x >> 5);
  if (i >= r.n || i >= __ldg(r.offsets + r.E)) return;
  const int64_t m = min(max(static_cast<int64_t>(__ldg(r.order + i)) / r.top_k, int64_t{0}), r.T - 1);
  const uint4* from = reinterpret_cast<const uint4*>(Q + m * K);
  uint4* to = reinterpret_cast<uint4*>(Q_out + i * K);
  const int64_t pieces = K / 16;
  for (int64_t c0 = lane; c0 < pieces; c0 += 4 * 32) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c0 + 32 * j < pieces) v[j] = __ldg(from + c0 + 32 * j);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c0 + 32 * j < pieces) to[c0 + 32 * j] = v[j];
  }
  for (int b = lane; b < KB; b += 32) s_out[i * KB + b] = __ldg(s + m * KB + b);
}

struct PackArgs {
  const void* X;
  int64_t ldx;
  uint32_t n_qblocks, KB, K;
  bool vec;
  const int32_t* place;  // null: rows by token
  int top_k;
  int64_t n;
  uint8_t* Q;
  float* s;
};
// The codes and scale of the 128 features of a token that eight lanes share
// (fp8_pack_kernel's), to the token's row or to every row that the plan gives it.
template <typename T>
__device__ __forceinline__ void pack_block(const PackArgs& a, uint32_t b) {
  const uint32_t sub = threadIdx.x & 7, row = b / a.KB, kb = b - row * a.KB, col = kb * fp8::QBLOCK + sub * 16;
  const bool on = b < a.n_qblocks && col < a.K;
  fp8::Pair x[8];
  if (on) {
    fp8::load16(static_cast<const T*>(a.X) + row * a.ldx + col, a.vec, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0ull;
  }
  float m = fp8::max_magnitude(x);
#pragma unroll
  for (int d = 1; d < 8; d *= 2) m = fp8::max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float sc = fp8::e4m3_scale(m);
  uint32_t c[4];
  fp8::e4m3_codes(x, sc, fp8::e4m3_factor(sc), c);
  if (!on) return;
  const uint4 codes = make_uint4(c[0], c[1], c[2], c[3]);
  if (!a.place) {
    *reinterpret_cast<uint4*>(a.Q + static_cast<int64_t>(row) * a.K + col) = codes;
    if (sub == 0) a.s[static_cast<int64_t>(row) * a.KB + kb] = sc;
    return;
  }
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t p = __ldg(a.place + static_cast<int64_t>(row) * a.top_k + j);
    if (p < 0 || p >= a.n) continue;
    *reinterpret_cast<uint4*>(a.Q + p * a.K + col) = codes;
    if (sub == 0) a.s[p * a.KB + kb] = sc;
  }
}

template <typename T>
__global__ void __launch_bounds__(ROW_THREADS, sizeof(T) == 2 ? 8 : 6) moe_pack_kernel(const __grid_constant__ PackArgs a) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  pack_block<T>(a, blockIdx.x * (ROW_THREADS / 8) + (threadIdx.x >> 3));
}

// A plan of few choices and the pack by token, which need nothing of each
// other, in one launch: the first `plan_ctas` CTAs plan.
template <typename T, int W>
__global__ void __launch_bounds__(PLAN_WARPS * 32)
moe_plan_pack_kernel(const int32_t* __restrict__ experts, int64_t n, int E, int32_t* __restrict__ order,
                     int32_t* __restrict__ place, int32_t* __restrict__ offsets, uint32_t plan_ctas,
                     const __grid_constant__ PackArgs a) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  if (blockIdx.x < plan_ctas) plan_experts<W>(experts, n, E, order, place, offsets);
  else pack_block<T>(a, (blockIdx.x - plan_ctas) * (PLAN_WARPS * 4) + (threadIdx.x >> 3));
}

// ---------------------------------------------------------------------------
// the weighted sum
// ---------------------------------------------------------------------------
//
//   Y[t] = residual[t] + sum_j weights[t,j] rows[place[t,j]], summed in fp32 in
// the order of j, one rounding at the end. Reads every row once. From HBM, 4096
// tokens: eight bf16 rows of 4096 each 51 us = 5.9 TB/s, four of 2048 19.7 us = 4.3
// TB/s (there a thread has four loads in flight, and waits for them).

// A token's rows are loaded several at a time: one after the other, their
// latencies add up (bf16 [32, 2048] of eight rows 7.5 us).

constexpr int COMBINE_THREADS = 128;

// Eight values of a row (one, without VEC) as they are in memory: loads that
// stay where they are written, before the first use of any of them.
template <typename T, bool VEC>
struct Raw {
  static constexpr int PIECES = VEC ? sizeof(T) / 2 : 1;
  uint4 v[PIECES];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                     : "l"(reinterpret_cast<const uint4*>(p) + i));
    } else if constexpr (sizeof(T) == 4) {
      asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v[0].x) : "l"(p));
    } else {
      uint16_t h;
      asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(h) : "l"(p));
      v[0].x = h;
    }
  }
  __device__ __forceinline__ void unpack(float (&x)[VEC ? 8 : 1]) const {
    if constexpr (!VEC && sizeof(T) == 4) {
      x[0] = __uint_as_float(v[0].x);
    } else if constexpr (!VEC) {
      float none;
      fp8::unpack2<T>(v[0].x, x[0], none);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[4 * i] = __uint_as_float(v[i].x);
        x[4 * i + 1] = __uint_as_float(v[i].y);
        x[4 * i + 2] = __uint_as_float(v[i].z);
        x[4 * i + 3] = __uint_as_float(v[i].w);
      }
    } else {
      fp8::unpack2<T>(v[0].x, x[0], x[1]);
      fp8::unpack2<T>(v[0].y, x[2], x[3]);
      fp8::unpack2<T>(v[0].z, x[4], x[5]);
      fp8::unpack2<T>(v[0].w, x[6], x[7]);
    }
  }
};

template <typename TR, typename TY, bool VEC>
__global__ void __launch_bounds__(COMBINE_THREADS, 8) moe_combine_kernel(const __grid_constant__ CombineArgs a, uint32_t chunks) {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  constexpr int E = VEC ? 8 : 1;                 // features per thread
  constexpr int BATCH = sizeof(TR) == 4 ? 4 : 8;  // rows loaded together
  const uint32_t token = blockIdx.x / chunks;
  const int64_t t = token, col = ((blockIdx.x - token * chunks) * blockDim.x + threadIdx.x) * static_cast<int64_t>(E);
  // lane j has the token's choice j (top_k <= 32)
  const int lane = threadIdx.x & 31;
  int mine = -1;
  float weight = 0.0f;
  if (lane < a.top_k) {
    mine = __ldg(a.place + t * a.top_k + lane);
    weight = __ldg(a.weights + t * a.top_k + lane);
    if (mine >= a.n) mine = -1;
  }
  const TR* rows = static_cast<const TR*>(a.rows) + col;
  float acc[E];
#pragma unroll
  for (int k = 0; k < E; ++k) acc[k] = 0.0f;
#pragma unroll 1
  for (int j0 = 0; j0 < a.top_k; j0 += BATCH) {
    Raw<TR, VEC> x[BATCH];
    float s[BATCH];
    int r[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      if (j0 + j >= a.top_k) break;
      r[j] = __shfl_sync(0xffffffffu, mine, j0 + j);
      if (r[j] < 0 || col >= a.N) continue;
      x[j].load(rows + r[j] * a.ldr);
      if (a.r_scale) s[j] = __ldg(a.r_scale + r[j] * a.r_blocks + col / fp8::QBLOCK);
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      if (j0 + j >= a.top_k) break;
      float f = __shfl_sync(0xffffffffu, weight, j0 + j);
      if (r[j] < 0) continue;
      float v[E];
      x[j].unpack(v);
      if (a.r_scale) f *= s[j];
      if constexpr (VEC) {
        const unsigned long long f2 = f32x2_pack(f, f);
#pragma unroll
        for (int k = 0; k < E; k += 2)
          f32x2_unpack(f32x2_fma(f2, f32x2_pack(v[k], v[k + 1]), f32x2_pack(acc[k], acc[k + 1])), acc[k], acc[k + 1]);
      } else {
        acc[0] = fmaf(f, v[0], acc[0]);
      }
    }
  }
  if (col >= a.N) return;
  TY* y = static_cast<TY*>(a.Y) + t * a.ldy + col;
  if (a.residual) {
    const TY* res = static_cast<const TY*>(a.residual) + t * a.ld_res + col;
    float v[E];
    if constexpr (VEC) {
      fp8::Pair q[4];
      fp8::load8(res, q);
#pragma unroll
      for (int k = 0; k < 4; ++k) f32x2_unpack(q[k], v[2 * k], v[2 * k + 1]);
    } else {
      v[0] = to_f32(*res);
    }
#pragma unroll
    for (int k = 0; k < E; ++k) acc[k] += v[k];
  }
  if constexpr (VEC) {
    fp8::Pair q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = f32x2_pack(acc[2 * k], acc[2 * k + 1]);
    fp8::store8(y, q);
  } else {
    *y = from_f32<TY>(acc[0]);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

template <typename T, int EPL>
int route_launch(const RouteParams& p, cudaStream_t stream) {
  const size_t smem =
      p.n_groups > 1 ? sizeof(float) * ROUTE_WARPS * 2 * p.n_groups * (p.per_group + p.lanes_per_group) : 0;
  Launch l(static_cast<unsigned>((p.T + ROUTE_WARPS - 1) / ROUTE_WARPS), ROUTE_WARPS * 32, smem, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, moe_route_kernel<T, EPL>, p);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

template <typename T>
int route_as(const RouteParams& p, cudaStream_t stream) {
  if (p.E <= 64) return route_launch<T, 2>(p, stream);
  if (p.E <= 128) return route_launch<T, 4>(p, stream);
  if (p.E <= 256) return route_launch<T, 8>(p, stream);
  if (p.E <= 512) return route_launch<T, 16>(p, stream);
  return route_launch<T, 32>(p, stream);
}

template <typename TR, typename TY>
int combine_as(const CombineArgs& a, cudaStream_t stream) {
  auto fits = [&](const void* p, int64_t ld, size_t size) { return aligned16(p) && (ld * size) % 16 == 0; };
  const bool vec = a.N % 8 == 0 && fits(a.rows, a.ldr, sizeof(TR)) && fits(a.Y, a.ldy, sizeof(TY)) &&
                   (!a.residual || fits(a.residual, a.ld_res, sizeof(TY)));
  const int64_t items = vec ? a.N / 8 : a.N;  // of a token
  const int64_t threads = std::min<int64_t>(COMBINE_THREADS, (items + 31) / 32 * 32);
  const int64_t chunks = (items + threads - 1) / threads;
  if (chunks * a.T > 0x7fffffff) return CONVROT_ERR_UNSUPPORTED;
  Launch l(static_cast<unsigned>(chunks * a.T), static_cast<unsigned>(threads), 0, stream);
  const uint32_t c = static_cast<uint32_t>(chunks);
  const cudaError_t e = vec ? cudaLaunchKernelEx(&l.cfg, moe_combine_kernel<TR, TY, true>, a, c)
                            : cudaLaunchKernelEx(&l.cfg, moe_combine_kernel<TR, TY, false>, a, c);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

template <typename TR>
int combine_rows(const CombineArgs& a, cudaStream_t stream) {
  if (a.y_dtype == CONVROT_F32) return combine_as<TR, float>(a, stream);
  if (a.y_dtype == CONVROT_F16) return combine_as<TR, __half>(a, stream);
  return combine_as<TR, __nv_bfloat16>(a, stream);
}

}  // namespace

int launch_route(const convrot_moe_route_args& a, cudaStream_t stream) {
  RouteParams p{};
  p.logits = a.logits;
  p.ld = a.ld;
  p.T = a.T;
  p.bias = a.bias;
  p.experts = a.experts;
  p.weights = a.weights;
  p.scale = a.scale;
  p.E = a.n_experts;
  p.top_k = a.top_k;
  p.n_groups = a.n_groups;
  p.per_group = a.n_experts / a.n_groups;
  p.group_factor = ((1u << 20) + p.per_group - 1) / p.per_group;
  p.top_groups = a.top_groups;
  p.group_top = a.group_top;
  p.lanes_per_group = 1;
  while (2 * p.lanes_per_group * a.n_groups <= 32) p.lanes_per_group *= 2;
  p.sigmoid = a.score == CONVROT_MOE_SIGMOID;
  p.renormalise = a.renormalise != 0;
  if (a.dtype == CONVROT_F32) return route_as<float>(p, stream);
  if (a.dtype == CONVROT_F16) return route_as<__half>(p, stream);
  return route_as<__nv_bfloat16>(p, stream);
}

template <int W>
static int plan_as(const int32_t* experts, int64_t n, int E, int32_t* order, int32_t* place, int32_t* offsets,
                   cudaStream_t stream) {
  Launch l(static_cast<unsigned>((E + W) / W), PLAN_WARPS * 32, 0, stream);  // E + 1 buckets
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, moe_plan_kernel<W>, experts, n, E, order, place, offsets);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

static int64_t plan_parts(int64_t n) { return n <= PLAN_ONE ? 0 : std::min(PLAN_PARTS, (n + PART_LEAST - 1) / PART_LEAST); }
size_t plan_workspace(int64_t n, int E) { return static_cast<size_t>(plan_parts(n)) * (E + 1) * sizeof(int32_t); }

int launch_plan(const int32_t* experts, int64_t n, int E, int32_t* order, int32_t* place, int32_t* offsets, void* workspace,
                cudaStream_t stream) {
  const int64_t parts = plan_parts(n);
  // As many experts per CTA as leave every SM about one CTA: 512 choices of 151,
  // 303, 607 and 1000 experts take 2.4, 2.6, 3.2 and 4.3 us.
  if (parts == 0) {
    if (E < 152) return plan_as<1>(experts, n, E, order, place, offsets, stream);
    if (E < 304) return plan_as<2>(experts, n, E, order, place, offsets, stream);
    if (E < 608) return plan_as<4>(experts, n, E, order, place, offsets, stream);
    return plan_as<8>(experts, n, E, order, place, offsets, stream);
  }
  int32_t* counts = static_cast<int32_t*>(workspace);
  static std::mutex mu;
  static uint64_t done = 0;
  constexpr int most = PART_WARPS * (MAX_EXPERTS + 1) * 4;
  static_assert(most <= 100 * 1024, "shared memory");
  if (int st = fp8::allow_smem(moe_place_kernel, most, done, mu)) return st;
  Launch count(static_cast<unsigned>(parts), PART_WARPS * 32, 0, stream);
  cudaError_t e = cudaLaunchKernelEx(&count.cfg, moe_count_kernel, experts, n, E, counts);
  if (e != cudaSuccess) return set_cuda_error(e);
  Launch put(static_cast<unsigned>(parts), PART_WARPS * 32, sizeof(int) * PART_WARPS * (E + 1), stream);
  e = cudaLaunchKernelEx(&put.cfg, moe_place_kernel, experts, n, E, static_cast<const int32_t*>(counts), order, place, offsets);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

int launch_gather(const uint8_t* Q, const float* s, int64_t K, const Rows& r, uint8_t* Q_out, float* s_out,
                  cudaStream_t stream) {
  const int64_t per = ROW_THREADS / 32;
  Launch l(static_cast<unsigned>((r.n + per - 1) / per), ROW_THREADS, 0, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, moe_gather_kernel, Q, s, K, static_cast<int>(fp8::n_blocks(K)), r, Q_out, s_out);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

static PackArgs pack_args(const void* X, int x_dtype, int64_t T, int64_t K, int64_t ldx, const int32_t* place, int top_k,
                          uint8_t* Q, float* s) {
  const int64_t KB = fp8::n_blocks(K);
  return PackArgs{X, ldx, static_cast<uint32_t>(T * KB), static_cast<uint32_t>(KB), static_cast<uint32_t>(K),
                  aligned16(X) && (ldx * fp8::dtype_size(x_dtype)) % 16 == 0, place, top_k, T * top_k, Q, s};
}

int launch_pack_sorted(const void* X, int x_dtype, int64_t T, int64_t K, int64_t ldx, const int32_t* place, int top_k,
                       uint8_t* Q, float* s, cudaStream_t stream) {
  const PackArgs a = pack_args(X, x_dtype, T, K, ldx, place, top_k, Q, s);
  const uint32_t per = ROW_THREADS / 8;
  Launch l((a.n_qblocks + per - 1) / per, ROW_THREADS, 0, stream);
  const cudaError_t e = x_dtype == CONVROT_F32   ? cudaLaunchKernelEx(&l.cfg, moe_pack_kernel<float>, a)
                        : x_dtype == CONVROT_F16 ? cudaLaunchKernelEx(&l.cfg, moe_pack_kernel<__half>, a)
                                                 : cudaLaunchKernelEx(&l.cfg, moe_pack_kernel<__nv_bfloat16>, a);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}

template <typename T, int W>
static int plan_pack_as(const int32_t* experts, int64_t n, int E, int32_t* order, int32_t* place, int32_t* offsets,
                        const PackArgs& a, cudaStream_t stream) {
  const uint32_t plan_ctas = static_cast<uint32_t>((E + W) / W), per = PLAN_WARPS * 4;
  Launch l(plan_ctas + (a.n_qblocks + per - 1) / per, PLAN_WARPS * 32, 0, stream);
  const cudaError_t e =
      cudaLaunchKernelEx(&l.cfg, moe_plan_pack_kernel<T, W>, experts, n, E, order, place, offsets, plan_ctas, a);
  return e == cudaSuccess ? check_launch() : set_cuda_error(e);
}
template <typename T>
static int plan_pack_of(const int32_t* experts, int64_t n, int E, int32_t* order, int32_t* place, int32_t* offsets,
                        const PackArgs& a, cudaStream_t stream) {
  if (E < 152) return plan_pack_as<T, 1>(experts, n, E, order, place, offsets, a, stream);
  if (E < 304) return plan_pack_as<T, 2>(experts, n, E, order, place, offsets, a, stream);
  // (for 304 to 607 experts a plan of four per CTA takes 1.2 us less by itself;
  // three more instances)
  return plan_pack_as<T, 8>(experts, n, E, order, place, offsets, a, stream);
}

int launch_plan_pack(const int32_t* experts, int64_t n, int E, int32_t* order, int32_t* place, int32_t* offsets,
                     void* workspace, const void* X, int x_dtype, int64_t T, int64_t K, int64_t ldx, int top_k, uint8_t* Q,
                     float* s, cudaStream_t stream) {
  if (plan_parts(n) > 0) {
    if (int st = launch_plan(experts, n, E, order, place, offsets, workspace, stream)) return st;
    return fp8::launch_fp8_pack(X, x_dtype, T, K, ldx, Q, s, stream);
  }
  const PackArgs a = pack_args(X, x_dtype, T, K, ldx, nullptr, top_k, Q, s);
  if (x_dtype == CONVROT_F32) return plan_pack_of<float>(experts, n, E, order, place, offsets, a, stream);
  if (x_dtype == CONVROT_F16) return plan_pack_of<__half>(experts, n, E, order, place, offsets, a, stream);
  return plan_pack_of<__nv_bfloat16>(experts, n, E, order, place, offsets, a, stream);
}

int launch_combine(const CombineArgs& a, cudaStream_t stream) {
  if (a.r_dtype == CONVROT_F32) return combine_rows<float>(a, stream);
  if (a.r_dtype == CONVROT_F16) return combine_rows<__half>(a, stream);
  return combine_rows<__nv_bfloat16>(a, stream);
}

cudaError_t route_error_word(int** p) { return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_moe_error); }

}  // namespace moe
}  // namespace convrot
