// moe_api.cu -- the extern "C" entry points of the experts' operators: argument
// checks on the host, then launches on the caller's stream. None allocates
// device memory.
#include "fp8_checks.cuh"
#include "moe_common.cuh"

#include <cmath>

using namespace convrot;
using namespace convrot::fp8;
using namespace convrot::moe;

namespace {

bool top_k_in_range(int top_k) { return top_k >= 1 && top_k <= MAX_TOP_K; }
int64_t size_of(int dtype) { return static_cast<int64_t>(dtype_size(dtype)); }

int route_checks(const convrot_moe_route_args& a) {
  if (a.T < 0 || a.n_experts < 1 || a.top_k < 1 || !known_dtype(a.dtype) || !std::isfinite(a.scale)) return CONVROT_ERR_ARG;
  if (a.score != CONVROT_MOE_SOFTMAX && a.score != CONVROT_MOE_SIGMOID) return CONVROT_ERR_ARG;
  if (a.n_groups < 1 || a.n_experts % a.n_groups != 0 || a.top_groups < 1 || a.top_groups > a.n_groups ||
      a.group_top < 1 || a.group_top > 2 ||
      a.top_k > static_cast<int64_t>(a.top_groups) * (a.n_experts / a.n_groups) || a.ld < a.n_experts)
    return CONVROT_ERR_ARG;
  if (a.n_experts > MAX_EXPERTS || !top_k_in_range(a.top_k) || a.n_groups > CONVROT_MOE_MAX_GROUPS) return CONVROT_ERR_UNSUPPORTED;
  if (a.T == 0) return CONVROT_OK;
  if (!a.logits || !a.experts || !a.weights) return CONVROT_ERR_ARG;
  const int64_t size = size_of(a.dtype);
  if (!aligned_to(a.logits, size) || !aligned_to(a.bias, 4) || !aligned_to(a.experts, 4) || !aligned_to(a.weights, 4))
    return CONVROT_ERR_ALIGN;
  if (!sane(a.T, a.ld) || a.T * a.top_k > MAX_ROWS) return CONVROT_ERR_UNSUPPORTED;
  const Region in[] = {{a.logits, a.T, a.n_experts * size, a.ld * size}, flat(a.bias, a.n_experts * 4)};
  const Region e = flat(a.experts, a.T * a.top_k * 4), w = flat(a.weights, a.T * a.top_k * 4);
  for (const Region& r : in)
    if (meet(r, e) || meet(r, w)) return CONVROT_ERR_ALIAS;
  return meet(e, w) ? CONVROT_ERR_ALIAS : CONVROT_OK;
}

// What a set of experts' matrices [N,K] spans.
struct Spans {
  Region q, scale, bias;
};
Spans spans(const convrot_experts& w, int64_t E, int64_t K) {
  const int64_t sc = n_blocks(w.N) * n_blocks(K) * 4;
  return Spans{{w.q, E, w.N * K, w.q_stride}, {w.scale, E, sc, w.scale_stride * 4}, {w.bias, E, w.N * 4, w.bias_stride * 4}};
}
bool meets(const Region& out, const Spans& s) { return meet(out, s.q) || meet(out, s.scale) || meet(out, s.bias); }

// The parts of a set of experts' matrices; N > 0.
int experts_checks(const convrot_experts& w, int64_t E, int64_t K) {
  const int64_t sc = n_blocks(w.N) * n_blocks(K);
  if (!w.q || !w.scale) return CONVROT_ERR_ARG;
  if (w.N > MAX_ROWS || K > MAX_LENGTH || n_blocks(w.N) > 0x7fffffff / n_blocks(K)) return CONVROT_ERR_UNSUPPORTED;
  if (E > 1 && (w.q_stride < w.N * K || w.scale_stride < sc || (w.bias && w.bias_stride < w.N))) return CONVROT_ERR_ARG;
  if (!aligned16(w.q) || (E > 1 && w.q_stride % 16 != 0) || !aligned_to(w.scale, 4) || !aligned_to(w.bias, 4))
    return CONVROT_ERR_ALIGN;
  if (E > 1 && (w.q_stride > (1ll << 38) || w.scale_stride > (1ll << 38) || (w.bias && w.bias_stride > (1ll << 38))))
    return CONVROT_ERR_UNSUPPORTED;
  return CONVROT_OK;
}

// What the two expert linears have in common, but for their outputs.
int expert_checks(const uint8_t* Q_x, const float* s_x, int64_t T, int64_t K, const int32_t* order,
                  const int32_t* offsets, int64_t n, int E, int top_k, const convrot_experts* w) {
  if (T < 0 || n < 0 || K <= 0 || E < 1 || top_k < 1 || !w || w->N < 0) return CONVROT_ERR_ARG;
  // n choices are of rows up to (n - 1) / top_k
  if (n > 0 && T <= (n - 1) / (order ? top_k : 1)) return CONVROT_ERR_ARG;
  if (E > MAX_EXPERTS) return CONVROT_ERR_UNSUPPORTED;
  if (n == 0 || w->N == 0) return CONVROT_OK;
  if (!Q_x || !s_x || !offsets) return CONVROT_ERR_ARG;
  if (K % 16 != 0 || !aligned16(Q_x) || !aligned_to(s_x, 4) || !aligned_to(order, 4) || !aligned_to(offsets, 4))
    return CONVROT_ERR_ALIGN;
  if (T > MAX_ROWS || n > MAX_ROWS || K > MAX_LENGTH || T > 0x7fffffff / n_blocks(K)) return CONVROT_ERR_UNSUPPORTED;
  return experts_checks(*w, E, K);
}

bool meets_inputs(const Region& out, const uint8_t* Q_x, const float* s_x, int64_t T, int64_t K, const int32_t* order,
                  const int32_t* offsets, int64_t n, int E) {
  return meet(out, flat(Q_x, T * K)) || meet(out, flat(s_x, T * n_blocks(K) * 4)) || meet(out, flat(order, n * 4)) ||
         meet(out, flat(offsets, (E + 1) * 4));
}

size_t sorted_bytes(int64_t n, int64_t K) {
  return round256(static_cast<size_t>(n) * K) + round256(static_cast<size_t>(n) * n_blocks(K) * 4);
}
// Where the linear wants its rows in the plan's order and they come by token,
// they are sorted into the workspace first: its checks (ws: the part in use) ...
int workspace_checks(void* workspace, size_t bytes, const uint8_t* Q_x, const float* s_x, int64_t T, int64_t K,
                     const int32_t* order, const int32_t* offsets, int64_t n, int E, Region& ws) {
  ws = flat(nullptr, 0);
  if (!order || !many_rows(n, E)) return CONVROT_OK;
  if (!workspace || bytes < sorted_bytes(n, K)) return CONVROT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return CONVROT_ERR_ALIGN;
  if (n > 0x7fffffff / n_blocks(K)) return CONVROT_ERR_UNSUPPORTED;
  ws = flat(workspace, static_cast<int64_t>(sorted_bytes(n, K)));
  return meets_inputs(ws, Q_x, s_x, T, K, order, offsets, n, E) ? CONVROT_ERR_ALIAS : CONVROT_OK;
}
// ... and the sort; Q_x, s_x and rows are the sorted ones from then on.
int sort_rows(const uint8_t*& Q_x, const float*& s_x, int64_t K, Rows& rows, const Region& ws, cudaStream_t stream) {
  if (!ws.p) return CONVROT_OK;
  uint8_t* q = static_cast<uint8_t*>(const_cast<void*>(ws.p));
  float* s = reinterpret_cast<float*>(q + round256(static_cast<size_t>(rows.n) * K));
  if (int st = launch_gather(Q_x, s_x, K, rows, q, s, stream)) return st;
  Q_x = q;
  s_x = s;
  rows = Rows{nullptr, rows.offsets, rows.n, rows.n, rows.E, 1};
  return CONVROT_OK;
}

int combine_checks(const CombineArgs& a) {
  if (a.T < 0 || a.n < 0 || a.N < 0 || a.top_k < 1 || !known_dtype(a.r_dtype) || !known_dtype(a.y_dtype) ||
      a.ldr < a.N || a.ldy < a.N || (a.residual && a.ld_res < a.N))
    return CONVROT_ERR_ARG;
  if (a.top_k > MAX_TOP_K) return CONVROT_ERR_UNSUPPORTED;
  if (a.T == 0 || a.N == 0) return CONVROT_OK;
  if (!a.place || !a.weights || !a.Y || (a.n > 0 && !a.rows)) return CONVROT_ERR_ARG;
  const int64_t rs = size_of(a.r_dtype), ys = size_of(a.y_dtype);
  if (!aligned_to(a.rows, rs) || !aligned_to(a.place, 4) || !aligned_to(a.weights, 4) || !aligned_to(a.residual, ys) ||
      !aligned_to(a.Y, ys))
    return CONVROT_ERR_ALIGN;
  if (!sane(a.n, a.ldr) || !sane(a.T, a.ldy) || (a.residual && !sane(a.T, a.ld_res)) || a.N > MAX_ROWS)
    return CONVROT_ERR_UNSUPPORTED;
  const Region y{a.Y, a.T, a.N * ys, a.ldy * ys};
  const bool in_place = a.residual == a.Y && a.ld_res == a.ldy;
  if (meet(y, Region{a.rows, a.n, a.N * rs, a.ldr * rs}) || meet(y, flat(a.place, a.T * a.top_k * 4)) ||
      meet(y, flat(a.weights, a.T * a.top_k * 4)) ||
      (!in_place && meet(y, Region{a.residual, a.T, a.N * ys, a.ld_res * ys})))
    return CONVROT_ERR_ALIAS;
  return CONVROT_OK;
}

// Where fp8_moe keeps what passes between its steps.
struct Workspace {
  size_t q_x, s_x, order, place, offsets, plan, q_h, s_h, rows, powers, bytes;
  int64_t ld;  // of the rows, elements
  Workspace(int64_t T, int64_t K, int64_t I, int64_t N, int64_t n, int E, int y_dtype) {
    size_t at = 0;
    auto take = [&](size_t b) {
      const size_t here = at;
      at += round256(b);
      return here;
    };
    const size_t m = static_cast<size_t>(many_rows(n, E) ? n : T);  // rows sorted by expert, or tokens
    q_x = take(m * K);
    s_x = take(m * n_blocks(K) * 4);
    order = take(static_cast<size_t>(n) * 4);
    place = take(static_cast<size_t>(n) * 4);
    offsets = take(static_cast<size_t>(E + 1) * 4);
    plan = take(plan_workspace(n, E));
    q_h = take(static_cast<size_t>(n) * I);
    s_h = take(static_cast<size_t>(n) * n_blocks(I) * 4);
    // rows that start on 16-byte boundaries: fp32, or binary16 with their powers of two
    const bool half = y_dtype == CONVROT_BF16;
    ld = half ? (N + 7) / 8 * 8 : (N + 3) / 4 * 4;
    rows = take(static_cast<size_t>(n) * ld * (half ? 2 : 4));
    powers = take(half ? static_cast<size_t>(n) * n_blocks(N) * 4 : 0);
    bytes = at;
  }
};
bool workspace_sizes(int64_t T, int64_t K, int64_t I, int64_t N, int top_k, int E, int y_dtype) {
  return T >= 0 && K > 0 && I > 0 && N >= 0 && top_k_in_range(top_k) && E >= 1 && E <= MAX_EXPERTS &&
         known_dtype(y_dtype) && T <= MAX_ROWS / top_k && K <= MAX_LENGTH && I <= MAX_LENGTH && N <= MAX_ROWS;
}

int moe_checks(const convrot_moe_args& a, void* workspace, size_t workspace_bytes) {
  if (a.T < 0 || a.K <= 0 || !known_dtype(a.x_dtype) || !known_dtype(a.y_dtype) || a.ldx < a.K || a.top_k < 1 ||
      a.n_experts < 1 || !a.gate || !a.up || !a.down)
    return CONVROT_ERR_ARG;
  const int64_t I = a.gate->N, N = a.down->N;
  if (I <= 0 || a.up->N != I || N < 0 || a.ldy < N || (a.residual && a.ld_res < N)) return CONVROT_ERR_ARG;
  if (!workspace_sizes(a.T, a.K, I, N, a.top_k, a.n_experts, a.y_dtype)) return CONVROT_ERR_UNSUPPORTED;
  if (a.T == 0 || N == 0) return CONVROT_OK;
  const int64_t n = a.T * a.top_k, xs = size_of(a.x_dtype), ys = size_of(a.y_dtype);
  if (!a.X || !a.experts || !a.weights || !a.Y) return CONVROT_ERR_ARG;
  const Workspace ws(a.T, a.K, I, N, n, a.n_experts, a.y_dtype);
  if (!workspace || workspace_bytes < ws.bytes) return CONVROT_ERR_WORKSPACE;
  if (a.K % 16 != 0 || I % 16 != 0 || !aligned16(workspace) || !aligned_to(a.X, xs) || !aligned_to(a.experts, 4) ||
      !aligned_to(a.weights, 4) || !aligned_to(a.Y, ys) || !aligned_to(a.residual, ys))
    return CONVROT_ERR_ALIGN;
  for (const auto& [w, K] : {std::pair{a.gate, a.K}, std::pair{a.up, a.K}, std::pair{a.down, I}})
    if (int st = experts_checks(*w, a.n_experts, K)) return st;
  if (!sane(a.T, a.ldx) || !sane(a.T, a.ldy) || (a.residual && !sane(a.T, a.ld_res)) ||
      n > 0x7fffffff / n_blocks(a.K) || n > 0x7fffffff / n_blocks(I))
    return CONVROT_ERR_UNSUPPORTED;
  const Region y{a.Y, a.T, N * ys, a.ldy * ys}, work = flat(workspace, static_cast<int64_t>(ws.bytes));
  const Region in[] = {{a.X, a.T, a.K * xs, a.ldx * xs}, flat(a.experts, n * 4), flat(a.weights, n * 4)};
  const Region res{a.residual, a.T, N * ys, a.ld_res * ys};
  const Spans sets[] = {spans(*a.gate, a.n_experts, a.K), spans(*a.up, a.n_experts, a.K), spans(*a.down, a.n_experts, I)};
  if (meet(y, work) || meet(res, work)) return CONVROT_ERR_ALIAS;
  if (!(a.residual == a.Y && a.ld_res == a.ldy) && meet(y, res)) return CONVROT_ERR_ALIAS;
  for (const Region& r : in)
    if (meet(y, r) || meet(work, r)) return CONVROT_ERR_ALIAS;
  for (const Spans& s : sets)
    if (meets(y, s) || meets(work, s)) return CONVROT_ERR_ALIAS;
  return CONVROT_OK;
}

}  // namespace

extern "C" {

int moe_route(const convrot_moe_route_args* args, void* stream) {
  if (!args) return CONVROT_ERR_ARG;
  if (int st = route_checks(*args)) return st;
  if (args->T == 0) return CONVROT_OK;
  if (int st = check_device()) return st;
  return launch_route(*args, static_cast<cudaStream_t>(stream));
}

int moe_plan(const int32_t* experts, int64_t n, int n_experts, int32_t* order, int32_t* place, int32_t* offsets,
             void* workspace, size_t workspace_bytes, void* stream) {
  if (n < 0 || n_experts < 1) return CONVROT_ERR_ARG;
  if (n_experts > MAX_EXPERTS || n > MAX_ROWS) return CONVROT_ERR_UNSUPPORTED;
  if (!offsets || (n > 0 && (!experts || !order || !place))) return CONVROT_ERR_ARG;
  const size_t need = plan_workspace(n, n_experts);
  if (need && (!workspace || workspace_bytes < need)) return CONVROT_ERR_WORKSPACE;
  const Region arrays[] = {flat(experts, n * 4), flat(order, n * 4), flat(place, n * 4),
                           flat(offsets, (n_experts + 1) * 4), flat(need ? workspace : nullptr, static_cast<int64_t>(need))};
  for (int i = 0; i < 5; ++i) {
    if (!aligned_to(arrays[i].p, 4)) return CONVROT_ERR_ALIGN;
    for (int j = 0; j < i; ++j)
      if (meet(arrays[i], arrays[j])) return CONVROT_ERR_ALIAS;
  }
  if (int st = check_device()) return st;
  return launch_plan(experts, n, n_experts, order, place, offsets, workspace, static_cast<cudaStream_t>(stream));
}

int fp8_expert_linear(const uint8_t* Q_x, const float* s_x, int64_t T, int64_t K, const int32_t* order,
                      const int32_t* offsets, int64_t n, int n_experts, int top_k, const convrot_experts* weight, void* Y,
                      int64_t ldy, int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!known_dtype(y_dtype)) return CONVROT_ERR_ARG;
  if (int st = expert_checks(Q_x, s_x, T, K, order, offsets, n, n_experts, top_k, weight)) return st;
  if (n == 0 || weight->N == 0) return CONVROT_OK;
  if (!Y || ldy < weight->N) return CONVROT_ERR_ARG;
  const int64_t size = size_of(y_dtype);
  if (!aligned_to(Y, size)) return CONVROT_ERR_ALIGN;
  if (!sane(n, ldy)) return CONVROT_ERR_UNSUPPORTED;
  const Region y{Y, n, weight->N * size, ldy * size};
  if (meets_inputs(y, Q_x, s_x, T, K, order, offsets, n, n_experts) || meets(y, spans(*weight, n_experts, K)))
    return CONVROT_ERR_ALIAS;
  Region ws;
  if (int st = workspace_checks(workspace, workspace_bytes, Q_x, s_x, T, K, order, offsets, n, n_experts, ws)) return st;
  if (meet(ws, y) || meets(ws, spans(*weight, n_experts, K))) return CONVROT_ERR_ALIAS;
  if (int st = check_device()) return st;
  Rows rows{order, offsets, n, T, n_experts, top_k};
  if (int st = sort_rows(Q_x, s_x, K, rows, ws, static_cast<cudaStream_t>(stream))) return st;
  return launch_expert_linear(Q_x, s_x, K, rows, *weight, Y, ldy, y_dtype, nullptr,
                              static_cast<cudaStream_t>(stream));
}

int fp8_expert_swiglu(const uint8_t* Q_x, const float* s_x, int64_t T, int64_t K, const int32_t* order,
                      const int32_t* offsets, int64_t n, int n_experts, int top_k, const convrot_experts* gate,
                      const convrot_experts* up, uint8_t* Q_h, float* s_h, void* workspace, size_t workspace_bytes,
                      void* stream) {
  for (const convrot_experts* w : {gate, up})
    if (int st = expert_checks(Q_x, s_x, T, K, order, offsets, n, n_experts, top_k, w)) return st;
  const int64_t N = gate->N;
  if (up->N != N) return CONVROT_ERR_ARG;
  if (n == 0 || N == 0) return CONVROT_OK;
  if (!Q_h || !s_h) return CONVROT_ERR_ARG;
  if (N % 16 != 0 || !aligned16(Q_h) || !aligned_to(s_h, 4)) return CONVROT_ERR_ALIGN;
  if (n > 0x7fffffff / n_blocks(N)) return CONVROT_ERR_UNSUPPORTED;
  const Region q = flat(Q_h, n * N), s = flat(s_h, n * n_blocks(N) * 4);
  if (meet(q, s)) return CONVROT_ERR_ALIAS;
  for (const Region& out : {q, s}) {
    if (meets_inputs(out, Q_x, s_x, T, K, order, offsets, n, n_experts)) return CONVROT_ERR_ALIAS;
    if (meets(out, spans(*gate, n_experts, K)) || meets(out, spans(*up, n_experts, K))) return CONVROT_ERR_ALIAS;
  }
  Region ws;
  if (int st = workspace_checks(workspace, workspace_bytes, Q_x, s_x, T, K, order, offsets, n, n_experts, ws)) return st;
  if (meet(ws, q) || meet(ws, s) || meets(ws, spans(*gate, n_experts, K)) || meets(ws, spans(*up, n_experts, K)))
    return CONVROT_ERR_ALIAS;
  if (int st = check_device()) return st;
  Rows rows{order, offsets, n, T, n_experts, top_k};
  if (int st = sort_rows(Q_x, s_x, K, rows, ws, static_cast<cudaStream_t>(stream))) return st;
  return launch_expert_swiglu(Q_x, s_x, K, rows, *gate, *up, Q_h, s_h, static_cast<cudaStream_t>(stream));
}

int fp8_test_expert_timeout(const uint8_t* Q_x, const float* s_x, int64_t n, int64_t K, const int32_t* offsets,
                            int n_experts, const convrot_experts* weight, const convrot_experts* up, void* out,
                            float* s_out, int64_t ld, int y_dtype, uint64_t wait_ns, void* stream) {
  if (wait_ns == 0 || n < 1 || !weight || !out || !known_dtype(y_dtype) || ld < weight->N || weight->N < 1 ||
      (up && (up->N != weight->N || !s_out)))
    return CONVROT_ERR_ARG;
  if (up && (ld != weight->N || ld % 16 != 0 || !aligned16(out))) return CONVROT_ERR_ALIGN;
  for (const convrot_experts* w : {weight, up})
    if (w)
      if (int st = expert_checks(Q_x, s_x, n, K, nullptr, offsets, n, n_experts, 1, w)) return st;
  if (int st = check_device()) return st;
  const Rows rows{nullptr, offsets, n, n, n_experts, 1};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (up) return launch_expert_swiglu(Q_x, s_x, K, rows, *weight, *up, static_cast<uint8_t*>(out), s_out, s, wait_ns);
  return launch_expert_linear(Q_x, s_x, K, rows, *weight, out, ld, y_dtype, nullptr, s, wait_ns);
}

int moe_combine(const void* rows, int r_dtype, int64_t ldr, int64_t n, const int32_t* place, const float* weights,
                int64_t T, int top_k, int64_t N, const void* residual, int64_t ld_res, void* Y, int64_t ldy,
                int y_dtype, void* stream) {
  const CombineArgs a{rows, r_dtype, ldr, n, place, weights, T, top_k, N, residual, ld_res, Y, ldy, y_dtype,
                      nullptr, 0};
  if (int st = combine_checks(a)) return st;
  if (T == 0 || N == 0) return CONVROT_OK;
  if (int st = check_device()) return st;
  return launch_combine(a, static_cast<cudaStream_t>(stream));
}

size_t moe_plan_workspace_size(int64_t n, int n_experts) {
  if (n < 0 || n > MAX_ROWS || n_experts < 1 || n_experts > MAX_EXPERTS) return 0;
  return plan_workspace(n, n_experts);
}

size_t fp8_expert_workspace_size(int64_t n, int64_t K, int n_experts) {
  if (n < 0 || K <= 0 || n > MAX_ROWS || K > MAX_LENGTH || n_experts < 1 || n_experts > MAX_EXPERTS) return 0;
  return many_rows(n, n_experts) ? sorted_bytes(n, K) : 0;
}

size_t fp8_moe_workspace_size(int64_t T, int64_t K, int64_t I, int64_t N, int top_k, int n_experts, int y_dtype) {
  if (!workspace_sizes(T, K, I, N, top_k, n_experts, y_dtype)) return 0;
  return Workspace(T, K, I, N, T * top_k, n_experts, y_dtype).bytes;
}

int fp8_moe(const convrot_moe_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  if (!args) return CONVROT_ERR_ARG;
  const convrot_moe_args& a = *args;
  if (int st = moe_checks(a, workspace, workspace_bytes)) return st;
  const int64_t I = a.gate->N, N = a.down->N, n = a.T * a.top_k;
  if (a.T == 0 || N == 0) return CONVROT_OK;
  if (int st = check_device()) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Workspace at(a.T, a.K, I, N, n, a.n_experts, a.y_dtype);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t *q_x = ws + at.q_x, *q_h = ws + at.q_h;
  float *s_x = reinterpret_cast<float*>(ws + at.s_x), *s_h = reinterpret_cast<float*>(ws + at.s_h);
  int32_t *order = reinterpret_cast<int32_t*>(ws + at.order), *place = reinterpret_cast<int32_t*>(ws + at.place);
  int32_t* offsets = reinterpret_cast<int32_t*>(ws + at.offsets);
  const Rows by_token{order, offsets, n, a.T, a.n_experts, a.top_k}, sorted{nullptr, offsets, n, n, a.n_experts, 1};
  const bool many = many_rows(n, a.n_experts);
  if (many) {
    if (int st = launch_plan(a.experts, n, a.n_experts, order, place, offsets, ws + at.plan, s)) return st;
    if (int st = launch_pack_sorted(a.X, a.x_dtype, a.T, a.K, a.ldx, place, a.top_k, q_x, s_x, s)) return st;
  } else if (int st = launch_plan_pack(a.experts, n, a.n_experts, order, place, offsets, ws + at.plan, a.X, a.x_dtype, a.T,
                                       a.K, a.ldx, a.top_k, q_x, s_x, s)) {
    return st;
  }
  if (int st = launch_expert_swiglu(q_x, s_x, a.K, many ? sorted : by_token, *a.gate, *a.up, q_h, s_h, s)) return st;
  const bool half = a.y_dtype == CONVROT_BF16;
  float* powers = half ? reinterpret_cast<float*>(ws + at.powers) : nullptr;
  const int rows = half ? CONVROT_F16 : CONVROT_F32;
  if (int st = launch_expert_linear(q_h, s_h, I, sorted, *a.down, ws + at.rows, at.ld, rows, powers, s)) return st;
  return launch_combine(CombineArgs{ws + at.rows, rows, at.ld, n, place, a.weights, a.T, a.top_k, N, a.residual,
                                    a.ld_res, a.Y, a.ldy, a.y_dtype, powers, n_blocks(N)}, s);
}

}  // extern "C"
