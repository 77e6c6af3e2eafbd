// fp8_api.cu -- the extern "C" entry points of the block norms and the 8-bit
// floating-point linears: argument checks on the host, then launches on the
// caller's stream. None allocates device memory.
#include "fp8_checks.cuh"

#include <cmath>

using namespace convrot;
using namespace convrot::fp8;

namespace {

int pack_checks(const void* X, int dtype, int64_t M, int64_t K, int64_t ldx, const uint8_t* Q, const float* s,
                int64_t n_scales) {
  if (M < 0 || K <= 0 || !known_dtype(dtype) || ldx < K) return CONVROT_ERR_ARG;
  if (M == 0) return CONVROT_OK;
  if (!X || !Q || !s) return CONVROT_ERR_ARG;
  const int64_t size = static_cast<int64_t>(dtype_size(dtype));
  if (K % 16 != 0 || !aligned16(Q) || !aligned_to(X, size) || !aligned_to(s, 4)) return CONVROT_ERR_ALIGN;
  if (!sane(M, ldx) || K > MAX_LENGTH || n_scales > 0x7fffffff) return CONVROT_ERR_UNSUPPORTED;
  const Region x{X, M, K * size, ldx * size}, q = flat(Q, M * K), sc = flat(s, n_scales * 4);
  if (meet(x, q) || meet(x, sc) || meet(q, sc)) return CONVROT_ERR_ALIAS;
  return CONVROT_OK;
}

// Checks of the linears against each other and against the packed activation
// and one more input (fp8_linear's X).
int linear_checks(const uint8_t* Qx, const float* s_x, int64_t M, int64_t K, const convrot_fp8_weight* weights, int n,
                  int y_dtype, const Region& extra) {
  if (M < 0 || K <= 0 || n < 1 || n > CONVROT_MAX_LINEARS || !weights || !known_dtype(y_dtype)) return CONVROT_ERR_ARG;
  const int64_t size = static_cast<int64_t>(dtype_size(y_dtype));
  for (int j = 0; j < n; ++j) {
    const convrot_fp8_weight& w = weights[j];
    if (w.N < 0) return CONVROT_ERR_ARG;
    if (w.N == 0 || M == 0) continue;
    if (!w.q || !w.scale || !w.Y || w.ldy < w.N) return CONVROT_ERR_ARG;
    if (!aligned16(w.q) || !aligned_to(w.scale, 4) || !aligned_to(w.bias, 4) || !aligned_to(w.Y, size))
      return CONVROT_ERR_ALIGN;
    if (!sane(M, w.ldy) || w.N > MAX_ROWS) return CONVROT_ERR_UNSUPPORTED;
  }
  if (M == 0) return CONVROT_OK;
  if (!Qx || !s_x) return CONVROT_ERR_ARG;
  if (K % 16 != 0 || !aligned16(Qx) || !aligned_to(s_x, 4)) return CONVROT_ERR_ALIGN;
  if (M > MAX_ROWS || K > MAX_LENGTH || M * n_blocks(K) > 0x7fffffff) return CONVROT_ERR_UNSUPPORTED;
  const Region qx = flat(Qx, M * K), sx = flat(s_x, M * n_blocks(K) * 4);
  for (int j = 0; j < n; ++j) {
    if (weights[j].N == 0) continue;
    const Region y{weights[j].Y, M, weights[j].N * size, weights[j].ldy * size};
    if (meet(y, qx) || meet(y, sx) || meet(y, extra)) return CONVROT_ERR_ALIAS;
    for (int i = 0; i < n; ++i) {
      const convrot_fp8_weight& w = weights[i];
      if (w.N == 0) continue;
      if (meet(y, flat(w.q, w.N * K)) || meet(y, flat(w.scale, n_blocks(w.N) * n_blocks(K) * 4)) ||
          (w.bias && meet(y, flat(w.bias, w.N * 4))))
        return CONVROT_ERR_ALIAS;
      if (i > j && meet(y, Region{w.Y, M, w.N * size, w.ldy * size})) return CONVROT_ERR_ALIAS;
    }
  }
  return CONVROT_OK;
}

// The linears that have outputs, to `w`; their number.
int with_output(const convrot_fp8_weight* weights, int n, convrot_fp8_weight (&w)[CONVROT_MAX_LINEARS]) {
  int k = 0;
  for (int j = 0; j < n; ++j)
    if (weights[j].N > 0) w[k++] = weights[j];
  return k;
}

int norm_checks(const convrot_block_norm_args& a) {
  if (a.M < 0 || a.K <= 0 || !known_dtype(a.dtype)) return CONVROT_ERR_ARG;
  for (int kind : {a.post_norm, a.pre_norm})
    if (kind != CONVROT_NORM_NONE && kind != CONVROT_NORM_RMS && kind != CONVROT_NORM_LAYER) return CONVROT_ERR_ARG;
  for (float v : {a.residual_scale, a.block_scale, a.post_eps, a.pre_eps})
    if (!std::isfinite(v)) return CONVROT_ERR_ARG;
  if (a.post_eps < 0.0f || a.pre_eps < 0.0f) return CONVROT_ERR_ARG;
  if (a.M == 0) return CONVROT_OK;
  if (!a.H || (!a.H_out && !a.U && !a.Q) || (a.U && a.Q) || (a.Q && !a.s)) return CONVROT_ERR_ARG;
  if (a.U && !known_dtype(a.u_dtype)) return CONVROT_ERR_ARG;
  if (a.ldh < a.K || (a.Y && a.ldy < a.K) || (a.H_out && a.ldho < a.K) || (a.U && a.ldu < a.K)) return CONVROT_ERR_ARG;
  const bool sampled = a.gate || a.scale || a.shift;
  if (a.gate && !a.Y) return CONVROT_ERR_ARG;
  if (sampled) {
    if (a.n_samples < 1 || a.rows_per_sample < 0) return CONVROT_ERR_ARG;
    if ((a.gate && a.ld_gate < a.K && a.n_samples > 1) ||
        ((a.scale || a.shift) && a.ld_mod < a.K && a.n_samples > 1))
      return CONVROT_ERR_ARG;
    if (!a.row_sample && a.rows_per_sample > 0 && (a.M - 1) / a.rows_per_sample >= a.n_samples) return CONVROT_ERR_ARG;
  }
  const int64_t size = static_cast<int64_t>(dtype_size(a.dtype)), usize = static_cast<int64_t>(dtype_size(a.u_dtype));
  if (!aligned_to(a.H, size) || !aligned_to(a.Y, size) || !aligned_to(a.H_out, size) || (a.U && !aligned_to(a.U, usize)))
    return CONVROT_ERR_ALIGN;
  for (const void* v : {static_cast<const void*>(a.post_weight), static_cast<const void*>(a.post_bias),
                        static_cast<const void*>(a.pre_weight), static_cast<const void*>(a.pre_bias),
                        static_cast<const void*>(a.gate), static_cast<const void*>(a.scale),
                        static_cast<const void*>(a.shift), static_cast<const void*>(a.row_sample)})
    if (!aligned_to(v, 4)) return CONVROT_ERR_ALIGN;
  if (a.Q && (a.K % 16 != 0 || !aligned16(a.Q) || !aligned_to(a.s, 4))) return CONVROT_ERR_ALIGN;
  if (a.K > CONVROT_NORM_MAX_K || !sane(a.M, a.ldh) || (a.Y && !sane(a.M, a.ldy)) || (a.H_out && !sane(a.M, a.ldho)) ||
      (a.U && !sane(a.M, a.ldu)) || (sampled && (!sane(a.n_samples, a.ld_gate) || !sane(a.n_samples, a.ld_mod))))
    return CONVROT_ERR_UNSUPPORTED;
  const int64_t kb = a.K * 4;
  const Region in[] = {
      {a.H, a.M, a.K * size, a.ldh * size},
      {a.Y, a.M, a.K * size, a.ldy * size},
      flat(a.post_weight, kb),
      flat(a.post_bias, kb),
      flat(a.pre_weight, kb),
      flat(a.pre_bias, kb),
      {a.gate, a.n_samples, kb, a.ld_gate * 4},
      {a.scale, a.n_samples, kb, a.ld_mod * 4},
      {a.shift, a.n_samples, kb, a.ld_mod * 4},
      flat(a.row_sample, a.M * 4),
  };
  const Region out[] = {
      {a.H_out, a.M, a.K * size, a.ldho * size},
      {a.U, a.M, a.K * usize, a.ldu * usize},
      flat(a.Q, a.M * a.K),
      flat(a.Q ? a.s : nullptr, a.M * n_blocks(a.K) * 4),
  };
  for (int i = 0; i < 4; ++i) {
    for (const Region& r : in) {
      const bool in_place = i == 0 && r.p == a.H && &r == &in[0] && a.H_out == a.H && a.ldho == a.ldh;
      if (!in_place && meet(out[i], r)) return CONVROT_ERR_ALIAS;
    }
    for (int k = i + 1; k < 4; ++k)
      if (meet(out[i], out[k])) return CONVROT_ERR_ALIAS;
  }
  return CONVROT_OK;
}

int linear_packed(const uint8_t* Q_x, const float* s_x, int64_t M, int64_t K, const convrot_fp8_weight* weights,
                  int n_weights, int y_dtype, uint64_t test_wait_ns, void* stream) {
  if (int st = linear_checks(Q_x, s_x, M, K, weights, n_weights, y_dtype, flat(nullptr, 0))) return st;
  convrot_fp8_weight w[CONVROT_MAX_LINEARS];
  const int n = with_output(weights, n_weights, w);
  if (M == 0 || n == 0) return CONVROT_OK;
  if (int st = check_device()) return st;
  return launch_fp8_gemm(Q_x, s_x, M, K, w, n, y_dtype, static_cast<cudaStream_t>(stream), test_wait_ns);
}

int launch_norm(const convrot_block_norm_args& a, void* stream, NormTimeoutTest test) {
  if (int st = check_device()) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.dtype == CONVROT_F32) return launch_block_norm_as<float>(a, s, test);
  if (a.dtype == CONVROT_F16) return launch_block_norm_as<__half>(a, s, test);
  return launch_block_norm_as<__nv_bfloat16>(a, s, test);
}

}  // namespace

extern "C" {

int convrot_block_norm(const convrot_block_norm_args* args, void* stream) {
  if (!args) return CONVROT_ERR_ARG;
  if (int st = norm_checks(*args)) return st;
  if (args->M == 0) return CONVROT_OK;
  return launch_norm(*args, stream, NormTimeoutTest());
}

int convrot_test_block_norm_timeout(const convrot_block_norm_args* args, int64_t row, uint64_t wait_ns, void* stream) {
  if (!args || wait_ns == 0) return CONVROT_ERR_ARG;
  if (int st = norm_checks(*args)) return st;
  if (row < 0 || row >= args->M) return CONVROT_ERR_ARG;
  return launch_norm(*args, stream, NormTimeoutTest{wait_ns, row});
}

int fp8_pack_activations(const void* X, int x_dtype, int64_t M, int64_t K, int64_t ldx, uint8_t* Q_x, float* s_x,
                         void* stream) {
  if (M > MAX_ROWS) return CONVROT_ERR_UNSUPPORTED;
  if (int st = pack_checks(X, x_dtype, M, K, ldx, Q_x, s_x, M * n_blocks(K))) return st;
  if (M == 0) return CONVROT_OK;
  if (int st = check_device()) return st;
  return launch_fp8_pack(X, x_dtype, M, K, ldx, Q_x, s_x, static_cast<cudaStream_t>(stream));
}

int fp8_prepare_weight(const void* W, int w_dtype, int64_t N, int64_t K, uint8_t* Q_w, float* s_w, void* stream) {
  if (N > MAX_ROWS) return CONVROT_ERR_UNSUPPORTED;
  if (int st = pack_checks(W, w_dtype, N, K, K, Q_w, s_w, n_blocks(N) * n_blocks(K))) return st;
  if (N == 0) return CONVROT_OK;
  if (int st = check_device()) return st;
  return launch_fp8_weight(W, w_dtype, N, K, Q_w, s_w, static_cast<cudaStream_t>(stream));
}

size_t fp8_linear_workspace_size(int64_t M, int64_t K) {
  if (M < 0 || K <= 0 || M > MAX_ROWS || K > MAX_LENGTH) return 0;
  return round256(static_cast<size_t>(M) * K) + round256(static_cast<size_t>(M) * n_blocks(K) * 4);
}

int fp8_linear_packed(const uint8_t* Q_x, const float* s_x, int64_t M, int64_t K, const convrot_fp8_weight* weights,
                      int n_weights, int y_dtype, void* stream) {
  return linear_packed(Q_x, s_x, M, K, weights, n_weights, y_dtype, 0, stream);
}

int fp8_test_linear_timeout(const uint8_t* Q_x, const float* s_x, int64_t M, int64_t K,
                            const convrot_fp8_weight* weights, int n_weights, int y_dtype, uint64_t wait_ns,
                            void* stream) {
  if (wait_ns == 0) return CONVROT_ERR_ARG;
  return linear_packed(Q_x, s_x, M, K, weights, n_weights, y_dtype, wait_ns, stream);
}

int fp8_linear(const void* X, int x_dtype, int64_t M, int64_t K, int64_t ldx, const convrot_fp8_weight* weights,
               int n_weights, int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (M < 0 || K <= 0 || !known_dtype(x_dtype) || ldx < K || !weights || n_weights < 1 ||
      n_weights > CONVROT_MAX_LINEARS || !known_dtype(y_dtype))
    return CONVROT_ERR_ARG;
  if (M > MAX_ROWS || K > MAX_LENGTH) return CONVROT_ERR_UNSUPPORTED;
  const size_t need = fp8_linear_workspace_size(M, K);
  uint8_t* q = static_cast<uint8_t*>(workspace);
  if (M > 0) {
    if (!workspace || workspace_bytes < need) return CONVROT_ERR_WORKSPACE;
    if (!aligned16(workspace)) return CONVROT_ERR_ALIGN;
  }
  float* s = reinterpret_cast<float*>(q + round256(static_cast<size_t>(M) * K));
  if (int st = pack_checks(X, x_dtype, M, K, ldx, q, s, M * n_blocks(K))) return st;
  const int64_t size = static_cast<int64_t>(dtype_size(x_dtype));
  if (int st = linear_checks(q, s, M, K, weights, n_weights, y_dtype, Region{X, M, K * size, ldx * size})) return st;
  convrot_fp8_weight lin[CONVROT_MAX_LINEARS];
  const int n = with_output(weights, n_weights, lin);
  if (M == 0 || n == 0) return CONVROT_OK;
  const Region ws = flat(workspace, static_cast<int64_t>(need));
  for (int j = 0; j < n_weights; ++j) {
    const convrot_fp8_weight& w = weights[j];
    if (w.N > 0 && (meet(ws, flat(w.q, w.N * K)) || meet(ws, flat(w.scale, n_blocks(w.N) * n_blocks(K) * 4)) ||
                    (w.bias && meet(ws, flat(w.bias, w.N * 4)))))
      return CONVROT_ERR_ALIAS;
  }
  if (int st = check_device()) return st;
  const cudaStream_t str = static_cast<cudaStream_t>(stream);
  bool launched = false;
  if (int st = launch_fp8_packing(X, x_dtype, M, K, ldx, lin, n, y_dtype, str, &launched)) return st;
  if (launched) return CONVROT_OK;
  if (int st = launch_fp8_pack(X, x_dtype, M, K, ldx, q, s, str)) return st;
  return launch_fp8_gemm(q, s, M, K, lin, n, y_dtype, str);
}

}  // extern "C"
