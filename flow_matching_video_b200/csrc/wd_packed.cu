// wd_packed.cu — the extern "C" entry points of the packed-batch operators:
// argument validation and the kernels' parameter structs.
#include "wd_internal.cuh"

namespace wd {

constexpr int64_t MAX_ROWS = int64_t(1) << 30;

// A row stride of `rs` elements for rows `width` wide: 16-byte steps, no overlap.
static wd_status check_stride(const char* what, int64_t rs, int64_t width) {
  if (rs < width || rs > (int64_t(1) << 36)) {
    set_error("%s: row stride %lld for rows of %lld", what, (long long)rs, (long long)width);
    return WD_ERR_SHAPE;
  }
  if (rs % 8) { set_error("%s: row stride %lld not a multiple of 8", what, (long long)rs); return WD_ERR_ALIGN; }
  return WD_OK;
}

static bool positive(double x) { return std::isfinite(x) && x > 0; }

// The pairs of one section: step * theta^(-2p/d) / 2 pi mod 1 in 2^-64 turns for p = 0 ..
// d/2 - 1, by repeated products in extended precision (64 of them keep 2^-57 of the value).
static void turn_fractions(double theta, double step, int d, uint64_t* out) {
  if (d == 0) return;
  const long double ratio = powl(theta, -2.0L / d);
  long double f = step / 6.283185307179586476925286766559006L;
  for (int p = 0; p < d / 2; ++p, f *= ratio)
    out[p] = static_cast<uint64_t>((f < 1 ? f : f - floorl(f)) * 18446744073709551616.0L);
}

}  // namespace wd

extern "C" {

wd_status wd_attention_packed(int dtype, int n_seq, int heads, int kv_heads, int dh, const void* q, int64_t q_rs,
                              int64_t q_rows, const int* cu_q, const void* k, const void* v, int64_t kv_rs,
                              int64_t k_rows, const int* cu_k, float scale, const float* bias, int radius, void* o,
                              int64_t o_rs, wd_stream stream) {
  WD_NEED(q); WD_NEED(cu_q); WD_NEED(k); WD_NEED(v); WD_NEED(cu_k); WD_OPT(bias); WD_NEED(o);
  if (dtype != WD_BF16 && dtype != WD_F16) {
    set_error("attention_packed: dtype %d (WD_BF16 or WD_F16)", dtype);
    return WD_ERR_DTYPE;
  }
  if (dh != 64 && dh != 128) { set_error("attention_packed: head dim %d (64 or 128)", dh); return WD_ERR_UNSUPPORTED; }
  if (n_seq <= 0 || q_rows <= 0 || k_rows <= 0 || n_seq > 65536 || q_rows > MAX_ROWS || k_rows > MAX_ROWS) {
    set_error("attention_packed: n_seq=%d, q_rows=%lld, k_rows=%lld", n_seq, (long long)q_rows, (long long)k_rows);
    return WD_ERR_SHAPE;
  }
  if (heads <= 0 || heads > 65535 || kv_heads <= 0 || heads % kv_heads) {
    set_error("attention_packed: %d heads over %d key/value heads", heads, kv_heads);
    return WD_ERR_SHAPE;
  }
  if ((bias == nullptr) != (radius == 0) || radius < 0 || radius > pka::MAX_RADIUS) {
    set_error("attention_packed: radius %d (1..%d with a bias, 0 without)", radius, pka::MAX_RADIUS);
    return WD_ERR_SHAPE;
  }
  if (!positive(scale) || !positive(scale * pka::LOG2E)) {
    set_error("attention_packed: scale %g", scale);
    return WD_ERR_ARG;
  }
  WD_TRY(check_stride("attention_packed q", q_rs, static_cast<int64_t>(heads) * dh));
  WD_TRY(check_stride("attention_packed k, v", kv_rs, static_cast<int64_t>(kv_heads) * dh));
  WD_TRY(check_stride("attention_packed o", o_rs, static_cast<int64_t>(heads) * dh));
  pka::Params p{};
  p.cu_q = cu_q; p.cu_k = cu_k;
  p.n_seq = n_seq; p.q_rows = static_cast<int>(q_rows); p.k_rows = static_cast<int>(k_rows);
  p.heads = heads; p.group = heads / kv_heads;
  p.scale_log2 = scale * pka::LOG2E;
  p.bias = bias; p.radius = radius;
  p.o = static_cast<bf16*>(o); p.o_rs = o_rs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == WD_BF16) return attention_packed_t<bf16>(dh, kv_heads, q, q_rs, k, v, kv_rs, p, st);
  return attention_packed_t<f16>(dh, kv_heads, q, q_rs, k, v, kv_rs, p, st);
}

wd_status wd_qknorm_rope_axes(int dtype, int64_t rows, int dh, const wd_rope_axes* axes, const int* pos, const void* q,
                              int64_t q_rs, int heads, const float* g_q, void* q_out, int64_t qo_rs, const void* k,
                              int64_t k_rs, int kv_heads, const float* g_k, void* k_out, int64_t ko_rs, float eps,
                              wd_stream stream) {
  if (!axes) { set_error("%s: axes is NULL", __func__); return WD_ERR_ARG; }
  WD_NEED(pos); WD_NEED(q); WD_NEED(q_out); WD_OPT(g_q);
  if (k) { WD_NEED(k); WD_NEED(k_out); WD_OPT(g_k); }
  if (dtype != WD_BF16 && dtype != WD_F32 && dtype != WD_F16) {
    set_error("qknorm_rope_axes: dtype %d", dtype);
    return WD_ERR_DTYPE;
  }
  if (rows <= 0 || rows > MAX_ROWS || dh < 8 || dh > 2 * rows::MAX_PAIRS || dh % 8) {
    set_error("qknorm_rope_axes: rows=%lld, dh=%d (a multiple of 8 in 8..%d)", (long long)rows, dh, 2 * rows::MAX_PAIRS);
    return WD_ERR_SHAPE;
  }
  int sum = 0;
  for (int i = 0; i < 3; ++i) {
    if (axes->sec[i] < 0 || axes->sec[i] % 2 || axes->sec[i] > dh) {
      set_error("qknorm_rope_axes: section of %d channels", axes->sec[i]);
      return WD_ERR_SHAPE;
    }
    sum += axes->sec[i];
  }
  if (sum != dh) { set_error("qknorm_rope_axes: sections add up to %d, not dh=%d", sum, dh); return WD_ERR_SHAPE; }
  if (!positive(axes->theta) || !positive(axes->step[0]) || !positive(axes->step[1]) || !positive(axes->step[2]) ||
      !(eps >= 0.f) || !std::isfinite(eps)) {
    set_error("qknorm_rope_axes: theta, step or eps");
    return WD_ERR_ARG;
  }
  rows::RopeArgs a{};
  a.pos = pos; a.rows = rows; a.dh = dh; a.eps = eps;
  a.p1 = axes->sec[0] / 2; a.p2 = a.p1 + axes->sec[1] / 2;
  a.in[0] = q; a.out[0] = q_out; a.gain[0] = g_q; a.in_rs[0] = q_rs; a.out_rs[0] = qo_rs;
  a.in[1] = k; a.out[1] = k_out; a.gain[1] = g_k; a.in_rs[1] = k_rs; a.out_rs[1] = ko_rs;
  for (int i = 0; i < (k ? 2 : 1); ++i) {
    const int64_t n = i ? kv_heads : heads;
    if (n <= 0 || n * dh > rows::ROW_MAX) {
      set_error("qknorm_rope_axes: %lld heads of %d (rows up to %d wide)", (long long)n, dh, rows::ROW_MAX);
      return WD_ERR_SHAPE;
    }
    a.D[i] = static_cast<int>(n) * dh;
    a.inv_D[i] = 1.f / a.D[i];
    WD_TRY(check_stride(i ? "qknorm_rope_axes k" : "qknorm_rope_axes q", a.in_rs[i], a.D[i]));
    WD_TRY(check_stride(i ? "qknorm_rope_axes k_out" : "qknorm_rope_axes q_out", a.out_rs[i], a.D[i]));
    if (a.in[i] == a.out[i] && a.in_rs[i] != a.out_rs[i]) {
      set_error("qknorm_rope_axes: in place with two row strides");
      return WD_ERR_ARG;
    }
  }
  for (int i = 0, p = 0; i < 3; p += axes->sec[i++] / 2) {
    if (i && axes->sec[i] == axes->sec[i - 1] && axes->step[i] == axes->step[i - 1])   // rows and columns, as a rule
      memcpy(a.freq + p, a.freq + p - axes->sec[i] / 2, axes->sec[i] / 2 * sizeof(a.freq[0]));
    else
      turn_fractions(axes->theta, axes->step[i], axes->sec[i], a.freq + p);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == WD_BF16) return qknorm_rope_axes<bf16>(a, st);
  if (dtype == WD_F16) return qknorm_rope_axes<f16>(a, st);
  return qknorm_rope_axes<float>(a, st);
}

wd_status wd_add_norm(int64_t rows, int D, int x_dtype, const void* x, int y_dtype, const void* y, int norm,
                      const float* gain, const float* beta, float eps, void* sum, int out_dtype, void* out,
                      float* scale, wd_stream stream) {
  WD_NEED(x); WD_OPT(y); WD_OPT(gain); WD_OPT(beta); WD_OPT(sum); WD_NEED(out);
  if ((x_dtype != WD_F32 && x_dtype != WD_BF16) || (y && y_dtype != WD_F32 && y_dtype != WD_BF16) ||
      (out_dtype != WD_F32 && out_dtype != WD_BF16 && out_dtype != WD_E4M3)) {
    set_error("add_norm: dtypes x %d, y %d, out %d", x_dtype, y_dtype, out_dtype);
    return WD_ERR_DTYPE;
  }
  if (out_dtype == WD_E4M3) { WD_NEED(scale); }
  if (rows <= 0 || rows > MAX_ROWS || D <= 0 || D % 8 || D > rows::ROW_MAX) {
    set_error("add_norm: rows=%lld, D=%d (a multiple of 8 up to %d)", (long long)rows, D, rows::ROW_MAX);
    return WD_ERR_SHAPE;
  }
  if ((norm != WD_NORM_LAYER && norm != WD_NORM_RMS) || !(eps >= 0.f) || !std::isfinite(eps)) {
    set_error("add_norm: norm %d, eps %g", norm, eps);
    return WD_ERR_ARG;
  }
  rows::AddNormArgs a{};
  a.x = x; a.y = y; a.gain = gain; a.beta = beta; a.sum = sum; a.out = out; a.scale = scale;
  a.rows = rows; a.D = D; a.rms = norm == WD_NORM_RMS; a.eps = eps;
  return add_norm(a, x_dtype, y ? y_dtype : x_dtype, out_dtype, static_cast<cudaStream_t>(stream));
}

size_t wd_gemm_lora_bytes(int M, int n_seg, int rank) {
  if (M <= 0 || M > (1 << 29) || n_seg <= 0 || n_seg > 65536 || rank <= 0 || rank % 8 || rank > lora::MAX_RANK) return 0;
  return gemm_lora_bytes(M, n_seg, rank);
}

wd_status wd_gemm_lora(int M, int N, int K, const void* A, const void* W, const float* bias, const wd_lora* lora,
                       int epilogue, void* out, const float* gate_a, const float* gate_b, void* ws, size_t ws_bytes,
                       wd_stream stream) {
  WD_NEED(A); WD_NEED(W); WD_OPT(bias); WD_NEED(out); WD_OPT(gate_a); WD_OPT(gate_b); WD_NEED(ws);
  if (!lora) { set_error("%s: lora is NULL", __func__); return WD_ERR_ARG; }
  WD_NEED(lora->seg); WD_NEED(lora->adapter); WD_NEED(lora->down); WD_NEED(lora->up); WD_OPT(lora->scale);
  if (epilogue < 0 || epilogue > EPI_STORE_F16 || epilogue == EPI_UNPATCH) {
    set_error("gemm_lora: epilogue %d", epilogue);
    return WD_ERR_ARG;
  }
  if (M <= 0 || M > (1 << 29) || N <= 0 || N % 64 || K <= 0 || K % 8) {
    set_error("gemm_lora: %d x %d x %d (N a multiple of 64, K of 8)", M, N, K);
    return WD_ERR_SHAPE;
  }
  const size_t need = wd_gemm_lora_bytes(M, lora->n_seg, lora->rank);
  const int64_t most = N > lora->rank ? N : lora->rank;   // rows of up or down an adapter has
  if (!need || lora->n_adapters <= 0 || lora->n_adapters * most > 0x7fffffff) {
    set_error("gemm_lora: n_seg=%d, n_adapters=%d, rank=%d (a multiple of 8 up to %d)", lora->n_seg, lora->n_adapters,
              lora->rank, lora::MAX_RANK);
    return WD_ERR_SHAPE;
  }
  if (ws_bytes < need) { set_error("gemm_lora: workspace %zu < %zu bytes", ws_bytes, need); return WD_ERR_WORKSPACE; }
  return gemm_lora(M, N, K, A, W, *lora, epilogue, epi(out, N, bias, gate_a, gate_b), ws,
                   static_cast<cudaStream_t>(stream));
}

}  // extern "C"
