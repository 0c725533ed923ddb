// extern "C" entry points of the operators on uncompressed 16-bit weights: argument checks and launches.
#include "dense_params.cuh"

using namespace sesg;

namespace {

constexpr int kMaxTokens = 1 << 20, kMaxOut = 1 << 20, kMaxIn = 1 << 18;
constexpr int kMaxDenseD = 16384, kMaxDenseF = 65536;
constexpr size_t kWsAlign = 256;

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// Whether a result of n bytes at y shares memory with an input of m bytes at p (NULL: none).
inline bool overlaps(const void* y, size_t n, const void* p, size_t m) {
  const uintptr_t a = (uintptr_t)y, b = (uintptr_t)p;
  return p && a < b + m && b < a + n;
}

// ... or with an expert stack's rows, which lie d or, interleaved, 2 d elements apart.
bool overlaps(const void* y, size_t n, const moe_dense_experts_t& ex) {
  const size_t rows = (size_t)ex.E * ex.f, d = ex.d;
  const size_t apart = ex.down == ex.gate_t + d ? 2 * d : d, bytes = ((rows - 1) * apart + d) * 2;
  return overlaps(y, n, ex.gate_t, bytes) || overlaps(y, n, ex.down, bytes) || overlaps(y, n, ex.up_t, rows * d * 2);
}

cudaError_t device_sizes(int& sms, int& smem) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  return e;
}

moe_status_t check_linear_sizes(int M, int N, int K) {
  if (M < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (M > kMaxTokens || N > kMaxOut || K > kMaxIn || K % 8) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

moe_status_t check_dense_sizes(int d, int f) {
  if (d <= 0 || f <= 0) return MOE_ERR_INVALID_ARG;
  if (d % 8 || f % 8 || d > kMaxDenseD || f > kMaxDenseF) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

moe_status_t check_dense_experts(const moe_dense_experts_t& ex, int d, int f, int dtype) {
  if (ex.E < 1 || ex.E > 256) return ex.E < 0 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED_SHAPE;
  if (ex.d != d || ex.f != f || ex.dtype != dtype) return MOE_ERR_INVALID_ARG;
  if (!ex.gate_t || !ex.up_t || !ex.down) return MOE_ERR_INVALID_ARG;
  if (!aligned(ex.gate_t, 16) || !aligned(ex.up_t, 16) || !aligned(ex.down, 16)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// Gate and down rows may lie interleaved in one buffer, as in moe_experts_t.
DenseExpertSet to_set(const moe_dense_experts_t& ex, int expert = -1) {
  DenseExpertSet s;
  const size_t d = ex.d;
  const uint16_t *g = ex.gate_t, *dn = ex.down;
  s.gate_rs = s.down_rs = dn == g + d ? 2 * d : d;
  s.up_rs = d;
  s.E = ex.E;
  s.gate_t = g;
  s.up_t = ex.up_t;
  s.down = dn;
  if (expert >= 0) {
    s.E = 1;
    s.gate_t = g + (size_t)expert * ex.f * s.gate_rs;
    s.up_t = ex.up_t + (size_t)expert * ex.f * s.up_rs;
    s.down = dn + (size_t)expert * ex.f * s.down_rs;
  }
  return s;
}

moe_status_t check_dense_layer(const moe_dense_layer_t* layer, int B) {
  if (!layer || B < 0) return MOE_ERR_INVALID_ARG;
  const moe_dense_experts_t& r = layer->routed;
  if (r.dtype != MOE_F16 && r.dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  moe_status_t s = check_dense_sizes(r.d, r.f);
  if (s != MOE_OK) return s;
  s = check_dense_experts(r, r.d, r.f, r.dtype);
  if (s != MOE_OK) return s;
  if (layer->shared.E != 0) {
    s = check_dense_experts(layer->shared, r.d, r.f, r.dtype);
    if (s != MOE_OK) return s;
    if (layer->shared.E > 8) return MOE_ERR_UNSUPPORTED_SHAPE;
  }
  if (layer->k < 1 || layer->k > r.E) return MOE_ERR_INVALID_ARG;
  if (layer->k > kMaxTok || B > kDenseMaxTok) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!layer->w_router) return MOE_ERR_INVALID_ARG;
  if (!aligned(layer->w_router, 16)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// Up to kDenseMaxTok tokens keep h as two 16-bit rows each, more round it.
inline int h_rows(int n) { return n <= kDenseMaxTok ? 2 * n : n; }
size_t expert_ws(int n, int f) { return align_up(linear_ws_bytes(), kWsAlign) + (size_t)h_rows(n) * f * 2; }

}  // namespace

extern "C" {

size_t moe_linear_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t gated) {
  if (check_linear_sizes(M, N, K) != MOE_OK) return 0;
  return linear_ws_bytes();
}

}  // extern "C"

namespace {

// tries: diagnostics (else 0), as in LinearCall
moe_status_t linear_call(const moe_linear_t* op, void* ws, size_t ws_bytes, uint32_t tries, void* stream) {
  if (!op) return MOE_ERR_INVALID_ARG;
  if (op->dtype != MOE_F16 && op->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (op->out_dtype != op->dtype && op->out_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (op->act < MOE_ACT_NONE || op->act > MOE_ACT_SILU) return MOE_ERR_INVALID_ARG;
  if (op->w_layout != MOE_W_NK && op->w_layout != MOE_W_KN) return MOE_ERR_INVALID_ARG;
  moe_status_t s = check_linear_sizes(op->M, op->N, op->K);
  if (s != MOE_OK) return s;
  if (op->w_layout == MOE_W_KN && op->N % 8) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (op->M == 0) return MOE_OK;
  if (!op->x || !op->w || !op->y || !ws) return MOE_ERR_INVALID_ARG;
  if (op->bias_mul && !op->w_mul) return MOE_ERR_INVALID_ARG;
  if (!aligned(op->x, 16) || !aligned(op->w, 16) || !aligned(op->w_mul, 16) || !aligned(op->bias, 16) ||
      !aligned(op->bias_mul, 16) || !aligned(op->residual, 16) || !aligned(op->y, 16) || !aligned(ws, kWsAlign))
    return MOE_ERR_ALIGNMENT;
  const size_t out = (size_t)op->M * op->N * (op->out_dtype == MOE_F32 ? 4 : 2), wn = (size_t)op->N * op->K * 2;
  if (overlaps(op->y, out, op->x, (size_t)op->M * op->K * 2) || overlaps(op->y, out, op->w, wn) ||
      overlaps(op->y, out, op->w_mul, wn) || overlaps(op->y, out, op->bias, (size_t)op->N * 2) ||
      overlaps(op->y, out, op->bias_mul, (size_t)op->N * 2))
    return MOE_ERR_INVALID_ARG;
  if ((op->y != op->residual || op->out_dtype != op->dtype) &&
      overlaps(op->y, out, op->residual, (size_t)op->M * op->N * 2))
    return MOE_ERR_INVALID_ARG;
  const size_t head = linear_ws_bytes();
  if (ws_bytes < head) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (overlaps(ws, head, op->y, out) || overlaps(ws, head, op->x, (size_t)op->M * op->K * 2) ||
      overlaps(ws, head, op->w, wn) || overlaps(ws, head, op->w_mul, wn) ||
      overlaps(ws, head, op->bias, (size_t)op->N * 2) || overlaps(ws, head, op->bias_mul, (size_t)op->N * 2) ||
      overlaps(ws, head, op->residual, (size_t)op->M * op->N * 2))
    return MOE_ERR_INVALID_ARG;
  int sms = 0, smem = 0;
  if (device_sizes(sms, smem) != cudaSuccess) return MOE_ERR_CUDA;
  LinearCall c = {};
  c.M = op->M;
  c.N = op->N;
  c.K = op->K;
  c.bf16 = op->dtype == MOE_BF16;
  c.kn = op->w_layout == MOE_W_KN;
  c.act = op->act;
  c.out_f32 = op->out_dtype == MOE_F32;
  c.x = op->x;
  c.w = op->w;
  c.w_mul = op->w_mul;
  c.bias = op->bias;
  c.bias_mul = op->bias_mul;
  c.residual = op->residual;
  c.y = op->y;
  c.w_stride = c.w_mul_stride = c.kn ? op->N : op->K;
  c.tries = tries;
  return cuda_status(launch_linear(c, ws, sms, smem, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

moe_status_t moe_linear(const moe_linear_t* op, void* ws, size_t ws_bytes, void* stream) {
  return linear_call(op, ws, ws_bytes, 0, stream);
}

moe_status_t moe_selftest_linear_timeout(const moe_linear_t* op, void* ws, size_t ws_bytes, uint32_t tries, void* stream) {
  if (tries < 1 || tries > 4000) return MOE_ERR_INVALID_ARG;
  return linear_call(op, ws, ws_bytes, tries, stream);
}

size_t moe_expert_dense_workspace_bytes(int32_t n, int32_t d, int32_t f) {
  if (n < 0 || n > kMaxTokens || check_dense_sizes(d, f) != MOE_OK) return 0;
  return expert_ws(n, f);
}

moe_status_t moe_expert_dense_swiglu(const uint16_t* x, int32_t n, const moe_dense_experts_t* experts,
                                     int32_t expert, const uint16_t* residual, uint16_t* y, void* ws,
                                     size_t ws_bytes, void* stream) {
  if (n < 0 || !experts) return MOE_ERR_INVALID_ARG;
  if (experts->dtype != MOE_F16 && experts->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  const int d = experts->d, f = experts->f;
  moe_status_t s = check_dense_sizes(d, f);
  if (s != MOE_OK) return s;
  if (n > kMaxTokens) return MOE_ERR_UNSUPPORTED_SHAPE;
  s = check_dense_experts(*experts, d, f, experts->dtype);
  if (s != MOE_OK) return s;
  if (expert < 0 || expert >= experts->E) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!x || !y || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(ws, kWsAlign)) return MOE_ERR_ALIGNMENT;
  // x is read before the first value of y is written
  const size_t bytes = (size_t)n * d * 2, need = expert_ws(n, f);
  if ((y != residual && overlaps(y, bytes, residual, bytes)) || overlaps(y, bytes, *experts)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (overlaps(ws, need, x, bytes) || overlaps(ws, need, y, bytes) || overlaps(ws, need, residual, bytes) ||
      overlaps(ws, need, *experts))
    return MOE_ERR_INVALID_ARG;
  int sms = 0, smem = 0;
  if (device_sizes(sms, smem) != cudaSuccess) return MOE_ERR_CUDA;
  const int bf16 = experts->dtype == MOE_BF16;
  const DenseExpertSet one = to_set(*experts, expert);
  cudaStream_t st = (cudaStream_t)stream;
  // Two products.  Up to 64 tokens are bound by the weights' bytes, and a second row for each token costs
  // nothing: h goes to the second product as hi + lo, to 2^-16 (bf16) or 2^-22 (fp16).  For more tokens
  // it would cost the tensor cores twice the work, and h is rounded to the type.
  const bool two = n <= kDenseMaxTok;
  void* h = reinterpret_cast<uint8_t*>(ws) + align_up(linear_ws_bytes(), kWsAlign);
  LinearCall c = {};
  c.M = n;
  c.N = f;
  c.K = d;
  c.bf16 = bf16;
  c.act = MOE_ACT_SILU;
  c.split = two;
  c.x = x;
  c.w = one.gate_t;
  c.w_mul = one.up_t;
  c.y = h;
  c.w_stride = one.gate_rs;
  c.w_mul_stride = one.up_rs;
  cudaError_t e = launch_linear(c, ws, sms, smem, st);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  LinearCall c2 = {};
  c2.M = h_rows(n);
  c2.pairs = two;
  c2.N = d;
  c2.K = f;
  c2.bf16 = bf16;
  c2.kn = 1;
  c2.x = h;
  c2.w = one.down;
  c2.residual = residual;
  c2.y = y;
  c2.w_stride = one.down_rs;
  return cuda_status(launch_linear(c2, ws, sms, smem, st));
}

size_t moe_layer_dense_workspace_bytes(const moe_dense_layer_t* layer, int32_t B) {
  if (check_dense_layer(layer, B) != MOE_OK) return 0;
  int sms = 0, smem = 0;
  if (device_sizes(sms, smem) != cudaSuccess) return 0;
  return dense_layer_ws_bytes(B, layer->routed.d, layer->routed.f, layer->routed.E, layer->k, layer->shared.E, sms);
}

}  // extern "C"

namespace {

// tries, missing: diagnostics (else 0), as in DenseLayerCall
moe_status_t layer_call(const uint16_t* x, int32_t B, const moe_dense_layer_t* layer, const uint16_t* residual,
                        uint16_t* y, int32_t rmsnorm_out, const moe_debug_t* dbg, void* ws, size_t ws_bytes,
                        uint32_t tries, int missing, void* stream) {
  moe_status_t s = check_dense_layer(layer, B);
  if (s != MOE_OK) return s;
  if (B == 0) return MOE_OK;
  if (!x || !y || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(ws, kWsAlign)) return MOE_ERR_ALIGNMENT;
  const size_t bytes = (size_t)B * layer->routed.d * 2;
  if (overlaps(y, bytes, x, bytes) || (y != residual && overlaps(y, bytes, residual, bytes))) return MOE_ERR_INVALID_ARG;
  const size_t router = (size_t)layer->routed.d * layer->routed.E * 2;
  auto in_weights = [&](const void* p, size_t n) {
    return overlaps(p, n, layer->w_router, router) || overlaps(p, n, layer->routed) ||
           (layer->shared.E > 0 && overlaps(p, n, layer->shared));
  };
  if (in_weights(y, bytes)) return MOE_ERR_INVALID_ARG;
  int sms = 0, smem = 0;
  if (device_sizes(sms, smem) != cudaSuccess) return MOE_ERR_CUDA;
  const moe_dense_experts_t& r = layer->routed;
  const size_t need = dense_layer_ws_bytes(B, r.d, r.f, r.E, layer->k, layer->shared.E, sms);
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (overlaps(ws, need, x, bytes) || overlaps(ws, need, y, bytes) || overlaps(ws, need, residual, bytes) ||
      in_weights(ws, need))
    return MOE_ERR_INVALID_ARG;
  DenseLayerCall c = {};
  c.B = B;
  c.d = r.d;
  c.f = r.f;
  c.k = layer->k;
  c.renorm = layer->renorm ? 1 : 0;
  c.rmsnorm = rmsnorm_out ? 1 : 0;
  c.bf16 = r.dtype == MOE_BF16;
  c.routed = to_set(r);
  if (layer->shared.E > 0) c.shared = to_set(layer->shared);
  c.x = x;
  c.w_router = layer->w_router;
  c.residual = residual;
  c.y = y;
  c.user_idx = dbg ? dbg->topk_idx : nullptr;
  c.user_w = dbg ? dbg->topk_w : nullptr;
  c.tries = tries;
  c.missing = missing;
  return cuda_status(launch_dense_layer(c, ws, sms, smem, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

moe_status_t moe_layer_dense_decode(const uint16_t* x, int32_t B, const moe_dense_layer_t* layer,
                                    const uint16_t* residual, uint16_t* y, int32_t rmsnorm_out,
                                    const moe_debug_t* dbg, void* ws, size_t ws_bytes, void* stream) {
  return layer_call(x, B, layer, residual, y, rmsnorm_out, dbg, ws, ws_bytes, 0, 0, stream);
}

moe_status_t moe_selftest_layer_dense_timeout(const uint16_t* x, int32_t B, const moe_dense_layer_t* layer, uint16_t* y,
                                              int32_t rmsnorm_out, int32_t barrier, void* ws, size_t ws_bytes,
                                              uint32_t tries, void* stream) {
  if (tries < 1 || tries > 4000 || barrier < 0 || barrier > (rmsnorm_out ? 3 : 2)) return MOE_ERR_INVALID_ARG;
  return layer_call(x, B, layer, nullptr, y, rmsnorm_out, nullptr, ws, ws_bytes, tries, barrier, stream);
}

}  // extern "C"
