// extern "C" entry points of the operators on 8-bit integers and of the norms around a block: argument checks and launches.
#include "dense_params.cuh"
#include "int8_params.cuh"

using namespace sesg;

namespace {

constexpr int kMaxTokens = 1 << 20, kMaxOut = 1 << 20, kMaxIn = 1 << 16;
constexpr int kMaxD = 16384;
constexpr size_t kWsAlign = 256;

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// A call's tensors: each with its bytes, NULL with any.
struct Span {
  const void* p;
  size_t bytes;
  bool overlaps(const Span& o) const {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)o.p;
    return p && o.p && a < b + o.bytes && b < a + bytes;
  }
  template <size_t N>
  bool overlaps_any(const Span (&o)[N]) const {
    for (const Span& s : o)
      if (overlaps(s)) return true;
    return false;
  }
};
template <size_t N>
bool all_aligned(const Span (&s)[N]) {
  for (const Span& t : s)
    if (!aligned(t.p, 16)) return false;
  return true;
}

inline size_t width(int dtype) { return dtype == MOE_I8 ? 1 : dtype == MOE_F32 ? 4 : 2; }
inline bool is16(int dtype) { return dtype == MOE_F16 || dtype == MOE_BF16; }

cudaError_t device_sizes(int& sms, int& smem) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  return e;
}

moe_status_t check_sizes(int M, int N, int K) {
  if (M < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (M > kMaxTokens || N > kMaxOut || K > kMaxIn || K % 16) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

moe_status_t check_expert_sizes(int n, int d, int f) {
  if (n < 0 || d <= 0 || f <= 0) return MOE_ERR_INVALID_ARG;
  if (n > kMaxTokens || d % 16 || f % 16 || d > kMaxD || f > kMaxIn) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

// Workspace of an expert: a product's, then h in fp32.
struct ExpertWs {
  size_t h, bytes;
  ExpertWs(int n, int d, int f) {
    h = align_up(Int8Ws(n, d > f ? d : f).bytes, kWsAlign);
    bytes = h + align_up((size_t)n * f * 4, kWsAlign);
  }
};

}  // namespace

extern "C" {

moe_status_t moe_quantize_int8(const void* x, int32_t dtype, int32_t rows, int32_t K, int8_t* q, float* scale,
                               void* stream) {
  if ((!is16(dtype) && dtype != MOE_F32) || rows < 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (K > kMaxIn || K % 16) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scale) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 16)) return MOE_ERR_ALIGNMENT;
  const Span in = {x, (size_t)rows * K * width(dtype)}, out = {q, (size_t)rows * K}, sc = {scale, (size_t)rows * 4};
  if (out.overlaps(in) || sc.overlaps(in) || sc.overlaps(out)) return MOE_ERR_INVALID_ARG;
  int sms = 0, smem = 0;
  if (device_sizes(sms, smem) != cudaSuccess) return MOE_ERR_CUDA;
  return cuda_status(launch_quantize(x, dtype, rows, K, q, scale, sms, (cudaStream_t)stream));
}

size_t moe_linear_int8_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t gated) {
  if (check_sizes(M, N, K) != MOE_OK) return 0;
  return Int8Ws(M, K).bytes;
}

}  // extern "C"

namespace {

// tries: diagnostics (else 0), as in LinearInt8Call
moe_status_t linear_int8_call(const moe_linear_int8_t* op, void* ws, size_t ws_bytes, uint32_t tries, void* stream) {
  if (!op) return MOE_ERR_INVALID_ARG;
  if (!is16(op->dtype) || (op->x_dtype != op->dtype && op->x_dtype != MOE_I8)) return MOE_ERR_INVALID_ARG;
  if (op->out_dtype != op->dtype && op->out_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (op->act < MOE_ACT_NONE || op->act > MOE_ACT_SILU) return MOE_ERR_INVALID_ARG;
  const moe_status_t s = check_sizes(op->M, op->N, op->K);
  if (s != MOE_OK || op->M == 0) return s;
  const bool x16 = op->x_dtype != MOE_I8;
  if (!op->x || !op->w || !op->w_scale || !op->y || !ws || x16 == (op->x_scale != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((op->w_mul == nullptr) != (op->w_mul_scale == nullptr) || (op->bias_mul && !op->w_mul)) return MOE_ERR_INVALID_ARG;
  const size_t M = op->M, N = op->N, K = op->K;
  const Span y = {op->y, M * N * width(op->out_dtype)}, residual = {op->residual, M * N * 2};
  const Span in[] = {{op->x, M * K * width(op->x_dtype)}, {op->x_scale, M * 4}, {op->w, N * K}, {op->w_scale, N * 4},
                     {op->w_mul, N * K}, {op->w_mul_scale, N * 4}, {op->bias, N * 2}, {op->bias_mul, N * 2}};
  if (!all_aligned(in) || !aligned(op->residual, 16) || !aligned(op->y, 16) || !aligned(ws, kWsAlign))
    return MOE_ERR_ALIGNMENT;
  if (y.overlaps_any(in)) return MOE_ERR_INVALID_ARG;
  if ((op->y != op->residual || op->out_dtype != op->dtype) && y.overlaps(residual)) return MOE_ERR_INVALID_ARG;
  const size_t need = Int8Ws(op->M, op->K).bytes;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const Span work = {ws, need};
  if (work.overlaps_any(in) || work.overlaps(y) || work.overlaps(residual)) return MOE_ERR_INVALID_ARG;
  int sms = 0, smem = 0;
  if (device_sizes(sms, smem) != cudaSuccess) return MOE_ERR_CUDA;
  LinearInt8Call c = {};
  c.M = op->M;
  c.N = op->N;
  c.K = op->K;
  c.x_dtype = op->x_dtype;
  c.bf16 = op->dtype == MOE_BF16;
  c.act = op->act;
  c.out_f32 = op->out_dtype == MOE_F32;
  c.x = op->x;
  c.x_scale = op->x_scale;
  c.w = op->w;
  c.w_mul = op->w_mul;
  c.w_scale = op->w_scale;
  c.w_mul_scale = op->w_mul_scale;
  c.bias = op->bias;
  c.bias_mul = op->bias_mul;
  c.residual = op->residual;
  c.y = op->y;
  c.tries = tries;
  return cuda_status(launch_linear_int8(c, ws, sms, smem, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

moe_status_t moe_linear_int8(const moe_linear_int8_t* op, void* ws, size_t ws_bytes, void* stream) {
  return linear_int8_call(op, ws, ws_bytes, 0, stream);
}

moe_status_t moe_selftest_linear_int8_timeout(const moe_linear_int8_t* op, void* ws, size_t ws_bytes, uint32_t tries,
                                              void* stream) {
  if (tries < 1 || tries > 4000) return MOE_ERR_INVALID_ARG;
  return linear_int8_call(op, ws, ws_bytes, tries, stream);
}

size_t moe_expert_int8_workspace_bytes(int32_t n, int32_t d, int32_t f) {
  return check_expert_sizes(n, d, f) == MOE_OK ? ExpertWs(n, d, f).bytes : 0;
}

moe_status_t moe_expert_int8_swiglu(const void* x, const float* x_scale, int32_t x_dtype, int32_t dtype, int32_t n,
                                    const moe_int8_experts_t* experts, int32_t expert, const void* residual, void* y,
                                    void* ws, size_t ws_bytes, void* stream) {
  if (!experts || !is16(dtype) || (x_dtype != dtype && x_dtype != MOE_I8)) return MOE_ERR_INVALID_ARG;
  const moe_int8_experts_t& ex = *experts;
  const moe_status_t s = check_expert_sizes(n, ex.d, ex.f);
  if (s != MOE_OK) return s;
  if (ex.E < 1 || ex.E > 256) return ex.E < 0 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED_SHAPE;
  if (expert < 0 || expert >= ex.E) return MOE_ERR_INVALID_ARG;
  const size_t E = ex.E, d = ex.d, f = ex.f;
  const Span weights[] = {{ex.gate_t, E * f * d}, {ex.up_t, E * f * d}, {ex.down_t, E * f * d},
                          {ex.gate_scale, E * f * 4}, {ex.up_scale, E * f * 4}, {ex.down_scale, E * d * 4}};
  for (const Span& w : weights)
    if (!w.p) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(weights)) return MOE_ERR_ALIGNMENT;
  if (n == 0) return MOE_OK;
  const bool x16 = x_dtype != MOE_I8;
  if (!x || !y || !ws || x16 == (x_scale != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(x_scale, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(ws, kWsAlign))
    return MOE_ERR_ALIGNMENT;
  const Span out = {y, n * d * 2}, in = {x, n * d * width(x_dtype)}, sc = {x_scale, (size_t)n * 4}, res = {residual, n * d * 2};
  // x is read before the first value of y is written: y may be x, not a part of it
  if ((y != residual && out.overlaps(res)) || out.overlaps_any(weights)) return MOE_ERR_INVALID_ARG;
  if ((!(x16 && y == x) && out.overlaps(in)) || out.overlaps(sc)) return MOE_ERR_INVALID_ARG;
  const ExpertWs at(n, ex.d, ex.f);
  if (ws_bytes < at.bytes) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const Span work = {ws, at.bytes};
  if (work.overlaps(in) || work.overlaps(sc) || work.overlaps(out) || work.overlaps(res) || work.overlaps_any(weights))
    return MOE_ERR_INVALID_ARG;
  int sms = 0, smem = 0;
  if (device_sizes(sms, smem) != cudaSuccess) return MOE_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  float* h = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + at.h);
  const size_t stack = (size_t)expert * f * d;
  LinearInt8Call c = {};
  c.M = n;
  c.N = ex.f;
  c.K = ex.d;
  c.x_dtype = x_dtype;
  c.bf16 = dtype == MOE_BF16;
  c.act = MOE_ACT_SILU;
  c.out_f32 = 1;
  c.x = x;
  c.x_scale = x_scale;
  c.w = ex.gate_t + stack;
  c.w_mul = ex.up_t + stack;
  c.w_scale = ex.gate_scale + expert * f;
  c.w_mul_scale = ex.up_scale + expert * f;
  c.y = h;
  const cudaError_t e = launch_linear_int8(c, ws, sms, smem, st);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  LinearInt8Call c2 = {};
  c2.M = n;
  c2.N = ex.d;
  c2.K = ex.f;
  c2.bf16 = dtype == MOE_BF16;
  c2.x_dtype = MOE_F32;
  c2.x = h;
  c2.w = ex.down_t + stack;
  c2.w_scale = ex.down_scale + expert * d;
  c2.residual = residual;
  c2.y = y;
  return cuda_status(launch_linear_int8(c2, ws, sms, smem, st));
}

moe_status_t moe_residual_norm(const moe_residual_norm_t* op, void* stream) {
  if (!op || op->M < 0 || op->d <= 0 || !is16(op->dtype)) return MOE_ERR_INVALID_ARG;
  if (op->s_dtype != op->dtype && op->s_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (op->y_dtype != op->dtype && op->y_dtype != MOE_I8) return MOE_ERR_INVALID_ARG;
  for (const int kind : {op->post, op->norm})
    if (kind < MOE_NORM_NONE || kind > MOE_NORM_LAYER) return MOE_ERR_INVALID_ARG;
  if (!(op->eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (op->M > kMaxTokens || op->d > kMaxD || op->d % (op->y_dtype == MOE_I8 ? 16 : 8)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (op->gate_rows < 0 || (op->gate_rows > 0) != (op->gate != nullptr)) return MOE_ERR_INVALID_ARG;
  if (op->M == 0) return MOE_OK;
  if (op->gate_rows > 0 && op->M % op->gate_rows) return MOE_ERR_INVALID_ARG;
  if (!op->x || (!op->s && !op->y) || (op->norm != MOE_NORM_NONE) != (op->y != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((op->y && op->y_dtype == MOE_I8) != (op->y_scale != nullptr)) return MOE_ERR_INVALID_ARG;
  if (op->post == MOE_NORM_NONE && (op->post_weight || op->post_bias)) return MOE_ERR_INVALID_ARG;
  if (op->norm == MOE_NORM_NONE && (op->weight || op->bias)) return MOE_ERR_INVALID_ARG;
  const size_t M = op->M, d = op->d;
  const Span vectors[] = {{op->gate, op->gate_rows * d * 2}, {op->post_weight, d * 2}, {op->post_bias, d * 2},
                          {op->weight, d * 2}, {op->bias, d * 2}};
  const Span x = {op->x, M * d * 2}, residual = {op->residual, M * d * width(op->s_dtype)};
  const Span s = {op->s, M * d * width(op->s_dtype)}, y = {op->y, M * d * width(op->y_dtype)}, sc = {op->y_scale, M * 4};
  for (const Span& t : {x, residual, s, y, sc})
    if (!aligned(t.p, 16)) return MOE_ERR_ALIGNMENT;
  if (!all_aligned(vectors)) return MOE_ERR_ALIGNMENT;
  // a thread reads its elements of x and the residual before it writes the same ones of s and y
  const bool s_in_x = s.p == x.p && op->s_dtype == op->dtype, y_in_x = y.p == x.p && op->y_dtype == op->dtype;
  if (s.overlaps_any(vectors) || y.overlaps_any(vectors) || sc.overlaps_any(vectors)) return MOE_ERR_INVALID_ARG;
  if ((!s_in_x && s.overlaps(x)) || (s.p != residual.p && s.overlaps(residual))) return MOE_ERR_INVALID_ARG;
  if ((!y_in_x && y.overlaps(x)) || y.overlaps(residual) || y.overlaps(s)) return MOE_ERR_INVALID_ARG;
  if (sc.overlaps(x) || sc.overlaps(residual) || sc.overlaps(s) || sc.overlaps(y)) return MOE_ERR_INVALID_ARG;
  int sms = 0, smem = 0;
  if (device_sizes(sms, smem) != cudaSuccess) return MOE_ERR_CUDA;
  return cuda_status(launch_residual_norm(*op, sms, (cudaStream_t)stream));
}

}  // extern "C"
