// Rows of 8-bit integers with a scale each (int8.cuh says how they are rounded).
//
// Bound by HBM: a row is read once and kept in registers, 16 bytes for each load, between the search for its largest value
// and the rounding.  One row has 32 to 1024 threads of up to 8 loads; rows of up to 32 threads share a CTA.  Measured: 14336 rows
// of 4096 bf16 31.5 us (176 MB, 5.6 TB/s; 26 us at a copy's rate, where the rounding of a row and the loads of the next
// would have to overlap more), 48 rows of 14336 fp16 2.4 us (launch, one latency of memory, one barrier), 14336 of 4096
// fp32 45.8 us (6.4 TB/s).  Short rows are bound by the CTAs' coming and going (65536 rows of 128: 15 us).
#include "int8.cuh"
#include "int8_params.cuh"
#include "int8_plan.h"

namespace sesg {

namespace {

template <bool F32>
__device__ __forceinline__ uint32_t most_of(uint32_t m, const uint4& v) {
  if constexpr (F32) return most32(m, v);
  else return most16(m, v);
}

// Eight 8-bit integers as fp16.
__device__ __forceinline__ uint4 widen8(const uint2& q) {
  uint4 r;
  to_f16(q.x, r.x, r.y);
  to_f16(q.y, r.z, r.w);
  return r;
}

// X: the type.  KEEP loads of 16 bytes are kept by a thread, of fp32 pairs of them (a thread's eight elements).  WIDE: q as fp16
// integers.
template <int X, int KEEP, bool WIDE, int MOST>
__global__ void __launch_bounds__(MOST) quantize_kernel(const void* x, int rows, int K, void* q, float* scale) {
  constexpr bool F32 = X == MOE_F32;
  constexpr int bf16 = X == MOE_BF16;
  constexpr int L = F32 ? 2 : 1;  // loads of eight elements
  __shared__ uint32_t part[32];
  // In this order: the product behind the tokens' kernel takes everything before this kernel for done.
  griddep_wait();
  griddep_launch_dependents();
  const int T = blockDim.x, tid = threadIdx.x, n = K / 8;
  const size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= (size_t)rows) return;  // whole warps, and the only row of a CTA that has barriers
  const uint4* from = reinterpret_cast<const uint4*>(x) + row * n * L;
  uint4 v[KEEP][L];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < KEEP; ++j)
#pragma unroll
    for (int l = 0; l < L; ++l) {
      const int i = tid + j * T;
      v[j][l] = i < n ? ld_stream_v4(from + i * L + l) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
  for (int j = 0; j < KEEP; ++j)
#pragma unroll
    for (int l = 0; l < L; ++l) m = most_of<F32>(m, v[j][l]);
  for (int i = tid + KEEP * T; i < n; i += T)  // longer rows: read twice
    for (int l = 0; l < L; ++l) m = most_of<F32>(m, from[i * L + l]);
  m = warp_most(F32 ? m : most_f32(m, bf16));
  if (T > 32) {
    if ((tid & 31) == 0) part[tid >> 5] = m;
    __syncthreads();
    m = warp_most((tid & 31) < T / 32 ? part[tid & 31] : 0);
  }
  const RowScale s = row_scale<!F32>(m);
  if (tid == 0) scale[row] = s.scale();
  auto eight = [&](const uint4* w, int i) {
    float t[8];
    if constexpr (F32) unpack8(w[0], w[1], t);
    else unpack8(w[0], bf16, t);
    const uint2 b = quantize8<!F32>(t, s);
    if constexpr (WIDE) reinterpret_cast<uint4*>(q)[row * n + i] = widen8(b);
    else reinterpret_cast<uint2*>(q)[row * n + i] = b;
  };
#pragma unroll
  for (int j = 0; j < KEEP; ++j)
    if (tid + j * T < n) eight(v[j], tid + j * T);
  for (int i = tid + KEEP * T; i < n; i += T) {
    uint4 w[L];
    for (int l = 0; l < L; ++l) w[l] = from[i * L + l];
    eight(w, i);
  }
}

// 8-bit tokens as fp16 integers, eight for each thread, and a copy of their scales.
__global__ void widen_kernel(const uint2* x, const float* x_scale, int M, size_t n, uint4* tokens, float* scales) {
  griddep_wait();
  griddep_launch_dependents();
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) tokens[i] = widen8(x[i]);
  if (i < (size_t)M) scales[i] = x_scale[i];
}

template <typename... Par, typename... Arg>
cudaError_t launch(void (*kernel)(Par...), dim3 grid, dim3 block, cudaStream_t st, Arg... arg) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, arg...);
}

// T threads for each row, which keep 2 loads or KEEP.
template <int X, int KEEP, bool WIDE>
cudaError_t launch_row_kernel(const void* x, int rows, int K, void* q, float* scale, int T, cudaStream_t st) {
  const int R = T == 32 ? 8 : 1;
  using Kernel = void (*)(const void*, int, int, void*, float*);
  const Kernel kernel = K / 8 <= 2 * T ? quantize_kernel<X, 2, WIDE, 1024>
                        : T <= 256     ? quantize_kernel<X, KEEP, WIDE, 256>
                                       : quantize_kernel<X, KEEP, WIDE, 1024>;
  return launch(kernel, dim3((unsigned)(((size_t)rows + R - 1) / R)), dim3(T, R), st, x, rows, K, q, scale);
}

template <bool WIDE>
cudaError_t launch_rows(const void* x, int dtype, int rows, int K, void* q, float* scale, int sms, cudaStream_t st) {
  const int T = quantize_threads(rows, K, dtype == MOE_F32, sms);
  return dtype == MOE_F32    ? launch_row_kernel<MOE_F32, 4, WIDE>(x, rows, K, q, scale, T, st)
         : dtype == MOE_BF16 ? launch_row_kernel<MOE_BF16, 8, WIDE>(x, rows, K, q, scale, T, st)
                             : launch_row_kernel<MOE_F16, 8, WIDE>(x, rows, K, q, scale, T, st);
}

}  // namespace

cudaError_t launch_quantize(const void* x, int dtype, int rows, int K, int8_t* q, float* scale, int sms, cudaStream_t st) {
  return launch_rows<false>(x, dtype, rows, K, q, scale, sms, st);
}

cudaError_t launch_tokens(const void* x, int dtype, const float* x_scale, int M, int K, void* tokens, float* scales, int sms,
                          cudaStream_t st) {
  if (dtype != MOE_I8) return launch_rows<true>(x, dtype, M, K, tokens, scales, sms, st);
  const size_t n = (size_t)M * K / 8;  // at least 2 M
  return launch(widen_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), st, reinterpret_cast<const uint2*>(x), x_scale, M,
                n, reinterpret_cast<uint4*>(tokens), scales);
}

}  // namespace sesg
