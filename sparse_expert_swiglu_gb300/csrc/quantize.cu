// Rows of 8-bit integers with a scale each (int8.cuh says how they are rounded).
//
// Bound by HBM: a row is read once and kept in registers, 16 bytes for each load, between the search for its largest value
// and the rounding.  One row has 32 to 1024 threads of up to 8 loads; rows of up to 32 threads share a CTA.
#include "int8.cuh"
#include "int8_params.cuh"

namespace sesg {

namespace {

template <bool F32>
__device__ __forceinline__ uint32_t most_of(uint32_t m, const uint4& v) {
  if constexpr (F32)
    return max(max(max(m, v.x & 0x7fffffffu), max(v.y & 0x7fffffffu, v.z & 0x7fffffffu)), v.w & 0x7fffffffu);
  else return most16(m, v);
}

// KEEP loads of 16 bytes are kept by a thread; F32: pairs of them (a thread's eight elements).
template <bool F32, int KEEP>
__global__ void __launch_bounds__(1024) quantize_kernel(const void* x, int bf16, int rows, int K, int8_t* q, float* scale) {
  constexpr int L = F32 ? 2 : 1;  // loads of eight elements
  __shared__ uint32_t part[32];
  griddep_launch_dependents();
  griddep_wait();
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
  const RowScale s = row_scale(m);
  if (tid == 0) scale[row] = s.scale;
  uint2* to = reinterpret_cast<uint2*>(q + row * K);
  auto eight = [&](const uint4* w, int i) {
    float t[8];
    if constexpr (F32) {
      const uint32_t b[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = __uint_as_float(b[e]);
    } else {
      unpack8(w[0], bf16, t);
    }
    to[i] = quantize8(t, s);
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

}  // namespace

cudaError_t launch_quantize(const void* x, int dtype, int rows, int K, int8_t* q, float* scale, cudaStream_t st) {
  const int n = K / 8;
  int T = 32;
  while (T < 1024 && T * 2 < n) T *= 2;
  const int R = T == 32 ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((size_t)rows + R - 1) / R));
  cfg.blockDim = dim3(T, R);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = dtype == MOE_F32 ? (n <= 2 * T ? quantize_kernel<true, 2> : quantize_kernel<true, 4>)
                                       : (n <= 2 * T ? quantize_kernel<false, 2> : quantize_kernel<false, 8>);
  return cudaLaunchKernelEx(&cfg, kernel, x, (int)(dtype == MOE_BF16), rows, K, q, scale);
}

}  // namespace sesg
