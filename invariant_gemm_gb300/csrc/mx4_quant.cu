// MX4 quantisation and its inverse (layout and rules in mx4.cuh).
#include "mx4.cuh"

namespace ig {

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p), v);
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0];
  const float4 b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__host__ __device__ inline uint32_t row_blocks(int64_t K) {
  return (uint32_t)((mx4_ktiles(K) * 16 + kThreads - 1) / kThreads);
}

// Thread = 8 values. A row's K / 8 threads are followed by those of the scale
// entries that only pad K to 128 (value 1).
template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_kernel(Mx4QuantParams p) {
  griddep_wait();
  uint32_t bid = blockIdx.x;
  const int64_t c = (int64_t)next_digit(bid, row_blocks(p.K)) * kThreads + threadIdx.x;
  const int64_t row = bid;                  // c: 8-value group of the row
  const bool in = c * 8 < p.K;
  float v[8] = {};
  if (in) load8(reinterpret_cast<const T*>(p.x) + row * p.ldx + c * 8, v);
  uint32_t byte;
  const uint32_t codes = mx4_encode8(v, byte);
  if (in) reinterpret_cast<uint32_t*>(p.codes)[row * (p.K / 8) + c] = codes;
  if (c % 4 == 0 && c / 16 < p.kt)
    p.scales[mx4_scale_at(row, c / 4, p.kt)] = in ? byte : 127;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(Mx4DequantParams p) {
  griddep_wait();
  uint32_t bid = blockIdx.x;
  const int64_t c = (int64_t)next_digit(bid, row_blocks(p.K)) * kThreads + threadIdx.x;
  const int64_t row = bid;
  if (c * 8 >= p.K) return;
  float v[8];
  e2m1_values(reinterpret_cast<const uint32_t*>(p.codes)[row * (p.K / 8) + c], v);
  const float s = e8m0_value(p.scales[mx4_scale_at(row, c / 4, p.kt)]);
  T* o = reinterpret_cast<T*>(p.out) + row * p.ldo + c * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (T)(v[i] * s);
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4QuantParams& p, bool f32, cudaStream_t st) {
  const dim3 grid((unsigned)(p.rows * row_blocks(p.K)));
  return f32 ? launch_pdl(quantize_kernel<float>, grid, kThreads, 0, st, p)
             : launch_pdl(quantize_kernel<__nv_bfloat16>, grid, kThreads, 0, st, p);
}

cudaError_t launch_mx4_dequantize(const Mx4DequantParams& p, bool f32, cudaStream_t st) {
  const dim3 grid((unsigned)(p.rows * row_blocks(p.K)));
  return f32 ? launch_pdl(dequantize_kernel<float>, grid, kThreads, 0, st, p)
             : launch_pdl(dequantize_kernel<__nv_bfloat16>, grid, kThreads, 0, st, p);
}

}  // namespace ig
