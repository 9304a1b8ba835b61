// MX4 quantisation and its inverse (layout and rules in mx4.cuh).
//
// Both are bound by memory: 2 or 4 bytes read and 17/32 of a byte written for
// each value, or the other way round. A thread takes U groups of 8 values, a
// block's groups following each other through the rows, so that short rows
// fill blocks too; all of a thread's loads are in flight before the first is
// used. A scale byte belongs to 4 lanes; 16 lanes hold the 4 bytes of a word of
// the scale tile, and one of them stores it.
#include "mx4.cuh"

namespace ig {

namespace {

constexpr int kThreads = 256;

template <typename T>
struct Raw;                                      // 8 values as they are loaded
template <>
struct Raw<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack8(a, v); }
  __device__ __forceinline__ uint32_t top() const { return top_of(a); }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ uint32_t top() const {
    float v[8];
    get(v);
    return top_of(v);
  }
};

// The rows' groups of 8 values, each row's padded to whole 128 values (16
// groups), numbered row by row; a block takes U * kThreads of them. next()
// goes kThreads groups on. Grids are below 2^26 blocks, so that the block's
// start in units of 16 groups is a 32-bit number.
template <int U>
struct Walk {
  int64_t row;
  uint32_t c, per;
  __device__ __forceinline__ Walk(int64_t kt) : per((uint32_t)kt * 16) {
    const uint32_t start = blockIdx.x * (uint32_t)(U * kThreads / 16);
    const uint32_t q = start / (uint32_t)kt;
    row = q;
    c = (start - q * (uint32_t)kt) * 16 + threadIdx.x;
    wrap();
  }
  __device__ __forceinline__ void wrap() {
    while (c >= per) {
      c -= per;
      ++row;
    }
  }
  __device__ __forceinline__ void next() {
    c += kThreads;
    wrap();
  }
};

// Groups that only pad a row write nothing but their scale, 1.
template <typename T, int U>
__global__ void __launch_bounds__(kThreads) quantize_kernel(Mx4QuantParams p) {
  const Walk<U> start(p.kt);
  const uint32_t groups = (uint32_t)(p.K / 8);
  griddep_launch();
  griddep_wait();
  Raw<T> raw[U];
  Walk<U> w = start;
#pragma unroll
  for (int j = 0; j < U; ++j, w.next()) {
    raw[j] = Raw<T>{};
    if (w.row < p.rows && w.c < groups)
      raw[j].load(static_cast<const T*>(p.x) + w.row * p.ldx + (int64_t)w.c * 8);
  }
  w = start;
#pragma unroll
  for (int j = 0; j < U; ++j, w.next()) {
    uint32_t byte;
    float v[8];
    raw[j].get(v);
    const uint32_t codes = mx4_encode8(v, raw[j].top(), byte);
    const bool in = w.c < groups;
    const uint32_t word = mx4_scale_word(in ? byte : 127u);
    if (w.row >= p.rows) continue;
    if (in) reinterpret_cast<uint32_t*>(p.codes)[w.row * groups + w.c] = codes;
    if (w.c % 16 == 0)
      *reinterpret_cast<uint32_t*>(p.scales + mx4_scale_at(w.row, w.c / 4, p.kt)) = word;
  }
}

template <typename T, int U>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(Mx4DequantParams p) {
  const Walk<U> start(p.kt);
  const uint32_t groups = (uint32_t)(p.K / 8);
  griddep_launch();
  griddep_wait();
  uint32_t codes[U], byte[U];
  Walk<U> w = start;
#pragma unroll
  for (int j = 0; j < U; ++j, w.next()) {
    codes[j] = byte[j] = 0;
    if (w.row >= p.rows || w.c >= groups) continue;
    codes[j] = __ldcs(reinterpret_cast<const uint32_t*>(p.codes) + w.row * groups + w.c);
    byte[j] = p.scales[mx4_scale_at(w.row, w.c / 4, p.kt)];
  }
  w = start;
#pragma unroll
  for (int j = 0; j < U; ++j, w.next()) {
    if (w.row >= p.rows || w.c >= groups) continue;
    const uint4 v = mx4_decode8(codes[j], byte[j]);
    T* o = static_cast<T*>(p.out) + w.row * p.ldo + (int64_t)w.c * 8;
    if constexpr (sizeof(T) == 4) {
      float f[8];
      unpack8(v, f);
      reinterpret_cast<float4*>(o)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(o)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      *reinterpret_cast<uint4*>(o) = v;
    }
  }
}

// Four groups a thread where that still gives every SM two blocks, else one:
// few rows are over soonest when each group has a thread.
template <typename P>
cudaError_t launch(void (*four)(P), void (*one)(P), const P& p, cudaStream_t st) {
  const int64_t groups = p.rows * p.kt * 16;
  const bool many = groups >= (int64_t)2 * sm_count() * 4 * kThreads;
  const int64_t per = many ? 4 * kThreads : kThreads;
  const int64_t grid = (groups + per - 1) / per;
  if (grid >= 1 << 26) return cudaErrorInvalidConfiguration;
  return launch_pdl(many ? four : one, dim3((unsigned)grid), dim3(kThreads), 0, st, p);
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4QuantParams& p, bool f32, cudaStream_t st) {
  return f32 ? launch(quantize_kernel<float, 4>, quantize_kernel<float, 1>, p, st)
             : launch(quantize_kernel<__nv_bfloat16, 4>, quantize_kernel<__nv_bfloat16, 1>, p, st);
}

cudaError_t launch_mx4_dequantize(const Mx4DequantParams& p, bool f32, cudaStream_t st) {
  return f32 ? launch(dequantize_kernel<float, 4>, dequantize_kernel<float, 1>, p, st)
             : launch(dequantize_kernel<__nv_bfloat16, 4>, dequantize_kernel<__nv_bfloat16, 1>, p,
                      st);
}

}  // namespace ig
