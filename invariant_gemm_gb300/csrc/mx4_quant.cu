// MX4 quantisation and its inverse (layout and rules in mx4.cuh).
//
// Both are bound by memory: 2 or 4 bytes read and 17/32 of a byte written for
// each value, or the other way round, and the bf16 quantiser nearly as much by
// instructions. A thread takes U groups of 16 (bf16) or 8 values, a block's
// groups following each other through the rows, so that short rows fill blocks
// too; all of a thread's loads are in flight before the first is used. The
// lanes of four blocks hold the 4 bytes of a word of the scale tile, and one
// of them stores it. 8192 x 28672: bf16 88 us (6.8 TB/s), FP32 150 us (7.1 TB/s),
// back to bf16 90 us (6.6 TB/s), to FP32 156 us (6.8 TB/s).
#include "mx4.cuh"

namespace ig {

namespace {

constexpr int kThreads = 256;

// A thread's consecutive values, as they are loaded: as many as one or two
// 16-byte words hold.
template <typename T>
struct Raw {
  static constexpr int kValues = 32 / sizeof(T);
  uint4 a, b;
  __device__ __forceinline__ void load(const T* p) {
    // the two words of a 32-byte sector: the second comes from L1
    a = __ldg(reinterpret_cast<const uint4*>(p));
    b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
};

__device__ __forceinline__ void floats(const Raw<float>& r, float (&v)[8]) {
  v[0] = __uint_as_float(r.a.x); v[1] = __uint_as_float(r.a.y);
  v[2] = __uint_as_float(r.a.z); v[3] = __uint_as_float(r.a.w);
  v[4] = __uint_as_float(r.b.x); v[5] = __uint_as_float(r.b.y);
  v[6] = __uint_as_float(r.b.z); v[7] = __uint_as_float(r.b.w);
}
__device__ __forceinline__ uint32_t raw_top(const Raw<float>& r) {
  float v[8];
  floats(r, v);
  return top_of(v);
}
__device__ __forceinline__ uint32_t raw_top(const Raw<__nv_bfloat16>& r) {
  return max(top_of(r.a), top_of(r.b));
}
__device__ __forceinline__ void store_codes(const Raw<float>& r, uint32_t byte, uint8_t* codes) {
  float v[8];
  floats(r, v);
  *reinterpret_cast<uint32_t*>(codes) = mx4_encode8(v, byte);
}
__device__ __forceinline__ void store_codes(const Raw<__nv_bfloat16>& r, uint32_t byte,
                                            uint8_t* codes) {
  float v[8];
  uint2 c;
  unpack8(r.a, v);
  c.x = mx4_encode8(v, byte);
  unpack8(r.b, v);
  c.y = mx4_encode8(v, byte);
  *reinterpret_cast<uint2*>(codes) = c;
}

// The rows' groups of G values, each row's padded to whole 128 values, numbered
// row by row; a block takes U * kThreads of them. next() goes kThreads groups
// on. Grids are below 2^26 blocks, so that the block's start in units of 128
// values is a 32-bit number.
template <int U, int G>
struct Walk {
  static constexpr uint32_t kTile = 128 / G;
  int64_t row;
  uint32_t c, per;
  __device__ __forceinline__ Walk(int64_t kt) : per((uint32_t)kt * kTile) {
    const uint32_t start = blockIdx.x * (uint32_t)(U * kThreads / kTile);
    const uint32_t q = start / (uint32_t)kt;
    row = q;
    c = (start - q * (uint32_t)kt) * kTile + threadIdx.x;
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
  constexpr int G = Raw<T>::kValues, kLanes = kMx4Block / G;
  const Walk<U, G> start(p.kt);
  const uint32_t groups = (uint32_t)(p.K / G);
  griddep_wait();
  Raw<T> raw[U];
  Walk<U, G> w = start;
#pragma unroll
  for (int j = 0; j < U; ++j, w.next()) {
    raw[j] = Raw<T>{};
    if (w.row < p.rows && w.c < groups)
      raw[j].load(static_cast<const T*>(p.x) + w.row * p.ldx + (int64_t)w.c * G);
  }
  w = start;
#pragma unroll
  for (int j = 0; j < U; ++j, w.next()) {
    const uint32_t byte = mx4_block_byte<kLanes>(raw_top(raw[j]));
    const bool in = w.c < groups;
    const uint32_t word = mx4_scale_word<kLanes>(in ? byte : 127u);
    if (w.row >= p.rows) continue;
    if (in) store_codes(raw[j], byte, p.codes + (w.row * groups + w.c) * (G / 2));
    if (w.c % (4 * kLanes) == 0)
      *reinterpret_cast<uint32_t*>(p.scales + mx4_scale_at(w.row, w.c / kLanes, p.kt)) = word;
  }
}

// 32 bytes to a 32-byte boundary in one store, or to a 16-byte boundary in two
// (which leaves each sector half written in between: 8192 x 28672 90 us against
// 97). `wide` is the same for the whole grid.
__device__ __forceinline__ void store32(void* at, const uint4& a, const uint4& b, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(at), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z),
                   "r"(b.w) : "memory");
  } else {
    static_cast<uint4*>(at)[0] = a;
    static_cast<uint4*>(at)[1] = b;
  }
}

template <typename T, int U>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(Mx4DequantParams p) {
  constexpr int G = Raw<T>::kValues, kLanes = kMx4Block / G;
  const Walk<U, G> start(p.kt);
  const uint32_t groups = (uint32_t)(p.K / G);
  griddep_wait();
  uint2 codes[U];              // .y for bf16 only
  uint32_t byte[U];
  Walk<U, G> w = start;
#pragma unroll
  for (int j = 0; j < U; ++j, w.next()) {
    codes[j] = make_uint2(0, 0);
    byte[j] = 0;
    if (w.row >= p.rows || w.c >= groups) continue;
    const uint8_t* at = p.codes + (w.row * groups + w.c) * (G / 2);
    if constexpr (G == 16) codes[j] = __ldcs(reinterpret_cast<const uint2*>(at));
    else codes[j].x = __ldcs(reinterpret_cast<const uint32_t*>(at));
    byte[j] = p.scales[mx4_scale_at(w.row, w.c / kLanes, p.kt)];
  }
  w = start;
#pragma unroll
  for (int j = 0; j < U; ++j, w.next()) {
    if (w.row >= p.rows || w.c >= groups) continue;
    T* o = static_cast<T*>(p.out) + w.row * p.ldo + (int64_t)w.c * G;
    uint4 a = mx4_decode8(codes[j].x, byte[j]), b;
    if constexpr (G == 16) {
      b = mx4_decode8(codes[j].y, byte[j]);
    } else {
      b = make_uint4(a.z << 16, a.z & 0xffff0000u, a.w << 16, a.w & 0xffff0000u);
      a = make_uint4(a.x << 16, a.x & 0xffff0000u, a.y << 16, a.y & 0xffff0000u);
    }
    store32(o, a, b, p.wide);
  }
}

// U groups a thread where that still gives every SM eight blocks, else one: few
// rows are over soonest when each group has a thread (1000 x 4096 bf16 back: 3.3
// us with one, 4.4 with four).
template <int U, int G, typename P>
cudaError_t launch(void (*several)(P), void (*one)(P), const P& p, cudaStream_t st) {
  const int64_t groups = p.rows * p.kt * (128 / G);
  const bool many = groups >= (int64_t)8 * sm_count() * U * kThreads;
  const int64_t per = many ? U * kThreads : kThreads;
  const int64_t grid = (groups + per - 1) / per;
  if (grid >= 1 << 26) return cudaErrorInvalidConfiguration;
  return launch_pdl(many ? several : one, dim3((unsigned)grid), dim3(kThreads), 0, st, p);
}

// Two groups a thread: 4095 x 11008 19.5 us with two, 20.7 with four; back 19.2
// and 19.5.
template <typename T>
cudaError_t quantize(const Mx4QuantParams& p, cudaStream_t st) {
  return launch<2, Raw<T>::kValues>(quantize_kernel<T, 2>, quantize_kernel<T, 1>, p, st);
}
template <typename T>
cudaError_t dequantize(const Mx4DequantParams& p, cudaStream_t st) {
  return launch<2, Raw<T>::kValues>(dequantize_kernel<T, 2>, dequantize_kernel<T, 1>, p, st);
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4QuantParams& p, bool f32, cudaStream_t st) {
  return f32 ? quantize<float>(p, st) : quantize<__nv_bfloat16>(p, st);
}

cudaError_t launch_mx4_dequantize(const Mx4DequantParams& p, bool f32, cudaStream_t st) {
  return f32 ? dequantize<float>(p, st) : dequantize<__nv_bfloat16>(p, st);
}

}  // namespace ig
