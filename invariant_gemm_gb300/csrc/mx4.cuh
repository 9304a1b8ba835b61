// MX4 (blocks of 32 values along K, one E8M0 scale byte each, E2M1 codes):
// what the quantiser, the block norm and the product share, and the launch
// parameter blocks of the quantised-block operators.
//
// Codes: [rows][K/2] bytes, the even k in the low four bits. Scales: tiles of
// 512 bytes, one per 128 rows x 4 blocks, [row % 32][row / 32 % 4][block % 4],
// the tiles of a row group following each other along K. That is the order in
// which tensor memory holds the scale factors of 128 rows x 128 k (32 lanes
// of 16 bytes), so the product copies a tile as it stands.
#pragma once

#include <atomic>

#include "ig_common.cuh"

namespace ig {

constexpr int kMx4Block = 32;           // values per scale
constexpr int kMx4TileBytes = 512;      // scale bytes of 128 rows x 128 k

constexpr int64_t kNormMaxH = 32768;    // block norm: 1024 threads with 4 vectors of 8 values each

__host__ __device__ inline int64_t mx4_ktiles(int64_t K) { return (K + 127) / 128; }

// Byte offset of the scale of (row, block kb); kt = mx4_ktiles(K).
__host__ __device__ inline int64_t mx4_scale_at(int64_t row, int64_t kb, int64_t kt) {
  return ((row >> 7) * kt + (kb >> 2)) * kMx4TileBytes + (row & 31) * 16 +
         ((row >> 5) & 3) * 4 + (kb & 3);
}

// SMs of the current device (cached per device; 152 on GB300).
int sm_count();

struct Mx4QuantParams {
  const void* x;
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows, K, ldx, kt;
};

struct Mx4DequantParams {
  const uint8_t* codes;
  const uint8_t* scales;
  void* out;
  int64_t rows, K, ldo, kt;
  bool wide;           // every row of out starts at a multiple of 32 bytes
};

struct Mx4GemmParams {
  CUtensorMap tm_w;    // codes as [N][K / 4] 2-byte words, box 64 x 128, 128-byte swizzle
  CUtensorMap tm_x;    // codes as [M][K / 4] 2-byte words, box 64 x BN (pairs: 64), 128-byte swizzle
  CUtensorMap tm_ws, tm_xs;   // scale tiles as rows of 256 2-byte words, box 256 x 2 (pairs)
  const uint8_t* xc;
  const uint8_t* xs;
  const uint8_t* wc;
  const uint8_t* ws;
  void* y;
  uint32_t* status;
  int64_t M, N, K, ldy, kt;
  int64_t k_part;      // k per part: whole 256-k stages
  int32_t S, ntiles;   // parts of K; 128-column tiles of N
  int32_t stages;      // of the ring (few tokens)
  uint32_t tmem_cols;
  int32_t y_f32, flags;
};

struct NormParams {
  const void* h;
  const __nv_bfloat16* y;
  const __nv_bfloat16* gate;
  const __nv_bfloat16* w_post;
  const __nv_bfloat16* w_pre;
  void* h_out;
  __nv_bfloat16* n_out;
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows, H, ld_h, ld_y, ld_ho, ld_n, gate_rs, kt;
  int32_t gate_cs, plus_one;
  float eps, scale;
};

cudaError_t launch_mx4_quantize(const Mx4QuantParams& p, bool f32, cudaStream_t st);
cudaError_t launch_mx4_dequantize(const Mx4DequantParams& p, bool f32, cudaStream_t st);
cudaError_t launch_mx4_gemm(Mx4GemmParams& p, cudaStream_t st);
cudaError_t launch_mx4_gemm_pair(Mx4GemmParams& p, int sms, cudaStream_t st);
cudaError_t launch_block_norm(const NormParams& p, bool h_f32, cudaStream_t st);

// Lets a kernel use all of an SM's shared memory (227 KB), once per device:
// `done` has a bit for each device it was set on. The call costs a product of
// one token a tenth of its host time.
inline cudaError_t allow_smem(const void* kern, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

#ifdef __CUDACC__

// Eight FP32 values -> eight E2M1 codes, value i in bits 4i..4i+3 (nearest,
// ties to even, held at +-6). Each conversion takes the high nibble first.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(f32x2_to_bf16x2_bits(f[0], f[1]), f32x2_to_bf16x2_bits(f[2], f[3]),
                    f32x2_to_bf16x2_bits(f[4], f[5]), f32x2_to_bf16x2_bits(f[6], f[7]));
}

// Eight codes -> the E2M1 values they stand for times 2^(byte - 127), two
// bf16 to a word, all exact. A code seem read as the bf16 bits s0000000 eem0..
// is its value times 2^-126 (the code's exponent 0 is a subnormal there too);
// a product by 2^126, then one by the scale (2^-127 is a subnormal bf16).
__device__ __forceinline__ uint4 mx4_decode8(uint32_t c, uint32_t byte) {
  const uint32_t bits = byte == 0 ? 0x0040u : byte == 255 ? 0x7fc0u : byte << 7;
  const uint32_t one = 0x7e807e80u, scale = bits | bits << 16;
  const uint32_t odd = c >> 4;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // byte i of c in the low half, byte i of c >> 4 in the high one
    const uint32_t u = __byte_perm(c, odd, i | i << 4 | (4 + i) << 8 | (4 + i) << 12);
    const uint32_t w = (u << 12 & 0x80008000u) | (u << 6 & 0x01c001c0u);
    __nv_bfloat162 v;
    *reinterpret_cast<uint32_t*>(&v) = w;
    v = __hmul2(v, *reinterpret_cast<const __nv_bfloat162*>(&one));
    v = __hmul2(v, *reinterpret_cast<const __nv_bfloat162*>(&scale));
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Scale byte of a block whose largest magnitude has FP32 bits `top`
// (non-negative; not below the bits of infinity for infinity and NaN):
// exponent floor(log2 top) - 2, at least -127; 255 where the block has a
// value that is not finite. A subnormal top has an exponent field of 0 and
// falls under the lower limit like every top below 2^-124.
__device__ __forceinline__ uint32_t e8m0_of(uint32_t top) {
  if (top >= 0x7f800000u) return 255u;
  const uint32_t e = top >> 23;      // floor(log2 top) + 127
  return e > 2u ? e - 2u : 0u;
}

// The factor 2^-(byte - 127) that takes a block's values to code range (of no
// use for 255).
__device__ __forceinline__ float e8m0_inverse(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// Largest magnitude of one thread's 8 values as FP32 bits, the bits of
// infinity or more where one is not finite.
__device__ __forceinline__ uint32_t top_of(const uint4& b16) {
  const uint32_t m = 0x7fff7fffu;     // bf16 magnitudes compare as integers
  const uint32_t t = __vmaxu2(__vmaxu2(b16.x & m, b16.y & m), __vmaxu2(b16.z & m, b16.w & m));
  return max(t << 16, t & 0xffff0000u);
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t top_of(const float (&v)[8]) {
  float t = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) t = max_nan(t, fabsf(v[i]));
  return __float_as_uint(t);
}

// The scale byte of the block that an aligned group of LANES lanes holds, in
// all of them, from each lane's top_of. Whole warps call it.
template <int LANES>
__device__ __forceinline__ uint32_t mx4_block_byte(uint32_t top) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  return e8m0_of(top);
}

// Codes of 8 values of a block with scale byte `byte`.
__device__ __forceinline__ uint32_t mx4_encode8(const float (&v)[8], uint32_t byte) {
  const float inv = e8m0_inverse(byte);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = v[i] * inv;
  const uint32_t codes = e2m1x8(q);
  return byte == 255u ? 0u : codes;
}

// The 4 scale bytes of 4 blocks of LANES lanes each, in the first of those
// lanes. Whole warps call it.
template <int LANES>
__device__ __forceinline__ uint32_t mx4_scale_word(uint32_t byte) {
  byte |= __shfl_down_sync(0xffffffffu, byte, LANES) << 8;
  return byte | __shfl_down_sync(0xffffffffu, byte, 2 * LANES) << 16;
}

#endif  // __CUDACC__

}  // namespace ig
