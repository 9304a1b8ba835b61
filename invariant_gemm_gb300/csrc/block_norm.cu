// Norm after a block, gate, residual and norm before the next block, one row
// per thread block:
//   t = y rsqrt(mean(y^2) + eps) w_post,  h' = h + scale gate t,
//   n = h' rsqrt(mean(h'^2) + eps) w_pre, and n in MX4.
#include "mx4.cuh"

namespace ig {

namespace {

constexpr int kMaxVec = 4;   // 8-element vectors per thread

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < nw ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void weight8(const __nv_bfloat16* w, int64_t at, bool plus_one,
                                        float (&f)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(w + at), f);
  if (plus_one) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += 1.0f;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(f32x2_to_bf16x2_bits(f[0], f[1]), f32x2_to_bf16x2_bits(f[2], f[3]),
                    f32x2_to_bf16x2_bits(f[4], f[5]), f32x2_to_bf16x2_bits(f[6], f[7]));
}

template <bool F32>
__global__ void __launch_bounds__(1024) norm_kernel(NormParams p) {
  __shared__ float red[2][32];
  griddep_wait();
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, T = blockDim.x;
  const int64_t vecs = p.H / 8;
  float h[kMaxVec][8];
  if (p.h) {
#pragma unroll
    for (int j = 0; j < kMaxVec; ++j) {
      const int64_t c = tid + (int64_t)j * T;
      if (c >= vecs) continue;
      if (F32) {
        const float4* q = reinterpret_cast<const float4*>(
            static_cast<const float*>(p.h) + row * p.ld_h + c * 8);
        const float4 a = q[0], b = q[1];
        h[j][0] = a.x; h[j][1] = a.y; h[j][2] = a.z; h[j][3] = a.w;
        h[j][4] = b.x; h[j][5] = b.y; h[j][6] = b.z; h[j][7] = b.w;
      } else {
        unpack8(*reinterpret_cast<const uint4*>(
                    static_cast<const __nv_bfloat16*>(p.h) + row * p.ld_h + c * 8), h[j]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kMaxVec; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = 0.0f;
  }
  if (p.y) {
    float y[kMaxVec][8];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < kMaxVec; ++j) {
      const int64_t c = tid + (int64_t)j * T;
      if (c >= vecs) continue;
      unpack8(*reinterpret_cast<const uint4*>(p.y + row * p.ld_y + c * 8), y[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(y[j][i], y[j][i], ss);
    }
    float f = 1.0f;
    if (p.w_post) f = rsqrtf(block_sum(ss, red[0]) / (float)p.H + p.eps);
    f *= p.scale;
    if (p.gate && p.gate_cs == 0) f *= __bfloat162float(p.gate[row * p.gate_rs]);
#pragma unroll
    for (int j = 0; j < kMaxVec; ++j) {
      const int64_t c = tid + (int64_t)j * T;
      if (c >= vecs) continue;
      if (p.w_post) {
        float w[8];
        weight8(p.w_post, c * 8, p.plus_one, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[j][i] *= w[i];
      }
      if (p.gate && p.gate_cs) {
        float g[8];
        unpack8(*reinterpret_cast<const uint4*>(p.gate + row * p.gate_rs + c * 8), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[j][i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = fmaf(y[j][i], f, h[j][i]);
    }
  }
  if (p.h_out) {
#pragma unroll
    for (int j = 0; j < kMaxVec; ++j) {
      const int64_t c = tid + (int64_t)j * T;
      if (c >= vecs) continue;
      if (F32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p.h_out) + row * p.ld_ho +
                                              c * 8);
        q[0] = make_float4(h[j][0], h[j][1], h[j][2], h[j][3]);
        q[1] = make_float4(h[j][4], h[j][5], h[j][6], h[j][7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.h_out) + row * p.ld_ho +
                                  c * 8) = pack8(h[j]);
      }
    }
  }
  if (!p.w_pre) return;
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < kMaxVec; ++j) {
    if (tid + (int64_t)j * T >= vecs) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(h[j][i], h[j][i], ss);
  }
  const float f = rsqrtf(block_sum(ss, red[1]) / (float)p.H + p.eps);
  const int64_t slots = p.codes ? p.kt * 16 : vecs;   // MX4 also writes the scales that pad K
#pragma unroll
  for (int j = 0; j < kMaxVec; ++j) {
    const int64_t c = tid + (int64_t)j * T;
    float n[8] = {};
    if (c < vecs) {
      float w[8];
      weight8(p.w_pre, c * 8, p.plus_one, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = h[j][i] * f * w[i];
      const uint4 o = pack8(n);
      if (p.n_out) *reinterpret_cast<uint4*>(p.n_out + row * p.ld_n + c * 8) = o;
      unpack8(o, n);
    }
    if (p.codes) {
      uint32_t byte;
      const uint32_t codes = mx4_encode8(n, byte);
      if (c < vecs) reinterpret_cast<uint32_t*>(p.codes)[row * vecs + c] = codes;
      if (c % 4 == 0 && c < slots)
        p.scales[mx4_scale_at(row, c / 4, p.kt)] = c < vecs ? byte : 127;
    }
  }
}

}  // namespace

cudaError_t launch_block_norm(const NormParams& p, bool h_f32, cudaStream_t st) {
  const int64_t slots = mx4_ktiles(p.H) * 16;
  int threads = 32;
  while (threads < 1024 && threads * 2 < slots) threads *= 2;
  return h_f32 ? launch_pdl(norm_kernel<true>, dim3((unsigned)p.rows), threads, 0, st, p)
               : launch_pdl(norm_kernel<false>, dim3((unsigned)p.rows), threads, 0, st, p);
}

}  // namespace ig
