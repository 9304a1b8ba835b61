// MX4 product: y[m][n] = sum_k x[m][k] w[n][k], both operands MX4.
#include "mx4.cuh"

namespace ig {

namespace {

constexpr int kTile = 32;     // tokens and output columns per block

// Block = 32 x 32 outputs, one scale block of K per step; thread = one token,
// four columns.
__global__ void __launch_bounds__(256) gemm_kernel(Mx4GemmParams p) {
  __shared__ float sx[kTile][kMx4Block + 1], sw[kTile][kMx4Block + 1];
  griddep_wait();
  uint32_t bid = blockIdx.x;
  const int64_t n0 = (int64_t)next_digit(bid, (uint32_t)((p.N + kTile - 1) / kTile)) * kTile;
  const int64_t m0 = (int64_t)bid * kTile;
  const int tid = threadIdx.x;
  float acc[4] = {};
  for (int64_t kb = 0; kb < p.K / kMx4Block; ++kb) {
    const int r = (tid & 127) >> 2, c = tid & 3;   // row of the tile, 8-value group
    const bool w = tid >= 128;
    const int64_t row = (w ? n0 : m0) + r;
    float v[8] = {};
    if (row < (w ? p.N : p.M)) {
      const uint8_t* codes = w ? p.wc : p.xc;
      e2m1_values(*reinterpret_cast<const uint32_t*>(codes + row * (p.K / 2) + kb * 16 + c * 4),
                  v);
      const float s = e8m0_value((w ? p.ws : p.xs)[mx4_scale_at(row, kb, p.kt)]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= s;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) (w ? sw : sx)[r][c * 8 + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMx4Block; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[j] = fmaf(sx[tid >> 3][k], sw[(tid & 7) + 8 * j][k], acc[j]);
    __syncthreads();
  }
  const int64_t m = m0 + (tid >> 3);
  if (m >= p.M) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t n = n0 + (tid & 7) + 8 * j;
    if (n >= p.N) continue;
    if (p.y_f32) static_cast<float*>(p.y)[m * p.ldy + n] = acc[j];
    else static_cast<__nv_bfloat16*>(p.y)[m * p.ldy + n] = __float2bfloat16_rn(acc[j]);
  }
}

}  // namespace

cudaError_t launch_mx4_gemm(const Mx4GemmParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)(((p.N + kTile - 1) / kTile) * ((p.M + kTile - 1) / kTile)));
  return launch_pdl(gemm_kernel, grid, 256, 0, st, p);
}

}  // namespace ig
