// MX4 product: y[m][n] = sum_k x[m][k] w[n][k], both operands MX4 (mx4.cuh),
// on the tcgen05 tensor cores.
//
// The weights are the MMA's A operand (128 output columns n are its 128
// rows), the tokens its B operand (BN of them), so that a decode batch of up
// to 16 tokens pads the MMA's N, its cheap side, and not its M.
//
// K is cut into S parts of whole 256-k stages; S depends on (N, K) only. Each
// part is one FP32 sum in tensor memory in increasing k, and the S sums are
// added to 0 in increasing order, so that a row's bits do not depend on M.
#include <algorithm>

#include "mx4.cuh"
#include "umma_mx4.cuh"

namespace ig {

namespace {

constexpr int kBM = 128;            // output columns (weight rows) per tile
constexpr int kBK = 256;            // k per stage: 128-byte rows of codes
constexpr int kThreads = 128;
constexpr int kWBytes = kBM * kBK / 2;
constexpr int kMaxStages = 8;

struct Ctl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t done;
  uint32_t tmem;
  int32_t issued;      // stages filled by the producer
  int32_t consumed;    // stages whose copies the MMA thread saw arrive
};

// Stage: W codes, x codes, W scales (2 tiles), x scales (2 tiles per 128 tokens).
__host__ __device__ constexpr int sf_groups(int bn) { return (bn + 127) / 128; }
__host__ __device__ constexpr int x_bytes(int bn) { return bn * kBK / 2; }
__host__ __device__ constexpr int stage_bytes(int bn) {
  return kWBytes + x_bytes(bn) + 2 * kMx4TileBytes * (1 + sf_groups(bn));
}
__host__ __device__ constexpr int stage_pitch(int bn) { return (stage_bytes(bn) + 1023) / 1024 * 1024; }
__host__ __device__ constexpr int stages_of(int bn) { return bn >= 256 ? 4 : bn >= 128 ? 5 : 4; }
// tensor memory: the accumulator, then the scale factors of each stage
__host__ __device__ constexpr int sf_col(int bn) { return bn < 32 ? 32 : bn; }
__host__ __device__ constexpr int sf_cols(int bn) { return 8 * (1 + sf_groups(bn)); }
__host__ __device__ constexpr int tmem_cols(int bn) {
  const int need = sf_col(bn) + stages_of(bn) * sf_cols(bn);
  return need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : 512;
}
// the part's sums [BN tokens][128] FP32 take the place of the stages
__host__ __device__ constexpr size_t smem_bytes(int bn) {
  const size_t ring = (size_t)stages_of(bn) * stage_pitch(bn);
  const size_t sums = (size_t)bn * kBM * 4;
  return 2048 + (ring > sums ? ring : sums);
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

template <int BN>
__global__ void __launch_bounds__(kThreads) gemm_kernel(const __grid_constant__ Mx4GemmParams p) {
  constexpr int NST = stages_of(BN), SG = sf_groups(BN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem);
  uint8_t* ring = smem + 1024;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = p.S;

  uint32_t bid = blockIdx.x;
  const int part = (int)next_digit(bid, (uint32_t)S);
  const int64_t n0 = (int64_t)next_digit(bid, (uint32_t)p.ntiles) * kBM;
  const int64_t m0 = (int64_t)bid * BN;
  const int64_t k0 = (int64_t)part * p.k_part;
  const int64_t k1 = min(p.K, k0 + p.k_part);
  const int nk = (int)((k1 - k0 + kBK - 1) / kBK);
  const int tok = (int)min((int64_t)BN, p.M - m0);         // tokens of the tile
  const int groups = (tok + 127) / 128;                    // their scale row groups

  if (tid == 0) {
    prefetch_tensormap(&p.tm_w);
    prefetch_tensormap(&p.tm_x);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    mbar_init(&ctl->done, 1);
    ctl->issued = ctl->consumed = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem, tmem_cols(BN));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  // The next kernel may start once every block is here: each has its tensor
  // memory by then, so no early block can hold what one of these still needs.
  griddep_launch();

  if (warp == 0 && lane == 0) {
    auto atoms = [&](int b) { return (int)min((int64_t)2, (k1 - k0 - (int64_t)b * kBK + 127) / 128); };
    auto arm = [&](int b) {
      mbar_arrive_expect_tx(&ctl->full[b % NST], (uint32_t)(kWBytes + x_bytes(BN) +
                                                            atoms(b) * kMx4TileBytes * (1 + groups)));
    };
    auto load_w = [&](int b) {
      uint8_t* st = ring + (b % NST) * stage_pitch(BN);
      const int64_t k = k0 + (int64_t)b * kBK;
      tma_load_2d(st, &p.tm_w, (int)(k / 4), (int)n0, &ctl->full[b % NST]);
      bulk_g2s(st + kWBytes + x_bytes(BN),
               p.ws + ((n0 / 128) * p.kt + k / 128) * kMx4TileBytes, atoms(b) * kMx4TileBytes,
               &ctl->full[b % NST]);
    };
    auto load_x = [&](int b) {
      uint8_t* st = ring + (b % NST) * stage_pitch(BN);
      const int64_t k = k0 + (int64_t)b * kBK;
      tma_load_2d(st + kWBytes, &p.tm_x, (int)(k / 4), (int)m0, &ctl->full[b % NST]);
      for (int g = 0; g < groups; ++g)
        bulk_g2s(st + kWBytes + x_bytes(BN) + 2 * kMx4TileBytes * (1 + g),
                 p.xs + ((m0 / 128 + g) * p.kt + k / 128) * kMx4TileBytes,
                 atoms(b) * kMx4TileBytes, &ctl->full[b % NST]);
    };
    const int first = min(nk, NST);
    const bool early = (p.flags & IG_FLAG_STATIC_WEIGHTS) != 0;
    for (int b = 0; b < first; ++b) {
      arm(b);
      if (early) load_w(b);
    }
    griddep_wait();
    for (int b = 0; b < first; ++b) {
      if (!early) load_w(b);
      load_x(b);
    }
    int b = first;
    for (; b < nk; ++b) {
      if (!mbar_wait_bounded(&ctl->empty[b % NST], (uint32_t)((b / NST - 1) & 1), p.status)) break;
      arm(b);
      load_w(b);
      load_x(b);
    }
    ctl->issued = b;
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = umma_idesc_mx4(kBM, BN);
    int b = 0;
    for (; b < nk; ++b) {
      const int s = b % NST;
      if (!mbar_wait_bounded(&ctl->full[s], (uint32_t)((b / NST) & 1), p.status)) break;
      tc_fence_after();
      const uint32_t wa = smem_u32(ring + s * stage_pitch(BN)), xa = wa + kWBytes;
      const uint32_t sfs = xa + x_bytes(BN);
      const uint32_t sfa = tmem + sf_col(BN) + s * sf_cols(BN), sfb = sfa + 8;
      const int64_t rem = k1 - k0 - (int64_t)b * kBK;
      const int steps = (int)min((int64_t)4, (rem + 63) / 64);
      for (int a = 0; a < (steps + 1) / 2; ++a) {
        sf_tile_to_tmem(sfa + 4 * a, sf_tile_desc(sfs + a * kMx4TileBytes));
        for (int g = 0; g < SG; ++g)
          sf_tile_to_tmem(sfb + 4 * (a * SG + g),
                          sf_tile_desc(sfs + (2 * (1 + g) + a) * kMx4TileBytes));
      }
      for (int i = 0; i < steps; ++i)
        umma_mx4(tmem, umma_desc_sw128(wa + 32 * i), umma_desc_sw128(xa + 32 * i),
                 umma_idesc_sf(idesc, 2 * (i & 1)), sfa + 4 * (i >> 1), sfb + 4 * SG * (i >> 1),
                 b > 0 || i > 0);
      umma_commit(&ctl->empty[s]);
    }
    umma_commit(&ctl->done);
    ctl->consumed = b;
  }
  __syncwarp();
  griddep_wait();
  bool ok = mbar_wait_bounded(&ctl->done, 0, p.status);
  __syncthreads();
  if (ctl->issued != nk || ctl->consumed != nk) {
    ok = false;                       // a copy never came: wait for those in flight
    if (tid == 0)
      for (int b = ctl->consumed; b < ctl->issued; ++b)
        mbar_wait_bounded(&ctl->full[b % NST], (uint32_t)((b / NST) & 1), p.status);
    __syncthreads();
  }
  tc_fence_after();

  // the part's sums -> shared memory [token][n], where the stages were
  float* sums = reinterpret_cast<float*>(ring);
  for (int c = 0; c < BN && c < tok; c += 32) {
    float v[32];
    tmem_ld32(tmem + ((uint32_t)(warp * 32) << 16) + c, v);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (BN >= 32 || i < BN) sums[(c + i) * kBM + tid] = v[i];
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, tmem_cols(BN));
  if (S > 1) cluster_sync_all();

  // block `part` of the cluster adds up and stores its share of the tokens
  const int share = (BN + S - 1) / S;
  const int n = 4 * lane;
  if (n0 + n < p.N && ok) {
    for (int t = part * share + warp; t < min((part + 1) * share, tok); t += kThreads / 32) {
      const float* own = sums + t * kBM + n;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int s = 0; s < S; ++s) {
        const float4 u = S == 1 ? *reinterpret_cast<const float4*>(own)
                                : ld_cluster_v4(map_rank(own, s));
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
      }
      const int64_t at = (m0 + t) * p.ldy + n0 + n;
      if (p.y_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = v;
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + at) =
            make_uint2(f32x2_to_bf16x2_bits(v.x, v.y), f32x2_to_bf16x2_bits(v.z, v.w));
    }
  }
  if (S > 1) cluster_sync_all();    // no block leaves while its sums are being read
}

template <int BN>
cudaError_t launch_bn(Mx4GemmParams& p, cudaStream_t st) {
  auto kern = gemm_kernel<BN>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem_bytes(BN));
  if (e != cudaSuccess) return e;
  if (encode_map_2d(&p.tm_x, p.xc, (uint64_t)p.M, (uint64_t)p.K / 4, (uint64_t)p.K / 2, 64, BN,
                    CU_TENSOR_MAP_SWIZZLE_128B) != IG_OK)
    return cudaErrorInvalidValue;
  const int64_t grid = (p.M + BN - 1) / BN * p.ntiles * p.S;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(BN);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.S;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx4_gemm(Mx4GemmParams& p, cudaStream_t st) {
  p.ntiles = (int32_t)((p.N + kBM - 1) / kBM);
  const int64_t stages = (p.K + kBK - 1) / kBK;
  int S = 1;
  while (S < 8 && (int64_t)p.ntiles * S < 128 && stages >= 4 * S) S *= 2;
  const int64_t per = (stages + S - 1) / S;
  p.k_part = per * kBK;
  p.S = (int32_t)((stages + per - 1) / per);   // no part is empty
  if (p.M > 512) return launch_mx4_gemm_pair(p, sm_count(), st);
  if (encode_map_2d(&p.tm_w, p.wc, (uint64_t)p.N, (uint64_t)p.K / 4, (uint64_t)p.K / 2, 64, kBM,
                    CU_TENSOR_MAP_SWIZZLE_128B) != IG_OK)
    return cudaErrorInvalidValue;
  if (p.M <= 16) return launch_bn<16>(p, st);
  if (p.M <= 32) return launch_bn<32>(p, st);
  if (p.M <= 64) return launch_bn<64>(p, st);
  if (p.M <= 128) return launch_bn<128>(p, st);
  return launch_bn<256>(p, st);
}

}  // namespace ig
