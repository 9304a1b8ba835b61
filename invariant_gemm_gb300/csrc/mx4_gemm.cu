// MX4 product: y[m][n] = sum_k x[m][k] w[n][k], both operands MX4 (mx4.cuh),
// on the tcgen05 tensor cores. This file: few tokens; mx4_gemm_pair.cu: many.
//
// The weights are the MMA's A operand (128 output columns n are its 128
// rows), the tokens its B operand (BN of them), so that a decode batch of up
// to 16 tokens pads the MMA's N, its cheap side, and not its M.
//
// K is cut into S parts of whole 256-k stages; S depends on (N, K) only. Each
// part is one FP32 sum in tensor memory in increasing k, and the S sums are
// added to 0 in increasing order, so that a row's bits do not depend on M. A
// part is a block here, the S blocks of a tile a cluster: each sends its sums,
// four tokens at a time, to the block that owns those tokens (the groups of
// four go round the blocks) through distributed shared memory, and the owner
// adds and stores them. A warp whose sums never came says so to the owners and
// counts its bytes as sent, so an owner's wait ends on every path, and never
// while sums are on their way to it.
//
// With few tokens the weights' bytes bound it: nearly all of shared memory is
// a ring of copies (17 KB of weights to a stage), and with
// IG_FLAG_STATIC_WEIGHTS the ring is filled while the kernel before ends. M = 16,
// K = 28672, N = 8192: 21.5 us, 5.8 TB/s. Small weights are over in the time from
// the first copy to the last store: M = 1, N = K = 4096 3.9 us, for 1.3 us of
// bytes.
//
// Warps: 0-3 take the sums out of tensor memory, 4 copies the weights, 6 the
// tokens, 5 issues the MMAs. Two warps copy because the tokens wait for the
// kernel before and static weights do not: with both after that wait M = 1, N =
// K = 4096 takes 4.7 us.
#include <algorithm>
#include <atomic>

#include "mx4.cuh"
#include "umma_mx4.cuh"

namespace ig {

namespace {

constexpr int kBM = 128;            // output columns (weight rows) per tile
constexpr int kBK = 256;            // k per stage: 128-byte rows of codes
constexpr int kCopyWarp = 4, kMmaWarp = 5, kCopyXWarp = 6;
constexpr int kThreads = 224;
constexpr int kWBytes = kBM * kBK / 2;
constexpr int kMaxStages = 10;

struct Ctl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t done;       // `consumed` is known, and the MMAs are complete
  uint64_t parts;      // the other blocks' sums (and the own ones) have come
  uint32_t tmem;
  int32_t issued[2];   // stages filled: weights, tokens
  int32_t consumed;    // stages whose copies the MMA thread saw arrive
  uint32_t missing;    // some sums of this owner's tokens never came
};

// Stage: W codes, x codes, W scales (2 tiles), x scales (2 tiles). A token tile
// (up to 128 tokens) lies in one scale row group of 128.
__host__ __device__ constexpr int x_bytes(int bn) { return bn * kBK / 2; }
__host__ __device__ constexpr int stage_bytes(int bn) {
  return kWBytes + x_bytes(bn) + 4 * kMx4TileBytes;
}
// tensor memory: the sums, then the scale factors of each stage
__host__ __device__ constexpr int sf_col(int bn) { return bn < 32 ? 32 : bn; }
constexpr int kSfCols = 16;
// The parts' sums [S][groups of four tokens of this owner][128][4] FP32: BN *
// 512 bytes, a little more where S does not divide the groups. Beside the ring
// for up to 32 tokens; else in its place once every block of the cluster is
// through with it (64 tokens, two blocks to an SM: a fourth stage instead, M =
// 256, N = K = 4096 8.6 -> 8.2 us). With one part they are not needed: the sums
// go from registers to memory.
__host__ __device__ constexpr bool own_sums(int bn) { return bn <= 32; }
__host__ __device__ inline int share_of(int bn, int S) { return (bn / 4 + S - 1) / S; }
__host__ __device__ inline int sums_bytes(int bn, int S) {
  return S > 1 ? share_of(bn, S) * S * kBM * 16 : 0;
}

// Four tokens' results of column n (0-127 of the tile; lanes hold neighbouring
// columns), tokens t0 ... of the tile, of which `tok` exist. y: the tile's
// first token and column.
template <typename T>
__device__ __forceinline__ void store4(T* y, int64_t ld, int n, bool in, int t0, int tok,
                                       const float4& v) {
  if constexpr (sizeof(T) == 4) {
    T* o = y + t0 * ld + n;
    if (in && t0 < tok) *o = v.x;
    if (in && t0 + 1 < tok) o[ld] = v.y;
    if (in && t0 + 2 < tok) o[2 * ld] = v.z;
    if (in && t0 + 3 < tok) o[3 * ld] = v.w;
  } else {
    // lanes 2 l, 2 l + 1 trade the rounded values of two tokens: the even one
    // stores both columns of tokens 0 and 2, the odd one of 1 and 3
    const bool odd = n & 1;
    const uint32_t pick = odd ? 0x3276u : 0x5410u;
    const uint32_t a = f32x2_to_bf16x2_bits(v.x, v.y), b = f32x2_to_bf16x2_bits(v.z, v.w);
    T* o = y + (t0 + odd) * ld + (n & ~1);
    const uint32_t va = __byte_perm(a, __shfl_xor_sync(0xffffffffu, a, 1), pick);
    const uint32_t vb = __byte_perm(b, __shfl_xor_sync(0xffffffffu, b, 1), pick);
    if (in && t0 + odd < tok) *reinterpret_cast<uint32_t*>(o) = va;
    if (in && t0 + 2 + odd < tok) *reinterpret_cast<uint32_t*>(o + 2 * ld) = vb;
  }
}

// Takes `bytes` off what a barrier of the cluster waits for, after setting the
// word at `flag` of the same block: a thread that sees the barrier's phase end
// sees the word.
__device__ __forceinline__ void give_up(uint32_t flag, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "st.shared::cluster.u32 [%0], 1;\n\t"
      "fence.acq_rel.cluster;\n\t"
      "mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%1], %2;"
      ::"r"(flag), "r"(bar), "r"(bytes) : "memory");
}

template <int BN>
__global__ void __launch_bounds__(kThreads) gemm_kernel(const __grid_constant__ Mx4GemmParams p) {
  constexpr int kStage = stage_bytes(BN);
  static_assert(kStage % 1024 == 0, "swizzled tiles start at multiples of 1024 bytes");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem);
  const int tid = threadIdx.x, warp = (int)uniform(tid >> 5), lane = tid & 31;
  const int S = p.S, NST = p.stages;
  uint8_t* ring = smem + 1024;
  float4* sums = reinterpret_cast<float4*>(own_sums(BN) ? ring + NST * kStage : ring);

  uint32_t bid = blockIdx.x;
  const int part = (int)next_digit(bid, (uint32_t)S);      // the block's rank in its cluster
  const int64_t n0 = (int64_t)next_digit(bid, (uint32_t)p.ntiles) * kBM;
  const int64_t m0 = (int64_t)bid * BN;
  const int64_t k0 = (int64_t)part * p.k_part;
  const int64_t k1 = min(p.K, k0 + p.k_part);
  const int nk = (int)((k1 - k0 + kBK - 1) / kBK);
  const int tok = (int)min((int64_t)BN, p.M - m0);         // tokens of the tile
  const int share = share_of(BN, S);
  const int quads = (tok + 3) / 4;                         // groups of four tokens
  auto owned_by = [&](int q) { return quads > q ? (quads - q - 1) / S + 1 : 0; };
  const int owned = owned_by(part);

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&ctl->full[i], 2);
      mbar_init(&ctl->empty[i], 1);
    }
    mbar_init(&ctl->done, 2);
    mbar_init(&ctl->parts, 1);
    ctl->issued[0] = ctl->issued[1] = ctl->consumed = 0;
    ctl->missing = 0;
    fence_mbar_init();
    if (S > 1) mbar_arrive_expect_tx(&ctl->parts, (uint32_t)(S * owned * kBM * 16));
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(ctl->tmem);
  if (S > 1 && own_sums(BN)) cluster_arrive_relaxed();

  bool ok = true;
  if (warp == kCopyWarp || warp == kCopyXWarp) {
    // Whole warps go through the loop and one lane issues.
    const bool leader = elect_one();
    const bool w = warp == kCopyWarp;
    const bool early = w && (p.flags & IG_FLAG_STATIC_WEIGHTS) != 0;
    const CUtensorMap* map = w ? &p.tm_w : &p.tm_x;
    const int row = (int)(w ? n0 : m0);
    const uint8_t* sf = (w ? p.ws : p.xs) + ((int64_t)(row >> 7) * p.kt + k0 / 128) * kMx4TileBytes;
    const uint32_t bytes = w ? kWBytes : x_bytes(BN);
    const int kc = (int)(k0 / 4);
    const int ntile = (int)((k1 - k0 + 127) / 128);       // scale tiles
    if (leader) prefetch_tensormap(map);
    if (!early) griddep_wait();
    // The next kernel may start once every block is here, all work before this
    // kernel is complete, and each block has its tensor memory: so no early
    // block can hold what one of these still needs.
    if (!w) griddep_launch();
    int b = 0, s = 0;
    uint32_t parity = 1;      // a stage's first use finds its barrier in the phase before
    for (; b < nk; ++b) {
      if (!warp_wait(&ctl->empty[s], parity, p.status)) break;
      if (leader) {
        const uint32_t sfb = (2 * b + 1 < ntile ? 2 : 1) * kMx4TileBytes;
        uint8_t* st = ring + s * kStage;
        uint8_t* st_sf = st + kWBytes + x_bytes(BN);
        mbar_arrive_expect_tx(&ctl->full[s], bytes + sfb);
        tma_load_2d(w ? st : st + kWBytes, map, kc + b * 64, row, &ctl->full[s]);
        bulk_g2s(w ? st_sf : st_sf + 2 * kMx4TileBytes, sf, sfb, &ctl->full[s]);
        sf += 2 * kMx4TileBytes;
      }
      if (++s == NST) {
        s = 0;
        parity ^= 1;
        griddep_wait();         // no bounded wait for a free stage spans the kernel before
      }
    }
    if (leader) ctl->issued[w ? 0 : 1] = b;
    __syncwarp();
    griddep_wait();
  } else if (warp == kMmaWarp) {
    constexpr uint32_t idesc0 = umma_idesc_mx4(kBM, BN), idesc1 = umma_idesc_sf(idesc0, 2);
    const uint64_t wd = umma_desc_sw128(smem_u32(ring)),
                   xd = umma_desc_sw128(smem_u32(ring) + kWBytes),
                   sfd = sf_tile_desc(smem_u32(ring) + kWBytes + x_bytes(BN));
    // A column holds the scales of 32 rows, and a 64-token tile may start at
    // row 64 of its group of 128, two columns on. (An odd column is not a valid
    // start: 32-token tiles only ever start at row 0.)
    const uint32_t shift = (uint32_t)(m0 & 127) / 32;
    const bool leader = elect_one();
    int b = 0, s = 0;
    uint32_t parity = 0;
    griddep_wait();           // as the tokens' copies do: the bounded waits start here
    for (; b < nk; ++b) {
      const bool expire = b == 0 && (p.flags & IG_FLAG_TEST_COPY_TIMEOUT) != 0;
      if (!warp_wait(&ctl->full[s], parity, p.status, expire ? 0 : 1ll << 31)) break;
      tc_fence_after();
      const uint64_t w = wd + s * (kStage >> 4), x = xd + s * (kStage >> 4);
      const uint64_t sf = sfd + s * (kStage >> 4);
      const uint32_t sfa = tmem + sf_col(BN) + s * kSfCols, sfc = sfa + 8, sfb = sfc + shift;
      const int rem = (int)min((int64_t)kBK, k1 - k0 - (int64_t)b * kBK);
      if (leader) {
        sf_tile_to_tmem(sfa, sf);
        sf_tile_to_tmem(sfc, sf + 64);
        umma_mx4(tmem, w, x, idesc0, sfa, sfb, b > 0);
        if (rem > 64) umma_mx4(tmem, w + 2, x + 2, idesc1, sfa, sfb, true);
        if (rem > 128) {
          sf_tile_to_tmem(sfa + 4, sf + 32);
          sf_tile_to_tmem(sfc + 4, sf + 96);
          umma_mx4(tmem, w + 4, x + 4, idesc0, sfa + 4, sfb + 4, true);
        }
        if (rem > 192) umma_mx4(tmem, w + 6, x + 6, idesc1, sfa + 4, sfb + 4, true);
        umma_commit(&ctl->empty[s]);
      }
      __syncwarp();
      if (++s == NST) {
        s = 0;
        parity ^= 1;
      }
    }
    if (leader) {
      ctl->consumed = b;
      mbar_arrive(&ctl->done);
      umma_commit(&ctl->done);
    }
    __syncwarp();
  } else {
    griddep_wait();
    ok = warp_wait(&ctl->done, 0, p.status) && ctl->consumed == nk;
    tc_fence_after();
  }
  if (!own_sums(BN)) {
    // the sums take the place of the stages
    __syncthreads();
    if (S > 1) cluster_arrive_relaxed();
  }
  if (S > 1) cluster_wait();

  float* y32 = static_cast<float*>(p.y) + m0 * p.ldy + n0;
  __nv_bfloat16* y16 = static_cast<__nv_bfloat16*>(p.y) + m0 * p.ldy + n0;
  if (warp < 4 && ok) {
    int owner = 0, at = 0;
    for (int c = 0; c < tok; c += 32) {
      float v[32];
      tmem_ld32(tmem + ((uint32_t)(warp * 32) << 16) + c, v);
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        if (c + i >= tok) continue;
        float4 q = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        if (S == 1) {
          q.x += 0.0f; q.y += 0.0f; q.z += 0.0f; q.w += 0.0f;
          const bool in = n0 + tid < p.N;
          if (p.y_f32) store4(y32, p.ldy, tid, in, c + i, tok, q);
          else store4(y16, p.ldy, tid, in, c + i, tok, q);
        } else {
          st_async_v4(map_rank(sums + (part * share + at) * kBM + tid, owner), q,
                      map_rank(&ctl->parts, owner));
          if (++owner == S) {
            owner = 0;
            ++at;
          }
        }
      }
    }
    tc_fence_before();
  } else if (S > 1 && warp < 4 && lane < min(S, quads)) {
    give_up(map_rank(&ctl->missing, lane), map_rank(&ctl->parts, lane), owned_by(lane) * 32 * 16);
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, p.tmem_cols);
  if (ctl->issued[0] != nk || ctl->issued[1] != nk || ctl->consumed != nk) {
    // a copy never came: wait for those in flight (the last to each stage),
    // store nothing
    ok = false;
    const int last = max(ctl->issued[0], ctl->issued[1]);
    if (tid == 0)
      for (int b = max(0, last - NST); b < last; ++b)
        mbar_wait_bounded(&ctl->full[b % NST], (b / NST) & 1, p.status, 1ll << 28);
    __syncthreads();
  }
  // The wait outlasts any sender's own bounded waits.
  if (S > 1)
    ok = mbar_wait_bounded(&ctl->parts, 0, p.status, 1ll << 36) && ok &&
         *static_cast<volatile uint32_t*>(&ctl->missing) == 0;

  // The owner of four tokens adds their sums up in order and stores them: a
  // lane two neighbouring columns, a warp 64, a line of 128 bytes in bf16.
  if (S == 1 || !__all_sync(0xffffffffu, ok)) return;
  for (int u = warp; u < 2 * owned; u += kThreads / 32) {
    const int g = u >> 1, n = (u & 1) * 64 + 2 * lane;
    if (n0 + n >= p.N) continue;
    float v[4][2] = {};
    for (int s = 0; s < S; ++s) {
      const float4* t = sums + (s * share + g) * kBM + n;
      const float4 a = t[0], b = t[1];
      v[0][0] += a.x; v[1][0] += a.y; v[2][0] += a.z; v[3][0] += a.w;
      v[0][1] += b.x; v[1][1] += b.y; v[2][1] += b.z; v[3][1] += b.w;
    }
    const int t0 = 4 * (part + g * S);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (t0 + i >= tok) break;
      const int64_t at = (t0 + i) * p.ldy + n;
      if (p.y_f32) *reinterpret_cast<float2*>(y32 + at) = make_float2(v[i][0], v[i][1]);
      else *reinterpret_cast<uint32_t*>(y16 + at) = f32x2_to_bf16x2_bits(v[i][0], v[i][1]);
    }
  }
}

template <int BN>
cudaError_t launch_bn(Mx4GemmParams& p, cudaStream_t st) {
  const int64_t grid = (p.M + BN - 1) / BN * p.ntiles * p.S;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // The ring: all of shared memory where every block has an SM to itself, else
  // half of it. Stages past the part's are of no use.
  const int sums = sums_bytes(BN, p.S);
  const int room = (grid <= sm_count() ? 220 : 110) * 1024 - (own_sums(BN) ? sums : 0);
  const int64_t nk = p.k_part / kBK;
  p.stages = (int32_t)std::min<int64_t>({kMaxStages, room / stage_bytes(BN), nk});
  const int cols = sf_col(BN) + p.stages * kSfCols;
  p.tmem_cols = cols <= 64 ? 64 : cols <= 128 ? 128 : cols <= 256 ? 256 : 512;
  const int ring = p.stages * stage_bytes(BN);
  const int smem = 2048 + (own_sums(BN) ? ring + sums : std::max(ring, sums));
  auto kern = gemm_kernel<BN>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), allowed);
  if (e != cudaSuccess) return e;
  if (encode_map_2d(&p.tm_x, p.xc, (uint64_t)p.M, (uint64_t)p.K / 4, (uint64_t)p.K / 2, 64, BN,
                    CU_TENSOR_MAP_SWIZZLE_128B) != IG_OK)
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.S;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// Which kernel is through soonest with more than 64 tokens, by a start and so
// much for each stage of K in hundredths of a microsecond (fitted to the times
// of 35 sizes, M 192-10000, N 128-12288, K 288-28672, within 20%). Here, the
// blocks of an SM count one by one, which has two at a time: tiles of 64 tokens
// only while all are at work at once; of 128 in waves (a last tile of up to 64
// tokens counts half). Pairs: rounds of tiles, 24 a stage for a last round of
// half tiles. us with 64 / 128 / pairs: M = 256, N = K = 4096 7.8 / 8.5 / 9.2; M
// = 192, K = 28672, N = 12288 43.5 / - / 40.1; 128 / pairs: M = 384, K = 4096, N =
// 2560 7.6 / 9.0; M = 512 11.0 / 9.3; M = 400, K = 11008 13.6 / 15.5; M = 512 19.8 /
// 15.8; M = 900, K = 28672, N = 520 19.5 / 31.2.
enum class Kind { k64, k128, kPairs };
Kind soonest(const Mx4GemmParams& p, int64_t stages, int64_t per) {
  const int64_t sms = sm_count(), pairs = sms / 2, halves = (p.M + 63) / 64;
  auto deep = [&](int64_t blocks) {
    return blocks > sms ? (blocks + 2 * sms - 1) / (2 * sms) * 2 : 1;
  };
  const int64_t b64 = halves * p.ntiles * p.S, b128 = (b64 + 1) / 2;
  const int64_t tiles = (p.N + 255) / 256 * ((p.M + 255) / 256), rest = tiles % pairs;
  const int64_t t64 = 420 + 18 * deep(b64) * per;
  const int64_t t128 = 300 + deep(b128) * (130 + 35 * per);
  const int64_t tpair =
      540 + (33 * (tiles / pairs) + (rest == 0 ? 0 : 2 * rest <= pairs ? 24 : 33)) * stages;
  if (b64 <= 2 * sms && t64 <= std::min(t128, tpair)) return Kind::k64;
  return t128 <= tpair ? Kind::k128 : Kind::kPairs;
}

}  // namespace

cudaError_t launch_mx4_gemm(Mx4GemmParams& p, cudaStream_t st) {
  p.ntiles = (int32_t)((p.N + kBM - 1) / kBM);
  // Parts of K: enough blocks for most SMs where the columns alone are few, and
  // no part under 8 stages, since the pairs of many tokens pay for each part.
  // N = K = 4096, us for M = 1 / 256 / 4096: S = 1 5.2 / 7.7 / 27.6, S = 2 3.9 /
  // 7.9 / 29.7, S = 4 3.4 / 9.6 / 35.8; N = 8192, K = 28672, M = 16 / 8192: 25.3 /
  // 506, 21.4 / 505, 20.7 / 512.
  const int64_t stages = (p.K + kBK - 1) / kBK;
  int S = 1;
  while (S < 8 && (int64_t)p.ntiles * S < 96 && stages >= 16 * S) S *= 2;
  const int64_t per = (stages + S - 1) / S;
  p.k_part = per * kBK;
  p.S = (int32_t)((stages + per - 1) / per);   // no part is empty
  const Kind kind = p.M > 64 ? soonest(p, stages, per) : Kind::k64;
  if (kind == Kind::kPairs) return launch_mx4_gemm_pair(p, sm_count(), st);
  if (encode_map_2d(&p.tm_w, p.wc, (uint64_t)p.N, (uint64_t)p.K / 4, (uint64_t)p.K / 2, 64, kBM,
                    CU_TENSOR_MAP_SWIZZLE_128B) != IG_OK)
    return cudaErrorInvalidValue;
  if (p.M <= 16) return launch_bn<16>(p, st);
  if (p.M <= 32) return launch_bn<32>(p, st);
  if (kind == Kind::k64) return launch_bn<64>(p, st);
  return launch_bn<128>(p, st);
}

}  // namespace ig
