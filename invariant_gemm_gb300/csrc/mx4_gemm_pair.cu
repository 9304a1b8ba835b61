// MX4 product for many tokens: the sums of mx4_gemm.cu, computed by pairs of
// blocks that share each MMA (cta_group::2).
//
// A pair takes tiles of 256 output columns x 256 tokens, one after the other:
// each of its two blocks holds 128 of the weight rows and 128 of the token
// rows, so that shared memory is filled and read at 16 KB + 16 KB per 256 k
// and block, where a block alone would need 16 KB + 32 KB for the same
// products. Both blocks keep 128 x 256 sums in tensor memory.
//
// Warps: 0-15 take the sums out of tensor memory (32 lanes and a quarter of
// the columns each), 16 copies, 17 (of the first block) issues the MMAs. The
// sums of a part of K go to registers at once (64 a thread) and tensor memory is
// free again: the stores of a tile run beside the products of the next.
//
// Bound by the tensor cores, and they by the board's power: M = N = 8192, K =
// 28672 498 us (7.7 PFLOP/s), 98% of the cycles in MMAs at 128 cycles each (K =
// 64), at a clock of about 1.5 GHz; M = 4096, K = 4096, N = 12288 64 us, 84% of the
// cycles (about 900 from a tile's last MMA to the next tile's first, and 10.1
// rounds of tiles), 76 us with an FP32 result. With K up to 512 by the stores, a
// tile's 5200 cycles in 64-byte pieces: M = N = 8192, K = 64 40 us (3.3 TB/s).
#include <atomic>

#include "mx4.cuh"
#include "umma_mx4.cuh"

namespace ig {

namespace {

constexpr int kBN = 256;                 // output columns per tile (128 per block)
constexpr int kBT = 256;                 // tokens per tile (128 rows of codes per block)
constexpr int kBK = 256;                 // k per stage
constexpr int kHalf = 128 * kBK / 2;     // codes of 128 rows
constexpr int kStage = 2 * kHalf + 6 * kMx4TileBytes;   // w, x, w scales (2 tiles), x scales (4)
constexpr int kHalfStage = kStage - kHalf / 2 - 2 * kMx4TileBytes;      // with 128 tokens
constexpr int kStages = 6;
constexpr int kEpiWarps = 16;
constexpr int kCols = kBT / (kEpiWarps / 4);   // token columns per warp
constexpr int kCopyWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
constexpr int kThreads = 32 * (kEpiWarps + 2);
constexpr uint32_t kSfCol = 256;         // tensor memory: sums 0-255, then scales
constexpr uint32_t kSfCols = 8 + 16;     // per stage: w 2 x 4, x 2 x 8
constexpr uint32_t kTmemCols = 512;
constexpr int kGroup = 16;               // token tiles that run through the columns together

struct Ctl {
  uint64_t full[kStages];       // of the first block: the copies of both blocks
  uint64_t empty[kStages];      // own: the MMAs that read the stage are done
  uint64_t sums_full;           // own: a part's sums are complete
  uint64_t sums_empty;          // of the first block: all warps have taken them out
  uint32_t tmem;
  int32_t fail;
};

constexpr size_t kSmem = 2048 + (size_t)kStages * kStage;

// A stage of the ring and the parity of its barriers' current phase.
struct Slot {
  uint32_t s = 0, parity = 0;
  __device__ __forceinline__ void next() {
    if (++s == kStages) {
      s = 0;
      parity ^= 1;
    }
  }
};

__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int c0, int c1,
                                              uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// Scale tile of each block's own shared memory -> its own tensor memory.
__device__ __forceinline__ void sf_tile_to_tmem_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

__device__ __forceinline__ void umma_mx4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                              bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X "
      "[%0], %1, %2, %3, [%4], [%5], p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb),
        "r"((uint32_t)accumulate)
      : "memory");
}

// One arrival on the barrier of both blocks of the pair once all earlier
// tcgen05 operations of this thread have completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}

// Arrival on a barrier of either block. It orders tensor memory (with the
// fences around it), not shared or global memory: nothing but tensor memory is
// handed over, and the cluster-wide release would make the warp wait for its
// stores.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

// 8 consecutive FP32 columns of this thread's lane (see tmem_ld32).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

struct Tile {
  int n0, m0;
  int rows;        // of its token rows, those that each block copies: 128 or 64
};

// Piece i: tile i, and from `whole` on half a tile, 128 tokens. Token tiles in
// groups of kGroup; within a group all column tiles, each with the group's
// token tiles, so that the pairs at work at a time share both operands in L2.
__device__ __forceinline__ Tile tile_at(uint32_t i, uint32_t whole, uint32_t nt, uint32_t mt) {
  const uint32_t half = i < whole ? 0 : (i - whole) & 1;
  const int rows = i < whole ? kBT / 2 : kBT / 4;
  if (i >= whole) i = whole + (i - whole) / 2;
  const uint32_t per = kGroup * nt;
  const uint32_t g = i / per, r = i - g * per;
  const uint32_t gm = min((uint32_t)kGroup, mt - g * kGroup);
  const uint32_t n = r / gm;
  return {(int)(n * kBN), (int)((g * kGroup + (r - n * gm)) * kBT + half * (kBT / 2)), rows};
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_pair_kernel(const __grid_constant__ Mx4GemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem);
  uint8_t* ring = smem + 1024;
  const int tid = threadIdx.x, warp = (int)uniform(tid >> 5), lane = tid & 31;
  const uint32_t rank = uniform(cluster_rank());
  const uint32_t nt = (uint32_t)((p.N + kBN - 1) / kBN), mt = (uint32_t)((p.M + kBT - 1) / kBT);
  // The last round of tiles, if it would give work to no more than half the
  // pairs, is cut into half tiles, which take three quarters of the time (us
  // before -> after: M = 384, K = 11008, N = 4096, 32 tiles 19.1 -> 16.4; M = N =
  // K = 4096, 256 tiles 28.9 -> 28.4; M = N = 8192, K = 28672 504 -> 498). The
  // bits stay: a sum's order is that of k alone.
  const uint32_t pairs = gridDim.x / 2, rest = nt * mt % pairs;
  const uint32_t whole = nt * mt - (2 * rest <= pairs ? rest : 0);
  const uint32_t pieces = whole + 2 * (nt * mt - whole);
  // k-blocks (stages) of a tile and of a part of K
  const int nkb = (int)((p.K + kBK - 1) / kBK), per_part = (int)(p.k_part / kBK);

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    mbar_init(&ctl->sums_full, 1);
    mbar_init(&ctl->sums_empty, 2 * kEpiWarps);
    ctl->fail = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(&ctl->tmem)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();        // barriers of both blocks are ready, both have their tensor memory
  tc_fence_after();
  const uint32_t tmem = uniform(ctl->tmem);
  griddep_wait();
  griddep_launch();

  // this pair's pieces, and their stages one after the other
  const uint32_t first = blockIdx.x / 2;
  const int64_t total = first < pieces ? (int64_t)((pieces - first - 1) / pairs + 1) * nkb : 0;

  // Copies. The whole warp goes through the loops and one lane issues: code
  // that the compiler knows to be uniform issues a copy in a few cycles, and a
  // second warp for the scales would gain nothing.
  if (warp == kCopyWarp) {
    const bool leader = elect_one();
    const uint32_t bar0 = map_rank(ctl->full, 0);
    const int kt = (int)p.kt;
    bool ok = true;
    Slot at;
    for (uint32_t i = first; i < pieces && ok; i += pairs) {
      const Tile t = tile_at(i, whole, nt, mt);
      const int wr = t.n0 + 128 * (int)rank, xr = t.m0 + t.rows * (int)rank;
      const bool full_tile = t.rows == 128;
      // scale tiles, as rows of the maps; rows past the last one (of rows of
      // the operands that do not exist) are filled with zeros
      int wrow = ((t.n0 >> 7) + (int)rank) * kt, xrow = (t.m0 >> 7) * kt;
      for (int kb = 0; kb < nkb; ++kb, at.next(), wrow += 2, xrow += 2) {
        // a stage's first use finds its barrier in the phase before: parity 1 passes
        if (!warp_wait(&ctl->empty[at.s], at.parity ^ 1, p.status)) {
          ok = false;
          break;
        }
        if (leader) {
          const uint32_t full = bar0 + 8 * at.s;
          if (rank == 0)
            mbar_arrive_expect_tx(&ctl->full[at.s], 2 * (full_tile ? kStage : kHalfStage));
          uint8_t* st = ring + at.s * kStage;
          uint8_t* sf = st + 2 * kHalf;
          tma_load_pair(st, &p.tm_w, kb * 64, wr, full);
          tma_load_pair(st + kHalf, &p.tm_x, kb * 64, xr, full);
          if (full_tile) tma_load_pair(st + kHalf + kHalf / 2, &p.tm_x, kb * 64, xr + 64, full);
          tma_load_pair(sf, &p.tm_ws, 0, wrow, full);
          tma_load_pair(sf + 2 * kMx4TileBytes, &p.tm_xs, 0, xrow, full);
          if (full_tile) tma_load_pair(sf + 4 * kMx4TileBytes, &p.tm_xs, 0, xrow + kt, full);
        }
      }
    }
    if (!ok && leader) ctl->fail = 1;
  } else if (warp == kMmaWarp) {
    if (rank == 0) {
      constexpr uint32_t of_tile = umma_idesc_mx4(256, kBT), of_half = umma_idesc_mx4(256, kBT / 2);
      const uint64_t wd = umma_desc_sw128(smem_u32(ring)),
                     xd = umma_desc_sw128(smem_u32(ring) + kHalf),
                     sfd = sf_tile_desc(smem_u32(ring) + 2 * kHalf);
      const bool leader = elect_one();
      Slot at;
      int kb = 0, part_end = 0;
      uint32_t part = 0, i = first;
      bool ok = true;
      for (int64_t it = 0; it < total; ++it, at.next()) {
        const bool begin = kb == part_end || kb == 0;
        if (begin) {
          part_end = min(nkb, kb + per_part);
          ok = part == 0 || warp_wait(&ctl->sums_empty, (part - 1) & 1, p.status);
        }
        const bool expire = it == 0 && (p.flags & IG_FLAG_TEST_COPY_TIMEOUT) != 0;
        ok = ok && warp_wait(&ctl->full[at.s], at.parity, p.status, expire ? 0 : 1ll << 31);
        if (!ok) break;
        tc_fence_after();
        const uint64_t w = wd + at.s * (kStage >> 4), x = xd + at.s * (kStage >> 4);
        const uint32_t sfa = tmem + kSfCol + at.s * kSfCols, sfb = sfa + 8;
        const int rem = (int)min((int64_t)kBK, p.K - (int64_t)kb * kBK);
        const bool end = kb + 1 == part_end, full_tile = i < whole;
        const uint32_t idesc0 = full_tile ? of_tile : of_half, idesc1 = umma_idesc_sf(idesc0, 2);
        const uint64_t sf = sfd + at.s * (kStage >> 4);      // tiles w0 w1 x0 x0' x1 x1'
        if (leader) {
          sf_tile_to_tmem_pair(sfa, sf);
          sf_tile_to_tmem_pair(sfb, sf + 64);
          if (full_tile) sf_tile_to_tmem_pair(sfb + 4, sf + 128);
          umma_mx4_pair(tmem, w, x, idesc0, sfa, sfb, !begin);
          if (rem > 64) umma_mx4_pair(tmem, w + 2, x + 2, idesc1, sfa, sfb, true);
          if (rem > 128) {
            sf_tile_to_tmem_pair(sfa + 4, sf + 32);
            sf_tile_to_tmem_pair(sfb + 8, sf + 96);
            if (full_tile) sf_tile_to_tmem_pair(sfb + 12, sf + 160);
            umma_mx4_pair(tmem, w + 4, x + 4, idesc0, sfa + 4, sfb + 8, true);
          }
          if (rem > 192) umma_mx4_pair(tmem, w + 6, x + 6, idesc1, sfa + 4, sfb + 8, true);
          umma_commit_pair(&ctl->empty[at.s]);
          if (end) umma_commit_pair(&ctl->sums_full);
        }
        __syncwarp();
        ++kb;
        if (end) {
          ++part;
          if (kb == nkb) {
            kb = 0;
            i += pairs;
          }
        }
      }
      if (!ok && leader) ctl->fail = 1;
    }
  } else {
    const uint32_t empty = map_rank(&ctl->sums_empty, 0);
    const int c0 = (warp >> 2) * kCols;                 // this warp's token columns
    const uint32_t src = tmem + ((uint32_t)((warp & 3) * 32) << 16) + c0;
    uint32_t part = 0;
    bool ok = true;
    for (uint32_t i = first; i < pieces && ok; i += pairs) {
      const Tile t = tile_at(i, whole, nt, mt);
      const bool mine = c0 < 2 * t.rows;       // the upper columns are not there in half a tile
      float acc[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) acc[j] = 0.0f;
      for (int kb0 = 0; kb0 < nkb; kb0 += per_part, ++part) {
        if (!warp_wait(&ctl->sums_full, part & 1, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kCols / 8; ++c) {
          if (!mine) break;
          float v[8];
          tmem_ld8(src + 8 * c, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[8 * c + j] += v[j];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(empty);
      }
      if (!ok) break;
      const int64_t n = t.n0 + 128 * (int)rank + (warp & 3) * 32;
      const int64_t m = t.m0 + c0;
      // the row stride, opaque to the compiler: multiples of it that are kept
      // over tiles would cost the registers that hold the sums
      int64_t ld = p.ldy;
      asm volatile("" : "+l"(ld));
      const int left = mine ? (int)min((int64_t)kCols, p.M - m) : 0;   // tokens of these columns
      if (p.y_f32) {
        float* y = static_cast<float*>(p.y) + m * ld + n + lane;
        if (n + lane < p.N) {
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            if (j < left) y[j * ld] = acc[j];
        }
      } else {
        // lanes 2 l, 2 l + 1 trade the rounded values of two tokens, so that each
        // stores two columns of one: the even lane of token j, the odd lane of
        // token j + 1
        const bool odd = lane & 1;
        const uint32_t pick = odd ? 0x3276u : 0x5410u;
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + (m + odd) * ld + n + (lane & ~1);
        const bool in = n + lane < p.N;
#pragma unroll
        for (int j = 0; j < kCols; j += 2) {
          const uint32_t own = f32x2_to_bf16x2_bits(acc[j], acc[j + 1]);
          const uint32_t v = __byte_perm(own, __shfl_xor_sync(0xffffffffu, own, 1), pick);
          if (in && j + odd < left) *reinterpret_cast<uint32_t*>(y + j * ld) = v;
        }
      }
    }
    if (!ok && lane == 0) ctl->fail = 1;
  }
  __syncthreads();
  if (ctl->fail && rank == 0 && tid == 0)
    // a wait ran out: give copies in flight time to land before leaving
    for (int s = 0; s < kStages; ++s)
      for (int ph = 0; ph < 2; ++ph) mbar_wait_bounded(&ctl->full[s], ph, p.status, 1ll << 28);
  tc_fence_before();
  cluster_sync_all();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                 ::"r"(tmem), "r"(kTmemCols) : "memory");
}

}  // namespace

cudaError_t launch_mx4_gemm_pair(Mx4GemmParams& p, int sms, cudaStream_t st) {
  const uint64_t words = (uint64_t)p.K / 4, row = (uint64_t)p.K / 2;
  const uint64_t wt = (uint64_t)((p.N + 127) / 128 * p.kt), xt = (uint64_t)((p.M + 127) / 128 * p.kt);
  if (encode_map_2d(&p.tm_x, p.xc, (uint64_t)p.M, words, row, 64, 64,
                    CU_TENSOR_MAP_SWIZZLE_128B) != IG_OK ||
      encode_map_2d(&p.tm_w, p.wc, (uint64_t)p.N, words, row, 64, 128,
                    CU_TENSOR_MAP_SWIZZLE_128B) != IG_OK ||
      encode_map_2d(&p.tm_ws, p.ws, wt, 256, kMx4TileBytes, 256, 2,
                    CU_TENSOR_MAP_SWIZZLE_NONE) != IG_OK ||
      encode_map_2d(&p.tm_xs, p.xs, xt, 256, kMx4TileBytes, 256, 2,
                    CU_TENSOR_MAP_SWIZZLE_NONE) != IG_OK)
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(gemm_pair_kernel), allowed);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (p.N + kBN - 1) / kBN * ((p.M + kBT - 1) / kBT);
  if (tiles > 0x3fffffffLL) return cudaErrorInvalidConfiguration;
  const int64_t pieces = 2 * tiles <= sms / 2 ? 2 * tiles : tiles;   // half tiles, if they all fit
  const int64_t pairs = pieces < sms / 2 ? pieces : sms / 2;
  return launch_pdl(gemm_pair_kernel, dim3((unsigned)(2 * pairs)), dim3(kThreads), kSmem, st, p);
}

}  // namespace ig
