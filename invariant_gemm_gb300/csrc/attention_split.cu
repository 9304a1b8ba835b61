// Attention of few query rows over the 8-bit paged cache: single tokens, drafted
// tokens, the ends of chunks.
//
// Rows are a kv head's: `group` query heads for each new token, 16 rows to a
// tile (the M of mma.sync.m16n8k16). A work item is one tile, one kv head and
// one part of the sequence's tokens (split_tokens); its four warps take the
// part's steps of 16 tokens, one block of the cache each, in turn. Each warp
// has a ring of its own: one TMA box for a step's keys and one for its values.
// Items are dealt to blocks that stay; a warp asks for the next item's steps
// while it computes this one's.
//
// FP16 tensor-core products: a code is exact in FP16, a query row too once it is
// scaled by a power of two to a maximum below 2^15. Scales, being powers of two,
// are applied outside the products: the keys' to the logits, the values' to p.
//
// Online softmax in base 2 with whole exponents: a row's m is raised only when a
// logit passes m + 7, to the next whole number, so that every rescaling is by
// an exact power of two and most steps have none. p = 2^(t - m + 8 + e - E), E
// the largest exponent of the value scales so far and e this step's, stays below
// 2^15; as FP16 it has 11 bits down to 2^-14. The sum of p is FP32.
//
// The K order of both products is free, so the fragments are what lies together:
// a lane's keys are 32 consecutive bytes of one token, its values 16 consecutive
// bytes of four tokens; the box's swizzle makes both 128-bit loads free of bank
// conflicts.
#include "attention.cuh"
#include "warp_mma.cuh"

namespace ig {

namespace {

constexpr int kWarps = 4;
constexpr int kStages = 4;              // steps of a warp in flight
constexpr int kStep = kKvBlock;
constexpr int kRows = 16;
constexpr float kHeadroom = 7.0f;       // a row's m is raised past m + this
constexpr float kBias = 8.0f;           // p is 2^kBias at m
constexpr int kMinShift = -40;          // value scales below 2^-40 of the largest: as 2^-40
constexpr uint32_t kAbsent = 1u << 16;  // slot word: the step's page does not exist

template <int D>
struct Smem {
  static constexpr int kBox = kStep * D;              // bytes of a step's keys (or values)
  static constexpr int kRing = kWarps * kStages * 2 * kBox;
  static constexpr int kPitch = D + 4;                // floats of a row of sums
  float o[kWarps][kRows][kPitch];
  float ml[kWarps][kRows][2];
  int expo[kWarps];
  int nan_at[2][D];
  uint64_t full[kWarps][kStages];
  uint32_t slot[kWarps][kStages];
  int scan[kWarps];
  int last;
};

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }
__device__ __forceinline__ float qnan() { return __uint_as_float(0x7fc00000u); }

// 2^d for a whole d <= 0 (0 below -126, NaN for NaN)
__device__ __forceinline__ float pow2_down(float d) {
  if (d != d) return d;
  return d < -126.0f ? 0.0f : pow2((int)d);
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t lo_f16(uint32_t v) { return e4m3x2_to_f16x2((uint16_t)v); }
__device__ __forceinline__ uint32_t hi_f16(uint32_t v) {
  return e4m3x2_to_f16x2((uint16_t)(v >> 16));
}
// 0x80 in each byte of w that is a NaN code
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// A tile of a sequence, one kv head, one part.
struct Item {
  int b, h, tile, split, tiles, ns;
  int row0, n, kv, rows;       // rows of the tile
  int t0, t1;                  // tokens of the part that the tile's rows see: t0 .. t1 - 1
  int low, high;               // last token that its first and its last row see
  int parts;                   // parts that its rows see
  int first;                   // number of the sequence's first item
};

__device__ __forceinline__ int seq_splits(int kv, int len) { return kv > 0 ? (kv + len - 1) / len : 1; }
__device__ __forceinline__ int part_len(int kv) { return max(split_tokens(kv), kSplitTokens); }

// prefix[b]: items of the sequences before b.
__device__ __forceinline__ Item item_of(const AttnParams& p, const int* prefix, int item) {
  int lo = 0, hi = p.c.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= item) lo = mid; else hi = mid;
  }
  Item it;
  it.b = lo;
  it.first = prefix[lo];
  sequence_of(p.c, lo, it.row0, it.n, it.kv);
  const int rows = it.n * p.group, len = part_len(it.kv);
  it.tiles = (rows + kRows - 1) / kRows;
  it.ns = seq_splits(it.kv, len);
  uint32_t v = (uint32_t)(item - it.first);
  it.tile = (int)next_digit(v, it.tiles);
  it.split = (int)next_digit(v, it.ns);
  it.h = (int)v;
  const int r = it.tile * kRows;
  it.rows = min(kRows, rows - r);
  it.low = it.kv - it.n + r / p.group;
  it.high = it.kv - it.n + (r + it.rows - 1) / p.group;
  const int end = max(it.high + 1, 0);
  it.parts = max(1, (end + len - 1) / len);
  it.t0 = it.split * len;
  it.t1 = max(it.t0, min(end, it.t0 + len));
  return it;
}
__device__ __forceinline__ int warp_steps(const Item& it, int warp) {
  const int steps = (it.t1 - it.t0 + kStep - 1) / kStep;
  return (steps - warp + kWarps - 1) / kWarps;         // steps warp, warp + 4, ...
}

// Copies of one warp's steps, item after item.
template <int D>
struct Feed {
  const AttnParams& p;
  const int* prefix;
  uint8_t* ring;               // of the warp
  uint64_t* full;
  uint32_t* slot;
  int warp, lane, total, item, steps, i, batch_at, t0, h;
  int32_t page;                // of the batch's step `lane`
  uint32_t info;
  uint32_t made;               // stages asked for so far
  const int32_t* table;
  bool done;

  __device__ __forceinline__ void open() {
    // the next item of this block with steps of this warp
    while (item < total) {
      const Item it = item_of(p, prefix, item);
      steps = it.split < it.parts ? warp_steps(it, warp) : 0;
      if (steps > 0) {
        t0 = it.t0;
        h = it.h;
        table = p.c.table + (int64_t)it.b * p.c.ld_table;
        i = 0;
        batch_at = -32;
        return;
      }
      item += gridDim.x;
    }
    done = true;
  }
  // Pages and scales of 32 steps, one to a lane.
  __device__ __forceinline__ void look() {
    batch_at = i;
    info = kAbsent;
    page = 0;
    if (i + lane < steps) {
      const int tok = t0 + (warp + kWarps * (i + lane)) * kStep;
      page = __ldg(table + (tok >> p.c.page_shift));
      if (page >= 0 && page < p.c.pages) {
        const int blocks = 1 << (p.c.page_shift - 4);
        const uint8_t* s = p.c.scales + page * p.c.scale_stride + h * blocks +
                           ((tok & ((1 << p.c.page_shift) - 1)) / kKvBlock);
        info = __ldg(s) | (uint32_t)__ldg(s + p.c.heads * blocks) << 8;
      } else {
        atomicOr(p.c.status, kStatusIndexRange);
      }
    }
  }
  // Asks for one more step. Call with done == false.
  __device__ __forceinline__ void push() {
    if (i >= batch_at + 32) look();
    const int32_t pg = __shfl_sync(0xffffffffu, page, i - batch_at);
    const uint32_t in = __shfl_sync(0xffffffffu, info, i - batch_at);
    const uint32_t st = made % kStages;
    if (lane == 0) {
      slot[st] = in;
      if (in & kAbsent) {
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(full + st))
                     : "memory");
      } else {
        const int tok = t0 + (warp + kWarps * i) * kStep;
        const int row = tok & ((1 << p.c.page_shift) - 1);
        uint8_t* at = ring + st * 2 * Smem<D>::kBox;
        mbar_arrive_expect_tx(full + st, 2 * Smem<D>::kBox);
        tma_load_3d(at, &p.tm, 0, (h << p.c.page_shift) + row, pg, full + st);
        tma_load_3d(at + Smem<D>::kBox, &p.tm, 0, ((p.c.heads + h) << p.c.page_shift) + row, pg,
                    full + st);
      }
    }
    ++made;
    if (++i == steps) {
      item += gridDim.x;
      open();
    }
  }
};

template <int D>
__global__ void __launch_bounds__(32 * kWarps, 2) split_kernel(const __grid_constant__ AttnParams p) {
  using S = Smem<D>;
  constexpr int KS = D / 16;            // steps of 16 along D
  constexpr int NT = D / 8;             // 8-column tiles of the output
  constexpr int VW = D / 32;            // words of a token's values in a lane
  extern __shared__ __align__(1024) uint8_t raw[];
  S& s = *reinterpret_cast<S*>(raw + S::kRing);
  int* prefix = reinterpret_cast<int*>(raw + S::kRing + sizeof(S));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;

  if (tid < kWarps * kStages) mbar_init(&s.full[0][0] + tid, 1);
  fence_mbar_init();
  prefetch_tensormap(&p.tm);
  for (int i = tid; i < 2 * D; i += 32 * kWarps) (&s.nan_at[0][0])[i] = 0x7fffffff;
  griddep_wait();

  // items of each sequence, summed up: 128 sequences at a time
  int carry = 0;
  for (int b0 = 0; b0 < p.c.batch; b0 += 32 * kWarps) {
    const int b = b0 + tid;
    int count = 0;
    if (b < p.c.batch) {
      int row0, n, kv;
      if (!sequence_of(p.c, b, row0, n, kv)) {
        if (blockIdx.x == 0) atomicOr(p.c.status, kStatusIndexRange);
      } else if (n > 0 && n * p.group <= p.few_rows) {
        count = (n * p.group + kRows - 1) / kRows * seq_splits(kv, part_len(kv)) * p.c.heads;
      }
    }
    int sum = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    __syncthreads();
    if (lane == 31) s.scan[warp] = sum;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s.scan[w];
      carry += s.scan[w];
    }
    if (b < p.c.batch) prefix[b] = before + sum - count;
  }
  __syncthreads();
  const int total = carry;

  Feed<D> feed{p, prefix, raw + warp * kStages * 2 * S::kBox, s.full[warp], s.slot[warp], warp, lane,
               total, (int)blockIdx.x, 0, 0, 0, 0, 0, 0, 0, 0, nullptr, false};
  feed.open();
  while (!feed.done && feed.made < kStages) feed.push();
  __syncwarp();

  uint32_t taken = 0;
  bool dead = false;                    // a copy did not come in time
  if (p.flags & IG_FLAG_TEST_COPY_TIMEOUT) {      // as if the first had not
    dead = true;
    atomicOr(p.c.status, kStatusTimeout);
  }
  int turn = 0;
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    const Item it = item_of(p, prefix, item);
    if (it.split >= it.parts) continue;
    const int steps = warp_steps(it, warp);

    // --- the tile's queries: rows g and g + 8, FP16 with a power of two apart
    uint32_t qa[KS][4];
    float f0, f1;                       // logit of a product: times scale_log2 and the row's power
    int lim0, lim1;                     // last token that the row sees
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = g + 8 * half, gr = it.tile * kRows + r;
      const bool in = r < it.rows;
      const int tok = gr / p.group, head = it.h * p.group + gr % p.group;
      uint32_t w[D / 8];                // D / 4 values of the lane, two to a word
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in)
          v = *(reinterpret_cast<const uint4*>(p.q + (int64_t)(it.row0 + tok) * p.ld_q +
                                               (int64_t)head * D + c * (D / 4)) + i);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int e = (int)(top >> 7);          // the largest value is below 2^(e - 126)
      const float up = e == 255 ? qnan() : pow2(141 - max(e, 20));
      const float f = p.scale_log2 * (e == 255 ? 1.0f : pow2(max(e, 20) - 141));
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qa[k][half] = f16x2_of(bf16lo(w[2 * k]) * up, bf16hi(w[2 * k]) * up);
        qa[k][2 + half] = f16x2_of(bf16lo(w[2 * k + 1]) * up, bf16hi(w[2 * k + 1]) * up);
      }
      const int lim = in ? it.kv - it.n + tok : 0x7fffffff;
      if (half) { f1 = f; lim1 = lim; } else { f0 = f; lim0 = lim; }
    }

    float o[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[j][k] = 0.0f;
    float m0 = neg_inf(), m1 = neg_inf(), l0 = 0.0f, l1 = 0.0f;
    int expo = -1000;                   // E; none yet

    for (int i = 0; i < steps; ++i) {
      const uint32_t st = taken % kStages;
      if (!dead && !mbar_wait_bounded(s.full[warp] + st, (taken / kStages) & 1, p.c.status))
        dead = true;
      dead = __any_sync(0xffffffffu, dead);
      if (dead) break;
      const uint32_t info = s.slot[warp][st];
      const int tok = it.t0 + (warp + kWarps * i) * kStep;
      const uint8_t* kb = raw + (warp * kStages + st) * 2 * S::kBox;
      const uint8_t* vb = kb + S::kBox;
      uint32_t vw[4][VW];               // values of tokens 2c, 2c + 1, 2c + 8, 2c + 9
      float sc[2][4];
      if (!(info & kAbsent)) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int r = 2 * c + (t & 1) + 8 * (t >> 1);
          if (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(vb + r * D + ((g ^ (r & 7)) << 4));
            vw[t][0] = v.x; vw[t][1] = v.y;
            vw[t][VW - 2] = v.z; vw[t][VW - 1] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(
                vb + r * D + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + ((g & 1) << 3));
            vw[t][0] = v.x; vw[t][1] = v.y;
          }
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int r = nt * 8 + g;
          uint32_t kw[D / 16];          // D / 4 bytes of token r
          if (D == 128) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint4 v =
                  *reinterpret_cast<const uint4*>(kb + r * D + (((2 * c + q) ^ (r & 7)) << 4));
              kw[(4 * q) % (D / 16)] = v.x; kw[(4 * q + 1) % (D / 16)] = v.y;
              kw[(4 * q + 2) % (D / 16)] = v.z; kw[(4 * q + 3) % (D / 16)] = v.w;
            }
          } else {
            const uint4 v =
                *reinterpret_cast<const uint4*>(kb + r * D + ((c ^ ((r >> 1) & 3)) << 4));
            kw[0] = v.x; kw[1] = v.y; kw[2] = v.z; kw[3] = v.w;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[nt][k] = 0.0f;
#pragma unroll
          for (int k = 0; k < KS; ++k) mma_f16(sc[nt], qa[k], lo_f16(kw[k]), hi_f16(kw[k]));
        }
      }
      ++taken;
      __syncwarp();                     // the stage has been read
      if (!feed.done) feed.push();
      if (info & kAbsent) continue;

      // logits in base 2, masks
      const float ks = e8m0_value(info & 0xffu);
      const float a0 = f0 * ks, a1 = f1 * ks;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        sc[nt][0] *= a0; sc[nt][1] *= a0;
        sc[nt][2] *= a1; sc[nt][3] *= a1;
      }
      const uint32_t vbyte = (info >> 8) & 0xffu;
      if (vbyte == 255) {               // the block's values are NaN
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int w = 0; w < VW; ++w) vw[t][w] = 0x7f7f7f7fu;
      }
      if (tok + kStep - 1 > it.low) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (tok + nt * 8 + 2 * c + (k & 1) > (k < 2 ? lim0 : lim1)) sc[nt][k] = neg_inf();
        // p is 0 there, but 0 times NaN is not: tokens that no row sees have
        // any bytes; a NaN of a token that some rows see is kept for those
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int at = tok + 2 * c + (t & 1) + 8 * (t >> 1);
          if (at > it.high) {
#pragma unroll
            for (int w = 0; w < VW; ++w) vw[t][w] = 0;
          } else if (at > it.low) {
#pragma unroll
            for (int w = 0; w < VW; ++w) {
              const uint32_t bad = nan_bytes(vw[t][w]);
              if (bad) {
                for (int q = 0; q < 4; ++q)
                  if (bad >> (8 * q + 7) & 1) atomicMin(&s.nan_at[turn & 1][g * (D / 8) + 4 * w + q], at);
                vw[t][w] &= ~((bad >> 7) * 0xffu);
              }
            }
          }
        }
      }

      // maxima: raised where a logit passes m + 7
      const float x0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
      const float x1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
      if (__any_sync(0xffffffffu, x0 > m0 + kHeadroom || x1 > m1 + kHeadroom)) {
        float y0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
        float y1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
        y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, 2));
        y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, 2));
        float d0 = 1.0f, d1 = 1.0f;
        if (y0 > m0 + kHeadroom) {
          const float to = ceilf(y0);
          d0 = m0 == neg_inf() ? 0.0f : pow2_down(m0 - to);
          m0 = to;
        }
        if (y1 > m1 + kHeadroom) {
          const float to = ceilf(y1);
          d1 = m1 == neg_inf() ? 0.0f : pow2_down(m1 - to);
          m1 = to;
        }
        l0 *= d0;
        l1 *= d1;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          o[j][0] *= d0; o[j][1] *= d0;
          o[j][2] *= d1; o[j][3] *= d1;
        }
      }
      // exponents of the value scales
      int shift = 0;
      if (vbyte != 255) {
        const int e = (int)vbyte - 127;
        if (e > expo) {
          if (expo > -1000) {
            const float d = pow2(max(expo - e, -126));
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int k = 0; k < 4; ++k) o[j][k] *= d;
          }
          expo = e;
        }
        shift = max(e - expo, kMinShift);
      }
      const float back = pow2(-shift);
      const float b0 = (m0 == neg_inf() ? 0.0f : m0) - (kBias + (float)shift);
      const float b1 = (m1 == neg_inf() ? 0.0f : m1) - (kBias + (float)shift);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        sc[nt][0] = ex2(sc[nt][0] - b0); sc[nt][1] = ex2(sc[nt][1] - b0);
        sc[nt][2] = ex2(sc[nt][2] - b1); sc[nt][3] = ex2(sc[nt][3] - b1);
        l0 = fmaf(sc[nt][0] + sc[nt][1], back, l0);
        l1 = fmaf(sc[nt][2] + sc[nt][3], back, l1);
      }
      uint32_t pa[4];
      pa[0] = f16x2_of(sc[0][0], sc[0][1]);
      pa[1] = f16x2_of(sc[0][2], sc[0][3]);
      pa[2] = f16x2_of(sc[1][0], sc[1][1]);
      pa[3] = f16x2_of(sc[1][2], sc[1][3]);
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        const uint32_t x01 = __byte_perm(vw[0][w], vw[1][w], 0x5140);
        const uint32_t x23 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
        const uint32_t y01 = __byte_perm(vw[2][w], vw[3][w], 0x5140);
        const uint32_t y23 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
        mma_f16(o[4 * w], pa, lo_f16(x01), lo_f16(y01));
        mma_f16(o[4 * w + 1], pa, hi_f16(x01), hi_f16(y01));
        mma_f16(o[4 * w + 2], pa, lo_f16(x23), lo_f16(y23));
        mma_f16(o[4 * w + 3], pa, hi_f16(x23), hi_f16(y23));
      }
    }

    // --- the four warps' sums, in their order
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (c == 0) {
      s.ml[warp][g][0] = m0; s.ml[warp][g][1] = l0;
      s.ml[warp][g + 8][0] = m1; s.ml[warp][g + 8][1] = l1;
    }
    if (lane == 0) s.expo[warp] = expo;
    __syncthreads();
    int top_e = s.expo[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top_e = max(top_e, s.expo[w]);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = g + 8 * half;
      if (r < it.rows) {
        float top = s.ml[0][r][0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s.ml[w][r][0]);
        const float m = half ? m1 : m0;
        const float d = m == neg_inf() ? 0.0f
                                       : pow2_down(m - top) * pow2(max(expo - top_e, -126));
        float* row = s.o[warp][r] + c * (D / 4);
#pragma unroll
        for (int j = 0; j < NT; j += 4) {
          *reinterpret_cast<float4*>(row + j) =
              make_float4(o[j][2 * half] * d, o[j + 1][2 * half] * d, o[j + 2][2 * half] * d,
                          o[j + 3][2 * half] * d);
          *reinterpret_cast<float4*>(row + D / 8 + j) =
              make_float4(o[j][2 * half + 1] * d, o[j + 1][2 * half + 1] * d,
                          o[j + 2][2 * half + 1] * d, o[j + 3][2 * half + 1] * d);
        }
      }
    }
    __syncthreads();
    const int* nan_at = s.nan_at[turn & 1];
    if (tid < D) s.nan_at[(turn + 1) & 1][tid] = 0x7fffffff;
    ++turn;
    const float out_e = top_e > -1000 ? e8m0_value(top_e + 127) : 0.0f;
    for (int i = tid; i < it.rows * (D / 4); i += 32 * kWarps) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float top = s.ml[0][r][0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s.ml[w][r][0]);
      float l = 0.0f;
      float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float m = s.ml[w][r][0];
        l += m == neg_inf() ? s.ml[w][r][1] : s.ml[w][r][1] * pow2_down(m - top);
        const float4 u = *reinterpret_cast<const float4*>(s.o[w][r] + d);
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
      }
      const int gr = it.tile * kRows + r, tok = gr / p.group;
      const int lim = it.kv - it.n + tok;
      if (lim >= nan_at[d]) v.x = qnan();
      if (lim >= nan_at[d + 1]) v.y = qnan();
      if (lim >= nan_at[d + 2]) v.z = qnan();
      if (lim >= nan_at[d + 3]) v.w = qnan();
      if (it.parts == 1) {
        const float inv = l == 0.0f ? 0.0f : out_e / l;
        *reinterpret_cast<uint2*>(p.out + (int64_t)(it.row0 + tok) * p.ld_out +
                                  (int64_t)(it.h * p.group + gr % p.group) * D + d) =
            make_uint2(f32x2_to_bf16x2_bits(v.x * inv, v.y * inv),
                       f32x2_to_bf16x2_bits(v.z * inv, v.w * inv));
      } else {
        const int64_t at = (int64_t)item * p.part_rows + r;
        *reinterpret_cast<float4*>(p.parts + at * D + d) = v;
        if (d == 0)
          *reinterpret_cast<float4*>(p.part_ml + at * kPartWords) =
              make_float4(top, l, __int_as_float(top_e), 0.0f);
      }
    }
    if (it.parts == 1) {
      __syncthreads();
      continue;
    }

    // --- the last of the tile's parts to come joins them, in their order
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      uint32_t* count = p.counters + ((int64_t)it.b * p.max_tiles + it.tile) * p.c.heads + it.h;
      const uint32_t old = atom_add_acq_rel_gpu(count, 1u);
      if (old >= (uint32_t)it.parts) atomicOr(p.c.status, kStatusCorrupt);
      s.last = old + 1 == (uint32_t)it.parts;
      if (s.last) *count = 0;
    }
    __syncthreads();
    if (!s.last) continue;
    __threadfence();
    for (int i = tid; i < it.rows * (D / 4); i += 32 * kWarps) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      const int64_t first = (int64_t)(it.first + (it.h * it.ns) * it.tiles + it.tile);
      float top = neg_inf();
      int te = -1000;
      for (int q = 0; q < it.parts; ++q) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(
            p.part_ml + ((first + (int64_t)q * it.tiles) * p.part_rows + r) * kPartWords));
        top = fmaxf(top, u.x);
        te = max(te, __float_as_int(u.z));
      }
      float l = 0.0f;
      float4 v = make_float4(0, 0, 0, 0);
      for (int q = 0; q < it.parts; ++q) {
        const int64_t at = (first + (int64_t)q * it.tiles) * p.part_rows + r;
        const float4 u = __ldcg(reinterpret_cast<const float4*>(p.part_ml + at * kPartWords));
        const float4 x = __ldcg(reinterpret_cast<const float4*>(p.parts + at * D + d));
        const float w = u.x == neg_inf() ? 1.0f : pow2_down(u.x - top);
        const float y = w * pow2(max(__float_as_int(u.z) - te, -126));
        l = fmaf(u.y, w, l);
        v.x = fmaf(x.x, y, v.x); v.y = fmaf(x.y, y, v.y);
        v.z = fmaf(x.z, y, v.z); v.w = fmaf(x.w, y, v.w);
      }
      const float inv = l == 0.0f ? 0.0f : (te > -1000 ? e8m0_value(te + 127) : 0.0f) / l;
      const int gr = it.tile * kRows + r, tok = gr / p.group;
      *reinterpret_cast<uint2*>(p.out + (int64_t)(it.row0 + tok) * p.ld_out +
                                (int64_t)(it.h * p.group + gr % p.group) * D + d) =
          make_uint2(f32x2_to_bf16x2_bits(v.x * inv, v.y * inv),
                     f32x2_to_bf16x2_bits(v.z * inv, v.w * inv));
    }
  }

  if (dead) {
    // own copies still in flight land before the block's memory is freed
    while (taken < feed.made) {
      mbar_wait_bounded(s.full[warp] + taken % kStages, (taken / kStages) & 1, p.c.status);
      ++taken;
    }
  }
}

template <int D>
cudaError_t launch(const AttnParams& p, cudaStream_t st) {
  const size_t smem = Smem<D>::kRing + sizeof(Smem<D>) + sizeof(int) * (size_t)p.c.batch;
  cudaError_t e = cudaFuncSetAttribute(split_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(split_kernel<D>, dim3(2 * sm_count()), dim3(32 * kWarps), smem, st, p);
}

}  // namespace

cudaError_t launch_attention_split(const AttnParams& p, int head_dim, cudaStream_t st) {
  return head_dim == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace ig
