// Attention of few query rows over the 8-bit paged cache: single tokens, drafted
// tokens, the ends of chunks.
//
// Rows are a kv head's: `group` query heads for each new token, 16 rows to a
// tile. A work item is one tile, one kv head and one part of the sequence's
// tokens (split_tokens). Items go to whichever block asks first (a counter in the
// workspace), of blocks that stay: three to an SM where a tile has 8 rows at most,
// else two (heads of 64: four and three). In a block four warps compute and one copies ahead:
//   copies   pages and scales of the part, a step of 16 tokens (a block of the
//            cache) to a lane, asked for while the part before is on its way;
//            then one TMA box for a step's keys and one for its values, four
//            steps to a stage of the ring; the item's queries
//   compute  a step of each stage to a warp; then a share each of the four warps'
//            sums, in their order, into the output or, where the rows see several
//            parts, into the workspace
// A second kernel joins the parts, in an order that their number fixes.
//
// FP16 tensor-core products with the tokens as rows (M) and the query rows as
// columns (N, 8 at a time): S^T = K Q^T and O^T = V^T P^T, so that 8 rows a kv
// head leave no part of an MMA unused. A code is exact in FP16, a query row too
// once it is scaled by a power of two to a maximum below 2^15 (but for values under
// 2^-31 of its largest, which are off by 2^-39 of that). Scales, being powers of two,
// are applied outside the products: the keys' to the logits, the values' to p.
//
// Online softmax in base 2 with whole exponents: a row's m is raised only when a
// logit passes m + 7, to the next whole number, so that every rescaling is by
// an exact power of two and most steps have none. A value's scale is part of its logit
// there ("a row's sums" in attention.cuh). p is 2^15 at most; as FP16 it has 11 bits down
// to 2^-14. The sum of p is FP32.
//
// The K order of both products is free, and so is the M order of the second, so
// the fragments are what lies together: a lane's keys are 32 consecutive bytes of
// two tokens, its values 16 consecutive bytes of four tokens; the box's swizzle
// makes both 128-bit loads free of bank conflicts.
//
// What bounds it: HBM. 64 sequences of up to 8192 tokens, 8 kv heads of 128, 8 rows each:
// 598 MB in 108 us (5.5 TB/s), issue slots half used; the join of the parts behind it 5
// us. 8 of up to 65536, 4 rows each: 103 us for 622 MB with the join (6.0 TB/s). Small
// calls are the chain start - lengths (0.9 us) - pages, queries, copies (1.8) - products of
// four steps to a warp (2.7) - join of the warps (0.6) - join of the parts (2): 777 tokens
// 8.9 us. With more than 16 rows each tile reads and converts the tokens again, from L2:
// 32 rows 302 us where 8 take 114. (Tiles of 32 rows, queries in shared memory, one block
// of 254 registers to an SM: 434 us.)
#include "attention.cuh"
#include "warp_mma.cuh"

namespace ig {

namespace {

constexpr int kTeam = 4;                // warps that compute
constexpr int kThreads = 32 * (kTeam + 1);
constexpr int kStep = kKvBlock;
constexpr int kRows = 16;               // of a tile
constexpr int kUnit = 32;               // steps looked up at a time
constexpr float kHeadroom = 7.0f;       // a row's m is raised past m + this
constexpr float kBias = 8.0f;           // p is 2^kBias at m
constexpr float kMost = 15.0f;          // of p's exponent: kHeadroom + kBias
constexpr int kNoExp = -1000;           // of no value scale yet
constexpr uint32_t kAbsent = 1u << 16;  // step's word: its page does not exist
constexpr int kSeqs = 128;              // sequences that a block keeps beside their items

// A tile of a sequence, one kv head, one part.
struct Item {
  int b, h, tile, split, tiles, ns;
  int row0, n, kv, rows;       // rows of the tile
  int t0, t1;                  // tokens of the part that the tile's rows see: t0 .. t1 - 1
  int low, high;               // last token that its first and its last row see
  int parts;                   // parts that its rows see
  int id;                      // -1: no more items
};

template <int D, int NT>
struct Smem {
  static constexpr int kStages = D == 128 && NT == 1 ? 3 : 4;
  static constexpr int kBlocks = (D == 128 ? 2 : 3) + (NT == 1);      // to an SM
  static constexpr int kBox = kStep * D;              // bytes of a step's keys (or values)
  static constexpr int kStage = 2 * kTeam * kBox;     // keys of four steps, then values
  static constexpr int kRing = kStages * kStage;
  static constexpr int kPitch = D + 4;                // floats of a row of sums
  float o[kTeam][8 * NT][kPitch];
  alignas(16) __nv_bfloat16 q[2][8 * NT][D];
  float ml[kTeam][8 * NT][2];
  int c[kTeam];
  alignas(16) int nan_at[2][D];
  Item item[2];
  uint64_t full[kStages], empty[kStages], item_full[2], item_empty[2], sums_full, sums_empty;
  uint32_t info[kStages][kTeam];
  int3 seq[kSeqs];                      // row0, n, kv of the first sequences
  int scan[kTeam + 1];
  int dead;
};

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }
__device__ __forceinline__ float qnan() { return __uint_as_float(0x7fc00000u); }

// 2^d for a whole d <= 0 (0 below -126, NaN for NaN): d + 127 is in the low bits
// of its sum with 1.5 * 2^23
__device__ __forceinline__ float pow2_down(float d) {
  const float r = __uint_as_float(__float_as_uint(d + (12582912.0f + 127.0f)) << 23);
  return d >= -126.0f ? r : d != d ? d : 0.0f;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// An exponent of p: logits past 2^22 come in steps by which it could pass what FP16 has (at
// the largest logit it is off by one of them at most, and not below 0 from steps of 16 on).
// NaN stays.
__device__ __forceinline__ float at_most(float x) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(kMost));
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
// Four codes -> FP16 values of the low two and of the high two.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(v));
}
// 8 x 8 values of 16 bits over the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// 0x80 in each byte of w that is a NaN code
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Bounded wait of a warp that also ends when any other wait of the block gave up.
template <typename S>
__device__ __forceinline__ bool wait(S& s, uint64_t* bar, uint32_t parity, uint32_t* status) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const long long t0 = clock64();
    while (!(ok = mbar_try_wait(bar, parity))) {
      if (*reinterpret_cast<volatile int*>(&s.dead)) break;
      if (clock64() - t0 > (1ll << 31)) {
        *reinterpret_cast<volatile int*>(&s.dead) = 1;
        atomicOr(status, kStatusTimeout);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// row / group for the few rows of a sequence here.
__device__ __forceinline__ int token_of(const AttnParams& p, int row) {
  return (int)((uint32_t)row * p.group_inv >> 16);
}

__device__ __forceinline__ int seq_splits(int kv, int len) { return kv > 0 ? (kv + len - 1) / len : 1; }

// Parts with tokens that a tile sees whose last row sees token `high`.
__device__ __forceinline__ int tile_parts(int high, int len) {
  return high < 0 ? 1 : high / len + 1;
}

// prefix[b]: items of the sequences before b.
__device__ __forceinline__ Item item_of(const AttnParams& p, const int* prefix, const int3* seq,
                                        int item) {
  int lo = 0, hi = p.c.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= item) lo = mid; else hi = mid;
  }
  Item it;
  it.id = item;
  it.b = lo;
  if (lo < kSeqs) {
    it.row0 = seq[lo].x;
    it.n = seq[lo].y;
    it.kv = seq[lo].z;
  } else {
    sequence_of(p.c, lo, it.row0, it.n, it.kv);
  }
  const int rows = it.n * p.group, len = split_tokens(it.kv);
  it.tiles = (rows + kRows - 1) / kRows;
  it.ns = seq_splits(it.kv, len);
  uint32_t v = (uint32_t)(item - prefix[lo]);
  it.tile = (int)next_digit(v, it.tiles);
  it.split = (int)next_digit(v, it.ns);
  it.h = (int)v;
  const int r = it.tile * kRows;
  it.rows = min(kRows, rows - r);
  it.low = it.kv - it.n + token_of(p, r);
  it.high = it.kv - it.n + token_of(p, r + it.rows - 1);
  const int end = max(it.high + 1, 0);
  it.parts = tile_parts(it.high, len);
  it.t0 = it.split * len;
  it.t1 = max(it.t0, min(end, it.t0 + len));
  return it;
}

// The copying warp's look at 32 steps of an item, a step to a lane.
struct Unit {
  Item it;
  int step;                    // first of the unit's steps
  int32_t page;
  uint32_t key, value;         // scales, not looked at before a step is handed on
};

// The unit after u: of the same item, else of the block's next item that has a
// part its rows see (id -1: none). Pages only.
// Which block takes an item does not show in its bits.
__device__ __forceinline__ void next_unit(const AttnParams& p, const int* prefix, const int3* seq,
                                          int total, int lane, Unit& u) {
  u.step += kUnit;
  if (u.it.id < 0 || u.it.t0 + u.step * kStep >= u.it.t1) {
    // a block's first item is its own, the others go to who asks first
    int id = (int)blockIdx.x;
    u.step = 0;
    for (bool own = u.it.id < 0;; own = false) {
      if (!own) {
        if (lane == 0) id = (int)(atomicAdd(p.next, 1u) + gridDim.x);
        id = __shfl_sync(0xffffffffu, id, 0);
      }
      if (id >= total) {
        u.it.id = -1;
        return;
      }
      u.it = item_of(p, prefix, seq, id);
      if (u.it.split < u.it.parts) break;
    }
  }
  u.key = kAbsent;
  u.value = 0;
  u.page = 0;
  const int tok = u.it.t0 + (u.step + lane) * kStep;
  if (tok < u.it.t1)
    u.page = __ldg(p.c.table + (int64_t)u.it.b * p.c.ld_table + (tok >> p.c.page_shift));
}
// Its scales.
__device__ __forceinline__ void unit_scales(const AttnParams& p, int lane, Unit& u) {
  const int tok = u.it.t0 + (u.step + lane) * kStep;
  if (u.it.id < 0 || tok >= u.it.t1) return;
  if (u.page >= 0 && u.page < p.c.pages) {
    const int blocks = 1 << (p.c.page_shift - 4);
    const uint8_t* s = p.c.scales + u.page * p.c.scale_stride + u.it.h * blocks +
                       ((tok & ((1 << p.c.page_shift) - 1)) / kKvBlock);
    u.key = __ldg(s);
    u.value = __ldg(s + p.c.heads * blocks);
  } else {
    atomicOr(p.c.status, kStatusIndexRange);
  }
}

template <int D, int NT>
__device__ void copy_warp(const AttnParams& p, Smem<D, NT>& s, uint8_t* ring, const int* prefix,
                          int total, int lane) {
  using S = Smem<D, NT>;
  Unit u;
  u.it.id = -1;
  u.step = 0;
  next_unit(p, prefix, s.seq, total, lane, u);
  unit_scales(p, lane, u);
  uint32_t items = 0, made = 0;
  bool ok = true;
  while (ok) {
    if (u.step == 0) {
      // the item and its queries: the heads of one kv head lie together
      const int buf = items & 1;
      ok = wait(s, &s.item_empty[buf], ((items >> 1) & 1) ^ 1, p.c.status);
      if (!ok) break;
      ++items;
      for (int d = lane; d < D; d += 32) s.nan_at[buf][d] = 0x7fffffff;
      __syncwarp();
      if (lane == 0) {
        s.item[buf] = u.it;
        const uint32_t bytes = u.it.id < 0 ? 0 : u.it.rows * D * 2;
        mbar_arrive_expect_tx(&s.item_full[buf], bytes);
      }
      __syncwarp();
      if (u.it.id < 0) break;
      const int r = u.it.tile * kRows, last = r + u.it.rows;      // rows of the sequence
      const int tok = token_of(p, r) + lane;
      const int from = max(r, tok * p.group), to = min(last, (tok + 1) * p.group);
      if (from < to)
        bulk_g2s(&s.q[buf][from - r][0],
                 p.q + (int64_t)(u.it.row0 + tok) * p.ld_q +
                     (int64_t)(u.it.h * p.group + from - tok * p.group) * D,
                 (uint32_t)(to - from) * D * 2, &s.item_full[buf]);
    }
    const Unit now = u;
    const int steps = min(kUnit, (now.it.t1 - now.it.t0 + kStep - 1) / kStep - now.step);
    const int row0 = now.it.t0 + now.step * kStep;
    for (int i = 0; i < steps || i == 0; i += kTeam) {
      if (steps > 0) {
        const uint32_t st = made % S::kStages;
        ok = wait(s, &s.empty[st], ((made / S::kStages) & 1) ^ 1, p.c.status);
        if (!ok) break;
        ++made;
        // lane l < 4: keys and values of step i + l; the scales may still be on
        // their way
        const int32_t page = __shfl_sync(0xffffffffu, now.page, (i + lane) & 31);
        const bool there = lane < kTeam && i + lane < steps && page >= 0 && page < p.c.pages;
        const uint32_t have = __popc(__ballot_sync(0xffffffffu, there));
        if (lane == 0) mbar_arrive_expect_tx(&s.full[st], have * 2 * S::kBox);
        __syncwarp();
        if (there) {
          const int row = (row0 + (i + lane) * kStep) & ((1 << p.c.page_shift) - 1);
          uint8_t* at = ring + st * S::kStage + lane * S::kBox;
          tma_load_3d(at, &p.tm, 0, (now.it.h << p.c.page_shift) + row, page, &s.full[st]);
          tma_load_3d(at + kTeam * S::kBox, &p.tm, 0,
                      ((p.c.heads + now.it.h) << p.c.page_shift) + row, page, &s.full[st]);
        }
        const uint32_t key = __shfl_sync(0xffffffffu, now.key, (i + lane) & 31);
        const uint32_t value = __shfl_sync(0xffffffffu, now.value, (i + lane) & 31);
        if (lane < kTeam) s.info[st][lane] = there ? key | value << 8 : kAbsent;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.full[st]);
        __syncwarp();
      }
      // the next unit's pages, and once they are here its scales
      if (i == 0) next_unit(p, prefix, s.seq, total, lane, u);
      if (i == 4 * kTeam) unit_scales(p, lane, u);
    }
    if (steps <= 4 * kTeam) unit_scales(p, lane, u);
  }
  if (*reinterpret_cast<volatile int*>(&s.dead)) {
    // copies still in flight land before the block leaves
    for (uint32_t m = made > S::kStages ? made - S::kStages : 0; m < made; ++m)
      mbar_wait_bounded(&s.full[m % S::kStages], (m / S::kStages) & 1, p.c.status);
    for (uint32_t m = items > 2 ? items - 2 : 0; m < items; ++m)
      mbar_wait_bounded(&s.item_full[m & 1], (m >> 1) & 1, p.c.status);
  }
}

// A warp's share of the rows: the four warps' sums, in their order.
template <int D, int NT>
__device__ __forceinline__ void join_sums(const AttnParams& p, const Smem<D, NT>& s, int buf,
                                          int warp, int lane) {
  constexpr int PER = 128 / D;          // rows of a pass, 4 values to a lane
  const int d = lane * 4 % D, sub = lane * 4 / D;
  const Item& it = s.item[buf];
  int c = s.c[0];
#pragma unroll
  for (int w = 1; w < kTeam; ++w) c = max(c, s.c[w]);
  float more[kTeam];
#pragma unroll
  for (int w = 0; w < kTeam; ++w) more[w] = pow2(c - s.c[w]);
  const int4 nan_at = *reinterpret_cast<const int4*>(&s.nan_at[buf][d]);
  const bool parts = it.parts > 1;
  const int64_t part =
      (((first_tile(p.tiles_by_row, it.b, it.row0, p.group, p.max_tiles) + it.tile) * p.c.heads +
        it.h) * p.max_parts + it.split) * p.part_rows;
#pragma unroll
  for (int i = 0; i < 2 * NT; i += PER) {
    const int r = i / PER * kTeam * PER + warp * PER + sub;
    if (r >= it.rows) break;
    float m[kTeam], top = neg_inf(), l = 0.0f;
    float4 u[kTeam], v = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < kTeam; ++w) {
      m[w] = s.ml[w][r][0];
      u[w] = *reinterpret_cast<const float4*>(&s.o[w][r][d]);
      top = fmaxf(top, m[w]);
    }
#pragma unroll
    for (int w = 0; w < kTeam; ++w) {
      // a warp that saw nothing has sums of 0, or of NaN
      const float y = m[w] == neg_inf() ? 1.0f : pow2_down(m[w] - top);
      l = fmaf(s.ml[w][r][1] * more[w], y, l);
      v.x = fmaf(u[w].x, y, v.x); v.y = fmaf(u[w].y, y, v.y);
      v.z = fmaf(u[w].z, y, v.z); v.w = fmaf(u[w].w, y, v.w);
    }
    const int gr = it.tile * kRows + r, tok = token_of(p, gr), lim = it.kv - it.n + tok;
    if (lim >= nan_at.x) v.x = qnan();
    if (lim >= nan_at.y) v.y = qnan();
    if (lim >= nan_at.z) v.z = qnan();
    if (lim >= nan_at.w) v.w = qnan();
    if (parts) {
      const int64_t at = part + r;
      *reinterpret_cast<float4*>(p.parts + at * D + d) = v;
      if (d == 0)
        *reinterpret_cast<float4*>(p.part_ml + at * kPartWords) =
            make_float4(top, l, __int_as_float(c), 0.0f);
    } else {
      // (one after the other: 2^c / l may be below FP32's range where the result is not)
      const float inv = l == 0.0f ? 0.0f : 1.0f / l, unit = pow2(c);
      v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
      *reinterpret_cast<uint2*>(p.out + (int64_t)(it.row0 + tok) * p.ld_out +
                                (it.h * p.group + gr - tok * p.group) * D + d) =
          make_uint2(f32x2_to_bf16x2_bits(v.x * unit, v.y * unit),
                     f32x2_to_bf16x2_bits(v.z * unit, v.w * unit));
    }
  }
}

template <int D, int NT>
__device__ void compute_warp(const AttnParams& p, Smem<D, NT>& s, const uint8_t* ring, int warp,
                             int lane) {
  using S = Smem<D, NT>;
  constexpr int KS = D / 16;            // steps of 16 along D
  constexpr int MT = D / 16;            // 16-row tiles of O^T
  constexpr int VW = D / 32;            // words of a token's values in a lane
  const int g = lane >> 2, c = lane & 3;
  uint32_t taken = 0;
  for (uint32_t turn = 0;; ++turn) {
    const int buf = turn & 1;
    if (!wait(s, &s.item_full[buf], (turn >> 1) & 1, p.c.status)) return;
    const Item& it = s.item[buf];
    if (it.id < 0) return;
    const int rows = it.rows, low = it.low, high = it.high, t0 = it.t0;
    const int steps = (it.t1 - t0 + kStep - 1) / kStep;

    // --- queries: row 8 nt + g as FP16 with a power of two apart
    uint32_t qb[NT][KS][2];
    float f[NT][2];                     // logit of a product, rows 2c and 2c + 1
    int lim[NT][2];                     // last token that they see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + g;
      uint32_t w[D / 8];                // D / 4 values, two to a word
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint4 v = *(reinterpret_cast<const uint4*>(&s.q[buf][r][c * (D / 4)]) + i);
        if (r >= rows) v = make_uint4(0, 0, 0, 0);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = (int)(top >> 7);    // the largest value is below 2^(e - 126)
      const float up = e == 255 ? qnan() : pow2(141 - max(e, 20));
      const float mine = p.scale_log2 * (e == 255 ? 1.0f : pow2(max(e, 20) - 141));
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qb[nt][k][0] = f16x2_of(bf16lo(w[2 * k]) * up, bf16hi(w[2 * k]) * up);
        qb[nt][k][1] = f16x2_of(bf16lo(w[2 * k + 1]) * up, bf16hi(w[2 * k + 1]) * up);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * nt + 2 * c + i;
        f[nt][i] = __shfl_sync(0xffffffffu, mine, (2 * c + i) * 4);
        lim[nt][i] = row < rows ? it.kv - it.n + token_of(p, it.tile * kRows + row) : 0x7fffffff;
      }
    }

    float o[MT][NT][4];
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[j][nt][k] = 0.0f;
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[nt][i] = neg_inf();
        l[nt][i] = 0.0f;
      }
    int expo = kNoExp;                  // largest exponent of a value scale so far

    for (int i = 0; i < steps; i += kTeam) {
      const uint32_t st = taken % S::kStages;
      if (!wait(s, &s.full[st], (taken / S::kStages) & 1, p.c.status)) return;
      ++taken;
      const uint32_t info = s.info[st][warp];
      const int tok = t0 + (i + warp) * kStep;
      const uint8_t* kb = ring + st * S::kStage + warp * S::kBox;
      const uint8_t* vb = kb + kTeam * S::kBox;
      if (info & kAbsent) {             // past the part's end, or no such page
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[st]);
        continue;
      }
      uint32_t kw[2][D / 16];           // D / 4 bytes of tokens g and g + 8
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int r = 8 * t + g;
        if constexpr (D == 128) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint4 v =
                *reinterpret_cast<const uint4*>(kb + r * D + (((2 * c + q) ^ (r & 7)) << 4));
            kw[t][4 * q] = v.x; kw[t][4 * q + 1] = v.y;
            kw[t][4 * q + 2] = v.z; kw[t][4 * q + 3] = v.w;
          }
        } else {
          const uint4 v =
              *reinterpret_cast<const uint4*>(kb + r * D + ((c ^ ((r >> 1) & 3)) << 4));
          kw[t][0] = v.x; kw[t][1] = v.y; kw[t][2] = v.z; kw[t][3] = v.w;
        }
      }
      uint32_t vw[4][VW];               // values of tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int r = 2 * c + (t & 1) + 8 * (t >> 1);
        if constexpr (D == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(vb + r * D + ((g ^ (r & 7)) << 4));
          vw[t][0] = v.x; vw[t][1] = v.y; vw[t][2] = v.z; vw[t][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(
              vb + r * D + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + ((g & 1) << 3));
          vw[t][0] = v.x; vw[t][1] = v.y;
        }
      }
      // tokens g (0, 1) and g + 8, rows 2c and 2c + 1; even and odd steps of K
      // apart: half as long a chain of MMAs
      float sc[NT][4], sd[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[nt][k] = sd[nt][k] = 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a[4];
        e4m3x4_to_f16(kw[0][k], a[0], a[2]);
        e4m3x4_to_f16(kw[1][k], a[1], a[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16(k & 1 ? sd[nt] : sc[nt], a, qb[nt][k][0], qb[nt][k][1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[nt][k] += sd[nt][k];
      __syncwarp();                     // the stage has been read
      if (lane == 0) mbar_arrive(&s.empty[st]);

      // logits in base 2, masks
      const float ks = e8m0_value(info & 0xffu);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float a0 = f[nt][0] * ks, a1 = f[nt][1] * ks;
        sc[nt][0] = __fmul_rn(sc[nt][0], a0); sc[nt][1] = __fmul_rn(sc[nt][1], a1);
        sc[nt][2] = __fmul_rn(sc[nt][2], a0); sc[nt][3] = __fmul_rn(sc[nt][3], a1);
      }
      const uint32_t vbyte = (info >> 8) & 0xffu;
      if (vbyte == 255) {               // the block's values are NaN
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int w = 0; w < VW; ++w) vw[t][w] = 0x7f7f7f7fu;
      }
      if (tok + kStep - 1 > low) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (tok + g + 8 * (k >> 1) > lim[nt][k & 1]) sc[nt][k] = neg_inf();
        // p is 0 there, but 0 times NaN is not: tokens that no row sees have
        // any bytes; a NaN of a token that some rows see is kept for those
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int at = tok + 2 * c + (t & 1) + 8 * (t >> 1);
          if (at > high) {
#pragma unroll
            for (int w = 0; w < VW; ++w) vw[t][w] = 0;
          } else if (at > low) {
#pragma unroll
            for (int w = 0; w < VW; ++w) {
              const uint32_t bad = nan_bytes(vw[t][w]);
              if (bad) {
                for (int q = 0; q < 4; ++q)
                  if (bad >> (8 * q + 7) & 1)
                    atomicMin(&s.nan_at[buf][g * (D / 8) + 4 * w + q], at);
                vw[t][w] &= ~((bad >> 7) * 0xffu);
              }
            }
          }
        }
      }

      // exponent of the value scale
      int e = 0;
      if (vbyte != 255) {
        e = (int)vbyte - 127;
        if (c_of(max(e, expo)) != c_of(expo)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) l[nt][r] *= pow2(c_of(64) - c_of(0));
        }
        expo = max(expo, e);
        e = max(e, expo - kSpread);
      }
      const float ef = (float)e, back = back_of(e, expo);
      // maxima: raised where a logit and e pass m + 7
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          raise |= fmaxf(sc[nt][r], sc[nt][2 + r]) > m[nt][r] + (kHeadroom - ef);
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float x = fmaxf(sc[nt][r], sc[nt][2 + r]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            x += ef;
            float d = 1.0f;
            if (x > m[nt][r] + kHeadroom) {
              const float to = ceilf(x);
              d = m[nt][r] == neg_inf() ? 0.0f : pow2_down(m[nt][r] - to);
              m[nt][r] = to;
            }
            l[nt][r] *= d;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              o[j][nt][r] *= d;
              o[j][nt][2 + r] *= d;
            }
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float b0 = (m[nt][0] == neg_inf() ? 0.0f : m[nt][0]) - (kBias + ef);
        const float b1 = (m[nt][1] == neg_inf() ? 0.0f : m[nt][1]) - (kBias + ef);
        const float p0 = ex2(at_most(sc[nt][0] - b0)), p1 = ex2(at_most(sc[nt][1] - b1));
        const float p2 = ex2(at_most(sc[nt][2] - b0)), p3 = ex2(at_most(sc[nt][3] - b1));
        l[nt][0] = fmaf(p0 + p2, back, l[nt][0]);
        l[nt][1] = fmaf(p1 + p3, back, l[nt][1]);
        pb[nt][0] = transpose8(f16x2_of(p0, p1));
        pb[nt][1] = transpose8(f16x2_of(p2, p3));
      }
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        uint32_t a[4], b[4];
        e4m3x4_to_f16(__byte_perm(vw[0][w], vw[1][w], 0x5140), a[0], a[1]);
        e4m3x4_to_f16(__byte_perm(vw[2][w], vw[3][w], 0x5140), a[2], a[3]);
        e4m3x4_to_f16(__byte_perm(vw[0][w], vw[1][w], 0x7362), b[0], b[1]);
        e4m3x4_to_f16(__byte_perm(vw[2][w], vw[3][w], 0x7362), b[2], b[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(o[2 * w][nt], a, pb[nt][0], pb[nt][1]);
          mma_f16(o[2 * w + 1][nt], b, pb[nt][0], pb[nt][1]);
        }
      }
    }

    // --- sums of all warps: rows 2c and 2c + 1, values (D / 8) g ..
    if (!wait(s, &s.sums_empty, (turn & 1) ^ 1, p.c.status)) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x = l[nt][r];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        const int row = 8 * nt + 2 * c + r;
        if (g == 0) {
          s.ml[warp][row][0] = m[nt][r];
          s.ml[warp][row][1] = x;
        }
        float* at = &s.o[warp][row][g * (D / 8)];
#pragma unroll
        for (int j = 0; j < MT; j += 2)
          *reinterpret_cast<float4*>(at + 2 * j) =
              make_float4(o[j][nt][r], o[j][nt][2 + r], o[j + 1][nt][r], o[j + 1][nt][2 + r]);
      }
    if (lane == 0) s.c[warp] = c_of(expo);
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.sums_full);
    if (!wait(s, &s.sums_full, turn & 1, p.c.status)) return;
    join_sums<D, NT>(p, s, buf, warp, lane);
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&s.sums_empty);
      mbar_arrive(&s.item_empty[buf]);
    }
  }
}

// The parts of a sequence's rows, joined: D / 4 lanes to a row of one query head,
// 4 values each, 128 / D rows to a block. Eight sums, of the parts w, w + 8, ... in
// their order, added in the order of w; W warps share them. Few rows are a matter
// of how long it takes to get at a row's parts (W = 8: 256 rows of up to 64 parts
// 5 us), many of how many rows there are at a time: the whole call with W = 1, 2 and 4
// 113.3, 114.7 and 115.8 us for 4096 rows of up to 16 parts, 73.9, 76.8 and 81.6 for
// 8192 of up to 4. 792 blocks of two rows: W = 8 18.7 us, 1 17.8.
constexpr int kJoinSums = 8;

template <int D, int W>
__global__ void __launch_bounds__(32 * W) join_kernel(const AttnJoinParams p) {
  constexpr int L = D / 4, PER = 32 / L, SL = kMaxSplits / 32;
  constexpr int C = kJoinSums / W;      // sums of a warp: w = warp, warp + W, ...
  constexpr int B = 8 / C;              // parts of each asked for at a time
  __shared__ float4 sums[kJoinSums][32];
  __shared__ float weight[PER][kMaxSplits], inverse[PER], unit[PER];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / L, d = lane % L * 4;
  const int heads = p.c.heads * p.group;
  uint32_t b = blockIdx.x * PER + sub;          // [sequence][token][head], below 2^30
  const int head = (int)next_digit(b, heads);
  const int tok = (int)next_digit(b, max(p.tokens, 1));
  // (the kernels before this one start behind all that was before them, so the lengths
  // are there already)
  int row0 = 0, n = 0, kv = 0;
  bool in = (int)b < p.c.batch && sequence_of(p.c, (int)b, row0, n, kv) && tok < n &&
            n * p.group <= p.few_rows;
  const int r = tok * p.group + head % p.group, tile = r / kRows;
  const int len = split_tokens(kv);
  const int last = min((tile + 1) * kRows, n * p.group) - 1;      // of the tile's rows
  int parts = in ? tile_parts(kv - n + last / p.group, len) : 1;
  in = in && parts > 1;
  griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x < 2) p.next[threadIdx.x] = 0;
  if (!__any_sync(0xffffffffu, in)) return;         // the same in all warps
  if (!in) parts = 1;
  const int64_t first =
      in ? ((first_tile(p.by_row, (int)b, row0, p.group, p.max_tiles) + tile) * p.c.heads +
            head / p.group) * p.max_parts
         : 0;
  const float* ml = p.part_ml + (first * p.part_rows + r % kRows) * kPartWords;
  const float* at = p.parts + (first * p.part_rows + r % kRows) * D + d;
  uint4 x[B][C];
  auto ask = [&](int q0) {
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int q = q0 + kJoinSums * i + W * k + warp;
        x[i][k] = make_uint4(0, 0, 0, 0);
        if (q < parts) x[i][k] = ldg_cg_v4(at + (int64_t)q * p.part_rows * D);
      }
  };
  ask(0);
  // m, l and c, by the first warps, a row each: parts `lane` and
  // `lane` + 32
  for (int k = warp; k < PER; k += W) {
    const float* from = reinterpret_cast<const float*>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(ml), k * L));
    const int count = __shfl_sync(0xffffffffu, parts, k * L);
    float4 u[SL];
    float top = neg_inf();
    int c = c_of(kNoExp);
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      u[i] = make_float4(neg_inf(), 0.0f, __int_as_float(c), 0.0f);
      if (lane + 32 * i < count && count > 1)
        u[i] = __ldcg(reinterpret_cast<const float4*>(
            from + (int64_t)(lane + 32 * i) * p.part_rows * kPartWords));
    }
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      top = fmaxf(top, u[i].x);
      c = max(c, __float_as_int(u[i].z));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    c = __reduce_max_sync(0xffffffffu, c);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const float y = u[i].x == neg_inf() ? 1.0f : pow2_down(u[i].x - top);
      weight[k][lane + 32 * i] = y;
      sum = fmaf(u[i].y * pow2(c - __float_as_int(u[i].z)), y, sum);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      inverse[k] = sum == 0.0f ? 0.0f : 1.0f / sum;
      unit[k] = pow2(c);
    }
  }
  __syncthreads();
  float4 v[C];
#pragma unroll
  for (int k = 0; k < C; ++k) v[k] = make_float4(0, 0, 0, 0);
  const int most = __reduce_max_sync(0xffffffffu, parts);
  for (int q0 = 0; q0 < most; q0 += kJoinSums * B) {
    if (q0) ask(q0);
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int q = q0 + kJoinSums * i + W * k + warp;
        if (q < parts) {
          const float y = weight[sub][q];
          v[k].x = fmaf(__uint_as_float(x[i][k].x), y, v[k].x);
          v[k].y = fmaf(__uint_as_float(x[i][k].y), y, v[k].y);
          v[k].z = fmaf(__uint_as_float(x[i][k].z), y, v[k].z);
          v[k].w = fmaf(__uint_as_float(x[i][k].w), y, v[k].w);
        }
      }
  }
#pragma unroll
  for (int k = 0; k < C; ++k) sums[warp + W * k][lane] = v[k];
  __syncthreads();
  if (warp != 0 || !in) return;
  float4 o = sums[0][lane];
#pragma unroll
  for (int i = 1; i < kJoinSums; ++i) {
    const float4 u = sums[i][lane];
    o.x += u.x; o.y += u.y; o.z += u.z; o.w += u.w;
  }
  const float inv = inverse[sub], by = unit[sub];
  o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
  *reinterpret_cast<uint2*>(p.out + (int64_t)(row0 + tok) * p.ld_out + (int64_t)head * D + d) =
      make_uint2(f32x2_to_bf16x2_bits(o.x * by, o.y * by),
                 f32x2_to_bf16x2_bits(o.z * by, o.w * by));
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Smem<D, NT>::kBlocks)
    split_kernel(const __grid_constant__ AttnParams p) {
  using S = Smem<D, NT>;
  extern __shared__ __align__(1024) uint8_t raw[];
  S& s = *reinterpret_cast<S*>(raw + S::kRing);
  int* prefix = reinterpret_cast<int*>(raw + S::kRing + sizeof(S));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&s.full[i], 2);
      mbar_init(&s.empty[i], kTeam);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.item_full[i], 1);
      mbar_init(&s.item_empty[i], kTeam);
    }
    mbar_init(&s.sums_full, kTeam);
    mbar_init(&s.sums_empty, kTeam);
    s.dead = 0;
    fence_mbar_init();
    prefetch_tensormap(&p.tm);
  }
  // (the prompt kernel lets this one start behind its own wait: what was before is there)
  if (!p.after_prompt) griddep_wait();
  griddep_launch();                     // of the join kernel, which waits for this one's end

  // items of each sequence, summed up
  int carry = 0;
  for (int b0 = 0; b0 < p.c.batch; b0 += kThreads) {
    const int b = b0 + tid;
    int count = 0;
    if (b < p.c.batch) {
      int row0, n, kv;
      const bool fine = sequence_of(p.c, b, row0, n, kv);
      if (b < kSeqs) s.seq[b] = make_int3(row0, n, kv);
      if (!fine) {
        if (blockIdx.x == 0) atomicOr(p.c.status, kStatusIndexRange);
      } else if (n > 0 && n * p.group <= p.few_rows) {
        count = (n * p.group + kRows - 1) / kRows * seq_splits(kv, split_tokens(kv)) * p.c.heads;
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
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += s.scan[w];
      carry += s.scan[w];
    }
    if (b < p.c.batch) prefix[b] = before + sum - count;
  }
  if (tid == 0 && (p.flags & IG_FLAG_TEST_COPY_TIMEOUT)) {      // as if a wait had expired
    s.dead = 1;
    atomicOr(p.c.status, kStatusTimeout);
  }
  __syncthreads();

  if (warp < kTeam)
    compute_warp<D, NT>(p, s, raw, warp, lane);
  else
    copy_warp<D, NT>(p, s, raw, prefix, carry, lane);
  if (p.after_prompt) griddep_wait();   // the joins wait for this kernel's end alone
}

template <int D, int NT>
cudaError_t launch(const AttnParams& p, cudaStream_t st) {
  const size_t smem = Smem<D, NT>::kRing + sizeof(Smem<D, NT>) + sizeof(int) * (size_t)p.c.batch;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(split_kernel<D, NT>), allowed);
  if (e != cudaSuccess) return e;
  return launch_pdl(split_kernel<D, NT>, dim3(Smem<D, NT>::kBlocks * sm_count()), dim3(kThreads),
                    smem, st, p);
}

template <int D>
cudaError_t launch_join(const AttnParams& p, cudaStream_t st) {
  AttnJoinParams j;
  j.next = p.next;
  j.c = p.c;
  j.out = p.out;
  j.parts = p.parts;
  j.part_ml = p.part_ml;
  j.ld_out = p.ld_out;
  j.group = p.group;
  j.few_rows = p.few_rows;
  j.max_tiles = p.max_tiles;
  j.by_row = p.tiles_by_row;
  j.max_parts = p.max_parts;
  j.part_rows = p.part_rows;
  const int most = p.few_rows / p.group;              // tokens of a sequence of this kernel
  j.tokens = p.c.max_q < most ? p.c.max_q : most;
  // (no tokens: a kv head has too many rows; one part: nothing to join. A block
  // all the same, for the items' counter)
  const bool any = j.tokens > 0 && p.max_parts > 1;
  const int64_t rows = any ? (int64_t)p.c.batch * j.tokens * p.c.heads * p.group : 1;
  if (!any) j.c.batch = 0;
  constexpr int PER = 128 / D;
  const dim3 grid((unsigned)((rows + PER - 1) / PER));
  if (grid.x > 4u * sm_count()) return launch_pdl(join_kernel<D, 1>, grid, dim3(32), 0, st, j);
  return launch_pdl(join_kernel<D, 8>, grid, dim3(256), 0, st, j);
}

}  // namespace

// A tile of 8 rows at most (as many as a kv head can have in this call) leaves
// half the 16 columns unused: one MMA less of two, and three blocks to an SM.
// The rows' bits are the same in both.
cudaError_t launch_attention_split(const AttnParams& p, int head_dim, cudaStream_t st) {
  if (p.part_rows <= 8) return head_dim == 128 ? launch<128, 1>(p, st) : launch<64, 1>(p, st);
  return head_dim == 128 ? launch<128, 2>(p, st) : launch<64, 2>(p, st);
}
cudaError_t launch_attention_join(const AttnParams& p, int head_dim, cudaStream_t st) {
  return head_dim == 128 ? launch_join<128>(p, st) : launch_join<64>(p, st);
}

}  // namespace ig
