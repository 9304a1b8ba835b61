// Attention of many query rows over the 8-bit paged cache: prompts and chunks of
// them, on the tcgen05 tensor cores.
//
// A block takes 256 rows of one kv head (`group` query heads for each new
// token), two tiles of 128 (the MMA's M), and walks the tokens that they see 128
// at a time:
//   S = Q K^T   kind::f8f6f4. The keys' codes are the B operand as TMA leaves
//               them. A query row, scaled by a power of two to a maximum of 128
//               to 256, is the sum of two e4m3 numbers: 8 significant bits are 4
//               and, of what is left, 4 more (values under 2^-9 of the row's
//               maximum are off by at most 2^-17 of it). Two MMAs at twice the
//               rate of one in FP16, and no conversion of the keys.
//   O += P V    kind::f16. P goes back to tensor memory over S, as FP16; the
//               values' codes are FP16 numbers too, converted by a warpgroup of
//               their own into the MMA's order (tokens along K, so V as it lies:
//               the MN-major operand).
// Softmax as in the split kernel: base 2, whole exponents, a row's maximum raised
// only past m + 7, value scales folded into P ("a row's sums" in attention.cuh), key
// scales into the logits.
//
// Warps: 0-7 and 8-15 the softmax of a tile each, half a row to a thread; 16-19
// the values; 20 the copies; 21 the MMAs; 22 the pages and scales. The two tiles
// take turns: while one is in the softmax the tensor cores work on the other. Where a
// block has 128 rows at most, both tiles have these rows, one the even steps and one
// the odd ones, and their sums are joined at the end (64 sequences of 64 rows over 8192
// tokens: a step 1700 clocks instead of 3500).
//
// What bounds it: a step of both tiles takes 3500 clocks of which the tensor cores work
// 2050 by their nominal rate; the rest is the chain products - maximum - exponentials -
// P of the two tiles, whose issue slots (54 %) and barriers do not all hide behind the
// other tile's. Beside its steps a block costs 23000 clocks: 2400 to find its rows,
// 9000 to load and convert 64 KB of queries, 1900 to the first products, 2300 from the
// last P to the last sums, 5500 for the results, 2100 to the next block. 2048 tokens over
// 32768 (32 query, 8 kv heads of 128): 884 us, 1205 TFLOP/s; three prompts of up to 4095
// tokens 217 us.
#include "attention.cuh"
#include "umma_mx4.cuh"

namespace ig {

namespace {

constexpr int kTile = 128;              // rows of a tile, tokens of a step
constexpr int kThreads = 768;
constexpr int kHalf = kTile / 2;        // columns of a thread
constexpr float kHeadroom = 7.0f;
constexpr float kBias = 8.0f;
constexpr float kFar = 1048576.0f;      // logits past this are rounded before they are used
constexpr int kNaNExp = 1000;           // of a block whose value scale is NaN
constexpr int kNoExp = -1000;           // of no block yet
constexpr int kNoBlock = 2000;          // tokens that no row sees, or an absent page
constexpr int kInfo = 8;                // steps whose pages and scales are held

// The block's rows.
struct Rows {
  int b, h, row0;              // sequence, kv head, the sequence's first row of q
  int tok0, rem;               // its token and query head that the block's first row is
  int rows;
  bool twin;                   // one tile of rows: the two take its steps in turn
  int low, high;               // last token that the first and the last row see
  int step0, steps;            // its steps: of the part of the tokens that is its
  int parts;                   // parts that the rows see; with several the results go to
  int64_t part;                // row `part` of the parts on
};

template <int D>
struct Smem {
  static constexpr int kPart = kTile * D;               // bytes of 128 rows of codes
  static constexpr int kQ = 0;                          // [tile][hi, lo]
  static constexpr int kK = kQ + 4 * kPart;             // [2]
  static constexpr int kV8 = kK + 2 * kPart;            // [2]
  static constexpr int kV16 = kV8 + 2 * kPart;          // [2]
  static constexpr int kEnd = kV16 + 4 * kPart;
  uint64_t k_full[2], k_empty[2], v8_full[2], v8_empty[2], v16_full[2], v16_empty[2];
  uint64_t s_full[2], p_full[2];
  uint64_t info_full[kInfo], info_empty[kInfo], q_full, drain;
  // of a step's 8 blocks: scale of the keys; e and 2^(c - e) for p; e or what is wrong with it
  alignas(16) float ks[kInfo][8], expo[kInfo][8], back[kInfo][8];
  int ve[kInfo][8];
  int page[kInfo][8];
  int partly[kInfo];                    // some block of the step is not there
  float more[kInfo];                    // 2^(c - c of the tile's step before)
  int c[2];                             // c in the end, of the even and the odd steps
  int nan_at[D], nans;                  // first token that makes each value NaN; whether one does
  float most[2][2][2 * kTile];          // [step % 2][half][row]: largest logit, sum
  float base[2 * kTile];                // m in the end
  uint32_t tmem;
  int dead;
  Rows it;
};

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }
__device__ __forceinline__ float qnan() { return __uint_as_float(0x7fc00000u); }
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

__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_minus(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// D[m][n] = sum_k A[m][k] B[n][k], FP32: e4m3 operands along K; FP16 with B in
// rows of n.
__host__ __device__ constexpr uint32_t idesc_f8(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_f16_nt(int m, int n) {
  return (1u << 4) | (1u << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// Rows of D bytes, swizzled by as much, 8-row groups 8 D bytes apart.
template <int D>
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)((8 * D) >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)(D == 128 ? 2 : 4) << 61;             // SWIZZLE_128B, SWIZZLE_64B
  return d;
}
// FP16 rows along n: atoms of 64 n (128 bytes) x 8 tokens, 1024 bytes, one after
// the other along the tokens; the next 64 n 128 tokens further.
__device__ __forceinline__ uint64_t desc_values(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((kTile * 128) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc) : "memory");
}
__device__ __forceinline__ void mma_f16_tm(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc) : "memory");
}
// 32 columns of this thread's lane, on their way until tmem_wait_ld; loaded32
// keeps their uses behind it.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void loaded32(float* v) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                    "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                    "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
  asm volatile("" : "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]),
                    "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]),
                    "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// N columns, 16 or 32, here when it returns.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[N]) {
  if constexpr (N == 32) {
    tmem_ld32_async(taddr, v);
    tmem_wait_ld();
    loaded32(v);
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15])
        : "r"(taddr) : "memory");
  }
}
// 16 bytes from global to shared memory, of which the first `bytes` are read and the
// others 0.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(bytes) : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Row's factor times a block's scale; not 0, which times -inf were no number.
__device__ __forceinline__ float factor(float f, float ks) {
  const float k = f * ks;
  return k < 1.18e-38f ? 1.18e-38f : k;
}
// A warpgroup's share of the block's registers (768 threads launched with 80).
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15]) : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Bounded wait that also ends when any other wait of the block gave up; with
// SLEEP a look may take 20 us, and the warp wakes up later than without (250
// clocks against 90) but issues nothing meanwhile.
__device__ __forceinline__ bool try_wait_long(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "r"(20000) : "memory");
  return ok != 0;
}
template <bool SLEEP = false, typename S>
__device__ __forceinline__ bool wait(S& s, uint64_t* bar, uint32_t parity, uint32_t* status) {
  auto look = [&] { return SLEEP ? try_wait_long(bar, parity) : mbar_try_wait(bar, parity); };
  if (look()) return true;
  const long long t0 = clock64();
  while (!look()) {
    __nanosleep(20);
    if (*reinterpret_cast<volatile int*>(&s.dead)) return false;
    if (clock64() - t0 > (1ll << 31)) {
      *reinterpret_cast<volatile int*>(&s.dead) = 1;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}

// Barrier of a tile's eight warps (or of both tiles'); whether all came with true.
template <int N = 256>
__device__ __forceinline__ bool all_of(int bar, bool mine) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "bar.red.and.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all) : "r"((uint32_t)mine), "r"(bar), "n"(N) : "memory");
  return all != 0;
}

// row / group for the rows of a block (and the first one's remainder): a float's
// rounding is far from the 0.5 / group that is between a half and a whole number.
__device__ __forceinline__ int token_of(const AttnParams& p, int row) {
  return (int)(((float)row + 0.5f) * p.group_rcp);
}

// The block's queries as the two numbers that make up each: of the warp's 32 rows and its
// half of D, 8 values of a row to a lane at a time, the row's 8 lanes (D = 64: 4) side by
// side. All rows are asked for at once and wait, as bf16, in the place of the first
// converted values. Returns what a product of the lane's own row is worth in the
// softmax's base 2. Rolled loops, and not inlined, as what stores the results: the code of
// what a block does once comes from far.
template <int D>
__device__ __noinline__ float convert_queries(const AttnParams& p, Smem<D>& s, uint8_t* raw) {
  using S = Smem<D>;
  constexpr int CH = D / 16;            // 16-byte chunks of half a row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = warp >> 3, half = (warp >> 2) & 1, ch = lane % CH;
  const int warp_row = t * kTile + (warp & 3) * 32;
  // (the two tiles have the same rows where they take turns)
  const Rows& it = s.it;
  const int same = it.twin ? t * kTile : 0, rows = it.rows + same;
  uint8_t* const from = raw + S::kV16 + half * D + ch * 16;
  {
    const __nv_bfloat16* q = p.q + (int64_t)(it.row0 + it.tok0) * p.ld_q +
                             (int64_t)it.h * p.group * D + half * (D / 2) + ch * 8;
#pragma unroll 1
    for (int r = warp_row + lane / CH; r < warp_row + 32; r += 32 / CH) {
      const int at = it.rem + r - same, tok = token_of(p, at);
      const bool in = r < rows;
      cp_async16(from + r * 2 * D, in ? q + tok * p.ld_q + (at - tok * p.group) * D : q, in ? 16 : 0);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  __syncwarp();
#pragma unroll 2
  for (int r = warp_row + lane / CH; r < warp_row + 32; r += 32 / CH) {
    const uint4 w = *reinterpret_cast<const uint4*>(from + r * 2 * D);
    // (magnitudes of bf16 compare as whole numbers do)
    uint32_t top = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                            __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
#pragma unroll
    for (int o = CH / 2; o; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (ch == 0) s.most[0][half][r] = __uint_as_float(max(top & 0xffffu, top >> 16));
  }
  asm volatile("bar.sync %0, 64;" ::"r"(1 + t * 4 + (warp & 3)) : "memory");
  auto exponent = [&](int r) {          // the row's largest value is below 2^(this - 126)
    return (int)(max(__float_as_uint(s.most[0][0][r]), __float_as_uint(s.most[0][1][r])) >> 7);
  };
#pragma unroll 1
  for (int r = warp_row + lane / CH; r < warp_row + 32; r += 32 / CH) {
    const uint4 w = *reinterpret_cast<const uint4*>(from + r * 2 * D);
    const int e = exponent(r);
    float up = e == 255 ? qnan() : pow2(134 - max(e, 20));
    if (p.scale_log2 < 0.0f) up = -up;
    // (as FP16 it loses what is under 2^-32 of the row's largest)
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = split2(mul2(pair2(bf16lo(u[k]), bf16hi(u[k])), pair2(up, up)));
      const uint32_t h = f16x2_of(x.x, x.y);
      hi[k] = f16x2_to_e4m3x2(h);
      lo[k] = f16x2_to_e4m3x2(f16x2_minus(h, e4m3x2_to_f16x2((uint16_t)hi[k])));
    }
    const int c16 = half * (D / 32) + ch / 2;           // 16-byte chunk of a row of codes
    const int at = (D == 128 ? c16 ^ (r & 7) : c16 ^ ((r >> 1) & 3)) * 16 + (ch & 1) * 8;
    uint8_t* dst = raw + S::kQ + t * 2 * S::kPart + (r & 127) * D + at;
    *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
    *reinterpret_cast<uint2*>(dst + S::kPart) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
  }
  const int e = exponent(warp_row + lane);
  return fabsf(p.scale_log2) * (e == 255 ? 1.0f : pow2(max(e, 20) - 134));
}

// What a thread has of the results, half a row (of two tiles that took turns over the
// same row a quarter, and both their sums): into the output or, of one part of
// several, as it stands into the workspace. m, l: maximum and sum of p of its tile.
template <int D>
__device__ __noinline__ void store_results(const AttnParams& p, Smem<D>& s, uint8_t* raw,
                                           float m, float l, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = (warp >> 2) & 1;
  const Rows& it = s.it;
  const bool twin = it.twin;
  const int t = warp >> 3, local = (warp & 3) * 32 + lane, my_row = twin ? local : t * kTile + local;
  const int first = twin ? (2 * t + half) * (D / 4) : half * (D / 2), count = twin ? D / 4 : D / 2;
  int c = s.c[1];
  float w0 = 1.0f, w1 = 0.0f;
  uint32_t from = tmem + 2 * kTile + ((uint32_t)((warp & 3) * 32) << 16) + first;
  if (!twin) {
    from += t * D;
    if (it.steps & 1) c = s.c[0];
  } else {
    const float m0 = s.base[local], m1 = s.base[kTile + local];
    const float l0 = s.most[1][0][local] + s.most[1][1][local];
    const float l1 = s.most[1][0][kTile + local] + s.most[1][1][kTile + local];
    c = max(s.c[0], s.c[1]);
    m = fmaxf(m0, m1);
    w0 = m0 == neg_inf() ? 1.0f : pow2_down(m0 - m);
    w1 = m1 == neg_inf() ? 1.0f : pow2_down(m1 - m);
    l = l0 * pow2(c - s.c[0]) * w0 + l1 * pow2(c - s.c[1]) * w1;
  }
  const bool whole = it.parts == 1;
  const int lim = it.low + token_of(p, it.rem + my_row);
  const bool nans = s.nans;
  // (where l is 0 so are the sums)
  // (one after the other: 2^c / l may be below FP32's range where the result is not)
  const float inv = !whole ? 1.0f : l == 0.0f ? 0.0f : __fdividef(1.0f, l), unit = pow2(c);
  // the warp's 32 rows of `chunks` 16-byte chunks, in shared memory that nothing else
  // uses any more: a lane has a row there, and takes whole lines of the rows from there
  const int shift = (whole ? 3 : 4) - (twin ? 1 : 0) - (D == 64 ? 1 : 0);
  const int chunks = 1 << shift;
  uint4* const mine = reinterpret_cast<uint4*>(raw) + (warp * 32 << shift);
  auto place = [&](int r, int ch) {
    return (r << shift) + (ch ^ (shift >= 3 ? r & 7 : shift == 2 ? r >> 1 & 3 : r >> 2 & 1));
  };
  constexpr int N = D / 4;              // columns at a time: all that a thread has of two tiles
#pragma unroll 1
  for (int c = 0; c < count; c += N) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    if (it.steps > 0) tmem_ld<N>(from + c, v);
    if (twin) {
      float u[N];
#pragma unroll
      for (int i = 0; i < N; ++i) u[i] = 0.0f;
      if (it.steps > 1) tmem_ld<N>(from + D + c, u);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] * w0 + u[i] * w1;
    }
    if (nans) {
#pragma unroll 1
      for (int i = 0; i < N; ++i) {
        const bool bad = lim >= s.nan_at[first + c + i];
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (k == i && bad) v[k] = qnan();
      }
    }
    if (whole) {
#pragma unroll
      for (int i = 0; i < N / 8; ++i) {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          u[k] = f32x2_to_bf16x2_bits(v[8 * i + 2 * k] * inv * unit, v[8 * i + 2 * k + 1] * inv * unit);
        mine[place(lane, c / 8 + i)] = make_uint4(u[0], u[1], u[2], u[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        *reinterpret_cast<float4*>(&mine[place(lane, c / 4 + i)]) =
            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  }
  if (my_row < it.rows && !whole && first == 0)
    *reinterpret_cast<float4*>(p.big_ml + (it.part + my_row) * kPartWords) =
        make_float4(m, l, __int_as_float(c), 0.0f);
  __syncwarp();
  const int ch = lane & (chunks - 1), row0 = my_row - lane;
#pragma unroll 1
  for (int r = lane >> shift; r < 32 && row0 + r < it.rows; r += 32 >> shift) {
    const uint4 u = mine[place(r, ch)];
    const int row = row0 + r;
    if (whole) {
      const int tok = token_of(p, it.rem + row);
      reinterpret_cast<uint4*>(p.out + (int64_t)(it.row0 + it.tok0 + tok) * p.ld_out +
                               (int64_t)(it.h * p.group + it.rem + row - tok * p.group) * D +
                               first)[ch] = u;
    } else {
      reinterpret_cast<uint4*>(p.big + (it.part + row) * D + first)[ch] = u;
    }
  }
}

// The parts of the rows of a token, joined in their order: D / 4 lanes to a query head,
// 4 values each; all parts of a row asked for together.
constexpr int kJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) prompt_join_kernel(const AttnJoinParams p) {
  constexpr int L = D / 4, PER = 32 / L;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / L, d = lane % L * 4;
  griddep_launch();                     // of the split kernel's join, which waits for the end
  griddep_wait();
  if (__ldcg(p.next + 1) == 0) return;  // no sequence was cut
  const int heads = p.c.heads * p.group;
  const unsigned chunks = (unsigned)(heads + kJoinWarps * PER - 1) / (kJoinWarps * PER);
  for (int64_t item = blockIdx.x; item < p.c.T * chunks; item += gridDim.x) {
    const int t = (int)(item / chunks);
    const int h0 = ((int)(item - (int64_t)t * chunks) * kJoinWarps + warp) * PER;
    int b = 0;
    for (int hi = p.c.batch; hi - b > 1;) {       // the last sequence that starts at or before t
      const int mid = (b + hi) >> 1;
      if (__ldg(p.c.cu + mid) <= t) b = mid; else hi = mid;
    }
    int row0, n, kv;
    if (!sequence_of(p.c, b, row0, n, kv) || t < row0 || t >= row0 + n || n * p.group <= p.few_rows)
      continue;
    const int cut = prompt_parts(n * p.group, kv, p.c.heads);
    if (cut == 1) continue;
    const int len = prompt_len(kv, cut), tok = t - row0;
    const int tiles = (n * p.group + kPromptRows - 1) / kPromptRows;
    if (h0 < heads) {
      const int h = min(h0 + sub, heads - 1), r = tok * p.group + h % p.group;
      const int tile = r / kPromptRows;
      const int last = min((tile + 1) * kPromptRows, n * p.group) - 1;
      const int parts = prompt_seen(kv - n + last / p.group, len);
      const bool in = h0 + sub < heads && parts > 1;
      // item (tiles - 1 - tile, part, kv head) of the sequence
      const int room = item_rows(n * p.group);
      const int64_t pitch = (int64_t)p.c.heads * room;
      const int64_t at = first_big(p.by_row, b, row0, p.group, p.part_rows) +
                         (int64_t)((tiles - 1 - tile) * cut * p.c.heads + h / p.group) * room +
                         r % kPromptRows;
      uint4 x[kPromptParts];
#pragma unroll
      for (int q = 0; q < kPromptParts; ++q) {
        x[q] = make_uint4(0, 0, 0, 0);
        if (in && q < parts) x[q] = ldg_cg_v4(p.parts + (at + q * pitch) * D + d);
      }
      float w = 0.0f, inv = 0.0f, unit = 0.0f;      // of part `lane % L` of this lane's row
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int64_t from = __shfl_sync(0xffffffffu, at, k * L);
        const int count = __shfl_sync(0xffffffffu, in ? parts : 0, k * L);
        float4 u = make_float4(neg_inf(), 0.0f, __int_as_float(c_of(kNoExp)), 0.0f);
        if (lane < count)
          u = __ldcg(reinterpret_cast<const float4*>(p.part_ml + (from + lane * pitch) * kPartWords));
        float top = u.x;
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int c = __reduce_max_sync(0xffffffffu, __float_as_int(u.z));
        const float y = u.x == neg_inf() ? 1.0f : pow2_down(u.x - top);
        float sum = u.y * pow2(c - __float_as_int(u.z)) * y;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float mine = __shfl_sync(0xffffffffu, y, lane % L);
        if (k == sub) {
          w = mine;
          inv = sum == 0.0f ? 0.0f : 1.0f / sum;
          unit = pow2(c);
        }
      }
      float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < kPromptParts; ++q) {
        const float y = __shfl_sync(0xffffffffu, w, sub * L + q);
        if (q < parts) {
          v.x = fmaf(__uint_as_float(x[q].x), y, v.x);
          v.y = fmaf(__uint_as_float(x[q].y), y, v.y);
          v.z = fmaf(__uint_as_float(x[q].z), y, v.z);
          v.w = fmaf(__uint_as_float(x[q].w), y, v.w);
        }
      }
      if (in)
        *reinterpret_cast<uint2*>(p.out + (int64_t)t * p.ld_out + (int64_t)h * D + d) =
            make_uint2(f32x2_to_bf16x2_bits(v.x * inv * unit, v.y * inv * unit),
                       f32x2_to_bf16x2_bits(v.z * inv * unit, v.w * inv * unit));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ AttnParams p) {
  using S = Smem<D>;
  extern __shared__ __align__(1024) uint8_t raw[];
  S& s = *reinterpret_cast<S*>(raw + S::kEnd);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // (not by warp 0, which looks for the block's rows)
  if (tid == 0) {
    s.dead = 0;
    s.nans = 0;
    s.c[0] = s.c[1] = c_of(kNoExp);     // (a block without steps reads it all the same)
  }
  if (tid == 64) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.k_full[i], 1);
      mbar_init(&s.k_empty[i], 1);
      mbar_init(&s.v8_full[i], 1);
      mbar_init(&s.v8_empty[i], 4);
      mbar_init(&s.v16_full[i], 4);
      mbar_init(&s.v16_empty[i], 1);
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], 8);
    }
    for (int i = 0; i < kInfo; ++i) mbar_init(&s.info_full[i], 1);
    mbar_init(&s.q_full, 16);
    mbar_init(&s.drain, 1);
    fence_mbar_init();
    prefetch_tensormap(&p.tm);
  }
  if (tid >= 128 && tid < 128 + D) s.nan_at[tid - 128] = 0x7fffffff;
  griddep_wait();
  griddep_launch();                     // of the split kernel: all it reads is there
  if (tid == 0 && (p.flags & IG_FLAG_TEST_COPY_TIMEOUT)) {      // as if a wait had expired
    s.dead = 1;
    atomicOr(p.c.status, kStatusTimeout);
  }

  // the block's rows: sequences in order, a sequence's last rows first
  if (warp == 0) {
    int at = blockIdx.x, found = -1;
    for (int b0 = 0; b0 < p.c.batch && found < 0; b0 += 32) {
      int row0, n, kv, count = 0, tiles = 0, cut = 1;
      if (b0 + lane < p.c.batch && sequence_of(p.c, b0 + lane, row0, n, kv) &&
          n * p.group > p.few_rows) {
        tiles = (n * p.group + 2 * kTile - 1) / (2 * kTile);
        cut = prompt_parts(n * p.group, kv, p.c.heads);
        count = tiles * p.c.heads * cut;
      }
      int sum = count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, at < sum);
      if (hit) {
        const int l = __ffs(hit) - 1;
        if (lane == l) {
          uint32_t v = at - (sum - count), rest;
          const int first = b0 + l, item = (int)v;
          Rows it;
          rest = v;
          v = divide(rest, p.c.heads, p.heads_magic);
          it.h = (int)rest;
          int part = 0;
          if (cut > 1) part = (int)next_digit(v, cut);
          const int row = (tiles - 1 - (int)v) * 2 * kTile;
          it.row0 = row0;
          rest = row;
          it.tok0 = (int)divide(rest, p.group, p.group_magic);
          it.rem = (int)rest;
          it.rows = min(2 * kTile, n * p.group - row);
          it.twin = it.rows <= kTile;
          it.low = kv - n + it.tok0;
          it.high = it.low + token_of(p, it.rem + it.rows - 1);
          it.step0 = 0;
          it.steps = it.high >= 0 ? it.high / kTile + 1 : 0;
          it.parts = 1;
          it.part = 0;
          if (cut > 1) {
            const int len = prompt_len(kv, cut);
            it.parts = prompt_seen(it.high, len);
            it.step0 = part * len;
            it.steps = max(0, min(it.steps, it.step0 + len) - it.step0);
            it.part = first_big(p.big_by_row, first, row0, p.group, p.big_rows) +
                      (int64_t)item * item_rows(n * p.group);
          }
          it.b = part < it.parts ? first : -1;
          s.it = it;
          if (it.parts > 1) p.next[1] = 1;      // there are parts to join
        }
        found = b0 + l;
      }
      at -= __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0 && found < 0) s.it.b = -1;
    __syncwarp();
    if (s.it.b >= 0) {
      // of a step's readers: softmax warps of one tile or of both, values, copies
      if (lane < kInfo) mbar_init(&s.info_empty[lane], (s.it.twin ? 8 : 16) + 5);
      fence_mbar_init();
    }
  } else if (warp == 1) {
    tmem_alloc(&s.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  if (s.it.b < 0) {
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }
  const int h = s.it.h, low = s.it.low, high = s.it.high, steps = s.it.steps;
  const bool twin = s.it.twin;
  const int tok0 = s.it.step0 * kTile;  // its first token
  const int half = (warp >> 2) & 1;

  // 512 threads with 96 registers and 256 with 48: the 61440 of the launch
  if (warp < 16) {
    // ---------------------------------------------------------------- softmax
    // a tile's steps: all, or every second one from its number on
    more_registers<96>();
    const int t = warp >> 3, mine = twin ? (steps + 1 - t) >> 1 : steps;
    const int slot = t * kTile + (warp & 3) * 32 + lane;
    const int my_row = twin ? slot - t * kTile : slot, top_row = twin ? 0 : t * kTile;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + t * kTile + lanes;
    const uint32_t to = tmem + 2 * kTile + t * D + half * (D / 2) + lanes;
    // (tokens from the part's first on)
    const int tile_low = low - tok0 + token_of(p, s.it.rem + top_row);
    const int lim = my_row < s.it.rows ? low - tok0 + token_of(p, s.it.rem + my_row)
                                       : 0x7fffffff;                    // last token it sees
    const int pair_bar = 1 + t * 4 + (warp & 3);        // the two warps of these rows
    bool ok = all_of(9 + t, !*reinterpret_cast<volatile int*>(&s.dead));
    float f = 0.0f;                     // logit of a product, base 2
    if (ok) {
      // (without steps nobody reads them, and the results go through their place)
      if (steps > 0) f = convert_queries<D>(p, s, raw);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.q_full);
    }
    float m = neg_inf(), l = 0.0f;
    for (int n = 0; ok && n < mine; ++n) {
      const int j = twin ? 2 * n + t : n, in = j % kInfo;
      ok = wait(s, &s.info_full[in], (j / kInfo) & 1, p.c.status);
      // what the scales have to say is here before the products are
      const float4 ks = *reinterpret_cast<const float4*>(&s.ks[in][4 * half]);
      const float4 expo = *reinterpret_cast<const float4*>(&s.expo[in][4 * half]);
      const float4 back = *reinterpret_cast<const float4*>(&s.back[in][4 * half]);
      float k[4] = {factor(f, ks.x), factor(f, ks.y), factor(f, ks.z), factor(f, ks.w)};
      const bool partly = s.partly[in];
      l *= s.more[in];
      // one warp of the tile looks for the products, the others wait for it: looks
      // share a queue with the exponentials
      if ((warp & 7) == 0) ok = ok && wait(s, &s.s_full[t], n & 1, p.c.status);
      ok = all_of(9 + t, ok);
      if (!ok) break;
      tc_fence_after();
      const int t0 = j * kTile + half * kHalf;
      // half a row's products, all in registers; columns that the row does not
      // see are -inf: in few steps, so the others have no look at them
      float v[kHalf];
      tmem_ld32_async(ts + half * kHalf, v);
      tmem_ld32_async(ts + half * kHalf + 32, v + 32);
      tmem_wait_ld();
      loaded32(v);
      loaded32(v + 32);
      if (t0 + kHalf - 1 > tile_low || partly) {
        const int seen = lim - t0;
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
          if (i > seen) v[i] = neg_inf();
        if (partly) {
#pragma unroll
          for (int i = 0; i < kHalf; ++i)
            if (s.ve[in][4 * half + i / 16] == kNoBlock) v[i] = neg_inf();
        }
      }
      float e[4] = {expo.x, expo.y, expo.z, expo.w}, y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) y[q] = max3(v[16 * q], v[16 * q + 1], v[16 * q + 2]);
#pragma unroll
      for (int i = 3; i < 15; i += 2)
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] = max3(y[q], v[16 * q + i], v[16 * q + i + 1]);
#pragma unroll
      for (int q = 0; q < 4; ++q) y[q] = __fmaf_rn(fmaxf(y[q], v[16 * q + 15]), k[q], e[q]);
      float x = fmaxf(max3(y[0], y[1], y[2]), y[3]);
      // the other half's; both have their products in registers from here on, so
      // P may take the place of S
      s.most[n & 1][half][slot] = x;
      asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
      x = fmaxf(x, s.most[n & 1][half ^ 1][slot]);
      float down = 1.0f;
      if (x > __fadd_rd(m, kHeadroom)) {
        const float up = ceilf(x);
        down = m == neg_inf() ? 0.0f : pow2_down(m - up);
        m = up;
        l *= down;
      }
      float base = m == neg_inf() ? 0.0f : m;
      if (__builtin_expect(fabsf(base) > kFar, 0)) {
        // m is a rounded logit, and what the product below has beyond it is no longer small
        // against p's range: logits as they were rounded for m. (That such rows are asked
        // for costs 1.1 %: 2048 tokens over 8192 222.4 us without, 224.9 with.)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int i = 16 * q; i < 16 * q + 16; ++i)
            v[i] = __fsub_rn(__fmaf_rn(v[i], k[q], e[q]), base);
          k[q] = 1.0f;
          e[q] = 0.0f;
        }
        base = 0.0f;
      }
      base -= kBias;
      const float off[4] = {e[0] - base, e[1] - base, e[2] - base, e[3] - base};
      float sums[4];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t u[16];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int blk = 2 * c + q;
          const uint64_t kk = pair2(k[blk], k[blk]), oo = pair2(off[blk], off[blk]);
          uint64_t sum = 0;
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float* at = v + 16 * blk + i;
            const float2 z = split2(fma2(pair2(at[0], at[1]), kk, oo));
            const float a = ex2(z.x), d = ex2(z.y);
            sum = add2(sum, pair2(a, d));
            u[8 * q + i / 2] = f16x2_of(a, d);
          }
          const float2 both = split2(sum);
          sums[blk] = both.x + both.y;
        }
        tmem_st16(ts + 32 * half + 16 * c, u);
      }
      l = fmaf(sums[0], back.x, l);
      l = fmaf(sums[1], back.y, l);
      l = fmaf(sums[2], back.z, l);
      l = fmaf(sums[3], back.w, l);
      // the sums so far by the new maximum
      if (n > 0 && __any_sync(0xffffffffu, down != 1.0f)) {
        constexpr int N = D / 2 < 32 ? D / 2 : 32;
#pragma unroll
        for (int c = 0; c < D / 2; c += N) {
          float o[32];
          tmem_ld32_async(to + c, o);
          tmem_wait_ld();
          loaded32(o);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t u[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) u[q] = __float_as_uint(o[16 * i + q] * down);
            tmem_st16(to + c + 16 * i, u);
          }
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s.info_empty[in]);
        mbar_arrive(&s.p_full[t]);
      }
    }
    // ---- the rows' results
    if (ok && mine > 0) {
      if ((warp & 7) == 0) ok = wait(s, &s.s_full[t], mine & 1, p.c.status);
      ok = all_of(9 + t, ok);
    }
    tc_fence_after();
    if (twin) {
      tc_fence_before();
      ok = all_of<512>(11, ok);         // no maximum is looked at any more
      s.most[1][half][slot] = l;
      if (half == 0) s.base[slot] = m;
      ok = all_of<512>(11, ok);
      tc_fence_after();
    } else if (ok) {
      // (the last step's maxima may still be read, in the place of its parity)
      s.most[mine & 1][half][slot] = l;
      asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
      // (first half) + (second half), for both the same
      l = s.most[mine & 1][0][slot] + s.most[mine & 1][1][slot];
    }
    if (ok) store_results<D>(p, s, raw, m, l, tmem);
  } else if (warp < 20) {
    // ----------------------------------------------------------------- values
    fewer_registers<48>();
    const int r = tid - 512;            // token of the step
    const int lo = low - tok0, hi = high - tok0;        // from the part's first token on
    bool ok = wait<true>(s, &s.q_full, 0, p.c.status);  // the queries were where the values go
    for (int j = 0; j < steps; ++j) {
      const int in = j % kInfo, st = j & 1;
      ok = ok && wait(s, &s.info_full[in], (j / kInfo) & 1, p.c.status) &&
                wait<true>(s, &s.v8_full[st], (j >> 1) & 1, p.c.status) &&
                wait<true>(s, &s.v16_empty[st], ((j >> 1) & 1) ^ 1, p.c.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int at = j * kTile + r, e = s.ve[in][r >> 4];
      const uint8_t* src = raw + S::kV8 + st * S::kPart + r * D;
      uint8_t* dst = raw + S::kV16 + st * 2 * S::kPart + r * 128;
#pragma unroll 1
      for (int d = 0; d < D / 64; ++d) {          // 64 values at a time
        uint32_t u[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ch = 4 * d + i;
          const uint4 x = *reinterpret_cast<const uint4*>(
              src + (D == 128 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3)) * 16);
          u[4 * i] = x.x; u[4 * i + 1] = x.y; u[4 * i + 2] = x.z; u[4 * i + 3] = x.w;
        }
        if (at > lo || e >= kNaNExp) {
          if (at > hi || e == kNoBlock) {
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = 0;     // p is 0, but 0 times NaN is not
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (e == kNaNExp) u[i] = 0x7f7f7f7fu;
              // seen by some rows only: a NaN is kept for those
              const uint32_t bad = ((u[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              if (at > lo && bad) {
                s.nans = 1;
                for (int q = 0; q < 4; ++q)
                  if (bad >> (8 * q + 7) & 1) atomicMin(&s.nan_at[64 * d + 4 * i + q], tok0 + at);
                u[i] &= ~((bad >> 7) * 0xffu);
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(dst + d * (kTile * 128) + (i ^ (r & 7)) * 16) =
              make_uint4(e4m3x2_to_f16x2((uint16_t)u[2 * i]),
                         e4m3x2_to_f16x2((uint16_t)(u[2 * i] >> 16)),
                         e4m3x2_to_f16x2((uint16_t)u[2 * i + 1]),
                         e4m3x2_to_f16x2((uint16_t)(u[2 * i + 1] >> 16)));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s.info_empty[in]);
        mbar_arrive(&s.v8_empty[st]);
        mbar_arrive(&s.v16_full[st]);
      }
    }
  } else {
   fewer_registers<48>();
   if (warp == 20) {
    // ----------------------------------------------------------------- copies
    int asked = 0;
    for (int j = 0; j < steps; ++j) {
      const int in = j % kInfo, st = j & 1;
      bool ok = wait<true>(s, &s.info_full[in], (j / kInfo) & 1, p.c.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      const bool there = lane < 8 && s.ve[in][lane & 7] != kNoBlock;
      const int32_t page = s.page[in][lane & 7];
      const int row = (tok0 + j * kTile + (lane & 7) * kKvBlock) & ((1 << p.c.page_shift) - 1);
      const uint32_t have = __ballot_sync(0xffffffffu, there);
      if (lane == 0) mbar_arrive(&s.info_empty[in]);
      ok = wait<true>(s, &s.k_empty[st], ((j >> 1) & 1) ^ 1, p.c.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint32_t bytes = __popc(have) * (kKvBlock * D);
      if (lane == 0) mbar_arrive_expect_tx(&s.k_full[st], bytes);
      __syncwarp();
      if (there)
        tma_load_3d(raw + S::kK + st * S::kPart + lane * (kKvBlock * D), &p.tm, 0,
                    (h << p.c.page_shift) + row, page, &s.k_full[st]);
      ok = wait<true>(s, &s.v8_empty[st], ((j >> 1) & 1) ^ 1, p.c.status);
      if (!__all_sync(0xffffffffu, ok)) {
        // the keys' copy of this step is in flight, the values' is not
        mbar_wait_bounded(&s.k_full[st], (j >> 1) & 1, p.c.status);
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(&s.v8_full[st], bytes);
      __syncwarp();
      if (there)
        tma_load_3d(raw + S::kV8 + st * S::kPart + lane * (kKvBlock * D), &p.tm, 0,
                    ((p.c.heads + h) << p.c.page_shift) + row, page, &s.v8_full[st]);
      asked = j + 1;
    }
    if (*reinterpret_cast<volatile int*>(&s.dead)) {
      // copies still in flight land before the block leaves
      for (int j = max(asked - 2, 0); j < asked; ++j) {
        mbar_wait_bounded(&s.k_full[j & 1], (j >> 1) & 1, p.c.status);
        mbar_wait_bounded(&s.v8_full[j & 1], (j >> 1) & 1, p.c.status);
      }
    }
   } else if (warp == 22) {
    // ------------------------------------------------------- pages and scales
    // a block to a lane, four steps at a time, ahead of the copies
    const int32_t* table = p.c.table + (int64_t)s.it.b * p.c.ld_table;
    const int blocks = 1 << (p.c.page_shift - 4);
    bool ok = true;
    int expo = kNoExp;                  // the largest exponent of a value scale so far
    int old[2] = {c_of(expo), c_of(expo)};        // c of the step before and of the one before that
    for (int j0 = 0; ok && j0 < steps; j0 += 4) {
      const int tok = tok0 + j0 * kTile + lane * kKvBlock;
      bool there = tok <= high;
      int32_t page = 0;
      uint32_t kb = 127, vb = 0;
      if (there) {
        page = __ldg(table + (tok >> p.c.page_shift));
        there = page >= 0 && page < p.c.pages;
        if (!there) atomicOr(p.c.status, kStatusIndexRange);
      }
      if (there) {
        const uint8_t* sc = p.c.scales + page * p.c.scale_stride + h * blocks +
                            (tok & ((1 << p.c.page_shift) - 1)) / kKvBlock;
        kb = __ldg(sc);
        vb = __ldg(sc + p.c.heads * blocks);
      }
      // a NaN scale of keys: rows that see the block are NaN, others are to know nothing of
      // it, so it stays out of the softmax and comes with the results
      for (uint32_t bad = __ballot_sync(0xffffffffu, there && kb == 255); bad; bad &= bad - 1) {
        const int first = tok0 + j0 * kTile + (__ffs(bad) - 1) * kKvBlock;
        for (int d = lane; d < D; d += 32) atomicMin(&s.nan_at[d], first);
        s.nans = 1;
      }
      if (kb == 255) kb = 127;
      const uint32_t have = __ballot_sync(0xffffffffu, there);
      for (int i = 0; i < 4 && j0 + i < steps; ++i) {
        const int in = (j0 + i) % kInfo;
        ok = wait<true>(s, &s.info_empty[in], (((j0 + i) / kInfo) & 1) ^ 1, p.c.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const bool mine = lane >> 3 == i, scaled = there && vb != 255;
        const int e = (int)vb - 127;
        expo = max(expo, __reduce_max_sync(0xffffffffu, mine && scaled ? e : kNoExp));
        const int c = c_of(expo);
        if (mine) {
          const int with = scaled ? max(e, expo - kSpread) : 0;
          s.ks[in][lane & 7] = e8m0_value(kb);
          s.expo[in][lane & 7] = (float)with;
          s.back[in][lane & 7] = back_of(with, expo);
          s.ve[in][lane & 7] = !there ? kNoBlock : vb == 255 ? kNaNExp : e;
          s.page[in][lane & 7] = page;
        }
        if (lane == 0) {
          s.partly[in] = (have >> (8 * i) & 0xffu) != 0xffu;
          s.more[in] = pow2(c - (twin ? old[1] : old[0]));
          s.c[(j0 + i) & 1] = c;
        }
        old[1] = old[0];
        old[0] = c;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.info_full[in]);
      }
    }
   } else if (warp == 21 && steps > 0) {
    // ------------------------------------------------------------------- MMAs
    constexpr uint32_t iqk = idesc_f8(kTile, kTile), ipv = idesc_f16_nt(kTile, D);
    const uint32_t base = smem_u32(raw);
    auto qk = [&](int t, int j) {
      const uint32_t q = base + S::kQ + t * 2 * S::kPart, k = base + S::kK + (j & 1) * S::kPart;
      if (elect_one()) {
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            mma_f8(tmem + t * kTile, desc_rows<D>(q + part * S::kPart + 32 * i),
                   desc_rows<D>(k + 32 * i), iqk, part + i > 0);
        umma_commit(&s.s_full[t]);
      }
      __syncwarp();
    };
    auto pv = [&](int t, int j, bool acc, bool last) {
      const uint32_t v = base + S::kV16 + (j & 1) * 2 * S::kPart;
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i)
          mma_f16_tm(tmem + 2 * kTile + t * D, tmem + t * kTile + 8 * i, desc_values(v + 2048 * i),
                     ipv, acc || i > 0);
        if (last) umma_commit(&s.s_full[t]);
      }
      __syncwarp();
    };
    auto free = [&](uint64_t* bar) {
      if (elect_one()) umma_commit(bar);
      __syncwarp();
    };
    bool ok = wait<true>(s, &s.q_full, 0, p.c.status) && wait(s, &s.k_full[0], 0, p.c.status);
    ok = __all_sync(0xffffffffu, ok);
    if (!twin) {
      if (ok) {
        qk(0, 0);
        qk(1, 0);
        free(&s.k_empty[0]);
      }
      for (int j = 0; ok && j < steps; ++j) {
        ok = wait(s, &s.v16_full[j & 1], (j >> 1) & 1, p.c.status);
        if (ok && j + 1 < steps)
          ok = wait(s, &s.k_full[(j + 1) & 1], ((j + 1) >> 1) & 1, p.c.status);
        for (int t = 0; t < 2; ++t) {
          ok = ok && wait(s, &s.p_full[t], j & 1, p.c.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          pv(t, j, j > 0, j + 1 == steps);
          if (j + 1 < steps) qk(t, j + 1);
        }
        if (!ok) break;
        free(&s.v16_empty[j & 1]);
        if (j + 1 < steps) free(&s.k_empty[(j + 1) & 1]);
      }
    } else {
      // step j is tile j % 2's; its next one is two steps on
      for (int j = 0; ok && j < 2 && j < steps; ++j) {
        ok = wait(s, &s.k_full[j], 0, p.c.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        qk(j, j);
        free(&s.k_empty[j]);
      }
      for (int j = 0; ok && j < steps; ++j) {
        const int t = j & 1;
        ok = wait(s, &s.v16_full[t], (j >> 1) & 1, p.c.status) &&
             wait(s, &s.p_full[t], (j >> 1) & 1, p.c.status);
        if (ok && j + 2 < steps) ok = wait(s, &s.k_full[t], ((j + 2) >> 1) & 1, p.c.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        pv(t, j, j > 1, j + 2 >= steps);
        free(&s.v16_empty[t]);
        if (j + 2 < steps) {
          qk(t, j + 2);
          free(&s.k_empty[t]);
        }
      }
    }
   }
  }

  tc_fence_before();
  __syncthreads();
  if (s.dead && warp == 21) {
    // MMAs still at work end before the tensor memory is given back
    tc_fence_after();
    if (elect_one()) umma_commit(&s.drain);
    __syncwarp();
    mbar_wait_bounded(&s.drain, 0, p.c.status);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const AttnParams& p, cudaStream_t st) {
  const size_t smem = Smem<D>::kEnd + sizeof(Smem<D>);
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(prompt_kernel<D>), allowed);
  if (e != cudaSuccess) return e;
  // at most so many tiles: whole ones, and one more for each sequence that can
  // have more rows than the split kernel takes
  const int64_t rows = p.c.T * p.group;
  const int64_t seqs = rows / (p.few_rows + 1);
  const int64_t some = seqs < p.c.batch ? seqs : p.c.batch;
  int64_t items = (rows / (2 * kTile) + some) * p.c.heads;
  // those that are cut have kPromptItems items at most
  if (p.big_rows) items += some * kPromptItems;
  return launch_pdl(prompt_kernel<D>, dim3((unsigned)items), dim3(kThreads), smem, st, p);
}

template <int D>
cudaError_t launch_join(const AttnParams& p, cudaStream_t st) {
  AttnJoinParams j;
  j.c = p.c;
  j.out = p.out;
  j.next = p.next;
  j.parts = p.big;
  j.part_ml = p.big_ml;
  j.ld_out = p.ld_out;
  j.group = p.group;
  j.few_rows = p.few_rows;
  j.part_rows = p.big_rows;
  j.by_row = p.big_by_row;
  constexpr int PER = kJoinWarps * 128 / D;             // heads to a block at a time
  const int64_t items = p.c.T * ((p.heads_q + PER - 1) / PER), most = 4 * sm_count();
  return launch_pdl(prompt_join_kernel<D>, dim3((unsigned)(items < most ? items : most)),
                    dim3(32 * kJoinWarps), 0, st, j);
}

}  // namespace

cudaError_t launch_attention_prompt(const AttnParams& p, int head_dim, cudaStream_t st) {
  return head_dim == 128 ? launch<128>(p, st) : launch<64>(p, st);
}
cudaError_t launch_attention_prompt_join(const AttnParams& p, int head_dim, cudaStream_t st) {
  return head_dim == 128 ? launch_join<128>(p, st) : launch_join<64>(p, st);
}

}  // namespace ig
