// What the calls of a served layer's attention share: the batch and cache as
// the kernels see them, the head norm's launch parameters, the e4m3 format.
//
// Cache: codes [pages][2][heads][page][D] (e4m3), scales [pages][2][heads]
// [page / 16] (E8M0). Scales are powers of two, so a code times its scale is
// exact in every format with e4m3's three mantissa bits and the range, and the
// kernels may apply a scale to codes, products or sums alike.
#pragma once

#include "mx4.cuh"

namespace ig {

constexpr int kKvBlock = 16;            // tokens that share a scale
constexpr int kKvMinExp = -120;         // least scale that the append writes: 2^-120

// Batch and cache.
struct KvParams {
  uint8_t* codes;
  uint8_t* scales;
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* table;
  uint32_t* status;
  int64_t pages, page_stride, scale_stride, ld_table;
  int64_t T;
  int32_t batch, max_q, heads, page_shift;
};

struct RopeParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* w_q;
  const __nv_bfloat16* w_k;
  const float* cos_sin;
  const int32_t* positions;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;
  uint32_t* status;
  int64_t T, table_rows, ld_q, ld_k, ld_qo, ld_ko;
  int32_t heads_q, heads_k, rot, interleaved, plus_one;
  float eps;
};

struct AppendParams {
  RopeParams r;
  KvParams c;
  const __nv_bfloat16* v;
  int64_t ld_v;
  int32_t nblocks;      // blocks of a sequence that max_q tokens can touch
};

struct GatherParams {
  KvParams c;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  int64_t ld_k, ld_v;
};

struct AttnParams {
  CUtensorMap tm;       // codes as {D, 2 heads page, pages} bytes, box {D, 16, 1}, swizzled by rows
  KvParams c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  uint32_t* next;       // [0] items of the split kernel taken beyond each block's first,
                        // [1] whether the prompt kernel cut a sequence; 0 between calls
  float* parts;         // results of parts [first_tile + tile][kv head][part][row][D]
  float* part_ml;       // [first_tile + tile][kv head][part][row][kPartWords]
  float* big;           // the prompt kernel's parts [first_big + row of an item][D]
  float* big_ml;        // [first_big + row of an item][kPartWords]
  int64_t ld_q, ld_out;
  int32_t big_rows;     // rows of an item of the prompt kernel's parts at most; 0: no parts
  int32_t big_by_row, tiles_by_row;     // see first_big, first_tile
  int32_t heads_q, group;   // query heads, and of one kv head
  uint32_t group_inv;   // 65536 / group, rounded up: row / group for few rows
  uint32_t group_magic, heads_magic;    // see divide
  float group_rcp;      // 1 / group
  int32_t few_rows;     // sequences with at most this many rows a kv head are the split kernel's
  int32_t max_tiles;    // 16-row tiles of such a sequence
  int32_t max_parts, part_rows;
  int32_t flags;
  int32_t after_prompt; // the split kernel runs beside the prompt kernel and ends behind it
  float scale_log2;     // scale * log2(e)
};

struct AttnJoinParams {
  KvParams c;
  __nv_bfloat16* out;
  uint32_t* next;
  const float* parts;
  const float* part_ml;
  int64_t ld_out;
  int32_t group, few_rows, tokens, max_tiles, max_parts, part_rows, by_row;
};

cudaError_t launch_qk_norm_rope(const RopeParams& p, int head_dim, cudaStream_t st);
cudaError_t launch_kv_append(const AppendParams& p, int head_dim, cudaStream_t st);
cudaError_t launch_kv_gather(const GatherParams& p, int head_dim, cudaStream_t st);
// Attention, in this order: the prompt kernel (where a sequence can have many rows), the
// split kernel, the prompt kernel's join (where it can cut a sequence), the split
// kernel's. The first lets the second start with its own last blocks; the second does
// not end before the first has; the joins wait for what is before them.
cudaError_t launch_attention_prompt(const AttnParams& p, int head_dim, cudaStream_t st);
cudaError_t launch_attention_split(const AttnParams& p, int head_dim, cudaStream_t st);
cudaError_t launch_attention_prompt_join(const AttnParams& p, int head_dim, cudaStream_t st);
cudaError_t launch_attention_join(const AttnParams& p, int head_dim, cudaStream_t st);

// {D, rows of a page, pages} of codes; box {D, 16, 1}, rows of 128 or 64 bytes
// swizzled by as much. IG_OK or IG_ERR_CUDA.
int encode_map_codes(CUtensorMap* map, const void* base, int head_dim, uint64_t rows,
                     uint64_t pages, uint64_t page_stride);

// Sequences of at most this many rows a kv head are the split kernel's, the
// others the prompt kernel's. (64 sequences of up to 8192 tokens, 64 query and 8 kv heads
// of 128: 32 rows 306 us by the one, 399 by the other, 64 rows 575 and 468; 64 rows of
// one sequence of 40000 89 and 44, of four of up to 1000 with 32 query heads 22 and 24, of
// one of 60000 with 8 query and 2 kv heads of 64 32 and 47. Fewer rows stay with the split
// kernel all the more: 20 over 500 tokens 13 and 21. The number of rows alone is not the
// best rule at the border: with 8 kv heads and long contexts 64 rows are slower by it.)
constexpr int kFewRows = 64;

// --- splitting a sequence ---------------------------------------------------
// A sequence's tokens are cut into parts of a length that kv_len alone fixes
// (so that a row's bits do not depend on the batch): 256 up to 4096 tokens, then
// whole 512s, at most 64 of them.
constexpr int kMaxSplits = 64;
constexpr int kPartWords = 4;           // of a row of a part: m, l, c (below), unused
__host__ __device__ inline int split_tokens(int kv) {
  return kv <= 4096 ? 256 : 512 * ((kv + 512 * kMaxSplits - 1) / (512 * kMaxSplits));
}

// The prompt kernel cuts a sequence's tokens too where its rows are few blocks' work
// (256 rows of a kv head each): into up to 16 parts, so many that blocks times parts
// fill a GPU's 152 SMs once at most, of six steps of 128 tokens at least. Again
// nothing but the sequence's own sizes decides. (A block costs 23000 clocks beside its
// steps of 3500. Parts of 3, 5, 8 and 12 steps at least, 32 query and 8 kv heads of 128:
// one sequence, 200 tokens over 2000 33, 35, 39, 44 us; 16 of up to 200 over up to
// 3000 199, 168, 141, 122 us.)
constexpr int kPromptRows = 256;
constexpr int kPromptStep = 128;
constexpr int kPromptItems = 152;       // of a sequence that is cut
constexpr int kPromptParts = 16;
__host__ __device__ inline int prompt_parts(int64_t rows, int kv, int heads) {
  const int64_t blocks = (rows + kPromptRows - 1) / kPromptRows * heads;
  if (blocks > kPromptItems / 2) return 1;
  int parts = kPromptItems / (int)blocks;
  const int steps = (kv + kPromptStep - 1) / kPromptStep;
  if (parts > steps / 6) parts = steps / 6;
  if (parts > kPromptParts) parts = kPromptParts;
  return parts < 1 ? 1 : parts;
}
// Where a sequence's parts are in the workspace: its first tile of the split kernel's,
// and its first row of the prompt kernel's (kPromptItems items at most, of item_rows rows
// each). By its number, or by where its rows begin where the rows of all sequences are too
// few for every one to have the most.
__host__ __device__ inline int64_t first_tile(bool by_row, int b, int64_t row0, int group,
                                              int max_tiles) {
  return by_row ? b + row0 * group / 16 : (int64_t)b * max_tiles;
}
__host__ __device__ inline int64_t first_big(bool by_row, int b, int64_t row0, int group,
                                             int big_rows) {
  return (by_row ? row0 * group : (int64_t)b * big_rows) * kPromptItems;
}
__host__ __device__ inline int item_rows(int rows) { return rows < kPromptRows ? rows : kPromptRows; }
// Steps to a part.
__host__ __device__ inline int prompt_len(int kv, int parts) {
  return ((kv + kPromptStep - 1) / kPromptStep + parts - 1) / parts;
}
// Parts that a tile sees whose last row sees token `high`.
__host__ __device__ inline int prompt_seen(int high, int len) {
  return high < 0 || len < 1 ? 1 : high / kPromptStep / len + 1;
}

// --- a row's sums -------------------------------------------------------------
// Of a token, t is the logit in base 2 and e the exponent of its value's scale. Its weight
// in the product with the values' codes is p = 2^(t + e - m + 8), m a whole number that the
// row's largest t + e passes by 7 at most: FP16 has 11 bits of it down to 2^-14, so that
// tokens lose bits against the row's own largest weight times scale, and against nothing
// that the row does not see. The products sum to 2^(8 - m) sum 2^t v, and
// l = sum p 2^(c - e) = 2^(8 - m + c) sum 2^t, so the result is their quotient times 2^c.
// Powers of two round nothing, and c is a matter of FP32's range alone: with -40 up to
// scales of 2^63, then 40, l is at least 2^-96 and at most 2^111 for each token where
// scales are no more than 2^kSpread apart (a smaller one counts as 2^-kSpread of the
// largest so far, or p could be 0 of a token that has its part in l).
constexpr int kSpread = 120;
__host__ __device__ constexpr int c_of(int largest_e) { return largest_e < 64 ? -40 : 40; }

// For divide(): (2^32 - 1) / d.
inline uint32_t magic_of(int d) { return 0xffffffffu / (uint32_t)d; }

#ifdef __CUDACC__
// v / d and, in v, the rest; with magic = (2^32 - 1) / d rounded down the product is two
// below the quotient at most.
__device__ __forceinline__ uint32_t divide(uint32_t& v, uint32_t d, uint32_t magic) {
  uint32_t q = __umulhi(v, magic);
  v -= q * d;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (v >= d) {
      v -= d;
      ++q;
    }
  return q;
}
// New tokens of sequence b: rows row0 .. row0 + n - 1, the last of kv tokens.
// False (and the status word says so) where they are out of range.
__device__ __forceinline__ bool sequence_of(const KvParams& c, int b, int& row0, int& n, int& kv) {
  row0 = __ldg(c.cu + b);
  n = __ldg(c.cu + b + 1) - row0;
  kv = __ldg(c.kv_len + b);
  return row0 >= 0 && n >= 0 && n <= c.max_q && (int64_t)row0 + n <= c.T && kv >= 0 &&
         (int64_t)kv <= (c.ld_table << c.page_shift);
}

// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}
// 2^e for e from -126 to 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// 2^(c - e) for a value scale's exponent e, E the largest so far
__device__ __forceinline__ float back_of(int e, int E) { return pow2(c_of(E) - e); }

// Two e4m3 codes (the low one in bits 0-7) -> two FP16 values, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
// Two FP32 values -> two e4m3 codes, to nearest, ties to even; NaN is NaN.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t v) {
  float lo, hi;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi) : "r"(v));
  return make_float2(lo, hi);
}
// Pairs of FP32 values: one instruction for both.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split2(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Eight values of eight codes.
__device__ __forceinline__ void e4m3_decode8(uint2 c, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? c.x : c.y;
    const float2 t = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(i & 1 ? w >> 16 : w & 0xffffu)));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ uint2 e4m3_encode8(const float (&f)[8]) {
  return make_uint2(f32x2_to_e4m3x2(f[0], f[1]) | f32x2_to_e4m3x2(f[2], f[3]) << 16,
                    f32x2_to_e4m3x2(f[4], f[5]) | f32x2_to_e4m3x2(f[6], f[7]) << 16);
}
#endif  // __CUDACC__

}  // namespace ig
