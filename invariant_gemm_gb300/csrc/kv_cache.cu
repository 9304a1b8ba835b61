// Head norms with the position rotation, and the 8-bit paged cache: append and
// read back.
//
// A head of D values is held by D / 8 lanes, two groups of 4 values each, so that
// both values of a rotated pair are in one lane: with halves as pairs a group of
// the first half and its partner, with neighbours as pairs 8 values in a row. 64-bit
// loads and stores, a butterfly over D / 8 lanes for the norm, nothing else between
// lanes. Arithmetic goes by pairs of FP32 values: with single ones and the weights apart
// from the rotation the instructions bound all three (8192 tokens of 64 + 8 heads of 128
// in 64.9 us at 73 % of the issue slots, now 54.1 us at 61 %: 5.7 TB/s, and HBM).
#include "attention.cuh"

namespace ig {

namespace {

// Where lane l of a head has its groups: values a .. a + 3 and b .. b + 3, and the
// first of the four pairs that they are (-1: not rotated).
struct Place {
  int a, b, pair;
};

template <bool INTER>
__device__ __forceinline__ Place place_of(const RopeParams& p, int l) {
  const int turning = p.rot >> 3;                     // lanes with rotated values
  if (INTER || l >= turning) return {8 * l, 8 * l + 4, l < turning ? 4 * l : -1};
  return {4 * l, (p.rot >> 1) + 4 * l, 4 * l};
}

// A lane's eight values as pairs: x[0], x[1] the first group, x[2], x[3] the second.
struct Values {
  uint64_t x[4];
};

__device__ __forceinline__ uint64_t bf16x2_to_pair(uint32_t u) {
  return pair2(bf16lo(u), bf16hi(u));
}
__device__ __forceinline__ Values unpack(uint2 a, uint2 b) {
  return {{bf16x2_to_pair(a.x), bf16x2_to_pair(a.y), bf16x2_to_pair(b.x), bf16x2_to_pair(b.y)}};
}
__device__ __forceinline__ uint32_t pair_to_bf16x2(uint64_t v) {
  const float2 f = split2(v);
  return f32x2_to_bf16x2_bits(f.x, f.y);
}

// What a head's norm weights w and its token's rotation do to a lane's values:
// y[i] = x[i] same[i] + partner(x)[i] other[i], with 1 / rms left to multiply. The
// products of w with cosines and sines are made once for all heads of a token.
struct Turn {
  uint64_t same[4], other[4];
};

// The value that turns with each: of the other group, or the neighbour.
template <bool INTER>
__device__ __forceinline__ uint64_t partner(const Values& v, int i) {
  if (!INTER) return v.x[i ^ 2];
  const float2 f = split2(v.x[i]);
  return pair2(f.y, f.x);
}

// Weights of the lane's values, 1 where there are none.
__device__ __forceinline__ Values load_weight(const RopeParams& p, const __nv_bfloat16* w,
                                              const Place& at) {
  const uint64_t one = pair2(1.0f, 1.0f);
  if (!w) return {{one, one, one, one}};
  Values v = unpack(__ldg(reinterpret_cast<const uint2*>(w + at.a)),
                    __ldg(reinterpret_cast<const uint2*>(w + at.b)));
  if (p.plus_one) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v.x[i] = add2(v.x[i], one);
  }
  return v;
}

// Row `pos` of the table, with the weights; where the lane's values are not rotated
// (`other` is not looked at) the weights alone.
template <bool INTER>
__device__ __forceinline__ Turn turn_of(const RopeParams& p, const Values& w, const Place& at,
                                        bool turned, int64_t pos) {
  Turn t = {};
  if (!turned) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t.same[i] = w.x[i];
    return t;
  }
  const float* row = p.cos_sin + pos * p.rot;
  const float4 c = __ldg(reinterpret_cast<const float4*>(row + at.pair));
  const float4 s = __ldg(reinterpret_cast<const float4*>(row + (p.rot >> 1) + at.pair));
  if (INTER) {
    const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.same[i] = mul2(w.x[i], pair2(cs[i], cs[i]));
      t.other[i] = mul2(partner<true>(w, i), pair2(-sn[i], sn[i]));
    }
  } else {
    const uint64_t cs[2] = {pair2(c.x, c.y), pair2(c.z, c.w)};
    const uint64_t sn[2] = {pair2(s.x, s.y), pair2(s.z, s.w)};
    const uint64_t neg[2] = {pair2(-s.x, -s.y), pair2(-s.z, -s.w)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.same[i] = mul2(w.x[i], cs[i & 1]);
      t.other[i] = mul2(w.x[i ^ 2], i < 2 ? neg[i] : sn[i & 1]);
    }
  }
  return t;
}

// Norm (where there is one) and rotation of the head that D / 8 lanes hold. Every
// lane of the warp takes part.
template <int D, bool INTER>
__device__ __forceinline__ Values norm_rotate(const RopeParams& p, bool norm, bool turned,
                                              const Turn& t, const Values& v) {
  constexpr int L = D / 8;
  Values y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y.x[i] = mul2(v.x[i], t.same[i]);
  if (turned) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y.x[i] = fma2(partner<INTER>(v, i), t.other[i], y.x[i]);
  }
  if (norm) {
    uint64_t sq = mul2(v.x[0], v.x[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) sq = fma2(v.x[i], v.x[i], sq);
    const float2 both = split2(sq);
    float ss = both.x + both.y;
#pragma unroll
    for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = rsqrtf(fmaf(ss, 1.0f / D, p.eps));
#pragma unroll
    for (int i = 0; i < 4; ++i) y.x[i] = mul2(y.x[i], pair2(inv, inv));
  }
  return y;
}

// Position of a token; false where the table does not have it.
__device__ __forceinline__ bool in_table(const RopeParams& p, int64_t pos) {
  const bool ok = pos >= 0 && pos < p.table_rows;
  if (!ok) atomicOr(p.status, kStatusIndexRange);
  return ok;
}

// Warps that the heads of a token take: those of q and of k have their own, so that
// a warp has one pointer and one set of weights.
template <int PER>
__host__ __device__ __forceinline__ uint32_t chunks_of(const RopeParams& p) {
  return (uint32_t)((p.heads_q + PER - 1) / PER + (p.heads_k + PER - 1) / PER);
}

// PASSES * (256 / D) heads of token t, the chunk's, of q or k into q_out or k_out by
// one warp; pos(): the token's position, asked for where there is a rotation, behind
// the loads of the heads.
template <int D, bool INTER, int PASSES, typename Pos>
__device__ __forceinline__ void heads_of_token(const RopeParams& p, int64_t t, int chunk, Pos pos) {
  constexpr int L = D / 8, PER = 32 / L;
  const int lane = threadIdx.x & 31, l = lane % L;
  const Place at = place_of<INTER>(p, l);
  const int chunks_q = (p.heads_q + PASSES * PER - 1) / (PASSES * PER);
  const bool is_q = chunk < chunks_q;
  const int first = (is_q ? chunk : chunk - chunks_q) * (PASSES * PER) + lane / L;
  const int heads = is_q ? p.heads_q : p.heads_k;
  const __nv_bfloat16* x = (is_q ? p.q + t * p.ld_q : p.k + t * p.ld_k) + first * D;
  __nv_bfloat16* y = (is_q ? p.q_out + t * p.ld_qo : p.k_out + t * p.ld_ko) + first * D;
  const __nv_bfloat16* weight = is_q ? p.w_q : p.w_k;
  uint2 raw[PASSES][2];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    raw[i][0] = raw[i][1] = make_uint2(0, 0);
    if (first + i * PER < heads) {
      raw[i][0] = *reinterpret_cast<const uint2*>(x + i * PER * D + at.a);
      raw[i][1] = *reinterpret_cast<const uint2*>(x + i * PER * D + at.b);
    }
  }
  const Values w = load_weight(p, weight, at);
  const int64_t row = p.cos_sin ? pos() : 0;
  const bool bad = p.cos_sin && !in_table(p, row), turned = p.cos_sin && !bad && at.pair >= 0;
  const Turn turn = turn_of<INTER>(p, w, at, turned, row);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const Values v = norm_rotate<D, INTER>(p, weight != nullptr, turned, turn,
                                           unpack(raw[i][0], raw[i][1]));
    uint2 o0 = make_uint2(pair_to_bf16x2(v.x[0]), pair_to_bf16x2(v.x[1]));
    uint2 o1 = make_uint2(pair_to_bf16x2(v.x[2]), pair_to_bf16x2(v.x[3]));
    if (bad) o0 = o1 = make_uint2(0x7fff7fffu, 0x7fff7fffu);
    if (first + i * PER < heads) {
      *reinterpret_cast<uint2*>(y + i * PER * D + at.a) = o0;
      *reinterpret_cast<uint2*>(y + i * PER * D + at.b) = o1;
    }
  }
}

constexpr int kWarps = 4;               // of a block of these kernels

template <int D, bool INTER, int PASSES>
__global__ void __launch_bounds__(32 * kWarps) qk_kernel(RopeParams p) {
  // (below 2^32: at most half as many as there are heads of tokens, and one a token)
  const uint32_t chunks = chunks_of<PASSES * 256 / D>(p);
  uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int chunk = (int)next_digit(item, chunks);
  griddep_wait();
  if (item >= p.T) return;
  heads_of_token<D, INTER, PASSES>(p, item, chunk,
                                   [&] { return (int64_t)__ldg(p.positions + item); });
}

// A key is off by a few units of the last place that FP32 has for the larger of it and the
// value that it is rotated with, and where it lies as near to the middle between two codes
// it would be rounded to the farther one: 1.2 of a million keys were. Those within 2^-20 of
// that larger one are worked out again in FP64 (4 us of 97, append and read-back of
// five prompts of up to 3001 tokens): 0.04 of a million are left.
//
// Whether a value in steps of the scale is that near: the middles of codes of 3 mantissa
// bits have the top one of the 20 bits below. (Under 2^-6 they lie elsewhere; there a code's
// step is 2^-17 of the largest code and its choice of no weight. The scale is by the
// largest key as FP32 has it.)
__device__ __forceinline__ bool near_middle(float x, float other) {
  const float middle = __uint_as_float((__float_as_uint(x) & 0xfff00000u) | 0x80000u);
  return fabsf(x - middle) <= fmaxf(fabsf(x), fabsf(other)) * 0x1p-20f;
}

// Keys as norm_rotate has them, from FP64, times 2^-e; rounded to FP32 towards 0, with
// the last bit set where that left anything, so that the next rounding is the only one.
template <int D, bool INTER>
__device__ __noinline__ Values keys_again(const RopeParams& p, Place at, uint2 a, uint2 b,
                                          bool turned, int64_t row, int e) {
  constexpr int L = D / 8;
  const uint32_t in[4] = {a.x, a.y, b.x, b.y};
  double x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (double)(i & 1 ? bf16hi(in[i >> 1]) : bf16lo(in[i >> 1]));
  double scale = __longlong_as_double((long long)(1023 - e) << 52);
  if (p.w_k) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
    for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    scale *= rsqrt(ss / D + (double)p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = __bfloat162float(p.w_k[(i < 4 ? at.a : at.b - 4) + i]);
      x[i] *= (double)w + (p.plus_one ? 1.0 : 0.0);
    }
  }
  if (turned) {
    const float* angles = p.cos_sin + row * p.rot + at.pair;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int one = INTER ? 2 * i : i, two = INTER ? 2 * i + 1 : i + 4;
      const double c = angles[i], n = angles[(p.rot >> 1) + i], x1 = x[one], x2 = x[two];
      x[one] = x1 * c - x2 * n;
      x[two] = x2 * c + x1 * n;
    }
  }
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double v = x[i] * scale;
    f[i] = __double2float_rz(v);
    if ((double)f[i] != v) f[i] = __uint_as_float(__float_as_uint(f[i]) | 1u);
  }
  return {{pair2(f[0], f[1]), pair2(f[2], f[3]), pair2(f[4], f[5]), pair2(f[6], f[7])}};
}

// One block of 16 tokens of one head and side, by W warps (of one thread block where
// they are four) that take its new tokens in turn, PASSES times 256 / D at most each.
template <int D, bool INTER, int W>
__device__ __forceinline__ void append_block(const AppendParams& p, int b, int blk, int h,
                                             int side, float* tops) {
  constexpr int L = D / 8, PER = 32 / L, PASSES = W == 1 ? 1 : kKvBlock / (W * PER);
  const int lane = threadIdx.x & 31, l = lane % L, warp = W == 1 ? 0 : threadIdx.x >> 5;
  const KvParams& c = p.c;
  int row0, n, kv;
  if (!sequence_of(c, b, row0, n, kv)) {
    if (blk == 0 && h == 0 && side == 0 && lane == 0) atomicOr(c.status, kStatusIndexRange);
    return;
  }
  // more new tokens than the sequence has in all: those before its first are
  // not in it
  const int first = kv - n;
  blk += max(first, 0) / kKvBlock;
  if (n == 0 || kv == 0 || blk > (kv - 1) / kKvBlock) return;
  // (kv may be close to 2^31, so what is behind the block's last token is not counted up to:
  // places from here on are the block's, 0 to 15)
  const int start = blk * kKvBlock;
  const int32_t page = __ldg(c.table + (int64_t)b * c.ld_table + (start >> c.page_shift));
  // the new tokens of this warp: begin + PER i, of those before end
  const int begin = max(first - start, 0) + warp * PASSES * PER + lane / L;
  const int end = min(kKvBlock, kv - start);
  const int row_at = row0 + (start - first);        // row of place 0
  const Place at = place_of<INTER>(p.r, l);
  const __nv_bfloat16* src = (side ? p.v : p.r.k) + (int64_t)h * D;
  const int64_t ld = side ? p.ld_v : p.r.ld_k;
  uint2 raw[PASSES][2];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int pos = begin + i * PER;
    raw[i][0] = raw[i][1] = make_uint2(0, 0);
    if (pos < end) {
      const int64_t t = row_at + pos;
      raw[i][0] = *reinterpret_cast<const uint2*>(src + t * ld + at.a);
      raw[i][1] = *reinterpret_cast<const uint2*>(src + t * ld + at.b);
    }
  }
  const bool there = page >= 0 && page < c.pages;
  const int in_page = start & ((1 << c.page_shift) - 1);
  const int64_t head = (((int64_t)side * c.heads + h) << c.page_shift) + in_page;
  uint8_t* rows = c.codes + page * c.page_stride + head * D;
  uint8_t* scale = c.scales + page * c.scale_stride + head / kKvBlock;
  const bool older = start < first;
  const int was = older && there ? *scale : 0;
  Values f[PASSES];
  float top = 0.0f;                     // largest magnitude, infinity among them, NaN not
  if (side == 0) {
    const Values w = load_weight(p.r, p.r.w_k, at);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int pos = begin + i * PER;
      bool bad = false;
      int64_t row = (int64_t)start + pos;
      if (p.r.cos_sin && pos < end) {
        if (p.r.positions) row = __ldg(p.r.positions + row_at + pos);
        bad = !in_table(p.r, row);
      }
      const bool turned = p.r.cos_sin && pos < end && !bad && at.pair >= 0;
      f[i] = norm_rotate<D, INTER>(p.r, p.r.w_k != nullptr, turned,
                                   turn_of<INTER>(p.r, w, at, turned, row),
                                   unpack(raw[i][0], raw[i][1]));
      if (bad) {
        const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i].x[j] = pair2(nan, nan);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) f[i] = unpack(raw[i][0], raw[i][1]);
  }
  auto largest = [&] {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = split2(f[i].x[j]);
        m = fmaxf(m, fmaxf(fabsf(x.x), fabsf(x.y)));
      }
    // (no value is negative, so whole numbers compare as they do)
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    if constexpr (W > 1) {
      if (lane == 0) tops[warp] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < W; ++i) m = fmaxf(m, tops[i]);
    }
    return m;
  };
  top = largest();
  if (top == __uint_as_float(0x7f800000u)) {
    // what is not finite is held as NaN, and has no say in the scale
    if constexpr (W > 1) __syncthreads();       // the warps' maxima are read
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 x = split2(f[i].x[j]);
        if (fabsf(x.x) == top) x.x = __uint_as_float(0x7fc00000u);
        if (fabsf(x.y) == top) x.y = __uint_as_float(0x7fc00000u);
        f[i].x[j] = pair2(x.x, x.y);
      }
    top = largest();
  }
  if (!there) {
    if (lane == 0) atomicOr(c.status, kStatusIndexRange);
    return;
  }
  // top = m 2^x, m in [1/2, 1): within 448 2^e = 7/8 2^(e + 9)
  const uint32_t bits = __float_as_uint(top);
  const int e = max((int)(bits >> 23) - 126 - 9 + ((bits & 0x7fffffu) > 0x600000u), kKvMinExp);
  const int byte = older ? max(e + 127, was) : e + 127;
  const float down = byte == 255 ? __uint_as_float(0x7fc00000u) : e8m0_value(254 - byte);
  const bool inexact = side == 0 && (p.r.w_k || p.r.cos_sin);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int pos = begin + i * PER;
    Values g;
#pragma unroll
    for (int j = 0; j < 4; ++j) g.x[j] = mul2(f[i].x[j], pair2(down, down));
    if (inexact) {
      uint32_t which = 0;               // of the eight
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = split2(g.x[j]), y = split2(partner<INTER>(g, j));
        which |= (near_middle(x.x, y.x) ? 1u : 0u) << 2 * j | (near_middle(x.y, y.y) ? 2u : 0u) << 2 * j;
      }
      if (__any_sync(0xffffffffu, which && pos < end)) {
        int64_t row = (int64_t)start + pos;
        uint2 a = make_uint2(0, 0), b = a;
        if (pos < end) {
          const int64_t t = row_at + pos;
          a = *reinterpret_cast<const uint2*>(src + t * ld + at.a);
          b = *reinterpret_cast<const uint2*>(src + t * ld + at.b);
          if (p.r.positions) row = __ldg(p.r.positions + t);
        }
        const bool turned = p.r.cos_sin && pos < end && at.pair >= 0 && row >= 0 &&
                            row < p.r.table_rows;
        const Values again = keys_again<D, INTER>(p.r, at, a, b, turned, row, byte - 127);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = split2(g.x[j]), y = split2(again.x[j]);
          g.x[j] = pair2(which >> 2 * j & 1 ? y.x : x.x, which >> 2 * j & 2 ? y.y : x.y);
        }
      }
    }
    if (pos >= end) continue;
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = split2(g.x[j]);
      q[j] = f32x2_to_e4m3x2(x.x, x.y);
    }
    *reinterpret_cast<uint32_t*>(rows + pos * D + at.a) = q[0] | q[1] << 16;
    *reinterpret_cast<uint32_t*>(rows + pos * D + at.b) = q[2] | q[3] << 16;
  }
  if (warp != 0) return;
  __syncwarp();                         // every lane has read the scale that was
  if (older && byte > was && byte < 255) {
    // the older tokens by the grown scale
    const float less = pow2(max(was - byte, -126));
    for (int i = lane; i < (first - start) * L; i += 32) {
      uint2* code = reinterpret_cast<uint2*>(rows) + i;
      float g[8];
      e4m3_decode8(*code, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] *= less;
      *code = e4m3_encode8(g);
    }
  }
  if (lane == 0) *scale = (uint8_t)byte;
}

// The sequence of row r: the last one that starts at or before it. 32 places a
// step.
__device__ __forceinline__ int sequence_at(const int32_t* cu, int batch, int64_t r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = batch;                       // cu[lo] <= r, the answer below hi
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool below = lane == 0 || (at < hi && __ldg(cu + at) <= r);
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, below));
    lo += last * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The blocks of k and v, behind them q: kv_blocks thread blocks and the others.
template <int D, bool INTER, int PASSES, int W>
__global__ void __launch_bounds__(32 * kWarps, 9) append_kernel(const AppendParams p,
                                                             unsigned kv_blocks) {
  constexpr int PER = PASSES * 256 / D;
  __shared__ float tops[kWarps];
  griddep_wait();
  if (blockIdx.x < kv_blocks) {
    uint32_t item = W == 1 ? blockIdx.x * kWarps + (threadIdx.x >> 5) : blockIdx.x;
    const int side = (int)next_digit(item, 2);
    const int h = (int)next_digit(item, p.c.heads);
    const int blk = (int)next_digit(item, p.nblocks);
    if ((int)item < p.c.batch) append_block<D, INTER, W>(p, (int)item, blk, h, side, tops);
    return;
  }
  uint32_t t = (blockIdx.x - kv_blocks) * kWarps + (threadIdx.x >> 5);
  const int chunk = (int)next_digit(t, chunks_of<PER>(p.r));
  if (t >= p.r.T) return;
  const int b = sequence_at(p.c.cu, p.c.batch, t);
  int row0, n, kv;
  if (!sequence_of(p.c, b, row0, n, kv) || (int)t < row0 || (int)t >= row0 + n) return;
  heads_of_token<D, INTER, PASSES>(p.r, t, chunk, [&] {
    return p.r.positions ? (int64_t)__ldg(p.r.positions + t) : (int64_t)kv - n + ((int)t - row0);
  });
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) gather_kernel(const GatherParams p) {
  constexpr int L = D / 16;                     // lanes to a head, 16 codes each
  const KvParams& c = p.c;
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  griddep_wait();
  if (r >= c.T) return;
  const int b = sequence_at(c.cu, c.batch, r);
  int row0, n, kv;
  const bool ok = sequence_of(c, b, row0, n, kv);
  if (!ok) {
    if (lane == 0) atomicOr(c.status, kStatusIndexRange);
    return;
  }
  if (r < row0 || r >= row0 + n) return;        // a row of no sequence
  const int64_t pos = kv - n + (r - row0);
  int32_t page = 0;
  bool absent = false;
  if (pos >= 0) {
    page = __ldg(c.table + (int64_t)b * c.ld_table + (pos >> c.page_shift));
    absent = page < 0 || page >= c.pages;
    if (absent && lane == 0) atomicOr(c.status, kStatusIndexRange);
  }
  const bool read = pos >= 0 && !absent;
  const int in_page = (int)(pos & ((1 << c.page_shift) - 1));
  // four vectors a lane at a time, all asked for before the first is used
  for (int i0 = lane; i0 < 2 * c.heads * L; i0 += 128) {
    uint4 raw[4];
    uint32_t byte[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + 32 * k;
      raw[k] = make_uint4(0, 0, 0, 0);
      byte[k] = 0;
      if (read && i < 2 * c.heads * L) {
        const int64_t row = ((int64_t)(i / L) << c.page_shift) + in_page;
        raw[k] = ldg_cg_v4(reinterpret_cast<const uint4*>(c.codes + page * c.page_stride + row * D) +
                           i % L);
        byte[k] = __ldg(c.scales + page * c.scale_stride + row / kKvBlock);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + 32 * k;
      if (i >= 2 * c.heads * L) break;
      const float scale = read ? e8m0_value(byte[k]) : absent ? __uint_as_float(0x7fc00000u) : 0.0f;
      const int64_t head = i / L;
      const bool is_v = head >= c.heads;
      __nv_bfloat16* out = is_v ? p.v_out + r * p.ld_v + (head - c.heads) * D
                                : p.k_out + r * p.ld_k + head * D;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float f[8];
        e4m3_decode8(j ? make_uint2(raw[k].z, raw[k].w) : make_uint2(raw[k].x, raw[k].y), f);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] *= scale;
        *(reinterpret_cast<uint4*>(out) + 2 * (i % L) + j) =
            make_uint4(f32x2_to_bf16x2_bits(f[0], f[1]), f32x2_to_bf16x2_bits(f[2], f[3]),
                       f32x2_to_bf16x2_bits(f[4], f[5]), f32x2_to_bf16x2_bits(f[6], f[7]));
      }
    }
  }
}

unsigned blocks_of(int64_t warps) { return (unsigned)((warps + kWarps - 1) / kWarps); }

// Passes: a warp takes four passes of heads of a token with one look at its angles
// where that leaves 16 warps to an SM at least, one pass where the call is smaller (a
// token of 40 heads of 128: 20 warps instead of 5). The bits are the same.
template <int D>
cudaError_t qk(const RopeParams& p, cudaStream_t st) {
  constexpr int PER = 256 / D;
  const int heads = p.heads_q + p.heads_k;
  const bool many = p.T * ((heads + PER - 1) / PER) > 64 * (int64_t)sm_count();
  auto go = [&](auto kern, int passes) {
    const int per = passes * PER;
    const int64_t chunks = (p.heads_q + per - 1) / per + (p.heads_k + per - 1) / per;
    return launch_pdl(kern, dim3(blocks_of(p.T * chunks)), dim3(32 * kWarps), 0, st, p);
  };
  if (p.interleaved) return many ? go(qk_kernel<D, true, 4>, 4) : go(qk_kernel<D, true, 1>, 1);
  return many ? go(qk_kernel<D, false, 4>, 4) : go(qk_kernel<D, false, 1>, 1);
}

template <int D, bool INTER, int PASSES, int W>
cudaError_t append_launch(const AppendParams& p, cudaStream_t st) {
  constexpr int PER = PASSES * 256 / D;
  const int64_t kv_items = 2ll * p.c.heads * p.nblocks * p.c.batch;
  const int64_t q_items = p.r.q ? p.r.T * ((p.r.heads_q + PER - 1) / PER) : 0;
  const unsigned kv_blocks = W == 1 ? blocks_of(kv_items) : (unsigned)kv_items;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kv_blocks + blocks_of(q_items));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_kernel<D, INTER, PASSES, W>, p, kv_blocks);
}

// One warp to a block of the cache where no sequence has more new tokens than it holds
// at a time (single tokens: 256 sequences 4096 warps), else four, whose loads are on their
// way together. Five prompts of up to 3001 tokens, 64 + 8 heads of 128: 84 us for 386 MB,
// 4.6 TB/s, issue slots 72 %: instructions bound it and not HBM, for each kv head's
// warps look up a token's angles and multiply them by the weights for themselves. (Nine
// blocks to an SM; with eight 103 us in place of 99, append and read-back.)
template <int D, bool INTER>
cudaError_t append(const AppendParams& p, cudaStream_t st) {
  constexpr int PER = 256 / D;
  const bool many = p.r.T * ((p.r.heads_q + PER - 1) / PER) > 64 * (int64_t)sm_count();
  if (p.c.max_q <= PER)
    return many ? append_launch<D, INTER, 4, 1>(p, st) : append_launch<D, INTER, 1, 1>(p, st);
  return many ? append_launch<D, INTER, 4, kWarps>(p, st) : append_launch<D, INTER, 1, kWarps>(p, st);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, int head_dim, cudaStream_t st) {
  return head_dim == 128 ? qk<128>(p, st) : qk<64>(p, st);
}

cudaError_t launch_kv_append(const AppendParams& p, int head_dim, cudaStream_t st) {
  if (p.r.interleaved) return head_dim == 128 ? append<128, true>(p, st) : append<64, true>(p, st);
  return head_dim == 128 ? append<128, false>(p, st) : append<64, false>(p, st);
}

cudaError_t launch_kv_gather(const GatherParams& p, int head_dim, cudaStream_t st) {
  if (head_dim == 128)
    return launch_pdl(gather_kernel<128>, dim3(blocks_of(p.c.T)), dim3(32 * kWarps), 0, st, p);
  return launch_pdl(gather_kernel<64>, dim3(blocks_of(p.c.T)), dim3(32 * kWarps), 0, st, p);
}

}  // namespace ig
