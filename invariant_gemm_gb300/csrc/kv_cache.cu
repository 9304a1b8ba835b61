// Head norms with the position rotation, and the 8-bit paged cache: append and
// read back.
//
// A head of D values is held by D / 8 lanes, two groups of 4 values each, so that
// both values of a rotated pair are in one lane: with halves as pairs a group of
// the first half and its partner, with neighbours as pairs 8 values in a row. 64-bit
// loads and stores, a butterfly over D / 8 lanes for the norm, nothing else between
// lanes.
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

struct Angles {
  float4 c, s;
};

__device__ __forceinline__ Angles load_angles(const RopeParams& p, int64_t pos, int pair) {
  const float* row = p.cos_sin + pos * p.rot;
  return {__ldg(reinterpret_cast<const float4*>(row + pair)),
          __ldg(reinterpret_cast<const float4*>(row + (p.rot >> 1) + pair))};
}

__device__ __forceinline__ void unpack4(uint2 u, float* f) {
  f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
}
__device__ __forceinline__ uint2 pack4(const float* f) {
  return make_uint2(f32x2_to_bf16x2_bits(f[0], f[1]), f32x2_to_bf16x2_bits(f[2], f[3]));
}

// Norm (the lane's own: w its 8 weights; others of the warp may have one where it
// has none) and rotation of the head that D / 8 lanes hold. Every lane of the warp
// takes part.
template <int D, bool INTER>
__device__ __forceinline__ void norm_rotate(const RopeParams& p, bool any, bool mine,
                                            const float (&w)[8], bool turned, const Angles& t,
                                            float (&f)[8]) {
  constexpr int L = D / 8;
  if (any) {
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      s0 = fmaf(f[i], f[i], s0);
      s1 = fmaf(f[i + 1], f[i + 1], s1);
    }
    float ss = s0 + s1;
#pragma unroll
    for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = mine ? rsqrtf(fmaf(ss, 1.0f / D, p.eps)) : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * w[i];
  }
  if (turned) {
    const float c[4] = {t.c.x, t.c.y, t.c.z, t.c.w}, s[4] = {t.s.x, t.s.y, t.s.z, t.s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int one = INTER ? 2 * i : i, two = INTER ? 2 * i + 1 : i + 4;
      const float x1 = f[one], x2 = f[two];
      f[one] = fmaf(-x2, s[i], x1 * c[i]);
      f[two] = fmaf(x1, s[i], x2 * c[i]);
    }
  }
}

// Weights of the lane's values, 1 where there are none.
__device__ __forceinline__ void load_weight(const RopeParams& p, const __nv_bfloat16* w,
                                            const Place& at, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 1.0f;
  if (!w) return;
  unpack4(__ldg(reinterpret_cast<const uint2*>(w + at.a)), f);
  unpack4(__ldg(reinterpret_cast<const uint2*>(w + at.b)), f + 4);
  if (p.plus_one) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += 1.0f;
  }
}

// Position of a token; false where the table does not have it.
__device__ __forceinline__ bool in_table(const RopeParams& p, int64_t pos) {
  const bool ok = pos >= 0 && pos < p.table_rows;
  if (!ok) atomicOr(p.status, kStatusIndexRange);
  return ok;
}

// Heads first .. first + PASSES * (256 / D) - 1 of token t, of the heads of q
// and then of k, into q_out and k_out by one warp; pos(): the token's position,
// asked for where there is a rotation, behind the loads of the heads.
template <int D, bool INTER, int PASSES, typename Pos>
__device__ __forceinline__ void heads_of_token(const RopeParams& p, int64_t t, int first, Pos pos) {
  constexpr int L = D / 8, PER = 32 / L;
  const int lane = threadIdx.x & 31, l = lane % L;
  const Place at = place_of<INTER>(p, l);
  const int heads = p.heads_q + p.heads_k;
  uint2 raw[PASSES][2];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int h = first + i * PER + lane / L;
    raw[i][0] = raw[i][1] = make_uint2(0, 0);
    if (h < heads) {
      const __nv_bfloat16* x = h < p.heads_q
                                   ? p.q + t * p.ld_q + (int64_t)h * D
                                   : p.k + t * p.ld_k + (int64_t)(h - p.heads_q) * D;
      raw[i][0] = *reinterpret_cast<const uint2*>(x + at.a);
      raw[i][1] = *reinterpret_cast<const uint2*>(x + at.b);
    }
  }
  Angles angles = {};
  bool bad = false, turned = false;
  if (p.cos_sin) {
    const int64_t row = pos();
    bad = !in_table(p, row);
    turned = !bad && at.pair >= 0;
    if (turned) angles = load_angles(p, row, at.pair);
  }
  float wq[8], wk[8];
  load_weight(p, p.w_q, at, wq);
  load_weight(p, p.w_k, at, wk);
  const bool any = p.w_q || p.w_k;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    if (first + i * PER >= heads) break;
    const int h = first + i * PER + lane / L;
    const bool is_q = h < p.heads_q;
    float f[8], w[8];
    unpack4(raw[i][0], f);
    unpack4(raw[i][1], f + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = is_q ? wq[j] : wk[j];
    norm_rotate<D, INTER>(p, any, is_q ? p.w_q != nullptr : p.w_k != nullptr, w, turned, angles, f);
    uint2 o0 = pack4(f), o1 = pack4(f + 4);
    if (bad) o0 = o1 = make_uint2(0x7fff7fffu, 0x7fff7fffu);
    if (h < heads) {
      __nv_bfloat16* y = is_q ? p.q_out + t * p.ld_qo + (int64_t)h * D
                              : p.k_out + t * p.ld_ko + (int64_t)(h - p.heads_q) * D;
      *reinterpret_cast<uint2*>(y + at.a) = o0;
      *reinterpret_cast<uint2*>(y + at.b) = o1;
    }
  }
}

constexpr int kWarps = 4;               // of a block of these kernels

template <int D, bool INTER, int PASSES>
__global__ void __launch_bounds__(32 * kWarps) qk_kernel(RopeParams p) {
  constexpr int PER = PASSES * 256 / D;
  const int chunks = (p.heads_q + p.heads_k + PER - 1) / PER;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = item / chunks;
  griddep_wait();
  if (t >= p.T) return;
  heads_of_token<D, INTER, PASSES>(p, t, (int)(item - t * chunks) * PER,
                                   [&] { return (int64_t)__ldg(p.positions + t); });
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
  const int start = (max(first, 0) / kKvBlock + blk) * kKvBlock;
  if (n == 0 || start >= kv) return;
  const int32_t page = __ldg(c.table + (int64_t)b * c.ld_table + (start >> c.page_shift));
  // the new tokens of this warp: begin + PER i, of those before end
  const int begin = max(start, first) + warp * PASSES * PER + lane / L;
  const int end = min(start + kKvBlock, kv);
  const Place at = place_of<INTER>(p.r, l);
  const __nv_bfloat16* src = (side ? p.v : p.r.k) + (int64_t)h * D;
  const int64_t ld = side ? p.ld_v : p.r.ld_k;
  uint2 raw[PASSES][2];
  Angles angles[PASSES];
  bool bad[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int pos = begin + i * PER;
    raw[i][0] = raw[i][1] = make_uint2(0, 0);
    bad[i] = false;
    if (pos < end) {
      const int64_t t = row0 + pos - first;
      raw[i][0] = *reinterpret_cast<const uint2*>(src + t * ld + at.a);
      raw[i][1] = *reinterpret_cast<const uint2*>(src + t * ld + at.b);
      if (side == 0 && p.r.cos_sin) {
        const int64_t row = p.r.positions ? (int64_t)__ldg(p.r.positions + t) : (int64_t)pos;
        bad[i] = !in_table(p.r, row);
        if (!bad[i] && at.pair >= 0) angles[i] = load_angles(p.r, row, at.pair);
      }
    }
  }
  const bool there = page >= 0 && page < c.pages;
  const int in_page = start & ((1 << c.page_shift) - 1);
  const int64_t head = (((int64_t)side * c.heads + h) << c.page_shift) + in_page;
  uint8_t* rows = c.codes + page * c.page_stride + head * D;
  uint8_t* scale = c.scales + page * c.scale_stride + head / kKvBlock;
  const bool older = start < first;
  const int was = older && there ? *scale : 0;
  float w[8];
  load_weight(p.r, side == 0 ? p.r.w_k : nullptr, at, w);
  const bool norm = side == 0 && p.r.w_k;
  float f[PASSES][8], top = 0.0f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const bool mine = begin + i * PER < end;
    unpack4(raw[i][0], f[i]);
    unpack4(raw[i][1], f[i] + 4);
    norm_rotate<D, INTER>(p.r, norm, norm, w,
                          side == 0 && p.r.cos_sin && mine && !bad[i] && at.pair >= 0, angles[i],
                          f[i]);
    if (mine) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (bad[i]) f[i][j] = __uint_as_float(0x7fc00000u);
        const float m = fabsf(f[i][j]);
        if (m < __uint_as_float(0x7f800000u)) top = fmaxf(top, m);
      }
    }
  }
  // (no value is negative, so whole numbers compare as they do)
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
  if constexpr (W > 1) {
    if (lane == 0) tops[warp] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) top = fmaxf(top, tops[i]);
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
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int pos = begin + i * PER;
    if (pos >= end) continue;
    float g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      g[j] = fabsf(f[i][j]) < __uint_as_float(0x7f800000u) ? f[i][j] * down
                                                          : __uint_as_float(0x7fc00000u);
    const uint2 q = e4m3_encode8(g);
    *reinterpret_cast<uint32_t*>(rows + (pos - start) * D + at.a) = q.x;
    *reinterpret_cast<uint32_t*>(rows + (pos - start) * D + at.b) = q.y;
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
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const AppendParams p,
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
  const int64_t item = (int64_t)(blockIdx.x - kv_blocks) * kWarps + (threadIdx.x >> 5);
  const int chunks = (p.r.heads_q + PER - 1) / PER;
  const int64_t t = item / chunks;
  if (t >= p.r.T) return;
  const int b = sequence_at(p.c.cu, p.c.batch, t);
  int row0, n, kv;
  if (!sequence_of(p.c, b, row0, n, kv) || t < row0 || t >= row0 + n) return;
  heads_of_token<D, INTER, PASSES>(p.r, t, (int)(item - t * chunks) * PER, [&] {
    return p.r.positions ? (int64_t)__ldg(p.r.positions + t) : (int64_t)kv - n + (t - row0);
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
        const uint2 lo = pack4(f), hi = pack4(f + 4);
        *(reinterpret_cast<uint4*>(out) + 2 * (i % L) + j) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  }
}

unsigned blocks_of(int64_t warps) { return (unsigned)((warps + kWarps - 1) / kWarps); }

// Passes: a warp takes several heads of a token with one look at its angles
// where there are many, one pass of them where the call is small.
template <int D>
cudaError_t qk(const RopeParams& p, cudaStream_t st) {
  constexpr int PER = 256 / D;
  const int heads = p.heads_q + p.heads_k;
  const bool many = p.T * ((heads + PER - 1) / PER) > 64 * (int64_t)sm_count();
  auto go = [&](auto kern, int passes) {
    const int per = passes * PER;
    return launch_pdl(kern, dim3(blocks_of(p.T * ((heads + per - 1) / per))), dim3(32 * kWarps), 0,
                      st, p);
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

// One warp a block where no sequence has more new tokens than it holds at a time,
// else four.
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
