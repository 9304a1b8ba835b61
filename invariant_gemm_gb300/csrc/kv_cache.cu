// Head norms with the position rotation, and the 8-bit paged cache: append and
// read back.
//
// A head of D values is held by D / 8 lanes, 8 consecutive values each: 128-bit
// loads and stores, a butterfly over D / 8 lanes for the norm, and the rotation's
// partner value either in the same lane (neighbours as pairs) or, at the same
// place, in one other lane (halves as pairs).
#include "attention.cuh"

namespace ig {

namespace {

// Cosines and sines of one token for the values of this lane: of the pairs that
// the lane holds one value of (halves: 8 of them) or both (neighbours: 4).
struct Angles {
  float c[8], s[8];
};

template <bool INTER>
__device__ __forceinline__ void load_angles(const RopeParams& p, int64_t pos, int l, Angles& a) {
  const int half = p.rot >> 1;
  const float* row = p.cos_sin + pos * p.rot;
  if (INTER) {
    if (8 * l < p.rot) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + 4 * l));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + 4 * l));
      a.c[0] = c.x; a.c[1] = c.y; a.c[2] = c.z; a.c[3] = c.w;
      a.s[0] = s.x; a.s[1] = s.y; a.s[2] = s.z; a.s[3] = s.w;
    }
  } else if (8 * l < p.rot) {
    const int i = 8 * l < half ? 8 * l : 8 * l - half;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + i) + j);
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + i) + j);
      a.c[4 * j] = c.x; a.c[4 * j + 1] = c.y; a.c[4 * j + 2] = c.z; a.c[4 * j + 3] = c.w;
      a.s[4 * j] = s.x; a.s[4 * j + 1] = s.y; a.s[4 * j + 2] = s.z; a.s[4 * j + 3] = s.w;
    }
  }
}

// Norm (w: the lane's 8 weights) and rotation of the head that D / 8 lanes hold,
// lane l of them its values 8 l .. 8 l + 7. Every lane of the warp takes part.
template <int D, bool INTER>
__device__ __forceinline__ void norm_rotate(const RopeParams& p, bool norm, const float (&w)[8],
                                            int l, const Angles& a, float (&f)[8]) {
  constexpr int L = D / 8;
  if (norm) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
    for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = __frsqrt_rn(ss * (1.0f / D) + p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * w[i];
  }
  if (!p.cos_sin) return;
  const bool in = 8 * l < p.rot;
  if (INTER) {
    if (in) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x1 = f[2 * i], x2 = f[2 * i + 1];
        f[2 * i] = fmaf(-x2, a.s[i], x1 * a.c[i]);
        f[2 * i + 1] = fmaf(x1, a.s[i], x2 * a.c[i]);
      }
    }
  } else {
    const int h8 = p.rot >> 4;                          // lanes to a half
    const bool first = l < h8;
    const int lane = threadIdx.x & 31;
    const int from = in ? (first ? lane + h8 : lane - h8) : lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_sync(0xffffffffu, f[i], from);
      if (in) f[i] = fmaf(first ? -other : other, a.s[i], f[i] * a.c[i]);
    }
  }
}

__device__ __forceinline__ void load_weight(const RopeParams& p, const __nv_bfloat16* w, int l,
                                            float (&f)[8]) {
  if (!w) return;
  unpack8(__ldg(reinterpret_cast<const uint4*>(w) + l), f);
  if (p.plus_one) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += 1.0f;
  }
}

__device__ __forceinline__ uint4 pack_bf16(const float (&f)[8]) {
  return make_uint4(f32x2_to_bf16x2_bits(f[0], f[1]), f32x2_to_bf16x2_bits(f[2], f[3]),
                    f32x2_to_bf16x2_bits(f[4], f[5]), f32x2_to_bf16x2_bits(f[6], f[7]));
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
  const int heads = p.heads_q + p.heads_k;
  uint4 raw[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int h = first + i * PER + lane / L;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (h < heads)
      raw[i] = h < p.heads_q
                   ? *(reinterpret_cast<const uint4*>(p.q + t * p.ld_q + (int64_t)h * D) + l)
                   : *(reinterpret_cast<const uint4*>(p.k + t * p.ld_k +
                                                      (int64_t)(h - p.heads_q) * D) + l);
  }
  Angles a = {};
  bool bad = false;
  if (p.cos_sin) {
    const int64_t at = pos();
    bad = !in_table(p, at);
    if (!bad) load_angles<INTER>(p, at, l, a);
  }
  float wq[8] = {}, wk[8] = {};
  load_weight(p, p.w_q, l, wq);
  load_weight(p, p.w_k, l, wk);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int h = first + i * PER + lane / L;
    if (first + i * PER >= heads) break;
    const bool is_q = h < p.heads_q;
    const bool norm = is_q ? p.w_q != nullptr : p.w_k != nullptr;
    float f[8], w[8];
    unpack8(raw[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = norm ? (is_q ? wq[j] : wk[j]) : 1.0f;
    // heads of both sides can share a warp: the norm is run for all if for any
    const bool any = __any_sync(0xffffffffu, norm);
    float g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = f[j];
    if (any) {
      norm_rotate<D, INTER>(p, true, w, l, a, f);
      if (!__all_sync(0xffffffffu, norm)) {
        norm_rotate<D, INTER>(p, false, w, l, a, g);
        if (!norm) {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = g[j];
        }
      }
    } else {
      norm_rotate<D, INTER>(p, false, w, l, a, f);
    }
    uint4 o = pack_bf16(f);
    if (bad) o = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
    if (h < heads) {
      if (is_q)
        *(reinterpret_cast<uint4*>(p.q_out + t * p.ld_qo + (int64_t)h * D) + l) = o;
      else
        *(reinterpret_cast<uint4*>(p.k_out + t * p.ld_ko + (int64_t)(h - p.heads_q) * D) + l) = o;
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

// One block of 16 tokens of one head and side by one warp.
template <int D, bool INTER>
__device__ __forceinline__ void append_block(const AppendParams& p, int b, int blk, int h,
                                             int side) {
  constexpr int L = D / 8, PER = 32 / L, PASSES = kKvBlock / PER;
  const int lane = threadIdx.x & 31, l = lane % L, sub = lane / L;
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
  if (page < 0 || page >= c.pages) {
    if (lane == 0) atomicOr(c.status, kStatusIndexRange);
    return;
  }
  const int in_page = start & ((1 << c.page_shift) - 1);
  const int64_t head = (int64_t)side * c.heads + h;
  uint8_t* rows = c.codes + page * c.page_stride + ((head << c.page_shift) + in_page) * D;
  uint8_t* scale = c.scales + page * c.scale_stride + ((head << c.page_shift) + in_page) / kKvBlock;
  const bool older = start < first;
  const int was = older ? *scale : 0;

  const __nv_bfloat16* src = side ? p.v : p.r.k;
  const int64_t ld = side ? p.ld_v : p.r.ld_k;
  uint4 raw[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int pos = start + i * PER + sub;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (pos >= first && pos < kv)
      raw[i] = *(reinterpret_cast<const uint4*>(src + (int64_t)(row0 + pos - first) * ld +
                                                (int64_t)h * D) + l);
  }
  float f[PASSES][8];
  float w[8] = {};
  if (side == 0) load_weight(p.r, p.r.w_k, l, w);
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int pos = start + i * PER + sub;
    const bool mine = pos >= first && pos < kv;
    unpack8(raw[i], f[i]);
    if (side == 0) {
      Angles a = {};
      bool bad = false;
      if (p.r.cos_sin && mine) {
        const int64_t at =
            p.r.positions ? __ldg(p.r.positions + row0 + pos - first) : (int64_t)pos;
        bad = !in_table(p.r, at);
        if (!bad) load_angles<INTER>(p.r, at, l, a);
      }
      norm_rotate<D, INTER>(p.r, p.r.w_k != nullptr, w, l, a, f[i]);
      if (bad) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = __uint_as_float(0x7fc00000u);
      }
    }
    if (mine) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float m = fabsf(f[i][j]);
        if (m < __uint_as_float(0x7f800000u)) top = fmaxf(top, m);
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  // top = m 2^x, m in [1/2, 1): within 448 2^e = 7/8 2^(e + 9)
  const uint32_t bits = __float_as_uint(top);
  int e = (int)(bits >> 23) - 126 - 9 + ((bits & 0x7fffffu) > 0x600000u);
  e = max(e, kKvMinExp);
  int byte = e + 127;
  if (older) byte = max(byte, was);
  const float down = byte == 255 ? __uint_as_float(0x7fc00000u) : e8m0_value(254 - byte);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int pos = start + i * PER + sub;
    if (pos >= first && pos < kv) {
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        g[j] = fabsf(f[i][j]) < __uint_as_float(0x7f800000u) ? f[i][j] * down
                                                            : __uint_as_float(0x7fc00000u);
      *(reinterpret_cast<uint2*>(rows + (i * PER + sub) * D) + l) = e4m3_encode8(g);
    } else if (older && byte > was && byte < 255 && pos < first) {
      uint2* at = reinterpret_cast<uint2*>(rows + (i * PER + sub) * D) + l;
      float g[8];
      e4m3_decode8(*at, g);
      const float less = pow2(max(was - byte, -126));
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] *= less;
      *at = e4m3_encode8(g);
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

// Warps 0 .. of the launch: the blocks of k and v; behind them q.
template <int D, bool INTER, int PASSES>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const AppendParams p, int64_t kv_items) {
  constexpr int PER = PASSES * 256 / D;
  int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  griddep_wait();
  if (item < kv_items) {
    const int side = (int)(item & 1);
    item >>= 1;
    const int h = (int)(item % p.c.heads);
    item /= p.c.heads;
    append_block<D, INTER>(p, (int)(item / p.nblocks), (int)(item % p.nblocks), h, side);
    return;
  }
  item -= kv_items;
  const int chunks = (p.r.heads_q + PER - 1) / PER;
  if (chunks == 0) return;
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
  for (int i = lane; i < 2 * c.heads * L; i += 32) {
    const int64_t head = i / L;
    const int l = i % L;
    uint4 raw = make_uint4(0, 0, 0, 0);
    float scale = absent ? __uint_as_float(0x7fc00000u) : 0.0f;
    if (read) {
      const int64_t row = (head << c.page_shift) + in_page;
      raw = *(reinterpret_cast<const uint4*>(c.codes + page * c.page_stride + row * D) + l);
      scale = e8m0_value(__ldg(c.scales + page * c.scale_stride + row / kKvBlock));
    }
    const bool is_v = head >= c.heads;
    __nv_bfloat16* out = is_v ? p.v_out + r * p.ld_v + (head - c.heads) * D
                              : p.k_out + r * p.ld_k + head * D;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float f[8];
      e4m3_decode8(j ? make_uint2(raw.z, raw.w) : make_uint2(raw.x, raw.y), f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= scale;
      *(reinterpret_cast<uint4*>(out) + 2 * l + j) = pack_bf16(f);
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

template <int D, bool INTER, int PASSES>
cudaError_t append_launch(const AppendParams& p, cudaStream_t st) {
  constexpr int PER = PASSES * 256 / D;
  const int64_t kv_items = 2ll * p.c.heads * p.nblocks * p.c.batch;
  const int64_t q_items = p.r.q ? p.r.T * ((p.r.heads_q + PER - 1) / PER) : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks_of(kv_items + q_items));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_kernel<D, INTER, PASSES>, p, kv_items);
}

template <int D>
cudaError_t append(const AppendParams& p, cudaStream_t st) {
  constexpr int PER = 256 / D;
  const bool many = p.r.T * ((p.r.heads_q + PER - 1) / PER) > 64 * (int64_t)sm_count();
  if (p.r.interleaved)
    return many ? append_launch<D, true, 4>(p, st) : append_launch<D, true, 1>(p, st);
  return many ? append_launch<D, false, 4>(p, st) : append_launch<D, false, 1>(p, st);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, int head_dim, cudaStream_t st) {
  return head_dim == 128 ? qk<128>(p, st) : qk<64>(p, st);
}

cudaError_t launch_kv_append(const AppendParams& p, int head_dim, cudaStream_t st) {
  return head_dim == 128 ? append<128>(p, st) : append<64>(p, st);
}

cudaError_t launch_kv_gather(const GatherParams& p, int head_dim, cudaStream_t st) {
  if (head_dim == 128)
    return launch_pdl(gather_kernel<128>, dim3(blocks_of(p.c.T)), dim3(32 * kWarps), 0, st, p);
  return launch_pdl(gather_kernel<64>, dim3(blocks_of(p.c.T)), dim3(32 * kWarps), 0, st, p);
}

}  // namespace ig
