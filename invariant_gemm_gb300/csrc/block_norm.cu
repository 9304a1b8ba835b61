// Norm after a block, gate, residual and norm before the next block:
//   t = y rsqrt(mean(y^2) + eps) w_post,  h' = h + scale gate t,
//   n = h' rsqrt(mean(h'^2) + eps) w_pre, and n in MX4.
//
// One row per thread block, one pass: a thread holds its vectors of 8 values
// of the row from the load to the last store, in registers but for a few words
// that go to local memory (stored + loaded bytes a thread by V and W, below:
// bf16 rows 0 for V = 2, W = 1, 36 + 36 for W = 2, 84 + 60 for V = 4; FP32 rows
// 12 + 8, 0 and 124 + 108).
//
// The order of the sums is fixed by H: a row has `slots` places for vectors,
// cut into V runs of T places; the values of the vectors at places t, t + T,
// ... are added one after the other (t < T; even and odd values apart, then
// together), the T sums by a butterfly over
// each 32 of them, then one over those. A thread does this for one t, or, in
// blocks of half the size, for two (W = 2) that lie T / 2 apart and so in
// different groups of 32: the same sums, the same bits.
//
// Bound by memory where there are many rows, and close to bound by
// instructions there. W = 2 has fewer, longer threads, so more rows at work
// per SM and less work per row; few rows are over sooner with W = 1
// (launch_block_norm has the figures). Copying rows ahead through shared memory by
// blocks that stay (cp.async, 3 rows deep) was slower than fresh blocks: 107
// against 87 us at 8192 x 8192, which now takes 82-84 us (bf16, 537 MB: 6.5 TB/s);
// 1001 x 11008 FP32 with a gate for each value 28-30 us (5.1-5.6 TB/s), 4000 of
// those rows 96 us (6.4 TB/s). With n in MX4 alone 8192 x 8192 takes 88 us (5.0
// TB/s, instructions issued in 77% of the cycles), the norm of h alone 49 us
// (268 MB: 5.5 TB/s) and with MX4 out 62 us (2.8 TB/s).
//
// Far from memory's rate: short rows, where a block has 64 threads for as few as
// 8 vectors (8192 rows of 64 to 256 values 9 us, of 512 10 us); FP32 rows above
// 12288 and all rows above 16384, whose blocks leave room for no other on their
// SM (4000 x 16384 FP32 168 us, 4.7 TB/s, where 12288 reach 6.5; 4000 x 32768 bf16
// 178 us, 5.9 TB/s, FP32 371 us, 4.2 TB/s).
//
// The next kernel on the stream starts when this one is complete (no early
// release): it may be one that reads n before its own wait, as the fused LoRA
// kernel does with IG_FLAG_INPUT_READY once one more kernel lies between.
#include "mx4.cuh"

namespace ig {

namespace {

// Sum over the block's T sums, W of them in a thread.
template <int W>
__device__ __forceinline__ float block_sum(float (&v)[W], float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < W; ++i) red[warp + i * nw] = v[i];
  }
  __syncthreads();
  float t = lane < W * nw ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// Pairs of FP32 values in one 64-bit register: products and sums of a pair are
// one instruction on this architecture. The kernel is close to bound by
// instructions where it is bound by memory, so everything between the loads
// and the stores works on pairs.
using f2 = uint64_t;

__device__ __forceinline__ f2 pair(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(f2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void unpack4(const uint4& u, f2 (&v)[4]) {
  v[0] = pair(bf16lo(u.x), bf16hi(u.x));
  v[1] = pair(bf16lo(u.y), bf16hi(u.y));
  v[2] = pair(bf16lo(u.z), bf16hi(u.z));
  v[3] = pair(bf16lo(u.w), bf16hi(u.w));
}
__device__ __forceinline__ uint4 pack4(const f2 (&v)[4]) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = split(v[i]);
    o[i] = f32x2_to_bf16x2_bits(t.x, t.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Threads and blocks per SM that the registers are cut for: 64 a thread, but
// 80 for two sums over FP32 rows, of which blocks of up to 384 threads share
// an SM in pairs (two of 96 registers would not fit).
__host__ __device__ constexpr int max_threads(bool f32, int w) {
  return w == 1 ? 1024 : f32 ? 384 : 512;
}

template <bool F32, int W, int V>
__global__ void __launch_bounds__(max_threads(F32, W), W) norm_kernel(NormParams p) {
  constexpr int HV = F32 ? 2 : 1;        // 16-byte words of h per vector
  __shared__ float red[2][32];
  const int tid = threadIdx.x, T = W * blockDim.x;
  const int vecs = (int)(p.H / 8);
  const int64_t row = blockIdx.x;
  const f2 offset = pair((float)p.plus_one, (float)p.plus_one);
  auto weight = [&](const uint4& raw, f2 (&w)[4]) {
    unpack4(raw, w);
    if (p.plus_one) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = add2(w[i], offset);
    }
  };
  // place of vector j of this thread's i-th sum
  auto place = [&](int i, int j) { return tid + i * (int)blockDim.x + j * T; };
  griddep_wait();

  uint4 y[W][V], h[W][V][HV], g[W][V];
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = place(i, j);
      y[i][j] = make_uint4(0, 0, 0, 0);
      if (p.y && c < vecs)
        y[i][j] = *(reinterpret_cast<const uint4*>(p.y + row * p.ld_y) + c);
    }
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = place(i, j);
#pragma unroll
      for (int q = 0; q < HV; ++q) h[i][j][q] = make_uint4(0, 0, 0, 0);
      if (!p.h || c >= vecs) continue;
      const uint4* at =
          F32 ? reinterpret_cast<const uint4*>(static_cast<const float*>(p.h) + row * p.ld_h)
              : reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.h) +
                                               row * p.ld_h);
#pragma unroll
      for (int q = 0; q < HV; ++q) h[i][j][q] = at[c * HV + q];
    }
  const bool gates = p.gate && p.gate_cs;     // a gate value for each place
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = place(i, j);
      g[i][j] = make_uint4(0, 0, 0, 0);
      if (gates && c < vecs)
        g[i][j] = *(reinterpret_cast<const uint4*>(p.gate + row * p.gate_rs) + c);
    }

  const float row_gate =
      p.gate && !gates ? __bfloat162float(p.gate[row * p.gate_rs]) : 1.0f;

  // u = y times its weights and gates, while the sum is on its way; what is
  // left after it is one product and sum a value; the second norm's weights are
  // on their way through its sum likewise (8192 x 8192 bf16: 82 us against 89
  // with both after the sums). Two sums over FP32 rows have no registers for
  // them beside h: 4000 x 11008 with full gates 118 us against 99.
  constexpr bool kEarly = !(F32 && W == 2);
  f2 u[kEarly ? W : 1][kEarly ? V : 1][4];
  auto weigh = [&](int i, int j, f2 (&v)[4]) {
    const int c = place(i, j);
    f2 w[4];
    if (p.w_post && c < vecs) {
      weight(__ldg(reinterpret_cast<const uint4*>(p.w_post) + c), w);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = mul2(v[k], w[k]);
    }
    if (gates) {
      unpack4(g[i][j], w);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = mul2(v[k], w[k]);
    }
  };
  if constexpr (!kEarly) {
    // the norm weights to L1, a line for each eight lanes (1001 x 11008: 33 ->
    // 30 us)
    auto touch = [&](const __nv_bfloat16* at, int c) {
      asm volatile("prefetch.global.L1 [%0];" ::"l"(reinterpret_cast<const uint4*>(at) + c));
    };
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = place(i, j);
        if (c >= vecs || (c & 7) != 0) continue;
        if (p.w_post) touch(p.w_post, c);
        if (p.w_pre) touch(p.w_pre, c);
      }
  }
  float s[W], f = p.scale;
  if (kEarly || p.w_post) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      f2 ss = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        f2 v[4];
        unpack4(y[i][j], v);
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = fma2(v[k], v[k], ss);
        if constexpr (kEarly) {
          weigh(i, j, v);
#pragma unroll
          for (int k = 0; k < 4; ++k) u[i][j][k] = v[k];
        }
      }
      const float2 t = split(ss);
      s[i] = t.x + t.y;
    }
    if (p.w_post) f *= rsqrtf(block_sum<W>(s, red[0]) / (float)p.H + p.eps);
  }
  if (p.gate && !gates) f *= row_gate;
  f2 r[W][V][4], ff = pair(f, f);         // h'
#pragma unroll
  for (int i = 0; i < W; ++i) {
    f2 ss = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = place(i, j);
      if (F32) {
        const uint4 a = h[i][j][0], b = h[i][j][HV - 1];
        r[i][j][0] = pair(__uint_as_float(a.x), __uint_as_float(a.y));
        r[i][j][1] = pair(__uint_as_float(a.z), __uint_as_float(a.w));
        r[i][j][2] = pair(__uint_as_float(b.x), __uint_as_float(b.y));
        r[i][j][3] = pair(__uint_as_float(b.z), __uint_as_float(b.w));
      } else {
        unpack4(h[i][j][0], r[i][j]);
      }
      if (c >= vecs) continue;
      if (p.y) {
        f2 v[4];
        if constexpr (kEarly) {
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = u[i][j][k];
        } else {
          unpack4(y[i][j], v);
          weigh(i, j, v);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) r[i][j][k] = fma2(v[k], ff, r[i][j][k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) ss = fma2(r[i][j][k], r[i][j][k], ss);
      if (p.h_out) {
        if (F32) {
          float4* q = reinterpret_cast<float4*>(static_cast<float*>(p.h_out) + row * p.ld_ho) +
                      2 * c;
          const float2 t0 = split(r[i][j][0]), t1 = split(r[i][j][1]), t2 = split(r[i][j][2]),
                       t3 = split(r[i][j][3]);
          q[0] = make_float4(t0.x, t0.y, t1.x, t1.y);
          q[1] = make_float4(t2.x, t2.y, t3.x, t3.y);
        } else {
          *(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.h_out) + row * p.ld_ho) + c) =
              pack4(r[i][j]);
        }
      }
    }
    const float2 t = split(ss);
    s[i] = t.x + t.y;
  }
  if (!p.w_pre) return;
  auto w_pre = [&](int c) { return __ldg(reinterpret_cast<const uint4*>(p.w_pre) + c); };
  uint4 wp[kEarly ? W : 1][kEarly ? V : 1];      // on their way through the second sum
  if constexpr (kEarly) {
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = place(i, j);
        wp[i][j] = make_uint4(0, 0, 0, 0);
        if (c < vecs) wp[i][j] = w_pre(c);
      }
  }
  f = rsqrtf(block_sum<W>(s, red[1]) / (float)p.H + p.eps);
  ff = pair(f, f);
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = place(i, j);
      const bool in = c < vecs;
      uint4 o = make_uint4(0, 0, 0, 0);
      if (in) {
        f2 n[4];
        if constexpr (kEarly) weight(wp[i][j], n);
        else weight(w_pre(c), n);
#pragma unroll
        for (int k = 0; k < 4; ++k) n[k] = mul2(mul2(r[i][j][k], ff), n[k]);
        o = pack4(n);
        if (p.n_out) *(reinterpret_cast<uint4*>(p.n_out + row * p.ld_n) + c) = o;
      }
      if (p.codes) {
        // places past the row's end are those that pad K to 128
        float n[8];
        unpack8(o, n);
        const uint32_t byte = mx4_block_byte<4>(top_of(o));
        const uint32_t codes = mx4_encode8(n, byte);
        const uint32_t word = mx4_scale_word<4>(in ? byte : 127u);
        if (in) reinterpret_cast<uint32_t*>(p.codes)[row * vecs + c] = codes;
        if (c % 16 == 0 && c < p.kt * 16)
          *reinterpret_cast<uint32_t*>(p.scales + mx4_scale_at(row, c / 4, p.kt)) = word;
      }
    }
}

template <bool F32, int W, int V>
cudaError_t launch(const NormParams& p, int threads, cudaStream_t st) {
  return launch_pdl(norm_kernel<F32, W, V>, dim3((unsigned)p.rows), dim3(threads), 0, st, p);
}

// V = 2 up to H = 16384, V = 4 to 32768 (always 1024 threads at most). Two sums
// a thread from where the rows at one a thread would not all be at work at
// once (1024 threads an SM). bf16 rows of 8192: 304 of them 6.2 us with one, 7.3
// with two; 608 of them 10.8 and 10.0; FP32 rows of 11008: 152 of them 7.6 and
// 7.6, 608 of them 25.1 and 18.4. Short rows (T < 256) keep one: 608 of 2048
// 4.6 and 6.0; so do those of V = 4, whose two sums would not fit the registers.
template <bool F32>
cudaError_t launch_rows(const NormParams& p, cudaStream_t st) {
  const int V = p.H <= 16384 ? 2 : 4;
  const int64_t slots = mx4_ktiles(p.H) * 16;
  const int T = (int)((slots + V * 64 - 1) / (V * 64) * 64);
  if (V == 4) return launch<F32, 1, 4>(p, T, st);
  const bool two = T >= 256 && T / 2 <= max_threads(F32, 2) && p.rows * T > 1024 * sm_count();
  return two ? launch<F32, 2, 2>(p, T / 2, st) : launch<F32, 1, 2>(p, T, st);
}

}  // namespace

cudaError_t launch_block_norm(const NormParams& p, bool h_f32, cudaStream_t st) {
  return h_f32 ? launch_rows<true>(p, st) : launch_rows<false>(p, st);
}

}  // namespace ig
