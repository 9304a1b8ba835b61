// Host side of the quantised-block entry points (MX4 quantisation, its
// inverse, the MX4 product, the block norm): argument checks, then one launch
// each. Nothing is enqueued for an argument error.
#include "mx4.cuh"

using namespace ig;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? IG_OK : IG_ERR_CUDA; }

bool known_type(int t) { return t == IG_TYPE_BF16 || t == IG_TYPE_F32; }

// rows x K of an MX4 operand. Coordinates and grids are 32-bit; offsets 64-bit.
int check_mx4(int64_t rows, int64_t K) {
  if (rows < 0 || K < kMx4Block || K % kMx4Block) return IG_ERR_SHAPE;
  if (rows > (1ll << 31) - 1 || K > (1ll << 31) - 128) return IG_ERR_UNSUPPORTED;
  if (rows > 0 && K > ((int64_t)1 << 44) / rows) return IG_ERR_UNSUPPORTED;
  return IG_OK;
}

int check_ld(int64_t ld, int64_t cols) { return ld < cols || ld % 8 ? IG_ERR_SHAPE : IG_OK; }

}  // namespace

extern "C" {

size_t ig_mx4_scale_bytes(int64_t rows, int64_t K) {
  if (check_mx4(rows, K) != IG_OK) return 0;
  return (size_t)((rows + 127) / 128 * mx4_ktiles(K) * kMx4TileBytes);
}

size_t ig_mx4_workspace_bytes(void) { return kMapOffset; }

int ig_mx4_quantize(int64_t rows, int64_t K, const void* x, int64_t ld_x, int x_type,
                    void* codes, void* scales, void* stream) {
  int rc = check_mx4(rows, K);
  if (rc != IG_OK) return rc;
  if (!known_type(x_type)) return IG_ERR_ARG;
  rc = check_ld(ld_x, K);
  if (rc != IG_OK) return rc;
  if (rows == 0) return IG_OK;
  if (!x || !codes || !scales) return IG_ERR_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return IG_ERR_ALIGN;
  Mx4QuantParams p;
  p.x = x;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  p.rows = rows;
  p.K = K;
  p.ldx = ld_x;
  p.kt = mx4_ktiles(K);
  return cuda_status(launch_mx4_quantize(p, x_type == IG_TYPE_F32,
                                         static_cast<cudaStream_t>(stream)));
}

int ig_mx4_dequantize(int64_t rows, int64_t K, const void* codes, const void* scales, void* out,
                      int64_t ld_out, int out_type, void* stream) {
  int rc = check_mx4(rows, K);
  if (rc != IG_OK) return rc;
  if (!known_type(out_type)) return IG_ERR_ARG;
  rc = check_ld(ld_out, K);
  if (rc != IG_OK) return rc;
  if (rows == 0) return IG_OK;
  if (!codes || !scales || !out) return IG_ERR_ARG;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(out)) return IG_ERR_ALIGN;
  Mx4DequantParams p;
  p.codes = static_cast<const uint8_t*>(codes);
  p.scales = static_cast<const uint8_t*>(scales);
  p.out = out;
  p.rows = rows;
  p.K = K;
  p.ldo = ld_out;
  p.kt = mx4_ktiles(K);
  const int64_t pitch = ld_out * (out_type == IG_TYPE_F32 ? 4 : 2);
  p.wide = (reinterpret_cast<uintptr_t>(out) % 32 == 0) && (rows == 1 || pitch % 32 == 0);
  return cuda_status(launch_mx4_dequantize(p, out_type == IG_TYPE_F32,
                                           static_cast<cudaStream_t>(stream)));
}

int ig_mx4_gemm(const ig_mx4_shape* shape, const void* x_codes, const void* x_scales,
                const void* w_codes, const void* w_scales, void* y, void* ws, size_t ws_bytes,
                void* stream) {
  if (!shape) return IG_ERR_ARG;
  if (shape->flags & ~(IG_FLAG_STATIC_WEIGHTS | IG_FLAG_TEST_COPY_TIMEOUT)) return IG_ERR_ARG;
  if (!known_type(shape->y_type)) return IG_ERR_ARG;
  int rc = check_mx4(shape->M, shape->K);
  if (rc != IG_OK) return rc;
  rc = check_mx4(shape->N, shape->K);
  if (rc != IG_OK) return rc;
  if (shape->N < 8 || shape->N % 8) return IG_ERR_SHAPE;
  rc = check_ld(shape->ld_y, shape->N);
  if (rc != IG_OK) return rc;
  if (shape->M == 0) return IG_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !y || !ws) return IG_ERR_ARG;
  if (!aligned16(x_codes) || !aligned16(x_scales) || !aligned16(w_codes) ||
      !aligned16(w_scales) || !aligned16(y) || !aligned16(ws))
    return IG_ERR_ALIGN;
  if (ws_bytes < ig_mx4_workspace_bytes()) return IG_ERR_WS_SMALL;
  Mx4GemmParams p;
  p.xc = static_cast<const uint8_t*>(x_codes);
  p.xs = static_cast<const uint8_t*>(x_scales);
  p.wc = static_cast<const uint8_t*>(w_codes);
  p.ws = static_cast<const uint8_t*>(w_scales);
  p.y = y;
  p.M = shape->M;
  p.N = shape->N;
  p.K = shape->K;
  p.ldy = shape->ld_y;
  p.kt = mx4_ktiles(shape->K);
  p.y_f32 = shape->y_type == IG_TYPE_F32;
  p.flags = shape->flags;
  p.status = static_cast<uint32_t*>(ws);
  return cuda_status(launch_mx4_gemm(p, static_cast<cudaStream_t>(stream)));
}

int ig_block_norm(const ig_norm_shape* s, const void* h, const void* y, const void* gate,
                  const void* w_post, const void* w_pre, void* h_out, void* n_out, void* codes,
                  void* scales, void* stream) {
  if (!s) return IG_ERR_ARG;
  if (s->flags & ~IG_NORM_WEIGHT_PLUS_ONE) return IG_ERR_ARG;
  if (!known_type(s->h_type)) return IG_ERR_ARG;
  if (s->gate_col_stride != 0 && s->gate_col_stride != 1) return IG_ERR_ARG;
  if (s->M < 0 || s->H < 8 || s->H % 8) return IG_ERR_SHAPE;
  if (s->M > (1ll << 31) - 1 || s->H > kNormMaxH) return IG_ERR_UNSUPPORTED;
  if (!(s->eps >= 0.0f)) return IG_ERR_ARG;
  if (s->M == 0) return IG_OK;        // an empty tensor may have no address
  // something to read, something to write; what belongs to a part of the
  // operator is given with that part only
  if ((!h && !y) || (!h_out && !n_out && !codes)) return IG_ERR_ARG;
  if (!y && (gate || w_post)) return IG_ERR_ARG;
  if (!w_pre != (!n_out && !codes)) return IG_ERR_ARG;
  if (!codes != !scales) return IG_ERR_ARG;
  if (codes && s->H % kMx4Block) return IG_ERR_SHAPE;
  if ((h && check_ld(s->ld_h, s->H) != IG_OK) || (y && check_ld(s->ld_y, s->H) != IG_OK) ||
      (h_out && check_ld(s->ld_h_out, s->H) != IG_OK) ||
      (n_out && check_ld(s->ld_n, s->H) != IG_OK))
    return IG_ERR_SHAPE;
  if (gate && (s->gate_row_stride < 0 || (s->gate_col_stride && s->gate_row_stride % 8)))
    return IG_ERR_SHAPE;
  if (!aligned16(h) || !aligned16(y) || !aligned16(w_post) || !aligned16(w_pre) ||
      !aligned16(h_out) || !aligned16(n_out) || !aligned16(codes) || !aligned16(scales))
    return IG_ERR_ALIGN;
  // one gate value per row is read by itself: a column of a wider tensor will do
  if ((uintptr_t)gate & (s->gate_col_stride ? 15u : 1u)) return IG_ERR_ALIGN;
  NormParams p;
  p.h = h;
  p.y = static_cast<const __nv_bfloat16*>(y);
  p.gate = static_cast<const __nv_bfloat16*>(gate);
  p.w_post = static_cast<const __nv_bfloat16*>(w_post);
  p.w_pre = static_cast<const __nv_bfloat16*>(w_pre);
  p.h_out = h_out;
  p.n_out = static_cast<__nv_bfloat16*>(n_out);
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  p.rows = s->M;
  p.H = s->H;
  p.ld_h = s->ld_h;
  p.ld_y = s->ld_y;
  p.ld_ho = s->ld_h_out;
  p.ld_n = s->ld_n;
  p.gate_rs = s->gate_row_stride;
  p.gate_cs = s->gate_col_stride;
  p.kt = mx4_ktiles(s->H);
  p.plus_one = s->flags & IG_NORM_WEIGHT_PLUS_ONE;
  p.eps = s->eps;
  p.scale = s->scale;
  return cuda_status(launch_block_norm(p, s->h_type == IG_TYPE_F32,
                                       static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
