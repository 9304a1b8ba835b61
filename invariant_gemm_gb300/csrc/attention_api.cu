// Host side of the calls of a served layer's attention (head norms with the
// rotation, the 8-bit paged cache, attention over it): argument checks, then the
// launches. Nothing is enqueued for an argument error.
#include "attention.cuh"

using namespace ig;

namespace {

bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? IG_OK : IG_ERR_CUDA; }

constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxBatch = 8192;

int check_ld(int64_t ld, int64_t cols) { return ld < cols || ld % 8 ? IG_ERR_SHAPE : IG_OK; }

int check_ws(const void* ws, size_t bytes, size_t need) {
  if (!ws) return IG_ERR_ARG;
  if (!aligned16(ws)) return IG_ERR_ALIGN;
  return bytes < need ? IG_ERR_WS_SMALL : IG_OK;
}

int check_heads(int32_t heads, int32_t head_dim) {
  if (heads < 1 || head_dim < 1) return IG_ERR_SHAPE;
  if ((head_dim != 64 && head_dim != 128) || heads > kMaxHeads) return IG_ERR_UNSUPPORTED;
  return IG_OK;
}

// Sizes of a cache, without its addresses.
int check_cache_sizes(const ig_kv_cache* c) {
  if (c->reserved != 0) return IG_ERR_ARG;
  const int rc = check_heads(c->heads, c->head_dim);
  if (rc != IG_OK) return rc;
  if (c->page < kKvBlock || (c->page & (c->page - 1))) return IG_ERR_SHAPE;
  return c->page > 256 ? IG_ERR_UNSUPPORTED : IG_OK;
}

int check_cache(const ig_kv_cache* c) {
  if (!c) return IG_ERR_ARG;
  int rc = check_cache_sizes(c);
  if (rc != IG_OK) return rc;
  const int64_t rows = 2ll * c->heads * c->page;
  if (c->pages < 1 || c->page_stride < rows * c->head_dim || c->page_stride % 16 ||
      c->scale_stride < rows / kKvBlock)
    return IG_ERR_SHAPE;
  if (c->pages > (1ll << 31) - 1 || c->page_stride > (1ll << 40) - 16 ||
      c->pages > ((int64_t)1 << 46) / c->page_stride || c->scale_stride > (1ll << 40))
    return IG_ERR_UNSUPPORTED;
  if (!c->codes || !c->scales) return IG_ERR_ARG;
  return aligned16(c->codes) ? IG_OK : IG_ERR_ALIGN;
}

int check_batch(const ig_batch* b) {
  if (!b) return IG_ERR_ARG;
  if (b->batch < 0 || b->max_q < 0 || b->ld_table < 1) return IG_ERR_SHAPE;
  if (b->batch > kMaxBatch || b->ld_table > (1 << 24)) return IG_ERR_UNSUPPORTED;
  if (b->batch == 0) return IG_OK;
  if (!b->cu || !b->kv_len || !b->page_table) return IG_ERR_ARG;
  return aligned(b->cu, 4) && aligned(b->kv_len, 4) && aligned(b->page_table, 4) ? IG_OK
                                                                                 : IG_ERR_ALIGN;
}

int check_tokens(int64_t T) {
  return T < 0 ? IG_ERR_SHAPE : T > (1ll << 30) ? IG_ERR_UNSUPPORTED : IG_OK;
}

KvParams kv_params(const ig_kv_cache* c, const ig_batch* b, int64_t T, void* ws) {
  KvParams p;
  p.codes = static_cast<uint8_t*>(c->codes);
  p.scales = static_cast<uint8_t*>(c->scales);
  p.cu = b->cu;
  p.kv_len = b->kv_len;
  p.table = b->page_table;
  p.status = static_cast<uint32_t*>(ws);
  p.pages = c->pages;
  p.page_stride = c->page_stride;
  p.scale_stride = c->scale_stride;
  p.ld_table = b->ld_table;
  p.T = T;
  p.batch = b->batch;
  p.max_q = b->max_q;
  p.heads = c->heads;
  p.page_shift = __builtin_ctz((unsigned)c->page);
  return p;
}

// Checks a rope shape with the sides that are given, and fills the parameters.
int rope_params(const ig_rope_shape* s, const void* q, const void* k, const void* w_q,
                const void* w_k, const float* cos_sin, const int32_t* positions, bool need_pos,
                void* q_out, RopeParams* p) {
  if (s->flags & ~(IG_NORM_WEIGHT_PLUS_ONE | IG_ROPE_INTERLEAVED)) return IG_ERR_ARG;
  if (!(s->eps >= 0.0f)) return IG_ERR_ARG;
  int rc = check_tokens(s->T);
  if (rc != IG_OK) return rc;
  if (q && (rc = check_heads(s->heads_q, s->head_dim)) != IG_OK) return rc;
  if (k && (rc = check_heads(s->heads_k, s->head_dim)) != IG_OK) return rc;
  if (cos_sin) {
    if (s->rot_dim < 16 || s->rot_dim % 16 || s->rot_dim > s->head_dim || s->table_rows < 1)
      return IG_ERR_SHAPE;
    if (s->table_rows > (1ll << 31) - 1) return IG_ERR_UNSUPPORTED;
    if (need_pos && !positions) return IG_ERR_ARG;
  } else if (positions) {
    return IG_ERR_ARG;
  }
  if ((!q && (w_q || q_out)) || (q && !q_out) || (!k && w_k)) return IG_ERR_ARG;
  if (s->T * ((int64_t)(q ? s->heads_q : 0) + (k ? s->heads_k : 0)) > (1ll << 32))
    return IG_ERR_UNSUPPORTED;
  const int64_t cq = (int64_t)s->heads_q * s->head_dim, ck = (int64_t)s->heads_k * s->head_dim;
  if ((q && (check_ld(s->ld_q, cq) != IG_OK || check_ld(s->ld_q_out, cq) != IG_OK)) ||
      (k && check_ld(s->ld_k, ck) != IG_OK))
    return IG_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(w_q) || !aligned16(w_k) ||
      !aligned16(cos_sin) || !aligned(positions, 4) || !aligned16(q_out))
    return IG_ERR_ALIGN;
  if (q && q == q_out && s->ld_q != s->ld_q_out) return IG_ERR_SHAPE;
  p->q = static_cast<const __nv_bfloat16*>(q);
  p->k = static_cast<const __nv_bfloat16*>(k);
  p->w_q = static_cast<const __nv_bfloat16*>(w_q);
  p->w_k = static_cast<const __nv_bfloat16*>(w_k);
  p->cos_sin = cos_sin;
  p->positions = positions;
  p->q_out = static_cast<__nv_bfloat16*>(q_out);
  p->k_out = nullptr;
  p->T = s->T;
  p->table_rows = s->table_rows;
  p->ld_q = s->ld_q;
  p->ld_k = s->ld_k;
  p->ld_qo = s->ld_q_out;
  p->ld_ko = 0;
  p->heads_q = q ? s->heads_q : 0;
  p->heads_k = k ? s->heads_k : 0;
  p->rot = cos_sin ? s->rot_dim : 0;
  p->interleaved = (s->flags & IG_ROPE_INTERLEAVED) != 0;
  p->plus_one = (s->flags & IG_NORM_WEIGHT_PLUS_ONE) != 0;
  p->eps = s->eps;
  return IG_OK;
}

// What the workspace of an attention call holds behind the status word and the
// counters (of which it uses two).
struct AttnPlan {
  int group, max_tiles, max_parts, part_rows;
  int big_rows, big_by_row, tiles_by_row;
  size_t ml_at, big_at, big_ml_at, total;    // behind the counters
};

int attn_plan(const ig_attn_shape* s, const ig_kv_cache* c, const ig_batch* b, AttnPlan* pl) {
  if (!s || !c || !b) return IG_ERR_ARG;
  if (s->flags & ~IG_FLAG_TEST_COPY_TIMEOUT || s->reserved != 0) return IG_ERR_ARG;
  int rc = check_cache_sizes(c);
  if (rc != IG_OK) return rc;
  rc = check_heads(s->heads_q, c->head_dim);
  if (rc != IG_OK) return rc;
  if (s->heads_q % c->heads) return IG_ERR_SHAPE;
  if ((rc = check_tokens(s->T)) != IG_OK) return rc;
  if (b->batch < 0 || b->max_q < 0 || b->ld_table < 1) return IG_ERR_SHAPE;
  if (b->batch > kMaxBatch || b->ld_table > (1 << 24) ||
      b->ld_table * c->page > (1ll << 30))
    return IG_ERR_UNSUPPORTED;
  pl->group = s->heads_q / c->heads;
  const int64_t rows = (int64_t)pl->group * b->max_q;
  if (rows > (1 << 28)) return IG_ERR_UNSUPPORTED;
  pl->max_tiles = (int)(((rows < kFewRows ? rows : kFewRows) + 15) / 16);
  pl->part_rows = (int)(rows < 16 ? rows : 16);
  const int64_t cap = b->ld_table * c->page;
  pl->max_parts = cap < 256 * kMaxSplits ? (int)((cap + 255) / 256) : kMaxSplits;
  const int64_t many = s->T * pl->group;        // rows of all sequences
  int64_t tiles = (int64_t)b->batch * pl->max_tiles;
  pl->tiles_by_row = b->batch + many / 16 < tiles;
  if (pl->tiles_by_row) tiles = b->batch + many / 16;
  const int64_t items = tiles * c->heads * pl->max_parts;
  if (items > (1ll << 30)) return IG_ERR_UNSUPPORTED;
  pl->ml_at = align_up((size_t)items * pl->part_rows * c->head_dim * 4, 256);
  pl->big_at = align_up(pl->ml_at + (size_t)items * pl->part_rows * kPartWords * 4, 256);
  // sequences that the prompt kernel may cut: more rows than the split kernel's, of
  // few enough tiles, long enough
  pl->big_rows = pl->big_by_row = 0;
  int64_t big = 0;
  if (rows > kFewRows && many > kFewRows && prompt_parts(kFewRows + 1, (int)cap, c->heads) > 1) {
    pl->big_rows = item_rows((int)rows);
    const int64_t most = (int64_t)b->batch * pl->big_rows;
    pl->big_by_row = many < most;
    big = (many < most ? many : most) * kPromptItems;
  }
  // (blocks of the prompt kernel: as its launch counts them)
  if ((many / kPromptRows + b->batch) * c->heads + (int64_t)b->batch * kPromptItems >= 1ll << 31)
    return IG_ERR_UNSUPPORTED;
  pl->big_ml_at = align_up(pl->big_at + (size_t)big * c->head_dim * 4, 256);
  pl->total = kMapOffset + pl->big_ml_at + (size_t)big * kPartWords * 4;
  return IG_OK;
}

}  // namespace

extern "C" {

int ig_qk_norm_rope(const ig_rope_shape* shape, const void* q, const void* k, const void* w_q,
                    const void* w_k, const float* cos_sin, const int32_t* positions, void* q_out,
                    void* k_out, void* ws, size_t ws_bytes, void* stream) {
  if (!shape || (!q && !k && shape->T != 0)) return IG_ERR_ARG;
  RopeParams p;
  int rc = rope_params(shape, q, k, w_q, w_k, cos_sin, positions, shape->T != 0, q_out, &p);
  if (rc != IG_OK) return rc;
  if (shape->T == 0) return IG_OK;
  if (!k != !k_out) return IG_ERR_ARG;
  if (k && check_ld(shape->ld_k_out, (int64_t)shape->heads_k * shape->head_dim) != IG_OK)
    return IG_ERR_SHAPE;
  if (!aligned16(k_out)) return IG_ERR_ALIGN;
  if (k && k == k_out && shape->ld_k != shape->ld_k_out) return IG_ERR_SHAPE;
  rc = check_ws(ws, ws_bytes, kMapOffset);
  if (rc != IG_OK) return rc;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.ld_ko = shape->ld_k_out;
  p.status = static_cast<uint32_t*>(ws);
  return cuda_status(launch_qk_norm_rope(p, shape->head_dim, static_cast<cudaStream_t>(stream)));
}

int ig_kv_append(const ig_rope_shape* shape, const ig_kv_cache* cache, const ig_batch* batch,
                 const void* k, const void* v, int64_t ld_v, const void* q, const void* w_q,
                 const void* w_k, const float* cos_sin, const int32_t* positions, void* q_out,
                 void* ws, size_t ws_bytes, void* stream) {
  if (!shape) return IG_ERR_ARG;
  int rc = check_cache(cache);
  if (rc != IG_OK) return rc;
  rc = check_batch(batch);
  if (rc != IG_OK) return rc;
  AppendParams p;
  rc = rope_params(shape, q, k, w_q, w_k, cos_sin, positions, false, q_out, &p.r);
  if (rc != IG_OK) return rc;
  if (shape->heads_k != cache->heads || shape->head_dim != cache->head_dim) return IG_ERR_SHAPE;
  rc = check_ld(ld_v, (int64_t)cache->heads * cache->head_dim);
  if (rc != IG_OK) return rc;
  if (shape->T == 0 || batch->batch == 0 || batch->max_q == 0) return IG_OK;
  if (!k || !v) return IG_ERR_ARG;
  if (!aligned16(v)) return IG_ERR_ALIGN;
  rc = check_ws(ws, ws_bytes, kMapOffset);
  if (rc != IG_OK) return rc;
  p.c = kv_params(cache, batch, shape->T, ws);
  p.r.status = p.c.status;
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.ld_v = ld_v;
  const int64_t most = batch->max_q < shape->T ? batch->max_q : shape->T;
  p.nblocks = (int)((most + 2 * kKvBlock - 2) / kKvBlock);
  p.r.heads_k = 0;
  if ((int64_t)p.nblocks * batch->batch * cache->heads > (1ll << 29)) return IG_ERR_UNSUPPORTED;
  return cuda_status(launch_kv_append(p, cache->head_dim, static_cast<cudaStream_t>(stream)));
}

int ig_kv_gather(const ig_kv_cache* cache, const ig_batch* batch, int64_t T, void* k_out,
                 int64_t ld_k_out, void* v_out, int64_t ld_v_out, void* ws, size_t ws_bytes,
                 void* stream) {
  int rc = check_cache(cache);
  if (rc != IG_OK) return rc;
  rc = check_batch(batch);
  if (rc != IG_OK) return rc;
  if ((rc = check_tokens(T)) != IG_OK) return rc;
  const int64_t cols = (int64_t)cache->heads * cache->head_dim;
  if (check_ld(ld_k_out, cols) != IG_OK || check_ld(ld_v_out, cols) != IG_OK) return IG_ERR_SHAPE;
  if (T == 0 || batch->batch == 0) return IG_OK;
  if (!k_out || !v_out) return IG_ERR_ARG;
  if (!aligned16(k_out) || !aligned16(v_out)) return IG_ERR_ALIGN;
  rc = check_ws(ws, ws_bytes, kMapOffset);
  if (rc != IG_OK) return rc;
  GatherParams p;
  p.c = kv_params(cache, batch, T, ws);
  p.c.max_q = 0x7fffffff;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.ld_k = ld_k_out;
  p.ld_v = ld_v_out;
  return cuda_status(launch_kv_gather(p, cache->head_dim, static_cast<cudaStream_t>(stream)));
}

size_t ig_attention_workspace_bytes(const ig_attn_shape* shape, const ig_kv_cache* cache,
                                    const ig_batch* batch) {
  AttnPlan pl;
  return attn_plan(shape, cache, batch, &pl) == IG_OK ? pl.total : 0;
}

int ig_paged_attention(const ig_attn_shape* shape, const ig_kv_cache* cache,
                       const ig_batch* batch, const void* q, void* out, void* ws,
                       size_t ws_bytes, void* stream) {
  AttnPlan pl;
  int rc = attn_plan(shape, cache, batch, &pl);
  if (rc != IG_OK) return rc;
  rc = check_cache(cache);
  if (rc != IG_OK) return rc;
  rc = check_batch(batch);
  if (rc != IG_OK) return rc;
  const int64_t cols = (int64_t)shape->heads_q * cache->head_dim;
  if (check_ld(shape->ld_q, cols) != IG_OK || check_ld(shape->ld_out, cols) != IG_OK)
    return IG_ERR_SHAPE;
  if (!(shape->scale > -3e38f && shape->scale < 3e38f)) return IG_ERR_ARG;
  if (shape->T == 0 || batch->batch == 0 || batch->max_q == 0) return IG_OK;
  if (!q || !out || q == out) return IG_ERR_ARG;
  if (!aligned16(q) || !aligned16(out)) return IG_ERR_ALIGN;
  rc = check_ws(ws, ws_bytes, pl.total);
  if (rc != IG_OK) return rc;
  AttnParams p;
  rc = encode_map_codes(&p.tm, cache->codes, cache->head_dim, 2ull * cache->heads * cache->page,
                        (uint64_t)cache->pages, (uint64_t)cache->page_stride);
  if (rc != IG_OK) return rc;
  p.c = kv_params(cache, batch, shape->T, ws);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.next = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + kCountersOffset);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kMapOffset);
  p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kMapOffset + pl.ml_at);
  p.big = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kMapOffset + pl.big_at);
  p.big_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kMapOffset + pl.big_ml_at);
  p.big_rows = pl.big_rows;
  p.big_by_row = pl.big_by_row;
  p.tiles_by_row = pl.tiles_by_row;
  p.ld_q = shape->ld_q;
  p.ld_out = shape->ld_out;
  p.heads_q = shape->heads_q;
  p.group = pl.group;
  p.group_rcp = 1.0f / (float)pl.group;
  p.group_inv = (uint32_t)((65536 + pl.group - 1) / pl.group);
  p.group_magic = magic_of(pl.group);
  p.heads_magic = magic_of(cache->heads);
  p.few_rows = kFewRows;
  p.max_tiles = pl.max_tiles;
  p.max_parts = pl.max_parts;
  p.part_rows = pl.part_rows;
  p.flags = shape->flags;
  p.scale_log2 = shape->scale * 1.4426950408889634f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int D = cache->head_dim;
  p.after_prompt = (int64_t)batch->max_q * pl.group > kFewRows && shape->T * pl.group > kFewRows;
  cudaError_t e = p.after_prompt ? launch_attention_prompt(p, D, st) : cudaSuccess;
  if (e == cudaSuccess) e = launch_attention_split(p, D, st);
  if (e == cudaSuccess && p.big_rows) e = launch_attention_prompt_join(p, D, st);
  if (e == cudaSuccess) e = launch_attention_join(p, D, st);
  return cuda_status(e);
}

}  // extern "C"
