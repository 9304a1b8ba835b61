/*
 * invariant_gemm — multi-adapter LoRA shrink / expand with a deterministic
 * Split-K reduction, for NVIDIA GB300 (sm_103a).
 *
 * The operations follow "Reproducible LoRA Inference Through Deterministic
 * Split-K Reduction" (Balusamy & Mohan):
 *   - Eq. 1: a LoRA linear layer computes Y = X W^T + s (X A^T) B^T with
 *     A in R^{r x H} and B in R^{Hout x r}. The shrink is Z = s X A^T (narrow,
 *     r columns); the expand adds Z B^T to Y.
 *   - Eq. 3 / Fig. 1: Split-K partitions the reduction index H into S parts,
 *     one thread block per (output tile, part).
 *   - Algorithm 1 / Fig. 2 / sec. 4.3: each block stores an FP32 partial into
 *     scratch, fences, and bumps a per-tile integer counter; the block that
 *     sees the previous value S-1 sums the S partials in increasing partition
 *     order, multiplies by the scale, writes the tile and resets the counter.
 *   - sec. 4.1: the atomic Split-K baseline adds partials with FP32 atomics.
 *   - sec. 4.2: the unsplit baseline (Split-K = 1) uses one block per tile.
 *   - sec. 4.3: an earlier deterministic design combined the partials in a
 *     separate kernel with a fixed pairwise tree (IG_MODE_DET_TREE).
 *   - sec. 6.2 / Fig. 5: the FP32 shrink output is rounded to BF16
 *     (round-to-nearest, ties to even) where the next operation reads it.
 *
 * Conventions for every entry point:
 *   - All tensor arguments are DEVICE pointers, owned by the caller, and must
 *     stay valid until the work queued on `stream` has finished. The library
 *     allocates no device memory.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream). Every call only enqueues work; none synchronises, except
 *     ig_check_status.
 *   - Layouts are dense row-major with the last index contiguous. bf16 is
 *     IEEE binary32 with the low 16 bits dropped, stored as 2 bytes.
 *       x        bf16  [M][K]
 *       A_stack  bf16  [L][slices][r][K]      (L = num_adapters)
 *       B_stack  bf16  [L][slices][N][r]
 *       z        f32   [slices][M][r]
 *       y        bf16  [M][slices*N]          (updated in place)
 *       adapter_idx int32 [M]; value a in [0, L) selects adapter a, -1 means
 *                the token has no adapter (its z row is 0 and its y row is
 *                left untouched). Any other value is an error: the row is
 *                treated as -1 and the device status word records
 *                IG_ERR_ADAPTER_RANGE (see ig_check_status).
 *   - Every pointer must be 16-byte aligned; K, N and r must be multiples of
 *     8 (so rows are whole 16-byte vectors).
 *   - Return value: IG_OK, or a negative ig_status. Argument errors are
 *     detected on the host before anything is enqueued. IG_ERR_CUDA reports
 *     a failed launch of this call.
 *   - Overlap: shrink and expand kernels are launched with programmatic
 *     dependent launch. A kernel may start while the previous kernel on the
 *     stream finishes, but it reads activations, z, y and the workspace
 *     (other than the token map) and writes anything only after that kernel
 *     has completed; only the token map (which is always complete before any
 *     later kernel starts) and, with IG_FLAG_STATIC_WEIGHTS, A_stack/B_stack
 *     are read earlier.
 *   - Determinism: in IG_MODE_DET, IG_MODE_DET_TREE and IG_MODE_UNSPLIT the
 *     bits of each z row
 *     and y row are a function of that row's inputs, its adapter and the plan
 *     only. The plan (ig_plan_query) is a function of
 *     (K, r, N, slices, split_k, mode, path) and never of M, so results do not
 *     depend on the batch size, the other rows of the batch, the row's
 *     position, or the run. IG_MODE_ATOMIC has no such property.
 */
#ifndef INVARIANT_GEMM_H
#define INVARIANT_GEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define IG_ABI_VERSION 1

typedef enum ig_status {
  IG_OK = 0,
  IG_ERR_ARG = -1,           /* null pointer or invalid enum value */
  IG_ERR_SHAPE = -2,         /* sizes invalid or not divisible as required */
  IG_ERR_ALIGN = -3,         /* a pointer is not 16-byte aligned */
  IG_ERR_WS_SMALL = -4,      /* workspace smaller than ig_workspace_bytes */
  IG_ERR_CUDA = -5,          /* a CUDA runtime call failed */
  IG_ERR_WS_CORRUPT = -6,    /* device: a completion counter held a value >= S */
  IG_ERR_ADAPTER_RANGE = -7, /* device: an adapter index outside [-1, L) */
  IG_ERR_TIMEOUT = -8,       /* device: a bounded wait expired */
  IG_ERR_UNSUPPORTED = -9,   /* valid request outside this build's limits */
  IG_ERR_INDEX_RANGE = -10   /* device: a position, page number or length of
                                the attention calls outside its range */
} ig_status;

/* Reduction variant of the shrink (sec. 4.1-4.3). */
typedef enum ig_mode {
  IG_MODE_DET = 0,     /* Split-K with FP32 partials in the workspace and a
                          last-arriver fixed-order combine (Algorithm 1) */
  IG_MODE_ATOMIC = 1,  /* Split-K with FP32 atomic adds into a zeroed z */
  IG_MODE_UNSPLIT = 2, /* Split-K = 1: one block per output tile */
  IG_MODE_DET_TREE = 3 /* Split-K with FP32 partials in the workspace, summed by
                          a second kernel with a fixed pairwise tree
                          ((P0+P1)+(P2+P3))+...: the earlier deterministic
                          design the pages describe in sec. 4.3 */
} ig_mode;

/* Arithmetic path. It is part of the determinism key: the same request on
 * another path gives results within tolerance but not bit-equal. */
typedef enum ig_path {
  IG_PATH_AUTO = 0,  /* chosen from (K, r, N, slices, flags) only, never
                        from M: IG_PATH_MMA for r >= 32 where it applies,
                        else IG_PATH_WARP */
  IG_PATH_WARP = 1,  /* small ranks: 8-token tiles on the warp-level tensor
                        cores (bf16 mma.sync m16n8k16, FP32 accumulation) */
  IG_PATH_MMA = 2,   /* 128-token tiles on the tcgen05 tensor cores, FP32
                        accumulation in TMEM; needs r and K/S multiples of
                        16, and r <= 192 with IG_FLAG_Z_FP32
                        (IG_ERR_UNSUPPORTED otherwise) */
  IG_PATH_FMA = 3    /* small ranks on CUDA cores: 8-token tiles, FP32 FMA in
                        increasing k per lane, warp-shuffle butterfly across
                        lanes; never chosen by IG_PATH_AUTO (the warp path
                        measured faster), kept as the CUDA-core baseline */
} ig_path;

typedef struct ig_shape {
  int64_t M;            /* tokens: rows of x, z and y; 0 is a valid no-op */
  int64_t K;            /* hidden size H: reduction length of the shrink
                           (< 2^31) */
  int64_t N;            /* output features per slice (Hout, < 2^31) */
  int64_t r;            /* adapter rank */
  int32_t slices;       /* stacked projections that share x, e.g. 3 for QKV */
  int32_t num_adapters; /* L: adapters held in A_stack and B_stack */
  int32_t split_k;      /* S: partitions of K; (K/8) % S == 0. Ignored (1)
                           in IG_MODE_UNSPLIT */
  int32_t mode;         /* ig_mode */
  int32_t path;         /* ig_path */
  int32_t flags;        /* 0 or IG_FLAG_* bits */
} ig_shape;

/* ig_shape.flags bits. */
#define IG_FLAG_STATIC_WEIGHTS 1 /* A_stack and B_stack are not written by any
                                    work still running on `stream` when the
                                    call is enqueued (true for inference
                                    weights). Lets a kernel start reading
                                    them while the previous kernel on the
                                    stream is still finishing. */
#define IG_FLAG_UNFUSED 2        /* IG_MODE_DET combines through the
                                    workspace with the completion counter
                                    (Algorithm 1) even where a cluster
                                    combine applies: lora_apply runs the
                                    Split-K shrink and the expand as two
                                    kernels instead of the fused one-launch
                                    kernel, and the tcgen05 shrink does not
                                    combine inside a thread-block cluster.
                                    Both give the same bits. */
#define IG_FLAG_Z_FP32 4         /* The expand reads Z in FP32 instead of
                                    rounding it to bf16 first (sec. 6.2 shows
                                    the bf16 boundary turning tiny FP32
                                    differences into visible ones). Tensor-
                                    core paths: Z = hi + mid + lo exactly,
                                    hi = bf16_rn(Z), mid = bf16_rn(Z - hi),
                                    lo = bf16_rn(Z - hi - mid), three MMAs
                                    per step of the rank sum; FMA path: Z
                                    used as stored. */

#define IG_FLAG_INPUT_READY 16   /* With IG_FLAG_STATIC_WEIGHTS: x is not written
                                    by any work still running on `stream`
                                    when the call is enqueued (true when x is
                                    the input of a base GEMM that runs just
                                    before the LoRA call, or comes from an
                                    earlier layer). The fused decode kernel
                                    of the warp path (lora_apply with
                                    ig_plan_info.apply_kernels == 1, not
                                    IG_PATH_FMA) then runs its shrink,
                                    partial exchange and combine while the
                                    previous kernel on the stream is still
                                    finishing; z and y are still read and
                                    written only after it has completed.
                                    Other kernels ignore the flag. Same
                                    results; not part of the determinism
                                    key. */
#define IG_FLAG_TEST_COPY_TIMEOUT 8 /* For testing the timeout path only; never
                                    set it in production. Warp-path shrink
                                    kernels (lora_shrink, and lora_apply's
                                    fused kernel) give their first A-copy wait
                                    no time at all: each block checks that
                                    copy once, right after issuing it, finds it
                                    still in flight, records IG_ERR_TIMEOUT,
                                    waits (bounded) for its own copies to land
                                    and leaves. The call's z and y are then
                                    unspecified, and ig_check_status reports
                                    IG_ERR_TIMEOUT and re-zeroes the counters.
                                    Not part of the determinism key. */

/* The resolved plan. Everything that fixes the arithmetic is in
 * determinism_key, which never depends on M. */
typedef struct ig_plan_info {
  int32_t path;             /* IG_PATH_WARP, IG_PATH_MMA or IG_PATH_FMA */
  int32_t split_k;          /* S used (1 for IG_MODE_UNSPLIT) */
  int64_t k_split;          /* K / S: elements per partition */
  int32_t shrink_bm;        /* shrink output tile: token rows ... */
  int32_t shrink_bn;        /* ... x rank columns */
  int32_t expand_bm;        /* expand tile: token rows ... */
  int32_t expand_bn;        /* ... x output columns */
  int64_t shrink_tiles_max; /* upper bound on shrink output tiles for this M */
  int64_t shrink_ctas_max;  /* shrink grid size for this M */
  int64_t workspace_bytes;  /* same as ig_workspace_bytes */
  uint64_t determinism_key; /* hash of the arithmetic-defining plan fields */
  int32_t apply_kernels;    /* kernels lora_apply launches after the token
                               map: 1 = fused shrink+expand (IG_MODE_DET,
                               r = 8 or 16, S <= 16, warp or FMA path), 2 = shrink
                               then expand */
  int32_t reserved;
} ig_plan_info;

/* Library version string and a message for a status code. Host only. */
const char* ig_version(void);
const char* ig_status_string(int status);

/* Bytes of device workspace a call with this shape needs: status word,
 * per-tile completion counters, the token map (rows grouped by adapter),
 * for IG_MODE_DET and IG_MODE_DET_TREE the FP32 partials [tiles][S][BM x BN],
 * and on the tcgen05 path in IG_MODE_DET and IG_MODE_UNSPLIT the expand's Z
 * operand that the shrink of lora_apply writes (bf16 z per tile, slice and
 * bf16 part). Returns 0 for an invalid shape. Host only. */
size_t ig_workspace_bytes(const ig_shape* shape);

/* Resolve the plan for a shape without touching the GPU. IG_OK or an
 * argument error. */
int ig_plan_query(const ig_shape* shape, ig_plan_info* out);

/* Zero the workspace's status word and completion counters (enqueued on
 * stream). Call once after allocating a workspace: afterwards the counters
 * reset themselves (Algorithm 1: the last block writes 0 back). */
int ig_workspace_init(void* ws, size_t ws_bytes, const ig_shape* shape, void* stream);

/* Group the tokens by adapter: a stable counting sort of adapter_idx[0..M)
 * written into the workspace's token map. lora_shrink, lora_expand and
 * lora_apply build the map themselves when given a non-NULL adapter_idx;
 * calling this once and then passing adapter_idx = NULL to several calls
 * with the same M, num_adapters and workspace reuses it (one map per batch,
 * shared by every LoRA layer of a forward pass). Supports num_adapters up to
 * 1023. */
int ig_map_tokens(const ig_shape* shape, const int32_t* adapter_idx,
                  void* ws, size_t ws_bytes, void* stream);

/* Shrink (Eq. 1, Eq. 3, Algorithm 1):
 *   z[sl][m][j] = scale * sum_k x[m][k] * A_stack[a_m][sl][j][k]
 * with FP32 accumulation of exact bf16 x bf16 products. The reduction over k
 * follows shape->mode; in IG_MODE_DET the S partials of a tile are summed in
 * increasing partition order by the last block to finish, then multiplied by
 * scale. IG_MODE_ATOMIC zeroes z (cudaMemsetAsync) and then adds
 * scale * partial with FP32 atomics. adapter_idx may be NULL to reuse the
 * token map already in ws (see ig_map_tokens). */
int lora_shrink(const ig_shape* shape, const void* x, const void* A_stack,
                const int32_t* adapter_idx, float scale, float* z,
                void* ws, size_t ws_bytes, void* stream);

/* Expand (Eq. 1, sec. 6.2):
 *   y[m][sl*N + n] = bf16_rn( f32(y[m][sl*N+n])
 *                             + sum_{j<r} bf16_rn(z[sl][m][j]) * B_stack[a_m][sl][n][j] )
 * (with IG_FLAG_Z_FP32: z[sl][m][j] itself instead of bf16_rn(z); the
 * tensor-core paths feed it as three bf16 parts that sum to it exactly)
 * The sum over j is an FP32 sum whose order is fixed by r and the path, not
 * by M: on the tensor-core paths (IG_PATH_WARP, IG_PATH_MMA) the rank axis
 * is taken in chunks of 16 in increasing order, one MMA per chunk, each
 * adding its 16 products into the FP32 accumulator inside the tensor core;
 * on IG_PATH_FMA a sequential FMA chain in increasing j. y is rounded once.
 * Rows with adapter -1 are not written. adapter_idx may be NULL to reuse the
 * token map in ws. */
int lora_expand(const ig_shape* shape, const float* z, const void* B_stack,
                const int32_t* adapter_idx, void* y,
                void* ws, size_t ws_bytes, void* stream);

/* Token map (if adapter_idx != NULL), shrink into z, then expand into y, all
 * on `stream`. z is caller-owned scratch of slices*M*r floats and holds the
 * shrink output afterwards. In IG_MODE_DET with r = 8 or 16 and S <= 16 the
 * shrink and expand run as one launch: the S partition blocks of a tile form
 * a thread-block cluster, sum their partials over distributed shared memory
 * in the same increasing partition order, and expand the tile's rows
 * (ig_plan_info.apply_kernels == 1; IG_FLAG_UNFUSED turns this off). On
 * the tcgen05 path (IG_PATH_MMA) in IG_MODE_DET and IG_MODE_UNSPLIT the
 * shrink also writes the expand's bf16 Z operand into ws, the expand copies
 * it instead of building it from z, and it starts its first y copies before
 * its dependency wait (the shrink writes no y). The results are
 * bit-identical to lora_shrink followed by lora_expand. */
int lora_apply(const ig_shape* shape, const void* x, void* y,
               const int32_t* adapter_idx, const void* A_stack,
               const void* B_stack, float scale, float* z,
               void* ws, size_t ws_bytes, void* stream);

/* lora_shrink without a caller-provided workspace. The paper has no
 * counterpart: it exists for callers that cannot allocate device memory
 * where they run the shrink (code that must not risk the device-wide
 * synchronisation an allocation can bring, runtimes that plan all memory
 * ahead and give libraries no allocator, plugin hosts that own every
 * allocation).
 *
 * Same arguments, arithmetic and results as lora_shrink (adapter_idx must be
 * non-NULL), but the token map, counters, status word and partials live in
 * a 4 MiB array inside the library, held by every GPU that loads it until
 * the process exits. This call allocates nothing: no cudaMalloc, no
 * cudaFree, no allocating library routine.
 *   - Shapes whose shrink needs more than 4 MiB of workspace are rejected
 *     with IG_ERR_WS_SMALL before anything is enqueued. That is
 *     ig_workspace_bytes without the expand's Z operand, which only
 *     lora_apply writes.
 *   - The first call on a device looks up the array's device address (with
 *     that device current). Make that first call before any stream capture.
 *   - Every call shares the one array and it keeps the previous call's
 *     contents; each call clears the status word and the counters it uses
 *     (a memset on `stream`). Calls that overlap on the GPU (other streams,
 *     other threads) race on the array and give wrong results: serialise
 *     them.
 *   - Device-side status (out-of-range adapter index, expired wait) is not
 *     reported; validate adapter_idx beforehand. */
int lora_shrink_noalloc(const ig_shape* shape, const void* x, const void* A_stack,
                        const int32_t* adapter_idx, float scale, float* z, void* stream);

/* ------------------------------------------------------------------------
 * The block around the adapters: MX4 weights and activations, and the norms.
 *
 * A served layer is  y = x W^T + s (x A^T) B^T  between two norms. lora_apply
 * adds the adapter term to a y that is already there; these calls make x, the
 * quantised W and that y, and take y up into the residual stream. As with the
 * LoRA calls, the bits of a row depend on that row, the weights and the sizes
 * (K, N; H) only: never on M, the other rows, the row's place or the run.
 *
 * MX4: a matrix [rows][K] with the product's reduction along K, K a multiple
 * of 32. Each 32 values of a row share one scale, held as an E8M0 byte b: the
 * value 2^(b - 127), 255 = NaN. A value is a 4-bit E2M1 float: 0, 0.5, 1, 1.5,
 * 2, 3, 4, 6 (codes 0-7) and their negatives (codes 8-15).
 *   codes   uint8 [rows][K/2], the even k in bits 0-3, the odd k in bits 4-7
 *   scales  uint8, ig_mx4_scale_bytes(rows, K) bytes: tiles of 512 bytes, one
 *           per 128 rows x 128 k, tile (row / 128) * ceil(K / 128) + k / 128;
 *           in a tile the byte of a block is at
 *           (row % 32) * 16 + (row / 32 % 4) * 4 + k / 32 % 4.
 *           Scale bytes of blocks past K are written as 127 by the calls
 *           below and must be finite; those of rows past the last are
 *           neither written nor of any effect.
 * These calls keep the conventions above (device pointers, 16-byte alignment,
 * enqueue only, argument errors before anything is enqueued); pointers and
 * stream belong to the current GPU; row strides (ld_*) are in elements and
 * multiples of 8. An operator with no rows is a no-op.
 * ------------------------------------------------------------------------ */
typedef enum ig_type { IG_TYPE_BF16 = 0, IG_TYPE_F32 = 1 } ig_type;

/* Bytes of the scales of a [rows][K] MX4 matrix; 0 for an invalid size. */
size_t ig_mx4_scale_bytes(int64_t rows, int64_t K);

/* x [rows][K] (bf16 or FP32) -> MX4. For a block with largest magnitude a the
 * scale is 2^e, e = max(floor(log2 a) - 2, -127); each value is divided by it
 * (exactly), rounded to the nearest E2M1 value, ties to the even code, and
 * held at +-6 (magnitudes between 6 and 8 times the scale, at most a quarter
 * off). A block that holds an infinity or a NaN gets the scale 255: all of it
 * reads as NaN. */
int ig_mx4_quantize(int64_t rows, int64_t K, const void* x, int64_t ld_x, int x_type,
                    void* codes, void* scales, void* stream);

/* The values an MX4 matrix stands for, rounded to the type of out
 * [rows][K]. Every value ig_mx4_quantize can produce is exact in bf16. */
int ig_mx4_dequantize(int64_t rows, int64_t K, const void* codes, const void* scales, void* out,
                      int64_t ld_out, int out_type, void* stream);

typedef struct ig_mx4_shape {
  int64_t M;      /* tokens: rows of x and y */
  int64_t N;      /* output features: rows of w (a multiple of 8) */
  int64_t K;      /* reduction length (a multiple of 32) */
  int64_t ld_y;   /* row stride of y */
  int32_t y_type; /* ig_type */
  int32_t flags;  /* 0, IG_FLAG_STATIC_WEIGHTS (w_codes and w_scales may be read
                     before earlier work on the stream has ended; products of
                     many tokens do not make use of it) and, for
                     tests only, IG_FLAG_TEST_COPY_TIMEOUT: the first wait for a
                     copy expires in every block, nothing is stored for its
                     tile and the status becomes IG_ERR_TIMEOUT */
} ig_mx4_shape;

/* Bytes of the workspace of ig_mx4_gemm: the status word and counters that a
 * workspace begins with (see ig_workspace_init, ig_check_status). Any
 * initialised workspace of the LoRA calls serves as it is; one of its own is
 * these bytes, zeroed once. */
size_t ig_mx4_workspace_bytes(void);

/* y[m][n] = sum_k x[m][k] w[n][k], x [M][K] and w [N][K] in MX4: exact
 * products, FP32 sums, one rounding to the type of y. A NaN scale makes the
 * rows (of x) or columns (of w) that it touches NaN. */
int ig_mx4_gemm(const ig_mx4_shape* shape, const void* x_codes, const void* x_scales,
                const void* w_codes, const void* w_scales, void* y, void* ws, size_t ws_bytes,
                void* stream);

#define IG_NORM_WEIGHT_PLUS_ONE 1 /* norm weights are stored as w - 1 */

typedef struct ig_norm_shape {
  int64_t M;               /* rows */
  int64_t H;               /* features: a multiple of 8, at most 32768 */
  int64_t ld_h, ld_y, ld_h_out, ld_n; /* row strides of what is given */
  int64_t gate_row_stride; /* 0: the same gate for every row */
  int32_t gate_col_stride; /* 1, or 0: one gate value per row (then
                              gate_row_stride may be any, and gate any
                              address of a bf16 value) */
  int32_t h_type;          /* ig_type of h and h_out */
  int32_t flags;           /* 0 or IG_NORM_WEIGHT_PLUS_ONE */
  float eps;               /* >= 0 */
  float scale;             /* residual scale */
} ig_norm_shape;

/* The norm after a block, its gate and residual scale, and the norm before
 * the next block, in one pass over the row:
 *   t  = y * rsqrt(mean(y^2) + eps) * w_post       (w_post NULL: t = y)
 *   h' = h + scale * gate * t                      (gate NULL: 1; h NULL: 0;
 *                                                   y NULL: h' = h)
 *   n  = h' * rsqrt(mean(h'^2) + eps) * w_pre
 * in FP32; h' goes to h_out (h_type; NULL: not wanted) and n, which is
 * computed from the FP32 h', to n_out (bf16; NULL: not wanted). codes and
 * scales (both or neither; H a multiple of 32) receive the bf16 n in MX4, the
 * same bits as ig_mx4_quantize of n_out. w_pre is given if and only if one of
 * n_out and codes is. y, gate, w_post and w_pre are bf16. h_out may be h, and
 * n_out may be y (same strides). */
int ig_block_norm(const ig_norm_shape* shape, const void* h, const void* y, const void* gate,
                  const void* w_post, const void* w_pre, void* h_out, void* n_out, void* codes,
                  void* scales, void* stream);

/* ------------------------------------------------------------------------
 * The attention of a served layer: head norms with the position rotation, a
 * paged key/value cache held in 8 bits, and attention over it. These calls
 * take the q, k and v that the stacked projections (slices = 3) leave and make
 * the input of the output projection.
 *
 * Tokens of a batch are stacked; sequence b has the rows cu[b] .. cu[b+1] - 1
 * and they are its last ones: positions kv_len[b] - rows .. kv_len[b] - 1.
 * Rows that belong to no sequence are neither read nor written. Token j of
 * sequence b is in row j % page of the page page_table[b][j / page].
 *
 * Cache, for each page, side (0 keys, 1 values) and kv head:
 *   codes   uint8 [pages][2][heads][page][head_dim], e4m3: sign, 4 exponent and
 *           3 mantissa bits, largest 448, 0x7f and 0xff NaN, no infinities
 *   scales  uint8 [pages][2][heads][page / 16]: 16 tokens of a head (a block)
 *           share the scale 2^(byte - 127); 255 = NaN
 * Pages may lie further apart than they are long (page_stride, scale_stride);
 * what is inside a page is dense.
 *
 * These calls keep the conventions above; pointers and stream belong to the
 * current GPU. q, k, v and their outputs are bf16 [T][heads][head_dim] with a
 * stride of ld_* elements (a multiple of 8) between tokens, so they may be
 * columns of one buffer. head_dim is 64 or 128. A sequence whose cu, kv_len or
 * page count is out of range (rows outside [0, T), more than max_q of them
 * where the call has one, kv_len beyond ld_table pages) is left out of the
 * call, tokens on pages outside [0, pages) are taken as absent, and the status
 * word of ws records IG_ERR_INDEX_RANGE. ws is any initialised workspace of the
 * library (ig_mx4_workspace_bytes() zeroed bytes will do), but for
 * ig_paged_attention, which says how much it needs.
 *
 * The bits of a row of q, k, v and of the attention's output depend on that
 * row, its sequence (kv_len, number of new tokens, cache content) and the sizes
 * of heads and pages only: never on the other sequences, the sequence's place
 * in the batch, the pages it is on or the run.
 * ------------------------------------------------------------------------ */
#define IG_ROPE_INTERLEAVED 2 /* rotated pairs are neighbours (x[2i], x[2i+1]);
                                 otherwise (x[i], x[i + rot_dim / 2]) */

typedef struct ig_rope_shape {
  int64_t T;               /* tokens */
  int64_t table_rows;      /* positions that cos_sin holds */
  int64_t ld_q, ld_k, ld_q_out, ld_k_out; /* strides of what is given */
  int32_t heads_q, heads_k;
  int32_t head_dim;        /* 64 or 128 */
  int32_t rot_dim;         /* values rotated, the first of each head: a multiple
                              of 16, at most head_dim */
  int32_t flags;           /* 0, IG_NORM_WEIGHT_PLUS_ONE, IG_ROPE_INTERLEAVED */
  float eps;               /* >= 0 */
} ig_rope_shape;

typedef struct ig_kv_cache {
  void* codes;
  void* scales;
  int64_t pages;
  int64_t page_stride;     /* bytes between pages of codes (a multiple of 16) */
  int64_t scale_stride;    /* bytes between pages of scales */
  int32_t page;            /* tokens to a page: 16, 32, 64, 128 or 256 */
  int32_t heads;           /* kv heads */
  int32_t head_dim;
  int32_t reserved;        /* 0 */
} ig_kv_cache;

typedef struct ig_batch {
  const int32_t* cu;         /* [batch + 1], not falling (where it falls, rows of the
                                sequences around are unspecified) */
  const int32_t* kv_len;     /* [batch] tokens in all, the new ones among them */
  const int32_t* page_table; /* [batch][ld_table] */
  int64_t ld_table;          /* pages that a row of page_table can name */
  int32_t batch;
  int32_t max_q;             /* no sequence has more new tokens than this */
} ig_batch;

/* Norms of queries and keys for each head and the position rotation, in one
 * pass, in FP32 with one rounding:
 *   n = x * rsqrt(mean(x^2) + eps) * w               (w NULL: n = x)
 *   (n1, n2) -> (n1 cos - n2 sin, n2 cos + n1 sin)    (cos_sin NULL: as it is)
 * for the rot_dim / 2 pairs, with the cosines cos_sin[p][0 .. rot_dim/2) and the
 * sines cos_sin[p][rot_dim/2 .. rot_dim) of the token's position p
 * (cos_sin FP32 [table_rows][rot_dim], positions int32 [T]). q or k may be NULL,
 * with their outputs. q_out may be q and k_out may be k (same strides). A token
 * whose position is outside the table gets NaN, and ws records
 * IG_ERR_INDEX_RANGE. w_q and w_k are bf16 [head_dim]. */
int ig_qk_norm_rope(const ig_rope_shape* shape, const void* q, const void* k, const void* w_q,
                    const void* w_k, const float* cos_sin, const int32_t* positions, void* q_out,
                    void* k_out, void* ws, size_t ws_bytes, void* stream);

/* Keys and values of the new tokens into the cache, keys (and q, where given,
 * into q_out) normed and rotated as by ig_qk_norm_rope; positions NULL: the
 * token's place in its sequence. Quantised from FP32: a block's scale is the
 * smallest 2^e, e >= -120, with max|value| <= 448 2^e over the finite values of
 * its new tokens; where older tokens of the sequence are in the block it is at
 * least their scale, and where it grew they are divided by as much. Values are
 * rounded to nearest, ties to even (keys of 2^-6 scale or more that FP32 cannot
 * tell from the middle between two codes by their FP64 values; smaller keys, and the
 * largest one for the scale, as FP32 has them); what is not finite is held as NaN.
 * Rows of the block behind the last token keep their bytes.
 * A block that is written must be one token range of one sequence: not shared
 * by two sequences, nor on a page that the page table names twice (its bytes are
 * unspecified otherwise; pages that are only read may be shared freely).
 * Tokens appended one by one and together get the same scales, and the same
 * codes but for values under 2^-6 scale, which a growing scale rounds again.
 * k and v have batch->cu's rows of shape->T; ld_k is the stride of k. */
int ig_kv_append(const ig_rope_shape* shape, const ig_kv_cache* cache, const ig_batch* batch,
                 const void* k, const void* v, int64_t ld_v, const void* q, const void* w_q,
                 const void* w_k, const float* cos_sin, const int32_t* positions, void* q_out,
                 void* ws, size_t ws_bytes, void* stream);

/* What the cache holds, as bf16 (exact but for what bf16 cannot hold: values
 * under 2^-126): row cu[b] + i of k_out and v_out [T][heads][head_dim] is token
 * kv_len[b] - rows + i of sequence b. max_q is not looked at. Rows of tokens
 * before the sequence's first (more rows than kv_len) are written as 0, of
 * absent tokens as NaN. */
int ig_kv_gather(const ig_kv_cache* cache, const ig_batch* batch, int64_t T, void* k_out,
                 int64_t ld_k_out, void* v_out, int64_t ld_v_out, void* ws, size_t ws_bytes,
                 void* stream);

typedef struct ig_attn_shape {
  int64_t T;               /* rows of q and out */
  int64_t ld_q, ld_out;
  int32_t heads_q;         /* a multiple of the cache's heads: query head h reads
                              kv head h / (heads_q / heads) */
  int32_t flags;           /* 0 or, for tests only, IG_FLAG_TEST_COPY_TIMEOUT: every
                              block acts as if its first wait for a copy had
                              expired; out is then unspecified and the status
                              IG_ERR_TIMEOUT */
  float scale;             /* of the products, usually 1 / sqrt(head_dim) */
  int32_t reserved;        /* 0 */
} ig_attn_shape;

/* Bytes of workspace of ig_paged_attention for these sizes (of batch: batch,
 * max_q and ld_table; of cache: page, heads and head_dim); 0 for invalid ones.
 * Enough for every call with fewer tokens, sequences, pages or a smaller max_q.
 * Zeroed once after it is allocated; calls that may overlap, captured ones too,
 * need one each. The library's other calls may share it where they do not overlap;
 * a token map in it does not outlive ig_paged_attention. After IG_ERR_CUDA of a call
 * it has to be zeroed again. */
size_t ig_attention_workspace_bytes(const ig_attn_shape* shape, const ig_kv_cache* cache,
                                    const ig_batch* batch);

/* Attention of the new tokens over the cache, causal at the sequence's end:
 *   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j),
 * over the tokens j <= kv_len - rows + i for row i of a sequence's `rows`. Rows
 * that see no token (rows > kv_len) are 0. Products of the held values in
 * the tensor cores with FP32 sums, softmax in FP32; for the product with the codes of
 * v, p times v's scale is rounded to 11 bits or to 2^-32 of the row's largest such product,
 * whichever is more (scales under 2^-120 of the largest up to the row's step of 128 tokens
 * count as that). A sequence of at most 64 rows a kv head (rows times heads_q / heads) is
 * one kernel's, which takes the values of a query under 2^-31 of its largest to within
 * 2^-39 of it, of more another's: under 2^-9, 2^-17. out may not be q, nor
 * overlap what the call reads. */
int ig_paged_attention(const ig_attn_shape* shape, const ig_kv_cache* cache,
                       const ig_batch* batch, const void* q, void* out, void* ws,
                       size_t ws_bytes, void* stream);

/* Synchronise `stream`, read and clear the workspace status word, and return
 * the most severe device-side error recorded since the last check
 * (IG_ERR_TIMEOUT, IG_ERR_WS_CORRUPT, IG_ERR_ADAPTER_RANGE,
 * IG_ERR_INDEX_RANGE) or IG_OK. After
 * IG_ERR_WS_CORRUPT or IG_ERR_TIMEOUT the completion counters are zeroed
 * again, so the workspace is usable for the next call. After IG_ERR_TIMEOUT
 * the z and y written by the calls since the last check are unspecified
 * (a block whose wait expired contributed nothing, or zeros); every block
 * still waited, bounded, for its own copies before it left. */
int ig_check_status(void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* INVARIANT_GEMM_H */
