/*
 * llsa.h -- C ABI of the B200 (sm_100a) implementation of Log-linear Sparse
 * Attention (LLSA) for pixel-space diffusion transformers.
 *
 * The method (cited by page title and section):
 *   [LLSA] "Trainable Log-linear Sparse Attention for Efficient Diffusion
 *          Transformers" (CVPR 2026), technical summary page: §三 hierarchical
 *          top-K, §四 hierarchical KV enrichment and KV reweighting, §4.1
 *          sparse backward, §4.2 / Fig. 2 index reordering.
 *   [ART]  popular write-up of arXiv:2512.16615, §三 (hierarchical selection,
 *          weight = block size of the level) and §四 (sparse-index forward,
 *          CSR->CSC index transpose, reordering).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * * Tensors are caller-owned DEVICE buffers, contiguous, 16-byte aligned.
 *   Token tensors are [batch, heads, N, d] with N = height * width, element
 *   type `dtype` (bf16 or fp32).  Every call except llsa_reorder takes them in
 *   HIERARCHICAL token order (see llsa_reorder).
 * * Level l = 1..L holds n_l = N / B^l pooled tokens.  Index lists have
 *   K_L = min(K, n_L) entries per token at the coarsest level and
 *   K_l = min(K, K_{l+1} * B) at finer levels ([LLSA] §三).
 * * Level-packed buffers hold level 1 first, then level 2, ...; inside a level
 *   the layout is [batch*heads][n_l][...].  Sizes come from llsa_query_sizes:
 *     pyramid   fp32  [BH][n_l][d]         per level
 *     idx       int32 [BH][n_l][K_l]       per level, each list ascending
 *     offs      int32 [BH][n_l + 1]        per level (CSC offsets)
 *     qlist     int32 [BH][n_l * K_l]      per level (CSC query ids, ascending per key)
 * * The library allocates nothing and keeps no state between calls; calls are
 *   asynchronous on `stream` (a cudaStream_t; NULL = legacy default stream).
 * * Host-detectable errors (bad shapes, NULL or misaligned pointers,
 *   unsupported sizes) return a status before anything is launched.  A
 *   launch failure returns LLSA_ERR_CUDA.  No exception crosses the ABI.
 * * Buffer sizes are queried with llsa_query_sizes (one call returns every
 *   size, the workspaces included); device-side timeouts are read with
 *   llsa_device_error.  The main entry points take no size arguments: their
 *   buffers must have the queried sizes.  LLSA_ERR_WORKSPACE is returned only
 *   by llsa_index_transpose_noalloc, whose scratch has a fixed size.
 * * Pooled tokens: pyrK / pyrV passed to the attention calls must be what
 *   llsa_pool wrote for the same k / v.  Level 1 is then the exact mean of
 *   the B key (value) rows it stands for, and the tensor-core kernels (bf16,
 *   d = 64, B = 16) use that identity: they form level-1 pooled logits and
 *   values from k / v themselves and do not read level 1 of pyrK / pyrV.  The
 *   CUDA-core kernels (every other problem) read it.  Levels >= 2 are read by
 *   both.
 */
#ifndef LLSA_H
#define LLSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Binary-compatible with cudaStream_t; no CUDA header needed to include this file. */
typedef struct CUstream_st* llsa_stream;

typedef enum {
  LLSA_OK = 0,
  LLSA_ERR_ARG = 1,          /* NULL pointer or invalid field */
  LLSA_ERR_SHAPE = 2,        /* image does not tile into sqrt(B)^L squares, or sizes overflow */
  LLSA_ERR_ALIGN = 3,        /* a buffer is not 16-byte aligned */
  LLSA_ERR_WORKSPACE = 4,    /* the fixed scratch of llsa_index_transpose_noalloc is too small */
  LLSA_ERR_CUDA = 5,         /* a CUDA launch or runtime call failed */
  LLSA_ERR_TIMEOUT = 6,      /* a bounded device-side wait gave up (see llsa_device_error) */
  LLSA_ERR_UNSUPPORTED = 7   /* valid problem outside what the kernels implement */
} llsa_status;

typedef enum { LLSA_BF16 = 0, LLSA_FP32 = 1 } llsa_dtype;

#define LLSA_MAX_LEVELS 12

typedef struct {
  int batch, heads;       /* independent (batch, head) slices */
  int height, width;      /* image size in pixels; N = height * width tokens */
  int d;                  /* head dimension (multiple of 8, at most 128) */
  int B;                  /* block size, a perfect square B = t * t, t >= 2 */
  int L;                  /* pooled levels, 1 <= L <= LLSA_MAX_LEVELS; height and width divisible by t^L */
  int K;                  /* top-K per level; K >= number of candidates keeps all of them */
  unsigned enrich_mask;   /* bit (l-1) set: level-l coarse K/V join the attention ([LLSA] §四) */
  float scale;            /* softmax scale; 0 selects 1/sqrt(d) */
  int dtype;              /* llsa_dtype of Q, K, V, O, dO, dQ, dK, dV */
} llsa_problem;

typedef struct {
  size_t tokens_bytes;              /* one [BH][N][d] tensor of `dtype` */
  size_t lse_bytes;                 /* fp32 [BH][N] */
  size_t pyramid_bytes;             /* one fp32 pyramid, levels 1..L */
  size_t idx_bytes;                 /* int32 index lists, all levels */
  size_t offs_bytes;                /* int32 CSC offsets, all levels */
  size_t qlist_bytes;               /* int32 CSC query ids, all levels */
  size_t transpose_scratch_bytes;   /* scratch for llsa_index_transpose */
  size_t bwd_workspace_bytes;       /* workspace for llsa_attn_bwd */
} llsa_sizes;

/* Human-readable name of a status. */
const char* llsa_status_string(llsa_status s);

/* Checks every field of *p; no launch.  LLSA_OK, LLSA_ERR_ARG, LLSA_ERR_SHAPE or
 * LLSA_ERR_UNSUPPORTED. */
llsa_status llsa_validate(const llsa_problem* p);

/* n[0..L] (tokens per level, n[0] = N) and Kl[0..L] (list length per level,
 * Kl[0] = 0).  Host memory, L+1 entries each. */
llsa_status llsa_level_sizes(const llsa_problem* p, int64_t* n, int64_t* Kl);

/* Byte sizes of every buffer the entry points take. */
llsa_status llsa_query_sizes(const llsa_problem* p, llsa_sizes* out);

/* Index reordering ([ART] §四; [LLSA] §4.2, Fig. 2).  Moves token rows between
 * raster order (row y*W + x) and hierarchical order: recursive sqrt(B) x sqrt(B)
 * tiles, row-major inside every tile and row-major over the top grid of
 * t^L x t^L squares, so that every aligned run of B^l hierarchical positions
 * is one t^l x t^l pixel square:
 *   hier(y,x) = (floor(y/t^L)*(W/t^L) + floor(x/t^L)) * B^L
 *             + sum_{l=1..L} ((floor(y/t^(l-1)) mod t)*t + floor(x/t^(l-1)) mod t) * B^(l-1).
 * in, out: [BH][N][d] of dtype; to_hier != 0 maps raster -> hierarchical,
 * 0 maps back.  in and out must not overlap. */
llsa_status llsa_reorder(const llsa_problem* p, const void* in, void* out, int to_hier, llsa_stream stream);

/* Hierarchical compression ([LLSA] §三): P_l[j] = mean of P_{l-1}[j*B .. j*B+B-1],
 * l = 1..L, P_0 = x.  x: hierarchical [BH][N][d] of dtype; pyramid: fp32, level
 * packed, pyramid_bytes.  Call once each for Q, K and V. */
llsa_status llsa_pool(const llsa_problem* p, const void* x, float* pyramid, llsa_stream stream);

/* Coarse-to-fine top-K selection ([LLSA] §三; [ART] §三).  Level L: every
 * level-L query token scores all n_L level-L keys.  Level l < L: query token a
 * scores only the B children of each pick of its parent floor(a/B) at level
 * l+1.  Score = pooled q . pooled k in fp32; the K_l best are kept (higher
 * score first, lower key id on equal scores) and stored ascending.
 * pyrQ, pyrK: pyramids from llsa_pool; idx: idx_bytes, all levels written. */
llsa_status llsa_select(const llsa_problem* p, const float* pyrQ, const float* pyrK, int32_t* idx,
                        llsa_stream stream);

/* One level of llsa_select: reads the level-(level+1) lists already in idx
 * (when level < L) and writes the level-`level` lists only. */
llsa_status llsa_select_level(const llsa_problem* p, int level, const float* pyrQ, const float* pyrK,
                              int32_t* idx, llsa_stream stream);

/* Sparse attention forward with hierarchical KV enrichment ([LLSA] §四;
 * [ART] §三, §四).  Fine query i (block a = floor(i/B)) attends to
 *   the B tokens of each level-1 block in S_1(a), logit scale * q.k, and
 *   for every level l set in enrich_mask the pooled tokens S_l(floor(i/B^l))
 *   of pyrK/pyrV, logit scale * q.P^K_l + ln(B^l)  (weight B^l).
 * Keys are gathered by index; no mask is built.
 * q, k, v: hierarchical [BH][N][d] of dtype; pyrK, pyrV: pyramids of K and V;
 * idx: from llsa_select; o: [BH][N][d] of dtype; lse: fp32 [BH][N], natural log
 * of the softmax denominator (with the weights). */
llsa_status llsa_attn_fwd(const llsa_problem* p, const void* q, const void* k, const void* v,
                          const float* pyrK, const float* pyrV, const int32_t* idx, void* o, float* lse,
                          llsa_stream stream);

/* Sparse index transpose, CSR -> CSC ([ART] §四; [LLSA] §4.1), every level:
 * per-key counts (warp-aggregated atomics), exclusive prefix sum into offs,
 * scatter of the query ids into qlist, each key's ids ascending.
 * scratch: transpose_scratch_bytes of device memory, contents ignored. */
llsa_status llsa_index_transpose(const llsa_problem* p, const int32_t* idx, int32_t* offs, int32_t* qlist,
                                 void* scratch, llsa_stream stream);

/* llsa_index_transpose without a scratch argument.  The pages have no
 * counterpart to this entry point; it exists for callers that cannot obtain
 * device memory at the point where they run the transpose -- for example a
 * plug-in whose host framework owns every device allocation and exposes no
 * allocator to it, or a latency-critical loop that must never call
 * cudaMalloc (which can synchronize the device).  Those callers still pass
 * idx, offs and qlist, but no scratch: the scratch lives in a fixed 16 MiB
 * device array inside this library (every GPU that loads the library holds
 * it until the process exits).  A problem whose transpose needs more than
 * that (transpose_scratch_bytes > 16 MiB) is rejected with
 * LLSA_ERR_WORKSPACE before anything is launched.  Nothing is allocated:
 * no cudaMalloc, no cudaFree.
 * Every call looks up the array's device address on the current device
 * (cudaGetSymbolAddress, a host-side lookup that launches nothing), so a
 * device reset between calls leaves no stale address behind.  The first call
 * on a device may load this library's device code there; make it before any
 * stream capture.  All calls share the one array and it
 * keeps whatever the last call left there (the parts that must start at zero
 * are cleared by every call), so two calls whose work overlaps on the GPU --
 * on different streams, or from different threads -- race and must be
 * serialized by the caller.  Results are identical to llsa_index_transpose. */
llsa_status llsa_index_transpose_noalloc(const llsa_problem* p, const int32_t* idx, int32_t* offs,
                                         int32_t* qlist, llsa_stream stream);

/* Sparse attention backward ([LLSA] §4.1), index lists held fixed.  With
 * P = exp(z - lse) and D_i = dO_i . o_i:  dq_i = scale * sum_j P_ij (dO_i.v_j - D_i) k_j;
 * fine keys gather their queries through the level-1 CSC lists (offs, qlist);
 * pooled keys accumulate into fp32 level gradients that are sent back to the
 * B^l tokens they average (dk_t += dPK_l[floor(t/B^l)] / B^l, the same for v).
 * Pooled Q receives no gradient.  o, lse: from llsa_attn_fwd; dO: upstream
 * gradient; dq, dk, dv: [BH][N][d] of dtype, fully written; workspace:
 * bwd_workspace_bytes of device memory, contents ignored. */
llsa_status llsa_attn_bwd(const llsa_problem* p, const void* q, const void* k, const void* v,
                          const void* o, const void* dO, const float* lse, const float* pyrK,
                          const float* pyrV, const int32_t* idx, const int32_t* offs, const int32_t* qlist,
                          void* dq, void* dk, void* dv, void* workspace, llsa_stream stream);

/* Which kernels llsa_attn_fwd and llsa_attn_bwd run for *p (host only, no
 * launch): *fwd_tc / *bwd_tc = 1 for the tensor-core kernels (tcgen05 /
 * TMEM, bf16, d = 64, B = 16, within the sizes they support), 0 for the
 * CUDA-core kernels.  Either pointer may be NULL. */
llsa_status llsa_attn_paths(const llsa_problem* p, int* fwd_tc, int* bwd_tc);

/* Number of CUDA kernels this library has launched in this process so far
 * (all entry points, all streams); for accounting in benchmarks. */
uint64_t llsa_kernel_launches(void);

/* Waits for `stream`, then reads and clears the device-side error word that
 * bounded waits inside the kernels set when they give up.  *code = 0 when no
 * wait gave up; returns LLSA_ERR_TIMEOUT when one did.  There is one word
 * per device, shared by every stream and thread of the process: a code
 * cannot be attributed to one stream, and a read clears it for all. */
llsa_status llsa_device_error(llsa_stream stream, int* code);

/* Self-test of the timeout path of the bounded device waits: launches one
 * thread on `stream` that waits, with the same bounded wait the pipelined
 * kernels use, on an mbarrier phase that nothing completes (arrive = 0) or
 * that it completed itself first (arrive = 1).  When the wait gives up after
 * limit_us microseconds the device error word is set to `code`, so that the
 * next llsa_device_error returns LLSA_ERR_TIMEOUT with *code = code; with
 * arrive = 1 it stays 0.  Neither faults nor hangs the GPU.  limit_us in
 * [1, 1000000], code != 0, arrive in {0, 1}, else LLSA_ERR_ARG before any
 * launch. */
llsa_status llsa_selftest_wait_timeout(unsigned limit_us, int code, int arrive, llsa_stream stream);

/* ------------------------------------------------------------------------
 * Around the self-attention of a conditional diffusion transformer: cross
 * attention to an encoder's states, and layer norm.
 *
 * These calls take token tensors [batch][heads][tokens][d] with element
 * strides per batch row, head and token (the channels of a token are
 * contiguous), so that slices of a projection's output are used in place.  A
 * llsa_strides of zeros means the contiguous layout above.  An input may
 * repeat itself (a stride of 0); tensors that are written may not overlap
 * themselves (LLSA_ERR_ARG), nor any other argument unless a call says so.
 * The buffers of cross attention and all workspaces are 16-byte aligned (a
 * workspace that is given is checked even where the call has no use for it);
 * the tensors of layer norm need their element's alignment only (with 16 bytes,
 * and widths and strides that are multiples of 8 elements, it is faster).
 * The conventions at the top of this file hold otherwise: asynchronous on
 * `stream`, on the current device, which owns every buffer; nothing is
 * allocated and nothing kept.  A workspace may be used by one call at a time
 * (give each graph that replays concurrently its own); its contents are
 * ignored on entry.  Calls give the same bits every time.
 * ---------------------------------------------------------------------- */

typedef struct {
  int64_t batch, head, token;   /* in elements */
} llsa_strides;

/* Cross attention: `nq` queries per head and batch row attend to the `nk`
 * states of an encoder; at most LLSA_CROSS_MAX_TOKENS of each, and four times as
 * many queries in the heads that share a key head (a head's 128 or more counted
 * in whole tiles of 128). */
#define LLSA_CROSS_MAX_TOKENS (1 << 24)

typedef struct {
  int batch, heads;       /* of the queries */
  int kv_heads;           /* of keys and values; divides heads: query head h reads key head h / (heads / kv_heads) */
  int nq, nk;
  int d;                  /* head dimension (multiple of 8, at most 128) */
  float scale;            /* softmax scale; 0 selects 1/sqrt(d) */
  int dtype;              /* llsa_dtype of q, k, v, o and of their gradients */
  /* strides: multiples of 8 elements (bf16) or 4 (fp32) */
  llsa_strides q, k, v, o, d_o, dq, dk, dv;
} llsa_cross_problem;

typedef struct {
  size_t lse_bytes;               /* fp32 [batch][heads][nq] */
  size_t fwd_workspace_bytes;     /* may be 0: then the workspace may be NULL */
  size_t bwd_workspace_bytes;
} llsa_cross_buffers;

/* Checks every field of *p; no launch. */
llsa_status llsa_cross_validate(const llsa_cross_problem* p);

/* Byte sizes of lse and of the workspaces; they depend on the sizes and types
 * in *p, not on its strides. */
llsa_status llsa_cross_query_sizes(const llsa_cross_problem* p, llsa_cross_buffers* out);

/* o_i = sum_j softmax_j(scale q_i . k_j) v_j over the batch row's valid keys,
 * lse_i = log sum_j exp(scale q_i . k_j).  Key j of batch row b is valid when
 * j < kv_len[b] and key_mask[b][j] != 0.  kv_len: int32 [batch] in device
 * memory, 4-byte aligned, clamped to 0..nk, or NULL (all nk); key_mask: uint8
 * [batch][nk] in device memory, or NULL (none masked).  k and v at keys that
 * are not valid are never used, whatever they hold.  Without a valid key
 * o = 0 and lse = -inf.  lse may be NULL. */
llsa_status llsa_cross_attn_fwd(const llsa_cross_problem* p, const void* q, const void* k, const void* v,
                                const int32_t* kv_len, const uint8_t* key_mask, void* o, float* lse,
                                void* workspace, llsa_stream stream);

/* Gradients of llsa_cross_attn_fwd.  With P = exp(z - lse), D_i = d_o_i . o_i
 * and dS = scale P (d_o v^T - D): dq = dS k, dk = dS^T q, dv = P^T d_o, the
 * last two summed over the query heads of a key head; zero for keys that are
 * not valid and queries without a valid key.  o, lse: from the forward call
 * with the same keys, kv_len and key_mask. */
llsa_status llsa_cross_attn_bwd(const llsa_cross_problem* p, const void* q, const void* k, const void* v,
                                const int32_t* kv_len, const uint8_t* key_mask, const void* o, const void* d_o,
                                const float* lse, void* dq, void* dk, void* dv, void* workspace,
                                llsa_stream stream);

/* Which kernels the two calls run for *p, its strides among it (host only, no
 * launch): 1 for the tensor-core kernels, 0 for the CUDA-core ones (fp32, and
 * bf16 with a token stride of 0 in q, k, v or, backward, d_o; the forward for
 * few queries takes those too).  Either pointer may be NULL. */
llsa_status llsa_cross_attn_paths(const llsa_cross_problem* p, int* fwd_tc, int* bwd_tc);

/* Layer norm of every token row over its c channels. */
typedef struct {
  int batch, heads, n;    /* rows: batch * heads * n */
  int c;                  /* channels, 1..LLSA_NORM_MAX_C */
  float eps;              /* added to the variance; >= 0 */
  int dtype;              /* llsa_dtype of x, y, dy, dx */
  int param_dtype;        /* of weight, bias and their gradients: dtype or LLSA_FP32 */
  int per_batch;          /* 0: weight, bias [c]; 1: [batch][c], a modulation of its own for each batch row (strided, as
                           * slices of a projection's output are) */
  llsa_strides x, y, dy, dx;   /* any strides */
  int64_t weight_batch, bias_batch; /* per_batch: elements between the batch rows; 0: c.  Not used otherwise */
} llsa_norm_problem;

#define LLSA_NORM_MAX_C 16384

typedef struct {
  size_t stat_bytes;              /* fp32 [batch][heads][n], mean and rstd each */
  size_t bwd_workspace_bytes;
} llsa_norm_buffers;

llsa_status llsa_norm_validate(const llsa_norm_problem* p);
/* Byte sizes; they depend on the sizes and types in *p, not on its strides. */
llsa_status llsa_norm_query_sizes(const llsa_norm_problem* p, llsa_norm_buffers* out);

/* y = (x - mean) * rstd * weight + bias with mean and rstd = 1 / sqrt(var + eps)
 * over the row's channels (var: mean of the squared deviations).  weight and
 * bias may be NULL (1 and 0); mean and rstd are written where not NULL.  y may
 * be x itself with the same strides. */
llsa_status llsa_layer_norm_fwd(const llsa_norm_problem* p, const void* x, const void* weight, const void* bias,
                                void* y, float* mean, float* rstd, llsa_stream stream);

/* Gradients: with g = dy * weight and xhat = (x - mean) * rstd,
 *   dx = rstd (g - mean_c(g) - xhat mean_c(g xhat)),
 *   dweight = sum over rows dy xhat, dbias = sum over rows dy (per batch row
 * when per_batch).  weight may be NULL as in the forward call; dx, dweight and
 * dbias are written where not NULL (not all three).  mean, rstd: from the
 * forward call.  dx may be dy itself with the same strides. */
llsa_status llsa_layer_norm_bwd(const llsa_norm_problem* p, const void* x, const void* dy, const void* weight,
                                const float* mean, const float* rstd, void* dx, void* dweight, void* dbias,
                                void* workspace, llsa_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* LLSA_H */
