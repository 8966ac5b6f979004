// llsa_ops_api.cu -- the C ABI of cross attention and layer norm: argument
// validation, buffer sizes, dispatch to the kernels.
#include <math.h>
#include <string.h>

#include <initializer_list>

#include "cross.cuh"
#include "norm.cuh"

namespace llsa {

constexpr int kSms = 148;                       // sizes follow from the problem alone, not from the device

static bool aligned(const void* p, size_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// The widest load of up to v values of `size` bytes that every address allows.
static int widest(int v, size_t size, std::initializer_list<const void*> all) {
  for (const void* p : all)
    while (v > 1 && !aligned(p, v * size > 16 ? 16 : v * size)) v /= 2;
  return v;
}

struct Dim {
  int64_t n, s;
};

// Whether no two elements of a tensor with these dimensions (beside `inner`
// contiguous channels) share an address: by growing stride, each step leaves
// everything inside it behind.
static bool distinct(Dim* d, int count, int64_t inner) {
  for (int i = 0; i < count; ++i)
    for (int j = i + 1; j < count; ++j)
      if (d[j].s < d[i].s) {
        Dim t = d[i];
        d[i] = d[j];
        d[j] = t;
      }
  int64_t extent = inner;
  for (int i = 0; i < count; ++i) {
    if (d[i].n == 1) continue;
    if (d[i].s < extent) return false;
    extent += (d[i].n - 1) * d[i].s;
  }
  return true;
}

// Strides of a [b][h][n][d] tensor: contiguous where all are zero; a
// dimension of one takes the contiguous stride.
static llsa_status layout(const llsa_strides& in, int64_t b, int64_t h, int64_t n, int64_t d, int64_t multiple,
                          bool written, int64_t* sb, int64_t* sh, int64_t* sn) {
  const bool none = in.batch == 0 && in.head == 0 && in.token == 0;
  const int64_t given[3] = {in.batch, in.head, in.token}, plain[3] = {h * n * d, n * d, d}, size[3] = {b, h, n};
  int64_t* out[3] = {sb, sh, sn};
  Dim dims[3];
  for (int i = 0; i < 3; ++i) {
    *out[i] = none || size[i] == 1 ? plain[i] : given[i];
    if (size[i] == 1 && !none) *out[i] = d;     // never multiplied by more than index 0
    if (*out[i] < 0) return LLSA_ERR_ARG;
    if (*out[i] >= (1ll << 37)) return LLSA_ERR_SHAPE;
    if (size[i] > 1 && *out[i] % multiple) return LLSA_ERR_ALIGN;
    dims[i] = Dim{size[i], *out[i]};
  }
  if (written && !distinct(dims, 3, d)) return LLSA_ERR_ARG;
  return LLSA_OK;
}

static llsa_status make_cross(const llsa_cross_problem* p, cross::Geo* g) {
  if (!p) return LLSA_ERR_ARG;
  memset(g, 0, sizeof(*g));
  if (p->batch < 1 || p->heads < 1 || p->kv_heads < 1 || p->nq < 1 || p->nk < 1 || p->d < 1) return LLSA_ERR_ARG;
  if (p->heads % p->kv_heads) return LLSA_ERR_ARG;
  if (p->dtype != LLSA_BF16 && p->dtype != LLSA_FP32) return LLSA_ERR_ARG;
  if (!(p->scale >= 0.0f) || isinf(p->scale)) return LLSA_ERR_ARG;
  if (p->d % 8 != 0 || p->d > 128) return LLSA_ERR_UNSUPPORTED;
  const int64_t b = p->batch, h = p->heads, hk = p->kv_heads, nq = p->nq, nk = p->nk, d = p->d;
  if (b * h > (1 << 24) || nq > LLSA_CROSS_MAX_TOKENS || nk > LLSA_CROSS_MAX_TOKENS) return LLSA_ERR_SHAPE;
  // a block's work between two hand-offs ends well before their waits give up: at most 2^19 tiles of 128 queries, each of
  // one head where a head fills a tile (3.2 us a tile in the longest chain: 1.7 s of 4)
  const int64_t padded = nq < 128 ? nq : (nq + 127) / 128 * 128;
  if (h / hk * padded > 4ll * LLSA_CROSS_MAX_TOKENS) return LLSA_ERR_SHAPE;
  if (b * h * nq >= (1ll << 34) || b * hk * nk >= (1ll << 34)) return LLSA_ERR_SHAPE;
  // one block per 32 queries or keys and head at most: a grid of fewer than 2^31 blocks
  if (b * h * ((nq + 31) / 32) >= (1ll << 31) || b * hk * ((nk + 31) / 32) >= (1ll << 31)) return LLSA_ERR_SHAPE;
  g->b = p->batch;
  g->h = p->heads;
  g->hk = p->kv_heads;
  g->group = p->heads / p->kv_heads;
  g->nq = p->nq;
  g->nk = p->nk;
  g->d = p->d;
  g->scale = p->scale > 0.0f ? p->scale : 1.0f / sqrtf((float)p->d);
  g->bf16 = p->dtype == LLSA_BF16;
  const int64_t m = g->bf16 ? 8 : 4;
  struct {
    const llsa_strides* in;
    cross::Lay* out;
    int64_t h, n;
    bool written;
  } all[8] = {{&p->q, &g->q, h, nq, false},    {&p->k, &g->k, hk, nk, false}, {&p->v, &g->v, hk, nk, false},
              {&p->o, &g->o, h, nq, true},     {&p->d_o, &g->dO, h, nq, false}, {&p->dq, &g->dq, h, nq, true},
              {&p->dk, &g->dk, hk, nk, true}, {&p->dv, &g->dv, hk, nk, true}};
  for (auto& t : all) {
    const llsa_status st = layout(*t.in, b, t.h, t.n, d, m, t.written, &t.out->b, &t.out->h, &t.out->n);
    if (st != LLSA_OK) return st;
  }
  return LLSA_OK;
}

// Rows as nested loops in the order of x's memory.
static llsa_status make_norm(const llsa_norm_problem* p, norm::Geo* g) {
  if (!p) return LLSA_ERR_ARG;
  memset(g, 0, sizeof(*g));
  if (p->batch < 1 || p->heads < 1 || p->n < 1 || p->c < 1) return LLSA_ERR_ARG;
  if (p->dtype != LLSA_BF16 && p->dtype != LLSA_FP32) return LLSA_ERR_ARG;
  if (p->param_dtype != p->dtype && p->param_dtype != LLSA_FP32) return LLSA_ERR_ARG;
  if (p->per_batch != 0 && p->per_batch != 1) return LLSA_ERR_ARG;
  if (!(p->eps >= 0.0f) || isinf(p->eps)) return LLSA_ERR_ARG;
  if (p->c > LLSA_NORM_MAX_C) return LLSA_ERR_UNSUPPORTED;
  const int64_t b = p->batch, h = p->heads, n = p->n, c = p->c;
  if (b * h > (1ll << 31) || b * h * n >= (1ll << 31)) return LLSA_ERR_SHAPE;
  if (p->per_batch && b > 65535) return LLSA_ERR_SHAPE;
  int64_t st[5][3];                             // x, y, dy, dx, mean / rstd; by dimension: batch, head, token
  const llsa_strides* in[4] = {&p->x, &p->y, &p->dy, &p->dx};
  for (int t = 0; t < 4; ++t) {
    const llsa_status e = layout(*in[t], b, h, n, c, 1, t == 1 || t == 3, &st[t][0], &st[t][1], &st[t][2]);
    if (e != LLSA_OK) return e;
  }
  st[4][0] = h * n;
  st[4][1] = n;
  st[4][2] = 1;
  const int64_t size[3] = {b, h, n};
  g->vec = p->dtype == LLSA_BF16 ? 8 : 4;
  while (c % g->vec) g->vec /= 2;
  for (int t = 0; t < 4; ++t)
    for (int i = 0; i < 3; ++i)
      while (size[i] > 1 && st[t][i] % g->vec) g->vec /= 2;
  g->ws = g->bs = p->c;
  if (p->per_batch) {
    if (p->weight_batch < 0 || p->bias_batch < 0) return LLSA_ERR_ARG;
    if (p->weight_batch >= (1ll << 37) || p->bias_batch >= (1ll << 37)) return LLSA_ERR_SHAPE;
    if (p->weight_batch) g->ws = p->weight_batch;
    if (p->bias_batch) g->bs = p->bias_batch;
    while (b > 1 && (g->ws % g->vec || g->bs % g->vec)) g->vec /= 2;
  }
  int64_t* out[5] = {g->x, g->y, g->dy, g->dx, g->s};
  // the loops over the group's rows, outermost first, in the order of x's strides; loops of one drop out
  int order[3], count = 0;
  for (int i = p->per_batch ? 1 : 0; i < 3; ++i)
    if (size[i] > 1) order[count++] = i;
  for (int i = 0; i < count; ++i)
    for (int j = i + 1; j < count; ++j)
      if (st[0][order[j]] > st[0][order[i]]) {
        const int t = order[i];
        order[i] = order[j];
        order[j] = t;
      }
  int64_t ln[3] = {1, 1, 1}, ls[5][3] = {};     // innermost first
  bool flat[4] = {true, true, true, true};
  for (int i = 0; i < count; ++i) {
    const int dim = order[count - 1 - i];
    ln[i] = size[dim];
    for (int t = 0; t < 5; ++t) ls[t][i] = st[t][dim];
    for (int t = 0; t < 4; ++t) flat[t] = flat[t] && (i == 0 || ls[t][i] == ls[t][i - 1] * ln[i - 1]);
  }
  g->flat_fwd = flat[0] && flat[1];
  g->flat_bwd = flat[0] && flat[2] && flat[3];
  g->groups = p->per_batch ? p->batch : 1;
  g->rows = ln[0] * ln[1] * ln[2];
  g->n2 = divisor((uint32_t)ln[0]);
  g->n1 = divisor((uint32_t)ln[1]);
  for (int t = 0; t < 5; ++t) {
    for (int i = 0; i < 3; ++i) out[t][2 - i] = ls[t][i];
    out[t][3] = st[t][0];
  }
  g->c = p->c;
  g->eps = p->eps;
  g->bf16 = p->dtype == LLSA_BF16;
  g->param_bf16 = p->param_dtype == LLSA_BF16;
  return LLSA_OK;
}

static llsa_status launched(cudaError_t e) {
  if (e != cudaSuccess) return LLSA_ERR_CUDA;
  return cudaPeekAtLastError() == cudaSuccess ? LLSA_OK : LLSA_ERR_CUDA;
}

}  // namespace llsa

#define LLSA_NEED(ptr)                                   \
  do {                                                   \
    if (!(ptr)) return LLSA_ERR_ARG;                     \
    if (!llsa::aligned(ptr, 16)) return LLSA_ERR_ALIGN;  \
  } while (0)
#define LLSA_MAY(ptr, to)                                \
  do {                                                   \
    if (!llsa::aligned(ptr, to)) return LLSA_ERR_ALIGN;  \
  } while (0)
#define LLSA_CROSS(p, g)                            \
  llsa::cross::Geo g;                               \
  do {                                              \
    llsa_status st_ = llsa::make_cross(p, &g);      \
    if (st_ != LLSA_OK) return st_;                 \
  } while (0)
#define LLSA_NORM(p, g)                             \
  llsa::norm::Geo g;                                \
  do {                                              \
    llsa_status st_ = llsa::make_norm(p, &g);       \
    if (st_ != LLSA_OK) return st_;                 \
  } while (0)

extern "C" {

llsa_status llsa_cross_validate(const llsa_cross_problem* p) {
  LLSA_CROSS(p, g);
  return LLSA_OK;
}

llsa_status llsa_cross_query_sizes(const llsa_cross_problem* p, llsa_cross_buffers* out) {
  if (!out) return LLSA_ERR_ARG;
  LLSA_CROSS(p, g);
  const llsa::cross::Plan plan = llsa::cross::plan_simt(g, llsa::kSms);
  out->lse_bytes = (size_t)llsa::cross::rows_of(g) * sizeof(float);
  out->fwd_workspace_bytes = llsa::cross::fwd_work_bytes(g, plan.fwd_ks);
  out->bwd_workspace_bytes = llsa::cross::bwd_work_bytes_simt(g, plan);
  if (g.bf16) {                                 // the strides decide which kernels run: room for either
    const size_t tc = llsa::cross::token_supported(g)
                          ? llsa::cross::token_work_bytes(g, llsa::kSms)
                          : llsa::cross::fwd_work_bytes(g, llsa::cross::plan_fwd_tc(g, llsa::kSms).ks);
    if (tc > out->fwd_workspace_bytes) out->fwd_workspace_bytes = tc;
    const size_t bwd = llsa::cross::bwd_work_bytes_tc(g, llsa::kSms);
    if (bwd > out->bwd_workspace_bytes) out->bwd_workspace_bytes = bwd;
  }
  return LLSA_OK;
}

llsa_status llsa_cross_attn_fwd(const llsa_cross_problem* p, const void* q, const void* k, const void* v,
                                const int32_t* kv_len, const uint8_t* key_mask, void* o, float* lse, void* workspace,
                                llsa_stream stream) {
  LLSA_CROSS(p, g);
  LLSA_NEED(q);
  LLSA_NEED(k);
  LLSA_NEED(v);
  LLSA_NEED(o);
  LLSA_MAY(kv_len, 4);
  LLSA_MAY(lse, 16);
  LLSA_MAY(workspace, 16);                      // of any call that is given one, whether its plan needs it or not
  const llsa::cross::Keys keys{kv_len, key_mask};
  if (llsa::cross::token_supported(g)) {
    LLSA_NEED(workspace);
    return llsa::launched(llsa::cross::launch_fwd_token(g, llsa::kSms, q, k, v, keys, o, lse, workspace, (cudaStream_t)stream));
  }
  if (llsa::cross::fwd_tc_supported(g)) {
    const llsa::cross::TcPlan plan = llsa::cross::plan_fwd_tc(g, llsa::kSms);
    if (plan.ks > 1) LLSA_NEED(workspace);
    return llsa::launched(llsa::cross::launch_fwd_tc(g, plan, q, k, v, keys, o, lse, workspace, (cudaStream_t)stream));
  }
  const llsa::cross::Plan plan = llsa::cross::plan_simt(g, llsa::kSms);
  if (plan.fwd_ks > 1) LLSA_NEED(workspace);
  return llsa::launched(llsa::cross::launch_fwd_simt(g, plan, q, k, v, keys, o, lse, workspace, (cudaStream_t)stream));
}

llsa_status llsa_cross_attn_bwd(const llsa_cross_problem* p, const void* q, const void* k, const void* v,
                                const int32_t* kv_len, const uint8_t* key_mask, const void* o, const void* d_o,
                                const float* lse, void* dq, void* dk, void* dv, void* workspace, llsa_stream stream) {
  LLSA_CROSS(p, g);
  LLSA_NEED(q);
  LLSA_NEED(k);
  LLSA_NEED(v);
  LLSA_MAY(kv_len, 4);
  LLSA_NEED(o);
  LLSA_NEED(d_o);
  LLSA_NEED(lse);
  LLSA_NEED(dq);
  LLSA_NEED(dk);
  LLSA_NEED(dv);
  LLSA_NEED(workspace);
  const llsa::cross::Keys keys{kv_len, key_mask};
  if (llsa::cross::bwd_tc_supported(g))
    return llsa::launched(llsa::cross::launch_bwd_tc(g, llsa::kSms, q, k, v, keys, o, d_o, lse, dq, dk, dv, workspace,
                                                     (cudaStream_t)stream));
  const llsa::cross::Plan plan = llsa::cross::plan_simt(g, llsa::kSms);
  return llsa::launched(llsa::cross::launch_bwd_simt(g, plan, q, k, v, keys, o, d_o, lse, dq, dk, dv, workspace,
                                                     (cudaStream_t)stream));
}

llsa_status llsa_cross_attn_paths(const llsa_cross_problem* p, int* fwd_tc, int* bwd_tc) {
  LLSA_CROSS(p, g);
  if (fwd_tc) *fwd_tc = llsa::cross::token_supported(g) || llsa::cross::fwd_tc_supported(g);
  if (bwd_tc) *bwd_tc = llsa::cross::bwd_tc_supported(g);
  return LLSA_OK;
}

llsa_status llsa_norm_validate(const llsa_norm_problem* p) {
  LLSA_NORM(p, g);
  return LLSA_OK;
}

llsa_status llsa_norm_query_sizes(const llsa_norm_problem* p, llsa_norm_buffers* out) {
  if (!out) return LLSA_ERR_ARG;
  LLSA_NORM(p, g);
  out->stat_bytes = (size_t)p->batch * p->heads * p->n * sizeof(float);
  out->bwd_workspace_bytes = llsa::norm::bwd_work_bytes(g);
  return LLSA_OK;
}

llsa_status llsa_layer_norm_fwd(const llsa_norm_problem* p, const void* x, const void* weight, const void* bias,
                                void* y, float* mean, float* rstd, llsa_stream stream) {
  LLSA_NORM(p, g);
  if (!x || !y) return LLSA_ERR_ARG;
  const size_t t = g.bf16 ? 2 : 4, pt = g.param_bf16 ? 2 : 4;
  LLSA_MAY(x, t);
  LLSA_MAY(y, t);
  LLSA_MAY(weight, pt);
  LLSA_MAY(bias, pt);
  LLSA_MAY(mean, 4);
  LLSA_MAY(rstd, 4);
  g.vec = llsa::widest(llsa::widest(g.vec, t, {x, y}), pt, {weight, bias});
  return llsa::launched(llsa::norm::launch_fwd(g, x, weight, bias, y, mean, rstd, (cudaStream_t)stream));
}

llsa_status llsa_layer_norm_bwd(const llsa_norm_problem* p, const void* x, const void* dy, const void* weight,
                                const float* mean, const float* rstd, void* dx, void* dweight, void* dbias,
                                void* workspace, llsa_stream stream) {
  LLSA_NORM(p, g);
  if (!x || !dy || !mean || !rstd) return LLSA_ERR_ARG;
  const size_t t = g.bf16 ? 2 : 4, pt = g.param_bf16 ? 2 : 4;
  LLSA_MAY(x, t);
  LLSA_MAY(dy, t);
  LLSA_MAY(dx, t);
  LLSA_MAY(weight, pt);
  LLSA_MAY(dweight, pt);
  LLSA_MAY(dbias, pt);
  LLSA_MAY(mean, 4);
  LLSA_MAY(rstd, 4);
  g.vec = llsa::widest(llsa::widest(g.vec, t, {x, dy, dx}), pt, {weight});
  if (!dx && !dweight && !dbias) return LLSA_ERR_ARG;
  LLSA_MAY(workspace, 16);
  if (dweight || dbias) LLSA_NEED(workspace);
  return llsa::launched(
      llsa::norm::launch_bwd(g, x, dy, weight, mean, rstd, dx, dweight, dbias, workspace, (cudaStream_t)stream));
}

}  // extern "C"
