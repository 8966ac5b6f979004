// k_cross_token.cu -- cross attention forward for few queries: at most 16 rows
// (the tokens of all query heads of a key head) against the states, bf16.
// One step of a decoder, or attention pooling.
//
// Bound by memory: every key and value is read once, 4 d bytes a pair for 4 d
// FLOPs a row.  All slices' valid keys, in blocks of 16, form one line that is
// cut into equal runs, one for each of 8 warps an SM, whatever the lengths are.
// A warp works on its own: cp.async brings its next blocks (K and V, three
// stages; an SM then has some 128 KB on their way) while it computes one:
//   S = Q K^T      mma.m16n8k16, Q in registers, K by ldmatrix
//   P = 2^(z - m)  the lazy running maximum of the row, its four lanes together
//   O += P V       the scores' registers are the left operand
// (The tiles of the 5th-generation tensor cores have 128 rows, of which these
// problems fill a few; there the chain of hand-offs between warps, 2.6 us for
// 128 keys, took 90 us where this takes a third.)  No block-wide step: each run leaves its
// part of a slice as fp32 O and LSE, and a second kernel joins a slice's parts.
// Run w's part of slice s stands at place w + s: either grows along the line.
#include <math.h>

#include "cross_tc.cuh"

namespace llsa {
namespace cross {
namespace token {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kHeadroom = 8.f;               // log2 of the largest weight before O is rescaled
constexpr int WARPS = 8, ROWS = 16, KEYS = 16; // KEYS: of a block
constexpr int MAX_BATCH = 2048;                // batch rows whose lengths a block keeps
constexpr int MIN_RUN = 4;                     // blocks of a run, at least
constexpr int SMS = 148, MAX_PARTS = SMS * WARPS;    // runs, and so parts of a slice, at most

struct Args {
  Geo g;
  Keys keys;
  Divisor by_hk, by_nq;
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* o;
  float* lse;
  int64_t* line;                               // [batch + 2] blocks before each batch row, all blocks; blocks of a run
  float* part;                                 // [runs + slices][rows][d]
  float* part_lse;                             // [runs + slices][rows]
};

__device__ __forceinline__ void copy16(void* dst, const void* src, bool any) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "r"(any ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int DP>
struct Smem {
  static constexpr int ST = DP == 64 ? 5 : 3;  // blocks of a warp in flight
  alignas(16) unsigned char kv[WARPS][ST][2][KEYS * DP * 2];   // K and V rows, 16-byte chunk c of row r at c ^ (r & 7)
  int64_t line[MAX_BATCH + 1];
};
static_assert(sizeof(Smem<64>) <= 232448 && sizeof(Smem<128>) <= 232448, "shared memory of one CTA");

template <int DP>
__global__ void __launch_bounds__(WARPS * 32, 1) token_kernel(const __grid_constant__ Args a) {
  using S = Smem<DP>;
  constexpr int ST = S::ST, CH = DP / 8, NT = DP / 8, KS = DP / 16;
  extern __shared__ __align__(16) unsigned char raw[];
  S& s = *reinterpret_cast<S*>(raw);
  const Geo& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // blocks before each batch row
  if (warp == 0) {
    int64_t sum = 0;
    for (int b0 = 0; b0 < g.b; b0 += 32) {
      const int b = b0 + lane;
      int64_t n = b < g.b ? (int64_t)g.hk * ((key_count(g, a.keys, b) + KEYS - 1) / KEYS) : 0;
#pragma unroll
      for (int w = 1; w < 32; w <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, n, w);
        if (lane >= w) n += up;
      }
      if (b < g.b) s.line[b + 1] = sum + n;
      sum += __shfl_sync(0xffffffffu, n, 31);
    }
    if (lane == 0) s.line[0] = 0;
  }
  __syncthreads();
  const int64_t total = s.line[g.b];
  const int runs = (int)gridDim.x * WARPS;
  int64_t per = (total + runs - 1) / runs;
  if (per < MIN_RUN) per = MIN_RUN;
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b <= g.b; b += WARPS * 32) a.line[b] = s.line[b];
    if (threadIdx.x == 0) a.line[g.b + 1] = per;
  }
  // runs go round the SMs, so that few of them use all
  const int run = warp * (int)gridDim.x + (int)blockIdx.x;
  int64_t at = run * per;
  const int64_t end = min(at + per, total);
  const float sc2 = g.scale * kLog2e;
  const int rows = g.group * g.nq;
  unsigned char(*stage)[2][KEYS * DP * 2] = s.kv[warp];
  // ldmatrix: matrix lane / 8, row lane % 8
  const int mi = lane >> 3, mr = lane & 7;
  while (at < end) {
    int lo = 0, hi = g.b - 1;                  // the batch row of block `at`
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s.line[mid] <= at) lo = mid; else hi = mid - 1;
    }
    const int b = lo;
    const int len = key_count(g, a.keys, b);
    const int nb = (len + KEYS - 1) / KEYS;
    const int hk = (int)((at - s.line[b]) / nb);
    const int first = (int)(at - s.line[b] - (int64_t)hk * nb);
    const int n = (int)min((int64_t)(nb - first), end - at);
    at += n;
    const uint8_t* mask = a.keys.mask ? a.keys.mask + (int64_t)b * g.nk : nullptr;
    const __nv_bfloat16* kb = a.k + b * g.k.b + hk * g.k.h;
    const __nv_bfloat16* vb = a.v + b * g.v.b + hk * g.v.h;
    auto valid = [&](int key) { return key < len && (!mask || mask[key]); };
    auto fetch = [&](int i) {                  // block i of the segment; keys that take no part are zero
      if (i < n) {
        unsigned char(*to)[KEYS * DP * 2] = stage[i % ST];
#pragma unroll
        for (int e = lane; e < KEYS * CH; e += 32) {
          const int r = e / CH, c = e % CH, key = (first + i) * KEYS + r;
          const bool any = c * 8 < g.d && valid(key);
          const int64_t off = any ? (int64_t)key : 0;
          const int cc = any ? c * 8 : 0;
          const int p = r * DP * 2 + ((c ^ (r & 7)) << 4);
          copy16(to[0] + p, kb + off * g.k.n + cc, any);
          copy16(to[1] + p, vb + off * g.v.n + cc, any);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) fetch(i);
    // Q: rows lane / 4 and + 8, channels 16 k + 2 (lane % 4) and + 8
    uint32_t qa[KS][4];
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = (lane >> 2) + 8 * (e & 1), c = 16 * k + 2 * (lane & 3) + 8 * (e >> 1);
        int t;
        const int h = hk * g.group + divide(r, a.by_nq, t);
        qa[k][e] = r < rows && c < g.d
                       ? *reinterpret_cast<const uint32_t*>(a.q + b * g.q.b + h * g.q.h + t * g.q.n + c)
                       : 0u;
      }
    float o[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};    // rows lane / 4 and + 8; l: of this lane's keys
    for (int i = 0; i < n; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(ST - 2) : "memory");
      __syncwarp();
      const uint32_t ks = ptx::smem_u32(stage[i % ST][0]), vs = ptx::smem_u32(stage[i % ST][1]);
      float z[2][4] = {};
#pragma unroll
      for (int k = 0; k < KS; ++k) {           // matrices: keys 0-7 and 8-15 (mi / 2), channels 0-7 and 8-15 (mi % 2)
        uint32_t w[4];
        const int r = (mi >> 1) * 8 + mr, c = 2 * k + (mi & 1);
        ldmatrix4(w, ks + r * DP * 2 + ((c ^ (r & 7)) << 4));
        mma16816(z[0], qa[k], w[0], w[1]);
        mma16816(z[1], qa[k], w[2], w[3]);
      }
      const int key0 = (first + i) * KEYS;
      if (mask || key0 + KEYS > len) {
        const uint32_t bits = __ballot_sync(0xffffffffu, lane < KEYS && valid(key0 + lane));
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((bits >> (8 * t + 2 * (lane & 3) + (e & 1))) & 1u)) z[t][e] = -INFINITY;
      }
      bool resc = false;
      float f[2] = {1.f, 1.f}, ref[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = fmaxf(fmaxf(z[0][2 * r], z[0][2 * r + 1]), fmaxf(z[1][2 * r], z[1][2 * r + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[r], mx * sc2);
        if (m[r] == -INFINITY) {
          m[r] = mn;
        } else if (mn > m[r] + kHeadroom) {
          resc = true;
          f[r] = ptx::ex2(m[r] - mn);
          m[r] = mn;
          l[r] *= f[r];
        }
        ref[r] = m[r] == -INFINITY ? 0.f : m[r];   // no key so far: every weight is 2^-inf = 0
      }
      if (__any_sync(0xffffffffu, resc)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][e] *= f[e >> 1];
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[t][e] = ptx::ex2(fmaf(z[t][e], sc2, -ref[e >> 1]));
          l[e >> 1] += z[t][e];
        }
      const uint32_t p[4] = {ptx::pack_bf16(z[0][0], z[0][1]), ptx::pack_bf16(z[0][2], z[0][3]),
                             ptx::pack_bf16(z[1][0], z[1][1]), ptx::pack_bf16(z[1][2], z[1][3])};
#pragma unroll
      for (int k = 0; k < KS; ++k) {           // matrices: keys 0-7 and 8-15 (mi % 2), channels 0-7 and 8-15 (mi / 2)
        uint32_t w[4];
        const int r = (mi & 1) * 8 + mr, c = 2 * k + (mi >> 1);
        ldmatrix4_t(w, vs + r * DP * 2 + ((c ^ (r & 7)) << 4));
        mma16816(o[2 * k], p, w[0], w[1]);
        mma16816(o[2 * k + 1], p, w[2], w[3]);
      }
      __syncwarp();                            // every lane has read the stage that comes next to be filled
      fetch(i + ST - 1);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    const int64_t place = (int64_t)run + (int64_t)b * g.hk + hk;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      const int row = (lane >> 2) + 8 * r;
      if (row >= rows) continue;
      const bool none = m[r] == -INFINITY && !(l[r] > 0.f) && l[r] == l[r];    // NaN sums pass through
      const float inv = none ? 0.f : 1.f / l[r];
      float* to = a.part + (place * rows + row) * g.d;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int c = 8 * t + 2 * (lane & 3);
        if (c < g.d)
          *reinterpret_cast<float2*>(to + c) = make_float2(none ? 0.f : o[t][2 * r] * inv, none ? 0.f : o[t][2 * r + 1] * inv);
      }
      if ((lane & 3) == 0) a.part_lse[place * rows + row] = none ? -INFINITY : (m[r] + log2f(l[r])) * kLn2;
    }
    __syncwarp();
  }
}

// One block per row: O = sum_w c_w O_w / sum_w c_w over the runs that hold a
// part of its slice, c_w = exp(LSE_w - max LSE).  128 threads: four channels
// each, the runs dealt to 128 / (d / 4) groups whose sums are added in order.
__global__ void __launch_bounds__(128) token_join_kernel(const __grid_constant__ Args a) {
  __shared__ float4 acc[128];
  __shared__ float red[4], tot[128];
  __shared__ float weight[MAX_PARTS];
  const Geo& g = a.g;
  const int rows = g.group * g.nq;
  const int64_t slice = blockIdx.x / rows;
  const int row = (int)(blockIdx.x % rows);
  int hk, t;
  const int b = divide((int)slice, a.by_hk, hk);
  const int64_t nb = (a.line[b + 1] - a.line[b]) / g.hk, per = a.line[g.b + 1];
  const int64_t s0 = a.line[b] + hk * nb;
  const int64_t w0 = s0 / per;               // (runs are at most MAX_PARTS)
  const int parts = nb > 0 ? (int)((s0 + nb - 1) / per - w0) + 1 : 0;
  const int64_t place = w0 + slice;
  const float* lse = a.part_lse + place * rows + row;
  float mx = -INFINITY;
  for (int i = threadIdx.x; i < parts; i += 128) {
    const float ls = lse[(int64_t)i * rows];
    weight[i] = ls;
    mx = fmaxf(mx, ls);
  }
#pragma unroll
  for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const int c4 = g.d / 4, groups = 128 / c4;
  const int grp = threadIdx.x / c4, c = (threadIdx.x % c4) * 4;
  const float ref = mx == -INFINITY ? 0.f : mx;
  for (int i = threadIdx.x; i < parts; i += 128) weight[i] = exp2f((weight[i] - ref) * kLog2e);   // a run without keys: 0
  __syncthreads();
  float sum = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (grp < groups)
#pragma unroll 8
    for (int i = grp; i < parts; i += groups) {
      const float4 y = *reinterpret_cast<const float4*>(a.part + ((place + i) * rows + row) * g.d + c);
      const float w = weight[i];
      sum += w;
      x.x = fmaf(w, y.x, x.x);
      x.y = fmaf(w, y.y, x.y);
      x.z = fmaf(w, y.z, x.z);
      x.w = fmaf(w, y.w, x.w);
    }
  acc[threadIdx.x] = x;
  tot[threadIdx.x] = sum;
  __syncthreads();
  if (grp != 0) return;
  for (int i = 1; i < groups; ++i) {
    const float4 y = acc[i * c4 + threadIdx.x];
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
    sum += tot[i * c4 + threadIdx.x];
  }
  const int h = hk * g.group + divide(row, a.by_nq, t);
  const bool none = mx == -INFINITY && sum == 0.f;
  const float inv = none ? 0.f : 1.f / sum;
  __nv_bfloat16* to = a.o + b * g.o.b + h * g.o.h + t * g.o.n + c;
  *reinterpret_cast<uint2*>(to) = make_uint2(ptx::pack_bf16(x.x * inv, x.y * inv), ptx::pack_bf16(x.z * inv, x.w * inv));
  if (a.lse && c == 0) a.lse[((int64_t)b * g.h + h) * g.nq + t] = none ? -INFINITY : mx + log2f(sum) * kLn2;
}

}  // namespace token

// Few rows a key head: what the tensor memory kernel would spend its 128-row tiles on.
bool token_supported(const Geo& g) {
  return g.bf16 && (int64_t)g.group * g.nq <= token::ROWS && g.b <= token::MAX_BATCH;
}

static int64_t token_places(const Geo& g, int sms) { return (int64_t)sms * token::WARPS + (int64_t)g.b * g.hk; }

static token::Args carve_token(const Geo& g, int sms, void* work, size_t* bytes) {
  token::Args a;
  const int64_t places = token_places(g, sms), rows = (int64_t)g.group * g.nq;
  const size_t line = round256(((size_t)g.b + 2) * 8), part = round256((size_t)(places * rows * g.d) * 4);
  char* w = static_cast<char*>(work);
  a.line = reinterpret_cast<int64_t*>(w);
  a.part = reinterpret_cast<float*>(w + line);
  a.part_lse = reinterpret_cast<float*>(w + line + part);
  if (bytes) *bytes = line + part + round256((size_t)(places * rows) * 4);
  return a;
}

size_t token_work_bytes(const Geo& g, int sms) {
  size_t n = 0;
  carve_token(g, sms, nullptr, &n);
  return n;
}

cudaError_t launch_fwd_token(const Geo& g, int sms, const void* q, const void* k, const void* v, const Keys& keys,
                             void* o, float* lse, void* work, cudaStream_t s) {
  token::Args a = carve_token(g, sms, work, nullptr);
  a.g = g;
  a.keys = keys;
  a.by_hk = divisor(g.hk);
  a.by_nq = divisor(g.nq);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  const bool narrow = g.d <= 64;
  const size_t smem = narrow ? sizeof(token::Smem<64>) : sizeof(token::Smem<128>);
  cudaError_t e = narrow ? cudaFuncSetAttribute(token::token_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                (int)smem)
                         : cudaFuncSetAttribute(token::token_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                (int)smem);
  if (e != cudaSuccess) return e;
  if (narrow)
    token::token_kernel<64><<<sms, token::WARPS * 32, smem, s>>>(a);
  else
    token::token_kernel<128><<<sms, token::WARPS * 32, smem, s>>>(a);
  note_launches(1);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  token::token_join_kernel<<<(unsigned)(rows_of(g)), 128, 0, s>>>(a);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace cross
}  // namespace llsa
