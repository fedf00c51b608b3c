// rlk_paged.cu -- the paged key-value cache: append, and the attention of new
// tokens over it.

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "rlk_rollout.h"
#include "rlk_host.h"

namespace rlk {

struct PagedParams {
  const void* k;
  const void* v;
  int64_t num_pages, page_stride, token_stride, head_stride;
  int page_size, kv_heads, max_pages;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  const int32_t* new_lens;
  int n;
  int32_t* err;
};

// Length and number of new tokens of sequence b, or false where they do not
// agree with each other or with the page table's width.
__device__ __forceinline__ bool seq_lens(const PagedParams& P, int b, int& len, int& nnew) {
  len = P.lens[b];
  nnew = P.new_lens ? P.new_lens[b] : P.n;
  return nnew >= 0 && nnew <= P.n && len >= nnew &&
         len <= static_cast<int64_t>(P.max_pages) * P.page_size;
}

// ------------------------------------------------------------ append

struct AppendParams {
  PagedParams c;
  const uint4* ksrc;
  const uint4* vsrc;
  rlk_bth_strides ks, vs;       // in 16-byte units
  int row16;                    // 16-byte pieces of a head row
  int64_t total;                // B * n * kv_heads * row16
};

// One thread per 16-byte piece of a new token's head row, keys and values.
__global__ void append_kernel(const AppendParams P) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t >= P.total) return;
  const int piece = static_cast<int>(t % P.row16);
  int64_t rest = t / P.row16;
  const int h = static_cast<int>(rest % P.c.kv_heads);
  rest /= P.c.kv_heads;
  const int i = static_cast<int>(rest % P.c.n);
  const int b = static_cast<int>(rest / P.c.n);
  int len, nnew;
  const bool first = piece == 0 && h == 0;
  if (!seq_lens(P.c, b, len, nnew)) {
    if (first && i == 0 && P.c.err) atomicAdd(P.c.err, 1);
    return;
  }
  if (i >= nnew) return;
  const int pos = len - nnew + i;
  const int page = P.c.table[b * P.c.table_stride + pos / P.c.page_size];
  if (page < 0 || page >= P.c.num_pages) {
    if (first && P.c.err) atomicAdd(P.c.err, 1);
    return;
  }
  const int64_t at = (page * P.c.page_stride + (pos % P.c.page_size) * P.c.token_stride + h * P.c.head_stride) / 8 + piece;
  reinterpret_cast<uint4*>(const_cast<void*>(P.c.k))[at] = P.ksrc[b * P.ks.batch + i * P.ks.token + h * P.ks.head + piece];
  reinterpret_cast<uint4*>(const_cast<void*>(P.c.v))[at] = P.vsrc[b * P.vs.batch + i * P.vs.token + h * P.vs.head + piece];
}

// ------------------------------------------------------------ attention

struct AttnParams {
  PagedParams c;
  const void* q;
  void* out;
  rlk_bth_strides qs, os;       // elements
  int q_heads;
  float scale;
  int window, sinks;
  float* lse;
};

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_float(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_float(float x, __half& y) { y = __float2half_rn(x); }

// One warp per query and head: every lane holds head_dim / 32 elements, the
// visible tokens go by one at a time with a running maximum and sum.
template <class T, int D>
__global__ void __launch_bounds__(128) attn_kernel(const AttnParams P, int64_t warps) {
  constexpr int E = D / 32;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
  if (w >= warps) return;
  const int lane = threadIdx.x & 31;
  const int hq = static_cast<int>(w % P.q_heads);
  const int i = static_cast<int>(w / P.q_heads % P.c.n);
  const int b = static_cast<int>(w / P.q_heads / P.c.n);
  const int hk = hq / (P.q_heads / P.c.kv_heads);
  T* out = static_cast<T*>(P.out) + b * P.os.batch + i * P.os.token + hq * P.os.head + lane * E;
  const float nan = __int_as_float(0x7fc00000);
  int len, nnew;
  bool ok = seq_lens(P.c, b, len, nnew);
  float m = -INFINITY, l = 0.0f, o[E] = {}, qv[E];
  if (ok && i < nnew) {
    const int pos = len - nnew + i;
    const T* qp = static_cast<const T*>(P.q) + b * P.qs.batch + i * P.qs.token + hq * P.qs.head + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) qv[e] = to_float(qp[e]);
    const int low = P.window > 0 ? max(0, pos - P.window + 1) : 0;
    for (int j = P.sinks > 0 ? 0 : low; j <= pos; ++j) {
      if (j < low && j >= P.sinks) j = low;
      const int page = P.c.table[b * P.c.table_stride + j / P.c.page_size];
      if (page < 0 || page >= P.c.num_pages) {
        ok = false;
        break;
      }
      const int64_t at = page * P.c.page_stride + (j % P.c.page_size) * P.c.token_stride + hk * P.c.head_stride + lane * E;
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) s += qv[e] * to_float(static_cast<const T*>(P.c.k)[at + e]);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= P.scale;
      const float mn = fmaxf(m, s);
      const float f = mn == -INFINITY ? 1.0f : expf(m - mn), p = mn == -INFINITY ? 0.0f : expf(s - mn);
      m = mn;
      l = l * f + p;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * to_float(static_cast<const T*>(P.c.v)[at + e]);
    }
  }
  if (!ok && lane == 0 && i == 0 && hq == 0 && P.c.err) atomicAdd(P.c.err, 1);
#pragma unroll
  for (int e = 0; e < E; ++e) from_float(!ok ? nan : l == 0.0f ? 0.0f : o[e] / l, out[e]);
  if (lane == 0 && P.lse) P.lse[(static_cast<int64_t>(b) * P.c.n + i) * P.q_heads + hq] = !ok ? nan : m + logf(l);
}

// ------------------------------------------------------------ host side

rlk_status check_cache(const rlk_kv_cache* c) {
  if (!c) return fail(RLK_EINVAL, "cache is NULL");
  if (c->B < 0 || c->B >= (1 << 16)) return fail(RLK_EINVAL, "B = %lld must be in 0..65535", (long long)c->B);
  if (c->n < 0 || c->n >= (1 << 16)) return fail(RLK_EINVAL, "n = %d must be in 0..65535", c->n);
  if (c->dtype != RLK_DT_BF16 && c->dtype != RLK_DT_F16)
    return fail(RLK_EINVAL, "dtype %d must be RLK_DT_BF16 or RLK_DT_F16", c->dtype);
  if (c->head_dim != 64 && c->head_dim != 128) return fail(RLK_EINVAL, "head_dim %d must be 64 or 128", c->head_dim);
  if (c->kv_heads < 1 || c->kv_heads > 1024) return fail(RLK_EINVAL, "kv_heads %d must be in 1..1024", c->kv_heads);
  if (c->page_size < 1) return fail(RLK_EINVAL, "page_size %d must be >= 1", c->page_size);
  if (c->max_pages < 0) return fail(RLK_EINVAL, "max_pages %d < 0", c->max_pages);
  if (static_cast<int64_t>(c->max_pages) * c->page_size >= (int64_t(1) << 31))
    return fail(RLK_EINVAL, "max_pages %d * page_size %d must be below 2^31", c->max_pages, c->page_size);
  if (c->num_pages < 0) return fail(RLK_EINVAL, "num_pages %lld < 0", (long long)c->num_pages);
  if (c->B == 0 || c->n == 0) return RLK_OK;
  if (c->table_stride < c->max_pages)
    return fail(RLK_EINVAL, "table_stride %lld < max_pages %d", (long long)c->table_stride, c->max_pages);
  if (c->num_pages > 0) {
    if (!c->k || !c->v) return fail(RLK_EINVAL, "k or v of the cache is NULL");
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return fail(RLK_EALIGN, "k or v of the cache is not 16-byte aligned");
    if (c->page_stride % 8 || c->token_stride % 8 || c->head_stride % 8)
      return fail(RLK_EALIGN, "a stride of the cache is not a multiple of 8 elements");
  }
  if (c->max_pages > 0 && !c->page_table) return fail(RLK_EINVAL, "page_table is NULL");
  if (!c->lens) return fail(RLK_EINVAL, "lens is NULL");
  if (!aligned(c->page_table, 4) || !aligned(c->lens, 4) || !aligned(c->new_lens, 4) || !aligned(c->err_count, 4))
    return fail(RLK_EALIGN, "page_table, lens, new_lens or err_count is not 4-byte aligned");
  return RLK_OK;
}

rlk_status check_bth(const void* p, const rlk_bth_strides* s, const char* what) {
  if (!p || !s) return fail(RLK_EINVAL, "%s or its strides are NULL", what);
  if (!aligned(p, 16)) return fail(RLK_EALIGN, "%s is not 16-byte aligned", what);
  if (s->batch % 8 || s->token % 8 || s->head % 8)
    return fail(RLK_EALIGN, "a stride of %s is not a multiple of 8 elements", what);
  return RLK_OK;
}

PagedParams paged_params(const rlk_kv_cache* c) {
  PagedParams P{};
  P.k = c->k;
  P.v = c->v;
  P.num_pages = c->num_pages;
  P.page_stride = c->page_stride;
  P.token_stride = c->token_stride;
  P.head_stride = c->head_stride;
  P.page_size = c->page_size;
  P.kv_heads = c->kv_heads;
  P.max_pages = c->max_pages;
  P.table = c->page_table;
  P.table_stride = c->table_stride;
  P.lens = c->lens;
  P.new_lens = c->new_lens;
  P.n = c->n;
  P.err = c->err_count;
  return P;
}

template <class T, int D>
void launch_attn(const AttnParams& P, int64_t B, cudaStream_t st) {
  const int64_t warps = B * P.c.n * P.q_heads;
  attn_kernel<T, D><<<static_cast<unsigned>((warps + 3) / 4), 128, 0, st>>>(P, warps);
}

}  // namespace rlk

using namespace rlk;

extern "C" {

rlk_status rlk_kv_append(const rlk_kv_cache* cache, const void* k, const rlk_bth_strides* k_strides,
                         const void* v, const rlk_bth_strides* v_strides, void* stream) {
  rlk_status s = check_cache(cache);
  if (s != RLK_OK || cache->B == 0 || cache->n == 0) return s;
  if ((s = check_bth(k, k_strides, "k")) != RLK_OK) return s;
  if ((s = check_bth(v, v_strides, "v")) != RLK_OK) return s;
  AppendParams P{};
  P.c = paged_params(cache);
  P.ksrc = static_cast<const uint4*>(k);
  P.vsrc = static_cast<const uint4*>(v);
  P.ks = {k_strides->batch / 8, k_strides->token / 8, k_strides->head / 8};
  P.vs = {v_strides->batch / 8, v_strides->token / 8, v_strides->head / 8};
  P.row16 = cache->head_dim / 8;
  P.total = cache->B * cache->n * cache->kv_heads * P.row16;
  const int64_t blocks = (P.total + 255) / 256;
  if (blocks >= (int64_t(1) << 31)) return fail(RLK_EINVAL, "B * n * kv_heads is too large for one call");
  append_kernel<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(P);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(RLK_ECUDA, "kernel launch: %s", cudaGetErrorString(e));
  return RLK_OK;
}

rlk_status rlk_paged_attention_workspace(int64_t B, int32_t n, int32_t q_heads, int32_t head_dim,
                                         int64_t max_tokens, size_t* bytes) {
  if (B < 0 || n < 0 || q_heads < 0 || head_dim < 0 || max_tokens < 0) return fail(RLK_EINVAL, "a size is negative");
  if (!bytes) return fail(RLK_EINVAL, "bytes is NULL");
  *bytes = 0;
  return RLK_OK;
}

rlk_status rlk_paged_attention(const rlk_kv_cache* cache, const void* q, const rlk_bth_strides* q_strides,
                               int32_t q_heads, float scale, int32_t window, int32_t sinks, void* out,
                               const rlk_bth_strides* out_strides, float* out_lse, void* workspace,
                               void* stream) {
  rlk_status s = check_cache(cache);
  if (s != RLK_OK) return s;
  if (q_heads < 1 || q_heads % cache->kv_heads || q_heads > 128 * cache->kv_heads)
    return fail(RLK_EINVAL, "q_heads %d must be 1 to 128 times kv_heads %d", q_heads, cache->kv_heads);
  if (!isfinite(scale)) return fail(RLK_EINVAL, "scale %g must be finite", (double)scale);
  if (window < 0 || sinks < 0) return fail(RLK_EINVAL, "window %d and sinks %d must be >= 0", window, sinks);
  if (cache->B == 0 || cache->n == 0) return RLK_OK;
  if ((s = check_bth(q, q_strides, "q")) != RLK_OK) return s;
  if ((s = check_bth(out, out_strides, "out")) != RLK_OK) return s;
  if ((s = check_out(out_lse, "out_lse", false)) != RLK_OK) return s;
  (void)workspace;
  AttnParams P{};
  P.c = paged_params(cache);
  P.q = q;
  P.out = out;
  P.qs = *q_strides;
  P.os = *out_strides;
  P.q_heads = q_heads;
  P.scale = scale;
  P.window = window;
  P.sinks = sinks;
  P.lse = out_lse;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = cache->dtype == RLK_DT_BF16, wide = cache->head_dim == 128;
  if (bf && wide) launch_attn<__nv_bfloat16, 128>(P, cache->B, st);
  else if (bf) launch_attn<__nv_bfloat16, 64>(P, cache->B, st);
  else if (wide) launch_attn<__half, 128>(P, cache->B, st);
  else launch_attn<__half, 64>(P, cache->B, st);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(RLK_ECUDA, "kernel launch: %s", cudaGetErrorString(e));
  return RLK_OK;
}

}  // extern "C"
