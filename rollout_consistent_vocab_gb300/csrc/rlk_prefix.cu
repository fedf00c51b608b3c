// rlk_prefix.cu -- attention of sequences that share a prefix: the shared tokens' part,
// for all queries of a group at once.
//
// plan_kernel looks the groups and lengths over.  The shared tokens of a group, rounded
// down to 32, go in pieces of a length that depends on theirs alone; a piece's result
// (maximum, sum, weighted sum of values of each query row) goes to the workspace.  Then
// paged attention takes every sequence's other tokens, and its join adds the pieces first.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "rlk_rollout.h"
#include "rlk_device.cuh"
#include "rlk_host.h"
#include "rlk_paged.h"

namespace rlk {

constexpr int PREFIX_STEP = 32;          // shared tokens come in multiples of this

// A group as the plan leaves it: its first sequence, how many, the shared tokens to take, and
// their pieces (0: nothing to do).
struct alignas(16) GroupPlan { int seq0, seqs, shared, pieces; };

struct PrefixParams {
  PagedParams c;
  const int32_t* group_start;
  const int32_t* shared_lens;
  int groups, max_shared;
  int64_t B;
  int32_t* first;               // [B], as in PrefixParts
  GroupPlan* plan;              // [groups]
  int32_t* busy;                // [groups] whether a sequence has new tokens
  uint32_t* base;               // [groups + 1] items before each group
  const void* q;
  rlk_bth_strides qs;
  int q_heads, group;           // group: query heads of a kv head
  int rows;                     // n * group: of a sequence and kv head
  int max_pieces;
  float c2;                     // scale * log2(e)
  float2* ml;
  float* o;
};

// ------------------------------------------------------------ the plan

constexpr int PLAN_THREADS = 1024;

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const PrefixParams P) {
  __shared__ uint32_t scan[PLAN_THREADS];
  const int tid = threadIdx.x, G = P.groups;
  const int64_t tokens = static_cast<int64_t>(P.c.max_pages) * P.c.page_size;
  bool fault = false;
  for (int g = tid; g < G; g += PLAN_THREADS) {
    const int a = P.group_start[g], e = P.group_start[g + 1];
    fault |= a < 0 || e < a || e > P.B;
    P.busy[g] = 0;
  }
  fault = __syncthreads_or(fault);
  for (int b = tid; b < P.B; b += PLAN_THREADS) {
    int len, nnew, first = -1;
    if (!fault && seq_lens(P.c, b, len, nnew)) {
      // the last group that begins at or before b
      int lo = -1, hi = G;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (P.group_start[mid] <= b) lo = mid;
        else hi = mid;
      }
      if (lo < 0 || b >= P.group_start[lo + 1]) {
        first = 0;
      } else {
        const int shared = P.shared_lens[lo];
        if (shared >= 0 && shared <= P.max_shared && shared <= tokens && (nnew == 0 || len - nnew >= shared)) {
          first = shared / PREFIX_STEP * PREFIX_STEP;
          if (nnew > 0 && first > 0) P.busy[lo] = 1;
        }
      }
    }
    P.first[b] = first;
  }
  __syncthreads();
  const int per = (G + PLAN_THREADS - 1) / PLAN_THREADS, g0 = min(G, tid * per), g1 = min(G, g0 + per);
  uint32_t mine = 0;
  for (int g = g0; g < g1; ++g) {
    GroupPlan p{0, 0, 0, 0};
    if (!fault && P.busy[g]) {
      p.seq0 = P.group_start[g];
      p.seqs = P.group_start[g + 1] - p.seq0;
      p.shared = min(max(P.shared_lens[g], 0), P.max_shared) / PREFIX_STEP * PREFIX_STEP;
      p.pieces = pieces_of(p.shared);
    }
    P.plan[g] = p;
    mine += p.pieces;
  }
  scan[tid] = mine;
  __syncthreads();
  for (int o = 1; o < PLAN_THREADS; o <<= 1) {
    const uint32_t x = tid >= o ? scan[tid - o] : 0u;
    __syncthreads();
    scan[tid] += x;
    __syncthreads();
  }
  uint32_t run = scan[tid] - mine;
  for (int g = g0; g < g1; ++g) {
    P.base[g] = run;
    run += P.plan[g].pieces;
  }
  if (tid == PLAN_THREADS - 1) P.base[G] = run;
}

// ------------------------------------------------------------ the shared tokens

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <class T> struct WeightUnit;    // paged attention's: weights are in units of 2^-OFF of the reference
template <> struct WeightUnit<__nv_bfloat16> { static constexpr float OFF = 0.0f; };
template <> struct WeightUnit<__half> { static constexpr float OFF = 8.0f; };

// A warp per query row and piece, one token after the other.
template <class T, int D>
__global__ void __launch_bounds__(256) prefix_kernel(const PrefixParams P) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  for (int g = 0; g < P.groups; ++g) {
    const GroupPlan pl = P.plan[g];
    const int size = piece_tokens(pl.shared);
    const int64_t all = static_cast<int64_t>(pl.seqs) * P.c.kv_heads * P.rows * pl.pieces;
    for (int64_t w = blockIdx.x * 8ll + threadIdx.x / 32; w < all; w += warps) {
      const int piece = static_cast<int>(w % pl.pieces);
      int64_t rest = w / pl.pieces;
      const int row = static_cast<int>(rest % P.rows);
      rest /= P.rows;
      const int h = static_cast<int>(rest % P.c.kv_heads), b = pl.seq0 + static_cast<int>(rest / P.c.kv_heads);
      const int i = row / P.group, nnew = P.c.new_lens ? P.c.new_lens[b] : P.c.n;
      if (P.first[b] < 0 || i >= nnew) continue;
      const T* q = static_cast<const T*>(P.q) + b * P.qs.batch + i * P.qs.token + (h * P.group + row % P.group) * P.qs.head + lane * E;
      float qv[E], o[E] = {}, m = -INFINITY, l = 0.0f;
      for (int e = 0; e < E; ++e) qv[e] = to_float(q[e]);
      for (int t = piece * size; t < min(pl.shared, (piece + 1) * size); ++t) {
        const int page = P.c.table[pl.seq0 * P.c.table_stride + t / P.c.page_size];
        if (page < 0 || page >= P.c.num_pages) {
          l = NAN;
          if (lane == 0 && P.c.err) atomicAdd(P.c.err, 1);
          break;
        }
        const int64_t at = page * P.c.page_stride + t % P.c.page_size * P.c.token_stride + h * P.c.head_stride + lane * E;
        const T* k = static_cast<const T*>(P.c.k) + at;
        const T* v = static_cast<const T*>(P.c.v) + at;
        float x = 0.0f;
        for (int e = 0; e < E; ++e) x += qv[e] * to_float(k[e]);
        for (int z = 16; z > 0; z >>= 1) x += __shfl_xor_sync(0xffffffffu, x, z);
        x *= P.c2;
        const float top = fmaxf(m, x);
        const float old = m == -INFINITY ? 0.0f : exp2f(m - top), wt = exp2f(x - (top == -INFINITY ? 0.0f : top) + WeightUnit<T>::OFF);
        m = top;
        l = l * old + wt;
        for (int e = 0; e < E; ++e) o[e] = o[e] * old + wt * to_float(v[e]);
      }
      const int64_t slot = ((static_cast<int64_t>(b) * P.c.kv_heads + h) * P.rows + row) * P.max_pieces + piece;
      if (lane == 0) P.ml[slot] = make_float2(m, l);
      for (int e = 0; e < E; ++e) P.o[slot * D + lane * E + e] = o[e];
    }
  }
}

// ------------------------------------------------------------ host side

// The workspace, in this order; each part on a line of its own.
struct PrefixLayout {
  size_t first, plan, busy, base, ml, o, rest, bytes;
  int pieces;
};
static size_t lined(size_t x) { return (x + 127) / 128 * 128; }
static PrefixLayout prefix_layout(int64_t B, int64_t n, int64_t q_heads, int64_t head_dim, int groups, int max_shared, size_t rest) {
  PrefixLayout y{};
  for (const int top : {max_shared < 8191 ? max_shared : 8191, max_shared < 32767 ? max_shared : 32767, max_shared}) {
    const int pieces = pieces_of(top / PREFIX_STEP * PREFIX_STEP);
    y.pieces = pieces > y.pieces ? pieces : y.pieces;
  }
  const size_t slots = static_cast<size_t>(B) * n * q_heads * y.pieces;
  y.first = 0;
  y.plan = y.first + lined(static_cast<size_t>(B) * 4);
  y.busy = y.plan + lined(static_cast<size_t>(groups) * sizeof(GroupPlan));
  y.base = y.busy + lined(static_cast<size_t>(groups) * 4);
  y.ml = y.base + lined(static_cast<size_t>(groups + 1) * 4);
  y.o = y.ml + lined(slots * 8);
  y.rest = y.o + lined(slots * head_dim * 4);
  y.bytes = y.rest + rest + 128;         // (the caller's memory may begin between two lines)
  return y;
}

}  // namespace rlk

using namespace rlk;

extern "C" {

rlk_status rlk_prefix_attention_workspace(int64_t B, int32_t n, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                          int64_t max_tokens, int32_t groups, int32_t max_shared, size_t* bytes) {
  size_t rest = 0;
  const rlk_status s = rlk_paged_attention_workspace(B, n, q_heads, kv_heads, head_dim, max_tokens, bytes ? &rest : nullptr);
  if (s != RLK_OK) return s;
  if (groups < 0 || groups >= (1 << 16)) return fail(RLK_EINVAL, "groups %d must be in 0..65535", groups);
  if (max_shared < 0 || max_shared > max_tokens)
    return fail(RLK_EINVAL, "max_shared %d must be in 0..%lld", max_shared, (long long)max_tokens);
  *bytes = B == 0 || n == 0 || q_heads == 0 ? 0 : prefix_layout(B, n, q_heads, head_dim, groups, max_shared, rest).bytes;
  return RLK_OK;
}

rlk_status rlk_prefix_attention(const rlk_kv_cache* cache, const rlk_prefix_groups* groups, const void* q,
                                const rlk_bth_strides* q_strides, int32_t q_heads, float scale, void* out,
                                const rlk_bth_strides* out_strides, float* out_lse, void* workspace, void* stream) {
  rlk_status s = check_cache(cache);
  if (s != RLK_OK) return s;
  if (!groups) return fail(RLK_EINVAL, "groups is NULL");
  if (q_heads < 1 || q_heads % cache->kv_heads || q_heads > 128 * cache->kv_heads)
    return fail(RLK_EINVAL, "q_heads %d must be 1 to 128 times kv_heads %d", q_heads, cache->kv_heads);
  if (!isfinite(scale)) return fail(RLK_EINVAL, "scale %g must be finite", (double)scale);
  const int64_t tokens = static_cast<int64_t>(cache->max_pages) * cache->page_size;
  size_t rest = 0, bytes = 0;
  if ((s = rlk_prefix_attention_workspace(cache->B, cache->n, q_heads, cache->kv_heads, cache->head_dim, tokens, groups->groups,
                                          groups->max_shared, &bytes)) != RLK_OK)
    return s;
  if (!aligned(groups->group_start, 4) || !aligned(groups->shared_lens, 4))
    return fail(RLK_EALIGN, "group_start or shared_lens is not 4-byte aligned");
  if (cache->B == 0 || cache->n == 0) return RLK_OK;
  if (groups->groups > 0 && (!groups->group_start || !groups->shared_lens))
    return fail(RLK_EINVAL, "group_start or shared_lens is NULL");
  if ((s = check_bth(q, q_strides, "q")) != RLK_OK) return s;
  if ((s = check_bth(out, out_strides, "out")) != RLK_OK) return s;
  if ((s = check_out(out_lse, "out_lse", false)) != RLK_OK) return s;
  if (!workspace) return fail(RLK_EINVAL, "workspace is NULL");
  if (!aligned(workspace, 16)) return fail(RLK_EALIGN, "workspace is not 16-byte aligned");
  rlk_paged_attention_workspace(cache->B, cache->n, q_heads, cache->kv_heads, cache->head_dim, tokens, &rest);
  const PrefixLayout y = prefix_layout(cache->B, cache->n, q_heads, cache->head_dim, groups->groups, groups->max_shared, rest);
  char* ws = reinterpret_cast<char*>(lined(reinterpret_cast<size_t>(workspace)));
  PrefixParams P{};
  P.c = paged_params(cache);
  P.group_start = groups->group_start;
  P.shared_lens = groups->shared_lens;
  P.groups = groups->groups;
  P.max_shared = groups->max_shared;
  P.B = cache->B;
  P.first = reinterpret_cast<int32_t*>(ws + y.first);
  P.plan = reinterpret_cast<GroupPlan*>(ws + y.plan);
  P.busy = reinterpret_cast<int32_t*>(ws + y.busy);
  P.base = reinterpret_cast<uint32_t*>(ws + y.base);
  P.ml = reinterpret_cast<float2*>(ws + y.ml);
  P.o = reinterpret_cast<float*>(ws + y.o);
  P.q = q;
  P.qs = *q_strides;
  P.q_heads = q_heads;
  P.group = q_heads / cache->kv_heads;
  P.rows = cache->n * P.group;
  P.max_pieces = y.pieces;
  P.c2 = scale * 1.4426950408889634f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  plan_kernel<<<1, PLAN_THREADS, 0, st>>>(P);
  if (y.pieces > 0 && groups->groups > 0) {
    const bool bf = cache->dtype == RLK_DT_BF16;
    if (cache->head_dim == 128) {
      if (bf) prefix_kernel<__nv_bfloat16, 128><<<152 * 8, 256, 0, st>>>(P);
      else prefix_kernel<__half, 128><<<152 * 8, 256, 0, st>>>(P);
    } else {
      if (bf) prefix_kernel<__nv_bfloat16, 64><<<152 * 8, 256, 0, st>>>(P);
      else prefix_kernel<__half, 64><<<152 * 8, 256, 0, st>>>(P);
    }
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(RLK_ECUDA, "kernel launch: %s", cudaGetErrorString(e));
  const PrefixParts parts{P.first, P.ml, P.o, y.pieces};
  return paged_attention(cache, q, q_strides, q_heads, scale, 0, 0, out, out_strides, out_lse, ws + y.rest, &parts, stream);
}

}  // extern "C"
