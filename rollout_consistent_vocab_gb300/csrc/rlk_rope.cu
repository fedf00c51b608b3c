// rlk_rope.cu -- the rotation of heads by position: alone, and on the way of keys
// into the paged cache.
//
// Angles.  A frequency is kept as a 64-bit fraction of a turn a position, so that
// position * frequency in 64-bit arithmetic is the angle modulo a turn, exact
// but for the frequency's own rounding (2^-52 of it: a rounded constant and a rounded product;
// a negative one is the positive one's complement) whatever the position.  Its upper
// 32 bits, taken to the nearest quarter turn, leave at most an eighth: sine and
// cosine of that, to float32's accuracy, then the quarters by exchange and sign.
//
// A block takes a few tokens: a thread has the same 16 elements of a few of their heads, whose loads go out
// first; meanwhile all threads take one sine and cosine per token and pair into shared memory,
// and those of the cache's places are looked up.  Bound by memory: 4 x 4096 tokens of 32 heads of 128
// elements, bf16, 268 MB, 0.041 ms = 6.5 TB/s; three axes, 28 heads, 117 MB, 0.0174 ms = 6.7 TB/s;
// append of 16 x 2048 tokens, 32 query heads on 8, 755 MB, 0.1175 ms = 6.4 TB/s.  Blocks of 256 threads:
// 0.041, 0.0185, 0.141 ms; loads behind the angles: 0.047, 0.025, 0.160.  The append's loads wait in shared
// memory: in registers three heads of a thread were under way, and it took 0.127 ms; 3, 4, 5, 6, 8 and 10 heads there
// 0.121, 0.123, 0.125, 0.1175, 0.1185, 0.125.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "rlk_rollout.h"
#include "rlk_host.h"
#include "rlk_paged.h"

namespace rlk {

constexpr int ROPE_THREADS = 128;
// heads of a thread whose loads are under way together: alone, and in the append
constexpr int ROPE_AHEAD = 4, APPEND_AHEAD = 6;
constexpr int ROPE_TOKENS = 8;           // of a block, at most

struct Turns {
  unsigned long long turn[RLK_ROPE_MAX_DIM / 2];   // 2^64 / (turns a position)
  uint8_t axis[RLK_ROPE_MAX_DIM / 2];
  const int32_t* positions;              // [axes][B][n] or NULL
  int64_t axis_stride;                   // B * n
  int pairs;
  bool interleaved, inverse;
};
struct HeadRows {                        // [B][n][heads][head_dim] in bytes
  const char* p;
  int64_t batch, token, head;
};

__device__ __forceinline__ float2 cos_sin(unsigned long long turn, int position) {
  const unsigned long long u = turn * static_cast<unsigned long long>(static_cast<long long>(position));
  const uint32_t hi = static_cast<uint32_t>(u >> 32), quarter = (hi + (1u << 29)) >> 30;
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(hi - (quarter << 30))) * 4.656612873077393e-10f, &s, &c);   // 2^-31 half turns
  if (quarter & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

template <class T> struct Eight;         // eight elements in registers as they lie in memory
template <> struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const char* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void store(char* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
};
struct Eight16 {
  uint4 w;
  __device__ __forceinline__ void load(const char* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void store(char* p) const { *reinterpret_cast<uint4*>(p) = w; }
};
template <> struct Eight<__nv_bfloat16> : Eight16 {
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[2 * j] = __uint_as_float(u[j] << 16), v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 r = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      u[j] = *reinterpret_cast<const uint32_t*>(&r);
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ void fill(float x) {
    const float v[8] = {x, x, x, x, x, x, x, x};
    set(v);
  }
};
template <> struct Eight<__half> : Eight16 {
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
      v[2 * j] = f.x, v[2 * j + 1] = f.y;
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 r = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
      u[j] = *reinterpret_cast<const uint32_t*>(&r);
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ void fill(float x) {
    const float v[8] = {x, x, x, x, x, x, x, x};
    set(v);
  }
};

__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
  const float a = __fmaf_rn(x, c, -__fmul_rn(y, s));
  y = __fmaf_rn(x, s, __fmul_rn(y, c));
  x = a;
}
// The thread's 16 elements: pairs between the two eights, or of neighbours in each.
template <class T>
__device__ __forceinline__ void turn(Eight<T>& lo, Eight<T>& hi, const float (&c)[8], const float (&s)[8], bool interleaved) {
  float a[8], b[8];
  lo.get(a);
  hi.get(b);
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      turn_pair(a[2 * j], a[2 * j + 1], c[j], s[j]);
      turn_pair(b[2 * j], b[2 * j + 1], c[4 + j], s[4 + j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) turn_pair(a[j], b[j], c[j], s[j]);
  }
  lo.set(a);
  hi.set(b);
}

struct RopeParams {
  Turns t;
  HeadRows x, out;
  int64_t tokens;                        // B * n
  uint32_t n;
  int heads, items;                      // items: 16-element pieces of a head
  int per;                               // tokens of a block
  bool in_place;
};

// The cosines and sines of a block's tokens, [token][cos, sin][pair]; place(token) is where positions has none.
template <class Place>
__device__ __forceinline__ void block_turns(const Turns& t, float* cs, int tokens, int64_t t0, Place place) {
  for (int e = threadIdx.x; e < tokens * t.pairs; e += ROPE_THREADS) {
    const int k = e / t.pairs, j = e - k * t.pairs;
    const int position = t.positions ? __ldg(t.positions + t.axis[j] * t.axis_stride + t0 + k) : place(k);
    const float2 v = cos_sin(t.turn[j], position);
    cs[k * (2 * t.pairs) + j] = v.x;
    cs[k * (2 * t.pairs) + t.pairs + j] = t.inverse ? -v.y : v.y;
  }
}
// Where a thread's two eights lie in a head, in elements, and its pairs' factors.
struct Item { int lo, hi; bool turns; };
__device__ __forceinline__ Item item_of(const Turns& t, int it) {
  const bool turns = it * 8 < t.pairs;
  return turns && !t.interleaved ? Item{it * 8, t.pairs + it * 8, true} : Item{it * 16, it * 16 + 8, turns};
}
__device__ __forceinline__ void load_factors(const Turns& t, const float* cs, int k, int it, float (&c)[8], float (&s)[8]) {
  const float4* p = reinterpret_cast<const float4*>(cs + k * (2 * t.pairs) + it * 8);   // (pairs is a multiple of 8)
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float4 x = p[j], y = p[t.pairs / 4 + j];
    c[4 * j] = x.x, c[4 * j + 1] = x.y, c[4 * j + 2] = x.z, c[4 * j + 3] = x.w;
    s[4 * j] = y.x, s[4 * j + 1] = y.y, s[4 * j + 2] = y.z, s[4 * j + 3] = y.w;
  }
}

template <class T>
__global__ void __launch_bounds__(ROPE_THREADS, sizeof(T) == 4 ? 4 : 6) rope_kernel(const __grid_constant__ RopeParams P) {
  __shared__ __align__(16) float cs[ROPE_TOKENS * RLK_ROPE_MAX_DIM];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * P.per;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(P.per), P.tokens - t0));
  // the threads as [head][token][item]
  const int row = tokens * P.items, slots = ROPE_THREADS / row;
  const int h0 = threadIdx.x / row, rest = threadIdx.x - h0 * row, k = rest / P.items, it = rest - k * P.items;
  const Item e = item_of(P.t, it);
  const bool works = h0 < slots && (e.turns || !P.in_place);
  const uint32_t at = static_cast<uint32_t>(t0) + k, b = at / P.n, i = at - b * P.n;     // (B * n is below 2^32)
  const char* src = P.x.p + b * P.x.batch + i * P.x.token;
  char* dst = const_cast<char*>(P.out.p) + b * P.out.batch + i * P.out.token;
  const int heads = works ? P.heads : 0;
  Eight<T> lo[ROPE_AHEAD], hi[ROPE_AHEAD];
  auto load = [&](int h) {
#pragma unroll
    for (int j = 0; j < ROPE_AHEAD; ++j)
      if (h + j * slots < heads) {
        const char* p = src + (h + j * slots) * P.x.head;
        lo[j].load(p + e.lo * sizeof(T));
        hi[j].load(p + e.hi * sizeof(T));
      }
  };
  load(h0);                              // (under way while the angles are taken)
  block_turns(P.t, cs, tokens, t0, [](int) { return 0; });
  __syncthreads();
  float c[8], s[8];
  if (e.turns && works) load_factors(P.t, cs, k, it, c, s);
  for (int h = h0; h < heads;) {
#pragma unroll
    for (int j = 0; j < ROPE_AHEAD; ++j)
      if (h + j * slots < heads) {
        if (e.turns) turn(lo[j], hi[j], c, s, P.t.interleaved);
        char* p = dst + (h + j * slots) * P.out.head;
        lo[j].store(p + e.lo * sizeof(T));
        hi[j].store(p + e.hi * sizeof(T));
      }
    h += slots * ROPE_AHEAD;
    load(h);
  }
}

// ------------------------------------------------------------ append

// 16 bytes on their way into shared memory, for the thread itself.
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

struct AppendRopeParams {
  Turns t;
  PagedParams c;
  HeadRows k, v, q, q_out;
  int64_t tokens;
  int q_heads, items, per;
};

template <class T>
__global__ void __launch_bounds__(ROPE_THREADS, 7) append_rope_kernel(const __grid_constant__ AppendRopeParams P) {
  __shared__ uint4 under_way[APPEND_AHEAD][2][ROPE_THREADS];       // each thread's own
  __shared__ __align__(16) float cs[ROPE_TOKENS * 128];         // (a cache's heads have up to 128 elements)
  __shared__ int64_t place[ROPE_TOKENS];           // of the token's first head in the cache, in elements; -1: none
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * P.per;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(P.per), P.tokens - t0));
  // the threads as [head][token][item]
  const int row = tokens * P.items, slots = ROPE_THREADS / row;
  const int h0 = threadIdx.x / row, rest = threadIdx.x - h0 * row, k = rest / P.items, it = rest - k * P.items;
  const Item e = item_of(P.t, it);
  const uint32_t n = P.c.n;
  const uint32_t at = static_cast<uint32_t>(t0) + k;       // (B * n is below 2^32)
  const int b = static_cast<int>(at / n), i = static_cast<int>(at - b * n);
  int len, nnew;
  const bool fine = seq_lens(P.c, b, len, nnew), there = fine && i < nnew;
  // queries, keys, values; of a place without a token only the queries' places are written
  const int heads = h0 >= slots ? 0 : there ? P.q_heads + 2 * P.c.kv_heads : P.q_heads;
  const bool in_place = P.q.p == P.q_out.p;
  const int64_t lo_at = e.lo * static_cast<int64_t>(sizeof(T)), hi_at = e.hi * static_cast<int64_t>(sizeof(T));
  auto load = [&](int h) {
#pragma unroll 1
    for (int j = 0; j < APPEND_AHEAD; ++j) {
      const int g = h + j * slots;
      if (g >= heads || !there) continue;
      const int z = g < P.q_heads ? g : g < P.q_heads + P.c.kv_heads ? g - P.q_heads : g - P.q_heads - P.c.kv_heads;
      const HeadRows& r = g < P.q_heads ? P.q : g < P.q_heads + P.c.kv_heads ? P.k : P.v;
      const char* p = r.p + b * r.batch + i * r.token + z * r.head;
      copy16(&under_way[j][0][threadIdx.x], p + lo_at);
      copy16(&under_way[j][1][threadIdx.x], p + hi_at);
    }
  };
  load(h0);                              // (under way while places and angles are looked up)
  if (threadIdx.x < row && it == 0) {
    int64_t to = -1;
    if (there) {
      const int pos = len - nnew + i, number = pos / P.c.page_size;
      const int page = P.c.table[b * P.c.table_stride + number];
      if (page >= 0 && page < P.c.num_pages)
        to = page * P.c.page_stride + (pos - number * P.c.page_size) * P.c.token_stride;
    }
    place[k] = to;
    if (P.c.err && (fine ? there && to < 0 : i == 0)) atomicAdd(P.c.err, 1);
  }
  block_turns(P.t, cs, tokens, t0, [&](int z) {
    const uint32_t u = static_cast<uint32_t>(t0) + z, s = u / n;
    int l, m;
    return seq_lens(P.c, static_cast<int>(s), l, m) ? l - m + static_cast<int>(u - s * n) : 0;
  });
  __syncthreads();
  float c[8], s[8];
  if (e.turns && heads > 0) load_factors(P.t, cs, k, it, c, s);
  const int64_t to = place[k];
  for (int h = h0; h < heads;) {
    copies_wait();
#pragma unroll 1
    for (int j = 0; j < APPEND_AHEAD; ++j) {
      const int g = h + j * slots;
      if (g >= heads) break;
      Eight<T> lo, hi;
      if (there) lo.w = under_way[j][0][threadIdx.x], hi.w = under_way[j][1][threadIdx.x];
      char* dst;
      if (g < P.q_heads) {
        if (!there) {
          lo.fill(fine ? 0.0f : __int_as_float(0x7fc00000));
          hi = lo;
        } else if (e.turns) {
          turn(lo, hi, c, s, P.t.interleaved);
        } else if (in_place) {
          continue;
        }
        dst = const_cast<char*>(P.q_out.p) + b * P.q_out.batch + i * P.q_out.token + g * P.q_out.head;
      } else {
        if (to < 0) continue;
        const bool key = g < P.q_heads + P.c.kv_heads;
        const int z = key ? g - P.q_heads : g - P.q_heads - P.c.kv_heads;
        if (key && e.turns) turn(lo, hi, c, s, P.t.interleaved);
        dst = static_cast<char*>(const_cast<void*>(key ? P.c.k : P.c.v)) + (to + z * P.c.head_stride) * static_cast<int64_t>(sizeof(T));
      }
      lo.store(dst + lo_at);
      hi.store(dst + hi_at);
    }
    h += slots * APPEND_AHEAD;
    load(h);
  }
}

// ------------------------------------------------------------ host side

// The checks of a rotation of heads of `dim` elements, and its kernel form.
static rlk_status make_turns(const rlk_rope_args* r, int dim, int64_t B, int64_t n, bool need_positions, bool inverse, Turns* t) {
  if (!r) return fail(RLK_EINVAL, "rope is NULL");
  if (r->rot_dim < 16 || r->rot_dim > dim || r->rot_dim % 16)
    return fail(RLK_EINVAL, "rot_dim %d must be a multiple of 16, 16 to the heads' %d", r->rot_dim, dim);
  if (r->interleaved != 0 && r->interleaved != 1) return fail(RLK_EINVAL, "interleaved %d must be 0 or 1", r->interleaved);
  if (r->axes < 1 || r->axes > RLK_ROPE_MAX_AXES)
    return fail(RLK_EINVAL, "axes %d must be 1..%d", r->axes, RLK_ROPE_MAX_AXES);
  if (!r->inv_freq) return fail(RLK_EINVAL, "inv_freq is NULL");
  if (!aligned(r->inv_freq, 8)) return fail(RLK_EALIGN, "inv_freq is not 8-byte aligned");
  if (!aligned(r->positions, 4)) return fail(RLK_EALIGN, "positions is not 4-byte aligned");
  t->pairs = r->rot_dim / 2;
  for (int j = 0; j < t->pairs; ++j) {
    const double f = fabs(r->inv_freq[j]) * 0.15915494309189535;         // 1 / (2 pi)
    if (!isfinite(f)) return fail(RLK_EINVAL, "inv_freq[%d] must be finite", j);
    // (exact, in [0, 1); a small negative one's fraction would be a rounded number next to 1)
    const unsigned long long part = static_cast<unsigned long long>((f - floor(f)) * 18446744073709551616.0);
    t->turn[j] = r->inv_freq[j] < 0.0 ? 0ull - part : part;
    t->axis[j] = r->pair_axis ? r->pair_axis[j] : 0;
    if (t->axis[j] >= r->axes) return fail(RLK_EINVAL, "pair_axis[%d] = %d must be below axes %d", j, t->axis[j], r->axes);
  }
  if (need_positions && !r->positions) return fail(RLK_EINVAL, "positions is NULL");
  t->positions = r->positions;
  t->axis_stride = B * n;
  t->interleaved = r->interleaved != 0;
  t->inverse = inverse;
  return RLK_OK;
}

static HeadRows head_rows(const void* p, const rlk_bth_strides* s, int size) {
  return {static_cast<const char*>(p), s->batch * size, s->token * size, s->head * size};
}

// Tokens of a block: as many as leave a thread no more heads than it loads at once, but as many
// blocks as two to an SM, where there are as many tokens.
static int tokens_per_block(int64_t tokens, int items, int heads, int ahead) {
  int per = 1;
  while (per < ROPE_TOKENS && 2 * per * items <= ROPE_THREADS &&
         ROPE_THREADS / (2 * per * items) * ahead >= heads && tokens > 2 * 152 * 2 * per)
    per *= 2;
  return per;
}

}  // namespace rlk

using namespace rlk;

extern "C" {

rlk_status rlk_rope(const rlk_rope_args* rope, int64_t B, int64_t n, int32_t heads, int32_t head_dim, int32_t dtype,
                    const void* x, const rlk_bth_strides* x_strides, void* out, const rlk_bth_strides* out_strides,
                    int32_t inverse, void* stream) {
  if (B < 0 || n < 0 || heads < 0) return fail(RLK_EINVAL, "B, n or heads is negative");
  if (B >= (int64_t(1) << 32) || n >= (int64_t(1) << 32) || B * n >= (int64_t(1) << 32))
    return fail(RLK_EINVAL, "B * n must be below 2^32");
  if (head_dim < 16 || head_dim > RLK_ROPE_MAX_DIM || head_dim % 16)
    return fail(RLK_EINVAL, "head_dim %d must be a multiple of 16, 16 to %d", head_dim, RLK_ROPE_MAX_DIM);
  if (dtype != RLK_DT_F32 && dtype != RLK_DT_BF16 && dtype != RLK_DT_F16)
    return fail(RLK_EINVAL, "dtype %d must be RLK_DT_F32, RLK_DT_BF16 or RLK_DT_F16", dtype);
  if (inverse != 0 && inverse != 1) return fail(RLK_EINVAL, "inverse %d must be 0 or 1", inverse);
  RopeParams P{};
  const bool empty = B == 0 || n == 0 || heads == 0;
  rlk_status s = make_turns(rope, head_dim, B, n, !empty, inverse != 0, &P.t);
  if (s != RLK_OK || empty) return s;
  const int size = dtype == RLK_DT_F32 ? 4 : 2;
  const void* ptr[2] = {x, out};
  const rlk_bth_strides* st[2] = {x_strides, out_strides};
  for (int j = 0; j < 2; ++j) {
    const char* what = j ? "out" : "x";
    if (!ptr[j] || !st[j]) return fail(RLK_EINVAL, "%s or its strides are NULL", what);
    if (!aligned(ptr[j], 16)) return fail(RLK_EALIGN, "%s is not 16-byte aligned", what);
    if (st[j]->batch * size % 16 || st[j]->token * size % 16 || st[j]->head * size % 16)
      return fail(RLK_EALIGN, "a stride of %s is not a multiple of 16 bytes", what);
  }
  P.x = head_rows(x, x_strides, size);
  P.out = head_rows(out, out_strides, size);
  P.in_place = x == out;
  if (P.in_place && (P.x.batch != P.out.batch || P.x.token != P.out.token || P.x.head != P.out.head))
    return fail(RLK_EINVAL, "x and out are the same memory with different strides");
  P.tokens = B * n;
  P.n = static_cast<uint32_t>(n);
  P.heads = heads;
  P.items = head_dim / 16;
  P.per = tokens_per_block(P.tokens, P.items, heads, ROPE_AHEAD);
  const int64_t blocks = (P.tokens + P.per - 1) / P.per;
  if (blocks >= (int64_t(1) << 31)) return fail(RLK_EINVAL, "B * n is too large for one call");
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(blocks);
  if (dtype == RLK_DT_F32) rope_kernel<float><<<grid, ROPE_THREADS, 0, cs>>>(P);
  else if (dtype == RLK_DT_BF16) rope_kernel<__nv_bfloat16><<<grid, ROPE_THREADS, 0, cs>>>(P);
  else rope_kernel<__half><<<grid, ROPE_THREADS, 0, cs>>>(P);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(RLK_ECUDA, "kernel launch: %s", cudaGetErrorString(e));
  return RLK_OK;
}

rlk_status rlk_kv_append_rope(const rlk_kv_cache* cache, const rlk_rope_args* rope, const void* k,
                              const rlk_bth_strides* k_strides, const void* v, const rlk_bth_strides* v_strides,
                              const void* q, const rlk_bth_strides* q_strides, int32_t q_heads, void* q_out,
                              const rlk_bth_strides* q_out_strides, void* stream) {
  rlk_status s = check_cache(cache);
  if (s != RLK_OK) return s;
  if (q_heads < 0 || q_heads > 128 * cache->kv_heads)
    return fail(RLK_EINVAL, "q_heads %d must be 0 to 128 times kv_heads %d", q_heads, cache->kv_heads);
  AppendRopeParams P{};
  if ((s = make_turns(rope, cache->head_dim, cache->B, cache->n, false, false, &P.t)) != RLK_OK) return s;
  if (cache->B == 0 || cache->n == 0) return RLK_OK;
  if ((s = check_bth(k, k_strides, "k")) != RLK_OK) return s;
  if ((s = check_bth(v, v_strides, "v")) != RLK_OK) return s;
  P.k = head_rows(k, k_strides, 2);
  P.v = head_rows(v, v_strides, 2);
  if (q_heads > 0) {
    if ((s = check_bth(q, q_strides, "q")) != RLK_OK) return s;
    if ((s = check_bth(q_out, q_out_strides, "q_out")) != RLK_OK) return s;
    P.q = head_rows(q, q_strides, 2);
    P.q_out = head_rows(q_out, q_out_strides, 2);
    if (q == q_out && (P.q.batch != P.q_out.batch || P.q.token != P.q_out.token || P.q.head != P.q_out.head))
      return fail(RLK_EINVAL, "q and q_out are the same memory with different strides");
  }
  P.c = paged_params(cache);
  P.tokens = cache->B * cache->n;
  P.q_heads = q_heads;
  P.items = cache->head_dim / 16;
  P.per = tokens_per_block(P.tokens, P.items, q_heads + 2 * cache->kv_heads, APPEND_AHEAD);
  const int64_t blocks = (P.tokens + P.per - 1) / P.per;
  if (blocks >= (int64_t(1) << 31)) return fail(RLK_EINVAL, "B * n is too large for one call");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(blocks);
  if (cache->dtype == RLK_DT_BF16) append_rope_kernel<__nv_bfloat16><<<grid, ROPE_THREADS, 0, st>>>(P);
  else append_rope_kernel<__half><<<grid, ROPE_THREADS, 0, st>>>(P);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(RLK_ECUDA, "kernel launch: %s", cudaGetErrorString(e));
  return RLK_OK;
}

}  // extern "C"
