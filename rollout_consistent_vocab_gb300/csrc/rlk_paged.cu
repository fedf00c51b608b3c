// rlk_paged.cu -- the paged key-value cache: append, and the attention of new
// tokens over it.

#include <type_traits>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "rlk_rollout.h"
#include "rlk_device.cuh"
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
  int pieces;                   // ... of a token
  int per;                      // tokens of a block
  int64_t tokens;               // B * n
};

// A block copies the head rows of `per` tokens, a thread two pieces of 16 bytes of
// the keys and of the values at once: all its loads are out before its first store.
// Bound by memory: 16 x 2048 tokens (ragged) of 8 heads of 128 elements, 252 MB read
// and written, 0.043 ms = 5.8 TB/s; with one piece to a thread and 64-bit places
// 0.048 ms, with four pieces 0.043 ms, with eight 0.053 ms.
constexpr int APPEND_THREADS = 256, APPEND_PIECES = 2;
__global__ void __launch_bounds__(APPEND_THREADS) append_kernel(const AppendParams P) {
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * P.per;
  const uint32_t n = P.c.n, b0 = static_cast<uint32_t>(t0 / n), i0 = static_cast<uint32_t>(t0 - static_cast<int64_t>(b0) * n);
  const uint32_t tokens = static_cast<uint32_t>(min(static_cast<int64_t>(P.per), P.tokens - t0));
  const uint32_t all = tokens * P.pieces;
  for (uint32_t e0 = threadIdx.x; e0 < all; e0 += APPEND_THREADS * APPEND_PIECES) {
    int64_t at[APPEND_PIECES];
    bool there[APPEND_PIECES];
    uint4 k[APPEND_PIECES], v[APPEND_PIECES];
#pragma unroll
    for (int j = 0; j < APPEND_PIECES; ++j) {
      const uint32_t e = e0 + j * APPEND_THREADS;
      there[j] = false;
      if (e >= all) continue;
      const uint32_t tok = e / P.pieces, h = (e - tok * P.pieces) / P.row16, piece = e % P.row16;
      const uint32_t up = i0 + tok, b = b0 + up / n;
      const int i = static_cast<int>(up % n);
      const bool first = piece == 0 && h == 0;
      int len, nnew;
      if (!seq_lens(P.c, static_cast<int>(b), len, nnew)) {
        if (first && i == 0 && P.c.err) atomicAdd(P.c.err, 1);
        continue;
      }
      if (i >= nnew) continue;
      const int pos = len - nnew + i, place = pos / P.c.page_size;
      const int page = P.c.table[b * P.c.table_stride + place];
      if (page < 0 || page >= P.c.num_pages) {
        if (first && P.c.err) atomicAdd(P.c.err, 1);
        continue;
      }
      at[j] = (page * P.c.page_stride + (pos - place * P.c.page_size) * P.c.token_stride + h * P.c.head_stride) / 8 + piece;
      there[j] = true;
      k[j] = __ldcs(P.ksrc + b * P.ks.batch + i * P.ks.token + h * P.ks.head + piece);
      v[j] = __ldcs(P.vsrc + b * P.vs.batch + i * P.vs.token + h * P.vs.head + piece);
    }
#pragma unroll
    for (int j = 0; j < APPEND_PIECES; ++j) {
      if (!there[j]) continue;
      reinterpret_cast<uint4*>(const_cast<void*>(P.c.k))[at[j]] = k[j];
      reinterpret_cast<uint4*>(const_cast<void*>(P.c.v))[at[j]] = v[j];
    }
  }
}

// ------------------------------------------------------------ attention
//
// The tokens of a sequence go in units of 512, at fixed places.  A unit is one
// CTA's: its four lanes take the unit's slices in turn.  A lane is a copying warp, which
// brings keys and values into the lane's ring in shared memory (TMA), and a working
// warp for each 8 query rows, all of which read what it brought.  S^T = K Q^T and
// O^T += V^T P^T run on the tensor cores with the slice's 16 tokens (or dims) as rows
// and 8 query rows as columns, with a running maximum and sum per query row; then
// the lanes' shares are summed in order.  What a row gets from a unit
// therefore does not depend on the other rows, nor on anything outside the unit.
// The units of a group (4 units, 2048 tokens, at fixed places too) are folded in
// order; the groups of a sequence are joined in a fixed tree.  Who folds is
// free: the units of the whole batch are dealt out in equal runs, and a run that
// holds all of a group folds it itself, otherwise the units' results go to the
// workspace and the join folds them, with the same arithmetic.  So no result
// depends on the batch.
//
// What bounds it.  One new token: memory.  64 sequences of up to 8192 tokens, 32 query
// heads on 8 of 128 elements, 0.69 GB of keys and values: 0.123 ms = 5.6 TB/s; 4 of up
// to 131071, 1.28 GB: 0.203 ms = 6.3 TB/s.  Several new tokens (128 sequences of up to
// 4096, 5 each, 0.65 GB): 0.170 ms = 3.8 TB/s, bound by the latency of the working
// warps' instructions (a slice takes one about 1800 cycles, a unit's sum 3500; with 24
// and 32 rows of 128 elements they also spill, 100 and 220 bytes a thread).  A
// window of 1024 (64 sequences, 64 heads on 8 of 64 elements, f16, 0.13 GB): 0.050 ms =
// 2.6 TB/s, where the units are few and their ends count.
// The extent of the work is the sequence's and the call's, not the tile's: every tile of
// n's rows goes over all that the sequence's new tokens see.  So prompts pay for their
// masked half (4 of 2048 tokens: 2.8 ms), and single tokens beside a prompt for its tiles.
//
// Why mma.sync.  With 8 query rows to a tile the products are small: K and V pass
// once through shared memory into registers, and a score never leaves the warp that
// takes its exponential.  The same tree on tcgen05 (128 tokens as rows, 16 to 64 query
// rows as columns, scores and results in tensor memory) took 0.172 ms where this takes
// 0.123, 0.243 for 0.203, 0.330 for 0.170 and 0.125 for 0.050: the weights' way through
// tensor memory and back lies between the two products, and its code (96 to 198 KB
// against 73 to 82) ran into the instruction cache.

// (units of 2048 tokens: 0.137 ms for 0.125 in the first case above, 0.274 for 0.253 in the third,
// when they were chosen; requests of a few units were not compared)
constexpr int UNIT = 512;                // tokens of a unit
constexpr int GROUP = 4;                 // units of a group
constexpr int AW = 4;                    // lanes of a CTA: every fourth slice of a unit is one's
constexpr int NUM_SMS = 152;

// Rows of a tile: the n * (q_heads / kv_heads) query rows of a kv head, in tiles of
// 8 NT.  A lane is a copying warp and NT working warps of 8 rows each, which share
// what it copies: slices of 32 tokens, in halves of 16, STAGES halves in its ring.
// (One working warp with all the rows: 0.223 ms for 0.185 with 20 rows.)  Two CTAs to an
// SM with 8 rows; from 16 rows on one, with the longer rings (16 rows, 64 sequences of
// up to 4096 tokens: 0.089 ms with one CTA, about 0.12 with two).
constexpr int SL = 32;
constexpr int HALF = SL / 2;
template <int D, int NT>
struct Shape {
  static constexpr int CTAS = NT == 1 ? 2 : 1;               // per SM
  static constexpr int WORKERS = NUM_SMS * CTAS;
  static constexpr int THREADS = (NT + 1) * AW * 32;
  // Registers of a thread: as many at the launch as an SM has for its CTAs, then what
  // the copying warps give back goes to the working ones.
  static constexpr int REGS = 65536 / (CTAS * THREADS) / 8 * 8;
  static constexpr int REGS_COPY = 40, REGS_WORK = (REGS * (NT + 1) - REGS_COPY) / NT / 8 * 8;
  // A half in shared memory: D / 64 panels of 16 rows of 128 bytes, the pieces of 16
  // bytes swizzled (piece p of row r at p ^ (r & 7)); keys, then values.
  static constexpr int PANEL = HALF * 128;
  static constexpr int KEYS = D / 64 * PANEL;
  static constexpr int STAGE = 2 * KEYS;
  // (as many as there is room for; with 10 of 64 elements 24 and 32 rows took a fifth longer, with 6 to 9 not)
  static constexpr int STAGES = D == 128 ? (NT == 1 ? 3 : NT == 2 ? 6 : 5) : NT == 1 ? 6 : 8;
  static constexpr int SLOTS = D / 16;                       // fragments (four floats a thread) of a warp's result
  static constexpr int PASSES = D == 128 && NT % 2 == 0 ? 2 : 1;
  static constexpr int XCH = SLOTS / PASSES * AW * 512;      // ... of 8 rows, exchanged in so many passes
  static constexpr bool QS = D == 128 && NT == 4;            // queries in shared memory, not in registers
  static constexpr int Q_AT = AW * STAGES * STAGE + NT * XCH;
  static constexpr int SMEM = Q_AT + (QS ? NT * SLOTS * 32 * 8 : 0);
  static_assert(SLOTS % PASSES == 0 && SLOTS / PASSES % AW == 0, "every warp sums as many fragments in each pass");
  static_assert(CTAS * (SMEM + (AW + 1) * NT * 64 + AW * STAGES * 16 + 128 + 1024) <= 228 * 1024,
                "as many CTAs in the shared memory of an SM");
};
constexpr int WORKERS = NUM_SMS * 2;     // at most

struct AttnParams {
  PagedParams c;
  const void* q;
  void* out;
  rlk_bth_strides qs, os;       // elements
  int q_heads, group;           // group: query heads of a kv head
  int rows;                     // n * group
  int tiles;                    // row tiles
  int64_t B;
  float c2;                     // |scale| * log2(e)
  uint32_t q_sign;              // 0x80008000: the queries change sign (scale < 0)
  int box;                      // tokens of a copy: the largest power of 2, up to 16, that divides page_size
  bool head_first;              // the tensor maps' second place is the head, not the token
  int window, sinks;
  float* lse;
  float2* unit_ml;              // [workers][2 GROUP][8 NT]: maximum, sum
  float* unit_o;                // ... and the weighted sum of values [D]
  float2* group_ml;             // [B * kv_heads * tiles * groups][8 NT]
  float* group_o;
  uint32_t page_magic;          // 2^32 / page_size, rounded up (page_size 1: 2^32 - 1)
  uint32_t group_magic;         // 2^32 / group, rounded up (group 1: 0)
  uint32_t workers;             // CTAs of the main kernel
  int groups;                   // groups of the longest sequence that the table can hold
};
struct AttnMaps {
  CUtensorMap k, v;             // (element, token of the page, head, page), or the head before the token
};

// Units of t tokens; t may be anything up to 2^31 - 1.
__device__ __forceinline__ int units_of(int t) { return t / UNIT + (t % UNIT != 0); }

// What of a sequence is visible to its new tokens: units [0, us) for the sinks
// and [ul, ul + nu - us) up to the end.
struct Seq {
  int len, nnew, low, us, ul, nu;
  bool ok;
  __device__ __forceinline__ int unit(int li) const { return li < us ? li : ul + (li - us); }
  // the units of group g, by their place in the sequence's list
  __device__ __forceinline__ int first(int g) const { return g * GROUP < us ? g * GROUP : us + max(0, g * GROUP - ul); }
  __device__ __forceinline__ int past(int g) const {
    const int e = (g + 1) * GROUP;
    return e <= ul ? min(us, e) : us + min(e - ul, nu - us);
  }
};
__device__ __forceinline__ Seq load_seq(const AttnParams& P, int b) {
  Seq s;
  s.ok = seq_lens(P.c, b, s.len, s.nnew);
  if (!s.ok) s.len = s.nnew = 0;
  s.low = s.us = s.ul = s.nu = 0;
  if (s.ok && s.nnew > 0) {
    if (P.window > 0) {
      s.low = max(0, s.len - s.nnew - P.window + 1);
      s.ul = s.low / UNIT;
      s.us = min(units_of(min(P.sinks, s.len)), s.ul);
    }
    s.nu = s.us + units_of(s.len) - s.ul;
  }
  return s;
}

// The units of the batch (fewer than 2^31) in equal runs, the first ones one longer.
struct Runs {
  uint32_t len, more, workers;
  __device__ __forceinline__ Runs(uint32_t units, uint32_t most) {
    workers = min(units, most);
    len = workers ? units / workers : 0;
    more = workers ? units - len * workers : 0;
  }
  __device__ __forceinline__ uint32_t start(uint32_t k) const { return k * len + min(k, more); }
};
// ... and the run that a unit is in, by multiplication: u d for a 32-bit u and
// d = ceil(2^64 / divisor) has the quotient in its upper 64 bits.
struct RunOf : Runs {
  unsigned long long inv, inv1;          // of len (0: len is 1) and of len + 1
  __device__ __forceinline__ RunOf(uint32_t units, uint32_t most) : Runs(units, most) {
    inv = len > 1 ? ~0ull / len + 1 : 0ull;
    inv1 = ~0ull / (len + 1) + 1;        // len + 1 >= 2 where it is used
  }
  __device__ __forceinline__ uint32_t of(uint32_t u) const {
    const uint32_t cut = more * (len + 1);
    if (u < cut) return static_cast<uint32_t>(__umul64hi(u, inv1));
    return more + (inv ? static_cast<uint32_t>(__umul64hi(u - cut, inv)) : u - cut);
  }
};

// Units (per kv head and tile) of the sequences before each block of sequences,
// thread by thread, into scan[THREADS], and of them all; the whole CTA.
template <int THREADS>
__device__ __forceinline__ int seqs_per(const AttnParams& P) { return static_cast<int>((P.B + THREADS - 1) / THREADS); }
template <int THREADS>
__device__ __forceinline__ int64_t unit_sums(const AttnParams& P, int64_t* scan) {
  const int tid = threadIdx.x, lane = tid & 31, per = seqs_per<THREADS>(P);
  const int lo = static_cast<int>(min(P.B, static_cast<int64_t>(tid) * per));
  const int hi = static_cast<int>(min(P.B, static_cast<int64_t>(lo) + per));
  int64_t mine = 0;
  for (int b = lo; b < hi; ++b) mine += load_seq(P, b).nu;
  scan[tid] = mine;
  __syncthreads();
  if (tid < 32) {
    constexpr int N = THREADS / 32;
    int64_t sum = 0;
    for (int j = 0; j < N; ++j) sum += scan[lane * N + j];
    int64_t run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    if (lane == 31) scan[THREADS] = run;
    run -= sum;
    for (int j = 0; j < N; ++j) {
      const int64_t v = scan[lane * N + j];
      scan[lane * N + j] = run;
      run += v;
    }
  }
  __syncthreads();
  return scan[THREADS];
}
template <int THREADS>
__device__ __forceinline__ int64_t units_before(const AttnParams& P, const int64_t* scan, int b) {
  const int per = seqs_per<THREADS>(P), blk = b / per;
  int64_t run = scan[blk];
  for (int i = blk * per; i < b; ++i) run += load_seq(P, i).nu;
  return run;
}

// The new token that a query row belongs to (row * group < 2^32: exact).
__device__ __forceinline__ int query_of(const AttnParams& P, int row) {
  return P.group_magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(row), P.group_magic)) : row;
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One more part of a row, of maximum m: the factors of what is there and of the
// part, with the new maximum in M.  A part that saw nothing (its sum is 0, since
// a part's largest weight is 1) is left out; one whose scores are all NaN has a
// NaN sum and m = -inf, and stays NaN.
struct Factors { float a, b; };
__device__ __forceinline__ Factors fold_factors(float& M, float m) {
  const float mx = fmaxf(M, m);
  const Factors f{M == -INFINITY ? 0.0f : ex2f(M - mx), ex2f(m - mx)};
  M = mx;
  return f;
}
// (b = 0: the part weighs nothing beside what is there, or saw only scores of -inf; its sum
// comes in all the same, so that values that are not finite are not lost)
__device__ __forceinline__ float fold(float x, float part, Factors f) { return __fmaf_rn(part, f.b, __fmul_rn(x, f.a)); }
// The part's maximum and sum into (M, L).
__device__ __forceinline__ Factors add_part(float& M, float& L, float m, float l) {
  if (l == 0.0f) return Factors{1.0f, 0.0f};
  Factors f = fold_factors(M, m);
  if (l != l) f.b = l;
  L = fold(L, l, f);
  return f;
}
// Four elements of a fragment: two each of its rows of even and odd number.
__device__ __forceinline__ void fold4(float4& x, const float4& part, Factors even, Factors odd) {
  x.x = fold(x.x, part.x, even);
  x.y = fold(x.y, part.y, odd);
  x.z = fold(x.z, part.z, even);
  x.w = fold(x.w, part.w, odd);
}
template <uint32_t EXP, uint32_t ONE>
struct OddElem {                         // which of a pair of elements are not finite: bits 15 and 31
  static __device__ __forceinline__ uint32_t of(uint32_t w) { return ((w & EXP) + ONE) & 0x80008000u; }
  static __device__ __forceinline__ bool odd(const uint4& w) { return (of(w.x) | of(w.y) | of(w.z) | of(w.w)) != 0; }
  static __device__ __forceinline__ void clear_odd(uint32_t (&a)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] &= ~((of(a[j]) >> 15) * 0xFFFFu);
  }
};
template <class T> struct Elem;
template <> struct Elem<__nv_bfloat16> : OddElem<0x7F807F80u, 0x00800080u> {
  static constexpr float OFF = 0.0f, SLACK = 8.0f;
  static constexpr uint32_t EXP = 0x7F807F80u;
  static __device__ __forceinline__ float value(uint32_t bits) { return __uint_as_float(bits << 16); }
  static constexpr float MORE = 1.0f + 2.384185791015625e-07f;   // 1 + 2^-22
  // The weights (a, b) >= 0 as the sum of two pairs of elements: hi is cut off, lo
  // is the rest and 2^-22 of the weight, a bias far below the result's own
  // rounding.  So both parts of a weight above 0 are above 0, and an infinite value
  // comes through as itself.
  static __device__ __forceinline__ void split(float a, float b, uint32_t& hi, uint32_t& lo) {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    hi = __byte_perm(x, y, 0x7632);
    const __nv_bfloat162 r = __floats2bfloat162_rn(__fmaf_rn(a, MORE, -__uint_as_float(x & 0xFFFF0000u)),
                                                   __fmaf_rn(b, MORE, -__uint_as_float(y & 0xFFFF0000u)));
    lo = *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  // The values of N fragments times the weights (tokens 0-7 and 8-15: hi, then lo).
  template <int N>
  static __device__ __forceinline__ void weigh(float (*o)[4], const uint32_t (&a)[N][4], const uint32_t (&p)[4]) {
#pragma unroll
    for (int z = 0; z < N; ++z) mma(o[z], a[z], p[2], p[3]);
#pragma unroll
    for (int z = 0; z < N; ++z) mma(o[z], a[z], p[0], p[1]);
  }
};
// f16: a weight's high part in units of 2^-8 of the row's reference, cut off, and the
// rest of it 2^12 times larger, whose products are scaled back as they join the others'.
// So a weight has 22 bits, down to 2^-44 of the reference; below that it is rounded to a
// multiple of it (with one scale for both that would be 2^-32, N 2^-33 of the values of N
// tokens).  The high part is below 2^15 and its rest below 2^3: both fit.
template <> struct Elem<__half> : OddElem<0x7C007C00u, 0x04000400u> {
  static constexpr float OFF = 8.0f, SLACK = 6.0f;
  static constexpr uint32_t EXP = 0x7C007C00u;
  static __device__ __forceinline__ float value(uint32_t bits) { return __half2float(__ushort_as_half(static_cast<unsigned short>(bits))); }
  static constexpr float TINY = 5.960464477539063e-08f;      // 2^-24, the smallest f16
  static constexpr float UP = 4096.0f, DOWN = 1.0f / 4096.0f;
  // The rest of a weight with a high part is never 0 (at most one step of the rest too
  // much), so that an infinite value comes through as itself.
  static __device__ __forceinline__ float rest(float a, float h) {
    const float r = __fmul_rn(__fsub_rn(a, h), UP);
    return a >= TINY ? fmaxf(r, TINY) : r;
  }
  static __device__ __forceinline__ void split(float a, float b, uint32_t& hi, uint32_t& lo) {
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    const __half2 r = __floats2half2_rn(rest(a, h.x), rest(b, h.y));
    lo = *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  template <int N>
  static __device__ __forceinline__ void weigh(float (*o)[4], const uint32_t (&a)[N][4], const uint32_t (&p)[4]) {
    constexpr int M = N > 2 ? 2 : N;     // (all four at once: 0.120 ms for 0.115, 20 rows, 64 sequences of up to 4096 tokens)
#pragma unroll
    for (int z0 = 0; z0 < N; z0 += M) {
      float low[M][4] = {};
#pragma unroll
      for (int z = 0; z < M; ++z) mma(low[z], a[z0 + z], p[2], p[3]);
#pragma unroll
      for (int z = 0; z < M; ++z) mma(o[z0 + z], a[z0 + z], p[0], p[1]);
#pragma unroll
      for (int z = 0; z < M; ++z)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[z0 + z][e] = __fmaf_rn(low[z][e], DOWN, o[z0 + z][e]);
    }
  }
};
__device__ __forceinline__ void from_float(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_float(float x, __half& y) { y = __float2half_rn(x); }

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap& map, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(&map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Waits for a phase of a barrier, at most TIMEOUT_NS twice over.
__device__ __forceinline__ bool mbar_wait_phase(uint32_t bar, uint32_t parity) {
  if (mbar_try(bar, parity)) return true;
  const unsigned long long t0 = global_timer();
  while (!mbar_try(bar, parity))
    if (global_timer() - t0 > 2 * TIMEOUT_NS) return false;
  return true;
}
// the four working warps of the tile's rows 8 x .. 8 x + 7
template <int NT>
__device__ __forceinline__ void rows_sync(int x) {
  if (NT <= 1 || (NT == 2 && x == 0)) asm volatile("bar.sync 1, %0;" ::"n"(AW * 32) : "memory");
  else if (NT == 2) asm volatile("bar.sync 2, %0;" ::"n"(AW * 32) : "memory");
  else asm volatile("bar.sync %0, %1;" ::"r"(x + 1), "n"(AW * 32) : "memory");
}

// A place in a worker's run: the sequence, kv head and tile, the unit in the
// sequence's list.
struct Place {
  Seq s;
  int b, head, tile, li;
  int left;                              // units of the run from this one on
};
// The slices of a unit that some new token sees, by bits; a lane's are every fourth.
__device__ __forceinline__ uint32_t slices_of(const AttnParams& P, const Place& p, int lane) {
  constexpr int N = UNIT / SL;
  const int t = p.s.unit(p.li) * UNIT;
  const int end = (min(max(0, p.s.len - t), UNIT) + SL - 1) / SL, from = min(N, max(0, p.s.low - t) / SL);
  const int sinks = (min(max(0, P.sinks - t), UNIT) + SL - 1) / SL;
  return ((1u << end) - 1u) & (((1u << N) - (1u << from)) | ((1u << sinks) - 1u)) & (0x1111u << lane);
}
// The next unit of the run; false at its end.
__device__ __forceinline__ bool next_unit(const AttnParams& P, Place& p) {
  if (--p.left <= 0) return false;
  if (++p.li == p.s.nu) {
    p.li = 0;
    if (++p.tile == P.tiles) p.tile = 0, ++p.head;
    if (p.head == P.c.kv_heads) {
      p.head = 0;
      // (where the lengths changed under the call there may be none left: then units without
      // tokens, so that every warp of a CTA goes through as many as the others)
      do {
        p.b = min(p.b + 1, static_cast<int>(P.B) - 1);
        p.s = load_seq(P, p.b);
      } while (p.s.nu == 0 && p.b + 1 < P.B);
    }
  }
  return true;
}

// Where the result of a row goes: out and lse, from the weighted sum o (this
// lane's share), the sum l and the maximum m (base 2).
template <class T>
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + (log2f(l) - Elem<T>::OFF)) * 0.6931471805599453f;
}

// A copying warp: the slices of its lane, by halves of 16 tokens, each half
// in boxes of P.box tokens that lie in one page.  Lane j looks token j of a slice
// up, while the slice before is copied.
template <int D, int NT>
__device__ __forceinline__ void copy_run(const AttnParams& P, const AttnMaps& maps, Place p, uint32_t ring, uint32_t full,
                                         uint32_t empty, uint8_t* bad_slice) {
  using S_ = Shape<D, NT>;
  const int lane = threadIdx.x & 31;
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the rings' front held the block sums
  int page = 0, place = 0;
  bool seen = false;
  uint32_t slices = slices_of(P, p, (threadIdx.x >> 5) % AW);
  auto seek = [&]() {
    while (slices == 0) {
      if (!next_unit(P, p)) return false;
      slices = slices_of(P, p, (threadIdx.x >> 5) % AW);
    }
    const int t = p.s.unit(p.li) * UNIT + (__ffs(slices) - 1) * SL + lane;
    slices &= slices - 1;
    seen = t < p.s.len && (t >= p.s.low || t < P.sinks);
    uint32_t n = __umulhi(static_cast<uint32_t>(t), P.page_magic);
    place = static_cast<int>(static_cast<uint32_t>(t) - n * static_cast<uint32_t>(P.c.page_size));
    if (place < 0) place += P.c.page_size, --n;            // the quotient is one off at most
    if (place >= P.c.page_size) place -= P.c.page_size, ++n;
    page = seen ? __ldg(P.c.table + p.b * P.c.table_stride + n) : -1;
    return true;
  };
  int stage = 0, phase = 1, number = 0;
  bool more = seek();
  while (more) {
    const int head = p.head, from = place;
    // the first lane of a box speaks for it: its page is that of any token seen in it
    const uint32_t in_box = (__ballot_sync(0xffffffffu, seen) >> lane) & ((1u << P.box) - 1u);
    const int at = __shfl_sync(0xffffffffu, page, in_box ? lane + __ffs(in_box) - 1 : lane);
    const bool speaks = lane % P.box == 0 && in_box;
    const bool copies = speaks && at >= 0 && at < P.c.num_pages;
    const bool bad = __any_sync(0xffffffffu, speaks && !copies);
    const uint32_t boxes = __ballot_sync(0xffffffffu, copies);
    more = seek();
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      const uint32_t bar = full + stage * 8;
      if (!mbar_wait_phase(empty + stage * 8, phase)) return;      // (the working warps give up too)
      if (lane == 0) {
        if (h == 0) bad_slice[number & 7] = bad;
        mbar_arrive_expect_tx(bar, __popc((boxes >> (h * HALF)) & 0xFFFFu) * P.box * D * 4);
      }
      __syncwarp();
      if (copies && lane / HALF == h) {
        const uint32_t dst = ring + stage * S_::STAGE + (lane & (HALF - 1)) * 128;
        const int c1 = P.head_first ? head : from, c2 = P.head_first ? from : head;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          copy_box(dst + c * S_::PANEL, maps.k, c * 64, c1, c2, at, bar);
          copy_box(dst + S_::KEYS + c * S_::PANEL, maps.v, c * 64, c1, c2, at, bar);
        }
      }
      if (++stage == S_::STAGES) stage = 0, phase ^= 1;
    }
    ++number;
  }
}

template <class T, int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::THREADS, Shape<D, NT>::CTAS)
attn_kernel(const __grid_constant__ AttnParams P, const __grid_constant__ AttnMaps maps) {
  using S_ = Shape<D, NT>;
  using E = Elem<T>;
  constexpr int KK = D / 16, DT = D / 16, MINE = S_::SLOTS / AW, THREADS = S_::THREADS;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ uint8_t bad_slice[AW][8];
  __shared__ float2 share[AW][NT * 8];   // maximum and sum of each lane's share
  __shared__ float2 group_ml[NT * 8];    // ... and of the group so far
  __shared__ uint64_t bars[2][AW][S_::STAGES];               // full, empty
  // until the runs are dealt out, the front of the rings holds the block sums
  int64_t* const scan = reinterpret_cast<int64_t*>(smem_raw);      // [THREADS], then the total
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t full = smem_addr(&bars[0][0][0]), empty = smem_addr(&bars[1][0][0]);
  if (tid < 2 * AW * S_::STAGES) {
    mbar_init(full + tid * 8, tid < AW * S_::STAGES ? 1 : NT);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }

  const int64_t total = unit_sums<THREADS>(P, scan);
  const int HT = P.c.kv_heads * P.tiles;
  const Runs runs(static_cast<uint32_t>(total * HT), S_::WORKERS);
  const uint32_t me = blockIdx.x;
  if (me >= runs.workers) return;        // every thread
  const uint32_t start = runs.start(me);
  Place cons;
  cons.left = static_cast<int>(runs.start(me + 1) - start);
  {
    const int64_t at = start / HT;       // the sequence that holds it: [run, run + nu)
    int blk = 0;                         // the last block of sequences that begins at or before it
#pragma unroll
    for (int j = 0; j < THREADS / 32; ++j) blk += __popc(__ballot_sync(0xffffffffu, scan[j * 32 + lane] <= at));
    blk -= 1;
    int b = blk * seqs_per<THREADS>(P);
    int64_t run = scan[blk];
    __syncthreads();                     // the rings are free
    Seq s = load_seq(P, b);
    while (run + s.nu <= at && b + 1 < P.B) {
      run += s.nu;
      s = load_seq(P, ++b);
    }
    // (within bounds, should the lengths have changed)
    const int64_t rest = static_cast<int64_t>(start) - run * HT;
    const int ht = min(static_cast<int>(rest / max(s.nu, 1)), HT - 1);
    cons.s = s;
    cons.b = b;
    cons.head = ht / P.tiles;
    cons.tile = ht - cons.head * P.tiles;
    cons.li = max(0, min(static_cast<int>(rest - static_cast<int64_t>(ht) * s.nu), s.nu - 1));
  }
  const int w = warp % AW, x = warp / AW;      // the lane; the working warp's rows, 8 x .. 8 x + 7 of a tile
  const uint32_t ring = smem_addr(smem_raw) + w * (S_::STAGES * S_::STAGE);
  const uint32_t my_full = full + w * S_::STAGES * 8, my_empty = empty + w * S_::STAGES * 8;
  if (x == NT) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S_::REGS_COPY));
    copy_run<D, NT>(P, maps, cons, ring, my_full, my_empty, bad_slice[w]);
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S_::REGS_WORK));

  // ---- a working warp
  // [fragment][lane of the CTA][thread]: four floats of a warp's result
  float4* const xch = reinterpret_cast<float4*>(smem_raw + AW * S_::STAGES * S_::STAGE + x * S_::XCH) + lane;
  int use_stage = 0, use_phase = 0, number = 0;
  bool dead = false;                     // a copy did not come
  const int g8 = lane >> 2, t4 = lane & 3;
  // this lane's row of an ldmatrix, with the swizzle of its first piece; pieces 2 k are at that ^ 32 k
  const uint32_t klane = (((lane >> 3) & 1) * 8 + (lane & 7)) * 128 + (((lane >> 4) ^ (lane & 7)) * 16);
  const uint32_t vlane = ((lane >> 4) * 8 + (lane & 7)) * 128 + ((((lane >> 3) & 1) ^ (lane & 7)) * 16);
  uint32_t kswz[4], vswz[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) kswz[k] = klane ^ (32 * k), vswz[k] = (vlane ^ (32 * k)) + S_::KEYS;
  uint32_t qf[S_::QS ? 1 : KK][2];
  uint2* const qsm = reinterpret_cast<uint2*>(smem_raw + S_::Q_AT) + x * KK * 32 + lane;       // [KK][thread]
  float o[DT][4], m[2], l[2];
  float4 gacc[MINE];
  bool fresh_group = true, folding = false, head_part = false, idle = false;
  int row0 = 0;
  uint32_t at = start;                   // the unit's number in the batch
  // the queries of a kv head and tile, as B operands: loaded, and where the tile's warps share them, put down
  uint32_t qr[S_::QS ? KK / AW : 1][2];
  auto fetch_queries = [&]() {
    row0 = (cons.tile * NT + x) * 8;
    idle = row0 >= P.rows || query_of(P, row0) >= cons.s.nnew;
    const int row = row0 + g8, i = query_of(P, row);
    const bool real = row < P.rows && i < cons.s.nnew;
    const T* qp = static_cast<const T*>(P.q) + cons.b * P.qs.batch + i * P.qs.token +
                  (cons.head * P.group + (row - i * P.group)) * P.qs.head + t4 * 2;
#pragma unroll
    for (int k = 0; k < KK / (S_::QS ? AW : 1); ++k) {
      const int c = (S_::QS ? k * AW + w : k) * 16;
      const uint32_t lo = real ? __ldg(reinterpret_cast<const uint32_t*>(qp + c)) ^ P.q_sign : 0u;
      const uint32_t hi = real ? __ldg(reinterpret_cast<const uint32_t*>(qp + c + 8)) ^ P.q_sign : 0u;
      if constexpr (S_::QS) qr[k][0] = lo, qr[k][1] = hi;
      else qf[k][0] = lo, qf[k][1] = hi;
    }
  };
  auto put_queries = [&]() {
#pragma unroll
    for (int k = 0; k < KK / AW; ++k) qsm[(k * AW + w) * 32] = make_uint2(qr[k][0], qr[k][1]);
  };
  fetch_queries();
  if constexpr (S_::QS) {
    put_queries();
    rows_sync<NT>(x);
  }
  for (;;) {
    const int u = cons.s.unit(cons.li), g = u / GROUP;
    if (fresh_group) {
      const int f = cons.s.first(g), e = cons.s.past(g);
      folding = cons.li == f && e - cons.li <= cons.left;
      head_part = start >= at - (cons.li - f);
#pragma unroll
      for (int j = 0; j < MINE; ++j) gacc[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] = 0.0f;
    m[0] = m[1] = -INFINITY, l[0] = l[1] = 0.0f;
    bool unit_bad = false;
#pragma unroll 1
    for (uint32_t slices = slices_of(P, cons, w); slices != 0; slices &= slices - 1) {
      // ---- one slice: its two halves, when they have landed
      uint32_t sk[2], done[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        sk[y] = ring + use_stage * S_::STAGE;
        done[y] = my_empty + use_stage * 8;
        if (!dead && !mbar_wait_phase(my_full + use_stage * 8, use_phase)) dead = true;
        if (++use_stage == S_::STAGES) use_stage = 0, use_phase ^= 1;
      }
      unit_bad |= dead || bad_slice[w][number & 7] != 0;
      ++number;
      const int t0 = u * UNIT + (__ffs(slices) - 1) * SL;
      if (idle) {                        // no query among the warp's rows
        if (lane == 0) mbar_arrive(done[0]), mbar_arrive(done[1]);
        continue;
      }
      float s[2][4];
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[y][e] = 0.0f;
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        uint2 bq;
        if constexpr (S_::QS) bq = qsm[k * 32];
        else bq = make_uint2(qf[k][0], qf[k][1]);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t a[4];
          ldsm(a, sk[y] + kswz[k % 4] + k / 4 * S_::PANEL);
          E::mma(s[y], a, bq.x, bq.y);
        }
      }
      // masks: the queries stand at p0 .. len - 1
      const int p0 = cons.s.len - cons.s.nnew;
      const bool masked = t0 + SL - 1 > p0 ||
                          (P.window > 0 && t0 <= cons.s.len - 1 - P.window && t0 > P.sinks - SL);
      uint32_t hidden = 0;               // bit 4 y + e (of the thread's scores)
      if (masked) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = query_of(P, row0 + 2 * t4 + e);        // at p0 + i, which 32 bits may not hold past the last token
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int t = t0 + y * HALF + g8 + 8 * f;
              if (t - p0 > i || t >= cons.s.len || (P.window > 0 && t - p0 <= i - P.window && t >= P.sinks)) {
                s[y][2 * f + e] = -INFINITY;
                hidden |= 1u << (y * 4 + 2 * f + e);
              }
            }
        }
      }
      // each query row's reference m (the threads of equal t4 share a row's tokens): it follows
      // the row's maximum where that runs SLACK ahead, so weights stay below 2^SLACK
      float top[2];
      bool ahead = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[e] = fmaxf(fmaxf(s[0][e], s[0][2 + e]), fmaxf(s[1][e], s[1][2 + e])) * P.c2;
        ahead |= top[e] > m[e] + E::SLACK;
      }
      if (__any_sync(0xffffffffu, ahead)) {
        bool scaled = false;
        float fac[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = top[e];
#pragma unroll
          for (int z = 4; z < 32; z <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, z));
          fac[e] = 1.0f;
          if (mx > m[e] + E::SLACK) {
            if (m[e] != -INFINITY) {
              fac[e] = ex2f(m[e] - mx);
              scaled = true;
            }
            m[e] = mx;
          }
        }
        if (__any_sync(0xffffffffu, scaled)) {
          l[0] *= fac[0], l[1] *= fac[1];
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] *= fac[e & 1];
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float sub = m[e] == -INFINITY ? E::OFF : E::OFF - m[e];
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int f = 0; f < 4; f += 2) s[y][f + e] = ex2f(__fmaf_rn(s[y][f + e], P.c2, sub));
      }
      // A masked token's value must not come in even as 0 * inf: where a masked slice
      // holds values that are not finite, they go straight into the rows that see them
      // (which they leave infinite or NaN), and the product takes zeros for them.
      bool odd = false;
      if (masked) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if ((hidden >> (y * 4 + e)) & 1u) s[y][e] = 0.0f;
#pragma unroll 8
        for (int z = lane * 16; z < 2 * S_::KEYS; z += 512) odd |= E::odd(lds128(z < S_::KEYS ? sk[0] + S_::KEYS + z : sk[1] + z));
        odd = __any_sync(0xffffffffu, odd);
        if (odd) {
#pragma unroll 1
          for (int r = 0; r < SL; ++r) {
            const int t = t0 + r;
            // (what lies in a place that nobody sees is of no account, whatever it is)
            if (t >= cons.s.len || (t < cons.s.low && t >= P.sinks)) continue;
            const uint32_t row = (r < HALF ? sk[0] : sk[1]) + S_::KEYS + (r & (HALF - 1)) * 128;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                const uint32_t bits = lds16(row + d / 4 * S_::PANEL + (((2 * (d % 4) + f) ^ (r & 7)) * 16) + g8 * 2);
                if ((bits & E::EXP & 0xFFFFu) != (E::EXP & 0xFFFFu)) continue;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int i = query_of(P, row0 + 2 * t4 + e);
                  if (t - p0 <= i && !(P.window > 0 && t - p0 <= i - P.window && t >= P.sinks)) o[d][2 * f + e] += E::value(bits);
                }
              }
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) l[e] += (s[0][e] + s[0][2 + e]) + (s[1][e] + s[1][2 + e]);
      uint32_t pf[2][4];                 // weights: tokens 0-7 and 8-15 of a half, then what the dtype dropped of them
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        E::split(s[y][0], s[y][1], pf[y][0], pf[y][2]);
        E::split(s[y][2], s[y][3], pf[y][1], pf[y][3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) pf[y][e] = movm(pf[y][e]);
      }
      if (odd) {
#pragma unroll 1
        for (int y = 0; y < 2; ++y) {
          const uint32_t base = y ? sk[1] : sk[0];
          uint32_t w4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w4[e] = y ? pf[1][e] : pf[0][e];
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            uint32_t a[1][4];
            ldsm_t(a[0], base + vswz[d % 4] + d / 4 * S_::PANEL);
            E::clear_odd(a[0]);
            E::weigh(o + d, a, w4);
          }
        }
      } else {
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int d = 0; d < DT; d += 4) {
            uint32_t a[4][4];
#pragma unroll
            for (int z = 0; z < 4; ++z) ldsm_t(a[z], sk[y] + vswz[z] + d / 4 * S_::PANEL);
            E::weigh(o + d, a, pf[y]);
          }
      }
      __syncwarp();                      // the stages may be filled again
      if (lane == 0) mbar_arrive(done[0]), mbar_arrive(done[1]);
    }

    // ---- where the unit's result goes; on to the next unit, whose queries come meanwhile
    const bool group_ends = cons.li + 1 == cons.s.past(g), store = !folding || group_ends;
    const bool direct = folding && cons.s.past(g) - cons.s.first(g) == cons.s.nu;
    const int64_t slot = folding ? (static_cast<int64_t>(cons.b) * HT + cons.head * P.tiles + cons.tile) * P.groups + g
                                 : static_cast<int64_t>(me) * (2 * GROUP) + (head_part ? 0 : GROUP) + u % GROUP;
    const int was_b = cons.b, was_head = cons.head, was_row0 = row0, was_nnew = cons.s.nnew;
    const bool head_ends = cons.li + 1 == cons.s.nu, more = next_unit(P, cons);
    if (head_ends && more) fetch_queries();
    ++at;

    // ---- the unit's result: the lanes' shares brought to one maximum and summed in order
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int z = 4; z < 32; z <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], z);
      if (unit_bad) m[e] = 0.0f, l[e] = __int_as_float(0x7fc00000);
      if (g8 == 0) share[w][x * 8 + 2 * t4 + e] = make_float2(m[e], l[e]);
    }
    if (unit_bad && x == 0 && lane == 0 && P.c.err) atomicAdd(P.c.err, 1);
    float UM[2], UL[2], wt[2][AW];
    float2 gml[2];
    float4 uacc[MINE];
    constexpr int PER_PASS = MINE / S_::PASSES;
#pragma unroll
    for (int pass = 0; pass < S_::PASSES; ++pass) {
      if (pass > 0) rows_sync<NT>(x);
#pragma unroll
      for (int f = 0; f < PER_PASS * AW; ++f) {
        const int d = pass * PER_PASS * AW + f;
        xch[(f * AW + w) * 32] = make_float4(o[d][0], o[d][1], o[d][2], o[d][3]);
      }
      rows_sync<NT>(x);
      if (pass == 0) {
        if constexpr (S_::QS)
          if (head_ends && more) put_queries();        // every warp is done with the head before
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float2 h[AW];
#pragma unroll
          for (int z = 0; z < AW; ++z) h[z] = share[z][x * 8 + 2 * t4 + e];
          float mx = -INFINITY, sum = 0.0f;
#pragma unroll
          for (int z = 0; z < AW; ++z) mx = fmaxf(mx, h[z].x);
#pragma unroll
          for (int z = 0; z < AW; ++z) {
            wt[e][z] = h[z].y == 0.0f ? 0.0f : ex2f(h[z].x - mx);
            sum = __fmaf_rn(h[z].y, wt[e][z], sum);
          }
          UM[e] = mx;
          UL[e] = sum;
          gml[e] = fresh_group ? make_float2(-INFINITY, 0.0f) : group_ml[x * 8 + 2 * t4 + e];
        }
      }
#pragma unroll
      for (int j = 0; j < PER_PASS; ++j) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int z = 0; z < AW; ++z) {
          const float4 part = xch[((j * AW + w) * AW + z) * 32];
          v.x = __fmaf_rn(part.x, wt[0][z], v.x);
          v.y = __fmaf_rn(part.y, wt[1][z], v.y);
          v.z = __fmaf_rn(part.z, wt[0][z], v.z);
          v.w = __fmaf_rn(part.w, wt[1][z], v.w);
        }
        uacc[pass * PER_PASS + j] = v;
      }
    }
    rows_sync<NT>(x);                        // the shares may be written again

    // ---- into the group, where this run holds all of it; otherwise out
    if (folding) {
      Factors f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f[e] = add_part(gml[e].x, gml[e].y, UM[e], UL[e]);
        UM[e] = gml[e].x;
        UL[e] = gml[e].y;
        if (w == 0 && g8 == 0) group_ml[x * 8 + 2 * t4 + e] = gml[e];
      }
#pragma unroll
      for (int j = 0; j < MINE; ++j) {
        fold4(gacc[j], uacc[j], f[0], f[1]);
        uacc[j] = gacc[j];
      }
    }
    if (store) {
      float2* const ml = folding ? P.group_ml : P.unit_ml;
      float* const po = folding ? P.group_o : P.unit_o;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = x * 8 + 2 * t4 + e, row = was_row0 + 2 * t4 + e, i = query_of(P, row);
        if (row >= P.rows || i >= was_nnew) continue;
        const float inv = UL[e] == 0.0f ? 0.0f : __frcp_rn(UL[e]);       // (nothing seen: o is 0)
        const int hq = was_head * P.group + (row - i * P.group);
        T* op = static_cast<T*>(P.out) + was_b * P.os.batch + i * P.os.token + hq * P.os.head + g8;
        float* dst = po + (slot * (NT * 8) + r) * D + g8;
#pragma unroll
        for (int j = 0; j < MINE; ++j) {
          const int d = j * AW + w;
          const float lo = e ? uacc[j].y : uacc[j].x, hi = e ? uacc[j].w : uacc[j].z;
          if (direct) {
            from_float(__fmul_rn(lo, inv), op[d * 16]);
            from_float(__fmul_rn(hi, inv), op[d * 16 + 8]);
          } else {
            dst[d * 16] = lo;
            dst[d * 16 + 8] = hi;
          }
        }
        if (w == 0 && g8 == 0) {
          if (!direct) ml[slot * (NT * 8) + r] = make_float2(UM[e], UL[e]);
          else if (P.lse) P.lse[(static_cast<int64_t>(was_b) * P.c.n + i) * P.q_heads + hq] = lse_of<T>(UM[e], UL[e]);
        }
      }
    }
    fresh_group = group_ends;
    if (!more) break;
  }
  // where a copy did not come in time, the CTA stays for the last ones, within limits
  if (dead) {
#pragma unroll 1
    for (int i = 0; i < S_::STAGES; ++i) {
      if (--use_stage < 0) use_stage = S_::STAGES - 1, use_phase ^= 1;
      mbar_wait_phase(my_full + use_stage * 8, use_phase);
    }
  }
}

// ------------------------------------------------------------ the join

constexpr int JW = 16;                   // warps of a join CTA, and chains of the tree
constexpr int JB = 4;                    // chains of a block

// A row of a sequence whose groups are not all in one run: group g goes to
// chain g mod 16, a chain folds its groups in order, a block its four chains,
// and the row its four blocks.  By how many rows there are, a chain, a block or
// a row is a warp's; it is the same tree.  The join also fills the rows without
// a query, and those of rejected sequences.
template <int D>
struct JoinRow {
  static constexpr int E = D / 32;       // elements of a lane
  float M = -INFINITY, L = 0.0f, o[E] = {};
  __device__ __forceinline__ void add(float m, float l, const float (&v)[E]) {
    const Factors f = add_part(M, L, m, l);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fold(o[e], v[e], f);
  }
  __device__ __forceinline__ void add(const JoinRow& r) { add(r.M, r.L, r.o); }
};
template <int E>
__device__ __forceinline__ void load_row(const float* p, float (&v)[E]) {
  if constexpr (E == 4) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else {
    const float2 x = *reinterpret_cast<const float2*>(p);
    v[0] = x.x, v[1] = x.y;
  }
}

template <class T, int D, int JR>        // JR: rows that a warp joins at once
__global__ void __launch_bounds__(JW * 32, 3 - JR) join_kernel(const AttnParams P, int tile_rows, int width, int64_t items) {
  constexpr int E = D / 32;
  __shared__ int64_t scan[JW * 32 + 1];
  __shared__ float2 chain_ml[JW][JR];
  __shared__ float chain_o[JW][JR][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int HT = P.c.kv_heads * P.tiles;
  const int blocks = (min(tile_rows, P.rows) + JR - 1) / JR;

  const bool chainwise = P.groups <= width || width == JW;
  const int w0 = warp % width;           // this warp's first chain
  const int64_t total = unit_sums<JW * 32>(P, scan);
  const RunOf runs(static_cast<uint32_t>(total * HT), P.workers);
  bool waited = false;
  for (int64_t round = blockIdx.x; round * (JW / width) < items; round += gridDim.x) {
    // ---- where everything is (the first time before the units are done).  An item is rows
    // [r, r + JR) of an entry (a sequence, kv head and tile), and `width` warps'
    const int64_t it = round * (JW / width) + warp / width;
    const bool mine = it < items;
    const int64_t entry = mine ? it / blocks : 0;
    const int r0 = static_cast<int>(it - entry * blocks) * JR;
    const int b = static_cast<int>(entry / HT), ht = static_cast<int>(entry - static_cast<int64_t>(b) * HT);
    const Seq s = load_seq(P, b);
    const uint32_t u0 = static_cast<uint32_t>(units_before<JW * 32>(P, scan, b) * HT) + static_cast<uint32_t>(ht) * s.nu;
    const int glast = s.nu > 0 ? s.unit(s.nu - 1) / GROUP : -1;
    const bool direct = s.nu > 0 && s.first(glast) == 0 && runs.of(u0) == runs.of(u0 + s.nu - 1);
    const bool work = mine && !(direct && s.nnew == P.c.n);
    if (mine && !s.ok && ht == 0 && r0 == 0 && w0 == 0 && lane == 0 && P.c.err) atomicAdd(P.c.err, 1);
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
    waited = true;
    if (!__syncthreads_or(work)) continue;

    // ---- this warp's chains, in order
    const int gl = s.ul / GROUP, gs = (s.us + GROUP - 1) / GROUP;            // groups [0, gs) and [gl, glast]
    JoinRow<D> acc[JR], blk[JR];
    if (work && !direct) {
      const int chains = chainwise ? 1 : JW / width;
      for (int c = w0 * chains; c < (w0 + 1) * chains && c <= glast; ++c) {     // (chainwise: chain w0)
        JoinRow<D> chain[JR];
        for (int g = c; g <= glast; g += JW) {
          if (g >= gs && g < gl) {
            g += (gl - g + JW - 1) / JW * JW;
            if (g > glast) break;
          }
          const int f = s.first(g), e = s.past(g);
          if (f >= e) continue;
          const uint32_t ua = u0 + f;
          // one part, where one run holds the group, or its units
          const bool whole = runs.start(runs.of(ua) + 1) >= u0 + e;
          const int parts = whole ? 1 : e - f;
          const float2* ml = whole ? P.group_ml : P.unit_ml;
          const float* po = whole ? P.group_o : P.unit_o;
          float2 h[GROUP][JR];
          float v[GROUP][JR][E];
#pragma unroll
          for (int k = 0; k < GROUP; ++k) {
            int64_t at = entry * P.groups + g;
            if (!whole) {
              const uint32_t w = runs.of(min(ua + k, u0 + e - 1));
              at = static_cast<int64_t>(w) * (2 * GROUP) + (runs.start(w) >= ua ? 0 : GROUP) + s.unit(min(f + k, e - 1)) % GROUP;
            }
            at = at * tile_rows + r0;
            // (past the last part: its place again)
#pragma unroll
            for (int j = 0; j < JR; ++j) {
              h[k][j] = ml[at + j];
              load_row<E>(po + (at + j) * D + lane * E, v[k][j]);
            }
          }
          JoinRow<D> inner[JR];
#pragma unroll
          for (int k = 0; k < GROUP; ++k)
            if (k < parts) {
#pragma unroll
              for (int j = 0; j < JR; ++j) inner[j].add(h[k][j].x, h[k][j].y, v[k][j]);
            }
#pragma unroll
          for (int j = 0; j < JR; ++j) chain[j].add(inner[j]);
        }
#pragma unroll
        for (int j = 0; j < JR; ++j) {
          if (chainwise) {
            acc[j] = chain[j];
          } else {
            blk[j].add(chain[j]);
            if (c % JB == JB - 1 || c == glast) {
              acc[j].add(blk[j]);
              blk[j] = JoinRow<D>();
            }
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < JR; ++j) {
      if (lane == 0) chain_ml[warp][j] = make_float2(acc[j].M, acc[j].L);
#pragma unroll
      for (int e = 0; e < E; ++e) chain_o[warp][j][lane * E + e] = acc[j].o[e];
    }
    __syncthreads();
    if (!work) continue;
    // ---- the item's warps in order, and the result: a row to a warp
    for (int j = w0; j < JR; j += width) {
      const int row = (ht % P.tiles) * tile_rows + r0 + j, i = query_of(P, row);
      if (row >= P.rows || (direct && i < s.nnew)) continue;
      JoinRow<D> all, part;
      for (int c = 0; c < width; ++c) {
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = chain_o[warp - w0 + c][j][lane * E + e];
        const float2 h = chain_ml[warp - w0 + c][j];
        if (!chainwise) {
          all.add(h.x, h.y, v);
          continue;
        }
        part.add(h.x, h.y, v);
        if (c % JB == JB - 1 || c == width - 1) {
          all.add(part);
          part = JoinRow<D>();
        }
      }
      const int hq = (ht / P.tiles) * P.group + (row - i * P.group);
      const bool query = i < s.nnew;
      const float inv = all.L == 0.0f ? 0.0f : __frcp_rn(all.L);
      const float nan = __int_as_float(0x7fc00000);
      T* op = static_cast<T*>(P.out) + b * P.os.batch + i * P.os.token + hq * P.os.head + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e)
        from_float(!s.ok ? nan : !query ? 0.0f : __fmul_rn(all.o[e], inv), op[e]);
      if (P.lse && lane == 0)
        P.lse[(static_cast<int64_t>(b) * P.c.n + i) * P.q_heads + hq] =
            !s.ok ? nan : !query ? -INFINITY : lse_of<T>(all.M, all.L);
    }
  }
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

// Row tiles of a call: as few as hold the rows in 32 each, then as narrow as they can be.
struct Tiling { int rows, tiles, nt; };
Tiling tiling_of(int64_t n, int64_t group) {
  const int64_t rows = n * group, tiles = (rows + 31) / 32;
  return {static_cast<int>(rows), static_cast<int>(tiles), static_cast<int>((rows + 8 * tiles - 1) / (8 * tiles))};
}

// The workspace, in this order: maxima and sums of units and of groups, their
// weighted sums.
struct Layout {
  size_t unit_ml, group_ml, unit_o, group_o, bytes;
  int64_t groups;
};
Layout layout_of(int64_t B, int64_t n, int64_t kv_heads, int64_t group, int64_t D, int64_t max_tokens) {
  const Tiling t = tiling_of(n, group);
  const int64_t entries = B * kv_heads * t.tiles, units = (max_tokens + UNIT - 1) / UNIT;
  const int64_t unit_slots = (entries * units < WORKERS ? entries * units : WORKERS) * 2 * GROUP;
  Layout y{};
  y.groups = (units + GROUP - 1) / GROUP;
  const size_t ur = static_cast<size_t>(unit_slots) * t.nt * 8, gr = static_cast<size_t>(entries * y.groups) * t.nt * 8;
  y.unit_ml = 0;
  y.group_ml = y.unit_ml + ur * 8;
  y.unit_o = y.group_ml + gr * 8;
  y.group_o = y.unit_o + ur * D * 4;
  y.bytes = y.group_o + gr * D * 4;
  return y;
}

// Function attributes are set once per device and kernel.
template <class K>
rlk_status allow_smem(K kernel, int bytes, int regs, bool (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(RLK_ECUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev >= 0 && dev < 64 && done[dev]) return RLK_OK;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  cudaFuncAttributes attr{};
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, kernel);
  if (e != cudaSuccess) return fail(RLK_ECUDA, "function attributes: %s", cudaGetErrorString(e));
  // (with fewer, the working warps would wait for registers without end)
  if (attr.numRegs != regs) return fail(RLK_ECUDA, "the kernel was built for %d registers, not %d", attr.numRegs, regs);
  if (dev >= 0 && dev < 64) done[dev] = true;
  return RLK_OK;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The cache's keys or values as a tensor of (element, token of the page, head, page),
// the middle two in the order of their strides; a copy takes 64 elements of
// P.box tokens of a head.
rlk_status map_cache(CUtensorMap* map, const AttnParams& P, const void* base, int D, bool bf16) {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !p)
      return fail(RLK_ECUDA, "cuTensorMapEncodeTiled is not available");
    fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  // a place of extent 1 is never stepped over: any stride does
  const cuuint64_t any = static_cast<cuuint64_t>(D) * 2;
  const cuuint64_t token = P.c.page_size > 1 ? static_cast<cuuint64_t>(P.c.token_stride) * 2 : any;
  const cuuint64_t head = P.c.kv_heads > 1 ? static_cast<cuuint64_t>(P.c.head_stride) * 2 : any;
  const cuuint64_t page = P.c.num_pages > 1 ? static_cast<cuuint64_t>(P.c.page_stride) * 2 : any;
  const cuuint64_t tokens = P.c.page_size, heads = P.c.kv_heads, pages = P.c.num_pages;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), P.head_first ? heads : tokens, P.head_first ? tokens : heads, pages};
  const cuuint64_t strides[3] = {P.head_first ? head : token, P.head_first ? token : head, page};
  const cuuint32_t box = static_cast<cuuint32_t>(P.box);
  const cuuint32_t boxes[4] = {64, P.head_first ? 1 : box, P.head_first ? box : 1, 1}, ones[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                        const_cast<void*>(base), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(RLK_EINVAL, "the cache's strides have no tensor map (%d): they must be positive and below 2^39 elements",
                static_cast<int>(r));
  return RLK_OK;
}

template <class T, int D, int NT>
rlk_status launch_attn(AttnParams P, cudaStream_t st) {
  static bool done[64] = {};
  rlk_status s = allow_smem(attn_kernel<T, D, NT>, Shape<D, NT>::SMEM, Shape<D, NT>::REGS, done);
  if (s != RLK_OK) return s;
  AttnMaps maps;
  constexpr bool bf16 = sizeof(T) == 2 && Elem<T>::EXP == 0x7F807F80u;
  if (P.c.num_pages > 0) {
    if ((s = map_cache(&maps.k, P, P.c.k, D, bf16)) != RLK_OK) return s;
    if ((s = map_cache(&maps.v, P, P.c.v, D, bf16)) != RLK_OK) return s;
  }
  P.workers = Shape<D, NT>::WORKERS;
  attn_kernel<T, D, NT><<<P.workers, Shape<D, NT>::THREADS, Shape<D, NT>::SMEM, st>>>(P, maps);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(RLK_ECUDA, "kernel launch: %s", cudaGetErrorString(e));
  // the join is launched while the units are at work, and waits for them.  A chain to a
  // warp, as far as one round of CTAs (one per SM) has the warps; two rows to a warp, unless
  // it has all their chains and there is room for a row to a warp in one round (the window's
  // 4096 rows: 0.065 ms the call with two, 0.060 with one; the drafts' 20480, which take
  // rounds: 0.188 with two, 0.195 with one)
  const int tile_rows = NT * 8, rows = tile_rows < P.rows ? tile_rows : P.rows;
  const int64_t entries = P.B * P.c.kv_heads * P.tiles, pairs = entries * ((rows + 1) / 2);
  int width = 1;
  while (width < JW && width < P.groups) width *= 2;
  if (pairs * width > NUM_SMS * JW) width = width > JB && pairs * JB <= NUM_SMS * JW ? JB : 1;
  const bool single = width == 1 && entries * rows <= 2 * NUM_SMS * JW;
  const int64_t items = single ? entries * rows : pairs, ctas = (items * width + JW - 1) / JW, most = NUM_SMS * (single ? 2 : 1);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas < most ? ctas : most));
  cfg.blockDim = dim3(JW * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, single ? join_kernel<T, D, 1> : join_kernel<T, D, 2>, P, tile_rows, width, items);
  if (e != cudaSuccess) return fail(RLK_ECUDA, "kernel launch: %s", cudaGetErrorString(e));
  return RLK_OK;
}
template <class T, int D>
rlk_status launch_rows(const AttnParams& P, int nt, cudaStream_t st) {
  switch (nt) {
    case 1: return launch_attn<T, D, 1>(P, st);
    case 2: return launch_attn<T, D, 2>(P, st);
    case 3: return launch_attn<T, D, 3>(P, st);
    default: return launch_attn<T, D, 4>(P, st);
  }
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
  P.pieces = cache->kv_heads * P.row16;
  P.per = APPEND_THREADS * APPEND_PIECES / P.pieces > 0 ? APPEND_THREADS * APPEND_PIECES / P.pieces : 1;
  P.tokens = cache->B * cache->n;
  const int64_t blocks = (P.tokens + P.per - 1) / P.per;
  if (blocks >= (int64_t(1) << 31)) return fail(RLK_EINVAL, "B * n * kv_heads is too large for one call");
  append_kernel<<<static_cast<unsigned>(blocks), APPEND_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(P);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(RLK_ECUDA, "kernel launch: %s", cudaGetErrorString(e));
  return RLK_OK;
}

rlk_status rlk_paged_attention_workspace(int64_t B, int32_t n, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                         int64_t max_tokens, size_t* bytes) {
  if (B < 0 || n < 0 || q_heads < 0 || head_dim < 0 || max_tokens < 0) return fail(RLK_EINVAL, "a size is negative");
  if (!bytes) return fail(RLK_EINVAL, "bytes is NULL");
  if (kv_heads < 1 || q_heads % kv_heads) return fail(RLK_EINVAL, "q_heads %d must be a multiple of kv_heads %d", q_heads, kv_heads);
  *bytes = B == 0 || n == 0 || q_heads == 0
               ? 0 : layout_of(B, n, kv_heads, q_heads / kv_heads, head_dim, max_tokens).bytes;
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
  if (!aligned(workspace, 16)) return fail(RLK_EALIGN, "workspace is not 16-byte aligned");
  const int group = q_heads / cache->kv_heads;
  const Tiling t = tiling_of(cache->n, group);
  const int64_t max_units = (static_cast<int64_t>(cache->max_pages) * cache->page_size + UNIT - 1) / UNIT;
  if (static_cast<double>(cache->B) * cache->kv_heads * t.tiles * max_units >= 2147483648.0)
    return fail(RLK_EINVAL, "too many tokens for one call: B * kv_heads * row tiles * max_pages * page_size / 512 must be below 2^31");
  const Layout y = layout_of(cache->B, cache->n, cache->kv_heads, group, cache->head_dim,
                             static_cast<int64_t>(cache->max_pages) * cache->page_size);
  if (!workspace && y.bytes > 0) return fail(RLK_EINVAL, "workspace is NULL");
  char* ws = static_cast<char*>(workspace);
  AttnParams P{};
  P.c = paged_params(cache);
  P.q = q;
  P.out = out;
  P.qs = *q_strides;
  P.os = *out_strides;
  P.q_heads = q_heads;
  P.group = group;
  P.rows = t.rows;
  P.tiles = t.tiles;
  P.B = cache->B;
  P.c2 = fabsf(scale) * 1.4426950408889634f;
  P.q_sign = scale < 0.0f ? 0x80008000u : 0u;
  P.window = window;
  P.sinks = window > 0 ? sinks : 0;
  P.lse = out_lse;
  P.unit_ml = reinterpret_cast<float2*>(ws + y.unit_ml);
  P.unit_o = reinterpret_cast<float*>(ws + y.unit_o);
  P.group_ml = reinterpret_cast<float2*>(ws + y.group_ml);
  P.group_o = reinterpret_cast<float*>(ws + y.group_o);
  P.page_magic = static_cast<uint32_t>(cache->page_size == 1 ? 0xFFFFFFFFull
                                       : ((1ull << 32) + cache->page_size - 1) / cache->page_size);
  P.groups = static_cast<int>(y.groups);
  P.group_magic = static_cast<uint32_t>(group == 1 ? 0 : ((1ull << 32) + group - 1) / group);
  P.box = 1;
  while (P.box < HALF && cache->page_size % (2 * P.box) == 0) P.box *= 2;
  P.head_first = cache->kv_heads > 1 && (cache->page_size == 1 || cache->head_stride < cache->token_stride);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = cache->dtype == RLK_DT_BF16;
  if (cache->head_dim == 128)
    return bf ? launch_rows<__nv_bfloat16, 128>(P, t.nt, st) : launch_rows<__half, 128>(P, t.nt, st);
  return bf ? launch_rows<__nv_bfloat16, 64>(P, t.nt, st) : launch_rows<__half, 64>(P, t.nt, st);
}

}  // extern "C"
