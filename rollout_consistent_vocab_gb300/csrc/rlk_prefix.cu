// rlk_prefix.cu -- attention of sequences that share a prefix: the shared tokens' part,
// for all queries of a group at once.
//
// plan_kernel looks the groups and lengths over.  The shared tokens of a group, rounded
// down to 32, go in pieces of a length that depends on theirs alone; a piece's result
// (maximum, sum, weighted sum of values of each query row) goes to the workspace.  Every
// sequence's other tokens, and the join of all, are a kernel each of rlk_tail.cu.  16 prompts
// of up to 8192 tokens with 16 samples each of up to 2048 more, 32 heads on 8 of 128: 786 MB, 150 us
// = 5.2 TB/s; 2 of up to 131071 with 32 samples each: 999 MB, 218 us = 4.6 TB/s (242 on another GB300).

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "rlk_rollout.h"
#include "rlk_device.cuh"
#include "rlk_host.h"
#include "rlk_paged.h"
#include "rlk_tcgen05.cuh"

namespace rlk {

constexpr int PREFIX_STEP = 32;          // shared tokens come in multiples of this

// A group as the plan leaves it: its first sequence, how many, the shared tokens to take, and
// their pieces (0: nothing to do).
struct alignas(16) GroupPlan { int seq0, seqs, shared, pieces; };

struct PrefixParams : PrefixParts {
  const int32_t* group_start;
  const int32_t* shared_lens;
  int groups, max_shared;
  int32_t* plan_first;          // as in PrefixParts, for the plan to write
  uint32_t* plan_tails;
  GroupPlan* plan;              // [groups]
  int32_t* busy;                // [groups] whether a sequence has new tokens
  uint32_t* base;               // units of work before each of [groups + 1], then the CTAs that share them (and `taken`)
  uint32_t unit_cost, tail_cost;         // of a unit, and of 16 own tokens of a sequence
  int box;                      // tokens of a copy: the largest power of 2, up to 64, that divides page_size
  bool merged;                  // a copy takes all 128 elements of its tokens (64 of them)
};

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// The work of a group in units: 512 shared tokens of a kv head for up to 128 query rows.  An
// item, a piece of a kv head for a block of up to 256 query rows, is so many of them.
constexpr int PIECE_UNIT = 512, PROWS = 256;
// What one costs, in steps of 16 own tokens for 8 query rows (a step of 64 elements is half as many bytes, a unit
// of them nearly as many exponentials).  By the times of 48, 72, 96 and 144: 8 x 16 samples with drafts 131, 112,
// 123, 123 us, in f16 143, 123, 134, 134; 16 x 16 samples 150, 150, 150, 150, in f16 160, 153, 151, 154; 8 x 4 with
// drafts and up to 20,000 own tokens 305, 245, 239, 236.  Of 60, 100, 140 and 200: uneven groups of 64 elements 166, 141, 143, 143.
constexpr uint32_t UNIT_COST_128 = 72, UNIT_COST_64 = 100;
constexpr int PSMS = 152;
__device__ __forceinline__ uint32_t units_of_head(const PrefixParams& P, const GroupPlan& p) {
  const uint32_t rows = static_cast<uint32_t>(p.seqs) * P.rows, full = rows / PROWS, rest = rows - full * PROWS;
  return (2u * full + (rest > PROWS / 2 ? 2u : rest > 0 ? 1u : 0u)) * p.pieces * (piece_tokens(p.shared) / PIECE_UNIT);
}

// ------------------------------------------------------------ the plan

constexpr int PLAN_THREADS = 1024, PLAN_GROUPS = 2048;         // groups that are kept in shared memory

// The sum of the values of the threads before this one; the whole CTA.
__device__ __forceinline__ uint32_t sum_before(uint32_t mine, uint32_t* scan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += x;
  }
  __syncthreads();
  if (lane == 31) scan[warp] = run;
  __syncthreads();
  if (warp == 0) {
    uint32_t sum = scan[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    scan[lane] = sum;
  }
  __syncthreads();
  return run - mine + (warp > 0 ? scan[warp - 1] : 0u);
}

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const PrefixParams P) {
  __shared__ int32_t near_start[PLAN_GROUPS + 1], near_shared[PLAN_GROUPS], near_busy[PLAN_GROUPS];
  __shared__ uint32_t scan[PLAN_THREADS / 32];
  __shared__ int most_own;               // tokens behind the shared ones, of the sequence with the most
  const int tid = threadIdx.x, G = P.groups;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t tokens = static_cast<int64_t>(P.c.max_pages) * P.c.page_size;
  const bool near = G <= PLAN_GROUPS;
  const int32_t* const start = near ? near_start : P.group_start;
  const int32_t* const shared = near ? near_shared : P.shared_lens;
  int32_t* const busy = near ? near_busy : P.busy;
  bool fault = false;
  if (tid == 0) most_own = 0;
  for (int g = tid; g < G; g += PLAN_THREADS) {
    const int a = P.group_start[g], e = P.group_start[g + 1];
    fault |= a < 0 || e < a || e > P.B;
    busy[g] = 0;
    if (near) {
      near_start[g] = a;
      near_shared[g] = P.shared_lens[g];
      if (g == G - 1) near_start[G] = e;
    }
  }
  fault = __syncthreads_or(fault);
  for (int b = tid; b < P.B; b += PLAN_THREADS) {
    int len, nnew, first = -1;
    if (!fault && seq_lens(P.c, b, len, nnew)) {
      // the last group that begins at or before b
      int lo = -1, hi = G;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (start[mid] <= b) lo = mid;
        else hi = mid;
      }
      if (lo < 0 || b >= start[lo + 1]) {
        first = 0;
      } else {
        const int in = shared[lo];
        if (in >= 0 && in <= P.max_shared && in <= tokens && (nnew == 0 || len - nnew >= in)) {
          first = in / PREFIX_STEP * PREFIX_STEP;
          if (nnew > 0 && first > 0) busy[lo] = 1;
        }
      }
      if (first >= 0 && nnew > 0) atomicMax(&most_own, len - first);
    }
    P.plan_first[b] = first;
  }
  __syncthreads();
  const int per = (G + PLAN_THREADS - 1) / PLAN_THREADS, g0 = min(G, tid * per), g1 = min(G, g0 + per);
  uint32_t mine = 0;
  for (int g = g0; g < g1; ++g) {
    GroupPlan p{0, 0, 0, 0};
    if (!fault && busy[g]) {
      p.seq0 = start[g];
      p.seqs = start[g + 1] - p.seq0;
      p.shared = min(max(shared[g], 0), P.max_shared) / PREFIX_STEP * PREFIX_STEP;
      p.pieces = pieces_of(p.shared);
    }
    P.plan[g] = p;
    mine += units_of_head(P, p) * P.c.kv_heads;
  }
  uint32_t run = sum_before(mine, scan);
  for (int g = g0; g < g1; ++g) {
    P.base[g] = run;
    run += units_of_head(P, P.plan[g]) * P.c.kv_heads;
  }
  const uint32_t units = run;            // (of the last thread: all)
  if (tid == PLAN_THREADS - 1) P.base[G] = run;
  // the steps of 16 tokens that the sequences have behind the shared ones, by the length of their parts
  const int seqs = static_cast<int>((P.B + PLAN_THREADS - 1) / PLAN_THREADS);
  const int b0 = static_cast<int>(min(P.B, static_cast<int64_t>(tid) * seqs)), b1 = static_cast<int>(min(P.B, static_cast<int64_t>(b0) + seqs));
  auto steps = [&](int b, int level) {
    const int first = P.plan_first[b];
    int len, nnew;
    if (first < 0 || !seq_lens(P.c, b, len, nnew) || nnew == 0) return 0u;
    const int in = min(len - first - tail_level_from(level), tail_level_tokens(level));
    return in > 0 ? (static_cast<uint32_t>(in) + 15u) / 16u : 0u;
  };
  const int top = tail_level(max(most_own, 1) - 1);
  uint32_t own_steps = 0;                // (of the last thread)
  for (int level = 0; level <= top; ++level) {
    uint32_t* const base = P.plan_tails + level * (P.B + 1);
    mine = 0;
    for (int b = b0; b < b1; ++b) mine += steps(b, level);
    run = sum_before(mine, scan);
    for (int b = b0; b < b1; ++b) {
      base[b] = run;
      run += steps(b, level);
    }
    if (tid == PLAN_THREADS - 1) base[P.B] = run;
    own_steps += run;
  }
  if (tid == PLAN_THREADS - 1) {
    // Shared tokens keep the tensor cores and exponentials busy, the others memory: the SMs are shared out
    // by the work that they are, so that both go on side by side to the end (16 groups of 16 samples took
    // 177 us one after the other).  Runs are of pairs of units, for the two streams.
    const uint64_t of_shared = static_cast<uint64_t>(units) * P.unit_cost, of_all = of_shared + static_cast<uint64_t>(own_steps) * P.tail_cost;
    uint32_t ctas = static_cast<uint32_t>((PSMS * of_shared + of_all) / (of_all + 1));
    ctas = max(1u, min(ctas, static_cast<uint32_t>(PSMS)));
    if (units > ctas) {
      const uint32_t per = ((units + ctas - 1) / ctas + 1) & ~1u;
      ctas = (units + per - 1) / per;
    }
    P.base[G + 1] = max(1u, min(units, ctas));
    P.taken[0] = 0u;
    P.taken[1] = static_cast<uint32_t>(top);
    P.taken[2] = own_steps;
  }
}

// ------------------------------------------------------------ the shared tokens
//
// S = Q K^T and O += P V run on tcgen05: 128 query rows as the accumulator's rows, 128
// tokens a tile, everything between in tensor memory.  A CTA has two streams of tiles, each
// with scores (128 columns of tensor memory) and a result (head_dim columns) of its own.
// The scores of a tile's halves come and go by themselves: while a stream's warps take the
// exponentials of one half, the tensor cores are at its other half, or at the other stream.
// A group with up to 128 query rows per kv head gives its streams pieces
// of their own; with more, both streams take the same piece, with 128 rows each, and
// every tile of keys and values is read once for 256 rows.
//
//   warps 0-3, 4-7   a stream's: a thread to a query row.  It reads 64 of its scores, keeps
//                    a reference maximum (which follows the row's maximum where that runs
//                    SLACK ahead; then the result so far is scaled in tensor memory) and
//                    the sum, and writes the weights over the scores as two elements
//                    of the cache's dtype each (hi, then what hi dropped): an operand of
//                    the second product as it lies.  At a piece's end it takes the result out.
//   warps 8, 9       a stream's: one thread issues the products
//   warps 10, 11     copy keys and values, half a tile each, into one ring of tiles, in the order in which they are
//                    needed (TMA boxes of as many tokens as lie together in a page)
//
// With 256 rows and more, bound by the tensor cores and the exponentials that do not go beside them:
// 131072 tokens, 8 kv heads, 1024 rows each of 128 elements, 597 us = 920 TFLOP/s (1380 with the second
// product of the low parts); 2.7 us for 128 tokens of 256 rows, of which the tensor cores need 2.0.  With
// 128 rows bound by memory (4.5 TB/s beside the pieces' results).  Pieces with one row's result behind the
// other's, their next pages looked up after the stores: 669 us.
//
// Shared tokens come in multiples of 32, so that a piece's last tile needs no masks: the
// scores of what is not there are not read, and the second product ends before it.

using bf16_t = __nv_bfloat16;

template <class T> struct Weights;
template <> struct Weights<bf16_t> {
  static constexpr uint32_t FORMAT = 1;            // of the instruction descriptor
  // weights are in units of 2^-OFF of the reference, so below 2^(OFF + SLACK); the pieces' in paged attention's
  static constexpr float OFF = 0.0f, SLACK = 8.0f, TO_PIECES = 1.0f;
  // hi is cut off; lo is the rest and 2^-22 of the weight, so that both parts of a weight
  // above 0 are above 0, and an infinite value comes through as itself
  static constexpr float MORE = 1.0f + 2.384185791015625e-07f;
  static __device__ __forceinline__ void split(float a, float b, uint32_t& hi, uint32_t& lo) {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    hi = __byte_perm(x, y, 0x7632);
    float c, d;
    unpack2(fma2(pack2(a, b), pack2(MORE, MORE), pack2(__uint_as_float((x & 0xFFFF0000u) ^ 0x80000000u),
                                                       __uint_as_float((y & 0xFFFF0000u) ^ 0x80000000u))), c, d);
    const __nv_bfloat162 r = __floats2bfloat162_rn(c, d);
    lo = *reinterpret_cast<const uint32_t*>(&r);
  }
};
// f16: 22 bits of a weight, and steps of 2^-24 below: 2^-37 of the reference.  (Paged attention
// gives the low parts a scale and an accumulator of their own; here tensor memory has no
// room for one, so the reference stays close to the maximum and the unit is as small as it can be.)
template <> struct Weights<__half> {
  static constexpr uint32_t FORMAT = 0;
  static constexpr float OFF = 13.0f, SLACK = 2.0f, TO_PIECES = 1.0f / 32.0f;
  // The rest of a weight with a high part is never 0 (at most one step of 2^-24 too much), so that an
  // infinite value comes through as itself; the words of numbers >= 0 are in their order.
  static __device__ __forceinline__ void split(float a, float b, uint32_t& hi, uint32_t& lo) {
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    float c, d;
    unpack2(fma2(pack2(h.x, h.y), pack2(-1.0f, -1.0f), pack2(a, b)), c, d);
    const __half2 r = __floats2half2_rn(c, d);
    lo = __vmaxu2(*reinterpret_cast<const uint32_t*>(&r), __vminu2(hi, 0x00010001u));
  }
};

constexpr int PTILE = 128;               // tokens of a tile, and rows
static_assert(PROWS == 2 * PTILE, "query rows of a CTA");
constexpr int PTHREADS = 384;
template <int D>
struct PShape {
  static constexpr int PANEL = PTILE * 128;        // 64 elements of every row, 128-byte swizzle
  static constexpr int TILE = D / 64 * PANEL;
  static constexpr int HALF = TILE / 2;            // keys and values: 64 tokens' panels, then the others'
  static constexpr int STAGES = D == 128 ? 5 : 10;
  static constexpr int BARS = 2 * STAGES + 2 * 7 + 1;
  static constexpr int SMEM = 1024 + (2 + STAGES) * TILE + BARS * 8 + 16;
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

// The units in equal runs, the first ones one longer (the CTAs without one make room at once).  An item is the CTA's whose run holds its first unit.
__device__ __forceinline__ uint32_t run_start(uint32_t units, uint32_t workers, uint32_t k) {
  const uint32_t len = units / workers, more = units - len * workers;
  return k * len + min(k, more);
}

// What the two streams take side by side: a piece each of a group's kv head, or one piece
// with rows of their own.
struct Step {
  int seq0, seqs, head, rb, piece;
  int t0, size;                          // the first piece's first token, tokens of a full piece
  int len0, len1;                        // tokens of the streams' pieces (0: none)
  bool both;                             // the same piece
  __device__ __forceinline__ int tokens(int s) const { return s ? len1 : len0; }
  __device__ __forceinline__ int tiles(int s) const { return (tokens(s) + PTILE - 1) / PTILE; }
  __device__ __forceinline__ int from(int s) const { return both || s == 0 ? t0 : t0 + size; }
  __device__ __forceinline__ int piece_of(int s) const { return both || s == 0 ? piece : piece + 1; }
};
// The rows that a stream has the queries of.
struct Rows {
  int seq0 = -1, head = 0, rb = 0;
  __device__ __forceinline__ bool of(const Step& x) const { return seq0 == x.seq0 && head == x.head && rb == x.rb; }
  __device__ __forceinline__ void take(const Step& x) { seq0 = x.seq0, head = x.head, rb = x.rb; }
};
// A stream's tile: tokens t .. t + count - 1 of a kv head; first: of its piece.
struct Tile {
  int seq0, head, t, count;
  bool both, first;
};
// A CTA's way through its run: `at` is the first unit of the item that is next.
struct Way {
  uint32_t at, end;
  int g, head, rb, piece, rows, rbs, size;
  GroupPlan pl;
  __device__ __forceinline__ void load(const PrefixParams& P) {
    pl = P.plan[g];
    size_up(P);
  }
  __device__ __forceinline__ void size_up(const PrefixParams& P) {
    rows = pl.seqs * P.rows;
    rbs = (rows + PROWS - 1) / PROWS;
    size = piece_tokens(pl.shared);
  }
  // the group that holds unit `at`, from g on; the whole warp
  __device__ __forceinline__ void find(const PrefixParams& P) {
    int hi = P.groups;
    while (hi - g > 1) {
      const int step = (hi - g + 31) / 32, mine = g + static_cast<int>(threadIdx.x & 31) * step;
      const uint32_t below = __ballot_sync(0xffffffffu, mine < hi && P.base[mine] <= at);      // (of g it is)
      g += (31 - __clz(below)) * step;
      hi = min(hi, g + step);
    }
    load(P);
  }
  __device__ __forceinline__ bool both() const { return rows - rb * PROWS > PTILE; }
  __device__ __forceinline__ uint32_t weight() const { return (both() ? 2u : 1u) * (size / PIECE_UNIT); }
  // where the pieces of a block end, the next block, head or group (with another item: at < end)
  __device__ __forceinline__ void settle(const PrefixParams& P) {
    if (piece < pl.pieces || at >= end) return;
    piece = 0;
    if (++rb == rbs) rb = 0, ++head;
    if (head == P.c.kv_heads) {
      head = 0;
      ++g;
      load(P);
      if (pl.pieces == 0) find(P);
    }
  }
  // The CTA's run, of equal ones; the whole warp.
  __device__ __forceinline__ void begin(const PrefixParams& P) {
    const int lane = threadIdx.x & 31, G = P.groups;
    g = 0;
    const bool few = G < 31;             // all of them are looked at at once
    uint32_t before = ~0u;
    GroupPlan mine{0, 0, 0, 0};
    if (few && lane <= G + 1) before = P.base[lane];
    if (few && lane < G) mine = P.plan[lane];
    const uint32_t units = few ? __shfl_sync(0xffffffffu, before, G) : P.base[G];
    const uint32_t workers = few ? __shfl_sync(0xffffffffu, before, G + 1) : P.base[G + 1], me = min(blockIdx.x, workers);
    at = run_start(units, workers, me), end = run_start(units, workers, min(me + 1, workers));
    if (at >= end) return;               // (a CTA without items goes through with an empty run)
    uint32_t rest = at;
    if (few) {
      g = 31 - __clz(__ballot_sync(0xffffffffu, lane < G && before <= at));
      pl = GroupPlan{__shfl_sync(0xffffffffu, mine.seq0, g), __shfl_sync(0xffffffffu, mine.seqs, g),
                     __shfl_sync(0xffffffffu, mine.shared, g), __shfl_sync(0xffffffffu, mine.pieces, g)};
      rest -= __shfl_sync(0xffffffffu, before, g);
      size_up(P);
    } else {
      find(P);
      rest -= P.base[g];
    }
    const uint32_t whole = units_of_head(P, pl), block = 2u * pl.pieces * (size / PIECE_UNIT);
    head = static_cast<int>(rest / whole);
    rest -= head * whole;
    rb = static_cast<int>(min(rest / block, static_cast<uint32_t>(rbs - 1)));
    rest -= rb * block;
    const uint32_t w = weight();
    piece = static_cast<int>((rest + w - 1) / w);
    at += piece * w - rest;
    settle(P);
  }
  // The next step; false at the run's end.
  __device__ __forceinline__ bool next(const PrefixParams& P, Step& s) {
    if (at >= end) return false;
    s.seq0 = pl.seq0, s.seqs = pl.seqs, s.head = head, s.rb = rb, s.piece = piece, s.t0 = piece * size, s.size = size;
    s.both = both();
    const uint32_t w = weight();
    const bool pair = !s.both && piece + 1 < pl.pieces && at + w < end;
    s.len0 = min(size, pl.shared - s.t0);
    s.len1 = s.both ? s.len0 : pair ? min(size, pl.shared - s.t0 - size) : 0;
    const int used = pair ? 2 : 1;
    at += used * w;
    piece += used;
    settle(P);
    return true;
  }
  // The products of the run in order: op(s, cur, next, asks) takes stream s from its tile cur to its tile
  // next (count 0: none).  The results of cur and the scores of next go together; asks: next's
  // queries are other ones than the stream had.
  template <class Op>
  __device__ __forceinline__ void walk(const PrefixParams& P, Op op) {
    Step cur, nxt;
    Rows held[2];
    bool have = next(P, cur);
    for (int j = -1; have; j = 0) {
      const bool more = next(P, nxt);
      const int tiles = max(cur.tiles(0), cur.tiles(1));
#pragma unroll 1
      for (; j < tiles; ++j) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int left = cur.tokens(s) - j * PTILE;            // of the stream's piece, from this tile on
          const Tile x{cur.seq0, cur.head, cur.from(s) + j * PTILE, j < 0 ? 0 : max(0, min(PTILE, left)), cur.both, j == 0};
          const bool here = left > PTILE, there = !here && j + 1 == tiles && more && nxt.tokens(s) > 0;
          const Tile y{here ? cur.seq0 : nxt.seq0, here ? cur.head : nxt.head, here ? cur.from(s) + (j + 1) * PTILE : nxt.from(s),
                       here ? min(PTILE, left - PTILE) : there ? min(PTILE, nxt.tokens(s)) : 0, here ? cur.both : nxt.both, !here || j < 0};
          bool asks = false;
          if (y.first && y.count > 0) {
            const int rb = here ? cur.rb : nxt.rb;
            asks = held[s].seq0 != y.seq0 || held[s].head != y.head || held[s].rb != rb;
            held[s].seq0 = y.seq0, held[s].head = y.head, held[s].rb = rb;
          }
          if (x.count > 0 || y.count > 0) op(s, x, y, asks);
        }
      }
      cur = nxt;
      have = more;
    }
  }
};

// true in one thread of a warp that is together
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
  return one != 0;
}
// D[tmem] (+)= A . B^T, one thread: A in shared or in tensor memory
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %3, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n}"
               :: "r"(d), "l"(a), "l"(b), "r"(static_cast<uint32_t>(accumulate)), "r"(idesc) : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %3, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n}"
               :: "r"(d), "r"(a), "l"(b), "r"(static_cast<uint32_t>(accumulate)), "r"(idesc) : "memory");
}
// 32 columns of the warp's 32 lanes of tensor memory, a lane to a thread; what is loaded is there after the wait
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// (keeps uses of the registers behind the wait)
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[32]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                    "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]) :: "memory");
  asm volatile("" : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                    "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) :: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
      :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  uint32_t a[16], b[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) a[j] = r[j], b[j] = r[16 + j];
  tmem_st16(taddr, a);
  tmem_st16(taddr + 16, b);
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The descriptor of the values' tile as the operand whose rows are the tokens (128-byte
// swizzle): 64 elements of 8 tokens are an atom of 1024 bytes, 8 tokens further on is
// 1024 bytes on, the next 64 elements a panel on.
__device__ __forceinline__ uint64_t values_desc(uint32_t saddr, uint32_t panel) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(panel >> 4) << 16) | (64ull << 32) | (1ull << 46) |
         (2ull << 61);
}
__device__ __forceinline__ void store8(float* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}

template <class T, int D>
__global__ void __launch_bounds__(PTHREADS, 1)
prefix_kernel(const __grid_constant__ PrefixParams P, const __grid_constant__ CacheMaps maps) {
  using S_ = PShape<D>;
  using W = Weights<T>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t raw = smem_addr(smem_raw), queries = (raw + 1023u) & ~1023u, ring = queries + 2 * S_::TILE;
  const uint32_t bars = ring + S_::STAGES * S_::TILE;
  const uint32_t full = bars, empty = bars + 8 * S_::STAGES, streams = empty + 8 * S_::STAGES;
  // of stream s, at 16 s + 8 h: half h of a tile has scores, or weights, an even or odd half's result is in; at 8 s: queries
  const uint32_t scored = streams, weighed = streams + 32, summed = streams + 64, asked = streams + 96, last = streams + 112;
  uint32_t* const slot = reinterpret_cast<uint32_t*>(smem_raw + (streams + 120 - raw));
  volatile uint32_t* const dead = slot + 1;        // a wait gave up: everything ends, within limits
  if (tid == 0) {
    for (int s = 0; s < S_::STAGES; ++s) mbar_init(full + 8 * s, 2), mbar_init(empty + 8 * s, 2);
    for (int s = 0; s < 2; ++s) {
      for (int h = 0; h < 2; ++h) mbar_init(scored + 16 * s + 8 * h, 1), mbar_init(weighed + 16 * s + 8 * h, 4), mbar_init(summed + 16 * s + 8 * h, 1);
      mbar_init(asked + 8 * s, 4);
    }
    mbar_init(last, 2);
    *dead = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 8) {
    tmem_alloc(smem_addr(slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  Way way;
  // The plan is made.  (tail_kernel and the join read it without a wait of their own: they are launched by this
  // kernel's signal, which must not come before the wait.)
  auto begin = [&]() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    way.begin(P);
  };
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (mbar_try(bar, parity & 1)) return true;
    const unsigned long long t0 = global_timer();
    while (!mbar_try(bar, parity & 1)) {
      if (*dead) return false;
      if (global_timer() - t0 > 2 * TIMEOUT_NS) {
        *dead = 1u;
        return false;
      }
    }
    return true;
  };

  if (warp >= 10) {
    // ---- copies: each of the two warps has half of the copies of every tile, a lane one of them: a box of
    // tokens and 64 of their elements, or all (P.merged).  Its page is looked up while the tile before
    // waits for its place.
    begin();
    const int panels = P.merged ? 1 : D / 64, copies = PTILE / P.box * panels;
    const uint32_t pages = static_cast<uint32_t>(P.c.num_pages), bytes = P.box * (P.merged ? 256 : 128);
    auto token_of = [&](int e) { return (D == 64 || P.merged ? e : e >> 1) * P.box; };
    auto panel_of = [&](int e) { return D == 64 || P.merged ? 0 : e & 1; };
    auto place_of = [&](int e) {         // of copy e in a tile: halves of 64 tokens, then panels of 64 elements
      const int token = token_of(e);
      return (token >> 6) * S_::HALF + panel_of(e) * (64 * 128) + (token & 63) * 128;
    };
    const int first = lane * 2 + (warp - 10), my_token = first < copies ? token_of(first) : PTILE, my_x = panel_of(first) * 64;
    const uint32_t my_place = ring + place_of(first);
    // (keys and values go first when the L2 is full: the pieces' results are to stay there for the join)
    const uint64_t policy = evict_first_policy();
    uint32_t stage = 0, phase = 1, n = 0;                // n: tiles so far
    // of the streams' last tile of keys, whose values come next: the page and place of this lane's copy (a page
    // number past the last: nothing to copy), and how many copies of the warp there are
    uint32_t page[2] = {~0u, ~0u}, count[2] = {0, 0};
    int place[2] = {0, 0};
    auto look = [&](const Tile& x, int token, uint32_t& pg, int& pl) {
      pg = ~0u;
      if (token < x.count) {
        const uint32_t number = page_of(P.c, P.page_magic, x.t + token, pl);
        pg = static_cast<uint32_t>(__ldg(P.c.table + x.seq0 * P.c.table_stride + number));
      }
    };
    auto copy = [&](const CUtensorMap& map, const Tile& x, uint32_t pg, int pl, uint32_t all) {
      const uint32_t bar = full + 8 * stage;
      if (copies > 64)                   // (boxes of 1 or 2 tokens)
        for (int e = first + 64; e < copies; e += 64) {
          uint32_t p2;
          int l2;
          look(x, token_of(e), p2, l2);
          all += __popc(__ballot_sync(0xffffffffu, p2 < pages));
        }
      const bool go = wait(empty + 8 * stage, phase);
      if (__all_sync(0xffffffffu, go)) {
        if (lane == 0) mbar_arrive_expect_tx(bar, all * bytes);
        __syncwarp();
        if (pg < pages) {
          const int c1 = P.head_first ? x.head : pl, c2 = P.head_first ? pl : x.head;
          if (P.merged) copy_box5(my_place + stage * S_::TILE, map, c1, c2, pg, bar, policy);
          else copy_box(my_place + stage * S_::TILE, map, my_x, c1, c2, pg, bar, policy);
        }
        if (copies > 64)
          for (int e = first + 64; e < copies; e += 64) {
            uint32_t p2;
            int l2;
            look(x, token_of(e), p2, l2);
            if (p2 < pages)
              copy_box(ring + stage * S_::TILE + place_of(e), map, panel_of(e) * 64, P.head_first ? x.head : l2,
                       P.head_first ? l2 : x.head, p2, bar, policy);
          }
        __syncwarp();
      }
      ++n;
      if (++stage == S_::STAGES) stage = 0, phase ^= 1;
    };
    way.walk(P, [&](int s, const Tile& x, const Tile& y, bool) {
      // the next keys are looked up while the values before them are copied
      const bool keys = y.count > 0 && !(y.both && s == 1);
      uint32_t pg = ~0u;
      int pl = 0;
      if (keys) look(y, my_token, pg, pl);
      if (x.count > 0 && !(x.both && s == 1)) copy(maps.v, x, page[s], place[s], count[s]);
      if (keys) {
        page[s] = pg;
        place[s] = pl;
        count[s] = __popc(__ballot_sync(0xffffffffu, pg < pages));
        copy(maps.k, y, pg, pl, count[s]);
      }
    });
    // where the products ended early, the CTA stays for its last copies
    if (*dead)
      for (uint32_t k = n > S_::STAGES ? n - S_::STAGES : 0; k < n; ++k) {
        const unsigned long long t0 = global_timer();
        while (!mbar_try(full + 8 * (k % S_::STAGES), (k / S_::STAGES) & 1) && global_timer() - t0 < TIMEOUT_NS) {}
      }
  } else if (warp >= 8) {
    // ---- a stream's products: the warp goes together, one thread issues
    constexpr uint32_t IDESC = (1u << 4) | (W::FORMAT << 7) | (W::FORMAT << 10) | (static_cast<uint32_t>(PTILE >> 4) << 24);
    constexpr uint32_t IDESC_QK = IDESC | (static_cast<uint32_t>(PTILE / 2 >> 3) << 17);
    constexpr uint32_t IDESC_PV = IDESC | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17);
    begin();
    const int mine = warp - 8;
    // whether a wait gave up: one answer for all lanes, which go on together
    auto ended = [&]() { return __any_sync(0xffffffffu, *dead != 0u) != 0; };
    const uint32_t scores = tmem + mine * PTILE, result = tmem + 2 * PTILE + mine * 128;
    uint32_t n = 0, value_at = 0, key_at = 0, uses[2] = {0, 0}, blocks = 0, halves = 0;   // tiles, waits, halves of tiles so far
    // Both streams' warps go by every tile, so that neither is ever more than one round of the ring
    // behind: a stage is free when both have let it go, at once where the tile is the other's.
    auto take = [&](int s, const Tile& x, uint32_t& at) {
      if (!(x.both && s == 1)) at = n++;
      if (s != mine && x.both) return;
      wait(full + 8 * (at % S_::STAGES), at / S_::STAGES);
      __syncwarp();
      if (s != mine && lane == 0) mbar_arrive(empty + 8 * (at % S_::STAGES));
    };
    way.walk(P, [&](int s, const Tile& x, const Tile& y, bool asks) {
      if (s != mine) {
        if (x.count > 0) take(s, x, value_at);
        if (y.count > 0) take(s, y, key_at);
        return;
      }
      if (x.count > 0) take(s, x, value_at);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // the results of half a tile
        if (h * 64 < x.count) {
          wait(weighed + 16 * mine + 8 * h, uses[h]++);
          if (!ended()) {
            tc_fence_after();
            const uint64_t b = values_desc(ring + value_at % S_::STAGES * S_::TILE + h * S_::HALF, 64 * 128);
            if (elect_one()) {
              // the low parts, then the high ones; two products of 16 tokens at a time
#pragma unroll
              for (int part = 1; part >= 0; --part)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  if (h * 64 + c * 32 < x.count) {
                    const uint32_t a = scores + h * 64 + c * 32 + part * 16;
                    umma_ts(result, a, b + 256 * c, IDESC_PV, !x.first || h > 0 || part == 0 || c > 0);
                    umma_ts(result, a + 8, b + 256 * c + 128, IDESC_PV, true);
                  }
              umma_commit(summed + 16 * mine + 8 * (halves & 1));
              if (x.count <= h * 64 + 64) umma_commit(empty + 8 * (value_at % S_::STAGES));
            }
            __syncwarp();
          }
          ++halves;
        }
        // the scores of half of the next, in the place of what was just used
        if (h * 64 < y.count) {
          if (h == 0) {
            take(s, y, key_at);
            if (asks) wait(asked + 8 * mine, blocks++);
          }
          if (!ended()) {
            tc_fence_after();
            const uint64_t a = sw128_desc(queries + mine * S_::TILE), b = sw128_desc(ring + key_at % S_::STAGES * S_::TILE + h * S_::HALF);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = k % 4 * 32 >> 4;
                umma_ss(scores + h * 64, a + off + (k / 4 * S_::PANEL >> 4), b + off + (k / 4 * 64 * 128 >> 4), IDESC_QK, k > 0);
              }
              umma_commit(scored + 16 * mine + 8 * h);
              if (y.count <= h * 64 + 64) umma_commit(empty + 8 * (key_at % S_::STAGES));
            }
            __syncwarp();
          }
        }
      }
    });
    if (elect_one()) umma_commit(last);  // nothing is left under way when tensor memory is given back
    __syncwarp();
    const unsigned long long t0 = global_timer();
    while (!mbar_try(last, 0) && global_timer() - t0 < TIMEOUT_NS) {}
    __syncwarp();
  } else {
    // ---- exponentials: a thread to a query row
    const int s = warp >> 2, row = tid & (PTILE - 1);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t scores = tmem + s * PTILE + lanes, result = tmem + 2 * PTILE + s * 128 + lanes;
    uint32_t used0 = 0, used1 = 0, total = 0;              // waits so far; halves of tiles so far
    // Half n's part of the result.  Even and odd halves have a barrier each: when a half has its scores, the
    // result of the one before the last is in, so that no wait is two rounds behind, whichever are left out.
    auto result_in = [&](uint32_t n) { return wait(summed + 16 * s + 8 * (n & 1), n >> 1); };
    Step st, nxt;
    Rows held;
    // Before the plan is made, half a tile without scores in the result's place: it brings the instructions,
    // which would be 3 us of the first half's 4.
    bool have = true, dry = true;
    st.len0 = st.len1 = 64;
    int64_t out = -1;                    // the first part of the row's sequence and kv head, in rows; -1: no query
    int row_in = 0;                      // the row in its sequence
    auto ask = [&](const Step& x) {      // the queries of the stream's rows of x
      held.take(x);
      const int at = x.rb * PROWS + (x.both ? s * PTILE : 0) + row, k = at / P.rows, r = at - k * P.rows, i = r / P.group, b = x.seq0 + k;
      out = -1;
      const uint4* src = nullptr;
      if (k < x.seqs) {
        const int nnew = P.c.new_lens ? P.c.new_lens[b] : P.c.n;
        if (P.first[b] >= 0 && i < nnew) {
          out = (static_cast<int64_t>(b) * P.c.kv_heads + x.head) * P.pieces * P.rows;
          row_in = r;
          src = reinterpret_cast<const uint4*>(static_cast<const T*>(P.q) + b * P.qs.batch + i * P.qs.token +
                                               (x.head * P.group + (r - i * P.group)) * P.qs.head);
        }
      }
      const uint32_t dst = queries + s * S_::TILE + row * 128;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        uint4 v = src ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
        v.x ^= P.q_sign, v.y ^= P.q_sign, v.z ^= P.q_sign, v.w ^= P.q_sign;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                     :: "r"(dst + c / 8 * S_::PANEL + ((c & 7) ^ (row & 7)) * 16), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(asked + 8 * s);
    };
    auto missing = [&](const Step& x) {  // whether one of the stream's pages of x that the lane looks at is not there
      bool bad = false;
      int place;
      const int to = static_cast<int>(page_of(P.c, P.page_magic, x.from(s) + x.tokens(s) - 1, place));
      for (int p = static_cast<int>(page_of(P.c, P.page_magic, x.from(s), place)) + lane; p <= to; p += 32) {
        const int page = __ldg(P.c.table + x.seq0 * P.c.table_stride + p);
        bad |= page < 0 || page >= P.c.num_pages;
      }
      return bad;
    };
    bool bad = false;
    for (; have; st = nxt) {
      bool more = false;
      const int all = st.tokens(s);
      if (all > 0) {
        float m = -INFINITY, l = 0.0f;
        const int halves = (all + 63) / 64;
#pragma unroll 1
        for (int h = 0; h < halves; ++h) {
          const bool two = all - h * 64 > 32;                    // 64 tokens, not 32
          const uint32_t at = dry ? result : scores + (h & 1) * 64;
          if (!dry) {
            if (h & 1) wait(scored + 16 * s + 8, used1++);
            else wait(scored + 16 * s, used0++);
          }
          __syncwarp();
          tc_fence_after();
          uint32_t x[2][32];
          tmem_ld32_async(at, x[0]);
          tmem_ld32_async(at + 32, x[1]);
          tmem_wait_ld();
          tmem_loaded(x[0]);
          tmem_loaded(x[1]);
          float top = -INFINITY, t2 = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            top = fmaxf(top, fmaxf(__uint_as_float(x[0][e]), __uint_as_float(x[0][e + 1])));
            t2 = fmaxf(t2, fmaxf(__uint_as_float(x[1][e]), __uint_as_float(x[1][e + 1])));
          }
          if (two) top = fmaxf(top, t2);
          top *= P.c2;
          float fac = 1.0f;
          if (top > m + W::SLACK) {
            if (m != -INFINITY) fac = ex2(m - top);
            m = top;
          }
          if (__any_sync(0xffffffffu, fac != 1.0f) && !dry) {
            l *= fac;
            result_in(total - 1);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t y[32];
              tmem_ld32_async(result + 32 * c, y);
              tmem_wait_ld();
              tmem_loaded(y);
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * fac);
              tmem_st32(result + 32 * c, y);
            }
          }
          const float sub = m == -INFINITY ? W::OFF : W::OFF - m;
          const uint64_t sub2 = pack2(sub, sub), c22 = pack2(P.c2, P.c2);
          uint64_t sum2 = 0;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (c == 1 && !two) continue;
            // 32 scores become 16 words of hi and 16 of lo, in their place
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float a, b;
              unpack2(fma2(pack2(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1])), c22, sub2), a, b);
              a = ex2(a);
              b = ex2(b);
              sum2 = add2(sum2, pack2(a, b));
              W::split(a, b, hi[e], lo[e]);
            }
            tmem_st16(at + 32 * c, hi);
            tmem_st16(at + 32 * c + 16, lo);
          }
          float sum0, sum1;
          unpack2(sum2, sum0, sum1);
          l += sum0 + sum1;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (!dry) {
            ++total;
            if (lane == 0) mbar_arrive(weighed + 16 * s + 8 * (h & 1));
          }
          __syncwarp();
        }
        const int64_t slot_at = out + static_cast<int64_t>(st.piece_of(s)) * P.rows;
        const bool query = out >= 0;
        const int r = row_in;
        if (dry) {
          dry = false;
          begin();
          have = way.next(P, nxt);
          if (have && nxt.tokens(s) > 0) {
            ask(nxt);
            bad = missing(nxt);
          }
          continue;
        }
        // What the next piece needs is looked up before this one's result goes out: a load waits for the stores
        // before it (2 us of them here).  All products with the queries of this one are done.
        more = way.next(P, nxt);
        bool bad_next = false;
        if (more && nxt.tokens(s) > 0) {
          if (!held.of(nxt)) ask(nxt);
          bad_next = missing(nxt);
        }
        bad |= !result_in(total - 1) || *dead != 0u;
        bad = __any_sync(0xffffffffu, bad);
        tc_fence_after();
        if (*dead && (warp & 3) == 0 && lane == 0 && P.c.err) atomicAdd(P.c.err, 1);         // (missing pages are the join's to count)
        const int64_t step = 8 * static_cast<int64_t>(P.rows);
        float* const to = P.piece_o + slot_at * D + 8 * static_cast<int64_t>(r);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t y[32];
          tmem_ld32_async(result + 32 * c, y);
          tmem_wait_ld();
          tmem_loaded(y);
          if (query) {
            if constexpr (W::TO_PIECES != 1.0f) {
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * W::TO_PIECES);
            }
#pragma unroll
            for (int e = 0; e < 32; e += 8) store8(to + (4 * c + e / 8) * step, y + e);
          }
          __syncwarp();
        }
        if (query) P.piece_ml[slot_at + r] = bad ? bad_part() : make_float2(m, l * W::TO_PIECES);
        bad = bad_next;
      } else {
        more = way.next(P, nxt);
        if (more && nxt.tokens(s) > 0) {
          if (!held.of(nxt)) ask(nxt);
          bad = missing(nxt);
        }
      }
      have = more;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------ host side

// The four launches, with all that can be refused before the first of them.
template <class T, int D>
static rlk_status launch_prefix(const PrefixParams& P, bool bf16, cudaStream_t st) {
  static bool done[64] = {};
  const bool shared = P.pieces > 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && shared && (dev >= 64 || !done[dev])) {
    e = cudaFuncSetAttribute(prefix_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, PShape<D>::SMEM);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
  }
  if (e != cudaSuccess) return fail(RLK_ECUDA, "function attributes: %s", cudaGetErrorString(e));
  CacheMaps maps{}, tail_maps{};
  rlk_status s;
  if (shared && P.c.num_pages > 0) {
    if ((s = map_cache(&maps.k, P.c, P.c.k, P.box, P.head_first, P.merged ? 2 : 1, D, bf16)) != RLK_OK) return s;
    if ((s = map_cache(&maps.v, P.c, P.c.v, P.box, P.head_first, P.merged ? 2 : 1, D, bf16)) != RLK_OK) return s;
  }
  if ((s = attend_tails(P, tail_maps, D, bf16, Tails::prepare, st)) != RLK_OK) return s;
  plan_kernel<<<1, PLAN_THREADS, 0, st>>>(P);
  e = cudaGetLastError();
  if (e != cudaSuccess) return fail(RLK_ECUDA, "kernel launch: %s", cudaGetErrorString(e));
  if (!shared) return attend_tails(P, tail_maps, D, bf16, Tails::alone, st);
  // launched while the plan is made, for which it waits
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(PSMS);
  cfg.blockDim = dim3(PTHREADS);
  cfg.dynamicSmemBytes = PShape<D>::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefix_kernel<T, D>, P, maps);
  if (e != cudaSuccess) return fail(RLK_ECUDA, "kernel launch: %s", cudaGetErrorString(e));
  return attend_tails(P, tail_maps, D, bf16, Tails::beside, st);
}

static size_t lined(size_t x) { return (x + 127) / 128 * 128; }

// The workspace, in this order; each part on a line of its own.
struct PrefixLayout {
  size_t first, tails_at, plan, busy, base, piece_ml, tail_ml, piece_o, tail_o, bytes;
  int pieces, tails;
};
static PrefixLayout prefix_layout(int64_t B, int64_t n, int64_t q_heads, int64_t head_dim, int64_t max_tokens, int groups, int max_shared) {
  PrefixLayout y{};
  for (const int most : {PIECES_1024 - 1, PIECES_2048 - 1, 0x7fffffff}) {
    const int pieces = pieces_of((max_shared < most ? max_shared : most) / PREFIX_STEP * PREFIX_STEP);
    y.pieces = pieces > y.pieces ? pieces : y.pieces;
  }
  if (groups == 0) y.pieces = 0;
  const int tokens = static_cast<int>(max_tokens < 0x7fffffff ? max_tokens : 0x7fffffff);
  y.tails = tail_parts(tokens);
  const size_t rows = static_cast<size_t>(B) * n * q_heads, pieces = rows * y.pieces, tails = rows * y.tails;
  size_t at = 0;
  auto next = [&](size_t bytes) {
    const size_t here = at;
    at += lined(bytes);
    return here;
  };
  y.first = next(static_cast<size_t>(B) * 4);
  y.tails_at = next(static_cast<size_t>(B + 1) * 4 * (tail_level(tokens > 0 ? tokens - 1 : 0) + 1));
  y.plan = next(static_cast<size_t>(groups) * sizeof(GroupPlan));
  y.busy = next(static_cast<size_t>(groups) * 4);
  y.base = next((static_cast<size_t>(groups) + 5) * 4);
  y.piece_ml = next(pieces * 8);
  y.tail_ml = next(tails * 8);
  y.piece_o = next(pieces * head_dim * 4);
  y.tail_o = next(tails * head_dim * 4);
  y.bytes = at + 128;                    // (the caller's memory may begin between two lines)
  return y;
}

}  // namespace rlk

using namespace rlk;

extern "C" {

rlk_status rlk_prefix_attention_workspace(int64_t B, int32_t n, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                          int64_t max_tokens, int32_t groups, int32_t max_shared, size_t* bytes) {
  if (B < 0 || n < 0 || q_heads < 0 || head_dim < 0 || max_tokens < 0) return fail(RLK_EINVAL, "a size is negative");
  if (!bytes) return fail(RLK_EINVAL, "bytes is NULL");
  if (kv_heads < 1 || q_heads % kv_heads) return fail(RLK_EINVAL, "q_heads %d must be a multiple of kv_heads %d", q_heads, kv_heads);
  if (groups < 0 || groups >= (1 << 16)) return fail(RLK_EINVAL, "groups %d must be in 0..65535", groups);
  if (max_shared < 0 || max_shared > max_tokens)
    return fail(RLK_EINVAL, "max_shared %d must be in 0..%lld", max_shared, (long long)max_tokens);
  *bytes = B == 0 || n == 0 || q_heads == 0 ? 0 : prefix_layout(B, n, q_heads, head_dim, max_tokens, groups, max_shared).bytes;
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
  size_t bytes = 0;
  if ((s = rlk_prefix_attention_workspace(cache->B, cache->n, q_heads, cache->kv_heads, cache->head_dim, tokens, groups->groups,
                                          groups->max_shared, &bytes)) != RLK_OK)
    return s;
  if (!aligned(groups->group_start, 4) || !aligned(groups->shared_lens, 4))
    return fail(RLK_EALIGN, "group_start or shared_lens is not 4-byte aligned");
  if (cache->B == 0 || cache->n == 0) return RLK_OK;
  if (groups->groups > 0 && (!groups->group_start || !groups->shared_lens))
    return fail(RLK_EINVAL, "group_start or shared_lens is NULL");
  if (tokens > 0x7fffffff - 64) return fail(RLK_EINVAL, "max_pages * page_size is above 2^31 - 65");
  const double rows = static_cast<double>(cache->B) * cache->n * (q_heads / cache->kv_heads);
  if (rows >= 2147483392.0 || (rows / 128 + groups->groups) * cache->kv_heads * (groups->max_shared / 512 + 4.0) >= 2147483648.0 ||
      static_cast<double>(cache->B) * (tokens / 16 + 1.0) >= 2147483648.0)
    return fail(RLK_EINVAL, "too many query rows or tokens for one call");
  if ((s = check_bth(q, q_strides, "q")) != RLK_OK) return s;
  if ((s = check_bth(out, out_strides, "out")) != RLK_OK) return s;
  if ((s = check_out(out_lse, "out_lse", false)) != RLK_OK) return s;
  if (!workspace) return fail(RLK_EINVAL, "workspace is NULL");
  if (!aligned(workspace, 16)) return fail(RLK_EALIGN, "workspace is not 16-byte aligned");
  const PrefixLayout y = prefix_layout(cache->B, cache->n, q_heads, cache->head_dim, tokens, groups->groups, groups->max_shared);
  char* ws = reinterpret_cast<char*>(lined(reinterpret_cast<size_t>(workspace)));
  PrefixParams P{};
  P.c = paged_params(cache);
  P.group_start = groups->group_start;
  P.shared_lens = groups->shared_lens;
  P.groups = groups->groups;
  P.max_shared = groups->max_shared;
  P.B = cache->B;
  P.plan_first = reinterpret_cast<int32_t*>(ws + y.first);
  P.plan_tails = reinterpret_cast<uint32_t*>(ws + y.tails_at);
  P.first = P.plan_first;
  P.tail_base = P.plan_tails;
  P.plan = reinterpret_cast<GroupPlan*>(ws + y.plan);
  P.busy = reinterpret_cast<int32_t*>(ws + y.busy);
  P.base = reinterpret_cast<uint32_t*>(ws + y.base);
  P.taken = P.base + groups->groups + 2;
  P.piece_ml = reinterpret_cast<float2*>(ws + y.piece_ml);
  P.piece_o = reinterpret_cast<float*>(ws + y.piece_o);
  P.tail_ml = reinterpret_cast<float2*>(ws + y.tail_ml);
  P.tail_o = reinterpret_cast<float*>(ws + y.tail_o);
  P.pieces = y.pieces;
  P.tails = y.tails;
  P.q = q;
  P.qs = *q_strides;
  P.out = out;
  P.os = *out_strides;
  P.lse = out_lse;
  P.q_heads = q_heads;
  P.group = q_heads / cache->kv_heads;
  P.rows = cache->n * P.group;
  P.c2 = fabsf(scale) * 1.4426950408889634f;
  P.q_sign = scale < 0.0f ? 0x80008000u : 0u;
  const TailTiles tt = tail_tiles(P.rows);
  P.unit_cost = cache->head_dim == 128 ? UNIT_COST_128 : UNIT_COST_64;
  P.tail_cost = static_cast<uint32_t>(tt.tiles) * tt.nt * cache->kv_heads;
  P.box = box_of(cache->page_size, PTILE / 2);
  P.merged = P.box == 64 && cache->head_dim == 128;
  P.head_first = heads_first(cache);
  P.page_magic = page_magic(cache->page_size);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = cache->dtype == RLK_DT_BF16;
  if (cache->head_dim == 128) return bf ? launch_prefix<bf16_t, 128>(P, bf, st) : launch_prefix<__half, 128>(P, bf, st);
  return bf ? launch_prefix<bf16_t, 64>(P, bf, st) : launch_prefix<__half, 64>(P, bf, st);
}

}  // extern "C"
