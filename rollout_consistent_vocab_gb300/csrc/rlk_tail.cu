// rlk_tail.cu -- attention over a shared prefix: every sequence's own tokens behind it, and
// the join with the shared tokens' parts.
//
// Own tokens are many short runs: hundreds of samples, each with some hundred tokens
// per kv head.  So a warp goes by itself: it takes a chunk of parts at a time (up to 256
// tokens of a sequence and kv head, more for long ones), brings its keys and values by TMA
// into a ring of its own, 16 tokens at a time, and meets no barrier but the ring's.  S^T = K Q^T and
// O^T += V^T P^T run on mma.sync with 16 tokens (or elements) as rows and 8 query rows as
// columns, up to three tiles of 8 rows on the same copy.  A part's maximum, sum and
// weighted sum of values go to the workspace, so that it is of no account which warp has it.
// The kernel's CTAs come to the SMs that the shared tokens' kernel leaves free, some at once
// and the others when it ends; chunks go to whoever is there.
//
// Bound by memory where rows are few: 256 sequences of up to 2048 own tokens, 8 kv heads of 128 with 4
// rows, 614 MB, 107 us by itself = 5.8 TB/s.  With 20 rows by the latency of a step's products and
// exponentials, of which an SM has eight warps (16 x 8 sequences of up to 1024 tokens, 154 MB, some 70 us).
// Equal runs of steps for all warps, dealt out beforehand and behind the other kernel: 16 x 16 samples 177 us
// for 158.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "rlk_attn.cuh"
#include "rlk_device.cuh"
#include "rlk_host.h"
#include "rlk_paged.h"
#include "rlk_tcgen05.cuh"

namespace rlk {

constexpr int TSTEP = 16;                // tokens of a step
constexpr int TWARPS = 8;                // of a CTA, one CTA to an SM
constexpr int TSMS = 152;
template <int D>
struct TShape {
  static constexpr int PANEL = TSTEP * 128;        // 64 elements of 16 tokens, 128-byte swizzle
  static constexpr int KEYS = D / 64 * PANEL;
  static constexpr int STAGE = 2 * KEYS;           // keys, then values
  static constexpr int STAGES = D == 128 ? 3 : 6;
  static constexpr int SMEM = TWARPS * STAGES * STAGE + 1024;
};

struct TailParams {
  PrefixParts p;
  int tiles, box;               // row tiles of 8 NT rows; tokens of a copy: the largest power of 2, up to 16, in a page
  bool merged;                  // a copy takes all 128 elements of its 16 tokens
};

// A place in a warp's chunk: a part of a sequence, kv head and row tile, tokens t .. end - 1.
struct TailPlace {
  int b, ht, part, t, end;
  int len, nnew, first;         // of the sequence: its lengths, where its own tokens begin
  int left;                     // steps of the chunk from this part's begin on (the part is the chunk's if there are any)
  __device__ __forceinline__ void load(const PrefixParts& P) {
    nnew = P.c.new_lens ? P.c.new_lens[b] : P.c.n;
    first = P.first[b];
    // (within bounds, should the lengths have changed since they were looked over)
    len = max(first, min(P.c.lens[b], static_cast<int>(min(static_cast<int64_t>(P.c.max_pages) * P.c.page_size, static_cast<int64_t>(0x7fffffff)))));
  }
  __device__ __forceinline__ void cut(int from) {
    t = from;
    end = min(len, t + min(tail_part_tokens(part), len - t));
  }
};

// The next part; false at the chunk's end.  The longest parts come first,
// so that none is begun when the others end (4 sequences of 100,000 tokens, parts of up to 4096 tokens: 380 us in the
// order of their places, 327 so).
__device__ __forceinline__ bool next_part(const TailParams& P, TailPlace& x, int HT) {
  do {
    x.left -= (x.end - x.first - tail_part_from(x.part) + TSTEP - 1) / TSTEP;
    if (x.left <= 0) return false;
    int level = tail_part_level(x.part), from = x.end;
    if (x.end < x.len && tail_part_level(x.part + 1) == level) {
      ++x.part;
    } else {
      if (++x.ht == HT) {
        x.ht = 0;
        const uint32_t* base;
        do {
          if (++x.b >= P.p.B) {
            if (level == 0) return false;
            --level;
            x.b = 0;
          }
          base = P.p.tail_base + level * (P.p.B + 1) + x.b;
        } while (base[1] == base[0]);
        x.load(P.p);
      }
      x.part = tail_level_part(level);
      from = x.first + tail_level_from(level);
    }
    x.cut(from);
  } while (x.t >= x.end);                // (only should the lengths have changed)
  return true;
}

__device__ __forceinline__ int row_query(const PrefixParts& P, int row) { return row / P.group; }

template <class T, int D, int NT>
__global__ void __launch_bounds__(TWARPS * 32, 1)
tail_kernel(const __grid_constant__ TailParams P, const __grid_constant__ CacheMaps maps) {
  using S_ = TShape<D>;
  using E = Elem<T>;
  constexpr int KK = D / 16, DT = D / 16;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ uint64_t bars[TWARPS][S_::STAGES];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t ring = ((smem_addr(smem_raw) + 1023u) & ~1023u) + warp * (S_::STAGES * S_::STAGE);
  const uint32_t full = smem_addr(&bars[warp][0]);
  if (lane < S_::STAGES) {
    mbar_init(full + lane * 8, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncwarp();

  const int HT = P.p.c.kv_heads * P.tiles;
  // A chunk: a quarter of an equal share (half of one is slower by a twentieth, an eighth no faster), but a
  // part's 16 steps where that is less, and a share where there are not so many.
  const int64_t each = static_cast<int64_t>(P.p.taken[2]) * HT / (TSMS * TWARPS);
  const int chunk = static_cast<int>(min(max(each / 4, min(max(each, static_cast<int64_t>(1)), static_cast<int64_t>(256 / TSTEP))), static_cast<int64_t>(1) << 29));
  TailPlace load_at, work_at;
  bool have = false;
  // ---- the next chunk of all steps that no warp has: the parts that begin there.  False where none is left.
  auto take = [&]() {
    uint32_t k = 0;
    // (looked up while the counter is; they would be in the products' way)
    int level = static_cast<int>(P.p.taken[1]);
    const uint32_t all = P.p.taken[2];
    if (lane == 0) k = atomicAdd(P.p.taken, 1u);
    const int64_t from = static_cast<int64_t>(__shfl_sync(0xffffffffu, k, 0)) * chunk, to = min(static_cast<int64_t>(all) * HT, from + chunk);
    if (from >= to) return false;
    // the last sequence that begins at or before it
    int64_t rest = from;
    const uint32_t* base = P.p.tail_base + level * (P.p.B + 1);
    for (; level > 0 && rest >= static_cast<int64_t>(base[P.p.B]) * HT; --level, base -= P.p.B + 1) rest -= static_cast<int64_t>(base[P.p.B]) * HT;
    const uint32_t at = static_cast<uint32_t>(rest / HT);
    int lo = 0, hi = static_cast<int>(P.p.B);
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, mine = lo + lane * step;
      const uint32_t below = __ballot_sync(0xffffffffu, mine < hi && base[mine] <= at);
      lo += (31 - __clz(below)) * step;
      hi = min(hi, lo + step);
    }
    TailPlace x;
    x.b = lo;
    x.load(P.p);
    const int64_t steps = base[lo + 1] - base[lo];
    rest -= static_cast<int64_t>(base[lo]) * HT;
    x.ht = static_cast<int>(min(rest / max(steps, static_cast<int64_t>(1)), static_cast<int64_t>(HT - 1)));
    const int64_t in = rest - x.ht * steps + tail_level_from(level) / TSTEP;
    // (within its tokens, should the lengths have changed)
    x.part = tail_part_of(static_cast<int>(min(in * TSTEP, static_cast<int64_t>(max(x.len - x.first, 1) - 1))));
    const int over = static_cast<int>(in - tail_part_from(x.part) / TSTEP);
    x.left = static_cast<int>(to - from) + over;           // (from where the part begins that holds the chunk's first step)
    x.cut(x.first + tail_part_from(x.part));
    have = over > 0 || x.t >= x.end ? next_part(P, x, HT) : true;
    work_at = load_at = x;
    return true;
  };

  // ---- copies: a step's pages are looked up while the step before is worked on.  Lanes 0-15 have the
  // tokens' keys, 16-31 their values; the first of a box speaks for it.
  constexpr int PANELS = D / 64;
  const uint64_t policy = evict_first_policy();            // (read once)
  bool more = false;
  int page = -1, place = 0;
  bool speaks = false;
  auto look = [&]() {
    const int in = lane & (TSTEP - 1), t = load_at.t + in;
    speaks = more && (in & (P.box - 1)) == 0 && t < load_at.end;
    if (speaks) page = __ldg(P.p.c.table + load_at.b * P.p.c.table_stride + page_of(P.p.c, P.p.page_magic, t, place));
  };
  uint32_t bad_stages = 0;
  int put = 0, under_way = 0;            // stage of the next copy; copies that were not waited for yet
  auto copy = [&]() {                    // the step that is looked up; on to the next one
    const bool copies = speaks && page >= 0 && page < P.p.c.num_pages;
    const uint32_t bar = full + put * 8;
    const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, copies));
    const bool bad = __any_sync(0xffffffffu, speaks && !copies);
    bad_stages = (bad_stages & ~(1u << put)) | (bad ? 1u << put : 0u);
    if (lane == 0) mbar_arrive_expect_tx(bar, boxes * P.box * D * 2);
    __syncwarp();
    if (copies) {
      const int head = load_at.ht / P.tiles;
      const int c1 = P.p.head_first ? head : place, c2 = P.p.head_first ? place : head;
      const CUtensorMap& map = lane < TSTEP ? maps.k : maps.v;
      const uint32_t dst = ring + put * S_::STAGE + (lane < TSTEP ? 0 : S_::KEYS) + (lane & (TSTEP - 1)) * 128;
      if (P.merged) {
        copy_box5(dst, map, c1, c2, page, bar, policy);
      } else {
        for (int c = 0; c < PANELS; ++c) copy_box(dst + c * S_::PANEL, map, c * 64, c1, c2, page, bar, policy);
      }
    }
    ++under_way;
    if (++put == S_::STAGES) put = 0;
    load_at.t += TSTEP;
    if (load_at.t >= load_at.end) more = next_part(P, load_at, HT);
    look();
  };
  const int g8 = lane >> 2, t4 = lane & 3;
  const uint32_t klane = (((lane >> 3) & 1) * 8 + (lane & 7)) * 128 + (((lane >> 4) ^ (lane & 7)) * 16);
  const uint32_t vlane = ((lane >> 4) * 8 + (lane & 7)) * 128 + ((((lane >> 3) & 1) ^ (lane & 7)) * 16);
  int get = 0, phase = 0;
  bool dead = false;                     // a copy did not come
  int held_b = -1, held_ht = -1;
  uint32_t qf[NT][KK][2];
#pragma unroll 1
  while (take()) {
    more = have && !dead;
    look();
#pragma unroll 1
    for (int i = 0; i < S_::STAGES - 1; ++i)
      if (more) copy();
#pragma unroll 1
    while (have) {
      const int head = work_at.ht / P.tiles, row0 = (work_at.ht - head * P.tiles) * (8 * NT);
      if (work_at.b != held_b || work_at.ht != held_ht) {
        held_b = work_at.b, held_ht = work_at.ht;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          const int row = row0 + x * 8 + g8, i = row_query(P.p, row);
          const bool real = row < P.p.rows && i < work_at.nnew;
          const T* qp = static_cast<const T*>(P.p.q) + work_at.b * P.p.qs.batch + i * P.p.qs.token +
                        (head * P.p.group + (row - i * P.p.group)) * P.p.qs.head + t4 * 2;
#pragma unroll
          for (int k = 0; k < KK; ++k) {
            qf[x][k][0] = real ? __ldg(reinterpret_cast<const uint32_t*>(qp + k * 16)) ^ P.p.q_sign : 0u;
            qf[x][k][1] = real ? __ldg(reinterpret_cast<const uint32_t*>(qp + k * 16 + 8)) ^ P.p.q_sign : 0u;
          }
        }
      }
      float o[NT][DT][4], m[NT][2], l[NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[x][d][e] = 0.0f;
        m[x][0] = m[x][1] = -INFINITY, l[x][0] = l[x][1] = 0.0f;
      }
      bool part_bad = false;
      const int p0 = work_at.len - work_at.nnew;             // the queries stand at p0 .. len - 1
#pragma unroll 1
      for (int t0 = work_at.t; t0 < work_at.end; t0 += TSTEP) {
        if (more) copy();
        // (one answer for all lanes: with some given up and some not, the next exchange would find no end)
        if (!dead && !__all_sync(0xffffffffu, mbar_wait_phase(full + get * 8, phase))) {
          dead = true;
          more = false;
        }
        part_bad |= dead || ((bad_stages >> get) & 1u);
        const uint32_t sk = ring + get * S_::STAGE, sv = sk + S_::KEYS;
        if (!dead) {                       // (else it stays, for the end)
          --under_way;
          if (++get == S_::STAGES) get = 0, phase ^= 1;
        }
        __syncwarp();
        float s[NT][4];
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[x][e] = 0.0f;
#pragma unroll
        for (int k = 0; k < KK; ++k) {
          uint32_t a[4];
          ldsm(a, sk + (klane ^ (32 * (k % 4))) + k / 4 * S_::PANEL);
#pragma unroll
          for (int x = 0; x < NT; ++x) E::mma(s[x], a, qf[x][k][0], qf[x][k][1]);
        }
        const bool masked = t0 + TSTEP - 1 > p0;
        bool odd = false;                  // values that are not finite among a masked step's
        if (masked) {
#pragma unroll
          for (int z = lane * 16; z < S_::KEYS; z += 512) odd |= E::odd(lds128(sv + z));
          odd = __any_sync(0xffffffffu, odd);
        }
        uint32_t pf[NT][4];                // weights: tokens 0-7 and 8-15, then what the dtype dropped of them
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          uint32_t hidden = 0;             // bit e (of the thread's scores)
          if (masked) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int i = row_query(P.p, row0 + x * 8 + 2 * t4 + e);           // at p0 + i, which 32 bits may not hold past the last token
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                const int t = t0 + g8 + 8 * f;
                if (t - p0 > i || t >= work_at.end) {
                  s[x][2 * f + e] = -INFINITY;
                  hidden |= 1u << (2 * f + e);
                }
              }
            }
          }
          // the reference m follows the row's maximum where that runs SLACK ahead, so weights stay below 2^SLACK
          float top[2];
          bool ahead = false;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[e] = fmaxf(s[x][e], s[x][2 + e]) * P.p.c2;
            ahead |= top[e] > m[x][e] + E::SLACK;
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
              if (mx > m[x][e] + E::SLACK) {
                if (m[x][e] != -INFINITY) {
                  fac[e] = ex2f(m[x][e] - mx);
                  scaled = true;
                }
                m[x][e] = mx;
              }
            }
            if (__any_sync(0xffffffffu, scaled)) {
              l[x][0] *= fac[0], l[x][1] *= fac[1];
#pragma unroll
              for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[x][d][e] *= fac[e & 1];
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float sub = m[x][e] == -INFINITY ? E::OFF : E::OFF - m[x][e];
#pragma unroll
            for (int f = 0; f < 4; f += 2) s[x][f + e] = ex2f(__fmaf_rn(s[x][f + e], P.p.c2, sub));
          }
          // A masked token's value must not come in even as 0 * inf: values that are not finite go straight
          // into the rows that see them, as the product would leave them (infinite, or NaN at a weight of 0), and
          // the product takes zeros for them.
          if (masked) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((hidden >> e) & 1u) s[x][e] = 0.0f;
            if (odd) {
#pragma unroll 1
              for (int r = 0; r < TSTEP; ++r) {
                const int t = t0 + r;
                if (t >= work_at.end) break;                       // (what lies in a place that nobody sees is of no account)
                bool w[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) w[e] = E::counts(__shfl_sync(0xffffffffu, r < 8 ? s[x][e] : s[x][2 + e], (r & 7) * 4 + t4));
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                  for (int f = 0; f < 2; ++f) {
                    const uint32_t bits = lds16(sv + r * 128 + d / 4 * S_::PANEL + (((2 * (d % 4) + f) ^ (r & 7)) * 16) + g8 * 2);
                    if ((bits & E::EXP & 0xFFFFu) != (E::EXP & 0xFFFFu)) continue;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                      if (t - p0 <= row_query(P.p, row0 + x * 8 + 2 * t4 + e)) o[x][d][2 * f + e] += w[e] ? E::value(bits) : __int_as_float(0x7fc00000);
                  }
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) l[x][e] += s[x][e] + s[x][2 + e];
          E::split(s[x][0], s[x][1], pf[x][0], pf[x][2]);
          E::split(s[x][2], s[x][3], pf[x][1], pf[x][3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) pf[x][e] = movm(pf[x][e]);
        }
        if (odd) {
#pragma unroll 1
          for (int d4 = 0; d4 < DT; d4 += 4) {
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              uint32_t a[1][4];
              ldsm_t(a[0], sv + (vlane ^ (32 * z)) + d4 / 4 * S_::PANEL);
              E::clear_odd(a[0]);
#pragma unroll
              for (int d = 0; d < DT; d += 4)
                if (d == d4) {
#pragma unroll
                  for (int x = 0; x < NT; ++x) E::weigh(o[x] + d + z, a, pf[x]);
                }
            }
          }
        } else {
#pragma unroll
          for (int d = 0; d < DT; d += 4) {
            uint32_t a[4][4];
#pragma unroll
            for (int z = 0; z < 4; ++z) ldsm_t(a[z], sv + (vlane ^ (32 * z)) + d / 4 * S_::PANEL);
#pragma unroll
            for (int x = 0; x < NT; ++x) E::weigh(o[x] + d, a, pf[x]);
          }
        }
        __syncwarp();                      // the stage may be filled again
      }
      // ---- the part's result
      if (dead && lane == 0 && P.p.c.err) atomicAdd(P.p.c.err, 1);         // (missing pages are the join's to count)
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[x][e];
#pragma unroll
          for (int z = 4; z < 32; z <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, z);
          const int row = row0 + x * 8 + 2 * t4 + e, i = row_query(P.p, row);
          if (row >= P.p.rows || i >= work_at.nnew) continue;
          const int64_t slot = ((static_cast<int64_t>(work_at.b) * P.p.c.kv_heads + head) * P.p.tails + work_at.part) * P.p.rows;
          float* dst = P.p.tail_o + slot * D + row * 8LL + g8;
          const int64_t chunk8 = P.p.rows * 8LL;
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            dst[2 * d * chunk8] = o[x][d][e];
            dst[(2 * d + 1) * chunk8] = o[x][d][2 + e];
          }
          if (g8 == 0) P.p.tail_ml[slot + row] = part_bad ? bad_part() : make_float2(m[x][e], sum);
        }
      have = next_part(P, work_at, HT);
    }
#pragma unroll 1
    for (; !dead && under_way > 0; --under_way) {            // (only should the lengths have changed)
      mbar_wait_phase(full + get * 8, phase);
      if (++get == S_::STAGES) get = 0, phase ^= 1;
    }
  }
  // Copies that nobody waited for (one did not come in time, or the lengths changed under the call): the
  // warp stays for them, within limits.
#pragma unroll 1
  for (; under_way > 0; --under_way) {
    mbar_wait_phase(full + get * 8, phase);
    if (++get == S_::STAGES) get = 0, phase ^= 1;
  }
  // (launched beside the shared tokens' kernel: the join goes by the end of this one alone)
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------ the join

// A thread to four elements of a row, in the order in which the parts lie: they go to two chains in
// turn, the shared tokens' first, whose sums are joined.  Bound by the latency of reads, of which each thread
// has a chain.  With more threads than are on the GPU at once each has two parts under way, and few registers;
// with fewer, eight (16 x 8 sequences with drafts, 655,360 threads: 14 us after the last part, with eight 24;
// 2 x 32 with 131,071 shared tokens, 65,536 threads: 15, with two 27).
constexpr int TJOIN = 256, JOIN_MANY = TSMS * 1024;        // threads of a CTA, and of all with two parts each
template <class T, int D, int AT_ONCE>
__global__ void __launch_bounds__(TJOIN, AT_ONCE == 2 ? 4 : 2) tail_join_kernel(const __grid_constant__ PrefixParts P) {
  const int64_t id = blockIdx.x * static_cast<int64_t>(TJOIN) + threadIdx.x, each = P.rows * static_cast<int64_t>(D / 4), bh = id / each;
  const uint32_t in = static_cast<uint32_t>(id - bh * each), two = in >> 1;        // (pairs of threads: 8 elements)
  const int d8 = two / P.rows, row = two - d8 * P.rows, i = row / P.group, half = (in & 1) * 4;
  const int b = static_cast<int>(bh / P.c.kv_heads), head = static_cast<int>(bh - static_cast<int64_t>(b) * P.c.kv_heads);
  if (b >= P.B) return;
  const int first = P.first[b], nnew = P.c.new_lens ? P.c.new_lens[b] : P.c.n, own = P.c.lens[b] - first;
  const bool ok = first >= 0, query = ok && i < nnew;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  JoinRow<128> chain[2];
  bool bad = !ok;
  if (query) {
    const int pieces = min(pieces_of(first), P.pieces), parts = pieces + min(tail_parts(own), P.tails);
    const int64_t shared = bh * P.pieces, tails = bh * P.tails - pieces;
    for (int p0 = 0; p0 < parts; p0 += AT_ONCE) {
      float2 h[AT_ONCE];
      float v[AT_ONCE][4];
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) {
        const int p = min(p0 + k, parts - 1);              // (past the last one: it again)
        const bool of_shared = p < pieces;
        const int64_t at = ((of_shared ? shared : tails) + p) * P.rows;
        h[k] = (of_shared ? P.piece_ml : P.tail_ml)[at + row];
        load_row<4>((of_shared ? P.piece_o : P.tail_o) + at * D + in * 4LL, v[k]);
      }
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k)
        if (p0 + k < parts) chain[k % 2].add(h[k].x, h[k].y, v[k]), bad |= h[k].x != h[k].x;
    }
    chain[0].add(chain[1]);
  }
  if (bad && in == 0 && head == 0 && P.c.err) atomicAdd(P.c.err, 1);       // a rejected sequence, once
  const JoinRow<128>& all = chain[0];
  const float inv = all.L == 0.0f ? 0.0f : __frcp_rn(all.L), nan = __int_as_float(0x7fc00000);
  const int hq = head * P.group + (row - i * P.group);
  T r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) from_float(!ok ? nan : !query ? 0.0f : __fmul_rn(all.o[e], inv), r[e]);
  T* op = static_cast<T*>(P.out) + b * P.os.batch + i * P.os.token + hq * P.os.head + d8 * 8 + half;
  *reinterpret_cast<uint2*>(op) = *reinterpret_cast<const uint2*>(r);
  if (P.lse && d8 == 0 && half == 0)
    P.lse[(static_cast<int64_t>(b) * P.c.n + i) * P.q_heads + hq] = !ok ? nan : !query ? -INFINITY : lse_of<T>(all.M, all.L);
}

// ------------------------------------------------------------ host side

template <class T, int D, int NT>
static rlk_status launch_tails(const TailParams& P, const CacheMaps& maps, Tails what, cudaStream_t st) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !done[dev])) {
    e = cudaFuncSetAttribute(tail_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, TShape<D>::SMEM);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
  }
  if (e != cudaSuccess) return fail(RLK_ECUDA, "function attributes: %s", cudaGetErrorString(e));
  if (what == Tails::prepare) return RLK_OK;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(TSMS);
  cfg.blockDim = dim3(TWARPS * 32);
  cfg.dynamicSmemBytes = TShape<D>::SMEM;
  cfg.stream = st;
  cfg.attrs = &attr;
  // (beside the shared tokens' kernel, which has waited for the plan)
  cfg.numAttrs = what == Tails::alone ? 0 : 1;
  e = cudaLaunchKernelEx(&cfg, tail_kernel<T, D, NT>, P, maps);
  if (e == cudaSuccess) {
    const int64_t threads = P.p.B * P.p.c.kv_heads * P.p.rows * (D / 4);
    cfg.gridDim = dim3(static_cast<unsigned>((threads + TJOIN - 1) / TJOIN));
    cfg.blockDim = dim3(TJOIN);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    e = threads > JOIN_MANY ? cudaLaunchKernelEx(&cfg, tail_join_kernel<T, D, 2>, P.p) : cudaLaunchKernelEx(&cfg, tail_join_kernel<T, D, 8>, P.p);
  }
  if (e != cudaSuccess) return fail(RLK_ECUDA, "kernel launch: %s", cudaGetErrorString(e));
  return RLK_OK;
}
template <class T, int D>
static rlk_status launch_tail_rows(const TailParams& P, const CacheMaps& maps, int nt, Tails what, cudaStream_t st) {
  switch (nt) {
    case 1: return launch_tails<T, D, 1>(P, maps, what, st);
    case 2: return launch_tails<T, D, 2>(P, maps, what, st);
    default: return launch_tails<T, D, 3>(P, maps, what, st);
  }
}

rlk_status attend_tails(const PrefixParts& parts, CacheMaps& maps, int head_dim, bool bf16, Tails what, cudaStream_t stream) {
  TailParams P{};
  P.p = parts;
  const TailTiles tt = tail_tiles(parts.rows);
  P.tiles = tt.tiles;
  const int nt = tt.nt;
  P.box = box_of(parts.c.page_size, TSTEP);
  P.merged = P.box == TSTEP && head_dim == 128;
  rlk_status s;
  if (what == Tails::prepare && parts.c.num_pages > 0) {
    if ((s = map_cache(&maps.k, parts.c, parts.c.k, P.box, parts.head_first, P.merged ? 2 : 1, head_dim, bf16)) != RLK_OK) return s;
    if ((s = map_cache(&maps.v, parts.c, parts.c.v, P.box, parts.head_first, P.merged ? 2 : 1, head_dim, bf16)) != RLK_OK) return s;
  }
  if (head_dim == 128)
    return bf16 ? launch_tail_rows<__nv_bfloat16, 128>(P, maps, nt, what, stream) : launch_tail_rows<__half, 128>(P, maps, nt, what, stream);
  return bf16 ? launch_tail_rows<__nv_bfloat16, 64>(P, maps, nt, what, stream) : launch_tail_rows<__half, 64>(P, maps, nt, what, stream);
}

}  // namespace rlk
