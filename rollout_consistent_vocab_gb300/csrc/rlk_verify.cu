// rlk_verify.cu -- verification of drafted tokens by rejection sampling.
//
// Two launches.  The first (verify_pass, a form of the fused logprob kernel)
// resolves every row of both models in one pass over the logits: maximum,
// normalisers, the support's lowest key, and the drafted token's probability,
// 32 bytes a row.  The second, here, takes one cluster of 8 CTAs per sequence:
// every CTA finds the first refused draft a from the records, and the cluster
// draws from row a, CTA r on shard r.
//
// The draw's masses are the selection's fixed-point masses, so that sums are
// exact whatever their order: P_j = exp((x_j - M) / tau) 2^44, rounded, for the
// support's columns.  A residual takes q_j in the same unit, Q_j = q_j Z_S 2^44
// rounded, and the mass is max(P_j - Q_j, 0).
//
// The pass is the sampler's, and bound as that is: by the exchanges between a row's
// eight CTAs.  128 sequences with 4 drafts of a draft model (1152 rows, 0.35 GB, top-k
// 128): 0.0925 ms = 3.8 TB/s, the pass 0.083 of it.  The draw is latency: a thread takes
// one marked chunk, and CTAs of 128 threads, many to an SM, wait beside each other
// (with 512 threads and every chunk of the shard looked at: 0.150 ms the call).  Rows
// without a bitmap (unfiltered, or nuclei of thousands) are read in full: the same call
// unfiltered takes 0.177 ms, with top-p 0.95 alone 0.164.

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>
#include <string.h>

#include "rlk_rollout.h"
#include "rlk_device.cuh"
#include "rlk_host.h"

namespace rlk {

constexpr int VT = 128;                                   // threads of a draw CTA
constexpr int VW = VT / 32;
constexpr int ROUNDS = (SHARD_CHUNKS + VT - 1) / VT;      // of a chunk to a thread, at most
static_assert(SAMP_BITWORDS <= VT, "a bitmap word to a thread");

struct DrawParams {
  VerifyPass ver;
  const uint16_t* logits;
  int64_t stride;
  const uint16_t* draft;              // NULL: point masses
  int64_t draft_stride;
  const float* tau_arr;
  float tau_s;
  const uint32_t* bits;
  const uint32_t* accept;
  const uint32_t* draw;
  int32_t* out_token;
  int32_t* out_accepted;
  float* out_restr;
  float* out_full;
  int32_t* err;
};

// What a row's masses are taken from: the target's row and, for a residual,
// the draft model's.
struct Masses {
  float M, c;
  __nv_bfloat162 vmin2;
  int skip;                           // a column without mass (a refused point mass), or -1
  bool with_q;
  float Mq, cq, ratio;                // q_j Z_S = exp((y_j - Mq) cq) ratio
  __nv_bfloat162 vminq2;
  int q_one;                          // greedy draft: the column that holds all of q
  float q_one_mass;                   // Z_S 2^44
};

// Fixed-point masses of the 8 columns of a chunk (x: the target's, y: the draft's).
__device__ __forceinline__ unsigned long long chunk_masses(const Masses& m, uint4 x, uint4 y, int col0,
                                                           unsigned long long (&mass)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w}, z[4] = {y.x, y.y, y.z, y.w};
  unsigned long long sum = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t in = __hge2_mask(as_bf2(w[j]), m.vmin2);
    const uint32_t inq = m.with_q ? __hge2_mask(as_bf2(z[j]), m.vminq2) : 0u;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = col0 + 2 * j + e;
      unsigned long long v = 0;
      if (((in >> (16 * e)) & 1u) && col != m.skip) {
        v = qfx(e ? bf16_hi(w[j]) : bf16_lo(w[j]), m.M, m.c);
        if (m.with_q) {
          float q = 0.0f;
          if (m.q_one >= 0) q = col == m.q_one ? m.q_one_mass : 0.0f;
          else if ((inq >> (16 * e)) & 1u)
            q = ex2(((e ? bf16_hi(z[j]) : bf16_lo(z[j])) - m.Mq) * m.cq) * m.ratio;
          const unsigned long long qi = __float2ull_rn(q);
          v = v > qi ? v - qi : 0ull;
        }
      }
      mass[2 * j + e] = v;
      sum += v;
    }
  }
  return sum;
}

// Sums over the CTA in thread order: this thread's exclusive prefix, and the total.
__device__ __forceinline__ unsigned long long cta_scan(unsigned long long v, unsigned long long (&part)[VW],
                                                       unsigned long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned long long incl = warp_incl_scan_u64(v);
  __syncthreads();                     // the parts of an earlier scan have been read
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  unsigned long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < VW; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  return before + incl - v;
}

__global__ void __cluster_dims__(NSHARD, 1, 1) __launch_bounds__(VT)
verify_draw_kernel(const DrawParams P) {
  __shared__ unsigned long long part[VW];
  __shared__ unsigned long long round_mass[ROUNDS];
  __shared__ unsigned long long shard_mass[2][NSHARD];
  __shared__ uint16_t list[SHARD_CHUNKS];
  const int tid = threadIdx.x, lane = tid & 31;
  const int r = static_cast<int>(cluster_rank());
  const int64_t b = blockIdx.x / NSHARD;
  const int n = P.ver.n;
  // what the pass does not write is here before it is done
  const int num_in = P.ver.num ? P.ver.num[b] : n;
  const uint32_t accept0 = lane < n ? P.accept[b * n + lane] : 0u, draw = P.draw[b];
  const float tau = P.tau_arr ? P.tau_arr[b] : P.tau_s;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const VerifyMsg* rec = P.ver.rec + b * (n + 1);
  const VerifyMsg* recq = P.draft ? P.ver.rec_draft + b * n : nullptr;

  // ---- the first place that is not an accepted draft (every warp, the same)
  bool bad = num_in < 0 || num_in > n;
  const int num = bad ? 0 : num_in;
  int a = num;
  for (int i0 = 0; i0 < num; i0 += 32) {
    const int i = i0 + lane;
    bool go_on = true;
    if (i < num) {
      const float u = static_cast<float>((i0 == 0 ? accept0 : P.accept[b * n + i]) >> 8) * 5.9604644775390625e-8f;
      const bool ok = (rec[i].flags & VER_OK) && (!recq || (recq[i].flags & VER_OK));
      const float q = recq ? recq[i].p_t : 1.0f;
      go_on = ok && __fmul_rn(u, q) < rec[i].p_t;
    }
    const unsigned stop = __ballot_sync(0xffffffffu, !go_on);
    if (stop) {
      a = i0 + __ffs(stop) - 1;
      break;
    }
  }
  const bool residual = a < num;
  if (!bad) bad = !(rec[a].flags & VER_OK) || (residual && recq && !(recq[a].flags & VER_OK));
  if (r == 0) {
    for (int i = tid; i <= n; i += VT) {
      const int64_t at = b * (n + 1) + i;
      if (i < a) {
        P.out_token[at] = P.ver.token[b * n + i];
        if (P.out_restr) P.out_restr[at] = rec[i].restr_t;
        if (P.out_full) P.out_full[at] = rec[i].full_t;
      } else if (i > a || bad) {
        P.out_token[at] = -1;
        const float v = i == a ? __int_as_float(0x7fc00000) : 0.0f;
        if (P.out_restr) P.out_restr[at] = v;
        if (P.out_full) P.out_full[at] = v;
      }
    }
    if (tid == 0) {
      P.out_accepted[b] = a;
      if (bad && P.err) atomicAdd(P.err, 1);
    }
  }
  if (bad) return;                     // the whole cluster
  const VerifyMsg rr = rec[a];
  const int64_t slot = b * (n + 1) + a;
  if (rr.flags & VER_GREEDY) {
    if (r == 0 && tid == 0) {
      P.out_token[slot] = rr.min_key;
      if (P.out_restr) P.out_restr[slot] = 0.0f;
      if (P.out_full) P.out_full[slot] = 0.0f;
    }
    return;
  }
  cluster_arrive_relaxed();            // met before the first store into a peer: every CTA is running

  // ---- the chunks that hold the support, in column order: those that the pass marked,
  // or all of the shard's
  const uint4* rowp = reinterpret_cast<const uint4*>(P.logits + slot * P.stride) + r * SHARD_CHUNKS;
  const bool with_y = residual && recq;
  const uint4* rowq = with_y ? reinterpret_cast<const uint4*>(P.draft + (b * n + a) * P.draft_stride) + r * SHARD_CHUNKS
                             : nullptr;
  int chunks = r == NSHARD - 1 ? LAST_CHUNKS : SHARD_CHUNKS;
  const bool marked = (rr.flags & SAMP_BITS) != 0;
  if (marked) {
    uint32_t word = tid < SAMP_BITWORDS ? P.bits[(slot * NSHARD + r) * SAMP_BITWORDS + tid] : 0u;
    unsigned long long total;
    int at = static_cast<int>(cta_scan(static_cast<unsigned long long>(__popc(word)), part, total));
    chunks = static_cast<int>(total);
    for (; word; word &= word - 1) list[at++] = static_cast<uint16_t>(tid * 32 + __ffs(word) - 1);
  }
  for (int i = tid; i < ROUNDS; i += VT) round_mass[i] = 0ull;
  __syncthreads();
  Masses m{};
  m.M = rr.M;
  m.c = __fdiv_rn(LOG2E, tau);
  const float vmin = rr.min_key <= KEY_NEG_INF ? -INFINITY : key_value(rr.min_key);
  m.vmin2 = __floats2bfloat162_rn(vmin, vmin);
  m.skip = residual && !recq ? P.ver.token[b * n + a] : -1;
  m.q_one = -1;
  if (with_y) {
    const VerifyMsg rq = recq[a];
    m.with_q = true;
    if (rq.flags & VER_GREEDY) {
      m.q_one = rq.min_key;
      m.q_one_mass = rr.zs * FX_SCALE;
    } else {
      const float tq = P.ver.tau_arr ? P.ver.tau_arr[b] : P.ver.tau_s;
      m.Mq = rq.M;
      m.cq = __fdiv_rn(LOG2E, tq);
      m.ratio = __fdiv_rn(rr.zs, rq.zs) * FX_SCALE;
      const float vq = rq.min_key <= KEY_NEG_INF ? -INFINITY : key_value(rq.min_key);
      m.vminq2 = __floats2bfloat162_rn(vq, vq);
    }
  }

  // ---- masses, a chunk to a thread in each round; where a residual has none anywhere,
  // once more for p itself
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  unsigned long long prefix = 0, total = 0, mine = 0;
  for (int turn = 0; turn < 2; ++turn) {
    unsigned long long sum = 0;
#pragma unroll 4
    for (int c = tid; c < chunks; c += VT) {
      const int g = marked ? list[c] : c;
      const uint4 x = __ldg(rowp + g), y = m.with_q ? __ldg(rowq + g) : none;
      unsigned long long e[8];
      const unsigned long long v = chunk_masses(m, x, y, r * SW + g * 8, e);
      if (v) atomicAdd(&round_mass[c / VT], v);            // integers: any order
      sum += v;
    }
    cta_scan(sum, part, mine);
    if (turn == 0) cluster_wait();
    if (tid < NSHARD) {
      const uint32_t dst = map_rank(smem_addr(&shard_mass[turn][r]), tid);
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(dst), "l"(mine) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    cluster_wait();
    prefix = total = 0;
#pragma unroll
    for (int q = 0; q < NSHARD; ++q) {
      if (q < r) prefix += shard_mass[turn][q];
      total += shard_mass[turn][q];
    }
    if (total != 0) break;             // the same in every CTA
    m.with_q = false;
    m.skip = -1;
  }
  if (total == 0) {                    // a row of zero mass: not a resolved row's case
    if (r == 0 && tid == 0) P.out_token[slot] = -1;
    return;
  }

  // ---- the shard, the round, the chunk and the column that hold the draw
  const unsigned long long t = scale_draw(draw, total);
  if (t < prefix || t - prefix >= mine) return;      // another CTA's
  unsigned long long left = t - prefix;
  int round = 0;
  while (left >= round_mass[round]) left -= round_mass[round++];
  const int c = round * VT + tid;
  const bool here = c < chunks;
  const int g = here ? (marked ? list[c] : c) : 0;
  unsigned long long e[8], mass = 0, all;
  uint4 x = none;
  if (here) {
    x = __ldg(rowp + g);
    mass = chunk_masses(m, x, m.with_q ? __ldg(rowq + g) : none, r * SW + g * 8, e);
  }
  const unsigned long long ex = cta_scan(mass, part, all);
  if (!here || left < ex || left - ex >= mass) return;
  left -= ex;
  const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
  int jstar = -1;
  float xa = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (jstar < 0) {
      if (left < e[j]) {
        jstar = j;
        xa = (j & 1) ? bf16_hi(w4[j >> 1]) : bf16_lo(w4[j >> 1]);
      } else {
        left -= e[j];
      }
    }
  }
  const float d = __fdiv_rn(xa - rr.M, tau);
  const float full = d - logf(rr.Z);
  P.out_token[slot] = r * SW + g * 8 + jstar;
  if (P.out_full) P.out_full[slot] = full;
  if (P.out_restr) P.out_restr[slot] = (rr.flags & SAMP_SEL) ? d - logf(rr.zs) : full;
}

}  // namespace rlk

using namespace rlk;

extern "C" rlk_status rlk_verify_drafts(const rlk_verify_args* a, int32_t* out_token, int32_t* out_accepted,
                                        float* out_restr, float* out_full, void* workspace, void* stream) {
  if (!a) return fail(RLK_EINVAL, "args is NULL");
  if (a->B < 0) return fail(RLK_EINVAL, "B = %lld < 0", (long long)a->B);
  if (a->n < 0 || a->n > 1024) return fail(RLK_EINVAL, "n = %d must be in 0..1024", a->n);
  if (a->B >= (int64_t(1) << 28) || a->B * (2 * int64_t(a->n) + 1) >= (int64_t(1) << 28))
    return fail(RLK_EINVAL, "B * (2 n + 1) must be below 2^28");
  rlk_logp_args t{};
  t.logits = a->logits;
  t.T = a->B * (a->n + 1);
  t.row_stride = a->row_stride;
  t.vocab_real = a->vocab_real;
  t.vocab_padded = a->vocab_padded;
  t.temperature = a->temperature;
  t.temperature_scalar = a->temperature_scalar;
  t.top_p = a->top_p;
  t.top_p_scalar = a->top_p_scalar;
  t.top_k = a->top_k;
  t.top_k_scalar = a->top_k_scalar;
  t.err_count = a->err_count;
  rlk_status s = check_args(&t, true, false);
  if (s != RLK_OK || a->B == 0) return s;
  const bool drafts = a->n > 0 && a->draft_logits;
  if (drafts) {
    if ((s = check_logits(a->draft_logits, a->B * a->n, a->draft_row_stride, "draft_logits")) != RLK_OK) return s;
    if ((s = check_tau(a->draft_temperature, a->draft_temperature_scalar)) != RLK_OK) return s;
    if ((s = check_top_p(a->draft_top_p, a->draft_top_p_scalar)) != RLK_OK) return s;
    if ((s = check_top_k(a->draft_top_k, a->draft_top_k_scalar)) != RLK_OK) return s;
  }
  if ((s = check_out(a->draft_token, "draft_token", a->n > 0)) != RLK_OK) return s;
  if ((s = check_out(a->accept_uniform, "accept_uniform", a->n > 0)) != RLK_OK) return s;
  if ((s = check_out(a->draw_uniform, "draw_uniform", true)) != RLK_OK) return s;
  if ((s = check_out(a->num_drafts, "num_drafts", false)) != RLK_OK) return s;
  if ((s = check_out(out_token, "out_token", true)) != RLK_OK) return s;
  if ((s = check_out(out_accepted, "out_accepted", true)) != RLK_OK) return s;
  if ((s = check_out(out_restr, "out_restr", false)) != RLK_OK) return s;
  if ((s = check_out(out_full, "out_full", false)) != RLK_OK) return s;
  if (!workspace) return fail(RLK_EINVAL, "workspace is NULL");
  if (!aligned(workspace, 16)) return fail(RLK_EALIGN, "workspace is not 16-byte aligned");

  DrawParams P{};
  P.ver.B = a->B;
  P.ver.n = a->n;
  P.ver.token = a->draft_token;
  P.ver.num = a->num_drafts;
  P.ver.tau_arr = a->draft_temperature;
  P.ver.p_arr = a->draft_top_p;
  P.ver.k_arr = a->draft_top_k;
  P.ver.tau_s = a->draft_temperature_scalar;
  P.ver.p_s = a->draft_top_p_scalar;
  P.ver.k_s = a->draft_top_k_scalar;
  P.ver.rec = static_cast<VerifyMsg*>(workspace);
  P.ver.rec_draft = P.ver.rec + a->B * (a->n + 1);
  uint32_t* bits = reinterpret_cast<uint32_t*>(P.ver.rec_draft + a->B * a->n);
  if ((s = verify_pass(&t, drafts ? a->draft_logits : nullptr, a->draft_row_stride, P.ver, bits, stream)) != RLK_OK)
    return s;
  P.logits = static_cast<const uint16_t*>(a->logits);
  P.stride = a->row_stride;
  P.draft = drafts ? static_cast<const uint16_t*>(a->draft_logits) : nullptr;
  P.draft_stride = a->draft_row_stride;
  P.tau_arr = a->temperature;
  P.tau_s = a->temperature_scalar;
  P.bits = bits;
  P.accept = a->accept_uniform;
  P.draw = a->draw_uniform;
  P.out_token = out_token;
  P.out_accepted = out_accepted;
  P.out_restr = out_restr;
  P.out_full = out_full;
  P.err = a->err_count;
  // launched while the pass's last rows are at work, and waits for them
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a->B * NSHARD));
  cfg.blockDim = dim3(VT);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_draw_kernel, P);
  if (e != cudaSuccess) return fail(RLK_ECUDA, "kernel launch: %s", cudaGetErrorString(e));
  return RLK_OK;
}
