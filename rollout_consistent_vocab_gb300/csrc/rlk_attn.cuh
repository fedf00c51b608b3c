// rlk_attn.cuh -- what the attention kernels share: the cache's dtypes on mma.sync, the
// arithmetic of a softmax that is taken part by part, fragments from shared memory.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "rlk_device.cuh"

namespace rlk {

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
  // whether both parts of a weight are above 0 (NaN's are not): a value that is not finite comes through as itself
  static __device__ __forceinline__ bool counts(float w) { return w > 0.0f; }
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
  static __device__ __forceinline__ bool counts(float w) { return w >= TINY; }
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
// Waits for a phase of a barrier, at most TIMEOUT_NS twice over.
__device__ __forceinline__ bool mbar_wait_phase(uint32_t bar, uint32_t parity) {
  if (mbar_try(bar, parity)) return true;
  const unsigned long long t0 = global_timer();
  while (!mbar_try(bar, parity))
    if (global_timer() - t0 > 2 * TIMEOUT_NS) return false;
  return true;
}
// Where the result of a row goes: out and lse, from the weighted sum o (this
// lane's share), the sum l and the maximum m (base 2).
template <class T>
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + (log2f(l) - Elem<T>::OFF)) * 0.6931471805599453f;
}

// A row's parts, joined one after the other; a warp's, 1 / 32 of the elements to a lane.
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

}  // namespace rlk
