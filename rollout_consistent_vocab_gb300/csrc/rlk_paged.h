// rlk_paged.h -- the paged key-value cache as the kernels see it, and what the
// translation units that work on it share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "rlk_rollout.h"

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

// 2^32 / page_size, rounded up (page_size 1: 2^32 - 1), and by it the page of token t in its
// sequence's list, with its place in the page.
inline uint32_t page_magic(int page_size) {
  return static_cast<uint32_t>(page_size == 1 ? 0xFFFFFFFFull : ((1ull << 32) + page_size - 1) / page_size);
}
__device__ __forceinline__ uint32_t page_of(const PagedParams& P, uint32_t magic, int t, int& place) {
  uint32_t n = __umulhi(static_cast<uint32_t>(t), magic);
  place = static_cast<int>(static_cast<uint32_t>(t) - n * static_cast<uint32_t>(P.page_size));
  if (place < 0) place += P.page_size, --n;                // the quotient is one off at most
  if (place >= P.page_size) place -= P.page_size, ++n;
  return n;
}
// Tokens of a copy: the largest power of 2, up to `most`, that divides the page.
inline int box_of(int page_size, int most) {
  int box = 1;
  while (box < most && page_size % (2 * box) == 0) box *= 2;
  return box;
}
// Whether the tensor maps' second place is the head, not the token.
inline bool heads_first(const rlk_kv_cache* c) {
  return c->kv_heads > 1 && (c->page_size == 1 || c->head_stride < c->token_stride);
}
// The cache's keys or values as a tensor of (element, token of the page, head, page),
// the middle two in the order of their strides; a copy takes 64 elements of
// `box` tokens of a head; with panels = 2 all 128 elements, the second 64 of every token
// behind the first 64 (a fifth place).
rlk_status map_cache(CUtensorMap* map, const PagedParams& c, const void* base, int box, bool head_first, int panels, int D, bool bf16);

// Attention over a shared prefix is taken in parts: of the shared tokens, that a group's
// queries go over together, and of each sequence's other ones.  How the shared ones are cut goes by
// their number alone, and how the others are by nothing but how far behind them each is: a token's
// result does not depend on its batch, nor on how many new tokens come with it.
//
// Tokens of a part of the shared ones: the fewer the longer, since a part costs as much as three tiles of
// 128 tokens, and a write and a read of 128 tokens' size for 128 rows; but as many as there are SMs, for a
// group or two (1 x 64 samples of 8190 tokens: parts of 1024 58 us, of 2048 71; 2 x 32 of 131071 tokens:
// parts of 1024 232 us, of 2048 213).
constexpr int PIECES_1024 = 1024, PIECES_2048 = 16384;     // shared tokens from which on parts are so long
__host__ __device__ __forceinline__ int piece_tokens(int shared) {
  return shared < PIECES_1024 ? 512 : shared < PIECES_2048 ? 1024 : 2048;
}
__host__ __device__ __forceinline__ int pieces_of(int shared) {
  const int t = piece_tokens(shared);
  return shared / t + (shared % t != 0);
}
// The parts of a sequence's other tokens: 64 of 256 tokens, then 32 to each doubling (of 512 from token 16384 on,
// of 1024 from 32768 on).  (Lengths that went by the number of all tokens made a token's bits depend on the
// drafts behind it.)  With half as many of twice the length from token 8192 on, 2 sequences of 500,000 tokens took
// 992 us for 710, 1 of 16,000 53 for 42; 64 of 16,000 672 for 684, whose results are half as many.
constexpr int TAIL_PART = 256;
__host__ __device__ __forceinline__ int tail_level(int token) {        // parts are TAIL_PART << level tokens
  int level = 0;
  while (token >> (13 + level) > 1) ++level;
  return level;
}
__host__ __device__ __forceinline__ int tail_part_of(int token) {
  const int level = tail_level(token);
  return (token >> (8 + level)) + 32 * level;
}
__host__ __device__ __forceinline__ int tail_parts(int tokens) { return tokens > 0 ? tail_part_of(tokens - 1) + 1 : 0; }
__host__ __device__ __forceinline__ int tail_part_level(int part) { return part < 64 ? 0 : part / 32 - 1; }
__host__ __device__ __forceinline__ int tail_part_from(int part) {
  const int level = tail_part_level(part);
  return (part - 32 * level) << (8 + level);
}
__host__ __device__ __forceinline__ int tail_part_tokens(int part) { return TAIL_PART << tail_part_level(part); }
// The parts of one length: the first of them, the token that it begins with, and the tokens of all.
__host__ __device__ __forceinline__ int tail_level_part(int level) { return level == 0 ? 0 : 32 + 32 * level; }
__host__ __device__ __forceinline__ int tail_level_from(int level) { return level == 0 ? 0 : 8192 << level; }
__host__ __device__ __forceinline__ int tail_level_tokens(int level) { return level == 0 ? 16384 : 8192 << level; }
// Their query rows go in tiles of 8 nt: as few as hold the rows in 24 each, then as narrow as they can be.
struct TailTiles { int tiles, nt; };
inline TailTiles tail_tiles(int rows) {
  const int tiles = (rows + 23) / 24;
  return {tiles, (rows + 8 * tiles - 1) / (8 * tiles)};
}
// What both kernels and the join go by.
struct PrefixParts {
  PagedParams c;
  const void* q;
  void* out;
  rlk_bth_strides qs, os;       // elements
  int64_t B;
  int q_heads, group;           // group: query heads of a kv head
  int rows;                     // n * group: of a sequence and kv head
  float c2;                     // |scale| * log2(e)
  uint32_t q_sign;              // 0x80008000: the queries change sign (scale < 0)
  uint32_t page_magic;
  bool head_first;              // the tensor maps' second place is the head, not the token
  float* lse;
  const int32_t* first;         // [B] tokens of the sequence that are taken as shared, a multiple of 32; -1: rejected
  // By the length of their parts, the level: steps of 16 other tokens (of a kv head) before each sequence
  const uint32_t* tail_base;    // [levels][B + 1]
  uint32_t* taken;              // chunks of those steps that warps have taken; then the highest level that there is, and all steps
  float2* piece_ml;             // [B][kv_heads][pieces][rows]: maximum (base 2), sum
  float* piece_o;               // ... and the weighted sum of values [B][kv_heads][pieces][head_dim / 8][rows][8]: a warp with a
                                // thread to a row has few lines to write at a time
  int pieces;                   // at most, of a sequence
  float2* tail_ml;              // the same of the tails
  float* tail_o;
  int tails;
};

// What is written of a part with a page that is not there: a sum that stays NaN, and a maximum that
// no other part has.
__device__ __forceinline__ float2 bad_part() { return make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000)); }

// The sequences' other tokens, and the join of all parts.  What can be refused is looked at before anything is
// launched (`prepare`); the launches follow the shared tokens' kernel, or where there is none (`alone`) the plan's.
struct CacheMaps { CUtensorMap k, v; };
enum class Tails { prepare, beside, alone };
rlk_status attend_tails(const PrefixParts& parts, CacheMaps& maps, int head_dim, bool bf16, Tails what, cudaStream_t stream);

rlk_status check_cache(const rlk_kv_cache* c);
rlk_status check_bth(const void* p, const rlk_bth_strides* s, const char* what);
PagedParams paged_params(const rlk_kv_cache* c);

}  // namespace rlk
