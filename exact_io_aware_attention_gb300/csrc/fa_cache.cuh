// Layout of the 4-bit K/V cache (fa_cache in include/fa.h), shared by the
// kernels that write it, read it back and attend over it.
//
// The pool is [num_pages][heads][page_size / 16] cells. A cell holds 16
// consecutive tokens of one head and is contiguous (20 d bytes), so one bulk
// copy brings a cell, or a run of cells of a page, into shared memory:
//
//   offset 0      K codes   16 rows of d/2 bytes
//          8 d    V codes   8 rows of d bytes, for pairs of tokens
//          16 d   K groups  16 rows of d/32 lo, d/32 s
//          18 d   V groups  s, then lo: 8 rows of d/32 words, for pairs of tokens
//
// Within a cell the order of rows and nibbles is that of the registers of the
// 16x8x16 matrix product the attention kernel runs on a cell, so a thread
// reads its operands as whole words without bank conflicts and one AND turns
// a word into two f16 operands: 4 bits in the low mantissa bits of an f16 are
// the subnormal u * 2^-24 (u * 2^-20 one nibble up), exact in the product.
//
//   token j of a cell is matrix row cell_slot(j); K codes and groups are in
//   slot order;
//   K: channel c = 32 g + 8 t + i is nibble i of word (t, g); channels i and
//   i + 4, in the two halves, are k-neighbours of the product;
//   V: channel c = 32 g + 4 r + i of tokens t + 8 y and t + 8 y + 4, which are
//   k-neighbours, is nibble i of the halves of word (y, t, r, g).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_internal.h"

namespace fa {

constexpr int kCellTokens = 16;

__host__ __device__ constexpr int cell_bytes(int d) { return 20 * d; }
__host__ __device__ constexpr int cell_v_codes(int d) { return 8 * d; }
__host__ __device__ constexpr int cell_k_groups(int d) { return 16 * d; }
__host__ __device__ constexpr int cell_v_groups(int d) { return 18 * d; }

// Matrix row of token j, and the token of matrix row s: the tokens of the
// four thread columns t of a V operand (slots 2t, 2t+1, 2t+8, 2t+9) are t,
// t + 4, t + 8 and t + 12, which lie in different banks.
__host__ __device__ constexpr int cell_slot(int j) {
  return ((j & 3) << 1) | ((j >> 2) & 1) | (j & 8);
}
__host__ __device__ constexpr int cell_token(int s) {
  return ((s >> 1) & 3) | ((s & 1) << 2) | (s & 8);
}

// Byte offset of K's code word (slot, t, g) in a cell: 8 channels. For d = 256
// the two 64-byte halves of a row (groups 0-3, 4-7) swap places in odd slots.
template <int D>
__host__ __device__ constexpr int k_word(int slot, int t, int g) {
  return D == 256 ? slot * 128 + (((g >> 2) ^ (slot & 1)) << 6) + t * 16 + (g & 3) * 4
                  : slot * (D / 2) + (t * (D / 32) + g) * 4;
}

// Byte offset of V's code word (y, t, r, g): 4 channels of tokens t + 8 y and
// t + 8 y + 4. Thread row r's words of a pair lie together (d = 256: four and
// four); their order depends on t so that the four threads t of a load lie in
// different banks (d = 96: they do as it is).
template <int D>
__host__ __device__ constexpr int v_word(int y, int t, int r, int g) {
  return cell_v_codes(D) +
         (D == 256   ? (g >> 2) * 1024 + (4 * y + t) * 128 + (r ^ (2 * t)) * 16 + (g & 3) * 4
          : D == 128 ? (4 * y + t) * 128 + (r ^ (2 * t)) * 16 + g * 4
          : D == 96  ? (4 * y + t) * 96 + (r * 3 + g) * 4
                     : (4 * y + t) * 64 + (r ^ (4 * (t >> 1))) * 8 + g * 4);
}
template <int D>
__host__ __device__ constexpr int v_half(int j, int r, int g) {
  return v_word<D>(j >> 3, j & 3, r, g) + ((j >> 2) & 1) * 2;
}

// Byte offsets of the 16-bit s and lo of K's group (slot, g): a row holds the
// lo of its groups, then their s, so that two groups' lo are a word.
template <int D>
__host__ __device__ constexpr int k_lo(int slot, int g) {
  return cell_k_groups(D) + slot * (D / 8) + g * 2;
}
template <int D>
__host__ __device__ constexpr int k_s(int slot, int g) {
  return k_lo<D>(slot, g) + D / 16;
}
// Byte offsets of V's words (y, t, g) of s and of lo: tokens t + 8 y (low half)
// and t + 8 y + 4.
template <int D>
__host__ __device__ constexpr int v_s(int y, int t, int g) {
  return cell_v_groups(D) + ((4 * y + t) * (D / 32) + g) * 4;
}
template <int D>
__host__ __device__ constexpr int v_lo(int y, int t, int g) {
  return v_s<D>(y, t, g) + D;
}

// Division of 0 <= x < 2^31 by a number known at the launch (d >= 1), as a
// product: mul = ceil(2^(31 + shift) / d) with 2^shift >= d exceeds the
// quotient 2^(31 + shift) / d by less than 1, which x / 2^31 < 1 of turns into
// less than the distance of x / d from the next whole number, 1 / d.
struct FastDiv {
  uint32_t mul;
  int shift, d;
  FastDiv() = default;
  __host__ explicit FastDiv(int by) : mul(0), shift(0), d(by) {
    while ((1ll << shift) < by) ++shift;
    mul = (uint32_t)((((1ull << 31) << shift) + by - 1) / by);
  }
  __host__ __device__ __forceinline__ int div(int x) const {
    return (int)(((uint64_t)(uint32_t)x * mul) >> (31 + shift));
  }
};

// The pool and the page table of a call. Cell c of sequence b and head h (its
// tokens 16 c .. 16 c + 15) is cell_ptr(page, h, c % page_cells), page =
// table[b * table_stride + c / page_cells].
struct CachePool {
  uint8_t *data;
  const int32_t *table;
  long long table_stride;
  int num_pages, heads, page_cells;   // page_cells = page_size / 16
  int table_cells;                    // cells a row of the table covers
  int d, f16;
  FastDiv by_page_cells;
  __device__ __forceinline__ bool page_ok(int page) const {
    return (unsigned)page < (unsigned)num_pages;
  }
  template <int D>
  __device__ __forceinline__ uint8_t *cell_ptr(int page, int h, int in_page) const {
    return data + (((size_t)page * heads + h) * page_cells + in_page) * (size_t)cell_bytes(D);
  }
};

// Writing n rows of each (b, head) into the cache, or reading them back: row i
// of sequence b is token start[b] + i, for i < counts[b] (n without counts).
struct CacheRowsParams {
  CachePool pool;
  const int32_t *start, *counts;
  void *k, *v;                        // 16-bit rows, strides sk / sv
  RowStrides sk, sv;
  int B, n;
  unsigned int *status;
};

// Attention over the cache. Query row (b, hq, i), i < counts[b] (nq without
// counts), is token lengths[b] - counts[b] + i of sequence b.
struct CacheFwdParams {
  CachePool pool;
  const int32_t *lengths, *counts;
  const void *q;                      // 16-bit rows, strides sq
  RowStrides sq;
  void *o;                            // 16-bit or fp32 rows, strides so
  RowStrides so;
  float *lse;                         // [B][Hq][nq]
  int o_f32;
  int B, hq, group, nq, causal;       // group = hq / heads of the pool
  FastDiv by_group, by_row_blocks;    // (row blocks: of the chosen row tiles)
  float scale_log2;
  float *part;                        // scratch: [ctas][2][rows][d] partial outputs,
  float *part_lse;                    // [ctas][2][rows] their log2-sum-exp,
  int4 *chain;                        // [ctas] where a segment's parts lie
  int block_rows;                     // query rows of a CTA
  int whole;                          // no segment is split: no scratch, no merge
  int ctas;                           // CTAs of the attention kernel
  unsigned int *status;
  uint32_t debug_flags;
  uint64_t wait_limit_ns;
};

cudaError_t launch_cache_write(const CacheRowsParams &p, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheRowsParams &p, cudaStream_t stream);
cudaError_t launch_cache_forward(const CacheFwdParams &p, cudaStream_t stream);

// The attention with 128 or 256 query rows a CTA on tcgen05 (fa_cache_fwd_tc.cu);
// the merge of its parts is launched by launch_cache_forward.
cudaError_t launch_cache_forward_tc(const CacheFwdParams &p, cudaStream_t stream);

// CTAs that one SM holds (its registers and shared memory allow).
constexpr int cache_forward_ctas_per_sm(int d, int block_rows) {
  return block_rows >= 128 ? 1
         : block_rows == 8 ? (d == 256 ? 2 : d == 128 ? 3 : 4)
                           : (d == 64 ? 3 : 2);
}

// Whether sequences of at most `tokens` tokens are not split between CTAs.
constexpr bool cache_forward_whole(long long tokens) { return tokens <= 1024; }

// Query rows (new tokens times query heads of one K/V head) that one CTA
// holds: 8 or 16 in the kernel for few rows, whose product has 8 columns a
// tile (d = 256: 8, two tiles' outputs would not fit the registers), 128 or 256
// (d = 256: 128) in the one for many.
//
// Up to 64 rows few: the other kernel needs 8 to 15 us more before and after its
// tiles, which only much work outweighs. Measured (few / many, whole calls), 4
// sequences of 6000 to 16000 keys on 2 K/V heads, 64 rows, bf16: 31 / 32 us at
// d = 64, 34 / 40 us at d = 128, 52 / 58 us at d = 256; one of 3000 keys on 4 heads
// 17 / 21, 18 / 24 and 21 / 32 us; 16 of 5000 to 8192 keys 44 / 38, 54 / 48 and
// 97 / 81 us. With 128 rows, 4 sequences on 2 heads: 92 / 52 us at d = 256.
//
// Where a segment stays whole, the few-row kernel is done sooner as long as all
// its segments run at once (d = 256: in two turns), and 128 rows sooner than 256
// as long as they do. Measured, up to 1000 keys, d = 128 (few / many): 8 heads
// of 512 rows, 256 segments, 23 / 36 us; 64 heads of 128 rows, 512 segments,
// 38 / 28 us; 12 heads of 1000 rows (128 / 256 rows a CTA) 27 / 36 us.
constexpr int cache_forward_block_rows(int d, long long rows, bool whole, double heads, int sms) {
  const int few = d == 256 || rows <= 8 ? 8 : 16;
  if (rows <= 64) return few;
  if (whole && heads * ((rows + few - 1) / few) <=
                   (d == 256 ? 2.0 : 1.0) * sms * cache_forward_ctas_per_sm(d, few))
    return few;
  return d == 256 || rows <= 128 || (whole && heads * ((rows + 127) / 128) <= sms) ? 128 : 256;
}

}  // namespace fa
