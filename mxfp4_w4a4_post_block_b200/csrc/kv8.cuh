// Shared by the kernels of the 8-bit paged cache (kv8_append.cu, attn_kv8.cu).
//
// The cache: pages of `page` tokens.  K and V each hold [num_pages][kv_heads][page][head_dim] E4M3
// bytes and one E8M0 scale byte per (page, kv head), value = code * 2^(byte - 127).  Page p of
// sequence b is page_table[b * max_pages + p]; a page id outside [0, num_pages) names no page.
#pragma once

#include <cstdint>

namespace batq {

// 2^(byte - 127) as fp32 (byte 0: the subnormal 2^-127; byte 255: NaN).
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  const uint32_t bits = byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23;
  return __uint_as_float(bits);
}

// Sequence b of a ragged batch: its rows [begin, begin + count) of the `rows` new tokens (or
// queries), and its tokens in the cache.  cu == nullptr: one row per sequence.  What the arrays
// must not hold (a range outside [0, rows], a negative count) gives a sequence without rows.
struct SeqRows {
  int begin, count, len;
};
__device__ __forceinline__ SeqRows seq_rows(const int* cu, const int* lens, int b, int rows, int max_len) {
  SeqRows s;
  s.begin = cu ? cu[b] : b;
  const int end = cu ? cu[b + 1] : b + 1;
  s.count = (s.begin < 0 || end > rows || end < s.begin) ? 0 : end - s.begin;
  s.len = min(lens[b], max_len);
  return s;
}

}  // namespace batq
