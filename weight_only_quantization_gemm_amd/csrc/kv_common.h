// The key-value cache's format, shared by the kernels that write, read and
// attend over it (and, being plain arithmetic, checked on the host by tests).
//
// One half (keys or values) of a cache of `pages` pages of P = 2^ps slots for
// H heads of D channels:
//   codes   uint32 [pages][H][P][D * bits / 32]
//   params  fp16   [pages][H][P][2]               scale, zero point (a whole number)
// so the slots of one head in one page are contiguous: 16 slots of 4-bit codes
// at D = 128 are 1 KB, one wave instruction of 16-byte loads.
#pragma once

#include <stdint.h>

#ifndef __host__
#define __host__
#define __device__
#endif

namespace awq {

struct KvShape {
  int64_t pages;
  int heads, ps;  // ps = log2 of the slots per page
};

// Whether `slot` (page * P + place in the page) is one of the cache's.
__host__ __device__ inline bool kv_slot_ok(const KvShape& s, int64_t slot) {
  return slot >= 0 && slot < (s.pages << s.ps);
}

// Row of (slot, head) among the pages * H * P rows of a half.
__host__ __device__ inline int64_t kv_row(const KvShape& s, int64_t slot, int head) {
  return ((((slot >> s.ps) * s.heads) + head) << s.ps) + (slot & ((int64_t(1) << s.ps) - 1));
}

// A page table's entry as a page of the cache, or -1 where it names none.
__host__ __device__ inline int kv_page(const KvShape& s, int32_t entry) {
  return entry >= 0 && entry < s.pages ? entry : -1;
}

// Row of (token t, head) where t is the first of 16 tokens that share the page
// `page` (t and a page's slots are multiples of 16).  For a page that is none
// the row is one of page 0: it may be read, and its tokens are masked.
__host__ __device__ inline int64_t kv_tile_row(const KvShape& s, int page, int64_t t, int head) {
  const int64_t place = t & ((int64_t(1) << s.ps) - 1);
  return kv_row(s, ((int64_t)(page < 0 ? 0 : page) << s.ps) + place, head);
}

// Tokens a sequence attends over: its length, within what the page table and
// the caller's bound hold.
__host__ __device__ inline int64_t kv_length(const KvShape& s, int32_t length, int64_t width, int64_t max_len) {
  int64_t n = length < 0 ? 0 : length;
  n = n < max_len ? n : max_len;
  return n < (width << s.ps) ? n : width << s.ps;
}

// Attention's split: sequences are counted in units of kKvUnit tokens (an empty one as
// one unit, whose block stores its zeros) and cut into pieces of at most 2^shift units,
// the pieces of a sequence as even as whole units allow; pieces are numbered sequence
// by sequence.
constexpr int kKvUnit = 128;

__host__ __device__ inline int kv_units(int len) { return len > 0 ? (len + kKvUnit - 1) / kKvUnit : 1; }

// log2 of the units of a piece: up to 4 units while all heads' pieces are more than about
// 512, and on while they are more than about `most`.
__host__ __device__ inline int kv_piece_shift(int64_t total, int heads, int most) {
  int shift = 0;
  while (shift < 2 && total * heads > (512 << shift)) ++shift;
  while (shift >= 2 && shift < 18 && total * heads > ((int64_t)most << shift)) ++shift;  // 2^18 units: any sequence
  return shift;
}
__host__ __device__ inline int kv_pieces(int units, int shift) { return (units + (1 << shift) - 1) >> shift; }

// The most pieces of a head: B sequences of at most max_len tokens.
__host__ __device__ inline int64_t kv_most_pieces(int64_t B, int max_len, int heads, int most) {
  const int64_t units = B * kv_units(max_len), pieces = (most > 512 ? most : 512) / heads + 1 + B;
  return pieces < units ? pieces : units;
}

}  // namespace awq
