// The 4-bit key/value cache as the kernels see it: addresses of a record and the checked view of a
// sequence's lengths and pages, which live in device memory and are never trusted.
//
// A record holds 16 tokens of one head (D = 2 dim stacked real and imaginary entries):
//   keys    8 D bytes: the 16 x D tile of q4_common.cuh, D / 64 times 512 bytes; row = token
//   values  8 D bytes: the same vectors turned round for O^T = V^T P^T: word 2 (q % 2) + h of lane
//           4 g + t in the 512 bytes of q / 2 holds entries 32 q + 4 g .. + 3 of tokens 2 t + 8 h (low
//           half, entry i in bits 4 i) and 2 t + 8 h + 1 (high half): key pairs adjacent for the matrix
//           instruction, and a token's values are whole half words, so that appending reads nothing
//   key parameters, value parameters  128 bytes each: per token bf16 {s_re, m_re, s_im, m_im}
#pragma once

#include "q4_common.cuh"

namespace ifq {

struct Kv4Arg {
  uint8_t* records;
  const int32_t* page_table;
  const int32_t* kv_lens;
  const int32_t* new_offsets;
  int64_t pages, table_cols, rows;
  int64_t record_bytes;
  int32_t page_tiles;  // records of a page and head
  int32_t kv_heads, B, n_new;
};

inline Kv4Arg kv4_arg(const ifq_kv4_cache& c) {
  Kv4Arg a;
  a.records = c.records;
  a.page_table = c.page_table;
  a.kv_lens = c.kv_lens;
  a.new_offsets = c.new_offsets;
  a.pages = c.pages;
  a.table_cols = c.table_cols;
  a.rows = c.rows;
  a.record_bytes = 32 * (int64_t)c.dim + 256;
  a.page_tiles = c.page_tokens / 16;
  a.kv_heads = c.kv_heads;
  a.B = c.B;
  a.n_new = c.n_new;
  return a;
}

// A sequence of the call: its new tokens are rows row0 .. row0 + n_new - 1 at positions len - n_new ..;
// ok is false where the device-side numbers are outside their ranges (then len = 0, and n_new = 0 too
// if the rows themselves are not usable).
struct Kv4Seq {
  int64_t row0;
  int32_t n_new, len;
  bool ok;
};

IFQ_DEVINL Kv4Seq kv4_seq(const Kv4Arg& c, int b) {
  Kv4Seq s;
  s.ok = true;
  s.len = ld_after(c.kv_lens + b);
  s.row0 = (int64_t)b * c.n_new;
  s.n_new = c.n_new;
  if (c.new_offsets) {
    const int32_t o0 = ld_after(c.new_offsets + b), o1 = ld_after(c.new_offsets + b + 1);
    s.row0 = o0;
    s.n_new = o1 - o0;
    if (o0 < 0 || o1 < o0 || o1 > c.rows || s.n_new > c.n_new) {
      s.ok = false;
      s.n_new = 0;
    }
  }
  if (s.len < s.n_new || s.len > c.table_cols * c.page_tiles * 16) s.ok = false;
  if (!s.ok) s.len = 0;
  return s;
}

// The record of head h that holds positions 16 tile .. 16 tile + 15 of sequence b, or null where the page
// table does not name a page of the cache.
IFQ_DEVINL uint8_t* kv4_record(const Kv4Arg& c, int b, int h, int32_t tile) {
  const int32_t pc = tile / c.page_tiles, in = tile - pc * c.page_tiles;
  const int32_t page = ld_after(c.page_table + (int64_t)b * c.table_cols + pc);
  if (page < 0 || page >= c.pages) return nullptr;
  return c.records + (((int64_t)page * c.kv_heads + h) * c.page_tiles + in) * c.record_bytes;
}

}  // namespace ifq
