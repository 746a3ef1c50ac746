// The paged cache of keys and values in 4 bits, as its kernels see it.
//
// Per page and key/value head, page_size rows of D / 2 bytes: the codes of one
// token's head, each c in [-7, 7] as the nibble c + 8, the low nibble first.
// k_codes holds a head's dimensions in order. v_codes holds them as
// [16][G][D / 16 / G]: sixteenth u of a row has D / 16 / G dimensions of every
// group, so that the 16 lanes of a matrix operand each read one sixteenth and
// every output tile of 16 dimensions belongs to one group of scales (G = 1: in
// order, too). Scales are fp32 [page][head][G][page_size]: four tokens' scales
// are one 16-byte load.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cider {

struct Kv4Cache {
  uint8_t* k_codes;
  float* k_scale;
  uint8_t* v_codes;
  float* v_scale;
  int64_t n_pages;
  int page_size, page_shift;   // tokens per page, a power of two
  int kv_heads, head_dim, groups;
};

}  // namespace cider
