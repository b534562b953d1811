// The 8-bit paged cache of grouped-query attention: E4M3 codes, 16 tokens of a
// key head a block with one power-of-two scale for its keys and one for its
// values (bytes e + 127, value = code 2^e).
//
// A block's 16 D codes lie in the order that the matrix instruction takes
// them, so that a wave reads whole 1 KB runs straight into operand registers:
//   keys    [D / 16][16 tokens][16 values]
//   values  [D / 2][2][2][2][4]: value pair d / 2, (t / 4) % 2, d % 2, t / 8, t % 4
// (a lane half's 8 tokens of one value are consecutive, in the order in which
// a score accumulator holds them, and 16 bytes hold them for two values).
// Blocks of a head follow one another within a page, heads within a page.
//
// The scale is the smallest power of two that brings the block's largest
// magnitude within 448. A finer scale would not gain: the codes have an
// exponent of their own. A later token that raises it leaves earlier codes
// their digits, except where they fall below the codes' normal range. It is not
// lowered while the block holds earlier tokens, also where a request goes back
// over the token that raised it: the digits that the second rounding took would
// not return.
#pragma once

#include "gqa.h"
#include "mx_codec.h"

namespace moe {
namespace gqa {

constexpr int kBlock = 16;

// smallest e in [-127, 127] with amax <= 448 2^e (0: -127); an infinity counts
// as the largest finite magnitude
__device__ __forceinline__ int scale_exponent(float amax) {
  if (!(amax > 0.f)) return -127;
  const uint32_t u = __float_as_uint(fminf(amax, 3.4028235e38f));
  const int e = floor_log2(__uint_as_float(u)) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < -127 ? -127 : e;
}

// ---- host side -----------------------------------------------------------------
inline int check_cache(const std::string& fn, int B, int T, int page_size, int n_pages, int max_pages, int nkv) {
  MOE_REQUIRE(B >= 0 && B <= 65536 && T >= 0, MOE_ERR_INVALID_ARG, fn + ": B must be in [0, 65536], T >= 0");
  // grids stay below 2^32 work items
  MOE_REQUIRE(static_cast<int64_t>(T) * nkv <= (1 << 24) && static_cast<int64_t>(B) * nkv <= (1 << 19),
              MOE_ERR_INVALID_ARG, fn + ": T * n_kv_heads must be <= 2^24, B * n_kv_heads <= 2^19");
  MOE_REQUIRE(page_size >= kBlock && page_size % kBlock == 0, MOE_ERR_INVALID_ARG,
              fn + ": page_size must be a multiple of 16");
  MOE_REQUIRE(n_pages >= 1 && max_pages >= 1 &&
                  static_cast<int64_t>(page_size) / kBlock * n_pages * nkv < (int64_t{1} << 31) &&
                  static_cast<int64_t>(page_size) * max_pages <= (1 << 30),
              MOE_ERR_INVALID_ARG,
              fn + ": n_pages and max_pages must be >= 1, the cache's blocks below 2^31, page_size * max_pages <= 2^30");
  return MOE_OK;
}

}  // namespace gqa
}  // namespace moe
