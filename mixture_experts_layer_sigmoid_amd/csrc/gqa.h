// Device helpers shared by the grouped-query attention kernels: n_heads query
// heads in groups of G share n_kv = n_heads / G key and value heads of D = 64
// or 128 values.
//
// The queries of a group and of consecutive tokens are packed as the rows of
// one product: row r of key head h is token r / G, query head h G + r % G.
// So a workgroup's rows span few tokens (128 rows of 8 heads: 16), which share
// the keys once loaded and cut the causal diagonal finely, and a token's heads
// lie side by side in memory.
#pragma once

#include "mla.h"

namespace moe {
namespace gqa {

using namespace mla;

// x / d and x % d for 0 <= x < 2^31, 1 <= d < 2^31: with 2^(s - 1) < d <= 2^s
// and m = ceil(2^(31 + s) / d) < 2^32, x m / 2^(31 + s) exceeds x / d by less
// than 1 / d.
struct Div {
  uint32_t magic;
  int shift, d;
};
inline Div make_div(int d) {
  int s = 0;
  while ((int64_t{1} << s) < d) ++s;
  return Div{static_cast<uint32_t>(((uint64_t{1} << (31 + s)) + d - 1) / d), s, d};
}
__device__ __forceinline__ int quot(int x, const Div& d) {
  return static_cast<int>(__umulhi(2 * static_cast<uint32_t>(x), d.magic) >> d.shift);
}

// Tile `index` of `per` rows over packed sequences whose tokens have `mult`
// rows each (find_tile with rows counted that way; n and tile are in rows,
// start, start2 and n2 in tokens).
__device__ __forceinline__ SeqTile find_rows(const int32_t* cu, const int32_t* cu2, int B, int total, int total2,
                                             int mult, int per, int index) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int b0 = 0; b0 < B; b0 += 64) {
    const int b = b0 + lane;
    int s = 0, n = 0, s2 = 0, n2 = 0;
    if (b < B) {
      const int a0 = cu[b], a1 = cu[b + 1], c0 = cu2[b], c1 = cu2[b + 1];
      s = clamp_int(a0, 0, total);
      n = (clamp_int(a1, s, total) - s) * mult;
      s2 = clamp_int(c0, 0, total2);
      n2 = clamp_int(c1, s2, total2) - s2;
    }
    const int tiles = (n + per - 1) / per;
    int sum = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(sum, o, 64);
      if (lane >= o) sum += u;
    }
    const uint64_t hit = __ballot(before + sum > index);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      SeqTile t;
      t.b = b0 + l;
      t.tile = index - before - (__builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(tiles, l));
      t.start = __builtin_amdgcn_readlane(s, l);
      t.n = __builtin_amdgcn_readlane(n, l);
      t.start2 = __builtin_amdgcn_readlane(s2, l);
      t.n2 = __builtin_amdgcn_readlane(n2, l);
      return t;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return SeqTile{-1, 0, 0, 0, 0, 0};
}

// Copies packed rows [r0, r0 + ROWS) of one key head into an LDS tile (the
// layout of tile_load). base: the sequence's first token at the group's first
// head; rows at or past n_rows (a whole number of tokens) are zero: they lie
// behind the buffer's end.
template <int RB, int ROWS, int NW>
__device__ __forceinline__ void rows_load(const uint16_t* base, int64_t ld, const Div& g, int r0, int n_rows,
                                          uint8_t* lds, int wave, int lane) {
  constexpr int kPer = 1024 / RB;
  constexpr int kIns = ROWS / kPer;
  static_assert(kIns % NW == 0, "whole instructions a wave");
  const int t0 = quot(r0, g), t_end = min(quot(r0 + ROWS - 1, g) + 1, quot(n_rows, g));
  const uint32_t ld_b = static_cast<uint32_t>(ld * 2);
  const uint32_t bytes = t_end > t0 ? (t_end - t0 - 1) * ld_b + g.d * RB : 0u;
  const __amdgpu_buffer_rsrc_t rs = buf_rsrc(base + static_cast<int64_t>(t0) * ld, bytes);
  const int c = lane & (RB / 16 - 1);
  const int lr = lane / (RB / 16);
#pragma unroll
  for (int i = 0; i < kIns / NW; ++i) {
    const int ins = wave + i * NW;
    const int r = ins * kPer + lr;
    const int t = quot(r0 + r, g);
    const uint32_t off = static_cast<uint32_t>(t - t0) * ld_b + static_cast<uint32_t>(r0 + r - t * g.d) * RB;
    lds_load16_buf(rs, off + ((c ^ tile_key<RB>(r)) << 4), 0, lds + ins * 1024);
  }
}

// The same for tiles that follow one another where the group divides the rows
// that the waves load at a time: a tile is whole tokens and all tiles' offsets
// are the first one's, so that nothing is left to compute per lane and tile
// (backward of 4096 tokens x 64 heads 1 to 2%).
template <int RB, int ROWS, int NW>
struct EvenRows {
  static constexpr int kPer = 1024 / RB, kStep = kPer * NW;
  const uint16_t* base;
  int64_t ld;
  uint32_t ld_b, off, step;
  int n_q, per;                                          // tokens of the sequence and of a tile

  static __device__ __forceinline__ bool fits(const Div& g) { return kStep % g.d == 0; }
  __device__ __forceinline__ EvenRows(const uint16_t* b, int64_t l, const Div& g, int n, int wave, int lane)
      : base(b), ld(l), ld_b(static_cast<uint32_t>(l * 2)), n_q(n), per(ROWS / g.d) {
    const int c = lane & (RB / 16 - 1), r = wave * kPer + lane / (RB / 16), t = quot(r, g);
    off = static_cast<uint32_t>(t) * ld_b + static_cast<uint32_t>(r - t * g.d) * RB + ((c ^ tile_key<RB>(r)) << 4);
    step = static_cast<uint32_t>(kStep / g.d) * ld_b;
  }
  __device__ __forceinline__ void load(int tile, const Div& g, uint8_t* lds, int wave) const {
    const int t0 = tile * per;
    const uint32_t bytes = static_cast<uint32_t>(min(per, n_q - t0) - 1) * ld_b + g.d * RB;
    const __amdgpu_buffer_rsrc_t rs = buf_rsrc(base + static_cast<int64_t>(t0) * ld, bytes);
#pragma unroll
    for (int i = 0; i < ROWS / kStep; ++i) lds_load16_buf(rs, off + i * step, 0, lds + (wave + i * NW) * 1024);
  }
};

// A wave's 32 result rows (packed rows r0 .. of one key head) from LDS to
// memory; dst: the sequence's first token at the group's first head.
template <int RB>
__device__ __forceinline__ void store_packed(const uint8_t* rows, uint16_t* dst, int64_t ld, const Div& g, int r0,
                                             int n_rows, int lane) {
  constexpr int kC = RB / 16;
#pragma unroll
  for (int i = 0; i < 32 * kC / 64; ++i) {
    const int c = i * 64 + lane, r = c / kC;
    if (r0 + r < n_rows) {
      const int t = quot(r0 + r, g);
      uint16_t* o = dst + static_cast<int64_t>(t) * ld + (r0 + r - t * g.d) * (RB / 2);
      *reinterpret_cast<u32x4_t*>(reinterpret_cast<uint8_t*>(o) + (c % kC) * 16) =
          *reinterpret_cast<const u32x4_t*>(rows + r * (RB + 16) + (c % kC) * 16);
    }
  }
}

// ---- host side -----------------------------------------------------------------
inline int check_heads(const std::string& fn, int fmt, int nh, int nkv, int D) {
  MOE_REQUIRE(nh >= 1 && nh <= 1024 && nkv >= 1 && nkv <= nh && nh % nkv == 0, MOE_ERR_INVALID_ARG,
              fn + ": n_heads must be in [1, 1024] and a multiple of n_kv_heads");
  MOE_REQUIRE(fmt == MOE_BF16, MOE_ERR_UNSUPPORTED, fn + ": fmt must be MOE_BF16");
  MOE_REQUIRE(D == 64 || D == 128, MOE_ERR_UNSUPPORTED, fn + ": head_dim must be 64 or 128");
  return MOE_OK;
}

inline int check_ld(const std::string& fn, const char* name, int64_t ld, int64_t row) {
  MOE_REQUIRE(ld >= row && ld <= kMaxLd, MOE_ERR_INVALID_ARG,
              fn + ": " + name + " is smaller than its row or above 2^23 elements");
  MOE_REQUIRE(ld % 8 == 0, MOE_ERR_ALIGNMENT, fn + ": " + name + " must be a multiple of 8 elements");
  return MOE_OK;
}

inline int check_sequences(const std::string& fn, int B, int Tq, int Tk, int nh, int causal, float scale) {
  MOE_REQUIRE(B >= 0 && Tq >= 0 && Tk >= 0 && Tq <= (1 << 27) && Tk <= (1 << 27), MOE_ERR_INVALID_ARG,
              fn + ": B must be >= 0, Tq and Tk in [0, 2^27]");
  // packed rows and grids stay far inside 31 bits
  MOE_REQUIRE(static_cast<int64_t>(Tq) * nh <= (1 << 27) && static_cast<int64_t>(Tk) * nh <= (1 << 27) &&
                  static_cast<int64_t>(B) * nh <= (1 << 22),
              MOE_ERR_INVALID_ARG, fn + ": Tq * n_heads and Tk * n_heads must be <= 2^27, B * n_heads <= 2^22");
  MOE_REQUIRE(causal == 0 || causal == 1, MOE_ERR_INVALID_ARG, fn + ": causal must be 0 or 1");
  MOE_REQUIRE(scale > 0.f && scale <= kMaxScale, MOE_ERR_INVALID_ARG, fn + ": scale must be in (0, 2.3e38]");
  return MOE_OK;
}

}  // namespace gqa
}  // namespace moe
