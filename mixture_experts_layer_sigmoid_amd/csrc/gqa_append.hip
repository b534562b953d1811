// moe_gqa_append: new keys and values into the 8-bit paged cache.
//
// Request b's n new tokens are its last: positions lens[b] - n .. lens[b] - 1.
// For every block of 16 positions that they touch, per key head, for keys and
// values apart:
//   e = smallest exponent with max |new values| <= 448 2^e,
//       not below the block's own where it holds earlier tokens
//   codes of the new tokens = E4M3(x 2^-e); earlier codes, if e grew, are
//   rounded again from code 2^(e_old - e)
// One wave owns a (block, key head, keys or values), so nothing is shared and
// no order matters; bytes of later positions stay as they are.
//
// Memory bounds a long prompt: 8192 tokens x 8 key heads of 128 take 11.7 to 13 us
// for 50 MB (3.9 to 4.3 TB/s); a single token for each of 64 requests is latency
// (5.4 us: the request's place, its page, then the block and the token side by
// side). Every wave walks through all requests to find its block: a token for
// each of 1024 takes 47 us, of 4096 0.51 ms.
#include "gqa_cache.h"

#include <cmath>

namespace moe {
namespace gqa {
namespace {

struct AppendArgs {
  const uint16_t* k;
  int64_t k_ld;
  const uint16_t* v;
  int64_t v_ld;
  uint8_t* k_cache;
  uint8_t* v_cache;
  uint8_t* k_scales;
  uint8_t* v_scales;
  int n_pages;
  Div bpp;                 // blocks per page
  const int32_t* table;
  int max_pages;
  const int32_t* lens;
  const int32_t* cu;
  int B, T, nkv;
};

struct Block {
  int b;                   // -1: none
  int block;               // of the request
  int first, len;          // positions of its new tokens: [first, len)
  int row;                 // row of the token at position 0 (may be negative)
};

// block `index` of the blocks that the requests' new tokens touch
__device__ __forceinline__ Block find_block(const AppendArgs& p, int index) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 64) {
    const int b = b0 + lane;
    int s = 0, n = 0, len = 0, first = 0, blocks = 0;
    if (b < p.B) {
      const int a0 = p.cu[b], a1 = p.cu[b + 1];
      len = clamp_int(p.lens[b], 0, p.max_pages * p.bpp.d * kBlock);
      s = clamp_int(a0, 0, p.T);
      n = clamp_int(a1, s, p.T) - s;
      first = max(len - n, 0);
      blocks = n > 0 && len > 0 ? (len - 1) / kBlock - first / kBlock + 1 : 0;
    }
    int sum = blocks;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(sum, o, 64);
      if (lane >= o) sum += u;
    }
    const uint64_t hit = __ballot(before + sum > index);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      Block r;
      r.b = b0 + l;
      r.first = __builtin_amdgcn_readlane(first, l);
      r.len = __builtin_amdgcn_readlane(len, l);
      r.block = index - before - (__builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(blocks, l)) +
                r.first / kBlock;
      r.row = __builtin_amdgcn_readlane(s, l) + __builtin_amdgcn_readlane(n, l) - r.len;
      return r;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return Block{-1, 0, 0, 0, 0};
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

// four values 2^-e as codes; four codes 2^d as codes
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, int e) {
  typedef short short2_t __attribute__((ext_vector_type(2)));
  short2_t o = {0, 0};
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, ldexpf(a, -e), ldexpf(b, -e), 1.f, false);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, ldexpf(c, -e), ldexpf(d, -e), 1.f, true);
  return __builtin_bit_cast(uint32_t, o);
}
__device__ __forceinline__ uint32_t move4(uint32_t w, int d) {
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, 1.f, false);
  const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, 1.f, true);
  return encode4(a[0], a[1], b[0], b[1], -d);
}

// The block's exponent: of the new values, and of the block's own where it
// holds earlier tokens (d: how much those codes move, never above 0).
__device__ __forceinline__ int merge_exponent(float amax, bool had, int old, int* d) {
  int e = scale_exponent(amax);
  *d = 0;
  if (had) {
    e = max(e, old);
    *d = old - e;
  }
  return e;
}

// Keys: 4 lanes a token, each every fourth chunk of 16 values.
template <int D>
__device__ __forceinline__ void append_keys(const AppendArgs& p, const Block& bl, int head, int64_t phys, int lane) {
  constexpr int kC = D / 64;                           // chunks a lane
  const int t = lane >> 2, pos = bl.block * kBlock + t;
  const bool mine = pos >= bl.first && pos < bl.len;
  const int start = bl.block * kBlock;
  const bool had = bl.first > start;
  uint8_t* sc = p.k_scales + phys;
  const int old = had ? static_cast<int>(*sc) - 127 : 0;
  float x[kC][16];
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[c][i] = 0.f;
    if (mine) {
      const uint16_t* src = p.k + static_cast<int64_t>(bl.row + pos) * p.k_ld + head * D + 16 * ((lane & 3) + 4 * c);
      const u32x4_t a = reinterpret_cast<const u32x4_t*>(src)[0], b = reinterpret_cast<const u32x4_t*>(src)[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[c][2 * i] = __uint_as_float(a[i] << 16), x[c][2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
        x[c][8 + 2 * i] = __uint_as_float(b[i] << 16), x[c][9 + 2 * i] = __uint_as_float(b[i] & 0xFFFF0000u);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[c][i]));
    }
  }
  int d;
  const int e = merge_exponent(wave_max(amax), had, old, &d);
  uint8_t* dst = p.k_cache + phys * (kBlock * D) + t * 16;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    u32x4_t* o = reinterpret_cast<u32x4_t*>(dst + ((lane & 3) + 4 * c) * 256);
    u32x4_t w;
    if (mine) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = encode4(x[c][4 * i], x[c][4 * i + 1], x[c][4 * i + 2], x[c][4 * i + 3], e);
      *o = w;
    } else if (d < 0 && pos < bl.first) {
      w = *o;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = move4(w[i], d);
      *o = w;
    }
  }
  if (lane == 0) *sc = static_cast<uint8_t>(e + 127);
}

// Values: a lane takes one pair of values (D = 128), or of two lanes each 8
// of the 16 tokens (D = 64): words (parity, t / 8) of 4 tokens each, for both
// or one of the halves (t / 4) % 2.
template <int D>
__device__ __forceinline__ void append_values(const AppendArgs& p, const Block& bl, int head, int64_t phys, int lane) {
  constexpr int kH = D / 64;                           // halves a lane
  const int pair = D == 128 ? lane : lane & 31;
  const int start = bl.block * kBlock;
  const bool had = bl.first > start;
  uint8_t* sc = p.v_scales + phys;
  const int old = had ? static_cast<int>(*sc) - 127 : 0;
  const uint16_t* src = p.v + static_cast<int64_t>(bl.row + start) * p.v_ld + head * D + 2 * pair;
  u32x4_t* dst = reinterpret_cast<u32x4_t*>(p.v_cache + phys * (kBlock * D) + pair * 32);
  const int lo = bl.first - start, hi = bl.len - start;  // new tokens of the block
  // a block that holds only new tokens, all 16, is written without being read
  const bool whole = lo <= 0 && hi >= kBlock;
  uint32_t x[kH][8];
  u32x4_t w[kH];
  float amax = 0.f;
#pragma unroll
  for (int h = 0; h < kH; ++h) {
    const int half = D == 128 ? h : lane >> 5;
    if (!whole) w[h] = dst[half];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = 8 * (i >> 2) + 4 * half + (i & 3);
      x[h][i] = t >= lo && t < hi ? *reinterpret_cast<const uint32_t*>(src + t * p.v_ld) : 0u;
      amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[h][i] << 16)), fabsf(__uint_as_float(x[h][i] & 0xFFFF0000u))));
    }
  }
  int d;
  const int e = merge_exponent(wave_max(amax), had, old, &d);
#pragma unroll
  for (int h = 0; h < kH; ++h) {
    const int half = D == 128 ? h : lane >> 5;
    u32x4_t r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {                      // parity j / 2, t / 8 = j % 2
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t y = x[h][4 * (j & 1) + i];
        f[i] = __uint_as_float(j >> 1 ? y & 0xFFFF0000u : y << 16);
      }
      const uint32_t fresh = encode4(f[0], f[1], f[2], f[3], e);
      if (whole) {
        r[j] = fresh;
      } else {
        const uint32_t prev = w[h][j], moved = d < 0 ? move4(prev, d) : prev;
        uint32_t o = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 8 * (j & 1) + 4 * half + i;
          o |= (t < lo ? moved : (t < hi ? fresh : prev)) & (0xFFu << (8 * i));
        }
        r[j] = o;
      }
    }
    dst[half] = r;
  }
  if (lane == 0) *sc = static_cast<uint8_t>(e + 127);
}

// a wave per (block, key head, keys or values)
template <int D>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = 2 * p.nkv;
  const int index = static_cast<int>(unit / per), which = static_cast<int>(unit - static_cast<int64_t>(index) * per);
  const Block bl = find_block(p, index);
  if (bl.b < 0) return;
  const int head = which >> 1;
  const int col = quot(bl.block, p.bpp);
  const int page = clamp_int(p.table[static_cast<int64_t>(bl.b) * p.max_pages + col], 0, p.n_pages - 1);
  const int64_t phys = (static_cast<int64_t>(page) * p.nkv + head) * p.bpp.d + (bl.block - col * p.bpp.d);
  if (which & 1) append_values<D>(p, bl, head, phys, lane);
  else append_keys<D>(p, bl, head, phys, lane);
}

}  // namespace
}  // namespace gqa
}  // namespace moe

extern "C" int moe_gqa_append(const void* k, int64_t k_ld, const void* v, int64_t v_ld, int fmt, void* k_cache,
                              void* v_cache, uint8_t* k_scales, uint8_t* v_scales, int page_size, int n_pages,
                              const int32_t* page_table, int max_pages, const int32_t* lens, const int32_t* cu, int B,
                              int T, int n_kv_heads, int head_dim, hipStream_t stream) {
  using namespace moe;
  using namespace moe::gqa;
  clear_error();
  const char* fn = "moe_gqa_append";
  if (const int rc = check_heads(fn, fmt, n_kv_heads, n_kv_heads, head_dim)) return rc;
  if (const int rc = check_cache(fn, B, T, page_size, n_pages, max_pages, n_kv_heads)) return rc;
  const int64_t row = static_cast<int64_t>(n_kv_heads) * head_dim;
  if (const int rc = check_ld(fn, "k_ld", k_ld, row)) return rc;
  if (const int rc = check_ld(fn, "v_ld", v_ld, row)) return rc;
  if (B == 0 || T == 0) return MOE_OK;
  MOE_REQUIRE(k && v && k_cache && v_cache && k_scales && v_scales && page_table && lens && cu, MOE_ERR_INVALID_ARG,
              "moe_gqa_append: null pointer");
  MOE_REQUIRE(aligned16(k) && aligned16(v) && aligned16(k_cache) && aligned16(v_cache), MOE_ERR_ALIGNMENT,
              "moe_gqa_append: k, v and the cache must be 16-byte aligned");
  AppendArgs a{static_cast<const uint16_t*>(k), k_ld, static_cast<const uint16_t*>(v), v_ld,
               static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), k_scales, v_scales, n_pages,
               make_div(page_size / kBlock), page_table, max_pages, lens, cu, B, T, n_kv_heads};
  // n tokens touch at most (n + 14) / 16 + 1 blocks
  const int64_t blocks = T / kBlock + 2 * static_cast<int64_t>(B < T ? B : T);
  const dim3 grid(static_cast<unsigned>((blocks * 2 * n_kv_heads + 3) / 4));
  if (head_dim == 128) hipLaunchKernelGGL(append_kernel<128>, grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL(append_kernel<64>, grid, dim3(256), 0, stream, a);
  return check_launch(fn);
}
