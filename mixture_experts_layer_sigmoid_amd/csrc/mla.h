// Device helpers shared by the latent-attention kernels: sizes, LDS tile
// layouts and their loaders, matrix-core operand reads, packed sequences.
//
// Latent attention keeps one latent vector c (512 values) and one rotary key
// (64 values) per token for all heads; head h's key is (W_UK[h] c | rotary
// key), its value W_UV[h] c. (TE DeepSeekV3Layer page, Description,
// MultiLatentAttention item.)
//
// Operand layout of the 32x32x16 bf16 matrix instruction (lane l, half
// g = l / 32): A holds row l % 32, B column l % 32, both k = 8 g .. 8 g + 7;
// the accumulator holds column l % 32 and rows 8 (i / 4) + 4 g + i % 4. The
// attention kernels compute scores transposed (keys as rows, queries as
// columns, or the other way round where the keys are the kept side), so the
// kept side is one lane's own and softmax statistics, masks and rescaling
// need no exchange beyond the two halves. The accumulator of such a product
// is at once the B operand of the next one: its rows 16 s + {4 g .. 4 g + 3,
// 8 + 4 g .. 8 + 4 g + 3} are taken as the k values of k-step s, and the A
// operand is read in the same order by two transposed LDS reads of four rows.
#pragma once

#include "gemm_util.h"

#include <type_traits>

namespace moe {
namespace mla {

constexpr int kDn = 128;              // per-head key values made from the latent
constexpr int kDr = 64;               // rotary key values, shared by the heads
constexpr int kDq = kDn + kDr;        // query / key size
constexpr int kDv = 128;              // value size
constexpr int kR = 512;               // latent
constexpr int kDc = kR + kDr;         // cache row
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMaxScale = 2.3e38f;  // its product with kLog2e is finite

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));

// ---- LDS tiles ---------------------------------------------------------------
// A tile of rows of RB bytes stores row r's 16-byte chunk c at chunk
// c ^ key(r). Two kinds of reads have to be free of bank conflicts over a
// 256-byte LDS line: 16 consecutive rows at one logical chunk (operands read
// as they lie), and 4 consecutive rows x 4 consecutive chunks (transposed
// reads). Rows of 256 bytes or a multiple: the low two row bits choose the
// group of 4 chunks, the next two the chunk within it. Rows of 128 bytes:
// two rows share a line, so the row's lowest bit is already in the address.
template <int RB>
__device__ __forceinline__ int tile_key(int r) {
  return RB == 128 ? (((r & 2) << 1) | ((r >> 2) & 3)) : (((r & 3) << 2) | ((r >> 2) & 3));
}

// Copies rows [0, ROWS) of RB bytes, `stride` bytes apart from `base`, into
// an LDS tile; rows at or past n_valid are zero (the buffer's range check).
// One instruction moves 1 KB; NW waves share the work.
template <int RB, int ROWS, int NW>
__device__ __forceinline__ void tile_load(const void* base, uint32_t stride, int n_valid,
                                          uint8_t* lds, int wave, int lane) {
  constexpr int kPer = 1024 / RB;              // rows per instruction
  constexpr int kIns = ROWS / kPer;
  const uint32_t bytes = n_valid > 0 ? (n_valid - 1) * stride + RB : 0u;
  const __amdgpu_buffer_rsrc_t rs = buf_rsrc(base, bytes);
  const int c = lane & (RB / 16 - 1);
  const int lr = lane / (RB / 16);
#pragma unroll
  for (int i = 0; i < (kIns + NW - 1) / NW; ++i) {
    const int ins = wave + i * NW;
    if (kIns % NW == 0 || ins < kIns) {
      const int r = ins * kPer + lr;
      lds_load16_buf(rs, r * stride + ((c ^ tile_key<RB>(r)) << 4), 0, lds + ins * 1024);
    }
  }
}

// A or B operand (32 rows as they lie): LDS byte offset of chunk 2 s + g of
// row l % 32; add 32 RB per row block.
template <int RB>
__device__ __forceinline__ uint32_t row_operand_offset(int lane, int s) {
  const int r = lane & 31, g = lane >> 5;
  return r * RB + (((2 * s + g) ^ tile_key<RB>(r)) << 4);
}
__device__ __forceinline__ bf16x8_t row_operand(const uint8_t* lds, uint32_t off) {
  return *reinterpret_cast<const bf16x8_t*>(lds + off);
}

// Transposed operand (columns of the tile as operand rows, tile rows as k, in
// the accumulator's order): byte offset of read p (0, 1) of 32-column block
// cb; add 16 RB per k-step of 16 tile rows.
template <int RB>
__device__ __forceinline__ uint32_t col_operand_offset(int lane, int cb, int p) {
  const int i = lane & 15, g = lane >> 5, m = (lane >> 4) & 1;
  const int r = 8 * p + 4 * g + (i >> 2);
  const int c = 4 * cb + 2 * m + ((i & 3) >> 1);
  return r * RB + ((c ^ tile_key<RB>(r)) << 4) + (i & 1) * 8;
}
__device__ __forceinline__ bf16x8_t col_operand(const uint8_t* __restrict__ lds, uint32_t off0, uint32_t off1) {
  typedef __attribute__((address_space(3))) bf16x4_t* lptr;
  const bf16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lptr)(lds + off0));
  const bf16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lptr)(lds + off1));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// f(integral_constant<0>) ... f(integral_constant<N - 1>), unrolled at compile time
template <int I, int N, typename Fn>
__device__ __forceinline__ void static_for_impl(Fn&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for_impl<I + 1, N>(f);
  }
}
template <int N, typename Fn>
__device__ __forceinline__ void static_for(Fn&& f) { static_for_impl<0, N>(f); }

__device__ __forceinline__ f32x16_t mfma(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Sums that stay in the accumulation registers from the first product to the
// last. Ordinary code that reads one (a rescaling, the final store) would make
// the compiler keep them in vector registers between the products and copy
// them all back and forth in every tile, so each tile's products end in
// keep_acc and such code reads through read_acc. The compiler does not know
// what read_acc's instruction reads, so the products that wrote the sums have
// to be over: acc_settled waits longer than the slowest product takes.
__device__ __forceinline__ void keep_acc(f32x16_t& v) { asm volatile("" : "+a"(v)); }
__device__ __forceinline__ float read_acc(float v) {
  float r;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(r) : "a"(v));
  return r;
}
__device__ __forceinline__ void acc_settled() { asm volatile("s_nop 15\n\ts_nop 15"); }

// accumulator rows of k-step s (values 8 s .. 8 s + 7) as a bf16 operand
__device__ __forceinline__ bf16x8_t pack_operand(const f32x16_t& v, int s) {
  typedef float f32x8_t __attribute__((ext_vector_type(8)));
  const f32x8_t w = {v[8 * s], v[8 * s + 1], v[8 * s + 2], v[8 * s + 3],
                     v[8 * s + 4], v[8 * s + 5], v[8 * s + 6], v[8 * s + 7]};
  return __builtin_convertvector(w, bf16x8_t);
}

__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d) {
  const bf16x4_t v = __builtin_convertvector((f32x4_t{a, b, c, d}), bf16x4_t);
  return __builtin_bit_cast(uint2, v);
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_hw(float x) { return __builtin_amdgcn_logf(x); }

// Running reference of a row's weights 2^(x - ref): it follows the maximum
// only once that has grown by more than 2^kLazy, so the sums are rescaled in
// few tiles instead of nearly every one (with 32 rows a wave some row's
// maximum grows almost always). Weights stay below 2^kLazy, far inside the
// range of bf16 and fp32, whose precision does not depend on the scale.
constexpr float kLazy = 8.f;
__device__ __forceinline__ float next_ref(float ref, float mx, float c2) {
  return (mx - ref) * c2 > kLazy ? mx : ref;       // ref -inf: taken whenever mx is finite
}

// value of the other half's lane (l ^ 32)
__device__ __forceinline__ float other_half(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// ---- results --------------------------------------------------------------------
// A wave's 32 result rows of RB bytes leave through LDS (`rows`, its own 32 x
// (RB + 16) bytes): out of the registers a store would touch 32 rows with 8
// bytes each, from here it writes whole rows.
template <int RB>
constexpr int result_bytes() { return 32 * (RB + 16); }
template <int RB>
__device__ __forceinline__ void store_rows(const uint8_t* rows, void* dst, int64_t ld_bytes, int n, int lane) {
  constexpr int kC = RB / 16;                            // 16-byte pieces a row
#pragma unroll
  for (int i = 0; i < 32 * kC / 64; ++i) {
    const int c = i * 64 + lane, r = c / kC;
    if (r < n)
      *reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(dst) + r * ld_bytes + (c % kC) * 16) =
          *reinterpret_cast<const u32x4_t*>(rows + r * (RB + 16) + (c % kC) * 16);
  }
}

// ---- packed sequences --------------------------------------------------------
// Sequence and tile of a work index: sequence b has ceil(n_b / per) tiles,
// n_b = cu[b + 1] - cu[b]; all 64 lanes of the wave take part. Offsets are
// clamped to [0, total] so no entry of cu can lead outside the tensors.
struct SeqTile {
  int b;         // -1: no such tile
  int tile;      // within the sequence
  int start, n;  // the sequence's rows
  int start2, n2;  // and those of the other side (keys for queries, queries for keys)
};
__device__ __forceinline__ int clamp_int(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

__device__ __forceinline__ SeqTile find_tile(const int32_t* cu, const int32_t* cu2, int B, int total, int total2,
                                             int per, int index) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int b0 = 0; b0 < B; b0 += 64) {
    const int b = b0 + lane;
    int s = 0, n = 0, s2 = 0, n2 = 0;
    if (b < B) {                       // both sides at once: one trip to memory
      const int a0 = cu[b], a1 = cu[b + 1], b0_ = cu2[b], b1 = cu2[b + 1];
      s = clamp_int(a0, 0, total);
      n = clamp_int(a1, s, total) - s;
      s2 = clamp_int(b0_, 0, total2);
      n2 = clamp_int(b1, s2, total2) - s2;
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

// Workgroups go to the XCDs round-robin; give each XCD a contiguous run of
// work indices, so that tiles that share keys share an L2.
__device__ __forceinline__ int xcd_contiguous(int id, int n) {
  const int x = id % kNumXcd, q = n / kNumXcd, rem = n % kNumXcd;
  return x * q + (x < rem ? x : rem) + id / kNumXcd;
}

// ---- host side -----------------------------------------------------------------
// upper bound of the tiles of `per` rows over B packed sequences of `total` rows
inline int seq_tiles_bound(int B, int total, int per) {
  const int seqs = B < total ? B : total;
  return total / per + seqs;
}

constexpr int64_t kMaxLd = int64_t{1} << 23;   // a 64-row tile stays below 2 GB

// argument checks shared by the expanded forward and backward
inline int check_expanded(const std::string& fn, int fmt, int B, int Tq, int Tk, int nh, int causal, float scale,
                          int64_t q_ld, int64_t kv_ld, int64_t kr_ld, int64_t out_ld) {
  MOE_REQUIRE(B >= 0 && Tq >= 0 && Tk >= 0 && Tq <= (1 << 28) && Tk <= (1 << 28), MOE_ERR_INVALID_ARG,
              fn + ": B must be >= 0, Tq and Tk in [0, 2^28]");
  MOE_REQUIRE(nh >= 1 && nh <= 1024, MOE_ERR_INVALID_ARG, fn + ": n_heads must be in [1, 1024]");
  // grids stay below 2^32 work items (the backward's sums of the heads' rotary
  // gradients, 64 work items a key, are cut into launches that do)
  MOE_REQUIRE(static_cast<int64_t>(Tq) * nh <= (1 << 27) && static_cast<int64_t>(Tk) * nh <= (1 << 27) &&
                  static_cast<int64_t>(B) * nh <= (1 << 22),
              MOE_ERR_INVALID_ARG, fn + ": Tq * n_heads and Tk * n_heads must be <= 2^27, B * n_heads <= 2^22");
  MOE_REQUIRE(fmt == MOE_BF16, MOE_ERR_UNSUPPORTED, fn + ": fmt must be MOE_BF16");
  MOE_REQUIRE(causal == 0 || causal == 1, MOE_ERR_INVALID_ARG, fn + ": causal must be 0 or 1");
  MOE_REQUIRE(scale > 0.f && scale <= kMaxScale, MOE_ERR_INVALID_ARG, fn + ": scale must be in (0, 2.3e38]");
  MOE_REQUIRE(q_ld >= static_cast<int64_t>(nh) * kDq && kv_ld >= static_cast<int64_t>(nh) * (kDn + kDv) &&
                  kr_ld >= kDr && out_ld >= static_cast<int64_t>(nh) * kDv && q_ld <= kMaxLd && kv_ld <= kMaxLd &&
                  kr_ld <= kMaxLd && out_ld <= kMaxLd,
              MOE_ERR_INVALID_ARG, fn + ": a row stride is smaller than its row or above 2^23 elements");
  MOE_REQUIRE(q_ld % 8 == 0 && kv_ld % 8 == 0 && kr_ld % 8 == 0 && out_ld % 8 == 0, MOE_ERR_ALIGNMENT,
              fn + ": row strides must be multiples of 8 elements");
  return MOE_OK;
}

}  // namespace mla
}  // namespace moe
