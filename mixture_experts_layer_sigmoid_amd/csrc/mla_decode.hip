// moe_mla_decode: latent attention over a paged cache, in absorbed form.
//
// With q_lat[t, h] = W_UK[h]^T q[t, h, :128] every head's scores are taken
// against the cached rows themselves:
//   s[j] = scale * (q_lat . c_j + q[t, h, 128:] . kr_j),  p = softmax(s)
//   o_lat = sum_j p_j c_j,   out[t, h] = W_UV[h] o_lat
// One cached row (512 latent values, 64 rotary ones) serves all heads as key
// and as value, so the heads of a request's new tokens are the rows of one
// matrix product over its cache.
//
// Three launches: the products with W_UK; the attention, its work cut evenly
// over the chip along the cached tokens; the joining of the pieces with the
// products with W_UV.
//
// Roundings: q_lat to bf16 and the weights p to bf16 (both operands of matrix
// instructions, rms 2^-9.2 of each; a wider q_lat would double the products
// of the scores); o_lat stays fp32 up to W_UV, where it enters as two bf16
// terms. A weight is rounded once more where the two halves of a token tile
// have other references and its own is brought to the larger. References in
// whole powers of two would spare that, but then the largest key's weight is
// no longer exactly 1, which costs more: out 2.60e-3 rms instead of 1.73e-3 (8
// long caches with lone tokens among them), 2.38 instead of 1.92 (64 ragged
// requests), 2.51 instead of 2.15 (trees of 32), the time the same. Scores,
// references, sums and pieces are fp32. Against 64 bits out has 1.7e-3 to
// 2.6e-3 rms: at 531 cached tokens 2.55e-3, the root of the squares of the
// output's own rounding (1.67), q_lat's (1.44) and the weights' (1.30).
//
// Bound, by size (an 8192^3 bf16 product reaches 1369 TFLOP/s here, a copy
// 4.87 TB/s):
//   256 tokens of 8 trees x 128 heads: 294 us attention (274-312) = 730
//     TFLOP/s. A tile of 64 tokens and 64 rows takes 4.9k cycles for 2.2k of
//     products: scores, softmax and value products follow one another between
//     barriers at one wave a SIMD (matrix unit 39% busy); join 42, q_lat 17;
//   64 ragged requests x 128 heads: 83-85 us, the same tiles (a workgroup has 22
//     on average, four fifths of its time) and the pieces' starts and ends
//     (queries in, sums out: about 18k cycles a piece, 1.4 a workgroup); matrix
//     unit 29% busy; join 20, q_lat 7.5 us;
//   8 long caches x 16 heads, 279k cached tokens: 63 us = 5.1 TB/s, at the
//     rate of a copy; join 14.5 us (its pieces' traffic);
//   one request x 16 heads, 531 tokens: 3 + 10 + 6.7 us, latency.
// The attention fills its registers: 256 and 230 to 250 accumulation registers
// a wave, one wave a SIMD; 61 to 69 scalar values (the work list's, page
// addresses) live in vector lanes. With 32 rows a workgroup has two waves and
// 148 KB of LDS, so two of a compute unit's four SIMDs are empty; long caches
// run at a copy's rate all the same.
#include "mla.h"

#include <cmath>

namespace moe {
namespace mla {
namespace {

constexpr int kTok = 64;                               // cached tokens per tile
constexpr int kLat = kTok * kR * 2, kRope = kTok * kDr * 2, kTile = kLat + kRope;
constexpr int kAhead = 6;                              // matrix operands read ahead
constexpr int kPieceCost = 4;                          // in token tiles; see the work list
constexpr int kShortRuns = 96;                         // more units: runs of two and more
constexpr int kGroups = 256;                           // workgroups of the attention

struct DecodeArgs {
  const uint16_t* q;
  int64_t q_ld;
  const uint16_t* w_uk;      // [nh, 512, 128] and [nh, 128, 512] in moe_pack_weights'
  const uint16_t* w_uv;      // order: per 32 rows and 16 columns one 1 KB operand
  const uint16_t* cache;
  int page_size, n_pages;
  uint32_t page_magic;       // x / page_size = umulhi(2 x, page_magic) >> page_shift for 0 <= x < 2^31
  int page_shift;
  const int32_t* table;
  int max_pages;
  const int32_t* lens;
  const int32_t* cu_q;
  const uint64_t* tree;
  int B, T, nh;
  int team;                  // workgroups that take neighbouring row tiles together
  float scale;
  uint16_t* out;
  int64_t out_ld;
  float* lse;
  uint16_t* q_lat;           // [T * nh, 512]
  float* o_full;             // [T * nh, 512]: rows whose cache one workgroup covered, not normalized
  float* part;               // [2 kGroups, rows, 512]: pieces, not normalized
  float2* part_ml;           // [2 kGroups, rows]: their (maximum, sum)
  int2* info;                // [T * nh]: (first piece, pieces + 2^16 row in the piece); 0 pieces: in o_full;
                             // -1: a row that no request holds
  float2* full_ml;           // [T * nh]: (maximum, sum) of o_full's rows
};

// ---- q_lat = q_nope . W_UK ---------------------------------------------------
// A wave keeps 32 latent columns of one head's matrix (32 registers) and
// takes up to 128 tokens in blocks of 32, whose queries come to LDS all at
// once: one trip to memory a workgroup, and the four waves share each row.
// The results go through LDS, so that a token's 128 columns leave as 256
// consecutive bytes. 64 tokens x 128 heads 7.6 us, 256 tokens 16.8 us for 59 MB
// = 3.5 TB/s (queries as 16-byte loads of each wave: 9.5 and 24.7).
constexpr int kAbsorbTok = 128;
constexpr int kAbsorbQ = 32 * kDn * 2;                 // one block's queries
constexpr int kAbsorbRow = 256 + 16;                   // padded: rows 16 bytes apart in the banks
__global__ __launch_bounds__(256) void absorb_kernel(DecodeArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kAbsorbTok / 32 * kAbsorbQ];
  __shared__ __attribute__((aligned(16))) uint8_t out[2][32 * kAbsorbRow];
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.y;
  const int r0 = blockIdx.x * 128;
  const int t_begin = blockIdx.z * kAbsorbTok;
  const int t_end = min(p.T, t_begin + kAbsorbTok);
  const uint16_t* q = p.q + static_cast<int64_t>(t_begin) * p.q_ld + h * kDq;
  for (int t0 = t_begin, k = 0; t0 < t_end; t0 += 32, ++k)
    tile_load<256, 32, 4>(q + 32 * k * p.q_ld, static_cast<uint32_t>(p.q_ld * 2), min(32, t_end - t0),
                          smem + k * kAbsorbQ, wave, lane);
  const uint16_t* w = p.w_uk + (static_cast<int64_t>(h) * kR + r0 + wave * 32) * kDn + lane * 8;
  bf16x8_t wf[8];
#pragma unroll
  for (int s = 0; s < 8; ++s) wf[s] = *reinterpret_cast<const bf16x8_t*>(w + 512 * s);
  uint32_t off[8];
#pragma unroll
  for (int s = 0; s < 8; ++s) off[s] = row_operand_offset<256>(lane, s);
  // rows that no request holds stay marked
  if (blockIdx.x == 0)
    for (int t = t_begin + threadIdx.x; t < t_end; t += 256)
      p.info[static_cast<int64_t>(t) * p.nh + h] = make_int2(0, -1);
  wait_vmcnt<0>();
  lds_barrier();
  int cur = 0;
  for (int t0 = t_begin; t0 < t_end; t0 += 32, cur ^= 1) {
    const uint8_t* qs = smem + (t0 - t_begin) / 32 * kAbsorbQ;
    f32x16_t a = f32x16_t{};
#pragma unroll
    for (int s = 0; s < 8; ++s) a = mfma(wf[s], row_operand(qs, off[s]), a);
    uint8_t* row = out[cur] + (lane & 31) * kAbsorbRow + wave * 64 + 8 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint2*>(row + 16 * i) = pack4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
    lds_barrier();                    // the other buffer's readers are a barrier behind
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * 16 + (threadIdx.x >> 4), c = threadIdx.x & 15;
      if (t0 + r < t_end)
        *reinterpret_cast<u32x4_t*>(p.q_lat + (static_cast<int64_t>(t0 + r) * p.nh + h) * kR + r0 + 8 * c) =
            *reinterpret_cast<const u32x4_t*>(out[cur] + r * kAbsorbRow + 16 * c);
    }
  }
}

// ---- the work list -------------------------------------------------------------
// Sequence b's new tokens and heads are n_q nh rows in ceil(n_q nh / rows)
// row tiles; each row tile has to pass max(1, ceil(len / 64)) token tiles.
// Neighbouring row tiles pass the same cached tokens, so `team` of them are
// taken by as many workgroups of one XCD in step, and share its L2. In the
// order sequence, group of `team` row tiles, token tile, every group is
// kPieceCost + its token tiles long (a group's start and end cost about as
// much as four tiles: queries in, sums out), and the whole is cut into equal
// runs, one for each team. A run's piece of a group is the token tiles in it;
// the part of a run in front of them stands for no work. kPieceCost 0 / 4 / 8:
// 64 ragged requests x 128 heads 95 / 82 / 87 us, long caches x 16 heads 77 /
// 63 / 63, trees of 32 x 128 heads 306 / 291 / 289.
// Little work is not cut to single tiles once there are more than kShortRuns
// units, as every piece is another one to join. Runs of one / two / three
// units, attention and join together: 136 units (7 tokens x 8 heads, 8404
// cached) 35.8 / 30.1 / 29.6 us, 63 units (7 x 16, 3 requests) 26.5 / 28.5 /
// 31, 13 units (1 x 16) 17.1 / 18.7 / 19.9.
struct Seq {
  int q0, nq, len, tok_tiles, units;
};
__device__ __forceinline__ Seq load_seq(const DecodeArgs& p, int b, int rows) {
  Seq s{0, 0, 0, 0, 0};
  if (b < p.B) {
    s.q0 = clamp_int(p.cu_q[b], 0, p.T);
    s.nq = clamp_int(p.cu_q[b + 1], s.q0, p.T) - s.q0;
    s.len = clamp_int(p.lens[b], 0, p.max_pages * p.page_size);
    const int per = rows * p.team;
    s.tok_tiles = s.len > 0 ? (s.len + kTok - 1) / kTok : 1;
    s.units = (s.nq * p.nh + per - 1) / per * (s.tok_tiles + kPieceCost);
  }
  return s;
}
__device__ __forceinline__ int wave_scan(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  return v;
}
// The lanes hold 64 sequences; up to 64 sequences are loaded once.
struct SeqBlock {
  Seq s;
  int sum;         // units up to and with this lane's sequence, within the block
};
__device__ __forceinline__ SeqBlock load_block(const DecodeArgs& p, int b0, int rows) {
  SeqBlock k;
  k.s = load_seq(p, b0 + (threadIdx.x & 63), rows);
  k.sum = wave_scan(k.s.units);
  return k;
}
__device__ __forceinline__ int total_units(const DecodeArgs& p, int rows, const SeqBlock& k0) {
  int n = __builtin_amdgcn_readlane(k0.sum, 63);
  for (int b0 = 64; b0 < p.B; b0 += 64) n += __builtin_amdgcn_readlane(load_block(p, b0, rows).sum, 63);
  return n;
}
// sequence of unit u (u < total): its data and first unit
__device__ __forceinline__ Seq find_unit(const DecodeArgs& p, int rows, const SeqBlock& k0, int u, int& b_out,
                                         int& first) {
  int before = 0;
  Seq r{0, 0, 0, 1, 0};
  b_out = 0;
  first = 0;
  SeqBlock k = k0;
  for (int b0 = 0; b0 < p.B; b0 += 64) {
    if (b0 > 0) k = load_block(p, b0, rows);
    const uint64_t hit = __ballot(before + k.sum > u);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      r.q0 = __builtin_amdgcn_readlane(k.s.q0, l);
      r.nq = __builtin_amdgcn_readlane(k.s.nq, l);
      r.len = __builtin_amdgcn_readlane(k.s.len, l);
      r.tok_tiles = __builtin_amdgcn_readlane(k.s.tok_tiles, l);
      r.units = __builtin_amdgcn_readlane(k.s.units, l);
      b_out = b0 + l;
      first = before + __builtin_amdgcn_readlane(k.sum, l) - r.units;
      return r;
    }
    before += __builtin_amdgcn_readlane(k.sum, 63);
  }
  return r;
}

// zero the bf16 values of a 16-byte piece that are infinite or NaN
__device__ __forceinline__ bool drop_nonfinite(u32x4_t& v) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((v[i] & 0x7F800000u) == 0x7F800000u) v[i] &= 0x0000FFFFu, bad = true;
    if ((v[i] & 0x00007F80u) == 0x00007F80u) v[i] &= 0xFFFF0000u, bad = true;
  }
  return bad;
}

__device__ __forceinline__ void scale_operand(bf16x8_t& v, float f) {
  typedef float f32x8_t __attribute__((ext_vector_type(8)));
  v = __builtin_convertvector(__builtin_convertvector(v, f32x8_t) * f, bf16x8_t);
}

// Workgroup: WR blocks of 32 rows, 2 WR waves. Wave (r, c) holds the queries
// of row block r (144 registers) and scores the 32 tokens of half c of a token
// tile; the weights go through LDS, and every wave multiplies all rows'
// weights with its share of the latent columns (512 / waves; 128 registers of
// sums), so that a value operand read from LDS serves every row block. (32
// rows x all 512 columns a wave would need 400 registers for the kept operands
// alone, and spills; 32 rows x 256 columns reads the values twice.)
// The halves' weights refer to each wave's own running reference; where one
// moved, both are brought to the larger before the product.
constexpr int kXchg = 64 * 32;                        // bytes of one wave's weights
// kRun: every run of kRpw token rows that a wave loads lies in one page, and
// takes one buffer resource (any other page size: one a row, which costs the
// trees of 32 x 128 heads 299 us instead of 291).
template <int WR, bool kRun>
__global__ __launch_bounds__(128 * WR) __attribute__((amdgpu_waves_per_eu(1, 1)))
void decode_attn_kernel(DecodeArgs p) {
  constexpr int NW = 2 * WR;
  constexpr int kRows = 32 * WR;
  constexpr int kRpw = kTok / NW;                     // token rows a wave loads
  constexpr int kCols = kR / NW, kCb = kCols / 32;    // latent columns of a wave, blocks of 32
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kTile + NW * kXchg + NW * 128];
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave >> 1, wc = wave & 1;
  uint8_t* xw = smem + 2 * kTile;
  float* xref = reinterpret_cast<float*>(xw + NW * kXchg);

  const SeqBlock seqs = load_block(p, 0, kRows);
  const int total = total_units(p, kRows, seqs);
  const int teams = kGroups / p.team;
  const int per = max(total > kShortRuns ? 2 : 1, (total + teams - 1) / teams);
  const int grp = xcd_contiguous(blockIdx.x, kGroups);
  const int my_team = grp / p.team, member = grp % p.team;
  int u = my_team * per;
  const int u_end = min(total, u + per);
  const int u_begin = u;

  uint32_t lat_off[8], rope_off[4], v_off[4][2];
#pragma unroll
  for (int s = 0; s < 8; ++s) lat_off[s] = row_operand_offset<1024>(lane, s) + wc * 32 * 1024;
#pragma unroll
  for (int s = 0; s < 4; ++s) rope_off[s] = kLat + row_operand_offset<128>(lane, s) + wc * 32 * 128;
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) v_off[c][h] = col_operand_offset<1024>(lane, c, h) + wave * (kCols * 2);
  const float c2 = p.scale * kLog2e;

  while (u < u_end) {
    int b, first;
    const Seq sq = find_unit(p, kRows, seqs, u, b, first);
    const int len_g = sq.tok_tiles + kPieceCost;
    const int rg = (u - first) / len_g;
    const int x0 = (u - first) - rg * len_g, x1 = min(len_g, x0 + (u_end - u));
    const int kt0 = max(0, x0 - kPieceCost), kt1 = max(0, x1 - kPieceCost);  // token tiles [kt0, kt1)
    const bool whole = kt0 == 0 && kt1 == sq.tok_tiles;
    const int rt = rg * p.team + member;
    const int slot = 2 * grp + (u == u_begin ? 0 : 1);
    u += x1 - x0;
    if (kt0 == kt1) continue;

    const int n_rows = sq.nq * p.nh;
    if (rt * kRows >= n_rows) continue;                         // the last group has fewer row tiles
    const int row = rt * kRows + wr * 32 + (lane & 31);
    const int rowc = min(row, n_rows - 1);
    const int tok = rowc / p.nh;                                // new token of the row
    const int prefix = sq.len - sq.nq;                          // cached tokens before the new ones

    // Page and place of the wave's token rows, lane i: row wave * kRpw + i
    // (rows past the cache's end repeat the last token's: their scores are
    // masked and their values meet weight 0), and from them the row's byte
    // address; apart, so that the page is waited for a tile later.
    int page = 0, place = 0;
    auto find_page = [&](int kt) {
      const int pos = min(kt * kTok + wave * kRpw + (lane & (kRpw - 1)), sq.len - 1);
      const int q = __umulhi(2 * static_cast<uint32_t>(pos), p.page_magic) >> p.page_shift;
      place = pos - q * p.page_size;
      page = p.table[static_cast<int64_t>(b) * p.max_pages + q];
    };
    auto row_address = [&]() -> uint64_t {
      const int slot = clamp_int(page, 0, p.n_pages - 1) * p.page_size + place;
      return reinterpret_cast<uint64_t>(p.cache) + static_cast<uint64_t>(slot) * (kDc * 2);
    };
    // Row i of the wave's share into lds: 64 lanes x 16 bytes. With kRun,
    // `rs` holds the share's valid rows and the others come as zeros; else
    // `addr` the rows' addresses and `bytes` 0 asks for zeros.
    auto load_row = [&](__amdgpu_buffer_rsrc_t rs, uint32_t bytes, uint64_t addr, uint8_t* lds, int i) {
      if constexpr (kRun) {
        lds_load16_buf(rs, ((lane ^ tile_key<1024>(i)) << 4) + i * (kDc * 2), 0, lds + i * 1024);
      } else {
        const uint64_t a = static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<int>(addr), i)) & 0xFFFFFFFFu;
        const uint64_t h = static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<int>(addr >> 32), i)) << 32;
        lds_load16_buf(buf_rsrc(reinterpret_cast<const void*>(h | a), bytes), (lane ^ tile_key<1024>(i)) << 4, 0,
                       lds + i * 1024);                          // kRpw % 16 == 0: key(row) = key(i)
      }
    };
    // the resource of the share's rows in token tile kt
    auto run_rsrc = [&](int kt, uint64_t addr) {
      const uint64_t a = static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<int>(addr), 0)) & 0xFFFFFFFFu;
      const uint64_t h = static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<int>(addr >> 32), 0)) << 32;
      const int n = kt < kt1 ? clamp_int(sq.len - kt * kTok - wave * kRpw, 0, kRpw) : 0;
      // (the same in all lanes; said so, or each load becomes a loop over them)
      const int bytes = __builtin_amdgcn_readfirstlane(n > 0 ? (n - 1) * (kDc * 2) + kR * 2 : 0);
      return buf_rsrc(reinterpret_cast<const void*>(h | a), bytes);
    };
    u32x4_t rope[kRpw / 8];
    auto load_rope = [&](uint64_t addr) {
      typedef const __attribute__((address_space(1))) u32x4_t* gptr;
#pragma unroll
      for (int i = 0; i < kRpw / 8; ++i) {
        const int lr = i * 8 + (lane >> 3);
        const uint32_t a = __shfl(static_cast<int>(addr), lr, 64), h = __shfl(static_cast<int>(addr >> 32), lr, 64);
        const uint64_t src = (static_cast<uint64_t>(h) << 32 | a) + kR * 2 + (lane & 7) * 16;
        rope[i] = *reinterpret_cast<gptr>(src);
      }
    };
    auto put_rope = [&](uint8_t* buf) {
#pragma unroll
      for (int i = 0; i < kRpw / 8; ++i) {
        const int r = wave * kRpw + i * 8 + (lane >> 3);
        *reinterpret_cast<u32x4_t*>(buf + kLat + r * 128 + (((lane & 7) ^ tile_key<128>(r)) << 4)) = rope[i];
      }
    };

    const bool any = sq.len > 0;
    const int w_row = wave * kRpw;                              // first row of the wave's share
    if (any) {
      find_page(kt0);
      const uint64_t a0 = row_address();
      load_rope(a0);
      const __amdgpu_buffer_rsrc_t rs = run_rsrc(kt0, a0);
#pragma unroll
      for (int i = 0; i < kRpw; ++i) load_row(rs, kR * 2, a0, smem + w_row * 1024, i);
      find_page(kt0 + 1);
    }
    // The queries come through the second tile buffer, like cached rows (64
    // or 32 consecutive rows of q_lat, and the rows' rotary parts): read from
    // memory as operands, each load would touch 32 rows.
    bf16x8_t qf[kDc / 16];
    if (any) {
      uint8_t* qb = smem + kTile;
      constexpr int kQr = kRows / NW;                            // rows a wave loads
      const int q_row = wave * kQr;
      const int64_t first_row = static_cast<int64_t>(sq.q0) * p.nh + rt * kRows;
      const int n_valid = __builtin_amdgcn_readfirstlane(clamp_int(n_rows - rt * kRows - q_row, 0, kQr));
      const __amdgpu_buffer_rsrc_t rs = buf_rsrc(p.q_lat + (first_row + q_row) * kR, n_valid * kR * 2);
#pragma unroll
      for (int i = 0; i < kQr; ++i)
        lds_load16_buf(rs, ((lane ^ tile_key<1024>(q_row + i)) << 4) + i * kR * 2, 0, qb + (q_row + i) * 1024);
#pragma unroll
      for (int i = 0; i < kQr / 8; ++i) {
        const int r = q_row + i * 8 + (lane >> 3);
        const int rr = min(rt * kRows + r, n_rows - 1), t = rr / p.nh;
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(
            p.q + (static_cast<int64_t>(sq.q0) + t) * p.q_ld + (rr - t * p.nh) * kDq + kDn + (lane & 7) * 8);
        *reinterpret_cast<u32x4_t*>(qb + kLat + r * 128 + (((lane & 7) ^ tile_key<128>(r)) << 4)) = v;
      }
      wait_vmcnt<0>();
      lds_barrier();
      // lat_off / rope_off are those of token half wc; here the row block is wr
      const int to_block = (wr - wc) * 32;
#pragma unroll
      for (int s = 0; s < 32; ++s)
        qf[s] = row_operand(qb, lat_off[s & 7] + (s >> 3) * 256 + to_block * 1024);
#pragma unroll
      for (int s = 0; s < 4; ++s) qf[32 + s] = row_operand(qb, rope_off[s] + to_block * 128);
    }
    const uint64_t sees = p.tree ? p.tree[sq.q0 + tok] : 0u;
    f32x16_t o[WR][kCb];
    float m[WR], l = 0.f;
#pragma unroll
    for (int r = 0; r < WR; ++r) {
      m[r] = -INFINITY;
#pragma unroll
      for (int c = 0; c < kCb; ++c) {
        o[r][c] = f32x16_t{};
        keep_acc(o[r][c]);
      }
    }

    for (int kt = kt0; any && kt < kt1; ++kt) {
      uint8_t* buf = smem + ((kt - kt0) & 1) * kTile;
      put_rope(buf);                  // the buffer's last readers are a barrier behind
      wait_vmcnt<0>();
      lds_barrier();
      // the next tile's rows (zeros behind the last)
      const uint32_t next_bytes = kt + 1 < kt1 ? kR * 2 : 0;
      const uint64_t next_addr = row_address();
      const __amdgpu_buffer_rsrc_t next_rs = run_rsrc(kt + 1, next_addr);
      uint32_t next_ofs = ((kt + 1 - kt0) & 1) * kTile + w_row * 1024;
      asm volatile("" : "+s"(next_ofs));                        // not one register per row
      const int t0 = kt * kTok;
      // scores: operands read kAhead steps ahead; the next tile's rows are
      // issued while the first operands arrive and between the products
      f32x16_t s = f32x16_t{};
      {
        bf16x8_t a[kAhead];
        auto fetch = [&](auto k_c) {
          constexpr int k = decltype(k_c)::value;
          if constexpr (k < 32) a[k % kAhead] = row_operand(buf, lat_off[k & 7] + (k >> 3) * 256);
          else a[k % kAhead] = row_operand(buf, rope_off[k - 32]);
        };
        static_for<kAhead>([&](auto k_c) { fetch(k_c); });
        load_rope(next_addr);
        static_for<kRpw / 2>([&](auto i_c) { load_row(next_rs, next_bytes, next_addr, smem + next_ofs, decltype(i_c)::value); });
        __builtin_amdgcn_sched_barrier(0);
        static_for<36>([&](auto k_c) {
          constexpr int k = decltype(k_c)::value;
          s = mfma(a[k % kAhead], qf[k], s);
          if constexpr (k + kAhead < 36) fetch(std::integral_constant<int, k + kAhead>{});
          if constexpr (k % 2 == 1 && k / 2 < kRpw / 2)
            load_row(next_rs, next_bytes, next_addr, smem + next_ofs, kRpw / 2 + k / 2);
          __builtin_amdgcn_sched_barrier(0);
        });
        find_page(kt + 2);
      }
      const bool tail = t0 + kTok > prefix;
      if (tail) {
        // the tile holds new tokens (or the end of the cache): bit j of
        // `hide` is place j of the tile
        const int first_new = prefix - t0;                     // may lie outside [0, 64)
        uint64_t hide;
        if (p.tree) {
          hide = first_new <= 0 ? ~uint64_t{0} : ~uint64_t{0} << first_new;
          hide &= ~(first_new >= 0 ? sees << first_new : (first_new > -64 ? sees >> -first_new : 0u));
        } else {
          const int n_shown = first_new + tok + 1;             // places before this one are shown
          hide = n_shown <= 0 ? ~uint64_t{0} : (n_shown < 64 ? ~uint64_t{0} << n_shown : 0u);
        }
        if (sq.len - t0 < kTok) hide |= ~uint64_t{0} << (sq.len - t0);
        const uint32_t w = static_cast<uint32_t>(hide >> (32 * wc)) >> (4 * g);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = (w >> (8 * (i >> 2) + (i & 3))) & 1u ? -INFINITY : s[i];
      }
      float mx = s[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[i]);
      mx = fmaxf(mx, other_half(mx));
      float m_own = m[0];
      if (WR == 2 && wr == 1) m_own = m[WR - 1];
      const float ref = next_ref(m_own, mx, c2);
      // rows that have seen no key yet keep -inf: exponents against 0
      const float rc = ref == -INFINITY ? 0.f : ref * c2;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = exp2_hw(fmaf(s[i], c2, -rc));
        sum += s[i];
      }
      bf16x8_t pf[WR][4];             // [row block][k-step of 16 tokens]
#pragma unroll
      for (int k = 0; k < 2; ++k)
        *reinterpret_cast<bf16x8_t*>(xw + wave * kXchg + k * 1024 + lane * 16) = pack_operand(s, k);
      if (g == 0) xref[wave * 32 + lane] = ref;
      constexpr int kN = 4 * kCb;     // value operands: k-step of 16 tokens, column block
      bf16x8_t va[kAhead];
      auto fetch_v = [&](auto n_c) {
        constexpr int n = decltype(n_c)::value, k = n / kCb, c = n % kCb;
        va[n % kAhead] = col_operand(buf, v_off[c & 3][0] + (c >> 2) * 256 + k * 16 * 1024,
                                     v_off[c & 3][1] + (c >> 2) * 256 + k * 16 * 1024);
      };
      static_for<kAhead>([&](auto n_c) { fetch_v(n_c); });
      lds_barrier();
      if (tail && (p.tree || sq.nq > 1)) {
        // a hidden token's row is still in the value product, with weight 0:
        // values that are not finite must not reach it (rows that see the
        // token have them in their scores already, as NaN, or with the whole
        // weight, or as -inf, which takes no weight)
        for (int i = threadIdx.x; i < kLat / 16; i += 64 * NW) {
          u32x4_t v = *reinterpret_cast<const u32x4_t*>(buf + i * 16);
          if (drop_nonfinite(v)) *reinterpret_cast<u32x4_t*>(buf + i * 16) = v;
        }
        lds_barrier();
        static_for<kAhead>([&](auto n_c) { fetch_v(n_c); });
      }
#pragma unroll
      for (int r = 0; r < WR; ++r) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          pf[r][k] = *reinterpret_cast<const bf16x8_t*>(xw + (2 * r + k / 2) * kXchg + (k % 2) * 1024 + lane * 16);
        const float ref0 = xref[2 * r * 32 + (lane & 31)], ref1 = xref[(2 * r + 1) * 32 + (lane & 31)];
        const float mn = fmaxf(ref0, ref1);
        if (__any(mn > m[r])) {
          const float mc = mn == -INFINITY ? 0.f : mn * c2;
          const float a = exp2_hw(fmaf(m[r], c2, -mc));
          const float f0 = exp2_hw(fmaf(ref0, c2, -mc)), f1 = exp2_hw(fmaf(ref1, c2, -mc));
          if (r == wr) {
            l *= a;
            sum *= wc == 0 ? f0 : f1;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) scale_operand(pf[r][k], k < 2 ? f0 : f1);
#pragma unroll
          for (int c = 0; c < kCb; ++c) {
#pragma unroll
            for (int i = 0; i < 16; ++i) o[r][c][i] = read_acc(o[r][c][i]) * a;
            keep_acc(o[r][c]);
          }
          m[r] = mn;
        }
      }
      l += sum;
      __builtin_amdgcn_sched_barrier(0);
      static_for<kN>([&](auto n_c) {
        constexpr int n = decltype(n_c)::value, k = n / kCb, c = n % kCb;
#pragma unroll
        for (int r = 0; r < WR; ++r) o[r][c] = mfma(va[n % kAhead], pf[r][k], o[r][c]);
        if constexpr (n + kAhead < kN) fetch_v(std::integral_constant<int, n + kAhead>{});
        __builtin_amdgcn_sched_barrier(0);
      });
#pragma unroll
      for (int r = 0; r < WR; ++r)
#pragma unroll
        for (int c = 0; c < kCb; ++c) keep_acc(o[r][c]);
    }
    acc_settled();
    wait_vmcnt<0>();                  // the zeros behind the last tile have arrived
    l += other_half(l);
    lds_barrier();                    // everyone is done with the buffers
    if (g == 0) xref[wave * 32 + lane] = l;
    lds_barrier();
    float lr[WR];                     // of every row block, added in the same order in all waves
#pragma unroll
    for (int r = 0; r < WR; ++r) lr[r] = xref[2 * r * 32 + (lane & 31)] + xref[(2 * r + 1) * 32 + (lane & 31)];
    lds_barrier();
    // The sums leave through LDS (each wave its own part of the tile
    // buffers), so that a row's columns are written as consecutive bytes: from
    // the registers, every store would touch 32 rows, and that took longer
    // than several token tiles.
    constexpr int kRowB = kCols * 4 + 16;
    static_assert(NW * kRows * kRowB <= 2 * kTile, "sums fit the tile buffers");
    uint8_t* ob = smem + wave * kRows * kRowB;
#pragma unroll
    for (int r = 0; r < WR; ++r)
#pragma unroll
      for (int c = 0; c < kCb; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<f32x4_t*>(ob + (r * 32 + (lane & 31)) * kRowB + (32 * c + 8 * i + 4 * g) * 4) =
              f32x4_t{read_acc(o[r][c][4 * i]), read_acc(o[r][c][4 * i + 1]), read_acc(o[r][c][4 * i + 2]),
                      read_acc(o[r][c][4 * i + 3])};
    const int64_t row0 = static_cast<int64_t>(sq.q0) * p.nh + rt * kRows;       // first row in o_full
    const int64_t part0 = static_cast<int64_t>(slot) * kRows;
    const int n_out = min(kRows, n_rows - rt * kRows);
    float* dst = (whole ? p.o_full + row0 * kR : p.part + part0 * kR) + wave * kCols;
    constexpr int kLpr = kCols / 4;                            // lanes a row
#pragma unroll 8
    for (int r0 = 0; r0 < kRows; r0 += 64 / kLpr) {
      const int r = r0 + lane / kLpr, c = lane % kLpr;
      if (r < n_out)
        *reinterpret_cast<f32x4_t*>(dst + static_cast<int64_t>(r) * kR + 4 * c) =
            *reinterpret_cast<const f32x4_t*>(ob + r * kRowB + 16 * c);
    }
    if (wave == 0 && g == 0) {
#pragma unroll
      for (int r = 0; r < WR; ++r) {
        const int lr_ = r * 32 + lane;
        if (lr_ >= n_out) continue;
        *(whole ? p.full_ml + row0 + lr_ : p.part_ml + part0 + lr_) = make_float2(m[r], lr[r]);
        if (kt0 == 0) {
          // pieces of the row tile: this one and one of each following team
          // up to the one that holds the last token tile
          const int last_unit = first + (rg + 1) * len_g - 1;
          const int n = whole ? 0 : last_unit / per - my_team + 1;
          p.info[row0 + lr_] = make_int2(slot, n | lr_ << 16);
        }
      }
    }
    lds_barrier();                    // before the next piece's tiles
  }
}

// ---- join the pieces, out = W_UV . o_lat --------------------------------------
// A workgroup takes one head of `toks` tokens (up to 32; fewer when there are
// few, so that the pieces' rows are read by enough workgroups). A wave joins
// the pieces of TPW tokens side by side (below 4 tokens several waves share
// one token's pieces in turn and their sums are added after), in an order that
// depends on the sizes alone, and puts the rows into LDS as two bf16 terms (16
// significant bits, so the product adds no rounding of its own); then each
// wave computes 32 of the 128 value columns. Pieces, conversion, barrier, W_UV
// and products follow one another: 42 us for 84 MB = 2 TB/s (256 tokens x 128
// heads). With TPW 8, 56 scalar values live in vector lanes (6 with TPW 4).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

template <int TPW>
__global__ __launch_bounds__(256) void decode_join_kernel(DecodeArgs p, int rows, int toks) {
  constexpr int kTokMax = 4 * TPW;
  constexpr int kUnroll = 8 / TPW;                     // pieces of a token read at once
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kTokMax * kR * 2];
  __shared__ float sums[TPW == 1 ? 4 : 1][kR];
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.x, t0 = blockIdx.y * toks;
  const float c2 = p.scale * kLog2e;
  const int share = toks >= 4 ? 1 : 4 / toks;          // waves of one token
  const int sub = wave % share;

  // What does not depend on another load is asked for at once: the rows'
  // pieces (info), and their whole rows in case that is what they have (else
  // what o_full holds there is not used). Token i of the wave is row
  // wave / share + 4 i.
  int64_t grow[TPW];
  float v[TPW][8], m[TPW], l[TPW];
  float2 ml[TPW];
#pragma unroll
  for (int i = 0; i < TPW; ++i)
    grow[i] = static_cast<int64_t>(min(t0 + wave / share + 4 * i, p.T - 1)) * p.nh + h;
  const int2 info = p.info[static_cast<int64_t>(min(t0 + wave / share + 4 * (lane & (TPW - 1)), p.T - 1)) * p.nh + h];
#pragma unroll
  for (int i = 0; i < TPW; ++i) {
    ml[i] = p.full_ml[grow[i]];
    load8_f32(p.o_full + grow[i] * kR + 8 * lane, v[i]);
  }
  int n[TPW], slot0[TPW], lr[TPW];
  bool held[TPW];
  int n_max = 0;
#pragma unroll
  for (int i = 0; i < TPW; ++i) {
    const int y = __builtin_amdgcn_readlane(info.y, i);
    held[i] = y >= 0 && t0 + wave / share + 4 * i < min(t0 + toks, p.T);
    slot0[i] = clamp_int(__builtin_amdgcn_readlane(info.x, i), 0, 2 * kGroups - 1);
    n[i] = held[i] ? clamp_int(y & 0xFFFF, 0, kGroups) : 0;
    lr[i] = clamp_int(y >> 16, 0, rows - 1);
    n_max = max(n_max, n[i]);
  }

  // row of a piece in part / part_ml: the first piece may be its workgroup's
  // second, the others are the first of the same member of the teams after it
  auto piece = [&](int i, int j) -> int64_t {
    const int s = j == 0 ? slot0[i] : min(2 * (slot0[i] / 2 + j * p.team), 2 * kGroups - 1);
    return static_cast<int64_t>(s) * rows + lr[i];
  };
  auto load_ml = [&](int i, int j) {
    return j < n[i] ? p.part_ml[piece(i, j)] : make_float2(-INFINITY, 0.f);
  };
  // the first pieces' rows are asked for along with the pieces' statistics
  float x[kUnroll][TPW][8];
  auto load_rows = [&](int j0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        const int k = j0 + u * share;
        if (k < n[i]) load8_f32(p.part + piece(i, k) * kR + 8 * lane, x[u][i]);
      }
  };
#pragma unroll
  for (int i = 0; i < TPW; ++i)
    if (n[i] > 0) ml[i] = load_ml(i, lane);
  load_rows(sub);
#pragma unroll
  for (int i = 0; i < TPW; ++i) {
    m[i] = ml[i].x;
    l[i] = ml[i].y;
    if (n[i] > 0) {
      for (int j = 64 + lane; j < n[i]; j += 64) m[i] = fmaxf(m[i], load_ml(i, j).x);
      m[i] = wave_max(m[i]);
      l[i] = 0.f;
    }
    // a whole row counts once where several waves share a token
    const bool keep = n[i] == 0 && sub == 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = keep ? v[i][e] : 0.f;
  }
  for (int c0 = 0; c0 < n_max; c0 += 64) {
    float a[TPW];                                      // weight of piece c0 + lane
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      if (n[i] == 0) continue;
      if (c0 > 0) ml[i] = load_ml(i, c0 + lane);
      a[i] = exp2_hw(fmaf(ml[i].x, c2, m[i] == -INFINITY ? 0.f : -m[i] * c2));
      l[i] += wave_sum(ml[i].y * a[i]);
    }
    const int c_end = min(64, n_max - c0);
    for (int j = sub; j < c_end; j += kUnroll * share) {
      if (c0 + j != sub) load_rows(c0 + j);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int i = 0; i < TPW; ++i) {
          const int k = j + u * share;
          if (k >= 64 || c0 + k >= n[i]) continue;
          const float f = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(a[i]), k));
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = fmaf(x[u][i][e], f, v[i][e]);
        }
    }
  }
  // the matrix, behind the pieces (loads return in order)
  constexpr int kW = TPW <= 4 ? 32 : 16;
  const uint16_t* w = p.w_uv + (static_cast<int64_t>(h) * kDv + wave * 32) * kR + lane * 8;
  bf16x8_t wf[kW];
#pragma unroll
  for (int s = 0; s < kW; ++s) wf[s] = *reinterpret_cast<const bf16x8_t*>(w + 512 * s);
  if constexpr (TPW == 1) {
    if (share > 1) {
      store8_f32(&sums[wave][8 * lane], v[0]);
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) v[0][e] = 0.f;
      for (int q = 0; q < share; ++q) {
        float x[8];
        load8_f32(&sums[wave - sub + q][8 * lane], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[0][e] += x[e];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < TPW; ++i) {
    const int r = wave / share + 4 * i;
    const float f = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);
    if (p.lse && held[i] && lane == 0 && sub == 0)
      p.lse[grow[i]] = l[i] == 0.f ? -INFINITY : fmaf(m[i], p.scale, log2_hw(l[i]) * kLn2);
    typedef float f32x8_t __attribute__((ext_vector_type(8)));
    const f32x8_t x = f32x8_t{v[i][0], v[i][1], v[i][2], v[i][3], v[i][4], v[i][5], v[i][6], v[i][7]} * f;
    const bf16x8_t a = __builtin_convertvector(x, bf16x8_t);
    const bf16x8_t b = __builtin_convertvector(x - __builtin_convertvector(a, f32x8_t), bf16x8_t);
    const uint32_t o = r * 1024 + ((lane ^ tile_key<1024>(r)) << 4);
    if (sub == 0 && r < kTokMax) {
      *reinterpret_cast<bf16x8_t*>(smem + o) = a;
      *reinterpret_cast<bf16x8_t*>(smem + kTokMax * 1024 + o) = b;
    }
  }
  __syncthreads();
  // token columns past the workgroup's repeat others and are not stored
  const int col = lane & 31, src = col & (kTokMax - 1);
  f32x16_t acc = f32x16_t{};
  static_for<32>([&](auto k_c) {
    constexpr int k = decltype(k_c)::value;
    const uint32_t o = src * 1024 + (((2 * (k & 7) + g) ^ tile_key<1024>(src)) << 4) + (k >> 3) * 256;
    acc = mfma(wf[k % kW], row_operand(smem, o), acc);
    acc = mfma(wf[k % kW], row_operand(smem + kTokMax * 1024, o), acc);
    if constexpr (k + kW < 32) wf[k % kW] = *reinterpret_cast<const bf16x8_t*>(w + 512 * (k + kW));
  });
  const int t = t0 + col;
  if (col >= toks || t >= p.T || p.info[static_cast<int64_t>(t) * p.nh + h].y < 0) return;
  uint16_t* o = p.out + static_cast<int64_t>(t) * p.out_ld + h * kDv + wave * 32 + 4 * g;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint2*>(o + 8 * i) = pack4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
}

constexpr int kJoinTok = 32;
// Tokens of a joining workgroup: more share a head's matrix, fewer join more
// pieces at once. As many as leave two workgroups a compute unit; always 32:
// 12 instead of 6.7 us (1 token x 16 heads), 44 instead of 9 (21), 77 instead
// of 14.5 (8 long caches); at most 16: 47 instead of 41 (256 x 128 heads).
int join_tokens(int T, int nh) {
  int n = kJoinTok;
  while (n > 1 && static_cast<int64_t>((T + n - 1) / n) * nh < 2 * kNumCu) n /= 2;
  return n;
}

// Row tiles taken in step by as many workgroups: the largest power of two (at
// most the 32 workgroups of an XCD) that leaves no more than a sixth of the
// places empty for a request of average size. Each by itself: 336 instead of
// 291 us (trees of 32 x 128 heads), 85 instead of 82 (one token x 128 heads).
int team_size(int64_t T, int B, int nh, int rows) {
  const int64_t tiles = ((T * nh + B - 1) / B + rows - 1) / rows;
  int n = kGroups / kNumXcd;
  while (n > 1 && (n > tiles || 6 * tiles < 5 * ((tiles + n - 1) / n * n))) n /= 2;
  return n;
}

// Rows of a row tile, by the new rows a request brings on average. 32 where
// 64 are taken: 121 instead of 82 us (one token x 128 heads), 485 instead of
// 291 (32 x 128), the same at 7 x 16; 64 where 32 are taken: 11.3 instead of
// 10.0 (one token x 16 heads), 67 instead of 63 (long caches).
int tile_rows(int64_t T, int B, int nh) {
  const int64_t avg = (T * nh + B - 1) / B;
  return avg <= 32 ? 32 : 64;
}

struct Layout {
  size_t q_lat, o_full, part, part_ml, info, full_ml, total;
};
Layout layout(int64_t T, int nh) {
  auto up = [](size_t v) { return (v + 255) & ~size_t{255}; };
  const size_t n = static_cast<size_t>(T) * nh;
  const size_t rows = n <= 32 ? 32 : 64;   // whatever B is
  Layout l;
  l.q_lat = 0;
  l.o_full = up(n * kR * 2);
  l.part = l.o_full + up(n * kR * 4);
  l.part_ml = l.part + 2 * kGroups * rows * kR * 4;
  l.info = l.part_ml + 2 * kGroups * rows * 8;
  l.full_ml = l.info + up(n * 8);
  l.total = l.full_ml + up(n * 8);
  return l;
}

}  // namespace
}  // namespace mla
}  // namespace moe

extern "C" size_t moe_mla_decode_workspace(int T, int n_heads) {
  if (T < 0 || n_heads < 1 || n_heads > 1024 || static_cast<int64_t>(T) * n_heads > (1 << 24)) return 0;
  return moe::mla::layout(T, n_heads).total;
}

extern "C" int moe_mla_decode(const void* q, int64_t q_ld, const void* w_uk, const void* w_uv, int fmt,
                              const void* cache, int page_size, int n_pages, const int32_t* page_table,
                              int max_pages, const int32_t* lens, const int32_t* cu_q, const int64_t* tree_mask,
                              int B, int T, int n_heads, float scale, void* out, int64_t out_ld, float* lse, void* ws,
                              size_t ws_bytes, hipStream_t stream) {
  using namespace moe;
  using namespace moe::mla;
  clear_error();
  MOE_REQUIRE(B >= 0 && B <= (1 << 16) && T >= 0, MOE_ERR_INVALID_ARG,
              "moe_mla_decode: need 0 <= B <= 65536 and T >= 0");
  MOE_REQUIRE(n_heads >= 1 && n_heads <= 1024 && static_cast<int64_t>(T) * n_heads <= (1 << 24), MOE_ERR_INVALID_ARG,
              "moe_mla_decode: n_heads must be in [1, 1024], T * n_heads <= 2^24");
  MOE_REQUIRE(fmt == MOE_BF16, MOE_ERR_UNSUPPORTED, "moe_mla_decode: fmt must be MOE_BF16");
  MOE_REQUIRE(page_size >= 1 && n_pages >= 1 && max_pages >= 1 &&
                  static_cast<int64_t>(page_size) * n_pages < (int64_t{1} << 31) &&
                  static_cast<int64_t>(page_size) * max_pages < (int64_t{1} << 31),
              MOE_ERR_INVALID_ARG,
              "moe_mla_decode: page_size, n_pages and max_pages must be >= 1, their products below 2^31");
  MOE_REQUIRE(scale > 0.f && scale <= kMaxScale, MOE_ERR_INVALID_ARG,
              "moe_mla_decode: scale must be in (0, 2.3e38]");
  MOE_REQUIRE(q_ld >= static_cast<int64_t>(n_heads) * kDq && out_ld >= static_cast<int64_t>(n_heads) * kDv &&
                  q_ld <= kMaxLd && out_ld <= kMaxLd,
              MOE_ERR_INVALID_ARG, "moe_mla_decode: a row stride is smaller than its row or above 2^23 elements");
  MOE_REQUIRE(q_ld % 8 == 0 && out_ld % 8 == 0, MOE_ERR_ALIGNMENT,
              "moe_mla_decode: row strides must be multiples of 8 elements");
  if (B == 0 || T == 0) return MOE_OK;
  const int rows = tile_rows(T, B, n_heads);
  const int64_t tiles = static_cast<int64_t>(T) * n_heads / rows + B;
  MOE_REQUIRE(tiles * ((static_cast<int64_t>(page_size) * max_pages + kTok - 1) / kTok + kPieceCost) < (int64_t{1} << 30),
              MOE_ERR_INVALID_ARG, "moe_mla_decode: too much work for one call (row tiles x cached tiles >= 2^30)");
  MOE_REQUIRE(q && w_uk && w_uv && cache && page_table && lens && cu_q && out, MOE_ERR_INVALID_ARG,
              "moe_mla_decode: null pointer");
  MOE_REQUIRE(aligned16(q) && aligned16(w_uk) && aligned16(w_uv) && aligned16(cache) && aligned16(out) &&
                  aligned16(ws),
              MOE_ERR_ALIGNMENT, "moe_mla_decode: tensors and ws must be 16-byte aligned");
  const Layout l = layout(T, n_heads);
  MOE_REQUIRE(ws && ws_bytes >= l.total, MOE_ERR_WORKSPACE,
              "moe_mla_decode: ws smaller than moe_mla_decode_workspace(T, n_heads)");
  uint8_t* w = static_cast<uint8_t*>(ws);
  DecodeArgs a{};
  a.q = static_cast<const uint16_t*>(q), a.q_ld = q_ld;
  a.w_uk = static_cast<const uint16_t*>(w_uk), a.w_uv = static_cast<const uint16_t*>(w_uv);
  a.cache = static_cast<const uint16_t*>(cache);
  a.page_size = page_size, a.n_pages = n_pages, a.table = page_table, a.max_pages = max_pages;
  int shift = 0;
  while ((int64_t{1} << shift) < page_size) ++shift;
  a.page_shift = shift;
  a.page_magic = static_cast<uint32_t>(((uint64_t{1} << (31 + shift)) + page_size - 1) / page_size);
  a.lens = lens, a.cu_q = cu_q, a.tree = reinterpret_cast<const uint64_t*>(tree_mask);
  a.B = B, a.T = T, a.nh = n_heads, a.scale = scale;
  a.out = static_cast<uint16_t*>(out), a.out_ld = out_ld, a.lse = lse;
  a.q_lat = reinterpret_cast<uint16_t*>(w + l.q_lat);
  a.o_full = reinterpret_cast<float*>(w + l.o_full);
  a.part = reinterpret_cast<float*>(w + l.part);
  a.part_ml = reinterpret_cast<float2*>(w + l.part_ml);
  a.info = reinterpret_cast<int2*>(w + l.info);
  a.full_ml = reinterpret_cast<float2*>(w + l.full_ml);
  a.team = team_size(T, B, n_heads, rows);
  const int toks = join_tokens(T, n_heads);
  hipLaunchKernelGGL(absorb_kernel, dim3(kR / 128, n_heads, (T + kAbsorbTok - 1) / kAbsorbTok), dim3(256), 0, stream,
                     a);
  auto attend = [&](auto kern, int waves) {
    hipLaunchKernelGGL(kern, dim3(kGroups), dim3(64 * waves), 0, stream, a);
  };
  if (rows == 32) {
    if (page_size % 32 == 0) attend(decode_attn_kernel<1, true>, 2);
    else attend(decode_attn_kernel<1, false>, 2);
  } else {
    if (page_size % 16 == 0) attend(decode_attn_kernel<2, true>, 4);
    else attend(decode_attn_kernel<2, false>, 4);
  }
  auto join = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(n_heads, (T + toks - 1) / toks), dim3(256), 0, stream, a, rows, toks);
  };
  if (toks <= 4) join(decode_join_kernel<1>);
  else if (toks == 8) join(decode_join_kernel<2>);
  else if (toks == 16) join(decode_join_kernel<4>);
  else join(decode_join_kernel<8>);
  return check_launch("moe_mla_decode");
}
