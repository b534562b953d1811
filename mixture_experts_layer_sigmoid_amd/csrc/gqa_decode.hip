// moe_gqa_decode: attention of the last tokens of B requests over the 8-bit
// paged cache, grouped heads.
//
// Per new token t, query head h, with the cache's codes times their scales:
//   s[j] = scale * q[t, h] . k_j,  p = softmax(s),  out[t, h] = sum_j p_j v_j
// over the tokens that it sees. The group's heads of a request's new tokens
// are the packed rows of one product over the head's cache, 32 at a time.
//
// Two launches. Attention: the cached tokens of each (request, key head, 32
// rows) are cut into pieces of about equal length, one workgroup each, whose
// four waves take 32 tokens in turn. A wave reads keys and values straight
// into registers (the cache lies in operand order), a tile ahead of its
// products, and turns codes into bf16 operands with the block's scale in the
// same instruction, exactly. So nothing passes LDS and no wave waits for
// another before the piece's end, where the four sums are added in order. The
// join adds the pieces in order; a row that one piece covers is stored at once.
//
// Roundings: the weights to bf16 as operands (their sum is taken before that).
// Codes times scales are exact in bf16; scores and all sums are fp32.
#include "gqa_cache.h"

#include <cmath>

namespace moe {
namespace gqa {
namespace {

constexpr int kTok = 32;                               // cached tokens a tile
constexpr int NW = 4;                                  // waves a workgroup
constexpr int kRows = 32;                              // packed rows a workgroup
constexpr int kPieces = 512;                           // pieces beside one a (request, head, rows)
constexpr int kLeast = NW;                             // tiles a piece, at least

struct DecodeArgs {
  const uint16_t* q;
  int64_t q_ld;
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  int n_pages;
  Div bpp;                   // blocks per page
  const int32_t* table;
  int max_pages;
  const int32_t* lens;
  const int32_t* cu_q;
  const uint64_t* tree;
  int B, T, nh, nkv;
  Div g;
  float scale;
  uint16_t* out;
  int64_t out_ld;
  float* lse;
  float* part;               // [workgroups, 32, D]: pieces, not normalized
  float2* part_ml;           // [workgroups, 32]: their (reference, sum)
  int wgs;                   // workgroups that part has room for
};

// A request's part of the work.
struct Seg {
  int b;                     // -1: none
  int start, n_q, len;       // rows of q, new tokens, cached tokens
  int tiles, pieces;         // of a (head, 32 rows)
  int row_tiles;
  int rest;                  // workgroup (or segment) within the request
  int first;                 // first workgroup of the request
};

// What each lane knows of one request.
__device__ __forceinline__ void request(const DecodeArgs& p, int b, int* start, int* n_q, int* len, int* tiles,
                                        int* row_tiles) {
  *start = *n_q = *len = *tiles = *row_tiles = 0;
  if (b >= p.B) return;
  const int a0 = p.cu_q[b], a1 = p.cu_q[b + 1], n = p.lens[b];
  *start = clamp_int(a0, 0, p.T);
  *n_q = clamp_int(a1, *start, p.T) - *start;
  *len = clamp_int(n, 0, p.max_pages * p.bpp.d * kBlock);
  *tiles = (*len + kTok - 1) / kTok;
  *row_tiles = (*n_q * p.g.d + kRows - 1) / kRows;
}

// Tiles of a piece: all tiles over kPieces workgroups, at least kLeast.
__device__ __forceinline__ int piece_tiles(const DecodeArgs& p) {
  const int lane = threadIdx.x & 63;
  int64_t all = 0;
  for (int b0 = 0; b0 < p.B; b0 += 64) {
    int s, n, len, tiles, rt;
    request(p, b0 + lane, &s, &n, &len, &tiles, &rt);
    all += static_cast<int64_t>(tiles) * rt * p.nkv;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) all += __shfl_xor(all, o, 64);
  const int64_t c = (all + kPieces - 1) / kPieces;
  return c > kLeast ? static_cast<int>(c < (1 << 30) ? c : (1 << 30)) : kLeast;
}

// Workgroup `index` (by_piece) or segment (request, head, rows) `index` of the
// call. The pieces of a request run slowest, its 32-row tiles fastest, so
// neighbours read the same tokens.
__device__ __forceinline__ Seg find_work(const DecodeArgs& p, int index, bool by_piece) {
  const int lane = threadIdx.x & 63;
  const int c = piece_tiles(p);
  int64_t before = 0, wgs = 0;
  for (int b0 = 0; b0 < p.B; b0 += 64) {
    int s, n, len, tiles, rt;
    request(p, b0 + lane, &s, &n, &len, &tiles, &rt);
    const int pieces = tiles > c ? (tiles + c - 1) / c : 1;
    const int seg = rt * p.nkv, groups = seg * pieces, count = by_piece ? groups : seg;
    int sum = count, gsum = groups;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(sum, o, 64), w = __shfl_up(gsum, o, 64);
      if (lane >= o) sum += u, gsum += w;
    }
    const uint64_t hit = __ballot(before + sum > index);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      Seg r;
      r.b = b0 + l;
      r.start = __builtin_amdgcn_readlane(s, l);
      r.n_q = __builtin_amdgcn_readlane(n, l);
      r.len = __builtin_amdgcn_readlane(len, l);
      r.tiles = __builtin_amdgcn_readlane(tiles, l);
      r.pieces = __builtin_amdgcn_readlane(pieces, l);
      r.row_tiles = __builtin_amdgcn_readlane(rt, l);
      r.rest = static_cast<int>(index - before) - (__builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(count, l));
      r.first = static_cast<int>(wgs) + __builtin_amdgcn_readlane(gsum, l) - __builtin_amdgcn_readlane(groups, l);
      return r;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
    wgs += __builtin_amdgcn_readlane(gsum, 63);
  }
  return Seg{-1, 0, 0, 0, 0, 0, 0, 0, 0};
}

// 8 codes times a scale as a bf16 operand
__device__ __forceinline__ bf16x8_t operand8(uint32_t lo, uint32_t hi, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// bit 7 of each byte that is a NaN code (0x7F, 0xFF): with the sign bit away
// only 0x7F carries into bit 7 when 1 is added
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}
__device__ __forceinline__ float scale_of(int byte) { return __uint_as_float(static_cast<uint32_t>(byte) << 23); }

template <int D>
constexpr int join_row() { return D + 4; }             // floats; padded against bank conflicts
template <int D>
constexpr int smem_bytes() { return (NW * kRows * join_row<D>() + 2 * NW * kRows) * 4; }

template <int D>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2)))
void decode_kernel(DecodeArgs p) {
  constexpr int S = D / 32, C = D / 32;                // key loads of 16 bytes, value blocks of 32
  __shared__ __attribute__((aligned(16))) float smem[smem_bytes<D>() / 4];
  const int lane = threadIdx.x & 63, g = lane >> 5, r32 = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Seg sg = find_work(p, blockIdx.x, true);
  if (sg.b < 0) return;
  const int rt = sg.rest % sg.row_tiles;
  const int hp = sg.rest / sg.row_tiles;
  const int head = hp % p.nkv, piece = hp / p.nkv;
  const int t_begin = static_cast<int>(static_cast<int64_t>(sg.tiles) * piece / sg.pieces);
  const int t_end = static_cast<int>(static_cast<int64_t>(sg.tiles) * (piece + 1) / sg.pieces);
  const int n_rows = sg.n_q * p.g.d;
  const int row = rt * kRows + r32;
  const int rowc = row < n_rows ? row : n_rows - 1;
  const int tok = quot(rowc, p.g), sub = rowc - tok * p.g.d;
  const int first_new = sg.len - sg.n_q;               // position of new token 0
  const int h = head * p.g.d + sub;

  // this wave's tiles are t_begin + wave + NW i; lane l keeps the place and
  // the scales of block l % 2 of tile l / 2 of the next 32 of them
  const int n_mine = t_begin + wave < t_end ? (t_end - t_begin - wave + NW - 1) / NW : 0;
  int place = 0, scales = 0;
  auto look_up = [&](int i0) {
    const int tile = t_begin + wave + NW * (i0 + (lane >> 1));
    const int blk = 2 * tile + (lane & 1);
    place = 0, scales = 127 | 127 << 8;                // a block without tokens: scale 1
    if (tile < t_end && blk * kBlock < sg.len) {
      const int col = quot(blk, p.bpp);
      const int page = clamp_int(p.table[static_cast<int64_t>(sg.b) * p.max_pages + col], 0, p.n_pages - 1);
      place = (page * p.nkv + head) * p.bpp.d + (blk - col * p.bpp.d);
      scales = p.k_scales[place] | p.v_scales[place] << 8;
    }
  };
  u32x4_t kr[S], vr[2][S / 2];
  auto load = [&](int i) {                             // tile i of this wave
    const int l = 2 * (i & 31);
    const int64_t b0 = static_cast<int64_t>(__builtin_amdgcn_readlane(place, l)) * (kBlock * D);
    const int64_t b1 = static_cast<int64_t>(__builtin_amdgcn_readlane(place, l + 1)) * (kBlock * D);
    const uint8_t* k = p.k + ((lane & 16) ? b1 : b0) + g * 256 + (lane & 15) * 16;
#pragma unroll
    for (int s = 0; s < S; ++s) kr[s] = *reinterpret_cast<const u32x4_t*>(k + s * 512);
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int j = 0; j < S / 2; ++j)
        vr[b][j] = *reinterpret_cast<const u32x4_t*>(p.v + (b ? b1 : b0) + j * 1024 + r32 * 32 + g * 16);
  };
  if (n_mine > 0) {
    look_up(0);
    load(0);
  }
  bf16x8_t qf[2 * S];
  {
    const uint16_t* q = p.q + (static_cast<int64_t>(sg.start) + tok) * p.q_ld + h * D + 16 * g;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) qf[2 * s + i] = *reinterpret_cast<const bf16x8_t*>(q + 32 * s + 8 * i);
  }
  const uint64_t word = p.tree ? p.tree[sg.start + tok] : 0;
  const int n_bits = min(64, sg.n_q);
  // whether the lane's row sees the token of accumulator row x of a tile
  auto visible = [&](int t0, int x) {
    const int j = t0 + 8 * (x >> 2) + 4 * g + (x & 3) - first_new;
    const int by_tree = static_cast<int>(word >> (j & 63)) & static_cast<int>(j < n_bits);
    return (j < 0) | static_cast<bool>(p.tree ? by_tree & 1 : static_cast<int>(j <= tok));
  };
  f32x16_t o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = f32x16_t{};
  float m = -INFINITY, l = 0.f;
  const float c2 = p.scale * kLog2e;

  for (int i = 0; i < n_mine; ++i) {
    const int t0 = (t_begin + wave + NW * i) * kTok;
    const int sc0 = __builtin_amdgcn_readlane(scales, 2 * (i & 31));
    const int sc1 = __builtin_amdgcn_readlane(scales, 2 * (i & 31) + 1);
    const float ks = scale_of(((lane & 16) ? sc1 : sc0) & 255);
    const float vs[2] = {scale_of(sc0 >> 8), scale_of(sc1 >> 8)};
    // codes behind the last token may be anything: as keys they are masked
    // below, as values they have to be finite beside weights of 0
    if (t0 + kTok > sg.len) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int n = sg.len - (t0 + 16 * b + 8 * w + 4 * g);
          const uint32_t keep = n >= 4 ? ~0u : (n <= 0 ? 0u : (1u << (8 * n)) - 1);
#pragma unroll
          for (int j = 0; j < S / 2; ++j) vr[b][j][w] &= keep, vr[b][j][2 + w] &= keep;
        }
    }
    // A NaN among the values of tokens that some rows see and others do not: it
    // is taken out of the product, where a weight of 0 would spread it, and put
    // into the sums of the rows that see it.
    if (t0 + kTok > first_new) {
      uint32_t bad = 0;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int j = 0; j < S / 2; ++j)
#pragma unroll
          for (int w = 0; w < 4; ++w) bad |= nan_bytes(vr[b][j][w]);
      if (__any(bad != 0)) {
        bf16x8_t seen[2];
#pragma unroll
        for (int x = 0; x < 16; ++x) seen[x >> 3][x & 7] = static_cast<__bf16>(visible(t0, x) ? 1.f : 0.f);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          f32x16_t n = {};
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            bf16x8_t is;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t codes = vr[b][c / 2][2 * (c % 2) + w], nan = nan_bytes(codes);
#pragma unroll
              for (int i = 0; i < 4; ++i) is[4 * w + i] = static_cast<__bf16>((nan >> (8 * i)) & 0x80u ? 1.f : 0.f);
              vr[b][c / 2][2 * (c % 2) + w] = codes & ~((nan >> 7) * 255u);
            }
            n = mfma(is, seen[b], n);
          }
#pragma unroll
          for (int x = 0; x < 16; ++x) o[c][x] = n[x] > 0.f ? NAN : o[c][x];
        }
      }
    }
    f32x16_t s = {};
#pragma unroll
    for (int x = 0; x < S; ++x) {
      s = mfma(operand8(kr[x][0], kr[x][1], ks), qf[2 * x], s);
      s = mfma(operand8(kr[x][2], kr[x][3], ks), qf[2 * x + 1], s);
    }
    bf16x8_t vf[2][C];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int c = 0; c < C; ++c) vf[b][c] = operand8(vr[b][c / 2][2 * (c % 2)], vr[b][c / 2][2 * (c % 2) + 1], vs[b]);
    if (i + 1 < n_mine) {
      if (((i + 1) & 31) == 0) look_up(i + 1);
      load(i + 1);
    }
    if (t0 + kTok > first_new) {
#pragma unroll
      for (int x = 0; x < 16; ++x) s[x] = visible(t0, x) ? s[x] : -INFINITY;
    }
    float mx = s[0];
#pragma unroll
    for (int x = 1; x < 16; ++x) mx = fmaxf(mx, s[x]);
    mx = fmaxf(mx, other_half(mx));
    const float mn = next_ref(m, mx, c2);
    const float mc = mn == -INFINITY ? 0.f : mn * c2;
    if (__any(mn > m)) {
      const float a = exp2_hw(fmaf(m, c2, -mc));
      l *= a;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int x = 0; x < 16; ++x) o[c][x] *= a;
      m = mn;
    }
    float sum = 0.f;
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      s[x] = exp2_hw(fmaf(s[x], c2, -mc));
      sum += s[x];
    }
    l += sum;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const bf16x8_t pf = pack_operand(s, b);
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = mfma(vf[b][c], pf, o[c]);
    }
  }
  l += other_half(l);

  // the four waves' sums, brought to the largest reference, added in order
  constexpr int kJ = join_row<D>();
  float2* ml = reinterpret_cast<float2*>(smem + NW * kRows * kJ);
  if (g == 0) ml[wave * kRows + r32] = make_float2(m, l);
  lds_barrier();
  float top = -INFINITY, all = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) top = fmaxf(top, ml[w * kRows + r32].x);
  const float tc = top == -INFINITY ? 0.f : top * c2;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const float2 x = ml[w * kRows + r32];
    all += x.y * exp2_hw(fmaf(x.x, c2, -tc));
  }
  const float mine = exp2_hw(fmaf(m, c2, -tc));
  // value block c = 2 j + parity holds values 64 j + 2 row + parity
  float* to = smem + (wave * kRows + r32) * kJ;
#pragma unroll
  for (int j = 0; j < C / 2; ++j)
#pragma unroll
    for (int x = 0; x < 16; x += 2) {
      const int d = 64 * j + 2 * (8 * (x >> 2) + 4 * g + (x & 3));
      *reinterpret_cast<f32x4_t*>(to + d) =
          f32x4_t{o[2 * j][x] * mine, o[2 * j + 1][x] * mine, o[2 * j][x + 1] * mine, o[2 * j + 1][x + 1] * mine};
    }
  lds_barrier();                                       // sums; ml has been read by everyone
  if (wave == 0 && g == 0) ml[r32] = make_float2(top, all);
  lds_barrier();
  const int n_out = min(kRows, n_rows - rt * kRows);
  for (int i = threadIdx.x; i < n_out * (D / 4); i += 64 * NW) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    f32x4_t x = *reinterpret_cast<const f32x4_t*>(smem + r * kJ + d);
#pragma unroll
    for (int w = 1; w < NW; ++w) x += *reinterpret_cast<const f32x4_t*>(smem + (w * kRows + r) * kJ + d);
    const float2 y = ml[r];
    if (sg.pieces == 1) {
      const float inv = y.y > 0.f ? 1.f / y.y : (y.y == 0.f ? 0.f : y.y);
      const int t = quot(rt * kRows + r, p.g), hh = head * p.g.d + rt * kRows + r - t * p.g.d;
      const int64_t at = static_cast<int64_t>(sg.start) + t;
      *reinterpret_cast<uint2*>(p.out + at * p.out_ld + hh * D + d) =
          pack4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
      if (p.lse && d == 0)
        p.lse[at * p.nh + hh] = y.y == 0.f ? -INFINITY : fmaf(y.x, p.scale, log2_hw(y.y) * kLn2);
    } else {
      const int64_t at = static_cast<int64_t>(blockIdx.x) * kRows + r;
      *reinterpret_cast<f32x4_t*>(p.part + at * D + d) = x;
      if (d == 0) p.part_ml[at] = y;
    }
  }
}

// ---- joining the pieces ------------------------------------------------------------
// A workgroup takes 256 / D of a segment's rows (2 or 4), its waves the pieces
// in turn; D / 4 lanes a row.
template <int D>
__global__ __launch_bounds__(256) void join_kernel(DecodeArgs p) {
  constexpr int kL = D / 4, kPer = 64 / kL, kSlots = kRows / kPer;
  __shared__ __attribute__((aligned(16))) float red[4][64][5];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Seg sg = find_work(p, blockIdx.x / kSlots, false);
  if (sg.b < 0 || sg.pieces == 1) return;
  // with offsets that overlap the work can exceed the grid: no such piece was stored
  if (static_cast<int64_t>(sg.first) + static_cast<int64_t>(p.nkv) * sg.row_tiles * sg.pieces > p.wgs) return;
  const int rt = sg.rest % sg.row_tiles, head = sg.rest / sg.row_tiles;
  const int n_out = min(kRows, sg.n_q * p.g.d - rt * kRows);
  const int r_first = (blockIdx.x % kSlots) * kPer;
  if (r_first >= n_out) return;
  const int r = r_first + lane / kL, d = (lane % kL) * 4;
  const int rc = min(r, n_out - 1);
  const int64_t step = static_cast<int64_t>(p.nkv) * sg.row_tiles * kRows;
  const int64_t at = (static_cast<int64_t>(sg.first) + head * sg.row_tiles + rt) * kRows + rc;
  const float c2 = p.scale * kLog2e;
  // largest reference of the row: the lanes of the row share the pieces
  float top = -INFINITY;
  for (int i = lane % kL; i < sg.pieces; i += kL) top = fmaxf(top, p.part_ml[at + i * step].x);
#pragma unroll
  for (int o = kL / 2; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  const float tc = top == -INFINITY ? 0.f : top * c2;
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
#pragma unroll 4
  for (int i = wave; i < sg.pieces; i += 4) {
    const float2 y = p.part_ml[at + i * step];
    const f32x4_t x = *reinterpret_cast<const f32x4_t*>(p.part + (at + i * step) * D + d);
    const float a = exp2_hw(fmaf(y.x, c2, -tc));
    l = fmaf(y.y, a, l);
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = fmaf(x[j], a, sum[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) red[wave][lane][j] = sum[j];
  red[wave][lane][4] = l;
  __syncthreads();
  if (wave == 0 && r < n_out) {
#pragma unroll
    for (int w = 1; w < 4; ++w) {
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += red[w][lane][j];
      l += red[w][lane][4];
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const int t = quot(rt * kRows + r, p.g), hh = head * p.g.d + rt * kRows + r - t * p.g.d;
    const int64_t o = static_cast<int64_t>(sg.start) + t;
    *reinterpret_cast<uint2*>(p.out + o * p.out_ld + hh * D + d) =
        pack4(sum[0] * inv, sum[1] * inv, sum[2] * inv, sum[3] * inv);
    if (p.lse && d == 0) p.lse[o * p.nh + hh] = l == 0.f ? -INFINITY : fmaf(top, p.scale, log2_hw(l) * kLn2);
  }
}

// (request, head, 32 rows) of a call: B requests share T tokens
int64_t segments(int B, int T, int nh, int nkv) {
  return (static_cast<int64_t>(T) * (nh / nkv) / kRows + (B < T ? B : T)) * nkv;
}

template <int D>
void launch_decode(const DecodeArgs& a, hipStream_t stream) {
  const int64_t segs = segments(a.B, a.T, a.nh, a.nkv);
  hipLaunchKernelGGL(decode_kernel<D>, dim3(static_cast<unsigned>(segs + kPieces)), dim3(64 * NW), 0, stream, a);
  constexpr int kSlots = kRows / (64 / (D / 4));
  hipLaunchKernelGGL(join_kernel<D>, dim3(static_cast<unsigned>(segs * kSlots)), dim3(256), 0, stream, a);
}

}  // namespace
}  // namespace gqa
}  // namespace moe

extern "C" size_t moe_gqa_decode_workspace(int B, int T, int n_heads, int n_kv_heads, int head_dim) {
  if (B < 1 || B > 65536 || T < 1 || n_heads < 1 || n_heads > 1024 || n_kv_heads < 1 || n_heads % n_kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128) || static_cast<int64_t>(T) * n_heads > (1 << 24))
    return 0;
  const size_t wgs = static_cast<size_t>(moe::gqa::segments(B, T, n_heads, n_kv_heads)) + moe::gqa::kPieces;
  return wgs * moe::gqa::kRows * (static_cast<size_t>(head_dim) * 4 + 8);
}

extern "C" int moe_gqa_decode(const void* q, int64_t q_ld, int fmt, const void* k_cache, const void* v_cache,
                              const uint8_t* k_scales, const uint8_t* v_scales, int page_size, int n_pages,
                              const int32_t* page_table, int max_pages, const int32_t* lens, const int32_t* cu_q,
                              const int64_t* tree_mask, int B, int T, int n_heads, int n_kv_heads, int head_dim,
                              float scale, void* out, int64_t out_ld, float* lse, void* ws, size_t ws_bytes,
                              hipStream_t stream) {
  using namespace moe;
  using namespace moe::gqa;
  clear_error();
  const char* fn = "moe_gqa_decode";
  if (const int rc = check_heads(fn, fmt, n_heads, n_kv_heads, head_dim)) return rc;
  if (const int rc = check_cache(fn, B, T, page_size, n_pages, max_pages, n_kv_heads)) return rc;
  MOE_REQUIRE(static_cast<int64_t>(T) * n_heads <= (1 << 24), MOE_ERR_INVALID_ARG,
              "moe_gqa_decode: T * n_heads must be <= 2^24");
  MOE_REQUIRE(scale > 0.f && scale <= kMaxScale, MOE_ERR_INVALID_ARG, "moe_gqa_decode: scale must be in (0, 2.3e38]");
  const int64_t row = static_cast<int64_t>(n_heads) * head_dim;
  if (const int rc = check_ld(fn, "q_ld", q_ld, row)) return rc;
  if (const int rc = check_ld(fn, "out_ld", out_ld, row)) return rc;
  if (B == 0 || T == 0) return MOE_OK;
  MOE_REQUIRE(q && k_cache && v_cache && k_scales && v_scales && page_table && lens && cu_q && out,
              MOE_ERR_INVALID_ARG, "moe_gqa_decode: null pointer");
  MOE_REQUIRE(aligned16(q) && aligned16(k_cache) && aligned16(v_cache) && aligned16(out) && aligned16(ws),
              MOE_ERR_ALIGNMENT, "moe_gqa_decode: q, the cache, out and ws must be 16-byte aligned");
  MOE_REQUIRE(ws && ws_bytes >= moe_gqa_decode_workspace(B, T, n_heads, n_kv_heads, head_dim), MOE_ERR_WORKSPACE,
              "moe_gqa_decode: ws smaller than moe_gqa_decode_workspace(...)");
  DecodeArgs a{};
  a.q = static_cast<const uint16_t*>(q), a.q_ld = q_ld;
  a.k = static_cast<const uint8_t*>(k_cache), a.v = static_cast<const uint8_t*>(v_cache);
  a.k_scales = k_scales, a.v_scales = v_scales;
  a.n_pages = n_pages, a.bpp = make_div(page_size / kBlock);
  a.table = page_table, a.max_pages = max_pages, a.lens = lens, a.cu_q = cu_q;
  a.tree = reinterpret_cast<const uint64_t*>(tree_mask);
  a.B = B, a.T = T, a.nh = n_heads, a.nkv = n_kv_heads, a.g = make_div(n_heads / n_kv_heads), a.scale = scale;
  a.out = static_cast<uint16_t*>(out), a.out_ld = out_ld, a.lse = lse;
  const size_t wgs = static_cast<size_t>(segments(B, T, n_heads, n_kv_heads)) + kPieces;
  a.wgs = static_cast<int>(wgs);
  a.part = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(a.part + wgs * kRows * head_dim);
  if (head_dim == 128) launch_decode<128>(a, stream);
  else launch_decode<64>(a, stream);
  return check_launch(fn);
}
