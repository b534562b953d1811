// moe_gqa_decode: attention of the last tokens of B requests over the 8-bit
// paged cache, grouped heads.
//
// Per new token t, query head h, with the cache's codes times their scales:
//   s[j] = scale * q[t, h] . k_j,  p = softmax(s),  out[t, h] = sum_j p_j v_j
// over the tokens that it sees. The group's heads of a request's new tokens
// are the packed rows of one product over the head's cache, 32 at a time.
//
// One launch. The cached tokens of each (request, key head, 32 rows) are cut
// into pieces of about equal length, one workgroup each, whose four waves take
// 32 tokens in turn. A wave reads keys and values straight into registers (the
// cache lies in operand order), a tile ahead of its products, and turns codes
// into bf16 operands with the block's scale in the same instruction, exactly.
// So nothing passes LDS and no wave waits for another before the piece's end,
// where the four sums are added in order. Pieces meet in the workspace: the
// workgroup that finishes a segment's last piece adds them, in their order
// whichever it is, so results repeat bit for bit.
//
// Roundings: the weights to bf16 as operands (their sum is taken before that).
// Codes times scales are exact in bf16; scores and all sums are fp32.
//
// Memory bounds long caches: 64 requests of 176k tokens x 8 key heads of 128
// take 78 to 83 us (4.5 to 4.7 TB/s of 372 MB), 8 of 279k x 2 heads 37 to 41
// (3.5 to 3.9 TB/s; the shorter the call, the more of it is start, join and the
// last pieces' ends). With 64 values a head a wave has half the bytes on their
// way: 49 us (3.8 TB/s) and 22.6 (3.2). Short ones are latency: 531 tokens x 8
// heads 9.5 us, 8.4 with 64 values. A join in a launch of its own took 8.5 to 20
// us more, eight waves a piece 154 instead of 118 for 256 requests of 1000 tokens.
//
// Every wave walks through all requests to find its place, so beside the memory's
// time a part grows with the square of their number: none is seen at 256, 1024
// requests of 200 tokens x 8 heads take 325 us (88 for their bytes), 4096 3.5 ms.
#include "gqa_cache.h"

#include <cmath>

namespace moe {
namespace gqa {
namespace {

constexpr int kTok = 32;                               // cached tokens a tile
constexpr int NW = 4;                                  // waves a workgroup
constexpr int kRows = 32;                              // packed rows a workgroup
// The most that pieces_of gives, two a compute unit; it sizes the workspace. (With
// one number for all calls 512 was the best: 768 and 1024 19 and 27% slower for
// 8 requests with 8 new tokens, 15 and 10% for 8 long caches, 64 requests the same
// within 3%. pieces_of's own numbers are below.)
constexpr int kPieces = 2 * kNumCu;                    // pieces beside one a (request, head, rows)
constexpr int kParts = 2 * kPieces;                    // pieces of segments that have several, at most
// 4 requests of 8000 tokens with 4 new each: pieces of at least 2 NW, 4 NW and
// 8 NW tiles 31, 21 and 19 us; one request of 4096 tokens 11.4, 12.3 and 15.3.
constexpr int kLeast = 4 * NW;                         // tiles a piece, at least
// one request of 531 tokens 9.6 us uncut, 11.2 cut (4 NW); 8 of 2000 tokens cut
// 15.1, uncut (16 NW) 17.7
constexpr int kAlone = 8 * NW;                         // tiles that are not cut
constexpr int kJoin = 16;                              // neighbouring pieces that are joined first

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
  float* part;               // [kParts, 32, D]: pieces of segments that have several, not normalized
  float2* part_ml;           // [kParts, 32]: their (reference, sum)
  int* done;                 // [2, kParts]: pieces of a group, and groups of a segment, that are in place;
                             // at the first piece's place; zero between calls
  int segs;                  // segments that the grid has room for
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

// n of which a call's tiles make pieces of 1 / n.
// A segment's last piece is half a piece on average, so there are about n +
// segs / 2 of them. Few segments: one piece a compute unit (a second does not
// read faster, and is joined: 8 long caches 38 us, two a unit 41; 8 requests
// with 8 new tokens 23.3 and 26). Some segments: as many as two a unit hold at
// once (20 of up to 8000 tokens 44.6 us, one a unit 46). Many: shorter pieces
// the more segments there are, so that the last to end are short (48 of up to
// 8000 tokens n = 256 98 us, 320 107; 64 of them 106, n = 512 113; 100 of them
// n = 512 175, 256 184).
__host__ __device__ constexpr int64_t pieces_of(int64_t segs) {
  return segs <= kNumCu / 2 ? kNumCu - segs / 2
         : segs <= kNumCu   ? kPieces - segs
         : segs < 3 * kNumCu ? kPieces / 2 : kPieces;
}
// Workgroups that n + segs pieces of at most so many segments need.
constexpr int64_t most_groups(int64_t segs) {
  const int64_t n = segs + pieces_of(segs);
  return segs > kNumCu / 2 && n < kPieces ? kPieces : n;
}

// Tiles of a piece: at least all tiles over kPieces (so fewer than kPieces
// segments have several pieces, and those fewer than 2 kPieces pieces), and at
// least kLeast. all, segs: one lane's share of the call's tiles and segments;
// most: the longest segment that the lane knows, then (of more than kNumCu) that
// of all.
__device__ __forceinline__ int piece_tiles(const DecodeArgs& p, int64_t all, int64_t segs, int* most) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    all += __shfl_xor(all, o, 64);
    segs += __shfl_xor(segs, o, 64);
    if (p.segs > kNumCu) *most = max(*most, __shfl_xor(*most, o, 64));
  }
  // requests whose rows overlap can exceed the grid: then nothing is cut
  if (segs > p.segs) return 1 << 30;
  const int64_t n = pieces_of(segs);
  const int64_t c = (all + n - 1) / n;
  return c > kLeast ? static_cast<int>(c < (1 << 30) ? c : (1 << 30)) : kLeast;
}

// A workgroup's part of the work.
struct Seg {
  int b;                     // -1: none
  int start, n_q, len;       // rows of q, new tokens, cached tokens
  int tiles, pieces;         // of a (head, 32 rows)
  int row_tiles;
  int rest;                  // workgroup within the request
  int part;                  // the request's first place in part
};

// The pieces of a request run slowest, its 32-row tiles fastest, so neighbours
// read the same tokens.
__device__ __forceinline__ Seg find_work(const DecodeArgs& p, int index) {
  const int lane = threadIdx.x & 63;
  int64_t all = 0, segs = 0;
  int s, n, len, tiles, rt, most = 0;
  for (int b0 = 0; b0 < p.B; b0 += 64) {
    request(p, b0 + lane, &s, &n, &len, &tiles, &rt);
    all += static_cast<int64_t>(tiles) * rt * p.nkv;
    segs += rt * p.nkv;
    most = max(most, tiles);
  }
  const int c = piece_tiles(p, all, segs, &most);
  // Where not all pieces run at once and some are cut, segments of half a piece
  // or less come last, so that the last to start are short (64 ragged requests 92
  // -> 78 us).
  const bool late = p.segs > kNumCu && most > c && most > kAlone;
  int64_t before = 0;
  for (int half = 0; half <= static_cast<int>(late); ++half) {
    int parts = 0;
    for (int b0 = 0; b0 < p.B; b0 += 64) {
      if (p.B > 64) request(p, b0 + lane, &s, &n, &len, &tiles, &rt);   // else they are at hand
      const int pieces = tiles > c && tiles > kAlone ? (tiles + c - 1) / c : 1;
      const int seg = rt * p.nkv, groups = (late && tiles <= c / 2) == (half == 1) ? seg * pieces : 0;
      const int cut = pieces > 1 ? seg : 0;
      int sum = groups, psum = cut * pieces;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(sum, o, 64), v = __shfl_up(psum, o, 64);
        if (lane >= o) sum += u, psum += v;
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
        r.rest = static_cast<int>(index - before) - __builtin_amdgcn_readlane(sum - groups, l);
        r.part = parts + __builtin_amdgcn_readlane(psum - cut * pieces, l);
        return r;
      }
      before += __builtin_amdgcn_readlane(sum, 63);
      parts += __builtin_amdgcn_readlane(psum, 63);
    }
  }
  return Seg{-1, 0, 0, 0, 0, 0, 0, 0, 0};
}

// Workgroups go to the XCDs in turn; runs of 8 work items stay on one, whose
// L2 then serves the row tiles that read the same tokens.
__device__ __forceinline__ int runs_of_8(int id, int n) {
  return id < (n & ~63) ? (id & ~63) + (id & 7) * 8 + ((id >> 3) & 7) : id;
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

// Pieces pass between compute units of different XCDs, whose L2 caches do not
// see each other's lines: device-scope accesses go past them. (Fences instead
// would write back and drop whole L2 caches under the other workgroups' loads:
// 81 against 40 us for 8 caches of 279k tokens in all x 2 key heads.)
__device__ __forceinline__ void put2(void* to, float a, float b) {
  const uint64_t v = static_cast<uint64_t>(__float_as_uint(b)) << 32 | __float_as_uint(a);
  __hip_atomic_store(static_cast<uint64_t*>(to), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 get2(const void* from) {
  const uint64_t v = __hip_atomic_load(static_cast<const uint64_t*>(from), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32)));
}

// Whether this workgroup is the last of n to arrive at a counter; all its
// stores have arrived before it counts. The last one leaves zero.
__device__ __forceinline__ bool last_of(int* count, int n, int* flag) {
  wait_vmcnt<0>();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int k = __hip_atomic_fetch_add(count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (k == n - 1) __hip_atomic_store(count, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *flag = k == n - 1;
  }
  __syncthreads();
  return *flag;
}

// Sum of n pieces, `step` places apart from place `at`, in order: D / 4 lanes a
// row, put(row, first value, sums, reference, sum of weights). U units (rows a
// lane) and K pieces are asked for at once.
template <int D, int U, int K, typename Put>
__device__ __forceinline__ void join_units(const DecodeArgs& p, float c2, int n_out, int at, int n, int step,
                                           Put&& put) {
  constexpr int kL = D / 4, kPer = 64 / kL;            // lanes a row, rows a wave
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int d = lane % kL * 4;
  f32x4_t x[U];
  float ref[U], sum[U];
  const float2* pm[U];
  const float* px[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = min((u * NW + wave) * kPer + lane / kL, n_out - 1);
    pm[u] = p.part_ml + static_cast<int64_t>(at) * kRows + r;
    px[u] = p.part + (static_cast<int64_t>(at) * kRows + r) * D + d;
    x[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    ref[u] = -INFINITY, sum[u] = 0.f;
  }
  for (int i0 = 0; i0 < n; i0 += K) {
    float2 y[U][K], z0[U][K], z1[U][K];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const int64_t o = static_cast<int64_t>(min(i0 + i, n - 1)) * step * kRows;
        y[u][i] = get2(pm[u] + o);
        z0[u][i] = get2(px[u] + o * D);
        z1[u][i] = get2(px[u] + o * D + 2);
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float top = ref[u];
#pragma unroll
      for (int i = 0; i < K; ++i) top = fmaxf(top, y[u][i].x);
      const float tc = top == -INFINITY ? 0.f : top * c2;
      const float old = exp2_hw(fmaf(ref[u], c2, -tc));
      ref[u] = top;
      sum[u] *= old;
      x[u] *= old;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const float a = i0 + i < n ? exp2_hw(fmaf(y[u][i].x, c2, -tc)) : 0.f;
        sum[u] = fmaf(y[u][i].y, a, sum[u]);
        x[u] = f32x4_t{fmaf(z0[u][i].x, a, x[u][0]), fmaf(z0[u][i].y, a, x[u][1]), fmaf(z1[u][i].x, a, x[u][2]),
                       fmaf(z1[u][i].y, a, x[u][3])};
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = (u * NW + wave) * kPer + lane / kL;
    if (r < n_out) put(r, d, x[u], ref[u], sum[u]);
  }
}
template <int D, typename Put>
__device__ __forceinline__ void join(const DecodeArgs& p, float c2, int n_out, int at, int n, int step, Put&& put) {
  constexpr int kPer = 256 / D * NW;                   // rows the workgroup takes at once
  if (n_out <= kPer) join_units<D, 1, 16>(p, c2, n_out, at, n, step, put);
  else join_units<D, kRows / kPer, 4 * kPer / 8>(p, c2, n_out, at, n, step, put);
}

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
  const Seg sg = find_work(p, runs_of_8(blockIdx.x, gridDim.x));
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

  // the waves' sums, brought to the largest reference, added in order
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
  auto store = [&](int r, int d, f32x4_t x, float ref, float sum) {
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    const int t = quot(rt * kRows + r, p.g), hh = head * p.g.d + rt * kRows + r - t * p.g.d;
    const int64_t at = static_cast<int64_t>(sg.start) + t;
    *reinterpret_cast<uint2*>(p.out + at * p.out_ld + hh * D + d) =
        pack4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    if (p.lse && d == 0) p.lse[at * p.nh + hh] = sum == 0.f ? -INFINITY : fmaf(ref, p.scale, log2_hw(sum) * kLn2);
  };
  // the segment's pieces are `step` places apart
  const int step = p.nkv * sg.row_tiles, first = sg.part + head * sg.row_tiles + rt;
  for (int i = threadIdx.x; i < n_out * (D / 4); i += 64 * NW) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    f32x4_t x = *reinterpret_cast<const f32x4_t*>(smem + r * kJ + d);
#pragma unroll
    for (int w = 1; w < NW; ++w) x += *reinterpret_cast<const f32x4_t*>(smem + (w * kRows + r) * kJ + d);
    const float2 y = ml[r];
    if (sg.pieces == 1) {
      store(r, d, x, y.x, y.y);
    } else {
      const int64_t at = static_cast<int64_t>(first + piece * step) * kRows + r;
      put2(p.part + at * D + d, x[0], x[1]);
      put2(p.part + at * D + d + 2, x[2], x[3]);
      if (d == 0) put2(p.part_ml + at, y.x, y.y);
    }
  }
  if (sg.pieces == 1) return;

  // The last piece of a group of kJoin joins them, the last group of the
  // segment the groups.
  int* flag = reinterpret_cast<int*>(smem);
  if (!last_of(p.done + first + piece / kJoin * kJoin * step, min(kJoin, sg.pieces - piece / kJoin * kJoin), flag))
    return;
  const bool one = sg.pieces <= kJoin;
  const int g0 = first + piece / kJoin * kJoin * step;
  auto keep = [&](int r, int d, f32x4_t x, float ref, float sum) {
    const int64_t at = static_cast<int64_t>(g0) * kRows + r;
    put2(p.part + at * D + d, x[0], x[1]);
    put2(p.part + at * D + d + 2, x[2], x[3]);
    if (d == 0) put2(p.part_ml + at, ref, sum);
  };
  auto both = [&](int r, int d, f32x4_t x, float ref, float sum) {
    if (one) store(r, d, x, ref, sum);
    else keep(r, d, x, ref, sum);
  };
  join<D>(p, c2, n_out, g0, min(kJoin, sg.pieces - piece / kJoin * kJoin), step, both);
  if (one) return;
  const int groups = (sg.pieces + kJoin - 1) / kJoin;
  if (!last_of(p.done + kParts + first, groups, flag)) return;
  join<D>(p, c2, n_out, first, groups, step * kJoin, store);
}

// (request, head, 32 rows) of a call: B requests share T tokens
int64_t segments(int B, int T, int nh, int nkv) {
  return (static_cast<int64_t>(T) * (nh / nkv) / kRows + (B < T ? B : T)) * nkv;
}

template <int D>
void launch_decode(const DecodeArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(decode_kernel<D>, dim3(static_cast<unsigned>(most_groups(a.segs))), dim3(64 * NW), 0, stream, a);
}

}  // namespace
}  // namespace gqa
}  // namespace moe

extern "C" size_t moe_gqa_decode_workspace(int head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return moe::gqa::kParts * 8 + static_cast<size_t>(moe::gqa::kParts) * moe::gqa::kRows * (head_dim * 4 + 8);
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
  MOE_REQUIRE(ws && ws_bytes >= moe_gqa_decode_workspace(head_dim), MOE_ERR_WORKSPACE,
              "moe_gqa_decode: ws smaller than moe_gqa_decode_workspace(head_dim)");
  DecodeArgs a{};
  a.q = static_cast<const uint16_t*>(q), a.q_ld = q_ld;
  a.k = static_cast<const uint8_t*>(k_cache), a.v = static_cast<const uint8_t*>(v_cache);
  a.k_scales = k_scales, a.v_scales = v_scales;
  a.n_pages = n_pages, a.bpp = make_div(page_size / kBlock);
  a.table = page_table, a.max_pages = max_pages, a.lens = lens, a.cu_q = cu_q;
  a.tree = reinterpret_cast<const uint64_t*>(tree_mask);
  a.B = B, a.T = T, a.nh = n_heads, a.nkv = n_kv_heads, a.g = make_div(n_heads / n_kv_heads), a.scale = scale;
  a.out = static_cast<uint16_t*>(out), a.out_ld = out_ld, a.lse = lse;
  a.segs = static_cast<int>(segments(B, T, n_heads, n_kv_heads));
  a.done = static_cast<int*>(ws);
  a.part = reinterpret_cast<float*>(a.done + 2 * kParts);
  a.part_ml = reinterpret_cast<float2*>(a.part + static_cast<size_t>(kParts) * kRows * head_dim);
  if (head_dim == 128) launch_decode<128>(a, stream);
  else launch_decode<64>(a, stream);
  return check_launch(fn);
}
