// moe_mla_attn_bwd: gradients of moe_mla_attn_fwd.
//
// With p the softmax weights, do the output's gradient:
//   delta[i] = do[i] . out[i]          (= sum_j p[i, j] dp[i, j])
//   dp = do v^T,  ds = p (dp - delta),  dv = p^T do
//   dq = scale ds k,  dk = scale ds^T q,  dk_rope = sum over heads of dk's
//   rotary columns
// p is computed again from the scores and the forward's lse.
//
// Three launches: the row statistics (lse in base 2, delta); the gradients,
// where one kind of workgroup keeps 32 keys a wave and walks the queries (dk,
// dv) and the other keeps 32 queries a wave and walks the keys (dq); the sum
// of the heads' rotary gradients. The scores are computed twice, so nothing
// is added up by atomics and the result does not depend on the order in which
// workgroups run.
//
// p and ds are rounded to bf16 as operands of dv, dk and dq (the matrix
// instruction's type; rms 2^-9.2 of each element, so a gradient, a sum of
// many, keeps that relative error: 2.5e-3 rms against 64 bits with its own
// rounding at the store). delta is formed from the stored out, which is
// rounded to bf16 and a sum of rounded weights (keeping it in fp32 would be
// another output of the forward, twice out's bytes); scores, dp, delta's sum
// and all other sums are fp32.
//
// Bound by the products and their operands from LDS: seven products of pairs
// x 128..192 (the formulas' five, scores and dp once more) = 1.44 TFLOP with
// the diagonal's tiles at 4096 tokens x 128 heads, causal; the gradients'
// kernel takes 1650 us on average of 20 calls (1514 for the first to 2038: the
// clock falls under this load) = 870 TFLOP/s (matrix unit 43% busy; an 8192^3
// bf16 product reaches 1369). The kept side's operands and sums (kv: 80
// operand, 160 sum, 64 score registers) bring a wave to 194 + 224 of 512
// registers, too many for two waves a SIMD; 81 of 160 KB LDS. What overlaps is
// written out: operands are read kAhead products ahead, and one block's
// element-wise work runs between another's products. A tile of 64
// queries takes 4.7k cycles against 2560 of products, a tile of 64 keys in the
// other part 3.4k against 2048; start and end (operands in, sums out through
// LDS) about 20k a workgroup, 15 to 25% of an average one here. Statistics (47
// us) and rotary sums (27 us) run at the rate of a copy. 515 tokens x 16 heads:
// 3.5 + 24.3 + 4.5 us: a workgroup walks up to seven tiles one after another.
// Measured and slower: nothing read ahead and two waves a SIMD for dq (1169 +
// 901 us for the two parts, against 954 + 779 then), two launches for the parts
// (1733), three stages with the barrier in mid-tile (1693), three blocks in
// flight at once with every element under two products (1817).
#include "mla.h"

#include <cmath>

namespace moe {
namespace mla {
namespace {

struct BwdArgs {
  const uint16_t* dout;
  int64_t dout_ld;
  const uint16_t* q;
  int64_t q_ld;
  const uint16_t* kv;
  int64_t kv_ld;
  const uint16_t* kr;
  int64_t kr_ld;
  const uint16_t* out;
  int64_t out_ld;
  const float* lse;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, Tq, Tk, nh, causal;
  float scale;
  uint16_t* dq;
  int64_t dq_ld;
  uint16_t* dkv;
  int64_t dkv_ld;
  uint16_t* dkr;
  int64_t dkr_ld;
  float2* stats;    // [nh, Tq]: (lse in base 2, delta); a row without keys: (+inf, 0)
  float* dkr_part;  // [nh, Tk, 64]
  int k_tiles, q_tiles;   // workgroups per head of the two parts
};

// 16 lanes per (token, head) row of 128 values
__global__ __launch_bounds__(256) void bwd_stats_kernel(BwdArgs p) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  if (row >= static_cast<int64_t>(p.Tq) * p.nh) return;
  const int64_t t = row / p.nh;
  const int h = static_cast<int>(row - t * p.nh);
  const int c = (threadIdx.x & 15) * 8;
  const u32x4_t a = *reinterpret_cast<const u32x4_t*>(p.out + t * p.out_ld + h * kDv + c);
  const u32x4_t b = *reinterpret_cast<const u32x4_t*>(p.dout + t * p.dout_ld + h * kDv + c);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), s);
    s = fmaf(__uint_as_float(a[i] & 0xFFFF0000u), __uint_as_float(b[i] & 0xFFFF0000u), s);
  }
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) s += __shfl_xor(s, o, 16);
  if ((threadIdx.x & 15) == 0) {
    const float l = p.lse[row];
    const bool none = l == -INFINITY;
    p.stats[static_cast<int64_t>(h) * p.Tq + t] = none ? make_float2(INFINITY, 0.f) : make_float2(l * kLog2e, s);
  }
}

// LDS offsets of the operands of one stage: a tile of 256-byte rows, one of
// 128-byte rows behind it (at N256), a second of 256-byte rows behind both,
// read with the first's offsets. They move with the stage in use, so no
// address is computed between the products.
template <int N256>
struct Operands {
  uint32_t r256[8], r128[4], c256[4][2], c128[2][2];
  __device__ __forceinline__ explicit Operands(int lane) {
#pragma unroll
    for (int s = 0; s < 8; ++s) r256[s] = row_operand_offset<256>(lane, s);
#pragma unroll
    for (int s = 0; s < 4; ++s) r128[s] = N256 + row_operand_offset<128>(lane, s);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int c = 0; c < 4; ++c) c256[c][h] = col_operand_offset<256>(lane, c, h);
#pragma unroll
      for (int c = 0; c < 2; ++c) c128[c][h] = N256 + col_operand_offset<128>(lane, c, h);
    }
  }
  __device__ __forceinline__ void move(int by) {
#pragma unroll
    for (int s = 0; s < 8; ++s) r256[s] += by;
#pragma unroll
    for (int s = 0; s < 4; ++s) r128[s] += by;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int c = 0; c < 4; ++c) c256[c][h] += by;
#pragma unroll
      for (int c = 0; c < 2; ++c) c128[c][h] += by;
    }
  }
};

// ---- dk, dv: a wave keeps 32 keys (the lanes' columns), queries pass by ------
constexpr int kQTile = 64;
constexpr int kAhead = 5;                               // matrix operands read ahead
constexpr int kKvWaves = 4;
constexpr int kKvKeys = 32 * kKvWaves;
constexpr int kLdsQn = kQTile * kDn * 2, kLdsQr = kQTile * kDr * 2, kLdsDo = kQTile * kDv * 2;
constexpr int kLdsStat = kQTile * 8;
constexpr int kLdsKvStage = kLdsQn + kLdsQr + kLdsDo + kLdsStat;

__device__ __forceinline__ void bwd_kv(const BwdArgs& p, int idx, uint8_t* smem) {
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int head = idx / p.k_tiles;
  const SeqTile st = find_tile(p.cu_k, p.cu_q, p.B, p.Tk, p.Tq, kKvKeys, idx % p.k_tiles);
  if (st.b < 0) return;
  const int n_k = st.n;
  const int q_start = st.start2, n_q = st.n2;
  const int k0 = st.tile * kKvKeys;
  const int key = k0 + wave * 32 + (lane & 31);
  const int keyc = key < n_k ? key : n_k - 1;
  const int shift = p.causal ? n_k - n_q : n_k;                // query i sees keys <= i + shift
  const int q_first = p.causal ? max(0, k0 - shift) : 0;       // first query that sees a key of the tile
  const int t_first = q_first / kQTile;
  const int t_end = (n_q + kQTile - 1) / kQTile;

  const uint16_t* q = p.q + static_cast<int64_t>(q_start) * p.q_ld + head * kDq;
  const uint16_t* dout = p.dout + static_cast<int64_t>(q_start) * p.dout_ld + head * kDv;
  const float2* stats = p.stats + static_cast<int64_t>(head) * p.Tq + q_start;
  float2 stat_next = make_float2(INFINITY, 0.f);
  auto load = [&](int t, uint8_t* buf) {
    const int n = n_q - t * kQTile;
    const int nv = n < kQTile ? n : kQTile;
    const uint16_t* qb = q + static_cast<int64_t>(t) * kQTile * p.q_ld;
    const uint32_t ld = static_cast<uint32_t>(p.q_ld * 2);
    tile_load<256, kQTile, kKvWaves>(qb, ld, nv, buf, wave, lane);
    tile_load<128, kQTile, kKvWaves>(qb + kDn, ld, nv, buf + kLdsQn, wave, lane);
    tile_load<256, kQTile, kKvWaves>(dout + static_cast<int64_t>(t) * kQTile * p.dout_ld,
                                     static_cast<uint32_t>(p.dout_ld * 2), nv, buf + kLdsQn + kLdsQr, wave, lane);
    if (wave == 0) stat_next = lane < nv ? stats[t * kQTile + lane] : make_float2(INFINITY, 0.f);
  };
  // the statistics of 64 queries as two arrays, read as broadcasts of 4
  auto put_stats = [&](uint8_t* buf) {
    if (wave == 0) {
      float* s = reinterpret_cast<float*>(buf + kLdsQn + kLdsQr + kLdsDo);
      s[lane] = stat_next.x;
      s[64 + lane] = stat_next.y;
    }
  };
  if (t_first < t_end) load(t_first, smem);

  bf16x8_t kf[kDq / 16], vf[kDv / 16];
  {
    const int64_t tok = static_cast<int64_t>(st.start) + keyc;
    const uint16_t* k = p.kv + tok * p.kv_ld + head * (kDn + kDv) + 8 * g;
    const uint16_t* r = p.kr + tok * p.kr_ld + 8 * g;
#pragma unroll
    for (int s = 0; s < 8; ++s) kf[s] = *reinterpret_cast<const bf16x8_t*>(k + 16 * s);
#pragma unroll
    for (int s = 0; s < 4; ++s) kf[8 + s] = *reinterpret_cast<const bf16x8_t*>(r + 16 * s);
#pragma unroll
    for (int s = 0; s < 8; ++s) vf[s] = *reinterpret_cast<const bf16x8_t*>(k + kDn + 16 * s);
  }
  Operands<kLdsQn> ops(lane);
  f32x16_t dk[6], dv[4];
#pragma unroll
  for (int c = 0; c < 6; ++c) {
    dk[c] = f32x16_t{};
    keep_acc(dk[c]);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    dv[c] = f32x16_t{};
    keep_acc(dv[c]);
  }
  const float c2 = p.scale * kLog2e;

  auto tile = [&](int t, auto cut_c) {
    constexpr bool kCut = decltype(cut_c)::value;
    uint8_t* buf = smem + ((t - t_first) & 1) * kLdsKvStage;
    put_stats(buf);                   // the other buffer's readers are a barrier behind
    wait_vmcnt<0>();
    lds_barrier();
    if (t + 1 < t_end) load(t + 1, smem + ((t + 1 - t_first) & 1) * kLdsKvStage);
    const uint8_t* dob = buf + kLdsQn + kLdsQr;
    const float* stat = reinterpret_cast<const float*>(dob + kLdsDo);
    // 80 products of two blocks of 32 queries: the scores and dp of block 0,
    // of block 1, then dv and dk from block 0 and from block 1. Their LDS
    // operands are read kAhead products ahead, and the element-wise work of
    // block 0 runs between the products of block 1's scores, that of block 1
    // between the products of block 0's gradients.
    constexpr int kDo = kLdsQn + kLdsQr;                // dO's place behind Q's
    {
      bf16x8_t a[kAhead], pf[2][2], sf[2][2];
      f32x16_t s[2], dp[2];
      f32x4_t l2[2], dl[2];
      typedef float f32x8_t __attribute__((ext_vector_type(8)));
      f32x8_t we, de;                 // elements of the current operand
      auto fetch = [&](auto n_c) {
        constexpr int n = decltype(n_c)::value, slot = n % kAhead;
        if constexpr (n < 40) {
          constexpr int b = n / 20, k = n % 20;
          if constexpr (k >= 16) a[slot] = row_operand(smem, ops.r128[k - 16] + b * 32 * 128);
          else a[slot] = row_operand(smem, ops.r256[k / 2] + (k % 2 ? kDo : 0) + b * 32 * 256);
        } else {
          constexpr int b = (n - 40) / 20, k = (n - 40) % 20 / 10, c = (n - 40) % 10;
          constexpr int o256 = (2 * b + k) * 16 * 256 + (c < 4 ? kDo : 0), o128 = (2 * b + k) * 16 * 128;
          if constexpr (c >= 8)
            a[slot] = col_operand(smem, ops.c128[c - 8][0] + o128, ops.c128[c - 8][1] + o128);
          else
            a[slot] = col_operand(smem, ops.c256[c % 4][0] + o256, ops.c256[c % 4][1] + o256);
        }
      };
      // statistics of 4 queries: elements 4 j .. 4 j + 3 of block b
      auto stats_of = [&](auto b_c, auto j_c) {
        constexpr int b = decltype(b_c)::value, j = decltype(j_c)::value;
        l2[j & 1] = *reinterpret_cast<const f32x4_t*>(stat + 32 * b + 8 * j + 4 * g);
        dl[j & 1] = *reinterpret_cast<const f32x4_t*>(stat + 64 + 32 * b + 8 * j + 4 * g);
      };
      auto element = [&](auto b_c, auto i_c) {
        constexpr int b = decltype(b_c)::value, i = decltype(i_c)::value;
        if constexpr (i % 4 == 0 && i < 12) stats_of(b_c, std::integral_constant<int, i / 4 + 1>{});
        float w = exp2_hw(fmaf(s[b][i], c2, -l2[(i >> 2) & 1][i & 3]));
        float d = w * (dp[b][i] - dl[(i >> 2) & 1][i & 3]);
        if constexpr (kCut) {
          const bool hidden = key > t * kQTile + 32 * b + 8 * (i >> 2) + 4 * g + (i & 3) + shift;
          w = hidden ? 0.f : w;
          d = hidden ? 0.f : d;
        }
        we[i % 8] = w;
        de[i % 8] = d;
        if constexpr (i % 8 == 7) {
          pf[b][i / 8] = __builtin_convertvector(we, bf16x8_t);
          sf[b][i / 8] = __builtin_convertvector(de, bf16x8_t);
        }
      };
      static_for<kAhead>([&](auto n_c) { fetch(n_c); });
      __builtin_amdgcn_sched_barrier(0);
      static_for<80>([&](auto n_c) {
        constexpr int n = decltype(n_c)::value, slot = n % kAhead;
        if constexpr (n < 40) {
          constexpr int b = n / 20, k = n % 20;
          if constexpr (k >= 16) s[b] = mfma(a[slot], kf[8 + k - 16], s[b]);
          else if constexpr (k % 2 == 0) s[b] = mfma(a[slot], kf[k / 2], k == 0 ? f32x16_t{} : s[b]);
          else dp[b] = mfma(a[slot], vf[k / 2], k == 1 ? f32x16_t{} : dp[b]);
        } else {
          constexpr int b = (n - 40) / 20, k = (n - 40) % 20 / 10, c = (n - 40) % 10;
          if constexpr (c < 4) dv[c] = mfma(a[slot], pf[b][k], dv[c]);
          else dk[c - 4] = mfma(a[slot], sf[b][k], dk[c - 4]);
        }
        if constexpr (n + kAhead < 80) fetch(std::integral_constant<int, n + kAhead>{});
        // element i of block b behind product 20 b + 22 + i
        if constexpr (n >= 22 && n < 38) element(std::integral_constant<int, 0>{}, std::integral_constant<int, n - 22>{});
        if constexpr (n == 18 || n == 38)
          stats_of(std::integral_constant<int, n / 20>{}, std::integral_constant<int, 0>{});
        if constexpr (n >= 42 && n < 58) element(std::integral_constant<int, 1>{}, std::integral_constant<int, n - 42>{});
        __builtin_amdgcn_sched_barrier(0);
      });
#pragma unroll
      for (int c = 0; c < 6; ++c) keep_acc(dk[c]);
#pragma unroll
      for (int c = 0; c < 4; ++c) keep_acc(dv[c]);
      ops.move((t - t_first) & 1 ? -kLdsKvStage : kLdsKvStage);
    }
  };
  // the tiles that the causal mask cuts come first; each loop has one body
  // (a choice inside it would cost copies of the sums where its sides meet)
  const int cut_end = p.causal ? min(t_end, max(t_first, (k0 + kKvKeys - shift + kQTile - 1) / kQTile)) : t_first;
  int t = t_first;
  for (; t < cut_end; ++t) tile(t, std::true_type{});
  for (; t < t_end; ++t) tile(t, std::false_type{});
  acc_settled();
  lds_barrier();                        // everyone is done with the tiles
  auto value = [&](const f32x16_t& v, int i) {
    return f32x4_t{read_acc(v[4 * i]), read_acc(v[4 * i + 1]), read_acc(v[4 * i + 2]), read_acc(v[4 * i + 3])};
  };
  constexpr int kRb = (kDn + kDv) * 2;
  static_assert(kKvWaves * result_bytes<kRb>() <= 2 * kLdsKvStage, "results fit the tile buffers");
  uint8_t* rows = smem + wave * result_bytes<kRb>();
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4_t x = value(dk[c], i) * p.scale, y = value(dv[c], i);
      uint8_t* o = rows + (lane & 31) * (kRb + 16) + (32 * c + 8 * i + 4 * g) * 2;
      *reinterpret_cast<uint2*>(o) = pack4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<uint2*>(o + kDn * 2) = pack4(y[0], y[1], y[2], y[3]);
    }
  const int64_t tok = static_cast<int64_t>(st.start) + k0 + wave * 32;
  const int n_out = n_k - k0 - wave * 32;
  store_rows<kRb>(rows, p.dkv + tok * p.dkv_ld + head * (kDn + kDv), p.dkv_ld * 2, n_out, lane);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f32x4_t*>(rows + (lane & 31) * (kDr * 4 + 16) + (32 * c + 8 * i + 4 * g) * 4) =
          value(dk[4 + c], i);
  store_rows<kDr * 4>(rows, p.dkr_part + (static_cast<int64_t>(head) * p.Tk + tok) * kDr, kDr * 4, n_out, lane);
}

// ---- dq: a wave keeps 32 queries (the lanes' columns), keys pass by ----------
constexpr int kKt = 64;
constexpr int kQWaves = 4;
constexpr int kQRows = 32 * kQWaves;
constexpr int kLdsKn = kKt * kDn * 2, kLdsKr = kKt * kDr * 2, kLdsV = kKt * kDv * 2;
constexpr int kLdsQStage = kLdsKn + kLdsKr + kLdsV;

__device__ __forceinline__ void bwd_q(const BwdArgs& p, int idx, uint8_t* smem) {
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int head = idx / p.q_tiles;
  const SeqTile st = find_tile(p.cu_q, p.cu_k, p.B, p.Tq, p.Tk, kQRows, p.q_tiles - 1 - idx % p.q_tiles);
  if (st.b < 0) return;
  const int k_start = st.start2, n_k = st.n2;
  const int n_q = st.n;
  const int q0 = st.tile * kQRows;
  const int row = q0 + wave * 32 + (lane & 31);
  const int rowc = row < n_q ? row : n_q - 1;
  const int shift = p.causal ? n_k - n_q : n_k;
  const int last = p.causal ? min(rowc + shift, n_k - 1) : n_k - 1;
  const int first_last = p.causal ? min(q0 + shift, n_k - 1) : n_k - 1;     // of the tile's first query
  const int tile_last = p.causal ? min(min(q0 + kQRows, n_q) - 1 + shift, n_k - 1) : n_k - 1;
  const int n_kt = tile_last < 0 ? 0 : tile_last / kKt + 1;
  const int n_full = first_last < 0 ? 0 : min(n_kt, (first_last + 1) / kKt); // tiles that every query sees whole

  const uint16_t* kv = p.kv + static_cast<int64_t>(k_start) * p.kv_ld + head * (kDn + kDv);
  const uint16_t* kr = p.kr + static_cast<int64_t>(k_start) * p.kr_ld;
  auto load = [&](int kt, uint8_t* buf) {
    const int n = n_k - kt * kKt;
    const int nv = n < kKt ? n : kKt;
    const uint16_t* b = kv + static_cast<int64_t>(kt) * kKt * p.kv_ld;
    const uint32_t ld = static_cast<uint32_t>(p.kv_ld * 2);
    tile_load<256, kKt, kQWaves>(b, ld, nv, buf, wave, lane);
    tile_load<128, kKt, kQWaves>(kr + static_cast<int64_t>(kt) * kKt * p.kr_ld, static_cast<uint32_t>(p.kr_ld * 2), nv,
                                 buf + kLdsKn, wave, lane);
    tile_load<256, kKt, kQWaves>(b + kDn, ld, nv, buf + kLdsKn + kLdsKr, wave, lane);
  };
  if (n_kt > 0) load(0, smem);

  const int64_t tokc = static_cast<int64_t>(st.start) + rowc;
  bf16x8_t qf[kDq / 16], df[kDv / 16];
  {
    const uint16_t* q = p.q + tokc * p.q_ld + head * kDq + 8 * g;
    const uint16_t* d = p.dout + tokc * p.dout_ld + head * kDv + 8 * g;
#pragma unroll
    for (int s = 0; s < kDq / 16; ++s) qf[s] = *reinterpret_cast<const bf16x8_t*>(q + 16 * s);
#pragma unroll
    for (int s = 0; s < kDv / 16; ++s) df[s] = *reinterpret_cast<const bf16x8_t*>(d + 16 * s);
  }
  const float2 stat = p.stats[static_cast<int64_t>(head) * p.Tq + tokc];
  Operands<kLdsKn> ops(lane);
  f32x16_t dq[6];
#pragma unroll
  for (int c = 0; c < 6; ++c) {
    dq[c] = f32x16_t{};
    keep_acc(dq[c]);
  }
  const float c2 = p.scale * kLog2e;

  auto tile = [&](int kt, auto cut_c) {
    constexpr bool kCut = decltype(cut_c)::value;
    wait_vmcnt<0>();
    lds_barrier();
    if (kt + 1 < n_kt) load(kt + 1, smem + ((kt + 1) & 1) * kLdsQStage);
    constexpr int kV = kLdsKn + kLdsKr;                 // V's place behind K's
    // 64 products, in the order of the kernel above: scores and dp of block 0
    // and block 1 of 32 keys, then dq from block 0 and from block 1; the
    // element-wise work of a block runs between the products after its scores
    bf16x8_t a[kAhead], sf[2][2];
    f32x16_t s[2], dp[2];
    typedef float f32x8_t __attribute__((ext_vector_type(8)));
    f32x8_t de;
    auto fetch = [&](auto n_c) {
      constexpr int n = decltype(n_c)::value, slot = n % kAhead;
      if constexpr (n < 40) {
        constexpr int b = n / 20, k = n % 20;
        if constexpr (k >= 16) a[slot] = row_operand(smem, ops.r128[k - 16] + b * 32 * 128);
        else a[slot] = row_operand(smem, ops.r256[k / 2] + (k % 2 ? kV : 0) + b * 32 * 256);
      } else {
        constexpr int k = (n - 40) / 6, c = (n - 40) % 6;
        constexpr int o256 = k * 16 * 256, o128 = k * 16 * 128;
        if constexpr (c >= 4)
          a[slot] = col_operand(smem, ops.c128[c - 4][0] + o128, ops.c128[c - 4][1] + o128);
        else
          a[slot] = col_operand(smem, ops.c256[c][0] + o256, ops.c256[c][1] + o256);
      }
    };
    auto element = [&](auto b_c, auto i_c) {
      constexpr int b = decltype(b_c)::value, i = decltype(i_c)::value;
      float d = exp2_hw(fmaf(s[b][i], c2, -stat.x)) * (dp[b][i] - stat.y);
      if constexpr (kCut) d = kt * kKt + 32 * b + 8 * (i >> 2) + 4 * g + (i & 3) > last ? 0.f : d;
      de[i % 8] = d;
      if constexpr (i % 8 == 7) sf[b][i / 8] = __builtin_convertvector(de, bf16x8_t);
    };
    static_for<kAhead>([&](auto n_c) { fetch(n_c); });
    __builtin_amdgcn_sched_barrier(0);
    static_for<64>([&](auto n_c) {
      constexpr int n = decltype(n_c)::value, slot = n % kAhead;
      if constexpr (n < 40) {
        constexpr int b = n / 20, k = n % 20;
        if constexpr (k >= 16) s[b] = mfma(a[slot], qf[8 + k - 16], s[b]);
        else if constexpr (k % 2 == 0) s[b] = mfma(a[slot], qf[k / 2], k == 0 ? f32x16_t{} : s[b]);
        else dp[b] = mfma(a[slot], df[k / 2], k == 1 ? f32x16_t{} : dp[b]);
      } else {
        constexpr int k = (n - 40) / 6, c = (n - 40) % 6;
        dq[c] = mfma(a[slot], sf[k / 2][k % 2], dq[c]);
      }
      if constexpr (n + kAhead < 64) fetch(std::integral_constant<int, n + kAhead>{});
      if constexpr (n >= 22 && n < 38) element(std::integral_constant<int, 0>{}, std::integral_constant<int, n - 22>{});
      if constexpr (n >= 42 && n < 58) element(std::integral_constant<int, 1>{}, std::integral_constant<int, n - 42>{});
      __builtin_amdgcn_sched_barrier(0);
    });
#pragma unroll
    for (int c = 0; c < 6; ++c) keep_acc(dq[c]);
    ops.move(kt & 1 ? -kLdsQStage : kLdsQStage);
  };
  int kt = 0;
  for (; kt < n_full; ++kt) tile(kt, std::false_type{});
  for (; kt < n_kt; ++kt) tile(kt, std::true_type{});

  acc_settled();
  lds_barrier();                        // everyone is done with the tiles
  uint8_t* rows = smem + wave * result_bytes<kDq * 2>();
#pragma unroll
  for (int c = 0; c < 6; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float sc = p.scale;
      *reinterpret_cast<uint2*>(rows + (lane & 31) * (kDq * 2 + 16) + (32 * c + 8 * i + 4 * g) * 2) =
          pack4(read_acc(dq[c][4 * i]) * sc, read_acc(dq[c][4 * i + 1]) * sc, read_acc(dq[c][4 * i + 2]) * sc,
                read_acc(dq[c][4 * i + 3]) * sc);
    }
  const int64_t tok = static_cast<int64_t>(st.start) + q0 + wave * 32;
  store_rows<kDq * 2>(rows, p.dq + tok * p.dq_ld + head * kDq, p.dq_ld * 2, n_q - q0 - wave * 32, lane);
}

// Both parts in one launch, dk / dv first: the second fills the compute units
// that the first's last workgroups leave, and short sequences need both to
// fill the chip.
static_assert(kKvWaves == kQWaves, "one workgroup size");
__global__ __launch_bounds__(64 * kQWaves) __attribute__((amdgpu_waves_per_eu(1, 1)))
void bwd_kernel(BwdArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * (kLdsKvStage > kLdsQStage ? kLdsKvStage : kLdsQStage)];
  const int n_kv = p.k_tiles * p.nh, n_q = p.q_tiles * p.nh;
  const int id = blockIdx.x;
  if (id < n_kv) bwd_kv(p, xcd_contiguous(id, n_kv), smem);
  else bwd_q(p, xcd_contiguous(id - n_kv, n_q), smem);
}

// ---- dk_rope[t] = scale * sum over heads, in head order ----------------------
// A workgroup takes 4 tokens: 16 lanes x 4 values a token, 4 groups of heads
// whose sums are joined in a fixed order. Only rows that a sequence holds;
// `skip` is where this launch's part of them starts.
constexpr int kRopeTok = 4;
constexpr int kRopeLaunch = 1 << 25;   // tokens of one launch: 64 work items each, below 2^32
__global__ __launch_bounds__(256) void bwd_rope_kernel(BwdArgs p, int skip) {
  __shared__ f32x4_t part[4][64];
  const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
  const int lo = clamp_int(p.cu_k[0], 0, p.Tk), hi = clamp_int(p.cu_k[p.B], lo, p.Tk);
  const int64_t t = static_cast<int64_t>(lo) + skip + blockIdx.x * kRopeTok + (lane >> 4);
  f32x4_t s = {0.f, 0.f, 0.f, 0.f};
  if (t < hi) {
    const float* src = p.dkr_part + t * kDr + (lane & 15) * 4;
#pragma unroll 8
    for (int h = grp; h < p.nh; h += 4) {
      const f32x4_t v = *reinterpret_cast<const f32x4_t*>(src + static_cast<int64_t>(h) * p.Tk * kDr);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += v[i];
    }
  }
  part[grp][lane] = s;
  __syncthreads();
  if (grp == 0 && t < hi) {
#pragma unroll
    for (int k = 1; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += part[k][lane][i];
    *reinterpret_cast<uint2*>(p.dkr + t * p.dkr_ld + (lane & 15) * 4) =
        pack4(s[0] * p.scale, s[1] * p.scale, s[2] * p.scale, s[3] * p.scale);
  }
}

size_t stats_bytes(int Tq, int nh) { return (static_cast<size_t>(Tq) * nh * 8 + 255) & ~size_t{255}; }

}  // namespace
}  // namespace mla
}  // namespace moe

extern "C" size_t moe_mla_attn_bwd_workspace(int Tq, int Tk, int n_heads) {
  if (Tq < 0 || Tk < 0 || Tq > (1 << 28) || Tk > (1 << 28) || n_heads < 1 || n_heads > 1024) return 0;
  return moe::mla::stats_bytes(Tq, n_heads) + static_cast<size_t>(Tk) * n_heads * moe::mla::kDr * 4;
}

extern "C" int moe_mla_attn_bwd(const void* dout, int64_t dout_ld, const void* q, int64_t q_ld, const void* kv,
                                int64_t kv_ld, const void* k_rope, int64_t kr_ld, int fmt, const void* out,
                                int64_t out_ld, const float* lse, const int32_t* cu_q, const int32_t* cu_k, int B,
                                int Tq, int Tk, int n_heads, int causal, float scale, void* dq, int64_t dq_ld,
                                void* dkv, int64_t dkv_ld, void* dk_rope, int64_t dkr_ld, void* ws, size_t ws_bytes,
                                hipStream_t stream) {
  using namespace moe;
  using namespace moe::mla;
  clear_error();
  const char* fn = "moe_mla_attn_bwd";
  if (const int rc = check_expanded(fn, fmt, B, Tq, Tk, n_heads, causal, scale, q_ld, kv_ld, kr_ld, out_ld)) return rc;
  if (const int rc = check_expanded(fn, fmt, B, Tq, Tk, n_heads, causal, scale, dq_ld, dkv_ld, dkr_ld, dout_ld))
    return rc;
  if (B == 0 || (Tq == 0 && Tk == 0)) return MOE_OK;
  MOE_REQUIRE(cu_q && cu_k && (Tq == 0 || (dout && q && out && lse && dq)) &&
                  (Tk == 0 || (kv && k_rope && dkv && dk_rope)),
              MOE_ERR_INVALID_ARG, "moe_mla_attn_bwd: null pointer");
  MOE_REQUIRE(aligned16(dout) && aligned16(q) && aligned16(kv) && aligned16(k_rope) && aligned16(out) &&
                  aligned16(dq) && aligned16(dkv) && aligned16(dk_rope) && aligned16(ws),
              MOE_ERR_ALIGNMENT, "moe_mla_attn_bwd: tensors and ws must be 16-byte aligned");
  MOE_REQUIRE(ws && ws_bytes >= moe_mla_attn_bwd_workspace(Tq, Tk, n_heads), MOE_ERR_WORKSPACE,
              "moe_mla_attn_bwd: ws smaller than moe_mla_attn_bwd_workspace(Tq, Tk, n_heads)");
  BwdArgs a{};
  a.dout = static_cast<const uint16_t*>(dout), a.dout_ld = dout_ld;
  a.q = static_cast<const uint16_t*>(q), a.q_ld = q_ld;
  a.kv = static_cast<const uint16_t*>(kv), a.kv_ld = kv_ld;
  a.kr = static_cast<const uint16_t*>(k_rope), a.kr_ld = kr_ld;
  a.out = static_cast<const uint16_t*>(out), a.out_ld = out_ld;
  a.lse = lse, a.cu_q = cu_q, a.cu_k = cu_k;
  a.B = B, a.Tq = Tq, a.Tk = Tk, a.nh = n_heads, a.causal = causal, a.scale = scale;
  a.dq = static_cast<uint16_t*>(dq), a.dq_ld = dq_ld;
  a.dkv = static_cast<uint16_t*>(dkv), a.dkv_ld = dkv_ld;
  a.dkr = static_cast<uint16_t*>(dk_rope), a.dkr_ld = dkr_ld;
  a.stats = static_cast<float2*>(ws);
  a.dkr_part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + stats_bytes(Tq, n_heads));
  if (Tq > 0) {
    const int64_t rows = static_cast<int64_t>(Tq) * n_heads;
    hipLaunchKernelGGL(bwd_stats_kernel, dim3(static_cast<unsigned>((rows + 15) / 16)), dim3(256), 0, stream, a);
  }
  a.k_tiles = Tk > 0 ? seq_tiles_bound(B, Tk, kKvKeys) : 0;
  a.q_tiles = Tq > 0 ? seq_tiles_bound(B, Tq, kQRows) : 0;
  hipLaunchKernelGGL(bwd_kernel, dim3(static_cast<unsigned>(a.k_tiles + a.q_tiles) * n_heads), dim3(64 * kQWaves), 0,
                     stream, a);
  for (int skip = 0; skip < Tk; skip += kRopeLaunch) {
    const int n = Tk - skip < kRopeLaunch ? Tk - skip : kRopeLaunch;
    hipLaunchKernelGGL(bwd_rope_kernel, dim3((n + kRopeTok - 1) / kRopeTok), dim3(256), 0, stream, a, skip);
  }
  return check_launch(fn);
}
