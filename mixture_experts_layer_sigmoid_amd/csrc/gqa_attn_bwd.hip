// moe_gqa_attn_bwd: gradients of moe_gqa_attn_fwd.
//
// With p the softmax weights, do the output's gradient:
//   delta[i] = do[i] . out[i]          (= sum_j p[i, j] dp[i, j])
//   dp = do v^T,  ds = p (dp - delta),  dv = p^T do
//   dq = scale ds k,  dk = scale ds^T q,  dk and dv summed over the queries of
//   all heads of the group
// p is computed again from the scores and the forward's lse.
//
// The row statistics (lse in base 2, delta) come first, then the gradients:
// one kind of workgroup keeps 32 keys a wave and walks the packed rows (dk, dv:
// the heads of the group are rows among others, so their sum needs no further
// step), the other keeps 32 packed rows a wave and walks the keys (dq). The
// scores are computed twice, so nothing is added up by atomics and the result
// does not depend on the order in which workgroups run. With few keys the rows
// are cut into parts whose dk and dv (fp32) a last launch adds up in order.
//
// p and ds are rounded to bf16 as operands of dv, dk and dq (the matrix
// instruction's type; rms 2^-9.2 of each element). delta is formed from the
// stored out, which is rounded to bf16: it is the output that a caller keeps
// anyway. An out of twice the digits beside it would take 0.1e-3 off errors of
// 2.5e-3 to 2.8e-3 of dq and dk, for 1% of the time and twice its memory. Scores,
// dp, delta's sum and all other sums are fp32.
//
// Seven products instead of five bound it, with the elements between them:
// 4096 tokens (2500 + 1596, causal) x 64 heads of 128 take 24 + 545 to 610 + 16 us
// (statistics, gradients, join). The seven are 505 GFLOP: 0.83 to 0.93 PFLOP/s,
// where a large library product reaches 1.10 to 1.37, with the matrix unit 43% and
// the vector unit 32% busy at a clock of 2.0 GHz. With 64 values a head 12 + 370
// to 395 + 8 us, 0.64 to 0.68 PFLOP/s (33% and 40%).
// One launch for both kinds: the kind with the longer workgroups goes first
// and the other fills the units it leaves (in two launches dq's three products
// 218 us, 0.99 PFLOP/s, and the four of dk and dv 390 us, 0.74: a read from LDS
// feeds one product there, 1.7 LDS instructions a product).
#include "gqa.h"

#include <cmath>

namespace moe {
namespace gqa {
namespace {

struct BwdArgs {
  const uint16_t* dout;
  int64_t dout_ld;
  const uint16_t* q;
  int64_t q_ld;
  const uint16_t* k;
  int64_t k_ld;
  const uint16_t* v;
  int64_t v_ld;
  const uint16_t* out;
  int64_t out_ld;
  const float* lse;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, Tq, Tk, nh, nkv, causal;
  Div g;
  float scale;
  uint16_t* dq;
  int64_t dq_ld;
  uint16_t* dk;
  int64_t dk_ld;
  uint16_t* dv;
  int64_t dv_ld;
  float2* stats;          // [Tq, nh]: (lse in base 2, delta); a row without keys: (+inf, 0)
  float* part;            // [parts, Tk, nkv, 2, D]: dk (not scaled) and dv of each part
  int parts;
  int k_tiles, q_tiles;   // workgroups per key head (and part) of the two kinds
  int q_first;            // dq's workgroups come first
};

// D / 8 lanes per (token, head) row
template <int D>
__global__ __launch_bounds__(256) void bwd_stats_kernel(BwdArgs p) {
  constexpr int kL = D / 8;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / kL) + threadIdx.x / kL;
  if (row >= static_cast<int64_t>(p.Tq) * p.nh) return;
  const int64_t t = row / p.nh;
  const int h = static_cast<int>(row - t * p.nh);
  const int c = (threadIdx.x & (kL - 1)) * 8;
  const u32x4_t a = *reinterpret_cast<const u32x4_t*>(p.out + t * p.out_ld + h * D + c);
  const u32x4_t b = *reinterpret_cast<const u32x4_t*>(p.dout + t * p.dout_ld + h * D + c);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), s);
    s = fmaf(__uint_as_float(a[i] & 0xFFFF0000u), __uint_as_float(b[i] & 0xFFFF0000u), s);
  }
#pragma unroll
  for (int o = kL / 2; o >= 1; o >>= 1) s += __shfl_xor(s, o, kL);
  if ((threadIdx.x & (kL - 1)) == 0) {
    const float l = p.lse[row];
    const bool none = l == -INFINITY;
    p.stats[row] = none ? make_float2(INFINITY, 0.f) : make_float2(l * kLog2e, s);
  }
}

// Two sizes of a workgroup. Eight waves keep 128 keys and take the rows in
// stages of 64; four keep 64 keys, take stages of 32 and leave room for a
// second workgroup on the compute unit. The larger moves each row half as often
// into LDS, the smaller fills the chip with short sequences (waves_of).
constexpr int kTile = 64;                               // keys that pass by at a time (dq)
constexpr int kPass = 64 * 4 * 16;                      // weights of 32 x 32 in fp32
template <int D, int W>
struct Shape {
  static constexpr int kKeys = 16 * W;                  // keys of a workgroup: 32 a pair of waves
  static constexpr int kKept = 32 * W;                  // packed rows of a workgroup (dq)
  static constexpr int kRows = 8 * W;                   // rows of a stage (dk, dv)
  static constexpr int kBlocks = kRows / 32;
  // stages in LDS: of dO the one in use and those on their way; Q and the
  // statistics stay one stage longer
  static constexpr int kDoStages = W == 8 ? 2 : 3, kQStages = kDoStages + 1;
  static constexpr int kDoBytes = kRows * D * 2, kQBytes = kDoBytes + kRows * 8;
  static constexpr int kQPlace = kDoStages * kDoBytes, kPassPlace = kQPlace + kQStages * kQBytes;
  static constexpr int kPassBytes = W / 2 * kBlocks * kPass;
  static constexpr int kKvBytes = kPassPlace + 2 * kPassBytes;
  static constexpr int kQStage = 2 * kTile * D * 2;
  static constexpr int kBytes = kKvBytes > 2 * kQStage ? kKvBytes : 2 * kQStage;
};

// ---- dk, dv: a pair of waves keeps 32 keys (the lanes' columns), rows pass by ---
// The first wave of a pair has the keys: scores, weights, dv = p^T do. The
// second has their values: dp, ds with the weights that the first left in LDS
// (fp32, as they lie in its accumulator), dk = ds^T q. So both take the same
// steps on the two tiles the other way round, and a wave's operands and sums
// leave room for two waves a SIMD. The second wave is a stage behind the first
// with ds and dk: between two barriers neither waits for the other, and its
// products fill the time of the first one's exponentials (forward and backward
// of 8 x 300 tokens x 64 heads 140 -> 127 us, 2 x 2000 x 16 234 -> 222, with eight
// waves no change).
template <int D, int W>
__device__ __forceinline__ void bwd_kv(const BwdArgs& p, int head, int part, int tile_index, uint8_t* smem) {
  typedef Shape<D, W> Sh;
  constexpr int RB = D * 2, S = D / 16, C = D / 32, R = Sh::kRows;
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pair = wave & (W / 2 - 1);
  const bool has_keys = wave < W / 2;
  const SeqTile st = find_rows(p.cu_k, p.cu_q, p.B, p.Tk, p.Tq, 1, Sh::kKeys, tile_index);
  if (st.b < 0) return;
  const int n_k = st.n;
  const int q_start = st.start2, n_q = st.n2, n_rows = n_q * p.g.d;
  const int k0 = st.tile * Sh::kKeys;
  const int key = k0 + pair * 32 + (lane & 31);
  const int keyc = key < n_k ? key : n_k - 1;
  const int shift = p.causal ? n_k - n_q : n_k;                // query i sees keys <= i + shift
  auto first_row = [&](int j) { return clamp_int(j - shift, 0, n_q) * p.g.d; };   // that sees key j
  const int t_lo = first_row(k0) / R, t_hi = (n_rows + R - 1) / R;
  // Row tiles are taken from the last one down, every parts-th: all workgroups
  // of a head, whose first rows differ, start with the same ones and meet them
  // in the XCD's L2.
  const int t_top = t_hi - 1 - part;
  const int n_t = t_top >= t_lo ? (t_top - t_lo) / p.parts + 1 : 0;
  const int row_min = first_row(keyc);                         // rows before it do not see this lane's key

  const uint16_t* q = p.q + static_cast<int64_t>(q_start) * p.q_ld + head * p.g.d * D;
  const uint16_t* dout = p.dout + static_cast<int64_t>(q_start) * p.dout_ld + head * p.g.d * D;
  // statistics of the group's rows: l2 of a stage's rows, then delta of them;
  // behind the last row they are 0, as its q and dO are
  const __amdgpu_buffer_rsrc_t stats =
      buf_rsrc(p.stats + static_cast<int64_t>(q_start) * p.nh, static_cast<uint32_t>(n_q) * p.nh * 8u);
  constexpr int kLoads = 2 * R * RB / 1024 / W;          // of a wave and stage, without the statistics
  auto do_at = [&](int i) { return smem + i % Sh::kDoStages * Sh::kDoBytes; };
  auto q_at = [&](int i) { return smem + Sh::kQPlace + i % Sh::kQStages * Sh::kQBytes; };
  typedef EvenRows<RB, R, W> Rows;
  const bool even = Rows::fits(p.g);
  const Rows q_rows(q, p.q_ld, p.g, n_q, wave, lane), do_rows(dout, p.dout_ld, p.g, n_q, wave, lane);
  auto load = [&](int i) {
    const int t = t_top - i * p.parts;
    if (even) {
      q_rows.load(t, p.g, q_at(i), wave);
      do_rows.load(t, p.g, do_at(i), wave);
    } else {
      rows_load<RB, R, W>(q, p.q_ld, p.g, t * R, n_rows, q_at(i), wave, lane);
      rows_load<RB, R, W>(dout, p.dout_ld, p.g, t * R, n_rows, do_at(i), wave, lane);
    }
    if (wave == 0) {
#pragma unroll
      for (int x = 0; x < Sh::kBlocks; ++x) {
        const int at = x * 64 + lane, r = t * R + (at & (R - 1)), tok = quot(r, p.g);
        lds_load4_buf(stats, static_cast<uint32_t>(tok * p.nh + head * p.g.d + r - tok * p.g.d) * 8u + at / R * 4, 0,
                      q_at(i) + Sh::kDoBytes + x * 256);
      }
    }
  };
#pragma unroll
  for (int i = 0; i + 1 < Sh::kDoStages; ++i)
    if (i < n_t) load(i);

  bf16x8_t kept[S];
  {
    const int64_t tok = static_cast<int64_t>(st.start) + keyc;
    const uint16_t* x = (has_keys ? p.k + tok * p.k_ld : p.v + tok * p.v_ld) + head * D + 8 * g;
#pragma unroll
    for (int s = 0; s < S; ++s) kept[s] = *reinterpret_cast<const bf16x8_t*>(x + 16 * s);
  }
  // rows of one tile as they lie, columns of the other
  uint32_t row_off[S], col_off[C][2];
#pragma unroll
  for (int s = 0; s < S; ++s) row_off[s] = row_operand_offset<RB>(lane, s);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) col_off[c][h] = col_operand_offset<RB>(lane, c, h);
  auto pass_at = [&](int i) {
    return reinterpret_cast<f32x4_t*>(smem + Sh::kPassPlace + (i & 1) * Sh::kPassBytes + pair * Sh::kBlocks * kPass) +
           lane;
  };
  f32x16_t sum[C], x[Sh::kBlocks];
#pragma unroll
  for (int c = 0; c < C; ++c) sum[c] = f32x16_t{};

  // Stage i is in place (those behind it may be on their way), all waves are
  // done with their last step, and the next stage is asked for.
  auto next = [&](int i) __attribute__((always_inline)) {
    if (i < n_t) {
      const int ahead = min(Sh::kDoStages - 2, n_t - 1 - i);
      if (ahead <= 0) wait_vmcnt<0>();
      else wave == 0 ? wait_vmcnt<kLoads + Sh::kBlocks>() : wait_vmcnt<kLoads>();
    }
    static_assert(Sh::kDoStages <= 3, "at most one stage behind");
    lds_barrier();
    if (i + Sh::kDoStages - 1 < n_t) load(i + Sh::kDoStages - 1);
  };
  auto rows_product = [&](const uint8_t* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < Sh::kBlocks; ++b)
#pragma unroll
      for (int k = 0; k < S; ++k)
        x[b] = mfma(row_operand(buf, row_off[k] + b * 32 * RB), kept[k], k == 0 ? f32x16_t{} : x[b]);
  };
  auto add_columns = [&](const uint8_t* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < Sh::kBlocks; ++b)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bf16x8_t f = pack_operand(x[b], k);
#pragma unroll
        for (int c = 0; c < C; ++c)
          sum[c] = mfma(col_operand(buf, col_off[c][0] + (2 * b + k) * 16 * RB, col_off[c][1] + (2 * b + k) * 16 * RB),
                        f, sum[c]);
      }
  };
  if (has_keys) {
    const float c2 = p.scale * kLog2e;
    auto step = [&](int i, auto cut_c) __attribute__((always_inline)) {
      constexpr bool kCut = decltype(cut_c)::value;
      next(i);
      rows_product(q_at(i));
      const float* stat = reinterpret_cast<const float*>(q_at(i) + Sh::kDoBytes) + 4 * g;
      f32x4_t* pass = pass_at(i);
      const int r0 = (t_top - i * p.parts) * R + 4 * g;
#pragma unroll
      for (int b = 0; b < Sh::kBlocks; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4_t l2 = *reinterpret_cast<const f32x4_t*>(stat + 32 * b + 8 * j);
          f32x4_t w;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[e] = exp2_hw(fmaf(x[b][4 * j + e], c2, -l2[e]));
            if constexpr (kCut) w[e] = r0 + 32 * b + 8 * j + e < row_min ? 0.f : w[e];
            x[b][4 * j + e] = w[e];
          }
          pass[(4 * b + j) * 64] = w;
        }
      add_columns(do_at(i));
    };
    // the tiles that the causal mask cuts come last
    const int cut_hi = p.causal ? (first_row(min(k0 + Sh::kKeys, n_k) - 1) + R - 1) / R : 0;
    const int n_whole = t_top >= cut_hi ? min(n_t, (t_top - cut_hi) / p.parts + 1) : 0;
    int i = 0;
    for (; i < n_whole; ++i) step(i, std::false_type{});
    for (; i < n_t; ++i) step(i, std::true_type{});
    next(n_t);
  } else {
    for (int i = 0; i <= n_t; ++i) {
      next(i);
      if (i > 0) {
        const float* stat = reinterpret_cast<const float*>(q_at(i - 1) + Sh::kDoBytes) + R + 4 * g;
        const f32x4_t* pass = pass_at(i - 1);
#pragma unroll
        for (int b = 0; b < Sh::kBlocks; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4_t delta = *reinterpret_cast<const f32x4_t*>(stat + 32 * b + 8 * j);
            const f32x4_t w = pass[(4 * b + j) * 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[b][4 * j + e] = w[e] * (x[b][4 * j + e] - delta[e]);
          }
        add_columns(q_at(i - 1));
      }
      if (i < n_t) rows_product(do_at(i));
    }
  }

  lds_barrier();                        // everyone is done with the tiles
  const int64_t tok = static_cast<int64_t>(st.start) + k0 + pair * 32;
  const int n_out = n_k - k0 - pair * 32;
  static_assert(W * result_bytes<RB>() <= Sh::kBytes, "results fit the tile buffers");
  if (p.parts == 1) {
    uint8_t* rows = smem + wave * result_bytes<RB>();
    const float sc = has_keys ? 1.f : p.scale;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint2*>(rows + (lane & 31) * (RB + 16) + (32 * c + 8 * j + 4 * g) * 2) =
            pack4(sum[c][4 * j] * sc, sum[c][4 * j + 1] * sc, sum[c][4 * j + 2] * sc, sum[c][4 * j + 3] * sc);
    const int64_t ld = has_keys ? p.dv_ld : p.dk_ld;
    store_rows<RB>(rows, (has_keys ? p.dv : p.dk) + tok * ld + head * D, ld * 2, n_out, lane);
  } else if ((lane & 31) < n_out) {
    float* dst = p.part + (((static_cast<int64_t>(part) * p.Tk + tok + (lane & 31)) * p.nkv + head) * 2 +
                           (has_keys ? 1 : 0)) * D + 4 * g;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<f32x4_t*>(dst + 32 * c + 8 * j) =
            f32x4_t{sum[c][4 * j], sum[c][4 * j + 1], sum[c][4 * j + 2], sum[c][4 * j + 3]};
  }
}

// ---- dq: a wave keeps 32 packed rows (the lanes' columns), keys pass by --------
template <int D, int W>
__device__ __forceinline__ void bwd_q(const BwdArgs& p, int head, int tile_index, uint8_t* smem) {
  constexpr int RB = D * 2, S = D / 16, C = D / 32;
  constexpr int kV = kTile * RB;                        // V's place behind K's
  constexpr int kStage = Shape<D, W>::kQStage, kKept = Shape<D, W>::kKept;
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const SeqTile st = find_rows(p.cu_q, p.cu_k, p.B, p.Tq, p.Tk, p.g.d, kKept, tile_index);
  if (st.b < 0) return;
  const int k_start = st.start2, n_k = st.n2;
  const int n_rows = st.n, n_q = quot(n_rows, p.g);
  const int r0 = st.tile * kKept;
  const int row = r0 + wave * 32 + (lane & 31);
  const int rowc = row < n_rows ? row : n_rows - 1;
  const int tok = quot(rowc, p.g), sub = rowc - tok * p.g.d;
  const int shift = p.causal ? n_k - n_q : n_k;
  auto last_of = [&](int r) {
    return p.causal ? min(quot(min(r, n_rows - 1), p.g) + shift, n_k - 1) : n_k - 1;
  };
  const int last = p.causal ? min(tok + shift, n_k - 1) : n_k - 1;
  const int first_last = last_of(r0), tile_last = last_of(r0 + kKept - 1);
  const int n_kt = tile_last < 0 ? 0 : tile_last / kTile + 1;
  const int n_full = first_last < 0 ? 0 : min(n_kt, (first_last + 1) / kTile);   // tiles that every row sees whole

  const uint16_t* kb = p.k + static_cast<int64_t>(k_start) * p.k_ld + head * D;
  const uint16_t* vb = p.v + static_cast<int64_t>(k_start) * p.v_ld + head * D;
  auto load = [&](int kt, uint8_t* buf) {
    const int n = n_k - kt * kTile;
    const int nv = n < kTile ? n : kTile;
    tile_load<RB, kTile, W>(kb + static_cast<int64_t>(kt) * kTile * p.k_ld, static_cast<uint32_t>(p.k_ld * 2), nv,
                                 buf, wave, lane);
    tile_load<RB, kTile, W>(vb + static_cast<int64_t>(kt) * kTile * p.v_ld, static_cast<uint32_t>(p.v_ld * 2), nv,
                                 buf + kV, wave, lane);
  };
  if (n_kt > 0) load(0, smem);

  const int64_t tokc = static_cast<int64_t>(st.start) + tok;
  const int h = head * p.g.d + sub;
  bf16x8_t qf[S], df[S];
  {
    const uint16_t* q = p.q + tokc * p.q_ld + h * D + 8 * g;
    const uint16_t* d = p.dout + tokc * p.dout_ld + h * D + 8 * g;
#pragma unroll
    for (int s = 0; s < S; ++s) qf[s] = *reinterpret_cast<const bf16x8_t*>(q + 16 * s);
#pragma unroll
    for (int s = 0; s < S; ++s) df[s] = *reinterpret_cast<const bf16x8_t*>(d + 16 * s);
  }
  const float2 stat = p.stats[tokc * p.nh + h];
  uint32_t row_off[S], col_off[C][2];
#pragma unroll
  for (int s = 0; s < S; ++s) row_off[s] = row_operand_offset<RB>(lane, s);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int k = 0; k < 2; ++k) col_off[c][k] = col_operand_offset<RB>(lane, c, k);
  f32x16_t dq[C];
#pragma unroll
  for (int c = 0; c < C; ++c) dq[c] = f32x16_t{};
  const float c2 = p.scale * kLog2e;

  auto tile = [&](int kt, auto cut_c) __attribute__((always_inline)) {
    constexpr bool kCut = decltype(cut_c)::value;
    wait_vmcnt<0>();
    lds_barrier();
    uint8_t* buf = smem + (kt & 1) * kStage;
    if (kt + 1 < n_kt) load(kt + 1, smem + ((kt + 1) & 1) * kStage);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f32x16_t s, dp;
#pragma unroll
      for (int k = 0; k < S; ++k) {
        s = mfma(row_operand(buf, row_off[k] + b * 32 * RB), qf[k], k == 0 ? f32x16_t{} : s);
        dp = mfma(row_operand(buf, row_off[k] + kV + b * 32 * RB), df[k], k == 0 ? f32x16_t{} : dp);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = exp2_hw(fmaf(s[i], c2, -stat.x)) * (dp[i] - stat.y);
        if constexpr (kCut) s[i] = kt * kTile + 32 * b + 8 * (i >> 2) + 4 * g + (i & 3) > last ? 0.f : s[i];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bf16x8_t f = pack_operand(s, k);
#pragma unroll
        for (int c = 0; c < C; ++c)
          dq[c] = mfma(col_operand(buf, col_off[c][0] + (2 * b + k) * 16 * RB, col_off[c][1] + (2 * b + k) * 16 * RB),
                       f, dq[c]);
      }
    }
  };
  int kt = 0;
  for (; kt < n_full; ++kt) tile(kt, std::false_type{});
  for (; kt < n_kt; ++kt) tile(kt, std::true_type{});

  lds_barrier();                        // everyone is done with the tiles
  uint8_t* rows = smem + wave * result_bytes<RB>();
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float sc = p.scale;
      *reinterpret_cast<uint2*>(rows + (lane & 31) * (RB + 16) + (32 * c + 8 * i + 4 * g) * 2) =
          pack4(dq[c][4 * i] * sc, dq[c][4 * i + 1] * sc, dq[c][4 * i + 2] * sc, dq[c][4 * i + 3] * sc);
    }
  store_packed<RB>(rows, p.dq + static_cast<int64_t>(st.start) * p.dq_ld + head * p.g.d * D, p.dq_ld, p.g,
                   r0 + wave * 32, n_rows, lane);
}

// Both kinds in one launch: the second fills the compute units that the
// first's last workgroups leave, and short sequences need both to fill the
// chip. The kind whose workgroups walk more tiles comes first. Heads run
// fastest (an XCD keeps to its own where their number is a multiple of 8); the
// tiles that see most come first.
template <int D, int W>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2, 2)))
void bwd_kernel(BwdArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[Shape<D, W>::kBytes];
  const int n_kv = p.k_tiles * p.nkv * p.parts, n_q = p.q_tiles * p.nkv;
  const int id = blockIdx.x;
  const int head = id % p.nkv;
  if (p.q_first ? id >= n_q : id < n_kv) {
    const int r = (p.q_first ? id - n_q : id) / p.nkv;
    bwd_kv<D, W>(p, head, r % p.parts, r / p.parts, smem);
  } else {
    bwd_q<D, W>(p, head, p.q_tiles - 1 - (p.q_first ? id : id - n_kv) / p.nkv, smem);
  }
}

// ---- dk, dv: the parts' sum, in order ------------------------------------------
// Only rows that a sequence holds.
template <int D>
__global__ __launch_bounds__(256) void bwd_join_kernel(BwdArgs p) {
  const int lo = clamp_int(p.cu_k[0], 0, p.Tk), hi = clamp_int(p.cu_k[p.B], lo, p.Tk);
  constexpr int kL = 2 * D / 4;                          // lanes a (token, head)
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (256 / kL) + threadIdx.x / kL;
  const int64_t t = unit / p.nkv;
  const int head = static_cast<int>(unit - t * p.nkv);
  if (t < lo || t >= hi) return;
  const int c = (threadIdx.x & (kL - 1)) * 4;            // of (dk | dv)
  const float* src = p.part + unit * 2 * D + c;
  const int64_t step = static_cast<int64_t>(p.Tk) * p.nkv * 2 * D;
  f32x4_t s = *reinterpret_cast<const f32x4_t*>(src);
#pragma unroll 4
  for (int i = 1; i < p.parts; ++i) {
    const f32x4_t x = *reinterpret_cast<const f32x4_t*>(src + i * step);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] += x[j];
  }
  if (c < D)
    *reinterpret_cast<uint2*>(p.dk + t * p.dk_ld + head * D + c) =
        pack4(s[0] * p.scale, s[1] * p.scale, s[2] * p.scale, s[3] * p.scale);
  else
    *reinterpret_cast<uint2*>(p.dv + t * p.dv_ld + head * D + c - D) = pack4(s[0], s[1], s[2], s[3]);
}

// Eight waves a workgroup where there are many rows (tokens x heads) and long
// sequences. Forward and backward in us, eight / four waves, 128 values a head:
// 4096 tokens in 2 sequences x 64 heads 725 / 768, 3500 in 2 x 32 287 / 321, 1500
// x 64 228 / 246; but 4096 x 16 400 / 363, 5 x 800 x 64 351 / 323, 8 x 300 x 64
// 155 / 129, 512 x 128 111 / 84. (64 values a head follow the same rule and were
// not measured on both sides; the sequences' mean length counts.)
constexpr int kManyRows = 90000, kLong = 1200;
int waves_of(int B, int Tq, int Tk, int nh) {
  return static_cast<int64_t>(Tq) * nh >= kManyRows && Tk / B >= kLong ? 8 : 4;
}
// Parts that the rows of a key tile are cut into: enough workgroups for two a
// compute unit, as far as a part keeps 12 stages of rows in the mean (forward
// and backward of 600 tokens x 4 heads 43 us, with 4 stages 49; 385 x 16 heads
// 38.6 and 42; 200 x 32 heads 35 and 33).
constexpr int kMaxParts = 32;
int parts_of(int w, int Tq, int Tk, int nh, int nkv) {
  if (Tk == 0) return 1;                                 // no dk and dv to add up: nothing for a join to do
  const int64_t wgs = (static_cast<int64_t>(Tk) + 16 * w - 1) / (16 * w) * nkv;
  const int64_t tiles = static_cast<int64_t>(Tq) * (nh / nkv) / (96 * w);
  int64_t n = 2 * kNumCu / wgs;
  n = n < tiles ? n : tiles;
  return n < 1 ? 1 : (n > kMaxParts ? kMaxParts : static_cast<int>(n));
}
// Rows of the parts' sums: parts_of never brings them above either bound, and
// both grow with the sizes, so a workspace serves every smaller call.
size_t part_rows(int Tk, int nkv) {
  const size_t all = size_t{kMaxParts} * Tk * nkv, most = size_t{2} * kNumCu * 128;
  return all < most ? all : most;
}
size_t stats_bytes(int Tq, int nh) { return (static_cast<size_t>(Tq) * nh * 8 + 255) & ~size_t{255}; }

template <int D>
void launch_bwd(BwdArgs a, int waves, hipStream_t stream) {
  if (a.Tq > 0) {
    const int64_t rows = static_cast<int64_t>(a.Tq) * a.nh;
    constexpr int kPer = 256 / (D / 8);
    hipLaunchKernelGGL(bwd_stats_kernel<D>, dim3(static_cast<unsigned>((rows + kPer - 1) / kPer)), dim3(256), 0, stream,
                       a);
  }
  a.k_tiles = a.Tk > 0 ? a.Tk / (16 * waves) + (a.B < a.Tk ? a.B : a.Tk) : 0;
  a.q_tiles = a.Tq > 0 ? a.Tq * a.g.d / (32 * waves) + (a.B < a.Tq ? a.B : a.Tq) : 0;
  const dim3 grid(static_cast<unsigned>(a.k_tiles * a.parts + a.q_tiles) * a.nkv);
  if (waves == 8) hipLaunchKernelGGL((bwd_kernel<D, 8>), grid, dim3(512), 0, stream, a);
  else hipLaunchKernelGGL((bwd_kernel<D, 4>), grid, dim3(256), 0, stream, a);
  if (a.parts > 1) {
    constexpr int kPer = 256 / (D / 2);
    const int64_t units = static_cast<int64_t>(a.Tk) * a.nkv;
    hipLaunchKernelGGL(bwd_join_kernel<D>, dim3(static_cast<unsigned>((units + kPer - 1) / kPer)), dim3(256), 0,
                       stream, a);
  }
}

}  // namespace
}  // namespace gqa
}  // namespace moe

extern "C" size_t moe_gqa_attn_bwd_workspace(int Tq, int Tk, int n_heads, int n_kv_heads, int head_dim) {
  if (Tq < 0 || Tk < 0 || Tq > (1 << 27) || Tk > (1 << 27) || n_heads < 1 || n_heads > 1024 || n_kv_heads < 1 ||
      n_heads % n_kv_heads != 0 || (head_dim != 64 && head_dim != 128))
    return 0;
  return moe::gqa::stats_bytes(Tq, n_heads) + moe::gqa::part_rows(Tk, n_kv_heads) * 2 * head_dim * 4;
}

extern "C" int moe_gqa_attn_bwd(const void* dout, int64_t dout_ld, const void* q, int64_t q_ld, const void* k,
                                int64_t k_ld, const void* v, int64_t v_ld, int fmt, const void* out, int64_t out_ld,
                                const float* lse, const int32_t* cu_q, const int32_t* cu_k, int B, int Tq, int Tk,
                                int n_heads, int n_kv_heads, int head_dim, int causal, float scale, void* dq,
                                int64_t dq_ld, void* dk, int64_t dk_ld, void* dv, int64_t dv_ld, void* ws,
                                size_t ws_bytes, hipStream_t stream) {
  using namespace moe;
  using namespace moe::gqa;
  clear_error();
  const char* fn = "moe_gqa_attn_bwd";
  if (const int rc = check_heads(fn, fmt, n_heads, n_kv_heads, head_dim)) return rc;
  if (const int rc = check_sequences(fn, B, Tq, Tk, n_heads, causal, scale)) return rc;
  const int64_t q_row = static_cast<int64_t>(n_heads) * head_dim, k_row = static_cast<int64_t>(n_kv_heads) * head_dim;
  const struct { const char* name; int64_t ld, row; } lds[] = {
      {"dout_ld", dout_ld, q_row}, {"q_ld", q_ld, q_row}, {"k_ld", k_ld, k_row}, {"v_ld", v_ld, k_row},
      {"out_ld", out_ld, q_row}, {"dq_ld", dq_ld, q_row}, {"dk_ld", dk_ld, k_row}, {"dv_ld", dv_ld, k_row}};
  for (const auto& x : lds)
    if (const int rc = check_ld(fn, x.name, x.ld, x.row)) return rc;
  if (B == 0 || (Tq == 0 && Tk == 0)) return MOE_OK;
  MOE_REQUIRE(cu_q && cu_k && (Tq == 0 || (dout && q && out && lse && dq)) && (Tk == 0 || (k && v && dk && dv)),
              MOE_ERR_INVALID_ARG, "moe_gqa_attn_bwd: null pointer");
  MOE_REQUIRE(aligned16(dout) && aligned16(q) && aligned16(k) && aligned16(v) && aligned16(out) && aligned16(dq) &&
                  aligned16(dk) && aligned16(dv) && aligned16(ws),
              MOE_ERR_ALIGNMENT, "moe_gqa_attn_bwd: tensors and ws must be 16-byte aligned");
  const size_t need = moe_gqa_attn_bwd_workspace(Tq, Tk, n_heads, n_kv_heads, head_dim);
  MOE_REQUIRE(need == 0 || (ws && ws_bytes >= need), MOE_ERR_WORKSPACE,
              "moe_gqa_attn_bwd: ws smaller than moe_gqa_attn_bwd_workspace(...)");
  BwdArgs a{};
  a.dout = static_cast<const uint16_t*>(dout), a.dout_ld = dout_ld;
  a.q = static_cast<const uint16_t*>(q), a.q_ld = q_ld;
  a.k = static_cast<const uint16_t*>(k), a.k_ld = k_ld;
  a.v = static_cast<const uint16_t*>(v), a.v_ld = v_ld;
  a.out = static_cast<const uint16_t*>(out), a.out_ld = out_ld;
  a.lse = lse, a.cu_q = cu_q, a.cu_k = cu_k;
  a.B = B, a.Tq = Tq, a.Tk = Tk, a.nh = n_heads, a.nkv = n_kv_heads, a.causal = causal, a.scale = scale;
  a.g = make_div(n_heads / n_kv_heads);
  a.dq = static_cast<uint16_t*>(dq), a.dq_ld = dq_ld;
  a.dk = static_cast<uint16_t*>(dk), a.dk_ld = dk_ld;
  a.dv = static_cast<uint16_t*>(dv), a.dv_ld = dv_ld;
  a.stats = static_cast<float2*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + stats_bytes(Tq, n_heads));
  const int waves = waves_of(B, Tq, Tk, n_heads);
  a.parts = parts_of(waves, Tq, Tk, n_heads, n_kv_heads);
  // the kind with the longer workgroups first (8 x 300 tokens x 64 heads, forward
  // and backward: 127 us, dq always first 160; short sequences in parts 31, dk and
  // dv always first 34)
  a.q_first = static_cast<int64_t>(Tq) * a.g.d / a.parts < Tk;
  if (head_dim == 128) launch_bwd<128>(a, waves, stream);
  else launch_bwd<64>(a, waves, stream);
  return check_launch(fn);
}
