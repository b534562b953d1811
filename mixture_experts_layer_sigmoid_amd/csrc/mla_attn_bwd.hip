// moe_mla_attn_bwd: gradients of moe_mla_attn_fwd.
//
// With p the softmax weights, do the output's gradient:
//   delta[i] = do[i] . out[i]          (= sum_j p[i, j] dp[i, j])
//   dp = do v^T,  ds = p (dp - delta),  dv = p^T do
//   dq = scale ds k,  dk = scale ds^T q,  dk_rope = sum over heads of dk's
//   rotary columns
// p is computed again from the scores and the forward's lse.
//
// Four launches: the row statistics (lse in base 2, delta); one that keeps
// 32 keys a wave and walks the queries (dk, dv); one that keeps 32 queries a
// wave and walks the keys (dq); the sum of the heads' rotary gradients. The
// scores are computed twice, so nothing is added up by atomics and the
// result does not depend on the order in which workgroups run.
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
  int n_tiles;
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

// ---- dk, dv: a wave keeps 32 keys (the lanes' columns), queries pass by ------
constexpr int kQTile = 64;
constexpr int kKvWaves = 4;
constexpr int kKvKeys = 32 * kKvWaves;
constexpr int kLdsQn = kQTile * kDn * 2, kLdsQr = kQTile * kDr * 2, kLdsDo = kQTile * kDv * 2;
constexpr int kLdsStat = kQTile * 8;
constexpr int kLdsKvStage = kLdsQn + kLdsQr + kLdsDo + kLdsStat;

__global__ __launch_bounds__(64 * kKvWaves) __attribute__((amdgpu_waves_per_eu(1, 1)))
void bwd_kv_kernel(BwdArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kLdsKvStage];
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int idx = xcd_contiguous(blockIdx.x, gridDim.x);
  const int head = idx / p.n_tiles;
  const SeqTile st = find_tile(p.cu_k, p.B, p.Tk, kKvKeys, idx % p.n_tiles);
  if (st.b < 0) return;
  const int n_k = st.n;
  const int q_start = clamp_int(p.cu_q[st.b], 0, p.Tq);
  const int n_q = clamp_int(p.cu_q[st.b + 1], q_start, p.Tq) - q_start;
  const int k0 = st.tile * kKvKeys;
  const int key = k0 + wave * 32 + (lane & 31);
  const int keyc = key < n_k ? key : n_k - 1;
  const int wave_last = min(k0 + wave * 32 + 31, n_k - 1);     // its last key
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
  uint32_t ro256[8], ro128[4], co256[4][2], co128[2][2];
#pragma unroll
  for (int s = 0; s < 8; ++s) ro256[s] = row_operand_offset<256>(lane, s);
#pragma unroll
  for (int s = 0; s < 4; ++s) ro128[s] = kLdsQn + row_operand_offset<128>(lane, s);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int c = 0; c < 4; ++c) co256[c][h] = col_operand_offset<256>(lane, c, h);
#pragma unroll
    for (int c = 0; c < 2; ++c) co128[c][h] = kLdsQn + col_operand_offset<128>(lane, c, h);
  }
  f32x16_t dk[6], dv[4];
#pragma unroll
  for (int c = 0; c < 6; ++c) dk[c] = f32x16_t{};
#pragma unroll
  for (int c = 0; c < 4; ++c) dv[c] = f32x16_t{};
  const float c2 = p.scale * kLog2e;

  for (int t = t_first; t < t_end; ++t) {
    uint8_t* buf = smem + ((t - t_first) & 1) * kLdsKvStage;
    put_stats(buf);                   // the other buffer's readers are a barrier behind
    wait_vmcnt<0>();
    lds_barrier();
    if (t + 1 < t_end) load(t + 1, smem + ((t + 1 - t_first) & 1) * kLdsKvStage);
    const uint8_t* dob = buf + kLdsQn + kLdsQr;
    const float* stat = reinterpret_cast<const float*>(dob + kLdsDo);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f32x16_t s = f32x16_t{}, dp = f32x16_t{};
#pragma unroll
      for (int k = 0; k < 8; ++k) s = mfma(row_operand(buf, ro256[k] + b * 32 * 256), kf[k], s);
#pragma unroll
      for (int k = 0; k < 4; ++k) s = mfma(row_operand(buf, ro128[k] + b * 32 * 128), kf[8 + k], s);
#pragma unroll
      for (int k = 0; k < 8; ++k) dp = mfma(row_operand(dob, ro256[k] + b * 32 * 256), vf[k], dp);
      const int q0 = t * kQTile + 32 * b;
      const bool cut = p.causal && q0 + shift < wave_last;
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        const f32x4_t l2 = *reinterpret_cast<const f32x4_t*>(stat + 32 * b + 8 * i4 + 4 * g);
        const f32x4_t dl = *reinterpret_cast<const f32x4_t*>(stat + 64 + 32 * b + 8 * i4 + 4 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 4 * i4 + e;
          s[i] = exp2_hw(fmaf(s[i], c2, -l2[e]));
          dp[i] = s[i] * (dp[i] - dl[e]);
        }
      }
      if (cut) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (key > q0 + 8 * (i >> 2) + 4 * g + (i & 3) + shift) {
            s[i] = 0.f;
            dp[i] = 0.f;
          }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bf16x8_t pf = pack_operand(s, k), sf = pack_operand(dp, k);
        const int o256 = (2 * b + k) * 16 * 256, o128 = (2 * b + k) * 16 * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) dv[c] = mfma(col_operand(dob, co256[c][0] + o256, co256[c][1] + o256), pf, dv[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) dk[c] = mfma(col_operand(buf, co256[c][0] + o256, co256[c][1] + o256), sf, dk[c]);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          dk[4 + c] = mfma(col_operand(buf, co128[c][0] + o128, co128[c][1] + o128), sf, dk[4 + c]);
      }
    }
  }
  if (key >= n_k) return;
  const int64_t tok = static_cast<int64_t>(st.start) + key;
  uint16_t* o = p.dkv + tok * p.dkv_ld + head * (kDn + kDv) + 4 * g;
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float sc = p.scale;
      *reinterpret_cast<uint2*>(o + 32 * c + 8 * i) =
          pack4(dk[c][4 * i] * sc, dk[c][4 * i + 1] * sc, dk[c][4 * i + 2] * sc, dk[c][4 * i + 3] * sc);
      *reinterpret_cast<uint2*>(o + kDn + 32 * c + 8 * i) =
          pack4(dv[c][4 * i], dv[c][4 * i + 1], dv[c][4 * i + 2], dv[c][4 * i + 3]);
    }
  float* r = p.dkr_part + (static_cast<int64_t>(head) * p.Tk + tok) * kDr + 4 * g;
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f32x4_t*>(r + 32 * c + 8 * i) =
          f32x4_t{dk[4 + c][4 * i], dk[4 + c][4 * i + 1], dk[4 + c][4 * i + 2], dk[4 + c][4 * i + 3]};
}

// ---- dq: a wave keeps 32 queries (the lanes' columns), keys pass by ----------
constexpr int kKt = 64;
constexpr int kLdsKn = kKt * kDn * 2, kLdsKr = kKt * kDr * 2, kLdsV = kKt * kDv * 2;
constexpr int kLdsQStage = kLdsKn + kLdsKr + kLdsV;

template <int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2)))
void bwd_q_kernel(BwdArgs p) {
  constexpr int kQt = 32 * NW;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kLdsQStage];
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int idx = xcd_contiguous(blockIdx.x, gridDim.x);
  const int head = idx / p.n_tiles;
  const SeqTile st = find_tile(p.cu_q, p.B, p.Tq, kQt, p.n_tiles - 1 - idx % p.n_tiles);
  if (st.b < 0) return;
  const int k_start = clamp_int(p.cu_k[st.b], 0, p.Tk);
  const int n_k = clamp_int(p.cu_k[st.b + 1], k_start, p.Tk) - k_start;
  const int n_q = st.n;
  const int w0 = st.tile * kQt + wave * 32;
  const int row = w0 + (lane & 31);
  const int rowc = row < n_q ? row : n_q - 1;
  const int shift = p.causal ? n_k - n_q : n_k;
  const int last = p.causal ? min(rowc + shift, n_k - 1) : n_k - 1;
  const int wave_first = p.causal ? min(min(w0, n_q - 1) + shift, n_k - 1) : n_k - 1;
  const int wave_last = p.causal ? min(min(w0 + 31, n_q - 1) + shift, n_k - 1) : n_k - 1;
  const int tile_last = p.causal ? min(min(st.tile * kQt + kQt, n_q) - 1 + shift, n_k - 1) : n_k - 1;
  const int n_kt = tile_last < 0 ? 0 : tile_last / kKt + 1;

  const uint16_t* kv = p.kv + static_cast<int64_t>(k_start) * p.kv_ld + head * (kDn + kDv);
  const uint16_t* kr = p.kr + static_cast<int64_t>(k_start) * p.kr_ld;
  auto load = [&](int kt, uint8_t* buf) {
    const int n = n_k - kt * kKt;
    const int nv = n < kKt ? n : kKt;
    const uint16_t* b = kv + static_cast<int64_t>(kt) * kKt * p.kv_ld;
    const uint32_t ld = static_cast<uint32_t>(p.kv_ld * 2);
    tile_load<256, kKt, NW>(b, ld, nv, buf, wave, lane);
    tile_load<128, kKt, NW>(kr + static_cast<int64_t>(kt) * kKt * p.kr_ld, static_cast<uint32_t>(p.kr_ld * 2), nv,
                            buf + kLdsKn, wave, lane);
    tile_load<256, kKt, NW>(b + kDn, ld, nv, buf + kLdsKn + kLdsKr, wave, lane);
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
  uint32_t ro256[8], ro128[4], co256[4][2], co128[2][2];
#pragma unroll
  for (int s = 0; s < 8; ++s) ro256[s] = row_operand_offset<256>(lane, s);
#pragma unroll
  for (int s = 0; s < 4; ++s) ro128[s] = kLdsKn + row_operand_offset<128>(lane, s);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int c = 0; c < 4; ++c) co256[c][h] = col_operand_offset<256>(lane, c, h);
#pragma unroll
    for (int c = 0; c < 2; ++c) co128[c][h] = kLdsKn + col_operand_offset<128>(lane, c, h);
  }
  f32x16_t dq[6];
#pragma unroll
  for (int c = 0; c < 6; ++c) dq[c] = f32x16_t{};
  const float c2 = p.scale * kLog2e;

  for (int kt = 0; kt < n_kt; ++kt) {
    wait_vmcnt<0>();
    lds_barrier();
    uint8_t* buf = smem + (kt & 1) * kLdsQStage;
    if (kt + 1 < n_kt) load(kt + 1, smem + ((kt + 1) & 1) * kLdsQStage);
    const int t0 = kt * kKt;
    if (t0 > wave_last) continue;
    const uint8_t* vb = buf + kLdsKn + kLdsKr;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f32x16_t s = f32x16_t{}, dp = f32x16_t{};
#pragma unroll
      for (int k = 0; k < 8; ++k) s = mfma(row_operand(buf, ro256[k] + b * 32 * 256), qf[k], s);
#pragma unroll
      for (int k = 0; k < 4; ++k) s = mfma(row_operand(buf, ro128[k] + b * 32 * 128), qf[8 + k], s);
#pragma unroll
      for (int k = 0; k < 8; ++k) dp = mfma(row_operand(vb, ro256[k] + b * 32 * 256), df[k], dp);
#pragma unroll
      for (int i = 0; i < 16; ++i) dp[i] = exp2_hw(fmaf(s[i], c2, -stat.x)) * (dp[i] - stat.y);
      if (t0 + 32 * b + 31 > wave_first) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (t0 + 32 * b + 8 * (i >> 2) + 4 * g + (i & 3) > last) dp[i] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bf16x8_t sf = pack_operand(dp, k);
        const int o256 = (2 * b + k) * 16 * 256, o128 = (2 * b + k) * 16 * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) dq[c] = mfma(col_operand(buf, co256[c][0] + o256, co256[c][1] + o256), sf, dq[c]);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          dq[4 + c] = mfma(col_operand(buf, co128[c][0] + o128, co128[c][1] + o128), sf, dq[4 + c]);
      }
    }
  }
  if (row >= n_q) return;
  uint16_t* o = p.dq + tokc * p.dq_ld + head * kDq + 4 * g;
#pragma unroll
  for (int c = 0; c < 6; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float sc = p.scale;
      *reinterpret_cast<uint2*>(o + 32 * c + 8 * i) =
          pack4(dq[c][4 * i] * sc, dq[c][4 * i + 1] * sc, dq[c][4 * i + 2] * sc, dq[c][4 * i + 3] * sc);
    }
}

// ---- dk_rope[t] = scale * sum over heads, in head order ----------------------
// A workgroup takes 4 tokens: 16 lanes x 4 values a token, 4 groups of heads
// whose sums are joined in a fixed order. Only rows that a sequence holds.
__global__ __launch_bounds__(256) void bwd_rope_kernel(BwdArgs p) {
  __shared__ f32x4_t part[4][64];
  const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
  const int lo = clamp_int(p.cu_k[0], 0, p.Tk), hi = clamp_int(p.cu_k[p.B], lo, p.Tk);
  const int t = lo + blockIdx.x * 4 + (lane >> 4);
  f32x4_t s = {0.f, 0.f, 0.f, 0.f};
  if (t < hi) {
    const float* src = p.dkr_part + static_cast<int64_t>(t) * kDr + (lane & 15) * 4;
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
    *reinterpret_cast<uint2*>(p.dkr + static_cast<int64_t>(t) * p.dkr_ld + (lane & 15) * 4) =
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
  if (Tk > 0) {
    a.n_tiles = seq_tiles_bound(B, Tk, kKvKeys);
    hipLaunchKernelGGL(bwd_kv_kernel, dim3(static_cast<unsigned>(a.n_tiles) * n_heads), dim3(64 * kKvWaves), 0,
                       stream, a);
    hipLaunchKernelGGL(bwd_rope_kernel, dim3((Tk + 3) / 4), dim3(256), 0, stream, a);
  }
  if (Tq > 0) {
    auto launch = [&](auto kern, int nw) {
      a.n_tiles = seq_tiles_bound(B, Tq, 32 * nw);
      hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(a.n_tiles) * n_heads), dim3(64 * nw), 0, stream, a);
    };
    if (Tq / B >= 512) launch(bwd_q_kernel<8>, 8);
    else launch(bwd_q_kernel<4>, 4);
  }
  return check_launch(fn);
}
