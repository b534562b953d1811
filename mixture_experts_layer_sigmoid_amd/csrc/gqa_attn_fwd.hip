// moe_gqa_attn_fwd: attention over packed sequences, grouped heads.
//
// Per query head h of key head h / G and packed sequence:
//   s[i, j] = scale * q[i, h] . k[j, h / G]
//   out[i, h] = sum_j softmax_j(s[i, :]) v[j, h / G],  lse[i, h] = log sum_j e^s
// over the keys the mask leaves; a row without keys has out 0 and lse -inf.
//
// One pass over the keys with a running reference and sum (fp32). A wave keeps
// 32 packed rows (tokens x heads of a group) as the columns of its
// accumulators: the scores are computed as k q^T, so a row's statistics belong
// to one lane and its mirror, and the weights in the accumulator are the next
// product's operand without moving. The weights are rounded to bf16, as the
// matrix instruction takes them; their sum is taken before that rounding.
//
// The power limit bounds it: 6144 queries x 64 heads of 128 over up to 9216 keys
// take 616 to 730 us by card and run, 0.92 to 1.08 PFLOP/s, with the matrix unit
// 55% and the vector unit 49% busy at a clock of 1.6 to 1.7 GHz instead of 2.4 (an
// 8192^3 library product reaches 1.10 to 1.37 PFLOP/s). With 64 values a head the
// products halve and the elements do not (11 vector instructions a product
// instead of 6): 4000 tokens x 64 heads take 164 to 192 us, 0.68 to 0.80 PFLOP/s,
// vector unit 62%, matrix unit 37% busy. Two workgroups of four waves a compute
// unit put one wave's exponentials beside another's products; within +-2% of
// it are eight waves a workgroup and raised priorities, slower are 64 rows a
// wave at one wave a SIMD (709) and products and softmax of neighbouring tiles
// interleaved in one wave (773).
#include "gqa.h"

#include <cmath>

namespace moe {
namespace gqa {
namespace {

struct FwdArgs {
  const uint16_t* q;
  int64_t q_ld;
  const uint16_t* k;
  int64_t k_ld;
  const uint16_t* v;
  int64_t v_ld;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, Tq, Tk, nh, nkv, causal;
  Div g;
  float scale;
  uint16_t* out;
  int64_t out_ld;
  float* lse;
  int n_tiles;
  int parts;               // of a sequence's keys, each a workgroup's
  float* part;             // [parts, Tq, nh, D]: sums of each part, not normalized
  float2* part_ml;         // [parts, Tq, nh]: their (reference, sum of weights)
};

constexpr int kKt = 64;                                  // keys per tile
constexpr int NW = 4;                                    // waves, 32 rows each

template <int D, bool kParts>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2)))
void attn_fwd_kernel(FwdArgs p) {
  constexpr int kQt = 32 * NW;
  constexpr int RB = D * 2;
  constexpr int kTileK = kKt * RB, kTileBytes = 2 * kTileK;
  constexpr int kRows = NW * result_bytes<RB>();
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kTileBytes > kRows ? 2 * kTileBytes : kRows];
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // heads run fastest: workgroups go to the XCDs in turn, so with 8 key heads
  // (or a multiple) an XCD keeps to its own; later tiles of a sequence see
  // more keys and come first
  const int head = blockIdx.x % p.nkv;
  const int index = blockIdx.x / p.nkv, part = kParts ? index % p.parts : 0;
  const SeqTile st = find_rows(p.cu_q, p.cu_k, p.B, p.Tq, p.Tk, p.g.d, kQt,
                               p.n_tiles - 1 - (kParts ? index / p.parts : index));
  if (st.b < 0) return;
  const int k_start = st.start2, n_k = st.n2;
  const int n_rows = st.n, n_q = quot(n_rows, p.g);

  const int r0 = st.tile * kQt + wave * 32;
  const int row = r0 + (lane & 31);                              // within the sequence
  const int rowc = row < n_rows ? row : n_rows - 1;
  const int tok = quot(rowc, p.g), sub = rowc - tok * p.g.d;
  // last visible key of this lane's row, and of the wave's and the tile's
  const int shift = p.causal ? n_k - n_q : n_k;
  auto last_of = [&](int r) {
    return p.causal ? min(quot(min(r, n_rows - 1), p.g) + shift, n_k - 1) : n_k - 1;
  };
  const int last = p.causal ? min(tok + shift, n_k - 1) : n_k - 1;
  const int wave_first = last_of(r0), wave_last = last_of(r0 + 31);
  const int tile_last = last_of(st.tile * kQt + kQt - 1);
  const int n_all = tile_last < 0 ? 0 : tile_last / kKt + 1;     // tiles of keys that some row sees
  const int first_kt = kParts ? static_cast<int>(static_cast<int64_t>(n_all) * part / p.parts) : 0;
  const int n_kt = kParts ? static_cast<int>(static_cast<int64_t>(n_all) * (part + 1) / p.parts) : n_all;

  const uint16_t* kb = p.k + static_cast<int64_t>(k_start) * p.k_ld + head * D;
  const uint16_t* vb = p.v + static_cast<int64_t>(k_start) * p.v_ld + head * D;
  auto load = [&](int kt, uint8_t* buf) {
    const int n = n_k - kt * kKt;
    const int nv = n < kKt ? n : kKt;
    tile_load<RB, kKt, NW>(kb + static_cast<int64_t>(kt) * kKt * p.k_ld, static_cast<uint32_t>(p.k_ld * 2), nv, buf,
                           wave, lane);
    tile_load<RB, kKt, NW>(vb + static_cast<int64_t>(kt) * kKt * p.v_ld, static_cast<uint32_t>(p.v_ld * 2), nv,
                           buf + kTileK, wave, lane);
  };
  if (first_kt < n_kt) load(first_kt, smem);

  bf16x8_t qf[D / 16];
  {
    const uint16_t* q = p.q + (static_cast<int64_t>(st.start) + tok) * p.q_ld + (head * p.g.d + sub) * D + 8 * g;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) qf[s] = *reinterpret_cast<const bf16x8_t*>(q + 16 * s);
  }
  uint32_t k_off[D / 16], v_off[D / 32][2];
#pragma unroll
  for (int s = 0; s < D / 16; ++s) k_off[s] = row_operand_offset<RB>(lane, s);
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) v_off[c][h] = kTileK + col_operand_offset<RB>(lane, c, h);

  f32x16_t o[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) o[c] = f32x16_t{};
  float m = -INFINITY, l = 0.f;
  const float c2 = p.scale * kLog2e;

  // the two buffers' places are constants of the two calls, so that operands'
  // addresses are an offset of the read instruction
  auto tile = [&](int kt, auto half_c) __attribute__((always_inline)) {
    constexpr int kHalf = decltype(half_c)::value;
    wait_vmcnt<0>();
    lds_barrier();
    const uint8_t* buf = smem + kHalf * kTileBytes;
    if (kt + 1 < n_kt) load(kt + 1, smem + (1 - kHalf) * kTileBytes);
    const int t0 = kt * kKt;
    if (t0 > wave_last) return;            // nothing of this tile is visible to the wave
    f32x16_t s[2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        s[b] = mfma(row_operand(buf, k_off[k] + b * 32 * RB), qf[k], k == 0 ? f32x16_t{} : s[b]);
    if (t0 + kKt - 1 > wave_first) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (t0 + 32 * b + 8 * (i >> 2) + 4 * g + (i & 3) > last) s[b][i] = -INFINITY;
    }
    float mx = s[0][0];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][i]);
    mx = fmaxf(mx, other_half(mx));
    const float mn = next_ref(m, mx, c2);
    // a row that has seen no key yet keeps the maximum -inf: its exponents
    // are taken against 0, so every weight is 2^-inf = 0 and not NaN
    const float mc = mn == -INFINITY ? 0.f : mn * c2;
    if (__any(mn > m)) {
      const float a = exp2_hw(fmaf(m, c2, -mc));
      l *= a;
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[c][i] *= a;
      m = mn;
    }
    float sum[4] = {};
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[b][i] = exp2_hw(fmaf(s[b][i], c2, -mc));
        sum[i & 3] += s[b][i];
      }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bf16x8_t pf = pack_operand(s[b], k);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          o[c] = mfma(col_operand(buf, v_off[c][0] + (2 * b + k) * 16 * RB, v_off[c][1] + (2 * b + k) * 16 * RB), pf,
                      o[c]);
      }
  };
  for (int kt = first_kt; kt < n_kt; kt += 2) {
    tile(kt, std::integral_constant<int, 0>{});
    if (kt + 1 < n_kt) tile(kt + 1, std::integral_constant<int, 1>{});
  }
  l += other_half(l);
  if constexpr (kParts) {
    if (row < n_rows) {
      const int64_t at = (static_cast<int64_t>(part) * p.Tq + st.start + tok) * p.nh + head * p.g.d + sub;
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<f32x4_t*>(p.part + at * D + 32 * c + 8 * i + 4 * g) =
              f32x4_t{o[c][4 * i], o[c][4 * i + 1], o[c][4 * i + 2], o[c][4 * i + 3]};
      if (g == 0) p.part_ml[at] = make_float2(m, l);
    }
    return;
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  lds_barrier();                        // everyone is done with the tiles
  uint8_t* rows = smem + wave * result_bytes<RB>();
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint2*>(rows + (lane & 31) * (RB + 16) + (32 * c + 8 * i + 4 * g) * 2) =
          pack4(o[c][4 * i] * inv, o[c][4 * i + 1] * inv, o[c][4 * i + 2] * inv, o[c][4 * i + 3] * inv);
  store_packed<RB>(rows, p.out + static_cast<int64_t>(st.start) * p.out_ld + head * p.g.d * D, p.out_ld, p.g, r0,
                   n_rows, lane);
  if (p.lse && g == 0 && row < n_rows)
    p.lse[(static_cast<int64_t>(st.start) + tok) * p.nh + head * p.g.d + sub] =
        l == 0.f ? -INFINITY : fmaf(m, p.scale, log2_hw(l) * kLn2);
}

// ---- joining the parts of the keys, in order -----------------------------------
// D / 4 lanes a row; only rows that a sequence holds.
template <int D>
__global__ __launch_bounds__(256) void fwd_join_kernel(FwdArgs p) {
  constexpr int kL = D / 4;
  const int lo = clamp_int(p.cu_q[0], 0, p.Tq), hi = clamp_int(p.cu_q[p.B], lo, p.Tq);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / kL) + threadIdx.x / kL;
  const int64_t t = row / p.nh;
  if (t < lo || t >= hi) return;
  const int d = (threadIdx.x & (kL - 1)) * 4;
  const int64_t step = static_cast<int64_t>(p.Tq) * p.nh;
  const float c2 = p.scale * kLog2e;
  float ref = -INFINITY;
  for (int i = 0; i < p.parts; ++i) ref = fmaxf(ref, p.part_ml[row + i * step].x);
  const float rc = ref == -INFINITY ? 0.f : ref * c2;
  f32x4_t x = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
#pragma unroll 8
  for (int i = 0; i < p.parts; ++i) {
    const float2 y = p.part_ml[row + i * step];
    const f32x4_t z = *reinterpret_cast<const f32x4_t*>(p.part + (row + i * step) * D + d);
    const float a = exp2_hw(fmaf(y.x, c2, -rc));
    sum = fmaf(y.y, a, sum);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = fmaf(z[j], a, x[j]);
  }
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  const int h = static_cast<int>(row - t * p.nh);
  *reinterpret_cast<uint2*>(p.out + t * p.out_ld + h * D + d) = pack4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
  if (p.lse && d == 0) p.lse[row] = sum == 0.f ? -INFINITY : fmaf(ref, p.scale, log2_hw(sum) * kLn2);
}

// Parts that the keys are cut into: few rows leave compute units without a
// workgroup, then as many as fill two a unit, of at least 6 tiles in the mean
// (16 tokens x 64 heads over 8000 keys 141 us in one part, 30 in parts of 8
// tiles, 53 in parts of 2: the join walks a row's parts one after another, 12 of
// the 29 us there, 34 of 78 over 30000 keys). The mean over the sequences counts,
// so a long one among short ones gets few parts: 16 tokens over 30000 keys packed
// with 15 prompts of 100 take 540 us.
constexpr int kMaxParts = 64;
int parts_of(int B, int Tq, int Tk, int nh, int nkv) {
  const int64_t wgs = (static_cast<int64_t>(Tq) * (nh / nkv) + 32 * NW - 1) / (32 * NW) * nkv;
  const int64_t tiles = static_cast<int64_t>(Tk) / B / (6 * kKt);
  int64_t n = 2 * kNumCu / (wgs > 0 ? wgs : 1);
  n = n < tiles ? n : tiles;
  return n < 2 ? 1 : (n > kMaxParts ? kMaxParts : static_cast<int>(n));
}
// Rows of the parts' sums: never above either bound, and both grow with Tq, so
// a workspace serves every smaller call.
size_t part_rows(int Tq, int nh) {
  const size_t all = size_t{kMaxParts} * Tq * nh, most = size_t{2} * kNumCu * 32 * NW;
  return all < most ? all : most;
}

template <int D>
void launch_fwd(const FwdArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.n_tiles) * a.nkv * a.parts);
  if (a.parts == 1) {
    hipLaunchKernelGGL((attn_fwd_kernel<D, false>), grid, dim3(64 * NW), 0, stream, a);
    return;
  }
  hipLaunchKernelGGL((attn_fwd_kernel<D, true>), grid, dim3(64 * NW), 0, stream, a);
  constexpr int kPer = 256 / (D / 4);
  const int64_t rows = static_cast<int64_t>(a.Tq) * a.nh;
  hipLaunchKernelGGL(fwd_join_kernel<D>, dim3(static_cast<unsigned>((rows + kPer - 1) / kPer)), dim3(256), 0, stream, a);
}

}  // namespace
}  // namespace gqa
}  // namespace moe

extern "C" size_t moe_gqa_attn_fwd_workspace(int Tq, int n_heads, int head_dim) {
  if (Tq < 0 || Tq > (1 << 27) || n_heads < 1 || n_heads > 1024 || (head_dim != 64 && head_dim != 128)) return 0;
  return moe::gqa::part_rows(Tq, n_heads) * (static_cast<size_t>(head_dim) * 4 + 8);
}

extern "C" int moe_gqa_attn_fwd(const void* q, int64_t q_ld, const void* k, int64_t k_ld, const void* v, int64_t v_ld,
                                int fmt, const int32_t* cu_q, const int32_t* cu_k, int B, int Tq, int Tk, int n_heads,
                                int n_kv_heads, int head_dim, int causal, float scale, void* out, int64_t out_ld,
                                float* lse, void* ws, size_t ws_bytes, hipStream_t stream) {
  using namespace moe;
  using namespace moe::gqa;
  clear_error();
  const char* fn = "moe_gqa_attn_fwd";
  if (const int rc = check_heads(fn, fmt, n_heads, n_kv_heads, head_dim)) return rc;
  if (const int rc = check_sequences(fn, B, Tq, Tk, n_heads, causal, scale)) return rc;
  const int64_t q_row = static_cast<int64_t>(n_heads) * head_dim, k_row = static_cast<int64_t>(n_kv_heads) * head_dim;
  if (const int rc = check_ld(fn, "q_ld", q_ld, q_row)) return rc;
  if (const int rc = check_ld(fn, "k_ld", k_ld, k_row)) return rc;
  if (const int rc = check_ld(fn, "v_ld", v_ld, k_row)) return rc;
  if (const int rc = check_ld(fn, "out_ld", out_ld, q_row)) return rc;
  if (B == 0 || Tq == 0) return MOE_OK;
  MOE_REQUIRE(q && cu_q && cu_k && out && (Tk == 0 || (k && v)), MOE_ERR_INVALID_ARG,
              "moe_gqa_attn_fwd: null pointer");
  MOE_REQUIRE(aligned16(q) && aligned16(k) && aligned16(v) && aligned16(out) && aligned16(ws), MOE_ERR_ALIGNMENT,
              "moe_gqa_attn_fwd: q, k, v, out and ws must be 16-byte aligned");
  const size_t need = moe_gqa_attn_fwd_workspace(Tq, n_heads, head_dim);
  MOE_REQUIRE(ws && ws_bytes >= need, MOE_ERR_WORKSPACE,
              "moe_gqa_attn_fwd: ws smaller than moe_gqa_attn_fwd_workspace(Tq, n_heads, head_dim)");
  FwdArgs a{static_cast<const uint16_t*>(q), q_ld, static_cast<const uint16_t*>(k), k_ld,
            static_cast<const uint16_t*>(v), v_ld, cu_q, cu_k, B, Tq, Tk, n_heads, n_kv_heads, causal,
            make_div(n_heads / n_kv_heads), scale, static_cast<uint16_t*>(out), out_ld, lse, 0, 1, nullptr, nullptr};
  a.n_tiles = Tq * a.g.d / (32 * NW) + (B < Tq ? B : Tq);
  a.parts = parts_of(B, Tq, Tk, n_heads, n_kv_heads);
  a.part = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(a.part + part_rows(Tq, n_heads) * head_dim);
  if (head_dim == 128) launch_fwd<128>(a, stream);
  else launch_fwd<64>(a, stream);
  return check_launch(fn);
}
