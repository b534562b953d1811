// moe_mla_attn_fwd: latent attention over expanded keys and values.
//
// Per head h and packed sequence:
//   s[i, j] = scale * (q[i, h, :128] . k[j, h, :] + q[i, h, 128:] . kr[j, :])
//   out[i, h] = sum_j softmax_j(s[i, :]) v[j, h],  lse[h, i] = log sum_j e^s
// over the keys the mask leaves; a row without keys has out 0 and lse -inf.
//
// One pass over the keys with a running reference and sum (fp32). A wave keeps
// 32 queries as the columns of its accumulators: the scores are computed as
// k q^T, so a query's statistics belong to one lane and its mirror, and the
// weights in the accumulator are the next product's operand without moving.
// The weights are rounded to bf16, as the matrix instruction takes them (rms
// 2^-9.2 of each, and out is rounded to bf16 as well: 2.0e-3 rms against 64
// bits, 1.66e-3 of it the output's own rounding); their sum is taken before
// that rounding.
//
// Bound by the matrix unit and the exponentials in turn: per 64 keys a wave
// has 40 products (1280 cycles) and 1024 elements' softmax (about 900 cycles
// of issue), which two waves a SIMD overlap. Four waves (128 queries) a
// workgroup and two workgroups a CU: keys and values pass LDS in tiles of 64,
// double buffered (80 KB a workgroup), loaded without registers. 3048 queries
// behind 11169 more keys x 128 heads 1835 us on average of 20 calls = 950
// TFLOP/s (1720 for the first to 2190: the clock falls under this load; matrix
// unit 57% busy; an 8192^3 bf16 product reaches 1369); 4096 tokens of three
// prompts, causal, 443 us (375-502) = 665, where the short rows of the mask's
// diagonal tiles and each workgroup's start (queries, first tile) count; 168
// tokens x 16 heads 8.8 us. Measured and slower: eight waves a workgroup (489
// against 440 us), 64 queries a wave at one wave a SIMD (560; 1951 against
// 1800 us: the softmax no longer runs under another wave's products).
#include "mla.h"

#include <cmath>

namespace moe {
namespace mla {
namespace {

constexpr int kKt = 64;                                  // keys per tile
constexpr int kTileKn = kKt * kDn * 2, kTileKr = kKt * kDr * 2, kTileV = kKt * kDv * 2;
constexpr int kTileBytes = kTileKn + kTileKr + kTileV;   // 40 KB

struct FwdArgs {
  const uint16_t* q;
  int64_t q_ld;
  const uint16_t* kv;
  int64_t kv_ld;
  const uint16_t* kr;
  int64_t kr_ld;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, Tq, Tk, nh, causal;
  float scale;
  uint16_t* out;
  int64_t out_ld;
  float* lse;
  int n_tiles;
};

constexpr int NW = 4;                                    // waves, 32 queries each
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2)))
void attn_fwd_kernel(FwdArgs p) {
  constexpr int kQt = 32 * NW;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kTileBytes];
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const int idx = xcd_contiguous(blockIdx.x, gridDim.x);
  const int head = idx / p.n_tiles;
  // later tiles of a sequence see more keys: longest first
  const SeqTile st = find_tile(p.cu_q, p.cu_k, p.B, p.Tq, p.Tk, kQt, p.n_tiles - 1 - idx % p.n_tiles);
  if (st.b < 0) return;
  const int k_start = st.start2, n_k = st.n2;
  const int n_q = st.n;

  const int row = st.tile * kQt + wave * 32 + (lane & 31);       // within the sequence
  const int rowc = row < n_q ? row : n_q - 1;
  // last visible key of this lane's row, and of the whole tile
  const int shift = p.causal ? n_k - n_q : n_k;
  const int last = p.causal ? min(rowc + shift, n_k - 1) : n_k - 1;
  const int wave_first = p.causal ? min(min(st.tile * kQt + wave * 32, n_q - 1) + shift, n_k - 1) : n_k - 1;
  const int tile_last = p.causal ? min(min(st.tile * kQt + kQt, n_q) - 1 + shift, n_k - 1) : n_k - 1;
  const int wave_last = p.causal ? min(min(st.tile * kQt + wave * 32 + 31, n_q - 1) + shift, n_k - 1) : n_k - 1;
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
                            buf + kTileKn, wave, lane);
    tile_load<256, kKt, NW>(b + kDn, ld, nv, buf + kTileKn + kTileKr, wave, lane);
  };
  if (n_kt > 0) load(0, smem);

  bf16x8_t qf[kDq / 16];
  {
    const uint16_t* q = p.q + (static_cast<int64_t>(st.start) + rowc) * p.q_ld + head * kDq + 8 * g;
#pragma unroll
    for (int s = 0; s < kDq / 16; ++s) qf[s] = *reinterpret_cast<const bf16x8_t*>(q + 16 * s);
  }
  uint32_t kn_off[8], kr_off[4], v_off[4][2];
#pragma unroll
  for (int s = 0; s < 8; ++s) kn_off[s] = row_operand_offset<256>(lane, s);
#pragma unroll
  for (int s = 0; s < 4; ++s) kr_off[s] = kTileKn + row_operand_offset<128>(lane, s);
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) v_off[c][h] = kTileKn + kTileKr + col_operand_offset<256>(lane, c, h);

  f32x16_t o[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) o[c] = f32x16_t{};
  float m = -INFINITY, l = 0.f;
  const float c2 = p.scale * kLog2e;

  for (int kt = 0; kt < n_kt; ++kt) {
    wait_vmcnt<0>();
    lds_barrier();
    uint8_t* buf = smem + (kt & 1) * kTileBytes;
    if (kt + 1 < n_kt) load(kt + 1, smem + ((kt + 1) & 1) * kTileBytes);
    const int t0 = kt * kKt;
    if (t0 > wave_last) continue;          // nothing of this tile is visible to the wave
    f32x16_t s[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      s[b] = f32x16_t{};
#pragma unroll
      for (int k = 0; k < 8; ++k) s[b] = mfma(row_operand(buf, kn_off[k] + b * 32 * 256), qf[k], s[b]);
#pragma unroll
      for (int k = 0; k < 4; ++k) s[b] = mfma(row_operand(buf, kr_off[k] + b * 32 * 128), qf[8 + k], s[b]);
    }
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
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[c][i] *= a;
      m = mn;
    }
    float sum = 0.f;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[b][i] = exp2_hw(fmaf(s[b][i], c2, -mc));
        sum += s[b][i];
      }
    l += sum;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bf16x8_t pf = pack_operand(s[b], k);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          o[c] = mfma(col_operand(buf, v_off[c][0] + (2 * b + k) * 16 * 256, v_off[c][1] + (2 * b + k) * 16 * 256),
                      pf, o[c]);
      }
  }
  l += other_half(l);
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  lds_barrier();                        // everyone is done with the tiles
  uint8_t* rows = smem + wave * result_bytes<kDv * 2>();
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint2*>(rows + (lane & 31) * (kDv * 2 + 16) + (32 * c + 8 * i + 4 * g) * 2) =
          pack4(o[c][4 * i] * inv, o[c][4 * i + 1] * inv, o[c][4 * i + 2] * inv, o[c][4 * i + 3] * inv);
  const int64_t tok = static_cast<int64_t>(st.start) + st.tile * kQt + wave * 32;
  store_rows<kDv * 2>(rows, p.out + tok * p.out_ld + head * kDv, p.out_ld * 2, n_q - st.tile * kQt - wave * 32, lane);
  if (p.lse && g == 0 && row < n_q)
    p.lse[(tok + lane) * p.nh + head] = l == 0.f ? -INFINITY : fmaf(m, p.scale, log2_hw(l) * kLn2);
}

}  // namespace
}  // namespace mla
}  // namespace moe

extern "C" int moe_mla_attn_fwd(const void* q, int64_t q_ld, const void* kv, int64_t kv_ld, const void* k_rope,
                                int64_t kr_ld, int fmt, const int32_t* cu_q, const int32_t* cu_k, int B, int Tq,
                                int Tk, int n_heads, int causal, float scale, void* out, int64_t out_ld, float* lse,
                                hipStream_t stream) {
  using namespace moe;
  using namespace moe::mla;
  clear_error();
  if (const int rc = check_expanded("moe_mla_attn_fwd", fmt, B, Tq, Tk, n_heads, causal, scale, q_ld, kv_ld, kr_ld,
                                    out_ld))
    return rc;
  if (B == 0 || Tq == 0) return MOE_OK;
  MOE_REQUIRE(q && cu_q && cu_k && out && (Tk == 0 || (kv && k_rope)), MOE_ERR_INVALID_ARG,
              "moe_mla_attn_fwd: null pointer");
  MOE_REQUIRE(aligned16(q) && aligned16(kv) && aligned16(k_rope) && aligned16(out), MOE_ERR_ALIGNMENT,
              "moe_mla_attn_fwd: q, kv, k_rope and out must be 16-byte aligned");
  FwdArgs a{static_cast<const uint16_t*>(q), q_ld, static_cast<const uint16_t*>(kv), kv_ld,
            static_cast<const uint16_t*>(k_rope), kr_ld, cu_q, cu_k, B, Tq, Tk, n_heads, causal, scale,
            static_cast<uint16_t*>(out), out_ld, lse, 0};
  a.n_tiles = seq_tiles_bound(B, Tq, 32 * NW);
  hipLaunchKernelGGL(attn_fwd_kernel, dim3(static_cast<unsigned>(a.n_tiles) * n_heads), dim3(64 * NW), 0, stream, a);
  return check_launch("moe_mla_attn_fwd");
}
