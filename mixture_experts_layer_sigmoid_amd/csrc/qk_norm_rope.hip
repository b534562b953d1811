// moe_qk_norm_rope and its backward: RMS norm of every head's query and key
// and the rotation of their first values by position, in one pass.
//
// Per token t and head, x of D values, w the weight of queries or keys:
//   r = 1 / sqrt(mean(x^2) + eps),  u = x r w,  y = R_t u
// R_t turns pair i < rotary / 2 of u by the angle of row positions[t]; pair i is
// (2 i, 2 i + 1) or (i, i + rotary / 2), values from `rotary` on stay. With g =
// R_t^T dy (the same turn backwards) and xh = x r:
//   dw = sum over tokens and heads of g xh,   dx = r (g w - xh mean(g w xh))
// All arithmetic in fp32, one rounding to bf16 at the store; dw stays fp32.
//
// D / 16 lanes take a head, 16 values each: the two 8-value pieces that hold 8
// pairs, so a rotation needs no exchange. A wave's groups of lanes walk the
// heads of one token, whose angles stay in registers.
//
// Memory bounds both: 8192 tokens x (64 + 8) heads of 128 take 61 to 65 us forward
// for 302 MB (4.6 to 4.9 TB/s) and 106 to 110 + 4.8 us backward for 453 MB (4.1 to
// 4.3 TB/s; the weights' gradients are summed in registers over a workgroup's
// tokens and in a second launch over the workgroups, so they repeat bit for bit).
#include "gqa.h"

#include <cmath>

namespace moe {
namespace gqa {
namespace {

struct NormArgs {
  const uint16_t* q;
  int64_t q_ld;
  const uint16_t* k;
  int64_t k_ld;
  const uint16_t* w_q;
  const uint16_t* w_k;
  float eps;
  const float* cos;
  const float* sin;
  int max_pos;
  const int32_t* pos;
  int rotary, interleaved;
  int T, nh, nkv;
  int wpt;                  // waves a token (forward)
  uint16_t* q_out;          // forward: results; backward: dq, dk
  int64_t qo_ld;
  uint16_t* k_out;
  int64_t ko_ld;
  const uint16_t* dq_out;   // backward: gradients of the results
  int64_t dqo_ld;
  const uint16_t* dk_out;
  int64_t dko_ld;
  float* dw_q;
  float* dw_k;
  float* part;              // [workgroups, 2, D]
  int n_parts;
};

__device__ __forceinline__ void unpack8(u32x4_t r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r[i] << 16);
    v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ u32x4_t pack8(const float* v) {
  const uint2 a = pack4(v[0], v[1], v[2], v[3]), b = pack4(v[4], v[5], v[6], v[7]);
  return u32x4_t{a.x, a.y, b.x, b.y};
}

// What a lane keeps for one token: its two pieces' places in a head, and the
// 8 angles of their pairs where they are rotated.
// IL: pairs are neighbours. (One kernel for both orders would keep both
// results of every rotation: 173 registers a lane of the backward.)
template <int D, bool IL>
struct Lane {
  int a, b;                 // first values of the two pieces
  bool turn;
  float c[8], s[8];
  __device__ __forceinline__ Lane(const NormArgs& p, int lane) {
    const int j = lane & (D / 16 - 1);
    turn = j < p.rotary / 16;
    a = turn && !IL ? 8 * j : 16 * j;
    b = turn && !IL ? 8 * j + p.rotary / 2 : 16 * j + 8;
  }
  __device__ __forceinline__ void angles(const NormArgs& p, int t, int lane) {
    if (!turn) return;
    const int64_t row = static_cast<int64_t>(clamp_int(p.pos[t], 0, p.max_pos - 1)) * (p.rotary / 2) +
                        8 * (lane & (D / 16 - 1));
    load8_f32(p.cos + row, c);
    load8_f32(p.sin + row, s);
  }
  __device__ __forceinline__ void load(const uint16_t* x, float* v) const {
    unpack8(*reinterpret_cast<const u32x4_t*>(x + a), v);
    unpack8(*reinterpret_cast<const u32x4_t*>(x + b), v + 8);
  }
  __device__ __forceinline__ void store(uint16_t* x, const float* v) const {
    *reinterpret_cast<u32x4_t*>(x + a) = pack8(v);
    *reinterpret_cast<u32x4_t*>(x + b) = pack8(v + 8);
  }
  // pairs turned by their angles, forwards (sign 1) or back (-1)
  __device__ __forceinline__ void rotate(float* v, float sign) const {
    if (!turn) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      constexpr int kStep = IL ? 2 : 1, kMate = IL ? 1 : 8;
      const float x = v[kStep * i], y = v[kStep * i + kMate], sn = sign * s[i];
      v[kStep * i] = x * c[i] - y * sn;
      v[kStep * i + kMate] = x * sn + y * c[i];
    }
  }
};

// sum over the lanes of a head
template <int D>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = D / 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

template <int D>
__device__ __forceinline__ float inv_rms(const float* x, float eps) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s = fmaf(x[i], x[i], s);
  return 1.f / sqrtf(head_sum<D>(s) / D + eps);
}

template <int D, bool IL>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormArgs p) {
  constexpr int kHeads = 64 / (D / 16);                // heads a wave takes at once
  const int lane = threadIdx.x & 63;
  const int wave = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int t = wave / p.wpt;
  if (t >= p.T) return;
  Lane<D, IL> ln(p, lane);
  ln.angles(p, t, lane);
  const int first = (wave - t * p.wpt) * kHeads + lane / (D / 16), step = p.wpt * kHeads;
  auto side = [&](const uint16_t* x, int64_t ld, const uint16_t* w, uint16_t* out, int64_t out_ld, int n, int from) {
    float wv[16];
    if (w) ln.load(w, wv);
    x += t * ld;
    out += t * out_ld;
    for (int h = from; h < n; h += step) {
      float v[16];
      ln.load(x + h * D, v);
      if (w) {
        const float r = inv_rms<D>(v, p.eps);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = v[i] * r * wv[i];
      }
      ln.rotate(v, 1.f);
      ln.store(out + h * D, v);
    }
  };
  side(p.q, p.q_ld, p.w_q, p.q_out, p.qo_ld, p.nh, first);
  // key heads follow the query heads in the same round of the waves
  side(p.k, p.k_ld, p.w_k, p.k_out, p.ko_ld, p.nkv, (first - p.nh % step + step) % step);
}

// ---- backward --------------------------------------------------------------------
// Workgroups take tokens in turn, the queries' heads first and then the keys',
// and add their share of dw up in registers; part holds one row a workgroup,
// which a second launch adds in order.
constexpr int kBwdGroups = 512, kBwdWaves = 8;

template <int D, bool IL>
__global__ __launch_bounds__(64 * kBwdWaves) void norm_rope_bwd_kernel(NormArgs p) {
  constexpr int kL = D / 16, kHeads = 64 / kL;
  __shared__ float red[kBwdWaves][2][D];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Lane<D, IL> ln(p, lane);
  auto side = [&](int which, const uint16_t* x0, int64_t ld, const uint16_t* w, const uint16_t* dy0, int64_t dy_ld,
                  uint16_t* dx0, int64_t dx_ld, int n) {
    float wv[16], dw[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[i] = 0.f;
    if (w) ln.load(w, wv);
    for (int t = blockIdx.x * kBwdWaves + wave; t < p.T; t += gridDim.x * kBwdWaves) {
      ln.angles(p, t, lane);
      const uint16_t* x = x0 + t * ld;
      const uint16_t* dy = dy0 + t * dy_ld;
      uint16_t* dx = dx0 + t * dx_ld;
      for (int h = lane / kL; h < n; h += kHeads) {
        float g[16];
        ln.load(dy + h * D, g);
        if (w) {
          float v[16];
          ln.load(x + h * D, v);
          const float r = inv_rms<D>(v, p.eps);
          ln.rotate(g, -1.f);
          float dot = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] *= r;
            dw[i] = fmaf(g[i], v[i], dw[i]);
            g[i] *= wv[i];
            dot = fmaf(g[i], v[i], dot);
          }
          dot = head_sum<D>(dot) / D;
#pragma unroll
          for (int i = 0; i < 16; ++i) g[i] = r * (g[i] - v[i] * dot);
        } else {
          ln.rotate(g, -1.f);
        }
        ln.store(dx + h * D, g);
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
      for (int o = kL; o < 64; o <<= 1) dw[i] += __shfl_xor(dw[i], o, 64);
      if (lane < kL) red[wave][which][i < 8 ? ln.a + i : ln.b + i - 8] = dw[i];
    }
  };
  side(0, p.q, p.q_ld, p.w_q, p.dq_out, p.dqo_ld, p.q_out, p.qo_ld, p.nh);
  side(1, p.k, p.k_ld, p.w_k, p.dk_out, p.dko_ld, p.k_out, p.ko_ld, p.nkv);
  if (!p.w_q && !p.w_k) return;
  __syncthreads();
  if (threadIdx.x < 2 * D) {
    const float* r = &red[0][0][0] + threadIdx.x;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kBwdWaves; ++i) s += r[i * 2 * D];
    p.part[static_cast<int64_t>(blockIdx.x) * 2 * D + threadIdx.x] = s;
  }
}

// 16 columns a workgroup, 64 rows of part at a time
template <int D>
__global__ __launch_bounds__(1024) void norm_rope_dw_kernel(NormArgs p) {
  __shared__ float red[64][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + c;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kBwdGroups / 64; ++i) {
    const int row = r + 64 * i;
    s += row < p.n_parts ? p.part[static_cast<int64_t>(row) * 2 * D + col] : 0.f;
  }
  red[r][c] = s;
  __syncthreads();
  if (r == 0) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 64; ++i) s += red[i][c];
    float* out = col < D ? (p.w_q ? p.dw_q + col : nullptr) : (p.w_k ? p.dw_k + col - D : nullptr);
    if (out) *out = s;
  }
}

int check_norm(const std::string& fn, int fmt, const void* w_q, const void* w_k, float eps, const float* cos,
               const float* sin, int max_pos, const int32_t* positions, int rotary, int interleaved, int T, int nh,
               int nkv, int D) {
  MOE_REQUIRE(T >= 0 && T <= (1 << 23), MOE_ERR_INVALID_ARG, fn + ": T must be in [0, 2^23]");
  MOE_REQUIRE(nh >= 1 && nh <= 1024 && nkv >= 1 && nkv <= 1024, MOE_ERR_INVALID_ARG,
              fn + ": n_heads and n_kv_heads must be in [1, 1024]");
  MOE_REQUIRE(fmt == MOE_BF16, MOE_ERR_UNSUPPORTED, fn + ": fmt must be MOE_BF16");
  MOE_REQUIRE(D == 64 || D == 128, MOE_ERR_UNSUPPORTED, fn + ": head_dim must be 64 or 128");
  MOE_REQUIRE((!w_q && !w_k) || (eps >= 0.f && eps <= 1.f), MOE_ERR_INVALID_ARG, fn + ": eps must be in [0, 1]");
  MOE_REQUIRE((cos != nullptr) == (sin != nullptr) && (!cos || (max_pos >= 1 && (T == 0 || positions))),
              MOE_ERR_INVALID_ARG, fn + ": cos and sin come together, with positions and max_pos >= 1");
  MOE_REQUIRE(!cos || (rotary >= 16 && rotary <= D && rotary % 16 == 0), MOE_ERR_INVALID_ARG,
              fn + ": rotary must be a multiple of 16 in [16, head_dim]");
  MOE_REQUIRE(interleaved == 0 || interleaved == 1, MOE_ERR_INVALID_ARG, fn + ": interleaved must be 0 or 1");
  MOE_REQUIRE(aligned16(w_q) && aligned16(w_k) && aligned16(cos) && aligned16(sin), MOE_ERR_ALIGNMENT,
              fn + ": weights, cos and sin must be 16-byte aligned");
  return MOE_OK;
}

}  // namespace
}  // namespace gqa
}  // namespace moe

extern "C" int moe_qk_norm_rope(const void* q, int64_t q_ld, const void* k, int64_t k_ld, int fmt, const void* w_q,
                                const void* w_k, float eps, const float* cos, const float* sin, int max_pos,
                                const int32_t* positions, int rotary, int interleaved, int T, int n_heads,
                                int n_kv_heads, int head_dim, void* q_out, int64_t qo_ld, void* k_out, int64_t ko_ld,
                                hipStream_t stream) {
  using namespace moe;
  using namespace moe::gqa;
  clear_error();
  const char* fn = "moe_qk_norm_rope";
  if (const int rc = check_norm(fn, fmt, w_q, w_k, eps, cos, sin, max_pos, positions, rotary, interleaved, T, n_heads,
                                n_kv_heads, head_dim))
    return rc;
  const int64_t q_row = static_cast<int64_t>(n_heads) * head_dim, k_row = static_cast<int64_t>(n_kv_heads) * head_dim;
  if (const int rc = check_ld(fn, "q_ld", q_ld, q_row)) return rc;
  if (const int rc = check_ld(fn, "k_ld", k_ld, k_row)) return rc;
  if (const int rc = check_ld(fn, "qo_ld", qo_ld, q_row)) return rc;
  if (const int rc = check_ld(fn, "ko_ld", ko_ld, k_row)) return rc;
  MOE_REQUIRE((q != q_out || q_ld == qo_ld) && (k != k_out || k_ld == ko_ld), MOE_ERR_INVALID_ARG,
              "moe_qk_norm_rope: in place, both row strides must be equal");
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(q && k && q_out && k_out, MOE_ERR_INVALID_ARG, "moe_qk_norm_rope: null pointer");
  MOE_REQUIRE(aligned16(q) && aligned16(k) && aligned16(q_out) && aligned16(k_out), MOE_ERR_ALIGNMENT,
              "moe_qk_norm_rope: tensors must be 16-byte aligned");
  NormArgs a{};
  a.q = static_cast<const uint16_t*>(q), a.q_ld = q_ld, a.k = static_cast<const uint16_t*>(k), a.k_ld = k_ld;
  a.w_q = static_cast<const uint16_t*>(w_q), a.w_k = static_cast<const uint16_t*>(w_k), a.eps = eps;
  a.cos = cos, a.sin = sin, a.max_pos = max_pos, a.pos = positions;
  a.rotary = cos ? rotary : 0, a.interleaved = interleaved, a.T = T, a.nh = n_heads, a.nkv = n_kv_heads;
  a.q_out = static_cast<uint16_t*>(q_out), a.qo_ld = qo_ld, a.k_out = static_cast<uint16_t*>(k_out), a.ko_ld = ko_ld;
  // few tokens: more waves a token, as far as they have heads
  const int rounds = (n_heads + n_kv_heads + 1024 / head_dim - 1) / (1024 / head_dim);
  a.wpt = 1;
  while (a.wpt < rounds && static_cast<int64_t>(T) * a.wpt < 8 * kNumCu) a.wpt *= 2;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(T) * a.wpt + 3) / 4));
  const auto kernel = head_dim == 128 ? (interleaved ? norm_rope_kernel<128, true> : norm_rope_kernel<128, false>)
                                      : (interleaved ? norm_rope_kernel<64, true> : norm_rope_kernel<64, false>);
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a);
  return check_launch(fn);
}

extern "C" size_t moe_qk_norm_rope_bwd_workspace(int head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return static_cast<size_t>(moe::gqa::kBwdGroups) * 2 * head_dim * 4;
}

extern "C" int moe_qk_norm_rope_bwd(const void* dq_out, int64_t dqo_ld, const void* dk_out, int64_t dko_ld,
                                    const void* q, int64_t q_ld, const void* k, int64_t k_ld, int fmt, const void* w_q,
                                    const void* w_k, float eps, const float* cos, const float* sin, int max_pos,
                                    const int32_t* positions, int rotary, int interleaved, int T, int n_heads,
                                    int n_kv_heads, int head_dim, void* dq, int64_t dq_ld, void* dk, int64_t dk_ld,
                                    float* dw_q, float* dw_k, void* ws, size_t ws_bytes, hipStream_t stream) {
  using namespace moe;
  using namespace moe::gqa;
  clear_error();
  const char* fn = "moe_qk_norm_rope_bwd";
  if (const int rc = check_norm(fn, fmt, w_q, w_k, eps, cos, sin, max_pos, positions, rotary, interleaved, T, n_heads,
                                n_kv_heads, head_dim))
    return rc;
  const int64_t q_row = static_cast<int64_t>(n_heads) * head_dim, k_row = static_cast<int64_t>(n_kv_heads) * head_dim;
  const struct { const char* name; int64_t ld, row; } lds[] = {{"dqo_ld", dqo_ld, q_row}, {"dko_ld", dko_ld, k_row},
                                                               {"q_ld", q_ld, q_row},     {"k_ld", k_ld, k_row},
                                                               {"dq_ld", dq_ld, q_row},   {"dk_ld", dk_ld, k_row}};
  for (const auto& x : lds)
    if (const int rc = check_ld(fn, x.name, x.ld, x.row)) return rc;
  MOE_REQUIRE((!w_q || dw_q) && (!w_k || dw_k), MOE_ERR_INVALID_ARG,
              "moe_qk_norm_rope_bwd: a weight's gradient has no place");
  MOE_REQUIRE(T == 0 || (dq_out && dk_out && dq && dk && (!w_q || q) && (!w_k || k)), MOE_ERR_INVALID_ARG,
              "moe_qk_norm_rope_bwd: null pointer");
  MOE_REQUIRE(aligned16(dq_out) && aligned16(dk_out) && aligned16(q) && aligned16(k) && aligned16(dq) &&
                  aligned16(dk) && aligned16(dw_q) && aligned16(dw_k) && aligned16(ws),
              MOE_ERR_ALIGNMENT, "moe_qk_norm_rope_bwd: tensors and ws must be 16-byte aligned");
  const bool norm = w_q || w_k;
  MOE_REQUIRE(!norm || (ws && ws_bytes >= moe_qk_norm_rope_bwd_workspace(head_dim)), MOE_ERR_WORKSPACE,
              "moe_qk_norm_rope_bwd: ws smaller than moe_qk_norm_rope_bwd_workspace(head_dim)");
  if (T == 0 && !norm) return MOE_OK;
  NormArgs a{};
  a.q = static_cast<const uint16_t*>(q), a.q_ld = q_ld, a.k = static_cast<const uint16_t*>(k), a.k_ld = k_ld;
  a.w_q = static_cast<const uint16_t*>(w_q), a.w_k = static_cast<const uint16_t*>(w_k), a.eps = eps;
  a.cos = cos, a.sin = sin, a.max_pos = max_pos, a.pos = positions;
  a.rotary = cos ? rotary : 0, a.interleaved = interleaved, a.T = T, a.nh = n_heads, a.nkv = n_kv_heads;
  a.q_out = static_cast<uint16_t*>(dq), a.qo_ld = dq_ld, a.k_out = static_cast<uint16_t*>(dk), a.ko_ld = dk_ld;
  a.dq_out = static_cast<const uint16_t*>(dq_out), a.dqo_ld = dqo_ld;
  a.dk_out = static_cast<const uint16_t*>(dk_out), a.dko_ld = dko_ld;
  a.dw_q = dw_q, a.dw_k = dw_k, a.part = static_cast<float*>(ws);
  const int groups = (T + kBwdWaves - 1) / kBwdWaves;
  a.n_parts = groups < kBwdGroups ? groups : kBwdGroups;
  if (T > 0) {
    const auto kernel = head_dim == 128
                            ? (interleaved ? norm_rope_bwd_kernel<128, true> : norm_rope_bwd_kernel<128, false>)
                            : (interleaved ? norm_rope_bwd_kernel<64, true> : norm_rope_bwd_kernel<64, false>);
    hipLaunchKernelGGL(kernel, dim3(a.n_parts), dim3(64 * kBwdWaves), 0, stream, a);
  }
  if (norm) {
    if (head_dim == 128) hipLaunchKernelGGL(norm_rope_dw_kernel<128>, dim3(16), dim3(1024), 0, stream, a);
    else hipLaunchKernelGGL(norm_rope_dw_kernel<64>, dim3(8), dim3(1024), 0, stream, a);
  }
  return check_launch(fn);
}
