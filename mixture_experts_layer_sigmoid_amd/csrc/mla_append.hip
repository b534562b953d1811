// moe_mla_append: new tokens into the latent cache.
//
// Per token t with slot s = slots[t] and angles a_i = angle(positions[t], i):
//   cache[s, :512] = c / sqrt(mean(c^2) + eps) * w,   c = kv_a[t, :512]
//   cache[s, 512:] = rotary(kv_a[t, 512:576])
//   q_out[t, h]    = (q[t, h, :128] | rotary(q[t, h, 128:192]))
// rotary turns the pair (x, y) into (x cos a_i - y sin a_i, x sin a_i +
// y cos a_i); pair i is (2 i, 2 i + 1) or (i, i + 32). All arithmetic in
// fp32, one rounding to bf16 at the store.
// One workgroup a token, so that a token's latent, its angles and its heads
// need no index arithmetic and the first wave's sum of squares stays in
// registers; 16-byte accesses. Bound by memory: 8192 tokens x 128 heads 160 us
// = 5.16 TB/s (a plain copy of 1 GiB: 4.87 TB/s). 64 tokens x 16 heads: 3.8 us,
// bound by two dependent trips to memory and the launch (1 MB).
#include "mla.h"

#include <cmath>

namespace moe {
namespace mla {
namespace {

struct AppendArgs {
  const uint16_t* kv_a;
  int64_t kv_ld;
  const uint16_t* w;
  float eps;
  const float* cos;
  const float* sin;
  int max_pos;
  const int32_t* pos;
  int interleaved;
  const int64_t* slots;
  int64_t n_slots;
  uint16_t* cache;
  const uint16_t* q;
  int64_t q_ld;
  uint16_t* q_out;
  int64_t qo_ld;
  int T, nh;
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

// Pairs 8 j .. 8 j + 7 (j < 4) of 64 rotary values: the two 16-byte pieces
// that hold them are 2 j, 2 j + 1 (interleaved) or j, j + 4 (halves).
__device__ __forceinline__ void rotate16(const uint16_t* src, uint16_t* dst, int j, bool interleaved,
                                         const float* cs, const float* sn) {
  const int a = interleaved ? 2 * j : j, b = interleaved ? 2 * j + 1 : j + 4;
  float x[16], c[8], s[8], y[16];
  unpack8(*reinterpret_cast<const u32x4_t*>(src + 8 * a), x);
  unpack8(*reinterpret_cast<const u32x4_t*>(src + 8 * b), x + 8);
  load8_f32(cs + 8 * j, c);
  load8_f32(sn + 8 * j, s);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[2 * i] = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
      y[2 * i + 1] = x[2 * i] * s[i] + x[2 * i + 1] * c[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = x[i] * c[i] - x[8 + i] * s[i];
      y[8 + i] = x[i] * s[i] + x[8 + i] * c[i];
    }
  }
  *reinterpret_cast<u32x4_t*>(dst + 8 * a) = pack8(y);
  *reinterpret_cast<u32x4_t*>(dst + 8 * b) = pack8(y + 8);
}

__global__ __launch_bounds__(256) void append_kernel(AppendArgs p) {
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int pos = clamp_int(p.pos ? p.pos[t] : 0, 0, p.max_pos - 1);
  const float* cs = p.cos + static_cast<int64_t>(pos) * 32;
  const float* sn = p.sin + static_cast<int64_t>(pos) * 32;
  if (wave == 0) {
    const int64_t slot = p.slots[t];
    const uint16_t* src = p.kv_a + static_cast<int64_t>(t) * p.kv_ld;
    float v[8], w[8];
    unpack8(*reinterpret_cast<const u32x4_t*>(src + 8 * lane), v);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
    if (slot >= 0 && slot < p.n_slots) {
      uint16_t* dst = p.cache + slot * kDc;
      if (p.w) {
        unpack8(*reinterpret_cast<const u32x4_t*>(p.w + 8 * lane), w);
        const float r = 1.f / sqrtf(s / kR + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[i];
      }
      *reinterpret_cast<u32x4_t*>(dst + 8 * lane) = pack8(v);
      if (p.cos) {
        if (lane < 4) rotate16(src + kR, dst + kR, lane, p.interleaved, cs, sn);
      } else if (lane < 8) {
        *reinterpret_cast<u32x4_t*>(dst + kR + 8 * lane) = *reinterpret_cast<const u32x4_t*>(src + kR + 8 * lane);
      }
    }
  }
  if (!p.q) return;
  const uint16_t* q = p.q + static_cast<int64_t>(t) * p.q_ld;
  uint16_t* qo = p.q_out + static_cast<int64_t>(t) * p.qo_ld;
  const int tid = static_cast<int>(threadIdx.x);
  if (p.cos)
    for (int i = tid; i < p.nh * 4; i += 256)
      rotate16(q + (i >> 2) * kDq + kDn, qo + (i >> 2) * kDq + kDn, i & 3, p.interleaved, cs, sn);
  if (q != qo) {
    const int per = p.cos ? 16 : 24;
    for (int i = tid; i < p.nh * per; i += 256) {
      const int o = (i / per) * kDq + (i % per) * 8;
      *reinterpret_cast<u32x4_t*>(qo + o) = *reinterpret_cast<const u32x4_t*>(q + o);
    }
  }
}

}  // namespace
}  // namespace mla
}  // namespace moe

extern "C" int moe_mla_append(const void* kv_a, int64_t kv_ld, int fmt, const void* norm_w, float eps,
                              const float* cos, const float* sin, int max_pos, const int32_t* positions,
                              int interleaved, const int64_t* slots, void* cache, int64_t n_slots, const void* q,
                              int64_t q_ld, void* q_out, int64_t qo_ld, int T, int n_heads, hipStream_t stream) {
  using namespace moe;
  using namespace moe::mla;
  clear_error();
  MOE_REQUIRE(T >= 0 && T <= (1 << 23) && n_slots >= 0, MOE_ERR_INVALID_ARG,
              "moe_mla_append: need 0 <= T <= 2^23 and n_slots >= 0");
  MOE_REQUIRE(fmt == MOE_BF16, MOE_ERR_UNSUPPORTED, "moe_mla_append: fmt must be MOE_BF16");
  MOE_REQUIRE(kv_ld >= kDc && kv_ld <= kMaxLd && kv_ld % 8 == 0, MOE_ERR_INVALID_ARG,
              "moe_mla_append: kv_ld must be a multiple of 8 in [576, 2^23]");
  MOE_REQUIRE(!norm_w || (eps >= 0.f && eps <= 1.f), MOE_ERR_INVALID_ARG, "moe_mla_append: eps must be in [0, 1]");
  MOE_REQUIRE((cos != nullptr) == (sin != nullptr) && (!cos || (positions && max_pos >= 1)), MOE_ERR_INVALID_ARG,
              "moe_mla_append: cos and sin come together, with positions and max_pos >= 1");
  MOE_REQUIRE(interleaved == 0 || interleaved == 1, MOE_ERR_INVALID_ARG,
              "moe_mla_append: interleaved must be 0 or 1");
  MOE_REQUIRE((q != nullptr) == (q_out != nullptr), MOE_ERR_INVALID_ARG,
              "moe_mla_append: q and q_out come together");
  if (q) {
    const int64_t row = static_cast<int64_t>(n_heads) * kDq;
    MOE_REQUIRE(n_heads >= 1 && n_heads <= 1024 && q_ld >= row && qo_ld >= row && q_ld <= kMaxLd && qo_ld <= kMaxLd &&
                    q_ld % 8 == 0 && qo_ld % 8 == 0,
                MOE_ERR_INVALID_ARG,
                "moe_mla_append: n_heads must be in [1, 1024], q strides multiples of 8 that hold n_heads * 192");
    MOE_REQUIRE(q != q_out || q_ld == qo_ld, MOE_ERR_INVALID_ARG,
                "moe_mla_append: in place, q_ld and qo_ld must be equal");
  }
  if (T == 0) return MOE_OK;
  MOE_REQUIRE(kv_a && slots && (cache || n_slots == 0), MOE_ERR_INVALID_ARG, "moe_mla_append: null pointer");
  MOE_REQUIRE(aligned16(kv_a) && aligned16(norm_w) && aligned16(cos) && aligned16(sin) && aligned16(cache) &&
                  aligned16(q) && aligned16(q_out),
              MOE_ERR_ALIGNMENT, "moe_mla_append: tensors must be 16-byte aligned");
  AppendArgs a{static_cast<const uint16_t*>(kv_a), kv_ld, static_cast<const uint16_t*>(norm_w), eps, cos, sin,
               cos ? max_pos : 1, cos ? positions : nullptr, interleaved, slots, n_slots,
               static_cast<uint16_t*>(cache), static_cast<const uint16_t*>(q), q_ld, static_cast<uint16_t*>(q_out),
               qo_ld, T, n_heads};
  hipLaunchKernelGGL(append_kernel, dim3(T), dim3(256), 0, stream, a);
  return check_launch("moe_mla_append");
}
