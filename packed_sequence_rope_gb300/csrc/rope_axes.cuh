// Rotation by positions with several axes, shared by aa_rope_axes_apply and
// the paged cache's append.
//
// Pair p of a row turns by pos[axis(p)][t] * theta_p (Eq. 6 of "When Precision
// Meets Position", architecture page, §3.4 "Rotary Positional Embedding
// (RoPE)", with one position per axis). The angle is taken in turns:
// theta_p / (2 pi) modulo 1 is kept as a 64-bit fraction, so its product with an
// integer position, modulo 2^64, is the angle modulo one turn without any
// rounding that grows with the position (fp32 products lose 0.008 rad at
// 1.3e5). The top 32 bits then go through sincospif.
#pragma once

#include "kcommon.cuh"

namespace aa {

// What a kernel needs of an aa_rope_axes (passed by value).
struct AxesTable {
  uint64_t turn[64];
  uint8_t axis[64];
};

inline AxesTable axes_table(const aa_rope_axes* r) {
  AxesTable t{};
  for (int p = 0; p < r->head_dim / 2; ++p) {
    t.turn[p] = r->turn[p];
    t.axis[p] = (uint8_t)r->axis_of_pair[p];
  }
  return t;
}

constexpr int32_t kAxesReady = 0x41786573;  // set by aa_rope_axes_init
inline bool axes_valid(const aa_rope_axes* r) { return r && r->ready == kAxesReady; }

__device__ __forceinline__ float2 axes_cs(const AxesTable& tab, const int32_t* __restrict__ pos, int64_t T, int64_t t,
                                          int p) {
  const int64_t at = __ldg(pos + tab.axis[p] * T + t);
  const uint64_t turns = (uint64_t)at * tab.turn[p];
  const int32_t half_turns = (int32_t)(uint32_t)((turns + (1ull << 31)) >> 32);  // angle / pi * 2^31
  float c, s;
  sincospif((float)half_turns * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

// Eight pairs of one row in registers: elements [16 i, 16 i + 16) for adjacent
// pairs (L = 0), [8 i, 8 i + 8) and HD / 2 further for split halves (L = 1).
template <int HD, int L>
struct Pairs8 {
  uint4 a, b;
  static __device__ __forceinline__ int off_a(int i) { return L == 0 ? 16 * i : 8 * i; }
  static __device__ __forceinline__ int off_b(int i) { return L == 0 ? 16 * i + 8 : HD / 2 + 8 * i; }
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int i) {
    a = *reinterpret_cast<const uint4*>(row + off_a(i));
    b = *reinterpret_cast<const uint4*>(row + off_b(i));
  }
  __device__ __forceinline__ void store(__nv_bfloat16* row, int i) const {
    *reinterpret_cast<uint4*>(row + off_a(i)) = a;
    *reinterpret_cast<uint4*>(row + off_b(i)) = b;
  }
  __device__ __forceinline__ void turn(const float2* cs) {
    uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if constexpr (L == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float2 v = ptx::unpack_bf16x2(u[e]);
        rope_pair(v.x, v.y, cs[e].x, cs[e].y);
        u[e] = ptx::pack_bf16x2(v.x, v.y);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 x = ptx::unpack_bf16x2(u[e]), y = ptx::unpack_bf16x2(u[4 + e]);
        rope_pair(x.x, y.x, cs[2 * e].x, cs[2 * e].y);
        rope_pair(x.y, y.y, cs[2 * e + 1].x, cs[2 * e + 1].y);
        u[e] = ptx::pack_bf16x2(x.x, x.y);
        u[4 + e] = ptx::pack_bf16x2(y.x, y.y);
      }
    }
    a = make_uint4(u[0], u[1], u[2], u[3]);
    b = make_uint4(u[4], u[5], u[6], u[7]);
  }
};

}  // namespace aa
