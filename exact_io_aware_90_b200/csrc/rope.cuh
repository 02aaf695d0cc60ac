// rope.cuh — the row arithmetic shared by the kernels that norm and rotate queries and keys: one row is
// the d features of one (token, head).
//
//   norm      n_f = x_f · r · w_f,  r = 1/√(mean_f x_f² + eps)              (optional)
//   rotation  (a, b) → (a·cos − b·sin, b·cos + a·sin) for each of the rot/2 pairs, cos and sin from the
//             caller's table at the token's position; features from rot on pass unrotated
//
// d/16 lanes work on a row.  Lane l holds two 8-feature chunks (16-byte loads) whose pairs it owns
// whole, so the rotation needs no exchange between lanes: with split halves (pairs (i, i + rot/2)) the
// chunks start at 8l and rot/2 + 8l, with neighbouring pairs (2i, 2i + 1) at 16l and 16l + 8.  Either
// way the lane's eight pairs are frequencies 8l .. 8l + 7, and the lanes from rot/16 on hold 16
// unrotated features each.
#pragma once

#include "fa_paged_internal.h"
#include "sm100.cuh"

namespace fa {

struct RopeLane {
  int c0, c1;  // first feature of the two chunks
  int f0;      // first of the eight frequencies
  bool rot;
};

template <bool INTER>
__device__ __forceinline__ RopeLane rope_lane(int l, int rot_dim) {
  RopeLane r;
  r.rot = 16 * l < rot_dim;
  r.f0 = 8 * l;
  if (INTER || !r.rot) {
    r.c0 = 16 * l;
    r.c1 = 16 * l + 8;
  } else {
    r.c0 = 8 * l;
    r.c1 = rot_dim / 2 + 8 * l;
  }
  return r;
}

// The positions that this lane's eight frequencies of token t go by, four by four: frequency i goes by the axis whose
// section holds i (sections are multiples of 4).  pos0 stands for positions == nullptr.
__device__ __forceinline__ int2 rope_positions(const RopeArgs& ra, int t, int T, int pos0, const RopeLane& rl) {
  if (ra.positions == nullptr) return make_int2(pos0, pos0);
  int axis[2] = {0, 0};
  if (ra.axes > 1) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int a = 0; a < kRopeMaxAxes - 1; ++a) axis[u] += (a + 1 < ra.axes && rl.f0 + 4 * u >= ra.section_end[a]) ? 1 : 0;
  }
  const int first = load_now(ra.positions + (size_t)axis[0] * T + t);
  return make_int2(first, axis[1] == axis[0] ? first : load_now(ra.positions + (size_t)axis[1] * T + t));
}

// cos and sin of this lane's eight frequencies at positions that are in the table.
__device__ __forceinline__ void rope_load(const RopeArgs& ra, int2 pos, const RopeLane& rl, float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const size_t at = (size_t)(u ? pos.y : pos.x) * (ra.rot_dim / 2) + rl.f0 + 4 * u;
    const float4 c = load_now(reinterpret_cast<const float4*>(ra.cos_t + at));
    const float4 s = load_now(reinterpret_cast<const float4*>(ra.sin_t + at));
    cs[4 * u] = c.x; cs[4 * u + 1] = c.y; cs[4 * u + 2] = c.z; cs[4 * u + 3] = c.w;
    sn[4 * u] = s.x; sn[4 * u + 1] = s.y; sn[4 * u + 2] = s.z; sn[4 * u + 3] = s.w;
  }
}

// cos and sin of this lane's eight frequencies.  False, with the status recorded, when a position that the warp's lanes
// read with is outside the table.
__device__ __forceinline__ bool rope_angles(const RopeArgs& ra, int2 pos, const RopeLane& rl, float (&cs)[8], float (&sn)[8]) {
  if (ra.cos_t == nullptr) return true;  // no rotation at all
  const bool ok = !rl.rot || ((unsigned)pos.x < (unsigned)ra.table_rows && (unsigned)pos.y < (unsigned)ra.table_rows);
  if (!__all_sync(0xffffffffu, ok)) {
    if (lane_id() == 0) record_status(1);
    return false;
  }
  if (rl.rot) rope_load(ra, pos, rl, cs, sn);
  return true;
}

// The same where the warp has several tokens, `width` lanes each (a power of two): a bad position leaves out its token alone,
// and leaves cos and sin as they were.  Lanes without a token (`on` false) ask for nothing.
__device__ __forceinline__ bool rope_angles_each(const RopeArgs& ra, int2 pos, const RopeLane& rl, float (&cs)[8], float (&sn)[8], bool on,
                                                 int width) {
  const bool bad = on && rl.rot && ((unsigned)pos.x >= (unsigned)ra.table_rows || (unsigned)pos.y >= (unsigned)ra.table_rows);
  const uint32_t votes = __ballot_sync(0xffffffffu, bad), lanes = 0xffffffffu >> (32 - width) << (lane_id() & ~(uint32_t)(width - 1));
  if ((votes & lanes) != 0u) {
    if ((lane_id() & (uint32_t)(width - 1)) == 0u) record_status(1);
    return false;
  }
  if (on && rl.rot) rope_load(ra, pos, rl, cs, sn);
  return on;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<BF16>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
}

// x[0..7], x[8..15]: the lane's two chunks.  BACK turns by the opposite angle (the transpose).
template <bool INTER, bool BACK>
__device__ __forceinline__ void rope_rotate(float (&x)[16], const float (&cs)[8], const float (&sn)[8]) {
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    const int i = INTER ? 2 * m : m, j = INTER ? 2 * m + 1 : m + 8;
    const float s = BACK ? -sn[m] : sn[m];
    const float a = x[i], b = x[j];
    x[i] = a * cs[m] - b * s;
    x[j] = b * cs[m] + a * s;
  }
}

// Sum over the d/16 lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = D / 32; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

template <int D>
__device__ __forceinline__ float row_rms_inv(const float (&x)[16], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
  return rsqrtf(row_sum<D>(ss) * (1.f / D) + eps);
}

}  // namespace fa
