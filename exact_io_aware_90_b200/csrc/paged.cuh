// paged.cuh — the paged key/value cache: addresses of its rows, the 4-bit row format, and the search for
// the sequence that owns a token.
//
// A cache is pages of page_size tokens; the keys and the values of one (page, head) are one contiguous
// block, so that a tile of a page is one contiguous copy.
//   16 bits  page_size rows of d elements
//   4 bits   page_size rows of d/2 bytes of numbers, then page_size rows of d/32 (scale, min) pairs of
//            fp16, one pair for each 32 features of the row: the value is number·scale + min
// The order of the numbers in a row is the order in which the decode kernel's lanes hold them (W = d/32):
//   key    feature 32w + 8t + n (t < 4, n < 8): nibble n of 32-bit word t·W + w
//   value  feature 32w + 4g + n (g < 8, n < 4): nibble n of 16-bit word g·W + w
#pragma once

#include "async_copy.cuh"
#include "fa_paged_internal.h"
#include "sm100.cuh"

namespace fa {

// Bytes of one (page, head) block.
__host__ __device__ constexpr size_t cache_block_bytes(int d, int page_size, bool q4) {
  return q4 ? (size_t)page_size * (d / 2 + d / 8) : (size_t)page_size * d * 2;
}

// The sequence that owns token t: the number of entries of cu[1..B] that are <= t (B when none owns it).
// All 32 lanes call it; each step looks at 32 evenly spaced entries.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int B, int t) {
  const int lane = (int)lane_id();
  int lo = 0, n = B;
  while (n > 32) {
    const int step = (n + 31) / 32;
    const int i = (lane + 1) * step - 1;
    const bool below = i < n && load_now(cu + 1 + lo + i) <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, below));
    lo += c * step;
    n = min(step, n - c * step);
    if (n <= 0) return lo;
  }
  const bool below = lane < n && load_now(cu + 1 + lo + lane) <= t;
  return lo + __popc(__ballot_sync(0xffffffffu, below));
}

// Page of position `at` of sequence b, or -1 with the status recorded (one lane's worth) when the
// position or the table's entry is out of range.
__device__ __forceinline__ int page_of(const PagedArgs& p, int b, int at, int& slot) {
  int page = -1;
  slot = 0;
  if (at >= 0 && at / p.page_size < p.max_pages) {
    const int i = at / p.page_size;
    slot = at - i * p.page_size;
    page = load_now(p.page_table + (size_t)b * p.max_pages + i);
    if (page >= p.num_pages) page = -1;
  }
  if (page < 0) {
    if (lane_id() == 0) record_status(1);
    return -1;
  }
  return page;
}

template <bool BF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16) asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 16 consecutive values of a row (half of a group of 32; the other half is in the neighbouring lane, lane
// xor 1) as 4-bit numbers: n[i] is 0x4B400000 plus the number (the fp32 bits of 1.5·2^23 + number), and the result the
// group's scale and minimum as fp16 bits (scale in the low half).  The minimum is rounded to fp16 first and the numbers
// are taken from it, so its rounding adds no error.
// A number is (x − min)/scale to nearest even, kept within 0..15.  The product with the reciprocal is rounded by adding
// 1.5·2^23; where some remainder x − min − n·scale (one rounding) reaches half a scale, the lane does its numbers again
// and lets the remainder decide.  An IEEE division per value took 65 us more for 33.9k tokens of 8 heads.
constexpr float kRound = 12582912.f;  // 1.5·2^23
template <bool BF16>
__device__ __forceinline__ uint32_t quantise16(const uint4& v0, const uint4& v1, uint32_t (&n)[16]) {
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  uint32_t lo2 = w[0], hi2 = w[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo2 = min2<BF16>(lo2, w[i]);
    hi2 = max2<BF16>(hi2, w[i]);
  }
  lo2 = min2<BF16>(lo2, __shfl_xor_sync(0xffffffffu, lo2, 1));
  hi2 = max2<BF16>(hi2, __shfl_xor_sync(0xffffffffu, hi2, 1));
  const float2 l = unpack2<BF16>(lo2), h = unpack2<BF16>(hi2);
  const float lo = fminf(l.x, l.y), hi = fmaxf(h.x, h.y);
  const __half hmin = __float2half_rn(fminf(fmaxf(lo, -65504.f), 65504.f));
  const __half hsc = __float2half_rn(fminf(__fdiv_rn(hi - lo, 15.f), 65504.f));
  const float mn = __half2float(hmin), sc = __half2float(hsc);
  const float inv = sc > 0.f ? __fdividef(1.f, sc) : 0.f, share = inv * (1.f / 15.f);
  const float half = sc > 0.f ? 0.5f * sc : INFINITY;
  bool close = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 x = unpack2<BF16>(w[i / 2]);
    const float a = ((i & 1) ? x.y : x.x) - mn;
    const float v = fmaf(__saturatef(a * share), 15.f, kRound);
    close |= fabsf(fmaf(v - kRound, -sc, a)) >= half;
    n[i] = __float_as_uint(v);
  }
  if (close) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 x = unpack2<BF16>(w[i / 2]);
      const float a = ((i & 1) ? x.y : x.x) - mn;
      float v = fmaf(fminf(fmaxf(a * inv, -1.f), 16.f), 1.f, kRound);
      const float rest = fmaf(v - kRound, -sc, a);
      // past the middle, or in it and odd
      if (fabsf(rest) > half || (fabsf(rest) == half && (__float_as_uint(v) & 1u) != 0u)) v += rest < 0.f ? -1.f : 1.f;
      n[i] = __float_as_uint(fminf(fmaxf(v, kRound), kRound + 15.f));
    }
  }
  return (uint32_t)__half_as_ushort(hsc) | ((uint32_t)__half_as_ushort(hmin) << 16);
}

// Eight of these numbers as the nibbles of a word: the sum of n[i]·16^i, less what 0x4B400000 adds to it.
__device__ __forceinline__ uint32_t nibbles8(const uint32_t* n) {
  uint32_t word = 0u - (0x4B400000u + 0xB4000000u + 0x40000000u);
#pragma unroll
  for (int i = 0; i < 8; ++i) word += n[i] << (4 * i);
  return word;
}

}  // namespace fa
