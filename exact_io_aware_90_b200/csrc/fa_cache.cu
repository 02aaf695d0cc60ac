// fa_cache.cu — writing a paged key/value cache and reading it back.
//
//   fa_cache_append_kernel  new keys (normed and rotated on the way, rope.cuh) and values to their places in
//                           the pages, 16-bit or 4-bit, and the new queries rotated into q_out, in one launch
//   fa_cache_gather_kernel  rows of the pages back into packed [T, Hk, d] arrays
//
// Both are streams bound by HBM bandwidth when there are many tokens, and by the launch when there are a
// few.  A warp takes one token and 512/d heads at a time (d/16 lanes per row, 16-byte accesses).  A 4-bit
// row is made from the row rounded to 16 bits — what the 16-bit cache would hold — so that both formats
// start from the same values.
#include "paged.cuh"
#include "rope.cuh"

namespace fa {

constexpr int kCacheThreads = 256;

// Sequence b of token t and its place in the sequence's new tokens; false when no sequence owns t.
// Records FA_ERR_INVALID_ARG for offsets that are inconsistent.
__device__ __forceinline__ bool owner_of(const int32_t* cu, int B, int T, int t, int& b, int& i, int& n) {
  if (cu == nullptr) {
    n = T / B;
    b = t / n;
    i = t - b * n;
    return true;
  }
  b = find_sequence(cu, B, t);
  if (b >= B) return false;
  const int first = __ldg(cu + b), end = __ldg(cu + b + 1);
  if (t < first) return false;  // before the first sequence
  if (first < 0 || end > T || t >= end) {
    if (lane_id() == 0) record_status(1);
    return false;
  }
  i = t - first;
  n = end - first;
  return true;
}

template <int D, bool BF16, bool INTER, bool Q4>
__global__ void __launch_bounds__(kCacheThreads) fa_cache_append_kernel(const AppendArgs a, const RopeArgs ra, const PagedArgs pg) {
  constexpr int G = D / 16, RPW = 32 / G, W = D / 32;
  __shared__ uint4 s_rows[Q4 ? kCacheThreads / 32 : 1][Q4 ? 64 : 1];  // a warp's rows, 512 values
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % G;
  const int t = blockIdx.x * (kCacheThreads / 32) + warp;
  if (t >= a.T) return;
  int b, i, n;
  if (!owner_of(a.cu_seqlens, pg.B, a.T, t, b, i, n)) return;
  const int len = __ldg(pg.seqlens_k + b);
  const int at = len - n + i;
  int slot;
  const int page = page_of(pg, b, len < n ? -1 : at, slot);
  if (page < 0) return;
  const RopeLane rl = rope_lane<INTER>(l, ra.rot_dim);
  float cs[8], sn[8];
  if (!rope_angles(ra, rope_positions(ra, t, a.T, at, rl), rl, cs, sn)) return;
  const int gq = (a.Hq + RPW - 1) / RPW, gk = (pg.Hk + RPW - 1) / RPW;
#pragma unroll 1
  for (int gi = blockIdx.y; gi < gq + 2 * gk; gi += gridDim.y) {
    const int part = gi < gq ? 0 : gi < gq + gk ? 1 : 2;  // queries, keys, values
    const int h = (part == 0 ? gi : part == 1 ? gi - gq : gi - gq - gk) * RPW + lane / G;
    const bool on = h < (part == 0 ? a.Hq : pg.Hk);
    const uint8_t* src = static_cast<const uint8_t*>(part == 0 ? a.q : part == 1 ? a.k : a.v) +
                         ((size_t)t * (part == 0 ? a.q_stride : part == 1 ? a.k_stride : a.v_stride) + (size_t)h * D) * 2;
    uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
    if (on) {
      u0 = *reinterpret_cast<const uint4*>(src + 2 * rl.c0);
      u1 = *reinterpret_cast<const uint4*>(src + 2 * rl.c1);
    }
    const void* wp = part == 0 ? a.wq : part == 1 ? a.wk : nullptr;
    if (part < 2 && (wp != nullptr || ra.cos_t != nullptr)) {
      float x[16];
      unpack8<BF16>(u0, x);
      unpack8<BF16>(u1, x + 8);
      if (wp != nullptr) {
        const float r = row_rms_inv<D>(x, a.eps);
        float w[16];
        const uint8_t* p = static_cast<const uint8_t*>(wp);
        unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(p + 2 * rl.c0)), w);
        unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(p + 2 * rl.c1)), w + 8);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = x[j] * r * w[j];
      }
      if (rl.rot && ra.cos_t != nullptr) rope_rotate<INTER, false>(x, cs, sn);
      u0 = pack8<BF16>(x);
      u1 = pack8<BF16>(x + 8);
    }
    if (part == 0) {
      if (on) {
        uint8_t* p = static_cast<uint8_t*>(a.q_out) + ((size_t)t * a.q_out_stride + (size_t)h * D) * 2;
        *reinterpret_cast<uint4*>(p + 2 * rl.c0) = u0;
        *reinterpret_cast<uint4*>(p + 2 * rl.c1) = u1;
      }
      continue;
    }
    uint8_t* block = static_cast<uint8_t*>(part == 1 ? pg.k_cache : pg.v_cache) +
                     ((size_t)page * pg.Hk + h) * cache_block_bytes(D, pg.page_size, Q4);
    if constexpr (!Q4) {
      if (on) {
        uint8_t* p = block + (size_t)slot * D * 2;
        *reinterpret_cast<uint4*>(p + 2 * rl.c0) = u0;
        *reinterpret_cast<uint4*>(p + 2 * rl.c1) = u1;
      }
    } else {
      // through shared memory: from the rotation's chunks to 16 consecutive features, half a group
      uint4* row = &s_rows[warp][(lane / G) * (D / 8)];
      row[rl.c0 / 8] = u0;
      row[rl.c1 / 8] = u1;
      __syncwarp();
      float x[16];
      unpack8<BF16>(row[2 * l], x);
      unpack8<BF16>(row[2 * l + 1], x + 8);
      __syncwarp();
      uint32_t num[16];
      const uint32_t pair = quantise16(x, num);
      const int w = l >> 1, half = l & 1;
      if (on) {
        uint8_t* p = block + (size_t)slot * (D / 2);
        if (part == 1) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) word |= num[8 * u + j] << (4 * j);
            reinterpret_cast<uint32_t*>(p)[(2 * half + u) * W + w] = word;
          }
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) word |= num[4 * u + j] << (4 * j);
            reinterpret_cast<uint16_t*>(p)[(4 * half + u) * W + w] = (uint16_t)word;
          }
        }
        if (half == 0)
          reinterpret_cast<uint32_t*>(block + (size_t)pg.page_size * (D / 2) + (size_t)slot * (D / 8))[w] = pair;
      }
    }
  }
}

// 16 consecutive values (half a group) from their 4-bit numbers.
__device__ __forceinline__ void dequantise16(const uint32_t (&n)[16], uint32_t pair, float (&x)[16]) {
  const float sc = __half2float(__ushort_as_half((unsigned short)(pair & 0xffffu)));
  const float mn = __half2float(__ushort_as_half((unsigned short)(pair >> 16)));
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = fmaf((float)n[i], sc, mn);
}

template <int D, bool BF16, bool Q4>
__global__ void __launch_bounds__(kCacheThreads) fa_cache_gather_kernel(const GatherArgs a, const PagedArgs pg) {
  constexpr int G = D / 16, RPW = 32 / G, W = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % G;
  const int t = blockIdx.x * (kCacheThreads / 32) + warp;
  if (t >= a.T) return;
  int b, i, n;
  if (!owner_of(a.cu_seqlens, pg.B, a.T, t, b, i, n)) return;
  const int start = a.starts != nullptr ? __ldg(a.starts + b) : 0;
  int slot;
  const int page = page_of(pg, b, start < 0 || start > 0x7fffffff - i ? -1 : start + i, slot);
  if (page < 0) return;
  const int gk = (pg.Hk + RPW - 1) / RPW;
#pragma unroll 1
  for (int gi = blockIdx.y; gi < 2 * gk; gi += gridDim.y) {
    const bool isv = gi >= gk;
    const int h = (isv ? gi - gk : gi) * RPW + lane / G;
    if (h >= pg.Hk) continue;
    const uint8_t* block = static_cast<const uint8_t*>(isv ? pg.v_cache : pg.k_cache) +
                           ((size_t)page * pg.Hk + h) * cache_block_bytes(D, pg.page_size, Q4);
    uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(isv ? a.v : a.k) + ((size_t)t * pg.Hk + h) * D * 2);
    if constexpr (!Q4) {
      const uint4* p = reinterpret_cast<const uint4*>(block + (size_t)slot * D * 2);
      const uint4 u0 = __ldg(p + l), u1 = __ldg(p + G + l);
      out[l] = u0;
      out[G + l] = u1;
    } else {
      const uint8_t* p = block + (size_t)slot * (D / 2);
      const int w = l >> 1, half = l & 1;
      const uint32_t pair = __ldg(reinterpret_cast<const uint32_t*>(block + (size_t)pg.page_size * (D / 2) + (size_t)slot * (D / 8)) + w);
      uint32_t num[16];
      if (!isv) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t word = __ldg(reinterpret_cast<const uint32_t*>(p) + (2 * half + u) * W + w);
#pragma unroll
          for (int j = 0; j < 8; ++j) num[8 * u + j] = (word >> (4 * j)) & 15u;
        }
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t word = __ldg(reinterpret_cast<const uint16_t*>(p) + (4 * half + u) * W + w);
#pragma unroll
          for (int j = 0; j < 4; ++j) num[4 * u + j] = (word >> (4 * j)) & 15u;
        }
      }
      float x[16];
      dequantise16(num, pair, x);
      out[2 * l] = pack8<BF16>(x);
      out[2 * l + 1] = pack8<BF16>(x + 8);
    }
  }
}

// Blocks of eight tokens; few of them: the head groups are spread over blocks too.
static dim3 cache_grid(int T, int groups) {
  const int blocks = (T + kCacheThreads / 32 - 1) / (kCacheThreads / 32);
  return dim3(blocks, max(1, min(groups, 2 * kSmCount / blocks)));
}

template <int D, bool BF16>
static cudaError_t launch_append_t(const AppendArgs& a, const RopeArgs& ra, const PagedArgs& pg, cudaStream_t stream) {
  constexpr int RPW = 512 / D;
  const dim3 grid = cache_grid(a.T, (a.Hq + RPW - 1) / RPW + 2 * ((pg.Hk + RPW - 1) / RPW));
  if (pg.q4) {
    if (ra.interleaved) fa_cache_append_kernel<D, BF16, true, true><<<grid, kCacheThreads, 0, stream>>>(a, ra, pg);
    else fa_cache_append_kernel<D, BF16, false, true><<<grid, kCacheThreads, 0, stream>>>(a, ra, pg);
  } else {
    if (ra.interleaved) fa_cache_append_kernel<D, BF16, true, false><<<grid, kCacheThreads, 0, stream>>>(a, ra, pg);
    else fa_cache_append_kernel<D, BF16, false, false><<<grid, kCacheThreads, 0, stream>>>(a, ra, pg);
  }
  return cudaPeekAtLastError();
}

cudaError_t launch_cache_append(const AppendArgs& a, const RopeArgs& ra, const PagedArgs& pg, cudaStream_t stream) {
  if (pg.d == 128) return pg.bf16 ? launch_append_t<128, true>(a, ra, pg, stream) : launch_append_t<128, false>(a, ra, pg, stream);
  return pg.bf16 ? launch_append_t<64, true>(a, ra, pg, stream) : launch_append_t<64, false>(a, ra, pg, stream);
}

template <int D, bool BF16>
static cudaError_t launch_gather_t(const GatherArgs& a, const PagedArgs& pg, cudaStream_t stream) {
  constexpr int RPW = 512 / D;
  const dim3 grid = cache_grid(a.T, 2 * ((pg.Hk + RPW - 1) / RPW));
  if (pg.q4) fa_cache_gather_kernel<D, BF16, true><<<grid, kCacheThreads, 0, stream>>>(a, pg);
  else fa_cache_gather_kernel<D, BF16, false><<<grid, kCacheThreads, 0, stream>>>(a, pg);
  return cudaPeekAtLastError();
}

cudaError_t launch_cache_gather(const GatherArgs& a, const PagedArgs& pg, cudaStream_t stream) {
  if (pg.d == 128) return pg.bf16 ? launch_gather_t<128, true>(a, pg, stream) : launch_gather_t<128, false>(a, pg, stream);
  return pg.bf16 ? launch_gather_t<64, true>(a, pg, stream) : launch_gather_t<64, false>(a, pg, stream);
}

}  // namespace fa
