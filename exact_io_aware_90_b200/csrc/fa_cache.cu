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

// The work is dealt out as units of 512/d rows: for each token the groups of its query heads, of its key heads, of its
// value heads.  A warp takes a run of units, so few tokens spread over as many warps as there are units, and many tokens
// keep their lookups and angles for a dozen units.  The rows come ahead through a ring in shared memory; each lane copies
// the pieces it will read itself, so nothing waits for another thread.
constexpr int kCacheStages = 8;
constexpr int kCacheRing = kCacheThreads / 32 * kCacheStages * 2 * 32 * 16;
constexpr int kCacheBlocks = 3;  // per SM: 168 KB in flight

template <int D, bool BF16, bool INTER, bool Q4>
__global__ void __launch_bounds__(kCacheThreads, kCacheBlocks) fa_cache_append_kernel(const AppendArgs a, const RopeArgs ra,
                                                                                      const PagedArgs pg, int share) {
  constexpr int G = D / 16, RPW = 32 / G, W = D / 32;
  extern __shared__ __align__(16) uint4 s_ring[];                      // [warps][stages][2 pieces][lanes]
  __shared__ uint4 s_rows[Q4 ? kCacheThreads / 32 : 1][Q4 ? 64 : 1];  // a warp's rows, 512 values
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % G;
  const int gq = (a.Hq + RPW - 1) / RPW, gk = (pg.Hk + RPW - 1) / RPW, groups = gq + 2 * gk;
  const long long u0 = ((long long)blockIdx.x * (kCacheThreads / 32) + warp) * share, all = (long long)a.T * groups;
  if (u0 >= all) return;
  int left = (int)min((long long)share, all - u0), to_copy = left;
  int t = (int)(u0 / groups), gi = (int)(u0 - (long long)t * groups);
  const RopeLane rl = rope_lane<INTER>(l, ra.rot_dim);
  uint4* mine = s_ring + warp * (kCacheStages * 2 * 32) + lane;
  int t_next = t, g_next = gi, stage = 0, stage_next = 0;
  auto issue = [&]() {
    if (to_copy > 0) {
      --to_copy;
      const int part = g_next < gq ? 0 : g_next < gq + gk ? 1 : 2;  // queries, keys, values
      const int h = (part == 0 ? g_next : part == 1 ? g_next - gq : g_next - gq - gk) * RPW + lane / G;
      if (h < (part == 0 ? a.Hq : pg.Hk)) {
        const uint8_t* src = static_cast<const uint8_t*>(part == 0 ? a.q : part == 1 ? a.k : a.v) +
                             ((size_t)t_next * (part == 0 ? a.q_stride : part == 1 ? a.k_stride : a.v_stride) + (size_t)h * D) * 2;
        const uint32_t to = smem_u32(mine + stage_next * 64);
        cp_async16(to, src + 2 * rl.c0);
        cp_async16(to + 512, src + 2 * rl.c1);
      }
      if (++g_next == groups) {
        g_next = 0;
        ++t_next;
      }
    }
    stage_next = stage_next + 1 == kCacheStages ? 0 : stage_next + 1;
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kCacheStages - 1; ++s) issue();
  float cs[8], sn[8];
  int page = -1, slot = 0;
  bool fresh = true;  // the token's lookups are to be made
#pragma unroll 1
  for (; left > 0; --left) {
    if (fresh) {
      fresh = false;
      int b, i, n;
      page = -1;
      if (owner_of(a.cu_seqlens, pg.B, a.T, t, b, i, n)) {
        const int len = __ldg(pg.seqlens_k + b);
        const int at = len - n + i;
        const int2 pos = rope_positions(ra, t, a.T, at, rl);
        page = page_of(pg, b, len < n ? -1 : at, slot);
        if (page >= 0 && !rope_angles(ra, pos, rl, cs, sn)) page = -1;
      }
    }
    const int part = gi < gq ? 0 : gi < gq + gk ? 1 : 2, t_now = t;
    const int h = (part == 0 ? gi : part == 1 ? gi - gq : gi - gq - gk) * RPW + lane / G;
    const bool on = h < (part == 0 ? a.Hq : pg.Hk);
    if (++gi == groups) {
      gi = 0;
      ++t;
      fresh = true;
    }
    cp_async_wait<kCacheStages - 2>();
    const uint4* from = mine + stage * 64;
    stage = stage + 1 == kCacheStages ? 0 : stage + 1;
    uint4 p0 = make_uint4(0, 0, 0, 0), p1 = p0;
    if (on) {
      p0 = from[0];
      p1 = from[32];
    }
    issue();  // into the place that the last turn read
    if (page < 0) continue;  // no sequence's token, or one that cannot be placed
    {
      const void* wp = part == 0 ? a.wq : part == 1 ? a.wk : nullptr;
      if (part < 2 && (wp != nullptr || ra.cos_t != nullptr)) {
        float x[16];
        unpack8<BF16>(p0, x);
        unpack8<BF16>(p1, x + 8);
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
        p0 = pack8<BF16>(x);
        p1 = pack8<BF16>(x + 8);
      }
      if (part == 0) {
        if (on) {
          uint8_t* p = static_cast<uint8_t*>(a.q_out) + ((size_t)t_now * a.q_out_stride + (size_t)h * D) * 2;
          __stcs(reinterpret_cast<uint4*>(p + 2 * rl.c0), p0);
          __stcs(reinterpret_cast<uint4*>(p + 2 * rl.c1), p1);
        }
        continue;
      }
      uint8_t* block = static_cast<uint8_t*>(part == 1 ? pg.k_cache : pg.v_cache) +
                       ((size_t)page * pg.Hk + h) * cache_block_bytes(D, pg.page_size, Q4);
      if constexpr (!Q4) {
        if (on) {
          uint8_t* p = block + (size_t)slot * D * 2;
          *reinterpret_cast<uint4*>(p + 2 * rl.c0) = p0;
          *reinterpret_cast<uint4*>(p + 2 * rl.c1) = p1;
        }
      } else {
        // through shared memory: from the rotation's chunks to 16 consecutive features, half a group
        uint4* row = &s_rows[warp][(lane / G) * (D / 8)];
        row[rl.c0 / 8] = p0;
        row[rl.c1 / 8] = p1;
        __syncwarp();
        float x[16];
        unpack8<BF16>(row[2 * l], x);
        unpack8<BF16>(row[2 * l + 1], x + 8);
        __syncwarp();
        uint32_t num[16];  // a number in the low 4 bits of each
        const uint32_t pair = quantise16(x, num);
        // and back, from the numbers to the row's bytes in the cache's order, 8 of them a lane
        const int w = l >> 1, half = l & 1;
        if (part == 1) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t word = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) word |= (num[8 * j + e] & 15u) << (4 * e);
            reinterpret_cast<uint32_t*>(row)[(2 * half + j) * W + w] = word;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t word = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) word |= (num[4 * j + e] & 15u) << (4 * e);
            reinterpret_cast<uint16_t*>(row)[(4 * half + j) * W + w] = (uint16_t)word;
          }
        }
        __syncwarp();
        if (on) {
          *reinterpret_cast<uint2*>(block + (size_t)slot * (D / 2) + 8 * l) = reinterpret_cast<const uint2*>(row)[l];
          if (half == 0)
            reinterpret_cast<uint32_t*>(block + (size_t)pg.page_size * (D / 2) + (size_t)slot * (D / 8))[w] = pair;
        }
        __syncwarp();
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

template <int D, bool BF16, bool INTER, bool Q4>
static cudaError_t launch_append_v(const AppendArgs& a, const RopeArgs& ra, const PagedArgs& pg, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  auto kernel = fa_cache_append_kernel<D, BF16, INTER, Q4>;
  cudaError_t e = set_smem_once(done, reinterpret_cast<const void*>(kernel), kCacheRing);
  if (e != cudaSuccess) return e;
  constexpr int RPW = 512 / D, WARPS = kCacheThreads / 32;
  const long long units = (long long)a.T * ((a.Hq + RPW - 1) / RPW + 2 * ((pg.Hk + RPW - 1) / RPW));
  const long long share = (units + kCacheBlocks * kSmCount * WARPS - 1) / (kCacheBlocks * kSmCount * WARPS);
  const int blocks = (int)((units + share * WARPS - 1) / (share * WARPS));
  kernel<<<blocks, kCacheThreads, kCacheRing, stream>>>(a, ra, pg, (int)share);
  return cudaPeekAtLastError();
}

template <int D, bool BF16>
static cudaError_t launch_append_t(const AppendArgs& a, const RopeArgs& ra, const PagedArgs& pg, cudaStream_t stream) {
  if (ra.interleaved) return pg.q4 ? launch_append_v<D, BF16, true, true>(a, ra, pg, stream) : launch_append_v<D, BF16, true, false>(a, ra, pg, stream);
  return pg.q4 ? launch_append_v<D, BF16, false, true>(a, ra, pg, stream) : launch_append_v<D, BF16, false, false>(a, ra, pg, stream);
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
