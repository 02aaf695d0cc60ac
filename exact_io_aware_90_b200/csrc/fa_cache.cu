// fa_cache.cu — writing a paged key/value cache and reading it back.
//
//   fa_cache_append_kernel  new keys (normed and rotated on the way, rope.cuh) and values to their places in
//                           the pages, 16-bit or 4-bit, and the new queries rotated into q_out, in one launch
//   fa_cache_gather_kernel  rows of the pages back into packed [T, Hk, d] arrays
//
// Streams.  A warp takes one token and 512/d heads at a time (d/16 lanes per row, 16-byte accesses).  A 4-bit
// row is made from the row rounded to 16 bits — what the 16-bit cache would hold — so that both formats
// start from the same values.
// Measured, bf16, d = 128: append of 31.6k tokens of 32 + 8 + 8 heads, 16 bits 776 MB in 136 us (87 % of the measured copy
// bandwidth), 4 bits 185 us: instructions bound it there (325 per 512/d rows on average, 64 % of the issue slots: the
// minimum, maximum and rounding of a 4-bit row cost twice its norm and rotation; held to 80 registers for three blocks a
// multiprocessor, a thread spills 100 bytes in 4 bits and 28 to 56 in 16, and warps wait for instructions).  Gather of 16 x 8192 keys of 8 heads,
// 16 bits 162 us (101 %), 4 bits 705 MB in 119 us (90 %).  16 tokens appended: 2.9 us, the launch and the chain of lookups.
// A ring of asynchronous copies, as in the norm's gradient, was no faster here: 139 us in 16 bits, and 4 bits the same.
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
  const int first = load_now(cu + b), end = load_now(cu + b + 1);
  if (t < first) return false;  // before the first sequence
  if (first < 0 || end > T || t >= end) {
    if (lane_id() == 0) record_status(1);
    return false;
  }
  i = t - first;
  n = end - first;
  return true;
}

// Stores 512/d rows (this lane's two chunks each) of keys or values as 4-bit rows.  `rows`: the warp's 1 KB in shared
// memory.  From the rotation's chunks to 16 consecutive features a lane (half a group), and from the numbers to the row's
// bytes in the cache's order, 8 of them a lane.
template <int D, bool BF16, bool VALUE>
__device__ __forceinline__ void store_q4(uint4* rows, const RopeLane& rl, int lane, const uint4& p0, const uint4& p1, uint8_t* numbers,
                                         uint8_t* pairs, bool on) {
  constexpr int G = D / 16, W = D / 32;
  const int l = lane % G, w = l >> 1, half = l & 1;
  uint4* row = rows + lane / G * (D / 8);
  __syncwarp();  // the rows before are read
  row[rl.c0 / 8] = p0;
  row[rl.c1 / 8] = p1;
  __syncwarp();
  const uint4 first = row[2 * l], second = row[2 * l + 1];
  __syncwarp();
  uint32_t num[16];
  const uint32_t pair = quantise16<BF16>(first, second, num);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t word = nibbles8(num + 8 * j);
    if constexpr (!VALUE) {
      reinterpret_cast<uint32_t*>(row)[(2 * half + j) * W + w] = word;
    } else {
      reinterpret_cast<uint16_t*>(row)[(4 * half + 2 * j) * W + w] = (uint16_t)word;
      reinterpret_cast<uint16_t*>(row)[(4 * half + 2 * j + 1) * W + w] = (uint16_t)(word >> 16);
    }
  }
  __syncwarp();
  if (on) {
    *reinterpret_cast<uint2*>(numbers + 8 * l) = reinterpret_cast<const uint2*>(row)[l];
    if (half == 0) *reinterpret_cast<uint32_t*>(pairs + 4 * w) = pair;
  }
}

// U: row groups (of 512/d rows) that are loaded together; the first ones are loaded ahead of the token's lookups.  A warp
// does its token's queries, keys and values, or (gridDim.z = 3) one of the three.
template <int D, bool BF16, bool INTER, bool Q4, int U>
__global__ void __launch_bounds__(kCacheThreads, U == 2 ? 3 : 2) fa_cache_append_kernel(const AppendArgs a, const RopeArgs ra, const PagedArgs pg) {
  constexpr int G = D / 16, RPW = 32 / G;
  after_earlier_kernels();
  __shared__ uint4 s_rows[Q4 ? kCacheThreads / 32 : 1][Q4 ? 64 : 1];  // a warp's rows, 512 values
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kCacheThreads / 32) + warp;
  if (t >= a.T) return;
  const RopeLane rl = rope_lane<INTER>(lane % G, ra.rot_dim);
  const int c0 = 2 * rl.c0, c1 = 2 * rl.c1, h_first = blockIdx.y * (RPW * U) + lane / G;
  const uint8_t* src = nullptr;
  int H = 0;
  uint4 v0[U], v1[U];
  auto begin = [&](const void* x, long long stride, int heads) {
    src = static_cast<const uint8_t*>(x) + (t * stride + (long long)h_first * D) * 2;
    H = heads;
  };
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v0[u] = v1[u] = make_uint4(0, 0, 0, 0);
      if (h + u * RPW < H) {
        v0[u] = load_once(reinterpret_cast<const uint4*>(src + u * RPW * D * 2 + c0));
        v1[u] = load_once(reinterpret_cast<const uint4*>(src + u * RPW * D * 2 + c1));
      }
    }
    src += (size_t)gridDim.y * (RPW * U * D * 2);
  };
  const int part0 = gridDim.z == 1 ? (a.Hq > 0 ? 0 : 1) : blockIdx.z, parts = gridDim.z == 1 ? 3 : part0 + 1;
  if (part0 == 0) begin(a.q, a.q_stride, a.Hq);
  else if (part0 == 1) begin(a.k, a.k_stride, pg.Hk);
  else begin(a.v, a.v_stride, pg.Hk);
  load(h_first);

  int b, i, n;
  if (!owner_of(a.cu_seqlens, pg.B, a.T, t, b, i, n)) return;
  const int len = load_now(pg.seqlens_k + b);
  const int at = len - n + i;
  const int2 pos = rope_positions(ra, t, a.T, at, rl);
  int slot;
  const int page = page_of(pg, b, len < n ? -1 : at, slot);
  if (page < 0) return;
  float cs[8], sn[8];
  if (!rope_angles(ra, pos, rl, cs, sn)) return;

  // queries and keys
#pragma unroll 1
  for (int part = part0; part < min(parts, 2); ++part) {
    const void* wp = part == 0 ? a.wq : a.wk;
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    if (wp != nullptr) {
      w0 = load_now(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(wp) + c0));
      w1 = load_now(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(wp) + c1));
    }
    const size_t block = cache_block_bytes(D, pg.page_size, Q4);
    uint8_t* dst = part == 0 ? static_cast<uint8_t*>(a.q_out) + (t * a.q_out_stride + (long long)h_first * D) * 2
                             : static_cast<uint8_t*>(pg.k_cache) + ((size_t)page * pg.Hk + h_first) * block + (size_t)slot * (Q4 ? D / 2 : D * 2);
    const size_t next = part == 0 ? (size_t)RPW * D * 2 : RPW * block;
    const bool packed = Q4 && part == 1;
#pragma unroll 1
    for (int h = h_first; h - lane / G < H; h += gridDim.y * (RPW * U)) {
      if (h != h_first) load(h);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[16];
        unpack8<BF16>(v0[u], x);
        unpack8<BF16>(v1[u], x + 8);
        if (wp != nullptr) {
          const float r = row_rms_inv<D>(x, a.eps);
          float w[16];
          unpack8<BF16>(w0, w);
          unpack8<BF16>(w1, w + 8);
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = x[j] * r * w[j];
        }
        if (rl.rot && ra.cos_t != nullptr) rope_rotate<INTER, false>(x, cs, sn);
        const uint4 p0 = pack8<BF16>(x), p1 = pack8<BF16>(x + 8);
        const bool on = h + u * RPW < H;
        if (packed) {
          if constexpr (Q4)
            store_q4<D, BF16, false>(s_rows[warp], rl, lane, p0, p1, dst + u * next,
                                     dst + u * next + (size_t)(pg.page_size - slot) * (D / 2) + (size_t)slot * (D / 8), on);
        } else if (on) {
          __stcs(reinterpret_cast<uint4*>(dst + u * next + c0), p0);
          __stcs(reinterpret_cast<uint4*>(dst + u * next + c1), p1);
        }
      }
      dst += gridDim.y * U * next;
    }
    if (part + 1 < parts) {
      if (part == 0) begin(a.k, a.k_stride, pg.Hk);
      else begin(a.v, a.v_stride, pg.Hk);
      load(h_first);
    }
  }
  if (parts < 3) return;
  // values
  const size_t next = RPW * cache_block_bytes(D, pg.page_size, Q4);
  uint8_t* dst = static_cast<uint8_t*>(pg.v_cache) + ((size_t)page * pg.Hk + h_first) * (next / RPW) + (size_t)slot * (Q4 ? D / 2 : D * 2);
#pragma unroll 1
  for (int h = h_first; h - lane / G < H; h += gridDim.y * (RPW * U)) {
    if (h != h_first) load(h);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool on = h + u * RPW < H;
      if constexpr (Q4) {
        store_q4<D, BF16, true>(s_rows[warp], rl, lane, v0[u], v1[u], dst + u * next,
                                dst + u * next + (size_t)(pg.page_size - slot) * (D / 2) + (size_t)slot * (D / 8), on);
      } else if (on) {
        __stcs(reinterpret_cast<uint4*>(dst + u * next + c0), v0[u]);
        __stcs(reinterpret_cast<uint4*>(dst + u * next + c1), v1[u]);
      }
    }
    dst += gridDim.y * U * next;
  }
}

// The eight numbers of a word as values x[0..7]: pairs (n, n + 4) under the exponent of 1024, the numbers exact in fp16.
__device__ __forceinline__ void dequantise8(uint32_t word, float2 p0, float2 p1, float* x) {
  const __half2 base = __float2half2_rn(1024.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = ((word >> (4 * i)) & 0x000f000fu) | 0x64006400u;
    const float2 n = __half22float2(__hsub2(*reinterpret_cast<const __half2*>(&m), base));
    x[i] = fmaf(n.x, p0.x, p0.y);
    x[i + 4] = fmaf(n.y, p1.x, p1.y);
  }
}

__device__ __forceinline__ float2 pair_of(uint32_t pair) { return __half22float2(*reinterpret_cast<const __half2*>(&pair)); }

// U groups of 512/d heads are loaded together, keys and values: a 4-bit row has few bytes, so many have to be in flight.
template <int D, bool BF16, bool Q4, int U>
__global__ void __launch_bounds__(kCacheThreads) fa_cache_gather_kernel(const GatherArgs a, const PagedArgs pg) {
  constexpr int G = D / 16, RPW = 32 / G, W = D / 32;
  after_earlier_kernels();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % G;
  const int t = blockIdx.x * (kCacheThreads / 32) + warp;
  if (t >= a.T) return;
  int b, i, n;
  if (!owner_of(a.cu_seqlens, pg.B, a.T, t, b, i, n)) return;
  const int start = a.starts != nullptr ? load_now(a.starts + b) : 0;
  int slot;
  const int page = page_of(pg, b, start < 0 || start > 0x7fffffff - i ? -1 : start + i, slot);
  if (page < 0) return;
  const size_t block = cache_block_bytes(D, pg.page_size, Q4);
  const size_t first = ((size_t)page * pg.Hk + lane / G) * block, row = (size_t)slot * (Q4 ? D / 2 : D * 2);
  const uint8_t* kb = static_cast<const uint8_t*>(pg.k_cache) + first;
  const uint8_t* vb = static_cast<const uint8_t*>(pg.v_cache) + first;
  const size_t out0 = ((size_t)t * pg.Hk + lane / G) * D * 2;
  uint8_t* ko = static_cast<uint8_t*>(a.k) + out0;
  uint8_t* vo = static_cast<uint8_t*>(a.v) + out0;
#pragma unroll 1
  for (int h = blockIdx.y * (RPW * U) + lane / G; h - lane / G < pg.Hk; h += gridDim.y * (RPW * U)) {
    const int off = h - lane / G;
    if constexpr (!Q4) {
      uint4 x[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * RPW < pg.Hk) {
          const uint4* pk = reinterpret_cast<const uint4*>(kb + (off + u * RPW) * block + row);
          const uint4* pv = reinterpret_cast<const uint4*>(vb + (off + u * RPW) * block + row);
          x[u][0] = load_once(pk + l);
          x[u][1] = load_once(pk + G + l);
          x[u][2] = load_once(pv + l);
          x[u][3] = load_once(pv + G + l);
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * RPW < pg.Hk) {
          uint4* qk = reinterpret_cast<uint4*>(ko + (size_t)(off + u * RPW) * D * 2);
          uint4* qv = reinterpret_cast<uint4*>(vo + (size_t)(off + u * RPW) * D * 2);
          __stcs(qk + l, x[u][0]);
          __stcs(qk + G + l, x[u][1]);
          __stcs(qv + l, x[u][2]);
          __stcs(qv + G + l, x[u][3]);
        }
    } else {
      // 8 bytes of a row a lane: of a key two words, 8 features each of two groups; of a value four half words, 4 each
      const int t4 = 2 * l / W, w2 = 2 * l % W;
      const size_t pairs = (size_t)pg.page_size * (D / 2) + (size_t)slot * (D / 8);
      uint2 kn[U], vn[U], kp[U];
      uint32_t vp[U][W];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * RPW < pg.Hk) {
          const uint8_t* pk = kb + (off + u * RPW) * block;
          const uint8_t* pv = vb + (off + u * RPW) * block;
          kn[u] = load_once(reinterpret_cast<const uint2*>(pk + row) + l);
          vn[u] = load_once(reinterpret_cast<const uint2*>(pv + row) + l);
          kp[u] = load_now(reinterpret_cast<const uint2*>(pk + pairs + 4 * w2));
          if constexpr (W == 4) {
            const uint4 v = load_now(reinterpret_cast<const uint4*>(pv + pairs));
            vp[u][0] = v.x; vp[u][1] = v.y; vp[u][2] = v.z; vp[u][3] = v.w;
          } else {
            const uint2 v = load_now(reinterpret_cast<const uint2*>(pv + pairs));
            vp[u][0] = v.x; vp[u][1] = v.y;
          }
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * RPW < pg.Hk) {
          uint4* qk = reinterpret_cast<uint4*>(ko + (size_t)(off + u * RPW) * D * 2);
          uint2* qv = reinterpret_cast<uint2*>(vo + (size_t)(off + u * RPW) * D * 2);
          const float2 p0 = pair_of(kp[u].x), p1 = pair_of(kp[u].y);
          float x[8];
          dequantise8(kn[u].x, p0, p0, x);
          __stcs(qk + 4 * w2 + t4, pack8<BF16>(x));
          dequantise8(kn[u].y, p1, p1, x);
          __stcs(qk + 4 * w2 + 4 + t4, pack8<BF16>(x));
#pragma unroll
          for (int j = 0; j < 4; j += 2) {  // half words 4l + j and 4l + j + 1, of groups w and w + 1
            const int g = 4 * l / W + j / W, w = j % W;
            dequantise8(j ? vn[u].y : vn[u].x, pair_of(vp[u][w]), pair_of(vp[u][w + 1]), x);
            __stcs(qv + 8 * w + g, make_uint2(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3])));
            __stcs(qv + 8 * (w + 1) + g, make_uint2(pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7])));
          }
        }
    }
  }
}

// Blocks of eight tokens; few of them: the head groups are spread over blocks too.
static dim3 cache_grid(int T, int groups) {
  const int blocks = (T + kCacheThreads / 32 - 1) / (kCacheThreads / 32);
  return dim3(blocks, max(1, min(groups, 2 * kSmCount / blocks)));
}

template <int D, bool BF16, bool Q4, int U>
static cudaError_t launch_append_u(const AppendArgs& a, const RopeArgs& ra, const PagedArgs& pg, cudaStream_t stream) {
  constexpr int ROWS = 512 / D * U;
  dim3 grid = cache_grid(a.T, (max(a.Hq, pg.Hk) + ROWS - 1) / ROWS);
  if (U == 1) grid.z = 3;
  return launch_after(ra.interleaved ? fa_cache_append_kernel<D, BF16, true, Q4, U> : fa_cache_append_kernel<D, BF16, false, Q4, U>, grid,
                      dim3(kCacheThreads), 0, stream, a, ra, pg);
}

// Two row groups together where the tokens fill the GPU; else one, with the heads, and queries, keys and values, spread
// over blocks too.
template <int D, bool BF16>
static cudaError_t launch_append_t(const AppendArgs& a, const RopeArgs& ra, const PagedArgs& pg, cudaStream_t stream) {
  const bool many = a.T >= 2 * kSmCount * (kCacheThreads / 32);
  if (pg.q4) return many ? launch_append_u<D, BF16, true, 2>(a, ra, pg, stream) : launch_append_u<D, BF16, true, 1>(a, ra, pg, stream);
  return many ? launch_append_u<D, BF16, false, 2>(a, ra, pg, stream) : launch_append_u<D, BF16, false, 1>(a, ra, pg, stream);
}

cudaError_t launch_cache_append(const AppendArgs& a, const RopeArgs& ra, const PagedArgs& pg, cudaStream_t stream) {
  if (pg.d == 128) return pg.bf16 ? launch_append_t<128, true>(a, ra, pg, stream) : launch_append_t<128, false>(a, ra, pg, stream);
  return pg.bf16 ? launch_append_t<64, true>(a, ra, pg, stream) : launch_append_t<64, false>(a, ra, pg, stream);
}

template <int D, bool BF16>
static cudaError_t launch_gather_t(const GatherArgs& a, const PagedArgs& pg, cudaStream_t stream) {
  constexpr int RPW = 512 / D;
  const bool many = a.T >= 2 * kSmCount * (kCacheThreads / 32) && pg.Hk > RPW;
  const dim3 grid = cache_grid(a.T, (pg.Hk + RPW - 1) / RPW);
  auto kernel = !pg.q4 ? fa_cache_gather_kernel<D, BF16, false, 1> : many ? fa_cache_gather_kernel<D, BF16, true, 2> : fa_cache_gather_kernel<D, BF16, true, 1>;
  return launch_after(kernel, grid, dim3(kCacheThreads), 0, stream, a, pg);
}

cudaError_t launch_cache_gather(const GatherArgs& a, const PagedArgs& pg, cudaStream_t stream) {
  if (pg.d == 128) return pg.bf16 ? launch_gather_t<128, true>(a, pg, stream) : launch_gather_t<128, false>(a, pg, stream);
  return pg.bf16 ? launch_gather_t<64, true>(a, pg, stream) : launch_gather_t<64, false>(a, pg, stream);
}

}  // namespace fa
