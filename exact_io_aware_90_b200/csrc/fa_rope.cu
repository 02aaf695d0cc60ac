// fa_rope.cu — queries and keys made ready for the attention: RMS norm of each head and the rotation by
// position in one pass, its gradient, and the table of angles (see rope.cuh for the row arithmetic).
//
// All three are streams: a few fp32 operations per value read and written, bound by HBM bandwidth.
//
//   fa_qk_norm_rope_kernel      a warp takes one token: its cos and sin are loaded once and serve every
//                               head; 512/d rows at a time, 16-byte loads and stores
//   fa_qk_norm_rope_bwd_kernel  with g the output's gradient turned back by the angle and n = x·r:
//                                 dx = r·(g∘w − n·mean(g∘w∘n)),   dw = Σ_{tokens, heads} g∘n
//                               a warp walks over tokens and keeps its part of dw in registers; the parts
//                               of a block are joined in shared memory and written to the workspace
//   fa_qk_norm_rope_dw_kernel   adds the blocks' parts of dw in a fixed order, so that equal calls give
//                               equal bits
#include "rope.cuh"

namespace fa {

constexpr int kRopeThreads = 256;

// ---------------------------------------------------------------- table
// cos and sin of p·base^(−2i/rot) in 64 bits: an fp32 angle would be off by 2^-24·p radians at position p.
__global__ void __launch_bounds__(256) fa_rope_table_kernel(float* cos_t, float* sin_t, long long n, int half, double log2_base) {
  const long long id = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= n) return;
  const long long p = id / half;
  const int i = (int)(id - p * half);
  double s, c;
  sincos((double)p * exp2(-log2_base * (double)i / (double)half), &s, &c);
  cos_t[id] = (float)c;
  sin_t[id] = (float)s;
}

// ---------------------------------------------------------------- forward
template <int D, bool BF16>
__device__ __forceinline__ void load_weights(const void* w, const RopeLane& rl, float (&x)[16]) {
  const uint8_t* p = static_cast<const uint8_t*>(w);
  unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(p + 2 * rl.c0)), x);
  unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(p + 2 * rl.c1)), x + 8);
}

template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) fa_qk_norm_rope_kernel(const QkArgs a, const RopeArgs ra) {
  constexpr int G = D / 16, RPW = 32 / G;  // lanes per row, rows per warp at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kRopeThreads / 32) + warp;
  if (t >= a.T) return;
  const RopeLane rl = rope_lane<INTER>(lane % G, ra.rot_dim);
  float cs[8], sn[8];
  if (!rope_angles(ra, t, a.T, 0, rl, cs, sn)) return;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int H = part == 0 ? a.Hq : a.Hk;
    const uint8_t* src = static_cast<const uint8_t*>(part == 0 ? a.q : a.k) + (size_t)t * (part == 0 ? a.q_stride : a.k_stride) * 2;
    uint8_t* dst = static_cast<uint8_t*>(part == 0 ? a.q_out : a.k_out) + (size_t)t * (part == 0 ? a.q_out_stride : a.k_out_stride) * 2;
    const void* wp = part == 0 ? a.wq : a.wk;
    float w[16];
    if (wp != nullptr) load_weights<D, BF16>(wp, rl, w);
#pragma unroll 1
    for (int h0 = blockIdx.y * RPW; h0 < H; h0 += gridDim.y * RPW) {
      const int h = h0 + lane / G;
      const bool on = h < H;
      float x[16];
      if (on) {
        const uint8_t* p = src + (size_t)h * D * 2;
        unpack8<BF16>(*reinterpret_cast<const uint4*>(p + 2 * rl.c0), x);
        unpack8<BF16>(*reinterpret_cast<const uint4*>(p + 2 * rl.c1), x + 8);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
      }
      if (wp != nullptr) {
        const float r = row_rms_inv<D>(x, a.eps);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
      }
      if (rl.rot) rope_rotate<INTER, false>(x, cs, sn);
      if (on) {
        uint8_t* p = dst + (size_t)h * D * 2;
        *reinterpret_cast<uint4*>(p + 2 * rl.c0) = pack8<BF16>(x);
        *reinterpret_cast<uint4*>(p + 2 * rl.c1) = pack8<BF16>(x + 8);
      }
    }
  }
}

// ---------------------------------------------------------------- backward
template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) fa_qk_norm_rope_bwd_kernel(const QkBwdArgs a, const RopeArgs ra) {
  constexpr int G = D / 16, RPW = 32 / G, WARPS = kRopeThreads / 32;
  __shared__ float s_dw[WARPS][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool isk = (int)blockIdx.x >= a.q_blocks;  // the first q_blocks blocks take the queries
  const int blk = isk ? blockIdx.x - a.q_blocks : blockIdx.x, nblk = isk ? gridDim.x - a.q_blocks : a.q_blocks;
  const int H = isk ? a.Hk : a.Hq;
  const uint8_t* gy = static_cast<const uint8_t*>(isk ? a.dk_out : a.dq_out);
  const uint8_t* xx = static_cast<const uint8_t*>(isk ? a.k : a.q);
  uint8_t* dx = static_cast<uint8_t*>(isk ? a.dk : a.dq);
  const long long gs = isk ? a.gk_stride : a.gq_stride, xs = isk ? a.k_stride : a.q_stride, ds = isk ? a.dk_stride : a.dq_stride;
  const void* wp = isk ? a.wk : a.wq;
  const RopeLane rl = rope_lane<INTER>(lane % G, ra.rot_dim);
  float w[16], dw[16];
  if (wp != nullptr) load_weights<D, BF16>(wp, rl, w);
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i] = 0.f;
#pragma unroll 1
  for (int t = blk * WARPS + warp; t < a.T; t += nblk * WARPS) {
    float cs[8], sn[8];
    if (!rope_angles(ra, t, a.T, 0, rl, cs, sn)) continue;
#pragma unroll 1
    for (int h0 = 0; h0 < H; h0 += RPW) {
      const int h = h0 + lane / G;
      const bool on = h < H;
      float g[16], x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) g[i] = x[i] = 0.f;
      if (on) {
        const uint8_t* p = gy + ((size_t)t * gs + (size_t)h * D) * 2;
        unpack8<BF16>(*reinterpret_cast<const uint4*>(p + 2 * rl.c0), g);
        unpack8<BF16>(*reinterpret_cast<const uint4*>(p + 2 * rl.c1), g + 8);
        if (wp != nullptr) {
          const uint8_t* px = xx + ((size_t)t * xs + (size_t)h * D) * 2;
          unpack8<BF16>(*reinterpret_cast<const uint4*>(px + 2 * rl.c0), x);
          unpack8<BF16>(*reinterpret_cast<const uint4*>(px + 2 * rl.c1), x + 8);
        }
      }
      if (rl.rot) rope_rotate<INTER, true>(g, cs, sn);
      if (wp != nullptr) {
        const float r = row_rms_inv<D>(x, a.eps);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[i] *= r;
          dw[i] = fmaf(g[i], x[i], dw[i]);
          g[i] *= w[i];
          dot = fmaf(g[i], x[i], dot);
        }
        dot = row_sum<D>(dot) * (1.f / D);
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] = r * (g[i] - x[i] * dot);
      }
      if (on) {
        uint8_t* p = dx + ((size_t)t * ds + (size_t)h * D) * 2;
        *reinterpret_cast<uint4*>(p + 2 * rl.c0) = pack8<BF16>(g);
        *reinterpret_cast<uint4*>(p + 2 * rl.c1) = pack8<BF16>(g + 8);
      }
    }
  }
  if (wp == nullptr) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
#pragma unroll
    for (int off = G; off < 32; off <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], off);
  }
  if (lane < G) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s_dw[warp][rl.c0 + i] = dw[i];
      s_dw[warp][rl.c1 + i] = dw[8 + i];
    }
  }
  __syncthreads();
  for (int f = threadIdx.x; f < D; f += kRopeThreads) {
    float v = 0.f;
#pragma unroll
    for (int u = 0; u < WARPS; ++u) v += s_dw[u][f];
    a.part[(size_t)blockIdx.x * D + f] = v;
  }
}

// Block (part, feature group): 32 features × 32 slices of the blocks' parts.
__global__ void __launch_bounds__(1024) fa_qk_norm_rope_dw_kernel(const float* part, float* dwq, float* dwk, int q_blocks,
                                                                   int k_blocks, int d) {
  __shared__ float s[32][33];
  const bool isk = blockIdx.y != 0;
  const int first = isk ? q_blocks : 0, n = isk ? k_blocks : q_blocks;
  const int f = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float v = 0.f;
  for (int b = slice; b < n; b += 32) v += part[(size_t)(first + b) * d + f];
  s[slice][threadIdx.x & 31] = v;
  __syncthreads();
  if (slice == 0) {
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < 32; ++u) sum += s[u][threadIdx.x];
    (isk ? dwk : dwq)[f] = sum;
  }
}

// ---------------------------------------------------------------- launches
template <int D, bool BF16>
static cudaError_t launch_qk_t(const QkArgs& a, const RopeArgs& ra, cudaStream_t stream) {
  constexpr int RPW = 512 / D;
  const int blocks = (a.T + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  const int most = (max(a.Hq, a.Hk) + RPW - 1) / RPW;
  // few tokens: spread the heads over blocks too, up to one row group each
  const int split = max(1, min(most, 2 * kSmCount / blocks));
  const dim3 grid(blocks, split);
  if (ra.interleaved) fa_qk_norm_rope_kernel<D, BF16, true><<<grid, kRopeThreads, 0, stream>>>(a, ra);
  else fa_qk_norm_rope_kernel<D, BF16, false><<<grid, kRopeThreads, 0, stream>>>(a, ra);
  return cudaPeekAtLastError();
}

cudaError_t launch_qk_norm_rope(const QkArgs& a, const RopeArgs& ra, int d, bool bf16, cudaStream_t stream) {
  if (d == 128) return bf16 ? launch_qk_t<128, true>(a, ra, stream) : launch_qk_t<128, false>(a, ra, stream);
  return bf16 ? launch_qk_t<64, true>(a, ra, stream) : launch_qk_t<64, false>(a, ra, stream);
}

// Blocks for the queries and for the keys: at most kQkBwdBlocks of each, a warp per token at least.
static int qk_bwd_side_blocks(int T) { return max(1, min(kQkBwdBlocks, (T + kRopeThreads / 32 - 1) / (kRopeThreads / 32))); }

template <int D, bool BF16>
static cudaError_t launch_qk_bwd_t(QkBwdArgs a, const RopeArgs& ra, cudaStream_t stream) {
  const int side = qk_bwd_side_blocks(a.T);
  a.q_blocks = side;
  if (ra.interleaved) fa_qk_norm_rope_bwd_kernel<D, BF16, true><<<2 * side, kRopeThreads, 0, stream>>>(a, ra);
  else fa_qk_norm_rope_bwd_kernel<D, BF16, false><<<2 * side, kRopeThreads, 0, stream>>>(a, ra);
  cudaError_t e = cudaPeekAtLastError();
  if (e != cudaSuccess || a.wq == nullptr) return e;
  fa_qk_norm_rope_dw_kernel<<<dim3(D / 32, 2), 1024, 0, stream>>>(a.part, a.dwq, a.dwk, side, side, D);
  return cudaPeekAtLastError();
}

cudaError_t launch_qk_norm_rope_bwd(const QkBwdArgs& a, const RopeArgs& ra, int d, bool bf16, cudaStream_t stream) {
  if (d == 128) return bf16 ? launch_qk_bwd_t<128, true>(a, ra, stream) : launch_qk_bwd_t<128, false>(a, ra, stream);
  return bf16 ? launch_qk_bwd_t<64, true>(a, ra, stream) : launch_qk_bwd_t<64, false>(a, ra, stream);
}

cudaError_t launch_rope_table(float* cos_t, float* sin_t, int rows, int rot_dim, double base, cudaStream_t stream) {
  const long long n = (long long)rows * (rot_dim / 2);
  fa_rope_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(cos_t, sin_t, n, rot_dim / 2, log2(base));
  return cudaPeekAtLastError();
}

}  // namespace fa
