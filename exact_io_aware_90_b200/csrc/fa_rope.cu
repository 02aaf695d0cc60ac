// fa_rope.cu — queries and keys made ready for the attention: RMS norm of each head and the rotation by
// position in one pass, its gradient, and the table of angles (see rope.cuh for the row arithmetic).
//
// Streams of a few fp32 operations per value read and written, bound by HBM bandwidth where there are many tokens
// (32768 tokens of 16 + 16 heads, d = 128, bf16: forward 541 MB in 91 us, gradient 810 MB in 132 us, 91 and 94 % of the
// measured copy bandwidth; under the power cap of long runs 93 and 142) and by the launch where there are few.
//
//   fa_qk_norm_rope_kernel      a warp takes one token: its cos and sin are loaded once and serve every
//                               head; 512/d rows at a time, 16-byte loads and stores
//   fa_qk_norm_rope_bwd_kernel  with g the output's gradient turned back by the angle and n = x·r:
//                                 dx = r·(g∘w − n·mean(g∘w∘n)),   dw = Σ_{tokens, heads} g∘n
//                               a warp walks over tokens and keeps its part of dw in registers; its rows come
//                               through a ring in shared memory (from registers alone, one group ahead: 176 us);
//                               the parts of a block are joined in shared memory and written to the workspace
//   fa_qk_norm_rope_dw_kernel   adds the blocks' parts of dw in a fixed order, so that equal calls give
//                               equal bits
#include "async_copy.cuh"
#include "rope.cuh"

namespace fa {

constexpr int kRopeThreads = 256;
constexpr int kRopeStages = 4;  // of the backward's ring: 64 KB per block, three stages (48 KB) in flight; two blocks per SM
constexpr int kRopeRing = kRopeThreads / 32 * kRopeStages * 4 * 32 * 16;

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
  unpack8<BF16>(load_now(reinterpret_cast<const uint4*>(p + 2 * rl.c0)), x);
  unpack8<BF16>(load_now(reinterpret_cast<const uint4*>(p + 2 * rl.c1)), x + 8);
}

// U: row groups (of 512/d rows) that a warp loads before it works on the first.
template <int D, bool BF16, bool INTER, int U>
__global__ void __launch_bounds__(kRopeThreads, 3) fa_qk_norm_rope_kernel(const QkArgs a, const RopeArgs ra) {
  constexpr int G = D / 16, RPW = 32 / G;  // lanes per row, rows per warp at a time
  after_earlier_kernels();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kRopeThreads / 32) + warp;
  if (t >= a.T) return;
  const RopeLane rl = rope_lane<INTER>(lane % G, ra.rot_dim);
  float cs[8], sn[8];
  if (!rope_angles(ra, rope_positions(ra, t, a.T, 0, rl), rl, cs, sn)) return;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int H = part == 0 ? a.Hq : a.Hk;
    const uint8_t* src = static_cast<const uint8_t*>(part == 0 ? a.q : a.k) + (size_t)t * (part == 0 ? a.q_stride : a.k_stride) * 2;
    uint8_t* dst = static_cast<uint8_t*>(part == 0 ? a.q_out : a.k_out) + (size_t)t * (part == 0 ? a.q_out_stride : a.k_out_stride) * 2;
    const void* wp = part == 0 ? a.wq : a.wk;
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;  // the weights stay packed: unpacking costs less than the registers
    if (wp != nullptr) {
      w0 = load_now(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(wp) + 2 * rl.c0));
      w1 = load_now(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(wp) + 2 * rl.c1));
    }
#pragma unroll 1
    for (int h0 = blockIdx.y * (RPW * U); h0 < H; h0 += gridDim.y * (RPW * U)) {
      const int h = h0 + lane / G;
      uint4 v0[U], v1[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v0[u] = v1[u] = make_uint4(0, 0, 0, 0);
        if (h + u * RPW < H) {
          const uint8_t* p = src + (size_t)(h + u * RPW) * D * 2;
          v0[u] = load_once(reinterpret_cast<const uint4*>(p + 2 * rl.c0));
          v1[u] = load_once(reinterpret_cast<const uint4*>(p + 2 * rl.c1));
        }
      }
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
          for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
        }
        if (rl.rot) rope_rotate<INTER, false>(x, cs, sn);
        if (h + u * RPW < H) {
          uint8_t* p = dst + (size_t)(h + u * RPW) * D * 2;
          __stcs(reinterpret_cast<uint4*>(p + 2 * rl.c0), pack8<BF16>(x));
          __stcs(reinterpret_cast<uint4*>(p + 2 * rl.c1), pack8<BF16>(x + 8));
        }
      }
    }
  }
}

// ---------------------------------------------------------------- backward
template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2) fa_qk_norm_rope_bwd_kernel(const QkBwdArgs a, const RopeArgs ra) {
  constexpr int G = D / 16, RPW = 32 / G, WARPS = kRopeThreads / 32;
  extern __shared__ __align__(16) uint4 s_ring[];  // [warps][stages][4 pieces][lanes]
  __shared__ float s_dw[WARPS][D];
  after_earlier_kernels();
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
  uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
  if (wp != nullptr) {
    w0 = load_now(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(wp) + 2 * rl.c0));
    w1 = load_now(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(wp) + 2 * rl.c1));
  }
  float dw[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i] = 0.f;
  // Each lane copies the pieces of its own rows ahead into its own places of the ring, so that no other thread is waited
  // for: the copies in flight, 2 KB a group, do not take registers.
  uint4* mine = s_ring + warp * (kRopeStages * 4 * 32) + lane;
  // Fewer heads than the warp has rows: it takes several tokens at a time, HP rows each (12527 tokens of 2 + 1 heads, d = 128:
  // 10.4 us against 22.6 with one token at a time).  t: this lane's token.
  const int bits = H >= RPW ? (D == 64 ? 3 : 2) : H > 4 ? 3 : H > 2 ? 2 : H - 1, HP = 1 << bits;
  const int first = lane / G >> bits, hl = lane / G & (HP - 1);
  const int step = nblk * WARPS * (RPW >> bits);
  int t = (blk * WARPS + warp) * (RPW >> bits) + first, h0 = 0, t_next = t, h_next = 0, stage = 0, stage_next = 0;
  auto issue = [&]() {
    const int h = h_next + hl;
    if (t_next < a.T && h < H) {
      const uint32_t to = smem_u32(mine + stage_next * 128);
      const uint8_t* p = gy + ((size_t)t_next * gs + (size_t)h * D) * 2;
      cp_async16(to, p + 2 * rl.c0);
      cp_async16(to + 512, p + 2 * rl.c1);
      if (wp != nullptr) {
        const uint8_t* px = xx + ((size_t)t_next * xs + (size_t)h * D) * 2;
        cp_async16(to + 1024, px + 2 * rl.c0);
        cp_async16(to + 1536, px + 2 * rl.c1);
      }
    }
    cp_async_commit();
    stage_next = stage_next + 1 == kRopeStages ? 0 : stage_next + 1;
    h_next += HP;
    if (h_next >= H) {
      h_next = 0;
      t_next += step;
    }
  };
#pragma unroll
  for (int s = 0; s < kRopeStages - 1; ++s) issue();
  float cs[8] = {}, sn[8] = {};
  bool ok = false;
  int2 pos = t < a.T ? rope_positions(ra, t, a.T, 0, rl) : make_int2(0, 0);
#pragma unroll 1
  while (t - first < a.T) {
    if (h0 == 0) ok = rope_angles_each(ra, pos, rl, cs, sn, t < a.T, G << bits);
    const int t_now = t, h = h0 + hl;
    h0 += HP;
    if (h0 >= H) {
      h0 = 0;
      t += step;
      if (t < a.T) pos = rope_positions(ra, t, a.T, 0, rl);
    }
    cp_async_wait<kRopeStages - 2>();
    const uint4* from = mine + stage * 128;
    stage = stage + 1 == kRopeStages ? 0 : stage + 1;
    float g[16], x[16];
    const bool on = h < H && ok;  // a position out of range: the token is left out
    const uint4 none = make_uint4(0, 0, 0, 0);
    unpack8<BF16>(on ? from[0] : none, g);
    unpack8<BF16>(on ? from[32] : none, g + 8);
    unpack8<BF16>(on && wp != nullptr ? from[64] : none, x);
    unpack8<BF16>(on && wp != nullptr ? from[96] : none, x + 8);
    issue();  // into the place that the last turn read
    if (rl.rot) rope_rotate<INTER, true>(g, cs, sn);
    if (wp != nullptr) {
      const float r = row_rms_inv<D>(x, a.eps);
      float dot = 0.f, w[16];
      unpack8<BF16>(w0, w);
      unpack8<BF16>(w1, w + 8);
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
      uint8_t* p = dx + ((size_t)t_now * ds + (size_t)h * D) * 2;
      __stcs(reinterpret_cast<uint4*>(p + 2 * rl.c0), pack8<BF16>(g));
      __stcs(reinterpret_cast<uint4*>(p + 2 * rl.c1), pack8<BF16>(g + 8));
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
  after_earlier_kernels();
  float v = 0.f;
#pragma unroll 4
  for (int b = slice; b < n; b += 32) v += load_now(part + (size_t)(first + b) * d + f);
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
template <int D, bool BF16, int U>
static cudaError_t launch_qk_u(const QkArgs& a, const RopeArgs& ra, int blocks, cudaStream_t stream) {
  const int most = (max(a.Hq, a.Hk) + 512 / D * U - 1) / (512 / D * U);
  const dim3 grid(blocks, max(1, min(most, 2 * kSmCount / blocks)));  // few tokens: the heads are spread over blocks too
  return launch_after(ra.interleaved ? fa_qk_norm_rope_kernel<D, BF16, true, U> : fa_qk_norm_rope_kernel<D, BF16, false, U>, grid,
                      dim3(kRopeThreads), 0, stream, a, ra);
}

// Two row groups ahead where the blocks fill the GPU (32768 tokens x 32 heads, d = 128: 89.6 us against 110.7 with one
// and 101 with four); one where they do not, so that there are more of them (1171 tokens: 3.7 us against 4.1).
template <int D, bool BF16>
static cudaError_t launch_qk_t(const QkArgs& a, const RopeArgs& ra, cudaStream_t stream) {
  const int blocks = (a.T + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  return blocks >= 2 * kSmCount ? launch_qk_u<D, BF16, 2>(a, ra, blocks, stream) : launch_qk_u<D, BF16, 1>(a, ra, blocks, stream);
}

cudaError_t launch_qk_norm_rope(const QkArgs& a, const RopeArgs& ra, int d, bool bf16, cudaStream_t stream) {
  if (d == 128) return bf16 ? launch_qk_t<128, true>(a, ra, stream) : launch_qk_t<128, false>(a, ra, stream);
  return bf16 ? launch_qk_t<64, true>(a, ra, stream) : launch_qk_t<64, false>(a, ra, stream);
}

// One wave of blocks (two per SM), shared between the queries and the keys by the row groups of a token, of which a small
// number of heads fills a part; a warp per group at least.
template <int D, bool BF16>
static cudaError_t launch_qk_bwd_t(QkBwdArgs a, const RopeArgs& ra, cudaStream_t stream) {
  constexpr int RPW = 512 / D, WARPS = kRopeThreads / 32;
  auto rows = [](int H) { return H >= RPW ? (H + RPW - 1) / RPW * RPW : H > 4 ? 8 : H > 2 ? 4 : H; };
  auto most = [&](int H) {
    const int tokens = H >= RPW ? WARPS : WARPS * RPW / rows(H);  // of a block
    return max(1, (a.T + tokens - 1) / tokens);
  };
  const int share = max(1, min(kQkBwdBlocks - 1, (int)((long long)kQkBwdBlocks * rows(a.Hq) / (rows(a.Hq) + rows(a.Hk)))));
  a.q_blocks = min(most(a.Hq), share);
  const int k_blocks = min(most(a.Hk), kQkBwdBlocks - share);
  auto kernel = ra.interleaved ? fa_qk_norm_rope_bwd_kernel<D, BF16, true> : fa_qk_norm_rope_bwd_kernel<D, BF16, false>;
  static std::atomic<unsigned long long> done[2] = {{0}, {0}};
  cudaError_t e = set_smem_once(done[ra.interleaved], reinterpret_cast<const void*>(kernel), kRopeRing);
  if (e != cudaSuccess) return e;
  e = launch_after(kernel, dim3(a.q_blocks + k_blocks), dim3(kRopeThreads), kRopeRing, stream, a, ra);
  if (e != cudaSuccess || a.wq == nullptr) return e;
  return launch_after(fa_qk_norm_rope_dw_kernel, dim3(D / 32, 2), dim3(1024), 0, stream, (const float*)a.part, a.dwq, a.dwk, a.q_blocks, k_blocks, D);
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
