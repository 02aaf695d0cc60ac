// fa_paged.cu — attention of a few new queries per sequence over a paged key/value cache, 16-bit or 4-bit.
//
//   fa_paged_split_kernel  one block per (sequence, key head, tile of query rows, chunk of keys): partial
//                          (m, ℓ, Õ = Σ_j 2^(s_j − m) v_j) of the chunk, s = scale·log2(e)·q·k (base 2)
//   fa_paged_merge_kernel  joins the chunks of a row: m = max m_c, ℓ = Σ ℓ_c·2^(m_c − m), Õ the same way
//
// The query rows of a key head are its H/Hk query heads times the Nq new tokens; 8 or 16 of them share one
// pass over the keys, so a key is read once for the whole group.  The call is a stream over the cache, and
// the products run on the tensor cores only so that 8 or 16 rows cost no more instructions than one.  The
// tile is small (16 keys by 8 rows), which the warp-level matrix instructions fit; tcgen05 would want 128
// rows of keys in shared memory in its own layout, and the 4-bit numbers would have to be written there
// after unpacking.
//
// Orders are chosen so that no operand moves between lanes.  With g = lane/4, t = lane%4:
//   scores   Sᵀ[16 keys × 8 rows] = K·qᵀ.  A lane loads whole 16-byte pieces of keys g and g + 8 and takes the
//            features in the order they arrive; the query operand is loaded in the same order.
//   output   Oᵀ[16 features × 8 rows] += Vᵀ·Pᵀ.  A lane loads pieces of keys 2t, 2t+1, 2t+8, 2t+9 and pairs
//            neighbouring keys with byte permutes; P is transposed in registers (movmatrix).
// A lane's scores and outputs belong to the same two rows (2t, 2t+1), so rescaling needs no exchange either.
//
// 4-bit numbers are used where they lie: a masked half word with n in bits 0-3 is the fp16 n·2^-24, with n in
// bits 4-7 n·2^-20 (subnormal, and exact in the products).  The queries are taken to fp16 by a power of two per
// row that brings the largest to 2^12 (exact but for features 2^-26 below it), those that meet the 2^-20 form by
// 2^-4 less.  Each group of 32 features has its own fp32 accumulator, so its scale and minimum enter once per key:
//   s = Σ_w scale_w·(q·n)_w + min_w·(Σ q)_w.
// For the output the value's scale multiplies P before P is rounded to fp16, and Σ_j p_j·min_j is kept in fp32.
// The reference of the exponent is the running maximum of s + log2(largest value scale), so that what is rounded
// is at most 2^14 whatever the scales are.
//
// The reference rises only when a score passes it by 2^8 (one vote per tile); P of 16-bit caches is the sum of two
// 16-bit parts, so its rounding stays behind the output's.
#include "paged.cuh"

namespace fa {

constexpr int kPagedWarps = 4;
constexpr int kPagedThreads = 32 * kPagedWarps;
constexpr float kRise = 8.f;  // how far a score may pass the reference before the reference follows

struct PagedParams {
  const uint8_t* q;
  void* o;
  float* lse;
  float* part_o;   // [rows, nchunk, d]
  float* part_ml;  // [rows, nchunk, 2]
  PagedArgs pg;
  int Nq, H, G, most, R, chunk, nchunk;  // G = H/Hk, most: the largest length allowed, R = G·Nq rows of a key head
  float scale_log2;
};

template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8×8 matrix of 16-bit elements: lane (g, t) gives row g, columns 2t, 2t+1 and gets the same of the transpose.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// The sequence's key count, or -1 (recorded) when it is out of range.
__device__ __forceinline__ int paged_length(const PagedParams& p, int b) {
  const int L = __ldg(p.pg.seqlens_k + b);
  if (L < 0 || L > p.most) {
    if (threadIdx.x == 0) record_status(1);
    return -1;
  }
  return L;
}

// What a part with maximum m weighs beside the maximum of all, M.  Parts without a key (m = -inf) hold zeros, or
// NaN where every score was NaN, which has to stay.
__device__ __forceinline__ float join_weight(float m, float M) { return m == M ? 1.f : ex2(m - M); }

// The row of q, o and lse for row r of key head hk.
__device__ __forceinline__ size_t paged_row(const PagedParams& p, int b, int hk, int r) {
  const int i = r / p.G, gh = r - i * p.G;
  return ((size_t)b * p.Nq + i) * p.H + (size_t)hk * p.G + gh;
}

template <int D, bool BF16>
__device__ __forceinline__ void store_out(void* o, size_t at, float v) {
  if constexpr (BF16) reinterpret_cast<__nv_bfloat16*>(o)[at] = __float2bfloat16_rn(v);
  else reinterpret_cast<__half*>(o)[at] = __float2half_rn(v);
}

template <int D, bool BF16, bool Q4, int NT>
__global__ void __launch_bounds__(kPagedThreads) fa_paged_split_kernel(const PagedParams p) {
  constexpr int W = D / 32;           // groups of 32 features
  constexpr int KS = D / 16;          // k-steps of the scores; feature tiles of the output
  constexpr bool MB = BF16 && !Q4;    // operand type of the products
  constexpr int ROWS = 8 * NT;
  __shared__ float s_m[kPagedWarps][ROWS], s_l[kPagedWarps][ROWS];
  __shared__ float s_o[kPagedWarps][ROWS][D + 4];
  const int c = blockIdx.x, b = blockIdx.z;
  const int hk = blockIdx.y % p.pg.Hk, r0 = (blockIdx.y / p.pg.Hk) * ROWS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int L = paged_length(p, b);
  if (L < 0) return;
  const int k0 = c * p.chunk, k1 = min(L, k0 + p.chunk);
  if (k0 >= L && c > 0) return;  // the merge reads the chunks inside the sequence, and the first one

  // ---- queries: operand registers, and for 4 bits the row's power of two and the sums of its groups
  uint32_t qb[NT][KS][2];
  float coef[NT][2], qsum[NT][2][Q4 ? W : 1];
  int lim[NT][2];  // the last key each of this lane's rows (2t, 2t+1) sees
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = r0 + 8 * nt + g;
    const bool on = r < p.R;
    const uint8_t* src = p.q + (on ? paged_row(p, b, hk, r) : 0) * D * 2;
    uint32_t w[W][4];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const uint4 v = on ? __ldg(reinterpret_cast<const uint4*>(src + (32 * j + 8 * t) * 2)) : make_uint4(0, 0, 0, 0);
      w[j][0] = v.x; w[j][1] = v.y; w[j][2] = v.z; w[j][3] = v.w;
    }
    if constexpr (!Q4) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        qb[nt][2 * j][0] = w[j][0];
        qb[nt][2 * j][1] = w[j][1];
        qb[nt][2 * j + 1][0] = w[j][2];
        qb[nt][2 * j + 1][1] = w[j][3];
      }
      coef[nt][0] = coef[nt][1] = p.scale_log2;
    } else {
      float f[W][8], most = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = unpack2<BF16>(w[j][i]);
          f[j][2 * i] = x.x;
          f[j][2 * i + 1] = x.y;
          most = fmaxf(most, fmaxf(fabsf(x.x), fabsf(x.y)));
        }
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // most = m·2^e, 1 <= m < 2; the row goes into the products as q·2^(12 − e)
      const int e = min(max((int)(__float_as_uint(most) >> 23) - 127, -100), 100);
      const float up = __uint_as_float((uint32_t)(127 + 12 - e) << 23);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float lo = up, hi = up * 0.0625f;  // the factors beside n·2^-24 and n·2^-20
        qb[nt][2 * j][0] = pack2<false>(f[j][0] * lo, f[j][4] * lo);
        qb[nt][2 * j][1] = pack2<false>(f[j][1] * hi, f[j][5] * hi);
        qb[nt][2 * j + 1][0] = pack2<false>(f[j][2] * lo, f[j][6] * lo);
        qb[nt][2 * j + 1][1] = pack2<false>(f[j][3] * hi, f[j][7] * hi);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += f[j][i];
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        // from the lanes of row g to the lanes that hold rows 2t, 2t+1
        qsum[nt][0][j] = __shfl_sync(0xffffffffu, s, 8 * t) * p.scale_log2;
        qsum[nt][1][j] = __shfl_sync(0xffffffffu, s, 8 * t + 4) * p.scale_log2;
      }
      const float back = __uint_as_float((uint32_t)(127 + 12 + e) << 23) * p.scale_log2;  // 2^(e − 12 + 24)
      coef[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);
      coef[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int rr = r0 + 8 * nt + 2 * t + u;
      lim[nt][u] = L - p.Nq + (rr < p.R ? rr / p.G : p.Nq - 1);
    }
  }

  float m[NT][2], l[NT][2], o[NT][KS][4], omin[NT][2][Q4 ? W : 1];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      m[nt][u] = -INFINITY;
      l[nt][u] = 0.f;
#pragma unroll
      for (int j = 0; j < (Q4 ? W : 1); ++j) omin[nt][u][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[nt][j][i] = 0.f;
  }

  const size_t block_bytes = cache_block_bytes(D, p.pg.page_size, Q4);
  const int ps = p.pg.page_size;
#pragma unroll 1
  for (int j0 = k0 + 16 * warp; j0 < k1; j0 += 16 * kPagedWarps) {
    int slot;
    const int page = page_of(p.pg, b, j0, slot);
    if (page < 0) continue;
    const size_t blk = ((size_t)page * p.pg.Hk + hk) * block_bytes;
    const uint8_t* kb = static_cast<const uint8_t*>(p.pg.k_cache) + blk;
    const uint8_t* vb = static_cast<const uint8_t*>(p.pg.v_cache) + blk;
    const bool tail = j0 + 16 > L;

    // ---- scores of keys j0 + g and j0 + g + 8
    float s[NT][4];
    uint32_t vpair[Q4 ? 2 : 1][Q4 ? W : 1];  // (scale, min) of the values of keys g, g + 8
    if constexpr (!Q4) {
      uint4 ka[W][2];
#pragma unroll
      for (int j = 0; j < W; ++j) {
        ka[j][0] = __ldg(reinterpret_cast<const uint4*>(kb + ((size_t)(slot + g) * D + 32 * j + 8 * t) * 2));
        ka[j][1] = __ldg(reinterpret_cast<const uint4*>(kb + ((size_t)(slot + g + 8) * D + 32 * j + 8 * t) * 2));
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          mma_16816<MB>(s[nt], ka[j][0].x, ka[j][1].x, ka[j][0].y, ka[j][1].y, qb[nt][2 * j][0], qb[nt][2 * j][1]);
          mma_16816<MB>(s[nt], ka[j][0].z, ka[j][1].z, ka[j][0].w, ka[j][1].w, qb[nt][2 * j + 1][0], qb[nt][2 * j + 1][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] *= p.scale_log2;
      }
    } else {
      uint32_t kn[2][W], kp[2][W];
      const uint8_t* kpair = kb + (size_t)ps * (D / 2);
      const uint8_t* vp = vb + (size_t)ps * (D / 2);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = slot + g + 8 * u;
        if constexpr (W == 4) {
          const uint4 a = __ldg(reinterpret_cast<const uint4*>(kb + (size_t)row * (D / 2)) + t);
          const uint4 y = __ldg(reinterpret_cast<const uint4*>(kpair + (size_t)row * (D / 8)));
          const uint4 z = __ldg(reinterpret_cast<const uint4*>(vp + (size_t)row * (D / 8)));
          kn[u][0] = a.x; kn[u][1] = a.y; kn[u][2] = a.z; kn[u][3] = a.w;
          kp[u][0] = y.x; kp[u][1] = y.y; kp[u][2] = y.z; kp[u][3] = y.w;
          vpair[u][0] = z.x; vpair[u][1] = z.y; vpair[u][2] = z.z; vpair[u][3] = z.w;
        } else {
          const uint2 a = __ldg(reinterpret_cast<const uint2*>(kb + (size_t)row * (D / 2)) + t);
          const uint2 y = __ldg(reinterpret_cast<const uint2*>(kpair + (size_t)row * (D / 8)));
          const uint2 z = __ldg(reinterpret_cast<const uint2*>(vp + (size_t)row * (D / 8)));
          kn[u][0] = a.x; kn[u][1] = a.y;
          kp[u][0] = y.x; kp[u][1] = y.y;
          vpair[u][0] = z.x; vpair[u][1] = z.y;
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint32_t x0 = kn[0][j], x1 = kn[1][j], y0 = x0 >> 8, y1 = x1 >> 8;
        const float2 p0 = __half22float2(*reinterpret_cast<const __half2*>(&kp[0][j]));
        const float2 p1 = __half22float2(*reinterpret_cast<const __half2*>(&kp[1][j]));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          mma_16816<false>(acc, x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, qb[nt][2 * j][0], qb[nt][2 * j][1]);
          mma_16816<false>(acc, y0 & 0x000f000fu, y1 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x00f000f0u, qb[nt][2 * j + 1][0],
                           qb[nt][2 * j + 1][1]);
          s[nt][0] = fmaf(p0.x, acc[0] * coef[nt][0], fmaf(p0.y, qsum[nt][0][j], s[nt][0]));
          s[nt][1] = fmaf(p0.x, acc[1] * coef[nt][1], fmaf(p0.y, qsum[nt][1][j], s[nt][1]));
          s[nt][2] = fmaf(p1.x, acc[2] * coef[nt][0], fmaf(p1.y, qsum[nt][0][j], s[nt][2]));
          s[nt][3] = fmaf(p1.x, acc[3] * coef[nt][1], fmaf(p1.y, qsum[nt][1][j], s[nt][3]));
        }
      }
    }
    // ---- keys behind a row's last one; rows behind the sequence's end hold anything, so they are replaced, not scaled
    if (j0 + 15 > L - p.Nq) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (j0 + g > lim[nt][0]) s[nt][0] = -INFINITY;
        if (j0 + g > lim[nt][1]) s[nt][1] = -INFINITY;
        if (j0 + g + 8 > lim[nt][0]) s[nt][2] = -INFINITY;
        if (j0 + g + 8 > lim[nt][1]) s[nt][3] = -INFINITY;
      }
    }
    float2 vsc[Q4 ? 2 : 1][Q4 ? W : 1];
    float lift[2] = {0.f, 0.f};
    if constexpr (Q4) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float most = 5.9604644775390625e-08f;  // 2^-24, the smallest scale above zero
#pragma unroll
        for (int j = 0; j < W; ++j) {
          vsc[u][j] = __half22float2(*reinterpret_cast<const __half2*>(&vpair[u][j]));
          if (tail && j0 + g + 8 * u >= L) vsc[u][j] = make_float2(0.f, 0.f);
          most = fmaxf(most, vsc[u][j].x);
        }
        lift[u] = __log2f(most);
      }
    }
    // ---- the reference
    bool rise = false;  // also for NaN, which then stays in the sum
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) rise = rise || !(s[nt][i] + lift[i >> 1] <= m[nt][i & 1] + kRise);
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float x = fmaxf(s[nt][u] + lift[0], s[nt][2 + u] + lift[1]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float mn = fmaxf(m[nt][u], x);
          const float alpha = m[nt][u] == -INFINITY ? 0.f : ex2(m[nt][u] - mn);
          m[nt][u] = mn;
          l[nt][u] *= alpha;
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            o[nt][j][u] *= alpha;
            o[nt][j][2 + u] *= alpha;
          }
          if constexpr (Q4) {
#pragma unroll
            for (int j = 0; j < W; ++j) omin[nt][u][j] *= alpha;
          }
        }
    }
    // ---- probabilities, relative to the reference
    float pr[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
      pr[nt][0] = ex2(s[nt][0] - m0);
      pr[nt][1] = ex2(s[nt][1] - m1);
      pr[nt][2] = ex2(s[nt][2] - m0);
      pr[nt][3] = ex2(s[nt][3] - m1);
      l[nt][0] += pr[nt][0] + pr[nt][2];
      l[nt][1] += pr[nt][1] + pr[nt][3];
    }
    // ---- output
    const int key[4] = {2 * t, 2 * t + 1, 2 * t + 8, 2 * t + 9};
    if constexpr (!Q4) {
      uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t hi = pack2<MB>(pr[nt][2 * u], pr[nt][2 * u + 1]);
          const float2 back = unpack2<MB>(hi);
          const uint32_t lo = pack2<MB>(pr[nt][2 * u] - back.x, pr[nt][2 * u + 1] - back.y);
          bh[nt][u] = movmatrix_trans(hi);
          bl[nt][u] = movmatrix_trans(lo);
        }
#pragma unroll
      for (int cc = 0; cc < D / 64; ++cc) {
        uint32_t v[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 x = __ldg(reinterpret_cast<const uint4*>(vb + ((size_t)(slot + key[i]) * D + 64 * cc + 8 * g) * 2));
          if (tail && j0 + key[i] >= L) x = make_uint4(0, 0, 0, 0);
          v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
        }
        if (j0 + 15 <= L - p.Nq || p.Nq == 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = prmt(v[0][i], v[1][i], 0x5410u), a1 = prmt(v[0][i], v[1][i], 0x7632u);
            const uint32_t a2 = prmt(v[2][i], v[3][i], 0x5410u), a3 = prmt(v[2][i], v[3][i], 0x7632u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_16816<MB>(o[nt][4 * cc + i], a0, a1, a2, a3, bh[nt][0], bh[nt][1]);
              mma_16816<MB>(o[nt][4 * cc + i], a0, a1, a2, a3, bl[nt][0], bl[nt][1]);
            }
          }
        } else {
          // the last keys, which the new tokens see one after another: a token at a time with the values behind
          // it taken out, since an infinity or NaN there would pass a zero probability
#pragma unroll 1
          for (int last = max(j0, L - p.Nq); last < min(j0 + 16, L); ++last) {
            // rows whose last key is `last`, or lies behind this tile when `last` is the tile's end
            const bool end = last == j0 + 15;
            uint32_t x[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) x[u][i] = j0 + key[u] <= last ? v[u][i] : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t a0 = prmt(x[0][i], x[1][i], 0x5410u), a1 = prmt(x[0][i], x[1][i], 0x7632u);
              const uint32_t a2 = prmt(x[2][i], x[3][i], 0x5410u), a3 = prmt(x[2][i], x[3][i], 0x7632u);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float tmp[4] = {0.f, 0.f, 0.f, 0.f};
                mma_16816<MB>(tmp, a0, a1, a2, a3, bh[nt][0], bh[nt][1]);
                mma_16816<MB>(tmp, a0, a1, a2, a3, bl[nt][0], bl[nt][1]);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  if (lim[nt][u & 1] == last || (end && lim[nt][u & 1] > last)) o[nt][4 * cc + i][u] += tmp[u];
              }
            }
          }
        }
      }
    } else {
      uint32_t v[4][W / 2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* row = vb + (size_t)(slot + key[i]) * (D / 2);
        if constexpr (W == 4) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(row) + g);
          v[i][0] = x.x;
          v[i][1] = x.y;
        } else {
          v[i][0] = __ldg(reinterpret_cast<const uint32_t*>(row) + g);
        }
      }
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
        const uint32_t e = prmt(v[0][j >> 1], v[1][j >> 1], sel), f = prmt(v[2][j >> 1], v[3][j >> 1], sel);
        const uint32_t e8 = e >> 8, f8 = f >> 8;
        const float s0 = vsc[0][j].x * 64.f, s1 = vsc[1][j].x * 64.f;  // P·scale up to 2^14
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t b0 = movmatrix_trans(pack2<false>(pr[nt][0] * s0, pr[nt][1] * s0));
          const uint32_t b1 = movmatrix_trans(pack2<false>(pr[nt][2] * s1, pr[nt][3] * s1));
          mma_16816<false>(o[nt][2 * j], e & 0x000f000fu, e & 0x00f000f0u, f & 0x000f000fu, f & 0x00f000f0u, b0, b1);
          mma_16816<false>(o[nt][2 * j + 1], e8 & 0x000f000fu, e8 & 0x00f000f0u, f8 & 0x000f000fu, f8 & 0x00f000f0u, b0, b1);
          omin[nt][0][j] = fmaf(pr[nt][0], vsc[0][j].y, fmaf(pr[nt][2], vsc[1][j].y, omin[nt][0][j]));
          omin[nt][1][j] = fmaf(pr[nt][1], vsc[0][j].y, fmaf(pr[nt][3], vsc[1][j].y, omin[nt][1][j]));
        }
      }
    }
  }

  // ---- the warp's partial result to shared memory
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = 8 * nt + 2 * t + u;
      float x = l[nt][u];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (g == 0) {
        s_m[warp][r] = m[nt][u];
        s_l[warp][r] = x;
      }
      if constexpr (!Q4) {
#pragma unroll
        for (int cc = 0; cc < D / 64; ++cc)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s_o[warp][r][64 * cc + 8 * g + 2 * i] = o[nt][4 * cc + i][u];
            s_o[warp][r][64 * cc + 8 * g + 2 * i + 1] = o[nt][4 * cc + i][2 + u];
          }
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) {
          float y = omin[nt][u][j];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
          float* dst = &s_o[warp][r][32 * j + 4 * g];
          dst[0] = fmaf(o[nt][2 * j][u], 262144.f, y);          // 2^(24 − 6)
          dst[1] = fmaf(o[nt][2 * j][2 + u], 16384.f, y);       // 2^(20 − 6)
          dst[2] = fmaf(o[nt][2 * j + 1][u], 262144.f, y);
          dst[3] = fmaf(o[nt][2 * j + 1][2 + u], 16384.f, y);
        }
      }
    }
  __syncthreads();
  // ---- the block's: a warp per row, d/32 features per lane
  for (int r = warp; r < ROWS && r0 + r < p.R; r += kPagedWarps) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kPagedWarps; ++w) M = fmaxf(M, s_m[w][r]);
    float ell = 0.f, acc[W];
#pragma unroll
    for (int j = 0; j < W; ++j) acc[j] = 0.f;
#pragma unroll
    for (int w = 0; w < kPagedWarps; ++w) {
      const float a = join_weight(s_m[w][r], M);
      ell = fmaf(s_l[w][r], a, ell);
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] = fmaf(s_o[w][r][32 * j + lane], a, acc[j]);
    }
    const size_t row = paged_row(p, b, hk, r0 + r);
    if (p.nchunk == 1) {
      const float inv = ell == 0.f ? 0.f : 1.f / ell;
#pragma unroll
      for (int j = 0; j < W; ++j) store_out<D, BF16>(p.o, row * D + 32 * j + lane, acc[j] * inv);
      if (lane == 0) p.lse[row] = ell == 0.f ? -INFINITY : (M + log2f(ell)) * 0.69314718055994531f;
    } else {
      const size_t slot = row * p.nchunk + c;
#pragma unroll
      for (int j = 0; j < W; ++j) p.part_o[slot * D + 32 * j + lane] = acc[j];
      if (lane == 0) {
        p.part_ml[2 * slot] = M;
        p.part_ml[2 * slot + 1] = ell;
      }
    }
  }
}

// One block per row of q: the warps take the chunks in turn, then join.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) fa_paged_merge_kernel(const PagedParams p) {
  constexpr int F = D / 32;
  __shared__ float s_o[4][D], s_l[4];
  const size_t row = blockIdx.x;
  const int b = (int)(row / ((size_t)p.Nq * p.H));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = paged_length(p, b);
  if (L < 0) return;
  const int nc = max(1, (L + p.chunk - 1) / p.chunk);
  const float* ml = p.part_ml + row * p.nchunk * 2;
  float M = -INFINITY;
  for (int c = lane; c < nc; c += 32) M = fmaxf(M, ml[2 * c]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float ell = 0.f, acc[F];
#pragma unroll
  for (int j = 0; j < F; ++j) acc[j] = 0.f;
#pragma unroll 4
  for (int c = warp; c < nc; c += 4) {
    const float a = join_weight(ml[2 * c], M);
    ell = fmaf(ml[2 * c + 1], a, ell);
    const float* src = p.part_o + (row * p.nchunk + c) * D;
#pragma unroll
    for (int j = 0; j < F; ++j) acc[j] = fmaf(src[32 * j + lane], a, acc[j]);
  }
#pragma unroll
  for (int j = 0; j < F; ++j) s_o[warp][32 * j + lane] = acc[j];
  if (lane == 0) s_l[warp] = ell;
  __syncthreads();
  ell = s_l[0] + s_l[1] + s_l[2] + s_l[3];
  const float inv = ell == 0.f ? 0.f : 1.f / ell;
  for (int f = threadIdx.x; f < D; f += 128)
    store_out<D, BF16>(p.o, row * D + f, (s_o[0][f] + s_o[1][f] + s_o[2][f] + s_o[3][f]) * inv);
  if (threadIdx.x == 0) p.lse[row] = ell == 0.f ? -INFINITY : (M + log2f(ell)) * 0.69314718055994531f;
}

// Keys per chunk: enough blocks to fill the GPU a few times over, whole tiles for every warp.
int paged_chunk(int B, int Nq, int H, int Hk, int Nk) {
  const int R = H / Hk * Nq;
  const long long units = (long long)B * Hk * (R <= 8 ? 1 : (R + 15) / 16);
  const int step = 16 * kPagedWarps;
  const long long want = std::max(1LL, std::min<long long>((8LL * kSmCount + units - 1) / units, (Nk + 2 * step - 1) / (2 * step)));
  const int chunk = (int)((Nk + want - 1) / want);
  return (chunk + step - 1) / step * step;
}

template <int D, bool BF16>
static cudaError_t launch_paged_t(const PagedParams& p, cudaStream_t stream) {
  const int rt = p.R <= 8 ? 1 : (p.R + 15) / 16;
  const dim3 grid((unsigned)p.nchunk, (unsigned)(p.pg.Hk * rt), (unsigned)p.pg.B);
  if (p.pg.q4) {
    if (p.R <= 8) fa_paged_split_kernel<D, BF16, true, 1><<<grid, kPagedThreads, 0, stream>>>(p);
    else fa_paged_split_kernel<D, BF16, true, 2><<<grid, kPagedThreads, 0, stream>>>(p);
  } else {
    if (p.R <= 8) fa_paged_split_kernel<D, BF16, false, 1><<<grid, kPagedThreads, 0, stream>>>(p);
    else fa_paged_split_kernel<D, BF16, false, 2><<<grid, kPagedThreads, 0, stream>>>(p);
  }
  cudaError_t e = cudaPeekAtLastError();
  if (e != cudaSuccess || p.nchunk == 1) return e;
  fa_paged_merge_kernel<D, BF16><<<(unsigned)((size_t)p.pg.B * p.Nq * p.H), 128, 0, stream>>>(p);
  return cudaPeekAtLastError();
}

cudaError_t launch_decode_paged(const PagedDecodeArgs& a, const PagedArgs& pg, cudaStream_t stream) {
  PagedParams p;
  p.q = static_cast<const uint8_t*>(a.q);
  p.o = a.o;
  p.lse = a.lse;
  p.part_o = a.part_o;
  p.part_ml = a.part_ml;
  p.pg = pg;
  p.Nq = a.Nq;
  p.H = a.H;
  p.G = a.H / pg.Hk;
  p.most = std::min(a.Nk, pg.max_pages * pg.page_size);
  p.R = p.G * a.Nq;
  p.chunk = paged_chunk(pg.B, a.Nq, a.H, pg.Hk, a.Nk);
  p.nchunk = (a.Nk + p.chunk - 1) / p.chunk;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  if (pg.d == 128) return pg.bf16 ? launch_paged_t<128, true>(p, stream) : launch_paged_t<128, false>(p, stream);
  return pg.bf16 ? launch_paged_t<64, true>(p, stream) : launch_paged_t<64, false>(p, stream);
}

}  // namespace fa
