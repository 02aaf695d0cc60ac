// fa_paged.cu — attention of a few new queries per sequence over a paged key/value cache, 16-bit or 4-bit.
//
//   fa_paged_split_kernel  one wave of blocks; the keys of all (sequence, key head, tile of query rows) units,
//                          in granules of 64 keys, are dealt out evenly: each block takes a run of granules,
//                          which may end inside a unit and may span several.  A unit that lies in one run is
//                          finished there; of others each block leaves its partial (m, ℓ, Õ = Σ_j 2^(s_j − m) v_j),
//                          s = scale·log2(e)·q·k (base 2)
//   fa_paged_merge_kernel  joins the parts of a row: m = max m_c, ℓ = Σ ℓ_c·2^(m_c − m), Õ the same way
//
// The query rows of a key head are its H/Hk query heads times the Nq new tokens; 8 or 16 of them share one
// pass over the keys, so a key is read once for the whole group.  The call is a stream over the cache, and
// the products run on the tensor cores only so that 8 or 16 rows cost no more instructions than one.  The
// tile is small (16 keys by 8 rows), which the warp-level matrix instructions fit; tcgen05 would want 128
// rows of keys in shared memory in its own layout, and the 4-bit numbers would have to be written there
// after unpacking.
//
// Each warp streams its own 16-key tiles (every fourth 16 keys of the run) through a ring in shared memory
// with asynchronous 16-byte copies; the ring's depth covers the latency of HBM, and no warp waits for another
// until the end of a unit.
//
// Orders are chosen so that no operand moves between lanes.  With g = lane/4, t = lane%4:
//   scores   Sᵀ[16 keys × 8 rows] = K·qᵀ.  A lane reads whole 16-byte pieces of keys g and g + 8 and takes the
//            features in the order they lie; the query operand is loaded in the same order.
//   output   Oᵀ[16 features × 8 rows] += Vᵀ·Pᵀ.  A lane reads pieces of keys 2t, 2t+1, 2t+8, 2t+9 and pairs
//            neighbouring keys with byte permutes; P is transposed in registers (movmatrix).
// A lane's scores and outputs belong to the same two rows (2t, 2t+1), so rescaling needs no exchange either.
// The pieces are written to shared memory at places that keep these reads free of bank conflicts.
//
// 4-bit numbers are used where they lie: a masked half word with n in bits 0-3 is the fp16 n·2^-24, with n in
// bits 4-7 n·2^-20 (subnormal, and exact in the products).  The queries are taken to fp16 by a power of two per
// row that brings the largest to 2^12 (exact but for features 2^-26 below it), those that meet the 2^-20 form by
// 2^-4 less.  Each group of 32 features has its own fp32 accumulator, so its scale and minimum enter once per key:
//   s = Σ_w scale_w·(q·n)_w + min_w·(Σ q)_w.
// For the output the values' numbers are taken to n − 8 (one exact fp16 subtraction), the value's scale multiplies P
// before P is rounded to fp16, and Σ_j p_j·(min_j + 8·scale_j) is kept in fp32.  Without the shift the products would
// add up to a mean of 2 standard deviations per key that the minimum takes away again: over 131071 keys the tensor
// cores' truncating sums then left 8e-4 of the output (now 2e-4, fp16's own rounding).  A power of two above every
// value scale the warp has met brings P·scale under 2^14; it follows the scales as the reference follows the scores.
//
// The reference rises only when a score passes it by 2^8 (one vote per tile); P of 16-bit caches is the sum of two
// 16-bit parts, so its rounding stays behind the output's.
#include "paged.cuh"

namespace fa {

constexpr int kPagedWarps = 4;
constexpr int kPagedThreads = 32 * kPagedWarps;
constexpr int kGranule = 16 * kPagedWarps;  // keys: one tile for each warp
constexpr float kRise = 8.f;  // how far a score may pass the reference before the reference follows

// Ring depth and blocks per SM of a variant: at least 40 KB in flight per SM (HBM latency times its bandwidth share),
// within 227 KB of shared memory and the registers.
template <int D, bool Q4, int NT>
struct PagedConfig {
  static constexpr int kTileBytes = 16 * (Q4 ? 2 * (D / 2 + D / 8) : 2 * D * 2);  // keys and values of 16 tokens
  static constexpr int kStages = Q4 ? 5 : 3;
  static constexpr int kBlocks = NT == 2 ? (D == 128 ? 2 : 4) : (!Q4 && D == 128 ? 2 : 4);
  static constexpr int kRing = kPagedWarps * kStages * kTileBytes;
  static constexpr int kRows = 8 * NT;
  static constexpr int kPitch = D + 4;  // floats per row of the warps' partial outputs
  static constexpr int kJoin = kPagedWarps * kRows * kPitch * 4;
  static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
};

struct PagedParams {
  const uint8_t* q;
  void* o;
  float* lse;
  float* part_o;   // [2·workers, rows of a tile, d]
  float* part_ml;  // [2·workers, rows of a tile, 2]
  PagedArgs pg;
  int Nq, H, G, most, R, tiles;  // G = H/Hk, most: the largest length allowed, R = G·Nq rows of a key head in `tiles` tiles
  int workers;
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

// The same with a zero sum to start from.
__device__ __forceinline__ void mma_16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Transpose of an 8×8 matrix of 16-bit elements: lane (g, t) gives row g, columns 2t, 2t+1 and gets the same of the transpose.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// The two 4-bit numbers at bits SHIFT and 16 + SHIFT of x as fp16: (n − 8)·2^-24 (SHIFT 0) or (n − 8)·2^-20 (SHIFT 4).
template <int SHIFT>
__device__ __forceinline__ uint32_t less8(uint32_t x) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x & (0x000f000fu << SHIFT)), "r"(0x00080008u << SHIFT));
  return d;
}

// The sequence's key count, or -1 when it is out of range.
__device__ __forceinline__ int paged_length(const PagedParams& p, int b) {
  const int L = __ldg(p.pg.seqlens_k + b);
  return L < 0 || L > p.most ? -1 : L;
}

__device__ __forceinline__ int granules(int L) { return L <= 0 ? 0 : (L + kGranule - 1) / kGranule; }

// Granules of the sequences before sequence `end` (one key head, one row tile).  Every lane gets the sum; a
// warp reads 128 lengths at a time (of at most 2^24 granules each).
__device__ __forceinline__ long long granules_before(const PagedParams& p, int end) {
  const int lane = (int)lane_id();
  long long sum = 0;
  for (int b0 = 0; b0 < end; b0 += 128) {
    unsigned n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = b0 + 32 * i + lane;
      if (b < end) n += granules(paged_length(p, b));
    }
    sum += __reduce_add_sync(0xffffffffu, n);
  }
  return sum;
}

// The sequence that holds granule `at` of the sequences' sum, and the granules before it.
__device__ __forceinline__ int find_granule(const PagedParams& p, long long at, long long& before) {
  const int lane = (int)lane_id();
  long long sum = 0;
  for (int b0 = 0; b0 < p.pg.B; b0 += 32) {
    const int n = b0 + lane < p.pg.B ? granules(paged_length(p, b0 + lane)) : 0;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, sum + incl > at);
    if (past != 0u) {
      const int l = __ffs(past) - 1;
      before = sum + __shfl_sync(0xffffffffu, incl - n, l);
      return b0 + l;
    }
    sum += __shfl_sync(0xffffffffu, incl, 31);
  }
  before = sum;
  return p.pg.B;
}

// Granules that each worker takes.
__device__ __forceinline__ long long granule_share(const PagedParams& p, long long total) {
  return max(1LL, (total + p.workers - 1) / p.workers);
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Shared-memory loads at a 32-bit address plus a constant.
template <int OFF>
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4 + %5];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2 + %3];" : "=r"(v.x), "=r"(v.y) : "r"(a), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1 + %2];" : "=r"(v) : "r"(a), "n"(OFF));
  return v;
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Places of 16-byte pieces in shared memory (c: piece of row r), such that the pieces one shared-memory access reads
// lie in different banks.  16 bits: eight lanes read four pieces of keys r, r + 1, or two pieces of values r, r + 2,
// r + 4, r + 6.  4-bit values: the same rows, two pieces in each half warp (d = 128) or the whole warp (d = 64).
template <int D>
__device__ __forceinline__ int k_piece(int r, int c) { return r * (D / 8) + (c ^ ((r & 1) << 2)); }
template <int D>
__device__ __forceinline__ int v_piece(int r, int c) { return r * (D / 8) + (c ^ (((r >> 1) & 3) << 1)); }
template <int D>
__device__ __forceinline__ int v4_piece(int r, int c) {
  const int i = r * (D / 32) + c;
  return i ^ (D == 128 ? ((r >> 1) & 3) << 1 : ((r >> 2) & 1) << 1);
}

// Copies tiles of a key head into one warp's ring.  All that does not change from tile to tile is kept per lane: where
// its pieces lie in a tile (the swizzles repeat after 32 pieces) and in a block of page 0.
template <int D, bool Q4>
struct TileCopy {
  static constexpr int kRow = Q4 ? D / 2 : D * 2;  // bytes of a row of elements or numbers
  static constexpr int kPer = 16 * kRow / 512;     // 32-piece copies of 16 rows
  static constexpr int kPairs = D / 8;             // 4 bits: pieces of 16 rows of pairs
  const uint8_t *k, *v, *pair;
  uint32_t dk, dv, dpair, page_bytes;
  bool has_pair;

  __device__ __forceinline__ TileCopy(const PagedArgs& pg, int hk, uint32_t ring, int lane) {
    const size_t block = cache_block_bytes(D, pg.page_size, Q4);
    k = static_cast<const uint8_t*>(pg.k_cache) + hk * block + lane * 16;
    v = static_cast<const uint8_t*>(pg.v_cache) + hk * block + lane * 16;
    page_bytes = (uint32_t)(block * pg.Hk);  // below 2^31 (checked on the host)
    const int r = lane / (kRow / 16), c = lane % (kRow / 16);
    if constexpr (Q4) {
      dk = ring + 16 * lane;
      dv = ring + 16 * kRow + 16 * v4_piece<D>(r, c);
      has_pair = lane < 2 * kPairs;
      pair = static_cast<const uint8_t*>(lane < kPairs ? pg.k_cache : pg.v_cache) + hk * block + (size_t)pg.page_size * kRow +
             lane % kPairs * 16;
      dpair = ring + 32 * kRow + 16 * lane;
    } else {
      dk = ring + 16 * k_piece<D>(r, c);
      dv = ring + 16 * kRow + 16 * v_piece<D>(r, c);
    }
  }

  // the 16 tokens from `slot` on of `page`, to the stage `at` bytes into the ring
  __device__ __forceinline__ void copy(int page, int slot, uint32_t at) const {
    const size_t off = (size_t)(uint32_t)page * page_bytes;
    const uint8_t* ks = k + off + slot * kRow;
    const uint8_t* vs = v + off + slot * kRow;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      // 16 bits: two (d = 128) or four rows per copy, so the values' swizzle changes with i
      const uint32_t turn = Q4 ? 0 : D == 128 ? i % 4 * 32 : i % 2 * 64;
      cp_async16(dk + at + 512 * i, ks + 512 * i);
      cp_async16(((dv + at) ^ turn) + 512 * i, vs + 512 * i);
    }
    if constexpr (Q4) {
      if (has_pair) cp_async16(dpair + at, pair + off + slot * (D / 8));
    }
  }
};

template <int D, bool BF16, bool Q4, int NT>
__global__ void __launch_bounds__(kPagedThreads, (PagedConfig<D, Q4, NT>::kBlocks)) fa_paged_split_kernel(const PagedParams p) {
  using Cfg = PagedConfig<D, Q4, NT>;
  constexpr int W = D / 32;           // groups of 32 features
  constexpr int KS = D / 16;          // k-steps of the scores; feature tiles of the output
  constexpr bool MB = BF16 && !Q4;    // operand type of the products
  constexpr int ROWS = 8 * NT, S = Cfg::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kPagedWarps][ROWS], s_l[kPagedWarps][ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  constexpr int ROW = TileCopy<D, Q4>::kRow;  // bytes of a row of elements or numbers
  const uint32_t ring = smem_u32(smem) + warp * S * Cfg::kTileBytes;
  // where this lane reads in a tile: everything else is a constant apart from these.  Keys of rows g (even and odd
  // pieces of 64 bytes: the swizzle swaps them in odd rows), values of row 2t, pairs of row g
  const uint32_t lane_k0 = Q4 ? lane * (D / 8) : 16 * k_piece<D>(g, t), lane_k1 = Q4 ? 0 : 16 * k_piece<D>(g, 4 + t);
  const uint32_t lane_v = 16 * ROW + (!Q4 ? 16 * v_piece<D>(2 * t, g)
                                          : D == 128 ? 16 * v4_piece<D>(2 * t, g >> 1) + 8 * (g & 1) : 16 * v4_piece<D>(2 * t, g >> 2) + 4 * (g & 3));
  const uint32_t lane_p = 32 * ROW + g * (D / 8);
  float* s_o = reinterpret_cast<float*>(smem);
  const int ps = p.pg.page_size;
  const int units = p.pg.Hk * p.tiles;  // of one sequence

  // ---- this block's run of granules
  for (int b = blockIdx.x; b < p.pg.B; b += gridDim.x)
    if (threadIdx.x == 0 && paged_length(p, b) < 0) record_status(1);
  const long long total = granules_before(p, p.pg.B) * units;
  const long long share = granule_share(p, total);
  long long at = blockIdx.x * share;
  const long long end = min(at + share, total);
  if (at >= end) return;
  long long before;
  int b = find_granule(p, at / units, before);
  int L = paged_length(p, b), n = granules(L);
  int unit = (int)((at - before * units) / n), first = (int)((at - before * units) - (long long)unit * n);

#pragma unroll 1
  for (;;) {
    const int last = (int)min((long long)n, first + (end - at));  // granules first .. last − 1 of this unit
    const int hk = unit % p.pg.Hk, r0 = (unit / p.pg.Hk) * ROWS;

    // ---- the warp's tiles: 16 keys from 64·i + 16·warp on; page lookups run one tile ahead of the copies
    const int32_t* table = p.pg.page_table + (size_t)b * p.pg.max_pages;
    const int tiles = last - first - (kGranule * (last - 1) + 16 * warp >= L ? 1 : 0);
    const TileCopy<D, Q4> copy(p.pg, hk, ring, lane);
    int page_i = (kGranule * first + 16 * warp) / ps, slot = (kGranule * first + 16 * warp) - page_i * ps;
    int page = tiles > 0 ? __ldg(table + page_i) : 0;
    int left = tiles;          // to be copied
    uint32_t copy_at = 0;      // the stage of the next one
    uint32_t valid = 0;        // bit i: the i-th last of them is there
    auto issue = [&]() {
      if (left > 0) {
        --left;
        const bool ok = (unsigned)page < (unsigned)p.pg.num_pages;
        valid = valid * 2 + (ok ? 1u : 0u);
        if (ok) copy.copy(page, slot, copy_at);
        else if (lane == 0) record_status(1);
        slot += kGranule;
        while (slot >= ps) {
          slot -= ps;
          ++page_i;
        }
        if (left > 0) page = __ldg(table + page_i);
      } else {
        valid *= 2;
      }
      copy_at = copy_at == (S - 1) * Cfg::kTileBytes ? 0 : copy_at + Cfg::kTileBytes;
      cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue();

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
        // most = m·2^e, 1 <= m < 2; the row goes into the products as q·2^(12 − e), times n·2^-24: s = s'·2^(e + 12)
        const int e = min(max((int)(__float_as_uint(most) >> 23) - 127, -100), 100);
        const float up = __uint_as_float((uint32_t)(127 + 12 - e) << 23);
        const float down = __uint_as_float((uint32_t)(127 - 12 - e) << 23);
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
          s *= down;
          // from the lanes of row g to the lanes that hold rows 2t, 2t+1
          qsum[nt][0][j] = __shfl_sync(0xffffffffu, s, 8 * t);
          qsum[nt][1][j] = __shfl_sync(0xffffffffu, s, 8 * t + 4);
        }
        const float back = __uint_as_float((uint32_t)(127 + 12 + e) << 23) * p.scale_log2;
        coef[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);
        coef[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int rr = r0 + 8 * nt + 2 * t + u;
        lim[nt][u] = L - p.Nq + (rr < p.R ? rr / p.G : p.Nq - 1);
      }
    }

    // m: the reference (base 2), mz: the same with 0 for −inf, rise_at: the dot product from which it has to rise
    float m[NT][2], mz[NT][2], rise_at[NT][2], l[NT][2], o[NT][KS][4], omin[NT][2][Q4 ? W : 1];
    float cap = 0.f, up = 1.f;  // 4 bits: a power of two no value scale of the warp passes, and 2^6 / cap
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        m[nt][u] = rise_at[nt][u] = -INFINITY;
        mz[nt][u] = 0.f;
        l[nt][u] = 0.f;
#pragma unroll
        for (int j = 0; j < (Q4 ? W : 1); ++j) omin[nt][u][j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][j][i] = 0.f;
    }

    uint32_t tile = ring + (S - 1) * Cfg::kTileBytes;
    int j0 = kGranule * (first - 1) + 16 * warp;
#pragma unroll 1
    for (int it = 0; it < tiles; ++it) {
      cp_async_wait<S - 2>();
      __syncwarp();  // the tile is here for every lane, and every lane is done with the one before
      const bool have = (valid >> (S - 2)) & 1u;
      issue();
      tile = tile == ring + (S - 1) * Cfg::kTileBytes ? ring : tile + Cfg::kTileBytes;
      j0 += kGranule;
      if (!have) continue;
      const bool tail = j0 + 16 > L;

      // ---- scores of keys j0 + g and j0 + g + 8
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
      uint32_t vp[Q4 ? 2 : 1][Q4 ? W : 1];  // (scale, min) of the values of keys g, g + 8
      float most = 0.f;                     // the largest of these scales
      if constexpr (!Q4) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const uint32_t a = tile + (j & 1 ? lane_k1 : lane_k0) + j / 2 * 128;
          const uint4 x = lds128<0>(a), y = lds128<8 * ROW>(a);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16816<MB>(s[nt], x.x, y.x, x.y, y.y, qb[nt][2 * j][0], qb[nt][2 * j][1]);
            mma_16816<MB>(s[nt], x.z, y.z, x.w, y.w, qb[nt][2 * j + 1][0], qb[nt][2 * j + 1][1]);
          }
        }
      } else {
        uint32_t kn[2][W], kp[2][W];
        const uint32_t ak = tile + lane_k0, ap = tile + lane_p;
        if constexpr (W == 4) {
          const uint4 x0 = lds128<0>(ak), x1 = lds128<8 * ROW>(ak), y0 = lds128<0>(ap), y1 = lds128<8 * 16>(ap);
          const uint4 z0 = lds128<16 * 16>(ap), z1 = lds128<24 * 16>(ap);
          kn[0][0] = x0.x; kn[0][1] = x0.y; kn[0][2] = x0.z; kn[0][3] = x0.w;
          kn[1][0] = x1.x; kn[1][1] = x1.y; kn[1][2] = x1.z; kn[1][3] = x1.w;
          kp[0][0] = y0.x; kp[0][1] = y0.y; kp[0][2] = y0.z; kp[0][3] = y0.w;
          kp[1][0] = y1.x; kp[1][1] = y1.y; kp[1][2] = y1.z; kp[1][3] = y1.w;
          vp[0][0] = z0.x; vp[0][1] = z0.y; vp[0][2] = z0.z; vp[0][3] = z0.w;
          vp[1][0] = z1.x; vp[1][1] = z1.y; vp[1][2] = z1.z; vp[1][3] = z1.w;
        } else {
          const uint2 x0 = lds64<0>(ak), x1 = lds64<8 * ROW>(ak), y0 = lds64<0>(ap), y1 = lds64<8 * 8>(ap);
          const uint2 z0 = lds64<16 * 8>(ap), z1 = lds64<24 * 8>(ap);
          kn[0][0] = x0.x; kn[0][1] = x0.y; kn[1][0] = x1.x; kn[1][1] = x1.y;
          kp[0][0] = y0.x; kp[0][1] = y0.y; kp[1][0] = y1.x; kp[1][1] = y1.y;
          vp[0][0] = z0.x; vp[0][1] = z0.y; vp[1][0] = z1.x; vp[1][1] = z1.y;
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const uint32_t x0 = kn[0][j], x1 = kn[1][j], y0 = x0 >> 8, y1 = x1 >> 8;
          const float2 p0 = __half22float2(*reinterpret_cast<const __half2*>(&kp[0][j]));
          const float2 p1 = __half22float2(*reinterpret_cast<const __half2*>(&kp[1][j]));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float acc[4];
            mma_16816_first(acc, x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, qb[nt][2 * j][0],
                             qb[nt][2 * j][1]);
            mma_16816<false>(acc, y0 & 0x000f000fu, y1 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x00f000f0u, qb[nt][2 * j + 1][0],
                             qb[nt][2 * j + 1][1]);
            s[nt][0] = fmaf(p0.x, acc[0], fmaf(p0.y, qsum[nt][0][j], s[nt][0]));
            s[nt][1] = fmaf(p0.x, acc[1], fmaf(p0.y, qsum[nt][1][j], s[nt][1]));
            s[nt][2] = fmaf(p1.x, acc[2], fmaf(p1.y, qsum[nt][0][j], s[nt][2]));
            s[nt][3] = fmaf(p1.x, acc[3], fmaf(p1.y, qsum[nt][1][j], s[nt][3]));
          }
        }
        if (tail) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < W; ++j)
              if (j0 + g + 8 * u >= L) vp[u][j] = 0u;
        }
        __half2 top = *reinterpret_cast<const __half2*>(&vp[0][0]);
#pragma unroll
        for (int j = 1; j < 2 * W; ++j) top = __hmax2(top, *reinterpret_cast<const __half2*>(&vp[j / W][j % W]));
        most = __low2float(top);
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
      // ---- the reference (NaN does not raise it: it reaches the sums all the same)
      bool rise = Q4 && most > cap;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        rise = rise || fmaxf(s[nt][0], s[nt][2]) > rise_at[nt][0] || fmaxf(s[nt][1], s[nt][3]) > rise_at[nt][1];
      if (__any_sync(0xffffffffu, rise)) {
        float grow = 1.f;
        if constexpr (Q4) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
          if (most > cap) {
            const uint32_t e = min((__float_as_uint(most) >> 23) + 1u, 160u);  // 2^(e − 127) is above it
            const float next = __uint_as_float(e << 23);
            grow = cap * __uint_as_float((254u - e) << 23);
            cap = next;
            up = 64.f * __uint_as_float((254u - e) << 23);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float x = fmaxf(s[nt][u], s[nt][2 + u]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float mn = fmaxf(m[nt][u], x * coef[nt][u]);
            const float alpha = m[nt][u] == -INFINITY ? 0.f : ex2(m[nt][u] - mn);
            m[nt][u] = mn;
            mz[nt][u] = mn == -INFINITY ? 0.f : mn;
            rise_at[nt][u] = (mn + kRise) / coef[nt][u];
            l[nt][u] *= alpha;
            const float ao = Q4 ? alpha * grow : alpha;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              o[nt][j][u] *= ao;
              o[nt][j][2 + u] *= ao;
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
#pragma unroll
        for (int i = 0; i < 4; ++i) pr[nt][i] = ex2(fmaf(s[nt][i], coef[nt][i & 1], -mz[nt][i & 1]));
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
            bh[nt][u] = movmatrix_trans(hi);
            bl[nt][u] = movmatrix_trans(pack2<MB>(pr[nt][2 * u] - back.x, pr[nt][2 * u + 1] - back.y));
          }
        const bool apart = p.Nq > 1 && j0 + 15 > L - p.Nq;
#pragma unroll
        for (int cc = 0; cc < D / 64; ++cc) {
          uint32_t v[4][4];
          const uint32_t av = tile + lane_v + 128 * cc;
          const uint4 rows[4] = {lds128<0>(av), lds128<ROW>(av), lds128<8 * ROW>(av), lds128<9 * ROW>(av)};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i][0] = rows[i].x; v[i][1] = rows[i].y; v[i][2] = rows[i].z; v[i][3] = rows[i].w;
          }
          if (tail) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int u = 0; u < 4; ++u)
                if (j0 + key[i] >= L) v[i][u] = 0u;
          }
          if (!apart) {
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
            for (int end_key = max(j0, L - p.Nq); end_key < min(j0 + 16, L); ++end_key) {
              const bool top = end_key == j0 + 15;  // rows that see all of this tile, and more
              uint32_t x[4][4];
#pragma unroll
              for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[u][i] = j0 + key[u] <= end_key ? v[u][i] : 0u;
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
                    if (lim[nt][u & 1] == end_key || (top && lim[nt][u & 1] > end_key)) o[nt][4 * cc + i][u] += tmp[u];
                }
              }
            }
          }
        }
      } else {
        uint32_t v[4][W / 2];
        const uint32_t av = tile + lane_v, odd = tile + (lane_v ^ ROW);  // row 2t + 1: the swizzle turns the row's bit too
        if constexpr (W == 4) {
          const uint2 rows[4] = {lds64<0>(av), lds64<0>(odd), lds64<8 * ROW>(av), lds64<8 * ROW>(odd)};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i][0] = rows[i].x;
            v[i][1] = rows[i].y;
          }
        } else {
          v[0][0] = lds32<0>(av);
          v[1][0] = lds32<0>(odd);
          v[2][0] = lds32<8 * ROW>(av);
          v[3][0] = lds32<8 * ROW>(odd);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
          const uint32_t e = prmt(v[0][j >> 1], v[1][j >> 1], sel), f = prmt(v[2][j >> 1], v[3][j >> 1], sel);
          const uint32_t a0 = less8<0>(e), a1 = less8<4>(e), a2 = less8<0>(f), a3 = less8<4>(f);
          const uint32_t d0 = less8<0>(e >> 8), d1 = less8<4>(e >> 8), d2 = less8<0>(f >> 8), d3 = less8<4>(f >> 8);
          const float2 p0 = __half22float2(*reinterpret_cast<const __half2*>(&vp[0][j]));
          const float2 p1 = __half22float2(*reinterpret_cast<const __half2*>(&vp[1][j]));
          const float s0 = p0.x * up, s1 = p1.x * up, n0 = fmaf(8.f, p0.x, p0.y), n1 = fmaf(8.f, p1.x, p1.y);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t b0 = movmatrix_trans(pack2<false>(pr[nt][0] * s0, pr[nt][1] * s0));
            const uint32_t b1 = movmatrix_trans(pack2<false>(pr[nt][2] * s1, pr[nt][3] * s1));
            mma_16816<false>(o[nt][2 * j], a0, a1, a2, a3, b0, b1);
            mma_16816<false>(o[nt][2 * j + 1], d0, d1, d2, d3, b0, b1);
            omin[nt][0][j] = fmaf(pr[nt][0], n0, fmaf(pr[nt][2], n1, omin[nt][0][j]));
            omin[nt][1][j] = fmaf(pr[nt][1], n0, fmaf(pr[nt][3], n1, omin[nt][1][j]));
          }
        }
      }
    }
    cp_async_wait<0>();
    __syncthreads();  // every warp is done with its ring: the memory now holds the warps' partial outputs
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = 8 * nt + 2 * t + u;
        float* row = s_o + (warp * ROWS + r) * Cfg::kPitch;
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
              row[64 * cc + 8 * g + 2 * i] = o[nt][4 * cc + i][u];
              row[64 * cc + 8 * g + 2 * i + 1] = o[nt][4 * cc + i][2 + u];
            }
        } else {
#pragma unroll
          for (int j = 0; j < W; ++j) {
            float y = omin[nt][u][j];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
            float* dst = row + 32 * j + 4 * g;
            const float even = cap * 262144.f, odd = cap * 16384.f;  // 2^24 and 2^20, over the 2^6 / cap of the products
            dst[0] = fmaf(o[nt][2 * j][u], even, y);
            dst[1] = fmaf(o[nt][2 * j][2 + u], odd, y);
            dst[2] = fmaf(o[nt][2 * j + 1][u], even, y);
            dst[3] = fmaf(o[nt][2 * j + 1][2 + u], odd, y);
          }
        }
      }
    __syncthreads();
    // ---- the block's: a warp per row, d/32 features per lane
    const bool whole = first == 0 && last == n;
    const int part = 2 * blockIdx.x + (first == 0 ? 1 : 0);
#pragma unroll 1
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
        for (int j = 0; j < W; ++j) acc[j] = fmaf(s_o[(w * ROWS + r) * Cfg::kPitch + 32 * j + lane], a, acc[j]);
      }
      if (whole) {
        const size_t row = paged_row(p, b, hk, r0 + r);
        const float inv = ell == 0.f ? 0.f : 1.f / ell;
#pragma unroll
        for (int j = 0; j < W; ++j) store_out<D, BF16>(p.o, row * D + 32 * j + lane, acc[j] * inv);
        if (lane == 0) p.lse[row] = ell == 0.f ? -INFINITY : (M + log2f(ell)) * 0.69314718055994531f;
      } else {
        const size_t row = (size_t)part * ROWS + r;
#pragma unroll
        for (int j = 0; j < W; ++j) p.part_o[row * D + 32 * j + lane] = acc[j];
        if (lane == 0) {
          p.part_ml[2 * row] = M;
          p.part_ml[2 * row + 1] = ell;
        }
      }
    }
    // ---- the next unit
    at += last - first;
    if (at >= end) break;
    __syncthreads();  // the partial outputs are read: the memory is the ring's again
    first = 0;
    if (++unit == units) {
      unit = 0;
      do {
        ++b;
        L = paged_length(p, b);
      } while (L <= 0);
      n = granules(L);
    }
  }
}

// One block per row of q.  A unit that lay in one run is already written; its row has nothing to join.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) fa_paged_merge_kernel(const PagedParams p, int tile_rows) {
  constexpr int F = D / 32;
  __shared__ float s_o[4][D], s_l[4];
  const size_t row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = (int)(row % p.H), i = (int)(row / p.H % p.Nq), b = (int)(row / p.H / p.Nq);
  const int r = i * p.G + head % p.G, units = p.pg.Hk * p.tiles;
  const int L = paged_length(p, b), n = granules(L);
  const long long total = granules_before(p, p.pg.B) * units, share = granule_share(p, total);
  const long long from = granules_before(p, b) * units + (long long)(r / tile_rows * p.pg.Hk + head / p.G) * n;
  const int w0 = (int)(from / share), w1 = n > 0 ? (int)((from + n - 1) / share) : w0 - 1;  // the blocks that hold a part
  asm volatile("griddepcontrol.wait;" ::: "memory");  // every block waits, so that this kernel ends after the other
  if (w0 == w1 || L < 0) return;
  // the first block's part is its last one (slot 1), the others' their first (slot 0)
  const int at = r % tile_rows;
  auto slot = [&](int w) { return (size_t)(2 * w + (w == w0 ? 1 : 0)) * tile_rows + at; };
  float M = -INFINITY;
  for (int w = w0 + lane; w <= w1; w += 32) M = fmaxf(M, p.part_ml[2 * slot(w)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float ell = 0.f, acc[F];
#pragma unroll
  for (int j = 0; j < F; ++j) acc[j] = 0.f;
#pragma unroll 4
  for (int w = w0 + warp; w <= w1; w += 4) {
    const size_t s = slot(w);
    const float a = join_weight(p.part_ml[2 * s], M);
    ell = fmaf(p.part_ml[2 * s + 1], a, ell);
    const float* src = p.part_o + s * D;
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

// Row tiles of a key head, and the rows of one.
static int paged_tile_rows(int R) { return R <= 8 ? 8 : 16; }

// Blocks that can take a run: all that fit the GPU at once (at most four per SM), or one per granule of the longest batch.
static int paged_workers(int B, int Hk, int tiles, int Nk, int per_sm) {
  const long long most = (long long)B * Hk * tiles * ((Nk + kGranule - 1) / kGranule);
  return (int)std::min<long long>(most, (long long)kSmCount * per_sm);
}

void paged_workspace(int B, int Nq, int H, int Hk, int Nk, int d, size_t* o_bytes, size_t* ml_bytes) {
  const int R = H / Hk * Nq, rows = paged_tile_rows(R), tiles = (R + rows - 1) / rows;
  const size_t slots = (size_t)2 * paged_workers(B, Hk, tiles, Nk, 4) * rows;
  *o_bytes = slots * d * sizeof(float);
  *ml_bytes = slots * 2 * sizeof(float);
}

template <int D, bool BF16, bool Q4, int NT>
static cudaError_t launch_paged_v(PagedParams p, int B, int Nk, cudaStream_t stream) {
  using Cfg = PagedConfig<D, Q4, NT>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = set_smem_once(done, reinterpret_cast<const void*>(fa_paged_split_kernel<D, BF16, Q4, NT>), Cfg::kSmem);
  if (e != cudaSuccess) return e;
  p.workers = paged_workers(B, p.pg.Hk, p.tiles, Nk, Cfg::kBlocks);
  fa_paged_split_kernel<D, BF16, Q4, NT><<<p.workers, kPagedThreads, Cfg::kSmem, stream>>>(p);
  e = cudaPeekAtLastError();
  if (e != cudaSuccess) return e;
  // the merge may start its index arithmetic while the last runs end; it waits for them before it reads a part
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((size_t)B * p.Nq * p.H));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_paged_merge_kernel<D, BF16>, p, 8 * NT);
}

template <int D, bool BF16>
static cudaError_t launch_paged_t(const PagedParams& p, int B, int Nk, cudaStream_t stream) {
  if (p.pg.q4)
    return p.R <= 8 ? launch_paged_v<D, BF16, true, 1>(p, B, Nk, stream) : launch_paged_v<D, BF16, true, 2>(p, B, Nk, stream);
  return p.R <= 8 ? launch_paged_v<D, BF16, false, 1>(p, B, Nk, stream) : launch_paged_v<D, BF16, false, 2>(p, B, Nk, stream);
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
  p.tiles = (p.R + paged_tile_rows(p.R) - 1) / paged_tile_rows(p.R);
  p.workers = 0;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  if (pg.d == 128) return pg.bf16 ? launch_paged_t<128, true>(p, pg.B, a.Nk, stream) : launch_paged_t<128, false>(p, pg.B, a.Nk, stream);
  return pg.bf16 ? launch_paged_t<64, true>(p, pg.B, a.Nk, stream) : launch_paged_t<64, false>(p, pg.B, a.Nk, stream);
}

}  // namespace fa
