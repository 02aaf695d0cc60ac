// fa_paged.cu — attention of a few new queries per sequence over a paged key/value cache, 16-bit or 4-bit.
//
//   fa_paged_split_kernel  one wave of blocks; the keys of all (sequence, key head, tile of query rows) units,
//                          in granules of four warps' tiles, are dealt out evenly: each block takes a run of
//                          granules, which may end inside a unit and may span several.  A unit that lies in one
//                          run is finished there; of others each block leaves its partial (m, ℓ, Õ = Σ_j 2^(s_j − m) v_j),
//                          s = scale·log2(e)·q·k (base 2)
//   fa_paged_merge_kernel  joins the parts of a row: m = max m_c, ℓ = Σ ℓ_c·2^(m_c − m), Õ the same way
//   fa_paged_cluster_kernel  small calls: a cluster of blocks per unit, joined through distributed shared memory, so that
//                          one launch does the call
//
// The query rows of a key head are its H/Hk query heads times the Nq new tokens; 8 or 16 of them share one
// pass over the keys, so a key is read once for the whole group.  The call is a stream over the cache, and
// the products run on the tensor cores only so that 8 or 16 rows cost no more instructions than one.  The
// tile is small (16 keys by 8 rows), which the warp-level matrix instructions fit; tcgen05 would want 128
// rows of keys in shared memory in its own layout, and the 4-bit numbers would have to be written there
// after unpacking.
//
// Each warp streams its own tiles (16 keys, or 32 of 4 bits) through a ring in shared memory with asynchronous
// 16-byte copies; the ring's depth covers the latency of HBM, and no warp waits for another until the end of
// a unit.
//
// Orders are chosen so that no operand moves between lanes.  With g = lane/4, t = lane%4:
//   scores   Sᵀ[16 keys × 8 rows] = K·qᵀ.  A lane reads whole 16-byte pieces of keys g and g + 8 and takes the
//            features in the order they lie; the query operand is loaded in the same order.
//   output   Oᵀ[16 features × 8 rows] += Vᵀ·Pᵀ.  A lane reads pieces of keys 2t, 2t+1, 2t+8, 2t+9 and pairs
//            neighbouring keys with byte permutes; P is transposed in registers (movmatrix).
// A lane's scores and outputs belong to the same two rows (2t, 2t+1), so rescaling needs no exchange either.
// The pieces are written to shared memory at places that keep these reads free of bank conflicts.
//
// Measured, d = 128: 16 x 8192 keys of 16 heads in 16 bits 1074 MB in 165 to 169 us (97 to 99 % of the measured copy
// bandwidth); 64 sequences of 512 to 16384 keys, 8 key heads, 4 query heads each, in 4 bits 744 MB in 167 us (68 %); 131071
// keys of 8 heads, 16 query rows, fp16, in 4 bits 168 MB in 72 us (35 %); one sequence of 777 keys and 16 heads 6.2 us (the
// launch and a chain of lookups and copies).  Over 16 rows a key head, each tile of 16 reads the keys again, from HBM where
// they do not fit L2: 1074 MB of 16-bit keys and values with 16, 32 and 60 rows 1.08, 2.15 and 4.28 GB, 181, 343 and 659 us.
//
// The reference of the exponents rises only when a score passes it by 2^8 (one vote per tile).  P of 16-bit caches is
// the sum of two 16-bit parts, so its rounding stays behind the output's; in fp16 the reference is 2^7 below the maximum,
// so that P, up to 2^15, keeps keys down to 2^-32 of the largest (many of them may outweigh it).
//
// 4 bits.  Instructions bound this path (16 keys by 8 rows of d = 128 have 2,560 bytes to read and 4,096 numbers to unpack;
// 362 instructions per warp, 52 % of the issue slots with three warps per scheduler, the integer pipe 46 % busy, HBM 68 %),
// so everything is arranged to keep their number low; the first arrangement, the plain formula, took 603:
//   * Numbers are used where they lie: a masked half word with n in bits 0-3 is the fp16 n·2^-24, with n in bits 4-7
//     n·2^-20 (subnormal, and exact in the products).  The queries are taken to fp16 by a power of two per row that
//     brings the largest to 2^12 (exact but for features 2^-26 below it), those that meet the 2^-20 form by 2^-4 less.
//   * Each group of 32 features has its own fp32 accumulator, which the key's scale multiplies; the minima times the
//     sums of q over the groups are one small product (the sums as two fp16 parts).
//   * P is rounded to fp16 and transposed once; for each group it is then multiplied by the values' scales of its keys.
//     That rounds a second time, which bf16 outputs do not show; for fp16 outputs what the second rounding takes away is
//     a product of its own (both roundings together left 1.8 times the output's own error, one leaves 1.4).
//   * Σ_j p_j·min_j and Σ_j p_j·scale_j are one small product more.  It takes the same rounded P, so what rounding
//     leaves is relative to the value, n·scale + min, and not to the larger min.
//   * The values enter as n − 8.  Without the shift the products would add up to a mean of 2 standard deviations per
//     key that the minimum takes away again: over 131071 keys the tensor cores' truncating sums left 8e-4 of the
//     output.  For one row tile −8·ΣP is a product of its own (no instruction per number); two row tiles share a
//     subtraction per number, and so do fp16 outputs.
//   * A key's minima and scales are divided by the power of two 2^e over the largest of them and its probability is multiplied
//     by it, and the reference is 2^7 under the largest p·2^e: fp16's range counts from the key whose values weigh most.  With
//     the reference under the largest p alone, small values beside a key that outweighs them lost their products with the
//     scale, and large values of no weight pushed the others out of the range (7 % of the output over 2048 keys).  Costs 30
//     instructions per tile: 64 sequences 161 -> 167 us, 131071 keys 71.8 -> 72.6.
#include <cooperative_groups.h>

#include <type_traits>

#include "paged.cuh"

namespace fa {

constexpr int kPagedWarps = 4;
constexpr int kPagedThreads = 32 * kPagedWarps;
constexpr float kRise = 8.f;  // how far a score may pass the reference before the reference follows

// Blocks per SM of a variant.
constexpr int paged_blocks(int d, bool q4, int nt) { return d == 64 ? (nt == 2 ? 3 : 4) : nt == 2 || !q4 ? 2 : 3; }

// Tile and ring depth of a variant: what all warps have in flight per SM is 96 to 128 KB in 16 bits and 40 to 60 KB in 4 bits
// (30 KB at d = 64 with two row tiles), against some 40 KB for HBM's latency times an SM's share of the bandwidth; within 227 KB
// of shared memory and the registers.
template <int D, bool Q4, int NT>
struct PagedConfig {
  static constexpr int kTile = Q4 ? 32 : 16;             // keys of a warp's tile
  static constexpr int kGranule = kTile * kPagedWarps;   // keys of all warps' tiles
  static constexpr int kTileBytes = kTile * (Q4 ? 2 * (D / 2 + D / 8) : 2 * D * 2);
  static constexpr int kStages = Q4 ? 2 : 3;
  static constexpr int kBlocks = paged_blocks(D, Q4, NT);
  static constexpr int kRing = kPagedWarps * kStages * kTileBytes;
  static constexpr int kRows = 8 * NT;
  static constexpr int kPitch = D + 4;  // floats per row of the warps' partial outputs
  static constexpr int kJoin = kPagedWarps * kRows * kPitch * 4;
  static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
};
constexpr int granule_keys(bool q4) { return q4 ? PagedConfig<64, true, 1>::kGranule : PagedConfig<64, false, 1>::kGranule; }

struct PagedParams {
  const uint8_t* q;
  void* o;
  float* lse;
  float* part_o;   // [2·workers, rows of a tile, d]
  float* part_ml;  // [2·workers, rows of a tile, 2]
  PagedArgs pg;
  int Nq, H, G, most, R, tiles;  // G = H/Hk, most: the largest length allowed, R = G·Nq rows of a key head in `tiles` tiles
  int workers, granule;
  bool by_unit;
  int4* units;  // what the merge joins, for each unit (by_unit) or for each worker: sequence, unit of it, the worker that
                // holds the first part, parts (0: nothing to join)
  float scale_log2;
};

template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with a zero sum to start from.
__device__ __forceinline__ void mma_16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 16 × 8 × 8 with a zero sum to start from.
__device__ __forceinline__ void mma_1688_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3]) : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}

// Transpose of an 8×8 matrix of 16-bit elements: lane (g, t) gives row g, columns 2t, 2t+1 and gets the same of the transpose.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
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
  const int L = load_now(p.pg.seqlens_k + b);
  return L < 0 || L > p.most ? -1 : L;
}

__device__ __forceinline__ int granules(const PagedParams& p, int L) { return L <= 0 ? 0 : (L + p.granule - 1) / p.granule; }

// 64-bit quotient; most are of 32-bit numbers, which are several times faster to divide.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (long long)((unsigned)a / (unsigned)b);
  return a / b;
}

// Sum over the block of the granules of all sequences (one key head, one row tile), and this thread's part of it: the
// sequences from `begin` on, `before` granules in front of them.
struct GranuleScan {
  long long total, before, mine;
  int begin, count;
};
__device__ __forceinline__ GranuleScan scan_granules(const PagedParams& p) {
  __shared__ long long s_sum[kPagedWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  GranuleScan s;
  const int per = (p.pg.B + kPagedThreads - 1) / kPagedThreads;
  s.begin = min((int)threadIdx.x * per, p.pg.B);
  s.count = min(per, p.pg.B - s.begin);
  s.mine = 0;
#pragma unroll 4
  for (int i = 0; i < s.count; ++i) s.mine += granules(p, paged_length(p, s.begin + i));
  long long incl = s.mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += x;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  long long base = 0;
  s.total = 0;
#pragma unroll
  for (int w = 0; w < kPagedWarps; ++w) {
    if (w < warp) base += s_sum[w];
    s.total += s_sum[w];
  }
  s.before = base + incl - s.mine;
  return s;
}

// Granules that each worker takes.
__device__ __forceinline__ long long granule_share(const PagedParams& p, long long total) {
  return max(1LL, quotient(total + p.workers - 1, p.workers));
}

// What rounding took from the products: a·b − ab, exact.
__device__ __forceinline__ uint32_t rest_f16x2(uint32_t a, uint32_t b, uint32_t ab) {
  uint32_t d;
  asm("{\n\t.reg .b32 t;\n\tneg.f16x2 t, %3;\n\tfma.rn.f16x2 %0, %1, %2, t;\n\t}" : "=r"(d) : "r"(a), "r"(b), "r"(ab));
  return d;
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
template <int OFF>
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint32_t v;
  asm volatile("{\n\t.reg .b16 h;\n\tld.shared.b16 h, [%1 + %2];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(v) : "r"(a), "n"(OFF));
  return v;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ void fma_pair(float& x, float& y, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\tfma.rn.f32x2 c, a, b, c;\n\t"
      "mov.b64 {%0, %1}, c;\n\t}" : "=f"(x), "=f"(y) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void sub_pair(float& x, float& y, float a0, float a1, float b0, float b1) {
  fma_pair(x, y, b0, b1, -1.f, -1.f, a0, a1);
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
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
// its pieces lie in a tile (the swizzles repeat after a copy of 32 pieces) and in a block of page 0.
// A 16-bit tile is 16 rows of keys, 16 of values; a 4-bit one 32 rows of the keys' numbers, of the values' numbers, of
// the keys' pairs, of the values' pairs.
template <int D, bool Q4>
struct TileCopy {
  static constexpr int kRow = Q4 ? D / 2 : D * 2;  // bytes of a row of elements or numbers
  static constexpr int kPair = D / 8;              // bytes of a row of pairs
  static constexpr int kT = Q4 ? 32 : 16;
  static constexpr int kPer = 16 * kRow / 512;     // copies of 16 rows
  const uint8_t *k, *v, *pair, *half_pair;
  uint32_t dk, dv, dpair, dhalf, page_bytes;
  uintptr_t to_v;  // from the keys' address to the values'
  int lane;

  __device__ __forceinline__ TileCopy(const PagedArgs& pg, int hk, uint32_t ring, int lane_) : lane(lane_) {
    const size_t block = cache_block_bytes(D, pg.page_size, Q4);
    const uint8_t* kb = static_cast<const uint8_t*>(pg.k_cache) + hk * block;
    const uint8_t* vb = static_cast<const uint8_t*>(pg.v_cache) + hk * block;
    k = kb + lane * 16;
    v = vb + lane * 16;
    to_v = reinterpret_cast<uintptr_t>(vb) - reinterpret_cast<uintptr_t>(kb);
    page_bytes = (uint32_t)(block * pg.Hk);  // below 2^31 (checked on the host)
    const int r = lane / (kRow / 16), c = lane % (kRow / 16);
    if constexpr (Q4) {
      dk = ring + 16 * lane;
      dv = ring + kT * kRow + 16 * v4_piece<D>(r, c);
      // pairs of 32 rows: d = 128 has 32 pieces of the keys' and of the values', d = 64 16 each, side by side
      const size_t rows = (size_t)pg.page_size * kRow;
      pair = D == 128 ? kb + rows + lane * 16 : (lane < 16 ? kb : vb) + rows + lane % 16 * 16;
      dpair = ring + 2 * kT * kRow + 16 * lane;
      // of 16 rows: half as many
      const int n = kPair, u = lane % n;
      half_pair = (lane < n ? kb : vb) + rows + u * 16;
      dhalf = ring + 2 * kT * kRow + (lane < n ? 0 : kT * kPair) + 16 * u;
    } else {
      dk = ring + 16 * k_piece<D>(r, c);
      dv = ring + kT * kRow + 16 * v_piece<D>(r, c);
    }
  }

  // N·16 tokens from `slot` on of `page`, to rows 16·half … of the stage `at` bytes into the ring
  template <int N>
  __device__ __forceinline__ void rows(int page, int slot, uint32_t at, int half) const {
    const size_t off = (size_t)(uint32_t)page * page_bytes;
    const uint8_t* ks = k + off + slot * kRow;
    const uint8_t* vs = v + off + slot * kRow;
    at += half * 16 * kRow;
#pragma unroll
    for (int i = 0; i < N * kPer; ++i) {
      // 16 bits: two (d = 128) or four rows per copy, so the values' swizzle changes with i
      const uint32_t turn = Q4 ? 0 : D == 128 ? i % 4 * 32 : i % 2 * 64;
      cp_async16(dk + at + 512 * i, ks + 512 * i);
      cp_async16(((dv + at) ^ turn) + 512 * i, vs + 512 * i);
    }
    if constexpr (Q4) {
      at -= half * 16 * kRow;
      if constexpr (N == 2) {
        const uint8_t* src = pair + off + slot * kPair;
        cp_async16(dpair + at, src);
        if constexpr (D == 128) cp_async16(dpair + at + kT * kPair, reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(src) + to_v));
      } else {
        if (lane < 2 * kPair) cp_async16(dhalf + at + half * 16 * kPair, half_pair + off + slot * kPair);
      }
    }
  }
};

// What a warp holds of its query rows, and one tile's work, for a 16-bit cache.
template <int D, bool BF16, int NT>
struct Rows16 {
  static constexpr int W = D / 32, KS = D / 16, ROW = D * 2;
  static constexpr float kDepth = BF16 ? 0.f : 7.f;  // how far the reference is under the maximum
  uint32_t qb[NT][KS][2];
  float m[NT][2], mz[NT][2], rise_at[NT][2];  // the reference, with 0 for −inf, and the dot product from which it has to rise
  float l[NT][2], o[NT][KS][4];
  int lim[NT][2];  // the last key each of this lane's rows (2t, 2t+1) sees
  uint32_t lane_k0, lane_k1, lane_v;
  float coef;
  int g, t, L, Nq;

  __device__ __forceinline__ void init(const PagedParams& p, int b, int hk, int r0, int len, int lane) {
    g = lane >> 2;
    t = lane & 3;
    L = len;
    Nq = p.Nq;
    coef = p.scale_log2;
    // where this lane reads in a tile, but for constants: keys of row g (even and odd 64-byte pieces, which the swizzle
    // swaps in odd rows), values of row 2t
    lane_k0 = 16 * k_piece<D>(g, t);
    lane_k1 = 16 * k_piece<D>(g, 4 + t);
    lane_v = 16 * ROW + 16 * v_piece<D>(2 * t, g);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + 8 * nt + g;
      const bool on = r < p.R;
      const uint8_t* src = p.q + (on ? paged_row(p, b, hk, r) : 0) * D * 2;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint4 v = on ? load_now(reinterpret_cast<const uint4*>(src + (32 * j + 8 * t) * 2)) : make_uint4(0, 0, 0, 0);
        qb[nt][2 * j][0] = v.x;
        qb[nt][2 * j][1] = v.y;
        qb[nt][2 * j + 1][0] = v.z;
        qb[nt][2 * j + 1][1] = v.w;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int rr = r0 + 8 * nt + 2 * t + u;
        lim[nt][u] = L - Nq + (rr < p.R ? rr / p.G : Nq - 1);
        m[nt][u] = rise_at[nt][u] = -INFINITY;
        mz[nt][u] = l[nt][u] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][j][i] = 0.f;
    }
  }

  __device__ __forceinline__ void step(uint32_t tile, int j0, uint32_t) {
    const bool tail = j0 + 16 > L;
    // ---- scores of keys j0 + g and j0 + g + 8
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const uint32_t a = tile + (j & 1 ? lane_k1 : lane_k0) + j / 2 * 128;
      const uint4 x = lds128<0>(a), y = lds128<8 * ROW>(a);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_16816<BF16>(s[nt], x.x, y.x, x.y, y.y, qb[nt][2 * j][0], qb[nt][2 * j][1]);
        mma_16816<BF16>(s[nt], x.z, y.z, x.w, y.w, qb[nt][2 * j + 1][0], qb[nt][2 * j + 1][1]);
      }
    }
    // ---- keys behind a row's last one; rows behind the sequence's end hold anything, so they are replaced, not scaled
    if (j0 + 15 > L - Nq) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j0 + g + 8 * (i >> 1) > lim[nt][i & 1]) s[nt][i] = -INFINITY;
    }
    // ---- the reference (NaN does not raise it: it reaches the sums all the same)
    bool rise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      rise |= (fmaxf(s[nt][0], s[nt][2]) > rise_at[nt][0]) | (fmaxf(s[nt][1], s[nt][3]) > rise_at[nt][1]);
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float x = fmaxf(s[nt][u], s[nt][2 + u]);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
          const float mn = fmaxf(m[nt][u], fmaf(x, coef, -kDepth));
          const float alpha = m[nt][u] == -INFINITY ? 0.f : ex2(m[nt][u] - mn);
          m[nt][u] = mn;
          mz[nt][u] = mn == -INFINITY ? 0.f : mn;
          rise_at[nt][u] = (mn + (kDepth + kRise)) / coef;
          l[nt][u] *= alpha;
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            o[nt][j][u] *= alpha;
            o[nt][j][2 + u] *= alpha;
          }
        }
    }
    // ---- probabilities, in two parts, transposed
    uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float pr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) pr[i] = ex2(fmaf(s[nt][i], coef, -mz[nt][i & 1]));
      l[nt][0] += pr[0] + pr[2];
      l[nt][1] += pr[1] + pr[3];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t hi = pack2<BF16>(pr[2 * u], pr[2 * u + 1]);
        const float2 back = unpack2<BF16>(hi);
        bh[nt][u] = movmatrix_trans(hi);
        bl[nt][u] = movmatrix_trans(pack2<BF16>(pr[2 * u] - back.x, pr[2 * u + 1] - back.y));
      }
    }
    // ---- output
    const int key[4] = {2 * t, 2 * t + 1, 2 * t + 8, 2 * t + 9};
    const bool apart = Nq > 1 && j0 + 15 > L - Nq;
#pragma unroll
    for (int cc = 0; cc < D / 64; ++cc) {
      uint32_t v[4][4];
      const uint32_t av = tile + lane_v + 128 * cc;
      const uint4 rows[4] = {lds128<0>(av), lds128<ROW>(av), lds128<8 * ROW>(av), lds128<9 * ROW>(av)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i][0] = rows[i].x;
        v[i][1] = rows[i].y;
        v[i][2] = rows[i].z;
        v[i][3] = rows[i].w;
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
            mma_16816<BF16>(o[nt][4 * cc + i], a0, a1, a2, a3, bh[nt][0], bh[nt][1]);
            mma_16816<BF16>(o[nt][4 * cc + i], a0, a1, a2, a3, bl[nt][0], bl[nt][1]);
          }
        }
      } else {
        // the last keys, which the new tokens see one after another: a token at a time with the values behind it
        // taken out, since an infinity or NaN there would pass a zero probability
#pragma unroll 1
        for (int end_key = max(j0, L - Nq); end_key < min(j0 + 16, L); ++end_key) {
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
              mma_16816<BF16>(tmp, a0, a1, a2, a3, bh[nt][0], bh[nt][1]);
              mma_16816<BF16>(tmp, a0, a1, a2, a3, bl[nt][0], bl[nt][1]);
#pragma unroll
              for (int u = 0; u < 4; ++u)
                if (lim[nt][u & 1] == end_key || (top && lim[nt][u & 1] > end_key)) o[nt][4 * cc + i][u] += tmp[u];
            }
          }
        }
      }
    }
  }

  // Row 8·nt + 2t + u of the warp's output (features [0, D) of `row`); its sum over this lane's keys is l[nt][u].
  __device__ __forceinline__ void store(float* row, int nt, int u) const {
#pragma unroll
    for (int cc = 0; cc < D / 64; ++cc)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        row[64 * cc + 8 * g + 2 * i] = o[nt][4 * cc + i][u];
        row[64 * cc + 8 * g + 2 * i + 1] = o[nt][4 * cc + i][2 + u];
      }
  }
};

// The same for a 4-bit cache; a tile is two sub-tiles of 16 keys.
template <int D, bool BF16, int NT>
struct Rows4 {
  static constexpr int W = D / 32, KS = D / 16, ROW = D / 2, PAIR = D / 8;
  static constexpr bool kRest = !BF16;              // P·scale in two parts
  static constexpr bool kCentre = NT == 1 && !kRest;  // −8·ΣP as a product
  static constexpr int NS = 2;  // sub-tiles in flight together
  static constexpr float kDepth = 7.f;      // the reference is 2^7 under the maximum
  static constexpr float kNone = -3.4028234663852886e38f;  // the reference of a row that has met no key: under every score
  uint32_t qb[NT][KS][2], qs[NT];
  float m[NT][2];  // the reference of s_j + e_j
  float l[NT][2], o[NT][KS][4], mins[NT][4], coef[NT][2];
  int lim[NT][2];
  uint32_t lane_k, lane_v, lane_p, lane_m, lane_a, lane_s;
  int g, t, lane, L, Nq;

  __device__ __forceinline__ void init(const PagedParams& p, int b, int hk, int r0, int len, int lane_) {
    lane = lane_;
    g = lane >> 2;
    t = lane & 3;
    L = len;
    Nq = p.Nq;
    lane_k = lane * PAIR;  // 16 (8) bytes of row g from 16t (8t) on
    lane_v = 32 * ROW + (D == 128 ? 16 * v4_piece<D>(2 * t, g >> 1) + 8 * (g & 1) : 16 * v4_piece<D>(2 * t, g >> 2) + 4 * (g & 3));
    lane_p = 64 * ROW + g * PAIR;                          // the keys' pairs of row g
    lane_m = lane_p + (W == 4 ? (t & 1) * 8 : 0);          // two of them: the minima of groups 2t, 2t + 1 (mod 4)
    lane_s = 64 * ROW + 32 * PAIR + 2 * t * PAIR;          // the values' pairs of row 2t
    lane_a = lane_s + (g & (W - 1)) * 4 + (g < 4 ? 2 : 0); // its minimum (g < 4) or scale of group g mod 4
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + 8 * nt + g;
      const bool on = r < p.R;
      const uint8_t* src = p.q + (on ? paged_row(p, b, hk, r) : 0) * D * 2;
      float f[W][8], most = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint4 v = on ? load_now(reinterpret_cast<const uint4*>(src + (32 * j + 8 * t) * 2)) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = unpack2<BF16>(w[i]);
          f[j][2 * i] = x.x;
          f[j][2 * i + 1] = x.y;
          most = fmaxf(most, fmaxf(fabsf(x.x), fabsf(x.y)));
        }
      }
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // most = x·2^e, 1 <= x < 2; the row goes into the products as q·2^(12 − e), times n·2^-24: s = s'·2^(e + 12).  The
      // sums of 32 features go as Σq·2^(8 − e), below 2^14, in two parts
      const int e = min(max((int)(__float_as_uint(most) >> 23) - 127, -100), 100);
      const float up = __uint_as_float((uint32_t)(127 + 12 - e) << 23);
      const float sums_up = __uint_as_float((uint32_t)(127 + 8 - e) << 23);
      float hi[4] = {0.f, 0.f, 0.f, 0.f}, lo[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float even = up, odd = up * 0.0625f;  // the factors beside n·2^-24 and n·2^-20
        qb[nt][2 * j][0] = pack2<false>(f[j][0] * even, f[j][4] * even);
        qb[nt][2 * j][1] = pack2<false>(f[j][1] * odd, f[j][5] * odd);
        qb[nt][2 * j + 1][0] = pack2<false>(f[j][2] * even, f[j][6] * even);
        qb[nt][2 * j + 1][1] = pack2<false>(f[j][3] * odd, f[j][7] * odd);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += f[j][i];
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        s *= sums_up;
        hi[j] = __half2float(__float2half_rn(s));
        lo[j] = s - hi[j];
      }
      // k-index 0-3: the first parts of groups 0-3, 4-7: the second parts
      qs[nt] = t == 0 ? pack2<false>(hi[0], hi[1]) : t == 1 ? pack2<false>(hi[2], hi[3])
             : t == 2 ? pack2<false>(lo[0], lo[1]) : pack2<false>(lo[2], lo[3]);
      // at least the smallest normal number: a factor of 0 would make a masked score of -inf NaN
      const float back = fmaxf(__uint_as_float((uint32_t)(127 + 12 + e) << 23) * p.scale_log2, 1.17549435e-38f);
      coef[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);
      coef[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int rr = r0 + 8 * nt + 2 * t + u;
        lim[nt][u] = L - Nq + (rr < p.R ? rr / p.G : Nq - 1);
        m[nt][u] = kNone;
        l[nt][u] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) mins[nt][i] = 0.f;
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][j][i] = 0.f;
    }
  }

  // Of s_j + e_j.
  static __device__ __forceinline__ float top_of(const float (&s)[NS][NT][4], int nt, int u) {
    float x = fmaxf(s[0][nt][u], s[0][nt][2 + u]);
#pragma unroll
    for (int ns = 1; ns < NS; ++ns) x = max3f(x, s[ns][nt][u], s[ns][nt][2 + u]);
    return x;
  }

  __device__ __forceinline__ void step(uint32_t tile, int j0, uint32_t flags) {
    const bool special = j0 + 32 > L || flags != 3u;  // some keys are not there
    auto live = [&](int sub, int key) { return ((flags >> sub) & 1u) != 0u && j0 + 16 * sub + key < L; };
    // ---- the values' pairs of row `lane`
    uint32_t w[W];
    const uint32_t aw = tile + 64 * ROW + 32 * PAIR + lane * PAIR;
    if constexpr (W == 4) {
      const uint4 x = lds128<0>(aw);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else {
      const uint2 x = lds64<0>(aw);
      w[0] = x.x; w[1] = x.y;
    }
    // ---- scores of keys j0 + 16·ns + g and + 8
    float s[NS][NT][4];
#pragma unroll
    for (int ns = 0; ns < NS; ++ns) {
      uint32_t kn[2][W], kp[2][W], mn[2];
      const uint32_t ak = tile + lane_k + ns * 16 * ROW, ap = tile + lane_p + ns * 16 * PAIR, am = tile + lane_m + ns * 16 * PAIR;
      if constexpr (W == 4) {
        const uint4 x0 = lds128<0>(ak), x1 = lds128<8 * ROW>(ak), y0 = lds128<0>(ap), y1 = lds128<8 * PAIR>(ap);
        kn[0][0] = x0.x; kn[0][1] = x0.y; kn[0][2] = x0.z; kn[0][3] = x0.w;
        kn[1][0] = x1.x; kn[1][1] = x1.y; kn[1][2] = x1.z; kn[1][3] = x1.w;
        kp[0][0] = y0.x; kp[0][1] = y0.y; kp[0][2] = y0.z; kp[0][3] = y0.w;
        kp[1][0] = y1.x; kp[1][1] = y1.y; kp[1][2] = y1.z; kp[1][3] = y1.w;
        const uint2 z0 = lds64<0>(am), z1 = lds64<8 * PAIR>(am);
        mn[0] = prmt(z0.x, z0.y, 0x7632u);
        mn[1] = prmt(z1.x, z1.y, 0x7632u);
      } else {
        const uint2 x0 = lds64<0>(ak), x1 = lds64<8 * ROW>(ak), y0 = lds64<0>(ap), y1 = lds64<8 * PAIR>(ap);
        kn[0][0] = x0.x; kn[0][1] = x0.y; kn[1][0] = x1.x; kn[1][1] = x1.y;
        kp[0][0] = y0.x; kp[0][1] = y0.y; kp[1][0] = y1.x; kp[1][1] = y1.y;
        mn[0] = prmt(y0.x, y0.y, 0x7632u);
        mn[1] = prmt(y1.x, y1.y, 0x7632u);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float acc[4];
        mma_1688_first(acc, mn[0], mn[1], qs[nt]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[ns][nt][i] = acc[i] * 9.5367431640625e-07f;  // 2^-20: from 2^(8 − e) to 2^-(e + 12)
      }
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint32_t x0 = kn[0][j], x1 = kn[1][j], y0 = x0 >> 8, y1 = x1 >> 8;
        const float p0 = __low2float(*reinterpret_cast<const __half2*>(&kp[0][j]));
        const float p1 = __low2float(*reinterpret_cast<const __half2*>(&kp[1][j]));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float acc[4];
          mma_16816_first(acc, x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, qb[nt][2 * j][0], qb[nt][2 * j][1]);
          mma_16816<false>(acc, y0 & 0x000f000fu, y1 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x00f000f0u, qb[nt][2 * j + 1][0],
                           qb[nt][2 * j + 1][1]);
          s[ns][nt][0] = fmaf(p0, acc[0], s[ns][nt][0]);
          s[ns][nt][1] = fmaf(p0, acc[1], s[ns][nt][1]);
          s[ns][nt][2] = fmaf(p1, acc[2], s[ns][nt][2]);
          s[ns][nt][3] = fmaf(p1, acc[3], s[ns][nt][3]);
        }
      }
    }
    // ---- they are divided by 2^e, which is over the largest of them; where the key is not there they become 0 (what the tile
    // holds may be anything)
    if (special && !live(lane >> 4, lane & 15)) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j] = 0u;
    }
    uint32_t top = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int j = 1; j < W; ++j) top = max2<false>(top, w[j] & 0x7fff7fffu);
    const int e = (int)(max(top & 0xffffu, top >> 16) >> 10) - 14;  // from fp16's exponent: -14 (0 too) … 16
    const uint32_t down = pack2<false>(__uint_as_float((uint32_t)(127 - e) << 23), __uint_as_float((uint32_t)(127 - e) << 23));
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = mul_f16x2(w[j], down);
    if constexpr (W == 4) st_shared_v4(aw, w[0], w[1], w[2], w[3]);
    else st_shared_v2(aw, w[0], w[1]);
    __syncwarp();
    int ek[NS][2];  // e of keys g, g + 8, g + 16 and g + 24
#pragma unroll
    for (int i = 0; i < 4; ++i) ek[i >> 1][i & 1] = __shfl_sync(0xffffffffu, e, g + 8 * i);
    // ---- keys behind a row's last one, or that are not there: they may hold anything, so they are replaced
    if (special || j0 + 31 > L - Nq) {
#pragma unroll
      for (int ns = 0; ns < NS; ++ns)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = g + 8 * (i >> 1);
            if (!live(ns, key) || j0 + 16 * ns + key > lim[nt][i & 1]) s[ns][nt][i] = -INFINITY;
          }
    }
#pragma unroll
    for (int ns = 0; ns < NS; ++ns)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float x = (float)ek[ns][i >> 1];
          fma_pair(s[ns][nt][i], s[ns][nt][i + 1], s[ns][nt][i], s[ns][nt][i + 1], coef[nt][0], coef[nt][1], x, x);
        }
    // ---- the reference (NaN does not raise it: it reaches the sums all the same)
    bool rise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int u = 0; u < 2; ++u) rise |= top_of(s, nt, u) > m[nt][u] + (kDepth + kRise);
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float x = top_of(s, nt, u);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
          const float r = fmaxf(m[nt][u], x - kDepth), alpha = ex2(m[nt][u] - r);
          m[nt][u] = r;
          l[nt][u] *= alpha;
          mins[nt][u] *= alpha;
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            o[nt][j][u] *= alpha;
            o[nt][j][2 + u] *= alpha;
          }
        }
    }
#pragma unroll
    for (int ns = 0; ns < NS; ++ns) {
      // ---- probabilities times 2^e (up to 2^15), rounded to fp16 and transposed; their sum without that factor
      uint32_t bh[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pr[4];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float w = __uint_as_float((uint32_t)(127 - ek[ns][i >> 1]) << 23);
          sub_pair(pr[i], pr[i + 1], s[ns][nt][i], s[ns][nt][i + 1], m[nt][0], m[nt][1]);
          pr[i] = ex2(pr[i]);
          pr[i + 1] = ex2(pr[i + 1]);
          fma_pair(l[nt][0], l[nt][1], pr[i], pr[i + 1], w, w, l[nt][0], l[nt][1]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) bh[nt][u] = movmatrix_trans(pack2<false>(pr[2 * u], pr[2 * u + 1]));
      }
      // ---- values of keys 2t, 2t + 1, 2t + 8, 2t + 9: numbers, pairs, and one minimum or scale of each
      uint32_t v[4][W / 2], pair[4][W], one[4];
      const uint32_t av = tile + lane_v + ns * 16 * ROW, odd = tile + (lane_v ^ ROW) + ns * 16 * ROW;  // row 2t + 1: the swizzle
      const uint32_t as = tile + lane_s + ns * 16 * PAIR, aa = tile + lane_a + ns * 16 * PAIR;         // turns the row's bit too
      one[0] = lds16<0>(aa);
      one[1] = lds16<PAIR>(aa);
      one[2] = lds16<8 * PAIR>(aa);
      one[3] = lds16<9 * PAIR>(aa);
      if constexpr (W == 4) {
        const uint2 n[4] = {lds64<0>(av), lds64<0>(odd), lds64<8 * ROW>(av), lds64<8 * ROW>(odd)};
        const uint4 y[4] = {lds128<0>(as), lds128<PAIR>(as), lds128<8 * PAIR>(as), lds128<9 * PAIR>(as)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i][0] = n[i].x;
          v[i][1] = n[i].y;
          pair[i][0] = y[i].x;
          pair[i][1] = y[i].y;
          pair[i][2] = y[i].z;
          pair[i][3] = y[i].w;
        }
      } else {
        const uint2 y[4] = {lds64<0>(as), lds64<PAIR>(as), lds64<8 * PAIR>(as), lds64<9 * PAIR>(as)};
        v[0][0] = lds32<0>(av);
        v[1][0] = lds32<0>(odd);
        v[2][0] = lds32<8 * ROW>(av);
        v[3][0] = lds32<8 * ROW>(odd);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pair[i][0] = y[i].x;
          pair[i][1] = y[i].y;
        }
      }
      // ---- Σ p·min (rows 0-3 of the product) and Σ p·scale (rows 4-7) of each group
      const uint32_t a01 = prmt(one[0], one[1], 0x5410u), a89 = prmt(one[2], one[3], 0x5410u);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_16816<false>(mins[nt], a01, 0u, a89, 0u, bh[nt][0], bh[nt][1]);
      // ---- Σ (P·scale)·(n − 8)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
        const uint32_t e = prmt(v[0][j >> 1], v[1][j >> 1], sel), f = prmt(v[2][j >> 1], v[3][j >> 1], sel);
        const uint32_t s01 = prmt(pair[0][j], pair[1][j], 0x5410u), s89 = prmt(pair[2][j], pair[3][j], 0x5410u);
        uint32_t a[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t x = u ? e >> 8 : e, y = u ? f >> 8 : f;
          if constexpr (kCentre) {
            a[u][0] = x & 0x000f000fu;
            a[u][1] = x & 0x00f000f0u;
            a[u][2] = y & 0x000f000fu;
            a[u][3] = y & 0x00f000f0u;
          } else {
            a[u][0] = less8<0>(x);
            a[u][1] = less8<4>(x);
            a[u][2] = less8<0>(y);
            a[u][3] = less8<4>(y);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t b0 = mul_f16x2(bh[nt][0], s01), b1 = mul_f16x2(bh[nt][1], s89);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if constexpr (kCentre)  // −8·2^-24 for the even numbers, −8·2^-20 for the odd ones
              mma_16816<false>(o[nt][2 * j + u], 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, b0, b1);
            mma_16816<false>(o[nt][2 * j + u], a[u][0], a[u][1], a[u][2], a[u][3], b0, b1);
          }
          if constexpr (kRest) {
            const uint32_t r0 = rest_f16x2(bh[nt][0], s01, b0), r1 = rest_f16x2(bh[nt][1], s89, b1);
#pragma unroll
            for (int u = 0; u < 2; ++u) mma_16816<false>(o[nt][2 * j + u], a[u][0], a[u][1], a[u][2], a[u][3], r0, r1);
          }
        }
      }
    }
  }

  __device__ __forceinline__ void store(float* row, int nt, int u) const {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float mn = __shfl_sync(0xffffffffu, mins[nt][u], 4 * j + t), sc = __shfl_sync(0xffffffffu, mins[nt][u], 4 * (j + 4) + t);
      const float y = fmaf(8.f, sc, mn);
      float* dst = row + 32 * j + 4 * g;
      dst[0] = fmaf(o[nt][2 * j][u], 16777216.f, y);
      dst[1] = fmaf(o[nt][2 * j][2 + u], 1048576.f, y);
      dst[2] = fmaf(o[nt][2 * j + 1][u], 16777216.f, y);
      dst[3] = fmaf(o[nt][2 * j + 1][2 + u], 1048576.f, y);
    }
  }
};

// One block's work on granules first .. last − 1 of a unit (first == last: none): every row's maximum, sum and output over
// those keys, `emit`ted by the row's warp, d/32 features a lane.  `smem`: Cfg::kSmem bytes; the caller synchronises before
// it calls again.
template <int D, bool BF16, bool Q4, int NT, typename Emit>
__device__ __forceinline__ void run_piece(const PagedParams& p, uint8_t* smem, int b, int hk, int r0, int L, int first, int last, Emit&& emit) {
  using Cfg = PagedConfig<D, Q4, NT>;
  using Rows = std::conditional_t<Q4, Rows4<D, BF16, NT>, Rows16<D, BF16, NT>>;
  constexpr int W = D / 32, ROWS = 8 * NT, S = Cfg::kStages, GK = Cfg::kGranule, T = Cfg::kTile;
  __shared__ float s_m[kPagedWarps][ROWS], s_l[kPagedWarps][ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem) + warp * S * Cfg::kTileBytes;
  float* s_o = reinterpret_cast<float*>(smem);
  const int ps = p.pg.page_size;
  const bool paired = Q4 && ps % 32 != 0;  // a tile's two halves may lie in two pages
  const int step_pages = GK / ps, step_slots = GK - step_pages * ps;

  // ---- the warp's tiles, keys GK·i + T·warp on; page lookups run one tile ahead of the copies
  const int32_t* table = p.pg.page_table + (size_t)b * p.pg.max_pages;
  const int tiles = last - first - (GK * (last - 1) + T * warp >= L ? 1 : 0);
  const TileCopy<D, Q4> copy(p.pg, hk, ring, lane);
  int next_j = GK * first + T * warp;  // the first key of the next tile to be copied
  int page_i = next_j / ps, slot = next_j - page_i * ps;
  int page = tiles > 0 ? load_now(table + page_i) : 0, page2 = 0;
  auto second = [&]() { return slot + 16 >= ps ? page_i + 1 : page_i; };  // the second half's page index
  if (paired && tiles > 0 && next_j + 16 < L) page2 = load_now(table + second());
  int left = tiles;      // to be copied
  uint32_t copy_at = 0;  // the stage of the next one
  uint32_t valid = 0;    // two bits for each of the last tiles copied: the halves that are there
  auto issue = [&]() {
    valid *= 4;
    if (left > 0) {
      --left;
      const bool ok = (unsigned)page < (unsigned)p.pg.num_pages;
      bool bad = !ok;
      if (!paired) {
        if (ok) copy.template rows<T / 16>(page, slot, copy_at, 0);
        valid += ok ? 3u : 0u;
      } else {
        if (ok) copy.template rows<1>(page, slot, copy_at, 0);
        valid += ok ? 1u : 0u;
        if (next_j + 16 < L) {
          const bool ok2 = (unsigned)page2 < (unsigned)p.pg.num_pages;
          if (ok2) copy.template rows<1>(page2, slot + 16 >= ps ? slot + 16 - ps : slot + 16, copy_at, 1);
          valid += ok2 ? 2u : 0u;
          bad = bad || !ok2;
        }
      }
      if (bad && lane == 0) record_status(1);
      next_j += GK;
      page_i += step_pages;
      slot += step_slots;
      if (slot >= ps) {
        slot -= ps;
        ++page_i;
      }
      if (left > 0) {
        page = load_now(table + page_i);
        if (paired && next_j + 16 < L) page2 = load_now(table + second());
      }
    }
    copy_at = copy_at == (S - 1) * Cfg::kTileBytes ? 0 : copy_at + Cfg::kTileBytes;
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue();

  Rows rows;
  rows.init(p, b, hk, r0, L, lane);
  uint32_t tile = ring + (S - 1) * Cfg::kTileBytes;
  int j0 = GK * (first - 1) + T * warp;
#pragma unroll 1
  for (int it = 0; it < tiles; ++it) {
    cp_async_wait<S - 2>();
    __syncwarp();  // the tile is here for every lane, and every lane is done with the one before
    const uint32_t flags = (valid >> (2 * (S - 2))) & 3u;
    issue();
    tile = tile == ring + (S - 1) * Cfg::kTileBytes ? ring : tile + Cfg::kTileBytes;
    j0 += GK;
    if (flags != 0u) rows.step(tile, j0, flags);
  }
  cp_async_wait<0>();
  __syncthreads();  // every warp is done with its ring: the memory now holds the warps' partial outputs
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = 8 * nt + 2 * (lane & 3) + u;
      float x = rows.l[nt][u];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (lane < 4) {
        s_m[warp][r] = rows.m[nt][u];
        s_l[warp][r] = x;
      }
      rows.store(s_o + (warp * ROWS + r) * Cfg::kPitch, nt, u);
    }
  __syncthreads();
  // ---- the block's: a warp per row, d/32 features per lane
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
    emit(r, M, ell, acc);
  }
}

// Output and log-sum-exp of a row from its maximum, sum and output, d/32 features a lane.
template <int D, bool BF16>
__device__ __forceinline__ void finish_row(const PagedParams& p, size_t row, int lane, float M, float ell, const float (&acc)[D / 32]) {
  const float inv = ell == 0.f ? 0.f : 1.f / ell;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) store_out<D, BF16>(p.o, row * D + 32 * j + lane, acc[j] * inv);
  if (lane == 0) p.lse[row] = ell == 0.f ? -INFINITY : (M + log2f(ell)) * 0.69314718055994531f;
}

template <int D, bool BF16, bool Q4, int NT>
__global__ void __launch_bounds__(kPagedThreads, (PagedConfig<D, Q4, NT>::kBlocks)) fa_paged_split_kernel(const PagedParams p) {
  using Cfg = PagedConfig<D, Q4, NT>;
  constexpr int W = D / 32, ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31;
  const int units = p.pg.Hk * p.tiles;  // of one sequence

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // for the merge
  after_earlier_kernels();

  // ---- this block's run of granules
  const GranuleScan scan = scan_granules(p);
  const long long total = scan.total * units, share = granule_share(p, total);
  long long at = blockIdx.x * share;
  const long long end = min(at + share, total);
  __shared__ int s_b;
  __shared__ long long s_before;
  const long long goal = quotient(at, units);
  if (goal >= scan.before && goal < scan.before + scan.mine) {
    long long before = scan.before;
    int b = scan.begin;
    for (;; ++b) {
      const int n = granules(p, paged_length(p, b));
      if (goal < before + n) break;
      before += n;
    }
    s_b = b;
    s_before = before;
  }
  // sequences without keys, and lengths that are out of range: the blocks share them out
  for (int b = blockIdx.x; b < p.pg.B; b += gridDim.x) {
    const int len = paged_length(p, b);
    if (len < 0 && threadIdx.x == 0) record_status(1);
    if (len == 0) {
      const size_t rows = (size_t)p.Nq * p.H;
      for (size_t i = threadIdx.x; i < rows * D; i += kPagedThreads) store_out<D, BF16>(p.o, b * rows * D + i, 0.f);
      for (size_t i = threadIdx.x; i < rows; i += kPagedThreads) p.lse[b * rows + i] = -INFINITY;
    }
    if (len <= 0 && p.by_unit)
      for (int i = threadIdx.x; i < units; i += kPagedThreads) p.units[b * units + i] = make_int4(0, 0, 0, 0);
  }
  if (threadIdx.x == 0 && !p.by_unit) p.units[blockIdx.x] = make_int4(0, 0, 0, 0);
  __syncthreads();
  if (at >= end) return;
  int b = s_b, L = paged_length(p, b), n = granules(p, L);
  const long long in_b = at - s_before * units;
  int unit = (int)quotient(in_b, n), first = (int)(in_b - (long long)unit * n);

#pragma unroll 1
  for (;;) {
    const int last = (int)min((long long)n, first + (end - at));  // granules first .. last − 1 of this unit
    const int hk = unit % p.pg.Hk, r0 = (unit / p.pg.Hk) * ROWS;

    const bool whole = first == 0 && last == n;
    const int part = 2 * blockIdx.x + (first == 0 ? 1 : 0);
    if (first == 0 && threadIdx.x == 0 && (p.by_unit || last < n))  // the blocks behind this one hold the rest
      p.units[p.by_unit ? b * units + unit : (int)blockIdx.x] =
          make_int4(b, unit, blockIdx.x, last < n ? 1 + (int)quotient(n - last + share - 1, share) : 0);
    run_piece<D, BF16, Q4, NT>(p, smem, b, hk, r0, L, first, last, [&](int r, float M, float ell, const float (&acc)[W]) {
      if (whole) {
        finish_row<D, BF16>(p, paged_row(p, b, hk, r0 + r), lane, M, ell, acc);
      } else {
        const size_t row = (size_t)part * ROWS + r;
#pragma unroll
        for (int j = 0; j < W; ++j) p.part_o[row * D + 32 * j + lane] = acc[j];
        if (lane == 0) {
          p.part_ml[2 * row] = M;
          p.part_ml[2 * row + 1] = ell;
        }
      }
    });
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
      n = granules(p, L);
    }
  }
}

// The same for small calls in one kernel without a workspace: a cluster of blocks takes a unit, each block a share of its
// granules, and joins the blocks' parts through distributed shared memory.
template <int D, bool BF16, bool Q4, int NT>
__global__ void __launch_bounds__(kPagedThreads, (PagedConfig<D, Q4, NT>::kBlocks)) fa_paged_cluster_kernel(const PagedParams p) {
  namespace cg = cooperative_groups;
  using Cfg = PagedConfig<D, Q4, NT>;
  constexpr int W = D / 32, ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_ml[ROWS][2];
  after_earlier_kernels();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int units = p.pg.Hk * p.tiles, u = blockIdx.x / C, b = u / units, unit = u - b * units;
  const int hk = unit % p.pg.Hk, r0 = (unit / p.pg.Hk) * ROWS;
  const int L = paged_length(p, b), n = granules(p, L);
  if (L < 0 && unit == 0 && rank == 0 && threadIdx.x == 0) record_status(1);
  const int share = (n + C - 1) / C, first = min(n, rank * share), last = min(n, first + share);
  float* s_o = reinterpret_cast<float*>(smem);
  run_piece<D, BF16, Q4, NT>(p, smem, b, hk, r0, L, first, last, [&](int r, float M, float ell, const float (&acc)[W]) {
    if (C == 1) {
      if (L >= 0) finish_row<D, BF16>(p, paged_row(p, b, hk, r0 + r), lane, M, ell, acc);
      return;
    }
    // in the place of the first warp's part, which this lane has read
#pragma unroll
    for (int j = 0; j < W; ++j) s_o[r * Cfg::kPitch + 32 * j + lane] = acc[j];
    if (lane == 0) {
      s_ml[r][0] = M;
      s_ml[r][1] = ell;
    }
  });
  if (C == 1) return;
  cluster.sync();
  if (L >= 0) {
    for (int r = rank + C * warp; r < ROWS && r0 + r < p.R; r += C * kPagedWarps) {
      float M = -INFINITY;
      for (int c = 0; c < C; ++c) M = fmaxf(M, cluster.map_shared_rank(&s_ml[r][0], c)[0]);
      float ell = 0.f, acc[W];
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] = 0.f;
#pragma unroll 4
      for (int c = 0; c < C; ++c) {
        const float* ml = cluster.map_shared_rank(&s_ml[r][0], c);
        const float* part = cluster.map_shared_rank(s_o + r * Cfg::kPitch, c);
        const float a = join_weight(ml[0], M);
        ell = fmaf(ml[1], a, ell);
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] = fmaf(part[32 * j + lane], a, acc[j]);
      }
      finish_row<D, BF16>(p, paged_row(p, b, hk, r0 + r), lane, M, ell, acc);
    }
  }
  cluster.sync();  // no block's shared memory goes while another reads it
}

// Block (note, row of a tile): joins that row of the unit, whose parts four warps share out.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) fa_paged_merge_kernel(const PagedParams p) {
  constexpr int F = D / 32;
  __shared__ float s_o[4][D], s_l[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.y, tile_rows = gridDim.y;
  after_earlier_kernels();
  const int4 note = load_now(p.units + blockIdx.x);  // sequence, unit of it, first worker, parts
  const int hk = note.y % p.pg.Hk, row = note.y / p.pg.Hk * tile_rows + r, w0 = note.z, parts = note.w;
  if (parts == 0 || row >= p.R) return;
  // the first worker's part is its last one (slot 1), the others' their first (slot 0)
  auto slot = [&](int i) { return (size_t)(2 * (w0 + i) + (i == 0 ? 1 : 0)) * tile_rows + r; };
  float M = -INFINITY;
  for (int i = lane; i < parts; i += 32) M = fmaxf(M, load_now(p.part_ml + 2 * slot(i)));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float ell = 0.f, acc[F];
#pragma unroll
  for (int j = 0; j < F; ++j) acc[j] = 0.f;
#pragma unroll 4
  for (int i = warp; i < parts; i += 4) {
    const size_t s = slot(i);
    const float a = join_weight(load_now(p.part_ml + 2 * s), M);
    ell = fmaf(load_now(p.part_ml + 2 * s + 1), a, ell);
    const float* src = p.part_o + s * D;
#pragma unroll
    for (int j = 0; j < F; ++j) acc[j] = fmaf(load_now(src + 32 * j + lane), a, acc[j]);
  }
#pragma unroll
  for (int j = 0; j < F; ++j) s_o[warp][32 * j + lane] = acc[j];
  if (lane == 0) s_l[warp] = ell;
  __syncthreads();
  if (warp > 0) return;
  ell = s_l[0] + s_l[1] + s_l[2] + s_l[3];
#pragma unroll
  for (int j = 0; j < F; ++j) acc[j] = s_o[0][32 * j + lane] + s_o[1][32 * j + lane] + s_o[2][32 * j + lane] + s_o[3][32 * j + lane];
  finish_row<D, BF16>(p, paged_row(p, note.x, hk, row), lane, M, ell, acc);
}

// Row tiles of a key head, and the rows of one (32, which d = 64 has registers for, were no faster: 27 x 8192 keys of 60 rows
// 41.2 us against 39.5).
static int paged_tile_rows(int R) { return R <= 8 ? 8 : 16; }

// Blocks that can take a run: all that fit the GPU at once (at most four per SM), or one per granule of the longest batch.
static int paged_workers(int B, int Hk, int tiles, int Nk, int granule, int per_sm) {
  const long long most = (long long)B * Hk * tiles * ((Nk + granule - 1) / granule);
  return (int)std::min<long long>(most, (long long)kSmCount * per_sm);
}

// Blocks of a cluster that takes one unit, 0 where the keys are dealt out instead.  Clusters need one launch and no second
// pass over partial outputs, but a cluster's blocks have to be on the GPU at once and all units take as long as the longest.
// As many blocks (1, 2, 4 or 8) as the keys fill (over 64 each) and the GPU holds beside one another (a sixteenth is left
// because clusters do not pack); the keys are dealt out where a block would get more than 1024 of them (2048 where the
// blocks fill the GPU).  Units that do not all fit at once take one block each up to 2048 keys.
// us of batches with half to all of the given keys, 16 bits, d = 128, clusters and dealt out: 12 x 256 keys x 16 heads 6.8 and
// 11.5; 37 x 512 x 4 heads of 20 rows 12.9 and 22.7; 37 x 1024 x 1 head of 16 rows 10.8 and 15.6; 1 x 4096 x
// 8 heads 10.3 and 11.4; 4 x 8192 x 4 heads of 20 rows 21.5 and 25.6, but 1 x 8192 x 16 heads 17.3 and 15.9; 4 bits:
// 37 x 2048 x 16 heads of 10 rows 56.3 and 64.3, 37 x 4096 x 16 heads of 1 row 83.9 and 68.8 (dealt out by the rule).
static int paged_cluster(int B, int Hk, int tiles, int Nk, int per_sm) {
  const long long units = (long long)B * Hk * tiles, room = kSmCount * per_sm * 15 / 16;
  if (units > room) return Nk <= 2048 ? 1 : 0;
  int C = 8;
  while (C > 1 && (Nk <= 64 * C || units * C > room)) C /= 2;
  return (Nk + C - 1) / C <= (10 * units * C >= 7 * room ? 2048 : 1024) ? C : 0;
}

void paged_workspace(int B, int Nq, int H, int Hk, int Nk, int d, size_t* o_bytes, size_t* ml_bytes, size_t* unit_bytes) {
  const int R = H / Hk * Nq, rows = paged_tile_rows(R), tiles = (R + rows - 1) / rows;
  const int nt = rows / 8;
  if (paged_cluster(B, Hk, tiles, Nk, paged_blocks(d, false, nt)) > 0 && paged_cluster(B, Hk, tiles, Nk, paged_blocks(d, true, nt)) > 0) {
    *o_bytes = *ml_bytes = *unit_bytes = 0;
    return;
  }
  const size_t workers = paged_workers(B, Hk, tiles, Nk, granule_keys(false), 4), slots = 2 * workers * rows;
  *unit_bytes = workers * sizeof(int4);
  *o_bytes = slots * d * sizeof(float);
  *ml_bytes = slots * 2 * sizeof(float);
}

template <int D, bool BF16, bool Q4, int NT>
static cudaError_t launch_paged_v(PagedParams p, int B, int Nk, cudaStream_t stream) {
  using Cfg = PagedConfig<D, Q4, NT>;
  static std::atomic<unsigned long long> done[2] = {{0}, {0}};
  p.granule = Cfg::kGranule;
  const int C = paged_cluster(B, p.pg.Hk, p.tiles, Nk, Cfg::kBlocks);
  const void* kernel = C > 0 ? reinterpret_cast<const void*>(fa_paged_cluster_kernel<D, BF16, Q4, NT>)
                             : reinterpret_cast<const void*>(fa_paged_split_kernel<D, BF16, Q4, NT>);
  cudaError_t e = set_smem_once(done[C > 0], kernel, Cfg::kSmem);
  if (e != cudaSuccess) return e;
  if (C > 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * p.pg.Hk * p.tiles * C));
    cfg.blockDim = dim3(kPagedThreads);
    cfg.dynamicSmemBytes = Cfg::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fa_paged_cluster_kernel<D, BF16, Q4, NT>, p);
  }
  p.workers = paged_workers(B, p.pg.Hk, p.tiles, Nk, Cfg::kGranule, Cfg::kBlocks);
  p.by_unit = (long long)B * p.pg.Hk * p.tiles <= p.workers;
  e = launch_after(fa_paged_split_kernel<D, BF16, Q4, NT>, dim3((unsigned)p.workers), dim3(kPagedThreads), Cfg::kSmem, stream, p);
  if (e != cudaSuccess) return e;
  // the merge is launched while the runs end; it waits for them before it reads
  const unsigned notes = (unsigned)(p.by_unit ? B * p.pg.Hk * p.tiles : p.workers);
  return launch_after(fa_paged_merge_kernel<D, BF16>, dim3(notes, 8 * NT), dim3(128), 0, stream, p);
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
  p.units = static_cast<int4*>(a.units);
  p.pg = pg;
  p.Nq = a.Nq;
  p.H = a.H;
  p.G = a.H / pg.Hk;
  p.most = std::min(a.Nk, pg.max_pages * pg.page_size);
  p.R = p.G * a.Nq;
  p.tiles = (p.R + paged_tile_rows(p.R) - 1) / paged_tile_rows(p.R);
  p.workers = p.granule = 0;
  p.by_unit = false;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  if (pg.d == 128) return pg.bf16 ? launch_paged_t<128, true>(p, pg.B, a.Nk, stream) : launch_paged_t<128, false>(p, pg.B, a.Nk, stream);
  return pg.bf16 ? launch_paged_t<64, true>(p, pg.B, a.Nk, stream) : launch_paged_t<64, false>(p, pg.B, a.Nk, stream);
}

}  // namespace fa
