// fa_paged_api.cu — the C ABI of what stands around the attention: the norm and rotation of queries and
// keys, and the paged key/value cache.  Validation as in fa_api.cu: everything that the host can see is
// checked before anything is launched; what only the device holds (positions, offsets, lengths, page
// numbers) is checked in the kernels, which skip what is out of range and record it.
#include <cmath>

#include "../../include/fa.h"
#include "fa_paged_internal.h"

namespace fa {

// [T, H, d] with a token stride: whole 16-byte pieces, rows that do not overlap.
static bool good_stride(long long stride, int H, int d) { return stride >= (long long)H * d && (stride & 7) == 0 && stride <= (1LL << 40); }

static int check_heads(int T, int Hq, int Hk, int d, int dtype) {
  if (T < 1 || Hq < 1 || Hk < 1 || (d != 64 && d != 128)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_INVALID_ARG;
  if (Hq > (1 << 20) || Hk > (1 << 20)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// The rotation's arguments.  cos_t == sin_t == nullptr: no rotation (only where `optional`).
static int set_rope(RopeArgs* r, const float* cos_t, const float* sin_t, const int32_t* positions, bool positions_optional,
                    bool optional, int d, int rot_dim, int table_rows, int axes, const int* sections, int interleaved) {
  *r = RopeArgs{};
  if (interleaved != 0 && interleaved != 1) return FA_ERR_INVALID_ARG;
  if (optional && cos_t == nullptr && sin_t == nullptr) return positions == nullptr ? FA_OK : FA_ERR_INVALID_ARG;
  if (!aligned16(cos_t) || !aligned16(sin_t)) return FA_ERR_INVALID_ARG;
  if (positions == nullptr ? !positions_optional : !aligned4(positions)) return FA_ERR_INVALID_ARG;
  if (rot_dim < 16 || rot_dim > d || (rot_dim & 15) != 0 || table_rows < 1) return FA_ERR_INVALID_ARG;
  if (axes < 1 || axes > kRopeMaxAxes || (axes > 1 && (sections == nullptr || positions == nullptr))) return FA_ERR_INVALID_ARG;
  int end = 0;
  for (int a = 0; a < axes; ++a) {
    const int n = axes == 1 ? rot_dim / 2 : sections[a];
    if (n < 4 || (n & 3) != 0 || n > rot_dim / 2) return FA_ERR_INVALID_ARG;
    end += n;
    r->section_end[a] = end;
  }
  if (end != rot_dim / 2) return FA_ERR_INVALID_ARG;
  r->cos_t = cos_t;
  r->sin_t = sin_t;
  r->positions = positions;
  r->rot_dim = rot_dim;
  r->table_rows = table_rows;
  r->axes = axes;
  r->interleaved = interleaved != 0;
  return FA_OK;
}

static bool good_eps(float eps) { return std::isfinite(eps) && eps > 0.f; }

static int set_paged(PagedArgs* p, const void* k_cache, const void* v_cache, const int32_t* page_table, const int32_t* seqlens_k,
                     bool need_lens, int B, int Hk, int d, int page_size, int num_pages, int max_pages, int dtype, int format) {
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned4(page_table)) return FA_ERR_INVALID_ARG;
  if (need_lens && !aligned4(seqlens_k)) return FA_ERR_INVALID_ARG;
  if (B < 1 || Hk < 1 || (d != 64 && d != 128) || page_size < 1 || num_pages < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_INVALID_ARG;
  if (format != FA_CACHE_16BIT && format != FA_CACHE_INT4) return FA_ERR_INVALID_ARG;
  if ((page_size & 15) != 0 || page_size > (1 << 20)) return FA_ERR_UNSUPPORTED;
  if ((long long)max_pages * page_size > (1LL << 30)) return FA_ERR_UNSUPPORTED;
  if ((long long)Hk * page_size > (1LL << 31) / (2 * d)) return FA_ERR_UNSUPPORTED;  // a page's bytes in 32 bits
  if (Hk > 65535 || B > (1 << 24)) return FA_ERR_UNSUPPORTED;
  p->k_cache = const_cast<void*>(k_cache);
  p->v_cache = const_cast<void*>(v_cache);
  p->page_table = page_table;
  p->seqlens_k = seqlens_k;
  p->B = B;
  p->Hk = Hk;
  p->d = d;
  p->page_size = page_size;
  p->num_pages = num_pages;
  p->max_pages = max_pages;
  p->bf16 = dtype == FA_BF16;
  p->q4 = format == FA_CACHE_INT4;
  return FA_OK;
}

static size_t qk_bwd_workspace(int d) { return align256((size_t)kQkBwdBlocks * d * sizeof(float)); }

static size_t decode_paged_workspace(int B, int Nq, int H, int Hk, int Nk, int d, size_t* ml_at, size_t* units_at) {
  size_t o_bytes, ml_bytes, unit_bytes;
  paged_workspace(B, Nq, H, Hk, Nk, d, &o_bytes, &ml_bytes, &unit_bytes);
  *ml_at = align256(o_bytes);
  *units_at = *ml_at + align256(ml_bytes);
  return *units_at + align256(unit_bytes);
}

}  // namespace fa

using namespace fa;

extern "C" {

int fa_rope_table(float* cos_t, float* sin_t, int table_rows, int rot_dim, double base, fa_stream_t stream) {
  if (!aligned16(cos_t) || !aligned16(sin_t)) return FA_ERR_INVALID_ARG;
  if (table_rows < 1 || rot_dim < 16 || rot_dim > 128 || (rot_dim & 15) != 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(base) || !(base > 1.0)) return FA_ERR_INVALID_ARG;
  return map_launch(launch_rope_table(cos_t, sin_t, table_rows, rot_dim, base, reinterpret_cast<cudaStream_t>(stream)));
}

int fa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const void* wq, const void* wk, const float* cos_t,
                    const float* sin_t, const int32_t* positions, int T, int Hq, int Hk, int d, long long q_stride,
                    long long k_stride, long long q_out_stride, long long k_out_stride, int rot_dim, int table_rows, int axes,
                    const int* sections, int interleaved, float eps, int dtype, fa_stream_t stream) {
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out)) return FA_ERR_INVALID_ARG;
  int st = check_heads(T, Hq, Hk, d, dtype);
  if (st != FA_OK) return st;
  if (!good_stride(q_stride, Hq, d) || !good_stride(k_stride, Hk, d) || !good_stride(q_out_stride, Hq, d) ||
      !good_stride(k_out_stride, Hk, d))
    return FA_ERR_INVALID_ARG;
  if ((wq == nullptr) != (wk == nullptr)) return FA_ERR_INVALID_ARG;
  if (wq != nullptr && (!aligned16(wq) || !aligned16(wk) || !good_eps(eps))) return FA_ERR_INVALID_ARG;
  RopeArgs ra;
  st = set_rope(&ra, cos_t, sin_t, positions, false, false, d, rot_dim, table_rows, axes, sections, interleaved);
  if (st != FA_OK) return st;
  const QkArgs a = {q, k, q_out, k_out, wq, wk, q_stride, k_stride, q_out_stride, k_out_stride, T, Hq, Hk, eps};
  return map_launch(launch_qk_norm_rope(a, ra, d, dtype == FA_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

size_t fa_qk_norm_rope_bwd_workspace_bytes(int d) { return d == 64 || d == 128 ? qk_bwd_workspace(d) : 0; }

int fa_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k, const void* wq, const void* wk,
                        const float* cos_t, const float* sin_t, const int32_t* positions, void* dq, void* dk, float* dwq,
                        float* dwk, int T, int Hq, int Hk, int d, long long dq_out_stride, long long dk_out_stride,
                        long long q_stride, long long k_stride, long long dq_stride, long long dk_stride, int rot_dim,
                        int table_rows, int axes, const int* sections, int interleaved, float eps, int dtype, void* workspace,
                        size_t workspace_bytes_, fa_stream_t stream) {
  if (!aligned16(dq_out) || !aligned16(dk_out) || !aligned16(dq) || !aligned16(dk)) return FA_ERR_INVALID_ARG;
  int st = check_heads(T, Hq, Hk, d, dtype);
  if (st != FA_OK) return st;
  if (!good_stride(dq_out_stride, Hq, d) || !good_stride(dk_out_stride, Hk, d) || !good_stride(dq_stride, Hq, d) ||
      !good_stride(dk_stride, Hk, d))
    return FA_ERR_INVALID_ARG;
  if ((wq == nullptr) != (wk == nullptr)) return FA_ERR_INVALID_ARG;
  QkBwdArgs a = {};
  if (wq != nullptr) {
    if (!aligned16(wq) || !aligned16(wk) || !aligned16(q) || !aligned16(k) || !aligned4(dwq) || !aligned4(dwk) || !good_eps(eps))
      return FA_ERR_INVALID_ARG;
    if (!good_stride(q_stride, Hq, d) || !good_stride(k_stride, Hk, d)) return FA_ERR_INVALID_ARG;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes_ < qk_bwd_workspace(d))
      return FA_ERR_INVALID_ARG;
    a.q = q;
    a.k = k;
    a.wq = wq;
    a.wk = wk;
    a.dwq = dwq;
    a.dwk = dwk;
    a.part = reinterpret_cast<float*>(workspace);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.eps = eps;
  }
  RopeArgs ra;
  st = set_rope(&ra, cos_t, sin_t, positions, false, false, d, rot_dim, table_rows, axes, sections, interleaved);
  if (st != FA_OK) return st;
  a.dq_out = dq_out;
  a.dk_out = dk_out;
  a.dq = dq;
  a.dk = dk;
  a.gq_stride = dq_out_stride;
  a.gk_stride = dk_out_stride;
  a.dq_stride = dq_stride;
  a.dk_stride = dk_stride;
  a.T = T;
  a.Hq = Hq;
  a.Hk = Hk;
  return map_launch(launch_qk_norm_rope_bwd(a, ra, d, dtype == FA_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

size_t fa_cache_bytes(int num_pages, int page_size, int Hk, int d, int cache_format) {
  if (num_pages < 1 || page_size < 1 || Hk < 1 || (d != 64 && d != 128)) return 0;
  if (cache_format != FA_CACHE_16BIT && cache_format != FA_CACHE_INT4) return 0;
  const size_t row = cache_format == FA_CACHE_INT4 ? (size_t)d * 5 / 8 : (size_t)d * 2;
  return (size_t)num_pages * page_size * Hk * row;
}

int fa_cache_append(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache, const void* wq,
                    const void* wk, const float* cos_t, const float* sin_t, const int32_t* positions, const int32_t* page_table,
                    const int32_t* seqlens_k, const int32_t* cu_seqlens, int B, int T, int Hq, int Hk, int d, long long q_stride,
                    long long k_stride, long long v_stride, long long q_out_stride, int page_size, int num_pages, int max_pages,
                    int rot_dim, int table_rows, int axes, const int* sections, int interleaved, float eps, int dtype,
                    int cache_format, fa_stream_t stream) {
  PagedArgs pg;
  int st = set_paged(&pg, k_cache, v_cache, page_table, seqlens_k, true, B, Hk, d, page_size, num_pages, max_pages, dtype, cache_format);
  if (st != FA_OK) return st;
  if (!aligned16(k) || !aligned16(v) || T < 1) return FA_ERR_INVALID_ARG;
  if (!good_stride(k_stride, Hk, d) || !good_stride(v_stride, Hk, d)) return FA_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr) || (q == nullptr) != (Hq == 0)) return FA_ERR_INVALID_ARG;
  if (q != nullptr) {
    st = check_heads(T, Hq, Hk, d, dtype);
    if (st != FA_OK) return st;
    if (!aligned16(q) || !aligned16(q_out) || !good_stride(q_stride, Hq, d) || !good_stride(q_out_stride, Hq, d))
      return FA_ERR_INVALID_ARG;
  }
  if ((wq != nullptr && q == nullptr) || (q != nullptr && (wq == nullptr) != (wk == nullptr))) return FA_ERR_INVALID_ARG;
  if (wk != nullptr && (!aligned16(wk) || !good_eps(eps))) return FA_ERR_INVALID_ARG;
  if (wq != nullptr && !aligned16(wq)) return FA_ERR_INVALID_ARG;
  if (cu_seqlens == nullptr ? T % B != 0 : !aligned4(cu_seqlens)) return FA_ERR_INVALID_ARG;
  RopeArgs ra;
  st = set_rope(&ra, cos_t, sin_t, positions, true, true, d, rot_dim, table_rows, axes, sections, interleaved);
  if (st != FA_OK) return st;
  const AppendArgs a = {q, k, v, q_out, wq, wk, cu_seqlens, q_stride, k_stride, v_stride, q_out_stride, T, Hq, eps};
  return map_launch(launch_cache_append(a, ra, pg, reinterpret_cast<cudaStream_t>(stream)));
}

int fa_cache_gather(const void* k_cache, const void* v_cache, void* k, void* v, const int32_t* page_table,
                    const int32_t* cu_seqlens_k, const int32_t* starts, int B, int total_keys, int Hk, int d, int page_size,
                    int num_pages, int max_pages, int dtype, int cache_format, fa_stream_t stream) {
  PagedArgs pg;
  int st = set_paged(&pg, k_cache, v_cache, page_table, nullptr, false, B, Hk, d, page_size, num_pages, max_pages, dtype, cache_format);
  if (st != FA_OK) return st;
  if (!aligned16(k) || !aligned16(v) || total_keys < 1) return FA_ERR_INVALID_ARG;
  if (starts != nullptr && !aligned4(starts)) return FA_ERR_INVALID_ARG;
  if (cu_seqlens_k == nullptr ? total_keys % B != 0 : !aligned4(cu_seqlens_k)) return FA_ERR_INVALID_ARG;
  const GatherArgs a = {k, v, cu_seqlens_k, starts, total_keys};
  return map_launch(launch_cache_gather(a, pg, reinterpret_cast<cudaStream_t>(stream)));
}

static bool paged_sizes(int B, int Nq, int H, int Hk, int Nk, int d) {
  if (B < 1 || Nq < 1 || H < 1 || Hk < 1 || Nk < 1 || (d != 64 && d != 128) || H % Hk != 0) return false;
  if (Nk > (1 << 30) || H > (1 << 20) || Nq > (1 << 20) || (long long)B * Nq * H > 0x7fffffffLL) return false;
  const long long rows = (long long)(H / Hk) * Nq;
  return B <= 65535 && rows <= 0x3fffffffLL && (rows + 15) / 16 * Hk <= 65535;  // units in 32 bits
}

size_t fa_decode_paged_workspace_bytes(int B, int Nq, int H, int Hk, int Nk, int d) {
  if (!paged_sizes(B, Nq, H, Hk, Nk, d)) return 0;
  size_t ml_at, units_at;
  return decode_paged_workspace(B, Nq, H, Hk, Nk, d, &ml_at, &units_at);
}

int fa_decode_paged(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse, const int32_t* page_table,
                    const int32_t* seqlens_k, int B, int Nq, int H, int Hk, int Nk, int d, float scale, int page_size,
                    int num_pages, int max_pages, int dtype, int cache_format, void* workspace, size_t workspace_bytes_,
                    fa_stream_t stream) {
  PagedArgs pg;
  int st = set_paged(&pg, k_cache, v_cache, page_table, seqlens_k, true, B, Hk, d, page_size, num_pages, max_pages, dtype, cache_format);
  if (st != FA_OK) return st;
  if (!aligned16(q) || !aligned16(o) || !aligned4(lse)) return FA_ERR_INVALID_ARG;
  if (Nq < 1 || H < 1 || Nk < 1 || H % Hk != 0 || !std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (!paged_sizes(B, Nq, H, Hk, Nk, d)) return FA_ERR_UNSUPPORTED;
  size_t ml_at, units_at;
  const size_t need = decode_paged_workspace(B, Nq, H, Hk, Nk, d, &ml_at, &units_at);
  if (need > 0 && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes_ < need))
    return FA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const PagedDecodeArgs a = {q, o, lse, reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + ml_at), ws + units_at, Nq, H, Nk, scale};
  return map_launch(launch_decode_paged(a, pg, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
