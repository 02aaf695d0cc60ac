// fa_paged_internal.h — declarations shared by the entry points (fa_paged_api.cu) and the kernels of what stands around
// the attention: the norm and rotation of queries and keys, and the paged key/value cache.
#pragma once

#include "fa_internal.h"

namespace fa {

// Launches a kernel that may be scheduled while the one before it in the stream ends (programmatic dependent launch);
// it waits for that one itself (after_earlier_kernels) before it touches global memory.
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The first statement of kernels launched by launch_after: waits until all kernels before this one are through, with what
// they wrote.  Blocks that are there before their turn hide the launch: a call of 777 keys decoded 8.2 -> 6.3 us, a gather of
// 2700 keys 6.2 -> 4.7.  (With launch_dependents in every kernel too, so that several calls queue up on the SMs, that gather
// took 7.4.)
__device__ __forceinline__ void after_earlier_kernels() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Loads behind that wait.  They are ordinary loads that the compiler keeps behind it; the read-only path (ld.global.nc) and
// the cache-hint intrinsics promise it data that no kernel at work writes, and may be moved.
template <typename T>
__device__ __forceinline__ T load_now(const T* p) { return *p; }
// The same for data that is read once.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load_once(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.cs.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// The grid rules' number of SMs (B200).
constexpr int kSmCount = 148;

// Rotation by position (rope.cuh): tables fp32 [table_rows, rot_dim/2] (nullptr: no rotation), positions
// int32 [axes, T] (nullptr where the kernel knows them); frequencies [section_end[a−1], section_end[a])
// go by axis a.
constexpr int kRopeMaxAxes = 4;
struct RopeArgs {
  const float* cos_t;
  const float* sin_t;
  const int32_t* positions;
  int rot_dim, table_rows, axes;
  int section_end[kRopeMaxAxes];
  bool interleaved;
};

// Norm and rotation of queries and keys (fa_rope.cu); strides in elements per token.
struct QkArgs {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const void* wq;  // norm weights (nullptr: no norm)
  const void* wk;
  long long q_stride, k_stride, q_out_stride, k_out_stride;
  int T, Hq, Hk;
  float eps;
};
constexpr int kQkBwdBlocks = 2 * kSmCount;  // at most, for the queries and the keys together
struct QkBwdArgs {
  const void* dq_out;
  const void* dk_out;
  const void* q;
  const void* k;
  const void* wq;
  const void* wk;
  void* dq;
  void* dk;
  float* dwq;
  float* dwk;
  float* part;  // [blocks, d]
  long long gq_stride, gk_stride, q_stride, k_stride, dq_stride, dk_stride;
  int T, Hq, Hk, q_blocks;
  float eps;
};
cudaError_t launch_qk_norm_rope(const QkArgs& a, const RopeArgs& ra, int d, bool bf16, cudaStream_t stream);
cudaError_t launch_qk_norm_rope_bwd(const QkBwdArgs& a, const RopeArgs& ra, int d, bool bf16, cudaStream_t stream);
cudaError_t launch_rope_table(float* cos_t, float* sin_t, int rows, int rot_dim, double base, cudaStream_t stream);

// A paged key/value cache (paged.cuh).
struct PagedArgs {
  void* k_cache;
  void* v_cache;
  const int32_t* page_table;  // [B, max_pages]
  const int32_t* seqlens_k;   // [B]
  int B, Hk, d, page_size, num_pages, max_pages;
  bool bf16, q4;
};
struct AppendArgs {
  const void* q;  // nullptr with Hq = 0: no queries
  const void* k;
  const void* v;
  void* q_out;
  const void* wq;
  const void* wk;
  const int32_t* cu_seqlens;
  long long q_stride, k_stride, v_stride, q_out_stride;
  int T, Hq;
  float eps;
};
struct GatherArgs {
  void* k;
  void* v;
  const int32_t* cu_seqlens;
  const int32_t* starts;
  int T;
};
struct PagedDecodeArgs {
  const void* q;
  void* o;
  float* lse;
  float* part_o;   // sizes from paged_workspace
  float* part_ml;
  void* units;
  int Nq, H, Nk;
  float scale;
};
void paged_workspace(int B, int Nq, int H, int Hk, int Nk, int d, size_t* o_bytes, size_t* ml_bytes,
                     size_t* unit_bytes);
cudaError_t launch_cache_append(const AppendArgs& a, const RopeArgs& ra, const PagedArgs& pg, cudaStream_t stream);
cudaError_t launch_cache_gather(const GatherArgs& a, const PagedArgs& pg, cudaStream_t stream);
cudaError_t launch_decode_paged(const PagedDecodeArgs& a, const PagedArgs& pg, cudaStream_t stream);

}  // namespace fa
