// serve_attn.cuh - launch parameters and device helpers of the two attention
// kernels over the paged 8-bit cache.
#pragma once

#include "serve_common.cuh"

namespace ajvp_serve {

struct CacheAttnParams {
  const void* q;  // [B, n, H, d] by strides
  int64_t q_seq, q_token, q_head;
  const uint8_t* codes[2];  // k, v
  const float* scale[2];
  int64_t page_stride, head_stride, token_stride, scale_page, scale_head;
  const int32_t* lens;
  const int32_t* table;
  int64_t table_stride;
  void* o;     // [B, n, H, d]
  float* lse;  // [B, H, n]
  unsigned int* status;
  int B, n, H, Hkv, group;  // group = H / Hkv
  int pages, table_width, page_shift;
  int causal;
  int row_tiles;  // tiles of query rows per (sequence, key head)
  int splits;     // blocks of a cluster that share one tile's keys
  float scale_log2;
};

constexpr float kMinScale = 9.094947017729282e-13f;  // 2^-40
constexpr float kMaxScale = 1.099511627776e12f;      // 2^40
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum is raised only when a score exceeds it by more than
// this many powers of two, so accumulators are rarely rescaled; p <= 2^8
// stays well inside fp16 and fp32.
constexpr float kLazyMax = 8.f;

__device__ __forceinline__ float read_scale(float s) {
  return fminf(fmaxf(s, kMinScale), kMaxScale);  // a NaN reads as the smallest
}

// Length of sequence b in the cache; 0 and an error if it is out of range.
__device__ __forceinline__ int checked_len(const CacheAttnParams& p, int b) {
  const int len = p.lens[b];
  if (len >= 0 && len <= (int64_t(p.table_width) << p.page_shift)) return len;
  if (threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
  return 0;
}

// Page of token j of sequence b; -1 (and an error) if it is out of range.
// `j` is below the sequence's length.
__device__ __forceinline__ int checked_page(const CacheAttnParams& p, int b, int j) {
  const int page = p.table[b * p.table_stride + (j >> p.page_shift)];
  if (page >= 0 && page < p.pages) return page;
  atomicOr(p.status, kStatusBadIndex);
  return -1;
}

__device__ __forceinline__ float rcp_approx(float x) {  // exact for powers of two
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Another block's shared memory.
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

constexpr int kRowsTile = 16;  // most query rows per key head of attn_cache_rows.cu
// attn_cache_tiles.cu: pairs of tiles of 128 query rows on tcgen05, split for
// sequences of up to `keys` tokens
cudaError_t cache_tiles_launch(const CacheAttnParams& p, int64_t keys, int d, int dtype, cudaStream_t st);
constexpr int kTilesRows = 256;

}  // namespace ajvp_serve
