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

constexpr float kLn2 = 0.6931471805599453f;

// e of the power of two 2^-e that scales a row of bf16 queries, amax the largest
// finite |q|, into fp16: to below 1, as far as 2^e and 2^-e are normal 32-bit
// numbers (subnormal rows have few bits anyway), and from 2^113 on only to below
// 2^15, which keeps 2^e times the softmax scale in range.
__device__ __forceinline__ int query_exp(float amax) {
  int e = 0;
  if (amax > 0.f) frexpf(amax, &e);
  return min(max(e, -126), 113);
}

// Length of sequence b in the cache; 0 and an error if it is out of range.
__device__ __forceinline__ int checked_len(const CacheAttnParams& p, int b) {
  const int len = p.lens[b];
  if (len >= 0 && len <= (int64_t(p.table_width) << p.page_shift)) return len;
  atomicOr(p.status, kStatusBadIndex);
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

// What a block of the shared-out steps leaves for the join, behind all places
// of the workspace (two places per block, for its first and its last piece).
struct Piece {
  static constexpr int kNone = -1;
  int went_on;  // number of a tile that an earlier block began (in its first place), or kNone
  int begun;    // that of a tile that it began and a later block goes on with, or kNone
  int place;    // where the begun tile's sums are
  int unused;
};

// The steps of all sequences in a row, own(b) of sequence b, are shared out to
// `blocks` blocks: block k has steps [all k / blocks, all (k + 1) / blocks). Of
// the blocks given only so many take part that each has `least` steps or more:
// the lengths may be far below what the host could know. Gives `all`, the
// blocks that take part, and for one of them the sequence that holds its first
// step, and the number of steps before that sequence. The whole block calls
// this.
template <int THREADS, typename Own>
__device__ __forceinline__ void find_step(int B, int64_t share, int least, Own own, int64_t& blocks,
                                          int64_t& all, int& b, int64_t& before) {
  __shared__ int64_t warp_sum[THREADS / 32];
  __shared__ int64_t at[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // inclusive sums over THREADS sequences at a time
  auto scan = [&](int64_t x, int64_t& total) -> int64_t {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    total = 0;
    int64_t base = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) base += warp_sum[w];
      total += warp_sum[w];
    }
    return base + x;
  };
  all = 0;
  const int64_t first = static_cast<int>(threadIdx.x) < B ? own(threadIdx.x) : 0;  // kept for the second pass
  for (int i0 = 0; i0 < B; i0 += THREADS) {
    const int i = i0 + threadIdx.x;
    int64_t total;
    scan(i0 == 0 ? first : i < B ? own(i) : 0, total);
    all += total;
  }
  blocks = max(min(blocks, all / least), int64_t(1));
  const int64_t w = all * min(share, blocks - 1) / blocks;
  int64_t passed = 0;
  for (int i0 = 0; i0 < B; i0 += THREADS) {
    const int i = i0 + threadIdx.x;
    const int64_t x = i0 == 0 ? first : i < B ? own(i) : 0;
    int64_t total;
    const int64_t end = passed + scan(x, total);
    if (w < end && w >= end - x) {
      at[0] = i;
      at[1] = end - x;
    }
    passed += total;
  }
  __syncthreads();
  b = static_cast<int>(at[0]);
  before = at[1];
}

// Running join of pieces' sums of p v, maxima and sums of p.
struct Join {
  float top = -INFINITY, sum = 0.f;
  __device__ __forceinline__ void add(float m, float l, float4* y, const float4* z, int n) {
    const float to = fmaxf(top, m);
    const float f = to == -INFINITY ? 1.f : ajvp::ex2_approx(top - to);
    const float g = to == -INFINITY ? 1.f : ajvp::ex2_approx(m - to);
    sum = sum * f + l * g;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      y[i].x = y[i].x * f + z[i].x * g, y[i].y = y[i].y * f + z[i].y * g;
      y[i].z = y[i].z * f + z[i].z * g, y[i].w = y[i].w * f + z[i].w * g;
    }
    top = to;
  }
};

// Blocks after `first`, in steps of 32 from k0 on, that went on with `tile`: a
// bit each; `more` if the next 32 have to be looked at too. A whole warp.
__device__ __forceinline__ uint32_t went_on(const Piece* pieces, int blocks, int k0, int tile, bool& more) {
  const int k = k0 + static_cast<int>(threadIdx.x & 31);
  const int on = k < blocks ? pieces[k].went_on : Piece::kNone;
  const uint32_t ends = __ballot_sync(0xffffffffu, on != tile);
  const uint32_t mine = __ballot_sync(0xffffffffu, on == tile);
  more = ends == 0 && k0 + 32 < blocks;
  return ends ? mine & ((ends & -ends) - 1) : mine;
}

constexpr int kRowsTile = 16;  // most query rows per key head of attn_cache_rows.cu
// attn_cache_tiles.cu: pairs of tiles of 128 query rows on tcgen05, on `blocks`
// blocks; `work` has tiles_work_bytes of each.
cudaError_t cache_tiles_launch(const CacheAttnParams& p, int d, int dtype, int blocks, float* work,
                               cudaStream_t st);
int64_t tiles_work_bytes(int64_t d);
constexpr int kTilesRows = 256;

}  // namespace ajvp_serve
