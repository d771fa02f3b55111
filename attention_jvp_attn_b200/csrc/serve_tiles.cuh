// serve_tiles.cuh - 128 x 128 attention tiles on tcgen05 for the serving
// operators: one thread per query row, scores and probabilities in tensor
// memory (the probabilities over their own scores), sums in tensor memory.
#pragma once

#include "serve_common.cuh"
#include "tiles.cuh"

namespace ajvp_serve {

using ajvp::named_bar_sync;
using ajvp::smem_u32;
using ajvp::umma_commit;
using ajvp::warp_uniform;

constexpr int kTile = 128;  // query rows and keys of a tile

// Instruction descriptor, kind::f16: fp32 sums, A and B both bf16 or both fp16.
template <bool F16>
__host__ __device__ constexpr uint32_t tile_idesc(int M, int N, int b_mn_major) {
  return F16 ? ajvp::idesc_bf16_f32(M, N, b_mn_major) & ~((1u << 7) | (1u << 10))
             : ajvp::idesc_bf16_f32(M, N, b_mn_major);
}

template <bool F16>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  return F16 ? Elem<__half>::pack(lo, hi) : ajvp::pack_bf16x2(lo, hi);
}

// D[tmem] (+)= P[tmem] V over one half of a tile's keys: P packed two keys to
// a column, 64 columns from a_tmem on; V a [128 keys x D] tile of 64-column
// chunks.
template <int D, int HALF>
__device__ __forceinline__ void mma_values_half(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_smem,
                                                uint32_t idesc, bool accumulate) {
  const uint64_t db = ajvp::smem_desc_sw128(b_smem, kTile * 128, 1024);
#pragma unroll
  for (int ks = 4 * HALF; ks < 4 * HALF + 4; ++ks)
    ajvp::umma_ts(d_tmem, a_tmem + 8 * ks, db + ((ks * 16 * 128) >> 4), idesc,
                  (accumulate || ks > 4 * HALF) ? 1u : 0u);
}

// 3-D tiled load, as tma_load_4d_hint.
__device__ __forceinline__ void tma_load_3d_hint(void* smem_dst, const void* map, uint64_t* bar,
                                                 int c0, int c1, int c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}

// Orders this thread's shared-memory stores before later reads of them by the
// tensor core or a bulk copy.
__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Scale the D sums of the warp's 32 rows, each by its lane's factor.
template <int D>
__device__ __forceinline__ void rescale_sums(uint32_t taddr, float f) {
  const float2 f2 = make_float2(f, f);
#pragma unroll 1  // seldom run: small
  for (int x = 0; x < D; x += 32) {
    uint32_t r[32];
    ajvp::tmem_ld32(taddr + x, r);
    ajvp::tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 y =
          __fmul2_rn(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), f2);
      r[j] = __float_as_uint(y.x);
      r[j + 1] = __float_as_uint(y.y);
    }
    ajvp::tmem_st32(taddr + x, r);
  }
  ajvp::tmem_wait_st();
}

// 64 scores of the lane's row.
__device__ __forceinline__ void load_scores(uint32_t taddr, uint32_t (&s)[64]) {
  ajvp::tmem_ld32(taddr, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
  ajvp::tmem_ld32(taddr + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
  ajvp::tmem_wait_ld();
}

// Largest of 128 scores.
__device__ __forceinline__ float max128(const uint32_t (&s)[kTile]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < kTile; j += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m[i] = ajvp::fmax3(m[i], __uint_as_float(s[j + 2 * i]), __uint_as_float(s[j + 2 * i + 1]));
  return fmaxf(ajvp::fmax3(m[0], m[1], m[2]), m[3]);
}

// 2^(s * sc - m) of 64 scores, packed in pairs, and their sum added to `sum`.
template <bool F16>
__device__ __forceinline__ void exp_half(const uint32_t* s, float2 sc, float m, uint32_t (&pk)[32],
                                         float2& sum) {
  const float base = m == -INFINITY ? 0.f : m;
  const float2 nb = make_float2(-base, -base);
  float2 other = make_float2(0.f, 0.f);
#pragma unroll
  for (int x = 0; x < 64; x += 4) {
    float2 a = __ffma2_rn(make_float2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), sc, nb);
    float2 c = __ffma2_rn(make_float2(__uint_as_float(s[x + 2]), __uint_as_float(s[x + 3])), sc, nb);
    a.x = ajvp::ex2_approx(a.x), a.y = ajvp::ex2_approx(a.y);
    c.x = ajvp::ex2_approx(c.x), c.y = ajvp::ex2_approx(c.y);
    sum = __fadd2_rn(sum, a);
    other = __fadd2_rn(other, c);
    pk[x / 2] = pack_pair<F16>(a.x, a.y);
    pk[x / 2 + 1] = pack_pair<F16>(c.x, c.y);
  }
  sum = __fadd2_rn(sum, other);
}

}  // namespace ajvp_serve
