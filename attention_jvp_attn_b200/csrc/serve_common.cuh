// serve_common.cuh - what the serving operators share: element types as 32-bit
// values, the checks of their arguments, the e4m3 conversions, and the search
// for the sequence that a piece of packed work belongs to.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <array>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "attn_jvp.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace ajvp_serve {

constexpr uint32_t kStatusBadIndex = 2u;  // bit of the device status word

// ---- host: argument checks ----
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A softmax scale (<= 0: the default), which the kernels take times log2 e.
constexpr float kLog2e = 1.4426950408889634f;
inline bool good_scale(float s) { return s <= 0.f || std::isfinite(s * kLog2e); }
inline float scale_log2(float s, int64_t d) {
  return (s > 0.f ? s : 1.0f / std::sqrt(static_cast<float>(d))) * kLog2e;
}

inline int dtype_bytes(int32_t dtype) {
  return dtype == ATTN_JVP_F32 ? 4 : (dtype == ATTN_JVP_BF16 || dtype == ATTN_JVP_F16) ? 2 : 0;
}

// A [rows, heads, d] array: pointer set and aligned, strides in whole 16 bytes.
// A stride that no second index uses is not looked at.
inline int check_rows(const void* p, attn_jvp_strides s, int64_t rows, int64_t heads, int bytes) {
  if (!p) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (!aligned16(p)) return ATTN_JVP_ERR_MISALIGNED;
  if ((rows > 1 && (s.token < 0 || s.token * bytes % 16)) ||
      (heads > 1 && (s.head < 0 || s.head * bytes % 16)))
    return ATTN_JVP_ERR_MISALIGNED;
  return ATTN_JVP_OK;
}

// The same for an input that tensor maps read: rows and heads may not be one
// and the same (a stride of 0).
inline int check_rows_map(const void* p, attn_jvp_strides s, int64_t rows, int64_t heads, int64_t d,
                          int bytes) {
  const int rc = check_rows(p, s, rows, heads, bytes);
  if (rc != ATTN_JVP_OK) return rc;
  return (rows > 1 && s.token < d) || (heads > 1 && s.head < d) ? ATTN_JVP_ERR_INVALID_ARGUMENT : ATTN_JVP_OK;
}

// The same for an output: rows and heads must not fall on one another.
inline int check_rows_out(const void* p, attn_jvp_strides s, int64_t rows, int64_t heads,
                          int64_t d, int bytes) {
  const int rc = check_rows(p, s, rows, heads, bytes);
  if (rc != ATTN_JVP_OK) return rc;
  const bool token_outside = (heads == 1 || s.head >= d) && (rows == 1 || s.token >= (heads - 1) * (heads > 1 ? s.head : 0) + d);
  const bool head_outside = (rows == 1 || s.token >= d) && (heads == 1 || s.head >= (rows - 1) * (rows > 1 ? s.token : 0) + d);
  return token_outside || head_outside ? ATTN_JVP_OK : ATTN_JVP_ERR_INVALID_ARGUMENT;
}

inline int check_tables(const attn_jvp_rope_tables* t, int64_t d) {
  if (!t) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (!t->cos || !t->sin || t->n_positions < 1 || t->n_positions > (int64_t(1) << 31) - 1)
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (!aligned16(t->cos) || !aligned16(t->sin)) return ATTN_JVP_ERR_MISALIGNED;
  if (t->rot < 16 || t->rot % 16 || t->rot > d) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (t->layout != ATTN_JVP_ROPE_INTERLEAVED && t->layout != ATTN_JVP_ROPE_HALF)
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  return ATTN_JVP_OK;
}

inline int check_cache(const attn_jvp_cache* c, int64_t Hkv, int64_t d) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (c->pages < 1 || c->pages > (int64_t(1) << 31) - 1) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
    return ATTN_JVP_ERR_UNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->k_scale) || !aligned4(c->v_scale))
    return ATTN_JVP_ERR_MISALIGNED;
  if (c->page_stride % 16 || c->head_stride % 16 || c->token_stride % 16)
    return ATTN_JVP_ERR_MISALIGNED;
  if (c->page_stride >= int64_t(1) << 32 || c->token_stride >= int64_t(1) << 32)
    return ATTN_JVP_ERR_UNSUPPORTED;  // far below what tensor maps take (2^40)
  if (c->token_stride < d || (Hkv > 1 && c->head_stride < d) || (c->pages > 1 && c->page_stride < d) ||
      (c->pages > 1 && c->scale_page_stride < 1) || (Hkv > 1 && c->scale_head_stride < 1))
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  return ATTN_JVP_OK;
}

// The running maximum m of a row's exponents (in powers of two) is kept kLead
// below the largest one at the time that it was raised, and raised again only
// when one exceeds it by more than kRaise, so that the sums are rarely rescaled.
// So probabilities 2^(t - m) are at most 2^15, which fp16 holds, and the row's
// largest is 2^kLead or more: fp16 rounds one by 2^-11 of itself, or by 2^-25,
// which is 2^-32 of the largest at most. At the largest itself (m = max t) the
// bits between 1 and 65,504 would lie idle and 2^-25 of the largest be lost.
constexpr float kLead = 7.f;
constexpr float kRaise = 15.f;

// Whether the elements of an array of `inner` adjacent ones, n[i] of them `stride[i]`
// apart in each of three dimensions, lie apart: each dimension steps over all that
// those of smaller strides span.
inline bool lie_apart(int64_t inner, std::array<int64_t, 3> n, std::array<int64_t, 3> stride) {
  std::array<int, 3> order = {0, 1, 2};
  std::sort(order.begin(), order.end(), [&](int a, int b) { return stride[a] < stride[b]; });
  __int128 span = inner;
  for (const int i : order) {
    if (n[i] <= 1) continue;
    if (stride[i] < span) return false;
    span += static_cast<__int128>(n[i] - 1) * stride[i];
  }
  return true;
}

// A cache that is written: no code or scale is another one's too.
inline bool writable(const attn_jvp_cache& c, int64_t Hkv, int64_t d) {
  return c.k != c.v && c.k_scale != c.v_scale &&
         lie_apart(d, {c.pages, Hkv, c.page_tokens}, {c.page_stride, c.head_stride, c.token_stride}) &&
         lie_apart(1, {c.pages, Hkv, 1}, {c.scale_page_stride, c.scale_head_stride, 0});
}

// Raises a kernel's shared-memory limit once per device (`done`: devices that
// have it; the kernel's own).
template <typename F>
cudaError_t allow_smem(F* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// ---- device: element types ----
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ void unpack(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return ajvp::pack_bf16x2(a, b);
  }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ void unpack(uint32_t w, float& a, float& b) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    a = f.x;
    b = f.y;
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// Eight adjacent elements as 32-bit values, and back.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    Elem<T>::unpack(u.x, x[0], x[1]);
    Elem<T>::unpack(u.y, x[2], x[3]);
    Elem<T>::unpack(u.z, x[4], x[5]);
    Elem<T>::unpack(u.w, x[6], x[7]);
  }
}
// The same eight elements as they lie in memory, and from there to 32 bits.
template <typename T>
struct Raw8 {
  uint4 u[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void unpack(float (&x)[8]) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        x[2 * i] = __uint_as_float(w[2 * i]);
        x[2 * i + 1] = __uint_as_float(w[2 * i + 1]);
      } else {
        Elem<T>::unpack(w[i], x[2 * i], x[2 * i + 1]);
      }
    }
  }
};
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(Elem<T>::pack(x[0], x[1]), Elem<T>::pack(x[2], x[3]),
                   Elem<T>::pack(x[4], x[5]), Elem<T>::pack(x[6], x[7]));
  }
}

__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
}

// ---- device: e4m3 ----
// Two values to two codes, to nearest even, beyond +-448 to the largest code.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two codes (the low 16 bits) to their values as an fp16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

// Four codes to their values as two fp16 pairs.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

// ---- device: page scales ----
constexpr float kMinScale = 9.094947017729282e-13f;  // 2^-40
constexpr float kMaxScale = 1.099511627776e12f;      // 2^40
__device__ __forceinline__ float read_scale(float s) {
  return fminf(fmaxf(s, kMinScale), kMaxScale);  // a NaN reads as the smallest
}

// The start of sequence b's rows in a packed array of T rows, from data that
// may be out of order: always in [0, T], so that no row outside is touched.
__device__ __forceinline__ int clamp_row(int start, int T) { return min(max(start, 0), T); }

// Work over packed sequences is cut into pieces of `unit` rows. Sequence b
// owns the pieces from starts[b] / unit + slack * b on: the next sequence's
// first piece lies at least rows / unit + slack further, which is enough for
// its rows however they straddle the pieces (slack = 1 for pieces that begin
// with the sequence, 2 for pieces that may begin inside a page). So a block
// finds its sequence without any scan of the lengths: by counting the first
// pieces at or before its own, in one round of loads for up to blockDim.x
// sequences, or by bisection if there are many more. Pieces that no sequence
// uses do nothing. Every thread of the block calls this; the result is the same
// in all of them. It relies on non-decreasing starts; others give some in-range
// sequence number.
__device__ __forceinline__ int find_sequence(const int32_t* starts, int B, int T, int unit,
                                             int slack, int piece) {
  auto at_or_before = [&](int b) {
    return clamp_row(starts[b], T) / unit + static_cast<int64_t>(slack) * b <= piece;
  };
  int before = 0;  // sequences whose first piece is at or before this one
  if (B <= 4 * static_cast<int>(blockDim.x)) {
    for (int b0 = 0; b0 < B; b0 += blockDim.x) {
      const int b = b0 + threadIdx.x;
      before += __syncthreads_count(b < B && at_or_before(b));
    }
  } else {
    for (int lo = 0, hi = B; lo < hi;) {
      const int mid = lo + (hi - lo) / 2;
      if (at_or_before(mid))
        before = lo = mid + 1;
      else
        hi = mid;
    }
  }
  return before > 0 ? before - 1 : 0;
}

}  // namespace ajvp_serve
