// attn_cache_append.cu - appending keys and values to a paged e4m3 cache, the
// keys rotated on the way (C ABI attn_jvp_cache_append).
//
// The pages describe an append mode of the key-value cache with keys cached
// after RoPE (Causal-rCM summary page, section 3, "KV Cache"); they give no
// format. Here a page and head has one scale 2^e with
//   e = min{ e : |x| <= 448 * 2^e for its finite values x }, -32 <= e <= 32.
// A power of two makes code = round(x / 2^e) one rounding from fp32, makes
// code * 2^e exact, and lets a page whose scale grows be rounded to the new
// scale without any error but for subnormal codes. It costs no precision, as
// e4m3 is a floating-point format; a free scale would gain at most one bit of
// range at its lower end.
//
// One block per (page that gets tokens, head, K or V): it alone reads and
// writes that page's codes and scale, so no atomics and no second launch are
// needed. Each thread holds its values in registers between the maximum and
// the rounding: one read of the input, one write of the codes. Bound by HBM
// for prompts, by latency for single tokens.
#include "serve_common.cuh"
#include "rope_math.cuh"

namespace ajvp_serve {

constexpr int kMinExp = -32, kMaxExp = 32;

struct AppendParams {
  const void* in[2];  // k, v
  int64_t in_token[2], in_head[2];
  uint8_t* codes[2];
  float* scale[2];
  int64_t page_stride, head_stride, token_stride, scale_page, scale_head;
  const int32_t* starts;
  const int32_t* cached;
  const int32_t* table;
  int64_t table_stride;
  const float* cos;  // null: no rotation
  const float* sin;
  unsigned int* status;
  int T, B, pages, table_width, n_positions;
  int d, half, half_layout;
};

// Eight rotated (K) or plain (V) values of one token's head, at column col.
template <typename T>
__device__ __forceinline__ void append_values(const AppendParams& p, const T* row, int col, bool turn,
                                              int64_t pos, float (&x)[8]) {
  load8(row + col, x);
  if (!turn || col >= 2 * p.half) return;
  const float* cp = p.cos + pos * p.half;
  const float* sp = p.sin + pos * p.half;
  if (!p.half_layout) {
    float c[4], s[4];
    load4(cp + col / 2, c);
    load4(sp + col / 2, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) ajvp::rope_rotate_pair(x[2 * i], x[2 * i + 1], c[i], s[i]);
    return;
  }
  // The other half of each pair is read too (by the thread that owns it as
  // well: from L1), and the half of the result that belongs here is kept.
  const bool upper = col >= p.half;
  const int at = upper ? col - p.half : col;
  float y[8], c[8], s[8];
  load8(row + (upper ? at : at + p.half), y);
  load4(cp + at, reinterpret_cast<float(&)[4]>(c[0]));
  load4(cp + at + 4, reinterpret_cast<float(&)[4]>(c[4]));
  load4(sp + at, reinterpret_cast<float(&)[4]>(s[0]));
  load4(sp + at + 4, reinterpret_cast<float(&)[4]>(s[4]));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a = upper ? y[i] : x[i], b = upper ? x[i] : y[i];
    ajvp::rope_rotate_pair(a, b, c[i], s[i]);
    x[i] = upper ? b : a;
  }
}

// PER: groups of 8 values per thread, page_tokens * d / 8 / THREADS.
template <typename T, int PER, int THREADS>
__global__ void __launch_bounds__(THREADS) append_kernel(const __grid_constant__ AppendParams p,
                                                         const int page_tokens) {
  __shared__ float red[THREADS / 32];
  const int which = blockIdx.z, head = blockIdx.y;
  const int b = find_sequence(p.starts, p.B, p.T, page_tokens, 2, blockIdx.x);
  const int raw0 = p.starts[b], raw1 = p.starts[b + 1];
  const int t0 = clamp_row(raw0, p.T), t1 = clamp_row(raw1, p.T);
  const int piece = static_cast<int>(blockIdx.x - (t0 / page_tokens + 2ll * b));
  if (threadIdx.x == 0 && (t0 != raw0 || t1 != raw1 || t1 < t0))
    atomicOr(p.status, kStatusBadIndex);
  const int old = p.cached[b];
  if (t1 <= t0 || piece < 0) return;
  if (old < 0) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
    return;
  }
  const int64_t index = int64_t(old / page_tokens) + piece;  // page of the sequence
  const int64_t first = index * page_tokens;                 // its first token
  const int64_t end = int64_t(old) + (t1 - t0);              // tokens after the call
  if (first >= end) return;
  const int lo = static_cast<int>(first < old ? old - first : 0);
  const int hi = static_cast<int>(end - first < page_tokens ? end - first : page_tokens);
  const int page = index < p.table_width ? p.table[b * p.table_stride + index] : -1;
  if (page < 0 || page >= p.pages || (p.cos && first + hi > p.n_positions)) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
    return;
  }
  const T* in = static_cast<const T*>(p.in[which]) + head * p.in_head[which];
  uint8_t* codes = p.codes[which] + page * p.page_stride + head * p.head_stride;
  float* scale = p.scale[which] + page * p.scale_page + head * p.scale_head;
  const float before = lo > 0 ? *scale : 0.f;
  const int per_row = p.d / 8;
  float x[PER][8];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int g = i * THREADS + threadIdx.x;
    const int row = g / per_row, col = (g - row * per_row) * 8;
    if (row >= lo && row < hi) {
      const int64_t pos = first + row;
      append_values(p, in + (t0 + pos - old) * p.in_token[which], col, which == 0 && p.cos, pos,
                    x[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = fabsf(x[i][j]);
        amax = fmaxf(amax, a < INFINITY ? a : 0.f);  // a NaN compares false
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) amax = fmaxf(amax, red[w]);
  // amax = m 2^e with 0.5 <= m < 1, and 448 = 0.875 * 2^9
  int e = kMinExp;
  if (amax > 0.f) {
    const float m = frexpf(amax, &e);
    e = min(max(e - 9 + (m > 0.875f ? 1 : 0), kMinExp), kMaxExp);
  }
  const float fresh = ldexpf(1.f, e);
  const float after = fmaxf(fresh, before);
  const float inv = 1.f / after;  // exact for powers of two
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int g = i * THREADS + threadIdx.x;
    const int row = g / per_row, col = (g - row * per_row) * 8;
    if (row >= hi) continue;
    uint2* at = reinterpret_cast<uint2*>(codes + row * p.token_stride + col);
    if (row >= lo) {
      uint2 r;
      r.x = e4m3x2(x[i][0] * inv, x[i][1] * inv) | (e4m3x2(x[i][2] * inv, x[i][3] * inv) << 16);
      r.y = e4m3x2(x[i][4] * inv, x[i][5] * inv) | (e4m3x2(x[i][6] * inv, x[i][7] * inv) << 16);
      *at = r;
    } else if (after != before) {  // an earlier token, to the larger scale
      const float ratio = before * inv;
      uint2 r = *at;
      uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float a, c, f, h;
        Elem<__half>::unpack(e4m3x2_to_f16x2(w[j] & 0xffffu), a, c);
        Elem<__half>::unpack(e4m3x2_to_f16x2(w[j] >> 16), f, h);
        w[j] = e4m3x2(a * ratio, c * ratio) | (e4m3x2(f * ratio, h * ratio) << 16);
      }
      *at = r;
    }
  }
  if (threadIdx.x == 0) *scale = after;
}

// A page's values over the block: 8 values a thread (128 to 256 threads) up
// to pages of 2048 values, then more per thread.
template <typename T>
void append_launch(const AppendParams& p, int page_tokens, dim3 grid, cudaStream_t st) {
  switch (page_tokens * p.d / 8) {
    case 128: append_kernel<T, 1, 128><<<grid, 128, 0, st>>>(p, page_tokens); break;
    case 256: append_kernel<T, 1, 256><<<grid, 256, 0, st>>>(p, page_tokens); break;
    case 512: append_kernel<T, 2, 256><<<grid, 256, 0, st>>>(p, page_tokens); break;
    case 1024: append_kernel<T, 4, 256><<<grid, 256, 0, st>>>(p, page_tokens); break;
    default: append_kernel<T, 8, 256><<<grid, 256, 0, st>>>(p, page_tokens); break;
  }
}

}  // namespace ajvp_serve

extern "C" int attn_jvp_cache_append(const attn_jvp_tokens* shape, const void* k,
                                     attn_jvp_strides k_strides, const void* v,
                                     attn_jvp_strides v_strides, const attn_jvp_cache* cache,
                                     int64_t B, const int32_t* starts, const int32_t* cached,
                                     const int32_t* table, int64_t table_width,
                                     int64_t table_stride, const attn_jvp_rope_tables* rope,
                                     void* stream) {
  using namespace ajvp_serve;
  if (!shape) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  const attn_jvp_tokens& s = *shape;
  const int bytes = dtype_bytes(s.dtype);
  if (!bytes || (s.d != 64 && s.d != 128)) return ATTN_JVP_ERR_UNSUPPORTED;
  if (s.T < 0 || s.T > (int64_t(1) << 30) || s.Hkv < 1 || s.Hkv > 65535 || B < 0 || B > (1 << 20))
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  int rc = check_cache(cache, s.Hkv, s.d);
  if (rc != ATTN_JVP_OK) return rc;
  if (rope && (rc = check_tables(rope, s.d)) != ATTN_JVP_OK) return rc;
  if (table_width < 1 || table_width > (int64_t(1) << 30) || (B > 1 && table_stride < table_width))
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (s.T == 0 || B == 0) return ATTN_JVP_OK;
  if (!starts || !cached || !table) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if ((rc = check_rows(k, k_strides, s.T, s.Hkv, bytes)) != ATTN_JVP_OK ||
      (rc = check_rows(v, v_strides, s.T, s.Hkv, bytes)) != ATTN_JVP_OK)
    return rc;
  AppendParams p;
  rc = ajvp::device_status_word(&p.status);
  if (rc != ATTN_JVP_OK) return rc;
  p.in[0] = k, p.in[1] = v;
  p.in_token[0] = k_strides.token, p.in_head[0] = k_strides.head;
  p.in_token[1] = v_strides.token, p.in_head[1] = v_strides.head;
  p.codes[0] = static_cast<uint8_t*>(cache->k), p.codes[1] = static_cast<uint8_t*>(cache->v);
  p.scale[0] = cache->k_scale, p.scale[1] = cache->v_scale;
  p.page_stride = cache->page_stride, p.head_stride = cache->head_stride;
  p.token_stride = cache->token_stride;
  p.scale_page = cache->scale_page_stride, p.scale_head = cache->scale_head_stride;
  p.starts = starts, p.cached = cached, p.table = table, p.table_stride = table_stride;
  p.cos = rope ? rope->cos : nullptr, p.sin = rope ? rope->sin : nullptr;
  p.n_positions = rope ? static_cast<int>(rope->n_positions) : 0;
  p.half = rope ? static_cast<int>(rope->rot / 2) : 0;
  p.half_layout = rope && rope->layout == ATTN_JVP_ROPE_HALF;
  p.T = static_cast<int>(s.T), p.B = static_cast<int>(B);
  p.pages = static_cast<int>(cache->pages), p.table_width = static_cast<int>(table_width);
  p.d = static_cast<int>(s.d);
  const int page = static_cast<int>(cache->page_tokens);
  const dim3 grid(static_cast<unsigned>(s.T / page + 2 * B), static_cast<unsigned>(s.Hkv), 2);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s.dtype == ATTN_JVP_BF16)
    append_launch<__nv_bfloat16>(p, page, grid, st);
  else if (s.dtype == ATTN_JVP_F16)
    append_launch<__half>(p, page, grid, st);
  else
    append_launch<float>(p, page, grid, st);
  return cudaGetLastError() == cudaSuccess ? ATTN_JVP_OK : ATTN_JVP_ERR_CUDA;
}
