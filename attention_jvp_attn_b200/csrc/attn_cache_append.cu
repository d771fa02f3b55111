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
// One block takes a (page that gets tokens, head, K or V) and some more: it alone
// reads and writes that page's codes and scale, so no atomics and no second
// launch are needed. Each thread holds its values in registers between the
// maximum and the rounding: one read of the input, one write of the codes.
// Bound by instructions and latency for prompts (32,800 tokens in pages of 16, 8
// heads, d = 128, 210 MB: 65 us, 3.2 TB/s, half of the copy rate; with one unit
// per block and 8 columns a thread 129 us), by the five reads one after the other
// for single tokens (64 sequences: 7.4 us).
#include "rope_slots.cuh"

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
  int T, B, heads, pages, table_width, n_positions;
  int d, half, half_layout;
};

// A block takes the new tokens of one page, for UN units (head, K or V) at
// once: the loads of all are in flight together behind one look-up of the
// page. PER: slots of 16 values of a unit per thread (rope_slots.cuh).
template <typename T, int D, int PER, int UN, int THREADS>
__global__ void __launch_bounds__(THREADS) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int per_row = D / 16;
  constexpr int page_tokens = PER * THREADS / per_row;
  __shared__ float red[UN][THREADS / 32];
  const int b = find_sequence(p.starts, p.B, p.T, page_tokens, 2, blockIdx.x);
  const int raw0 = p.starts[b], raw1 = p.starts[b + 1];
  const int old = p.cached[b];
  const int t0 = clamp_row(raw0, p.T), t1 = clamp_row(raw1, p.T);
  const int piece = static_cast<int>(blockIdx.x - (t0 / page_tokens + 2ll * b));
  if (threadIdx.x == 0 && (t0 != raw0 || t1 != raw1 || t1 < t0))
    atomicOr(p.status, kStatusBadIndex);
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
  const int unit0 = blockIdx.y * UN, units = 2 * p.heads;
  float x[UN][PER][16], amax[UN], before[UN];
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    const int which = unit0 + u >= p.heads ? 1 : 0, head = unit0 + u - which * p.heads;
    const bool has = unit0 + u < units;
    before[u] = 0.f;
    if (has && lo > 0) before[u] = p.scale[which][page * p.scale_page + head * p.scale_head];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int g = i * THREADS + threadIdx.x;
      const int row = g / per_row;
      float (&a)[8] = reinterpret_cast<float(&)[8]>(x[u][i][0]);
      float (&c)[8] = reinterpret_cast<float(&)[8]>(x[u][i][8]);
      if (has && row >= lo && row < hi) {
        const RopeSlot sl(g % per_row, which ? 0 : p.half, p.half_layout);
        const int64_t pos = first + row;
        load_slot(static_cast<const T*>(p.in[which]) + head * p.in_head[which] +
                      (t0 + pos - old) * p.in_token[which],
                  sl, a, c);
        if (sl.pair >= 0) {
          float co[8], si[8];
          load_turn(p.cos, p.sin, pos, p.half, sl, co, si);
          turn_slot(sl.split, a, c, co, si);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[u][i][j] = 0.f;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    amax[u] = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) amax[u] = fmaxf(amax[u], fabsf(x[u][i][j]));  // a NaN is passed over
    if (amax[u] == INFINITY) {  // once more, without infinities
      amax[u] = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float a = fabsf(x[u][i][j]);
          amax[u] = fmaxf(amax[u], a < INFINITY ? a : 0.f);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      amax[u] = fmaxf(amax[u], __shfl_xor_sync(0xffffffffu, amax[u], o));
    if ((threadIdx.x & 31) == 0) red[u][threadIdx.x >> 5] = amax[u];
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    if (unit0 + u >= units) break;
    const int which = unit0 + u >= p.heads ? 1 : 0, head = unit0 + u - which * p.heads;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) amax[u] = fmaxf(amax[u], red[u][w]);
    // amax = f 2^E with 1 <= f < 2, and 448 = 1.75 * 2^8 (a subnormal amax is
    // below the smallest scale anyway)
    const uint32_t bits = __float_as_uint(amax[u]);
    const int e = min(max(static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0),
                          kMinExp), kMaxExp);
    const float fresh = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    const float after = fmaxf(fresh, before[u]);
    const float inv = after == fresh ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 1.f / after;
    uint8_t* codes = p.codes[which] + page * p.page_stride + head * p.head_stride;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int g = i * THREADS + threadIdx.x;
      const int row = g / per_row;
      if (row >= hi) continue;
      const RopeSlot sl(g % per_row, which ? 0 : p.half, p.half_layout);
      uint8_t* at = codes + row * p.token_stride;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint2* to = reinterpret_cast<uint2*>(at + (k ? sl.c1 : sl.c0));
        if (row >= lo) {
          const float* y = &x[u][i][8 * k];
          uint2 r;
          r.x = e4m3x2(y[0] * inv, y[1] * inv) | (e4m3x2(y[2] * inv, y[3] * inv) << 16);
          r.y = e4m3x2(y[4] * inv, y[5] * inv) | (e4m3x2(y[6] * inv, y[7] * inv) << 16);
          *to = r;
        } else if (after != before[u]) {  // an earlier token, to the larger scale
          const float ratio = before[u] * inv;
          uint2 r = *to;
          uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float a, c, f, h;
            Elem<__half>::unpack(e4m3x2_to_f16x2(w[j] & 0xffffu), a, c);
            Elem<__half>::unpack(e4m3x2_to_f16x2(w[j] >> 16), f, h);
            w[j] = e4m3x2(a * ratio, c * ratio) | (e4m3x2(f * ratio, h * ratio) << 16);
          }
          *to = r;
        }
      }
    }
    if (threadIdx.x == 0) p.scale[which][page * p.scale_page + head * p.scale_head] = after;
  }
}

// 32 values a thread in flight (64 for the largest pages), whatever the page.
template <typename T, int D>
void append_launch(const AppendParams& p, int page_tokens, int pieces, cudaStream_t st) {
  constexpr int R = D / 64;  // 1 or 2
  auto grid = [&](int un) { return dim3(pieces, (2 * p.heads + un - 1) / un); };
  switch (page_tokens) {
    case 16: append_kernel<T, D, 1, 2, 64 * R><<<grid(2), 64 * R, 0, st>>>(p); break;
    case 32: append_kernel<T, D, 1, 2, 128 * R><<<grid(2), 128 * R, 0, st>>>(p); break;
    case 64: append_kernel<T, D, R, 2 / R, 256><<<grid(2 / R), 256, 0, st>>>(p); break;
    default: append_kernel<T, D, 2 * R, 1, 256><<<grid(1), 256, 0, st>>>(p); break;
  }
}

template <typename T>
void append_launch(const AppendParams& p, int page_tokens, int pieces, cudaStream_t st) {
  if (p.d == 128)
    append_launch<T, 128>(p, page_tokens, pieces, st);
  else
    append_launch<T, 64>(p, page_tokens, pieces, st);
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
  if (s.T < 0 || s.T > (int64_t(1) << 30) || s.Hkv < 1 || s.Hkv > 32767 || B < 0 || B > (1 << 20))
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  int rc = check_cache(cache, s.Hkv, s.d);
  if (rc != ATTN_JVP_OK) return rc;
  if (rope && (rc = check_tables(rope, s.d)) != ATTN_JVP_OK) return rc;
  if (table_width < 1 || table_width > (int64_t(1) << 30) || (B > 1 && table_stride < table_width))
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (s.T == 0 || B == 0) return ATTN_JVP_OK;
  if (!starts || !cached || !table) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (!aligned4(starts) || !aligned4(cached) || !aligned4(table)) return ATTN_JVP_ERR_MISALIGNED;
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
  p.d = static_cast<int>(s.d), p.heads = static_cast<int>(s.Hkv);
  const int page = static_cast<int>(cache->page_tokens);
  const int pieces = static_cast<int>(s.T / page + 2 * B);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s.dtype == ATTN_JVP_BF16)
    append_launch<__nv_bfloat16>(p, page, pieces, st);
  else if (s.dtype == ATTN_JVP_F16)
    append_launch<__half>(p, page, pieces, st);
  else
    append_launch<float>(p, page, pieces, st);
  return cudaGetLastError() == cudaSuccess ? ATTN_JVP_OK : ATTN_JVP_ERR_CUDA;
}
