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
// maximum and the rounding: one read of the input, one write of the codes. Three
// reads depend on one another: the sequence, then its page beside the values and
// the tables' rows, then the page's scale.
// Bound by instructions and latency for prompts (32,800 tokens in pages of 16, 8
// heads, d = 128, 210 MB: 54 us, 3.9 TB/s, 59 % of the copy rate; 63 us with the
// values read after the page, 129 us with one unit per block and 8 columns a
// thread besides; fp32, 344 MB: 59 us), by the three reads for single tokens (64
// sequences: 2.9 us, fp32 3.2). A chunk of 1,560 tokens, 12 heads, pages of 64: 5.9
// us (fp32 8.4), some 624 blocks where 592 fit at once.
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

// What a block works on: new tokens [lo, hi) of a page, the page's first token
// being the sequence's token `first` and the packed rows' row from + first.
struct Part {
  int64_t first, from;
  int lo, hi;
  int page;    // not checked yet: its number may still be on its way
  bool known;  // the positions are in the tables
};

// Block blockIdx.x's part; false if it has none. The whole block calls this.
template <int THREADS>
__device__ __forceinline__ bool find_part(const AppendParams& p, int page_tokens, Part& part) {
  __shared__ int found[3];
  int b, raw0, raw1, old;
  if (p.B <= THREADS) {  // as find_sequence, with what belongs to the sequence in the same round of loads
    const int i = threadIdx.x;
    int s0 = 0, s1 = 0, c0 = 0;
    if (i < p.B) s0 = p.starts[i], s1 = p.starts[i + 1], c0 = p.cached[i];
    const bool at = i < p.B && clamp_row(s0, p.T) / page_tokens + 2 * i <= static_cast<int>(blockIdx.x);
    b = max(__syncthreads_count(at) - 1, 0);
    if (i == b) found[0] = s0, found[1] = s1, found[2] = c0;
    __syncthreads();
    raw0 = found[0], raw1 = found[1], old = found[2];
  } else {
    b = find_sequence(p.starts, p.B, p.T, page_tokens, 2, blockIdx.x);
    raw0 = p.starts[b], raw1 = p.starts[b + 1], old = p.cached[b];
  }
  const int t0 = clamp_row(raw0, p.T), t1 = clamp_row(raw1, p.T);
  const int piece = static_cast<int>(blockIdx.x - (t0 / page_tokens + 2ll * b));
  if (threadIdx.x == 0 && (t0 != raw0 || t1 != raw1 || t1 < t0 || (t1 > t0 && old < 0)))
    atomicOr(p.status, kStatusBadIndex);
  if (t1 <= t0 || piece < 0 || old < 0) return false;
  const int64_t index = int64_t(old / page_tokens) + piece;  // page of the sequence
  const int64_t end = int64_t(old) + (t1 - t0);              // tokens after the call
  part.first = index * page_tokens;
  if (part.first >= end) return false;
  part.from = int64_t(t0) - old;
  part.lo = static_cast<int>(part.first < old ? old - part.first : 0);
  part.hi = static_cast<int>(end - part.first < page_tokens ? end - part.first : page_tokens);
  part.known = !p.cos || part.first + part.hi <= p.n_positions;
  part.page = part.known && index < p.table_width ? p.table[b * p.table_stride + index] : -1;
  return true;
}

// Whether the part's page is one; else an error, and nothing is written.
__device__ __forceinline__ bool page_exists(const AppendParams& p, const Part& part) {
  if (part.page >= 0 && part.page < p.pages) return true;
  if (threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
  return false;
}

__device__ __forceinline__ float max_finite(const float* x, int n) {  // a NaN is passed over
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < n; ++j) top = fmaxf(top, fabsf(x[j]));
  if (top == INFINITY) {  // once more, without infinities
    top = 0.f;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float a = fabsf(x[j]);
      top = fmaxf(top, a < INFINITY ? a : 0.f);
    }
  }
  return top;
}

// A page's scale for new values up to amax, `before` being its scale where it
// `keeps` earlier tokens, and the scale's inverse. `before` becomes what it counts
// as (0 without such tokens), only here: looked at where it is loaded, it would be
// waited for there, 0.2 us before the maximum is found.
__device__ __forceinline__ void page_scale(float amax, bool keeps, float& before, float& after, float& inv) {
  before = keeps ? read_scale(before) : 0.f;
  // amax = f 2^E with 1 <= f < 2, and 448 = 1.75 * 2^8 (a subnormal amax is
  // below the smallest scale anyway)
  const uint32_t bits = __float_as_uint(amax);
  const int e = min(max(static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0),
                        kMinExp), kMaxExp);
  const float fresh = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  after = fmaxf(fresh, before);
  inv = after == fresh ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 1.f / after;
}

__device__ __forceinline__ void write8(uint8_t* to, const float* y, float inv) {
  uint2 r;
  r.x = e4m3x2(y[0] * inv, y[1] * inv) | (e4m3x2(y[2] * inv, y[3] * inv) << 16);
  r.y = e4m3x2(y[4] * inv, y[5] * inv) | (e4m3x2(y[6] * inv, y[7] * inv) << 16);
  *reinterpret_cast<uint2*>(to) = r;
}

// Eight codes of an earlier token, to a larger scale.
__device__ __forceinline__ void rescale8(uint8_t* to, float ratio) {
  uint2 r = *reinterpret_cast<uint2*>(to);
  uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float a, c, f, h;
    Elem<__half>::unpack(e4m3x2_to_f16x2(w[j] & 0xffffu), a, c);
    Elem<__half>::unpack(e4m3x2_to_f16x2(w[j] >> 16), f, h);
    w[j] = e4m3x2(a * ratio, c * ratio) | (e4m3x2(f * ratio, h * ratio) << 16);
  }
  *reinterpret_cast<uint2*>(to) = r;
}

// A block takes the new tokens of one page, for UN units (head, K or V) at
// once: the loads of all are in flight together, beside the look-up of the
// page. PER: slots of 16 values of a unit per thread (rope_slots.cuh). 64
// registers up to two slots of 16-bit values, for the blocks in flight.
template <typename T, int D, int PER, int UN, int THREADS>
__global__ void __launch_bounds__(THREADS, PER * sizeof(T) <= 4 ? 1024 / THREADS : 1)
    append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int per_row = D / 16;
  constexpr int page_tokens = PER * THREADS / per_row;
  __shared__ float red[UN][THREADS / 32];
  Part part;
  if (!find_part<THREADS>(p, page_tokens, part)) return;
  const int lo = part.lo, hi = part.hi;
  const int unit0 = blockIdx.y * UN, units = 2 * p.heads;
  Raw8<T> ra[UN][PER], rb[UN][PER];
  float co[PER][8], si[PER][8];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int g = i * THREADS + threadIdx.x, row = g / per_row;
    const bool fresh = part.known && row >= lo && row < hi;
    const int64_t pos = part.first + row;
    const RopeSlot sl(g % per_row, p.half, p.half_layout);
    if (fresh && sl.pair >= 0 && unit0 < p.heads) load_turn(p.cos, p.sin, pos, p.half, sl, co[i], si[i]);
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int which = unit0 + u >= p.heads ? 1 : 0, head = unit0 + u - which * p.heads;
      ra[u][i] = {}, rb[u][i] = {};
      if (fresh && unit0 + u < units) {
        const RopeSlot at(g % per_row, which ? 0 : p.half, p.half_layout);
        const T* src = static_cast<const T*>(p.in[which]) + head * p.in_head[which] +
                       (part.from + pos) * p.in_token[which];
        ra[u][i].load(src + at.c0);
        rb[u][i].load(src + at.c1);
      }
    }
  }
  if (!page_exists(p, part)) return;
  const int64_t page = part.page;
  float x[UN][PER][16], amax[UN], before[UN];
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    const int which = unit0 + u >= p.heads ? 1 : 0, head = unit0 + u - which * p.heads;
    before[u] = 0.f;
    if (unit0 + u < units && lo > 0) before[u] = p.scale[which][page * p.scale_page + head * p.scale_head];
  }
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    const bool key = unit0 + u < p.heads;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int g = i * THREADS + threadIdx.x, row = g / per_row;
      const RopeSlot sl(g % per_row, p.half, p.half_layout);
      float (&a)[8] = reinterpret_cast<float(&)[8]>(x[u][i][0]);
      float (&c)[8] = reinterpret_cast<float(&)[8]>(x[u][i][8]);
      ra[u][i].unpack(a);
      rb[u][i].unpack(c);
      if (key && sl.pair >= 0 && row >= lo && row < hi) turn_slot(sl.split, a, c, co[i], si[i]);
    }
  }
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    amax[u] = max_finite(&x[u][0][0], PER * 16);
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
    float after, inv;
    page_scale(amax[u], lo > 0, before[u], after, inv);
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
        uint8_t* to = at + (k ? sl.c1 : sl.c0);
        if (row >= lo)
          write8(to, &x[u][i][8 * k], inv);
        else if (after != before[u])
          rescale8(to, before[u] * inv);
      }
    }
    if (threadIdx.x == 0) p.scale[which][page * p.scale_page + head * p.scale_head] = after;
  }
}

// The same for calls with few new tokens per sequence: a warp takes a unit, and
// rounds of 32 slots of the new tokens only (the first stays in registers, any
// further ones are read twice).
constexpr int kFewWarps = 8;
template <typename T, int D>
__global__ void __launch_bounds__(kFewWarps * 32)
    append_few_kernel(const __grid_constant__ AppendParams p, const int page_tokens) {
  constexpr int per_row = D / 16, STEP = 32 / per_row;
  Part part;
  if (!find_part<kFewWarps * 32>(p, page_tokens, part)) return;
  const int lane = threadIdx.x & 31, sub = lane / per_row;
  const int unit = blockIdx.y * kFewWarps + (threadIdx.x >> 5);
  const bool has = unit < 2 * p.heads;
  const int which = unit >= p.heads ? 1 : 0, head = unit - which * p.heads;
  const RopeSlot sl(lane % per_row, which ? 0 : p.half, p.half_layout);
  const T* src = static_cast<const T*>(p.in[which]) + head * p.in_head[which];
  Raw8<T> ra = {}, rb = {};
  float co[8], si[8];
  auto load = [&](int row) {
    const int64_t pos = part.first + row;
    if (sl.pair >= 0) load_turn(p.cos, p.sin, pos, p.half, sl, co, si);
    ra.load(src + (part.from + pos) * p.in_token[which] + sl.c0);
    rb.load(src + (part.from + pos) * p.in_token[which] + sl.c1);
  };
  auto value = [&](float (&y)[16]) {
    float (&a)[8] = reinterpret_cast<float(&)[8]>(y[0]);
    float (&c)[8] = reinterpret_cast<float(&)[8]>(y[8]);
    ra.unpack(a);
    rb.unpack(c);
    if (sl.pair >= 0) turn_slot(sl.split, a, c, co, si);
  };
  const int row0 = part.lo + sub;
  const bool mine = has && part.known && row0 < part.hi;
  if (mine) load(row0);
  if (!page_exists(p, part) || !has) return;
  float* scale = p.scale[which] + part.page * p.scale_page + head * p.scale_head;
  float before = part.lo > 0 ? *scale : 0.f;
  float x[16], amax = 0.f;
  if (mine) {
    value(x);
    amax = max_finite(x, 16);
    for (int row = row0 + STEP; row < part.hi; row += STEP) {
      float y[16];
      load(row);
      value(y);
      amax = fmaxf(amax, max_finite(y, 16));
    }
  }
  __syncwarp();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  float after, inv;
  page_scale(amax, part.lo > 0, before, after, inv);
  uint8_t* codes = p.codes[which] + part.page * p.page_stride + head * p.head_stride;
  if (mine) {
    write8(codes + row0 * p.token_stride + sl.c0, x, inv);
    write8(codes + row0 * p.token_stride + sl.c1, x + 8, inv);
    for (int row = row0 + STEP; row < part.hi; row += STEP) {
      load(row);
      value(x);
      write8(codes + row * p.token_stride + sl.c0, x, inv);
      write8(codes + row * p.token_stride + sl.c1, x + 8, inv);
    }
  }
  if (after != before)
    for (int row = sub; row < part.lo; row += STEP) {
      rescale8(codes + row * p.token_stride + sl.c0, before * inv);
      rescale8(codes + row * p.token_stride + sl.c1, before * inv);
    }
  if (lane == 0) *scale = after;
}

// New tokens per sequence, on average, up to which a warp takes a unit: one round
// of it at d = 128. us, a warp / a block per unit, d = 128, 8 heads, new tokens of
// each sequence:
//   64 sequences, pages of 64:   1: 2.9 / 7.4   4: 3.0 / 7.8   8: 4.2 / 8.3   32: 9.2 / 10.4
//   500 sequences, pages of 32:  1: 13 / 30     4: 14 / 33     8: 18 / 35     32: 51 / 58
//   1 sequence, pages of 64:     1: 2.6 / 2.6   4: 2.7 / 2.7   8: 3.4 / 2.6   32: 7.4 / 2.7
// Beyond it one long sequence would wait for its rounds. The mean decides, as the
// host knows no lengths, so a chunk among single tokens may have to do just that, in
// up to 32 rounds a page: sequences of one token and one of n, 8 heads, d = 128, us:
//   pages of 16:   63 + one of 190: 4.8 / 4.0     255 + one of 760: 8.1 / 10.6   1,023 + one of 3,000: 36 / 49
//   pages of 64:   63 + one of 190: 9.5 / 7.8     255 + one of 760: 14 / 24      1,023 + one of 3,000: 35 / 121
//   pages of 128:  63 + one of 190: 16 / 12       255 + one of 760: 24 / 40      1,023 + one of 3,000: 45 / 208
constexpr int kFewTokens = 4;

// 32 values a thread in flight (64 for the largest pages), whatever the page.
template <typename T, int D>
void append_launch(const AppendParams& p, int page_tokens, int pieces, cudaStream_t st) {
  constexpr int R = D / 64;  // 1 or 2
  if (p.T <= int64_t(kFewTokens) * p.B) {
    append_few_kernel<T, D><<<dim3(pieces, (2 * p.heads + kFewWarps - 1) / kFewWarps), kFewWarps * 32, 0, st>>>(
        p, page_tokens);
    return;
  }
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
  if (!writable(*cache, s.Hkv, s.d)) return ATTN_JVP_ERR_INVALID_ARGUMENT;
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
