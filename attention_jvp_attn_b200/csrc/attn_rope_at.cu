// attn_rope_at.cu - rotary embedding of queries and keys at given positions
// (C ABI attn_jvp_rope_at): adjacent or half-split pairs, any leading part of
// the head, and the transposed rotation for the backward pass.
//
// The pages name RoPE before and after caching as the positional treatment of
// queries and keys (Causal-rCM summary page, section 3, "KV Cache"). With
// p = positions[t] and a pair (a, b) of columns:
//   a' = a cos[p] - b sin[p],   b' = a sin[p] + b cos[p]
// in 32 bits with the rounding of rope_rotate_pair, rounded once to the type.
// The matrix's transpose negates sin; a magnitude in the tables scales both.
//
// Bound by HBM: each value is read and written once, the tables' row once per
// token. A block takes whole tokens, so a thread keeps its columns' cosines
// and sines in registers over the heads that it turns.
#include "serve_common.cuh"
#include "rope_math.cuh"

namespace ajvp_serve {

constexpr int kRopeThreads = 256;

struct RopeAtParams {
  const void* in[2];  // q, k
  void* out[2];
  int64_t in_token[2], in_head[2], out_token[2], out_head[2];
  int heads[2];  // H, Hkv (0: no k)
  const void* positions;
  const float* cos;
  const float* sin;
  unsigned int* status;
  int64_t T;
  int n_positions;
  int d, half;  // head dim, rot / 2
  int wide;     // positions are 64-bit
  float sign;   // +1, or -1 for the transpose
};

// Column groups of a head: a group is 8 adjacent columns (interleaved pairs,
// or the columns behind the rotated part), or two times 8 columns half a
// rotation apart.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) rope_at_kernel(const __grid_constant__ RopeAtParams p) {
  const int turned = HALF ? p.half / 8 : p.half / 4;  // groups with a rotation
  const int groups = turned + (p.d - 2 * p.half) / 8;
  const int lanes = kRopeThreads / groups;            // heads in flight
  const int lane = threadIdx.x / groups, g = threadIdx.x - lane * groups;
  if (lane >= lanes) return;
  const int col = g < turned ? 8 * g : 2 * p.half + 8 * (g - turned);
  const int heads = p.heads[0] + p.heads[1];
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int64_t pos = p.wide ? static_cast<const int64_t*>(p.positions)[t]
                               : static_cast<const int32_t*>(p.positions)[t];
    if (pos < 0 || pos >= p.n_positions) {
      if (threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
      continue;
    }
    float c[8], s[8];
    if (g < turned) {
      const float* cp = p.cos + pos * p.half + (HALF ? col : col / 2);
      const float* sp = p.sin + pos * p.half + (HALF ? col : col / 2);
#pragma unroll
      for (int i = 0; i < (HALF ? 8 : 4); i += 4) {
        load4(cp + i, reinterpret_cast<float(&)[4]>(c[i]));
        load4(sp + i, reinterpret_cast<float(&)[4]>(s[i]));
      }
#pragma unroll
      for (int i = 0; i < (HALF ? 8 : 4); ++i) s[i] *= p.sign;
    }
    for (int h = lane; h < heads; h += lanes) {
      const int w = h < p.heads[0] ? 0 : 1, hh = w ? h - p.heads[0] : h;
      const T* src = static_cast<const T*>(p.in[w]) + t * p.in_token[w] + hh * p.in_head[w] + col;
      T* dst = static_cast<T*>(p.out[w]) + t * p.out_token[w] + hh * p.out_head[w] + col;
      float x[8];
      load8(src, x);
      if (HALF && g < turned) {
        float y[8];
        load8(src + p.half, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) ajvp::rope_rotate_pair(x[i], y[i], c[i], s[i]);
        store8(dst + p.half, y);
      } else if (!HALF && g < turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) ajvp::rope_rotate_pair(x[2 * i], x[2 * i + 1], c[i], s[i]);
      }
      store8(dst, x);
    }
  }
}

template <typename T>
void rope_at_launch(const RopeAtParams& p, int layout, int grid, cudaStream_t st) {
  if (layout == ATTN_JVP_ROPE_HALF)
    rope_at_kernel<T, true><<<grid, kRopeThreads, 0, st>>>(p);
  else
    rope_at_kernel<T, false><<<grid, kRopeThreads, 0, st>>>(p);
}

}  // namespace ajvp_serve

extern "C" int attn_jvp_rope_at(const attn_jvp_tokens* shape, const void* q,
                                attn_jvp_strides q_strides, const void* k,
                                attn_jvp_strides k_strides, const void* positions,
                                int32_t position_bytes, const attn_jvp_rope_tables* tables,
                                int32_t transpose, void* q_out, attn_jvp_strides q_out_strides,
                                void* k_out, attn_jvp_strides k_out_strides, void* stream) {
  using namespace ajvp_serve;
  if (!shape) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  const attn_jvp_tokens& s = *shape;
  const int bytes = dtype_bytes(s.dtype);
  if (!bytes || (s.d != 64 && s.d != 128)) return ATTN_JVP_ERR_UNSUPPORTED;
  if (s.T < 0 || s.H < 1 || s.H > 65535 || (k && (s.Hkv < 1 || s.Hkv > 65535)) ||
      (k == nullptr) != (k_out == nullptr) || (position_bytes != 4 && position_bytes != 8))
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  int rc = check_tables(tables, s.d);
  if (rc != ATTN_JVP_OK) return rc;
  if (s.T == 0) return ATTN_JVP_OK;
  if (!positions) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (reinterpret_cast<uintptr_t>(positions) % position_bytes) return ATTN_JVP_ERR_MISALIGNED;
  if ((rc = check_rows(q, q_strides, s.T, s.H, bytes)) != ATTN_JVP_OK ||
      (rc = check_rows_out(q_out, q_out_strides, s.T, s.H, s.d, bytes)) != ATTN_JVP_OK)
    return rc;
  if (k && ((rc = check_rows(k, k_strides, s.T, s.Hkv, bytes)) != ATTN_JVP_OK ||
            (rc = check_rows_out(k_out, k_out_strides, s.T, s.Hkv, s.d, bytes)) != ATTN_JVP_OK))
    return rc;
  RopeAtParams p;
  int sms = 0;
  rc = ajvp::device_status_word(&p.status, &sms);
  if (rc != ATTN_JVP_OK) return rc;
  p.in[0] = q, p.in[1] = k, p.out[0] = q_out, p.out[1] = k_out;
  p.in_token[0] = q_strides.token, p.in_head[0] = q_strides.head;
  p.in_token[1] = k_strides.token, p.in_head[1] = k_strides.head;
  p.out_token[0] = q_out_strides.token, p.out_head[0] = q_out_strides.head;
  p.out_token[1] = k_out_strides.token, p.out_head[1] = k_out_strides.head;
  p.heads[0] = static_cast<int>(s.H);
  p.heads[1] = k ? static_cast<int>(s.Hkv) : 0;
  p.positions = positions;
  p.wide = position_bytes == 8;
  p.cos = tables->cos, p.sin = tables->sin;
  p.n_positions = static_cast<int>(tables->n_positions);
  p.T = s.T;
  p.d = static_cast<int>(s.d);
  p.half = static_cast<int>(tables->rot / 2);
  p.sign = transpose ? -1.f : 1.f;
  const int64_t cap = int64_t(sms) * 8;
  const int grid = static_cast<int>(s.T < cap ? s.T : cap);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s.dtype == ATTN_JVP_BF16)
    rope_at_launch<__nv_bfloat16>(p, tables->layout, grid, st);
  else if (s.dtype == ATTN_JVP_F16)
    rope_at_launch<__half>(p, tables->layout, grid, st);
  else
    rope_at_launch<float>(p, tables->layout, grid, st);
  return cudaGetLastError() == cudaSuccess ? ATTN_JVP_OK : ATTN_JVP_ERR_CUDA;
}
