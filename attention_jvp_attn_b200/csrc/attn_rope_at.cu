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
// Bound by HBM: each value is read and written once; the tables' row of a token
// comes from L1 or L2 for all heads but the first. The position, then the
// table's row, are two reads one after the other, so many warps are wanted; and
// a thread keeps its columns' cosines and sines over its heads. Three blocks per
// SM, so 80 registers, spill 20 to 28 bytes a thread (fp32: 76 to 104). Measured (one
// B200): 32,760 tokens of 24 heads, d = 128, bf16, 419 MB: 75 to 77 us, 5.44 TB/s, 83
// % of the copy rate (half layout: 73); with 8 columns of one head a thread 104 us
// (126 instructions per 8 values), with a block per token that walks on to the next
// 107 us. fp32, 822 MB: 155 us, 5.3 TB/s (half layout, whose runs of 8 columns a warp
// reads side by side: 128 us, 6.4 TB/s). 64 tokens of 40 heads: 3.0 us (fp32 4.6).
#include "rope_slots.cuh"

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
  int parts;    // warps that share a token's heads
  float sign;   // +1, or -1 for the transpose
};

// A warp takes heads [n part / parts, n (part + 1) / parts) of q, then of k, of
// one token: a lane takes a slot of 16 columns (rope_slots.cuh) of every
// (32 / slots)-th head, two heads' loads in flight at a time. The first loads
// go out before the position's and the table's, which wait for one another.
template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_at_kernel(const __grid_constant__ RopeAtParams p) {
  constexpr int SLOTS = D / 16, STEP = 32 / SLOTS, U = 2;
  const int lane = threadIdx.x & 31;
  const int64_t warp = int64_t(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = warp / p.parts;
  if (t >= p.T) return;
  const int part = static_cast<int>(warp - t * p.parts);
  const RopeSlot sl(lane % SLOTS, p.half, HALF);
  const int sub = lane / SLOTS;
  const int64_t pos = p.wide ? static_cast<const int64_t*>(p.positions)[t]
                             : static_cast<const int32_t*>(p.positions)[t];
  float c[8], s[8];
  bool ready = false, good = true;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int hi = p.heads[w] * (part + 1) / p.parts;
    int h = p.heads[w] * part / p.parts + sub;
    const T* src = static_cast<const T*>(p.in[w]) + t * p.in_token[w] + h * p.in_head[w];
    T* dst = static_cast<T*>(p.out[w]) + t * p.out_token[w] + h * p.out_head[w];
    const int64_t in_step = STEP * p.in_head[w], out_step = STEP * p.out_head[w];
    for (; h < hi; h += U * STEP) {
      Raw8<T> ra[U], rb[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * STEP < hi) {
          ra[u].load(src + u * in_step + sl.c0);
          rb[u].load(src + u * in_step + sl.c1);
        }
      if (!ready) {
        ready = true;
        good = pos >= 0 && pos < p.n_positions;
        if (good && sl.pair >= 0) {
          load_turn(p.cos, p.sin, pos, p.half, sl, c, s);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] *= p.sign;
        }
      }
      if (!good) break;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * STEP < hi) {
          float a[8], b[8];
          ra[u].unpack(a);
          rb[u].unpack(b);
          if (sl.pair >= 0) turn_slot(HALF, a, b, c, s);  // a rotated slot is split in the half layout
          store8(dst + u * out_step + sl.c0, a);
          store8(dst + u * out_step + sl.c1, b);
        }
      src += U * in_step;
      dst += U * out_step;
    }
  }
  if (!good && sub == 0) atomicOr(p.status, kStatusBadIndex);
}

template <typename T>
void rope_at_launch(RopeAtParams& p, bool half_layout, int sms, cudaStream_t st) {
  // Warps of a token: one, so that the position and the table's row are read
  // once, unless the tokens are too few to fill the SMs.
  const int slots = p.d / 16, batch = 2 * (32 / slots);  // heads of about a round
  const int rounds = (p.heads[0] + batch - 1) / batch;
  const int64_t want = (int64_t(sms) * 32 + p.T - 1) / p.T;
  p.parts = static_cast<int>(want < rounds ? want : rounds);
  const int64_t warps = p.T * p.parts, per = kRopeThreads / 32;
  const unsigned blocks = static_cast<unsigned>((warps + per - 1) / per);
  if (p.d == 128)
    (half_layout ? rope_at_kernel<T, 128, true> : rope_at_kernel<T, 128, false>)<<<blocks, kRopeThreads, 0, st>>>(p);
  else
    (half_layout ? rope_at_kernel<T, 64, true> : rope_at_kernel<T, 64, false>)<<<blocks, kRopeThreads, 0, st>>>(p);
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
  if (s.T < 0 || s.T > (int64_t(1) << 31) - 1 || s.H < 1 || s.H > 65535 || (k && (s.Hkv < 1 || s.Hkv > 65535)) ||
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
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s.dtype == ATTN_JVP_BF16)
    rope_at_launch<__nv_bfloat16>(p, tables->layout == ATTN_JVP_ROPE_HALF, sms, st);
  else if (s.dtype == ATTN_JVP_F16)
    rope_at_launch<__half>(p, tables->layout == ATTN_JVP_ROPE_HALF, sms, st);
  else
    rope_at_launch<float>(p, tables->layout == ATTN_JVP_ROPE_HALF, sms, st);
  return cudaGetLastError() == cudaSuccess ? ATTN_JVP_OK : ATTN_JVP_ERR_CUDA;
}
