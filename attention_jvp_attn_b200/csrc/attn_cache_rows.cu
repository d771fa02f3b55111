// attn_cache_rows.cu - attention of a few query rows over the paged e4m3 cache
// (C ABI attn_jvp_cache_attn): single tokens and short runs of tokens.
//
// For each row, over the keys that it sees, with code values k_j, v_j and the
// page scales a_j, b_j:
//   x_j = s a_j <q, k_j>,  O = sum_j e^(x_j) b_j v_j / sum_j e^(x_j)
// One pass with a running maximum, in powers of two. The value scale goes into
// the exponent: with t_j = x_j log2 e + log2 b_j and m near max t_j (kLead),
//   p_j = 2^(t_j - m),  O = sum_j p_j v_j / sum_j p_j / b_j,
// so p is at most 2^kRaise however the scales differ. What fp16 takes from a p_j,
// 2^-11 of it or 2^-32 of the row's largest p, is small against the largest e^x b,
// a bound on a contribution to O, not a contribution: where the page of the
// largest holds codes near 0 (one token of the page is far larger than the others)
// and the other pages' scales are below some 2^-20 of its own, O is made of
// probabilities of few bits. The sum of p / b is of the unrounded ones.
//
// Bound by HBM: a cached token is 2 d bytes per key head, read once; the rows
// (all query heads of the key head, and the newest tokens) share it. Codes are
// exact in fp16, so both products run on m16n8k16 fp16 matrix instructions
// with fp32 sums; bf16 queries are scaled by a power of two per row into fp16
// (exact within 2^-14 of the row's largest, absolute error 2^-25 of it below).
// Tokens are the instruction's 16 rows and query rows its 8 columns
// (S^T = K Q^T, O^T = V^T P^T), so 8 query rows cost no padding and each code
// is converted once however many query rows there are; 128-row tensor-memory
// tiles would be mostly empty here.
//
// Layout: each warp streams its own steps of 32 tokens through a private ring
// of TMA copies (no block-wide barrier in the loop), so a stall of one warp
// holds up no other. The order of the head dimension inside the products is
// free, so a lane takes 16 adjacent codes at a time for four matrix
// instructions, and the column order of O lets a lane own adjacent columns: no
// shared-memory transposes.
//
// The key axis is split in one of two ways, both with a fixed order of sums:
//   - short sequences: over the blocks of a cluster, which join their sums
//     through distributed shared memory. One launch, which counts there;
//   - long ones: all steps of all sequences and heads in a row are shared out
//     evenly to as many blocks as fit at once, so sequences of any lengths
//     load the SMs evenly. A block's first and last pieces may be parts of a
//     sequence; their sums go to the workspace, and a second, small kernel
//     joins them.
// Measured (one B200, d = 128): 64 sequences of 500 to 8,192 tokens, 32 query and 8
// key heads, 586 MB: 112 us, 5.2 TB/s, 80 % of the copy rate (query rows as the
// instruction's rows, codes copied by the lanes: 241 us); 3 sequences of 40,000 to
// 131,072 tokens, 16 rows, 592 MB: 133 us, 4.4 TB/s.
#include <cuda.h>

#include "serve_attn.cuh"

#include <type_traits>

namespace ajvp_serve {

namespace {

constexpr int kRowsWarps = 4;
constexpr int kStep = 32;                  // tokens per step of a warp
constexpr int kMostSplits = 8;             // blocks of a cluster
constexpr int kLeastSteps = 8;             // steps of a block: two of a warp
constexpr uint32_t kHidden = 0xffffffffu;  // in place of a key scale: no page there

struct RowsParams {
  CUtensorMap map_k, map_v;  // codes (d, page tokens, heads, pages), boxes of d x box tokens
  CacheAttnParams c;
  int box;      // 16 or 32 tokens, one page's
  float* work;  // sums of partial pieces, two places per block; null: clusters
};

template <int D, int NT>
struct RowsCfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int STAGES = NT == 1 ? 2 : 3;
  static constexpr int KV = kStep * D;                // bytes of a step's keys (or values)
  static constexpr int RING = STAGES * 2 * KV;        // per warp
  static constexpr int PITCH = D + 4;                 // floats per row of a warp's sums
  static constexpr int PART = ROWS * PITCH * 4;
  static constexpr int SLOT = RING;                   // the sums lie over the ring
  static constexpr int SCALES = STAGES * 8 * 4;       // per warp: see `scales` below
  static constexpr int AT_WHOLE = kRowsWarps * SLOT;  // the block's sums
  static constexpr int AT_STATS = AT_WHOLE + PART;
  static constexpr int AT_SCALES = AT_STATS + (2 * kRowsWarps + 2) * ROWS * 4;
  static constexpr int AT_BARS = AT_SCALES + kRowsWarps * SCALES;
  static constexpr int BYTES = 1024 + AT_BARS + kRowsWarps * STAGES * 8 + 16;
  static_assert(PART <= SLOT && SLOT % 1024 == 0 && AT_BARS % 8 == 0, "layout");
  // a place of the workspace: the block's sums, then maxima and sums of p
  static constexpr int PLACE = ROWS * (D + 2);
};

// Steps of a sequence of which `reach` tokens are seen; one without tokens
// takes a step of its own, in which its empty rows are written.
__device__ __forceinline__ int steps_of(int reach) { return max((reach + kStep - 1) / kStep, 1); }

// Tokens that the last of sequence b's new ones sees (all of them: rows <= 16).
__device__ __forceinline__ int reach_of(const CacheAttnParams& p, int b) {
  return checked_len(p, b);
}

// A lane's place in the instruction: g = lane / 4 its token (or column of O),
// c = lane % 4 its columns (or tokens). Which tokens and which 16 codes those
// stand for is free, and chosen so that the eight lanes of a shared-memory
// phase hit all banks of the TMA-swizzled rows (128-byte swizzle for d = 128,
// 64-byte for d = 64).
template <int D>
__device__ __forceinline__ int token_of(int g) {  // of row g of the instruction's first 8
  return D == 128 ? (g >> 1) | ((g & 1) << 2) : g ^ ((g >> 1) & 1);
}
template <int D>
__device__ __forceinline__ int place(int r, int q) {  // 16-byte chunk q of token row r
  return D == 128 ? r * 128 + ((q ^ (r & 7)) << 4) : r * 64 + ((q ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) { return Elem<__half>::pack(a, b); }

// Four columns of row r of (b, hk) from its sums.
template <typename T, int D>
__device__ __forceinline__ void write_row(const CacheAttnParams& p, int b, int hk, int r, int col,
                                          const float4& y, float top, float sum) {
  const int token = r / p.group, head = hk * p.group + r - token * p.group;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key seen (a NaN sum is not 0)
  T* dst = static_cast<T*>(p.o) + ((int64_t(b) * p.n + token) * p.H + head) * D + col;
  uint2 u;
  u.x = Elem<T>::pack(y.x * inv, y.y * inv);
  u.y = Elem<T>::pack(y.z * inv, y.w * inv);
  *reinterpret_cast<uint2*>(dst) = u;
  if (col == 0)
    p.lse[(int64_t(b) * p.H + head) * p.n + token] =
        sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// Orders this thread's shared-memory accesses before later copies into it.
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kRowsWarps * 32, NT == 1 ? 3 : 2) cache_rows_kernel(const __grid_constant__ RowsParams params) {
  using C = RowsCfg<D, NT>;
  const CacheAttnParams& p = params.c;
  constexpr int H2 = D / 64;  // 64-column parts of the head dimension
  constexpr int VB = D / 8;   // output columns (value bytes) per lane
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::AT_BARS) + warp * C::STAGES;
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(smem + C::AT_BARS + kRowsWarps * C::STAGES * 8);

  const int rows = p.n * p.group;  // rows of a key head: token-major, then head of the group
  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int i = 0; i < C::STAGES; ++i) ajvp::mbar_init(&full[i], 1);
    ajvp::fence_barrier_init();
  }
  __syncthreads();

  // This block's pieces: steps [s_begin, s_end) of sequence b and key head hk,
  // one piece of a cluster's, or the steps [w, w_end) of all in a row.
  int b, hk, rank = 0;
  int64_t w = 0, w_end = 1, base = 0;  // base: the first step of (b, hk)
  if (params.work) {
    int64_t all, blocks = gridDim.x;
    find_step<kRowsWarps * 32>(
        p.B, blockIdx.x, kLeastSteps,
        [&](int i) { return int64_t(p.Hkv) * steps_of(reach_of(p, i)); }, blocks, all, b, base);
    if (blockIdx.x < blocks) {
      w = all * blockIdx.x / blocks;
      w_end = all * (blockIdx.x + 1) / blocks;
    } else {
      w = w_end = 0;
    }
    const int steps = steps_of(reach_of(p, b));
    hk = static_cast<int>((w - base) / steps);
    base += int64_t(hk) * steps;
  } else {
    const int tile = blockIdx.x / p.splits;
    rank = blockIdx.x - tile * p.splits;
    b = tile / p.Hkv;
    hk = tile - b * p.Hkv;
  }
  uint8_t* ring = smem + warp * C::SLOT;
  float* scales = reinterpret_cast<float*>(smem + C::AT_SCALES + warp * C::SCALES);
  int issued = 0, taken = 0;  // steps whose copies were issued, and waited for
  bool first_piece = true;
  Piece left = {Piece::kNone, Piece::kNone, 0, 0};
  while (w < w_end) {
    const int len = checked_len(p, b);
    const int reach = len;  // most keys seen
    const int all = p.causal ? max(len - p.n + 1, 0) : len;  // keys all rows see
    const int steps = params.work ? steps_of(reach) : (reach + kStep - 1) / kStep;
    int s_begin, s_end;
    if (params.work) {
      s_begin = static_cast<int>(w - base);
      s_end = static_cast<int>(min(w_end - base, int64_t(steps)));
    } else {
      s_begin = static_cast<int>(int64_t(steps) * rank / p.splits);
      s_end = static_cast<int>(int64_t(steps) * (rank + 1) / p.splits);
    }
    const bool whole = s_begin == 0 && s_end == steps;

    // Pages of step s: lanes 0 and 1 those of its 16-token halves; -1: none.
    auto page_of = [&](int s) -> int {
      const int j = s * kStep + (lane & 1) * 16;
      return lane < 2 && s < s_end && j < reach ? checked_page(p, b, j) : -1;
    };
    // Copies step s, whose pages are `page`, into the next stage, and reads the
    // scales of its 16-token halves: keys in lanes 0, 1, values in lanes 2, 3.
    auto fetch = [&](int s, int page) -> float {
      float sc = __uint_as_float(kHidden);
      if (s < s_end) {
        const int page0 = __shfl_sync(0xffffffffu, page, 0), page1 = __shfl_sync(0xffffffffu, page, 1);
        const int st = issued++ % C::STAGES;
        uint8_t* at = ring + st * 2 * C::KV;
        const int j = (s * kStep) & ((1 << p.page_shift) - 1);
        if (lane == 0) {
          const int boxes = params.box == kStep ? (page0 >= 0) : (page0 >= 0) + (page1 >= 0);
          ajvp::mbar_arrive_expect_tx(&full[st], boxes * params.box * D * 2);
          if (page0 >= 0) {
            ajvp::tma_load_4d(at, &params.map_k, &full[st], 0, j, hk, page0);
            ajvp::tma_load_4d(at + C::KV, &params.map_v, &full[st], 0, j, hk, page0);
          }
          if (params.box != kStep && page1 >= 0) {
            ajvp::tma_load_4d(at + 16 * D, &params.map_k, &full[st], 0, 0, hk, page1);
            ajvp::tma_load_4d(at + C::KV + 16 * D, &params.map_v, &full[st], 0, 0, hk, page1);
          }
        }
        const int pg = (lane & 1) ? page1 : page0;
        if (lane < 4 && pg >= 0) sc = p.scale[lane >> 1][pg * p.scale_page + hk * p.scale_head];
      }
      return sc;
    };
    // Writes what the softmax needs of those into stage st's scales: for the
    // two halves the key scales (a mark for a hidden half), log2 of the value
    // scales, and their inverses.
    auto keep_scales = [&](int st, float sc) {
      if (lane < 4) {
        const bool none = __float_as_uint(sc) == kHidden;
        float* to = scales + 8 * st + (lane & 1);
        const float r = none ? 1.f : read_scale(sc);
        if (lane < 2) {
          to[0] = none ? sc : r;
        } else {
          to[2] = log2_approx(r);
          to[4] = rcp_approx(r);
        }
      }
    };

    int next = s_begin + warp;  // next step to copy
    int page = page_of(next);
    float pending = 0.f;
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) {
      const int st = issued % C::STAGES;
      pending = fetch(next, page);
      next += kRowsWarps;
      page = page_of(next);
      keep_scales(st, pending);
    }

    // Queries as fp16 fragments: k-step (h, s) holds columns (c + 4h) 16 + 4s + 0..3 of row g.
    uint32_t q[NT][H2][4][2];
    float row_scale[NT][2];  // of rows 2c, 2c + 1
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 8 * t + g;
      float x[H2][16];
      float amax = 0.f;
      const int token = r / p.group, head = hk * p.group + r - token * p.group;
      const T* src = static_cast<const T*>(p.q) + b * p.q_seq + token * p.q_token + head * p.q_head;
#pragma unroll
      for (int h = 0; h < H2; ++h) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float (&y)[8] = reinterpret_cast<float(&)[8]>(x[h][8 * j]);
          if (r < rows) {
            load8(src + (c + 4 * h) * 16 + 8 * j, y);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = fabsf(y[e]);
            amax = fmaxf(amax, a < INFINITY ? a : 0.f);
          }
        }
      }
      float inv = 1.f, mine = p.scale_log2;
      if constexpr (!std::is_same<T, __half>::value) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = query_exp(amax);
        inv = ldexpf(1.f, -e);
        mine *= ldexpf(1.f, e);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) row_scale[t][i] = __shfl_sync(0xffffffffu, mine, 4 * (2 * c + i));
#pragma unroll
      for (int h = 0; h < H2; ++h)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          q[t][h][s][0] = pack_f16(x[h][4 * s] * inv, x[h][4 * s + 1] * inv);
          q[t][h][s][1] = pack_f16(x[h][4 * s + 2] * inv, x[h][4 * s + 3] * inv);
        }
    }
    int seen[NT][2];  // keys that rows 2c, 2c + 1 see
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = min(8 * t + 2 * c + i, rows - 1);
        seen[t][i] = p.causal ? max(len - p.n + r / p.group + 1, 0) : len;
      }

    float m[NT][2], l[NT][2], acc[NT][VB / 2][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 2; ++i) m[t][i] = -INFINITY, l[t][i] = 0.f;
#pragma unroll
      for (int j = 0; j < VB / 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][j][i] = 0.f;
    }

    int late = -1;  // the stage that `pending` belongs to
    __syncwarp();
    for (int s = s_begin + warp; s < s_end; s += kRowsWarps) {
      if (late >= 0) keep_scales(late, pending);
      // The next stage's reads are over since the end of the last round: the matrix
      // instructions, which the whole warp issues, have taken all that was read.
      late = next < s_end ? issued % C::STAGES : -1;
      pending = fetch(next, page);
      next += kRowsWarps;
      page = page_of(next);
      const int stage = taken % C::STAGES;
      if (!ajvp::warp_wait(&full[stage], (taken / C::STAGES) & 1, abort_flag, p.status)) break;
      ++taken;
      __syncwarp();
      const uint8_t* sk = ring + stage * 2 * C::KV;
      const uint8_t* sv = sk + C::KV;
      const float4 ss = *reinterpret_cast<const float4*>(scales + 8 * stage);
      const float2 iv = *reinterpret_cast<const float2*>(scales + 8 * stage + 4);

      float x[NT][2][4];  // 16-token halves: token g (0, 1) and g + 8 (2, 3), rows 2c (0, 2), 2c + 1
#pragma unroll
      for (int f = 0; f < 2; ++f) {
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t][f][0] = x[t][f][1] = x[t][f][2] = x[t][f][3] = 0.f;
        const int r = 16 * f + token_of<D>(g);
#pragma unroll
        for (int h = 0; h < H2; ++h) {
          const uint4 u = *reinterpret_cast<const uint4*>(sk + place<D>(r, c + 4 * h));
          const uint4 w = *reinterpret_cast<const uint4*>(sk + place<D>(r + 8, c + 4 * h));
          const uint32_t us[4] = {u.x, u.y, u.z, u.w}, ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x4(us[e], a0, a2);
            e4m3x4_to_f16x4(ws[e], a1, a3);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma_f16(x[t][f], a0, a1, a2, a3, q[t][h][e][0], q[t][h][e][1]);
          }
        }
      }
      // scores in powers of two, the value scale in the exponent
      const bool hidden[2] = {__float_as_uint(ss.x) == kHidden, __float_as_uint(ss.y) == kHidden};
      const float ks[2] = {ss.x, ss.y}, lv[2] = {ss.z, ss.w}, inv_v[2] = {iv.x, iv.y};
      const int j0 = s * kStep;
      const bool edge = j0 + kStep > all || hidden[0] || hidden[1];
      float top[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[t][f][e] = fmaf(x[t][f][e], row_scale[t][e & 1] * ks[f], lv[f]);
        if (edge) {
#pragma unroll
          for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (hidden[f] || j0 + 16 * f + token_of<D>(g) + 8 * (e >> 1) >= seen[t][e & 1])
                x[t][f][e] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          top[t][i] = fmaxf(fmaxf(x[t][0][i], x[t][0][i + 2]), fmaxf(x[t][1][i], x[t][1][i + 2]));
      }
      bool raise = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) raise |= top[t][i] > m[t][i] + kRaise;
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float to = top[t][i];
            to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, 4));
            to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, 8));
            to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, 16));
            to = fmaxf(to - kLead, m[t][i]);
            const float f = to == -INFINITY ? 1.f : ajvp::ex2_approx(m[t][i] - to);
            m[t][i] = to;
            l[t][i] *= f;
#pragma unroll
            for (int j = 0; j < VB / 2; ++j) {
              acc[t][j][i] *= f;
              acc[t][j][2 + i] *= f;
            }
          }
      }
      uint32_t pk[NT][2][2], vis[NT][2][2];  // probabilities, and 1.0 where a row sees a token
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float base[2] = {m[t][0] == -INFINITY ? 0.f : m[t][0], m[t][1] == -INFINITY ? 0.f : m[t][1]};
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          if (edge) {
            vis[t][f][0] = transpose8(pack_f16(x[t][f][0] != -INFINITY, x[t][f][1] != -INFINITY));
            vis[t][f][1] = transpose8(pack_f16(x[t][f][2] != -INFINITY, x[t][f][3] != -INFINITY));
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) x[t][f][e] = ajvp::ex2_approx(x[t][f][e] - base[e & 1]);
          l[t][0] = fmaf(x[t][f][0] + x[t][f][2], inv_v[f], l[t][0]);
          l[t][1] = fmaf(x[t][f][1] + x[t][f][3], inv_v[f], l[t][1]);
          pk[t][f][0] = transpose8(pack_f16(x[t][f][0], x[t][f][1]));
          pk[t][f][1] = transpose8(pack_f16(x[t][f][2], x[t][f][3]));
        }
      }
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        // values of the instruction's tokens 2c, 2c + 1, 2c + 8, 2c + 9, the lane's columns
        uint32_t w[4][VB / 4];
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 16 * f + token_of<D>(2 * c + (i & 1)) + 8 * (i >> 1);
          if constexpr (D == 128) {
            const uint4 u = *reinterpret_cast<const uint4*>(sv + place<D>(r, token_of<D>(g)));
            w[i][0] = u.x, w[i][1] = u.y, w[i][2] = u.z, w[i][3] = u.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(sv + place<D>(r, g >> 1) + 8 * (g & 1));
            w[i][0] = u.x, w[i][1] = u.y;
          }
          if (edge) {
#pragma unroll
            for (int e = 0; e < VB / 4; ++e)
              nan |= (((w[i][e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
          }
        }
        // A NaN value where some rows see the token and some do not (or none: what
        // an earlier owner of the page left there): it must not reach the rows
        // that do not (0 * NaN). It is taken out of the product, and a second
        // product, of what each row sees and where the NaN are, says which sums
        // become NaN.
        if (edge && __any_sync(0xffffffffu, nan)) {
#pragma unroll
          for (int e = 0; e < VB / 4; ++e) {
            uint32_t mark[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              mark[i] = (((w[i][e] & 0x7f7f7f7fu) + 0x01010101u) >> 7) & 0x01010101u;
              w[i][e] &= ~(mark[i] * 0xffu);
              mark[i] *= 0x38u;  // the e4m3 code of 1
            }
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
              const uint32_t sel = hi ? 0x7362u : 0x5140u;
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16x4(__byte_perm(mark[0], mark[1], sel), a0, a1);
              e4m3x4_to_f16x4(__byte_perm(mark[2], mark[3], sel), a2, a3);
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                float hit[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(hit, a0, a1, a2, a3, vis[t][f][0], vis[t][f][1]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (hit[i] > 0.f) acc[t][2 * e + hi][i] = NAN;
              }
            }
          }
        }
#pragma unroll
        for (int e = 0; e < VB / 4; ++e)
#pragma unroll
          for (int hi = 0; hi < 2; ++hi) {
            // bytes 2hi, 2hi + 1 of the two tokens of a pair, interleaved
            const uint32_t sel = hi ? 0x7362u : 0x5140u;
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x4(__byte_perm(w[0][e], w[1][e], sel), a0, a1);
            e4m3x4_to_f16x4(__byte_perm(w[2][e], w[3][e], sel), a2, a3);
#pragma unroll
            for (int t = 0; t < NT; ++t)
              mma_f16(acc[t][2 * e + hi], a0, a1, a2, a3, pk[t][f][0], pk[t][f][1]);
          }
      }
      __syncwarp();
    }
    // After an abort copies may still be on their way: they land before the ring
    // is written over. (A normal end has waited for each.)
    for (; taken < issued; ++taken)
      ajvp::mbar_wait_drain(&full[taken % C::STAGES], (taken / C::STAGES) & 1, 200000000ull);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 4);
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 8);
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 16);
      }

    // Join the warps: each leaves its sums in its ring, then the block adds them
    // up into `whole`, and the cluster's blocks add those up.
    float* sums = reinterpret_cast<float*>(smem + C::AT_WHOLE);
    float* wm = reinterpret_cast<float*>(smem + C::AT_STATS);  // [warps][ROWS]: running maxima
    float* wl = wm + C::ROWS * kRowsWarps;                     // [warps][ROWS]: sums
    float* bm = wl + C::ROWS * kRowsWarps;                     // [ROWS]: the block's maxima, then sums
    __syncwarp();
    {
      float* part = reinterpret_cast<float*>(ring);
      const int col = D == 128 ? token_of<D>(g) * VB : g * VB;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 8 * t + 2 * c + i;
#pragma unroll
          for (int j = 0; j < VB / 2; j += 2)
            *reinterpret_cast<float4*>(part + r * C::PITCH + col + 2 * j) =
                make_float4(acc[t][j][i], acc[t][j][2 + i], acc[t][j + 1][i], acc[t][j + 1][2 + i]);
          if (g == 0) {
            wm[warp * C::ROWS + r] = m[t][i];
            wl[warp * C::ROWS + r] = l[t][i];
          }
        }
    }
    __syncthreads();
    constexpr int kThreads = kRowsWarps * 32;
    // what the block's warps have of 4 columns of row r
    auto block_sums = [&](int r, int col, float& top, float& sum) -> float4 {
      top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) top = fmaxf(top, wm[w * C::ROWS + r]);
      sum = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) {
        // a warp that saw no key has sum 0 and maximum -inf; NaN sums pass on
        const float f = top == -INFINITY ? 1.f : ajvp::ex2_approx(wm[w * C::ROWS + r] - top);
        sum = fmaf(wl[w * C::ROWS + r], f, sum);
        const float4 z = *reinterpret_cast<const float4*>(smem + w * C::SLOT + (r * C::PITCH + col) * 4);
        y.x = fmaf(z.x, f, y.x), y.y = fmaf(z.y, f, y.y);
        y.z = fmaf(z.z, f, y.z), y.w = fmaf(z.w, f, y.w);
      }
      return y;
    };
    if (params.work || p.splits == 1) {
      float* place = params.work + (2 * int64_t(blockIdx.x) + (first_piece ? 0 : 1)) * C::PLACE;
      for (int item = threadIdx.x; item < C::ROWS * (D / 4); item += kThreads) {
        const int r = item / (D / 4), col = (item % (D / 4)) * 4;
        if (r >= rows) continue;
        float top, sum;
        const float4 y = block_sums(r, col, top, sum);
        if (whole) {
          write_row<T, D>(p, b, hk, r, col, y, top, sum);
        } else {
          *reinterpret_cast<float4*>(place + r * D + col) = y;
          if (col == 0) place[C::ROWS * D + r] = top, place[C::ROWS * (D + 1) + r] = sum;
        }
      }
      if (!whole) {
        if (s_begin > 0)
          left.went_on = b * p.Hkv + hk;
        else
          left.begun = b * p.Hkv + hk, left.place = first_piece ? 0 : 1;
      }
      // on to the next piece, whose copies go where these sums are
      first_piece = false;
      w = base + s_end;
      if (!params.work || w >= w_end) break;
      base = w;
      if (++hk == p.Hkv) hk = 0, ++b;
      fence_async();
      __syncthreads();
      continue;
    }
    // one of a cluster's blocks
    for (int item = threadIdx.x; item < C::ROWS * (D / 4); item += kThreads) {
      const int r = item / (D / 4), col = (item % (D / 4)) * 4;
      float top, sum;
      *reinterpret_cast<float4*>(sums + r * C::PITCH + col) = block_sums(r, col, top, sum);
      if (col == 0) bm[r] = top, bm[C::ROWS + r] = sum;
    }
    ajvp::cluster_sync_all();
    // Block `rank` of the cluster joins and writes every splits-th group of 4 columns.
    const uint32_t sums_addr = ajvp::smem_u32(sums), bm_addr = ajvp::smem_u32(bm);
    for (int item = rank + threadIdx.x * p.splits; item < C::ROWS * (D / 4); item += kThreads * p.splits) {
      const int r = item / (D / 4), col = (item % (D / 4)) * 4;
      if (r >= rows) continue;
      // all blocks' reads are in flight together
      float mk[kMostSplits], lk[kMostSplits], top = -INFINITY, sum = 0.f;
      float4 z[kMostSplits], y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMostSplits; ++k) {
        mk[k] = -INFINITY, lk[k] = 0.f, z[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < p.splits) {
          mk[k] = ld_cluster_f32(ajvp::mapa_shared(bm_addr + r * 4, k));
          lk[k] = ld_cluster_f32(ajvp::mapa_shared(bm_addr + (C::ROWS + r) * 4, k));
          z[k] = ld_cluster_f32x4(ajvp::mapa_shared(sums_addr + (r * C::PITCH + col) * 4, k));
        }
      }
#pragma unroll
      for (int k = 0; k < kMostSplits; ++k) top = fmaxf(top, mk[k]);
#pragma unroll
      for (int k = 0; k < kMostSplits; ++k) {
        const float f = top == -INFINITY ? 1.f : ajvp::ex2_approx(mk[k] - top);
        sum = fmaf(lk[k], f, sum);
        y.x = fmaf(z[k].x, f, y.x), y.y = fmaf(z[k].y, f, y.y);
        y.z = fmaf(z[k].z, f, y.z), y.w = fmaf(z[k].w, f, y.w);
      }
      write_row<T, D>(p, b, hk, r, col, y, top, sum);
    }
    ajvp::cluster_sync_all();  // no block leaves while its sums are read
    break;
  }
  if (params.work && threadIdx.x == 0)
    reinterpret_cast<Piece*>(params.work + 2 * int64_t(gridDim.x) * C::PLACE)[blockIdx.x] = left;
}

// Joins the pieces of the (sequence, key head) that block blockIdx.x began and
// later blocks went on with. A block takes 32 groups of 4 columns; its warps
// take every fourth piece, four at a time, and join what they have.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kRowsWarps * 32) join_rows_kernel(const CacheAttnParams p,
                                                                    const float* work, const int blocks) {
  using C = RowsCfg<D, NT>;
  __shared__ float stats[2][kRowsWarps][32];
  __shared__ float4 part[kRowsWarps][32];
  cudaGridDependencySynchronize();  // launched early: the pieces are complete from here on
  const Piece* pieces = reinterpret_cast<const Piece*>(work + 2 * int64_t(blocks) * C::PLACE);
  const int first = blockIdx.x, tile = pieces[first].begun;
  if (tile < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = blockIdx.y * 32 + lane;
  const int r = item / (D / 4), col = (item % (D / 4)) * 4;
  const int rows = p.n * p.group;
  Join join;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  if (warp == 0 && r < rows) {
    const float* at = work + (2 * int64_t(first) + pieces[first].place) * C::PLACE;
    const float4 z = *reinterpret_cast<const float4*>(at + r * D + col);
    join.add(at[C::ROWS * D + r], at[C::ROWS * (D + 1) + r], &y, &z, 1);
  }
  bool more = true;
  for (int k0 = first + 1; more; k0 += 32) {
    const uint32_t use = went_on(pieces, blocks, k0, tile, more);
    if (r < rows) {
      for (int i0 = warp; i0 < 32; i0 += 4 * kRowsWarps) {
        float mk[4], lk[4];
        float4 z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = i0 + i * kRowsWarps;
          mk[i] = -INFINITY, lk[i] = 0.f, z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if ((use >> j) & 1u) {
            const float* at = work + 2 * int64_t(k0 + j) * C::PLACE;
            mk[i] = at[C::ROWS * D + r];
            lk[i] = at[C::ROWS * (D + 1) + r];
            z[i] = *reinterpret_cast<const float4*>(at + r * D + col);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) join.add(mk[i], lk[i], &y, &z[i], 1);
      }
    }
  }
  stats[0][warp][lane] = join.top, stats[1][warp][lane] = join.sum;
  part[warp][lane] = y;
  __syncthreads();
  if (warp == 0 && r < rows) {
#pragma unroll
    for (int w = 1; w < kRowsWarps; ++w) join.add(stats[0][w][lane], stats[1][w][lane], &y, &part[w][lane], 1);
    write_row<T, D>(p, tile / p.Hkv, tile % p.Hkv, r, col, y, join.top, join.sum);
  }
}

template <typename T, int D, int NT>
cudaError_t rows_launch(const RowsParams& p, int blocks, cudaStream_t st) {
  using C = RowsCfg<D, NT>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(cache_rows_kernel<T, D, NT>, C::BYTES, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.work ? blocks : p.c.B * p.c.Hkv * p.c.splits));
  cfg.blockDim = dim3(kRowsWarps * 32);
  cfg.dynamicSmemBytes = C::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.c.splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, cache_rows_kernel<T, D, NT>, p);
  if (e != cudaSuccess || !p.work) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks),
                     static_cast<unsigned>((p.c.n * p.c.group * (D / 4) + 31) / 32));
  cfg.dynamicSmemBytes = 0;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, join_rows_kernel<T, D, NT>, p.c, static_cast<const float*>(p.work),
                            blocks);
}

template <typename T, int D>
cudaError_t rows_launch(const RowsParams& p, int blocks, cudaStream_t st) {
  return p.c.n * p.c.group <= 8 ? rows_launch<T, D, 1>(p, blocks, st)
                                : rows_launch<T, D, 2>(p, blocks, st);
}

// Tiles of 8 or 16 query rows.
cudaError_t cache_rows_launch(const RowsParams& p, int d, int dtype, int blocks, cudaStream_t st) {
  if (dtype == ATTN_JVP_BF16)
    return d == 128 ? rows_launch<__nv_bfloat16, 128>(p, blocks, st)
                    : rows_launch<__nv_bfloat16, 64>(p, blocks, st);
  return d == 128 ? rows_launch<__half, 128>(p, blocks, st) : rows_launch<__half, 64>(p, blocks, st);
}

// Blocks that share out the steps: as many per SM as fit (8 rows: 168 registers,
// 12 bytes spilled at d = 128, and 70 KB; 16 rows: 255 and 104 KB. At 16 rows three blocks per SM spill and
// took 231 us where two take 134).
constexpr int blocks_per_sm(int64_t rows) { return rows <= 8 ? 3 : 2; }

// How the work of a call with `rows` query rows per key head is shared out, for
// sequences of up to `len` tokens: blocks (0: clusters, no workspace) and bytes
// of workspace for each.
//   - More than 16 rows go to the tcgen05 kernel. 8 sequences of 8,192 tokens, 8
//     key heads, us of the GPU in a graph, d = 128 (64), here: 4 rows 34 (25), 8: 35
//     (25), 9: 44 (34), 16: 46 (34); there: 17 and 20 rows 89 (72), 32: 90 (72), 64:
//     94 (73), 128: 99 (76), 129: 115 (89), 256: 124 (93). A second call here for
//     the rows beyond 16 would bring 17 to 24 rows to 81 (59) and 25 to 32 to 91
//     (68), and three or more calls are behind.
//   - Up to 16 rows, clusters (one launch) up to 512 tokens, or 4,096 if they are
//     all resident at once; shared out evenly (two launches) beyond. us, clusters
//     / shared out, single tokens, d = 128, by sequences x key heads and tokens:
//       1 x 8:  512: 7.1 / 10.4   4,096: 11.5 / 12.1   16,384: 26.9 / 21.5
//       16 x 2: 512: 7.5 / 10.7   4,096: 13.2 / 17.7   16,384: 32.4 / 34.8
//       64 x 8: 512: 19.8 / 24.7  1,024: 36.7 / 35.1    8,192: 228 / 171
//     and sequences of different lengths add to the second's advantage.
struct Share {
  int blocks;
  int64_t bytes;
  Share(int64_t rows, int64_t B, int64_t Hkv, int64_t d, int64_t len, int sms) : blocks(0), bytes(0) {
    if (rows > kRowsTile) {
      // a block per SM, but no more than give each four key tiles
      const int64_t steps = B * Hkv * ((rows + kTilesRows - 1) / kTilesRows) * ((len + 127) / 128);
      const int64_t most = (steps + 3) / 4;
      blocks = static_cast<int>(most < sms ? most : sms);
      bytes = tiles_work_bytes(d);
    } else if (len > 512 && (len > 4096 || B * Hkv * 8 > 2 * sms)) {
      blocks = blocks_per_sm(rows) * sms;
      bytes = 2 * (rows <= 8 ? 8 : 16) * (d + 2) * 4 + static_cast<int64_t>(sizeof(Piece));
    }
  }
};

int check_attn_shape(const attn_jvp_shape& s, int64_t Hkv) {
  if ((s.dtype != ATTN_JVP_BF16 && s.dtype != ATTN_JVP_F16) || (s.d != 64 && s.d != 128))
    return ATTN_JVP_ERR_UNSUPPORTED;
  if (s.B < 0 || s.B > 65535 || s.L < 0 || s.L > (1 << 24) || s.H < 1 || s.H > 65535 || Hkv < 1 || s.H % Hkv)
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  return ATTN_JVP_OK;
}

}  // namespace

}  // namespace ajvp_serve

extern "C" int64_t attn_jvp_cache_attn_workspace_bytes(const attn_jvp_shape* shape, int64_t Hkv,
                                                       int64_t max_len) {
  using namespace ajvp_serve;
  if (!shape || check_attn_shape(*shape, Hkv) || max_len < 0 || max_len > (int64_t(1) << 30)) return -1;
  unsigned int* status = nullptr;
  int sms = 0;
  if (ajvp::device_status_word(&status, &sms) != ATTN_JVP_OK) return -1;
  const Share share(shape->L * (shape->H / Hkv), shape->B, Hkv, shape->d, max_len, sms);
  return share.blocks * share.bytes;
}

extern "C" int attn_jvp_cache_attn(const attn_jvp_shape* shape, int64_t Hkv, const void* q,
                                   const int64_t* q_strides, const attn_jvp_cache* cache,
                                   const int32_t* lens, const int32_t* table, int64_t table_width,
                                   int64_t table_stride, int64_t max_len, int32_t causal,
                                   void* workspace, int64_t workspace_bytes, void* o, float* lse,
                                   void* stream) {
  using namespace ajvp_serve;
  if (!shape || !q_strides) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  const attn_jvp_shape& s = *shape;
  int rc = check_attn_shape(s, Hkv);
  if (rc != ATTN_JVP_OK) return rc;
  if (max_len < 0 || !good_scale(s.scale)) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if ((rc = check_cache(cache, Hkv, s.d)) != ATTN_JVP_OK) return rc;
  if (table_width < 1 || table_width > (int64_t(1) << 30) / cache->page_tokens ||
      (s.B > 1 && table_stride < table_width))
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (s.B == 0 || s.L == 0) return ATTN_JVP_OK;
  if (!q || !lens || !table || !o || !lse) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(o) || !aligned4(lse) || !aligned4(lens) || !aligned4(table) ||
      (s.B > 1 && q_strides[0] % 8) ||
      (s.L > 1 && q_strides[1] % 8) || (s.H > 1 && q_strides[2] % 8))
    return ATTN_JVP_ERR_MISALIGNED;
  if ((s.B > 1 && q_strides[0] < 0) || (s.L > 1 && q_strides[1] < 0) || (s.H > 1 && q_strides[2] < 0))
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  RowsParams rp;
  CacheAttnParams& p = rp.c;
  int sms = 0;
  rc = ajvp::device_status_word(&p.status, &sms);
  if (rc != ATTN_JVP_OK) return rc;
  p.q = q, p.q_seq = q_strides[0], p.q_token = q_strides[1], p.q_head = q_strides[2];
  p.codes[0] = static_cast<const uint8_t*>(cache->k);
  p.codes[1] = static_cast<const uint8_t*>(cache->v);
  p.scale[0] = cache->k_scale, p.scale[1] = cache->v_scale;
  p.page_stride = cache->page_stride, p.head_stride = cache->head_stride;
  p.token_stride = cache->token_stride;
  p.scale_page = cache->scale_page_stride, p.scale_head = cache->scale_head_stride;
  p.lens = lens, p.table = table, p.table_stride = table_stride;
  p.o = o, p.lse = lse;
  p.B = static_cast<int>(s.B), p.n = static_cast<int>(s.L), p.H = static_cast<int>(s.H);
  p.Hkv = static_cast<int>(Hkv), p.group = p.H / p.Hkv;
  p.pages = static_cast<int>(cache->pages), p.table_width = static_cast<int>(table_width);
  p.page_shift = 4;
  while ((1 << p.page_shift) < cache->page_tokens) ++p.page_shift;
  p.causal = causal != 0;
  p.scale_log2 = scale_log2(s.scale, s.d);
  const int64_t bound = table_width * cache->page_tokens;
  const int64_t len = max_len > 0 && max_len < bound ? max_len : bound;
  const int64_t rows = s.L * p.group;
  const bool few = rows <= kRowsTile;
  const int per_tile = few ? kRowsTile : kTilesRows;
  const int64_t row_tiles = (rows + per_tile - 1) / per_tile;
  const int64_t tiles = s.B * Hkv * row_tiles;
  if (rows > (int64_t(1) << 30) || tiles > (int64_t(1) << 27)) return ATTN_JVP_ERR_UNSUPPORTED;
  p.row_tiles = static_cast<int>(row_tiles);
  p.splits = 1;
  const Share share(rows, s.B, Hkv, s.d, len, sms);
  if (share.blocks) {
    if (!workspace || workspace_bytes < share.blocks * share.bytes) return ATTN_JVP_ERR_INVALID_ARGUMENT;
    if (!aligned16(workspace)) return ATTN_JVP_ERR_MISALIGNED;
  } else {
    while (p.splits < kMostSplits && tiles * p.splits < 2 * sms && len >= 256 * p.splits) p.splits *= 2;
  }
  rp.work = share.blocks ? static_cast<float*>(workspace) : nullptr;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (few) {
    rp.box = cache->page_tokens < kStep ? static_cast<int>(cache->page_tokens) : kStep;
    if (!ajvp::encode_cache_map(&rp.map_k, cache->k, s.d, cache->page_tokens, Hkv, cache->pages,
                                p.token_stride, p.head_stride, p.page_stride, rp.box) ||
        !ajvp::encode_cache_map(&rp.map_v, cache->v, s.d, cache->page_tokens, Hkv, cache->pages,
                                p.token_stride, p.head_stride, p.page_stride, rp.box))
      return ATTN_JVP_ERR_INVALID_ARGUMENT;
    e = cache_rows_launch(rp, static_cast<int>(s.d), s.dtype, share.blocks, st);
  } else {
    e = cache_tiles_launch(p, static_cast<int>(s.d), s.dtype, share.blocks, rp.work, st);
  }
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? ATTN_JVP_OK : ATTN_JVP_ERR_CUDA;
}
