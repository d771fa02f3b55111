// attn_cache_rows.cu - attention of a few query rows over the paged e4m3 cache
// (C ABI attn_jvp_cache_attn): single tokens and short runs of tokens.
//
// For each row, over the keys that it sees, with code values k_j, v_j and the
// page scales a_j, b_j:
//   x_j = s a_j <q, k_j>,  O = sum_j e^(x_j) b_j v_j / sum_j e^(x_j)
// One pass with a running maximum, in powers of two. The value scale goes into
// the exponent: with t_j = x_j log2 e + log2 b_j and m = max t_j,
//   p_j = 2^(t_j - m),  O = sum_j p_j v_j / sum_j p_j / b_j,
// so p is at most 2^kLazyMax however the scales differ, and what fp16 rounds
// away of p is small against the largest contribution to O.
//
// Bound by HBM: a cached token is 2 d bytes per key head, read once; 16 rows
// (all query heads of the key head, and the newest tokens) share it. Codes are
// exact in fp16, so both products run on m16n8k16 fp16 matrix instructions
// with fp32 sums; bf16 queries are scaled by a power of two per row into fp16
// (exact within 2^-14 of the row's largest, absolute error 2^-25 of it below).
// 128-row tensor-memory tiles would leave 7/8 of the rows unused here.
//
// Layout: each warp streams its own steps of 32 tokens through a private ring
// of asynchronous copies (no block-wide barrier in the loop), so a stall of
// one warp holds up no other. The order of the head dimension inside the
// products is free, so a lane takes 16 adjacent codes at a time for four
// matrix instructions, and the column order of O lets a lane own adjacent
// columns: no shared-memory transposes. The key axis of one tile is split
// over the blocks of a cluster, which join their sums through distributed
// shared memory: one launch, no workspace, a fixed order of sums.
#include "serve_attn.cuh"

#include <type_traits>

namespace ajvp_serve {

constexpr int kRowsWarps = 4;
constexpr int kStep = 32;  // tokens per step of a warp
constexpr uint32_t kHidden = 0xffffffffu;  // in place of a key scale: no page there

template <int D>
struct RowsCfg {
  static constexpr int STAGES = D == 128 ? 3 : 4;
  static constexpr int KV = kStep * D;            // bytes of a step's keys (or values)
  static constexpr int STAGE = 2 * KV + 16;       // and k, v scales of its two 16-token halves
  static constexpr int RING = STAGES * STAGE;     // per warp
  static constexpr int PART = kRowsTile * D * 4;  // one warp's sums
  static constexpr int BYTES = kRowsWarps * (RING > PART ? RING : PART) + PART + 3 * 4 * kRowsTile * kRowsWarps;
};

// Where 16-byte chunk q of token row r lies in a step's keys or values, so
// that the lanes of a quarter warp hit all banks: they read 2 rows x 4 chunks
// of the keys, 4 even rows x 2 chunks of the values.
template <int D>
__device__ __forceinline__ int k_place(int r, int q) {
  return D == 128 ? r * 128 + ((q ^ ((r & 1) << 2)) << 4) : r * 64 + (q << 4);
}
template <int D>
__device__ __forceinline__ int v_place(int r, int q) {
  return D == 128 ? r * 128 + ((q ^ (((r >> 1) & 3) << 1)) << 4)
                  : (r >> 1) * 128 + (((((r & 1) << 2) + q) ^ (((r >> 1) & 3) << 1)) << 4);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  return Elem<__half>::pack(a, b);
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowsWarps * 32) cache_rows_kernel(const __grid_constant__ CacheAttnParams p) {
  using C = RowsCfg<D>;
  constexpr int H2 = D / 64;  // 64-column parts of the head dimension
  constexpr int VB = D / 8;   // output columns (value bytes) per lane and row
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;

  const int tile = blockIdx.x / p.splits, rank = blockIdx.x - tile * p.splits;
  const int rt = tile % p.row_tiles, bh = tile / p.row_tiles;
  const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const int rows = p.n * p.group;  // rows of this key head: token-major, then head of the group
  const int row0 = rt * kRowsTile;
  const int len = checked_len(p, b);

  // This lane's rows g and g + 8: keys they see.
  int seen[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = min(row0 + g + 8 * i, rows - 1);
    seen[i] = p.causal ? max(len - p.n + r / p.group + 1, 0) : len;
  }
  const int last = min(row0 + kRowsTile, rows) - 1;
  const int reach = p.causal ? max(len - p.n + last / p.group + 1, 0) : len;   // most keys seen
  const int all = p.causal ? max(len - p.n + row0 / p.group + 1, 0) : len;     // keys all rows see
  const int steps = (reach + kStep - 1) / kStep;
  const int s_begin = static_cast<int>(int64_t(steps) * rank / p.splits);
  const int s_end = static_cast<int>(int64_t(steps) * (rank + 1) / p.splits);

  // Queries as fp16 fragments: k-step (h, s) holds columns (c + 4h) 16 + 4s + 0..3.
  uint32_t q[H2][4][4];
  float row_scale[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = row0 + g + 8 * i;
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
    float inv = 1.f;
    row_scale[i] = p.scale_log2;
    if constexpr (sizeof(T) == 2 && !std::is_same<T, __half>::value) {
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      int e = 0;
      if (amax > 0.f) frexpf(amax, &e);
      e = min(max(e, -100), 100);
      inv = ldexpf(1.f, -e);
      row_scale[i] *= ldexpf(1.f, e);
    }
#pragma unroll
    for (int h = 0; h < H2; ++h)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        q[h][s][i] = pack_f16(x[h][4 * s] * inv, x[h][4 * s + 1] * inv);
        q[h][s][2 + i] = pack_f16(x[h][4 * s + 2] * inv, x[h][4 * s + 3] * inv);
      }
  }

  uint8_t* ring = smem + warp * (C::RING > C::PART ? C::RING : C::PART);
  const uint32_t ring_addr = ajvp::smem_u32(ring);
  const uint8_t* kb = p.codes[0] + hk * p.head_stride;
  const uint8_t* vb = p.codes[1] + hk * p.head_stride;
  const int in_page = (1 << p.page_shift) - 1;

  // The page of this lane's 16-token half (lane / 16) of step s; -1: none.
  auto page_of = [&](int s) -> int {
    const int j = s * kStep + (lane & 16);
    return s < s_end && j < reach ? checked_page(p, b, j) : -1;
  };
  // Copies step s, whose pages are `page`, into stage st.
  auto fetch = [&](int s, int st, int page) {
    if (s < s_end) {
      const uint32_t at = ring_addr + st * C::STAGE;
      constexpr int Q = D / 16, PER = 32 / Q;  // chunks of a row, rows per round of the warp
      const int chunk = lane % Q, first = lane / Q;
#pragma unroll
      for (int i = 0; i < kStep / PER; ++i) {
        const int r = first + i * PER;
        const int j = s * kStep + r;
        const int pg = __shfl_sync(0xffffffffu, page, r & 16);
        const bool valid = pg >= 0 && j < reach;
        const int64_t off = valid ? pg * p.page_stride + (j & in_page) * p.token_stride + chunk * 16 : 0;
        copy16(at + k_place<D>(r, chunk), kb + off, valid);
        copy16(at + C::KV + v_place<D>(r, chunk), vb + off, valid);
      }
      // scales of the halves: lanes 0, 16 keys, 1, 17 values; a hidden half has the mark
      if ((lane & 15) < 2) {
        float* dst = reinterpret_cast<float*>(ring + st * C::STAGE + 2 * C::KV) + (lane & 1) * 2 + (lane >> 4);
        if (page >= 0) {
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ajvp::smem_u32(dst)),
                       "l"(p.scale[lane & 1] + page * p.scale_page + hk * p.scale_head)
                       : "memory");
        } else {
          *dst = (lane & 1) ? 1.f : __uint_as_float(kHidden);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float acc[VB][4];
#pragma unroll
  for (int j = 0; j < VB; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

  int next = s_begin + warp;  // next step to copy
  int page = page_of(next);
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) {
    fetch(next, i, page);
    next += kRowsWarps;
    page = page_of(next);
  }
  int stage = 0;
  for (int s = s_begin + warp; s < s_end; s += kRowsWarps) {
    asm volatile("cp.async.wait_group %0;" ::"n"(C::STAGES - 2) : "memory");
    __syncwarp();
    {
      int into = stage + C::STAGES - 1;
      if (into >= C::STAGES) into -= C::STAGES;
      fetch(next, into, page);
      next += kRowsWarps;
      page = page_of(next);
    }
    const uint8_t* sk = ring + stage * C::STAGE;
    const uint8_t* sv = sk + C::KV;
    const float* ss = reinterpret_cast<const float*>(sv + C::KV);
    float t[4][4];  // 8-token tiles: rows g (0, 1), g + 8 (2, 3), tokens 8 i + 2c, + 1
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[i][0] = t[i][1] = t[i][2] = t[i][3] = 0.f;
#pragma unroll
      for (int h = 0; h < H2; ++h) {
        const uint4 w = *reinterpret_cast<const uint4*>(sk + k_place<D>(8 * i + g, c + 4 * h));
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mma_f16(t[i], q[h][e][0], q[h][e][1], q[h][e][2], q[h][e][3],
                  e4m3x2_to_f16x2(ws[e] & 0xffffu), e4m3x2_to_f16x2(ws[e] >> 16));
      }
    }
    // scores in powers of two, the value scale in the exponent
    float inv_v[2];
    const int j0 = s * kStep;
    const bool edge = j0 + kStep > all;
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const float ks = ss[f], vs = read_scale(ss[2 + f]);
      inv_v[f] = 1.f / vs;
      const float lv = log2_approx(vs);
      const bool none = __float_as_uint(ks) == kHidden;
      const float kr = read_scale(ks);
      const float a[2] = {row_scale[0] * kr, row_scale[1] * kr};
#pragma unroll
      for (int i = 2 * f; i < 2 * f + 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = fmaf(t[i][e], a[e >> 1], lv);
          if (none || (edge && j0 + 8 * i + 2 * c + (e & 1) >= seen[e >> 1])) x = -INFINITY;
          t[i][e] = x;
          top[e >> 1] = fmaxf(top[e >> 1], x);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
    }
    if (__any_sync(0xffffffffu, top[0] > m[0] + kLazyMax || top[1] > m[1] + kLazyMax)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float to = fmaxf(m[i], top[i]);
        const float f = to == -INFINITY ? 1.f : ajvp::ex2_approx(m[i] - to);
        m[i] = to;
        l[i] *= f;
#pragma unroll
        for (int j = 0; j < VB; ++j) {
          acc[j][2 * i] *= f;
          acc[j][2 * i + 1] *= f;
        }
      }
    }
    const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      float sum[2] = {0.f, 0.f};
      uint32_t seen_pairs[4] = {0, 0, 0, 0};  // 1.0 where a row sees the token (the slow path below)
      uint32_t pk[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float (&x)[4] = t[2 * f + i];
        if (edge) {
          seen_pairs[2 * i] = pack_f16(x[0] != -INFINITY, x[1] != -INFINITY);
          seen_pairs[2 * i + 1] = pack_f16(x[2] != -INFINITY, x[3] != -INFINITY);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = ajvp::ex2_approx(x[e] - base[e >> 1]);
          sum[e >> 1] += x[e];
        }
        pk[2 * i] = pack_f16(x[0], x[1]);
        pk[2 * i + 1] = pack_f16(x[2], x[3]);
      }
      l[0] = fmaf(sum[0], inv_v[f], l[0]);
      l[1] = fmaf(sum[1], inv_v[f], l[1]);
      // values of tokens 2c, 2c + 1, 2c + 8, 2c + 9, columns VB g .. + VB
      uint32_t w[4][VB / 4];
      bool nan = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 16 * f + 2 * c + (i & 1) + 8 * (i >> 1);
        if constexpr (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(sv + v_place<D>(r, g));
          w[i][0] = u.x, w[i][1] = u.y, w[i][2] = u.z, w[i][3] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(sv + v_place<D>(r, g >> 1) + 8 * (g & 1));
          w[i][0] = u.x, w[i][1] = u.y;
        }
        if (edge) {
#pragma unroll
          for (int e = 0; e < VB / 4; ++e)
            nan |= (((w[i][e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
        }
      }
      // A NaN value where some rows see the token and some do not: it must not
      // reach the rows that do not (0 * NaN). It is taken out of the product,
      // and a second product, of what each row sees and where the NaN are,
      // says which sums become NaN.
      const bool apart = edge && __any_sync(0xffffffffu, nan);
#pragma unroll
      for (int e = 0; e < VB / 4; ++e) {
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          // bytes 2hi, 2hi + 1 of the two tokens of a pair, interleaved
          const uint32_t sel = hi ? 0x7362u : 0x5140u;
          uint32_t p0 = __byte_perm(w[0][e], w[1][e], sel), p1 = __byte_perm(w[2][e], w[3][e], sel);
          if (apart) {
            const uint32_t n0 = (((p0 & 0x7f7f7f7fu) + 0x01010101u) >> 7) & 0x01010101u;
            const uint32_t n1 = (((p1 & 0x7f7f7f7fu) + 0x01010101u) >> 7) & 0x01010101u;
            p0 &= ~(n0 * 0xffu);
            p1 &= ~(n1 * 0xffu);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float hit[4] = {0.f, 0.f, 0.f, 0.f};
              // 0x38 is the e4m3 code of 1
              mma_f16(hit, seen_pairs[0], seen_pairs[1], seen_pairs[2], seen_pairs[3],
                      e4m3x2_to_f16x2(((n0 * 0x38u) >> (16 * k)) & 0xffffu),
                      e4m3x2_to_f16x2(((n1 * 0x38u) >> (16 * k)) & 0xffffu));
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (hit[x] > 0.f) acc[4 * e + 2 * hi + k][x] = NAN;
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k)
            mma_f16(acc[4 * e + 2 * hi + k], pk[0], pk[1], pk[2], pk[3],
                    e4m3x2_to_f16x2((p0 >> (16 * k)) & 0xffffu),
                    e4m3x2_to_f16x2((p1 >> (16 * k)) & 0xffffu));
        }
      }
    }
    __syncwarp();
    if (++stage == C::STAGES) stage = 0;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
  }

  // Join the warps: each leaves its sums in its ring, then the block adds them
  // up into `whole`, and the cluster's blocks add those up.
  constexpr int SLOT = C::RING > C::PART ? C::RING : C::PART;
  float* whole = reinterpret_cast<float*>(smem + kRowsWarps * SLOT);
  float* wm = whole + kRowsTile * D;              // [warps][16]: running maxima
  float* wl = wm + kRowsTile * kRowsWarps;        // [warps][16]: sums
  float* bm = wl + kRowsTile * kRowsWarps;        // [16]: the block's maxima, then [16] sums
  __syncwarp();
  {
    float* part = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < VB; j += 4)
          *reinterpret_cast<float4*>(part + (g + 8 * i) * D + (2 * c + u) * VB + j) =
              make_float4(acc[j][2 * i + u], acc[j + 1][2 * i + u], acc[j + 2][2 * i + u],
                          acc[j + 3][2 * i + u]);
    if (c == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        wm[warp * kRowsTile + g + 8 * i] = m[i];
        wl[warp * kRowsTile + g + 8 * i] = l[i];
      }
    }
  }
  __syncthreads();
  constexpr int TPR = kRowsWarps * 32 / kRowsTile;  // threads per row
  const int jr = threadIdx.x / TPR, jc = threadIdx.x % TPR;
  {
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w) top = fmaxf(top, wm[w * kRowsTile + jr]);
    float f[kRowsWarps], sum = 0.f;
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w) {
      f[w] = top == -INFINITY ? 0.f : ajvp::ex2_approx(wm[w * kRowsTile + jr] - top);
      // a warp that saw no key has sum 0 and maximum -inf; NaN sums pass on
      sum += wl[w * kRowsTile + jr] * f[w];
    }
    for (int x = jc * 4; x < D; x += TPR * 4) {
      float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(smem + w * SLOT + (jr * D + x) * 4);
        r.x = fmaf(y.x, f[w], r.x), r.y = fmaf(y.y, f[w], r.y);
        r.z = fmaf(y.z, f[w], r.z), r.w = fmaf(y.w, f[w], r.w);
      }
      *reinterpret_cast<float4*>(whole + jr * D + x) = r;
    }
    if (jc == 0) {
      bm[jr] = top;
      bm[kRowsTile + jr] = sum;
    }
  }
  if (p.splits > 1)
    ajvp::cluster_sync_all();
  else
    __syncthreads();

  // Rank r of the cluster joins and writes rows r, r + splits, ...
  const uint32_t whole_addr = ajvp::smem_u32(whole), bm_addr = ajvp::smem_u32(bm);
  for (int item = threadIdx.x; item < kRowsTile * (D / 8); item += kRowsWarps * 32) {
    const int r = (item / (D / 8)) * 1, x = (item % (D / 8)) * 8;
    const int row = row0 + r;
    if (r % p.splits != rank || row >= rows) continue;
    float top = -INFINITY, sum = 0.f, y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < p.splits; ++k)
      top = fmaxf(top, ld_cluster_f32(ajvp::mapa_shared(bm_addr + r * 4, k)));
    for (int k = 0; k < p.splits; ++k) {
      const float mk = ld_cluster_f32(ajvp::mapa_shared(bm_addr + r * 4, k));
      const float f = top == -INFINITY ? 0.f : ajvp::ex2_approx(mk - top);
      sum = fmaf(ld_cluster_f32(ajvp::mapa_shared(bm_addr + (kRowsTile + r) * 4, k)), f, sum);
      const uint32_t at = ajvp::mapa_shared(whole_addr + (r * D + x) * 4, k);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fmaf(ld_cluster_f32(at + 4 * e), f, y[e]);
    }
    const int token = row / p.group, head = hk * p.group + row - token * p.group;
    const float inv = top == -INFINITY && sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= inv;
    T* dst = static_cast<T*>(p.o) + ((int64_t(b) * p.n + token) * p.H + head) * D + x;
    store8(dst, y);
    if (x == 0)
      p.lse[(int64_t(b) * p.H + head) * p.n + token] =
          top == -INFINITY && sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
  if (p.splits > 1) ajvp::cluster_sync_all();  // no block leaves while its sums are read
}

template <typename T, int D>
cudaError_t rows_launch(const CacheAttnParams& p, cudaStream_t st) {
  using C = RowsCfg<D>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(cache_rows_kernel<T, D>, C::BYTES, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B * p.Hkv * p.row_tiles * p.splits));
  cfg.blockDim = dim3(kRowsWarps * 32);
  cfg.dynamicSmemBytes = C::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_rows_kernel<T, D>, p);
}

cudaError_t cache_rows_launch(const CacheAttnParams& p, int d, int dtype, cudaStream_t st) {
  if (dtype == ATTN_JVP_BF16)
    return d == 128 ? rows_launch<__nv_bfloat16, 128>(p, st) : rows_launch<__nv_bfloat16, 64>(p, st);
  return d == 128 ? rows_launch<__half, 128>(p, st) : rows_launch<__half, 64>(p, st);
}

}  // namespace ajvp_serve

extern "C" int attn_jvp_cache_attn(const attn_jvp_shape* shape, int64_t Hkv, const void* q,
                                   const int64_t* q_strides, const attn_jvp_cache* cache,
                                   const int32_t* lens, const int32_t* table, int64_t table_width,
                                   int64_t table_stride, int64_t max_len, int32_t causal, void* o,
                                   float* lse, void* stream) {
  using namespace ajvp_serve;
  if (!shape || !q_strides) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  const attn_jvp_shape& s = *shape;
  if ((s.dtype != ATTN_JVP_BF16 && s.dtype != ATTN_JVP_F16) || (s.d != 64 && s.d != 128))
    return ATTN_JVP_ERR_UNSUPPORTED;
  if (s.B < 0 || s.B > 65535 || s.L < 0 || s.L > (1 << 24) || s.H < 1 || s.H > 65535 || Hkv < 1 ||
      s.H % Hkv || max_len < 0 || !(s.scale <= 0.f || std::isfinite(s.scale)))
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  int rc = check_cache(cache, Hkv, s.d);
  if (rc != ATTN_JVP_OK) return rc;
  if (table_width < 1 || table_width * cache->page_tokens > (int64_t(1) << 30) ||
      (s.B > 1 && table_stride < table_width))
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (s.B == 0 || s.L == 0) return ATTN_JVP_OK;
  if (!q || !lens || !table || !o || !lse) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(o) || (s.B > 1 && q_strides[0] % 8) ||
      (s.L > 1 && q_strides[1] % 8) || (s.H > 1 && q_strides[2] % 8))
    return ATTN_JVP_ERR_MISALIGNED;
  if ((s.B > 1 && q_strides[0] < 0) || (s.L > 1 && q_strides[1] < 0) || (s.H > 1 && q_strides[2] < 0))
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  CacheAttnParams p;
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
  const float scale = s.scale > 0.f ? s.scale : 1.0f / std::sqrt(static_cast<float>(s.d));
  p.scale_log2 = scale * 1.4426950408889634f;
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
  if (few)
    while (p.splits < 8 && tiles * p.splits < 2 * sms && len >= 256 * p.splits) p.splits *= 2;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = few ? cache_rows_launch(p, static_cast<int>(s.d), s.dtype, st)
                            : cache_tiles_launch(p, len, static_cast<int>(s.d), s.dtype, st);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? ATTN_JVP_OK : ATTN_JVP_ERR_CUDA;
}
