// attn_cache_tiles.cu - attention of many query rows over the paged e4m3 cache
// (C ABI attn_jvp_cache_attn) on tcgen05: chunks of tokens, or many query
// heads per key head. The formulas are those of attn_cache_rows.cu.
//
// Bound by the tensor cores (4 d operations per row and key) and the
// exponentials from some 200 rows per key head on, by HBM below. A block takes
// two tiles of 128 rows (the rows of a key head: token-major, then the heads
// of its group), as in attn_prompt.cu:
//   - warps 0-3 and 4-7: the softmax of the two row tiles, one thread per row.
//     A key's page scale multiplies its column of scores, its value scale goes
//     into the exponent; tokens come in groups of 16 of one page, so both cost
//     a few instructions per group;
//   - warp 8: issues the products, fp16 with fp32 sums (codes are exact);
//   - warp 9: copies the codes of a key tile by TMA, page by page, into a stage;
//   - warps 12-15: write them as fp16 into the swizzled ring that the tensor
//     core reads (warps 10 and 11 do nothing: registers are given out by four
//     warps).
// The key tiles are split over the blocks of a cluster where the row tiles are
// few or fill the SMs badly; the blocks join their sums through distributed
// shared memory, so there is one launch and no workspace.
//
// NaN values of tokens that some rows must not see are taken out of the
// product and marked, as in attn_prompt.cu; a row that sees a marked token
// gets NaN in its columns at the end.
#include <cuda.h>

#include "serve_attn.cuh"

#include <type_traits>

#include "serve_tiles.cuh"

namespace ajvp_serve {

namespace {

using namespace ajvp;

constexpr int kTilesThreads = 512;
constexpr int kGroup = 16;        // tokens that share a page for certain
constexpr int kScaleSlots = 8;    // key tiles whose scales are kept: more than the ring may run ahead

struct TilesParams {
  CUtensorMap map_k, map_v;  // codes (d, page tokens, heads, pages), boxes of a page's tokens
  CacheAttnParams c;
};

template <int D>
struct TilesCfg {
  static constexpr int TILE = kTile * D * 2;
  static constexpr int NS = D == 128 ? 4 : 8;   // ring slots, K and V tiles in turn
  static constexpr int RAW = D == 128 ? 2 : 4;  // stages of codes; the block has room for
  static constexpr int RAW_ONE = 4;             // so many if it has one row tile only
  static constexpr int RAW_AT = (2 + NS) * TILE;
  static constexpr int DATA = RAW_AT + RAW * TILE / 2;
  static constexpr int PITCH = D + 4;           // floats per row of the joined sums
  static constexpr int SCALES = kScaleSlots * (kTile / kGroup) * 16;
  // maxima and sums of the 256 rows, at the end, behind the joined sums
  static constexpr int STATS_AT = 2 * kTile * PITCH * 4;
  static constexpr int NBAR = 2 * NS + 5 * 2 + kScaleSlots + 2 * RAW_ONE + 2;
  static constexpr int BYTES = 1024 + DATA + SCALES + NBAR * 8 + 16 * 4 + 16;
  static constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;  // S_t at 128 t, O_t at 256 + D t
  static_assert(BYTES <= 232448, "shared memory budget");
  static_assert(STATS_AT + 2 * 2 * kTile * 4 <= DATA, "the joined sums lie over the tiles");
};

// The address with bits of its offset flipped (the base is aligned beyond them).
__device__ __forceinline__ const uint8_t* smem_xor(const uint8_t* p, uint32_t bits) {
  return reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(p) ^ bits);
}

// 64 scores of the lane's row.
__device__ __forceinline__ void load_scores(uint32_t taddr, uint32_t (&s)[64]) {
  tmem_ld32(taddr, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
  tmem_ld32(taddr + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
  tmem_wait_ld();
}

// What the softmax needs of the four groups of 64 scores.
struct Groups {
  float a[4];    // score = a * product + lv, in powers of two with the value scale
  float lv[4];   // log2 of the value scale; -inf for a group without a page
  float inv[4];  // 1 / value scale
  bool hidden;   // some group of the key tile has no page (the same for the whole block)
  __device__ __forceinline__ Groups(const float4* sc, float row_scale) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float4 f = sc[g];
      a[g] = row_scale * f.x, lv[g] = f.y, inv[g] = f.z;
      hidden = f.w != 0.f;
    }
  }
};

// Scores of tokens that the row does not see, from the left-th of 64 on or in
// a group without a page, become -inf.
__device__ __forceinline__ void hide(uint32_t (&s)[64], Groups& gr, int left) {
  if (left < 64) {
#pragma unroll
    for (int x = 0; x < 64; ++x)
      if (x >= left) s[x] = __float_as_uint(-INFINITY);
  }
  if (gr.hidden) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (gr.lv[g] == -INFINITY) {
        gr.lv[g] = 0.f;  // any finite addend will do
#pragma unroll
        for (int x = 0; x < kGroup; ++x) s[g * kGroup + x] = __float_as_uint(-INFINITY);
      }
  }
}

// Largest of 64 scores.
__device__ __forceinline__ float max_groups(const uint32_t (&s)[64], const Groups& gr) {
  float top[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float a = -INFINITY, c = -INFINITY;
#pragma unroll
    for (int x = 0; x < kGroup; x += 4) {
      const uint32_t* y = &s[g * kGroup + x];
      a = fmax3(a, __uint_as_float(y[0]), __uint_as_float(y[1]));
      c = fmax3(c, __uint_as_float(y[2]), __uint_as_float(y[3]));
    }
    top[g] = fmaf(fmaxf(a, c), gr.a[g], gr.lv[g]);
  }
  return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
}

// p = 2^(score - m) of 64 scores, packed in pairs; returns the sum of p / value
// scale.
__device__ __forceinline__ float exp_groups(const uint32_t (&s)[64], const Groups& gr, float m,
                                            uint32_t (&pk)[32]) {
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const float2 a2 = make_float2(gr.a[g], gr.a[g]);
    const float2 b2 = make_float2(gr.lv[g] - base, gr.lv[g] - base);
    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
    for (int x = 0; x < kGroup; x += 4) {
      const uint32_t* y = &s[g * kGroup + x];
      float2 u = __ffma2_rn(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), a2, b2);
      float2 v = __ffma2_rn(make_float2(__uint_as_float(y[2]), __uint_as_float(y[3])), a2, b2);
      u.x = ex2_approx(u.x), u.y = ex2_approx(u.y);
      v.x = ex2_approx(v.x), v.y = ex2_approx(v.y);
      sum0 = __fadd2_rn(sum0, u);
      sum1 = __fadd2_rn(sum1, v);
      pk[(g * kGroup + x) / 2] = pack_pair<true>(u.x, u.y);
      pk[(g * kGroup + x) / 2 + 1] = pack_pair<true>(v.x, v.y);
    }
    sum0 = __fadd2_rn(sum0, sum1);
    l = fmaf(sum0.x + sum0.y, gr.inv[g], l);
  }
  return l;
}

template <int D, typename T>
__global__ void __launch_bounds__(kTilesThreads, 1) cache_tiles_kernel(const __grid_constant__ TilesParams params) {
  using C = TilesCfg<D>;
  const CacheAttnParams& p = params.c;
  extern __shared__ uint8_t smem_raw[];
  // The same offset in every block of a cluster: the dynamic shared memory
  // starts at the same address in each.
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + 2 * C::TILE;
  // per group of a key tile: the key scale, log2 of the value scale (-inf: no
  // page), its inverse, and whether any group of the tile has no page
  float4* scales = reinterpret_cast<float4*>(smem + C::DATA);
  float* stats = reinterpret_cast<float*>(smem + C::STATS_AT);  // [256] maxima, [256] sums
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::DATA + C::SCALES);
  uint64_t* full = bars;                // [NS] ring slot written
  uint64_t* empty = bars + C::NS;       // [NS] ring slot read
  uint64_t* q_full = bars + 2 * C::NS;  // [2]
  uint64_t* s_full = q_full + 2;        // [2] scores of the row tile's current key tile
  uint64_t* p_full = q_full + 4;        // [2] its probabilities, first half
  uint64_t* p_late = q_full + 6;        // [2] second half
  uint64_t* pv_done = q_full + 8;       // [2] its sums
  uint64_t* sc_full = q_full + 10;       // [kScaleSlots] scales of a key tile
  uint64_t* raw_full = sc_full + kScaleSlots;    // [RAW_ONE] codes of a half tile landed
  uint64_t* raw_empty = raw_full + C::RAW_ONE;   // [RAW_ONE] codes read
  uint64_t* loaded = raw_empty + C::RAW_ONE;  // all tiles written, all marks made
  uint64_t* drain = loaded + 1;
  uint32_t* marked = reinterpret_cast<uint32_t*>(bars + C::NBAR);  // [4][4] tokens with NaN values
  uint32_t* tmem_slot = marked + 16;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tile = blockIdx.x / p.splits, rank = blockIdx.x - tile * p.splits;
  const int rt = tile % p.row_tiles, bh = tile / p.row_tiles;
  const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const int rows = p.n * p.group;
  const int row0 = rt * 2 * kTile;
  const int len = checked_len(p, b);
  const bool two = row0 + kTile < rows;  // the second row tile has rows
  const int last = min(row0 + 2 * kTile, rows) - 1;
  const int reach = p.causal ? max(len - p.n + last / p.group + 1, 0) : len;  // most keys seen
  const int all = p.causal ? max(len - p.n + row0 / p.group + 1, 0) : len;    // keys all rows see
  const int tiles = (reach + kTile - 1) / kTile;
  const int j_begin = static_cast<int>(int64_t(tiles) * rank / p.splits);
  const int j_end = static_cast<int>(int64_t(tiles) * (rank + 1) / p.splits);
  const int n = j_end - j_begin;  // key tiles of this block; may be 0
  const int first_edge = all / kTile;  // key tiles from here on have hidden tokens

  const int warp = warp_uniform(static_cast<int>(threadIdx.x >> 5));
  const int lane = threadIdx.x & 31;
  auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return warp_wait(bar, parity, abort_flag, p.status);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&full[i], 4);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&p_late[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) mbar_init(&sc_full[i], 1);
    for (int i = 0; i < C::RAW_ONE; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    mbar_init(loaded, 4);
    mbar_init(drain, 1);
    for (int i = 0; i < 16; ++i) marked[i] = 0;
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(warp_uniform(static_cast<int>(*tmem_slot)));

  const int stages = two ? C::RAW : C::RAW_ONE;
  auto stage_at = [&](int s) {  // the second row tile's queries' place is free without one
    return s < C::RAW ? smem + C::RAW_AT + s * (C::TILE / 2)
                      : sQ + C::TILE + (s - C::RAW) * (C::TILE / 2);
  };

  if (warp >= 8 && warp < 12) {
    setmaxnreg_dec<88>();
    if (warp == 8) {
      // ------------------------------------------------------------ products
      // As in attn_prompt.cu, with both row tiles over the same key tiles.
      const uint32_t idesc_s = tile_idesc<true>(kTile, kTile, 0);
      const uint32_t idesc_v = tile_idesc<true>(kTile, D, 1);
      const uint32_t aQ = smem_u32(sQ), aR = smem_u32(sRing);
      const int nt = two ? 2 : 1;
      auto slot_addr = [&](int i) { return aR + (i % C::NS) * C::TILE; };
      auto landed = [&](int i) { return wwait(&full[i % C::NS], (i / C::NS) & 1); };
      auto scores = [&](int t, int j) {
        mma_scores<D, kTile, kTile, false>(tmem + C::TM_S + kTile * t, aQ + t * C::TILE,
                                           slot_addr(2 * j), idesc_s, false);
        umma_commit(&s_full[t]);
      };
      bool ok = n > 0 && landed(0);
      for (int t = 0; ok && t < nt; ++t) {
        ok = wwait(&q_full[t], 0);
        tc_fence_after();
        if (ok) scores(t, 0);
      }
      if (ok) umma_commit(&empty[0]);
      for (int j = 0; ok && j < n; ++j) {
        const int vi = 2 * j + 1, ki = 2 * j + 2;
        ok = landed(vi);
        for (int t = 0; ok && t < nt; ++t) {
          ok = wwait(&p_full[t], j & 1);
          if (!ok) break;
          tc_fence_after();
          mma_values_half<D, 0>(tmem + C::TM_O + D * t, tmem + C::TM_S + kTile * t, slot_addr(vi),
                                idesc_v, j > 0);
          if (t == 0 && j + 1 < n) ok = landed(ki);
          ok = ok && wwait(&p_late[t], j & 1);
          if (!ok) break;
          tc_fence_after();
          mma_values_half<D, 1>(tmem + C::TM_O + D * t, tmem + C::TM_S + kTile * t, slot_addr(vi),
                                idesc_v, true);
          umma_commit(&pv_done[t]);
          if (j + 1 < n) scores(t, j + 1);
        }
        if (!ok) break;
        umma_commit(&empty[vi % C::NS]);
        if (j + 1 < n) umma_commit(&empty[ki % C::NS]);
      }
      umma_commit(drain);  // every product ends before tensor memory is released
      if (lane == 0) mbar_wait_drain(drain, 0, 1000000000ull);
      __syncwarp();
    } else if (warp == 9) {
      // ------------------------------------------------------------ copies
      // Half tile i is the keys (even i) or values (odd) of key tile i / 2. Its
      // codes are copied page by page into a stage.
      // Pages of the eight groups of 16 tokens of a key tile, one per lane. They
      // are loaded a tile before they are used, and looked at then: -1 if hidden.
      const int32_t* table = p.table + b * p.table_stride;
      int raw_page = -1, page = -1;
      auto load_page = [&](int j) {
        const int token = (j_begin + j) * kTile + lane * kGroup;
        raw_page = lane < kTile / kGroup && j < n && token < reach ? table[token >> p.page_shift] : -1;
      };
      load_page(0);
      float2 sc = make_float2(0.f, 0.f);
      int i = 0;
      for (; i < 2 * n; ++i) {
        const int j = i >> 1, st = i % stages;
        if (i & 1) {
          // the scales, read before the keys' copies, are there by now
          const float some = __any_sync(0xffffffffu, lane < kTile / kGroup && page < 0);
          if (lane < kTile / kGroup) {
            float4 f = make_float4(1.f, -INFINITY, 1.f, some);  // hidden
            if (page >= 0) {
              const float vs = read_scale(sc.y);
              f = make_float4(read_scale(sc.x), log2_approx(vs), rcp_approx(vs), some);
            }
            scales[(j % kScaleSlots) * (kTile / kGroup) + lane] = f;
          }
          __syncwarp();
          mbar_arrive_if(&sc_full[j % kScaleSlots], lane == 0);
        } else {
          const int token = (j_begin + j) * kTile + lane * kGroup;
          page = raw_page >= 0 && raw_page < p.pages ? raw_page : -1;
          if (page < 0 && lane < kTile / kGroup && token < reach) atomicOr(p.status, kStatusBadIndex);
          if (page >= 0) {
            const int64_t at = page * p.scale_page + hk * p.scale_head;
            sc = make_float2(p.scale[0][at], p.scale[1][at]);
          }
          load_page(j + 1);
        }
        if (!wwait(&raw_empty[st], ((i / stages) & 1) ^ 1)) break;
        const bool box = page >= 0 && ((lane * kGroup) & ((1 << p.page_shift) - 1)) == 0;
        const int boxes = __popc(__ballot_sync(0xffffffffu, box));
        if (lane == 0) mbar_arrive_expect_tx(&raw_full[st], boxes * (D << p.page_shift));
        __syncwarp();
        if (box)
          tma_load_4d(stage_at(st) + lane * kGroup * D, (i & 1) ? &params.map_v : &params.map_k,
                      &raw_full[st], 0, 0, hk, page);
        __syncwarp();
      }
      // after an abort: every copy issued lands before the block ends
      if (i < 2 * n)
        for (int k = max(i - stages, 0); k < i; ++k)
          mbar_wait_drain(&raw_full[k % stages], (k / stages) & 1, 200000000ull);
    }
  } else if (warp >= 12) {
    setmaxnreg_dec<96>();
    // -------------------------------------------------------------- codes to fp16
    // Each lane takes 16 codes of a token at a time. A quarter warp takes four
    // adjacent ones of two rows whose places differ in bits 0 and 2, which puts
    // its reads (of rows swizzled by the copies) and its writes (of the ring's
    // swizzled rows) on all banks; a warp takes 8 rows at a time.
    constexpr int CH = D / 64;            // 64-column parts
    constexpr int COUNT = 4 * CH;         // pieces of a lane: 16 blocks of 8 rows, 4 warps
    const int r7 = (lane >> 3) ^ ((lane & 4) ? 5 : 0), q = lane & 3;
    const int from_at = D == 128 ? r7 * 128 + ((q ^ r7) << 4) : r7 * 64 + ((q ^ ((r7 >> 1) & 3)) << 4);
    const int to_lo = r7 * 128 + (((2 * q) ^ r7) << 4), to_hi = r7 * 128 + (((2 * q + 1) ^ r7) << 4);
    uint32_t hidden = 0;  // groups of the key tile without a page
    for (int i = 0; i < 2 * n; ++i) {
      const int slot = i % C::NS, st = i % stages, j = j_begin + (i >> 1);
      if (!(i & 1)) {
        const int k = (i >> 1) % kScaleSlots;
        if (!wwait(&sc_full[k], ((i >> 1) / kScaleSlots) & 1)) break;
        hidden = __ballot_sync(0xffffffffu,
                               lane < kTile / kGroup &&
                                   scales[k * (kTile / kGroup) + lane % (kTile / kGroup)].y == -INFINITY);
      }
      if (!wwait(&raw_full[st], (i / stages) & 1)) break;
      const uint8_t* from = stage_at(st) + from_at;
      // all pieces are read before the first is written: the compiler cannot
      // tell the two places apart
      uint4 u[COUNT];
#pragma unroll
      for (int k = 0; k < COUNT; ++k) {
        const int block = (k / CH) * 4 + warp - 12;
        // the second part of a 128-byte row: chunk 4 + q, so bit 2 of its place
        u[k] = *reinterpret_cast<const uint4*>(D == 128 ? smem_xor(from + block * 1024, (k % CH) << 6)
                                                        : from + block * 512);
      }
      __syncwarp();
      mbar_arrive_if(&raw_empty[st], lane == 0);
      // tokens that nobody sees, or without a page, become zeros
      const int left = reach - j * kTile;
      if (left < kTile || hidden != 0) {
#pragma unroll
        for (int k = 0; k < COUNT; ++k) {
          const int r = ((k / CH) * 4 + warp - 12) * 8 + r7;
          if (r >= left || ((hidden >> (r / kGroup)) & 1u)) u[k] = make_uint4(0, 0, 0, 0);
        }
      }
      if ((i & 1) && j >= first_edge) {
#pragma unroll
        for (int k = 0; k < COUNT; ++k) {
          const int r = ((k / CH) * 4 + warp - 12) * 8 + r7;
          uint32_t* w = reinterpret_cast<uint32_t*>(&u[k]);
          bool nan = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t m = (((w[e] & 0x7f7f7f7fu) + 0x01010101u) >> 7) & 0x01010101u;
            nan |= m != 0;
            w[e] &= ~(m * 0xffu);
          }
          if (nan) atomicOr(&marked[4 * (j - first_edge) + (r >> 5)], 1u << (r & 31));
        }
      }
      if (!wwait(&empty[slot], ((i / C::NS) & 1) ^ 1)) break;
      uint8_t* to = sRing + slot * C::TILE;
#pragma unroll
      for (int k = 0; k < COUNT; ++k) {
        const int block = (k / CH) * 4 + warp - 12;
        uint32_t h[8];
        e4m3x4_to_f16x4(u[k].x, h[0], h[1]);
        e4m3x4_to_f16x4(u[k].y, h[2], h[3]);
        e4m3x4_to_f16x4(u[k].z, h[4], h[5]);
        e4m3x4_to_f16x4(u[k].w, h[6], h[7]);
        uint8_t* part = to + (k % CH) * kTile * 128 + block * 1024;
        *reinterpret_cast<uint4*>(part + to_lo) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(part + to_hi) = make_uint4(h[4], h[5], h[6], h[7]);
      }
      fence_proxy_async_shared();
      __syncwarp();
      mbar_arrive_if(&full[slot], lane == 0);
    }
    __syncwarp();
    mbar_arrive_if(loaded, lane == 0);
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<160>();
    const int t = warp >> 2, sub = warp & 3;
    const int row = sub * 32 + lane;
    const int r = row0 + t * kTile + row;  // row of the key head
    const bool mine = r < rows;
    const int token = min(r, rows - 1) / p.group, head = hk * p.group + min(r, rows - 1) - token * p.group;
    const int seen = p.causal ? max(len - p.n + token + 1, 0) : len;
    const bool active = t == 0 || two;
    const uint32_t lane_off = static_cast<uint32_t>(sub * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::TM_S + kTile * t;
    const uint32_t tO = tmem + lane_off + C::TM_O + D * t;
    float row_scale = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    if (active && n > 0) {
      // this row's query as fp16, bf16 scaled by a power of two (see attn_cache_rows.cu)
      const T* src = static_cast<const T*>(p.q) + b * p.q_seq + token * p.q_token + head * p.q_head;
      float inv = 1.f;
      if constexpr (!std::is_same<T, __half>::value) {
        float amax = 0.f;
#pragma unroll 4
        for (int x = 0; x < D; x += 8) {
          float y[8];
          load8(src + x, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = fabsf(y[e]);
            amax = fmaxf(amax, a < INFINITY ? a : 0.f);
          }
        }
        int e = 0;
        if (amax > 0.f) frexpf(amax, &e);
        e = min(max(e, -100), 100);
        inv = ldexpf(1.f, -e);
        row_scale *= ldexpf(1.f, e);
      }
#pragma unroll 4
      for (int x = 0; x < D; x += 8) {
        float y[8];
        load8(src + x, y);
        uint4 u;
        u.x = Elem<__half>::pack(y[0] * inv, y[1] * inv);
        u.y = Elem<__half>::pack(y[2] * inv, y[3] * inv);
        u.z = Elem<__half>::pack(y[4] * inv, y[5] * inv);
        u.w = Elem<__half>::pack(y[6] * inv, y[7] * inv);
        *reinterpret_cast<uint4*>(sQ + t * C::TILE + (x >> 6) * kTile * 128 + row * 128 +
                                  ((((x >> 3) & 7) ^ (row & 7)) << 4)) = u;
      }
      fence_proxy_async_shared();
      __syncwarp();
      mbar_arrive_if(&q_full[t], lane == 0);
    }
    for (int j = 0; active && j < n; ++j) {
      if (!wwait(&sc_full[j % kScaleSlots], (j / kScaleSlots) & 1) || !wwait(&s_full[t], j & 1) ||
          (j > 0 && !wwait(&pv_done[t], (j - 1) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float4* sc = scales + (j % kScaleSlots) * (kTile / kGroup);
      const int left = j_begin + j >= first_edge ? seen - (j_begin + j) * kTile : kTile;
      // As in attn_prompt.cu: the first half's probabilities are formed at the
      // running maximum while the row's largest score is being found, and
      // again only if that is much larger. The scores stay in tensor memory
      // until then, and 64 at a time in registers.
      uint32_t s[64], pk[32];
      float top, add;
      load_scores(tS, s);
      Groups gr(sc, row_scale);
      hide(s, gr, left);
      top = max_groups(s, gr);
      add = exp_groups(s, gr, m, pk);
      load_scores(tS + 64, s);
      Groups late(sc + 4, row_scale);
      hide(s, late, left - 64);
      top = fmaxf(top, max_groups(s, late));
      if (__any_sync(0xffffffffu, top > m + kLazyMax)) {
        const float to = fmaxf(m, top);
        const float f = to == -INFINITY ? 1.f : ex2_approx(m - to);
        m = to;
        l *= f;
        if (j > 0) rescale_sums<D>(tO, f);
        load_scores(tS, s);
        gr = Groups(sc, row_scale);
        hide(s, gr, left);
        add = exp_groups(s, gr, m, pk);
        load_scores(tS + 64, s);
        late = Groups(sc + 4, row_scale);
        hide(s, late, left - 64);
      }
      tmem_st32(tS, pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_if(&p_full[t], lane == 0);
      add += exp_groups(s, late, m, pk);
      tmem_st32(tS + 32, pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_if(&p_late[t], lane == 0);
      l += add;
    }
    // ---------------------------------------------------------- sums
    ok = ok && active && (n == 0 || wwait(&pv_done[t], (n - 1) & 1)) && wwait(loaded, 0);
    // the sums to be joined lie over the operands: the other row tile's products are done with them
    if (ok && p.splits > 1) ok = wwait(drain, 0);
    if (ok) {
      tc_fence_after();
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) any |= marked[i];
      const bool none = l == 0.f;  // no key seen (a NaN sum is not 0)
      const float inv = p.splits > 1 ? 1.f : none ? 0.f : 1.f / l;
      float* part = reinterpret_cast<float*>(smem) + (t * kTile + row) * C::PITCH;
      T* dst = static_cast<T*>(p.o) + ((int64_t(b) * p.n + token) * p.H + head) * D;
#pragma unroll 1
      for (int x = 0; x < D; x += 32) {
        uint32_t y[32];
        if (n > 0) {
          tmem_ld32(tO + x, y);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) y[c] = 0;
        }
        if (any && mine) {
          for (int key = first_edge * kTile; key < seen; ++key) {
            const int k = key - first_edge * kTile;
            if (!((marked[k >> 5] >> (k & 31)) & 1u)) continue;
            const uint8_t* v = p.codes[1] + p.table[b * p.table_stride + (key >> p.page_shift)] * p.page_stride +
                               hk * p.head_stride +
                               (key & ((1 << p.page_shift) - 1)) * p.token_stride + x;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if ((v[c] & 0x7fu) == 0x7fu) y[c] = 0x7fffffffu;
          }
        }
        if (p.splits > 1) {
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            *reinterpret_cast<uint4*>(part + x + c) = make_uint4(y[c], y[c + 1], y[c + 2], y[c + 3]);
        } else if (mine) {
#pragma unroll
          for (int c = 0; c < 32; c += 8) {
            float z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = none ? 0.f : __uint_as_float(y[c + e]) * inv;
            store8(dst + x + c, z);
          }
        }
      }
      if (p.splits > 1) {
        stats[t * kTile + row] = m;
        stats[2 * kTile + t * kTile + row] = l;
      } else if (mine) {
        p.lse[(int64_t(b) * p.H + head) * p.n + token] = none ? -INFINITY : (m + log2f(l)) * kLn2;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, C::TM_COLS);
  if (p.splits == 1) return;

  // ------------------------------------------------------------ join
  // Block `rank` of the cluster joins every splits-th row, a warp per row.
  cluster_sync_all();
  const uint32_t part = smem_u32(smem), st = smem_u32(stats);
  constexpr int kLanes = D / 4;  // lanes of a row
  const int at = lane % kLanes;
  const int sub_row = (warp * 32 + lane) / kLanes;
  constexpr int kRows = kTilesThreads / kLanes;  // rows in flight
  for (int i = rank + sub_row * p.splits; i < min(2 * kTile, rows - row0); i += kRows * p.splits) {
    float top = -INFINITY, sum = 0.f;
    for (int k = 0; k < p.splits; ++k) top = fmaxf(top, ld_cluster_f32(mapa_shared(st + i * 4, k)));
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < p.splits; ++k) {
      const float mk = ld_cluster_f32(mapa_shared(st + i * 4, k));
      const float f = top == -INFINITY ? 1.f : ex2_approx(mk - top);
      const float4 z = ld_cluster_f32x4(mapa_shared(part + (i * C::PITCH + 4 * at) * 4, k));
      sum = fmaf(ld_cluster_f32(mapa_shared(st + (2 * kTile + i) * 4, k)), f, sum);
      y.x = fmaf(z.x, f, y.x), y.y = fmaf(z.y, f, y.y);
      y.z = fmaf(z.z, f, y.z), y.w = fmaf(z.w, f, y.w);
    }
    const int r = row0 + i, token = r / p.group, head = hk * p.group + r - token * p.group;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    T* dst = static_cast<T*>(p.o) + ((int64_t(b) * p.n + token) * p.H + head) * D + 4 * at;
    uint2 u;
    u.x = pack_pair<std::is_same<T, __half>::value>(y.x * inv, y.y * inv);
    u.y = pack_pair<std::is_same<T, __half>::value>(y.z * inv, y.w * inv);
    *reinterpret_cast<uint2*>(dst) = u;
    if (at == 0)
      p.lse[(int64_t(b) * p.H + head) * p.n + token] =
          sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
  cluster_sync_all();  // no block leaves while its sums are read
}

template <int D, typename T>
struct TilesKernel {
  static cudaError_t prepare() {
    static std::atomic<uint64_t> done{0};
    return allow_smem(cache_tiles_kernel<D, T>, TilesCfg<D>::BYTES, done);
  }
  static void config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int blocks, int splits,
                     cudaStream_t st) {
    cfg->gridDim = dim3(static_cast<unsigned>(blocks));
    cfg->blockDim = dim3(kTilesThreads);
    cfg->dynamicSmemBytes = TilesCfg<D>::BYTES;
    cfg->stream = st;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = splits;
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cfg->attrs = attr;
    cfg->numAttrs = 1;
  }
  // Clusters of k blocks resident at once, k = 1 .. 8: asked for once per device.
  static cudaError_t clusters(int (&at_once)[9]) {
    static std::atomic<int> known[64][9];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = prepare()) != cudaSuccess) return e;
    for (int k = 1; k <= 8; ++k) {
      int n = known[dev & 63][k].load(std::memory_order_relaxed);
      if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr;
        config(&cfg, &attr, k, k, nullptr);
        e = cudaOccupancyMaxActiveClusters(&n, cache_tiles_kernel<D, T>, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) n = 1;
        known[dev & 63][k].store(n, std::memory_order_relaxed);
      }
      at_once[k] = n;
    }
    return cudaSuccess;
  }
  static cudaError_t launch(TilesParams& params, int64_t keys, cudaStream_t st) {
    CacheAttnParams& p = params.c;
    // The number of splits that ends first, in key tiles per block and round
    // of the clusters that run at once: clusters above 2 leave some SMs out
    // (15 clusters of 8 fit, but 74 of 2). A block takes about 2 tiles' time to
    // start and end, the join about 3 more.
    int at_once[9];
    cudaError_t err = clusters(at_once);
    if (err != cudaSuccess) return err;
    const int64_t tiles = int64_t(p.B) * p.Hkv * p.row_tiles, len = (keys + kTile - 1) / kTile;
    int64_t best = INT64_MAX;
    for (int k = 1; k <= 8 && (k == 1 || 2 * k <= len); ++k) {
      const int64_t rounds = (tiles + at_once[k] - 1) / at_once[k];
      const int64_t cost = rounds * ((len + k - 1) / k + 2 + (k > 1 ? 3 : 0));
      if (cost < best) best = cost, p.splits = k;
    }
    cudaError_t e = prepare();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    config(&cfg, &attr, p.B * p.Hkv * p.row_tiles * p.splits, p.splits, st);
    return cudaLaunchKernelEx(&cfg, cache_tiles_kernel<D, T>, params);
  }
};

}  // namespace

cudaError_t cache_tiles_launch(const CacheAttnParams& p, int64_t keys, int d, int dtype, cudaStream_t st) {
  TilesParams t;
  t.c = p;
  const int page = 1 << p.page_shift;
  if (!encode_cache_map(&t.map_k, p.codes[0], d, page, p.Hkv, p.pages, p.token_stride, p.head_stride,
                        p.page_stride, page) ||
      !encode_cache_map(&t.map_v, p.codes[1], d, page, p.Hkv, p.pages, p.token_stride, p.head_stride,
                        p.page_stride, page))
    return cudaErrorInvalidValue;
  if (dtype == ATTN_JVP_BF16)
    return d == 128 ? TilesKernel<128, __nv_bfloat16>::launch(t, keys, st)
                    : TilesKernel<64, __nv_bfloat16>::launch(t, keys, st);
  return d == 128 ? TilesKernel<128, __half>::launch(t, keys, st)
                  : TilesKernel<64, __half>::launch(t, keys, st);
}

}  // namespace ajvp_serve
