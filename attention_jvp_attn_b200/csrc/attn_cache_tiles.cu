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
// The key tiles of all sequences, heads and row tile pairs in a row are shared
// out evenly, as in attn_cache_rows.cu: whatever the shapes, every SM has the
// same number of tiles, give or take one. Partial sums go to the workspace and
// a second, small kernel joins them.
//
// Measured (one B200): 1,560 queries over 32,760 tokens, 12 heads, d = 128, 314
// GFLOP: 409 to 426 us, 740 to 770 TFLOP/s (418 at a median of 1,935 MHz), causal
// or not; 1,536 queries, which fill their row tiles, 359 us. The bound is the chain
// scores -> softmax -> products of a row tile, 4,100 to 4,600 cycles per key tile
// against 2,048 of tensor work; the conversion is beside it (without it the time is
// the same). With one row tile (17 to 128 rows) nothing runs beside that chain: see
// Share in attn_cache_rows.cu.
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
constexpr int kLeastTiles = 2;    // key tiles of a block that takes part
constexpr int kGroup = 16;        // tokens that share a page for certain
constexpr int kScaleSlots = 8;    // key tiles whose scales are kept: more than the ring may run ahead

struct TilesParams {
  CUtensorMap map_k, map_v;  // codes (d, page tokens, heads, pages), boxes of a page's tokens
  CacheAttnParams c;
  float* work;  // sums of partial pieces, two places per block, and the pieces
  int blocks;
};

template <int D>
struct TilesCfg {
  static constexpr int TILE = kTile * D * 2;
  static constexpr int NS = D == 128 ? 4 : 8;   // ring slots, K and V tiles in turn
  static constexpr int RAW = D == 128 ? 2 : 4;  // stages of codes; the block has room for
  static constexpr int RAW_ONE = 4;             // so many if it has one row tile only
  static constexpr int RAW_AT = (2 + NS) * TILE;
  static constexpr int DATA = RAW_AT + RAW * TILE / 2;
  static constexpr int SCALES = kScaleSlots * (kTile / kGroup) * 16;
  static constexpr int NBAR = 2 * NS + 6 * 2 + kScaleSlots + 2 * RAW_ONE + 2;
  static constexpr int BYTES = 1024 + DATA + SCALES + NBAR * 8 + 16 * 4 + 16;
  static constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;  // S_t at 128 t, O_t at 256 + D t
  static_assert(BYTES <= 232448, "shared memory budget");
  // a place of the workspace: sums of the 256 rows, four columns of all rows
  // after one another (so that a warp's rows lie together), then maxima and
  // sums of p
  static constexpr int PLACE = 2 * kTile * (D + 2);
};

// Key tiles that a row tile pair of a sequence of `len` tokens reaches; one at
// least, in which rows without keys are written.
__device__ __forceinline__ int reach_of(const CacheAttnParams& p, int len, int rt) {
  const int last = min((rt + 1) * 2 * kTile, p.n * p.group) - 1;
  return p.causal ? max(len - p.n + last / p.group + 1, 0) : len;
}
__device__ __forceinline__ int tiles_of(const CacheAttnParams& p, int len, int rt) {
  return max((reach_of(p, len, rt) + kTile - 1) / kTile, 1);
}
__device__ __forceinline__ int64_t head_steps(const CacheAttnParams& p, int len) {
  if (!p.causal) return int64_t(p.row_tiles) * tiles_of(p, len, 0);
  int64_t x = 0;
  for (int i = 0; i < p.row_tiles; ++i) x += tiles_of(p, len, i);
  return x;
}

// The block's current piece, in shared memory (it would cost every role some
// twenty registers): key tiles [j_begin, j_begin + n) of sequence b, key head hk
// and row tile pair rt. One thread moves it on.
struct Current {
  int64_t w, w_end, base;  // steps from w on are left; base: the row tile pair's first step
  int b, hk, rt;
  int index, done;         // pieces, and key tiles, before this one
  int twos, two_done;      // those that had a second row tile
  int len, reach, first_edge, j_begin, n;
  int two, whole, valid;

  __device__ void start(const CacheAttnParams& p, int64_t all, int b_, int64_t before, int64_t blocks) {
    index = done = twos = two_done = 0;
    w = all * blockIdx.x / blocks;
    w_end = all * (blockIdx.x + 1) / blocks;
    b = b_;
    base = before;
    len = checked_len(p, b);
    const int64_t per = head_steps(p, len);
    hk = static_cast<int>((w - base) / per);
    base += hk * per;
    for (rt = 0; rt + 1 < p.row_tiles; ++rt) {
      const int x = tiles_of(p, len, rt);
      if (w < base + x) break;
      base += x;
    }
    look(p);
  }
  __device__ int number(const CacheAttnParams& p) const { return (b * p.Hkv + hk) * p.row_tiles + rt; }
  __device__ void look(const CacheAttnParams& p) {
    valid = w < w_end;
    if (!valid) return;
    const int tiles = tiles_of(p, len, rt);
    reach = reach_of(p, len, rt);
    const int all = p.causal ? max(len - p.n + rt * 2 * kTile / p.group + 1, 0) : len;
    first_edge = all / kTile;  // key tiles from here on have hidden tokens
    j_begin = static_cast<int>(w - base);
    n = static_cast<int>(min(w_end - base, int64_t(tiles))) - j_begin;
    two = rt * 2 * kTile + kTile < p.n * p.group;
    whole = n == tiles;
  }
  __device__ void next(const CacheAttnParams& p) {
    ++index;
    done += n;
    if (two) ++twos, two_done += n;
    w += n;
    base = w;
    if (w < w_end && ++rt == p.row_tiles) {
      rt = 0;
      if (++hk == p.Hkv) {
        hk = 0;
        ++b;
        len = checked_len(p, b);
      }
    }
    look(p);
  }
};

// The address with bits of its offset flipped (the base is aligned beyond them).
__device__ __forceinline__ uint8_t* smem_xor(uint8_t* p, uint32_t bits) {
  return reinterpret_cast<uint8_t*>(reinterpret_cast<uintptr_t>(p) ^ bits);
}

// What the softmax needs of the four groups of 64 scores.
struct Groups {
  float a[4];    // score = a * product + lv, in powers of two with the value scale
  float lv[4];   // log2 of the value scale
  float inv[4];  // 1 / value scale
  __device__ __forceinline__ Groups(const float4* sc, float row_scale) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float4 f = sc[g];
      // a group without a page has scores of -inf, and any finite addend will do
      a[g] = row_scale * f.x, lv[g] = fmaxf(f.y, -64.f), inv[g] = f.z;
    }
  }
};

// Scores of tokens that the row does not see, from the left-th of 64 on or in a
// group without a page, become -inf. In tensor memory, a group at a time:
// seldom needed, so its code is kept small.
__device__ __forceinline__ void hide(uint32_t taddr, const float4* sc, int left) {
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    const int here = sc[g].y == -INFINITY ? 0 : left - 16 * g;
    uint32_t s[16];
    ajvp::tmem_ld16(taddr + 16 * g, s);
    ajvp::tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 16; ++x)
      if (x >= here) s[x] = __float_as_uint(-INFINITY);
    ajvp::tmem_st16(taddr + 16 * g, s);
  }
  ajvp::tmem_wait_st();
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
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + 2 * C::TILE;
  // per group of a key tile: the key scale, log2 of the value scale (-inf: no
  // page), its inverse, and whether any group of the tile has no page
  float4* scales = reinterpret_cast<float4*>(smem + C::DATA);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::DATA + C::SCALES);
  uint64_t* full = bars;                // [NS] ring slot written
  uint64_t* empty = bars + C::NS;       // [NS] ring slot read
  uint64_t* q_full = bars + 2 * C::NS;  // [2]
  uint64_t* s_full = q_full + 2;        // [2] scores of the row tile's current key tile
  uint64_t* p_full = q_full + 4;        // [2] its probabilities, first half
  uint64_t* p_late = q_full + 6;        // [2] second half
  uint64_t* pv_done = q_full + 8;       // [2] its sums
  uint64_t* pv_half = q_full + 10;      // [2] its sums over the first half
  uint64_t* sc_full = q_full + 12;      // [kScaleSlots] scales of a key tile
  uint64_t* raw_full = sc_full + kScaleSlots;    // [RAW_ONE] codes of a half tile landed
  uint64_t* raw_empty = raw_full + C::RAW_ONE;   // [RAW_ONE] codes read
  uint64_t* loaded = raw_empty + C::RAW_ONE;  // all tiles written, all marks made
  uint64_t* drain = loaded + 1;
  uint32_t* marked = reinterpret_cast<uint32_t*>(bars + C::NBAR);  // [4][4] tokens with NaN values
  uint32_t* tmem_slot = marked + 16;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int rows = p.n * p.group;
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
      mbar_init(&pv_half[i], 1);
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
  __shared__ Current pc;
  __shared__ Piece left;  // what the join will know of this block
  {
    int64_t blocks = params.blocks, all, before;
    int b;
    find_step<kTilesThreads>(
        p.B, blockIdx.x, kLeastTiles, [&](int i) { return p.Hkv * head_steps(p, checked_len(p, i)); },
        blocks, all, b, before);
    if (threadIdx.x == 0) {
      pc.valid = 0;
      if (blockIdx.x < blocks) pc.start(p, all, b, before, blocks);
      left = {Piece::kNone, Piece::kNone, 0, 0};
    }
    __syncthreads();
  }
  const uint32_t tmem = static_cast<uint32_t>(warp_uniform(static_cast<int>(*tmem_slot)));

  // The end of a piece for the whole block: queries, ring and marks are free for
  // the next one (none after an abort).
  auto end_piece = [&]() {
    tc_fence_before();
    named_bar_sync(1, kTilesThreads);
    tc_fence_after();
    if (threadIdx.x < 16) marked[threadIdx.x] = 0;
    if (threadIdx.x == kTilesThreads - 1) {
      if (!pc.whole) {
        if (pc.j_begin > 0)
          left.went_on = pc.number(p);
        else
          left.begun = pc.number(p), left.place = pc.index ? 1 : 0;
      }
      pc.next(p);
      if (*abort_flag) pc.valid = 0;
    }
    named_bar_sync(1, kTilesThreads);
  };

  // Without a second row tile its queries' place is free for stages of codes.
  const int stages = rows > kTile ? C::RAW : C::RAW_ONE;
  auto stage_at = [&](int s) {
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
      auto slot_addr = [&](int i) { return aR + (i % C::NS) * C::TILE; };
      auto landed = [&](int i) { return wwait(&full[i % C::NS], (i / C::NS) & 1); };
      auto scores = [&](int t, int j) {
        mma_scores<D, kTile, kTile, false>(tmem + C::TM_S + kTile * t, aQ + t * C::TILE,
                                           slot_addr(2 * j), idesc_s, false);
        umma_commit(&s_full[t]);
      };
      while (warp_uniform(pc.valid)) {
        const int nt = warp_uniform(pc.two ? 2 : 1), j0 = warp_uniform(pc.done), j1 = j0 + warp_uniform(pc.n);
        const int index = warp_uniform(pc.index), twos = warp_uniform(pc.twos);
        const int shift = warp_uniform(pc.two_done) - j0;
        bool ok = landed(2 * j0);
        for (int t = 0; ok && t < nt; ++t) {
          ok = wwait(&q_full[t], (t ? twos : index) & 1);
          tc_fence_after();
          if (ok) scores(t, j0);
        }
        if (ok) umma_commit(&empty[2 * j0 % C::NS]);
        for (int j = j0; ok && j < j1; ++j) {
          const int vi = 2 * j + 1, ki = 2 * j + 2;
          ok = landed(vi);
          for (int t = 0; ok && t < nt; ++t) {
            const int phase = (t ? j + shift : j) & 1;
            ok = wwait(&p_full[t], phase);
            if (!ok) break;
            tc_fence_after();
            mma_values_half<D, 0>(tmem + C::TM_O + D * t, tmem + C::TM_S + kTile * t, slot_addr(vi),
                                  idesc_v, j > j0);
            if (t == 0 && j + 1 < j1) ok = landed(ki);
            umma_commit(&pv_half[t]);
            ok = ok && wwait(&p_late[t], phase);
            if (!ok) break;
            tc_fence_after();
            mma_values_half<D, 1>(tmem + C::TM_O + D * t, tmem + C::TM_S + kTile * t, slot_addr(vi),
                                  idesc_v, true);
            umma_commit(&pv_done[t]);
            if (j + 1 < j1) scores(t, j + 1);
          }
          if (!ok) break;
          umma_commit(&empty[vi % C::NS]);
          if (j + 1 < j1) umma_commit(&empty[ki % C::NS]);
        }
        umma_commit(drain);  // every product ends before the piece does
        if (lane == 0) mbar_wait_drain(drain, index & 1, 1000000000ull);
        __syncwarp();
        end_piece();
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------ copies
      // Half tile i is the keys (even i) or values (odd) of key tile i / 2. Its
      // codes are copied page by page into a stage.
      // Pages of the eight groups of 16 tokens of a key tile, one per lane. They
      // are loaded a tile before they are used, and looked at then: -1 if hidden.
      while (pc.valid) {
        const int n = pc.n, done = pc.done, reach = pc.reach, j_begin = pc.j_begin, hk = pc.hk;
        const int32_t* table = p.table + pc.b * p.table_stride;
        int raw_page = -1, page = -1;
        auto load_page = [&](int j) {
          const int token = (j_begin + j) * kTile + lane * kGroup;
          raw_page = lane < kTile / kGroup && j < n && token < reach ? table[token >> p.page_shift] : -1;
        };
        load_page(0);
        float2 sc = make_float2(0.f, 0.f);
        int i = 0;
        for (; i < 2 * n; ++i) {
          const int j = i >> 1, run = 2 * done + i, st = run % stages;
          if (i & 1) {
            // the scales, read before the keys' copies, are there by now
            const float some = __any_sync(0xffffffffu, lane < kTile / kGroup && page < 0);
            const int slot = (done + j) % kScaleSlots;
            if (lane < kTile / kGroup) {
              float4 f = make_float4(1.f, -INFINITY, 1.f, some);  // hidden
              if (page >= 0) {
                const float vs = read_scale(sc.y);
                f = make_float4(read_scale(sc.x), log2_approx(vs), rcp_approx(vs), some);
              }
              scales[slot * (kTile / kGroup) + lane] = f;
            }
            __syncwarp();
            mbar_arrive_if(&sc_full[slot], lane == 0);
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
          if (!wwait(&raw_empty[st], ((run / stages) & 1) ^ 1)) break;
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
          for (int k = max(i - stages, 0); k < i; ++k) {
            const int run = 2 * done + k;
            mbar_wait_drain(&raw_full[run % stages], (run / stages) & 1, 200000000ull);
          }
        end_piece();
      }
    } else {
      while (pc.valid) end_piece();
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
    while (pc.valid) {
      const int n = pc.n, done = pc.done, reach = pc.reach, j_begin = pc.j_begin, first_edge = pc.first_edge;
      uint32_t hidden = 0;  // groups of the key tile without a page
      for (int i = 0; i < 2 * n; ++i) {
        const int run = 2 * done + i;  // half tiles of all pieces
        const int slot = run % C::NS, st = run % stages, j = j_begin + (i >> 1);
        if (!(i & 1)) {
          const int k = (run >> 1) % kScaleSlots;
          if (!wwait(&sc_full[k], ((run >> 1) / kScaleSlots) & 1)) break;
          hidden = __ballot_sync(0xffffffffu,
                                 lane < kTile / kGroup &&
                                     scales[k * (kTile / kGroup) + lane % (kTile / kGroup)].y == -INFINITY);
        }
        if (!wwait(&raw_full[st], (run / stages) & 1)) break;
        uint8_t* from = stage_at(st) + from_at;
        const int left = reach - j * kTile;
        const bool look = (i & 1) && j >= first_edge;
        // Seldom, and so in the stage itself, a piece at a time (the lane's own):
        // tokens that nobody sees, or without a page, become zeros; NaN values of
        // tokens that some rows do not see too, and are marked.
        if (left < kTile || hidden != 0 || look) {
#pragma unroll 1
          for (int k = 0; k < COUNT; ++k) {
            const int block = (k / CH) * 4 + warp - 12, r = block * 8 + r7;
            uint32_t* at = reinterpret_cast<uint32_t*>(
                D == 128 ? smem_xor(from + block * 1024, (k % CH) << 6) : from + block * 512);
            const bool none = r >= left || ((hidden >> (r / kGroup)) & 1u);
            bool nan = false;
#pragma unroll 1
            for (int e = 0; e < 4; ++e) {
              const uint32_t w = none ? 0u : at[e];
              const uint32_t m = look ? (((w & 0x7f7f7f7fu) + 0x01010101u) >> 7) & 0x01010101u : 0u;
              nan |= m != 0;
              at[e] = w & ~(m * 0xffu);
            }
            if (nan) atomicOr(&marked[4 * (j - first_edge) + (r >> 5)], 1u << (r & 31));
          }
        }
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
        if (!wwait(&empty[slot], ((run / C::NS) & 1) ^ 1)) break;
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
        // The stage is given back only here, behind the stores that need its codes
        // and behind the proxy fence. The stores make sure that every lane's reads
        // are over: given back right after the reads, they were seen to return the
        // next copy's codes (nothing had used them yet). The fence orders this warp's
        // own stores into the stage (hidden tokens, above) before that copy.
        mbar_arrive_if(&raw_empty[st], lane == 0);
      }
      __syncwarp();
      mbar_arrive_if(loaded, lane == 0);
      end_piece();
    }
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<160>();
    const int t = warp >> 2, sub = warp & 3;
    const int row = sub * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(sub * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::TM_S + kTile * t;
    const uint32_t tO = tmem + lane_off + C::TM_O + D * t;
    while (pc.valid) {
      const int n = pc.n, done = pc.done, j_begin = pc.j_begin, first_edge = pc.first_edge;
      const int r = pc.rt * 2 * kTile + t * kTile + row;  // row of the key head
      const bool mine = r < rows;
      const int token = min(r, rows - 1) / p.group, head = pc.hk * p.group + min(r, rows - 1) - token * p.group;
      const int seen = p.causal ? max(pc.len - p.n + token + 1, 0) : pc.len;
      const bool active = t == 0 || pc.two;
      const int base = t ? pc.two_done : done;  // key tiles of this row tile before
      float row_scale = p.scale_log2;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      if (active) {
        // this row's query as fp16, bf16 scaled by a power of two (see attn_cache_rows.cu)
        const T* src = static_cast<const T*>(p.q) + pc.b * p.q_seq + token * p.q_token + head * p.q_head;
        float inv = 1.f;
        if constexpr (!std::is_same<T, __half>::value) {
          float amax = 0.f;
#pragma unroll 1
          for (int x = 0; x < D; x += 8) {
            float y[8];
            load8(src + x, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float a = fabsf(y[e]);
              amax = fmaxf(amax, a < INFINITY ? a : 0.f);
            }
          }
          const int e = query_exp(amax);
          inv = ldexpf(1.f, -e);
          row_scale *= ldexpf(1.f, e);
        }
#pragma unroll 1
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
        const int slot = (done + j) % kScaleSlots;
        if (!wwait(&sc_full[slot], ((done + j) / kScaleSlots) & 1) || !wwait(&s_full[t], (base + j) & 1) ||
            (j > 0 && !wwait(&pv_done[t], (base + j - 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float4* sc = scales + slot * (kTile / kGroup);
        const int left = j_begin + j >= first_edge ? seen - (j_begin + j) * kTile : kTile;
        // Each half of the tile is a step of the online softmax of its own. Its
        // probabilities are formed at the running maximum while its largest
        // score is being found, and once more only if that is much larger. One
        // copy of the code for all that: the kernel's instructions, of four
        // roles at once, barely fit their cache.
#pragma unroll 1
        for (int h = 0; ok && h < 2; ++h) {
          uint32_t pk[32];
          float add;
          if (j_begin + j >= first_edge || sc[0].w != 0.f) hide(tS + 64 * h, sc + 4 * h, left - 64 * h);
#pragma unroll 1
          while (true) {
            uint32_t s[64];
            load_scores(tS + 64 * h, s);  // anew the second time: they need not be kept
            const Groups gr(sc + 4 * h, row_scale);
            const float top = max_groups(s, gr);
            add = exp_groups(s, gr, m, pk);
            if (!__any_sync(0xffffffffu, top > m + kRaise)) break;
            const float to = fmaxf(m, top - kLead);
            const float f = to == -INFINITY ? 1.f : ex2_approx(m - to);
            m = to;
            l *= f;
            if (h && !(ok = wwait(&pv_half[t], (base + j) & 1))) break;
            tc_fence_after();
            if (j > 0 || h) rescale_sums<D>(tO, f);
          }
          tmem_st32(tS + 32 * h, pk);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive_if(h ? &p_late[t] : &p_full[t], lane == 0);
          l += add;
        }
      }
      // ---------------------------------------------------------- sums
      if (ok && active && wwait(&pv_done[t], (base + pc.n - 1) & 1) && wwait(loaded, pc.index & 1)) {
        tc_fence_after();
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) any |= marked[i];
        const bool none = l == 0.f;  // no key seen (a NaN sum is not 0)
        const float inv = none ? 0.f : 1.f / l;
        float* place = params.work + (2 * int64_t(blockIdx.x) + (pc.index ? 1 : 0)) * C::PLACE;
        T* dst = static_cast<T*>(p.o) + ((int64_t(pc.b) * p.n + token) * p.H + head) * D;
#pragma unroll 1
        for (int x = 0; x < D; x += 32) {
          uint32_t y[32];
          tmem_ld32(tO + x, y);
          tmem_wait_ld();
          if (any && mine) {
            for (int key = pc.first_edge * kTile; key < seen; ++key) {
              const int k = key - pc.first_edge * kTile;
              if (!((marked[k >> 5] >> (k & 31)) & 1u)) continue;
              const int page = p.table[pc.b * p.table_stride + (key >> p.page_shift)];
              const uint8_t* v = p.codes[1] + page * p.page_stride + pc.hk * p.head_stride +
                                 (key & ((1 << p.page_shift) - 1)) * p.token_stride + x;
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if ((v[c] & 0x7fu) == 0x7fu) y[c] = 0x7fffffffu;
            }
          }
          if (!pc.whole) {
#pragma unroll
            for (int c = 0; c < 32; c += 4)
              *reinterpret_cast<uint4*>(place + (((x + c) / 4) * 2 * kTile + t * kTile + row) * 4) =
                  make_uint4(y[c], y[c + 1], y[c + 2], y[c + 3]);
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
        if (!pc.whole) {
          place[2 * kTile * D + t * kTile + row] = m;
          place[2 * kTile * (D + 1) + t * kTile + row] = l;
        } else if (mine) {
          p.lse[(int64_t(pc.b) * p.H + head) * p.n + token] = none ? -INFINITY : (m + log2f(l)) * kLn2;
        }
      }
      end_piece();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, C::TM_COLS);
  if (threadIdx.x == 0)
    reinterpret_cast<Piece*>(params.work + 2 * int64_t(params.blocks) * C::PLACE)[blockIdx.x] = left;
}

// Joins the pieces of the row tile pair that block blockIdx.x began and later
// blocks went on with: 32 rows (a lane each) and 32 columns per block, the
// pieces shared out to its warps.
constexpr int kJoinWarps = 8;
template <int D, typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) join_tiles_kernel(const CacheAttnParams p,
                                                                     const float* work, const int blocks) {
  using C = TilesCfg<D>;
  constexpr int COLS = 8;  // groups of 4 columns
  __shared__ float stats[2][kJoinWarps][32];
  __shared__ float4 part[kJoinWarps][COLS][32];
  cudaGridDependencySynchronize();  // launched early: the pieces are complete from here on
  const Piece* pieces = reinterpret_cast<const Piece*>(work + 2 * int64_t(blocks) * C::PLACE);
  const int first = blockIdx.x, tile = pieces[first].begun;
  if (tile < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rt = tile % p.row_tiles, bh = tile / p.row_tiles, b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const int row = blockIdx.y * 32 + lane, col0 = blockIdx.z * COLS;
  const int r = rt * 2 * kTile + row, rows = p.n * p.group;
  if (rt * 2 * kTile + static_cast<int>(blockIdx.y) * 32 >= rows) return;
  Join join;
  float4 y[COLS];
#pragma unroll
  for (int c = 0; c < COLS; ++c) y[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto take = [&](const float* at) {
    float4 z[COLS];
#pragma unroll
    for (int c = 0; c < COLS; ++c)
      z[c] = *reinterpret_cast<const float4*>(at + ((col0 + c) * 2 * kTile + row) * 4);
    join.add(at[2 * kTile * D + row], at[2 * kTile * (D + 1) + row], y, z, COLS);
  };
  if (r < rows) {
    if (warp == 0) take(work + (2 * int64_t(first) + pieces[first].place) * C::PLACE);
  }
  bool more = true;
  for (int k0 = first + 1; more; k0 += 32) {
    const uint32_t use = went_on(pieces, blocks, k0, tile, more);
    if (r < rows)
      for (int j = (warp + kJoinWarps - 1) % kJoinWarps; j < 32; j += kJoinWarps)
        if ((use >> j) & 1u) take(work + 2 * int64_t(k0 + j) * C::PLACE);
  }
  stats[0][warp][lane] = join.top, stats[1][warp][lane] = join.sum;
#pragma unroll
  for (int c = 0; c < COLS; ++c) part[warp][c][lane] = y[c];
  __syncthreads();
  // warp w joins and writes group w of the columns
  if (r >= rows) return;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  Join all;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w)
    all.add(stats[0][w][lane], stats[1][w][lane], &o, &part[w][warp][lane], 1);
  const int token = r / p.group, head = hk * p.group + r - token * p.group;
  const float inv = all.sum == 0.f ? 0.f : 1.f / all.sum;  // no key seen (a NaN sum is not 0)
  T* dst = static_cast<T*>(p.o) + ((int64_t(b) * p.n + token) * p.H + head) * D + 4 * (col0 + warp);
  uint2 u;
  u.x = Elem<T>::pack(o.x * inv, o.y * inv);
  u.y = Elem<T>::pack(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(dst) = u;
  if (col0 + warp == 0)
    p.lse[(int64_t(b) * p.H + head) * p.n + token] =
        all.sum == 0.f ? -INFINITY : (all.top + log2f(all.sum)) * kLn2;
}

template <int D, typename T>
cudaError_t tiles_launch(const TilesParams& params, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(cache_tiles_kernel<D, T>, TilesCfg<D>::BYTES, done);
  if (e != cudaSuccess) return e;
  cache_tiles_kernel<D, T><<<params.blocks, kTilesThreads, TilesCfg<D>::BYTES, st>>>(params);
  e = cudaGetLastError();
  if (e != cudaSuccess || params.blocks == 1) return e;
  const int rows = params.c.n * params.c.group;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(params.blocks, ((rows < 2 * kTile ? rows : 2 * kTile) + 31) / 32, D / 32);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_tiles_kernel<D, T>, params.c,
                            static_cast<const float*>(params.work), params.blocks);
}

}  // namespace

int64_t tiles_work_bytes(int64_t d) {
  return 2 * 2 * kTile * (d + 2) * 4 + static_cast<int64_t>(sizeof(Piece));
}

cudaError_t cache_tiles_launch(const CacheAttnParams& p, int d, int dtype, int blocks, float* work,
                               cudaStream_t st) {
  TilesParams t;
  t.c = p;
  t.work = work;
  t.blocks = blocks;
  const int page = 1 << p.page_shift;
  if (!encode_cache_map(&t.map_k, p.codes[0], d, page, p.Hkv, p.pages, p.token_stride, p.head_stride,
                        p.page_stride, page) ||
      !encode_cache_map(&t.map_v, p.codes[1], d, page, p.Hkv, p.pages, p.token_stride, p.head_stride,
                        p.page_stride, page))
    return cudaErrorInvalidValue;
  if (dtype == ATTN_JVP_BF16)
    return d == 128 ? tiles_launch<128, __nv_bfloat16>(t, st) : tiles_launch<64, __nv_bfloat16>(t, st);
  return d == 128 ? tiles_launch<128, __half>(t, st) : tiles_launch<64, __half>(t, st);
}

}  // namespace ajvp_serve
