// attn_prompt.cu - causal attention over packed prompts with grouped heads
// (C ABI attn_jvp_prompt_attn), bf16 or fp16.
//
// Row t of sequence b (rows starts[b] .. starts[b+1]) and query head h:
//   x_j = s <q_t, k_j>,  O_t = sum_j e^(x_j) v_j / sum_j e^(x_j),  j <= t
// in one pass over the keys with a running maximum (the standard online
// softmax; statistics and sums in fp32, the probabilities rounded to the
// inputs' type for the second product, at most 2^kRaise).
//
// Bound by the tensor cores (4 d operations per pair) and, about as much, by
// the exponentials: a tile of 128 x 128 scores takes 1,024 cycles of MMA at
// d = 128 and 1,024 cycles of MUFU. One block per SM takes two tiles of 128
// query rows of one head, so that one tile's softmax runs beside the other
// tile's products:
//   - warps 0-3 and 4-7: the softmax of tile 0 and 1, one thread per row, so
//     that maxima and sums need no exchange;
//   - warp 8: TMA loads, a ring of K and V tiles shared by the two row tiles;
//   - warp 9: issues the products. Scores S_t and, over them, probabilities
//     P_t are in tensor memory (128 columns each), the sums O_t beside them;
//   - warps 10 and 11: look through the values of the tiles on the diagonal,
//     whose keys some rows must not see (below).
// Key tiles behind a row tile's last row are never visited. The first half of a
// tile's probabilities is handed to the products before the second half is
// formed. Measured (one B200, bf16): 32,760 tokens, 8 query and 2 key heads, d =
// 128: 1.77 ms, 1,240 TFLOP/s, in a long row of calls (median 1,582 MHz, power-capped;
// the first ten after a pause, at up to 1,965 MHz, 1.54 ms); five prompts of 61 to
// 8,192 tokens: 0.64 ms (1,687 MHz; 0.59); 1,333 tokens, d = 64: 17.3 us. A pair of
// key tiles takes 3,200 cycles, 2,048 of them tensor work. d = 64: 32,760 tokens 1.39
// ms, 790 TFLOP/s (1,957 MHz), bound by the exponentials. Many short prompts are
// bound by the blocks' start and end, one block per SM: 40 of 16 to 200 tokens, 16
// heads, 36 us at d = 64 and 47 at 128.
//
// A masked key's probability is 0, but 0 times an infinity or NaN among its
// values is not. So non-finite values in the tiles on the diagonal (which hold
// the rows behind the sequence too) are set to 0 in shared memory, their keys
// are marked, and at the end each row that sees a marked key adds the key's
// non-finite values to its sums: p > 0 times infinity is infinity.
#include <cuda.h>

#include "serve_tiles.cuh"

namespace ajvp_serve {

namespace {

using namespace ajvp;

constexpr int kThreads = 384;
constexpr float kLn2F = 0.6931471805599453f;

struct PromptParams {
  CUtensorMap map_q, map_k, map_v;  // (d, heads, T), boxes of 64 columns x 128 tokens
  const void* v;
  int64_t v_token, v_head;
  void* o;     // [T, H, d]
  float* lse;  // [H, T]
  const int32_t* starts;
  unsigned int* status;
  int T, B, H, group, pieces;
  float scale_log2;
};

template <int D>
struct PromptCfg {
  static constexpr int CH = D / 64;
  static constexpr int TILE = kTile * D * 2;
  static constexpr int NS = D == 128 ? 5 : 10;  // ring slots, K and V tiles in turn
  static constexpr int DATA = (2 + NS) * TILE;
  static constexpr int NBAR = 2 * NS + 7 * 2 + 2;
  static constexpr int BYTES = 1024 + DATA + NBAR * 8 + 2 * 4 * 4 + 16;
  static constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;  // S_t at 128 t, O_t at 256 + D t
  static_assert(BYTES <= 232448, "shared memory budget");
};

// Bits of the two 16-bit halves that are infinities or NaN, at bits 0 and 16.
template <bool F16>
__device__ __forceinline__ uint32_t non_finite(uint32_t w) {
  return F16 ? (((w & 0x7c007c00u) + 0x04000400u) >> 15) & 0x00010001u
             : (((w & 0x7f807f80u) + 0x00800080u) >> 15) & 0x00010001u;
}

// The rank-th block of `unit` query rows (a "pair" of row tiles below) of all
// sequences: its sequence b and its index k in it. Up to kThreads sequences:
// those that see the most keys first, so that the blocks started last are short
// whatever the sequences' order. Pairs of index k or above number sum_b max(0, pairs(b) - k), so k is found by
// bisection and b among the sequences that have a pair k: one round of loads
// and log2 (T / unit) sums over the block. More sequences: in their order, by
// find_sequence. Every thread of the block calls this; false if there is no
// such pair.
__device__ __forceinline__ bool find_pair(const PromptParams& p, int unit, int rank, int& b, int& k) {
  __shared__ int sums[kThreads / 32];
  __shared__ int found;
  auto pairs = [&](int i) -> int {
    const int raw0 = p.starts[i], raw1 = p.starts[i + 1];
    const int t0 = clamp_row(raw0, p.T), t1 = clamp_row(raw1, p.T);
    if (t0 != raw0 || t1 != raw1 || t1 < t0) atomicOr(p.status, kStatusBadIndex);
    return t1 > t0 ? (t1 - t0 + unit - 1) / unit : 0;
  };
  if (p.B > kThreads) {
    b = find_sequence(p.starts, p.B, p.T, unit, 1, rank);
    k = rank - (clamp_row(p.starts[b], p.T) / unit + b);
    return k >= 0 && k < pairs(b);
  }
  const int warp = threadIdx.x >> 5;
  const int own = static_cast<int>(threadIdx.x) < p.B ? pairs(threadIdx.x) : 0;
  auto total = [&](int x) -> int {  // over the block
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sums[warp] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) x += sums[w];
    return x;
  };
  auto from = [&](int at) { return total(max(own - at, 0)); };  // pairs of index `at` or above
  int lo = 0, hi = p.T / unit + 1;  // from(lo) > rank >= from(hi)
  int above = 0;
  if (from(0) <= rank) return false;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2, x = from(mid);
    if (x > rank) {
      lo = mid;
    } else {
      hi = mid;
      above = x;
    }
  }
  k = lo;
  // the (rank - above)-th of the sequences with a pair k
  const bool has = own > k;
  const uint32_t votes = __ballot_sync(0xffffffffu, has);
  total((threadIdx.x & 31) == 0 ? __popc(votes) : 0);
  int before = __popc(votes & ((1u << (threadIdx.x & 31)) - 1u));
  for (int w = 0; w < warp; ++w) before += sums[w];
  if (has && before == rank - above) found = threadIdx.x;
  __syncthreads();
  b = found;
  return true;
}

// SINGLE: the block has one row tile, whose key tiles are taken in turn by the
// two sets of scores, softmax warps and sums that otherwise belong to two row
// tiles ("t" below: row tile, or key tiles 2 i + t); their sums are joined at the
// end.
template <int D, bool F16, bool SINGLE>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
  using C = PromptCfg<D>;
  using T = typename std::conditional<F16, __half, __nv_bfloat16>::type;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + 2 * C::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::DATA);
  uint64_t* full = bars;              // [NS] ring slot landed
  uint64_t* empty = bars + C::NS;     // [NS] ring slot read
  uint64_t* q_full = bars + 2 * C::NS;  // [2]
  uint64_t* s_full = q_full + 2;      // [2] scores of the row tile's current key tile
  uint64_t* p_full = q_full + 4;      // [2] its probabilities, first half
  uint64_t* p_late = q_full + 12;     // [2] second half
  uint64_t* pv_done = q_full + 6;     // [2] its sums
  uint64_t* clean = q_full + 8;       // [2] values of a diagonal tile looked through
  uint64_t* sent = q_full + 10;       // [2] the copy of a diagonal tile's values is on its way
  uint64_t* drain = q_full + 14;
  uint64_t* joined = q_full + 15;     // SINGLE: the second set's sums and statistics
  uint32_t* marked = reinterpret_cast<uint32_t*>(bars + C::NBAR);  // [2][4] keys with non-finite values
  uint32_t* tmem_slot = marked + 8;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  constexpr int unit = SINGLE ? kTile : 2 * kTile;
  const int head = blockIdx.x % p.H;
  __shared__ int where[2];
  {
    int b, block;
    if (!find_pair(p, unit, static_cast<int>(blockIdx.x / p.H), b, block)) return;
    if (threadIdx.x == 0) where[0] = b, where[1] = block;
    __syncthreads();
  }
  const int b = where[0], block = where[1];
  const int t0 = clamp_row(p.starts[b], p.T), t1 = clamp_row(p.starts[b + 1], p.T);
  const int first = block * unit;  // the block's first row
  const int len = t1 - t0;
  // Key tiles of the two row tiles; the last one of each is on its diagonal.
  const int n0 = first / kTile + 1;
  const int n1 = !SINGLE && first + kTile < len ? n0 + 1 : 0;
  const int n = n1 ? n1 : n0;

  const int warp = warp_uniform(static_cast<int>(threadIdx.x >> 5));
  const int lane = threadIdx.x & 31;
  auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return warp_wait(bar, parity, abort_flag, p.status);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&p_late[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&clean[i], 2);
      mbar_init(&sent[i], 1);
    }
    mbar_init(drain, 1);
    mbar_init(joined, 4);
    for (int i = 0; i < 8; ++i) marked[i] = 0;
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(warp_uniform(static_cast<int>(*tmem_slot)));
  const int kv_head = head / p.group;

  if (warp >= 8) {
    setmaxnreg_dec<80>();
    if (warp == 8) {
      // ------------------------------------------------------------ loads
      const uint64_t keep = l2_policy_evict_last();   // K, V: read by every later block
      const uint64_t once = l2_policy_evict_first();  // Q: this block only
      const int nq = n1 ? 2 : 1;
      if (elect_one()) {
        tma_prefetch_desc(&p.map_k);
        tma_prefetch_desc(&p.map_v);
        for (int t = 0; t < nq; ++t) {
          mbar_arrive_expect_tx(&q_full[t], C::TILE);
#pragma unroll
          for (int c = 0; c < C::CH; ++c)
            tma_load_3d_hint(sQ + t * C::TILE + c * kTile * 128, &p.map_q, &q_full[t], c * 64, head,
                             t0 + first + t * kTile, once);
        }
      }
      __syncwarp();
      int i = 0;
      bool ok = true;
      for (; i < 2 * n; ++i) {
        const int slot = i % C::NS;
        if (!wwait(&empty[slot], ((i / C::NS) & 1) ^ 1)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[slot], C::TILE);
#pragma unroll
          for (int c = 0; c < C::CH; ++c)
            tma_load_3d_hint(sRing + slot * C::TILE + c * kTile * 128, (i & 1) ? &p.map_v : &p.map_k,
                             &full[slot], c * 64, kv_head, t0 + (i >> 1) * kTile, keep);
        }
        __syncwarp();
        if ((i & 1) && (i >> 1) >= n0 - 1) mbar_arrive_if(&sent[(i >> 1) - (n0 - 1)], lane == 0);
      }
      if (!ok && lane == 0) {  // every copy issued lands before the block ends
        for (int t = 0; t < nq; ++t) mbar_wait_drain(&q_full[t], 0, 200000000ull);
        for (int j = i - 1; j >= 0 && j >= i - C::NS; --j)
          mbar_wait_drain(&full[j % C::NS], (j / C::NS) & 1, 200000000ull);
      }
      __syncwarp();
    } else if (warp == 9) {
      // ------------------------------------------------------------ products
      const uint32_t idesc_s = tile_idesc<F16>(kTile, kTile, 0);
      const uint32_t idesc_v = tile_idesc<F16>(kTile, D, 1);
      const uint32_t aQ = smem_u32(sQ), aR = smem_u32(sRing);
      auto slot_addr = [&](int i) { return aR + (i % C::NS) * C::TILE; };
      auto landed = [&](int i) { return wwait(&full[i % C::NS], (i / C::NS) & 1); };
      auto scores = [&](int t, int j) {
        mma_scores<D, kTile, kTile, false>(tmem + C::TM_S + kTile * t, aQ + (SINGLE ? 0 : t * C::TILE),
                                           slot_addr(2 * j), idesc_s, false);
        umma_commit(&s_full[t]);
      };
      bool ok = wwait(&q_full[0], 0) && landed(0);
      if (ok) {
        tc_fence_after();
        scores(0, 0);
        if (n1) {
          ok = wwait(&q_full[1], 0);
          tc_fence_after();
          if (ok) scores(1, 0);
        }
        umma_commit(&empty[0]);
        if (SINGLE && n > 1) {
          ok = landed(2);
          tc_fence_after();
          if (ok) scores(1, 1);
          umma_commit(&empty[2]);
        }
      }
      // Per key tile j and row tile t: O_t += P_t V_j, then the next scores
      // over P_t (one thread's products execute in order), which the softmax
      // of row tile t turns into probabilities beside the other row tile's
      // products.
      for (int j = 0; ok && j < n; ++j) {
        const int vi = 2 * j + 1, ahead = SINGLE ? 2 : 1, ki = 2 * (j + ahead);
        ok = landed(vi) && (j < n0 - 1 || wwait(&clean[j - (n0 - 1)], 0));
        for (int t = 0; ok && t < 2; ++t) {
          const int nt = !SINGLE && t ? n1 : n0;
          if (SINGLE ? t != (j & 1) : j >= nt) continue;
          const int phase = SINGLE ? (j >> 1) & 1 : j & 1;
          ok = wwait(&p_full[t], phase);
          if (!ok) break;
          tc_fence_after();
          mma_values_half<D, 0>(tmem + C::TM_O + D * t, tmem + C::TM_S + kTile * t, slot_addr(vi),
                                idesc_v, SINGLE ? j > 1 : j > 0);
          // the next keys, while the second half's probabilities are formed
          if (j + ahead < nt) ok = landed(ki);
          ok = ok && wwait(&p_late[t], phase);
          if (!ok) break;
          tc_fence_after();
          mma_values_half<D, 1>(tmem + C::TM_O + D * t, tmem + C::TM_S + kTile * t, slot_addr(vi),
                                idesc_v, true);
          umma_commit(&pv_done[t]);
          if (j + ahead < nt) scores(t, j + ahead);
        }
        if (!ok) break;
        umma_commit(&empty[vi % C::NS]);
        if (j + ahead < n) umma_commit(&empty[ki % C::NS]);
      }
      umma_commit(drain);  // every product ends before tensor memory is released
      if (lane == 0) mbar_wait_drain(drain, 0, 1000000000ull);
      __syncwarp();
    } else {
      // ------------------------------------------------------------ diagonal values
      const int part = (warp - 10) * 32 + lane;
      for (int d = 0; d < (n1 ? 2 : 1); ++d) {
        const int i = 2 * (n0 - 1 + d) + 1, slot = i % C::NS;
        // These warps do not follow the ring: once the copy has been issued, the
        // slot's earlier phases are over, and its parity says this copy's.
        if (!wwait(&sent[d], 0) || !wwait(&full[slot], (i / C::NS) & 1)) break;
#pragma unroll 1
        for (int r = part; r < kTile; r += 64) {
          bool bad = false;
#pragma unroll
          for (int c = 0; c < C::CH; ++c)
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              // the row's 16-byte pieces in an order that spreads the banks
              uint4* at = reinterpret_cast<uint4*>(sRing + slot * C::TILE + c * kTile * 128 + r * 128 +
                                                   ((x + r) & 7) * 16);
              uint4 u = *at;
              const uint32_t m0 = non_finite<F16>(u.x), m1 = non_finite<F16>(u.y),
                             m2 = non_finite<F16>(u.z), m3 = non_finite<F16>(u.w);
              if (m0 | m1 | m2 | m3) {
                bad = true;
                u.x &= ~(m0 * 0xffffu), u.y &= ~(m1 * 0xffffu);
                u.z &= ~(m2 * 0xffffu), u.w &= ~(m3 * 0xffffu);
                *at = u;
              }
            }
          if (bad) atomicOr(&marked[4 * d + (r >> 5)], 1u << (r & 31));
        }
        fence_proxy_async_shared();
        __syncwarp();
        mbar_arrive_if(&clean[d], lane == 0);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<208>();
    const int t = warp >> 2, sub = warp & 3;
    const int row = sub * 32 + lane;
    const int nt = SINGLE ? (n0 + 1 - t) / 2 : t ? n1 : n0;
    const uint32_t lane_off = static_cast<uint32_t>(sub * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::TM_S + kTile * t;
    const uint32_t tO = tmem + lane_off + C::TM_O + D * t;
    const float sc = p.scale_log2;
    const float2 sc2 = make_float2(sc, sc);
    float m = -INFINITY;  // running maximum of x log2 e
    float l = 0.f;
    bool ok = true;
    for (int j = 0; j < nt; ++j) {
      // the sums of the tile before are complete once these scores are; every
      // phase of their barrier is waited for in turn
      if (!wwait(&s_full[t], j & 1) || (j > 0 && !wwait(&pv_done[t], (j - 1) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t s[kTile];
#pragma unroll
      for (int x = 0; x < kTile; x += 32)
        tmem_ld32(tS + x, *reinterpret_cast<uint32_t(*)[32]>(&s[x]));
      tmem_wait_ld();
      if (SINGLE ? 2 * j + t == n0 - 1 : j == nt - 1) {
#pragma unroll
        for (int x = 0; x < kTile; ++x)
          if (x > row) s[x] = __float_as_uint(-INFINITY);
      }
      // The first half's probabilities are formed at the running maximum while
      // the row's largest score is still being found, and again only if it
      // exceeds that maximum by more than 2^kRaise.
      uint32_t pk[32];
      float2 sum = make_float2(0.f, 0.f);
      exp_half<F16>(&s[0], sc2, m, pk, sum);
      const float top = max128(s) * sc;
      if (__any_sync(0xffffffffu, top > m + kRaise)) {
        const float to = fmaxf(m, top - kLead);
        const float f = to == -INFINITY ? 1.f : ex2_approx(m - to);
        m = to;
        l *= f;
        if (j > 0) rescale_sums<D>(tO, f);
        sum = make_float2(0.f, 0.f);
        exp_half<F16>(&s[0], sc2, m, pk, sum);
      }
      tmem_st32(tS, pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_if(&p_full[t], lane == 0);
      exp_half<F16>(&s[64], sc2, m, pk, sum);
      tmem_st32(tS + 32, pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_if(&p_late[t], lane == 0);
      l += sum.x + sum.y;
    }
    bool writes = nt > 0;
    float* stats = reinterpret_cast<float*>(sQ + C::TILE);  // SINGLE: m and l of the second set
    if (SINGLE && t == 1) {
      writes = false;
      if (ok && (nt == 0 || wwait(&pv_done[1], (nt - 1) & 1))) {
        tc_fence_after();
        stats[row] = m, stats[kTile + row] = l;
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(joined, lane == 0);
      }
    }
    if (ok && writes && wwait(&pv_done[t], (nt - 1) & 1) && wwait(&clean[0], 0) &&
        (t == 0 || wwait(&clean[1], 0)) && (!SINGLE || wwait(joined, 0))) {
      tc_fence_after();
      const int r = first + (SINGLE ? 0 : t * kTile) + row;  // row of the sequence
      const bool mine = r < len;
      float f0 = 1.f, f1 = 0.f;
      if (SINGLE && n0 > 1) {
        const float other = stats[row], to = fmaxf(m, other);
        f0 = to == -INFINITY ? 1.f : ex2_approx(m - to);
        f1 = to == -INFINITY ? 1.f : ex2_approx(other - to);
        m = to;
        l = l * f0 + stats[kTile + row] * f1;
      }
      const float inv = 1.f / l;
      // keys with non-finite values that this row sees: all marked ones of the
      // first diagonal tile up to the row, or of the second too
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) any |= marked[i];
      T* dst = static_cast<T*>(p.o) + (int64_t(t0 + r) * p.H + head) * D;
#pragma unroll 1
      for (int x = 0; x < D; x += 32) {
        uint32_t y[32];
        tmem_ld32(tO + x, y);
        tmem_wait_ld();
        if (SINGLE && n0 > 1) {
          uint32_t z[32];
          tmem_ld32(tO + D + x, z);  // the second set's, in the same lanes
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c)
            y[c] = __float_as_uint(__uint_as_float(y[c]) * f0 + __uint_as_float(z[c]) * f1);
        }
        if (any && mine) {
          for (int k = 0; k < (t + 1) * kTile; ++k) {
            const int key = first + k;
            if (key > r || !((marked[k >> 5] >> (k & 31)) & 1u)) continue;
            const T* v = static_cast<const T*>(p.v) + int64_t(t0 + key) * p.v_token +
                         kv_head * p.v_head + x;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float z = static_cast<float>(v[c]);
              if (!isfinite(z)) y[c] = __float_as_uint(__uint_as_float(y[c]) + z);
            }
          }
        }
        if (mine) {
#pragma unroll
          for (int c = 0; c < 32; c += 8) {
            uint4 u;
            u.x = pack_pair<F16>(__uint_as_float(y[c]) * inv, __uint_as_float(y[c + 1]) * inv);
            u.y = pack_pair<F16>(__uint_as_float(y[c + 2]) * inv, __uint_as_float(y[c + 3]) * inv);
            u.z = pack_pair<F16>(__uint_as_float(y[c + 4]) * inv, __uint_as_float(y[c + 5]) * inv);
            u.w = pack_pair<F16>(__uint_as_float(y[c + 6]) * inv, __uint_as_float(y[c + 7]) * inv);
            *reinterpret_cast<uint4*>(dst + x + c) = u;
          }
        }
      }
      if (mine) p.lse[int64_t(head) * p.T + t0 + r] = (m + log2f(l)) * kLn2F;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, C::TM_COLS);
}

template <int D, bool F16, bool SINGLE>
cudaError_t prompt_launch(const PromptParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(prompt_kernel<D, F16, SINGLE>, PromptCfg<D>::BYTES, done);
  if (e != cudaSuccess) return e;
  prompt_kernel<D, F16, SINGLE><<<p.pieces * p.H, kThreads, PromptCfg<D>::BYTES, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

}  // namespace ajvp_serve

extern "C" int attn_jvp_prompt_attn(const attn_jvp_tokens* shape, const void* q,
                                    attn_jvp_strides q_strides, const void* k,
                                    attn_jvp_strides k_strides, const void* v,
                                    attn_jvp_strides v_strides, int64_t B, const int32_t* starts,
                                    void* o, float* lse, void* stream) {
  using namespace ajvp_serve;
  if (!shape) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  const attn_jvp_tokens& s = *shape;
  if ((s.dtype != ATTN_JVP_BF16 && s.dtype != ATTN_JVP_F16) || (s.d != 64 && s.d != 128))
    return ATTN_JVP_ERR_UNSUPPORTED;
  if (s.T < 0 || s.T > (int64_t(1) << 30) || s.H < 1 || s.H > 65535 || s.Hkv < 1 || s.H % s.Hkv ||
      B < 0 || B > (1 << 20) || !good_scale(s.scale))
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (s.T == 0 || B == 0) return ATTN_JVP_OK;
  if (!starts || !o || !lse) return ATTN_JVP_ERR_INVALID_ARGUMENT;
  if (!aligned16(o) || !aligned4(lse) || !aligned4(starts)) return ATTN_JVP_ERR_MISALIGNED;
  int rc;
  if ((rc = check_rows_map(q, q_strides, s.T, s.H, s.d, 2)) != ATTN_JVP_OK ||
      (rc = check_rows_map(k, k_strides, s.T, s.Hkv, s.d, 2)) != ATTN_JVP_OK ||
      (rc = check_rows_map(v, v_strides, s.T, s.Hkv, s.d, 2)) != ATTN_JVP_OK)
    return rc;
  int64_t pieces = s.T / (2 * kTile) + B;
  if (pieces * s.H > (int64_t(1) << 30)) return ATTN_JVP_ERR_UNSUPPORTED;
  PromptParams p;
  int sms = 0;
  rc = ajvp::device_status_word(&p.status, &sms);
  if (rc != ATTN_JVP_OK) return rc;
  if (!ajvp::encode_token_rows_map(&p.map_q, q, s.dtype, s.T, s.H, s.d, q_strides.token,
                                   q_strides.head, kTile) ||
      !ajvp::encode_token_rows_map(&p.map_k, k, s.dtype, s.T, s.Hkv, s.d, k_strides.token,
                                   k_strides.head, kTile) ||
      !ajvp::encode_token_rows_map(&p.map_v, v, s.dtype, s.T, s.Hkv, s.d, v_strides.token,
                                   v_strides.head, kTile))
    return ATTN_JVP_ERR_INVALID_ARGUMENT;
  p.v = v, p.v_token = v_strides.token, p.v_head = v_strides.head;
  p.o = o, p.lse = lse, p.starts = starts;
  p.T = static_cast<int>(s.T), p.B = static_cast<int>(B), p.H = static_cast<int>(s.H);
  p.group = static_cast<int>(s.H / s.Hkv);
  // Blocks of one row tile where blocks of two would not fill the SMs (they read
  // each key twice as often). us, one / two, by length and heads:
  //                       d = 64         d = 128                       d = 64         d = 128
  //   300 x 4:            8.8 / 9.1      9.8 / 12.3   2,600 x 16:      39.1 / 37.5    50.0 / 41.5
  //   2 of 300, 16 heads: 9.2 / 9.6     10.1 / 12.6   4,000 x 16:      69.0 / 58.7    90.4 / 66.9
  //   1,333 x 16:        17.3 / 21.8    21.7 / 25.0   1,300 x 32:      30.3 / 26.6    38.8 / 32.5
  //   4,000 x 8:         34.7 / 54.3    45.1 / 57.7   8 of 500, 8 heads: 17.7 / 14.0  21.5 / 16.4
  //   8,000 x 4:         53.6 / 99.5    69.3 / 104
  const bool single = pieces * s.H <= sms;
  if (single) pieces = s.T / kTile + B;
  p.pieces = static_cast<int>(pieces);
  p.scale_log2 = scale_log2(s.scale, s.d);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  auto launch = [&](auto one) {
    constexpr bool S = decltype(one)::value;
    if (s.dtype == ATTN_JVP_BF16)
      return s.d == 128 ? prompt_launch<128, false, S>(p, st) : prompt_launch<64, false, S>(p, st);
    return s.d == 128 ? prompt_launch<128, true, S>(p, st) : prompt_launch<64, true, S>(p, st);
  };
  e = single ? launch(std::true_type()) : launch(std::false_type());
  return e == cudaSuccess ? ATTN_JVP_OK : ATTN_JVP_ERR_CUDA;
}
