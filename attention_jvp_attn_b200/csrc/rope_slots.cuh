// rope_slots.cuh - a head's row in slots of 16 columns, each two runs of 8
// adjacent columns that hold whole pairs of the rotation, for one thread each:
// shared by the rotation at positions and the append to the cache, so both
// give the same values.
#pragma once

#include "rope_math.cuh"
#include "serve_common.cuh"

namespace ajvp_serve {

// Slot g of d / 16. half = rot / 2 (a multiple of 8), 0 for no rotation.
struct RopeSlot {
  int c0, c1;  // first columns of the two runs
  int pair;    // first of the slot's 8 pairs; -1: not rotated
  bool split;  // pairs are (c0 + i, c1 + i); else adjacent columns
  __device__ __forceinline__ RopeSlot(int g, int half, bool half_layout) {
    const int turned = half >> 3;  // rotated slots: the first ones
    split = half_layout && g < turned;
    c0 = split ? 8 * g : 16 * g;
    c1 = split ? c0 + half : c0 + 8;
    pair = g < turned ? 8 * g : -1;
  }
};

// The slot's cosines and sines from a row [half] of the tables.
__device__ __forceinline__ void load_turn(const float* cos, const float* sin, int64_t row, int half,
                                          const RopeSlot& sl, float (&c)[8], float (&s)[8]) {
  const int64_t at = row * half + sl.pair;
  load4(cos + at, reinterpret_cast<float(&)[4]>(c[0]));
  load4(cos + at + 4, reinterpret_cast<float(&)[4]>(c[4]));
  load4(sin + at, reinterpret_cast<float(&)[4]>(s[0]));
  load4(sin + at + 4, reinterpret_cast<float(&)[4]>(s[4]));
}

// `split` is sl.split, given apart where the compiler may know it.
__device__ __forceinline__ void turn_slot(bool split, float (&a)[8], float (&b)[8],
                                          const float (&c)[8], const float (&s)[8]) {
  if (split) {
#pragma unroll
    for (int i = 0; i < 8; ++i) ajvp::rope_rotate_pair(a[i], b[i], c[i], s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ajvp::rope_rotate_pair(a[2 * i], a[2 * i + 1], c[i], s[i]);
      ajvp::rope_rotate_pair(b[2 * i], b[2 * i + 1], c[4 + i], s[4 + i]);
    }
  }
}

}  // namespace ajvp_serve
