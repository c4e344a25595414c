// rope.cuh -- rotary angles, shared by the rotation kernel and the cache write.
#pragma once

#include <cuda_bf16.h>

#include "kdv_internal.cuh"

namespace kdv {

// Pair frequencies in turns per position (inv_freq / 2 pi), by value in the
// kernel parameters.
template <int N>
struct RopeTurns {
  double f[N];
};

// Positions of a call: explicit, or prefix_len + depth of the tree's nodes.
struct RopePos {
  const int32_t* pos;
  const int32_t* tree_off;
  const int32_t* prefix_len;
  const int32_t* depth;
  int32_t batch;
};

// Request of tree node i: the last b with tree_off[b] <= i. -1 when no
// request holds it.
__device__ inline int node_request(const int32_t* tree_off, int batch, int i) {
  int lo = 0, hi = batch;            // tree_off[lo] <= i < tree_off[hi] when i is in range
  if (i < tree_off[0] || i >= tree_off[batch]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tree_off[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ inline int32_t rope_position(const RopePos& r, int i) {
  if (r.pos != nullptr) return r.pos[i];
  const int b = node_request(r.tree_off, r.batch, i);
  return b < 0 ? 0 : r.prefix_len[b] + r.depth[i];
}

// (cos, sin) of pos * inv_freq, times mscale. The angle is formed in turns in
// 64 bits and reduced to [-1/2, 1/2] there. The frequency in turns and the product round
// by 2^-53 each: for frequencies up to 1, 5e-7 radians at a position of 2^31, and below half
// of fp32's step of the result to 2^27.
__device__ inline float2 rope_cos_sin(int32_t pos, double turns_per_pos, float mscale) {
  double t = (double)pos * turns_per_pos;
  t -= rint(t);
  float s, c;
  sincospif(2.0f * (float)t, &s, &c);
  return make_float2(c * mscale, s * mscale);
}

}  // namespace kdv
