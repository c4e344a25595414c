// latent8_write.cu -- quantising write of latent rows into the 8-bit cache.
//
// Row i: s = least power of two (>= 2^-100) with amax |c_i| <= 448 s, or the
// slot's block scale; c8 = e4m3(c / s), kr = bf16(R(pos) k / s).
// A power of two keeps c / s exact, so a code is off by e4m3's half step and
// nothing else, and the stored rope part keeps bf16's own precision under the
// row's scale.
//
// Bound: HBM (reads 576 elements, writes 644 bytes a row); at a verify step's
// row counts launch latency. One warp takes a row: each lane holds 16 latent
// elements in registers between the maximum and the rounding (one read), and
// one rope pair, whose angle it forms itself; everything a row needs from memory is asked
// for at once, the next row's slot and position before that. A scale that is a power of two divides as a product (exact). 65536 bf16 rows: 30 us
// (device time in a graph, 31-32 a call; 49 us with a division for each element and the position read last).
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "rope.cuh"

namespace kdv {
namespace {

constexpr int WARPS = 8;
constexpr int PER_LANE = 16;          // latent elements a lane holds: D_c <= 512
constexpr int MAX_DR = 64;

struct WriteArgs {
  const void* c;
  const void* k;
  int64_t c_stride, k_stride;
  const int32_t* slot;
  const int32_t* tree_off;
  const int32_t* prefix_len;
  const int32_t* kv_off;
  const int32_t* page_table;
  RopePos pos;
  uint8_t* c8;
  __nv_bfloat16* kr;
  float* scale;
  int64_t num_slots;
  int32_t* d_err;
  int32_t rows, d_c, d_r, rot, half, batch, block_log2, static_scale;
  float mscale;
};

// The least e >= -100 with x <= 448 * 2^e = 1.75 * 2^(e + 8), from x's bits (x > 0, finite; what is too
// small to be normal is below every e that counts).
__device__ inline int scale_exponent(uint32_t bits) {
  return max((int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), -100);
}

__device__ inline bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// e4m3 of v / s, saturating; the NaN code where v is not finite. inv: 1 / s where s is a power of two, else 0.
__device__ inline uint32_t e4m3x4(float a, float b, float c, float d, float s, float inv) {
  if (inv != 0.f) {
    a *= inv; b *= inv; c *= inv; d *= inv;
  } else {
    a /= s; b /= s; c /= s; d /= s;
  }
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Row i's slot: -1 skipped, -2 outside the pool, -3 not a node of a request.
__device__ inline int64_t find_slot(const WriteArgs& a, int i) {
  int64_t slot;
  if (a.slot != nullptr) {
    slot = a.slot[i];
    if (slot == -1) return -1;
    // a row that takes its position from the tree has to be one of its nodes
    if (a.rot > 0 && a.pos.pos == nullptr && (i < a.tree_off[0] || i >= a.tree_off[a.batch])) return -3;
  } else {
    const int b = node_request(a.tree_off, a.batch, i);
    const int64_t at = b < 0 ? 0 : (int64_t)a.kv_off[b] + a.prefix_len[b] + (i - a.tree_off[b]);
    if (b < 0 || a.prefix_len[b] < 0 || at < 0 || at >= a.kv_off[b + 1]) return -3;
    slot = a.page_table != nullptr ? a.page_table[at] : at;
  }
  return slot < 0 || slot >= a.num_slots ? -2 : slot;
}

// A row's inputs as this lane holds them. FAST: D_c = 512, D_r = 64 and
// 16-byte aligned rows: lane l holds elements 8 l .. 8 l + 7 of each half of
// the row. Otherwise lane l holds l + 32 i.
template <typename T, bool FAST>
struct RowIn {
  static constexpr int WORDS = FAST ? PER_LANE * (int)sizeof(T) / 16 : 1;
  uint4 w[WORDS];
  float f[FAST ? 1 : PER_LANE];
  T ku, kv;
  int32_t pos;
  int64_t slot;
  __device__ __forceinline__ void load(const WriteArgs& a, int i, int lane) {
    const T* c = static_cast<const T*>(a.c) + (int64_t)i * a.c_stride;
    if constexpr (FAST) {
#pragma unroll
      for (int g = 0; g < WORDS; ++g)
        w[g] = reinterpret_cast<const uint4*>(c + g / (WORDS / 2) * 256 + lane * 8)[g % (WORDS / 2)];
    } else {
#pragma unroll
      for (int j = 0; j < PER_LANE; ++j) f[j] = lane + 32 * j < a.d_c ? (float)c[lane + 32 * j] : 0.f;
    }
    const T* k = static_cast<const T*>(a.k) + (int64_t)i * a.k_stride;
    const int npair = a.rot / 2;
    ku = kv = T(0.f);
    pos = 0;
    if (lane < npair) {
      ku = k[a.half ? lane : 2 * lane];
      kv = k[a.half ? lane + npair : 2 * lane + 1];
      pos = rope_position(a.pos, i);
    }
    slot = find_slot(a, i);
  }
  // the largest magnitude of this lane's elements, as the bits of a float
  __device__ __forceinline__ uint32_t magnitude() const {
    uint32_t m = 0;
    if constexpr (!FAST) {
#pragma unroll
      for (int j = 0; j < PER_LANE; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
      return m;
    } else {
#pragma unroll
      for (int g = 0; g < WORDS; ++g) {
        const uint32_t u[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = sizeof(T) == 2 ? __vmaxu2(m, u[j] & 0x7fff7fffu) : max(m, u[j] & 0x7fffffffu);
      }
      return sizeof(T) == 2 ? max(m & 0xffff0000u, m << 16) : m;
    }
  }
  __device__ __forceinline__ void get(float (&v)[PER_LANE]) const {
    if constexpr (!FAST) {
#pragma unroll
      for (int j = 0; j < PER_LANE; ++j) v[j] = f[j];
    } else {
#pragma unroll
      for (int g = 0; g < WORDS; ++g) {
        const uint32_t u[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (sizeof(T) == 2) {
            v[g * 8 + 2 * j] = __uint_as_float(u[j] << 16);
            v[g * 8 + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
          } else {
            v[g * 4 + j] = __uint_as_float(u[j]);
          }
        }
      }
    }
  }
};

template <typename T, bool FAST>
__device__ __forceinline__ void write_row(const WriteArgs& a, int i, const RowIn<T, FAST>& in, double turns_per_pos, int lane) {
  const int64_t slot = in.slot;
  float s = a.static_scale ? a.scale[slot >> a.block_log2] : 0.f;
  float v[PER_LANE];
  in.get(v);
  const int npair = a.rot / 2;
  const int first = a.half ? lane : 2 * lane, second = a.half ? lane + npair : 2 * lane + 1;
  const float ku = (float)in.ku, kv = (float)in.kv;

  // magnitudes order as their bits do, infinities and NaN above all
  uint32_t top = __reduce_max_sync(0xffffffffu, in.magnitude());
  if (top >= 0x7f800000u) {                        // left out of the maximum, stored as NaN
    if (lane == 0) record_error(a.d_err, KDV_DERR_RANGE);
    top = 0;
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) {
      const bool ok = finite(v[j]);
      top = max(top, ok ? __float_as_uint(fabsf(v[j])) : 0u);
      v[j] = ok ? v[j] : __int_as_float(0x7fc00000);
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  if (a.static_scale) {
    if (!(s > 0.f) || !finite(s)) {
      if (lane == 0) record_error(a.d_err, KDV_DERR_RANGE);
      return;
    }
  } else {
    s = top == 0u ? 1.f : __int_as_float((127 + scale_exponent(top)) << 23);
    if (lane == 0) a.scale[slot] = s;
  }
  // 2^-e of s = 2^e, for every e whose inverse is a normal number
  const uint32_t sb = __float_as_uint(s);
  const float inv = (sb & 0x7fffffu) == 0u && sb >= 0x01000000u && sb <= 0x7e000000u ? __uint_as_float(0x7f000000u - sb) : 0.f;
  uint8_t* dst = a.c8 + slot * a.d_c;
  if constexpr (FAST) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float* w = v + g * 8;
      *reinterpret_cast<uint2*>(dst + g * 256 + lane * 8) =
          make_uint2(e4m3x4(w[0], w[1], w[2], w[3], s, inv), e4m3x4(w[4], w[5], w[6], w[7], s, inv));
    }
  } else {
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j)
      if (lane + 32 * j < a.d_c) dst[lane + 32 * j] = (uint8_t)e4m3x4(v[j], 0.f, 0.f, 0.f, s, inv);
  }
  if (a.d_r == 0) return;
  __nv_bfloat16* out = a.kr + slot * a.d_r;
  if (lane < npair) {
    const float2 w = rope_cos_sin(in.pos, turns_per_pos, a.mscale);
    const float x0 = ku * w.x - kv * w.y, x1 = ku * w.y + kv * w.x;
    const float r0 = inv != 0.f ? x0 * inv : x0 / s, r1 = inv != 0.f ? x1 * inv : x1 / s;
    if (FAST && !a.half) {
      *reinterpret_cast<__nv_bfloat162*>(out + first) = __floats2bfloat162_rn(r0, r1);
    } else {
      out[first] = __float2bfloat16_rn(r0);
      out[second] = __float2bfloat16_rn(r1);
    }
  }
  const T* kp = static_cast<const T*>(a.k) + (int64_t)i * a.k_stride;
  for (int d = a.rot + lane; d < a.d_r; d += 32) out[d] = __float2bfloat16_rn((float)kp[d] / s);
}

template <typename T, bool FAST>
__global__ void __launch_bounds__(WARPS * 32, 4) latent8_write_kernel(const __grid_constant__ WriteArgs a,
                                                                    const __grid_constant__ RopeTurns<MAX_DR / 2> turns) {
  const int lane = threadIdx.x & 31;
  const int npair = a.rot / 2;
  // lane-dependent indexes into the parameters are read one lane at a time: once a warp, not once a row
  const double turns_per_pos = lane < npair ? turns.f[lane] : 0.0;
  const int stride = gridDim.x * WARPS;
  int i = blockIdx.x * WARPS + (threadIdx.x >> 5);
  if (i >= a.rows) return;
  RowIn<T, FAST> in;
  in.load(a, i, lane);
  for (;;) {
    const bool more = i < a.rows - stride;
    RowIn<T, FAST> next = in;
    if (more) next.load(a, i + stride, lane);
    if (in.slot >= 0) write_row<T, FAST>(a, i, in, turns_per_pos, lane);
    else if (in.slot < -1 && lane == 0) record_error(a.d_err, in.slot == -2 ? KDV_DERR_BAD_SLOT : KDV_DERR_BAD_LENGTH);
    if (!more) break;
    in = next;
    i += stride;
  }
}

bool al16(const void* p, int64_t stride, int esz) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (stride * esz) % 16 == 0;
}

template <typename T>
void launch_write(const WriteArgs& a, const RopeTurns<MAX_DR / 2>& f, bool fast, cudaStream_t s) {
  // enough CTAs to fill the GPU once, each warp then steps through rows
  const int grid = (int)std::min<int64_t>(((int64_t)a.rows + WARPS - 1) / WARPS, 148 * 4);
  if (fast) latent8_write_kernel<T, true><<<grid, WARPS * 32, 0, s>>>(a, f);
  else latent8_write_kernel<T, false><<<grid, WARPS * 32, 0, s>>>(a, f);
}

}  // namespace
}  // namespace kdv

using namespace kdv;

extern "C" kdv_status kdv_latent8_write(const kdv_latent8_params* p, void* stream) {
  if (p == nullptr || p->rows < 0) return KDV_ERR_INVALID_ARG;
  if (p->d_latent < 1 || p->d_rope < 0) return KDV_ERR_INVALID_ARG;
  if (p->d_latent > 512 || p->d_rope > MAX_DR) return KDV_ERR_UNSUPPORTED;
  if (p->dtype != KDV_BF16 && p->dtype != KDV_F32) return KDV_ERR_INVALID_ARG;
  if (p->c_stride < p->d_latent || (p->d_rope > 0 && p->k_stride < p->d_rope)) return KDV_ERR_INVALID_ARG;
  if (p->scale_block < 1 || p->scale_block > 4096 || (p->scale_block & (p->scale_block - 1)))
    return KDV_ERR_INVALID_ARG;
  if (p->static_scale != 0 && p->static_scale != 1) return KDV_ERR_INVALID_ARG;
  if (!p->static_scale && p->scale_block != 1) return KDV_ERR_UNSUPPORTED;   // a shared scale cannot follow one row
  if (p->num_slots < 0) return KDV_ERR_INVALID_ARG;
  const bool rot = p->h_inv_freq != nullptr;
  if (rot) {
    if (p->rot_dim < 2 || p->rot_dim % 2 || p->rot_dim > p->d_rope) return KDV_ERR_INVALID_ARG;
    if (p->layout != KDV_ROPE_INTERLEAVED && p->layout != KDV_ROPE_HALF) return KDV_ERR_INVALID_ARG;
    if (!std::isfinite(p->mscale)) return KDV_ERR_INVALID_ARG;
    for (int k = 0; k < p->rot_dim / 2; ++k)
      if (!std::isfinite(p->h_inv_freq[k])) return KDV_ERR_INVALID_ARG;
  }
  if (p->rows == 0) return KDV_OK;
  const bool nodes = p->slot == nullptr, tree_pos = rot && p->pos == nullptr;
  if (nodes || tree_pos) {
    if (p->batch < 1 || !p->tree_off || !p->prefix_len) return KDV_ERR_INVALID_ARG;
    if (p->batch > KDV_MAX_BATCH) return KDV_ERR_UNSUPPORTED;
    if ((nodes && !p->kv_off) || (tree_pos && !p->depth)) return KDV_ERR_INVALID_ARG;
  }
  if (!p->c || !p->c8 || !p->kv_scale || (p->d_rope > 0 && (!p->k_rope || !p->kr))) return KDV_ERR_INVALID_ARG;
  const int esz = p->dtype == KDV_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(p->c) % esz || reinterpret_cast<uintptr_t>(p->k_rope) % esz ||
      reinterpret_cast<uintptr_t>(p->kr) % 2 || reinterpret_cast<uintptr_t>(p->kv_scale) % 4)
    return KDV_ERR_INVALID_ARG;
  WriteArgs a = {};
  a.c = p->c;
  a.k = p->k_rope;
  a.c_stride = p->c_stride;
  a.k_stride = p->k_stride;
  a.slot = p->slot;
  a.tree_off = p->tree_off;
  a.prefix_len = p->prefix_len;
  a.kv_off = p->kv_off;
  a.page_table = p->page_table;
  a.pos = {p->pos, p->tree_off, p->prefix_len, p->depth, p->batch};
  a.c8 = p->c8;
  a.kr = static_cast<__nv_bfloat16*>(p->kr);
  a.scale = p->kv_scale;
  a.num_slots = p->num_slots;
  a.d_err = p->d_err;
  a.rows = p->rows;
  a.d_c = p->d_latent;
  a.d_r = p->d_rope;
  a.rot = rot ? p->rot_dim : 0;
  a.half = rot && p->layout == KDV_ROPE_HALF;
  a.batch = p->batch;
  while ((1 << a.block_log2) < p->scale_block) ++a.block_log2;
  a.static_scale = p->static_scale;
  a.mscale = p->mscale;
  RopeTurns<MAX_DR / 2> f = {};
  for (int k = 0; k < a.rot / 2; ++k) f.f[k] = p->h_inv_freq[k] / 6.283185307179586476925286766559;
  const bool fast = p->d_latent == 512 && p->d_rope == 64 && al16(p->c, p->c_stride, esz) && al16(p->c8, 512, 1) &&
                    reinterpret_cast<uintptr_t>(p->kr) % 4 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->dtype == KDV_BF16) launch_write<__nv_bfloat16>(a, f, fast, s);
  else launch_write<float>(a, f, fast, s);
  return cudaGetLastError() == cudaSuccess ? KDV_OK : KDV_ERR_CUDA;
}
