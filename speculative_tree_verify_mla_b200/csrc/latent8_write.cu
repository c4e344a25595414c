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
// one rope pair, whose angle it forms itself.
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

// The least e with x <= 448 * 2^e = 0.875 * 2^(e + 9), clamped below at -100.
__device__ inline int scale_exponent(float amax) {
  int e;
  const float m = frexpf(amax, &e);                 // amax = m 2^e, m in [1/2, 1)
  return max(m <= 0.875f ? e - 9 : e - 8, -100);
}

__device__ inline bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// e4m3 of v, saturating; the NaN code where the source value was not finite.
__device__ inline uint8_t e4m3(float v, bool ok) {
  return ok ? (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3) : (uint8_t)0x7F;
}

// FAST: D_c = 512, D_r = 64 and 16-byte aligned rows: lane l holds elements
// 8 l .. 8 l + 7 of each half of the row. Otherwise lane l holds l + 32 i.
template <typename T, bool FAST>
__global__ void __launch_bounds__(WARPS * 32) latent8_write_kernel(const __grid_constant__ WriteArgs a,
                                                                    const __grid_constant__ RopeTurns<MAX_DR / 2> turns) {
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * WARPS + (threadIdx.x >> 5);
  if (i >= a.rows) return;
  int64_t slot;
  if (a.slot != nullptr) {
    slot = a.slot[i];
    if (slot == -1) return;
  } else {
    const int b = node_request(a.tree_off, a.batch, i);
    const int64_t at = b < 0 ? 0 : (int64_t)a.kv_off[b] + a.prefix_len[b] + (i - a.tree_off[b]);
    if (b < 0 || a.prefix_len[b] < 0 || at < 0 || at >= a.kv_off[b + 1]) {
      if (lane == 0) record_error(a.d_err, KDV_DERR_BAD_LENGTH);
      return;
    }
    slot = a.page_table != nullptr ? a.page_table[at] : at;
  }
  if (slot < 0 || slot >= a.num_slots) {
    if (lane == 0) record_error(a.d_err, KDV_DERR_BAD_SLOT);
    return;
  }
  const T* c = static_cast<const T*>(a.c) + (int64_t)i * a.c_stride;
  float v[PER_LANE];
  if constexpr (FAST) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const T* src = c + g * 256 + lane * 8;
      if constexpr (sizeof(T) == 2) {
        const uint4 w = *reinterpret_cast<const uint4*>(src);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[g * 8 + 2 * j] = __uint_as_float(u[j] << 16);
          v[g * 8 + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 w = reinterpret_cast<const float4*>(src)[j];
          v[g * 8 + 4 * j] = w.x; v[g * 8 + 4 * j + 1] = w.y;
          v[g * 8 + 4 * j + 2] = w.z; v[g * 8 + 4 * j + 3] = w.w;
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j) v[j] = lane + 32 * j < a.d_c ? (float)c[lane + 32 * j] : 0.f;
  }
  // this lane's rope pair: read before the reduction, so that both loads are in flight together
  const int npair = a.rot / 2;
  const T* kp = static_cast<const T*>(a.k) + (int64_t)i * a.k_stride;
  const int first = a.half ? lane : 2 * lane, second = a.half ? lane + npair : 2 * lane + 1;
  float ku = 0.f, kv = 0.f;
  if (lane < npair) {
    ku = (float)kp[first];
    kv = (float)kp[second];
  }

  float amax = 0.f;
  bool all_ok = true;
#pragma unroll
  for (int j = 0; j < PER_LANE; ++j) {
    const bool ok = finite(v[j]);
    all_ok &= ok;
    amax = fmaxf(amax, ok ? fabsf(v[j]) : 0.f);
  }
  if (__any_sync(0xffffffffu, !all_ok) && lane == 0) record_error(a.d_err, KDV_DERR_RANGE);
  float s;
  if (a.static_scale) {
    s = a.scale[slot >> a.block_log2];
    if (!(s > 0.f) || !finite(s)) {
      if (lane == 0) record_error(a.d_err, KDV_DERR_RANGE);
      return;
    }
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    s = amax == 0.f ? 1.f : ldexpf(1.f, scale_exponent(amax));
    if (lane == 0) a.scale[slot] = s;
  }
  uint8_t* dst = a.c8 + slot * a.d_c;
  if constexpr (FAST) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j / 4] |= (uint32_t)e4m3(v[g * 8 + j] / s, finite(v[g * 8 + j])) << (8 * (j % 4));
      *reinterpret_cast<uint2*>(dst + g * 256 + lane * 8) = make_uint2(w[0], w[1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < PER_LANE; ++j)
      if (lane + 32 * j < a.d_c) dst[lane + 32 * j] = e4m3(v[j] / s, finite(v[j]));
  }
  if (a.d_r == 0) return;
  __nv_bfloat16* out = a.kr + slot * a.d_r;
  if (lane < npair) {
    const float2 w = rope_cos_sin(rope_position(a.pos, i), turns.f[lane], a.mscale);
    const float r0 = (ku * w.x - kv * w.y) / s, r1 = (ku * w.y + kv * w.x) / s;
    if (FAST && !a.half) {
      *reinterpret_cast<__nv_bfloat162*>(out + first) = __floats2bfloat162_rn(r0, r1);
    } else {
      out[first] = __float2bfloat16_rn(r0);
      out[second] = __float2bfloat16_rn(r1);
    }
  }
  for (int d = a.rot + lane; d < a.d_r; d += 32) out[d] = __float2bfloat16_rn((float)kp[d] / s);
}

bool al16(const void* p, int64_t stride, int esz) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (stride * esz) % 16 == 0;
}

template <typename T>
void launch_write(const WriteArgs& a, const RopeTurns<MAX_DR / 2>& f, bool fast, cudaStream_t s) {
  const int grid = (a.rows + WARPS - 1) / WARPS;
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
