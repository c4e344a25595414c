// rope.cu -- rotary positions for head vectors (kdv_rope, kdv_rope_freqs).
//
// (u, v) -> mscale (u cos a - v sin a, u sin a + v cos a), a = pos * inv_freq,
// for rot_dim/2 pairs of each head vector; the rest is copied.
//
// Bound: HBM for many rows (every element read and written once), launch
// latency for a verify step's. One CTA takes a group of tokens and a range of
// heads: it forms the group's (cos, sin) table once in shared memory (the
// 64-bit angles are what a per-element version would spend its time on: a
// head count of 64 would repeat each one 64 times), while the first vectors
// are on their way, then streams the vectors through registers, four 16-byte units in flight a
// thread. 8192 tokens x 64 heads x 128 dims, half of them rotated: 48.2 us (86 us with
// the loads behind the table and a division for each unit). CTAs are small, so that some load while others store: 4096
// tokens x 64 heads x 64 dims 11.0 us, 13.0 with 256 threads. (Device times in a graph; calls among others take 51 us for
// the first. In 32 bits it takes 80 us, 103 %, and with interleaved pairs 43 us, 96 % of the measured copy bandwidth.)
#include <algorithm>
#include <cmath>

#include "rope.cuh"

namespace kdv {
namespace {

constexpr int THREADS = 128;
constexpr int TABLE = 1024;      // (cos, sin) entries a CTA holds (8 KB)
constexpr int INFLIGHT = 4;      // units a thread loads before it stores the first

struct RopeArgs {
  const void* x;
  void* y;
  int64_t xt, xh, yt, yh;
  RopePos pos;
  int32_t tokens, heads, dim, rot;
  int32_t group, heads_per_cta;  // tokens and heads of one CTA
  uint32_t by_units;             // ceil(2^32 / units of a vector): i / units = i * by_units >> 32 for every i of a CTA (0: no CTA has two vectors)
  float mscale, sign;            // sign -1: the inverse turn
};

template <typename T, int V> struct Vec;
template <> struct Vec<__nv_bfloat16, 8> {
  uint4 w;
  __device__ Vec from_lane(int lane) const {
    Vec r;
    r.w = make_uint4(__shfl_sync(0xffffffffu, w.x, lane), __shfl_sync(0xffffffffu, w.y, lane), __shfl_sync(0xffffffffu, w.z, lane),
                     __shfl_sync(0xffffffffu, w.w, lane));
    return r;
  }
  __device__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ static void store(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <> struct Vec<float, 8> {
  float4 a, b;
  __device__ Vec from_lane(int lane) const {
    Vec r;
    r.a = make_float4(__shfl_sync(0xffffffffu, a.x, lane), __shfl_sync(0xffffffffu, a.y, lane), __shfl_sync(0xffffffffu, a.z, lane),
                      __shfl_sync(0xffffffffu, a.w, lane));
    r.b = make_float4(__shfl_sync(0xffffffffu, b.x, lane), __shfl_sync(0xffffffffu, b.y, lane), __shfl_sync(0xffffffffu, b.z, lane),
                      __shfl_sync(0xffffffffu, b.w, lane));
    return r;
  }
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ static void store(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};
template <typename T> struct Vec<T, 1> {
  T w;
  __device__ void load(const T* p) { w = *p; }
  __device__ void get(float (&f)[1]) const { f[0] = (float)w; }
  __device__ static void store(T* p, const float (&f)[1]) { *p = (T)f[0]; }
};

template <int N> __device__ __forceinline__ void read_pairs(float2 (&out)[N], const float2* at) {
  if constexpr (N == 1) {
    out[0] = *at;
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float4 w = reinterpret_cast<const float4*>(at)[i];
      out[2 * i] = make_float2(w.x, w.y);
      out[2 * i + 1] = make_float2(w.z, w.w);
    }
  }
}

// A unit is V elements (both members of its pairs): with V = 8 four
// interleaved pairs (NEIGHBOURS), or eight of the first half with their eight partners
// (HALVES: two Vecs); with V = 1 one pair as two scalars. Units behind the rotated
// part copy V elements. HALVES_BY_LANES: every unit is eight elements where they lie and the partner's
// come from another lane, so that a warp's accesses are whole lines (two Vecs a thread leave gaps:
// 49 us instead of 57); it takes partners that are a power of two of units apart, and vectors of whole such groups.
enum { NEIGHBOURS, HALVES, HALVES_BY_LANES };
template <typename TX, typename TY, int V, int PAIRING>
__global__ void __launch_bounds__(THREADS) rope_kernel(const __grid_constant__ RopeArgs a,
                                                       const __grid_constant__ RopeTurns<KDV_MAX_ROT / 2> turns) {
  __shared__ __align__(16) float2 table[TABLE];
  constexpr bool HALF = PAIRING != NEIGHBOURS, LANES = PAIRING == HALVES_BY_LANES;
  constexpr bool TWO = (HALF && !LANES) || V == 1;      // the pair's members are in two Vecs of a thread
  const int pairs = a.rot / 2;
  const int t0 = blockIdx.x * a.group;
  const int nt = min(a.group, a.tokens - t0);
  const int h0 = blockIdx.y * a.heads_per_cta;
  const int nh = min(a.heads_per_cta, a.heads - h0);
  const TX* x = static_cast<const TX*>(a.x);
  TY* y = static_cast<TY*>(a.y);
  const int rot_units = TWO ? pairs / V : a.rot / V;
  const int units = rot_units + (a.dim - a.rot) / V;
  const int total = nt * nh * units;
  Vec<TX, V> u[INFLIGHT], v[INFLIGHT];
  int64_t yo[INFLIGHT];
  int cs_at[INFLIGHT];                                  // the unit's place in the table, -1 behind the rotated part
  auto load = [&](int base) {
#pragma unroll
    for (int n = 0; n < INFLIGHT; ++n) {
      const int i = base + n * THREADS;
      if (i < total) {
        const int th = units == 1 ? i : (int)__umulhi((uint32_t)i, a.by_units), un = i - th * units;
        const int t = nt == 1 ? 0 : th / nh, h = th - t * nh;
        int e, second = 0;                              // the unit's element, and its partner's distance
        if (un >= rot_units) {
          e = a.rot + (un - rot_units) * V;
        } else if (HALF && !LANES) {
          e = un * V;
          second = pairs;
        } else if (V == 1) {
          e = 2 * un;
          second = 1;
        } else {
          e = un * V;
        }
        const int64_t xo = (int64_t)(t0 + t) * a.xt + (int64_t)(h0 + h) * a.xh + e;
        yo[n] = (int64_t)(t0 + t) * a.yt + (int64_t)(h0 + h) * a.yh + e;
        cs_at[n] = un < rot_units ? t * pairs + (LANES ? un * V & (pairs - 1) : un * (TWO ? V : V / 2)) : -1;
        u[n].load(x + xo);
        if (TWO && un < rot_units) v[n].load(x + xo + second);
      }
    }
  };
  load(threadIdx.x);
  for (int i = threadIdx.x; i < nt * pairs; i += THREADS) {
    const int t = i / pairs, k = i - t * pairs;
    float2 cs = rope_cos_sin(rope_position(a.pos, t0 + t), turns.f[k], a.mscale);
    cs.y *= a.sign;
    table[i] = cs;
  }
  __syncthreads();
  for (int base = threadIdx.x; base - (int)(threadIdx.x & 31) < total; base += THREADS * INFLIGHT) {
    if (base != (int)threadIdx.x) load(base);
#pragma unroll
    for (int n = 0; n < INFLIGHT; ++n) {
      const int i = base + n * THREADS;
      if constexpr (LANES) {
        // the partner's elements are `apart` lanes away; its lane is in range where this one is
        const int apart = pairs / V;
        v[n] = u[n].from_lane((threadIdx.x & 31) ^ apart);
        if (i < total) {
          float f[V], g[V];
          u[n].get(f);
          if (cs_at[n] >= 0) {
            float2 cs[V];
            read_pairs(cs, table + cs_at[n]);
            const float side = i & apart ? 1.f : -1.f;  // second halves add u sin, first ones take v sin away
            v[n].get(g);
#pragma unroll
            for (int k = 0; k < V; ++k) f[k] = f[k] * cs[k].x + side * cs[k].y * g[k];
          }
          Vec<TY, V>::store(y + yo[n], f);
        }
        continue;
      }
      if (i < total) {
        float f[V], g[V];
        u[n].get(f);
        if (cs_at[n] >= 0) {
          float2 cs[TWO || LANES ? V : V / 2];                   // (in 16-byte pieces: a unit's entries begin at one)
          read_pairs(cs, table + cs_at[n]);
          if constexpr (TWO) {
            v[n].get(g);
#pragma unroll
            for (int k = 0; k < V; ++k) {
              const float2 w = cs[k];
              const float p = f[k], q = g[k];
              f[k] = p * w.x - q * w.y;
              g[k] = p * w.y + q * w.x;
            }
            Vec<TY, V>::store(y + yo[n] + (HALF ? pairs : 1), g);
          } else {
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
              const float2 w = cs[k];
              const float p = f[2 * k], q = f[2 * k + 1];
              f[2 * k] = p * w.x - q * w.y;
              f[2 * k + 1] = p * w.y + q * w.x;
            }
          }
        }
        Vec<TY, V>::store(y + yo[n], f);
      }
    }
  }
}

template <typename TX, typename TY>
void launch_typed(const RopeArgs& a, const RopeTurns<KDV_MAX_ROT / 2>& f, bool half, bool vec, bool lanes, dim3 grid, cudaStream_t s) {
  if (vec) {
    if (lanes) rope_kernel<TX, TY, 8, HALVES_BY_LANES><<<grid, THREADS, 0, s>>>(a, f);
    else if (half) rope_kernel<TX, TY, 8, HALVES><<<grid, THREADS, 0, s>>>(a, f);
    else rope_kernel<TX, TY, 8, NEIGHBOURS><<<grid, THREADS, 0, s>>>(a, f);
  } else {
    if (half) rope_kernel<TX, TY, 1, HALVES><<<grid, THREADS, 0, s>>>(a, f);
    else rope_kernel<TX, TY, 1, NEIGHBOURS><<<grid, THREADS, 0, s>>>(a, f);
  }
}

// Whether two of the n x m vectors of dim elements at i * s + j * t (i < n, j < m) overlap; s and t >= 0.
bool vectors_overlap(int64_t n, int64_t s, int64_t m, int64_t t, int64_t dim) {
  if (n > m) return vectors_overlap(m, t, n, s, dim);
  if (m > 1 && t < dim) return true;
  if (n == 1 || (__int128)s >= (__int128)(m - 1) * t + dim) return false;            // whole rows apart,
  if (s >= dim && (__int128)t >= (__int128)(n - 1) * s + dim) return false;         // or whole columns
  for (int64_t i = 1; i < n; ++i) {                     // i s apart along one axis: against the nearest multiples of t
    const __int128 d = (__int128)i * s;
    const __int128 j = m > 1 ? d / t : 0;
    if (j >= m) return false;                           // behind the last vector, by t or more; so are all the others
    if (d - j * t < dim || (j + 1 < m && (j + 1) * t - d < dim)) return true;
  }
  return false;
}

bool rows16(const void* p, int64_t ts, int64_t hs, int esz) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ts * esz) % 16 == 0 && (hs * esz) % 16 == 0;
}

}  // namespace
}  // namespace kdv

using namespace kdv;

extern "C" {

kdv_status kdv_rope_freqs(int32_t rot_dim, double base, int32_t rule, double factor, double trained_len,
                          double beta_fast, double beta_slow, double* inv_freq, double* mscale) {
  if (inv_freq == nullptr || rot_dim < 2 || rot_dim % 2 || rot_dim > KDV_MAX_ROT) return KDV_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base)) return KDV_ERR_INVALID_ARG;
  if (rule < KDV_ROPE_SCALE_NONE || rule > KDV_ROPE_SCALE_YARN) return KDV_ERR_INVALID_ARG;
  if (rule != KDV_ROPE_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return KDV_ERR_INVALID_ARG;
  if (rule == KDV_ROPE_SCALE_NTK) {
    if (rot_dim < 4) return KDV_ERR_INVALID_ARG;
    base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  }
  double low = 0.0, high = 0.0;
  if (rule == KDV_ROPE_SCALE_YARN) {
    if (!(trained_len >= 1.0) || !std::isfinite(trained_len) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) ||
        !std::isfinite(beta_fast))
      return KDV_ERR_INVALID_ARG;
    // the pair index that makes `turns` turns over the trained length
    const double two_pi = 6.283185307179586476925286766559;
    auto index = [&](double turns) {
      return rot_dim * std::log(trained_len / (turns * two_pi)) / (2.0 * std::log(base));
    };
    low = std::max(std::floor(index(beta_fast)), 0.0);
    high = std::min(std::ceil(index(beta_slow)), (double)rot_dim - 1.0);
  }
  for (int k = 0; k < rot_dim / 2; ++k) {
    const double f = std::pow(base, -2.0 * k / rot_dim);
    if (rule == KDV_ROPE_SCALE_LINEAR) {
      inv_freq[k] = f / factor;
    } else if (rule == KDV_ROPE_SCALE_YARN) {
      const double r = std::min(std::max((k - low) / std::max(high - low, 1e-3), 0.0), 1.0);
      inv_freq[k] = f / factor * r + f * (1.0 - r);
    } else {
      inv_freq[k] = f;
    }
  }
  if (mscale != nullptr) *mscale = rule == KDV_ROPE_SCALE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return KDV_OK;
}

kdv_status kdv_rope(const kdv_rope_params* p, void* stream) {
  if (p == nullptr) return KDV_ERR_INVALID_ARG;
  if (p->tokens < 0 || p->heads < 1 || p->dim < 1) return KDV_ERR_INVALID_ARG;
  if (p->rot_dim < 2 || p->rot_dim % 2 || p->rot_dim > p->dim) return KDV_ERR_INVALID_ARG;
  if (p->rot_dim > KDV_MAX_ROT) return KDV_ERR_UNSUPPORTED;
  if (p->layout != KDV_ROPE_INTERLEAVED && p->layout != KDV_ROPE_HALF) return KDV_ERR_INVALID_ARG;
  if (p->inverse != 0 && p->inverse != 1) return KDV_ERR_INVALID_ARG;
  if ((p->x_dtype != KDV_BF16 && p->x_dtype != KDV_F32) || (p->y_dtype != KDV_BF16 && p->y_dtype != KDV_F32))
    return KDV_ERR_INVALID_ARG;
  if (p->h_inv_freq == nullptr || !std::isfinite(p->mscale)) return KDV_ERR_INVALID_ARG;
  for (int k = 0; k < p->rot_dim / 2; ++k)
    if (!std::isfinite(p->h_inv_freq[k])) return KDV_ERR_INVALID_ARG;
  for (const int64_t stride : {p->x_head_stride, p->y_token_stride, p->y_head_stride})
    if (stride == INT64_MIN) return KDV_ERR_INVALID_ARG;                // (has no magnitude)
  if (p->heads > 1 && (std::llabs(p->x_head_stride) < p->dim || std::llabs(p->y_head_stride) < p->dim))
    return KDV_ERR_INVALID_ARG;
  if (p->tokens == 0) return KDV_OK;
  if (p->x == nullptr || p->y == nullptr) return KDV_ERR_INVALID_ARG;
  if (vectors_overlap(p->tokens, std::llabs(p->y_token_stride), p->heads, std::llabs(p->y_head_stride), p->dim))
    return KDV_ERR_INVALID_ARG;                                         // elements written twice
  const int xe = p->x_dtype == KDV_BF16 ? 2 : 4, ye = p->y_dtype == KDV_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(p->x) % xe || reinterpret_cast<uintptr_t>(p->y) % ye) return KDV_ERR_INVALID_ARG;
  if (p->x == p->y && (xe != ye || (p->tokens > 1 && p->x_token_stride != p->y_token_stride) ||
                       (p->heads > 1 && p->x_head_stride != p->y_head_stride)))
    return KDV_ERR_INVALID_ARG;
  if (p->pos == nullptr) {
    if (p->batch < 1 || !p->tree_off || !p->prefix_len || !p->depth) return KDV_ERR_INVALID_ARG;
    if (p->batch > KDV_MAX_BATCH) return KDV_ERR_UNSUPPORTED;
  }
  RopeArgs a = {};
  a.x = p->x;
  a.y = p->y;
  a.xt = p->tokens > 1 ? p->x_token_stride : 0;
  a.yt = p->tokens > 1 ? p->y_token_stride : 0;
  a.xh = p->heads > 1 ? p->x_head_stride : 0;
  a.yh = p->heads > 1 ? p->y_head_stride : 0;
  a.pos = {p->pos, p->tree_off, p->prefix_len, p->depth, p->batch};
  a.tokens = p->tokens;
  a.heads = p->heads;
  a.dim = p->dim;
  a.rot = p->rot_dim;
  a.mscale = p->mscale;
  a.sign = p->inverse ? -1.f : 1.f;
  RopeTurns<KDV_MAX_ROT / 2> f = {};
  for (int k = 0; k < p->rot_dim / 2; ++k) f.f[k] = p->h_inv_freq[k] / 6.283185307179586476925286766559;
  const bool half = p->layout == KDV_ROPE_HALF;
  const bool vec = p->rot_dim % (half ? 16 : 8) == 0 && p->dim % 8 == 0 && rows16(p->x, a.xt, a.xh, xe) &&
                   rows16(p->y, a.yt, a.yh, ye);
  // One pass of the CTA's threads (INFLIGHT units each) is its share: whole
  // tokens while their vectors are few, else a range of one token's heads. (Four passes a CTA
  // measured 65 us where one takes 57: CTAs that wait for their angles cover one another.)
  const int V = vec ? 8 : 1, pairs = p->rot_dim / 2, apart = pairs / 8;
  const bool lanes = vec && half && (apart & (apart - 1)) == 0 && apart <= 16 && p->dim / 8 % (2 * apart) == 0;
  const int64_t units = (((half && !lanes) || V == 1) ? pairs / V : p->rot_dim / V) + (p->dim - p->rot_dim) / V;
  // A CTA's units: one a thread until every SM has four CTAs, then up to as many as are in flight. 13 tokens x 64 heads
  // x 64 dims: 2.4 us (3.2 in CTAs of four units a thread, of which there are 7); 416 tokens: 3.2 us (3.8).
  const int64_t deep = std::max<int64_t>(1, std::min<int64_t>(INFLIGHT, (int64_t)p->tokens * p->heads * units / (4 * 148 * THREADS)));
  const int64_t share = THREADS * deep;
  a.heads_per_cta = (int)std::max<int64_t>(1, std::min<int64_t>(p->heads, share / std::max<int64_t>(1, units)));
  a.group = a.heads_per_cta < p->heads
                ? 1
                : (int)std::max<int64_t>(1, std::min<int64_t>(TABLE / pairs, share / (units * p->heads)));
  a.by_units = units == 1 || units > 65535 ? 0 : (uint32_t)(((1ull << 32) + units - 1) / units);
  const int64_t gx = ((int64_t)p->tokens + a.group - 1) / a.group;
  const int64_t gy = ((int64_t)p->heads + a.heads_per_cta - 1) / a.heads_per_cta;
  if (gy > 65535 || units * a.heads_per_cta * a.group > INT32_MAX / 2) return KDV_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)gx, (unsigned)gy);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (xe == 2 && ye == 2) launch_typed<__nv_bfloat16, __nv_bfloat16>(a, f, half, vec, lanes, grid, s);
  else if (xe == 2) launch_typed<__nv_bfloat16, float>(a, f, half, vec, lanes, grid, s);
  else if (ye == 2) launch_typed<float, __nv_bfloat16>(a, f, half, vec, lanes, grid, s);
  else launch_typed<float, float>(a, f, half, vec, lanes, grid, s);
  return cudaGetLastError() == cudaSuccess ? KDV_OK : KDV_ERR_CUDA;
}

}  // extern "C"
