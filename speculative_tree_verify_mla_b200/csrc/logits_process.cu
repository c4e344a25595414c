// logits_process.cu -- penalties, biases and grammar masks on the target
// logits of a draft tree's nodes (kdv_logits_process).
//
//   x > 0 ? x / r : x * r where the token was seen; x - f made - p [made > 0]
//   + bias; -inf where the grammar forbids it. made counts the request's own
//   output tokens in its history plus the drafted tokens on the node's path.
//
// Bound: HBM (every logit read and written once, 1/8 byte of grammar mask);
// for one request's tree the fixed part: launch, and the history's way from L2.
// One CTA takes a tile of the vocabulary for some nodes of one request. It counts the
// request's history into a table of the tile's tokens in shared memory (the
// history is read from L2 by every tile's CTA; a table of counts in memory would be 4 bytes a token
// a request, twice a bf16 row). A thread then notes whether any of its eight tokens has a count or a
// bias at all and streams the logits, two nodes in flight, the first two asked for before the history is read. Drafted tokens are not counted into the table:
// each one in the tile has a number there, and a small matrix says how often
// node t's path holds it, so the nodes need no barrier between them.
// 13 nodes of 163840 tokens with 5553 of history: 9.8 us (38 with the tile's nodes one after
// another and the path counted in and out around each); 160 nodes in fp32: 49 us (87), the logits
// read as streaming data, so that the results stay in L2 (53 otherwise); in bf16
// 40 us. (Device times in a graph; calls among others take 12, 52 and 42 us. 64 registers a thread for four CTAs an SM,
// 36 to 44 bytes of them spilled.)
#include <cuda_bf16.h>

#include <algorithm>

#include "kdv_internal.cuh"

namespace kdv {
namespace {

constexpr int THREADS = 256;
constexpr int TOKENS = 8;                  // tokens a thread holds
constexpr int TILE = THREADS * TOKENS;     // tokens a CTA holds
constexpr int NODES = 2;                   // a CTA's nodes at least: one in hand, one on its way
constexpr int L2_AHEAD = 3;                // nodes behind the one in hand whose logits are asked for into L2

struct LogitsArgs {
  const void* x;
  void* y;
  int64_t x_ld, y_ld;
  const int32_t* tree_off;
  const int32_t* parent;
  const int32_t* token;
  const int32_t* hist;
  int64_t hist_ld;
  const int32_t* hist_len;
  const int32_t* prompt_len;
  const float* repetition;
  const float* presence;
  const float* frequency;
  const int32_t* bias_off;
  const int32_t* bias_token;
  const float* bias_value;
  const uint32_t* allow;
  int64_t allow_ld;
  const int32_t* allow_row;
  int32_t* d_err;
  int32_t allow_rows, max_T, total_nodes, vocab;
  int32_t chunk;           // nodes of one CTA
};

// word: 2 * made + (1 if the prompt holds the token)
__device__ __forceinline__ float process(float x, uint32_t word, float bias, float rep, float inv, bool normal, float pres, float freq) {
  if (word != 0u) {
    const float low = normal ? x * inv : x / rep;
    x = x > 0.f ? low : x * rep;
    const uint32_t made = word >> 1;
    x -= freq * (float)made;
    if (made != 0u) x -= pres;
  }
  return x + bias;
}

// A thread's eight logits of a node: neighbours in 16-byte pieces (VEC), or 256 apart.
template <typename T, bool VEC> struct Row;
template <> struct Row<__nv_bfloat16, true> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int) { w = __ldcs(reinterpret_cast<const uint4*>(p + TOKENS * threadIdx.x)); }
  __device__ __forceinline__ float get(int j) const {
    const uint32_t u = j < 2 ? w.x : j < 4 ? w.y : j < 6 ? w.z : w.w;
    return __uint_as_float(j % 2 ? u & 0xffff0000u : u << 16);
  }
};
template <> struct Row<float, true> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, int) {
    a = __ldcs(reinterpret_cast<const float4*>(p + TOKENS * threadIdx.x));
    b = __ldcs(reinterpret_cast<const float4*>(p + TOKENS * threadIdx.x) + 1);
  }
  __device__ __forceinline__ float get(int j) const {
    return j == 0 ? a.x : j == 1 ? a.y : j == 2 ? a.z : j == 3 ? a.w : j == 4 ? b.x : j == 5 ? b.y : j == 6 ? b.z : b.w;
  }
};
template <typename T> struct Row<T, false> {
  T v[TOKENS];
  __device__ __forceinline__ void load(const T* p, int n) {
#pragma unroll
    for (int j = 0; j < TOKENS; ++j)
      if ((int)threadIdx.x + j * THREADS < n) v[j] = p[threadIdx.x + j * THREADS];
  }
  __device__ __forceinline__ float get(int j) const { return (float)v[j]; }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// grid (batch, tiles, chunks of nodes). VEC: rows of both sides 16-byte
// aligned and the tile whole; the launch's other tiles (the last one) take the scalar form.
template <typename TX, typename TY, bool VEC>
__device__ __forceinline__ void process_tile(const LogitsArgs& a, uint32_t* count, float* bias, uint8_t* number,
                                             uint8_t (*times)[KDV_MAX_TREE], int* par, int* tok) {
  const int tid = threadIdx.x, b = blockIdx.x, v0 = blockIdx.y * TILE, n = min(TILE, a.vocab - v0);
  const bool reports = blockIdx.y == 0 && blockIdx.z == 0;  // what every CTA of the request sees
  // the request's scalars, all asked for at once
  const int t0 = a.tree_off[b], T = a.tree_off[b + 1] - t0;
  int len = a.hist ? a.hist_len[b] : 0;
  const int pl = a.hist && a.prompt_len ? a.prompt_len[b] : 0;
  const int bias_lo = a.bias_off ? a.bias_off[b] : 0, bias_hi = a.bias_off ? a.bias_off[b + 1] : 0;
  float rep = a.repetition ? a.repetition[b] : 1.f;
  const float pres = a.presence ? a.presence[b] : 0.f, freq = a.frequency ? a.frequency[b] : 0.f;
  if (T < 0 || T > a.max_T || t0 < 0 || t0 > a.total_nodes - T) {
    if (reports && tid == 0) record_error(a.d_err, KDV_DERR_BAD_LENGTH);
    return;
  }
  const int first = blockIdx.z * a.chunk, last = min(T, first + a.chunk);
  if (first >= last) return;
  const TX* x = static_cast<const TX*>(a.x) + (int64_t)t0 * a.x_ld + v0;
  TY* y = static_cast<TY*>(a.y) + (int64_t)t0 * a.y_ld + v0;
  // grammar row of node t (null: unconstrained)
  auto allowed = [&](int t) -> const uint32_t* {
    if (a.allow == nullptr) return nullptr;
    const int row = a.allow_row ? a.allow_row[t0 + t] : t0 + t;
    if (row >= a.allow_rows) {
      if (blockIdx.y == 0 && tid == 0) record_error(a.d_err, KDV_DERR_BAD_TOKEN);
      return nullptr;
    }
    return row < 0 ? nullptr : a.allow + (int64_t)row * a.allow_ld + v0 / 32;
  };
  auto bits_of = [&](const uint32_t* row) -> uint32_t {     // bit j: this thread's token j
    if (row == nullptr) return 0xffu;
    if (VEC) return reinterpret_cast<const uint8_t*>(row)[tid];
    uint32_t bits = 0;
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) {
      const int i = tid + j * THREADS;
      if (i < n) bits |= ((row[i / 32] >> (i % 32)) & 1u) << j;
    }
    return bits;
  };
  int node_parent = -1, node_token = 0;
  if (a.parent != nullptr && tid < T) {
    node_parent = a.parent[t0 + tid];
    node_token = a.token[t0 + tid];
  }
  Row<TX, VEC> r, ahead;
  uint32_t bits = 0xffu, bits_ahead = 0xffu;
  r.load(x + (int64_t)first * a.x_ld, n);
  bits = bits_of(allowed(first));

  // The CTA's next rows come into L2 while it counts the history (160 nodes in fp32: 53 us, 59 without).
  auto to_l2 = [&](int t) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(x + (int64_t)t * a.x_ld), "r"((uint32_t)(TILE * sizeof(TX))) : "memory");
  };
  if (VEC && tid > 0 && tid <= L2_AHEAD && first + tid < last) to_l2(first + tid);

  for (int i = tid; i < TILE / 4; i += THREADS) {
    reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
    reinterpret_cast<uint4*>(bias)[i] = make_uint4(0, 0, 0, 0);
    reinterpret_cast<uint32_t*>(number)[i] = 0u;
  }
  if (!(rep > 0.f) || !(rep <= 3.402823466e38f)) {
    if (reports && tid == 0) record_error(a.d_err, KDV_DERR_BAD_SCORE);
    rep = 1.f;
  }
  // the tree's path data
  bool bad = false, mine = false;
  if (a.parent != nullptr && tid < T) {
    const int p = node_parent, k = node_token;
    bad = p < -1 || p >= tid;
    const bool bad_tok = p >= 0 && (k < 0 || k >= a.vocab);
    if (reports && (bad || bad_tok)) record_error(a.d_err, bad ? KDV_DERR_BAD_PARENT : KDV_DERR_BAD_TOKEN);
    par[tid] = p;
    mine = p >= 0 && k >= v0 && k - v0 < n;                 // roots are in the history already
    tok[tid] = mine ? k - v0 : -1;
  }
  const bool tree_ok = !__syncthreads_or(bad);
  const bool drafted = __syncthreads_or(mine) && tree_ok;   // else no node of this tile needs its path
  if (drafted) {
    if (mine) {                                             // the token's number: 1 + its first node
      int w = 0;
      while (tok[w] != tok[tid]) ++w;
      number[tok[tid]] = (uint8_t)(w + 1);
    }
    for (int i = tid; i < T * T; i += THREADS) times[i / T][i % T] = 0;
  }
  // history: made tokens add 2, prompt tokens set bit 0
  if (a.hist != nullptr) {
    if (len < 0 || len > a.hist_ld || pl < 0 || pl > a.hist_ld) {   // (pl needs no clamp: i < len <= hist_ld)
      if (reports && tid == 0) record_error(a.d_err, KDV_DERR_BAD_LENGTH);
      len = (int)min((int64_t)max(len, 0), a.hist_ld);
    }
    const int32_t* h = a.hist + b * a.hist_ld;
    auto add = [&](uint32_t i, uint32_t at) {
      if (at < (uint32_t)n) {
        if ((int)i < pl) atomicOr(&count[at], 1u); else atomicAdd(&count[at], 2u);
      }
    };
    // Nearly every token is another tile's: four at a time, one branch for them all.
    const uint32_t fours = reinterpret_cast<uintptr_t>(h) % 16 == 0 ? (uint32_t)len / 4 : 0u;
    constexpr int FLIGHT = 4;
    for (uint32_t base = tid; base < fours; base += THREADS * FLIGHT) {
      int4 k[FLIGHT];
#pragma unroll
      for (int j = 0; j < FLIGHT; ++j)
        k[j] = base + j * THREADS < fours ? reinterpret_cast<const int4*>(h)[base + j * THREADS] : make_int4(v0 - 1, v0 - 1, v0 - 1, v0 - 1);
#pragma unroll
      for (int j = 0; j < FLIGHT; ++j) {
        const uint32_t i = 4 * (base + j * THREADS);
        const uint32_t w = (uint32_t)k[j].x - v0, x = (uint32_t)k[j].y - v0, y = (uint32_t)k[j].z - v0, z = (uint32_t)k[j].w - v0;
        if (min(min(w, x), min(y, z)) < (uint32_t)n) {
          add(i, w);
          add(i + 1, x);
          add(i + 2, y);
          add(i + 3, z);
        }
      }
    }
    for (uint32_t i = 4 * fours + tid; i < (uint32_t)len; i += THREADS) add(i, (uint32_t)h[i] - v0);
    if (reports)
      for (uint32_t i = tid; i < (uint32_t)len; i += THREADS)
        if (h[i] < 0 || h[i] >= a.vocab) record_error(a.d_err, KDV_DERR_BAD_TOKEN);
  }
  // biases: ascending tokens, so the tile's entries are one range
  if (a.bias_off != nullptr) {
    const int lo = bias_lo, hi = bias_hi;
    int s = lo, e = hi;
    // first entry with token >= v0; a short list is read through instead (the search's steps wait for one another)
    while (hi - lo > 16 * THREADS && s < e) {
      const int mid = s + (e - s) / 2;
      if (a.bias_token[mid] < v0) s = mid + 1; else e = mid;
    }
    for (int i = s + tid; i < hi; i += THREADS) {
      const int k = a.bias_token[i];
      if (k >= v0 + n) break;
      if (k >= v0 && (i == lo || a.bias_token[i - 1] < k)) bias[k - v0] = a.bias_value[i];
    }
    if (reports)
      for (int i = lo + tid; i < hi; i += THREADS) {
        const int k = a.bias_token[i];
        if (k < 0 || k >= a.vocab || (i > lo && a.bias_token[i - 1] >= k)) record_error(a.d_err, KDV_DERR_BAD_TOKEN);
      }
  }
  __syncthreads();
  if (drafted) {
    if (tid < T)
      for (int u = tid; u >= 0; u = par[u])
        if (tok[u] >= 0) ++times[tid][number[tok[u]] - 1];
    __syncthreads();
  }

  auto at = [&](int j) { return VEC ? TOKENS * tid + j : tid + j * THREADS; };
  uint32_t touched = 0;                                     // not 0: some of this thread's tokens have a count or a bias
  if (VEC) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint4 x = reinterpret_cast<const uint4*>(count)[2 * tid + q], z = reinterpret_cast<const uint4*>(bias)[2 * tid + q];
      touched |= x.x | x.y | x.z | x.w | z.x | z.y | z.z | z.w;
      if (drafted) touched |= reinterpret_cast<const uint32_t*>(number)[2 * tid + q];
    }
  } else {
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) touched |= count[at(j)] | __float_as_uint(bias[at(j)]) | number[at(j)];
  }
  // x / rep as a product where 1 / rep is a normal number (an fp32 rounding more; dividing takes 10.6 us where this takes
  // 9.8, and 39.5 for 2 x 64 bf16 nodes where this takes 32.5)
  const float inv = 1.f / rep;
  const bool normal = inv >= 1.17549435e-38f && inv <= 3.402823466e38f;
  for (int t = first; t < last; ++t) {
    if (t + 1 < last) {
      ahead.load(x + (int64_t)(t + 1) * a.x_ld, n);
      bits_ahead = bits_of(allowed(t + 1));
      if (VEC && tid == 0 && t + 1 + L2_AHEAD < last) to_l2(t + 1 + L2_AHEAD);
    }
    float f[TOKENS];
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) f[j] = r.get(j);
    if (touched != 0) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {                         // four tokens at a time
        uint32_t w[4], id[4] = {0, 0, 0, 0};
        float add[4];
        if (VEC) {
          const uint4 c = reinterpret_cast<const uint4*>(count)[2 * tid + q];
          const float4 z = reinterpret_cast<const float4*>(bias)[2 * tid + q];
          w[0] = c.x; w[1] = c.y; w[2] = c.z; w[3] = c.w;
          add[0] = z.x; add[1] = z.y; add[2] = z.z; add[3] = z.w;
          if (drafted) {
            const uint32_t u = reinterpret_cast<const uint32_t*>(number)[2 * tid + q];
#pragma unroll
            for (int j = 0; j < 4; ++j) id[j] = (u >> (8 * j)) & 0xffu;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w[j] = count[at(4 * q + j)];
            add[j] = bias[at(4 * q + j)];
            if (drafted) id[j] = number[at(4 * q + j)];
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (id[j] != 0) w[j] += 2u * times[t][id[j] - 1];
          f[4 * q + j] = process(f[4 * q + j], w[j], add[j], rep, inv, normal, pres, freq);
        }
      }
    }
    if (bits != 0xffu) {
#pragma unroll
      for (int j = 0; j < TOKENS; ++j)
        if (!((bits >> j) & 1u)) f[j] = __int_as_float(0xff800000);
    }
    TY* row = y + (int64_t)t * a.y_ld;
    if (VEC) {
      store8(row + TOKENS * tid, f);
    } else {
#pragma unroll
      for (int j = 0; j < TOKENS; ++j)
        if (at(j) < n) row[at(j)] = (TY)f[j];
    }
    r = ahead;
    bits = bits_ahead;
  }
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(THREADS, 4) logits_process_kernel(const __grid_constant__ LogitsArgs a, int vec) {
  __shared__ __align__(16) uint32_t count[TILE];
  __shared__ __align__(16) float bias[TILE];
  __shared__ __align__(16) uint8_t number[TILE], times[KDV_MAX_TREE][KDV_MAX_TREE];
  __shared__ int par[KDV_MAX_TREE], tok[KDV_MAX_TREE];
  if (vec && (int64_t)(blockIdx.y + 1) * TILE <= a.vocab) process_tile<TX, TY, true>(a, count, bias, number, times, par, tok);
  else process_tile<TX, TY, false>(a, count, bias, number, times, par, tok);
}

template <typename TX, typename TY>
cudaError_t launch_logits(const LogitsArgs& a, int batch, bool vec, cudaStream_t s) {
  const dim3 grid((unsigned)batch, (unsigned)(((int64_t)a.vocab + TILE - 1) / TILE), (unsigned)((a.max_T + a.chunk - 1) / a.chunk));
  logits_process_kernel<TX, TY><<<grid, THREADS, 0, s>>>(a, vec ? 1 : 0);
  return cudaGetLastError();
}

bool rows_aligned(const void* p, int64_t ld, int esz) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * esz) % 16 == 0;
}

}  // namespace
}  // namespace kdv

using namespace kdv;

extern "C" kdv_status kdv_logits_process(const kdv_logits_params* p, void* stream) {
  if (p == nullptr || p->batch < 1 || p->max_T < 1 || p->total_nodes < 0 || p->vocab < 1) return KDV_ERR_INVALID_ARG;
  if (p->batch > KDV_MAX_BATCH || p->max_T > KDV_MAX_TREE || p->vocab > 65535 * TILE) return KDV_ERR_UNSUPPORTED;
  if ((p->dtype != KDV_BF16 && p->dtype != KDV_F32) || (p->out_dtype != KDV_BF16 && p->out_dtype != KDV_F32))
    return KDV_ERR_INVALID_ARG;
  if (p->logits_ld < p->vocab || p->out_ld < p->vocab) return KDV_ERR_INVALID_ARG;
  if (p->total_nodes == 0) return KDV_OK;
  if (!p->logits || !p->out || !p->tree_off) return KDV_ERR_INVALID_ARG;
  if ((p->parent == nullptr) != (p->token == nullptr)) return KDV_ERR_INVALID_ARG;
  if (p->hist && (!p->hist_len || p->hist_ld < 0)) return KDV_ERR_INVALID_ARG;
  if (p->bias_off && (!p->bias_token || !p->bias_value)) return KDV_ERR_INVALID_ARG;
  if (p->allow && (p->allow_ld < (p->vocab + 31) / 32 || p->allow_rows < 0)) return KDV_ERR_INVALID_ARG;
  if (p->allow && !p->allow_row && p->allow_rows < p->total_nodes) return KDV_ERR_INVALID_ARG;
  const int xe = p->dtype == KDV_BF16 ? 2 : 4, ye = p->out_dtype == KDV_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(p->logits) % xe || reinterpret_cast<uintptr_t>(p->out) % ye) return KDV_ERR_INVALID_ARG;
  if (p->logits == p->out && (xe != ye || p->logits_ld != p->out_ld)) return KDV_ERR_INVALID_ARG;
  LogitsArgs a = {};
  a.x = p->logits;
  a.y = p->out;
  a.x_ld = p->logits_ld;
  a.y_ld = p->out_ld;
  a.tree_off = p->tree_off;
  a.parent = p->parent;
  a.token = p->token;
  a.hist = p->hist;
  a.hist_ld = p->hist_ld;
  a.hist_len = p->hist_len;
  a.prompt_len = p->prompt_len;
  a.repetition = p->repetition;
  a.presence = p->presence;
  a.frequency = p->frequency;
  a.bias_off = p->bias_off;
  a.bias_token = p->bias_token;
  a.bias_value = p->bias_value;
  a.allow = p->allow;
  a.allow_ld = p->allow_ld;
  a.allow_row = p->allow_row;
  a.allow_rows = p->allow_rows;
  a.d_err = p->d_err;
  a.max_T = p->max_T;
  a.total_nodes = p->total_nodes;
  a.vocab = p->vocab;
  // Nodes of a CTA: all of a tree once the tiles alone fill the GPU (each more
  // CTA counts the history again), else as few as are in flight at once.
  const int64_t tiles = ((int64_t)p->vocab + TILE - 1) / TILE * p->batch;
  const int64_t chunks = std::max<int64_t>(1, std::min<int64_t>((p->max_T + NODES - 1) / NODES, (4 * 148 + tiles - 1) / tiles));
  a.chunk = (int)(((p->max_T + chunks - 1) / chunks + NODES - 1) / NODES * NODES);
  const bool vec = rows_aligned(p->logits, p->logits_ld, xe) && rows_aligned(p->out, p->out_ld, ye);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (xe == 2 && ye == 2) e = launch_logits<__nv_bfloat16, __nv_bfloat16>(a, p->batch, vec, s);
  else if (xe == 2) e = launch_logits<__nv_bfloat16, float>(a, p->batch, vec, s);
  else if (ye == 2) e = launch_logits<float, __nv_bfloat16>(a, p->batch, vec, s);
  else e = launch_logits<float, float>(a, p->batch, vec, s);
  return e == cudaSuccess ? KDV_OK : KDV_ERR_CUDA;
}
