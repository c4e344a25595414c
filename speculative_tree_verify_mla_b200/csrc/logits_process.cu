// logits_process.cu -- penalties, biases and grammar masks on the target
// logits of a draft tree's nodes (kdv_logits_process).
//
//   x > 0 ? x / r : x * r where the token was seen; x - f made - p [made > 0]
//   + bias; -inf where the grammar forbids it. made counts the request's own
//   output tokens in its history plus the drafted tokens on the node's path.
//
// Bound: HBM (every logit read and written once, 1/8 byte of grammar mask).
// One CTA takes a tile of the vocabulary for all nodes of one request: it
// counts the request's history into a table of the tile's tokens in shared
// memory once (the history is read from L2 by every tile's CTA; a table of
// counts in memory would be 4 bytes a token a request, twice a bf16 row), adds
// the biases, and then streams each node's logits through registers. A node's
// path holds at most 64 tokens: where some of them fall into the tile, their
// counts are added for that node and taken away again after it.
#include <cuda_bf16.h>

#include <algorithm>

#include "kdv_internal.cuh"

namespace kdv {
namespace {

constexpr int THREADS = 256;

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
  int32_t allow_rows, max_T, total_nodes, vocab, tile;
};

// count word: 2 * made + (1 if the prompt holds the token)
__device__ __forceinline__ float process(float x, uint32_t word, float bias, float rep, float pres, float freq) {
  if (word != 0u) {
    x = x > 0.f ? x / rep : x * rep;
    const uint32_t made = word >> 1;
    x -= freq * (float)made;
    if (made != 0u) x -= pres;
  }
  return x + bias;
}

template <typename T> __device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}
template <typename T> __device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// grid (tiles, batch). VEC: rows of both sides 16-byte aligned.
template <typename TX, typename TY, bool VEC>
__global__ void __launch_bounds__(THREADS) logits_process_kernel(const __grid_constant__ LogitsArgs a) {
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* count = smem;                                   // [tile]
  float* bias = reinterpret_cast<float*>(smem + a.tile);    // [tile]
  __shared__ int par[KDV_MAX_TREE], tok[KDV_MAX_TREE];
  const int b = blockIdx.y, v0 = blockIdx.x * a.tile, n = min(a.tile, a.vocab - v0);
  const bool first = blockIdx.x == 0 && threadIdx.x == 0;   // reports what every tile sees
  const int t0 = a.tree_off[b], T = a.tree_off[b + 1] - t0;
  if (T < 0 || T > a.max_T || t0 < 0 || t0 > a.total_nodes - T) {
    if (first) record_error(a.d_err, KDV_DERR_BAD_LENGTH);
    return;
  }
  if (T == 0) return;
  for (int i = threadIdx.x; i < a.tile; i += THREADS) {
    count[i] = 0u;
    bias[i] = 0.f;
  }
  float rep = a.repetition ? a.repetition[b] : 1.f;
  const float pres = a.presence ? a.presence[b] : 0.f, freq = a.frequency ? a.frequency[b] : 0.f;
  if (!(rep > 0.f) || !(rep <= 3.402823466e38f)) {
    if (first) record_error(a.d_err, KDV_DERR_BAD_SCORE);
    rep = 1.f;
  }
  // the tree's path data
  const bool paths = a.parent != nullptr;
  if (threadIdx.x < T && paths) {
    const int u = threadIdx.x, p = a.parent[t0 + u], k = a.token[t0 + u];
    const bool bad = p < -1 || p >= u;
    const bool bad_tok = p >= 0 && (k < 0 || k >= a.vocab);
    if (blockIdx.x == 0 && (bad || bad_tok)) record_error(a.d_err, bad ? KDV_DERR_BAD_PARENT : KDV_DERR_BAD_TOKEN);
    par[u] = p;
    tok[u] = (p < 0 || bad_tok) ? -1 : k;                   // roots are in the history already
  }
  const bool tree_ok = !__syncthreads_or(threadIdx.x < T && paths && (par[threadIdx.x] < -1 || par[threadIdx.x] >= (int)threadIdx.x));
  // history: made tokens add 2, prompt tokens set bit 0
  if (a.hist != nullptr) {
    int len = a.hist_len[b], pl = a.prompt_len ? a.prompt_len[b] : 0;
    if (len < 0 || len > a.hist_ld || pl < 0) {
      if (first) record_error(a.d_err, KDV_DERR_BAD_LENGTH);
      len = (int)min((int64_t)max(len, 0), a.hist_ld);
    }
    const int32_t* h = a.hist + b * a.hist_ld;
    for (int base = threadIdx.x; base < len; base += THREADS * 4) {
      int k[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = base + j * THREADS < len ? h[base + j * THREADS] : v0 - 1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = base + j * THREADS;
        if (i < len && blockIdx.x == 0 && (k[j] < 0 || k[j] >= a.vocab)) record_error(a.d_err, KDV_DERR_BAD_TOKEN);
        const uint32_t at = (uint32_t)k[j] - (uint32_t)v0;
        if (i < len && at < (uint32_t)n) {
          if (i < pl) atomicOr(&count[at], 1u); else atomicAdd(&count[at], 2u);
        }
      }
    }
  }
  // biases: ascending tokens, so the tile's entries are one range
  if (a.bias_off != nullptr) {
    const int lo = a.bias_off[b], hi = a.bias_off[b + 1];
    int s = lo, e = hi;
    while (s < e) {                                         // first entry with token >= v0
      const int mid = s + (e - s) / 2;
      if (a.bias_token[mid] < v0) s = mid + 1; else e = mid;
    }
    for (int i = s + threadIdx.x; i < hi; i += THREADS) {
      const int k = a.bias_token[i];
      if (k >= v0 + n) break;
      if (k >= v0 && (i == lo || a.bias_token[i - 1] < k)) bias[k - v0] = a.bias_value[i];
    }
    if (blockIdx.x == 0)
      for (int i = lo + threadIdx.x; i < hi; i += THREADS) {
        const int k = a.bias_token[i];
        if (k < 0 || k >= a.vocab || (i > lo && a.bias_token[i - 1] >= k)) record_error(a.d_err, KDV_DERR_BAD_TOKEN);
      }
  }
  __syncthreads();
  // does any drafted token fall into the tile? (else no node needs its path)
  const bool mine = paths && tree_ok && threadIdx.x < T && (uint32_t)tok[threadIdx.x] - (uint32_t)v0 < (uint32_t)n &&
                    tok[threadIdx.x] >= 0;
  const bool drafted = __syncthreads_or(mine);

  const TX* x = static_cast<const TX*>(a.x);
  TY* y = static_cast<TY*>(a.y);
  for (int t = 0; t < T; ++t) {
    const int node = t0 + t;
    if (drafted) {
      __syncthreads();
      if (threadIdx.x == 0)
        for (int u = t; u >= 0; u = par[u])
          if (tok[u] >= v0 && tok[u] - v0 < n) count[tok[u] - v0] += 2u;
      __syncthreads();
    }
    int arow = a.allow_row ? a.allow_row[node] : node;
    if (a.allow != nullptr && arow >= a.allow_rows) {
      if (first) record_error(a.d_err, KDV_DERR_BAD_TOKEN);
      arow = -1;
    }
    const uint32_t* allow = a.allow != nullptr && arow >= 0 ? a.allow + (int64_t)arow * a.allow_ld + v0 / 32 : nullptr;
    const TX* xr = x + (int64_t)node * a.x_ld + v0;
    TY* yr = y + (int64_t)node * a.y_ld + v0;
    const int nv = VEC ? n / 8 * 8 : 0;
    for (int i = threadIdx.x * 8; i < nv; i += THREADS * 8) {
      float f[8];
      load8(xr + i, f);
      const uint32_t bits = allow ? allow[i / 32] >> (i % 32) : 0xffffffffu;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[j] = process(f[j], count[i + j], bias[i + j], rep, pres, freq);
        if (!((bits >> j) & 1u)) f[j] = __int_as_float(0xff800000);
      }
      store8(yr + i, f);
    }
    for (int i = nv + threadIdx.x; i < n; i += THREADS) {
      float f = process((float)xr[i], count[i], bias[i], rep, pres, freq);
      if (allow && !((allow[i / 32] >> (i % 32)) & 1u)) f = __int_as_float(0xff800000);
      yr[i] = (TY)f;
    }
    if (drafted) {
      __syncthreads();
      if (threadIdx.x == 0)
        for (int u = t; u >= 0; u = par[u])
          if (tok[u] >= v0 && tok[u] - v0 < n) count[tok[u] - v0] -= 2u;
    }
  }
}

template <typename TX, typename TY>
cudaError_t launch_logits(const LogitsArgs& a, int batch, bool vec, cudaStream_t s) {
  const size_t smem = (size_t)a.tile * 8;
  const dim3 grid((unsigned)((a.vocab + a.tile - 1) / a.tile), (unsigned)batch);
  auto k = vec ? logits_process_kernel<TX, TY, true> : logits_process_kernel<TX, TY, false>;
  k<<<grid, THREADS, smem, s>>>(a);
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
  if (p->batch > KDV_MAX_BATCH || p->max_T > KDV_MAX_TREE) return KDV_ERR_UNSUPPORTED;
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
  a.tile = 2048;
  const bool vec = rows_aligned(p->logits, p->logits_ld, xe) && rows_aligned(p->out, p->out_ld, ye);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (xe == 2 && ye == 2) e = launch_logits<__nv_bfloat16, __nv_bfloat16>(a, p->batch, vec, s);
  else if (xe == 2) e = launch_logits<__nv_bfloat16, float>(a, p->batch, vec, s);
  else if (ye == 2) e = launch_logits<float, __nv_bfloat16>(a, p->batch, vec, s);
  else e = launch_logits<float, float>(a, p->batch, vec, s);
  return e == cudaSuccess ? KDV_OK : KDV_ERR_CUDA;
}
