// verify8_simt.cu -- attention over the 8-bit latent cache on CUDA cores, for
// the types and dims that the tensor-core kernel does not take.
//
// s_j = scale * kv_scale_j (q_lat . c8_j + q_rope . kr_j), softmax over the
// keys that the row's node sees, o = sum_j p_j kv_scale_j c8_j. One warp owns
// a query row; a CTA of eight warps stages 32 keys at a time in shared memory
// as fp32 (scaled), lane k scores key k, then every lane accumulates its
// D_c / 32 output dims. Bound by the shared-memory reads of the staged keys.
#include <cuda_fp8.h>

#include "verify8.cuh"

namespace kdv {
namespace {

constexpr int KT = 32;                 // keys per shared-memory tile
constexpr int WARPS = SIMT_ROWS;       // one warp per query row
constexpr int DC_PER_LANE = 16;        // D_c <= 512

__device__ inline float code_value(uint8_t c) {
  __nv_fp8_e4m3 v;
  v.__x = c;
  return (float)v;
}
__device__ inline float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = (v > w || isnan(v)) ? v : w;   // a NaN logit of a visible key stays
  }
  return v;
}
__device__ inline float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename TQ>
__global__ void __launch_bounds__(WARPS * 32) verify8_simt_kernel(const __grid_constant__ Verify8Args a,
                                                                  const __grid_constant__ VerifyPlan p) {
  extern __shared__ float smem[];
  const int D_c = a.D_c, D_q = a.D_c + a.D_r, KS = D_q + 1;
  float* Ks = smem;                            // [KT][KS]
  float* Qs = smem + KT * KS;                  // [WARPS][D_q]
  __shared__ int64_t key_slot[KT];             // -1: not readable
  const int item = blockIdx.x;
  const int b = plan_request(p, item);
  const int local = item - p.item_base[b];
  const int s = local / p.tiles[b];
  const int rt = local - s * p.tiles[b];
  const int L = p.L[b], n_keys = L + p.T[b], rows_b = p.T[b] * p.H;
  const bool ok = request_ok(a, p, b, threadIdx.x == 0 && local == 0);
  const int64_t lo64 = (int64_t)s * p.chunk[b];
  const int k_lo = (int)min(lo64, (int64_t)n_keys);
  const int k_hi = ok ? (int)min(lo64 + p.chunk[b], (int64_t)n_keys) : k_lo;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t kv_base = a.kv_off[b];
  const TQ* q = static_cast<const TQ*>(a.q);

  const int r = rt * WARPS + warp;
  const bool row_ok = r < rows_b;
  const uint64_t mask_t = row_ok ? node_mask(a, p, b, r / p.H) : 0ull;
  const int64_t row_global = (int64_t)p.tree_base[b] * p.H + r;
  for (int d = lane; d < D_q; d += 32)
    Qs[warp * D_q + d] = row_ok ? (float)q[row_global * a.q_row_stride + d] : 0.f;

  float o[DC_PER_LANE];
#pragma unroll
  for (int i = 0; i < DC_PER_LANE; ++i) o[i] = 0.f;
  float m = -INFINITY, l = 0.f;

  for (int j0 = k_lo; j0 < k_hi; j0 += KT) {
    __syncthreads();
    if (threadIdx.x < KT) {
      const int j = j0 + threadIdx.x;
      int64_t slot = -1;
      if (j < k_hi) {
        slot = a.page_table ? (int64_t)a.page_table[kv_base + j] : kv_base + j;
        if (slot < 0 || slot >= a.num_slots) {
          record_error(a.d_err, KDV_DERR_BAD_SLOT);
          slot = -1;
        }
      }
      key_slot[threadIdx.x] = slot;
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < KT * D_q; idx += WARPS * 32) {
      const int k = idx / D_q, d = idx - k * D_q;
      const int64_t slot = key_slot[k];
      float v = 0.f;
      if (slot >= 0) {
        v = d < D_c ? code_value(a.c8[slot * D_c + d]) : __bfloat162float(a.kr[slot * a.D_r + d - D_c]);
        v *= a.kv_scale[slot >> a.block_log2];
      }
      Ks[k * KS + d] = v;
    }
    __syncthreads();
    if (!row_ok) continue;

    const int j = j0 + lane;
    const bool vis = j < k_hi && key_slot[lane] >= 0 && (j < L || ((mask_t >> (j - L)) & 1ull));
    float sc = -INFINITY;
    if (vis) {
      // eight interleaved sums: an eighth of one chain's roundings
      float acc[8] = {};
      const float* qr = Qs + warp * D_q;
      const float* kk = Ks + lane * KS;
      int d = 0;
      for (; d + 8 <= D_q; d += 8)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(qr[d + i], kk[d + i], acc[i]);
      for (; d < D_q; ++d) acc[0] = fmaf(qr[d], kk[d], acc[0]);
      sc = a.scale * (((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7])));
    }
    const float tile_max = warp_max(sc);
    const float m_new = (m > tile_max || isnan(m)) ? m : tile_max;
    if (m_new == -INFINITY) continue;          // nothing visible yet (warp-uniform)
    const float corr = m == m_new ? 1.f : expf(m - m_new);
    const float pk = vis ? expf(sc - m_new) : 0.f;
    l = l * corr + warp_sum(pk);
#pragma unroll
    for (int i = 0; i < DC_PER_LANE; ++i) o[i] *= corr;
    for (int k = 0; k < KT; ++k) {
      const float pv = __shfl_sync(0xffffffffu, pk, k);
      if (pv == 0.f) continue;                  // warp-uniform
      const float* vr = Ks + k * KS;
#pragma unroll
      for (int i = 0; i < DC_PER_LANE; ++i) {
        const int d = lane + 32 * i;
        if (d < D_c) o[i] = fmaf(pv, vr[d], o[i]);
      }
    }
    m = m_new;
  }

  if (!row_ok) return;
  const int64_t orow = out_row_index(p, b, s, r);
  const bool none = l == 0.f && m == -INFINITY;
  const float inv = none ? 0.f : 1.f / l;
  const float lse = none ? -INFINITY : m + logf(l);
#pragma unroll
  for (int i = 0; i < DC_PER_LANE; ++i) {
    const int d = lane + 32 * i;
    if (d >= D_c) continue;
    const float v = o[i] * inv;
    if (p.out_mode == OUT_WORKSPACE) static_cast<float*>(a.part_o)[orow * D_c + d] = v;
    else if (a.out_f32) static_cast<float*>(a.o)[orow * D_c + d] = v;
    else static_cast<__nv_bfloat16*>(a.o)[orow * D_c + d] = __float2bfloat16_rn(v);
  }
  if (lane == 0) {
    if (p.out_mode == OUT_WORKSPACE) a.part_s[orow] = make_float2(lse, 1.f);
    else if (a.lse != nullptr) a.lse[orow] = lse;
  }
}

// Merge of a request's split partials: LSE = ln sum_k exp(lse_k), o = sum_k
// exp(lse_k - LSE) unit_k o_k. One warp a row, each lane two neighbouring
// dims of every 64, so a warp reads 128 (fp16) or 256 bytes at a time. Reads
// S * rows * D_c partials that the attention kernel has just left in L2.
template <typename TP>
__global__ void __launch_bounds__(256) combine8_kernel(const __grid_constant__ Verify8Args a,
                                                       const __grid_constant__ VerifyPlan p) {
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= p.total_rows) return;
  int b = 0;
  while (b + 1 < p.B && p.tree_base[b + 1] * p.H <= row) ++b;
  const int rows_b = p.T[b] * p.H, r = row - p.tree_base[b] * p.H, S = p.S[b];
  const int64_t base = p.part_base[b] + r;
  float m = -INFINITY;
  bool bad = false;                       // a NaN part makes the row NaN
  for (int k = lane; k < S; k += 32) {
    const float l = a.part_s[base + (int64_t)k * rows_b].x;
    bad |= isnan(l);
    m = fmaxf(m, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (__any_sync(0xffffffffu, bad)) m = __int_as_float(0x7fc00000);
  float sum = 0.f;
  for (int k = lane; k < S; k += 32) {
    const float l = a.part_s[base + (int64_t)k * rows_b].x;
    sum += l == -INFINITY ? 0.f : expf(l - m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const bool none = m == -INFINITY;
  const float inv = none ? 0.f : 1.f / sum;
  if (lane == 0 && a.lse != nullptr) a.lse[row] = none ? -INFINITY : m + logf(sum);
  const TP* part = static_cast<const TP*>(a.part_o);
  for (int d0 = 0; d0 < a.D_c; d0 += 512) {
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    for (int k = 0; k < S; ++k) {
      const float2 su = a.part_s[base + (int64_t)k * rows_b];
      if (su.x == -INFINITY) continue;
      const float w = expf(su.x - m) * inv * su.y;
      const TP* src = part + (base + (int64_t)k * rows_b) * a.D_c;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d = d0 + 64 * i + 2 * lane;
        if (d < a.D_c) acc[2 * i] = fmaf(w, (float)src[d], acc[2 * i]);
        if (d + 1 < a.D_c) acc[2 * i + 1] = fmaf(w, (float)src[d + 1], acc[2 * i + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int d = d0 + 64 * (i / 2) + 2 * lane + (i & 1);
      if (d >= a.D_c) continue;
      if (a.out_f32) static_cast<float*>(a.o)[(int64_t)row * a.D_c + d] = acc[i];
      else static_cast<__nv_bfloat16*>(a.o)[(int64_t)row * a.D_c + d] = __float2bfloat16_rn(acc[i]);
    }
  }
}

}  // namespace

cudaError_t launch_verify8_simt(const Verify8Args& a, const VerifyPlan& p, cudaStream_t stream) {
  const int D_q = a.D_c + a.D_r;
  const size_t smem = (size_t)(KT * (D_q + 1) + WARPS * D_q) * sizeof(float);
  auto k = a.q_f32 ? verify8_simt_kernel<float> : verify8_simt_kernel<__nv_bfloat16>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  k<<<p.n_items, WARPS * 32, smem, stream>>>(a, p);
  return cudaGetLastError();
}

cudaError_t launch_combine8(const Verify8Args& a, const VerifyPlan& p, cudaStream_t stream) {
  const int grid = (p.total_rows + 7) / 8;
  if (p.part_f16) combine8_kernel<__half><<<grid, 256, 0, stream>>>(a, p);
  else combine8_kernel<float><<<grid, 256, 0, stream>>>(a, p);
  return cudaGetLastError();
}

}  // namespace kdv
