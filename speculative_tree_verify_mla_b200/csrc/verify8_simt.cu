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
constexpr int smem_bytes(int D_q) { return (KT * (D_q + 1) + WARPS * D_q) * (int)sizeof(float); }

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
// exp(lse_k - LSE) unit_k o_k. Reads S * rows * D_c partials that the attention
// kernel has just left in L2, so it is a matter of loads in flight: one CTA a
// row, a thread holds four neighbouring dims and reads eight parts at a time;
// the parts' weights are formed once, 128 of them at a time, in shared memory.
constexpr int MERGE_THREADS = 128;
__global__ void __launch_bounds__(MERGE_THREADS) combine8_kernel(const __grid_constant__ Verify8Args a,
                                                                 const __grid_constant__ VerifyPlan p) {
  __shared__ float weight[MERGE_THREADS];
  __shared__ float red[2][MERGE_THREADS / 32];
  const int tid = threadIdx.x, row = blockIdx.x, D = a.D_c;
  int b = 0;
  while (b + 1 < p.B && p.tree_base[b + 1] * p.H <= row) ++b;
  const int rows_b = p.T[b] * p.H, r = row - p.tree_base[b] * p.H, S = p.S[b];
  const int64_t base = p.part_base[b] + r;
  asm volatile("griddepcontrol.launch_dependents;");       // the next launch may prepare itself
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the attention kernel's parts
  float m = -INFINITY;
  bool bad = false;                       // a NaN part makes the row NaN
  for (int k = tid; k < S; k += MERGE_THREADS) {
    const float l = a.part_s[base + (int64_t)k * rows_b].x;
    bad |= isnan(l);
    m = fmaxf(m, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (__any_sync(0xffffffffu, bad)) m = INFINITY;          // lse is never +inf otherwise
  if (tid % 32 == 0) red[0][tid / 32] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  if (m == INFINITY) m = __int_as_float(0x7fc00000);
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
  const float* part = static_cast<const float*>(a.part_o);
  const int d0 = 4 * tid;                                  // D_c <= 512
  const bool whole = D % 4 == 0;
  for (int k0 = 0; k0 < S; k0 += MERGE_THREADS) {
    const int n = min(MERGE_THREADS, S - k0);
    if (k0 > 0) __syncthreads();
    if (tid < n) {
      const float2 su = a.part_s[base + (int64_t)(k0 + tid) * rows_b];
      const float e = su.x == -INFINITY ? 0.f : expf(su.x - m);
      sum += e;
      weight[tid] = e * su.y;
    }
    __syncthreads();
    if (d0 >= D) continue;
    const float* src = part + (base + (int64_t)k0 * rows_b) * D + d0;
    const int64_t step = (int64_t)rows_b * D;
    for (int k = 0; k < n; k += 8) {
      float v[8][4];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = 0.f;
        if (k + j >= n) continue;
        if (whole) {
          const float4 w = *reinterpret_cast<const float4*>(src + j * step);
          v[j][0] = w.x; v[j][1] = w.y; v[j][2] = w.z; v[j][3] = w.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) if (d0 + i < D) v[j][i] = (float)src[j * step + i];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float w = k + j < n ? weight[k + j] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(w, v[j][i], acc[i]);
      }
      src += 8 * step;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (tid % 32 == 0) red[1][tid / 32] = sum;
  __syncthreads();
  sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  const bool none = m == -INFINITY;
  const float inv = none ? 0.f : 1.f / sum;
  if (tid == 0 && a.lse != nullptr) a.lse[row] = none ? -INFINITY : m + logf(sum);
  if (d0 >= D) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = none ? 0.f : acc[i] * inv;
  const int64_t at = (int64_t)row * D + d0;
  if (whole && reinterpret_cast<uintptr_t>(a.o) % 16 == 0) {
    if (a.out_f32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.o) + at) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    } else {
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc[0], acc[1]), y = __floats2bfloat162_rn(acc[2], acc[3]);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (d0 + i >= D) break;
      if (a.out_f32) static_cast<float*>(a.o)[at + i] = acc[i];
      else static_cast<__nv_bfloat16*>(a.o)[at + i] = __float2bfloat16_rn(acc[i]);
    }
  }
}

// The same for the tensor-core kernel's parts (fp16, 512 dims): one warp half a row, no barrier;
// the first eight parts are on their way before their weights are known. 5.5k layer (832 rows, 10
// parts): 0.3 us more with a warp a row and four parts in flight, 0.7 with a CTA a row as above (28.4 us in all then, 26.2 now).
constexpr int ROW_WARPS = 4;
__global__ void __launch_bounds__(ROW_WARPS * 32) combine8_rows_kernel(const __grid_constant__ Verify8Args a,
                                                                       const __grid_constant__ VerifyPlan p) {
  constexpr int AHEAD = 8;
  const int lane = threadIdx.x & 31, warp = blockIdx.x * ROW_WARPS + (threadIdx.x >> 5);
  const int row = warp >> 1, piece = (warp & 1) * 32 + lane;               // eight of the row's dims
  asm volatile("griddepcontrol.launch_dependents;");       // the next launch may prepare itself
  if (row >= p.total_rows) return;
  int b = 0;
  while (b + 1 < p.B && p.tree_base[b + 1] * p.H <= row) ++b;
  const int rows_b = p.T[b] * p.H, S = p.S[b];
  const int64_t base = (int64_t)p.part_base[b] + row - p.tree_base[b] * p.H;
  const uint4* part = static_cast<const uint4*>(a.part_o) + base * 64 + piece;
  const int64_t step = (int64_t)rows_b * 64;
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the attention kernel's parts
  uint4 x[AHEAD];
  auto load = [&](int k0) {
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (k0 + j < S) x[j] = part[(k0 + j) * step];
  };
  float2 su = lane < S ? a.part_s[base + (int64_t)lane * rows_b] : make_float2(-INFINITY, 0.f);   // of part `lane`
  load(0);
  float m = su.x;
  bool bad = isnan(su.x);                                  // a NaN part makes the row NaN
  for (int k = lane + 32; k < S; k += 32) {
    const float v = a.part_s[base + (int64_t)k * rows_b].x;
    bad |= isnan(v);
    m = fmaxf(m, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (__any_sync(0xffffffffu, bad)) m = __int_as_float(0x7fc00000);
  float acc[8], sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int k0 = 0; k0 < S; k0 += 32) {                     // 32 parts' weights at a time, one a lane
    if (k0 > 0) su = k0 + lane < S ? a.part_s[base + (int64_t)(k0 + lane) * rows_b] : make_float2(-INFINITY, 0.f);
    const float e = su.x == -INFINITY ? 0.f : expf(su.x - m);
    const float weight = e * su.y;
    sum += e;
    const int n = min(32, S - k0);
    for (int k = 0; k < n; k += AHEAD) {
      if (k0 + k > 0) load(k0 + k);
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const float w = __shfl_sync(0xffffffffu, weight, (k + j) & 31);
        if (k + j >= n) break;
        const uint32_t u[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
          acc[2 * i] = fmaf(w, f.x, acc[2 * i]);
          acc[2 * i + 1] = fmaf(w, f.y, acc[2 * i + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const bool none = m == -INFINITY;
  const float inv = none ? 0.f : 1.f / sum;
  if (piece == 0 && a.lse != nullptr) a.lse[row] = none ? -INFINITY : m + logf(sum);
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = none ? 0.f : acc[i] * inv;
  const int64_t at = (int64_t)row * 64 + piece;            // o is 16-byte aligned here
  if (a.out_f32) {
    static_cast<float4*>(a.o)[2 * at] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    static_cast<float4*>(a.o)[2 * at + 1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 y = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    static_cast<uint4*>(a.o)[at] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

}  // namespace

cudaError_t launch_verify8_simt(const Verify8Args& a, const VerifyPlan& p, cudaStream_t stream) {
  constexpr int MOST = smem_bytes(512 + 64);
  const int smem = smem_bytes(a.D_c + a.D_r);
  cudaError_t e = a.q_f32 ? allow_smem<verify8_simt_kernel<float>>(MOST) : allow_smem<verify8_simt_kernel<__nv_bfloat16>>(MOST);
  if (e != cudaSuccess) return e;
  if (a.q_f32) verify8_simt_kernel<float><<<p.n_items, WARPS * 32, smem, stream>>>(a, p);
  else verify8_simt_kernel<__nv_bfloat16><<<p.n_items, WARPS * 32, smem, stream>>>(a, p);
  return cudaGetLastError();
}

cudaError_t launch_combine8(const Verify8Args& a, const VerifyPlan& p, cudaStream_t stream) {
  // a programmatic dependent of the attention kernel: its launch overlaps that
  // kernel's end, its reads wait for it
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.part_f16 ? (2 * p.total_rows + ROW_WARPS - 1) / ROW_WARPS : p.total_rows));
  cfg.blockDim = dim3(p.part_f16 ? ROW_WARPS * 32 : MERGE_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, p.part_f16 ? combine8_rows_kernel : combine8_kernel, a, p);
}

}  // namespace kdv
