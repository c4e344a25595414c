// verify8_api.cu -- kdv_verify_attn8: argument checks, split planning, launches.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "verify8.cuh"

using namespace kdv;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      n <= 0) {
    cudaGetLastError();
    return 148;
  }
  return n;
}

// types and dims of the tensor-core kernel (its row maxima are taken with a
// positive scale); pointer alignment is checked separately
bool tc_shape(const kdv_verify8_params* p) {
  return p->dtype == KDV_BF16 && p->d_latent == 512 && p->d_rope == 64 && p->scale > 0.f;
}
bool tc_pointers(const kdv_verify8_params* p) {
  const int64_t stride = p->q_row_stride == 0 ? (int64_t)p->d_latent + p->d_rope : p->q_row_stride;
  return aligned16(p->q) && aligned16(p->c8) && aligned16(p->kr) && aligned16(p->o) && stride % 8 == 0;
}

int resolve(const kdv_verify8_params* p) {
  if (p->impl != KDV_IMPL_AUTO) return p->impl;
  return tc_shape(p) && tc_pointers(p) ? KDV_IMPL_TC : KDV_IMPL_SIMT;
}

kdv_status check(const kdv_verify8_params* p) {
  if (p == nullptr) return KDV_ERR_INVALID_ARG;
  if (p->batch < 1 || p->num_heads < 1 || p->d_latent < 1 || p->d_rope < 0) return KDV_ERR_INVALID_ARG;
  if (p->batch > KDV_MAX_BATCH || p->d_latent > 512 || p->d_rope > 64) return KDV_ERR_UNSUPPORTED;
  if ((p->dtype != KDV_BF16 && p->dtype != KDV_F32) || (p->out_dtype != KDV_BF16 && p->out_dtype != KDV_F32))
    return KDV_ERR_INVALID_ARG;
  if (p->impl < KDV_IMPL_AUTO || p->impl > KDV_IMPL_TC_STAGED) return KDV_ERR_INVALID_ARG;
  if (p->impl == KDV_IMPL_TC_1SM || p->impl == KDV_IMPL_TC_STAGED) return KDV_ERR_UNSUPPORTED;
  if (!std::isfinite(p->scale) || p->num_splits < 0) return KDV_ERR_INVALID_ARG;
  if (p->scale_block < 1 || p->scale_block > 4096 || (p->scale_block & (p->scale_block - 1)))
    return KDV_ERR_INVALID_ARG;
  if (p->h_prefix_len == nullptr || p->h_tree_T == nullptr) return KDV_ERR_INVALID_ARG;
  for (int b = 0; b < p->batch; ++b) {
    if (p->h_prefix_len[b] < 0 || p->h_tree_T[b] < 1) return KDV_ERR_INVALID_ARG;
    if (p->h_tree_T[b] > KDV_MAX_TREE || p->h_prefix_len[b] > INT_MAX / 2) return KDV_ERR_UNSUPPORTED;
  }
  if (p->impl == KDV_IMPL_TC && !tc_shape(p)) return KDV_ERR_UNSUPPORTED;
  const int64_t D_q = (int64_t)p->d_latent + p->d_rope;
  if (p->q_row_stride != 0 && p->q_row_stride < D_q) return KDV_ERR_INVALID_ARG;
  return KDV_OK;
}

kdv_status check_pointers(const kdv_verify8_params* p, int impl) {
  if (!p->q || !p->c8 || (p->d_rope > 0 && !p->kr) || !p->kv_scale || !p->kv_off || !p->tree_off || !p->o)
    return KDV_ERR_INVALID_ARG;
  if (p->num_slots < 0) return KDV_ERR_INVALID_ARG;
  const uintptr_t qe = p->dtype == KDV_BF16 ? 2 : 4, oe = p->out_dtype == KDV_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(p->q) % qe || reinterpret_cast<uintptr_t>(p->o) % oe ||
      reinterpret_cast<uintptr_t>(p->kr) % 2 || reinterpret_cast<uintptr_t>(p->kv_scale) % 4 ||
      reinterpret_cast<uintptr_t>(p->lse) % 4 || reinterpret_cast<uintptr_t>(p->mask) % 8)
    return KDV_ERR_INVALID_ARG;
  if (impl == KDV_IMPL_TC && !tc_pointers(p)) return KDV_ERR_INVALID_ARG;
  return KDV_OK;
}

int64_t parts_of(const VerifyPlan& v) {
  const int b = v.B - 1;
  return (int64_t)v.part_base[b] + (int64_t)v.S[b] * v.T[b] * v.H;
}
size_t part_o_bytes(const VerifyPlan& v, int d) { return align256((size_t)parts_of(v) * d * (v.part_f16 ? 2 : 4)); }

// Work items and splits. Splits cover whole key tiles. Automatic: the
// chunk of X keys that minimises a cost in keys of one item: one wave of
// items costs its longest, X + C; two or three waves as much each (few items even
// nothing out); more their mean each and the last one its longest. C is an item's fixed cost (queries, pipeline fill, epilogue, its part of the merge)
// in keys of steady state. Tensor cores: 8 requests x 13 nodes x 64 heads over 5.5k keys take
// 136 us unsplit (104 items), 156, 165, 148 us in 2, 3, 4 splits, which fits 48 keys a us and C = 700.
kdv_status make_plan(const kdv_verify8_params* p, int impl, VerifyPlan* v, size_t* bytes) {
  std::memset(v, 0, sizeof(*v));
  const bool tc = impl == KDV_IMPL_TC;
  const int B = p->batch, H = p->num_heads, per = tc ? V8_ROWS : SIMT_ROWS;
  v->B = B;
  v->H = H;
  v->rows_per_tile = per;
  v->part_f16 = tc ? 1 : 0;
  int64_t nodes = 0, max_n = 1;
  double work = 0.0;
  for (int b = 0; b < B; ++b) {
    v->L[b] = p->h_prefix_len[b];
    v->T[b] = p->h_tree_T[b];
    v->tree_base[b] = (int32_t)nodes;
    nodes += v->T[b];
    const int64_t rows = (int64_t)v->T[b] * H, n = (int64_t)v->L[b] + v->T[b];
    if (rows > INT_MAX / 4) return KDV_ERR_UNSUPPORTED;
    v->tiles[b] = (int32_t)((rows + per - 1) / per);
    max_n = std::max(max_n, n);
    work += (double)v->tiles[b] * n;
  }
  if (nodes * H > INT_MAX / 4) return KDV_ERR_UNSUPPORTED;
  v->total_rows = (int32_t)(nodes * H);
  const double slots = tc ? sm_count() : 4.0 * sm_count();
  const double C = tc ? 700.0 : 128.0;
  auto items_for = [&](int64_t X) {
    double n = 0.0;
    for (int b = 0; b < B; ++b) n += (double)v->tiles[b] * (double)((uint32_t)(v->L[b] + v->T[b] + X - 1) / (uint32_t)X);
    return n;
  };
  auto cost = [&](int64_t X) {
    const double n = items_for(X);
    const double waves = std::ceil(n / slots);
    return waves <= 3.0 ? waves * (X + C) : (waves - 1.0) * (work / n + C) + X + C;
  };
  const int64_t align = tc ? V8_KEYS : SPLIT_ALIGN, x_hi = (max_n + align - 1) / align * align;
  int64_t X = x_hi;
  double best = cost(x_hi);
  for (double xf = (double)align; xf < (double)x_hi; xf = std::max(xf * 1.05, xf + align)) {
    const int64_t x = (int64_t)xf / align * align;
    if (cost(x) < best) {
      best = cost(x);
      X = x;
    }
  }
  int64_t items = 0, parts = 0;
  bool all_one = true;
  for (int b = 0; b < B; ++b) {
    const int64_t n = (int64_t)v->L[b] + v->T[b];
    int64_t S = p->num_splits >= 1 ? p->num_splits : (n + X - 1) / X;
    if (S > 4096) return KDV_ERR_UNSUPPORTED;
    v->chunk[b] = (int32_t)(align * ((n + align * S - 1) / (align * S)));
    if (p->num_splits == 0) S = (n + v->chunk[b] - 1) / v->chunk[b];   // whole tiles may need fewer
    v->S[b] = (int32_t)S;
    v->item_base[b] = (int32_t)items;
    v->part_base[b] = (int32_t)parts;
    items += (int64_t)v->tiles[b] * S;
    parts += S * v->T[b] * H;
    if (S != 1) all_one = false;
    if (items > INT_MAX / 4 || parts > INT_MAX / 4) return KDV_ERR_UNSUPPORTED;
  }
  v->item_base[B] = (int32_t)items;
  v->n_items = (int32_t)items;
  v->out_mode = all_one ? OUT_DIRECT : OUT_WORKSPACE;
  *bytes = all_one ? 0 : part_o_bytes(*v, p->d_latent) + (size_t)parts * sizeof(float2);
  return KDV_OK;
}

}  // namespace

extern "C" {

kdv_status kdv_verify_attn8_workspace(const kdv_verify8_params* p, size_t* bytes) {
  if (bytes == nullptr) return KDV_ERR_INVALID_ARG;
  kdv_status st = check(p);
  if (st != KDV_OK) return st;
  VerifyPlan v;
  st = make_plan(p, resolve(p), &v, bytes);
  // AUTO also goes by the pointers' alignment, which may not be final yet:
  // the answer covers both kernels
  if (st == KDV_OK && p->impl == KDV_IMPL_AUTO && tc_shape(p)) {
    size_t simt = 0, tc = 0;
    st = make_plan(p, KDV_IMPL_SIMT, &v, &simt);
    if (st == KDV_OK) st = make_plan(p, KDV_IMPL_TC, &v, &tc);
    *bytes = std::max(simt, tc);
  }
  return st;
}

kdv_status kdv_verify_attn8_plan(const kdv_verify8_params* p, int32_t* splits, int32_t* grid_items) {
  kdv_status st = check(p);
  if (st != KDV_OK) return st;
  VerifyPlan v;
  size_t bytes = 0;
  st = make_plan(p, resolve(p), &v, &bytes);
  if (st != KDV_OK) return st;
  if (splits)
    for (int b = 0; b < v.B; ++b) splits[b] = v.S[b];
  if (grid_items) *grid_items = v.n_items;
  return KDV_OK;
}

kdv_status kdv_verify_attn8(const kdv_verify8_params* p, void* stream) {
  kdv_status st = check(p);
  if (st != KDV_OK) return st;
  const int impl = resolve(p);
  st = check_pointers(p, impl);
  if (st != KDV_OK) return st;
  VerifyPlan v;
  size_t need = 0;
  st = make_plan(p, impl, &v, &need);
  if (st != KDV_OK) return st;
  if (need > 0 && (p->workspace == nullptr || p->workspace_bytes < need || !aligned16(p->workspace)))
    return KDV_ERR_WORKSPACE;
  Verify8Args a = {};
  a.q = p->q;
  a.q_row_stride = p->q_row_stride == 0 ? (int64_t)p->d_latent + p->d_rope : p->q_row_stride;
  a.c8 = p->c8;
  a.kr = static_cast<const __nv_bfloat16*>(p->kr);
  a.kv_scale = p->kv_scale;
  while ((1 << a.block_log2) < p->scale_block) ++a.block_log2;
  a.num_slots = p->num_slots;
  a.page_table = p->page_table;
  a.kv_off = p->kv_off;
  a.tree_off = p->tree_off;
  a.prefix_len = p->prefix_len;
  a.mask = p->mask;
  a.D_c = p->d_latent;
  a.D_r = p->d_rope;
  a.scale = p->scale;
  a.scale_part = std::ldexp(std::frexp(p->scale, &a.scale_exponent) * 2.f * 1.4426950408889634f, -11);   // (0 stays 0)
  a.scale_exponent += 10;
  a.q_f32 = p->dtype == KDV_F32;
  a.out_f32 = p->out_dtype == KDV_F32;
  a.o = p->o;
  a.lse = p->lse;
  a.d_err = p->d_err;
  a.wait_limit_ns = p->wait_limit_ns;
  if (v.out_mode == OUT_WORKSPACE) {
    a.part_o = p->workspace;
    a.part_s = reinterpret_cast<float2*>(static_cast<char*>(p->workspace) + part_o_bytes(v, p->d_latent));
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = impl == KDV_IMPL_TC ? launch_verify8_tc(a, v, s) : launch_verify8_simt(a, v, s);
  if (e == cudaSuccess && v.out_mode == OUT_WORKSPACE) e = launch_combine8(a, v, s);
  return e == cudaSuccess ? KDV_OK : KDV_ERR_CUDA;
}

}  // extern "C"
