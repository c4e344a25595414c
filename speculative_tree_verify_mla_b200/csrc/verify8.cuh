// verify8.cuh -- shared declarations of the 8-bit-cache attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "kdv_internal.cuh"

namespace kdv {

// Everything the kernels read or write besides the plan. The plan is a
// VerifyPlan: out_mode OUT_DIRECT (o / lse) or OUT_WORKSPACE (the part_*
// arrays, row out_row_index; part_f16 is 1 for the tensor-core kernel).
struct Verify8Args {
  const void* q;
  int64_t q_row_stride;
  const uint8_t* c8;
  const __nv_bfloat16* kr;
  const float* kv_scale;
  int32_t block_log2;
  int64_t num_slots;
  const int32_t* page_table;
  const int32_t* kv_off;
  const int32_t* tree_off;
  const int32_t* prefix_len;
  const uint64_t* mask;      // null: chain
  int32_t D_c, D_r;
  float scale;
  // scale log2(e) = scale_part 2^scale_exponent for the tensor-core kernel, 2^-11 <= scale_part < 2^-9: a staged query row
  // times a key is below 2^26, so with the key's scale, below 2^111, nothing overflows before the row's own power of two
  float scale_part;
  int32_t scale_exponent;
  int32_t q_f32, out_f32;
  void* o;
  float* lse;
  void* part_o;              // [parts][D_c]: fp32 o_k (SIMT), fp16 o_k / unit_k (tensor cores)
  float2* part_s;            // [parts]: (lse_k, unit_k)
  int32_t* d_err;
  uint64_t wait_limit_ns;
};

constexpr int V8_ROWS = 64;      // query rows of a tensor-core work item
constexpr int V8_KEYS = 96;      // keys of its tiles

// mask word of node t
__device__ inline uint64_t node_mask(const Verify8Args& a, const VerifyPlan& p, int b, int t) {
  return a.mask != nullptr ? a.mask[p.tree_base[b] + t] : (2ull << t) - 1ull;
}

// Checks the device-side lengths of request b once (thread 0 of an item
// calls it) and says whether its key range can be read.
__device__ inline bool request_ok(const Verify8Args& a, const VerifyPlan& p, int b, bool report) {
  bool ok = (int64_t)a.kv_off[b + 1] - a.kv_off[b] >= (int64_t)p.L[b] + p.T[b] && a.kv_off[b] >= 0;
  if (report && (!ok || (a.prefix_len != nullptr && a.prefix_len[b] != p.L[b]) || a.tree_off[b] != p.tree_base[b]))
    record_error(a.d_err, KDV_DERR_BAD_LENGTH);
  return ok;
}

// Raises a kernel's dynamic shared memory limit to the most that its launches take, once for each kernel and device.
// (The limit is the kernel's, whoever launches it: one that a call lowers is missing in another thread's launch.)
template <auto Kernel> cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done[4];                    // devices below 256
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < 256;
  if (known && (done[dev / 64].load(std::memory_order_acquire) >> (dev % 64)) & 1u) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && known) done[dev / 64].fetch_or(1ull << (dev % 64), std::memory_order_release);
  return e;
}

cudaError_t launch_verify8_simt(const Verify8Args& a, const VerifyPlan& p, cudaStream_t stream);
cudaError_t launch_verify8_tc(const Verify8Args& a, const VerifyPlan& p, cudaStream_t stream);
cudaError_t launch_combine8(const Verify8Args& a, const VerifyPlan& p, cudaStream_t stream);

}  // namespace kdv
