// verify8_tc.cu -- attention over the 8-bit latent cache on tcgen05 tensor cores.
//
//   x[r,j] = scale s_j (q_lat[r] . c8[j] + q_rope[r] . kr[j])      (s_j = kv_scale of key j)
//   o[r]   = sum_j p[r,j] s_j c8[j] / sum_j p[r,j],  p = exp(x - max)
//
// The codes are multiplied as they are stored, so a key costs 512 + 128 bytes
// of memory and of shared memory, and nothing is converted:
//   Q.K^T  q_lat times a power of two per row is split in two e4m3 terms,
//          q = hi + lo / 16. bf16 holds 8 significant bits and a term 4, so the
//          split is exact down to 2^-21 of the row's largest element. The rope
//          part is a bf16 product into the same sums. Products of e4m3 codes and
//          their fp32 sums are exact to fp32's rounding (measured: 3e-8).
//   P.V    p s_j is rounded to fp16 and split in three e5m2 terms, the first
//          two truncated (an e5m2 is an fp16's upper byte, so a term is a
//          mask and the rest an exact subtraction), the last one rounded:
//          2^-9 of p at most, against 2^-8 for a bf16 numerator. e5m2 reaches
//          down to 2^-16 and the largest p is kept within [2^12, 2^15], so
//          keys 2^-28 below the largest still count; with e4m3 terms a long
//          tail of small weights would vanish (2^-18). Two terms would be
//          off by 2.7e-3 (rms) at 0.85 of the time.
//
// Both products are formed transposed, keys resp. latent dims as the rows (M)
// of an MMA and 64 query rows as its columns (N): one token of 64 heads fills
// a tile, where rows of queries would leave half of M = 128 empty, and the fp32
// output (64 columns for each of four 128-dim blocks) takes 256 columns of
// TMEM instead of all 512. The same 16 KB block of 128 keys x 128 dims in the
// 128-byte swizzle is A of Q.K^T (K-major) and A of P.V (M-major).
//
// One CTA per work item: 64 query rows of one request, one key split, tiles
// of 128 keys:
//   warps 9-12  producers: gather 128-byte row pieces through the page table
//               with cp.async into a ring of seven 16 KB blocks (a tile is
//               the rope block and four latent blocks), one warp a block, four
//               in flight. (tile::gather4 issues one 512-byte gather in ~65
//               cycles on this part, 8 B/clk; cp.async beside these MMAs
//               reached 28 B/clk, of the 20 B/clk that the MMAs consume.)
//   warp 8      MMA issue: the next tile's Q.K^T (as far as its blocks are
//               here and the ring holds them) runs while the softmax works on this tile;
//               then P.V; a block is freed by the last MMA that reads it.
//   warps 0-7   two warpgroups: queries in, softmax, output. Lane = key, so a
//               warpgroup owns 32 query rows, a thread one key of them; a row's
//               maximum is only looked for across lanes when some logit passes
//               the reference by 2^3 (a vote), then O is rescaled in TMEM.
//
// What bounds it: shared-memory reads of the MMAs. Per tile 16 (N = 128) + 4
// + 48 (N = 64) MMAs of 64, 64 and 48 cycles at 128 B/clk: 3.6k cycles, the
// same as 82 KB of HBM at this SM's share of 6.46 TB/s.
#include <cuda_fp8.h>

#include "sm100_ptx.cuh"
#include "verify8.cuh"

namespace kdv {
namespace {

using namespace ptx;

constexpr int ROWS = V8_ROWS, KEYS = V8_KEYS, DC = 512, DR = 64;
constexpr int BLOCK = 16384;                 // 128 keys x 128 bytes, or 128 stacked query rows x 128 bytes
constexpr int PARTS = 5;                     // blocks of a tile: rope, latent 0..3
constexpr int RING = 7;
constexpr int TERMS = 3, P_BYTES = KEYS * ROWS;
constexpr int KS_BUFS = 4;
constexpr int SOFTMAX_WARPS = 8, MMA_WARP = 8, PRODUCER_WARPS = 4;
constexpr int THREADS = (SOFTMAX_WARPS + 1 + PRODUCER_WARPS) * 32;
constexpr float P_TOP = 12.f, P_GROW = 15.f; // log2 of the largest p when the reference is set / allowed later
constexpr float NO_MAX = -1e30f;             // the reference of a row that has seen no key
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr uint64_t TIMEOUT_NS = 1000000000ull;

constexpr int OFF_Q = 0;                                   // 4 blocks: rows 0-63 hi, 64-127 lo
constexpr int OFF_QR = OFF_Q + 4 * BLOCK;                  // rows 0-63 q_rope bf16, 64-127 zero
constexpr int OFF_P = OFF_QR + BLOCK;
constexpr int OFF_RING = OFF_P + TERMS * P_BYTES;
constexpr int OFF_KS = OFF_RING + RING * BLOCK;            // float [KS_BUFS][128] key scales
constexpr int OFF_OK = OFF_KS + KS_BUFS * KEYS * 4;        // u32 [KS_BUFS][4] readable keys
constexpr int OFF_MASK = OFF_OK + KS_BUFS * 16;            // u64 [64] node masks by row
constexpr int OFF_CM = OFF_MASK + ROWS * 8;                // float4 [32]: (c, c', -m, -m') of a row pair
constexpr int OFF_RED = OFF_CM + 32 * 16;                  // float [2][4][32]
constexpr int OFF_FAC = OFF_RED + 2 * 4 * 32 * 4;          // float [64] per-row factors
constexpr int OFF_RED2 = OFF_FAC + ROWS * 4;               // float [2][4]
constexpr int OFF_BAR = OFF_RED2 + 32;
constexpr int B_FULL = 0, B_EMPTY = B_FULL + RING, B_KS = B_EMPTY + RING, B_S = B_KS + KS_BUFS, B_P = B_S + 2, B_ROPE = B_P + 1,
              B_Q = B_ROPE + 1, B_FIN = B_Q + 1, NUM_BARS = B_FIN + 1;
constexpr int OFF_TMEM = OFF_BAR + NUM_BARS * 8;
constexpr int OFF_ABORT = OFF_TMEM + 4;
constexpr int SMEM_BYTES = OFF_ABORT + 4 + 1024;
static_assert(OFF_BAR % 8 == 0 && OFF_MASK % 8 == 0 && OFF_CM % 16 == 0, "alignment");
static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory");
constexpr uint32_t TM_S = 256;                             // S buffers behind the 4 x 64 output columns

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// kind::f8f6f4 with fp32 D: formats 0 e4m3, 1 e5m2
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a_fmt, int b_fmt, bool a_mn, bool b_mn) {
  return (1u << 4) | ((uint32_t)a_fmt << 7) | ((uint32_t)b_fmt << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t IDESC_QK = idesc_f8(128, 128, 0, 0, false, false);
constexpr uint32_t IDESC_ROPE = idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t IDESC_PV = idesc_f8(128, 64, 0, 1, true, true);

// 64-byte-swizzled descriptor (P: 64 query rows of a key are one 64-byte row, eight keys a group of 512 bytes)
__device__ __forceinline__ uint64_t sw64_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) | ((uint64_t)4 << 61);
}
__device__ __forceinline__ uint32_t swz128(uint32_t o) { return o ^ ((o >> 3) & 0x70u); }

__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Bounded waits: a wait that runs out reports, raises the CTA's abort flag and
// returns false; from then on every other wait of the CTA returns at once.
struct Waiter {
  volatile int* abort;
  int32_t* d_err;
  uint64_t limit;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return true;
    return slow(bar, parity);
  }
  __device__ __noinline__ bool slow(uint32_t bar, uint32_t parity) const {
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(bar, parity)) {
      if (*abort) return false;
      if (global_ns() - t0 > limit) {
        *abort = 1;
        record_error(d_err, KDV_DERR_TIMEOUT);
        return false;
      }
    }
    return true;
  }
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// largest |x| of a warp / largest x, through the order-preserving integer image of a float
__device__ __forceinline__ float warp_max(float x) {
  int i = __float_as_int(x);
  i ^= (i >> 31) & 0x7fffffff;
  i = __reduce_max_sync(0xffffffffu, i);
  return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

// ------------------------------------------------------------------ queries
// One row by one warp: lane l holds latent elements 16 l .. 16 l + 15 and rope
// elements 2 l, 2 l + 1. Returns the row's logit factor scale log2(e) 2^-k.
__device__ __forceinline__ float stage_query(const Verify8Args& a, const __nv_bfloat16* row, bool valid, int r, uint8_t* sp, int lane) {
  float v[16];
  uint32_t rope = 0;
  if (valid) {
    const uint4 w0 = reinterpret_cast<const uint4*>(row)[2 * lane], w1 = reinterpret_cast<const uint4*>(row)[2 * lane + 1];
    const uint32_t u[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
    rope = reinterpret_cast<const uint32_t*>(row + DC)[lane];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, finite(v[i]) ? fabsf(v[i]) : 0.f);
  top = warp_max(top);
  // the power of two that brings the largest element into [128, 256)
  int e = top > 0.f ? 7 - ilogbf(top) : 0;
  e = max(-120, min(60, e));
  const float up = ldexpf(1.f, e);
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[4], y[4];
    uint32_t h = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = finite(v[4 * i + j]) ? v[4 * i + j] * up : __int_as_float(0x7fc00000);
    h = e4m3x4(x[0], x[1], x[2], x[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __nv_fp8_e4m3 t;
      t.__x = (uint8_t)(h >> (8 * j));
      y[j] = isnan(x[j]) ? 0.f : 16.f * (x[j] - (float)t);   // the low terms stay finite, see the softmax
    }
    hi[i] = h;
    lo[i] = e4m3x4(y[0], y[1], y[2], y[3]);
  }
  const uint32_t blk = (uint32_t)(lane / 8) * BLOCK, col = (uint32_t)(lane % 8) * 16;
  *reinterpret_cast<uint4*>(sp + OFF_Q + blk + swz128(r * 128 + col)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  *reinterpret_cast<uint4*>(sp + OFF_Q + blk + swz128((r + ROWS) * 128 + col)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  const float ra = __uint_as_float(rope << 16) * up, rb = __uint_as_float(rope & 0xffff0000u) * up;
  *reinterpret_cast<uint32_t*>(sp + OFF_QR + swz128(r * 128 + lane * 4)) = pack_bf16x2(ra, rb);
  *reinterpret_cast<uint32_t*>(sp + OFF_QR + swz128((r + ROWS) * 128 + lane * 4)) = 0u;
  return fminf(fmaxf(a.scale * LOG2E * ldexpf(1.f, -e), 1.17549435e-38f), 3.402823466e38f);
}

// Two fp16 numerators -> their three e5m2 terms: the upper bytes of the first
// two words' halves, and both bytes of the third packed in 16 bits.
__device__ __forceinline__ void split_p(uint32_t h, uint32_t& t0, uint32_t& t1, uint32_t& t2) {
  t0 = h & 0xff00ff00u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&t0));
  const uint32_t ru = *reinterpret_cast<const uint32_t*>(&r);
  t1 = ru & 0xff00ff00u;
  const __half2 s = __hsub2(r, *reinterpret_cast<const __half2*>(&t1));
  uint16_t c;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(*reinterpret_cast<const uint32_t*>(&s)));
  t2 = c;
}

__global__ void __launch_bounds__(THREADS, 1) verify8_tc_kernel(const __grid_constant__ Verify8Args a,
                                                                const __grid_constant__ VerifyPlan p) {
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* sp = raw + (base - smem_u32(raw));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](int i) { return base + OFF_BAR + 8 * i; };
  volatile int* abort = reinterpret_cast<volatile int*>(sp + OFF_ABORT);
  const Waiter wait{abort, a.d_err, a.wait_limit_ns ? a.wait_limit_ns : TIMEOUT_NS};

  const int item = blockIdx.x;
  const int b = plan_request(p, item);
  const int local = item - p.item_base[b];
  const int split = local / p.tiles[b], rt = local - split * p.tiles[b];
  const int L = p.L[b], n_keys = L + p.T[b], rows_b = p.T[b] * p.H;
  const bool ok = request_ok(a, p, b, tid == 0 && local == 0);
  const int64_t lo64 = (int64_t)split * p.chunk[b];
  const int k_lo = (int)min(lo64, (int64_t)n_keys);
  const int k_hi = ok ? (int)min(lo64 + p.chunk[b], (int64_t)n_keys) : k_lo;
  const int NT = (k_hi - k_lo + KEYS - 1) / KEYS;
  const int r0 = rt * ROWS;

  if (tid == 0) {
    for (int i = 0; i < RING; ++i) {
      mbar_init(bar(B_FULL + i), 1);
      mbar_init(bar(B_EMPTY + i), 1);
    }
    for (int i = 0; i < KS_BUFS; ++i) mbar_init(bar(B_KS + i), 1);
    mbar_init(bar(B_S), 1);
    mbar_init(bar(B_S + 1), 1);
    mbar_init(bar(B_P), SOFTMAX_WARPS);
    mbar_init(bar(B_ROPE), 1);
    mbar_init(bar(B_Q), SOFTMAX_WARPS);
    mbar_init(bar(B_FIN), 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(base + OFF_TMEM, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sp + OFF_TMEM);

  if (warp > MMA_WARP) {
    // ---------------------------------------------------------- producers
    const int64_t kv_base = a.kv_off[b];
    auto load_slots = [&](int tile, int (&slot)[4]) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int j = k_lo + tile * KEYS + g * 32 + lane;
        slot[g] = -1;
        if (tile < NT && j < k_hi) {
          const int64_t s = a.page_table ? (int64_t)a.page_table[kv_base + j] : kv_base + j;
          if (s >= 0 && s < a.num_slots) slot[g] = (int)s; else slot[g] = -2;
        }
      }
    };
    int next[4];
    int n = warp - MMA_WARP - 1;
    load_slots(n / PARTS, next);
    for (; n < NT * PARTS; n += PRODUCER_WARPS) {
      const int tile = n / PARTS, part = n % PARTS, pos = n % RING, use = n / RING;
      int slot[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) slot[g] = next[g];
      load_slots((n + PRODUCER_WARPS) / PARTS, next);
      if (use > 0 && !__all_sync(0xffffffffu, wait(bar(B_EMPTY + pos), (use - 1) & 1))) break;
      const uint32_t dst = base + OFF_RING + pos * BLOCK;
      const int sub = lane >> 3, col = (lane & 7) * 16;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int row = g * 32 + q * 4 + sub;
          const int s = __shfl_sync(0xffffffffu, slot[g], q * 4 + sub);
          const int64_t at = s < 0 ? 0 : s;
          const uint8_t* src = part == 0 ? reinterpret_cast<const uint8_t*>(a.kr) + at * (DR * 2) + col
                                         : a.c8 + at * DC + (part - 1) * 128 + col;
          cp_async16(dst + swz128(row * 128 + col), src, s < 0 ? 0 : 16);
        }
      }
      if (part == 0) {
        float* ks = reinterpret_cast<float*>(sp + OFF_KS) + (tile % KS_BUFS) * KEYS;
        uint32_t* okw = reinterpret_cast<uint32_t*>(sp + OFF_OK) + (tile % KS_BUFS) * 4;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float s = slot[g] < 0 ? 0.f : a.kv_scale[slot[g] >> a.block_log2];
          ks[g * 32 + lane] = finite(s) ? s : __int_as_float(0x7fc00000);   // a row of infinities has NaN logits
          const uint32_t m = __ballot_sync(0xffffffffu, slot[g] >= 0);
          if (lane == 0) okw[g] = m;
          if (slot[g] == -2) record_error(a.d_err, KDV_DERR_BAD_SLOT);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_KS + tile % KS_BUFS));
      }
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_FULL + pos));
    }
    cp_async_wait_all();
  } else if (warp == MMA_WARP) {
    // ---------------------------------------------------------- MMA issue
    if (lane == 0 && NT > 0) {
      const uint32_t qb = base + OFF_Q, qr = base + OFF_QR, pb = base + OFF_P, ring = base + OFF_RING;
      // Q.K^T of block n (its barrier has been waited for)
      auto qk = [&](int n) {
        const int tile = n / PARTS, part = n % PARTS, pos = n % RING;
        const uint32_t kb = ring + pos * BLOCK, d = tmem + TM_S + (tile & 1) * 128;
        tc_fence_after();
        if (part == 0) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(d, sw128_desc(kb + k * 32, 16, 1024), sw128_desc(qr + k * 32, 16, 1024), IDESC_ROPE, k > 0);
          tc_commit(bar(B_EMPTY + pos));
          // products of two kinds into one accumulator: the second kind waits
          // for the first (it has the softmax's time for that)
          tc_commit(bar(B_ROPE));
          return wait(bar(B_ROPE), tile & 1);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8(d, sw128_desc(kb + k * 32, 16, 1024), sw128_desc(qb + (part - 1) * BLOCK + k * 32, 16, 1024), IDESC_QK, 1u);
        return true;
      };
      bool go = wait(bar(B_Q), 0);
      int n = 0;                                     // next block of Q.K^T
      for (int i = -1; i < NT && go; ++i) {
        if (i >= 0) {
          // the next tile's blocks while this tile's numerators are not ready;
          // the ring holds up to its third
          const int most = (i + 1 < NT) ? (i + 1) * PARTS + 3 : n;
          while (n < most && go && !mbar_test_wait(bar(B_P), i & 1)) {
            if (mbar_test_wait(bar(B_FULL + n % RING), (n / RING) & 1)) {
              go = qk(n);
              ++n;
            } else if (*abort) {
              go = false;
            }
          }
          if (!go || !(go = wait(bar(B_P), i & 1))) break;
          tc_fence_after();
#pragma unroll 1
          for (int mt = 0; mt < 4; ++mt) {
            const int pos = (i * PARTS + 1 + mt) % RING;
            const uint32_t vb = ring + pos * BLOCK;
#pragma unroll
            for (int t = 0; t < TERMS; ++t)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_f8(tmem + mt * 64, sw128_desc(vb + k * 4096, BLOCK, 1024), sw64_desc(pb + t * P_BYTES + k * 2048, P_BYTES, 512),
                       IDESC_PV, (i > 0 || t > 0 || k > 0) ? 1u : 0u);
            tc_commit(bar(B_EMPTY + pos));
          }
        }
        if (i + 1 < NT) {
          const int end = (i + 2) * PARTS;
          while (n < end && go) {
            go = wait(bar(B_FULL + n % RING), (n / RING) & 1) && qk(n);
            ++n;
          }
          if (go) tc_commit(bar(B_S + ((i + 1) & 1)));
        }
      }
      // nothing of this CTA may still run when its tensor memory is given
      // back: a wait of its own, whatever happened before
      tc_commit(bar(B_FIN));
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(bar(B_FIN), 0) && global_ns() - t0 < TIMEOUT_NS) {}
    }
    __syncwarp();
  } else {
    // ------------------------------------------------- queries and softmax
    const int g = warp >> 2, w = warp & 3;           // warpgroup, lane quarter
    float4* cm = reinterpret_cast<float4*>(sp + OFF_CM);
    uint64_t* rmask = reinterpret_cast<uint64_t*>(sp + OFF_MASK);
    float* fac = reinterpret_cast<float*>(sp + OFF_FAC);
    float* red = reinterpret_cast<float*>(sp + OFF_RED) + g * 128;
    float* red2 = reinterpret_cast<float*>(sp + OFF_RED2) + g * 4;
    const uint32_t wg_bar = 1 + g;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    for (int r = warp; r < ROWS; r += SOFTMAX_WARPS) {
      const int lr = r0 + r;
      const bool valid = lr < rows_b;
      const float c = stage_query(a, q + ((int64_t)p.tree_base[b] * p.H + lr) * a.q_row_stride, valid, r, sp, lane);
      if (lane == 0) {
        float* f = reinterpret_cast<float*>(cm + r / 2) + (r & 1);
        f[0] = c;
        f[2] = -NO_MAX;
        rmask[r] = valid ? node_mask(a, p, b, lr / p.H) : 0ull;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(B_Q));
    named_bar_sync(3, SOFTMAX_WARPS * 32);           // both groups have written cm and rmask

    float l[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) l[i] = 0.f;
    float unit = 0.f, inv_unit = 0.f;                // the power of two that s_j is taken relative to
    const uint32_t quarter = (uint32_t)(w * 32) << 16;
    const int key = w * 32 + lane;
    uint8_t* prow = sp + OFF_P + key * ROWS;
    const uint32_t psw = ((uint32_t)key >> 1) & 3u;  // 64-byte swizzle of this key's row

    for (int i = 0; i < NT; ++i) {
      wait(bar(B_KS + i % KS_BUFS), (i / KS_BUFS) & 1);
      const float s = reinterpret_cast<const float*>(sp + OFF_KS)[(i % KS_BUFS) * KEYS + key];
      const uint32_t okw = reinterpret_cast<const uint32_t*>(sp + OFF_OK)[(i % KS_BUFS) * 4 + w];
      const int u = k_lo + i * KEYS + key - L;       // tree key if >= 0
      const bool readable = (okw >> lane) & 1u;
      const bool plain = __all_sync(0xffffffffu, readable && u < 0);
      wait(bar(B_S + (i & 1)), (i >> 1) & 1);
      tc_fence_after();
      float t[32];
      bool dirty;
      {
        uint32_t hi[32], lo[32];
        const uint32_t sb = tmem + quarter + TM_S + (i & 1) * 128 + 32 * g;
        tmem_ld32(sb, hi);
        tmem_ld32(sb + 64, lo);
        tmem_wait_ld();
        dirty = isnan(__uint_as_float(lo[0]));
#pragma unroll
        for (int r = 0; r < 32; ++r) t[r] = fmaf(__uint_as_float(lo[r]), 0.0625f, __uint_as_float(hi[r]));
      }
      // The low terms of a query are finite whatever the query holds, so a NaN
      // in their sums is the key's: its row of V becomes zeros, or 0 * NaN would
      // reach rows that do not see it. (Rows that see it get their NaN from p.)
      if (dirty) {
#pragma unroll 1
        for (int mt = 0; mt < 4; ++mt) {
          uint4* v = reinterpret_cast<uint4*>(sp + OFF_RING + ((i * PARTS + 1 + mt) % RING) * BLOCK + key * 128);
          for (int x = 0; x < 8; ++x) v[x] = make_uint4(0, 0, 0, 0);
        }
      }
      if (plain) {
#pragma unroll
        for (int r = 0; r < 32; ++r) t[r] *= s;
      } else {
#pragma unroll
        for (int r = 0; r < 32; ++r) {
          const bool vis = readable && (u < 0 || ((rmask[32 * g + r] >> u) & 1ull));
          t[r] = vis ? t[r] * s : -INFINITY;
        }
      }
      bool move = fabsf(s) > unit;
#pragma unroll
      for (int r = 0; r < 32; r += 2) {
        const float4 f = cm[16 * g + r / 2];
        const float2 d = fma_f32x2(make_float2(t[r], t[r + 1]), make_float2(f.x, f.y), make_float2(f.z, f.w));
        move |= fmaxf(d.x, d.y) > P_GROW;
      }
      if (named_bar_or(wg_bar, 128, move)) {
        // ---- some reference moves: maxima over the tile's keys, per row
        float mine = 0.f;                            // of row `lane`
#pragma unroll
        for (int r = 0; r < 32; ++r) {
          const float4 f = cm[16 * g + r / 2];
          float x = t[r] * ((r & 1) ? f.y : f.x);
          x = isnan(x) ? -INFINITY : x;
          const float top = warp_max(x);
          if (lane == r) mine = top;
        }
        red[w * 32 + lane] = mine;
        const float smax = warp_max(isnan(s) ? 0.f : fabsf(s));
        if (lane == 0) red2[w] = smax;
        named_bar_sync(wg_bar, 128);
        const float top = fmaxf(fmaxf(red[lane], red[32 + lane]), fmaxf(red[64 + lane], red[96 + lane]));
        const float st = fmaxf(fmaxf(red2[0], red2[1]), fmaxf(red2[2], red2[3]));
        float* cr = reinterpret_cast<float*>(cm + 16 * g + lane / 2) + (lane & 1);
        const float m_old = -cr[2];
        const float m_new = top - P_TOP > m_old ? top - P_TOP : m_old;
        float unit_new = unit;
        if (st > unit) {
          int e;
          const float m = frexpf(st, &e);
          unit_new = ldexpf(1.f, max(m == 0.5f ? e - 1 : e, -120));
        } else if (unit == 0.f) {
          unit_new = ldexpf(1.f, -120);              // scales of 0 so far
        }
        const float shift = ex2(m_old - m_new);
        named_bar_sync(wg_bar, 128);                 // all have read red, red2 and cm
        if (w == 0) {
          cr[2] = -m_new;
          fac[32 * g + lane] = shift;
        }
        named_bar_sync(wg_bar, 128);
        const float us = unit / unit_new;
        unit = unit_new;
        inv_unit = 1.f / unit_new;
#pragma unroll
        for (int r = 0; r < 32; ++r) l[r] *= fac[32 * g + r];
        if (i > 0) {
          // P.V of the tiles before is complete: this tile's S was committed behind it
#pragma unroll 1
          for (int mt = 0; mt < 4; ++mt) {
            uint32_t o[32];
            tmem_ld32(tmem + quarter + mt * 64 + 32 * g, o);
            tmem_wait_ld();
#pragma unroll
            for (int r = 0; r < 32; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * (fac[32 * g + r] * us));
            tmem_st32(tmem + quarter + mt * 64 + 32 * g, o);
          }
          tmem_wait_st();
        }
      }
      const float sr = s * inv_unit;
#pragma unroll
      for (int h = 0; h < 2; ++h) {                  // 16 rows = 16 bytes of each term
        uint32_t w0[4], w1[4], w2[4];
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          uint32_t t0[2], t1[2], t2[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = 16 * h + 4 * q4 + 2 * k;
            const float4 f = cm[16 * g + r / 2];
            const float2 d = fma_f32x2(make_float2(t[r], t[r + 1]), make_float2(f.x, f.y), make_float2(f.z, f.w));
            const float p0 = ex2(d.x), p1 = ex2(d.y);
            l[r] += p0;
            l[r + 1] += p1;
            float e0 = p0 * sr, e1 = p1 * sr;
            if (!plain) {                            // an unseen key's scale may be NaN
              e0 = p0 == 0.f ? 0.f : e0;
              e1 = p1 == 0.f ? 0.f : e1;
            }
            split_p(pack_f16x2(e0, e1), t0[k], t1[k], t2[k]);
          }
          w0[q4] = __byte_perm(t0[0], t0[1], 0x7531);
          w1[q4] = __byte_perm(t1[0], t1[1], 0x7531);
          w2[q4] = t2[0] | (t2[1] << 16);
        }
        uint8_t* at = prow + ((((uint32_t)(2 * g + h)) ^ psw) << 4);
        *reinterpret_cast<uint4*>(at) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
        *reinterpret_cast<uint4*>(at + P_BYTES) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        *reinterpret_cast<uint4*>(at + 2 * P_BYTES) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_P));
    }

    // ---- row sums over the 128 lanes: halves of the rows swap sides, so lane r ends with row r
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int k = 0; k < o; ++k) {
        const float keep = up ? l[k + o] : l[k], send = up ? l[k] : l[k + o];
        l[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
    named_bar_sync(wg_bar, 128);
    red[w * 32 + lane] = l[0];
    named_bar_sync(wg_bar, 128);
    const float sum = (red[lane] + red[32 + lane]) + (red[64 + lane] + red[96 + lane]);
    const float m = -(reinterpret_cast<const float*>(cm + 16 * g + lane / 2) + (lane & 1))[2];
    const bool none = sum == 0.f;
    const float inv = none ? 0.f : 1.f / sum;
    const float lse = none ? -INFINITY : LN2 * (m + log2f(sum));
    const bool direct = p.out_mode == OUT_DIRECT;
    if (w == 0) {
      const int lr = r0 + 32 * g + lane;
      fac[32 * g + lane] = direct ? inv * unit : inv;
      if (lr < rows_b) {
        const int64_t orow = out_row_index(p, b, split, lr);
        if (!direct) a.part_s[orow] = make_float2(lse, unit);
        else if (a.lse != nullptr) a.lse[orow] = lse;
      }
    }
    named_bar_sync(wg_bar, 128);
    if (NT > 0) wait(bar(B_FIN), 0);
    tc_fence_after();
    const int64_t orow0 = out_row_index(p, b, split, r0 + 32 * g);
    const int nr = min(32, rows_b - r0 - 32 * g);
#pragma unroll 1
    for (int mt = 0; mt < 4; ++mt) {
      uint32_t o[32];
      if (NT > 0) {
        tmem_ld32(tmem + quarter + mt * 64 + 32 * g, o);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int r = 0; r < 32; ++r) o[r] = 0u;
      }
      const int dim = mt * 128 + w * 32 + lane;
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        if (r >= nr) break;
        const float f = fac[32 * g + r];
        const float v = f == 0.f ? 0.f : __uint_as_float(o[r]) * f;
        const int64_t at = (orow0 + r) * DC + dim;
        if (!direct) static_cast<__half*>(a.part_o)[at] = __float2half_rn(v);
        else if (a.out_f32) static_cast<float*>(a.o)[at] = v;
        else static_cast<__nv_bfloat16*>(a.o)[at] = __float2bfloat16_rn(v);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == MMA_WARP) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_verify8_tc(const Verify8Args& a, const VerifyPlan& p, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(verify8_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  verify8_tc_kernel<<<p.n_items, THREADS, SMEM_BYTES, stream>>>(a, p);
  return cudaGetLastError();
}

}  // namespace kdv
