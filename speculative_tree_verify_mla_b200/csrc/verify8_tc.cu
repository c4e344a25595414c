// verify8_tc.cu -- attention over the 8-bit latent cache on tcgen05 tensor cores.
//
//   x[r,j] = scale s_j (q_lat[r] . c8[j] + q_rope[r] . kr[j])      (s_j = kv_scale of key j)
//   o[r]   = sum_j p[r,j] s_j c8[j] / sum_j p[r,j],  p = exp(x - max)
//
// The codes are multiplied as they are stored, so a key costs 512 + 128 bytes
// of memory and of shared memory, and nothing is converted:
//   Q.K^T  q_lat times a power of two per row is split in two e4m3 terms,
//          q = hi + lo / 16. bf16 holds 8 significant bits and a term 4, so the
//          split is exact down to 2^-21 of the row's largest latent element, whatever that is
//          (beside a rope element 2^53 times as large: to 2^-74 of the rope element). The rope
//          part is a bf16 product into the same sums. Products of e4m3 codes and
//          their fp32 sums are exact to fp32's rounding (measured: 3e-8).
//   P.V    p s_j is rounded to fp16 and split in three e5m2 terms, the first
//          two truncated (an e5m2 is an fp16's upper byte, so a term is a
//          mask and the rest an exact subtraction), the last one rounded:
//          2^-9 of p s at most, against 2^-8 for a bf16 numerator. e5m2 reaches
//          down to 2^-16 and a row's largest p s is kept within [2^8, 2^15], so
//          keys 2^-24 below the largest still count; with e4m3 terms a long
//          tail of small weights would vanish (2^-18). Two terms would be
//          off by 2.7e-3 (rms) at 0.85 of the time. The reference of a row's exponents
//          is the largest log2(p s_j) of the keys that this row sees, not the largest logit:
//          scales that differ widely, and those of keys that it does not see, take no precision from it.
//
// Both products are formed transposed, keys resp. latent dims as the rows (M)
// of an MMA and 64 query rows as its columns (N): one token of 64 heads fills
// a tile, where rows of queries would leave half of M = 128 empty, and the fp32
// output (64 columns for each of four 128-dim blocks) takes 256 columns of
// TMEM instead of all 512. The same block of keys x 128 dims in the
// 128-byte swizzle is A of Q.K^T (K-major) and A of P.V (M-major). The three terms' MMAs of P.V
// have the same A one after another, which the tensor core keeps: 36 clocks an MMA instead of 48.
//
// One CTA per work item: 64 query rows of one request, one key split, tiles
// of 96 keys. (The queries take 80 KB of shared memory. Beside them two tiles of 96
// fit, so that the softmax of one runs during P.V of the one before and Q.K^T of the one behind; two
// of 128 do not: 7 % slower over 200k keys. The MMAs' rows 96-127 are
// whatever follows a block; nothing reads what they give.)
//   warps 17-19 producers: gather 128-byte row pieces through the page table
//               with cp.async into a ring of ten 12 KB blocks (two rope blocks,
//               two tiles of four latent blocks), each warp a third of every block.
//               (tile::gather4 issues one 512-byte gather in ~65 clocks, 8 B/clk;
//               cp.async beside these MMAs reaches ~28 B/clk.)
//   warp 16     MMA issue, one thread.
//   warps 0-15  four warpgroups: queries in, softmax, output. Lane = key, so a
//               warpgroup owns 16 query rows, a thread one key of them; a row's
//               maximum is only looked for across lanes when some p s passes
//               the reference by 2^7 (a vote), then O is rescaled in TMEM.
//
// What bounds it: the tensor core and shared memory. A tile's 16 (N = 128) + 4 + 36 (N = 64) MMAs take
// 2.55k clocks alone and 3.4k beside the copies and the softmax (71 % of them tensor-active over 200k keys); one
// cp.async block of 12 KB takes ~400. Over 200k keys the part runs into its power cap: 461 us in bursts (about 1.7 GHz),
// 529 us sustained (1.58 GHz; 16 nodes x 64 heads, 967 and 843 TFLOP/s of the logical products, 2176 a row and key).
// As bf16 products its own operations are 2688 of them, 323 us at the measured 1702 TFLOP/s. Contiguous pools through TMA
// boxes instead of the gather: 20 and 11 us more, so there is one way to bring keys in. Few rows over short contexts: 16k
// clocks an item for set-up, queries, first tile and output, and the merge (2.5-4 us): 13 nodes x 64 heads x 5.5k keys 26.2 us.
// (Device times in a graph with the cache warm, but for the 200k keys. 96 registers a thread, 12 bytes of them spilled.)
#include <cuda_fp8.h>

#include "sm100_ptx.cuh"
#include "verify8.cuh"

namespace kdv {
namespace {

using namespace ptx;

constexpr int ROWS = V8_ROWS, KEYS = V8_KEYS, DC = 512, DR = 64;
constexpr int QBLOCK = 16384;                // 128 stacked query rows x 128 bytes
constexpr int BLOCK = KEYS * 128;            // a tile's keys x 128 bytes
constexpr int BLOCKS = 4;                    // latent blocks of a tile, behind its rope block
constexpr int ROPE_PLACES = 2, RING = ROPE_PLACES + 2 * BLOCKS;   // two tiles
constexpr int TERMS = 3, P_BYTES = KEYS * ROWS;   // terms of a numerator (a fill, a use and a last use of V's operand)
constexpr int GROUPS = 4, GROUP_ROWS = ROWS / GROUPS;       // softmax warpgroups, 16 query rows each
constexpr int SOFTMAX_WARPS = 4 * GROUPS, MMA_WARP = SOFTMAX_WARPS, PRODUCER_WARPS = 3;
constexpr int FIRST_PRODUCER = MMA_WARP + 1;
constexpr int THREADS = (FIRST_PRODUCER + PRODUCER_WARPS) * 32;   // 640: 96 registers a thread
// log2 of a row's largest numerator p s when its reference is set, and the most that it may grow to (5.5k layer: 26.2 us,
// 27.0 with a reference set to 10, 28.9 with 12: references move less often)
constexpr float P_TOP = 8.f, P_GROW = 15.f;
// Scales are taken times 2^16: those of 2^-108 to 2^111 have room, smaller ones lose precision and larger ones count as infinite.
// (p = 2^8 / (2^16 s) for the key that sets the reference, and ex2 flushes below 2^-126: from s = 2^94 on the smallest weights go.)
constexpr float SCALE_UP = 65536.f, SCALE_UP_LOG2 = 16.f;
constexpr float SCALE_MIN = -92.f;           // log2 of the least that a reference counts: p stays below 2^107, sums of 2^20 in fp32
// |o| <= 448 n 2^15 / l for n keys: 57344 in units of 256 n / l. Where one key of a part holds all the weight, p s >= 2^8
// leaves code / 2 n of it, and fp16's step of 2^-24 is off by n 2^-24 of a code at most: at 32768 keys e4m3's own least step.
// (A second bound, by the largest scale seen, would lift that for 0.5 us of a 5.5k layer's 26.5.)
constexpr float PART_UNIT = 256.f;
constexpr float NO_MAX = -1e30f;             // the reference of a row that has seen no key
constexpr float LN2 = 0.6931471805599453f;
constexpr uint64_t TIMEOUT_NS = 1000000000ull;
constexpr uint32_t POLLS = 64;               // between two looks at the clock,
constexpr uint64_t SHORT_NS = 100000;        // unless the limit is shorter than they may take

constexpr int OFF_Q = 0;                                   // 4 blocks: rows 0-63 hi, 64-127 lo
constexpr int OFF_QR = OFF_Q + 4 * QBLOCK;                 // rows 0-63 q_rope bf16, 64-127 zero
constexpr int OFF_P = OFF_QR + QBLOCK;
constexpr int OFF_RING = OFF_P + TERMS * P_BYTES;
// an MMA reads 128 rows of a block: the last one's end is 4 KB further
constexpr int OFF_MASK = OFF_RING + RING * BLOCK;          // u64 [64] node masks by row
constexpr int OFF_CM = OFF_MASK + ROWS * 8;                // float4 [32]: (c, c', -m, -m') of a row pair
constexpr int OFF_RED = OFF_CM + 32 * 16;                  // float [GROUPS][4][16]
constexpr int OFF_FAC = OFF_RED + GROUPS * 4 * GROUP_ROWS * 4;   // float [64] per-row factors
constexpr int OFF_BAR = OFF_FAC + ROWS * 4;
constexpr int B_FULL = 0, B_EMPTY = B_FULL + RING, B_S = B_EMPTY + RING, B_P = B_S + 2,
              B_PV = B_P + 1, B_ROPE = B_PV + 1, B_Q = B_ROPE + 1, B_FIN = B_Q + 1, NUM_BARS = B_FIN + 1;
constexpr int OFF_TMEM = OFF_BAR + NUM_BARS * 8;
constexpr int OFF_ABORT = OFF_TMEM + 4;
constexpr int SMEM_BYTES = (OFF_ABORT + 4 > OFF_MASK + (128 - KEYS) * 128 ? OFF_ABORT + 4 : OFF_MASK + (128 - KEYS) * 128) + 1024;
static_assert(KEYS == 96 && KEYS * ROWS % 512 == 0, "tile");
static_assert(OFF_BAR % 8 == 0 && OFF_MASK % 8 == 0 && OFF_CM % 16 == 0, "alignment");
static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory");
constexpr uint32_t TM_S = BLOCKS * ROWS;                   // S buffers behind the output columns
static_assert(TM_S + 4 * ROWS <= 512, "tensor memory");

// KEEP: what happens to A in the tensor core's operand buffer. Three MMAs in
// a row with the same A read it from shared memory once: 36 clocks each (M 128, N 64), 48 without.
enum class A { ONCE, FILL, USE, LAST };
template <A KEEP = A::ONCE>
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
#define KDV_MMA_F8(COLLECT) \
  asm volatile( \
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t" \
      "tcgen05.mma.cta_group::1.kind::f8f6f4" COLLECT " [%0], %1, %2, %3, p;\n\t}" \
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory")
  if constexpr (KEEP == A::FILL) KDV_MMA_F8(".collector::a::fill");
  else if constexpr (KEEP == A::USE) KDV_MMA_F8(".collector::a::use");
  else if constexpr (KEEP == A::LAST) KDV_MMA_F8(".collector::a::lastuse");
  else KDV_MMA_F8("");
#undef KDV_MMA_F8
}
// One lane of a converged warp, the same at every call. The issuing warp runs
// its loop with all lanes and elects around each block of MMAs: measured 48 clocks an
// N = 64 MMA, 69 with a predicate on each (which is what their operands take to read: 46).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// kind::f8f6f4 with fp32 D: formats 0 e4m3, 1 e5m2
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a_fmt, int b_fmt, bool a_mn, bool b_mn) {
  return (1u << 4) | ((uint32_t)a_fmt << 7) | ((uint32_t)b_fmt << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t IDESC_QK = idesc_f8(128, 128, 0, 0, false, false);
constexpr uint32_t IDESC_ROPE = idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t IDESC_PV = idesc_f8(128, ROWS, 0, 1, true, true);

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
// Waits within the CTA. (The cluster-scope forms of the shared header cost this
// kernel about 500 clocks each.)
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" :: "l"(p)); }
// Arrives on `bar` when all of this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Bounded waits: a wait that runs out reports, raises the CTA's abort flag and
// returns false; from then on every other wait of the CTA returns at once.
struct Waiter {
  volatile int* abort;
  int32_t* d_err;
  uint64_t limit;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (mbar_try(bar, parity)) return true;
    return slow(bar, parity);
  }
  // (Reading the global timer takes hundreds of clocks, so it is looked at
  // once in many polls: with one read a poll each wait ended that much late.)
  __device__ __forceinline__ bool slow(uint32_t bar, uint32_t parity) const {
    uint64_t t0 = 0;
    for (uint32_t n = 1;; ++n) {
      if (mbar_try(bar, parity)) return true;
      if (n % POLLS != 0 && limit >= SHORT_NS) continue;
      if (*abort) return false;
      const uint64_t now = global_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit) {
        *abort = 1;
        record_error(d_err, KDV_DERR_TIMEOUT);
        return false;
      }
    }
  }
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }
__device__ __forceinline__ uint32_t e4m3x2(uint32_t f16x2) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(f16x2));
  return c;
}
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return h;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^k: infinite where it is no float, 2^-149 at least (the product with a logit of -inf has to stay that)
__device__ __forceinline__ float power_of_two(int k) {
  return __int_as_float(k > 127 ? 0x7f800000 : k >= -126 ? (k + 127) << 23 : 1 << max(k + 149, 0));
}

// ------------------------------------------------------------------ queries
constexpr uint32_t PLAIN_LATENT = (127 - 21) << 7, PLAIN_ROPE = (127 + 32) << 7;   // bf16 bits of 2^-21 and 2^32
// One row by one warp: lane l holds latent elements 16 l .. 16 l + 15 and rope
// elements 2 l, 2 l + 1.
struct QueryRow {
  uint32_t u[8], rope;
  __device__ __forceinline__ void load(const __nv_bfloat16* row, bool valid, int lane) {
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    rope = 0;
    if (valid) {
      w0 = reinterpret_cast<const uint4*>(row)[2 * lane];
      w1 = reinterpret_cast<const uint4*>(row)[2 * lane + 1];
      rope = reinterpret_cast<const uint32_t*>(row + DC)[lane];
    }
    u[0] = w0.x; u[1] = w0.y; u[2] = w0.z; u[3] = w0.w;
    u[4] = w1.x; u[5] = w1.y; u[6] = w1.z; u[7] = w1.w;
  }
  // The row's largest magnitude, as the bits of a bf16: 0x7f80 or more where it holds an infinity or a NaN.
  __device__ __forceinline__ uint32_t magnitude() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, u[i] & 0x7fff7fffu);
    return __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  }
  // The same of its finite elements alone.
  __device__ __forceinline__ uint32_t finite_magnitude() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t lo = u[i] & 0x7fffu, hi = (u[i] >> 16) & 0x7fffu;
      m = max(m, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
    }
    return __reduce_max_sync(0xffffffffu, m);
  }
  // The magnitudes of this lane's rope elements.
  __device__ __forceinline__ uint32_t rope_magnitudes() const { return rope & 0x7fff7fffu; }
  // The exponent of the power of two that the row is staged times. Plain rows: largest latent element of 2^-21 or more,
  // which comes into [128, 256) (or a row of zeros), rope elements below 2^32.
  __device__ __forceinline__ static bool plain(uint32_t top) { return top == 0u || (top >= PLAIN_LATENT && top < 0x7f80u); }
  __device__ __forceinline__ static int plain_exponent(uint32_t top) { return top == 0u ? 0 : 7 + 127 - (int)(top >> 7); }
  // Any row: the same of its finite elements, but rope elements stay below 2^61. A row without latents goes by its rope part.
  __device__ __forceinline__ int any_exponent(bool& zeros) const {
    const uint32_t lat = finite_magnitude(), lo = rope & 0x7fffu, hi = (rope >> 16) & 0x7fffu;
    const uint32_t rp = __reduce_max_sync(0xffffffffu, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
    auto exponent = [](uint32_t m) { return m >= 0x80u ? (int)(m >> 7) - 127 : -102 - __clz(m); };   // floor(log2), m > 0
    zeros = lat == 0u && rp == 0u;
    if (lat == 0u) return zeros ? 0 : 7 - exponent(rp);
    return rp == 0u ? 7 - exponent(lat) : min(7 - exponent(lat), 60 - exponent(rp));
  }
  // Writes the row's terms times 2^e. bad: some element is not finite, or 2^e is no float.
  template <bool bad> __device__ __forceinline__ void stage(int e, int r, uint8_t* sp, int lane) const {
    const uint32_t blk = (uint32_t)(lane / 8) * QBLOCK, col = (uint32_t)(lane % 8) * 16;
    *reinterpret_cast<uint32_t*>(sp + OFF_QR + swz128((r + ROWS) * 128 + lane * 4)) = 0u;
    const int first = bad ? min(e, 100) : e;              // -120 <= e <= 140: in two steps
    const float up = __int_as_float((first + 127) << 23), rest = bad ? __int_as_float((e - first + 127) << 23) : 1.f;
    // (fp16 holds the scaled elements: exact down to 2^-14, off by 2^-25 at most below)
    uint32_t hi[4], lo[4];
    const __half2 sixteen = __float2half2_rn(16.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x0 = __uint_as_float(u[2 * i + j] << 16) * up, x1 = __uint_as_float(u[2 * i + j] & 0xffff0000u) * up;
        if (bad) {
          x0 *= rest;
          x1 *= rest;
          x0 = finite(x0) ? x0 : __int_as_float(0x7fc00000);
          x1 = finite(x1) ? x1 : __int_as_float(0x7fc00000);
        }
        const uint32_t x = pack_f16x2(x0, x1), h = e4m3x2(x), back = e4m3x2_f16(h);
        __half2 y = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&back)), sixteen);
        if (bad) {                                   // the low terms stay finite, see the softmax
          y.x = __hisnan(y.x) ? __half(0.f) : y.x;
          y.y = __hisnan(y.y) ? __half(0.f) : y.y;
        }
        const uint32_t l = e4m3x2(*reinterpret_cast<const uint32_t*>(&y));
        hi[i] = j == 0 ? h : hi[i] | (h << 16);
        lo[i] = j == 0 ? l : lo[i] | (l << 16);
      }
    }
    *reinterpret_cast<uint4*>(sp + OFF_Q + blk + swz128(r * 128 + col)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(sp + OFF_Q + blk + swz128((r + ROWS) * 128 + col)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    const float ra = __uint_as_float(rope << 16) * up * rest, rb = __uint_as_float(rope & 0xffff0000u) * up * rest;
    *reinterpret_cast<uint32_t*>(sp + OFF_QR + swz128(r * 128 + lane * 4)) = pack_bf16x2(ra, rb);
  }
};

// Reduction of 16 values a lane over the warp's lanes: halves of the rows swap
// sides, so that lane r ends with row r mod 16 (16 shuffles, where a reduction for each row takes 80).
template <typename F> __device__ __forceinline__ float transpose_reduce(float (&v)[16], int lane, F join) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int k = 0; k < o; ++k) {
      const float keep = up ? v[k + o] : v[k], send = up ? v[k] : v[k + o];
      v[k] = join(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  return join(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
         "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
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

// Places of the ring: rope blocks alternate between two, latent blocks between two sets.
__device__ __forceinline__ int rope_place(int tile) { return tile & 1; }
__device__ __forceinline__ int latent_place(int tile, int x) { return ROPE_PLACES + (tile & 1) * BLOCKS + x; }

__global__ void __launch_bounds__(THREADS, 1) verify8_tc_kernel(const __grid_constant__ Verify8Args a,
                                                                const __grid_constant__ VerifyPlan p) {
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* sp = raw + (base - smem_u32(raw));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](int i) { return base + OFF_BAR + 8 * i; };
  volatile int* abort = reinterpret_cast<volatile int*>(sp + OFF_ABORT);
  const Waiter wait{abort, a.d_err, a.wait_limit_ns ? a.wait_limit_ns : TIMEOUT_NS};

  if (tid == FIRST_PRODUCER * 32) {
    for (int i = 0; i < RING; ++i) {
      mbar_init(bar(B_FULL + i), 32 * PRODUCER_WARPS);
      mbar_init(bar(B_EMPTY + i), 1);
    }
    mbar_init(bar(B_S), 1);
    mbar_init(bar(B_S + 1), 1);
    mbar_init(bar(B_PV), 1);
    mbar_init(bar(B_FIN), 1);
    mbar_init(bar(B_P), SOFTMAX_WARPS);
    mbar_init(bar(B_ROPE), 1);
    mbar_init(bar(B_Q), SOFTMAX_WARPS);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(base + OFF_TMEM, 512);
    tmem_relinquish();
  }
  const int item = blockIdx.x;
  const int b = plan_request(p, item);
  // The launch overlaps the end of the kernel before it on the stream; from here on its results are read.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int local = item - p.item_base[b];
  const int split = local / p.tiles[b], rt = local - split * p.tiles[b];
  const int rows_b = p.T[b] * p.H, r0 = rt * ROWS;
  // this warp's query rows and a lane's row's mask: on their way while the CTA sets up
  QueryRow row[4];
  uint64_t qmask = 0;
  if (warp < SOFTMAX_WARPS) {
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + ((int64_t)p.tree_base[b] * p.H + r0 + 4 * warp) * a.q_row_stride;
#pragma unroll
    for (int k = 0; k < 4; ++k) row[k].load(q + k * a.q_row_stride, r0 + 4 * warp + k < rows_b, lane);
    const int lr = r0 + 4 * warp + lane;
    if (lane < 4 && lr < rows_b) qmask = node_mask(a, p, b, lr / p.H);
  }
  const int L = p.L[b], n_keys = L + p.T[b];
  const bool ok = request_ok(a, p, b, tid == 0 && local == 0);
  const int64_t lo64 = (int64_t)split * p.chunk[b];
  const int k_lo = (int)min(lo64, (int64_t)n_keys);
  const int k_hi = ok ? (int)min(lo64 + p.chunk[b], (int64_t)n_keys) : k_lo;
  const int NT = (k_hi - k_lo + KEYS - 1) / KEYS;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sp + OFF_TMEM);

  // A key's pool slot in two steps, so that nothing waits for the page table
  // where it is read: its entry, and a tile later what that means (-1 no key, -2 outside the pool).
  const int64_t kv_base = a.kv_off[b];
  auto entry_of = [&](int j) { return j >= k_hi ? -1 : a.page_table ? a.page_table[kv_base + j] : (int)(kv_base + j); };
  auto slot_of = [&](int j, int entry) { return j >= k_hi ? -1 : entry >= 0 && entry < a.num_slots ? entry : -2; };
  if (warp >= FIRST_PRODUCER) {
    // ---------------------------------------------------------- producers
    // Every warp brings a third of each block (four rows a copy), so that a block freed
    // by P.V is full again as soon as may be. A lane's copies arrive on the block's
    // barrier by themselves; the fence between them and the tensor cores' reads is the issuing
    // thread's, behind its wait (a fence here drains the copies in flight: measured 900 clocks a block instead of 350).
    constexpr int COPIES = KEYS / 4 / PRODUCER_WARPS;
    static_assert(COPIES * PRODUCER_WARPS * 4 == KEYS, "a warp's share of a block");
    const int mine = warp - FIRST_PRODUCER, sub = lane >> 3, col = (lane & 7) * 16;
    auto row = [&](int q) { return (mine + PRODUCER_WARPS * q) * 4 + sub; };
    int next[COPIES];                                // this lane's rows in the page table, read a tile ahead
    auto load_slots = [&](int tile) {
#pragma unroll
      for (int q = 0; q < COPIES; ++q) next[q] = entry_of(k_lo + tile * KEYS + row(q));
    };
    const uint8_t* c8 = a.c8 + col;
    const uint8_t* kr = reinterpret_cast<const uint8_t*>(a.kr) + col;
    const uint32_t ring = base + OFF_RING;
    load_slots(0);
    for (int tile = 0; tile < NT; ++tile) {
      uint32_t s[COPIES], take = 0;                  // which rows are readable; the others become zeros
#pragma unroll
      for (int q = 0; q < COPIES; ++q) {
        const int slot = slot_of(k_lo + tile * KEYS + row(q), next[q]);
        s[q] = (uint32_t)max(slot, 0);
        take |= slot >= 0 ? 1u << q : 0u;
      }
      load_slots(tile + 1);
      bool go = true;
#pragma unroll
      for (int part = 0; part <= BLOCKS; ++part) {
        const int pos = part == 0 ? rope_place(tile) : latent_place(tile, part - 1), use = tile >> 1;
        if (use > 0 && !(go = __all_sync(0xffffffffu, wait(bar(B_EMPTY + pos), (use - 1) & 1)))) break;
        const uint8_t* src = part == 0 ? kr : c8 + (part - 1) * 128;
        const uint32_t pitch = part == 0 ? DR * 2 : DC;
#pragma unroll
        for (int q = 0; q < COPIES; ++q)
          cp_async16_or_zero(ring + pos * BLOCK + swz128(row(q) * 128 + col), src + (uint64_t)s[q] * pitch, (take >> q) & 1u ? 16 : 0);
        cp_async_arrive(bar(B_FULL + pos));
      }
      if (!go) break;
    }
    cp_async_wait_all();
  } else if (warp == MMA_WARP) {
    // ---------------------------------------------------------- MMA issue
    // One thread. The pipe takes few MMAs ahead, so the time between two of
    // them is its idle time: blocks of MMAs are long and their waits lie behind others.
    // P.V of tile i, then Q.K^T of tile i + 2, while the softmax works on tile i + 1. (Products of
    // another kind into the same sums wait for the rope part's end, which P.V's last block covers.)
    if (NT > 0 && elect_one()) {
      const uint64_t q_desc = sw128_desc(base + OFF_Q, 16, 1024), qr_desc = sw128_desc(base + OFF_QR, 16, 1024);
      const uint64_t p_desc = sw64_desc(base + OFF_P, P_BYTES, 512);
      const uint64_t k_desc = sw128_desc(base + OFF_RING, 16, 1024), v_desc = sw128_desc(base + OFF_RING, BLOCK, 1024);
      auto rope = [&](int i) {
        const int at = rope_place(i);
        if (!wait(bar(B_FULL + at), (i >> 1) & 1)) return false;
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t kb = k_desc + (uint32_t)(at * (BLOCK / 16));
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_ss(tmem + TM_S + (i & 1) * 128, kb + 2 * k, qr_desc + 2 * k, IDESC_ROPE, k > 0);
        tc_commit(bar(B_EMPTY + at));
        tc_commit(bar(B_ROPE));
        return true;
      };
      auto latents = [&](int i) {
        if (!wait(bar(B_ROPE), i & 1)) return false;
#pragma unroll
        for (int x = 0; x < BLOCKS; ++x) {
          const int at = latent_place(i, x);
          const uint64_t kb = k_desc + (uint32_t)(at * (BLOCK / 16)), qb = q_desc + (uint32_t)(x * (QBLOCK / 16));
          if (!wait(bar(B_FULL + at), (i >> 1) & 1)) return false;
          fence_proxy_async_smem();
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f8(tmem + TM_S + (i & 1) * 128, kb + 2 * k, qb + 2 * k, IDESC_QK, 1u);
        }
        tc_commit(bar(B_S + (i & 1)));
        return true;
      };
      auto values = [&](int i, int x) {
        const int at = latent_place(i, x);
        const uint64_t vb = v_desc + (uint32_t)(at * (BLOCK / 16));
        const uint32_t d = tmem + x * ROWS;
#pragma unroll
        for (int k = 0; k < KEYS / 32; ++k) {
          const uint64_t v = vb + k * 256, p = p_desc + k * (2048 / 16);
          mma_f8<A::FILL>(d, v, p, IDESC_PV, k > 0 ? 1u : (uint32_t)(i > 0));
          mma_f8<A::USE>(d, v, p + P_BYTES / 16, IDESC_PV, 1u);
          mma_f8<A::LAST>(d, v, p + 2 * P_BYTES / 16, IDESC_PV, 1u);
        }
        tc_commit(bar(B_EMPTY + at));
      };
      bool go = wait(bar(B_Q), 0);
      for (int i = 0; i < 2 && i < NT && go; ++i) go = rope(i) && latents(i);
      for (int i = 0; i < NT && go; ++i) {
        const bool more = i + 2 < NT;
        if (!(go = wait(bar(B_P), i & 1))) break;
        tc_fence_after();
        values(i, 0);
        values(i, 1);
        values(i, 2);
        if (more) go = rope(i + 2);
        values(i, 3);
        tc_commit(bar(B_PV));
        if (more) go = go && latents(i + 2);
      }
      // nothing of this CTA may still run when its tensor memory is given
      // back: a wait of its own, whatever happened before
      tc_commit(bar(B_FIN));
      const uint64_t t0 = global_ns();
      while (!mbar_try(bar(B_FIN), 0) && global_ns() - t0 < TIMEOUT_NS) {}
    }
    __syncwarp();
  } else if (warp < SOFTMAX_WARPS) {
    // ------------------------------------------------- queries and softmax
    const int g = warp >> 2, w = warp & 3;           // warpgroup, lane quarter
    float4* cm = reinterpret_cast<float4*>(sp + OFF_CM) + g * (GROUP_ROWS / 2);    // this group's
    uint64_t* rmask = reinterpret_cast<uint64_t*>(sp + OFF_MASK) + g * GROUP_ROWS;
    float* fac = reinterpret_cast<float*>(sp + OFF_FAC) + g * GROUP_ROWS;
    float* red = reinterpret_cast<float*>(sp + OFF_RED) + g * 4 * GROUP_ROWS;
    const uint32_t wg_bar = 1 + g;
    {
      // a warp stages four rows of its group, all loads in flight
      int e[4];
      uint32_t top[4], rope = 0;
      bool odd = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) top[k] = row[k].magnitude();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        rope = __vmaxu2(rope, row[k].rope_magnitudes());
        odd |= !QueryRow::plain(top[k]) || (top[k] == 0u && row[k].rope_magnitudes() != 0u);
      }
      odd |= (rope & 0xffffu) >= PLAIN_ROPE || (rope >> 16) >= PLAIN_ROPE;
      if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          bool zeros;
          e[k] = row[k].any_exponent(zeros);
          row[k].stage<true>(e[k], 4 * warp + k, sp, lane);
          if (zeros) e[k] = a.scale_exponent;        // logits of 0 take the factor 1 at any softmax scale
        }
      } else {                                       // four independent streams of instructions
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          e[k] = QueryRow::plain_exponent(top[k]);
          row[k].stage<false>(e[k], 4 * warp + k, sp, lane);
          if (top[k] == 0u) e[k] = a.scale_exponent;
        }
      }
      if (lane < 4) {
        const int r = 4 * warp + lane;
        float* f = reinterpret_cast<float*>(sp + OFF_CM) + (r / 2) * 4 + (r & 1);
        f[0] = power_of_two(a.scale_exponent - (lane == 0 ? e[0] : lane == 1 ? e[1] : lane == 2 ? e[2] : e[3]));
        f[2] = -NO_MAX;
        reinterpret_cast<uint64_t*>(sp + OFF_MASK)[r] = qmask;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(B_Q));
    named_bar_sync(wg_bar, 128);                     // the group's cm and rmask are written

    float l[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) l[i] = 0.f;
    const uint32_t quarter = tmem + ((uint32_t)(w * 32) << 16);
    const int key = w * 32 + lane;                   // also the dim of a block; the last quarter has no keys
    auto key_of = [&](int tile) { return key < KEYS ? k_lo + tile * KEYS + key : k_hi; };   // k_hi: no key
    uint8_t* prow = sp + OFF_P + key * ROWS + (((uint32_t)g ^ (((uint32_t)key >> 1) & 3u)) << 4);   // 64-byte swizzle

    // This key's scale is read a tile ahead, its slot two. The ring holds little more
    // than a tile, so a block's copies start late: its rows are asked into L2 when their
    // slots are known, a 128-byte line by each group, for all row tiles of a request by the
    // first one (measured over 200k keys: 466 us, 479 with every row tile's own requests, 488 with none).
    auto scale_of = [&](int slot) { return slot < 0 ? 0.f : a.kv_scale[slot >> a.block_log2]; };
    auto prefetch = [&](int slot) {
      if (slot < 0 || rt != 0) return;
      prefetch_l2(a.c8 + (int64_t)slot * DC + 128 * g);
      if (g == 0) prefetch_l2(static_cast<const __nv_bfloat16*>(a.kr) + (int64_t)slot * DR);
    };
    int slot = entry_of(key_of(0)), slot_next = entry_of(key_of(1)), entry = entry_of(key_of(2));
    slot = slot_of(key_of(0), slot);
    slot_next = slot_of(key_of(1), slot_next);
    float ks = scale_of(slot), ks_next = scale_of(slot_next);
    prefetch(slot_next);

    for (int i = 0; i < NT; ++i) {
      if (g == 0 && slot == -2) record_error(a.d_err, KDV_DERR_BAD_SLOT);
      const float sr = ks * SCALE_UP;
      const float s = finite(sr) ? ks : __int_as_float(0x7fc00000);   // a row of infinities has NaN logits
      const bool readable = slot >= 0;
      const int u = k_lo + i * KEYS + key - L;       // tree key if >= 0
      const bool plain = __all_sync(0xffffffffu, readable && u < 0);
      wait(bar(B_S + (i & 1)), (i >> 1) & 1);
      tc_fence_after();
      const float sl = s * a.scale_part;
      float t[16], d[16];
      bool dirty;
      {                                              // t = scale_part s_j (q . k) 2^e, -inf where the row does not see the key
        uint32_t hi[16], lo[16];
        const uint32_t sb = quarter + TM_S + (i & 1) * 128 + GROUP_ROWS * g;
        tmem_ld16(sb, hi);
        tmem_ld16(sb + ROWS, lo);
        tmem_wait_ld();
        dirty = key < KEYS && isnan(__uint_as_float(lo[0]));
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
          float2 x = fma_f32x2(make_float2(__uint_as_float(lo[r]), __uint_as_float(lo[r + 1])), make_float2(0.0625f, 0.0625f),
                               make_float2(__uint_as_float(hi[r]), __uint_as_float(hi[r + 1])));
          x = mul_f32x2(x, make_float2(sl, sl));
          t[r] = x.x;
          t[r + 1] = x.y;
        }
        if (!plain) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const bool vis = readable && (u < 0 || ((rmask[r] >> u) & 1ull));
            t[r] = vis ? t[r] : -INFINITY;
          }
        }
      }
      const float ls = fmaxf(lg2(fabsf(s)) + SCALE_UP_LOG2, SCALE_MIN);
      // d = log2 of p; the largest. The rows' factors 2^(scale_exponent - e) are powers of two, so a product is exact and the reference one
      // of these products: the largest key's difference stays small at any size of the logits.
      auto exponents = [&]() {
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
          const float4 f = cm[r / 2];
          const float2 x = fma_f32x2(make_float2(t[r], t[r + 1]), make_float2(f.x, f.y), make_float2(f.z, f.w));
          d[r] = x.x;
          d[r + 1] = x.y;
          top = fmaxf(top, fmaxf(x.x, x.y));
        }
        return top;
      };
      // The low terms of a query are finite whatever the query holds, so a NaN
      // in their sums is the key's: its row of V becomes zeros, or 0 * NaN would
      // reach rows that do not see it. (Rows that see it get their NaN from p.)
      if (dirty) {
#pragma unroll 1
        for (int mt = 0; mt < BLOCKS; ++mt) {
          uint4* v = reinterpret_cast<uint4*>(sp + OFF_RING + latent_place(i, mt) * BLOCK + key * 128);
          for (int x = 0; x < 8; ++x) v[x] = make_uint4(0, 0, 0, 0);
        }
      }
      // the first tile sets the reference in any case
      const bool move = i == 0 || exponents() + ls > P_GROW;
      if (i == 0 || named_bar_or(wg_bar, 128, move)) {
        // ---- some reference moves: maxima over the tile's keys, per row
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
          const float4 f = cm[r / 2];
          const float2 x = fma_f32x2(make_float2(t[r], t[r + 1]), make_float2(f.x, f.y), make_float2(ls, ls));
          d[r] = x.x;
          d[r + 1] = x.y;
        }
        const float mine = transpose_reduce(d, lane, [](float x, float y) { return fmaxf(x, y); });   // of row `lane`
        if (lane < GROUP_ROWS) red[w * GROUP_ROWS + lane] = mine;
        named_bar_sync(wg_bar, 128);
        if (w == 0) {                                // one warp moves the rows' references
          const int row = lane & (GROUP_ROWS - 1);
          const float top = fmaxf(fmaxf(red[row], red[16 + row]), fmaxf(red[32 + row], red[48 + row]));   // NaN: no key moves it
          float* cr = reinterpret_cast<float*>(cm + row / 2) + (row & 1);
          const float m_old = -cr[2], m_new = top - m_old > P_GROW ? top - P_TOP : m_old;   // a row's own keys decide
          __syncwarp();
          if (lane < GROUP_ROWS) {
            cr[2] = -m_new;
            fac[lane] = ex2(m_old - m_new);
          }
        }
        named_bar_sync(wg_bar, 128);
        if (i > 0) {
          wait(bar(B_PV), (i - 1) & 1);              // P.V of the tiles before is complete
          tc_fence_after();
#pragma unroll
          for (int r = 0; r < 16; ++r) l[r] *= fac[r];
#pragma unroll 1
          for (int x = 0; x < BLOCKS; ++x) {
            uint32_t o[16];
            tmem_ld16(quarter + x * ROWS + GROUP_ROWS * g, o);
            tmem_wait_ld();
#pragma unroll
            for (int r = 0; r < 16; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * fac[r]);
            tmem_st16(quarter + x * ROWS + GROUP_ROWS * g, o);
          }
          tmem_wait_st();
        }
        exponents();
        // A reference of 2^24 and more is rounded to whole units.
#pragma unroll
        for (int r = 0; r < 16; ++r) d[r] = d[r] > P_GROW - ls ? P_GROW - ls : d[r];
      }
      uint32_t w0[4], w1[4], w2[4];                  // 16 rows = 16 bytes of each term
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) {
        uint32_t t0[2], t1[2], t2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = 4 * q4 + 2 * k;
          const float p0 = ex2(d[r]), p1 = ex2(d[r + 1]);
          const float2 sum = add_f32x2(make_float2(l[r], l[r + 1]), make_float2(p0, p1));
          l[r] = sum.x;
          l[r + 1] = sum.y;
          float2 e = mul_f32x2(make_float2(p0, p1), make_float2(sr, sr));
          if (!plain) {                              // an unseen key's scale may be NaN
            e.x = p0 == 0.f ? 0.f : e.x;
            e.y = p1 == 0.f ? 0.f : e.y;
          }
          split_p(pack_f16x2(e.x, e.y), t0[k], t1[k], t2[k]);
        }
        w0[q4] = __byte_perm(t0[0], t0[1], 0x7531);
        w1[q4] = __byte_perm(t1[0], t1[1], 0x7531);
        w2[q4] = t2[0] | (t2[1] << 16);
      }
      if (i > 0) wait(bar(B_PV), (i - 1) & 1);       // the numerators' place is free
      if (key < KEYS) {
        *reinterpret_cast<uint4*>(prow) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
        *reinterpret_cast<uint4*>(prow + P_BYTES) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        *reinterpret_cast<uint4*>(prow + 2 * P_BYTES) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_P));
      slot = slot_next;
      ks = ks_next;
      slot_next = slot_of(key_of(i + 2), entry);
      ks_next = scale_of(slot_next);
      prefetch(slot_next);
      entry = entry_of(key_of(i + 3));
    }

    if (tid == 0) asm volatile("griddepcontrol.launch_dependents;");   // the merge's launch overlaps the rest
    // ---- row sums over the 128 lanes
    const float part = transpose_reduce(l, lane, [](float x, float y) { return x + y; });
    named_bar_sync(wg_bar, 128);
    if (lane < GROUP_ROWS) red[w * GROUP_ROWS + lane] = part;
    named_bar_sync(wg_bar, 128);
    const bool direct = p.out_mode == OUT_DIRECT;
    const int64_t orow0 = out_row_index(p, b, split, r0 + GROUP_ROWS * g);
    const int nr = min(GROUP_ROWS, rows_b - r0 - GROUP_ROWS * g);      // rows to write, may be below 0
    if (w == 0 && lane < GROUP_ROWS) {
      const float sum = (red[lane] + red[16 + lane]) + (red[32 + lane] + red[48 + lane]);
      const float m = -(reinterpret_cast<const float*>(cm + lane / 2) + (lane & 1))[2];
      const bool none = sum == 0.f;
      const float inv = none ? 0.f : 1.f / sum / SCALE_UP;
      const float lse = none ? -INFINITY : LN2 * (m + log2f(sum));
      // a part's unit: a power of two
      const float u = fminf(inv * (PART_UNIT * (float)(NT * KEYS)), 0x1p126f);
      const float unit = none ? 1.f : __uint_as_float((__float_as_uint(u) + 0x7fffffu) & 0xff800000u);
      fac[lane] = direct ? inv : inv * (1.f / unit);
      if (lane < nr) {
        if (!direct) a.part_s[orow0 + lane] = make_float2(lse, unit);
        else if (a.lse != nullptr) a.lse[orow0 + lane] = lse;
      }
    }
    named_bar_sync(wg_bar, 128);
    if (NT > 0) wait(bar(B_FIN), 0);
    tc_fence_after();
    // Output: lanes are dims and columns rows, so a block of 128 dims goes
    // through shared memory (the ring is free) and leaves in 16-byte pieces of rows.
    uint8_t* stage = sp + OFF_RING + g * (2 * GROUP_ROWS * 512);
    auto write = [&](auto zero, auto convert, void* dst) {
      using T = decltype(zero);
      constexpr int LINE = 128 * sizeof(T), PER = LINE / 16;
      uint8_t* out = static_cast<uint8_t*>(dst) + orow0 * 4 * LINE;
      float f[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) f[r] = fac[r];
      uint32_t o[16], ahead[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) o[r] = ahead[r] = 0u;
      if (NT > 0) {
        tmem_ld16(quarter + GROUP_ROWS * g, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int mt = 0; mt < BLOCKS; ++mt) {
        T* buf = reinterpret_cast<T*>(stage + (mt & 1) * (GROUP_ROWS * 512));
        if (NT > 0 && mt + 1 < BLOCKS) tmem_ld16(quarter + (mt + 1) * ROWS + GROUP_ROWS * g, ahead);
#pragma unroll
        for (int r = 0; r < 16; ++r) buf[r * 128 + key] = convert(f[r] == 0.f ? 0.f : __uint_as_float(o[r]) * f[r]);
        named_bar_sync(wg_bar, 128);                 // the other buffer's readers have passed the barrier before this one
#pragma unroll
        for (int x = key; x < GROUP_ROWS * PER; x += 128) {
          const int r = x / PER, c = x % PER;
          if (r < nr) reinterpret_cast<uint4*>(out + (r * 4 + mt) * LINE)[c] = reinterpret_cast<const uint4*>(buf + r * 128)[c];
        }
        if (NT > 0) tmem_wait_ld();
#pragma unroll
        for (int r = 0; r < 16; ++r) o[r] = ahead[r];
      }
    };
    if (nr <= 0) {
      // no rows of this group
    } else if (!direct) write(__half(), [](float v) { return __float2half_rn(v); }, a.part_o);
    else if (a.out_f32) write(float(), [](float v) { return v; }, a.o);
    else write(__nv_bfloat16(), [](float v) { return __float2bfloat16_rn(v); }, a.o);
    tc_fence_before();
  }
  __syncthreads();
  if (warp == MMA_WARP) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_verify8_tc(const Verify8Args& a, const VerifyPlan& p, cudaStream_t stream) {
  cudaError_t e = allow_smem<verify8_tc_kernel>(SMEM_BYTES);
  if (e != cudaSuccess) return e;
  // a programmatic dependent: it waits itself, before its first read
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.n_items);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify8_tc_kernel, a, p);
}

}  // namespace kdv
