// k_paged.cu -- the paged latent cache: rows appended with their position's rotation
// (paged_append_kernel), and dense attention of one new token per query over a sequence's
// pages (paged_attn_kernel, paged_join_kernel).
//
// A cache row is one 512-d latent, key and value of every head.  Pages hold page_rows rows;
// table[b][j / page_rows] is the page of row j of sequence b.
#include <cuda_fp8.h>

#include "common.cuh"
#include "compress_dev.cuh"

CSA2_DEFINE_FAULT_FLAG(paged)

namespace csa2 {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// ================================ append ================================================
//
// A warp per token, kTok tokens at a time: a lane holds the 16-byte chunks `lane` (dims 8 l ..)
// and, below lane 24, 32 + lane (dims 256 + 8 l ..) of the row, and one rotation pair each: dims
// 448 + 2 l, 449 + 2 l, so the 32 angles of a row take one sine and cosine per lane.  bf16 rows
// outside the rotated dims are copied as they are.  Bound by the bytes moved: 1024 read, 1024
// or 528 written per token.  The lanes' angular steps (64-bit floating point, of which an SM does
// two a cycle) are computed once per warp, so many tokens run on a grid that stays (kTok = 4,
// whose rows load together); few tokens take a warp each (kTok = 1).  Measured: 57.7 us for
// four bf16 prompts of 16384 to 65535 tokens (86 % of the copy rate), 5 us for 4096 FP8_E8M0
// tokens, 3 us for 64 tokens.

constexpr int kAppWarps = 8;
constexpr int kAppCtas = 6;  // CTAs of an SM with many tokens (three at a time, by registers)

// E4M3 codes of v over scale s, as products with r = 1 / s: within 2^-23 of the quotients, against
// the 2^-4 of a code, and equal to them when s is a power of two.  (Eighteen divisions a lane
// took longer than the row's bytes.)  A scale below 2^-126, whose reciprocal may overflow,
// divides.
__device__ __forceinline__ uint32_t codes2(float x, float y, float s, float r) {
  return s >= 1.1754944e-38f ? cvt_e4m3x2(x * r, y * r) : cvt_e4m3x2(x / s, y / s);
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float s, float r) {
  uint32_t c[4];
  if (s >= 1.1754944e-38f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = cvt_e4m3x2(v[2 * i] * r, v[2 * i + 1] * r);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = cvt_e4m3x2(v[2 * i] / s, v[2 * i + 1] / s);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The smallest exponent byte e in [0, 254] with top <= 448 * 2^(e - 127); 127 for zero.
__device__ __forceinline__ uint32_t e8m0_of(float top) {
  if (!(top > 0.f)) return 127u;
  // top = m 2^x with m in [1, 2): 448 = 1.75 * 2^8, so e - 127 = x - 8, one more when m > 1.75.
  // Values below 2^-118 need no exact x: e is clamped to 0 there.
  const uint32_t u = __float_as_uint(top);
  const int x = (int)(u >> 23) - 127;
  const int e = x - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0) + 127;
  return (uint32_t)min(max(e, 0), 254);
}
__device__ __forceinline__ float e8m0_value(uint32_t e) {
  return e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23);
}

__device__ __forceinline__ float top8(const float (&v)[8]) {
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) t = fmaxf(t, fabsf(v[i]));
  return t;
}
// Maximum over aligned groups of `n` lanes.
template <int N>
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Stores token row (c0, c1: chunks; pr: rotation pair) as row j of sequence b.
__device__ __forceinline__ void append_row(const PagedAppendArgs& a, uint4 c0, uint4 c1, uint32_t pr,
                                           int b, int64_t j, uint64_t turn, int lane) {
  int32_t page = -1, row = 0;
  if (j >= 0 && j < a.cap_rows) {
    const int32_t lp = (int32_t)(__umulhi((uint32_t)j, a.page_mul) >> a.page_shift);
    row = (int32_t)j - lp * a.cache.page_rows;
    page = a.cache.table[(int64_t)b * a.cache.table_ld + lp];
  }
  if (page < 0 || page >= a.cache.n_pages) {
    if (lane == 0) raise_fault(kFaultBounds);
    return;
  }
  uint8_t* dst = a.cache.data + (int64_t)page * a.cache.page_stride +
                 (int64_t)row * (a.cache.dtype == 0 ? 1024 : 528);
  float x0 = __uint_as_float(pr << 16), x1 = __uint_as_float(pr & 0xFFFF0000u);
  if (a.inv_freq) {
    float s, c;
    sincosf(rope_angle(turn, (uint64_t)j * (uint64_t)a.ratio), &s, &c);
    const float y0 = x0 * c - x1 * s;
    x1 = x0 * s + x1 * c;
    x0 = y0;
  }
  if (a.cache.dtype == 0) {
    *(reinterpret_cast<uint4*>(dst) + lane) = c0;
    if (lane < 24) *(reinterpret_cast<uint4*>(dst) + 32 + lane) = c1;
    *(reinterpret_cast<uint32_t*>(dst + 2 * kRopeDim0) + lane) = pack_bf16x2(x0, x1);
    return;
  }
  float v0[8], v1[8];
  unpack8(c0, v0);
  unpack8(c1, v1);
  const float tr = fmaxf(fabsf(x0), fabsf(x1));
  float s0, s1, sr, r0, r1, rr;  // scales, reciprocals
  if (a.cache.dtype == 1) {
    // groups of 128 dims: 16 lanes of a chunk; the last one is lanes 16..23's second chunks
    // and all 32 pairs
    const float m0 = lanes_max<16>(top8(v0)), m1 = lanes_max<16>(top8(v1));
    const float m3 = fmaxf(__shfl_sync(0xFFFFFFFFu, m1, 16), lanes_max<32>(tr));
    s0 = m0 > 0.f ? m0 / 448.f : 1.f;
    s1 = lane < 16 ? m1 : m3;
    s1 = s1 > 0.f ? s1 / 448.f : 1.f;
    sr = m3 > 0.f ? m3 / 448.f : 1.f;
    float* sc = reinterpret_cast<float*>(dst + 512);
    if ((lane & 15) == 0) {
      sc[lane >> 4] = s0;
      sc[2 + (lane >> 4)] = s1;
    }
    r0 = 1.f / s0;
    r1 = 1.f / s1;
    rr = 1.f / sr;
  } else {
    // groups of 32 dims: four lanes of a chunk, 16 lanes' pairs
    const uint32_t e0 = e8m0_of(lanes_max<4>(top8(v0))), e1 = e8m0_of(lanes_max<4>(top8(v1)));
    const uint32_t er = e8m0_of(lanes_max<16>(tr));
    s0 = s1 = sr = 1.f;
    r0 = e8m0_value(254u - e0);  // 2^(127 - e)
    r1 = e8m0_value(254u - e1);
    rr = e8m0_value(254u - er);
    uint8_t* sc = dst + 512;
    if ((lane & 3) == 0) {
      sc[lane >> 2] = (uint8_t)e0;
      if (lane < 24) sc[8 + (lane >> 2)] = (uint8_t)e1;
    }
    if ((lane & 15) == 0) sc[14 + (lane >> 4)] = (uint8_t)er;
  }
  *(reinterpret_cast<uint2*>(dst) + lane) = codes8(v0, s0, r0);
  if (lane < 24) *(reinterpret_cast<uint2*>(dst + 256) + lane) = codes8(v1, s1, r1);
  *(reinterpret_cast<uint16_t*>(dst + kRopeDim0) + lane) = (uint16_t)codes2(x0, x1, sr, rr);
}

template <int kTok>
__global__ void __launch_bounds__(kAppWarps * 32) paged_append_kernel(PagedAppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * kAppWarps * kTok;
  const uint64_t turn = a.inv_freq ? rope_turn(a.inv_freq[lane]) : 0;
  for (int64_t t = ((int64_t)blockIdx.x * kAppWarps + (threadIdx.x >> 5)) * kTok; t < a.T; t += step) {
    uint4 c0[kTok], c1[kTok];
    uint32_t pr[kTok];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      c1[i] = make_uint4(0u, 0u, 0u, 0u);
      if (t + i < a.T) {
        const uint16_t* src = a.kv + (t + i) * a.kv_ld;
        c0[i] = __ldcs(reinterpret_cast<const uint4*>(src) + lane);
        if (lane < 24) c1[i] = __ldcs(reinterpret_cast<const uint4*>(src) + 32 + lane);
        pr[i] = __ldcs(reinterpret_cast<const uint32_t*>(src + kRopeDim0) + lane);
      }
    }
    int b = cdev::warp_find_seq(a.cu_seqlens, a.cache.B, t, lane);
    int64_t t0 = a.cu_seqlens[b], t1 = a.cu_seqlens[b + 1], first = a.start_row[b];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      if (t + i >= a.T) break;
      if (i > 0 && t + i >= t1) {  // on to the token's sequence
        b = cdev::warp_find_seq(a.cu_seqlens, a.cache.B, t + i, lane);
        t0 = a.cu_seqlens[b];
        t1 = a.cu_seqlens[b + 1];
        first = a.start_row[b];
      }
      // a token behind the last sequence is padding
      if (t + i >= t0 && t + i < t1)
        append_row(a, c0[i], c1[i], pr[i], b, first + (t + i - t0), turn, lane);
    }
  }
}

// ================================ attention =============================================
//
// An item is a query and up to 64 of its heads; its visible rows lo .. hi - 1 form tiles of
// 64 rows (tile boundaries at multiples of 64), and `ut` tiles a unit.  The units of all
// items, in order, are dealt evenly to the CTAs (one per SM), so a CTA works on a run of
// tiles of one item (a segment), then of the next: batches of unequal lengths and single
// long sequences alike keep every SM busy.  An item that lies within one CTA is finished
// there; of the others each CTA writes its part (O^T unscaled, running maximum and sums, in
// fp32) to the workspace and paged_join_kernel joins them.
//
// A small call (kDirect, see paged_cluster) deals a.cluster CTAs to each item instead, one or a
// cluster that shares the item's tiles and joins in distributed shared memory: no plan over
// all items, one launch, no workspace.
//
// A tile passes through a ring of 16 KiB slots, each a quarter of it (64 rows x 128 dims, as
// eight groups of 8 rows, two 128-byte-swizzled blocks of 64 dims each):
//   load     warps 12..15, a quarter each: one tensor copy per page piece (bf16 rows), or
//            warps 12..27, which load FP8 rows into registers a tile ahead and store them as
//            bf16.  A tensor copy takes its warp 50 to 100 cycles to issue, so one warp alone
//            held the tile rate to 3200 cycles (a tile of HBM time per SM is 2800)
//   S        warp 8: Q[64 x 512] . X^T, a quarter as it lands; head h in TMEM lane
//            32 (h / 16) + h % 16, column = row
//   softmax  warps 0..7, half of the rows each four: P = 2^(s - m) with the running maximum m,
//            which moves only when a score exceeds it by more than 2^64 (P <= 2^64 keeps bf16
//            P and fp32 sums finite), so a tile's usual pass needs no maximum across threads,
//            one vote only
//   O^T     += X^T[512 x 64] . P^T: warp 9, four M = 128 tiles of dims, each releasing its
//            slot, so the quarter of a later tile starts to load while this one is finished
// Rows outside lo .. hi - 1 or on a bad page get P = 0 and are zeroed before the product
// (what the page holds there may be NaN).
//
// Measured, 64 heads: 16 sequences of 262144 rows 664 us in bf16 (95 % of the copy rate), 964 us
// as FP8_S128, 853 us as FP8_E8M0; 64 sequences of 8192 to 32768 rows 234 us in bf16, 343 us as
// FP8_S128.  bf16 rows are bound by HBM.  FP8 rows are bound by the data pipe of L1 and shared
// memory (78 % busy: a tile takes 1780 cycles of operand reads, 1010 of row loads, 890 of
// stores, 650 of loads and waits) and by what waits for it: a slot's way round the ring.
//
// The sum of P exists twice: of the bf16-rounded values, which the output is divided by (a
// common rounding error of the largest weights cancels), and of the unrounded ones for lse.

constexpr int kSlotBytes = 16384;
constexpr int kBlock = 1024;  // 64 dims of 8 rows
constexpr int kGroup = 2048;  // 128 dims of 8 rows
constexpr int kMaxSmem = 232448;
constexpr float kLazy = 64.0f;
// Most tiles that O^T sums up, a power of two.  The tensor core cuts the low bits of its running
// sums instead of rounding them, so sums of one sign come out short by some 2^-24 of themselves per
// product of 16 rows: 0.04 % after 65536 rows, a tenth of the output's own rounding, but 0.6 % after
// a million.  A longer segment is done in runs, whose parts are added up in fp32.
constexpr int kRunTiles = 1024;
constexpr float kLowSink = -1048576.0f;  // from here on fp32's steps are 1/8 and less
constexpr uint32_t kColO = 256;  // O^T tiles at 256 + 64 mt

// What lives in P's buffers while they hold no P: from the end of a tile's products to the next
// tile's weights, and in a segment's end.
struct __align__(16) PagedSpare {
  float top[2][64];     // largest score above the running maximum, by part of the rows
  float lsum[2][64], rsum[2][64];  // sums of P by part: unrounded, rounded
  float m_run[64], sink2[64];
};
static_assert(sizeof(PagedSpare) <= 8192, "it shares P's memory");

struct __align__(16) PagedAux {
  uint64_t full[12], empty[12];  // ring slots
  uint64_t landed[12];           // FP8 rows: written by the loaders, not yet fenced
  uint64_t q_full, q_empty;
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[2], pv_done;  // p_full: [1] with FP8_S128 rows only
  uint64_t fin[2];
  uint64_t mask[4];     // valid rows of tile c at c & 3
  int it0, it0_unit;    // first item of this CTA and the units before it within the item
  __align__(16) float fac[64];  // rescale factor or 1 / sum, per head
  float rope_c[32], rope_s[32];
  uint32_t tmem_slot;
  int abort;
};

// kMode 0: bf16 rows; 1: FP8_S128 (fp32 scales stay outside the products: one accumulator
// and one P per 128 dims); 2: FP8_E8M0 (a power of two times a code is exact in bf16 for scale
// bytes from 3 on; below, values under 2^-127 may lose their last bits).
template <int kHp, int kMode>
struct PagedCfg {
  static constexpr bool kScaled = kMode == 1;
  // softmax warps: kParts of four, each with 64 / kParts rows of a tile
  static constexpr int kParts = 2;
  static constexpr int kSoft = 128 * kParts;         // softmax threads
  static constexpr int kWarpS = 4 * kParts;          // a warp issues S,
  static constexpr int kWarpO = kWarpS + 1;          // one O^T, one loads Q,
  static constexpr int kWarpQ = kWarpS + 2;
  static constexpr int kWarpF = kWarpS + 3;          // one fences FP8 rows (spare with bf16),
  static constexpr int kWarpL = kWarpS + 4;          // the others load rows
  static constexpr int kLoadWarps = kMode == 0 ? 4 : 16;
  static constexpr int kThreads = 32 * (kWarpL + kLoadWarps);
  static constexpr int kQBlock = kHp * 128;
  static constexpr int kQBytes = 8 * kQBlock;
  static constexpr int kPBufs = kScaled ? 4 : 1;  // scaled rows have a P per quarter
  // P's memory also stages the output: a KiB for each softmax warp
  static constexpr int kPUsed = kHp * 128 * kPBufs;
  static constexpr int kPBytes = kPUsed > 8192 ? kPUsed : 8192;
  // scales [tile][quarter][row] of the last kScTiles tiles, the eight rows of a softmax thread
  // side by side (row bits 5, 2..1, 4..3, 0): a tile's are written with its last quarter, whose
  // slot with eight slots was the last quarter's two tiles before
  static constexpr int kScTiles = kHp == 64 ? 2 : 4;
  static constexpr int kScBytes = kScaled ? kScTiles * 4 * 64 * 4 : 0;
  static constexpr int kFree =
      (kMaxSmem - kQBytes - kPBytes - kScBytes - (int)sizeof(PagedAux)) / kSlotBytes;
  static constexpr int kSlots = kFree < 12 ? kFree : 12;
  static_assert(!kScaled || kScTiles == 4 || kSlots <= 8, "scales are overwritten too early");
  static constexpr int kSmem =
      kQBytes + kSlots * kSlotBytes + kPBytes + kScBytes + (int)sizeof(PagedAux);
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Wait for a phase; false once something in the CTA has given up.  The flag is read only while
// the phase is incomplete: a read of shared memory takes some hundred cycles while the tensor
// core's operand reads fill it, and the waits stand on the path from scores to values.
__device__ __forceinline__ bool wait_phase(PagedAux& X, uint64_t& bar, uint32_t parity,
                                           uint64_t limit_ns = 2000000000ull) {
  const uint32_t b = smem_u32(&bar);
  if (mbar_try_wait(b, parity)) return true;
  const volatile int* abort = &X.abort;
  if (*abort) return false;
  if (mbar_wait(b, parity, limit_ns)) return true;
  X.abort = 1;
  return false;
}

// One lane of the warp, and values that the compiler may take to be the same in all of it.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r));
  return r;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }
__device__ __forceinline__ bool all_ok(bool x) { return __all_sync(0xFFFFFFFFu, x); }

// Four 8 x 8 matrices of 16-bit values: thread t holds (t / 4, 2 (t % 4) + {0, 1}) of each; lane
// 8 i + r gives the address of row r of matrix i.  (No memory clobber: what it writes is read
// after a fence and a barrier, which have one, and loads of scales may move past it.)
__device__ __forceinline__ void store_matrices(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]));
}

// The same, each matrix transposed: lane 8 i + r gives the address of column r of matrix i.
__device__ __forceinline__ void store_matrices_t(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

template <int kSoft>
__device__ __forceinline__ void soft_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoft) : "memory");
}
template <int kSoft>
__device__ __forceinline__ bool soft_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.or.pred po, 1, %2, pi;\n\tselp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "n"(kSoft)
      : "memory");
  return r != 0;
}

// Two fp32 lanes at once: a * b + c and a + b.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// 16 TMEM lanes x 32 columns: thread t receives lanes t / 4 and t / 4 + 8 of columns
// 8 i + 2 (t % 4) + {0, 1} at r[4 i ..] (as tmem_ld_16x256b, four times).
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// The same, two times 8 columns.
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// A box of a page's rows from group y of 8 rows on, dim blocks db and db + 1 (of 64), page z.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int32_t db,
                                            int32_t y, int32_t z, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(db), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}

// What an item sees: rows lo .. hi - 1 of sequence seq in `tiles` tiles from tile0, `units`
// units (0: a padded query, or one whose sequence is outside the table).
struct Item {
  int64_t q;
  int hg;     // head group
  int seq;
  int lo, hi;
  int tile0, tiles, units;
};

__device__ __forceinline__ Item load_item(const PagedAttnArgs& a, int64_t it, bool report) {
  Item i;
  i.q = a.ng == 2 ? it >> 1 : it;
  i.hg = a.ng == 2 ? (int)(it & 1) : 0;
  i.seq = a.q_seq[i.q];
  const int64_t p = a.q_pos[i.q];
  i.lo = i.hi = i.tile0 = 0;
  i.tiles = i.units = 0;
  if (i.seq < 0 || i.seq >= a.cache.B) {
    if (report && i.seq != -1) raise_fault(kFaultBounds);
    return i;
  }
  int64_t hi;  // (p + 1) / ratio
  if (p < 0) hi = 0;
  else if (p < 0x7FFFFFFF) hi = (uint32_t)(p + 1) / (uint32_t)a.ratio;
  else hi = (int64_t)min(((uint64_t)p + 1) / (uint64_t)a.ratio, (uint64_t)1 << 62);
  int64_t lo = a.window > 0 && hi > a.window ? hi - a.window : 0;
  if (hi > a.cap_rows) {
    if (report) raise_fault(kFaultBounds);
    hi = a.cap_rows;
    lo = lo < hi ? lo : hi;
  }
  i.lo = (int)lo;
  i.hi = (int)hi;
  i.tile0 = i.lo >> 6;
  // an empty item is one masked tile, which writes its zeros
  i.tiles = i.hi > i.lo ? ((i.hi + 63) >> 6) - i.tile0 : 1;
  i.units = (i.tiles + a.ut - 1) / a.ut;
  return i;
}

// j / page_rows for j < 2^31.
__device__ __forceinline__ int32_t page_of(const PagedAttnArgs& a, uint32_t j) {
  return (int32_t)(__umulhi(j, a.page_mul) >> a.page_shift);
}

// A CTA's walk over its segments: item it, tiles t .. t_end - 1 of it.
struct Walk {
  int it;          // item
  int64_t left;    // units of this CTA from this segment on
  int unit;        // unit within the item where the segment begins
  Item i;
  int t, t_end;    // tiles of the segment, relative to i.tile0
  int seg_units;
};
__device__ __forceinline__ void walk_fit(const PagedAttnArgs& a, Walk& w) {
  const int rest = w.i.units - w.unit;
  w.seg_units = rest < w.left ? rest : (int)w.left;
  w.t = w.unit * a.ut;
  const int e = (w.unit + w.seg_units) * a.ut;
  w.t_end = e < w.i.tiles ? e : w.i.tiles;
}
__device__ __forceinline__ void walk_start(const PagedAttnArgs& a, const PagedAux& X, int64_t left,
                                           Walk& w) {
  w.it = X.it0;
  w.unit = X.it0_unit;
  w.left = left;
  w.i = load_item(a, w.it, false);
  walk_fit(a, w);
}
// The next segment; false when the CTA is done.
__device__ __forceinline__ bool walk_next(const PagedAttnArgs& a, Walk& w) {
  w.left -= w.seg_units;
  if (w.left <= 0) return false;
  w.unit = 0;
  do {
    if (++w.it >= a.Q * a.ng) return false;
    w.i = load_item(a, w.it, false);
  } while (w.i.units == 0);
  walk_fit(a, w);
  return true;
}

// Four heads of a pair of dims: (x, y) += w * (part's two dims).
__device__ __forceinline__ void join_add(float (&acc)[8], const float4& x, const float4& y,
                                         const float4& w) {
  acc[0] = fmaf(x.x, w.x, acc[0]);
  acc[1] = fmaf(x.y, w.y, acc[1]);
  acc[2] = fmaf(x.z, w.z, acc[2]);
  acc[3] = fmaf(x.w, w.w, acc[3]);
  acc[4] = fmaf(y.x, w.x, acc[4]);
  acc[5] = fmaf(y.y, w.y, acc[5]);
  acc[6] = fmaf(y.z, w.z, acc[6]);
  acc[7] = fmaf(y.w, w.w, acc[7]);
}

// A 32-bit store into shared memory of a CTA of the cluster.
__device__ __forceinline__ void st_cluster32(uint32_t dst, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(dst), "r"(v) : "memory");
}

// ln Z of sums l (of rows and sink) under the maximum M; the sink itself where the rows' sum is 0.
__device__ __forceinline__ float head_lse(float M, float l, float rows, float sink) {
  return rows == 0.f ? sink : (M + __log2f(l)) * kLn2;
}

// A head's running maximum and sums over the parts of the softmax warps.
struct HeadSums {
  float m, l, r;  // maximum; sums of P, unrounded and rounded
};
template <int kParts>
__device__ __forceinline__ HeadSums head_sums(const PagedSpare& Y, int h) {
  HeadSums s = {Y.m_run[h], Y.lsum[0][h], Y.rsum[0][h]};
#pragma unroll
  for (int i = 1; i < kParts; ++i) {
    s.l += Y.lsum[i][h];
    s.r += Y.rsum[i][h];
  }
  return s;
}
// Adds the sink's mass, stores lse and leaves 2^(m - M) / Z in X.fac, M the larger of m and sink
// (log2).
__device__ __forceinline__ void finish_head(const PagedAttnArgs& a, PagedAux& X, HeadSums s,
                                            float sink, int h, const Item& i) {
  // (the sink is above the rows' maximum only where that did not start at it)
  const float M = fmaxf(s.m, sink), Mf = M == -INFINITY ? 0.f : M, w = ex2(s.m - Mf);
  const float rows = s.l *= w;
  s.r *= w;
  if (sink > -INFINITY) {
    s.l += ex2(sink - Mf);
    s.r += ex2(sink - Mf);
  }
  X.fac[h] = s.r > 0.f || s.r != s.r ? w / s.r : 0.f;  // no row and no sink: zeros
  if (a.lse) {
    const int hq = 64 * i.hg + h;
    a.lse[i.q * a.H + hq] = head_lse(Mf, s.l, rows, a.sink ? a.sink[hq] : -INFINITY);
  }
}

// Adds the part of an item's earlier runs (po: this lane's place in it, st: this thread's head's m,
// l, r) to the run in TMEM and Y, both under the larger maximum; the sum goes to both places.
template <int kHp, int kSoft, int kParts>
__device__ __forceinline__ void fold_run(float* po, float* st, PagedAux& X, PagedSpare& Y, uint32_t tq,
                                      int half, int Hg, int tid) {
  if (tid < Hg) {
    const HeadSums h = head_sums<kParts>(Y, tid);
    const float M = fmaxf(st[0], h.m), Mf = M == -INFINITY ? 0.f : M;
    const float f0 = ex2(st[0] - Mf), f1 = ex2(h.m - Mf);
    Y.top[0][tid] = f0;
    X.fac[tid] = f1;
    st[0] = M;
    st[kHp] = h.l * f1 + st[kHp] * f0;
    st[2 * kHp] = h.r * f1 + st[2 * kHp] * f0;
  }
  soft_sync<kSoft>();
#pragma unroll 1
  for (int mt = half; mt < 4; mt += kParts) {
#pragma unroll 1
    for (int hb = 0; hb < Hg; hb += 16) {
      uint32_t v[16];
      tmem_ld16(tq + kColO + 64 * mt + hb, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        float4* to = reinterpret_cast<float4*>(po + (mt * (kHp / 4) + ((hb + j) >> 2)) * 512);
        const float4 f0 = *reinterpret_cast<const float4*>(&Y.top[0][hb + j]);
        const float4 f1 = *reinterpret_cast<const float4*>(&X.fac[hb + j]);
        float4 x = *to;
        x.x = x.x * f0.x + __uint_as_float(v[j]) * f1.x;
        x.y = x.y * f0.y + __uint_as_float(v[j + 1]) * f1.y;
        x.z = x.z * f0.z + __uint_as_float(v[j + 2]) * f1.z;
        x.w = x.w * f0.w + __uint_as_float(v[j + 3]) * f1.w;
        *to = x;
        v[j] = __float_as_uint(x.x);
        v[j + 1] = __float_as_uint(x.y);
        v[j + 2] = __float_as_uint(x.z);
        v[j + 3] = __float_as_uint(x.w);
      }
      tmem_st16(tq + kColO + 64 * mt + hb, v);
    }
  }
  tmem_st_wait();
  soft_sync<kSoft>();  // the factors are read
}

// The same as a call: rare as it is, inline it costs the loop over the tiles registers.  Inline / as
// a call, us: 64 bf16 sequences of 8192 to 32768 rows 234.6 / 233.8, 200 short ones with 16 heads
// 152.6 / 151.8, FP8_E8M0 rows of eight sequences with four tokens each 105.8 / 102.6; but FP8_S128
// rows of the 64 sequences 343 / 358.
template <int kHp, int kSoft, int kParts>
__device__ __noinline__ void call_fold_run(float* po, float* st, PagedAux& X, PagedSpare& Y,
                                           uint32_t tq, int half, int Hg, int tid) {
  fold_run<kHp, kSoft, kParts>(po, st, X, Y, tq, half, Hg, tid);
}

// Dims 128 mt + 32 quad .. + 31 of all heads by one warp: O^T from TMEM (lane = dim) times 1 / Z
// and rotated back, in bf16 through a KiB of shared memory at `stage` ([16 heads][32 dims],
// written as transposed 8 x 8 matrices; 16-byte chunk i of head h at i ^ (h / 2 % 4), free of bank
// conflicts).  Stores of single values from a lane per dim took twice as long.
__device__ __forceinline__ void store_tile(const PagedAttnArgs& a, const PagedAux& X, uint32_t tq,
                                           int mt, int quad, int lane, int Hg, uint32_t stage,
                                           uint16_t* out) {
  const int d0 = mt * 128 + quad * 32, r4 = lane & 3;
  const bool rot = a.inv_freq && d0 >= kRopeDim0;  // the same in a warp
  // this thread's dims: d0 + 8 i + lane / 4, i < 4; of a pair (2 k, 2 k + 1) the other is lane ^ 4
  float cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
    if (rot) {
      const int k = ((d0 - kRopeDim0) >> 1) + 4 * i + (lane >> 3);
      cs[i] = X.rope_c[k];
      sn[i] = (lane & 4) ? -X.rope_s[k] : X.rope_s[k];
    }
  }
  const uint32_t swz = (uint32_t)(lane & 7) * 64 + ((uint32_t)((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
  const uint32_t rd = stage + (uint32_t)(lane >> 2) * 64 + ((uint32_t)(r4 ^ (lane >> 3)) << 4);
#pragma unroll 1
  for (int hb = 0; hb < Hg; hb += 16) {
    uint32_t v[2][8];
    tmem_ld_16x256b_x2(tq + kColO + 64 * mt + hb, v[0]);
    tmem_ld_16x256b_x2(tq + (16u << 16) + kColO + 64 * mt + hb, v[1]);
    tmem_ld_wait();
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float2 f = *reinterpret_cast<const float2*>(&X.fac[hb + 8 * g + 2 * r4]);
      uint32_t m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x = __uint_as_float(v[i >> 1][4 * g + 2 * (i & 1)]) * f.x;
        float y = __uint_as_float(v[i >> 1][4 * g + 2 * (i & 1) + 1]) * f.y;
        if (rot) {  // pair (2k, 2k + 1) times e^{-i p theta_k}
          x = x * cs[i] + __shfl_xor_sync(0xFFFFFFFFu, x, 4) * sn[i];
          y = y * cs[i] + __shfl_xor_sync(0xFFFFFFFFu, y, 4) * sn[i];
        }
        m[i] = pack_bf16x2(x, y);
      }
      store_matrices_t(stage + g * 512 + swz, m);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int h = hb + 8 * i + (lane >> 2);
      const uint4 x = ld_shared16(rd + i * 512);
      if (h < Hg)
        __stcs(reinterpret_cast<uint4*>(out + h * kDLat + mt * 128 + quad * 32) + (lane & 3), x);
    }
    __syncwarp();
  }
}

// Valid rows of the 64-row tile that begins at row r0, as bits.
__device__ __forceinline__ uint64_t tile_mask(int64_t r0, int lo, int hi) {
  const int64_t f = lo - r0, l = hi - r0;  // first valid, end
  uint64_t m = l >= 64 ? ~0ull : l <= 0 ? 0ull : (1ull << l) - 1;
  if (f >= 64) m = 0;
  else if (f > 0) m &= ~0ull << f;
  return m;
}

template <int kHp, int kMode, bool kDirect>
__global__ void __launch_bounds__(PagedCfg<kHp, kMode>::kThreads, 1)
    paged_attn_kernel(PagedAttnArgs a, const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap) {
  using C = PagedCfg<kHp, kMode>;
  constexpr int NS = C::kSlots;
  // no static shared memory in this kernel: the dynamic part begins at a 1024-byte boundary,
  // as the swizzled tiles need (checked below)
  extern __shared__ __align__(1024) uint8_t smem[];
  // Q first: the S products read 64 rows of each Q block, with fewer heads past the block
  // (into what follows it; those TMEM lanes are never used)
  const uint32_t q_s = smem_u32(smem), ring = q_s + C::kQBytes, p_s = ring + NS * kSlotBytes;
  float* sc_s = reinterpret_cast<float*>(smem + C::kQBytes + NS * kSlotBytes + C::kPBytes);
  PagedAux& X = *reinterpret_cast<PagedAux*>(reinterpret_cast<uint8_t*>(sc_s) + C::kScBytes);
  PagedSpare& Y = *reinterpret_cast<PagedSpare*>(smem + C::kQBytes + NS * kSlotBytes);
  // the warp index as a value that the compiler knows to be the same in the whole warp
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;

  griddep_launch_dependents();
  if ((smem_u32(smem) & 1023u) != 0) {  // the same in every thread
    griddep_wait();
    if (tid == 0) raise_fault(kFaultBounds);
    return;
  }
  if (tid == 0) {
    prefetch_tensormap(&qmap);
    if (kMode == 0) prefetch_tensormap(&kmap);
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&X.full[s]), 1);
      mbar_init(smem_u32(&X.landed[s]), 8);
      mbar_init(smem_u32(&X.empty[s]), 1);
    }
    mbar_init(smem_u32(&X.q_full), 1);
    mbar_init(smem_u32(&X.q_empty), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&X.s_full[b]), 2);
      mbar_init(smem_u32(&X.s_empty[b]), C::kWarpS);
    }
    for (int b = 0; b < 2; ++b) mbar_init(smem_u32(&X.fin[b]), 1);
    for (int k = 0; k < 2; ++k) mbar_init(smem_u32(&X.p_full[k]), C::kWarpS);
    mbar_init(smem_u32(&X.pv_done), 1);
    X.abort = 0;
    mbar_fence_init();
  }
  if (warp == C::kWarpS) {
    tmem_alloc(smem_u32(&X.tmem_slot), 512);
    tmem_relinquish();
  }
  // Every thread waits here: queries, positions, page ids and rows may come from the kernel
  // before this one, and the output and the workspace may still be in use by it.  The waits
  // below, which are bounded, then time this kernel's work alone.
  griddep_wait();
  // ---- the plan: every CTA sums the units of all items and finds its share of them ----
  int64_t u0, u1, U = 0;
  int64_t ncta = 1;
  const int cl = kDirect ? a.cluster : 1, crank = kDirect && cl > 1 ? (int)cluster_ctarank() : 0;
  if (kDirect) {
    const int it = blockIdx.x / cl;
    const int tiles = load_item(a, it, crank == 0 && tid == 0).units;
    u0 = (int64_t)tiles * crank / cl;
    u1 = (int64_t)tiles * (crank + 1) / cl;
    if (tid == 0) {
      X.it0 = it;
      X.it0_unit = (int)u0;
    }
  } else {
    const int64_t items = (int64_t)a.Q * a.ng;
    const int64_t per = (items + C::kThreads - 1) / C::kThreads;
    const int64_t i0 = tid * per, i1 = i0 + per < items ? i0 + per : items;
    int64_t s = 0;
    for (int64_t i = i0; i < i1; ++i) s += load_item(a, i, blockIdx.x == 0).units;
    int64_t x = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    int64_t* sums = reinterpret_cast<int64_t*>(smem + C::kQBytes);  // the ring is not in use yet
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < C::kThreads / 32; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    before += x - s;  // units of the items before this thread's
    U = total;
    ncta = (int64_t)gridDim.x < U ? (int64_t)gridDim.x : U;
    const int64_t c = blockIdx.x;
    u0 = c < ncta ? U * c / ncta : 0;
    u1 = c < ncta ? U * (c + 1) / ncta : 0;
    if (u1 > u0 && before <= u0 && u0 < before + s) {  // one thread
      int64_t at = before;
      for (int64_t i = i0; i < i1; ++i) {
        const int n = load_item(a, i, false).units;
        if (u0 < at + n) {
          X.it0 = (int)i;
          X.it0_unit = (int)(u0 - at);
          break;
        }
        at += n;
      }
    }
    fence_proxy_async_smem();  // the scan's sums lie where copies will land
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, X.tmem_slot, 0);

  // the rotation of a small call's output, by a warp that has time, where the CTA stores
  // rotated dims
  if (kDirect && a.inv_freq && warp == C::kWarpF && (crank + 1) * (kDLat / cl) > kRopeDim0) {
    const int64_t it = blockIdx.x / cl, q = a.ng == 2 ? it >> 1 : it;
    float s, c;
    sincosf(rope_angle(rope_turn(a.inv_freq[lane]), (uint64_t)a.q_pos[q]), &s, &c);
    X.rope_c[lane] = c;
    X.rope_s[lane] = s;
  }
  if (u1 > u0) {
    if (warp < C::kWarpS) {
      // ================= softmax, rescale, output =================
      // Warp w holds heads 16 (w % 4) .. + 15 (TMEM lanes 32 (w % 4) ..) and rows kRows (w / 4) ..
      // of a tile; thread t the heads hA = 16 (w % 4) + t / 4 and hB = hA + 8 and of its rows
      // 8 g + 2 (t % 4) + {0, 1}, g < kG.
      constexpr int kParts = C::kParts, kRows = 64 / kParts, kG = kRows / 8;
      const int quad = warp & 3, half = warp >> 2, r4 = lane & 3;
      const int hA = 16 * quad + (lane >> 2), hB = hA + 8;
      const bool on = 16 * quad < kHp;  // this warp's 16 heads exist
      const uint32_t lrow = (uint32_t)(quad * 32) << 16;
      const float sc2 = a.scale * kLog2e;
      Walk w;
      walk_start(a, X, u1 - u0, w);
      int c = 0;                       // tiles of this CTA so far
      int sl = 0;                      // ring slot of the tile's first quarter
      uint32_t sph = 0;                // its phase
      int64_t u = u0;                  // unit where the segment begins
      int t0 = w.t;                    // tile where the run begins
      for (;;) {
        const int Hg = min(64, a.H - 64 * w.i.hg);
        float mA = -INFINITY, mB = -INFINITY;
        float2 lA = make_float2(0.f, 0.f), lB = lA, rA = lA, rB = lA;  // unrounded, rounded
        if (a.sink) {
          if (hA < Hg) mA = sink_log2(a.sink[64 * w.i.hg + hA]);
          if (hB < Hg) mB = sink_log2(a.sink[64 * w.i.hg + hB]);
        }
        const bool whole = kDirect ? cl == 1 : w.unit == 0 && w.seg_units == w.i.units;
        const float sinkA = mA, sinkB = mB;
        // A maximum is moved by adding a score's distance to it, which loses the score where the
        // two are far apart: from a sink far below all scores no maximum starts.
        if (mA < kLowSink) mA = -INFINITY;
        if (mB < kLowSink) mB = -INFINITY;
        // what the output needs is computed while the first tile loads
        if (!kDirect && whole && a.inv_freq && warp == C::kWarpS - 1) {
          float s, cs;
          sincosf(rope_angle(rope_turn(a.inv_freq[lane]), (uint64_t)a.q_pos[w.i.q]), &s, &cs);
          X.rope_c[lane] = cs;
          X.rope_s[lane] = s;
        }
        const int t_run = kDirect ? w.t_end : min(t0 + kRunTiles, w.t_end);
        for (int t = t0; t < t_run; ++t, ++c) {
          const int sb = C::kScaled ? 0 : c & 1;
          const uint32_t sphase = C::kScaled ? (uint32_t)c & 1 : (uint32_t)(c >> 1) & 1;
          // P's memory and O^T are free once the previous tile's products are done.  With bf16
          // rows they are before this tile's scores (the loads are the limit), and waiting for
          // them here keeps that wait off the path from scores to values; with FP8 rows the
          // scores come earlier, so the wait stands before the first use.
          auto products_done = [&]() {
            if (c > 0) wait_phase(X, X.pv_done, (uint32_t)(c - 1) & 1);
          };
          if (kMode == 0) products_done();
          // the scores, and with them (the issuers have seen the tile land and arrive here too)
          // the mask and the scales that its loader wrote
          wait_phase(X, X.s_full[sb], sphase);
          tc_fence_after();
          const uint64_t mask = X.mask[c & 3];
          const bool all = mask == ~0ull;
          // bit 8 g: row 8 g + 2 r4 of this part, bit 8 g + 1 the one after it
          const uint32_t mk = (uint32_t)(mask >> (kRows * half + 2 * r4));
          float2 xA[kG], xB[kG];
          if (on) {
            if (!C::kScaled) {
              uint32_t x[4 * kG];
              tmem_ld_16x256b_x4(tmem + lrow + 64 * sb + kRows * half, x);
              tmem_ld_wait();
#pragma unroll
              for (int g = 0; g < kG; ++g) {
                xA[g] = make_float2(__uint_as_float(x[4 * g]), __uint_as_float(x[4 * g + 1]));
                xB[g] = make_float2(__uint_as_float(x[4 * g + 2]), __uint_as_float(x[4 * g + 3]));
              }
            } else {
#pragma unroll
              for (int g = 0; g < kG; ++g) xA[g] = xB[g] = make_float2(0.f, 0.f);
#pragma unroll
              for (int k2 = 0; k2 < 4; k2 += 2) {
                uint32_t x[2][4 * kG];
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  tmem_ld_16x256b_x4(tmem + lrow + 64 * (k2 + k) + kRows * half, x[k]);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const float4* sc = reinterpret_cast<const float4*>(
                      sc_s + ((c & (C::kScTiles - 1)) * 4 + k2 + k) * 64 + kRows * half + 8 * r4);
                  const float4 f4[2] = {sc[0], sc[1]};
#pragma unroll
                  for (int g = 0; g < kG; ++g) {
                    const float2 f = g & 1 ? make_float2(f4[g >> 1].z, f4[g >> 1].w)
                                           : make_float2(f4[g >> 1].x, f4[g >> 1].y);
                    xA[g] = fma2(
                        make_float2(__uint_as_float(x[k][4 * g]), __uint_as_float(x[k][4 * g + 1])), f,
                        xA[g]);
                    xB[g] = fma2(
                        make_float2(__uint_as_float(x[k][4 * g + 2]), __uint_as_float(x[k][4 * g + 3])),
                        f, xB[g]);
                  }
                }
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&X.s_empty[sb]));
          // P = 2^(score - m), m the running maximum (no score yet: 0); the largest exponent
          // met and the sums of P
          uint32_t pa[kG], pb[kG];
          float2 eA[kG], eB[kG];
          float tA, tB;
          float2 sA, sB, uA, uB;
          auto weights = [&]() {
            const float nA = mA == -INFINITY ? 0.f : -mA, nB = mB == -INFINITY ? 0.f : -mB;
            tA = tB = -INFINITY;
            sA = sB = uA = uB = make_float2(0.f, 0.f);
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              float2 y = fma2(xA[g], make_float2(sc2, sc2), make_float2(nA, nA));
              float2 z = fma2(xB[g], make_float2(sc2, sc2), make_float2(nB, nB));
              if (!all) {
                if (!(mk >> (8 * g) & 1u)) y.x = z.x = -INFINITY;
                if (!(mk >> (8 * g + 1) & 1u)) y.y = z.y = -INFINITY;
              }
              tA = fmaxf(tA, fmaxf(y.x, y.y));
              tB = fmaxf(tB, fmaxf(z.x, z.y));
              y = make_float2(ex2(y.x), ex2(y.y));
              z = make_float2(ex2(z.x), ex2(z.y));
              sA = add2(sA, y);
              sB = add2(sB, z);
              if (C::kScaled) {
                eA[g] = y;
                eB[g] = z;
              } else {
                pa[g] = pack_bf16x2(y.x, y.y);
                pb[g] = pack_bf16x2(z.x, z.y);
                uA = add2(uA, make_float2(__uint_as_float(pa[g] << 16),
                                          __uint_as_float(pa[g] & 0xFFFF0000u)));
                uB = add2(uB, make_float2(__uint_as_float(pb[g] << 16),
                                          __uint_as_float(pb[g] & 0xFFFF0000u)));
              }
            }
          };
          for (int pass = 0;; ++pass) {
            bool need = false;
            if (on) {
              weights();
              need = (hA < Hg && (tA > kLazy || (mA == -INFINITY && tA > -INFINITY))) ||
                     (hB < Hg && (tB > kLazy || (mB == -INFINITY && tB > -INFINITY)));
            }
            if (!soft_any<C::kSoft>(need) || pass == 1) break;
            if (kMode != 0) products_done();
            // a head's maximum moves: the largest exponent of its rows in all parts; the weights
            // are taken again
            if (on) {
              tA = fmaxf(tA, __shfl_xor_sync(0xFFFFFFFFu, tA, 1));
              tA = fmaxf(tA, __shfl_xor_sync(0xFFFFFFFFu, tA, 2));
              tB = fmaxf(tB, __shfl_xor_sync(0xFFFFFFFFu, tB, 1));
              tB = fmaxf(tB, __shfl_xor_sync(0xFFFFFFFFu, tB, 2));
              if (r4 == 0) {
                Y.top[half][hA] = tA;
                Y.top[half][hB] = tB;
              }
            }
            soft_sync<C::kSoft>();
            if (on) {
              float fA = 1.f, fB = 1.f;
              tA = Y.top[0][hA];
              tB = Y.top[0][hB];
#pragma unroll
              for (int i = 1; i < kParts; ++i) {
                tA = fmaxf(tA, Y.top[i][hA]);
                tB = fmaxf(tB, Y.top[i][hB]);
              }
              if (tA > kLazy || (mA == -INFINITY && tA > -INFINITY)) {
                fA = mA == -INFINITY ? 0.f : ex2(-tA);
                mA = mA == -INFINITY ? tA : mA + tA;
              }
              if (tB > kLazy || (mB == -INFINITY && tB > -INFINITY)) {
                fB = mB == -INFINITY ? 0.f : ex2(-tB);
                mB = mB == -INFINITY ? tB : mB + tB;
              }
              if (half == 0 && r4 == 0) {
                X.fac[hA] = fA;
                X.fac[hB] = fB;
              }
              const float2 qA = make_float2(fA, fA), qB = make_float2(fB, fB);
              const float2 o0 = make_float2(0.f, 0.f);
              lA = fma2(lA, qA, o0);
              lB = fma2(lB, qB, o0);
              rA = fma2(rA, qA, o0);
              rB = fma2(rB, qB, o0);
            }
            soft_sync<C::kSoft>();  // fac is written, and top read, by all
            if (t > t0) {
              tc_fence_after();
#pragma unroll 1
              for (int mt = half; mt < 4; mt += kParts) {
#pragma unroll 1
                for (int hb = 0; hb < kHp; hb += 16) {
                  uint32_t v[16];
                  const uint32_t ta = tmem + lrow + kColO + 64 * mt + hb;
                  tmem_ld16(ta, v);
                  tmem_ld_wait();
#pragma unroll
                  for (int j = 0; j < 16; ++j)
                    v[j] = __float_as_uint(__uint_as_float(v[j]) * X.fac[hb + j]);
                  tmem_st16(ta, v);
                }
              }
              tmem_st_wait();
            }
            // (the next pass' vote comes after all have read fac: P may then be written over it)
          }
          if (on) {
            lA = add2(lA, sA);
            lB = add2(lB, sB);
            if (!C::kScaled) {
              rA = add2(rA, uA);
              rB = add2(rB, uB);
            }
          }
          if (kMode != 0) products_done();
          if (kMode == 0 && !all) {
            // rows outside the item: whatever the page holds there must not meet P's zeros
            for (int k = 0; k < 4; ++k) {  // the copies themselves, too, are complete
              const int i = sl + k;
              wait_phase(X, X.full[i >= NS ? i - NS : i], i >= NS ? sph ^ 1 : sph);
            }
            const int piece = tid & 63;
            for (int r = tid >> 6; r < 64; r += C::kSoft / 64) {
              if ((mask >> r) & 1) continue;
              int s = sl + (piece >> 4);
              if (s >= NS) s -= NS;
              st_shared16(ring + s * kSlotBytes + (r >> 3) * kGroup + ((piece >> 3) & 1) * kBlock +
                              (r & 7) * 128 + (piece & 7) * 16,
                          make_uint4(0u, 0u, 0u, 0u));
            }
          }
          // P [head][64 rows], 128-byte swizzled: matrix i is this part's rows 8 i .. of eight
          // heads
          static_assert(kG == 4, "a warp's rows are four matrices");
          const uint32_t pA = p_s + (16 * quad + (lane & 7)) * 128 +
                              (((kG * half + (lane >> 3)) ^ (lane & 7)) << 4);
#pragma unroll
          for (int k = 0; k < C::kPBufs; ++k) {
            if (on) {
              if (C::kScaled) {
                const float4* sc = reinterpret_cast<const float4*>(
                    sc_s + ((c & (C::kScTiles - 1)) * 4 + k) * 64 + kRows * half + 8 * r4);
                const float4 f4[2] = {sc[0], sc[1]};
#pragma unroll
                for (int g = 0; g < kG; ++g) {
                  const float2 f = g & 1 ? make_float2(f4[g >> 1].z, f4[g >> 1].w)
                                         : make_float2(f4[g >> 1].x, f4[g >> 1].y);
                  const float2 o0 = make_float2(0.f, 0.f);
                  const float2 x = fma2(eA[g], f, o0), y = fma2(eB[g], f, o0);
                  pa[g] = pack_bf16x2(x.x, x.y);
                  pb[g] = pack_bf16x2(y.x, y.y);
                }
              }
              const uint32_t pk = pA + k * (kHp * 128);
              store_matrices(pk, pa);
              store_matrices(pk + 8 * 128, pb);
            }
          }
          // one fence for all: with FP8_S128 rows two, each for two quarters' P, took 2 % longer
          // (64 sequences of 8192 to 32768 rows)
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&X.p_full[0]));
            if (C::kScaled) mbar_arrive(smem_u32(&X.p_full[1]));
          }
          sl += 4;
          if (sl >= NS) { sl -= NS; sph ^= 1; }
        }
        // ---- the segment's end: sums of each head, then its part or its output ----
        wait_phase(X, X.pv_done, (uint32_t)(c - 1) & 1);
        tc_fence_after();
        if (on) {
          float v[4] = {lA.x + lA.y, lB.x + lB.y, rA.x + rA.y, rB.x + rB.y};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], 1);
            v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], 2);
          }
          if (r4 == 0) {
            Y.lsum[half][hA] = v[0];
            Y.lsum[half][hB] = v[1];
            // with scaled weights no rounded sum stands for the output's weights
            Y.rsum[half][hA] = C::kScaled ? v[0] : v[2];
            Y.rsum[half][hB] = C::kScaled ? v[1] : v[3];
            if (half == 0) {
              Y.m_run[hA] = mA;
              Y.m_run[hB] = mB;
              Y.sink2[hA] = sinkA;
              Y.sink2[hB] = sinkB;
            }
          }
        }
        const int64_t part = 2 * (int64_t)blockIdx.x + (w.unit == 0 ? 1 : 0);
        soft_sync<C::kSoft>();
        if (kDirect) break;  // the output, by more warps, or the cluster's join follows below
        float* st = a.pstat + part * (3 * kHp) + tid;
        // [dim tile][four heads][even dims, odd dims][4]: a lane writes 16 bytes, and the
        // join's threads, which have a pair of dims each, read them side by side
        float* po = a.part + part * (int64_t)(kHp * kDLat) +
                    (((quad * 32 + lane) >> 1) + (lane & 1) * 64) * 4;
        const bool onto = t0 > w.t, last = t_run == w.t_end;  // of the segment's runs
        if (onto) {
          if (C::kScaled)
            fold_run<kHp, C::kSoft, kParts>(po, st, X, Y, tmem + lrow, half, Hg, tid);
          else
            call_fold_run<kHp, C::kSoft, kParts>(po, st, X, Y, tmem + lrow, half, Hg, tid);
        }
        if (tid < Hg) {
          if (whole && last) {
            const HeadSums h =
                onto ? HeadSums{st[0], st[kHp], st[2 * kHp]} : head_sums<kParts>(Y, tid);
            finish_head(a, X, h, Y.sink2[tid], tid, w.i);
          } else if (!onto) {
            const HeadSums h = head_sums<kParts>(Y, tid);
            st[0] = h.m;
            st[kHp] = h.l;
            st[2 * kHp] = h.r;
          }
        }
        if (a.rec && last && w.unit == 0 && tid == 0) {
          // CTAs of the item's first and last unit; (-1, -1): finished here
          const int64_t ul = u + w.i.units - 1;
          a.rec[w.it] = whole ? make_int2(-1, -1)
                             : make_int2((int)blockIdx.x, (int)(((ul + 1) * ncta - 1) / U));
        }
        soft_sync<C::kSoft>();
        if (whole && last) {
          uint16_t* out = a.out + (w.i.q * a.H + 64 * w.i.hg) * kDLat;
          for (int mt = half; mt < 4; mt += kParts)
            store_tile(a, X, tmem + lrow, mt, quad, lane, Hg, p_s + warp * 1024, out);
        } else if (!onto) {
#pragma unroll 1
          for (int mt = half; mt < 4; mt += kParts) {
#pragma unroll 1
            for (int hb = 0; hb < Hg; hb += 16) {
              uint32_t v[16];
              tmem_ld16(tmem + lrow + kColO + 64 * mt + hb, v);
              tmem_ld_wait();
#pragma unroll
              for (int j4 = 0; j4 < 4; ++j4)
                *reinterpret_cast<uint4*>(po + (mt * (kHp / 4) + (hb >> 2) + j4) * 512) =
                    make_uint4(v[4 * j4], v[4 * j4 + 1], v[4 * j4 + 2], v[4 * j4 + 3]);
            }
          }
        }
        tc_fence_before();
        soft_sync<C::kSoft>();  // fac, the sums and the rotation are read before the next segment's
        if (!last) {
          t0 = t_run;
          continue;
        }
        u += w.seg_units;
        if (!walk_next(a, w)) break;
        t0 = w.t;
      }
    } else if (warp == C::kWarpS) {
      // ================= S products =================
      // The whole warp walks the loop and one elected lane issues: with operands the same in
      // the warp an MMA takes 32 cycles (its reads of shared memory), where a lane in a branch
      // of its own took 47 and far more beside busy warps.
      const uint32_t lead = elect_lane();
      Walk w;
      walk_start(a, X, u1 - u0, w);
      int c = 0, sl = 0;
      uint32_t sph = 0, n = 0;  // n: segments so far
      const uint32_t id = idesc_bf16(64, 64, 0, 0);
      const uint64_t q_d = sdesc_sw128(q_s, 16, 1024), r_d = sdesc_sw128(ring, 16, kGroup);
      bool ok = true, next;
      do {
        ok = all_ok(wait_phase(X, X.q_full, n & 1));
        ++n;
        const int tiles = uniform(w.t_end - w.t);
        for (int t = 0; ok && t < tiles; ++t, ++c) {
          const int sb = C::kScaled ? 0 : c & 1;
          const int lag = C::kScaled ? 1 : 2;
          if (c >= lag)
            ok = all_ok(wait_phase(X, X.s_empty[sb], C::kScaled ? (uint32_t)(c - 1) & 1
                                                                : (uint32_t)((c - 2) >> 1) & 1));
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            ok = ok && all_ok(wait_phase(X, X.full[sl], sph));
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + 64 * (C::kScaled ? k : sb);
            const uint64_t rd = r_d + ((uint32_t)(sl * kSlotBytes) >> 4);
            if (lead) {
              // the tile's mask came with its first quarter, the scales with each
              if (k == (C::kScaled ? 3 : 0)) mbar_arrive(smem_u32(&X.s_full[sb]));
#pragma unroll
              for (int i = 0; i < 8; ++i)
                umma_bf16(d, q_d + (((2 * k + (i >> 2)) * C::kQBlock + (i & 3) * 32) >> 4),
                          rd + (((i >> 2) * kBlock + (i & 3) * 32) >> 4), id,
                          i > 0 || (!C::kScaled && k > 0));
              if (k == 3) umma_commit(smem_u32(&X.s_full[sb]));
            }
            __syncwarp();
            if (++sl == NS) { sl = 0; sph ^= 1; }
          }
        }
        if (!ok) break;
        if (lead) umma_commit(smem_u32(&X.q_empty));
        __syncwarp();
        next = uniform(walk_next(a, w)) != 0;
      } while (next);
      // no MMA may still be running when the TMEM is released, whatever happened above
      if (lead) umma_commit(smem_u32(&X.fin[0]));
      __syncwarp();
      mbar_wait(smem_u32(&X.fin[0]), 0, 100000000ull);
    } else if (warp == C::kWarpO) {
      // ================= O^T products =================
      const uint32_t lead = elect_lane();
      Walk w;
      walk_start(a, X, u1 - u0, w);
      int c = 0, sl = 0;
      const uint32_t id = idesc_bf16(128, kHp, 1, 0);
      const uint64_t r_d = sdesc_sw128(ring, kBlock, kGroup), p_d = sdesc_sw128(p_s, 16, 1024);
      bool ok = true, next;
      do {
        const int tiles = uniform(w.t_end - w.t);
        for (int t = 0; ok && t < tiles; ++t, ++c) {
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            // (with FP8_S128 rows a second wait, for what is then there, lets the other issuer's
            // products in between: 3 % less for 64 sequences of 8192 to 32768 rows)
            if (mt == 0 || (C::kScaled && mt == 2)) {
              ok = ok && all_ok(wait_phase(X, X.p_full[mt >> 1], (uint32_t)c & 1));
              if (!ok) break;
              tc_fence_after();
            }
            const uint64_t rd = r_d + ((uint32_t)(sl * kSlotBytes) >> 4);
            const uint64_t pd = p_d + ((uint32_t)((C::kScaled ? mt : 0) * (kHp * 128)) >> 4);
            if (lead) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_bf16(tmem + kColO + 64 * mt, rd + ((kk * 2 * kGroup) >> 4),
                          pd + ((kk * 32) >> 4), id, (t & (kRunTiles - 1)) > 0 || kk > 0);
              umma_commit(smem_u32(&X.empty[sl]));
              if (mt == 3) umma_commit(smem_u32(&X.pv_done));
            }
            __syncwarp();
            if (++sl == NS) sl = 0;
          }
        }
        if (!ok) break;
        next = uniform(walk_next(a, w)) != 0;
      } while (next);
      if (lead) umma_commit(smem_u32(&X.fin[1]));
      __syncwarp();
      mbar_wait(smem_u32(&X.fin[1]), 0, 100000000ull);
    } else if (warp == C::kWarpQ) {
      // ================= Q of each segment =================
      if (lane == 0) {
        Walk w;
        walk_start(a, X, u1 - u0, w);
        const uint64_t pol = policy_evict_first();
        uint32_t n = 0;  // segments so far
        int tiles = 0;   // of the last one
        const uint32_t qf = smem_u32(&X.q_full);
        do {
          // this wait lasts as long as a segment, which may be millions of tiles of some 2 us
          if (n > 0 &&
              !wait_phase(X, X.q_empty, (n - 1) & 1, 2000000000ull + 50000ull * (uint32_t)tiles))
            break;
          tiles = w.t_end - w.t;
          mbar_arrive_expect_tx(qf, C::kQBytes);
#pragma unroll
          for (int db = 0; db < 8; ++db)
            tma_load_2d(q_s + db * C::kQBlock, &qmap, 64 * db, (int32_t)(w.i.q * a.H + 64 * w.i.hg),
                        qf, pol);
          ++n;
        } while (walk_next(a, w));
        mbar_wait(qf, (n - 1) & 1, 100000000ull);  // no copy may land after the CTA's exit
      }
    } else if (warp == C::kWarpF) {
      // ================= FP8 rows: from the threads' writes to the tensor core's reads ========
      // The fence between the two takes hundreds of cycles while the MMAs' reads fill shared
      // memory; a warp of its own takes it off the loaders' and the issuer's way.
      if (kMode != 0) {
        Walk w;
        walk_start(a, X, u1 - u0, w);
        int sl = 0;
        uint32_t ph = 0;
        bool ok = true;
        do {
          for (int i = 4 * (w.t_end - w.t); ok && i > 0; --i) {
            ok = wait_phase(X, X.landed[sl], ph);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&X.full[sl]));
            if (++sl == NS) { sl = 0; ph ^= 1; }
          }
        } while (ok && walk_next(a, w));
      }
    } else if (kMode == 0) {
      // ================= bf16 rows by tensor copies: warp k quarter k =================
      const int k = warp - C::kWarpL;
      Walk w;
      walk_start(a, X, u1 - u0, w);
      const uint64_t pol = a.shared ? policy_evict_normal() : policy_evict_first();
      const int R = a.box_rows, nc = 64 / R;      // page pieces per tile
      const int tb = 32 / nc;                     // tiles whose pieces the lanes look up at once
      const int cl = lane & (nc - 1);             // this lane's piece of a tile
      int sl = k, c = 0;
      uint32_t ph = 0;  // how often the ring has come round, modulo 2
      bool again = false, ok = true;
      do {
        for (int tbeg = w.t; ok && tbeg < w.t_end; tbeg += tb) {
          // piece `lane` of the next tb tiles: its page and row, valid rows
          const int64_t row = ((int64_t)w.i.tile0 + tbeg) * 64 + (int64_t)lane * R;
          int32_t py = 0, pz = (int32_t)a.cache.n_pages;  // beyond the pool: zeros
          uint64_t m = 0;
          if (row < w.i.hi && row + R > w.i.lo && tbeg + lane / nc < w.t_end) {
            const int32_t lp = page_of(a, (uint32_t)row);
            const int32_t page = a.cache.table[(int64_t)w.i.seq * a.cache.table_ld + lp];
            if (page >= 0 && page < a.cache.n_pages) {
              py = ((int32_t)row - lp * a.cache.page_rows) >> 3;
              pz = page;
              m = tile_mask(row, w.i.lo, w.i.hi);
              if (R < 64) m &= (1ull << R) - 1;
            } else if (k == 0) {
              raise_fault(kFaultBounds);
            }
          }
          m <<= cl * R;
          for (int o = 1; o < nc; o <<= 1) m |= __shfl_xor_sync(0xFFFFFFFFu, m, o);
          const int te = min(tbeg + tb, w.t_end);
          for (int t = tbeg; ok && t < te; ++t, ++c) {
            const int src = (t - tbeg) * nc;
            const int32_t y = __shfl_sync(0xFFFFFFFFu, py, src + cl);
            const int32_t z = __shfl_sync(0xFFFFFFFFu, pz, src + cl);
            const uint64_t mk = __shfl_sync(0xFFFFFFFFu, m, src);
            const uint32_t bar = smem_u32(&X.full[sl]);
            if (again) ok = wait_phase(X, X.empty[sl], ph ^ 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (lane == 0) {
              if (k == 0) X.mask[c & 3] = mk;
              mbar_arrive_expect_tx(bar, kSlotBytes);
            }
            __syncwarp();
            if (lane < nc) tma_load_5d(ring + sl * kSlotBytes + lane * R * 256, &kmap, 2 * k, y, z, bar, pol);
            sl += 4;
            if (sl >= NS) { sl -= NS; ph ^= 1; again = true; }
          }
        }
        if (!ok) break;
      } while (walk_next(a, w));
      if (!ok) X.abort = 1;
      // No copy may still be landing when the CTA exits: wait for this warp's last three, but
      // for those whose slot another quarter has taken since (they have long landed, and the
      // barrier is in a later phase).
      if (lane < 3 && lane < c && 4 * (c - 1 - lane) + k + NS >= 4 * c) {
        int s = sl - 4 * (lane + 1);
        if (s < 0) { s += NS; ph ^= 1; }
        if (s < 0) { s += NS; ph ^= 1; }
        mbar_wait(smem_u32(&X.full[s]), ph, 100000000ull);
      }
    } else {
      // ================= FP8 rows through registers =================
      // Two groups of eight warps take turns at the tiles, so a group's tile loads into its
      // registers while the other group converts and stores (a group that loaded the next
      // quarter after each one waited for that load before it could use the one already there:
      // registers wait for all loads behind one counter).  Thread t of a group: row t / 4 of a
      // tile and of each quarter dims 16 (t % 4) .. and 64 + 16 (t % 4) .., two loads of 64 whole
      // bytes a row and stores free of bank conflicts; a thread has one row, whose page is looked
      // up a turn ahead.  (Eight lanes a row, whole lines: 2 % less time for FP8_S128 rows, 3 %
      // more for FP8_E8M0.)
      const int grp = (warp - C::kWarpL) >> 3, t256 = (tid - 32 * C::kWarpL) & 255;
      const int r = t256 >> 2, pc = t256 & 3;
      Walk w;
      walk_start(a, X, u1 - u0, w);
      int tn = w.t;  // next tile to look up
      bool more = true;
      auto step = [&]() {
        if (more && ++tn == w.t_end) {
          more = walk_next(a, w);
          tn = w.t;
        }
      };
      // The page and the row within it of the next tile's row (row -1: none), and past the other
      // group's tile; false: no further tile.
      auto look = [&](int& page, int& row) -> bool {
        page = row = -1;
        if (!more) return false;
        const int64_t j = ((int64_t)w.i.tile0 + tn) * 64 + r;
        if (j >= w.i.lo && j < w.i.hi) {
          const int32_t lp = page_of(a, (uint32_t)j);
          row = (int32_t)j - lp * a.cache.page_rows;
          page = a.cache.table[(int64_t)w.i.seq * a.cache.table_ld + lp];
        }
        step();
        step();
        return true;
      };
      // Address of the row (null: none), and the tile's valid rows among this warp's eight.
      auto place = [&](int page, int row, const uint8_t*& src) -> uint32_t {
        src = nullptr;
        if (row >= 0) {
          if (page >= 0 && page < a.cache.n_pages)
            src = a.cache.data + (int64_t)page * a.cache.page_stride + (int64_t)row * 528;
          else if (pc == 0)
            raise_fault(kFaultBounds);
        }
        uint32_t m = __ballot_sync(0xFFFFFFFFu, src != nullptr) & 0x11111111u;
        m = (m | (m >> 3)) & 0x03030303u;
        m = (m | (m >> 6)) & 0x000F000Fu;
        return (m | (m >> 12)) & 0xFFu;
      };
      uint4 buf[2][4];
      uint32_t scl;  // scale word pc of the row: an fp32 scale (FP8_S128) or four bytes
      auto fetch = [&](const uint8_t* src) {
        scl = 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) buf[0][k] = buf[1][k] = make_uint4(0u, 0u, 0u, 0u);
        if (src) {
          scl = __ldcs(reinterpret_cast<const uint32_t*>(src + 512) + pc);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            buf[0][k] = __ldcs(reinterpret_cast<const uint4*>(src + 16 * pc + 128 * k));
            buf[1][k] = __ldcs(reinterpret_cast<const uint4*>(src + 16 * pc + 128 * k + 64));
          }
        }
      };
      int page, row;
      const uint8_t* src;
      if (grp == 1) step();
      bool have = look(page, row);
      uint32_t bits = place(page, row, src);
      fetch(src);
      bool nxt = look(page, row);
      int c = grp, sl = 4 * grp;
      uint32_t ph = 0;
      const uint32_t off0 = ring + (r >> 3) * kGroup + sw128_off(r & 7, 2 * pc);
      const uint32_t off1 = ring + (r >> 3) * kGroup + sw128_off(r & 7, 2 * pc + 1);
      for (; have; c += 2) {
        // the slots become free in order: one look at the last one's often stands for all four
        bool free;
        {
          const int i = sl + 3;
          free = 4 * c + 3 < NS ||
                 all_ok(mbar_test_wait(smem_u32(&X.empty[i >= NS ? i - NS : i]),
                                       i >= NS ? ph : ph ^ 1));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (!free && 4 * c + k >= NS) wait_phase(X, X.empty[sl], ph ^ 1);
          if (k == 0 && lane == 0)
            reinterpret_cast<uint8_t*>(&X.mask[c & 3])[(warp - C::kWarpL) & 7] = (uint8_t)bits;
          // (with the last quarter: its slot is free once the tile before the last one has read
          // its scales)
          if (kMode == 1 && k == 3)
            sc_s[((c & (C::kScTiles - 1)) * 4 + pc) * 64 + (r & 33) + ((r & 6) << 2) +
                 ((r & 24) >> 2)] = __uint_as_float(scl);
          uint32_t word = 0;
          if (kMode == 2) word = __shfl_sync(0xFFFFFFFFu, scl, (lane & 28) + k) >> (8 * (pc >> 1));
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // dim block i of the quarter
            // 2^(e - 127) twice in bf16: exponent field e, the subnormal 0x0040 for e = 0
            const uint32_t sc2 = max(((word >> (16 * i)) & 0xFFu) * 0x00800080u, 0x00400040u);
            const uint32_t w4[4] = {buf[i][k].x, buf[i][k].y, buf[i][k].z, buf[i][k].w};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t packed[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                    (__nv_fp8x2_storage_t)((w4[2 * h + (j >> 1)] >> (16 * (j & 1))) & 0xFFFFu),
                    __NV_E4M3);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
                packed[j] = pack_bf16x2(f.x, f.y);  // exact: four significant bits
                if (kMode == 2) {
                  const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&packed[j]),
                                                   *reinterpret_cast<const __nv_bfloat162*>(&sc2));
                  packed[j] = *reinterpret_cast<const uint32_t*>(&v);
                }
              }
              st_shared16((h ? off1 : off0) + sl * kSlotBytes + i * kBlock,
                          make_uint4(packed[0], packed[1], packed[2], packed[3]));
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&X.landed[sl]));
          if (++sl == NS) { sl = 0; ph ^= 1; }
        }
        sl += 4;  // the other group's tile
        if (sl >= NS) { sl -= NS; ph ^= 1; }
        have = nxt;
        if (have) {
          bits = place(page, row, src);
          fetch(src);
          nxt = look(page, row);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (kDirect && cl == 1 && u1 > u0) {
    // the item's output by sixteen warps (the ring is empty: it stages them)
    const Item I = load_item(a, X.it0, false);
    const int Hg = min(64, a.H - 64 * I.hg);
    if (tid < Hg) finish_head(a, X, head_sums<C::kParts>(Y, tid), Y.sink2[tid], tid, I);
    __syncthreads();
    if (warp < 16)
      store_tile(a, X, tmem + ((uint32_t)((warp & 3) * 32) << 16), warp >> 2, warp & 3, lane, Hg,
                 ring + warp * 1024, a.out + (I.q * a.H + 64 * I.hg) * kDLat);
    tc_fence_before();
    __syncthreads();
  }
  if (kDirect && cl > 1) {
    // Each CTA owns 512 / cluster dims.  Once all are done with their rings, every CTA writes its
    // O^T (unscaled) into the rings of the dims' owners and its m, l, r to all; then the owners
    // weigh, sum and store.
    const int lg = cl == 8 ? 3 : cl == 4 ? 2 : 1;
    const int slice = kDLat >> lg, half = slice >> 1;  // dims, pairs of them
    static_assert(NS * kSlotBytes >= kHp * 2048, "room for the parts, [ranks][heads][a rank's dims]");
    constexpr bool kTail = NS * kSlotBytes >= kHp * 2048 + 8 * 3 * kHp * 4;
    // [rank][m, l, r][head], in every CTA
    const uint32_t st_off = kTail ? (uint32_t)(C::kQBytes + kHp * 2048)
                                  : (uint32_t)(C::kQBytes + NS * kSlotBytes + sizeof(PagedSpare));
    static_assert(kTail || C::kPBytes >= (int)sizeof(PagedSpare) + 8 * 3 * kHp * 4, "room for m, l, r");
    float* st = reinterpret_cast<float*>(smem + st_off);
    const Item I = load_item(a, blockIdx.x / cl, false);
    const bool live = I.units > 0;  // the same in the whole cluster
    const int Hg = min(64, a.H - 64 * I.hg);
    float own[3] = {-INFINITY, 0.f, 0.f};
    if (live && tid < kHp && u1 > u0) {
      own[0] = Y.m_run[tid];
#pragma unroll
      for (int i = 0; i < C::kParts; ++i) {
        own[1] += Y.lsum[i][tid];
        own[2] += Y.rsum[i][tid];
      }
    }
    cluster_sync();
    if (live && tid < kHp)
      for (int o = 0; o < cl; ++o)
#pragma unroll
        for (int i = 0; i < 3; ++i)
          st_cluster32(dsmem_addr(smem_u32(st + (crank * 3 + i) * kHp + tid), o),
                       __float_as_uint(own[i]));
    if (live && u1 > u0 && warp < 16) {
      const int mt = warp >> 2, d = mt * 128 + (warp & 3) * 32 + lane;
      // [rank][four heads][even dims, odd dims][4]: the owner reads a pair's dims by neighbouring
      // lanes without bank conflicts
      const int at = ((d & (slice - 1)) >> 1) + (d & 1) * half;
      const uint32_t to =
          dsmem_addr(ring + (uint32_t)((crank * (kHp / 4)) * slice + at) * 16, d >> (9 - lg));
#pragma unroll 1
      for (int hb = 0; hb < Hg; hb += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColO + 64 * mt + hb, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          st_cluster16(to + (uint32_t)((hb >> 2) + j) * slice * 16,
                       make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
      }
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    // weights and 1 / Z: eight lanes a head, one for each rank
    for (int i = tid; live && i < 8 * kHp; i += C::kThreads) {
      const int h = i >> 3, o = i & 7;
      const bool in = o < cl && h < Hg;  // heads that are padding weigh nothing
      const float logit = a.sink && h < Hg ? a.sink[64 * I.hg + h] : -INFINITY;
      const float sink = sink_log2(logit);
      float* so = st + o * 3 * kHp + h;
      const float m = in ? so[0] : -INFINITY;
      float M = fmaxf(m, sink);
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, x));
      const float Mf = M == -INFINITY ? 0.f : M, w = ex2(m - Mf);
      float l = in ? w * so[kHp] : 0.f, r = in ? w * so[2 * kHp] : 0.f;
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) {
        l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
        r += __shfl_xor_sync(0xFFFFFFFFu, r, x);
      }
      if (o < cl) so[0] = in ? w : 0.f;
      if (o > 0 || h >= Hg) continue;
      const float rows = l;
      if (sink > -INFINITY) {
        l += ex2(sink - Mf);
        r += ex2(sink - Mf);
      }
      X.fac[h] = r > 0.f || r != r ? 1.f / r : 0.f;
      if (a.lse && crank == 0)
        a.lse[I.q * a.H + 64 * I.hg + h] = head_lse(Mf, l, rows, logit);
    }
    __syncthreads();
    if (live) {
      for (int i = tid; i < (kHp / 4) * half; i += C::kThreads) {
        const int hc = i >> (8 - lg), pair = i & (half - 1);
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int o = 0; o < cl; ++o) {
          const float4 w = *reinterpret_cast<const float4*>(st + o * 3 * kHp + 4 * hc);
          // a CTA without tiles wrote nothing, and its weights are zero
          if (!(w.x != 0.f || w.y != 0.f || w.z != 0.f || w.w != 0.f)) continue;
          const float4* b = reinterpret_cast<const float4*>(smem + C::kQBytes) +
                            (o * (kHp / 4) + hc) * slice + pair;
          join_add(acc, b[0], b[half], w);
        }
        const int d = crank * slice + 2 * pair;
        float cs = 1.f, sn = 0.f;
        if (a.inv_freq && d >= kRopeDim0) {
          cs = X.rope_c[(d - kRopeDim0) >> 1];
          sn = X.rope_s[(d - kRopeDim0) >> 1];
        }
        uint16_t* out = a.out + (I.q * a.H + 64 * I.hg) * kDLat + d;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (4 * hc + h >= Hg) break;
          const float x0 = acc[h] * X.fac[4 * hc + h], x1 = acc[4 + h] * X.fac[4 * hc + h];
          __stcs(reinterpret_cast<unsigned int*>(out + (4 * hc + h) * kDLat),
                 pack_bf16x2(x0 * cs + x1 * sn, x1 * cs - x0 * sn));
        }
      }
    }
    __syncthreads();
  }
  if (warp == C::kWarpS) tmem_dealloc(tmem, 512);
}

// ================================ join ===================================================
//
// Joins the parts of the items that several CTAs worked on: with M the largest running
// maximum (and the sink logit), weights 2^(m - M) and Z = 2^(sink - M) + sum 2^(m - M) l,
// out = sum 2^(m - M) O / Z.  A CTA takes one item, 2 kPairs dims and kSets times four heads, a
// thread a pair of dims of four heads; its kGroups groups take every kGroups-th part, the first
// kAhead of them loaded before the weights are known.  Bound by latency: the parts come from L2.
// Many items, of few parts each, take four sets and no groups: few CTAs with long loads.  Fewer
// items take four groups and a set; a single long one, which may have 152 parts, 32 groups and
// CTAs of 64 dims (whole calls, us: 64 items of 128 to 512 tiles 234 with sets / 240 with groups,
// 16 of 256 to 512 tiles 88 / 87, 8 of them 62 / 54; one item of 1024 tiles 31.8 with 32 groups
// / 45.4 with four, two 46.7 / 49.9).
constexpr int kMaxCtas = 152;
constexpr int kAhead = 4;

template <int kGroups, int kSets, int kPairs>
__global__ void __launch_bounds__(kPairs * kGroups * kSets)
    paged_join_kernel(PagedAttnArgs a, int hp) {
  static_assert(kGroups == 1 || kSets == 1, "the groups' sums fold over one set");
  constexpr int kWarps = kPairs * kGroups * kSets / 32;
  __shared__ float4 wt[kMaxCtas][kSets];
  __shared__ float4 inv_s[kSets];
  __shared__ float acc_s[kGroups > 1 ? kGroups / 2 : 1][8][kPairs];
  __shared__ float rope_c[32], rope_s[32];
  griddep_launch_dependents();
  griddep_wait();  // for the parts, and for what the attention's call was given
  const int64_t it = blockIdx.x;
  constexpr int kCuts = 256 / kPairs;  // CTAs of the same heads
  const int cut = blockIdx.y % kCuts, hc0 = kSets * (blockIdx.y / kCuts);
  const int64_t q = a.ng == 2 ? it >> 1 : it;
  const int hg = a.ng == 2 ? (int)(it & 1) : 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pair = tid % kPairs, set = tid / kPairs % kSets, grp = tid / (kPairs * kSets);
  const int2 rec = a.rec[it];  // (of an item that is not live: not written, and not used)
  const int seq = a.q_seq[q];
  const bool live = 64 * hg + 4 * hc0 < a.H && seq >= 0 && seq < a.cache.B;
  // the rotation by one warp, where this CTA has rotated dims
  if (a.inv_freq && live && warp == kWarps - 1 && 2 * kPairs * (cut + 1) > kRopeDim0) {
    sincosf(rope_angle(rope_turn(a.inv_freq[lane]), (uint64_t)a.q_pos[q]), &rope_s[lane],
            &rope_c[lane]);
  }
  if (!live || rec.x < 0) return;
  const int n = min(rec.y - rec.x + 1, kMaxCtas);
  auto part = [&](int s) -> int64_t { return 2 * (int64_t)(rec.x + s) + (s == 0 ? 1 : 0); };
  const int hc = hc0 + set;
  const bool mine = 64 * hg + 4 * hc < a.H && 4 * hc < hp;
  const int d = 2 * (cut * kPairs + pair);  // this thread's dims d, d + 1
  const float4* src = reinterpret_cast<const float4*>(a.part) + ((d >> 7) * (hp / 4) + hc) * 128 +
                      ((d & 127) >> 1);
  float4 x[kAhead], y[kAhead];
  auto load = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int s = s0 + i * kGroups;
      if (s < n && mine) {
        const float4* p = src + part(s) * (int64_t)(hp * kDLat / 4);
        x[i] = __ldcs(p);
        y[i] = __ldcs(p + 64);
      }
    }
  };
  load(grp);
  // weights and 1 / Z of a head by one warp
  for (int hh = warp; hh < 4 * kSets; hh += kWarps) {
    const int hb = 4 * hc0 + hh, hq = 64 * hg + hb;
    const bool there = hq < a.H && hb < hp;
    const float logit = a.sink && there ? a.sink[hq] : -INFINITY, sink = sink_log2(logit);
    float m[(kMaxCtas + 31) / 32], M = sink;
#pragma unroll
    for (int i = 0; i < (kMaxCtas + 31) / 32; ++i) {
      const int s = lane + 32 * i;
      m[i] = s < n && there ? a.pstat[part(s) * (3 * hp) + hb] : -INFINITY;
      M = fmaxf(M, m[i]);
    }
    M = lanes_max<32>(M);
    const float Mf = M == -INFINITY ? 0.f : M;
    float l = 0.f, r = 0.f;
#pragma unroll
    for (int i = 0; i < (kMaxCtas + 31) / 32; ++i) {
      const int s = lane + 32 * i;
      if (s < n) {
        const float w = there ? ex2(m[i] - Mf) : 0.f;
        reinterpret_cast<float*>(&wt[s][0])[hh] = w;
        if (there) {
          const float* st = a.pstat + part(s) * (3 * hp) + hb;
          l = fmaf(w, st[hp], l);
          r = fmaf(w, st[2 * hp], r);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
      r += __shfl_xor_sync(0xFFFFFFFFu, r, o);
    }
    const float sk = sink == -INFINITY ? 0.f : ex2(sink - Mf), rows = l;
    l += sk;
    r += sk;
    if (lane == 0) {
      reinterpret_cast<float*>(inv_s)[hh] = r > 0.f || r != r ? 1.f / r : 0.f;
      if (a.lse && cut == 0 && there)
        a.lse[q * a.H + hq] = head_lse(Mf, l, rows, logit);
    }
  }
  __syncthreads();
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s0 = grp; s0 < n; s0 += kAhead * kGroups) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int s = s0 + i * kGroups;
      if (s < n && mine) join_add(acc, x[i], y[i], wt[s][set]);
    }
    load(s0 + kAhead * kGroups);
  }
  if (kGroups > 1) {
#pragma unroll
    for (int low = kGroups / 2; low > 0; low >>= 1) {  // the groups' sums fold in halves
      if (grp >= low && grp < 2 * low) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc_s[grp - low][i][pair] = acc[i];
      }
      __syncthreads();
      if (grp < low) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += acc_s[grp][i][pair];
      }
      __syncthreads();
    }
    if (grp > 0) return;
  }
  if (!mine) return;
  float cs = 1.f, sn = 0.f;
  if (a.inv_freq && d >= kRopeDim0) {
    cs = rope_c[(d - kRopeDim0) >> 1];
    sn = rope_s[(d - kRopeDim0) >> 1];
  }
  const float4 iv = inv_s[set];
  const float inv[4] = {iv.x, iv.y, iv.z, iv.w};
  const int h0 = 64 * hg + 4 * hc;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    if (h0 + h >= a.H) break;
    const float x0 = acc[h] * inv[h], x1 = acc[4 + h] * inv[h];
    __stcs(reinterpret_cast<unsigned int*>(a.out + (q * a.H + h0 + h) * kDLat + d),
           pack_bf16x2(x0 * cs + x1 * sn, x1 * cs - x0 * sn));
  }
}

template <int kHp, int kMode, bool kDirect>
cudaError_t launch_attn_inst(const PagedAttnArgs& a, const CUtensorMap& qm, const CUtensorMap& km,
                             cudaStream_t s) {
  using C = PagedCfg<kHp, kMode>;
  auto kern = paged_attn_kernel<kHp, kMode, kDirect>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)a.nctas), block(C::kThreads);
  return kDirect && a.cluster > 1
             ? launch_pdl_cluster(kern, grid, block, C::kSmem, s, (unsigned)a.cluster, a, qm, km)
             : launch_pdl(kern, grid, block, C::kSmem, s, a, qm, km);
}

template <int kHp, int kMode>
cudaError_t launch_attn_kind(const PagedAttnArgs& a, const CUtensorMap& qm, const CUtensorMap& km,
                             cudaStream_t s) {
  return a.cluster > 0 ? launch_attn_inst<kHp, kMode, true>(a, qm, km, s)
                       : launch_attn_inst<kHp, kMode, false>(a, qm, km, s);
}

template <int kHp>
cudaError_t launch_attn_mode(const PagedAttnArgs& a, const CUtensorMap& qm, const CUtensorMap& km,
                             cudaStream_t s) {
  switch (a.cache.dtype) {
    case 0: return launch_attn_kind<kHp, 0>(a, qm, km, s);
    case 1: return launch_attn_kind<kHp, 1>(a, qm, km, s);
    default: return launch_attn_kind<kHp, 2>(a, qm, km, s);
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, int sms, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  // Four tokens a warp at a time once every SM has 64 tokens: 10000 bf16 tokens 5.9 us against
  // 7.4 with a warp each, 4900 FP8 tokens 7.3 us against 5.9
  if (a.T >= 8 * kAppWarps * sms) {
    const int64_t need = (a.T + 4 * kAppWarps - 1) / (4 * kAppWarps), most = (int64_t)sms * kAppCtas;
    return launch_pdl(paged_append_kernel<4>, dim3((unsigned)(need < most ? need : most)),
                      dim3(kAppWarps * 32), 0, s, a);
  }
  return launch_pdl(paged_append_kernel<1>, dim3((unsigned)((a.T + kAppWarps - 1) / kAppWarps)),
                    dim3(kAppWarps * 32), 0, s, a);
}

int paged_head_pad(int H) { return H <= 16 ? 16 : H <= 32 ? 32 : 64; }

// Tiles of a unit: the share of an item that is not split further.
int paged_unit_tiles() { return 4; }

int paged_max_ctas() { return kMaxCtas; }

// CTAs per item of a small call, 0 for one whose tiles are dealt evenly to all CTAs and joined
// through the workspace.  An item of up to four tiles takes one CTA.  The tiles of a
// longer one are shared by 8, 4 or 2, as many as all items leave room for (clusters of eight do
// not fill every SM): up to 32 tiles an item, where lengths below the caller's bound cost
// little.  Measured, us, bf16, equal lengths, clusters against even dealing: 8 sequences of
// 16 tiles 16.0 / 17.7, 33 of 32 tiles 26.6 / 36.8, 66 of 16 tiles 26.3 / 38.6; of 32 tiles six
// sequences 18.4 / 17.8 and five 17.9 / 17.6 (FP8_S128 23.3 / 23.7 and 22.8 / 23.5).
int paged_cluster(int64_t items, int64_t tiles, int sms) {
  if (tiles <= paged_unit_tiles()) return items <= sms ? 1 : 0;
  if (tiles > 32 || (tiles > 16 && items < 6)) return 0;
  return items <= sms / 10 ? 8 : items <= (sms - 16) / 4 ? 4 : items <= (sms - 16) / 2 ? 2 : 0;
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int units, cudaStream_t s) {
  if (a.Q == 0) return cudaSuccess;
  const int hp = paged_head_pad(a.H);
  CUtensorMap qm, km;
  if (!encode_rows_bf16(&qm, a.q, (uint64_t)a.Q * a.H, kDLat, 64, (uint32_t)hp))
    return cudaErrorInvalidValue;
  km = qm;
  if (a.cache.dtype == 0) {
    // a page as [8-row groups][8 dim blocks][8 rows][128 bytes]
    const uint64_t dims[5] = {128, 8, 8, (uint64_t)a.cache.page_rows / 8, (uint64_t)a.cache.n_pages};
    const uint64_t strides[4] = {1024, 128, 8192, (uint64_t)a.cache.page_stride};
    const uint32_t box[5] = {128, 8, 2, (uint32_t)a.box_rows / 8, 1};
    if (!encode_bytes(&km, a.cache.data, 5, dims, strides, box)) return cudaErrorInvalidValue;
  }
  cudaError_t e = hp == 16   ? launch_attn_mode<16>(a, qm, km, s)
                  : hp == 32 ? launch_attn_mode<32>(a, qm, km, s)
                             : launch_attn_mode<64>(a, qm, km, s);
  if (e != cudaSuccess || units <= 1) return e;
  const unsigned items = (unsigned)(a.Q * a.ng);
  if (items == 1 && units > 64)
    return launch_pdl(paged_join_kernel<32, 1, 32>, dim3(items, 2u * hp), dim3(1024), 0, s, a, hp);
  return items >= 16
             ? launch_pdl(paged_join_kernel<1, 4, 64>, dim3(items, hp / 4u), dim3(256), 0, s, a, hp)
             : launch_pdl(paged_join_kernel<4, 1, 64>, dim3(items, (unsigned)hp), dim3(256), 0, s, a, hp);
}

}  // namespace csa2
