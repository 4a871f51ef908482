// k_chunk.cu -- chunks of new tokens over the paged latent cache, and its rows read back
// (paged_read_kernel).
#include <cuda_fp16.h>

#include "common.cuh"
#include "compress_dev.cuh"

CSA2_DEFINE_FAULT_FLAG(chunk)

namespace csa2 {
namespace {

// ================================ read ==================================================
//
// The inverse of paged_append_kernel.  A warp takes runs of up to 32 rows: first each lane finds where one of
// them lies, then the rows are loaded kTok at a time, the next ones before these are written.  An FP8 lane
// has dims 16 l .. of a row, one 16-byte load and two 16-byte stores; a bf16 lane the chunks l and 32 + l of
// eight dims.  Lane i has the angle of rotation pair i, which the lanes of dims 448.. fetch.  x = code *
// scale in fp32, rounded once to bf16 (exact for FP8_E8M0 scales of 2^-124 to 2^119).  Bound by the
// bytes moved, 1024 or 528 read and 1024 written per row: 163835 FP8_E8M0 rows, rotated back, in 49 to 52 us
// (5.0 TB/s of 6.8), as many bf16 rows in 69; few rows by the launch (300 in 4.5 us).  The grid stays: with one
// CTA for each four runs 60 us, with a row looked up at a time 92.

constexpr int kReadWarps = 4;
constexpr int read_ctas(int mode) { return mode == 0 ? 4 : 5; }  // an SM, by registers

__device__ __forceinline__ float2 e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float e8m0_scale(uint32_t e) {  // 2^(e - 127); 255 is NaN
  return e == 0 ? __uint_as_float(0x00400000u) : e == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(e << 23);
}
__device__ __forceinline__ void turn_back(float& x0, float& x1, float c, float s) {  // times e^{-i p theta}
  const float y = x0 * c + x1 * s;
  x1 = x1 * c - x0 * s;
  x0 = y;
}

// What a lane loads of a row, and the row written from it.
template <int kMode>
struct RowPart {
  uint4 a, b;   // bf16: two chunks; FP8: sixteen codes in a
  uint32_t sc;  // FP8: the scale

  __device__ __forceinline__ void load(const uint8_t* src, int lane) {
    a = __ldcs(reinterpret_cast<const uint4*>(src) + lane);
    if (kMode == 0) b = __ldcs(reinterpret_cast<const uint4*>(src) + 32 + lane);
    if (kMode == 1) sc = __ldcs(reinterpret_cast<const uint32_t*>(src + 512) + (lane >> 3));
    if (kMode == 2) sc = __ldcs(src + 512 + (lane >> 1));
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); sc = 0u; }
  // ang: cosine and sine of the row's 32 rotation pairs, or null.  low: where what the rounding leaves of
  // FP8_S128 values goes (nothing of those that overflow), or null.
  __device__ __forceinline__ void store(uint16_t* dst, int lane, const float2* ang, uint16_t* low) const {
    if (kMode == 0) {
      uint4 w = b;
      if (ang && lane >= 24) {
        float y[8];
        unpack_bf16x8(b, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 g = ang[4 * (lane - 24) + i];
          turn_back(y[2 * i], y[2 * i + 1], g.x, g.y);
        }
        w = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                       pack_bf16x2(y[6], y[7]));
      }
      __stcs(reinterpret_cast<uint4*>(dst) + lane, a);
      __stcs(reinterpret_cast<uint4*>(dst) + 32 + lane, w);
    } else {
      const float scale = kMode == 1 ? __uint_as_float(sc) : e8m0_scale(sc);
      const float2 f = make_float2(scale, scale);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
      float2 y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = mul2(e4m3x2(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu), f);
      if (ang && lane >= 28) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 g = ang[8 * (lane - 28) + i];
          turn_back(y[i].x, y[i].y, g.x, g.y);
        }
      }
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = pack_bf16x2(y[i].x, y[i].y);
      __stcs(reinterpret_cast<uint4*>(dst) + 2 * lane, make_uint4(o[0], o[1], o[2], o[3]));
      __stcs(reinterpret_cast<uint4*>(dst) + 2 * lane + 1, make_uint4(o[4], o[5], o[6], o[7]));
      if (kMode == 1 && low) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float h0 = __uint_as_float(o[i] << 16), h1 = __uint_as_float(o[i] & 0xFFFF0000u);
          o[i] = pack_bf16x2(isfinite(h0) ? y[i].x - h0 : 0.f, isfinite(h1) ? y[i].y - h1 : 0.f);
        }
        __stcs(reinterpret_cast<uint4*>(low) + 2 * lane, make_uint4(o[0], o[1], o[2], o[3]));
        __stcs(reinterpret_cast<uint4*>(low) + 2 * lane + 1, make_uint4(o[4], o[5], o[6], o[7]));
      }
    }
  }
};

template <int kMode, int kTok>
__global__ void __launch_bounds__(kReadWarps * 32, read_ctas(kMode)) paged_read_kernel(PagedReadArgs a, int run) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ __align__(16) float2 ang_s[kReadWarps][kTok][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t step = (int64_t)gridDim.x * kReadWarps * run;
  const uint64_t turn = a.inv_freq ? rope_turn(a.inv_freq[lane]) : 0;
  const int64_t rows = a.cu_seqlens[a.cache.B];
  // (with row_end a key tile's length of zeros more, which a tile that ends there reads)
  const int64_t total = min((int64_t)a.T, rows + (a.row_end ? 256 : 0));
  for (int64_t t = ((int64_t)blockIdx.x * kReadWarps + (threadIdx.x >> 5)) * run; t < total; t += step) {
    // lane l: row t + l
    const int n = (int)min(total - t, (int64_t)run);
    const uint8_t* src = nullptr;
    int64_t j = 0;
    const bool zero = a.row_end != nullptr;
    {
      const int64_t tl = t + min(lane, n - 1);
      int b = cdev::warp_find_seq(a.cu_seqlens, a.cache.B, t, lane);
      if (tl < rows) {  // (the rows behind the last sequence's are no sequence's)
        if (a.cu_seqlens[b + 1] <= tl) {  // in a later sequence
          int hi = a.cache.B - 1;
          for (++b; b < hi;) {
            const int m = (b + hi + 1) >> 1;
            if (a.cu_seqlens[m] <= tl) b = m;
            else hi = m - 1;
          }
        }
        j = a.start_row[b] + (tl - a.cu_seqlens[b]);
      }
      if (tl < rows && (!zero || j < a.row_end[b])) {
        int32_t page = -1, row = 0;
        if (j >= 0 && j < a.cap_rows) {
          const int32_t lp = (int32_t)(__umulhi((uint32_t)j, a.page_mul) >> a.page_shift);
          row = (int32_t)j - lp * a.cache.page_rows;
          page = a.cache.table[(int64_t)b * a.cache.table_ld + lp];
        }
        if (page < 0 || page >= a.cache.n_pages) {
          if (lane < n) raise_fault(kFaultBounds);
        } else {
          src = a.cache.data + (int64_t)page * a.cache.page_stride + (int64_t)row * (kMode == 0 ? 1024 : 528);
        }
      }
    }
    __syncwarp();
    const uint64_t p = (uint64_t)j * (uint64_t)a.ratio;
    const uint32_t skips = __ballot_sync(0xFFFFFFFFu, !src && !zero);  // rows of out that are left as they are
    RowPart<kMode> cur[kTok], nxt[kTok];
    auto fetch = [&](RowPart<kMode>(&r)[kTok], int i0) {
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        const uint64_t at = __shfl_sync(0xFFFFFFFFu, (unsigned long long)src, (i0 + i) & 31);
        if (at && i0 + i < n) r[i].load(reinterpret_cast<const uint8_t*>(at), lane);
        else r[i].zero();
      }
    };
    fetch(cur, 0);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kTok) {
      if (i0 + kTok < n) fetch(nxt, i0 + kTok);
      if (a.inv_freq) {
        __syncwarp();  // the last rows' angles are read
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
          const uint64_t pi = __shfl_sync(0xFFFFFFFFu, (unsigned long long)p, (i0 + i) & 31);
          sincosf(rope_angle(turn, pi), &ang_s[warp][i][lane].y, &ang_s[warp][i][lane].x);
        }
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        const bool none = (skips >> ((i0 + i) & 31) & 1u) != 0;
        if (none || i0 + i >= n) continue;  // (the same in the warp)
        const int64_t at = (t + i0 + i) * a.out_ld;
        cur[i].store(a.out + at, lane, a.inv_freq ? ang_s[warp][i] : nullptr, a.low ? a.low + at : nullptr);
      }
#pragma unroll
      for (int i = 0; i < kTok; ++i) cur[i] = nxt[i];
    }
  }
}

// ================================ chunk attention =======================================
//
// Rows (token, head) of a sequence's new tokens form tiles of 128, in the order of q; all of them
// share the keys, so the scores of a tile are one product of 128 x 512 by 512 x 256 cache rows (a
// key tile), and the output another of 128 x 256 by 256 x 512.
//
// A pair of CTAs works on a tile (tcgen05 with cta_group::2, M = 128: 64 rows in each CTA), because
// the output's 512 fp32 columns for 128 rows are all of an SM's tensor memory: here each CTA holds
// them for its 64 rows in 256 columns, folded over 128 lanes (lane r and 64 + r are row r: the first
// and second half of a product's columns), beside two buffers of scores of 128 columns.  For S a CTA
// brings 128 of the key tile's rows, for O 256 of the 512 dims of all its rows, so a cache row is
// loaded once as key and once as value by a pair, in slots of 16 KiB that one ring of 8 holds:
//   K slot k        this CTA's 128 rows x dims 64 k .. 64 k + 63
//   V slot (c, h)   rows 64 c .. 64 c + 63 x this CTA's dims 256 h + 128 rank .. + 127
// A key tile is eight slots of each, a revolution of the ring: K(0) K(1) V(0) K(2) V(1) ..
//   warps 0..7   softmax: thread (lane r or 64 + r, half of its columns) has 64 scores of a row, all in
//                one 64-row block of P.  The running maximum m moves only when a score exceeds it by
//                2^64, so a tile's usual pass is one vote
//   warp 8       issues all products (even CTA)
//   warps 9, 10  load the even and the odd slots, the first of them each tile's Q
//   warp 11      cleans values that must not be read (below)
// The plan deals the key tiles of all tiles evenly to the pairs; a tile that several pairs work on is
// joined from their parts by chunk_join_kernel.
//
// A key tile takes 4096 cycles of products (an MMA of 128 x 256 x 16 by a pair 64, probed; with N = 128 it takes
// 52) and about 5400 in all: reads of Q, P, K and V by the products and writes of the slots and P share an SM's
// shared memory.  2048 tokens of 64 heads over 32768 rows take 5.0 to 5.5 ms, 1.57 to 1.7 PFLOP/s of 1.9
// (1.70 is what a library's product of matrices sustains at the power limit).  The loops over slots are
// rolled: unrolled, this took 6.0 ms, for the code of four kinds of warp then left the instruction cache.
//
// A row that some tokens of a tile see and others do not may hold NaN or infinities, which must not
// reach those others through 0 * NaN.  Such a row makes its scores non-finite for every query, so
// where a key tile is masked for some row, a masked score that is not finite flags the cache row, and
// the values of flagged rows lose their non-finite elements before the product.  A token that sees the row
// has a NaN weight and shows it all the same, unless its score is -inf: then the weight is 0, and
// 0 times the elements that were lost is NaN in their dims (poison_outputs), as it is in a key tile that all
// tokens see.  Rows behind the last visible one are garbage and are treated so too.  Rows in two
// parts lose the elements of the first; the second holds zeros there, and is finite everywhere.

constexpr int kQRows = 128, kKeys = 256;
constexpr int kSlotBytes = 16384, kSlots = 8;
constexpr int kQBytes = 65536, kPBytes = 32768;
constexpr int kSoftWarps = 8, kSoft = 32 * kSoftWarps;
constexpr int kWarpMma = 8, kWarpLoad = 9, kLoadWarps = 2, kWarpClean = 11, kThreads = 32 * 12;
constexpr uint32_t kColS = 256;
constexpr float kLazy = 64.0f;
// Key tiles that O sums up in tensor memory (65536 rows; the tensor core cuts the low bits of its
// running sums).  A longer segment is done in runs, which add up in fp32 in the pair's part.
constexpr int kRun = 256;

// A key tile of a pair's work, for the warps that do it; the loader writes them ahead.
struct __align__(16) ChunkStep {
  uint32_t groups;  // groups of eight rows that are on a page
  int base;         // first cache row
  int i;            // key tile of the segment, -1: no further one
  int kind;         // 1: the segment's last, 2: not all of its rows are seen by all tokens
};
enum : int { kStepLast = 1, kStepMasked = 2 };
// A segment: key tiles of a tile of queries.
struct __align__(16) ChunkSegment {
  int64_t start;
  int row0, rows, tok0, clip;  // as in ChunkTile
  int whole;                   // all of the tile's key tiles
  int slot;                    // its part
  int seq;
};

struct __align__(16) ChunkAux {
  uint64_t full[kSlots], empty[kSlots];
  uint64_t q_full, q_empty;
  uint64_t s_full[2];
  uint64_t p_full[4], p_free[4];  // P's blocks of 64 cache rows: written; read by their products
  uint64_t step_full[4];
  uint64_t clean_req, clean_done;
  uint64_t fin;
  ChunkStep step[4];      // of key tile c & 3 (three at most are in use)
  ChunkSegment seg[4];    // of segment s & 3 (four)
  uint32_t flags[2][8];   // even CTA: rows of key tile c & 1 to be cleaned
  uint32_t clean[8];      // rows to be cleaned now
  uint64_t turn[32];
  float top[4][64], sum[4][64];
  uint32_t tmem_slot;
  int abort, done, work;
  int odd[2];             // of key tile c & 1: a token sees a row with a score that is not finite
};
constexpr int kSmem = kQBytes + kSlots * kSlotBytes + kPBytes + (int)sizeof(ChunkAux);
static_assert(kSmem <= 232448, "shared memory of a CTA");

// Wait for a phase; false once something in the CTA has given up.  kPair: one that threads of both CTAs
// complete with what they wrote.
template <bool kPair = false>
__device__ __forceinline__ bool wait_phase(ChunkAux& X, uint64_t& bar, uint32_t parity,
                                           uint64_t limit_ns = 2000000000ull) {
  const uint32_t b = smem_u32(&bar);
  auto done = [&]() { return kPair ? mbar_try_wait_cluster(b, parity) : mbar_try_wait(b, parity); };
  if (done()) return true;
  const volatile int* abort = &X.abort;
  if (*abort) return false;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    for (int i = 0; i < 64; ++i)
      if (done()) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      raise_fault(kFaultTimeout);
      X.abort = 1;
      return false;
    }
  }
}

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoft) : "memory"); }
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

// 32 bytes to global memory, 16-byte aligned; in one store where they are a sector.
__device__ __forceinline__ void store_sector(uint16_t* to, const uint32_t (&b)[8]) {
  if ((reinterpret_cast<uintptr_t>(to) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(b[0]), "r"(b[1]),
                 "r"(b[2]), "r"(b[3]), "r"(b[4]), "r"(b[5]), "r"(b[6]), "r"(b[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(to)[0] = make_uint4(b[0], b[1], b[2], b[3]);
    reinterpret_cast<uint4*>(to)[1] = make_uint4(b[4], b[5], b[6], b[7]);
  }
}

// x / d for x < 2^31 by the factor and shift of d (Divide): see there.
__device__ __forceinline__ uint32_t divide(uint32_t x, const Divide& d) {
  return d.shift < 0 ? x : __umulhi(x, d.mul) >> d.shift;
}

// Rows lo .. hi - 1 that the token at position p sees, of at most clip; true if there were more.
__device__ __forceinline__ bool token_rows(const ChunkArgs& a, int64_t p, int64_t clip, int& lo, int& hi) {
  int64_t h;
  if (p < 0) h = 0;
  else if (p < 0x7FFFFFFF) h = divide((uint32_t)(p + 1), a.by_ratio);
  else h = (int64_t)min(((uint64_t)p + 1) / (uint64_t)a.ratio, (uint64_t)1 << 62);
  int64_t l = a.window > 0 && h > a.window ? h - a.window : 0;
  const bool over = h > clip;
  if (over) {
    h = clip;
    l = l < h ? l : h;
  }
  lo = (int)l;
  hi = (int)h;
  return over;
}

// ---- plan ------------------------------------------------------------------------------
//
// One CTA: the tiles of all sequences with their key tiles, the staged rows' places, and each pair's
// share.  Up to as many tiles as pairs, none longer than kWhole, go to a pair each.  Otherwise the cost of
// all tiles, 2 a key tile and kTileCost a tile (what begins and ends it takes as long as 1.5 key tiles), is
// cut evenly: pair c begins at cost W c / C, C as many pairs as leave each kShare key tiles or a tile.  A cut
// within the first kTileCost of a tile is one before it.  Up to kPlanFew tiles and sequences are planned by as
// many threads, whose barriers are shorter (with the fewer CTAs of the join: 35 sequences of two tokens 40.1 ->
// 36.5 us, 45 of eight 44.7 -> 40.4).  kMaxPairs: a pair for each two of the GPU's 152 SMs.
constexpr int kPlanThreads = 1024, kPlanFew = 256, kMaxPairs = 76;
constexpr int kWhole = 6, kShare = 4, kTileCost = 3;

// Exclusive prefix of x over the CTA's threads; *total gets the sum.
template <int kN>
__device__ __forceinline__ int64_t plan_scan(int64_t x, int64_t* sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t z = __shfl_up_sync(0xFFFFFFFFu, y, o);
    if (lane >= o) y += z;
  }
  if (lane == 31) sums[warp] = y;
  __syncthreads();
  if (warp == 0) {
    int64_t v = lane < kN / 32 ? sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += z;
    }
    sums[lane] = v;
  }
  __syncthreads();
  *total = sums[31];
  const int64_t before = (warp ? sums[warp - 1] : 0) + y - x;
  __syncthreads();
  return before;
}

// x / y, mostly in 32 bits (a division in 64 takes four times as long).
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

// Tile k of a sequence of `count` tokens from tok0 on, the first at position start; true if a token sees
// more rows than it may.
__device__ __forceinline__ bool make_tile(const ChunkArgs& a, ChunkTile& t, int seq, int tok0, int count, int64_t start,
                                          int64_t off, int clip, int k) {
  const int64_t rows = (int64_t)count * a.H - (int64_t)k * kQRows;
  t.seq = seq;
  t.rows = (int)min(rows, (int64_t)kQRows);
  t.row0 = tok0 * a.H + k * kQRows;
  t.tok0 = tok0;
  t.start = start;
  t.off = off;
  t.clip = clip;
  t.c0 = t.c1 = 0;
  int lo, hi, y;
  bool over = token_rows(a, start + (int)(divide(t.row0, a.by_heads) - tok0), clip, lo, y);
  over |= token_rows(a, start + (int)(divide(t.row0 + t.rows - 1, a.by_heads) - tok0), clip, y, hi);
  t.k0 = hi > lo ? lo / kKeys : 0;
  t.kn = hi > lo ? (hi + kKeys - 1) / kKeys - t.k0 : 1;
  return over;
}

template <int kN>
__global__ void __launch_bounds__(kN) chunk_plan_kernel(ChunkArgs a) {
  constexpr int kTiles = 4;  // of a thread at a time, at most
  __shared__ int64_t sums[32];
  __shared__ int tile0[kN], tok0[kN], count[kN], clip[kN];
  __shared__ int64_t off[kN], start[kN];
  __shared__ int cut_tile[kMaxPairs + 1], cut_at[kMaxPairs + 1];
  __shared__ int64_t cut_keys[kMaxPairs + 1];
  __shared__ int longest, splits;
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  if (tid == 0) longest = splits = 0;
  int64_t tiles = 0, units = 0, staged = 0;
  int most = 0;
  const int B = a.cache.B;
  for (int b0 = 0; b0 < B; b0 += kN) {
    const int b = b0 + tid;
    int t0 = 0, n = 0, c = (int)a.cap_rows;
    int64_t s = 0, first = 0, len = 0, end = 0;
    if (b < B) {
      t0 = min(max(a.cu_seqlens[b], 0), a.T);
      n = max(0, min(a.cu_seqlens[b + 1], a.T) - t0);
      s = a.start_pos[b];
    }
    if (a.stage && n > 0) {
      int lo, hi, x;
      token_rows(a, s, a.cap_rows, lo, x);
      token_rows(a, s + n - 1, a.cap_rows, x, hi);
      first = lo & ~7;
      end = hi > lo ? hi : first;
      len = (end - first + 7) & ~(int64_t)7;
    }
    int64_t total = 0;
    if (a.stage) {
      const int64_t at = staged + plan_scan<kN>(len, sums, &total);
      if (at + len > a.stage_rows) {  // more rows than announced
        raise_fault(kFaultBounds);
        len = max((int64_t)0, a.stage_rows - at) & ~(int64_t)7;
        end = min(end, first + len);
        c = (int)end;
      }
      if (b < B) {
        a.stage_cu[b] = (int32_t)min(at, a.stage_rows);
        a.stage_first[b] = first;
        a.stage_end[b] = end;
      }
      off[tid] = at - first;
      staged += total;
    } else {
      off[tid] = 0;
    }
    const int64_t nt = ((int64_t)n * a.H + kQRows - 1) / kQRows;
    const int64_t mine = plan_scan<kN>(nt, sums, &total);
    tile0[tid] = (int)mine;
    tok0[tid] = t0;
    count[tid] = n;
    clip[tid] = c;
    start[tid] = s;
    __syncthreads();
    const int here = (int)total;
    const int per = here > kN ? kTiles : 1;
    for (int x0 = 0; x0 < here; x0 += per * kN) {
      const int x = x0 + per * tid;
      int i = 0, e = kN;  // the last sequence with tile0 <= x
      while (e - i > 1) {
        const int m = (i + e) >> 1;
        if (tile0[m] <= x) i = m;
        else e = m;
      }
      int cost[kTiles], sum = 0;
#pragma unroll
      for (int q = 0; q < kTiles; ++q) {
        cost[q] = 0;
        if (q < per && x + q < here && tiles + x + q < a.max_tiles) {
          while (i + 1 < kN && tile0[i + 1] <= x + q) ++i;  // (past empty sequences)
          ChunkTile t{};
          if (make_tile(a, t, b0 + i, tok0[i], count[i], start[i], off[i], clip[i], x + q - tile0[i]) &&
              clip[i] == a.cap_rows)
            raise_fault(kFaultBounds);
          a.tile[tiles + x + q] = t;
          cost[q] = 2 * t.kn + kTileCost;
          most = max(most, t.kn);
        }
        sum += cost[q];
      }
      int64_t before = units + plan_scan<kN>(sum, sums, &total);
#pragma unroll
      for (int q = 0; q < kTiles; ++q) {
        if (cost[q]) a.prefix[tiles + x + q] = before;
        before += cost[q];
      }
      units += total;
    }
    tiles += here;
    __syncthreads();
  }
  if (a.stage && tid == 0) a.stage_cu[B] = (int32_t)min(staged, a.stage_rows);
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if ((tid & 31) == 0) atomicMax(&longest, most);
  __syncthreads();
  const int64_t n = min(tiles, (int64_t)a.max_tiles);
  if (n <= a.pairs && longest <= kWhole) {
    if (tid < a.pairs) a.share[tid] = tid < n ? ChunkShare{tid, 0, a.tile[tid].kn} : ChunkShare{0, 0, 0};
    if (tid == 0) a.split[0] = 0;
    return;
  }
  int64_t C = max(n, ((units - kTileCost * n) / 2 + kShare - 1) / kShare);
  C = C < a.pairs ? C : a.pairs;
  // Where each pair begins: the last tile that does at or before its cut, searched for in every so manieth
  // tile's prefix first.
  int64_t* sample = start;
  const int64_t every = (n + kN - 1) / kN;
  if (tid * every < n) sample[tid] = a.prefix[tid * every];
  __syncthreads();
  if (tid <= C) {
    if (tid == C) {
      cut_tile[tid] = (int)n;
      cut_at[tid] = 0;
      cut_keys[tid] = (units - kTileCost * n) / 2;
    } else {
      const int64_t u = quotient(units * tid, C);
      int lo = 0, hi = (int)((n - 1) / every);
      while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (sample[m] <= u) lo = m;
        else hi = m - 1;
      }
      int64_t x = lo * every, e = min(n, x + every) - 1;
      while (x < e) {
        const int64_t m = (x + e + 1) >> 1;
        if (a.prefix[m] <= u) x = m;
        else e = m - 1;
      }
      const int64_t p = a.prefix[x], at = u - p - kTileCost;
      cut_tile[tid] = (int)x;
      cut_at[tid] = at > 0 ? (int)(at >> 1) : 0;
      cut_keys[tid] = (p - kTileCost * x) / 2 + cut_at[tid];
    }
  }
  __syncthreads();
  if (tid < a.pairs)
    a.share[tid] = tid < C ? ChunkShare{cut_tile[tid], cut_at[tid], cut_keys[tid + 1] - cut_keys[tid]}
                           : ChunkShare{0, 0, 0};
  // the tiles that are cut, each by the first pair that begins within it
  if (tid > 0 && tid < C && cut_at[tid] > 0 && !(cut_tile[tid - 1] == cut_tile[tid] && cut_at[tid - 1] > 0)) {
    int last = tid;
    while (last + 1 < C && cut_tile[last + 1] == cut_tile[tid]) ++last;
    a.tile[cut_tile[tid]].c0 = tid - 1;
    a.tile[cut_tile[tid]].c1 = last;
    a.split[1 + atomicAdd(&splits, 1)] = cut_tile[tid];
  }
  __syncthreads();
  if (tid == 0) a.split[0] = splits;
}

// Few short sequences: tile `pair` by a warp of its own, without a plan; false when there is none.  All lanes
// get the tile.
__device__ __forceinline__ bool plan_alone(const ChunkArgs& a, ChunkTile& t, int pair, int lane, bool report) {
  int tiles = 0;
  for (int b0 = 0; b0 < a.cache.B; b0 += 32) {
    const int b = b0 + lane;
    int tok0 = 0, n = 0;
    if (b < a.cache.B) {
      tok0 = min(max(a.cu_seqlens[b], 0), a.T);
      n = max(0, min(a.cu_seqlens[b + 1], a.T) - tok0);
    }
    const int mine = (int)(((int64_t)n * a.H + kQRows - 1) / kQRows);
    int to = mine;  // tiles of this and the sequences before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, to, o);
      if (lane >= o) to += x;
    }
    const uint32_t here = __ballot_sync(0xFFFFFFFFu, tiles + to > pair);
    if (here) {
      const int l = __ffs(here) - 1;
      const int first = tiles + __shfl_sync(0xFFFFFFFFu, to - mine, l);
      const int seq = b0 + l;
      if (make_tile(a, t, seq, __shfl_sync(0xFFFFFFFFu, tok0, l), __shfl_sync(0xFFFFFFFFu, n, l), a.start_pos[seq], 0,
                    (int)a.cap_rows, pair - first) && report && lane == 0)
        raise_fault(kFaultBounds);
      return true;
    }
    tiles += __shfl_sync(0xFFFFFFFFu, to, 31);
  }
  return false;
}

// ---- attention -------------------------------------------------------------------------

// A pair's walk over its key tiles: i of n of the segment (tile, from key tile `unit` of it on).  The next
// tile's record is read a segment ahead.
struct ChunkWalk {
  int64_t left;  // units behind this segment
  int tile, unit, n, i;
  ChunkTile t, next;
};
__device__ __forceinline__ void walk_fit(const ChunkArgs& a, ChunkWalk& w) {
  const int rest = w.t.kn - w.unit;
  w.n = rest < w.left ? rest : (int)w.left;
  w.left -= w.n;
  w.i = 0;
  if (w.left > 0) w.next = a.tile[w.tile + 1];
}
template <bool kAlone>
__device__ __forceinline__ bool walk_start(const ChunkArgs& a, int pair, int lane, bool report, ChunkWalk& w) {
  if (kAlone) {
    w.left = 0;
    w.tile = w.unit = w.i = 0;
    if (!plan_alone(a, w.t, pair, lane, report)) return false;
    w.n = w.t.kn;
    return true;
  }
  const ChunkShare s = a.share[pair];
  w.left = s.count;
  if (w.left <= 0) return false;
  w.tile = s.tile;
  w.unit = s.unit;
  w.t = a.tile[w.tile];
  walk_fit(a, w);
  return true;
}
// On to the next key tile; false when there is none.
__device__ __forceinline__ bool walk_next(const ChunkArgs& a, ChunkWalk& w) {
  if (++w.i < w.n) return true;
  if (w.left <= 0) return false;
  w.unit = 0;
  ++w.tile;
  w.t = w.next;
  walk_fit(a, w);
  return true;
}
// What the tokens of a tile see: the first's lo, the last's hi.
__device__ __forceinline__ void tile_rows(const ChunkArgs& a, const ChunkTile& t, int& lo0, int& hi0,
                                          int& lo1, int& hi1) {
  token_rows(a, t.start + (int)(divide(t.row0, a.by_heads) - t.tok0), t.clip, lo0, hi0);
  token_rows(a, t.start + (int)(divide(t.row0 + t.rows - 1, a.by_heads) - t.tok0), t.clip, lo1, hi1);
}

// Groups of eight rows of a key tile, one a lane: where each lies.
struct Places {
  int32_t y, z;  // group within the page, page
  bool good;     // on a page, or not needed
};
__device__ __forceinline__ Places place_groups(const ChunkArgs& a, const ChunkTile& t, int64_t base, int lo,
                                               int hi, int lane, bool report) {
  Places p;
  const int64_t j = base + 8 * lane;
  const bool needed = j < hi && j + 8 > lo;
  p.y = a.cache.page_rows >> 3;  // outside every page: reads as zeros
  p.z = 0;
  p.good = true;
  if (j < t.clip) {
    const int32_t lp = (int32_t)(__umulhi((uint32_t)j, a.page_mul) >> a.page_shift);
    const int32_t page = a.cache.table[(int64_t)t.seq * a.cache.table_ld + lp];
    if (page >= 0 && page < a.cache.n_pages) {
      if (!a.stage) {
        p.y = (int32_t)(j - (int64_t)lp * a.cache.page_rows) >> 3;
        p.z = page;
      }
    } else if (needed) {
      p.good = false;
      if (report) raise_fault(kFaultBounds);
    }
  }
  if (a.stage) p.y = (int32_t)((j + t.off) >> 3);
  return p;
}

// Rows of block `blk` of a key tile that a token sees (they are on a page, and lo .. hi - 1).
__device__ __forceinline__ uint64_t rows_seen(int base, uint32_t groups, int blk, int lo, int hi) {
  uint64_t seen = tile_mask((int64_t)base + 64 * blk, lo, hi);
  const uint32_t g8 = (groups >> (8 * blk)) & 0xFFu;
#pragma unroll
  for (int g = 0; g < 8; ++g)
    if (!(g8 >> g & 1u)) seen &= ~(0xFFull << (8 * g));
  return seen;
}

// Those of them whose scores, in the 64 columns from `scores` on, are not finite, as bits for the token of row `row`.
__device__ __forceinline__ void note_rows(ChunkAux& X, uint32_t scores, int base, uint32_t groups, int lo, int hi,
                                          bool any, int blk, int row) {
  uint64_t odd = 0;
#pragma unroll 1
  for (int k = 0; k < 64; k += 16) {
    uint32_t v[16], w = 0;
    __syncwarp();
    tmem_ld16(scores + k, v);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 16; ++j) w |= (v[j] & 0x7F800000u) == 0x7F800000u ? 1u << j : 0u;
    odd |= (uint64_t)w << k;
  }
  odd = any ? odd & rows_seen(base, groups, blk, lo, hi) : 0;
  X.top[blk][row] = __uint_as_float((uint32_t)odd);
  X.sum[blk][row] = __uint_as_float((uint32_t)(odd >> 32));
}

// The O of such a token gets NaN in the dims in which one of these rows, of the key tile from row `base` on, is not
// finite.  O is in the 64 columns from `o` and `o` + 128 on, dims d.. and d + 256 ...  By whole warps, hardly ever.
__device__ __forceinline__ void poison_outputs(const ChunkArgs& a, const ChunkAux& X, int seq, int base, int row,
                                               int d, uint32_t o) {
  const int64_t off = a.stage ? a.stage_cu[seq] - a.stage_first[seq] : 0;
#pragma unroll 1
  for (int k = 0; k < 8; ++k) {
    const int col = 16 * (k & 3), dim = d + 256 * (k >> 2) + col;
    uint32_t gone = 0;  // columns
#pragma unroll 1
    for (int b = 0; b < 8; ++b) {
      uint32_t bits = __float_as_uint((b & 1 ? X.sum : X.top)[b >> 1][row]);
      for (; bits; bits &= bits - 1) {
        const int64_t j = (int64_t)base + 32 * b + __ffs(bits) - 1;
        const uint16_t* at;
        if (a.stage) {
          at = a.stage + (j + off) * kDLat;
        } else {
          const int32_t lp = (int32_t)(__umulhi((uint32_t)j, a.page_mul) >> a.page_shift);
          at = reinterpret_cast<const uint16_t*>(a.cache.data + a.cache.table[(int64_t)seq * a.cache.table_ld + lp] *
                                                                    a.cache.page_stride) +
               (j - (int64_t)lp * a.cache.page_rows) * kDLat;
        }
        for (int i = 0; i < 16; ++i)
          if ((at[dim + i] & 0x7F80u) == 0x7F80u) gone |= 1u << i;
      }
    }
    if (__any_sync(0xFFFFFFFFu, gone != 0)) {
      uint32_t v[16];
      __syncwarp();
      tmem_ld16(o + 128 * (k >> 2) + col, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (gone >> i & 1u) v[i] = 0x7FC00000u;
      tmem_st16(o + 128 * (k >> 2) + col, v);
      tmem_st_wait();
    }
  }
}

// What the softmax warps do with such a key tile c in place of handing on their blocks of P alone.  (A call of its
// own: as two calls or inlined, 2048 tokens over 32768 rows, which never come here, took 2 to 6 % longer.)
__device__ __noinline__ void poison_tile(const ChunkArgs& a, ChunkAux& X, int seg, int c, int base, uint32_t groups, int lo,
                                         int hi, bool any, uint32_t tlane, uint32_t p_full) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = warp >> 2, L = 32 * (warp & 3) + lane;
  const int row = L & 63, kh = L >> 6, blk = 2 * kh + half;
  note_rows(X, tlane + kColS + 128 * (c & 1) + 64 * half, base, groups, lo, hi, any, blk, row);  // while they are there
  fence_proxy_async_smem();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive_cluster(p_full);
  soft_sync();
  wait_phase(X, X.p_free[3], (uint32_t)c & 1);  // the values' products are done
  tc_fence_after();
  poison_outputs(a, X, X.seg[(seg - 1) & 3].seq, base, row, kh * 128 + half * 64, tlane + 64 * half);
  tc_fence_before();
  soft_sync();
  if (threadIdx.x == 0) X.odd[c & 1] = 0;  // (set again by tile c + 2, barriers from here)
}

// kAlone: without a plan, pair c works on tile c.  kParts: of a staged row.  (Instances of their own, as code that is
// not used lies in the way of what is: with kAlone's in it, ragged chunks took 531 us in place of 509, with
// kParts as a number 525.)
template <bool kAlone, int kParts>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t q_s = smem_u32(smem), ring = q_s + kQBytes, p_s = ring + kSlots * kSlotBytes;
  ChunkAux& X = *reinterpret_cast<ChunkAux*>(smem + kQBytes + kSlots * kSlotBytes + kPBytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1;
  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&X.full[i]), 1);
      mbar_init(smem_u32(&X.empty[i]), 1);
    }
    mbar_init(smem_u32(&X.q_full), 1);
    mbar_init(smem_u32(&X.q_empty), 1);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&X.s_full[i]), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&X.p_full[i]), 2 * kSoftWarps / 4);
      mbar_init(smem_u32(&X.p_free[i]), 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&X.step_full[i]), 1);
    mbar_init(smem_u32(&X.clean_req), 1);
    mbar_init(smem_u32(&X.clean_done), 2);
    mbar_init(smem_u32(&X.fin), 1);
    X.abort = X.done = 0;
    X.odd[0] = X.odd[1] = 0;
    mbar_fence_init();
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  if (tid < 16) X.flags[tid >> 3][tid & 7] = 0;
  if (warp == kWarpMma) {
    tmem_alloc_pair(smem_u32(&X.tmem_slot), 512);
    tmem_relinquish_pair();
  }
  griddep_wait();
  if (a.inv_freq && tid < 32) X.turn[tid] = rope_turn(a.inv_freq[tid]);
  ChunkWalk w;  // the loaders'
  if (warp >= kWarpLoad && warp < kWarpLoad + kLoadWarps) {
    const bool any = walk_start<kAlone>(a, pair, lane, rank == 0 && warp == kWarpLoad, w);
    if (warp == kWarpLoad && lane == 0) X.work = any;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const bool work = X.work != 0;
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, X.tmem_slot, 0);

  if (work && warp < kSoftWarps) {
    // ================= softmax, rescale, output =================
    // (a wait that gave up is not acted on here: the loop's barriers need every thread)
    const int quad = warp & 3, half = warp >> 2;
    const int L = 32 * quad + lane, row = L & 63, kh = L >> 6, blk = 2 * kh + half;
    const uint32_t tlane = tmem + ((uint32_t)(32 * quad) << 16);
    const float sc2 = a.scale * kLog2e;
    const uint32_t p_full = dsmem_addr(smem_u32(&X.p_full[blk]), 0);
    const uint32_t flags = dsmem_addr(smem_u32(&X.flags[0][2 * blk]), 0);
    int seg = 0;  // segments so far
    // of the segment: what this thread's row sees; the running maximum,
    // that of what the part holds, and the sums of P (unrounded, rounded)
    int lo = 0, hi = 0;
    float m = -INFINITY, mslot = -INFINITY;
    float2 l2 = make_float2(0.f, 0.f), r2 = l2;
    float logit = -INFINITY;  // the row's sink
    auto part_of = [&](int sl) {
      return reinterpret_cast<float4*>(a.part) + (((int64_t)sl * 2 + rank) * 64 + 16 * half) * 128 + L;
    };
    for (int c = 0;; ++c) {
      // (the loader ends the steps, too, when something has given up: all threads see the same end)
      mbar_wait(smem_u32(&X.step_full[c & 3]), (uint32_t)(c >> 2) & 1, 60000000000ull);
      const ChunkStep st = X.step[c & 3];
      const bool have = st.i >= 0, first = st.i <= 0;
      uint32_t pk[32];
      bool masked = false;
      bool poison = false;  // a thread sees a row with a score that is not finite
      // of the segment before, until its end is done
      const float m_end = m, mslot_end = mslot;
      const float2 l_end = l2, r_end = r2;
      const float logit_end = logit;
      if (have) {
        if (first) {
          m = mslot = -INFINITY;
          l2 = r2 = make_float2(0.f, 0.f);
          const ChunkSegment& t = X.seg[seg & 3];
          const int grow = t.row0 + min((int)rank * 64 + row, t.rows - 1);  // rows behind the last follow it
          const int tok = (int)divide(grow, a.by_heads);
          token_rows(a, t.start + (tok - t.tok0), t.clip, lo, hi);
          if (a.sink) logit = a.sink[grow - tok * a.H];
          ++seg;
        }
        wait_phase(X, X.s_full[c & 1], (uint32_t)(c >> 1) & 1);
        tc_fence_after();
        const uint32_t scores = tlane + kColS + 128 * (c & 1) + 64 * half;
        masked = (st.kind & kStepMasked) != 0;
        const uint64_t seen = masked ? rows_seen(st.base, st.groups, blk, lo, hi) : ~0ull;
        // Exponents of columns 2 j, 2 j + 1: v two of the scores.
        auto scaled = [&](int j, const uint32_t* v, float nm) {
          float2 y = fma2(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), make_float2(sc2, sc2),
                          make_float2(nm, nm));
          if (masked) {
            if (!(seen >> (2 * j) & 1u)) y.x = -INFINITY;
            if (!(seen >> (2 * j + 1) & 1u)) y.y = -INFINITY;
          }
          return y;
        };
        // The largest exponent of a row, of its four threads.
        auto row_top = [&](float top) {
          X.top[blk][row] = top;
          soft_sync();
          float mx = X.top[0][row];
#pragma unroll
          for (int k = 1; k < 4; ++k) mx = fmaxf(mx, X.top[k][row]);
          return mx;
        };
        // P = 2^(score - m), m the running maximum (none yet: 0)
        float top;
        float2 ls, rs;
        auto weights = [&]() {
          const float nm = m == -INFINITY ? 0.f : -m;
          top = -INFINITY;
          ls = rs = make_float2(0.f, 0.f);
          uint32_t v[64];
          tmem_ld32(scores, *reinterpret_cast<uint32_t(*)[32]>(v));
          tmem_ld32(scores + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float2 y = scaled(j, v + 2 * j, nm);
            top = fmaxf(top, fmaxf(y.x, y.y));
            y = make_float2(ex2(y.x), ex2(y.y));
            ls = add2(ls, y);
            pk[j] = pack_bf16x2(y.x, y.y);
            rs = add2(rs, make_float2(__uint_as_float(pk[j] << 16), __uint_as_float(pk[j] & 0xFFFF0000u)));
          }
        };
        // a segment's first tile begins with its own maximum, which the weights then need not move
        for (int pass = first ? 1 : 0;; ++pass) {
          if (pass == 1 || masked) {
            // the largest exponent; and rows that must not be seen and whose scores are not finite
            uint32_t v[64], bad[2] = {0u, 0u};
            tmem_ld32(scores, *reinterpret_cast<uint32_t(*)[32]>(v));
            tmem_ld32(scores + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
            tmem_ld_wait();
            const float nm = m == -INFINITY ? 0.f : -m;
            top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float2 y = scaled(j, v + 2 * j, nm);
              top = fmaxf(top, fmaxf(y.x, y.y));
              if (masked) {
                if ((v[2 * j] & 0x7F800000u) == 0x7F800000u) bad[j >> 4] |= 1u << (2 * (j & 15));
                if ((v[2 * j + 1] & 0x7F800000u) == 0x7F800000u) bad[j >> 4] |= 2u << (2 * (j & 15));
              }
            }
            if (masked) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                if (bad[k] & (uint32_t)(seen >> (32 * k))) *reinterpret_cast<volatile int*>(&X.odd[c & 1]) = 1;
                bad[k] = __reduce_or_sync(0xFFFFFFFFu, bad[k] & ~(uint32_t)(seen >> (32 * k)));
                if (lane == 0 && bad[k]) red_or_cluster(flags + (c & 1) * 32 + k * 4, bad[k]);
              }
            }
          }
          if (pass == 1) {  // a row's maximum moves
            const float mx = row_top(top);
            float f = 1.f;
            if (mx > kLazy || (m == -INFINITY && mx > -INFINITY)) {
              f = m == -INFINITY ? 0.f : ex2(-mx);
              m = m == -INFINITY ? mx : m + mx;
              const float2 ff = make_float2(f, f), o = make_float2(0.f, 0.f);
              l2 = fma2(l2, ff, o);
              r2 = fma2(r2, ff, o);
            }
            if ((st.i & (kRun - 1)) != 0) {
              wait_phase(X, X.p_free[3], (uint32_t)(c - 1) & 1);
              tc_fence_after();
              if (__any_sync(0xFFFFFFFFu, f != 1.f)) {
#pragma unroll 1
                for (int k = 0; k < 128; k += 16) {
                  uint32_t v[16];
                  tmem_ld16(tlane + 128 * half + k, v);
                  tmem_ld_wait();
#pragma unroll
                  for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * f);
                  tmem_st16(tlane + 128 * half + k, v);
                }
                tmem_st_wait();
              }
            }
          }
          weights();
          if (pass == 1) {
            // all have read top, and have rescaled O: no block of P is handed on before
            tc_fence_before();
            soft_sync();
            break;
          }
          if (!soft_any(top > kLazy || (m == -INFINITY && top > -INFINITY))) break;
        }
        l2 = add2(l2, ls);
        r2 = add2(r2, rs);
        if (masked) poison = *reinterpret_cast<volatile int*>(&X.odd[c & 1]) != 0;
      }
      // ---- the end of the segment before: O is read and stored before the next values' products may
      // start (those of scores run on) ----
      const ChunkSegment& e = X.seg[(seg - (have ? 2 : 1)) & 3];
      // (what it needs of the record is read before the products start: the loader may then write it over)
      const bool end = first && c > 0, store = end && e.whole;
      const int wrow = (int)rank * 64 + 32 * (quad & 1);  // this warp's rows within the tile
      // the output's rotation: lane i has the angles of pair i, of the first kTok tokens of this warp's rows
      constexpr int kTok = 2;
      float2 ang[kTok] = {};
      int tok = 0, ntok = 0;
      if (store && blk == 3 && a.inv_freq) {
        tok = (int)divide(e.row0 + wrow, a.by_heads);
        ntok = (int)divide(e.row0 + wrow + 31, a.by_heads) - tok + 1;
#pragma unroll
        for (int k = 0; k < kTok; ++k)
          if (k < ntok)
            sincosf(rope_angle(X.turn[lane], (uint64_t)(e.start + (tok + k - e.tok0))), &ang[k].y, &ang[k].x);
      }
      if (c > 0) wait_phase(X, X.p_free[blk], (uint32_t)(c - 1) & 1);
      if (have) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          st_shared16(p_s + blk * 8192 + sw128_off(row, k),
                      make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]));
      }
      if (end) {
        wait_phase(X, X.p_free[3], (uint32_t)(c - 1) & 1);
        tc_fence_after();
        X.top[blk][row] = l_end.x + l_end.y;
        X.sum[blk][row] = r_end.x + r_end.y;
        soft_sync();
        float l = 0.f, r = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          l += X.top[k][row];
          r += X.sum[k][row];
        }
        const bool live = (int)rank * 64 + row < e.rows;
        float fac = 0.f;
        if (e.whole) {
          const float sink = sink_log2(logit_end);
          const float M = fmaxf(m_end, sink), Mf = M == -INFINITY ? 0.f : M, x = ex2(m_end - Mf);
          const float rows = l * x;
          float z = rows, zr = r * x;
          if (sink > -INFINITY) {
            z += ex2(sink - Mf);
            zr += ex2(sink - Mf);
          }
          fac = zr > 0.f || zr != zr ? x / zr : 0.f;  // no row and no sink: zeros
          if (a.lse && live && blk == 0)
            a.lse[e.row0 + (int)rank * 64 + row] = head_lse(Mf, z, rows, logit_end);
        } else if (blk == 0) {
          float* to = a.pstat + ((int64_t)e.slot * 2 + rank) * 192 + row;
          to[0] = m_end;
          to[64] = l;
          to[128] = r;
        }
        __syncwarp();
        const float f0 = mslot_end == -INFINITY ? 0.f : ex2(mslot_end - m_end);
        const bool folded = mslot_end != -INFINITY;
        const int mytok = ntok ? (int)divide(e.row0 + wrow + lane, a.by_heads) - tok : 0;
        // A lane has 32 columns of its row at a time; their 64 bytes go out as two whole sectors (stores of
        // 16 bytes a row took prompts twice as long; through shared memory a tile's end took 2000 cycles more).
        uint16_t* out = a.out + (int64_t)(e.row0 + (int)rank * 64 + row) * kDLat + kh * 128 + half * 64;
        float4* to = part_of(e.slot);
#pragma unroll 1
        for (int k = 0; k < 4; ++k, to += (k & 1 ? 8 : 24) * 128, out += k & 1 ? 32 : 224) {
          uint32_t v[32];
          tmem_ld32(tlane + 128 * (k >> 1) + 64 * half + 32 * (k & 1), v);
          tmem_ld_wait();
          if (folded || !store) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float4 o = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                     __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
              if (folded) {
                const float4 q = to[j * 128];
                o.x = fmaf(q.x, f0, o.x);
                o.y = fmaf(q.y, f0, o.y);
                o.z = fmaf(q.z, f0, o.z);
                o.w = fmaf(q.w, f0, o.w);
              }
              if (!store) to[j * 128] = o;
              v[4 * j] = __float_as_uint(o.x);
              v[4 * j + 1] = __float_as_uint(o.y);
              v[4 * j + 2] = __float_as_uint(o.z);
              v[4 * j + 3] = __float_as_uint(o.w);
            }
            if (!store) {
              __syncwarp();
              continue;
            }
          }
          if (k >= 2) {  // pair 16 (k - 2) + j times e^{-i p theta}
#pragma unroll 1
            for (int n = 0; n < ntok; ++n) {
              float2 an = n == 0 ? ang[0] : ang[1];
              if (n >= kTok) sincosf(rope_angle(X.turn[lane], (uint64_t)(e.start + (tok + n - e.tok0))), &an.y, &an.x);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float cs = __shfl_sync(0xFFFFFFFFu, an.x, 16 * (k - 2) + j);
                const float sn = __shfl_sync(0xFFFFFFFFu, an.y, 16 * (k - 2) + j);
                const float y0 = __uint_as_float(v[2 * j]), y1 = __uint_as_float(v[2 * j + 1]);
                if (mytok == n) {
                  v[2 * j] = __float_as_uint(y0 * cs + y1 * sn);
                  v[2 * j + 1] = __float_as_uint(y1 * cs - y0 * sn);
                }
              }
            }
          }
          if (live) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t b[8];
#pragma unroll
              for (int j = 0; j < 8; ++j)
                b[j] = pack_bf16x2(__uint_as_float(v[16 * q + 2 * j]) * fac, __uint_as_float(v[16 * q + 2 * j + 1]) * fac);
              store_sector(out + 16 * q, b);
            }
          }
          __syncwarp();  // (what follows wants whole warps)
        }
      }
      // A block of P lets the first products overwrite O, whichever warps have read it: none is handed on
      // before all have.  (The sums, too, are read before others are written.)
      if (end) {
        tc_fence_before();
        soft_sync();
      }
      if (!have) break;
      if (poison) {
        poison_tile(a, X, seg, c, st.base, st.groups, lo, hi, l2.x + l2.y == l2.x + l2.y, tlane, p_full);
      } else {
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(p_full);
      }
      if (!(st.kind & kStepLast) && ((st.i + 1) & (kRun - 1)) == 0) {
        // a run's end: O joins what the part holds
        wait_phase(X, X.p_free[3], (uint32_t)c & 1);
        tc_fence_after();
        const float f = mslot == -INFINITY ? 0.f : ex2(mslot - m);
        const bool onto = st.i + 1 > kRun;
        float4* part = part_of(X.seg[(seg - 1) & 3].slot);
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
          const int hh = k >> 2, col = 16 * (k & 3);
          uint32_t v[16];
          tmem_ld16(tlane + 128 * hh + 64 * half + col, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float4* to = part + (hh * 32 + (col >> 2) + j) * 128;
            float4 o = onto ? *to : make_float4(0.f, 0.f, 0.f, 0.f);
            o.x = fmaf(o.x, f, __uint_as_float(v[4 * j]));
            o.y = fmaf(o.y, f, __uint_as_float(v[4 * j + 1]));
            o.z = fmaf(o.z, f, __uint_as_float(v[4 * j + 2]));
            o.w = fmaf(o.w, f, __uint_as_float(v[4 * j + 3]));
            *to = o;
          }
        }
        mslot = m;
        tc_fence_before();
        soft_sync();  // (as above: the next block of P lets O be overwritten)
      }
    }
    if (tid == 0) *reinterpret_cast<volatile int*>(&X.done) = 1;
  } else if (work && warp == kWarpMma && rank == 0) {
    // ================= products =================
    const uint32_t lead = elect_lane();
    const uint32_t id_s = idesc_bf16(128, 256, 0, 0), id_o = idesc_bf16(128, 256, 0, 1);
    const uint64_t q_d = sdesc_sw128(q_s, 16, 1024), p_d = sdesc_sw128(p_s, 16, 1024);
    const uint64_t k_d = sdesc_sw128(ring, 16, 1024), v_d = sdesc_sw128(ring, 1024, 2048);
    bool ok = true;
    int rev = 0;
    int cleaned = 0;
    // The values of key tile c of this pair, the run's run-th.
    auto values = [&](int c, int run, bool masked) {
      if (masked) {  // every row is flagged that is to be
#pragma unroll 1
        for (int k = 0; k < 4; ++k) ok = ok && all_ok(wait_phase<true>(X, X.p_full[k], (uint32_t)c & 1));
        const uint32_t bad = lane < 8 && ok ? X.flags[c & 1][lane] : 0u;
        if (__any_sync(0xFFFFFFFFu, bad != 0u)) {
          // rows to be cleaned, by a warp of each CTA, once all of the tile's values are there
#pragma unroll 1
          for (int k = 0; k < kSlots; ++k) ok = ok && all_ok(wait_phase(X, X.full[k], (uint32_t)rev & 1));
          if (lane < 8) {
            X.flags[c & 1][lane] = 0u;
            X.clean[lane] = bad;
            st_cluster32(dsmem_addr(smem_u32(&X.clean[lane]), 1), bad);
          }
          __syncwarp();
          if (lane < 2) mbar_arrive_cluster(dsmem_addr(smem_u32(&X.clean_req), lane));
          ok = ok && all_ok(wait_phase<true>(X, X.clean_done, (uint32_t)cleaned & 1));
          ++cleaned;
        }
      }
#pragma unroll 1
      for (int n = 0; n < 4 * kParts; ++n) {
        const int b = n & 3;
        ok = ok && all_ok(wait_phase<true>(X, X.p_full[b], (uint32_t)c & 1));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ok = ok && all_ok(wait_phase(X, X.full[2 * b + h], (uint32_t)(kParts == 1 ? rev : rev + n / 4) & 1));
          if (!ok) return;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              umma_pair_bf16(tmem + 128 * h, p_d + ((b * 8192 + s * 32) >> 4),
                             v_d + (((2 * b + h) * kSlotBytes + s * 4096) >> 4), id_o, run > 0 || n > 0 || s > 0);
            umma_commit_pair(smem_u32(&X.empty[2 * b + h]));
            if (h == 1 && n >= 4 * (kParts - 1)) umma_commit_pair(smem_u32(&X.p_free[b]));
          }
          __syncwarp();
        }
      }
      rev += kParts;
    };
    int c = 0, seg = 0, run = 0;
    bool masked = false;
    // What key tile c is, read while the products of the one before are under way.
    int i = 0, kind = 0;
    auto step = [&]() {
      ok = ok && all_ok(wait_phase(X, X.step_full[c & 3], (uint32_t)(c >> 2) & 1));
      i = ok ? uniform(X.step[c & 3].i) : -1;
      kind = uniform(X.step[c & 3].kind);
    };
    step();
    while (i >= 0) {
      if (i == 0) {
        ok = all_ok(wait_phase(X, X.q_full, (uint32_t)seg & 1));
        ++seg;
      }
#pragma unroll 1
      for (int n = 0; n < kSlots * kParts; ++n) {
        const int k = kParts == 1 ? n : n & (kSlots - 1);
        ok = ok && all_ok(wait_phase(X, X.full[k], (uint32_t)(kParts == 1 ? rev : rev + n / kSlots) & 1));
        if (!ok) break;
        tc_fence_after();
        if (lead) {
#pragma unroll
          for (int s = 0; s < 4; ++s)
            umma_pair_bf16(tmem + kColS + 128 * (c & 1), q_d + ((k * 8192 + s * 32) >> 4),
                           k_d + ((k * kSlotBytes + s * 32) >> 4), id_s, n > 0 || s > 0);
          umma_commit_pair(smem_u32(&X.empty[k]));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (lead) {
        umma_commit_pair(smem_u32(&X.s_full[c & 1]));
        if (kind & kStepLast) umma_commit_pair(smem_u32(&X.q_empty));
      }
      __syncwarp();
      rev += kParts;
      if (c > 0) values(c - 1, run, masked);
      run = i & (kRun - 1);
      masked = (kind & kStepMasked) != 0;
      ++c;
      step();
    }
    if (ok) values(c - 1, run, masked);
    // no product may still be running when the tensor memory is released, whatever happened above
    if (lead) umma_commit_pair(smem_u32(&X.fin));
    __syncwarp();
    mbar_wait(smem_u32(&X.fin), 0, 100000000ull);
  } else if (work && warp == kWarpClean) {
    // ================= values that must not be read =================
    for (uint32_t n = 0;;) {
      // (a try_wait may sleep for microseconds, which would hold up the kernel's end)
      if (!mbar_test_wait(smem_u32(&X.clean_req), n & 1)) {
        if (*reinterpret_cast<volatile int*>(&X.done)) break;
        __nanosleep(200);
        continue;
      }
      mbar_try_wait_cluster(smem_u32(&X.clean_req), n & 1);  // (complete: for what the request brings)
      // row r's values: slots (r / 64, 0) and (r / 64, 1), group r % 64 / 8, two blocks of 64 dims
      for (int r = 0; r < kKeys; ++r) {
        if (!(X.clean[r >> 5] >> (r & 31) & 1u)) continue;
        const uint32_t at = ring + (uint32_t)((r >> 6) * 2 + (lane >> 4)) * kSlotBytes + ((r & 63) >> 3) * 2048 +
                            ((lane >> 3) & 1) * 1024 + (r & 7) * 128 + (lane & 7) * 16;
        uint4 v = ld_shared16(at);
        uint32_t* x = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if ((x[k] & 0x7F80u) == 0x7F80u) x[k] &= 0xFFFF0000u;
          if ((x[k] & 0x7F800000u) == 0x7F800000u) x[k] &= 0x0000FFFFu;
        }
        st_shared16(at, v);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(dsmem_addr(smem_u32(&X.clean_done), 0));
      ++n;
    }
  } else if (work && warp >= kWarpLoad) {
    // ================= loads =================
    const uint64_t pol = policy_evict_normal();
    const int k0 = warp - kWarpLoad;  // this warp's slots: k0, k0 + kLoadWarps, ..
    const uint32_t q_full = dsmem_addr(smem_u32(&X.q_full), 0), full = dsmem_addr(smem_u32(&X.full[0]), 0);
    const int lg = 31 - __clz(a.box_rows);
    bool ok = true;
    int rev = 0, c = 0, seg = 0, n_last = 0;
    int lo0 = 0, hi0 = 0, lo1 = 0, hi1 = 0;
    // Eight slots of each part, each in pieces of box_rows rows, one a lane.
    auto slots = [&](const Places& at, const CUtensorMap* map, bool values) {
      constexpr int count = kSlots * kParts;
      const int piece = lane << lg;
      const bool mine = piece < (values ? 64 : 128);
      const uint32_t dst = ring + (uint32_t)piece * (values ? 256 : 128);
      int g = (16 * (int)rank + (piece >> 3)) & 31;
      int32_t y = __shfl_sync(0xFFFFFFFFu, at.y, g), z = __shfl_sync(0xFFFFFFFFu, at.z, g);
#pragma unroll 1
      for (int n = k0; n < count; n += kLoadWarps) {
        const int k = kParts == 1 ? n : n & (kSlots - 1), r = kParts == 1 ? rev : rev + n / kSlots;
        if (values) {
          g = (8 * (k >> 1) + (piece >> 3)) & 31;
          y = __shfl_sync(0xFFFFFFFFu, at.y, g);
          z = __shfl_sync(0xFFFFFFFFu, at.z, g);
        }
        if (r > 0) ok = ok && all_ok(wait_phase(X, X.empty[k], (uint32_t)(r - 1) & 1));
        if (!ok) return;
        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(smem_u32(&X.full[k]), 2 * kSlotBytes);
        if (mine)
          tma_load_5d_pair(dst + k * kSlotBytes, map, values ? 4 * (k & 1) + 2 * (int)rank : k, y, kParts == 1 ? z : z + n / kSlots,
                           full + 8 * k, pol);
        __syncwarp();
      }
      rev += kParts;
    };
    // The places of the walk's key tile (a segment's first: with its bounds).
    auto places = [&]() {
      if (w.i == 0) tile_rows(a, w.t, lo0, hi0, lo1, hi1);
      return place_groups(a, w.t, (int64_t)(w.t.k0 + w.unit + w.i) * kKeys, lo0, hi1, lane,
                          rank == 0 && k0 == 0);
    };
    Places cur = places(), last = cur;
    bool have = true;
    while (ok && have) {
      if (k0 == 0) {
        if (w.i == 0) {
          if (seg > 0)
            ok = all_ok(wait_phase(X, X.q_empty, (uint32_t)(seg - 1) & 1,
                                   2000000000ull + 100000ull * (uint32_t)n_last));
          if (!ok) break;
          if (lane == 0) {
            if (rank == 0) mbar_arrive_expect_tx(smem_u32(&X.q_full), 2 * kQBytes);
#pragma unroll 1
            for (int k = 0; k < 8; ++k)
              tma_load_2d_pair(q_s + k * 8192, &qmap, 64 * k, w.t.row0 + (int)rank * 64, q_full, pol);
          }
          if (lane == 0)
            X.seg[seg & 3] = ChunkSegment{w.t.start, w.t.row0, w.t.rows, w.t.tok0, w.t.clip,
                                          w.t.c0 == w.t.c1, 2 * pair + (w.unit == 0 ? 1 : 0), w.t.seq};
          __syncwarp();
          ++seg;
          n_last = w.n;
        }
        const uint32_t groups = __ballot_sync(0xFFFFFFFFu, cur.good);
        if (lane == 0) {
          const int at = (w.t.k0 + w.unit + w.i) * kKeys;
          X.step[c & 3] = ChunkStep{groups, at, w.i,
                                    (w.i + 1 == w.n ? kStepLast : 0) |
                                        (at < lo1 || at + kKeys > hi0 || ~groups ? kStepMasked : 0)};
          mbar_arrive(smem_u32(&X.step_full[c & 3]));
        }
      }
      const Places now = cur;
      have = uniform(walk_next(a, w)) != 0;
      slots(now, &kmap, false);
      if (ok && c > 0) slots(last, &vmap, true);
      if (have) cur = places();  // (read while the slots issued last are still in use)
      last = now;
      ++c;
    }
    if (k0 == 0 && lane == 0) {  // (after a wait that gave up, too)
      X.step[c & 3] = ChunkStep{0u, 0, -1, 0};
      mbar_arrive(smem_u32(&X.step_full[c & 3]));
    }
    if (ok) slots(last, &vmap, true);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (X.abort) {  // copies in flight land within microseconds
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
    __syncthreads();
  }
  if (warp == kWarpMma) tmem_dealloc_pair(tmem, 512);
}

// ---- join ------------------------------------------------------------------------------
//
// A tile that pairs c0 .. c1 worked on: with M the largest running maximum (and the sink's logit) of
// a row, out = sum 2^(m - M) O / Z.  kJoin CTAs a tile, a thread 16 bytes of every part at a time.  Bound by
// the parts' way from L2.
// At most kJoinFew tiles at a time after a small plan: a CTA without a tile takes its time, too.
constexpr int kJoin = 64, kJoinFew = 16;

__global__ void __launch_bounds__(256) chunk_join_kernel(ChunkArgs a) {
  __shared__ float wt[kMaxPairs][64];
  __shared__ float red[3][4][64];
  __shared__ float inv[64];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, splits = a.split[0];
  for (int y = blockIdx.y; y < splits; y += gridDim.y) {
    const ChunkTile t = a.tile[a.split[1 + y]];
    const int n = min(t.c1 - t.c0 + 1, kMaxPairs);
    const int rank = blockIdx.x / (kJoin / 2);  // the CTA whose 64 rows these are
    auto slot = [&](int i) -> int64_t { return (2 * (int64_t)(t.c0 + i) + (i == 0 ? 1 : 0)) * 2 + rank; };
    const int row = tid & 63, quarter = tid >> 6, r = 64 * rank + row;
    const int grow = t.row0 + min(r, t.rows - 1), h = grow % a.H;
    const bool live = r < t.rows;
    {
      float m = -INFINITY;
      for (int i = quarter; i < n; i += 4) {
        const float x = a.pstat[slot(i) * 192 + row];
        wt[i][row] = x;
        m = fmaxf(m, x);
      }
      red[0][quarter][row] = m;
      __syncthreads();
      const float logit = a.sink ? a.sink[h] : -INFINITY, sink = sink_log2(logit);
      float M = sink;
  #pragma unroll
      for (int k = 0; k < 4; ++k) M = fmaxf(M, red[0][k][row]);
      const float Mf = M == -INFINITY ? 0.f : M;
      float l = 0.f, z = 0.f;
      for (int i = quarter; i < n; i += 4) {
        const float e = ex2(wt[i][row] - Mf);
        wt[i][row] = e;
        l = fmaf(e, a.pstat[slot(i) * 192 + 64 + row], l);
        z = fmaf(e, a.pstat[slot(i) * 192 + 128 + row], z);
      }
      red[1][quarter][row] = l;
      red[2][quarter][row] = z;
      __syncthreads();
      if (quarter == 0) {
        l = red[1][0][row] + red[1][1][row] + red[1][2][row] + red[1][3][row];
        z = red[2][0][row] + red[2][1][row] + red[2][2][row] + red[2][3][row];
        const float rows = l;
        if (sink > -INFINITY) {
          l += ex2(sink - Mf);
          z += ex2(sink - Mf);
        }
        inv[row] = z > 0.f || z != z ? 1.f / z : 0.f;
        if (a.lse && live && blockIdx.x % (kJoin / 2) == 0) a.lse[grow] = head_lse(Mf, l, rows, logit);
      }
      __syncthreads();
    }
    // 8192 float4 of this CTA's rows, columns by kJoin / 2 CTAs
    for (int x = (blockIdx.x % (kJoin / 2)) * 256 + tid; x < 8192; x += 256 * (kJoin / 2)) {
      const int L = x & 127, col = x >> 7;
      const float4* p = reinterpret_cast<const float4*>(a.part) + col * 128 + L;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  #pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float4 v = p[slot(i) * 8192];
        const float e = wt[i][row];
        // (a part that saw nothing has weight zero and may hold anything finite)
        o.x = fmaf(v.x, e, o.x);
        o.y = fmaf(v.y, e, o.y);
        o.z = fmaf(v.z, e, o.z);
        o.w = fmaf(v.w, e, o.w);
      }
      const int d = (col >> 5) * 256 + (L >> 6) * 128 + ((col >> 4) & 1) * 64 + 4 * (col & 15);
      const float f = inv[row];
      o.x *= f;
      o.y *= f;
      o.z *= f;
      o.w *= f;
      if (a.inv_freq && d >= kRopeDim0) {
        const uint64_t pos = (uint64_t)(t.start + (grow / a.H - t.tok0));
        float sn, cs;
        sincosf(rope_angle(rope_turn(a.inv_freq[(d - kRopeDim0) >> 1]), pos), &sn, &cs);
        float z = o.x * cs + o.y * sn;
        o.y = o.y * cs - o.x * sn;
        o.x = z;
        sincosf(rope_angle(rope_turn(a.inv_freq[((d - kRopeDim0) >> 1) + 1]), pos), &sn, &cs);
        z = o.z * cs + o.w * sn;
        o.w = o.w * cs - o.z * sn;
        o.z = z;
      }
      if (live)
        *reinterpret_cast<uint2*>(a.out + (int64_t)grow * kDLat + d) =
            make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    }
    __syncthreads();  // wt and inv are read
  }
}
}  // namespace

namespace {

template <int kMode>
cudaError_t launch_read(const PagedReadArgs& a, int sms, cudaStream_t s) {
  // Runs of up to 32 rows, as many to each warp of a grid that stays.
  const int64_t most = (int64_t)sms * read_ctas(kMode), warps = most * kReadWarps, passes = ((int64_t)a.T + warps * 32 - 1) / (warps * 32);
  const int run = (int)(((int64_t)a.T + warps * passes - 1) / (warps * passes));
  const int64_t need = ((int64_t)a.T + kReadWarps * run - 1) / (kReadWarps * run);
  const dim3 grid((unsigned)(need < most ? need : most));
  return run >= 4 ? launch_pdl(paged_read_kernel<kMode, 4>, grid, dim3(kReadWarps * 32), 0, s, a, run)
                  : launch_pdl(paged_read_kernel<kMode, 1>, grid, dim3(kReadWarps * 32), 0, s, a, run);
}

}  // namespace

cudaError_t launch_paged_read(const PagedReadArgs& a, int sms, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  return a.cache.dtype == 0   ? launch_read<0>(a, sms, s)
         : a.cache.dtype == 1 ? launch_read<1>(a, sms, s)
                              : launch_read<2>(a, sms, s);
}

int chunk_max_pairs() { return kMaxPairs; }
int chunk_whole_keys() { return kWhole; }

cudaError_t launch_chunk_attn(const ChunkArgs& a, int sms, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  CUtensorMap qm, km, vm;
  if (!encode_rows_bf16(&qm, a.q, (uint64_t)a.T * a.H, kDLat, 64, 64)) return cudaErrorInvalidValue;
  // a page (or all staged rows) as [8-row groups][8 dim blocks][8 rows][128 bytes]
  const uint64_t groups = a.stage ? (uint64_t)a.stage_rows / 8 : (uint64_t)a.cache.page_rows / 8;
  const uint64_t dims[5] = {128, 8, 8, groups, a.stage ? (uint64_t)a.parts : (uint64_t)a.cache.n_pages};
  const uint64_t strides[4] = {1024, 128, 8192,
                               a.stage ? groups * 8192 : (uint64_t)a.cache.page_stride};
  const uint32_t kbox[5] = {128, 8, 1, (uint32_t)a.box_rows / 8, 1};
  const uint32_t vbox[5] = {128, 8, 2, (uint32_t)a.box_rows / 8, 1};
  const void* rows = a.stage ? (const void*)a.stage : (const void*)a.cache.data;
  if (!encode_bytes(&km, rows, 5, dims, strides, kbox) || !encode_bytes(&vm, rows, 5, dims, strides, vbox))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (!a.alone)
    e = a.max_tiles <= kPlanFew && a.cache.B <= kPlanFew
            ? launch_pdl(chunk_plan_kernel<kPlanFew>, dim3(1), dim3(kPlanFew), 0, s, a)
            : launch_pdl(chunk_plan_kernel<kPlanThreads>, dim3(1), dim3(kPlanThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  if (a.stage) {
    PagedReadArgs r{};
    r.out = a.stage;
    r.out_ld = kDLat;
    r.low = a.parts == 2 ? a.stage + a.stage_rows * kDLat : nullptr;
    r.T = (int)a.stage_rows;
    r.row_end = a.stage_end;
    r.cu_seqlens = a.stage_cu;
    r.start_row = a.stage_first;
    r.ratio = 1;
    r.cache = a.cache;
    r.cap_rows = a.cap_rows;
    r.page_mul = a.page_mul;
    r.page_shift = a.page_shift;
    e = launch_paged_read(r, sms, s);
    if (e != cudaSuccess) return e;
  }
  auto kern = a.alone            ? chunk_attn_kernel<true, 1>
              : a.parts == 1 ? chunk_attn_kernel<false, 1>
                                 : chunk_attn_kernel<false, 2>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl_cluster(kern, dim3(2u * a.pairs), dim3(kThreads), kSmem, s, 2u, a, qm, km, vm);
  if (e != cudaSuccess || !a.part) return e;
  const int few = a.max_tiles <= kPlanFew ? kJoinFew : a.pairs, y = a.max_tiles < few ? a.max_tiles : few;
  return launch_pdl(chunk_join_kernel, dim3(kJoin, (unsigned)y), dim3(256), 0, s, a);
}

}  // namespace csa2
