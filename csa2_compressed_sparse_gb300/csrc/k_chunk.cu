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
// The inverse of paged_append_kernel, laid out as it is: a warp per row, kTok rows at a time; a lane
// holds the chunks `lane` (dims 8 l ..) and, below lane 24, 32 + lane (dims 256 + 8 l ..), and the
// rotation pair 448 + 2 l, 449 + 2 l.  x = code * scale in fp32, rounded once to bf16 (exact for
// FP8_E8M0 scales of 2^-124 to 2^119).  Bound by the bytes moved: 1024 or 528 read, 1024 written per row.

constexpr int kReadWarps = 8;
constexpr int kReadCtas = 6;

__device__ __forceinline__ float2 e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Eight codes times a scale, to bf16.
__device__ __forceinline__ uint4 decode8(uint2 c, float s) {
  uint32_t r[4];
  const uint32_t w[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = e4m3x2(w[i]);
    r[i] = pack_bf16x2(v.x * s, v.y * s);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ float e8m0_scale(uint32_t e) {  // 2^(e - 127); 255 is NaN
  return e == 0 ? __uint_as_float(0x00400000u) : e == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(e << 23);
}

template <int kTok>
__global__ void __launch_bounds__(kReadWarps * 32) paged_read_kernel(PagedReadArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * kReadWarps * kTok;
  const uint64_t turn = a.inv_freq ? rope_turn(a.inv_freq[lane]) : 0;
  const int64_t total = min((int64_t)a.T, (int64_t)a.cu_seqlens[a.cache.B]);
  for (int64_t t = ((int64_t)blockIdx.x * kReadWarps + (threadIdx.x >> 5)) * kTok; t < total; t += step) {
    // where the rows are
    const uint8_t* src[kTok];
    int64_t j[kTok];
    int b = cdev::warp_find_seq(a.cu_seqlens, a.cache.B, t, lane);
    int64_t t0 = a.cu_seqlens[b], t1 = a.cu_seqlens[b + 1], first = a.start_row[b];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      src[i] = nullptr;
      if (t + i >= total) continue;
      if (i > 0 && t + i >= t1) {  // on to the row's sequence
        b = cdev::warp_find_seq(a.cu_seqlens, a.cache.B, t + i, lane);
        t0 = a.cu_seqlens[b];
        t1 = a.cu_seqlens[b + 1];
        first = a.start_row[b];
      }
      j[i] = first + (t + i - t0);
      int32_t page = -1, row = 0;
      if (j[i] >= 0 && j[i] < a.cap_rows) {
        const int32_t lp = (int32_t)(__umulhi((uint32_t)j[i], a.page_mul) >> a.page_shift);
        row = (int32_t)j[i] - lp * a.cache.page_rows;
        page = a.cache.table[(int64_t)b * a.cache.table_ld + lp];
      }
      if (page < 0 || page >= a.cache.n_pages) {
        if (lane == 0) raise_fault(kFaultBounds);
        continue;
      }
      src[i] = a.cache.data + (int64_t)page * a.cache.page_stride +
               (int64_t)row * (a.cache.dtype == 0 ? 1024 : 528);
    }
    uint4 c0[kTok], c1[kTok];
    float x0[kTok], x1[kTok];
    if (a.cache.dtype == 0) {
      uint32_t pr[kTok];
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        if (!src[i]) continue;
        c0[i] = __ldcs(reinterpret_cast<const uint4*>(src[i]) + lane);
        if (lane < 24) c1[i] = __ldcs(reinterpret_cast<const uint4*>(src[i]) + 32 + lane);
        pr[i] = __ldcs(reinterpret_cast<const uint32_t*>(src[i] + 2 * kRopeDim0) + lane);
      }
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        x0[i] = __uint_as_float(pr[i] << 16);
        x1[i] = __uint_as_float(pr[i] & 0xFFFF0000u);
      }
    } else {
      uint2 d0[kTok], d1[kTok];
      uint32_t pr[kTok];
      float s0[kTok], s1[kTok], sr[kTok];
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        if (!src[i]) continue;
        d0[i] = __ldcs(reinterpret_cast<const uint2*>(src[i]) + lane);
        if (lane < 24) d1[i] = __ldcs(reinterpret_cast<const uint2*>(src[i] + 256) + lane);
        pr[i] = __ldcs(reinterpret_cast<const uint16_t*>(src[i] + kRopeDim0) + lane);
        if (a.cache.dtype == 1) {
          const float* sc = reinterpret_cast<const float*>(src[i] + 512);
          s0[i] = sc[lane >> 4];
          s1[i] = sc[2 + (lane >> 4)];
          sr[i] = sc[3];
        } else {
          const uint8_t* sc = src[i] + 512;
          s0[i] = e8m0_scale(sc[lane >> 2]);
          s1[i] = e8m0_scale(sc[8 + (lane >> 2)]);
          sr[i] = e8m0_scale(sc[14 + (lane >> 4)]);
        }
      }
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        if (!src[i]) continue;
        c0[i] = decode8(d0[i], s0[i]);
        if (lane < 24) c1[i] = decode8(d1[i], s1[i]);
        const float2 v = e4m3x2(pr[i]);
        x0[i] = v.x * sr[i];
        x1[i] = v.y * sr[i];
      }
    }
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      if (!src[i]) continue;
      if (a.inv_freq) {  // times e^{-i p theta}
        float s, c;
        sincosf(rope_angle(turn, (uint64_t)j[i] * (uint64_t)a.ratio), &s, &c);
        const float y0 = x0[i] * c + x1[i] * s;
        x1[i] = x1[i] * c - x0[i] * s;
        x0[i] = y0;
      }
      uint16_t* dst = a.out + (t + i) * a.out_ld;
      *(reinterpret_cast<uint4*>(dst) + lane) = c0[i];
      if (lane < 24) *(reinterpret_cast<uint4*>(dst) + 32 + lane) = c1[i];
      *(reinterpret_cast<uint32_t*>(dst + kRopeDim0) + lane) = pack_bf16x2(x0[i], x1[i]);
    }
  }
}

// ================================ chunk =================================================

// The sequence and position of each token, for attention token by token.
__global__ void __launch_bounds__(256) chunk_tokens_kernel(ChunkArgs a, int32_t* q_seq, int64_t* q_pos) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int b = cdev::warp_find_seq(a.cu_seqlens, a.cache.B, t, lane);
  const int64_t t0 = a.cu_seqlens[b];
  const bool live = t >= t0 && t < a.cu_seqlens[b + 1];
  if (lane == 0) {
    q_seq[t] = live ? b : -1;
    q_pos[t] = live ? a.start_pos[b] + (t - t0) : 0;
  }
}

}  // namespace

cudaError_t launch_paged_read(const PagedReadArgs& a, int sms, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (a.T >= 8 * kReadWarps * sms) {
    const int64_t need = (a.T + 4 * kReadWarps - 1) / (4 * kReadWarps), most = (int64_t)sms * kReadCtas;
    return launch_pdl(paged_read_kernel<4>, dim3((unsigned)(need < most ? need : most)),
                      dim3(kReadWarps * 32), 0, s, a);
  }
  return launch_pdl(paged_read_kernel<1>, dim3((unsigned)((a.T + kReadWarps - 1) / kReadWarps)),
                    dim3(kReadWarps * 32), 0, s, a);
}

cudaError_t launch_chunk_tokens(const ChunkArgs& a, int32_t* q_seq, int64_t* q_pos, cudaStream_t s) {
  return launch_pdl(chunk_tokens_kernel, dim3((unsigned)((a.T + 7) / 8)), dim3(256), 0, s, a, q_seq, q_pos);
}

}  // namespace csa2
