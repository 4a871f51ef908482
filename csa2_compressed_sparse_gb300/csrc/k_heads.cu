// k_heads.cu -- the norm of queries and keys for each head, with the rotation of the token's
// position in the same pass (qk_norm_rope_kernel).
//
// A row is a token's head: y = x / sqrt(mean x^2 + eps) * w in fp32, then R of its dims from r0 on
// rotated, pair i by the angle p theta_i (the phase exact, as in the compressor) and scaled by
// `factor`, rounded once to bf16.  Pairs are neighbours (2 i, 2 i + 1) or halves (i, i + R / 2).
//
// A group of kG lanes has a row, a lane kC 16-byte chunks of it (chunk lane + 32 c), so a warp
// reads whole rows in order; kU rows a lane are loaded at once.  The angles of a lane's dims are
// computed once per item, which is a token and up to `rows` of its heads.
#include "common.cuh"
#include "compress_dev.cuh"

namespace csa2 {
namespace {

constexpr int kWarps = 8;

template <int kG, int kC, bool kHalf, int kU>
__global__ void __launch_bounds__(kWarps * 32) qk_norm_rope_kernel(HeadsArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kRows = 32 / kG;          // rows side by side in a warp
  constexpr int kPairs = kHalf ? 8 : 4;   // angles of a chunk
  const int lane = threadIdx.x & 31, sub = lane / kG, l = lane % kG;
  const int half = a.rope_dims >> 1;
  // a lane's chunks: first dim, whether it exists, whether it is rotated, and its pairs' steps
  int dim[kC], mate[kC];
  bool have[kC], rot[kC];
  float sign[kC];
  uint64_t turn[kC][kPairs];
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    dim[c] = 8 * (l + 32 * c);
    have[c] = dim[c] < a.D;
    const int e = dim[c] - a.rope_dim0;
    rot[c] = have[c] && e >= 0 && e < a.rope_dims;
    // halves: the chunk with the other dims of the pairs; -x1 s for the first, + x0 s for the second
    mate[c] = dim[c] + (e < half ? half : -half);
    sign[c] = e < half ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
      turn[c][i] = rot[c] ? rope_turn(a.inv_freq[kHalf ? (e < half ? e : e - half) + i : e / 2 + i]) : 0;
  }
  const int64_t nq = (a.q.H + a.rows - 1) / a.rows, nk = (a.k.H + a.rows - 1) / a.rows;
  const int64_t items = (nq + nk) * a.T, step = (int64_t)gridDim.x * kWarps;
  for (int64_t it = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); it < items; it += step) {
    const int64_t t = it / (nq + nk);
    int64_t blk = it - t * (nq + nk);
    const HeadSet& s = blk < nq ? a.q : a.k;
    if (blk >= nq) blk -= nq;
    const int h0 = (int)blk * a.rows, h1 = min(s.H, h0 + a.rows);
    const uint16_t* x = s.x + t * s.x_token;
    uint16_t* out = s.out + t * s.out_token;
    const uint64_t p = a.rope_dims > 0 ? (uint64_t)a.pos[t] : 0;
    float cs[kC][kPairs], sn[kC][kPairs], w[kC][8], wm[kC][8];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[c][i] = wm[c][i] = 1.f;
      if (have[c] && s.norm_w) cdev::load8_f32(s.norm_w + dim[c], w[c]);
      if (!rot[c]) continue;
      if (kHalf && s.norm_w) cdev::load8_f32(s.norm_w + mate[c], wm[c]);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        sincosf(rope_angle(turn[c][i], p), &sn[c][i], &cs[c][i]);
        cs[c][i] *= a.factor;
        sn[c][i] *= a.factor;
      }
    }
    for (int h = h0; h < h1; h += kRows * kU) {
      uint4 v[kU][kC], m[kU][kHalf ? kC : 1];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int r = h + u * kRows + sub;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          v[u][c] = make_uint4(0u, 0u, 0u, 0u);
          if (r < h1 && have[c])
            v[u][c] = __ldcs(reinterpret_cast<const uint4*>(x + r * s.x_head + dim[c]));
          if (kHalf && r < h1 && rot[c])
            m[u][c] = *reinterpret_cast<const uint4*>(x + r * s.x_head + mate[c]);
        }
      }
      __syncwarp();  // every lane has its part of these rows: they may be written over in place
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int r = h + u * kRows + sub;
        float y[kC][8];
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          unpack_bf16x8(v[u][c], y[c]);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(y[c][i], y[c][i], ss);
        }
#pragma unroll
        for (int o = kG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float rstd = s.norm ? 1.0f / sqrtf(ss / (float)a.D + a.eps) : 1.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[c][i] *= rstd * w[c][i];
          if (rot[c]) {
            if (kHalf) {
              float z[8];
              unpack_bf16x8(m[u][c], z);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                y[c][i] = y[c][i] * cs[c][i] + sign[c] * (z[i] * (rstd * wm[c][i])) * sn[c][i];
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float x0 = y[c][2 * i], x1 = y[c][2 * i + 1];
                y[c][2 * i] = x0 * cs[c][i] - x1 * sn[c][i];
                y[c][2 * i + 1] = x0 * sn[c][i] + x1 * cs[c][i];
              }
            }
          }
          if (r < h1 && have[c]) {
            const uint4 o = make_uint4(pack_bf16x2(y[c][0], y[c][1]), pack_bf16x2(y[c][2], y[c][3]),
                                       pack_bf16x2(y[c][4], y[c][5]), pack_bf16x2(y[c][6], y[c][7]));
            __stcs(reinterpret_cast<uint4*>(out + r * s.out_head + dim[c]), o);
          }
        }
      }
    }
  }
}

template <int kG, int kC, bool kHalf>
cudaError_t launch_rows(HeadsArgs a, int sms, cudaStream_t s) {
  constexpr int kU = 4, kRows = 32 / kG;
  // heads of an item: as many as leave every SM some 32 warps' worth of items
  const int64_t heads = (int64_t)a.q.H + a.k.H;
  int rows = 16 * kRows;
  while (rows > kRows && a.T * ((heads + rows - 1) / rows) < (int64_t)sms * 32) rows >>= 1;
  a.rows = rows;
  const int64_t items = a.T * (((int64_t)a.q.H + rows - 1) / rows + ((int64_t)a.k.H + rows - 1) / rows);
  const int64_t need = (items + kWarps - 1) / kWarps, most = (int64_t)sms * 8;
  const dim3 grid((unsigned)(need < most ? need : most));
  if (rows >= kU * kRows)
    return launch_pdl(qk_norm_rope_kernel<kG, kC, kHalf, kU>, grid, dim3(kWarps * 32), 0, s, a);
  return launch_pdl(qk_norm_rope_kernel<kG, kC, kHalf, 1>, grid, dim3(kWarps * 32), 0, s, a);
}

template <int kG, int kC>
cudaError_t launch_layout(const HeadsArgs& a, int sms, cudaStream_t s) {
  return a.halves ? launch_rows<kG, kC, true>(a, sms, s) : launch_rows<kG, kC, false>(a, sms, s);
}

}  // namespace

cudaError_t launch_heads(const HeadsArgs& a, int sms, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  return a.D <= 64    ? launch_layout<8, 1>(a, sms, s)
         : a.D <= 128 ? launch_layout<16, 1>(a, sms, s)
         : a.D <= 256 ? launch_layout<32, 1>(a, sms, s)
                      : launch_layout<32, 2>(a, sms, s);
}

}  // namespace csa2
