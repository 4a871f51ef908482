// k_heads.cu -- the norm of queries and keys for each head, with the rotation of the token's
// position in the same pass (qk_norm_rope_kernel).
//
// A row is a token's head: y = x / sqrt(mean x^2 + eps) * w in fp32, then R of its dims from r0 on
// rotated, pair i by the angle p theta_i (the phase exact, as in the compressor) and scaled by
// `factor`, rounded once to bf16.  Pairs are neighbours (2 i, 2 i + 1) or halves (i, i + R / 2).
//
// A group of kG lanes has a row, a lane kC 16-byte chunks of it (chunk lane + 32 c), so a warp reads
// whole rows in order.  A warp takes an item, a token's rows or a run of them, a row a lane at a time,
// the next one loaded before this is written; the token's angles it computes once, through shared
// memory.  Angular steps (64-bit floating point, of which an SM does two a cycle) are computed once a CTA.
// Bound by the bytes moved: 4096 tokens of 65 heads of 512 take 98 us (5.6 of 6.8 TB/s; what is missing is
// bytes in flight, a row and the next two of each of 24 warps an SM), 64 tokens the launch and a chain of latencies (7 us).
//
// The attention of the sparse step reads its queries and window rows before its dependency wait, and this
// kernel is what writes them: it lets no dependent start before its CTAs have ended (of calls in a row, 1001 tokens
// of 65 heads of 128 take 14.7 us in place of 14.1, 4096 of 512 98.7 in place of 98.1).
#include "common.cuh"
#include "compress_dev.cuh"

namespace csa2 {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxPairs = 256;

// Two bf16 values in fp32, and back.
__device__ __forceinline__ float2 wide2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// CTAs of an SM, by registers: halves of wide heads take more, and so do two rows ahead
template <int kC, bool kHalf, bool kTwo>
constexpr int kCtas = kC == 1 ? 4 : kHalf ? 2 : kTwo ? 3 : 4;

// kTwo: the next two rows are loaded ahead, not one.
template <int kG, int kC, bool kHalf, bool kTwo>
__global__ void __launch_bounds__(kWarps * 32, kCtas<kC, kHalf, kTwo>) qk_norm_rope_kernel(HeadsArgs a) {
  __shared__ uint64_t turn_s[kMaxPairs];
  __shared__ __align__(16) float cs_s[kWarps][kMaxPairs], sn_s[kWarps][kMaxPairs];
  griddep_wait();
  constexpr int kRows = 32 / kG;  // rows of a unit
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane / kG, l = lane % kG;
  const int half = a.rope_dims >> 1;
  const float inv_d = 1.f / (float)a.D;
  if (tid < half) turn_s[tid] = rope_turn(a.inv_freq[tid]);
  __syncthreads();
  // a lane's chunks: first dim, whether it exists, whether it is rotated, its pairs
  int dim[kC], mate[kC], pair[kC];
  bool have[kC], rot[kC];
  float sign[kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    dim[c] = 8 * (l + 32 * c);
    have[c] = dim[c] < a.D;
    const int e = dim[c] - a.rope_dim0;
    rot[c] = have[c] && e >= 0 && e < a.rope_dims;
    // halves: the chunk with the other dims of the pairs; -x1 s for the first, + x0 s for the second
    mate[c] = dim[c] + (e < half ? half : -half);
    sign[c] = e < half ? -1.f : 1.f;
    pair[c] = rot[c] ? (kHalf ? (e < half ? e : e - half) : e / 2) : 0;
  }
  const int nq = (a.q.H + kRows - 1) / kRows, nk = (a.k.H + kRows - 1) / kRows;
  const int blocks = (nq + nk + a.units - 1) / a.units;
  const int64_t items = (int64_t)a.T * blocks, step = (int64_t)gridDim.x * kWarps;
  for (int64_t it = (int64_t)blockIdx.x * kWarps + warp; it < items; it += step) {
    const int64_t t = it / blocks;
    const int u0 = (int)(it - t * blocks) * a.units, u1 = min(nq + nk, u0 + a.units);
    uint4 v[kC], m[kHalf ? kC : 1], vn[kC], mn[kHalf ? kC : 1], vf[kTwo ? kC : 1];
    auto fetch = [&](int u, uint4(&x)[kC], uint4(&y)[kHalf ? kC : 1]) {
      const bool q = u < nq;
      const HeadSet& s = q ? a.q : a.k;
      const int r = (q ? u : u - nq) * kRows + sub;
      const uint16_t* src = s.x + t * s.x_token + r * s.x_head;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        x[c] = make_uint4(0u, 0u, 0u, 0u);
        if (r < s.H && have[c]) x[c] = __ldcs(reinterpret_cast<const uint4*>(src + dim[c]));
        if (kHalf && r < s.H && rot[c]) y[kHalf ? c : 0] = *reinterpret_cast<const uint4*>(src + mate[c]);
      }
    };
    fetch(u0, v, m);
    if (kTwo && u0 + 1 < u1) fetch(u0 + 1, vn, mn);
    if (half > 0) {
      const uint64_t p = (uint64_t)a.pos[t];
      __syncwarp();  // the last token's angles are read
      for (int i = lane; i < half; i += 32) {
        float s, c;
        sincosf(rope_angle(turn_s[i], p), &s, &c);
        cs_s[warp][i] = c * a.factor;
        sn_s[warp][i] = s * a.factor;
      }
      __syncwarp();
    }
    float2 w[kC][4], wm[kHalf ? kC : 1][4];  // the set's weights, of the lane's dims and their mates
#pragma unroll 1
    for (int u = u0; u < u1; ++u) {
      const bool q = u < nq;
      const HeadSet& s = q ? a.q : a.k;
      const int r = (q ? u : u - nq) * kRows + sub;
      uint16_t* out = s.out + t * s.out_token + r * s.out_head;
      if constexpr (kTwo) {
        if (u + 2 < u1) fetch(u + 2, vf, mn);
      } else {
        if (u + 1 < u1) fetch(u + 1, vn, mn);
      }
      if (u == u0 || u == nq) {
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const bool use = have[c] && s.norm_w;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            w[c][k] = use ? *reinterpret_cast<const float2*>(s.norm_w + dim[c] + 2 * k) : make_float2(1.f, 1.f);
            if (kHalf)
              wm[kHalf ? c : 0][k] = use && rot[c] ? *reinterpret_cast<const float2*>(s.norm_w + mate[c] + 2 * k)
                                                   : make_float2(1.f, 1.f);
          }
        }
      }
      __syncwarp();  // every lane has its part of these rows: they may be written over in place
      float2 ss = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 y = wide2(word(v[c], k));
          ss = fma2(y, y, ss);
        }
      float sum = ss.x + ss.y;
#pragma unroll
      for (int o = kG / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      // (rsqrtf is within 2 units: 2^-22)
      const float rstd = s.norm ? rsqrtf(fmaf(sum, inv_d, a.eps)) : 1.f;
      const float2 rr = make_float2(rstd, rstd);
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        float2 y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = mul2(mul2(wide2(word(v[c], k)), rr), w[c][k]);
        if (rot[c]) {
          const float4* cs = reinterpret_cast<const float4*>(&cs_s[warp][pair[c]]);
          const float4* sn = reinterpret_cast<const float4*>(&sn_s[warp][pair[c]]);
          if (kHalf) {
            const float2 sg = make_float2(sign[c], sign[c]);
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const float4 co = cs[k >> 1], si = sn[k >> 1];
              const float2 z0 = mul2(mul2(wide2(word(m[kHalf ? c : 0], k)), rr), wm[kHalf ? c : 0][k]);
              const float2 z1 = mul2(mul2(wide2(word(m[kHalf ? c : 0], k + 1)), rr), wm[kHalf ? c : 0][k + 1]);
              y[k] = fma2(mul2(z0, sg), make_float2(si.x, si.y), mul2(y[k], make_float2(co.x, co.y)));
              y[k + 1] = fma2(mul2(z1, sg), make_float2(si.z, si.w), mul2(y[k + 1], make_float2(co.z, co.w)));
            }
          } else {
            const float4 co = cs[0], si = sn[0];
            const float cc[4] = {co.x, co.y, co.z, co.w}, sc[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              y[k] = make_float2(y[k].x * cc[k] - y[k].y * sc[k], y[k].x * sc[k] + y[k].y * cc[k]);
          }
        }
        if (r < s.H && have[c])
          __stcs(reinterpret_cast<uint4*>(out + dim[c]),
                 make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y),
                            pack_bf16x2(y[2].x, y[2].y), pack_bf16x2(y[3].x, y[3].y)));
      }
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        v[c] = vn[c];
        if (kTwo) vn[c] = vf[kTwo ? c : 0];
        if (kHalf) m[kHalf ? c : 0] = mn[kHalf ? c : 0];
      }
    }
  }
  __threadfence();  // (what ends a CTA need not make its rows visible to what starts then)
}

template <int kG, int kC, bool kHalf>
cudaError_t launch_rows(HeadsArgs a, int sms, cudaStream_t s) {
  constexpr int kRows = 32 / kG;
  // Much work on heads that fill a warp has two rows ahead (4096 tokens of 65 heads of 512 103 -> 98 us, 5000
  // 127 -> 116, heads of 192 and 256 10 % less; little work took 13.8 in place of 13.0, narrower heads as long
  // or up to 9 % longer, and so halves of any width, whose rows take twice the registers).
  constexpr bool kTwo = kG == 32 && !kHalf;
  const int units = (a.q.H + kRows - 1) / kRows + (a.k.H + kRows - 1) / kRows;
  // Much work goes in runs of which the GPU's warps take at least two each, the last ones as nearly at the same
  // time as may be; what begins a run counts as a unit of 1 KiB, or three of fewer bytes.  Of 65 heads of 512,
  // 5000 tokens took 173 us with a token's rows to a warp (one each, and 136 over) and 127 so.
  constexpr int kStart = kC == 2 ? 1 : 3;
  const int64_t cap = (int64_t)sms * kCtas<kC, kHalf, kTwo> * kWarps;
  int64_t best = INT64_MAX;
  a.units = units;
  for (int blocks = 1; (int64_t)a.T * units >= 8 * cap && blocks <= 16 && blocks <= units; ++blocks) {
    const int n = (units + blocks - 1) / blocks;
    const int64_t rounds = ((int64_t)a.T * ((units + n - 1) / n) + cap - 1) / cap;
    if (rounds > 1 && rounds * (n + kStart) < best) {
      best = rounds * (n + kStart);
      a.units = n;
    }
  }
  // Otherwise: a token's rows to a warp, or as few of them as it takes to give each SM some 24 warps.
  const bool much = best != INT64_MAX;
  while (!much && a.units > 1 && (int64_t)a.T * ((units + a.units - 1) / a.units) < (int64_t)sms * 24)
    a.units = (a.units + 1) / 2;
  const int64_t items = (int64_t)a.T * ((units + a.units - 1) / a.units);
  const int64_t need = (items + kWarps - 1) / kWarps;
  const int64_t most = (int64_t)sms * (much ? kCtas<kC, kHalf, kTwo> : kCtas<kC, kHalf, false>);
  return launch_pdl(much ? qk_norm_rope_kernel<kG, kC, kHalf, kTwo> : qk_norm_rope_kernel<kG, kC, kHalf, false>,
                    dim3((unsigned)(need < most ? need : most)), dim3(kWarps * 32), 0, s, a);
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
