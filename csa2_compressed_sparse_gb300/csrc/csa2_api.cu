// csa2_api.cu -- the extern "C" entry points declared in include/csa2.h: argument
// validation on the host, workspace layout, kernel dispatch and error reporting.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include <cudaTypedefs.h>

#include "../../include/csa2.h"
#include "common.cuh"

namespace {

thread_local std::string g_last_error;

csa2_status fail(csa2_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

csa2_status cuda_fail(cudaError_t e, const char* where) {
  return fail(CSA2_ECUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned_to(size_t n, const void* p) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool aligned16(const void* p) { return aligned_to(16, p); }

#define REQUIRE(cond, ...)                         \
  do {                                             \
    if (!(cond)) return fail(CSA2_EINVAL, __VA_ARGS__); \
  } while (0)

int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace of csa2_index_topk.
struct IndexWs {
  size_t keys, n_scored, grp, cta, n_groups, count, part, total;
  int nchunk;
  // candidate pool (nbk > 0): merge counters and partial lists of the block selection
  size_t pcount, ppart;
  // FP8 plane (qrows > 0): the quantised queries and their scales
  size_t q8, qscale;
  int64_t nb_max;
  int pnchunk;
};

// Blocks of 8 positions in a row of ld positions.
int64_t pool_blocks(int64_t ld) { return (ld + 7) / 8; }

// Chunks of the candidate-block selection.  A chunk CTA reads 8 position keys per block;
// when few queries have long rows (a long-context decode batch) most SMs would idle
// while a handful of CTAs each stream 1 MiB, so the rows are cut into chunks of 8192
// blocks (256 KiB of keys) as long as the merge holds their lists and the chunks fit
// twice over on the SMs; otherwise chunks of up to 32768 blocks.  sms == 0 gives the
// most chunks any call can use (for the workspace size).
int pool_chunks(int64_t nb, int nbk, int Q, int sms) {
  const int big = csa2::topk_num_chunks(nb);
  const int64_t small = (nb + 8191) / 8192;
  if (small > big && small * nbk <= 32768 && (sms == 0 || (int64_t)Q * small <= 2 * sms))
    return (int)small;
  return big;
}

IndexWs index_ws_layout(int Q, int64_t ld, int k, int nbk = 0, int64_t qrows = 0) {
  IndexWs w{};
  size_t o = 0;
  w.keys = o; o = up256(o + (size_t)Q * (size_t)((ld + 3) & ~int64_t(3)) * 4);
  w.n_scored = o; o = up256(o + (size_t)Q * 4);
  w.grp = o; o = up256(o + (size_t)Q * sizeof(csa2::GroupRec));
  w.cta = o; o = up256(o + (size_t)csa2::kMaxIndexCtas * sizeof(csa2::CtaRec));
  w.n_groups = o; o = up256(o + 8);
  w.count = o; o = up256(o + (size_t)Q * 4);
  w.nchunk = csa2::topk_row_num_chunks(ld);
  w.part = o;
  if (w.nchunk > 1) o = up256(o + (size_t)Q * w.nchunk * k * 8);
  if (nbk > 0) {
    w.nb_max = pool_blocks(ld);
    w.pnchunk = pool_chunks(w.nb_max, nbk, Q, 0);
    w.pcount = o; o = up256(o + (size_t)Q * 4);
    w.ppart = o;
    if (w.pnchunk > 1) o = up256(o + (size_t)Q * w.pnchunk * nbk * 8);
  }
  if (qrows > 0) {
    w.q8 = o; o = up256(o + (size_t)qrows * 128);
    w.qscale = o; o = up256(o + (size_t)qrows * 4);
  }
  w.total = o;
  return w;
}

// csa2_topk_scores: per-row arrival counters, then the partial lists.
size_t topk_ws_bytes(int Q, int64_t ld, int k) {
  const int nchunk = csa2::topk_row_num_chunks(ld);
  return nchunk > 1 ? up256((size_t)Q * 4) + up256((size_t)Q * nchunk * k * 8) : 0;
}


csa2_status attn_common(const char* name, const csa2_bf16* q, int Q, const int32_t* q_seq,
                        const int64_t* q_pos, const csa2_swa* swa, const void* plane,
                        int64_t plane_rows, const int64_t* row_base, const int32_t* sel, int nsel,
                        const float* sink, float scale, csa2_bf16* out, float* lse, void* ws,
                        size_t ws_bytes, const float* inv_freq, int plane_dtype, csa2_stream stream) {
  REQUIRE(Q >= 0 && Q <= 65535, "%s: Q must be in [0, 65535] (got %d)", name, Q);
  if (Q == 0) return CSA2_OK;
  REQUIRE(q && q_seq && q_pos && swa && out, "%s: q, q_seq, q_pos, swa and out are required", name);
  REQUIRE(aligned16(q) && aligned16(out), "%s: q and out must be 16-byte aligned", name);
  REQUIRE(nsel >= 0 && nsel <= 512, "%s: nsel must be in [0, 512] (got %d)", name, nsel);
  REQUIRE(nsel == 0 || (sel && plane && row_base), "%s: sel, plane and row_base are required when nsel > 0", name);
  REQUIRE(plane == nullptr || aligned16(plane), "%s: plane must be 16-byte aligned", name);
  REQUIRE(swa->mode == CSA2_SWA_RING || swa->mode == CSA2_SWA_LINEAR, "%s: bad swa.mode %d", name, swa->mode);
  REQUIRE(swa->dtype == CSA2_SWA_BF16 || swa->dtype == CSA2_SWA_FP8_S128 ||
              swa->dtype == CSA2_SWA_FP8_E8M0,
          "%s: bad swa.dtype %d", name, swa->dtype);
  REQUIRE(swa->data && aligned16(swa->data), "%s: swa.data must be a 16-byte aligned pointer", name);
  REQUIRE(swa->n_rows >= 0, "%s: swa.n_rows must be >= 0", name);
  REQUIRE(swa->mode == CSA2_SWA_RING || (swa->lin_base && swa->lin_pos0),
          "%s: LINEAR windows need lin_base and lin_pos0", name);
  REQUIRE(std::isfinite(scale), "%s: scale must be finite", name);
  REQUIRE(plane_rows >= 0 && plane_rows < ((int64_t)1 << 31),
          "%s: plane_rows must be in [0, 2^31)", name);
  REQUIRE(swa->n_rows < ((int64_t)1 << 31), "%s: swa.n_rows must be < 2^31", name);
  csa2::AttnArgs a{};
  a.q = q; a.Q = Q; a.q_seq = q_seq; a.q_pos = q_pos;
  a.swa_mode = swa->mode; a.swa_dtype = swa->dtype;
  a.swa = static_cast<const uint8_t*>(swa->data); a.swa_rows = swa->n_rows;
  a.lin_base = swa->lin_base; a.lin_pos0 = swa->lin_pos0;
  a.plane = static_cast<const uint16_t*>(plane); a.plane_rows = plane_rows; a.row_base = row_base;
  a.plane_dtype = plane_dtype;
  a.sel = sel; a.nsel = nsel; a.sink = sink; a.scale = scale; a.out = out; a.lse = lse;
  a.inv_freq = inv_freq;
  // rows read about once (a decode batch) are streamed through L2; a prefill chunk's
  // queries share the plane's rows, which stay
  a.stream_rows = (int64_t)Q * (128 + nsel) <= plane_rows ? 1 : 0;
  REQUIRE(ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) == 0,
          "%s: ws must be 256-byte aligned", name);
  const int sms = num_sms();
  if (sms <= 0) return fail(CSA2_ECUDA, "%s: no CUDA device", name);
  (void)ws_bytes;  // the attention needs no workspace (see csa2_attn_workspace_size)
  const int nsplit = csa2::attn_num_splits(Q, nsel, sms);
  // more queries than SMs: one CTA per SM walks its queries, overlapping a query's output
  // and the next query's set-up with the gathers
  a.persist = nsplit == 1 && Q > sms ? sms : 0;
  cudaError_t e = csa2::launch_attn(a, nsplit, stream);
  if (e != cudaSuccess) return cuda_fail(e, name);
  return CSA2_OK;
}

}  // namespace

namespace csa2 {
void set_last_error(const char* msg) { g_last_error = msg; }
}  // namespace csa2

extern "C" {

const char* csa2_last_error(void) { return g_last_error.c_str(); }

const char* csa2_version(void) { return "csa2 0.1 sm_103a"; }

csa2_status csa2_device_status(csa2_stream stream) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail(e, "csa2_device_status");
  int f = 0;
  for (int v : {csa2::take_fault_compress(), csa2::take_fault_index(), csa2::take_fault_topk(),
                csa2::take_fault_attn(), csa2::take_fault_paged(), csa2::take_fault_chunk()})
    if (!f) f = v;
  if (f == csa2::kFaultTimeout) return fail(CSA2_ETIMEOUT, "a kernel gave up a bounded wait");
  if (f == csa2::kFaultBounds) return fail(CSA2_EBOUNDS, "a kernel met an index outside its buffer");
  return CSA2_OK;
}

csa2_status csa2_selftest_wait_timeout(int64_t limit_ns, csa2_stream stream) {
  REQUIRE(limit_ns >= 1000 && limit_ns <= 1000000000,
          "csa2_selftest_wait_timeout: limit_ns must be in [1e3, 1e9] (got %lld)",
          (long long)limit_ns);
  cudaError_t e = csa2::launch_wait_timeout((uint64_t)limit_ns, stream);
  if (e != cudaSuccess) return cuda_fail(e, "csa2_selftest_wait_timeout");
  return CSA2_OK;
}

namespace {

// Checks of the compressor's arguments (csa2_compress and the calls that include it);
// fills *a (a->T == 0: nothing to compress).
csa2_status compress_args(const char* name, const csa2_bf16* kv, const csa2_bf16* score, int T,
                          const int32_t* cu_seqlens, int B, const int64_t* start_pos, int ratio,
                          float* kv_state, float* score_state, csa2_bf16* plane,
                          int64_t plane_rows, const int64_t* row_base, const float* norm_w,
                          float eps, const float* inv_freq, csa2::CompressArgs* a) {
  *a = csa2::CompressArgs{};
  REQUIRE(ratio == 1 || ratio == 2, "%s: ratio must be 1 or 2 (got %d)", name, ratio);
  REQUIRE(B >= 1 && B <= 8192, "%s: B must be in [1, 8192] (got %d)", name, B);
  REQUIRE(T >= 0, "%s: T must be >= 0 (got %d)", name, T);
  if (T == 0) return CSA2_OK;
  REQUIRE(kv && cu_seqlens && start_pos && plane && row_base && inv_freq,
          "%s: kv, cu_seqlens, start_pos, plane, row_base and inv_freq are required", name);
  REQUIRE(ratio == 1 || (score && kv_state && score_state),
          "%s: ratio 2 needs score, kv_state and score_state", name);
  REQUIRE(aligned16(kv) && aligned16(plane) && (!score || aligned16(score)) &&
              (!kv_state || aligned16(kv_state)) && (!score_state || aligned16(score_state)) &&
              (!norm_w || aligned16(norm_w)),
          "%s: kv, score, plane, states and norm_w must be 16-byte aligned", name);
  REQUIRE(eps >= 0.f && std::isfinite(eps), "%s: eps must be finite and >= 0", name);
  REQUIRE(plane_rows >= 0, "%s: plane_rows must be >= 0", name);
  *a = csa2::CompressArgs{kv, score, T, cu_seqlens, B, start_pos, ratio, kv_state, score_state,
                          plane, plane_rows, row_base, norm_w, eps, inv_freq,
                          nullptr, nullptr, nullptr};
  return CSA2_OK;
}

}  // namespace

csa2_status csa2_compress(const csa2_bf16* kv, const csa2_bf16* score, int T,
                          const int32_t* cu_seqlens, int B, const int64_t* start_pos, int ratio,
                          float* kv_state, float* score_state, csa2_bf16* plane,
                          int64_t plane_rows, const int64_t* row_base, const float* norm_w,
                          float eps, const float* inv_freq, csa2_stream stream) {
  csa2::CompressArgs a;
  const csa2_status st = compress_args("csa2_compress", kv, score, T, cu_seqlens, B, start_pos,
                                       ratio, kv_state, score_state, plane, plane_rows, row_base,
                                       norm_w, eps, inv_freq, &a);
  if (st != CSA2_OK || a.T == 0) return st;
  cudaError_t e = csa2::launch_compress(a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "csa2_compress");
  return CSA2_OK;
}

csa2_status csa2_compress_index(const csa2_bf16* kv, const csa2_bf16* score, int T,
                                const int32_t* cu_seqlens, int B, const int64_t* start_pos,
                                int ratio, float* kv_state, float* score_state, csa2_bf16* plane,
                                int64_t plane_rows, const int64_t* row_base, const float* norm_w,
                                float eps, const float* inv_freq, const csa2_bf16* wk,
                                const float* knorm_w, csa2_bf16* index_plane,
                                csa2_stream stream) {
  REQUIRE(T <= 0 || (wk && index_plane), "csa2_compress_index: wk and index_plane are required");
  REQUIRE(!wk || (aligned16(wk) && aligned16(index_plane)),
          "csa2_compress_index: wk and index_plane must be 16-byte aligned");
  // the plain compressor's checks next
  csa2::CompressArgs a;
  const csa2_status st = compress_args("csa2_compress", kv, score, T, cu_seqlens, B, start_pos,
                                       ratio, kv_state, score_state, plane, plane_rows, row_base,
                                       norm_w, eps, inv_freq, &a);
  if (st != CSA2_OK || a.T == 0) return st;
  a.wk = reinterpret_cast<const uint16_t*>(wk);
  a.knorm_w = knorm_w;
  a.index_plane = reinterpret_cast<uint16_t*>(index_plane);
  cudaError_t e = csa2::launch_compress(a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "csa2_compress_index");
  return CSA2_OK;
}

size_t csa2_index_topk_workspace_size(int Q, int H, int64_t max_scored, int k) {
  (void)H;
  if (Q < 0 || max_scored < 1 || k < 1 || k > 512) return 0;
  return index_ws_layout(Q, max_scored, k).total;
}

namespace {

// plane_fmt: 1 = FP8 blocks (plane), 2 = MXFP4 blocks (plane); 0 = bf16 rows (index_k)
csa2_status index_topk_impl(const csa2_bf16* iq, const float* w, int Q, int H,
                            const csa2_bf16* index_k, const uint8_t* plane, int plane_fmt,
                            int64_t index_rows,
                            const int64_t* row_base, const int32_t* q_seq, const int64_t* q_pos,
                            int ratio, const int32_t* cand, int ncb, int k, int relu,
                            int64_t max_scored, int32_t* sel, float* sel_scores,
                            float* scores_out, int nbk, int32_t* pool, void* ws, size_t ws_bytes,
                            csa2_stream stream, const csa2::CompressArgs* comp = nullptr) {
  REQUIRE(Q >= 0, "csa2_index_topk: Q must be >= 0 (got %d)", Q);
  REQUIRE(H == 32 || H == 64, "csa2_index_topk: H must be 32 or 64 (got %d)", H);
  REQUIRE(ratio == 1 || ratio == 2, "csa2_index_topk: ratio must be 1 or 2 (got %d)", ratio);
  REQUIRE(k >= 1 && k <= 512, "csa2_index_topk: k must be in [1, 512] (got %d)", k);
  REQUIRE(max_scored >= 1, "csa2_index_topk: max_scored must be >= 1");
  if (cand) {
    REQUIRE(ncb >= 1, "csa2_index_topk: ncb must be >= 1 with a candidate pool");
    REQUIRE((int64_t)ncb * 8 >= k,
            "csa2_index_topk: candidate pool of %d blocks x 8 rows cannot hold top-%d", ncb, k);
    REQUIRE(max_scored == (int64_t)ncb * 8, "csa2_index_topk: REINDEX needs max_scored == ncb * 8");
  }
  REQUIRE(max_scored <= csa2::topk_max_len(),
          "csa2_index_topk: max_scored %lld exceeds the supported %lld positions",
          (long long)max_scored, (long long)csa2::topk_max_len());
  if (Q == 0) {  // nothing to score: the compressor's tokens (if any) run on their own
    if (comp && comp->T > 0) {
      cudaError_t e = csa2::launch_compress(*comp, stream);
      if (e != cudaSuccess) return cuda_fail(e, "csa2_compress_index_topk (compress)");
    }
    return CSA2_OK;
  }
  REQUIRE(iq && w && (plane_fmt ? plane != nullptr : index_k != nullptr) && row_base && q_seq &&
              q_pos && sel && ws,
          "csa2_index_topk: iq, w, the index plane, row_base, q_seq, q_pos, sel and ws are required");
  REQUIRE(aligned16(iq) && aligned16(plane_fmt ? (const void*)plane : (const void*)index_k),
          "csa2_index_topk: iq and the index plane must be 16-byte aligned");
  REQUIRE(index_rows >= 1 && index_rows < (int64_t)1 << 31, "csa2_index_topk: index_rows out of range");
  REQUIRE((int64_t)Q * H < (int64_t)1 << 31, "csa2_index_topk: Q * H out of range");
  REQUIRE((reinterpret_cast<uintptr_t>(ws) & 255u) == 0, "csa2_index_topk: ws must be 256-byte aligned");
  const IndexWs L = index_ws_layout(Q, max_scored, k, nbk, plane_fmt == 1 ? (int64_t)Q * H : 0);
  if (ws_bytes < L.total)
    return fail(CSA2_ENOSPACE, "csa2_index_topk: workspace %zu bytes < required %zu", ws_bytes, L.total);
  uint8_t* base = static_cast<uint8_t*>(ws);
  csa2::IndexArgs a{};
  a.iq = iq; a.w = w; a.Q = Q; a.H = H; a.index_k = index_k; a.index_rows = index_rows;
  a.row_base = row_base; a.q_seq = q_seq; a.q_pos = q_pos; a.ratio = ratio; a.cand = cand;
  a.ncb = cand ? ncb : 0; a.relu = relu ? 1 : 0; a.ld = max_scored; a.scores_out = scores_out;
  a.ldk = (max_scored + 3) & ~int64_t(3);
  a.keys = reinterpret_cast<uint32_t*>(base + L.keys);
  a.n_scored = reinterpret_cast<int32_t*>(base + L.n_scored);
  a.grp = reinterpret_cast<csa2::GroupRec*>(base + L.grp);
  a.cta = reinterpret_cast<csa2::CtaRec*>(base + L.cta);
  a.n_groups = reinterpret_cast<int32_t*>(base + L.n_groups);
  a.topk_count = reinterpret_cast<int32_t*>(base + L.count);
  a.group_max = cand ? 1 : 256 / H;
  if (nbk > 0) a.pool_count = reinterpret_cast<int32_t*>(base + L.pcount);
  if (plane_fmt == 1) {
    a.index_k = nullptr;
    a.plane8 = plane;
    a.q8 = base + L.q8;
    a.qscale = reinterpret_cast<float*>(base + L.qscale);
  } else if (plane_fmt == 2) {
    a.index_k = nullptr;
    a.plane4 = plane;
  }
  const int sms = num_sms();
  if (sms <= 0) return fail(CSA2_ECUDA, "csa2_index_topk: no CUDA device");
  cudaError_t e = csa2::launch_index(a, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "csa2_index_topk (scores)");
  csa2::TopkArgs t{};
  t.keys = a.keys; t.scores = nullptr; t.n = a.n_scored; t.Q = Q; t.ld = a.ldk; t.k = k;
  t.cand = cand; t.ncb = a.ncb; t.sel = sel; t.sel_scores = sel_scores;
  t.part = reinterpret_cast<uint64_t*>(base + L.part); t.nchunk = L.nchunk;
  t.count = a.topk_count;
  t.chunk = csa2::topk_row_chunk_len(max_scored);
  t.q_pos = q_pos;
  t.ratio = ratio;
  // n_scored <= max_scored <= ldk: the chunking of max_scored covers every row
  csa2::TopkArgs p{};
  if (nbk > 0) {  // the candidate blocks, from the same keys, in the same launch
    p = t;
    p.sel_scores = nullptr;
    p.k = nbk; p.sel = pool; p.blocks = 1;
    p.part = reinterpret_cast<uint64_t*>(base + L.ppart);
    p.nchunk = pool_chunks(L.nb_max, nbk, Q, sms);
    p.count = a.pool_count;
    p.chunk = (int)((L.nb_max + p.nchunk - 1) / p.nchunk);
  }
  // the block selection's CTAs (the longer ones) first
  e = nbk > 0 ? csa2::launch_topk(p, stream, &t, comp) : csa2::launch_topk(t, stream, nullptr, comp);
  if (e != cudaSuccess) return cuda_fail(e, "csa2_index_topk (top-k)");
  return CSA2_OK;
}

}  // namespace

csa2_status csa2_index_topk(const csa2_bf16* iq, const float* w, int Q, int H,
                            const csa2_bf16* index_k, int64_t index_rows,
                            const int64_t* row_base, const int32_t* q_seq, const int64_t* q_pos,
                            int ratio, const int32_t* cand, int ncb, int k, int relu,
                            int64_t max_scored, int32_t* sel, float* sel_scores,
                            float* scores_out, void* ws, size_t ws_bytes, csa2_stream stream) {
  return index_topk_impl(iq, w, Q, H, index_k, nullptr, 0, index_rows, row_base, q_seq, q_pos,
                         ratio, cand, ncb, k, relu, max_scored, sel, sel_scores, scores_out, 0,
                         nullptr, ws, ws_bytes, stream);
}

csa2_status csa2_compress_index_topk(
    const csa2_bf16* kv, const csa2_bf16* score, int T, const int32_t* cu_seqlens, int B,
    const int64_t* start_pos, float* kv_state, float* score_state, csa2_bf16* plane,
    int64_t plane_rows, const float* norm_w, float eps, const float* inv_freq,
    const csa2_bf16* iq, const float* w, int Q, int H, const csa2_bf16* index_k,
    int64_t index_rows, const int64_t* row_base, const int32_t* q_seq, const int64_t* q_pos,
    int ratio, const int32_t* cand, int ncb, int k, int relu, int64_t max_scored, int32_t* sel,
    float* sel_scores, float* scores_out, void* ws, size_t ws_bytes, csa2_stream stream) {
  csa2::CompressArgs c;
  const csa2_status st = compress_args("csa2_compress_index_topk", kv, score, T, cu_seqlens, B,
                                       start_pos, ratio, kv_state, score_state, plane,
                                       plane_rows, row_base, norm_w, eps, inv_freq, &c);
  if (st != CSA2_OK) return st;
  return index_topk_impl(iq, w, Q, H, index_k, nullptr, 0, index_rows, row_base, q_seq, q_pos,
                         ratio, cand, ncb, k, relu, max_scored, sel, sel_scores, scores_out, 0,
                         nullptr, ws, ws_bytes, stream, c.T > 0 ? &c : nullptr);
}

size_t csa2_index_topk_pool_workspace_size(int Q, int H, int64_t max_scored, int k, int nbk) {
  (void)H;
  if (Q < 0 || max_scored < 1 || k < 1 || k > 512 || nbk < 1 || nbk > 2048) return 0;
  return index_ws_layout(Q, max_scored, k, nbk).total;
}

csa2_status csa2_index_topk_pool(const csa2_bf16* iq, const float* w, int Q, int H,
                                 const csa2_bf16* index_k, int64_t index_rows,
                                 const int64_t* row_base, const int32_t* q_seq,
                                 const int64_t* q_pos, int ratio, int k, int relu,
                                 int64_t max_scored, int32_t* sel, float* sel_scores,
                                 float* scores_out, int nbk, int32_t* pool, void* ws,
                                 size_t ws_bytes, csa2_stream stream) {
  REQUIRE(nbk >= 1 && nbk <= 2048, "csa2_index_topk_pool: nbk must be in [1, 2048] (got %d)", nbk);
  REQUIRE(max_scored >= 1 && csa2::topk_fits(pool_blocks(max_scored), nbk),
          "csa2_index_topk_pool: %lld blocks per row with nbk = %d exceed the block selection",
          (long long)pool_blocks(max_scored), nbk);
  REQUIRE(Q == 0 || pool, "csa2_index_topk_pool: pool is required");
  return index_topk_impl(iq, w, Q, H, index_k, nullptr, 0, index_rows, row_base, q_seq, q_pos,
                         ratio, nullptr, 0, k, relu, max_scored, sel, sel_scores, scores_out,
                         nbk, pool, ws, ws_bytes, stream);
}

size_t csa2_index_topk_fp8_workspace_size(int Q, int H, int64_t max_scored, int k) {
  if (Q < 0 || (H != 32 && H != 64) || max_scored < 1 || k < 1 || k > 512) return 0;
  return index_ws_layout(Q, max_scored, k, 0, (int64_t)Q * H).total;
}

csa2_status csa2_index_topk_fp8(const csa2_bf16* iq, const float* w, int Q, int H,
                                const uint8_t* plane, int64_t index_rows,
                                const int64_t* row_base, const int32_t* q_seq,
                                const int64_t* q_pos, int ratio, const int32_t* cand, int ncb,
                                int k, int relu, int64_t max_scored, int32_t* sel,
                                float* sel_scores, float* scores_out, void* ws, size_t ws_bytes,
                                csa2_stream stream) {
  REQUIRE(Q == 0 || plane, "csa2_index_topk_fp8: plane is required");
  return index_topk_impl(iq, w, Q, H, nullptr, plane, 1, index_rows, row_base, q_seq, q_pos,
                         ratio, cand, ncb, k, relu, max_scored, sel, sel_scores, scores_out, 0,
                         nullptr, ws, ws_bytes, stream);
}

size_t csa2_index_topk_fp4_workspace_size(int Q, int H, int64_t max_scored, int k) {
  if (Q < 0 || (H != 32 && H != 64) || max_scored < 1 || k < 1 || k > 512) return 0;
  return index_ws_layout(Q, max_scored, k).total;
}

csa2_status csa2_index_topk_fp4(const csa2_bf16* iq, const float* w, int Q, int H,
                                const uint8_t* plane, int64_t index_rows,
                                const int64_t* row_base, const int32_t* q_seq,
                                const int64_t* q_pos, int ratio, const int32_t* cand, int ncb,
                                int k, int relu, int64_t max_scored, int32_t* sel,
                                float* sel_scores, float* scores_out, void* ws, size_t ws_bytes,
                                csa2_stream stream) {
  REQUIRE(Q == 0 || plane, "csa2_index_topk_fp4: plane is required");
  return index_topk_impl(iq, w, Q, H, nullptr, plane, 2, index_rows, row_base, q_seq, q_pos,
                         ratio, cand, ncb, k, relu, max_scored, sel, sel_scores, scores_out, 0,
                         nullptr, ws, ws_bytes, stream);
}

size_t csa2_index_plane_fp4_bytes(int64_t rows) {
  return rows <= 0 ? 0 : (size_t)((rows + 7) / 8) * 544;
}

csa2_status csa2_index_plane_fp4(const csa2_bf16* index_k, int64_t rows, uint8_t* plane,
                                 csa2_stream stream) {
  REQUIRE(rows >= 0 && rows < (int64_t)1 << 34, "csa2_index_plane_fp4: rows out of range");
  if (rows == 0) return CSA2_OK;
  REQUIRE(index_k && plane, "csa2_index_plane_fp4: index_k and plane are required");
  REQUIRE(aligned16(index_k) && aligned16(plane),
          "csa2_index_plane_fp4: index_k and plane must be 16-byte aligned");
  cudaError_t e = csa2::launch_plane_fp4_index(reinterpret_cast<const uint16_t*>(index_k), rows,
                                               plane, stream);
  if (e != cudaSuccess) return cuda_fail(e, "csa2_index_plane_fp4");
  return CSA2_OK;
}

size_t csa2_index_plane_fp8_bytes(int64_t rows) {
  return rows <= 0 ? 0 : (size_t)((rows + 7) / 8) * 1056;
}

csa2_status csa2_index_plane_fp8(const csa2_bf16* index_k, int64_t rows, uint8_t* plane,
                                 csa2_stream stream) {
  REQUIRE(rows >= 0 && rows < (int64_t)1 << 34, "csa2_index_plane_fp8: rows out of range");
  if (rows == 0) return CSA2_OK;
  REQUIRE(index_k && plane, "csa2_index_plane_fp8: index_k and plane are required");
  REQUIRE(aligned16(index_k) && aligned16(plane),
          "csa2_index_plane_fp8: index_k and plane must be 16-byte aligned");
  cudaError_t e = csa2::launch_plane_fp8(reinterpret_cast<const uint16_t*>(index_k), rows, plane,
                                         stream);
  if (e != cudaSuccess) return cuda_fail(e, "csa2_index_plane_fp8");
  return CSA2_OK;
}

size_t csa2_topk_workspace_size(int Q, int64_t ld, int k) {
  if (Q < 0 || ld < 1 || k < 1 || k > 2048 || !csa2::topk_row_fits(ld, k)) return 0;
  return topk_ws_bytes(Q, ld, k);
}

csa2_status csa2_topk_scores(const float* scores, const int32_t* n, int Q, int64_t ld, int k,
                             int32_t* sel, float* sel_scores, void* ws, size_t ws_bytes,
                             csa2_stream stream) {
  REQUIRE(Q >= 0, "csa2_topk_scores: Q must be >= 0");
  REQUIRE(k >= 1 && k <= 2048, "csa2_topk_scores: k must be in [1, 2048] (got %d)", k);
  REQUIRE(ld >= 1, "csa2_topk_scores: ld must be >= 1");
  REQUIRE(ld <= csa2::topk_max_len(),
          "csa2_topk_scores: ld %lld exceeds the supported %lld positions", (long long)ld,
          (long long)csa2::topk_max_len());
  REQUIRE(csa2::topk_row_fits(ld, k),
          "csa2_topk_scores: rows of %lld positions with k = %d exceed the chunk merge "
          "(chunks of 32768 positions x k must be <= 32768)", (long long)ld, k);
  if (Q == 0) return CSA2_OK;
  REQUIRE(scores && n && sel, "csa2_topk_scores: scores, n and sel are required");
  const size_t need = topk_ws_bytes(Q, ld, k);
  if (need) {
    REQUIRE(ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0,
            "csa2_topk_scores: ws must be a 256-byte aligned pointer");
    if (ws_bytes < need)
      return fail(CSA2_ENOSPACE, "csa2_topk_scores: workspace %zu bytes < required %zu", ws_bytes, need);
  }
  csa2::TopkArgs t{};
  t.keys = nullptr; t.scores = scores; t.n = n; t.Q = Q; t.ld = ld; t.k = k; t.cand = nullptr;
  t.ncb = 0; t.sel = sel; t.sel_scores = sel_scores;
  t.nchunk = csa2::topk_row_num_chunks(ld);
  t.chunk = csa2::topk_row_chunk_len(ld);
  if (t.nchunk > 1) {
    t.count = static_cast<int32_t*>(ws);
    t.part = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(ws) + up256((size_t)Q * 4));
    cudaError_t z = cudaMemsetAsync(t.count, 0, (size_t)Q * 4, stream);
    if (z != cudaSuccess) return cuda_fail(z, "csa2_topk_scores");
  }
  cudaError_t e = csa2::launch_topk(t, stream);
  if (e != cudaSuccess) return cuda_fail(e, "csa2_topk_scores");
  return CSA2_OK;
}

size_t csa2_attn_workspace_size(int Q, int nsel) {
  (void)Q;
  (void)nsel;
  return 0;  // one or two CTAs per query, merging in distributed shared memory
}

csa2_status csa2_sparse_attn(const csa2_bf16* q, int Q, const int32_t* q_seq,
                             const int64_t* q_pos, const csa2_swa* swa, const csa2_bf16* plane,
                             int64_t plane_rows, const int64_t* row_base, const int32_t* sel,
                             int nsel, const float* sink, float scale, csa2_bf16* out, float* lse,
                             void* ws, size_t ws_bytes, csa2_stream stream) {
  return attn_common("csa2_sparse_attn", q, Q, q_seq, q_pos, swa, plane, plane_rows, row_base,
                     sel, nsel, sink, scale, out, lse, ws, ws_bytes, nullptr, 0, stream);
}

csa2_status csa2_reuse_attn(const csa2_bf16* q, int Q, const int32_t* q_seq,
                            const int64_t* q_pos, const csa2_swa* swa, const csa2_bf16* plane,
                            int64_t plane_rows, const int64_t* row_base, const int32_t* sel,
                            int nsel, const float* sink, float scale, csa2_bf16* out, float* lse,
                            void* ws, size_t ws_bytes, csa2_stream stream) {
  return attn_common("csa2_reuse_attn", q, Q, q_seq, q_pos, swa, plane, plane_rows, row_base,
                     sel, nsel, sink, scale, out, lse, ws, ws_bytes, nullptr, 0, stream);
}

csa2_status csa2_sparse_attn_rope(const csa2_bf16* q, int Q, const int32_t* q_seq,
                                  const int64_t* q_pos, const csa2_swa* swa,
                                  const csa2_bf16* plane, int64_t plane_rows,
                                  const int64_t* row_base, const int32_t* sel, int nsel,
                                  const float* sink, float scale, csa2_bf16* out, float* lse,
                                  void* ws, size_t ws_bytes, const float* inv_freq,
                                  csa2_stream stream) {
  REQUIRE(inv_freq != nullptr, "csa2_sparse_attn_rope: inv_freq is required");
  return attn_common("csa2_sparse_attn_rope", q, Q, q_seq, q_pos, swa, plane, plane_rows,
                     row_base, sel, nsel, sink, scale, out, lse, ws, ws_bytes, inv_freq, 0,
                     stream);
}

csa2_status csa2_reuse_attn_rope(const csa2_bf16* q, int Q, const int32_t* q_seq,
                                 const int64_t* q_pos, const csa2_swa* swa,
                                 const csa2_bf16* plane, int64_t plane_rows,
                                 const int64_t* row_base, const int32_t* sel, int nsel,
                                 const float* sink, float scale, csa2_bf16* out, float* lse,
                                 void* ws, size_t ws_bytes, const float* inv_freq,
                                 csa2_stream stream) {
  REQUIRE(inv_freq != nullptr, "csa2_reuse_attn_rope: inv_freq is required");
  return attn_common("csa2_reuse_attn_rope", q, Q, q_seq, q_pos, swa, plane, plane_rows,
                     row_base, sel, nsel, sink, scale, out, lse, ws, ws_bytes, inv_freq, 0,
                     stream);
}

csa2_status csa2_sparse_attn_fp4(const csa2_bf16* q, int Q, const int32_t* q_seq,
                                 const int64_t* q_pos, const csa2_swa* swa, const uint8_t* plane,
                                 int64_t plane_rows, const int64_t* row_base, const int32_t* sel,
                                 int nsel, const float* sink, float scale, csa2_bf16* out,
                                 float* lse, void* ws, size_t ws_bytes, const float* inv_freq,
                                 csa2_stream stream) {
  return attn_common("csa2_sparse_attn_fp4", q, Q, q_seq, q_pos, swa, plane, plane_rows,
                     row_base, sel, nsel, sink, scale, out, lse, ws, ws_bytes, inv_freq, 1,
                     stream);
}

namespace {

// Checks of a paged cache; fills *c.
csa2_status paged_args(const char* name, const csa2_paged* p, csa2::PagedCache* c) {
  REQUIRE(p, "%s: cache is required", name);
  REQUIRE(p->dtype == CSA2_SWA_BF16 || p->dtype == CSA2_SWA_FP8_S128 ||
              p->dtype == CSA2_SWA_FP8_E8M0,
          "%s: bad cache.dtype %d", name, p->dtype);
  REQUIRE(p->page_rows >= 8 && p->page_rows <= 65536 && p->page_rows % 8 == 0,
          "%s: cache.page_rows must be a multiple of 8 in [8, 65536] (got %d)", name, p->page_rows);
  REQUIRE(p->data && aligned16(p->data), "%s: cache.data must be a 16-byte aligned pointer", name);
  REQUIRE(p->n_pages >= 1 && p->n_pages < ((int64_t)1 << 31),
          "%s: cache.n_pages must be in [1, 2^31) (got %lld)", name, (long long)p->n_pages);
  const int64_t page = (int64_t)p->page_rows * (p->dtype == CSA2_SWA_BF16 ? 1024 : 528);
  REQUIRE(p->page_stride >= page && p->page_stride % 16 == 0 &&
              p->page_stride < ((int64_t)1 << 40),
          "%s: cache.page_stride must be a multiple of 16 in [%lld, 2^40) (got %lld)", name,
          (long long)page, (long long)p->page_stride);
  REQUIRE(p->B >= 1 && p->B <= 65535, "%s: cache.B must be in [1, 65535] (got %d)", name, p->B);
  REQUIRE(p->table, "%s: cache.table is required", name);
  REQUIRE(aligned_to(4, p->table), "%s: cache.table must be 4-byte aligned", name);
  REQUIRE(p->table_cols >= 1 && p->table_ld >= p->table_cols,
          "%s: cache.table_cols must be in [1, table_ld] (got %lld, table_ld %lld)", name,
          (long long)p->table_cols, (long long)p->table_ld);
  c->dtype = p->dtype; c->page_rows = p->page_rows; c->data = static_cast<uint8_t*>(p->data);
  c->n_pages = p->n_pages; c->page_stride = p->page_stride; c->table = p->table; c->B = p->B;
  c->table_ld = p->table_ld; c->table_cols = p->table_cols;
  return CSA2_OK;
}

csa2::Divide divide_by(int d) {
  int lg = 0;
  while ((1 << lg) < d) ++lg;
  return {(uint32_t)((((uint64_t)1 << (31 + lg)) + d - 1) / d), lg - 1};
}

// Factor and shift of a division by page_rows: with s = ceil(log2 d) and mul = ceil(2^(31 + s) /
// d), j mul exceeds j 2^(31 + s) / d by less than j <= 2^31 times 1, so the floor of
// j mul / 2^(31 + s) is exact for j < 2^31.
void page_division(const csa2::PagedCache& c, uint32_t* mul, int* shift) {
  int lg = 3;  // page_rows >= 8
  while ((1 << lg) < c.page_rows) ++lg;
  *mul = (uint32_t)((((uint64_t)1 << (31 + lg)) + c.page_rows - 1) / c.page_rows);
  *shift = lg - 1;
}

// Rows that the table holds per sequence, at most 2^31 - 256.
int64_t table_rows(const csa2::PagedCache& c) {
  const int64_t most = 0x7FFFFF00;
  return c.table_cols >= most / c.page_rows ? most : c.table_cols * c.page_rows;
}

// Workspace of csa2_paged_attn: the parts of items that more than one CTA works on.
struct PagedWs {
  size_t part, pstat, rec, total;
  int nctas;   // most CTAs the call uses
  bool split;  // an item can be split
};
PagedWs paged_ws_layout(int Q, int H, int64_t max_rows) {
  PagedWs w{};
  const int ut = csa2::paged_unit_tiles();
  const int64_t items = (int64_t)Q * (H > 64 ? 2 : 1);
  // a window that begins inside a tile adds one tile
  const int64_t units = ((max_rows + 63) / 64 + 1 + ut - 1) / ut;
  const int64_t all = items * units;
  w.nctas = (int)(all < csa2::paged_max_ctas() ? all : csa2::paged_max_ctas());
  w.split = (max_rows + 63) / 64 > ut;
  size_t o = 0;
  const size_t hp = (size_t)csa2::paged_head_pad(H);
  if (w.split) {
    w.part = o; o = up256(o + (size_t)w.nctas * 2 * hp * 512 * 4);
    w.pstat = o; o = up256(o + (size_t)w.nctas * 2 * hp * 3 * 4);
    w.rec = o; o = up256(o + (size_t)items * 8);
  }
  w.total = o;
  return w;
}

}  // namespace

csa2_status csa2_paged_append(const csa2_bf16* kv, int64_t kv_ld, int T, const int32_t* cu_seqlens,
                              const int64_t* start_row, int ratio, const csa2_paged* cache,
                              const float* inv_freq, csa2_stream stream) {
  const char* name = "csa2_paged_append";
  REQUIRE(T >= 0, "%s: T must be >= 0 (got %d)", name, T);
  if (T == 0) return CSA2_OK;
  csa2::PagedAppendArgs a{};
  csa2_status st = paged_args(name, cache, &a.cache);
  if (st != CSA2_OK) return st;
  REQUIRE(kv && cu_seqlens && start_row, "%s: kv, cu_seqlens and start_row are required", name);
  REQUIRE(aligned16(kv), "%s: kv must be 16-byte aligned", name);
  REQUIRE(aligned_to(4, cu_seqlens) && aligned_to(8, start_row) && aligned_to(4, inv_freq),
          "%s: cu_seqlens, start_row and inv_freq must be aligned to their elements", name);
  REQUIRE(kv_ld >= 512 && kv_ld % 8 == 0, "%s: kv_ld must be a multiple of 8, >= 512 (got %lld)",
          name, (long long)kv_ld);
  REQUIRE(ratio >= 1 && ratio <= 65536, "%s: ratio must be in [1, 65536] (got %d)", name, ratio);
  a.kv = kv; a.kv_ld = kv_ld; a.T = T; a.cu_seqlens = cu_seqlens; a.start_row = start_row;
  a.ratio = ratio; a.inv_freq = inv_freq;
  a.cap_rows = table_rows(a.cache);
  page_division(a.cache, &a.page_mul, &a.page_shift);
  const int sms = num_sms();
  if (sms <= 0) return fail(CSA2_ECUDA, "%s: no CUDA device", name);
  cudaError_t e = csa2::launch_paged_append(a, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, name);
  return CSA2_OK;
}

size_t csa2_paged_attn_workspace_size(int Q, int H, int64_t max_rows) {
  if (Q < 0 || Q > 65535 || H < 1 || H > 128 || max_rows < 0 || max_rows > 0x7FFFFF00) return 0;
  if (Q == 0) return 0;
  return paged_ws_layout(Q, H, max_rows).total;
}

csa2_status csa2_paged_attn(const csa2_bf16* q, int Q, int H, const int32_t* q_seq,
                            const int64_t* q_pos, const csa2_paged* cache, int ratio,
                            int64_t window, int64_t max_rows, const float* sink, float scale,
                            csa2_bf16* out, float* lse, const float* inv_freq, void* ws,
                            size_t ws_bytes, csa2_stream stream) {
  const char* name = "csa2_paged_attn";
  REQUIRE(Q >= 0 && Q <= 65535, "%s: Q must be in [0, 65535] (got %d)", name, Q);
  if (Q == 0) return CSA2_OK;
  csa2::PagedAttnArgs a{};
  csa2_status st = paged_args(name, cache, &a.cache);
  if (st != CSA2_OK) return st;
  REQUIRE(q && q_seq && q_pos && out, "%s: q, q_seq, q_pos and out are required", name);
  REQUIRE(aligned16(q) && aligned16(out), "%s: q and out must be 16-byte aligned", name);
  REQUIRE(aligned_to(4, q_seq) && aligned_to(8, q_pos) && aligned_to(4, sink) &&
              aligned_to(4, lse) && aligned_to(4, inv_freq),
          "%s: q_seq, q_pos, sink, lse and inv_freq must be aligned to their elements", name);
  REQUIRE(H >= 1 && H <= 128, "%s: H must be in [1, 128] (got %d)", name, H);
  REQUIRE(ratio >= 1 && ratio <= 65536, "%s: ratio must be in [1, 65536] (got %d)", name, ratio);
  REQUIRE(window >= 0, "%s: window must be >= 0 (got %lld)", name, (long long)window);
  REQUIRE(max_rows >= 0 && max_rows <= 0x7FFFFF00,
          "%s: max_rows must be in [0, 2^31 - 256] (got %lld)", name, (long long)max_rows);
  REQUIRE(std::isfinite(scale), "%s: scale must be finite", name);
  REQUIRE((reinterpret_cast<uintptr_t>(ws) & 255u) == 0, "%s: ws must be 256-byte aligned", name);
  const PagedWs w = paged_ws_layout(Q, H, max_rows);
  if (w.split && (!ws || ws_bytes < w.total))
    return fail(CSA2_ENOSPACE, "%s: workspace of %zu bytes, %zu needed", name, ws ? ws_bytes : 0,
                w.total);
  const int sms = num_sms();
  if (sms <= 0) return fail(CSA2_ECUDA, "%s: no CUDA device", name);
  a.q = q; a.Q = Q; a.H = H; a.ng = H > 64 ? 2 : 1; a.q_seq = q_seq; a.q_pos = q_pos;
  a.cap_rows = table_rows(a.cache) < max_rows ? table_rows(a.cache) : max_rows;
  a.ratio = ratio; a.window = window; a.sink = sink; a.scale = scale; a.out = out; a.lse = lse;
  a.inv_freq = inv_freq; a.ut = csa2::paged_unit_tiles();
  a.box_rows = a.cache.page_rows % 64 == 0 ? 64 : a.cache.page_rows % 32 == 0 ? 32
               : a.cache.page_rows % 16 == 0 ? 16 : 8;
  page_division(a.cache, &a.page_mul, &a.page_shift);
  a.shared = (int64_t)Q * a.ng > a.cache.B ? 1 : 0;
  a.nctas = w.nctas < sms ? w.nctas : sms;
  uint8_t* base = static_cast<uint8_t*>(ws);
  if (w.split) {
    a.part = reinterpret_cast<float*>(base + w.part);
    a.pstat = reinterpret_cast<float*>(base + w.pstat);
    a.rec = reinterpret_cast<int2*>(base + w.rec);
  }
  // tiles an item can have: a window of w rows touches at most (w + 62) / 64 + 1
  const int64_t most = (a.cap_rows + 63) / 64;
  const bool narrow = window > 0 && window < a.cap_rows && (window + 62) / 64 + 1 < most;
  const int64_t tiles = narrow ? (window + 62) / 64 + 1 : most;
  const int64_t items = (int64_t)Q * a.ng;
  a.cluster = csa2::paged_cluster(items, tiles, sms);
  if (a.cluster > 0) {
    a.ut = 1;
    a.nctas = (int)items * a.cluster;
  }
  const int units = a.cluster > 0 ? 1 : (int)((tiles + a.ut - 1) / a.ut);
  cudaError_t e = csa2::launch_paged_attn(a, units, stream);
  if (e != cudaSuccess) return cuda_fail(e, name);
  return CSA2_OK;
}

csa2_status csa2_paged_read(csa2_bf16* out, int64_t out_ld, int T, const int32_t* cu_seqlens,
                            const int64_t* start_row, int ratio, const csa2_paged* cache,
                            const float* inv_freq, csa2_stream stream) {
  const char* name = "csa2_paged_read";
  REQUIRE(T >= 0, "%s: T must be >= 0 (got %d)", name, T);
  if (T == 0) return CSA2_OK;
  csa2::PagedReadArgs a{};
  csa2_status st = paged_args(name, cache, &a.cache);
  if (st != CSA2_OK) return st;
  REQUIRE(out && cu_seqlens && start_row, "%s: out, cu_seqlens and start_row are required", name);
  REQUIRE(aligned16(out), "%s: out must be 16-byte aligned", name);
  REQUIRE(aligned_to(4, cu_seqlens) && aligned_to(8, start_row) && aligned_to(4, inv_freq),
          "%s: cu_seqlens, start_row and inv_freq must be aligned to their elements", name);
  REQUIRE(out_ld >= 512 && out_ld % 8 == 0, "%s: out_ld must be a multiple of 8, >= 512 (got %lld)",
          name, (long long)out_ld);
  REQUIRE(ratio >= 1 && ratio <= 65536, "%s: ratio must be in [1, 65536] (got %d)", name, ratio);
  a.out = out; a.out_ld = out_ld; a.T = T; a.cu_seqlens = cu_seqlens; a.start_row = start_row;
  a.ratio = ratio; a.inv_freq = inv_freq;
  a.cap_rows = table_rows(a.cache);
  page_division(a.cache, &a.page_mul, &a.page_shift);
  const int sms = num_sms();
  if (sms <= 0) return fail(CSA2_ECUDA, "%s: no CUDA device", name);
  cudaError_t e = csa2::launch_paged_read(a, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, name);
  return CSA2_OK;
}

namespace {

// Whether two of the runs of D elements at t * token + h * head, t < T, h < H, share an element (strides >= 0).
bool rows_overlap(int T, int H, int D, int64_t token, int64_t head) {
  if ((T > 1 && token < D) || (H > 1 && head < D)) return true;
  if (T == 1 || H == 1) return false;
  // one stride beyond all that the other spans: the usual layouts
  typedef __int128 wide;
  if (token >= (wide)head * (H - 1) + D || head >= (wide)token * (T - 1) + D) return false;
  // otherwise the nearest token to each head
  for (int h = 1; h < H; ++h) {
    const wide to = (wide)head * h, most = T - 1, t = to / token < most ? to / token : most, past = to - t * token;
    if (past < D || (t < most && token - past < D)) return true;
  }
  return false;
}

// Checks of one set of heads; fills *s.
csa2_status head_args(const char* name, const char* which, const csa2_heads* h, int T, int D,
                      csa2::HeadSet* s) {
  REQUIRE(h->H >= 1 && h->H <= 1024, "%s: %s.H must be in [1, 1024] (got %d)", name, which, h->H);
  REQUIRE(h->x && h->out, "%s: %s.x and %s.out are required", name, which, which);
  REQUIRE(aligned16(h->x) && aligned16(h->out), "%s: %s.x and %s.out must be 16-byte aligned", name,
          which, which);
  REQUIRE(h->x_token >= 0 && h->x_head >= 0 && h->out_token >= 0 && h->out_head >= 0 &&
              ((h->x_token | h->x_head | h->out_token | h->out_head) & 7) == 0,
          "%s: %s's strides must be multiples of 8, >= 0", name, which);
  REQUIRE(!rows_overlap(T, h->H, D, h->out_token, h->out_head), "%s: %s.out's heads or tokens overlap", name, which);
  REQUIRE(aligned16(h->norm_w), "%s: %s.norm_w must be 16-byte aligned", name, which);
  s->x = h->x; s->out = h->out; s->x_token = h->x_token; s->x_head = h->x_head;
  s->out_token = h->out_token; s->out_head = h->out_head; s->H = h->H; s->norm = h->norm ? 1 : 0;
  s->norm_w = h->norm ? h->norm_w : nullptr;
  return CSA2_OK;
}

}  // namespace

csa2_status csa2_qk_norm_rope(const csa2_heads* q, const csa2_heads* k, int T, int D, float eps,
                              const int64_t* pos, const float* inv_freq, int rope_dim0,
                              int rope_dims, int layout, float factor, csa2_stream stream) {
  const char* name = "csa2_qk_norm_rope";
  REQUIRE(T >= 0, "%s: T must be >= 0 (got %d)", name, T);
  if (T == 0) return CSA2_OK;
  REQUIRE(q || k, "%s: q or k is required", name);
  REQUIRE(D >= 8 && D <= 512 && D % 8 == 0, "%s: D must be a multiple of 8 in [8, 512] (got %d)", name,
          D);
  REQUIRE(layout == CSA2_ROPE_PAIRS || layout == CSA2_ROPE_HALVES, "%s: bad layout %d", name, layout);
  REQUIRE(rope_dim0 >= 0 && rope_dims >= 0 && rope_dim0 % 8 == 0 && rope_dims % 8 == 0 &&
              rope_dims <= D && rope_dim0 <= D - rope_dims,
          "%s: rope_dim0 and rope_dims must be multiples of 8 within D (got %d, %d)", name, rope_dim0,
          rope_dims);
  REQUIRE(layout == CSA2_ROPE_PAIRS || rope_dims % 16 == 0,
          "%s: rope_dims must be a multiple of 16 with halves (got %d)", name, rope_dims);
  REQUIRE(rope_dims == 0 || (pos && inv_freq), "%s: pos and inv_freq are required", name);
  REQUIRE(aligned_to(8, pos) && aligned_to(4, inv_freq),
          "%s: pos and inv_freq must be aligned to their elements", name);
  REQUIRE(std::isfinite(eps) && eps >= 0.f, "%s: eps must be finite and >= 0", name);
  REQUIRE(std::isfinite(factor), "%s: factor must be finite", name);
  csa2::HeadsArgs a{};
  if (q) {
    csa2_status st = head_args(name, "q", q, T, D, &a.q);
    if (st != CSA2_OK) return st;
  }
  if (k) {
    csa2_status st = head_args(name, "k", k, T, D, &a.k);
    if (st != CSA2_OK) return st;
  }
  a.T = T; a.D = D; a.eps = eps; a.pos = pos; a.inv_freq = inv_freq; a.rope_dim0 = rope_dim0;
  a.rope_dims = rope_dims; a.halves = layout == CSA2_ROPE_HALVES; a.factor = factor;
  const int sms = num_sms();
  if (sms <= 0) return fail(CSA2_ECUDA, "%s: no CUDA device", name);
  cudaError_t e = csa2::launch_heads(a, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, name);
  return CSA2_OK;
}

namespace {

// Workspace of csa2_paged_chunk_attn.
struct ChunkWs {
  size_t tile, prefix, share, split_list, part, pstat, stage, stage_cu, stage_first, stage_end, total;
  int max_tiles, pairs;
  bool split;      // a tile may need parts
  int64_t rows;    // staged
  int parts;       // whose sum the staged rows are
};
// Rows that a tensor copy brings at once: the largest of 64, 32, 16, 8 dividing page_rows.
int page_box(int page_rows) {
  return page_rows % 64 == 0 ? 64 : page_rows % 32 == 0 ? 32 : page_rows % 16 == 0 ? 16 : 8;
}

// FP8 rows are staged as dense bf16 rows first: decoding a row once for all tiles that read it.  So are bf16
// rows on small pages where a sequence has tiles enough to read them, as copies of 16 or 8 rows take the
// loaders longer than the products take: us direct / staged, chunks of 8 sequences with 150 tiles each
// 795 / 678 at 16-row pages and 1048 / 679 at 8-row ones (688 / 710 at 32), 24 with 31 tiles 536 / 509 and
// 754 / 536, 8 with 8 tiles 149 / 161 and 193 / 164, 64 with 2 tiles 171 / 271 and 194 / 274.
bool chunk_stages(int T, int H, const csa2_paged& c) {
  if (c.dtype != CSA2_SWA_BF16) return true;
  const int64_t seqs = c.B < T ? c.B : T, tiles = ((int64_t)T * H + 127) / 128;
  const int box = page_box(c.page_rows);
  return box == 8 ? tiles >= 4 * seqs : box == 16 ? tiles >= 24 * seqs : false;
}

ChunkWs chunk_ws_layout(int T, int H, const csa2_paged& c, int64_t max_rows, int64_t total_rows) {
  ChunkWs w{};
  // sequences with tokens; each may have an incomplete tile
  const int64_t seqs = c.B < T ? c.B : T;
  const int64_t tiles = ((int64_t)T * H + 127) / 128 + seqs;
  // key tiles of a tile: a window that begins inside one adds one
  const int64_t keys = (max_rows + 255) / 256 + 1;
  w.max_tiles = (int)tiles;
  w.split = tiles > csa2::chunk_max_pairs() || keys > csa2::chunk_whole_keys();
  const int64_t most = w.split ? tiles * keys : tiles;
  w.pairs = (int)(most < csa2::chunk_max_pairs() ? most : csa2::chunk_max_pairs());
  // A code of four bits times a scale of 24 is more than bf16 holds: FP8_S128 rows are staged in two parts, the
  // value rounded and what that leaves, rounded, 2^-16 off in all.  In one part lse came out 1e-5 off and out
  // half as far again as that of bf16 rows; four chunks over 16000 rows took 1040 us in place of 2010.
  w.parts = c.dtype == CSA2_SWA_FP8_S128 ? 2 : 1;
  size_t o = 0;
  w.tile = o; o = up256(o + (size_t)tiles * sizeof(csa2::ChunkTile));
  w.prefix = o; o = up256(o + (size_t)tiles * 8);
  w.share = o; o = up256(o + (size_t)w.pairs * sizeof(csa2::ChunkShare));
  w.split_list = o; o = up256(o + (size_t)(w.pairs + 1) * 4);
  if (w.split) {
    w.part = o; o = up256(o + (size_t)w.pairs * 2 * 128 * 512 * 4);
    w.pstat = o; o = up256(o + (size_t)w.pairs * 2 * 128 * 3 * 4);
  }
  if (chunk_stages(T, H, c)) {
    // whole groups of eight rows of each sequence, and a key tile's rows of zeros behind the last (with copies
    // that reach beyond the tensor instead, 1295 tokens over 38 rows took 380 us in place of 97)
    w.rows = ((total_rows + 7) & ~(int64_t)7) + 16 * seqs + 256;
    w.stage = o; o = up256(o + (size_t)w.parts * w.rows * 1024);
    w.stage_cu = o; o = up256(o + (size_t)(c.B + 1) * 4);
    w.stage_first = o; o = up256(o + (size_t)c.B * 8);
    w.stage_end = o; o = up256(o + (size_t)c.B * 8);
  }
  w.total = o;
  return w;
}

}  // namespace

size_t csa2_paged_chunk_attn_workspace_size(int T, int H, const csa2_paged* cache, int64_t max_rows,
                                            int64_t total_rows) {
  if (T < 0 || T > 1048576 || H < 1 || H > 128 || max_rows < 0 || max_rows > 0x7FFFFF00 ||
      total_rows < 0 || total_rows > (1 << 30) || !cache || cache->B < 1 || cache->B > 65535)
    return 0;
  if (T == 0) return 0;
  return chunk_ws_layout(T, H, *cache, max_rows, total_rows).total;
}

csa2_status csa2_paged_chunk_attn(const csa2_bf16* q, int T, int H, const int32_t* cu_seqlens,
                                  const int64_t* start_pos, const csa2_paged* cache, int ratio,
                                  int64_t window, int64_t max_rows, int64_t total_rows,
                                  const float* sink, float scale, csa2_bf16* out, float* lse,
                                  const float* inv_freq, void* ws, size_t ws_bytes,
                                  csa2_stream stream) {
  const char* name = "csa2_paged_chunk_attn";
  REQUIRE(T >= 0 && T <= 1048576, "%s: T must be in [0, 1048576] (got %d)", name, T);
  if (T == 0) return CSA2_OK;
  csa2::ChunkArgs a{};
  csa2_status st = paged_args(name, cache, &a.cache);
  if (st != CSA2_OK) return st;
  REQUIRE(q && cu_seqlens && start_pos && out, "%s: q, cu_seqlens, start_pos and out are required",
          name);
  REQUIRE(aligned16(q) && aligned16(out), "%s: q and out must be 16-byte aligned", name);
  REQUIRE(aligned_to(4, cu_seqlens) && aligned_to(8, start_pos) && aligned_to(4, sink) &&
              aligned_to(4, lse) && aligned_to(4, inv_freq),
          "%s: cu_seqlens, start_pos, sink, lse and inv_freq must be aligned to their elements", name);
  REQUIRE(H >= 1 && H <= 128, "%s: H must be in [1, 128] (got %d)", name, H);
  REQUIRE(ratio >= 1 && ratio <= 65536, "%s: ratio must be in [1, 65536] (got %d)", name, ratio);
  REQUIRE(window >= 0, "%s: window must be >= 0 (got %lld)", name, (long long)window);
  REQUIRE(max_rows >= 0 && max_rows <= 0x7FFFFF00,
          "%s: max_rows must be in [0, 2^31 - 256] (got %lld)", name, (long long)max_rows);
  REQUIRE(total_rows >= 0 && total_rows <= (1 << 30),
          "%s: total_rows must be in [0, 2^30] (got %lld)", name, (long long)total_rows);
  REQUIRE(std::isfinite(scale), "%s: scale must be finite", name);
  REQUIRE((reinterpret_cast<uintptr_t>(ws) & 255u) == 0, "%s: ws must be 256-byte aligned", name);
  const ChunkWs w = chunk_ws_layout(T, H, *cache, max_rows, total_rows);
  if (!ws || ws_bytes < w.total)
    return fail(CSA2_ENOSPACE, "%s: workspace of %zu bytes, %zu needed", name, ws ? ws_bytes : 0,
                w.total);
  const int sms = num_sms();
  if (sms <= 0) return fail(CSA2_ECUDA, "%s: no CUDA device", name);
  a.q = q; a.T = T; a.H = H; a.cu_seqlens = cu_seqlens; a.start_pos = start_pos;
  a.cap_rows = table_rows(a.cache) < max_rows ? table_rows(a.cache) : max_rows;
  a.ratio = ratio; a.window = window; a.sink = sink; a.scale = scale; a.out = out; a.lse = lse;
  a.inv_freq = inv_freq;
  page_division(a.cache, &a.page_mul, &a.page_shift);
  a.pairs = w.pairs;
  a.by_ratio = divide_by(ratio);
  a.by_heads = divide_by(H);
  a.alone = !w.split && w.rows == 0 && a.cache.B <= 256 ? 1 : 0;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.tile = reinterpret_cast<csa2::ChunkTile*>(base + w.tile);
  a.prefix = reinterpret_cast<int64_t*>(base + w.prefix);
  a.max_tiles = w.max_tiles;
  a.share = reinterpret_cast<csa2::ChunkShare*>(base + w.share);
  a.split = reinterpret_cast<int32_t*>(base + w.split_list);
  if (w.split) {
    a.part = reinterpret_cast<float*>(base + w.part);
    a.pstat = reinterpret_cast<float*>(base + w.pstat);
  }
  a.box_rows = page_box(a.cache.page_rows);
  a.parts = w.parts;
  if (w.rows > 0) {
    a.box_rows = 64;
    a.stage = reinterpret_cast<uint16_t*>(base + w.stage);
    a.stage_rows = w.rows;
    a.stage_cu = reinterpret_cast<int32_t*>(base + w.stage_cu);
    a.stage_first = reinterpret_cast<int64_t*>(base + w.stage_first);
    a.stage_end = reinterpret_cast<int64_t*>(base + w.stage_end);
  }
  cudaError_t e = csa2::launch_chunk_attn(a, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, name);
  return CSA2_OK;
}

size_t csa2_plane_fp4_bytes(int64_t rows) { return rows <= 0 ? 0 : (size_t)rows * 288; }

csa2_status csa2_plane_fp4(const csa2_bf16* plane, int64_t rows, uint8_t* out,
                           csa2_stream stream) {
  REQUIRE(rows >= 0 && rows < (int64_t)1 << 31, "csa2_plane_fp4: rows out of range");
  if (rows == 0) return CSA2_OK;
  REQUIRE(plane && out, "csa2_plane_fp4: plane and out are required");
  REQUIRE(aligned16(plane) && aligned16(out), "csa2_plane_fp4: plane and out must be 16-byte aligned");
  cudaError_t e =
      csa2::launch_plane_fp4(reinterpret_cast<const uint16_t*>(plane), rows, out, stream);
  if (e != cudaSuccess) return cuda_fail(e, "csa2_plane_fp4");
  return CSA2_OK;
}

}  // extern "C"

namespace csa2 {

static PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

bool encode_bytes(CUtensorMap* m, const void* base, int rank, const uint64_t* dims,
                  const uint64_t* strides, const uint32_t* box) {
  auto fn = tensor_map_encoder();
  if (!fn || !base || rank < 2 || rank > 5) return false;
  cuuint64_t d[5], st[4];
  cuuint32_t bx[5], es[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    bx[i] = box[i];
    if (dims[i] == 0) return false;
  }
  for (int i = 0; i + 1 < rank; ++i) st[i] = strides[i];
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(base), d,
                  st, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_rows_bf16(CUtensorMap* m, const void* base, uint64_t rows, uint32_t cols,
                      uint32_t box_cols, uint32_t box_rows) {
  auto fn = tensor_map_encoder();
  if (!fn || !base || rows == 0) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace csa2
