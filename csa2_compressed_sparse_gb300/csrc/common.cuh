// common.cuh -- argument blocks shared by the C-ABI layer and the kernels, plus the
// per-translation-unit fault flag helpers.
#pragma once

#include <cfloat>

#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "ptx.cuh"

namespace csa2 {

constexpr int kDLat = 512;   // latent width (K = V)
constexpr int kDIdx = 128;   // indexer head width
constexpr int kHeads = 64;   // attention query heads
constexpr int kRing = 128;   // sliding-window slots
constexpr int kRopeDim0 = 448;
constexpr int kMaxK = 512;   // largest top-k
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct CompressArgs {
  const uint16_t* kv;
  const uint16_t* score;
  int T;
  const int32_t* cu_seqlens;
  int B;
  const int64_t* start_pos;
  int ratio;
  float* kv_state;
  float* score_state;
  uint16_t* plane;
  int64_t plane_rows;
  const int64_t* row_base;
  const float* norm_w;
  float eps;
  const float* inv_freq;
  // index K of each row (null wk: none): wk [128][512] bf16, knorm_w [128] (null: ones),
  // index_plane [plane_rows][128] bf16
  const uint16_t* wk;
  const float* knorm_w;
  uint16_t* index_plane;
};

// A query group of the indexer: queries q0 .. q0 + nq - 1 of sequence seq (row_base rb)
// own the work tiles tile0 .. tile1 - 1.
struct __align__(16) GroupRec {
  int32_t q0, nq, seq, pad0;
  int64_t tile0, tile1;
  int64_t rb, pad1;
};
// A score CTA's work: tiles it_lo .. it_hi - 1, starting in group g_first.
struct __align__(16) CtaRec {
  int32_t g_first, pad0;
  int64_t it_lo, it_hi, pad1;
};
constexpr int kMaxIndexCtas = 1024;

struct IndexArgs {
  const uint16_t* iq;   // [Q][H][128]
  const float* w;       // [Q][H]
  int Q, H;
  const uint16_t* index_k;
  int64_t index_rows;
  const int64_t* row_base;
  const int32_t* q_seq;
  const int64_t* q_pos;
  int ratio;
  const int32_t* cand;  // [Q][ncb] or null
  int ncb;
  int relu;
  int64_t ld;           // max_scored: positions per query (row stride of scores_out)
  int64_t ldk;          // row stride of keys (ld rounded up to a multiple of 4)
  float* scores_out;    // optional [Q][ld]
  // workspace views
  uint32_t* keys;       // [Q][ldk]
  int32_t* n_scored;    // [Q]
  struct GroupRec* grp;  // [Q]  query groups (written by the prep kernel)
  struct CtaRec* cta;    // [nctas] each score CTA's tile range and first group
  int nctas;             // score kernel CTAs (<= kMaxIndexCtas)
  int32_t* n_groups;     // [2]  groups, largest group size
  int32_t* topk_count;  // [Q]  zeroed by the prep kernel for the top-k merge
  int group_max;        // queries per group (FULL: 256 / H; REINDEX: 1)
  int32_t* pool_count;  // [Q]  or null: zeroed by the prep kernel for the candidate
                        //      pool's top-k merge
  // FP8 index plane (null: index_k is bf16): blocks of 8 rows, 8 x 128 E4M3 codes then
  // 8 fp32 scales (1056 bytes); row_base values are multiples of 8
  const uint8_t* plane8;
  const uint8_t* plane4;  // MXFP4 index plane (blocks of 8 rows, 544 bytes), or null
  uint8_t* q8;          // [Q*H][128] E4M3 codes of the quantised queries (workspace)
  float* qscale;        // [Q*H] their power-of-two scales (workspace)
};

struct TopkArgs {
  const uint32_t* keys;   // [Q][ld] order-preserving keys (0 = not scored), or
  const float* scores;    // [Q][ld] raw fp32 scores (converted on load)
  const int32_t* n;       // [Q] positions per row
  int Q;
  int64_t ld;
  int k;
  const int32_t* cand;    // [Q][ncb] position -> row map for REINDEX, else null
  int ncb;
  int32_t* sel;           // [Q][k]
  float* sel_scores;      // [Q][k] or null
  uint64_t* part;         // [Q][nchunk][k] (key << 32 | position) partial results
  int32_t* count;         // [Q] chunk arrivals (zero before the call; reset by the merge)
  int nchunk;             // chunks per row (1 = single pass)
  int chunk;              // positions (blocks) per chunk
  int blocks;             // 1: select blocks of 8 positions of `keys` instead (candidate
                          //    pool): a block's key is the largest key of its positions
                          //    < n[q], the newest block ceil(n[q] / 8) - 1 is pinned to
                          //    ~0, and the output holds block ids
  const int64_t* q_pos;   // or null: n[q] = min(ld, cand ? ncb * 8 : (q_pos[q] + 1) / ratio),
  int ratio;              //    the index call's scored count, known before its prep ends
};

struct AttnArgs {
  const uint16_t* q;
  int Q;
  const int32_t* q_seq;
  const int64_t* q_pos;
  int swa_mode, swa_dtype;
  const uint8_t* swa;
  int64_t swa_rows;
  const int64_t* lin_base;
  const int64_t* lin_pos0;
  const uint16_t* plane;
  int64_t plane_rows;
  const int64_t* row_base;
  const int32_t* sel;
  int nsel;
  const float* sink;
  float scale;
  uint16_t* out;
  float* lse;
  int cluster;     // nsplit == 2: the two CTAs of a query form a cluster and merge in place
  const float* inv_freq;  // [32] or null: rotate the output's dims 448..511 back by q_pos
  int plane_dtype;        // 0: bf16 plane rows [512]; 1: FP4 rows of 288 bytes (E2M1 codes,
                          //    low nibble first, then 32 E4M3 scales, one per 16 dims)
  int stream_rows;        // 1: the call reads fewer rows than the plane holds, so a row is
                          //    read about once: gathered bf16 rows are evicted from L2 first
  int persist;            // > 0 (one CTA per query, more queries than SMs): that many CTAs,
                          //    each carrying on from query to query
};

// A paged latent cache: row j of sequence b is row j % page_rows of page
// table[b * table_ld + j / page_rows], page_stride bytes from page to page.
struct PagedCache {
  int dtype;              // 0: bf16 rows of 1024 bytes; 1: FP8_S128, 2: FP8_E8M0 (528 bytes)
  int page_rows;
  uint8_t* data;
  int64_t n_pages;
  int64_t page_stride;
  const int32_t* table;
  int B;
  int64_t table_ld, table_cols;
};

struct PagedAppendArgs {
  const uint16_t* kv;
  int64_t kv_ld;          // elements from token to token
  int T;
  const int32_t* cu_seqlens;
  const int64_t* start_row;
  int ratio;              // position of cache row j: j * ratio
  const float* inv_freq;  // [32] or null: rows are stored as they are
  PagedCache cache;
  int64_t cap_rows;       // rows that the table holds per sequence (below 2^31)
  uint32_t page_mul;      // j / page_rows = (j * page_mul >> 32) >> page_shift
  int page_shift;
};

struct PagedAttnArgs {
  const uint16_t* q;
  int Q, H;
  int ng;                 // head groups of up to 64
  const int32_t* q_seq;
  const int64_t* q_pos;
  PagedCache cache;
  int64_t cap_rows;       // rows a query may see: the caller's bound and the table's capacity
  int ratio;
  int64_t window;         // 0: all visible rows
  const float* sink;
  float scale;
  uint16_t* out;
  float* lse;
  const float* inv_freq;
  int ut;                 // tiles of 64 rows per unit
  uint32_t page_mul;      // as in PagedAppendArgs
  int page_shift;
  int box_rows;           // rows per tensor copy: the largest of 64, 32, 16, 8 dividing page_rows
  int shared;             // more items than sequences: rows are read more than once
  int nctas;
  int cluster;            // CTAs per item of a small call (a cluster if more than one), else 0
  // workspace: parts [2 nctas][padded heads * 512], their m, l, r, and each item's CTA range
  float* part;
  float* pstat;
  int2* rec;
};

// Rows start_row[b] + i of the cache to row cu_seqlens[b] + i of out, as bf16.
struct PagedReadArgs {
  uint16_t* out;
  const int64_t* row_end; // or null; rows from row_end[b] on, and those on bad pages, become zeros
  uint16_t* low;          // or null: what FP8_S128 rows lose when rounded, rounded itself, as rows of out
  int64_t out_ld;         // elements from row to row
  int T;
  const int32_t* cu_seqlens;
  const int64_t* start_row;
  int ratio;
  const float* inv_freq;  // [32] or null: the rotation by j * ratio is undone
  PagedCache cache;
  int64_t cap_rows;       // these three as in PagedAppendArgs
  uint32_t page_mul;
  int page_shift;
};

// Division of x < 2^31 by d in 1 .. 2^16: with s = ceil(log2 d) and mul = ceil(2^(31 + s) / d), j mul exceeds
// j 2^(31 + s) / d by less than 2^31, so the floor of j mul / 2^(31 + s) is exact.  shift = s - 1.
struct Divide {
  uint32_t mul;
  int shift;
};

// A tile of a chunk's attention: 128 rows (token, head) of one sequence, and its key tiles.
struct __align__(16) ChunkTile {
  int32_t seq, row0, rows;  // rows row0 .. row0 + rows - 1 of [T * H]
  int32_t k0, kn;           // key tiles of 256 cache rows: k0 .. k0 + kn - 1
  int32_t c0, c1;           // the first and last CTA pair that works on it
  int32_t tok0;             // the sequence's first token,
  int64_t start;            // and its position
  int64_t off;              // staged rows: cache row j is row j + off
  int32_t clip;             // rows the sequence may see
  int32_t pad[3];
};
// A pair's share: `count` units (key tiles) from key tile `unit` of tile `tile` on.
struct __align__(16) ChunkShare {
  int32_t tile, unit;
  int64_t count;
};

// Attention of a chunk of new tokens: token cu_seqlens[b] + i of q sits at start_pos[b] + i.
struct ChunkArgs {
  const uint16_t* q;      // [T][H][512]
  int T, H;
  const int32_t* cu_seqlens;
  const int64_t* start_pos;
  PagedCache cache;
  int64_t cap_rows;       // rows a token may see: the caller's bound and the table's capacity
  int ratio;
  int64_t window;
  const float* sink;
  float scale;
  uint16_t* out;
  float* lse;
  const float* inv_freq;
  uint32_t page_mul;      // as in PagedAppendArgs
  int page_shift;
  int box_rows;           // rows per tensor copy
  Divide by_ratio, by_heads;
  int alone;              // no plan: pair c works on tile c
  int pairs;              // CTA pairs of the launch
  // workspace
  ChunkTile* tile;        // [max_tiles]
  int64_t* prefix;        // [max_tiles] units before each tile
  int max_tiles;
  ChunkShare* share;      // [pairs]
  int32_t* split;         // [1 + pairs] how many tiles several pairs work on, and which
  float* part;            // [2 pairs][2 CTAs][64 float4 columns][128 lanes][4]
  float* pstat;           // [2 pairs][2 CTAs][m, l, r][64]
  // rows that are not read from their pages: staged as dense bf16 rows (stage null: none are)
  uint16_t* stage;        // [parts][stage_rows][512]
  int parts;              // 2: a row is the sum of both parts'
  int64_t stage_rows;
  int32_t* stage_cu;      // [B + 1]
  int64_t* stage_first;   // [B]
  int64_t* stage_end;     // [B]
};

// Heads of queries or of keys: token t's head h at x + t x_token + h x_head (elements).
struct HeadSet {
  const uint16_t* x;
  uint16_t* out;
  int64_t x_token, x_head, out_token, out_head;
  int H;                  // 0: none
  int norm;
  const float* norm_w;    // [D] or null: ones
};
struct HeadsArgs {
  HeadSet q, k;
  int T, D;
  float eps;
  const int64_t* pos;     // [T]
  const float* inv_freq;  // [rope_dims / 2]
  int rope_dim0, rope_dims, halves;
  float factor;
  int units;              // units of rows of an item
};

cudaError_t launch_compress(const CompressArgs& a, cudaStream_t s);
cudaError_t launch_heads(const HeadsArgs& a, int sms, cudaStream_t s);
cudaError_t launch_paged_read(const PagedReadArgs& a, int sms, cudaStream_t s);
cudaError_t launch_chunk_attn(const ChunkArgs& a, int sms, cudaStream_t s);
int chunk_max_pairs();        // most CTA pairs of a chunk's attention
int chunk_whole_keys();       // key tiles up to which few tiles go to a pair each
cudaError_t launch_paged_append(const PagedAppendArgs& a, int sms, cudaStream_t s);
int paged_head_pad(int H);    // heads of an item, padded: 16, 32 or 64
int paged_unit_tiles();
int paged_max_ctas();         // most CTAs of one attention call
int paged_cluster(int64_t items, int64_t tiles, int sms);  // PagedAttnArgs::cluster
// units: the most units an item can have that are joined through the workspace (1: none is)
cudaError_t launch_paged_attn(const PagedAttnArgs& a, int units, cudaStream_t s);
// One CTA whose bounded wait runs out after limit_ns (test of the timeout path).
cudaError_t launch_wait_timeout(uint64_t limit_ns, cudaStream_t s);
cudaError_t launch_index(const IndexArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_plane_fp4_index(const uint16_t* k, int64_t n, uint8_t* plane, cudaStream_t s);
// bf16 plane rows [n][512] -> FP4 rows [n][288].
cudaError_t launch_plane_fp4(const uint16_t* rows, int64_t n, uint8_t* out, cudaStream_t s);
// bf16 index rows [n][128] -> FP8 plane (ceil(n / 8) blocks of 1056 bytes).
cudaError_t launch_plane_fp8(const uint16_t* k, int64_t n, uint8_t* plane, cudaStream_t s);
// One launch for selection `a` and, when b != null, a second selection over the same
// queries that runs beside it; when comp != null (comp->T > 0) further CTAs of the same
// launch run the compressor's tokens (csa2_compress_index_topk).
cudaError_t launch_topk(const TopkArgs& a, cudaStream_t s, const TopkArgs* b = nullptr,
                        const CompressArgs* comp = nullptr);
int attn_num_splits(int Q, int nsel, int num_sms);

// 2-D tensor map over `rows` bf16 rows of `cols` elements (row stride cols * 2 bytes),
// boxes of box_cols x box_rows, 128-byte swizzle, out-of-range elements read as zero.
// A tensor map over bytes: rank 2 to 5, dims[0] contiguous, strides[i] = byte stride of
// dims[i + 1]; 128-byte swizzle (box[0] must be 128).
bool encode_bytes(CUtensorMap* m, const void* base, int rank, const uint64_t* dims,
                  const uint64_t* strides, const uint32_t* box);
bool encode_rows_bf16(CUtensorMap* m, const void* base, uint64_t rows, uint32_t cols,
                      uint32_t box_cols, uint32_t box_rows);
cudaError_t launch_attn(const AttnArgs& a, int nsplit, cudaStream_t s);

int topk_chunk_len(int64_t ld);
int topk_num_chunks(int64_t ld);
int64_t topk_max_len();
// Can one call select the top-k of rows of ld items?  (the chunk merge holds chunks * k
// pairs)  topk_chunk_len / topk_num_chunks / topk_fits: the staged select of the
// candidate pool's blocks; topk_row_*: the row selection, whose rows of up to 65536
// positions run on one CTA.
bool topk_fits(int64_t ld, int k);
int topk_row_chunk_len(int64_t ld);
int topk_row_num_chunks(int64_t ld);
bool topk_row_fits(int64_t ld, int k);

// Replace the calling thread's csa2_last_error() text.
void set_last_error(const char* msg);

// Fault flags of each translation unit (read and cleared, host side).
int take_fault_compress();
int take_fault_index();
int take_fault_topk();
int take_fault_attn();
int take_fault_paged();
int take_fault_chunk();

// Order-preserving map of fp32 scores to uint32 keys: NaN ranks as -inf, -0 as +0,
// and every key of a real score is >= 1 so that 0 can mark "not scored".
// RoPE phase of position p for frequency theta: theta / (2 pi) is kept as a 64-bit binary
// fraction of a turn (its fractional part only), so (p * turn) mod 2^64 is the phase of
// p exactly in integer arithmetic; read as a signed fraction it is an angle in [-pi, pi).
__device__ __forceinline__ uint64_t rope_turn(float theta) {
  double tr = (double)theta * 0.15915494309189535;
  tr -= floor(tr);
  const double sc = tr * 18446744073709551616.0;  // 2^64
  return sc >= 18446744073709551615.0 ? ~0ull : (uint64_t)sc;
}
__device__ __forceinline__ float rope_angle(uint64_t turn, uint64_t p) {
  return (float)(int64_t)(p * turn) * 3.4061215800865545e-19f;  // 2 pi / 2^64
}

__device__ __forceinline__ void unpack_bf16x8(uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// A sink's logit in log2.  A finite one stays finite: the largest and lowest of fp32 overflow.
__device__ __forceinline__ float sink_log2(float sink) {
  const float y = sink * kLog2e;
  return isinf(y) && !isinf(sink) ? copysignf(FLT_MAX, sink) : y;
}

// ln Z of sums l (of rows and sink) under the maximum M; the sink itself where the rows' sum is 0.
__device__ __forceinline__ float head_lse(float M, float l, float rows, float sink) {
  return rows == 0.f ? sink : (M + __log2f(l)) * kLn2;
}

// Valid rows of the 64-row tile that begins at row r0, as bits.
__device__ __forceinline__ uint64_t tile_mask(int64_t r0, int lo, int hi) {
  const int64_t f = lo - r0, l = hi - r0;  // first valid, end
  uint64_t m = l >= 64 ? ~0ull : l <= 0 ? 0ull : (1ull << l) - 1;
  if (f >= 64) m = 0;
  else if (f > 0) m &= ~0ull << f;
  return m;
}

__host__ __device__ __forceinline__ uint32_t score_key(float f) {
  uint32_t u;
#ifdef __CUDA_ARCH__
  u = __float_as_uint(f);
#else
  memcpy(&u, &f, 4);
#endif
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) u = 0xFF800000u;  // NaN -> -inf
  if (u == 0x80000000u) u = 0u;                           // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__host__ __device__ __forceinline__ float key_score(uint32_t k) {
  uint32_t u = (k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k;
#ifdef __CUDA_ARCH__
  return __uint_as_float(u);
#else
  float f;
  memcpy(&f, &u, 4);
  return f;
#endif
}

}  // namespace csa2

// Host reader of this translation unit's fault flag.
#define CSA2_DEFINE_FAULT_FLAG(NAME)                                     \
  namespace csa2 {                                                       \
  int take_fault_##NAME() {                                              \
    int v = 0, z = 0;                                                    \
    if (cudaMemcpyFromSymbol(&v, g_fault, sizeof(int)) != cudaSuccess)   \
      return 0;                                                          \
    if (v) cudaMemcpyToSymbol(g_fault, &z, sizeof(int));                 \
    return v;                                                            \
  }                                                                      \
  }
