// Plans of the attention operators over the paged cache (swiftkv_attend, swiftkv_attention_weights
// and the model's own layers when a window or score pools are set): the host side lists the work of
// a ragged batch once, one upload takes it to the device, and any number of layers run from it.
#pragma once

#include <vector>

#include "launch.h"
#include "model_state.h"

namespace skv {

// A row at position p sees key j <= p when window == 0 or j > p - window or j < sinks. Pages that
// hold no visible key are not read, whatever their block-table entry; an entry outside the pool that
// is needed sets kStatusBadPage. Cached rows that no row sees may hold anything, NaN included.
// First key, past the sinks, that a row at position p sees.
__host__ __device__ __forceinline__ int window_begin(int p, int window) { return window > 0 && p >= window ? p - window + 1 : 0; }
__host__ __device__ __forceinline__ bool attn_visible(int key, int p, int window, int sinks) {
  return key <= p && (window <= 0 || key > p - window || key < sinks);
}
// Copies of the pages of V that a chunk sees in part, with the rows that none of its rows sees (past
// the sequence's end, before the first row's window, between the sinks and it) zero: out
// [P][kTailSlots][n_kv][16][d_head], slot 0 the last page, 1 the window's first, 2 the sinks' last.
// The tensor core multiplies whole pages, and a NaN in such a row would reach every output
// through 0 * NaN.
constexpr int kTailSlots = 3;
struct TailPages {
  int page[kTailSlots];  // page index within the sequence, -1: none
  int first, end, sinks;
  __host__ __device__ bool seen(int key) const { return key < end && (key >= first || key < sinks); }
};
__host__ __device__ __forceinline__ TailPages tail_pages(int c0, int n, int window, int sinks) {
  TailPages t;
  t.end = c0 + n;
  t.first = window_begin(c0, window);
  t.sinks = window > 0 && sinks < t.first ? sinks : t.first;
  t.page[0] = t.end % kPageSize ? t.end / kPageSize : -1;
  t.page[1] = t.first % kPageSize ? t.first / kPageSize : -1;
  t.page[2] = t.first > 0 && t.sinks % kPageSize ? t.sinks / kPageSize : -1;
  return t;
}
cudaError_t launch_v_tail(const bf16* v_pool, const int* block_table, int max_pages, int num_pages, const int* cu,
                          const int* ctx, int P, int n_kv, int d_head, int window, int sinks, bf16* out,
                          cudaStream_t stream);
// One FP8 cache, and a dense bf16 copy of the pages a call needs (codes as bf16 values, scales
// beside them, rows that no row of the sequence's chunk sees as zeros): item i = (sequence, page
// index) becomes page i, which `dst.block_table`, of the same shape as src's, then names. Dense
// and per sequence, so that sequences may share pages and the copy is no larger than what is read.
// Value scales are copied times kValueShift, which whoever multiplies P by them takes back: P times a
// scale goes to bf16, and value scales near float32's smallest would end up among bf16's subnormals.
constexpr float kValueShift = 65536.f;
struct KVPool8 {
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  const int* block_table;
};
struct KVExpansion {
  bf16 *k, *v;
  float *k_scale, *v_scale;
  int* block_table;
};
cudaError_t launch_kv_expand_seen(const int* items, int num_items, const KVPool8& src, int max_pages, int num_pages,
                                  const int* cu, const int* ctx, int n_kv, int d_head, int window, int sinks,
                                  const KVExpansion& dst, int* status, cudaStream_t stream);

// Host lists of a small call travel in the kernels' parameters instead of an upload of their own
// (which costs a launch: 2 us of a 26 us decode attention, a third of a tiny one). A kernel that may
// get them so reads its lists at list_base(dev, inl) + offset.
constexpr int kInlineInts = 1000;
struct alignas(16) InlineInts {
  int v[kInlineInts];
};
__device__ __forceinline__ const int* list_base(const int* dev, const InlineInts& inl) { return dev ? dev : inl.v; }

// Bump allocator over the model's operator workspace: sized by a first pass without a base.
struct Arena {
  char* base = nullptr;
  size_t used = 0;
  template <typename T>
  T* take(size_t count) {
    T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += (count * sizeof(T) + 255) / 256 * 256;
    return p;
  }
};
// Gives the arena `bytes` of the model's operator workspace, growing it where needed: refused
// (SWIFTKV_ESTATE) while `stream` is being captured, since that would need an allocation. One call of
// the library makes at most one reservation: a larger one later on would free what it uses.
int reserve(swiftkv_model* m, size_t bytes, cudaStream_t stream, Arena* arena);

// A ragged batch: chunk s is rows [cu[s], cu[s + 1]) at positions ctx[s] .. of sequence s.
struct Batch {
  int P = 0, T = 0;
  bool fp8 = false;
  int window = 0, sinks = 0;
  int max_pages = 0;
};

struct AttendPlan {
  Batch b;
  bool head_pairs = false;
  // host lists, and their places in one device upload
  std::vector<int> ints;
  int o_cu = 0, o_ctx = 0, o_tiles = 0, o_items = 0, o_units = 0, o_ubeg = 0, o_exp = 0;
  int num_tiles = 0, num_items = 0, max_cols = 0, num_units = 0, num_exp = 0;
  // device (lists: null where the kernels take them inline)
  int* dev = nullptr;
  float* part = nullptr;
  bf16* v_tail = nullptr;
  KVExpansion exp{};
  double keys = 0, pairs = 0;  // cached keys some row sees, and (row, key) pairs, for profiling

  // Validates cu / ctx against the block table and lists the work.
  int make(const swiftkv_model* m, const int32_t* cu, const int32_t* ctx, int P, const swiftkv_kv_pages* kv,
           int window, int sinks);
  void place(const swiftkv_model* m, Arena* a);
  int upload(cudaStream_t s) const;
  // Attention of q's rows over cache `c`; lse [n_q][ldl] may be null.
  int run(swiftkv_model* m, const swiftkv_kv_pages* kv, int c, const bf16* q, int ldq, bf16* out, int ldo, float* lse,
          int ldl, cudaStream_t s) const;
  int kernels() const;
};

struct WeightsPlan {
  Batch b;
  std::vector<int> ints;
  int o_cu = 0, o_ctx = 0, o_units = 0, o_tiles = 0, o_exp = 0;
  int num_units = 0, max_cols = 0, num_tiles = 0, num_exp = 0;
  int* dev = nullptr;
  KVExpansion exp{};
  double keys = 0, pairs = 0;

  int make(const swiftkv_model* m, const int32_t* cu, const int32_t* ctx, int P, const swiftkv_kv_pages* kv,
           int window, int sinks);
  void place(const swiftkv_model* m, Arena* a);
  int upload(cudaStream_t s) const;
  // scores[page][head][row] = decay * scores + the weight that q's rows gave to the key.
  int run(swiftkv_model* m, const swiftkv_kv_pages* kv, int c, const bf16* q, int ldq, const float* lse, int ldl,
          float decay, float* scores, cudaStream_t s) const;
  int kernels() const;
};

// ---- kernels (attn_chunk.cu, attn_rows.cu, attn_weights.cu, evict.cu) --------------------------------------
// Query tiles of longer chunks: tiles (seq << 16 | tile), heaviest first, of 128 rows (head_pairs:
// an item is a tile for two query heads of one KV head, num_items = tiles * n_q / 2) or of 256 rows
// (an item is a tile for one head, num_items = tiles * n_q).
struct ChunkArgs {
  const float *k_scale, *v_scale;  // FP8: the expansion's scales; else null
  const int* bt;
  int max_pages, num_pages;
  const int *cu, *ctx, *tiles;
  int num_items;
  bool head_pairs;
  int n_q, n_kv;
  int window, sinks;
  bf16* out;
  int ldo;
  float* lse;              // [n_q][ldl] or null
  int ldl;
  const bf16* v_tail;      // bf16 cache: launch_v_tail's copies of tail_seqs sequences
  int tail_seqs;
  int* status;
};
cudaError_t launch_attn_chunk(const ChunkArgs& a, const bf16* q, int ldq, int T, const bf16* k, const bf16* v, int d_head,
                              int num_sms, cudaStream_t s);
// Rows of short chunks: items [4 * n] = (first row, rows, sequence, first position), rows x group <=
// kRowsCols; units [3 * num_units] = (item, first key, keys) of keys some row sees, item-major; ubeg
// [n + 1]; part: num_units * n_kv * max_cols records of d_head + 4 floats (several units an item).
constexpr int kRowsCols = 16;
constexpr int kRowsWarps = 8, kRowsWarps8 = 12;  // warps per SM that walk units: bf16, FP8
struct RowsArgs {
  const bf16* q;
  int ldq;
  const int* bt;
  int max_pages, num_pages;
  const int* lists;  // null: inline
  int o_items, o_units, o_ubeg;
  int num_units, max_cols;
  int n_q, n_kv;
  int window, sinks;
  bf16* out;
  int ldo;
  float* lse;
  int ldl;
  float* part;
  int* status;
};
cudaError_t launch_attn_rows(const RowsArgs& a, const InlineInts& inl, const void* k, const void* v, const float* k_scale, const float* v_scale,
                             int d_head, int num_items, int num_sms, cudaStream_t s);
struct WeightsArgs {
  const bf16* q;
  int ldq, T;
  const float* lse;
  int ldl;
  const int* bt;
  int max_pages, num_pages;
  const int* lists;  // null: inline (rows kernel only)
  int o_cu, o_ctx, o_units;
  int window, sinks;
  int n_q, n_kv;
  float decay;
  float* scores;
  int* status;
};
// Chunks of few rows (rows x group <= kWeightCols): units [3 * num_units] = (sequence, first key,
// keys), one warp per unit and KV head at a time. FP8 cache: codes and scales of K.
constexpr int kWeightCols = 32;
constexpr int kWeightTile = 256;  // keys of an item of the tcgen05 kernel
constexpr int kWeightWarps = 12;  // warps per SM that walk units
cudaError_t launch_weights_rows(const WeightsArgs& a, const InlineInts& inl, const bf16* k, const uint8_t* k8,
                                const float* k_scale, int d_head, int max_cols, int num_units, int num_sms,
                                cudaStream_t s);
// Longer chunks on tcgen05: tiles [2 * num_tiles] = (sequence, kWeightTile-key tile), heaviest first. FP8:
// k / k_scale are an expansion (pages named by a.bt's counterpart `bt_k` of the same shape).
cudaError_t launch_weights_tc(const WeightsArgs& a, const bf16* k, const float* k_scale, const int* bt_k, int pages_k,
                              int d_head, const int* tiles, int num_tiles, int num_sms, cudaStream_t s);

struct EvictArgs {
  const int* lists;         // null: inline; [0, P): keys each sequence holds, then at o_ptrs the
  int o_ptrs, num_ptrs;     // pools of all num_ptrs caches: K, V, scores and, for FP8, both scales
  int P, first_cache, num_caches;
  int n_kv, row_bytes;      // bytes of one K or V row
  const int *src_bt, *dst_bt;
  int src_pages, dst_pages; // pages per block-table row
  int num_pages;
  int keep, sinks, recent;
  bool fp8;
  int* kept;                // [num_caches][P][n_kv][keep]
  int* status;
  bool in_place;
};
cudaError_t launch_evict(const EvictArgs& a, const InlineInts& inl, int max_len, cudaStream_t s);

}  // namespace skv
