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
  __host__ __device__ bool pages_seen(int p, int q) const {  // pages p .. q all hold such keys, all of the sinks or all behind them
    return q * kPageSize < sinks || ((p + 1) * kPageSize > first && q * kPageSize < end);
  }
  __host__ __device__ bool page_seen(int p) const { return pages_seen(p, p); }  // page p holds a key that some row sees
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
// An 8-bit cache, and a dense bf16 copy of the pages a call needs: codes as bf16 values, scales beside them,
// rows that no row of the sequence's chunk sees as zeros. An item (sequence, page index, place)
// becomes the page at that place of the copy; places ascend, and those of `places` that no item names get scales that
// do no harm and nothing else. Dense and per sequence, so that sequences may share pages and the copy is no larger than
// what is read. by_head: the copy is [n_kv][places][16][d_head], a head's pages neighbours, so that one TMA copy takes
// a block of them; else [places][n_kv][16][d_head], every place an item's, and `block_table`, of the same shape as
// src's, names its pages.
// FP8: scales [...][16] likewise. Value scales are copied times kValueShift, which whoever multiplies P by them takes
// back: P times a scale goes to bf16, and value scales near float32's smallest would end up among bf16's subnormals.
// int8 (by_head): k_scale alone, [n_kv][places] records of a float4: the key scale times log2(e) / sqrt(d_head); lv,
// the binary logarithm of the value scale times kPageShift, by which exp2's argument rises so that P carries the
// value scale; 2^-lv; 0. Where that product is below 1, lv is what it has above a power of two and the copy's values
// carry that power, so that lv is never negative and P as far from float32's smallest as it is without it. Scales have
// to stay below 2^64.
constexpr float kValueShift = 65536.f;
constexpr float kPageShift = 268435456.f;
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
cudaError_t launch_kv_expand_seen(const int* items, int num_items, int places, int kind, bool by_head, const KVPool8& src, int max_pages,
                                  int num_pages, const int* cu, const int* ctx, int n_kv, int d_head, int window, int sinks,
                                  const KVExpansion& dst, int* status, cudaStream_t stream);

// Keys of a block of the tcgen05 attention, and where a sequence's blocks are in the expansion, behind its first:
// those of the sinks, then the others.
__host__ __device__ constexpr int chunk_block(int d_head) { return d_head == 128 ? 80 : 128; }
struct BlockOrder {
  int sinks, rest, end;  // blocks of the sinks alone; first of the others; past the last
  __host__ __device__ BlockOrder(int c0, int n, int window, int num_sinks, int bkv) {
    const TailPages t = tail_pages(c0, n, window, num_sinks);
    sinks = t.sinks > 0 && t.sinks < t.first ? (t.sinks + bkv - 1) / bkv : 0;
    rest = t.sinks >= t.first ? 0 : t.first / bkv > sinks ? t.first / bkv : sinks;
    end = (t.end + bkv - 1) / bkv;
  }
  __host__ __device__ int place(int block) const { return block < sinks ? block : block - rest + sinks; }
  __host__ __device__ int count() const { return place(end); }
};

// The blocks of a query tile, or of two, that starts at row q0 of its chunk and whose last starts at q1: those of the
// sinks [0, sinks), then [rest, end), one list of which a tile that ends before needs a prefix.
struct TileBlocks {
  int sinks, rest, end;
  __host__ __device__ TileBlocks(int c0, int n, int q0, int q1, int window, int num_sinks, int bkv) {
    const int seen = c0 + n < c0 + q1 + 128 ? c0 + n : c0 + q1 + 128, w0 = window_begin(c0 + q0, window);
    const int near = num_sinks < w0 ? num_sinks : w0;
    end = (seen + bkv - 1) / bkv;
    sinks = (near + bkv - 1) / bkv < end ? (near + bkv - 1) / bkv : end;
    rest = w0 / bkv > sinks ? w0 / bkv : sinks;
  }
  __host__ __device__ int entries(int last) const {
    return (sinks < last ? sinks : last) + (last > rest ? last - rest : 0);
  }
};

// kv_dtype of a cache
constexpr int kKvBf16 = 0, kKvFp8 = 1, kKvInt8 = 2;

// Host lists of a small call travel in the kernels' parameters instead of an upload of their own
// (which costs a launch: 2 us of a 26 us decode attention, a third of a tiny one). A kernel that may
// get them so reads its lists at list_base(dev, inl) + offset.
constexpr int kInlineInts = 1000;
struct alignas(16) InlineInts {
  int v[kInlineInts];
};
// The lists for the kernels' parameters (nothing of them where they were uploaded).
InlineInts inline_of(const std::vector<int>& ints, const int* dev);
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
  int kind = 0;  // kv_dtype
  int window = 0, sinks = 0;
  int max_pages = 0;
};

struct AttendPlan {
  Batch b;
  bool head_pairs = false;
  // host lists, and their places in one device upload
  std::vector<int> ints;
  int o_cu = 0, o_ctx = 0, o_tiles = 0, o_items = 0, o_units = 0, o_ubeg = 0, o_exp = 0, o_first = 0, o_merges = 0;
  int num_slots = 0, num_merges = 0;
  int num_tiles = 0, num_items = 0, max_cols = 0, num_units = 0;
  int num_exp = 0, places = 0;  // pages of the expansion, and places for them
  // device (lists: null where the kernels take them inline)
  int* dev = nullptr;
  float *part = nullptr, *tile_part = nullptr;
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
// (an item is a tile for one head, num_items = tiles * n_q). int8 with num_merges > 0: tiles [4 * n] = (seq << 16 | tile,
// first entry of its list of blocks, entries, slot of its partial result or -1), merges [3 * num_merges] = (tile, first
// slot, parts).
struct ChunkArgs {
  int kind;                        // kv_dtype
  const float *k_scale, *v_scale;  // 8-bit caches: the expansion's
  const int* exp_first;            // 8-bit caches: [P] each sequence's first page in the expansion of num_pages pages
  const int* bt;                   // bf16 cache
  int max_pages, num_pages;
  const int *cu, *ctx, *tiles;
  int num_items;
  const int* merges;
  int num_merges;
  float* part;             // [slots][items of a tile][2][128 * (d_head + 2)]
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
constexpr int kRowsWarps = 8, kRowsWarps8 = 12;  // warps per SM that walk units: bf16, 8-bit codes
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
cudaError_t launch_attn_rows(const RowsArgs& a, int kind, const InlineInts& inl, const void* k, const void* v, const float* k_scale, const float* v_scale,
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

// New rows of `caches` caches (append.cu): k and v [T] rows, ldk / ldv elements apart, a cache's heads k_step /
// v_step elements behind the one before; q [T] rows or null. Lists (null: inline): cu [P + 1], ctx [P], o_off
// (-1: none) [P] added to the positions of the rotation.
struct AppendArgs {
  const bf16* q;
  int ldq;
  bf16* q_out;
  int ldq_out;
  const bf16 *k, *v;
  int ldk, ldv;
  long long k_step, v_step;
  int caches, n_q, n_kv;
  int P, T;
  const int* lists;
  int o_cu, o_ctx, o_off;
  // addresses of the caches' K pools, and pool_step entries on of V's, of K's scales and of V's
  const long long* pools;  // null: in the lists, at o_pools
  int o_pools, pool_step;
  const int* bt;
  int max_pages, num_pages;
  bool rotate;
  const float2* rope_tab;
  int rope_len;
  const unsigned long long* rope_turn;
  int* status;
  // set by launch_append
  uint32_t per_cache;
  int splits, pages;
  unsigned row_warps;
};
// launch_append with the model's shape, rotation and status word.
cudaError_t launch_append_on(const swiftkv_model* m, AppendArgs a, int kind, const InlineInts& inl, cudaStream_t s);
cudaError_t launch_append(AppendArgs a, int kind, int d_head, const InlineInts& inl, int num_sms, cudaStream_t s);

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
