// Plans of the attention operators over the paged cache (swiftkv_attend, swiftkv_attention_weights
// and the model's own layers when a window or score pools are set): the host side lists the work of
// a ragged batch once, one upload takes it to the device, and any number of layers run from it.
#pragma once

#include <vector>

#include "launch.h"
#include "model_state.h"

namespace skv {

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
// (SWIFTKV_ESTATE) while `stream` is being captured, since that would need an allocation.
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
  bool tc = false, head_pairs = false;
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

// ---- kernels (attn_rows.cu, attn_weights.cu, evict.cu) --------------------------------------
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
constexpr int kWeightWarps = 12;  // warps per SM that walk units
cudaError_t launch_weights_rows(const WeightsArgs& a, const InlineInts& inl, const bf16* k, const uint8_t* k8,
                                const float* k_scale, int d_head, int max_cols, int num_units, int num_sms,
                                cudaStream_t s);
// Longer chunks on tcgen05: tiles [2 * num_tiles] = (sequence, 128-key tile), heaviest first. FP8:
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
