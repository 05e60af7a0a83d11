// C-ABI entries of the operators over the paged cache: attention of new tokens with a window and
// sinks, the attention weight each cached key received, and eviction by it.
#include "serving.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

namespace skv {

namespace {

// Chunks of at most this many rows go to the row kernel, split along their keys; a 128-row query
// tile would be nearly empty (the serving forward's rule). Tiles over bf16 and FP8 are not split along the keys, so few
// short chunks after a long prefix leave SMs idle: one sequence, 32 / 8 heads x 128, bf16, 4 rows after
// 16000 keys 37 us, 5 rows 176; 8 sequences 98 and 179.
constexpr int kRowChunk = 4;
// Over an int8 cache, where tiles are cut along their keys (cut_tiles), by the same measure. us as rows for 5 / 8 / 12 / 16
// rows, and as tiles, for which these are all one:
//                            32 / 8 heads               40 / 8 heads               64 / 8 heads
//   1 sequence after 300     17 / 19 / 19 / 19    21    19 / 19 / 19 / 19    19    19 / 19 / 19 / 19    21
//   1 after 16000            46 / 46 / 52 / 56    64    47 / 51 / 56 / 68    82    48 / 56 / 68 / 82    88
//   8 after 300              19 / 21 / 21 / 23    23    21 / 21 / 23 / 27    29    21 / 23 / 27 / 31    29
//   8 after 16000            138 / 140 / 207 / 259 328  139 / 205 / 259 / 430 580  203 / 259 / 431 / 570 504
//   32 after 300             31 / 31 / 41 / 54    45    31 / 41 / 53 / 47    62    41 / 52 / 48 / 76    64
//   32 after 4000            158 / 160 / 234 / 352 340  160 / 232 / 351 / 426 489  230 / 353 / 429 / 565 479
// Rows take a pass over the keys for each 16 query heads and rows, so that the last of these 16 rows are dearer than a
// tile at 4 heads a KV head with many short sequences (by 4 to 18 %) and at 8 with several sequences (7 to 23 %).
constexpr int kRowChunkInt8 = 16;

int check_batch(const swiftkv_model* m, const int32_t* cu, const int32_t* ctx, int P, const swiftkv_kv_pages* kv,
                int window, int sinks, Batch* b) {
  if (cu[0] != 0) return fail(SWIFTKV_EINVAL_SEQLENS, "cu_seqlens[0] != 0");
  for (int i = 0; i < P; ++i) {
    const long long n = (long long)cu[i + 1] - cu[i], c0 = ctx ? ctx[i] : 0;
    if (n < 0) return fail(SWIFTKV_EINVAL_SEQLENS, "chunk %d has %lld tokens", i, n);
    if (c0 < 0) return fail(SWIFTKV_EINVAL_SEQLENS, "ctx_lens[%d] = %lld < 0", i, c0);
    if (c0 + n > (long long)kv->max_pages_per_seq * kPageSize)
      return fail(SWIFTKV_ENO_PAGES, "sequence %d needs %lld pages, block table holds %d", i, (c0 + n + 15) / 16,
                  kv->max_pages_per_seq);
    if (n > 65535LL * 64) return fail(SWIFTKV_EUNSUPPORTED, "chunk %d has more than 4194240 tokens", i);
  }
  if (window < 0 || sinks < 0) return fail(SWIFTKV_EINVAL, "negative window or sinks");
  if ((long long)kv->num_pages * m->cfg.n_kv * kPageSize >= 1LL << 31)
    return fail(SWIFTKV_EUNSUPPORTED, "a pool of 2^31 rows or more");
  if (kv->max_pages_per_seq > (1 << 26)) return fail(SWIFTKV_EUNSUPPORTED, "max_pages_per_seq above 2^26");
  b->P = P;
  b->T = cu[P];
  b->kind = kv->kv_dtype;
  b->window = window;
  b->sinks = window > 0 ? std::min(sinks, 1 << 30) : 0;
  b->max_pages = kv->max_pages_per_seq;
  return SWIFTKV_OK;
}

// Key ranges [k0, k1) that some row of a chunk sees: the sinks', then the rest.
struct Ranges {
  int n = 0, k0[2], k1[2];
};
Ranges seen_ranges(int c0, int n, int window, int sinks) {
  Ranges r;
  if (n < 1) return r;
  const TailPages t = tail_pages(c0, n, window, sinks);
  if (t.sinks > 0 && t.sinks < t.first) {
    r.k0[r.n] = 0;
    r.k1[r.n++] = t.sinks;
  }
  r.k0[r.n] = t.sinks >= t.first ? 0 : t.first;
  r.k1[r.n++] = t.end;
  return r;
}

int pages_of(int k0, int k1) { return k1 > k0 ? (k1 - 1) / kPageSize - k0 / kPageSize + 1 : 0; }

// Cuts the items' key ranges into units (item, first key, keys) of whole pages and about the same
// length, so that each of `warps` warps gets one per KV head: units of a fixed 128 or 256 keys left
// the last round of warps half empty (with the row kernel as it then was, attention of 24 rows of
// ~1100 keys, 40 / 8 heads: 22 against 25 us; 16 windows of 4100 FP8 keys: 60 against 83 us). The rounding of a row split this way
// depends on the call it is part of. ubeg [items + 1]: each item's first unit.
constexpr int kMinUnitPages = 4;   // below this a unit's partial result costs more than it spreads
constexpr int kMaxUnitPages = 64;  // with more items than warps: the last round stays short
void cut_units(const std::vector<int>& item_ids, const std::vector<Ranges>& seen, int n_kv, long long warps,
               std::vector<int>* units, std::vector<int>* ubeg) {
  auto count = [&](int len) {
    long long n = 0;
    for (const Ranges& r : seen)
      for (int i = 0; i < r.n; ++i) n += (pages_of(r.k0[i], r.k1[i]) + len - 1) / len;
    return n;
  };
  const long long budget = std::max(1LL, warps / n_kv);
  int lo = kMinUnitPages, hi = kMinUnitPages;
  for (const Ranges& r : seen)
    for (int i = 0; i < r.n; ++i) hi = std::max(hi, pages_of(r.k0[i], r.k1[i]));
  if (count(hi) > budget) lo = hi = std::min(hi, kMaxUnitPages);
  while (lo < hi) {  // the shortest length that fits the budget
    const int mid = (lo + hi) / 2;
    if (count(mid) <= budget) hi = mid;
    else lo = mid + 1;
  }
  units->reserve(3 * count(lo));
  if (ubeg) ubeg->assign(1, 0);
  for (size_t b = 0; b < seen.size(); ++b) {
    for (int i = 0; i < seen[b].n; ++i) {
      const int k0 = seen[b].k0[i], k1 = seen[b].k1[i], p0 = k0 / kPageSize;
      const long long np = pages_of(k0, k1), nu = (np + lo - 1) / lo;
      for (long long u = 0; u < nu; ++u) {
        const int a = std::max(k0, (p0 + (int)(np * u / nu)) * kPageSize);
        const int e = (int)std::min<long long>(k1, (p0 + np * (u + 1) / nu) * kPageSize);
        units->insert(units->end(), {item_ids[b], a, e - a});
      }
    }
    if (ubeg) ubeg->push_back((int)(units->size() / 3));
  }
}

// (sequence, page, place) of the pages some row of the chunk sees.
void list_pages(int s, int c0, int n, int window, int sinks, std::vector<int>* out) {
  const Ranges r = seen_ranges(c0, n, window, sinks);
  int next = 0;
  for (int i = 0; i < r.n; ++i)
    for (int p = std::max(next, r.k0[i] / kPageSize); p < (r.k1[i] + kPageSize - 1) / kPageSize; ++p) {
      out->insert(out->end(), {s, p, (int)(out->size() / 3)});
      next = p + 1;
    }
}

// The same in blocks of `bkv` keys that hold such a page, in BlockOrder's order: all pages of a block take a place.
void list_blocks(int s, int c0, int n, int window, int sinks, int bkv, int* places, std::vector<int>* out) {
  const BlockOrder o(c0, n, window, sinks, bkv);
  const TailPages t = tail_pages(c0, n, window, sinks);
  auto put_block = [&](int b) {
    for (int p = b * (bkv / kPageSize); p < (b + 1) * (bkv / kPageSize); ++p, ++*places)
      if (t.page_seen(p)) out->insert(out->end(), {s, p, *places});
  };
  for (int b = 0; b < o.sinks; ++b) put_block(b);
  for (int b = o.rest; b < o.end; ++b) put_block(b);
}

void count_work(const int32_t* cu, const int32_t* ctx, const Batch& b, double* keys, double* pairs) {
  for (int i = 0; i < b.P; ++i) {
    const int n = cu[i + 1] - cu[i], c0 = ctx ? ctx[i] : 0;
    const Ranges r = seen_ranges(c0, n, b.window, b.sinks);
    for (int k = 0; k < r.n; ++k) *keys += r.k1[k] - r.k0[k];
    const double w = b.window > 0 ? b.window : 1e18, s = b.sinks;
    // rows at c0 .. c0 + n - 1 see min(p + 1, w) keys of the window and min(s, p + 1 - w) sinks
    auto sum = [&](double lim, double shift) {  // sum over p of clamp(p + 1 - shift, 0, lim)
      double t = 0;
      const double a = c0 + 1 - shift, z = c0 + n - shift;  // first and last p + 1 - shift
      const double u = std::min(z, lim), l = std::max(a, 1.0);
      if (u >= l) t += (u - l + 1) * (u + l) / 2;
      if (z > lim) t += (z - std::max(lim, a - 1)) * lim;
      return t;
    };
    if (n > 0) *pairs += sum(w, 0) + (b.window > 0 ? sum(s, w) : 0);
  }
}

// Cuts tiles (seq << 16 | tile, of so many blocks each, heaviest first) along their lists of blocks where there are too
// few to keep the SMs busy: entries of ChunkArgs::tiles, heaviest first, and its merges; none of the two where whole tiles
// are as good. `per` items run for each. Parts fill the rounds that whole tiles take, the last of which would be half
// empty, and are no shorter than kMinPart blocks. Whether that pays is counted as the kernel deals items out, with
// kStart blocks' time for an item's start and end, twice that for a part's, and kMerge for the join.
// int8, 32 / 8 heads x 128, us whole / cut: 1 sequence, 24 and 64 rows after 16000 keys 206 / 62, 128 after 6048 93 / 41, 512
// 98 / 70, 2016 191 / 185 (2016 after none 49 / 55: left whole); 2 and 4 sequences, 32 rows after 8000 121 / 64 and 140 / 103.
constexpr int kMinPart = 8, kStart = 2, kMerge = 6, kFullRounds = 4;
void cut_tiles(const std::vector<int>& tiles, const std::vector<int>& blocks, int per, int num_sms, std::vector<int>* out,
               std::vector<int>* merges, int* num_slots) {
  struct Part {
    int tile, from, n, slot;
  };
  const long long items = (long long)tiles.size() * per, rounds = (items + num_sms - 1) / num_sms;
  if (items >= (long long)kFullRounds * num_sms) return;
  auto longest = [&](const std::vector<Part>& parts) {  // blocks of the SM that has most
    std::vector<long long> load(num_sms, 0);
    long long w = 0, most = 0;
    for (const Part& p : parts)
      for (int k = 0; k < per; ++k, ++w) {
        const long long it = w / num_sms, c = w % num_sms;
        most = std::max(most, load[it & 1 ? num_sms - 1 - c : c] += p.n + (p.slot < 0 ? kStart : 2 * kStart));
      }
    return most;
  };
  std::vector<Part> whole, parts;
  long long most = 1;
  for (size_t i = 0; i < tiles.size(); ++i) {
    whole.push_back({tiles[i], 0, blocks[i], -1});
    most = std::max<long long>(most, blocks[i]);
  }
  int lo = (int)std::min<long long>(kMinPart, most), len = (int)most;
  while (lo < len) {  // the shortest length that keeps to the rounds
    const int mid = (lo + len) / 2;
    long long n = 0;
    for (int b : blocks) n += (b + mid - 1) / mid;
    if (n * per <= rounds * num_sms) len = mid;
    else lo = mid + 1;
  }
  std::vector<int> joins;
  int slots = 0;
  for (size_t i = 0; i < tiles.size(); ++i) {
    const int n = blocks[i], p = (n + len - 1) / len;
    if (p <= 1) {
      parts.push_back(whole[i]);
      continue;
    }
    joins.insert(joins.end(), {tiles[i], slots, p});
    for (int k = 0; k < p; ++k) {
      const int a = (int)((long long)n * k / p), e = (int)((long long)n * (k + 1) / p);
      parts.push_back({tiles[i], a, e - a, slots++});
    }
  }
  auto heavier = [](const Part& x, const Part& y) { return x.n > y.n; };
  std::stable_sort(whole.begin(), whole.end(), heavier);
  std::stable_sort(parts.begin(), parts.end(), heavier);
  if (joins.empty() || longest(parts) + kMerge >= longest(whole)) return;
  for (const Part& p : parts) out->insert(out->end(), {p.tile, p.from, p.n, p.slot});
  merges->swap(joins);
  *num_slots = slots;
}

int put(std::vector<int>* ints, const std::vector<int>& v) {
  const int at = (int)ints->size();
  ints->insert(ints->end(), v.begin(), v.end());
  return at;
}

void place_expansion(const swiftkv_model* m, Arena* a, int pages, const Batch& b, bool with_v, KVExpansion* e) {
  if (pages <= 0) return;
  const size_t rows = (size_t)pages * m->cfg.n_kv * kPageSize;
  e->k = a->take<bf16>(rows * m->cfg.d_head);
  e->v = with_v ? a->take<bf16>(rows * m->cfg.d_head) : nullptr;
  e->k_scale = a->take<float>(b.kind == kKvInt8 ? rows / kPageSize * 4 : rows);  // int8: a record a page and head
  e->v_scale = with_v && b.kind == kKvFp8 ? a->take<float>(rows) : nullptr;
  e->block_table = with_v ? nullptr : a->take<int>((size_t)b.P * b.max_pages);
}

int expand(swiftkv_model* m, const swiftkv_kv_pages* kv, int c, const Batch& b, const int* items, int num,
           int places, const int* cu, const int* ctx, bool by_head, const KVExpansion& e, cudaStream_t s) {
  KVPool8 src;
  src.k = static_cast<const uint8_t*>(kv->k_pool[c]);
  src.v = static_cast<const uint8_t*>(kv->v_pool[c]);
  src.k_scale = static_cast<const float*>(kv->k_scale[c]);
  src.v_scale = static_cast<const float*>(kv->v_scale[c]);
  src.block_table = kv->block_table;
  CK(launch_kv_expand_seen(items, num, places, b.kind, by_head, src, b.max_pages, kv->num_pages, cu, ctx, m->cfg.n_kv, m->cfg.d_head, b.window,
                           b.sinks, e, m->status, s));
  return SWIFTKV_OK;
}

// The model's operator workspace holds `bytes`. One that a captured graph uses stays when it is outgrown.
int hold(swiftkv_model* m, size_t bytes, cudaStream_t stream) {
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  CK(cudaStreamIsCapturing(stream, &cap));
  const bool capturing = cap != cudaStreamCaptureStatusNone;
  if (bytes > m->ops_bytes) {
    if (capturing)
      return fail(SWIFTKV_ESTATE, "the workspace must grow to %zu bytes: make one such call before the capture", bytes);
    if (m->ops_ws && m->ops_captured) {
      m->allocs.push_back(m->ops_ws);
      m->ops_kept_bytes += m->ops_bytes;
    } else if (m->ops_ws) {
      CK(cudaFree(m->ops_ws));  // synchronises the device: no enqueued work still uses it
    }
    m->ops_ws = nullptr;
    m->ops_bytes = 0;
    m->ops_captured = false;
    const size_t want = std::max(bytes + bytes / 4, (size_t)1 << 20);
    void* p = nullptr;
    const cudaError_t e = cudaMalloc(&p, want);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return fail(SWIFTKV_EOOM, "workspace cudaMalloc(%zu): %s", want, cudaGetErrorString(e));
    }
    m->ops_ws = static_cast<char*>(p);
    m->ops_bytes = want;
  }
  m->ops_captured |= capturing;
  return SWIFTKV_OK;
}

}  // namespace

InlineInts inline_of(const std::vector<int>& ints, const int* dev) {
  InlineInts r;
  if (!dev) memcpy(r.v, ints.data(), ints.size() * 4);
  return r;
}

int reserve(swiftkv_model* m, size_t bytes, cudaStream_t stream, Arena* arena) {
  if (bytes > 0) RET(guarded([&] { return hold(m, bytes, stream); }));
  arena->base = m->ops_ws;
  arena->used = 0;
  return SWIFTKV_OK;
}

cudaError_t launch_append_on(const swiftkv_model* m, AppendArgs a, int kind, const InlineInts& inl, cudaStream_t s) {
  a.n_q = m->cfg.n_q;
  a.n_kv = m->cfg.n_kv;
  a.rope_tab = m->rope_tab;
  a.rope_len = kRopeLen;
  a.rope_turn = m->rope_turn;
  a.status = m->status;
  return launch_append(a, kind, m->cfg.d_head, inl, m->num_sms, s);
}

// ---------------------------------------------------------------------------- attention

int AttendPlan::make(const swiftkv_model* m, const int32_t* cu, const int32_t* ctx, int P, const swiftkv_kv_pages* kv,
                     int window, int sinks) {
  RET(check_batch(m, cu, ctx, P, kv, window, sinks, &b));
  const auto& c = m->cfg;
  head_pairs = (c.n_q / c.n_kv) % 2 == 0;
  const int tile_rows = head_pairs ? 128 : 256;
  std::vector<int> cuv(cu, cu + P + 1), ctxv(P, 0), tiles, items, ids, exp_items, first;
  if (b.kind != kKvBf16) first.assign(P, 0);
  std::vector<Ranges> seen;
  items.reserve(4 * P);
  ids.reserve(P);
  seen.reserve(P);
  const int G = c.n_q / c.n_kv, group = kRowsCols / G;  // rows of an item of the row kernel
  for (int i = 0; i < P; ++i) {
    const int n = cu[i + 1] - cu[i], c0 = ctx ? ctx[i] : 0;
    ctxv[i] = c0;
    if (n <= (b.kind == kKvInt8 ? kRowChunkInt8 : kRowChunk)) {
      for (int r = 0; r < n; r += group) {
        const int rows = std::min(group, n - r);
        ids.push_back((int)ids.size());
        items.insert(items.end(), {cu[i] + r, rows, i, c0 + r});
        seen.push_back(seen_ranges(c0 + r, rows, b.window, b.sinks));
        max_cols = std::max(max_cols, rows * G);
      }
      continue;
    }
    for (int t = 0; t < (n + tile_rows - 1) / tile_rows; ++t) tiles.push_back((i << 16) | t);
    if (b.kind != kKvBf16) {
      first[i] = places;
      list_blocks(i, c0, n, b.window, b.sinks, chunk_block(c.d_head), &places, &exp_items);
      if (places >= 1 << 27) return fail(SWIFTKV_EUNSUPPORTED, "batch too large");
    }
  }
  // heaviest first: the keys that a tile's last row sees
  auto keys_of = [&](int tl) {
    const int p = ctxv[tl >> 16] + ((tl & 0xffff) + 1) * tile_rows;
    return b.window > 0 ? std::min((long long)p, (long long)b.window + b.sinks + tile_rows) : (long long)p;
  };
  std::stable_sort(tiles.begin(), tiles.end(), [&](int x, int y) { return keys_of(x) > keys_of(y); });
  num_tiles = (int)tiles.size();
  std::vector<int> merges;
  if (b.kind == kKvInt8 && num_tiles > 0) {
    std::vector<int> blocks, cut;
    for (int tl : tiles) {
      const int i = tl >> 16, n = cu[i + 1] - cu[i], q0 = (tl & 0xffff) * tile_rows;
      const int q1 = !head_pairs && q0 + 128 < n ? q0 + 128 : q0;
      const TileBlocks t(ctxv[i], n, q0, q1, b.window, b.sinks, chunk_block(c.d_head));
      blocks.push_back(t.entries(t.end));
    }
    cut_tiles(tiles, blocks, head_pairs ? c.n_q / 2 : c.n_q, m->num_sms, &cut, &merges, &num_slots);
    num_merges = (int)(merges.size() / 3);
    if (num_merges > 0) {
      num_tiles = (int)(cut.size() / 4);
      tiles.swap(cut);
    }
  }
  std::vector<int> units, ubeg;
  if (!ids.empty())
    cut_units(ids, seen, c.n_kv, (long long)m->num_sms * (b.kind != kKvBf16 ? kRowsWarps8 : kRowsWarps), &units, &ubeg);
  num_items = (int)ids.size();
  num_units = (int)(units.size() / 3);
  num_exp = (int)(exp_items.size() / 3);
  // offsets into the lists and the kernels' item counts are ints
  if (std::max({units.size(), tiles.size(), exp_items.size()}) >= (size_t)1 << 28 ||
      (long long)num_units * c.n_kv >= (1LL << 31) || (long long)num_tiles * c.n_q >= (1LL << 31))
    return fail(SWIFTKV_EUNSUPPORTED, "batch too large");
  ints.reserve(3 * cuv.size() + tiles.size() + merges.size() + 8 + units.size() + exp_items.size() + ubeg.size() + items.size());
  o_cu = put(&ints, cuv);
  o_ctx = put(&ints, ctxv);
  while (num_merges > 0 && ints.size() % 4) ints.push_back(0);  // entries of 16 bytes
  o_tiles = put(&ints, tiles);
  o_merges = put(&ints, merges);
  o_items = put(&ints, items);
  o_units = put(&ints, units);
  o_ubeg = put(&ints, ubeg);
  if (num_exp > 0) {
    o_exp = put(&ints, exp_items);
    o_first = put(&ints, first);
  }
  if (m->prof_on) count_work(cu, ctx, b, &keys, &pairs);
  return SWIFTKV_OK;
}

void AttendPlan::place(const swiftkv_model* m, Arena* a) {
  const auto& c = m->cfg;
  dev = num_tiles > 0 || ints.size() > kInlineInts ? a->take<int>(ints.size()) : nullptr;
  part = a->take<float>(num_units > num_items ? (size_t)num_units * c.n_kv * max_cols * (c.d_head + 4) : 0);
  tile_part = a->take<float>((size_t)num_slots * (head_pairs ? c.n_q / 2 : c.n_q) * 2 * 128 * (c.d_head + 2));
  v_tail = nullptr;
  if (num_tiles > 0 && b.kind == kKvBf16)
    v_tail = a->take<bf16>((size_t)b.P * kTailSlots * c.n_kv * kPageSize * c.d_head);
  place_expansion(m, a, places, b, true, &exp);
}

int AttendPlan::upload(cudaStream_t s) const {
  if (dev) CK(upload_ints(dev, ints.data(), (int)ints.size(), s));
  return SWIFTKV_OK;
}

int AttendPlan::run(swiftkv_model* m, const swiftkv_kv_pages* kv, int c, const bf16* q, int ldq, bf16* out, int ldo,
                    float* lse, int ldl, cudaStream_t s) const {
  const auto& g = m->cfg;
  cudaError_t e = cudaSuccess;
  if (num_tiles > 0) {
    ChunkArgs t;
    const bf16* k = static_cast<const bf16*>(kv->k_pool[c]);
    const bf16* v = static_cast<const bf16*>(kv->v_pool[c]);
    t.kind = b.kind;
    t.k_scale = t.v_scale = nullptr;
    t.exp_first = nullptr;
    t.bt = kv->block_table;
    t.num_pages = kv->num_pages;
    t.v_tail = nullptr;
    t.tail_seqs = b.P;
    t.cu = dev + o_cu;
    t.ctx = dev + o_ctx;
    if (b.kind != kKvBf16) {
      RET(expand(m, kv, c, b, dev + o_exp, num_exp, places, t.cu, t.ctx, true, exp, s));
      t.exp_first = dev + o_first;
      k = exp.k;
      v = exp.v;
      t.k_scale = exp.k_scale;
      t.v_scale = exp.v_scale;
      t.bt = nullptr;
      t.num_pages = places;
    } else {
      CK(launch_v_tail(v, t.bt, b.max_pages, t.num_pages, t.cu, t.ctx, b.P, g.n_kv, g.d_head, b.window, b.sinks, v_tail, s));
      t.v_tail = v_tail;
    }
    t.max_pages = b.max_pages;
    t.tiles = dev + o_tiles;
    t.merges = dev + o_merges;
    t.num_merges = num_merges;
    t.part = tile_part;
    t.num_items = num_tiles * (head_pairs ? g.n_q / 2 : g.n_q);
    t.head_pairs = head_pairs;
    t.n_q = g.n_q;
    t.n_kv = g.n_kv;
    t.window = b.window;
    t.sinks = b.sinks;
    t.out = out;
    t.ldo = ldo;
    t.lse = lse;
    t.ldl = ldl;
    t.status = m->status;
    e = launch_attn_chunk(t, q, ldq, b.T, k, v, g.d_head, m->num_sms, s);
  }
  if (e == cudaSuccess && num_items > 0) {
    RowsArgs r;
    r.q = q;
    r.ldq = ldq;
    r.bt = kv->block_table;
    r.max_pages = b.max_pages;
    r.num_pages = kv->num_pages;
    r.lists = dev;
    r.o_items = o_items;
    r.o_units = o_units;
    r.o_ubeg = o_ubeg;
    r.num_units = num_units;
    r.max_cols = max_cols;
    r.n_q = g.n_q;
    r.n_kv = g.n_kv;
    r.window = b.window;
    r.sinks = b.sinks;
    r.out = out;
    r.ldo = ldo;
    r.lse = lse;
    r.ldl = ldl;
    r.part = part;
    r.status = m->status;
    e = launch_attn_rows(r, b.kind, inline_of(ints, dev), kv->k_pool[c], kv->v_pool[c],
                         b.kind != kKvBf16 ? static_cast<const float*>(kv->k_scale[c]) : nullptr,
                         b.kind != kKvBf16 ? static_cast<const float*>(kv->v_scale[c]) : nullptr, g.d_head, num_items, m->num_sms, s);
  }
  if (e != cudaSuccess)
    return fail(e == cudaErrorNotSupported ? SWIFTKV_EUNSUPPORTED : SWIFTKV_ECUDA, "attention: %s", cudaGetErrorString(e));
  return SWIFTKV_OK;
}

int AttendPlan::kernels() const {
  return (num_tiles > 0 ? 2 + (num_merges > 0) : 0) + (num_items > 0 ? 1 + (num_units > num_items) : 0);
}

// ---------------------------------------------------------------------------- attention weights

int WeightsPlan::make(const swiftkv_model* m, const int32_t* cu, const int32_t* ctx, int P, const swiftkv_kv_pages* kv,
                      int window, int sinks) {
  RET(check_batch(m, cu, ctx, P, kv, window, sinks, &b));
  const auto& c = m->cfg;
  const int G = c.n_q / c.n_kv;
  std::vector<int> cuv(cu, cu + P + 1), ctxv(P, 0), ids, units, tiles, exp_items;
  std::vector<Ranges> seen;
  std::vector<std::pair<long long, std::pair<int, int>>> heavy;  // (rows that see the tile, (sequence, tile))
  for (int i = 0; i < P; ++i) {
    const int n = cu[i + 1] - cu[i], c0 = ctx ? ctx[i] : 0;
    ctxv[i] = c0;
    const Ranges r = seen_ranges(c0, n, b.window, b.sinks);
    if (n * (long long)G <= kWeightCols) {
      max_cols = std::max(max_cols, n * G);
      if (r.n > 0) {
        ids.push_back(i);
        seen.push_back(r);
      }
      continue;
    }
    int next = 0;
    for (int k = 0; k < r.n; ++k)
      for (int t = std::max(next, r.k0[k] / kWeightTile); t < (r.k1[k] + kWeightTile - 1) / kWeightTile; ++t) {
        const long long key0 = (long long)t * kWeightTile, first = std::max(0LL, key0 - c0);
        long long last = n;
        if (b.window > 0 && key0 >= b.sinks) last = std::min<long long>(n, key0 + kWeightTile - 1 + b.window - c0);
        heavy.push_back({last - first, {i, t}});
        next = t + 1;
      }
    if (b.kind != kKvBf16) list_pages(i, c0, n, b.window, b.sinks, &exp_items);
  }
  if (!ids.empty()) cut_units(ids, seen, c.n_kv, (long long)m->num_sms * kWeightWarps, &units, nullptr);
  std::stable_sort(heavy.begin(), heavy.end(), [](const auto& x, const auto& y) { return x.first > y.first; });
  for (const auto& h : heavy) {
    tiles.push_back(h.second.first);
    tiles.push_back(h.second.second);
  }
  num_units = (int)(units.size() / 3);
  num_tiles = (int)(tiles.size() / 2);
  num_exp = (int)(exp_items.size() / 3);
  if (std::max({units.size(), tiles.size(), exp_items.size()}) >= (size_t)1 << 28 ||
      (long long)num_units * c.n_kv >= (1LL << 31) || (long long)num_tiles * c.n_kv >= (1LL << 31))
    return fail(SWIFTKV_EUNSUPPORTED, "batch too large");
  ints.reserve(2 * cuv.size() + tiles.size() + units.size() + exp_items.size());
  o_cu = put(&ints, cuv);
  o_ctx = put(&ints, ctxv);
  o_units = put(&ints, units);
  o_tiles = put(&ints, tiles);
  o_exp = put(&ints, exp_items);
  if (m->prof_on) count_work(cu, ctx, b, &keys, &pairs);
  return SWIFTKV_OK;
}

void WeightsPlan::place(const swiftkv_model* m, Arena* a) {
  dev = num_tiles > 0 || ints.size() > kInlineInts ? a->take<int>(ints.size()) : nullptr;
  place_expansion(m, a, num_exp, b, false, &exp);
}

int WeightsPlan::upload(cudaStream_t s) const {
  if (dev) CK(upload_ints(dev, ints.data(), (int)ints.size(), s));
  return SWIFTKV_OK;
}

int WeightsPlan::run(swiftkv_model* m, const swiftkv_kv_pages* kv, int c, const bf16* q, int ldq, const float* lse,
                     int ldl, float decay, float* scores, cudaStream_t s) const {
  const auto& g = m->cfg;
  WeightsArgs a;
  a.q = q;
  a.ldq = ldq;
  a.T = b.T;
  a.lse = lse;
  a.ldl = ldl;
  a.bt = kv->block_table;
  a.max_pages = b.max_pages;
  a.num_pages = kv->num_pages;
  a.lists = dev;
  a.o_cu = o_cu;
  a.o_ctx = o_ctx;
  a.o_units = o_units;
  a.window = b.window;
  a.sinks = b.sinks;
  a.n_q = g.n_q;
  a.n_kv = g.n_kv;
  a.decay = decay;
  a.scores = scores;
  a.status = m->status;
  cudaError_t e = cudaSuccess;
  if (num_units > 0)
    e = launch_weights_rows(a, inline_of(ints, dev), (b.kind == kKvFp8) ? nullptr : static_cast<const bf16*>(kv->k_pool[c]),
                            (b.kind == kKvFp8) ? static_cast<const uint8_t*>(kv->k_pool[c]) : nullptr,
                            (b.kind == kKvFp8) ? static_cast<const float*>(kv->k_scale[c]) : nullptr, g.d_head, max_cols,
                            num_units, m->num_sms, s);
  if (e == cudaSuccess && num_tiles > 0) {
    if ((b.kind == kKvFp8)) {
      RET(expand(m, kv, c, b, dev + o_exp, num_exp, num_exp, dev + o_cu, dev + o_ctx, false, exp, s));
      e = launch_weights_tc(a, exp.k, exp.k_scale, exp.block_table, num_exp, g.d_head, dev + o_tiles, num_tiles,
                            m->num_sms, s);
    } else {
      e = launch_weights_tc(a, static_cast<const bf16*>(kv->k_pool[c]), nullptr, kv->block_table, kv->num_pages,
                            g.d_head, dev + o_tiles, num_tiles, m->num_sms, s);
    }
  }
  if (e != cudaSuccess)
    return fail(e == cudaErrorNotSupported ? SWIFTKV_EUNSUPPORTED : SWIFTKV_ECUDA, "attention weights: %s",
                cudaGetErrorString(e));
  return SWIFTKV_OK;
}

int WeightsPlan::kernels() const { return (num_units > 0) + (num_tiles > 0 ? 1 + (b.kind == kKvFp8) : 0); }

}  // namespace skv

// ============================================================================ C ABI

using namespace skv;

namespace {

int check_call(const swiftkv_model* m, int cache, int P, const swiftkv_kv_pages* kv) {
  if (!m) return fail(SWIFTKV_EINVAL, "null model");
  if (P < 0 || P > 32767) return fail(SWIFTKV_EINVAL, "num_seqs %d outside [0, 32767]", P);
  RET(check_kv(m, kv));
  if (cache < 0 || cache >= m->C) return fail(SWIFTKV_EINVAL, "cache %d outside [0, %d)", cache, m->C);
  return SWIFTKV_OK;
}

// The caches' operators that know no block scales: weights by the key, and moves between pages.
int check_no_blocks(const swiftkv_kv_pages* kv, const char* name) {
  return kv->kv_dtype == kKvInt8 ? fail(SWIFTKV_EUNSUPPORTED, "%s over an int8 cache", name) : (int)SWIFTKV_OK;
}

// Keys of a sequence, and of its kept list: the kernels step through them in ints, past the end.
constexpr int kMaxKeys = 1 << 30;

int check_width(const void* p, int ld, long long width, const char* name) {
  if (!p) return fail(SWIFTKV_EINVAL, "null %s", name);
  if (ld < width || ld % 8 || (reinterpret_cast<uintptr_t>(p) & 15))
    return fail(SWIFTKV_EINVAL, "%s: rows need a stride of at least %lld, a multiple of 8, and 16-byte alignment", name,
                width);
  return SWIFTKV_OK;
}
int check_rows(const swiftkv_model* m, const void* p, int ld, const char* name) { return check_width(p, ld, m->Nq, name); }

}  // namespace

extern "C" {

int swiftkv_attend(swiftkv_model* m, int cache, const void* q, int ldq, const int32_t* cu, const int32_t* ctx, int P,
                   const swiftkv_kv_pages* kv, int window, int sinks, void* out, int ldo, float* lse,
                   swiftkv_stream stream) {
  return guarded([&]() -> int {
    RET(check_call(m, cache, P, kv));
    if (P == 0) return SWIFTKV_OK;
    if (!cu) return fail(SWIFTKV_EINVAL, "null cu_seqlens");
    AttendPlan p;
    RET(p.make(m, cu, ctx, P, kv, window, sinks));
    if (p.b.T == 0) return SWIFTKV_OK;
    RET(check_rows(m, q, ldq, "q"));
    RET(check_rows(m, out, ldo, "out"));
    const char *qa = static_cast<const char*>(q), *oa = static_cast<const char*>(out);
    const size_t qn = ((size_t)(p.b.T - 1) * ldq + m->Nq) * 2, on = ((size_t)(p.b.T - 1) * ldo + m->Nq) * 2;
    if (qa < oa + on && oa < qa + qn) return fail(SWIFTKV_EINVAL, "out overlaps q");
    if (reinterpret_cast<uintptr_t>(lse) & 3) return fail(SWIFTKV_EINVAL, "misaligned lse");
    OnDevice on_device(m);
    cudaStream_t s = (cudaStream_t)stream;
    Arena size, arena;
    p.place(m, &size);
    RET(reserve(m, size.used, s, &arena));
    p.place(m, &arena);
    RET(p.upload(s));
    return p.run(m, kv, cache, static_cast<const bf16*>(q), ldq, static_cast<bf16*>(out), ldo, lse, p.b.T, s);
  });
}

int swiftkv_append(swiftkv_model* m, int cache, int caches, const swiftkv_new_rows* rows, const int32_t* cu,
                   const int32_t* ctx, const int32_t* pos_off, int P, const swiftkv_kv_pages* kv, int rotate,
                   swiftkv_stream stream) {
  return guarded([&]() -> int {
    RET(check_call(m, cache, P, kv));
    if (caches < 1 || caches > m->C - cache)
      return fail(SWIFTKV_EINVAL, "caches %d .. %lld of %d", cache, (long long)cache + caches - 1, m->C);
    if (P == 0) return SWIFTKV_OK;
    if (!cu || !rows) return fail(SWIFTKV_EINVAL, "null cu_seqlens / rows");
    Batch b;
    RET(check_batch(m, cu, ctx, P, kv, 0, 0, &b));
    for (int i = 0; i < P; ++i) {
      const long long end = (ctx ? ctx[i] : 0) + (long long)(cu[i + 1] - cu[i]), off = pos_off ? pos_off[i] : 0;
      if (off < 0 || off + end > (1LL << 30))
        return fail(SWIFTKV_EINVAL_SEQLENS, "sequence %d: positions outside [0, 2^30)", i);
    }
    if (b.T == 0) return SWIFTKV_OK;
    const long long Nkv = m->Nkv, most = 0x7fffffff;  // no step is longer than a row
    if (caches > 1 && (rows->k_step < Nkv || rows->v_step < Nkv || rows->k_step > most || rows->v_step > most ||
                       rows->k_step % 8 || rows->v_step % 8))
      return fail(SWIFTKV_EINVAL, "k_step, v_step: from %lld to a row's stride and a multiple of 8", Nkv);
    const long long k_width = caches > 1 ? (caches - 1) * rows->k_step + Nkv : Nkv;
    const long long v_width = caches > 1 ? (caches - 1) * rows->v_step + Nkv : Nkv;
    RET(check_width(rows->k, rows->ldk, k_width, "k"));
    RET(check_width(rows->v, rows->ldv, v_width, "v"));
    if (rows->q) {
      RET(check_rows(m, rows->q, rows->ldq, "q"));
      RET(check_rows(m, rows->q_out, rows->ldq_out, "q_out"));
      if (!(rows->q == rows->q_out && (rows->ldq == rows->ldq_out || b.T == 1)) &&
          rows_meet(rows->q, 2LL * rows->ldq, 2LL * m->Nq, rows->q_out, 2LL * rows->ldq_out, 2LL * m->Nq, b.T))
        return fail(SWIFTKV_EINVAL, "q_out overlaps q without being it");
      for (int i = 0; i < caches; ++i) {  // other warps read them while these are written
        const bf16 *ki = static_cast<const bf16*>(rows->k) + i * rows->k_step, *vi = static_cast<const bf16*>(rows->v) + i * rows->v_step;
        if (rows_meet(rows->q_out, 2LL * rows->ldq_out, 2LL * m->Nq, ki, 2LL * rows->ldk, 2 * Nkv, b.T) ||
            rows_meet(rows->q_out, 2LL * rows->ldq_out, 2LL * m->Nq, vi, 2LL * rows->ldv, 2 * Nkv, b.T))
          return fail(SWIFTKV_EINVAL, "q_out overlaps k or v");
      }
    }
    OnDevice on_device(m);
    cudaStream_t s = (cudaStream_t)stream;
    AppendArgs a;
    // lists and pool addresses: in the kernel's parameters where they fit, straight from here
    const int planes = b.kind != kKvBf16 ? 4 : 2;
    a.o_cu = 0;
    a.o_ctx = P + 1;
    a.o_off = pos_off ? 2 * P + 1 : -1;
    a.o_pools = ((pos_off ? 3 : 2) * P + 2) & ~1;
    const size_t total = (size_t)a.o_pools + 2 * (size_t)planes * caches;
    InlineInts inl;
    std::vector<int> many(total > kInlineInts ? total : 0);
    int* to = many.empty() ? inl.v : many.data();
    memcpy(to, cu, (size_t)(P + 1) * 4);
    if (ctx) memcpy(to + a.o_ctx, ctx, (size_t)P * 4);
    else memset(to + a.o_ctx, 0, (size_t)P * 4);
    if (pos_off) memcpy(to + a.o_off, pos_off, (size_t)P * 4);
    void* const* const pools[4] = {kv->k_pool, kv->v_pool, kv->k_scale, kv->v_scale};
    for (int i = 0; i < planes; ++i)
      memcpy(to + a.o_pools + 2 * (size_t)i * caches, pools[i] + cache, (size_t)caches * sizeof(void*));
    int* dev = nullptr;
    if (!many.empty()) {
      Arena arena;
      RET(reserve(m, total * 4, s, &arena));
      dev = arena.take<int>(total);
      CK(upload_ints(dev, to, (int)total, s));
    }
    a.lists = dev;
    a.pools = nullptr;
    a.pool_step = caches;
    a.q = static_cast<const bf16*>(rows->q);
    a.ldq = rows->ldq;
    a.q_out = static_cast<bf16*>(rows->q_out);
    a.ldq_out = rows->ldq_out;
    a.k = static_cast<const bf16*>(rows->k);
    a.v = static_cast<const bf16*>(rows->v);
    a.ldk = rows->ldk;
    a.ldv = rows->ldv;
    a.k_step = rows->k_step;
    a.v_step = rows->v_step;
    a.caches = caches;
    a.P = P;
    a.T = b.T;
    a.bt = kv->block_table;
    a.max_pages = kv->max_pages_per_seq;
    a.num_pages = kv->num_pages;
    a.rotate = rotate != 0;
    const cudaError_t e = launch_append_on(m, a, b.kind, inl, s);
    if (e != cudaSuccess)
      return fail(e == cudaErrorNotSupported ? SWIFTKV_EUNSUPPORTED : SWIFTKV_ECUDA, "append: %s", cudaGetErrorString(e));
    return SWIFTKV_OK;
  });
}

int swiftkv_attention_weights(swiftkv_model* m, int cache, const void* q, int ldq, const float* lse, const int32_t* cu,
                              const int32_t* ctx, int P, const swiftkv_kv_pages* kv, int window, int sinks, float decay,
                              float* scores, swiftkv_stream stream) {
  return guarded([&]() -> int {
    RET(check_call(m, cache, P, kv));
    if (P == 0) return SWIFTKV_OK;
    if (!cu) return fail(SWIFTKV_EINVAL, "null cu_seqlens");
    if (!(std::fabs(decay) <= 3.0e38f)) return fail(SWIFTKV_EINVAL, "decay is not finite");
    RET(check_no_blocks(kv, "attention weights"));
    WeightsPlan p;
    RET(p.make(m, cu, ctx, P, kv, window, sinks));
    if (p.b.T == 0) return SWIFTKV_OK;
    RET(check_rows(m, q, ldq, "q"));
    if (!lse || !scores) return fail(SWIFTKV_EINVAL, "null lse / scores");
    if ((reinterpret_cast<uintptr_t>(lse) & 3) || (reinterpret_cast<uintptr_t>(scores) & 15))
      return fail(SWIFTKV_EINVAL, "misaligned lse (4 bytes) or scores (16 bytes)");
    OnDevice on_device(m);
    cudaStream_t s = (cudaStream_t)stream;
    Arena size, arena;
    p.place(m, &size);
    RET(reserve(m, size.used, s, &arena));
    p.place(m, &arena);
    RET(p.upload(s));
    return p.run(m, kv, cache, static_cast<const bf16*>(q), ldq, lse, p.b.T, decay, scores, s);
  });
}

int swiftkv_evict(swiftkv_model* m, int cache, const swiftkv_kv_pages* kv, float* const* scores,
                  const int32_t* seq_lens, int P, int keep, int sinks, int recent, const int32_t* dst_block_table,
                  int dst_max_pages, int32_t* kept, swiftkv_stream stream) {
  return guarded([&]() -> int {
    RET(check_call(m, cache < 0 ? 0 : cache, P, kv));
    if (P == 0) return SWIFTKV_OK;
    if (cache < -1) return fail(SWIFTKV_EINVAL, "cache %d outside [-1, %d)", cache, m->C);
    RET(check_no_blocks(kv, "eviction"));
    if (!scores || !seq_lens || !kept) return fail(SWIFTKV_EINVAL, "null scores / seq_lens / kept");
    if ((reinterpret_cast<uintptr_t>(kept) | reinterpret_cast<uintptr_t>(dst_block_table)) & 3)
      return fail(SWIFTKV_EINVAL, "misaligned kept or destination block table");
    const int first = cache < 0 ? 0 : cache, C = cache < 0 ? m->C : 1;
    for (int c = first; c < first + C; ++c)
      if (!scores[c] || (reinterpret_cast<uintptr_t>(scores[c]) & 15))
        return fail(SWIFTKV_EINVAL, "null or misaligned score pool for cache %d", c);
    if (keep < 1 || sinks < 0 || recent < 0 || (long long)sinks + recent > keep)
      return fail(SWIFTKV_EINVAL, "need keep >= 1, sinks >= 0, recent >= 0 and sinks + recent <= keep");
    if (keep > kMaxKeys) return fail(SWIFTKV_EUNSUPPORTED, "keep above 2^30");
    const int dst_width = dst_block_table ? dst_max_pages : kv->max_pages_per_seq;
    if (dst_block_table && dst_max_pages < 1) return fail(SWIFTKV_EINVAL, "empty destination block table");
    int longest = 0;
    for (int i = 0; i < P; ++i) {
      const long long n = seq_lens[i];
      if (n < 0) return fail(SWIFTKV_EINVAL_SEQLENS, "seq_lens[%d] < 0", i);
      if (n > kMaxKeys) return fail(SWIFTKV_EUNSUPPORTED, "seq_lens[%d] above 2^30", i);
      if (n > (long long)kv->max_pages_per_seq * kPageSize)
        return fail(SWIFTKV_ENO_PAGES, "sequence %d needs %lld pages, block table holds %d", i, (n + 15) / 16,
                    kv->max_pages_per_seq);
      const long long left = std::min<long long>(n, keep);
      if (left > (long long)dst_width * kPageSize)
        return fail(SWIFTKV_ENO_PAGES, "sequence %d keeps %lld pages, destination block table holds %d", i,
                    (left + 15) / 16, dst_width);
      longest = std::max(longest, (int)n);
    }
    OnDevice on_device(m);
    cudaStream_t s = (cudaStream_t)stream;
    // lengths and the caches' pool pointers in one list
    const bool fp8 = kv->kv_dtype == 1;
    std::vector<int> ints(seq_lens, seq_lens + P);
    if (ints.size() % 2) ints.push_back(0);
    const size_t at = ints.size();
    std::vector<const void*> ptrs;
    for (int c = 0; c < m->C; ++c) ptrs.push_back(kv->k_pool[c]);
    for (int c = 0; c < m->C; ++c) ptrs.push_back(kv->v_pool[c]);
    for (int c = 0; c < m->C; ++c) ptrs.push_back(c >= first && c < first + C ? scores[c] : nullptr);
    for (int c = 0; fp8 && c < m->C; ++c) ptrs.push_back(kv->k_scale[c]);
    for (int c = 0; fp8 && c < m->C; ++c) ptrs.push_back(kv->v_scale[c]);
    ints.resize(at + 2 * ptrs.size());
    memcpy(ints.data() + at, ptrs.data(), ptrs.size() * 8);
    int* dev = nullptr;
    if (ints.size() > kInlineInts) {
      Arena arena;
      RET(reserve(m, ints.size() * 4, s, &arena));
      dev = arena.take<int>(ints.size());
      CK(upload_ints(dev, ints.data(), (int)ints.size(), s));
    }
    EvictArgs a;
    a.lists = dev;
    a.o_ptrs = (int)at;
    a.num_ptrs = m->C;
    a.fp8 = fp8;
    a.P = P;
    a.first_cache = first;
    a.num_caches = C;
    a.n_kv = m->cfg.n_kv;
    a.row_bytes = m->cfg.d_head * (fp8 ? 1 : 2);
    a.src_bt = kv->block_table;
    a.src_pages = kv->max_pages_per_seq;
    a.dst_bt = dst_block_table ? dst_block_table : kv->block_table;
    a.dst_pages = dst_width;
    a.num_pages = kv->num_pages;
    a.keep = keep;
    a.sinks = sinks;
    a.recent = recent;
    a.kept = kept;
    a.status = m->status;
    a.in_place = !dst_block_table;
    const cudaError_t e = launch_evict(a, inline_of(ints, dev), longest, s);
    if (e != cudaSuccess)
      return fail(e == cudaErrorNotSupported ? SWIFTKV_EUNSUPPORTED : SWIFTKV_ECUDA, "evict: %s", cudaGetErrorString(e));
    return SWIFTKV_OK;
  });
}

}  // extern "C"
