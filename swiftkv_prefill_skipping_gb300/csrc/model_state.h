// The model handle and error helpers shared by the C-ABI implementation files.
#pragma once

#include <cuda_runtime.h>

#include <new>
#include <string>
#include <vector>

#include "launch.h"
#include "swiftkv.h"

namespace skv {

// Records the message as the calling thread's swiftkv_last_error() and returns `code`.
int fail(int code, const char* fmt, ...);

#define CK(call)                                                                              \
  do {                                                                                        \
    cudaError_t e_ = (call);                                                                  \
    if (e_ != cudaSuccess) return skv::fail(SWIFTKV_ECUDA, "%s: %s", #call, cudaGetErrorString(e_)); \
  } while (0)

#define RET(x)                 \
  do {                         \
    int r_ = (x);              \
    if (r_ != SWIFTKV_OK) return r_; \
  } while (0)


struct LayerW {
  float* g_attn = nullptr;
  float* g_mlp = nullptr;
  bf16* wqkv = nullptr;  // full layer: [Nq + 2 Nkv][d]; skipped layer: W_Q only [Nq][d]
  float* bqkv = nullptr;
  bf16* wo = nullptr;    // [d][Nq]
  bf16* wgu = nullptr;   // [2 Fp][d], gate/up interleaved in 64-row blocks
  bf16* wd = nullptr;    // [d][Fp]
  bool loaded = false;
};

}  // namespace skv

struct swiftkv_model {
  swiftkv_model_config cfg;
  int l, g, C, G;
  int Nq, Nkv, Fp, Nwide;
  int device, num_sms;
  std::vector<skv::LayerW> layers;
  skv::bf16 *embed = nullptr, *lm_head = nullptr;
  float* g_final = nullptr;
  skv::bf16* w_wide = nullptr;
  float* b_wide = nullptr;
  float2* rope_tab = nullptr;
  unsigned long long* rope_turn = nullptr;
  int* status = nullptr;
  std::vector<void*> allocs;
  size_t weight_bytes = 0;
  char* ws = nullptr;
  size_t ws_bytes = 0;
  char* ops_ws = nullptr;  // workspace of the operators of serving.h
  size_t ops_bytes = 0;
  bool ops_captured = false;   // a captured graph uses ops_ws: when outgrown it stays, in `allocs`
  size_t ops_kept_bytes = 0;   // of the blocks that stayed so
  bool globals_loaded = false;
  int gemm_impl = 0;  // 0 tcgen05 CTA pairs, 1 mma.sync tiles, 2 tcgen05 single CTA (GEMMs with > 64 rows)
  int attn_impl = 0;  // 0 tcgen05 when d_head == 128, 1 mma.sync
  bool norm_fusion = false;  // prompt rows: RMSNorm in the tcgen05 GEMM epilogues (else its own pass)
  int rows_impl = 1;  // tail / decode rows after attention: 0 one chained launch, 1 a launch per GEMM / norm
  unsigned* chain_count = nullptr;  // grid-barrier arrivals of the chained launches (device)
  unsigned chain_base = 0;          // ... and their count so far (host)
  int window = 0, sinks = 0;          // attention window of the model's layers (0: none)
  std::vector<float*> score_pools;    // per cache, where the layers' attention weights are added (empty: off)
  int score_pages = 0;                // pages of each
  float score_decay = 1.f;
  // profiling (swiftkv_profile_begin/end)
  bool prof_on = false;
  struct Rec {
    std::string name;
    cudaEvent_t a, b;
    int kernels;
    double flops, bytes;
  };
  std::vector<Rec> recs;
  std::vector<cudaEvent_t> ev_pool;
  size_t ev_used = 0;
};

namespace skv {

constexpr int kRopeLen = 32768;  // positions of rope_tab

// f() for a C entry: host lists that do not fit the memory become an error code.
template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(SWIFTKV_EOOM, "host memory");
  } catch (const std::exception& e) {  // std::length_error
    return fail(SWIFTKV_EUNSUPPORTED, "%s", e.what());
  }
}

// The caches a call names: counts, page size and pointers against the model's.
int check_kv(const swiftkv_model* m, const swiftkv_kv_pages* kv);

// Makes the model's device current for a scope and the caller's again after it.
struct OnDevice {
  int was = -1;
  explicit OnDevice(const swiftkv_model* m) {
    int now = -1;
    if (cudaGetDevice(&now) == cudaSuccess && now != m->device && cudaSetDevice(m->device) == cudaSuccess) was = now;
  }
  ~OnDevice() {
    if (was >= 0) cudaSetDevice(was);
  }
  OnDevice(const OnDevice&) = delete;
  OnDevice& operator=(const OnDevice&) = delete;
};

}  // namespace skv
