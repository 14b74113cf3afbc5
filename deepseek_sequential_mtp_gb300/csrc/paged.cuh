// Internal interface of the paged key/value cache (paged.cu, paged_attn.cu).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace mtp {

// The checks of a cache that every entry point makes.
mtp_status paged_cache_check(const mtp_paged_cache* c, bool pointers);

// One attention over a paged cache: q [R, L, H] rows of head_dim, strides in elements.
struct PagedAttn {
  mtp_paged_cache c{};
  int R = 0, L = 1, H = 0;
  bool causal = true;
  float scale = 0.f;
  const __nv_bfloat16* q = nullptr;
  long long q_r = 0, q_l = 0, q_h = 0;
  const int32_t* ctx_len = nullptr;
  const int32_t* n_new = nullptr;  // null: L
  // results: o [R, L, H, hd] bf16 and lse [R, L, H] (nullable), or one record
  // (maximum, sum, unnormalised o[hd]) per (request, token, head), rec_stride floats apart
  __nv_bfloat16* o = nullptr;
  float* lse = nullptr;
  float* rec = nullptr;
  long long rec_stride = 0;
};

// The rows that a request holds as dense bf16 rows [R, T, Hkv, hd], those behind them left as they are but for, if causal,
// L - n_new[r] rows of zeros; ctx_out[r] = ctx_len[r] and those (n_new null: L).  Nothing of a request with n_new[r] = 0:
// ctx_out[r] = 0, its pages are not looked up.
mtp_status kv_dense_launch(const mtp_paged_cache& c, int R, int L, long long T, const int32_t* ctx_len, const int32_t* n_new,
                           bool causal, void* k_out, void* v_out, int32_t* ctx_out, cudaStream_t st);

bool paged_attn_sizes_ok(int R, int L, int H, const mtp_paged_cache& c);
size_t paged_attn_workspace_bytes(int R, int L, int H, const mtp_paged_cache& c);
mtp_status paged_attn_launch(const PagedAttn& p, void* ws, size_t ws_bytes, cudaStream_t stream);

}  // namespace mtp
