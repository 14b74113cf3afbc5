// Internal interface of the shared-prefix attention (prefix_attn.cu).
#pragma once

#include "common.cuh"

namespace mtp {

// One call: q [R, L, H] rows of head_dim, a prefix [P, Hkv] shared by all
// requests and a cache [R, T, Hkv] of each request's own; strides in elements.
struct PrefixAttn {
  int R = 0, L = 1, H = 0, Hkv = 0, hd = 0, P = 0, T = 0;
  bool causal = true;
  float scale = 0.f;
  const __nv_bfloat16* q = nullptr;
  long long q_r = 0, q_l = 0, q_h = 0;
  const __nv_bfloat16 *pk = nullptr, *pv = nullptr;
  long long p_t = 0, p_h = 0;
  const __nv_bfloat16 *kk = nullptr, *kv = nullptr;
  long long k_r = 0, k_t = 0, k_h = 0;
  const int32_t* ctx_len = nullptr;  // null: T
  // results: o [R, L, H, hd] bf16 and lse [R, L, H] (nullable), or one record
  // (maximum, sum, unnormalised o[hd]) per (request, token, head), rec_stride floats apart
  __nv_bfloat16* o = nullptr;
  float* lse = nullptr;
  float* rec = nullptr;
  long long rec_stride = 0;
};

bool prefix_attn_sizes_ok(int R, int L, int H, int Hkv, int hd, int P, int T);
size_t prefix_attn_workspace_bytes(int R, int L, int H, int Hkv, int hd, int P, int T);
mtp_status prefix_attn_launch(const PrefixAttn& p, void* ws, size_t ws_bytes, cudaStream_t stream);

}  // namespace mtp
