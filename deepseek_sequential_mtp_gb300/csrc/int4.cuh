// Internal interface of the 4-bit weight GEMM (int4.cu) used by the draft
// step's linear maps.
#pragma once

#include "common.cuh"

namespace mtp {

// One weight matrix of a grouped call: codes q [n, K/2] (two per byte, the
// lower k in the low half), scale [n, ceil(K/group)] bf16, zero the same shape
// of bytes or null (8); out: fp32 [R, ldo] whose columns [0, n) receive the product.
struct Int4Seg {
  const uint8_t* q = nullptr;
  const __nv_bfloat16* scale = nullptr;
  const uint8_t* zero = nullptr;
  int n = 0;
  float* out = nullptr;
};

// out_s[r, :] = (accumulate ? out_s[r, :] : 0) + x[r, :] · w_s^T for 1..3
// segments sharing x [R, K] bf16 (row stride K).  R in [1, 32], K % 32 == 0,
// group in {32, 64, 128}, x and q_s 16-byte aligned, scale_s 2-byte, ldo >= n.
mtp_status int4w_gemm_launch(const Int4Seg* segs, int nseg, int K, int group, const __nv_bfloat16* x, int R, int ldo,
                             bool accumulate, cudaStream_t stream);

}  // namespace mtp
