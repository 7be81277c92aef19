// query_attn.cuh -- what the kernels of kvq_attention share: the rows of a sequence and the
// keys that each of them sees.
#pragma once

#include "attn_tile.cuh"

namespace kvq {

namespace {

constexpr float kNoKey = -1e30f;  // the softmax reference before the first key

// tanh(x) = 1 - 2 / (1 + e^2x): an absolute error of a few 2^-23, which is what a capped
// logit needs (tanh.approx is off by 2^-11 of the cap).
__device__ __forceinline__ float tanh_abs(float x) {
  return __fmaf_rn(-2.0f, rcp_approx(1.0f + ex2(2.0f * kLog2e * x)), 1.0f);
}

// Range of keys that query token `tok` at position pos sees.
__device__ __forceinline__ void key_range(const QueryAttnParams& p, int s, int tok, int pos, int len, int& lo, int& hi) {
  lo = 0;
  hi = pos + 1;
  if (p.prefix != nullptr) hi = max(hi, min(LDX(p.prefix + s), len));
  if (p.window > 0) lo = max(lo, pos + 1 - p.window);
  if (p.key_starts != nullptr) lo = max(lo, LDX(p.key_starts + tok));
}

// First query token and number of query tokens of sequence s; false where they do not fit
// the arrays or the sequence.
__device__ __forceinline__ bool query_range(const QueryAttnParams& p, int s, int& q0, int& n, int& len) {
  q0 = LDX(p.starts + s);
  const int q1 = LDX(p.starts + s + 1);
  len = LDX(p.a.seq_lens + s);
  n = 0;
  if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || q1 - q0 > p.max_q || len < 0 || len > p.a.seq_cap || q1 - q0 > len)
    return false;
  n = q1 - q0;
  return true;
}

}  // namespace

}  // namespace kvq
