// query_attn.cuh -- what the kernels of kvq_attention share: the rows of a sequence and the
// keys that each of them sees.
#pragma once

#include "attn_tile.cuh"

namespace kvq {

namespace {

constexpr float kNoKey = -1e30f;  // the softmax reference before the first key

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

// Logits of a tile's scores: sc[nh][e] belongs to row 8 nh + 2c + (e & 1) and token t +
// 8 (e >> 1).  Without a cap and a bias the scores stay as they are (qmul then carries the
// row's factor and log2 e); with one of them they become base-2 logits (qmul is 1).  The
// mask is skipped on tiles that every row of the warp sees whole.
template <int kNH>
struct QueryMod {
  static constexpr bool kActive = true;
  float fac[kNH][2], slope[kNH][2];
  int lo[kNH][2], hi[kNH][2], pos[kNH][2];
  int lo_all, hi_all;  // keys that every row sees
  float cap, icap;
  bool biased, linear;
  int t, t0;  // token of e = 0, 1; first token of the tile

  // The values of this lane's rows, and qmul.  Row r of the CTA has its lo and hi in lane r
  // and its factor in row_fac[r / 8] of the four lanes with g = r % 8.
  __device__ __forceinline__ void init(const QueryAttnParams& qp, int lane, int h, int row0, int rows, int first_pos,
                                       int lane_lo, int lane_hi, const float (&row_fac)[kNH], float (&qmul)[kNH][2]) {
    const int c = lane & 3;
    cap = qp.softcap;
    icap = cap > 0.0f ? 1.0f / cap : 0.0f;
    biased = qp.slopes != nullptr;
    linear = !biased && !(cap > 0.0f);
    const bool live = lane < 8 * kNH && row0 + lane < rows;
    lo_all = __reduce_max_sync(0xFFFFFFFFu, live ? lane_lo : 0);  // INT_MAX with a row that sees nothing
    hi_all = __reduce_min_sync(0xFFFFFFFFu, live ? lane_hi : 0x7FFFFFFF);
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nh + 2 * c + e;
        fac[nh][e] = __shfl_sync(0xFFFFFFFFu, row_fac[nh], 4 * (2 * c + e));
        qmul[nh][e] = linear ? fac[nh][e] * kLog2e : 1.0f;
        lo[nh][e] = __shfl_sync(0xFFFFFFFFu, lane_lo, r);
        hi[nh][e] = __shfl_sync(0xFFFFFFFFu, lane_hi, r);
        const int row = min(row0 + r, rows - 1), i = row / qp.a.group;
        pos[nh][e] = first_pos + i;
        slope[nh][e] = biased ? LDX(qp.slopes + h * qp.a.group + row - i * qp.a.group) : 0.0f;
      }
  }
  __device__ __forceinline__ void operator()(float (&sc)[kNH][4]) const {
    if (!linear) {
#pragma unroll
      for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = sc[nh][e] * fac[nh][e & 1];
          // tanh(x) = 1 - 2 / (1 + e^2x): an absolute error of a few 2^-23, which is what a
          // capped logit needs (tanh.approx is off by 2^-11 of the cap)
          if (cap > 0.0f) x = cap * __fmaf_rn(-2.0f, rcp_ftz(1.0f + ex2_ftz(2.0f * kLog2e * icap * x)), 1.0f);
          if (biased) x = __fmaf_rn(slope[nh][e & 1], static_cast<float>(t + 8 * (e >> 1) - pos[nh][e & 1]), x);
          sc[nh][e] = x * kLog2e;
        }
    }
    if (t0 < lo_all || t0 + 16 > hi_all) {  // uniform
#pragma unroll
      for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tt = t + 8 * (e >> 1);
          if (tt < lo[nh][e & 1] || tt >= hi[nh][e & 1]) sc[nh][e] = kNegInf;
        }
    }
  }
};

// Range of lane r's row of a CTA's rows (lo = INT_MAX: none), for r < n.
__device__ __forceinline__ void lane_range(const QueryAttnParams& qp, int lane, int n, int s, int q0, int nq, int len,
                                           int row0, int rows, int& lo, int& hi) {
  lo = 0x7FFFFFFF;
  hi = 0;
  if (lane < n && row0 + lane < rows) {
    const int i = (row0 + lane) / qp.a.group;
    int l, u;
    key_range(qp, s, q0 + i, len - nq + i, len, l, u);
    if (l < u) {
      lo = l;
      hi = u;
    }
  }
}

// This lane's Q^T fragments of one n-tile (`row` = its row g), scaled by a power of two into
// f16; returns the row's factor.
template <int D>
__device__ __forceinline__ float query_fragments(const AttnParams& p, int lane, int h, int q0, int row, int rows,
                                                 uint2 (&frag)[D / 16]) {
  const int c = lane & 3;
  uint32_t w[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) w[i] = 0u;
  if (row < rows) {
    const int i = row / p.group;
    const uint16_t* q = p.q + static_cast<int64_t>(q0 + i) * p.q_row_pitch +
                        static_cast<int64_t>(h * p.group + row - i * p.group) * p.q_head_pitch + c * (D / 4);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      uint32_t v4[4];
      load16B(q + 8 * j, v4);
      w[4 * j] = v4[0];
      w[4 * j + 1] = v4[1];
      w[4 * j + 2] = v4[2];
      w[4 * j + 3] = v4[3];
    }
  }
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) am = fmaxf(am, fmaxf(fabsf(bf16lo(w[i])), fabsf(bf16hi(w[i]))));
  am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
  am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
  int k = 0;
  if (am > 0.0f) k = 14 - (static_cast<int>((__float_as_uint(am) >> 23) & 0xFF) - 127);
  k = max(-100, min(120, k));
  const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
#pragma unroll
  for (int kb = 0; kb < D / 16; ++kb)
    frag[kb] = make_uint2(f32x2_to_f16x2(bf16lo(w[2 * kb]) * up, bf16hi(w[2 * kb]) * up),
                          f32x2_to_f16x2(bf16lo(w[2 * kb + 1]) * up, bf16hi(w[2 * kb + 1]) * up));
  return p.scale * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
}

}  // namespace

}  // namespace kvq
