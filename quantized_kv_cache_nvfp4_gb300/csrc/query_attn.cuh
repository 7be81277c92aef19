// query_attn.cuh -- what the kernels of kvq_attention share: the rows of a sequence and the
// keys that each of them sees.
#pragma once

#include "attn_tile.cuh"

namespace kvq {

namespace {

// Range of keys that query token `tok` at position pos sees.
__device__ __forceinline__ void key_range(const QueryAttnParams& p, int s, int tok, int pos, int len, int& lo, int& hi) {
  lo = 0;
  hi = pos + 1;
  if (p.prefix != nullptr) hi = max(hi, min(LDX(p.prefix + s), len));
  if (p.window > 0) lo = max(lo, pos + 1 - p.window);
  if (p.key_starts != nullptr) lo = max(lo, LDX(p.key_starts + tok));
}

// First query token and number of query tokens of sequence s; false where they do not fit
// the arrays or the sequence.  Without starts (decode) token s is sequence s's only one.
__device__ __forceinline__ bool query_range(const QueryAttnParams& p, int s, int& q0, int& n, int& len) {
  len = LDX(p.a.seq_lens + s);
  n = 0;
  if (p.starts == nullptr) {
    q0 = s;
    if (len < 0 || len > p.a.seq_cap) return false;
    n = 1;
    return true;
  }
  q0 = LDX(p.starts + s);
  const int q1 = LDX(p.starts + s + 1);
  if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || q1 - q0 > p.max_q || len < 0 || len > p.a.seq_cap || q1 - q0 > len)
    return false;
  n = q1 - q0;
  return true;
}

// Whether the keys [lo, hi) of sequence s need a block entry outside the pool, for a whole warp
// (32 entries at a time: pages may be single tokens).  Only rows of a block that met such an entry
// ask.
__device__ __forceinline__ bool needs_bad_block(const AttnParams& p, int s, int lo, int hi) {
  if (lo >= hi) return false;
  const int32_t* const table = p.block_table + static_cast<int64_t>(s) * p.max_blocks;
  const uint32_t last = p.div_bs.div(static_cast<uint32_t>(hi) - 1), lane = threadIdx.x & 31;
#pragma unroll 1
  for (uint32_t b = p.div_bs.div(static_cast<uint32_t>(lo)); b <= last; b += 32) {
    const int32_t blk = b + lane <= last ? LDX(table + b + lane) : 0;
    if (__any_sync(0xFFFFFFFFu, b + lane <= last && (blk < 0 || blk >= p.num_blocks))) return true;
  }
  return false;
}

// Logits of a tile's scores: sc[nh][e] belongs to row 8 nh + 2c + (e & 1) and token t0 + g +
// 8 (e >> 1).  Without a cap and a bias the scores stay as they are (qmul then carries the
// row's factor and log2 e); with one of them they become base-2 logits (qmul is 1).  The
// mask is skipped on tiles that every row of the block sees whole; what it and the bias need
// stays in shared memory, since registers are what these kernels run out of.
template <int kNH>
struct QueryMod {
  static constexpr bool kActive = true;
  // Shared: the rows' key ranges, and for each row of the warp's head {slope log2 e, position};
  // positions count from the block's first row's, so that near keys' distances are exact at any
  // position (those of keys farther than 2^24 are rounded).
  struct Tables {
    int2 range[8 * kNH];
    float2 bias[16][8 * kNH];
  };
  const Tables* tab;
  int hw;               // the head's place in tab->bias
  float f[kNH][2];      // the row's factor: times 2 log2 e / cap, else times log2 e
  int lo_all, hi_all;   // keys that every row sees
  bool mixed;           // and whether some see others too
  float c2;             // cap log2 e, 0: no cap
  bool biased;
  int base;             // position of the block's first row
  int t0, g;            // first token of the tile; this lane's tokens are t0 + g and + 8

  // Fills the tables (a barrier follows): the block's ranges (row r's in lane r) by one warp,
  // the head's biases by one warp of each head.
  static __device__ __forceinline__ void fill(Tables* tab, const QueryAttnParams& qp, int lane, int h, int hw, int row0,
                                              int rows, int lo, int hi, bool ranges, bool biases) {
    if (lane >= 8 * kNH) return;
    if (ranges) tab->range[lane] = make_int2(lo, hi);
    if (biases && qp.slopes != nullptr) {
      const int row = min(row0 + lane, rows - 1), i = row / qp.a.group;
      tab->bias[hw][lane] = make_float2(LDX(qp.slopes + h * qp.a.group + row - i * qp.a.group) * kLog2e,
                                        static_cast<float>(i - row0 / qp.a.group));
    }
  }
  // row_fac[nh]: the factor of row 8 nh + g; lo, hi: the range of row `lane`.
  __device__ __forceinline__ void init(const Tables* t, const QueryAttnParams& qp, int lane, int head_place, int row0, int rows,
                                       int first_pos, int lo, int hi, const float (&row_fac)[kNH], float (&qmul)[kNH][2]) {
    const int c = lane & 3;
    tab = t;
    hw = head_place;
    base = first_pos + row0 / qp.a.group;
    g = lane >> 2;
    c2 = qp.softcap * kLog2e;
    biased = qp.slopes != nullptr;
    const bool linear = !biased && !(c2 > 0.0f);
    const float unit = c2 > 0.0f ? 2.0f * kLog2e / qp.softcap : kLog2e;
    const bool live = lane < 8 * kNH && row0 + lane < rows;
    lo_all = __reduce_max_sync(0xFFFFFFFFu, live ? lo : 0);  // INT_MAX with a row that sees nothing
    hi_all = __reduce_min_sync(0xFFFFFFFFu, live ? hi : 0x7FFFFFFF);
    mixed = __any_sync(0xFFFFFFFFu, live && (lo != lo_all || hi != hi_all));
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f[nh][e] = __shfl_sync(0xFFFFFFFFu, row_fac[nh], 4 * (2 * c + e)) * unit;
        qmul[nh][e] = linear ? f[nh][e] : 1.0f;
      }
  }
  __device__ __forceinline__ void operator()(float (&sc)[kNH][4]) const {
    const int c = threadIdx.x & 3;
    if (c2 > 0.0f) {
      // c2 tanh(x) = c2 - 2 c2 / (1 + e^2x): an absolute error of a few 2^-23 of the cap, which
      // is what a capped logit needs (tanh.approx is off by 2^-11 of it)
#pragma unroll
      for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sc[nh][e] = __fmaf_rn(-2.0f * c2, rcp_ftz(1.0f + ex2_ftz(sc[nh][e] * f[nh][e & 1])), c2);
    } else if (biased) {
#pragma unroll
      for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nh][e] *= f[nh][e & 1];
    }
    if (biased) {
      const float t[2] = {static_cast<float>(t0 - base + g), static_cast<float>(t0 - base + g + 8)};
#pragma unroll
      for (int nh = 0; nh < kNH; ++nh) {
        const float4 b = *reinterpret_cast<const float4*>(&tab->bias[hw][8 * nh + 2 * c]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sc[nh][e] = __fmaf_rn(e & 1 ? b.z : b.x, t[e >> 1] - (e & 1 ? b.w : b.y), sc[nh][e]);
      }
    }
    if (t0 < lo_all || t0 + 16 > hi_all) {  // uniform
#pragma unroll
      for (int nh = 0; nh < kNH; ++nh) {
        const int4 q = *reinterpret_cast<const int4*>(&tab->range[8 * nh + 2 * c]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tt = t0 + g + 8 * (e >> 1);
          if (tt < (e & 1 ? q.z : q.x) || tt >= (e & 1 ? q.w : q.y)) sc[nh][e] = kNegInf;
        }
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
  k = max(-113, min(120, k));
  const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
#pragma unroll
  for (int kb = 0; kb < D / 16; ++kb)
    frag[kb] = make_uint2(f32x2_to_f16x2(bf16lo(w[2 * kb]) * up, bf16hi(w[2 * kb]) * up),
                          f32x2_to_f16x2(bf16lo(w[2 * kb + 1]) * up, bf16hi(w[2 * kb + 1]) * up));
  return p.scale * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
}

}  // namespace

}  // namespace kvq
