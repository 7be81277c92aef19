// attn_kernels.cu -- paged decode attention that reads the quantised pool directly.
//
// The step downstream of the paged restore: instead of restoring K and V to bf16,
// decode attention dequantises them in registers ("feat(kvcache): add nvfp4 kv
// quantization (FreeToken PR #408)", Summary -- the restore paths -- and fp8 store
// notes, where the row scale multiplies the score and the output; "vllm-rlt PR #166",
// review by 0z5a: dequantise to 16 bits in registers and keep the 16-bit MMA).
//
// One query token per sequence; query head qh reads KV head qh / group:
//   o[s][qh] = softmax_t(scale * q . k_t) . v_t   over tokens t < seq_lens[s].
//
// Mapping (mma.sync m16n8k16, f16 operands, f32 accumulators), token-major.  A CTA
// takes one (split of a sequence's tokens, KV head, sequence); its 4 warps take
// 16-token tiles in turn, each through its own cp.async ring of pool tiles in shared
// memory.
//  * M = the tile's 16 tokens, N = the group's query heads in n-tiles of 8 (one for
//    groups up to 8, two up to 16): a warp computes S^T = K Q^T, 16 tokens x 8 heads
//    per n-tile, with K as the A operand, so no MMA row is padding.
//  * S^T contracts over the head dimension in a permuted order: k-step kb of lane c
//    (c = lane % 4) covers dims c*D/4 + 4kb .. + 3, so a lane's K operand for one token
//    is one contiguous run of code bytes; Q^T is permuted the same way and stays in
//    registers when its fragments fit in 16 of them (D = 64, or D = 128 with one
//    n-tile), else it is read from shared memory per k-step.
//  * The probabilities leave the S^T accumulators in the C layout (a lane holds two
//    heads of tokens g and g + 8); an 8x8 transpose in registers (movmatrix) turns
//    them into the B operand of O^T = V^T P^T (two tokens of one head).
//  * O^T: m-tile mt, rows g and g + 8 = dims g*D/8 + 2mt and + 1, so a lane's V operand
//    for one token is again one contiguous run; the nibbles (or bytes) of the two
//    tokens a register pairs are interleaved by a mask-and-shift (or byte-permute)
//    transpose.
//  * K and V decode exactly to f16: e2m1 x e4m3 has at most 2 x 4 significant bits,
//    and e4m3 fits f16.  K's FP32 row scale multiplies the score; V's multiplies P
//    relative to a reference R of the tile row scales.  R and the softmax reference m
//    move only when a tile exceeds them by more than 2^6 and 2^8 (O is rescaled then),
//    so P' = exp2(s - m) * rs / R stays below 2^14 and f16 holds it.
//  * Q enters f16 exactly: each query row is scaled by a power of two that puts its
//    largest element in [2^14, 2^15), undone in the score multiplier.
//  * The warps of a CTA merge through shared memory; several splits of a sequence
//    merge through the caller's workspace in a second small kernel.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "attn_tile.cuh"

namespace kvq {

namespace {

template <int D, int kFK, int kFV, int kNH>
__global__ void __launch_bounds__(kAttnThreads) decode_attn_kernel(const AttnParams p) {
  using T = AttnTile<D, kFK, kFV>;
  constexpr int kKS = D / 16;  // k-steps of S^T = K Q^T
  constexpr int kMT = D / 16;  // m-tiles of O^T = V^T P^T
  constexpr bool kQReg = kNH * kKS <= 8;  // Q^T fragments kept in registers
  extern __shared__ __align__(16) unsigned char smem[];

  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int g = lane >> 2;
  const int c = lane & 3;
  const int split = blockIdx.x, h = blockIdx.y, s = blockIdx.z;

  const int len = LDX(p.seq_lens + s);
  const bool bad_len = len < 0 || len > p.seq_cap;
  const int t_begin = split * p.split_len;
  const int t_end = bad_len ? t_begin : t_begin + min(p.split_len, len - t_begin);
  const int ntile = t_end > t_begin ? (t_end - t_begin + 15) / 16 : 0;
  if (bad_len && threadIdx.x == 0 && split == 0 && h == 0) set_status(p.status, 8u);

  // ---- Q^T fragments (query head 8nh + g of the group, scaled by 2^k into f16) and
  // the per-head score factors, built once by warp 0 into shared memory ----
  uint2* const qfrag = reinterpret_cast<uint2*>(smem);                         // [nh][k-step][32 lanes]
  float* const qfac = reinterpret_cast<float*>(smem + kNH * kKS * 32 * 8);  // [8 kNH heads]
  if (warp == 0) {
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh) {
      const int row = 8 * nh + g;
      uint32_t w[D / 8];  // this lane's D/4 dims as bf16 pairs
#pragma unroll
      for (int i = 0; i < D / 8; ++i) w[i] = 0u;
      if (row < p.group) {
        const uint16_t* qp = p.q + static_cast<int64_t>(s) * p.q_row_pitch +
                             static_cast<int64_t>(h * p.group + row) * p.q_head_pitch + c * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t v4[4];
          load16B(qp + 8 * i, v4);
          w[4 * i] = v4[0];
          w[4 * i + 1] = v4[1];
          w[4 * i + 2] = v4[2];
          w[4 * i + 3] = v4[3];
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
      if (c == 0) qfac[row] = p.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
      for (int kb = 0; kb < kKS; ++kb)
        qfrag[(nh * kKS + kb) * 32 + lane] =
            make_uint2(f32x2_to_f16x2(bf16lo(w[2 * kb]) * up, bf16hi(w[2 * kb]) * up),            // dims 4kb, +1
                       f32x2_to_f16x2(bf16lo(w[2 * kb + 1]) * up, bf16hi(w[2 * kb + 1]) * up));  // dims 4kb+2, +3
    }
  }
  __syncthreads();
  float qmul[kNH][2];  // heads 8nh + 2c, + 1
#pragma unroll
  for (int nh = 0; nh < kNH; ++nh) {
    qmul[nh][0] = qfac[8 * nh + 2 * c];
    qmul[nh][1] = qfac[8 * nh + 2 * c + 1];
  }
  uint2 qreg[kQReg ? kNH : 1][kQReg ? kKS : 1];
  if constexpr (kQReg) {
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
      for (int kb = 0; kb < kKS; ++kb) qreg[nh][kb] = qfrag[(nh * kKS + kb) * 32 + lane];
  }
  auto qb = [&](int nh, int kb) -> uint2 {
    if constexpr (kQReg) {
      return qreg[nh][kb];
    } else {
      return qfrag[(nh * kKS + kb) * 32 + lane];
    }
  };

  // ---- the warp's tiles through its cp.async ring ----
  unsigned char* const ring = smem + T::kQ + warp * T::kStages * T::kBytes;
  bool bad = false;
  // pool row of token (lane & 15) of the warp's tile number `it` (-1 past the end); the
  // block-table load is issued a tile ahead of its copies, so its latency overlaps
  // the current tile's arithmetic.  srow: the scale this lane copies (lanes 0-15 K's,
  // 16-31 V's), the row's own or its page's
  const bool lane_page = lane < 16 ? p.k_page : p.v_page;
  auto row_of = [&](int it, int64_t& srow) -> int64_t {
    const int tile = warp + it * kAttnWarps;
    srow = 0;
    if (tile >= ntile) return -1;
    int t = t_begin + tile * 16 + (lane & 15);
    if (t >= t_end) t = t_end - 1;  // a valid token's address; masked later
    uint32_t bi, bo;
    p.div_bs.divmod(static_cast<uint32_t>(t), bi, bo);
    int64_t blk = LDX(p.block_table + static_cast<int64_t>(s) * p.max_blocks + bi);
    if (blk < 0 || blk >= p.num_blocks) {
      bad = true;
      blk = 0;
    }
    const int64_t row = (blk * p.block_size + bo) * p.H + h;
    srow = lane_page ? blk * p.H + h : row;
    return row;
  };
  // copies of a tile (rows from row_of, uniform -1 when there is none) into stage st:
  // the 32 lanes take consecutive 16-byte pieces of the 16 rows (whole sectors), then
  // lanes 0-15 the K block and row scales and lanes 16-31 the V ones
  auto issue = [&](int64_t row, int64_t srow, int st) {
    if (__shfl_sync(0xFFFFFFFFu, row, 0) < 0) return;
    unsigned char* const sb = ring + st * T::kBytes;
    const int tt = lane & 15;
    constexpr int kPK = T::kCK / 16, kPV = T::kCV / 16;
    if constexpr (kPK == kPV) {  // the same piece of K and V: one row exchange for both
#pragma unroll
      for (int i = lane; i < 16 * kPK; i += 32) {
        const int64_t rr = shfl64(row, i / kPK);
        cp_async16(sb + T::kOffKC + (i / kPK) * T::kSK + (i % kPK) * 16, p.k.codes + rr * T::kCK + (i % kPK) * 16);
        cp_async16(sb + T::kOffVC + (i / kPV) * T::kSV + (i % kPV) * 16, p.v.codes + rr * T::kCV + (i % kPV) * 16);
      }
    } else {
#pragma unroll
      for (int i = lane; i < 16 * kPK; i += 32) {
        const int64_t rr = shfl64(row, i / kPK);
        cp_async16(sb + T::kOffKC + (i / kPK) * T::kSK + (i % kPK) * 16, p.k.codes + rr * T::kCK + (i % kPK) * 16);
      }
#pragma unroll
      for (int i = lane; i < 16 * kPV; i += 32) {
        const int64_t rr = shfl64(row, i / kPV);
        cp_async16(sb + T::kOffVC + (i / kPV) * T::kSV + (i % kPV) * 16, p.v.codes + rr * T::kCV + (i % kPV) * 16);
      }
    }
    if (lane < 16) {
      if constexpr (T::kBK > 0) cp_async_n<T::kBK>(sb + T::kOffKB + tt * T::kBK, p.k.bscale + row * T::kBK);
      cp_async_small<4>(sb + T::kOffKR + tt * 4, p.k.rscale + srow);
    } else {
      if constexpr (T::kBV > 0) cp_async_n<T::kBV>(sb + T::kOffVB + tt * T::kBV, p.v.bscale + row * T::kBV);
      cp_async_small<4>(sb + T::kOffVR + tt * 4, p.v.rscale + srow);
    }
  };

  AttnState<D, kNH> st;
  st.init();

#pragma unroll
  for (int j = 0; j < T::kStages - 1; ++j) {
    int64_t srow;
    const int64_t row = row_of(j, srow);
    issue(row, srow, j);
    cp_async_commit();
  }
  const int my_tiles = ntile > warp ? (ntile - warp + kAttnWarps - 1) / kAttnWarps : 0;
  for (int it = 0; it < my_tiles; ++it) {
    int64_t srow_next;
    const int64_t row_next = row_of(it + T::kStages - 1, srow_next);  // the refill's rows, loaded early
    cp_async_wait<T::kStages - 2>();
    __syncwarp();
    const unsigned char* const sb = ring + (it % T::kStages) * T::kBytes;
    const int t0 = t_begin + (warp + it * kAttnWarps) * 16;

    const TileView tv{sb + T::kOffKC, sb + T::kOffVC, sb + T::kOffKB, sb + T::kOffVB, sb + T::kOffKR, sb + T::kOffVR,
                      T::kSK, T::kSV, T::kBK, T::kBV, 4, 4};
    attn_tile<D, kFK, kFV, kNH>(tv, qb, qmul, lane, t_end - t0, st, NoMod{});
    __syncwarp();  // every lane has read this stage before it is refilled
    issue(row_next, srow_next, (it + T::kStages - 1) % T::kStages);
    cp_async_commit();
  }
  cp_async_wait<0>();
  // the merge kernel (when the sequence is split) may be scheduled from here on; it
  // waits for this grid's writes before it reads them
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) set_status(p.status, 2u);
  // row sums over the 8 lanes (tokens) of each head
#pragma unroll
  for (int off = 4; off <= 16; off <<= 1)
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh) {
      st.l[nh][0] += __shfl_xor_sync(0xFFFFFFFFu, st.l[nh][0], off);
      st.l[nh][1] += __shfl_xor_sync(0xFFFFFFFFu, st.l[nh][1], off);
    }
  const bool cta_bad = __syncthreads_or(bad ? 1 : 0) != 0 || bad_len;  // the ring is free after this

  // per warp: O (true scale: O * R) by head and natural dim, and m, l per head
  constexpr int kHeads = 8 * kNH;
  float* const mo = reinterpret_cast<float*>(smem + T::kQ) + warp * kHeads * (D + 2);
#pragma unroll
  for (int q = 0; q < kMT; ++q)
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int head = 8 * nh + 2 * c + (e & 1);
        const int d = g * (D / 8) + 2 * q + (e >> 1);
        mo[head * (D + 2) + d] = st.o[q][nh][e] * st.R;
      }
  if (g == 0) {
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int head = 8 * nh + 2 * c + e;
        mo[head * (D + 2) + D] = st.m[nh][e];
        mo[head * (D + 2) + D + 1] = st.l[nh][e];
      }
  }
  __syncthreads();
  const float* const mall = reinterpret_cast<const float*>(smem + T::kQ);
  for (int idx = threadIdx.x; idx < p.group * D; idx += kAttnThreads) {
    const int row = idx / D, d = idx % D;
    float M = kNegInf;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) M = fmaxf(M, mall[(w * kHeads + row) * (D + 2) + D]);
    float L = 0.0f, O = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      const float mw = mall[(w * kHeads + row) * (D + 2) + D];
      const float f = mw == kNegInf ? 0.0f : ex2(mw - M);
      L += mall[(w * kHeads + row) * (D + 2) + D + 1] * f;
      O += mall[(w * kHeads + row) * (D + 2) + d] * f;
    }
    const int qh = h * p.group + row;
    if (p.nsplit == 1) {
      if (cta_bad) continue;  // a bad sequence leaves its output untouched
      const float y = L == 0.0f ? 0.0f : O / L;  // a NaN stays one
      STX(p.out + static_cast<int64_t>(s) * p.o_row_pitch + static_cast<int64_t>(qh) * p.o_head_pitch + d,
          static_cast<uint16_t>(pack_bf16x2(y, 0.0f) & 0xFFFFu));
    } else {
      float* const wsr = p.ws + ((static_cast<int64_t>(s) * p.Hq + qh) * p.nsplit + split) * (D + 2);
      STX(wsr + d, O);
      if (d == 0) {
        STX(wsr + D, cta_bad ? __int_as_float(0x7FC00000) : M);  // NaN marks a bad sequence (M never is one)
        STX(wsr + D + 1, L);
      }
    }
  }
}

// Merge of the splits of each (sequence, query head): o = sum_k O_k 2^(M_k - M) /
// sum_k L_k 2^(M_k - M), one warp per (sequence, query head).  Lane k holds split k's
// M and L (32 splits at a time), the warp reduces them, and each lane sums its D/32
// dims over the splits.  The O rows of the first kPre splits are loaded together with
// M and L, so a call with up to kPre splits waits for memory once.  A NaN M (bad
// sequence) leaves the output untouched; a NaN L is a NaN score's and reaches the output.
constexpr int kMergeWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) decode_attn_merge_kernel(const AttnParams p) {
  constexpr int kDL = D / 32 > 0 ? D / 32 : 1;  // dims per lane (D >= 64: 2, 4 or 8)
  constexpr int kPre = 64 / kDL;               // splits whose O is loaded up front
  // launched as a programmatic dependent of the attention kernel: wait for its results
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int sq = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);  // s * Hq + qh
  if (sq >= p.S * p.Hq) return;
  const int s = sq / p.Hq, qh = sq % p.Hq;
  const float* const base = p.ws + static_cast<int64_t>(sq) * p.nsplit * (D + 2);
  const int npre = min(p.nsplit, kPre);
  float2 pre[kPre][kDL / 2];
#pragma unroll
  for (int k = 0; k < kPre; ++k)
#pragma unroll
    for (int i = 0; i < kDL / 2; ++i)
      pre[k][i] = k < npre ? LDX(reinterpret_cast<const float2*>(base + k * (D + 2) + kDL * lane + 2 * i))
                           : make_float2(0.0f, 0.0f);  // (D + 2) * 4 bytes is a multiple of 8
  float M = kNegInf;
  bool bad = false;
  for (int k0 = 0; k0 < p.nsplit; k0 += 32) {
    const int k = k0 + lane;
    if (k < p.nsplit) {
      const float mk = LDX(base + k * (D + 2) + D);
      M = fmaxf(M, mk);
      bad = bad || isnan(mk);
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
  if (__any_sync(0xFFFFFFFFu, bad)) return;
  float L = 0.0f;
  float o[kDL];
#pragma unroll
  for (int i = 0; i < kDL; ++i) o[i] = 0.0f;
  for (int k0 = 0; k0 < p.nsplit; k0 += 32) {
    float f = 0.0f;
    const int kk = k0 + lane;
    if (kk < p.nsplit) {
      const float mk = LDX(base + kk * (D + 2) + D);
      f = mk == kNegInf ? 0.0f : ex2(mk - M);
      L += LDX(base + kk * (D + 2) + D + 1) * f;
    }
    if (k0 == 0) {
#pragma unroll
      for (int k = 0; k < kPre; ++k) {
        const float fk = __shfl_sync(0xFFFFFFFFu, f, k);  // 0 past the last split
#pragma unroll
        for (int i = 0; i < kDL / 2; ++i) {
          o[2 * i] += pre[k][i].x * fk;
          o[2 * i + 1] += pre[k][i].y * fk;
        }
      }
    }
    const int kfirst = k0 == 0 ? kPre : 0;
    const int nk = min(32, p.nsplit - k0);
#pragma unroll 4
    for (int k = kfirst; k < nk; ++k) {
      const float fk = __shfl_sync(0xFFFFFFFFu, f, k);
      const float* const ok = base + (k0 + k) * (D + 2) + kDL * lane;
#pragma unroll
      for (int i = 0; i < kDL; i += 2) {
        const float2 v = LDX(reinterpret_cast<const float2*>(ok + i));
        o[i] += v.x * fk;
        o[i + 1] += v.y * fk;
      }
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, off);
  uint16_t* const out = p.out + static_cast<int64_t>(s) * p.o_row_pitch + static_cast<int64_t>(qh) * p.o_head_pitch;
#pragma unroll
  for (int i = 0; i < kDL; i += 2) {
    const float y0 = L == 0.0f ? 0.0f : o[i] / L;
    const float y1 = L == 0.0f ? 0.0f : o[i + 1] / L;
    STX(reinterpret_cast<uint32_t*>(out + kDL * lane + i), pack_bf16x2(y0, y1));
  }
}

// ---------------------------------------------------------------------------------
// Page-major decode attention: one block per (token split, sequence) that covers every
// KV head.  16 consecutive tokens of a page (block_size a multiple of 16) hold, for all
// H heads, one contiguous range of each pool plane: H x 16 code rows, block-scale rows
// and row scales.  So a producer warp moves a stage of P = W / H such 16-token chunks
// with 6 P bulk copies (cp.async.bulk, completion on the stage's "full" mbarrier), and
// W consumer warps each take one (chunk, head) of every stage: warp w serves head w % H
// and chunk w / H, with the tile arithmetic of the head-major kernel above.  A consumer
// releases a stage on its "empty" mbarrier (W arrivals) before the producer refills it.
// Warps of one head (P > 1) merge through shared memory at the end; each head's result
// (or split partial) is written by its chunk-0 warp.
// ---------------------------------------------------------------------------------
// kPg: a plane may be page-scaled (p.k_page / p.v_page); its chunk's H scales are then
// one 4 H-byte copy (a multiple of 16, H >= 4) that all 16 tokens of the chunk read.
template <int D, int kFK, int kFV, int W, int H, bool kPg>
__global__ void __launch_bounds__((W + 1) * 32, W == 8 ? 2 : 1) decode_attn_page_kernel(const AttnParams p) {
  using T = PageStage<D, kFK, kFV, W>;
  constexpr int kKS = D / 16;
  constexpr int kMT = D / 16;
  static_assert(kKS <= 8, "Q^T fragments of one head n-tile in registers");
  extern __shared__ __align__(128) unsigned char page_smem[];
  unsigned char* const smem = page_smem;

  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int g = lane >> 2;
  const int c = lane & 3;
  const int split = blockIdx.x, s = blockIdx.z;
  constexpr int P = W / H;  // 16-token chunks per stage (the KV head count H is fixed per instance)

  const int len = LDX(p.seq_lens + s);
  const bool bad_len = len < 0 || len > p.seq_cap;
  const int t_begin = split * p.split_len;
  const int t_end = bad_len ? t_begin : t_begin + min(p.split_len, len - t_begin);
  const int nstage = t_end > t_begin ? (t_end - t_begin + 16 * P - 1) / (16 * P) : 0;
  if (bad_len && threadIdx.x == 0 && split == 0) set_status(p.status, 8u);

  const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const uint32_t full0 = ring_s + T::kOffBar;          // full[st] at full0 + 8 st
  const uint32_t empty0 = full0 + 8 * T::kStages;      // empty[st] at empty0 + 8 st
  int* const bad_flag = reinterpret_cast<int*>(smem + T::kOffBar + 16 * T::kStages);
  if (threadIdx.x == 0) {
#pragma unroll
    for (int st = 0; st < T::kStages; ++st) {
      mbar_init(full0 + 8 * st, 1);
      mbar_init(empty0 + 8 * st, W);
    }
    *bad_flag = 0;
    mbar_init_fence();
  }
  __syncthreads();

  if (warp == W) {
    // ---- producer: lane j < P resolves chunk j of each stage and issues its copies ----
    bool timed_out = false, bad = false;
    for (int k = 0; k < nstage; ++k) {
      const int st = k % T::kStages;
      const int t0 = t_begin + 16 * (P * k + lane);
      bool have = false;
      int64_t r0 = 0;  // pool row (slot, head 0) of the chunk's first token
      int64_t pg = 0;  // its page
      if (lane < P && t0 < t_end) {
        uint32_t bi, bo;
        p.div_bs.divmod(static_cast<uint32_t>(t0), bi, bo);
        const int64_t blk = LDX(p.block_table + static_cast<int64_t>(s) * p.max_blocks + bi);
        if (blk < 0 || blk >= p.num_blocks) {
          bad = true;
        } else {
          have = true;
          r0 = (blk * p.block_size + bo) * H;
          pg = blk;
        }
      }
      const uint32_t ksc = kPg && p.k_page ? 4u * H : 64u * H, vsc = kPg && p.v_page ? 4u * H : 64u * H;
      const uint32_t bytes = __reduce_add_sync(0xFFFFFFFFu, have ? 16u * H * (T::kRow - 8) + ksc + vsc : 0u);
      const bool any_bad = __any_sync(0xFFFFFFFFu, bad);
      if (k >= T::kStages && !mbar_wait(empty0 + 8 * st, ((k / T::kStages) - 1) & 1)) timed_out = true;
      if (lane == 0) {
        if (any_bad) *bad_flag = 1;  // published by the arrival below
        mbar_arrive_expect_tx(full0 + 8 * st, bytes);
      }
      __syncwarp();
      if (have) {
        const uint32_t sb = ring_s + st * T::kBytes;
        const int jr = 16 * H * lane;  // the chunk's first row in the stage planes
        const uint32_t full = full0 + 8 * st;
        bulk_copy_g2s(sb + T::kOffKC + jr * T::kCK, p.k.codes + r0 * T::kCK, 16u * H * T::kCK, full);
        bulk_copy_g2s(sb + T::kOffVC + jr * T::kCV, p.v.codes + r0 * T::kCV, 16u * H * T::kCV, full);
        if constexpr (T::kBK > 0) bulk_copy_g2s(sb + T::kOffKB + jr * T::kBK, p.k.bscale + r0 * T::kBK, 16u * H * T::kBK, full);
        if constexpr (T::kBV > 0) bulk_copy_g2s(sb + T::kOffVB + jr * T::kBV, p.v.bscale + r0 * T::kBV, 16u * H * T::kBV, full);
        bulk_copy_g2s(sb + T::kOffKR + jr * 4, p.k.rscale + (kPg && p.k_page ? pg * H : r0), ksc, full);
        bulk_copy_g2s(sb + T::kOffVR + jr * 4, p.v.rscale + (kPg && p.v_page ? pg * H : r0), vsc, full);
      }
    }
    const bool bad_any = __any_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      if (bad_any) set_status(p.status, 2u);
      if (timed_out) set_status(p.status, 16u);
    }
    return;  // the consumers' own barrier below leaves this warp out
  }

  // ---- consumers: warp w serves head h = w % H, chunk j = w / H of every stage ----
  const int h = warp % H, j = warp / H;
  // Q^T fragments (query head h * group + g, this lane's dims c*D/4 + 4kb .. + 3, scaled
  // by a power of two into f16 exactly) and the per-head query factors
  uint2 qreg[kKS];
  float qfac = 0.0f;
  {
    uint32_t w[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) w[i] = 0u;
    if (g < p.group) {
      const uint16_t* qp = p.q + static_cast<int64_t>(s) * p.q_row_pitch +
                           static_cast<int64_t>(h * p.group + g) * p.q_head_pitch + c * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t v4[4];
        load16B(qp + 8 * i, v4);
        w[4 * i] = v4[0];
        w[4 * i + 1] = v4[1];
        w[4 * i + 2] = v4[2];
        w[4 * i + 3] = v4[3];
      }
    }
    float am = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) am = fmaxf(am, fmaxf(fabsf(bf16lo(w[i])), fabsf(bf16hi(w[i]))));
    am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
    am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
    int kq = 0;
    if (am > 0.0f) kq = 14 - (static_cast<int>((__float_as_uint(am) >> 23) & 0xFF) - 127);
    kq = max(-113, min(120, kq));
    const float up = __uint_as_float(static_cast<uint32_t>(127 + kq) << 23);
    qfac = p.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - kq) << 23);
#pragma unroll
    for (int kb = 0; kb < kKS; ++kb)
      qreg[kb] = make_uint2(f32x2_to_f16x2(bf16lo(w[2 * kb]) * up, bf16hi(w[2 * kb]) * up),
                            f32x2_to_f16x2(bf16lo(w[2 * kb + 1]) * up, bf16hi(w[2 * kb + 1]) * up));
  }
  float qmul[1][2];  // heads 2c, 2c + 1: the factors of lanes (2c, 0) and (2c + 1, 0)
  qmul[0][0] = __shfl_sync(0xFFFFFFFFu, qfac, 8 * c);
  qmul[0][1] = __shfl_sync(0xFFFFFFFFu, qfac, 8 * c + 4);
  auto qb = [&](int, int kb) -> uint2 { return qreg[kb]; };

  AttnState<D, 1> st;
  st.init();
  bool timed_out = false;
  for (int k = 0; k < nstage; ++k) {
    const int stg = k % T::kStages;
    if (!mbar_wait(full0 + 8 * stg, (k / T::kStages) & 1)) timed_out = true;
    const int t0 = t_begin + 16 * (P * k + j);
    if (t0 < t_end) {
      const unsigned char* const sb = smem + stg * T::kBytes;
      const int r = 16 * H * j + h;  // row of this chunk's token 0, head h; tokens H rows apart
      const TileView tv{sb + T::kOffKC + r * T::kCK, sb + T::kOffVC + r * T::kCV, sb + T::kOffKB + r * T::kBK,
                        sb + T::kOffVB + r * T::kBV, sb + T::kOffKR + r * 4, sb + T::kOffVR + r * 4,
                        H * T::kCK, H * T::kCV, H * T::kBK, H * T::kBV,
                        kPg && p.k_page ? 0 : H * 4, kPg && p.v_page ? 0 : H * 4};
      attn_tile<D, kFK, kFV, 1>(tv, qb, qmul, lane, t_end - t0, st, NoMod{});
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8 * stg);
  }
  // the merge kernel (when the sequence is split) may be scheduled from here on; it
  // waits for this grid's writes before it reads them
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // row sums over the 8 lanes (tokens) of each head
#pragma unroll
  for (int off = 4; off <= 16; off <<= 1) {
    st.l[0][0] += __shfl_xor_sync(0xFFFFFFFFu, st.l[0][0], off);
    st.l[0][1] += __shfl_xor_sync(0xFFFFFFFFu, st.l[0][1], off);
  }
  if (__any_sync(0xFFFFFFFFu, timed_out) && lane == 0) set_status(p.status, 16u);
  // the producer's bad flag is visible: it was set before the arrival of a stage this
  // warp has waited for (or nothing was issued, and it is still 0)
  const bool cta_bad = bad_len || *bad_flag != 0;

  // this lane's O (true scale O * R), m and l for heads 2c, 2c + 1
  float O[kMT][4], M[2], L[2];
#pragma unroll
  for (int q = 0; q < kMT; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) O[q][e] = st.o[q][0][e] * st.R;
  M[0] = st.m[0][0];
  M[1] = st.m[0][1];
  L[0] = st.l[0][0];
  L[1] = st.l[0][1];
  if (P > 1) {
    // the P warps of a head merge through shared memory (the ring is free once every
    // consumer has waited for every stage): warp w's lane values at [w][lane][.]
    asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory");
    float* const mine = reinterpret_cast<float*>(smem) + (warp * 32 + lane) * T::kLaneFloats;
#pragma unroll
    for (int q = 0; q < kMT; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) mine[4 * q + e] = O[q][e];
    mine[4 * kMT] = M[0];
    mine[4 * kMT + 1] = M[1];
    mine[4 * kMT + 2] = L[0];
    mine[4 * kMT + 3] = L[1];
    asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory");
    if (j != 0) return;
    const float* const all = reinterpret_cast<const float*>(smem);
    float Mn[2] = {M[0], M[1]};
    for (int jj = 1; jj < P; ++jj) {
      const float* const o = all + ((jj * H + h) * 32 + lane) * T::kLaneFloats;
      Mn[0] = fmaxf(Mn[0], o[4 * kMT]);
      Mn[1] = fmaxf(Mn[1], o[4 * kMT + 1]);
    }
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      f[e] = M[e] == kNegInf ? 0.0f : ex2(M[e] - Mn[e]);
      L[e] *= f[e];
    }
#pragma unroll
    for (int q = 0; q < kMT; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) O[q][e] *= f[e & 1];
    for (int jj = 1; jj < P; ++jj) {
      const float* const o = all + ((jj * H + h) * 32 + lane) * T::kLaneFloats;
      float fj[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mj = o[4 * kMT + e];
        fj[e] = mj == kNegInf ? 0.0f : ex2(mj - Mn[e]);
        L[e] += o[4 * kMT + 2 + e] * fj[e];
      }
#pragma unroll
      for (int q = 0; q < kMT; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[q][e] += o[4 * q + e] * fj[e & 1];
    }
    M[0] = Mn[0];
    M[1] = Mn[1];
  }
  // heads 2c + e (e = 0, 1) of this KV head's group; dims g*D/8 + 2q and + 1
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int head = 2 * c + e;
    if (head >= p.group) continue;
    const int qh = h * p.group + head;
    if (p.nsplit == 1) {
      if (cta_bad) continue;  // a bad sequence leaves its output untouched
      uint16_t* const out = p.out + static_cast<int64_t>(s) * p.o_row_pitch + static_cast<int64_t>(qh) * p.o_head_pitch;
#pragma unroll
      for (int q = 0; q < kMT; ++q) {
        const int d = g * (D / 8) + 2 * q;
        const float y0 = L[e] == 0.0f ? 0.0f : O[q][e] / L[e];
        const float y1 = L[e] == 0.0f ? 0.0f : O[q][e + 2] / L[e];
        STX(reinterpret_cast<uint32_t*>(out + d), pack_bf16x2(y0, y1));
      }
    } else {
      float* const wsr = p.ws + ((static_cast<int64_t>(s) * p.Hq + qh) * p.nsplit + split) * (D + 2);
#pragma unroll
      for (int q = 0; q < kMT; ++q) {
        const int d = g * (D / 8) + 2 * q;
        STX(wsr + d, O[q][e]);
        STX(wsr + d + 1, O[q][e + 2]);
      }
      if (g == 0) {
        STX(wsr + D, cta_bad ? __int_as_float(0x7FC00000) : M[e]);  // NaN marks a bad sequence
        STX(wsr + D + 1, L[e]);
      }
    }
  }
}

// The merge as a programmatic dependent launch: it may be scheduled while the attention
// kernel drains and waits (griddepcontrol.wait) for that kernel's writes.
template <int D>
cudaError_t launch_merge(const AttnParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.S * p.Hq + kMergeWarps - 1) / kMergeWarps);
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_attn_merge_kernel<D>, p);
}

template <int D, int kFK, int kFV, int kNH>
cudaError_t attn_launch(const AttnParams& p, cudaStream_t s) {
  using T = AttnTile<D, kFK, kFV>;
  auto k = decode_attn_kernel<D, kFK, kFV, kNH>;
  if (T::kSmem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = cudaSuccess;
  const dim3 grid(p.nsplit, p.H, p.S);
  KVQ_LAUNCH("decode_attn_kernel", s, k<<<grid, kAttnThreads, T::kSmem, s>>>(p); e = cudaGetLastError());
  if (e != cudaSuccess || p.nsplit == 1) return e;
  KVQ_LAUNCH("decode_attn_merge_kernel", s, e = launch_merge<D>(p, s));
  return e;
}

template <int D, int kNH>
cudaError_t attn_dispatch_fmt(const AttnParams& p, cudaStream_t s) {
  const bool k8 = p.fmt_k == 3, v8 = p.fmt_v == 3;
  if (!k8 && !v8) return attn_launch<D, 1, 1, kNH>(p, s);
  if (k8 && !v8) return attn_launch<D, 3, 1, kNH>(p, s);
  if (!k8 && v8) return attn_launch<D, 1, 3, kNH>(p, s);
  return attn_launch<D, 3, 3, kNH>(p, s);
}

// Query heads per KV head: one n-tile of 8 heads, or two for 9 to 16.
template <int D>
cudaError_t attn_dispatch_group(const AttnParams& p, cudaStream_t s) {
  return p.group <= 8 ? attn_dispatch_fmt<D, 1>(p, s) : attn_dispatch_fmt<D, 2>(p, s);
}

template <int D, int kFK, int kFV, int W, int H, bool kPg = false>
cudaError_t page_launch(const AttnParams& p, cudaStream_t s) {
  using T = PageStage<D, kFK, kFV, W>;
  auto k = decode_attn_page_kernel<D, kFK, kFV, W, H, kPg>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.nsplit, 1, p.S);
  KVQ_LAUNCH("decode_attn_page_kernel", s, k<<<grid, (W + 1) * 32, T::kSmem, s>>>(p); e = cudaGetLastError());
  if (e != cudaSuccess || p.nsplit == 1) return e;
  if constexpr (kPg) {  // page-scaled calls split further: the merge that shares splits among warps
    QueryAttnParams q{};
    q.a = p;
    q.num_tokens = p.S;
    q.max_q = 1;
    return launch_query_merge_splits(q, s);
  } else {
    KVQ_LAUNCH("decode_attn_merge_kernel", s, e = launch_merge<D>(p, s));
    return e;
  }
}

template <int D, int W, int H>
cudaError_t page_dispatch_fmt(const AttnParams& p, cudaStream_t s) {
  const bool k8 = p.fmt_k == 3, v8 = p.fmt_v == 3;
  if constexpr (H >= 4) {
    if (p.k_page || p.v_page) {
      if (k8 && !v8) return page_launch<D, 3, 1, W, H, true>(p, s);
      if (!k8 && v8) return page_launch<D, 1, 3, W, H, true>(p, s);
      return page_launch<D, 3, 3, W, H, true>(p, s);
    }
  }
  if (!k8 && !v8) return page_launch<D, 1, 1, W, H>(p, s);
  if (k8 && !v8) return page_launch<D, 3, 1, W, H>(p, s);
  if (!k8 && v8) return page_launch<D, 1, 3, W, H>(p, s);
  return page_launch<D, 3, 3, W, H>(p, s);
}

// One instance per KV head count: the stage layout's strides are then constants.
template <int D>
cudaError_t page_dispatch(const AttnParams& p, cudaStream_t s) {
  switch (p.H) {
    case 1: return page_dispatch_fmt<D, 8, 1>(p, s);
    case 2: return page_dispatch_fmt<D, 8, 2>(p, s);
    case 4: return page_dispatch_fmt<D, 8, 4>(p, s);
    case 8: return page_dispatch_fmt<D, 8, 8>(p, s);
    case 16: return page_dispatch_fmt<D, 16, 16>(p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// Split policy: CTAs resident per SM assumed by the wave count (4 at D <= 128), and
// the most waves a split may create.
constexpr int kAttnCtasPerSm = 4;
constexpr int kAttnMaxWaves = 4;

// Built-in split scratch for kvq_decode_attention_noalloc, for callers that cannot
// allocate device memory: it is part of the library image, so every GPU that loads
// the library holds these 48 MiB until the process exits, and no call allocates.
// One array per device, shared by every call on it: calls that overlap on the GPU
// race on it.  Each call writes every partial it later reads, so nothing in it needs
// clearing between calls.  The policy above keeps S*H*nsplit <= 4 waves = 16 * SMs
// CTAs, so the partials take at most 16 * SMs * 16 query heads * (256 + 2) * 4
// bytes: 40.2 MB on 152 SMs.
constexpr size_t kAttnScratchBytes = size_t{48} << 20;
static __device__ __align__(256) float g_attn_scratch[kAttnScratchBytes / sizeof(float)];

// Host code may not pass g_attn_scratch itself to a kernel: on the host that name is a
// stand-in, not a device address.  The device address is looked up once per device,
// with that device current, on the first call there, and kept.
constexpr int kScratchDevices = 64;
static std::atomic<void*> g_scratch_addr[kScratchDevices];
static std::mutex g_scratch_mu;

cudaError_t attn_builtin_scratch(void** ptr, size_t* bytes) {
  *bytes = kAttnScratchBytes;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kScratchDevices) return cudaErrorInvalidDevice;
  void* addr = g_scratch_addr[dev].load(std::memory_order_acquire);
  if (addr == nullptr) {
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    addr = g_scratch_addr[dev].load(std::memory_order_relaxed);
    if (addr == nullptr) {
      e = cudaGetSymbolAddress(&addr, g_attn_scratch);
      if (e != cudaSuccess || addr == nullptr) {
        cudaGetLastError();  // leave no error behind for the launch check
        return e != cudaSuccess ? e : cudaErrorInvalidSymbol;
      }
      g_scratch_addr[dev].store(addr, std::memory_order_release);
    }
  }
  *ptr = addr;
  return cudaSuccess;
}

size_t attn_builtin_scratch_bytes() { return kAttnScratchBytes; }

int attn_num_splits(int32_t S, int32_t H, int32_t max_seq_len) {
  const int64_t pairs = static_cast<int64_t>(S) * H;
  if (pairs <= 0 || max_seq_len <= 0) return 1;
  const int64_t slots = static_cast<int64_t>(kAttnCtasPerSm) * num_sms();  // CTAs resident at once
  int64_t cap = (static_cast<int64_t>(max_seq_len) + 255) / 256;                                  // >= 256 tokens per split
  const int64_t waves_cap = (kAttnMaxWaves * slots) / pairs;                  // <= kAttnMaxWaves waves
  if (waves_cap < cap) cap = waves_cap;
  if (cap > 64) cap = 64;
  // the split count whose last wave is fullest (least idle CTA time), the smallest on ties
  int best = 1;
  double best_fill = 0.0;
  for (int64_t n = 1; n <= cap; ++n) {
    const int64_t ctas = pairs * n;
    const int64_t waves = (ctas + slots - 1) / slots;
    const double fill = static_cast<double>(ctas) / static_cast<double>(waves * slots);
    if (fill > best_fill + 0.01) {
      best_fill = fill;
      best = static_cast<int>(n);
    }
  }
  return best;
}

// The page-major kernel serves pages of whole 16-token chunks (block_size a multiple of
// 16), head_dim 64 or 128, up to 8 query heads per KV head, and H in {1, 2, 4, 8, 16}
// (W = 8 consumer warps, or 16 at H = 16, P = W / H chunks per stage).  The H scales of
// a page are one bulk copy only from H = 4 (16 bytes).
bool attn_page_ok(int32_t block_size, int32_t H, int32_t D, int32_t group, bool page_scaled) {
  return block_size % 16 == 0 && (D == 64 || D == 128) && group <= 8 &&
         (H == 1 || H == 2 || H == 4 || H == 8 || H == 16) && (!page_scaled || H >= 4);
}

// Splits of the page-major kernel: one block per (split, sequence), 2 resident per SM
// (1 at H = 16); at least 256 tokens a split, and S * H * nsplit <= 16 * SMs so the
// partials stay within the bound of the built-in scratch; the count whose last wave is
// fullest, the smallest on ties.
int attn_page_splits(int32_t S, int32_t H, int32_t max_seq_len) {
  if (S <= 0 || H <= 0 || max_seq_len <= 0) return 1;
  const int64_t slots = static_cast<int64_t>(H == 16 ? 1 : 2) * num_sms();
  int64_t cap = (static_cast<int64_t>(max_seq_len) + 255) / 256;
  const int64_t scratch_cap = (static_cast<int64_t>(kAttnCtasPerSm) * kAttnMaxWaves * num_sms()) /
                              (static_cast<int64_t>(S) * H);
  if (scratch_cap < cap) cap = scratch_cap;
  if (cap > 64) cap = 64;
  int best = 1;
  double best_fill = 0.0;
  for (int64_t n = 1; n <= cap; ++n) {
    const int64_t ctas = static_cast<int64_t>(S) * n;
    const int64_t waves = (ctas + slots - 1) / slots;
    const double fill = static_cast<double>(ctas) / static_cast<double>(waves * slots);
    if (fill > best_fill + 0.01) {
      best_fill = fill;
      best = static_cast<int>(n);
    }
  }
  return best;
}

// Splits of a page-scaled pool's calls in the page-major kernel: 2 blocks an SM (1 at H = 16), at
// least 64 tokens a split, so that short sequences spread over the GPU too.  At most two waves,
// 4 SMs x 64 query heads x 130 (or 2 SMs x 128 x 130) partials of 4 bytes: 20.2 MB on 152 SMs.
int attn_page_scaled_splits(int32_t S, int32_t H, int32_t Hq, int32_t D, int32_t max_seq_len) {
  const bool ok = (D == 64 || D == 128) && (H == 4 || H == 8 || H == 16) && Hq / H <= 8;
  if (!ok || S <= 0 || max_seq_len <= 0) return 1;
  return fill_splits(S, static_cast<int64_t>(H == 16 ? 1 : 2) * num_sms(), max_seq_len, 64, 384);
}

// Tokens per split: the splits cover max_seq_len in multiples of `unit` tokens.
static int attn_split_len(int32_t max_seq_len, int nsplit, int unit) {
  const int64_t per = (static_cast<int64_t>(max_seq_len) + nsplit - 1) / nsplit;
  const int64_t len = ((per + unit - 1) / unit) * unit;
  return len > 0 ? static_cast<int>(std::min(len, int64_t{0x7FFFFFC0})) : unit;  // a multiple of both units
}

size_t attn_workspace_bytes(int32_t S, int32_t H, int32_t Hq, int32_t D, int32_t max_seq_len, bool page_scaled) {
  if (S <= 0 || H <= 0 || Hq <= 0 || D <= 0 || max_seq_len <= 0) return 0;
  // either kernel may serve the call (the choice also depends on the pool's block size)
  int n = attn_num_splits(S, H, max_seq_len);
  const int np = attn_page_splits(S, H, max_seq_len);
  if (np > n) n = np;
  const int ns = page_scaled ? attn_page_scaled_splits(S, H, Hq, D, max_seq_len) : 1;
  if (ns > n) n = ns;
  const size_t bytes = n <= 1 ? 0 : static_cast<size_t>(S) * Hq * n * (D + 2) * sizeof(float);
  // the whole-page kernel's partials: at most 8 SMs x 64 query heads x 130, or 4 SMs x 128 x 130, or
  // 4 SMs x 64 x 258 of 4 bytes, 40.5 MB on 152 SMs
  if (!page_scaled || (H != 4 && H != 8) || Hq / H > 16) return bytes;
  const size_t pages = query_pages_workspace_bytes(S, S, Hq, D, Hq / H, max_seq_len);
  return pages > bytes ? pages : bytes;
}

cudaError_t launch_decode_attention(const AttnParams& p_in, cudaStream_t s) {
  AttnParams p = p_in;
  if ((p.k_page || p.v_page) && p.H <= 8 && query_pages_ok(p.block_size, p.H, true) &&
      (p.D == 256 || p.group > 8 || query_pages_share(p.S, p.D, p.group, p.max_len))) {
    // what the page-major kernel does not take, or takes in equal parts only: the whole-page
    // kernel of kvq_attention, one query token a sequence (head_dim 256, 2 x 65536 tokens, H4: 58 us;
    // 91 us by the head-major kernel below)
    QueryAttnParams q{};
    q.a = p;
    q.num_tokens = p.S;
    q.max_q = 1;
    return launch_query_pages(q, p.max_len, s);
  }
  if (attn_page_ok(p.block_size, p.H, p.D, p.group, p.k_page || p.v_page)) {
    p.nsplit = p.k_page || p.v_page ? attn_page_scaled_splits(p.S, p.H, p.Hq, p.D, p.max_len)
                                    : attn_page_splits(p.S, p.H, p.max_len);
    p.split_len = attn_split_len(p.max_len, p.nsplit, 16);
    switch (p.D) {
      case 64: return page_dispatch<64>(p, s);
      case 128: return page_dispatch<128>(p, s);
    }
    return cudaErrorInvalidValue;
  }
  p.nsplit = attn_num_splits(p.S, p.H, p.max_len);
  p.split_len = attn_split_len(p.max_len, p.nsplit, 64);
  switch (p.D) {
    case 64: return attn_dispatch_group<64>(p, s);
    case 128: return attn_dispatch_group<128>(p, s);
    case 256: return attn_dispatch_group<256>(p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
