// query_attn_kernels.cu -- paged attention of several query tokens per sequence.
//
// Sequence s has n = starts[s + 1] - starts[s] query tokens, its last ones: token i sits
// at position pos = seq_lens[s] - n + i and sees the keys t of [lo, hi),
//   hi = max(pos + 1, min(prefix, len)),  lo = max(0, pos + 1 - window, key_start),
// with logits  cap(scale q . k_t) + slope (t - pos),  cap(x) = softcap tanh(x / softcap).
// A row that sees no key is 0.
//
// Rows kernel (few rows; many go to query_tile_kernels.cu): a CTA takes 8 or 16 rows (token i, query head of the group) of
// one KV head and one split of the keys that any of its rows sees; its 4 warps take
// 16-token tiles in turn through cp.async rings, with the tile arithmetic of the decode
// kernels (attn_tile.cuh), the score modifier between its two products.  Splits of a
// sequence merge through the caller's workspace in a second small kernel.  Bound: issue and
// latency of the tile arithmetic, and gathers of 64 to 256 bytes (16 x 5000 tokens over NVFP4 with
// bias, 64 query heads, 8-token pages: 46.5 us; 39.5 by whole pages of 16 tokens).
#include <algorithm>

#include "query_attn.cuh"

namespace kvq {

namespace {

template <int D, int kFK, int kFV, int kNH>
__global__ void __launch_bounds__(kAttnThreads) query_rows_kernel(const QueryAttnParams qp) {
  using T = AttnTile<D, kFK, kFV>;
  const AttnParams& p = qp.a;
  constexpr int kKS = D / 16;
  constexpr int kMT = D / 16;
  constexpr int kRows = 8 * kNH;
  constexpr bool kQReg = kNH * kKS <= 8;
  extern __shared__ __align__(16) unsigned char smem[];

  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int g = lane >> 2;
  const int c = lane & 3;
  const int s = blockIdx.z, h = blockIdx.y;
  const int tile = blockIdx.x / p.nsplit, split = blockIdx.x - tile * p.nsplit;
  const int row0 = tile * kRows;  // first row (i * group + head) of the CTA

  int q0, nq, len;
  const bool ok = query_range(qp, s, q0, nq, len);
  if (!ok && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) set_status(p.status, 8u);
  const int rows = nq * p.group;
  if (row0 >= rows) return;

  int lo, hi;  // lane r < kRows: row r's range; the CTA's keys are the union
  lane_range(qp, lane, kRows, s, q0, nq, len, row0, rows, lo, hi);
  const int lo_min = __reduce_min_sync(0xFFFFFFFFu, lo);
  const int hi_max = __reduce_max_sync(0xFFFFFFFFu, hi);
  int t_begin = 0, t_end = 0;
  if (lo_min < hi_max) {  // equal splits, in whole tiles for the four warps
    const int per = ((hi_max - lo_min + p.nsplit - 1) / p.nsplit + 63) / 64 * 64;
    t_begin = static_cast<int>(min(static_cast<int64_t>(lo_min) + static_cast<int64_t>(split) * per, static_cast<int64_t>(hi_max)));
    t_end = t_begin + min(per, hi_max - t_begin);
  }
  const int ntile = (t_end - t_begin + 15) / 16;

  // ---- Q^T fragments: in registers, or warp 0's in shared memory ----
  uint2* const qfrag = reinterpret_cast<uint2*>(smem);
  uint2 qreg[kQReg ? kNH : 1][kKS];
  float row_fac[kNH];
#pragma unroll
  for (int nh = 0; nh < kNH; ++nh) {
    uint2(&f)[kKS] = qreg[kQReg ? nh : 0];
    row_fac[nh] = query_fragments<D>(p, lane, h, q0, row0 + 8 * nh + g, rows, f);
    if (!kQReg && warp == 0) {
#pragma unroll
      for (int kb = 0; kb < kKS; ++kb) qfrag[(nh * kKS + kb) * 32 + lane] = f[kb];
    }
  }
  __shared__ __align__(16) typename QueryMod<kNH>::Tables tab;
  QueryMod<kNH>::fill(&tab, qp, lane, h, 0, row0, rows, lo, hi, warp == 0, warp == 0);
  __syncthreads();
  QueryMod<kNH> mod;
  float qmul[kNH][2];
  mod.init(&tab, qp, lane, 0, row0, rows, len - nq, lo, hi, row_fac, qmul);
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
  const bool lane_page = lane < 16 ? p.k_page : p.v_page;
  auto row_of = [&](int it, int64_t& srow) -> int64_t {
    const int kt = warp + it * kAttnWarps;
    srow = 0;
    if (kt >= ntile) return -1;
    int t = t_begin + kt * 16 + (lane & 15);
    if (t >= t_end) t = t_end - 1;  // a token that is read anyway; masked later
    uint32_t bi, bo;
    p.div_bs.divmod(static_cast<uint32_t>(t), bi, bo);
    int64_t blk = LDX(p.block_table + static_cast<int64_t>(s) * p.max_blocks + bi);
    if (blk < 0 || blk >= p.num_blocks) {
      bad = true;
      return -2;
    }
    const int64_t row = (blk * p.block_size + bo) * p.H + h;
    srow = lane_page ? blk * p.H + h : row;
    return row;
  };
  // a tile with tokens of bad block entries: those become zeros, which rows that do not see
  // them may meet
  auto issue_around_gaps = [&](int64_t row, int64_t srow, unsigned char* sb) {
    for (int j = 0; j < 16; ++j) {
      const int64_t rr = shfl64(row, j);
      for (int i = lane; i < T::kCK / 16; i += 32) {
        if (rr >= 0) cp_async16(sb + T::kOffKC + j * T::kSK + i * 16, p.k.codes + rr * T::kCK + i * 16);
        else *reinterpret_cast<uint4*>(sb + T::kOffKC + j * T::kSK + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      for (int i = lane; i < T::kCV / 16; i += 32) {
        if (rr >= 0) cp_async16(sb + T::kOffVC + j * T::kSV + i * 16, p.v.codes + rr * T::kCV + i * 16);
        else *reinterpret_cast<uint4*>(sb + T::kOffVC + j * T::kSV + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    const int tt = lane & 15;
    if (row < 0) {
      unsigned char* const b = lane < 16 ? sb + T::kOffKB + tt * T::kBK : sb + T::kOffVB + tt * T::kBV;
      for (int i = 0; i < (lane < 16 ? T::kBK : T::kBV); ++i) b[i] = 0;
      *reinterpret_cast<float*>(sb + (lane < 16 ? T::kOffKR : T::kOffVR) + tt * 4) = 0.0f;
    } else if (lane < 16) {
      if constexpr (T::kBK > 0) cp_async_n<T::kBK>(sb + T::kOffKB + tt * T::kBK, p.k.bscale + row * T::kBK);
      cp_async_small<4>(sb + T::kOffKR + tt * 4, p.k.rscale + srow);
    } else {
      if constexpr (T::kBV > 0) cp_async_n<T::kBV>(sb + T::kOffVB + tt * T::kBV, p.v.bscale + row * T::kBV);
      cp_async_small<4>(sb + T::kOffVR + tt * 4, p.v.rscale + srow);
    }
  };
  auto issue = [&](int64_t row, int64_t srow, int st) {
    if (__shfl_sync(0xFFFFFFFFu, row, 0) == -1) return;
    unsigned char* const sb = ring + st * T::kBytes;
    if (__any_sync(0xFFFFFFFFu, row < 0)) {
      issue_around_gaps(row, srow, sb);
      return;
    }
    const int tt = lane & 15;
    constexpr int kPK = T::kCK / 16, kPV = T::kCV / 16;
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
    if (lane < 16) {
      if constexpr (T::kBK > 0) cp_async_n<T::kBK>(sb + T::kOffKB + tt * T::kBK, p.k.bscale + row * T::kBK);
      cp_async_small<4>(sb + T::kOffKR + tt * 4, p.k.rscale + srow);
    } else {
      if constexpr (T::kBV > 0) cp_async_n<T::kBV>(sb + T::kOffVB + tt * T::kBV, p.v.bscale + row * T::kBV);
      cp_async_small<4>(sb + T::kOffVR + tt * 4, p.v.rscale + srow);
    }
  };

  AttnState<D, kNH> st;
  st.init(kNoKey);
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
    const int64_t row_next = row_of(it + T::kStages - 1, srow_next);
    cp_async_wait<T::kStages - 2>();
    __syncwarp();
    const unsigned char* const sb = ring + (it % T::kStages) * T::kBytes;
    const int t0 = t_begin + (warp + it * kAttnWarps) * 16;
    const TileView tv{sb + T::kOffKC, sb + T::kOffVC, sb + T::kOffKB, sb + T::kOffVB, sb + T::kOffKR, sb + T::kOffVR,
                      T::kSK, T::kSV, T::kBK, T::kBV, 4, 4};
    mod.t0 = t0;
    attn_tile<D, kFK, kFV, kNH>(tv, qb, qmul, lane, t_end - t0, st, mod);
    __syncwarp();
    issue(row_next, srow_next, (it + T::kStages - 1) % T::kStages);
    cp_async_commit();
  }
  cp_async_wait<0>();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) set_status(p.status, 2u);
#pragma unroll
  for (int off = 4; off <= 16; off <<= 1)
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh) {
      st.l[nh][0] += __shfl_xor_sync(0xFFFFFFFFu, st.l[nh][0], off);
      st.l[nh][1] += __shfl_xor_sync(0xFFFFFFFFu, st.l[nh][1], off);
    }
  __shared__ uint32_t bad_rows;
  if (threadIdx.x == 0) bad_rows = 0u;
  if (__syncthreads_or(bad ? 1 : 0) != 0) {  // (the ring is free after this)
    for (int r = warp; r < min(kRows, rows - row0); r += kAttnWarps)
      if (needs_bad_block(p, s, max(tab.range[r].x, t_begin), min(tab.range[r].y, t_end)) && lane == 0)
        atomicOr(&bad_rows, 1u << r);
  }

  float* const mo = reinterpret_cast<float*>(smem + T::kQ) + warp * kRows * (D + 2);
#pragma unroll
  for (int q = 0; q < kMT; ++q)
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        mo[(8 * nh + 2 * c + (e & 1)) * (D + 2) + g * (D / 8) + 2 * q + (e >> 1)] = st.o[q][nh][e] * st.R;
  if (g == 0) {
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mo[(8 * nh + 2 * c + e) * (D + 2) + D] = st.m[nh][e];
        mo[(8 * nh + 2 * c + e) * (D + 2) + D + 1] = st.l[nh][e];
      }
  }
  __syncthreads();
  const float* const mall = reinterpret_cast<const float*>(smem + T::kQ);
  const int live = min(kRows, rows - row0);
  for (int idx = threadIdx.x; idx < live * D; idx += kAttnThreads) {
    const int row = idx / D, d = idx % D;
    float M = kNoKey;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) M = fmaxf(M, mall[(w * kRows + row) * (D + 2) + D]);
    float L = 0.0f, O = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      const float f = ex2(mall[(w * kRows + row) * (D + 2) + D] - M);
      L += mall[(w * kRows + row) * (D + 2) + D + 1] * f;
      O += mall[(w * kRows + row) * (D + 2) + d] * f;
    }
    const int i = (row0 + row) / p.group;
    const int qh = h * p.group + row0 + row - i * p.group;
    const int64_t tok = q0 + i;
    const bool row_bad = ((bad_rows >> row) & 1u) != 0u;
    if (p.nsplit == 1) {
      if (row_bad) continue;
      const float y = L == 0.0f ? 0.0f : O / L;
      STX(p.out + tok * p.o_row_pitch + static_cast<int64_t>(qh) * p.o_head_pitch + d,
          static_cast<uint16_t>(pack_bf16x2(y, 0.0f) & 0xFFFFu));
    } else {
      float* const wsr = p.ws + ((tok * p.Hq + qh) * p.nsplit + split) * (D + 2);
      STX(wsr + d, O);
      if (d == 0) {
        STX(wsr + D, row_bad ? __int_as_float(0x7FC00000) : M);  // NaN marks a bad block entry (M never is one)
        STX(wsr + D + 1, L);
      }
    }
  }
}

// Merge of the splits of each (token, query head): o = sum_k O_k 2^(M_k - M) / sum_k L_k 2^(M_k -
// M), by kPer warps a row, which share the splits (one warp walking 76 splits of two rows took
// longer than their attention's last wave).  A row's warps first find its token's sequence
// (32-way search over starts): rows of no sequence, or of a refused one, have no partials and
// stay as they are, as do rows with a NaN mark in place of an M.  A NaN L is a NaN score's and
// reaches the output.
template <int kPer>
constexpr int kMergeWarps = kPer > 4 ? kPer : 4;  // of a block

template <int D, int kPer>
__global__ void __launch_bounds__(32 * kMergeWarps<kPer>) query_merge_kernel(const QueryAttnParams qp) {
  const AttnParams& p = qp.a;
  constexpr int kDL = D / 32;
  constexpr int kWarps = kMergeWarps<kPer>;
  constexpr int kRows = kWarps / kPer;  // a block
  __shared__ float2 part_ml[kWarps];
  __shared__ float part_o[kPer > 1 ? kWarps : 1][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % kPer;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + warp / kPer;
  const bool live = row < static_cast<int64_t>(qp.num_tokens) * p.Hq;
  const int tok = live ? static_cast<int>(row / p.Hq) : 0, qh = static_cast<int>(row - static_cast<int64_t>(tok) * p.Hq);
  int lo = 0, hi = p.S;  // the last s < S with starts[s] <= tok lies in [lo, hi)
  if (qp.starts == nullptr) lo = hi = tok;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool below = at < hi && LDX(qp.starts + at) <= tok;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, below);
    const int last = m != 0u ? 31 - __clz(m) : 0;
    hi = min(hi, lo + (last + 1) * step);
    lo += last * step;
  }
  int q0, n, len;
  const bool owned = query_range(qp, lo, q0, n, len) && tok >= q0 && tok < q0 + n;
  // launched as a programmatic dependent of the attention kernel: wait for its results
  // (every block does, so that this grid's end implies the other's)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool mine = live && owned;  // the same for all of a row's warps
  if (kPer == 1 && !mine) return;
  const float* const base = p.ws + row * p.nsplit * (D + 2);
  const int nsplit = !mine ? 0 : qp.parts != nullptr ? LDX(qp.parts + lo) : p.nsplit;
  const bool done = qp.parts != nullptr && nsplit == 1;  // written by the attention kernel
  if (kPer == 1 && done) return;
  const int per = (nsplit + kPer - 1) / kPer;
  const int k_begin = done ? 0 : min(part * per, nsplit), k_end = done ? 0 : min(k_begin + per, nsplit);
  // the O rows of the first kPre splits are loaded together with M and L: one wait for memory
  constexpr int kPre = 64 / kDL;
  float2 pre[kPre][kDL / 2];
#pragma unroll
  for (int k = 0; k < kPre; ++k)
#pragma unroll
    for (int i = 0; i < kDL / 2; ++i)
      pre[k][i] = k_begin + k < k_end ? LDX(reinterpret_cast<const float2*>(base + (k_begin + k) * (D + 2) + kDL * lane + 2 * i))
                                      : make_float2(0.0f, 0.0f);
  float M = kNoKey, L = 0.0f;
  bool bad = false;
  for (int k = k_begin + lane; k < k_end; k += 32) {
    const float2 ml = LDX(reinterpret_cast<const float2*>(base + k * (D + 2) + D));
    M = fmaxf(M, ml.x);
    bad = bad || isnan(ml.x);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
  float o[kDL];
#pragma unroll
  for (int i = 0; i < kDL; ++i) o[i] = 0.0f;
  for (int k0 = k_begin; k0 < k_end; k0 += 32) {
    float f = 0.0f;
    if (k0 + lane < k_end) {
      const float2 ml = LDX(reinterpret_cast<const float2*>(base + (k0 + lane) * (D + 2) + D));
      f = ex2(ml.x - M);
      L += ml.y * f;
    }
    if (k0 == k_begin) {
#pragma unroll
      for (int k = 0; k < kPre; ++k) {
        const float fk = __shfl_sync(0xFFFFFFFFu, f, k);  // 0 past the last split
#pragma unroll
        for (int i = 0; i < kDL / 2; ++i) {
          o[2 * i] = __fmaf_rn(pre[k][i].x, fk, o[2 * i]);
          o[2 * i + 1] = __fmaf_rn(pre[k][i].y, fk, o[2 * i + 1]);
        }
      }
    }
    const int nk = min(32, k_end - k0);
#pragma unroll 8
    for (int k = k0 == k_begin ? kPre : 0; k < nk; ++k) {
      const float fk = __shfl_sync(0xFFFFFFFFu, f, k);
      const float* const ok = base + (k0 + k) * (D + 2) + kDL * lane;
#pragma unroll
      for (int i = 0; i < kDL; i += 2) {
        const float2 v = LDX(reinterpret_cast<const float2*>(ok + i));
        o[i] = __fmaf_rn(v.x, fk, o[i]);
        o[i + 1] = __fmaf_rn(v.y, fk, o[i + 1]);
      }
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, off);
  bad = __any_sync(0xFFFFFFFFu, bad);
  if constexpr (kPer > 1) {
    if (lane == 0) part_ml[warp] = make_float2(bad ? __int_as_float(0x7FC00000) : M, L);
#pragma unroll
    for (int i = 0; i < kDL; ++i) part_o[warp][kDL * lane + i] = o[i];
    __syncthreads();
    if (part != 0 || !mine || done) return;
#pragma unroll
    for (int w = 1; w < kPer; ++w) M = fmaxf(M, part_ml[warp + w].x);
    L = 0.0f;
#pragma unroll
    for (int i = 0; i < kDL; ++i) o[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < kPer; ++w) {
      const float2 ml = part_ml[warp + w];
      bad = bad || isnan(ml.x);
      const float f = ex2(ml.x - M);
      L += ml.y * f;
#pragma unroll
      for (int i = 0; i < kDL; ++i) o[i] = __fmaf_rn(part_o[warp + w][kDL * lane + i], f, o[i]);
    }
  }
  if (bad) return;
  uint16_t* const out = p.out + static_cast<int64_t>(tok) * p.o_row_pitch + static_cast<int64_t>(qh) * p.o_head_pitch;
#pragma unroll
  for (int i = 0; i < kDL; i += 2) {
    const float y0 = L == 0.0f ? 0.0f : o[i] / L;
    const float y1 = L == 0.0f ? 0.0f : o[i + 1] / L;
    STX(reinterpret_cast<uint32_t*>(out + kDL * lane + i), pack_bf16x2(y0, y1));
  }
}

template <int D, int kPer>
cudaError_t launch_query_merge(const QueryAttnParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int64_t rows = static_cast<int64_t>(p.num_tokens) * p.a.Hq;
  constexpr int kWarps = kMergeWarps<kPer>;
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kWarps / kPer - 1) / (kWarps / kPer)));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, query_merge_kernel<D, kPer>, p);
}

template <int D>
cudaError_t launch_query_merge(const QueryAttnParams& p, cudaStream_t s) {
  // Warps a row by its splits (of shared blocks the usual count, half the most).  us of the whole
  // call by fewer warps and by these: 188 splits of 32 rows 21.5 by four, 16.8 by 8, 15.2 by 16; 76 of
  // 256 rows 32.8 by four, 31.0 by 8, 34.2 by 16; 6 of 1600 rows, the merge alone, 10.2 by four, 5.6 by one
  const int n = p.parts != nullptr ? p.a.nsplit / 2 : p.a.nsplit;
  if (n >= 96) return launch_query_merge<D, 16>(p, s);
  if (n >= 32) return launch_query_merge<D, 8>(p, s);
  return n >= 12 ? launch_query_merge<D, 4>(p, s) : launch_query_merge<D, 1>(p, s);
}

template <int D, int kFK, int kFV, int kNH>
cudaError_t rows_launch(const QueryAttnParams& p, cudaStream_t s) {
  using T = AttnTile<D, kFK, kFV>;
  auto k = query_rows_kernel<D, kFK, kFV, kNH>;
  if (T::kSmem + sizeof(typename QueryMod<kNH>::Tables) > 48 * 1024) {  // what needs no opt-in
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = cudaSuccess;
  const int64_t tiles = (static_cast<int64_t>(p.max_q) * p.a.group + 8 * kNH - 1) / (8 * kNH);
  const dim3 grid(static_cast<unsigned>(tiles * p.a.nsplit), p.a.H, p.a.S);
  KVQ_LAUNCH("query_rows_kernel", s, k<<<grid, kAttnThreads, T::kSmem, s>>>(p); e = cudaGetLastError());
  return e;
}

template <int D, int kNH>
cudaError_t rows_dispatch_fmt(const QueryAttnParams& p, cudaStream_t s) {
  const bool k8 = p.a.fmt_k == 3, v8 = p.a.fmt_v == 3;
  if (!k8 && !v8) return rows_launch<D, 1, 1, kNH>(p, s);
  if (k8 && !v8) return rows_launch<D, 3, 1, kNH>(p, s);
  if (!k8 && v8) return rows_launch<D, 1, 3, kNH>(p, s);
  return rows_launch<D, 3, 3, kNH>(p, s);
}

template <int D>
cudaError_t rows_dispatch(const QueryAttnParams& p, int rows, cudaStream_t s) {
  return rows <= 8 ? rows_dispatch_fmt<D, 1>(p, s) : rows_dispatch_fmt<D, 2>(p, s);
}

// Kernels and their split counts.  The tile kernel from 17 rows a sequence and KV head on (its
// cost hardly grows up to 128 rows; the others take 16 at a time); below, whole pages where
// the layout allows it, else the rows kernel.  16 sequences of 3000 page-scaled tokens, 8 KV heads,
// head_dim 128, tile and whole-page kernel: 16 rows 52.0, 34.1 us; 20 rows 52.0, 53.3; 32 rows 52.3,
// 55.9.
constexpr int kTileFrom = 17;

int tile_splits(int32_t S, int32_t H, int32_t D, int64_t rows, int32_t span) {
  // one CTA an SM, at least 512 tokens a split (160 rows a KV head of one sequence: 3000 tokens
  // 25.6 us, 25.2 at 256, 31.9 at 1024; 12,000 tokens 32.6, 32.7, 35.7)
  const int64_t ctas = static_cast<int64_t>(S) * H * ((rows + query_tile_rows(D) - 1) / query_tile_rows(D));
  return fill_splits(ctas, num_sms(), span, 512, 512);
}
bool page_two(int32_t D, int64_t rows) { return rows > 8 && D != 256; }  // 16 rows a block spill at head_dim 256

// The whole-page kernel's blocks.  Several sequences share one or two waves of them by length
// (page_job): in equal parts their longest sets the time.  GPU us in equal parts and shared (as the
// rule was taken), one
// token each: lengths of 1 to L, NVFP4 with bias, 16 x 5000 34.4, 29.9; page-scaled, 24 x 6000 42.3,
// 35.9; 50 x 6000 76.7, 55.7; 100 x 6000 145, 120; 250 x 6000 396, 329; all of one length, 32 x 8192
// 86.4, 88.9; 50 x 6000 98.3, 101; 250 x 6000 449, 482.  Not where there is little to share: below
// 96 keys a resident block (every block reads all lengths first, 1 us), or below 4096 keys
// where it takes two waves (100 x 1500: ragged 45.7, 45.6, of one length 56.9, 67.4); nor for more
// tiles than a wave holds, or for more than 512 sequences.  One line of all the work in equal
// shares, several sequences' parts to a block, was better for many (250 x 6000 269) and worse for
// few (16 x 6000 30, against 25.9): a second part's start costs as much as five stages.
struct PagePlan {
  int nsplit;  // partials a row
  int blocks;  // when balanced, else 0
  int wave;
};
PagePlan page_plan(int32_t S, int32_t D, int64_t rows, int32_t span) {
  // two blocks an SM (one with 16 rows or head_dim 256); at least 64 keys a split (one sequence
  // of 500 10.3 us, 11.7 at 96, 13.3 at 128; of 2000 10.7, 12.2, 13.6)
  const int64_t per = page_two(D, rows) ? 16 : 8;
  const int64_t slots = static_cast<int64_t>(per == 16 || D == 256 ? 1 : 2) * num_sms();
  const int64_t ctas = static_cast<int64_t>(S) * ((rows + per - 1) / per);
  const int n = fill_splits(ctas, slots, span, 64, 384);
  if (S == 1 || S > 512 || ctas > slots || ctas * span < 96 * slots) return PagePlan{n, 0, 0};
  const bool two = 4 * ctas > slots;
  if (two && span < 4096) return PagePlan{n, 0, 0};
  const int64_t blocks = two ? 2 * slots : slots;
  const int64_t most = std::min((static_cast<int64_t>(span) + 63) / 64, 2 * blocks / ctas);
  return PagePlan{static_cast<int>(std::min(std::max(most, static_cast<int64_t>(n)), int64_t{256})),
                  static_cast<int>(blocks), static_cast<int>(slots)};
}
int row_splits(int32_t S, int32_t H, int64_t rows, int32_t span) {
  // four CTAs an SM; at least 256 tokens a split (8 KV heads, 1 x 1000 tokens 9.1 us, 7.6 at 128;
  // 1 x 12,000 11.8, 16.9; 4 x 3000 11.7, 15.9)
  const int64_t ctas = static_cast<int64_t>(S) * H * (rows <= 8 ? 1 : (rows + 15) / 16);
  return fill_splits(ctas, 4ll * num_sms(), span, 256, 256);
}

}  // namespace

int fill_splits(int64_t ctas, int64_t slots, int32_t tokens, int32_t min_one, int32_t min_two) {
  // within a number of waves more splits fill them better, so each bound is its best count
  auto most = [&](int64_t waves, int32_t least) {
    const int64_t cap = std::min((static_cast<int64_t>(tokens) + least - 1) / least, waves * slots / ctas);
    return std::max(int64_t{1}, std::min(cap, int64_t{256}));
  };
  auto fill = [&](int64_t n) {
    const int64_t waves = (ctas * n + slots - 1) / slots;
    return static_cast<double>(ctas * n) / static_cast<double>(waves * slots);
  };
  const int64_t one = most(1, min_one), two = most(2, min_two);
  return static_cast<int>(two > one && fill(two) > 1.08 * fill(one) ? two : one);
}

cudaError_t launch_query_merge_splits(const QueryAttnParams& p, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (p.a.nsplit == 1) return e;
  KVQ_LAUNCH("query_merge_kernel", s,
             e = p.a.D == 64    ? launch_query_merge<64>(p, s)
                 : p.a.D == 128 ? launch_query_merge<128>(p, s)
                                : launch_query_merge<256>(p, s));
  return e;
}

bool query_pages_ok(int32_t block_size, int32_t H, bool page_scaled) {
  return block_size % 16 == 0 && (H == 1 || H == 2 || H == 4 || H == 8) && (H >= 4 || !page_scaled);
}

bool query_pages_share(int32_t S, int32_t D, int64_t rows, int32_t span) { return page_plan(S, D, rows, span).blocks > 0; }

size_t query_pages_workspace_bytes(int32_t S, int32_t num_tokens, int32_t Hq, int32_t D, int64_t rows, int32_t max_len) {
  const PagePlan plan = page_plan(S, D, rows, max_len);
  if (plan.nsplit <= 1) return 0;
  return static_cast<size_t>(num_tokens) * Hq * plan.nsplit * (D + 2) * sizeof(float) + (plan.blocks > 0 ? 4 * static_cast<size_t>(S) : 0);
}

cudaError_t launch_query_pages(const QueryAttnParams& p_in, int32_t span, cudaStream_t s) {
  QueryAttnParams p = p_in;
  const int64_t rows = static_cast<int64_t>(p.max_q) * p.a.group;
  // the workspace query knows the longest sequence but no window: never more partials than it
  // counted
  const PagePlan plan = page_plan(p.a.S, p.a.D, rows, span), most = page_plan(p.a.S, p.a.D, rows, p.a.max_len);
  p.a.nsplit = std::min(plan.nsplit, most.nsplit);
  if (plan.blocks > 0 && most.blocks > 0 && p.a.nsplit > 1) {
    p.parts = reinterpret_cast<int32_t*>(p.a.ws + static_cast<int64_t>(p.num_tokens) * p.a.Hq * p.a.nsplit * (p.a.D + 2));
    p.blocks = plan.blocks;
    p.wave = plan.wave;
  }
  const cudaError_t e = p.a.D == 64    ? launch_query_pages_64(p, page_two(64, rows), s)
                        : p.a.D == 128 ? launch_query_pages_128(p, page_two(128, rows), s)
                                       : launch_query_pages_256(p, s);
  return e == cudaSuccess ? launch_query_merge_splits(p, s) : e;
}

size_t query_attn_workspace_bytes(int32_t S, int32_t num_tokens, int32_t H, int32_t Hq, int32_t D, int32_t max_q,
                                  int32_t max_len) {
  if (S <= 0 || num_tokens <= 0 || H <= 0 || Hq < H || D <= 0 || max_q <= 0 || max_len <= 0) return 0;
  if (max_q > max_len) max_q = max_len;  // as the call does
  // whichever kernel serves the call: the choice also depends on the pool
  const int64_t rows = static_cast<int64_t>(max_q) * (Hq / H);
  int n;
  if (rows >= kTileFrom) {
    n = tile_splits(S, H, D, rows, max_len);
  } else {
    n = row_splits(S, H, rows, max_len);
  }
  const size_t bytes = n <= 1 ? 0 : static_cast<size_t>(num_tokens) * Hq * n * (D + 2) * sizeof(float);
  return rows >= kTileFrom ? bytes : std::max(bytes, query_pages_workspace_bytes(S, num_tokens, Hq, D, rows, max_len));
}

cudaError_t launch_query_attention(const QueryAttnParams& p_in, cudaStream_t s) {
  QueryAttnParams p = p_in;
  const int rows = p.max_q * p.a.group;
  // tokens that a sequence's rows can see: less than all of them under a window (never more
  // splits than the workspace query counted, which knows the window not)
  const int64_t seen = static_cast<int64_t>(p.window) + p.max_q;
  const int32_t span = p.window > 0 && p.prefix == nullptr && seen < p.a.max_len ? static_cast<int32_t>(seen) : p.a.max_len;
  if (rows < kTileFrom) {
    if (query_pages_ok(p.a.block_size, p.a.H, p.a.k_page || p.a.v_page)) return launch_query_pages(p, span, s);
    p.a.nsplit = std::min(row_splits(p.a.S, p.a.H, rows, span), row_splits(p.a.S, p.a.H, rows, p.a.max_len));
    const cudaError_t e = p.a.D == 64    ? rows_dispatch<64>(p, rows, s)
                          : p.a.D == 128 ? rows_dispatch<128>(p, rows, s)
                                         : rows_dispatch<256>(p, rows, s);
    return e == cudaSuccess ? launch_query_merge_splits(p, s) : e;
  }
  p.a.nsplit = std::min(tile_splits(p.a.S, p.a.H, p.a.D, rows, span), tile_splits(p.a.S, p.a.H, p.a.D, rows, p.a.max_len));
  const cudaError_t e = launch_query_tiles(p, s);
  return e == cudaSuccess ? launch_query_merge_splits(p, s) : e;
}

}  // namespace kvq
