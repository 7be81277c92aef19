// query_page.cuh -- paged attention of up to 16 query rows per KV head and block, whole
// pages at a time: the page-major decode kernel's layout (attn_kernels.cu) with the rows, masks
// and logits of query_attn_kernels.cu.
//
// One block covers every KV head of one (split of the keys, 8 kNH rows, sequence).  A producer
// warp moves 16-token chunks of whole pages with bulk copies through a ring of stages; consumer
// warp w serves head w % H and chunk w / H of every stage with the shared tile arithmetic; the
// warps of one head merge through shared memory.  It serves block sizes that are multiples of
// 16 and H in {1, 2, 4, 8} (page-scaled planes from H = 4 on, whose H scales are one copy of
// 16 bytes at least).  H is a run-time value here: with a modifier between the products the
// strides' constants measured no gain, and there are a quarter of the instances.
//
// Bound: HBM with up to 8 rows a KV head and plain logits over FP8 planes (32 x 8192 tokens, 8 KV heads, 32 query
// heads, head_dim 128, page scales: 88.0 us, 6.12 TB/s, 90% of a plain copy's rate); issue and
// latency of a 16-token tile's arithmetic once options join in or the planes are NVFP4 (16 ragged sequences of up to 5000 tokens over
// NVFP4 with bias: 30.6 us, 2.0 TB/s; 32 of up to 4 draft tokens, capped, window 1024: 27.0 us).
// Blocks of every head and whole pages move 16 KB and more with one copy, where a block of one
// head would gather rows of 64 to 256 bytes (47 us for each of the last two).
#pragma once

#include "query_attn.cuh"

namespace kvq {

namespace {

// The job of block `cta` where sequences share the blocks by length: with T row tiles and w =
// (stages of its keys + 2 for a block's start) a sequence has T p blocks,
//   p = 1 + floor(w (n - sum T) / sum T w),
// at most a.nsplit and one for 64 keys; blocks go to the sequences in order.  n is one wave of
// blocks, or two where the longest share of one is above 1.3 times the mean by 4 stages and more (a
// second wave's starts and partials cost 12 to 19% on equal lengths of 3000).  One warp; its notes take
// 8 S bytes of shared memory.
struct PageJob {
  int s, tile, part, parts;  // parts 0: nothing to do
};
template <int kRows>
__device__ __forceinline__ PageJob page_job(const QueryAttnParams& qp, int lane, int unit, int cta, int2* note) {
  const int S = qp.a.S;
  auto sum = [](int64_t v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  };
  int64_t tiles = 0, work = 0;
#pragma unroll 4
  for (int s = lane; s < S; s += 32) {  // note: {w, T}
    int q0, n, len;
    int2 wt = make_int2(0, 0);
    if (query_range(qp, s, q0, n, len)) {
      wt.y = (n * qp.a.group + kRows - 1) / kRows;
      const int64_t near = static_cast<int64_t>(qp.window) + n;
      const int span = qp.window > 0 && qp.prefix == nullptr && near < len ? static_cast<int>(near) : len;
      wt.x = static_cast<int>((static_cast<uint32_t>(span) + unit - 1) / unit) + 2;
    } else if (cta == 0) {
      set_status(qp.a.status, 8u);
    }
    note[s] = wt;
    tiles += wt.y;
    work += static_cast<int64_t>(wt.x) * wt.y;
  }
  tiles = sum(tiles);
  work = max(sum(work), int64_t{1});
  int64_t spare = max(qp.wave - tiles, int64_t{0});
  float per_w = static_cast<float>(spare) / static_cast<float>(work);
  auto parts_of = [&](int2 wt) {
    // the quotient in 32 bits, at most one low or one high, then put right
    const int64_t all = wt.x * spare;
    int q = static_cast<int>(static_cast<float>(wt.x) * per_w);
    if (q * work > all) --q;
    if ((q + 1) * work <= all) ++q;
    const int most = static_cast<int>((static_cast<uint32_t>(wt.x - 2) * unit + 63u) / 64u);
    return max(1, min(min(most, qp.a.nsplit), 1 + q));
  };
  if (qp.blocks > qp.wave) {
    int longest = 0;
    for (int s = lane; s < S; s += 32) {
      const int2 wt = note[s];
      if (wt.y > 0) {
        const int n = parts_of(wt);
        longest = max(longest, (wt.x + n - 1) / n);
      }
    }
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    if (static_cast<float>(longest - 4) * static_cast<float>(qp.wave) > 1.3f * static_cast<float>(work)) {
      spare = max(qp.blocks - tiles, int64_t{0});
      per_w = static_cast<float>(spare) / static_cast<float>(work);
    }
  }
  int64_t before = 0;
  for (int s0 = 0; s0 < S; s0 += 32) {
    const int2 wt = s0 + lane < S ? note[s0 + lane] : make_int2(0, 0);
    const int parts = wt.y > 0 ? parts_of(wt) : 0;
    const int64_t mine = static_cast<int64_t>(wt.y) * parts;
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    const int64_t at = cta - before - (upto - mine);
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, at >= 0 && at < mine);
    if (hit != 0u) {
      const int src = __ffs(hit) - 1;
      const int off = __shfl_sync(0xFFFFFFFFu, static_cast<int>(at), src), n = __shfl_sync(0xFFFFFFFFu, parts, src);
      return PageJob{s0 + src, off / n, off % n, n};
    }
    before += __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  return PageJob{0, 0, 0, 0};
}

template <int D, int kFK, int kFV, int kNH>
struct QueryPage {
  static constexpr int kW = 8;
  static constexpr int kBlocks = D == 256 || kNH == 2 ? 1 : 2;
  static constexpr bool kQReg = kNH * (D / 16) <= 8;  // Q^T fragments in registers, else shared
  static constexpr int kFragBytes = kNH * (D / 16) * 32 * 8;  // of one head
  static constexpr int kQBytes = kQReg ? 0 : kW * kFragBytes;
  using Stage = PageStage<D, kFK, kFV, kW, kBlocks, kNH, kQBytes>;
  static constexpr int kOffQ = (Stage::kSmem + 15) / 16 * 16;
  static constexpr int kSmem = kOffQ + kQBytes;
};

template <int D, int kFK, int kFV, int kNH>
__global__ void __launch_bounds__(32 * (QueryPage<D, kFK, kFV, kNH>::kW + 1), QueryPage<D, kFK, kFV, kNH>::kBlocks)
    query_page_kernel(const QueryAttnParams qp) {
  using QP = QueryPage<D, kFK, kFV, kNH>;
  using T = typename QP::Stage;
  constexpr int W = QP::kW, kKS = D / 16, kMT = D / 16, kRows = 8 * kNH;
  constexpr bool kQReg = QP::kQReg;
  const AttnParams& p = qp.a;
  extern __shared__ __align__(128) unsigned char query_smem[];
  unsigned char* const smem = query_smem;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int H = p.H, P = W / H;
  __shared__ PageJob job;

  const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const uint32_t full0 = ring_s + T::kOffBar, empty0 = full0 + 8 * T::kStages;
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
  if (warp == W) {
    PageJob mine;
    if (qp.parts != nullptr) {
      mine = page_job<kRows>(qp, lane, 16 * P, blockIdx.x, reinterpret_cast<int2*>(smem));
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // its notes lie where copies will land
    } else {
      const int t = static_cast<int>(blockIdx.x) / p.nsplit;
      mine = PageJob{static_cast<int>(blockIdx.z), t, static_cast<int>(blockIdx.x) - t * p.nsplit, p.nsplit};
    }
    if (lane == 0) {
      job = mine;
      if (qp.parts != nullptr && mine.parts > 0 && mine.tile == 0 && mine.part == 0) STX(qp.parts + mine.s, mine.parts);
    }
  }
  __syncthreads();
  const int s = job.s, split = job.part, nsplit = job.parts;
  const int row0 = job.tile * kRows;
  if (nsplit == 0) return;

  int q0, nq, len;
  const bool ok = query_range(qp, s, q0, nq, len);
  if (!ok && threadIdx.x == 0 && blockIdx.x == 0) set_status(p.status, 8u);  // (page_job did it before)
  const int rows = nq * p.group;
  if (row0 >= rows) return;
  int lo, hi;
  lane_range(qp, lane, kRows, s, q0, nq, len, row0, rows, lo, hi);
  const int lo_min = __reduce_min_sync(0xFFFFFFFFu, lo), hi_max = __reduce_max_sync(0xFFFFFFFFu, hi);
  int t_begin = 0, t_end = 0;
  if (lo_min < hi_max) {  // equal splits in whole stages, from a chunk's start
    const int first = lo_min & ~15, unit = 16 * P;
    const int per = ((hi_max - first + nsplit - 1) / nsplit + unit - 1) / unit * unit;
    t_begin = static_cast<int>(min(static_cast<int64_t>(first) + static_cast<int64_t>(split) * per, static_cast<int64_t>(hi_max)));
    t_end = t_begin + min(per, hi_max - t_begin);
  }
  const int nstage = t_end > t_begin ? (t_end - t_begin + 16 * P - 1) / (16 * P) : 0;

  if (warp == W) {
    // ---- producer: lane j < P resolves chunk j of each stage, its table entry loaded a stage
    // ahead, and issues its copies ----
    bool timed_out = false, bad = false;
    const int32_t* const table = p.block_table + static_cast<int64_t>(s) * p.max_blocks;
    auto entry = [&](int k) -> int32_t {
      const int t0 = t_begin + 16 * (P * k + lane);
      return lane < P && t0 < t_end ? LDX(table + p.div_bs.div(static_cast<uint32_t>(t0))) : -1;
    };
    int32_t next = entry(0);
    for (int k = 0; k < nstage; ++k) {
      const int st = k % T::kStages;
      const int t0 = t_begin + 16 * (P * k + lane);
      const int64_t blk = next;
      next = entry(k + 1);
      bool have = false;
      int64_t r0 = 0;  // pool row (slot, head 0) of the chunk's first token
      if (lane < P && t0 < t_end) {
        if (blk < 0 || blk >= p.num_blocks) {
          bad = true;
        } else {
          uint32_t bi, bo;
          p.div_bs.divmod(static_cast<uint32_t>(t0), bi, bo);
          have = true;
          r0 = (blk * p.block_size + bo) * H;
        }
      }
      const uint32_t ksc = (p.k_page ? 4u : 64u) * H, vsc = (p.v_page ? 4u : 64u) * H;
      const uint32_t bytes = __reduce_add_sync(0xFFFFFFFFu, have ? 16u * H * (T::kRow - 8) + ksc + vsc : 0u);
      const bool any_bad = __any_sync(0xFFFFFFFFu, bad);
      if (k >= T::kStages && !mbar_wait(empty0 + 8 * st, ((k / T::kStages) - 1) & 1)) timed_out = true;
      const uint32_t gaps = __ballot_sync(0xFFFFFFFFu, lane < P && t0 < t_end && !have);
      if (gaps != 0u) {  // zeros where rows that do not see them meet them
        auto clear = [&](uint32_t at, uint32_t n) {
          for (uint32_t o = 16u * lane; o < n; o += 512u)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(ring_s + st * T::kBytes + at + o), "r"(0u) : "memory");
        };
        for (uint32_t left = gaps; left != 0u; left &= left - 1) {
          const uint32_t jr = 16u * H * (__ffs(left) - 1);
          clear(T::kOffKC + jr * T::kCK, 16u * H * T::kCK);
          clear(T::kOffVC + jr * T::kCV, 16u * H * T::kCV);
          clear(T::kOffKB + jr * T::kBK, 16u * H * T::kBK);
          clear(T::kOffVB + jr * T::kBV, 16u * H * T::kBV);
          clear(T::kOffKR + jr * 4, ksc);
          clear(T::kOffVR + jr * 4, vsc);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // copies land here later
        __syncwarp();
      }
      if (lane == 0) {
        if (any_bad) *bad_flag = 1;  // published by the arrival below
        mbar_arrive_expect_tx(full0 + 8 * st, bytes);
      }
      __syncwarp();
      if (have) {
        const uint32_t sb = ring_s + st * T::kBytes;
        const int jr = 16 * H * lane;
        const uint32_t full = full0 + 8 * st;
        bulk_copy_g2s(sb + T::kOffKC + jr * T::kCK, p.k.codes + r0 * T::kCK, 16u * H * T::kCK, full);
        bulk_copy_g2s(sb + T::kOffVC + jr * T::kCV, p.v.codes + r0 * T::kCV, 16u * H * T::kCV, full);
        if constexpr (T::kBK > 0) bulk_copy_g2s(sb + T::kOffKB + jr * T::kBK, p.k.bscale + r0 * T::kBK, 16u * H * T::kBK, full);
        if constexpr (T::kBV > 0) bulk_copy_g2s(sb + T::kOffVB + jr * T::kBV, p.v.bscale + r0 * T::kBV, 16u * H * T::kBV, full);
        bulk_copy_g2s(sb + T::kOffKR + jr * 4, p.k.rscale + (p.k_page ? blk * H : r0), ksc, full);
        bulk_copy_g2s(sb + T::kOffVR + jr * 4, p.v.rscale + (p.v_page ? blk * H : r0), vsc, full);
      }
    }
    const bool bad_any = __any_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      if (bad_any) set_status(p.status, 2u);
      if (timed_out) set_status(p.status, 16u);
    }
    return;  // the consumers' barriers leave this warp out
  }

  // ---- consumers ----
  const int h = warp % H, j = warp / H;
  uint2* const qfrag = reinterpret_cast<uint2*>(smem + QP::kOffQ + h * QP::kFragBytes);
  uint2 qreg[kQReg ? kNH : 1][kKS];
  float row_fac[kNH];
#pragma unroll
  for (int nh = 0; nh < kNH; ++nh) {
    uint2(&f)[kKS] = qreg[kQReg ? nh : 0];
    row_fac[nh] = query_fragments<D>(p, lane, h, q0, row0 + 8 * nh + g, rows, f);
    if (!kQReg && j == 0) {
#pragma unroll
      for (int kb = 0; kb < kKS; ++kb) qfrag[(nh * kKS + kb) * 32 + lane] = f[kb];
    }
  }
  __shared__ __align__(16) typename QueryMod<kNH>::Tables tab;
  QueryMod<kNH>::fill(&tab, qp, lane, h, h, row0, rows, lo, hi, warp == 0, j == 0);
  asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory");
  QueryMod<kNH> mod;
  float qmul[kNH][2];
  mod.init(&tab, qp, lane, h, row0, rows, len - nq, lo, hi, row_fac, qmul);
  auto qb = [&](int nh, int kb) -> uint2 {
    if constexpr (kQReg) {
      return qreg[nh][kb];
    } else {
      return qfrag[(nh * kKS + kb) * 32 + lane];
    }
  };

  AttnState<D, kNH> st;
  st.init(kNoKey);
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
                        H * T::kCK, H * T::kCV, H * T::kBK, H * T::kBV, p.k_page ? 0 : H * 4, p.v_page ? 0 : H * 4};
      mod.t0 = t0;
      attn_tile<D, kFK, kFV, kNH>(tv, qb, qmul, lane, t_end - t0, st, mod, lo_min - t0);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8 * stg);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll
  for (int off = 4; off <= 16; off <<= 1)
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh) {
      st.l[nh][0] += __shfl_xor_sync(0xFFFFFFFFu, st.l[nh][0], off);
      st.l[nh][1] += __shfl_xor_sync(0xFFFFFFFFu, st.l[nh][1], off);
    }
  if (__any_sync(0xFFFFFFFFu, timed_out) && lane == 0) set_status(p.status, 16u);
  // visible: set before the arrival of a stage this warp has waited for
  const bool cta_bad = *bad_flag != 0;

#pragma unroll
  for (int q = 0; q < kMT; ++q)
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[q][nh][e] *= st.R;
  if (P > 1) {
    asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory");  // the ring is free
    constexpr int kLane = T::kLaneFloats / kNH;  // floats of one n-tile
    float* const mine = reinterpret_cast<float*>(smem) + (warp * 32 + lane) * T::kLaneFloats;
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh) {
#pragma unroll
      for (int q = 0; q < kMT; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) mine[nh * kLane + 4 * q + e] = st.o[q][nh][e];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mine[nh * kLane + 4 * kMT + e] = st.m[nh][e];
        mine[nh * kLane + 4 * kMT + 2 + e] = st.l[nh][e];
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory");
    if (j != 0) return;
    const float* const all = reinterpret_cast<const float*>(smem);
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh) {
      float Mn[2] = {st.m[nh][0], st.m[nh][1]};
      for (int jj = 1; jj < P; ++jj) {
        const float* const o = all + ((jj * H + h) * 32 + lane) * T::kLaneFloats + nh * kLane;
        Mn[0] = fmaxf(Mn[0], o[4 * kMT]);
        Mn[1] = fmaxf(Mn[1], o[4 * kMT + 1]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float f = ex2(st.m[nh][e] - Mn[e]);
        st.l[nh][e] *= f;
        st.m[nh][e] = Mn[e];
#pragma unroll
        for (int q = 0; q < kMT; ++q) {
          st.o[q][nh][e] *= f;
          st.o[q][nh][e + 2] *= f;
        }
      }
      for (int jj = 1; jj < P; ++jj) {
        const float* const o = all + ((jj * H + h) * 32 + lane) * T::kLaneFloats + nh * kLane;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = ex2(o[4 * kMT + e] - Mn[e]);
          st.l[nh][e] = __fmaf_rn(o[4 * kMT + 2 + e], f, st.l[nh][e]);
#pragma unroll
          for (int q = 0; q < kMT; ++q) {
            st.o[q][nh][e] = __fmaf_rn(o[4 * q + e], f, st.o[q][nh][e]);
            st.o[q][nh][e + 2] = __fmaf_rn(o[4 * q + e + 2], f, st.o[q][nh][e + 2]);
          }
        }
      }
    }
  }
  uint32_t bad_rows = 0;
  if (cta_bad) {
    for (int r = 0; r < min(kRows, rows - row0); ++r)
      if (needs_bad_block(p, s, max(tab.range[r].x, t_begin), min(tab.range[r].y, t_end))) bad_rows |= 1u << r;
  }
  // rows 8 nh + 2c + e; dims g*D/8 + 2q and + 1
#pragma unroll
  for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = row0 + 8 * nh + 2 * c + e;
      if (row >= rows) continue;
      const int i = row / p.group, qh = h * p.group + row - i * p.group;
      const int64_t tok = q0 + i;
      const float L = st.l[nh][e];
      const bool bad = ((bad_rows >> (8 * nh + 2 * c + e)) & 1u) != 0u;
      if (nsplit == 1) {
        if (bad) continue;
        uint16_t* const out = p.out + tok * p.o_row_pitch + static_cast<int64_t>(qh) * p.o_head_pitch;
#pragma unroll
        for (int q = 0; q < kMT; ++q) {
          const float y0 = L == 0.0f ? 0.0f : st.o[q][nh][e] / L, y1 = L == 0.0f ? 0.0f : st.o[q][nh][e + 2] / L;
          STX(reinterpret_cast<uint32_t*>(out + g * (D / 8) + 2 * q), pack_bf16x2(y0, y1));
        }
      } else {
        float* const wsr = p.ws + ((tok * p.Hq + qh) * p.nsplit + split) * (D + 2);
#pragma unroll
        for (int q = 0; q < kMT; ++q)
          STX(reinterpret_cast<float2*>(wsr + g * (D / 8) + 2 * q), make_float2(st.o[q][nh][e], st.o[q][nh][e + 2]));
        if (g == 0)  // a NaN M marks a bad block entry
          STX(reinterpret_cast<float2*>(wsr + D), make_float2(bad ? __int_as_float(0x7FC00000) : st.m[nh][e], L));
      }
    }
}

template <int D, int kFK, int kFV, int kNH>
cudaError_t query_page_launch(const QueryAttnParams& p, cudaStream_t s) {
  using QP = QueryPage<D, kFK, kFV, kNH>;
  auto k = query_page_kernel<D, kFK, kFV, kNH>;
  static_assert(QP::kSmem <= 227 * 1024 && QP::Stage::kStages >= 2, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, QP::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (static_cast<int64_t>(p.max_q) * p.a.group + 8 * kNH - 1) / (8 * kNH);
  const dim3 grid(p.parts != nullptr ? p.blocks : static_cast<unsigned>(tiles * p.a.nsplit), 1, p.parts != nullptr ? 1 : p.a.S);
  KVQ_LAUNCH("query_page_kernel", s, k<<<grid, 32 * (QP::kW + 1), QP::kSmem, s>>>(p); e = cudaGetLastError());
  return e;
}

template <int D, int kNH>
cudaError_t query_page_fmt(const QueryAttnParams& p, cudaStream_t s) {
  const bool k8 = p.a.fmt_k == 3, v8 = p.a.fmt_v == 3;
  if (!k8 && !v8) return query_page_launch<D, 1, 1, kNH>(p, s);
  if (k8 && !v8) return query_page_launch<D, 3, 1, kNH>(p, s);
  if (!k8 && v8) return query_page_launch<D, 1, 3, kNH>(p, s);
  return query_page_launch<D, 3, 3, kNH>(p, s);
}

}  // namespace

}  // namespace kvq
