// select_kernels.cu -- for each query token and KV head, the blocks of a paged cache with the
// highest bound on a score.
//
// With the g query heads of a KV head and lo_b, hi_b the least and the largest keys of block b,
// channel by channel,
//   q+ = sum_g max(q_g, 0),  q- = sum_g min(q_g, 0),  score(b) = q+ . hi_b + q- . lo_b,
// which no key t of the block exceeds: score(b) >= sum_g q_g . k_t.  One dot product of 2 D values
// serves all heads of the group.  The `first` first and `last` last blocks up to the query's own are
// listed in any case, then the highest scores up to `topk` blocks, ties to the lowest index.
//
// The list is that of the exact scores.  The score kernels work in binary32; their roundings stay
// within e = err * a, a = sum_d (|q+_d| max |hi_d| + |q-_d| max |lo_d|) (err counts them; the maxima
// are over the row's blocks).  A score above the best unlisted one by more than 2 e is listed for
// certain, one below the lowest listed one by as much is not; what lies between is scored again, by
// one warp a block: a few blocks in pairs of binary32 numbers (one row in eight has two or three; on this
// GPU binary64 runs at two operations a cycle and SM, and took 6 us of such a call), more than 32, or what
// binary32 cannot bound (sums that may overflow), in binary64 and ranked by the upper and then the lower
// bits of that.  Exact ties go the same way to the index.
//
// Both score kernels take the dot products on the tensor cores, q split into bf16 parts: with the blocks
// as rows and the parts as columns for few queries a sequence (score_kernel; bound: HBM), by tiles of 64
// queries and 128 blocks from kTileQueries on (score_tile_kernel).
#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_params.h"

namespace kvq {

namespace {

// Keys: scores in the order of unsigned integers; below them what has none.
constexpr uint32_t kKeyBad = 1u;  // a table entry outside the pool
constexpr uint32_t kKeyNan = 2u;
constexpr uint32_t kKeyNan64 = 3u;          // of the second scores, which begin above it
constexpr uint32_t kKeyListed = 0xFFFFFFFEu;  // listed for certain
__device__ __forceinline__ uint32_t score_key(float x) {
  if (isnan(x)) return kKeyNan;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 as 0
  return (u & 0x80000000u) != 0u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) != 0u ? k & 0x7FFFFFFFu : ~k);
}

constexpr int kScoreQueries = 8;  // of a sequence, at most; more go to the tile kernel
constexpr int kTileQueries = kScoreQueries + 1;

// The score kernel's shared memory, for hc KV heads a thread block: stages of 16 `part` blocks of the
// cache (rows of the heads' bounds, 16 bytes apart: conflict-free ldmatrix), q as operand fragments, a
// row of zeros, the warps' sizes.
template <int D>
constexpr int kScoreWarps = D == 256 ? 4 : 8;  // and one that copies
struct ScorePlan {
  int hc, part, row, stage, stages, groups, frag, smem;
  __host__ __device__ ScorePlan(int H, int D, int max_q) {
    const int warps = D == 256 ? 4 : 8;
    hc = H < warps ? H : warps;
    part = warps / hc;  // warps of a head
    row = hc * 4 * D + 16;
    stage = 16 * part * row;
    groups = max_q <= 4 ? 1 : 2;  // of 8 operand columns: 2 queries in three parts, or 4 in two
    frag = hc * groups * (D / 8) * 256;
    const int rest = 4 * D + warps * kScoreQueries * 4;
    stages = (227 * 1024 - 512 - frag - rest) / stage;
    if (stages > 6) stages = 6;
    smem = stages * stage + frag + rest;
  }
};

// First query token and number of query tokens of sequence s (see query_range, query_attn.cuh).
__device__ __forceinline__ bool select_range(const SelectParams& p, int s, int& q0, int& n, int& len) {
  len = LDX(p.seq_lens + s);
  q0 = LDX(p.starts + s);
  const int q1 = LDX(p.starts + s + 1);
  n = 0;
  if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || q1 - q0 > p.max_q || len < 0 || len > p.seq_cap || q1 - q0 > len)
    return false;
  n = q1 - q0;
  return true;
}

// Sums over the heads of one token's q- and q+ at channels d .. d + 7.
__device__ __forceinline__ void sum_heads(const SelectParams& p, int tok, int h, int d, float (&minus)[8], float (&plus)[8]) {
  const uint16_t* const x = p.q + tok * p.q_row_pitch + static_cast<int64_t>(h) * p.group * p.q_head_pitch + d;
#pragma unroll
  for (int i = 0; i < 8; ++i) minus[i] = plus[i] = 0.0f;
#pragma unroll 1
  for (int j0 = 0; j0 < p.group; j0 += 8) {  // 8 heads' loads at a time: the loop waits for memory
    uint32_t v[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0u;
      if (j0 + j < p.group) load16B(x + (j0 + j) * p.q_head_pitch, v[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = i % 2 == 0 ? bf16lo(v[j][i / 2]) : bf16hi(v[j][i / 2]);
        minus[i] = __fadd_rn(minus[i], y > 0.0f ? 0.0f : y);  // a NaN goes on
        plus[i] = __fadd_rn(plus[i], y > 0.0f ? y : 0.0f);
      }
  }
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Scores of a segment of a sequence's blocks for up to 8 KV heads and up to 8 query tokens.  A producer
// warp copies the heads' bounds of whole blocks (one run of memory each) through a ring of stages;
// consumer warp w serves head w % hc and 16 blocks of a stage: mma.sync m16n8k16 with the blocks as rows
// and the queries as columns, q+ and q- in three bf16 parts (q exactly, up to 2 queries) or two (what
// is left below 2^-18 of it), a column each.  The products of a step of 16 channels are added up by the
// tensor cores, the steps in binary32 registers, which keeps the bound on the roundings 16 times
// smaller than one chain would.  (Dot products by FMA, 8 blocks a warp and a reduction over its
// lanes, took 73 us of 32 x 2048 blocks and 8 heads at head_dim 128, the copies alone 44.)
template <int D>
__global__ void __launch_bounds__(32 * (kScoreWarps<D> + 1), 1) score_kernel(const SelectParams p) {
  constexpr int kW = kScoreWarps<D>, kSteps = 2 * D / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[2][6];
  __shared__ uint32_t have[6][4];  // bit j of [x]: block 32 x + j of the stage has bounds
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int segment = blockIdx.x, s = blockIdx.z;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int q0, n, len;
  if (!select_range(p, s, q0, n, len) || n == 0) return;
  const int blocks = static_cast<int>(p.div_bs.div(static_cast<uint32_t>(len - 1))) + 1;
  if (blocks <= p.topk) return;
  const ScorePlan plan(p.H, D, p.max_q);
  const bool three = p.max_q <= 2;
  const int h0 = static_cast<int>(blockIdx.y) * plan.hc, hn = min(plan.hc, p.H - h0);  // heads h0 .. h0 + hn - 1
  // equal segments in groups of 16 blocks; a stage takes `part` of them
  const int groups = (blocks + 15) / 16, per = (groups + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  const int first = 16 * min(segment * per, groups), last = min(blocks, first + 16 * per);
  const int stage_blocks = 16 * plan.part, count = first < last ? (last - first + stage_blocks - 1) / stage_blocks : 0;
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const uint32_t full0 = static_cast<uint32_t>(__cvta_generic_to_shared(&bars[0][0]));
  const uint32_t empty0 = static_cast<uint32_t>(__cvta_generic_to_shared(&bars[1][0]));
  unsigned char* const frag = smem + plan.stages * plan.stage;  // [head][column group][step][lane] {k 2c, 2c + 1 | + 8, + 9}
  const int off_zero = plan.stages * plan.stage + plan.frag;
  if (threadIdx.x == 0) {
    for (int st = 0; st < plan.stages; ++st) {
      mbar_init(full0 + 8 * st, 1);
      mbar_init(empty0 + 8 * st, kW);
    }
    mbar_init_fence();
  }
  __syncthreads();
  bool timed_out = false;
  if (warp == kW) {
    // ---- producer: lanes take a stage's blocks, whose table entries are loaded a stage ahead ----
    constexpr int kX = kW / 2;  // 16 kW blocks at most
    const uint32_t bytes = 4u * D * hn;
    auto entry = [&](int k, int x) -> int32_t {
      const int j = 32 * x + lane, b = first + k * stage_blocks + j;
      return j < stage_blocks && b < last ? LDX(p.table + static_cast<int64_t>(s) * p.max_blocks + b) : -1;
    };
    int32_t next[kX];
#pragma unroll
    for (int x = 0; x < kX; ++x) next[x] = entry(0, x);
    int st = 0, turn = 0;
    for (int k = 0; k < count; ++k) {
      int64_t blk[kX];
      uint32_t ok[kX], sum = 0u;
#pragma unroll
      for (int x = 0; x < kX; ++x) {
        const int j = 32 * x + lane;
        blk[x] = next[x] >= 0 && next[x] < p.num_blocks ? next[x] : -1;
        const bool in = j < stage_blocks && first + k * stage_blocks + j < last;
        if (__any_sync(0xFFFFFFFFu, in && blk[x] < 0) && lane == 0) set_status(p.status, 2u);
        ok[x] = __ballot_sync(0xFFFFFFFFu, blk[x] >= 0);
        sum += __popc(ok[x]);
        next[x] = entry(k + 1, x);
      }
      if (k >= plan.stages && !mbar_wait(empty0 + 8 * st, turn ^ 1)) timed_out = true;
      if (lane == 0) {
#pragma unroll
        for (int x = 0; x < kX; ++x) have[st][x] = ok[x];  // published by the arrival
        mbar_arrive_expect_tx(full0 + 8 * st, bytes * sum);
      }
      __syncwarp();
#pragma unroll
      for (int x = 0; x < kX; ++x)
        if (blk[x] >= 0)
          bulk_copy_g2s(base + st * plan.stage + (32 * x + lane) * plan.row, p.bounds + (blk[x] * p.H + h0) * (2 * D), bytes,
                        full0 + 8 * st);
      if (++st == plan.stages) {
        st = 0;
        turn ^= 1;
      }
    }
    if (__any_sync(0xFFFFFFFFu, timed_out) && lane == 0) set_status(p.status, 16u);
    return;  // the others' barriers leave this warp out
  }
  auto together = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * kW) : "memory"); };
  for (int at = threadIdx.x; at < (plan.frag + 4 * D) / 16; at += 32 * kW)
    reinterpret_cast<uint4*>(frag)[at] = make_uint4(0u, 0u, 0u, 0u);
  together();
  for (int at = threadIdx.x; at < n * hn * (D / 8); at += 32 * kW) {
    const int d = 8 * (at % (D / 8)), ih = at / (D / 8), i = ih / hn, h = ih - i * hn;
    float v[2][8];  // q-, q+
    sum_heads(p, q0 + i, h0 + h, d, v[0], v[1]);
    const int col = three ? 4 * (i % 2) : 2 * (i % 4), group = three ? i / 2 : i / 4;
    unsigned char* const to = frag + (h * plan.groups + group) * (kSteps * 256);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = j * D + d;
      unsigned char* const at_k = to + (k / 16) * 256 + (k % 16 / 8) * 4;
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        if (part == 2 && !three) break;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t w = pack_bf16x2(v[j][2 * x], v[j][2 * x + 1]);
          v[j][2 * x] = __fsub_rn(v[j][2 * x], bf16lo(w));
          v[j][2 * x + 1] = __fsub_rn(v[j][2 * x + 1], bf16hi(w));
          *reinterpret_cast<uint32_t*>(at_k + ((col + part) * 4 + x) * 8) = w;
        }
      }
    }
  }
  together();
  const int h = warp % plan.hc, part = warp / plan.hc, g = lane >> 2, c = lane & 3;
  const bool works = h < hn && part < plan.part;
  const bool two = plan.groups == 2;
  const uint2* const q_at = reinterpret_cast<const uint2*>(frag + h * plan.groups * (kSteps * 256)) + lane;
  uint32_t top[kSteps][2] = {};  // largest |bound| of the lane's channels, packed
  int st = 0, turn = 0;
#pragma unroll 1
  for (int k = 0; k < count; ++k) {
    if (!mbar_wait(full0 + 8 * st, turn)) timed_out = true;
    const int b0 = first + k * stage_blocks + 16 * part;
    if (works && b0 < last) {  // the same in the whole warp
      const uint32_t here = have[st][part / 2] >> (16 * (part % 2)) & 0xFFFFu;
      const int r = lane & 15;
      const uint32_t at = base + (lane >> 4) * 16 +
                          ((here >> r) & 1u ? st * plan.stage + (16 * part + r) * plan.row + h * 4 * D : off_zero);
      float acc[2][4] = {};
#pragma unroll
      for (int t = 0; t < kSteps; ++t) {
        uint32_t a[4];
        ldmatrix_x4(a, at + 32 * t);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(top[t][x / 2]) : "r"(top[t][x / 2]), "r"(a[x]));
        const uint2 b = q_at[t * 32];
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        mma_bf16_16816(d, a, b.x, b.y);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][e] = __fadd_rn(acc[0][e], d[e]);
        if (two) {
          const uint2 b2 = q_at[(kSteps + t) * 32];
          float d2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_bf16_16816(d2, a, b2.x, b2.y);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[1][e] = __fadd_rn(acc[1][e], d2[e]);
        }
      }
#pragma unroll
      for (int gr = 0; gr < 2; ++gr) {
        if (gr == 1 && !two) break;
        float v[2] = {__fadd_rn(acc[gr][0], acc[gr][1]), __fadd_rn(acc[gr][2], acc[gr][3])};  // rows g, g + 8
        int i = 4 * gr + c;
        if (three) {
          v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 1));
          v[1] = __fadd_rn(v[1], __shfl_xor_sync(0xFFFFFFFFu, v[1], 1));
          i = c / 2;
        }
        uint32_t* const to = p.keys + (static_cast<int64_t>(q0 + i) * p.H + h0 + h) * p.pitch + b0 + g;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (i < n && b0 + g + 8 * e < last && !(three && e != (c & 1)))
            STX(to + 8 * e, (here >> (g + 8 * e)) & 1u ? score_key(v[e]) : kKeyBad);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8 * st);
    if (++st == plan.stages) {
      st = 0;
      turn ^= 1;
    }
  }
  // ---- sizes: sum_d |q_d| top_d.  Lanes of one c hold the same channels: their maxima, then lane g
  // adds up query g's.  2^-100 on both sides covers what the tensor cores may take for zero (subnormal
  // parts); 0 only for a query of zeros.  A NaN in q would make the size one (those of the bounds do not count
  // in top); fmaxf makes it 2^-149, which does no harm: all of that query's scores are NaN, in any precision.
  float* const sizes = reinterpret_cast<float*>(smem + off_zero + 4 * D);  // [warp][query]
  float size = 0.0f;
  bool none = true;
  const int col = three ? 4 * (g % 2) : 2 * (g % 4), group = three ? g / 2 : g / 4;
  const uint2* const mine = reinterpret_cast<const uint2*>(frag + (h * plan.groups + (group < plan.groups ? group : 0)) * (kSteps * 256)) +
                            col * 4 + c;
#pragma unroll
  for (int t = 0; t < kSteps; ++t) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t m = top[t][x];
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) {
        const uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, m, o);
        asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(y));
      }
      const uint32_t w = x == 0 ? mine[t * 32].x : mine[t * 32].y;
      none = none && (w & 0x7FFF7FFFu) == 0u;
      size += (fabsf(bf16lo(w)) * 1.01f + 0x1p-100f) * (fabsf(bf16lo(m)) + 0x1p-100f);
      size += (fabsf(bf16hi(w)) * 1.01f + 0x1p-100f) * (fabsf(bf16hi(m)) + 0x1p-100f);
    }
  }
  if (!works || g >= n) none = true;
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    size += __shfl_xor_sync(0xFFFFFFFFu, size, o);
    none = __shfl_xor_sync(0xFFFFFFFFu, none ? 1 : 0, o) != 0 && none;
  }
  if (c == 0) sizes[warp * kScoreQueries + g] = none ? 0.0f : fmaxf(size, 0x1p-149f);
  together();
  for (int at = threadIdx.x; at < n * hn; at += 32 * kW) {
    const int i = at / hn, hh = at - i * hn;
    float a = 0.0f;
    for (int x = 0; x < plan.part; ++x) a = fmaxf(a, sizes[(x * plan.hc + hh) * kScoreQueries + i]);
    STX(p.sizes + (static_cast<int64_t>(q0 + i) * p.H + h0 + hh) * p.sizes_pitch + segment, a);
  }
  if (__any_sync(0xFFFFFFFFu, timed_out) && lane == 0) set_status(p.status, 16u);
}

// The same by tiles of kM queries and kN blocks: mma.sync m16n8k16 over 2 D channels, q = hi + lo in
// bf16 (rest below 2^-18 of it), the bounds as they are.  The products of a step of 16 channels are
// added up by the tensor cores, the steps in binary32 registers, which keeps the bound on the
// roundings 16 times smaller than one chain would.  A block takes a segment of the sequence's blocks:
// q is split once, tiles of bounds follow through two stages of bulk copies.
template <int D>
struct ScoreTile {
  static constexpr int kM = D == 256 ? 32 : 64, kN = D == 256 ? 64 : 128;
  static constexpr int kPitch = 4 * D + 16;  // bytes of a row (conflict-free ldmatrix)
  static constexpr int kOffLo = kM * kPitch;
  static constexpr int kOffB = 2 * kM * kPitch;
  static constexpr int kStage = kN * kPitch;
  static constexpr int kOffTop = kOffB + 2 * kStage;  // largest |bound| of each channel, f32
  static constexpr int kSmem = kOffTop + 2 * D * 4;
  static constexpr int kWarps = D == 256 ? 8 : 16;  // 2 by kWarps / 2 over the tile; and one that copies
};

template <int D>
__global__ void __launch_bounds__(32 * (ScoreTile<D>::kWarps + 1), 1) score_tile_kernel(const SelectParams p) {
  using T = ScoreTile<D>;
  constexpr int kMT = T::kM / 32, kNT = T::kN / (4 * T::kWarps), kThreads = 32 * T::kWarps;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[4];  // full and empty, a stage each
  __shared__ uint32_t have[2][T::kN / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int qt = static_cast<int>(blockIdx.x) / p.H, h = static_cast<int>(blockIdx.x) - qt * p.H, s = blockIdx.z;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int q0, n, len;
  if (!select_range(p, s, q0, n, len) || qt * T::kM >= n) return;
  const int nq = min(T::kM, n - qt * T::kM), tok0 = q0 + qt * T::kM;
  // blocks that this tile's last query sees
  const int blocks = static_cast<int>(p.div_bs.div(static_cast<uint32_t>(len - n + qt * T::kM + nq - 1))) + 1;
  const int first = static_cast<int>(blockIdx.y) * p.segment;
  if (blocks <= p.topk) return;
  if (first >= blocks) {  // nothing of this segment: nothing to round
    for (int i = threadIdx.x; i < nq; i += static_cast<int>(blockDim.x))
      STX(p.sizes + (static_cast<int64_t>(tok0 + i) * p.H + h) * p.sizes_pitch + blockIdx.y, 0.0f);
    return;
  }
  const int last = min(blocks, first + p.segment), tiles = (last - first + T::kN - 1) / T::kN;
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const uint32_t full0 = static_cast<uint32_t>(__cvta_generic_to_shared(bars)), empty0 = full0 + 16;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      mbar_init(full0 + 8 * st, 1);
      mbar_init(empty0 + 8 * st, T::kWarps);
    }
    mbar_init_fence();
  }
  __syncthreads();
  bool timed_out = false;
  if (warp == T::kWarps) {
    // ---- producer: a tile's table entries are loaded while the one before it is copied ----
    constexpr int kX = T::kN / 32;
    auto entry = [&](int t, int x) -> int32_t {
      const int b = first + t * T::kN + 32 * x + lane;
      return b < last ? LDX(p.table + static_cast<int64_t>(s) * p.max_blocks + b) : -1;
    };
    int32_t next[kX];
#pragma unroll
    for (int x = 0; x < kX; ++x) next[x] = entry(0, x);
    for (int t = 0; t < tiles; ++t) {
      const int st = t & 1;
      int64_t blk[kX];
      uint32_t ok[kX], count = 0u;
#pragma unroll
      for (int x = 0; x < kX; ++x) {
        blk[x] = next[x] >= 0 && next[x] < p.num_blocks ? next[x] : -1;
        if (__any_sync(0xFFFFFFFFu, blk[x] < 0 && first + t * T::kN + 32 * x + lane < last) && lane == 0)
          set_status(p.status, 2u);
        ok[x] = __ballot_sync(0xFFFFFFFFu, blk[x] >= 0);
        count += __popc(ok[x]);
        next[x] = entry(t + 1, x);
      }
      if (t >= 2 && !mbar_wait(empty0 + 8 * st, ((t >> 1) - 1) & 1)) timed_out = true;
      if (lane == 0) {
#pragma unroll
        for (int x = 0; x < kX; ++x) have[st][x] = ok[x];  // published by the arrival
        mbar_arrive_expect_tx(full0 + 8 * st, count * 4u * D);
      }
      __syncwarp();
#pragma unroll
      for (int x = 0; x < kX; ++x) {
        const uint32_t at = base + T::kOffB + st * T::kStage + (32 * x + lane) * T::kPitch;
        if (blk[x] >= 0) bulk_copy_g2s(at, p.bounds + (blk[x] * p.H + h) * (2 * D), 4u * D, full0 + 8 * st);
      }
    }
    if (__any_sync(0xFFFFFFFFu, timed_out) && lane == 0) set_status(p.status, 16u);
    return;  // the others' barriers leave this warp out
  }
  auto together = [] { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); };
  for (int at = threadIdx.x; at < T::kM * (D / 8); at += kThreads) {
    const int i = at / (D / 8), d = 8 * (at - i * (D / 8));
    float v[2][8];  // q-, q+
    if (i < nq) {
      sum_heads(p, tok0 + i, h, d, v[0], v[1]);
    } else {
#pragma unroll
      for (int x = 0; x < 8; ++x) v[0][x] = v[1][x] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float a = v[j][2 * x], b = v[j][2 * x + 1];
        hi[x] = pack_bf16x2(a, b);
        lo[x] = pack_bf16x2(__fsub_rn(a, bf16lo(hi[x])), __fsub_rn(b, bf16hi(hi[x])));
      }
      unsigned char* const row = smem + i * T::kPitch + 2 * (j * D + d);
      *reinterpret_cast<uint4*>(row) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(row + T::kOffLo) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  together();

  const int m0 = (warp & 1) * (T::kM / 2), n0 = (warp >> 1) * (8 * kNT);
  const uint32_t a_at = base + (m0 + (lane & 15)) * T::kPitch + (lane >> 4) * 16;
  const uint32_t b_row = (n0 + (lane & 7) + ((lane >> 4) << 3)) * T::kPitch + ((lane >> 3) & 1) * 16;
  uint32_t top[2 * D / kThreads > 0 ? 2 * D / kThreads : 1] = {};
  constexpr int kWords = D;  // of a row
  for (int t = 0; t < tiles; ++t) {
    const int st = t & 1;
    if (!mbar_wait(full0 + 8 * st, (t >> 1) & 1)) timed_out = true;
    const unsigned char* const tile = smem + T::kOffB + st * T::kStage;
    // rows without bounds: zeros, which no copy writes
    uint32_t gaps = 0u;
#pragma unroll
    for (int x = 0; x < T::kN / 32; ++x) gaps |= ~have[st][x];
    if (gaps != 0u) {
      for (int at = threadIdx.x; at < T::kN * (D / 4); at += kThreads) {
        const int r = at / (D / 4), x = at - r * (D / 4);
        if (((have[st][r / 32] >> (r % 32)) & 1u) == 0u)
          *reinterpret_cast<uint4*>(smem + T::kOffB + st * T::kStage + r * T::kPitch + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // copies land here later
      together();
    }
    float acc[kMT][kNT][4];
#pragma unroll
    for (int a = 0; a < kMT; ++a)
#pragma unroll
      for (int b = 0; b < kNT; ++b) acc[a][b][0] = acc[a][b][1] = acc[a][b][2] = acc[a][b][3] = 0.0f;
    const uint32_t b_at = base + T::kOffB + st * T::kStage + b_row;
#pragma unroll 2
    for (int k = 0; k < 2 * D / 16; ++k) {
      uint32_t hi[kMT][4], lo[kMT][4], bb[kNT / 2][4];
#pragma unroll
      for (int a = 0; a < kMT; ++a) {
        ldmatrix_x4(hi[a], a_at + a * 16 * T::kPitch + 32 * k);
        ldmatrix_x4(lo[a], a_at + T::kOffLo + a * 16 * T::kPitch + 32 * k);
      }
#pragma unroll
      for (int b = 0; b < kNT / 2; ++b) ldmatrix_x4(bb[b], b_at + b * 16 * T::kPitch + 32 * k);
      float step[kMT][kNT][4];  // chains of two, as many at a time as there are
#pragma unroll
      for (int a = 0; a < kMT; ++a)
#pragma unroll
        for (int b = 0; b < kNT; ++b) {
          step[a][b][0] = step[a][b][1] = step[a][b][2] = step[a][b][3] = 0.0f;
          mma_bf16_16816(step[a][b], lo[a], bb[b / 2][2 * (b % 2)], bb[b / 2][2 * (b % 2) + 1]);
        }
#pragma unroll
      for (int a = 0; a < kMT; ++a)
#pragma unroll
        for (int b = 0; b < kNT; ++b) mma_bf16_16816(step[a][b], hi[a], bb[b / 2][2 * (b % 2)], bb[b / 2][2 * (b % 2) + 1]);
#pragma unroll
      for (int a = 0; a < kMT; ++a)
#pragma unroll
        for (int b = 0; b < kNT; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[a][b][e] = __fadd_rn(acc[a][b][e], step[a][b][e]);
    }
    // largest |bound| of each channel: thread x has words x, x + kThreads
#pragma unroll
    for (int x = 0; x < (kWords + kThreads - 1) / kThreads; ++x) {
      const int word = threadIdx.x % kWords + x * kThreads, r0 = threadIdx.x / kWords;
      constexpr int kShare = kThreads > kWords ? kThreads / kWords : 1;  // threads of a word
#pragma unroll 8
      for (int r = r0; r < T::kN; r += kShare)
        asm("max.xorsign.abs.bf16x2 %0, %1, %2;"
            : "=r"(top[x])
            : "r"(top[x]), "r"(*reinterpret_cast<const uint32_t*>(tile + r * T::kPitch + 4 * word)));
    }
    const int g = lane >> 2, c = lane & 3, col0 = n0 + 2 * c, left = last - (first + t * T::kN);
    uint32_t* const to = p.keys + (static_cast<int64_t>(tok0 + m0 + g) * p.H + h) * p.pitch + first + t * T::kN;
    const int64_t rows8 = static_cast<int64_t>(8 * p.H) * p.pitch;
#pragma unroll
    for (int b = 0; b < kNT; ++b) {
      const int col = col0 + 8 * b;
      const uint32_t ok = have[st][col / 32] >> (col % 32);
#pragma unroll
      for (int a = 0; a < kMT; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (m0 + 16 * a + g + 8 * e >= nq || col >= left) continue;
          uint2 v = make_uint2(score_key(acc[a][b][2 * e]), score_key(acc[a][b][2 * e + 1]));
          if ((ok & 3u) != 3u) v = make_uint2(ok & 1u ? v.x : kKeyBad, ok & 2u ? v.y : kKeyBad);
          STX(reinterpret_cast<uint2*>(to + (2 * a + e) * rows8 + col), v);  // pitch is even: the pair lies in the row
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8 * st);  // this warp has read the stage, and its notes
  }
  // ---- sizes: sum_d |q_d| top_d; what the tensor cores may take for zero (subnormal parts) is
  // covered by 2^-100 on both sides; a NaN as in score_kernel ----
  float* const tops = reinterpret_cast<float*>(smem + T::kOffTop);
  constexpr int kShare = kThreads > kWords ? kThreads / kWords : 1;
  for (int share = 0; share < kShare; ++share) {
    if (static_cast<int>(threadIdx.x) / kWords == share) {
#pragma unroll
      for (int x = 0; x < (kWords + kThreads - 1) / kThreads; ++x) {
        const int word = threadIdx.x % kWords + x * kThreads;
        const float a = fabsf(bf16lo(top[x])), b = fabsf(bf16hi(top[x]));
        tops[2 * word] = share == 0 ? a : fmaxf(tops[2 * word], a);
        tops[2 * word + 1] = share == 0 ? b : fmaxf(tops[2 * word + 1], b);
      }
    }
    together();
  }
  for (int i = warp; i < nq; i += T::kWarps) {
    float size = 0.0f;
    bool none = true;
    for (int x = lane; x < kWords; x += 32) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(smem + i * T::kPitch + 4 * x);
      const float a = fabsf(bf16lo(w)), b = fabsf(bf16hi(w));
      none = none && a == 0.0f && b == 0.0f;
      size += (a * 1.01f + 0x1p-100f) * (tops[2 * x] + 0x1p-100f);
      size += (b * 1.01f + 0x1p-100f) * (tops[2 * x + 1] + 0x1p-100f);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) size += __shfl_xor_sync(0xFFFFFFFFu, size, o);
    none = __all_sync(0xFFFFFFFFu, none);
    if (lane == 0)
      STX(p.sizes + (static_cast<int64_t>(tok0 + i) * p.H + h) * p.sizes_pitch + blockIdx.y, none ? 0.0f : fmaxf(size, 0x1p-149f));
  }
  if (__any_sync(0xFFFFFFFFu, timed_out) && lane == 0) set_status(p.status, 16u);
}

// What the threads of one list share.  A list of one warp needs no barrier.
constexpr uint32_t kFewTies = 32u;  // blocks to score again, where they are few
template <int kThreads>
struct ListShared {
  static constexpr int kBins = kThreads == 32 ? 256 : 1024;
  uint32_t slot[2][64];
  uint32_t bin[kBins];  // from the highest keys down
  uint32_t found[3];    // bin of the k-th key, keys above it, keys in it
  uint32_t count;       // entries below
  uint32_t entry[kFewTies];
  uint64_t score[kFewTies];
};

template <int kThreads>
struct ListThreads {
  static constexpr int kWarps = kThreads / 32;
  ListShared<kThreads>& sh;
  int turn;  // of the slots, so that one barrier does for each exchange

  __device__ __forceinline__ void sync() {
    if constexpr (kThreads == 32) {
      __syncwarp();
    } else {
      __syncthreads();
    }
  }
  __device__ __forceinline__ uint32_t sum(uint32_t v) {
    v = __reduce_add_sync(0xFFFFFFFFu, v);
    if constexpr (kWarps == 1) return v;
    return exchange(v, 0u, [](uint32_t x) { return __reduce_add_sync(0xFFFFFFFFu, x); });
  }
  __device__ __forceinline__ uint32_t max(uint32_t v) {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if constexpr (kWarps == 1) return v;
    return exchange(v, 0u, [](uint32_t x) { return __reduce_max_sync(0xFFFFFFFFu, x); });
  }
  // least of lo and largest of hi
  __device__ __forceinline__ void range(uint32_t& lo, uint32_t& hi) {
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    if constexpr (kWarps > 1) {
      const int lane = threadIdx.x & 31;
      uint32_t* const at = sh.slot[turn];
      turn ^= 1;
      if (lane == 0) {
        at[threadIdx.x >> 5] = lo;
        at[32 + (threadIdx.x >> 5)] = hi;
      }
      __syncthreads();
      lo = __reduce_min_sync(0xFFFFFFFFu, lane < kWarps ? at[lane] : 0xFFFFFFFFu);
      hi = __reduce_max_sync(0xFFFFFFFFu, lane < kWarps ? at[32 + lane] : 0u);
    }
  }
  // sum over the threads before this one
  __device__ __forceinline__ uint32_t before(uint32_t v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t upto = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    if constexpr (kWarps == 1) return upto - v;
    uint32_t* const at = sh.slot[turn];
    turn ^= 1;
    if (lane == 31) at[warp] = upto;
    __syncthreads();
    return upto - v + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? at[lane] : 0u);
  }

 private:
  template <typename F>
  __device__ __forceinline__ uint32_t exchange(uint32_t v, uint32_t none, F reduce) {
    uint32_t* const at = sh.slot[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return reduce(lane < kWarps ? at[lane] : none);
  }
};

// The border of the k highest keys (0: none) that lie in from .. to: at least k keys are >= hi, fewer are
// above it; lo is the largest key below hi (0: none) where exactly k are, else hi.  By histograms of
// the range, each of the part that holds the k-th key, until that has at most 32 keys (or one value),
// which a warp ranks.  Keys that are scores spread well: one histogram does for nearly all lists.  (A
// search by halves took 16 counts over the thread block, 7500 cycles for 2048 keys; keys in shared memory
// and short loops over them, 3 us more of 58 for 256 lists of 2048.)
struct Border {
  uint32_t hi, lo, count;
};
template <int kThreads, int P>
__device__ __forceinline__ Border find_border(const uint32_t (&key)[P], uint32_t k, uint32_t from, uint32_t to,
                                              ListThreads<kThreads>& th) {
  ListShared<kThreads>& sh = th.sh;
  constexpr int kBins = ListShared<kThreads>::kBins, kEach = kBins / kThreads, kBits = kThreads == 32 ? 8 : 10;
  const int lane = threadIdx.x & 31, me = threadIdx.x % kThreads;
  uint32_t above = 0u, inside = 0u;
  for (int round = 0;; ++round) {
    const int shift = max(0, 32 - __clz(to - from) - kBits);
#pragma unroll
    for (int x = 0; x < kEach; ++x) sh.bin[me + x * kThreads] = 0u;
    if (me == 0) sh.count = 0u;
    th.sync();
#pragma unroll
    for (int j = 0; j < P; ++j)
      if (key[j] - from <= to - from) atomicAdd(&sh.bin[kBins - 1 - ((key[j] - from) >> shift)], 1u);  // from > 0
    th.sync();
    uint32_t each[kEach], sum = 0u;
#pragma unroll
    for (int x = 0; x < kEach; ++x) sum += each[x] = sh.bin[me * kEach + x];
    uint32_t upto = above + th.before(sum);
    if (upto < k && upto + sum >= k) {
#pragma unroll
      for (int x = 0; x < kEach; ++x) {
        if (upto < k && upto + each[x] >= k) {
          sh.found[0] = kBins - 1 - (me * kEach + x);
          sh.found[1] = upto;
          sh.found[2] = each[x];
        }
        upto += each[x];
      }
    }
    th.sync();
    const uint32_t low = from + (sh.found[0] << shift);
    to = shift == 0 ? low : min(to, low + ((1u << shift) - 1u));
    from = low;
    above = sh.found[1];
    inside = sh.found[2];
    // four rounds narrow 32 bits; keys that another call overwrote (a shared workspace) end here as well
    if (inside <= 32u || from >= to || round == 4) break;
    th.sync();  // found is read before it is written again
  }
  inside = from != to ? min(inside, 32u) : inside;
  Border at{from, from, above + inside};
  uint32_t below = 0u;  // the largest key below `from`
#pragma unroll
  for (int j = 0; j < P; ++j) {
    if (key[j] < from) below = max(below, key[j]);
    if (from != to && key[j] - from <= to - from) sh.entry[atomicAdd(&sh.count, 1u) % kFewTies] = key[j];
  }
  below = th.max(below);  // (a barrier, or)
  if constexpr (kThreads == 32) __syncwarp();
  if (from != to) {
    const uint32_t mine = lane < static_cast<int>(inside) ? sh.entry[lane] : 0u;
    uint32_t greater = above, equal = 0u, next = 0u;  // next: the largest entry below mine
#pragma unroll 1
    for (uint32_t x = 0; x < inside; ++x) {
      const uint32_t other = sh.entry[x];
      greater += other > mine ? 1u : 0u;
      equal += other == mine ? 1u : 0u;
      if (other < mine) next = max(next, other);
    }
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, lane < static_cast<int>(inside) && greater < k && greater + equal >= k);
    const int src = __ffs(hit) - 1;
    at.hi = __shfl_sync(0xFFFFFFFFu, mine, src);
    at.count = __shfl_sync(0xFFFFFFFFu, greater + equal, src);
    below = max(below, __shfl_sync(0xFFFFFFFFu, next, src));
  }
  at.lo = at.count == k ? below : at.hi;
  return at;
}

// s + e = a + b exactly (Knuth's sum of two).
__device__ __forceinline__ float two_sum(float a, float b, float& e) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
  return s;
}

// The score of one block in twice binary32's precision, by a warp, as an ordered integer; NaN: 0.  Lanes take 8
// channels of q- . lo, q+ . hi at a time, with kC such chunks' (2 at head_dim 256) and kJ heads' loads in flight
// (one and two where many lists share an SM, or where 1024 threads have 64 registers each: two and four cost
// 40 registers, 8192 lists 10 us, 32 lists of 30,000 blocks 10 of 127).
template <int kC, int kJ>
__device__ __noinline__ uint64_t score_pair(const SelectParams& p, int tok, int h, int64_t blk) {
  const int lane = threadIdx.x & 31;
  const uint16_t* const q = p.q + tok * p.q_row_pitch + static_cast<int64_t>(h) * p.group * p.q_head_pitch;
  float sum = 0.0f, rest = 0.0f;
#pragma unroll 1
  for (int d0 = 8 * lane; d0 < 2 * p.D; d0 += 256 * kC) {
    uint32_t w[kC][4] = {};
    float qh[kC][8] = {}, ql[kC][8] = {};
#pragma unroll
    for (int c = 0; c < kC; ++c)
      if (d0 + 256 * c < 2 * p.D) load16B(p.bounds + (blk * p.H + h) * (2 * p.D) + d0 + 256 * c, w[c]);
#pragma unroll 1
    for (int j0 = 0; j0 < p.group; j0 += kJ) {
      uint32_t v[kJ][kC][4];
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const int d = d0 + 256 * c;
          v[j][c][0] = v[j][c][1] = v[j][c][2] = v[j][c][3] = 0u;
          if (d < 2 * p.D && j0 + j < p.group) load16B(q + (j0 + j) * p.q_head_pitch + (d < p.D ? d : d - p.D), v[j][c]);
        }
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const bool low = d0 + 256 * c < p.D;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float y = x % 2 == 0 ? bf16lo(v[j][c][x / 2]) : bf16hi(v[j][c][x / 2]);
            float e;
            qh[c][x] = two_sum(qh[c][x], low != (y > 0.0f) ? y : 0.0f, e);
            ql[c][x] = __fadd_rn(ql[c][x], e);
          }
        }
    }
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float y = x % 2 == 0 ? bf16lo(w[c][x / 2]) : bf16hi(w[c][x / 2]);
        const float t = __fmul_rn(qh[c][x], y);
        float e;
        sum = two_sum(sum, t, e);
        rest = __fadd_rn(rest, __fadd_rn(e, __fmaf_rn(ql[c][x], y, __fmaf_rn(qh[c][x], y, -t))));
      }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    float e;
    const float rest2 = __shfl_xor_sync(0xFFFFFFFFu, rest, o);
    sum = two_sum(sum, __shfl_xor_sync(0xFFFFFFFFu, sum, o), e);
    rest = __fadd_rn(__fadd_rn(rest, rest2), e);
  }
  sum = two_sum(sum, rest, rest);
  return isnan(sum) ? 0ull : static_cast<uint64_t>(score_key(sum)) << 32 | score_key(rest);
}

// The same in binary64 (two operations a cycle and SM on this GPU), an ordered integer; NaN: 0.
__device__ __noinline__ uint64_t score_wide(const SelectParams& p, int tok, int h, int64_t blk) {
  const int lane = threadIdx.x & 31;
  double sum = 0.0;
  for (int d = lane; d < 2 * p.D; d += 32) {
    const bool low = d < p.D;
    const uint16_t* const q = p.q + tok * p.q_row_pitch + static_cast<int64_t>(h) * p.group * p.q_head_pitch + (low ? d : d - p.D);
    double qd = 0.0;
    for (int j = 0; j < p.group; ++j) {
      const float v = __uint_as_float(static_cast<uint32_t>(LDX(q + j * p.q_head_pitch)) << 16);
      if (low != (v > 0.0f)) qd += static_cast<double>(v);
    }
    sum = fma(qd, static_cast<double>(__uint_as_float(static_cast<uint32_t>(LDX(p.bounds + (blk * p.H + h) * (2 * p.D) + d)) << 16)), sum);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(sum + 0.0));
  return isnan(sum) ? 0ull : (u >> 63) != 0ull ? ~u : u | 0x8000000000000000ull;
}

// The list of one (query token, KV head): of its kThreads threads, t holds the keys of P blocks from t P on;
// a thread block has 128 / kThreads lists, or one.  Bound: latency of a dozen barriers and exchanges
// between the threads, and of the first use of each instruction line.
template <int kThreads, int P>
__global__ void __launch_bounds__(kThreads < 128 ? 128 : kThreads) select_kernel(const SelectParams p) {
  constexpr int kRows = kThreads < 128 ? 128 / kThreads : 1, kWarps = kThreads / 32;
  static_assert(kThreads == 32 || kRows == 1, "lists of one warp, or of the block");
  static_assert(P % 4 == 0 && P <= 32, "vectors of keys, bits of a word");
  __shared__ ListShared<kThreads> shared[kRows];
  const int lane = threadIdx.x & 31, warp = kThreads == 32 ? 0 : threadIdx.x >> 5;  // of the list
  const int me = threadIdx.x % kThreads, mine = threadIdx.x / kThreads;
  const int64_t at_row = static_cast<int64_t>(blockIdx.x) * kRows + mine;  // i H + h
  const int i = static_cast<int>(at_row / p.H), h = static_cast<int>(at_row - static_cast<int64_t>(i) * p.H), s = blockIdx.y;
  ListShared<kThreads>& sh = shared[mine];
  ListThreads<kThreads> th{sh, 0};
  int q0, n, len;
  const bool ok = select_range(p, s, q0, n, len);
  if (!ok && threadIdx.x == 0 && blockIdx.x == 0) set_status(p.status, 8u);
  // launched as a programmatic dependent of the score kernel: wait for its results (every
  // block does, so that this grid's end implies the other's)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (i >= n) return;
  const int pos = len - n + i;
  const int vis = static_cast<int>(p.div_bs.div(static_cast<uint32_t>(pos))) + 1;
  const int64_t row = static_cast<int64_t>(q0 + i) * p.H + h;
  int32_t* const out = p.selected + row * p.topk;
  if (vis <= p.topk) {
    for (int j = me; j < p.topk; j += kThreads) STX(out + j, j < vis ? j : -1);
    return;
  }
  float size = 0.0f;  // over the error bound of the scores
  bool bounded = true;
  for (int x = lane; x < p.sizes_n; x += 32) {
    const float y = LDX(p.sizes + row * p.sizes_pitch + x);
    bounded = bounded && y <= 1e38f;  // not: sums that may overflow, an infinite q or bound
    size = fmaxf(size, y);
  }
  // blocks below `head` and from `tail` on are listed in any case: their keys become 0
  const int head = min(p.first, vis), tail = max(vis - p.last, head);
  const uint32_t k = static_cast<uint32_t>(p.topk - head - (vis - tail));
  const int b0 = me * P;
  uint32_t key[P];
#pragma unroll
  for (int j = 0; j < P; j += 4) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (b0 + j < vis) v = LDX(reinterpret_cast<const uint4*>(p.keys + row * p.pitch + b0 + j));
    key[j] = v.x, key[j + 1] = v.y, key[j + 2] = v.z, key[j + 3] = v.w;
  }
  uint32_t least = 0xFFFFFFFFu, most = 0u;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    if (b0 + j < head || b0 + j >= tail) key[j] = 0u;
    least = min(least, key[j] - 1u);  // 0 as the largest
    most = max(most, key[j]);
  }
  size = group_max<32>(size);
  bounded = __all_sync(0xFFFFFFFFu, bounded);
  const float e = size > 0.0f ? size * p.err + 0x1p-130f : 0.0f;  // + roundings below the normal numbers

  Border at{kKeyListed, kKeyListed, 0u};  // listed: keys above at.hi, and of those equal to it the first
  if (k > 0u) {
    th.range(least, most);
    at = find_border<kThreads, P>(key, k, least + 1u, most, th);
    const bool scored = at.hi > kKeyNan;  // not: blocks without a score fill the list
    const float hi = key_score(at.hi), lo = at.lo > kKeyNan ? key_score(at.lo) : -__int_as_float(0x7F800000);
    if (!bounded || (scored && e > 0.0f && !(hi - lo > 2.0f * e))) {
      th.sync();  // the entries are read
      if (me == 0) sh.count = 0u;
      th.sync();
      uint32_t again = 0u, certain = 0u;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        if (key[j] <= kKeyBad || (bounded && key[j] == kKeyNan)) continue;  // last in any case
        const float x = key_score(key[j]);
        if (bounded && x > lo + 2.0f * e) {
          key[j] = kKeyListed;
          ++certain;
        } else if (bounded && x < hi - 2.0f * e) {
          key[j] = 0u;
        } else {
          again |= 1u << j;
        }
      }
      for (uint32_t left = again; left != 0u; left &= left - 1u) {
        const uint32_t place = atomicAdd(&sh.count, 1u);
        if (place < kFewTies) sh.entry[place] = b0 + __ffs(left) - 1;
      }
      const uint32_t need = k - th.sum(certain);
      th.sync();
      const uint32_t m = sh.count;
      const int32_t* const table = p.table + static_cast<int64_t>(s) * p.max_blocks;  // what has a score lies in the pool
      if (m <= kFewTies && m >= need && size > 0x1p-60f && size < 0x1p100f) {
        // few, and nothing that overflows or underflows: a warp scores one at a time, then each one's rank
        for (uint32_t x = warp; x < m; x += kWarps) {
          constexpr bool kNarrow = kThreads == 32 || kThreads == 1024;
          const uint64_t u = score_pair<kNarrow ? 1 : 2, kNarrow ? 2 : 4>(p, q0 + i, h, LDX(table + sh.entry[x]));
          if (lane == 0) sh.score[x] = u;
        }
        th.sync();
        if (me < static_cast<int>(m)) {
          const uint64_t u = sh.score[me];
          const uint32_t b = sh.entry[me];
          uint32_t rank = 0u;
          for (uint32_t x = 0; x < m; ++x) {
            const uint64_t other = sh.score[x];
            rank += other > u || (other == u && sh.entry[x] < b) ? 1u : 0u;
          }
          sh.bin[me] = rank < need ? b : 0xFFFFFFFFu;  // the winners
        }
        th.sync();
#pragma unroll
        for (int j = 0; j < P; ++j)
          if ((again >> j) & 1u) key[j] = 0u;
        for (uint32_t x = 0; x < m; ++x) {
          const uint32_t j = sh.bin[x] - static_cast<uint32_t>(b0);
          if (j < static_cast<uint32_t>(P)) {
#pragma unroll
            for (int y = 0; y < P; ++y)
              if (y == static_cast<int>(j)) key[y] = kKeyListed;
          }
        }
        at = Border{kKeyListed, 0u, k};
      } else {
#pragma unroll 1
        for (int stage = 0; stage < 2; ++stage) {
#pragma unroll 1
          for (uint32_t left = again;;) {
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, left != 0u);
            if (who == 0u) break;
            const int src = __ffs(who) - 1;
            const int j = __shfl_sync(0xFFFFFFFFu, __ffs(left) - 1, src);
            const uint64_t u = score_wide(p, q0 + i, h, LDX(table + (warp * 32 + src) * P + j));
            const uint32_t bits = static_cast<uint32_t>(stage == 0 ? u >> 33 : (u >> 2) & 0x7FFFFFFFull);
            if (lane == src) {
              left &= left - 1u;
#pragma unroll
              for (int x = 0; x < P; ++x)
                if (x == j) key[x] = u == 0ull ? kKeyNan64 : kKeyNan64 + 1u + bits;
            }
          }
          least = 0xFFFFFFFFu;
          most = 0u;
#pragma unroll
          for (int j = 0; j < P; ++j) {
            least = min(least, key[j] - 1u);
            most = max(most, key[j]);
          }
          th.range(least, most);
          at = find_border<kThreads, P>(key, k, least + 1u, most, th);
          if (at.count == k || stage == 1 || at.hi <= kKeyNan64) break;
          again = 0u;
#pragma unroll
          for (int j = 0; j < P; ++j) {
            if (key[j] == at.hi) {
              again |= 1u << j;
            } else {
              key[j] = key[j] > at.hi ? kKeyListed : 0u;
            }
          }
          th.sync();  // the entries are read
        }
      }
    }
  }
  // ---- the list, in the order of the blocks ----
  uint32_t listed = 0u, ties = 0u;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    if (key[j] > at.hi || (b0 + j < vis && (b0 + j < head || b0 + j >= tail))) listed |= 1u << j;
    if (key[j] == at.hi) ties |= 1u << j;
  }
  if (at.count > k) {  // more equal ones than the list takes; uniform
    const uint32_t left = static_cast<uint32_t>(p.topk) - th.sum(__popc(listed));
    uint32_t before = th.before(__popc(ties));
    for (; ties != 0u; ties &= ties - 1u, ++before)
      if (before < left) listed |= ties & (0u - ties);
  } else {
    listed |= ties;
  }
  uint32_t before = th.before(__popc(listed));
  for (; listed != 0u; listed &= listed - 1u, ++before) STX(out + before, b0 + __ffs(listed) - 1);
}

template <int kThreads, int P>
cudaError_t select_launch(const SelectParams& p, bool dependent, cudaStream_t s) {
  constexpr int kRows = kThreads < 128 ? 128 / kThreads : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(p.max_q) * p.H + kRows - 1) / kRows),
                     static_cast<unsigned>(p.S));
  cfg.blockDim = dim3(kThreads < 128 ? 128 : kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, select_kernel<kThreads, P>, p);
}

template <int D>
cudaError_t score_launch(SelectParams& p, cudaStream_t s) {
  cudaError_t e;
  if (p.max_q < kTileQueries) {
    const ScorePlan plan(p.H, D, p.max_q);
    // segments of each sequence that fill the GPU once, of 16 blocks at least
    const int heads = (p.H + plan.hc - 1) / plan.hc;
    const int64_t rows = static_cast<int64_t>(p.S) * heads;
    const int64_t segments = std::max(int64_t{1}, std::min(num_sms() / rows, static_cast<int64_t>(p.most) / 16));
    p.sizes_n = static_cast<int>(segments);
    // in units of 2^-23: 16 additions a step of 16 channels, which the tensor cores may round towards
    // zero, half a unit for each step's sum, one for each part's and half for each head's; two parts: as
    // much as 2^-18 for what they leave of q
    p.err = 1.02f * static_cast<float>(16 + D / 16 + 4 + p.group + (p.max_q <= 2 ? 0 : 33)) * 0x1p-23f;
    struct Tag {};
    e = allow_smem<Tag>(reinterpret_cast<const void*>(score_kernel<D>), 227 * 1024 - 512);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(segments), heads, p.S);
    KVQ_LAUNCH("score_kernel", s, score_kernel<D><<<grid, 32 * (kScoreWarps<D> + 1), plan.smem, s>>>(p); e = cudaGetLastError());
    return e;
  }
  using T = ScoreTile<D>;
  // segments of whole tiles, as many as fill the GPU once
  const int64_t rows = static_cast<int64_t>((p.max_q + T::kM - 1) / T::kM) * p.H, tiles = (p.most + T::kN - 1) / T::kN;
  const int64_t segments = std::max(int64_t{1}, std::min(tiles, num_sms() / (rows * p.S)));
  p.segment = static_cast<int>((tiles + segments - 1) / segments) * T::kN;
  p.sizes_n = (p.most + p.segment - 1) / p.segment;
  // in units of 2^-23: 32 additions a step of 16 channels (hi and lo), which the tensor cores may round
  // towards zero, the same again for what hi + lo leaves of q (2^-18), half a unit for each step's sum
  // and for each head's
  p.err = 1.02f * static_cast<float>(64 + D / 16 + p.group) * 0x1p-23f;
  struct Tag {};
  e = allow_smem<Tag>(reinterpret_cast<const void*>(score_tile_kernel<D>), T::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(p.sizes_n), p.S);
  KVQ_LAUNCH("score_tile_kernel", s, score_tile_kernel<D><<<grid, 32 * (T::kWarps + 1), T::kSmem, s>>>(p); e = cudaGetLastError());
  return e;
}

template <int D>
cudaError_t select_dim(SelectParams& p, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const bool scores = p.most > p.topk;
  if (scores && (e = score_launch<D>(p, s)) != cudaSuccess) return e;
  // threads of a list: a warp where lists are many and short (8192 lists of 1024 blocks: 91 us with their scores,
  // 101 by 128 threads, 96 by 64; 32 lists of 375: 10.6 by 128, 12.3 by a warp).  1024 threads have 64 registers
  // each and spill, so they take only the longest (32 lists of 12,500: 61.5, by 1024 threads 72.7)
  const int64_t lists = static_cast<int64_t>(p.max_q) * p.H * p.S;
  const bool many = lists >= 8 * num_sms();
  KVQ_LAUNCH("select_kernel", s,
             e = many && p.most <= 512    ? select_launch<32, 16>(p, scores, s)
                 : many && p.most <= 1024 ? select_launch<32, 32>(p, scores, s)
                 : p.most <= 512          ? select_launch<128, 4>(p, scores, s)
                 : p.most <= 2048         ? select_launch<256, 8>(p, scores, s)
                 : p.most <= 8192         ? select_launch<512, 16>(p, scores, s)
                 : p.most <= 16384        ? select_launch<512, 32>(p, scores, s)
                                          : select_launch<1024, 32>(p, scores, s));
  return e;
}

int32_t key_pitch(int32_t most) { return (most + 31) / 32 * 32; }
int32_t sizes_pitch(int32_t most) { return (most + 15) / 16; }  // parts of 16 blocks or more

}  // namespace

// Keys of every (token, head), then the sizes of their parts.
size_t select_workspace_bytes(int32_t T, int32_t H, int32_t most) {
  if (T <= 0 || H <= 0 || most <= 0) return 0;
  return static_cast<size_t>(T) * H * (static_cast<size_t>(key_pitch(most)) + sizes_pitch(most)) * 4;
}

cudaError_t launch_select_blocks(const SelectParams& p_in, void* workspace, cudaStream_t s) {
  SelectParams p = p_in;
  p.pitch = key_pitch(p.most);
  p.sizes_pitch = sizes_pitch(p.most);
  p.keys = static_cast<uint32_t*>(workspace);
  p.sizes = reinterpret_cast<float*>(p.keys + static_cast<int64_t>(p.num_tokens) * p.H * p.pitch);
  switch (p.D) {
    case 64: return select_dim<64>(p, s);
    case 128: return select_dim<128>(p, s);
    case 256: return select_dim<256>(p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
