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
// certain, one below the lowest listed one by as much is not; what lies between is scored again in
// binary64, by one warp a block, and ranked by the upper and then the lower bits of that.  One row in
// fifty has such blocks; exact ties go the same way to the index.  What binary32 cannot bound (sums that
// may overflow) all goes to binary64.
//
// Few queries a sequence (score_kernel): a warp streams blocks' bounds by bulk copies and takes the
// dot products in registers.  Bound: HBM.  From kTileQueries queries on (score_tile_kernel): a product
// of 64 queries and 128 blocks on the tensor cores, q split into two bf16 parts.
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

constexpr int kScoreWarps = 4;
constexpr int kScoreQueries = 8;  // of one pass over the bounds
constexpr int kScoreBytes = 16384;  // of bounds that a warp has in flight
template <int D>
constexpr int kScoreBlocks = kScoreBytes / (4 * D);  // cache blocks of a warp
constexpr int kTileQueries = 9;  // queries a sequence from which on the tile kernel takes the call

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

// The lane's part of a block's bounds, 2 D bf16 over the warp: D / 16 of them, D / 32 words.
template <int D>
__device__ __forceinline__ void load_bounds(const uint16_t* at, uint32_t (&w)[D / 32]) {
  if constexpr (D == 64) {
    load8B(at, w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      uint32_t v[4];
      load16B(at + 8 * i, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
    }
  }
}

// Sums over the heads of one token's q- and q+ at channels d .. d + 7.
__device__ __forceinline__ void sum_heads(const SelectParams& p, int tok, int h, int d, float (&minus)[8], float (&plus)[8]) {
  const uint16_t* const x = p.q + tok * p.q_row_pitch + static_cast<int64_t>(h) * p.group * p.q_head_pitch + d;
#pragma unroll
  for (int i = 0; i < 8; ++i) minus[i] = plus[i] = 0.0f;
#pragma unroll 4
  for (int j = 0; j < p.group; ++j) {
    uint32_t v[4];
    load16B(x + j * p.q_head_pitch, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = i % 2 == 0 ? bf16lo(v[i / 2]) : bf16hi(v[i / 2]);
      minus[i] = __fadd_rn(minus[i], y > 0.0f ? 0.0f : y);  // a NaN goes on
      plus[i] = __fadd_rn(plus[i], y > 0.0f ? y : 0.0f);
    }
  }
}

__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Scores of a run of blocks of one (sequence, KV head) for all its query tokens.  Each lane of a warp
// copies its blocks' bounds to shared memory, all at once (16 KB a warp in flight); then the warp
// reads one block's with one load a lane, and adds up the sums of 8 blocks over its lanes by 9
// shuffles (halving the sums with the lanes).
template <int D>
__global__ void __launch_bounds__(32 * kScoreWarps, 3) score_kernel(const SelectParams p) {
  constexpr int kC = D / 16;  // values of a lane
  constexpr int kB = kScoreBlocks<D>, kGroups = kB / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(16) float coef[kScoreQueries][2 * D];
  __shared__ __align__(8) uint64_t bars[kScoreWarps][kGroups];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, s = blockIdx.z;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int q0, n, len;
  if (!select_range(p, s, q0, n, len) || n == 0) return;
  const int blocks = static_cast<int>(p.div_bs.div(static_cast<uint32_t>(len - 1))) + 1;
  const int c0 = static_cast<int>(blockIdx.x) * kScoreWarps * kB;
  if (blocks <= p.topk || c0 >= blocks) return;
  const int b0 = c0 + warp * kB;
  unsigned char* const ring = smem + warp * kScoreBytes;
  const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const uint32_t bar0 = static_cast<uint32_t>(__cvta_generic_to_shared(&bars[warp][0]));
  if (lane == 0) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) mbar_init(bar0 + 8 * g, 1);
    mbar_init_fence();
  }
  __syncwarp();
  uint32_t have[(kB + 31) / 32];  // bit j: block b0 + 32 x + j has bounds
#pragma unroll
  for (int x = 0; x < (kB + 31) / 32; ++x) {
    const int j = 32 * x + lane, b = b0 + j;
    const bool in = j < kB && b < blocks;
    const int64_t blk = in ? LDX(p.table + static_cast<int64_t>(s) * p.max_blocks + b) : -1;
    const bool ok = in && blk >= 0 && blk < p.num_blocks;
    if (__any_sync(0xFFFFFFFFu, in && !ok) && lane == 0) set_status(p.status, 2u);
    have[x] = __ballot_sync(0xFFFFFFFFu, ok);
    if (lane % 8 == 0 && j < kB)
      mbar_arrive_expect_tx(bar0 + 8 * (j / 8), 4u * D * __popc((have[x] >> lane) & 0xFFu));
    __syncwarp();
    if (ok) bulk_copy_g2s(ring_s + j * 4 * D, p.bounds + (blk * p.H + h) * (2 * D), 4u * D, bar0 + 8 * (j / 8));
  }
  uint32_t top[D / 32] = {};  // largest |bound| of the lane's channels, packed
  bool timed_out = false;
  for (int i0 = 0; i0 < n; i0 += kScoreQueries) {
    const int ni = min(kScoreQueries, n - i0);
    if (i0 > 0) __syncthreads();
    for (int at = threadIdx.x; at < ni * (D / 8); at += 32 * kScoreWarps) {
      const int i = at / (D / 8), d = 8 * (at - i * (D / 8));
      float minus[8], plus[8];
      sum_heads(p, q0 + i0 + i, h, d, minus, plus);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        coef[i][d + x] = minus[x];
        coef[i][D + d + x] = plus[x];
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int g8 = 0; g8 < kGroups; ++g8) {
      if (b0 + 8 * g8 >= blocks) break;
      if (i0 == 0 && !mbar_wait(bar0 + 8 * g8, 0)) timed_out = true;
      const uint32_t here = (have[g8 / 4] >> (8 * (g8 % 4))) & 0xFFu;
      uint32_t w[8][D / 32];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t* const at = reinterpret_cast<const uint32_t*>(ring + (8 * g8 + j) * 4 * D) + lane * (D / 32);
#pragma unroll
        for (int x = 0; x < D / 32; x += 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(at + x);
          const bool ok = (here >> j) & 1u;
          w[j][x] = ok ? v.x : 0u;
          w[j][x + 1] = ok ? v.y : 0u;
        }
      }
      if (i0 == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int x = 0; x < D / 32; ++x)
            asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(top[x]) : "r"(top[x]), "r"(w[j][x]));
      }
      for (int i = 0; i < ni; ++i) {
        const uint64_t* const c = reinterpret_cast<const uint64_t*>(&coef[i][lane * kC]);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint64_t acc = 0ull;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) acc = fma_f32x2(pack_f32x2(w[j][x] << 16, w[j][x] & 0xFFFF0000u), c[x], acc);
          uint32_t a, b;
          unpack_f32x2(acc, a, b);
          v[j] = __fadd_rn(__uint_as_float(a), __uint_as_float(b));
        }
#pragma unroll
        for (int o = 16, m = 4; m >= 1; o >>= 1, m >>= 1) {
          const bool up = (lane & o) != 0;
#pragma unroll
          for (int j = 0; j < m; ++j) {
            const float give = up ? v[j] : v[j + m], keep = up ? v[j + m] : v[j];
            v[j] = __fadd_rn(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
          }
        }
        v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 2));
        v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 1));
        const int j = lane >> 2, b = b0 + 8 * g8 + j;
        if ((lane & 3) == 0 && b < blocks)
          STX(p.keys + (static_cast<int64_t>(q0 + i0 + i) * p.H + h) * p.pitch + b,
              (here >> j) & 1u ? score_key(v[0]) : kKeyBad);
      }
    }
    if (b0 < blocks) {
      for (int i = 0; i < ni; ++i) {
        float a = 0.0f;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          // 0 only where there is nothing to round: a product that underflows counts 2^-149
          const float c0 = fabsf(coef[i][lane * kC + 2 * x]), c1 = fabsf(coef[i][lane * kC + 2 * x + 1]);
          const float t0 = fabsf(bf16lo(top[x])), t1 = fabsf(bf16hi(top[x]));
          a += c0 * t0 + (c0 > 0.0f && t0 > 0.0f ? 0x1p-149f : 0.0f);
          a += c1 * t1 + (c1 > 0.0f && t1 > 0.0f ? 0x1p-149f : 0.0f);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        if (lane == 0)
          STX(p.sizes + (static_cast<int64_t>(q0 + i0 + i) * p.H + h) * p.sizes_pitch + b0 / kB, a);
      }
    }
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
  static constexpr int kWarps = 8;
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(32 * ScoreTile<D>::kWarps, 1) score_tile_kernel(const SelectParams p) {
  using T = ScoreTile<D>;
  constexpr int kMT = T::kM / 32, kNT = T::kN / 32, kThreads = 32 * T::kWarps;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ uint32_t have[2][T::kN / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int qt = static_cast<int>(blockIdx.x) / p.H, h = static_cast<int>(blockIdx.x) - qt * p.H, s = blockIdx.z;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int q0, n, len;
  if (!select_range(p, s, q0, n, len) || qt * T::kM >= n) return;
  const int nq = min(T::kM, n - qt * T::kM), tok0 = q0 + qt * T::kM;
  // blocks that this tile's last query sees
  const int blocks = static_cast<int>(p.div_bs.div(static_cast<uint32_t>(len - n + qt * T::kM + nq - 1))) + 1;
  const int first = static_cast<int>(blockIdx.y) * p.sizes_step;
  if (blocks <= p.topk || first >= blocks) return;
  const int last = min(blocks, first + p.sizes_step), tiles = (last - first + T::kN - 1) / T::kN;
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const uint32_t bar0 = static_cast<uint32_t>(__cvta_generic_to_shared(bars));
  if (threadIdx.x == 0) {
    mbar_init(bar0, 1);
    mbar_init(bar0 + 8, 1);
    mbar_init_fence();
  }
  __syncthreads();
  // warp 0: copies of tile t into its stage
  auto fetch = [&](int t) {
    const int st = t & 1;
    int64_t blk[T::kN / 32];
    uint32_t count = 0u;
#pragma unroll
    for (int x = 0; x < T::kN / 32; ++x) {
      const int b = first + t * T::kN + 32 * x + lane;
      const bool in = b < last;
      blk[x] = in ? LDX(p.table + static_cast<int64_t>(s) * p.max_blocks + b) : -1;
      if (blk[x] < 0 || blk[x] >= p.num_blocks) blk[x] = -1;
      if (__any_sync(0xFFFFFFFFu, in && blk[x] < 0) && lane == 0) set_status(p.status, 2u);
      const uint32_t ok = __ballot_sync(0xFFFFFFFFu, blk[x] >= 0);
      if (lane == 0) have[st][x] = ok;
      count += __popc(ok);
    }
    if (lane == 0) mbar_arrive_expect_tx(bar0 + 8 * st, count * 4u * D);
    __syncwarp();
#pragma unroll
    for (int x = 0; x < T::kN / 32; ++x) {
      const uint32_t at = base + T::kOffB + st * T::kStage + (32 * x + lane) * T::kPitch;
      if (blk[x] >= 0) bulk_copy_g2s(at, p.bounds + (blk[x] * p.H + h) * (2 * D), 4u * D, bar0 + 8 * st);
    }
  };
  if (warp == 0) {
    fetch(0);
    if (tiles > 1) fetch(1);
  }
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
  __syncthreads();

  const int m0 = (warp & 1) * (T::kM / 2), n0 = (warp >> 1) * (T::kN / 4);
  const uint32_t a_at = base + (m0 + (lane & 15)) * T::kPitch + (lane >> 4) * 16;
  const uint32_t b_row = (n0 + (lane & 7) + ((lane >> 4) << 3)) * T::kPitch + ((lane >> 3) & 1) * 16;
  uint32_t top[2 * D / kThreads > 0 ? 2 * D / kThreads : 1] = {};
  constexpr int kWords = D;  // of a row
  bool timed_out = false;
  for (int t = 0; t < tiles; ++t) {
    const int st = t & 1;
    if (!mbar_wait(bar0 + 8 * st, (t >> 1) & 1)) timed_out = true;
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
      __syncthreads();
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
#pragma unroll
      for (int a = 0; a < kMT; ++a)
#pragma unroll
        for (int b = 0; b < kNT; ++b) {
          float step[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_bf16_16816(step, lo[a], bb[b / 2][2 * (b % 2)], bb[b / 2][2 * (b % 2) + 1]);
          mma_bf16_16816(step, hi[a], bb[b / 2][2 * (b % 2)], bb[b / 2][2 * (b % 2) + 1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[a][b][e] = __fadd_rn(acc[a][b][e], step[e]);
        }
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
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int a = 0; a < kMT; ++a)
#pragma unroll
      for (int b = 0; b < kNT; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = m0 + 16 * a + g + 8 * e, col = n0 + 8 * b + 2 * c, at = first + t * T::kN + col;
          if (i >= nq || at >= last) continue;
          uint32_t* const to = p.keys + (static_cast<int64_t>(tok0 + i) * p.H + h) * p.pitch + at;
          const uint32_t ok = have[st][col / 32] >> (col % 32);
          const uint2 v = make_uint2(ok & 1u ? score_key(acc[a][b][2 * e]) : kKeyBad,
                                     ok & 2u ? score_key(acc[a][b][2 * e + 1]) : kKeyBad);
          STX(reinterpret_cast<uint2*>(to), v);  // pitch is even: the pair lies in the row
        }
    __syncthreads();  // the stage is free
    if (warp == 0 && t + 2 < tiles) fetch(t + 2);
  }
  // ---- sizes: sum_d |q_d| top_d; what the tensor cores may take for zero (subnormal parts) is
  // covered by 2^-100 on both sides ----
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
    __syncthreads();
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

// Sums, maxima or minima over the threads of a row, the same in all of them.  A row of one warp needs
// no barrier; wider ones need one each (the slots alternate).
template <int kThreads>
struct RowReduce {
  uint32_t (*slot)[32];
  int turn;
  template <typename F>
  __device__ __forceinline__ uint32_t run(uint32_t v, F warp_reduce, uint32_t none) {
    constexpr int kWarps = kThreads / 32;
    v = warp_reduce(v);
    if constexpr (kWarps == 1) {
      return v;
    } else {
      uint32_t* const at = slot[turn];
      turn ^= 1;
      if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = v;
      __syncthreads();
      const int lane = threadIdx.x & 31;
      return warp_reduce(lane < kWarps ? at[lane] : none);
    }
  }
  __device__ __forceinline__ uint32_t sum(uint32_t v) {
    return run(v, [](uint32_t x) { return __reduce_add_sync(0xFFFFFFFFu, x); }, 0u);
  }
  __device__ __forceinline__ uint32_t max(uint32_t v) {
    return run(v, [](uint32_t x) { return __reduce_max_sync(0xFFFFFFFFu, x); }, 0u);
  }
  __device__ __forceinline__ uint32_t min(uint32_t v) {
    return run(v, [](uint32_t x) { return __reduce_min_sync(0xFFFFFFFFu, x); }, 0xFFFFFFFFu);
  }
  // Sum over the threads before this one.
  __device__ __forceinline__ uint32_t before(uint32_t v) {
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t upto = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    if constexpr (kWarps == 1) {
      return upto - v;
    } else {
      uint32_t* const at = slot[turn];
      turn ^= 1;
      if (lane == 31) at[warp] = upto;
      __syncthreads();
      return upto - v + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? at[lane] : 0u);
    }
  }
};

// The border of the k highest keys: at least k keys are >= hi, fewer are above it; lo is the
// largest key below hi (0: none) where exactly k are, else hi.
struct Border {
  uint32_t hi, lo, count;
};
template <int kThreads, int P>
__device__ __forceinline__ Border find_border(const uint32_t (&key)[P], uint32_t k, RowReduce<kThreads>& red) {
  uint32_t least = 0xFFFFFFFFu, most = 0u;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    if (key[j] == 0u) continue;
    least = min(least, key[j]);
    most = max(most, key[j]);
  }
  // count(>= from) >= k > count(>= to)
  uint32_t from = red.min(least), to = red.max(most) + 1u;
  uint32_t at = from, count = 0u;
  while (to - from > 1u) {
    const uint32_t mid = from + (to - from) / 2u;
    uint32_t c = 0u;
#pragma unroll
    for (int j = 0; j < P; ++j) c += key[j] >= mid ? 1u : 0u;
    c = red.sum(c);
    if (c >= k) from = mid;
    if (c < k) to = mid;
    if (c == k) break;
  }
  at = from;
  uint32_t hi = 0xFFFFFFFFu, lo = 0u, c = 0u;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    if (key[j] >= at) {
      hi = min(hi, key[j]);
      ++c;
    } else {
      lo = max(lo, key[j]);
    }
  }
  count = red.sum(c);
  hi = red.min(hi);
  lo = red.max(lo);
  return Border{hi, count > k ? hi : lo, count};
}

// The list of one (query token, KV head): of the row's kThreads threads, t holds the keys of P
// blocks from t P on; a thread block has 128 / kThreads rows, or one.  A search by halves over the
// keys' range finds the border (it ends as soon as a bound parts k keys from the rest).  Bound: latency
// of some 15 counts over the row's threads where there are few rows, else their issue.
template <int D, int kThreads, int P>
__global__ void __launch_bounds__(kThreads < 128 ? 128 : kThreads) select_kernel(const SelectParams p) {
  constexpr int kC = D / 16, kRows = kThreads < 128 ? 128 / kThreads : 1;
  static_assert(kThreads == 32 || kRows == 1, "rows of one warp, or of the block");
  const int lane = threadIdx.x & 31, warp = kThreads == 32 ? 0 : threadIdx.x >> 5;  // of the row
  const int me = threadIdx.x % kThreads;
  const int64_t at_row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kThreads;  // i H + h
  const int i = static_cast<int>(at_row / p.H), h = static_cast<int>(at_row - static_cast<int64_t>(i) * p.H), s = blockIdx.y;
  __shared__ uint32_t slots[2][32];
  RowReduce<kThreads> red{slots, 0};
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
  // blocks below `head` and from `tail` on are listed in any case
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
  // the error bound of the scores
  float size = 0.0f;
  bool bounded = true;
  for (int at = lane; at * p.sizes_step < vis; at += 32) {
    const float x = LDX(p.sizes + row * p.sizes_pitch + at);
    bounded = bounded && x <= 1e38f;  // not: sums that may overflow, NaN
    size = fmaxf(size, x);
  }
  size = group_max<32>(size);
  bounded = __all_sync(0xFFFFFFFFu, bounded);
  const float e = size > 0.0f ? size * p.err + 0x1p-130f : 0.0f;  // + roundings below the normal numbers
#pragma unroll
  for (int j = 0; j < P; ++j)
    if (b0 + j < head || b0 + j >= tail) key[j] = 0u;  // out of the search

  uint32_t listed = 0u;  // bits of this thread's blocks
  if (k > 0u) {
    Border at = find_border<kThreads, P>(key, k, red);
    const bool scored = at.hi > kKeyNan;  // not: blocks without a score fill the list
    const float hi = key_score(at.hi), lo = at.lo > kKeyNan ? key_score(at.lo) : -__int_as_float(0x7F800000);
    if (!bounded || (scored && e > 0.0f && !(hi - lo > 2.0f * e))) {
      uint32_t again = 0u;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        if (key[j] <= kKeyBad || (bounded && key[j] == kKeyNan)) continue;  // last in any case
        const float x = key_score(key[j]);
        if (bounded && x > lo + 2.0f * e) {
          key[j] = kKeyListed;
        } else if (bounded && x < hi - 2.0f * e) {
          key[j] = 0u;
        } else {
          again |= 1u << j;
        }
      }
      // the lane's channels of q+ or q-, in binary64
      double qd[kC];
#pragma unroll
      for (int x = 0; x < kC; ++x) qd[x] = 0.0;
#pragma unroll 1
      for (int j = 0; j < p.group; ++j) {
        uint32_t w[D / 32];
        load_bounds<D>(p.q + (q0 + i) * p.q_row_pitch + (static_cast<int64_t>(h) * p.group + j) * p.q_head_pitch +
                           (lane % 16) * kC, w);
#pragma unroll
        for (int x = 0; x < kC; ++x) {
          const float v = x % 2 == 0 ? bf16lo(w[x / 2]) : bf16hi(w[x / 2]);
          qd[x] += (lane < 16 ? !(v > 0.0f) : v > 0.0f) ? static_cast<double>(v) : 0.0;
        }
      }
#pragma unroll 1
      for (int stage = 0; stage < 2; ++stage) {
        uint32_t left = again;
        while (true) {
          const uint32_t who = __ballot_sync(0xFFFFFFFFu, left != 0u);
          if (who == 0u) break;
          const int src = __ffs(who) - 1;
          const int j = __shfl_sync(0xFFFFFFFFu, __ffs(left) - 1, src);
          const int b = (warp * 32 + src) * P + j;
          // one that has a score lies in the pool
          const int64_t blk = LDX(p.table + static_cast<int64_t>(s) * p.max_blocks + b);
          uint32_t w[D / 32];
          load_bounds<D>(p.bounds + (blk * p.H + h) * (2 * D) + lane * kC, w);
          double sum = 0.0;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            sum = fma(qd[2 * x], static_cast<double>(bf16lo(w[x])), sum);
            sum = fma(qd[2 * x + 1], static_cast<double>(bf16hi(w[x])), sum);
          }
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
          uint64_t u = static_cast<uint64_t>(__double_as_longlong(sum + 0.0));
          u = (u >> 63) != 0ull ? ~u : u | 0x8000000000000000ull;
          const uint32_t bits = static_cast<uint32_t>(stage == 0 ? u >> 33 : (u >> 2) & 0x7FFFFFFFull);
          const uint32_t fresh = isnan(sum) ? kKeyNan64 : kKeyNan64 + 1u + bits;
          if (lane == src) {
            left &= left - 1u;
#pragma unroll
            for (int x = 0; x < P; ++x)
              if (x == j) key[x] = fresh;
          }
        }
        at = find_border<kThreads, P>(key, k, red);
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
      }
    }
    // the keys above the border, and of those on it the first
    uint32_t ties = 0u;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      if (key[j] > at.hi) listed |= 1u << j;
      if (key[j] == at.hi) ties |= 1u << j;
    }
    if (at.count > k) {  // uniform
      const uint32_t need = k - red.sum(__popc(listed));
      uint32_t before = red.before(__popc(ties));
      for (; ties != 0u; ties &= ties - 1u, ++before)
        if (before < need) listed |= ties & (0u - ties);
    } else {
      listed |= ties;
    }
  }
#pragma unroll
  for (int j = 0; j < P; ++j)
    if (b0 + j < vis && (b0 + j < head || b0 + j >= tail)) listed |= 1u << j;
  uint32_t before = red.before(__popc(listed));
  for (; listed != 0u; listed &= listed - 1u, ++before) STX(out + before, b0 + __ffs(listed) - 1);
}

template <int D, int kThreads, int P>
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
  return cudaLaunchKernelEx(&cfg, select_kernel<D, kThreads, P>, p);
}

template <int D>
cudaError_t score_launch(SelectParams& p, cudaStream_t s) {
  cudaError_t e;
  if (p.max_q < kTileQueries) {
    constexpr int kSmem = kScoreWarps * kScoreBytes, kB = kScoreBlocks<D>;
    p.sizes_step = kB;
    // roundings on a product's way into a score, of 2^-24 each: the sum over the heads, a chain of
    // D / 32 products, the two chains' sum and 5 steps over the lanes; a fiftieth for those of
    // the bound itself and of the comparisons with it
    p.err = 1.02f * static_cast<float>(p.group + D / 32 + 8) * 0x1p-24f;
    e = cudaFuncSetAttribute(score_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>((p.most + kScoreWarps * kB - 1) / (kScoreWarps * kB)), p.H, p.S);
    KVQ_LAUNCH("score_kernel", s, score_kernel<D><<<grid, 32 * kScoreWarps, kSmem, s>>>(p); e = cudaGetLastError());
    return e;
  }
  using T = ScoreTile<D>;
  // segments of whole tiles, as many as fill the GPU once
  const int64_t rows = static_cast<int64_t>((p.max_q + T::kM - 1) / T::kM) * p.H, tiles = (p.most + T::kN - 1) / T::kN;
  const int64_t segments = std::max(int64_t{1}, std::min(tiles, num_sms() / (rows * p.S)));
  p.sizes_step = static_cast<int>((tiles + segments - 1) / segments) * T::kN;
  // in units of 2^-23: 32 additions a step of 16 channels (hi and lo), which the tensor cores may round
  // towards zero, the same again for what hi + lo leaves of q (2^-18), half a unit for each step's sum
  // and for each head's
  p.err = 1.02f * static_cast<float>(64 + D / 16 + p.group) * 0x1p-23f;
  e = cudaFuncSetAttribute(score_tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>((p.most + p.sizes_step - 1) / p.sizes_step), p.S);
  KVQ_LAUNCH("score_tile_kernel", s, score_tile_kernel<D><<<grid, 32 * T::kWarps, T::kSmem, s>>>(p); e = cudaGetLastError());
  return e;
}

template <int D>
cudaError_t select_dim(SelectParams& p, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const bool scores = p.most > p.topk;
  if (scores && (e = score_launch<D>(p, s)) != cudaSuccess) return e;
  if (p.most <= 512) {
    KVQ_LAUNCH("select_kernel", s, e = (select_launch<D, 32, 16>(p, scores, s)));
  } else if (p.most <= 1024) {
    KVQ_LAUNCH("select_kernel", s, e = (select_launch<D, 32, 32>(p, scores, s)));
  } else if (p.most <= 4096) {
    KVQ_LAUNCH("select_kernel", s, e = (select_launch<D, 256, 16>(p, scores, s)));
  } else {
    KVQ_LAUNCH("select_kernel", s, e = (select_launch<D, 1024, 32>(p, scores, s)));
  }
  return e;
}

int32_t key_pitch(int32_t most) { return (most + 31) / 32 * 32; }
int32_t sizes_pitch(int32_t most) { return (most + 15) / 16; }  // the smallest step

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
