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
// The list is that of the exact scores.  The score kernel works in binary32; its roundings stay
// within e = err * |q|_1 * max |bound|  (err counts them, 2^-24 each, with the sum over the heads;
// |q|_1 over all heads).  A score above the best unlisted one by more than 2 e is listed for certain, one below
// the lowest listed one by as much is not; what lies between is scored again in binary64, by one
// warp a block, and ranked by the upper and then the lower bits of that.  A few blocks of
// some rows are; exact ties go the same way to the index.  What binary32 cannot bound (sums that
// may overflow) all goes to binary64.
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
constexpr int kScoreBlocks = 32 * kScoreWarps;  // cache blocks of a thread block

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

__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Scores of 128 blocks of one (sequence, KV head) for all its query tokens: a warp reads one
// block's bounds with one load a lane, 8 blocks in flight, and adds up 8 sums over its lanes by
// 9 shuffles (halving the sums with the lanes).
template <int D>
__global__ void __launch_bounds__(32 * kScoreWarps) score_kernel(const SelectParams p) {
  constexpr int kC = D / 16;  // values of a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = blockIdx.x, h = blockIdx.y, s = blockIdx.z;
  __shared__ __align__(16) float coef[kScoreQueries][2 * D];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int q0, n, len;
  if (!select_range(p, s, q0, n, len) || n == 0) return;
  const int blocks = static_cast<int>(p.div_bs.div(static_cast<uint32_t>(len - 1))) + 1;
  if (blocks <= p.topk || chunk * kScoreBlocks >= blocks) return;
  const int b0 = chunk * kScoreBlocks + 32 * warp;
  const int32_t mine = b0 + lane < blocks ? LDX(p.table + static_cast<int64_t>(s) * p.max_blocks + b0 + lane) : -1;
  const bool bad = b0 + lane < blocks && (mine < 0 || mine >= p.num_blocks);
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) set_status(p.status, 2u);
  const uint32_t have = __ballot_sync(0xFFFFFFFFu, b0 + lane < blocks && !bad);
  uint32_t top = 0u;  // largest |bound| of the lane's, packed
  for (int i0 = 0; i0 < n; i0 += kScoreQueries) {
    const int ni = min(kScoreQueries, n - i0);
    if (i0 > 0) __syncthreads();
    for (int at = threadIdx.x; at < ni * D; at += 32 * kScoreWarps) {
      const int i = at / D, d = at - i * D;
      const uint16_t* const x = p.q + static_cast<int64_t>(q0 + i0 + i) * p.q_row_pitch +
                                static_cast<int64_t>(h) * p.group * p.q_head_pitch + d;
      float minus = 0.0f, plus = 0.0f;
      for (int j = 0; j < p.group; ++j) {
        const float v = __uint_as_float(static_cast<uint32_t>(LDX(x + j * p.q_head_pitch)) << 16);
        minus = __fadd_rn(minus, v < 0.0f || isnan(v) ? v : 0.0f);
        plus = __fadd_rn(plus, v > 0.0f ? v : 0.0f);
      }
      coef[i][d] = minus;
      coef[i][D + d] = plus;
    }
    __syncthreads();
    for (int g8 = 0; g8 < 4; ++g8) {
      if (b0 + 8 * g8 >= blocks) break;
      uint32_t w[8][D / 32];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int32_t blk = __shfl_sync(0xFFFFFFFFu, mine, 8 * g8 + j);
        if ((have >> (8 * g8 + j)) & 1u) {
          load_bounds<D>(p.bounds + (static_cast<int64_t>(blk) * p.H + h) * (2 * D) + lane * kC, w[j]);
        } else {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) w[j][i] = 0u;
        }
      }
      if (i0 == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < D / 32; ++i) asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(top) : "r"(top), "r"(w[j][i]));
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
              (have >> (8 * g8 + j)) & 1u ? score_key(v[0]) : kKeyBad);
      }
    }
  }
  top &= 0x7FFF7FFFu;
  float m = fmaxf(bf16lo(top), bf16hi(top));
  m = group_max<32>(m);
  if (lane == 0) STX(p.tops + (static_cast<int64_t>(q0) * p.H + h) * p.tops_pitch + chunk * kScoreWarps + warp, m);
}

// Sums, maxima or minima over a thread block, the same in all threads; one barrier each (the
// slots alternate).
template <int kThreads>
struct BlockReduce {
  uint32_t (*slot)[32];
  int turn;
  template <typename F>
  __device__ __forceinline__ uint32_t run(uint32_t v, F warp_reduce, uint32_t none) {
    constexpr int kWarps = kThreads / 32;
    v = warp_reduce(v);
    uint32_t* const at = slot[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_reduce(lane < kWarps ? at[lane] : none);
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
};

// The border of the k highest keys: at least k keys are >= hi, fewer are above it; lo is the
// largest key below hi (0: none) where exactly k are, else hi.
struct Border {
  uint32_t hi, lo, count;
};
template <int kThreads, int P>
__device__ __forceinline__ Border find_border(const uint32_t (&key)[P], uint32_t k, BlockReduce<kThreads>& red) {
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

// The list of one (query token, KV head): thread t holds the keys of P blocks from t P on.
// A search by halves over the keys' range finds the border (it ends as soon as a bound parts k keys
// from the rest).  Bound: latency, some 15 rounds of a count over the thread block.
template <int D, int kThreads, int P>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p) {
  constexpr int kC = D / 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = static_cast<int>(blockIdx.x) / p.H, h = static_cast<int>(blockIdx.x) - i * p.H, s = blockIdx.y;
  __shared__ uint32_t slots[2][32];
  BlockReduce<kThreads> red{slots, 0};
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
    for (int j = threadIdx.x; j < p.topk; j += kThreads) STX(out + j, j < vis ? j : -1);
    return;
  }
  // blocks below `head` and from `tail` on are listed in any case
  const int head = min(p.first, vis), tail = max(vis - p.last, head);
  const uint32_t k = static_cast<uint32_t>(p.topk - head - (vis - tail));
  const int b0 = threadIdx.x * P;
  uint32_t key[P];
#pragma unroll
  for (int j = 0; j < P; j += 4) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (b0 + j < vis) v = LDX(reinterpret_cast<const uint4*>(p.keys + row * p.pitch + b0 + j));
    key[j] = v.x, key[j + 1] = v.y, key[j + 2] = v.z, key[j + 3] = v.w;
  }
#pragma unroll
  for (int j = 0; j < P; ++j)
    if (b0 + j < head || b0 + j >= tail) key[j] = 0u;  // out of the search

  uint32_t listed = 0u;  // bits of this thread's blocks
  if (k > 0u) {
    // |q|_1 over the heads and the largest bound: the error bound of the binary32 scores
    float q1 = 0.0f, top = 0.0f;
    for (int at = lane; at < p.group * (D / 8); at += 32) {
      const int j = at / (D / 8), d = 8 * (at - j * (D / 8));
      uint32_t v[4];
      load16B(p.q + (q0 + i) * p.q_row_pitch + (static_cast<int64_t>(h) * p.group + j) * p.q_head_pitch + d, v);
#pragma unroll
      for (int x = 0; x < 4; ++x) q1 += fabsf(bf16lo(v[x])) + fabsf(bf16hi(v[x]));
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) q1 += __shfl_xor_sync(0xFFFFFFFFu, q1, o);
    const float* const tops = p.tops + (static_cast<int64_t>(q0) * p.H + h) * p.tops_pitch;
    for (int at = lane; at < (vis + 31) / 32; at += 32) top = fmaxf(top, LDX(tops + at));
    top = group_max<32>(top);
    const float size = q1 * top;
    // + 2^-130: roundings below the normal numbers.  NaN and what may overflow: no bound
    const float e = size <= 1e38f ? (size > 0.0f ? size * p.err + 0x1p-130f : 0.0f) : __int_as_float(0x7F800000);

    Border at = find_border<kThreads, P>(key, k, red);
    const bool bounded = !isinf(e), scored = at.hi > kKeyNan;  // not: blocks without a score fill the list
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
      const int d0 = (lane % 16) * kC;
      auto load_q = [&]() {
#pragma unroll
        for (int x = 0; x < kC; ++x) qd[x] = 0.0;
        for (int j = 0; j < p.group; ++j)
#pragma unroll
          for (int x = 0; x < kC; ++x) {
            const float v = __uint_as_float(static_cast<uint32_t>(LDX(
                                p.q + (q0 + i) * p.q_row_pitch + (static_cast<int64_t>(h) * p.group + j) * p.q_head_pitch + d0 + x))
                                            << 16);
            qd[x] += (lane < 16 ? v < 0.0f || isnan(v) : v > 0.0f) ? static_cast<double>(v) : 0.0;
          }
      };
      load_q();
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
    uint32_t above = 0u, ties = 0u;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      if (key[j] > at.hi) listed |= 1u << j;
      if (key[j] == at.hi) ties |= 1u << j;
    }
    above = red.sum(__popc(listed));
    uint32_t need = k - above;
    if (at.count > k) {  // uniform
      const uint32_t mine = __popc(ties);
      uint32_t upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += y;
      }
      __syncthreads();
      if (lane == 31) slots[0][warp] = upto;
      __syncthreads();
      uint32_t before = upto - mine;
      for (int x = 0; x < warp; ++x) before += slots[0][x];
      __syncthreads();
      for (; ties != 0u; ties &= ties - 1u, ++before)
        if (before < need) listed |= ties & (0u - ties);
    } else {
      listed |= ties;
    }
  }
#pragma unroll
  for (int j = 0; j < P; ++j)
    if (b0 + j < vis && (b0 + j < head || b0 + j >= tail)) listed |= 1u << j;
  const uint32_t mine = __popc(listed);
  uint32_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += y;
  }
  __syncthreads();
  if (lane == 31) slots[0][warp] = upto;
  __syncthreads();
  uint32_t before = upto - mine;
  for (int x = 0; x < warp; ++x) before += slots[0][x];
  for (; listed != 0u; listed &= listed - 1u, ++before) STX(out + before, b0 + __ffs(listed) - 1);
}

template <int D, int kThreads, int P>
cudaError_t select_launch(const SelectParams& p, bool dependent, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(p.max_q) * p.H), static_cast<unsigned>(p.S));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, select_kernel<D, kThreads, P>, p);
}

template <int D>
cudaError_t select_dim(const SelectParams& p, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const bool scores = p.most > p.topk;
  if (scores) {
    const dim3 grid(static_cast<unsigned>((p.most + kScoreBlocks - 1) / kScoreBlocks), p.H, p.S);
    KVQ_LAUNCH("score_kernel", s, score_kernel<D><<<grid, 32 * kScoreWarps, 0, s>>>(p); e = cudaGetLastError());
    if (e != cudaSuccess) return e;
  }
  if (p.most <= 512) {
    KVQ_LAUNCH("select_kernel", s, e = (select_launch<D, 128, 4>(p, scores, s)));
  } else if (p.most <= 4096) {
    KVQ_LAUNCH("select_kernel", s, e = (select_launch<D, 256, 16>(p, scores, s)));
  } else {
    KVQ_LAUNCH("select_kernel", s, e = (select_launch<D, 1024, 32>(p, scores, s)));
  }
  return e;
}

int32_t key_pitch(int32_t most) { return (most + 31) / 32 * 32; }
int64_t tops_pitch(int32_t most) { return static_cast<int64_t>(most + kScoreBlocks - 1) / kScoreBlocks * kScoreWarps; }

}  // namespace

// Keys of every (token, head), then the largest bounds of each 32 blocks of every (sequence,
// head), under the sequence's first token.
size_t select_workspace_bytes(int32_t T, int32_t H, int32_t most) {
  if (T <= 0 || H <= 0 || most <= 0) return 0;
  return static_cast<size_t>(T) * H * (key_pitch(most) + static_cast<size_t>(tops_pitch(most))) * 4;
}

cudaError_t launch_select_blocks(const SelectParams& p_in, void* workspace, cudaStream_t s) {
  SelectParams p = p_in;
  p.pitch = key_pitch(p.most);
  p.tops_pitch = static_cast<int32_t>(tops_pitch(p.most));
  p.keys = static_cast<uint32_t*>(workspace);
  p.tops = reinterpret_cast<float*>(p.keys + static_cast<int64_t>(p.num_tokens) * p.H * p.pitch);
  // roundings on a product's way into a score, of 2^-24 each: the sum over the heads, a chain of
  // D / 32 products, the two chains' sum and 5 steps over the lanes; two more and a fiftieth for those
  // of |q|_1, of the bound itself and of the comparisons with it
  p.err = 1.02f * static_cast<float>(p.group + p.D / 32 + 8) * 0x1p-24f;
  switch (p.D) {
    case 64: return select_dim<64>(p, s);
    case 128: return select_dim<128>(p, s);
    case 256: return select_dim<256>(p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
