// page_scale_kernels.cu -- scatter into an FP8 cache with one scale per (block, head).
//
// A page is block_size tokens of one head; its scale s is a power of two, so x / s is
// exact and E4M3 keeps the relative precision that a scale of amax / 448 would give (a
// float code loses nothing but its smallest binade to the factor below 2).  For the rows
// that a call writes into a page, with s0 the page's stored scale (none where the call
// writes the page's first slot, which starts the page over):
//   need = the smallest power of two with amax <= 448 need (at least 2^-126), amax the largest
//          finite |x| (an infinity saturates: as part of amax it would round the page's other rows
//          to 0 for good)
//   s    = max(s0, need)
//   code = E4M3(x / s);  the page's other rows, where s > s0 > 0:  E4M3(code * (s0 / s))
// The second rounding of a held row is exact but for codes that fall below E4M3's normal
// range.  Each raise of the scale rounds those again, so a page filled token by token holds
// what one call would have written, or is off by one subnormal step of the final scale.
//
// Mapping: rows of one page that stand next to each other in slot_ids form a run; one
// warp serves (run, head, tensor), so no two warps write one (page, head) and no atomics
// are needed.  L = D / 16 lanes (rounded up to a power of two) read a row as 32 bytes
// each; 32 / L rows go at once, and the first kHold such passes stay in registers between
// the maximum and the codes, so pages up to 8 * 32 / L rows are read once.
// Bound: HBM, 2 D bytes read and D written per row.  Measured: 37 prompts of 55,500 tokens in
// all, 8 heads, head_dim 128, 32-token pages: 63.2 us, 5.40 TB/s, 80% of a plain copy's rate;
// 64 single tokens into half-filled pages 3.3 us, one launch and one chain of loads.  More
// resident blocks (fewer registers, 102 against 72 us with events around each call) measured
// slower.
#include "kvq_device.cuh"
#include "kvq_params.h"

namespace kvq {

namespace {

constexpr int kPageThreads = 128;
constexpr int kHold = 8;  // passes kept in registers (64 registers)

// The smallest power of two s >= 2^-126 with amax <= 448 s (448 = 1.75 * 2^8).
__device__ __forceinline__ float page_scale_need(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < 1 ? 1 : e;  // also for a subnormal amax
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// Four E4M3 codes times f (a power of two unless the stored scale was not one).
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h2;
    const uint16_t two = static_cast<uint16_t>((w >> (16 * i)) & 0xFFFFu);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
    float lo, hi;
    f16x2_to_f32(h2, lo, hi);
    r |= e4m3x2_from_f32(__fmul_rn(lo, f), __fmul_rn(hi, f)) << (16 * i);
  }
  return r | (w & 0x80808080u);  // a NaN code (a row never written) keeps its sign too
}

__device__ __forceinline__ int run_bits(uint32_t m) { return m == 0xFFFFFFFFu ? 32 : __ffs(~m) - 1; }

template <int L, bool kV8>
__global__ void __launch_bounds__(kPageThreads) page_encode_kernel(const PageEncodeParams p) {
  constexpr int R = 32 / L;  // rows per pass
  const int lane = threadIdx.x & 31;
  const int li = lane % L, sub = lane / L;
  const bool act = li < p.nb;
  // warp -> (chunk, tensor, head), heads fastest: neighbouring warps read neighbouring rows
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kPageThreads / 32) + (threadIdx.x >> 5);
  const int per = p.H * p.ntensors;
  const int64_t ci = w / per;
  const int rem = static_cast<int>(w - ci * per);
  const int tensor = rem / p.H, h = rem - tensor * p.H;
  const int64_t t0 = ci * p.chunk;
  if (t0 >= p.T) return;
  const EncodeTensor ten = p.ten[tensor];

  // pages of tokens t0 - 1 .. t0 + 31 (-1: skipped)
  auto slot_of = [&](int64_t t) -> int64_t {
    if (t < 0 || t >= p.T) return -1;
    const int64_t s = LDX(p.slot_ids + t);
    if (s >= p.num_slots) {
      if (rem == 0) set_status(p.status, 1u);
      return -1;
    }
    return s;
  };
  auto page_of = [&](int64_t slot) -> int64_t { return slot < 0 ? -1 : slot / p.block_size; };
  const int64_t slot = slot_of(t0 + lane);
  const int64_t before = lane == 0 ? page_of(slot_of(t0 - 1)) : -1;
  const int64_t page = page_of(slot);
  int64_t prev = __shfl_up_sync(0xFFFFFFFFu, page, 1);
  if (lane == 0) prev = before;
  uint32_t leaders = __ballot_sync(0xFFFFFFFFu, lane < p.chunk && page >= 0 && page != prev);
  const uint32_t firsts = __ballot_sync(0xFFFFFFFFu, page >= 0 && slot - page * p.block_size == 0);

  while (leaders != 0u) {
    const int b = __ffs(leaders) - 1;
    leaders &= leaders - 1;
    const int64_t pg = __shfl_sync(0xFFFFFFFFu, page, b);
    const int64_t ts = t0 + b;
    // run length, and whether it holds the page's first slot
    int n = run_bits(__ballot_sync(0xFFFFFFFFu, page == pg) >> b);  // zeros come in from the top
    bool begins = ((firsts >> b) & (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u)) != 0u;
    if (b + n == 32) {
      for (int64_t t = t0 + 32; t < p.T; t += 32) {
        const int64_t s2 = slot_of(t + lane);
        const int64_t p2 = page_of(s2);
        const int m = run_bits(__ballot_sync(0xFFFFFFFFu, p2 == pg));
        begins = begins || __any_sync(0xFFFFFFFFu, lane < m && s2 == pg * p.block_size);
        n += m;
        if (m < 32) break;
      }
    }
    float* const sp = ten.dst.rscale + pg * p.H + h;
    float s0 = 0.0f;
    if (!begins && lane == 0) s0 = LDX(sp);
    s0 = __shfl_sync(0xFFFFFFFFu, s0, 0);
    const uint16_t* const x = ten.x + ts * ten.row_pitch + h * ten.head_pitch + 16 * li;

    uint32_t hold[kHold][8];
    float am = 0.0f;
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      const int r = k * R + sub;
#pragma unroll
      for (int i = 0; i < 8; ++i) hold[k][i] = 0u;
      if (act && r < n) load32B<kV8, true>(x + r * ten.row_pitch, hold[k]);
    }
#pragma unroll
    for (int k = 0; k < kHold; ++k) am = fmaxf(am, absmax16(hold[k]));
    for (int r = kHold * R + sub; r < n; r += R) {
      uint32_t v[8];
      if (act) {
        load32B<kV8, true>(x + r * ten.row_pitch, v);
        am = fmaxf(am, absmax16(v));
      }
    }
    am = group_max<32>(am);
    if (am > 3.4028235e38f) {  // an infinity among them, the same in all lanes: once more without
      am = 0.0f;
      for (int r = sub; r < n; r += R) {
        uint32_t v[8];
        if (!act) continue;
        load32B<kV8, true>(x + r * ten.row_pitch, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float lo = fabsf(bf16lo(v[i])), hi = fabsf(bf16hi(v[i]));
          am = fmaxf(am, fmaxf(lo <= 3.4028235e38f ? lo : 0.0f, hi <= 3.4028235e38f ? hi : 0.0f));
        }
      }
      am = group_max<32>(am);
    }
    if (!(s0 > 0.0f && s0 <= 3.4028235e38f)) s0 = 0.0f;  // no scale stored yet
    const float need = page_scale_need(am);
    const float s = fmaxf(s0, need);
    uint8_t* const cp = ten.dst.codes + ((pg * p.block_size) * p.H + h) * (16 * p.nb) + 16 * li;
    const int64_t cpitch = static_cast<int64_t>(p.H) * 16 * p.nb;
    if (s0 > 0.0f && s > s0) {  // the rows that the page holds, under the new scale
      const float f = __fdiv_rn(s0, s);
      for (int r = sub; r < p.block_size; r += R) {
        if (!act) continue;
        uint32_t c[4];
        load16B_rw(cp + r * cpitch, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = rescale4(c[i], f);
        store16B(cp + r * cpitch, c);
      }
      __syncwarp();  // before the call's own rows go over them
    }
    if (lane == 0 && s != s0) STX(sp, s);
    const float inv = __frcp_rn(s);
    auto put = [&](const uint32_t (&v)[8], int r) {
      const int64_t off = LDX(p.slot_ids + ts + r) - pg * p.block_size;
      uint32_t c[4];
      fp8_quantize16(v, s, inv, c);
      store16B(cp + off * cpitch, c);
    };
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      const int r = k * R + sub;
      if (act && r < n) put(hold[k], r);
    }
    for (int r = kHold * R + sub; r < n; r += R) {
      uint32_t v[8];
      if (act) {
        load32B<kV8, true>(x + r * ten.row_pitch, v);
        put(v, r);
      }
    }
  }
}

template <int L, bool kV8>
cudaError_t page_launch_encode(const PageEncodeParams& p_in, cudaStream_t s) {
  PageEncodeParams p = p_in;
  auto k = page_encode_kernel<L, kV8>;
  // tokens per warp: as many as leave 16 warps an SM (one token a warp in a decode step,
  // whose runs are single rows; 32 in a prompt)
  const int64_t rows = static_cast<int64_t>(p.T) * p.H * p.ntensors;
  p.chunk = 32;
  while (p.chunk > 1 && rows < static_cast<int64_t>(p.chunk) * 16 * num_sms()) p.chunk >>= 1;
  const int64_t warps = (static_cast<int64_t>(p.T) + p.chunk - 1) / p.chunk * p.H * p.ntensors;
  const int64_t blocks = (warps + kPageThreads / 32 - 1) / (kPageThreads / 32);
  cudaError_t e = cudaSuccess;
  KVQ_LAUNCH("page_encode_kernel", s, k<<<static_cast<unsigned>(blocks), kPageThreads, 0, s>>>(p);
             e = cudaGetLastError());
  return e;
}

}  // namespace

cudaError_t launch_page_encode(const PageEncodeParams& p, bool v8, cudaStream_t s) {
  int L = 1;
  while (L < p.nb) L <<= 1;
#define KVQ_PAGE(N) \
  if (L == N) return v8 ? page_launch_encode<N, true>(p, s) : page_launch_encode<N, false>(p, s);
  KVQ_PAGE(1) KVQ_PAGE(2) KVQ_PAGE(4) KVQ_PAGE(8) KVQ_PAGE(16) KVQ_PAGE(32)
#undef KVQ_PAGE
  return cudaErrorInvalidValue;
}

}  // namespace kvq
