// attn_tile.cuh -- the tile arithmetic that the paged attention kernels share: one
// 16-token tile of one KV head, dequantised in registers, against up to 16 query rows
// (mma.sync m16n8k16, f16 operands, f32 accumulators).  The layout of the operands is
// described at the head of attn_kernels.cu.
#pragma once

#include "kvq_device.cuh"
#include "kvq_params.h"

namespace kvq {

namespace {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kNoKey = -1e30f;  // the softmax reference before the first key, under a mask

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Both E4M3 bytes of `two` (low byte -> low half) to f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  const uint16_t in = static_cast<uint16_t>(two & 0xFFFFu);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(in));
  return r;
}

// The four E2M1 pairs of a word, byte i -> f16x2 i (low nibble in the low half),
// exactly; the bytes go to the conversions as .b8 registers (no shifts or masks).
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// The two E4M3 pairs of a word, bytes 0-1 -> f16x2 0 and bytes 2-3 -> f16x2 1, exactly.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t (&h)[2]) {
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(w));
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The same with results below 2^-126 flushed to zero: used for probabilities, whose
// row sum is at least 1, so a flushed term is below the sum's own rounding.
__device__ __forceinline__ float ex2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Asynchronous 4- / 8-byte copies into shared memory (cp.async.ca; 16-byte copies use
// cp_async16).  The checked build stores zeros instead of copying from outside a
// registered range.
template <int N>
__device__ __forceinline__ void cp_async_small(void* smem_dst, const void* gsrc) {
  static_assert(N == 4 || N == 8, "4 or 8 bytes");
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(smem_dst));
  if (!KVQ_OK(gsrc, N, N)) {
    if constexpr (N == 4) {
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(d), "r"(0u) : "memory");
    } else {
      asm volatile("st.shared.v2.b32 [%0], {%1, %1};" ::"r"(d), "r"(0u) : "memory");
    }
    return;
  }
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(gsrc), "n"(N) : "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_n(void* smem_dst, const void* gsrc) {
  if constexpr (N == 16) {
    cp_async16(smem_dst, gsrc);
  } else {
    cp_async_small<N>(smem_dst, gsrc);
  }
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int src) {
  const int lo = __shfl_sync(0xFFFFFFFFu, static_cast<int>(v & 0xFFFFFFFF), src);
  const int hi = __shfl_sync(0xFFFFFFFFu, static_cast<int>(v >> 32), src);
  return (static_cast<int64_t>(hi) << 32) | static_cast<uint32_t>(lo);
}

// Shared-memory layout of one 16-token tile of one KV head (both K and V).  Row
// strides are chosen so that each access phase of a warp covers 32 distinct banks:
// a K read is one lane's contiguous chunk (D/8 or D/4 bytes at lane c's offset) of
// token 8j + g; a V read is D/16 or D/8 bytes at lane g's offset of token 2c (+1,
// +8, +9), which needs a row stride of 4 mod 16 words (the code bytes + 16).
template <int D, int kFK, int kFV>
struct AttnTile {
  static constexpr int kCK = kFK == 3 ? D : D / 2;  // code bytes per row
  static constexpr int kCV = kFV == 3 ? D : D / 2;
  static constexpr int kSK = kFK == 3 ? (D == 128 ? 144 : D) : (D == 256 ? 144 : D / 2);  // smem row strides
  static constexpr int kSV = kCV + 16;
  static constexpr int kBK = kFK == 3 ? 0 : D / 16;  // block-scale bytes per row
  static constexpr int kBV = kFV == 3 ? 0 : D / 16;
  static constexpr int kOffKC = 0;
  static constexpr int kOffVC = kOffKC + 16 * kSK;
  static constexpr int kOffKB = kOffVC + 16 * kSV;
  static constexpr int kOffVB = kOffKB + 16 * kBK;
  static constexpr int kOffKR = kOffVB + 16 * kBV;
  static constexpr int kOffVR = kOffKR + 64;
  static constexpr int kBytes = kOffVR + 64;
  static constexpr int kStages = kBytes > 4096 ? 3 : 4;
  static constexpr int kRing = kAttnWarps * kStages * kBytes;
  // per warp: up to 16 query heads x (O, m, l); Q^T fragments [n-tile][k-step][lane]
  // (8 B each, up to two n-tiles) + up to 16 head factors
  static constexpr int kMerge = kAttnWarps * 16 * (D + 2) * 4;
  static constexpr int kQ = (D / 16) * 32 * 16 + 64;
  static constexpr int kSmem = kQ + (kRing > kMerge ? kRing : kMerge);
};

// NW words from shared memory at p (aligned to the access), in 16-, 8- or 4-byte loads.
template <int NW>
__device__ __forceinline__ void lds_words(const unsigned char* p, uint32_t (&w)[NW]) {
  if constexpr (NW % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NW / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  } else if constexpr (NW == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// Transpose of an 8x8 f16 matrix held as one m16n8 fragment quarter: lane (g, c) gives
// row g, columns 2c and 2c + 1, and receives row g, columns 2c and 2c + 1 of the
// transpose.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Shared-memory view of one 16-token tile of one KV head: the code, block-scale and row
// scale rows of token i start at kc / vc / kb / vb / kr / vr + i * stride (bytes; the
// scale strides are 0 where the tile lies in one page of a page-scaled plane).
struct TileView {
  const unsigned char *kc, *vc, *kb, *vb, *kr, *vr;
  int sk, sv, sbk, sbv, skr, svr;
};

// Score modifier of a tile: none (one query token that sees every key of its sequence).
struct NoMod {
  static constexpr bool kActive = false;
  __device__ __forceinline__ void operator()(float (&)[1][4]) const {}
};

// A warp's running softmax state over its tiles: per head (8nh + 2c + e) the reference
// m (mlag: the logit from which on it moves), the partial sum l of this lane's tokens, the V
// row-scale reference R (Rlag: the scale from which on it moves, rR = 1 / R), and the O^T
// accumulators o[mt][nh] (dims g*D/8 + 2mt, e = 0, 1, and + 1, e = 2, 3, of heads 8nh + 2c and
// + 1), relative to R.
// Under a mask R may come from rows of V that a query does not see.  A query whose own V scales
// are 2^kLagR and more below R takes m lower by the difference in powers of two (its shift), so
// that P' keeps its precision; mlag tells the reference of its logits.  While any query of the
// warp is shifted, every tile sets the references anew.  (Where all rows see the same keys, as the
// heads of one token do, none of this runs: in every tile that moves m it cost 5%.)
template <int D, int kNH>
struct AttnState {
  float m[kNH][2], mlag[kNH][2], l[kNH][2], R, Rlag, rR;
  bool shifted;
  float o[D / 16][kNH][4];
  // m0: the reference before any key; finite where a tile may hold no key that a row sees
  __device__ __forceinline__ void init(float m0 = kNegInf) {
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh) {
      m[nh][0] = m[nh][1] = mlag[nh][0] = mlag[nh][1] = m0;
      l[nh][0] = l[nh][1] = 0.0f;
    }
    R = Rlag = rR = 0.0f;
    shifted = false;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int nh = 0; nh < kNH; ++nh) o[mt][nh][0] = o[mt][nh][1] = o[mt][nh][2] = o[mt][nh][3] = 0.0f;
  }
};

// One 16-token tile of one KV head into the warp's state: S^T = K Q^T, the softmax
// update, O^T += V^T P'^T.  nvalid = tokens of the tile inside the sequence (16 but on
// a split's last tile), nfirst those before it (active mods only); the rest of the tile
// may hold anything, NaN codes and scales among it.  qb(nh, kb) gives the Q^T fragment, qmul the per-head query factors (scale,
// log2 e, Q's power of two).  An active mod turns the scores (rows 8nh + 2c and + 1,
// tokens g and g + 8) into base-2 logits with the masked ones at -inf; qmul is then 1.
//
// How far the references lag: m is set kUp below a row's largest logit and moves when a tile
// exceeds that by kLag, R when a V scale exceeds it by 2^kLagR, so P' = exp2(s - m) * rs_v / R
// stays below 2^14 and f16 holds it, and O is rescaled on few tiles.  A key whose P' falls below
// f16's 2^-25 counts in the row sum but not in O: below 2^-31 of the largest weight with a
// modifier, whose rows may look back over a whole long cache in one block, 2^-25 without.
template <int D, int kFK, int kFV, int kNH, typename QB, typename Mod>
__device__ __forceinline__ void attn_tile(const TileView& tv, const QB& qb, const float (&qmul)[kNH][2], int lane,
                                          int nvalid, AttnState<D, kNH>& st, const Mod& mod, int nfirst = 0) {
  constexpr int kKS = D / 16;
  constexpr int kMT = D / 16;
  constexpr int kUp = Mod::kActive ? 6 : 0, kLag = Mod::kActive ? 4 : 8, kLagR = Mod::kActive ? 4 : 6;
  const int g = lane >> 2;
  const int c = lane & 3;
  // S^T = K Q^T: rows g and g + 8 are tokens g and 8 + g (this lane's K rows), each
  // K fragment serves every head n-tile
  float sc[kNH][4];
#pragma unroll
  for (int nh = 0; nh < kNH; ++nh) sc[nh][0] = sc[nh][1] = sc[nh][2] = sc[nh][3] = 0.0f;
  if constexpr (kFK == 3) {
    uint32_t kw[2][D / 16];  // this lane's D/4 code bytes of tokens g and 8 + g
    lds_words<D / 16>(tv.kc + g * tv.sk + c * (D / 4), kw[0]);
    lds_words<D / 16>(tv.kc + (8 + g) * tv.sk + c * (D / 4), kw[1]);
#pragma unroll
    for (int kb = 0; kb < kKS; ++kb) {
      uint32_t k0[2], k1[2];
      e4m3x4_to_f16x2(kw[0][kb], k0);  // dims 4kb, 4kb+1 | 4kb+2, 4kb+3
      e4m3x4_to_f16x2(kw[1][kb], k1);
      const uint32_t a[4] = {k0[0], k1[0], k0[1], k1[1]};
#pragma unroll
      for (int nh = 0; nh < kNH; ++nh) {
        const uint2 b = qb(nh, kb);
        mma_f16_16816(sc[nh], a, b.x, b.y);
      }
    }
  } else {
    uint32_t kw[2][D / 32];  // this lane's D/8 code bytes of tokens g and 8 + g
    lds_words<D / 32>(tv.kc + g * tv.sk + c * (D / 8), kw[0]);
    lds_words<D / 32>(tv.kc + (8 + g) * tv.sk + c * (D / 8), kw[1]);
    constexpr int kNB = D / 64 > 0 ? D / 64 : 1;  // blocks of this lane's dims
    uint32_t bsb[2][kNB];                         // their scales, f16 in both halves
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint8_t* kbs = tv.kb + (8 * j + g) * tv.sbk + c * (D / 64);
      if constexpr (kNB == 1) {
        const uint32_t bsh = e4m3_to_f16x2(kbs[0]) & 0xFFFFu;
        bsb[j][0] = bsh | (bsh << 16);
      } else {  // pairs of scale bytes, one conversion each, halves spread by a permute
#pragma unroll
        for (int i = 0; i < kNB; i += 2) {
          const uint32_t two = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(kbs + i));
          bsb[j][i] = __byte_perm(two, 0u, 0x1010);
          bsb[j][i + 1] = __byte_perm(two, 0u, 0x3232);
        }
      }
    }
#pragma unroll
    for (int wi = 0; wi < D / 32; ++wi) {  // one code word = k-steps 2wi and 2wi + 1
      uint32_t hk[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        e2m1x8_to_f16x2(kw[j][wi], hk[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) hk[j][i] = hmul2(hk[j][i], bsb[j][(2 * wi) / 4]);
      }
#pragma unroll
      for (int hs = 0; hs < 2; ++hs) {
        const uint32_t a[4] = {hk[0][2 * hs], hk[1][2 * hs], hk[0][2 * hs + 1], hk[1][2 * hs + 1]};
#pragma unroll
        for (int nh = 0; nh < kNH; ++nh) {
          const uint2 b = qb(nh, 2 * wi + hs);
          mma_f16_16816(sc[nh], a, b.x, b.y);
        }
      }
    }
  }
  // scores times K's row scale; the query factor (scale, log2 e, Q's power of two,
  // positive) enters with the reference in one FMA below, and the maxima are scaled
  // by it once.  Tokens past the end are masked (only a split's last tile can hold
  // any).
  const float kr0 = *reinterpret_cast<const float*>(tv.kr + g * tv.skr);
  const float kr1 = *reinterpret_cast<const float*>(tv.kr + (g + 8) * tv.skr);
  float vr0 = *reinterpret_cast<const float*>(tv.vr + g * tv.svr);
  float vr1 = *reinterpret_cast<const float*>(tv.vr + (g + 8) * tv.svr);
  // tokens outside the sequence (a split's first and last tiles only)
  const bool edge = nvalid < 16 || (Mod::kActive && nfirst > 0);
  const bool dead0 = g >= nvalid || (Mod::kActive && g < nfirst);
  const bool dead1 = g + 8 >= nvalid || (Mod::kActive && g + 8 < nfirst);
  // this lane's maxima (two tokens per head) first: the references move when any
  // lane's exceed them, and only then are the tile's maxima reduced across lanes
  float mt[kNH][2];
  bool move = false;
#pragma unroll
  for (int nh = 0; nh < kNH; ++nh) {
    sc[nh][0] *= kr0;
    sc[nh][1] *= kr0;
    sc[nh][2] *= kr1;
    sc[nh][3] *= kr1;
  }
  if constexpr (Mod::kActive) mod(sc);
  if (edge) {  // uniform
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh) {
      if (dead0) sc[nh][0] = sc[nh][1] = kNegInf;
      if (dead1) sc[nh][2] = sc[nh][3] = kNegInf;
    }
    if (dead0) vr0 = 0.0f;
    if (dead1) vr1 = 0.0f;
    if constexpr (kFV != 3) {
      // 0 * NaN would reach O (E2M1 holds no NaN, a block scale may): V's block scales of tokens
      // outside become 0 where they lie, in rows that no other warp reads.  (Masked in
      // registers, in the loop below, they cost every tile 2.6% of the decode kernel's time.)
      if (lane < 16 && (lane >= nvalid || (Mod::kActive && lane < nfirst))) {
        uint32_t* const w = reinterpret_cast<uint32_t*>(const_cast<uint8_t*>(tv.vb) + lane * tv.sbv);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) w[i] = 0u;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // a copy may land here next
      }
      __syncwarp();
    }
  }
#pragma unroll
  for (int nh = 0; nh < kNH; ++nh) {
    mt[nh][0] = fmaxf(sc[nh][0], sc[nh][2]) * qmul[nh][0];
    mt[nh][1] = fmaxf(sc[nh][1], sc[nh][3]) * qmul[nh][1];
    move = move || mt[nh][0] > st.mlag[nh][0] || mt[nh][1] > st.mlag[nh][1];
  }
  float rmax = fmaxf(vr0, vr1);
  move = move || rmax > st.Rlag || (Mod::kActive && st.shifted);
  if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
    for (int off = 4; off <= 16; off <<= 1) {
#pragma unroll
      for (int nh = 0; nh < kNH; ++nh) {
        mt[nh][0] = fmaxf(mt[nh][0], __shfl_xor_sync(0xFFFFFFFFu, mt[nh][0], off));
        mt[nh][1] = fmaxf(mt[nh][1], __shfl_xor_sync(0xFFFFFFFFu, mt[nh][1], off));
      }
      rmax = fmaxf(rmax, __shfl_xor_sync(0xFFFFFFFFu, rmax, off));
    }
    // with a mask R holds until a scale exceeds it by 2^kLagR: the smallest shift then tells
    bool mixed = false;
    if constexpr (Mod::kActive) mixed = mod.mixed;
    const bool jump = !mixed || rmax > st.Rlag || st.R == 0.0f;
    const float Rn = jump ? fmaxf(fmaxf(st.R, rmax), 0x1p-126f) : st.R;
    const float rr = st.R / Rn;
    int shift[kNH][2] = {};
    bool reset = false;  // the shifts
    if (mixed) {
      reset = jump || st.shifted;
#pragma unroll
      for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
        for (int e = 0; e < 2; ++e) reset = reset || (st.m[nh][e] == kNoKey && mt[nh][e] > kNoKey);
      reset = __any_sync(0xFFFFFFFFu, reset);
      if (reset) {
        auto exponent = [](float x) { return static_cast<int>(__float_as_uint(x) >> 23); };
        bool any = false;
#pragma unroll
        for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // the largest scale that the query sees in this tile, and saw before
            float own = fmaxf(sc[nh][e] > kNegInf ? vr0 : 0.0f, sc[nh][2 + e] > kNegInf ? vr1 : 0.0f);
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) own = fmaxf(own, __shfl_xor_sync(0xFFFFFFFFu, own, off));
            int top = exponent(own);
            if (st.m[nh][e] > kNoKey) {
              const float was = st.shifted ? rintf((st.mlag[nh][e] - kLag) - (st.m[nh][e] + kUp)) : 0.0f;
              top = max(top, exponent(st.R) - static_cast<int>(was));
            }
            const int below = min(exponent(Rn) - top, 100);
            shift[nh][e] = below >= kLagR && fmaxf(st.m[nh][e], mt[nh][e]) > kNoKey ? below : 0;
            any = any || shift[nh][e] > 0;
            if (st.shifted) mt[nh][e] = fmaxf(mt[nh][e], st.mlag[nh][e] - kLag);
          }
        any = __any_sync(0xFFFFFFFFu, any);
        if (!st.shifted) {
#pragma unroll
          for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
            for (int e = 0; e < 2; ++e) mt[nh][e] = fmaxf(mt[nh][e], st.m[nh][e] + kUp);
        }
        st.shifted = any;
      }
    }
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ref = reset ? mt[nh][e] : fmaxf(st.m[nh][e] + kUp, mt[nh][e]);  // of the logits
        const float mn = Mod::kActive ? ref - static_cast<float>(shift[nh][e] + kUp) : ref;
        const float a = ex2(st.m[nh][e] - mn);  // 0 while m is -inf
        const float f = a * rr;
#pragma unroll
        for (int q = 0; q < kMT; ++q) {
          st.o[q][nh][e] *= f;
          st.o[q][nh][e + 2] *= f;
        }
        st.l[nh][e] *= a;
        st.m[nh][e] = mn;
        st.mlag[nh][e] = ref + kLag;
      }
    }
    st.R = Rn;
    st.Rlag = Rn * static_cast<float>(1 << kLagR);
    st.rR = rcp_approx(Rn);
  }
  // P'^T = exp2(s - m) * rs_v / st.R, transposed in registers into the B operand of
  // O^T += V^T P'^T: pb[nh][0] holds tokens 2c, 2c + 1 of head 8nh + g, pb[nh][1]
  // tokens 2c + 8, 2c + 9
  const float r0 = vr0 * st.rR, r1 = vr1 * st.rR;
  uint32_t pb[kNH][2];
#pragma unroll
  for (int nh = 0; nh < kNH; ++nh) {
    const float p0 = ex2_ftz(__fmaf_rn(sc[nh][0], qmul[nh][0], -st.m[nh][0]));  // token g
    const float p1 = ex2_ftz(__fmaf_rn(sc[nh][1], qmul[nh][1], -st.m[nh][1]));
    const float p2 = ex2_ftz(__fmaf_rn(sc[nh][2], qmul[nh][0], -st.m[nh][0]));  // token g + 8
    const float p3 = ex2_ftz(__fmaf_rn(sc[nh][3], qmul[nh][1], -st.m[nh][1]));
    st.l[nh][0] += p0 + p2;
    st.l[nh][1] += p1 + p3;
    pb[nh][0] = transpose8x8(f32x2_to_f16x2(p0 * r0, p1 * r0));
    pb[nh][1] = transpose8x8(f32x2_to_f16x2(p2 * r1, p3 * r1));
  }
  // O^T += V^T P'^T: m-tile mt, rows g and g + 8 = dims g * D/8 + 2mt and + 1; this
  // lane supplies V for tokens (2c, 2c + 1) and (2c + 8, 2c + 9) at those dims
  {
    const int ta0 = 2 * c, ta1 = 2 * c + 8;
    if constexpr (kFV == 3) {
      uint32_t v0[D / 32], v1[D / 32], v2[D / 32], v3[D / 32];  // D/8 bytes of each token
      lds_words<D / 32>(tv.vc + ta0 * tv.sv + g * (D / 8), v0);
      lds_words<D / 32>(tv.vc + (ta0 + 1) * tv.sv + g * (D / 8), v1);
      lds_words<D / 32>(tv.vc + ta1 * tv.sv + g * (D / 8), v2);
      lds_words<D / 32>(tv.vc + (ta1 + 1) * tv.sv + g * (D / 8), v3);
      if (edge) {  // 0 * NaN would reach O: tokens outside decode to 0
        auto in = [&](int t) { return t < nvalid && (!Mod::kActive || t >= nfirst); };
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          v0[i] = in(ta0) ? v0[i] : 0u;
          v1[i] = in(ta0 + 1) ? v1[i] : 0u;
          v2[i] = in(ta1) ? v2[i] : 0u;
          v3[i] = in(ta1 + 1) ? v3[i] : 0u;
        }
      }
#pragma unroll
      for (int q = 0; q < kMT; ++q) {  // dims 2q, 2q + 1: bytes of one half word
        const int wd = q / 2, bo2 = 2 * (q % 2);
        const uint32_t sel = bo2 | ((4 + bo2) << 4) | ((bo2 + 1) << 8) | ((5 + bo2) << 12);
        uint32_t h01[2], h23[2];
        e4m3x4_to_f16x2(__byte_perm(v0[wd], v1[wd], sel), h01);
        e4m3x4_to_f16x2(__byte_perm(v2[wd], v3[wd], sel), h23);
        const uint32_t a[4] = {h01[0], h01[1], h23[0], h23[1]};
#pragma unroll
        for (int nh = 0; nh < kNH; ++nh) mma_f16_16816(st.o[q][nh], a, pb[nh][0], pb[nh][1]);
      }
    } else {
      constexpr int kW = D / 64;  // code words per lane per token (D/16 bytes)
      uint32_t v0[kW], v1[kW], v2[kW], v3[kW];
      lds_words<kW>(tv.vc + ta0 * tv.sv + g * (D / 16), v0);
      lds_words<kW>(tv.vc + (ta0 + 1) * tv.sv + g * (D / 16), v1);
      lds_words<kW>(tv.vc + ta1 * tv.sv + g * (D / 16), v2);
      lds_words<kW>(tv.vc + (ta1 + 1) * tv.sv + g * (D / 16), v3);
      // block scales of this lane's dims g * D/8 .. + D/8 - 1 for its four tokens: one
      // 16-dim block (D <= 128) or two (D = 256), as f16x2 pairs (tokens ta, ta + 1)
      constexpr int kVB = D / 8 > 16 ? D / 128 : 1;
      const uint8_t* vbs = tv.vb;
      uint32_t bs01[kVB], bs23[kVB];
#pragma unroll
      for (int q = 0; q < kVB; ++q) {
        const int blk = (g * (D / 8)) / 16 + q;
        bs01[q] = e4m3x2_to_f16x2(vbs[ta0 * tv.sbv + blk] | (vbs[(ta0 + 1) * tv.sbv + blk] << 8));
        bs23[q] = e4m3x2_to_f16x2(vbs[ta1 * tv.sbv + blk] | (vbs[(ta1 + 1) * tv.sbv + blk] << 8));
      }
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        // nibble transpose: X byte b = (dim 2(4i+b) of token a | the same dim of token
        // b << 4), Y: the odd dims; then byte b of X / Y is m-tile 4i + b, row g / g + 8
        const uint32_t x01 = (v0[i] & 0x0F0F0F0Fu) | ((v1[i] & 0x0F0F0F0Fu) << 4);
        const uint32_t y01 = ((v0[i] >> 4) & 0x0F0F0F0Fu) | (v1[i] & 0xF0F0F0F0u);
        const uint32_t x23 = (v2[i] & 0x0F0F0F0Fu) | ((v3[i] & 0x0F0F0F0Fu) << 4);
        const uint32_t y23 = ((v2[i] >> 4) & 0x0F0F0F0Fu) | (v3[i] & 0xF0F0F0F0u);
        uint32_t hx01[4], hy01[4], hx23[4], hy23[4];
        e2m1x8_to_f16x2(x01, hx01);
        e2m1x8_to_f16x2(y01, hy01);
        e2m1x8_to_f16x2(x23, hx23);
        e2m1x8_to_f16x2(y23, hy23);
#pragma unroll
        for (int bb = 0; bb < 4; ++bb) {
          const int q = 4 * i + bb;             // m-tile: dims 2q, 2q + 1, one 16-block
          const int vb = kVB == 1 ? 0 : q / 8;  // g * D/8 is a multiple of 16 when D = 256
          const uint32_t a[4] = {hmul2(hx01[bb], bs01[vb]), hmul2(hy01[bb], bs01[vb]),
                                 hmul2(hx23[bb], bs23[vb]), hmul2(hy23[bb], bs23[vb])};
#pragma unroll
          for (int nh = 0; nh < kNH; ++nh) mma_f16_16816(st.o[q][nh], a, pb[nh][0], pb[nh][1]);
        }
      }
    }
  }}

// A stage of the page-major kernels: 16 W (token, head) rows of every plane, and the ring
// that holds kStages of them.  kNH: head n-tiles of a warp (its share of the merge).
template <int D, int kFK, int kFV, int W, int kBlocks = (W == 8 ? 2 : 1), int kNH = 1, int kExtra = 0>
struct PageStage {
  static constexpr int kCK = kFK == 3 ? D : D / 2;
  static constexpr int kCV = kFV == 3 ? D : D / 2;
  static constexpr int kBK = kFK == 3 ? 0 : D / 16;
  static constexpr int kBV = kFV == 3 ? 0 : D / 16;
  static constexpr int kRow = kCK + kCV + kBK + kBV + 8;  // pool bytes per (token, KV head)
  // a stage: 16 W (token, head) rows of every plane; chunk j's rows start at 16 H j
  static constexpr int kOffKC = 0;
  static constexpr int kOffVC = kOffKC + 16 * W * kCK;
  static constexpr int kOffKB = kOffVC + 16 * W * kCV;
  static constexpr int kOffVB = kOffKB + 16 * W * kBK;
  static constexpr int kOffKR = kOffVB + 16 * W * kBV;
  static constexpr int kOffVR = kOffKR + 16 * W * 4;
  static constexpr int kBytes = kOffVR + 16 * W * 4;
  // kBlocks blocks per SM; kExtra bytes of a block go to something else
  static constexpr int kBudget = (kBlocks == 2 ? 108 * 1024 : 216 * 1024) - kExtra;
  static constexpr int kStagesFit = kBudget / kBytes;
  static constexpr int kStages = kStagesFit > 6 ? 6 : (kStagesFit < 2 ? 2 : kStagesFit);
  static constexpr int kRing = kStages * kBytes;
  // end-of-block merge: per consumer warp and lane, O (D/16 m-tiles x 4) + m, l (2 each), per n-tile
  static constexpr int kLaneFloats = kNH * ((D / 16) * 4 + 4);
  static constexpr int kMerge = W * 32 * kLaneFloats * 4;
  static constexpr int kOffBar = kRing > kMerge ? kRing : kMerge;
  static constexpr int kSmem = kOffBar + 2 * kStages * 8 + 16;  // full + empty barriers, the bad flag
};

}  // namespace

}  // namespace kvq
