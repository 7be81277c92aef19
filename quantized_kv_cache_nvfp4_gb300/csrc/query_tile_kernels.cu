// query_tile_kernels.cu -- paged attention of many query rows per KV head on tcgen05.
//
// The mathematics and the row layout are those of query_attn_kernels.cu.  A CTA takes kNT
// tiles of 128 rows (row = query token * group + query head of the group) of one KV head
// and walks the keys that any of its rows sees, kBN tokens at a time:
//   S = Q K^T   tcgen05.mma kind::f16, f16 operands in shared memory, S in tensor memory;
//   P'          softmax warps, one thread a row: p = 2^(y - M) from the logits y, their sum
//               l, P' = p * (V's scale) as f16 over S's columns of tensor memory;
//   O += P' V   P' from tensor memory, V from shared memory, O in tensor memory.
// K and V enter as the f16 values of their codes (exact: E4M3, or E2M1 times its E4M3 block
// scale); K's FP32 scale multiplies the score, V's the probability, so codes are converted
// once for kNT * 128 rows.  The reference M covers logit and V's scale together: it is set 6 below
// a tile's largest logit plus log2 of its largest V scale, and moves, and O and l are rescaled,
// only when those exceed it by 14.  P' is then 2^6 to 2^14 for the largest, which f16 holds, most
// tiles leave O alone, and keys of 2^-30 of the largest weight still count (set at the largest
// itself, half a million keys of 2^-26 behind one sink vanished from O, though not from l).
//
// Warps: 4 kNT softmax warps; one that looks the step's tokens up in the block table (any
// block size) some steps ahead; 4 producer warps, which load the rows, convert them and
// store them in the 128-byte-swizzled layout the matrix unit reads (K with the head
// dimension contiguous, V the same rows read "MN-major"); one that issues the products.  Loads of the next step are in flight in registers while the current one is
// converted.  The tiles of a CTA take turns on the tensor cores, so one's softmax runs
// while the other's products do.
//
// Bound: the softmax warps (an exponential, a maximum, a sum and a conversion for each score, and
// the waits of their tensor-memory loads), with the tensor cores busy about half the time.
// Measured at 4096 queries behind 8192 cached tokens, 8 KV heads, 32 query heads, page-scaled:
// head_dim 128 632 us, 1087 Tflop/s (56% of the library GEMM rate), 817 over NVFP4 (its block scales
// join the conversion), 860 capped (799 Tflop/s), 838 with bias; head_dim 64 559, 256 869 us.  (Row
// references that leave out hidden keys' scales, and sums that keep keys of tiny V, cost 2 to 3%
// of the plain and biased ones.)  The 14 warps of head_dim 64 and 128 leave 128 registers a thread,
// and the head_dim 128 instances spill 132 to 136 bytes.  The rows kernel took 4706 us for the
// capped one.  Other arrangements measured slower: P' kept in registers for
// one pass (1104 against 912 us at that step: spills), 16 and 32 tensor-memory columns at a time
// in two buffers (1120, 975), an issuing warp for each tile (996).
#include "query_attn.cuh"

namespace kvq {

namespace {

// ---- tcgen05 / tensor memory -------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The warp that issues the products runs its loop as a whole (addresses and descriptors are
// then uniform registers, which the instructions want; one thread's own loop measured twice
// the issue time), and one lane of it, `leader`, issues.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t leader;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
  return leader;
}
// Arrives on the mbarrier once all products issued so far by this thread are complete.
__device__ __forceinline__ void tc_commit(uint32_t leader, uint32_t mbar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %0, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(leader),
      "r"(mbar)
      : "memory");
}
// D (tensor memory) (+)= A B: both from shared memory, or A from tensor memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %0, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], %2, %3, %4, p;\n\t}" ::"r"(leader),
      "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %0, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], %3, %4, p;\n\t}" ::"r"(leader),
      "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
// 32 columns of this warp's 32 lanes, one lane a row; the wait is part of the load.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
// 64 columns: half as many waits for tensor memory as 32 at a time.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,"
      "%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,"
      "%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, "
      "[%64];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]),
        "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]),
        "=r"(v[40]), "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]),
        "=r"(v[48]), "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]),
        "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
      : "r"(taddr)
      : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[N]) {
  if constexpr (N == 64) tmem_ld64(taddr, v);
  else tmem_ld32(taddr, v);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[N]) {
  if constexpr (N == 32) tmem_st32(taddr, v);
  else tmem_st16(taddr, v);
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory operand descriptor, 128-byte swizzle: rows of 128 bytes in groups of 8
// (1024 bytes apart); `lbo` is the distance of the next 64 elements along the contiguous
// axis where that axis is M or N.
// Only the low word differs between operands, and a step along an operand adds to it.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ uint64_t smem_desc(uint32_t lo, uint32_t step_bytes) {
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
  return (static_cast<uint64_t>(hi) << 32) | (lo + (step_bytes >> 4));
}

__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t dup_f32x2(float x) { return pack_f32x2(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The larger one, NaN if either is (a select for this took 2% of the capped chunk's time).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// ---- shapes ------------------------------------------------------------------------
template <int D>
struct QTile {
  static constexpr int kBN = D == 256 ? 64 : 128;       // tokens per step
  static constexpr int kNT = D == 256 ? 1 : 2;          // 128-row tiles per CTA (tensor memory: 512 columns)
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kRows = 128 * kNT;
  static constexpr int kSoft = 4 * kNT;                 // softmax warps
  static constexpr int kIssuer = kSoft + 4;             // the warp that issues the products
  static constexpr int kResolver = kIssuer + 1;         // the warp that looks the tokens up
  static constexpr int kWarps = kResolver + 1;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kQBytes = 128 * D * 2;           // per row tile
  static constexpr int kKVBytes = kBN * D * 2;          // per stage and tensor
  static constexpr int kSlots = 4;                      // steps whose rows and scales are held
  static constexpr int kOffK = kNT * kQBytes;
  static constexpr int kOffV = kOffK + kStages * kKVBytes;
  static constexpr int kOffKS = kOffV + kStages * kKVBytes;        // [slots][kBN] K scales
  static constexpr int kOffVS = kOffKS + kSlots * kBN * 4;    // [slots][kBN] V scales
  static constexpr int kOffVM = kOffVS + kSlots * kBN * 4;         // [slots] the largest V scale
  static constexpr int kOffRow = kOffVM + 16 * kSlots;             // [slots][kBN] pool rows (int64)
  static constexpr int kOffBar = kOffRow + kSlots * kBN * 8;
  static constexpr int kNumBars = 4 * kStages + 2 * kSlots + 4 * kNT + 1;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;          // tensor memory address, key range, flags
  static constexpr int kSmem = kOffMisc + 32 + 1024;               // + alignment of the base
  static_assert(kSmem > 114 * 1024 && kSmem <= 227 * 1024, "one block per SM, since each takes all of tensor memory");
  // tensor-memory columns
  static constexpr int kColS = 0;                        // kNT x kBN
  static constexpr int kColO = 256;                      // kNT x D
};

struct TileMisc {
  uint32_t tmem;
  int lo, hi;   // keys that any row sees
  int bad;      // a block entry outside the pool
  int give_up;  // a wait ran out
};

// A wait that gives up (after about 0.1 s, or soon after another one did).
__device__ __forceinline__ void tile_wait(uint32_t bar, uint32_t parity, volatile TileMisc* misc, uint32_t* status) {
  for (int n = 0; n < kMbarTries; ++n) {
    if (mbar_try_wait(bar, parity)) return;
    if ((n & 15) == 15 && misc->give_up != 0) return;
  }
  misc->give_up = 1;
  set_status(status, 16u);
}

// ---- logits ------------------------------------------------------------------------
enum LogitMode : int { kPlain, kCapped, kNearCap, kBiased, kBoth /* cap and bias */ };

// A capped logit costs 2^x and a reciprocal beside the probability's own 2^x, and the unit
// that computes these is then the kernel's bound (8 results a clock and scheduler for 2^x).
// Where every score of a warp's step is below 3/4 of the cap (kNearCap), tanh comes from an
// odd polynomial of degree 9 instead: the minimax fit on [-3/4, 3/4] (iteratively reweighted
// least squares on a Chebyshev grid), off by at most 0.3 * 2^-20 with its binary32 rounding.
constexpr float kTanhRange = 0.75f;
constexpr float kTanh0 = 0.9999971985816956f, kTanh1 = -0.33323076367378235f, kTanh2 = 0.13226091861724854f,
                kTanh3 = -0.049280449748039246f, kTanh4 = 0.012318833731114864f;

struct RowLogit {
  float f;       // query factor times log2 e (plain, biased without cap)
  float fz;      // capped: 2 log2 e / softcap times the query factor
  float fu;      // capped: the query factor over softcap
  float c2;      // capped: softcap log2 e
  bool cap;      // whether there is one
  float slope;   // times log2 e
  int pos;
  int lo, hi;
};

// Base-2 logit of a scaled score x = s * ks at column col of a tile that starts at t0 (tf =
// t0 - pos as a float).
template <int kMode>
__device__ __forceinline__ float logit(const RowLogit& r, float x, float tf, int col) {
  float y;
  if (kMode == kCapped || kMode == kBoth) {
    y = __fmaf_rn(-2.0f * r.c2, rcp_ftz(1.0f + ex2_ftz(x * r.fz)), r.c2);
  } else {
    y = x * r.f;
  }
  if (kMode == kBoth) y = __fmaf_rn(r.slope, tf + static_cast<float>(col), y);
  return y;
}

// The first half of a step's P' is in tensor memory: its products may begin while the second
// half is computed.  Not where the planes are page-scaled and a step has 128 columns: those
// take 64 columns at a time, and one hand-over is faster then (624 against 639 us on 4096
// queries in 12288 tokens at head_dim 128; at 256, 845 against 929 us the other way).
__device__ __forceinline__ void half_ready(uint32_t bar) {
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// y - M + add for a pair of scores x in kPlain (f2 the factor), kCapped (f2 = 2 log2 e / cap
// times the factor, y = c2 - 2 c2 / (1 + 2^(x f2)), c2 part of add) or kNearCap (f2 the factor
// over cap, y = c2 tanh(x f2)).
struct CapPairs {
  uint64_t one, m2c, k[5];  // 1, -2 c2, and the polynomial's coefficients times c2
  template <int kMode>
  __device__ __forceinline__ void init(float c2) {
    if (kMode == kCapped) {
      one = dup_f32x2(1.0f);
      m2c = dup_f32x2(-2.0f * c2);
    }
    if (kMode == kNearCap) {
      k[0] = dup_f32x2(kTanh0 * c2);
      k[1] = dup_f32x2(kTanh1 * c2);
      k[2] = dup_f32x2(kTanh2 * c2);
      k[3] = dup_f32x2(kTanh3 * c2);
      k[4] = dup_f32x2(kTanh4 * c2);
    }
  }
  template <int kMode>
  __device__ __forceinline__ uint64_t logit2(uint64_t x, uint64_t f2, uint64_t add) const {
    if constexpr (kMode == kPlain || kMode == kBiased) {
      return fma_f32x2(x, f2, add);
    } else if constexpr (kMode == kNearCap) {
      const uint64_t u = mul_f32x2(x, f2), t = mul_f32x2(u, u);
      uint64_t P = fma_f32x2(k[4], t, k[3]);
      P = fma_f32x2(P, t, k[2]);
      P = fma_f32x2(P, t, k[1]);
      P = fma_f32x2(P, t, k[0]);
      return fma_f32x2(u, P, add);
    } else {
      uint32_t a, b;
      unpack_f32x2(mul_f32x2(x, f2), a, b);
      unpack_f32x2(add_f32x2(pack_f32x2(__float_as_uint(ex2_ftz(__uint_as_float(a))), __float_as_uint(ex2_ftz(__uint_as_float(b)))),
                             one), a, b);
      return fma_f32x2(pack_f32x2(__float_as_uint(rcp_ftz(__uint_as_float(a))), __float_as_uint(rcp_ftz(__uint_as_float(b)))),
                       m2c, add);
    }
  }
};

// slope * col + base for the columns col and col + 1 (kBiased).
__device__ __forceinline__ uint64_t bias2(uint64_t slope, int col, uint64_t base) {
  return fma_f32x2(slope, pack_f32x2(__float_as_uint(static_cast<float>(col)), __float_as_uint(static_cast<float>(col + 1))), base);
}

// log2 of the largest V scale as the reference takes it, clamped far outside what rows of
// ordinary size need.
__device__ __forceinline__ float scale_log2(float v) { return fminf(fmaxf(lg2(v), -100.0f), 100.0f); }

// Largest logit of a tile's row (-inf where it sees no key of the tile).
// most: the largest |score| (kCapped only).  lv: log2 of the largest V scale of the keys that the
// row sees, where the mask leaves some out (a row that took louder ones into its reference would
// lose its own P' to f16's range).
template <int kMode, bool kMask, int kBN>
__device__ __forceinline__ float tile_max(const RowLogit& r, uint32_t taddr, const float* ks, const float* vs, int t0, float& most,
                                          float& lv) {
  const int lo = r.lo - t0, hi = r.hi - t0;
  const float tf = static_cast<float>(t0 - r.pos);
  float m0 = kNegInf, m1 = kNegInf, a0 = 0.0f, v0 = 0.0f;
  const uint64_t f2 = dup_f32x2(r.f), s2 = dup_f32x2(r.slope);
#pragma unroll 1
  for (int c0 = 0; c0 < kBN; c0 += 32) {
    const uint64_t base = dup_f32x2(r.slope * (tf + static_cast<float>(c0)));
    uint32_t v[32];
    tmem_ld32(taddr + c0, v);
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(ks + c0 + i);
      uint64_t xa = mul_f32x2(pack_f32x2(v[i], v[i + 1]), k4.x);
      uint64_t xb = mul_f32x2(pack_f32x2(v[i + 2], v[i + 3]), k4.y);
      if (kMode == kBiased) {
        xa = fma_f32x2(xa, f2, bias2(s2, i, base));
        xb = fma_f32x2(xb, f2, bias2(s2, i + 2, base));
      }
      uint32_t x0, x1, x2, x3;
      unpack_f32x2(xa, x0, x1);
      unpack_f32x2(xb, x2, x3);
      float y[4] = {__uint_as_float(x0), __uint_as_float(x1), __uint_as_float(x2), __uint_as_float(x3)};
      if (kMode == kCapped) a0 = max3(max3(a0, fabsf(y[0]), fabsf(y[1])), fabsf(y[2]), fabsf(y[3]));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (kMode == kBoth) y[e] = logit<kMode>(r, y[e], tf, c0 + i + e);
        if (kMask) {
          const bool in = c0 + i + e >= lo && c0 + i + e < hi;
          y[e] = in ? y[e] : kNegInf;
          v0 = fmaxf(v0, in ? vs[c0 + i + e] : 0.0f);
        }
      }
      m0 = max3(m0, y[0], y[1]);
      m1 = max3(m1, y[2], y[3]);
    }
  }
  const float m = fmaxf(m0, m1);
  most = a0;
  if (kMask) lv = scale_log2(v0);
  // without a bias the logit grows with the score, so it is taken once
  if (kMode == kBiased || kMode == kBoth || (kMask && m == kNegInf)) return m;
  return logit<kMode>(r, m, 0.0f, 0);
}

// P' of a tile's row over the first half of its score columns; returns the row sum of p.
template <int kMode, bool kMask, int kBN>
__device__ __forceinline__ float tile_probs(const RowLogit& r, uint32_t taddr, const float* ks, const float* vs, int t0,
                                            float M, uint32_t half) {
  const int lo = r.lo - t0, hi = r.hi - t0;
  const float tf = static_cast<float>(t0 - r.pos);
  const uint64_t f2 = dup_f32x2(kMode == kNearCap ? r.fu : kMode == kCapped ? r.fz : r.f), s2 = dup_f32x2(r.slope);
  const uint64_t add = dup_f32x2(kMode == kCapped ? r.c2 - M : -M);
  CapPairs cp;
  cp.init<kMode>(r.c2);
  uint64_t l0 = 0, l1 = 0;  // two pairs of partial sums
#pragma unroll 1
  for (int c0 = 0; c0 < kBN; c0 += 32) {
    const uint64_t base = dup_f32x2(__fmaf_rn(r.slope, tf + static_cast<float>(c0), -M));
    uint32_t v[32], h[16];
    tmem_ld32(taddr + c0, v);
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(ks + c0 + i);
      const ulonglong2 v4 = *reinterpret_cast<const ulonglong2*>(vs + c0 + i);
      uint64_t xa = mul_f32x2(pack_f32x2(v[i], v[i + 1]), k4.x);
      uint64_t xb = mul_f32x2(pack_f32x2(v[i + 2], v[i + 3]), k4.y);
      if (kMode == kBiased) {
        xa = fma_f32x2(xa, f2, bias2(s2, i, base));
        xb = fma_f32x2(xb, f2, bias2(s2, i + 2, base));
      } else if (kMode != kBoth) {
        xa = cp.logit2<kMode>(xa, f2, add);
        xb = cp.logit2<kMode>(xb, f2, add);
      }
      uint32_t x[4];
      unpack_f32x2(xa, x[0], x[1]);
      unpack_f32x2(xb, x[2], x[3]);
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y = __uint_as_float(x[e]);
        if (kMode == kBoth) y = logit<kMode>(r, y, tf, c0 + i + e) - M;
        if (kMask) y = c0 + i + e >= lo && c0 + i + e < hi ? y : kNegInf;
        p[e] = ex2_ftz(y);
      }
      const uint64_t pa = pack_f32x2(__float_as_uint(p[0]), __float_as_uint(p[1]));
      const uint64_t pb = pack_f32x2(__float_as_uint(p[2]), __float_as_uint(p[3]));
      l0 = add_f32x2(l0, pa);
      l1 = add_f32x2(l1, pb);
      uint32_t q[4];
      unpack_f32x2(mul_f32x2(pa, v4.x), q[0], q[1]);
      unpack_f32x2(mul_f32x2(pb, v4.y), q[2], q[3]);
      // one rounding of P' to f16: relative 2^-11 of the largest |v| the row attends to
      h[i / 2] = f32x2_to_f16x2(__uint_as_float(q[0]), __uint_as_float(q[1]));
      h[i / 2 + 1] = f32x2_to_f16x2(__uint_as_float(q[2]), __uint_as_float(q[3]));
    }
    tmem_st16(taddr + c0 / 2, h);  // columns whose scores are already read
    if (c0 + 32 == kBN / 2) half_ready(half);
  }
  uint32_t a, b, c, d;
  unpack_f32x2(l0, a, b);
  unpack_f32x2(l1, c, d);
  return (__uint_as_float(a) + __uint_as_float(b)) + (__uint_as_float(c) + __uint_as_float(d));
}

// The same where both planes are page-scaled and pages are whole groups of 16 columns: K's
// scale and V's (as its log2) are one pair a group, gs[group] = {ks, log2 vs}.  The scale of
// the scores is then part of the row's factor, and P' = 2^(y - M + log2 vs) needs no product;
// the group's sum of P' is divided by vs for l.  M may come from steps with much larger scales (a
// page of zeros has 2^-126), and l has to keep p where P' vanishes: with mx the step's largest
// logit of the row, log2 vs - M counts as -mx - 40 where it is below that.  P' is then at most
// 2^-40, 0 in f16 either way, and the sum loses nothing above 2^-86 of the step's largest p.
template <int kMode, bool kMask, int kBN>
__device__ __forceinline__ float tile_max_pages(const RowLogit& r, uint32_t taddr, const float2* gs, int t0, float& most,
                                                float& lv) {
  constexpr int kCols = kBN == 128 ? 64 : 32;  // at a time
  const int lo = r.lo - t0, hi = r.hi - t0;
  const float tf = static_cast<float>(t0 - r.pos);
  const uint64_t s2 = dup_f32x2(r.slope);
  float best = kNegInf;
  most = 0.0f;
  if (kMask) lv = -100.0f;
#pragma unroll 1
  for (int c0 = 0; c0 < kBN; c0 += kCols) {
    uint32_t v[kCols];
    tmem_ld(taddr + c0, v);
#pragma unroll
    for (int g = 0; g < kCols / 16; ++g) {
      const float ks = gs[c0 / 16 + g].x;
      if (kMask) lv = fmaxf(lv, c0 + 16 * g < hi && c0 + 16 * g + 16 > lo ? fminf(gs[c0 / 16 + g].y, 100.0f) : -100.0f);
      float m[2] = {kNegInf, kNegInf}, a = 0.0f;
      const uint64_t f2 = dup_f32x2(r.f * ks);
      const uint64_t base = dup_f32x2(r.slope * (tf + static_cast<float>(c0 + 16 * g)));
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const int col = c0 + 16 * g + i;
        float x0 = __uint_as_float(v[16 * g + i]), x1 = __uint_as_float(v[16 * g + i + 1]);
        if (kMode == kBiased) {
          uint32_t b0, b1;
          unpack_f32x2(fma_f32x2(pack_f32x2(v[16 * g + i], v[16 * g + i + 1]), f2, bias2(s2, i, base)), b0, b1);
          x0 = __uint_as_float(b0);
          x1 = __uint_as_float(b1);
        }
        if (kMode == kCapped) a = max3(a, fabsf(x0), fabsf(x1));
        if (kMode == kBoth) {
          x0 = logit<kMode>(r, x0 * ks, tf, col);
          x1 = logit<kMode>(r, x1 * ks, tf, col + 1);
        }
        if (kMask) {
          x0 = col >= lo && col < hi ? x0 : kNegInf;
          x1 = col + 1 >= lo && col + 1 < hi ? x1 : kNegInf;
        }
        m[i / 2 % 2] = max3(m[i / 2 % 2], x0, x1);
      }
      const float mg = fmaxf(m[0], m[1]);
      if (kMode == kCapped) most = fmaxf(most, a * ks);
      best = fmaxf(best, kMode == kBiased || kMode == kBoth || (kMask && mg == kNegInf) ? mg : mg * ks);
    }
  }
  if (kMode == kBiased || kMode == kBoth || (kMask && best == kNegInf)) return best;
  return logit<kMode>(r, best, 0.0f, 0);
}

template <int kMode, bool kMask, int kBN>
__device__ __forceinline__ float tile_probs_pages(const RowLogit& r, uint32_t taddr, const float2* gs, int t0, float M, float mx, uint32_t half) {
  constexpr int kCols = kBN == 128 ? 64 : 32;  // at a time
  const int lo = r.lo - t0, hi = r.hi - t0;
  const float tf = static_cast<float>(t0 - r.pos);
  CapPairs cp;
  cp.init<kMode>(r.c2);
  const uint64_t s2 = dup_f32x2(r.slope);
  float L = 0.0f;
  const float least = -40.0f - mx;
#pragma unroll 1
  for (int c0 = 0; c0 < kBN; c0 += kCols) {
    uint32_t v[kCols], h[kCols / 2];
    tmem_ld(taddr + c0, v);
#pragma unroll
    for (int g = 0; g < kCols / 16; ++g) {
      const float2 s = gs[c0 / 16 + g];
      const float ref = max_nan(s.y - M, least);
      const uint64_t f2 = dup_f32x2((kMode == kNearCap ? r.fu : kMode == kCapped ? r.fz : r.f) * s.x);
      const uint64_t base = dup_f32x2(__fmaf_rn(r.slope, tf + static_cast<float>(c0 + 16 * g), ref));
      const uint64_t add = dup_f32x2(kMode == kCapped ? r.c2 + ref : ref);
      uint64_t l[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const int col = c0 + 16 * g + i;
        const uint64_t x2 = pack_f32x2(v[16 * g + i], v[16 * g + i + 1]);
        float y0, y1;
        uint32_t a, b;
        if (kMode == kBoth) {
          y0 = logit<kMode>(r, __uint_as_float(v[16 * g + i]) * s.x, tf, col) + ref;
          y1 = logit<kMode>(r, __uint_as_float(v[16 * g + i + 1]) * s.x, tf, col + 1) + ref;
        } else {
          unpack_f32x2(kMode == kBiased ? fma_f32x2(x2, f2, bias2(s2, i, base)) : cp.logit2<kMode>(x2, f2, add), a, b);
          y0 = __uint_as_float(a);
          y1 = __uint_as_float(b);
        }
        if (kMask) {
          y0 = col >= lo && col < hi ? y0 : kNegInf;
          y1 = col + 1 >= lo && col + 1 < hi ? y1 : kNegInf;
        }
        const float p0 = ex2_ftz(y0), p1 = ex2_ftz(y1);
        l[(i / 2) % 2] = add_f32x2(l[(i / 2) % 2], pack_f32x2(__float_as_uint(p0), __float_as_uint(p1)));
        // one rounding of P' to f16: relative 2^-11 of the largest |v| the row attends to
        h[8 * g + i / 2] = f32x2_to_f16x2(p0, p1);
      }
      uint32_t a, b;
      unpack_f32x2(add_f32x2(l[0], l[1]), a, b);
      L = __fmaf_rn(__uint_as_float(a) + __uint_as_float(b), ex2_ftz(-(ref + M)), L);
    }
    tmem_st(taddr + c0 / 2, h);  // columns whose scores are already read
    if (kBN == 64 && c0 == 0) half_ready(half);
  }
  return L;
}

// Where a step's scales are: K's and V's by token, or the groups' pairs.
struct StepScales {
  const float *ks, *vs;
  const float2* gs;
};

template <int kMode, int kBN, bool kPages>
__device__ __forceinline__ float tile_max_any(bool mask, const RowLogit& r, uint32_t ta, const StepScales& sc, int t0, float& most,
                                              float& lv) {
  if constexpr (kPages)
    return mask ? tile_max_pages<kMode, true, kBN>(r, ta, sc.gs, t0, most, lv) : tile_max_pages<kMode, false, kBN>(r, ta, sc.gs, t0, most, lv);
  else
    return mask ? tile_max<kMode, true, kBN>(r, ta, sc.ks, sc.vs, t0, most, lv)
                : tile_max<kMode, false, kBN>(r, ta, sc.ks, sc.vs, t0, most, lv);
}
template <int kMode, int kBN, bool kPages>
__device__ __forceinline__ float tile_probs_any(bool mask, const RowLogit& r, uint32_t ta, const StepScales& sc, int t0, float M, float mx, uint32_t half) {
  if constexpr (kPages)
    return mask ? tile_probs_pages<kMode, true, kBN>(r, ta, sc.gs, t0, M, mx, half)
                : tile_probs_pages<kMode, false, kBN>(r, ta, sc.gs, t0, M, mx, half);
  else
    return mask ? tile_probs<kMode, true, kBN>(r, ta, sc.ks, sc.vs, t0, M, half) : tile_probs<kMode, false, kBN>(r, ta, sc.ks, sc.vs, t0, M, half);
}

// ---- producers: one tensor's rows of a step ------------------------------------------
// 128 threads; a thread takes the same 16-byte piece of kPer code rows, kRowStep rows apart.
// Eight threads that store together hold the pieces of one 64-dim panel in as many
// neighbouring rows as make their swizzled chunks cover all banks (FP8: 4 pieces of two
// chunks, 2 rows; NVFP4: 2 pieces of four chunks, 4 rows).  kRowStep is a multiple of 8, so a
// thread's swizzle is the same for all its rows and its addresses differ by constants.
template <int D, int kFmt>
struct TileLoad {
  static constexpr int kBN = QTile<D>::kBN;
  static constexpr int kCB = kFmt == 3 ? D : D / 2;     // code bytes per row
  static constexpr int kPieces = kCB / 16;              // per row
  static constexpr int kPer = kBN * kPieces / 128;      // per thread
  static constexpr int kRowStep = 128 / kPieces;
  static constexpr int kPanelPieces = kFmt == 3 ? 4 : 2;  // pieces of a 64-dim panel
  static constexpr int kRowsTogether = 8 / kPanelPieces;
  static constexpr int kPanels = kPieces / kPanelPieces;
  static_assert(kRowStep % 8 == 0, "the swizzle repeats every 8 rows");
  uint32_t w[kPer][4];
  uint32_t bs[kFmt == 3 ? 1 : kPer];                    // NVFP4: the piece's two block scales

  static __device__ __forceinline__ int piece(int tid) { return tid % kPanelPieces; }  // within the panel
  static __device__ __forceinline__ int panel(int tid) { return tid / 8 % kPanels; }
  static __device__ __forceinline__ int row0(int tid) {
    return tid / (8 * kPanels) * kRowsTogether + tid / kPanelPieces % kRowsTogether;
  }
  __device__ __forceinline__ void load(const AttnPlane& pl, const int64_t* rows, int tid) {
    const int c = panel(tid) * kPanelPieces + piece(tid);
    const int64_t* const mine = rows + row0(tid);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t row = mine[i * kRowStep];
      w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0u;
      if constexpr (kFmt != 3) bs[i] = 0u;
      if (row >= 0) {
        load16B(pl.codes + row * kCB + 16 * c, w[i]);
        if constexpr (kFmt != 3) bs[i] = LDX(reinterpret_cast<const uint16_t*>(pl.bscale + row * (D / 16) + 2 * c));
      }
    }
  }
  // f16 values into the swizzled tile at shared address dst: panels of 64 dims, [kBN][128 B]
  __device__ __forceinline__ void store(uint32_t dst, int tid) const {
    const int r = row0(tid);
    const uint32_t base = dst + panel(tid) * (kBN * 128) + r * 128;
    constexpr int kChunks = 8 / kPanelPieces;  // of a piece
    uint32_t at[kChunks];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) at[j] = base + (((kChunks * piece(tid) + j) ^ (r & 7)) * 16);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t down = i * kRowStep * 128;
      if constexpr (kFmt == 3) {  // 16 dims: two 16-byte chunks
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t h0[2], h1[2];
          e4m3x4_to_f16x2(w[i][2 * j], h0);
          e4m3x4_to_f16x2(w[i][2 * j + 1], h1);
          sts16(at[j] + down, h0[0], h0[1], h1[0], h1[1]);
        }
      } else {  // 32 dims: four chunks, two block scales
        const uint32_t two = e4m3x2_to_f16x2(bs[i]);
        const uint32_t s0 = __byte_perm(two, 0u, 0x1010), s1 = __byte_perm(two, 0u, 0x3232);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t h[4];
          e2m1x8_to_f16x2(w[i][j], h);
          const uint32_t s = j < 2 ? s0 : s1;
          sts16(at[j] + down, hmul2(h[0], s), hmul2(h[1], s), hmul2(h[2], s), hmul2(h[3], s));
        }
      }
    }
  }
};

// kPages: both planes page-scaled, block_size a multiple of 16 (FP8 codes).
template <int D, int kFK, int kFV, bool kPages>
__global__ void __launch_bounds__(QTile<D>::kThreads, 1) query_tile_kernel(const QueryAttnParams qp) {
  using T = QTile<D>;
  constexpr int kBN = T::kBN, kNT = T::kNT, kStages = T::kStages;
  constexpr bool kHalves = !(kPages && kBN == 128);
  const AttnParams& p = qp.a;
  extern __shared__ unsigned char tile_smem_raw[];
  const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(tile_smem_raw));
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* const smem = tile_smem_raw + (sbase - raw);
  TileMisc* const misc = reinterpret_cast<TileMisc*>(smem + T::kOffMisc);

  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform for the compiler too
  const int s = blockIdx.z, h = blockIdx.y;
  // the last rows first: under a causal mask they see the most keys
  const int ntiles = gridDim.x / p.nsplit;
  const int ct = ntiles - 1 - static_cast<int>(blockIdx.x) / p.nsplit, split = blockIdx.x % p.nsplit;
  const int row0 = ct * T::kRows;

  int q0, nq, len;
  const bool ok = query_range(qp, s, q0, nq, len);
  if (!ok && threadIdx.x == 0 && blockIdx.x == 0 && h == 0) set_status(p.status, 8u);
  const int rows = nq * p.group;
  if (row0 >= rows) return;

  const int nt = kNT == 2 && rows - row0 <= 128 ? 1 : kNT;  // row tiles that hold rows

  const uint32_t bar0 = sbase + T::kOffBar;
  const uint32_t k_full = bar0, k_empty = k_full + 8 * kStages, v_full = k_empty + 8 * kStages, v_empty = v_full + 8 * kStages;
  const uint32_t sc_full = v_empty + 8 * kStages, sc_empty = sc_full + 8 * T::kSlots, s_full = sc_empty + 8 * T::kSlots;
  const uint32_t p_ready = s_full + 8 * kNT, o_done = p_ready + 8 * kNT, q_full = o_done + 8 * kNT;
  const uint32_t p_half = q_full + 8;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(k_full + 8 * i, 4);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, 4);
      mbar_init(v_empty + 8 * i, 1);
    }
    for (int i = 0; i < T::kSlots; ++i) {
      mbar_init(sc_full + 8 * i, 1);
      mbar_init(sc_empty + 8 * i, 4 + 4 * nt);  // the producer and the softmax warps
    }
    for (int i = 0; i < kNT; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_ready + 8 * i, 4);
      mbar_init(p_half + 8 * i, 4);
      mbar_init(o_done + 8 * i, 1);
    }
    mbar_init(q_full, 4 * nt);
    misc->lo = 0x7FFFFFFF;
    misc->hi = 0;
    misc->bad = 0;
    misc->give_up = 0;
    mbar_init_fence();
  }
  __syncthreads();
  if (warp == T::kIssuer) {
    tmem_alloc(sbase + T::kOffMisc, 512);
    tmem_relinquish();
  }

  // ---- softmax threads: the keys that their row sees (lookup and loads of K and V wait for
  // them, not for Q) ----
  RowLogit rl;
  int row = -1;  // the thread's row within the sequence; -1: none
  int head = 0;
  int64_t tok = 0;
  bool sees = false;
  rl.lo = 0;
  rl.hi = 0x7FFFFFFF;  // a thread without a row masks nothing
  rl.pos = 0;
  if (warp < 4 * nt) {
    if (row0 + static_cast<int>(threadIdx.x) < rows) row = row0 + threadIdx.x;
    if (row >= 0) {
      const int i = row / p.group;
      head = h * p.group + row - i * p.group;
      tok = q0 + i;
      rl.pos = len - nq + i;
      int lo, hi;
      key_range(qp, s, q0 + i, rl.pos, len, lo, hi);
      sees = lo < hi;
      if (sees) {
        rl.lo = lo;
        rl.hi = hi;
      }
    }
    const int lo = __reduce_min_sync(0xFFFFFFFFu, sees ? rl.lo : 0x7FFFFFFF);
    const int hi = __reduce_max_sync(0xFFFFFFFFu, sees ? rl.hi : 0);
    if (lane == 0) {
      atomicMin(&misc->lo, lo);
      atomicMax(&misc->hi, hi);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, misc->tmem, 0);
  const int key_lo = misc->lo, key_hi = misc->hi;
  int t_begin = 0, t_end = 0;
  if (key_lo < key_hi) {  // equal splits in whole steps
    const int first = kPages ? key_lo & ~15 : key_lo;  // groups of 16 columns lie in one page
    const int per = ((key_hi - first + p.nsplit - 1) / p.nsplit + kBN - 1) / kBN * kBN;
    t_begin = static_cast<int>(min(static_cast<int64_t>(first) + static_cast<int64_t>(split) * per, static_cast<int64_t>(key_hi)));
    t_end = t_begin + min(per, key_hi - t_begin);
  }
  const int steps = (t_end - t_begin + kBN - 1) / kBN;

  if (warp == T::kResolver) {
    // ---- pool rows and scales of each step's tokens, up to kSlots steps ahead ----
    int64_t* const rowbuf = reinterpret_cast<int64_t*>(smem + T::kOffRow);
    float* const ksb = reinterpret_cast<float*>(smem + T::kOffKS);
    float* const vsb = reinterpret_cast<float*>(smem + T::kOffVS);
    float2* const gsb = reinterpret_cast<float2*>(smem + T::kOffKS);  // [slots][groups], in K's place
    float* const vmb = reinterpret_cast<float*>(smem + T::kOffVM);
    constexpr int kPer = kBN / 32;  // tokens a lane
    const int32_t* const table = p.block_table + static_cast<int64_t>(s) * p.max_blocks;
    // a step's table entries are on their way two steps ahead of its scales' use, its
    // scales one step ahead: the two dependent loads never wait for each other
    int32_t blk[kPer];
    int64_t row[kPer];
    float ks[kPer], vs[kPer];
    auto entries = [&](int j) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int t = t_begin + j * kBN + 32 * i + lane;
        blk[i] = t < t_end ? LDX(table + p.div_bs.div(static_cast<uint32_t>(t))) : -1;
      }
    };
    auto scales = [&](int j) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int t = t_begin + j * kBN + 32 * i + lane;
        row[i] = -1;
        ks[i] = vs[i] = 0.0f;
        if (t >= t_end || t < key_lo) continue;
        if (blk[i] < 0 || blk[i] >= p.num_blocks) {
          misc->bad = 1;
          continue;
        }
        uint32_t bi, bo;
        p.div_bs.divmod(static_cast<uint32_t>(t), bi, bo);
        const int64_t pg = static_cast<int64_t>(blk[i]);
        row[i] = (pg * p.block_size + bo) * p.H + h;
        ks[i] = LDX(p.k.rscale + (p.k_page ? pg * p.H + h : row[i]));
        vs[i] = LDX(p.v.rscale + (p.v_page ? pg * p.H + h : row[i]));
      }
    };
    entries(0);
    scales(0);
    entries(1);
    for (int j = 0; j < steps; ++j) {
      const int slot = j % T::kSlots;
      if (j >= T::kSlots) tile_wait(sc_empty + 8 * slot, ((j / T::kSlots) - 1) & 1, misc, p.status);
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) m = fmaxf(m, vs[i]);
      m = group_max<32>(m);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        rowbuf[slot * kBN + 32 * i + lane] = row[i];
        if constexpr (kPages) {
          // a group's scales are those of any of its tokens within the keys (0 without one); a V
          // scale of 0 counts as 2^-126
          const uint32_t has = __ballot_sync(0xFFFFFFFFu, row[i] >= 0) & (lane < 16 ? 0xFFFFu : 0xFFFF0000u);
          const int from = has != 0u ? __ffs(has) - 1 : lane;
          const float kg = __shfl_sync(0xFFFFFFFFu, ks[i], from), vg = __shfl_sync(0xFFFFFFFFu, vs[i], from);
          if (lane % 16 == 0)
            gsb[slot * (kBN / 16) + 2 * i + lane / 16] = make_float2(kg, lg2(vg < 0x1p-126f ? 0x1p-126f : vg));
        } else {
          ksb[slot * kBN + 32 * i + lane] = ks[i];
          vsb[slot * kBN + 32 * i + lane] = vs[i];
        }
      }
      scales(j + 1);  // nothing past t_end is read
      entries(j + 2);
      if (lane == 0) vmb[4 * slot] = m;
      __syncwarp();
      if (lane == 0) mbar_arrive(sc_full + 8 * slot);
    }
  } else if (warp >= T::kIssuer) {
    // ---- the products ----
    if (steps > 0) {
      const uint32_t leader = elect_one();
      constexpr uint32_t kBase = (1u << 4) | (8u << 24);  // f16 x f16 -> f32, M = 128
      constexpr uint32_t kIdS = kBase | (static_cast<uint32_t>(kBN / 8) << 17);
      constexpr uint32_t kIdO = kBase | (1u << 16) | (static_cast<uint32_t>(D / 8) << 17);  // B is MN-major
      auto scores = [&](int i, int j) {
        const uint32_t qa = desc_lo(sbase + i * T::kQBytes, 16);
        const uint32_t ka = desc_lo(sbase + T::kOffK + (j % kStages) * T::kKVBytes, 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma_ss(leader, tmem + T::kColS + i * kBN, smem_desc(qa, (k / 4) * (128 * 128) + (k % 4) * 32),
                    smem_desc(ka, (k / 4) * (kBN * 128) + (k % 4) * 32), kIdS, k > 0);
        tc_commit(leader, s_full + 8 * i);
        if (i == nt - 1) tc_commit(leader, k_empty + 8 * (j % kStages));
      };
      tile_wait(q_full, 0, misc, p.status);
      tile_wait(k_full, 0, misc, p.status);
      tc_fence_after();
      for (int i = 0; i < nt; ++i) scores(i, 0);
      for (int j = 0; j < steps; ++j) {
        const int st = j % kStages;
        tile_wait(v_full + 8 * st, (j / kStages) & 1, misc, p.status);
        for (int i = 0; i < nt; ++i) {
          const uint32_t va = desc_lo(sbase + T::kOffV + st * T::kKVBytes, kBN * 128);
          tile_wait((kHalves ? p_half : p_ready) + 8 * i, j & 1, misc, p.status);
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kBN / 32; ++k)
            tc_mma_ts(leader, tmem + T::kColO + i * D, tmem + T::kColS + i * kBN + 8 * k, smem_desc(va, k * 2048), kIdO, j > 0 || k > 0);
          if constexpr (kHalves) {
            tile_wait(p_ready + 8 * i, j & 1, misc, p.status);
            tc_fence_after();
          }
#pragma unroll
          for (int k = kBN / 32; k < kBN / 16; ++k)
            tc_mma_ts(leader, tmem + T::kColO + i * D, tmem + T::kColS + i * kBN + 8 * k, smem_desc(va, k * 2048), kIdO, j > 0 || k > 0);
          if (i == nt - 1) tc_commit(leader, v_empty + 8 * st);
          if (j + 1 < steps) {
            if (i == 0) {
              tile_wait(k_full + 8 * ((j + 1) % kStages), ((j + 1) / kStages) & 1, misc, p.status);
              tc_fence_after();
            }
            scores(i, j + 1);
          } else {
            tc_commit(leader, o_done + 8 * i);
          }
        }
      }
    }
    __syncwarp();
  } else if (warp >= T::kSoft) {
    // ---- producers ----
    const int tid = threadIdx.x - 32 * T::kSoft;
    const int64_t* const rowbuf = reinterpret_cast<const int64_t*>(smem + T::kOffRow);
    TileLoad<D, kFK> lk;
    TileLoad<D, kFV> lv;
    // K of step j + 1 is loaded into registers while K and V of step j are stored, V likewise
    auto rows = [&](int j) {
      tile_wait(sc_full + 8 * (j % T::kSlots), (j / T::kSlots) & 1, misc, p.status);
      return rowbuf + (j % T::kSlots) * kBN;
    };
    if (steps > 0) {
      const int64_t* const first = rows(0);
      lk.load(p.k, first, tid);
      lv.load(p.v, first, tid);
      __syncwarp();
      if (lane == 0) mbar_arrive(sc_empty);
    }
    for (int j = 0; j < steps; ++j) {
      const int st = j % kStages;
      if (j >= kStages) tile_wait(k_empty + 8 * st, ((j / kStages) - 1) & 1, misc, p.status);
      lk.store(sbase + T::kOffK + st * T::kKVBytes, tid);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full + 8 * st);
      const int64_t* const next = j + 1 < steps ? rows(j + 1) : nullptr;
      if (next != nullptr) lk.load(p.k, next, tid);
      if (j >= kStages) tile_wait(v_empty + 8 * st, ((j / kStages) - 1) & 1, misc, p.status);
      lv.store(sbase + T::kOffV + st * T::kKVBytes, tid);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full + 8 * st);
      if (next != nullptr) {
        lv.load(p.v, next, tid);
        __syncwarp();
        if (lane == 0) mbar_arrive(sc_empty + 8 * ((j + 1) % T::kSlots));
      }
    }
  } else if (warp < 4 * nt) {
    // ---- softmax: one thread a row.  First its row of Q as f16, scaled by a power of two so
    // that the largest element lies in [2^14, 2^15): exact ----
    {
      const int r = threadIdx.x;
      const uint32_t qs = sbase + (r / 128) * T::kQBytes + (r % 128) * 128;
      const uint16_t* const q = p.q + tok * p.q_row_pitch + static_cast<int64_t>(head) * p.q_head_pitch;
      rl.slope = row >= 0 && qp.slopes != nullptr ? LDX(qp.slopes + head) * kLog2e : 0.0f;
      constexpr int kC = D / 8, kHold = kC < 16 ? kC : 16;  // 16-byte pieces; those in flight at once
      uint32_t w[kHold][4];
      auto load = [&](int c0) {
#pragma unroll
        for (int c = 0; c < kHold; ++c) {
          w[c][0] = w[c][1] = w[c][2] = w[c][3] = 0u;
          if (row >= 0) load16B(q + 8 * (c0 + c), w[c]);
        }
      };
      float am = 0.0f;
#pragma unroll
      for (int c0 = 0; c0 < kC; c0 += kHold) {
        load(c0);
#pragma unroll
        for (int c = 0; c < kHold; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) am = max3(am, fabsf(bf16lo(w[c][e])), fabsf(bf16hi(w[c][e])));
      }
      int k = 0;
      if (am > 0.0f) k = 14 - (static_cast<int>((__float_as_uint(am) >> 23) & 0xFF) - 127);
      k = max(-113, min(120, k));
      const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
      const float fac = row >= 0 ? p.scale * __uint_as_float(static_cast<uint32_t>(127 - k) << 23) : 0.0f;
#pragma unroll
      for (int c0 = 0; c0 < kC; c0 += kHold) {
        if (kC > kHold) load(c0);
#pragma unroll
        for (int c = 0; c < kHold; ++c) {
          uint32_t f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = f32x2_to_f16x2(bf16lo(w[c][e]) * up, bf16hi(w[c][e]) * up);
          sts16(qs + ((c0 + c) / 8) * (128 * 128) + ((((c0 + c) % 8) ^ (r & 7)) * 16), f[0], f[1], f[2], f[3]);
        }
      }
      rl.f = fac * kLog2e;
      rl.cap = qp.softcap > 0.0f;
      rl.c2 = qp.softcap * kLog2e;
      rl.fu = rl.cap ? fac / qp.softcap : 0.0f;
      rl.fz = rl.cap ? 2.0f * kLog2e / qp.softcap * fac : 0.0f;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const int i = warp / 4;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + T::kColS + i * kBN, to = tmem + lanes + T::kColO + i * D;
    const int mode = qp.slopes != nullptr ? (rl.cap ? kBoth : kBiased) : rl.cap ? kCapped : kPlain;
    float M = kNoKey, L = 0.0f;
    for (int j = 0; j < steps; ++j) {
      const int slot = j % T::kSlots;
      const int t0 = t_begin + j * kBN;
      tile_wait(sc_full + 8 * slot, (j / T::kSlots) & 1, misc, p.status);
      tile_wait(s_full + 8 * i, j & 1, misc, p.status);
      tc_fence_after();
      __syncwarp();
      const StepScales sc{reinterpret_cast<const float*>(smem + T::kOffKS) + slot * kBN,
                          reinterpret_cast<const float*>(smem + T::kOffVS) + slot * kBN,
                          reinterpret_cast<const float2*>(smem + T::kOffKS) + slot * (kBN / 16)};
      const float vm = *reinterpret_cast<const float*>(smem + T::kOffVM + 16 * slot);
      const bool mask = __any_sync(0xFFFFFFFFu, rl.lo > t0 || rl.hi < t0 + kBN);
      const bool none = __all_sync(0xFFFFFFFFu, rl.lo >= t0 + kBN || rl.hi <= t0 || row < 0 || !sees);
      if (none) {  // no row of the warp sees a key of this step
        uint32_t z[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) z[e] = 0u;
#pragma unroll
        for (int c = 0; c < kBN / 2; c += 16) tmem_st16(ts + c, z);
        if (kHalves) half_ready(p_half + 8 * i);
      } else {
        float mx, most, lv = scale_log2(vm);
        if (mode == kPlain) mx = tile_max_any<kPlain, kBN, kPages>(mask, rl, ts, sc, t0, most, lv);
        else if (mode == kCapped) mx = tile_max_any<kCapped, kBN, kPages>(mask, rl, ts, sc, t0, most, lv);
        else if (mode == kBiased) mx = tile_max_any<kBiased, kBN, kPages>(mask, rl, ts, sc, t0, most, lv);
        else mx = tile_max_any<kBoth, kBN, kPages>(mask, rl, ts, sc, t0, most, lv);
        // V's scales enter P', so the reference covers them
        const bool move = mx + lv > M + 14.0f;
        if (__any_sync(0xFFFFFFFFu, move)) {
          const float Mn = move ? mx + lv - 6.0f : M;
          const float a = ex2(M - Mn);
          M = Mn;
          L *= a;
          if (j > 0) {  // the products of the steps before are complete: s_full came after them
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(to + c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
              tmem_st32(to + c, o);
            }
          }
        }
        if (mode == kPlain) L += tile_probs_any<kPlain, kBN, kPages>(mask, rl, ts, sc, t0, M, mx, p_half + 8 * i);
        else if (mode == kCapped && __all_sync(0xFFFFFFFFu, most * rl.fu <= kTanhRange))
          L += tile_probs_any<kNearCap, kBN, kPages>(mask, rl, ts, sc, t0, M, mx, p_half + 8 * i);
        else if (mode == kCapped) L += tile_probs_any<kCapped, kBN, kPages>(mask, rl, ts, sc, t0, M, mx, p_half + 8 * i);
        else if (mode == kBiased) L += tile_probs_any<kBiased, kBN, kPages>(mask, rl, ts, sc, t0, M, mx, p_half + 8 * i);
        else L += tile_probs_any<kBoth, kBN, kPages>(mask, rl, ts, sc, t0, M, mx, p_half + 8 * i);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(p_ready + 8 * i);
        mbar_arrive(sc_empty + 8 * slot);
      }
    }
    if (steps > 0) {
      tile_wait(o_done + 8 * i, 0, misc, p.status);
      tc_fence_after();
      __syncwarp();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    bool bad = false;
    if (*reinterpret_cast<volatile int*>(&misc->bad) != 0) {
      for (int l = 0; l < 32; ++l) {
        const int lo = __shfl_sync(0xFFFFFFFFu, sees ? rl.lo : t_end, l), hi = __shfl_sync(0xFFFFFFFFu, rl.hi, l);
        if (needs_bad_block(p, s, max(lo, t_begin), min(hi, t_end)) && lane == l) bad = true;
      }
    }
    if (!sees) L = 0.0f;
    uint16_t* const out = p.out + tok * p.o_row_pitch + static_cast<int64_t>(head) * p.o_head_pitch;
    float* const wsr = p.ws + ((tok * p.Hq + head) * p.nsplit + split) * (D + 2);
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;  // a NaN stays one
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t o[32];
      __syncwarp();
      if (steps > 0) {
        tmem_ld32(to + c, o);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
      }
      if (row < 0) continue;
      if (p.nsplit == 1) {
        if (bad) continue;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint32_t w[4];
#pragma unroll
          for (int b = 0; b < 4; ++b)
            w[b] = L != 0.0f ? pack_bf16x2(__uint_as_float(o[e + 2 * b]) * inv, __uint_as_float(o[e + 2 * b + 1]) * inv) : 0u;
          store16B(out + c + e, w);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; e += 2)  // (D + 2) * 4 bytes is a multiple of 8
          STX(reinterpret_cast<float2*>(wsr + c + e),
              sees ? make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])) : make_float2(0.0f, 0.0f));
      }
    }
    if (row >= 0 && p.nsplit > 1)
      STX(reinterpret_cast<float2*>(wsr + D), make_float2(bad ? __int_as_float(0x7FC00000) : sees ? M : kNoKey, L));
    tc_fence_before();
  }
  __syncthreads();
  if (warp == T::kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && misc->bad != 0) set_status(p.status, 2u);
}

template <int D, int kFK, int kFV, bool kPages = false>
cudaError_t tile_launch(const QueryAttnParams& p, cudaStream_t s) {
  using T = QTile<D>;
  auto k = query_tile_kernel<D, kFK, kFV, kPages>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (static_cast<int64_t>(p.max_q) * p.a.group + T::kRows - 1) / T::kRows;
  const dim3 grid(static_cast<unsigned>(tiles * p.a.nsplit), p.a.H, p.a.S);
  KVQ_LAUNCH("query_tile_kernel", s, k<<<grid, T::kThreads, T::kSmem, s>>>(p); e = cudaGetLastError());
  return e;
}

template <int D>
cudaError_t tile_dispatch(const QueryAttnParams& p, cudaStream_t s) {
  const bool k8 = p.a.fmt_k == 3, v8 = p.a.fmt_v == 3;
  if (p.a.k_page && p.a.v_page && p.a.block_size % 16 == 0) return tile_launch<D, 3, 3, true>(p, s);
  if (!k8 && !v8) return tile_launch<D, 1, 1>(p, s);
  if (k8 && !v8) return tile_launch<D, 3, 1>(p, s);
  if (!k8 && v8) return tile_launch<D, 1, 3>(p, s);
  return tile_launch<D, 3, 3>(p, s);
}

}  // namespace

int query_tile_rows(int32_t D) { return D == 256 ? QTile<256>::kRows : QTile<128>::kRows; }

cudaError_t launch_query_tiles(const QueryAttnParams& p, cudaStream_t s) {
  switch (p.a.D) {
    case 64: return tile_dispatch<64>(p, s);
    case 128: return tile_dispatch<128>(p, s);
    case 256: return tile_dispatch<256>(p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
