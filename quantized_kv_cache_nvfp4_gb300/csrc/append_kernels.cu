// append_kernels.cu -- K and V rows into a paged cache, K turned by its position's angles on
// the way, with the bounds of each block's keys; Q turned beside them.
//
// Position p has the angles whose cosines and sines stand in row p of a table; with c, s those
// of a pair (a, b) of channels
//   a' = a c - b s,   b' = b c + a s        (binary32, every product and sum rounded once)
// the pairs being (i, i + rot/2) or (2i, 2i + 1); channels from rot on pass.  K' goes from
// binary32 into the pool's format with the codec's arithmetic (nvfp4_kernels.cu,
// page_scale_kernels.cu): rounding it to bf16 first, as a store of turned bf16 rows has to,
// would round twice.  Q' is rounded to bf16 once.  The bounds of (block, head) are the least
// and the largest bf16(K') of its rows, channel by channel.
//
// Mapping: tokens of one page that stand next to each other in slot_ids form a run; one warp serves
// (run, head, tensor), so scales and bounds need no atomics.  A thread block looks the runs of a chunk of
// tokens up once and shares them, heads fastest, among its warps.  D / 16 lanes (rounded up to a power of
// two) hold a row, 8 channels of a half and their partners of the other half each, so that pairs need no
// exchange and share their angles; 32 / lanes rows a pass.  The rows come through shared memory, a run or
// 4 KB of it ahead of the arithmetic: in registers, one pass ahead left too little in flight (27,000
// tokens, 8 heads, head_dim 128: K alone 40 us), and a whole run unrolled outgrew the instruction cache
// (48).  Page scales need the maximum before the codes, and take a run twice.  The blocks behind
// turn Q: a warp holds a token's angles in registers and walks its heads (evenly among the others it took 5%
// longer).
//
// Bound: HBM for Q, issue and 16 resident warps an SM (128 registers a thread) for K and V.
// Measured: 27,000 tokens of 24 prompts, 32 and 8 heads, head_dim 128, FP8 rows of K and pages of V, 16-token
// blocks, with bounds: 127 us, 4.9 TB/s, 73% of a plain copy's rate; Q alone 71 us (93%), K 54, V
// 32; 64 single tokens 5.1 us.  (Without packed products 2 us more; stages of 8 KB, half the warps: 236.)
#include <algorithm>

#include "page_scale.cuh"
#include "kvq_params.h"

namespace kvq {

namespace {

// Four warps a block, four blocks an SM (24 prompts as above: 127 us; eight warps and two blocks 136, two and
// eight 135: Q's blocks start as those of K and V end one by one).
constexpr int kAppendWarps = 4, kAppendBlocks = 4;
constexpr int kChunk = 32;  // most tokens of a block

// The two 8-channel chunks of a lane: c and c + half of the turned channels where those are rot / 2 apart
// (half chunks each), else neighbours.  at: the first angle of each (-1: not turned).
struct Lane {
  int ch[2], at[2];
  bool act;    // the lane has channels
  bool apart;  // ch[0] and ch[1] are partners
};
__device__ __forceinline__ Lane make_lane(int rot, bool pairs, int li, int D) {
  const int half = pairs ? 0 : rot / 16;
  Lane l;
  l.act = 16 * li < D;
  l.apart = li < half;
  l.ch[0] = l.apart ? li : 2 * li;
  l.ch[1] = l.apart ? li + half : 2 * li + 1;
#pragma unroll
  for (int j = 0; j < 2; ++j) l.at[j] = pairs ? (8 * l.ch[j] < rot ? 4 * l.ch[j] : -1) : l.apart ? 8 * li : -1;
  return l;
}

// Angles of the lane at a position, from its row of the table: apart, 8 cosines and 8 sines for both
// chunks; neighbours, 4 and 4 for each.
struct Angles {
  uint4 c[2], s[2];
};
__device__ __forceinline__ void load_angles(const Lane& l, int rot, bool pairs, const float* row, Angles& a) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int at = pairs ? l.at[j] : l.at[0] + 4 * j;
    if (l.at[pairs ? j : 0] < 0) continue;
    a.c[j] = LDX(reinterpret_cast<const uint4*>(row + at));
    a.s[j] = LDX(reinterpret_cast<const uint4*>(row + rot / 2 + at));
  }
}

// Products and sums one rounding each: packed products, single sums (a packed sum of packed products comes
// out as one rounding).
__device__ __forceinline__ void mul2(float a0, float a1, uint32_t b0, uint32_t b1, float& r0, float& r1) {
  uint32_t u, v;
  unpack_f32x2(mul_f32x2(pack_f32x2(__float_as_uint(a0), __float_as_uint(a1)), pack_f32x2(b0, b1)), u, v);
  r0 = __uint_as_float(u);
  r1 = __uint_as_float(v);
}

// The lane's 16 channels in binary32, turned (rot: uniform, 0 for none).
__device__ __forceinline__ void turn16(const Lane& l, const Angles& a, int rot, bool pairs, const uint32_t (&w)[2][4],
                                       float (&y)[2][8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[j][2 * i] = bf16lo(w[j][i]);
      y[j][2 * i + 1] = bf16hi(w[j][i]);
    }
  if (rot == 0) return;
  if (pairs) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (l.at[j] < 0) continue;
      const uint32_t c[4] = {a.c[j].x, a.c[j].y, a.c[j].z, a.c[j].w}, s[4] = {a.s[j].x, a.s[j].y, a.s[j].z, a.s[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float ac, bc, as, bs;
        mul2(y[j][2 * i], y[j][2 * i + 1], c[i], c[i], ac, bc);
        mul2(y[j][2 * i], y[j][2 * i + 1], s[i], s[i], as, bs);
        y[j][2 * i] = __fsub_rn(ac, bs);
        y[j][2 * i + 1] = __fadd_rn(bc, as);
      }
    }
  } else if (l.apart) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // channels 4 j .. 4 j + 3 of both chunks
      const uint32_t c[4] = {a.c[j].x, a.c[j].y, a.c[j].z, a.c[j].w}, s[4] = {a.s[j].x, a.s[j].y, a.s[j].z, a.s[j].w};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float &a0 = y[0][4 * j + 2 * i], &a1 = y[0][4 * j + 2 * i + 1], &b0 = y[1][4 * j + 2 * i], &b1 = y[1][4 * j + 2 * i + 1];
        float ac0, ac1, as0, as1, bc0, bc1, bs0, bs1;
        mul2(a0, a1, c[2 * i], c[2 * i + 1], ac0, ac1);
        mul2(a0, a1, s[2 * i], s[2 * i + 1], as0, as1);
        mul2(b0, b1, c[2 * i], c[2 * i + 1], bc0, bc1);
        mul2(b0, b1, s[2 * i], s[2 * i + 1], bs0, bs1);
        a0 = __fsub_rn(ac0, bs0);
        a1 = __fsub_rn(ac1, bs1);
        b0 = __fadd_rn(bc0, as0);
        b1 = __fadd_rn(bc1, as1);
      }
    }
  }
}

__device__ __forceinline__ float absmax8(const float (&y)[8]) {
  float m = fabsf(y[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
  return m;
}

// quantize_block and fp8_quantize16 (kvq_device.cuh) of 8 binary32 values; inv = 1 / s (0 when s is 0).
__device__ __forceinline__ float inverse(float s) { return (s != 0.0f) ? __frcp_rn(s) : 0.0f; }
__device__ __forceinline__ uint32_t quantize8(const float (&y)[8], float s, float inv) {
  uint32_t byte[4];
  if (!isinf(inv)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float q0, q1;
      mul2(y[2 * i], y[2 * i + 1], __float_as_uint(inv), __float_as_uint(inv), q0, q1);
      byte[i] = e2m1x2_from_f32(q0, q1);
    }
  } else {  // the reciprocal overflowed, divide directly
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const float a = i == 0 ? y[0] : i == 1 ? y[2] : i == 2 ? y[4] : y[6], b = i == 0 ? y[1] : i == 1 ? y[3] : i == 2 ? y[5] : y[7];
      const uint32_t v = e2m1x2_from_f32(__fdiv_rn(a, s), __fdiv_rn(b, s));
      byte[0] = i == 0 ? v : byte[0], byte[1] = i == 1 ? v : byte[1], byte[2] = i == 2 ? v : byte[2], byte[3] = i == 3 ? v : byte[3];
    }
  }
  return bytes4(byte[0], byte[1], byte[2], byte[3]);
}
__device__ __forceinline__ uint2 fp8_quantize8(const float (&y)[8], float s, float inv) {
  uint32_t w[4];
  if (!isinf(inv)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float q0, q1;
      mul2(y[2 * i], y[2 * i + 1], __float_as_uint(inv), __float_as_uint(inv), q0, q1);
      w[i] = e4m3x2_from_f32(q0, q1);
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const float a = i == 0 ? y[0] : i == 1 ? y[2] : i == 2 ? y[4] : y[6], b = i == 0 ? y[1] : i == 1 ? y[3] : i == 2 ? y[5] : y[7];
      const uint32_t v = e4m3x2_from_f32(__fdiv_rn(a, s), __fdiv_rn(b, s));
      w[0] = i == 0 ? v : w[0], w[1] = i == 1 ? v : w[1], w[2] = i == 2 ? v : w[2], w[3] = i == 3 ? v : w[3];
    }
  }
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// bf16 minima and maxima of packed pairs (a NaN loses against a number).
__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A token's slot and position as they stand in memory; nothing (a negative slot) for tokens outside the call.
struct Token {
  int64_t slot;
  int pos;
};
__device__ __forceinline__ Token load_token(const AppendParams& p, int64_t t) {
  Token k{-1, 0};
  if (t < 0 || t >= p.T) return k;
  k.slot = LDX(p.slot_ids + t);
  if (p.cos_sin != nullptr) k.pos = LDX(p.positions + t);
  return k;
}
// Its slot: -1 where it has none in the pool.  `report`: the block that speaks for the token.
__device__ __forceinline__ int64_t token_slot(const AppendParams& p, const Token& k, bool report) {
  if (k.slot >= p.num_slots && report) set_status(p.status, 1u);
  if (k.pos >= p.num_positions && p.cos_sin != nullptr && report) set_status(p.status, 4u);
  return k.slot >= p.num_slots ? -1 : k.slot;
}
// Whether its position lets it in.
__device__ __forceinline__ bool turnable(const AppendParams& p, int pos) {
  return p.cos_sin == nullptr || (pos >= 0 && pos < p.num_positions);
}

// The runs that begin in a chunk of tokens, and the chunk's tokens.  A run goes by slots alone: a token that its
// position keeps out stays in it as a row that is not live (a run cut there would give a page's scale and
// bounds to two warps at once).  A run without a live row is none.
struct Chunk {
  int64_t page[kChunk];  // of a run
  int start[kChunk];     // its first token, from the chunk's
  int length[kChunk];
  bool begins[kChunk];   // a live row holds the page's first slot
  bool whole[kChunk];    // all its rows are live
  int place[kChunk];     // of a token in its page, -1: not live
  int pos[kChunk];
  int runs;
};
__device__ __forceinline__ void find_runs(const AppendParams& p, int64_t t0, bool report, Chunk& ck) {  // one warp
  const int lane = threadIdx.x & 31;
  auto page_of = [&](int64_t slot) -> int64_t {
    return slot < 0 ? -1 : p.small ? static_cast<int64_t>(p.div_bs.div(static_cast<uint32_t>(slot))) : slot / p.block_size;
  };
  // all loads at once (one behind the other they were most of a block's start; K of 27,000 tokens 39.6 us, 36.6)
  const Token token = load_token(p, t0 + lane), ahead = load_token(p, lane == 0 ? t0 - 1 : -1);
  Token behind = load_token(p, t0 + 32 + lane);
  const int64_t slot = token_slot(p, token, report);
  const int64_t page = page_of(slot);
  const int64_t before = page_of(token_slot(p, ahead, false));
  int64_t prev = __shfl_up_sync(0xFFFFFFFFu, page, 1);
  if (lane == 0) prev = before;
  const bool live = page >= 0 && turnable(p, token.pos);
  const int place = live ? static_cast<int>(slot - page * p.block_size) : -1;
  ck.place[lane] = place;
  ck.pos[lane] = live ? token.pos : 0;  // any that has angles, as a live row of the run does
  const uint32_t leaders = __ballot_sync(0xFFFFFFFFu, lane < p.chunk && page >= 0 && page != prev);
  const uint32_t same = __ballot_sync(0xFFFFFFFFu, page >= 0 && page == prev);  // goes on with the token before
  const uint32_t firsts = __ballot_sync(0xFFFFFFFFu, place == 0), lives = __ballot_sync(0xFFFFFFFFu, live);
  const bool leads = ((leaders >> lane) & 1u) != 0u;
  int n = leads ? min(1 + (lane == 31 ? 0 : run_bits(same >> (lane + 1))), 32 - lane) : 0;
  const uint32_t mine = n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
  bool any = ((lives >> lane) & mine) != 0u, whole = ((~lives >> lane) & mine) == 0u, begins = ((firsts >> lane) & mine) != 0u;
  const uint32_t reach = __ballot_sync(0xFFFFFFFFu, leads && lane + n == 32);
  if (reach != 0u) {  // the last run may go on behind the 32 tokens
    const int b = __ffs(reach) - 1;
    const int64_t pg = __shfl_sync(0xFFFFFFFFu, page, b);
    for (int64_t t = t0 + 32; t < p.T; t += 32) {
      const int64_t s2 = token_slot(p, behind, false);
      const int m = run_bits(__ballot_sync(0xFFFFFFFFu, page_of(s2) == pg));
      const bool in = lane < m && turnable(p, behind.pos);
      const bool more = __any_sync(0xFFFFFFFFu, in), gap = __any_sync(0xFFFFFFFFu, lane < m && !in);
      const bool first = __any_sync(0xFFFFFFFFu, in && s2 == pg * p.block_size);
      if (lane == b) {
        n += m;
        any = any || more;
        whole = whole && !gap;
        begins = begins || first;
      }
      if (m < 32) break;
      behind = load_token(p, t + 32 + lane);
    }
  }
  const uint32_t runs = __ballot_sync(0xFFFFFFFFu, leads && any);
  if (leads && any) {
    const int at = __popc(runs & ((1u << lane) - 1u));
    ck.page[at] = page;
    ck.start[at] = lane;
    ck.length[at] = n;
    ck.begins[at] = begins;
    ck.whole[at] = whole;
  }
  if (lane == 0) ck.runs = __popc(runs);
}

// The rows of a warp's items (run, tensor, head) pass through two stages of its own in shared memory,
// up to kStageBytes of rows each: one is filled by cp.async while the other is worked on.  An item of page
// scales that takes more than one stage passes twice.
constexpr int kStageBytes = 4096;

template <int L>
__device__ __forceinline__ void append_items(const AppendParams& p, const Chunk& ck, int64_t t0, int first, int step,
                                             unsigned char* stages) {
  constexpr int R = 32 / L;  // rows per pass
  const int lane = threadIdx.x & 31, li = lane % L, sub = lane / L;
  const int D = p.D, per = p.H * p.ntensors, items = ck.runs * per, rows = kStageBytes / (2 * D), pieces = D / 8;

  struct Place {  // in the sequence of stages
    int it, r0;   // item and first row
    bool again;   // the second time through the item
  };
  Place now{first, 0, false};
  struct Item {
    int run, tensor, h;
  };
  auto item_of = [&](int it) {
    Item m;
    uint32_t run, rem;
    p.div_per.divmod(static_cast<uint32_t>(it), run, rem);
    m.run = static_cast<int>(run);
    m.tensor = static_cast<int>(rem) >= p.H ? 1 : 0;
    m.h = static_cast<int>(rem) - m.tensor * p.H;
    return m;
  };
  auto after = [&](Place c, int length, bool paged) {
    c.r0 += rows;
    if (c.r0 < length) return c;
    c.again = !c.again && length > rows && paged;
    c.r0 = 0;
    if (!c.again) c.it += step;
    return c;
  };
  auto fetch = [&](const Place& c, unsigned char* to) {
    if (c.it < items) {
      const Item m = item_of(c.it);
      const AppendTensor& ten = p.ten[m.tensor];
      const int n = min(rows, ck.length[m.run] - c.r0);
      const int64_t pitch = ten.row_pitch;
      const uint16_t* x = ten.x + (t0 + ck.start[m.run] + c.r0) * pitch + m.h * ten.head_pitch;
      if constexpr (L <= 16) {  // a lane copies one piece of every (16 / L)-th row
        const int c8 = lane % (2 * L), r = lane / (2 * L);
        x += r * pitch + 8 * c8;
        to += 16 * (r * pieces + c8);
        for (int q = r; q < n; q += 16 / L, x += (16 / L) * pitch, to += 16 * (16 / L) * pieces)
          if (c8 < pieces) cp_async16(to, x);
      } else {
        for (int q = 0; q < n; ++q, x += pitch, to += 16 * pieces)
          for (int c8 = lane; c8 < pieces; c8 += 32) cp_async16(to + 16 * c8, x + 8 * c8);
      }
    }
    cp_async_commit();
  };
  fetch(now, stages);

  float am = 0.0f, s0 = 0.0f, s = 0.0f;
#pragma unroll 1
  for (int stage = 0; now.it < items; stage ^= 1) {
    const Item item = item_of(now.it);
    const int run = item.run, tensor = item.tensor, h = item.h;
    const Place next = after(now, ck.length[run], p.ten[tensor].fmt == 5);
    fetch(next, stages + (stage ^ 1) * kStageBytes);
    const bool key = p.ten[tensor].key;
    const int fmt = p.ten[tensor].fmt;
    const Nvfp4Planes dst = p.ten[tensor].dst;
    const int rot = key && p.cos_sin != nullptr ? p.rot : 0;
    const int length = ck.length[run], n = min(rows, length - now.r0), b = ck.start[run] + now.r0;
    const int64_t prow = ck.page[run] * p.H + h, row0 = ck.page[run] * p.block_size;
    const bool begins = ck.begins[run], whole = ck.whole[run], paged = fmt == 5;
    uint16_t* const bounds = key ? p.bounds : nullptr;
    const Lane ln = make_lane(rot, p.pairs, li, D);
    if (now.r0 == 0 && !now.again) {
      am = s0 = 0.0f;
      if (paged && !begins && lane == 0) s0 = LDX(dst.rscale + prow);
    }
    unsigned char* const at_stage = stages + stage * kStageBytes + 2 * D * sub;
    // row 0 of the page: a row's bytes are `at` times the row's of all heads behind it
    const int row_bytes = fmt == 1 ? D / 2 : D, codes_pitch = p.H * row_bytes;
    uint8_t* const codes = dst.codes + (row0 * p.H + h) * row_bytes;
    // rows of the stage that are not live, filled with a word (rare: a uniform branch beside the loops)
    auto fill_dead = [&](uint32_t word) {
      for (int r = 0; r < n; ++r) {
        if (b + r < kChunk ? ck.place[b + r] >= 0 : turnable(p, LDX(p.positions + t0 + b + r))) continue;
        for (int c8 = lane; c8 < pieces; c8 += 32)
          *reinterpret_cast<uint4*>(stages + stage * kStageBytes + 2 * D * r + 16 * c8) = make_uint4(word, word, word, word);
      }
      __syncwarp();
    };
    // the stage's rows: the lane's channels and angles, the row, its place in the page (below 0: not live)
    auto each_row = [&](auto&& f) {
#pragma unroll 1
      for (int q = 0; q < n; q += R) {
        const int r = q + sub;
        int at = 0, pos = 0;
        if (b + r < kChunk) {
          at = ck.place[b + r];
          pos = ck.pos[b + r];
        } else if (r < n) {
          at = static_cast<int>(LDX(p.slot_ids + t0 + b + r) - row0);
          if (rot != 0 || !whole) pos = LDX(p.positions + t0 + b + r);
          if (!whole && !turnable(p, pos)) at = -1, pos = 0;
        }
        Angles a;
        if (rot != 0 && r < n) load_angles(ln, rot, p.pairs, p.cos_sin + static_cast<int64_t>(pos) * rot, a);
        uint32_t v[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 u = ln.act && r < n ? *reinterpret_cast<const uint4*>(at_stage + 2 * D * q + 16 * ln.ch[j]) : make_uint4(0u, 0u, 0u, 0u);
          v[j][0] = u.x, v[j][1] = u.y, v[j][2] = u.z, v[j][3] = u.w;
        }
        f(v, a, r, at);
      }
    };
    // turned rows in bf16 over the rows as they came, for the bounds
    auto put_back = [&](const float (&y)[2][8], int r) {
      if (!(ln.act && r < n)) return;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<uint4*>(at_stage + 2 * D * (r - sub) + 16 * ln.ch[j]) =
            make_uint4(pack_bf16x2(y[j][0], y[j][1]), pack_bf16x2(y[j][2], y[j][3]), pack_bf16x2(y[j][4], y[j][5]),
                       pack_bf16x2(y[j][6], y[j][7]));
    };
    cp_async_wait<1>();
    __syncwarp();
    if (!whole) fill_dead(0u);  // no part in the maxima
    bool turned = rot != 0 || !paged;
    if (!now.again && !turned) {  // page scales of rows as they are: maxima of packed bf16
      uint32_t m = 0u;
      each_row([&](const uint32_t (&v)[2][4], const Angles&, int, int) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(v[j][i]));
      });
      m &= 0x7FFF7FFFu;
      const float most = fmaxf(bf16lo(m), bf16hi(m));
      turned = __any_sync(0xFFFFFFFFu, most > 3.4028235e38f);  // an infinity: the other way
      if (!turned) am = fmaxf(am, most);
    }
    if (!now.again && turned) {
      each_row([&](const uint32_t (&v)[2][4], const Angles& a, int r, int at) {
        float y[2][8];
        turn16(ln, a, rot, p.pairs, v, y);
        const bool live = ln.act && r < n && at >= 0;
        const float vb[2] = {absmax8(y[0]), absmax8(y[1])};  // 0 in lanes without a row
        if (bounds != nullptr && !paged) put_back(y, r);
        if (paged) {  // the largest finite one: an infinity costs its own element only
          if (fmaxf(vb[0], vb[1]) <= 3.4028235e38f) {
            am = fmaxf(am, fmaxf(vb[0], vb[1]));
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(y[j][i]) <= 3.4028235e38f ? fabsf(y[j][i]) : 0.0f);
          }
          return;
        }
        const float amax = group_max<L>(fmaxf(vb[0], vb[1]));
        const float rs = __fdiv_rn(amax, fmt == 3 ? kE4M3Max : kE2M1Max * kE4M3Max);
        const float rinv = inverse(rs);
        if (fmt == 3) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint2 c = fp8_quantize8(y[j], rs, rinv);
            if (live) store8B(codes + static_cast<int64_t>(at) * codes_pitch + 8 * ln.ch[j], c.x, c.y);
          }
        } else {
          // a block of 16 is chunks 2 k and 2 k + 1: the other one's lane and place there
          float other[2] = {vb[1], vb[0]};
          if (rot != 0 && !p.pairs) {  // uniform
            const int half = rot / 16, base = lane - li;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int c = ln.ch[j] ^ 1;
              const int src = c < half ? c : c < 2 * half ? c - half : c / 2;
              const float o0 = __shfl_sync(0xFFFFFFFFu, vb[0], base + src % L), o1 = __shfl_sync(0xFFFFFFFFu, vb[1], base + src % L);
              other[j] = (c < half ? 0 : c < 2 * half ? 1 : c % 2) == 0 ? o0 : o1;
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t bsb = block_scale_code(fmaxf(vb[j], other[j]), rs, rinv);
            const float bs = __fmul_rn(e4m3_to_f32(bsb), rs);
            const uint32_t c = quantize8(y[j], bs, inverse(bs));
            if (live) {
              STX(reinterpret_cast<uint32_t*>(codes + static_cast<int64_t>(at) * codes_pitch) + ln.ch[j], c);
              if (ln.ch[j] % 2 == 0)
                STX(dst.bscale + ((row0 + at) * p.H + h) * (D / 16) + ln.ch[j] / 2, static_cast<uint8_t>(bsb));
            }
          }
        }
        if (li == 0 && live) STX(dst.rscale + (row0 + at) * p.H + h, rs);
      });
    }
    if (!now.again) {
      if (now.r0 + rows >= length) {  // all of the item's rows
        if (paged) {
          s0 = __shfl_sync(0xFFFFFFFFu, s0, 0);
          if (!(s0 > 0.0f && s0 <= 3.4028235e38f)) s0 = 0.0f;  // no scale stored yet
          s = fmaxf(s0, page_scale_need(group_max<32>(am)));
          if (s0 > 0.0f && s > s0) {  // the rows that the page holds, under the new scale
            const float f = __fdiv_rn(s0, s);
            uint8_t* const cp = dst.codes + (row0 * p.H + h) * D;
            const int64_t cpitch = static_cast<int64_t>(p.H) * D;
            const int each = D / 16;  // 16-byte pieces of a row
            for (int at = lane; at < p.block_size * each; at += 32) {
              uint8_t* const to = cp + (at / each) * cpitch + 16 * (at % each);
              uint32_t c[4];
              load16B_rw(to, c);
#pragma unroll
              for (int i = 0; i < 4; ++i) c[i] = rescale4(c[i], f);
              store16B(to, c);
            }
            __syncwarp();  // before the call's own rows go over them
          }
          if (lane == 0 && s != s0) STX(dst.rscale + prow, s);
        }
      }
    }
    if (paged && (now.again || length <= rows)) {
      const float inv = inverse(s);
      each_row([&](const uint32_t (&v)[2][4], const Angles& a, int r, int at) {
        float y[2][8];
        turn16(ln, a, rot, p.pairs, v, y);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint2 c = fp8_quantize8(y[j], s, inv);
          if (ln.act && r < n && at >= 0) store8B(codes + static_cast<int64_t>(at) * codes_pitch + 8 * ln.ch[j], c.x, c.y);
        }
        if (bounds != nullptr) put_back(y, r);
      });
    }
    // ---- bounds of the stage's rows, a lane 8 channels, with the stored ones but where the item's first
    // rows start the block over ----
    if (bounds != nullptr && (!paged || now.again || length <= rows)) {
      __syncwarp();
      if (!whole) fill_dead(0x7FFF7FFFu);  // NaN: no part in the bounds
      for (int c8 = lane; c8 < pieces; c8 += 32) {
        uint16_t* const at = bounds + prow * 2 * D + 8 * c8;
        uint32_t lo[4], hi[4];
        if (begins && now.r0 == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lo[i] = 0x7F807F80u;
            hi[i] = 0xFF80FF80u;
          }
        } else {
          load16B_rw(at, lo);
          load16B_rw(at + D, hi);
        }
        const unsigned char* from = stages + stage * kStageBytes + 16 * c8;
#pragma unroll 4
        for (int r = 0; r < n; ++r, from += 2 * D) {
          const uint4 u = *reinterpret_cast<const uint4*>(from);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lo[i] = bf16x2_min(lo[i], w[i]);
            hi[i] = bf16x2_max(hi[i], w[i]);
          }
        }
        store16B(at, lo);
        store16B(at + D, hi);
      }
    }
    __syncwarp();  // the stage is read
    now = next;
  }
  cp_async_wait<0>();
}

// Q: warp w takes heads first .. of one token, 32 / L at a time.
template <int L>
__device__ __forceinline__ void append_turn_q(const AppendParams& p, int64_t w) {
  constexpr int R = 32 / L;
  constexpr int kBatch = 4;  // passes in flight (27,000 tokens of 32 heads, head_dim 128: 73 us, with 2 84)
  const int lane = threadIdx.x & 31;
  const int li = lane % L, sub = lane / L;
  const int64_t t = w / p.q_parts;
  if (t >= p.T) return;
  const int first = static_cast<int>(w - t * p.q_parts) * p.q_heads;
  const int32_t pos = LDX(p.positions + t);
  if (pos < 0) return;
  if (pos >= p.num_positions) {
    if (lane == 0 && first == 0) set_status(p.status, 4u);
    return;
  }
  const Lane ln = make_lane(p.rot, p.pairs, li, p.D);
  Angles a;
  load_angles(ln, p.rot, p.pairs, p.cos_sin + static_cast<int64_t>(pos) * p.rot, a);
  const uint16_t* const x = p.q + t * p.q_row_pitch;
  uint16_t* const y_at = p.q_out + t * p.qo_row_pitch;
  const int end = min(first + p.q_heads, p.Hq);
#pragma unroll 1
  for (int h0 = first; h0 < end; h0 += kBatch * R) {
    uint32_t raw[kBatch][2][4];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h0 + k * R + sub;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (ln.act && h < end) load16B_rw(x + h * p.q_head_pitch + 8 * ln.ch[j], raw[k][j]);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h0 + k * R + sub;
      if (!(ln.act && h < end)) continue;
      float y[2][8];
      turn16(ln, a, p.rot, p.pairs, raw[k], y);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(y[j][2 * i], y[j][2 * i + 1]);
        store16B(y_at + h * p.qo_head_pitch + 8 * ln.ch[j], o);
      }
    }
  }
}

template <int L>
__global__ void __launch_bounds__(32 * kAppendWarps, kAppendBlocks) append_kernel(const AppendParams p) {
  __shared__ Chunk ck;
  extern __shared__ __align__(16) unsigned char stages[];
  const int warp = threadIdx.x >> 5;
  const int64_t block = blockIdx.x;
  if (block >= p.row_blocks) {
    append_turn_q<L>(p, (block - p.row_blocks) * kAppendWarps + warp);
    return;
  }
  const int64_t chunk = block / p.parts;
  const int part = static_cast<int>(block - chunk * p.parts);
  const int64_t t0 = chunk * p.chunk;
  if (warp == 0) find_runs(p, t0, part == 0, ck);
  __syncthreads();
  append_items<L>(p, ck, t0, part * kAppendWarps + warp, p.parts * kAppendWarps, stages + warp * 2 * kStageBytes);
}

template <int L>
cudaError_t append_launch(const AppendParams& p_in, cudaStream_t s) {
  AppendParams p = p_in;
  constexpr int R = 32 / L;
  auto k = append_kernel<L>;
  const int64_t per = static_cast<int64_t>(p.H) * p.ntensors, fill = 16ll * num_sms();
  int64_t blocks = 0;
  p.div_per = FastDiv(static_cast<uint32_t>(per > 0 ? per : 1));
  p.parts = 1;
  if (p.ntensors > 0) {
    // tokens per block: even turns of the resident blocks, as few as chunks of 32 allow (27,000 tokens, K alone: 54 us,
    // by whole chunks of 32 60).  Where that is less than a common page, chunks of 32 whose runs and heads several
    // blocks share: short chunks leave the runs to a few of them (1000 tokens in 64-token pages, 8 heads of 256:
    // 59 us, by chunks of 2 185; 64 single tokens take 0.2 of 5 us more)
    const int64_t slots = static_cast<int64_t>(kAppendBlocks) * num_sms();
    const int64_t turns = (p.T + kChunk * slots - 1) / (kChunk * slots);
    p.chunk = 2ll * p.T > kChunk * slots ? static_cast<int>((p.T + slots * turns - 1) / (slots * turns)) : kChunk;
    const int64_t chunks = (static_cast<int64_t>(p.T) + p.chunk - 1) / p.chunk;
    const int64_t most = (std::min<int64_t>(p.chunk, p.T) * per + kAppendWarps - 1) / kAppendWarps;  // an item a warp
    p.parts = static_cast<int>(std::max(int64_t{1}, std::min(slots / chunks, most)));
    p.row_blocks = chunks * p.parts;
    blocks = p.row_blocks;
  }
  if (p.q != nullptr) {
    // heads per warp, in whole passes: as many as leave 16 warps an SM
    p.q_heads = (p.Hq + R - 1) / R * R;
    while (p.q_heads > R && static_cast<int64_t>(p.T) * ((p.Hq + p.q_heads - 1) / p.q_heads) < fill)
      p.q_heads = (p.q_heads / R + 1) / 2 * R;
    p.q_parts = (p.Hq + p.q_heads - 1) / p.q_heads;
    blocks += (static_cast<int64_t>(p.T) * p.q_parts + kAppendWarps - 1) / kAppendWarps;
  }
  cudaError_t e = cudaSuccess;
  constexpr int kSmem = kAppendWarps * 2 * kStageBytes;
  struct Tag {};
  if ((e = allow_smem<Tag>(reinterpret_cast<const void*>(k), kSmem)) != cudaSuccess) return e;
  KVQ_LAUNCH("append_kernel", s, k<<<static_cast<unsigned>(blocks), 32 * kAppendWarps, kSmem, s>>>(p); e = cudaGetLastError());
  return e;
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
  int L = 1;
  while (16 * L < p.D) L <<= 1;
  switch (L) {
    case 1: return append_launch<1>(p, s);
    case 2: return append_launch<2>(p, s);
    case 4: return append_launch<4>(p, s);
    case 8: return append_launch<8>(p, s);
    case 16: return append_launch<16>(p, s);
  }
  return append_launch<32>(p, s);
}

}  // namespace kvq
