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
// Mapping: rows of one page that stand next to each other in slot_ids form a run; one warp
// serves (run, head, tensor), so scales and bounds need no atomics.  L = D / 8 lanes (rounded up to a
// power of two; at most 32, with two chunks each above head_dim 256) hold 8 channels of a row each,
// 32 / L rows a pass, kBatch passes' loads in flight; halves of a pair in different lanes meet by shuffles.
// Pages up to kBatch passes stay in registers, as they came, between the maximum and the codes
// (page scales), larger ones are read twice; both turn K twice.  Neighbouring warps take the heads of the
// same tokens, so a token's angles come from L1 but once.  Behind those blocks of the grid, others
// turn Q: a warp holds a token's angles in registers and walks its heads.
#include "page_scale.cuh"
#include "kvq_params.h"

namespace kvq {

namespace {

constexpr int kAppendThreads = 128;

// What a lane does for its chunk ch of 8 channels: where the chunk's first angle stands (-1: not turned),
// and, with pairs rot / 2 apart, where the partner chunk is and whether this one holds the b of its pairs.
struct Turn {
  int at, lane, slot;
  bool second;
};
__device__ __forceinline__ Turn make_turn(int rot, bool pairs, int ch, int base) {
  const int half = rot / 16;  // chunks of a half
  Turn t;
  const bool in = ch < 2 * half;
  t.second = !pairs && in && ch >= half;
  const int partner = pairs || !in ? ch : (t.second ? ch - half : ch + half);
  t.lane = base + partner % 32;
  t.slot = partner / 32;
  t.at = !in ? -1 : pairs ? 4 * ch : 8 * (t.second ? ch - half : ch);
  return t;
}

// Cosines and signed sines of the chunk as pairs of neighbouring channels: y = x c + p s with p the
// partner channel, s negative where the channel is the a of its pair.
struct Angles {
  uint64_t c[4], s[4];
};
__device__ __forceinline__ void load_angles(const Turn& t, int rot, bool pairs, const float* row, Angles& a) {
  if (t.at < 0) return;
  const uint4* const c = reinterpret_cast<const uint4*>(row + t.at);
  const uint4* const s = reinterpret_cast<const uint4*>(row + rot / 2 + t.at);
  if (pairs) {
    const uint4 u = LDX(c), v = LDX(s);
    constexpr uint32_t kNeg = 0x80000000u;
    a.c[0] = pack_f32x2(u.x, u.x), a.c[1] = pack_f32x2(u.y, u.y), a.c[2] = pack_f32x2(u.z, u.z), a.c[3] = pack_f32x2(u.w, u.w);
    a.s[0] = pack_f32x2(v.x ^ kNeg, v.x), a.s[1] = pack_f32x2(v.y ^ kNeg, v.y);
    a.s[2] = pack_f32x2(v.z ^ kNeg, v.z), a.s[3] = pack_f32x2(v.w ^ kNeg, v.w);
  } else {
    const uint4 u0 = LDX(c), u1 = LDX(c + 1), v0 = LDX(s), v1 = LDX(s + 1);
    const uint32_t n = t.second ? 0u : 0x80000000u;
    a.c[0] = pack_f32x2(u0.x, u0.y), a.c[1] = pack_f32x2(u0.z, u0.w), a.c[2] = pack_f32x2(u1.x, u1.y), a.c[3] = pack_f32x2(u1.z, u1.w);
    a.s[0] = pack_f32x2(v0.x ^ n, v0.y ^ n), a.s[1] = pack_f32x2(v0.z ^ n, v0.w ^ n);
    a.s[2] = pack_f32x2(v1.x ^ n, v1.y ^ n), a.s[3] = pack_f32x2(v1.z ^ n, v1.w ^ n);
  }
}

// The lane's chunks in binary32, turned.  Every lane of the warp takes part (rot: uniform, 0 for none).
template <int C>
__device__ __forceinline__ void turn8(const Turn (&t)[C], const Angles (&a)[C], int rot, bool pairs, const uint32_t (&w)[C][4],
                                      float (&y)[C][8]) {
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[j][2 * i] = bf16lo(w[j][i]);
      y[j][2 * i + 1] = bf16hi(w[j][i]);
    }
  if (rot == 0) return;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (pairs) {
        o[i] = __byte_perm(w[j][i], 0u, 0x1032);  // the neighbour
      } else {
        o[i] = __shfl_sync(0xFFFFFFFFu, w[0][i], t[j].lane);
        if constexpr (C == 2) {
          const uint32_t o2 = __shfl_sync(0xFFFFFFFFu, w[1][i], t[j].lane);
          o[i] = t[j].slot != 0 ? o2 : o[i];
        }
      }
    }
    if (t[j].at < 0) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t x = pack_f32x2(__float_as_uint(y[j][2 * i]), __float_as_uint(y[j][2 * i + 1]));
      const uint64_t p = pack_f32x2(o[i] << 16, o[i] & 0xFFFF0000u);
      // the sums one by one: the packed sum of packed products came out as one rounding
      uint32_t m0, m1, n0, n1;
      unpack_f32x2(mul_f32x2(x, a[j].c[i]), m0, m1);
      unpack_f32x2(mul_f32x2(p, a[j].s[i]), n0, n1);
      y[j][2 * i] = __fadd_rn(__uint_as_float(m0), __uint_as_float(n0));
      y[j][2 * i + 1] = __fadd_rn(__uint_as_float(m1), __uint_as_float(n1));
    }
  }
}

__device__ __forceinline__ float absmax8(const float (&y)[8]) {
  float m = fabsf(y[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
  return m;
}

// quantize_block and fp8_quantize16 (kvq_device.cuh) of 8 binary32 values.
__device__ __forceinline__ uint32_t quantize8(const float (&y)[8], float s) {
  const float inv = (s != 0.0f) ? __frcp_rn(s) : 0.0f;
  uint32_t byte[4];
  if (!isinf(inv)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) byte[i] = e2m1x2_from_f32(__fmul_rn(y[2 * i], inv), __fmul_rn(y[2 * i + 1], inv));
  } else {  // the reciprocal overflowed, divide directly
#pragma unroll
    for (int i = 0; i < 4; ++i) byte[i] = e2m1x2_from_f32(__fdiv_rn(y[2 * i], s), __fdiv_rn(y[2 * i + 1], s));
  }
  return bytes4(byte[0], byte[1], byte[2], byte[3]);
}
__device__ __forceinline__ void fp8_quantize8(const float (&y)[8], float rs, uint32_t& c0, uint32_t& c1) {
  const float inv = (rs != 0.0f) ? __frcp_rn(rs) : 0.0f;
  uint32_t w[4];
  if (!isinf(inv)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = e4m3x2_from_f32(__fmul_rn(y[2 * i], inv), __fmul_rn(y[2 * i + 1], inv));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = e4m3x2_from_f32(__fdiv_rn(y[2 * i], rs), __fdiv_rn(y[2 * i + 1], rs));
  }
  c0 = w[0] | w[1] << 16;
  c1 = w[2] | w[3] << 16;
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

// 16 bytes that this launch reads once, or (rw) may write too.
__device__ __forceinline__ void load_row16(const void* p, uint32_t (&w)[4]) {
  if (!KVQ_OK(p, 16, 16)) {
    w[0] = w[1] = w[2] = w[3] = 0u;
    return;
  }
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "l"(p));
}

// Slot of token t: -1 where it is skipped.  `report`: the warp that speaks for the token.
__device__ __forceinline__ int64_t append_slot(const AppendParams& p, int64_t t, bool report) {
  if (t < 0 || t >= p.T) return -1;
  const int64_t s = LDX(p.slot_ids + t);
  if (s >= p.num_slots && report) set_status(p.status, 1u);
  if (p.cos_sin != nullptr) {
    const int32_t pos = LDX(p.positions + t);
    if (pos >= p.num_positions && report) set_status(p.status, 4u);
    if (pos < 0 || pos >= p.num_positions) return -1;
  }
  return s >= p.num_slots ? -1 : s;
}

template <int L, int C>
__device__ __forceinline__ void append_rows(const AppendParams& p, int64_t w) {
  constexpr int R = 32 / L;       // rows per pass
  constexpr int kBatch = 8 / C;
  const int lane = threadIdx.x & 31;
  const int li = lane % L, sub = lane / L;
  const int per = p.H * p.ntensors;
  const int64_t ci = w / per;
  const int rem = static_cast<int>(w - ci * per);
  const int tensor = rem / p.H, h = rem - tensor * p.H;
  const int64_t t0 = ci * p.chunk;
  if (t0 >= p.T) return;
  const AppendTensor ten = p.ten[tensor];
  const int rot = ten.key && p.cos_sin != nullptr ? p.rot : 0;
  const int D = p.D;
  uint16_t* const bounds = ten.key ? p.bounds : nullptr;
  Turn turn[C];
  bool act[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    turn[j] = make_turn(rot, p.pairs, li + 32 * j, lane - li);
    act[j] = 8 * (li + 32 * j) < D;
  }

  auto page_of = [&](int64_t slot) -> int64_t { return slot < 0 ? -1 : slot / p.block_size; };
  const int64_t slot = append_slot(p, t0 + lane, rem == 0);
  const int64_t before = lane == 0 ? page_of(append_slot(p, t0 - 1, false)) : -1;
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
        const int64_t s2 = append_slot(p, t + lane, false);
        const int64_t p2 = page_of(s2);
        const int m = run_bits(__ballot_sync(0xFFFFFFFFu, p2 == pg));
        begins = begins || __any_sync(0xFFFFFFFFu, lane < m && s2 == pg * p.block_size);
        n += m;
        if (m < 32) break;
      }
    }
    const bool paged = ten.fmt == 5;
    const int64_t prow = pg * p.H + h;
    float s0 = 0.0f;
    if (paged && !begins && lane == 0) s0 = LDX(ten.dst.rscale + prow);
    s0 = __shfl_sync(0xFFFFFFFFu, s0, 0);
    const uint16_t* const x = ten.x + ts * ten.row_pitch + h * ten.head_pitch + 8 * li;

    uint32_t raw[kBatch][C][4];
    auto load = [&](int r, uint32_t (&v)[C][4]) {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0u;
        if (act[j] && r < n) load_row16(x + r * ten.row_pitch + 256 * j, v[j]);
      }
    };
    auto turned = [&](int r, const uint32_t (&v)[C][4], float (&y)[C][8]) {
      Angles a[C];
      if (rot != 0 && r < n) {
        const float* const row = p.cos_sin + static_cast<int64_t>(LDX(p.positions + ts + r)) * rot;
#pragma unroll
        for (int j = 0; j < C; ++j) load_angles(turn[j], rot, p.pairs, row, a[j]);
      }
      turn8<C>(turn, a, rot, p.pairs, v, y);
    };
    auto row_of = [&](int r) -> int64_t { return LDX(p.slot_ids + ts + r) * p.H + h; };

    uint32_t lo[C][4], hi[C][4];
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[j][i] = 0x7F807F80u;
        hi[j][i] = 0xFF80FF80u;
      }
    float am = 0.0f;
    for (int k0 = 0; k0 * R < n; k0 += kBatch) {  // uniform
#pragma unroll
      for (int k = 0; k < kBatch; ++k) load((k0 + k) * R + sub, raw[k]);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int r = (k0 + k) * R + sub;
        if ((k0 + k) * R >= n) break;  // uniform
        float y[C][8];
        turned(r, raw[k], y);
        if (bounds != nullptr && r < n) {
#pragma unroll
          for (int j = 0; j < C; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t b2 = pack_bf16x2(y[j][2 * i], y[j][2 * i + 1]);
              lo[j][i] = bf16x2_min(lo[j][i], b2);
              hi[j][i] = bf16x2_max(hi[j][i], b2);
            }
        }
        float vb[C];  // 0 in lanes without a row
        float row_max = 0.0f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
          vb[j] = absmax8(y[j]);
          row_max = fmaxf(row_max, vb[j]);
        }
        if (paged) {
          am = fmaxf(am, row_max);
          continue;
        }
        const float amax = group_max<L>(row_max);
        if (ten.fmt == 3) {
          const float rs = __fdiv_rn(amax, kE4M3Max);
          const int64_t row = r < n ? row_of(r) : 0;
#pragma unroll
          for (int j = 0; j < C; ++j) {
            uint32_t c0, c1;
            fp8_quantize8(y[j], rs, c0, c1);
            if (act[j] && r < n) store8B(ten.dst.codes + row * D + 8 * (li + 32 * j), c0, c1);
          }
          if (li == 0 && r < n) STX(ten.dst.rscale + row, rs);
        } else {
          const float rs = __fdiv_rn(amax, kE2M1Max * kE4M3Max);
          const float rinv = (rs != 0.0f) ? __frcp_rn(rs) : 0.0f;
          const int64_t row = r < n ? row_of(r) : 0;
#pragma unroll
          for (int j = 0; j < C; ++j) {
            const float block = fmaxf(vb[j], __shfl_xor_sync(0xFFFFFFFFu, vb[j], 1));
            const uint32_t bsb = block_scale_code(block, rs, rinv);
            const uint32_t c = quantize8(y[j], __fmul_rn(e4m3_to_f32(bsb), rs));
            if (act[j] && r < n) {
              const int ch = li + 32 * j;
              STX(reinterpret_cast<uint32_t*>(ten.dst.codes + row * (D / 2)) + ch, c);
              if (ch % 2 == 0) STX(ten.dst.bscale + row * (D / 16) + ch / 2, static_cast<uint8_t>(bsb));
            }
          }
          if (li == 0 && r < n) STX(ten.dst.rscale + row, rs);
        }
      }
    }

    if (bounds != nullptr) {
#pragma unroll
      for (int j = 0; j < C; ++j) {
#pragma unroll
        for (int o = L; o < 32; o <<= 1)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lo[j][i] = bf16x2_min(lo[j][i], __shfl_xor_sync(0xFFFFFFFFu, lo[j][i], o));
            hi[j][i] = bf16x2_max(hi[j][i], __shfl_xor_sync(0xFFFFFFFFu, hi[j][i], o));
          }
        if (act[j] && sub == 0) {
          uint16_t* const at = bounds + prow * 2 * D + 8 * (li + 32 * j);
          if (!begins) {
            uint32_t was[4];
            load16B_rw(at, was);
#pragma unroll
            for (int i = 0; i < 4; ++i) lo[j][i] = bf16x2_min(lo[j][i], was[i]);
            load16B_rw(at + D, was);
#pragma unroll
            for (int i = 0; i < 4; ++i) hi[j][i] = bf16x2_max(hi[j][i], was[i]);
          }
          store16B(at, lo[j]);
          store16B(at + D, hi[j]);
        }
      }
    }
    if (!paged) continue;

    am = group_max<32>(am);
    if (am > 3.4028235e38f) {  // an infinity among them, the same in all lanes: once more without
      am = 0.0f;
      for (int k = 0; k * R < n; ++k) {
        const int r = k * R + sub;
        uint32_t v[C][4];
        float y[C][8];
        load(r, v);
        turned(r, v, y);
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(y[j][i]) <= 3.4028235e38f ? fabsf(y[j][i]) : 0.0f);
      }
      am = group_max<32>(am);
    }
    if (!(s0 > 0.0f && s0 <= 3.4028235e38f)) s0 = 0.0f;  // no scale stored yet
    const float s = fmaxf(s0, page_scale_need(am));
    const int64_t cpitch = static_cast<int64_t>(p.H) * D;
    if (s0 > 0.0f && s > s0) {  // the rows that the page holds, under the new scale
      const float f = __fdiv_rn(s0, s);
      uint8_t* const cp = ten.dst.codes + (pg * p.block_size * p.H + h) * D;
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
    if (lane == 0 && s != s0) STX(ten.dst.rscale + prow, s);
    const bool kept = n <= kBatch * R;  // in raw
    for (int k0 = 0; k0 * R < n; k0 += kBatch) {
      if (!kept) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) load((k0 + k) * R + sub, raw[k]);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int r = (k0 + k) * R + sub;
        if ((k0 + k) * R >= n) break;  // uniform
        float y[C][8];
        turned(r, raw[k], y);
        if (r >= n) continue;
        const int64_t row = row_of(r);
#pragma unroll
        for (int j = 0; j < C; ++j) {
          uint32_t c0, c1;
          fp8_quantize8(y[j], s, c0, c1);
          if (act[j]) store8B(ten.dst.codes + row * D + 8 * (li + 32 * j), c0, c1);
        }
      }
    }
  }
}

// Q: warp w takes heads first .. of one token, 32 / L at a time.
template <int L, int C>
__device__ __forceinline__ void append_turn_q(const AppendParams& p, int64_t w) {
  constexpr int R = 32 / L;
  constexpr int kBatch = 4 / C;
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
  Turn turn[C];
  Angles a[C];
  bool act[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    turn[j] = make_turn(p.rot, p.pairs, li + 32 * j, lane - li);
    act[j] = 8 * (li + 32 * j) < p.D;
    load_angles(turn[j], p.rot, p.pairs, p.cos_sin + static_cast<int64_t>(pos) * p.rot, a[j]);
  }
  const uint16_t* const x = p.q + t * p.q_row_pitch + 8 * li;
  uint16_t* const y_at = p.q_out + t * p.qo_row_pitch + 8 * li;
  const int end = min(first + p.q_heads, p.Hq);
  for (int h0 = first; h0 < end; h0 += kBatch * R) {
    uint32_t raw[kBatch][C][4];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h0 + k * R + sub;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        raw[k][j][0] = raw[k][j][1] = raw[k][j][2] = raw[k][j][3] = 0u;
        if (act[j] && h < end) load16B_rw(x + h * p.q_head_pitch + 256 * j, raw[k][j]);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h0 + k * R + sub;
      float y[C][8];
      turn8<C>(turn, a, p.rot, p.pairs, raw[k], y);
#pragma unroll
      for (int j = 0; j < C; ++j) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(y[j][2 * i], y[j][2 * i + 1]);
        if (act[j] && h < end) store16B(y_at + h * p.qo_head_pitch + 256 * j, o);
      }
    }
  }
}

template <int L, int C>
__global__ void __launch_bounds__(kAppendThreads, 4) append_kernel(const AppendParams p) {
  const int64_t warp = threadIdx.x >> 5;
  const int64_t block = blockIdx.x;
  if (block < p.row_blocks) {
    append_rows<L, C>(p, block * (kAppendThreads / 32) + warp);
  } else {
    append_turn_q<L, C>(p, (block - p.row_blocks) * (kAppendThreads / 32) + warp);
  }
}

template <int L, int C>
cudaError_t append_launch(const AppendParams& p_in, cudaStream_t s) {
  AppendParams p = p_in;
  constexpr int kW = kAppendThreads / 32, R = 32 / L;
  auto k = append_kernel<L, C>;
  // tokens per warp: as many as leave 16 warps an SM (one token a warp in a decode step, whose
  // runs are single rows; 32 in a prompt)
  const int64_t rows = static_cast<int64_t>(p.T) * p.H * p.ntensors, fill = 16ll * num_sms();
  p.chunk = 32;
  while (p.chunk > 1 && rows < p.chunk * fill) p.chunk >>= 1;
  const int64_t warps = (static_cast<int64_t>(p.T) + p.chunk - 1) / p.chunk * p.H * p.ntensors;
  p.row_blocks = (warps + kW - 1) / kW;
  int64_t blocks = p.row_blocks;
  if (p.q != nullptr) {
    // heads per warp, in whole passes: likewise
    p.q_heads = (p.Hq + R - 1) / R * R;
    while (p.q_heads > R && static_cast<int64_t>(p.T) * ((p.Hq + p.q_heads - 1) / p.q_heads) < fill)
      p.q_heads = (p.q_heads / R + 1) / 2 * R;
    p.q_parts = (p.Hq + p.q_heads - 1) / p.q_heads;
    blocks += (static_cast<int64_t>(p.T) * p.q_parts + kW - 1) / kW;
  }
  cudaError_t e = cudaSuccess;
  KVQ_LAUNCH("append_kernel", s, k<<<static_cast<unsigned>(blocks), kAppendThreads, 0, s>>>(p); e = cudaGetLastError());
  return e;
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
  if (p.D > 256) return append_launch<32, 2>(p, s);
  int L = 2;
  while (8 * L < p.D) L <<= 1;
  switch (L) {
    case 2: return append_launch<2, 1>(p, s);
    case 4: return append_launch<4, 1>(p, s);
    case 8: return append_launch<8, 1>(p, s);
    case 16: return append_launch<16, 1>(p, s);
  }
  return append_launch<32, 1>(p, s);
}

}  // namespace kvq
