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
// serves (run, head, tensor), so scales and bounds need no atomics.  L = D / 16 lanes (rounded
// up to a power of two) read a row as 32 bytes each, 32 / L rows a pass, kBatch passes' loads in
// flight; halves of a pair in different lanes meet by shuffles.  Pages up to kBatch passes stay in
// registers between the maximum and the codes (page scales), larger ones are read twice.
// Neighbouring warps take the heads of the same tokens, so a token's angles come from L1 but
// once.  Behind those blocks of the grid, others turn Q: a warp holds a token's angles in
// registers and walks its heads.
#include "page_scale.cuh"
#include "kvq_params.h"

namespace kvq {

namespace {

constexpr int kAppendThreads = 128;
constexpr int kBatch = 4;

// Cosines and sines of a lane's two 8-channel chunks: 8 pairs a chunk where the halves of a
// pair are rot / 2 apart, 4 where they are neighbours.
struct Angles {
  float c[2][8], s[2][8];
};

// What a lane does for its chunks 2 li and 2 li + 1.
struct Turn {
  int rot;           // channels turned; 0: none
  bool pairs;        // neighbours
  bool cross;        // a partner chunk is the other half of its lane's
  int src[2];        // lane of the partner chunk
  int at[2];         // first angle of the chunk; -1: not turned
  bool second[2];    // the chunk holds the b of its pairs
};

template <int L>
__device__ __forceinline__ Turn make_turn(int rot, bool pairs, int lane) {
  Turn t;
  t.rot = rot;
  t.pairs = pairs;
  const int li = lane % L, base = lane - li, half = rot / 16;  // chunks of a half
  t.cross = !pairs && (half & 1) != 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int ch = 2 * li + j;
    const bool in = ch < 2 * half;
    t.second[j] = !pairs && in && ch >= half;
    const int partner = pairs || !in ? ch : (t.second[j] ? ch - half : ch + half);
    t.src[j] = base + partner / 2;
    t.at[j] = !in ? -1 : pairs ? 4 * ch : 8 * (t.second[j] ? ch - half : ch);
  }
  return t;
}

__device__ __forceinline__ void load_angles(const Turn& t, const float* row, Angles& a) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (t.at[j] < 0) continue;
    const float4* const c = reinterpret_cast<const float4*>(row + t.at[j]);
    const float4* const s = reinterpret_cast<const float4*>(row + t.rot / 2 + t.at[j]);
    const float4 c0 = LDX(c), s0 = LDX(s);
    a.c[j][0] = c0.x, a.c[j][1] = c0.y, a.c[j][2] = c0.z, a.c[j][3] = c0.w;
    a.s[j][0] = s0.x, a.s[j][1] = s0.y, a.s[j][2] = s0.z, a.s[j][3] = s0.w;
    if (!t.pairs) {
      const float4 c1 = LDX(c + 1), s1 = LDX(s + 1);
      a.c[j][4] = c1.x, a.c[j][5] = c1.y, a.c[j][6] = c1.z, a.c[j][7] = c1.w;
      a.s[j][4] = s1.x, a.s[j][5] = s1.y, a.s[j][6] = s1.z, a.s[j][7] = s1.w;
    }
  }
}

// The lane's 16 channels in binary32, turned.  Every lane of the warp takes part.
__device__ __forceinline__ void turn16(const Turn& t, const Angles& a, const uint32_t (&w)[8], float (&y)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[2 * i] = bf16lo(w[i]);
    y[2 * i + 1] = bf16hi(w[i]);
  }
  if (t.rot == 0) return;  // uniform
  if (t.pairs) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (t.at[j] < 0) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x0 = y[8 * j + 2 * i], x1 = y[8 * j + 2 * i + 1];
        y[8 * j + 2 * i] = __fsub_rn(__fmul_rn(x0, a.c[j][i]), __fmul_rn(x1, a.s[j][i]));
        y[8 * j + 2 * i + 1] = __fadd_rn(__fmul_rn(x1, a.c[j][i]), __fmul_rn(x0, a.s[j][i]));
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = __shfl_sync(0xFFFFFFFFu, t.cross ? w[4 * (1 - j) + i] : w[4 * j + i], t.src[j]);
    if (t.at[j] < 0) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p0 = bf16lo(o[i]), p1 = bf16hi(o[i]);
      float &y0 = y[8 * j + 2 * i], &y1 = y[8 * j + 2 * i + 1];
      const float m0 = __fmul_rn(y0, a.c[j][2 * i]), n0 = __fmul_rn(p0, a.s[j][2 * i]);
      const float m1 = __fmul_rn(y1, a.c[j][2 * i + 1]), n1 = __fmul_rn(p1, a.s[j][2 * i + 1]);
      y0 = t.second[j] ? __fadd_rn(m0, n0) : __fsub_rn(m0, n0);
      y1 = t.second[j] ? __fadd_rn(m1, n1) : __fsub_rn(m1, n1);
    }
  }
}

__device__ __forceinline__ float absmax16f(const float (&y)[16]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(y[i]));
  return m;
}

// quantize_block and fp8_quantize16 (kvq_device.cuh) of binary32 values.
__device__ __forceinline__ void quantize_block_f(const float (&y)[16], float s, uint32_t& c0, uint32_t& c1) {
  const float inv = (s != 0.0f) ? __frcp_rn(s) : 0.0f;
  const bool tiny = isinf(inv);  // the reciprocal overflowed, divide directly
  uint32_t byte[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    byte[i] = tiny ? e2m1x2_from_f32(__fdiv_rn(y[2 * i], s), __fdiv_rn(y[2 * i + 1], s))
                   : e2m1x2_from_f32(__fmul_rn(y[2 * i], inv), __fmul_rn(y[2 * i + 1], inv));
  c0 = bytes4(byte[0], byte[1], byte[2], byte[3]);
  c1 = bytes4(byte[4], byte[5], byte[6], byte[7]);
}
__device__ __forceinline__ void fp8_quantize16_f(const float (&y)[16], float rs, uint32_t (&c)[4]) {
  const float inv = (rs != 0.0f) ? __frcp_rn(rs) : 0.0f;
  const bool tiny = isinf(inv);
  c[0] = c[1] = c[2] = c[3] = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i / 2] |= (tiny ? e4m3x2_from_f32(__fdiv_rn(y[2 * i], rs), __fdiv_rn(y[2 * i + 1], rs))
                      : e4m3x2_from_f32(__fmul_rn(y[2 * i], inv), __fmul_rn(y[2 * i + 1], inv)))
                << (16 * (i % 2));
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

template <int L, bool kV8>
__device__ __forceinline__ void append_rows(const AppendParams& p, int64_t w) {
  constexpr int R = 32 / L;  // rows per pass
  const int lane = threadIdx.x & 31;
  const int li = lane % L, sub = lane / L;
  const bool act = li < p.nb;
  const int per = p.H * p.ntensors;
  const int64_t ci = w / per;
  const int rem = static_cast<int>(w - ci * per);
  const int tensor = rem / p.H, h = rem - tensor * p.H;
  const int64_t t0 = ci * p.chunk;
  if (t0 >= p.T) return;
  const AppendTensor ten = p.ten[tensor];
  const Turn turn = make_turn<L>(ten.key && p.cos_sin != nullptr ? p.rot : 0, p.pairs, lane);
  uint16_t* const bounds = ten.key ? p.bounds : nullptr;
  const int D = 16 * p.nb;

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
    const uint16_t* const x = ten.x + ts * ten.row_pitch + h * ten.head_pitch + 16 * li;
    const int code_bytes = ten.fmt == 1 ? D / 2 : D;

    auto load = [&](int r, uint32_t (&v)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0u;
      if (act && r < n) load32B<kV8, true>(x + r * ten.row_pitch, v);
    };
    auto turned = [&](int r, const uint32_t (&v)[8], float (&y)[16]) {
      Angles a;
      if (turn.rot != 0 && r < n)
        load_angles(turn, p.cos_sin + static_cast<int64_t>(LDX(p.positions + ts + r)) * p.rot, a);
      turn16(turn, a, v, y);
    };
    auto row_of = [&](int r) -> int64_t { return LDX(p.slot_ids + ts + r) * p.H + h; };

    uint32_t lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = 0x7F807F80u;
      hi[i] = 0xFF80FF80u;
    }
    float held[kBatch][16];
    float am = 0.0f;
    for (int k0 = 0; k0 * R < n; k0 += kBatch) {  // uniform
      uint32_t raw[kBatch][8];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) load((k0 + k) * R + sub, raw[k]);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int r = (k0 + k) * R + sub;
        if ((k0 + k) * R >= n) break;  // uniform
        float y[16];
        turned(r, raw[k], y);
        const bool live = act && r < n;
        if (bounds != nullptr && live) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t b2 = pack_bf16x2(y[2 * i], y[2 * i + 1]);
            lo[i] = bf16x2_min(lo[i], b2);
            hi[i] = bf16x2_max(hi[i], b2);
          }
        }
        const float vb = absmax16f(y);  // 0 in lanes without a row
        if (paged) {
          am = fmaxf(am, vb);
          if (k0 == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) held[k][i] = y[i];
          }
          continue;
        }
        const float amax = group_max<L>(vb);
        if (ten.fmt == 3) {
          const float rs = __fdiv_rn(amax, kE4M3Max);
          uint32_t c[4];
          fp8_quantize16_f(y, rs, c);
          if (live) {
            const int64_t row = row_of(r);
            store16B(ten.dst.codes + row * code_bytes + 16 * li, c);
            if (li == 0) STX(ten.dst.rscale + row, rs);
          }
        } else {
          const float rs = __fdiv_rn(amax, kE2M1Max * kE4M3Max);
          const float rinv = (rs != 0.0f) ? __frcp_rn(rs) : 0.0f;
          const uint32_t bsb = block_scale_code(vb, rs, rinv);
          uint32_t c0, c1;
          quantize_block_f(y, __fmul_rn(e4m3_to_f32(bsb), rs), c0, c1);
          if (live) {
            const int64_t row = row_of(r);
            store8B(ten.dst.codes + row * code_bytes + 8 * li, c0, c1);
            STX(ten.dst.bscale + row * p.nb + li, static_cast<uint8_t>(bsb));
            if (li == 0) STX(ten.dst.rscale + row, rs);
          }
        }
      }
    }

    if (bounds != nullptr) {
#pragma unroll
      for (int o = L; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          lo[i] = bf16x2_min(lo[i], __shfl_xor_sync(0xFFFFFFFFu, lo[i], o));
          hi[i] = bf16x2_max(hi[i], __shfl_xor_sync(0xFFFFFFFFu, hi[i], o));
        }
      if (act && sub == 0) {
        uint16_t* const at = bounds + prow * 2 * D + 16 * li;
        if (!begins) {
          uint32_t was[8];
          load32B<false, false>(at, was);
#pragma unroll
          for (int i = 0; i < 8; ++i) lo[i] = bf16x2_min(lo[i], was[i]);
          load32B<false, false>(at + D, was);
#pragma unroll
          for (int i = 0; i < 8; ++i) hi[i] = bf16x2_max(hi[i], was[i]);
        }
        store32B<false>(at, lo);
        store32B<false>(at + D, hi);
      }
    }
    if (!paged) continue;

    am = group_max<32>(am);
    if (am > 3.4028235e38f) {  // an infinity among them, the same in all lanes: once more without
      am = 0.0f;
      for (int k = 0; k * R < n; ++k) {
        const int r = k * R + sub;
        uint32_t v[8];
        float y[16];
        load(r, v);
        turned(r, v, y);
#pragma unroll
        for (int i = 0; i < 16; ++i) am = fmaxf(am, fabsf(y[i]) <= 3.4028235e38f ? fabsf(y[i]) : 0.0f);
      }
      am = group_max<32>(am);
    }
    if (!(s0 > 0.0f && s0 <= 3.4028235e38f)) s0 = 0.0f;  // no scale stored yet
    const float s = fmaxf(s0, page_scale_need(am));
    uint8_t* const cp = ten.dst.codes + (pg * p.block_size * p.H + h) * D + 16 * li;
    const int64_t cpitch = static_cast<int64_t>(p.H) * D;
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
    if (lane == 0 && s != s0) STX(ten.dst.rscale + prow, s);
    auto put = [&](const float (&y)[16], int r) {
      if (!(act && r < n)) return;
      uint32_t c[4];
      fp8_quantize16_f(y, s, c);
      store16B(ten.dst.codes + row_of(r) * D + 16 * li, c);
    };
#pragma unroll
    for (int k = 0; k < kBatch; ++k) put(held[k], k * R + sub);
    for (int k = kBatch; k * R < n; ++k) {
      const int r = k * R + sub;
      uint32_t v[8];
      float y[16];
      load(r, v);
      turned(r, v, y);
      put(y, r);
    }
  }
}

// Q: warp w takes heads first .. of one token, 32 / L at a time.
template <int L, bool kV8>
__device__ __forceinline__ void append_turn_q(const AppendParams& p, int64_t w) {
  constexpr int R = 32 / L;
  const int lane = threadIdx.x & 31;
  const int li = lane % L, sub = lane / L;
  const bool act = li < p.nb;
  const int64_t t = w / p.q_parts;
  if (t >= p.T) return;
  const int first = static_cast<int>(w - t * p.q_parts) * p.q_heads;
  const int32_t pos = LDX(p.positions + t);
  if (pos < 0) return;
  if (pos >= p.num_positions) {
    if (lane == 0 && first == 0) set_status(p.status, 4u);
    return;
  }
  const Turn turn = make_turn<L>(p.rot, p.pairs, lane);
  Angles a;
  if (act) load_angles(turn, p.cos_sin + static_cast<int64_t>(pos) * p.rot, a);
  const uint16_t* const x = p.q + t * p.q_row_pitch + 16 * li;
  uint16_t* const y_at = p.q_out + t * p.qo_row_pitch + 16 * li;
  const int end = min(first + p.q_heads, p.Hq);
  for (int h0 = first; h0 < end; h0 += kBatch * R) {
    uint32_t raw[kBatch][8];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h0 + k * R + sub;
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[k][i] = 0u;
      if (act && h < end) load32B<kV8, false>(x + h * p.q_head_pitch, raw[k]);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h0 + k * R + sub;
      float y[16];
      turn16(turn, a, raw[k], y);
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
      if (act && h < end) store32B<kV8>(y_at + h * p.qo_head_pitch, o);
    }
  }
}

template <int L, bool kV8>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  const int64_t warp = threadIdx.x >> 5;
  const int64_t block = blockIdx.x;
  if (block < p.row_blocks) {
    append_rows<L, kV8>(p, block * (kAppendThreads / 32) + warp);
  } else {
    append_turn_q<L, kV8>(p, (block - p.row_blocks) * (kAppendThreads / 32) + warp);
  }
}

template <int L, bool kV8>
cudaError_t append_launch(const AppendParams& p_in, cudaStream_t s) {
  AppendParams p = p_in;
  constexpr int kW = kAppendThreads / 32, R = 32 / L;
  auto k = append_kernel<L, kV8>;
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

cudaError_t launch_append(const AppendParams& p, bool v8, cudaStream_t s) {
  int L = 1;
  while (L < p.nb) L <<= 1;
#define KVQ_APPEND(N) \
  if (L == N) return v8 ? append_launch<N, true>(p, s) : append_launch<N, false>(p, s);
  KVQ_APPEND(1) KVQ_APPEND(2) KVQ_APPEND(4) KVQ_APPEND(8) KVQ_APPEND(16) KVQ_APPEND(32)
#undef KVQ_APPEND
  return cudaErrorInvalidValue;
}

}  // namespace kvq
