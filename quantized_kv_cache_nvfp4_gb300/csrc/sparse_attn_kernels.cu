// sparse_attn_kernels.cu -- paged attention over the listed blocks of each (query token, KV head).
//
// Token i of a sequence's last n sits at p = len - n + i; KV head h of it has a list of topk
// blocks, and its query heads see the keys t <= p of those (an entry below 0 or past p has none;
// one that stands there twice counts twice).  Logits are cap(scale q . k_t); a row that sees no key
// is 0.
//
// A thread block takes one (split of the list, KV head, token): the group's query heads are the
// rows of the tiles, since they alone share a list.  It first looks its entries up (list and block
// table, all at once) into shared memory; then its 4 warps take 16 of the listed keys in turn
// through cp.async rings with the tile arithmetic of the other attention kernels (attn_tile.cuh).
// Keys outside the row's sight become zeros in shared memory and -inf among the scores.  Up to 8 splits
// of a list merge as a cluster, more through the caller's workspace in the merge kernel of kvq_attention.
#include <algorithm>

#include "query_attn.cuh"

namespace kvq {

namespace {

// Logits of a tile whose rows all see the same keys: a cap, and the keys that are not there.
template <int kNH>
struct SparseMod {
  static constexpr bool kActive = true;
  static constexpr bool mixed = false;
  float f[kNH][2];  // the row's factor: times 2 log2 e / cap, else 1 (qmul carries it)
  float c2;         // cap log2 e, 0: no cap
  uint32_t keys;    // bit j: key j of the tile is seen

  __device__ __forceinline__ void operator()(float (&sc)[kNH][4]) const {
    if (c2 > 0.0f) {  // c2 tanh(x) = c2 - 2 c2 / (1 + e^2x), as in QueryMod
#pragma unroll
      for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sc[nh][e] = __fmaf_rn(-2.0f * c2, rcp_ftz(1.0f + ex2_ftz(sc[nh][e] * f[nh][e & 1])), c2);
    }
    if (keys != 0xFFFFu) {  // uniform
      const int g = (threadIdx.x & 31) >> 2;
      const bool off0 = ((keys >> g) & 1u) == 0u, off1 = ((keys >> (g + 8)) & 1u) == 0u;
#pragma unroll
      for (int nh = 0; nh < kNH; ++nh) {
        if (off0) sc[nh][0] = sc[nh][1] = kNegInf;
        if (off1) sc[nh][2] = sc[nh][3] = kNegInf;
      }
    }
  }
};

// The ring and shared memory of a thread block.  Two stages where a tile is over 4 KB: four blocks an SM
// instead of three, and one tile a warp ahead (32 x 8 lists of 128 16-token blocks, head_dim 128, page
// scales: 36.6 us, with three stages 38.2; 512 x 8 lists of 32 64-token blocks 282 and 316).  Three at
// head_dim 256, where two blocks fit either way (27 x 4 lists 16.1 us, with two stages 18.5).
template <int D, int kFK, int kFV>
struct SparseRing {
  using T = AttnTile<D, kFK, kFV>;
  static constexpr int kStages = D == 256 && T::kBytes > 4096 ? 3 : T::kBytes > 4096 ? 2 : 4;
  static constexpr int kRing = kAttnWarps * kStages * T::kBytes;
  static constexpr int kMerge = kAttnWarps * 16 * (D + 4) * 4;
  static constexpr int kSmem = T::kQ + (kRing > kMerge ? kRing : kMerge);
};

// Up to this many splits of a list are one thread-block cluster and merge through each other's shared
// memory: a second kernel costs 4 us.
constexpr int kClusterSplits = 8;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A float of this thread block's shared memory, read in block `rank` of the cluster.
__device__ __forceinline__ float peer_float(const float* mine, uint32_t rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(mine))), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ float4 peer_float4(const float* mine, uint32_t rank) {
  uint32_t at;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(mine))), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

template <int D, int kFK, int kFV, int kNH>
__global__ void __launch_bounds__(kAttnThreads, D == 128 && kNH == 1 ? 4 : 1) sparse_rows_kernel(const SparseAttnParams sp) {
  using T = AttnTile<D, kFK, kFV>;
  using Ring = SparseRing<D, kFK, kFV>;
  constexpr int kStages = Ring::kStages;
  const QueryAttnParams& qp = sp.q;
  const AttnParams& p = qp.a;
  constexpr int kKS = D / 16, kMT = D / 16, kRows = 8 * kNH;
  constexpr bool kQReg = kNH * kKS <= 8;
  extern __shared__ __align__(16) unsigned char smem[];
  int2* const entries = reinterpret_cast<int2*>(smem + Ring::kSmem);  // {block of the pool or -1, first token}
  __shared__ uint32_t seen[kAttnWarps][kStages];
  __shared__ int last_entry;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int s = blockIdx.z, h = blockIdx.y;
  const int i = static_cast<int>(blockIdx.x) / p.nsplit, split = static_cast<int>(blockIdx.x) - i * p.nsplit;

  int q0, nq, len;
  const bool ok = query_range(qp, s, q0, nq, len);
  if (!ok && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) set_status(p.status, 8u);
  if (i >= nq) return;
  const int64_t tok = q0 + i;
  const int pos = len - nq + i, rows = p.group;
  const int32_t own_block = static_cast<int32_t>(p.div_bs.div(static_cast<uint32_t>(pos)));

  // ---- Q^T fragments (rows: query heads of the group) ----
  uint2* const qfrag = reinterpret_cast<uint2*>(smem);
  uint2 qreg[kQReg ? kNH : 1][kKS];
  float row_fac[kNH];
#pragma unroll
  for (int nh = 0; nh < kNH; ++nh) {
    uint2(&f)[kKS] = qreg[kQReg ? nh : 0];
    row_fac[nh] = query_fragments<D>(p, lane, h, static_cast<int>(tok), 8 * nh + g, rows, f);
    if (!kQReg && warp == 0) {
#pragma unroll
      for (int kb = 0; kb < kKS; ++kb) qfrag[(nh * kKS + kb) * 32 + lane] = f[kb];
    }
  }

  // ---- the list: up to its last entry in sight, shared in equal splits of whole tiles ----
  const int32_t* const list = sp.selected + (tok * p.H + h) * sp.topk;
  if (threadIdx.x == 0) last_entry = 0;
  __syncthreads();
  const int32_t* const table = p.block_table + static_cast<int64_t>(s) * p.max_blocks;
  int upto = 0;
  int32_t first_b = -1, first_blk = -1;  // of entry threadIdx.x, whose table entry is not waited for here
  for (int e = threadIdx.x; e < sp.topk; e += kAttnThreads) {
    const int32_t b = LDX(list + e);
    const bool in = b >= 0 && b <= own_block;
    if (in) upto = e + 1;
    if (e < kAttnThreads) {
      first_b = b;
      if (in) first_blk = LDX(table + b);
    }
  }
  upto = __reduce_max_sync(0xFFFFFFFFu, upto);
  if (lane == 0 && upto > 0) atomicMax(&last_entry, upto);
  __syncthreads();
  const int64_t all = static_cast<int64_t>(last_entry) * p.block_size;  // keys, seen or not (below 2^31)
  const int per = static_cast<int>(((all + p.nsplit - 1) / p.nsplit + 63) / 64 * 64);
  const int v_begin = static_cast<int>(min(static_cast<int64_t>(split) * per, all));
  const int v_end = static_cast<int>(min(static_cast<int64_t>(v_begin) + per, all));
  const int ntile = (v_end - v_begin + 15) / 16;
  const int e0 = static_cast<int>(p.div_bs.div(static_cast<uint32_t>(v_begin)));
  const int e1 = v_end > v_begin ? static_cast<int>(p.div_bs.div(static_cast<uint32_t>(v_end - 1))) + 1 : e0;
  bool bad = false;
  for (int e = threadIdx.x; e < e1; e += kAttnThreads) {
    if (e < e0) continue;
    const int32_t b = e < kAttnThreads ? first_b : LDX(list + e);
    int2 at = make_int2(-1, 0);
    if (b >= 0 && b <= own_block) {
      const int32_t blk = e < kAttnThreads ? first_blk : LDX(table + b);
      if (blk < 0 || blk >= p.num_blocks) {
        bad = true;
      } else {
        at = make_int2(blk, b * p.block_size);
      }
    }
    entries[e - e0] = at;
  }
  const bool cta_bad = __syncthreads_or(bad ? 1 : 0) != 0;
  if (cta_bad && threadIdx.x == 0) set_status(p.status, 2u);

  SparseMod<kNH> mod;
  float qmul[kNH][2];
  mod.c2 = qp.softcap * kLog2e;
#pragma unroll
  for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float f = __shfl_sync(0xFFFFFFFFu, row_fac[nh], 4 * (2 * c + e));
      mod.f[nh][e] = qp.softcap > 0.0f ? f * (2.0f * kLog2e / qp.softcap) : 1.0f;
      qmul[nh][e] = qp.softcap > 0.0f ? 1.0f : f * kLog2e;
    }
  auto qb = [&](int nh, int kb) -> uint2 {
    if constexpr (kQReg) {
      return qreg[nh][kb];
    } else {
      return qfrag[(nh * kKS + kb) * 32 + lane];
    }
  };

  // ---- the warp's tiles through its cp.async ring ----
  unsigned char* const ring = smem + T::kQ + warp * kStages * T::kBytes;
  const bool lane_page = lane < 16 ? p.k_page : p.v_page;
  // copies of the warp's tile number `it` into stage st; keys out of sight become zeros
  auto issue = [&](int it, int st) {
    const int kt = warp + it * kAttnWarps;
    if (kt >= ntile) return;
    unsigned char* const sb = ring + st * T::kBytes;
    const int tt = lane & 15;
    constexpr int kPK = T::kCK / 16, kPV = T::kCV / 16;
    if (sp.whole) {  // the tile lies in one block
      uint32_t e, off;
      p.div_bs.divmod(static_cast<uint32_t>(v_begin + kt * 16), e, off);
      const int2 at = entries[e - e0];
      if (at.x < 0 || at.y + static_cast<int>(off) > pos) {
        if (lane == 0) seen[warp][st] = 0u;
        return;
      }
      if (at.y + static_cast<int>(off) + 15 <= pos) {  // and in sight: rows a fixed pitch apart
        const int64_t r0 = (static_cast<int64_t>(at.x) * p.block_size + off) * p.H + h;
        const int pk = p.H * T::kCK, pv = p.H * T::kCV;
        const uint8_t* ks = p.k.codes + r0 * T::kCK + (lane / kPK) * pk + (lane % kPK) * 16;
        const uint8_t* vs = p.v.codes + r0 * T::kCV + (lane / kPV) * pv + (lane % kPV) * 16;
        unsigned char* const kd = sb + T::kOffKC + (lane / kPK) * T::kSK + (lane % kPK) * 16;
        unsigned char* const vd = sb + T::kOffVC + (lane / kPV) * T::kSV + (lane % kPV) * 16;
#pragma unroll
        for (int x = 0; x < kPK / 2; ++x) cp_async16(kd + x * (32 / kPK) * T::kSK, ks + static_cast<int64_t>(x * (32 / kPK)) * pk);
#pragma unroll
        for (int x = 0; x < kPV / 2; ++x) cp_async16(vd + x * (32 / kPV) * T::kSV, vs + static_cast<int64_t>(x * (32 / kPV)) * pv);
        const int64_t row = r0 + static_cast<int64_t>(tt) * p.H, srow = lane_page ? static_cast<int64_t>(at.x) * p.H + h : row;
        if (lane < 16) {
          if constexpr (T::kBK > 0) cp_async_n<T::kBK>(sb + T::kOffKB + tt * T::kBK, p.k.bscale + row * T::kBK);
          cp_async_small<4>(sb + T::kOffKR + tt * 4, p.k.rscale + srow);
        } else {
          if constexpr (T::kBV > 0) cp_async_n<T::kBV>(sb + T::kOffVB + tt * T::kBV, p.v.bscale + row * T::kBV);
          cp_async_small<4>(sb + T::kOffVR + tt * 4, p.v.rscale + srow);
        }
        if (lane == 0) seen[warp][st] = 0xFFFFu;
        return;
      }
    }
    const int v = v_begin + kt * 16 + tt;
    int64_t row = -1, srow = 0;
    if (v < v_end) {
      uint32_t e, off;
      p.div_bs.divmod(static_cast<uint32_t>(v), e, off);
      const int2 at = entries[e - e0];
      if (at.x >= 0 && at.y + static_cast<int>(off) <= pos) {
        row = (static_cast<int64_t>(at.x) * p.block_size + off) * p.H + h;
        srow = lane_page ? static_cast<int64_t>(at.x) * p.H + h : row;
      }
    }
    const uint32_t keys = __ballot_sync(0xFFFFFFFFu, row >= 0) & 0xFFFFu;
    if (lane == 0) seen[warp][st] = keys;
    if (keys == 0u) return;
    auto piece = [&](unsigned char* dst, const uint8_t* src, int64_t rr) {
      if (rr >= 0) cp_async16(dst, src);
      else *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
    };
#pragma unroll
    for (int x = lane; x < 16 * kPK; x += 32) {
      const int64_t rr = shfl64(row, x / kPK);
      piece(sb + T::kOffKC + (x / kPK) * T::kSK + (x % kPK) * 16, p.k.codes + rr * T::kCK + (x % kPK) * 16, rr);
    }
#pragma unroll
    for (int x = lane; x < 16 * kPV; x += 32) {
      const int64_t rr = shfl64(row, x / kPV);
      piece(sb + T::kOffVC + (x / kPV) * T::kSV + (x % kPV) * 16, p.v.codes + rr * T::kCV + (x % kPV) * 16, rr);
    }
    if (row < 0) {
      uint32_t* const b = reinterpret_cast<uint32_t*>(lane < 16 ? sb + T::kOffKB + tt * T::kBK : sb + T::kOffVB + tt * T::kBV);
      for (int x = 0; x < (lane < 16 ? T::kBK : T::kBV) / 4; ++x) b[x] = 0u;
      *reinterpret_cast<float*>(sb + (lane < 16 ? T::kOffKR : T::kOffVR) + tt * 4) = 0.0f;
    } else if (lane < 16) {
      if constexpr (T::kBK > 0) cp_async_n<T::kBK>(sb + T::kOffKB + tt * T::kBK, p.k.bscale + row * T::kBK);
      cp_async_small<4>(sb + T::kOffKR + tt * 4, p.k.rscale + srow);
    } else {
      if constexpr (T::kBV > 0) cp_async_n<T::kBV>(sb + T::kOffVB + tt * T::kBV, p.v.bscale + row * T::kBV);
      cp_async_small<4>(sb + T::kOffVR + tt * 4, p.v.rscale + srow);
    }
  };

  AttnState<D, kNH> st;
  st.init(kNoKey);
#pragma unroll
  for (int j = 0; j < kStages - 1; ++j) {
    issue(j, j);
    cp_async_commit();
  }

  const int my_tiles = ntile > warp ? (ntile - warp + kAttnWarps - 1) / kAttnWarps : 0;
  for (int it = 0; it < my_tiles; ++it) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    const int stage = it % kStages;
    const unsigned char* const sb = ring + stage * T::kBytes;
    mod.keys = seen[warp][stage];
    if (mod.keys != 0u) {
      const TileView tv{sb + T::kOffKC, sb + T::kOffVC, sb + T::kOffKB, sb + T::kOffVB, sb + T::kOffKR, sb + T::kOffVR,
                        T::kSK, T::kSV, T::kBK, T::kBV, 4, 4};
      attn_tile<D, kFK, kFV, kNH>(tv, qb, qmul, lane, 16, st, mod);
    }
    __syncwarp();
    issue(it + kStages - 1, (it + kStages - 1) % kStages);
    cp_async_commit();
  }
  cp_async_wait<0>();
  if (!sp.cluster) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll
  for (int off = 4; off <= 16; off <<= 1)
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh) {
      st.l[nh][0] += __shfl_xor_sync(0xFFFFFFFFu, st.l[nh][0], off);
      st.l[nh][1] += __shfl_xor_sync(0xFFFFFFFFu, st.l[nh][1], off);
    }
  // ---- the warps' parts, on one reference: M of the four, then O and L scaled as they are written ----
  constexpr int kPitch = D + 4;  // floats of a row
  __shared__ float warp_m[kAttnWarps][kRows], warp_l[kAttnWarps][kRows];
  __shared__ __align__(16) float merged[2 * kRows];  // M, then L
  if (g == 0) {
#pragma unroll
    for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
      for (int e = 0; e < 2; ++e) warp_m[warp][8 * nh + 2 * c + e] = st.m[nh][e];
  }
  __syncthreads();  // and the ring is free
  float* const mo = reinterpret_cast<float*>(smem + T::kQ);  // [warp][row][kPitch]
#pragma unroll
  for (int nh = 0; nh < kNH; ++nh)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 8 * nh + 2 * c + e;
      float M = kNoKey;
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) M = fmaxf(M, warp_m[w][row]);
      const float f = ex2(st.m[nh][e] - M), fo = f * st.R;
      if (g == 0) {
        warp_l[warp][row] = st.l[nh][e] * f;
        if (warp == 0) merged[row] = cta_bad ? __int_as_float(0x7FC00000) : M;  // NaN marks a bad block entry (M never is one)
      }
      float* const to = mo + (warp * kRows + row) * kPitch + g * (D / 8);
#pragma unroll
      for (int q = 0; q < kMT; q += 2)
        *reinterpret_cast<float4*>(to + 2 * q) = make_float4(st.o[q][nh][e] * fo, st.o[q][nh][e + 2] * fo,
                                                             st.o[q + 1][nh][e] * fo, st.o[q + 1][nh][e + 2] * fo);
    }
  __syncthreads();
  auto put = [&](int row, int d, float4 o, float L) {
    uint32_t* const out = reinterpret_cast<uint32_t*>(p.out + tok * p.o_row_pitch +
                                                      static_cast<int64_t>(h * p.group + row) * p.o_head_pitch + d);
    const bool none = L == 0.0f;  // a NaN goes on
    STX(reinterpret_cast<uint2*>(out), make_uint2(none ? 0u : pack_bf16x2(o.x / L, o.y / L), none ? 0u : pack_bf16x2(o.z / L, o.w / L)));
  };
  for (int idx = threadIdx.x; idx < rows * (D / 4); idx += kAttnThreads) {
    const int row = idx / (D / 4), d = 4 * (idx % (D / 4));
    float L = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(mo + (w * kRows + row) * kPitch + d);
      L += warp_l[w][row];
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
    }
    if (p.nsplit == 1) {
      if (!cta_bad) put(row, d, o, L);
    } else if (sp.cluster) {
      *reinterpret_cast<float4*>(mo + row * kPitch + d) = o;  // what no other thread reads
      if (d == 0) merged[kRows + row] = L;
    } else {
      float* const wsr = p.ws + ((tok * p.Hq + h * p.group + row) * p.nsplit + split) * (D + 2);
      STX(reinterpret_cast<float2*>(wsr + d), make_float2(o.x, o.y));
      STX(reinterpret_cast<float2*>(wsr + d + 2), make_float2(o.z, o.w));
      if (d == 0) STX(reinterpret_cast<float2*>(wsr + D), make_float2(merged[row], L));
    }
  }
  if (!sp.cluster) return;
  cluster_sync();
  // four channels a thread, shared among the cluster's blocks (block `split` of it is this one)
  for (int idx = split * kAttnThreads + static_cast<int>(threadIdx.x); idx < rows * (D / 4); idx += p.nsplit * kAttnThreads) {
    const int row = idx / (D / 4), d = 4 * (idx % (D / 4));
    float m[kClusterSplits], M = kNoKey;
    bool skip = false;
#pragma unroll
    for (int x = 0; x < kClusterSplits; ++x) {
      m[x] = x < p.nsplit ? peer_float(merged + row, x) : kNegInf;
      skip = skip || isnan(m[x]);
      M = fmaxf(M, m[x]);
    }
    float L = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
    for (int x = 0; x < p.nsplit; ++x) {
      const float4 y = peer_float4(mo + row * kPitch + d, x);
      float f = ex2(peer_float(merged + row, x) - M);
      L = __fmaf_rn(peer_float(merged + kRows + row, x), f, L);
      o.x = __fmaf_rn(y.x, f, o.x), o.y = __fmaf_rn(y.y, f, o.y), o.z = __fmaf_rn(y.z, f, o.z), o.w = __fmaf_rn(y.w, f, o.w);
    }
    if (!skip) put(row, d, o, L);
  }
  cluster_sync();  // its shared memory is read
}

template <int D, int kFK, int kFV, int kNH>
cudaError_t sparse_launch(const SparseAttnParams& p, cudaStream_t s) {
  auto k = sparse_rows_kernel<D, kFK, kFV, kNH>;
  const int64_t keys = static_cast<int64_t>(p.topk) * p.q.a.block_size;
  const int64_t per = ((keys + p.q.a.nsplit - 1) / p.q.a.nsplit + 63) / 64 * 64;
  const int64_t entries = std::min(static_cast<int64_t>(p.topk), per / p.q.a.block_size + 2);
  const size_t smem = SparseRing<D, kFK, kFV>::kSmem + static_cast<size_t>(entries) * sizeof(int2);
  struct Tag {};
  cudaError_t e = allow_smem<Tag>(reinterpret_cast<const void*>(k), 200 * 1024);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(p.q.max_q) * p.q.a.nsplit), p.q.a.H, p.q.a.S);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kAttnThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.q.a.nsplit);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster ? 1 : 0;
  KVQ_LAUNCH("sparse_rows_kernel", s, e = cudaLaunchKernelEx(&cfg, k, p));
  return e;
}

template <int D, int kNH>
cudaError_t sparse_fmt(const SparseAttnParams& p, cudaStream_t s) {
  const bool k8 = p.q.a.fmt_k == 3, v8 = p.q.a.fmt_v == 3;
  if (!k8 && !v8) return sparse_launch<D, 1, 1, kNH>(p, s);
  if (k8 && !v8) return sparse_launch<D, 3, 1, kNH>(p, s);
  if (!k8 && v8) return sparse_launch<D, 1, 3, kNH>(p, s);
  return sparse_launch<D, 3, 3, kNH>(p, s);
}

template <int D>
cudaError_t sparse_dim(const SparseAttnParams& p, cudaStream_t s) {
  return p.q.a.group <= 8 ? sparse_fmt<D, 1>(p, s) : sparse_fmt<D, 2>(p, s);
}

// Splits of a list: as many as the resident blocks take at once, of 128 keys or more (4 x 8 lists of 512 keys:
// 7.9 us, of 256 keys or more 9.1; 16 x 8 lists of up to 1536 do as well with half as many, 19.7 against 21.9).
constexpr int kLeastKeys = 128;  // of a split
int64_t list_keys(int32_t topk, int32_t block_size) {
  return std::min(static_cast<int64_t>(topk) * block_size, int64_t{0x7FFF0000});
}
int64_t sparse_slots(int32_t D) { return (D == 256 ? 2ll : 4ll) * num_sms(); }
int sparse_splits(int32_t T, int32_t H, int32_t D, int32_t topk, int32_t block_size) {
  return fill_splits(static_cast<int64_t>(T) * H, sparse_slots(D), static_cast<int32_t>(list_keys(topk, block_size)), kLeastKeys,
                     2 * kLeastKeys);
}

// Not at head_dim 256 (27 lists of 64 16-token blocks in 2 splits: 24.7 us as clusters, 16.3 with the merge
// kernel).
bool use_cluster(int32_t D, int nsplit) { return nsplit > 1 && nsplit <= kClusterSplits && D <= 128; }

}  // namespace

size_t sparse_attn_workspace_bytes(int32_t T, int32_t H, int32_t Hq, int32_t D, int32_t block_size, int32_t topk) {
  if (T <= 0 || H <= 0 || Hq < H || D <= 0 || block_size <= 0 || topk <= 0) return 0;
  const int n = sparse_splits(T, H, D, topk, block_size);
  return n <= 1 || use_cluster(D, n) ? 0 : static_cast<size_t>(T) * Hq * n * (D + 2) * sizeof(float);
}

// Fewer tokens take more splits, so what a call needs does not grow with them.  Split lists fill at most two waves
// of the resident blocks (fill_splits), by at most as many splits as a list has room for: that grows with
// both, and is the same for every larger batch.
size_t sparse_attn_workspace_bound(int32_t T, int32_t H, int32_t Hq, int32_t D, int32_t block_size, int32_t topk) {
  if (T <= 0 || H <= 0 || Hq < H || D <= 0 || block_size <= 0 || topk <= 0) return 0;
  const int64_t most = std::min((list_keys(topk, block_size) + kLeastKeys - 1) / kLeastKeys, int64_t{256});
  if (most <= 1 || use_cluster(D, static_cast<int>(most))) return 0;
  const int64_t parts = std::min(static_cast<int64_t>(T) * H * most, 2 * sparse_slots(D));
  return static_cast<size_t>((parts * Hq + H - 1) / H) * (D + 2) * sizeof(float);
}

cudaError_t launch_sparse_attention(const SparseAttnParams& p_in, cudaStream_t s) {
  SparseAttnParams p = p_in;
  AttnParams& a = p.q.a;
  p.whole = a.block_size % 16 == 0;
  a.nsplit = sparse_splits(p.q.num_tokens, a.H, a.D, p.topk, a.block_size);
  p.cluster = use_cluster(a.D, a.nsplit);
  const cudaError_t e = a.D == 64 ? sparse_dim<64>(p, s) : a.D == 128 ? sparse_dim<128>(p, s) : sparse_dim<256>(p, s);
  return e == cudaSuccess && !p.cluster ? launch_query_merge_splits(p.q, s) : e;
}

}  // namespace kvq
