// Attention of drafted trees over a cache on the tcgen05 tensor cores: bf16 operands, fp32 accumulation and
// softmax statistics. Bound by reading the cache: a tile of 128 keys and values moves 64 KB (d = 128), about
// 2800 cycles of one SM's share of HBM, against 1024 or 2048 cycles of products.
//
// A persistent CTA walks its share of the stream of tiles (tree.cuh), one CTA per SM, with two slots that
// alternate on the tensor cores: while the softmax of one slot runs, the products of the other do.
//   SPLIT (up to 128 rows a unit): both slots hold the same rows and take the even and the odd tiles of the
//     segment, each with its own statistics and accumulator; they are merged at the segment's end.
//   else (two 128-row tiles): slot s holds row tile s, every K/V tile serves both.
//   warps 0-3, 4-7  softmax of slot 0 and 1, one thread a row     warp 8   TMA
//   warp 9          S = Q K^T     warp 10  O += P V               warp 11  the trees' masks
// A row tile holds the T rows of 128 / T heads, in the order of the TMA box that loads them.
// Measured (32/8 heads of 128), whole calls with the join: 32 sequences of 1 to 131056 tokens, 16 drafts: 1.02 ms,
// 6.8 TB/s in a burst, 1.23 ms over a second of calls, at the power cap; one token each: 0.98 and 1.18 ms. 4 sequences
// of 511 to 32000, 64 drafts: 92 us in a burst, 96 over a second (this kernel alone 72 us under a profiler). No unit
// is near its limit there: the two slots' softmax runs in step, 3600 to 3850 cycles against 2048 of products.
// Rows of V that no token sees (behind the drafts, absent slots) are zeroed in shared memory before P V: the
// cache may hold anything there, and 0 * NaN is NaN. Such rows of K only reach scores that are masked.
#include "tc_softmax.cuh"
#include "tree.cuh"

namespace pyr {

namespace {

using namespace tc;

constexpr int kThreads = 384;

template <int D, bool SPLIT>
struct TPlan {
  static constexpr int TB = 128 * D * 2;
  static constexpr int MT = SPLIT ? 1 : 2;
  static constexpr int NS = D == 64 ? 8 : SPLIT ? 5 : 4;
  static constexpr int kQ = 0;
  static constexpr int kRing = MT * TB;
  static constexpr int kMasks = kRing + NS * TB;  // [2]
  static constexpr int kPieces = kMasks + 2 * (int)sizeof(TreeMaskBuf);  // [2], with the masks
  static constexpr int kMl = kPieces + 2 * 64;  // [128][2] fp32: slot 1's maximum and sum
  static constexpr int kBar = kMl + 1024;
  static constexpr int kNumBars = 2 + 2 * NS + 2 + 4 + 2 + 2 + 4 + 2 + 2;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kSums = kMisc + 16;
  static constexpr int kPre = kSums + 128;
  static constexpr int kBytes = kPre + 1024;  // + 4 (B + 1)
};

// a piece, with what the issuing warps take from it in uniform registers
__device__ __forceinline__ bool piece_at(const TreeGeo& g, const TreeArgs& a, const TreeStream& ts, int x, int x1,
                                         TreePiece* p) {
  if (!uniform(tree_piece(g, a, ts, x, x1, p))) return false;
  p->b = uniform(p->b);
  p->hk = uniform(p->hk);
  p->rg = uniform(p->rg);
  p->len = uniform(p->len);
  p->t0 = uniform(p->t0);
  p->steps = uniform(p->steps);
  p->next = uniform(p->next);
  return true;
}

// bit c: key u0 + c, counted from the first drafted token, is visible to a row with this (non-zero) mask
__device__ __forceinline__ unsigned long long visible64(int u0, unsigned long long mask) {
  if (mask == 0 || u0 >= 64) return 0ull;
  if (u0 >= 0) return mask >> u0;
  if (u0 <= -64) return ~0ull;
  return (mask << -u0) | ((1ull << -u0) - 1);
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, TreeGeo g, TreeArgs a, int q_bytes) {
  using PL = TPlan<D, SPLIT>;
  constexpr int NS = PL::NS, TB = PL::TB, MT = PL::MT;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_align<1024>(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + PL::kBar);
  uint64_t* bar_q_full = bars;
  uint64_t* bar_q_free = bars + 1;
  uint64_t* bar_full = bars + 2;          // [NS]
  uint64_t* bar_free = bar_full + NS;     // [NS]
  uint64_t* bar_s_full = bar_free + NS;   // [2] slot
  uint64_t* bar_p_full = bar_s_full + 2;  // [2][2] slot, half
  uint64_t* bar_pv = bar_p_full + 4;      // [2]
  uint64_t* bar_o_free = bar_pv + 2;      // [2]
  uint64_t* bar_m_full = bar_o_free + 2;  // [2] masks of a segment
  uint64_t* bar_m_free = bar_m_full + 2;  // [2]
  uint64_t* bar_ml_full = bar_m_free + 2;
  uint64_t* bar_ml_free = bar_ml_full + 1;
  uint64_t* bar_drain = bar_ml_free + 1;  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + PL::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + PL::kMisc + 4);
  TreeMaskBuf* masks = reinterpret_cast<TreeMaskBuf*>(smem + PL::kMasks);
  TreePiece* pieces = reinterpret_cast<TreePiece*>(smem + PL::kPieces);
  float2* ml = reinterpret_cast<float2*>(smem + PL::kMl);
  int* pre = reinterpret_cast<int*>(smem + PL::kPre);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
    mbar_init(bar_q_full, 1);
    mbar_init(bar_q_free, 1);
    for (int s = 0; s < NS; s++) {
      mbar_init(bar_full + s, 1);
      mbar_init(bar_free + s, 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(bar_s_full + i, 1);
      mbar_init(bar_p_full + 2 * i, 4);
      mbar_init(bar_p_full + 2 * i + 1, 4);
      mbar_init(bar_pv + i, 1);
      mbar_init(bar_o_free + i, 4);
      mbar_init(bar_m_full + i, 1);
      mbar_init(bar_m_free + i, 9);  // softmax warps and the P V warp
      mbar_init(bar_drain + i, 1);
    }
    mbar_init(bar_ml_full, 4);
    mbar_init(bar_ml_free, 4);
    fence_mbar_init();
    *abort_flag = 0;
  }
  grid_launch();
  tree_prefix(g, a, pre, reinterpret_cast<int*>(smem + PL::kSums));
  const TreeStream ts(g, pre);
  const int x0 = blockIdx.x * ts.per, x1 = min(x0 + ts.per, ts.total);
  if (x0 >= x1) return;
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tO = tmem + 256;
  unsigned char* sQ = smem + PL::kQ;
  unsigned char* ring = smem + PL::kRing;
  TreePiece sg;

  if (warp == 8) {
    regs_dec<88>();
    // ------------------------------------------------------------ TMA producer
    bool ok = true;
    int u = 0, segs = 0;
    for (int x = x0; ok && piece_at(g, a, ts, x, x1, &sg); x = sg.next) {
      auto load = [&](const CUtensorMap* map, int t) {
        const int s = u % NS, k = u / NS;
        if (k > 0 && ok) ok = warp_wait(bar_free + s, (k - 1) & 1, abort_flag);
        if (!ok) return;
        if (elect_one()) {
          mbar_expect_tx(bar_full + s, TB);
          for (int h = 0; h < D / 64; h++)
            tma_load_4d(ring + s * TB + h * 16384, map, h * 64, t * 128, sg.hk, sg.b, bar_full + s);
        }
        u++;
      };
      // the first K tile may be in flight while the last S of the segment before still reads Q
      load(&tmK, sg.t0);
      if (ok && segs > 0) ok = warp_wait(bar_q_free, (segs - 1) & 1, abort_flag);
      if (!ok) break;
      if (elect_one()) {
        mbar_expect_tx(bar_q_full, MT * q_bytes);
        for (int mt = 0; mt < MT; mt++)
          for (int h = 0; h < D / 64; h++)
            tma_load_4d(sQ + mt * TB + h * 16384, &tmQ, h * 64, 0, sg.hk * g.G + (sg.rg * MT + mt) * g.HM, sg.b,
                        bar_q_full);
      }
      segs++;
      load(&tmV, sg.t0);
      for (int i = 1; i < sg.steps && ok; i++) {
        load(&tmK, sg.t0 + i);
        load(&tmV, sg.t0 + i);
      }
    }
    // drain: every copy issued must land (bounded) before the CTA may exit
    volatile int no_abort = 0;
    if (segs > 0) mbar_wait(bar_q_full, (segs - 1) & 1, &no_abort);
    for (int v = max(0, u - NS); v < u; v++) mbar_wait(bar_full + v % NS, (v / NS) & 1, &no_abort);
    __syncwarp();
  } else if (warp == 9) {
    regs_dec<88>();
    // ------------------------------------------------------------ S = Q K^T
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 0, 0);
    const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024), dK = sdesc_sw128(smem_u32(ring), 16, 1024);
    bool ok = true;
    int u = 0, segs = 0, ns[2] = {0, 0};
    for (int x = x0; ok && piece_at(g, a, ts, x, x1, &sg); x = sg.next, segs++) {
      for (int i = 0; i < sg.steps && ok; i++, u += 2) {
        const int s = u % NS;
        ok = warp_wait(bar_full + s, (u / NS) & 1, abort_flag);
        if (ok && i == 0) ok = warp_wait(bar_q_full, segs & 1, abort_flag);
        const uint64_t dKs = dK + (uint64_t)(s * (TB >> 4));
#pragma unroll
        for (int sl = 0; sl < 2; sl++) {
          if (!ok || (SPLIT && sl != (i & 1))) continue;
          if (ns[sl] > 0) ok = warp_wait(bar_pv + sl, (ns[sl] - 1) & 1, abort_flag);
          if (!ok) continue;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; kk++)
              umma_bf16(tS + sl * 128,
                        dQ + (uint64_t)(((SPLIT ? 0 : sl) * TB + (kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                        dKs + (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4), idesc, kk > 0);
            umma_commit(bar_s_full + sl);
          }
          __syncwarp();
          ns[sl]++;
        }
        if (ok && elect_one()) umma_commit(bar_free + s);
        __syncwarp();
      }
      if (ok && elect_one()) umma_commit(bar_q_free);
      __syncwarp();
    }
    drain(bar_drain);
  } else if (warp == 10) {
    regs_dec<88>();
    // ------------------------------------------------------------ O += P V
    constexpr uint32_t idesc = idesc_bf16_f32(128, D, 0, 1);
    const uint64_t dV = sdesc_sw128(smem_u32(ring), 16384, 1024);
    bool ok = true;
    int u = 1, segs = 0, np[2] = {0, 0}, no[2] = {0, 0};
    for (int x = x0; ok && piece_at(g, a, ts, x, x1, &sg); x = sg.next, segs++) {
      unsigned long long used = 0;
      ok = warp_wait(bar_m_full + (segs & 1), (segs >> 1) & 1, abort_flag);
      if (!ok) break;
      if ((sg.t0 + sg.steps) * 128 > sg.len) used = tree_used(masks + (segs & 1));
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_m_free + (segs & 1));
      for (int i = 0; i < sg.steps && ok; i++, u += 2) {
        const int s = u % NS;
        ok = warp_wait(bar_full + s, (u / NS) & 1, abort_flag);
        if (!ok) break;
        const int k0 = (sg.t0 + i) * 128;
        if (k0 + 128 > sg.len) {
          for (int r = lane; r < 128; r += 32) {
            const int v = k0 + r - sg.len;
            if (v < 0 || (v < g.T && ((used >> v) & 1))) continue;
#pragma unroll
            for (int c = 0; c < D / 8; c++)
              *reinterpret_cast<uint4*>(ring + s * TB + (c >> 3) * 16384 + r * 128 + (c & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        const uint64_t dVs = dV + (uint64_t)(s * (TB >> 4));
#pragma unroll
        for (int sl = 0; sl < 2; sl++) {
          if (!ok || (SPLIT && sl != (i & 1))) continue;
          const bool first = i == (SPLIT ? sl : 0);
          // O still holds the segment before until its epilogue has read it
          if (first && no[sl]++ > 0) ok = warp_wait(bar_o_free + sl, (no[sl] - 2) & 1, abort_flag);
          for (int half = 0; half < 2 && ok; half++) {
            ok = warp_wait(bar_p_full + 2 * sl + half, np[sl] & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; kk++)
                umma_bf16_ts(tO + sl * D, tS + sl * 128 + half * 32 + kk * 8,
                             dVs + (uint64_t)(((half * 4 + kk) * 2048) >> 4), idesc, !first || half > 0 || kk > 0);
              if (half) umma_commit(bar_pv + sl);
            }
            __syncwarp();
          }
          if (!ok) continue;
          np[sl]++;
        }
        if (ok && elect_one()) umma_commit(bar_free + s);
        __syncwarp();
      }
    }
    drain(bar_drain + 1);
  } else if (warp == 11) {
    regs_dec<88>();
    // ------------------------------------------------------------ masks
    // (and the pieces, so that the softmax warps need not hold more of them than they use)
    bool more = true;
    int segs = 0;
    for (int x = x0; more; x = sg.next, segs++) {
      more = piece_at(g, a, ts, x, x1, &sg);
      if (segs >= 2 && !warp_wait(bar_m_free + (segs & 1), ((segs >> 1) - 1) & 1, abort_flag)) break;
      if (more)
        tree_masks(g, a, sg.b, sg.good, masks + (segs & 1));
      else
        sg.steps = 0;
      if (lane == 0) pieces[segs & 1] = sg;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_m_full + (segs & 1));
    }
  } else {
    regs_inc<208>();  // 2 * 128 * 208 + 128 * 88 = 384 * 168
    // ------------------------------------------------------------ softmax
    const int sl = warp >> 2, wq = warp & 3;
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const uint32_t tS_row = tS + lane_base + sl * 128;
    const uint32_t tO_row = tO + lane_base + sl * D;
    const float sl2 = rsqrtf((float)D) * kLog2e;
    const int rt = wq * 32 + lane;  // row of the tile: token tok of the tile's head hl
    const int hl = rt / g.T, tok = rt - hl * g.T;
    bool ok = true;
    int n = 0, n1 = 0, segs = 0, twos = 0;  // so far: S tiles of this slot, of slot 1, segments, with two slots
    for (;; segs++) {
      ok = warp_wait(bar_m_full + (segs & 1), (segs >> 1) & 1, abort_flag);
      if (!ok) break;
      const TreePiece* pc = pieces + (segs & 1);
      const int steps = uniform(pc->steps);
      if (steps == 0) break;
      // head of the group this row belongs to
      const bool row_ok = hl < g.HM && (pc->rg * MT + (SPLIT ? 0 : sl)) * g.HM + hl < g.G;
      const unsigned long long mask = row_ok ? masks[segs & 1].mask[tok] : 0ull;
      const bool live = __any_sync(0xffffffffu, mask != 0);
      // first key of the next tile, counted from the first drafted token
      int v0 = ((pc->t0 + (SPLIT ? sl : 0)) * 128) - pc->len;
      float m_ref = -INFINITY, l_sum = 0.f;
      for (int i = SPLIT ? sl : 0; i < steps; i += SPLIT ? 2 : 1, n++, v0 += SPLIT ? 256 : 128) {
        ok = warp_wait(bar_s_full + sl, n & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (!live) {
          // what S left in place of P reaches rows that are not used
          if (lane == 0) {
            mbar_arrive(bar_p_full + 2 * sl);
            mbar_arrive(bar_p_full + 2 * sl + 1);
          }
          continue;
        }
        float s[128];
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_ld32(tS_row + c, s + c);
        tmem_wait_ld();
        if (v0 > -128) {
          const unsigned long long m0 = visible64(v0, mask), m1 = visible64(v0 + 64, mask);
#pragma unroll
          for (int c = 0; c < 64; c++) {
            s[c] = (m0 >> c) & 1 ? s[c] : -INFINITY;
            s[c + 64] = (m1 >> c) & 1 ? s[c + 64] : -INFINITY;
          }
        }
        const float mx = fmaxf(fmaxf(max32(s), max32(s + 32)), fmaxf(max32(s + 64), max32(s + 96)));
        const float m_new = fmaxf(m_ref, mx * sl2);
        const bool need = (m_ref != -INFINITY) && (m_new > m_ref + kRescale);
        float factor = 1.f;
        if (need) {
          factor = ex2(m_ref - m_new);
          l_sum *= factor;
          m_ref = m_new;
        } else if (m_ref == -INFINITY) {
          m_ref = m_new;
        }
        if (__any_sync(0xffffffffu, need)) {
          float o[32];
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            tmem_ld32(tO_row + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; k++) o[k] *= factor;
            tmem_st32(tO_row + c, o);
          }
        }
        const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
        const float2 scl = make_float2(sl2, sl2), off = make_float2(-m_use, -m_use);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int half = 0; half < 2; half++) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; c++) {
            const float2 y = __ffma2_rn(make_float2(s[half * 64 + 2 * c], s[half * 64 + 2 * c + 1]), scl, off);
            const float2 e = make_float2(ex2(y.x), ex2(y.y));
            acc[c & 3] = __fadd2_rn(acc[c & 3], e);
            pk[c] = pack_bf16(e.x, e.y);
          }
          tmem_st32u(tS_row + half * 32, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_p_full + 2 * sl + half);
        }
        const float2 s01 = __fadd2_rn(acc[0], acc[1]), s23 = __fadd2_rn(acc[2], acc[3]);
        const float2 sall = __fadd2_rn(s01, s23);
        l_sum += sall.x + sall.y;
      }
      if (!ok) break;
      // ---- the segment's end ----
      const bool seen = mask != 0;
      if (!seen) {
        m_ref = -INFINITY;
        l_sum = 0.f;
      }
      const bool two = SPLIT && steps > 1;  // slot 1 has part of the keys
      if (SPLIT && sl == 1) {
        if (lane == 0) mbar_arrive(bar_m_free + (segs & 1));
        if (!two) continue;
        if (twos > 0) ok = warp_wait(bar_ml_free, (twos - 1) & 1, abort_flag);
        if (!ok) break;
        ml[rt] = make_float2(m_ref, l_sum);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_ml_full);
        twos++;
        continue;
      }
      // the last P V of the slot (the one before it was done when the last S arrived)
      ok = warp_wait(bar_pv + sl, (n - 1) & 1, abort_flag);
      float w0 = 1.f, w1 = 0.f;
      if (two) {
        n1 += steps >> 1;
        if (ok) ok = warp_wait(bar_ml_full, twos & 1, abort_flag);
        if (ok) ok = warp_wait(bar_pv + 1, (n1 - 1) & 1, abort_flag);
        if (!ok) break;
        const float2 other = ml[rt];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_ml_free);
        twos++;
        const float m = fmaxf(m_ref, other.x), mu = m == -INFINITY ? 0.f : m;
        w0 = ex2(m_ref - mu);
        w1 = ex2(other.x - mu);
        m_ref = m;
        l_sum = l_sum * w0 + other.y * w1;
      }
      if (!ok) break;
      tc_fence_after();
      const int b = pc->b, hg = (pc->rg * MT + (SPLIT ? 0 : sl)) * g.HM + hl, head = pc->hk * g.G + hg;
      const bool whole = pc->whole;
      const int64_t part =
          (int64_t)(blockIdx.x * 2 + pc->part) * g.RR + (SPLIT ? 0 : sl) * 128 + rt;
      if (whole) {
        const float inv = l_sum != 0.f ? 1.f / l_sum : 0.f;  // 0: absent (a NaN score's sum is NaN)
        w0 *= inv;
        w1 *= inv;
      }
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        if (live) {
          tmem_ld32(tO_row + c, o);
          if (two) {
            float o1[32];
            tmem_ld32(tO_row + D + c, o1);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; k++) o[k] = fmaf(o1[k], w1, o[k] * w0);
          } else {
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; k++) o[k] *= w0;
          }
        }
#pragma unroll
        for (int k = 0; k < 32; k++) o[k] = seen ? o[k] : 0.f;
        if (row_ok && whole) {
          store32_bf16(view_at<__nv_bfloat16>(a.o, b, head, tok) + c, o, 1.f);
        } else if (row_ok) {
          float4* dst = reinterpret_cast<float4*>(a.part_o + part * D + c);
#pragma unroll
          for (int k = 0; k < 8; k++) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar_m_free + (segs & 1));
        mbar_arrive(bar_o_free + sl);
        if (two) mbar_arrive(bar_o_free + 1);
      }
      if (row_ok && whole) {
        if (a.lse)
          a.lse[((int64_t)b * g.Hq + head) * g.T + tok] =
              l_sum != 0.f ? (m_ref + log2f(l_sum)) * kLn2 : -INFINITY;
      } else if (row_ok) {
        *reinterpret_cast<float2*>(a.part_ml + 2 * part) = make_float2(m_ref, l_sum);
      }
    }
  }

  // ---- teardown ----
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) report(a.status, PYR_ETIMEOUT);
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool SPLIT>
cudaError_t launch(const TreeGeo& g, const TreeArgs& a, cudaStream_t st) {
  const int heads = g.HM < g.G ? g.HM : g.G;  // of a row tile
  CUtensorMap mq, mk, mv;
  if (!make_tmap_bf16_view(&mq, a.q.data, a.q.batch, a.q.head, a.q.row, D, g.T, g.Hq, g.B, g.T, heads) ||
      !make_tmap_bf16_view(&mk, a.k.data, a.k.batch, a.k.head, a.k.row, D, g.N, g.Hkv, g.B, 128) ||
      !make_tmap_bf16_view(&mv, a.v.data, a.v.batch, a.v.head, a.v.row, D, g.N, g.Hkv, g.B, 128))
    return cudaErrorInvalidValue;
  auto kern = tree_tc_kernel<D, SPLIT>;
  // the limit is the kernel's, not the call's: the same in every call, as two threads may be here at once
  constexpr int most = TPlan<D, SPLIT>::kBytes + 4 * (kTreeMaxB + 1);
  static_assert(most <= 227 * 1024, "shared memory of a CTA");
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  kern<<<g.C, kThreads, TPlan<D, SPLIT>::kBytes + 4 * (g.B + 1), st>>>(mq, mk, mv, g, a, heads * g.T * D * 2);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_tc(const TreeGeo& g, const TreeArgs& a, cudaStream_t st) {
  if (g.RR == 128) return g.d == 64 ? launch<64, true>(g, a, st) : launch<128, true>(g, a, st);
  return g.d == 64 ? launch<64, false>(g, a, st) : launch<128, false>(g, a, st);
}

}  // namespace pyr
