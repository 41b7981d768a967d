// Causal attention of packed prompts on the tcgen05 tensor cores: bf16 operands, fp32 accumulation and
// softmax statistics, P rounded to bf16 for the second product.
//
// A persistent CTA works on two 128-row tiles at a time that share every K/V tile: the same 128 rows of two
// heads of a group (G even: no tile of the pair crosses the diagonal later than the other), or 256 rows of
// one head. Keys come in tiles of 128 counted from the sequence's start, so the diagonal tile is square.
//   warps 0-3, 4-7   softmax of row tile 0 and 1, one thread a row
//   warp 8           TMA: Q of both tiles, then K and V tiles through one ring
//   warp 9           issues S = Q K^T   (M = 128, N = 128)
//   warp 10          issues O += P V    (P from tensor memory), in two halves of 64 keys
//   warp 11          idle (it completes the warpgroup that gives up registers)
// Tensor memory: S of each tile 128 columns (P overwrites the first 64 as bf16), O of each tile D columns.
// A tile has one S buffer; the two tiles alternate: while the softmax of one runs, the tensor cores serve
// the other. S(t + 1) of a tile is issued after P V(t) of that tile is done, so when the softmax sees
// S(t + 1), O is at rest and may be rescaled without a wait.
// A row sees 128 scores: the maximum comes first over all of them (so that the first half's P V may start
// while the second half's exponentials run), O is rescaled only if the maximum grew by more than 2^8.
// Measured (heads of 128): 24001 + 6000 + 2500 + 267 tokens, 16 heads: 1.95 ms in a burst, 1300 TFLOP/s, 78 % of
// the measured peak; 2.3 ms over a second of calls, at the power cap. 8192 tokens: 211 us, tensor pipe 67 % busy,
// about 2990 cycles a step of which 2048 are the products'.
// Rows of V behind the sequence's end belong to others and may hold anything (0 * NaN is NaN): the P V
// warp zeroes them in shared memory. Rows of K there only reach scores that the causal mask drops, rows of
// Q only outputs that are not stored.
#include "packed.cuh"
#include "tc_softmax.cuh"

namespace pyr {

namespace {

using namespace tc;

// of 32 pairs of exponentials, on the FMA pipe. Kernel time against it is rugged at d = 128 (32K tokens, 16 heads,
// timed for a second: none 2.53 ms, the last 10 2.33, 11 2.45, 12 2.26, 14 2.49, 12 spread evenly 2.31; 8K tokens, in a
// burst: none 262 us, 8 248, 12 233, 14 262). At d = 64 (8K tokens): none 225 us, 8 203, 12 211, 14 217
constexpr int kFma = 12;

template <int D>
struct FPlan {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int NS = D == 128 ? 5 : 8;  // K/V ring stages
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kBar = kRing + NS * kTileBytes;
  static constexpr int kNumBars = 2 + 2 + 2 * NS + 2 + 4 + 2 + 2 + 2 + 8;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kBytes = kMisc + 16 + 1024;
  static constexpr int kThreads = 384;
};

// one unit of work of a CTA: what the two row tiles are and how many key tiles each walks
struct FItem {
  int start, end, row0, hk;
  int head[2], row[2], n[2];  // row: first row of the tile; n: key tiles (0: no row of the sequence in it)
  int steps;
};

__device__ __forceinline__ bool fwd_item(const PackedGeo& g, const int32_t* plan, int tiles, int64_t at, FItem* it) {
  const bool pair = g.G % 2 == 0;
  const int units = pair ? g.Hq / 2 : g.Hq;
  const int64_t tile = at / units;
  if (tile >= tiles) return false;
  const int u = (int)(at - tile * units);
  int4 w = __ldg(reinterpret_cast<const int4*>(plan + packed_list_at(g, kListFwd)) + tile);
  w.x = it->start = uniform(w.x);
  w.y = it->end = uniform(w.y);
  w.z = it->row0 = uniform(w.z);
#pragma unroll
  for (int mt = 0; mt < 2; mt++) {
    it->head[mt] = pair ? 2 * u + mt : u;
    it->row[mt] = pair ? w.z : w.z + 128 * mt;
    it->n[mt] = it->row[mt] < w.y ? (it->row[mt] - w.x) / 128 + 1 : 0;
  }
  it->hk = it->head[0] / g.G;
  it->steps = max(it->n[0], it->n[1]);
  return true;
}

template <int D>
__global__ void __launch_bounds__(FPlan<D>::kThreads, 1)
    packed_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, PackedGeo g, PackedFwdArgs a) {
  using PL = FPlan<D>;
  constexpr int NS = PL::NS, TB = PL::kTileBytes;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_align<1024>(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + PL::kBar);
  uint64_t* bar_q_full = bars;               // [2]
  uint64_t* bar_q_free = bars + 2;           // [2]
  uint64_t* bar_full = bars + 4;             // [NS]
  uint64_t* bar_free = bar_full + NS;        // [NS]
  uint64_t* bar_s_full = bar_free + NS;      // [2]
  uint64_t* bar_p_full = bar_s_full + 2;     // [2][2]: tile, half
  uint64_t* bar_pv = bar_p_full + 4;         // [2] P V(t) of the tile done: S is free, O at rest
  uint64_t* bar_o_free = bar_pv + 2;         // [2] the epilogue has read O
  uint64_t* bar_drain = bar_o_free + 2;      // [2]
  uint64_t* bar_turn = bar_drain + 2;        // [2][4] exponentials of a tile done, by row tile and scheduler
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + PL::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + PL::kMisc + 4);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
    for (int i = 0; i < 2; i++) {
      mbar_init(bar_q_full + i, 1);
      mbar_init(bar_q_free + i, 1);
      mbar_init(bar_s_full + i, 1);
      mbar_init(bar_p_full + 2 * i, 4);
      mbar_init(bar_p_full + 2 * i + 1, 4);
      mbar_init(bar_pv + i, 1);
      mbar_init(bar_o_free + i, 4);
      mbar_init(bar_drain + i, 1);
      for (int w = 0; w < 4; w++) mbar_init(bar_turn + 4 * i + w, 1);
    }
    for (int s = 0; s < NS; s++) {
      mbar_init(bar_full + s, 1);
      mbar_init(bar_free + s, 1);
    }
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tO = tmem + 256;  // S[mt] at mt * 128, O[mt] at 256 + mt * D
  unsigned char* sQ = smem + PL::kQ;
  unsigned char* ring = smem + PL::kRing;

  FItem it;
  const int tiles = uniform(packed_tiles(g, a.plan, kListFwd, a.status));
  // a softmax thread holds a row of 128 scores; the other warpgroup needs few registers
  // (2 * 128 * 208 + 128 * 88 = 384 * 168)
  if (warp == 8) {
    regs_dec<88>();
    // ------------------------------------------------------------ TMA producer
    bool ok = true;
    int u = 0;  // ring uses so far
    int nq[2] = {0, 0};
    for (int r = 0; ok && fwd_item(g, a.plan, tiles, list_at(r), &it); r++) {
      auto load = [&](const CUtensorMap* map, int row) {
        const int s = u % NS, k = u / NS;
        if (k > 0 && ok) ok = warp_wait(bar_free + s, (k - 1) & 1, abort_flag);
        if (!ok) return;
        if (elect_one()) {
          mbar_expect_tx(bar_full + s, TB);
          for (int h = 0; h < D / 64; h++)
            tma_load_4d(ring + s * TB + h * 16384, map, h * 64, row, it.hk, 0, bar_full + s);
        }
        u++;
      };
      // the first K tile may be in flight while the last S of the previous item still reads Q
      load(&tmK, it.start);
#pragma unroll
      for (int mt = 0; mt < 2; mt++) {
        if (!it.n[mt]) continue;
        if (nq[mt] > 0 && ok) ok = warp_wait(bar_q_free + mt, (nq[mt] - 1) & 1, abort_flag);
        if (!ok) continue;
        if (elect_one()) {
          mbar_expect_tx(bar_q_full + mt, TB);
          for (int h = 0; h < D / 64; h++)
            tma_load_4d(sQ + mt * TB + h * 16384, &tmQ, h * 64, it.row[mt], it.head[mt], 0, bar_q_full + mt);
        }
        nq[mt]++;
      }
      load(&tmV, it.start);
      for (int t = 1; t < it.steps && ok; t++) {
        load(&tmK, it.start + t * 128);
        load(&tmV, it.start + t * 128);
      }
    }
    // drain: every copy issued must land (bounded) before the CTA may exit
    volatile int no_abort = 0;
    for (int i = 0; i < 2; i++)
      if (nq[i] > 0) mbar_wait(bar_q_full + i, (nq[i] - 1) & 1, &no_abort);
    for (int v = max(0, u - NS); v < u; v++) mbar_wait(bar_full + v % NS, (v / NS) & 1, &no_abort);
    __syncwarp();
  } else if (warp == 9) {
    regs_dec<88>();
    // ------------------------------------------------------------ S = Q K^T
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 0, 0);
    const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024), dK = sdesc_sw128(smem_u32(ring), 16, 1024);
    bool ok = true;
    int u = 0, nq[2] = {0, 0}, ns[2] = {0, 0};
    for (int r = 0; ok && fwd_item(g, a.plan, tiles, list_at(r), &it); r++) {
      for (int t = 0; t < it.steps; t++, u += 2) {
        const int s = u % NS;
        ok = warp_wait(bar_full + s, (u / NS) & 1, abort_flag);
        if (!ok) break;
        const uint64_t dKs = dK + (uint64_t)(s * (TB >> 4));
#pragma unroll
        for (int mt = 0; mt < 2; mt++) {
          if (!ok || t >= it.n[mt]) continue;
          if (t == 0) ok = warp_wait(bar_q_full + mt, nq[mt]++ & 1, abort_flag);
          if (ok && ns[mt] > 0) ok = warp_wait(bar_pv + mt, (ns[mt] - 1) & 1, abort_flag);
          if (!ok) continue;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; kk++)
              umma_bf16(tS + mt * 128, dQ + (uint64_t)((mt * TB + (kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                        dKs + (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4), idesc, kk > 0);
            umma_commit(bar_s_full + mt);
            if (t == it.n[mt] - 1) umma_commit(bar_q_free + mt);
          }
          __syncwarp();
          ns[mt]++;
        }
        if (ok && elect_one()) umma_commit(bar_free + s);
        __syncwarp();
        if (!ok) break;
      }
    }
    drain(bar_drain);
  } else if (warp == 10) {
    regs_dec<88>();
    // ------------------------------------------------------------ O += P V
    constexpr uint32_t idesc = idesc_bf16_f32(128, D, 0, 1);
    const uint64_t dV = sdesc_sw128(smem_u32(ring), 16384, 1024);
    bool ok = true;
    int u = 1, np[2] = {0, 0}, no[2] = {0, 0};
    for (int r = 0; ok && fwd_item(g, a.plan, tiles, list_at(r), &it); r++) {
      for (int t = 0; t < it.steps && ok; t++, u += 2) {
        const int s = u % NS;
        ok = warp_wait(bar_full + s, (u / NS) & 1, abort_flag);
        if (!ok) break;
        const int valid = it.end - (it.start + t * 128);
        if (valid < 128) {
          for (int x = lane; x < (128 - valid) * 8; x += 32)
#pragma unroll
            for (int h = 0; h < D / 64; h++)
              *reinterpret_cast<uint4*>(ring + s * TB + h * 16384 + valid * 128 + x * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        const uint64_t dVs = dV + (uint64_t)(s * (TB >> 4));
#pragma unroll
        for (int mt = 0; mt < 2; mt++) {
          if (!ok || t >= it.n[mt]) continue;
          // O still holds the previous item's result until its epilogue has read it
          if (t == 0 && no[mt]++ > 0) ok = warp_wait(bar_o_free + mt, (no[mt] - 2) & 1, abort_flag);
          for (int half = 0; half < 2 && ok; half++) {
            ok = warp_wait(bar_p_full + 2 * mt + half, np[mt] & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; kk++)
                umma_bf16_ts(tO + mt * D, tS + mt * 128 + half * 32 + kk * 8,
                             dVs + (uint64_t)(((half * 4 + kk) * 2048) >> 4), idesc, t > 0 || half > 0 || kk > 0);
              if (half) umma_commit(bar_pv + mt);
            }
            __syncwarp();
          }
          if (!ok) continue;
          np[mt]++;
        }
        if (ok && elect_one()) umma_commit(bar_free + s);
        __syncwarp();
      }
    }
    drain(bar_drain + 1);
  } else if (warp == 11) {
    regs_dec<88>();
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<208>();  // 2 * 128 * 208 + 128 * 88 = 384 * 168
    const int mt = warp >> 2, wq = warp & 3;
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const uint32_t tS_row = tS + lane_base + mt * 128;
    const uint32_t tO_row = tO + lane_base + mt * D;
    const float sl2 = rsqrtf((float)D) * kLog2e;
    bool ok = true;
    int n = 0, turns = 0;  // so far: tiles of S, turns of the other row tile waited for
    for (int r = 0; ok && fwd_item(g, a.plan, tiles, list_at(r), &it); r++) {
      const int steps = mt ? it.n[1] : it.n[0], row_mt = mt ? it.row[1] : it.row[0];
      const int head = mt ? it.head[1] : it.head[0];
      if (!steps) continue;
      const int others = mt ? it.n[0] : it.n[1];  // key tiles of the other row tile
      const int row = row_mt + wq * 32 + lane;
      const bool live = row_mt + wq * 32 < it.end;  // some row of the warp is in the sequence
      float m_ref = -INFINITY, l_sum = 0.f;
      for (int t = 0; t < steps; t++, n++) {
        ok = warp_wait(bar_s_full + mt, n & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        // the turns go tile 0, tile 1 for every key tile that both have. At d = 64 the exponentials take longer
        // than the products and turns gain 10 % (8K tokens, 16 heads: 241 -> 217 us); at d = 128 they cost 5 %
        const bool take = D == 64 && (mt ? t < others : t > 0 && t - 1 < others);
        const bool give = D == 64 && (mt ? t + 1 < others : t < others);
        if (!live) {
          // P stays what S left there: it reaches rows that nobody stores
          turns += take;
          if (lane == 0) {
            if (give) mbar_arrive(bar_turn + 4 * mt + wq);
            mbar_arrive(bar_p_full + 2 * mt);
            mbar_arrive(bar_p_full + 2 * mt + 1);
          }
          continue;
        }
        const int lim = row - (it.start + t * 128) + 1;  // keys this row may see
        const bool masked = t == steps - 1;
        float s[128];
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_ld32(tS_row + c, s + c);
        tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int c = 0; c < 128; c++) s[c] = c < lim ? s[c] : -INFINITY;
        }
        // a NaN score makes the row's maximum, and with it all that follows, NaN
        const float mx = max_nan(max_nan(max32(s), max32(s + 32)), max_nan(max32(s + 64), max32(s + 96)));
        const float m_new = max_nan(m_ref, mx * sl2);
        const bool need = (m_ref != -INFINITY) && !(m_new <= m_ref + kRescale);
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
        if (take) turn_wait(bar_turn + 4 * (1 - mt) + wq, turns++ & 1);
        const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
        const float2 scl = make_float2(sl2, sl2), off = make_float2(-m_use, -m_use);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int half = 0; half < 2; half++) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; c++) {
            const float2 x = __ffma2_rn(make_float2(s[half * 64 + 2 * c], s[half * 64 + 2 * c + 1]), scl, off);
            const float2 e = exp2_mix<32, kFma, 4, false>(c, x);
            acc[c & 3] = __fadd2_rn(acc[c & 3], e);
            pk[c] = pack_bf16(e.x, e.y);
          }
          if (half && give && lane == 0) mbar_arrive(bar_turn + 4 * mt + wq);
          tmem_st32u(tS_row + half * 32, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_p_full + 2 * mt + half);
        }
        const float2 s01 = __fadd2_rn(acc[0], acc[1]), s23 = __fadd2_rn(acc[2], acc[3]);
        const float2 sall = __fadd2_rn(s01, s23);
        l_sum += sall.x + sall.y;
      }
      if (!ok) break;
      // ---- epilogue: the last P V (the one before it was done when the last S arrived) ----
      ok = warp_wait(bar_pv + mt, (n - 1) & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const bool store = row < it.end;
      const float inv = 1.f / l_sum;
      __nv_bfloat16* dst = view_at<__nv_bfloat16>(a.o, 0, head, row);
      if (live) {
        float o[32];
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          tmem_ld32(tO_row + c, o);
          tmem_wait_ld();
          if (store) store32_bf16(dst + c, o, inv);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_o_free + mt);
      if (store && a.lse) a.lse[(int64_t)head * g.T + row] = (m_ref + log2f(l_sum)) * kLn2;
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

template <int D>
cudaError_t launch_d(const PackedGeo& g, const PackedFwdArgs& a, cudaStream_t st) {
  CUtensorMap mq, mk, mv;
  if (!make_tmap_bf16_view(&mq, a.q.data, a.q.batch, a.q.head, a.q.row, D, g.T, g.Hq, 1, 128) ||
      !make_tmap_bf16_view(&mk, a.k.data, a.k.batch, a.k.head, a.k.row, D, g.T, g.Hkv, 1, 128) ||
      !make_tmap_bf16_view(&mv, a.v.data, a.v.batch, a.v.head, a.v.row, D, g.T, g.Hkv, 1, 128))
    return cudaErrorInvalidValue;
  auto kern = packed_fwd_tc_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, FPlan<D>::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t items = packed_list_cap(g, kListFwd) * (g.G % 2 ? g.Hq : g.Hq / 2);
  kern<<<(unsigned)(items < 148 ? items : 148), FPlan<D>::kThreads, FPlan<D>::kBytes, st>>>(mq, mk, mv, g, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_fwd_tc(const PackedGeo& g, const PackedFwdArgs& a, cudaStream_t st) {
  return g.d == 64 ? launch_d<64>(g, a, st) : launch_d<128>(g, a, st);
}

}  // namespace pyr
