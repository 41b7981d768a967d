// Gradients of packed-prompt attention on the tcgen05 tensor cores: bf16 operands, fp32 accumulation; P and
// dS are rounded to bf16 for the products that read them. Two kernels, so that every gradient is summed by
// one CTA in a fixed order (no atomics): S and dP are computed twice, and P K besides, 8 products of 128 x 128 x D
// where a single pass with atomic sums of dQ would need 5, or 6 with P K.
//
// dK/dV: a CTA owns 128 keys of a key/value head and walks the 128-row query tiles from its own to the
//   sequence's end, over the heads of the group:
//     S^T = K Q^T, dP^T = V dO^T           (rows = keys: P^T and dS^T come out as A operands in tensor memory)
//     P^T = 2^(S^T c - lse2), dS^T = P^T (dP^T - delta)
//     dV += P^T dO, dK += dS^T Q
//   Tensor memory is full: S^T 128 columns, dP^T 128, dV D, dK D; P^T and dS^T overwrite their sources as
//   bf16. While the softmax works on P^T(t), the tensor cores run dP^T(t) and dK(t - 1).
// dQ: a CTA owns 128 queries of a head and walks the key tiles up to the diagonal:
//     S = Q K^T, dP = dO V^T, dS = P (dP - delta), dQ += dS K, PK += P K
//   Tensor memory is full: S (P goes over it as bf16) 128 columns, dP (dS goes over it) 128, dQ D, PK D.
// Both: persistent CTAs over the plan's lists (longest first, back and forth over the CTAs).
//   warps 0-15  softmax: warpgroup w takes the columns 32 w .. 32 w + 31 of every row; its bf16 results go to
//               columns 32 w .. 32 w + 15 of the buffer, so that no warpgroup touches another's columns. Four
//               warps a scheduler: with two, the waits and tensor-memory loads of a step were not covered
//   warp 16     TMA      warp 17  products      warp 19  lse, delta and tails (dK/dV only)
// delta = dO . O comes from the rounded O and is off by about 2^-9 |(dO_i O_i)_i|. The rounding of dS is small
// against |dP - delta|, that error only against |O|, and the two have nothing to do with each other: values with a
// component in common, peaked scores or few keys in a row make the error the larger one (values and keys with a
// common component of 4 and 2 times their spread: dQ 13 % off). The dQ kernel has all of a row's P and dP, and
//   rest = sum_k P (dP - delta)   makes   delta + rest = sum_k P dP   up to the rounding of the differences alone,
// so it subtracts rest PK from dQ, and writes delta + rest back for the dK/dV kernel, which therefore runs second.
// The rows of a sequence's first tile see one key tile: they get delta + rest before dS is formed, which leaves
// exactly 0 where a row sees one key. (8192 tokens, 16 heads, all of the gradients: without PK and rest 748 us, with
// them 823.)
// Measured (8192 tokens, 16 heads of 128): 2840 cycles a step in both kernels, tensor pipe 72 % busy, 0.4 ms each.
// dK/dV has shared memory close behind (256 KB a step, 2048 cycles), dQ the softmax warps' chain of loads,
// exponentials and stores. 32K tokens: 7.3 ms in a burst, 8.5 ms over a second, at the power cap.
// Rows behind the sequence's end may hold anything. As rows of A they only reach outputs that are not
// stored; where they are summed over (B of dK, dV and dQ) they are zeroed in shared memory.
#include "packed.cuh"
#include "tc_softmax.cuh"

namespace pyr {

namespace {

using namespace tc;

constexpr int kSoftmax = 16;                    // softmax warps
constexpr int kThreads = (kSoftmax + 4) * 32;
// of 16 pairs of exponentials, on the FMA pipe (dK/dV kernel: none 3 % slower; dQ kernel: none 8 % slower, 4 pairs 1 %)
constexpr int kFma = 6;

// zero the rows valid .. 127 of a 128-row operand tile (64-element halves of 128 rows x 128 bytes); one warp
template <int D>
__device__ __forceinline__ void zero_tail(unsigned char* tile, int valid) {
  const int lane = threadIdx.x & 31;
  for (int x = lane; x < (128 - valid) * 8; x += 32)
#pragma unroll
    for (int h = 0; h < D / 64; h++)
      *reinterpret_cast<uint4*>(tile + h * 16384 + valid * 128 + x * 16) = make_uint4(0, 0, 0, 0);
}

template <int D>
__device__ __forceinline__ void load_tile(unsigned char* dst, const CUtensorMap* map, int row, int head, uint64_t* bar) {
  mbar_expect_tx(bar, 128 * D * 2);
#pragma unroll
  for (int h = 0; h < D / 64; h++) tma_load_4d(dst + h * 16384, map, h * 64, row, head, 0, bar);
}

// D[tmem] = A B^T over D elements, both operands 128-row tiles in shared memory
template <int D>
__device__ __forceinline__ void mma_nt(uint32_t d, uint64_t da, uint64_t db) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 0, 0);
#pragma unroll
  for (int kk = 0; kk < D / 16; kk++) {
    const uint64_t o = (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
    umma_bf16(d, da + o, db + o, idesc, kk > 0);
  }
}

// D[tmem] (+)= A B over the rows 16 K0 .. 16 (K0 + NK) - 1 of B: A bf16 in tensor memory, its elements 32 w ..
// 32 w + 31 of a row at a + 32 w; B a 128-row tile in shared memory
template <int D, int K0, int NK>
__device__ __forceinline__ void mma_acc(uint32_t d, uint32_t a, uint64_t db, bool add) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, D, 0, 1);
#pragma unroll
  for (int kk = K0; kk < K0 + NK; kk++)
    umma_bf16_ts(d, a + (kk >> 1) * 32 + (kk & 1) * 8, db + (uint64_t)((kk * 2048) >> 4), idesc, add || kk > K0);
}

// N columns of a row of an fp32 accumulator in tensor memory, times f, to memory
template <int N>
__device__ __forceinline__ void store_acc(uint32_t t, __nv_bfloat16* dst, float f, bool store) {
#pragma unroll 1
  for (int c = 0; c < N; c += 32) {
    float o[32];
    tmem_ld32(t + c, o);
    tmem_wait_ld();
    if (store) store32_bf16(dst + c, o, f);
  }
}

// ---------------------------------------------------------------------------------------------- dK, dV

template <int D>
struct KPlan {
  static constexpr int TB = 128 * D * 2;
  static constexpr int NS = 2;  // stages of the Q and of the dO ring
  static constexpr int kK = 0, kV = TB, kQ = 2 * TB, kG = kQ + NS * TB;
  static constexpr int kStat = kG + NS * TB;  // [NS][2][128] fp32: -lse2, -delta
  static constexpr int kBar = kStat + NS * 1024;
  static constexpr int kNumBars = 2 + 6 * NS + 9;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kBytes = kMisc + 16 + 1024;
};

struct KItem {
  int end, key0, hk, nq, steps;
};

__device__ __forceinline__ bool k_item(const PackedGeo& g, const int32_t* plan, int tiles, int64_t at, KItem* it) {
  const int64_t tile = at / g.Hkv;
  if (tile >= tiles) return false;
  const int4 w = __ldg(reinterpret_cast<const int4*>(plan + packed_list_at(g, kListK)) + tile);
  it->hk = (int)(at - tile * g.Hkv);
  it->end = uniform(w.y);
  it->key0 = uniform(w.z);
  it->nq = (it->end - it->key0 + 127) / 128;
  it->steps = it->nq * g.G;
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dkdv_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
                          PackedGeo g, PackedBwdArgs a) {
  using PL = KPlan<D>;
  constexpr int NS = PL::NS, TB = PL::TB;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_align<1024>(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + PL::kBar);
  uint64_t* bar_kv_full = bars;            // K and V of the item
  uint64_t* bar_kv_free = bars + 1;
  uint64_t* bar_q_full = bars + 2;         // [NS]
  uint64_t* bar_q_free = bar_q_full + NS;  // [NS]
  uint64_t* bar_g_full = bar_q_free + NS;  // [NS] dO
  uint64_t* bar_g_free = bar_g_full + NS;  // [NS]
  uint64_t* bar_st_full = bar_g_free + NS;   // [NS] lse and delta there, tails zeroed
  uint64_t* bar_st_free = bar_st_full + NS;  // [NS]
  uint64_t* bar_s_full = bar_st_free + NS;
  uint64_t* bar_p_full = bar_s_full + 1;    // [2] half of the columns
  uint64_t* bar_dp_full = bar_p_full + 2;
  uint64_t* bar_ds_full = bar_dp_full + 1;  // [2] half of the columns
  uint64_t* bar_acc_full = bar_ds_full + 2;
  uint64_t* bar_acc_free = bar_acc_full + 1;
  uint64_t* bar_drain = bar_acc_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + PL::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + PL::kMisc + 4);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
    tma_prefetch_map(&tmG);
    mbar_init(bar_kv_full, 1);
    mbar_init(bar_kv_free, 1);
    for (int s = 0; s < NS; s++) {
      mbar_init(bar_q_full + s, 1);
      mbar_init(bar_q_free + s, 1);
      mbar_init(bar_g_full + s, 1);
      mbar_init(bar_g_free + s, 1);
      mbar_init(bar_st_full + s, 1);
      mbar_init(bar_st_free + s, kSoftmax);
    }
    mbar_init(bar_s_full, 1);
    mbar_init(bar_dp_full, 1);
    for (int c = 0; c < 2; c++) {
      mbar_init(bar_p_full + c, kSoftmax / 2);
      mbar_init(bar_ds_full + c, kSoftmax / 2);
    }
    mbar_init(bar_acc_full, 1);
    mbar_init(bar_acc_free, kSoftmax);
    mbar_init(bar_drain, 1);
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == kSoftmax + 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tP = tmem + 128, tDV = tmem + 256, tDK = tmem + 256 + D;
  const uint64_t dK = sdesc_sw128(smem_u32(smem + PL::kK), 16, 1024), dV = sdesc_sw128(smem_u32(smem + PL::kV), 16, 1024);
  KItem it;
  const int tiles = uniform(packed_tiles(g, a.plan, kListK, a.status));

  if (warp == kSoftmax + 0) {
    regs_dec<64>();
    // ------------------------------------------------------------ TMA producer
    bool ok = true;
    int items = 0, u = 0;
    for (int r = 0; ok && k_item(g, a.plan, tiles, list_at(r), &it); r++, items++) {
      if (items > 0) ok = warp_wait(bar_kv_free, (items - 1) & 1, abort_flag);
      if (!ok) break;
      if (elect_one()) {
        mbar_expect_tx(bar_kv_full, 2 * TB);
        for (int h = 0; h < D / 64; h++) {
          tma_load_4d(smem + PL::kK + h * 16384, &tmK, h * 64, it.key0, it.hk, 0, bar_kv_full);
          tma_load_4d(smem + PL::kV + h * 16384, &tmV, h * 64, it.key0, it.hk, 0, bar_kv_full);
        }
      }
      int head = it.hk * g.G, j = 0;
      for (int i = 0; i < it.steps; i++, u++) {
        const int s = u % NS, k = u / NS, q0 = it.key0 + j * 128;
        if (k > 0) ok = warp_wait(bar_q_free + s, (k - 1) & 1, abort_flag);
        if (ok && k > 0) ok = warp_wait(bar_g_free + s, (k - 1) & 1, abort_flag);
        if (!ok) break;
        if (elect_one()) {
          load_tile<D>(smem + PL::kQ + s * TB, &tmQ, q0, head, bar_q_full + s);
          load_tile<D>(smem + PL::kG + s * TB, &tmG, q0, head, bar_g_full + s);
        }
        if (++j == it.nq) j = 0, head++;
      }
    }
    // drain: every copy issued must land (bounded) before the CTA may exit
    volatile int no_abort = 0;
    for (int v = max(0, u - NS); v < u; v++) {
      mbar_wait(bar_q_full + v % NS, (v / NS) & 1, &no_abort);
      mbar_wait(bar_g_full + v % NS, (v / NS) & 1, &no_abort);
    }
    if (items > 0) mbar_wait(bar_kv_full, (items - 1) & 1, &no_abort);
    __syncwarp();
  } else if (warp == kSoftmax + 1) {
    regs_dec<64>();
    // ------------------------------------------------------------ all products, in the order that keeps
    // S(i + 1) ahead of dK(i): the softmax waits for S, and dK(i) and dP(i + 1) fill its time
    const uint64_t dQ = sdesc_sw128(smem_u32(smem + PL::kQ), 16, 1024), dG = sdesc_sw128(smem_u32(smem + PL::kG), 16, 1024);
    const uint64_t dQm = sdesc_sw128(smem_u32(smem + PL::kQ), 16384, 1024);
    const uint64_t dGm = sdesc_sw128(smem_u32(smem + PL::kG), 16384, 1024);
    bool ok = true;
    int items = 0, u = 0;
    for (int r = 0; ok && k_item(g, a.plan, tiles, list_at(r), &it); r++, items++) {
      int j = 0;  // query tile that the next S reads
      auto scores = [&](int v) {
        const int s = v % NS;
        ok = warp_wait(bar_q_full + s, (v / NS) & 1, abort_flag);
        if (ok && it.key0 + j * 128 + 128 > it.end) ok = warp_wait(bar_st_full + s, (v / NS) & 1, abort_flag);
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
          mma_nt<D>(tS, dK, dQ + (uint64_t)(s * (TB >> 4)));
          umma_commit(bar_s_full);
        }
        __syncwarp();
        if (++j == it.nq) j = 0;
      };
      auto dprob = [&](int v) {
        const int s = v % NS;
        ok = warp_wait(bar_g_full + s, (v / NS) & 1, abort_flag);  // (a tail's zeroing: waited for above)
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
          mma_nt<D>(tP, dV, dG + (uint64_t)(s * (TB >> 4)));
          umma_commit(bar_dp_full);
        }
        __syncwarp();
      };
      ok = warp_wait(bar_kv_full, items & 1, abort_flag);
      if (ok) scores(u);
      if (ok) dprob(u);
      for (int i = 0; i < it.steps && ok; i++, u++) {
        const int s = u % NS;
        const uint64_t at = (uint64_t)(s * (TB >> 4));
        if (i == 0 && items > 0) ok = warp_wait(bar_acc_free, (items - 1) & 1, abort_flag);
#pragma unroll
        for (int c = 0; c < 2; c++) {
          if (ok) ok = warp_wait(bar_p_full + c, u & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            if (c == 0)
              mma_acc<D, 0, 4>(tDV, tS, dGm + at, i > 0);
            else
              mma_acc<D, 4, 4>(tDV, tS, dGm + at, true);
            if (c == 1) umma_commit(bar_g_free + s);
          }
          __syncwarp();
        }
        // over P^T(i): products of one thread run in the order of issue
        if (ok && i + 1 < it.steps) scores(u + 1);
#pragma unroll
        for (int c = 0; c < 2; c++) {
          if (ok) ok = warp_wait(bar_ds_full + c, u & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            if (c == 0)
              mma_acc<D, 0, 4>(tDK, tP, dQm + at, i > 0);
            else
              mma_acc<D, 4, 4>(tDK, tP, dQm + at, true);
            if (c == 1) umma_commit(bar_q_free + s);
          }
          __syncwarp();
        }
        if (ok && i + 1 < it.steps) dprob(u + 1);
      }
      if (ok && elect_one()) {
        umma_commit(bar_kv_free);
        umma_commit(bar_acc_full);
      }
      __syncwarp();
    }
    drain(bar_drain);
  } else if (warp == kSoftmax + 2) {
    regs_dec<64>();
  } else if (warp == kSoftmax + 3) {
    regs_dec<64>();
    // ------------------------------------------------------------ lse, delta, tails
    bool ok = true;
    int u = 0;
    for (int r = 0; ok && k_item(g, a.plan, tiles, list_at(r), &it); r++) {
      for (int i = 0; i < it.steps; i++, u++) {
        const int s = u % NS, k = u / NS, head = it.hk * g.G + i / it.nq, q0 = it.key0 + i % it.nq * 128;
        if (k > 0) ok = warp_wait(bar_st_free + s, (k - 1) & 1, abort_flag);
        if (!ok) break;
        float* st = reinterpret_cast<float*>(smem + PL::kStat + s * 1024);
        const int64_t at = (int64_t)head * g.T;
#pragma unroll
        for (int c = lane; c < 128; c += 32) {
          const int q = q0 + c;
          st[c] = q < it.end ? -kLog2e * a.lse[at + q] : -INFINITY;
          st[128 + c] = q < it.end ? -a.delta[at + q] : 0.f;
        }
        if (q0 + 128 > it.end) {
          ok = warp_wait(bar_q_full + s, k & 1, abort_flag);
          if (ok) ok = warp_wait(bar_g_full + s, k & 1, abort_flag);
          if (!ok) break;
          zero_tail<D>(smem + PL::kQ + s * TB, it.end - q0);
          zero_tail<D>(smem + PL::kG + s * TB, it.end - q0);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_st_full + s);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<104>();  // 512 * 104 + 128 * 64 = 640 * 96
    const int wg = warp >> 2, wq = warp & 3, half = wg >> 1;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16, base = lanes + wg * 32;
    const float scale = rsqrtf((float)D), sl2 = scale * kLog2e;
    const float2 scl = make_float2(sl2, sl2);
    const int rr = wq * 32 + lane;
    bool ok = true;
    int items = 0, u = 0;
    for (int r = 0; ok && k_item(g, a.plan, tiles, list_at(r), &it); r++, items++) {
      const bool live = it.key0 + wq * 32 < it.end;
      int j = 0;
      for (int i = 0; i < it.steps; i++, u++) {
        const int st_i = u % NS;
        const float4* st = reinterpret_cast<const float4*>(smem + PL::kStat + st_i * 1024) + wg * 8;
        const bool diag = j == 0;
        if (++j == it.nq) j = 0;
        ok = warp_wait(bar_s_full, u & 1, abort_flag);
        if (ok) ok = warp_wait(bar_st_full + st_i, (u / NS) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        float p[32];
        if (live) {
          uint32_t pk[16];
          tmem_ld32(tS + base, p);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float4 nl = st[e / 2];
            const int o = 2 * e;
            const float2 x = exp2_mix<16, kFma, 3, true>(e, __ffma2_rn(make_float2(p[o], p[o + 1]), scl, make_float2(nl.x, nl.y)));
            const float2 y =
                exp2_mix<16, kFma, 3, true>(e + 1, __ffma2_rn(make_float2(p[o + 2], p[o + 3]), scl, make_float2(nl.z, nl.w)));
            p[o] = x.x, p[o + 1] = x.y, p[o + 2] = y.x, p[o + 3] = y.y;
          }
          if (diag) {
#pragma unroll
            for (int e = 0; e < 32; e++) p[e] = wg * 32 + e >= rr ? p[e] : 0.f;
          }
#pragma unroll
          for (int e = 0; e < 16; e++) pk[e] = pack_bf16(p[2 * e], p[2 * e + 1]);
          tmem_st16u(tS + base, pk);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p_full + half);
        ok = warp_wait(bar_dp_full, u & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (live) {
          float d[32];
          uint32_t pk[16];
          tmem_ld32(tP + base, d);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float4 nd = st[32 + e / 2];  // -delta
            const int o = 2 * e;
            const float2 x = __fmul2_rn(make_float2(p[o], p[o + 1]),
                                        __fadd2_rn(make_float2(d[o], d[o + 1]), make_float2(nd.x, nd.y)));
            const float2 y = __fmul2_rn(make_float2(p[o + 2], p[o + 3]),
                                        __fadd2_rn(make_float2(d[o + 2], d[o + 3]), make_float2(nd.z, nd.w)));
            pk[e] = pack_bf16(x.x, x.y);
            pk[e + 1] = pack_bf16(y.x, y.y);
          }
          tmem_st16u(tP + base, pk);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar_ds_full + half);
          mbar_arrive(bar_st_free + st_i);
        }
      }
      if (!ok) break;
      // ---- epilogue: two warpgroups store dV, two dK, half of the columns each ----
      ok = warp_wait(bar_acc_full, items & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const int key = it.key0 + rr, c0 = (wg & 1) * (D / 2);
      if (live)
        store_acc<D / 2>((half ? tDK : tDV) + lanes + c0,
                         view_at<__nv_bfloat16>(half ? a.dk : a.dv, 0, it.hk, key) + c0, half ? scale : 1.f,
                         key < it.end);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_acc_free);
    }
  }

  // ---- teardown ----
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) report(a.status, PYR_ETIMEOUT);
  if (warp == kSoftmax + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// -------------------------------------------------------------------------------------------------- dQ

template <int D>
struct QPlan {
  static constexpr int TB = 128 * D * 2;
  static constexpr int NK = 3, NV = 2;  // K stages (a K tile lives until dQ has read it), V stages
  static constexpr int kQ = 0, kG = TB, kK = 2 * TB, kV = kK + NK * TB;
  static constexpr int kSum = kV + NV * TB;  // [2][128] fp32: row sums on their way through the warpgroups
  static constexpr int kBar = kSum + 1024;
  static constexpr int kNumBars = 2 + 2 * NK + 2 * NV + 2 + 2 + 2 + 1 + 16;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kBytes = kMisc + 16 + 1024;
};

struct QItem {
  int start, end, row0, head, hk, steps;
};

__device__ __forceinline__ bool q_item(const PackedGeo& g, const int32_t* plan, int tiles, int64_t at, QItem* it) {
  const int64_t tile = at / g.Hq;
  if (tile >= tiles) return false;
  const int4 w = __ldg(reinterpret_cast<const int4*>(plan + packed_list_at(g, kListQ)) + tile);
  it->head = (int)(at - tile * g.Hq);
  it->hk = it->head / g.G;
  it->start = uniform(w.x);
  it->end = uniform(w.y);
  it->row0 = uniform(w.z);
  it->steps = (it->row0 - it->start) / 128 + 1;
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dq_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG, PackedGeo g,
                        PackedBwdArgs a) {
  using PL = QPlan<D>;
  constexpr int NK = PL::NK, NV = PL::NV, TB = PL::TB;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_align<1024>(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + PL::kBar);
  uint64_t* bar_q_full = bars;      // Q and dO of the item
  uint64_t* bar_q_free = bars + 1;  // its last S and dP have read them
  uint64_t* bar_k_full = bars + 2;
  uint64_t* bar_k_free = bar_k_full + NK;
  uint64_t* bar_v_full = bar_k_free + NK;
  uint64_t* bar_v_free = bar_v_full + NV;
  uint64_t* bar_s_full = bar_v_free + NV;
  uint64_t* bar_p_full = bar_s_full + 1;    // P stands where S was
  uint64_t* bar_dp_full = bar_p_full + 1;
  uint64_t* bar_ds_full = bar_dp_full + 1;  // dS stands where dP was
  uint64_t* bar_acc_full = bar_ds_full + 1;
  uint64_t* bar_acc_free = bar_acc_full + 1;
  uint64_t* bar_drain = bar_acc_free + 1;
  uint64_t* bar_sum = bar_drain + 1;  // [4][4] rows, warpgroup: has added its part
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + PL::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + PL::kMisc + 4);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
    tma_prefetch_map(&tmG);
    mbar_init(bar_q_full, 1);
    mbar_init(bar_q_free, 1);
    for (int s = 0; s < NK; s++) {
      mbar_init(bar_k_full + s, 1);
      mbar_init(bar_k_free + s, 1);
    }
    for (int s = 0; s < NV; s++) {
      mbar_init(bar_v_full + s, 1);
      mbar_init(bar_v_free + s, 1);
    }
    mbar_init(bar_s_full, 1);
    mbar_init(bar_p_full, kSoftmax);
    mbar_init(bar_dp_full, 1);
    mbar_init(bar_ds_full, kSoftmax);
    mbar_init(bar_acc_full, 1);
    mbar_init(bar_acc_free, kSoftmax);
    mbar_init(bar_drain, 1);
    for (int i = 0; i < 16; i++) mbar_init(bar_sum + i, 1);
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == kSoftmax + 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tP = tmem + 128, tDQ = tmem + 256, tPK = tmem + 256 + D;
  QItem it;
  const int tiles = uniform(packed_tiles(g, a.plan, kListQ, a.status));

  if (warp == kSoftmax + 0) {
    regs_dec<64>();
    // ------------------------------------------------------------ TMA producer
    bool ok = true;
    int items = 0, u = 0;
    for (int r = 0; ok && q_item(g, a.plan, tiles, list_at(r), &it); r++, items++) {
      if (items > 0) ok = warp_wait(bar_q_free, (items - 1) & 1, abort_flag);
      if (!ok) break;
      if (elect_one()) {
        mbar_expect_tx(bar_q_full, 2 * TB);
        for (int h = 0; h < D / 64; h++) {
          tma_load_4d(smem + PL::kQ + h * 16384, &tmQ, h * 64, it.row0, it.head, 0, bar_q_full);
          tma_load_4d(smem + PL::kG + h * 16384, &tmG, h * 64, it.row0, it.head, 0, bar_q_full);
        }
      }
      for (int i = 0; i < it.steps; i++, u++) {
        const int sk = u % NK, kk = u / NK, sv = u % NV, kv = u / NV;
        if (kk > 0) ok = warp_wait(bar_k_free + sk, (kk - 1) & 1, abort_flag);
        if (ok && kv > 0) ok = warp_wait(bar_v_free + sv, (kv - 1) & 1, abort_flag);
        if (!ok) break;
        if (elect_one()) {
          load_tile<D>(smem + PL::kK + sk * TB, &tmK, it.start + i * 128, it.hk, bar_k_full + sk);
          load_tile<D>(smem + PL::kV + sv * TB, &tmV, it.start + i * 128, it.hk, bar_v_full + sv);
        }
      }
    }
    volatile int no_abort = 0;
    for (int v = max(0, u - NK); v < u; v++) mbar_wait(bar_k_full + v % NK, (v / NK) & 1, &no_abort);
    for (int v = max(0, u - NV); v < u; v++) mbar_wait(bar_v_full + v % NV, (v / NV) & 1, &no_abort);
    if (items > 0) mbar_wait(bar_q_full, (items - 1) & 1, &no_abort);
    __syncwarp();
  } else if (warp == kSoftmax + 1) {
    regs_dec<64>();
    // ------------------------------------------------------------ all products: P K(u) and S(u + 1) while the
    // softmax works on dS(u), dQ(u) and dP(u + 1) while it works on P(u + 1). S(u + 1) goes over P(u) and dP(u + 1)
    // over dS(u) behind the products that read them, as products of one thread run in the order of issue. At an
    // item's end S(u + 1) comes behind dQ(u), which would otherwise wait for the next item's Q.
    const uint64_t dQ = sdesc_sw128(smem_u32(smem + PL::kQ), 16, 1024), dG = sdesc_sw128(smem_u32(smem + PL::kG), 16, 1024);
    const uint64_t dK = sdesc_sw128(smem_u32(smem + PL::kK), 16, 1024), dV = sdesc_sw128(smem_u32(smem + PL::kV), 16, 1024);
    const uint64_t dKm = sdesc_sw128(smem_u32(smem + PL::kK), 16384, 1024);
    bool ok = true, last = false;
    int us = 0, si = 0, sr = 0, sitems = 0;  // next S: step, step of its item, its item in the list and here
    QItem is;
    bool more = q_item(g, a.plan, tiles, list_at(0), &is);
    auto scores = [&]() {
      if (!more || !ok) return;
      const int s = us % NK;
      if (si == 0) ok = warp_wait(bar_q_full, sitems & 1, abort_flag);
      if (ok) ok = warp_wait(bar_k_full + s, (us / NK) & 1, abort_flag);
      if (!ok) return;
      const int valid = is.end - (is.start + si * 128);
      if (valid < 128) {
        // dQ sums over the rows of K
        zero_tail<D>(smem + PL::kK + s * TB, valid);
        fence_proxy_async_smem();
        __syncwarp();
      }
      tc_fence_after();
      if (elect_one()) {
        mma_nt<D>(tS, dQ, dK + (uint64_t)(s * (TB >> 4)));
        umma_commit(bar_s_full);
      }
      __syncwarp();
      us++;
      last = ++si == is.steps;
      if (last) {
        si = 0;
        sitems++;
        more = q_item(g, a.plan, tiles, list_at(++sr), &is);
      }
    };
    auto dprob = [&](int v) {  // of the step whose S was the last to be issued
      if (!ok || us <= v) return;
      const int s = v % NV;
      ok = warp_wait(bar_v_full + s, (v / NV) & 1, abort_flag);
      if (!ok) return;
      tc_fence_after();
      if (elect_one()) {
        mma_nt<D>(tP, dG, dV + (uint64_t)(s * (TB >> 4)));
        umma_commit(bar_dp_full);
        umma_commit(bar_v_free + s);
        if (last) umma_commit(bar_q_free);
      }
      __syncwarp();
    };
    scores();
    dprob(0);
    int items = 0, u = 0;
    for (int r = 0; ok && q_item(g, a.plan, tiles, list_at(r), &it); r++, items++) {
      for (int i = 0; i < it.steps && ok; i++, u++) {
        const int s = u % NK;
        const uint64_t at = (uint64_t)(s * (TB >> 4));
        ok = warp_wait(bar_p_full, u & 1, abort_flag);
        if (ok && i == 0 && items > 0) ok = warp_wait(bar_acc_free, (items - 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (it.steps > 1) {
          if (elect_one()) mma_acc<D, 0, 8>(tPK, tS, dKm + at, i > 0);
          __syncwarp();
        }
        if (i + 1 < it.steps) scores();
        if (ok) ok = warp_wait(bar_ds_full, u & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          mma_acc<D, 0, 8>(tDQ, tP, dKm + at, i > 0);
          umma_commit(bar_k_free + s);
          if (i == it.steps - 1) umma_commit(bar_acc_full);
        }
        __syncwarp();
        if (i + 1 == it.steps) scores();
        dprob(u + 1);
      }
    }
    drain(bar_drain);
  } else if (warp >= kSoftmax + 2) {
    regs_dec<64>();
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<104>();  // 512 * 104 + 128 * 64 = 640 * 96
    const int wg = warp >> 2, wq = warp & 3;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16, base = lanes + wg * 32;
    const float scale = rsqrtf((float)D), sl2 = scale * kLog2e;
    const int rr = wq * 32 + lane;
    bool ok = true;
    int items = 0, u = 0, sums = 0;  // sums: rounds of the row sums so far
    // A row's sum over its four warpgroups' parts, added in their order. Two buffers: a warpgroup that is a round
    // ahead writes into the other one, and cannot be two ahead, as every round waits for all four.
    auto row_sum = [&](float part) {
      volatile float* sum = reinterpret_cast<volatile float*>(smem + PL::kSum) + (sums & 1) * 128 + rr;
      if (wg > 0) {
        ok = warp_wait(bar_sum + 4 * wq + wg - 1, sums & 1, abort_flag);
        part += *sum;
      }
      *sum = part;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_sum + 4 * wq + wg);
      if (ok) ok = warp_wait(bar_sum + 4 * wq + 3, sums & 1, abort_flag);
      sums++;
      return *sum;
    };
    for (int r = 0; ok && q_item(g, a.plan, tiles, list_at(r), &it); r++, items++) {
      const int row = it.row0 + rr;
      const bool live = it.row0 + wq * 32 < it.end;
      const int64_t at = (int64_t)it.head * g.T + min(row, it.end - 1);
      const float nl = -kLog2e * a.lse[at], nd = -a.delta[at];
      const float2 scl = make_float2(sl2, sl2), off = make_float2(nl, nl);
      float2 del = make_float2(nd, nd), rest = make_float2(0.f, 0.f);
      for (int i = 0; i < it.steps; i++, u++) {
        const bool diag = i == it.steps - 1;
        ok = warp_wait(bar_s_full, u & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        float p[32];
        if (live) {
          uint32_t pk[16];
          tmem_ld32(tS + base, p);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; c++) {
            const float2 x = exp2_mix<16, kFma, 3, true>(c, __ffma2_rn(make_float2(p[2 * c], p[2 * c + 1]), scl, off));
            p[2 * c] = x.x, p[2 * c + 1] = x.y;
          }
          if (diag) {
#pragma unroll
            for (int c = 0; c < 32; c++) p[c] = wg * 32 + c <= rr ? p[c] : 0.f;
          }
#pragma unroll
          for (int c = 0; c < 16; c++) pk[c] = pack_bf16(p[2 * c], p[2 * c + 1]);
          tmem_st16u(tS + base, pk);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p_full);
        ok = warp_wait(bar_dp_full, u & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (live) {
          float d[32];
          uint32_t pk[16];
          tmem_ld32(tP + base, d);
          tmem_wait_ld();
          if (diag) {
            // columns behind the row may hold another sequence's values
#pragma unroll
            for (int c = 0; c < 32; c++) d[c] = wg * 32 + c <= rr ? d[c] : 0.f;
          }
          if (it.steps == 1) {  // all that the row sees
            float part = 0.f;
#pragma unroll
            for (int c = 0; c < 32; c++) part = fmaf(p[c], d[c] + nd, part);
            const float refined = -nd + row_sum(part);
            del = make_float2(-refined, -refined);
            if (wg == 0 && row < it.end) a.delta[at] = refined;
          }
#pragma unroll
          for (int c = 0; c < 16; c++) {
            const float2 x =
                __fmul2_rn(make_float2(p[2 * c], p[2 * c + 1]), __fadd2_rn(make_float2(d[2 * c], d[2 * c + 1]), del));
            rest = __fadd2_rn(rest, x);
            pk[c] = pack_bf16(x.x, x.y);
          }
          tmem_st16u(tP + base, pk);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (!ok) break;
        if (lane == 0) mbar_arrive(bar_ds_full);
      }
      if (!ok) break;
      // ---- epilogue: 32 columns a warpgroup ----
      float c = 0.f;
      if (live && it.steps > 1) {
        c = row_sum(rest.x + rest.y);
        if (wg == 0 && row < it.end) a.delta[at] = -nd + c;  // for the dK/dV kernel
        if (!ok) break;
      }
      ok = warp_wait(bar_acc_full, items & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      if (live && wg * 32 < D) {
        float o[32];
        tmem_ld32(tDQ + base, o);
        if (it.steps > 1) {
          float k[32];
          tmem_ld32(tPK + base, k);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e++) o[e] = fmaf(-c, k[e], o[e]);
        } else {
          tmem_wait_ld();
        }
        if (row < it.end) store32_bf16(view_at<__nv_bfloat16>(a.dq, 0, it.head, row) + wg * 32, o, scale);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_acc_free);
    }
  }

  // ---- teardown ----
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) report(a.status, PYR_ETIMEOUT);
  if (warp == kSoftmax + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_d(const PackedGeo& g, const PackedBwdArgs& a, cudaStream_t st) {
  CUtensorMap mq, mk, mv, mg;
  if (!make_tmap_bf16_view(&mq, a.q.data, a.q.batch, a.q.head, a.q.row, D, g.T, g.Hq, 1, 128) ||
      !make_tmap_bf16_view(&mk, a.k.data, a.k.batch, a.k.head, a.k.row, D, g.T, g.Hkv, 1, 128) ||
      !make_tmap_bf16_view(&mv, a.v.data, a.v.batch, a.v.head, a.v.row, D, g.T, g.Hkv, 1, 128) ||
      !make_tmap_bf16_view(&mg, a.dout.data, a.dout.batch, a.dout.head, a.dout.row, D, g.T, g.Hq, 1, 128))
    return cudaErrorInvalidValue;
  auto kq = packed_dq_tc_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, QPlan<D>::kBytes);
  if (e != cudaSuccess) return e;
  int64_t items = packed_list_cap(g, kListQ) * g.Hq;
  kq<<<(unsigned)(items < 148 ? items : 148), kThreads, QPlan<D>::kBytes, st>>>(mq, mk, mv, mg, g, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  auto kk = packed_dkdv_tc_kernel<D>;
  e = cudaFuncSetAttribute(kk, cudaFuncAttributeMaxDynamicSharedMemorySize, KPlan<D>::kBytes);
  if (e != cudaSuccess) return e;
  items = packed_list_cap(g, kListK) * g.Hkv;
  kk<<<(unsigned)(items < 148 ? items : 148), kThreads, KPlan<D>::kBytes, st>>>(mq, mk, mv, mg, g, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_bwd_tc(const PackedGeo& g, const PackedBwdArgs& a, cudaStream_t st) {
  return g.d == 64 ? launch_d<64>(g, a, st) : launch_d<128>(g, a, st);
}

}  // namespace pyr
