// Drafted trees over a cache: geometry, the split of the work over the GPU, the trees' masks.
#pragma once

#include "view.cuh"

namespace pyr {

// Rows of a unit (sequence, key/value head): drafted token t of the group's head h. They are cut into row
// groups of RR rows, and the keys into tiles of BK. On the CUDA cores (HM = 0) row r = h * T + t is row
// r % RR of group r / RR; on the tensor cores a group is RR / 128 tiles that hold the T rows of HM heads each.
struct TreeGeo {
  int B, Hq, Hkv, G, N, T, d, dtype;
  int HM;      // heads per 128-row tile, or 0
  int RR, RG;  // rows per row group, row groups per unit
  int BK;      // keys per tile
  int C;       // CTAs the tiles are split over
};

struct TreeArgs {
  View q, k, v, o;
  const int32_t* len;
  const int32_t* parent;
  float* lse;
  float* part_o;   // [C][2][RR][d] accumulators of the segments a CTA holds in part, against their maximum
  float* part_ml;  // [C][2][RR][2] their row maximum (log2 units) and sum
  int* status;
};

constexpr int kTreeMaxT = 64;

// head of the group and token of row rr of row group rg; false: the row holds nothing
__device__ __forceinline__ bool tree_row(const TreeGeo& g, int rg, int rr, int* h, int* t) {
  if (g.HM) {
    const int w = rr & 127, hl = w / g.T;
    *h = (rg * (g.RR >> 7) + (rr >> 7)) * g.HM + hl;
    *t = w - hl * g.T;
    return hl < g.HM && *h < g.G;
  }
  const int r = rg * g.RR + rr;
  *h = r / g.T;
  *t = r - *h * g.T;
  return *h < g.G;
}

// keys of sequence b, tile count; a sequence with a bad length has one tile without keys, so that some
// CTA writes its outputs
__device__ __forceinline__ bool tree_len(const TreeGeo& g, const TreeArgs& a, int b, int* len) {
  *len = __ldg(a.len + b);
  return *len >= 0 && *len <= g.N - g.T;
}
__device__ __forceinline__ int tree_tiles(const TreeGeo& g, const TreeArgs& a, int b) {
  int n;
  return tree_len(g, a, b, &n) ? (n + g.T + g.BK - 1) / g.BK : 1;
}

// The tiles of all (sequence, unit, row group) in that order form one stream; CTA c < C takes the positions
// [cut(c), cut(c + 1)), at least one, whatever segments they fall in. pre[b] = tiles of one row group of
// the sequences before b (in shared memory, B + 1 entries).
struct TreeStream {
  const int* pre;
  int B, HR;  // HR: row groups of a sequence
  int64_t total;
  int C;
  __device__ TreeStream(const TreeGeo& g, const int* p)
      : pre(p), B(g.B), HR(g.Hkv * g.RG), total((int64_t)p[g.B] * g.Hkv * g.RG), C(total < g.C ? (int)total : g.C) {}
  __device__ int64_t cut(int c) const { return total / C * c + total % C * c / C; }
  // the segment that holds position x: sequence, unit and row group, first position, tiles
  __device__ void find(int64_t x, int* b, int* hr, int64_t* first, int* tiles) const {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)pre[mid] * HR <= x)
        lo = mid;
      else
        hi = mid;
    }
    const int nt = pre[lo + 1] - pre[lo];
    const int64_t at = (int64_t)pre[lo] * HR;
    *b = lo;
    *hr = (int)((x - at) / nt);
    *first = at + (int64_t)*hr * nt;
    *tiles = nt;
  }
};

// pre[0 .. B] by the whole block (blockDim.x a multiple of 32, at most 1024); warp_sums: 32 ints
__device__ __forceinline__ void tree_prefix(const TreeGeo& g, const TreeArgs& a, int* pre, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int carry = 0;
  for (int base = 0; base < g.B; base += blockDim.x) {
    const int b = base + threadIdx.x;
    int x = b < g.B ? tree_tiles(g, a, b) : 0;
    const int own = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += u;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = carry, all = carry;
    for (int w = 0; w < nw; w++) {
      if (w < warp) before += warp_sums[w];
      all += warp_sums[w];
    }
    if (b < g.B) pre[b] = before + x - own;
    carry = all;
    __syncthreads();
  }
  if (threadIdx.x == 0) pre[g.B] = carry;
  __syncthreads();
}

// masks[t] = the drafted tokens that token t sees (itself and its ancestors), 0 if the slot is absent, by
// one warp. Pointer jumping: after k rounds a token has the 2^k nearest of its path.
// buf: 2 * 64 uint64 and 64 ints of scratch in shared memory.
struct TreeMaskBuf {
  unsigned long long mask[kTreeMaxT];
  int ptr[kTreeMaxT];  // next ancestor not yet merged; -1: none; -2: the path holds an absent slot
};

__device__ __forceinline__ void tree_masks(const TreeGeo& g, const TreeArgs& a, int b, bool ok, TreeMaskBuf* s) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int t = lane + 32 * i;
    int p = PYR_TREE_ABSENT;
    if (t < g.T && ok) {
      p = a.parent ? a.parent[(int64_t)b * g.T + t] : t - 1;
      if (p < PYR_TREE_ABSENT || p >= t) {
        report(a.status, PYR_EBADSEQ);
        p = PYR_TREE_ABSENT;
      }
    }
    s->mask[t] = p == PYR_TREE_ABSENT ? 0ull : 1ull << t;
    s->ptr[t] = p;
  }
  if (!ok && lane == 0) report(a.status, PYR_EBADSEQ);
  __syncwarp();
  for (int k = 0; k < 6; k++) {
    unsigned long long m[2];
    int p[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int t = lane + 32 * i;
      m[i] = s->mask[t];
      p[i] = s->ptr[t];
      if (p[i] >= 0) {
        m[i] |= s->mask[p[i]];
        p[i] = s->ptr[p[i]];
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; i++) {
      s->mask[lane + 32 * i] = m[i];
      s->ptr[lane + 32 * i] = p[i];
    }
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < 2; i++)
    if (s->ptr[lane + 32 * i] == PYR_TREE_ABSENT) s->mask[lane + 32 * i] = 0ull;
  __syncwarp();
}

// of the drafted tokens, those that some token sees: the others' cache rows may hold anything
__device__ __forceinline__ unsigned long long tree_used(const TreeMaskBuf* s) {
  unsigned long long m = 0;
  for (int t = 0; t < kTreeMaxT; t++) m |= s->mask[t];
  return m;
}

__device__ __forceinline__ bool tree_sees(int key, int len, unsigned long long mask) {
  return mask != 0 && (key < len || (key - len < kTreeMaxT && ((mask >> (key - len)) & 1)));
}

cudaError_t launch_tree_tc(const TreeGeo& g, const TreeArgs& a, cudaStream_t st);
cudaError_t launch_tree_simt(const TreeGeo& g, const TreeArgs& a, cudaStream_t st);
// joins the parts of every segment that more than one CTA worked on
cudaError_t launch_tree_join(const TreeGeo& g, const TreeArgs& a, cudaStream_t st);

}  // namespace pyr
