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

constexpr int kTreeMaxT = 64, kTreeMaxB = 4096;

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

// The tiles of all segments (sequence, unit, row group) in that order form one stream, which is cut into C
// equal shares. A segment costs its tiles and, for its queries, masks and epilogue, about kSegCost tiles
// more: positions 0 .. nt + cost - 1, tile 0 at position 0 and tile t > 0 at position cost + t. (Measured on
// 4 sequences of 511 to 32000 tokens, 64 drafts: without the cost, CTAs that got the short sequences ran 1.7
// times as long as the others.) The cost counts only if a share is longer than it, so that every CTA between
// the first and the last of a segment has a tile of it.
constexpr int kSegCost = 3, kSegCostFrom = 8;  // tiles; from this many tiles a CTA on

struct TreeStream {
  const int* pre;  // tiles of one row group of the sequences before b (shared memory, B + 1 entries)
  int B, HR;       // HR: row groups of a sequence
  int cost, total, per;  // positions of a segment beyond its tiles, of the stream, of a CTA
  __device__ TreeStream(const TreeGeo& g, const int* p) : pre(p), B(g.B), HR(g.Hkv * g.RG) {
    const int tiles = p[g.B] * HR;
    cost = tiles >= kSegCostFrom * g.C ? kSegCost : 0;
    total = tiles + g.B * HR * cost;
    per = (total + g.C - 1) / g.C;
  }
  __device__ int start(int b) const { return (pre[b] + b * cost) * HR; }
  // the segment that holds position x: sequence, row group, first position, tiles
  __device__ void find(int x, int* b, int* hr, int* first, int* tiles) const {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start(mid) <= x)
        lo = mid;
      else
        hi = mid;
    }
    const int nt = pre[lo + 1] - pre[lo], at = start(lo);
    *b = lo;
    *hr = (x - at) / (nt + cost);
    *first = at + *hr * (nt + cost);
    *tiles = nt;
  }
};

// A CTA's pieces of segments, in stream order.
struct TreePiece {
  int b, hk, rg, len;
  int t0, steps;  // first tile, tiles
  bool good;      // the sequence's length is in range
  bool whole;     // the CTA holds the whole segment
  int part;       // else: which of the CTA's two parts this is. 0 continues a segment, 1 begins one
  int next;       // position behind the segment
};

// the first piece with tiles at or behind position x of a CTA whose share ends at x1
__device__ __forceinline__ bool tree_piece(const TreeGeo& g, const TreeArgs& a, const TreeStream& ts, int x, int x1,
                                           TreePiece* p) {
  for (; x < x1; x = p->next) {
    int hr, first, tiles;
    ts.find(x, &p->b, &hr, &first, &tiles);
    p->next = first + tiles + ts.cost;
    p->t0 = x == first ? 0 : max(1, x - first - ts.cost);
    const int t1 = x1 >= p->next ? tiles : max(p->t0 == 0 ? 1 : p->t0, x1 - first - ts.cost);
    p->steps = t1 - p->t0;
    if (p->steps <= 0) continue;
    p->hk = hr / g.RG;
    p->rg = hr - p->hk * g.RG;
    p->whole = p->t0 == 0 && t1 == tiles;
    p->part = p->t0 == 0;
    p->good = tree_len(g, a, p->b, &p->len);
    if (!p->good) p->len = 0;
    return true;
  }
  return false;
}

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
