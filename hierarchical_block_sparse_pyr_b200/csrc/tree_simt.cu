// Attention of drafted trees over a cache on the CUDA cores, fp32 arithmetic: 32 or 64 rows x 64 keys a step.
// Every CTA walks its share of the stream of tiles (tree.cuh) and writes the rows of a segment itself where
// it holds the whole segment, else a part for the join.
#include "simt_tile.cuh"
#include "tree.cuh"

namespace pyr {

namespace {

using namespace simt;

template <int D, int ROWS>
constexpr int tree_smem() {
  return ((ROWS + kTile) * (D + 4) + kTile * D) * 4;
}

template <int D, int ROWS>
__global__ void __launch_bounds__(4 * ROWS) tree_simt_kernel(TreeGeo g, TreeArgs a) {
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm, *Ks = Qs + ROWS * (D + 4), *Vs = Ks + kTile * (D + 4), *Ps = Ks;
  int* pre = reinterpret_cast<int*>(Vs + kTile * D);
  __shared__ int warp_sums[32];
  __shared__ TreeMaskBuf masks;
  grid_launch();
  tree_prefix(g, a, pre, warp_sums);
  const TreeStream ts(g, pre);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const float sl2 = rsqrtf((float)D) * 1.4426950408889634f;
  const int x1 = min((blockIdx.x + 1) * ts.per, ts.total);
  TreePiece pc;
  for (int x = blockIdx.x * ts.per; tree_piece(g, a, ts, x, x1, &pc); x = pc.next) {
    const int b = pc.b, hk = pc.hk, len = pc.len, t0 = pc.t0, t1 = pc.t0 + pc.steps, r0 = pc.rg * g.RR;
    const bool good = pc.good;
    __syncthreads();
    if (threadIdx.x < 32) tree_masks(g, a, b, good, &masks);
    const int nr = min(ROWS, g.G * g.T - r0);
    for (int i = threadIdx.x; i < ROWS * (D / 4); i += 4 * ROWS) {
      const int r = i / (D / 4), c = 4 * (i - r * (D / 4)), ra = r0 + r;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nr) v = *reinterpret_cast<const float4*>(view_at<float>(a.q, b, hk * g.G + ra / g.T, ra % g.T) + c);
      *reinterpret_cast<float4*>(Qs + r * (D + 4) + c) = v;
    }
    __syncthreads();
    const unsigned long long used = tree_used(&masks);
    float m[4], l[4], acc[4][D / 16];
    unsigned long long mask[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      const int r = 4 * ty + i;
      mask[i] = r < nr ? masks.mask[(r0 + r) % g.T] : 0ull;
#pragma unroll
      for (int c = 0; c < D / 16; c++) acc[i][c] = 0.f;
    }
    for (int t = t0; t < t1; t++) {
      const int k0 = t * kTile;
      auto wanted = [&](int r) {
        const int u = k0 + r - len;
        return good && (u < 0 || (u < g.T && ((used >> u) & 1)));
      };
      __syncthreads();
      load_rows_if<4 * ROWS, D, kTile>(Ks, D + 4, view_at<float>(a.k, b, hk, k0), a.k.row, wanted);
      load_rows_if<4 * ROWS, D, kTile>(Vs, D, view_at<float>(a.v, b, hk, k0), a.v.row, wanted);
      __syncthreads();
      float s[4][4];
      mul_nt<4 * ROWS, D>(s, Qs, D + 4, Ks, D + 4);
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++)
          s[i][j] = tree_sees(k0 + tx + 16 * j, len, mask[i]) && good ? s[i][j] * sl2 : -INFINITY;
      softmax_step<D>(s, m, l, acc);
      __syncthreads();
      store_p<4 * ROWS>(Ps, s);
      __syncwarp();
      mul_acc<4 * ROWS, D>(acc, Ps, Vs, D);
    }
    const bool whole = pc.whole;
    const int64_t part = (int64_t)(blockIdx.x * 2 + pc.part) * g.RR;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int r = 4 * ty + i;
      if (r >= nr) continue;
      if (mask[i] == 0) {  // an absent slot: what it summed is not its own
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; c++) acc[i][c] = 0.f;
      }
      if (whole) {
        const int h = hk * g.G + (r0 + r) / g.T, t = (r0 + r) % g.T;
        store_row<D>(view_at<float>(a.o, b, h, t), acc[i], l[i] != 0.f ? 1.f / l[i] : 0.f);
        if (a.lse && tx == 0)
          a.lse[((int64_t)b * g.Hq + h) * g.T + t] =
              l[i] != 0.f ? (m[i] + log2f(l[i])) * 0.6931471805599453f : -INFINITY;
      } else {
        store_row<D>(a.part_o + (part + r) * D, acc[i], 1.f);
        if (tx == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * (part + r)) = make_float2(m[i], l[i]);
      }
    }
  }
}

template <int D, int ROWS>
cudaError_t launch(const TreeGeo& g, const TreeArgs& a, cudaStream_t st) {
  auto kern = tree_simt_kernel<D, ROWS>;
  // the limit is the kernel's, not the call's: the same in every call, as two threads may be here at once
  constexpr int most = tree_smem<D, ROWS>() + (kTreeMaxB + 1) * 4;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  kern<<<g.C, 4 * ROWS, tree_smem<D, ROWS>() + (g.B + 1) * 4, st>>>(g, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_simt(const TreeGeo& g, const TreeArgs& a, cudaStream_t st) {
  if (g.RR == 32) return g.d == 64 ? launch<64, 32>(g, a, st) : launch<128, 32>(g, a, st);
  return g.d == 64 ? launch<64, 64>(g, a, st) : launch<128, 64>(g, a, st);
}

}  // namespace pyr
