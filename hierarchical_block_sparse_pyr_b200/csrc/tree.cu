// Drafted trees over a cache: the C entry point and the kernel that joins the parts.
#include "tree.cuh"

namespace pyr {

namespace {

constexpr int kJoinWarps = 8;

template <int E>
struct Part;  // the E = D / 32 elements of a row that a lane owns
template <>
struct Part<2> {
  float x[2];
  __device__ __forceinline__ void load(const float* p) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x, x[1] = v.y;
  }
  __device__ __forceinline__ void store(float* p, float f) const {
    *reinterpret_cast<float2*>(p) = make_float2(x[0] * f, x[1] * f);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, float f) const {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x[0] * f, x[1] * f);
  }
};
template <>
struct Part<4> {
  float x[4];
  __device__ __forceinline__ void load(const float* p) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  }
  __device__ __forceinline__ void store(float* p, float f) const {
    *reinterpret_cast<float4*>(p) = make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, float f) const {
    const __nv_bfloat162 u = __floats2bfloat162_rn(x[0] * f, x[1] * f), v = __floats2bfloat162_rn(x[2] * f, x[3] * f);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
  }
};

// One warp a row: O = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over the parts of the row's segment in
// stream order. Segments that one CTA held whole were written by it. blockIdx.x is a segment, or (where
// there are more segments than cuts between CTAs) a cut: the first cut of a segment does its rows. A sum of 0 is an
// absent slot's; a NaN score's is NaN.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) tree_join_kernel(TreeGeo g, TreeArgs a, bool by_cut) {
  extern __shared__ int s_pre[];
  __shared__ int warp_sums[32];
  tree_prefix(g, a, s_pre, warp_sums);
  const TreeStream ts(g, s_pre);
  int b, hr, first, nt;
  bool mine = true;
  if (by_cut) {
    const int cut = blockIdx.x + 1;
    mine = cut < g.C && cut * ts.per < ts.total;
    ts.find(mine ? cut * ts.per : 0, &b, &hr, &first, &nt);
    mine = mine && first / ts.per == cut - 1;
  } else {
    b = blockIdx.x / ts.HR;
    hr = blockIdx.x - b * ts.HR;
    nt = s_pre[b + 1] - s_pre[b];
    first = ts.start(b) + hr * (nt + ts.cost);
  }
  // first and last CTA of the segment
  const int c0 = first / ts.per, c1 = (nt == 1 ? first : first + ts.cost + nt - 1) / ts.per;
  // the parts are written by the kernel before, which may still run. Every block waits, so that this kernel
  // cannot end, and what follows it start, before that one has ended
  grid_wait();
  if (!mine || c0 == c1) return;
  const int hk = hr / g.RG, rg = hr - hk * g.RG, lane = threadIdx.x & 31, n = c1 - c0 + 1;
  constexpr int E = D / 32;
  for (int rr = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); rr < g.RR; rr += gridDim.y * kJoinWarps) {
    int hg, t;
    if (!tree_row(g, rg, rr, &hg, &t)) continue;
    auto part = [&](int i) { return ((int64_t)(c0 + i) * 2 + (i == 0)) * g.RR + rr; };
    constexpr int kAhead = 8;  // parts fetched before their weights are known
    Part<E> ahead[kAhead], acc;
#pragma unroll
    for (int i = 0; i < kAhead; i++) ahead[i].load(a.part_o + part(min(i, n - 1)) * D + lane * E);
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, a.part_ml[2 * part(i)]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float mu = m == -INFINITY ? 0.f : m;
    float l = 0.f;
#pragma unroll
    for (int e = 0; e < E; e++) acc.x[e] = 0.f;
    for (int base = 0; base < n; base += 32) {
      float w = 0.f;
      if (base + lane < n) {
        const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * part(base + lane));
        w = exp2f(ml.x - mu);
        l += w * ml.y;
      }
      if (base == 0) {
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
          const float wi = __shfl_sync(0xffffffffu, w, i);  // 0 behind the last part
#pragma unroll
          for (int e = 0; e < E; e++) acc.x[e] = fmaf(wi, ahead[i].x[e], acc.x[e]);
        }
      }
      const int cnt = min(32, n - base);
#pragma unroll 4
      for (int i = base ? 0 : kAhead; i < cnt; i++) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        Part<E> p;
        p.load(a.part_o + part(base + i) * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e++) acc.x[e] = fmaf(wi, p.x[e], acc.x[e]);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const int h = hk * g.G + hg;
    acc.store(view_at<T>(a.o, b, h, t) + lane * E, l != 0.f ? 1.f / l : 0.f);
    if (a.lse && lane == 0)
      a.lse[((int64_t)b * g.Hq + h) * g.T + t] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
  }
}

template <typename T, int D>
cudaError_t launch_join(const TreeGeo& g, const TreeArgs& a, cudaStream_t st) {
  const int used = g.HM ? g.G * g.T <= 128 ? g.G * g.T : g.RR : g.G * g.T;
  const int rows = used < g.RR ? used : g.RR, segments = g.B * g.Hkv * g.RG;
  const bool by_cut = segments > g.C - 1;
  const int x = by_cut ? g.C - 1 : segments;
  // a warp a row, as long as about eight blocks an SM do
  const int all = (rows + kJoinWarps - 1) / kJoinWarps, some = 8 * 148 / x;
  const dim3 grid(x, all <= some ? all : some < 1 ? 1 : some);
  // launched while the kernel before it still runs; it works out its segments and then waits for the parts
  return launch_early(tree_join_kernel<T, D>, grid, dim3(kJoinWarps * 32), (g.B + 1) * sizeof(int), st, g, a, by_cut);
}

int make_tree_geo(const tree_shape* s, TreeGeo* g) {
  if (!s || s->B <= 0 || s->Hq <= 0 || s->Hkv <= 0 || s->Hq % s->Hkv || s->T <= 0 || s->N < s->T) return PYR_EINVAL;
  if (s->dtype != PYR_F32 && s->dtype != PYR_BF16) return PYR_EUNSUPPORTED;
  if (s->d != 64 && s->d != 128) return PYR_EUNSUPPORTED;
  if (s->T > kTreeMaxT || s->B > kTreeMaxB || s->Hq > 65535 || s->N > (1 << 28)) return PYR_EUNSUPPORTED;
  TreeGeo t = {s->B, s->Hq, s->Hkv, s->Hq / s->Hkv, s->N, s->T, s->d, s->dtype};
  if (t.dtype == PYR_BF16) {
    // one CTA per SM (148): two 128-row tiles where the group's heads do not fit in one
    t.HM = 128 / t.T;
    t.RR = t.G > t.HM ? 256 : 128;
    t.BK = 128;
    t.C = 148;
    t.RG = (t.G + t.HM * (t.RR / 128) - 1) / (t.HM * (t.RR / 128));
  } else {
    t.HM = 0;
    t.RR = t.G * t.T <= 32 ? 32 : 64;  // more rows share a key tile, fewer waste nothing
    t.BK = 64;
    t.C = 296;  // two CTAs per SM
    t.RG = (t.G * t.T + t.RR - 1) / t.RR;
  }
  // positions of the stream are 32-bit
  if ((((int64_t)t.N + t.BK - 1) / t.BK + kSegCost) * t.B > 0x7fffffff / t.Hkv / t.RG - t.C) return PYR_EUNSUPPORTED;
  *g = t;
  return PYR_OK;
}

size_t tree_part_rows(const TreeGeo& g) { return (size_t)g.C * 2 * g.RR; }

}  // namespace

cudaError_t launch_tree_join(const TreeGeo& g, const TreeArgs& a, cudaStream_t st) {
  if (g.dtype == PYR_F32) return g.d == 64 ? launch_join<float, 64>(g, a, st) : launch_join<float, 128>(g, a, st);
  return g.d == 64 ? launch_join<__nv_bfloat16, 64>(g, a, st) : launch_join<__nv_bfloat16, 128>(g, a, st);
}

}  // namespace pyr

extern "C" {

size_t tree_workspace_bytes(const tree_shape* s) {
  pyr::TreeGeo g;
  return pyr::make_tree_geo(s, &g) == PYR_OK ? pyr::tree_part_rows(g) * (g.d + 2) * sizeof(float) : 0;
}

int tree_forward(const tree_shape* s, const pyr_view* Q, const pyr_view* K, const pyr_view* V, const int32_t* len,
                 const int32_t* parent, const pyr_view* O, float* lse, void* workspace, size_t workspace_bytes,
                 int* dev_status, void* stream) {
  pyr::TreeGeo g;
  const int rc = pyr::make_tree_geo(s, &g);
  if (rc) return rc;
  pyr::TreeArgs a;
  if (!pyr::check_view(Q, g.B, g.Hq, g.T, g.d, g.dtype, false, &a.q) ||
      !pyr::check_view(K, g.B, g.Hkv, g.N, g.d, g.dtype, false, &a.k) ||
      !pyr::check_view(V, g.B, g.Hkv, g.N, g.d, g.dtype, false, &a.v) ||
      !pyr::check_view(O, g.B, g.Hq, g.T, g.d, g.dtype, true, &a.o) || !len || !workspace || !pyr::aligned4(len) ||
      !pyr::aligned4(parent) || !pyr::aligned4(lse) || !pyr::aligned16(workspace) ||
      workspace_bytes < tree_workspace_bytes(s))
    return PYR_EINVAL;
  a.len = len;
  a.parent = parent;
  a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = a.part_o + pyr::tree_part_rows(g) * g.d;
  a.status = dev_status;
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = g.dtype == PYR_F32 ? pyr::launch_tree_simt(g, a, st) : pyr::launch_tree_tc(g, a, st);
  if (e == cudaSuccess) e = pyr::launch_tree_join(g, a, st);
  return e == cudaSuccess ? PYR_OK : PYR_ECUDA;
}

}  // extern "C"
