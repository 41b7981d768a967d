// Packed prompts: the C entry points and the planner.
#include "packed.cuh"

namespace pyr {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 2048;

// exclusive prefix sum over the block; total in *sum. Barriers inside.
__device__ int block_scan(int x, int* warp_sums, int* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += u;
  }
  if (lane == 31) warp_sums[warp] = y;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const int r = y - x + (warp ? warp_sums[warp - 1] : 0);
  *sum = warp_sums[31];
  __syncthreads();
  return r;
}

// One block writes the three lists. Each: tile counts summed over the sequences, then a counting sort of
// all tiles by work in 2048 buckets. Tiles of one bucket come in no fixed order; every tile's result is
// its own, so the order moves no bit of the output. Bound by the latency of its passes: 9 us for a few sequences (32K
// tokens in 4), 14 us for 512 of 64 tokens, 44 us for 16 of 64K, 0.47 ms for 32768 of 8.
__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(PackedGeo g, const int32_t* __restrict__ cu,
                                                                   int32_t* __restrict__ plan, int* status) {
  __shared__ int hist[kBuckets];
  __shared__ int warp_sums[32];
  __shared__ int s_bad, s_most;
  const int tid = threadIdx.x;
  if (tid == 0) s_bad = 0;
  if (tid < kPlanHeader) plan[tid] = tid == 3 ? packed_plan_mark(g) : 0;
  __syncthreads();
  for (int s = tid; s < g.S; s += kPlanThreads) {
    const int a = cu[s], b = cu[s + 1];
    if (a < 0 || b < a || b > g.T) s_bad = 1;
  }
  __syncthreads();
  if (s_bad) {
    if (tid == 0) report(status, PYR_EBADSEQ);
    return;
  }
  int32_t* first = plan + packed_list_at(g, 3);
  for (int list = 0; list < 3; list++) {
    const int rows = packed_tile_rows(g, list);
    int4* out = reinterpret_cast<int4*>(plan + packed_list_at(g, list));
    if (tid == 0) s_most = 1;
    for (int i = tid; i < kBuckets; i += kPlanThreads) hist[i] = 0;
    __syncthreads();
    int total = 0;
    for (int base = 0; base < g.S; base += kPlanThreads) {
      const int s = base + tid;
      const int nt = s < g.S ? (cu[s + 1] - cu[s] + rows - 1) / rows : 0;
      int sum;
      const int at = block_scan(nt, warp_sums, &sum);
      if (s < g.S) first[s] = total + at;
      if (nt > 1) atomicMax(&s_most, nt);
      total += sum;
    }
    if (tid == 0) {
      first[g.S] = total;
      plan[list] = total;
    }
    __syncthreads();
    const int most = s_most;
    for (int pass = 0; pass < 2; pass++) {
      for (int x = tid; x < total; x += kPlanThreads) {
        int lo = 0, hi = g.S;  // first[lo] <= x < first[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (first[mid] <= x)
            lo = mid;
          else
            hi = mid;
        }
        const int j = x - first[lo], nt = first[lo + 1] - first[lo];
        const int w = list == kListK ? nt - j : j + 1;  // 1 .. most
        const int bucket = kBuckets - 1 - (int)((int64_t)(w - 1) * kBuckets / most);
        const int slot = atomicAdd(&hist[bucket], 1);
        if (pass) out[slot] = make_int4(cu[lo], cu[lo + 1], cu[lo] + j * rows, 0);
      }
      __syncthreads();
      if (pass == 0) {
        const int a = hist[2 * tid], b = hist[2 * tid + 1];
        int sum;
        const int at = block_scan(a + b, warp_sums, &sum);
        hist[2 * tid] = at;
        hist[2 * tid + 1] = at + a;
        __syncthreads();
      }
    }
  }
}

int make_packed_geo(const packed_shape* s, PackedGeo* g) {
  if (!s || s->S <= 0 || s->T <= 0 || s->Hq <= 0 || s->Hkv <= 0 || s->Hq % s->Hkv) return PYR_EINVAL;
  if (s->dtype != PYR_F32 && s->dtype != PYR_BF16) return PYR_EUNSUPPORTED;
  if (s->d != 64 && s->d != 128) return PYR_EUNSUPPORTED;
  if (s->T > (1 << 28) || s->S > (1 << 28) || s->Hq > 65535) return PYR_EUNSUPPORTED;
  *g = {s->S, s->T, s->Hq, s->Hkv, s->Hq / s->Hkv, s->d, s->dtype};
  for (int i = 0; i < 3; i++)  // one thread block per (tile, head) at most
    if (packed_list_cap(*g, i) * s->Hq > 0x7fffffff) return PYR_EUNSUPPORTED;
  return PYR_OK;
}

}  // namespace

cudaError_t launch_packed_plan(const PackedGeo& g, const int32_t* cu, int32_t* plan, int* status, cudaStream_t st) {
  packed_plan_kernel<<<1, kPlanThreads, 0, st>>>(g, cu, plan, status);
  return cudaGetLastError();
}

}  // namespace pyr

using pyr::check_view;
using pyr::PackedGeo;

extern "C" {

size_t packed_plan_elems(const packed_shape* s) {
  PackedGeo g;
  return pyr::make_packed_geo(s, &g) == PYR_OK ? (size_t)pyr::packed_plan_words(g) : 0;
}

int packed_plan(const packed_shape* s, const int32_t* cu, int32_t* plan, int* dev_status, void* stream) {
  PackedGeo g;
  const int rc = pyr::make_packed_geo(s, &g);
  if (rc) return rc;
  if (!cu || !plan || !pyr::aligned4(cu) || !pyr::aligned16(plan)) return PYR_EINVAL;
  return pyr::launch_packed_plan(g, cu, plan, dev_status, (cudaStream_t)stream) == cudaSuccess ? PYR_OK : PYR_ECUDA;
}

int packed_forward(const packed_shape* s, const pyr_view* Q, const pyr_view* K, const pyr_view* V,
                   const int32_t* plan, const pyr_view* O, float* lse, int* dev_status, void* stream) {
  PackedGeo g;
  const int rc = pyr::make_packed_geo(s, &g);
  if (rc) return rc;
  pyr::PackedFwdArgs a;
  if (!check_view(Q, 1, g.Hq, g.T, g.d, g.dtype, false, &a.q) ||
      !check_view(K, 1, g.Hkv, g.T, g.d, g.dtype, false, &a.k) ||
      !check_view(V, 1, g.Hkv, g.T, g.d, g.dtype, false, &a.v) ||
      !check_view(O, 1, g.Hq, g.T, g.d, g.dtype, true, &a.o) || !plan || !pyr::aligned16(plan) ||
      !pyr::aligned4(lse))
    return PYR_EINVAL;
  a.plan = plan;
  a.lse = lse;
  a.status = dev_status;
  const cudaError_t e = g.dtype == PYR_F32 ? pyr::launch_packed_fwd_simt(g, a, (cudaStream_t)stream)
                                           : pyr::launch_packed_fwd_tc(g, a, (cudaStream_t)stream);
  return e == cudaSuccess ? PYR_OK : PYR_ECUDA;
}

int packed_backward(const packed_shape* s, const pyr_view* Q, const pyr_view* K, const pyr_view* V,
                    const int32_t* plan, const pyr_view* O, const float* lse, const pyr_view* dO, float* delta,
                    const pyr_view* dQ, const pyr_view* dK, const pyr_view* dV, int* dev_status, void* stream) {
  PackedGeo g;
  const int rc = pyr::make_packed_geo(s, &g);
  if (rc) return rc;
  pyr::PackedBwdArgs a;
  if (!check_view(Q, 1, g.Hq, g.T, g.d, g.dtype, false, &a.q) ||
      !check_view(K, 1, g.Hkv, g.T, g.d, g.dtype, false, &a.k) ||
      !check_view(V, 1, g.Hkv, g.T, g.d, g.dtype, false, &a.v) ||
      !check_view(O, 1, g.Hq, g.T, g.d, g.dtype, false, &a.o) ||
      !check_view(dO, 1, g.Hq, g.T, g.d, g.dtype, false, &a.dout) ||
      !check_view(dQ, 1, g.Hq, g.T, g.d, g.dtype, true, &a.dq) ||
      !check_view(dK, 1, g.Hkv, g.T, g.d, g.dtype, true, &a.dk) ||
      !check_view(dV, 1, g.Hkv, g.T, g.d, g.dtype, true, &a.dv) || !plan || !lse || !delta ||
      !pyr::aligned16(plan) || !pyr::aligned4(lse) || !pyr::aligned4(delta))
    return PYR_EINVAL;
  a.plan = plan;
  a.lse = lse;
  a.delta = delta;
  a.status = dev_status;
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = pyr::launch_packed_delta(g, a, st);
  if (e == cudaSuccess)
    e = g.dtype == PYR_F32 ? pyr::launch_packed_bwd_simt(g, a, st) : pyr::launch_packed_bwd_tc(g, a, st);
  return e == cudaSuccess ? PYR_OK : PYR_ECUDA;
}

}  // extern "C"
