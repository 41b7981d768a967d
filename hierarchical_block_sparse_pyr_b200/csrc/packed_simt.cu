// Causal attention of packed prompts and its gradients on the CUDA cores, fp32 arithmetic throughout: the
// fp32 path (reduced-precision tensor-core operands would lose what fp32 callers keep).
//
// Forward and dQ: one CTA per (32-row tile, query head), walking the keys up to the tile's end. dK/dV: one per
// (32-key tile, key/value head), walking the rows from the tile's start on, over the heads of its group, so
// that every gradient is summed by one CTA in a fixed order. Tiles come longest first from the plan.
// A CTA is two (d = 128) or four (d = 64) teams of 128 threads that take the steps of its walk in turn with sums
// of their own, added in the teams' order at the end: the longest walk bounds small calls (2 heads of 64, 4K
// tokens, gradients: one team 450 us, two 267, four 231).
// Rows behind the sequence's end are loaded as zeros, never from memory.
#include "packed.cuh"
#include "simt_tile.cuh"

namespace pyr {

namespace {

using namespace simt;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 32;         // rows of a tile, packed_tile_rows() of fp32
constexpr int kTeam = 4 * kRows;  // threads of a team
template <int D>
constexpr int kTeams = D == 64 ? 4 : 2;  // as many as shared memory holds
template <int D>
constexpr int kThreads = kTeams<D> * kTeam;

__device__ __forceinline__ int team() { return threadIdx.x / kTeam; }
__device__ __forceinline__ void team_sync() { asm volatile("bar.sync %0, %1;" ::"r"(1 + team()), "n"(kTeam) : "memory"); }

// the teams' 32 x D sums on their way to team 0, in shared memory that all have finished with
template <int D>
__device__ __forceinline__ void put_acc(float* buf, const float (&acc)[4][D / 16]) {
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int c = 0; c < D / 16; c++) buf[(i * (D / 16) + c) * kTeam + team_tid<kTeam>()] = acc[i][c];
}
template <int D>
__device__ __forceinline__ float got_acc(const float* buf, int i, int c) {
  return buf[(i * (D / 16) + c) * kTeam + team_tid<kTeam>()];
}

template <int D>
constexpr int fwd_team() { return kTile * (D + 4) + kTile * D; }  // K (P over K), V
template <int D>
constexpr int fwd_smem() {
  return (kRows * (D + 4) + kTeams<D> * fwd_team<D>()) * 4;  // Q, and the teams' tiles
}

// S = Q K^T, online softmax, O += P V over 64-key tiles; P goes over K's buffer.
template <int D>
__global__ void __launch_bounds__(kThreads<D>) packed_fwd_simt_kernel(PackedGeo g, PackedFwdArgs a) {
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm, *Ks = Qs + kRows * (D + 4) + team() * fwd_team<D>(), *Vs = Ks + kTile * (D + 4), *Ps = Ks;
  const int tile = blockIdx.x / g.Hq, h = blockIdx.x - tile * g.Hq;
  if (tile >= packed_tiles(g, a.plan, kListFwd, a.status)) return;
  const int4 w = reinterpret_cast<const int4*>(a.plan + packed_list_at(g, kListFwd))[tile];
  const int start = w.x, end = w.y, row0 = w.z, hk = h / g.G;
  const int tx = threadIdx.x & 15, ty = team_tid<kTeam>() >> 4;
  const float sl2 = rsqrtf((float)D) * kLog2e;
  const int nrow = min(kRows, end - row0);
  load_rows<kThreads<D>, D, kRows>(Qs, D + 4, view_at<float>(a.q, 0, h, row0), a.q.row, nrow);
  __syncthreads();
  float m[4], l[4], acc[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; c++) acc[i][c] = 0.f;
  }
  const int stop = row0 + nrow;
  for (int k0 = start + team() * kTile; k0 < stop; k0 += kTeams<D> * kTile) {
    const int nk = min(kTile, stop - k0);
    team_sync();
    load_rows<kTeam, D, kTile>(Ks, D + 4, view_at<float>(a.k, 0, hk, k0), a.k.row, nk);
    load_rows<kTeam, D, kTile>(Vs, D, view_at<float>(a.v, 0, hk, k0), a.v.row, nk);
    team_sync();
    float s[4][4];
    mul_nt<kTeam, D>(s, Qs, D + 4, Ks, D + 4);
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) s[i][j] = k0 + tx + 16 * j <= row0 + 4 * ty + i ? s[i][j] * sl2 : -INFINITY;
    softmax_step<D>(s, m, l, acc);
    team_sync();  // every thread is done with K
    store_p<kTeam>(Ps, s);
    __syncwarp();  // a row of P is written and read by one half-warp
    mul_acc<kTeam, D>(acc, Ps, Vs, D);
  }
  __syncthreads();
  // per team behind the first: 32 x D sums, then maximum and sum of the rows (each thread's own copy)
  constexpr int kMl = kRows * D, kPart = kMl + 8 * kTeam;
  if (team() > 0) {
    float* buf = sm + (team() - 1) * kPart;
    put_acc<D>(buf, acc);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      buf[kMl + (2 * i) * kTeam + team_tid<kTeam>()] = m[i];
      buf[kMl + (2 * i + 1) * kTeam + team_tid<kTeam>()] = l[i];
    }
  }
  __syncthreads();
  if (team() > 0) return;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int t = row0 + 4 * ty + i;
    if (t >= end) continue;
    // team 0 has seen the first tile, which every row sees; the others may have seen nothing (m = -inf)
#pragma unroll
    for (int k = 1; k < kTeams<D>; k++) {
      const float* buf = sm + (k - 1) * kPart;
      const float m1 = buf[kMl + (2 * i) * kTeam + team_tid<kTeam>()];
      const float mm = fmaxf(m[i], m1), f0 = exp2f(m[i] - mm), f1 = exp2f(m1 - mm);
      l[i] = l[i] * f0 + buf[kMl + (2 * i + 1) * kTeam + team_tid<kTeam>()] * f1;
      m[i] = mm;
#pragma unroll
      for (int c = 0; c < D / 16; c++) acc[i][c] = acc[i][c] * f0 + got_acc<D>(buf, i, c) * f1;
    }
    store_row<D>(view_at<float>(a.o, 0, h, t), acc[i], 1.f / l[i]);
    if (a.lse && tx == 0) a.lse[(int64_t)h * g.T + t] = (m[i] + log2f(l[i])) * 0.6931471805599453f;
  }
}

// delta[t] = dO_t . O_t for the rows of the sequences. A row is read by as many lanes as it has 16-byte
// chunks, and a thread has four rows' chunks of both tensors in flight: one pass, bound by HBM.
template <typename T, int D>
__global__ void __launch_bounds__(256) packed_delta_kernel(PackedGeo g, PackedBwdArgs a) {
  constexpr int E = 16 / sizeof(T), L = D / E, U = 4;  // elements a chunk, lanes a row, rows a thread
  const int tile = blockIdx.x / g.Hq, h = blockIdx.x - tile * g.Hq;
  if (tile >= packed_tiles(g, a.plan, kListQ, a.status)) return;
  const int4 w = reinterpret_cast<const int4*>(a.plan + packed_list_at(g, kListQ))[tile];
  const int lane = threadIdx.x % L;
  const int stop = min(w.z + packed_tile_rows(g, kListQ), w.y);
  // the loop is the block's as a whole: the sums below are exchanged by whole warps, whose rows may end at different t
  for (int base = w.z; base < stop; base += U * (256 / L)) {
    const int t0 = base + threadIdx.x / L;
    uint4 o[U], d[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int t = t0 + u * (256 / L);
      o[u] = d[u] = make_uint4(0, 0, 0, 0);
      if (t < stop) {
        o[u] = __ldcs(reinterpret_cast<const uint4*>(view_at<T>(a.o, 0, h, t)) + lane);
        d[u] = __ldg(reinterpret_cast<const uint4*>(view_at<T>(a.dout, 0, h, t)) + lane);
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const T *x = reinterpret_cast<const T*>(&o[u]), *y = reinterpret_cast<const T*>(&d[u]);
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; e++) s = fmaf(to_f32(x[e]), to_f32(y[e]), s);
#pragma unroll
      for (int m = L / 2; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
      const int t = t0 + u * (256 / L);
      if (lane == 0 && t < stop) a.delta[(int64_t)h * g.T + t] = s;
    }
  }
}

template <int D>
constexpr int bwd_team() { return 2 * kTile * (D + 4) + kRows * kPitchP; }  // a tile of two operands, P or dS
template <int D>
constexpr int bwd_smem() {
  return (2 * kRows * (D + 4) + kTeams<D> * bwd_team<D>()) * 4;  // two operands of the CTA's rows, and the teams' tiles
}

// dS = P (dO V^T - delta), dQ += dS K
template <int D>
__global__ void __launch_bounds__(kThreads<D>) packed_dq_simt_kernel(PackedGeo g, PackedBwdArgs a) {
  extern __shared__ __align__(16) float sm[];
  constexpr int P = D + 4;
  float *Qs = sm, *Gs = Qs + kRows * P, *Ks = Gs + kRows * P + team() * bwd_team<D>(), *Vs = Ks + kTile * P,
        *Ps = Vs + kTile * P;
  const int tile = blockIdx.x / g.Hq, h = blockIdx.x - tile * g.Hq;
  if (tile >= packed_tiles(g, a.plan, kListQ, a.status)) return;
  const int4 w = reinterpret_cast<const int4*>(a.plan + packed_list_at(g, kListQ))[tile];
  const int start = w.x, end = w.y, row0 = w.z, hk = h / g.G;
  const int tx = threadIdx.x & 15, ty = team_tid<kTeam>() >> 4;
  const float scale = rsqrtf((float)D), sl2 = scale * kLog2e;
  const int nrow = min(kRows, end - row0);
  load_rows<kThreads<D>, D, kRows>(Qs, P, view_at<float>(a.q, 0, h, row0), a.q.row, nrow);
  load_rows<kThreads<D>, D, kRows>(Gs, P, view_at<float>(a.dout, 0, h, row0), a.dout.row, nrow);
  float lse2[4], del[4], acc[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int t = min(row0 + 4 * ty + i, end - 1);
    lse2[i] = a.lse[(int64_t)h * g.T + t] * kLog2e;
    del[i] = a.delta[(int64_t)h * g.T + t];
#pragma unroll
    for (int c = 0; c < D / 16; c++) acc[i][c] = 0.f;
  }
  __syncthreads();
  const int stop = row0 + nrow;
  for (int k0 = start + team() * kTile; k0 < stop; k0 += kTeams<D> * kTile) {
    const int nk = min(kTile, stop - k0);
    team_sync();
    load_rows<kTeam, D, kTile>(Ks, P, view_at<float>(a.k, 0, hk, k0), a.k.row, nk);
    load_rows<kTeam, D, kTile>(Vs, P, view_at<float>(a.v, 0, hk, k0), a.v.row, nk);
    team_sync();
    float s[4][4], dp[4][4];
    mul_nt<kTeam, D>(s, Qs, P, Ks, P);
    mul_nt<kTeam, D>(dp, Gs, P, Vs, P);
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 4; j++)
        s[i][j] = k0 + tx + 16 * j <= row0 + 4 * ty + i ? exp2f(s[i][j] * sl2 - lse2[i]) : 0.f;
    if (stop - start <= kTile) {
      // The row sees this tile alone, perhaps one key, where dP and delta cancel: delta += sum_k P (dP - delta),
      // which is sum_k P dP up to the rounding of the difference. The dK/dV kernel, which runs second, reads it.
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; j++) sum = fmaf(s[i][j], dp[i][j] - del[i], sum);
#pragma unroll
        for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        del[i] += sum;
        const int t = row0 + 4 * ty + i;
        if (tx == 0 && t < end) a.delta[(int64_t)h * g.T + t] = del[i];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) s[i][j] *= dp[i][j] - del[i];
    store_p<kTeam>(Ps, s);
    __syncwarp();
    mul_acc<kTeam, D>(acc, Ps, Ks, P);
    __syncwarp();
  }
  __syncthreads();
  if (team() > 0) put_acc<D>(sm + (team() - 1) * kRows * D, acc);
  __syncthreads();
  if (team() > 0) return;
#pragma unroll
  for (int i = 0; i < 4; i++) {
#pragma unroll
    for (int k = 0; k < kTeams<D> - 1; k++)
#pragma unroll
      for (int c = 0; c < D / 16; c++) acc[i][c] += got_acc<D>(sm + k * kRows * D, i, c);
    if (row0 + 4 * ty + i < end) store_row<D>(view_at<float>(a.dq, 0, h, row0 + 4 * ty + i), acc[i], scale);
  }
}

// rows = keys, columns = queries: dV += P^T dO, dK += dS^T Q over the rows of the group's heads
template <int D>
__global__ void __launch_bounds__(kThreads<D>) packed_dkdv_simt_kernel(PackedGeo g, PackedBwdArgs a) {
  extern __shared__ __align__(16) float sm[];
  constexpr int P = D + 4;
  float *Ks = sm, *Vs = Ks + kRows * P, *Qs = Vs + kRows * P + team() * bwd_team<D>(), *Gs = Qs + kTile * P,
        *Ps = Gs + kTile * P;
  const int tile = blockIdx.x / g.Hkv, hk = blockIdx.x - tile * g.Hkv;
  if (tile >= packed_tiles(g, a.plan, kListK, a.status)) return;
  const int4 w = reinterpret_cast<const int4*>(a.plan + packed_list_at(g, kListK))[tile];
  const int end = w.y, key0 = w.z;
  const int tx = threadIdx.x & 15, ty = team_tid<kTeam>() >> 4;
  const float scale = rsqrtf((float)D), sl2 = scale * kLog2e;
  const int nk = min(kRows, end - key0);
  load_rows<kThreads<D>, D, kRows>(Ks, P, view_at<float>(a.k, 0, hk, key0), a.k.row, nk);
  load_rows<kThreads<D>, D, kRows>(Vs, P, view_at<float>(a.v, 0, hk, key0), a.v.row, nk);
  __syncthreads();
  float dk[4][D / 16], dv[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int c = 0; c < D / 16; c++) dk[i][c] = dv[i][c] = 0.f;
  const int nq_tiles = (end - key0 + kTile - 1) / kTile, steps = nq_tiles * g.G;
  for (int step = team(); step < steps; step += kTeams<D>) {
    const int h = hk * g.G + step / nq_tiles, q0 = key0 + step % nq_tiles * kTile;
    const int nq = min(kTile, end - q0);
    team_sync();
    load_rows<kTeam, D, kTile>(Qs, P, view_at<float>(a.q, 0, h, q0), a.q.row, nq);
    load_rows<kTeam, D, kTile>(Gs, P, view_at<float>(a.dout, 0, h, q0), a.dout.row, nq);
    team_sync();
    float s[4][4], dp[4][4];
    mul_nt<kTeam, D>(s, Ks, P, Qs, P);
    mul_nt<kTeam, D>(dp, Vs, P, Gs, P);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int t = q0 + tx + 16 * j, tc = min(t, end - 1);
      const float lse2 = a.lse[(int64_t)h * g.T + tc] * kLog2e, del = a.delta[(int64_t)h * g.T + tc];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        s[i][j] = key0 + 4 * ty + i <= t && t < end ? exp2f(s[i][j] * sl2 - lse2) : 0.f;
        dp[i][j] = s[i][j] * (dp[i][j] - del);
      }
    }
    store_p<kTeam>(Ps, s);
    __syncwarp();
    mul_acc<kTeam, D>(dv, Ps, Gs, P);
    __syncwarp();
    store_p<kTeam>(Ps, dp);
    __syncwarp();
    mul_acc<kTeam, D>(dk, Ps, Qs, P);
    __syncwarp();
  }
  __syncthreads();
  if (team() > 0) {
    put_acc<D>(sm + (2 * team() - 2) * kRows * D, dk);
    put_acc<D>(sm + (2 * team() - 1) * kRows * D, dv);
  }
  __syncthreads();
  if (team() > 0) return;
#pragma unroll
  for (int i = 0; i < 4; i++) {
#pragma unroll
    for (int k = 0; k < kTeams<D> - 1; k++)
#pragma unroll
      for (int c = 0; c < D / 16; c++) {
        dk[i][c] += got_acc<D>(sm + 2 * k * kRows * D, i, c);
        dv[i][c] += got_acc<D>(sm + (2 * k + 1) * kRows * D, i, c);
      }
    if (4 * ty + i >= nk) continue;
    store_row<D>(view_at<float>(a.dk, 0, hk, key0 + 4 * ty + i), dk[i], scale);
    store_row<D>(view_at<float>(a.dv, 0, hk, key0 + 4 * ty + i), dv[i], 1.f);
  }
}

template <typename K, typename A>
cudaError_t launch(K kern, int64_t blocks, int threads, int smem, const PackedGeo& g, const A& a, cudaStream_t st) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<(unsigned)blocks, threads, smem, st>>>(g, a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_bwd(const PackedGeo& g, const PackedBwdArgs& a, cudaStream_t st) {
  const cudaError_t e =
      launch(packed_dq_simt_kernel<D>, packed_list_cap(g, kListQ) * g.Hq, kThreads<D>, bwd_smem<D>(), g, a, st);
  if (e != cudaSuccess) return e;
  return launch(packed_dkdv_simt_kernel<D>, packed_list_cap(g, kListK) * g.Hkv, kThreads<D>, bwd_smem<D>(), g, a, st);
}

}  // namespace

cudaError_t launch_packed_fwd_simt(const PackedGeo& g, const PackedFwdArgs& a, cudaStream_t st) {
  const int64_t blocks = packed_list_cap(g, kListFwd) * g.Hq;
  return g.d == 64 ? launch(packed_fwd_simt_kernel<64>, blocks, kThreads<64>, fwd_smem<64>(), g, a, st)
                   : launch(packed_fwd_simt_kernel<128>, blocks, kThreads<128>, fwd_smem<128>(), g, a, st);
}

cudaError_t launch_packed_delta(const PackedGeo& g, const PackedBwdArgs& a, cudaStream_t st) {
  const int64_t blocks = packed_list_cap(g, kListQ) * g.Hq;
  if (g.dtype == PYR_F32)
    return g.d == 64 ? launch(packed_delta_kernel<float, 64>, blocks, 256, 0, g, a, st)
                     : launch(packed_delta_kernel<float, 128>, blocks, 256, 0, g, a, st);
  return g.d == 64 ? launch(packed_delta_kernel<__nv_bfloat16, 64>, blocks, 256, 0, g, a, st)
                   : launch(packed_delta_kernel<__nv_bfloat16, 128>, blocks, 256, 0, g, a, st);
}

cudaError_t launch_packed_bwd_simt(const PackedGeo& g, const PackedBwdArgs& a, cudaStream_t st) {
  return g.d == 64 ? launch_bwd<64>(g, a, st) : launch_bwd<128>(g, a, st);
}

}  // namespace pyr
