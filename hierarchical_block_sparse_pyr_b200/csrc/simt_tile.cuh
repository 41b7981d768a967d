// ROWS x 64 tiles of fp32 attention on the CUDA cores by a team of NT = 4 ROWS threads (a block may hold
// several teams, each of consecutive threads). Thread (tx, ty) = (tid % 16, tid / 16) of its team
// owns rows 4 ty .. 4 ty + 3 of every product; of a ROWS x 64 product it owns the columns tx + 16 j (four,
// which keeps the 16-byte reads of the other operand's rows conflict-free with a row pitch of D + 4), of a
// ROWS x D product the columns 4 tx + 64 j .. + 3. Rows of the result are written and read by one half-warp.
#pragma once

#include "view.cuh"

namespace pyr {
namespace simt {

constexpr int kTile = 64;            // columns of a step
constexpr int kPitchP = kTile + 4;

template <int NT>
__device__ __forceinline__ int team_tid() { return threadIdx.x & (NT - 1); }

// dst[r][0 .. D) = row r of src where wanted(r), zeros in the other of the N rows
template <int NT, int D, int N, typename F>
__device__ __forceinline__ void load_rows_if(float* dst, int pitch, const float* src, int64_t stride, F wanted) {
  constexpr int C = D / 4;
#pragma unroll 4
  for (int x = team_tid<NT>(); x < N * C; x += NT) {
    const int r = x / C, c = 4 * (x - r * C);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (wanted(r)) v = *reinterpret_cast<const float4*>(src + r * stride + c);
    *reinterpret_cast<float4*>(dst + r * pitch + c) = v;
  }
}

template <int NT, int D, int N>
__device__ __forceinline__ void load_rows(float* dst, int pitch, const float* src, int64_t stride, int n) {
  load_rows_if<NT, D, N>(dst, pitch, src, stride, [n](int r) { return r < n; });
}

// acc[i][j] = A[4 ty + i] . B[tx + 16 j] over D elements
template <int NT, int D>
__device__ __forceinline__ void mul_nt(float (&acc)[4][4], const float* A, int pa, const float* B, int pb) {
  const int tx = threadIdx.x & 15, ty = team_tid<NT>() >> 4;
  float2 sum[4][4];  // of the even and of the odd elements
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) sum[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int e = 0; e < D; e += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; i++) a[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * pa + e);
#pragma unroll
    for (int j = 0; j < 4; j++) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * pb + e);
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) {
        sum[i][j] = __ffma2_rn(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), sum[i][j]);
        sum[i][j] = __ffma2_rn(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), sum[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) acc[i][j] = sum[i][j].x + sum[i][j].y;
}

// acc[i][4 j + c] += sum_k P[4 ty + i][k] V[k][4 tx + 64 j + c], k = 0 .. 63
template <int NT, int D>
__device__ __forceinline__ void mul_acc(float (&acc)[4][D / 16], const float* P, const float* V, int pv) {
  const int tx = threadIdx.x & 15, ty = team_tid<NT>() >> 4;
#pragma unroll 2
  for (int k = 0; k < kTile; k += 4) {
    float p[4][4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float4 x = *reinterpret_cast<const float4*>(P + (4 * ty + i) * kPitchP + k);
      p[i][0] = x.x, p[i][1] = x.y, p[i][2] = x.z, p[i][3] = x.w;
    }
#pragma unroll
    for (int kk = 0; kk < 4; kk++)
#pragma unroll
      for (int j = 0; j < D / 64; j++) {
        const float4 v = *reinterpret_cast<const float4*>(V + (k + kk) * pv + 4 * tx + 64 * j);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          float2* c = reinterpret_cast<float2*>(&acc[i][4 * j]);
          const float2 w = make_float2(p[i][kk], p[i][kk]);
          c[0] = __ffma2_rn(w, make_float2(v.x, v.y), c[0]);
          c[1] = __ffma2_rn(w, make_float2(v.z, v.w), c[1]);
        }
      }
  }
}

template <int NT>
__device__ __forceinline__ void store_p(float* P, const float (&s)[4][4]) {
  const int tx = threadIdx.x & 15, ty = team_tid<NT>() >> 4;
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) P[(4 * ty + i) * kPitchP + tx + 16 * j] = s[i][j];
}

// one step of the online softmax over a 64-column tile of scores in log2 units (-inf: not attended):
// s becomes the probabilities against the new maximum, acc is rescaled
template <int D>
__device__ __forceinline__ void softmax_step(float (&s)[4][4], float (&m)[4], float (&l)[4],
                                             float (&acc)[4][D / 16]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    float mx = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
    for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m[i], mx);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m[i] - mu);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      s[i][j] = exp2f(s[i][j] - mu);
      sum += s[i][j];
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l[i] = l[i] * f + sum;
    m[i] = mn;
#pragma unroll
    for (int c = 0; c < D / 16; c++) acc[i][c] *= f;
  }
}

// row 4 ty + i of a 64 x D accumulator, times f, to memory
template <int D>
__device__ __forceinline__ void store_row(float* dst, const float (&acc)[D / 16], float f) {
  const int tx = threadIdx.x & 15;
#pragma unroll
  for (int j = 0; j < D / 64; j++)
    *reinterpret_cast<float4*>(dst + 4 * tx + 64 * j) =
        make_float4(acc[4 * j] * f, acc[4 * j + 1] * f, acc[4 * j + 2] * f, acc[4 * j + 3] * f);
}

}  // namespace simt
}  // namespace pyr
