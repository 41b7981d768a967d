// What the softmax warps of the tensor-core kernels over strided operands share: rows of scores in
// registers, exponentials on two pipes, register shares of the warpgroups, work order of persistent CTAs.
#pragma once

#include <cuda_bf16.h>

#include "tc_util.cuh"

namespace pyr {
namespace tc {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;  // an accumulator is rescaled when the row maximum grew by more (log2 units)

// Wait whose outcome the whole warp shares, so that a timeout never leaves the warp diverged in front of
// a .sync.aligned instruction.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  const bool ok = mbar_wait(bar, parity, abort_flag);
  return __all_sync(0xffffffffu, ok);
}

// Warps that issue tensor-core products run their loops as a whole and elect one lane for the issue alone:
// with loop bounds, stages and descriptors the same in every lane by construction, these stay in uniform
// registers, which is where the instruction takes its operands from. Issued under a branch on the lane, each
// product has to move its operands there first and takes about 100 cycles while the softmax warps compete
// for issue slots, against 64 of execution.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void drain(uint64_t* bar) {  // every product issued so far, by the whole warp
  if (elect_one()) umma_commit(bar);
  __syncwarp();
  volatile int no_abort = 0;
  mbar_wait(bar, 0, &no_abort);
  __syncwarp();
}

// Registers move from the warpgroup that loads and issues to those that hold rows of scores. The shares have
// to add up to what the block was launched with.
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// maxima that are NaN if an operand is
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max32(const float* s) {
  float a[11];
#pragma unroll
  for (int k = 0; k < 10; k++) a[k] = max3_nan(s[3 * k], s[3 * k + 1], s[3 * k + 2]);
  a[10] = max_nan(s[30], s[31]);
  const float x = max3_nan(a[0], a[1], a[2]), y = max3_nan(a[3], a[4], a[5]), z = max3_nan(a[6], a[7], a[8]);
  return max_nan(max3_nan(x, y, z), max_nan(a[9], a[10]));
}

// 16 consecutive 32-bit columns of this thread's lane, stored from registers.
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 2^x on the FMA pipe for x <= 127 (the MUFU unit gives 16 results a cycle and SM, and a 128 x 128 tile's
// exponentials on it alone take as long as two of its products). x = n + f with n the nearest integer
// (adding 1.5 * 2^23 leaves n in the low bits) and f in [-1/2, 1/2]; 2^f is 1 + f (c1 + f (c2 + ...)) with
// the coefficients of least maximum relative error for that form (found by linear programming on a grid of
// 4001 points): 1.0e-4 for degree 3, 2.9e-6 for degree 4, against 2^-9 = 2e-3 of the rounding to bf16 that
// follows. Below -127 the clamp makes n = -127, f = 0, and the exponent gives exactly 0.
// KEEP_NAN: NaN stays NaN, as on the MUFU unit: the clamp hands it on, and 2^n is a factor instead of an addition to
// the exponent's bits, which would make a number of it. Without, NaN becomes 0, for rows whose other columns are NaN
// as well.
template <int DEG, bool KEEP_NAN>
__device__ __forceinline__ float2 exp2_fma(float2 x) {
  constexpr float kMagic = 12582912.f;
  x.x = KEEP_NAN ? max_nan(x.x, -127.f) : fmaxf(x.x, -127.f);
  x.y = KEEP_NAN ? max_nan(x.y, -127.f) : fmaxf(x.y, -127.f);
  const float2 t = __fadd2_rn(x, make_float2(kMagic, kMagic));
  const float2 n = __fadd2_rn(t, make_float2(-kMagic, -kMagic));
  const float2 f = __ffma2_rn(n, make_float2(-1.f, -1.f), x);
  float2 p;
  if (DEG == 3) {
    p = __ffma2_rn(f, make_float2(0.05500906f, 0.05500906f), make_float2(0.24221097f, 0.24221097f));
    p = __ffma2_rn(f, p, make_float2(0.6932829f, 0.6932829f));
  } else {
    p = __ffma2_rn(f, make_float2(0.009582576f, 0.009582576f), make_float2(0.05590683f, 0.05590683f));
    p = __ffma2_rn(f, p, make_float2(0.24024107f, 0.24024107f));
    p = __ffma2_rn(f, p, make_float2(0.6931241f, 0.6931241f));
  }
  p = __ffma2_rn(f, p, make_float2(1.f, 1.f));
  if (!KEEP_NAN)
    return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23)),
                       __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23)));
  return __fmul2_rn(p, make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + 0x3f800000u),
                                   __uint_as_float((__float_as_uint(t.y) << 23) + 0x3f800000u)));
}

// 2^x of the c-th of N pairs: the last FMA of them on the FMA pipe, the others on MUFU
template <int N, int FMA, int DEG, bool KEEP_NAN>
__device__ __forceinline__ float2 exp2_mix(int c, float2 x) {
  if (c >= N - FMA) return exp2_fma<DEG, KEEP_NAN>(x);
  return make_float2(ex2(x.x), ex2(x.y));
}

// Two softmax warps of a scheduler take turns with their exponentials, so that the one's run while the
// other's products do; left alone, both end up waiting for the tensor cores, and then for the MUFU unit, at
// the same time. A turn is a hint: it is not waited for longer than a step takes.
__device__ __forceinline__ void turn_wait(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity) && clock64() - t0 < 4096) {
  }
  __syncwarp();
}

// position in a work list of a persistent CTA's r-th item: the lists are sorted by work, and going back and
// forth over the CTAs evens out their sums
__device__ __forceinline__ int64_t list_at(int r) {
  return (int64_t)r * gridDim.x + (r & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// 32 columns of a row, times f, as bf16
__device__ __forceinline__ void store32_bf16(__nv_bfloat16* dst, const float* o, float f) {
#pragma unroll
  for (int k = 0; k < 4; k++)
    reinterpret_cast<uint4*>(dst)[k] =
        make_uint4(pack_bf16(o[8 * k + 0] * f, o[8 * k + 1] * f), pack_bf16(o[8 * k + 2] * f, o[8 * k + 3] * f),
                   pack_bf16(o[8 * k + 4] * f, o[8 * k + 5] * f), pack_bf16(o[8 * k + 6] * f, o[8 * k + 7] * f));
}

}  // namespace tc
}  // namespace pyr
