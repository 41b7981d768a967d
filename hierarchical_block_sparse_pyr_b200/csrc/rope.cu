// Rotary positions: y = scale * R(p * w_i) x for every pair i of a head's first `rot` elements, or the
// transposed map (the gradient). One pass, bound by HBM: 2 * B * (Hq + Hkv) * N * d elements move.
//
// The angle depends on the position and the pair, not on the head, so a thread owns one 16-byte chunk of
// pairs of one token, takes its sines and cosines once and walks over several heads with them. Angles: the
// product of the position and the pair's turns per position in double (at position 10^6 a product in single
// precision would be off by 2^-24 * 10^6 radians), reduced to a fraction of a turn in [-1/2, 1/2], and only
// that fraction goes to single precision.
// Measured: 32K tokens, 32 heads of 128, bf16: 81.8 us, 6.56 TB/s (the copy rate); 8194 tokens, 40 heads of 64 of
// which half rotates, fp32, token-major: 29 us, 5.8 TB/s.
#include <math.h>

#include "view.cuh"

namespace pyr {

namespace {

struct RopeArgs {
  View q, k, qo, ko;
  const int32_t* pos;
  int64_t pos_stride;
  int pos_offset;
  int B, Hq, Hkv, N, d, rot, inverse;
  int copy_q, copy_k;  // pass the elements behind rot through (not needed in place)
  int heads_per_thread;
  float scale;
  double turns[64];  // freq / (2 pi)
};

__device__ __forceinline__ void rope_angle(const RopeArgs& a, int pos, int pair, float* c, float* s) {
  const double x = (double)pos * a.turns[pair];
  const float r = (float)(x - rint(x));
  float sn, cs;
  sincospif(2.f * r, &sn, &cs);
  *c = cs * a.scale;
  *s = (a.inverse ? -sn : sn) * a.scale;
}

template <typename T>
struct Vec;  // a 16-byte chunk as floats
template <>
struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Whole 16-byte chunks. Item x of a token: rotated items first (ROPE_HALF: the chunk pair (x, x + rot/2);
// interleaved: one chunk), then the chunks behind rot.
template <typename T, int LAYOUT, int HPT>
__global__ void __launch_bounds__(256) rope_vec_kernel(RopeArgs a, int items, int rot_items) {
  constexpr int E = Vec<T>::E;
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t n64 = id / items;
  if (n64 >= a.N) return;
  const int x = (int)(id - n64 * items), n = (int)n64, b = blockIdx.z;
  const int h0 = blockIdx.y * HPT, hn = min(HPT, a.Hq + a.Hkv - h0);
  const bool copy = x >= rot_items;
  const int e0 = copy ? a.rot + (x - rot_items) * E : x * E;
  const int e1 = e0 + a.rot / 2;  // ROPE_HALF partner

  uint4 v0[HPT], v1[HPT];
#pragma unroll
  for (int i = 0; i < HPT; i++) {
    if (i >= hn) break;
    const int h = h0 + i;
    const T* src = h < a.Hq ? view_at<T>(a.q, b, h, n) : view_at<T>(a.k, b, h - a.Hq, n);
    v0[i] = __ldcs(reinterpret_cast<const uint4*>(src + e0));
    if (LAYOUT == ROPE_HALF && !copy) v1[i] = __ldcs(reinterpret_cast<const uint4*>(src + e1));
  }
  if (copy) {
#pragma unroll
    for (int i = 0; i < HPT; i++) {
      if (i >= hn) break;
      const int h = h0 + i;
      if (h < a.Hq ? !a.copy_q : !a.copy_k) continue;
      T* dst = h < a.Hq ? view_at<T>(a.qo, b, h, n) : view_at<T>(a.ko, b, h - a.Hq, n);
      *reinterpret_cast<uint4*>(dst + e0) = v0[i];
    }
    return;
  }
  const int pos = a.pos ? a.pos[b * a.pos_stride + n] : a.pos_offset + n;
  constexpr int NP = LAYOUT == ROPE_HALF ? E : E / 2;  // pairs of this item
  float c[NP], s[NP];
#pragma unroll
  for (int i = 0; i < NP; i++) rope_angle(a, pos, x * NP + i, c + i, s + i);
#pragma unroll
  for (int i = 0; i < HPT; i++) {
    if (i >= hn) break;
    const int h = h0 + i;
    T* dst = h < a.Hq ? view_at<T>(a.qo, b, h, n) : view_at<T>(a.ko, b, h - a.Hq, n);
    float f[E];
    Vec<T>::unpack(v0[i], f);
    if (LAYOUT == ROPE_HALF) {
      float g[E];
      Vec<T>::unpack(v1[i], g);
#pragma unroll
      for (int j = 0; j < E; j++) {
        const float u = f[j], w = g[j];
        f[j] = u * c[j] - w * s[j];
        g[j] = u * s[j] + w * c[j];
      }
      *reinterpret_cast<uint4*>(dst + e0) = Vec<T>::pack(f);
      *reinterpret_cast<uint4*>(dst + e1) = Vec<T>::pack(g);
    } else {
#pragma unroll
      for (int j = 0; j < E / 2; j++) {
        const float u = f[2 * j], w = f[2 * j + 1];
        f[2 * j] = u * c[j] - w * s[j];
        f[2 * j + 1] = u * s[j] + w * c[j];
      }
      *reinterpret_cast<uint4*>(dst + e0) = Vec<T>::pack(f);
    }
  }
}

// Any even rot, one element pair (or one element behind rot) per thread and head: for a rot whose chunks
// would straddle 16-byte boundaries (rot / 2, or rot when interleaved, not a whole number of chunks).
template <typename T>
__global__ void __launch_bounds__(256) rope_pair_kernel(RopeArgs a, int layout, int items) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t n64 = id / items;
  if (n64 >= a.N) return;
  const int x = (int)(id - n64 * items), n = (int)n64, b = blockIdx.z;
  const int np = a.rot / 2;
  const int h0 = blockIdx.y * a.heads_per_thread, h1 = min(h0 + a.heads_per_thread, a.Hq + a.Hkv);
  float c = 1.f, s = 0.f;
  if (x < np) rope_angle(a, a.pos ? a.pos[b * a.pos_stride + n] : a.pos_offset + n, x, &c, &s);
  for (int h = h0; h < h1; h++) {
    const T* src = h < a.Hq ? view_at<T>(a.q, b, h, n) : view_at<T>(a.k, b, h - a.Hq, n);
    T* dst = h < a.Hq ? view_at<T>(a.qo, b, h, n) : view_at<T>(a.ko, b, h - a.Hq, n);
    if (x >= np) {
      if (h < a.Hq ? a.copy_q : a.copy_k) dst[np + x] = src[np + x];  // element rot + (x - np)
      continue;
    }
    const int i = layout == ROPE_HALF ? x : 2 * x, j = layout == ROPE_HALF ? x + np : 2 * x + 1;
    const float u = to_f32(src[i]), w = to_f32(src[j]);
    dst[i] = (T)(u * c - w * s);
    dst[j] = (T)(u * s + w * c);
  }
}

template <typename T, int LAYOUT, int HPT>
void launch_vec(const RopeArgs& a, cudaStream_t st) {
  constexpr int E = Vec<T>::E;
  const int rot_items = LAYOUT == ROPE_HALF ? a.rot / 2 / E : a.rot / E;
  const int items = rot_items + ((a.copy_q || a.copy_k) ? (a.d - a.rot) / E : 0);
  const dim3 grid((unsigned)(((int64_t)a.N * items + 255) / 256), (a.Hq + a.Hkv + HPT - 1) / HPT, a.B);
  rope_vec_kernel<T, LAYOUT, HPT><<<grid, 256, 0, st>>>(a, items, rot_items);
}

template <typename T, int LAYOUT>
void launch_layout(const RopeArgs& a, cudaStream_t st) {
  // few tokens: one head a thread, so that the heads spread over the GPU; else four share their angles (32K
  // tokens, 32 heads of 128, bf16: 81.8 us; two 100.5, eight 83.4)
  const int64_t threads = (int64_t)a.B * a.N * (a.Hq + a.Hkv) * a.d / (2 * Vec<T>::E);
  if (threads <= 148 * 2048)
    launch_vec<T, LAYOUT, 1>(a, st);
  else
    launch_vec<T, LAYOUT, 4>(a, st);
}

template <typename T>
cudaError_t launch_rope(RopeArgs a, int layout, cudaStream_t st) {
  constexpr int E = Vec<T>::E;
  if ((layout == ROPE_HALF ? a.rot / 2 : a.rot) % E == 0) {
    if (layout == ROPE_HALF)
      launch_layout<T, ROPE_HALF>(a, st);
    else
      launch_layout<T, ROPE_INTERLEAVED>(a, st);
  } else {
    const int items = a.rot / 2 + ((a.copy_q || a.copy_k) ? a.d - a.rot : 0);
    a.heads_per_thread = 8;
    const dim3 grid((unsigned)(((int64_t)a.N * items + 255) / 256), (a.Hq + a.Hkv + 7) / 8, a.B);
    rope_pair_kernel<T><<<grid, 256, 0, st>>>(a, layout, items);
  }
  return cudaGetLastError();
}

bool same_view(const View& a, const View& b) {
  return a.data == b.data && a.batch == b.batch && a.head == b.head && a.row == b.row;
}

}  // namespace

}  // namespace pyr

extern "C" {

int rope_spec_init(rope_spec* spec, int d, int rot, int layout, double base, int scaling, double factor,
                   int trained) {
  if (!spec || (d != 64 && d != 128) || rot < 2 || rot > d || rot % 2 ||
      (layout != ROPE_HALF && layout != ROPE_INTERLEAVED) || scaling < ROPE_SCALE_NONE || scaling > ROPE_SCALE_YARN ||
      !(base > 1.0) || !(base < 1e300))
    return PYR_EINVAL;
  if (scaling != ROPE_SCALE_NONE && (!(factor >= 1.0) || !(factor < 1e30))) return PYR_EINVAL;
  if (scaling == ROPE_SCALE_NTK && rot < 4) return PYR_EINVAL;
  if (scaling == ROPE_SCALE_YARN && (trained < 1 || rot < 4)) return PYR_EINVAL;
  spec->d = d;
  spec->rot = rot;
  spec->layout = layout;
  spec->reserved = 0;
  spec->scale = 1.0;
  if (scaling == ROPE_SCALE_NTK) base *= pow(factor, rot / (rot - 2.0));
  double lo = 0.0, hi = 0.0;
  if (scaling == ROPE_SCALE_YARN) {
    // pair index at which the trained length makes 32 turns, and one turn
    const double two_pi = 6.283185307179586476925286766559;
    lo = floor(rot * log(trained / (32.0 * two_pi)) / (2.0 * log(base)));
    hi = ceil(rot * log(trained / two_pi) / (2.0 * log(base)));
    if (lo < 0.0) lo = 0.0;
    if (hi > rot - 1.0) hi = rot - 1.0;
    if (hi - lo < 0.001) hi = lo + 0.001;
    spec->scale = 0.1 * log(factor) + 1.0;
  }
  for (int i = 0; i < 64; i++) {
    double f = i < rot / 2 ? pow(base, -2.0 * i / rot) : 0.0;
    if (scaling == ROPE_SCALE_LINEAR) f /= factor;
    if (scaling == ROPE_SCALE_YARN) {
      double r = (i - lo) / (hi - lo);
      r = r < 0.0 ? 0.0 : (r > 1.0 ? 1.0 : r);
      f = f / factor * r + f * (1.0 - r);
    }
    spec->freq[i] = f;
  }
  return PYR_OK;
}

int rope_apply(const rope_spec* spec, int B, int Hq, int Hkv, int N, int dtype, const pyr_view* Q, const pyr_view* K,
               const int32_t* pos, int64_t pos_stride, int pos_offset, const pyr_view* Qo, const pyr_view* Ko,
               int inverse, int* dev_status, void* stream) {
  (void)dev_status;
  if (!spec || B <= 0 || N <= 0 || Hq < 0 || Hkv < 0 || (int64_t)Hq + Hkv <= 0) return PYR_EINVAL;
  if (dtype != PYR_F32 && dtype != PYR_BF16) return PYR_EUNSUPPORTED;
  if (spec->d != 64 && spec->d != 128) return PYR_EUNSUPPORTED;
  if (spec->rot < 2 || spec->rot > spec->d || spec->rot % 2 ||
      (spec->layout != ROPE_HALF && spec->layout != ROPE_INTERLEAVED) || !(fabs(spec->scale) < INFINITY))
    return PYR_EINVAL;
  for (int i = 0; i < spec->rot / 2; i++)
    if (!(fabs(spec->freq[i]) <= 1e9)) return PYR_EINVAL;
  if (B > 65535 || (int64_t)Hq + Hkv > 65535 || (int64_t)N * spec->d > ((int64_t)1 << 38)) return PYR_EUNSUPPORTED;
  if ((Hq > 0) != (Q != nullptr) || (Hq > 0) != (Qo != nullptr) || (Hkv > 0) != (K != nullptr) ||
      (Hkv > 0) != (Ko != nullptr))
    return PYR_EINVAL;
  pyr::RopeArgs a = {};
  if (Hq > 0 && (!pyr::check_view(Q, B, Hq, N, spec->d, dtype, false, &a.q) ||
                 !pyr::check_view(Qo, B, Hq, N, spec->d, dtype, true, &a.qo)))
    return PYR_EINVAL;
  if (Hkv > 0 && (!pyr::check_view(K, B, Hkv, N, spec->d, dtype, false, &a.k) ||
                  !pyr::check_view(Ko, B, Hkv, N, spec->d, dtype, true, &a.ko)))
    return PYR_EINVAL;
  if (pos ? (!pyr::aligned4(pos) || pos_stride < 0 || (pos_stride > 0 && pos_stride < N && B > 1))
          : (int64_t)pos_offset + N - 1 > INT32_MAX)
    return PYR_EINVAL;
  a.pos = pos;
  a.pos_stride = pos_stride;
  a.pos_offset = pos_offset;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.N = N;
  a.d = spec->d;
  a.rot = spec->rot;
  a.inverse = inverse != 0;
  a.copy_q = Hq > 0 && spec->rot < spec->d && !pyr::same_view(a.q, a.qo);
  a.copy_k = Hkv > 0 && spec->rot < spec->d && !pyr::same_view(a.k, a.ko);
  a.scale = (float)spec->scale;
  for (int i = 0; i < spec->rot / 2; i++) a.turns[i] = spec->freq[i] / 6.283185307179586476925286766559;
  const cudaError_t e = dtype == PYR_F32 ? pyr::launch_rope<float>(a, spec->layout, (cudaStream_t)stream)
                                         : pyr::launch_rope<__nv_bfloat16>(a, spec->layout, (cudaStream_t)stream);
  return e == cudaSuccess ? PYR_OK : PYR_ECUDA;
}

}  // extern "C"
