// Strided [batch][head][row][d] operands: the device-side form and the host-side checks.
#pragma once

#include "pyr_common.cuh"

namespace pyr {

struct View {
  void* data;
  int64_t batch, head, row;  // strides in elements
};

template <typename T>
__device__ __forceinline__ T* view_at(const View& v, int b, int h, int64_t n) {
  return reinterpret_cast<T*>(v.data) + (b * v.batch + h * v.head + n * v.row);
}

// Overlap of two kernels of a stream: the second may start once every block of the first has called
// grid_launch (or has ended), and waits in grid_wait until the first has ended and its writes are visible.
__device__ __forceinline__ void grid_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch a kernel that may start early in this sense.
template <typename... P, typename... A>
inline cudaError_t launch_early(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
inline int elt_bytes(int dtype) { return dtype == PYR_F32 ? 4 : 2; }

// Check a view of extents B x H x N x d and copy it to `out`; the stride of an axis with one entry is
// never used and becomes d. written: the rows must not overlap, which is checked by nesting the axes by
// stride. False: the entry point returns PYR_EINVAL.
inline bool check_view(const pyr_view* v, int B, int H, int64_t N, int d, int dtype, bool written, View* out) {
  if (!v || !v->data || !aligned16(v->data)) return false;
  const int64_t ext[3] = {B, H, N}, given[3] = {v->batch, v->head, v->row};
  int64_t st[3];
  const int64_t unit = 16 / elt_bytes(dtype);
  for (int i = 0; i < 3; i++) {
    st[i] = ext[i] > 1 ? given[i] : d;
    if (st[i] < d || st[i] % unit || st[i] >= ((int64_t)1 << 38)) return false;
  }
  if (written) {
    int o[3] = {0, 1, 2};
    for (int i = 0; i < 2; i++)
      for (int j = 0; j < 2 - i; j++)
        if (st[o[j]] > st[o[j + 1]]) {
          const int t = o[j];
          o[j] = o[j + 1];
          o[j + 1] = t;
        }
    int64_t span = d;  // elements from the first to behind the last of the axes seen so far
    for (int i = 0; i < 3; i++) {
      if (ext[o[i]] <= 1) continue;
      if (st[o[i]] < span) return false;
      span += (ext[o[i]] - 1) * st[o[i]];
    }
  }
  out->data = v->data;
  out->batch = st[0];
  out->head = st[1];
  out->row = st[2];
  return true;
}

}  // namespace pyr
