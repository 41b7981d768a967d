// Packed prompts: geometry, plan layout and launchers.
#pragma once

#include "view.cuh"

namespace pyr {

struct PackedGeo {
  int S, T, Hq, Hkv, G, d, dtype;
};

// A plan is three work lists, each sorted by work (longest first), behind a header of kPlanHeader int32
// words of which the first three are the lists' lengths and the fourth marks the geometry they are for
// (entries of another shape, or a buffer that holds no plan, would send the kernels out of bounds):
//   kListFwd   row tiles of the forward pass,   work ~ keys up to the tile's end
//   kListQ     row tiles of the dQ kernel,      same
//   kListK     key tiles of the dK/dV kernel,   work ~ rows from the tile's start to the sequence's end
// An entry is (start, end of its sequence, first token of the tile, 0). The tail of the buffer is the
// planner's scratch: tile counts summed over the sequences (S + 1 words).
constexpr int kPlanHeader = 16;
constexpr int kListFwd = 0, kListQ = 1, kListK = 2;

// tokens per tile of a list. fp32: 32 (packed_simt.cu). bf16: 128, and in the forward pass 256 where the two 128-row tiles of
// a CTA come from one head (packed_fwd_tc.cu).
__host__ __device__ inline int packed_tile_rows(const PackedGeo& g, int list) {
  if (g.dtype == PYR_F32) return 32;
  return list == kListFwd && g.G % 2 ? 256 : 128;
}

__host__ __device__ inline int64_t packed_list_cap(const PackedGeo& g, int list) {
  const int rows = packed_tile_rows(g, list);
  return (int64_t)(g.T + rows - 1) / rows + g.S;  // a sequence has at most one tile that is not full
}
// first int32 word of a list
__host__ __device__ inline int64_t packed_list_at(const PackedGeo& g, int list) {
  int64_t at = kPlanHeader;
  for (int i = 0; i < list; i++) at += 4 * packed_list_cap(g, i);
  return at;
}
__host__ __device__ inline int64_t packed_plan_words(const PackedGeo& g) { return packed_list_at(g, 3) + g.S + 1; }

__host__ __device__ inline int packed_plan_mark(const PackedGeo& g) {
  const uint32_t v[7] = {(uint32_t)g.S, (uint32_t)g.T, (uint32_t)g.Hq, (uint32_t)g.Hkv, (uint32_t)g.d, (uint32_t)g.dtype,
                         0x706c616eu};
  uint32_t h = 2166136261u;  // FNV-1a over the words
  for (int i = 0; i < 7; i++) h = (h ^ v[i]) * 16777619u;
  return (int)(h | 1u);
}

// Length of a list, 0 where the plan is not one of this geometry (reported once by the grid).
__device__ __forceinline__ int packed_tiles(const PackedGeo& g, const int32_t* plan, int list, int* status) {
  if (plan[3] != packed_plan_mark(g)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(status, PYR_EBADSEQ);
    return 0;
  }
  return plan[list];
}

struct PackedFwdArgs {
  View q, k, v, o;
  const int32_t* plan;
  float* lse;
  int* status;
};

struct PackedBwdArgs {
  View q, k, v, o, dout, dq, dk, dv;
  const int32_t* plan;
  const float* lse;
  float* delta;
  int* status;
};

cudaError_t launch_packed_plan(const PackedGeo& g, const int32_t* cu, int32_t* plan, int* status, cudaStream_t st);
cudaError_t launch_packed_fwd_simt(const PackedGeo& g, const PackedFwdArgs& a, cudaStream_t st);
cudaError_t launch_packed_fwd_tc(const PackedGeo& g, const PackedFwdArgs& a, cudaStream_t st);
cudaError_t launch_packed_bwd_simt(const PackedGeo& g, const PackedBwdArgs& a, cudaStream_t st);
cudaError_t launch_packed_bwd_tc(const PackedGeo& g, const PackedBwdArgs& a, cudaStream_t st);
// delta = rowsum(dO * O) of the rows of every sequence
cudaError_t launch_packed_delta(const PackedGeo& g, const PackedBwdArgs& a, cudaStream_t st);

}  // namespace pyr
