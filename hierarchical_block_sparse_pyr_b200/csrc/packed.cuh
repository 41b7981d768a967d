// Packed prompts: geometry, plan layout and launchers.
#pragma once

#include "view.cuh"

namespace pyr {

struct PackedGeo {
  int S, T, Hq, Hkv, G, d, dtype;
};

// A plan is three work lists, each sorted by work (longest first), behind a header of kPlanHeader int32
// words of which the first three are the lists' lengths:
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
