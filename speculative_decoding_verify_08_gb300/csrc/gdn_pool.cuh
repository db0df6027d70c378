// gdn_pool.cuh -- the gated delta rule over a pool of states: what its token
// kernel (gdn_step.cu) and its chunk kernel (gdn_chunk.cu) share.
#pragma once

#include "paged.cuh"

namespace sv {
namespace gdn {

constexpr int MAX_POOL_B = 65535;

// Rows of a call: the sequence's own (row offsets cu, or `M` each) and, before
// them, those of the tape that it accepted.
struct PoolParams {
  sv_states states;
  const int *slots;
  sv_rows tk, tv, q, k, v, o;
  const float *tg, *tb, *g, *b;
  const int *n_replay;  // NULL: no tape
  const int *cu;        // NULL: M rows each
  unsigned *err;
  int B, T, M, tape_M, Hk, Hv, dv;
  int commit;  // the rows after the tape go into the state too
  int o_f32;
  int stage;   // tokens held in shared memory at a time
};

// The state of sequence b: its slot, or -1 (starts from zeros, not kept).
__device__ __forceinline__ int slot_of(const PoolParams &P, int b, bool report) {
  const int s = P.slots[b];
  if (s >= P.states.num_slots) {
    if (report) atomicOr(P.err, ERR_INDEX);
    return -1;
  }
  return s;
}

// First row and rows of sequence b; no rows if its offsets are out of order or range.
__device__ __forceinline__ int2 rows_of(const PoolParams &P, int b, bool report) {
  if (!P.cu) return make_int2(b * P.M, P.M);
  const int r0 = P.cu[b], r1 = P.cu[b + 1];
  if (r0 < 0 || r1 < r0 || r1 > P.T) {
    if (report) atomicOr(P.err, ERR_INDEX);
    return make_int2(0, 0);
  }
  return make_int2(r0, r1 - r0);
}

inline sv_status check_states(const sv_states *s, int Hv, int dk, int dv) {
  if (!s || !s->ptr || !paged::aligned(s->ptr, 16) || s->num_slots < 1) return SV_ERR_INVALID_ARG;
  const int64_t one = (int64_t)Hv * dv * dk;
  if (s->slot_stride < 0 || s->slot_stride % 4 != 0) return SV_ERR_INVALID_ARG;
  if (s->num_slots > 1 && s->slot_stride < one) return SV_ERR_INVALID_ARG;
  if (s->num_slots > 0x7fffffffLL || s->slot_stride > ((int64_t)1 << 40)) return SV_ERR_UNSUPPORTED;
  return SV_OK;
}

// The token kernel (gdn_step.cu).
sv_status launch_tokens(PoolParams &P, int dk, cudaStream_t s);

}  // namespace gdn
}  // namespace sv
