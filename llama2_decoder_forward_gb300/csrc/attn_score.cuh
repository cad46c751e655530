// Pieces shared by the attention kernels with capped or biased scores: a
// document's rows, a decode row's last key, the cap, how partial results are merged.
#pragma once

#include "common.cuh"

namespace llgb {

// Document b's rows [lo, lo + n) of the packed n_rows; bounds outside
// [0, n_rows] or decreasing are flagged and cut to what exists.
__device__ __forceinline__ void doc_rows(const int32_t* cu, int b, int n_rows, uint32_t* status,
                                         int& lo, int& n) {
  const int a = cu[b], e = cu[b + 1];
  lo = min(max(a, 0), n_rows);
  const int hi = min(max(e, lo), n_rows);
  n = hi - lo;
  if (lo != a || hi != e) flag(status, LLAMA_FLAG_POS_RANGE);
}

// The position that a decode row attends up to: one past the limit (flagged by the
// caller) attends the keys in range, as the last one does; the distance bias then
// counts from there, which shifts all scores of the row alike. -1: no keys.
__device__ __forceinline__ int key_position(int pos, int key_limit) {
  return max(min(pos, key_limit - 1), -1);
}

// The maximum that a partial result of sum l is merged with: a maximum passes over
// NaN scores, and without a finite one beside them the part would count as
// empty, so a NaN sum takes part as +inf, which the merge turns into NaN.
__device__ __forceinline__ float merge_max(float m, float l) { return l != l ? INFINITY : m; }

// tanh(y) = y R(y^2): weighted least-squares fits of smallest relative error
// with 3 coefficients for |y| <= 1/4, 4 for 1/2 and 6 for 1 (below 7e-7 each,
// evaluated in fp32).
constexpr float kTanh[13] = {
    0.9999995827674866f, -0.33321908116340637f, 0.12841613590717316f,
    0.999999463558197f, -0.33326318860054016f, 0.13190296292304993f, -0.04440222680568695f,
    0.9999994039535522f, -0.3332904279232025f, 0.13281433284282684f, -0.051605671644210815f,
    0.016743114218115807f, -0.0030670599080622196f};

}  // namespace llgb
