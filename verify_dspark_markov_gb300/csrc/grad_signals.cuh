// Which slice and which mbarrier a row of the distillation gradient's pipeline
// uses (distill.cu).  Rows are numbered within their cluster.
//
// A slice is used by every kSlices-th row.  Those rows are of either parity in
// turn, and the rows of one parity are taken by one warp A, so the slice's
// copies are announced on two mbarriers, one for either warp: a warp that waits
// for alternate phases of a barrier can be two phases behind, and a wait for a
// phase's parity returns at once when the phase two before it is the one in
// flight.  Row n and row n + kFull are of one parity: the warp that waits for
// one has waited for the other.
//
// What orders row n + kSlices after row n: its barrier's phase ends only after
// warp D has arrived on it, and D does so once row n's gradient is stored.
#pragma once

#include <stdint.h>

namespace dspark {

constexpr int kSlices = 3;
constexpr int kFull = 2 * kSlices;  // mbarriers of copies
static_assert(kFull % 2 == 0, "the rows of a barrier are of one parity");

__host__ __device__ inline int slice_of(int n) { return n % kSlices; }
__host__ __device__ inline int full_of(int n) { return n % kFull; }
__host__ __device__ inline uint32_t full_parity(int n) { return static_cast<uint32_t>(n / kFull) & 1u; }

}  // namespace dspark
