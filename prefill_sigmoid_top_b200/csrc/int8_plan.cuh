// What the int8 expert products read of a plan.  The plan is the caller's: one of another shape, or one whose making met
// an expert id out of range, must not move a read or a store out of the buffers.  Counts are held to the slots that
// there are and rows to the plan's capacity; what falls outside sets the error word and is left out.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moe {

// Tokens of expert e.
__device__ __forceinline__ int plan_count(const Int8GemmArgs& args, int e) {
  const int n = args.counts[e];
  const int held = min(max(n, 0), args.M * args.top_k);
  if (held != n) set_error(args.err, kErrInvalidInput);
  return held;
}

// Slot of plan row r, or -1: a row outside the plan, or a slot that there is not.
__device__ __forceinline__ int plan_slot(const Int8GemmArgs& args, int r) {
  if (static_cast<unsigned>(r) >= static_cast<unsigned>(args.cap)) return -1;
  const int id = args.sorted_ids[r];
  return id < args.M * args.top_k ? id : -1;
}

}  // namespace moe
