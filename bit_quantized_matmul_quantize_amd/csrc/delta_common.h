// What the kernels of the gated delta rule share: their arguments and a
// sequence's range of tokens and place in the state.
#pragma once

#include "bqmm_internal.h"

namespace bqmm {

struct DeltaSeq {
  uint32_t begin, end;  // tokens
  int slot;             // place in the state; -1: starts from zeros, and the end is not kept
  bool fresh;           // starts from zeros
};

// The token ranges come from the device, so they are held to the arrays here:
// a range outside [0, tokens) is cut off, one that runs backwards is empty.
__device__ __forceinline__ DeltaSeq delta_sequence(const DeltaArgs &a, uint32_t seq) {
  DeltaSeq s;
  const int b = a.starts[seq], e = a.starts[seq + 1u];
  s.begin = min((uint32_t)max(b, 0), a.tokens);
  s.end = max(min((uint32_t)max(e, 0), a.tokens), s.begin);
  const int slot = a.slots ? a.slots[seq] : (int)seq;
  s.slot = slot >= 0 && (uint32_t)slot < a.state_slots ? slot : -1;
  s.fresh = a.fresh != nullptr && a.fresh[seq] != 0u;
  return s;
}

}  // namespace bqmm
