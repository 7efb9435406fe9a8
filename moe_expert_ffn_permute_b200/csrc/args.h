// args.h -- what the plan-free calls (row operators, MXFP4 operators) check of
// their arguments on the host: element types, alignment, overlap.
#pragma once
#include <cstddef>
#include <cstdint>

#include "../../include/moe.h"

namespace moe {

inline int elem_bytes(int dtype) { return dtype == MOE_T_FP32 ? 4 : 2; }
inline bool elem_ok(int dtype) {
  return dtype == MOE_T_BF16 || dtype == MOE_T_FP16 || dtype == MOE_T_FP32;
}

// Most slots of a token the row operators and the quantiser take: their loops
// step past k by up to a group of slots.
constexpr int kMaxSlotsPerToken = 1 << 24;

// A buffer of a call.  The operators read through the read-only path and in no
// set order, so an output may lie neither in an input nor in another output.
struct Buffer {
  const void* p;
  long long bytes;
  bool out;
};

// Whether an output shares a byte with another buffer (a null one shares none).
template <int kN>
inline bool outputs_overlap(const Buffer (&b)[kN]) {
  for (int i = 0; i < kN; ++i)
    for (int j = i + 1; j < kN; ++j) {
      if ((!b[i].out && !b[j].out) || b[i].p == nullptr || b[j].p == nullptr) continue;
      const auto x = reinterpret_cast<uintptr_t>(b[i].p), y = reinterpret_cast<uintptr_t>(b[j].p);
      if (x < y + static_cast<uintptr_t>(b[j].bytes) && y < x + static_cast<uintptr_t>(b[i].bytes))
        return true;
    }
  return false;
}

inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace moe
