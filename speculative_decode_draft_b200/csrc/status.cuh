// Device status bits and the way kernels report them.
#pragma once

#include <stdint.h>

namespace wmtp {

// Status bits (mirror include/wmtp.h and include/wmtp_step.h).
constexpr int kDevPageOob = 0x1;
constexpr int kDevLenOob = 0x2;
constexpr int kDevRingState = 0x4;
constexpr int kDevUndoFull = 0x8;
constexpr int kDevTimeout = 0x10;
constexpr int kDevPool = 0x40;
constexpr int kDevLogits = 0x80;
constexpr int kDevTokenOob = 0x100;

__device__ __forceinline__ void set_status(int32_t* status, int bits) {
  if (status != nullptr) atomicOr(status, bits);
}

}  // namespace wmtp
