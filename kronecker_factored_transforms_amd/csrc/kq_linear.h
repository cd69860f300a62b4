// Device helpers shared by the operators around a linear layer (kq_norm.hip, kq_grouped.hip,
// kq_adapter.hip).
#pragma once

#include "kq_common.h"

namespace {

// fp32 -> fp16, round to nearest even, of the fp32 value as it stands: the value is opaque to
// the compiler, which would otherwise fold a preceding product or sum into an instruction that
// rounds its exact result to fp16 at once (one rounding instead of the two that are meant).
__device__ __forceinline__ _Float16 half_rne(float v) {
  asm("" : "+v"(v));
  return (_Float16)v;
}

// 16 zero bytes, for DMA past the end of a row
__device__ __align__(16) const unsigned char kZeros[16] = {};

// The same address, in scalar registers (it is the same in every lane)
__device__ __forceinline__ const unsigned char *uniform(const void *p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const unsigned char *>((uint64_t)hi << 32 | lo);
}

}  // namespace
