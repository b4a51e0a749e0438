// Host helpers of the entry points' argument checks.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "q8d_internal.cuh"

namespace q8d {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && x < y + nb && y < x + na;
}

// Bytes of n cache elements of a type (a whole number of blocks for the
// packed types).
inline long long kv_bytes(int kv_dtype, long long n) {
  switch (kv_dtype) {
    case Q8D_KV_F32: return n * 4;
    case Q8D_KV_F16: return n * 2;
    case Q8D_KV_Q8_0: return n / 32 * 34;
    default: return n / 32 * 18;
  }
}
inline bool kv_known(int kv_dtype) {
  return kv_dtype == Q8D_KV_F32 || kv_dtype == Q8D_KV_F16 || kv_dtype == Q8D_KV_Q8_0 ||
         kv_dtype == Q8D_KV_Q4;
}
inline bool kv_packed(int kv_dtype) { return kv_dtype == Q8D_KV_Q8_0 || kv_dtype == Q8D_KV_Q4; }

}  // namespace q8d
