// Counter-based random bits: Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011).  The four words of a
// counter are a bijection of it under the key, so any element's bits come
// from its index alone: nothing is stored between forward and backward.
#pragma once

#include "common.hpp"

namespace dlrm {

struct DropState {
  uint64_t seed, offset;
};
__device__ __forceinline__ DropState drop_state(const int64_t* rng) {
  return DropState{(uint64_t)rng[0], (uint64_t)rng[1]};
}

// the four words of counter (offset + i, 0) under the key `seed`
__device__ __forceinline__ uint4 philox(const DropState& s, uint64_t i) {
  const uint64_t c = s.offset + i;
  uint32_t x0 = (uint32_t)c, x1 = (uint32_t)(c >> 32), x2 = 0u, x3 = 0u;
  uint32_t k0 = (uint32_t)s.seed, k1 = (uint32_t)(s.seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * x0, b = (uint64_t)0xCD9E8D57u * x2;
    x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
    x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
    x1 = (uint32_t)b;
    x3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(x0, x1, x2, x3);
}

// bit j: element 8 i + j is kept (its 16-bit field is at least cut)
__device__ __forceinline__ uint32_t keep8(const DropState& s, uint64_t i, uint32_t cut) {
  const uint4 w = philox(s, i);
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m |= (uint32_t)((x[j] & 0xffffu) >= cut) << (2 * j);
    m |= (uint32_t)((x[j] >> 16) >= cut) << (2 * j + 1);
  }
  return m;
}

inline uint32_t drop_cut(float p) { return (uint32_t)(p * 65536.0 + 0.5); }
inline float drop_factor(uint32_t cut) { return cut < 65536u ? 65536.f / (float)(65536u - cut) : 0.f; }

}  // namespace dlrm
