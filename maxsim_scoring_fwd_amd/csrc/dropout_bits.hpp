// Dropout's random bits (include/maxsim.h, maxsim_dropout): Philox4x32 (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) with 7 rounds, the fewest that the
// paper found to pass every statistical test. A block of 128 bits serves 8 entries of a row, 16
// bits each, so a mask costs some 10 instructions an entry and is made again wherever it is
// needed: it is never stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace maxsim {

constexpr int DROP_ROUNDS = 7;
constexpr int DROP_CHUNK = 8;  // entries of a block

struct DropArgs {
  const int64_t *rng;  // key and step, on the device; NULL: no dropout
  uint32_t call;
  uint32_t least;      // an entry is kept where its 16 bits are not below
  float up;            // what is kept is multiplied by this
};

// Host side: p in steps of 2^-16, so that what is kept is scaled by its true rate.
inline DropArgs drop_args(double p, const int64_t *rng, int call) {
  DropArgs a;
  a.least = (uint32_t)__builtin_rint(p * 65536.0);
  a.rng = a.least ? rng : nullptr;
  a.call = (uint32_t)call;
  a.up = a.least < 65536 ? (float)(65536.0 / (double)(65536 - a.least)) : 0.0f;
  return a;
}

// The generator's state: the same for every thread of a launch.
struct DropKey {
  uint32_t k0, k1, step;
  __device__ __forceinline__ void load(const int64_t *rng) {
    const uint64_t k = (uint64_t)rng[0];
    k0 = __builtin_amdgcn_readfirstlane((uint32_t)k);
    k1 = __builtin_amdgcn_readfirstlane((uint32_t)(k >> 32));
    step = __builtin_amdgcn_readfirstlane((uint32_t)rng[1]);
  }
};

// The bits of a block: 16 for each of its 8 entries.
struct DropBits {
  uint32_t w[4];
  __device__ __forceinline__ void make(const DropKey &key, const DropArgs &a, uint64_t block) {
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = key.step, c3 = a.call;
    uint32_t k0 = key.k0, k1 = key.k1;
    constexpr int XOR3 = 0x96;  // truth table of a ^ b ^ c
#pragma unroll
    for (int r = 0; r < DROP_ROUNDS; r++) {
      const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
      c0 = __builtin_amdgcn_bitop3_b32((uint32_t)(p1 >> 32), c1, k0, XOR3);
      c2 = __builtin_amdgcn_bitop3_b32((uint32_t)(p0 >> 32), c3, k1, XOR3);
      c1 = (uint32_t)p1;
      c3 = (uint32_t)p0;
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
  }
  // x * up where entry e (a constant) is kept, else 0.
  __device__ __forceinline__ float apply(const DropArgs &a, int e, float x) const {
#pragma clang fp contract(off)  // the product is rounded, whatever it is added to
    const uint32_t u = e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu;
    return u >= a.least ? x * a.up : 0.0f;
  }
};

}  // namespace maxsim
