// philox.cuh - the adapter dropout's mask: a counter-based generator, so the
// mask is computed wherever it is needed and never stored.
//
// Philox4x32 with 7 rounds (Salmon, Moraes, Dror, Shaw: "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011, where 7 is the fewest rounds that
// pass the paper's statistical batteries and 10 the default margin; a mask
// needs no margin, and the three rounds less are a third of its cost).
// Element (i, k) of X takes 16 bits: the block with
//     counter = (k / 8, i, offset low, offset high),  key = (seed low, high)
// gives 8 lanes of 16 bits (word 0 low half, word 0 high half, word 1 ...),
// and lane k % 8 keeps the element when it is >= thr = round(65536 p).  16
// bits place p on a grid of 2^-16 (the kept values are scaled by the exact
// 65536 / (65536 - thr)) and let one block serve one 16-byte chunk of bf16.
#pragma once

#include "common.cuh"

namespace lora {

struct DropArgs {
  const uint64_t* rng;  // device: {seed, offset}; NULL = no dropout
  uint32_t thr;         // keep when the 16-bit lane is >= thr, thr in [0, 65535]
  float inv_keep;       // 65536 / (65536 - thr)
};

// The generator's constants of one call: the round keys (kept in registers;
// stepping them in every block costs two additions a round) and the first
// round's product of the offset word.
struct DropState {
  uint32_t k0[7], k1[7];
  uint32_t o_hi, o_lo;  // words of offset low * 0xCD9E8D57
  uint32_t o1;
  uint32_t thr_hi;      // thr << 16
};

// Reads the seed and offset (after the kernel's dependency wait).
__device__ __forceinline__ DropState drop_load(const DropArgs& d) {
  const uint64_t seed = d.rng[0], off = d.rng[1];
  DropState s;
#pragma unroll
  for (uint32_t i = 0; i < 7; ++i) {
    s.k0[i] = uint32_t(seed) + i * 0x9E3779B9u;
    s.k1[i] = uint32_t(seed >> 32) + i * 0xBB67AE85u;
  }
  const uint64_t b = (off & 0xFFFFFFFFu) * 0xCD9E8D57u;
  s.o_hi = uint32_t(b >> 32);
  s.o_lo = uint32_t(b);
  s.o1 = uint32_t(off >> 32);
  s.thr_hi = d.thr << 16;
  return s;
}

// The random block of the 8 elements (row, 8 c8 .. 8 c8 + 7).
__device__ __forceinline__ uint4 drop_block(const DropState& s, uint32_t c8, uint32_t row) {
  const uint64_t a0 = uint64_t(c8) * 0xD2511F53u;
  uint32_t c0 = s.o_hi ^ row ^ s.k0[0], c1 = s.o_lo;
  uint32_t c2 = uint32_t(a0 >> 32) ^ s.o1 ^ s.k1[0], c3 = uint32_t(a0);
#pragma unroll
  for (int i = 1; i < 7; ++i) {
    const uint64_t a = uint64_t(c0) * 0xD2511F53u, b = uint64_t(c2) * 0xCD9E8D57u;
    c0 = uint32_t(b >> 32) ^ c1 ^ s.k0[i];
    c2 = uint32_t(a >> 32) ^ c3 ^ s.k1[i];
    c1 = uint32_t(b);
    c3 = uint32_t(a);
  }
  return make_uint4(c0, c1, c2, c3);
}

// Zero the dropped ones of two bf16 values packed in `x` (`w` holds their
// two lanes).  A select, not a product: a dropped infinity or NaN is gone.
__device__ __forceinline__ uint32_t drop_pair(uint32_t x, uint32_t w, uint32_t thr_hi) {
  if ((w << 16) < thr_hi) x &= 0xFFFF0000u;
  if (w < thr_hi) x &= 0x0000FFFFu;
  return x;
}

__device__ __forceinline__ uint4 drop_bf16x8(uint4 x, uint4 w, uint32_t thr_hi) {
  return make_uint4(drop_pair(x.x, w.x, thr_hi), drop_pair(x.y, w.y, thr_hi), drop_pair(x.z, w.z, thr_hi),
                    drop_pair(x.w, w.w, thr_hi));
}

}  // namespace lora
