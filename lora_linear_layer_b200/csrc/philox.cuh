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

struct DropState {
  uint32_t k0, k1, o0, o1;
  uint32_t thr_hi;      // thr << 16
};

// Reads the seed and offset (after the kernel's dependency wait).
__device__ __forceinline__ DropState drop_load(const DropArgs& d) {
  const uint64_t seed = d.rng[0], off = d.rng[1];
  return DropState{uint32_t(seed), uint32_t(seed >> 32), uint32_t(off), uint32_t(off >> 32), d.thr << 16};
}

__device__ __forceinline__ uint4 philox4x32_7(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                              uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t a = uint64_t(c0) * 0xD2511F53u, b = uint64_t(c2) * 0xCD9E8D57u;
    const uint32_t n0 = uint32_t(b >> 32) ^ c1 ^ k0, n2 = uint32_t(a >> 32) ^ c3 ^ k1;
    c1 = uint32_t(b);
    c3 = uint32_t(a);
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The random block of the 8 elements (row, 8 c8 .. 8 c8 + 7).
__device__ __forceinline__ uint4 drop_block(const DropState& s, uint32_t c8, uint32_t row) {
  return philox4x32_7(c8, row, s.o0, s.o1, s.k0, s.k1);
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
