// fp8.cuh - e4m3 with a power-of-two scale for each block of 128.
//
// A group of values (a 128 x 128 block of a weight; 128 consecutive values
// of one row of an activation or gradient) is held as e4m3 codes q and one
// e8m0 byte b:  value = q 2^(b - 127).  2^(b - 127) is the smallest power of
// two, at least 2^-127, with which the largest magnitude of the group is at
// most 448, the largest e4m3 value; an empty (all zero) group has b = 127.
// The division by a power of two is exact, so a code is the value's only
// rounding (nearest even), and tcgen05.mma applies such scales itself.
// A group that holds an infinity or a NaN gets b = 255, e8m0's NaN: every
// product it enters is NaN, as in the unquantised layer's affected rows.
//
// The two weight kernels move 3 bytes an element and do nothing else of
// weight: memory bound.  One block of 256 threads takes one 128 x 128 block
// in registers (each thread 4 rows of 16 consecutive values: 8 16-byte loads
// in flight), so W is read once, between the maximum and the codes.
#pragma once

#include "common.cuh"

namespace lora {

constexpr int kQBlock = 128;

// Largest magnitudes of packed bf16 pairs; a NaN wins.  The result's sign is
// the xor of the operands' (the form that needs no separate absolute values);
// abs_bf16x2 clears it at the end.
__device__ __forceinline__ uint32_t amax_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t abs_bf16x2(uint32_t v) { return v & 0x7FFF7FFFu; }

__device__ __forceinline__ uint32_t amax_bf16x16(uint4 x, uint4 y) {
  return amax_bf16x2(amax_bf16x2(amax_bf16x2(x.x, x.y), amax_bf16x2(x.z, x.w)),
                     amax_bf16x2(amax_bf16x2(y.x, y.y), amax_bf16x2(y.z, y.w)));
}

// The e8m0 byte of a group whose largest magnitude has these bf16 bits.
// amax = 1.f * 2^x fits under 448 * 2^e = 1.75 * 2^(e + 8) with e = x - 8
// when its fraction is at most .75 (96 of 128), else with e = x - 7: adding
// 31 carries exactly then.  A subnormal bf16 (x < -126) is below
// 448 * 2^-127 in any case.
__device__ __forceinline__ uint32_t e8m0_of_amax(uint32_t amax_bits) {
  const uint32_t b = uint32_t(max(int((amax_bits + 31u) >> 7) - 8, 0));
  return amax_bits >= 0x7F80u ? 255u : amax_bits == 0u ? 127u : b;  // (selects: a branch costs more)
}

// The same for the larger of two packed magnitudes (signs are ignored).
__device__ __forceinline__ uint32_t e8m0_of_pair(uint32_t m) {
  m = abs_bf16x2(m);
  return e8m0_of_amax(max(m & 0xFFFFu, m >> 16));
}

// 2^-(b - 127) as two packed bf16, the factor that values are multiplied by
// (b is at most 247; 1 for the NaN scale).  The product of a bf16 value is
// exact in bf16, except far below the smallest e4m3 value, where the code is
// zero in any case.
__device__ __forceinline__ uint32_t e8m0_inverse(uint32_t b) {
  return b == 255u ? 0x3F803F80u : ((254u - b) << 7) * 0x10001u;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7FC00000u) : b == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

// Two fp32 -> packed e4m3x2 (nearest even; magnitudes are at most 448 here),
// `lo` in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four scaled bf16 (two words) -> four codes.
__device__ __forceinline__ uint32_t quant4(uint32_t a, uint32_t b, uint32_t f) {
  a = mul_bf16x2(a, f);
  b = mul_bf16x2(b, f);
  const uint32_t lo = pack_e4m3x2(bf16lo_to_f32(a), bf16hi_to_f32(a));
  const uint32_t hi = pack_e4m3x2(bf16lo_to_f32(b), bf16hi_to_f32(b));
  return lo | (hi << 16);
}

// 8 consecutive bf16 with the scale's inverse -> 8 codes.
__device__ __forceinline__ uint2 quant8(uint4 x, uint32_t f) {
  return make_uint2(quant4(x.x, x.y, f), quant4(x.z, x.w, f));
}

// Two e4m3 codes (low 16 bits) -> two fp32 (through fp16, which holds every
// e4m3 value).
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(v)));
  float2 f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}\n"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// ---------------------------------------------------- scales of a product ----
//
// tcgen05.mma reads its scales from TMEM as 32 lanes x 4 columns of 32-bit
// words for 128 rows (columns) of a tile: row r is lane r % 32, column r / 32,
// and the four bytes of a word are the scales of four consecutive blocks of
// 128 values of K.  One such "atom" is 512 bytes, 16 a lane.
//   rows of X or dY:    [ceil(K / 512)][ceil(M / 128)] atoms, written by the
//                       pass that rounds them;
//   columns of a tile:  [tile][ceil(K / 512)][2] atoms for the tile's up to
//                       256 columns, laid out from the weight's bytes for
//                       each call (scale_atoms) since a tile's columns need
//                       not begin on a block of 128.

// Byte offset of the scale of (row, block kb of K), `blocks` = ceil(M / 128).
__device__ __forceinline__ size_t scale_atom_offset(int row, int kb, int blocks) {
  return (size_t(kb >> 2) * size_t(blocks) + size_t(row >> 7)) * 512 +
         size_t((row & 31) * 16 + ((row >> 5) & 3) * 4 + (kb & 3));
}

struct ScaleAtomArgs {
  const uint8_t* bytes;   // the weight's scales, or NULL: no atoms to lay out
  uint8_t* atoms;         // [tiles][groups][2][512]
  int32_t tiles, groups;  // of the product
  int32_t bn;             // columns of a tile
  int32_t n_blocks, k_blocks, ld_n, ld_k;  // of `bytes`, along the product's N and K
};

// One warp's share of the column atoms: every `step`-th atom from `item` on.
__device__ __forceinline__ void scale_atoms(const ScaleAtomArgs& a, int item, int step, int lane) {
  for (; item < a.tiles * a.groups * 2; item += step) {
    const int tile = item / (2 * a.groups), g = (item >> 1) % a.groups, half = item & 1;
    // byte lane & 3 of word (lane >> 2) & 3
    const int n = tile * a.bn + 128 * half + 32 * ((lane >> 2) & 3);
    const int nb = imin(n >> 7, a.n_blocks - 1), kb = imin(4 * g + (lane & 3), a.k_blocks - 1);
    uint32_t v = uint32_t(a.bytes[size_t(nb) * size_t(a.ld_n) + size_t(kb) * size_t(a.ld_k)]) << (8 * (lane & 3));
    v |= __shfl_xor_sync(0xffffffffu, v, 1);
    v |= __shfl_xor_sync(0xffffffffu, v, 2);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __shfl_sync(0xffffffffu, v, 4 * i);
    reinterpret_cast<uint4*>(a.atoms)[size_t(item) * 32 + size_t(lane)] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

constexpr int kQuantThreads = 256;

// W[rows, cols] bf16 -> Wq codes (same layout) and Ws[ceil(rows/128),
// ceil(cols/128)] bytes.  cols is a multiple of 16.  Grid: one block for each
// 128 x 128 block of W, columns fastest.
__global__ void __launch_bounds__(kQuantThreads)
    quantize_block_kernel(const uint8_t* W, uint8_t* Wq, uint8_t* Ws, int32_t rows, int32_t cols,
                          int32_t col_blocks) {
  __shared__ uint32_t warp_max[kQuantThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int cb = int(blockIdx.x) % col_blocks, rb = int(blockIdx.x) / col_blocks;
  const int col = cb * kQBlock + int(threadIdx.x & 7u) * 16;
  const int row0 = rb * kQBlock + int(threadIdx.x >> 3);
  uint4 v[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + 32 * i;
    v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
    // (a branch: with clamped addresses and selects behind them 14336 x 4096
    // takes 33 us instead of 26.5, 32768 x 8192 136 instead of 120)
    if (row < rows && col < cols) {
      const uint8_t* src = W + (size_t(row) * size_t(cols) + size_t(col)) * 2;
      v[i][0] = ld_global_cs_v4(src);
      v[i][1] = ld_global_cs_v4(src + 16);
    }
  }
  uint32_t m = amax_bf16x16(v[0][0], v[0][1]);
#pragma unroll
  for (int i = 1; i < 4; ++i) m = amax_bf16x2(m, amax_bf16x16(v[i][0], v[i][1]));
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m = amax_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, s));
  if ((threadIdx.x & 31u) == 0u) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQuantThreads / 32; ++i) m = amax_bf16x2(m, warp_max[i]);
  const uint32_t b = e8m0_of_pair(m);
  const uint32_t f = e8m0_inverse(b);
  if (threadIdx.x == 0) Ws[blockIdx.x] = uint8_t(b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + 32 * i;
    const uint2 lo = quant8(v[i][0], f), hi = quant8(v[i][1], f);
    if (row < rows && col < cols)
      *reinterpret_cast<uint4*>(Wq + size_t(row) * size_t(cols) + size_t(col)) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
}

// Wq, Ws -> W (bf16): each value q 2^(b - 127) rounded once (it is exact
// unless it is below bf16's normal range).  Eight values a lane, so that a
// warp's store is 512 consecutive bytes of two rows (16 values a lane, stored
// in two halves of each 32-byte sector, take 40 us instead of 30.5 on 14336 x
// 4096, launched one by one).
__global__ void __launch_bounds__(kQuantThreads)
    dequantize_block_kernel(const uint8_t* Wq, const uint8_t* Ws, uint8_t* W, int32_t rows, int32_t cols,
                            int32_t col_blocks) {
  griddep_wait();
  griddep_launch_dependents();
  const int cb = int(blockIdx.x) % col_blocks, rb = int(blockIdx.x) / col_blocks;
  const int col = cb * kQBlock + int(threadIdx.x & 15u) * 8;
  const int row0 = rb * kQBlock + int(threadIdx.x >> 4);
  if (col >= cols) return;
  const float s = e8m0_value(ld_global_u8(Ws + blockIdx.x));
  uint2 q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = imin(row0 + 16 * i, rows - 1);
    q[i] = ld_global_cs_v2(Wq + size_t(row) * size_t(cols) + size_t(col));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 16 * i;
    if (row >= rows) return;
    const float2 a = e4m3x2_to_f32(q[i].x), b = e4m3x2_to_f32(q[i].x >> 16);
    const float2 c = e4m3x2_to_f32(q[i].y), d = e4m3x2_to_f32(q[i].y >> 16);
    *reinterpret_cast<uint4*>(W + (size_t(row) * size_t(cols) + size_t(col)) * 2) =
        make_uint4(pack_bf16x2(a.x * s, a.y * s), pack_bf16x2(b.x * s, b.y * s), pack_bf16x2(c.x * s, c.y * s),
                   pack_bf16x2(d.x * s, d.y * s));
  }
}

}  // namespace lora
