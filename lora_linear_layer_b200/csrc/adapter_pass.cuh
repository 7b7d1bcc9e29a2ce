// adapter_pass.cuh - the rank-sized products with the adapter's dropout and
// the 8-bit rounding done on the way:
//     OUT[i, j] = scale * sum_k (m * P)(i, k) R(j, k),  j < r_pad
// and, with QUANT, P itself as e4m3 codes with one power-of-two scale for
// each row and 128 values of k (fp8.cuh), from the same read of P.
//   T  = s/(1-p) (m * X) A^T  (+ Xq)  P = X[M, d_in],  R = A[r, d_in] (K-major)
//   dT = s dY B               (+ dYq) P = dY[M, d_out], R(j,k) = B[k, j] (MN)
//   dB = dY^T T                       P(i,k) = dY[k, i] (MN), R(j,k) = T[k, j]
//   dA = dT^T (m * X)/(1-p)           P(i,k) = X[k, i] (MN),  R(j,k) = dT[k, j]
// Tiles, splits and the cluster reduction are those of skinny.cuh: i runs
// over 128-row tiles (UMMA M = 128), the rank is the UMMA N, and the
// contraction is split over a cluster whose partials are added in split
// order (no atomics: results repeat bit for bit).
//
// What bounds it is the read of P (and the write of its codes).  So P comes
// by TMA as in the plain product, several stages ahead, and 8 or 16 warps
// (pass_workers) work on each stage in shared memory between the copy and
// the MMA: they take the maximum of a row's 128 values over 4 lanes, write
// the codes to global memory, and put the masked values back where the MMA
// reads them (a dropped value is set to zero by a select, so the product
// needs no mask and a dropped infinity or NaN is gone; 1/(1-p) is in the
// scale).  The mask is computed here, 8 values at a time, for the chunk in
// hand.
#pragma once

#include "common.cuh"
#include "fp8.cuh"
#include "philox.cuh"
#include "skinny.cuh"

namespace lora {

// Warps that work on the stages, beside the TMA and the MMA warp: 16, one
// block an SM and a deep ring, where P is rounded (X[8192, 4096] at r = 16: 21
// us against 24 us with two blocks of 8) or the rank's operand is wide (stages
// of 48 KB and more); else 8 and two blocks an SM (masked, X[32768, 4096]: 78
// us against 83 us).
__host__ __device__ constexpr int pass_workers(int rcw, bool p_mn, bool quant) {
  return !p_mn && (quant || rcw == 64) ? 16 : 8;
}
__host__ __device__ constexpr int pass_threads(int rcw, bool p_mn, bool quant) {
  return 64 + 32 * pass_workers(rcw, p_mn, quant);
}

struct PassArgs {
  int32_t rows;           // output rows (size of the i dimension)
  int32_t K;              // contraction length
  int32_t r_pad;          // rank rounded up to 16
  int32_t r;              // rank
  int32_t n_rchunks;      // r_pad / RCW rounded up
  int32_t stages;
  int32_t nb_per_split;   // stages' worth of K (128 K-major, 64 MN) per split
  int32_t splits;         // gridDim.y; the cluster size
  int32_t out_mode;       // SkinnyOut
  int32_t r_mn;           // R is read MN-major
  int32_t out_f32;        // OUT_ROWS_R / OUT_COLS_R: write fp32
  float scale;            // applied to the reduced fp32 sum before rounding
  __nv_bfloat16* out;     // (a float* when out_f32)
  DropArgs drop;          // rng NULL: P is used as it is
  uint8_t* codes;         // QUANT: [rows, K] e4m3
  uint8_t* scales;        // QUANT: e8m0 bytes (scale_atom_offset)
  uint64_t wait_limit_ns;
};

// One stage: SUB sub-stages of 64 values of K, each P (16 KB) then R.
struct PassLayout {
  uint32_t sub_bytes, stage_bytes, red_stride, off_bar, total;
  __host__ __device__ PassLayout(bool p_mn, bool r_mn, int rcw, int r_pad, int n_rchunks, int stages) {
    const uint32_t r_bytes = r_mn ? uint32_t(n_rchunks * rcw * 128) : uint32_t(r_pad * 128);
    sub_bytes = 16384u + r_bytes;
    stage_bytes = sub_bytes * (p_mn ? 1u : 2u);
    const uint32_t ring = stage_bytes * uint32_t(stages);
    red_stride = uint32_t((r_pad + 4) * 4);  // padded as in skinny.cuh
    const uint32_t red = 128u * red_stride;
    off_bar = ((ring > red ? ring : red) + 1023u) & ~1023u;
    total = off_bar + 256;
  }
};

template <bool P_MN, int RCW, bool QUANT>
__global__ void __launch_bounds__(pass_threads(RCW, P_MN, QUANT), pass_workers(RCW, P_MN, QUANT) == 16 ? 1 : 2)
    adapter_pass_kernel(const __grid_constant__ CUtensorMap tmP0, const __grid_constant__ CUtensorMap tmR0,
                        const __grid_constant__ CUtensorMap tmP1, const __grid_constant__ CUtensorMap tmR1,
                        const __grid_constant__ PassArgs a0, const __grid_constant__ PassArgs a1,
                        const int32_t x_split, const int32_t x_atoms, const __grid_constant__ ScaleAtomArgs atoms) {
  static_assert(!(P_MN && QUANT), "codes are written row by row");
  constexpr int kPassWorkers = pass_workers(RCW, P_MN, QUANT), kPassThreads = pass_threads(RCW, P_MN, QUANT);
  if constexpr (QUANT) {
    if (int(blockIdx.x) >= x_atoms) {  // blocks behind the row tiles: the other operand's scales
      griddep_wait();  // must come first, as below
      griddep_launch_dependents();
      const int blocks = int(gridDim.x) - x_atoms, block = int(blockIdx.x) - x_atoms + blocks * int(blockIdx.y);
      scale_atoms(atoms, block * (kPassThreads / 32) + int(threadIdx.x >> 5),
                  blocks * int(gridDim.y) * (kPassThreads / 32), int(threadIdx.x & 31u));
      return;
    }
  }
  const bool second = int(blockIdx.x) >= x_split;
  const PassArgs& a = second ? a1 : a0;
  const int bx = second ? int(blockIdx.x) - x_split : int(blockIdx.x);
  constexpr uint32_t kRSwz = RCW == 16 ? SWZ_32B : RCW == 32 ? SWZ_64B : SWZ_128B;
  constexpr uint32_t kRSpan = RCW * 2;
  constexpr int kSub = P_MN ? 1 : 2;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (sbase - raw);
  const bool r_mn = a.r_mn != 0;
  const PassLayout L(P_MN, r_mn, RCW, a.r_pad, a.n_rchunks, a.stages);
  const int S = a.stages;
  const uint32_t bar0 = sbase + L.off_bar;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto ready_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto empty_bar = [&](int s) { return bar0 + 8u * (2 * S + s); };
  const uint32_t accfull = bar0 + 8u * (3 * S);
  const uint32_t drain = bar0 + 8u * (3 * S + 1);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + L.off_bar + 8 * (3 * S + 2));
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t ncols = tmem_cols_for(a.r_pad);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(ready_bar(s), kPassWorkers);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(accfull, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(second ? &tmP1 : &tmP0);
    tma_prefetch_desc(second ? &tmR1 : &tmR0);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), ncols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The wait must come first, in every block: token_stream_kernel and
  // lowrank_gemm_kernel (late_wait) behind this one read, before their own
  // wait, what was written before this one.  That is complete only if this
  // one lets them go after it has waited itself.
  griddep_wait();
  griddep_launch_dependents();

  const int i0 = bx * 128;
  const int split = blockIdx.y;
  constexpr int kStageK = 64 * kSub;
  const int nb_total = (a.K + kStageK - 1) / kStageK;
  const int kb0 = imin(nb_total, split * a.nb_per_split);
  const int kb1 = imin(nb_total, kb0 + a.nb_per_split);
  const int nkb = kb1 - kb0;
  const uint64_t lim = a.wait_limit_ns;
  const bool drop = a.drop.rng != nullptr;
  const bool work = QUANT || drop;  // the stages pass through the worker warps

  if (warp == 0) {
    auto produce = [&](const CUtensorMap& tmP, const CUtensorMap& tmR) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, lim, SITE_EMPTY)) break;
        const uint32_t fb = full_bar(stage);
        mbar_arrive_expect_tx(fb, L.stage_bytes);
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
          const uint32_t st = sbase + uint32_t(stage) * L.stage_bytes + uint32_t(sub) * L.sub_bytes;
          const int k0 = kb * kStageK + sub * 64;
          if (!P_MN) {
            tma_load_2d(st, &tmP, fb, k0, i0);
          } else {
            tma_load_2d(st, &tmP, fb, i0, k0);
            tma_load_2d(st + 8192u, &tmP, fb, i0 + 64, k0);
          }
          const uint32_t sr = st + 16384u;
          if (!r_mn) {
            tma_load_2d(sr, &tmR, fb, k0, 0);
          } else {
            for (int c = 0; c < a.n_rchunks; ++c)
              tma_load_2d(sr + uint32_t(c) * (64u * kRSpan), &tmR, fb, c * RCW, k0);
          }
        }
        if (++stage == S) { stage = 0; phase ^= 1u; }
      }
    };
    if (lane == 0) {
      if (second) produce(tmP1, tmR1);
      else produce(tmP0, tmR0);
      if (*abort_flag) settle_ns(200000);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(128, a.r_pad, P_MN, r_mn);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = 0; kb < nkb; ++kb) {
        if (!wait_bounded(full_bar(stage), phase, abort_flag, lim, SITE_FULL) ||
            (work && !wait_bounded(ready_bar(stage), phase, abort_flag, lim, SITE_VFULL))) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
          const uint32_t st = sbase + uint32_t(stage) * L.stage_bytes + uint32_t(sub) * L.sub_bytes;
          const uint32_t sr = st + 16384u;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t ad = P_MN ? smem_desc(st + kk * 2048u, 8192u, 1024u, SWZ_128B)
                                     : smem_desc(st + kk * 32u, 16u, 1024u, SWZ_128B);
            const uint64_t bd = r_mn ? smem_desc(sr + kk * (16u * kRSpan), 64u * kRSpan, 8u * kRSpan, kRSwz)
                                     : smem_desc(sr + kk * 32u, 16u, 1024u, SWZ_128B);
            umma_bf16(tmem, ad, bd, idesc, (kb | sub | kk) != 0);
          }
        }
        umma_commit(empty_bar(stage));
        if (++stage == S) { stage = 0; phase ^= 1u; }
      }
      if (ok) umma_commit(accfull);
      umma_commit(drain);
      wait_bounded(drain, 0u, abort_flag, lim, SITE_DRAIN);
    }
  } else if (work) {
    // -------------------------------------------- workers on a stage ----
    const int w = warp - 2;
    DropState ds{};
    if (drop) ds = drop_load(a.drop);
    int stage = 0;
    uint32_t phase = 0;
    // What bounds these warps is their instructions (at 8 lanes a row and one
    // address calculation a store X[32768, 4096] took 88 us rounded and 75 us
    // masked, against 48 us untouched), so a lane takes as much of a row as it
    // can, and pointers run along.
    constexpr int kRows = 128 / kPassWorkers;
    if constexpr (!P_MN) {
      // Eight rows at a time, 4 lanes a row; a lane has 16 consecutive values
      // (two 16-byte chunks) of each sub-stage, so that the row's codes leave
      // in two stores of 64 consecutive bytes.  The 8 lanes of two rows touch
      // 8 different bank groups: even chunks of one row, odd ones of the other.
      constexpr int kIts = kRows / 8;
      const int c = lane & 3, r8 = lane >> 2;
      const int row0 = i0 + w * kRows + r8;
      uint32_t at[4];  // inside a stage: chunks 2 c and 2 c + 1 of the first sub-stage, then of the second
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        at[j] = (j >> 1) * L.sub_bytes + uint32_t(w * kRows + r8) * 128u +
                ((uint32_t(c) * 2u + (j & 1u)) ^ uint32_t(r8)) * 16u;
      const bool any = i0 + w * kRows < a.rows;  // (rows past the end are zero fill)
      uint8_t* code = QUANT ? a.codes + size_t(row0) * size_t(a.K) + size_t(kb0) * 128 + size_t(c * 16) : nullptr;
      const size_t code_step = size_t(8) * size_t(a.K);
      const int row_blocks = (a.rows + 127) / 128;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait_bounded(full_bar(stage), phase, abort_flag, lim, SITE_FULL)) break;
        if (any) {
          const uint32_t st = sbase + uint32_t(stage) * L.stage_bytes;
          const int k = kb * 128 + c * 16;
          uint4 v[kIts][4];
#pragma unroll
          for (int it = 0; it < kIts; ++it)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[it][j] = ld_shared_v4(st + at[j] + uint32_t(it) * 1024u);
          if constexpr (QUANT) {
            uint8_t* const scale = a.scales + scale_atom_offset(row0, kb, row_blocks);  // 8 rows on: 128 bytes on
            uint32_t m[kIts];
#pragma unroll
            for (int it = 0; it < kIts; ++it)
              m[it] = amax_bf16x2(amax_bf16x16(v[it][0], v[it][1]), amax_bf16x16(v[it][2], v[it][3]));
#pragma unroll
            for (int s = 2; s > 0; s >>= 1)
#pragma unroll
              for (int it = 0; it < kIts; ++it) m[it] = amax_bf16x2(m[it], __shfl_xor_sync(0xffffffffu, m[it], s));
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
              const uint32_t b = e8m0_of_pair(m[it]), f = e8m0_inverse(b);
              const uint2 q0 = quant8(v[it][0], f), q1 = quant8(v[it][1], f);
              const uint2 q2 = quant8(v[it][2], f), q3 = quant8(v[it][3], f);
              if (row0 + 8 * it < a.rows) {
                uint8_t* const dst = code + size_t(it) * code_step;
                // (K is a multiple of 16)
                if (k < a.K) *reinterpret_cast<uint4*>(dst) = make_uint4(q0.x, q0.y, q1.x, q1.y);
                if (k + 64 < a.K) *reinterpret_cast<uint4*>(dst + 64) = make_uint4(q2.x, q2.y, q3.x, q3.y);
                if (c == 0) scale[it * 128] = uint8_t(b);
              }
            }
            code += 128;
          }
          if (drop) {
            const uint32_t c8 = uint32_t(k) >> 3;
#pragma unroll
            for (int it = 0; it < kIts; ++it)
#pragma unroll
              for (uint32_t j = 0; j < 4; ++j)
                st_shared_v4(st + at[j] + uint32_t(it) * 1024u,
                             drop_bf16x8(v[it][j], drop_block(ds, c8 + (j >> 1) * 8u + (j & 1u), uint32_t(row0 + 8 * it)), ds.thr_hi));
          }
        }
        if (drop) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(ready_bar(stage));
        if (++stage == S) { stage = 0; phase ^= 1u; }
      }
    } else {
      // 64 tokens x two chunks of 64 columns: 128 rows of 8 lanes, four at a time
      const int c = lane & 7, r4 = lane >> 3;
      uint32_t off[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t row = uint32_t(w * kRows + 4 * i + r4);
        off[i] = (row >> 6) * 8192u + swz_offset(row & 63u, uint32_t(c), 128u);
      }
      const int tok0 = (w * kRows + r4) & 63;
      const uint32_t c8 = uint32_t(i0 + (w * kRows >> 6) * 64) / 8u + uint32_t(c);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait_bounded(full_bar(stage), phase, abort_flag, lim, SITE_FULL)) break;
        const uint32_t st = sbase + uint32_t(stage) * L.stage_bytes;
#pragma unroll
        for (int it = 0; it < kRows / 4; ++it) {
          const uint32_t addr = st + off[it & 1] + uint32_t(it >> 1) * 1024u;
          const uint32_t tok = uint32_t(kb * 64 + tok0 + 4 * it);
          st_shared_v4(addr, drop_bf16x8(ld_shared_v4(addr), drop_block(ds, c8, tok), ds.thr_hi));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(ready_bar(stage));
        if (++stage == S) { stage = 0; phase ^= 1u; }
      }
    }
  }

  // ---------------------------------------------- partial / output -----
  uint8_t* const red = gbase;  // fp32 partial rows (reuses the ring once the MMAs are done)
  if (warp >= 2) {
    bool have = true;
    if (nkb > 0) {
      have = warp_wait_bounded(accfull, 0u, abort_flag, lim, SITE_ACCFULL);
      tc_fence_after();
    }
    if (have) {
      const int q = warp & 3;
      const uint32_t lane_base = uint32_t(q * 32) << 16;
      for (int col = 16 * ((warp - 2) >> 2); col < a.r_pad; col += 4 * kPassWorkers) {
        uint32_t v[16];
        if (nkb > 0) {
          tmem_ld_x16(tmem + lane_base + uint32_t(col), v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = 0u;  // empty split: contributes zero
        }
        uint4* dst = reinterpret_cast<uint4*>(red + uint32_t(q * 32 + lane) * L.red_stride + col * 4);
#pragma unroll
        for (int g = 0; g < 4; ++g) dst[g] = make_uint4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier_sync();  // every split's partial is in its shared memory
  // Every CTA of the cluster reduces its own slice of the 128 rows: four
  // consecutive columns per task, the S partials added in split order.
  if (warp >= 2 && !*abort_flag) {
    const int n_splits = a.splits;
    const int f4_per_row = a.r_pad / 4;
    const int rows_per = (128 + n_splits - 1) / n_splits;
    const int r0 = split * rows_per;
    const int n_rows = imin(128, r0 + rows_per) - r0;
    for (int task = int(threadIdx.x) - 64; task < n_rows * f4_per_row; task += 32 * kPassWorkers) {
      // (transposed output: rows fastest, so a warp writes neighbours)
      const bool cols = a.out_mode == OUT_COLS_R;
      const int rr = r0 + (cols ? task % n_rows : task / f4_per_row);
      const int c4 = cols ? task / n_rows : task % f4_per_row;
      const uint32_t off = smem_addr(red + rr * L.red_stride + c4 * 16);
      float4 p[8];
#pragma unroll
      for (int s2 = 0; s2 < 8; ++s2)
        if (s2 < n_splits) p[s2] = ld_shared_cluster_f4(mapa_shared(off, uint32_t(s2)));
      float4 acc = p[0];
#pragma unroll
      for (int s2 = 1; s2 < 8; ++s2)
        if (s2 < n_splits) {
          acc.x += p[s2].x;
          acc.y += p[s2].y;
          acc.z += p[s2].z;
          acc.w += p[s2].w;
        }
      const int g = i0 + rr;
      const int j0 = c4 * 4;
      if (g >= a.rows) continue;
      const float v[4] = {acc.x * a.scale, acc.y * a.scale, acc.z * a.scale, acc.w * a.scale};
      if (a.out_mode == OUT_ROWS_RPAD) {
        // T and dT go to bf16 because they are the operands of the next
        // product, whose other side is bf16 (kind::f16 takes one type for
        // both).  Columns past the rank are zero and not the sum: a row with
        // an infinity has NaN there (infinity times zero fill), which the
        // next product would spread over its whole row.
        if (j0 >= a.r) {  // r % 8 == 0: the 4 columns are all in or all out
          *reinterpret_cast<uint2*>(a.out + size_t(g) * size_t(a.r_pad) + j0) = make_uint2(0u, 0u);
          continue;
        }
        *reinterpret_cast<uint2*>(a.out + size_t(g) * size_t(a.r_pad) + j0) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      } else if (a.out_mode == OUT_ROWS_R) {
        if (j0 >= a.r) continue;
        const size_t o = size_t(g) * size_t(a.r) + j0;
        if (a.out_f32)
          *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + o) = make_float4(v[0], v[1], v[2], v[3]);
        else
          *reinterpret_cast<uint2*>(a.out + o) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (j0 + e >= a.r) continue;
          const size_t o = size_t(j0 + e) * size_t(a.rows) + g;
          if (a.out_f32) reinterpret_cast<float*>(a.out)[o] = v[e];
          else a.out[o] = __float2bfloat16_rn(v[e]);
        }
      }
    }
  }
  cluster_barrier_sync();  // peers keep their shared memory until every slice is done
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, ncols);
  }
}

}  // namespace lora
