// token.cuh - the layer for few tokens:
//     Y  = X W^T + T B^T,                 T = s/(1-p) (m * X) A^T
//     dX = dY W + m * (dT A)/(1-p)
// over a bf16 base or an 8-bit one (Xq, dYq and Wq in the base product).
//
// At this size the layer is one read of the weight and the latency around
// it.  Two launches forward:
//  1. token_prep_kernel: T, and with an 8-bit base the codes and scales of X,
//     beside each other in one grid of small blocks that read straight into
//     registers.
//  2. token_stream_kernel: W streamed through the tensor pipe, with W's rows
//     (columns for dX) as the MMA's 128 rows and the tokens as its N columns,
//     so that no row of a tile is empty and each W tile is read once.
// The second launch starts while the first runs (programmatic dependent
// launch) and fetches its first stages of W before it waits: W was complete
// before the first kernel began, since that one waits before it lets a
// dependent launch go.
#pragma once

#include "common.cuh"
#include "fp8.cuh"
#include "philox.cuh"

namespace lora {

constexpr int kPrepThreads = 256;
constexpr int kPrepWarps = kPrepThreads / 32;
constexpr int kPrepTokens = 16;  // tokens of a block of T (the m16n8k16 MMA's rows)
constexpr int kPrepRanks = 16;   // and its rank rows
constexpr int kPrepSplits = 4;   // blocks (a cluster) that share one such sum

struct PrepArgs {
  const uint8_t* X;      // bf16 [M, K]
  const uint8_t* A;      // bf16 [r, K]
  __nv_bfloat16* T;      // [M, r_pad]
  uint8_t* codes;        // [M, K] (with an 8-bit base)
  uint8_t* scales;       // e8m0 bytes (scale_atom_offset)
  int32_t M, K, r, r_pad, t_blocks, q_blocks;
  float scale;
  DropArgs drop;
  ScaleAtomArgs atoms;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Blocks [0, t_blocks): T for 16 tokens and 16 rank rows.  The warps take 32
// values of K in turn; a lane loads 8 consecutive values (16 bytes) of its
// two tokens and of its two rank rows, which are the operands of two MMAs:
// the order of K inside the 32 is free as long as both sides agree on it.
// K is split over a cluster of four, so that one token's T is not a chain of
// memory latencies: 4096 values are one round of loads.  The sums of the
// warps, then of the blocks, are added in order.
// The other blocks: codes and scales of X, one warp for each row and 512
// values.
__global__ void __launch_bounds__(kPrepThreads) token_prep_kernel(const PrepArgs a) {
  __shared__ float part[kPrepWarps][kPrepTokens][kPrepRanks + 1];
  __shared__ __align__(16) float sums[kPrepTokens * kPrepRanks];
  // The wait must come first, in every block: token_stream_kernel behind this
  // one reads the weight before its own wait (see adapter_pass_kernel).
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (int(blockIdx.x) >= a.t_blocks + a.q_blocks) {  // the weight's scales for the product, where it wants them
    const int block = int(blockIdx.x) - a.t_blocks - a.q_blocks, blocks = int(gridDim.x) - a.t_blocks - a.q_blocks;
    scale_atoms(a.atoms, block * kPrepWarps + warp, blocks * kPrepWarps, lane);
    return;
  }
  if (int(blockIdx.x) >= a.t_blocks) {  // (a whole cluster of them)
    // 8 lanes a group of 128 values, 4 groups (one scale word) a warp
    const int groups = (a.K + 511) / 512;
    const int item = (int(blockIdx.x) - a.t_blocks) * kPrepWarps + warp;
    if (item >= a.M * groups) return;
    const int row = item / groups, g = item - row * groups;
    const int k = g * 512 + lane * 16;
    const bool in = k < a.K;  // K is a multiple of 16
    const size_t at = size_t(row) * size_t(a.K) + size_t(k);
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    if (in) {
      const uint4* src = reinterpret_cast<const uint4*>(a.X + at * 2);
      v0 = src[0];
      v1 = src[1];
    }
    uint32_t m = amax_bf16x16(v0, v1);
#pragma unroll
    for (int s = 4; s > 0; s >>= 1) m = amax_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, s));
    const uint32_t b = e8m0_of_pair(m), f = e8m0_inverse(b);
    const uint2 q0 = quant8(v0, f), q1 = quant8(v1, f);
    if (in) *reinterpret_cast<uint4*>(a.codes + at) = make_uint4(q0.x, q0.y, q1.x, q1.y);
    if ((lane & 7) == 0) a.scales[scale_atom_offset(row, 4 * g + (lane >> 3), (a.M + 127) / 128)] = uint8_t(b);
    return;
  }
  const int j_blocks = a.r_pad / kPrepRanks;
  const int tile = int(blockIdx.x) / kPrepSplits, split = int(blockIdx.x) % kPrepSplits;
  const int j0 = (tile % j_blocks) * kPrepRanks, m0 = (tile / j_blocks) * kPrepTokens;
  const int g = lane >> 2, t = lane & 3;
  // Rows that are not there repeat the last one; their sums are not used.
  // (Every load is unconditional: as branches they ran one after the other.)
  const uint8_t* src[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    src[i] = a.X + size_t(imin(m0 + g + 8 * i, a.M - 1)) * size_t(a.K) * 2;
    src[2 + i] = a.A + size_t(imin(j0 + g + 8 * i, a.r - 1)) * size_t(a.K) * 2;
  }
  const bool drop = a.drop.rng != nullptr;
  DropState ds{};
  if (drop) ds = drop_load(a.drop);
  float d[2][4] = {};
  constexpr int kUnroll = 4;
  constexpr int kStep = kPrepSplits * kPrepWarps * 32;
  for (int k0 = (split * kPrepWarps + warp) * 32; k0 < a.K; k0 += kStep * kUnroll) {
    uint4 v[kUnroll][4];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = k0 + u * kStep + t * 8;
      const size_t at = size_t(imin(k, a.K - 8)) * 2;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[u][i] = ld_global_v4(src[i] + at);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (k0 + u * kStep + t * 8 >= a.K) {  // past the end of K: zero
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = make_uint4(0, 0, 0, 0);
      }
    if (drop) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          v[u][i] = drop_bf16x8(v[u][i], drop_block(ds, uint32_t(k0 + u * kStep) / 8u + uint32_t(t), uint32_t(m0 + g + 8 * i)),
                                ds.thr_hi);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mma_bf16(d[j], v[u][0].x, v[u][1].x, v[u][0].y, v[u][1].y, v[u][2 + j].x, v[u][2 + j].y);
        mma_bf16(d[j], v[u][0].z, v[u][1].z, v[u][0].w, v[u][1].w, v[u][2 + j].z, v[u][2 + j].w);
      }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][g + 8 * (e >> 1)][8 * j + 2 * t + (e & 1)] = d[j][e];
  __syncthreads();
  {
    const int tok = int(threadIdx.x) / kPrepRanks, j = int(threadIdx.x) % kPrepRanks;  // 256 threads, 16 x 16 sums
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kPrepWarps; ++w) s += part[w][tok][j];
    sums[threadIdx.x] = s;
  }
  cluster_barrier_sync();
  constexpr int kShare = kPrepTokens * kPrepRanks / kPrepSplits;  // this block's share of the 16 x 16
  if (int(threadIdx.x) < kShare) {
    const int i = split * kShare + int(threadIdx.x), tok = i / kPrepRanks, j = i % kPrepRanks;
    float s = 0.0f;
#pragma unroll
    for (uint32_t c = 0; c < uint32_t(kPrepSplits); ++c) s += ld_shared_cluster_f32(mapa_shared(smem_addr(sums + i), c));
    if (m0 + tok < a.M)  // (bf16, and zero past the rank, as adapter_pass_kernel leaves it)
      a.T[size_t(m0 + tok) * size_t(a.r_pad) + size_t(j0 + j)] =
          __float2bfloat16_rn(j0 + j < a.r ? s * a.scale : 0.0f);
  }
  cluster_barrier_sync();  // peers keep their sums until they are read
}

// The contraction of the second launch is split over a cluster whose fp32
// partials are added in split order through distributed shared memory, as in
// skinny.cuh; the rank product is one or two more K blocks of the first split.
// The scales go to TMEM as in lowrank_gemm.cuh; W's are one for the whole
// tile.  DROP (dX with a mask): the rank product has an accumulator of its
// own, and the first split masks and adds it when it takes its partial out.
constexpr int kStreamMax = 256;
constexpr int kStreamMaxDrop = 192;  // two accumulators
constexpr int kStreamThreads = 192;
constexpr int kStreamScaleBufs = 4;
constexpr uint32_t kStreamScaleBytes = 512u * 3u;

struct StreamArgs {
  const uint8_t* w_scales;   // 8-bit base: bytes of its blocks
  int32_t ws_row, ws_k;      // strides along the MMA's rows and along K
  const uint32_t* x_scales;  // 8-bit base: words of 4 scale bytes (scale_atom_offset)
  __nv_bfloat16* out;        // [M, N]
  int32_t M, N, K, r_pad;
  int32_t tok_pad;           // tokens rounded up to 16 (UMMA N)
  int32_t stages, kb_per_split, splits;
  DropArgs drop;
  uint64_t wait_limit_ns;
};

struct StreamLayout {
  uint32_t stage_bytes, off_sf, off_bar, red_stride, total;
  __host__ __device__ StreamLayout(int tok_pad, int stages) {
    stage_bytes = 16384u + uint32_t(tok_pad) * 128u;
    const uint32_t ring = stage_bytes * uint32_t(stages);
    red_stride = uint32_t(tok_pad + 4) * 4u;
    const uint32_t red = 128u * red_stride;
    off_sf = ((ring > red ? ring : red) + 1023u) & ~1023u;
    off_bar = off_sf + kStreamScaleBufs * kStreamScaleBytes;
    total = off_bar + 512;
  }
};

// Accumulators and, in the last 64 columns, the scales.
__host__ __device__ inline uint32_t stream_tmem_cols(int tok_pad, bool drop) {
  const int need = tok_pad * (drop ? 2 : 1) + 16 * kStreamScaleBufs;
  return need <= 128 ? 128u : need <= 256 ? 256u : 512u;
}

template <bool FP8, bool MN, bool DROP>
__global__ void __launch_bounds__(kStreamThreads)
    token_stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmU,
                        const __grid_constant__ StreamArgs a) {
  static_assert(!DROP || MN, "only dX masks its rank product");
  constexpr int kStageK = FP8 ? 128 : 64;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (sbase - raw);
  const StreamLayout L(a.tok_pad, a.stages);
  const int S = a.stages;
  const uint32_t bar0 = sbase + L.off_bar;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  const uint32_t accfull = bar0 + 8u * (2 * S);
  const uint32_t drain = bar0 + 8u * (2 * S + 1);
  const uint32_t sffull0 = bar0 + 8u * (2 * S + 2);
  const uint32_t sfempty0 = sffull0 + 8u * kStreamScaleBufs;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + L.off_bar + 8 * (2 * S + 2 + 2 * kStreamScaleBufs));
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ncols = stream_tmem_cols(a.tok_pad, DROP);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(accfull, 1);
    mbar_init(drain, 1);
    for (int i = 0; i < 2 * kStreamScaleBufs; ++i) mbar_init(sffull0 + 8u * i, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmU);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), ncols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int n0 = int(blockIdx.x) * 128;
  const int split = blockIdx.y;
  const int nk = (a.K + kStageK - 1) / kStageK;
  const int kb0 = imin(nk, split * a.kb_per_split);
  const int nkb = imin(nk, kb0 + a.kb_per_split) - kb0;
  const int nr = split == 0 ? (a.r_pad + 63) / 64 : 0;  // rank blocks
  const uint64_t lim = a.wait_limit_ns;

  if (warp == 0) {
    if (lane == 0) {
      // the weight's 128 rows (columns with MN) of one K block into a stage
      auto load_w = [&](uint32_t st, uint32_t fb, int kb) {
        const int k0 = kb * kStageK;
        if constexpr (!MN) {
          tma_load_2d(st, &tmW, fb, k0, n0);
        } else if constexpr (FP8) {
          tma_load_2d(st, &tmW, fb, n0, k0);
        } else {
          tma_load_2d(st, &tmW, fb, n0, k0);
          tma_load_2d(st + 8192u, &tmW, fb, n0 + 64, k0);
        }
      };
      const int pre = imin(S, nkb);
      for (int i = 0; i < pre; ++i) {
        mbar_arrive_expect_tx(full_bar(i), L.stage_bytes);
        load_w(sbase + uint32_t(i) * L.stage_bytes, full_bar(i), kb0 + i);
      }
      griddep_wait();
      griddep_launch_dependents();
      for (int i = 0; i < pre; ++i)
        tma_load_2d(sbase + uint32_t(i) * L.stage_bytes + 16384u, &tmX, full_bar(i), (kb0 + i) * kStageK, 0);
      int stage = pre % S;
      uint32_t phase = pre == S ? 1u : 0u;
      for (int i = pre; i < nkb + nr; ++i) {
        if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, lim, SITE_EMPTY)) break;
        const uint32_t st = sbase + uint32_t(stage) * L.stage_bytes, fb = full_bar(stage);
        mbar_arrive_expect_tx(fb, L.stage_bytes);
        if (i < nkb) {
          load_w(st, fb, kb0 + i);
          tma_load_2d(st + 16384u, &tmX, fb, (kb0 + i) * kStageK, 0);
        } else {
          const int r0 = (i - nkb) * 64;
          if constexpr (!MN) {
            tma_load_2d(st, &tmV, fb, r0, n0);
          } else {
            tma_load_2d(st, &tmV, fb, n0, r0);
            tma_load_2d(st + 8192u, &tmV, fb, n0 + 64, r0);
          }
          tma_load_2d(st + 16384u, &tmU, fb, r0, 0);
        }
        if (++stage == S) { stage = 0; phase ^= 1u; }
      }
      if (*abort_flag) settle_ns(200000);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t id_bf16 = idesc_bf16(128, uint32_t(a.tok_pad), MN, false);
      const uint32_t sf_base = tmem + ncols - 16u * kStreamScaleBufs;
      auto w_desc = [&](uint32_t st, uint32_t kk) {  // bf16: 16 values of K on
        return MN ? smem_desc(st + kk * 2048u, 8192u, 1024u, SWZ_128B) : smem_desc(st + kk * 32u, 16u, 1024u, SWZ_128B);
      };
      int stage = 0;
      uint32_t phase = 0, sf_tmem = 0;
      bool ok = true;
      for (int i = 0; i < nkb + nr && ok; ++i) {
        if (!wait_bounded(full_bar(stage), phase, abort_flag, lim, SITE_FULL)) { ok = false; break; }
        tc_fence_after();
        const uint32_t st = sbase + uint32_t(stage) * L.stage_bytes, sx = st + 16384u;
        if (i >= nkb) {
          const uint32_t d = tmem + (DROP ? uint32_t(a.tok_pad) : 0u);
          const int kk_n = imin(4, (a.r_pad - (i - nkb) * 64) / 16);
          for (int kk = 0; kk < kk_n; ++kk)
            umma_bf16(d, w_desc(st, uint32_t(kk)), smem_desc(sx + kk * 32u, 16u, 1024u, SWZ_128B), id_bf16,
                      DROP ? (i - nkb | kk) != 0 : 1u);
        } else if constexpr (FP8) {
          if ((i & 3) == 0) {
            const uint32_t n = uint32_t(i) >> 2, buf = n % kStreamScaleBufs;
            if (!wait_bounded(sffull0 + 8u * buf, (n / kStreamScaleBufs) & 1u, abort_flag, lim, SITE_TXMSG)) {
              ok = false;
              break;
            }
            tc_fence_after();
            sf_tmem = sf_base + 16u * buf;
            const uint32_t src = sbase + L.off_sf + buf * kStreamScaleBytes;
#pragma unroll
            for (uint32_t c = 0; c < 3; ++c)
              tmem_cp_scales(sf_tmem + 4u * c, smem_desc(src + 512u * c, 16u, 128u, SWZ_NONE));
            umma_commit(sfempty0 + 8u * buf);
          }
          const uint32_t id = idesc_mxf8(128, uint32_t(a.tok_pad), MN, false, uint32_t(i & 3));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_mxf8(tmem,
                      MN ? smem_desc(st + kk * 4096u, 16384u, 1024u, SWZ_128B)
                         : smem_desc(st + kk * 32u, 16u, 1024u, SWZ_128B),
                      smem_desc(sx + kk * 32u, 16u, 1024u, SWZ_128B), id, sf_tmem, sf_tmem + 4u, (i | kk) != 0);
        } else {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem, w_desc(st, uint32_t(kk)), smem_desc(sx + kk * 32u, 16u, 1024u, SWZ_128B), id_bf16,
                      (i | kk) != 0);
        }
        umma_commit(empty_bar(stage));
        if (++stage == S) { stage = 0; phase ^= 1u; }
      }
      if (ok) umma_commit(accfull);
      umma_commit(drain);
      wait_bounded(drain, 0u, abort_flag, lim, SITE_DRAIN);
    }
  } else {
    griddep_wait();
    if constexpr (FP8) {
      // Scale words: W's are one for the whole tile, the tokens' one each.  The
      // four warps take the groups of four stages in turn, one buffer each.
      const uint8_t* const ws = a.w_scales + size_t(n0 >> 7) * size_t(a.ws_row);
      const int last_group = (nk - 1) >> 2, x_blocks = (a.M + 127) / 128;
      const uint32_t buf = uint32_t(warp - 2);
      const uint32_t dst = sbase + L.off_sf + buf * kStreamScaleBytes + 16u * uint32_t(lane);
      uint32_t use = 0;
      for (int g = int(buf); g * 4 < nkb; g += kStreamScaleBufs) {
        const int kb = kb0 + 4 * g;
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) w |= uint32_t(ws[size_t(imin(kb + e, nk - 1)) * size_t(a.ws_k)]) << (8 * e);
        uint32_t x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (32 * i >= a.tok_pad) { x[i] = 0u; continue; }
          const int tok = imin(32 * i + lane, a.M - 1);
          const uint32_t lo = a.x_scales[scale_atom_offset(tok, kb & ~3, x_blocks) / 4];
          const uint32_t hi = a.x_scales[scale_atom_offset(tok, imin((kb & ~3) + 4, 4 * last_group), x_blocks) / 4];
          x[i] = __funnelshift_r(lo, hi, 8 * (kb & 3));
        }
        if (!warp_wait_bounded(sfempty0 + 8u * buf, (use++ & 1u) ^ 1u, abort_flag, lim, SITE_VEMPTY)) break;
        st_shared_v4(dst, make_uint4(w, w, w, w));
        st_shared_v4(dst + 512u, make_uint4(x[0], x[1], x[2], x[3]));
        st_shared_v4(dst + 1024u, make_uint4(x[4], x[5], x[6], x[7]));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(sffull0 + 8u * buf);
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
      const bool masked = DROP && split == 0;
      DropState ds{};
      if (masked) ds = drop_load(a.drop);
      for (int col = 0; col < a.tok_pad; col += 16) {
        uint32_t v[16];
        if (nkb > 0) {
          tmem_ld_x16(tmem + lane_base + uint32_t(col), v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = 0u;  // empty split: contributes zero
        }
        if (masked) {
          // This lane's column i = n0 + 32 q + lane of dX is one of 8 that
          // share a random block; each of the 8 lanes makes two of the 16
          // tokens' blocks and hands the words around.
          uint32_t u[16];
          tmem_ld_x16(tmem + lane_base + uint32_t(a.tok_pad + col), u);
          tmem_ld_wait();
          const uint32_t c8 = uint32_t(n0 + q * 32 + lane) / 8u;
          const int home = lane & 24, mine = lane & 7;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 r = drop_block(ds, c8, uint32_t(col + 8 * h + mine));
#pragma unroll
            for (int t = 0; t < 8; ++t) {
              const uint32_t w0 = __shfl_sync(0xffffffffu, r.x, home + t), w1 = __shfl_sync(0xffffffffu, r.y, home + t);
              const uint32_t w2 = __shfl_sync(0xffffffffu, r.z, home + t), w3 = __shfl_sync(0xffffffffu, r.w, home + t);
              const uint32_t w = mine < 4 ? (mine < 2 ? w0 : w1) : (mine < 6 ? w2 : w3);
              const bool keep = (mine & 1 ? w : w << 16) >= ds.thr_hi;
              const int e = 8 * h + t;
              const float x = __uint_as_float(u[e]) * a.drop.inv_keep;
              v[e] = __float_as_uint(__uint_as_float(v[e]) + (keep ? x : 0.0f));
            }
          }
        }
        uint4* dst = reinterpret_cast<uint4*>(red + uint32_t(q * 32 + lane) * L.red_stride + col * 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) dst[c] = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier_sync();  // every split's partial is in its shared memory
  if (warp >= 2 && !*abort_flag) {
    // this CTA's slice of the 128 rows, rows fastest: a warp writes neighbours
    const int rows_per = (128 + a.splits - 1) / a.splits;
    const int r0 = split * rows_per;
    const int n_rows = imin(128, r0 + rows_per) - r0;
    const int tok4 = (a.M + 3) / 4;
    for (int task = int(threadIdx.x) - 64; task < n_rows * tok4; task += kStreamThreads - 64) {
      const int rr = r0 + task % n_rows, t4 = task / n_rows;
      const uint32_t off = smem_addr(red + uint32_t(rr) * L.red_stride + t4 * 16);
      float4 p[8];
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s < a.splits) p[s] = ld_shared_cluster_f4(mapa_shared(off, uint32_t(s)));
      float4 acc = p[0];
#pragma unroll
      for (int s = 1; s < 8; ++s)
        if (s < a.splits) {
          acc.x += p[s].x;
          acc.y += p[s].y;
          acc.z += p[s].z;
          acc.w += p[s].w;
        }
      const int n = n0 + rr;
      if (n >= a.N) continue;
      const float v[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * t4 + e < a.M) a.out[size_t(4 * t4 + e) * size_t(a.N) + size_t(n)] = __float2bfloat16_rn(v[e]);
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
