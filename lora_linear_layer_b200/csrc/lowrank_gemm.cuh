// lowrank_gemm.cuh - OUT = P Q + m * (U V), the products that carry an
// adapter whose rank-side operand U is already in memory:
//   Y  = X W^T    + T B^T           (bf16 base, T with dropout: adapter_pass.cuh)
//   Y  = Xq Wq^T  + T B^T           (8-bit base)
//   dX = dY W     + m * (dT A)/(1-p)
//   dX = dYq Wq   + m * (dT A)/(1-p)
// One accumulator holds both products.  The rank side is one or two K blocks
// of the same ring, issued before the base blocks: where the mask m applies
// to it alone (DROP), eight warps take the rank product out of TMEM, mask and
// scale it, and put it back, and the base product then accumulates
// onto it.  That costs no extra accumulator and no extra pass over OUT, and
// it hides behind another tile's K loop: the rank blocks of the next tile
// are issued in the middle of the current one, into the other accumulator.
//
// FP8: operands are e4m3 with power-of-two scales for 128 values of K, which
// is what kind::mxf8f6f4 applies itself (it takes one scale for 32 values of
// K; the four of a block are the same byte).  A stage holds 128 values of K
// (128-byte rows, as 64 bf16 are), so the ring, the swizzle and the
// descriptors are those of the bf16 form.  The scales of four stages are the
// four bytes of one 32-bit word for each row (column) of the tile, selected
// by the scale index of the instruction descriptor.  They lie in memory as
// the tensor core reads them (scale_atom_offset) and come with the first of
// the four stages, by TMA and on its barrier; the MMA thread copies them to
// TMEM (tcgen05.cp) and does nothing else for them: its own instructions are
// what keeps the tensor pipe waiting at 8 bits.  (A warp that built the words
// in shared memory cost a wait and a commit there: 123 us against 109 us on
// 8192 x 4096 x 4096.)  Two accumulators of 224 columns leave 64 columns of
// TMEM for scales: four buffers of 16 columns.  A buffer comes round again
// after four groups of stages, which are seven stages or more (a group is one
// stage only where K <= 128, and then each but the last tile's has a rank
// block before it); the ring has at most seven, so the MMAs that read a buffer
// are done when the stage that brings its next scales can be filled.
//
// dX (late_wait) begins before the kernel in front of it, dA's and dB's, has
// ended: its inputs were complete when that one began its work, since that one
// waits before it lets a dependent launch go (adapter_pass_kernel must).  It
// waits at its end, so that what follows it still finds everything before it
// done.
//
// Tiles are CTA pairs (cta_group::2) of 256 x BN.  What bounds it is the
// tensor pipe.
#pragma once

#include "common.cuh"
#include "fused.cuh"
#include "philox.cuh"

namespace lora {

constexpr int kLrScaleBufs = 4;
constexpr int kLrMaxStagesFp8 = 7;
constexpr uint32_t kLrScaleBytes = 512u * 3u;  // A: 128 rows, B: 256 columns, 4 bytes each

struct LrArgs {
  FusedArgs f;               // sizes, tile counts, stages, ep_bufs
  int32_t group_m;           // M blocks walked together (LrSched)
  int32_t late_wait;         // the inputs were complete before the kernel before this one began its work
  DropArgs drop;             // DROP: the mask of OUT's [M, N]
};

// Tiles are dealt one at a time, group by group of `group_m` M blocks and M
// fastest inside a group: the tiles in flight share their rows of P, which
// stay in L2 for the whole group, and the same few columns of Q, so Q is read
// from memory once a group.
struct LrSched {
  int num_m, num_n, group_m, G, t;
  __device__ LrSched(const LrArgs& a, int G_, int c)
      : num_m(a.f.num_m), num_n(a.f.num_n), group_m(a.group_m), G(G_), t(c) {}
  __device__ bool next(int& m, int& n) {
    if (t >= num_m * num_n) return false;
    const int per = group_m * num_n;
    const int g = t / per, i = t - g * per;
    const int w = imin(group_m, num_m - g * group_m);
    n = i / w;
    m = g * group_m + (i - n * w);
    t += G;
    return true;
  }
};

template <bool FP8, bool MN, int BN>
struct LrShape {
  static constexpr int kBNC = BN / 2;                     // columns of OUT whose Q values a CTA holds
  static constexpr int kChunks = (kBNC + 63) / 64;        // 64-column chunks of bf16 MN-major operands
  static constexpr uint32_t kQBase = !MN ? kBNC * 128u : FP8 ? 16384u : kChunks * 8192u;  // bytes loaded, base block
  static constexpr uint32_t kQRank = !MN ? kBNC * 128u : kChunks * 8192u;                 // bytes loaded, rank block
  static constexpr uint32_t kQSlot = kQBase > kQRank ? kQBase : kQRank;
  static constexpr uint32_t kStage = 16384u + kQSlot;
};

struct LrLayout {
  uint32_t off_sf, off_ep, off_bar, total;
  __host__ __device__ LrLayout(uint32_t stage_bytes, bool fp8, int stages, int ep_bufs) {
    off_sf = stage_bytes * uint32_t(stages);
    off_ep = off_sf + (fp8 ? kLrScaleBufs * kLrScaleBytes : 0u);
    off_bar = off_ep + 4u * uint32_t(ep_bufs) * kEpBufBytes;
    total = off_bar + 512;
  }
};

// Warps 0 TMA, 1 MMA, 2-5 epilogue, and with DROP 6-13 the mask: with the
// epilogue's warps for it a tile of 1024 contracted values took 7.5 us, mask
// and store one after the other, where its products take 5.
constexpr int lr_threads(bool drop) { return kFusedThreads + (drop ? 256 : 0); }

template <bool FP8, bool MN, bool DROP, int BN>
__global__ void __launch_bounds__(lr_threads(DROP), 1)
    lowrank_gemm_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                        const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmPS,
                        const __grid_constant__ CUtensorMap tmQS, const __grid_constant__ LrArgs la) {
  static_assert(BN % 32 == 0 && 2 * BN + (FP8 ? 16 * kLrScaleBufs : 0) <= 512, "TMEM");
  static_assert(!DROP || MN, "only dX masks its rank product");
  using Sh = LrShape<FP8, MN, BN>;
  using G = Group<2>;
  constexpr int BNC = Sh::kBNC;
  constexpr int kStageK = FP8 ? 128 : 64;
  const FusedArgs& a = la.f;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (sbase - raw);
  const LrLayout L(Sh::kStage, FP8, a.stages, a.ep_bufs);
  const int S = a.stages;
  const uint32_t bar0 = sbase + L.off_bar;
  // full, accempty, masked and drain are used on the even CTA only
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  const uint32_t accfull0 = bar0 + 8u * (2 * S);        // +8*b
  const uint32_t accempty0 = bar0 + 8u * (2 * S + 2);   // +8*b
  const uint32_t rankfull = bar0 + 8u * (2 * S + 4);    // DROP: a rank product is in its accumulator
  const uint32_t masked = bar0 + 8u * (2 * S + 5);      // DROP: ... and masked
  const uint32_t drain = bar0 + 8u * (2 * S + 6);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + L.off_bar + 8 * (2 * S + 7));
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accfull0 + 8u * b, 1);
      mbar_init(accempty0 + 8u * b, 8);
    }
    mbar_init(rankfull, 1);
    mbar_init(masked, 16);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmU);
    tma_prefetch_desc(&tmV);
    if constexpr (FP8) {
      tma_prefetch_desc(&tmPS);
      tma_prefetch_desc(&tmQS);
    }
  }
  if (warp == 2 && lane == 0) tma_prefetch_desc(&tmO);
  if (warp == 1) G::alloc(smem_addr(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  G::cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (la.late_wait == 0) {
    griddep_wait();
    griddep_launch_dependents();
  }

  const int nk = (a.K + kStageK - 1) / kStageK;
  const int nr = (a.r_pad + 63) / 64;  // rank blocks
  // DROP: the next tile's rank blocks go before this base block
  const int ahead = nk / 2;
  const uint64_t lim = a.wait_limit_ns;
  const int n_clusters = int(gridDim.x) / 2;
  const int cluster_id = int(blockIdx.x) / 2;

  if (warp == 0) {
    // ------------------------------------------------ TMA producer ----
    if (lane == 0) {
      LrSched sch(la, n_clusters, cluster_id);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t sf_n = 0;                      // scale groups so far
      const int groups = (nk + 3) / 4, p_blocks = (a.M + 127) / 128;
      auto claim = [&](uint32_t bytes, uint32_t& st, uint32_t& fb) -> bool {
        if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, lim, SITE_EMPTY, true)) return false;
        st = sbase + uint32_t(stage) * Sh::kStage;
        fb = G::leader_addr(full_bar(stage));
        if (leader) mbar_arrive_expect_tx(full_bar(stage), 2u * bytes);
        if (++stage == S) { stage = 0; phase ^= 1u; }
        return true;
      };
      auto rank_blocks = [&](int m, int n) -> bool {
        const int row0 = m * 256 + int(rank) * kBM;
        const int q0 = n * BN + int(rank) * BNC;
        for (int rb = 0; rb < nr; ++rb) {
          uint32_t st, fb;
          if (!claim(16384u + Sh::kQRank, st, fb)) return false;
          G::load(st, &tmU, fb, rb * 64, row0);
          if constexpr (!MN) {
            G::load(st + 16384u, &tmV, fb, rb * 64, q0);
          } else {
#pragma unroll
            for (int i = 0; i < Sh::kChunks; ++i)
              G::load(st + 16384u + uint32_t(i) * 8192u, &tmV, fb, q0 + 64 * i, rb * 64);
          }
        }
        return true;
      };
      auto base_blocks = [&](int m, int n, int from, int to) -> bool {
        const int row0 = m * 256 + int(rank) * kBM;
        const int q0 = n * BN + int(rank) * BNC;
        for (int kb = from; kb < to; ++kb) {
          uint32_t st, fb;
          const bool scales = FP8 && (kb & 3) == 0;
          if (!claim(16384u + Sh::kQBase + (scales ? kLrScaleBytes : 0u), st, fb)) return false;
          const int k0 = kb * kStageK;
          if constexpr (FP8) {
            if (scales) {
              const uint32_t sf = sbase + L.off_sf + (sf_n++ % kLrScaleBufs) * kLrScaleBytes;
              G::load(sf, &tmPS, fb, 0, (kb >> 2) * p_blocks + 2 * m + int(rank));
              G::load(sf + 512u, &tmQS, fb, 0, 2 * (n * groups + (kb >> 2)));
            }
          }
          G::load(st, &tmP, fb, k0, row0);
          if constexpr (!MN) {
            G::load(st + 16384u, &tmQ, fb, k0, q0);
          } else if constexpr (FP8) {
            G::load(st + 16384u, &tmQ, fb, q0, k0);
          } else {
#pragma unroll
            for (int i = 0; i < Sh::kChunks; ++i)
              G::load(st + 16384u + uint32_t(i) * 8192u, &tmQ, fb, q0 + 64 * i, k0);
          }
        }
        return true;
      };
      int m, n, mn = 0, nn = 0;
      bool have = sch.next(m, n);
      bool ok = !(DROP && have) || rank_blocks(m, n);
      while (ok && have) {
        const bool more = sch.next(mn, nn);
        if constexpr (DROP) {
          ok = base_blocks(m, n, 0, ahead) && (!more || rank_blocks(mn, nn)) && base_blocks(m, n, ahead, nk);
        } else {
          ok = rank_blocks(m, n) && base_blocks(m, n, 0, nk);
        }
        m = mn;
        n = nn;
        have = more;
      }
      if (*abort_flag) settle_ns(200000);  // let copies in flight land
    }
  } else if (warp == 1) {
    // ------------------------------------------------- MMA issuer ----
    if (lane == 0 && leader) {
      const uint32_t id_base = idesc_bf16(256, BN, false, MN);  // also the rank blocks' (V has Q's layout)
      LrSched sch(la, n_clusters, cluster_id);
      int stage = 0;
      uint32_t phase = 0, sf_n = 0, marks = 0;
      uint32_t acc_waits[2] = {0u, 0u};
      // Descriptors of stage 0; a stage's are these plus its offset (in units
      // of 16 bytes: the start address is the descriptor's low field).  This
      // thread's own instructions are what keeps the tensor pipe waiting at
      // 8 bits, so it does as little as it can.
      const uint64_t p_desc = smem_desc(sbase, 16u, 1024u, SWZ_128B);
      const uint64_t v_desc = MN ? smem_desc(sbase + 16384u, 8192u, 1024u, SWZ_128B)   // bf16 (rank blocks, base)
                                 : smem_desc(sbase + 16384u, 16u, 1024u, SWZ_128B);
      const uint64_t q_desc = MN && FP8 ? smem_desc(sbase + 16384u, 16384u, 1024u, SWZ_128B) : v_desc;
      const uint64_t sf_desc = smem_desc(sbase + L.off_sf, 16u, 128u, SWZ_NONE);
      auto take = [&](uint64_t& st) -> bool {
        if (!wait_bounded(full_bar(stage), phase, abort_flag, lim, SITE_FULL, true)) return false;
        tc_fence_after();
        st = uint64_t(uint32_t(stage) * (Sh::kStage >> 4));
        return true;
      };
      auto give = [&]() {
        G::commit_all(empty_bar(stage));
        if (++stage == S) { stage = 0; phase ^= 1u; }
      };
      // waits for the accumulator and starts it with the rank product
      auto rank_blocks = [&](uint32_t b) -> bool {
        const uint32_t w = b ? acc_waits[1]++ : acc_waits[0]++;
        if (!wait_bounded(accempty0 + 8u * b, (w & 1u) ^ 1u, abort_flag, lim, SITE_ACCEMPTY, true)) return false;
        tc_fence_after();
        const uint32_t d = tmem + b * BN;
        for (int rb = 0; rb < nr; ++rb) {
          uint64_t st;
          if (!take(st)) return false;
          const int kk_n = imin(4, (a.r_pad - rb * 64) / 16);
          for (int kk = 0; kk < kk_n; ++kk)
            G::mma(d, p_desc + st + uint32_t(kk) * 2u, v_desc + st + uint32_t(kk) * (MN ? 128u : 2u), id_base,
                   (rb | kk) != 0);
          give();
        }
        if constexpr (DROP) G::commit_all(rankfull);
        return true;
      };
      auto base_blocks = [&](uint32_t b, int from, int to) -> bool {
        const uint32_t d = tmem + b * BN;
        uint32_t sf_tmem = 0;
        if constexpr (FP8) sf_tmem = tmem + 2 * BN + 16u * ((sf_n - 1u) % kLrScaleBufs);
        for (int kb = from; kb < to; ++kb) {
          uint64_t st;
          if (!take(st)) return false;
          if constexpr (FP8) {
            if ((kb & 3) == 0) {
              const uint32_t buf = sf_n++ % kLrScaleBufs;
              sf_tmem = tmem + 2 * BN + 16u * buf;
              const uint64_t src = sf_desc + ((buf * kLrScaleBytes) >> 4);
#pragma unroll
              for (uint32_t i = 0; i < 3; ++i) tmem_cp_scales_pair(sf_tmem + 4u * i, src + 32u * i);
            }
            const uint32_t id = idesc_mxf8(256, BN, false, MN, uint32_t(kb & 3));
#pragma unroll
            for (uint32_t kk = 0; kk < 4; ++kk)
              umma_mxf8_pair(d, p_desc + st + kk * 2u, q_desc + st + kk * (MN ? 256u : 2u), id, sf_tmem, sf_tmem + 4u,
                             1u);
          } else {
#pragma unroll
            for (uint32_t kk = 0; kk < 4; ++kk)
              G::mma(d, p_desc + st + kk * 2u, v_desc + st + kk * (MN ? 128u : 2u), id_base, 1u);
          }
          give();
        }
        return true;
      };
      int m, n;
      bool have = sch.next(m, n);
      uint32_t b = 0;
      bool ok = !(DROP && have) || rank_blocks(0);
      while (ok && have) {
        const bool more = sch.next(m, n);
        if constexpr (DROP) {
          ok = wait_bounded(masked, marks++ & 1u, abort_flag, lim, SITE_STFULL, true);
          tc_fence_after();
          ok = ok && base_blocks(b, 0, ahead) && (!more || rank_blocks(b ^ 1u)) && base_blocks(b, ahead, nk);
        } else {
          ok = rank_blocks(b) && base_blocks(b, 0, nk);
        }
        if (!ok) break;
        G::commit_all(accfull0 + 8u * b);
        b ^= 1u;
        have = more;
      }
      // make sure no tcgen05 op is still running before TMEM is released
      G::commit_local(drain);
      wait_bounded(drain, 0u, abort_flag, lim, SITE_DRAIN, false);
    }
  } else if (warp < 6) {
    // ---------------------------------------------------- epilogue ----
    const int q = warp & 3;            // TMEM lane quarter of this warp
    const uint32_t lane_base = uint32_t(q * 32) << 16;
    LrSched sch(la, n_clusters, cluster_id);
    uint32_t full_waits[2] = {0u, 0u};
    const uint32_t ep_off = L.off_ep + uint32_t(q * a.ep_bufs) * kEpBufBytes;
    uint32_t epc = 0;  // output blocks staged so far
    int m, n;
    uint32_t b = 0;
    while (sch.next(m, n)) {
      const uint32_t fpar = (b ? full_waits[1]++ : full_waits[0]++) & 1u;
      if (!warp_wait_bounded(accfull0 + 8u * b, fpar, abort_flag, lim, SITE_ACCFULL, true)) break;
      tc_fence_after();
      const int wrow0 = m * 256 + int(rank) * kBM + q * 32;
#pragma unroll 1
      for (int ch = 0; ch < BN / kEpCols; ++ch) {
        uint32_t v[32];
        tmem_ld_x32(tmem + lane_base + b * BN + uint32_t(ch * kEpCols), v);
        tmem_ld_wait();
        const int col0 = n * BN + ch * kEpCols;
        if (col0 >= a.N || wrow0 >= a.M) continue;
        uint4 pk[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          pk[g].x = pack_bf16x2(__uint_as_float(v[8 * g + 0]), __uint_as_float(v[8 * g + 1]));
          pk[g].y = pack_bf16x2(__uint_as_float(v[8 * g + 2]), __uint_as_float(v[8 * g + 3]));
          pk[g].z = pack_bf16x2(__uint_as_float(v[8 * g + 4]), __uint_as_float(v[8 * g + 5]));
          pk[g].w = pack_bf16x2(__uint_as_float(v[8 * g + 6]), __uint_as_float(v[8 * g + 7]));
        }
        // the store that last used this buffer has read it
        if (lane == 0) {
          if (a.ep_bufs == 2) bulk_wait_group_read1();
          else bulk_wait_group_read0();
        }
        __syncwarp();
        const uint32_t bo = ep_off + (a.ep_bufs == 2 ? (epc & 1u) * kEpBufBytes : 0u);
        ++epc;
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<uint4*>(gbase + bo + swz_offset(uint32_t(lane), uint32_t(g), kEpCols * 2)) = pk[g];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tmO, sbase + bo, col0, wrow0);
          bulk_commit_group();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) G::arrive_leader(accempty0 + 8u * b);
      b ^= 1u;
    }
    if (lane == 0) bulk_wait_group0();  // every output store has completed
  } else if constexpr (DROP) {
    // -------------------------------------------------------- mask ----
    // Two warps a lane quarter, every other 32 columns each.
    const int q = warp & 3;
    const uint32_t lane_base = uint32_t(q * 32) << 16;
    LrSched sch(la, n_clusters, cluster_id);
    const DropState ds = drop_load(la.drop);
    int m, n;
    uint32_t tiles = 0;
    while (sch.next(m, n)) {
      const uint32_t b = tiles & 1u;
      if (!warp_wait_bounded(rankfull, tiles & 1u, abort_flag, lim, SITE_TFULL, true)) break;
      ++tiles;
      tc_fence_after();
      const uint32_t row = uint32_t(m * 256 + int(rank) * kBM + q * 32 + lane);
#pragma unroll 1
      for (int ch = (warp - 6) >> 2; ch < BN / 32; ch += 2) {
        const uint32_t col = tmem + lane_base + b * BN + uint32_t(ch * 32);
        uint32_t v[32];
        tmem_ld_x32(col, v);
        const uint32_t c8 = uint32_t(n * BN + ch * 32) / 8u;
        uint4 r[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) r[g] = drop_block(ds, c8 + g, row);
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t w[4] = {r[g].x, r[g].y, r[g].z, r[g].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float lo = __uint_as_float(v[8 * g + 2 * i]) * la.drop.inv_keep;
            const float hi = __uint_as_float(v[8 * g + 2 * i + 1]) * la.drop.inv_keep;
            v[8 * g + 2 * i] = (w[i] << 16) < ds.thr_hi ? 0u : __float_as_uint(lo);
            v[8 * g + 2 * i + 1] = w[i] < ds.thr_hi ? 0u : __float_as_uint(hi);
          }
        }
        tmem_st_x32(col, v);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) G::arrive_leader(masked);
    }
  }

  if (la.late_wait != 0) {  // what follows this kernel may rely on all that came before it
    griddep_wait();
    griddep_launch_dependents();
  }
  tc_fence_before();
  __syncthreads();
  G::cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    G::dealloc(tmem, 512);
  }
}

}  // namespace lora
