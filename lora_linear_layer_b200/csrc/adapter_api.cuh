// adapter_api.cuh - entry points of the adapter with dropout and of the
// 8-bit base: argument rules, launch configuration, launches.
// Part of the single translation unit built from lora_api.cu.
#pragma once

#include "adapter_pass.cuh"
#include "lowrank_gemm.cuh"
#include "token.cuh"

namespace {

// ------------------------------------------------------------- arguments ----

// p and rng -> the mask's arguments.  p == 0 is no dropout (rng is ignored).
lora_status_t drop_args(float p, const void* rng, DropArgs& d) {
  d = DropArgs{nullptr, 0u, 1.0f};
  if (!(p >= 0.0f) || p >= 1.0f) return LORA_ERR_DROPOUT;
  const int thr = int(double(p) * 65536.0 + 0.5);
  if (thr > 65535) return LORA_ERR_DROPOUT;
  if (p == 0.0f) return LORA_OK;
  if (rng == nullptr) return LORA_ERR_DROPOUT;
  if (!aligned16(rng)) return LORA_ERR_ALIGN;
  d.rng = reinterpret_cast<const uint64_t*>(rng);
  d.thr = uint32_t(thr);
  d.inv_keep = float(65536.0 / double(65536 - thr));
  return LORA_OK;
}

int64_t qblocks(int64_t n) { return (n + kQBlock - 1) / kQBlock; }

lora_status_t check_sizes_fp8(int64_t M, int64_t d_in, int64_t d_out, int32_t r) {
  const lora_status_t s = check_sizes(M, d_in, d_out, r);
  if (s != LORA_OK) return s;
  return (d_in % 16) != 0 || (d_out % 16) != 0 ? LORA_ERR_SHAPE : LORA_OK;
}

// The 8-bit layer's workspace: T and dT as the backward's, then the codes of
// X or dY, their scales and the weight's as the product reads them.
struct Fp8Workspace {
  size_t off_codes, off_scales, off_atoms, total;
};

// Scale atoms of a product's N columns (tiles are at least 128 wide) over K.
size_t atom_bytes(int64_t N, int64_t K) { return size_t((N + 127) / 128) * size_t((K + 511) / 512) * 1024; }

Fp8Workspace fp8_workspace(int64_t M, int64_t d_in, int64_t d_out, int32_t r) {
  const size_t wide = size_t(std::max(d_in, d_out));
  Fp8Workspace w;
  w.off_codes = bwd_workspace(M, r).total;
  w.off_scales = w.off_codes + align256(size_t(M) * wide);
  w.off_atoms = w.off_scales + size_t((M + 127) / 128) * ((wide + 511) / 512) * 512;
  w.total = w.off_atoms + std::max(atom_bytes(d_out, d_in), atom_bytes(d_in, d_out));
  return w;
}

// Base weight of a call: bf16 (scales NULL) or e4m3 codes with block scales.
struct Base {
  const void* w;
  const void* scales;
  bool fp8() const { return scales != nullptr; }
};

// -------------------------------------------------------- adapter passes ----

struct PassCfg {
  int RCW;
  uint32_t smem;
  PassArgs args;
};

// Three stages where two blocks share an SM (37 KB each at r = 16), else as
// many as fit, at most six.  The splits of a row tile form one cluster: as many
// as fill the block slots that shared memory and threads leave, at most 8 and
// at least 256 values of the contraction each.
// For dA and dB (66 registers, 320 threads) these are more slots than there
// are: shared memory has room for 3 or 4 blocks, the registers for 2.  The
// blocks past the resident ones even out the masked row tiles of dA and the
// cheaper ones of dB.  With the slots held to 2 an SM the launch takes 290-320
// us against 230-240 on 16384 x 4096 x 14336, r = 64, p = 0.1, and 67 against
// 58-63 on 8192 x 4096 x 4096, r = 16; less only where a few row tiles remain
// (2400 x 4096 x 4096, r = 32, no mask: 24 against 30).  (The occupancy query
// does not say how many are resident: for a kernel that allocates tensor memory
// it answers one block an SM, where two and three were seen to run.)
void pick_pass(int64_t rows, int64_t K, int r, bool p_mn, bool r_mn, bool quant, int out_mode, int64_t launch_tiles,
               int sm_count, PassCfg& c) {
  const int r_pad = r_pad_of(r);
  c.RCW = rcw_of(r_pad);
  PassArgs& a = c.args;
  std::memset(&a, 0, sizeof(a));
  a.n_rchunks = (r_pad + c.RCW - 1) / c.RCW;
  auto smem = [&](int stages) { return PassLayout(p_mn, r_mn, c.RCW, r_pad, a.n_rchunks, stages).total + 1024; };
  a.stages = pass_workers(c.RCW, p_mn, quant) == 16 ? 6 : 3;
  while (a.stages > 2 && smem(a.stages) > kSmemMax) --a.stages;
  c.smem = smem(a.stages);
  const int per_sm =
      std::max(1, std::min<int>(int(kSmemPerSM / (c.smem + 1024)), 2048 / pass_threads(c.RCW, p_mn, quant)));
  const int block_k = p_mn ? 64 : 128;
  const int nb = int((K + block_k - 1) / block_k);
  const int tiles = int(std::max<int64_t>(1, launch_tiles));
  // One block an SM: two clusters of 8 fit most GPCs, 15 the chip (and 15 of 7,
  // 22 of 6, 33 of 4), so that 17 row tiles took two rounds, 28 us on
  // X[2051, 2560] at r = 128 against 15-17 us in fours; sixes are no faster
  // (14.5, and dT 22 in either).
  const int most = per_sm == 1 && tiles > 14 ? 4 : 8;
  int splits = std::max(1, std::min({per_sm * sm_count / tiles, most, std::max(1, nb * block_k / 256)}));
  a.nb_per_split = std::max(1, (nb + splits - 1) / splits);
  splits = std::max(1, (nb + a.nb_per_split - 1) / a.nb_per_split);
  a.rows = int32_t(rows);
  a.K = int32_t(K);
  a.r_pad = r_pad;
  a.r = r;
  a.splits = splits;
  a.out_mode = out_mode;
  a.r_mn = r_mn ? 1 : 0;
  a.scale = 1.0f;
  a.drop = DropArgs{nullptr, 0u, 1.0f};
  a.wait_limit_ns = kWaitLimitNs;
}

// Two jobs of one launch share its split count.
void resplit_pass(PassCfg& c, int splits, bool p_mn) {
  const int block_k = p_mn ? 64 : 128;
  const int nb = int((int64_t(c.args.K) + block_k - 1) / block_k);
  c.args.splits = splits;
  c.args.nb_per_split = std::max(1, (nb + splits - 1) / splits);
}

struct PassMaps {
  CUtensorMap p, r;
};

constexpr int kAtomBlocks = 16;  // blocks (times the splits) that lay out the weight's scales

template <bool P_MN, int RCW, bool QUANT>
lora_status_t launch_pass_t(const PassMaps& m0, const PassCfg& c0, const PassMaps* m1, const PassCfg* c1,
                            const ScaleAtomArgs& atoms, cudaStream_t st) {
  auto kern = adapter_pass_kernel<P_MN, RCW, QUANT>;
  const uint32_t smem = c1 != nullptr ? std::max(c0.smem, c1->smem) : c0.smem;
  if (!ensure_smem_attr(kern, smem)) return LORA_ERR_CUDA;
  const int t0 = int((int64_t(c0.args.rows) + 127) / 128);
  const int t1 = c1 != nullptr ? int((int64_t(c1->args.rows) + 127) / 128) : 0;
  const dim3 cl(1, unsigned(c0.args.splits), 1);
  const PassMaps& second = m1 != nullptr ? *m1 : m0;
  const int ta = atoms.bytes != nullptr ? kAtomBlocks : 0;
  return launch_ex("adapter pass", kern, dim3(unsigned(t0 + t1 + ta), unsigned(c0.args.splits)), dim3(pass_threads(RCW, P_MN, QUANT)),
                   smem, st, &cl, m0.p, m0.r, second.p, second.r, c0.args, c1 != nullptr ? c1->args : c0.args,
                   int32_t(t0), int32_t(t0 + t1), atoms);
}

template <bool P_MN, bool QUANT>
lora_status_t launch_pass(const PassMaps& m0, const PassCfg& c0, cudaStream_t st, const PassMaps* m1 = nullptr,
                          const PassCfg* c1 = nullptr, const ScaleAtomArgs& atoms = ScaleAtomArgs{}) {
  if (c0.RCW == 16) return launch_pass_t<P_MN, 16, QUANT>(m0, c0, m1, c1, atoms, st);
  if (c0.RCW == 32) return launch_pass_t<P_MN, 32, QUANT>(m0, c0, m1, c1, atoms, st);
  return launch_pass_t<P_MN, 64, QUANT>(m0, c0, m1, c1, atoms, st);
}

// What a pass over an 8-bit layer's operand leaves for the product.
struct Rounded {
  uint8_t* codes;
  uint8_t* scales;
  ScaleAtomArgs atoms;  // the weight's scales, to be laid out beside
};

// T = scale (m * X) A^T into `Tws`; with `q`, X's codes and scales too.
lora_status_t launch_down(const void* X, const void* A, int64_t M, int64_t d_in, int32_t r, float scale,
                          const DropArgs& drop, __nv_bfloat16* Tws, const Rounded* q, int sm_count, cudaStream_t st) {
  PassCfg c;
  pick_pass(M, d_in, r, false, false, q != nullptr, OUT_ROWS_RPAD, (M + 127) / 128, sm_count, c);
  c.args.out = Tws;
  c.args.scale = scale * drop.inv_keep;
  c.args.drop = drop;
  PassMaps m;
  if (!make_map(&m.p, X, d_in, M, d_in, 64, 128, 128) ||
      !make_map(&m.r, A, d_in, r, d_in, 64, uint32_t(c.args.r_pad), 128))
    return LORA_ERR_CUDA;
  if (q == nullptr) return launch_pass<false, false>(m, c, st);
  c.args.codes = q->codes;
  c.args.scales = q->scales;
  return launch_pass<false, true>(m, c, st, nullptr, nullptr, q->atoms);
}

// -------------------------------------------------------- low-rank GEMMs ----

struct LrCfg {
  int BN;
  uint32_t smem;
  LrArgs args;
};

uint32_t lr_stage_bytes(bool fp8, bool mn, int BN) {
  if (fp8) {
    return mn ? (BN == 224 ? LrShape<true, true, 224>::kStage : LrShape<true, true, 128>::kStage)
              : (BN == 224 ? LrShape<true, false, 224>::kStage : LrShape<true, false, 128>::kStage);
  }
  return mn ? (BN == 256 ? LrShape<false, true, 256>::kStage : LrShape<false, true, 128>::kStage)
            : (BN == 256 ? LrShape<false, false, 256>::kStage : LrShape<false, false, 128>::kStage);
}

// OUT[M, N] over the contraction K: the wide tile (224 columns for 8 bits,
// 256 for bf16) or 128 columns, whichever needs fewer rounds of the clusters.
// A round takes nearly the same time with either (what bounds one tile a pair
// is its operands' way from L2; X[2048, 4096], N = 4096: 4 rounds of 128 in 49
// us, 3 of 224 in 38 us at 8 bits, 4 in 81 and 2 of 256 in 50 us for bf16); at
// equal rounds the narrow one is a little shorter (512 x 4096 x 4096 bf16: 25
// against 28 us).
void pick_lr(int64_t M, int64_t N, int64_t K, int r, bool fp8, bool mn, int sm_count, LrCfg& c) {
  const int64_t clusters = sm_count / 2;
  const int64_t num_m = (M + 255) / 256;
  auto cost = [&](int bn) {
    const int64_t tiles = num_m * ((N + bn - 1) / bn);
    return ((tiles + clusters - 1) / clusters) * int64_t(bn + 1024);
  };
  const int wide = fp8 ? 224 : 256;
  c.BN = cost(128) < cost(wide) ? 128 : wide;
  const uint32_t stage = lr_stage_bytes(fp8, mn, c.BN);
  auto stages_for = [&](int ep_bufs) {
    return std::min(fp8 ? kLrMaxStagesFp8 : 8, int((kSmemMax - LrLayout(stage, fp8, 0, ep_bufs).total - 1024) / stage));
  };
  std::memset(&c.args, 0, sizeof(c.args));
  FusedArgs& a = c.args.f;
  a.stages = stages_for(1);
  a.ep_bufs = stages_for(2) >= a.stages ? 2 : 1;
  c.smem = LrLayout(stage, fp8, a.stages, a.ep_bufs).total + 1024;
  a.M = int32_t(M);
  a.N = int32_t(N);
  a.K = int32_t(K);
  a.r_pad = r_pad_of(r);
  a.scale = 1.0f;
  a.num_m = int32_t(num_m);
  a.num_n = int32_t((N + c.BN - 1) / c.BN);
  // as many M blocks together as keep their rows of P in about a third of
  // the 126 MB L2
  const int64_t block_bytes = 256 * K * (fp8 ? 1 : 2);
  c.args.group_m = int32_t(std::max<int64_t>(1, std::min<int64_t>({num_m, 16, (int64_t(40) << 20) / block_bytes})));
  a.wait_limit_ns = kWaitLimitNs;
  c.args.drop = DropArgs{nullptr, 0u, 1.0f};
}

template <bool FP8, bool MN, bool DROP, int BN>
lora_status_t launch_lr_t(const CUtensorMap* maps, const LrCfg& c, int sm_count, cudaStream_t st) {
  auto kern = lowrank_gemm_kernel<FP8, MN, DROP, BN>;
  if (!ensure_smem_attr(kern, c.smem)) return LORA_ERR_CUDA;
  const int64_t tiles = int64_t(c.args.f.num_m) * c.args.f.num_n;
  const int clusters = int(std::min<int64_t>(tiles, max_clusters(kern, 2, c.smem, sm_count)));
  const dim3 cl(2, 1, 1);
  return launch_ex("low-rank GEMM", kern, dim3(unsigned(clusters * 2)), dim3(lr_threads(DROP)), c.smem, st, &cl,
                   maps[0], maps[1], maps[2], maps[3], maps[4], maps[5], maps[6], c.args);
}

template <bool MN, bool DROP>
lora_status_t launch_lr(bool fp8, const CUtensorMap* maps, const LrCfg& c, int sm_count, cudaStream_t st) {
  if (fp8)
    return c.BN == 224 ? launch_lr_t<true, MN, DROP, 224>(maps, c, sm_count, st)
                       : launch_lr_t<true, MN, DROP, 128>(maps, c, sm_count, st);
  return c.BN == 256 ? launch_lr_t<false, MN, DROP, 256>(maps, c, sm_count, st)
                     : launch_lr_t<false, MN, DROP, 128>(maps, c, sm_count, st);
}

// The product's view of the weight's scales: columns of the forward are rows
// of W, those of dX columns.
ScaleAtomArgs scale_atom_args(const Base& W, const Rounded& q, const LrCfg& c, bool mn, int64_t d_in, int64_t d_out) {
  ScaleAtomArgs a;
  const int32_t out_b = int32_t(qblocks(d_out)), in_b = int32_t(qblocks(d_in));
  a.bytes = reinterpret_cast<const uint8_t*>(W.scales);
  a.atoms = q.atoms.atoms;
  a.tiles = c.args.f.num_n;
  a.groups = (c.args.f.K + 511) / 512;
  a.bn = c.BN;
  a.n_blocks = mn ? in_b : out_b;
  a.k_blocks = mn ? out_b : in_b;
  a.ld_n = mn ? 1 : in_b;
  a.ld_k = mn ? in_b : 1;
  return a;
}

bool scale_maps(CUtensorMap* maps, const Rounded& q, const LrCfg& c) {
  const uint64_t groups = uint64_t((c.args.f.K + 511) / 512);
  return make_map_atoms(&maps[0], q.scales, groups * uint64_t((c.args.f.M + 127) / 128), 1) &&
         make_map_atoms(&maps[1], q.atoms.atoms, groups * uint64_t(c.args.f.num_n) * 2, 2);
}

// Y = X W^T + T B^T from T (bf16 [M, r_pad], scale included); for an 8-bit
// base from X's codes in `q`.
lora_status_t launch_up(const void* X, const Rounded& q, const Base& W, const void* B, void* Y,
                        const __nv_bfloat16* Tws, const LrCfg& c, int32_t r, int sm_count, cudaStream_t st) {
  const int64_t M = c.args.f.M, d_in = c.args.f.K, d_out = c.args.f.N;
  const bool fp8 = W.fp8();
  const uint32_t bnc = uint32_t(c.BN / 2);
  const uint64_t r_pad = uint64_t(r_pad_of(r));
  CUtensorMap maps[7];
  const bool ok = fp8 ? make_map_u8(&maps[0], q.codes, d_in, M, d_in, 128, 128) &&
                            make_map_u8(&maps[1], W.w, d_in, d_out, d_in, 128, bnc) && scale_maps(maps + 5, q, c)
                      : make_map(&maps[0], X, d_in, M, d_in, 64, 128, 128) &&
                            make_map(&maps[1], W.w, d_in, d_out, d_in, 64, bnc, 128);
  if (!ok || !make_map(&maps[2], Tws, r_pad, M, r_pad, 64, 128, 128) ||
      !make_map(&maps[3], B, r, d_out, r, 64, bnc, 128) ||
      !make_map(&maps[4], Y, d_out, M, d_out, kEpCols, 32, kEpCols * 2))
    return LORA_ERR_CUDA;
  if (!fp8) maps[5] = maps[6] = maps[0];  // (unused)
  return launch_lr<false, false>(fp8, maps, c, sm_count, st);
}

// dX = dY W + m * (dT A)/(1-p); for an 8-bit base from dY's codes in `q`.
lora_status_t launch_dx(const void* dY, const Rounded& q, const Base& W, const void* A, void* dX,
                        const __nv_bfloat16* dTws, const LrCfg& c, int32_t r, int sm_count, cudaStream_t st) {
  const int64_t M = c.args.f.M, d_in = c.args.f.N, d_out = c.args.f.K;
  const bool fp8 = W.fp8();
  const uint64_t r_pad = uint64_t(r_pad_of(r));
  CUtensorMap maps[7];
  const bool ok = fp8 ? make_map_u8(&maps[0], q.codes, d_out, M, d_out, 128, 128) &&
                            make_map_u8(&maps[1], W.w, d_in, d_out, d_in, 128, 128) && scale_maps(maps + 5, q, c)
                      : make_map(&maps[0], dY, d_out, M, d_out, 64, 128, 128) &&
                            make_map(&maps[1], W.w, d_in, d_out, d_in, 64, 64, 128);
  if (!ok || !make_map(&maps[2], dTws, r_pad, M, r_pad, 64, 128, 128) ||
      !make_map(&maps[3], A, d_in, r, d_in, 64, 64, 128) ||
      !make_map(&maps[4], dX, d_in, M, d_in, kEpCols, 32, kEpCols * 2))
    return LORA_ERR_CUDA;
  if (!fp8) maps[5] = maps[6] = maps[0];  // (unused)
  return c.args.drop.rng != nullptr ? launch_lr<true, true>(fp8, maps, c, sm_count, st)
                                    : launch_lr<true, false>(fp8, maps, c, sm_count, st);
}

// -------------------------------------------------------------- tokens ----

// Whether launch_prep is used: its blocks read X again for every 16 rank
// rows, which costs less than the pass's long prologue and few blocks up to
// M * r_pad = 8192 (X[512, 8192] at r = 16: 14 against 18 us; at M = 1024 they
// tie, and X[512, 4096] at r = 128 takes 29 against 17 us).
bool use_prep(int64_t M, int32_t r) { return M * r_pad_of(r) <= 8192; }

// T and, with `q`, the codes of X for few tokens.
lora_status_t launch_prep(const void* X, const void* A, int64_t M, int64_t d_in, int32_t r, float scale,
                          const DropArgs& drop, __nv_bfloat16* Tws, const Rounded* q, cudaStream_t st) {
  PrepArgs p;
  std::memset(&p, 0, sizeof(p));
  p.X = reinterpret_cast<const uint8_t*>(X);
  p.A = reinterpret_cast<const uint8_t*>(A);
  p.T = Tws;
  p.drop = drop;
  p.M = int32_t(M);
  p.K = int32_t(d_in);
  p.r = r;
  p.r_pad = r_pad_of(r);
  p.t_blocks = kPrepSplits * (p.r_pad / kPrepRanks) * ((p.M + kPrepTokens - 1) / kPrepTokens);
  p.scale = scale * drop.inv_keep;
  auto blocks = [](int64_t items) {  // whole clusters of blocks, a warp an item
    return (items + kPrepWarps * kPrepSplits - 1) / (kPrepWarps * kPrepSplits) * kPrepSplits;
  };
  int64_t a_blocks = 0;
  if (q != nullptr) {
    p.codes = q->codes;
    p.scales = q->scales;
    p.atoms = q->atoms;
    p.q_blocks = int32_t(blocks(M * ((d_in + 511) / 512)));
    if (q->atoms.bytes != nullptr) a_blocks = blocks(int64_t(q->atoms.tiles) * q->atoms.groups * 2);
  }
  const unsigned grid = unsigned(p.t_blocks + p.q_blocks + a_blocks);
  const dim3 cl(kPrepSplits, 1, 1);
  return launch_ex("token prep", token_prep_kernel, dim3(grid), dim3(kPrepThreads), 0, st, &cl, p);
}

template <bool FP8, bool MN, bool DROP>
lora_status_t launch_stream_t(const CUtensorMap* maps, const StreamArgs& a, int tiles, uint32_t smem, cudaStream_t st) {
  auto kern = token_stream_kernel<FP8, MN, DROP>;
  if (!ensure_smem_attr(kern, smem)) return LORA_ERR_CUDA;
  const dim3 cl(1, unsigned(a.splits), 1);
  return launch_ex("token stream", kern, dim3(unsigned(tiles), unsigned(a.splits)), dim3(kStreamThreads), smem, st, &cl,
                   maps[0], maps[1], maps[2], maps[3], a);
}

// Few enough tokens for launch_stream (`drop`: the product masks its rank
// side).  Above 128 tokens its blocks' way out, 128 rows by every token, costs
// as much as a short contraction (X[223, 288], N = 1664 at 8 bits: 21 us
// against 9 us by tiles; [256, 4096], N = 4096: 22 against 17 us), and it
// pays for splitting a long one alone ([256, 14336], N = 4096: 32 against 74);
// K = 6144 lies between these two.
bool use_stream(int64_t M, int64_t K, bool drop) {
  return M <= 128 || (M <= (drop ? kStreamMaxDrop : kStreamMax) && K > 6144);
}

// Y (mn = false, from T in `U`) or dX (mn = true, from dT in `U`) for few
// tokens; `in` is X or dY.
lora_status_t launch_stream(bool mn, const void* in, const Rounded& q, const Base& W, const void* V, void* out,
                            const __nv_bfloat16* U, int64_t M, int64_t d_in, int64_t d_out, int32_t r,
                            const DropArgs& drop, int sm_count, cudaStream_t st) {
  const bool fp8 = W.fp8(), masked = mn && drop.rng != nullptr;
  const int64_t N = mn ? d_in : d_out, K = mn ? d_out : d_in;
  StreamArgs a;
  std::memset(&a, 0, sizeof(a));
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.M = int32_t(M);
  a.N = int32_t(N);
  a.K = int32_t(K);
  a.r_pad = r_pad_of(r);
  a.tok_pad = (a.M + 15) / 16 * 16;
  a.drop = masked ? drop : DropArgs{nullptr, 0u, 1.0f};
  if (fp8) {
    a.w_scales = reinterpret_cast<const uint8_t*>(W.scales);
    a.x_scales = reinterpret_cast<const uint32_t*>(q.scales);
    a.ws_row = mn ? 1 : int32_t(qblocks(d_in));
    a.ws_k = mn ? int32_t(qblocks(d_in)) : 1;
  }
  const uint32_t stage = StreamLayout(a.tok_pad, 0).stage_bytes;
  const uint32_t fixed = kStreamScaleBufs * kStreamScaleBytes + 2048;
  // two blocks an SM where four stages fit in half of it
  const uint32_t half = kSmemPerSM / 2 - 1024 - fixed;
  a.stages = std::min(8, int((half / stage >= 4 ? half : kSmemMax - fixed) / stage));
  const uint32_t smem = StreamLayout(a.tok_pad, a.stages).total + 1024;
  const int per_sm =
      std::max(1, std::min(int(kSmemPerSM / (smem + 1024)), int(512 / stream_tmem_cols(a.tok_pad, masked))));
  const int tiles = int((N + 127) / 128), block_k = fp8 ? 128 : 64, nk = int((K + block_k - 1) / block_k);
  const int splits = std::max(1, std::min({8, per_sm * sm_count / tiles, nk / 2}));
  a.kb_per_split = (nk + splits - 1) / splits;
  a.splits = (nk + a.kb_per_split - 1) / a.kb_per_split;
  a.wait_limit_ns = kWaitLimitNs;
  const uint32_t box_m = uint32_t(a.tok_pad);
  CUtensorMap maps[4];
  bool ok;
  if (fp8)  // (128 codes x 128 rows either way)
    ok = make_map_u8(&maps[0], W.w, d_in, d_out, d_in, 128, 128) && make_map_u8(&maps[1], q.codes, K, M, K, 128, box_m);
  else
    ok = make_map(&maps[0], W.w, d_in, d_out, d_in, 64, mn ? 64 : 128, 128) &&
         make_map(&maps[1], in, K, M, K, 64, box_m, 128);
  ok = ok && (mn ? make_map(&maps[2], V, d_in, r, d_in, 64, 64, 128) : make_map(&maps[2], V, r, d_out, r, 64, 128, 128)) &&
       make_map(&maps[3], U, uint64_t(a.r_pad), M, uint64_t(a.r_pad), 64, box_m, 128);
  if (!ok) return LORA_ERR_CUDA;
  if (masked)
    return fp8 ? launch_stream_t<true, true, true>(maps, a, tiles, smem, st)
               : launch_stream_t<false, true, true>(maps, a, tiles, smem, st);
  if (mn)
    return fp8 ? launch_stream_t<true, true, false>(maps, a, tiles, smem, st)
               : launch_stream_t<false, true, false>(maps, a, tiles, smem, st);
  return fp8 ? launch_stream_t<true, false, false>(maps, a, tiles, smem, st)
             : launch_stream_t<false, false, false>(maps, a, tiles, smem, st);
}

// --------------------------------------------------------- whole layers ----

// T into the workspace; with an 8-bit base (`q`) X's codes and scales too.
lora_status_t launch_t_codes(const void* X, const void* A, int64_t M, int64_t d_in, int32_t r, float scale,
                             const DropArgs& drop, __nv_bfloat16* Tws, const Rounded* q, int sm_count,
                             cudaStream_t st) {
  if (use_prep(M, r)) return launch_prep(X, A, M, d_in, r, scale, drop, Tws, q, st);
  return launch_down(X, A, M, d_in, r, scale, drop, Tws, q, sm_count, st);
}

// Where a call's intermediate values lie in its workspace.
struct Places {
  __nv_bfloat16 *T, *dT;
  Rounded q;  // (8-bit base)
  Places(void* workspace, int64_t M, int64_t d_in, int64_t d_out, int32_t r) {
    uint8_t* const ws = reinterpret_cast<uint8_t*>(workspace);
    const BwdWorkspace w = bwd_workspace(M, r);
    const Fp8Workspace f = fp8_workspace(M, d_in, d_out, r);
    T = reinterpret_cast<__nv_bfloat16*>(ws + w.off_t);
    dT = reinterpret_cast<__nv_bfloat16*>(ws + w.off_dt);
    q = Rounded{ws + f.off_codes, ws + f.off_scales, ScaleAtomArgs{}};
    q.atoms.atoms = ws + f.off_atoms;
  }
};

// Forward.  Arguments already validated.
lora_status_t adapter_fwd_run(const void* X, const Base& W, const void* A, const void* B, void* Y, int64_t M,
                              int64_t d_in, int64_t d_out, int32_t r, float scale, const DropArgs& drop,
                              void* workspace, cudaStream_t st) {
  DeviceInfo dev;
  lora_status_t s = device_info(dev);
  if (s != LORA_OK || M == 0) return s;
  const int sms = dev.sm_count;
  const bool fp8 = W.fp8(), stream = use_stream(M, d_in, false);
  Places at(workspace, M, d_in, d_out, r);
  LrCfg c;
  if (!stream) pick_lr(M, d_out, d_in, r, fp8, false, sms, c);
  if (fp8 && !stream) at.q.atoms = scale_atom_args(W, at.q, c, false, d_in, d_out);
  if ((s = launch_t_codes(X, A, M, d_in, r, scale, drop, at.T, fp8 ? &at.q : nullptr, sms, st)) != LORA_OK) return s;
  if (stream) return launch_stream(false, X, at.q, W, B, Y, at.T, M, d_in, d_out, r, drop, sms, st);
  c.args.f.out = reinterpret_cast<__nv_bfloat16*>(Y);
  return launch_up(X, at.q, W, B, Y, at.T, c, r, sms, st);
}

// Backward.  Arguments already validated.
//  1. T unless saved, and dT = s dY B (with an 8-bit base also dY's codes);
//  2. dB = dY^T T and dA = dT^T (m * X)/(1-p);
//  3. dX.
lora_status_t adapter_bwd_run(const void* X, const Base& W, const void* A, const void* B, const void* dY, void* dX,
                              void* dA, void* dB, int64_t M, int64_t d_in, int64_t d_out, int32_t r, float scale,
                              const DropArgs& drop, void* workspace, uint32_t flags, cudaStream_t st) {
  const bool f32 = (flags & LORA_BWD_FP32_GRADS) != 0u;
  const bool saved = (flags & LORA_BWD_T_SAVED) != 0u;
  const bool fp8 = W.fp8();
  DeviceInfo dev;
  lora_status_t s = device_info(dev);
  if (s != LORA_OK) return s;
  if (M == 0) {
    const size_t gb = f32 ? 4 : 2;
    if ((s = zero_bytes(dA, size_t(r) * size_t(d_in) * gb, st)) != LORA_OK) return s;
    return zero_bytes(dB, size_t(d_out) * size_t(r) * gb, st);
  }
  const int sms = dev.sm_count;
  Places at(workspace, M, d_in, d_out, r);
  const int r_pad = r_pad_of(r);
  const int rcw = rcw_of(r_pad);

  // (X's codes are not needed here, but this way T is the forward's bit for bit)
  if (!saved &&
      (s = launch_t_codes(X, A, M, d_in, r, scale, drop, at.T, fp8 ? &at.q : nullptr, sms, st)) != LORA_OK)
    return s;
  const bool stream = use_stream(M, d_out, drop.rng != nullptr);
  LrCfg c;
  if (!stream) {
    pick_lr(M, d_in, d_out, r, fp8, true, sms, c);
    c.args.f.out = reinterpret_cast<__nv_bfloat16*>(dX);
    c.args.drop = drop;
    // dA's and dB's launch lies between: it lets dX's go only once dT (and the
    // codes) are complete, and dX shares no buffer that either writes, so dX's
    // tiles fill the SMs that its tail leaves (8-bit step on X[2051, 2560],
    // d_out = 1024: 69.8 -> 68.3 us; large ones the same).
    c.args.late_wait = 1;
  }
  {
    PassCfg p;
    pick_pass(M, d_out, r, false, true, fp8, OUT_ROWS_RPAD, (M + 127) / 128, sms, p);
    p.args.out = at.dT;
    p.args.scale = scale;
    PassMaps m;
    if (!make_map(&m.p, dY, d_out, M, d_out, 64, 128, 128) || !make_map(&m.r, B, r, d_out, r, rcw, 64, rcw * 2))
      return LORA_ERR_CUDA;
    if (fp8) {
      p.args.codes = at.q.codes;
      p.args.scales = at.q.scales;
      if (!stream) at.q.atoms = scale_atom_args(W, at.q, c, true, d_in, d_out);
      s = launch_pass<false, true>(m, p, st, nullptr, nullptr, at.q.atoms);
    } else {
      s = launch_pass<false, false>(m, p, st);
    }
    if (s != LORA_OK) return s;
  }
  {
    // One launch, dA's row tiles first: with a mask a stage of theirs takes
    // twice dB's time (16384 x 4096 x 14336, r = 64, p = 0.1: 142 us against
    // 215 us with dB's first, and 187 us as two launches).
    PassCfg cb, ca;
    const int64_t tiles = (d_out + 127) / 128 + (d_in + 127) / 128;
    pick_pass(d_in, M, r, true, true, false, OUT_COLS_R, tiles, sms, ca);
    pick_pass(d_out, M, r, true, true, false, OUT_ROWS_R, tiles, sms, cb);
    resplit_pass(cb, ca.args.splits, true);
    cb.args.out = reinterpret_cast<__nv_bfloat16*>(dB);
    cb.args.out_f32 = f32 ? 1 : 0;
    ca.args.out = reinterpret_cast<__nv_bfloat16*>(dA);
    ca.args.out_f32 = f32 ? 1 : 0;
    ca.args.scale = drop.inv_keep;
    ca.args.drop = drop;
    PassMaps mb, ma;
    if (!make_map(&mb.p, dY, d_out, M, d_out, 64, 64, 128) ||
        !make_map(&mb.r, at.T, r_pad, M, r_pad, rcw, 64, rcw * 2) ||
        !make_map(&ma.p, X, d_in, M, d_in, 64, 64, 128) ||
        !make_map(&ma.r, at.dT, r_pad, M, r_pad, rcw, 64, rcw * 2))
      return LORA_ERR_CUDA;
    if ((s = launch_pass<true, false>(ma, ca, st, &mb, &cb)) != LORA_OK) return s;
  }
  if (stream) return launch_stream(true, dY, at.q, W, A, dX, at.dT, M, d_in, d_out, r, drop, sms, st);
  return launch_dx(dY, at.q, W, A, dX, at.dT, c, r, sms, st);
}

// Pointer and workspace rules of the four layer entry points (sizes already
// checked); `grads`: dY, dX, dA, dB or NULL for a forward.
lora_status_t check_adapter(const void* X, const Base& W, const void* A, const void* B, void* Y, const void* dY,
                            void* dX, void* dA, void* dB, const DropArgs& drop, int64_t M, int64_t d_in,
                            int64_t d_out, int32_t r, int gb, void* workspace, size_t workspace_bytes, bool fwd) {
  const bool fp8 = W.fp8(), rows = M > 0;
  const uint64_t m = uint64_t(M), k = uint64_t(d_in), n = uint64_t(d_out), rr = uint64_t(r);
  const size_t need = !rows ? 0 : fp8 ? fp8_workspace(M, d_in, d_out, r).total : bwd_workspace(M, r).total;
  const BufSpec in[7] = {{X, m * k * 2, rows},
                         {W.w, k * n * (fp8 ? 1 : 2), true},
                         {A, rr * k * 2, true},
                         {B, n * rr * 2, true},
                         {dY, m * n * 2, rows && !fwd},
                         {drop.rng, 16, false},
                         {W.scales, uint64_t(qblocks(d_in)) * uint64_t(qblocks(d_out)), fp8}};
  const BufSpec ws{rows ? workspace : nullptr, need, false};
  const BufSpec out_f[2] = {{Y, m * n * 2, rows}, ws};
  const BufSpec out_b[4] = {{dX, m * k * 2, rows}, {dA, rr * k * uint64_t(gb), true},
                            {dB, n * rr * uint64_t(gb), true}, ws};
  const lora_status_t s = fwd ? check_bufs(in, 7, out_f, 2) : check_bufs(in, 7, out_b, 4);
  if (s != LORA_OK) return s;
  return check_workspace(workspace, workspace_bytes, need);
}

}  // namespace

extern "C" {

lora_status_t lora_fwd_dropout(const void* X, const void* W, const void* A, const void* B, void* Y, int64_t M,
                               int64_t d_in, int64_t d_out, int32_t r, float scale, float p, const void* rng,
                               void* workspace, size_t workspace_bytes, void* stream) {
  lora_status_t s = check_sizes(M, d_in, d_out, r);
  DropArgs drop;
  if (s != LORA_OK || (s = drop_args(p, rng, drop)) != LORA_OK) return s;
  const Base base{W, nullptr};
  if ((s = check_adapter(X, base, A, B, Y, nullptr, nullptr, nullptr, nullptr, drop, M, d_in, d_out, r, 2, workspace,
                         workspace_bytes, true)) != LORA_OK)
    return s;
  return adapter_fwd_run(X, base, A, B, Y, M, d_in, d_out, r, scale, drop, workspace,
                         reinterpret_cast<cudaStream_t>(stream));
}

lora_status_t lora_bwd_dropout(const void* X, const void* W, const void* A, const void* B, const void* dY, void* dX,
                               void* dA, void* dB, int64_t M, int64_t d_in, int64_t d_out, int32_t r, float scale,
                               float p, const void* rng, void* workspace, size_t workspace_bytes, uint32_t flags,
                               void* stream) {
  if ((flags & ~kBwdFlags) != 0u) return LORA_ERR_FLAGS;
  lora_status_t s = check_sizes(M, d_in, d_out, r);
  DropArgs drop;
  if (s != LORA_OK || (s = drop_args(p, rng, drop)) != LORA_OK) return s;
  const Base base{W, nullptr};
  const int gb = (flags & LORA_BWD_FP32_GRADS) != 0u ? 4 : 2;
  if ((s = check_adapter(X, base, A, B, nullptr, dY, dX, dA, dB, drop, M, d_in, d_out, r, gb, workspace,
                         workspace_bytes, false)) != LORA_OK)
    return s;
  return adapter_bwd_run(X, base, A, B, dY, dX, dA, dB, M, d_in, d_out, r, scale, drop, workspace, flags,
                         reinterpret_cast<cudaStream_t>(stream));
}

size_t lora_fp8_workspace_size(int64_t M, int64_t d_in, int64_t d_out, int32_t r) {
  if (check_sizes_fp8(M, d_in, d_out, r) != LORA_OK || M == 0) return 0;
  return fp8_workspace(M, d_in, d_out, r).total;
}

lora_status_t lora_fwd_fp8(const void* X, const void* Wq, const void* Ws, const void* A, const void* B, void* Y,
                           int64_t M, int64_t d_in, int64_t d_out, int32_t r, float scale, float p, const void* rng,
                           void* workspace, size_t workspace_bytes, void* stream) {
  lora_status_t s = check_sizes_fp8(M, d_in, d_out, r);
  DropArgs drop;
  if (s != LORA_OK || (s = drop_args(p, rng, drop)) != LORA_OK) return s;
  if (Ws == nullptr) return LORA_ERR_NULL;
  const Base base{Wq, Ws};
  if ((s = check_adapter(X, base, A, B, Y, nullptr, nullptr, nullptr, nullptr, drop, M, d_in, d_out, r, 2, workspace,
                         workspace_bytes, true)) != LORA_OK)
    return s;
  return adapter_fwd_run(X, base, A, B, Y, M, d_in, d_out, r, scale, drop, workspace,
                         reinterpret_cast<cudaStream_t>(stream));
}

lora_status_t lora_bwd_fp8(const void* X, const void* Wq, const void* Ws, const void* A, const void* B,
                           const void* dY, void* dX, void* dA, void* dB, int64_t M, int64_t d_in, int64_t d_out,
                           int32_t r, float scale, float p, const void* rng, void* workspace, size_t workspace_bytes,
                           uint32_t flags, void* stream) {
  if ((flags & ~kBwdFlags) != 0u) return LORA_ERR_FLAGS;
  lora_status_t s = check_sizes_fp8(M, d_in, d_out, r);
  DropArgs drop;
  if (s != LORA_OK || (s = drop_args(p, rng, drop)) != LORA_OK) return s;
  if (Ws == nullptr) return LORA_ERR_NULL;
  const Base base{Wq, Ws};
  const int gb = (flags & LORA_BWD_FP32_GRADS) != 0u ? 4 : 2;
  if ((s = check_adapter(X, base, A, B, nullptr, dY, dX, dA, dB, drop, M, d_in, d_out, r, gb, workspace,
                         workspace_bytes, false)) != LORA_OK)
    return s;
  return adapter_bwd_run(X, base, A, B, dY, dX, dA, dB, M, d_in, d_out, r, scale, drop, workspace, flags,
                         reinterpret_cast<cudaStream_t>(stream));
}

// Sizes and buffers of the two weight conversions.
static lora_status_t check_quant(const void* src, uint64_t src_b, const void* scales_in, const void* dst,
                                 uint64_t dst_b, const void* scales_out, int64_t d_out, int64_t d_in) {
  if (d_in <= 0 || d_out <= 0 || (d_in % 16) != 0 || d_in > (int64_t(1) << 30) || d_out > (int64_t(1) << 30))
    return LORA_ERR_SHAPE;
  const uint64_t nb = uint64_t(qblocks(d_in)) * uint64_t(qblocks(d_out));
  if (nb > 0x7FFFFFFFull) return LORA_ERR_SHAPE;
  const uint64_t e = uint64_t(d_in) * uint64_t(d_out);
  const BufSpec in[2] = {{src, e * src_b, true}, {scales_in, nb, scales_out == nullptr}};
  const BufSpec out[2] = {{dst, e * dst_b, true}, {scales_out, nb, scales_in == nullptr}};
  return check_bufs(in, 2, out, 2);
}

lora_status_t lora_quantize_fp8(const void* W, void* Wq, void* Ws, int64_t d_out, int64_t d_in, void* stream) {
  if (Ws == nullptr) return LORA_ERR_NULL;
  lora_status_t s = check_quant(W, 2, nullptr, Wq, 1, Ws, d_out, d_in);
  DeviceInfo dev;
  if (s != LORA_OK || (s = device_info(dev)) != LORA_OK) return s;
  const int64_t cb = qblocks(d_in);
  return launch_ex("quantize", quantize_block_kernel, dim3(unsigned(cb * qblocks(d_out))), dim3(kQuantThreads), 0,
                   reinterpret_cast<cudaStream_t>(stream), nullptr, reinterpret_cast<const uint8_t*>(W),
                   reinterpret_cast<uint8_t*>(Wq), reinterpret_cast<uint8_t*>(Ws), int32_t(d_out), int32_t(d_in),
                   int32_t(cb));
}

lora_status_t lora_dequantize_fp8(const void* Wq, const void* Ws, void* W, int64_t d_out, int64_t d_in, void* stream) {
  if (Ws == nullptr) return LORA_ERR_NULL;
  lora_status_t s = check_quant(Wq, 1, Ws, W, 2, nullptr, d_out, d_in);
  DeviceInfo dev;
  if (s != LORA_OK || (s = device_info(dev)) != LORA_OK) return s;
  const int64_t cb = qblocks(d_in);
  return launch_ex("dequantize", dequantize_block_kernel, dim3(unsigned(cb * qblocks(d_out))), dim3(kQuantThreads), 0,
                   reinterpret_cast<cudaStream_t>(stream), nullptr, reinterpret_cast<const uint8_t*>(Wq),
                   reinterpret_cast<const uint8_t*>(Ws), reinterpret_cast<uint8_t*>(W), int32_t(d_out), int32_t(d_in),
                   int32_t(cb));
}

}  // extern "C"
