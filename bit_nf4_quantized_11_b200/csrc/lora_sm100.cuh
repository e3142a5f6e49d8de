// lora_sm100.cuh -- the rank-r contractions of the QLoRA layer on tcgen05.
//
// ("QLoRA", llm-compass, 方法与公式: h = dequant(W0) x + (alpha/r) B A x, with
// gradients for A and B only; aigrafen.se, opening paragraph.)
//
// All four products have one dimension equal to the LoRA rank r and stream a
// token-sized operand from HBM once, so they are bound by that read.  Each is
// one tcgen05 tile product D[128 x N] (+)= A . B^T with N = r rounded up to a
// multiple of 16 (at most 256), fp32 accumulation in tensor memory, both
// operands staged by TMA (128-byte swizzle) in a ring of shared-memory stages:
//
//   row form  out[m][j] = bf16(scale * sum_k act[m][k] * w(j, k))
//     us = bf16(s x A^T)   act = x  [M, in]  (K-major), w = A [r, in]  (K-major)
//     du = bf16(s dh B)    act = dh [M, out] (K-major), w = B [out, r] (N-major)
//   col form  D[f][j] = scale * sum_m act[m][f] * u[m][j]
//     dB   = dh^T us       act = dh [M, out] (MN-major), u = us [M, r] (N-major)
//     dA^T = x^T du        act = x  [M, in]  (MN-major), u = du [M, r] (N-major)
//
// The tile rows are tokens (row form) or features (col form); the
// contraction (K of the row form, the tokens of the col form) is split over
// the CTAs of a thread-block cluster (at most 8).  Each CTA moves its fp32
// partial tile from tensor memory to its own shared memory; then every CTA
// adds up its share of the tile's rows over distributed shared memory,
// partials in rank order (deterministic), and stores it.
//
// Roles (128 threads, 320 with a keep mask): warp 0 lane 0 issues the TMA
// loads, warp 1 allocates tensor memory and its lane 0 issues the MMAs, and
// with a LoRA-dropout keep mask warps 2-9 zero the dropped activations of
// each landed stage in shared memory (bit c % 8 of byte c / 8 of a token's
// row keeps column c) before the MMAs read it; afterwards warps 0-3 read the
// accumulator (warp w owns rows 32 w .. 32 w + 31, its TMEM lanes) and all
// warps take part in the cluster reduction.
// Every wait is bounded: on timeout the CTA sets the device error flag,
// issues nothing more, waits (bounded) for what it issued and exits.
// No TMA multicast is used.
//
// kRng: the same products for counter-based LoRA dropout (philox.cuh).
//   * The masking warps draw the keep bits of the staged tile instead of
//     loading them.
//   * dA is a sum over tokens of du x, so du rounded to bf16 would leave a
//     relative error of 2^-9 in the fp32 gradient.  du is kept as three bf16
//     parts whose sum is its fp32 value (hi, mid, lo columns side by side, at
//     most 80 ranks per column group so that 3 x 80 <= 256), dA multiplies by
//     all three and adds the three results.
//   * The tensor cores cut the fp32 sum at every step, always towards zero:
//     of positive products, 391 steps of 16 tokens lost 1e-5 and 1024 steps
//     4e-5.  The stages take turns over several accumulators, which the
//     epilogue adds up; in the col form, whose tokens have no end, in rounds of
//     64 steps each: between two rounds the masking warps add the accumulators
//     to a total that takes the place of the last one, by rounded additions
//     (positive products of 262144 tokens, rank 64: 6e-7.  A backward of 65536
//     tokens, 1024 -> 11008, takes 2.3 ms, 2.1 without rounds and 2.6 with one
//     launch per round).
#pragma once

#include "common.cuh"
#include "philox.cuh"

namespace qnf4 {

constexpr int kLrThreads = 128;
constexpr int kLrMaskThreads = 320;                        // with a keep mask: eight masking warps
constexpr int kLrMaxStages = 8;
constexpr int kLrRound = 16;                              // (kRng, col form) stages per accumulator and round
constexpr int kLrTileRows = 128;
constexpr int kLrAStage = kLrTileRows * 64 * 2;           // 16 KB: 128 rows x 64 k (or two 64-wide MN atoms)

// Instruction descriptor, kind::f16 with bf16 A and B, fp32 D; either
// operand K-major or MN-major.
__host__ __device__ constexpr uint32_t umma_idesc_bf16_ab(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

struct LrProblem {
  void* out;             // row form: bf16 [rows, r]; col form: fp32 [rows, r] or, transposed, [r, rows]
  int rows;              // tokens (row form) or features (col form)
  int tiles;             // ceil(rows / 128)
  int transpose_out;     // col form: write D^T (dA [r, in])
  float scale;
  const uint8_t* keep;   // LoRA dropout keep bits of the token operand [tokens, features / 8], or null
  int features;          // columns of the token operand (row form: K; col form: rows)
  // kRng only:
  int masked;            // draw the keep bits
  int N;                 // columns of the product
  int parts;             // row form: bf16 parts written per value; col form: column sets added up
  int groups;            // col form: column groups (tiles of group g follow those of g - 1)
  int group_ranks;       // ranks per column group
};

struct LrArgs {
  LrProblem p[2];        // blockIdx.x < p[0].tiles: problem 0, else problem 1
  int K;                 // contraction length (row form: features; col form: tokens)
  int r;                 // rank
  int N;                 // r rounded up to 16
  int n_alloc;           // TMEM columns (power of two >= 32, >= N)
  int stages_per_split;  // 64-wide contraction stages per CTA of the cluster
  int ring;              // shared-memory stages in flight (<= kLrMaxStages)
  uint64_t timeout_ns;
  DropoutRng rng;        // kRng only
};

// du as parts: rank j of a row lies at (j / kLrPartRanks) 3 kLrPartRanks + part * ranks-of-its-group + ...
constexpr int kLrPartRanks = 80;
// Ranks per column group and columns of a row of du in parts, for a rank r (r % 8 == 0).
__host__ __device__ constexpr int lr_group_ranks(int r) { return r <= kLrPartRanks ? r : kLrPartRanks; }
__host__ __device__ constexpr int lr_groups(int r) { return (r + lr_group_ranks(r) - 1) / lr_group_ranks(r); }
__host__ __device__ constexpr int lr_part_cols(int r) { return lr_groups(r) * 3 * lr_group_ranks(r); }

// Shared bytes of one stage of the B operand (N rows x 64 k K-major, or
// ceil(N / 64) atoms of 64 n x 64 k) and of the fp32 partial tile (padded rows).
__host__ __device__ constexpr int lr_b_stage(int N, bool b_mn_major) {
  return b_mn_major ? ((N + 63) / 64) * 8192 : ((N * 128 + 1023) / 1024) * 1024;
}
__host__ __device__ constexpr int lr_partial_pitch(int N) { return N * 4 + 16; }
__host__ __device__ constexpr int lr_smem_bytes(int N, bool b_mn_major, int stages) {
  const int ring = stages * (kLrAStage + lr_b_stage(N, b_mn_major));
  const int part = kLrTileRows * lr_partial_pitch(N);
  return (ring > part ? ring : part) + 512 + 1024;
}

// kCol: col form (A MN-major, output fp32); otherwise row form (A K-major,
// output bf16).  kBMN: B operand N-major.  kRounds (kRng, col form): a CTA may
// have more than kLrRound stages per accumulator.
template <bool kCol, bool kBMN, bool kRng = false, bool kRounds = false>
__global__ void __launch_bounds__(kLrMaskThreads) lora_umma_kernel(
    const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_b0,
    const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_b1, const LrArgs args) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const int N = args.N;
  const int b_stage = lr_b_stage(N, kBMN);
  const int S = args.ring;                                           // stages of the ring
  const int ring_bytes = S * (kLrAStage + b_stage);
  const int part_bytes = kLrTileRows * lr_partial_pitch(N);
  uint8_t* a_ring = smem;
  uint8_t* b_ring = smem + S * kLrAStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (ring_bytes > part_bytes ? ring_bytes : part_bytes));
  uint64_t* full = bars;
  uint64_t* empty = bars + kLrMaxStages;
  uint64_t* masked = bars + 2 * kLrMaxStages;                        // (keep mask) the stage is masked
  uint64_t* acc_full = bars + 3 * kLrMaxStages;
  uint64_t* round_full = acc_full + 1;                               // a round's sums are complete
  uint64_t* round_empty = acc_full + 2;                              // and added to the total
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_full + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int prob = static_cast<int>(blockIdx.x) < args.p[0].tiles ? 0 : 1;
  // fields of this CTA's problem (selected, not indexed: no local-memory copy)
  void* const p_out = prob == 0 ? args.p[0].out : args.p[1].out;
  const int p_rows = prob == 0 ? args.p[0].rows : args.p[1].rows;
  const bool p_transpose = (prob == 0 ? args.p[0].transpose_out : args.p[1].transpose_out) != 0;
  const float p_scale = prob == 0 ? args.p[0].scale : args.p[1].scale;
  const uint8_t* const p_keep = prob == 0 ? args.p[0].keep : args.p[1].keep;
  const int p_features = prob == 0 ? args.p[0].features : args.p[1].features;
  const bool do_mask = kRng ? (prob == 0 ? args.p[0].masked : args.p[1].masked) != 0
                            : p_keep != nullptr;                     // CTA-uniform
  const int p_tile = prob == 0 ? static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x) - args.p[0].tiles;
  // (kRng) this CTA's columns: width, first column, bf16 parts
  const int p_N = kRng ? (prob == 0 ? args.p[0].N : args.p[1].N) : N;
  const int p_parts = kRng ? (prob == 0 ? args.p[0].parts : args.p[1].parts) : 1;
  const int p_ranks = kRng ? (prob == 0 ? args.p[0].group_ranks : args.p[1].group_ranks) : args.r;
  const int p_row_tiles = (p_rows + kLrTileRows - 1) / kLrTileRows;
  const int p_group = kRng && kCol ? p_tile / p_row_tiles : 0;
  const int tile = kRng && kCol ? p_tile % p_row_tiles : p_tile;
  // accumulators that the stages take turns over
  const int acc_stride = (p_N + 31) / 32 * 32;
  const int n_acc = kRng ? max(1, min(8, args.n_alloc / acc_stride)) : 1;
  const CUtensorMap* tm_a = prob == 0 ? &tm_a0 : &tm_a1;
  const CUtensorMap* tm_b = prob == 0 ? &tm_b0 : &tm_b1;
  const int row0 = tile * kLrTileRows;
  const int ks = static_cast<int>(gridDim.y);
  const int split = static_cast<int>(blockIdx.y);
  const int n_stages_total = (args.K + 63) / 64;
  const int st_begin = split * args.stages_per_split;
  const int st_end = min(n_stages_total, st_begin + args.stages_per_split);
  const int n_iter = max(0, st_end - st_begin);
  const uint64_t tmo = args.timeout_ns;
  // (kRounds) accumulators in use, stages of a round, rounds
  const bool in_rounds = kRounds && n_acc > 1 && n_iter > kLrRound * n_acc;
  const int n_live = in_rounds ? n_acc - 1 : n_acc;
  const int round = in_rounds ? kLrRound * n_live : n_iter;
  const int n_rounds = in_rounds ? (n_iter + round - 1) / round : 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
      mbar_init(masked + s, (blockDim.x - 64) / 32);                 // one arrive per masking warp
    }
    mbar_init(acc_full, 1);
    if (kRounds) {
      mbar_init(round_full, 1);
      mbar_init(round_empty, 8);                                     // the masking warps
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, static_cast<uint32_t>(args.n_alloc));
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_holder;

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (*abort_flag) return;
    if (!mbar_wait_bounded(bar, parity, tmo)) {
      *abort_flag = 1;
      raise_device_error(1);
    }
  };

  // Round k's accumulators, and the total so far, added up over the last one:
  // warps 2-9, two per 32 rows with every other 16 columns each.
  auto end_round = [&](int k) -> bool {
    wait(round_full, k & 1u);
    if (__any_sync(0xFFFFFFFFu, *abort_flag)) return false;
    tc_fence_after_sync();
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    for (int c0 = 16 * ((warp - 2) >> 2); c0 < p_N; c0 += 32) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(lanes + c0, v);
      tmem_ld_wait();
      for (int g = 1; g < n_live + (k > 0 ? 1 : 0); ++g) {
        uint32_t w[16];
        tmem_ld_32x32b_x16(lanes + g * acc_stride + c0, w);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
      }
      tmem_st_32x32b_x16(lanes + n_live * acc_stride + c0, v);
    }
    tmem_st_wait();
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(round_empty);
    return true;
  };

  const uint32_t stage_tx = static_cast<uint32_t>(kLrAStage + (kRng ? lr_b_stage(p_N, kBMN) : b_stage));
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      tma_prefetch_desc(tm_a);
      tma_prefetch_desc(tm_b);
      int issued = 0;
      for (int it = 0; it < n_iter; ++it) {
        const int s = it % S;
        wait(empty + s, ((it / S) & 1u) ^ 1u);
        if (*abort_flag) break;
        mbar_arrive_expect_tx(full + s, stage_tx);
        const uint32_t a_dst = smem_u32(a_ring + s * kLrAStage);
        const uint32_t b_dst = smem_u32(b_ring + s * b_stage);
        const int k0 = (st_begin + it) * 64;
        if (!kCol) {
          tma_load_2d(a_dst, tm_a, full + s, k0, row0);                      // [128 rows x 64 k]
        } else {
          tma_load_2d(a_dst, tm_a, full + s, row0, k0);                      // two atoms of 64 features x 64 tokens
          tma_load_2d(a_dst + 8192, tm_a, full + s, row0 + 64, k0);
        }
        if (!kBMN) {
          tma_load_2d(b_dst, tm_b, full + s, k0, 0);                         // [N rows x 64 k]
        } else {
          const int c0 = kRng ? p_group * p_parts * p_ranks : 0;
          for (int a = 0; a * 64 < p_N; ++a) tma_load_2d(b_dst + a * 8192, tm_b, full + s, c0 + a * 64, k0);
        }
        ++issued;
      }
      // only the last S issued stages can still be in flight
      for (int it = issued > S ? issued - S : 0; it < issued; ++it)
        mbar_wait_bounded(full + (it % S), (it / S) & 1u, tmo);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      const uint32_t idesc = umma_idesc_bf16_ab(kLrTileRows, p_N, kCol, kBMN);
      int lo = 0, rounds_done = 0;                                   // (kRounds) the round's first stage
      for (int it = 0; it < n_iter; ++it) {
        const int s = it % S;
        if (kRounds && it - lo == round) {
          umma_commit(round_full);
          wait(round_empty, rounds_done & 1u);
          ++rounds_done;
          lo = it;
        }
        const int turn = kRounds ? it - lo : it;
        wait(full + s, (it / S) & 1u);
        if (do_mask) wait(masked + s, (it / S) & 1u);
        if (*abort_flag) break;
        tc_fence_after_sync();
        const uint32_t a_base = smem_u32(a_ring + s * kLrAStage);
        const uint32_t b_base = smem_u32(b_ring + s * b_stage);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t adesc = kCol ? umma_desc_sw128(a_base + kk * 2048, 8192, 1024)
                                      : umma_desc_sw128(a_base + kk * 32, 16, 1024);
          const uint64_t bdesc = kBMN ? umma_desc_sw128(b_base + kk * 2048, 8192, 1024)
                                      : umma_desc_sw128(b_base + kk * 32, 16, 1024);
          if (kRng)
            umma_bf16_ss(tmem_base + (turn % n_live) * acc_stride, adesc, bdesc, idesc,
                         (turn >= n_live || kk > 0) ? 1u : 0u);
          else
            umma_bf16_ss(tmem_base, adesc, bdesc, idesc, (it > 0 || kk > 0) ? 1u : 0u);
        }
        umma_commit(empty + s);
      }
      umma_commit(acc_full);
      mbar_wait_bounded(acc_full, 0, tmo);
    }
  } else if (do_mask) {
    // ------------------------------------------------------------ keep mask
    // The MT = blockDim - 64 masking threads split a stage into 256 items,
    // (row i, half q) = (j % 128, j / 128) for j = t + MT h: row form, token
    // row0 + i; col form, token k0 + i % 64 of the 64-feature atom i / 64;
    // half q is 16-byte chunks 4q .. 4q + 3 of the row (32 values, one
    // 32-bit word of keep bits).  In each landed stage the thread zeroes the
    // values of its items whose keep bit is 0.
    const int t = threadIdx.x - 64;
    const int MT = static_cast<int>(blockDim.x) - 64;
    const int n_items = 2 * kLrTileRows / MT;                        // 1, 2 or 4 per thread
    const int64_t kb_row = p_features / 8;                           // keep bytes per token
    auto mask_chunk16 = [](uint32_t addr, uint32_t bits) {           // 8 bf16 at addr, bit e keeps value e
      uint32_t v[4];
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                   : "r"(addr) : "memory");
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] &= ((bits >> (2 * e)) & 1u ? 0x0000FFFFu : 0u) | ((bits >> (2 * e + 1)) & 1u ? 0xFFFF0000u : 0u);
      sts_v4(addr, v[0], v[1], v[2], v[3]);
    };
    // keep-bit address of item h of stage `it`, or null past the token or feature end
    auto keep_ptr = [&](int it, int h) -> const uint32_t* {
      if (it >= n_iter || h >= n_items) return nullptr;
      const int j = t + MT * h, i = j & (kLrTileRows - 1), q = j >> 7;
      const int k0 = (st_begin + it) * 64;
      int64_t tok, f0;
      if (!kCol) { tok = row0 + i; f0 = k0; }
      else { tok = k0 + (i & 63); f0 = row0 + 64 * (i >> 6); }
      const int64_t n_tok = kCol ? args.K : p_rows;
      if (tok >= n_tok || f0 >= p_features) return nullptr;
      return reinterpret_cast<const uint32_t*>(p_keep + tok * kb_row + f0 / 8) + q;   // 4-byte aligned
    };
    auto load_keep = [&](int it, uint32_t (&kb)[4]) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint32_t* src = keep_ptr(it, h);
        kb[h] = src != nullptr ? __ldg(src) : 0u;
      }
    };
    // loaded into registers two stages ahead and brought into L2 six stages
    // ahead, so their latency overlaps the stream
    auto prefetch_keep = [&](int it) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint32_t* src = keep_ptr(it, h);
        if (src != nullptr) asm volatile("prefetch.global.L2 [%0];" :: "l"(src));
      }
    };
    PhiloxKey key{};
    if (kRng) key = philox_key(args.rng.state);
    if (kRng) {
      // one item per thread (256 masking threads); its 32 values' masks are
      // drawn before the stage lands (past the tokens or features nothing
      // reads them)
      const int i = t & (kLrTileRows - 1), q = t >> 7;
      const int r = kCol ? (i & 63) : i;
      const uint32_t row_off = (kCol ? (i >> 6) * 8192 : 0) + r * 128;
      for (int it = 0; it < n_iter; ++it) {
        const int s = it % S;
        if (kRounds && it > 0 && it % round == 0 && !end_round(it / round - 1)) break;
        const int k0 = (st_begin + it) * 64;
        const int tok = kCol ? k0 + (i & 63) : row0 + i;
        const int f0 = kCol ? row0 + 64 * (i >> 6) : k0;
        uint32_t drop[4][4];
        const uint64_t first = philox_first(static_cast<uint32_t>(f0 / 8 + 4 * q));
#pragma unroll
        for (int c = 0; c < 4; ++c)
          philox_drop8(key, args.rng.threshold, static_cast<uint32_t>(tok), first + c * kPhiloxA, drop[c]);
        wait(full + s, (it / S) & 1u);
        if (*abort_flag) break;
        const uint32_t rbase = smem_u32(a_ring + s * kLrAStage) + row_off;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t addr = rbase + ((((4 * q + c) ^ r) & 7) << 4);
          uint32_t v[4];
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                       : "r"(addr) : "memory");
          sts_v4(addr, v[0] & ~drop[c][0], v[1] & ~drop[c][1], v[2] & ~drop[c][2], v[3] & ~drop[c][3]);
        }
        fence_proxy_async_smem();                                   // generic writes before the MMAs read
        __syncwarp();
        if (lane == 0) mbar_arrive(masked + s);
      }
    }
    if (!kRng)
      for (int i = 2; i < 6; ++i) prefetch_keep(i);
    uint32_t kb_n1[4], kb_n2[4];
    if (!kRng) {
      load_keep(0, kb_n1);
      load_keep(1, kb_n2);
    }
    for (int it = 0; !kRng && it < n_iter; ++it) {
      const int s = it % S;
      uint32_t kb[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        kb[h] = kb_n1[h];
        kb_n1[h] = kb_n2[h];
      }
      load_keep(it + 2, kb_n2);
      prefetch_keep(it + 6);
      wait(full + s, (it / S) & 1u);
      if (*abort_flag) break;
      const uint32_t a_base = smem_u32(a_ring + s * kLrAStage);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if (h >= n_items) continue;
        const int j = t + MT * h, i = j & (kLrTileRows - 1), q = j >> 7;
        // row form: row i of the 128-row tile; col form: row i % 64 of atom i / 64
        const int r = kCol ? (i & 63) : i;
        const uint32_t rbase = a_base + (kCol ? (i >> 6) * 8192 : 0) + r * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t bits = (kb[h] >> (8 * c)) & 0xFFu;
          if (bits != 0xFFu) mask_chunk16(rbase + ((((4 * q + c) ^ r) & 7) << 4), bits);
        }
      }
      fence_proxy_async_smem();                                     // generic writes before the MMAs read
      __syncwarp();
      if (lane == 0) mbar_arrive(masked + s);
    }
  } else if (kRounds) {
    for (int k = 0; k + 1 < n_rounds && end_round(k); ++k) {}
  }

  // ---------------------------------------------------------------- epilogue
  // Wait for the accumulator (the commit arrives even when no stage was
  // issued; an empty split leaves zeros).
  __syncwarp();
  wait(acc_full, 0);
  tc_fence_after_sync();
  const int row = warp * 32 + lane;                                  // this thread's TMEM lane / tile row
  const int pitch = lr_partial_pitch(p_N);
  uint8_t* part = smem;                                              // the ring is free once acc_full completed
  __syncthreads();                                                   // every stage read by the tensor cores
  for (int c0 = 0; warp < 4 && c0 < p_N; c0 += 32) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(warp * 32) << 16) + c0, v);
    tmem_ld_wait();
    if (kRng) {
      auto add = [&](int g) {
        uint32_t w[32];
        tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(warp * 32) << 16) + g * acc_stride + c0, w);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
      };
      const int n_last = kRounds ? n_iter - (n_rounds - 1) * round : n_iter;       // stages of the last round
      for (int g = 1; g < n_live && g < n_last; ++g) add(g);
      if (kRounds && n_rounds > 1) add(n_live);                      // the total of the rounds before
    }
    if (n_iter == 0) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0u;                        // nothing accumulated
    }
    const uint32_t dst = smem_u32(part + row * pitch + c0 * 4);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + 4 * i < p_N) sts_v4(dst + 16 * i, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (ks > 1) cluster_sync_all();                                    // every CTA's partial is in place

  // this CTA's share of the tile's rows, summed over the cluster in rank order
  const int share = kLrTileRows / ks;
  const int r_lo = split * share;
  // float4 groups of this CTA's ranks
  const int n4 = (kRng ? min(p_ranks, args.r - p_group * p_ranks) : args.r) / 4;
  for (int e = threadIdx.x; e < share * n4; e += static_cast<int>(blockDim.x)) {
    int rr, c4;
    if (kCol && p_transpose) {                                   // rows fastest: coalesced dA^T stores
      rr = r_lo + e % share;
      c4 = e / share;
    } else {
      rr = r_lo + e / n4;
      c4 = e % n4;
    }
    const int grow = row0 + rr;
    const uint32_t addr = smem_u32(part + rr * pitch + c4 * 16);
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int rk = 0; rk < ks; ++rk) {
      float4 u;
      if (ks == 1) {
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(u.x), "=f"(u.y), "=f"(u.z), "=f"(u.w)
                     : "r"(addr) : "memory");
      } else {
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(u.x), "=f"(u.y), "=f"(u.z), "=f"(u.w) : "r"(mapa_shared(addr, rk)) : "memory");
      }
      t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
      if (kRng && kCol) {
        for (int q = 1; q < p_parts; ++q) {                          // the parts of du: hi, then mid, then lo
          const uint32_t addr_q = addr + q * p_ranks * 4;
          if (ks == 1) {
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(u.x), "=f"(u.y), "=f"(u.z), "=f"(u.w)
                         : "r"(addr_q) : "memory");
          } else {
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(u.x), "=f"(u.y), "=f"(u.z), "=f"(u.w) : "r"(mapa_shared(addr_q, rk)) : "memory");
          }
          t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
        }
      }
    }
    if (grow >= p_rows) continue;
    const float sc = p_scale;
    if (kRng && !kCol && p_parts == 3) {
      // du in three bf16 parts, each the rounding of what the ones before leave
      const int j = c4 * 4, gr = lr_group_ranks(args.r);
      uint16_t* o = static_cast<uint16_t*>(p_out) + static_cast<int64_t>(grow) * lr_part_cols(args.r) +
                    j / gr * 3 * gr + j % gr;                        // (gr % 8 == 0: four ranks of one group)
      float f[4] = {t.x * sc, t.y * sc, t.z * sc, t.w * sc};
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] = pack_bf16x2_rn(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<uint2*>(o + q * gr) = make_uint2(w[0], w[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {                                // exact; 0 past an infinity or NaN
          const float lo = f[2 * i] - __uint_as_float(w[i] << 16);
          const float hi = f[2 * i + 1] - __uint_as_float(w[i] & 0xFFFF0000u);
          f[2 * i] = isfinite(lo) ? lo : 0.f;
          f[2 * i + 1] = isfinite(hi) ? hi : 0.f;
        }
      }
    } else if (!kCol) {
      uint16_t* o = static_cast<uint16_t*>(p_out) + static_cast<int64_t>(grow) * args.r + c4 * 4;
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2_rn(t.x * sc, t.y * sc), pack_bf16x2_rn(t.z * sc, t.w * sc));
    } else if (!p_transpose) {
      float* o = static_cast<float*>(p_out) + static_cast<int64_t>(grow) * args.r + c4 * 4;
      *reinterpret_cast<float4*>(o) = make_float4(t.x * sc, t.y * sc, t.z * sc, t.w * sc);
    } else {
      const int64_t ld = p_rows;
      float* o = static_cast<float*>(p_out) + static_cast<int64_t>(kRng ? p_group * p_ranks : 0) * ld;
      o[static_cast<int64_t>(c4 * 4 + 0) * ld + grow] = t.x * sc;
      o[static_cast<int64_t>(c4 * 4 + 1) * ld + grow] = t.y * sc;
      o[static_cast<int64_t>(c4 * 4 + 2) * ld + grow] = t.z * sc;
      o[static_cast<int64_t>(c4 * 4 + 3) * ld + grow] = t.w * sc;
    }
  }
  if (ks > 1) cluster_sync_all();                                    // no CTA leaves while others read it
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, static_cast<uint32_t>(args.n_alloc));
  }
}

}  // namespace qnf4
