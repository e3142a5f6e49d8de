// gemm_pair_sm100.cuh -- fused dequant-in-mainloop QLoRA GEMM on a CTA pair
// (tcgen05 cta_group::2).
//
// Same products as gemm_sm100.cuh ("QLoRA", llm-compass, 方法与公式):
//   forward  h [M, out] = [x | us] . [W0 | B]^T       K = in  + r
//   backward dx[M, in ] = [dh | du] . [W0 ; A]        K = out + r
// with W0 dequantized on the fly, but one output tile of 512 token rows x 256
// columns is computed by a pair of CTAs on two SMs.  Each UMMA is
// 256 x 256 x 16 (cta_group::2): its A rows come half from each CTA and its B
// columns half from each CTA, so each SM dequantizes only its 128-column half
// of the weight tile and its tensor core reads that half once per UMMA.
// Compared with one CTA on a 256 x 256 tile this halves both the dequant work
// per tensor-core FLOP and the shared-memory traffic for the weight operand.
//
// Per CTA (576 threads, 4-stage ring of 32 KB activation + 16 KB weight):
//   warp 0     TMA producer for this CTA's two 128-row activation tiles; the
//              copies of both CTAs complete on the even CTA's "full" barrier
//   warp 1     TMEM allocation (both CTAs); UMMA issue for the pair (even CTA)
//   warps 2-17 dequant producers in four groups of 4, each group taking every
//              fourth stage:
//              a thread decodes its next stage into registers before it
//              waits for the buffer, then stores, fences and (one lane per
//              warp) arrives on the even CTA's "full" barrier; afterwards
//              the epilogue of this CTA's 256 accumulator rows
// TMEM: two 256-column fp32 accumulators per CTA (token sub-tiles 0 and 1).
// The even CTA's "full" barrier counts its TMA arrive (with the byte count of
// both CTAs' copies) and the 8 dequant warps of both CTAs.  The even CTA
// commits each stage with a multicast arrive on both CTAs' "empty" barriers,
// and the end of the accumulation on both "acc_full".
// Every wait is bounded (see gemm_sm100.cuh); no TMA multicast is used.
//
// kSlots: the forward with one adapter per token (h[m] = W0 x[m] + B_a us[m],
// a = ids[m]).  A kernel before lists the distinct adapters of each tile of
// 512 tokens (slots.cuh); the rank columns of the listed adapters, one after
// another, are K slices before the base's (before: their loads then overlap
// the filling of the pipeline).  There the dequant groups write both operands: B_a rows
// as they are, and the token rows of us under the columns of the token's own
// adapter with zeros elsewhere.  A B value that is infinite or NaN would reach
// the other tokens through those zeros: it is carried as 0 and both CTAs are
// marked, and the epilogue adds its products to the adapter's own tokens.
// Prompts of few requests cost a slice or two this way, against a second pass
// over h (M out 4 bytes) for adding the adapters behind the GEMM.
//
// kDrop: dx under counter-based LoRA dropout, dx = dh W0 + (du A) k / (1 - q)
// with the mask drawn in the epilogue (philox.cuh).  The masked term cannot be
// a K slice, and the two base accumulators fill tensor memory.  So the rank
// slices stay in the ring, and for each half of the tile's columns the
// epilogue warps take the base into registers (64 columns each), the UMMAs
// write P = du A over it, and the warps add the masked P and round once.
// Against a pass over dx behind the GEMM this saves one rounding and takes a
// 7B attention backward of 4096 tokens from 160 to 153 us, of 8192 tokens of
// 4096 -> 11008 from 704 to 643, although it waits for du (15 us) first.
#pragma once

#include "common.cuh"
#include "gemm_sm100.cuh"
#include "philox.cuh"
#include "slots.cuh"

namespace qnf4 {

struct PairCfg {
  static constexpr int kStages = 4;
  static constexpr int BM = 512;                       // token rows per pair
  static constexpr int BN = 256;                       // output columns per pair
  static constexpr int A_SUB = 128 * 64 * 2;           // one 128-row activation tile
  static constexpr int A_STAGE = 2 * A_SUB;            // two token sub-tiles per CTA
  static constexpr int B_STAGE = 128 * 64 * 2;         // this CTA's half of the weight tile
  static constexpr int RING = kStages * (A_STAGE + B_STAGE);
  static constexpr int SMEM = RING + 256 + 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int kGroups = 4;                    // dequant groups, one stage each in turn
  static constexpr int THREADS = 64 + kGroups * 128;   // 2 + 16 warps
  static constexpr int SLOTS_SMEM = SMEM + BM * 4 + 16;   // kSlots: per token its first rank column; a flag
};

struct PairExtra {
  // kSlots
  const SlotsTile* tiles;   // per 512 tokens
  const uint16_t* us;       // [M, r8]
  int r8;                   // r rounded up to 8
  // kDrop
  DropoutRng rng;
  float inv_keep;           // 1 / (1 - q)
};

template <bool kDx, bool kSlots = false, bool kDrop = false>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairCfg::THREADS, 1)
qlora_gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_act,
                       const __grid_constant__ CUtensorMap tm_lora,
                       const GemmArgs args, const PairExtra slots) {
  using Cfg = PairCfg;
  constexpr int kStages = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* a_ring = smem;
  uint8_t* b_ring = smem + kStages * Cfg::A_STAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::RING);
  uint64_t* full = bars;                       // (even CTA) both CTAs' stage is complete
  uint64_t* empty = bars + kStages;            // the pair's UMMAs on the stage finished
  uint64_t* acc_full = bars + 2 * kStages;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  // (even CTA) the number of stages whose copies each CTA of the pair issued
  volatile int* issued_by = reinterpret_cast<volatile int*>(tmem_holder + 2);
  // kDrop, one phase per half: (even CTA) the base columns of the half are in
  // registers; the half's P is complete
  uint64_t* p_ready = reinterpret_cast<uint64_t*>(tmem_holder + 4);
  uint64_t* p_full = p_ready + 1;

  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int pair = blockIdx.x >> 1;
  const int tiles_m = (args.M + Cfg::BM - 1) / Cfg::BM;
  const int tile_m = pair % tiles_m;
  const int tile_n = pair / tiles_m;
  const int m0 = tile_m * Cfg::BM;
  const int n0 = tile_n * Cfg::BN;
  const int n0_half = n0 + 128 * static_cast<int>(rank);
  const int n_main = args.K / 64;
  const uint64_t tmo = args.timeout_ns;
  int32_t* tok_col = reinterpret_cast<int32_t*>(smem + Cfg::RING + 256);   // kSlots
  volatile int32_t* odd = tok_col + Cfg::BM;           // a B value of either CTA was not finite
  const int32_t* list = nullptr;                       // the tile's adapters
  int k_low = args.r;                                  // rank columns beside the base
  int n_list = 0;
  if constexpr (kSlots) {
    const SlotsTile& tile = slots.tiles[tile_m];
    n_list = __ldg(&tile.n);
    list = tile.list;
    if (threadIdx.x < Cfg::BM) tok_col[threadIdx.x] = __ldg(tile.col + threadIdx.x);
    if (threadIdx.x == 0) *odd = 0;
    k_low = n_list * slots.r8;
  }
  const int n_lora = (k_low + 63) / 64;
  const int n_iter = n_main + n_lora;
  // the rank slices come behind the base's, with kSlots before them
  auto is_low = [&](int it) { return kSlots ? it < n_lora : it >= n_main; };
  auto main_of = [&](int it) { return kSlots ? it - n_lora : it; };
  auto low_of = [&](int it) { return kSlots ? it : it - n_main; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1 + 8);     // TMA arrive + 4 dequant warps (one group) per CTA
      mbar_init(empty + s, 1);
    }
    mbar_init(acc_full, 1);
    if (kDrop) {
      mbar_init(p_ready, 2 * 4 * Cfg::kGroups);            // the epilogue warps of both CTAs
      mbar_init(p_full, 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, Cfg::TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();                 // both CTAs' barriers exist before any remote arrive
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_holder;

  // bounded waits (cluster-scope acquire: other CTAs and the pair's tensor
  // cores arrive on these barriers)
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (*abort_flag) return;
    if (!mbar_wait_cluster_bounded(bar, parity, tmo)) {
      *abort_flag = 1;
      raise_device_error(1);
    }
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_act);
      tma_prefetch_desc(&tm_lora);
      int issued = 0;
      for (int it = 0; it < n_iter; ++it) {
        const int s = it % kStages;
        const uint32_t ph = (it / kStages) & 1u;
        wait(empty + s, ph ^ 1u);
        if (*abort_flag) break;                           // a wait timed out: issue nothing more
        if (kSlots && is_low(it)) {                       // the dequant groups write the token operand
          if (leader) mbar_arrive(full + s);
          ++issued;
          continue;
        }
        if (leader) mbar_arrive_expect_tx(full + s, 2 * Cfg::A_STAGE);    // both CTAs' bytes
        const uint32_t bar = mapa_shared(smem_u32(full + s), 0);
        const uint32_t dst = smem_u32(a_ring + s * Cfg::A_STAGE);
        if (main_of(it) + kStages < n_main) {             // warm L2 for a later stage
#pragma unroll
          for (int sub = 0; sub < 2; ++sub)
            tma_prefetch_l2_2d(&tm_act, (main_of(it) + kStages) * 64, m0 + sub * 256 + static_cast<int>(rank) * 128);
        }
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          const int row = m0 + sub * 256 + static_cast<int>(rank) * 128;
          if (!is_low(it))
            tma_load_2d_pair(dst + sub * Cfg::A_SUB, &tm_act, bar, main_of(it) * 64, row);
          else
            tma_load_2d_pair(dst + sub * Cfg::A_SUB, &tm_lora, bar, low_of(it) * 64, row);
        }
        ++issued;
      }
      // Copies of both CTAs complete on the even CTA's barriers, which drains
      // them after the cluster barrier below; it needs both issued counts.
      asm volatile("st.shared::cluster.u32 [%0], %1;"
                   :: "r"(mapa_shared(smem_u32(const_cast<int*>(issued_by + rank)), 0)), "r"(issued) : "memory");
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------------------------------------------------- UMMA issuer
      constexpr uint32_t idesc = umma_idesc_bf16(256, 256, kDx);
      const int n_acc = kDrop ? n_main : n_iter;            // stages of the accumulation
      for (int it = 0; it < n_acc; ++it) {
        const int s = it % kStages;
        const uint32_t ph = (it / kStages) & 1u;
        wait(full + s, ph);
        if (*abort_flag) break;                           // commit what was issued, then finish
        tc_fence_after_sync();
        const uint32_t a_base = smem_u32(a_ring + s * Cfg::A_STAGE);
        const uint32_t b_base = smem_u32(b_ring + s * Cfg::B_STAGE);
        int ksteps = 4;
        // (args.r by name: through k_low the plain forward and dx took 0.8 % longer)
        if (is_low(it)) ksteps = min(4, ((kSlots ? k_low : args.r) - low_of(it) * 64 + 15) / 16);
        for (int kk = 0; kk < ksteps; ++kk) {
          const uint64_t bdesc = kDx ? umma_desc_sw128(b_base + kk * 2048, 8192, 1024)
                                     : umma_desc_sw128(b_base + kk * 32, 16, 1024);
#pragma unroll
          for (int sub = 0; sub < 2; ++sub) {
            const uint64_t adesc = umma_desc_sw128(a_base + sub * Cfg::A_SUB + kk * 32, 16, 1024);
            umma_bf16_ss_pair(tmem_base + sub * 256, adesc, bdesc, idesc, (it > 0 || kk > 0) ? 1u : 0u);
          }
        }
        umma_commit_pair_multicast(empty + s, 0x3);
      }
      umma_commit_pair_multicast(acc_full, 0x3);
      if constexpr (kDrop) {
        // P of each half of the columns, over the base columns that the
        // epilogue has taken into registers; the rank stages stay in the ring
        constexpr uint32_t pdesc = umma_idesc_bf16(256, 128, true);
        for (int it = n_main; it < n_iter; ++it) wait(full + (it % kStages), (it / kStages) & 1u);
        for (int a = 0; a < 2 && !*abort_flag; ++a) {
          wait(p_ready, a);
          if (*abort_flag) break;
          tc_fence_after_sync();
          for (int it = n_main; it < n_iter; ++it) {
            const int s = it % kStages;
            const uint32_t a_base = smem_u32(a_ring + s * Cfg::A_STAGE);
            const uint32_t b_base = smem_u32(b_ring + s * Cfg::B_STAGE) + a * 8192;
            const int ksteps = min(4, (args.r - (it - n_main) * 64 + 15) / 16);
            for (int kk = 0; kk < ksteps; ++kk) {
              const uint64_t bdesc = umma_desc_sw128(b_base + kk * 2048, 8192, 1024);
#pragma unroll
              for (int sub = 0; sub < 2; ++sub)
                umma_bf16_ss_pair(tmem_base + sub * 256 + a * 128,
                                  umma_desc_sw128(a_base + sub * Cfg::A_SUB + kk * 32, 16, 1024), bdesc, pdesc,
                                  (it > n_main || kk > 0) ? 1u : 0u);
            }
          }
          umma_commit_pair_multicast(p_full, 0x3);
        }
        // whatever was issued last is done before the pair may leave
        if (!*abort_flag) mbar_wait_cluster_bounded(p_full, 1, tmo);
      }
      mbar_wait_cluster_bounded(acc_full, 0, tmo);
    }
  } else {
    // -------------------------------------------------- dequant producers
    constexpr int G = Cfg::kGroups;
    const int group = (warp - 2) >> 2;                    // stages it = group, group+G, ...
    const int t = (threadIdx.x - 64) & 127;               // 0..127 within the group
    const int64_t w_row_bytes = args.w_cols / 2;
    const int64_t w_row_blocks = args.w_cols / 64;
    const float mu = __ldg(args.mean);

    const uint8_t* code_ptr;
    int64_t code_step, q8_idx, q8_step;
    uint32_t row_off, key;
    bool col_valid;
    int lora_row;
    if (!kDx) {
      col_valid = (n0_half + t) < args.N;
      const int64_t wr = col_valid ? (n0_half + t) : 0;
      code_ptr = args.codes + wr * w_row_bytes;
      code_step = 32;
      q8_idx = wr * w_row_blocks;
      q8_step = 1;
      row_off = t * 128;
      key = t & 7;
      lora_row = n0_half + t;
    } else {
      const int k = t & 63, a = t >> 6;
      col_valid = (n0_half + 64 * a) < args.N;
      const int64_t wc = col_valid ? (n0_half + 64 * a) : 0;
      code_ptr = args.codes + static_cast<int64_t>(k) * w_row_bytes + wc / 2;
      code_step = 64 * w_row_bytes;
      q8_idx = static_cast<int64_t>(k) * w_row_blocks + wc / 64;
      q8_step = 64 * w_row_blocks;
      row_off = a * 8192 + k * 128;
      key = k & 7;
      lora_row = k;
    }

    struct StageIn {
      uint4 c0, c1;
      int q;
      float st;
    };
    auto load_stage = [&](int it, StageIn& d) {
      const int k = main_of(it);
      if (col_valid && (!kSlots || k >= 0) && k < n_main) {
        const uint8_t* p = code_ptr + k * code_step;
        const int64_t blk = q8_idx + k * q8_step;
        if (args.codes_32b) {
          ld_nc_v8(p, d.c0, d.c1);
        } else {
          d.c0 = ld_nc_v4(p);
          d.c1 = ld_nc_v4(p + 16);
        }
        d.q = __ldg(args.q8 + blk);
        d.st = __ldg(args.step2 + blk / 256);
      }
    };

    // Decode (or fetch the LoRA rows of) stage `it` into 8 x 16 B of registers.
    auto produce = [&](int it, const StageIn& in, uint4 (&v)[8]) {
      if (!is_low(it)) {
        if (col_valid) {
          const float c_hat = block_scale(in.q, in.st, mu);
          const Nf4Table tb = make_table(args.L, c_hat);
          const uint32_t w[8] = {in.c0.x, in.c0.y, in.c0.z, in.c0.w, in.c1.x, in.c1.y, in.c1.z, in.c1.w};
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t o[4];
            decode8(tb, w[c], o);
            v[c] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] = make_uint4(0, 0, 0, 0);
        }
      } else if constexpr (kSlots) {
        // rank columns [64 j, 64 j + 64) of the listed adapters, in chunks of 8
        const int j = low_of(it);
        int li = j * 64 / slots.r8, c0 = j * 64 - li * slots.r8;
        uint32_t exps = 0;                                // bit 15 or 31: an exponent of all ones
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          v[c] = make_uint4(0, 0, 0, 0);
          if (col_valid && li < n_list) {
            const uint16_t* src = args.lora_w + (static_cast<int64_t>(__ldg(list + li)) * args.N + lora_row) * args.r + c0;
            if ((args.r & 7) == 0) {
              v[c] = ld_nc_v4(src);
            } else {
              uint32_t w[4] = {0, 0, 0, 0};
              for (int i = 0; i < 8; ++i)
                if (c0 + i < args.r) w[i >> 1] |= static_cast<uint32_t>(__ldg(src + i)) << (16 * (i & 1));
              v[c] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          c0 += 8;
          if (c0 == slots.r8) { c0 = 0; ++li; }
        }
#pragma unroll
        for (int c = 0; c < 8; ++c)
          exps |= ((v[c].x & 0x7F807F80u) + 0x00800080u) | ((v[c].y & 0x7F807F80u) + 0x00800080u) |
                  ((v[c].z & 0x7F807F80u) + 0x00800080u) | ((v[c].w & 0x7F807F80u) + 0x00800080u);
        if (exps & 0x80008000u) {
          auto finite = [](uint32_t& w) {
            if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
            if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
          };
#pragma unroll
          for (int c = 0; c < 8; ++c) { finite(v[c].x); finite(v[c].y); finite(v[c].z); finite(v[c].w); }
          const uint32_t at = smem_u32(const_cast<int32_t*>(odd));
          for (uint32_t k = 0; k < 2; ++k)                // before this warp's arrive on "full"
            asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(mapa_shared(at, k)), "r"(1) : "memory");
        }
      } else {
        const int j = low_of(it);
        const uint16_t* src = nullptr;
        int count = 0;
        if (!kDx) {
          if (col_valid) {
            src = args.lora_w + static_cast<int64_t>(lora_row) * args.r + j * 64;
            count = min(64, args.r - j * 64);
          }
        } else {
          const int kr = j * 64 + lora_row;
          if constexpr (kDrop) {
            // atom a of both CTAs together is half a of the tile's columns
            const int c0 = n0 + 128 * (t >> 6) + 64 * static_cast<int>(rank);
            if (c0 < args.N && kr < args.r) {
              src = args.lora_w + static_cast<int64_t>(kr) * args.w_cols + c0;
              count = 64;
            }
          } else if (col_valid && kr < args.r) {
            src = args.lora_w + static_cast<int64_t>(kr) * args.w_cols + n0_half + 64 * (t >> 6);
            count = 64;
          }
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = (c * 8 < count) ? ld_nc_v4(src + c * 8) : make_uint4(0, 0, 0, 0);
      }
    };

    // codes and scale codes are loaded two of this group's turns ahead (eight
    // stages), so their global-load latency overlaps two turns of MMAs
    StageIn na{}, nb{};
    load_stage(group, na);
    load_stage(group + G, nb);
    const bool warp_lead = lane == 0;

    for (int it = group; it < n_iter; it += G) {
      const StageIn cur = na;
      na = nb;
      load_stage(it + 2 * G, nb);
      uint4 v[8];
      produce(it, cur, v);                          // before waiting for the buffer

      const int s = it % kStages;
      const uint32_t ph = (it / kStages) & 1u;
      const uint32_t dst = smem_u32(b_ring + s * Cfg::B_STAGE) + row_off;
      wait(empty + s, ph ^ 1u);
#pragma unroll
      for (int c = 0; c < 8; ++c) sts_v4(dst + ((c ^ key) << 4), v[c].x, v[c].y, v[c].z, v[c].w);
      if constexpr (kSlots) {
        if (is_low(it)) {
          // token rows t of both sub-tiles: us under the columns of the token's adapter
          const int e = low_of(it);
#pragma unroll
          for (int sub = 0; sub < 2; ++sub) {
            const int i = sub * 256 + static_cast<int>(rank) * 128 + t;         // of the 512 tokens
            const uint32_t row = smem_u32(a_ring + s * Cfg::A_STAGE) + sub * Cfg::A_SUB + t * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c) sts_v4(row + ((c ^ (t & 7)) << 4), 0, 0, 0, 0);
            const int col = tok_col[i] - e * 64;
            const uint16_t* src = slots.us + static_cast<int64_t>(m0 + i) * slots.r8;
#pragma unroll 2
            for (int j = max(0, -col); j < slots.r8 && col + j < 64; j += 8) {
              const uint4 u = *reinterpret_cast<const uint4*>(src + j);
              sts_v4(row + ((((col + j) >> 3) ^ (t & 7)) << 4), u.x, u.y, u.z, u.w);
            }
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (warp_lead) mbar_arrive_remote(mapa_shared(smem_u32(full + s), 0));
    }

    // ------------------------------------------------------------ epilogue
    // This CTA's TMEM holds 128 rows (lanes) x 256 columns for each token
    // sub-tile; each of the 16 warps writes 128 columns of one sub-tile for
    // the 32 lanes of its quadrant.
    wait(acc_full, 0);
    tc_fence_after_sync();
    const int q = warp & 3;
    const int part = (warp - 2) >> 2;                     // 0..3
    const int sub = part >> 1;
    const int m = m0 + sub * 256 + static_cast<int>(rank) * 128 + q * 32 + lane;
    if constexpr (kDrop) {
      const PhiloxKey key = philox_key(slots.rng.state);
      const uint32_t lanes = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + sub * 256;
      for (int a = 0; a < 2; ++a) {
        const int col0 = a * 128 + (part & 1) * 64;         // this warp's 64 columns of half a
        const uint64_t first = philox_first(static_cast<uint32_t>((n0 + col0) / 8));
        uint32_t base[64];
        tmem_ld_32x32b_x32(lanes + col0, *reinterpret_cast<uint32_t(*)[32]>(&base[0]));
        tmem_ld_32x32b_x32(lanes + col0 + 32, *reinterpret_cast<uint32_t(*)[32]>(&base[32]));
        tmem_ld_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (warp_lead) mbar_arrive_remote(mapa_shared(smem_u32(p_ready), 0));
        wait(p_full, a);
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16], drop[2][4];
          tmem_ld_32x32b_x16(lanes + col0 + 16 * c, p);
#pragma unroll
          for (int g = 0; g < 2; ++g)
            philox_drop8(key, slots.rng.threshold, static_cast<uint32_t>(m), first + (2 * c + g) * kPhiloxA, drop[g]);
          tmem_ld_wait();
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t d = drop[i >> 2][i & 3];         // columns 2 i, 2 i + 1
            const float k0 = d & 0xFFFFu ? 0.f : slots.inv_keep, k1 = d >> 16 ? 0.f : slots.inv_keep;
            // (a dropped column adds nothing, whatever its P is)
            const float p0 = d & 0xFFFFu ? 0.f : __uint_as_float(p[2 * i]);
            const float p1 = d >> 16 ? 0.f : __uint_as_float(p[2 * i + 1]);
            o[i] = pack_bf16x2_rn(fmaf(k0, p0, __uint_as_float(base[16 * c + 2 * i])),
                                  fmaf(k1, p1, __uint_as_float(base[16 * c + 2 * i + 1])));
          }
          if (m < args.M && n0 + col0 < args.N) {
            uint16_t* dstp = args.out + static_cast<int64_t>(m) * args.N + n0 + col0 + 16 * c;
            st_v4(dstp, make_uint4(o[0], o[1], o[2], o[3]));
            st_v4(dstp + 8, make_uint4(o[4], o[5], o[6], o[7]));
          }
        }
      }
    }
    for (int col = (part & 1) * 128; !kDrop && col < (part & 1) * 128 + 128; col += 32) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + sub * 256 + col, v);
      tmem_ld_wait();
      if constexpr (kSlots) {
        const int c = tok_col[m - m0];
        if (*odd && m < args.M && n0 + col < args.N && c >= 0) {
          const int64_t a = list[c / slots.r8];
#pragma unroll 1
          for (int i = 0; i < 32; ++i) {
            const float f = slots_odd_term(args.lora_w + (a * args.N + n0 + col + i) * args.r,
                                           slots.us + static_cast<int64_t>(m) * slots.r8, args.r);
#pragma unroll
            for (int k = 0; k < 32; ++k)                  // (constant indices keep v in registers)
              if (k == i) v[k] = __float_as_uint(__uint_as_float(v[k]) + f);
          }
        }
      }
      if (m < args.M && n0 + col < args.N) {
        uint16_t* dstp = args.out + static_cast<int64_t>(m) * args.N + n0 + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 o = make_uint4(
              pack_bf16x2_rn(__uint_as_float(v[8 * i + 0]), __uint_as_float(v[8 * i + 1])),
              pack_bf16x2_rn(__uint_as_float(v[8 * i + 2]), __uint_as_float(v[8 * i + 3])),
              pack_bf16x2_rn(__uint_as_float(v[8 * i + 4]), __uint_as_float(v[8 * i + 5])),
              pack_bf16x2_rn(__uint_as_float(v[8 * i + 6]), __uint_as_float(v[8 * i + 7])));
          st_v4(dstp + 8 * i, o);
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();                 // both issued counts are visible to the even CTA
  if (leader && warp == 0 && lane == 0) {
    // Wait (bounded) for the stages whose copies may still be in flight: a
    // stage more than kStages behind the last one issued was consumed, so
    // its copies have landed.  Without a timeout every phase has completed
    // and these waits return at once.
    const int n = max(issued_by[0], issued_by[1]);
    for (int it = n > kStages ? n - kStages : 0; it < n; ++it)
      mbar_wait_cluster_bounded(full + (it % kStages), (it / kStages) & 1u, tmo);
  }
  cluster_sync_all();                 // no CTA leaves while its pair may still use its memory
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
  }
}

}  // namespace qnf4
