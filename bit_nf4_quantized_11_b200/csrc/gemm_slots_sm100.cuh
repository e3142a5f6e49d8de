// gemm_slots_sm100.cuh -- the QLoRA forward with one adapter per token for
// small and middle token counts:
//   h[m][n] = sum_k W0[n][k] x[m][k] + sum_j B_a[n][j] us[m][j],  a = ids[m]
// ("QLoRA", llm-compass, 方法与公式, the displayed formula, per token).
//
// The output is computed transposed: a CTA owns 128 weight rows (the UMMA's M
// dimension) and a tile of N <= 256 tokens (its N dimension), so a decode
// batch does not pad the UMMA and every weight is dequantized once per token
// tile.  The dequantized weight never touches shared memory: thread t of a
// dequant group decodes the 64-weight block of weight row t straight into the
// 32 tensor-memory columns that the UMMA reads as its A operand, and x comes
// as the B operand through TMA.
//
// The adapters ride along as extra K stages.  The CTA lists the distinct
// adapters of its token tile (first appearance first); the rank columns of
// the listed adapters, one after another, form a K axis that is cut into
// stages: the A operand is B_a[n][j], the B operand us[m][j] where token m
// uses that adapter and zero elsewhere.
//
// A B value that is infinite or NaN would reach the other tokens of the tile
// through their zeros, so the stages carry 0 in its place and the tile is
// marked; the epilogue then adds those products to the adapter's own tokens.
//
// The K axis is split over the CTAs of a cluster (256-column units of the
// base, and the adapter stages, each evenly); the fp32 partial tiles are
// added over distributed shared memory in rank order (deterministic).
//
// Roles per CTA (8 + 4 G warps):
//   warp 0        TMA of the x tiles (one copy per stage)
//   warp 1        TMEM allocation; UMMA issue
//   warp 2        TMA of the code tiles (128 rows x 128 bytes: 256 K columns)
//   warps 4-7     block scales of each code tile (one row per thread)
//   warps 8-23    four dequant groups of 4 warps, group g takes the 64-wide
//                 K blocks g, g + 4, ..
// A stage is KB = 4 blocks of K (2 above 128 tokens, where two stages of x
// would not fit otherwise).  The issuing warp runs its loop as a whole, with
// one elected lane inside the instruction: its operands then stay uniform and
// an UMMA of 16 tokens issues in 10 clocks; from a one-lane branch it took 118.
// Every wait is bounded, as in gemm_sm100.cuh; no TMA multicast.
#pragma once

#include "common.cuh"

namespace qnf4 {

constexpr int kSgRows = 128;                  // weight rows per CTA
constexpr int kSgMaxN = 256;                  // tokens per CTA
constexpr int kSgUnits = 4;                   // code tiles in flight
constexpr int kSgCodeTile = kSgRows * 128;    // 16 KB: 256 K columns
constexpr int kSgABlock = kSgRows * 128;      // 16 KB: one 64-wide block of the A operand
constexpr int kSgABlocks = 8;                 // blocks of the tensor-memory A ring, 32 columns each
constexpr uint32_t kSgAccCol = 256;           // the accumulator, behind the A ring
constexpr int kSgMaxStages = 4;
constexpr int kSgGroups = 4;                  // dequant groups
constexpr int kSgThreads = (8 + 4 * kSgGroups) * 32;

// K blocks per stage, and x stages in flight (at most 64 KB).
__host__ __device__ constexpr int sg_kb(int N) { return N <= 128 ? 4 : 2; }
__host__ __device__ constexpr int sg_stages(int N) { return N <= 64 ? 4 : 2; }
__host__ __device__ constexpr int sg_x_bytes(int N) { return sg_stages(N) * sg_kb(N) * N * 128; }
__host__ __device__ constexpr int sg_list_bytes() { return 2 * kSgMaxN * 4 + 64; }
// The fp32 partial tile lies over the rings once they are done with.
__host__ __device__ constexpr int sg_ring_bytes(int N) {
  return sg_x_bytes(N) + kSgUnits * kSgCodeTile;
}
// At least kSgMinSmem, so that no other CTA of this library that allocates
// tensor memory fits beside this one (the rank-r kernels take 72 KB or more):
// two CTAs that wait for each other's tensor memory while both wait for their
// clusters could not finish.
constexpr int kSgMinSmem = 160 * 1024;
__host__ __device__ constexpr int sg_smem_bytes(int N) {
  const int need = sg_ring_bytes(N) + kSgUnits * kSgRows * 16 + sg_list_bytes() + 512 + 1024;
  return need > kSgMinSmem ? need : kSgMinSmem;
}
static_assert(kSgMaxN * kSgRows * 4 <= sg_ring_bytes(kSgMaxN) && 16 * kSgRows * 4 <= sg_ring_bytes(16),
              "the partial tile fits the rings");
__host__ __device__ constexpr int sg_tmem_cols(int) { return 512; }

struct SlotsGemmArgs {
  const int8_t* q8;
  const float* step2;
  const float* mean;
  const uint16_t* us;       // [M, r8]
  const uint16_t* B;        // [n_adapters, out, r]
  const int32_t* ids;       // [M]
  uint16_t* h;              // [M, out]
  int64_t n_adapters;
  int M, out, K, r, r8;
  int N;                    // tokens per tile (a multiple of 16)
  Levels L;
  uint64_t timeout_ns;
};

// mbar_try_wait that lets the hardware suspend the warp for up to 20 us: two
// dozen warps share the SM here.
__device__ __forceinline__ bool mbar_try_wait_hint(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok) : "r"(bar), "r"(parity), "r"(20000u) : "memory");
  return ok != 0;
}
// D[tmem] (+)= A[tmem] * B[smem desc]^T, bf16 inputs, fp32 accumulate; the
// descriptor's halves apart, since only the low one changes along K.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi,
                                             uint32_t idesc, uint32_t accumulate, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n"
      :: "r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(elected) : "memory");
}
// umma_commit by the elected lane.
__device__ __forceinline__ void umma_commit_elected(uint32_t bar, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n"
      :: "r"(bar), "r"(elected) : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
  return r;
}
// 32 lanes x 32 consecutive 32-bit columns; thread t writes lane (base+t).
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
         "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
         "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t x,
                                            int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(smem_dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)) : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void lds_v4(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}

// KB, S: sg_kb(N), sg_stages(N).
template <int KB, int S>
__global__ void __launch_bounds__(kSgThreads, 1)
slots_gemm_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_x,
                  const SlotsGemmArgs args) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const int N = args.N;
  constexpr int SA = kSgABlocks / KB;                            // stages of the A ring
  const int x_blk = N * 128, x_stage = KB * x_blk;
  uint8_t* x_ring = smem;
  uint8_t* c_ring = x_ring + S * x_stage;
  float* s_ring = reinterpret_cast<float*>(c_ring + kSgUnits * kSgCodeTile);   // [unit][block][row]
  int32_t* tok_id = reinterpret_cast<int32_t*>(s_ring + kSgUnits * kSgRows * 4);
  int32_t* list = tok_id + kSgMaxN;                          // distinct adapters, first appearance first
  int32_t* counts = list + kSgMaxN;                          // [8] leaders per warp of 32 tokens
  int32_t* odd = counts + 8;                                 // some B value of a stage was not finite
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(tok_id) + sg_list_bytes());
  uint64_t* xfull = bars;                                    // the stage's x tile landed
  uint64_t* xempty = xfull + kSgMaxStages;                   // the UMMAs on the x tile finished
  uint64_t* afull = xempty + kSgMaxStages;                   // the stage's A operand is written
  uint64_t* aempty = afull + kSgMaxStages;                   // the UMMAs on it finished
  uint64_t* cfull = aempty + kSgMaxStages;                   // the code tile landed
  uint64_t* sfull = cfull + kSgUnits;                        // its scales are written
  uint64_t* cempty = sfull + kSgUnits;                       // codes and scales are read
  uint64_t* acc_full = cempty + kSgUnits;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_tiles = (args.out + kSgRows - 1) / kSgRows;
  const int n0 = (static_cast<int>(blockIdx.x) % row_tiles) * kSgRows;
  const int m0 = (static_cast<int>(blockIdx.x) / row_tiles) * N;
  const int ks = static_cast<int>(gridDim.y), split = static_cast<int>(blockIdx.y);
  const uint64_t tmo = args.timeout_ns;
  const int n_blk = args.K / 64;
  const int n_units = (n_blk + 3) / 4;
  const int u_begin = static_cast<int>(static_cast<int64_t>(n_units) * split / ks);
  const int u_end = static_cast<int>(static_cast<int64_t>(n_units) * (split + 1) / ks);
  const int n_base = (u_end - u_begin) * 4 / KB;             // stages of the base; blocks past K are zero

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSgMaxStages; ++s) {
      mbar_init(xfull + s, 1);
      mbar_init(xempty + s, 1);
      mbar_init(afull + s, 4 * KB);                          // one arrive per warp of the stage's groups
      mbar_init(aempty + s, 1);
    }
    for (int u = 0; u < kSgUnits; ++u) {
      mbar_init(cfull + u, 1);
      mbar_init(sfull + u, 4);
      mbar_init(cempty + u, 16);                             // four blocks x four warps
    }
    mbar_init(acc_full, 1);
    *abort_flag = 0;
    *odd = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, static_cast<uint32_t>(sg_tmem_cols(N)));
    tmem_relinquish();
  }
  // the token tile's slots; -1 for no adapter and for tokens past the batch
  if (threadIdx.x < kSgMaxN) {
    const int m = m0 + static_cast<int>(threadIdx.x);
    int32_t a = -1;
    if (static_cast<int>(threadIdx.x) < N && m < args.M) {
      a = __ldg(args.ids + m);
      if (a < 0 || a >= args.n_adapters) a = -1;
    }
    tok_id[threadIdx.x] = a;
  }
  __syncthreads();
  bool leader = false;
  if (threadIdx.x < kSgMaxN) {                               // whole warps
    const int t = threadIdx.x;
    const int32_t a = tok_id[t];
    leader = a >= 0;
    for (int i = 0; leader && i < t; ++i)
      if (tok_id[i] == a) leader = false;
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, leader);
    if (lane == 0) counts[warp] = __popc(b);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  int n_list = 0;
  {
    int before = 0;
#pragma unroll
    for (int w = 0; w < kSgMaxN / 32; ++w) {
      if (w < warp) before += counts[w];
      n_list += counts[w];
    }
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, leader);
    if (leader) list[before + __popc(b & ((1u << lane) - 1u))] = tok_id[threadIdx.x];
  }
  __syncthreads();
  const uint32_t tmem_base = *tmem_holder;
  const int k_low = n_list * args.r8;                        // rank columns of the listed adapters
  const int n_low_all = (k_low + 64 * KB - 1) / (64 * KB);   // adapter stages
  const int l_begin = static_cast<int>(static_cast<int64_t>(n_low_all) * split / ks);
  const int n_low = static_cast<int>(static_cast<int64_t>(n_low_all) * (split + 1) / ks) - l_begin;
  const int n_it = n_base + n_low;

  // Bounded wait; false once it, or any other wait of the CTA, ran out of time.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    const uint32_t a = smem_u32(bar);
    if (mbar_try_wait_hint(a, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait_hint(a, parity)) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > tmo) {
        *abort_flag = 1;
        raise_device_error(1);
        return false;
      }
    }
    return true;
  };
  // the same answer for every lane of a warp (the roles that work as whole warps)
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity)) != 0; };

  if (warp == 0) {
    // ------------------------------------------------------------ x tiles
    if (lane == 0) {
      tma_prefetch_desc(&tm_x);
      int issued = 0;
      for (int it = 0; it < n_base; ++it) {
        const int s = it % S;
        if (!wait(xempty + s, ((it / S) & 1u) ^ 1u)) break;
        mbar_arrive_expect_tx(xfull + s, static_cast<uint32_t>(x_stage));
        tma_load_3d(smem_u32(x_ring + s * x_stage), &tm_x, xfull + s, 0, m0, 4 * u_begin + it * KB);
        ++issued;
      }
      // only the last S issued stages can still be in flight
      for (int it = issued > S ? issued - S : 0; it < issued; ++it)
        mbar_wait_bounded(xfull + (it % S), (it / S) & 1u, tmo);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ UMMA issuer
    const uint32_t idesc = umma_idesc_bf16(kSgRows, N, false);
    const uint64_t desc_x = umma_desc_sw128(smem_u32(x_ring), 16, 1024);
    const uint32_t hi = static_cast<uint32_t>(desc_x >> 32);
    const uint32_t x_lo = static_cast<uint32_t>(desc_x);
    const uint32_t elected = elect_one();
    uint32_t acc = 0;
    for (int it = 0; it < n_it; ++it) {
      const int s = it % S, sa = it % SA;
      int blocks;                                            // blocks that hold anything
      if (it < n_base) {
        blocks = min(KB, n_blk - 4 * u_begin - it * KB);
        if (!wait_warp(xfull + s, (it / S) & 1u)) break;     // an adapter stage's x tile comes with its A operand
      } else {
        blocks = min(KB, (k_low + 63) / 64 - (l_begin + it - n_base) * KB);
      }
      if (!wait_warp(afull + sa, (it / SA) & 1u)) break;
      tc_fence_after_sync();
      uint32_t b = x_lo + ((s * x_stage) >> 4);
      uint32_t a = tmem_base + sa * KB * 32;
#pragma unroll
      for (int blk = 0; blk < KB; ++blk, b += x_blk >> 4, a += 32) {
        if (blk >= blocks) break;
        umma_bf16_ts(tmem_base + kSgAccCol, a, b, hi, idesc, acc, elected);
        umma_bf16_ts(tmem_base + kSgAccCol, a + 8, b + 2, hi, idesc, 1u, elected);
        umma_bf16_ts(tmem_base + kSgAccCol, a + 16, b + 4, hi, idesc, 1u, elected);
        umma_bf16_ts(tmem_base + kSgAccCol, a + 24, b + 6, hi, idesc, 1u, elected);
        acc = 1u;
      }
      umma_commit_elected(smem_u32(aempty + sa), elected);
      umma_commit_elected(smem_u32(xempty + s), elected);
    }
    umma_commit_elected(smem_u32(acc_full), elected);
    mbar_wait_bounded(acc_full, 0, tmo);
  } else if (warp == 2) {
    // ------------------------------------------------------------ code tiles
    if (lane == 0) {
      tma_prefetch_desc(&tm_codes);
      int issued = 0;
      for (int u = 0; u < u_end - u_begin; ++u) {
        const int s = u % kSgUnits;
        if (!wait(cempty + s, ((u / kSgUnits) & 1u) ^ 1u)) break;
        mbar_arrive_expect_tx(cfull + s, kSgCodeTile);
        tma_load_2d(smem_u32(c_ring + s * kSgCodeTile), &tm_codes, cfull + s, (u_begin + u) * 128, n0);
        ++issued;
      }
      for (int u = issued > kSgUnits ? issued - kSgUnits : 0; u < issued; ++u)
        mbar_wait_bounded(cfull + (u % kSgUnits), (u / kSgUnits) & 1u, tmo);
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ block scales
    // Thread t owns weight row n0 + t: the four scales of each code tile,
    // loaded two tiles ahead.
    const int t = threadIdx.x - 128;
    const int64_t row_blk = static_cast<int64_t>(n0 + t) * n_blk;
    const bool row_ok = n0 + t < args.out;
    const float mu = __ldg(args.mean);
    const bool word = (n_blk & 3) == 0;                      // a tile's four codes are one aligned word
    struct In { uint32_t q; float s0, s3; };
    auto load = [&](int u, In& d) {
      if (!row_ok || u >= u_end) return;
      const int64_t i = row_blk + 4 * u;
      const int last = min(3, n_blk - 1 - 4 * u);
      if (word) {
        d.q = __ldg(reinterpret_cast<const uint32_t*>(args.q8 + i));
      } else {
        d.q = 0;
        for (int b = 0; b <= last; ++b) d.q |= static_cast<uint32_t>(static_cast<uint8_t>(__ldg(args.q8 + i + b))) << (8 * b);
      }
      d.s0 = __ldg(args.step2 + i / 256);
      d.s3 = __ldg(args.step2 + (i + last) / 256);
    };
    In a{}, b{};
    load(u_begin, a);
    load(u_begin + 1, b);
    for (int u = u_begin; u < u_end; ++u) {
      const In cur = a;
      a = b;
      load(u + 2, b);
      const int k = u - u_begin, s = k % kSgUnits;
      if (!wait_warp(cempty + s, ((k / kSgUnits) & 1u) ^ 1u)) break;
      const int64_t i = row_blk + 4 * u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float st = ((i + e) / 256 == i / 256) ? cur.s0 : cur.s3;
        const int q = static_cast<int8_t>(cur.q >> (8 * e));
        s_ring[(s * 4 + e) * kSgRows + t] = row_ok && 4 * u + e < n_blk ? block_scale(q, st, mu) : 0.f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sfull + s);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ dequant groups
    const int g = (warp - 8) >> 2;
    const int quad = warp & 3;
    const int t = quad * 32 + lane;                          // weight row of the tile
    // Above 128 tokens a group's x slot is also that of the groups two stages
    // away: its last stage before `it` must be done before an adapter
    // stage writes the slot.  Waited for at every stage, so that no phase of
    // that barrier is skipped.
    auto x_done = [&](int it) { return it < 2 || wait_warp(aempty + (it - 2) % SA, ((it - 2) / SA) & 1u); };
    for (int i = g; i < n_it * KB; i += kSgGroups) {         // 64-wide blocks of the stages
      const int it = i / KB, s = it % S, sa = it % SA, ib = i % KB;
      uint32_t v[32];
      if (it < n_base) {
        const int k = i >> 2, cs = k % kSgUnits, blk = i & 3;
        const uint32_t par = (k / kSgUnits) & 1u;
        if (!wait_warp(cfull + cs, par) || !wait_warp(sfull + cs, par)) break;
        const uint32_t crow = smem_u32(c_ring + cs * kSgCodeTile) + t * 128;
        uint32_t c[8];
        lds_v4(crow + (((2 * blk) ^ (t & 7)) << 4), *reinterpret_cast<uint32_t(*)[4]>(&c[0]));
        lds_v4(crow + (((2 * blk + 1) ^ (t & 7)) << 4), *reinterpret_cast<uint32_t(*)[4]>(&c[4]));
        const float c_hat = s_ring[(cs * 4 + blk) * kSgRows + t];
        __syncwarp();
        if (lane == 0) mbar_arrive(cempty + cs);
        const Nf4Table tb = make_table(args.L, c_hat);
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          uint32_t o[4];
          decode8(tb, c[w], o);
          v[4 * w] = o[0]; v[4 * w + 1] = o[1]; v[4 * w + 2] = o[2]; v[4 * w + 3] = o[3];
        }
        if (!wait_warp(aempty + sa, ((it / SA) & 1u) ^ 1u)) break;
      } else {
        // adapter stage: rank columns [64 e, 64 e + 64) of the listed adapters, in chunks of 8
        const int e = (l_begin + it - n_base) * KB + ib;
        const bool row_ok = n0 + t < args.out;
        if (!wait_warp(aempty + sa, ((it / SA) & 1u) ^ 1u)) break;
        if (SA > S && !x_done(it)) break;
        const uint32_t x_base = smem_u32(x_ring + s * x_stage + ib * x_blk);
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const int kk = e * 64 + ch * 8;
          const int li = kk / args.r8, j0 = kk - li * args.r8;
          const bool live = kk < k_low;
          const int32_t a = live ? list[li] : -2;
          uint4 bv = make_uint4(0, 0, 0, 0);
          if (live && row_ok) {
            const uint16_t* src = args.B + (static_cast<int64_t>(a) * args.out + n0 + t) * args.r + j0;
            if ((args.r & 7) == 0) {
              bv = ld_nc_v4(src);
            } else {
              uint32_t w[4] = {0, 0, 0, 0};
              for (int c = 0; c < 8; ++c)
                if (j0 + c < args.r) w[c >> 1] |= static_cast<uint32_t>(__ldg(src + c)) << (16 * (c & 1));
              bv = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          v[4 * ch] = bv.x; v[4 * ch + 1] = bv.y; v[4 * ch + 2] = bv.z; v[4 * ch + 3] = bv.w;
#pragma unroll
          for (int w = 4 * ch; w < 4 * ch + 4; ++w) {
            if ((v[w] & 0x7F80u) == 0x7F80u) { v[w] &= 0xFFFF0000u; *odd = 1; }
            if ((v[w] & 0x7F800000u) == 0x7F800000u) { v[w] &= 0xFFFFu; *odd = 1; }
          }
          for (int m = t; m < N; m += 128) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (tok_id[m] == a) u = *reinterpret_cast<const uint4*>(args.us + static_cast<int64_t>(m0 + m) * args.r8 + j0);
            sts_v4(x_base + m * 128 + ((ch ^ (m & 7)) << 4), u.x, u.y, u.z, u.w);
          }
        }
        fence_proxy_async_smem();                            // generic writes before the UMMA reads
      }
      tmem_st_32x32b_x32(tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + (sa * KB + ib) * 32, v);
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(afull + sa);
      if (SA > S && it < n_base && !x_done(it)) break;
    }
  }

  // ---------------------------------------------------------------- epilogue
  __syncwarp();
  wait(acc_full, 0);
  tc_fence_after_sync();
  __syncthreads();                                           // every copy has landed, every stage is read
  float* part = reinterpret_cast<float*>(smem);              // [token][row], over the rings
  if (warp >= 8) {
    const int quad = warp & 3;
    for (int c0 = ((warp - 8) >> 2) * 16; c0 < N; c0 += 16 * kSgGroups) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(tmem_base + kSgAccCol + (static_cast<uint32_t>(quad * 32) << 16) + c0, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) part[(c0 + i) * kSgRows + quad * 32 + lane] = __uint_as_float(v[i]);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (ks > 1) cluster_sync_all();                            // every CTA's partial is in place
  int any_odd = 0;
  for (int rk = 0; rk < ks; ++rk) {
    int o;
    if (ks == 1) o = *odd;
    else asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(o) : "r"(mapa_shared(smem_u32(odd), rk)) : "memory");
    any_odd |= o;
  }
  // this CTA's tokens: split, split + ks, ...; one warp per token, four rows per lane
  const int n = n0 + 4 * lane;
  for (int t = split + ks * warp; t < N; t += ks * (kSgThreads / 32)) {
    const int m = m0 + t;
    if (m >= args.M) break;
    const uint32_t addr = smem_u32(part + t * kSgRows + 4 * lane);
    float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int rk = 0; rk < ks; ++rk) {
      float4 p;
      if (ks == 1) {
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(p.x), "=f"(p.y), "=f"(p.z), "=f"(p.w)
                     : "r"(addr) : "memory");
      } else {
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(p.x), "=f"(p.y), "=f"(p.z), "=f"(p.w) : "r"(mapa_shared(addr, rk)) : "memory");
      }
      d.x += p.x; d.y += p.y; d.z += p.z; d.w += p.w;
    }
    if (any_odd && n < args.out && tok_id[t] >= 0) {         // the products left out of the stages
      float* dd[4] = {&d.x, &d.y, &d.z, &d.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint16_t* src = args.B + (static_cast<int64_t>(tok_id[t]) * args.out + n + e) * args.r;
        for (int j = 0; j < args.r; ++j) {
          const uint32_t b = __ldg(src + j);
          if ((b & 0x7F80u) == 0x7F80u)
            *dd[e] = fmaf(__uint_as_float(static_cast<uint32_t>(args.us[static_cast<int64_t>(m) * args.r8 + j]) << 16),
                          __uint_as_float(b << 16), *dd[e]);
        }
      }
    }
    if (n < args.out)
      *reinterpret_cast<uint2*>(args.h + static_cast<int64_t>(m) * args.out + n) =
          make_uint2(pack_bf16x2_rn(d.x, d.y), pack_bf16x2_rn(d.z, d.w));
  }
  if (ks > 1) cluster_sync_all();                            // no CTA leaves while others read it
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, static_cast<uint32_t>(sg_tmem_cols(N)));
  }
}

}  // namespace qnf4
