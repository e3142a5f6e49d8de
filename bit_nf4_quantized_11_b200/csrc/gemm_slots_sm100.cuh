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
// The adapters ride along as extra K.  The CTA lists the distinct adapters of
// the tokens (first appearance first); the rank columns of the listed
// adapters, one after another, form a K axis behind that of the base: the A
// operand is B_a[n][j], the B operand us[m][j] where token m uses that adapter
// and zero elsewhere.  A B value that is infinite or NaN would reach the other
// tokens through their zeros, so it is carried as 0 and the tile is marked;
// the epilogue then adds those products to the adapter's own tokens.
//
// Schedule: K is cut into units of 256; the units of all row tiles, tile after
// tile, are dealt out evenly to a persistent grid of one CTA per SM, so every
// CTA streams the same amount whatever the shape.  A tile that one CTA holds
// goes straight to h; of a tile cut between CTAs each leaves an fp32 partial,
// and the one that finishes last (a ticket per tile) adds them in CTA order,
// so the result does not depend on which CTA ran when.  (Rounds of whole
// tiles, split over clusters, lost a quarter to the last round and paid a
// prologue per round: 125 us for the 70B up projection at 16 tokens.)
//
// Decode.  The integer pipe (64 lanes per clock) bounds a decode by byte
// permutes, about 4 operations per weight.  Up to 128 tokens there is room
// for a 64 KB table instead, for every byte of two codes the two fp32 levels,
// one copy per lane: a pair of weights takes one prmt (the address), one
// 8-byte shared load, one packed fp32 multiply and one conversion, and every
// weight is bf16(level * scale) as everywhere else.  Under that load every
// shared-memory access (a barrier poll too) takes about 300 clocks (counted
// likewise), so the
// chain of a block counts: its lookups go out in four batches of 8, the next
// one before the last is converted, and the barriers ahead are polled before
// the last batches and looked at behind them.
//
// Roles per CTA (24 warps):
//   warp 0        TMA of the x tiles (one copy per stage)
//   warp 1        TMEM allocation; UMMA issue
//   warp 2        TMA of the code tiles (128 rows x 128 bytes: one unit)
//   warp 3        waits for the kernel before, so that no CTA ends ahead of it
//   warps 4-7     block scales of each code tile (one row per thread)
//   warps 8-23    four dequant groups of 4 warps, group g takes the g-th
//                 64-wide block of every unit; then the epilogue
// A stage is KB = 4 blocks of K (2 above 64 tokens, where two stages of x
// would not fit otherwise).  The issuing warp runs its loop as a whole, with
// one elected lane inside the instruction: its operands then stay uniform and
// an UMMA of 16 tokens issues in 10 clocks; from a one-lane branch it took 118
// (clock counters around the loop, in a build for it).
// Every wait is bounded, as in gemm_sm100.cuh; no TMA multicast.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "slots.cuh"

namespace qnf4 {

constexpr int kSgRows = 128;                  // weight rows per tile
constexpr int kSgMaxN = 256;                  // tokens per launch
constexpr int kSgMaxCtas = 256;
constexpr int kSgHash = 512;
constexpr int kSgUnits = 3;                   // code tiles in flight
constexpr int kSgCodeTile = kSgRows * 128;    // 16 KB: 256 K columns
constexpr int kSgABlocks = 8;                 // blocks of the tensor-memory A ring, 32 columns each
constexpr uint32_t kSgAccCol = 256;           // the accumulator, behind the A ring
constexpr uint32_t kSgTmemCols = 512;
constexpr int kSgMaxStages = 4;
constexpr int kSgGroups = 4;                  // dequant groups
constexpr int kSgDecThreads = kSgGroups * 128;
constexpr int kSgThreads = 256 + kSgDecThreads;

// K blocks per stage; two x stages in flight (64 KB, without the table 128 KB).
__host__ __device__ constexpr int sg_kb(int N) { return N <= 64 ? 4 : 2; }
constexpr int kSgXStages = 2;
__host__ __device__ constexpr bool sg_lut(int N) { return N <= 128; }
// Shared memory by absolute shared address: the level table sits on a 64 KB
// boundary (prmt assembles its addresses), x behind it; codes, scales, lists
// and barriers before it.  Without the table x starts at the boundary.
constexpr uint32_t kSgTableAt = 0x10000;
__host__ __device__ constexpr int sg_low_bytes() {
  return kSgUnits * (kSgCodeTile + kSgRows * 16) + 2 * kSgMaxN * 4 + 64 + 512;
}
// No other CTA of this library that allocates tensor memory fits beside this
// one (the rank-r kernels take 72 KB or more): two that waited for each
// other's columns while both wait for their clusters could not finish.
constexpr int kSgMinSmem = 160 * 1024;
__host__ __device__ constexpr int sg_smem_bytes(int N) {   // (the window starts at or above address 0)
  const int need = static_cast<int>(kSgTableAt) + (sg_lut(N) ? 65536 + kSgXStages * sg_kb(N) * N * 128 : 131072);
  return need > kSgMinSmem ? need : kSgMinSmem;
}
static_assert(sg_low_bytes() + 1024 + 1024 <= static_cast<int>(kSgTableAt), "the low part fits below the table");
static_assert(sg_smem_bytes(kSgMaxN) <= 227 * 1024 && sg_smem_bytes(128) <= 227 * 1024, "shared memory of a CTA");
static_assert(kSgMinSmem > (228 - 72) * 1024, "one CTA with tensor memory per SM");

struct SlotsGemmArgs {
  const int8_t* q8;
  const float* step2;
  const float* mean;
  const uint16_t* us;       // [M, r8]
  const uint16_t* B;        // [n_adapters, out, r]
  const int32_t* ids;       // [M], or null: adapter 0 throughout
  uint16_t* h;              // [M, out]
  float* part;              // [2 * CTAs][N][128]: a CTA's first and last tile, where cut
  uint32_t* tickets;        // [row tiles], zero before the launch
  int64_t n_adapters;
  int M, out, K, r, r8;     // M <= 256
  int N;                    // M rounded up to 16
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
// The waiting part of a bounded wait, out of line: two dozen copies of it cost
// instruction fetches in the roles' loops.
__device__ __noinline__ bool sg_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort_flag) {
  if (mbar_try_wait_hint(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait_hint(bar, parity)) {
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > timeout_ns) {
      *abort_flag = 1;
      raise_device_error(1);
      return false;
    }
  }
  return true;
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
// Whether a phase is complete, without waiting: asked early, looked at late.
__device__ __forceinline__ uint32_t mbar_probe(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok;
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t x,
                                            int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(smem_dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void lds_v4(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// T units dealt out to G CTAs: CTA c begins at floor(T c / G).  (T fits 32 bits:
// at most 2^23 row tiles with 256 adapter units each, and 2^40 weights.)
struct SgDeal {
  uint32_t T, G, each, rest;
  __device__ SgDeal(uint32_t T_, uint32_t G_) : T(T_), G(G_), each(T_ / G_), rest(T_ % G_) {}
  __device__ __forceinline__ uint32_t begin(uint32_t c) const { return each * c + rest * c / G; }
  // the CTA that holds unit u
  __device__ __forceinline__ int holder(uint32_t u) const {
    int c = min(static_cast<int>(G) - 1, static_cast<int>(static_cast<float>(u) * (static_cast<float>(G) / static_cast<float>(T))));
    while (c > 0 && begin(c) > u) --c;
    while (c + 1 < static_cast<int>(G) && begin(c + 1) <= u) ++c;
    return c;
  }
};

// KB, kLut: sg_kb(N), sg_lut(N).
template <int KB, bool kLut>
__global__ void __launch_bounds__(kSgThreads, 1)
slots_gemm_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_x,
                  const SlotsGemmArgs args) {
  constexpr int S = kSgXStages;
  constexpr int SA = kSgABlocks / KB;                        // stages of the A ring
  constexpr bool kOneRing = S == SA;                         // x and A slots are freed together
  constexpr int SPU = 4 / KB;                                // stages per unit
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* low = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* table = smem_raw + (kSgTableAt - raw_addr);
  const int N = args.N;
  const int x_blk = N * 128, x_stage = KB * x_blk;
  uint8_t* c_ring = low;
  float* s_ring = reinterpret_cast<float*>(c_ring + kSgUnits * kSgCodeTile);   // [unit][block][row]
  int32_t* list = reinterpret_cast<int32_t*>(s_ring + kSgUnits * kSgRows * 4);
                                                                                    // distinct adapters, first appearance first
  int32_t* tok_col = list + kSgMaxN;                         // a token's first rank column, or far past the last
  int32_t* counts = tok_col + kSgMaxN;                       // [8] leaders per warp of 32 tokens
  volatile int32_t* odd = counts + 8;                        // [2] by segment: a B value was not finite
  volatile int32_t* last_flag = counts + 10;                 // [2]: the ticket of the CTA's first and last tile
  volatile int32_t* cut = counts + 12;                       // [2][2]: their first CTA's partial, how many CTAs share them
  uint8_t* x_ring = kLut ? table + 65536 : table;
  uint64_t* bars = reinterpret_cast<uint64_t*>(counts + 16);
  uint64_t* xfull = bars;                                    // the stage's x tile landed
  uint64_t* xempty = xfull + kSgMaxStages;                   // the UMMAs on the x tile finished
  uint64_t* afull = xempty + kSgMaxStages;                   // the stage's A operand is written
  uint64_t* aempty = afull + kSgMaxStages;                   // the UMMAs on it finished
  uint64_t* cfull = aempty + kSgMaxStages;                   // the code tile landed
  uint64_t* sfull = cfull + kSgUnits;                        // its scales are written too
  uint64_t* cempty = sfull + kSgUnits;                       // codes and scales are read
  uint64_t* acc_full = cempty + kSgUnits;                    // a segment's accumulator is complete
  uint64_t* acc_empty = acc_full + 1;                        // and read
  uint64_t* dec_bar = acc_empty + 1;                         // the dequant warps among themselves
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(dec_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t tmo = args.timeout_ns;
  const int n_blk = args.K / 64;
  const int UB = (n_blk + 3) / 4;                            // base units per tile

  // The tokens' slots (-1: no adapter, or past the batch): of up to 32 tokens
  // every warp looks at all, of more each thread has its own.
  const bool one_warp = args.M <= 32;
  int32_t my_id = -1;
  if (one_warp && lane < args.M) my_id = args.ids != nullptr ? __ldg(args.ids + lane) : 0;
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
    mbar_init(acc_empty, 16);
    mbar_init(dec_bar, 16);
    *abort_flag = 0;
    odd[0] = odd[1] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_codes);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, kSgTmemCols);
    tmem_relinquish();
  }
  if (kLut && warp >= 8) {
    // row b (256 bytes): lane l's copy of {level of the low code, level of the high code} at 8 l
    const float low_level = args.L.v[warp - 8];
    static_assert(kSgDecThreads == 512, "a warp fills the rows of one low code");
#pragma unroll
    for (int hi = 0; hi < 16; ++hi)
      *reinterpret_cast<float2*>(table + (16 * hi + warp - 8) * 256 + lane * 8) = make_float2(low_level, args.L.v[hi]);
  }
  if (!one_warp && threadIdx.x < kSgMaxN && static_cast<int>(threadIdx.x) < args.M)
    my_id = args.ids != nullptr ? __ldg(args.ids + threadIdx.x) : 0;
  if (my_id < 0 || my_id >= args.n_adapters) my_id = -1;
  int n_list, place;
  if (one_warp) {                                            // every warp for itself
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, my_id);
    const int first = __ffs(static_cast<int>(same)) - 1;
    const uint32_t lead = __ballot_sync(0xFFFFFFFFu, my_id >= 0 && first == lane);
    n_list = __popc(lead);
    place = my_id < 0 ? -1 : __popc(lead & ((1u << first) - 1u));
    if (warp == 3) {
      if (my_id >= 0 && first == lane) list[place] = my_id;
      tok_col[lane] = place < 0 ? -(1 << 29) : place * args.r8;
    }
  } else {                                                   // the hash table lies over the code ring, not in use yet
    n_list = distinct_slots<kSgMaxN, kSgHash>(my_id, reinterpret_cast<int32_t*>(c_ring), list, counts, place);
    if (threadIdx.x < kSgMaxN) tok_col[threadIdx.x] = place < 0 ? -(1 << 29) : place * args.r8;
    fence_proxy_async_smem();                                // the table's words before the copies over them
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_holder;
  const int k_low = n_list * args.r8;                        // rank columns of the listed adapters
  const int low_blk = (k_low + 63) / 64;
  const int UPT = UB + (low_blk + 3) / 4;                    // units per tile
  const SgDeal deal(static_cast<uint32_t>((args.out + kSgRows - 1) / kSgRows) * UPT, gridDim.x);
  const uint32_t g0 = deal.begin(blockIdx.x);
  const int n_u = static_cast<int>(deal.begin(blockIdx.x + 1) - g0);           // this CTA's units
  const int tile0 = static_cast<int>(g0 / UPT), uu0 = static_cast<int>(g0 % UPT);

  // Bounded wait; false once it, or any other wait of the CTA, ran out of time.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return mbar_probe(smem_u32(bar), parity) != 0 || sg_wait(smem_u32(bar), parity, tmo, abort_flag);
  };
  // the same answer for every lane of a warp (the roles that work as whole warps)
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity)) != 0; };
  // by address, after a probe that was taken earlier
  auto settled = [&](uint32_t probed, uint32_t bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, probed || mbar_probe(bar, parity) || sg_wait(bar, parity, tmo, abort_flag)) != 0;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ x tiles
    if (lane == 0) {
      int it = 0, uu = uu0;
      bool ok = true;
      for (int i = 0; i < n_u && ok; ++i) {
        for (int j = 0; j < SPU; ++j, ++it) {
          const int s = it % S;
          if (!(ok = wait((kOneRing ? aempty : xempty) + s, ((it / S) & 1u) ^ 1u))) break;
          if (uu < UB) {
            mbar_arrive_expect_tx(xfull + s, static_cast<uint32_t>(x_stage));
            tma_load_3d(smem_u32(x_ring + s * x_stage), &tm_x, xfull + s, 0, 0, uu * 4 + j * KB);
          } else {
            mbar_arrive(xfull + s);                          // an adapter stage: the dequant groups fill it
          }
        }
        if (++uu == UPT) uu = 0;
      }
      // only the last S stages can still be in flight
      for (int k = it > S ? it - S : 0; k < it; ++k) mbar_wait_bounded(xfull + (k % S), (k / S) & 1u, tmo);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ UMMA issuer
    const uint32_t idesc = umma_idesc_bf16(kSgRows, N, false);
    const uint64_t desc_x = umma_desc_sw128(smem_u32(x_ring), 16, 1024);
    const uint32_t hi = static_cast<uint32_t>(desc_x >> 32);
    const uint32_t x_lo = static_cast<uint32_t>(desc_x);
    const uint32_t d = tmem_base + kSgAccCol;
    const uint32_t elected = elect_one();
    uint32_t acc = 0;
    int it = 0, uu = uu0, seg = 0;
    bool ok = true;
    for (int i = 0; i < n_u && ok; ++i) {
      if (acc == 0 && seg > 0 && !(ok = wait_warp(acc_empty, (seg - 1) & 1u))) break;
      for (int j = 0; j < SPU; ++j, ++it) {
        const int s = it % S, sa = it % SA;
        const int blocks = uu < UB ? n_blk - uu * 4 - j * KB : low_blk - (uu - UB) * 4 - j * KB;
        if (!(ok = wait_warp(xfull + s, (it / S) & 1u) && wait_warp(afull + sa, (it / SA) & 1u))) break;
        tc_fence_after_sync();
        uint32_t b = x_lo + ((s * x_stage) >> 4);
        uint32_t a = tmem_base + sa * KB * 32;
#pragma unroll
        for (int blk = 0; blk < KB; ++blk, b += x_blk >> 4, a += 32) {
          if (blk >= blocks) break;
          umma_bf16_ts(d, a, b, hi, idesc, acc, elected);
          umma_bf16_ts(d, a + 8, b + 2, hi, idesc, 1u, elected);
          umma_bf16_ts(d, a + 16, b + 4, hi, idesc, 1u, elected);
          umma_bf16_ts(d, a + 24, b + 6, hi, idesc, 1u, elected);
          acc = 1u;
        }
        umma_commit_elected(smem_u32(aempty + sa), elected);
        if (!kOneRing) umma_commit_elected(smem_u32(xempty + s), elected);
      }
      if (++uu == UPT || i == n_u - 1) {                     // the segment ends
        uu = 0;
        acc = 0;
        ++seg;
        umma_commit_elected(smem_u32(acc_full), elected);
      }
    }
    // every UMMA finished before the CTA may leave
    if (ok) mbar_wait_bounded(acc_full, (seg - 1) & 1u, tmo);
    else {
      umma_commit_elected(smem_u32(acc_full), elected);
      mbar_wait_bounded(acc_full, seg & 1u, tmo);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ code tiles
    if (lane == 0) {
      int uu = uu0, tile = tile0, s = 0, issued = 0;
      uint32_t ph = 1;
      for (int i = 0; i < n_u; ++i) {
        if (uu < UB) {
          if (!wait(cempty + s, ph)) break;
          mbar_arrive_expect_tx(cfull + s, kSgCodeTile);
          tma_load_2d(smem_u32(c_ring + s * kSgCodeTile), &tm_codes, cfull + s, uu * 128, tile * kSgRows);
          ++issued;
          if (++s == kSgUnits) { s = 0; ph ^= 1u; }
        }
        if (++uu == UPT) { uu = 0; ++tile; }
      }
      for (int k = issued > kSgUnits ? issued - kSgUnits : 0; k < issued; ++k)
        mbar_wait_bounded(cfull + (k % kSgUnits), (k / kSgUnits) & 1u, tmo);
    }
  } else if (warp == 3) {
    // With no adapter in use and no tile cut nothing else waits for the kernel
    // before; what follows this one in the stream relies on it too.
    grid_dependency_wait();
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ block scales
    // Thread t owns row t of each tile: the four scales of each code tile,
    // loaded two units ahead.
    const int t = threadIdx.x - 128;
    const float mu = __ldg(args.mean);
    const bool word = (n_blk & 3) == 0;                      // a unit's four codes are one aligned word
    struct In { uint32_t q; float s0, s3; };
    int l_uu = uu0, l_tile = tile0, l_i = 0;                 // the next unit to load
    auto load = [&](In& d) {
      if (l_i++ >= n_u) return;
      const int row = l_tile * kSgRows + t;
      if (l_uu < UB && row < args.out) {
        const int64_t i = static_cast<int64_t>(row) * n_blk + 4 * l_uu;
        const int last = min(3, n_blk - 1 - 4 * l_uu);
        if (word) {
          d.q = __ldg(reinterpret_cast<const uint32_t*>(args.q8 + i));
        } else {
          d.q = 0;
          for (int b = 0; b <= last; ++b)
            d.q |= static_cast<uint32_t>(static_cast<uint8_t>(__ldg(args.q8 + i + b))) << (8 * b);
        }
        d.s0 = __ldg(args.step2 + i / 256);
        d.s3 = __ldg(args.step2 + (i + last) / 256);
      }
      if (++l_uu == UPT) { l_uu = 0; ++l_tile; }
    };
    In a{}, b{};
    load(a);
    load(b);
    int uu = uu0, tile = tile0, s = 0;
    uint32_t ph = 1;
    for (int i = 0; i < n_u; ++i) {
      const In cur = a;
      a = b;
      load(b);
      if (uu < UB) {
        if (!wait_warp(cempty + s, ph)) break;
        const int row = tile * kSgRows + t;
        const int64_t idx = static_cast<int64_t>(row) * n_blk + 4 * uu;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float st = ((idx + e) / 256 == idx / 256) ? cur.s0 : cur.s3;
          const int q = static_cast<int8_t>(cur.q >> (8 * e));
          s_ring[(s * 4 + e) * kSgRows + t] = row < args.out && 4 * uu + e < n_blk ? block_scale(q, st, mu) : 0.f;
        }
        if (!wait_warp(cfull + s, ph ^ 1u)) break;           // codes too: the dequant groups wait for sfull alone
        __syncwarp();
        if (lane == 0) mbar_arrive(sfull + s);
        if (++s == kSgUnits) { s = 0; ph ^= 1u; }
      }
      if (++uu == UPT) { uu = 0; ++tile; }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ dequant groups
    const int g = (warp - 8) >> 2;
    const int quad = warp & 3;
    const int t = quad * 32 + lane;                          // weight row of the tile
    const int ib = g % KB;                                   // the group's block within its stage
    const uint32_t a_lane = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    // prmt operand that completes a code byte to its table address
    const uint32_t lut_base = kSgTableAt | (static_cast<uint32_t>(lane) * 8u);
    // Above 64 tokens a group's x slot is also that of the groups two stages
    // away: its last stage before `it` must be done before an adapter stage
    // writes the slot.  Waited for at every stage, so that no phase of that
    // barrier is skipped.
    auto x_done = [&](int it) { return it < 2 || wait_warp(aempty + (it - 2) % SA, ((it - 2) / SA) & 1u); };
    auto odd_term = [&](int m, int n) {
      if (tok_col[m] < 0) return 0.f;
      const int64_t a = list[tok_col[m] / args.r8];
      return slots_odd_term(args.B + (a * args.out + n) * args.r,
                                          args.us + static_cast<int64_t>(m) * args.r8, args.r);
    };
    uint32_t dph = 0;
    auto dec_sync = [&]() {                                  // all dequant warps, bounded
      __syncwarp();
      if (lane == 0) mbar_arrive(dec_bar);
      const bool done = wait_warp(dec_bar, dph);
      dph ^= 1u;
      return done;
    };
    int uu = uu0, tile = tile0, seg = 0, seg_uu = uu0;
    uint32_t cph = 0;
    // The CTA's first and last tile, cut between CTAs or not: which CTAs hold
    // units of them.  Found here, while the first codes are on their way.
    if (threadIdx.x < 256 + 2) {
      const int c = static_cast<int>(threadIdx.x) - 256;
      const uint32_t u_lo = (c == 0 ? static_cast<uint32_t>(tile0) : (g0 + n_u - 1) / UPT) * UPT;
      const int c_first = deal.holder(u_lo);
      // (a CTA leaves the part of its first tile in its first partial, that of its last one in its second)
      cut[2 * c] = 2 * c_first + (deal.begin(c_first) < u_lo ? 1 : 0);
      cut[2 * c + 1] = deal.holder(u_lo + UPT - 1) - c_first + 1;
      last_flag[c] = -1;
    }
    // The codes and the scale of a unit's block are read while the store of the
    // block before it completes.
    uint32_t c[8];
    float c_hat = 0.f;
    const uint32_t sfull_a = smem_u32(sfull), cempty_a = smem_u32(cempty), afull_a = smem_u32(afull),
                   aempty_a = smem_u32(aempty);
    const uint32_t codes_a = smem_u32(c_ring) + t * 128 + (((2 * g) ^ (t & 7)) << 4);      // the block's two 16-byte chunks:
    const uint32_t scale_a = smem_u32(s_ring) + (g * kSgRows + t) * 4;                     // here and 16 bytes across
    uint32_t cs_codes = codes_a, cs_scale = scale_a, cs_bar = 0;                           // of the ring's slot in turn
    auto read_codes = [&](uint32_t probed) {
      if (!settled(probed, sfull_a + cs_bar, cph)) return false;
      lds_v4(cs_codes, *reinterpret_cast<uint32_t(*)[4]>(&c[0]));
      lds_v4(cs_codes ^ 16u, *reinterpret_cast<uint32_t(*)[4]>(&c[4]));
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(c_hat) : "r"(cs_scale));
      __syncwarp();
      if (lane == 0) mbar_arrive_at(cempty_a + cs_bar);
      cs_codes += kSgCodeTile;
      cs_scale += kSgRows * 16;
      cs_bar += 8;
      if (cs_bar == 8 * kSgUnits) { cs_codes = codes_a; cs_scale = scale_a; cs_bar = 0; cph ^= 1u; }
      return true;
    };
    bool ok = true;
    if (uu < UB) ok = read_codes(0);
    for (int i = 0; i < n_u && ok; ++i) {
      const int it = i * SPU + g / KB, sa = it % SA;
      const bool more = i + 1 < n_u && (uu + 1 == UPT || uu + 1 < UB);    // a base unit follows
      const uint32_t a_blk = a_lane + (sa * KB + ib) * 32, a_par = ((it / SA) & 1u) ^ 1u;
      uint32_t next = 0;                                     // its codes are there
      if (kLut && uu < UB) {
        const uint32_t free = mbar_probe(aempty_a + 8 * sa, a_par);
        uint64_t c2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(c2) : "f"(c_hat));
        uint64_t lv[4][8];
        uint32_t w[16];
        auto lookup = [&](int q) {                           // the 8 bytes of codes 2 q, 2 q + 1
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            // bytes of the address: {lane copy, code byte, table, 0}
            const uint32_t addr = prmt(lut_base, c[2 * q + (b >> 2)], 0x3200u | ((4u + (b & 3)) << 4));
            asm volatile("ld.shared.b64 %0, [%1];" : "=l"(lv[q][b]) : "r"(addr));
          }
        };
        auto convert = [&](int q) {
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(lv[q][b]) : "l"(c2));
            float lo, hi2;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi2) : "l"(lv[q][b]));
            w[8 * (q & 1) + b] = pack_bf16x2_rn(lo, hi2);
          }
        };
        lookup(0);
        lookup(1);
        convert(0);
        lookup(2);
        convert(1);
        if (!(ok = settled(free, aempty_a + 8 * sa, a_par))) break;
        tc_fence_after_sync();                               // the UMMAs that read the slot, before the store over it
        tmem_st_32x32b_x16(a_blk, w);
        if (more) next = mbar_probe(sfull_a + cs_bar, cph);
        lookup(3);
        convert(2);
        convert(3);
        tmem_st_32x32b_x16(a_blk + 16, w);
      } else if (uu < UB) {
        uint32_t v[32];
        {
          const Nf4Table tb = make_table(args.L, c_hat);
#pragma unroll
          for (int w = 0; w < 8; ++w) {
            uint32_t o[4];
            decode8(tb, c[w], o);
            v[4 * w] = o[0]; v[4 * w + 1] = o[1]; v[4 * w + 2] = o[2]; v[4 * w + 3] = o[3];
          }
        }
        if (!(ok = wait_warp(aempty + sa, a_par))) break;
        tc_fence_after_sync();
        tmem_st_32x32b_x32(a_blk, v);
      } else {
        uint32_t v[32];
        // adapter block: rank columns [64 e, 64 e + 64) of the listed adapters, in chunks of 8
        const int e = (uu - UB) * 4 + g;
        const int row = tile * kSgRows + t;
        const bool row_ok = row < args.out;
        // the 8 chunks of this row's B values, all loads under way together
        int li = e * 64 / args.r8, j0 = e * 64 - li * args.r8;
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          uint4 bv = make_uint4(0, 0, 0, 0);
          if (row_ok && li < n_list) {
            const uint16_t* src = args.B + (static_cast<int64_t>(list[li]) * args.out + row) * args.r + j0;
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
          j0 += 8;
          if (j0 == args.r8) { j0 = 0; ++li; }
        }
        if (!(ok = wait_warp(aempty + sa, a_par))) break;
        tc_fence_after_sync();
        if (SA > S && !(ok = x_done(it))) break;
        grid_dependency_wait();                              // us comes from the kernel before
        // the tokens' us under the columns of their own adapter, zero elsewhere
        const uint32_t x_base = smem_u32(x_ring + (it % S) * x_stage + ib * x_blk);
        for (int m = t; m < N; m += 128) {
          const uint32_t x_row = x_base + m * 128;
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) sts_v4(x_row + ((ch ^ (m & 7)) << 4), 0, 0, 0, 0);
          const int col = tok_col[m] - e * 64;               // the token's first column in this block
          const uint16_t* src = args.us + static_cast<int64_t>(m) * args.r8;
#pragma unroll 2
          for (int j = max(0, -col); j < args.r8 && col + j < 64; j += 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(src + j);
            sts_v4(x_row + ((((col + j) >> 3) ^ (m & 7)) << 4), u.x, u.y, u.z, u.w);
          }
        }
        fence_proxy_async_smem();                            // generic writes before the UMMA reads
        uint32_t exps = 0;                                   // bit 15 or 31: an exponent of all ones
#pragma unroll
        for (int w = 0; w < 32; ++w) exps |= (v[w] & 0x7F807F80u) + 0x00800080u;
        if (exps & 0x80008000u) {
          odd[seg & 1] = 1;
#pragma unroll
          for (int w = 0; w < 32; ++w) {
            if ((v[w] & 0x7F80u) == 0x7F80u) v[w] &= 0xFFFF0000u;
            if ((v[w] & 0x7F800000u) == 0x7F800000u) v[w] &= 0xFFFFu;
          }
        }
        tmem_st_32x32b_x32(a_blk, v);
      }
      if (more && !(ok = read_codes(next))) break;
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(afull_a + 8 * sa);
      if (SA > S && uu < UB && !(ok = x_done(it))) break;

      if (++uu != UPT && i != n_u - 1) continue;
      // ---------------------------------------------------------- the segment ends
      const bool whole = seg_uu == 0 && uu == UPT;           // this CTA holds all of the tile
      const int n0 = tile * kSgRows;
      if (!(ok = wait_warp(acc_full, seg & 1u))) break;
      tc_fence_after_sync();
      const int my_odd = odd[seg & 1];
      float* part = args.part + (static_cast<int64_t>(blockIdx.x) * 2 + (seg > 0 ? 1 : 0)) * N * kSgRows;
      for (int c0 = g * 16; c0 < N; c0 += 16 * kSgGroups) {
        uint32_t d[16];
        tmem_ld_32x32b_x16(a_lane + kSgAccCol + c0, d);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int m = c0 + k;
          if (!whole) {
            part[m * kSgRows + t] = __uint_as_float(d[k]);
          } else if (m < args.M && n0 + t < args.out) {
            float f = __uint_as_float(d[k]);
            if (my_odd) f += odd_term(m, n0 + t);
            args.h[static_cast<int64_t>(m) * args.out + n0 + t] = __bfloat16_as_ushort(__float2bfloat16_rn(f));
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
      if (!whole) __threadfence();
      if (!(ok = dec_sync())) break;
      if (threadIdx.x == 256) odd[seg & 1] = 0;              // written again two segments on
      if (!whole) {
        // the answer is read when this CTA is done with its units: the part
        // that ends here is rarely the tile's last
        if (threadIdx.x == 256) {
          grid_dependency_wait();                            // the kernel before zeroes the tickets
          const uint32_t mine = 1u | (my_odd ? 0x10000u : 0u);
          last_flag[seg > 0 ? 1 : 0] = static_cast<int32_t>(atomicAdd(args.tickets + tile, mine) + mine);
        }
      }
      ++seg;
      seg_uu = 0;
      if (uu == UPT) { uu = 0; ++tile; }
    }
    // ------------------------------------------------------------ tiles cut between CTAs
    if (ok) ok = dec_sync();                                 // the tickets are there
    int32_t ticket[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      ticket[c] = last_flag[c];
      if (!ok || ticket[c] < 0 || (ticket[c] & 0xFFFF) != cut[2 * c + 1]) ticket[c] = 0;    // not the last to finish
    }
    if ((ticket[0] | ticket[1]) != 0) {
      __threadfence();
      // Four rows per lane; the loads of 8 values under way together: of up to
      // 16 tokens one per warp and 8 parts, of more four tokens and two parts.
      // Added in CTA order.
      auto add_up = [&](auto tokens) {
        constexpr int kTok = decltype(tokens)::value, kPart = 8 / kTok;
        const int steps = (args.M + kTok - 1) / kTok;
        for (int e = warp - 8; e < 2 * steps; e += kSgDecThreads / 32) {
          const int c = e < steps ? 0 : 1, m0 = (e - c * steps) * kTok;
          if (ticket[c] == 0) continue;
          const int tl = c == 0 ? tile0 : static_cast<int>((g0 + n_u - 1) / UPT);
          const int n = tl * kSgRows + 4 * lane, p_first = cut[2 * c], n_parts = cut[2 * c + 1];
          float4 d[kTok];
#pragma unroll
          for (int k = 0; k < kTok; ++k) d[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int p0 = 0; p0 < n_parts; p0 += kPart) {
            float4 p[kPart][kTok];
#pragma unroll
            for (int j = 0; j < kPart; ++j) {
              if (p0 + j >= n_parts) break;
              // the CTAs behind the first begin within the tile: their first partial
              const int at = p0 + j == 0 ? p_first : (p_first & ~1) + 2 * (p0 + j);
              const float* src = args.part + (static_cast<int64_t>(at) * N + m0) * kSgRows + 4 * lane;
#pragma unroll
              for (int k = 0; k < kTok; ++k)                 // (rows up to N, a multiple of 16, are there)
                p[j][k] = __ldcg(reinterpret_cast<const float4*>(src + k * kSgRows));
            }
#pragma unroll
            for (int j = 0; j < kPart; ++j) {
              if (p0 + j >= n_parts) break;
#pragma unroll
              for (int k = 0; k < kTok; ++k) {
                d[k].x += p[j][k].x; d[k].y += p[j][k].y; d[k].z += p[j][k].z; d[k].w += p[j][k].w;
              }
            }
          }
#pragma unroll
          for (int k = 0; k < kTok; ++k) {
            const int m = m0 + k;
            if (m >= args.M || n >= args.out) break;
            if (ticket[c] > 0xFFFF) {                        // some part was marked
              d[k].x += odd_term(m, n);
              d[k].y += odd_term(m, n + 1);
              d[k].z += odd_term(m, n + 2);
              d[k].w += odd_term(m, n + 3);
            }
            *reinterpret_cast<uint2*>(args.h + static_cast<int64_t>(m) * args.out + n) =
                make_uint2(pack_bf16x2_rn(d[k].x, d[k].y), pack_bf16x2_rn(d[k].z, d[k].w));
          }
        }
      };
      if (args.M <= 16) add_up(std::integral_constant<int, 1>{});
      else add_up(std::integral_constant<int, 4>{});
    }
  }

  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, kSgTmemCols);
  }
}

}  // namespace qnf4
