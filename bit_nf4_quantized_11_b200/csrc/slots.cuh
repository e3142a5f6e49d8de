// slots.cuh -- one low-rank adapter per request beside the shared NF4 base:
//   h[m] = W0 x[m] + scale_a B_a (A_a x[m]),   a = ids[m]
// ("QLoRA", llm-compass, 方法与公式, the displayed formula, with an adapter
// chosen per token; skillbyai, Merging the adapter for serving: one base
// serves several adapters as long as they are not merged into it).
//
// token_slots_kernel   ids from request lengths
// slots_us_kernel      us[m][j] = bf16(scale_a sum_k x[m][k] A_a[j][k])
//
// The second product is part of the base GEMM (gemm_slots_sm100.cuh).
#pragma once

#include "common.cuh"
#include "fewtok.cuh"

namespace qnf4 {

// ids[t] = slots[k] of the request k whose tokens [start_k, start_k + len_k)
// hold t, with start_k the sum of the lengths before it (a negative length
// counts as 0); -1 behind the last request.
//
// Bound by latency: 8 bytes per request and 4 per token.  One launch: every
// CTA owns 1024 consecutive tokens and walks the lengths in tiles of 1024,
// scanning each tile in shared memory (a warp scan per 32 lengths, then the
// warp totals); the tokens that fall into the tile find their request by
// bisection.  A CTA stops at the tile that passes its last token.
constexpr int kTsThreads = 256;
constexpr int kTsTile = 1024;        // lengths per scan, and tokens per CTA

__global__ void __launch_bounds__(kTsThreads) token_slots_kernel(const int32_t* __restrict__ lengths,
                                                                 const int32_t* __restrict__ slots,
                                                                 int64_t n_requests, int64_t n_tokens,
                                                                 int32_t* __restrict__ ids) {
  constexpr int kPer = kTsTile / kTsThreads;                         // 4 lengths and 4 tokens per thread
  __shared__ int64_t ends[kTsTile];                                  // end of each request of the tile
  __shared__ int64_t warp_sum[kTsThreads / 32];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * kTsTile;
  const int64_t tok_end = tok0 + kTsTile < n_tokens ? tok0 + kTsTile : n_tokens;
  int32_t found[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) found[i] = -1;
  int64_t base = 0;                                                  // tokens of the tiles before this one
  for (int64_t r0 = 0; r0 < n_requests && base < tok_end; r0 += kTsTile) {
    int64_t v[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t k = r0 + t * kPer + i;
      const int32_t len = k < n_requests ? __ldg(lengths + k) : 0;
      sum += len > 0 ? len : 0;
      v[i] = sum;                                                    // inclusive within the thread
    }
    int64_t incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
      if (lane >= off) incl += o;
    }
    __syncthreads();                                                 // the previous tile's ends are read
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int64_t before = base + incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kTsThreads / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) ends[t * kPer + i] = before + v[i];
    __syncthreads();
    const int64_t tile_end = base + total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t tok = tok0 + t + i * kTsThreads;
      if (tok < base || tok >= tile_end) continue;
      int lo = 0, hi = kTsTile - 1;                                  // first request whose end passes tok
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > tok) hi = mid;
        else lo = mid + 1;
      }
      found[i] = __ldg(slots + r0 + lo);
    }
    base = tile_end;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t tok = tok0 + t + i * kTsThreads;
    if (tok < n_tokens) ids[tok] = found[i];
  }
}

// ---------------------------------------------------------------------------
// The distinct adapters of a tile of tokens, in order of first appearance.
// Thread t holds token t's slot (-1: none); all threads of the CTA take part,
// kTok of them with a token (a multiple of 32).  A hash table (2 * kHash
// ints, kHash >= 2 kTok a power of two) keeps each slot's first token.
// list: the distinct slots; the return value is how many; `place` is the
// token's index into the list, -1 for none.  counts: kTok / 32 ints.
template <int kTok, int kHash>
__device__ __forceinline__ int distinct_slots(int32_t id, int32_t* hash, int32_t* list, int32_t* counts, int& place) {
  static_assert(kHash >= 2 * kTok && (kHash & (kHash - 1)) == 0, "half-empty power-of-two table");
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  int32_t* key = hash;
  int32_t* first = hash + kHash;
  for (int i = t; i < kHash; i += static_cast<int>(blockDim.x)) {
    key[i] = -1;
    first[i] = kTok;
  }
  __syncthreads();
  int at = -1;
  if (t < kTok && id >= 0) {
    at = static_cast<int>((static_cast<uint32_t>(id) * 2654435761u) >> 16) & (kHash - 1);
    while (true) {                                           // ends: half of the places stay free
      const int32_t was = atomicCAS(key + at, -1, id);
      if (was == -1 || was == id) break;
      at = (at + 1) & (kHash - 1);
    }
    atomicMin(first + at, t);
  }
  __syncthreads();
  const bool leader = at >= 0 && first[at] == t;
  const uint32_t lead = __ballot_sync(0xFFFFFFFFu, leader);
  if (warp < kTok / 32 && lane == 0) counts[warp] = __popc(lead);
  __syncthreads();
  int n = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kTok / 32; ++w) {
    const int c = counts[w];
    if (w < warp) before += c;
    n += c;
  }
  if (leader) {
    const int li = before + __popc(lead & ((1u << lane) - 1u));
    list[li] = id;
    key[at] = li;                                            // (nobody looks keys up any more)
  }
  __syncthreads();
  place = at < 0 ? -1 : key[at];
  return n;
}

// What the CTA-pair GEMM needs to know about each tile of 512 tokens: the
// distinct adapters, and each token's first rank column among theirs (far
// below 0 for none).  One CTA per tile, once per call: inside the GEMM every
// wave of tiles would build the list again (about 2.5 us each).
constexpr int kSlotsTile = 512;
struct SlotsTile {
  int32_t n;                             // adapters in the list
  int32_t pad[3];
  int32_t list[kSlotsTile];
  int32_t col[kSlotsTile];
};

__global__ void __launch_bounds__(kSlotsTile) slots_tiles_kernel(const int32_t* __restrict__ ids, int64_t M,
                                                                 int64_t n_adapters, int r8,
                                                                 SlotsTile* __restrict__ tiles) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int32_t hash[4 * kSlotsTile], list[kSlotsTile], counts[kSlotsTile / 32];
  const int64_t m = static_cast<int64_t>(blockIdx.x) * kSlotsTile + threadIdx.x;
  int32_t id = -1;
  if (m < M) {
    id = __ldg(ids + m);
    if (id < 0 || id >= n_adapters) id = -1;
  }
  int place;
  const int n = distinct_slots<kSlotsTile, 2 * kSlotsTile>(id, hash, list, counts, place);
  SlotsTile& t = tiles[blockIdx.x];
  t.col[threadIdx.x] = place < 0 ? -(1 << 29) : place * r8;
  if (static_cast<int>(threadIdx.x) < n) t.list[threadIdx.x] = list[threadIdx.x];
  if (threadIdx.x == 0) t.n = n;
}

// The products of an adapter row's infinite or NaN B values with a token's us.
__device__ __noinline__ float slots_odd_term(const uint16_t* B_row, const uint16_t* us, int r) {
  float f = 0.f;
  for (int j = 0; j < r; ++j) {
    const uint32_t b = __ldg(B_row + j);
    if ((b & 0x7F80u) == 0x7F80u)
      f = fmaf(__uint_as_float(static_cast<uint32_t>(us[j]) << 16), __uint_as_float(b << 16), f);
  }
  return f;
}

// us of at most 256 tokens.  One CTA per (token, 4 rank columns): its warps
// share the K axis (thread t takes the 8-column chunks t, t + 256, ...), then
// add up over a butterfly and shared memory in warp order.  Tokens of one
// adapter go in fours, in token order: the CTA of the first of four reads the
// adapter once for all of them, the other three leave (128 tokens of 64
// adapters, 28672 wide, rank 16: 31 us each for itself, 24 so; the adapters'
// and x's bytes out of L2 bound it; at three CTAs per SM its registers spill
// 140 bytes).  A token's sum is the same in any
// company.  us has rows of r8 = r
// rounded up to 8; its columns past r, and the rows of tokens without an
// adapter, are zero.  The CTAs also zero the tickets of the GEMM behind, and
// let it start beside them.
constexpr int kUsThreads = 256;
constexpr int kUsRanks = 4;
constexpr int kUsTokens = 4;

// acc[i][j] = thread's share of the products of token tok[i] with adapter row j
template <int kTok>
__device__ __forceinline__ void slots_us_part(const uint16_t* __restrict__ x, const uint16_t* __restrict__ Ar,
                                              const int* tok, int64_t K, int rows, float (&acc)[kUsTokens][kUsRanks]) {
  const int chunks = static_cast<int>(K / 8);
  const uint16_t* xr[kTok];
#pragma unroll
  for (int i = 0; i < kTok; ++i) xr[i] = x + tok[i] * K;
#pragma unroll 2
  for (int c = threadIdx.x; c < chunks; c += kUsThreads) {
    uint4 xv[kTok], av[kUsRanks];
#pragma unroll
    for (int i = 0; i < kTok; ++i) xv[i] = ld_nc_v4(xr[i] + c * 8);
#pragma unroll
    for (int j = 0; j < kUsRanks; ++j)
      av[j] = j < rows ? ld_nc_v4(Ar + j * K + c * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      const uint32_t xw[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
#pragma unroll
      for (int j = 0; j < kUsRanks; ++j) {
        const uint32_t aw[4] = {av[j].x, av[j].y, av[j].z, av[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[i][j] = fmaf(fewtok_bf16_lo(xw[e]), fewtok_bf16_lo(aw[e]), acc[i][j]);
          acc[i][j] = fmaf(fewtok_bf16_hi(xw[e]), fewtok_bf16_hi(aw[e]), acc[i][j]);
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kUsThreads, 3) slots_us_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ A, const float* __restrict__ scale,
    const int32_t* __restrict__ ids, int M, int64_t K, int64_t n_adapters, int r, int r8, uint16_t* __restrict__ us,
    uint32_t* __restrict__ tickets, int n_tickets) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float sums[kUsThreads / 32][kUsTokens][kUsRanks];
  __shared__ uint32_t same[kUsThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = blockIdx.x * kUsThreads + threadIdx.x; i < n_tickets; i += gridDim.x * kUsThreads) tickets[i] = 0u;
  const int per_tok = r8 / kUsRanks;
  const int m = static_cast<int>(blockIdx.x) / per_tok;
  const int j0 = static_cast<int>(blockIdx.x % per_tok) * kUsRanks;
  const int32_t a = __ldg(ids + m);
  const int t = static_cast<int>(threadIdx.x);
  const int32_t other = t < M ? __ldg(ids + t) : -1;         // thread t looks at token t
  if (a < 0 || a >= n_adapters) {
    if (t < kUsRanks) us[static_cast<int64_t>(m) * r8 + j0 + t] = 0;
    return;
  }
  const uint32_t hit = __ballot_sync(0xFFFFFFFFu, t < M && other == a);
  if (lane == 0) same[warp] = hit;
  __syncthreads();
  // the tokens of this adapter before this one, and this one with the next three
  int before = 0, n_tok = 0, tok[kUsTokens];
#pragma unroll
  for (int i = 0; i < kUsTokens; ++i) tok[i] = m;
#pragma unroll
  for (int w = 0; w < kUsThreads / 32; ++w) {
    uint32_t bits = same[w];
    const int base = 32 * w;
    if (base < m) before += __popc(m - base >= 32 ? bits : bits & ((1u << (m - base)) - 1u));
    if (base + 31 < m) continue;
    if (base < m) bits &= ~((1u << (m - base)) - 1u);
#pragma unroll
    for (int i = 0; i < kUsTokens; ++i)
      if (i == n_tok && bits != 0) {
        tok[i] = base + __ffs(static_cast<int>(bits)) - 1;
        bits &= bits - 1;
        ++n_tok;
      }
  }
  if (before % kUsTokens != 0) return;
  float acc[kUsTokens][kUsRanks] = {};
  const uint16_t* Ar = A + (static_cast<int64_t>(a) * r + j0) * K;
  if (n_tok == 1) slots_us_part<1>(x, Ar, tok, K, r - j0, acc);
  else if (n_tok == 2) slots_us_part<2>(x, Ar, tok, K, r - j0, acc);
  else slots_us_part<4>(x, Ar, tok, K, r - j0, acc);         // (of three the first stands in for a fourth)
#pragma unroll
  for (int i = 0; i < kUsTokens; ++i) {
    if (i >= n_tok) break;
#pragma unroll
    for (int j = 0; j < kUsRanks; ++j) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) acc[i][j] += __shfl_xor_sync(0xFFFFFFFFu, acc[i][j], off);
      if (lane == 0) sums[warp][i][j] = acc[i][j];
    }
  }
  __syncthreads();
  if (t < n_tok * kUsRanks) {
    const int i = t / kUsRanks, j = t % kUsRanks;
    float v = 0.f;
    if (j0 + j < r) {                                        // (a NaN in x times a zero of the padding is no result)
      for (int w = 0; w < kUsThreads / 32; ++w) v += sums[w][i][j];
      v *= __ldg(scale + a);
    }
    int at = tok[0];
#pragma unroll
    for (int k = 1; k < kUsTokens; ++k)
      if (i == k) at = tok[k];
    us[static_cast<int64_t>(at) * r8 + j0 + j] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
}

}  // namespace qnf4
