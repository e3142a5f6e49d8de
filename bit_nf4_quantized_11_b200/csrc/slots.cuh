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

// One warp per (token, 8 rank columns): lane l takes the 8-column chunks
// l, l + 32, ... of the token's row.  us has rows of r8 = r rounded up to 8;
// its columns past r, and the rows of tokens without an adapter, are zero.
__global__ void __launch_bounds__(256) slots_us_kernel(const uint16_t* __restrict__ x,
                                                       const uint16_t* __restrict__ A,
                                                       const float* __restrict__ scale,
                                                       const int32_t* __restrict__ ids, int64_t M, int64_t K,
                                                       int64_t n_adapters, int r, int r8, uint16_t* __restrict__ us) {
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t m = item / (r8 / 8);
  const int j0 = static_cast<int>(item % (r8 / 8)) * 8;
  if (m >= M) return;
  const int32_t a = __ldg(ids + m);
  float acc[8] = {};
  float s = 0.f;
  if (a >= 0 && a < n_adapters) {
    s = __ldg(scale + a);
    for (int64_t c = lane; c < K / 8; c += 32) {
      const uint4 xv = ld_nc_v4(x + m * K + c * 8);
      const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j0 + j >= r) break;
        const uint4 av = ld_nc_v4(A + (static_cast<int64_t>(a) * r + j0 + j) * K + c * 8);
        const uint32_t aw[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[j] = fmaf(fewtok_bf16_lo(xw[e]), fewtok_bf16_lo(aw[e]), acc[j]);
          acc[j] = fmaf(fewtok_bf16_hi(xw[e]), fewtok_bf16_hi(aw[e]), acc[j]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], off);
    if (lane == j) us[m * r8 + j0 + j] = __bfloat16_as_ushort(__float2bfloat16_rn(s * acc[j]));
  }
}

}  // namespace qnf4
