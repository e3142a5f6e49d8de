// philox.cuh -- the keep mask of counter-based LoRA dropout.
//
// Philox4x32 (J. Salmon, M. Moraes, R. Dror and D. Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011) with 7 rounds, the fewest that the
// paper finds to pass its statistical tests.  The key is the 64-bit seed, the
// counter (column / 8, row, offset low, offset high); 16-bit half i of the
// four words (word i / 2, low half first) decides column 8 (column / 8) + i:
// it is dropped when the half is below T = rint(65536 p).  A value therefore
// depends on (seed, offset, row, column) alone, so that the forward and every
// kernel of the backward draw the same mask and none is stored.
//
// Cost per 8 values: 7 rounds of two 32 x 32 -> 64 multiplications and two
// 3-input xors, and two or three instructions per value to compare and pack.
#pragma once

#include "common.cuh"

namespace qnf4 {

struct DropoutRng {
  const uint64_t* state;    // {seed, offset}
  uint32_t threshold;       // T
};

struct PhiloxKey { uint32_t k0, k1, c2, c3; };

__device__ __forceinline__ PhiloxKey philox_key(const uint64_t* state) {
  const uint64_t seed = __ldg(reinterpret_cast<const unsigned long long*>(state));
  const uint64_t off = __ldg(reinterpret_cast<const unsigned long long*>(state) + 1);
  return PhiloxKey{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(off),
                   static_cast<uint32_t>(off >> 32)};
}

// The first product of a column group's rounds; the next group's is this one
// plus kPhiloxA.
constexpr uint64_t kPhiloxA = 0xD2511F53u;
__device__ __forceinline__ uint64_t philox_first(uint32_t group) { return kPhiloxA * group; }

// The four words for columns 8 group .. 8 group + 7 of a row, from
// philox_first(group): the low half of word i decides column 2 i, the high
// half column 2 i + 1.
__device__ __forceinline__ void philox_words(const PhiloxKey& key, uint32_t row, uint64_t first, uint32_t (&w)[4]) {
  uint32_t c0 = 0, c1 = row, c2 = key.c2, c3 = key.c3, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t a = i == 0 ? first : kPhiloxA * c0, b = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = c0; w[1] = c1; w[2] = c2; w[3] = c3;
}

// Those columns as bf16x2 masks of the dropped values (all ones in a dropped
// half): half - T is negative exactly when the half is dropped, and a prmt
// that replicates signs widens the two signs to halves.
__device__ __forceinline__ void philox_drop8(const PhiloxKey& key, uint32_t threshold, uint32_t row, uint64_t first,
                                             uint32_t (&drop)[4]) {
  uint32_t w[4];
  philox_words(key, row, first, w);
#pragma unroll
  for (int i = 0; i < 4; ++i) drop[i] = prmt((w[i] & 0xFFFFu) - threshold, (w[i] >> 16) - threshold, 0xFFBBu);
}

// The keep bits of columns 8 group .. 8 group + 7, shifted into `bits` from
// below (column 8 group + 7 first): for T > 0, 2^16 half + (2^32 - 2^16 T)
// carries exactly when half >= T, whatever lies below the half, and an add with
// carry takes that in: two instructions per value.
__device__ __forceinline__ uint32_t philox_shift8(const PhiloxKey& key, uint32_t threshold, uint32_t row,
                                                  uint64_t first, uint32_t bits) {
  uint32_t w[4];
  philox_words(key, row, first, w);
  const uint32_t lift = 0u - (threshold << 16);
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    asm("{\n\t.reg .u32 t;\n\t"
        "add.cc.u32 t, %1, %2;\n\t"
        "addc.u32 %0, %0, %0;\n\t"
        "add.cc.u32 t, %3, %2;\n\t"
        "addc.u32 %0, %0, %0;\n\t}"
        : "+&r"(bits) : "r"(w[i]), "r"(lift), "r"(w[i] << 16));    // (bits is written before the last input is read)
  }
  return threshold != 0 ? bits : 0xFFFFFFFFu;
}

// Keep bits of columns 8 group .. 8 group + 7 of a row, bit i for column i.
__device__ __forceinline__ uint32_t philox_keep8(const PhiloxKey& key, uint32_t threshold, uint32_t row,
                                                 uint32_t group) {
  return philox_shift8(key, threshold, row, philox_first(group), 0u) & 0xFFu;
}

// Keep bits of the 32 columns from 8-column group `group` on.
__device__ __forceinline__ uint32_t philox_keep32(const PhiloxKey& key, uint32_t threshold, uint32_t row,
                                                  uint32_t group) {
  const uint64_t first = philox_first(group);
  uint32_t bits = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) bits = philox_shift8(key, threshold, row, first + i * kPhiloxA, bits);
  return bits;
}

// The mask as bits, [M, n / 8] (the layout of the calls that take a mask):
// one 32-bit word per thread and step.  n % 32 == 0.  Bound by the 64-bit
// products, not by its M n / 8 bytes: of the 14 of a group, those that the four
// groups of a word share leave 11.5, and 8192 x 11008 values take 33.4 us,
// which is 14 of them per clock and SM (the add-with-carry packing took the
// rest out of the way: 35.4 us with two operations more per value).
__global__ void __launch_bounds__(256) keep_bits_kernel(DropoutRng rng, int64_t M, int64_t n, uint32_t* bits) {
  const PhiloxKey key = philox_key(rng.state);
  const int64_t words = n / 32, total = M * words;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * 256) {
    // (total below 2^32: a 32-bit division)
    const int64_t m = total <= 0xFFFFFFFFll ? static_cast<uint32_t>(e) / static_cast<uint32_t>(words) : e / words;
    bits[e] = philox_keep32(key, rng.threshold, static_cast<uint32_t>(m), static_cast<uint32_t>(4 * (e - m * words)));
  }
}

}  // namespace qnf4
