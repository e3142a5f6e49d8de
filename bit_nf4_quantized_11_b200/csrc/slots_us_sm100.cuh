// slots_us_sm100.cuh -- the rank-r product of the many-adapter layer on tcgen05:
//   us[m][j] = bf16(scale_a sum_k x[m][k] A_a[j][k]),   a = ids[m]
// ("QLoRA", llm-compass, 方法与公式: the B A x branch, per token).
//
// A tile of 128 tokens is multiplied by the rank rows of a group of its
// distinct adapters at once, at most floor(256 / r8) (r8 = r rounded up to 8;
// UMMA 128 x N x 16, N <= 256, fp32 accumulation in tensor memory), and every
// token keeps the r columns of its own adapter.  The other columns are wasted
// work that the tensor cores do not notice: the kernel is bound by reading x
// and the adapters once per such group.  K is split over the CTAs of a cluster
// (at most 8); each CTA leaves its partial tile in shared memory and the
// cluster adds them in rank order over distributed shared memory.
//
// blockIdx.x = token tile * groups + group: the host launches the largest
// number of groups a tile can have; a cluster whose group does not exist
// leaves at once.  Rows of tokens without an adapter are not written (nothing
// reads them).  Roles and bounded waits as in lora_sm100.cuh.
#pragma once

#include "common.cuh"
#include "slots.cuh"

namespace qnf4 {

constexpr int kUuThreads = 160;               // TMA warp, MMA warp; five warps in prologue and epilogue
constexpr int kUuRing = 4;
constexpr int kUuATile = 128 * 64 * 2;        // 16 KB of x

// The UMMA's N for a group of adapters.
__host__ __device__ constexpr int uu_cols(int adapters, int r8) { return (adapters * r8 + 15) / 16 * 16; }
__host__ __device__ constexpr int uu_pitch(int N) { return N * 4 + 16; }
__host__ __device__ constexpr int uu_smem_bytes(int N) {
  const int ring = kUuRing * (kUuATile + N * 128);
  const int part = 128 * uu_pitch(N);
  return (ring > part ? ring : part) + 2 * 128 * 4 + 64 + 256 + 1024;
}

struct SlotsUsArgs {
  const float* scale;
  const int32_t* ids;
  uint16_t* us;             // [M, r8]
  uint32_t* tickets;        // zeroed for the GEMM behind, or none
  int64_t n_adapters;
  int n_tickets;
  int M, K, r, r8;
  int per;                  // adapters per group
  int groups;               // groups per token tile in the grid
  int N, n_alloc;           // columns of a full group, TMEM columns
  int stages_per_split;
  uint64_t timeout_ns;
};

__global__ void __launch_bounds__(kUuThreads) slots_us_umma_kernel(const __grid_constant__ CUtensorMap tm_x,
                                                                   const __grid_constant__ CUtensorMap tm_a,
                                                                   const SlotsUsArgs args) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const int N = args.N;
  const int b_stage = N * 128;
  const int ring_bytes = kUuRing * (kUuATile + b_stage), part_bytes = 128 * uu_pitch(N);
  uint8_t* a_ring = smem;
  uint8_t* b_ring = smem + kUuRing * kUuATile;
  int32_t* list = reinterpret_cast<int32_t*>(smem + (ring_bytes > part_bytes ? ring_bytes : part_bytes));
  int32_t* tok_place = list + 128;
  int32_t* counts = tok_place + 128;                         // 16 ints
  uint64_t* full = reinterpret_cast<uint64_t*>(counts + 16);
  uint64_t* empty = full + kUuRing;
  uint64_t* acc_full = empty + kUuRing;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = static_cast<int>(blockIdx.x) / args.groups, group = static_cast<int>(blockIdx.x) % args.groups;
  const int m0 = tile * 128;
  const int ks = static_cast<int>(gridDim.y), split = static_cast<int>(blockIdx.y);
  const uint64_t tmo = args.timeout_ns;
  if (split == 0)
    for (int i = blockIdx.x * kUuThreads + threadIdx.x; i < args.n_tickets; i += gridDim.x * kUuThreads)
      args.tickets[i] = 0u;

  int32_t my_id = -1;
  if (threadIdx.x < 128 && m0 + static_cast<int>(threadIdx.x) < args.M) {
    my_id = __ldg(args.ids + m0 + threadIdx.x);
    if (my_id < 0 || my_id >= args.n_adapters) my_id = -1;
  }
  int place;
  const int n_list = distinct_slots<128, 256>(my_id, reinterpret_cast<int32_t*>(smem), list, counts, place);
  const int per = args.per;
  const int first = group * per;                             // the group's adapters in the list
  const int n_ad = min(per, n_list - first);
  // The kernel before (the tiles' adapter lists) may still run: what follows
  // this one relies on it too, so no CTA leaves before it is done.
  if (n_ad <= 0) {                                           // every CTA of the cluster alike
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  if (threadIdx.x < 128) tok_place[threadIdx.x] = place;
  const int cols = uu_cols(n_ad, args.r8);
  fence_proxy_async_smem();                                  // the hash table before the copies over it

  const int n_stages = (args.K + 63) / 64;
  const int st_begin = split * args.stages_per_split;
  const int n_iter = max(0, min(n_stages, st_begin + args.stages_per_split) - st_begin);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kUuRing; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    mbar_init(acc_full, 1);
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

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_x);
      tma_prefetch_desc(&tm_a);
      int issued = 0;
      for (int it = 0; it < n_iter; ++it) {
        const int s = it % kUuRing;
        wait(empty + s, ((it / kUuRing) & 1u) ^ 1u);
        if (*abort_flag) break;
        // (the columns past the adapters' rows, when cols is rounded up, keep
        // what the slot held: nothing reads them)
        mbar_arrive_expect_tx(full + s, static_cast<uint32_t>(kUuATile + n_ad * args.r8 * 128));
        const int k0 = (st_begin + it) * 64;
        tma_load_2d(smem_u32(a_ring + s * kUuATile), &tm_x, full + s, k0, m0);
        for (int i = 0; i < n_ad; ++i)                       // r8 rows from the adapter's first
          tma_load_2d(smem_u32(b_ring + s * b_stage) + i * args.r8 * 128, &tm_a, full + s, k0,
                      list[first + i] * args.r);
        ++issued;
      }
      for (int it = issued > kUuRing ? issued - kUuRing : 0; it < issued; ++it)
        mbar_wait_bounded(full + (it % kUuRing), (it / kUuRing) & 1u, tmo);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = umma_idesc_bf16(128, cols, false);
      for (int it = 0; it < n_iter; ++it) {
        const int s = it % kUuRing;
        wait(full + s, (it / kUuRing) & 1u);
        if (*abort_flag) break;
        tc_fence_after_sync();
        const uint32_t a_base = smem_u32(a_ring + s * kUuATile);
        const uint32_t b_base = smem_u32(b_ring + s * b_stage);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16_ss(tmem_base, umma_desc_sw128(a_base + kk * 32, 16, 1024),
                       umma_desc_sw128(b_base + kk * 32, 16, 1024), idesc, (it > 0 || kk > 0) ? 1u : 0u);
        umma_commit(empty + s);
      }
      umma_commit(acc_full);
      mbar_wait_bounded(acc_full, 0, tmo);
    }
  }

  __syncwarp();
  wait(acc_full, 0);
  tc_fence_after_sync();
  __syncthreads();                                           // every stage is read
  const int pitch = uu_pitch(N);
  for (int c0 = 0; warp < 4 && c0 < cols; c0 += 16) {
    uint32_t v[16];
    tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(warp * 32) << 16) + c0, v);
    tmem_ld_wait();
    const uint32_t dst = smem_u32(smem + (warp * 32 + lane) * pitch + c0 * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sts_v4(dst + 16 * i, n_iter ? v[4 * i] : 0u, n_iter ? v[4 * i + 1] : 0u, n_iter ? v[4 * i + 2] : 0u,
             n_iter ? v[4 * i + 3] : 0u);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (ks > 1) cluster_sync_all();                            // every CTA's partial is in place
  // this CTA's tokens split, split + ks, ...: the columns of their own adapter
  const int r4 = args.r8 / 4;
  const int n_tok = (128 - split + ks - 1) / ks;
  for (int e = threadIdx.x; e < n_tok * r4; e += kUuThreads) {
    const int t = split + (e / r4) * ks, c4 = (e % r4) * 4;
    const int p = tok_place[t] - first;
    if (p < 0 || p >= n_ad) continue;                        // another group's, or no adapter
    const uint32_t addr = smem_u32(smem + t * pitch + (p * args.r8 + c4) * 4);
    float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int rk = 0; rk < ks; ++rk) {
      float4 u;
      if (ks == 1) {
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(u.x), "=f"(u.y), "=f"(u.z), "=f"(u.w)
                     : "r"(addr) : "memory");
      } else {
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(u.x), "=f"(u.y), "=f"(u.z), "=f"(u.w) : "r"(mapa_shared(addr, rk)) : "memory");
      }
      d.x += u.x; d.y += u.y; d.z += u.z; d.w += u.w;
    }
    const float s = __ldg(args.scale + list[first + p]);
    // the columns past r came from the next adapter's rows
    const float f[4] = {c4 < args.r ? s * d.x : 0.f, c4 + 1 < args.r ? s * d.y : 0.f, c4 + 2 < args.r ? s * d.z : 0.f,
                        c4 + 3 < args.r ? s * d.w : 0.f};
    *reinterpret_cast<uint2*>(args.us + static_cast<int64_t>(m0 + t) * args.r8 + c4) =
        make_uint2(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]));
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (ks > 1) cluster_sync_all();                            // no CTA leaves while others read it
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, static_cast<uint32_t>(args.n_alloc));
  }
}

}  // namespace qnf4
