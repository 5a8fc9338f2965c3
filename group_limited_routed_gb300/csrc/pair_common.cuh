// Pieces shared by the CTA-pair products of the training operators
// (pair_product_kernel.cuh, ortho_chain.cu): tile constants, loads and
// descriptors of both operand orders, accumulator loads, staged stores.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "gemm_common.cuh"
#include "ptx.cuh"

namespace beam {
namespace {

using gemm::Waiter;

constexpr int kPBK = 64;                       // k elements per block (128 bytes)
constexpr uint32_t kPABytes = 128 * 128;       // one CTA's A per stage
constexpr int kPEpiWarps = 16;
constexpr int kPThreads = 96 + 32 * kPEpiWarps;
constexpr uint32_t kPRing = 216 * 1024;
constexpr uint64_t kPPeerDrainNs = 1000000ull; // see the producers' teardown
constexpr uint32_t kAtom = 64 * 128;           // MN-major atom: 64 k rows of 64 elements

// Results that leave through shared memory: a warp stages 2 KB (16 rows of 32
// FP32 columns, or 32 rows of 16-bit ones) and one bulk copy writes them.
constexpr uint32_t kStaging = kPEpiWarps * 2048;

// True on one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// 32 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// 3-D tiled load into this CTA's shared memory, bytes counted on a barrier of
// either CTA of the pair.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* m,
                                                 uint32_t cluster_bar, int32_t x, int32_t y,
                                                 int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(cluster_bar), "l"(policy)
      : "memory");
}

// Shared-memory descriptor of an MN-major operand as a 128-byte-swizzled TMA
// load of a 64 x 64 box leaves it: each k row is 128 bytes of 64 consecutive
// elements; 8 k rows make a 1024-byte group (stride byte offset); the next 64
// elements of the operand's own axis are one box further (leading byte offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kAtom >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// Arrive on either CTA's barrier without a release.  It frees TMEM columns
// whose loads have completed (tcgen05.wait::ld): no memory is handed over,
// and a release would wait for the warp's earlier global stores.
__device__ __forceinline__ void arrive_relaxed_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}
// Arrive on either CTA's barrier, releasing the warp's writes to its own
// shared memory (ordered before by __syncwarp) and nothing else: a release of
// everything would wait for the CTA's global stores in flight, 1500 to 3400
// cycles.
__device__ __forceinline__ void arrive_release_smem_cluster(uint32_t cluster_bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  arrive_relaxed_cluster(cluster_bar);
}
// Waiter::wait for a barrier whose arrivals release at cluster scope.
__device__ __forceinline__ bool wait_cluster(const Waiter& w, uint32_t bar, uint32_t parity) {
  auto done = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
  };
  if (done()) return true;
  const uint64_t t0 = ptx::globaltimer();
  for (uint32_t n = 1;; ++n) {
    if (done()) return true;
    if ((n & 63u) == 0) {
      if (*w.abort_flag) return false;
      if (ptx::globaltimer() - t0 > w.limit_ns) {
        *w.abort_flag = 1;
        latch_status(w.status, kStatusTimeout);
        return false;
      }
    }
  }
}
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[16]) { ptx::tmem_ld16(at, r); }
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[32]) { tmem_ld32(at, r); }

// Two values rounded to the 16-bit output type, the first in the low half.
__device__ __forceinline__ uint32_t pack_out(float lo, float hi, bool f16) {
  if (f16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Bulk copy of a warp's staged rows, shared -> global; ADD: += in FP32.
template <bool ADD>
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, uint32_t src, int32_t x,
                                             int32_t y, int32_t z) {
  if constexpr (ADD)
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group "
        "[%0, {%1, %2, %3}], [%4];" ::"l"(reinterpret_cast<uint64_t>(m)),
        "r"(x), "r"(y), "r"(z), "r"(src)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::
            "l"(reinterpret_cast<uint64_t>(m)),
        "r"(x), "r"(y), "r"(z), "r"(src)
        : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Every staged row of this thread's copies has been read / written.
__device__ __forceinline__ void tma_store_read_done() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void tma_store_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Two 16-bit values of one lane's column (rows j, j + 1) and its neighbour's
// -> the word this lane stores: even lanes row j, odd lanes row j + 1, two
// columns each.
__device__ __forceinline__ uint32_t swap_pair(uint32_t mine, int lane) {
  const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
  return (lane & 1) ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
}

}  // namespace
}  // namespace beam
