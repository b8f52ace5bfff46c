// Clusters of the layer kernels: ranks, barriers and reads of the peers' shared memory.
#pragma once

#include "common.cuh"

namespace dt {

DT_DEVINL uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of every CTA; what was written to shared memory before is seen behind it.
DT_DEVINL void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `p` (shared memory of this CTA) in the shared memory of CTA `rank`.
DT_DEVINL uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
DT_DEVINL float4 peer_ld4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
DT_DEVINL float peer_ld(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
DT_DEVINL uint32_t peer_ld_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
DT_DEVINL uint64_t peer_ld_u64(uint32_t a) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

// What a warp whose wait gave up has to tell the cluster's other CTAs: a word of shared memory, 0 at first, that it sets before the
// cluster's barrier.  Behind it, in every lane of a warp, not 0 in one of them where any of the `ctas` has set its own.
DT_DEVINL uint32_t gave_up_beside(const uint32_t* word, int ctas) {
  const uint32_t lane = threadIdx.x & 31u;
  return ctas == 1 ? *const_cast<const volatile uint32_t*>(word) : lane < static_cast<uint32_t>(ctas) ? peer_ld_u32(peer_addr(word, lane)) : 0u;
}

// Whether a phase is complete, without waiting (try_wait may hold the thread for microseconds).
DT_DEVINL bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

}  // namespace dt
