// cfa_tensor_pair.cuh -- tcgen05 instructions that span the two blocks of a cluster (cta_group::2).
#pragma once

#include <cstdint>

#include "cfa_device.cuh"

namespace cfa {

// Arrive on the barrier at this offset in both blocks once all earlier products have ended.
__device__ __forceinline__ void umma2_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
}
// D[tmem] (+)= A[smem] . B[smem] of both blocks, issued by one thread of the first.
__device__ __forceinline__ void umma2_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           bool accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
                 : "memory");
}
// Arrives on a barrier of either block (an address from map_to_rank). What it tells of are writes of the
// asynchronous proxy, or ones that a proxy fence has put in front of it, to the arriving
// block's own shared memory, which that block's own tensor core reads. The form that releases at cluster scope
// takes 1100 clocks each time: 16,000 for a block of keys that should take 3000. By the letter of the memory model
// this one, which releases at block scope, does not order those writes for the other block's issuing thread: that a
// product that it issues behind its wait reads them is an assumption about the hardware.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t remote_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(remote_bar) : "memory");
}
// By one warp of each block.
__device__ __forceinline__ void tmem2_alloc(uint32_t slot_smem_addr, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(slot_smem_addr), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem2_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(taddr), "r"(ncols) : "memory");
}
// The same with A in TMEM: either block's rows in its own lanes, two bf16 a column.
__device__ __forceinline__ void umma2_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              bool accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
                 : "memory");
}

}  // namespace cfa
