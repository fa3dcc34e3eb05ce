// cfa_tensor.cuh -- what the tensor-core attention kernels share: TMEM and mma.sync accesses, packed
// fp32 arithmetic, copies, and a bounded wait in few instructions.
#pragma once

#include <cstdint>

#include "cfa_device.cuh"

namespace cfa {

// D[tmem] (+)= A[tmem] . B[smem]: A's row r in lane r, two bf16 a column.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, bool accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
                 : "memory");
}

// 32 consecutive fp32 columns of this warp's 32 lanes; valid after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
                   "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
                   "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                   "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
                   "=r"(r[31])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                    "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
                    "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2^x by the hardware's base-2 exponential (relative error about 2^-22), results below
// 2^-126 flushed to 0: one instruction, where the form that keeps them takes four.
__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// All bits of those of two bf16 that are infinite or NaN: an exponent of ones and the 1 added to
// it carry into the sign's place.
__device__ __forceinline__ uint32_t odd_bf16x2(uint32_t v) {
    return ((((v & 0x7f807f80u) + 0x00800080u) >> 15) & 0x00010001u) * 0xffffu;
}
// The larger magnitudes of two pairs of bf16, NaN where there is one (signs mean nothing); and of 16 bytes.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}
__device__ __forceinline__ uint32_t max_abs_bf16x8(uint32_t m, uint4 v) {
    return max_abs_bf16x2(max_abs_bf16x2(m, max_abs_bf16x2(v.x, v.y)), max_abs_bf16x2(v.z, v.w));
}

// Two fp32 lanes in one instruction.
__device__ __forceinline__ uint64_t pair_f32(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair_f32(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// True in one lane of the warp, the same one every time. A warp whose lanes all run an
// issue loop keeps its operands in uniform registers; a loop inside "if (lane == 0)" moves
// them there for every instruction (measured: 100 clocks a product, 250 a copy).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(~0u, v, 0); }

// Lanes hold rows, an even lane's and the next one's behind one another in memory, and w 32 bytes of each: two lanes write
// 32 bytes of a row together, then the other's. A lane's own 16, in 32 rows at once, take a transaction each.
// `out` is the even row's 32 bytes, at this lane's half of them; `next` elements on are the odd row's. By a whole warp.
__device__ __forceinline__ void write_rows_in_pairs(uint16_t *out, size_t next, const uint32_t *w, bool even_live, bool odd_live) {
    const bool odd = threadIdx.x & 1;
    uint32_t other[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) other[c] = __shfl_xor_sync(~0u, odd ? w[c] : w[4 + c], 1);
    if (even_live)
        *reinterpret_cast<uint4 *>(out) = odd ? make_uint4(other[0], other[1], other[2], other[3]) : make_uint4(w[0], w[1], w[2], w[3]);
    if (odd_live)
        *reinterpret_cast<uint4 *>(out + next) = odd ? make_uint4(w[4], w[5], w[6], w[7]) : make_uint4(other[0], other[1], other[2], other[3]);
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
// Arrives on the barrier when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void prefetch_tensor_map(const void *tmap) {
    asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(tmap)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(n) : "memory");
}

// The library's bounded wait in few instructions: the kernel's many waits would otherwise
// crowd its loops out of the instruction cache, and a call in their place keeps the
// compiler from giving the warpgroups different registers.
__device__ __forceinline__ uint32_t timer_lo_ns() {
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}
template <typename Done>
__device__ __forceinline__ bool bounded_wait(Done done, uint32_t timeout_ns, volatile int *timed_out, unsigned *status,
                                           unsigned site) {
    if (done()) return true;
    const uint32_t t0 = timer_lo_ns();
    CFA_ROLLED while (!done()) {
        if (*timed_out) return false;
        if (timer_lo_ns() - t0 > timeout_ns) {
            *timed_out = 1;
            atomicOr(status, kStatusTimeoutBit | (site << kStatusSiteShift));
            return false;
        }
    }
    return true;
}

}  // namespace cfa
