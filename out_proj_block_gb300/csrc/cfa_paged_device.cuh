// cfa_paged_device.cuh -- what the paged-cache kernels share on the device.
#pragma once

#include <cstdint>

namespace cfa {

// Two fp32 to packed bf16, rounded to nearest even, in one conversion.
__device__ __forceinline__ uint32_t pack2_bf16_cvt(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace cfa
