// cfa_host_util.h -- what the paged entry points' host code shares: argument checks, the
// plan's device, launches, and the rotation's frequencies.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "cfa.h"

namespace cfa {

inline bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

struct Span {
    const void *at;
    size_t n;
};

// The plan's device is the current one for the length of a call.
class OnDevice {
  public:
    explicit OnDevice(int device) {
        if (cudaGetDevice(&was_) != cudaSuccess) was_ = -1;
        ok_ = was_ == device || cudaSetDevice(device) == cudaSuccess;
        if (was_ == device) was_ = -1;
        if (!ok_) cudaGetLastError();
    }
    ~OnDevice() {
        if (was_ >= 0) cudaSetDevice(was_);
    }
    bool ok() const { return ok_; }

  private:
    int was_ = -1;
    bool ok_ = false;
};

// Launches with programmatic stream serialization; cluster 1: no cluster.
inline cfa_status launch_kernel(const void *kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                void **args, int cluster = 1) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelExC(&cfg, kernel, args) != cudaSuccess) {
        cudaGetLastError();
        return CFA_ERR_CUDA;
    }
    return CFA_OK;
}

// Clears words of a plan. A memset may run after the call that asks for it has returned, and
// streams that do not wait for the legacy one would launch on what the words held before.
inline bool clear_words(unsigned *words, int n) {
    return cudaMemset(words, 0, sizeof(unsigned) * n) == cudaSuccess && cudaStreamSynchronize(nullptr) == cudaSuccess;
}

// Turns per position of each pair of rotary_dim dims as fractions of 2^64, or why not
// (cfa_paged_set_rope says what the arguments mean).
inline cfa_status rope_turns(double theta, int rotary_dim, int scaling, double factor, double low_turns,
                             double high_turns, int original_ctx, double magnitude, unsigned long long *turns) {
    if (!(theta >= 1.0) || !std::isfinite(theta) || !(factor >= 1.0) || !std::isfinite(factor) ||
        !(magnitude > 0.0) || !std::isfinite(magnitude) || magnitude > 1e6 ||
        scaling < CFA_ROPE_PLAIN || scaling > CFA_ROPE_BY_PARTS)
        return CFA_ERR_INVALID_ARG;
    if (scaling == CFA_ROPE_BY_PARTS &&
        (!(low_turns >= 0.0) || !(high_turns > low_turns) || !std::isfinite(high_turns) || original_ctx < 1))
        return CFA_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925287;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rotary_dim);
        if (scaling == CFA_ROPE_LINEAR) f /= factor;
        if (scaling == CFA_ROPE_BY_PARTS) {
            const double r = original_ctx * f / two_pi;
            const double g = std::min(1.0, std::max(0.0, (r - low_turns) / (high_turns - low_turns)));
            f = g * f + (1.0 - g) * f / factor;
        }
        // f <= 1, so below 1/6 of a turn: the product stays far below 2^64
        turns[i] = static_cast<unsigned long long>(std::ldexp(f / two_pi, 64));
    }
    return CFA_OK;
}

}  // namespace cfa
