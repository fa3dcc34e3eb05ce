// Instantiations of the paged latent-cache kernels.
#include "cfa_latent_attn.cuh"
#include "cfa_latent_cache.cuh"
#include "cfa_latent_expanded.cuh"
#include "cfa_latent_heads.cuh"

namespace cfa {

const void *latent_append_kernel_ptr(bool interleaved) {
    return interleaved ? reinterpret_cast<const void *>(&latent_append_kernel<true>)
                       : reinterpret_cast<const void *>(&latent_append_kernel<false>);
}
const void *latent_fold_kernel_ptr() { return reinterpret_cast<const void *>(&latent_fold_kernel); }
const void *latent_unfold_kernel_ptr() { return reinterpret_cast<const void *>(&latent_unfold_kernel); }
const void *latent_attention_kernel_ptr() { return reinterpret_cast<const void *>(&latent_attention_kernel); }
const void *latent_merge_kernel_ptr() { return reinterpret_cast<const void *>(&latent_merge_kernel); }
int latent_attention_smem() { return LatSmem::kBytes; }
const void *latent_expanded_kernel_ptr() { return reinterpret_cast<const void *>(&latent_expanded_kernel); }
const void *latent_expanded_merge_kernel_ptr() { return reinterpret_cast<const void *>(&latent_expanded_merge_kernel); }
int latent_expanded_smem() { return ExpSmem::kBytes; }

}  // namespace cfa
