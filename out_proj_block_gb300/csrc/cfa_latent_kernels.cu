// Instantiations of the paged latent-cache kernels.
#include "cfa_latent_attn.cuh"
#include "cfa_latent_cache.cuh"
#include "cfa_latent_expanded.cuh"
#include "cfa_latent_heads.cuh"
#include "cfa_latent_heads_mma.cuh"

namespace cfa {

const void *latent_append_kernel_ptr(bool interleaved) {
    return interleaved ? reinterpret_cast<const void *>(&latent_append_kernel<true>)
                       : reinterpret_cast<const void *>(&latent_append_kernel<false>);
}
const void *latent_heads_kernel_ptr(bool fold) {
    return fold ? reinterpret_cast<const void *>(&latent_fold_kernel) : reinterpret_cast<const void *>(&latent_unfold_kernel);
}
int latent_heads_smem(bool fold) { return fold ? 0 : UnfoldSmem::kBytes; }
const void *latent_heads_mma_kernel_ptr(bool fold) {
    return fold ? reinterpret_cast<const void *>(&latent_heads_mma_kernel<true>)
                : reinterpret_cast<const void *>(&latent_heads_mma_kernel<false>);
}
int latent_heads_mma_smem(bool fold) { return fold ? HeadsMma<true>::kBytes : HeadsMma<false>::kBytes; }
const void *latent_attention_kernel_ptr() { return reinterpret_cast<const void *>(&latent_attention_kernel); }
const void *latent_merge_kernel_ptr() { return reinterpret_cast<const void *>(&latent_merge_kernel); }
int latent_attention_smem() { return LatSmem::kBytes; }
const void *latent_expanded_kernel_ptr() { return reinterpret_cast<const void *>(&latent_expanded_kernel); }
const void *latent_expanded_merge_kernel_ptr() { return reinterpret_cast<const void *>(&latent_expanded_merge_kernel); }
int latent_expanded_smem() { return ExpSmem::kBytes; }

}  // namespace cfa
