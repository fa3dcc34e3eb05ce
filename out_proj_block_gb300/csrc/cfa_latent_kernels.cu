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
// Kernels of blocks of tm tokens: 16, 64 or 128.
const void *latent_fold_kernel_ptr(int tm) {
    return tm == 16   ? reinterpret_cast<const void *>(&latent_fold_kernel<16>)
           : tm == 64 ? reinterpret_cast<const void *>(&latent_fold_kernel<64>)
                      : reinterpret_cast<const void *>(&latent_fold_kernel<128>);
}
int latent_fold_smem(int tm) { return (kHeadsCols + tm) * 256; }
const void *latent_unfold_kernel_ptr(int tm) {
    return tm == 16   ? reinterpret_cast<const void *>(&latent_unfold_few_kernel)
           : tm == 64 ? reinterpret_cast<const void *>(&latent_unfold_kernel<64>)
                      : reinterpret_cast<const void *>(&latent_unfold_kernel<128>);
}
int latent_unfold_smem(int tm) {
    return tm == 16 ? UnfoldFewSmem::kBytes : tm == 64 ? UnfoldSmem<64>::kBytes : UnfoldSmem<128>::kBytes;
}
const void *latent_attention_kernel_ptr() { return reinterpret_cast<const void *>(&latent_attention_kernel); }
const void *latent_merge_kernel_ptr() { return reinterpret_cast<const void *>(&latent_merge_kernel); }
int latent_attention_smem() { return LatSmem::kBytes; }
const void *latent_expanded_kernel_ptr() { return reinterpret_cast<const void *>(&latent_expanded_kernel); }
const void *latent_expanded_merge_kernel_ptr() { return reinterpret_cast<const void *>(&latent_expanded_merge_kernel); }
int latent_expanded_smem() { return ExpSmem::kBytes; }

}  // namespace cfa
