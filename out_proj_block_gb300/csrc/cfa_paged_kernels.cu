// Instantiations of the paged-cache kernels.
#include "cfa_paged_attn.cuh"
#include "cfa_paged_cache.cuh"

namespace cfa {

const void *paged_tables_kernel_ptr() { return reinterpret_cast<const void *>(&paged_tables_kernel); }
const void *paged_append_kernel_ptr(bool interleaved) {
    return interleaved ? reinterpret_cast<const void *>(&paged_append_kernel<true>)
                       : reinterpret_cast<const void *>(&paged_append_kernel<false>);
}
const void *paged_attention_kernel_ptr(int d) {
    return d == 128 ? reinterpret_cast<const void *>(&paged_attention_kernel<128>)
                    : reinterpret_cast<const void *>(&paged_attention_kernel<64>);
}
const void *paged_merge_kernel_ptr(int d) {
    return d == 128 ? reinterpret_cast<const void *>(&paged_merge_kernel<128>)
                    : reinterpret_cast<const void *>(&paged_merge_kernel<64>);
}
int paged_attention_smem(int d, int seqs) {
    return d == 128 ? PagedSmem<128>::bytes(seqs) : PagedSmem<64>::bytes(seqs);
}

}  // namespace cfa
