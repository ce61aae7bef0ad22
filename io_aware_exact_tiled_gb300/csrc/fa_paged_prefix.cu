// Attention over the paged 8-bit cache for a batch whose requests share prefixes.
//
// Two passes of the kernels of fa_paged_split.cuh and fa_paged_tile.cu. In the
// first, a group of requests is one request whose new tokens are all of theirs
// and whose keys are the prefix, so that a prefix is read once for all rows that
// share it; it leaves each row's maximum and sum and its output, normalised, in
// fp32. The second is each request over its own tokens, and joins the two.
#include "fa_paged_split.cuh"

namespace fa {

cudaError_t launch_fwd_paged_prefix(const PagedArgs& prefix, const PagedArgs& own, cudaStream_t stream, int* nlaunch) {
    *nlaunch = 0;
    cudaError_t e = cudaSuccess;
    if (own.ev_begin) cudaEventRecord(own.ev_begin, stream);
    for (const PagedArgs* a : {&prefix, &own}) {
        if (e == cudaSuccess && a->split_rows > 0) {
            e = launch_split<true>(*a, stream);
            ++*nlaunch;
        }
        if (e == cudaSuccess && paged_has_tiles(a->max_new, a->Hq / a->Hkv, a->d)) {
            e = launch_paged_tile(*a, stream);
            ++*nlaunch;
        }
    }
    if (own.ev_end) cudaEventRecord(own.ev_end, stream);
    return e;
}

}  // namespace fa
