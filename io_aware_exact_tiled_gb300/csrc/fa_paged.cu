// Attention over the paged 8-bit cache: the split-key kernel, and the choice
// between it and the row-tile kernel.
#include "fa_paged_split.cuh"

namespace fa {

cudaError_t launch_fwd_paged(const PagedArgs& a, cudaStream_t stream, int* nlaunch) {
    if (a.ev_begin) cudaEventRecord(a.ev_begin, stream);
    cudaError_t e = launch_split<false>(a, stream);
    *nlaunch = 1;
    if (e == cudaSuccess && paged_has_tiles(a.max_new, a.Hq / a.Hkv, a.d)) {
        e = launch_paged_tile(a, stream);
        *nlaunch = 2;
    }
    if (a.ev_end) cudaEventRecord(a.ev_end, stream);
    return e;
}

}  // namespace fa
