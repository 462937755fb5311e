// select_attn.hip -- attention of one new token over the pages that a list names for each
// (row, kv head): the kernels of paged_attn_kernel.hpp with such a list.
//
// Bound: HBM, the listed pages.  32 rows of 128 pages of 16 tokens, 32 + 8 heads of 128, bf16 (250 MB): 60 us, 4.2 TB/s, of which
// 5 join the pieces.  One row of 32 pages of 64, 16 + 2 heads of 128, 8 bits: 10.8, the chain of lists, pages, keys and two launches.
#include "paged_attn_kernel.hpp"

namespace ssm {

hipError_t launch_select_attn(const PagedAttnArgs &a, hipStream_t stream, const char **kernel_name) {
    return launch_form<true>(a, stream, kernel_name);
}

}  // namespace ssm
