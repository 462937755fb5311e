// select_attn.hip -- attention of one new token over the pages that a list names for each
// (row, kv head): the kernels of paged_attn_kernel.hpp with such a list.
#include "paged_attn_kernel.hpp"

namespace ssm {

hipError_t launch_select_attn(const PagedAttnArgs &a, hipStream_t stream, const char **kernel_name) {
    return launch_form<true>(a, stream, kernel_name);
}

}  // namespace ssm
