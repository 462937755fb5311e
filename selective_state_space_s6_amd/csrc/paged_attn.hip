// paged_attn.hip -- attention of one new token over all of its cached tokens: the kernels of
// paged_attn_kernel.hpp without a list of pages.
#include "paged_attn_kernel.hpp"

namespace ssm {

// (of the smallest unit, a tile of one wave)
double paged_attn_max_units(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t max_pages, int64_t page_size) {
    const double len = (double)max_pages * (double)page_size;
    return (double)batch * (double)n_kv_heads * (double)passes_of(n_heads / n_kv_heads) * (len / 16 + 1.0);
}

size_t paged_attn_workspace_bytes(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                                  int64_t max_pages, int64_t page_size) {
    const int64_t group = n_heads / n_kv_heads, gmax = std::min<int64_t>(group, kHeads);
    const int64_t places = 2 * most_blocks(batch, n_heads, n_kv_heads, headdim, max_pages, page_size) * gmax;
    return (size_t)(align16((batch + 1) * 4) + align16(places * 8) + places * headdim * 4);
}

hipError_t launch_paged_attn(const PagedAttnArgs &a, hipStream_t stream, const char **kernel_name) {
    return launch_form<false>(a, stream, kernel_name);
}

}  // namespace ssm
