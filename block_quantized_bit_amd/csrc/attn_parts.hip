// attn_parts.hip -- the attention kernels for rows that see parts: first tokens and a window, or a tree of drafted tokens.
#include "attn_kernel.h"

namespace wq {

void launch_parts_token(const AttnArgs& a, dim3 grid, bool few, hipStream_t s) { launch_token<true>(a, grid, few, s); }
void launch_parts_rows(const AttnArgs& a, dim3 grid, bool wide, hipStream_t s) { launch_rows<true>(a, grid, wide, s); }

}  // namespace wq
