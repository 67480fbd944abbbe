// attn_parts.hip -- the attention kernels for rows that see parts: first tokens and a window, or a tree of drafted tokens.
#include "attn_kernel.h"

namespace wq {

namespace {

template <int NB, int NW, int KS>
void launch_shared_as(const AttnArgs& a, dim3 grid, hipStream_t s) {
    if (a.q41) hipLaunchKernelGGL((k_attn_rows_shared<NB, true, NW, KS>), grid, dim3(NW * 64), 0, s, a);
    else hipLaunchKernelGGL((k_attn_rows_shared<NB, false, NW, KS>), grid, dim3(NW * 64), 0, s, a);
}

}  // namespace

void launch_parts_shared(const AttnArgs& a, dim3 grid, bool wide, hipStream_t s) {
    switch (a.dim) {
    case 64: wide ? launch_shared_as<2, 8, 2>(a, grid, s) : launch_shared_as<2, 4, 2>(a, grid, s); break;
    case 96: wide ? launch_shared_as<3, 8, 2>(a, grid, s) : launch_shared_as<3, 4, 1>(a, grid, s); break;
    case 128: wide ? launch_shared_as<4, 8, 2>(a, grid, s) : launch_shared_as<4, 4, 1>(a, grid, s); break;
    default: launch_shared_as<8, 4, 1>(a, grid, s); break;
    }
}

void launch_parts_token(const AttnArgs& a, dim3 grid, bool few, hipStream_t s) { launch_token<true>(a, grid, few, s); }
void launch_parts_rows(const AttnArgs& a, dim3 grid, bool wide, hipStream_t s) { launch_rows<true>(a, grid, wide, s); }

}  // namespace wq
