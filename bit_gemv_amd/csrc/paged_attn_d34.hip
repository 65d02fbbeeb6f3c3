// The paged attention for heads of 96 and 128 values (a file of its own so that the
// sizes compile side by side).
#include "paged_attn_kernel.h"

namespace rfp2 {

hipError_t launch_paged_attn_34(const AttnArgs& a, bool i8, int nb, int rows, int grid,
                                hipStream_t stream) {
  return nb == 3 ? launch_attn_nb<3>(a, i8, rows, grid, stream)
                 : launch_attn_nb<4>(a, i8, rows, grid, stream);
}

}  // namespace rfp2
