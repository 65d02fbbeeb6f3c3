// The paged attention for heads of 160 and 192 values (a file of its own so that the
// sizes compile side by side).
#include "paged_attn_kernel.h"

namespace rfp2 {

hipError_t launch_paged_attn_56(const AttnArgs& a, bool i8, int nb, int rows, int grid,
                                hipStream_t stream) {
  return nb == 5 ? launch_attn_nb<5>(a, i8, rows, grid, stream)
                 : launch_attn_nb<6>(a, i8, rows, grid, stream);
}

}  // namespace rfp2
